"""Inputs, tolerances and checks shared by the tests of the latent cache."""
import numpy as np
import torch

from oracle import int4, latent

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step relative to the value
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
LEAST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the subnormals


def bits16(rng, *shape, dtype, size=1.0):
    return int4.narrow(rng.standard_normal(shape) * size, dtype)


def dev(b, dtype):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(TORCH[dtype])


def back(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def table(positions, factor=1.0):
    angle = np.arange(positions)[:, None] * 1000.0 ** (-np.arange(0, 64, 2) / 64)
    return (factor * np.concatenate([np.cos(angle), np.sin(angle)], 1)).astype(np.float32)


def check(got, ref, bound, what=""):
    g = int4.widen(back(got), "f16" if got.dtype == torch.float16 else "bf16")
    assert g.shape == ref.shape, (g.shape, ref.shape)
    bad = ~(abs(g - ref) <= bound)
    if bad.any():
        at = np.argwhere(bad)[:4].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first {at}: "
                             f"{g[bad][:4]} for {ref[bad][:4]}, bound {np.broadcast_to(bound, g.shape)[bad][:4]}")


def attention_bound(ref, size, terms, dtype, positions, width, largest):
    """How far an output may be off its fp64 value.  u is half a step of dtype.
    - the output's own rounding: u |ref|, or half a step of the subnormals;
    - the weights' rounding to dtype: u sum w |v| (their sum is not rounded);
    - a score's error e changes every weight by a factor within exp(+-2 e) of one
      another: 2 e (sum w |v| + |ref|).  e: products of 16-bit values are exact in
      fp32; a sum of `width` of them, in whatever order and cut rather than
      rounded, is off by width 2^-23 of the absolute terms; its scaling and the
      distance from the running maximum, two fp32 roundings of a score (2^-22 of
      its terms);
    - 2^x, fp32 sums of the products with V and of the weights over `positions`
      (256 partial sums of at most 64 terms each in sequence, rescaled): 2^-14;
    - f16 weights below the least normal: positions 2^-32 of the largest |v|."""
    u = UNIT[dtype]
    e = terms[..., None] * (width * 2.0 ** -23 + 2.0 ** -22)
    bound = u * abs(ref) + LEAST[dtype] + (u + 2.0 ** -14) * size + 2 * e * (size + abs(ref))
    if dtype == "f16":
        bound = bound + positions * 2.0 ** -32 * largest
    return bound


class Decode:
    """A batch over a latent pool whose stale slots and unused blocks hold NaN and infinities."""

    def __init__(self, rng, dtype, lens, heads, rank=512, block=16, size=1.0, poison=True, spare=3):
        lens = np.asarray(lens, np.int32)
        self.dtype, self.lens, self.heads, self.rank, self.block = dtype, lens, heads, rank, block
        count = -(-lens // block)
        total = int(count.sum()) + spare
        self.tables = np.full((len(lens), max(1, int(count.max(initial=0)))), 0, np.int32)
        order = rng.permutation(total)
        self.pool = np.full((total, block, rank + 64), 0x7E00 if dtype == "f16" else 0x7FC0, np.uint16)
        if poison:
            self.pool[:, 1::2] = 0xFC00 if dtype == "f16" else 0xFF80
        else:
            self.pool[:] = 0
        at = 0
        for i, L in enumerate(lens):
            mine = order[at:at + count[i]]
            at += count[i]
            self.tables[i, :count[i]] = mine
            rows = bits16(rng, count[i] * block, rank + 64, dtype=dtype)
            for j, b in enumerate(mine):
                n = min(block, L - j * block)
                self.pool[b, :n] = rows[j * block:j * block + n]
        self.q = bits16(rng, len(lens), heads, rank + 64, dtype=dtype, size=size)
        self.scale = 192 ** -0.5
        self.max_len = int(lens.max(initial=0))

    def reference(self):
        ref, size, terms = latent.decode(self.q, self.pool, self.tables, self.lens, self.scale, self.dtype)
        live = int4.widen(self.pool, self.dtype)
        largest = abs(live[np.isfinite(live)]).max(initial=0.0)
        return ref, attention_bound(ref, size, terms, self.dtype, self.max_len, self.rank + 64, largest)

    def gpu(self):
        self.g = dict(q=dev(self.q, self.dtype), pool=dev(self.pool, self.dtype),
                      block_tables=torch.as_tensor(self.tables).cuda(),
                      seq_lens=torch.as_tensor(self.lens).cuda(), max_seq_len=self.max_len,
                      scale=self.scale)
        return self.g

    def empty(self):
        return torch.full((len(self.lens), self.heads, self.rank), float("nan"), dtype=TORCH[self.dtype],
                          device="cuda")


class Prefill:
    """Ragged prompts; tokens before, between and behind the sequences hold NaN."""

    def __init__(self, rng, dtype, n_q, n_k, heads, causal, size=1.0, gap=3):
        self.dtype, self.heads, self.causal = dtype, heads, causal
        self.n_q, self.n_k = np.asarray(n_q), np.asarray(n_k)
        self.q_starts = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
        self.k_starts = (np.concatenate([[0], np.cumsum(n_k)]) + gap).astype(np.int32)
        self.q_starts += gap
        tq, tk = int(self.q_starts[-1]) + gap, int(self.k_starts[-1]) + gap
        self.q = bits16(rng, tq, heads, 192, dtype=dtype, size=size)
        self.kv = bits16(rng, tk, heads, 256, dtype=dtype)
        self.rows = bits16(rng, tk, 320, dtype=dtype)
        nan = 0x7E00 if dtype == "f16" else 0x7FC0
        for a, first, last in ((self.q, self.q_starts[0], self.q_starts[-1]),
                               (self.kv, self.k_starts[0], self.k_starts[-1]),
                               (self.rows, self.k_starts[0], self.k_starts[-1])):
            a[:first] = nan
            a[last:] = nan
        self.scale = 192 ** -0.5

    def reference(self):
        ref, size, terms = latent.prefill(self.q, self.kv[..., :128], self.kv[..., 128:],
                                          self.rows[:, 256:], self.q_starts, self.k_starts, self.scale,
                                          self.causal, self.dtype)
        v = int4.widen(self.kv[..., 128:], self.dtype)
        largest = abs(v[np.isfinite(v)]).max(initial=0.0)
        return ref, attention_bound(ref, size, terms, self.dtype, int(self.n_k.max(initial=0)), 192, largest)

    def gpu(self):
        kv, rows = dev(self.kv, self.dtype), dev(self.rows, self.dtype)
        return dict(q=dev(self.q, self.dtype), k=kv[..., :128], v=kv[..., 128:], k_pe=rows[:, 256:],
                    q_starts=torch.as_tensor(self.q_starts).cuda(),
                    k_starts=torch.as_tensor(self.k_starts).cuda(),
                    max_q_len=int(self.n_q.max(initial=0)), scale=self.scale, causal=self.causal)

    def empty(self):
        return torch.full((len(self.q), self.heads, 128), 7.0, dtype=TORCH[self.dtype], device="cuda")

    def check(self, out, what=""):
        ref, bound = self.reference()
        a, b = int(self.q_starts[0]), int(self.q_starts[-1])
        check(out[a:b], ref[a:b], bound[a:b], what)
        assert (out[:a] == 7.0).all() and (out[b:] == 7.0).all(), "rows of no sequence were written"
