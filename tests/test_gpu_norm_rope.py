"""GPU parity of the q/k norm with rotation and cache write against the fp64
oracle, for pools of 16-bit values, E4M3 codes and 4-bit records, and a run of
the whole chain: norm and rotation into a 4-bit cache, then decode.

Tolerance of a turned value: half a step of its type, and for fp32 arithmetic
2^-20 of the two values it is made of: the mean (8 products and their sums, a
tree of 4 more), the root and the two products with weights round about 16
times, each by 2^-24 of the value."""
import numpy as np
import pytest
import torch

from oracle import int4
from paged_kv_cache_64_gb300 import api, workloads

from _parity import bits
from test_gpu_decode_int4 import HALF, Case, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_errors():
    assert torch.cuda.is_available()
    yield
    api.check_error()


def table(positions, rot, base=10000.0):
    rate = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(positions)[:, None] * rate
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Inputs:
    def __init__(self, T, hq, hkv, d, block, dtype, rot, seed=0, positions=500, skip=()):
        rng = np.random.default_rng(seed)
        self.dtype, self.block, self.d, self.hkv = dtype, block, d, hkv
        self.qkv = int4.narrow(rng.standard_normal((T, (hq + 2 * hkv) * d)) *
                               rng.choice([0.02, 1.0, 30.0], (T, 1)), dtype)
        cut = [0, hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
        self.q, self.k, self.v = (self.qkv[:, a:b].reshape(T, -1, d) for a, b in zip(cut, cut[1:]))
        g = to_gpu(self.qkv, dtype)
        self.gq, self.gk, self.gv = (g[:, a:b].view(T, -1, d) for a, b in zip(cut, cut[1:]))
        self.qw, self.kw = (int4.narrow(1 + 0.2 * rng.standard_normal(d), dtype) for _ in range(2))
        self.gqw, self.gkw = to_gpu(self.qw, dtype), to_gpu(self.kw, dtype)
        self.eps = 1e-5
        self.cs = table(positions, rot)
        self.gcs = torch.as_tensor(self.cs, device="cuda")
        self.pos = rng.integers(0, positions, T)
        self.nb = -(-T // block) + 2
        self.slots = rng.permutation(self.nb * block)[:T].astype(np.int64)
        self.slots[list(skip)] = -1
        self.gpos, self.gslots = (torch.as_tensor(x, device="cuda") for x in (self.pos, self.slots))

    def pools(self, fmt):
        shape = (self.nb, self.hkv, self.block, self.d)
        if fmt == "int4":
            return [torch.full(api.int4_pool_shape(self.nb, self.hkv, self.block, self.d), 0x33,
                               dtype=torch.uint8, device="cuda") for _ in range(2)]
        dt = torch.uint8 if fmt == "e4m3" else workloads.torch_dtype(self.dtype)
        return [torch.full(shape, 3, dtype=dt, device="cuda") for _ in range(2)]

    def run(self, pools, interleaved, q_out=None, **kw):
        out = torch.full(self.gq.shape, float("nan"), dtype=self.gq.dtype, device="cuda") \
            if q_out is None else q_out
        api.qk_norm_rope(out, self.gq, self.gk, self.gv, self.gqw, self.gkw, self.eps, self.gcs,
                         self.gpos, self.gslots, *pools, interleaved=interleaved, **kw)
        return out

    def check(self, got, x, w, interleaved):
        ref = int4.norm_rope(x, w, self.eps, self.cs, self.pos, interleaved, self.dtype)
        half = self.cs.shape[1] // 2
        one = np.ones_like(self.cs)
        one[:, half:] = -1  # |a| + |b| of a pair, by a turn of (1, -1) of absolute values
        y = np.abs(int4.norm_rope(x, w, self.eps, np.concatenate([one[:, :half], 0 * one[:, half:]], 1),
                                  self.pos, interleaved, self.dtype))
        pair = y.copy()
        if interleaved:
            pair[..., 0:2 * half:2] += y[..., 1:2 * half:2]
            pair[..., 1:2 * half:2] += y[..., 0:2 * half:2]
        else:
            pair[..., :half] += y[..., half:2 * half]
            pair[..., half:2 * half] += y[..., :half]
        tol = HALF[self.dtype] * (1 + 2.0**-8) * np.abs(ref) + 2.0**-20 * pair + 2.0**-25
        g = int4.widen(bits(got), self.dtype)
        bad = ~(np.abs(g - ref) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), g[bad][:4], ref[bad][:4])


def gathered(pool, slots, block):
    s = torch.as_tensor(slots, device="cuda")
    return pool[s // block, :, s % block]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112),
                                   (128, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_16bit_pools(dtype, d, rot, interleaved):
    x = Inputs(21, 6, 2, d, 16, dtype, rot, seed=rot, skip=(4, 20))
    pools = x.pools("16")
    before = [p.clone() for p in pools]
    q = x.run(pools, interleaved)
    x.check(q, x.q, x.qw, interleaved)
    keep = x.slots >= 0
    x16 = gathered(pools[0], np.maximum(x.slots, 0), 16)
    x16[4] = x16[20] = x16[0]  # skipped tokens: looked at below
    kept = x.k.copy()
    kept[4] = kept[20] = kept[0]
    pos = x.pos.copy()
    x.pos[[4, 20]] = x.pos[0]
    x.check(x16, kept, x.kw, interleaved)
    x.pos = pos
    assert torch.equal(gathered(pools[1], x.slots[keep], 16).view(torch.int16),
                       x.gv[torch.as_tensor(keep, device="cuda")].view(torch.int16))
    # every other slot as it was
    for p, b in zip(pools, before):
        s = torch.as_tensor(x.slots[keep], device="cuda")
        b[s // 16, :, s % 16] = p[s // 16, :, s % 16]
        assert torch.equal(p, b)


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 32)])
@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (37, 21, 3), (600, 8, 1)])
def test_coded_pools_hold_what_the_writes_would_write(fmt, dtype, d, block, T, hq, hkv):
    """The cache gets the 16-bit keys' and values' codes, byte for byte those
    of cache_write_fp8 / cache_write_int4."""
    x = Inputs(T, hq, hkv, d, block, dtype, d, seed=T, skip=(5,) if T > 5 else ())
    wide, pools, want = x.pools("16"), x.pools(fmt), x.pools(fmt)
    q16 = x.run(wide, False)
    kw = dict(k_scale=0.037, v_scale=0.9) if fmt == "e4m3" else {}
    q = x.run(pools, False, **kw)
    assert torch.equal(q, q16)
    k16 = gathered(wide[0], np.maximum(x.slots, 0), block).contiguous()
    v = x.gv.contiguous()
    if fmt == "e4m3":
        api.cache_write_fp8(k16, v, x.gslots, *want, 0.037, 0.9)
    else:
        api.cache_write_int4(k16, v, x.gslots, *want)
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])


@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (2, 7, 7), (3, 14, 2), (300, 64, 8), (2500, 5, 5)])
def test_counts_and_head_layouts(T, hq, hkv):
    x = Inputs(T, hq, hkv, 128, 16, "bf16", 128, seed=hq)
    pools = x.pools("16")
    q = x.run(pools, False)
    x.check(q, x.q, x.qw, False)
    x.check(gathered(pools[0], x.slots, 16), x.k, x.kw, False)
    assert torch.equal(gathered(pools[1], x.slots, 16), x.gv)


def test_in_place_and_other_strides():
    x = Inputs(33, 6, 2, 64, 16, "bf16", 64)
    want = x.run(x.pools("16"), True)
    wide = torch.zeros(33, 1000, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 8:8 + 6 * 64].view(33, 6, 64)
    x.run(x.pools("16"), True, q_out=out)
    assert torch.equal(out, want)
    assert not wide[:, :8].any() and not wide[:, 8 + 384:].any()
    x.run(x.pools("16"), True, q_out=x.gq)  # a column range of the projection, in place
    assert torch.equal(x.gq, want)


def test_bad_positions_and_slots_are_recorded_and_skipped():
    x = Inputs(8, 4, 2, 64, 16, "f16", 64)
    pools = x.pools("int4")
    want = x.run(pools, False)
    x.gpos[1], x.gpos[5] = -1, 500
    x.gslots[3] = x.nb * 16
    fresh = x.pools("int4")
    out = x.run(fresh, False)
    with pytest.raises(Exception, match="PA_ERR_BAD_INDEX"):
        api.check_error()
    api.check_error()
    assert torch.isnan(out[[1, 5]]).all()
    rest = [0, 2, 3, 4, 6, 7]
    assert torch.equal(out[rest], want[rest])
    got, exp = ([torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
                for _ in range(2))
    s = torch.as_tensor(x.slots, device="cuda")
    api.cache_read_int4(*got, s, *fresh)
    api.cache_read_int4(*exp, s, *pools)
    ok = [0, 2, 4, 6, 7]
    assert torch.equal(got[0][ok], exp[0][ok]) and torch.equal(got[1][ok], exp[1][ok])
    untouched = torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda"), \
        torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda")
    api.cache_read_int4(*untouched, s, *x.pools("int4"))
    assert torch.equal(got[0][[1, 3, 5]], untouched[0][[1, 3, 5]])


@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 16), ("f16", 64, 32)])
def test_a_serving_run(dtype, d, block):
    """Prompt, then steps: norm, rotation and write into a 4-bit cache, decode
    over it; every step's output against the oracle's decode over the oracle's
    own quantisation of the keys (16-bit, from a 16-bit cache beside it)."""
    hq, hkv, steps = 6, 2, 5
    prompts = [40, 7, 129]
    S = len(prompts)
    alloc = api.BlockAllocator(64, block)
    for i in range(S):
        alloc.add(i)
    tdt = workloads.torch_dtype(dtype)
    shape = (64, hkv, block, d)
    wide = [torch.zeros(shape, dtype=tdt, device="cuda") for _ in range(2)]
    four = [torch.zeros(api.int4_pool_shape(64, hkv, block, d), dtype=torch.uint8, device="cuda")
            for _ in range(2)]
    host = [p.cpu().numpy() for p in four]
    ws = None
    for step in range(steps):
        counts = prompts if step == 0 else [1] * S
        start = [0 if step == 0 else alloc.length(i) for i in range(S)]
        slots = np.concatenate([alloc.append(i, n)[0] for i, n in enumerate(counts)]).astype(np.int64)
        x = Inputs(len(slots), hq, hkv, d, block, dtype, d, seed=step)
        x.gslots = torch.as_tensor(slots, device="cuda")
        x.gpos = torch.as_tensor(np.concatenate([np.arange(s, s + n) for s, n in zip(start, counts)]),
                                 device="cuda")
        q = x.run(wide, False)
        assert torch.equal(q, x.run(four, False))
        s = torch.as_tensor(slots, device="cuda")
        k16 = wide[0][s // block, :, s % block]
        int4.cache_write(host, [bits(k16), x.v], slots, block, dtype)
        tables, lens = alloc.export(list(range(S)), 16)
        last = torch.as_tensor(np.cumsum(counts) - 1, device="cuda")
        c = Case.__new__(Case)
        c.d, c.block, c.dtype, c.scale = d, block, dtype, d ** -0.5
        c.tables, c.lens, (c.kp, c.vp) = tables, lens, host
        c.gq = q[last].contiguous()
        c.q = bits(c.gq)
        out = torch.empty_like(c.gq)
        ws = api.decode_int4(out, c.gq, *four, torch.as_tensor(tables, device="cuda").contiguous(),
                             torch.as_tensor(lens, device="cuda"), int(lens.max()), c.scale,
                             partition_tokens=32, workspace=ws)
        c.check(out, step)
    for g, h in zip(four, host):
        assert np.array_equal(g.cpu().numpy(), h)
