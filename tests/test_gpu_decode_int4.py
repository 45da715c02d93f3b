"""GPU parity of decode attention over 4-bit pools against the fp64 oracle.

Tolerance, per sequence and head: half a step of the output type, plus what
fp32 arithmetic can move.  A score is a sum whose running value stays below
A = max_p sum_i |q_i k_i| * scale * log2 e; its dozen roundings (products in
the matrix unit, partial sums, scale) move it by under 2^-19 A, so a weight by
under 2^-19 A ln 2 relative and the normalised sum by twice that, times the
largest |v|: 2^-17 A |v| leaves a factor of about 4.  exp2's and the sums' own
roundings add 2^-18 |v| and, one for each few positions, L 2^-28 |v|."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import int4
from paged_kv_cache_64_gb300 import _lib, api, workloads

from _parity import bits

pytestmark = pytest.mark.gpu

HALF = {"f16": 2.0**-11, "bf16": 2.0**-8}


@pytest.fixture(autouse=True)
def clean_errors():
    assert torch.cuda.is_available()
    yield
    api.check_error()


def to_gpu(b, dtype):
    t = torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).to("cuda")
    return t.view(workloads.torch_dtype(dtype))


class Case:
    """Sequences of the given lengths whose blocks lie anywhere in pools of
    quantised normal rows; every slot no sequence reaches holds NaN rows."""

    def __init__(self, lens, hkv, group, d, block, dtype, seed=0, k_rows=None, v_rows=None, q=None,
                 max_len=None):
        rng = np.random.default_rng(seed)
        self.d, self.block, self.dtype = d, block, dtype
        self.lens = np.asarray(lens, np.int32)
        S = len(lens)
        count = -(-self.lens // block)
        most = max(1, int(count.max(initial=0)))
        nb = int(count.sum()) + 3
        order = rng.permutation(nb)
        self.tables = np.full((S, most), 1 << 30, np.int32)  # unused entries are never looked at
        slots, at = [], 0
        for i in range(S):
            t = order[at:at + count[i]]
            at += count[i]
            self.tables[i, :count[i]] = t
            p = np.arange(self.lens[i])
            slots.append(t[p // block].astype(np.int64) * block + p % block if len(t) else
                         np.zeros(0, np.int64))
        slots = np.concatenate(slots) if S else np.zeros(0, np.int64)
        T = len(slots)
        shape = api.int4_pool_shape(nb, hkv, block, d)
        self.kp, self.vp = np.full(shape, 0xFF, np.uint8), np.full(shape, 0xFF, np.uint8)
        k = rng.standard_normal((T, hkv, d)) if k_rows is None else k_rows(rng, (T, hkv, d))
        v = rng.standard_normal((T, hkv, d)) if v_rows is None else v_rows(rng, (T, hkv, d))
        qv = rng.standard_normal((S, hkv * group, d)) if q is None else q(rng, (S, hkv * group, d))
        self.q = int4.narrow(qv, dtype)
        self.scale = d ** -0.5
        tdt = workloads.torch_dtype(dtype)
        self.gk, self.gv = (torch.from_numpy(x).to("cuda") for x in (self.kp, self.vp))
        if T:  # the write is bit-exact against the oracle (its own tests)
            api.cache_write_int4(torch.tensor(k, device="cuda").to(tdt),
                                 torch.tensor(v, device="cuda").to(tdt),
                                 torch.as_tensor(slots, device="cuda"), self.gk, self.gv)
        self.kp, self.vp = self.gk.cpu().numpy(), self.gv.cpu().numpy()
        self.gq = to_gpu(self.q, dtype)
        self.gt = torch.as_tensor(self.tables, device="cuda")
        self.gl = torch.as_tensor(self.lens, device="cuda")
        self.max_len = int(self.lens.max(initial=0)) if max_len is None else max_len

    def gpu(self, partition=0, workspace=None, stream=None):
        out = torch.full_like(self.gq, float("nan"))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        api.decode_int4(out, self.gq, self.gk, self.gv, self.gt, self.gl, self.max_len, self.scale,
                        partition_tokens=partition, workspace=workspace, stream=stream)
        return out

    def oracle(self):
        return int4.decode(self.q, self.kp, self.vp, self.tables, self.lens, self.scale, self.block,
                           self.dtype)

    def allowed(self, ref):
        kv, vv = (int4.values(p, self.d, self.block, self.dtype) for p in (self.kp, self.vp))
        q = np.abs(int4.widen(self.q, self.dtype))
        S, hq, d = q.shape
        hkv = kv.shape[1]
        tol = HALF[self.dtype] * (1 + 2.0**-8) * np.abs(ref) + 2.0**-25
        for i, L in enumerate(self.lens.tolist()):
            if not L:
                continue
            t = self.tables[i, :-(-L // self.block)]
            for h in range(hkv):
                k = np.abs(kv[t, h].reshape(-1, d)[:L])
                v = np.abs(vv[t, h].reshape(-1, d)[:L]).max()
                mine = slice(h * hq // hkv, (h + 1) * hq // hkv)
                A = (q[i, mine] @ k.T).max(-1, keepdims=True) * self.scale * 1.4427
                tol[i, mine] += v * (A * 2.0**-17 + 2.0**-18 + L * 2.0**-28)
        return tol

    def check(self, out, what=""):
        ref = self.oracle()
        assert np.isfinite(ref).all()
        o = int4.widen(bits(out), self.dtype)
        bad = ~(np.abs(o - ref) <= self.allowed(ref))
        assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), o[bad][:4],
                               ref[bad][:4], self.allowed(ref)[bad][:4])


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 64, 100, 0, 511, 513, 700]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("partition", [0, -1, 32, 256])
def test_edge_lengths(dtype, d, block, partition):
    c = Case(EDGES, 2, 3, d, block, dtype, seed=d + block)
    out = c.gpu(partition)
    c.check(out)
    assert not out[torch.as_tensor(c.lens == 0, device="cuda")].any()


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 128), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_every_group(dtype, d, group):
    c = Case([40, 1, 333], 2, group, d, 16, dtype, seed=group)
    c.check(c.gpu(0))
    c.check(c.gpu(64))


@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_long_and_many_partitions(hkv):
    c = Case([5000, 3, 2049], hkv, 4, 128, 16, "bf16", seed=hkv)
    for partition in (0, -1, 512, 2048, 96):  # 96: more partials than one launch combines
        c.check(c.gpu(partition), partition)


def test_a_maximum_length_past_the_lengths():
    c = Case([40, 0, 90], 2, 2, 128, 16, "f16", max_len=96)
    c.check(c.gpu(0))
    c.check(c.gpu(16))


def test_no_sequences_and_no_tokens():
    c = Case([0, 0], 2, 2, 64, 16, "f16")
    assert not c.gpu(0).any()
    e = Case([], 2, 2, 64, 16, "f16")
    assert e.gpu(0).shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_scales(dtype, d):
    """Scales of V from 2^-20 to 2^8 within a sequence, rows of equal values
    (s = 0), offsets far over the range, and the last rows the largest, so the
    running scale has to move."""
    def rows(rng, shape):
        x = rng.standard_normal(shape) * 2.0 ** rng.integers(-20, 5, (*shape[:2], 1))
        x += rng.choice([0.0, 0.0, 30.0], (*shape[:2], 1))
        x[::7] = rng.standard_normal((len(x[::7]), shape[1], 1))
        x[-60:] *= 2.0 ** np.linspace(0, 8, len(x[-60:]))[:, None, None]
        return x
    c = Case([333, 1, 64], 2, 5, d, 16, dtype, v_rows=rows)
    c.check(c.gpu(-1))
    c.check(c.gpu(64))
    small = Case([200], 1, 8, d, 16, "bf16", v_rows=lambda r, s: r.standard_normal(s) * 1e-9)
    ref = small.oracle()
    o = int4.widen(bits(small.gpu(0)), "bf16")
    assert (np.abs(o - ref) <= 2.0**-8 * 1.01 * np.abs(ref) + 2.0**-16 * 5e-9).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_and_keys_of_many_magnitudes(dtype, d):
    def q(rng, shape):
        x = rng.standard_normal(shape) * 2.0 ** rng.integers(-20, 1, shape)
        x[:, 0] *= 2.0**-14
        x[:, 1] = rng.standard_normal(shape[2]) * 50.0
        x[:, 2] = 0.0
        return x

    def k(rng, shape):
        return rng.standard_normal(shape) * 2.0 ** rng.integers(-6, 2, (1, shape[1], shape[2]))
    c = Case([200, 17], 2, 4, d, 16, dtype, q=q, k_rows=k)
    c.check(c.gpu(0))
    # scores that rise along the sequence: the running maximum moves in every tile
    up = Case([400], 1, 8, d, 16, dtype, q=lambda r, s: np.ones(s),
              k_rows=lambda r, s: r.standard_normal(s) * 0.1 + np.linspace(0, 12, s[0])[:, None, None])
    up.check(up.gpu(-1))
    up.check(up.gpu(32))


def test_nan_rows_reach_only_their_own_heads():
    def rows(rng, shape):
        x = rng.standard_normal(shape)
        x[50, 1, 3] = np.nan  # sequence 1 (positions 40 ..), KV head 1
        return x
    for where in ("k_rows", "v_rows"):
        c = Case([40, 30, 20], 2, 2, 64, 16, "bf16", **{where: rows})
        out = c.gpu(0).float()
        assert torch.isnan(out[1, 2:]).all()
        out[1, 2:] = 0
        assert torch.isfinite(out).all()


def test_sequences_of_nan_rows_alone():
    def rows(rng, shape):
        return np.full(shape, np.nan)
    for where in ("k_rows", "v_rows"):
        c = Case([1, 0, 70], 1, 3, 64, 16, "bf16", **{where: rows})
        for partition in (-1, 16, 0):
            out = c.gpu(partition).float()
            assert torch.isnan(out[[0, 2]]).all() and not out[1].any()


def test_workspace_of_garbage_is_scratch():
    c = Case([700, 90, 1500], 2, 4, 128, 16, "bf16")
    for partition in (256, 96):
        need = api.int4_workspace_size(3, 8, 2, 128, 16, c.max_len, partition, c.gq.dtype)
        assert need > 0
        for fill in (0, 0xFF, 0x5A):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            a = c.gpu(partition, workspace=ws)
            b = c.gpu(partition, workspace=ws)
            c.check(a)
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_a_missing_small_or_crooked_workspace_is_refused():
    """Host checks, before any launch."""
    c = Case([700], 2, 4, 128, 16, "bf16")
    need = api.int4_workspace_size(1, 8, 2, 128, 16, c.max_len, 128, c.gq.dtype)
    buf = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    vp = lambda t: ctypes.c_void_p(t.data_ptr())
    out = torch.empty_like(c.gq)
    for ws, size in ((ctypes.c_void_p(0), need), (vp(buf), need - 1), (vp(buf[16:]), need)):
        rc = _lib.load().pa_decode_int4(
            vp(out), vp(c.gq), vp(c.gk), vp(c.gv), c.gk.shape[0], vp(c.gt), c.gt.shape[1], vp(c.gl),
            c.max_len, 1, 8, 2, 128, 16, ctypes.c_float(c.scale), 128, ws, size, _lib.PA_BF16,
            ctypes.c_void_p(0))
        assert rc == 1  # PA_ERR_INVALID


@pytest.mark.parametrize("cut", [256, 0])
def test_two_graphs_share_a_workspace_and_replay(cut):
    a = Case([700, 90, 1500], 2, 4, 128, 16, "bf16", seed=1)
    b = Case([1900, 33], 3, 8, 64, 32, "f16", seed=2)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    a.gpu(0, workspace=ws), b.gpu(0, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, partition in ((a, cut), (b, cut)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.gpu(partition, workspace=ws))
        graphs.append(g)
    for _ in range(4):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        a.check(outs[0])
        b.check(outs[1])


@pytest.mark.parametrize("cut", [256, 0])
def test_two_streams_with_workspaces_of_their_own(cut):
    a = Case([700, 90, 1500], 2, 4, 128, 16, "bf16", seed=1)
    b = Case([1900, 33], 2, 4, 128, 16, "bf16", seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            x = a.gpu(cut)
        with torch.cuda.stream(s2):
            y = b.gpu(cut)
        outs.append((x, y))
    torch.cuda.synchronize()
    for x, y in outs:
        a.check(x)
        b.check(y)


def test_bad_lengths_and_entries_are_recorded():
    """Lengths past the maximum are cut to it, negative ones count as none,
    and entries outside the pool are never followed; each is reported."""
    c = Case([40, 50], 1, 2, 64, 16, "f16")
    good = c.gpu(0)
    c.gl = torch.tensor([40, -3], dtype=torch.int32, device="cuda")
    out = c.gpu(0)
    with pytest.raises(Exception, match="PA_ERR_BAD_INDEX"):
        api.check_error()
    assert torch.equal(out[0], good[0]) and not out[1].any()
    c.gl = torch.tensor([40, 1 << 20], dtype=torch.int32, device="cuda")
    out = c.gpu(0)  # cut to max_len = 50
    with pytest.raises(Exception, match="PA_ERR_BAD_INDEX"):
        api.check_error()
    assert torch.equal(out, good)
    c.gl = torch.as_tensor(c.lens, device="cuda")
    for bad in (-1, c.kp.shape[0], 1 << 29):
        c.gt = torch.as_tensor(c.tables, device="cuda").clone()
        c.gt[1, 1] = bad
        out = c.gpu(0)
        with pytest.raises(Exception, match="PA_ERR_BAD_INDEX"):
            api.check_error()
        assert torch.equal(out[0], good[0])


def test_offsets_past_32_bits():
    """Pools over 4 GiB with the sequence in their last blocks."""
    hkv, d, block, dtype = 8, 128, 16, "bf16"
    nb = (1 << 32) // (hkv * 1088) + 40
    kp = torch.empty(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
    vp = torch.empty_like(kp)
    L, small = 300, 19
    at = torch.arange(nb - small, nb, device="cuda").flip(0)
    p = torch.arange(L, device="cuda")
    slots = at[p // block] * block + p % block
    k = torch.randn(L, hkv, d, device="cuda").to(torch.bfloat16)
    v = torch.randn(L, hkv, d, device="cuda").to(torch.bfloat16)
    api.cache_write_int4(k, v, slots, kp, vp)
    sk = torch.empty(api.int4_pool_shape(small, hkv, block, d), dtype=torch.uint8, device="cuda")
    sv = torch.empty_like(sk)
    api.cache_write_int4(k, v, p, sk, sv)
    a, b = torch.empty_like(k), torch.empty_like(k)
    e, f = torch.empty_like(k), torch.empty_like(k)
    api.cache_read_int4(a, b, slots, kp, vp)
    api.cache_read_int4(e, f, p, sk, sv)
    assert torch.equal(a, e) and torch.equal(b, f)
    q = torch.randn(1, hkv * 4, d, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    x, y = torch.empty_like(q), torch.empty_like(q)
    api.decode_int4(x, q, kp, vp, at[None].to(torch.int32).contiguous(), lens, L, d ** -0.5)
    api.decode_int4(y, q, sk, sv, torch.arange(small, device="cuda", dtype=torch.int32)[None], lens,
                    L, d ** -0.5)
    assert torch.equal(x, y)


@pytest.mark.parametrize("hkv,group,block", [(5, 2, 16), (11, 1, 32), (16, 3, 16), (2, 8, 32)])
def test_head_counts_of_every_bundle(hkv, group, block):
    """Lengths that the automatic choice cuts, for head counts whose bundles
    are 5, 1, 8 and 2; sequences without tokens between them."""
    c = Case([0, 4000, 1, 2100, 0, 1300, 130, 0], hkv, group, 64, block, "f16", seed=hkv)
    c.check(c.gpu(0))


@pytest.mark.parametrize("lens", [[1025], [3000] * 3, [0, 0, 9000], [1100] * 40, [20000, 3, 3, 3]])
def test_automatic_choice_against_single_pass(lens):
    c = Case(lens, 2, 4, 128, 16, "f16", seed=len(lens))
    c.check(c.gpu(0))
    c.check(c.gpu(-1))


def test_a_long_batch_with_a_second_wave():
    """Fifty sequences of 12,000 to 16,384 positions: shares of over 64 units, so
    two waves of CTAs; single pass gives the same sums in another order, and two
    sequences go through the oracle."""
    rng = np.random.default_rng(0)
    S, hkv, group, d, block = 50, 8, 2, 64, 16
    lens = rng.integers(12000, 16385, S)
    lens[7] = 0
    count = -(-lens // block)
    nb = int(count.sum())
    order = rng.permutation(nb)
    tables = np.zeros((S, count.max()), np.int32)
    used = np.arange(count.max())[None] < count[:, None]
    tables[used] = order
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kp, vp = (torch.empty(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
              for _ in range(2))
    slots = torch.arange(nb * block, device="cuda")
    for p in (kp, vp):
        x = torch.randn(nb * block, hkv, d, generator=g, device="cuda").to(torch.float16)
        api.cache_write_int4(x, x, slots, p, p.clone())
    q = torch.randn(S, hkv * group, d, generator=g, device="cuda").to(torch.float16)
    gt, gl = torch.as_tensor(tables, device="cuda"), torch.as_tensor(lens, device="cuda").int()
    out, one = torch.empty_like(q), torch.empty_like(q)
    ws = api.decode_int4(out, q, kp, vp, gt, gl, int(lens.max()), d ** -0.5)
    api.decode_int4(one, q, kp, vp, gt, gl, int(lens.max()), d ** -0.5, partition_tokens=-1)
    api.check_error()
    assert not out[7].any()
    for _ in range(3):  # the same bits every time, whatever the order of the CTAs
        again = torch.empty_like(q)
        api.decode_int4(again, q, kp, vp, gt, gl, int(lens.max()), d ** -0.5, workspace=ws)
        assert torch.equal(again, out)
    a, b = out.double(), one.double()
    # both within half a step and fp32's share of the true value (see above)
    assert ((a - b).abs() <= 2.0**-10 * 1.01 * b.abs() + 2.0**-14).all()
    for i in (0, 33):
        at = tables[i, :count[i]]
        small = Case.__new__(Case)
        small.d, small.block, small.dtype, small.scale = d, block, "f16", d ** -0.5
        small.kp, small.vp = (p[torch.as_tensor(at, device="cuda").long()].cpu().numpy()
                              for p in (kp, vp))
        small.tables = np.arange(len(at), dtype=np.int32)[None]
        small.lens, small.q = lens[i:i + 1], bits(q[i:i + 1])
        small.check(out[i:i + 1], i)


def test_a_given_stream_without_a_workspace():
    c = Case([4000, 70], 2, 4, 128, 16, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [c.gpu(0, stream=side) for _ in range(3)]
    side.synchronize()
    for o in outs:
        c.check(o)


@pytest.mark.parametrize("hkv,group", [(2, 4), (1, 8)])
def test_small_outputs_of_a_long_sequence_keep_their_digits(hkv, group):
    """Over 120,000 positions the weights average V to about 1/200 of its size,
    while the sums of codes that the kernel forms are of V's whole range.  What
    fp32 loses of them has to stay below f16's rounding of the result: in the
    2-norm, half a step (2^-11)."""
    c = Case([120000], hkv, group, 128, 16, "f16", seed=hkv)
    out = int4.widen(bits(c.gpu(0)), "f16")
    ref = c.oracle()
    assert np.linalg.norm(out - ref) <= 2.0**-11 * np.linalg.norm(ref)
    one = int4.widen(bits(c.gpu(-1)), "f16")  # 940 steps of a warp in one sum
    assert np.linalg.norm(one - ref) <= 2.0**-11 * np.linalg.norm(ref)


@pytest.mark.parametrize("d,block", [(64, 16), (128, 32)])
def test_more_sequences_than_a_compact_grid(d, block):
    """Over 128 sequences a CTA stands for every chunk of the longest; chunks
    that begin at a sequence's end must not touch its output."""
    lens = [0, 64, 128, 192, 1, 63, 65, 127, 129, 191] * 14
    c = Case(lens, 2, 3, d, block, "f16", seed=d)
    for partition in (64, 128, -1, 0):
        c.check(c.gpu(partition), partition)


def test_more_sequences_than_balanced_ranges_take():
    lens = [3, 0, 17, 1, 40] * 210
    lens[7], lens[1000], lens[1049] = 2048, 1500, 1024
    c = Case(lens, 1, 4, 64, 16, "bf16")
    c.check(c.gpu(0))
    c.check(c.gpu(512))


def test_a_captured_call_follows_the_lengths():
    """The lengths are read on the device: a graph captured once serves them as
    they grow and shrink under the maximum it was captured with."""
    c = Case([3000, 2900, 1500, 10], 2, 4, 64, 16, "f16", seed=3)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    c.gpu(0, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.gpu(0, workspace=ws)
    for lens in ([3000, 2900, 1500, 10], [1, 2900, 0, 10], [0, 0, 0, 0], [2999, 17, 1500, 1]):
        c.lens = np.asarray(lens, np.int32)
        c.gl.copy_(torch.as_tensor(c.lens))
        g.replay()
        c.check(out, lens)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0, 1e-6])
def test_scales_of_every_kind(scale):
    c = Case([700, 2000, 3], 2, 4, 64, 16, "f16", seed=4)
    c.scale = scale
    ref = c.oracle()
    c.scale = abs(scale)  # the bound on a score goes by its size
    tol = c.allowed(ref)
    c.scale = scale
    for partition in (0, -1):
        assert (np.abs(int4.widen(bits(c.gpu(partition)), "f16") - ref) <= tol).all()
