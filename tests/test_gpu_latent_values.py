"""Latent attention and its rows at unusual values: scales far below the scores' sizes;
infinities and NaN in rows."""
import numpy as np
import pytest
import torch

from _latent import LEAST, TORCH, UNIT, Decode, Prefill, bits16, check, dev, table
from oracle import int4, latent
from paged_kv_cache_64_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,scale", [(1e30, 5e-32), (1e30, -5e-32), (1e35, 4e-37), (1e36, 0.0),
                                        (1e36, -0.0), (1e36, 1e-41)])
def test_small_scales_of_large_scores(size, scale):
    """Products of bf16 values as large as fp32 holds: how small the scale is says nothing
    about the scores.  (Scores stay at a few units, or at 0 beside the bound's 2^-14; the
    last scale is no normal number, off by half a step of 2^-149 or 7e-46: 1e-7 of a score.)"""
    rng = np.random.default_rng(31)
    case = Decode(rng, "bf16", [1, 63, 64, 200, 0, 700], 9, 256, 16, size=size)
    case.scale = scale
    out = case.empty()
    api.decode_latent(out, **case.gpu())
    api.check_error()
    ref, bound = case.reference()
    check(out, ref, bound)
    case = Prefill(rng, "bf16", [130, 3, 20], [130, 0, 300], 3, True, size=size)
    case.scale = scale
    out = case.empty()
    api.prefill_latent(out, **case.gpu())
    api.check_error()
    case.check(out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rank", [256, 512])
def test_rows_with_infinities(dtype, interleaved, rank):
    """An infinity or a NaN of a rotary part stays in its pair, one of the latent part in
    that part: 0 beside an infinity, NaN beside a NaN."""
    rng = np.random.default_rng(32)
    tokens, heads, nan = 6, 3, float("nan")
    q = bits16(rng, tokens, heads, 64, dtype=dtype)
    x = bits16(rng, tokens, rank + 64, dtype=dtype)
    weight, cs = bits16(rng, rank, dtype=dtype), table(50)
    pos = np.array([1, 7, 20, 33, 48, 5])

    def put(a, value):
        a[...] = int4.narrow(np.float64(value), dtype)

    put(x[1, rank + 3:rank + 4], np.inf)
    put(x[2, rank + 10:rank + 11], nan)
    put(x[3, 5:6], -np.inf)
    put(x[4, rank - 1:rank], nan)
    put(q[1, 0, 40:41], -np.inf)
    put(q[2, 2, 63:64], nan)
    pool = torch.zeros(2, 16, rank + 64, dtype=TORCH[dtype], device="cuda")
    rows = torch.zeros(tokens, rank + 64, dtype=TORCH[dtype], device="cuda")
    q_out = torch.zeros(tokens, heads, 64, dtype=TORCH[dtype], device="cuda")
    slots = torch.as_tensor(np.array([3, 31, 0, 17, -1, 9])).cuda()
    api.latent_norm_rope(q_out, dev(q, dtype), dev(x, dtype), dev(weight, dtype), 1e-5,
                         torch.as_tensor(cs).cuda(), torch.as_tensor(pos).cuda(), slots, pool,
                         rows_out=rows, interleaved=interleaved)
    api.check_error()
    with np.errstate(invalid="ignore"):
        ref = latent.norm_rope(q, x, weight, 1e-5, cs, pos, interleaved, dtype)
    assert not np.isfinite(ref[0][1, 0]).all() and np.isfinite(ref[0]).sum() >= ref[0].size - 4
    assert np.isfinite(ref[2][[0, 5]]).all() and (~np.isfinite(ref[2][[1, 2], rank:])).any(1).all()
    assert (ref[2][3, :rank] == 0).sum() == rank - 1 and np.isnan(ref[2][4, :rank]).all()
    assert np.isfinite(ref[2][[1, 2], :rank]).all() and np.isfinite(ref[2][[3, 4], rank:]).all()
    for got, y, size in ((q_out, ref[0], ref[1]), (rows, ref[2], ref[3])):
        g = got.double().cpu().numpy()
        live = np.isfinite(y)
        assert np.array_equal(g[~live], y[~live], equal_nan=True)
        # half a step of the result, and fp32 sums of few terms: below 2^-18
        bound = UNIT[dtype] * abs(y) + LEAST[dtype] + 2.0 ** -18 * size
        assert (abs(g[live] - y[live]) <= bound[live]).all()
    kept = slots >= 0
    assert torch.equal(pool.view(-1, rank + 64)[slots[kept]].view(torch.int16), rows[kept].view(torch.int16))


@pytest.mark.parametrize("bound", [5000, (1 << 31) - 1, (1 << 32) + 3, 1 << 40])
def test_bounds_on_lengths_past_every_length(bound):
    """max_seq_len and max_q_len are bounds: however large, also past 32 bits."""
    rng = np.random.default_rng(33)
    case = Decode(rng, "bf16", rng.integers(0, 200, 70), 5, 256, 16)
    out = case.empty()
    api.decode_latent(out, **{**case.gpu(), "max_seq_len": bound})
    api.check_error()
    ref, far = case.reference()
    check(out, ref, far)
    case = Prefill(rng, "bf16", [30, 300, 1], [30, 310, 5], 2, True)
    out = case.empty()
    api.prefill_latent(out, **{**case.gpu(), "max_q_len": bound})
    api.check_error()
    case.check(out)


def test_prompt_keys_of_nan_behind_the_causal_limit():
    """A key of NaN, or of infinities, reaches only the queries that meet it."""
    rng = np.random.default_rng(34)
    case = Prefill(rng, "bf16", [200, 140], [330, 140], 2, True)
    keys = [int(case.k_starts[1]) - 1, int(case.k_starts[2]) - 20]
    case.kv[keys[0], :, :128] = 0x7FC0
    case.kv[keys[1], 0, :128] = 0x7F80
    case.rows[keys[1], 256:] = 0xFF80
    out = case.empty()
    api.prefill_latent(out, **case.gpu())
    api.check_error()
    live = np.ones(len(case.q), bool)
    live[:case.q_starts[0]] = live[case.q_starts[2]:] = False
    live[case.q_starts[1] - 1] = False
    live[case.q_starts[2] - 20:] = False
    with np.errstate(invalid="ignore"):
        ref, bound = case.reference()
    check(out[torch.as_tensor(live).cuda()], ref[live], bound[live])
    assert torch.isnan(out[int(case.q_starts[1]) - 1]).all()


def test_tables_with_entries_of_no_block_behind_the_lengths():
    """Entries past a sequence's blocks may hold anything: they are not looked at."""
    rng = np.random.default_rng(35)
    case = Decode(rng, "f16", [1, 16, 17, 513, 0, 2000], 20, 512, 16)
    wide = np.full((6, 500), -1, np.int32)
    wide[:, 1::3] = 1 << 30
    for i, n in enumerate(case.lens):
        count = -(-n // 16)
        wide[i, :count] = case.tables[i, :count]
    case.tables = wide
    out = case.empty()
    api.decode_latent(out, **{**case.gpu(), "max_seq_len": 8000})
    api.check_error()
    ref, bound = case.reference()
    check(out, ref, bound)
