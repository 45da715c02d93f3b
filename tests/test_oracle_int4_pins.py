"""Pins of the 4-bit cache's oracle: hand-worked rows, the error bound, the
record layout, and the 16-bit rounding it rests on."""
import numpy as np
import pytest
import torch

from oracle import int4


def row(values, dtype):
    return int4.narrow(np.asarray(values, np.float64), dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_hand_worked_rows(dtype):
    # 0 .. 15 eight times over: s = 1, m = 0, codes the values themselves
    x = np.tile(np.arange(16.0), 8)
    codes, s, m = int4.quantise(row(x, dtype)[None], dtype)
    assert codes[0].tolist() == x.astype(int).tolist()
    assert int4.widen(s, dtype)[0] == 1.0 and int4.widen(m, dtype)[0] == 0.0
    # span 15 from -3; ties: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    x = np.array([-3.0, 12.0, -2.5, -1.5, -0.5] + [-3.0] * 59)
    codes, s, m = int4.quantise(row(x, dtype)[None], dtype)
    assert codes[0, :5].tolist() == [0, 15, 0, 2, 2]
    assert int4.widen(m, dtype)[0] == -3.0
    # equal values; -0 as the minimum is +0; a NaN, an infinity
    codes, s, m = int4.quantise(row([[2.5] * 64, [-0.0] * 64, [np.nan] + [1.0] * 63,
                                     [-np.inf] + [1.0] * 63], dtype), dtype)
    assert not codes.any()
    assert s[0] == 0 and int4.widen(m, dtype)[0] == 2.5 and m[1] == 0
    assert np.isnan(int4.widen(s, dtype)[2:]).all() and np.isnan(int4.widen(m, dtype)[2:]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_error_is_at_most_half_a_step_and_s_is_smallest(dtype):
    rng = np.random.default_rng(7)
    x = rng.standard_normal((200, 64)) * rng.choice([1e-6, 1e-3, 1.0, 300.0], (200, 1)) + \
        rng.choice([0.0, 5.0, -100.0], (200, 1))
    b = row(x, dtype)
    v = int4.widen(b, dtype)
    codes, s, m = int4.quantise(b, dtype)
    step, low = int4.widen(s, dtype)[:, None], int4.widen(m, dtype)[:, None]
    # fp32's rounding of x - m: 2^-24 of at most 16 steps
    assert (np.abs(v - (low + step * codes)) <= step * (0.5 + 16 * 2.0**-24)).all()
    span = v.max(-1) - v.min(-1)
    assert (15 * step[:, 0] >= span * (1 - 2.0**-24)).all()
    below = int4.widen((s - 1).astype(np.uint16), dtype)
    assert (15 * below < span)[s > 0].all()


def test_bf16_span_past_fp32_is_nan():
    codes, s, m = int4.quantise(row([3e38, -3e38] + [0.0] * 62, "bf16")[None], "bf16")
    assert np.isnan(int4.widen(s, "bf16")).all()


@pytest.mark.parametrize("d,block", [(64, 16), (128, 16), (64, 32), (128, 32)])
def test_record_layout(d, block):
    pool = np.zeros((3, 2, block * (d // 2 + 4)), np.uint8)
    x = np.tile(np.arange(16.0), d // 16)[None, None].repeat(2, 1)  # [1, 2, d]
    x[0, 1] = 15 - x[0, 1] + 4
    int4.cache_write([pool], [row(x, "f16")], [block + 5], block, "f16")
    rec = pool[1, 0]
    assert rec[5 * d // 2:5 * d // 2 + 4].tolist() == [0x10, 0x32, 0x54, 0x76]
    at = block * d // 2 + 4 * 5
    assert rec[at:at + 4].tolist() == [0x00, 0x3C, 0x00, 0x00]      # s = 1.0, m = 0
    assert pool[1, 1][5 * d // 2:5 * d // 2 + 2].tolist() == [0xEF, 0xCD]
    assert pool[1, 1][at:at + 4].tolist() == [0x00, 0x3C, 0x00, 0x44]  # s = 1.0, m = 4
    assert not pool[0].any() and not pool[2].any()
    assert np.array_equal(int4.values(pool, d, block, "f16")[1, :, 5], x[0])
    assert np.array_equal(int4.cache_read(pool, [block + 5], d, block, "f16"), row(x, "f16"))


def test_narrow_matches_torch():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(4000).astype(np.float32) * rng.choice([1e-40, 1e-6, 1.0, 7e4], 4000).astype(np.float32)
    for dtype, t in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        want = torch.tensor(x).to(t).view(torch.int16).numpy().view(np.uint16)
        assert np.array_equal(int4.narrow(x, dtype), want)


def test_norm_rope_turns_by_the_angle():
    # unit weights: a rotated pair keeps its length, and position 0 is the norm alone
    rng = np.random.default_rng(5)
    x = row(rng.standard_normal((3, 2, 64)), "f16")
    w = row(np.ones(64), "f16")
    ang = np.array([0.0, 0.7, -2.0])[:, None] * np.array([1.0, 0.25, 0.5, 2.0, 1, 1, 1, 1])[None]
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    v = int4.widen(x, "f16")
    norm = v / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6)
    for inter in (False, True):
        y = int4.norm_rope(x, w, 1e-6, cs, np.array([0, 1, 2]), inter, "f16")
        assert np.allclose(y[0], norm[0], atol=1e-12)
        assert np.array_equal(y[..., 16:], norm[..., 16:])
        i, j = (0, 1) if inter else (0, 8)
        z = (norm[1, 0, i] + 1j * norm[1, 0, j]) * np.exp(0.7j)
        assert abs(y[1, 0, i] - z.real) < 1e-6 and abs(y[1, 0, j] - z.imag) < 1e-6
