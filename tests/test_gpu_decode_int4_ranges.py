"""4-bit decode where the sizes within a sequence differ by many powers of ten:
rows of V, queries.  Bounds go by the weights, so that a row without weight
allows nothing.

Tolerance, per sequence and head, with P the softmax weights, v_p the largest
|V| of row p and W = sum_p P_p v_p: half a step of the output type, and
 - a score's dozen roundings, each of a running value below A_p = sum_i |q_i
   k_pi| * scale * log2 e, and that of its difference from the maximum |M|: under
   2^-19 (A_p + |M|) together, so a weight is off by less than e_p =
   2^-18 (A_p + |M|) of itself; numerator and sum: sum_p P_p e_p (v_p + W);
 - exp2, the products and the 22 bits of a weight: 2^-18 W;
 - the sums, a rounding of 2^-23 of sums below 2 W for each 64 positions, and the
   grid of the weights' second terms, 2^-31 of the largest P_p v_p for each
   position: both below L 2^-28 W;
 - weights below 2^-126 of the largest are 0: 2^-126 sum_p v_p."""
import numpy as np
import pytest
import torch

from oracle import int4
from paged_kv_cache_64_gb300 import api

from _parity import bits
from test_gpu_decode_int4 import HALF, Case

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


@pytest.fixture(autouse=True)
def clean_errors():
    assert torch.cuda.is_available()
    yield
    api.check_error()


def allowed(c, ref):
    kv, vv = (int4.values(p, c.d, c.block, c.dtype) for p in (c.kp, c.vp))
    q = int4.widen(c.q, c.dtype)
    S, hq, d = q.shape
    hkv = kv.shape[1]
    tol = HALF[c.dtype] * (1 + 2.0**-8) * np.abs(ref) + (2.0**-25 if c.dtype == "f16" else 0.0)
    for i, L in enumerate(c.lens.tolist()):
        if not L:
            continue
        t = c.tables[i, :-(-L // c.block)]
        for h in range(hkv):
            k = kv[t, h].reshape(-1, d)[:L]
            v = np.abs(vv[t, h].reshape(-1, d)[:L]).max(-1)
            mine = slice(h * hq // hkv, (h + 1) * hq // hkv)
            s = q[i, mine] @ k.T * c.scale * LOG2E
            A = np.abs(q[i, mine]) @ np.abs(k).T * abs(c.scale) * LOG2E
            M = s.max(-1, keepdims=True)
            P = np.exp2(s - M)
            P /= P.sum(-1, keepdims=True)
            W = (P * v).sum(-1, keepdims=True)
            e = 2.0**-18 * (A + np.abs(M))
            tol[i, mine] += ((P * e * (v + W)).sum(-1, keepdims=True) + W * (2.0**-18 + L * 2.0**-28) +
                             2.0**-126 * v.sum())
    return tol


def check(c, out, what=""):
    ref = c.oracle()
    assert np.isfinite(ref).all()
    tol = allowed(c, ref)
    o = int4.widen(bits(out), c.dtype)
    bad = ~(np.abs(o - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), o[bad][:4],
                           ref[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("dtype,small,large", [
    ("f16", 0.05, 6e4), ("f16", 1e-3, 6e4), ("f16", 1e-4, 6e4), ("bf16", 1.0, 1e6),
    ("bf16", 1.0, 1e8), ("bf16", 1.0, 1e10), ("bf16", 1e-3, 1e30)])
@pytest.mark.parametrize("d,group", [(64, 5), (128, 3), (64, 4), (128, 8)])
def test_one_row_far_larger_than_the_rest(dtype, small, large, d, group):
    """First, in the middle or last of a sequence; of the heads that share it
    some give it no weight, some as much as the others' sum, some a full one."""
    lens, at = [333, 333, 333, 40], [0, 333 + 150, 999 - 1, 999 + 17]

    def v(rng, shape):
        x = rng.standard_normal(shape) * small
        x[at] = np.clip(rng.standard_normal((len(at), *shape[1:])), -1, 1) * large
        return x

    def k(rng, shape):
        x = rng.standard_normal(shape)
        x[at] = 0.0
        x[at, :, 0] = -300.0
        return x

    def q(rng, shape):
        x = rng.standard_normal(shape)
        x[:, 0::3, 0] = 8.0
        x[:, 1::3, 0] = 0.0
        x[:, 2::3, 0] = np.log(large / small) / (300.0 * d ** -0.5)
        return x
    c = Case(lens, 2, group, d, 16, dtype, seed=group, q=q, k_rows=k, v_rows=v)
    for partition in (-1, 64, 0):
        check(c, c.gpu(partition), partition)


@pytest.mark.parametrize("d,group", [(64, 2), (128, 7)])
@pytest.mark.parametrize("dtype,first,last", [("f16", 12, -12), ("bf16", 100, -20),
                                              ("f16", -12, 12), ("bf16", -100, 110)])
def test_sizes_that_change_along_rising_scores(d, group, dtype, first, last):
    """The largest weight moves along the sequence, so the sums' scale has to
    come down (and up) with it."""
    def v(rng, shape):
        return rng.standard_normal(shape) * 2.0 ** np.linspace(first, last, shape[0])[:, None, None]

    def k(rng, shape):
        return rng.standard_normal(shape) * 0.1 + np.linspace(0, 30, shape[0])[:, None, None]
    c = Case([700], 2, group, d, 32, dtype, seed=3, v_rows=v, k_rows=k,
             q=lambda r, s: np.ones(s) + 0.1 * r.standard_normal(s))
    for partition in (-1, 96):
        check(c, c.gpu(partition), partition)


def test_ordinary_rows_keep_the_bound():
    c = Case([700, 0, 90, 1500, 1], 2, 4, 128, 16, "bf16")
    for partition in (-1, 256, 0):
        check(c, c.gpu(partition), partition)


@pytest.mark.parametrize("d,group", [(64, 3), (128, 6)])
@pytest.mark.parametrize("eq,ek,escale", [
    (127, -127, -3), (122, -122, -3), (116, -118, -3), (110, -110, -3), (92, -92, -3), (88, -90, 0),
    (70, -118, 40), (20, -118, 90), (-20, 20, -3), (-100, 100, -3), (-115, 115, -3), (-124, 125, -3),
    (-130, 126, -3), (-60, -40, 97)])
def test_queries_of_every_size_bf16_holds(d, group, eq, ek, escale):
    """Queries around 2^eq (from bf16's subnormals to its largest), keys and scale
    such that the scores are ordinary; some heads' queries are 2^20 smaller."""
    def q(rng, shape):
        x = rng.uniform(-1, 1, shape) * 2.0**eq
        x[:, 1::4] *= 2.0**-20 if eq > -100 else 1.0
        x[0, 0] = 0.0
        x[0, -1, 0] = 0.99 * 2.0**eq
        return x
    c = Case([150, 1, 40], 2, group, d, 16, "bf16", seed=5, q=q,
             k_rows=lambda r, s: r.uniform(-1, 1, s) * 2.0**ek)
    c.scale = 2.0**escale
    assert np.isfinite(int4.widen(c.q, "bf16")).all() and np.isfinite(
        int4.values(c.kp, d, 16, "bf16")[c.tables[0, :9]]).all()
    for partition in (-1, 32):
        check(c, c.gpu(partition), partition)
