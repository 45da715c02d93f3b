"""Latent attention and its rows at unusual values: scales far below the scores' sizes."""
import numpy as np
import pytest

from _latent import Decode, Prefill, check
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
