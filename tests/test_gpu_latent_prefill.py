"""Prompts' expanded attention where a CTA takes over many pieces of work: pieces
without keys among them."""
import numpy as np
import pytest

from _latent import Prefill
from paged_kv_cache_64_gb300 import api

pytestmark = pytest.mark.gpu


def run(case, **kw):
    out = case.empty()
    api.prefill_latent(out, **{**case.gpu(), **kw})
    api.check_error()
    case.check(out)
    return out


# ------------------------------------------------------------------ works without keys
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("share", [0.1, 0.5, 0.9, 1.0])
def test_sequences_without_keys_among_others(share, causal):
    """Several pieces of work an SM, runs of them without keys between, before and behind
    those with keys."""
    rng = np.random.default_rng(int(10 * share))
    n_q = np.where(rng.random(200) < 0.15, rng.integers(1, 300, 200), rng.integers(1, 40, 200))
    n_k = np.where(rng.random(200) < share, 0, n_q + rng.integers(0, 150, 200))
    run(Prefill(rng, "bf16", n_q, n_k, 8, causal))


@pytest.mark.parametrize("length", [1, 2, 3, 4])
def test_runs_of_works_without_keys(length):
    """One sequence with keys, `length` without, and so on, the last ones without."""
    rng = np.random.default_rng(length)
    n_k = np.where(np.arange(240) % (length + 1) == 0, rng.integers(1, 400, 240), 0)
    run(Prefill(rng, "f16", rng.integers(1, 40, 240), n_k, 8, False))


@pytest.mark.parametrize("heads,n_q,n_k", [(8, 9000, 130), (40, 1500, 1), (16, 4000, 300)])
def test_many_more_queries_than_keys(heads, n_q, n_k):
    """Causal: all queries but the last n_k meet no key, whole pieces of work of them."""
    run(Prefill(np.random.default_rng(heads), "bf16", [n_q], [n_k], heads, True))
