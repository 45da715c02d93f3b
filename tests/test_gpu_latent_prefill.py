"""Prompts' expanded attention where a CTA takes over many pieces of work: pieces
without keys among them, and batches of many sequences and of very different lengths."""
import numpy as np
import pytest
import torch

from _latent import Prefill, check
from paged_kv_cache_64_gb300 import _lib, api

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


# ------------------------------------------------------------------ which work a block is
@pytest.mark.parametrize("max_q_len", [100, 1 << 20, (1 << 31) - 1])
def test_bound_on_queries_far_above_them(max_q_len):
    rng = np.random.default_rng(20)
    n_q = rng.integers(0, 20, 300)
    run(Prefill(rng, "bf16", n_q, n_q + rng.integers(0, 9, 300), 2, True), max_q_len=max_q_len)


@pytest.mark.parametrize("heads,context", [(3, 20), (12, 110)])
@pytest.mark.parametrize("at", [0, 200, 290, 399])
def test_one_long_prompt_among_many_short(heads, context, at):
    """More sequences than the fetching warp holds at once, in either order of work."""
    rng = np.random.default_rng(at)
    n_q = rng.integers(0, 6, 400)
    n_q[at] = 900
    n_k = n_q + rng.integers(context // 2, context, 400)
    case = Prefill(rng, "bf16", n_q, n_k, heads, True)
    assert (len(case.kv) * heads > 400000) == (heads == 12)
    run(case)


@pytest.mark.parametrize("full", [[0], [599], [255, 256], [10, 511, 512]])
def test_padded_batches(full):
    """Most sequences are empty."""
    rng = np.random.default_rng(full[0])
    n_q = np.zeros(600, np.int64)
    n_q[full] = rng.integers(200, 700, len(full))
    run(Prefill(rng, "f16", n_q, n_q, 2, False))


def test_more_pieces_of_work_than_blocks():
    """65,535 sequences of a token with one key: each output is that key's value."""
    S, heads = 65535, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.empty(S, heads, w, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
               for w in (192, 128, 128))
    k_pe = torch.empty(S, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    starts = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    out = torch.full_like(v, 7.0)
    api.prefill_latent(out, q, k, v, k_pe, starts, starts, 1, 0.1)
    api.check_error()
    assert torch.equal(out, v)


def test_starts_that_go_back():
    """Sequences that repeat others' queries behind a bad one: more pieces of work than
    as many tokens and sequences have in order."""
    rng = np.random.default_rng(21)
    case = Prefill(rng, "bf16", [600, 600], [600, 600], 1, True, gap=0)
    ref, bound = case.reference()
    starts = torch.tensor([0, 600] * 9 + [1200], dtype=torch.int32, device="cuda")
    out = case.empty()
    api.prefill_latent(out, **{**case.gpu(), "q_starts": starts, "k_starts": starts})
    with pytest.raises(_lib.PagedAttentionError) as e:
        api.check_error()
    assert e.value.code == 6
    check(out, ref, bound)


def test_bad_starts_far_behind():
    """A bad sequence behind the last piece of work is reported too."""
    rng = np.random.default_rng(22)
    n = np.zeros(700, np.int64)
    n[3] = 40
    case = Prefill(rng, "bf16", n, n, 2, True)
    g, out = case.gpu(), case.empty()
    g["k_starts"][700] += 1 << 20
    api.prefill_latent(out, **g)
    with pytest.raises(_lib.PagedAttentionError):
        api.check_error()
    case.check(out)


@pytest.mark.parametrize("max_q_len", [300, 3000])
def test_lengths_change_between_replays(max_q_len):
    """A graph's launch is of the tokens and bounds it was captured with; which work its
    blocks are follows the starts at each replay."""
    rng = np.random.default_rng(23)
    n = np.full(250, 12)
    case = Prefill(rng, "bf16", n, n, 3, True, gap=0)
    g, out = case.gpu(), case.empty()
    g["max_q_len"] = max_q_len
    api.prefill_latent(out, **g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.prefill_latent(out, **g)
    for kind in range(4):
        n = rng.multinomial(3000, rng.dirichlet(np.full(250, 0.05 if kind % 2 else 5.0)))
        n = np.minimum(n, max_q_len)
        case.n_q = n
        case.n_k = np.where(rng.random(250) < 0.3, 0, n) if kind > 1 else n
        case.q_starts, case.k_starts = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32)
                                        for x in (case.n_q, case.n_k))
        g["q_starts"].copy_(torch.as_tensor(case.q_starts))
        g["k_starts"].copy_(torch.as_tensor(case.k_starts))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        api.check_error()
        case.check(out)
