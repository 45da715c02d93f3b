"""Plain fp64 oracle of latent attention over a paged cache of shared rows.

TEST INFRASTRUCTURE (see oracle/__init__.py): numpy only, shares no code with
the library.  Arrays of 16-bit elements are uint16 bit patterns; dtype is
"f16" or "bf16".  A row is rank latent values and 64 shared key values; a pool
is [blocks][block size][rank + 64].  Beside each result comes the size that its
rounding errors scale with.
"""
import numpy as np

from .int4 import widen

ROPE = 64


def turn(x, cos_sin, interleaved):
    """Rotary parts x [..., 64] (fp64) by table rows cos_sin [..., 64]; also |a c| + |b s|."""
    c, s = cos_sin[..., :32].astype(np.float64), cos_sin[..., 32:].astype(np.float64)
    first = slice(0, None, 2) if interleaved else slice(0, 32)
    second = slice(1, None, 2) if interleaved else slice(32, 64)
    a, b = x[..., first], x[..., second]
    y, size = np.empty_like(x), np.empty_like(x)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first], size[..., second] = abs(a * c) + abs(b * s), abs(b * c) + abs(a * s)
    return y, size


def norm_rope(q, latent, weight, eps, cos_sin, positions, interleaved, dtype):
    """(turned q [T, H, 64], its size, rows [T, rank + 64], their size), fp64."""
    rank = latent.shape[1] - ROPE
    table = cos_sin[positions]
    yq, size_q = turn(widen(q, dtype), table[:, None, :], interleaved)
    x = widen(latent, dtype)
    c = x[:, :rank] / np.sqrt((x[:, :rank] ** 2).mean(-1, keepdims=True) + eps) * widen(weight, dtype)
    pe, size_pe = turn(x[:, rank:], table, interleaved)
    return yq, size_q, np.concatenate([c, pe], 1), np.concatenate([abs(c), size_pe], 1)


def _attend(q, keys, values, scale):
    """Scores scale q keys^T for q [H, n, w], keys [H, m, w], the sums of their absolute terms,
    and the values [H, m, d] as they are: what _weigh takes."""
    with np.errstate(invalid="ignore"):
        s = np.einsum("hnw,hmw->hnm", q, keys) * scale
        terms = np.einsum("hnw,hmw->hnm", abs(q), abs(keys)) * abs(scale)
    return s, terms, values


def _weigh(s, terms, values):
    """softmax(s) values, with the weights' sum of |values| and the largest of the terms of a
    row's live scores; zeros where a row has none."""
    if s.shape[-1] == 0:
        shape = (*s.shape[:-1], values.shape[-1])
        return np.zeros(shape), np.zeros(shape), np.zeros(s.shape[:-1])
    top = s.max(-1, keepdims=True)
    live = np.isfinite(top)
    w = np.where(live, np.exp(s - np.where(live, top, 0.0)), 0.0)
    total = w.sum(-1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return w @ values, w @ abs(values), np.where(np.isfinite(s), terms, 0.0).max(-1)


def decode(q, pool, tables, lens, scale, dtype):
    """(out [S, H, rank], weighted |values| like out, score terms [S, H]), fp64."""
    S, H, width = q.shape
    block = pool.shape[1]
    out, size = np.zeros((S, H, width - ROPE)), np.zeros((S, H, width - ROPE))
    terms = np.zeros((S, H))
    for i in range(S):
        L = int(lens[i])
        if L == 0:
            continue
        rows = widen(pool[tables[i, :-(-L // block)]].reshape(-1, width)[:L], dtype)
        qi = widen(q[i], dtype)
        s, t, v = _attend(qi[None], rows[None], rows[None, :, :width - ROPE], scale)
        o, a, t = _weigh(s, t, v)
        out[i], size[i], terms[i] = o[0], a[0], t[0]
    return out, size, terms


def prefill(q, k, v, k_pe, q_starts, k_starts, scale, causal, dtype):
    """(out [Tq, H, 128], weighted |values|, score terms [Tq, H]), fp64; rows of no sequence are zero."""
    Tq, H, _ = q.shape
    out, size, terms = np.zeros((Tq, H, 128)), np.zeros((Tq, H, 128)), np.zeros((Tq, H))
    for i in range(len(q_starts) - 1):
        a0, a1, b0, b1 = q_starts[i], q_starts[i + 1], k_starts[i], k_starts[i + 1]
        n_q, n_k = a1 - a0, b1 - b0
        if n_q == 0:
            continue
        keys = np.concatenate([widen(k[b0:b1], dtype),
                               np.broadcast_to(widen(k_pe[b0:b1], dtype)[:, None], (n_k, H, ROPE))], 2)
        s, t, values = _attend(widen(q[a0:a1], dtype).transpose(1, 0, 2), keys.transpose(1, 0, 2),
                               widen(v[b0:b1], dtype).transpose(1, 0, 2), scale)
        if causal:
            hidden = np.arange(n_k)[None, :] > n_k - n_q + np.arange(n_q)[:, None]
            s = np.where(hidden[None], -np.inf, s)
        o, z, t = _weigh(s, t, values)
        out[a0:a1], size[a0:a1] = o.transpose(1, 0, 2), z.transpose(1, 0, 2)
        terms[a0:a1] = t.transpose(1, 0)
    return out, size, terms
