"""Pins of the latent cache's fp64 oracle: closed forms and independent ways to
the same values."""
import numpy as np
import pytest

from oracle import int4, latent


def bits16(rng, *shape, dtype="f16"):
    return int4.narrow(rng.standard_normal(shape), dtype)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_pairs_by_their_angle(interleaved):
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((5, 64)), rng.uniform(-3, 3, (5, 32))
    y, size = latent.turn(x, np.concatenate([np.cos(angle), np.sin(angle)], 1), interleaved)
    pair = lambda v: (v[:, 0::2] + 1j * v[:, 1::2]) if interleaved else (v[:, :32] + 1j * v[:, 32:])
    assert np.allclose(pair(y), pair(x) * np.exp(1j * angle), atol=1e-14)
    assert (abs(y) <= size + 1e-15).all()


def test_rows_are_normed_and_scaled():
    rng = np.random.default_rng(2)
    x, w = bits16(rng, 3, 320), int4.narrow(np.full(256, 2.0), "f16")
    cs = np.concatenate([np.ones((1, 32)), np.zeros((1, 32))], 1)  # no turn
    yq, _, rows, _ = latent.norm_rope(bits16(rng, 3, 2, 64), x, w, 0.0, cs, np.zeros(3, int), False, "f16")
    assert np.allclose((rows[:, :256] ** 2).mean(1), 4.0)
    assert np.array_equal(rows[:, 256:], int4.widen(x[:, 256:], "f16"))


def test_decode_is_softmax_attention_over_the_tables_rows():
    rng = np.random.default_rng(3)
    pool, q = bits16(rng, 6, 16, 320), bits16(rng, 2, 3, 320)
    tables, lens = np.array([[4, 1], [0, 0]]), np.array([21, 0])
    out, size, _ = latent.decode(q, pool, tables, lens, 0.3, "f16")
    rows = np.concatenate([int4.widen(pool[4], "f16"), int4.widen(pool[1], "f16")])[:21]
    for h in range(3):
        w = np.exp(0.3 * rows @ int4.widen(q[0, h], "f16"))
        assert np.allclose(out[0, h], (w / w.sum()) @ rows[:, :256], atol=1e-13)
    assert (out[1] == 0).all() and (abs(out) <= size + 1e-15).all()
    one, _, _ = latent.decode(q, pool, tables, np.array([1, 1]), 0.3, "f16")
    assert np.allclose(one[0], int4.widen(pool[4, 0, :256], "f16"))


@pytest.mark.parametrize("causal", [True, False])
def test_expanded_attention_is_the_absorbed_one(causal):
    """Keys and values that are products of the rows: both forms give the same mixture."""
    rng = np.random.default_rng(4)
    n, rank = 9, 256
    up = rng.integers(-2, 3, (rank, 256)).astype(float)  # products that 16 bits hold
    rows = np.zeros((n, rank + 64))
    rows[:, rng.integers(0, rank, 3)] = rng.integers(-3, 4, (n, 3))
    rows[:, rank:] = rng.integers(-2, 3, (n, 64))
    q = rng.integers(-2, 3, (n, 1, 192)).astype(float)
    f16 = lambda a: int4.narrow(a, "f16")
    kv = rows[:, None, :rank] @ up
    starts = np.array([0, n])
    got, _, _ = latent.prefill(f16(q), f16(kv[..., :128]), f16(kv[..., 128:]), f16(rows[:, rank:]), starts,
                               starts, 0.05, causal, "f16")
    absorbed = np.concatenate([q[..., :128] @ up[:, :128].T, q[..., 128:]], 2)
    for i in range(n):
        last = i + 1 if causal else n
        mix, _, _ = latent.decode(f16(absorbed[i:i + 1]), f16(rows)[None], np.array([[0]]), np.array([last]),
                                  0.05, "f16")
        assert np.allclose(mix[0] @ up[:, 128:], got[i], atol=1e-12)


def test_prompt_behind_a_context_and_queries_without_keys():
    rng = np.random.default_rng(5)
    q, k, v, e = bits16(rng, 4, 2, 192), bits16(rng, 7, 2, 128), bits16(rng, 7, 2, 128), bits16(rng, 7, 64)
    whole = latent.prefill(q, k[:4], v[:4], e[:4], [0, 4], [0, 4], 0.1, True, "f16")[0]
    part = latent.prefill(q[2:], k[:4], v[:4], e[:4], [0, 2], [0, 4], 0.1, True, "f16")[0]
    assert np.allclose(part, whole[2:], atol=1e-14)
    few = latent.prefill(q, k[:2], v[:2], e[:2], [0, 4], [0, 2], 0.1, True, "f16")[0]
    assert (few[:2] == 0).all() and np.allclose(few[2], int4.widen(v[0], "f16"))
