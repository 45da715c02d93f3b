"""Plain fp64 oracle of the 4-bit KV cache and of the norm-and-rotation step.

TEST INFRASTRUCTURE (see oracle/__init__.py): numpy only, shares no code with
the library.  Arrays of 16-bit elements are uint16 bit patterns; dtype is
"f16" or "bf16".  Pools are uint8 [blocks][KV heads][record], a record being
block_size * d / 2 bytes of codes (element 2i in the low half of byte i) and
then block_size pairs (s, m) of 16-bit values.
"""
import numpy as np

LARGEST = {"f16": 65504.0, "bf16": float(np.float32(3.38953138925e38))}


def widen(bits, dtype):
    """uint16 bit patterns as float64."""
    bits = np.asarray(bits, dtype=np.uint16)
    if dtype == "f16":
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def narrow(values, dtype):
    """float64 -> bit patterns of the nearest 16-bit values, ties to even."""
    values = np.asarray(values, dtype=np.float64)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return values.astype(np.float16).view(np.uint16)
    with np.errstate(over="ignore", invalid="ignore"):
        exponent = np.maximum(np.frexp(values)[1], -125)
        unit = np.ldexp(1.0, exponent - 8)  # 8 significant bits, subnormals from 2^-133
        near = np.where(np.isfinite(values), np.rint(values / unit) * unit, values)
        out = near.astype(np.float32).view(np.uint32) >> 16
    return np.where(np.isnan(values), 0x7FC0, out).astype(np.uint16)


def quantise(bits, dtype):
    """Rows [..., d] -> (codes [..., d] uint8, s [...] uint16, m [...] uint16)."""
    x = widen(bits, dtype)
    shape = x.shape[:-1]
    x = x.reshape(-1, x.shape[-1])
    codes = np.zeros(x.shape, np.uint8)
    s_bits, m_bits = np.zeros(len(x), np.uint16), np.zeros(len(x), np.uint16)
    nan = 0x7E00 if dtype == "f16" else 0x7FC0
    for r, row in enumerate(x):
        with np.errstate(over="ignore", invalid="ignore"):
            span = np.float32(row.max()) - np.float32(row.min())  # fp32
        if not np.isfinite(row).all() or not np.isfinite(span):
            s_bits[r] = m_bits[r] = nan
            continue
        m = row.min() + 0.0  # -0 becomes +0
        step = float(span) / 15
        b = narrow(step, dtype)[()]
        while widen(b, dtype) * 15 < float(span):
            b = np.uint16(b + 1)
        while b > 0 and widen(np.uint16(b - 1), dtype) * 15 >= float(span):
            b = np.uint16(b - 1)
        s_bits[r], m_bits[r] = b, narrow(m, dtype)
        s = float(widen(b, dtype))
        if s > 0:
            a = (row.astype(np.float32) - np.float32(m)).astype(np.float64)
            codes[r] = np.clip(np.rint(a / s), 0, 15)
    return codes.reshape(*shape, -1), s_bits.reshape(shape), m_bits.reshape(shape)


def split_pool(pool, d, block_size):
    """(codes [NB, H, B, d], params uint16 [NB, H, B, 2]) of a pool."""
    nb, h, rec = pool.shape
    assert rec == block_size * (d // 2 + 4)
    packed = pool[:, :, :block_size * d // 2].reshape(nb, h, block_size, d // 2)
    codes = np.empty((nb, h, block_size, d), np.uint8)
    codes[..., 0::2] = packed & 15
    codes[..., 1::2] = packed >> 4
    pairs = np.ascontiguousarray(pool[:, :, block_size * d // 2:]).view(np.uint16)
    return codes, pairs.reshape(nb, h, block_size, 2)


def cache_write(pools, news, slots, block_size, dtype):
    """Write rows news[i] [T, H, d] (bits) into pools[i] (in place)."""
    for pool, new in zip(pools, news):
        d = new.shape[-1]
        codes, s, m = quantise(new, dtype)
        for t, slot in enumerate(slots):
            if slot < 0:
                continue
            b, o = divmod(int(slot), block_size)
            pool[b, :, o * d // 2:(o + 1) * d // 2] = codes[t, :, 0::2] | (codes[t, :, 1::2] << 4)
            at = block_size * d // 2 + 4 * o
            pool[b, :, at:at + 4] = np.stack([s[t], m[t]], -1).astype("<u2").view(np.uint8).reshape(-1, 4)


def values(pool, d, block_size, dtype):
    """The fp64 values m + s n of a whole pool [NB, H, B, d]."""
    codes, pairs = split_pool(pool, d, block_size)
    p = widen(pairs, dtype)
    return p[..., 1:2] + p[..., 0:1] * codes


def cache_read(pool, slots, d, block_size, dtype):
    """Bits of the rows at slots [T, H, d]: fl32(m + s n), saturated, to 16 bits."""
    v = values(pool, d, block_size, dtype)
    rows = np.stack([v[int(s) // block_size, :, int(s) % block_size] for s in slots])
    rows = np.clip(rows.astype(np.float32).astype(np.float64), -LARGEST[dtype], LARGEST[dtype])
    return narrow(rows, dtype)


def decode(q_bits, k_pool, v_pool, block_tables, seq_lens, scale, block_size, dtype):
    """fp64 decode attention over 4-bit pools: [S, Hq, d]."""
    q = widen(q_bits, dtype)
    S, hq, d = q.shape
    hkv = k_pool.shape[1]
    G = hq // hkv
    kcodes, kpairs = split_pool(k_pool, d, block_size)
    vcodes, vpairs = split_pool(v_pool, d, block_size)
    out = np.zeros((S, hq, d))
    for i in range(S):
        L = int(seq_lens[i])
        if L == 0:
            continue
        at = block_tables[i, :-(-L // block_size)]
        for h in range(hkv):
            def rows(codes, pairs):
                p = widen(pairs[at, h], dtype)
                return (p[..., 1:2] + p[..., 0:1] * codes[at, h]).reshape(-1, d)[:L]
            s = q[i, h * G:(h + 1) * G] @ rows(kcodes, kpairs).T * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            out[i, h * G:(h + 1) * G] = (w @ rows(vcodes, vpairs)) / w.sum(-1, keepdims=True)
    return out


def norm_rope(x_bits, weight_bits, eps, cos_sin, positions, interleaved, dtype):
    """fp64 RMS norm over the last axis and rotation of rows [T, H, d]."""
    x = widen(x_bits, dtype)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * widen(weight_bits, dtype)
    half = cos_sin.shape[1] // 2
    cs = cos_sin[positions].astype(np.float64)[:, None, :]
    c, s = cs[..., :half], cs[..., half:]
    out = y.copy()
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    out[..., first] = y[..., first] * c - y[..., second] * s
    out[..., second] = y[..., second] * c + y[..., first] * s
    return out
