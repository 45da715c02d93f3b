"""Cases of the 4-bit KV cache and of the norm-and-rotation step that feeds a cache, with plain forms.

Four operators, as a serving program calls them in `paged_kv_cache_64_gb300.api`:

- `cache_write_int4`: new tokens' K and V quantised into paged pools of 4-bit codes, here with the
  stored values returned (what a prompt's own attention then uses);
- `cache_read_int4`: cached tokens back as 16-bit values;
- `decode_int4`: decode attention, one query token a sequence, over such pools;
- `qk_norm_rope`: per-head RMS norm of q and k, rotary positions, and the cache write, in one pass.

A row (one token of one KV head: d values x of a 16-bit type) is held as m = min x, s = the smallest
value of the type that is >= (max x - min x) / 15, and codes n = nearest integer to (x - m) / s, ties
to even (the differences rounded to fp32, the quotients not); it stands for m + s n.  A (block, KV head) record is B * d / 2 bytes of codes (two a byte, the
even element low) followed by B pairs (s, m); a pool is uint8 [blocks][KV heads][B * (d / 2 + 4)].

`own` selects the library's kernels; otherwise `run` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's new tokens of a small model's batch, one layer
        {"name": "write step", "op": "write", "tokens": 128, "kv": 2, "d": 64, "block": 16,
         "dtype": "f16", "pad": 0.0},
        # prompts of a batch, ragged, a few padded tokens behind them
        {"name": "write prompts", "op": "write", "tokens": 40003, "kv": 8, "d": 128, "block": 16,
         "dtype": "bf16", "pad": 0.02},
        # a short cached prompt taken back, for the prompt pass that continues it
        {"name": "read short", "op": "read", "tokens": 517, "kv": 2, "d": 64, "block": 16,
         "dtype": "f16"},
        # long cached prompts taken back
        {"name": "read long", "op": "read", "tokens": 65537, "kv": 8, "d": 128, "block": 16,
         "dtype": "bf16"},
        # the smallest batch: latency
        {"name": "decode tiny", "op": "decode", "seqs": 4, "kv": 2, "group": 2, "d": 64, "block": 16,
         "dtype": "f16", "lengths": "uniform", "low": 6, "high": 65},
        # a chat batch of a small model: many short contexts, some long, one layer
        {"name": "decode chat", "op": "decode", "seqs": 128, "kv": 2, "group": 7, "d": 64,
         "block": 16, "dtype": "f16", "lengths": "lognormal", "low": 2, "high": 2049},
        # a full batch of a mid-size model
        {"name": "decode full batch", "op": "decode", "seqs": 256, "kv": 8, "group": 4, "d": 128,
         "block": 16, "dtype": "bf16", "lengths": "uniform", "low": 513, "high": 8193},
        # long documents
        {"name": "decode long", "op": "decode", "seqs": 16, "kv": 8, "group": 8, "d": 128,
         "block": 16, "dtype": "bf16", "lengths": "uniform", "low": 16385, "high": 32769},
        # one user with a very long context
        {"name": "decode one long", "op": "decode", "seqs": 1, "kv": 8, "group": 4, "d": 128,
         "block": 32, "dtype": "bf16", "lengths": "uniform", "low": 200003, "high": 200003},
        # the step of a few users of a small model, partly rotated heads
        {"name": "rope step small", "op": "rope", "tokens": 5, "kv": 2, "group": 7, "d": 64,
         "block": 16, "dtype": "f16", "rot": 32, "interleaved": True, "pad": 0.0},
        # the decode step of a full batch
        {"name": "rope step", "op": "rope", "tokens": 256, "kv": 8, "group": 4, "d": 128,
         "block": 16, "dtype": "bf16", "rot": 128, "interleaved": False, "pad": 0.05},
        # prompts of a batch
        {"name": "rope prompts", "op": "rope", "tokens": 16411, "kv": 8, "group": 4, "d": 128,
         "block": 16, "dtype": "bf16", "rot": 128, "interleaved": False, "pad": 0.0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "rope"])
    d = rng.choice([64, 128])
    case = {"op": op, "kv": rng.choice([1, 2, 4, 8]), "d": d, "block": rng.choice([16, 32]),
            "dtype": rng.choice(["f16", "bf16"])}
    if op in ("write", "read"):
        case["tokens"] = _log(rng, 1, 40000)
        if op == "write":
            case["pad"] = rng.choice([0.0, 0.03, 0.3])
    elif op == "rope":
        case["tokens"] = _log(rng, 1, 16000)
        case["group"] = rng.randint(1, 8)
        case["rot"] = 16 * rng.randint(1, d // 16)
        case["interleaved"] = rng.random() < 0.5
        case["pad"] = rng.choice([0.0, 0.03, 0.3])
    else:
        case["group"] = rng.randint(1, 8)
        case["seqs"] = _log(rng, 1, 200)
        # at most two thirds of a million positions, padded to the longest
        case["high"] = _log(rng, 8, min(120000, 650000 // case["seqs"]))
        case["low"] = rng.choice([0, 1, max(1, case["high"] // 2), case["high"]])
        case["lengths"] = rng.choice(["uniform", "lognormal"])
    return case


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """Codes (int16), s and m (the type of x) of rows x [..., d] of a 16-bit type: differences in 32
    bits, quotients in 64, so that values next to a border fall on the right side."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    span = (hi.float() - lo.float()).double()
    step = span / torch.full_like(span, 15)  # a tensor: by a number it would be a product with 1/15
    s = step.to(x.dtype)
    s = torch.where(s.double() < step, (s.view(torch.int16) + 1).view(x.dtype), s)
    t = (x.float() - lo.float()).double() / s.double()
    n = torch.where(s == 0, 0.0, t).round().clamp(0, 15)
    return n.to(torch.int16), s, lo


def _records(n, s, m):
    """Pool records [blocks, heads, B * (d/2 + 4)] of codes [blocks, heads, B, d] and s, m [.., 1]."""
    blocks, heads = n.shape[:2]
    packed = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8).reshape(blocks, heads, -1)
    params = torch.cat([s, m], -1).contiguous().view(torch.uint8).reshape(blocks, heads, -1)
    return torch.cat([packed, params], -1)


def _pool(g, blocks, case, spread):
    """A pool whose every slot holds a quantised row of normal values, each channel with its own scale."""
    kv, d, block, dtype = case["kv"], case["d"], case["block"], DTYPES[case["dtype"]]
    out = torch.empty(blocks, kv, block * (d // 2 + 4), dtype=torch.uint8, device="cuda")
    channel = torch.exp(spread * torch.randn(kv, 1, d, generator=g, device="cuda"))
    piece = max(1, (1 << 27) // (kv * block * d))
    for b in range(0, blocks, piece):
        n = min(piece, blocks - b)
        x = torch.randn(n, kv, block, d, generator=g, device="cuda") * channel
        out[b:b + n] = _records(*_quantise(x.to(dtype)))
    return out


def _slots(rng, tokens, case):
    """Slots of the tokens of consecutive sequences whose blocks lie anywhere in the pool."""
    block = case["block"]
    need = -(-tokens // block)
    blocks = need + max(1, need // 5)
    order = rng.permutation(blocks)[:need]
    slots = (order[:, None] * block + np.arange(block)[None, :]).reshape(-1)[:tokens].astype(np.int64)
    return blocks, slots


def _lengths(rng, case):
    low, high, seqs = case["low"], case["high"], case["seqs"]
    if case["lengths"] == "lognormal":
        v = np.round(rng.lognormal(math.log(max(1, high / 10)), 0.858, seqs)).astype(np.int64)
        return np.clip(v, low, high)
    return rng.integers(low, high + 1, seqs)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dtype, kv, d, block = DTYPES[case["dtype"]], case["kv"], case["d"], case["block"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def dev(a):
        return torch.as_tensor(a, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "decode":
        lens = _lengths(rng, case)
        count = -(-lens // block)
        most = int(max(1, count.max()))
        total = int(count.sum())
        blocks = total + max(1, total // 5)
        tables = np.zeros((case["seqs"], most), np.int32)
        used = np.arange(most)[None, :] < count[:, None]
        tables[used] = rng.permutation(blocks)[:total]
        s["q"] = normal(case["seqs"], kv * case["group"], d).to(dtype)
        s["out"] = torch.empty_like(s["q"])
        s["k_pool"], s["v_pool"] = _pool(g, blocks, case, 0.4), _pool(g, blocks, case, 0.1)
        s["tables"], s["lens"] = dev(tables), dev(lens.astype(np.int32))
        s["max_len"], s["scale"], s["workspace"] = int(lens.max()), d ** -0.5, None
        return s
    tokens = case["tokens"]
    blocks, slots = _slots(rng, tokens, case)
    if case.get("pad"):
        slots[rng.random(tokens) < case["pad"]] = -1
    s["slots"] = dev(slots)
    if case["op"] == "read":
        s["k_pool"], s["v_pool"] = _pool(g, blocks, case, 0.4), _pool(g, blocks, case, 0.1)
        s["k_out"] = torch.zeros(tokens, kv, d, dtype=dtype, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    if case["op"] == "write":
        channel = torch.exp(0.4 * normal(1, kv, d))
        s["k"] = (normal(tokens, kv, d) * channel).to(dtype)
        s["v"] = normal(tokens, kv, d).to(dtype)
        s["k_pool"] = torch.zeros(blocks, kv, block * (d // 2 + 4), dtype=torch.uint8, device="cuda")
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
        return s
    # rope: q, k and v are column ranges of one projection's output, as a program has them
    heads = kv * case["group"]
    qkv = normal(tokens, (heads + 2 * kv) * d).to(dtype)
    s["q"] = qkv[:, :heads * d].view(tokens, heads, d)
    s["k"] = qkv[:, heads * d:(heads + kv) * d].view(tokens, kv, d)
    s["v"] = qkv[:, (heads + kv) * d:].view(tokens, kv, d)
    s["q_weight"] = (1 + 0.1 * normal(d)).to(dtype)
    s["k_weight"] = (1 + 0.1 * normal(d)).to(dtype)
    s["eps"] = 1e-6
    positions = 32768
    rate = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * rate
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["positions"] = dev(rng.integers(0, positions, tokens))
    s["k_pool"] = torch.zeros(blocks, kv, block, d, dtype=dtype, device="cuda")
    s["v_pool"] = torch.zeros_like(s["k_pool"])
    s["q_out"] = torch.empty(tokens, heads, d, dtype=dtype, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _split(rows, case, codes_shape):
    """fp32 (codes, s, m) of record bytes [..., B * (d/2 + 4)]."""
    d, block, dtype = case["d"], case["block"], DTYPES[case["dtype"]]
    cut = block * d // 2
    packed = rows[..., :cut]
    n = torch.stack([packed & 15, packed >> 4], -1).reshape(*codes_shape, block, d).float()
    params = rows[..., cut:].contiguous().view(dtype).reshape(*codes_shape, block, 2).float()
    return n, params[..., 0:1], params[..., 1:2]


def _values(n, s, m, dtype):
    top = torch.finfo(dtype).max
    return (m.float() + s.float() * n.float()).clamp(-top, top).to(dtype)


def _plain_write(s):
    case = s["case"]
    d, block = case["d"], case["block"]
    cut, kv = block * d // 2, case["kv"]
    keep = s["slots"] >= 0
    blk, off = s["slots"][keep] // block, s["slots"][keep] % block
    done = {}
    for name in ("k", "v"):
        x = s[name]
        n, scale, low = _quantise(x)
        pool = s[name + "_pool"]
        codes = pool[..., :cut].view(-1, kv, block, d // 2)
        params = pool[..., cut:].view(-1, kv, block, 4)
        codes[blk, :, off] = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)[keep]
        params[blk, :, off] = torch.cat([scale, low], -1).contiguous().view(torch.uint8)[keep]
        values = _values(n, scale, low, x.dtype)
        done[name] = torch.where(keep[:, None, None], values, s[name + "_out"])
    return done


def _plain_read(s):
    case = s["case"]
    block = case["block"]
    blk, off = s["slots"] // block, s["slots"] % block
    done = {}
    for name in ("k", "v"):
        pool = s[name + "_pool"]
        n, scale, low = _split(pool, case, pool.shape[:2])
        done[name] = _values(n[blk, :, off], scale[blk, :, off], low[blk, :, off],
                             DTYPES[case["dtype"]])
    return done


def _plain_decode(s):
    case = s["case"]
    kv, d, seqs = case["kv"], case["d"], case["seqs"]
    table = s["tables"].long()

    def values(pool):  # [seqs, heads, positions, d]
        n, scale, low = _split(pool[table], case, (*table.shape, kv))
        return (low + scale * n).permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, d)

    q = s["q"].float().view(seqs, kv, -1, d)
    score = torch.matmul(q, values(s["k_pool"]).transpose(-1, -2)) * s["scale"]
    seen = torch.arange(score.shape[-1], device="cuda")[None, :] < s["lens"][:, None]
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = weight.sum(-1, keepdim=True)
    weight = weight / torch.where(total == 0, 1.0, total)
    return torch.matmul(weight, values(s["v_pool"])).reshape(seqs, -1, d).to(s["q"].dtype)


def _plain_rope(s):
    case = s["case"]
    rot, block = case["rot"], case["block"]
    table = s["cos_sin"][s["positions"]][:, None, :]
    cos, sin = table[..., :rot // 2], table[..., rot // 2:]

    def turned(x, weight):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
        if case["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            y[..., :rot] = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            y[..., :rot] = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return y

    dtype = s["q"].dtype
    keep = s["slots"] >= 0
    blk, off = s["slots"][keep] // block, s["slots"][keep] % block
    s["k_pool"][blk, :, off] = turned(s["k"], s["k_weight"]).to(dtype)[keep]
    s["v_pool"][blk, :, off] = s["v"][keep]
    return {"q": turned(s["q"], s["q_weight"]).to(dtype), "k": s["k_pool"], "v": s["v_pool"]}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from paged_kv_cache_64_gb300 import api
        if op == "write":
            api.cache_write_int4(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"],
                                 k_out=s["k_out"], v_out=s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if op == "read":
            api.cache_read_int4(s["k_out"], s["v_out"], s["slots"], s["k_pool"], s["v_pool"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if op == "decode":
            s["workspace"] = api.decode_int4(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"],
                                             s["lens"], s["max_len"], s["scale"],
                                             workspace=s["workspace"])
            return {"out": s["out"]}
        api.qk_norm_rope(s["q_out"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["eps"],
                         s["cos_sin"], s["positions"], s["slots"], s["k_pool"], s["v_pool"],
                         interleaved=s["case"]["interleaved"])
        return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}
    if op == "decode":
        return {"out": _plain_decode(s)}
    return {"write": _plain_write, "read": _plain_read, "rope": _plain_rope}[op](s)


# ------------------------------------------------------------------ work
def work(case):
    kv, d, op = case["kv"], case["d"], case["op"]
    row = d // 2 + 4
    if op == "decode":
        # the expected lengths; the drawn ones are near
        rng = np.random.default_rng(0)
        lens = _lengths(rng, {**case, "seqs": 4096}).mean() * case["seqs"]
        heads = kv * case["group"]
        return {"bytes": float(lens * kv * 2 * row + 4 * lens / case["block"]
                               + case["seqs"] * (4 * heads * d + 4)),
                "flops": float(4 * lens * heads * d)}
    tokens = case["tokens"]
    kept = tokens * (1 - case.get("pad", 0.0))
    wide = 2 * kv * d * 2  # K and V of a token in 16 bits
    if op == "write":
        return {"bytes": float(kept * (2 * wide + 2 * kv * row) + 8 * tokens),
                "flops": float(kept * 2 * kv * d * 8)}
    if op == "read":
        return {"bytes": float(tokens * (wide + 2 * kv * row + 8)), "flops": float(tokens * 2 * kv * d * 2)}
    heads = kv * case["group"]
    return {"bytes": float(tokens * (2 * 2 * heads * d + 4 * case["rot"] + 16) + kept * 2 * wide + 4 * d),
            "flops": float(tokens * heads * d * 8 + kept * kv * d * 8)}


# ------------------------------------------------------------------ exact values
def _wide(records, case):
    """fp64 values [n, heads, B, d] of pool records [n, heads, bytes]."""
    d, block = case["d"], case["block"]
    code = records[:, :, :block * d // 2].to(torch.int64).view(*records.shape[:2], block, d // 2)
    pair = records[:, :, block * d // 2:].clone().view(DTYPES[case["dtype"]])
    pair = pair.view(*records.shape[:2], block, 2).double()
    value = torch.empty(*code.shape[:3], d, dtype=torch.float64, device=records.device)
    value[..., 0::2] = (code % 16).double()
    value[..., 1::2] = (code // 16).double()
    return value * pair[..., :1] + pair[..., 1:]


def _exact_rows(x):
    """What rows x stand for once quantised, in 64 bits."""
    v = x.double()
    low = v.min(-1, keepdim=True).values
    step = (v.max(-1, keepdim=True).values - low).cpu().numpy() / 15
    exponent = np.frexp(step)[1]
    bits, least = (11, -24) if x.dtype == torch.float16 else (8, -133)
    unit = np.ldexp(1.0, np.maximum(exponent - bits, least))
    s = torch.as_tensor(np.ceil(step / unit) * unit, device=x.device)
    n = torch.round((v - low) / torch.where(s > 0, s, 1.0))
    return low + n * s


def exact(case, seed):
    s = prepare(case, seed)
    block, d, kv, op = case["block"], case["d"], case["kv"], case["op"]
    if op == "write":
        keep = (s["slots"] >= 0)[:, None, None]
        return {n: torch.where(keep, _exact_rows(s[n]), 0.0) for n in ("k", "v")}
    if op == "read":
        done = {}
        for name in ("k", "v"):
            parts = []
            for at in torch.split(s["slots"], 4096):
                rows = _wide(s[name + "_pool"][at // block], case)
                parts.append(rows[torch.arange(len(at), device="cuda"), :, at % block])
            done[name] = torch.cat(parts)
        return done
    if op == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for i, length in enumerate(s["lens"].tolist()):
            if length == 0:
                continue
            at = s["tables"][i, :-(-length // block)].long()
            for h in range(kv):
                k = _wide(s["k_pool"][at, h:h + 1], case).reshape(-1, d)[:length]
                v = _wide(s["v_pool"][at, h:h + 1], case).reshape(-1, d)[:length]
                mine = slice(h * case["group"], (h + 1) * case["group"])
                score = s["q"][i, mine].double() @ k.T * s["scale"]
                out[i, mine] = torch.softmax(score, -1) @ v
        return {"out": out}
    half = case["rot"] // 2
    cs = s["cos_sin"][s["positions"]].double()
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]

    def turned(x, weight):
        v = x.double()
        y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + s["eps"]) * weight.double()
        if case["interleaved"]:
            z = torch.complex(y[..., 0:2 * half:2].contiguous(), y[..., 1:2 * half:2].contiguous()) * turn
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    pools = {n: torch.zeros(s[n + "_pool"].shape, dtype=torch.float64, device="cuda") for n in ("k", "v")}
    kept = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][kept]
    pools["k"][at // block, :, at % block] = turned(s["k"], s["k_weight"])[kept]
    pools["v"][at // block, :, at % block] = s["v"].double()[kept]
    return {"q": turned(s["q"], s["q_weight"]), **pools}
