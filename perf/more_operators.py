"""Cases of latent attention over a paged cache (one shared latent row a token), with plain forms.

A token's row holds `rank` latent values, which every head's key and value are products of, and 64 values
of a rotated key part that the heads share; a pool is [blocks][block size][rank + 64].  Four operators, as
a serving program calls them in `paged_kv_cache_64_gb300.api`:

- `latent_norm_rope`: RMS norm of the latent part, rotary positions of the shared key part and of every
  query head's rotary part, and the write of the rows into the pool (for prompts, the rows themselves too);
- `cache_read_latent`: cached tokens' rows back, in the order of their slots (what a prompt's expanded
  attention over cached context starts from);
- `decode_latent`: one query token a sequence in the absorbed form: with queries already multiplied by the
  key expansion, scores are products with whole rows and outputs are weighted sums of the latent parts;
- `prefill_latent`: prompts in the expanded form: every head has keys of 128 values beside the shared 64
  and values of 128, ragged sequences packed one behind the other, each with its cached context.

`own` selects the library's kernels; otherwise `run` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ROPE = 64    # rotary values of a row and of a query head
NOPE = 128   # a head's own key values in the expanded form
VALUE = 128  # a head's values in the expanded form


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the step of a few users of a small model, interleaved pairs
        {"name": "rows step small", "op": "rows", "tokens": 5, "heads": 16, "rank": 256, "block": 16,
         "dtype": "f16", "interleaved": True, "pad": 0.0, "rows_out": False},
        # the decode step of a full batch, a few padded tokens among them
        {"name": "rows step", "op": "rows", "tokens": 256, "heads": 128, "rank": 512, "block": 32,
         "dtype": "bf16", "interleaved": False, "pad": 0.05, "rows_out": False},
        # prompts of a batch, the rows wanted for the expansion too
        {"name": "rows prompts", "op": "rows", "tokens": 16411, "heads": 32, "rank": 512, "block": 16,
         "dtype": "bf16", "interleaved": True, "pad": 0.0, "rows_out": True},
        # a short cached prompt taken back, for the prompt pass that continues it
        {"name": "read short", "op": "read", "tokens": 517, "rank": 256, "block": 16, "dtype": "f16"},
        # long cached prompts taken back
        {"name": "read long", "op": "read", "tokens": 131073, "rank": 512, "block": 16, "dtype": "bf16"},
        # the smallest batch: latency
        {"name": "decode tiny", "op": "decode", "seqs": 4, "heads": 16, "rank": 256, "block": 16,
         "dtype": "f16", "lengths": "uniform", "low": 6, "high": 65},
        # a chat batch of many short contexts, some long
        {"name": "decode chat", "op": "decode", "seqs": 128, "heads": 16, "rank": 512, "block": 16,
         "dtype": "bf16", "lengths": "lognormal", "low": 2, "high": 2049},
        # a full batch, every head on one GPU
        {"name": "decode full batch", "op": "decode", "seqs": 128, "heads": 128, "rank": 512,
         "block": 32, "dtype": "bf16", "lengths": "uniform", "low": 513, "high": 8193},
        # long documents
        {"name": "decode long", "op": "decode", "seqs": 16, "heads": 64, "rank": 512, "block": 16,
         "dtype": "bf16", "lengths": "uniform", "low": 16385, "high": 32769},
        # one user with a very long context
        {"name": "decode one long", "op": "decode", "seqs": 1, "heads": 32, "rank": 512, "block": 16,
         "dtype": "bf16", "lengths": "uniform", "low": 200003, "high": 200003},
        # prompts of a chat batch, nothing cached before them
        {"name": "prefill prompts", "op": "prefill", "seqs": 16, "heads": 16, "dtype": "bf16",
         "low": 31, "high": 2049, "context": 0, "causal": True},
        # pieces of two long prompts behind their cached context
        {"name": "prefill pieces", "op": "prefill", "seqs": 2, "heads": 32, "dtype": "bf16",
         "low": 2048, "high": 4096, "context": 12003, "causal": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rows", "read", "decode", "decode", "prefill", "prefill"])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"])}
    if op != "prefill":
        case["rank"] = rng.choice([256, 512])
        case["block"] = rng.choice([16, 32, 64])
    if op != "read":
        case["heads"] = _log(rng, 1, 128)
    if op == "rows":
        case["tokens"] = _log(rng, 1, 16000)
        case["interleaved"] = rng.random() < 0.5
        case["pad"] = rng.choice([0.0, 0.03, 0.3])
        case["rows_out"] = rng.random() < 0.5
    elif op == "read":
        case["tokens"] = _log(rng, 1, 100000)
    elif op == "decode":
        case["seqs"] = _log(rng, 1, 200)
        # at most half a million positions, padded to the longest
        case["high"] = _log(rng, 8, min(150000, 500000 // case["seqs"]))
        case["low"] = rng.choice([0, 1, max(1, case["high"] // 2), case["high"]])
        case["lengths"] = rng.choice(["uniform", "lognormal"])
    else:
        case["seqs"] = _log(rng, 1, 12)
        case["high"] = _log(rng, 1, 16000 // case["seqs"])
        case["low"] = rng.choice([1, max(1, case["high"] // 2), case["high"]])
        case["context"] = rng.choice([0, 0, _log(rng, 1, 8000)])
        case["causal"] = rng.random() < 0.75
        # no more pairs of a query and a key than the largest listed case has
        pairs = case["seqs"] * case["high"] * (case["high"] + case["context"])
        case["heads"] = max(1, min(case["heads"], int(2.5e9 // pairs)))
    return case


# ------------------------------------------------------------------ inputs
def _slots(rng, tokens, block):
    """Slots of the tokens of consecutive sequences whose blocks lie anywhere in the pool."""
    need = -(-tokens // block)
    blocks = need + max(1, need // 5)
    order = rng.permutation(blocks)[:need]
    slots = (order[:, None] * block + np.arange(block)[None, :]).reshape(-1)[:tokens].astype(np.int64)
    return blocks, slots


def _lengths(rng, case):
    low, high, seqs = case["low"], case["high"], case["seqs"]
    if case.get("lengths") == "lognormal":
        v = np.round(rng.lognormal(math.log(max(1, high / 10)), 0.858, seqs)).astype(np.int64)
        return np.clip(v, low, high)
    return rng.integers(low, high + 1, seqs)


def _angles(positions):
    """Table [positions, 64] of cosines and sines; slow pairs' angles shrunk for long contexts, and
    lengths grown a little, as models trained on short contexts do."""
    rate = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    keep = torch.clamp((torch.arange(ROPE // 2, device="cuda") - 8.0) / 12.0, 0.0, 1.0).double()
    rate = rate * (1 - keep) + rate / 8 * keep
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * rate
    return (torch.cat([angle.cos(), angle.sin()], 1) * (1 + 0.1 * math.log(8))).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def dev(a):
        return torch.as_tensor(a, device="cuda")

    s = {"case": dict(case)}
    op = case["op"]
    if op == "prefill":
        heads = case["heads"]
        # the lengths are the case's, as the outputs' sizes follow from them; their order is
        # the seed's, and what is cached before each
        n_q = rng.permutation(_lengths(np.random.default_rng(case["high"]), case))
        n_k = n_q + (rng.integers(case["context"] // 2, case["context"] + 1, case["seqs"])
                     if case["context"] else 0)
        total_q, total_k = int(n_q.sum()), int(n_k.sum())
        s["q"] = normal(total_q, heads, NOPE + ROPE).to(dtype)
        # keys and values as one product with the expansion leaves them; the shared
        # part is the end of the rows
        expanded = torch.empty(total_k, heads, NOPE + VALUE, dtype=dtype, device="cuda")
        for at in range(0, total_k, 4096):
            expanded[at:at + 4096] = normal(min(4096, total_k - at), heads, NOPE + VALUE)
        s["k"], s["v"] = expanded[..., :NOPE], expanded[..., NOPE:]
        s["k_pe"] = normal(total_k, 512 + ROPE).to(dtype)[:, 512:]
        s["q_starts"] = dev(np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32))
        s["k_starts"] = dev(np.concatenate([[0], np.cumsum(n_k)]).astype(np.int32))
        s["lengths"] = list(zip(n_q.tolist(), n_k.tolist()))
        s["max_q"], s["scale"] = int(n_q.max()), (NOPE + ROPE) ** -0.5
        s["out"] = torch.empty(total_q, heads, VALUE, dtype=dtype, device="cuda")
        return s
    rank, block = case["rank"], case["block"]
    if op == "decode":
        lens = _lengths(rng, case)
        count = -(-lens // block)
        most = int(max(1, count.max()))
        total = int(count.sum())
        blocks = total + max(1, total // 5)
        tables = np.zeros((case["seqs"], most), np.int32)
        used = np.arange(most)[None, :] < count[:, None]
        tables[used] = rng.permutation(blocks)[:total]
        s["q"] = normal(case["seqs"], case["heads"], rank + ROPE).to(dtype)
        s["out"] = torch.empty(case["seqs"], case["heads"], rank, dtype=dtype, device="cuda")
        s["pool"] = torch.empty(blocks, block, rank + ROPE, dtype=dtype, device="cuda")
        for at in range(0, blocks, 8192):
            n = min(8192, blocks - at)
            s["pool"][at:at + n] = normal(n, block, rank + ROPE)
        s["tables"], s["lens"] = dev(tables), dev(lens.astype(np.int32))
        s["max_len"], s["scale"], s["workspace"] = int(lens.max()), (NOPE + ROPE) ** -0.5, None
        return s
    tokens = case["tokens"]
    blocks, slots = _slots(rng, tokens, block)
    if case.get("pad"):
        slots[rng.random(tokens) < case["pad"]] = -1
    s["slots"] = dev(slots)
    if op == "read":
        s["pool"] = normal(blocks, block, rank + ROPE).to(dtype)
        s["rows"] = torch.zeros(tokens, rank + ROPE, dtype=dtype, device="cuda")
        return s
    heads = case["heads"]
    # the query heads' rotary parts lie behind their other parts; they go behind the
    # absorbed queries; the latents are a column range of a down projection's output
    s["q_pe"] = normal(tokens, heads, NOPE + ROPE).to(dtype)[..., NOPE:]
    s["q"] = torch.zeros(tokens, heads, rank + ROPE, dtype=dtype, device="cuda")
    s["latent"] = normal(tokens, 768 + rank + ROPE).to(dtype)[:, 768:]
    s["weight"] = (1 + 0.1 * normal(rank)).to(dtype)
    s["eps"] = 1e-6
    positions = 32768
    s["cos_sin"] = _angles(positions)
    s["positions"] = dev(rng.integers(0, positions, tokens))
    s["pool"] = torch.zeros(blocks, block, rank + ROPE, dtype=dtype, device="cuda")
    s["rows"] = (torch.zeros(tokens, rank + ROPE, dtype=dtype, device="cuda") if case["rows_out"]
                 else None)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_rows(s):
    case = s["case"]
    rank, block = case["rank"], case["block"]
    table = s["cos_sin"][s["positions"]]
    cos, sin = table[:, :ROPE // 2], table[:, ROPE // 2:]

    def turned(x, cos, sin):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    dtype = s["q"].dtype
    s["q"][..., rank:] = turned(s["q_pe"], cos[:, None, :], sin[:, None, :]).to(dtype)
    x = s["latent"].float()
    c = x[:, :rank]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    rows = torch.cat([c, turned(x[:, rank:], cos, sin)], -1).to(dtype)
    keep = s["slots"] >= 0
    s["pool"][s["slots"][keep] // block, s["slots"][keep] % block] = rows[keep]
    return {"q": s["q"], "pool": s["pool"], **({"rows": rows} if case["rows_out"] else {})}


def _plain_read(s):
    block = s["case"]["block"]
    return {"rows": s["pool"][s["slots"] // block, s["slots"] % block]}


def _plain_decode(s):
    rank = s["case"]["rank"]
    seqs, heads, width = s["q"].shape
    piece = max(1, (1 << 30) // max(1, s["tables"].shape[1] * s["case"]["block"] * (width + heads)))
    parts = []
    for at in range(0, seqs, piece):
        rows = s["pool"][s["tables"][at:at + piece].long()].float().flatten(1, 2)
        score = torch.matmul(s["q"][at:at + piece].float(), rows.transpose(1, 2)) * s["scale"]
        seen = (torch.arange(rows.shape[1], device="cuda")[None, :]
                < s["lens"][at:at + piece, None])[:, None, :]
        score = torch.where(seen, score, -math.inf)
        top = score.amax(-1, keepdim=True)
        weight = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
        total = weight.sum(-1, keepdim=True)
        weight = weight / torch.where(total == 0, 1.0, total)
        parts.append(torch.matmul(weight, rows[..., :rank]).to(s["q"].dtype))
    return torch.cat(parts)


def _plain_prefill(s):
    out = torch.empty_like(s["out"])
    a = b = 0
    for n_q, n_k in s["lengths"]:
        k = torch.cat([s["k"][b:b + n_k].float(),
                       s["k_pe"][b:b + n_k, None, :].float().expand(-1, s["k"].shape[1], -1)], -1)
        k, v = k.permute(1, 2, 0), s["v"][b:b + n_k].float().transpose(0, 1)
        for at in range(0, n_q, 512):
            n = min(512, n_q - at)
            q = s["q"][a + at:a + at + n].float().transpose(0, 1)
            score = torch.matmul(q, k) * s["scale"]
            if s["case"]["causal"]:
                last = n_k - n_q + at + torch.arange(n, device="cuda")
                seen = torch.arange(n_k, device="cuda")[None, :] <= last[:, None]
                score = torch.where(seen, score, -math.inf)
            weight = torch.exp(score - score.amax(-1, keepdim=True))
            weight = weight / weight.sum(-1, keepdim=True)
            out[a + at:a + at + n] = torch.matmul(weight, v).transpose(0, 1).to(out.dtype)
        a, b = a + n_q, b + n_k
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from paged_kv_cache_64_gb300 import api
        if op == "rows":
            api.latent_norm_rope(s["q"][..., s["case"]["rank"]:], s["q_pe"], s["latent"], s["weight"],
                                 s["eps"], s["cos_sin"], s["positions"], s["slots"], s["pool"],
                                 rows_out=s["rows"], interleaved=s["case"]["interleaved"])
            return {"q": s["q"], "pool": s["pool"],
                    **({"rows": s["rows"]} if s["case"]["rows_out"] else {})}
        if op == "read":
            api.cache_read_latent(s["rows"], s["slots"], s["pool"])
            return {"rows": s["rows"]}
        if op == "decode":
            s["workspace"] = api.decode_latent(s["out"], s["q"], s["pool"], s["tables"], s["lens"],
                                               s["max_len"], s["scale"], workspace=s["workspace"])
            return {"out": s["out"]}
        api.prefill_latent(s["out"], s["q"], s["k"], s["v"], s["k_pe"], s["q_starts"], s["k_starts"],
                           s["max_q"], s["scale"], causal=s["case"]["causal"])
        return {"out": s["out"]}
    if op == "decode":
        return {"out": _plain_decode(s)}
    if op == "prefill":
        return {"out": _plain_prefill(s)}
    return {"rows": _plain_rows, "read": _plain_read}[op](s)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "prefill":
        many = _lengths(np.random.default_rng(case["high"]), case).astype(np.float64)
        seqs, heads, before = case["seqs"], case["heads"], 0.75 * case["context"]
        tokens = many.sum()
        seen = ((many * (many + 1) / 2 if case["causal"] else many * many) + many * before).mean()
        return {"bytes": float(2 * heads * (tokens * (NOPE + ROPE + VALUE)
                                            + (tokens + before * seqs) * (NOPE + VALUE))
                               + 2 * ROPE * (tokens + before * seqs)),
                "flops": float(2 * seen * seqs * heads * (NOPE + ROPE + VALUE))}
    rank = case["rank"]
    row = 2 * (rank + ROPE)
    if op == "decode":
        # the expected lengths; the drawn ones are near
        rng = np.random.default_rng(0)
        lens = _lengths(rng, {**case, "seqs": 4096}).mean() * case["seqs"]
        return {"bytes": float(lens * row + 4 * lens / case["block"]
                               + case["seqs"] * (2 * case["heads"] * (2 * rank + ROPE) + 4)),
                "flops": float(2 * lens * case["heads"] * (2 * rank + ROPE))}
    tokens = case["tokens"]
    if op == "read":
        return {"bytes": float(tokens * (2 * row + 8)), "flops": 0.0}
    copies = 1 - case["pad"] + (2 if case["rows_out"] else 1)
    return {"bytes": float(tokens * (2 * 2 * ROPE * case["heads"] + copies * row + 4 * ROPE + 16)
                           + 2 * rank),
            "flops": float(tokens * (3 * ROPE * (case["heads"] + 1) + 4 * rank))}


# ------------------------------------------------------------------ exact values
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "read":
        flat = s["pool"].double().view(-1, s["pool"].shape[-1])
        return {"rows": flat.index_select(0, s["slots"])}
    if op == "rows":
        rank, half = case["rank"], ROPE // 2
        table = s["cos_sin"].double()[s["positions"]]
        turn = torch.complex(table[:, :half].contiguous(), table[:, half:].contiguous())

        def turned(x, turn):
            v = x.double()
            if case["interleaved"]:
                z = torch.view_as_complex(v.reshape(*v.shape[:-1], half, 2).contiguous()) * turn
                return torch.view_as_real(z).reshape(v.shape)
            z = torch.complex(v[..., :half].contiguous(), v[..., half:].contiguous()) * turn
            return torch.cat([z.real, z.imag], -1)

        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        q[..., rank:] = turned(s["q_pe"], turn[:, None])
        c = s["latent"][:, :rank].double()
        c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / rank + s["eps"]) * s["weight"].double()
        rows = torch.cat([c, turned(s["latent"][:, rank:], turn)], -1)
        pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
        kept = torch.nonzero(s["slots"] >= 0)[:, 0]
        pool.view(-1, rank + ROPE)[s["slots"][kept]] = rows[kept]
        return {"q": q, "pool": pool, **({"rows": rows} if case["rows_out"] else {})}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if op == "decode":
        rank = case["rank"]
        for i, length in enumerate(s["lens"].tolist()):
            if length == 0:
                continue
            at = s["tables"][i, :-(-length // case["block"])].long()
            rows = s["pool"][at].reshape(-1, rank + ROPE)[:length].double()
            score = s["q"][i].double() @ rows.T * s["scale"]
            out[i] = torch.softmax(score, -1) @ rows[:, :rank]
        return {"out": out}
    a = b = 0
    for n_q, n_k in s["lengths"]:
        shared = s["k_pe"][b:b + n_k].double()
        for h in range(case["heads"] if n_q else 0):
            keys = s["k"][b:b + n_k, h].double()
            values = s["v"][b:b + n_k, h].double()
            for at in range(0, n_q, 2048):
                q = s["q"][a + at:a + min(at + 2048, n_q), h].double()
                score = (q[:, :NOPE] @ keys.T + q[:, NOPE:] @ shared.T) * s["scale"]
                if case["causal"]:
                    hidden = torch.ones(len(q), n_k, dtype=torch.bool, device="cuda")
                    score.masked_fill_(hidden.triu(n_k - n_q + at + 1), -math.inf)
                out[a + at:a + at + len(q), h] = torch.softmax(score, -1) @ values
        a, b = a + n_q, b + n_k
    return {"out": out}
