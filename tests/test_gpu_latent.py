"""The latent cache on the GPU: norm, rotation and write; read-back; absorbed
decode; expanded prompts; and all of them together."""
import numpy as np
import pytest
import torch

from _latent import (LEAST, UNIT, Decode, Prefill, TORCH, attention_bound, back, bits16, check, dev,
                     table)
from oracle import int4, latent
from paged_kv_cache_64_gb300 import _lib, api

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("dtype", ["f16", "bf16"])


# ------------------------------------------------------------------ rows
class Rows:
    def __init__(self, rng, dtype, tokens, heads, rank, block, wide=0):
        self.dtype, self.rank, self.block = dtype, rank, block
        self.q = bits16(rng, tokens, heads, 128 + 64, dtype=dtype)
        self.latent = bits16(rng, tokens, wide + rank + 64, dtype=dtype, size=3.0)
        self.weight = bits16(rng, rank, dtype=dtype)
        self.cs = table(50, 1.2)
        self.pos = rng.integers(0, 50, tokens)
        blocks = tokens // block + 3
        self.slots = rng.permutation(blocks * block)[:tokens].astype(np.int64)
        self.pool = bits16(rng, blocks, block, rank + 64, dtype=dtype)
        self.wide, self.eps = wide, 1e-5

    def reference(self, interleaved):
        yq, sq, rows, sr = latent.norm_rope(self.q[..., 128:], self.latent[:, self.wide:], self.weight,
                                            self.eps, self.cs, np.clip(self.pos, 0, 49), interleaved,
                                            self.dtype)
        # half a step of the result; fp32: the norm's sum (rank / 32 terms a lane, five
        # levels), its root and two products, or two products and a sum: below 2^-18
        bound = lambda y, size: UNIT[self.dtype] * abs(y) + LEAST[self.dtype] + 2.0 ** -18 * size
        return (yq, bound(yq, sq)), (rows, bound(rows, sr))

    def gpu(self):
        c = lambda a: torch.as_tensor(a).cuda()
        return dict(q=dev(self.q, self.dtype)[..., 128:], latent=dev(self.latent, self.dtype)[:, self.wide:],
                    weight=dev(self.weight, self.dtype), eps=self.eps, cos_sin=c(self.cs),
                    positions=c(self.pos), slot_mapping=c(self.slots), pool=dev(self.pool, self.dtype))


@BOTH
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,rank,block,wide", [
    (1, 1, 256, 16, 0), (5, 16, 512, 32, 8), (7, 17, 256, 64, 24), (33, 128, 512, 16, 0),
    (3, 1024, 256, 16, 0), (1300, 3, 512, 32, 768)])
def test_norm_rope(dtype, interleaved, tokens, heads, rank, block, wide):
    rng = np.random.default_rng(tokens + heads)
    r = Rows(rng, dtype, tokens, heads, rank, block, wide)
    r.slots[rng.random(tokens) < 0.2] = -1
    g = r.gpu()
    q_out = torch.full((tokens, heads, rank + 64), 5.0, dtype=TORCH[dtype], device="cuda")
    rows = torch.full((tokens, rank + 64), 5.0, dtype=TORCH[dtype], device="cuda")
    api.latent_norm_rope(q_out[..., rank:], rows_out=rows, interleaved=interleaved, **g)
    api.check_error()
    (yq, bq), (yr, br) = r.reference(interleaved)
    check(q_out[..., rank:], yq, bq, "queries")
    assert (q_out[..., :rank] == 5.0).all()
    check(rows, yr, br, "rows")
    want = r.pool.copy().reshape(-1, rank + 64)
    kept = r.slots >= 0
    want[r.slots[kept]] = back(rows)[kept]
    assert np.array_equal(back(g["pool"]).reshape(-1, rank + 64), want)
    # without rows_out, in place: the same bits
    pool, q = dev(r.pool, dtype), dev(r.q, dtype)
    api.latent_norm_rope(q[..., 128:], **{**g, "q": q[..., 128:], "pool": pool}, interleaved=interleaved)
    assert torch.equal(pool.view(torch.int16), g["pool"].view(torch.int16))
    assert torch.equal(q[..., 128:], q_out[..., rank:])
    assert np.array_equal(back(q[..., :128]), r.q[..., :128])


def test_norm_rope_bad_positions_and_slots():
    rng = np.random.default_rng(2)
    r = Rows(rng, "bf16", 40, 20, 256, 16)
    r.pos[[3, 9]] = [-1, 50]
    r.slots[[5, 11]] = [len(r.pool) * 16, 1 << 40]
    g = r.gpu()
    q_out = torch.full((40, 20, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.full((40, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    api.latent_norm_rope(q_out, rows_out=rows, **g)
    with pytest.raises(_lib.PagedAttentionError) as e:
        api.check_error()
    assert e.value.code == 6
    (yq, bq), (yr, br) = r.reference(False)
    live = ~np.isin(np.arange(40), [3, 9])
    mine = torch.as_tensor(live).cuda()
    check(q_out[mine], yq[live], bq[live])
    check(rows[mine], yr[live], br[live])
    assert (q_out[~mine] == 5.0).all() and (rows[~mine] == 5.0).all()
    want = r.pool.copy().reshape(-1, 320)
    kept = live & (r.slots < len(r.pool) * 16)
    want[r.slots[kept]] = back(rows)[kept]
    assert np.array_equal(back(g["pool"]).reshape(-1, 320), want)


@BOTH
def test_norm_rope_of_extreme_rows(dtype):
    """Rows of zeros (eps alone), of one large value, and of infinities in the shared part."""
    rng = np.random.default_rng(3)
    r = Rows(rng, dtype, 4, 2, 512, 16)
    r.latent[0] = 0
    r.latent[1] = 0
    r.latent[1, 7] = int4.narrow(3e4, dtype)
    g = r.gpu()
    rows = torch.empty(4, 576, dtype=TORCH[dtype], device="cuda")
    q_out = torch.empty(4, 2, 64, dtype=TORCH[dtype], device="cuda")
    api.latent_norm_rope(q_out, rows_out=rows, **g)
    api.check_error()
    (_, _), (yr, br) = r.reference(False)
    check(rows, yr, br)


# ------------------------------------------------------------------ read-back
@BOTH
@pytest.mark.parametrize("tokens,rank,block", [(0, 512, 16), (1, 256, 16), (57, 512, 64), (1025, 256, 32),
                                               (4099, 512, 16)])
def test_read(dtype, tokens, rank, block):
    rng = np.random.default_rng(tokens)
    pool = rng.integers(0, 1 << 16, (90, block, rank + 64)).astype(np.uint16)  # any bits
    slots = rng.integers(-1, 90 * block, tokens).astype(np.int64)  # some twice, some skipped
    out = torch.full((tokens, rank + 64), 5.0, dtype=TORCH[dtype], device="cuda")
    want = back(out)
    api.cache_read_latent(out, torch.as_tensor(slots).cuda(), dev(pool, dtype))
    api.check_error()
    want[slots >= 0] = pool.reshape(-1, rank + 64)[slots[slots >= 0]]
    assert np.array_equal(back(out), want)


def test_read_slots_past_the_pool():
    pool = torch.randn(4, 16, 320, device="cuda").half()
    out = torch.full((3, 320), 5.0, device="cuda", dtype=torch.float16)
    api.cache_read_latent(out, torch.tensor([1, 64, 1 << 50], device="cuda"), pool)
    with pytest.raises(_lib.PagedAttentionError):
        api.check_error()
    assert torch.equal(out[0], pool[0, 1]) and (out[1:] == 5.0).all()


# ------------------------------------------------------------------ decode
def run_decode(case, what="", **kw):
    ref, bound = case.reference()
    out = case.empty()
    api.decode_latent(out, **case.gpu(), **kw)
    api.check_error()
    check(out, ref, bound, what)
    return out


@BOTH
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("heads", [1, 7, 16, 17, 32, 40, 64, 65, 128, 130])
def test_decode_heads(dtype, rank, heads):
    run_decode(Decode(np.random.default_rng(heads), dtype, [70, 0, 1, 131], heads, rank, 16))


@BOTH
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("rank,heads", [(512, 16), (256, 64)])
def test_decode_lengths(dtype, block, rank, heads):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 191, 200, 256, 257, 300, 0]
    run_decode(Decode(np.random.default_rng(block), dtype, lens, heads, rank, block))


@BOTH
@pytest.mark.parametrize("rank,heads", [(512, 128), (512, 3), (256, 33)])
def test_decode_one_long(dtype, rank, heads):
    run_decode(Decode(np.random.default_rng(5), dtype, [20011], heads, rank, 32))


@pytest.mark.parametrize("heads", [5, 64, 100])
def test_decode_ragged_batch(heads):
    rng = np.random.default_rng(8)
    lens = np.clip(np.round(rng.lognormal(4.5, 1.2, 60)), 0, 3000).astype(int)
    lens[[4, 50]] = 0
    run_decode(Decode(rng, "bf16", lens, heads, 512, 16))


def test_decode_many_sequences():
    rng = np.random.default_rng(9)
    run_decode(Decode(rng, "f16", rng.integers(0, 40, 700), 4, 256, 16))


@BOTH
def test_decode_sharp_scores(dtype):
    """Large queries: softmax near one position, running maxima that jump from tile to tile."""
    run_decode(Decode(np.random.default_rng(10), dtype, [900, 65, 1], 20, 512, 16, size=12.0))


def test_decode_rising_scores():
    """Scores that grow along the sequence: the running maximum moves in every tile."""
    case = Decode(np.random.default_rng(11), "bf16", [1500], 30, 256, 16, poison=False)
    q = np.zeros((1, 30, 320))
    q[..., 256] = 1.0
    case.q = int4.narrow(q, "bf16")
    for p in range(1500):
        case.pool[case.tables[0, p // 16], p % 16, 256] = int4.narrow(p * 3.0, "bf16")
    run_decode(case)
    for p in range(1500):  # and that fall
        case.pool[case.tables[0, p // 16], p % 16, 256] = int4.narrow(-p * 3.0, "bf16")
    run_decode(case)


def test_decode_f16_small_weights():
    """One position far above many others whose weights together count."""
    case = Decode(np.random.default_rng(12), "f16", [30000], 2, 256, 64, poison=False)
    q = np.zeros((1, 2, 320))
    q[..., 256] = 1.0
    case.q, case.scale = int4.narrow(q, "f16"), 1.0
    case.pool[:] = 0
    case.pool[..., :256] = int4.narrow(1.0, "f16")
    case.pool[case.tables[0, 3], 5, 256] = int4.narrow(13.0, "f16")
    case.pool[case.tables[0, 3], 5, :256] = int4.narrow(-1.0, "f16")
    run_decode(case)


def test_decode_equal_scores_give_the_mean():
    case = Decode(np.random.default_rng(13), "bf16", [333], 16, 512, 16)
    case.q[:] = 0
    run_decode(case)


def test_decode_minus_infinite_key():
    """A key of -inf in a live position has no weight."""
    case = Decode(np.random.default_rng(14), "f16", [100], 16, 256, 16)
    case.q[..., 256:] = int4.narrow(1.0, "f16")
    case.pool[case.tables[0, 2], 3, 300] = 0xFC00
    live = int4.widen(case.q, "f16")
    assert (live[..., 300] > 0).all()
    out = case.empty()
    api.decode_latent(out, **case.gpu())
    api.check_error()
    assert torch.isfinite(out).all()
    case.pool[case.tables[0, 2], 3, 300] = int4.narrow(-60000.0, "f16")
    ref, bound = case.reference()
    check(out, ref, bound)


@BOTH
@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-20])
def test_attention_of_unusual_scales(dtype, scale):
    """No scale (the mean of the values) and negative ones, masked positions among the tiles."""
    case = Decode(np.random.default_rng(19), dtype, [77, 200, 64], 20, 256, 16)
    case.scale = scale
    run_decode(case)
    case = Prefill(np.random.default_rng(20), dtype, [150, 7], [200, 7], 2, True)
    case.scale = scale
    run_prefill(case)


def test_decode_more_heads_than_two_groups():
    run_decode(Decode(np.random.default_rng(21), "bf16", [300, 5, 0, 64], 300, 256, 32))


def test_decode_rows_far_into_a_large_pool():
    """Rows whose elements lie past 2^32 (written, read back and attended)."""
    rng = np.random.default_rng(22)
    case = Decode(rng, "bf16", [150, 40], 3, 512, 64, poison=False, spare=0)
    blocks = (1 << 32) // (64 * 576) + 20
    pool = torch.empty(blocks, 64, 576, dtype=torch.bfloat16, device="cuda")
    far = blocks - len(case.pool)
    pool[far:] = dev(case.pool, "bf16")
    g = case.gpu()
    g["block_tables"] = g["block_tables"] + far
    ref, bound = case.reference()
    out = case.empty()
    api.decode_latent(out, **{**g, "pool": pool})
    api.check_error()
    check(out, ref, bound)
    slots = torch.tensor([blocks * 64 - 1, 5, far * 64 + 3], device="cuda")
    rows = torch.empty(3, 576, dtype=torch.bfloat16, device="cuda")
    r = Rows(rng, "bf16", 3, 2, 512, 64).gpu()
    api.latent_norm_rope(torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda"),
                         **{**r, "pool": pool, "slot_mapping": slots}, rows_out=rows)
    again = torch.empty_like(rows)
    api.cache_read_latent(again, slots, pool)
    api.check_error()
    assert torch.equal(rows, again)


def test_decode_a_head_of_nan_stays_alone():
    """A query head of NaN spoils its own outputs only."""
    case = Decode(np.random.default_rng(23), "bf16", [500, 70], 9, 256, 16)
    ref, bound = case.reference()
    g, out = case.gpu(), case.empty()
    g["q"][0, 4] = float("nan")
    api.decode_latent(out, **g)
    api.check_error()
    assert torch.isnan(out[0, 4]).all()
    rest = [h for h in range(9) if h != 4]
    check(out[0, rest], ref[0, rest], bound[0, rest])
    check(out[1], ref[1], bound[1])


def test_decode_thousands_of_sequences():
    rng = np.random.default_rng(25)
    lens = rng.integers(0, 3, 5000)
    lens[[0, 17, 4999]] = [700, 300, 129]
    run_decode(Decode(rng, "bf16", lens, 2, 256, 16))


def test_attention_of_large_values():
    """Values near the largest whose sums fp32 is said to hold (2^119 over the keys)."""
    case = Decode(np.random.default_rng(26), "bf16", [500, 60], 5, 256, 16, poison=False)
    size = 2.0 ** (119 - 9 - 2)
    wide = int4.widen(case.pool, "bf16")
    wide[..., :256] *= size
    case.pool = int4.narrow(wide, "bf16")
    wide = int4.widen(case.q, "bf16")
    wide[..., :256] /= size
    case.q = int4.narrow(wide, "bf16")
    run_decode(case)
    case = Prefill(np.random.default_rng(27), "bf16", [300], [500], 2, True)
    wide = int4.widen(case.kv, "bf16")
    wide[..., 128:] *= size
    case.kv = int4.narrow(wide, "bf16")
    run_prefill(case)


def test_decode_shared_and_repeated_blocks():
    """Sequences that share blocks, and one that names a block twice."""
    case = Decode(np.random.default_rng(24), "f16", [160, 96, 64], 6, 512, 32, poison=False)
    case.tables[1, :2] = case.tables[0, :2]
    case.tables[2, 1] = case.tables[2, 0]
    run_decode(case)


def test_decode_empty_batches():
    g = Decode(np.random.default_rng(15), "bf16", [3, 5], 8, 256, 16).gpu()
    out = torch.full((2, 8, 256), 5.0, device="cuda", dtype=torch.bfloat16)
    g["seq_lens"].zero_()
    api.decode_latent(out, **g)
    assert (out == 0).all()
    api.decode_latent(out, **{**g, "max_seq_len": 0})
    assert (out == 0).all()
    api.decode_latent(out[:0], **{**g, "q": g["q"][:0], "block_tables": g["block_tables"][:0],
                                  "seq_lens": g["seq_lens"][:0]})
    api.check_error()


def test_decode_bad_indexes():
    case = Decode(np.random.default_rng(16), "bf16", [100, 50, 70], 8, 256, 16)
    ref, bound = case.reference()
    for what, i in (("table", 1), ("table", 1), ("long", 2), ("negative", 0)):
        out = case.empty()
        g = case.gpu()
        if what == "table":
            g["block_tables"][1, 2] = 1 << 30
        else:
            g["seq_lens"][i] = 1 << 20 if what == "long" else -4
        api.decode_latent(out, **g)
        with pytest.raises(_lib.PagedAttentionError) as e:
            api.check_error()
        assert e.value.code == 6
        rest = [s for s in range(3) if s != i]
        check(out[rest], ref[rest], bound[rest])
        if what == "negative":
            assert (out[i] == 0).all()


def test_decode_workspace_and_determinism():
    rng = np.random.default_rng(17)
    case = Decode(rng, "bf16", [5000, 17, 2500], 64, 512, 16)
    ref, bound = case.reference()
    g, out = case.gpu(), case.empty()
    ws = api.decode_latent(out, **g)
    need = api.latent_workspace_size(3, 64, 512, 16, case.max_len, torch.bfloat16)
    assert (ws is None) == (need == 0)
    check(out, ref, bound)
    for fill in (0, 255):
        again = case.empty()
        if ws is not None:
            ws.fill_(fill)
        assert api.decode_latent(again, **g, workspace=ws) is ws
        assert torch.equal(out, again)
    if ws is not None:
        with pytest.raises(_lib.PagedAttentionError):
            _lib.check("x", _lib.load().pa_decode_latent(
                out.data_ptr(), g["q"].data_ptr(), g["pool"].data_ptr(), g["pool"].shape[0],
                g["block_tables"].data_ptr(), g["block_tables"].shape[1], g["seq_lens"].data_ptr(),
                case.max_len, 3, 64, 512, 16, 0.1, ws.data_ptr(), need - 1, 1, 0))


def test_decode_on_streams_and_in_graphs():
    """A captured call replayed under other lengths, beside an eager one on another stream."""
    rng = np.random.default_rng(18)
    a, b = Decode(rng, "bf16", [700, 3000, 1], 40, 512, 16), Decode(rng, "bf16", [90] * 30, 40, 512, 16)
    ga, gb, oa, ob = a.gpu(), b.gpu(), a.empty(), b.empty()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        wa = api.decode_latent(oa, **ga)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decode_latent(oa, **ga, workspace=wa)
    for lens in ([700, 3000, 1], [0, 64, 0], [1, 2999, 1]):
        a.lens[:] = lens
        ga["seq_lens"].copy_(torch.as_tensor(a.lens))
        oa.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        api.decode_latent(ob, **gb, stream=side)
        torch.cuda.synchronize()
        api.check_error()
        ref, bound = a.reference()
        check(oa, ref, bound)
        ref, bound = b.reference()
        check(ob, ref, bound)


def test_two_graphs_share_a_workspace():
    """Graphs of batches that are cut and that are not, replayed in turn over one workspace."""
    rng = np.random.default_rng(28)
    cases = [Decode(rng, "bf16", [2500, 300], 33, 256, 16), Decode(rng, "bf16", [400, 390], 33, 256, 16)]
    gs, outs = [c.gpu() for c in cases], [c.empty() for c in cases]
    ws = api.alloc_workspace(max(api.latent_workspace_size(2, 33, 256, 16, c.max_len, torch.bfloat16)
                                 for c in cases), "cuda")
    graphs = []
    for g, out in zip(gs, outs):
        api.decode_latent(out, **g, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            api.decode_latent(out, **g, workspace=ws)
    for _ in range(3):
        for out in outs:
            out.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        api.check_error()
        for c, out in zip(cases, outs):
            ref, bound = c.reference()
            check(out, ref, bound)


def test_a_step_on_another_stream():
    """Rows written, read back and attended on a stream that is not the current one, in order."""
    rng = np.random.default_rng(29)
    case = Decode(rng, "f16", [200, 65], 10, 512, 32, poison=False)
    g, out, side = case.gpu(), case.empty(), torch.cuda.Stream()
    r = Rows(rng, "f16", 2, 10, 512, 32)
    last = [int(case.tables[i, (n - 1) // 32]) * 32 + (n - 1) % 32 for i, n in enumerate(case.lens.tolist())]
    rows, back_rows = (torch.zeros(2, 576, dtype=torch.float16, device="cuda") for _ in range(2))
    slots, args = torch.tensor(last, device="cuda"), r.gpu()
    torch.cuda.synchronize()
    api.latent_norm_rope(g["q"][..., 512:], **{**args, "pool": g["pool"], "slot_mapping": slots},
                         rows_out=rows, stream=side)
    api.cache_read_latent(back_rows, slots, g["pool"], stream=side)
    api.decode_latent(out, **g, stream=side)
    side.synchronize()
    api.check_error(side)
    assert torch.equal(rows, back_rows)
    case.pool, case.q = back(g["pool"]), back(g["q"])
    ref, bound = case.reference()
    check(out, ref, bound)


# ------------------------------------------------------------------ prompts
def run_prefill(case, what=""):
    out = case.empty()
    api.prefill_latent(out, **case.gpu())
    api.check_error()
    case.check(out, what)
    return out


@BOTH
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 3, 16])
def test_prefill_ragged(dtype, causal, heads):
    n = [1, 0, 63, 64, 65, 127, 128, 129, 2, 255, 257]
    run_prefill(Prefill(np.random.default_rng(heads), dtype, n, n, heads, causal))


@BOTH
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_behind_a_context(dtype, causal):
    n_q = np.array([1, 5, 128, 200, 300, 0, 7])
    run_prefill(Prefill(np.random.default_rng(3), dtype, n_q, n_q + [100, 0, 77, 1, 129, 50, 640], 4, causal))


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_queries_without_keys(causal):
    """Fewer keys than queries (the first queries meet none), and none at all."""
    run_prefill(Prefill(np.random.default_rng(4), "bf16", [10, 200, 300, 5], [3, 70, 0, 5], 2, causal))


@BOTH
@pytest.mark.parametrize("size", [0.0, 12.0])
def test_prefill_flat_and_sharp_scores(dtype, size):
    run_prefill(Prefill(np.random.default_rng(5), dtype, [400, 130], [400, 500], 2, True, size=size))


def test_prefill_long():
    run_prefill(Prefill(np.random.default_rng(6), "bf16", [700, 1], [5003, 4097], 2, True))


def test_prefill_dense_and_empty_arguments():
    case = Prefill(np.random.default_rng(7), "f16", [50, 60], [50, 60], 3, True, gap=0)
    g = case.gpu()
    out = case.empty()
    dense = {n: g[n].contiguous() for n in ("q", "k", "v", "k_pe")}
    api.prefill_latent(out, **{**g, **dense})
    case.check(out)
    again = case.empty()
    api.prefill_latent(again, **g)
    assert torch.equal(out, again)
    # heads first in memory: a head's tokens lie together
    swapped = {n: g[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v")}
    again = case.empty()
    api.prefill_latent(again, **{**g, **swapped})
    assert torch.equal(out, again)
    starts = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 3, 128, dtype=torch.float16, device="cuda")
    out.fill_(7.0)
    api.prefill_latent(out, **{**g, "k": none, "v": none, "k_pe": none[:, 0, :64], "k_starts": starts})
    assert (out == 0).all()
    api.prefill_latent(out[:0], **{**g, "q": g["q"][:0], "q_starts": starts, "max_q_len": 0})
    api.check_error()


def test_prefill_bad_starts():
    case = Prefill(np.random.default_rng(8), "bf16", [40, 50, 60], [40, 50, 60], 2, True)
    ref, bound = case.reference()
    s = case.q_starts
    for name, at, value in (("q_starts", 3, 1 << 20), ("k_starts", 3, 1 << 20), ("q_starts", 0, -5),
                            ("k_starts", 0, 200)):
        g, out = case.gpu(), case.empty()
        g[name][at] = value
        api.prefill_latent(out, **g)
        with pytest.raises(_lib.PagedAttentionError) as e:
            api.check_error()
        assert e.value.code == 6
        lost = 2 if at == 3 else 0
        for i in range(3):
            part = slice(int(s[i]), int(s[i + 1]))
            if i == lost:
                assert (out[part] == 7.0).all()
            else:
                check(out[part], ref[part], bound[part])
    g, out = case.gpu(), case.empty()
    api.prefill_latent(out, **{**g, "max_q_len": 55})
    with pytest.raises(_lib.PagedAttentionError):
        api.check_error()
    assert (out[int(s[2]):] == 7.0).all()
    check(out[int(s[0]):int(s[2])], ref[s[0]:s[2]], bound[s[0]:s[2]])


@BOTH
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n_q,n_k,heads", [
    ([1], [3000], 3), ([200, 0, 37], [2500, 2600, 2700], 5), ([300, 129], [1100, 1500], 20),
    ([600], [400], 4), ([1, 1, 1], [5000, 0, 130], 2), ([700], [1200], 30)])
def test_prefill_keys_shared_out(dtype, causal, n_q, n_k, heads):
    """Few pieces of work with many keys: two to eight CTAs share the keys of one, some with none."""
    run_prefill(Prefill(np.random.default_rng(heads), dtype, n_q, n_k, heads, causal))


def test_prefill_keys_shared_out_of_bad_starts():
    case = Prefill(np.random.default_rng(13), "bf16", [40, 50], [3000, 2000], 2, True)
    ref, bound = case.reference()
    g, out = case.gpu(), case.empty()
    g["k_starts"][0] = 1 << 20
    api.prefill_latent(out, **g)
    with pytest.raises(_lib.PagedAttentionError):
        api.check_error()
    a, b = int(case.q_starts[1]), int(case.q_starts[2])
    assert (out[:a] == 7.0).all()
    check(out[a:b], ref[a:b], bound[a:b])


def test_prefill_many_short_prompts():
    rng = np.random.default_rng(10)
    n_q = rng.integers(0, 4, 3000)
    run_prefill(Prefill(rng, "bf16", n_q, n_q + rng.integers(0, 3, 3000), 2, True))


def test_prefill_output_off_a_32_byte_boundary():
    case = Prefill(np.random.default_rng(11), "bf16", [300], [300], 3, True)
    n = case.empty().numel()
    out = torch.full((n + 8,), 7.0, dtype=torch.bfloat16, device="cuda")[8:].view(-1, 3, 128)
    assert out.data_ptr() % 32 == 16
    api.prefill_latent(out, **case.gpu())
    api.check_error()
    case.check(out)


@pytest.mark.parametrize("heads,n_q,n_k", [(70, 300, 6100), (1, 9000, 9000)])
def test_prefill_orders_of_work(heads, n_q, n_k):
    """More (key, head) pairs than the order by length takes; more queries than one wave."""
    rng = np.random.default_rng(heads)
    case = Prefill(rng, "bf16", [n_q], [n_k], heads, True)
    out = case.empty()
    api.prefill_latent(out, **case.gpu())
    api.check_error()
    pick = np.unique(np.concatenate([rng.integers(0, n_q, 40), [0, n_q - 1]]))
    for h in (0, heads - 1):  # some rows of two heads
        for i in pick:
            last = n_k - n_q + i + 1
            a, b = int(case.q_starts[0] + i), int(case.k_starts[0])
            ref, size, terms = latent.prefill(
                case.q[a:a + 1, h:h + 1], case.kv[b:b + last, h:h + 1, :128],
                case.kv[b:b + last, h:h + 1, 128:], case.rows[b:b + last, 256:], np.array([0, 1]),
                np.array([0, last]), case.scale, True, "bf16")
            check(out[a:a + 1, h:h + 1], ref, attention_bound(ref, size, terms, "bf16", last, 192, 0.0))


def test_prefill_on_two_streams_at_once():
    cases = [Prefill(np.random.default_rng(12 + i), "f16", [500, 40 + i], [700, 90], 4, True)
             for i in range(2)]
    gs, outs = [c.gpu() for c in cases], [c.empty() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for g, out, stream in zip(gs, outs, streams):
            api.prefill_latent(out, **g, stream=stream)
    torch.cuda.synchronize()
    api.check_error()
    for c, out in zip(cases, outs):
        c.check(out)


def test_prefill_in_a_graph():
    case = Prefill(np.random.default_rng(9), "bf16", [300, 20], [300, 90], 4, True)
    g, out = case.gpu(), case.empty()
    api.prefill_latent(out, **g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.prefill_latent(out, **g)
    for _ in range(2):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        case.check(out)


# ------------------------------------------------------------------ all together
@BOTH
def test_a_sequence_through_all_of_them(dtype):
    """A prompt of two pieces and three decoded tokens: rows written by
    latent_norm_rope, the first piece's read back for the second, prompts attended
    in the expanded form, new tokens in the absorbed one; each against fp64
    attention over the rows that the cache holds."""
    rng = np.random.default_rng(20)
    heads, rank, block, n1, n2, n3 = 6, 256, 16, 45, 30, 3
    total, t = n1 + n2 + n3, TORCH[dtype]
    x = bits16(rng, total, rank + 64, dtype=dtype)
    q = dev(bits16(rng, total, heads, 192, dtype=dtype), dtype)
    weight = dev(bits16(rng, rank, dtype=dtype), dtype)
    up = torch.from_numpy(rng.standard_normal((rank, heads, 256)) / 16).cuda()  # fp64
    cs, lat = torch.as_tensor(table(100)).cuda(), dev(x, dtype)
    alloc = api.BlockAllocator(9, block, rng.permutation(9))
    alloc.add(1)
    slots = torch.tensor(alloc.append(1, total)[0], device="cuda")
    tables, _ = alloc.export([1], 6)
    pool = torch.full((9, block, rank + 64), float("nan"), dtype=t, device="cuda")
    positions = torch.arange(total, device="cuda")
    scale = 192 ** -0.5

    def rows_of(a, b):
        rows = torch.empty(b - a, rank + 64, dtype=t, device="cuda")
        api.latent_norm_rope(q[a:b, :, 128:], q[a:b, :, 128:], lat[a:b], weight, 1e-6, cs, positions[a:b],
                             slots[a:b], pool, rows_out=rows)
        return rows

    def want(a, b, up_k, up_v):
        """fp64 attention of queries a .. b over the cache, with its bound's sizes."""
        seen = torch.as_tensor(int4.widen(back(pool), dtype)).cuda().view(-1, rank + 64)[slots[:b]]
        keys = torch.cat([torch.einsum("tr,rhd->thd", seen[:, :rank], up_k),
                          seen[:, None, rank:].expand(-1, heads, -1)], 2)
        values = torch.einsum("tr,rhd->thd", seen[:, :rank], up_v)
        s = torch.einsum("qhd,khd->hqk", q[a:b].double(), keys) * scale
        terms = torch.einsum("qhd,khd->hqk", q[a:b].double().abs(), keys.abs()) * scale
        hidden = torch.arange(b, device="cuda")[None, :] > torch.arange(a, b, device="cuda")[:, None]
        w = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
        return (torch.einsum("hqk,khd->qhd", w, values), torch.einsum("hqk,khd->qhd", w, values.abs()),
                terms.amax(-1).T)

    # keys and values as the 16-bit products that the prompts' attention is given
    def expanded(rows):
        return torch.einsum("tr,rhd->thd", rows[:, :rank].double(), up).to(t)

    first = rows_of(0, n1)
    out = torch.empty(n1, heads, 128, dtype=t, device="cuda")
    kv = expanded(first)
    starts = torch.tensor([0, n1], dtype=torch.int32, device="cuda")
    api.prefill_latent(out, q[:n1], kv[..., :128], kv[..., 128:], first[:, rank:], starts, starts, n1, scale)
    second = rows_of(n1, n1 + n2)
    cached = torch.empty(n1, rank + 64, dtype=t, device="cuda")
    api.cache_read_latent(cached, slots[:n1], pool)
    assert torch.equal(cached, first)
    rows = torch.cat([cached, second])
    kv = expanded(rows)
    out2 = torch.empty(n2, heads, 128, dtype=t, device="cuda")
    api.prefill_latent(out2, q[n1:n1 + n2], kv[..., :128], kv[..., 128:], rows[:, rank:],
                       torch.tensor([0, n2], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, n1 + n2], dtype=torch.int32, device="cuda"), n2, scale)
    u = UNIT[dtype]
    for got, a, b in ((out, 0, n1), (out2, n1, n1 + n2)):
        ref, size, terms = (v.cpu().numpy() for v in want(a, b, up[..., :128], up[..., 128:]))
        # beside the kernel's own: keys and values rounded once each, so scores off by
        # u of their terms and values by u of theirs
        bound = attention_bound(ref, size, terms, dtype, total, 192, 20.0)
        bound += u * size + 2 * u * terms[..., None] * (size + abs(ref))
        check(got, ref, bound)
    ws = None
    for i in range(n1 + n2, total):
        rows_of(i, i + 1)
        absorbed = torch.cat([torch.einsum("hd,rhd->hr", q[i, :, :128].double(), up[..., :128]).to(t),
                              q[i, :, 128:]], -1)[None].contiguous()
        mixed = torch.empty(1, heads, rank, dtype=t, device="cuda")
        ws = api.decode_latent(mixed, absorbed, pool, torch.as_tensor(tables).cuda(),
                               torch.tensor([i + 1], dtype=torch.int32, device="cuda"), i + 1, scale,
                               workspace=ws)
        ref, size, terms = latent.decode(back(absorbed), back(pool), tables, np.array([i + 1]), scale, dtype)
        check(mixed, ref, attention_bound(ref, size, terms, dtype, total, rank + 64, 20.0))
        # and the expanded form's result: the absorbed queries and the mixture rounded once
        got = torch.einsum("hr,rhd->hd", mixed[0].double(), up[..., 128:]).cpu().numpy()
        far = want(i, i + 1, up[..., :128], up[..., 128:])[0][0].cpu().numpy()
        weights = torch.einsum("hr,rhd->hd", torch.as_tensor(size[0]).cuda(), up[..., 128:].abs()).cpu().numpy()
        e = 2 * (2 * u * terms[0][:, None] + 2.0 ** -12)
        assert (abs(got - far) <= (2 * u + e) * 2 * weights).all()
    api.check_error()
