"""GPU parity of the 4-bit KV cache against the fp64 oracle: the quantising
write and the read-back bit for bit.

The format is exact by construction (fp32 differences, exact quotients), so
codes, scales, minima and read-back values are compared as bits."""
import numpy as np
import pytest
import torch

from oracle import int4
from paged_kv_cache_64_gb300 import api, workloads

from _parity import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_errors():
    assert torch.cuda.is_available()
    yield
    api.check_error()


def as_bits(values, dtype):
    return int4.narrow(values, dtype)


def to_gpu(b, dtype):
    t = torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).to("cuda")
    return t.view(workloads.torch_dtype(dtype))


def rows_of_every_kind(T, H, d, dtype, seed):
    """Bits [T, H, d]: ordinary rows, offset ones, tiny and huge ones, ties,
    equal values, non-finite ones."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, d))
    scale = [1e-7, 1e-4, 1.0, 50.0, 1.5e4] if dtype == "f16" else [1e-40, 1e-36, 1e-3, 1.0, 1e30]
    x *= rng.choice(scale, (T, H, 1))
    x += rng.choice([0.0, 0.0, 3.0, -40.0], (T, H, 1))
    kinds = rng.integers(0, 12, (T, H))
    x[kinds == 0] = rng.integers(-8, 8, (int((kinds == 0).sum()), d)) / 2    # ties
    x[kinds == 1] = rng.integers(0, 31, (int((kinds == 1).sum()), d)) * 3.0  # ties, s = 6
    x[kinds == 2] = rng.choice([-0.0, 0.0, 7.25, -1e-3], (int((kinds == 2).sum()), 1))
    big = int4.LARGEST[dtype]
    some = np.argwhere(kinds == 3)
    for t, h in some:  # the whole range next to the smallest values
        x[t, h, ::5] = rng.choice([big, -big, 2.0**-24, -(2.0**-20), 0.0], len(x[t, h, ::5]))
    for n, (t, h) in enumerate(np.argwhere(kinds == 4)):
        x[t, h, rng.integers(d)] = [np.nan, np.inf, -np.inf][n % 3]
    return as_bits(x, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block,hkv", [(16, 2), (32, 3), (16, 1)])
def test_write_and_read_bit_exact(dtype, d, block, hkv):
    T, nb = 301, 37 if block == 16 else 19
    rng = np.random.default_rng(d + block + hkv)
    k = rows_of_every_kind(T, hkv, d, dtype, 1 + hkv)
    v = rows_of_every_kind(T, hkv, d, dtype, 2 + hkv)
    slots = rng.permutation(nb * block)[:T].astype(np.int64)
    slots[[3, 100]] = [-1, -7]  # skipped
    shape = api.int4_pool_shape(nb, hkv, block, d)
    kp = torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda")
    vp = torch.full(shape, 0x5A, dtype=torch.uint8, device="cuda")
    rk, rv = kp.cpu().numpy(), vp.cpu().numpy()
    gk, gv, gs = to_gpu(k, dtype), to_gpu(v, dtype), torch.as_tensor(slots, device="cuda")
    api.cache_write_int4(gk, gv, gs, kp, vp)
    int4.cache_write([rk, rv], [k, v], slots, block, dtype)
    assert np.array_equal(kp.cpu().numpy(), rk)
    assert np.array_equal(vp.cpu().numpy(), rv)

    # the values, by the write itself and by a read of a permutation with
    # repeats; skipped rows stay as they were
    ko, vo = torch.full_like(gk, 7.5), torch.full_like(gv, 7.5)
    api.cache_write_int4(gk, gv, gs, kp, vp, k_out=ko, v_out=vo)
    assert np.array_equal(kp.cpu().numpy(), rk)
    order = rng.integers(0, T, 2 * T)
    ro, wo = torch.full((2 * T, hkv, d), 7.5, dtype=gk.dtype, device="cuda"), None
    wo = ro.clone()
    api.cache_read_int4(ro, wo, gs[torch.as_tensor(order, device="cuda")], kp, vp)
    for pool, out, got in ((rk, ko, ro), (rv, vo, wo)):
        keep = slots >= 0
        want = np.full((T, hkv, d), as_bits(7.5, dtype)[()], np.uint16)
        want[keep] = int4.cache_read(pool, slots[keep], d, block, dtype)
        nan = np.isnan(int4.widen(want, dtype))
        o, g = bits(out), bits(got)
        assert np.array_equal(np.isnan(int4.widen(o, dtype)), nan)
        assert np.array_equal(o[~nan], want[~nan])
        assert np.array_equal(np.isnan(int4.widen(g, dtype)), nan[order])
        assert np.array_equal(g[~nan[order]], want[order][~nan[order]])

    # in place: the values over the new tokens
    api.cache_write_int4(gk, gv, gs, kp, vp, k_out=gk, v_out=gv)
    keep = torch.as_tensor(slots >= 0, device="cuda")
    assert torch.equal(gk[keep].view(torch.int16), ko[keep].view(torch.int16))
    assert torch.equal(gv[~keep].view(torch.int16).cpu(),
                       torch.from_numpy(v.view(np.int16))[~keep.cpu()])
    assert np.array_equal(kp.cpu().numpy(), rk)


@pytest.mark.parametrize("T", [1, 2, 15, 5000])
def test_write_and_read_of_any_count(T):
    hkv, d, block, dtype = 8, 128, 16, "bf16"
    nb = -(-T // block) + 2
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    k = torch.randn(T, hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(T, hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(nb * block, generator=g, device="cuda")[:T]
    kp = torch.zeros(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    api.cache_write_int4(k, v, slots, kp, vp)
    api.cache_read_int4(ko, vo, slots, kp, vp)
    n = min(T, 40)
    for x, o in ((k, ko), (v, vo)):
        codes, s, m = int4.quantise(bits(x[-n:]), dtype)
        want = int4.widen(m, dtype)[..., None] + int4.widen(s, dtype)[..., None] * codes
        assert np.array_equal(bits(o[-n:]), int4.narrow(want.astype(np.float32), dtype))
        # half a step, and half a bf16 step of the largest value
        step = (x.amax(-1, keepdim=True).double() - x.amin(-1, keepdim=True).double()) / 15
        assert ((o.double() - x.double()).abs() <= step * 0.5 * (1 + 2.0**-7)
                + 2.0**-8 * x.abs().amax(-1, keepdim=True).double()).all()


def test_bad_slots_are_recorded_and_skipped():
    hkv, d, block, nb = 2, 64, 16, 4
    k = torch.ones(3, hkv, d, dtype=torch.float16, device="cuda")
    slots = torch.tensor([5, nb * block, 1 << 40], device="cuda")
    pools = [torch.zeros(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    api.cache_write_int4(k, k, slots, *pools)
    with pytest.raises(Exception, match="PA_ERR_BAD_INDEX"):
        api.check_error()
    api.check_error()
    ko, vo = torch.full_like(k, 9.0), torch.full_like(k, 9.0)
    api.cache_read_int4(ko, vo, slots, *pools)
    with pytest.raises(Exception, match="PA_ERR_BAD_INDEX"):
        api.check_error()
    assert (ko[0] == 1).all() and (vo[0] == 1).all()
    assert (ko[1:] == 9).all() and (vo[1:] == 9).all()


def test_copied_blocks_read_the_same():
    """Copy-on-write over 4-bit pools: pa_copy_blocks moves whole records."""
    hkv, d, block, nb = 2, 128, 16, 6
    k = torch.randn(block, hkv, d, device="cuda").to(torch.float16)
    slots = torch.arange(block, device="cuda") + 2 * block
    pools = [torch.zeros(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    api.cache_write_int4(k, 2 * k, slots, *pools)
    api.copy_blocks([pools[0]], [pools[1]], torch.tensor([[2, 5]], device="cuda"))
    a, b, c, e = (torch.empty_like(k) for _ in range(4))
    api.cache_read_int4(a, b, slots, *pools)
    api.cache_read_int4(c, e, slots + 3 * block, *pools)
    assert torch.equal(a, c) and torch.equal(b, e)


def test_captured_and_replayed():
    """A write and a read in one CUDA graph, replayed over new inputs."""
    hkv, d, block, nb = 2, 64, 16, 8
    k = torch.randn(50, hkv, d, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(nb * block, device="cuda")[:50]
    pools = [torch.zeros(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.cache_write_int4(k, k, slots, *pools)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_write_int4(k, k, slots, *pools)
        api.cache_read_int4(ko, vo, slots, *pools)
    for seed in range(3):
        k.copy_(torch.randn(50, hkv, d, device="cuda"))
        graph.replay()
        a, b = torch.empty_like(k), torch.empty_like(k)
        fresh = [torch.zeros_like(p) for p in pools]
        api.cache_write_int4(k, k, slots, *fresh, k_out=a, v_out=b)
        assert torch.equal(ko, a) and torch.equal(vo, b)


@pytest.mark.parametrize("hkv", [5, 7, 12, 31, 33, 100])
def test_every_row_finds_its_token(hkv):
    """Row to token and head for head counts that are no power of two."""
    T, d, block = 67, 64, 16
    nb = -(-T // block) + 1
    k = torch.arange(T * hkv, device="cuda").view(T, hkv, 1).expand(T, hkv, d)
    k = (k % 2048).to(torch.float16).contiguous()  # rows of one value each: exact
    v = (k + 1).contiguous()
    slots = torch.randperm(nb * block, device="cuda")[:T]
    pools = [torch.zeros(api.int4_pool_shape(nb, hkv, block, d), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    api.cache_write_int4(k, v, slots, *pools)
    rows = [int4.values(p.cpu().numpy(), d, block, "f16") for p in pools]
    at = slots.cpu().numpy()
    for got, want in zip(rows, (k, v)):
        assert np.array_equal(got[at // block, :, at % block], want.double().cpu().numpy())
    a, b = torch.empty_like(k), torch.empty_like(v)
    api.cache_read_int4(a, b, slots, *pools)
    assert torch.equal(a, k) and torch.equal(b, v)
