"""The ways through 4-bit decode and the norm-rope write that other tests do not
reach: automatic chunks, balanced ranges over many heads, coded pools under every
rotation.  Each decode test first asserts, by the workspace, which way it takes."""
import numpy as np
import pytest
import torch

from paged_kv_cache_64_gb300 import api

from test_gpu_decode_int4 import Case
from test_gpu_norm_rope import Inputs, gathered

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_errors():
    assert torch.cuda.is_available()
    yield
    api.check_error()


def workspace(c, partition=0):
    S, hq, d = c.gq.shape
    return api.int4_workspace_size(S, hq, c.gk.shape[1], d, c.block, c.max_len, partition, c.gq.dtype)


@pytest.mark.parametrize("longest", [4097, 9000, 40000])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "f16")])
def test_automatic_chunks_of_more_than_1024_sequences(longest, d, dtype):
    lens = [3, 0, 17, 1, 40] * 210
    lens[7], lens[300], lens[1000], lens[1049] = longest, 4096, 8192, 4097
    lens = [min(x, longest) for x in lens]
    c = Case(lens, 1, 4, d, 16, dtype, seed=longest)
    assert workspace(c) > 0
    c.check(c.gpu(0))


@pytest.mark.parametrize("lens,hkv,group,d", [
    ([2300] * 40, 2, 4, 64), ([2049, 2300, 2177] * 22, 2, 3, 64), ([1500] * 40, 2, 6, 128),
    ([1100, 1025, 0, 1281] * 15, 2, 8, 128), ([2049] + [2048] * 17, 8, 5, 128)])
def test_balanced_ranges_over_many_heads(lens, hkv, group, d):
    """Heads of a few units each, cut next to the slack; with more heads than an
    eighth of the CTAs (at most four an SM) the partials are merged by bounds."""
    c = Case(lens, hkv, group, d, 16, "bf16", seed=group)
    assert workspace(c) > 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert 8 * len(lens) * hkv > 4 * sms
    out = c.gpu(0)
    c.check(out)
    for _ in range(3):
        assert torch.equal(c.gpu(0).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 32), (64, 48), (128, 128), (128, 16),
                                   (128, 64), (128, 80), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_coded_pools_under_every_rotation(fmt, dtype, d, rot, interleaved):
    """Queries against the oracle; keys' and values' codes byte for byte those that
    cache_write_fp8 / cache_write_int4 give for the 16-bit pool's."""
    block = 16 if d == 64 else 32
    x = Inputs(39, 14, 2, d, block, dtype, rot, seed=rot, skip=(0, 5))
    wide, pools, want = x.pools("16"), x.pools(fmt), x.pools(fmt)
    kw = dict(k_scale=0.05, v_scale=0.7) if fmt == "e4m3" else {}
    q = x.run(pools, interleaved, **kw)
    x.check(q, x.q, x.qw, interleaved)
    assert torch.equal(q, x.run(wide, interleaved))
    keep = torch.as_tensor(x.slots >= 0, device="cuda")
    k16 = gathered(wide[0], np.maximum(x.slots, 0), block).contiguous()
    if fmt == "e4m3":
        api.cache_write_fp8(k16, x.gv.contiguous(), x.gslots, *want, 0.05, 0.7)
    else:
        api.cache_write_int4(k16, x.gv.contiguous(), x.gslots, *want)
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])
    assert keep.sum() == 37
