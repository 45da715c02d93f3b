"""What decode_int4 chooses for partition_tokens = 0, by the workspace that it asks
for: none for a single pass (no device call is needed)."""
import pytest

from paged_kv_cache_64_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_64_gb300 import build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("seqs,hkv", [(1, 1), (8, 2), (32, 2), (8, 8), (127, 1), (64, 2), (128, 2),
                                      (16, 8), (256, 8), (512, 2)])
def test_single_pass_up_to_a_length_that_goes_by_the_heads(lib, seqs, hkv):
    def single(max_len):
        return lib.pa_decode_int4_workspace_size(seqs, 4 * hkv, hkv, 128, 16, max_len, 0, 1) == 0
    bound = 2048 if seqs * hkv >= 128 else 1024
    assert single(1) and single(bound)
    assert not single(bound + 1) and not single(100000)


@pytest.mark.parametrize("max_len", [4097, 9000, 40000])
def test_more_sequences_than_balanced_ranges_are_cut_into_chunks(lib, max_len):
    """A partial (8 m, 8 l, G rows of D fp32) for each of up to eight chunks."""
    seqs, hkv, G, D = 1100, 2, 3, 64
    P = max(4096, (-(-max_len // 8) + 31) // 32 * 32)
    chunks = -(-max_len // P)
    slots = seqs * hkv * chunks
    up = lambda x: (x + 255) // 256 * 256
    want = 2 * up(slots * 8 * 4) + up(slots * G * D * 4)
    assert lib.pa_decode_int4_workspace_size(seqs, G * hkv, hkv, D, 16, max_len, 0, 1) == want
    assert lib.pa_decode_int4_workspace_size(seqs, G * hkv, hkv, D, 16, 4096, 0, 1) == 0
