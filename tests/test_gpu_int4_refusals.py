"""The 4-bit and norm-rope wrappers say which argument they refuse.  Host checks
alone: none of these calls launches anything."""
import pytest
import torch

from paged_kv_cache_64_gb300 import api

pytestmark = pytest.mark.gpu


def shifted(t):
    """t's values two elements into a buffer: dense, on no 16-byte boundary."""
    flat = torch.empty(t.numel() + 2, dtype=t.dtype, device=t.device)[2:]
    flat.copy_(t.reshape(-1))
    assert flat.data_ptr() % 16
    return flat.view(t.shape)


def rope_args(T=3, hq=4, hkv=2, d=64):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(T, dtype=torch.int64, device="cuda")
    return dict(q_out=z(T, hq, d), q=z(T, hq, d), k=z(T, hkv, d), v=z(T, hkv, d), q_weight=z(d),
                k_weight=z(d), eps=1e-6, cos_sin=torch.zeros(9, d, device="cuda"), positions=n,
                slot_mapping=n - 1, k_pool=z(4, hkv, 16, d), v_pool=z(4, hkv, 16, d))


@pytest.mark.parametrize("name", ["q_out", "q", "k", "v", "q_weight", "k_weight", "cos_sin", "k_pool",
                                  "v_pool"])
def test_norm_rope_names_what_is_not_aligned(name):
    args = rope_args()
    args[name] = shifted(args[name])
    with pytest.raises(ValueError, match=rf"\b{name}\b.*16"):
        api.qk_norm_rope(**args)


@pytest.mark.parametrize("name", ["q_out", "q", "k", "v"])
def test_norm_rope_names_a_crooked_step(name):
    args = rope_args()
    t = args[name]
    wide = torch.zeros(3, t[0].numel() + 4, dtype=t.dtype, device="cuda")
    args[name] = wide[:, :t[0].numel()].view(t.shape)
    with pytest.raises(ValueError, match=rf"\b{name}\b.*multiple of 8"):
        api.qk_norm_rope(**args)
    args[name] = args[name][:1]  # of one token no step is taken
    for other in ("q_out", "q", "k", "v", "positions", "slot_mapping"):
        args[other] = args[other][:1]
    api.qk_norm_rope(**args)
    api.check_error()


def test_write_read_and_decode_name_what_is_not_aligned():
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    pool = torch.zeros(api.int4_pool_shape(4, 2, 16, 64), dtype=torch.uint8, device="cuda")
    bent = torch.empty(pool.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(pool.shape)
    slots = torch.full((3,), -1, device="cuda")
    for name in ("k_new", "v_new", "k_pool", "v_pool", "k_out", "v_out"):
        args = dict(k_new=k, v_new=k, slot_mapping=slots, k_pool=pool, v_pool=pool, k_out=k, v_out=k)
        args[name] = bent if "pool" in name else shifted(k)
        with pytest.raises(ValueError, match=rf"\b{name}\b.*16"):
            api.cache_write_int4(**args)
    for name in ("k_out", "v_out", "k_pool", "v_pool"):
        args = dict(k_out=k, v_out=k, slot_mapping=slots, k_pool=pool, v_pool=pool)
        args[name] = bent if "pool" in name else shifted(k)
        with pytest.raises(ValueError, match=rf"\b{name}\b.*16"):
            api.cache_read_int4(**args)
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    tables = torch.zeros(1, 64, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    for name in ("q", "out", "k_pool", "v_pool"):
        args = dict(out=q.clone(), q=q, k_pool=pool, v_pool=pool, block_tables=tables, seq_lens=lens,
                    max_seq_len=1000, scale=1.0)
        args[name] = bent if "pool" in name else shifted(q)
        with pytest.raises(ValueError, match=rf"\b{name}\b.*16"):
            api.decode_int4(**args)
    need = api.int4_workspace_size(1, 4, 2, 64, 16, 1000, 64, q.dtype)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    with pytest.raises(ValueError, match="workspace.*256"):
        api.decode_int4(q.clone(), q, pool, pool, tables, lens, 1000, 1.0, partition_tokens=64,
                        workspace=ws)
