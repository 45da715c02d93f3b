"""Python binding of the C ABI (include/pa.h) for torch tensors.

Argument marshalling only: every function checks devices, dtypes, shapes and
contiguity, passes raw pointers and sizes to libpa.so, and raises on a
non-OK status.  All computation runs in the library's CUDA kernels; nothing
here computes on the host or falls back to PyTorch ops.
"""
import ctypes

import numpy as np
import torch

from . import _lib

_DTYPES = {torch.float16: _lib.PA_F16, torch.bfloat16: _lib.PA_BF16}


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dt(t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported element type {t.dtype}; use float16 or bfloat16") from None


def _cuda(t, name, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def version():
    return _lib.load().pa_version()


def check_error(stream=None):
    """Synchronise the stream and raise if a kernel recorded a device error
    (PA_ERR_BAD_INDEX, PA_ERR_DEVICE_TIMEOUT)."""
    _lib.check("pa_check_error", _lib.load().pa_check_error(_stream_handle(stream)))


def selftest_wait_timeout(stream=None):
    """Launch the bounded-wait self-test kernel (see pa.h)."""
    _lib.check("pa_selftest_wait_timeout",
               _lib.load().pa_selftest_wait_timeout(_stream_handle(stream)))


def cache_write(k_new, v_new, slot_mapping, k_pool, v_pool, stream=None):
    """reshape_and_cache: k_new/v_new [T, Hkv, d] into pools [NB, Hkv, B, d]
    at slot_mapping (int64 [T]; slot = block * B + offset, < 0 skips)."""
    nb, hkv, bs, d = k_pool.shape
    if v_pool.shape != k_pool.shape or k_new.shape != v_new.shape:
        raise ValueError("pool / new-token shapes differ")
    if k_new.dim() != 3 or k_new.shape[1:] != (hkv, d):
        raise ValueError(f"k_new must be [T, {hkv}, {d}], got {tuple(k_new.shape)}")
    T = k_new.shape[0]
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    for t in (k_new, v_new, v_pool):
        if t.dtype != k_pool.dtype:
            raise TypeError("element types differ")
    rc = _lib.load().pa_cache_write(
        _cuda(k_new, "k_new"), _cuda(v_new, "v_new"),
        _cuda(slot_mapping, "slot_mapping", torch.int64), T,
        _cuda(k_pool, "k_pool", ndim=4), _cuda(v_pool, "v_pool", ndim=4), nb, hkv, d, bs,
        _dt(k_pool), _stream_handle(stream))
    _lib.check("pa_cache_write", rc)


def copy_blocks(k_pools, v_pools, block_mapping, stream=None):
    """Copy-on-write block copies: for each (src, dst) row of block_mapping
    (int64 [n, 2], CUDA), pool[dst] = pool[src] in every layer's K and V
    pool."""
    if len(k_pools) != len(v_pools) or not k_pools:
        raise ValueError("need the same non-zero number of K and V pools")
    shape, dtype = k_pools[0].shape, k_pools[0].dtype
    for t in list(k_pools) + list(v_pools):
        if t.shape != shape or t.dtype != dtype:
            raise ValueError("all pools must share shape and dtype")
    n = 0 if block_mapping.numel() == 0 else block_mapping.shape[0]
    if block_mapping.numel() and (block_mapping.dim() != 2 or block_mapping.shape[1] != 2):
        raise ValueError("block_mapping must be [n, 2]")
    L = len(k_pools)
    kp = (ctypes.c_void_p * L)(*[_cuda(t, "k_pool").value for t in k_pools])
    vp = (ctypes.c_void_p * L)(*[_cuda(t, "v_pool").value for t in v_pools])
    block_bytes = int(np.prod(shape[1:])) * k_pools[0].element_size()
    mp = _cuda(block_mapping, "block_mapping", torch.int64) if n else ctypes.c_void_p(0)
    rc = _lib.load().pa_copy_blocks(kp, vp, L, mp, n, shape[0], block_bytes,
                                    _stream_handle(stream))
    _lib.check("pa_copy_blocks", rc)


def _decode_dims(q, k_pool, block_tables, seq_lens):
    S, hq, d = q.shape
    nb, hkv, bs, d2 = k_pool.shape
    if d2 != d:
        raise ValueError("head_dim of q and pools differ")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be [S, max_blocks], seq_lens [S]")
    return S, hq, hkv, d, nb, bs


def auto_partition(num_seqs, num_kv_heads, max_seq_len, head_dim, block_size, group, dtype,
                   fp8=False):
    """Partition size decode (fp8=False) or decode_fp8 (fp8=True) uses for
    partition_tokens=0; -1 for single pass."""
    fn = _lib.load().pa_decode_fp8_auto_partition if fp8 else _lib.load().pa_decode_auto_partition
    return fn(num_seqs, num_kv_heads, max_seq_len, head_dim, block_size, group, _DTYPES[dtype])


def partial_tokens(num_seqs, num_kv_heads, max_seq_len, head_dim, block_size, group, dtype,
                   partition_tokens=0, fp8=False):
    """Positions each split-KV partial of decode (or decode_fp8) covers: the
    partition size times the partitions one CTA merges; -1 for single pass."""
    return _lib.load().pa_decode_partial_tokens(num_seqs, num_kv_heads, max_seq_len, head_dim,
                                                block_size, group, int(partition_tokens),
                                                _DTYPES[dtype], int(bool(fp8)))


DECODE_IMPLS = {"auto": 0, "cuda_cores": 1, "tensor_cores": 2}


def set_decode_impl(name):
    """Select the decode kernel for later calls ("auto", "cuda_cores",
    "tensor_cores"); returns the previous name."""
    prev = _lib.load().pa_set_decode_impl(DECODE_IMPLS[name])
    if prev < 0:
        raise ValueError(name)
    return {v: k for k, v in DECODE_IMPLS.items()}[prev]


def get_decode_impl():
    return {v: k for k, v in DECODE_IMPLS.items()}[_lib.load().pa_get_decode_impl()]


def set_decode_span(span):
    """Split-KV partitions per tensor-core CTA for later calls (0 = automatic);
    returns the previous setting."""
    prev = _lib.load().pa_set_decode_span(int(span))
    if prev < 0:
        raise ValueError(span)
    return prev


def ctas_per_sm(head_dim, group, dtype):
    return _lib.load().pa_decode_ctas_per_sm(head_dim, group, _DTYPES[dtype])


def workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                   partition_tokens, dtype):
    return _lib.load().pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                block_size, max_seq_len, partition_tokens,
                                                _DTYPES[dtype])


def alloc_workspace(nbytes, device):
    """Device scratch for split-KV (256-byte aligned by the caching allocator)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def decode(out, q, k_pool, v_pool, block_tables, seq_lens, max_seq_len, scale,
           partition_tokens=0, workspace=None, stream=None):
    """Paged decode attention into out [S, Hq, d].  partition_tokens: -1
    single pass, 0 automatic, >0 split-KV partition size.  workspace: a
    device buffer of at least workspace_size(...) bytes (alloc_workspace);
    when it is missing or too small one is allocated here, so a decode loop
    passes its own.  Returns the workspace used."""
    S, hq, hkv, d, nb, bs = _decode_dims(q, k_pool, block_tables, seq_lens)
    if out.shape != q.shape or out.dtype != q.dtype or k_pool.dtype != q.dtype:
        raise ValueError("out/q/pool shapes or types differ")
    need = workspace_size(S, hq, hkv, d, bs, max_seq_len, partition_tokens, q.dtype)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = alloc_workspace(need, q.device)
    ws = _cuda(workspace, "workspace") if workspace is not None else ctypes.c_void_p(0)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.load().pa_decode(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_pool, "k_pool"), _cuda(v_pool, "v_pool"), nb,
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), int(max_seq_len), S, hq, hkv, d, bs,
        float(scale), int(partition_tokens), ws, wbytes, _dt(q), _stream_handle(stream))
    _lib.check("pa_decode", rc)
    return workspace


def decode_step(out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables, seq_lens,
                max_seq_len, scale, partition_tokens=0, workspace=None, stream=None):
    """One fused decode step: write each sequence's newest token (k_new /
    v_new [S, Hkv, d] at slot_mapping [S], the slot of position seq_lens-1)
    and attend over seq_lens positions, in one launch.  workspace as for
    decode."""
    S, hq, hkv, d, nb, bs = _decode_dims(q, k_pool, block_tables, seq_lens)
    if out.shape != q.shape or out.dtype != q.dtype or k_pool.dtype != q.dtype:
        raise ValueError("out/q/pool shapes or types differ")
    if k_new.shape != (S, hkv, d) or v_new.shape != k_new.shape or slot_mapping.shape != (S,):
        raise ValueError("k_new/v_new must be [S, Hkv, d] and slot_mapping [S]")
    need = workspace_size(S, hq, hkv, d, bs, max_seq_len, partition_tokens, q.dtype)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = alloc_workspace(need, q.device)
    ws = _cuda(workspace, "workspace") if workspace is not None else ctypes.c_void_p(0)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.load().pa_decode_step(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_new, "k_new"), _cuda(v_new, "v_new"),
        _cuda(slot_mapping, "slot_mapping", torch.int64), _cuda(k_pool, "k_pool"),
        _cuda(v_pool, "v_pool"), nb, _cuda(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _cuda(seq_lens, "seq_lens", torch.int32), int(max_seq_len), S, hq,
        hkv, d, bs, float(scale), int(partition_tokens), ws, wbytes, _dt(q),
        _stream_handle(stream))
    _lib.check("pa_decode_step", rc)
    return workspace


def shared_prefix_len(block_tables, seq_lens, block_size):
    """Longest whole-block prefix that every sequence reaches through the
    same block-table entries (host arrays), capped by the shortest sequence:
    the prefix_len decode_cascade can be given for this batch
    (pa_shared_prefix_len)."""
    t = np.ascontiguousarray(block_tables, dtype=np.int32)
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    if t.ndim != 2 or lens.shape != (t.shape[0],):
        raise ValueError("block_tables must be [S, max_blocks], seq_lens [S]")
    out = ctypes.c_int(0)
    rc = _lib.load().pa_shared_prefix_len(
        t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), t.shape[1],
        lens.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), t.shape[0], int(block_size),
        ctypes.byref(out))
    _lib.check("pa_shared_prefix_len", rc)
    return out.value


def cache_write_fp8(k_new, v_new, slot_mapping, k_pool, v_pool, k_scale, v_scale, stream=None):
    """reshape_and_cache into E4M3 pools (uint8 [NB, Hkv, B, d]): k_new /
    v_new (16-bit [T, Hkv, d]) quantised with the pools' scales."""
    nb, hkv, bs, d = k_pool.shape
    T = k_new.shape[0]
    if k_pool.dtype != torch.uint8 or v_pool.dtype != torch.uint8:
        raise ValueError("E4M3 pools are uint8 tensors of codes")
    if k_new.shape != (T, hkv, d) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [T, Hkv, d]")
    rc = _lib.load().pa_cache_write_fp8(
        _cuda(k_new, "k_new"), _cuda(v_new, "v_new"),
        _cuda(slot_mapping, "slot_mapping", torch.int64), T, _cuda(k_pool, "k_pool"),
        _cuda(v_pool, "v_pool"), nb, hkv, d, bs, float(k_scale), float(v_scale), _dt(k_new),
        _stream_handle(stream))
    _lib.check("pa_cache_write_fp8", rc)


def fp8_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                       partition_tokens, dtype):
    return _lib.load().pa_decode_fp8_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                    head_dim, block_size, max_seq_len,
                                                    partition_tokens, _DTYPES[dtype])


def decode_fp8(out, q, k_pool, v_pool, block_tables, seq_lens, max_seq_len, scale, k_scale,
               v_scale, partition_tokens=0, k_new=None, v_new=None, slot_mapping=None,
               workspace=None, stream=None):
    """Paged decode over E4M3 pools (uint8 codes, element = scale * code);
    q / out 16-bit.  With k_new / v_new / slot_mapping, each sequence's newest
    token is quantised and written first (the fused step)."""
    S, hq, d = q.shape
    nb, hkv, bs, d2 = k_pool.shape
    if d2 != d or block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape != (S,):
        raise ValueError("shapes of q, pools, block_tables, seq_lens disagree")
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    if k_pool.dtype != torch.uint8 or v_pool.dtype != torch.uint8:
        raise ValueError("E4M3 pools are uint8 tensors of codes")
    step = k_new is not None
    if step and (k_new.shape != (S, hkv, d) or v_new is None or v_new.shape != k_new.shape
                 or slot_mapping is None or slot_mapping.shape != (S,)):
        raise ValueError("k_new/v_new must be [S, Hkv, d] and slot_mapping [S]")
    need = fp8_workspace_size(S, hq, hkv, d, bs, max_seq_len, partition_tokens, q.dtype)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = alloc_workspace(need, q.device)
    ws = _cuda(workspace, "workspace") if workspace is not None else ctypes.c_void_p(0)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    null = ctypes.c_void_p(0)
    rc = _lib.load().pa_decode_fp8(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_new, "k_new") if step else null,
        _cuda(v_new, "v_new") if step else null,
        _cuda(slot_mapping, "slot_mapping", torch.int64) if step else null,
        _cuda(k_pool, "k_pool"), _cuda(v_pool, "v_pool"), nb,
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), int(max_seq_len), S, hq, hkv, d, bs,
        float(scale), float(k_scale), float(v_scale), int(partition_tokens), ws, wbytes, _dt(q),
        _stream_handle(stream))
    _lib.check("pa_decode_fp8", rc)
    return workspace


# The checks below are written out in each wrapper as one condition (a call
# costs more than the kernel of a small batch); when it fails, _explain finds
# the argument and says what is wrong with it.


def _explain(dev, **tensors):
    """Raise for the first of name=(tensor, dtype or None) that is not a dense
    CUDA tensor of that type on device `dev` (the first tensor's)."""
    for name, (t, dtype) in tensors.items():
        if t is None:
            continue
        _cuda(t, name, dtype)
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the device of the other tensors (cuda:{dev})")
    raise ValueError("arguments must be dense CUDA tensors on one device")


def _check(fn_name, rc, **tensors):
    """Raise unless rc is PA_OK; for PA_ERR_INVALID name the first of the tensors
    that the library refuses for its address."""
    if rc == _lib.PA_ERR_INVALID:
        for name, t in tensors.items():
            if t is not None and t.data_ptr() % 16:
                raise ValueError(f"{name} must start on a 16-byte boundary")
    _lib.check(fn_name, rc)


def _run(dev, stream, fn, args):
    """fn(*args, stream handle) with `dev` current; stream None: its current
    stream.  (What torch.cuda's own calls end in, looked up here: builds of torch
    without CUDA lack them, and the host parts of this module need none.)"""
    cuda = torch._C
    if dev != cuda._cuda_getDevice():
        with torch.cuda.device(dev):
            return _run(dev, stream, fn, args)
    return fn(*args, cuda._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def int4_pool_shape(num_blocks, num_kv_heads, block_size, head_dim):
    """Shape of a 4-bit pool (a uint8 tensor): one record a (block, KV head),
    block_size * (head_dim / 2 + 4) bytes (layout in pa.h)."""
    rec = _lib.load().pa_int4_record_bytes(int(head_dim), int(block_size))
    if not rec:
        raise ValueError("4-bit pools hold head_dim 64 or 128 in blocks of 16 or 32")
    return (int(num_blocks), int(num_kv_heads), rec)


def _int4_pools(k_pool, v_pool, hkv, d):
    """(blocks, block size) of a pair of 4-bit pools."""
    if k_pool.dtype is not torch.uint8 or v_pool.dtype is not torch.uint8:
        raise TypeError("4-bit pools are uint8 tensors of records")
    shape = k_pool.shape
    if len(shape) != 3 or shape[1] != hkv or v_pool.shape != shape:
        raise ValueError(f"4-bit pools must both be [blocks, {hkv}, record bytes] (int4_pool_shape)")
    bs, rest = divmod(shape[2], d // 2 + 4)
    if rest or (bs != 16 and bs != 32):
        raise ValueError(f"a record of {shape[2]} bytes is no block of 16 or 32 rows of head_dim {d}")
    return shape[0], bs


def cache_write_int4(k_new, v_new, slot_mapping, k_pool, v_pool, k_out=None, v_out=None,
                     stream=None):
    """reshape_and_cache into 4-bit pools (uint8, int4_pool_shape): each row
    of k_new / v_new (16-bit [T, Hkv, d]) quantised with its own scale and
    minimum at its slot (int64 [T]; < 0 skips; distinct).  k_out / v_out (like
    k_new; may be k_new / v_new) receive the values the stored rows stand for."""
    shape, dtype = k_new.shape, k_new.dtype
    if len(shape) != 3 or v_new.shape != shape or v_new.dtype is not dtype:
        raise ValueError("k_new and v_new must both be [T, Hkv, d] of one type")
    T, hkv, d = shape
    nb, bs = _int4_pools(k_pool, v_pool, hkv, d)
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    code = _dt(k_new)
    dev = k_new.get_device()
    if not (dev >= 0 and k_new.is_contiguous() and v_new.is_contiguous()
            and slot_mapping.is_contiguous() and k_pool.is_contiguous() and v_pool.is_contiguous()
            and v_new.get_device() == dev and slot_mapping.get_device() == dev
            and k_pool.get_device() == dev and v_pool.get_device() == dev
            and slot_mapping.dtype is torch.int64):
        _explain(dev, k_new=(k_new, None), v_new=(v_new, None),
                 slot_mapping=(slot_mapping, torch.int64), k_pool=(k_pool, None),
                 v_pool=(v_pool, None))
    ko = vo = None
    if k_out is not None:
        for t in (k_out, v_out):
            if t.shape != shape or t.dtype is not dtype:
                raise ValueError("k_out and v_out must be like k_new")
            if t.get_device() != dev or not t.is_contiguous():
                _explain(dev, k_out=(k_out, None), v_out=(v_out, None))
        ko, vo = k_out.data_ptr(), v_out.data_ptr()
    rc = _run(dev, stream, _lib.load().pa_cache_write_int4,
              (k_new.data_ptr(), v_new.data_ptr(), slot_mapping.data_ptr(), T, k_pool.data_ptr(),
               v_pool.data_ptr(), nb, hkv, d, bs, ko, vo, code))
    _check("pa_cache_write_int4", rc, k_new=k_new, v_new=v_new, k_pool=k_pool, v_pool=v_pool,
           k_out=k_out, v_out=v_out)


def cache_read_int4(k_out, v_out, slot_mapping, k_pool, v_pool, stream=None):
    """Rows of 4-bit pools back as 16-bit values: k_out / v_out [T, Hkv, d]
    at slot_mapping (int64 [T]; rows of a negative slot are left alone)."""
    shape, dtype = k_out.shape, k_out.dtype
    if len(shape) != 3 or v_out.shape != shape or v_out.dtype is not dtype:
        raise ValueError("k_out and v_out must both be [T, Hkv, d] of one type")
    T, hkv, d = shape
    nb, bs = _int4_pools(k_pool, v_pool, hkv, d)
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    code = _dt(k_out)
    dev = k_out.get_device()
    if not (dev >= 0 and k_out.is_contiguous() and v_out.is_contiguous()
            and slot_mapping.is_contiguous() and k_pool.is_contiguous() and v_pool.is_contiguous()
            and v_out.get_device() == dev and slot_mapping.get_device() == dev
            and k_pool.get_device() == dev and v_pool.get_device() == dev
            and slot_mapping.dtype is torch.int64):
        _explain(dev, k_out=(k_out, None), v_out=(v_out, None),
                 slot_mapping=(slot_mapping, torch.int64), k_pool=(k_pool, None),
                 v_pool=(v_pool, None))
    rc = _run(dev, stream, _lib.load().pa_cache_read_int4,
              (k_out.data_ptr(), v_out.data_ptr(), slot_mapping.data_ptr(), T, k_pool.data_ptr(),
               v_pool.data_ptr(), nb, hkv, d, bs, code))
    _check("pa_cache_read_int4", rc, k_out=k_out, v_out=v_out, k_pool=k_pool, v_pool=v_pool)


def int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                        partition_tokens, dtype):
    return _lib.load().pa_decode_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                     block_size, max_seq_len, partition_tokens,
                                                     _DTYPES[dtype])


def decode_int4(out, q, k_pool, v_pool, block_tables, seq_lens, max_seq_len, scale,
                partition_tokens=0, workspace=None, stream=None):
    """Paged decode attention over 4-bit pools (uint8, int4_pool_shape) into
    out [S, Hq, d]; q / out 16-bit.  partition_tokens and workspace as for
    decode (a workspace allocated here is of int4_workspace_size bytes and
    tied to the stream)."""
    shape = q.shape
    if len(shape) != 3 or out.shape != shape or out.dtype is not q.dtype:
        raise ValueError("q and out must both be [S, Hq, d] of one type")
    S, hq, d = shape
    if k_pool.dim() != 3:
        raise ValueError("4-bit pools are [blocks, Hkv, record bytes] (int4_pool_shape)")
    hkv = k_pool.shape[1]
    nb, bs = _int4_pools(k_pool, v_pool, hkv, d)
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != S or seq_lens.shape != (S,):
        raise ValueError("block_tables must be [S, max_blocks], seq_lens [S]")
    code = _dt(q)
    dev = q.get_device()
    if not (dev >= 0 and q.is_contiguous() and out.is_contiguous() and k_pool.is_contiguous()
            and v_pool.is_contiguous() and block_tables.is_contiguous() and seq_lens.is_contiguous()
            and out.get_device() == dev and k_pool.get_device() == dev
            and v_pool.get_device() == dev and block_tables.get_device() == dev
            and seq_lens.get_device() == dev and block_tables.dtype is torch.int32
            and seq_lens.dtype is torch.int32):
        _explain(dev, q=(q, None), out=(out, None), k_pool=(k_pool, None), v_pool=(v_pool, None),
                 block_tables=(block_tables, torch.int32), seq_lens=(seq_lens, torch.int32))
    fn = _lib.load().pa_decode_int4
    max_len, part = int(max_seq_len), int(partition_tokens)
    args = (out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), nb,
            block_tables.data_ptr(), tables[1], seq_lens.data_ptr(), max_len, S, hq, hkv, d, bs,
            float(scale), part)

    def run(ws):
        if ws is None:
            return _run(dev, stream, fn, args + (None, 0, code))
        if ws.get_device() != dev or not ws.is_contiguous():
            _explain(dev, workspace=(ws, None))
        return _run(dev, stream, fn, args + (ws.data_ptr(), ws.nbytes, code))

    rc = run(workspace)
    if rc == _lib.PA_ERR_INVALID:  # perhaps for want of a workspace: nothing was launched
        with torch.cuda.device(dev):
            need = int4_workspace_size(S, hq, hkv, d, bs, max_len, part, q.dtype)
        if need and (workspace is None or workspace.nbytes < need):
            # from the stream's own memory: a block freed on another stream may
            # still be in use there
            with torch.cuda.stream(stream):
                workspace = alloc_workspace(need, q.device)
            rc = run(workspace)
        elif need and workspace.data_ptr() % 256:
            raise ValueError("workspace must start on a 256-byte boundary")
    _check("pa_decode_int4", rc, out=out, q=q, k_pool=k_pool, v_pool=v_pool)
    return workspace


def _token_step(t, name, T, own, d):
    """Elements from a token to the next of t [T, heads, d] whose heads, `own`
    elements, are dense."""
    step, head, one = t.stride()
    if T <= 1:
        step = own
    if one != 1 or (head != d and own != d) or step < own:
        raise ValueError(f"{name}: each token's heads must be dense and apart from the next's")
    if step % 8:
        raise ValueError(f"{name}: the step from a token to the next must be a multiple of 8 elements")
    return step


def qk_norm_rope(q_out, q, k, v, q_weight, k_weight, eps, cos_sin, positions, slot_mapping, k_pool,
                 v_pool, interleaved=False, k_scale=None, v_scale=None, stream=None):
    """RMS norm of every q and k head, rotary positions and the cache write in
    one pass (pa_qk_norm_rope).  q, q_out [T, Hq, d]; k, v [T, Hkv, d] (tokens
    may be strided: column ranges of one projection; q_out may be q);
    weights [d]; cos_sin float32 [positions, rotary_dim] (cosines, sines);
    positions, slot_mapping int64 [T].  The pools' form is theirs: like q
    [NB, Hkv, B, d], E4M3 codes (uint8, the same shape, with k_scale and
    v_scale) or 4-bit records (uint8, int4_pool_shape)."""
    qs, ks_, dt = q.shape, k.shape, q.dtype
    if len(qs) != 3 or len(ks_) != 3 or v.shape != ks_ or q_out.shape != qs or ks_[0] != qs[0] \
            or ks_[2] != qs[2]:
        raise ValueError("q and q_out must be [T, Hq, d], k and v [T, Hkv, d]")
    T, hq, d = qs
    hkv = ks_[1]
    if not (k.dtype is dt and v.dtype is dt and q_out.dtype is dt and q_weight.dtype is dt
            and k_weight.dtype is dt):
        raise TypeError("q, q_out, k, v and the weights must have one type")
    if q_weight.shape != (d,) or k_weight.shape != (d,):
        raise ValueError("the weights must be [head_dim]")
    if positions.shape != (T,) or slot_mapping.shape != (T,):
        raise ValueError("positions and slot_mapping must be [T]")
    table = cos_sin.shape
    if len(table) != 2:
        raise ValueError("cos_sin must be [positions, rotary_dim]")
    ks = vs = 1.0
    pool = k_pool.shape
    if len(pool) == 3:
        fmt = _lib.PA_KV_INT4
        nb, bs = _int4_pools(k_pool, v_pool, hkv, d)
    else:
        if len(pool) != 4 or v_pool.shape != pool or pool[1] != hkv or pool[3] != d:
            raise ValueError(f"pools must both be [blocks, {hkv}, block size, {d}] or 4-bit records")
        nb, bs = pool[0], pool[2]
        if k_pool.dtype is dt and v_pool.dtype is dt:
            fmt = _lib.PA_KV_16BIT
        elif k_pool.dtype is torch.uint8 and v_pool.dtype is torch.uint8:
            fmt = _lib.PA_KV_E4M3
            if k_scale is None or v_scale is None:
                raise ValueError("E4M3 pools need k_scale and v_scale")
            ks, vs = float(k_scale), float(v_scale)
        else:
            raise TypeError("pools must have q's type or be uint8 codes")
    code = _dt(q)
    dev = q.get_device()
    if not (dev >= 0 and k.get_device() == dev and v.get_device() == dev
            and q_out.get_device() == dev and q_weight.get_device() == dev
            and k_weight.get_device() == dev and cos_sin.get_device() == dev
            and positions.get_device() == dev and slot_mapping.get_device() == dev
            and k_pool.get_device() == dev and v_pool.get_device() == dev
            and q_weight.is_contiguous() and k_weight.is_contiguous() and cos_sin.is_contiguous()
            and positions.is_contiguous() and slot_mapping.is_contiguous()
            and k_pool.is_contiguous() and v_pool.is_contiguous()
            and cos_sin.dtype is torch.float32 and positions.dtype is torch.int64
            and slot_mapping.dtype is torch.int64):
        for name, t in (("q", q), ("k", k), ("v", v), ("q_out", q_out)):  # may be strided
            if t.get_device() != dev or dev < 0:
                raise ValueError(f"{name} must be a CUDA tensor on the device of the others")
        _explain(dev, q_weight=(q_weight, None), k_weight=(k_weight, None),
                 cos_sin=(cos_sin, torch.float32), positions=(positions, torch.int64),
                 slot_mapping=(slot_mapping, torch.int64), k_pool=(k_pool, None),
                 v_pool=(v_pool, None))
    rc = _run(dev, stream, _lib.load().pa_qk_norm_rope,
              (q_out.data_ptr(), _token_step(q_out, "q_out", T, hq * d, d), q.data_ptr(),
               _token_step(q, "q", T, hq * d, d), k.data_ptr(), _token_step(k, "k", T, hkv * d, d),
               v.data_ptr(), _token_step(v, "v", T, hkv * d, d), q_weight.data_ptr(),
               k_weight.data_ptr(), float(eps), cos_sin.data_ptr(), table[0], table[1],
               1 if interleaved else 0, positions.data_ptr(), slot_mapping.data_ptr(), T,
               k_pool.data_ptr(), v_pool.data_ptr(), nb, hq, hkv, d, bs, fmt, ks, vs, code))
    _check("pa_qk_norm_rope", rc, q_out=q_out, q=q, k=k, v=v, q_weight=q_weight, k_weight=k_weight,
           cos_sin=cos_sin, k_pool=k_pool, v_pool=v_pool)


def cascade_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                           max_seq_len, prefix_len, dtype):
    return _lib.load().pa_decode_cascade_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                        head_dim, block_size, max_seq_len,
                                                        prefix_len, _DTYPES[dtype])


def decode_cascade(out, q, k_pool, v_pool, block_tables, seq_lens, max_seq_len, scale,
                   prefix_len, k_new=None, v_new=None, slot_mapping=None, workspace=None,
                   stream=None):
    """Decode of a batch whose sequences share their first prefix_len
    positions (the same first prefix_len / block_size block-table entries):
    the prefix is attended once per KV head for every sequence's queries,
    each tail separately, and the two merged.  With k_new / v_new /
    slot_mapping, each sequence's newest token is written first, as in
    decode_step."""
    S, hq, hkv, d, nb, bs = _decode_dims(q, k_pool, block_tables, seq_lens)
    if out.shape != q.shape or out.dtype != q.dtype or k_pool.dtype != q.dtype:
        raise ValueError("out/q/pool shapes or types differ")
    step = k_new is not None
    if step and (k_new.shape != (S, hkv, d) or v_new is None or v_new.shape != k_new.shape
                 or slot_mapping is None or slot_mapping.shape != (S,)):
        raise ValueError("k_new/v_new must be [S, Hkv, d] and slot_mapping [S]")
    need = cascade_workspace_size(S, hq, hkv, d, bs, max_seq_len, prefix_len, q.dtype)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = alloc_workspace(need, q.device)
    ws = _cuda(workspace, "workspace") if workspace is not None else ctypes.c_void_p(0)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    null = ctypes.c_void_p(0)
    rc = _lib.load().pa_decode_cascade(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_new, "k_new") if step else null,
        _cuda(v_new, "v_new") if step else null,
        _cuda(slot_mapping, "slot_mapping", torch.int64) if step else null,
        _cuda(k_pool, "k_pool"), _cuda(v_pool, "v_pool"), nb,
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), int(max_seq_len), S, hq, hkv, d, bs,
        float(scale), int(prefix_len), ws, wbytes, _dt(q), _stream_handle(stream))
    _lib.check("pa_decode_cascade", rc)
    return workspace


def decode_static_scratch(out, q, k_pool, v_pool, block_tables, seq_lens, max_seq_len, scale,
                          partition_tokens=0, stream=None):
    """Same result as decode(), for callers that cannot allocate device
    memory: split-KV partials go to the library's fixed device array
    (_lib.STATIC_SCRATCH_BYTES per GPU) instead of a workspace.  Raises
    PagedAttentionError (PA_ERR_TOO_LARGE) when they would not fit; calls on
    one device share that array, so they must not overlap on the GPU."""
    S, hq, hkv, d, nb, bs = _decode_dims(q, k_pool, block_tables, seq_lens)
    if out.shape != q.shape or out.dtype != q.dtype or k_pool.dtype != q.dtype:
        raise ValueError("out/q/pool shapes or types differ")
    rc = _lib.load().pa_decode_static_scratch(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_pool, "k_pool"), _cuda(v_pool, "v_pool"), nb,
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), int(max_seq_len), S, hq, hkv, d, bs,
        float(scale), int(partition_tokens), _dt(q), _stream_handle(stream))
    _lib.check("pa_decode_static_scratch", rc)


def partition_count(max_seq_len, partition_tokens):
    return max(1, -(-int(max_seq_len) // int(partition_tokens)))


def partials_view(workspace, num_seqs, num_q_heads, head_dim, max_seq_len, partition_tokens):
    """Views (m, l, O) of the partials in a workspace, per the layout in pa.h."""
    NP = partition_count(max_seq_len, partition_tokens)
    rows = num_seqs * num_q_heads * NP
    a = lambda x: (x + 255) // 256 * 256
    m_off, l_off = 0, a(rows * 4)
    o_off = l_off + a(rows * 4)
    f = workspace.view(torch.uint8)
    m = f[m_off:m_off + rows * 4].view(torch.float32).view(num_seqs, num_q_heads, NP)
    l = f[l_off:l_off + rows * 4].view(torch.float32).view(num_seqs, num_q_heads, NP)
    o = f[o_off:o_off + rows * head_dim * 4].view(torch.float32).view(
        num_seqs, num_q_heads, NP, head_dim)
    return m, l, o


def decode_partitions(q, k_pool, v_pool, block_tables, seq_lens, max_seq_len, scale,
                      partition_tokens, workspace, stream=None):
    """Split-KV step 2 only: partials into the workspace."""
    S, hq, hkv, d, nb, bs = _decode_dims(q, k_pool, block_tables, seq_lens)
    rc = _lib.load().pa_decode_partitions(
        _cuda(q, "q"), _cuda(k_pool, "k_pool"), _cuda(v_pool, "v_pool"), nb,
        _cuda(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _cuda(seq_lens, "seq_lens", torch.int32), int(max_seq_len), S, hq, hkv, d, bs,
        float(scale), int(partition_tokens), _cuda(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _dt(q), _stream_handle(stream))
    _lib.check("pa_decode_partitions", rc)


def split_kv_reduce(out, workspace, seq_lens, max_seq_len, partition_tokens, stream=None):
    """Split-KV step 3 only: combine the partials in the workspace into out."""
    S, hq, d = out.shape
    rc = _lib.load().pa_split_kv_reduce(
        _cuda(out, "out"), _cuda(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _cuda(seq_lens, "seq_lens", torch.int32),
        int(max_seq_len), S, hq, d, int(partition_tokens), _dt(out), _stream_handle(stream))
    _lib.check("pa_split_kv_reduce", rc)


class BlockAllocator:
    """Host block allocator (free list, refcounts, fork, copy-on-write)."""

    def __init__(self, num_blocks, block_size, free_order=None):
        self._lib = _lib.load()
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)
        handle = ctypes.c_void_p()
        order = None
        if free_order is not None:
            arr = np.ascontiguousarray(free_order, dtype=np.int32)
            if arr.shape != (self.num_blocks,):
                raise ValueError("free_order must list every block once")
            order = arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        _lib.check("pa_alloc_create", self._lib.pa_alloc_create(
            self.num_blocks, self.block_size, order, ctypes.byref(handle)))
        self._h = handle

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._lib.pa_alloc_destroy(h)
            self._h = None

    def add(self, seq):
        _lib.check("pa_seq_add", self._lib.pa_seq_add(self._h, int(seq)))

    def append(self, seq, n=1):
        """Returns (slots, copies) like the allocator model: flat slots of the
        new tokens and the (src, dst) copy-on-write pair(s)."""
        slots = np.empty(max(int(n), 1), dtype=np.int64)
        pair = np.empty(2, dtype=np.int64)
        ncow = ctypes.c_int(0)
        rc = self._lib.pa_seq_append(
            self._h, int(seq), int(n), slots.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
            pair.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), ctypes.byref(ncow))
        _lib.check("pa_seq_append", rc)
        copies = [(int(pair[0]), int(pair[1]))] if ncow.value else []
        return slots[:int(n)].tolist(), copies

    def fork(self, parent, child):
        _lib.check("pa_seq_fork", self._lib.pa_seq_fork(self._h, int(parent), int(child)))

    def release(self, seq):
        _lib.check("pa_seq_free", self._lib.pa_seq_free(self._h, int(seq)))

    def length(self, seq):
        v = ctypes.c_int64()
        _lib.check("pa_seq_len", self._lib.pa_seq_len(self._h, int(seq), ctypes.byref(v)))
        return v.value

    def table(self, seq):
        n = ctypes.c_int()
        cap = self.num_blocks
        out = np.empty(max(cap, 1), dtype=np.int32)
        rc = self._lib.pa_seq_block_table(self._h, int(seq),
                                          out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                          cap, ctypes.byref(n))
        _lib.check("pa_seq_block_table", rc)
        return out[:n.value].tolist()

    def export(self, seqs, max_blocks_per_seq):
        """Dense int32 [n, max_blocks] tables and int32 [n] lengths."""
        ids = np.ascontiguousarray(seqs, dtype=np.int64)
        tables = np.zeros((len(ids), max(int(max_blocks_per_seq), 1)), dtype=np.int32)
        lens = np.zeros(len(ids), dtype=np.int32)
        rc = self._lib.pa_alloc_export(
            self._h, ids.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), len(ids),
            tables.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(max_blocks_per_seq),
            lens.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
        _lib.check("pa_alloc_export", rc)
        return tables[:, :int(max_blocks_per_seq)], lens

    def num_free(self):
        return self._lib.pa_alloc_num_free(self._h)

    def free_list(self):
        n = ctypes.c_int()
        out = np.empty(max(self.num_blocks, 1), dtype=np.int32)
        rc = self._lib.pa_alloc_free_list(self._h,
                                          out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                          self.num_blocks, ctypes.byref(n))
        _lib.check("pa_alloc_free_list", rc)
        return out[:n.value].tolist()

    def refcount(self, block):
        return self._lib.pa_block_refcount(self._h, int(block))


class PrefixCachePool:
    """Host block pool with automatic prefix caching (pa_pcache_*): requests
    whose prompts begin with cached full blocks share them; freed hashed
    blocks stay cached until the pool needs them (LRU)."""

    def __init__(self, num_blocks, block_size, free_order=None):
        self._lib = _lib.load()
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)
        handle = ctypes.c_void_p()
        order = None
        if free_order is not None:
            arr = np.ascontiguousarray(free_order, dtype=np.int32)
            if arr.shape != (self.num_blocks,):
                raise ValueError("free_order must list every block once")
            self._order = arr
            order = arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        _lib.check("pa_pcache_create", self._lib.pa_pcache_create(
            self.num_blocks, self.block_size, order, ctypes.byref(handle)))
        self._h = handle

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._lib.pa_pcache_destroy(h)
            self._h = None

    @staticmethod
    def _tokens(tokens):
        arr = np.ascontiguousarray(tokens, dtype=np.int32).reshape(-1)
        return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    def lookup(self, tokens, salt=0):
        """Number of leading full blocks of the prompt that are cached."""
        arr, ptr = self._tokens(tokens)
        n = ctypes.c_int()
        _lib.check("pa_pcache_lookup", self._lib.pa_pcache_lookup(
            self._h, ptr, arr.size, int(salt) & (2**64 - 1), ctypes.byref(n)))
        return n.value

    def add_request(self, seq, tokens, salt=0):
        """Returns (cached tokens, slot of every prompt position)."""
        arr, ptr = self._tokens(tokens)
        slots = np.empty(max(arr.size, 1), dtype=np.int64)
        cached = ctypes.c_int()
        _lib.check("pa_pcache_add", self._lib.pa_pcache_add(
            self._h, int(seq), ptr, arr.size, int(salt) & (2**64 - 1), ctypes.byref(cached),
            slots.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))))
        return cached.value, slots[:arr.size].tolist()

    def append(self, seq, token):
        slot = ctypes.c_int64()
        _lib.check("pa_pcache_append", self._lib.pa_pcache_append(
            self._h, int(seq), int(token), ctypes.byref(slot)))
        return slot.value

    def release(self, seq):
        _lib.check("pa_pcache_free", self._lib.pa_pcache_free(self._h, int(seq)))

    def table(self, seq):
        n = ctypes.c_int()
        out = np.empty(max(self.num_blocks, 1), dtype=np.int32)
        _lib.check("pa_pcache_block_table", self._lib.pa_pcache_block_table(
            self._h, int(seq), out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
            self.num_blocks, ctypes.byref(n)))
        return out[:n.value].tolist()

    def length(self, seq):
        v = ctypes.c_int64()
        _lib.check("pa_pcache_len", self._lib.pa_pcache_len(self._h, int(seq), ctypes.byref(v)))
        return v.value

    def free_list(self):
        n = ctypes.c_int()
        out = np.empty(max(self.num_blocks, 1), dtype=np.int32)
        _lib.check("pa_pcache_free_queue", self._lib.pa_pcache_free_queue(
            self._h, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), self.num_blocks,
            ctypes.byref(n)))
        return out[:n.value].tolist()

    def num_free(self):
        return self._lib.pa_pcache_num_free(self._h)

    def refcount(self, blk):
        return self._lib.pa_pcache_refcount(self._h, int(blk))

    def block_hash(self, blk):
        """The block's hash, or None when it is not cached."""
        h = ctypes.c_uint64()
        c = ctypes.c_int()
        _lib.check("pa_pcache_block_hash", self._lib.pa_pcache_block_hash(
            self._h, int(blk), ctypes.byref(h), ctypes.byref(c)))
        return h.value if c.value else None

    def hash_block(self, prev, tokens):
        arr, ptr = self._tokens(tokens)
        return int(self._lib.pa_pcache_hash_block(int(prev) & (2**64 - 1), ptr, arr.size))
