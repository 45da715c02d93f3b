// pa_cache_write_int4 and pa_cache_read_int4: rows into and out of paged
// 4-bit pools (see pa_int4.cuh for the format).
//
// A row of D values is D/8 consecutive lanes, 8 elements (16 bytes of 16-bit
// values, 4 bytes of codes) a lane, so a warp reads and writes whole rows.
// Bound by HBM: 2 bytes an element on the 16-bit side, 0.53 (D = 128) or 0.56
// (D = 64) in the pool.
#include <cstdint>

#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

struct Int4IoParams {
    const uint4 *src[2];  // K and V rows to store (write)
    uint4 *dst[2];        // values out, or nullptr (write)
    uint8_t *pool[2];
    const int64_t *slots;
    int64_t num_slots;
    int rows;             // tokens * KV heads
    int num_kv_heads;
    int log2_block;
    int *err;
};

// Byte offset of slot `slot`'s codes in the pool and of its (s, m) pair from
// the start of its record.
template <int D>
__device__ __forceinline__ int64_t int4_record(const Int4IoParams &p, int64_t slot, int head,
                                               int *off) {
    const int64_t blk = slot >> p.log2_block;
    *off = (int)(slot & ((1 << p.log2_block) - 1));
    return (blk * p.num_kv_heads + head) * (int64_t)int4_record_bytes<D>(1 << p.log2_block);
}

constexpr int kInt4Threads = 256;

// blockIdx.y: 0 K, 1 V.  READ: pool -> values; otherwise values -> pool, and
// the stored values out when dst is given.
template <bool BF16, int D, bool READ>
__global__ void __launch_bounds__(kInt4Threads) int4_rows_kernel(const Int4IoParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // programmatic dependent launch
    constexpr int LANES = D / 8, ROWS = kInt4Threads / LANES;
    const int which = blockIdx.y, c = threadIdx.x % LANES;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < p.rows; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = r0 + threadIdx.x / LANES;
        int64_t slot = -1;
        int head = 0;
        if (row < p.rows) {
            const int t = (int)row / p.num_kv_heads;
            head = (int)row - t * p.num_kv_heads;
            slot = p.slots[t];
            if (slot >= p.num_slots) {
                if (c == 0) record_error(p.err, PA_ERR_BAD_INDEX);
                slot = -1;
            }
        }
        int off = 0;
        uint8_t *rec = nullptr;
        if (slot >= 0) rec = p.pool[which] + int4_record<D>(p, slot, head, &off);
        const int64_t piece = row * LANES + c;
        Int4Row q;
        if constexpr (READ) {
            if (slot < 0) continue;
            q.codes = *reinterpret_cast<const uint32_t *>(rec + off * (D / 2) + c * 4);
            q.params = *reinterpret_cast<const uint32_t *>(rec + (D / 2 << p.log2_block) + off * 4);
            p.dst[which][piece] = read8_int4<BF16>(q.codes, q.params);
        } else {
            float x[8];
            widen8<BF16>(slot >= 0 ? p.src[which][piece] : make_uint4(0, 0, 0, 0), x);
            q = quantise_row_int4<BF16, LANES>(x);
            if (slot < 0) continue;  // after the row's shuffles
            *reinterpret_cast<uint32_t *>(rec + off * (D / 2) + c * 4) = q.codes;
            if (c == 0)
                *reinterpret_cast<uint32_t *>(rec + (D / 2 << p.log2_block) + off * 4) = q.params;
            if (p.dst[which]) p.dst[which][piece] = read8_int4<BF16>(q.codes, q.params);
        }
    }
}

static pa_status int4_rows(bool read, Int4IoParams p, int num_tokens, const void *k_pool,
                           const void *v_pool, const int64_t *slots, int num_blocks,
                           int num_kv_heads, int head_dim, int block_size, pa_dtype dtype,
                           void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_INVALID;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if ((int64_t)num_tokens * num_kv_heads > 0x7fffffff) return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    if (!k_pool || !v_pool || !slots || !aligned16(k_pool) || !aligned16(v_pool))
        return PA_ERR_INVALID;
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.pool[0] = static_cast<uint8_t *>(const_cast<void *>(k_pool));
    p.pool[1] = static_cast<uint8_t *>(const_cast<void *>(v_pool));
    p.slots = slots;
    p.num_slots = (int64_t)num_blocks * block_size;
    p.rows = num_tokens * num_kv_heads;
    p.num_kv_heads = num_kv_heads;
    p.log2_block = block_size == 16 ? 4 : 5;
    const int rows_per_block = kInt4Threads / (head_dim / 8);
    const int64_t blocks = ((int64_t)p.rows + rows_per_block - 1) / rows_per_block;
    const int64_t cap = 16ll * (sm_count() > 0 ? sm_count() : 152);
    const dim3 grid((unsigned)(blocks < cap ? blocks : cap), 2);
    auto kern = int4_rows_kernel<false, 64, false>;
#define PA_CASE(BF, DD, RR) \
    if ((dtype == PA_BF16) == BF && head_dim == DD && read == RR) kern = int4_rows_kernel<BF, DD, RR>;
    PA_CASE(false, 64, true) PA_CASE(false, 128, false) PA_CASE(false, 128, true)
    PA_CASE(true, 64, false) PA_CASE(true, 64, true) PA_CASE(true, 128, false)
    PA_CASE(true, 128, true)
#undef PA_CASE
    kern<<<grid, kInt4Threads, 0, as_stream(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_int4_record_bytes(int head_dim, int block_size) {
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32)) return 0;
    return (size_t)block_size * (head_dim / 2 + 4);
}

pa_status pa_cache_write_int4(const void *k_new, const void *v_new, const int64_t *slot_mapping,
                              int num_tokens, void *k_pool, void *v_pool, int num_blocks,
                              int num_kv_heads, int head_dim, int block_size, void *k_out,
                              void *v_out, pa_dtype dtype, void *stream) {
    if (num_tokens > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new) ||
                           !k_out != !v_out || !aligned16(k_out) || !aligned16(v_out)))
        return PA_ERR_INVALID;
    Int4IoParams p = {};
    p.src[0] = static_cast<const uint4 *>(k_new);
    p.src[1] = static_cast<const uint4 *>(v_new);
    p.dst[0] = static_cast<uint4 *>(k_out);
    p.dst[1] = static_cast<uint4 *>(v_out);
    return int4_rows(false, p, num_tokens, k_pool, v_pool, slot_mapping, num_blocks, num_kv_heads,
                     head_dim, block_size, dtype, stream);
}

pa_status pa_cache_read_int4(void *k_out, void *v_out, const int64_t *slot_mapping, int num_tokens,
                             const void *k_pool, const void *v_pool, int num_blocks,
                             int num_kv_heads, int head_dim, int block_size, pa_dtype dtype,
                             void *stream) {
    if (num_tokens > 0 && (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)))
        return PA_ERR_INVALID;
    Int4IoParams p = {};
    p.dst[0] = static_cast<uint4 *>(k_out);
    p.dst[1] = static_cast<uint4 *>(v_out);
    return int4_rows(true, p, num_tokens, k_pool, v_pool, slot_mapping, num_blocks, num_kv_heads,
                     head_dim, block_size, dtype, stream);
}

}  // extern "C"
