// pa_cache_write_int4 and pa_cache_read_int4: rows into and out of paged
// 4-bit pools (see pa_int4.cuh for the format).
//
// A row of D values is D/16 consecutive lanes, 16 elements (32 bytes of 16-bit
// values, 8 bytes of codes) a lane, so a warp reads and writes whole rows.
// Bound by HBM: 2 bytes an element on the 16-bit side, 0.53 (D = 128) or 0.56
// (D = 64) in the pool.  A write forms the stored values whether or not they are
// asked for: 40,003 tokens of 8 heads of 128 take 61 us with them (floor 54) and 55
// without (floor 31).
#include <cstdint>

#include "pa_decode.cuh"
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
    // row / num_kv_heads = (row * magic) >> (32 + shift) for row < 2^31 (one
    // head: magic 0)
    uint32_t magic;
    int shift;
    int log2_block;
    int *err;
};

constexpr int kInt4Threads = 256;
// Two rows a lane in flight, both ways.  Measured for 8 heads of 128: reading
// 65,537 tokens 58 us as one wave of 6 CTAs an SM, 61 us as several waves or with
// four rows; writing 40,003 tokens 61 us in 64 registers (4 CTAs an SM) over
// several waves, 62 us as one, 67 us in 74 registers.
constexpr int kInt4Unroll = 2;

// blockIdx.y: 0 K, 1 V.  READ: pool -> values; otherwise values -> pool, and
// the stored values out when dst is given.
template <bool BF16, int D, bool READ>
__global__ void __launch_bounds__(kInt4Threads, READ ? 6 : 4) int4_rows_kernel(const Int4IoParams p) {
    pdl_wait();
    constexpr int LANES = D / 16, ROWS = kInt4Threads / LANES, U = kInt4Unroll;
    const int which = blockIdx.y, c = threadIdx.x % LANES;
    const uint4 *src = which ? p.src[1] : p.src[0];
    uint4 *dst = which ? p.dst[1] : p.dst[0];
    uint8_t *pool = which ? p.pool[1] : p.pool[0];
    const int block = 1 << p.log2_block, record = int4_record_bytes<D>(block);
    for (int64_t r0 = (int64_t)blockIdx.x * (ROWS * U); r0 < p.rows;
         r0 += (int64_t)gridDim.x * (ROWS * U)) {
        int64_t slot[U];
        int row[U], head[U];
        uint4 raw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * ROWS + threadIdx.x / LANES;
            row[u] = r < p.rows ? (int)r : -1;
            if (!READ) raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            slot[u] = -1;
            if (row[u] < 0) continue;
            const int t = p.magic ? (int)(__umulhi((uint32_t)row[u], p.magic) >> p.shift) : row[u];
            head[u] = row[u] - t * p.num_kv_heads;
            slot[u] = p.slots[t];
            if (!READ) {  // also of skipped tokens: not to wait for the slot
                const uint4 *from = src + (int64_t)row[u] * (D / 8) + 2 * c;
                raw[u][0] = from[0];
                raw[u][1] = from[1];
            }
        }
        uint2 q[U];
        uint32_t sm[U];
        uint8_t *codes[U], *pair[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (slot[u] >= p.num_slots) {
                if (c == 0) record_error(p.err, PA_ERR_BAD_INDEX);
                slot[u] = -1;
            }
            if (slot[u] < 0) continue;
            const int off = (int)slot[u] & (block - 1), blk = (int)(slot[u] >> p.log2_block);
            uint8_t *rec = pool + ((int64_t)blk * p.num_kv_heads + head[u]) * record;
            codes[u] = rec + off * (D / 2) + c * 8;
            pair[u] = rec + block * (D / 2) + off * 4;
            if (READ) {
                q[u] = *reinterpret_cast<const uint2 *>(codes[u]);
                sm[u] = *reinterpret_cast<const uint32_t *>(pair[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 y[2];
            if constexpr (READ) {
                if (slot[u] < 0) continue;
                y[0] = read8_int4<BF16>(q[u].x, sm[u]);
                y[1] = read8_int4<BF16>(q[u].y, sm[u]);
            } else {
                const Int4Row<2> z = quantise_row_int4<BF16, LANES, 2, true>(raw[u], y);
                if (slot[u] < 0) continue;  // after the row's shuffles
                *reinterpret_cast<uint2 *>(codes[u]) = make_uint2(z.codes[0], z.codes[1]);
                if (c == 0) *reinterpret_cast<uint32_t *>(pair[u]) = z.params;
            }
            if (READ || dst) {
                uint4 *to = dst + (int64_t)row[u] * (D / 8) + 2 * c;
                to[0] = y[0];
                to[1] = y[1];
            }
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
    if (num_kv_heads > 1) {
        // l = ceil(log2 H), magic = ceil(2^(31 + l) / H) < 2^32: exact below 2^31
        int l = 1;
        while ((1ll << l) < num_kv_heads) ++l;
        p.magic = (uint32_t)(((1ull << (31 + l)) + num_kv_heads - 1) / num_kv_heads);
        p.shift = l - 1;
    }
    p.log2_block = block_size == 16 ? 4 : 5;
    const int rows_per_block = kInt4Threads / (head_dim / 16) * kInt4Unroll;
    const int64_t blocks = ((int64_t)p.rows + rows_per_block - 1) / rows_per_block;
    const int64_t cap = (read ? 3ll : 16ll) * (sm_count() > 0 ? sm_count() : 152);  // for K, for V
    const dim3 grid((unsigned)(blocks < cap ? blocks : cap), 2);
    auto kern = int4_rows_kernel<false, 64, false>;
#define PA_CASE(BF, DD, RR) \
    if ((dtype == PA_BF16) == BF && head_dim == DD && read == RR) kern = int4_rows_kernel<BF, DD, RR>;
    PA_CASE(false, 64, true) PA_CASE(false, 128, false) PA_CASE(false, 128, true)
    PA_CASE(true, 64, false) PA_CASE(true, 64, true) PA_CASE(true, 128, false)
    PA_CASE(true, 128, true)
#undef PA_CASE
    if (launch_pdl(kern, grid, dim3(kInt4Threads), 0, as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
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
