// The latent cache's rows: pa_latent_norm_rope (what lies between a layer's
// projections and its attention) and pa_cache_read_latent.
//
//   c = x w / sqrt(mean x^2 + eps) over a row's RANK values;
//   (a, b) -> (a c - b s, b c + a s) over its 64 rotary values and those of
//   every query head.
//
// A 16-byte chunk is 8 elements.  A rotary part is 8 chunks: lane j of four
// holds chunks j and j + 4, so that the pairs of either layout lie in one lane
// (halves: element i of chunk j with element i of chunk j + 4; interleaved:
// neighbours in a chunk), and the token's cosines and sines stay in its
// registers for all heads that it works on.  A row's latent part is a warp's:
// RANK / 256 chunks a lane, the sum of squares a shuffle sum.  Bound by HBM:
// every element is read and written once.
#include <cmath>
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kRope = 64;  // rotary values of a row and of a query head
constexpr int kLatentThreads = 64;

struct LatentRopeParams {
    uint16_t *q_out;
    const uint16_t *q;
    const uint16_t *latent;
    const uint4 *weight;
    const float *cos_sin;
    const int64_t *positions;
    const int64_t *slots;
    uint16_t *rows_out;  // or null
    uint16_t *pool;
    int64_t q_out_token, q_out_head, q_token, q_head, latent_token;  // steps, in elements
    int64_t num_slots;
    float eps;
    int num_positions;
    int num_heads;
    int heads_per_cta;
    int *err;
};

struct Vec8 {
    float v[8];
};

template <bool BF16>
__device__ __forceinline__ Vec8 widen8(uint4 w) {
    const float2 a = widen2<BF16>(w.x), b = widen2<BF16>(w.y), c = widen2<BF16>(w.z),
                 d = widen2<BF16>(w.w);
    return {{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y}};
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const Vec8 &x) {
    return make_uint4(narrow2<BF16>(x.v[0], x.v[1]), narrow2<BF16>(x.v[2], x.v[3]),
                      narrow2<BF16>(x.v[4], x.v[5]), narrow2<BF16>(x.v[6], x.v[7]));
}

// Chunks j and j + 4 of a rotary part, turned in place.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void turn(uint4 (&w)[2], const Vec8 &c, const Vec8 &s) {
    const Vec8 a = widen8<BF16>(w[0]), b = widen8<BF16>(w[1]);
    Vec8 x, y;
    if constexpr (PAIRS) {  // c, s: the four pairs of chunk j, then those of j + 4
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x.v[2 * i] = a.v[2 * i] * c.v[i] - a.v[2 * i + 1] * s.v[i];
            x.v[2 * i + 1] = a.v[2 * i + 1] * c.v[i] + a.v[2 * i] * s.v[i];
            y.v[2 * i] = b.v[2 * i] * c.v[4 + i] - b.v[2 * i + 1] * s.v[4 + i];
            y.v[2 * i + 1] = b.v[2 * i + 1] * c.v[4 + i] + b.v[2 * i] * s.v[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x.v[i] = a.v[i] * c.v[i] - b.v[i] * s.v[i];
            y.v[i] = b.v[i] * c.v[i] + a.v[i] * s.v[i];
        }
    }
    w[0] = narrow8<BF16>(x);
    w[1] = narrow8<BF16>(y);
}

// (18 CTAs an SM: 16,411 tokens of 32 heads in 33.7 us, 5.8 TB/s of the 195.6 MB that
// they have to move; 35.5 with 14, 36.9 with 20, 38.0 with CTAs of four warps, 36.4
// with a token's heads over two CTAs.)
template <bool BF16, int RANK, bool PAIRS>
__global__ void __launch_bounds__(kLatentThreads, 18) latent_norm_rope_kernel(
    const __grid_constant__ LatentRopeParams p) {
    constexpr int ROW = RANK + kRope, PER = RANK / 256;
    const int j = threadIdx.x & 3, g = threadIdx.x >> 2, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    pdl_wait();
    const int64_t pos = p.positions[t];
    // the first chunk of the CTA's heads is on its way while the table's row is
    const int first = blockIdx.y * p.heads_per_cta;
    const int last = min(first + p.heads_per_cta, p.num_heads);
    const uint16_t *src = p.q + t * p.q_token;
    uint4 next[2] = {};
    auto load = [&](int h) {
        if (h < last) {
            const uint4 *from = reinterpret_cast<const uint4 *>(src + h * p.q_head);
            next[0] = from[j];
            next[1] = from[j + 4];
        }
    };
    load(first + g);
    const bool row_cta = blockIdx.y == 0 && threadIdx.x < 32;  // the warp that has the row
    uint4 x[PER], pe[2] = {};
    int64_t slot = -1;
    if (row_cta) {
        const uint4 *from = reinterpret_cast<const uint4 *>(p.latent + t * p.latent_token);
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = from[lane + 32 * i];
        pe[0] = from[RANK / 8 + j];
        pe[1] = from[RANK / 8 + j + 4];
        slot = p.slots[t];
    }
    if (pos < 0 || pos >= p.num_positions) {  // the same for the whole CTA
        if (threadIdx.x == 0 && blockIdx.y == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        return;
    }
    Vec8 c, s;
    {
        const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + pos * kRope);
        const int lo = PAIRS ? j : 2 * j, hi = PAIRS ? j + 4 : 2 * j + 1;
        const float4 c0 = row[lo], c1 = row[hi], s0 = row[8 + lo], s1 = row[8 + hi];
        c = {{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}};
        s = {{s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w}};
    }
    if (row_cta) {
        if (slot >= p.num_slots) {
            if (lane == 0) record_error(p.err, PA_ERR_BAD_INDEX);
            slot = -1;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const Vec8 v = widen8<BF16>(x[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(v.v[k], v.v[k], sum);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        const float inv = __frsqrt_rn(sum * (1.f / RANK) + p.eps);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            Vec8 v = widen8<BF16>(x[i]);
            const Vec8 w = widen8<BF16>(p.weight[lane + 32 * i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) v.v[k] = v.v[k] * inv * w.v[k];
            x[i] = narrow8<BF16>(v);
        }
        turn<BF16, PAIRS>(pe, c, s);
        auto store = [&](uint16_t *row) {
            uint4 *to = reinterpret_cast<uint4 *>(row);
#pragma unroll
            for (int i = 0; i < PER; ++i) to[lane + 32 * i] = x[i];
            if (lane < 4) {
                to[RANK / 8 + j] = pe[0];
                to[RANK / 8 + j + 4] = pe[1];
            }
        };
        if (slot >= 0) store(p.pool + slot * ROW);
        if (p.rows_out) store(p.rows_out + t * ROW);
    }
    uint16_t *dst = p.q_out + t * p.q_out_token;
    for (int h = first + g; h < last; h += kLatentThreads / 4) {
        uint4 w[2] = {next[0], next[1]};
        load(h + kLatentThreads / 4);
        turn<BF16, PAIRS>(w, c, s);
        uint4 *to = reinterpret_cast<uint4 *>(dst + h * p.q_out_head);
        to[j] = w[0];
        to[j + 4] = w[1];
    }
}

using LatentRopeKernel = void (*)(const LatentRopeParams);

template <bool BF16, int RANK>
static LatentRopeKernel latent_rope_variant(bool pairs) {
    return pairs ? latent_norm_rope_kernel<BF16, RANK, true>
                 : latent_norm_rope_kernel<BF16, RANK, false>;
}

// Rows out of the pool: thread-linear over the rows' 16-byte chunks, four loads
// in flight a thread.  Bound by HBM: a row is read and written once (131,073 rows of
// 1,152 bytes in 46.0 us, 6.6 TB/s; eight loads in flight, or half as many threads a
// CTA, take as long).
constexpr int kReadThreads = 256, kReadPer = 4;

template <int CHUNKS>
__global__ void __launch_bounds__(kReadThreads) latent_read_kernel(
    uint4 *out, const uint4 *pool, const int64_t *slots, int64_t total, int64_t num_slots, int *err) {
    pdl_wait();
    const int64_t i0 = (int64_t)blockIdx.x * (kReadThreads * kReadPer) + threadIdx.x;
    uint4 v[kReadPer];
    int64_t slot[kReadPer];
#pragma unroll
    for (int k = 0; k < kReadPer; ++k) {
        const int64_t i = i0 + k * kReadThreads;
        slot[k] = i < total ? slots[i / CHUNKS] : -1;
    }
#pragma unroll
    for (int k = 0; k < kReadPer; ++k) {
        const int64_t i = i0 + k * kReadThreads;
        if (slot[k] >= num_slots) {
            record_error(err, PA_ERR_BAD_INDEX);
            slot[k] = -1;
        }
        if (slot[k] >= 0) v[k] = pool[slot[k] * CHUNKS + i % CHUNKS];
    }
#pragma unroll
    for (int k = 0; k < kReadPer; ++k)
        if (slot[k] >= 0) out[i0 + k * kReadThreads] = v[k];
}

static bool latent_shape(int rank, int block_size) {
    return (rank == 256 || rank == 512) &&
           (block_size == 16 || block_size == 32 || block_size == 64);
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_latent_norm_rope(
    void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, const void *q,
    int64_t q_token_stride, int64_t q_head_stride, const void *latent, int64_t latent_stride,
    const void *weight, float eps, const float *cos_sin, int num_positions, int interleaved,
    const int64_t *positions, const int64_t *slot_mapping, int num_tokens, void *rows_out,
    void *pool, int num_blocks, int num_heads, int rank, int block_size, pa_dtype dtype,
    void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || num_heads <= 0 || num_positions <= 0 ||
        !(eps >= 0.f) || !std::isfinite(eps) || (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID;
    if (!latent_shape(rank, block_size)) return PA_ERR_UNSUPPORTED;
    const int64_t steps[] = {q_out_token_stride, q_out_head_stride, q_token_stride, q_head_stride};
    for (int64_t s : steps)
        if (s < kRope || s % 8 || s > (1ll << 40)) return PA_ERR_INVALID;
    if (latent_stride < rank + kRope || latent_stride % 8 || num_heads > 0x7fffff)
        return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    const void *ptrs[] = {q_out, q, latent, weight, cos_sin, pool};
    for (const void *ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return PA_ERR_INVALID;
    if ((rows_out && !aligned16(rows_out)) || !positions || !slot_mapping) return PA_ERR_INVALID;
    LatentRopeParams p = {};
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.q = static_cast<const uint16_t *>(q);
    p.latent = static_cast<const uint16_t *>(latent);
    p.weight = static_cast<const uint4 *>(weight);
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slot_mapping;
    p.rows_out = static_cast<uint16_t *>(rows_out);
    p.pool = static_cast<uint16_t *>(pool);
    p.q_out_token = q_out_token_stride;
    p.q_out_head = q_out_head_stride;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.latent_token = latent_stride;
    p.num_slots = (int64_t)num_blocks * block_size;
    p.eps = eps;
    p.num_positions = num_positions;
    p.num_heads = num_heads;
    // one CTA a token; tokens too few to fill the GPU are split over their heads
    const int groups = kLatentThreads / 4, most = (num_heads + groups - 1) / groups;
    int chunks = 1;
    while (chunks < most && (int64_t)num_tokens * chunks < 8ll * sm_count()) ++chunks;
    const int per = (most + chunks - 1) / chunks;
    p.heads_per_cta = per * groups;
    const dim3 grid((unsigned)num_tokens, (unsigned)((most + per - 1) / per));
    if (grid.y > 65535) return PA_ERR_INVALID;
    const bool pairs = interleaved != 0;
    LatentRopeKernel kern =
        dtype == PA_BF16
            ? (rank == 512 ? latent_rope_variant<true, 512>(pairs) : latent_rope_variant<true, 256>(pairs))
            : (rank == 512 ? latent_rope_variant<false, 512>(pairs)
                           : latent_rope_variant<false, 256>(pairs));
    if (launch_pdl(kern, grid, dim3(kLatentThreads), 0, as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_cache_read_latent(void *rows_out, const int64_t *slot_mapping,
                                          int num_tokens, const void *pool, int num_blocks,
                                          int rank, int block_size, pa_dtype dtype, void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID;
    if (!latent_shape(rank, block_size)) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!rows_out || !pool || !slot_mapping || !aligned16(rows_out) || !aligned16(pool))
        return PA_ERR_INVALID;
    int *err = error_word();
    if (!err) return PA_ERR_CUDA;
    const int chunks = (rank + kRope) / 8;
    const int64_t total = (int64_t)num_tokens * chunks;
    const int64_t ctas = (total + kReadThreads * kReadPer - 1) / (kReadThreads * kReadPer);
    auto kern = rank == 512 ? latent_read_kernel<(512 + kRope) / 8> : latent_read_kernel<(256 + kRope) / 8>;
    if (launch_pdl(kern, dim3((unsigned)ctas), dim3(kReadThreads), 0, as_stream(stream),
                   static_cast<uint4 *>(rows_out), static_cast<const uint4 *>(pool), slot_mapping,
                   total, (int64_t)num_blocks * block_size, err) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
