// pa_qk_norm_rope: RMS norm of every query and key head, rotary positions and
// the cache write, in one pass over a token's heads.
//
//   y = x w / sqrt(mean x^2 + eps);  (a, b) -> (a c - b s, b c + a s)
//
// A head is D/8 consecutive lanes, 8 elements (16 bytes) a lane; the sum of
// squares is a shuffle sum over them.  Rotated pairs that lie D apart sit in
// lanes rotary_dim / 16 apart and change places by shuffles; interleaved pairs
// sit in one lane.  A CTA works on one token, so the position's cosines and
// sines are loaded once a lane and kept for all its heads.  Bound by HBM:
// every element is read and written once (E4M3 and 4-bit pools: 1 and 0.53
// bytes instead of 2 on the way out).
#include <cmath>
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

struct NormRopeParams {
    const uint16_t *src[3];  // q, k, v
    int64_t stride[3];       // elements from a token to the next
    uint16_t *q_out;
    int64_t q_out_stride;
    const uint4 *weight[2];  // q, k
    const float *cos_sin;
    const int64_t *positions;
    const int64_t *slots;
    uint8_t *pool[2];        // K, V
    float inv_scale[2];      // E4M3: fl32(1 / scale)
    float eps;
    int num_positions;
    int rotary_dim;
    int interleaved;
    int num_q_heads;
    int num_kv_heads;
    int rows_per_cta;        // heads of a token one CTA works on
    int log2_block;
    int64_t num_slots;
    int *err;
};

constexpr int kNormRopeThreads = 128;

template <bool BF16, int D, int FMT>
__global__ void __launch_bounds__(kNormRopeThreads) norm_rope_kernel(const NormRopeParams p) {
    constexpr int LANES = D / 8, GROUPS = kNormRopeThreads / LANES;
    const int c = threadIdx.x % LANES, g = threadIdx.x / LANES;
    const int64_t t = blockIdx.x;
    pdl_wait();
    const int64_t pos = p.positions[t];
    int64_t slot = p.slots[t];
    if (pos < 0 || pos >= p.num_positions) {  // the same for the whole CTA
        if (threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        return;
    }
    if (slot >= p.num_slots) {
        if (threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        slot = -1;
    }
    const int64_t blk = slot >> p.log2_block;
    const int off = (int)(slot & ((1 << p.log2_block) - 1));

    // this lane's cosines and sines: of its 8 elements' angles (halves: the sine
    // with the sign of the partner's term), or of its four pairs (interleaved);
    // 1 and 0 where nothing turns
    const int half = p.rotary_dim >> 1, hc = p.rotary_dim >> 4;  // hc: lanes in a half
    const bool turns = c < 2 * hc;
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (turns) {
        const float *row = p.cos_sin + pos * p.rotary_dim;
        const float *a = row + (p.interleaved ? 4 * c : 8 * (c < hc ? c : c - hc));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i && p.interleaved) break;
            const float4 u = reinterpret_cast<const float4 *>(a)[i];
            const float4 w = reinterpret_cast<const float4 *>(a + half)[i];
            cs[4 * i] = u.x; cs[4 * i + 1] = u.y; cs[4 * i + 2] = u.z; cs[4 * i + 3] = u.w;
            sn[4 * i] = w.x; sn[4 * i + 1] = w.y; sn[4 * i + 2] = w.z; sn[4 * i + 3] = w.w;
        }
        if (!p.interleaved && c < hc) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
        }
    }
    // lane that holds the other element of a pair (itself where nothing turns)
    const int partner = (threadIdx.x & 31) + (turns ? (c < hc ? hc : -hc) : 0);

    const int nq = p.num_q_heads, nk = p.num_kv_heads, heads = nq + 2 * nk;
    const int first = blockIdx.y * p.rows_per_cta;
    const int last = min(first + p.rows_per_cta, heads);
    auto kind_of = [&](int r) { return r < nq ? 0 : r < nq + nk ? 1 : 2; };
    auto load = [&](int r) {
        if (r >= last) return make_uint4(0, 0, 0, 0);
        const int kind = kind_of(r), head = r - (kind > 0 ? nq : 0) - (kind > 1 ? nk : 0);
        return reinterpret_cast<const uint4 *>(p.src[kind] + t * p.stride[kind] +
                                               (int64_t)head * D)[c];
    };
    // two heads ahead in flight
    uint4 next[2] = {load(first + g), load(first + GROUPS + g)};
    for (int r0 = first; r0 < last; r0 += GROUPS) {
        const int r = r0 + g;
        const bool live = r < last;
        const int kind = kind_of(r), head = r - (kind > 0 ? nq : 0) - (kind > 1 ? nk : 0);
        const uint4 raw = next[0];
        next[0] = next[1];
        next[1] = load(r + 2 * GROUPS);
        uint4 y16 = raw;
        if (__any_sync(kFullMask, live && kind < 2)) {
            float x[8], w[8];
            widen8<BF16>(raw, x);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
            for (int o = LANES / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
            widen8<BF16>(p.weight[kind == 0 ? 0 : 1][c], w);
            const float inv = __frsqrt_rn(ss * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
            float z[8];
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    z[2 * i] = a * cs[i] - b * sn[i];
                    z[2 * i + 1] = b * cs[i] + a * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[i] = x[i] * cs[i] + __shfl_sync(kFullMask, x[i], partner) * sn[i];
            }
            if (kind < 2)
                y16 = make_uint4(narrow2<BF16>(z[0], z[1]), narrow2<BF16>(z[2], z[3]),
                                 narrow2<BF16>(z[4], z[5]), narrow2<BF16>(z[6], z[7]));
        }
        const bool store = live && kind > 0 && slot >= 0;
        if (live && kind == 0)
            reinterpret_cast<uint4 *>(p.q_out + t * p.q_out_stride + (int64_t)head * D)[c] = y16;
        uint8_t *pool = p.pool[kind == 2];
        const int64_t rec = blk * nk + head;
        const int64_t at = (rec << p.log2_block) + off;
        if constexpr (FMT == PA_KV_16BIT) {
            if (store) reinterpret_cast<uint4 *>(pool)[at * LANES + c] = y16;
        } else if constexpr (FMT == PA_KV_E4M3) {
            if (store) {
                const uint4 q = quantize16_e4m3<BF16>(y16, y16, p.inv_scale[kind == 2]);
                reinterpret_cast<uint2 *>(pool)[at * LANES + c] = make_uint2(q.x, q.y);
            }
        } else {
            if (__any_sync(kFullMask, store)) {
                const uint4 row[1] = {y16};
                const Int4Row<1> q = quantise_row_int4<BF16, LANES, 1>(row);
                if (store) {
                    uint8_t *dst = pool + rec * int4_record_bytes<D>(1 << p.log2_block);
                    *reinterpret_cast<uint32_t *>(dst + off * (D / 2) + c * 4) = q.codes[0];
                    if (c == 0)
                        *reinterpret_cast<uint32_t *>(dst + ((D / 2) << p.log2_block) + off * 4) =
                            q.params;
                }
            }
        }
    }
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_qk_norm_rope(
    void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k,
    int64_t k_stride, const void *v, int64_t v_stride, const void *q_weight, const void *k_weight,
    float eps, const float *cos_sin, int num_positions, int rotary_dim, int interleaved,
    const int64_t *positions, const int64_t *slot_mapping, int num_tokens, void *k_pool,
    void *v_pool, int num_blocks, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    pa_kv_format kv_format, float k_scale, float v_scale, pa_dtype dtype, void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_positions <= 0 || num_q_heads % num_kv_heads || !(eps >= 0.f) || !std::isfinite(eps))
        return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_INVALID;
    if (kv_format != PA_KV_16BIT && kv_format != PA_KV_E4M3 && kv_format != PA_KV_INT4)
        return PA_ERR_INVALID;
    if (kv_format == PA_KV_E4M3 && (!(k_scale > 0.f) || !(v_scale > 0.f) ||
                                    !std::isfinite(k_scale) || !std::isfinite(v_scale)))
        return PA_ERR_INVALID;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16) return PA_ERR_UNSUPPORTED;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (q_out_stride < q_row || q_stride < q_row || k_stride < kv_row || v_stride < kv_row ||
        q_out_stride % 8 || q_stride % 8 || k_stride % 8 || v_stride % 8)
        return PA_ERR_INVALID;
    if ((int64_t)num_q_heads + 2ll * num_kv_heads > 0x7fffff) return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    const void *ptrs[] = {q_out, q, k, v, q_weight, k_weight, cos_sin, k_pool, v_pool};
    for (const void *ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return PA_ERR_INVALID;
    if (!positions || !slot_mapping) return PA_ERR_INVALID;
    NormRopeParams p = {};
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.src[0] = static_cast<const uint16_t *>(q);
    p.src[1] = static_cast<const uint16_t *>(k);
    p.src[2] = static_cast<const uint16_t *>(v);
    p.stride[0] = q_stride;
    p.stride[1] = k_stride;
    p.stride[2] = v_stride;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.q_out_stride = q_out_stride;
    p.weight[0] = static_cast<const uint4 *>(q_weight);
    p.weight[1] = static_cast<const uint4 *>(k_weight);
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slot_mapping;
    p.pool[0] = static_cast<uint8_t *>(k_pool);
    p.pool[1] = static_cast<uint8_t *>(v_pool);
    p.inv_scale[0] = 1.0f / k_scale;
    p.inv_scale[1] = 1.0f / v_scale;
    p.eps = eps;
    p.num_positions = num_positions;
    p.rotary_dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.log2_block = block_size == 16 ? 4 : 5;
    p.num_slots = (int64_t)num_blocks * block_size;
    const int groups = kNormRopeThreads / (head_dim / 8), heads = num_q_heads + 2 * num_kv_heads;
    // one CTA a token; tokens too few to fill the GPU are split over their heads
    int chunks = 1;
    const int most = (heads + groups - 1) / groups;
    while (chunks < most && (int64_t)num_tokens * chunks < 8ll * sm_count()) ++chunks;
    int per = (most + chunks - 1) / chunks;
    p.rows_per_cta = per * groups;
    const dim3 grid((unsigned)num_tokens, (unsigned)((most + per - 1) / per));
    if (grid.y > 65535) return PA_ERR_INVALID;
    auto kern = norm_rope_kernel<false, 64, PA_KV_16BIT>;
#define PA_CASE(BF, DD, FF)                                                      \
    if ((dtype == PA_BF16) == BF && head_dim == DD && kv_format == FF)           \
        kern = norm_rope_kernel<BF, DD, FF>;
#define PA_CASES(FF) PA_CASE(false, 64, FF) PA_CASE(false, 128, FF) PA_CASE(true, 64, FF) \
    PA_CASE(true, 128, FF)
    PA_CASES(PA_KV_16BIT) PA_CASES(PA_KV_E4M3) PA_CASES(PA_KV_INT4)
#undef PA_CASES
#undef PA_CASE
    if (launch_pdl(kern, grid, dim3(kNormRopeThreads), 0, as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
