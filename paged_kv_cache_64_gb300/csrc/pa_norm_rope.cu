// pa_qk_norm_rope: RMS norm of every query and key head, rotary positions and
// the cache write, in one pass over a token's heads.
//
//   y = x w / sqrt(mean x^2 + eps);  (a, b) -> (a c - b s, b c + a s)
//
// A head is D/16 consecutive lanes; lane c holds its chunks (8 elements, 16
// bytes) c and c + D/16.  The sum of squares is a shuffle sum.  With the whole
// head rotated by halves, a pair's elements then lie in one lane, as interleaved
// pairs always do; with a part of it rotated by halves they change places by
// shuffles.  A CTA works on one token, so the position's cosines and sines are
// loaded once a lane and kept for all its heads.  Arithmetic is on packed fp32
// pairs where it can be.  Bound by HBM: every element is read and written once
// (E4M3 and 4-bit pools: 1 and 0.53 bytes instead of 2 on the way out).
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
    int num_q_heads;
    int num_kv_heads;
    int rows_per_cta;        // heads of a token one CTA works on
    int log2_block;
    int64_t num_slots;
    int *err;
};

constexpr int kNormRopeThreads = 64;

// 8 fp32 values as four packed pairs.
struct Chunk {
    float2 p[4];
};

template <bool BF16>
__device__ __forceinline__ Chunk widen_chunk(uint4 v) {
    return {{widen2<BF16>(v.x), widen2<BF16>(v.y), widen2<BF16>(v.z), widen2<BF16>(v.w)}};
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow_chunk(const Chunk &x) {
    return make_uint4(narrow2<BF16>(x.p[0].x, x.p[0].y), narrow2<BF16>(x.p[1].x, x.p[1].y),
                      narrow2<BF16>(x.p[2].x, x.p[2].y), narrow2<BF16>(x.p[3].x, x.p[3].y));
}

__device__ __forceinline__ Chunk load_chunk(const float *src) {
    const float4 a = reinterpret_cast<const float4 *>(src)[0];
    const float4 b = reinterpret_cast<const float4 *>(src)[1];
    return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y),
             make_float2(b.z, b.w)}};
}

__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

// How a lane's chunks are rotated: interleaved pairs; halves of the whole head
// (chunk c with chunk c + D/16); halves of a part of it.
enum RopeKind { kRopePairs, kRopeWhole, kRopePart };

// CTAs an SM, at least: two warps of 64 registers a thread (16,411 tokens of 32 +
// 8 + 8 heads of 128: 69.6 us; four warps a CTA 71 to 73 us, 80 registers 77 us,
// 48 registers 76 us); up to 96 for the quantiser (78 us) and the shuffles of partly
// rotated heads (half the head 77 us, 105 with 64; seven eighths 80), which would
// spill much in 64.  Interleaved pairs keep 64 and spill 20 bytes: 71 us, 76 in 96.
template <int FMT, int ROPE>
constexpr int kNormRopeCtas = FMT == PA_KV_INT4 || ROPE == kRopePart ? 10 : 16;

template <bool BF16, int D, int FMT, int ROPE>
__global__ void __launch_bounds__(kNormRopeThreads, (kNormRopeCtas<FMT, ROPE>)) norm_rope_kernel(
    const __grid_constant__ NormRopeParams p) {
    constexpr int LANES = D / 16, GROUPS = kNormRopeThreads / LANES;
    const int c = threadIdx.x % LANES, g = threadIdx.x / LANES;
    const int64_t t = blockIdx.x;
    pdl_wait();
    const int nq = p.num_q_heads, nk = p.num_kv_heads, heads = nq + 2 * nk;
    const int first = blockIdx.y * p.rows_per_cta;
    const int last = min(first + p.rows_per_cta, heads);
    struct Row {
        uint4 v[2];
    };
    auto load = [&](int r) {
        Row x = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
        if (r < last) {
            const uint16_t *src = r < nq ? p.src[0] + t * p.stride[0] + (int64_t)r * D
                                  : r < nq + nk
                                      ? p.src[1] + t * p.stride[1] + (int64_t)(r - nq) * D
                                      : p.src[2] + t * p.stride[2] + (int64_t)(r - nq - nk) * D;
            x.v[0] = reinterpret_cast<const uint4 *>(src)[c];
            x.v[1] = reinterpret_cast<const uint4 *>(src)[c + LANES];
        }
        return x;
    };
    // heads ahead in flight: two where fewer CTAs share an SM and the quantiser
    // does not set the pace (half the head turned: 83 us for 98 with one)
    constexpr int AHEAD = kNormRopeCtas<FMT, ROPE> < 16 && FMT != PA_KV_INT4 ? 2 : 1;
    Row next[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) next[i] = load(first + i * GROUPS + g);
    const int64_t pos = p.positions[t];
    int64_t slot = p.slots[t];
    if (pos < 0 || pos >= p.num_positions) {  // the same for the whole CTA
        if (threadIdx.x == 0 && blockIdx.y == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        return;
    }
    if (slot >= p.num_slots) {
        if (threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        slot = -1;
    }
    const int64_t blk = slot >> p.log2_block;
    const int off = (int)slot & ((1 << p.log2_block) - 1);

    // Cosines and sines of the lane's chunks; 1 and 0 where nothing turns.
    // kRopePairs: of a chunk's four pairs, each twice, the sine as (-s, s);
    // kRopeWhole: of its eight pairs in cs[0], sn[0]; kRopePart: of each
    // chunk's eight elements, the sine with the sign of the partner's term.
    const int half = p.rotary_dim >> 1, hc = p.rotary_dim >> 4;  // hc: chunks in a half
    Chunk cs[2], sn[2];
    int partner[2] = {c, c};  // kRopePart: chunk that holds the pairs' other elements
    {
        const float *row = p.cos_sin + pos * p.rotary_dim;
        if constexpr (ROPE == kRopeWhole) {
            cs[0] = load_chunk(row + 8 * c);
            sn[0] = load_chunk(row + half + 8 * c);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int chunk = c + i * LANES;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cs[i].p[j] = make_float2(1.f, 1.f);
                    sn[i].p[j] = make_float2(0.f, 0.f);
                }
                partner[i] = chunk;
                if (chunk >= 2 * hc) continue;
                if constexpr (ROPE == kRopePairs) {
                    const float4 u = reinterpret_cast<const float4 *>(row)[chunk];
                    const float4 w = reinterpret_cast<const float4 *>(row + half)[chunk];
                    cs[i] = {{make_float2(u.x, u.x), make_float2(u.y, u.y), make_float2(u.z, u.z),
                              make_float2(u.w, u.w)}};
                    sn[i] = {{make_float2(-w.x, w.x), make_float2(-w.y, w.y), make_float2(-w.z, w.z),
                              make_float2(-w.w, w.w)}};
                } else {
                    const bool low = chunk < hc;
                    partner[i] = low ? chunk + hc : chunk - hc;
                    cs[i] = load_chunk(row + 8 * (low ? chunk : chunk - hc));
                    sn[i] = load_chunk(row + half + 8 * (low ? chunk : chunk - hc));
                    if (low) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) sn[i].p[j] = neg2(sn[i].p[j]);
                    }
                }
            }
        }
    }

    for (int r0 = first; r0 < last; r0 += GROUPS) {
        const int r = r0 + g;
        const bool live = r < last;
        const int kind = r < nq ? 0 : r < nq + nk ? 1 : 2;
        const Row raw = next[0];
        if (AHEAD > 1) next[0] = next[AHEAD - 1];
        next[AHEAD - 1] = load(r + AHEAD * GROUPS);
        uint4 y16[2] = {raw.v[0], raw.v[1]};
        if (__any_sync(kFullMask, live && kind < 2)) {
            Chunk x[2];
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[i] = widen_chunk<BF16>(raw.v[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = __ffma2_rn(x[i].p[j], x[i].p[j], ss);
            }
            float sum = ss.x + ss.y;
#pragma unroll
            for (int o = LANES / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
            const float inv = __frsqrt_rn(sum * (1.f / D) + p.eps);
            const float2 inv2 = make_float2(inv, inv);
            const uint4 *weight = kind == 0 ? p.weight[0] : p.weight[1];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Chunk w = widen_chunk<BF16>(weight[c + i * LANES]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i].p[j] = __fmul2_rn(__fmul2_rn(x[i].p[j], inv2), w.p[j]);
            }
            Chunk z[2];
            if constexpr (ROPE == kRopeWhole) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = x[0].p[j], b = x[1].p[j];
                    z[0].p[j] = __ffma2_rn(a, cs[0].p[j], neg2(__fmul2_rn(b, sn[0].p[j])));
                    z[1].p[j] = __ffma2_rn(b, cs[0].p[j], __fmul2_rn(a, sn[0].p[j]));
                }
            } else if constexpr (ROPE == kRopePairs) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = x[i].p[j];
                        z[i].p[j] = __ffma2_rn(a, cs[i].p[j],
                                               __fmul2_rn(make_float2(a.y, a.x), sn[i].p[j]));
                    }
            } else {
                // chunk k is half k / LANES of lane k % LANES
                const int base = (threadIdx.x & 31) - c;
                const int from0 = base + partner[0] % LANES, from1 = base + partner[1] % LANES;
                if (2 * hc <= LANES) {  // at most half the head turns: first halves only
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 q =
                            make_float2(__shfl_sync(kFullMask, x[0].p[j].x, from0),
                                        __shfl_sync(kFullMask, x[0].p[j].y, from0));
                        z[0].p[j] = __ffma2_rn(x[0].p[j], cs[0].p[j], __fmul2_rn(q, sn[0].p[j]));
                        z[1].p[j] = x[1].p[j];
                    }
                } else {
                    // a chunk of the second half turns with one of the first (where
                    // it does not turn its sine is 0)
                    auto both = [&](float a, float b, float *q0, float *q1) {
                        const float u = __shfl_sync(kFullMask, a, from0);
                        const float w = __shfl_sync(kFullMask, b, from0);
                        *q0 = partner[0] < LANES ? u : w;
                        *q1 = __shfl_sync(kFullMask, a, from1);
                    };
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 q0, q1;
                        both(x[0].p[j].x, x[1].p[j].x, &q0.x, &q1.x);
                        both(x[0].p[j].y, x[1].p[j].y, &q0.y, &q1.y);
                        z[0].p[j] = __ffma2_rn(x[0].p[j], cs[0].p[j], __fmul2_rn(q0, sn[0].p[j]));
                        z[1].p[j] = __ffma2_rn(x[1].p[j], cs[1].p[j], __fmul2_rn(q1, sn[1].p[j]));
                    }
                }
            }
            if (kind < 2) {
                y16[0] = narrow_chunk<BF16>(z[0]);
                y16[1] = narrow_chunk<BF16>(z[1]);
            }
        }
        if (live && kind == 0) {
            uint4 *to = reinterpret_cast<uint4 *>(p.q_out + t * p.q_out_stride + (int64_t)r * D);
            to[c] = y16[0];
            to[c + LANES] = y16[1];
        }
        const bool store = live && kind > 0 && slot >= 0;
        uint8_t *pool = kind == 1 ? p.pool[0] : p.pool[1];
        const int64_t rec = blk * nk + (r - (kind == 1 ? nq : nq + nk));
        const int64_t at = (rec << p.log2_block) + off;
        if constexpr (FMT == PA_KV_16BIT) {
            if (store) {
                uint4 *to = reinterpret_cast<uint4 *>(pool) + at * (D / 8);
                to[c] = y16[0];
                to[c + LANES] = y16[1];
            }
        } else if constexpr (FMT == PA_KV_E4M3) {
            if (store) {
                const uint4 q = quantize16_e4m3<BF16>(
                    y16[0], y16[1], kind == 1 ? p.inv_scale[0] : p.inv_scale[1]);
                uint2 *to = reinterpret_cast<uint2 *>(pool) + at * (D / 8);
                to[c] = make_uint2(q.x, q.y);
                to[c + LANES] = make_uint2(q.z, q.w);
            }
        } else {
            if (__any_sync(kFullMask, store)) {
                const Int4Row<2> q = quantise_row_int4<BF16, LANES, 2, false>(y16, nullptr);
                if (store) {
                    uint8_t *dst = pool + rec * int4_record_bytes<D>(1 << p.log2_block);
                    uint32_t *to = reinterpret_cast<uint32_t *>(dst + off * (D / 2));
                    to[c] = q.codes[0];
                    to[c + LANES] = q.codes[1];
                    if (c == 0)
                        *reinterpret_cast<uint32_t *>(dst + ((D / 2) << p.log2_block) + off * 4) =
                            q.params;
                }
            }
        }
    }
}

using NormRopeKernel = void (*)(const NormRopeParams);

template <bool BF16, int D, int FMT>
static NormRopeKernel rope_variant(int rope) {
    return rope == kRopePairs   ? norm_rope_kernel<BF16, D, FMT, kRopePairs>
           : rope == kRopeWhole ? norm_rope_kernel<BF16, D, FMT, kRopeWhole>
                                : norm_rope_kernel<BF16, D, FMT, kRopePart>;
}

template <bool BF16, int D>
static NormRopeKernel format_variant(int fmt, int rope) {
    return fmt == PA_KV_16BIT  ? rope_variant<BF16, D, PA_KV_16BIT>(rope)
           : fmt == PA_KV_E4M3 ? rope_variant<BF16, D, PA_KV_E4M3>(rope)
                               : rope_variant<BF16, D, PA_KV_INT4>(rope);
}

static NormRopeKernel pick_norm_rope(bool bf16, int D, int fmt, int rope) {
    if (D == 64) return bf16 ? format_variant<true, 64>(fmt, rope) : format_variant<false, 64>(fmt, rope);
    return bf16 ? format_variant<true, 128>(fmt, rope) : format_variant<false, 128>(fmt, rope);
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
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.log2_block = block_size == 16 ? 4 : 5;
    p.num_slots = (int64_t)num_blocks * block_size;
    const int groups = kNormRopeThreads / (head_dim / 16), heads = num_q_heads + 2 * num_kv_heads;
    // one CTA a token; tokens too few to fill the GPU are split over their heads
    int chunks = 1;
    const int most = (heads + groups - 1) / groups;
    while (chunks < most && (int64_t)num_tokens * chunks < 8ll * sm_count()) ++chunks;
    int per = (most + chunks - 1) / chunks;
    p.rows_per_cta = per * groups;
    const dim3 grid((unsigned)num_tokens, (unsigned)((most + per - 1) / per));
    if (grid.y > 65535) return PA_ERR_INVALID;
    const int rope = interleaved               ? kRopePairs
                     : rotary_dim == head_dim ? kRopeWhole
                                              : kRopePart;
    NormRopeKernel kern = pick_norm_rope(dtype == PA_BF16, head_dim, kv_format, rope);
    if (launch_pdl(kern, grid, dim3(kNormRopeThreads), 0, as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
