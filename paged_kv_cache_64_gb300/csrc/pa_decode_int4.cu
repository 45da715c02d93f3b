// Decode attention over 4-bit pools (pa_decode_int4), simplest form: a warp a
// position, a lane D/32 dimensions, fp32 throughout.
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kInt4Warps = 4;
constexpr int kInt4MaxG = 8;

template <int D>
struct Int4Shape {
    static constexpr int RED_BYTES = kInt4Warps * kInt4MaxG * (D + 2) * 4;
    static constexpr int SMEM_BYTES = RED_BYTES;
};

template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kInt4Warps) decode_int4_kernel(const DecodeParams p) {
    constexpr int V = D / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int chunk = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
    const int L = item_len(p, seq, threadIdx.x == 0 && chunk == 0 && kvh == 0);
    const int G = p.group, P = p.partition_tokens;
    const int nparts = L == 0 ? 0 : (L - 1) / P + 1;
    const int start = chunk * P;
    uint16_t *out = static_cast<uint16_t *>(p.out) + ((int64_t)seq * p.num_q_heads + kvh * G) * D;
    if (L == 0) {
        if (chunk == 0)
            for (int i = threadIdx.x; i < G * D; i += blockDim.x) out[i] = 0;
        return;
    }
    if (chunk >= nparts) return;
    const int end = L < start + P ? L : start + P;

    float q[kInt4MaxG][V], acc[kInt4MaxG][V], m[kInt4MaxG], l[kInt4MaxG];
#pragma unroll
    for (int g = 0; g < kInt4MaxG; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            acc[g][i] = 0.f;
            q[g][i] = g < G ? from16<BF16>(p.q[((int64_t)seq * p.num_q_heads + kvh * G + g) * D +
                                              lane * V + i]) * p.scale_log2
                            : 0.f;
        }
    }
    const int rec_bytes = int4_record_bytes<D>(p.block_size);
    const uint8_t *pools[2] = {reinterpret_cast<const uint8_t *>(p.k_pool),
                               reinterpret_cast<const uint8_t *>(p.v_pool)};
    for (int pos = start + warp; pos < end; pos += kInt4Warps) {
        const int phys = seq_table(p, seq)[pos >> p.log2_block];
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
            if (lane == 0) record_error(p.err, PA_ERR_BAD_INDEX);
            continue;
        }
        const int off = pos & (p.block_size - 1);
        float x[2][V];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint8_t *rec = pools[w] + ((int64_t)phys * p.num_kv_heads + kvh) * rec_bytes;
            const uint32_t par =
                *reinterpret_cast<const uint32_t *>(rec + p.block_size * (D / 2) + off * 4);
            const float s = from16<BF16>(par & 0xffffu), lo = from16<BF16>(par >> 16);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const int b = rec[off * (D / 2) + lane * (V / 2) + i];
                x[w][2 * i] = fmaf(s, (float)(b & 15), lo);
                x[w][2 * i + 1] = fmaf(s, (float)(b >> 4), lo);
            }
        }
#pragma unroll
        for (int g = 0; g < kInt4MaxG; ++g) {
            if (g >= G) continue;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) s += q[g][i] * x[0][i];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
            const float mn = fmaxf(m[g], s), a = fast_exp2(m[g] - mn), w = fast_exp2(s - mn);
            m[g] = mn;
            l[g] = l[g] * a + w;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[g][i] = acc[g][i] * a + w * x[1][i];
        }
    }

    float *red = reinterpret_cast<float *>(smem);                 // [W][8][D]
    float *red_m = red + kInt4Warps * kInt4MaxG * D, *red_l = red_m + kInt4Warps * kInt4MaxG;
#pragma unroll
    for (int g = 0; g < kInt4MaxG; ++g) {
#pragma unroll
        for (int i = 0; i < V; ++i) red[(warp * kInt4MaxG + g) * D + lane * V + i] = acc[g][i];
        if (lane == 0) {
            red_m[warp * kInt4MaxG + g] = m[g];
            red_l[warp * kInt4MaxG + g] = l[g];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * (D / 2); i += blockDim.x) {
        const int g = i / (D / 2), x0 = i % (D / 2) * 2;
        float M = -INFINITY;
        for (int w = 0; w < kInt4Warps; ++w) M = fmaxf(M, red_m[w * kInt4MaxG + g]);
        float lsum = 0.f, o0 = 0.f, o1 = 0.f;
        for (int w = 0; w < kInt4Warps; ++w) {
            const int at = w * kInt4MaxG + g;
            const float f = red_m[at] == -INFINITY ? 0.f : fast_exp2(red_m[at] - M);
            lsum += f * red_l[at];
            o0 += f * red[at * D + x0];
            o1 += f * red[at * D + x0 + 1];
        }
        const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
        if (nparts == 1) {
            *reinterpret_cast<uint32_t *>(out + g * D + x0) = narrow2<BF16>(o0 * inv, o1 * inv);
        } else {
            const int64_t row = part_row(p, seq, kvh * G + g, chunk);
            if (x0 == 0) {
                p.part_m[row] = M;
                p.part_l[row] = lsum;
            }
            *reinterpret_cast<float2 *>(p.part_o + row * D + x0) = make_float2(o0 * inv, o1 * inv);
        }
    }
    if (nparts > 1 && p.counters != nullptr)
        finish_item<BF16, D>(p, seq, kvh, nparts, chunk, nparts, false,
                             reinterpret_cast<float *>(smem), Int4Shape<D>::SMEM_BYTES);
}

using Int4Kernel = void (*)(const DecodeParams);

static Int4Kernel pick_int4(bool bf16, int D, int *smem) {
    *smem = D == 64 ? Int4Shape<64>::SMEM_BYTES : Int4Shape<128>::SMEM_BYTES;
    if (D == 64) return bf16 ? decode_int4_kernel<true, 64> : decode_int4_kernel<false, 64>;
    return bf16 ? decode_int4_kernel<true, 128> : decode_int4_kernel<false, 128>;
}

int int4_ctas_per_sm(bool bf16, int head_dim) {
    int smem = 0, n = 0;
    Int4Kernel k = pick_int4(bf16, head_dim, &smem);
    if (!ensure_smem_attr(reinterpret_cast<const void *>(k), smem)) return 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, 32 * kInt4Warps, smem) != cudaSuccess)
        return 1;
    return n > 0 ? n : 1;
}

pa_status launch_decode_int4(const DecodeParams &prm, bool bf16, int head_dim, int num_partitions,
                             int num_kv_heads, int num_seqs, cudaStream_t stream) {
    if (num_seqs == 0) return PA_OK;
    int smem = 0;
    Int4Kernel k = pick_int4(bf16, head_dim, &smem);
    if (!ensure_smem_attr(reinterpret_cast<const void *>(k), smem)) return PA_ERR_CUDA;
    const dim3 grid((unsigned)num_partitions, (unsigned)num_kv_heads, (unsigned)num_seqs);
    if (launch_pdl(k, grid, dim3(32 * kInt4Warps), (size_t)smem, stream, prm) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
