// pa_prefill_latent: attention of ragged prompts in the expanded form of latent
// attention.  The simplest form: one CTA a (query, head), 32 keys a step on
// CUDA cores.
#include <cmath>
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kRope = 64, kNope = 128, kValue = 128;

struct PrefillLatentParams {
    uint16_t *out;
    const uint16_t *q, *k, *v, *k_pe;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, k_pe_token;
    const int32_t *q_starts, *k_starts;
    int num_seqs, total_q, total_k, max_q, num_heads, causal;
    float scale_log2;
    int *err;
};

template <bool BF16>
__global__ void __launch_bounds__(128) prefill_latent_kernel(
    const __grid_constant__ PrefillLatentParams p) {
    constexpr int TILE = 32;
    __shared__ float q[kNope + kRope], score[TILE];
    pdl_wait();
    const int i = blockIdx.x, h = blockIdx.y, seq = blockIdx.z, warp = threadIdx.x >> 5,
              lane = threadIdx.x & 31;
    const int q0 = p.q_starts[seq], n_q = p.q_starts[seq + 1] - q0;
    const int k0 = p.k_starts[seq], n_k = p.k_starts[seq + 1] - k0;
    if (q0 < 0 || n_q < 0 || n_q > p.max_q || n_q > p.total_q - q0 || k0 < 0 || n_k < 0 ||
        n_k > p.total_k - k0) {
        if (threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        return;
    }
    if (i >= n_q) return;
    const uint16_t *src = p.q + (int64_t)(q0 + i) * p.q_token + h * p.q_head;
    for (int c = threadIdx.x; c < kNope + kRope; c += 128) q[c] = widen2<BF16>(src[c]).x * p.scale_log2;
    const int L = p.causal ? max(0, n_k - n_q + i + 1) : n_k;
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int t = 0; t < L; t += TILE) {
        const int n = min(TILE, L - t);
        __syncthreads();
        for (int j = warp; j < n; j += 4) {
            const int64_t tok = k0 + t + j;
            float s = 0.f;
            for (int c = lane; c < kNope; c += 32)
                s += q[c] * widen2<BF16>(p.k[tok * p.k_token + h * p.k_head + c]).x;
            for (int c = lane; c < kRope; c += 32)
                s += q[kNope + c] * widen2<BF16>(p.k_pe[tok * p.k_pe_token + c]).x;
            for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
            if (lane == 0) score[j] = s;
        }
        __syncthreads();
        float top = m;
        for (int j = 0; j < n; ++j) top = fmaxf(top, score[j]);
        const float alpha = fast_exp2(m - top);
        m = top;
        l *= alpha;
        acc *= alpha;
        for (int j = 0; j < n; ++j) {
            const float w = fast_exp2(score[j] - m);
            l += w;
            acc += w * widen2<BF16>(p.v[(int64_t)(k0 + t + j) * p.v_token + h * p.v_head + threadIdx.x]).x;
        }
    }
    p.out[((int64_t)(q0 + i) * p.num_heads + h) * kValue + threadIdx.x] =
        (uint16_t)narrow2<BF16>(L > 0 ? acc / l : 0.f, 0.f);
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_prefill_latent(
    void *out, const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
    int64_t v_head_stride, const void *k_pe, int64_t k_pe_stride, const int32_t *q_starts,
    const int32_t *k_starts, int num_seqs, int total_q, int total_k, int max_q_len, int num_heads,
    float scale, int causal, pa_dtype dtype, void *stream) {
    if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_q_len < 0 || num_heads <= 0 ||
        num_heads > 1024 || num_seqs > 65535 || !std::isfinite(scale) ||
        (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID;
    const int64_t steps[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                             v_token_stride, v_head_stride, k_pe_stride};
    const int least[] = {kNope + kRope, kNope + kRope, kNope, kNope, kValue, kValue, kRope};
    for (int i = 0; i < 7; ++i)
        if (steps[i] < least[i] || steps[i] % 8 || steps[i] > (1ll << 38)) return PA_ERR_INVALID;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
    if (!out || !q || !q_starts || !k_starts || !aligned16(out) || !aligned16(q)) return PA_ERR_INVALID;
    if (total_k > 0 && (!k || !v || !k_pe)) return PA_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pe)) return PA_ERR_INVALID;
    PrefillLatentParams p = {};
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.out = static_cast<uint16_t *>(out);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.k_pe = static_cast<const uint16_t *>(k_pe);
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    p.k_pe_token = k_pe_stride;
    p.q_starts = q_starts;
    p.k_starts = k_starts;
    p.num_seqs = num_seqs;
    p.total_q = total_q;
    p.total_k = total_k;
    p.max_q = max_q_len;
    p.num_heads = num_heads;
    p.causal = causal != 0;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    auto kern = dtype == PA_BF16 ? prefill_latent_kernel<true> : prefill_latent_kernel<false>;
    if (launch_pdl(kern, dim3((unsigned)max_q_len, (unsigned)num_heads, (unsigned)num_seqs), dim3(128),
                   0, as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
