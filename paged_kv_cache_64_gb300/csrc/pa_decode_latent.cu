// pa_decode_latent: decode attention, one query token a sequence, over a paged
// cache of latent rows (absorbed form).  The simplest form: one CTA a
// (sequence, head), 32 positions a step on CUDA cores.
#include <cmath>
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kRope = 64;

struct DecodeLatentParams {
    uint16_t *out;
    const uint16_t *q;
    const uint16_t *pool;
    const int32_t *tables;
    const int32_t *lens;
    int num_blocks, max_blocks, max_len, num_heads, log2_block;
    float scale_log2;
    int *err;
};

template <bool BF16, int RANK>
__global__ void __launch_bounds__(256) decode_latent_kernel(
    const __grid_constant__ DecodeLatentParams p) {
    constexpr int ROW = RANK + kRope, TILE = 32;
    __shared__ float q[ROW], score[TILE];
    __shared__ int64_t at[TILE];
    pdl_wait();
    const int h = blockIdx.x, seq = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)seq * p.num_heads + h;
    int L = p.lens[seq];
    const int64_t cover = (int64_t)p.max_blocks << p.log2_block;
    const int cap = (int)(cover < p.max_len ? cover : p.max_len);
    if (L < 0 || L > cap) {
        if (threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_INDEX);
        L = L < 0 ? 0 : cap;
    }
    for (int i = threadIdx.x; i < ROW; i += 256)
        q[i] = widen2<BF16>(p.q[row * ROW + i]).x * p.scale_log2;
    float m = -INFINITY, l = 0.f, acc[RANK / 256] = {};
    for (int t = 0; t < L; t += TILE) {
        const int n = min(TILE, L - t);
        __syncthreads();
        if (threadIdx.x < n) {
            const int pos = t + threadIdx.x;
            int blk = p.tables[(int64_t)seq * p.max_blocks + (pos >> p.log2_block)];
            if ((unsigned)blk >= (unsigned)p.num_blocks) {
                record_error(p.err, PA_ERR_BAD_INDEX);
                blk = 0;
            }
            at[threadIdx.x] = (((int64_t)blk << p.log2_block) + (pos & ((1 << p.log2_block) - 1))) * ROW;
        }
        __syncthreads();
        for (int i = warp; i < n; i += 8) {
            float s = 0.f;
            for (int c = lane; c < ROW; c += 32) s += q[c] * widen2<BF16>(p.pool[at[i] + c]).x;
            for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
            if (lane == 0) score[i] = s;
        }
        __syncthreads();
        float top = m;
        for (int i = 0; i < n; ++i) top = fmaxf(top, score[i]);
        const float alpha = fast_exp2(m - top);
        m = top;
        l *= alpha;
        for (int k = 0; k < RANK / 256; ++k) acc[k] *= alpha;
        for (int i = 0; i < n; ++i) {
            const float w = fast_exp2(score[i] - m);
            l += w;
            for (int k = 0; k < RANK / 256; ++k)
                acc[k] += w * widen2<BF16>(p.pool[at[i] + threadIdx.x + 256 * k]).x;
        }
    }
    for (int k = 0; k < RANK / 256; ++k)
        p.out[row * RANK + threadIdx.x + 256 * k] =
            (uint16_t)narrow2<BF16>(L > 0 ? acc[k] / l : 0.f, 0.f);
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_latent_workspace_size(int num_seqs, int num_heads, int rank,
                                                  int block_size, int max_seq_len, pa_dtype dtype) {
    (void)num_seqs, (void)num_heads, (void)rank, (void)block_size, (void)max_seq_len, (void)dtype;
    return 0;
}

extern "C" pa_status pa_decode_latent(void *out, const void *q, const void *pool, int num_blocks,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      const int32_t *seq_lens, int max_seq_len, int num_seqs,
                                      int num_heads, int rank, int block_size, float scale,
                                      void *workspace, size_t workspace_bytes, pa_dtype dtype,
                                      void *stream) {
    (void)workspace, (void)workspace_bytes;
    if (num_seqs < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_seq_len < 0 ||
        num_heads <= 0 || num_heads > 1024 || num_seqs > 65535 || !std::isfinite(scale) ||
        (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID;
    if ((rank != 256 && rank != 512) || (block_size != 16 && block_size != 32 && block_size != 64))
        return PA_ERR_UNSUPPORTED;
    if ((int64_t)num_blocks * block_size >= 1ll << 31 ||
        (int64_t)max_blocks_per_seq * block_size >= 1ll << 31)
        return PA_ERR_INVALID;
    if (num_seqs == 0) return PA_OK;
    const void *ptrs[] = {out, q, pool};
    for (const void *ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return PA_ERR_INVALID;
    if (!block_tables || !seq_lens) return PA_ERR_INVALID;
    DecodeLatentParams p = {};
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.out = static_cast<uint16_t *>(out);
    p.q = static_cast<const uint16_t *>(q);
    p.pool = static_cast<const uint16_t *>(pool);
    p.tables = block_tables;
    p.lens = seq_lens;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.max_len = max_seq_len;
    p.num_heads = num_heads;
    p.log2_block = block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const bool bf16 = dtype == PA_BF16;
    auto kern = rank == 512 ? (bf16 ? decode_latent_kernel<true, 512> : decode_latent_kernel<false, 512>)
                            : (bf16 ? decode_latent_kernel<true, 256> : decode_latent_kernel<false, 256>);
    if (launch_pdl(kern, dim3((unsigned)num_heads, (unsigned)num_seqs), dim3(256), 0,
                   as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
