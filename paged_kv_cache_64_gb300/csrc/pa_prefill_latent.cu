// pa_prefill_latent: attention of ragged prompts in the expanded form of latent
// attention, on the 5th-generation tensor cores.
//
//   s = scale (q[0..128) . k + q[128..192) . k_pe);  out = softmax(s) v
//
// One CTA a (256 queries, head, sequence): two query tiles of 128 rows that take
// turns, so that one tile's softmax runs while the other's products do.  Per tile
// X and 128 keys:
//
//   S_X[128 rows x 128 keys] = Q_X . [K | K_pe]^T   (M=128, N=128, K=192)
//   O_X[128 rows x 128]     += P_X . V              (M=128, N=64 twice, K=128)
//
// K and the shared part meet only in shared memory: the concatenated keys are
// never formed.  TMEM: S_A, S_B, O_A, O_B of 128 columns each; P_X takes the place
// of S_X (two 16-bit weights a column) and is the A operand of P.V from there.
// Shared memory: Q (96 KiB) and a ring of eight 16 KiB slabs (128 keys x 64
// values) that K (three slabs a tile) and V (two) pass through in turn.
//
// Roles (10 warps): 0 producer (TMA); 1 issues every product (and owns TMEM);
// 2-5 softmax and epilogue of tile A, 6-9 of tile B: thread r of four warps owns
// row r (TMEM lane r), so maxima and sums need no exchange.  The products of a
// tile are issued in the order q.K(t), P.V(t), q.K(t + 1): S(t + 1) may take P(t)'s
// place, and once it is there, O is at rest for the lazy rescale.
#include <cmath>
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kPreRope = 64, kPreNope = 128, kPreValue = 128;
constexpr int kPreRows = 128;   // query rows of a tile
constexpr int kPreKeys = 128;   // keys of a tile
constexpr int kPreSlab = kPreKeys * 128;
constexpr int kPreSlots = 8;    // slabs of the ring
constexpr int kPreWarps = 10;
constexpr int kPreThreads = kPreWarps * 32;
constexpr int kPreOffRing = 2 * 3 * kPreSlab;
constexpr int kPreOffBar = kPreOffRing + kPreSlots * kPreSlab;
constexpr int kPreSmem = kPreOffBar + 512 + 1024;  // + slack to align the base to 1 KiB
constexpr int kPreColS = 0, kPreColO = 256;        // TMEM columns: S_A S_B O_A O_B
static_assert(kPreSmem <= 232448, "shared memory");

enum PreBar { kPreFull = 0, kPreEmpty = kPreSlots, kPreQFull = 2 * kPreSlots,
              kPreSFull = kPreQFull + 2, kPrePReady = kPreSFull + 2, kPreODone = kPrePReady + 2,
              kPreDrain = kPreODone + 2, kPreBars };

struct PrefillLatentParams {
    uint16_t *out;
    const int32_t *q_starts, *k_starts;
    int total_q, total_k, max_q, num_heads, causal;
    float scale_log2;
    int *err;
};

template <bool BF16>
__global__ void __launch_bounds__(kPreThreads, 1)
    prefill_latent_kernel(const __grid_constant__ PrefillLatentParams p,
                          const __grid_constant__ CUtensorMap map_q,
                          const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v,
                          const __grid_constant__ CUtensorMap map_pe) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kPreOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kPreOffBar + 384);
    int *flag = reinterpret_cast<int *>(smem + kPreOffBar + 392);
    volatile int *abort_flag = flag;
    static_assert(kPreBars * 8 <= 384, "barriers");

    // the longest tiles of a causal sequence first
    const int qt = gridDim.x - 1 - blockIdx.x, head = blockIdx.y, seq = blockIdx.z;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    pdl_wait();
    const int q0 = p.q_starts[seq], n_q = p.q_starts[seq + 1] - q0;
    const int k0 = p.k_starts[seq], n_k = p.k_starts[seq + 1] - k0;
    if (q0 < 0 || n_q < 0 || n_q > p.max_q || n_q > p.total_q - q0 || k0 < 0 || n_k < 0 ||
        n_k > p.total_k - k0) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            record_error(p.err, PA_ERR_BAD_INDEX);
        return;
    }
    const int first = qt * 2 * kPreRows;  // the CTA's first query in the sequence
    if (first >= n_q) return;
    // keys that a tile's rows meet: row i those below reach + i (causal) or n_k
    const int reach = p.causal ? n_k - n_q + 1 : n_k;
    auto tiles_of = [&](int x) -> int {
        const int a = first + x * kPreRows, b = min(a + kPreRows, n_q);
        if (a >= n_q) return 0;
        const int keys = p.causal ? min(reach + b - 1, n_k) : n_k;
        return keys > 0 ? (keys + kPreKeys - 1) / kPreKeys : 0;
    };
    const int tiles0 = tiles_of(0), tiles1 = tiles_of(1), most = max(tiles0, tiles1);

    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        prefetch_tensormap(&map_pe);
        for (int b = 0; b < kPreBars; ++b)
            mbar_init(&bar[b], b >= kPrePReady && b < kPreODone ? 4 : 1);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    bool ok = true;

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        if (lane == 0 && most > 0) {
            auto load_q = [&](int x) {
                mbar_arrive_expect_tx(&bar[kPreQFull + x], 3 * kPreSlab);
                for (int i = 0; i < 3; ++i)
                    tma_load_3d(smem + (3 * x + i) * kPreSlab, &map_q, 64 * i, q0 + first + x * kPreRows,
                                head, &bar[kPreQFull + x]);
            };
            // slab u: of tile u / 5 the keys' own values (two), the shared ones, V (two)
            auto load = [&](int u) -> bool {
                const int slot = u % kPreSlots, use = u / kPreSlots, t = u / 5, i = u % 5;
                if (use > 0 && !mbar_wait_or(&bar[kPreEmpty + slot], (use - 1) & 1, abort_flag))
                    return false;
                uint8_t *to = smem + kPreOffRing + slot * kPreSlab;
                uint64_t *full = &bar[kPreFull + slot];
                mbar_arrive_expect_tx(full, kPreSlab);
                const int key = k0 + t * kPreKeys;
                if (i == 2)
                    tma_load_2d(to, &map_pe, 0, key, full);
                else
                    tma_load_3d(to, i < 2 ? &map_k : &map_v, 64 * (i < 2 ? i : i - 3), key, head, full);
                return true;
            };
            int u = 0;
            if (tiles0 > 0) load_q(0);
            for (; u < 3; ++u) load(u);
            if (tiles1 > 0) load_q(1);
            for (; ok && u < 5 * most; u += ok) ok = load(u);
            // every copy has landed before shared memory goes (each slot's last use)
            for (int s = max(0, u - kPreSlots); s < u; ++s)
                (void)mbar_wait(&bar[kPreFull + s % kPreSlots], (s / kPreSlots) & 1);
            if (tiles0 > 0) (void)mbar_wait(&bar[kPreQFull], 0);
            if (tiles1 > 0) (void)mbar_wait(&bar[kPreQFull + 1], 0);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- products
        constexpr uint32_t idesc_qk = f16_idesc(BF16, false, false, kPreRows, kPreKeys);
        constexpr uint32_t idesc_pv = f16_idesc(BF16, false, true, kPreRows, 64);
        const uint32_t base = smem_addr(smem);
        const uint64_t q_desc = sw128_desc(base, 16, 1024);
        const uint64_t k_desc = sw128_desc(base + kPreOffRing, 16, 1024);
        const uint64_t v_desc = sw128_desc(base + kPreOffRing, kPreSlab, 1024);
        auto issue_qk = [&](int x, int t) {
            if (t == 0) mbar_wait_flow(&bar[kPreQFull + x], 0, flag);
            const bool last = x == 1 || t >= tiles1;  // tile B uses a slab last where it reaches it
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int u = 5 * t + i, slot = u % kPreSlots;
                mbar_wait_flow(&bar[kPreFull + slot], (u / kPreSlots) & 1, flag);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t q = q_desc + ((3 * x + i) * kPreSlab >> 4);
                    const uint64_t k = k_desc + slot * (kPreSlab >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma(tmem + kPreColS + 128 * x, q + ks * 2, k + ks * 2, idesc_qk, i > 0 || ks > 0);
                    if (last) tc_commit(&bar[kPreEmpty + slot]);
                    if (i == 2) tc_commit(&bar[kPreSFull + x]);
                }
                __syncwarp();
            }
        };
        auto issue_pv = [&](int x, int t) {
            mbar_wait_flow(&bar[kPrePReady + x], t & 1, flag);
            const bool last = x == 1 || t >= tiles1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int u = 5 * t + 3 + i, slot = u % kPreSlots;
                mbar_wait_flow(&bar[kPreFull + slot], (u / kPreSlots) & 1, flag);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t v = v_desc + slot * (kPreSlab >> 4);
#pragma unroll
                    for (int ks = 0; ks < kPreKeys / 16; ++ks)
                        tc_mma_ts(tmem + kPreColO + 128 * x + 64 * i, tmem + kPreColS + 128 * x + 8 * ks,
                                  v + ks * (2048 >> 4), idesc_pv, t > 0 || ks > 0);
                    if (last) tc_commit(&bar[kPreEmpty + slot]);
                    if (i == 1 && t + 1 == (x ? tiles1 : tiles0)) tc_commit(&bar[kPreODone + x]);
                }
                __syncwarp();
            }
        };
        if (tiles0 > 0) issue_qk(0, 0);
        if (tiles1 > 0) issue_qk(1, 0);
        for (int t = 0; t < most; ++t) {
            if (t < tiles0) issue_pv(0, t);
            if (t + 1 < tiles0) issue_qk(0, t + 1);
            if (t < tiles1) issue_pv(1, t);
            if (t + 1 < tiles1) issue_qk(1, t + 1);
        }
        if (elect_one()) tc_commit(&bar[kPreDrain]);
        (void)mbar_wait(&bar[kPreDrain], 0);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax / epilogue
        const int x = (warp - 2) >> 2, tiles = x ? tiles1 : tiles0;
        const int quad = warp & 3, r = quad * 32 + lane;  // TMEM lane = row of the tile
        const int row = first + x * kPreRows + r;         // query in the sequence
        const uint32_t s_at = tmem + ((uint32_t)(quad * 32) << 16) + kPreColS + 128 * x;
        const uint32_t o_at = tmem + ((uint32_t)(quad * 32) << 16) + kPreColO + 128 * x;
        const int limit = p.causal ? min(reach + row, n_k) : n_k;  // keys below it are met
        // up to here no row of the tile has a masked key
        const int clear = p.causal ? min(reach + first + x * kPreRows, n_k) : n_k;
        // f16 weights as 2^7 of themselves: at most 2^15 with the lag of the maximum, and
        // normal down to 2^-21 of the largest
        constexpr float kLift = BF16 ? 0.f : 7.f;
        float m_run = -INFINITY, l_run = 0.f;
        for (int t = 0; ok && t < tiles; ++t) {
            ok = __all_sync(kFullMask, mbar_wait_or(&bar[kPreSFull + x], t & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            float s[kPreKeys];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, s + 32 * c);
            const int here = t * kPreKeys;
            const float sc = p.scale_log2;
            float mx = -INFINITY;
            if (here + kPreKeys <= clear) {
#pragma unroll
                for (int j = 0; j < kPreKeys; ++j) {
                    s[j] *= sc;
                    mx = fmaxf(mx, s[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kPreKeys; ++j) {
                    s[j] = here + j < limit ? s[j] * sc : -INFINITY;  // NaN-safe select
                    mx = fmaxf(mx, s[j]);
                }
            }
            const bool need = mx > m_run + kLazyRescale;
            float alpha = 1.f;
            if (need) {
                alpha = fast_exp2(m_run - mx);  // 0 from an empty maximum
                m_run = mx;
                l_run *= alpha;
            }
            if (t > 0 && __any_sync(kFullMask, need)) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    float o[16];
                    tmem_load16(o_at + 16 * c, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= alpha;
                    tmem_store16(o_at + 16 * c, o);
                }
            }
            const float from = (m_run == -INFINITY ? 0.f : m_run) - kLift;
            float sum[4] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float a = fast_exp2(s[32 * c + 2 * j] - from);
                    const float b = fast_exp2(s[32 * c + 2 * j + 1] - from);
                    sum[j & 3] += a + b;
                    w[j] = __uint_as_float(narrow2<BF16>(a, b));
                }
                tmem_store16(s_at + 16 * c, w);
            }
            l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            if (here + kPreKeys > n_k && (x == 0 || t >= tiles0)) {
                // rows past the sequence's keys: P is 0 there, and V must be finite.  Tile B's
                // product follows A's, so the first tile to reach them clears them.
                for (int i = 0; i < 2; ++i) {
                    const int u = 5 * t + 3 + i;
                    ok = ok && mbar_wait_or(&bar[kPreFull + u % kPreSlots], (u / kPreSlots) & 1, abort_flag);
                    uint4 *z = reinterpret_cast<uint4 *>(smem + kPreOffRing + (u % kPreSlots) * kPreSlab);
                    for (int k = (n_k - here) * 8 + r; k < kPreKeys * 8; k += 128)
                        z[k] = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kPrePReady + x]);
        }
        if (tiles > 0 && ok)
            ok = __all_sync(kFullMask, mbar_wait_or(&bar[kPreODone + x], 0, abort_flag));
        if (ok) {
            tc_fence_after();
            const float inv = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : l_run;
            uint4 *to = reinterpret_cast<uint4 *>(
                p.out + ((int64_t)(q0 + row) * p.num_heads + head) * kPreValue);
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0.f;
                if (tiles > 0) tmem_load16(o_at + 16 * c, o);
                if (row < n_q) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = l_run == 0.f ? 0.f : o[i] * inv;
                    to[2 * c] = make_uint4(narrow2<BF16>(o[0], o[1]), narrow2<BF16>(o[2], o[3]),
                                           narrow2<BF16>(o[4], o[5]), narrow2<BF16>(o[6], o[7]));
                    to[2 * c + 1] = make_uint4(narrow2<BF16>(o[8], o[9]), narrow2<BF16>(o[10], o[11]),
                                               narrow2<BF16>(o[12], o[13]), narrow2<BF16>(o[14], o[15]));
                }
            }
        }
    }
    if (!ok) *abort_flag = 1;
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_error(p.err, PA_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
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
    const int least[] = {kPreNope + kPreRope, kPreNope + kPreRope, kPreNope, kPreNope, kPreValue,
                         kPreValue, kPreRope};
    for (int i = 0; i < 7; ++i)
        if (steps[i] < least[i] || steps[i] % 8 || steps[i] >= (1ll << 38)) return PA_ERR_INVALID;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
    if (!out || !q || !q_starts || !k_starts || !aligned16(out) || !aligned16(q)) return PA_ERR_INVALID;
    if (total_k > 0 && (!k || !v || !k_pe)) return PA_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pe)) return PA_ERR_INVALID;
    PrefillLatentParams p = {};
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.out = static_cast<uint16_t *>(out);
    p.q_starts = q_starts;
    p.k_starts = k_starts;
    p.total_q = total_q;
    p.total_k = total_k;
    p.max_q = max_q_len;
    p.num_heads = num_heads;
    p.causal = causal != 0;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const bool bf16 = dtype == PA_BF16;
    // without keys no map of theirs is used: q stands in
    const bool keys = total_k > 0;
    const int box[3] = {64, kPreKeys, 1};
    auto map3 = [&](CUtensorMap *map, const void *base, int width, int tokens, int64_t token, int64_t head) {
        const int64_t dims[3] = {width, tokens, num_heads}, step[2] = {token, head};
        return boxed_tensor_map(map, base, 3, dims, step, box, bf16);
    };
    CUtensorMap map_q, map_k, map_v, map_pe;
    const int64_t pe_dims[2] = {kPreRope, keys ? total_k : total_q}, pe_step[1] = {keys ? k_pe_stride : q_token_stride};
    if (!map3(&map_q, q, kPreNope + kPreRope, total_q, q_token_stride, q_head_stride) ||
        !(keys ? map3(&map_k, k, kPreNope, total_k, k_token_stride, k_head_stride) &&
                     map3(&map_v, v, kPreValue, total_k, v_token_stride, v_head_stride)
               : map3(&map_k, q, kPreNope, total_q, q_token_stride, q_head_stride) &&
                     map3(&map_v, q, kPreValue, total_q, q_token_stride, q_head_stride)) ||
        !boxed_tensor_map(&map_pe, keys ? k_pe : q, 2, pe_dims, pe_step, box, bf16))
        return PA_ERR_CUDA;
    auto kern = bf16 ? prefill_latent_kernel<true> : prefill_latent_kernel<false>;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(kern), kPreSmem)) return PA_ERR_CUDA;
    const dim3 grid((unsigned)(((int64_t)max_q_len + 2 * kPreRows - 1) / (2 * kPreRows)),
                    (unsigned)num_heads, (unsigned)num_seqs);
    if (launch_pdl(kern, grid, dim3(kPreThreads), kPreSmem, as_stream(stream), p, map_q, map_k, map_v,
                   map_pe) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
