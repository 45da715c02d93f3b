// pa_decode_latent: decode attention, one query token a sequence, over a paged
// cache of latent rows (absorbed form), on the 5th-generation tensor cores.
//
//   s_p = scale q . row_p over RANK + 64 values;  out = softmax(s) . row[0 .. RANK)
//
// A row is key and value at once, so a tile of 64 rows is staged once for both
// products.  Per tile and group of up to NH heads (one CTA):
//
//   S[heads x 64 pos]    = Q[heads x (RANK + 64)] . K_tile^T        (M=64, N=64)
//   O^T[128 dims x heads] += V_tile^T[128 x 64 pos] . P^T, RANK/128 times (N=NH)
//
// S with the heads on the lanes: a thread owns a head's row, so maxima and sums
// need no exchange.  O transposed: 128 dims fill the lanes whatever the number of
// heads, RANK/128 * NH columns hold it, and the staged rows are its A operand as
// they lie (MN-major).  Two S buffers and O are in TMEM; Q stays in shared memory,
// the rows pass through rings of 64-column slabs (16 KiB pairs of the latent part,
// freed after P.V; 8 KiB of the rotary part, freed after q.K).
//
// Roles (8 warps): 0 producer of rows (TMA boxes of 16 rows through the block
// table); 1 issues q.K^T (and owns TMEM); 2-5 softmax and epilogue; 6 issues P.V;
// 7 loads Q.  The running maximum moves only when a tile exceeds it by more than
// kLazyRescale; then O's columns are rescaled in TMEM.
//
// The batch's tiles are shared out evenly: range b of the launch is tiles
// [b per, (b + 1) per) of all sequences' tiles in a row, found from the lengths on
// the device.  A CTA goes through its range's pieces of sequences; Q and the rows
// of the next piece are on their way while one ends.  A piece that is a whole
// sequence is written out; the others leave (m, l, O) and a second launch joins
// them.
#include <cmath>
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kLatRope = 64;      // shared key values of a row
constexpr int kLatTile = 64;      // positions of a tile
constexpr int kLatWarps = 8;
constexpr int kLatThreads = kLatWarps * 32;
constexpr int kLatSmem = 232448;  // what a CTA may have
constexpr int kLatMisc = 2048;    // barriers and exchange
constexpr int kLatMinTiles = 4;   // tiles of a range, at least
constexpr int kLatWhole = 8;      // up to so many tiles a sequence is never cut

struct DecodeLatentParams {
    uint16_t *out;
    const int32_t *tables;
    const int32_t *lens;
    float *part_o;   // [ranges][groups][2][NH][RANK]
    float *part_ml;  // [ranges][groups][2][NH][2]: maximum (base 2), sum
    int4 *plan;      // [ranges]: sequence whose pieces begin in the range and go on, or -1
    int num_blocks, max_blocks, max_len, num_seqs, num_heads, log2_block;
    int ranges, groups;
    int whole;       // range b is sequence b
    float scale_log2;
    int *err;
};

template <int RANK, int NH>
struct LatShape {
    static constexpr int SLABS = RANK / 64 + 1;    // the last one rotary
    static constexpr int PAIRS = RANK / 128;
    static constexpr int Q_SLAB = NH * 128;
    static constexpr int SLAB = kLatTile * 128;
    static constexpr int P_BYTES = NH * 128;
    static constexpr int P_BUFS = RANK == 512 && NH == 64 ? 1 : 2;
    static constexpr int ROPE_SLOTS = RANK == 256 ? (NH == 64 ? 4 : 5) : (NH == 64 ? 2 : 3);
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + SLABS * Q_SLAB;
    static constexpr int OFF_ROPE = OFF_P + P_BUFS * P_BYTES;
    static constexpr int OFF_PAIR = OFF_ROPE + ROPE_SLOTS * SLAB;
    static constexpr int PAIR_SLOTS = (kLatSmem - 1024 - kLatMisc - OFF_PAIR) / (2 * SLAB);
    static constexpr int OFF_MISC = OFF_PAIR + PAIR_SLOTS * 2 * SLAB;
    static constexpr int SMEM_BYTES = OFF_MISC + kLatMisc + 1024;  // + slack to align the base
    static constexpr int S_COL = PAIRS * NH;       // TMEM: O first, then two S buffers
    // barriers
    static constexpr int PAIR_FULL = 0, PAIR_EMPTY = PAIR_SLOTS, ROPE_FULL = 2 * PAIR_SLOTS,
                         ROPE_EMPTY = ROPE_FULL + ROPE_SLOTS, Q_FULL = ROPE_EMPTY + ROPE_SLOTS,
                         Q_FREE = Q_FULL + 1, S_FULL = Q_FREE + 1, S_FREE = S_FULL + 2,
                         P_FULL = S_FREE + 2, PV_DONE = P_FULL + 2, O_FREE = PV_DONE + 2,
                         DRAIN = O_FREE + 1, BARS = DRAIN + 2;
    // behind the barriers: TMEM address, abort flag, scan scratch, then alphas / sums
    static constexpr int OFF_WORDS = OFF_MISC + 512, OFF_ALPHA = OFF_MISC + 1024;
    static_assert(BARS * 8 <= 512 && NH * 4 <= 1024, "misc");
    static_assert(PAIR_SLOTS >= 2 * PAIRS && S_COL + 2 * kLatTile <= 512, "rings, TMEM");
    static_assert(OFF_P % 1024 == 0 && OFF_PAIR % 1024 == 0 && SMEM_BYTES <= kLatSmem, "layout");
    // q.K reads 64 rows of A whatever NH: past a slab's own rows it meets other
    // operands, whose products end in lanes that nothing reads
    static_assert(OFF_P - Q_SLAB + 64 * 128 <= OFF_MISC, "A rows in shared memory");
};

// Length of a sequence, clamped to what the launch and the table cover.
__device__ __forceinline__ int latent_len(const DecodeLatentParams &p, int seq, bool report) {
    int L = p.lens[seq];
    const int cover = p.max_blocks << p.log2_block;
    const int cap = cover < p.max_len ? cover : p.max_len;
    if (L < 0 || L > cap) {
        if (report) record_error(p.err, PA_ERR_BAD_INDEX);
        L = L < 0 ? 0 : cap;
    }
    return L;
}
// Tiles of a sequence; an empty one counts as one, in which its zeros are written.
__device__ __forceinline__ int latent_tiles(int len) {
    return len > 0 ? (len + kLatTile - 1) / kLatTile : 1;
}

// The pieces of a range, in order: every role walks them by itself.
struct LatWalk {
    const DecodeLatentParams &p;
    int seq, tile, left;
    int len, n;    // of the current piece: the sequence's length, tiles
    bool more;     // the sequence goes on behind the range
    __device__ __forceinline__ LatWalk(const DecodeLatentParams &prm, int s, int t, int l)
        : p(prm), seq(s), tile(t), left(l) {}
    __device__ __forceinline__ bool next() {  // the current piece's data, false at the end
        if (left <= 0 || seq >= p.num_seqs) return false;
        len = latent_len(p, seq, false);
        n = latent_tiles(len) - tile;
        more = n > left;
        if (more) n = left;
        return true;
    }
    __device__ __forceinline__ void advance() {
        left -= n;
        tile = 0;
        ++seq;
    }
};

// Named barrier 1 over the 128 softmax threads, true on all if any passed true.
__device__ __forceinline__ bool softmax_bar128_or(bool v) {
    int any;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.s32 pi, %1, 0;\n\t"
        "bar.red.or.pred po, 1, 128, pi;\n\t"
        "selp.s32 %0, 1, 0, po;\n\t}"
        : "=r"(any)
        : "r"((int)v)
        : "memory");
    return any != 0;
}

template <bool BF16, int RANK, int NH>
__global__ void __launch_bounds__(kLatThreads, 1)
    decode_latent_kernel(const __grid_constant__ DecodeLatentParams p,
                         const __grid_constant__ CUtensorMap map_rows,
                         const __grid_constant__ CUtensorMap map_q) {
    using S = LatShape<RANK, NH>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + S::OFF_MISC);
    int *words = reinterpret_cast<int *>(smem + S::OFF_WORDS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(words);
    int *flag = words + 1;
    volatile int *abort_flag = flag;
    int *scan = words + 8;  // [8] warp sums, then start sequence and tile
    float *alphas = reinterpret_cast<float *>(smem + S::OFF_ALPHA);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int group = blockIdx.x % p.groups, range = blockIdx.x / p.groups;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_rows);
        prefetch_tensormap(&map_q);
        for (int b = 0; b < S::BARS; ++b)
            mbar_init(&bar[b], (b >= S::S_FREE && b < S::PV_DONE) || b == S::O_FREE ? 4 : 1);
        *abort_flag = 0;
        scan[8] = p.num_seqs;
        scan[9] = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();

    // ---------------------------------------------------------- this CTA's range
    int seq0 = range, tile0 = 0, left;
    if (p.whole) {
        left = latent_tiles(latent_len(p, range, group == 0));
        tc_fence_before();
        __syncthreads();
    } else {
        int sum = 0;
        for (int i = threadIdx.x; i < p.num_seqs; i += kLatThreads)
            sum += latent_tiles(latent_len(p, i, blockIdx.x == 0));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        if (lane == 0) scan[warp] = sum;
        tc_fence_before();
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < kLatWarps; ++w) total += scan[w];
        int per = (total + p.ranges - 1) / p.ranges;
        if (per < kLatMinTiles) per = kLatMinTiles;
        const int start = (int)min((int64_t)range * per, (int64_t)total);
        left = min(per, total - start);
        // the sequence and tile that the range begins with
        int before = 0;
        for (int base = 0; base < p.num_seqs && left > 0; base += kLatThreads) {
            const int i = base + (int)threadIdx.x;
            const int mine = i < p.num_seqs ? latent_tiles(latent_len(p, i, false)) : 0;
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFullMask, incl, o);
                if (lane >= o) incl += v;
            }
            __syncthreads();
            if (lane == 31) scan[warp] = incl;
            __syncthreads();
            int all = 0;
#pragma unroll
            for (int w = 0; w < kLatWarps; ++w) {
                if (w == warp) incl += all;
                all += scan[w];
            }
            const int first = before + incl - mine;
            if (start >= first && start < first + mine) {
                scan[8] = i;
                scan[9] = start - first;
            }
            before += all;
            if (before > start) break;  // the same for all threads
        }
        __syncthreads();
        seq0 = scan[8];
        tile0 = scan[9];
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();  // the joining launch waits for this one's end by itself

    LatWalk walk(p, seq0, tile0, left);
    bool ok = true;

    if (warp == 0) {
        // ---------------------------------------------------------- producer of rows
        int pair = 0, pair_use = 0, rope = 0, rope_use = 0;
        for (; ok && walk.next(); walk.advance()) {
            if (walk.len == 0) continue;
            const int first = walk.tile * kLatTile;
            const int units = (min(walk.len - first, walk.n * kLatTile) + kUnit - 1) / kUnit;
            const int32_t *table = p.tables + (int64_t)walk.seq * p.max_blocks;
            auto unit_row = [&](int u) -> int {  // first row of a unit in the pool
                if (u >= units) return 0;
                const int pos = first + u * kUnit;
                int phys = table[pos >> p.log2_block];
                if ((unsigned)phys >= (unsigned)p.num_blocks) {
                    record_error(p.err, PA_ERR_BAD_INDEX);
                    phys = 0;
                }
                return (phys << p.log2_block) + (pos & ((1 << p.log2_block) - 1));
            };
            int rows_cur = unit_row(lane), rows_next = unit_row(32 + lane);
            for (int t = 0; ok && t < walk.n; ++t) {
                if (t > 0 && (t & 7) == 0) {
                    rows_cur = rows_next;
                    rows_next = unit_row(32 * ((t >> 3) + 1) + lane);
                }
                const int nu = min(units - 4 * t, 4);
                const int row = __shfl_sync(kFullMask, rows_cur, ((t & 7) * 4 + (lane & 3)) & 31);
                if (rope_use > 0)
                    ok = mbar_wait_or(&bar[S::ROPE_EMPTY + rope], (rope_use - 1) & 1, abort_flag);
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&bar[S::ROPE_FULL + rope], nu * 2048);
                __syncwarp();
                if (lane < nu)
                    tma_load_2d(smem + S::OFF_ROPE + rope * S::SLAB + lane * 2048, &map_rows, RANK, row,
                                &bar[S::ROPE_FULL + rope]);
                if (++rope == S::ROPE_SLOTS) rope = 0, ++rope_use;
#pragma unroll
                for (int j = 0; j < S::PAIRS; ++j) {
                    if (ok && pair_use > 0)
                        ok = mbar_wait_or(&bar[S::PAIR_EMPTY + pair], (pair_use - 1) & 1, abort_flag);
                    ok = __all_sync(kFullMask, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bar[S::PAIR_FULL + pair], nu * 4096);
                    __syncwarp();
                    if (lane < 8 && (lane & 3) < nu)
                        tma_load_2d(smem + S::OFF_PAIR + pair * 2 * S::SLAB + (lane >> 2) * S::SLAB +
                                        (lane & 3) * 2048,
                                    &map_rows, 128 * j + 64 * (lane >> 2), row, &bar[S::PAIR_FULL + pair]);
                    if (++pair == S::PAIR_SLOTS) pair = 0, ++pair_use;
                }
            }
        }
        // every copy has landed before shared memory goes (a slot's last use)
        for (int i = 0; i < S::PAIR_SLOTS; ++i) {
            const int uses = pair_use + (i < pair);
            if (uses > 0) (void)mbar_wait(&bar[S::PAIR_FULL + i], (uses - 1) & 1);
        }
        for (int i = 0; i < S::ROPE_SLOTS; ++i) {
            const int uses = rope_use + (i < rope);
            if (uses > 0) (void)mbar_wait(&bar[S::ROPE_FULL + i], (uses - 1) & 1);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- q.K^T
        constexpr uint32_t idesc = f16_idesc(BF16, false, false, 64, kLatTile);
        const uint32_t base = smem_addr(smem);
        const uint64_t q_desc = sw128_desc(base + S::OFF_Q, 16, 1024);
        const uint64_t pair_desc = sw128_desc(base + S::OFF_PAIR, 16, 1024);
        const uint64_t rope_desc = sw128_desc(base + S::OFF_ROPE, 16, 1024);
        int pair = 0, pair_use = 0, rope = 0, rope_use = 0, g = 0, piece = 0;
        for (; walk.next(); walk.advance()) {
            if (walk.len == 0) continue;
            mbar_wait_flow(&bar[S::Q_FULL], piece & 1, flag);
            for (int t = 0; t < walk.n; ++t, ++g) {
                const int b = g & 1;
                if (g >= 2) mbar_wait_flow(&bar[S::S_FREE + b], ((g >> 1) - 1) & 1, flag);
                mbar_wait_flow(&bar[S::ROPE_FULL + rope], rope_use & 1, flag);
                tc_fence_after();
                const uint32_t d = tmem + S::S_COL + kLatTile * b;
                if (elect_one()) {
                    const uint64_t k = rope_desc + rope * (S::SLAB >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma(d, q_desc + (((S::SLABS - 1) * S::Q_SLAB + ks * 32) >> 4), k + ks * 2,
                               idesc, ks > 0);
                    tc_commit(&bar[S::ROPE_EMPTY + rope]);
                }
                __syncwarp();
                if (++rope == S::ROPE_SLOTS) rope = 0, ++rope_use;
#pragma unroll
                for (int j = 0; j < S::PAIRS; ++j) {
                    mbar_wait_flow(&bar[S::PAIR_FULL + pair], pair_use & 1, flag);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t k = pair_desc + pair * (2 * S::SLAB >> 4);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            tc_mma(d,
                                   q_desc + (((2 * j + (ks >> 2)) * S::Q_SLAB + (ks & 3) * 32) >> 4),
                                   k + (((ks >> 2) * S::SLAB + (ks & 3) * 32) >> 4), idesc, 1);
                        if (j + 1 == S::PAIRS) {
                            if (t + 1 == walk.n) tc_commit(&bar[S::Q_FREE]);
                            tc_commit(&bar[S::S_FULL + b]);
                        }
                    }
                    __syncwarp();
                    if (++pair == S::PAIR_SLOTS) pair = 0, ++pair_use;
                }
            }
            ++piece;
        }
        if (elect_one()) tc_commit(&bar[S::DRAIN]);
        (void)mbar_wait(&bar[S::DRAIN], 0);
        __syncwarp();
    } else if (warp == 6) {
        // ---------------------------------------------------------- P.V
        constexpr uint32_t idesc = f16_idesc(BF16, true, false, 128, NH);
        const uint32_t base = smem_addr(smem);
        const uint64_t p_desc = sw128_desc(base + S::OFF_P, 16, 1024);
        const uint64_t pair_desc = sw128_desc(base + S::OFF_PAIR, S::SLAB, 1024);
        int pair = 0, pair_use = 0, g = 0, piece = 0;
        for (; walk.next(); walk.advance()) {
            if (walk.len == 0) continue;
            if (piece > 0) mbar_wait_flow(&bar[S::O_FREE], (piece - 1) & 1, flag);
            for (int t = 0; t < walk.n; ++t, ++g) {
                const int pb = g % S::P_BUFS;
                mbar_wait_flow(&bar[S::P_FULL + pb], (g / S::P_BUFS) & 1, flag);
                const uint64_t w = p_desc + pb * (S::P_BYTES >> 4);
#pragma unroll
                for (int j = 0; j < S::PAIRS; ++j) {
                    mbar_wait_flow(&bar[S::PAIR_FULL + pair], pair_use & 1, flag);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t v = pair_desc + pair * (2 * S::SLAB >> 4);
#pragma unroll
                        for (int ks = 0; ks < kLatTile / 16; ++ks)
                            tc_mma(tmem + j * NH, v + ks * (2048 >> 4), w + ks * 2, idesc, t > 0 || ks > 0);
                        tc_commit(&bar[S::PAIR_EMPTY + pair]);
                        if (j + 1 == S::PAIRS) tc_commit(&bar[S::PV_DONE + pb]);
                    }
                    __syncwarp();
                    if (++pair == S::PAIR_SLOTS) pair = 0, ++pair_use;
                }
            }
            ++piece;
        }
        if (elect_one()) tc_commit(&bar[S::DRAIN + 1]);
        (void)mbar_wait(&bar[S::DRAIN + 1], 0);
        __syncwarp();
    } else if (warp == 7) {
        // ---------------------------------------------------------- Q
        if (lane == 0) {
            int piece = 0;
            for (; ok && walk.next(); walk.advance()) {
                if (walk.len == 0) continue;
                if (piece > 0) ok = mbar_wait_or(&bar[S::Q_FREE], (piece - 1) & 1, abort_flag);
                if (!ok) break;
                mbar_arrive_expect_tx(&bar[S::Q_FULL], S::SLABS * S::Q_SLAB);
                // rows past the last sequence read as zero, other heads' rows as they are
                for (int i = 0; i < S::SLABS; ++i)
                    tma_load_2d(smem + S::OFF_Q + i * S::Q_SLAB, &map_q, 64 * i,
                                walk.seq * p.num_heads + group * NH, &bar[S::Q_FULL]);
                ++piece;
            }
            if (piece > 0) (void)mbar_wait(&bar[S::Q_FULL], (piece - 1) & 1);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax / epilogue
        const int quad = warp & 3;                 // TMEM lanes this warp may access
        const int row = quad * 16 + lane;          // head of lanes 0-15 (M = 64: 16 lanes a quadrant)
        const int heads = min(NH, p.num_heads - group * NH);
        const bool mine = lane < 16 && row < heads;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        // f16 weights as 2^7 of themselves: at most 2^15 with the lag of the maximum, and
        // normal down to 2^-21 of the largest
        constexpr float kLift = BF16 ? 0.f : 7.f;
        int g = 0, pair0 = 0;
        int4 plan = make_int4(-1, 0, 0, 0);
        // P.V of tile k (counted over all pieces) is done.  One barrier a P buffer, whose
        // phases are waited for in turn: a tile's is, at the latest, before P goes into
        // its buffer again.
        auto pv_done = [&](int k) -> bool {
            return mbar_wait_or(&bar[S::PV_DONE + k % S::P_BUFS], (k / S::P_BUFS) & 1, abort_flag);
        };
        for (; ok && walk.next(); walk.advance()) {
            const int64_t out_row = (int64_t)walk.seq * p.num_heads + group * NH;
            const int dim = quad * 32 + lane;
            if (walk.len == 0) {
                for (int h = 0; h < heads; ++h)
#pragma unroll
                    for (int j = 0; j < S::PAIRS; ++j) p.out[(out_row + h) * RANK + 128 * j + dim] = 0;
                continue;
            }
            float m_run = -INFINITY, l_run = 0.f;
            for (int t = 0; t < walk.n; ++t, ++g) {
                const int b = g & 1;
                bool fine = mbar_wait_or(&bar[S::S_FULL + b], (g >> 1) & 1, abort_flag);
                fine = __all_sync(kFullMask, fine);
                float s[kLatTile];
                if (fine) {
                    tc_fence_after();
                    tmem_ld32(tmem + lanes + S::S_COL + kLatTile * b, s);
                    tmem_ld32(tmem + lanes + S::S_COL + kLatTile * b + 32, s + 32);
                    tc_fence_before();
                } else {
#pragma unroll
                    for (int j = 0; j < kLatTile; ++j) s[j] = 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[S::S_FREE + b]);
                const int valid = min(walk.len - (walk.tile + t) * kLatTile, kLatTile);
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < kLatTile; ++j) {
                    s[j] = j < valid ? s[j] * p.scale_log2 : -INFINITY;  // NaN-safe select
                    mx = fmaxf(mx, s[j]);
                }
                float alpha = 1.f;
                bool need = mx > m_run + kLazyRescale;
                if (need) {
                    alpha = fast_exp2(m_run - mx);  // 0 from an empty maximum
                    m_run = mx;
                    l_run *= alpha;
                }
                need = need && mine && t > 0;
                if (mine) alphas[row] = alpha;
                const float from = (m_run == -INFINITY ? 0.f : m_run) - kLift;
                uint32_t w[kLatTile / 2];
#pragma unroll
                for (int j = 0; j < kLatTile / 2; ++j) {
                    const float a = fast_exp2(s[2 * j] - from), c = fast_exp2(s[2 * j + 1] - from);
                    l_run += a + c;
                    w[j] = narrow2<BF16>(a, c);
                }
                const bool any = softmax_bar128_or(need || !fine);
                // P's buffer is free, and O at rest where it is rescaled
                if (g >= S::P_BUFS) fine = fine && pv_done(g - S::P_BUFS);
                if (any && g > 0) fine = fine && pv_done(g - 1);
                if (valid < kLatTile) {
                    // rows past the length: P is 0 there, and V must be finite
                    int pair = pair0;
                    for (int j = 0; j < S::PAIRS; ++j) {
                        fine = fine && mbar_wait_or(&bar[S::PAIR_FULL + pair],
                                                ((g * S::PAIRS + j) / S::PAIR_SLOTS) & 1, abort_flag);
                        uint8_t *slab = smem + S::OFF_PAIR + pair * 2 * S::SLAB;
                        for (int i = valid * 8 + quad * 32 + lane; i < kLatTile * 8; i += 128) {
                            reinterpret_cast<uint4 *>(slab)[i] = make_uint4(0, 0, 0, 0);
                            reinterpret_cast<uint4 *>(slab + S::SLAB)[i] = make_uint4(0, 0, 0, 0);
                        }
                        if (++pair == S::PAIR_SLOTS) pair = 0;
                    }
                }
                fine = __all_sync(kFullMask, fine);
                if (any) {
                    // rescale O, or end together
                    if (softmax_bar128_or(!fine)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < S::PAIRS * NH; c += 16) {
                        float o[16];
                        tmem_load16(tmem + lanes + c, o);
                        const float4 *a = reinterpret_cast<const float4 *>(alphas + c % NH);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 f = a[i];
                            o[4 * i] *= f.x, o[4 * i + 1] *= f.y, o[4 * i + 2] *= f.z, o[4 * i + 3] *= f.w;
                        }
                        tmem_store16(tmem + lanes + c, o);
                    }
                    tmem_wait_st();
                    softmax_bar128_or(false);  // the alphas are free again
                } else if (!fine) {
                    *abort_flag = 1;
                }
                if (mine) {
                    uint8_t *to = smem + S::OFF_P + (g % S::P_BUFS) * S::P_BYTES + (row >> 3) * 1024 +
                                  (row & 7) * 128;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4 *>(to + ((j ^ (row & 7)) << 4)) =
                            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[S::P_FULL + g % S::P_BUFS]);
                pair0 = (pair0 + S::PAIRS) % S::PAIR_SLOTS;
            }
            if (!ok) break;
            const bool fine = pv_done(g - 1);
            if (softmax_bar128_or(!fine)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool whole = walk.tile == 0 && !walk.more;
            if (whole) {
                if (mine) alphas[row] = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : l_run;
                softmax_bar128_or(false);
#pragma unroll 1
                for (int c = 0; c < S::PAIRS * NH; c += 16) {
                    float o[16];
                    tmem_load16(tmem + lanes + c, o);
                    const int h0 = c % NH, j = c / NH;
                    uint16_t *to = p.out + (out_row + h0) * RANK + 128 * j + dim;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (h0 + i < heads) to[i * RANK] = narrow1<BF16>(o[i] * alphas[h0 + i]);
                }
            } else {
                const int cut = walk.seq == seq0 && walk.tile == tile0 ? 0 : 1;
                const int64_t slot = ((int64_t)range * p.groups + group) * 2 + cut;
                if (walk.more && walk.tile == 0) {
                    const int rest = latent_tiles(walk.len) - walk.n;
                    plan = make_int4(walk.seq, cut, rest, 0);
                }
                if (mine) {
                    p.part_ml[(slot * NH + row) * 2] = m_run;
                    p.part_ml[(slot * NH + row) * 2 + 1] = l_run;
                }
                float *part = p.part_o + slot * NH * RANK + dim;
#pragma unroll 1
                for (int c = 0; c < S::PAIRS * NH; c += 16) {
                    float o[16];
                    tmem_load16(tmem + lanes + c, o);
                    const int h0 = c % NH, j = c / NH;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (h0 + i < heads) part[(h0 + i) * RANK + 128 * j] = o[i];
                }
            }
            tc_fence_before();
            softmax_bar128_or(false);  // O and the alphas have been read
            if (lane == 0) mbar_arrive(&bar[S::O_FREE]);
        }
        if (!p.whole && group == 0 && threadIdx.x == 64) {
            // the ranges that the rest of the sequence lies in (all but the last full)
            const int per = left;  // a range that a sequence goes on behind is full
            if (plan.x >= 0) plan.z = (plan.z + per - 1) / per;
            p.plan[range] = ok ? plan : make_int4(-1, 0, 0, 0);
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

// Joins the pieces of the sequences that ranges cut: block (range, head) the
// sequence that begins in the range and goes on.
//   M = max m_i;  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i
constexpr int kLatJoinThreads = 512;

template <bool BF16, int RANK, int NH>
__global__ void __launch_bounds__(kLatJoinThreads) latent_join_kernel(
    const __grid_constant__ DecodeLatentParams p) {
    constexpr int D4 = RANK / 4, PARTS = kLatJoinThreads / D4;
    __shared__ float weight[1024];
    __shared__ float4 sums[PARTS][D4];
    pdl_wait();
    const int range = blockIdx.x, h = blockIdx.y, group = h / NH, row = h % NH;
    const int4 plan = p.plan[range];
    if (plan.x < 0) return;
    const int n = plan.z + 1;
    auto slot_of = [&](int i) -> int64_t {
        return ((int64_t)(range + i) * p.groups + group) * 2 + (i == 0 ? plan.y : 0);
    };
    if (threadIdx.x < 32) {
        float M = -INFINITY;
        for (int i = threadIdx.x; i < n; i += 32)
            M = fmaxf(M, p.part_ml[(slot_of(i) * NH + row) * 2]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
        float total = 0.f;
        for (int i = threadIdx.x; i < n; i += 32) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + (slot_of(i) * NH + row) * 2);
            const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
            weight[i] = w;
            total += w * ml.y;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
        const float inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
        for (int i = threadIdx.x; i < n; i += 32) weight[i] *= inv;
    }
    __syncthreads();
    const int d = threadIdx.x % D4, part = threadIdx.x / D4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = part; i < n; i += PARTS) {
        const float4 v = reinterpret_cast<const float4 *>(p.part_o + (slot_of(i) * NH + row) * RANK)[d];
        const float w = weight[i];
        acc.x += w * v.x, acc.y += w * v.y, acc.z += w * v.z, acc.w += w * v.w;
    }
    sums[part][d] = acc;
    __syncthreads();
    if (part == 0) {
#pragma unroll
        for (int k = 1; k < PARTS; ++k) {
            const float4 v = sums[k][d];
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        reinterpret_cast<uint2 *>(p.out + ((int64_t)plan.x * p.num_heads + h) * RANK)[d] =
            make_uint2(narrow2<BF16>(acc.x, acc.y), narrow2<BF16>(acc.z, acc.w));
    }
}

// ------------------------------------------------------------------ host side
struct LatentLaunch {
    int nh, groups, ranges, whole;
    size_t o_bytes, ml_bytes, plan_bytes;
    size_t bytes() const { return whole ? 0 : o_bytes + ml_bytes + plan_bytes; }
};

static LatentLaunch latent_launch(int num_seqs, int num_heads, int rank, int max_seq_len, int sms) {
    LatentLaunch c = {};
    c.nh = num_heads <= 16 ? 16 : num_heads <= 32 ? 32 : 64;
    c.groups = (num_heads + c.nh - 1) / c.nh;
    c.ranges = sms / c.groups > 0 ? sms / c.groups : 1;
    const int tiles = (max_seq_len + kLatTile - 1) / kLatTile;
    c.whole = num_seqs <= c.ranges && tiles <= kLatWhole;
    if (c.whole) c.ranges = num_seqs;
    const size_t pieces = (size_t)c.ranges * c.groups * 2 * c.nh;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    c.o_bytes = up(pieces * rank * 4);
    c.ml_bytes = up(pieces * 8);
    c.plan_bytes = up((size_t)c.ranges * 16);
    return c;
}

struct LatentKernels {
    void (*decode)(const DecodeLatentParams, const CUtensorMap, const CUtensorMap);
    void (*join)(const DecodeLatentParams);
    int smem;
};

template <bool BF16, int RANK>
static LatentKernels latent_kernels(int nh) {
    if (nh == 16)
        return {decode_latent_kernel<BF16, RANK, 16>, latent_join_kernel<BF16, RANK, 16>,
                LatShape<RANK, 16>::SMEM_BYTES};
    if (nh == 32)
        return {decode_latent_kernel<BF16, RANK, 32>, latent_join_kernel<BF16, RANK, 32>,
                LatShape<RANK, 32>::SMEM_BYTES};
    return {decode_latent_kernel<BF16, RANK, 64>, latent_join_kernel<BF16, RANK, 64>,
            LatShape<RANK, 64>::SMEM_BYTES};
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_latent_workspace_size(int num_seqs, int num_heads, int rank,
                                                  int block_size, int max_seq_len, pa_dtype dtype) {
    (void)block_size, (void)dtype;
    if (num_seqs <= 0 || num_heads <= 0 || num_heads > 1024 || max_seq_len < 0 ||
        (rank != 256 && rank != 512))
        return 0;
    return latent_launch(num_seqs, num_heads, rank, max_seq_len, sm_count()).bytes();
}

extern "C" pa_status pa_decode_latent(void *out, const void *q, const void *pool, int num_blocks,
                                      const int32_t *block_tables, int max_blocks_per_seq,
                                      const int32_t *seq_lens, int max_seq_len, int num_seqs,
                                      int num_heads, int rank, int block_size, float scale,
                                      void *workspace, size_t workspace_bytes, pa_dtype dtype,
                                      void *stream) {
    if (num_seqs < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_seq_len < 0 ||
        num_heads <= 0 || num_heads > 1024 || num_seqs > 65535 || !std::isfinite(scale) ||
        (dtype != PA_F16 && dtype != PA_BF16))
        return PA_ERR_INVALID;
    if ((rank != 256 && rank != 512) || (block_size != 16 && block_size != 32 && block_size != 64))
        return PA_ERR_UNSUPPORTED;
    if ((int64_t)num_blocks * block_size >= 1ll << 31 ||
        (int64_t)max_blocks_per_seq * block_size >= 1ll << 31 ||
        ((int64_t)max_seq_len / kLatTile + 1) * num_seqs >= 1ll << 31)
        return PA_ERR_INVALID;
    if (num_seqs == 0) return PA_OK;
    const void *ptrs[] = {out, q, pool};
    for (const void *ptr : ptrs)
        if (!ptr || !aligned16(ptr)) return PA_ERR_INVALID;
    if (!block_tables || !seq_lens) return PA_ERR_INVALID;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const LatentLaunch c = latent_launch(num_seqs, num_heads, rank, max_seq_len, sms);
    if (c.bytes() > 0 && (!workspace || workspace_bytes < c.bytes() ||
                          (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return PA_ERR_INVALID;
    DecodeLatentParams p = {};
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.out = static_cast<uint16_t *>(out);
    p.tables = block_tables;
    p.lens = seq_lens;
    if (!c.whole) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        p.part_o = reinterpret_cast<float *>(ws);
        p.part_ml = reinterpret_cast<float *>(ws + c.o_bytes);
        p.plan = reinterpret_cast<int4 *>(ws + c.o_bytes + c.ml_bytes);
    }
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.max_len = max_seq_len;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.log2_block = block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    p.ranges = c.ranges;
    p.groups = c.groups;
    p.whole = c.whole;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const bool bf16 = dtype == PA_BF16;
    const LatentKernels k = rank == 512 ? (bf16 ? latent_kernels<true, 512>(c.nh) : latent_kernels<false, 512>(c.nh))
                                        : (bf16 ? latent_kernels<true, 256>(c.nh) : latent_kernels<false, 256>(c.nh));
    CUtensorMap map_rows, map_q;
    const int64_t row = rank + kLatRope;
    const int64_t dims[2] = {row, (int64_t)num_blocks * block_size}, step[1] = {row};
    const int64_t qdims[2] = {row, (int64_t)num_seqs * num_heads};
    if (!rows_tensor_map(&map_rows, pool, 2, dims, step, kUnit, bf16) ||
        !rows_tensor_map(&map_q, q, 2, qdims, step, c.nh, bf16) ||
        !ensure_smem_attr(reinterpret_cast<const void *>(k.decode), k.smem))
        return PA_ERR_CUDA;
    if (launch_pdl(k.decode, dim3((unsigned)(c.ranges * c.groups)), dim3(kLatThreads), (size_t)k.smem,
                   as_stream(stream), p, map_rows, map_q) != cudaSuccess)
        return PA_ERR_CUDA;
    if (!c.whole &&
        launch_pdl(k.join, dim3((unsigned)c.ranges, (unsigned)num_heads), dim3(kLatJoinThreads), 0,
                   as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
