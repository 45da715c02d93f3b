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
// S with the heads on the lanes: a thread owns a head's row.  O transposed: 128
// dims fill the lanes whatever the number of heads, RANK/128 * NH columns hold it,
// and the staged rows are its A operand as they lie (MN-major).  Two S buffers and O
// are in TMEM; Q stays in shared memory, the rows pass through a ring of tiles.
//
// A unit of 16 rows is one TMA copy: the pool seen as [rows / 8][RANK / 64 + 1 slabs]
// [8 rows][64 columns], a box of two 8-row groups with all their slabs (a copy a unit
// and slab, 36 a tile, is bound by the issue of copies: 85 clocks each).  So a slab's
// 8-row groups lie (RANK / 64 + 1) KiB apart, which is the operands' group stride.
// P.V takes a unit at a time and frees it.
//
// Roles (12 warps): 0 producer of rows (TMA boxes of 16 rows through the block
// table, and prefetches of whole units to L2 some tiles ahead); 1 issues q.K^T (and
// owns TMEM); 2-9 softmax and epilogue, two warpgroups that share the heads: one
// takes positions 0-31 of every tile and the first half of O's columns, the other
// the rest; 10 issues P.V; 11 loads Q.  The running maximum moves only when a tile
// exceeds it by more than kLazyRescale; then the halves exchange their maxima and
// O's columns are rescaled in TMEM.
//
// The batch's tiles are shared out evenly: range b of the launch is tiles
// [b per, (b + 1) per) of all sequences' tiles in a row, found from the lengths on
// the device, or sequence b where they are about even.  A CTA goes through its range's
// pieces of sequences; Q and the rows of the next piece are on their way while one
// ends.  A piece that is a whole sequence is written out; the others leave (m, l, O)
// and a second launch joins them.
//
// What bounds it (rank 512).  A tile's products are 36 instructions of 32 clocks for
// q.K^T (M = N = 64: their operands' 4 KiB from shared memory) and 16 of 48 for P.V,
// 1,920 clocks for up to 64 heads; its 73.7 KB are 3,150 clocks of an SM's share of the
// copy peak.  So up to 64 heads HBM bounds it, 128 heads (two CTAs on the same rows) the
// tensor pipe.  Beside 64 heads' queries two tiles fit: a stage's way (copy about 950
// clocks from L2, q.K 1,300, softmax 1,000, P.V 900) is longer than two tiles' products,
// which leaves the tensor pipe 71% busy in steady state.  Measured: 128 sequences of
// 513-8192 positions, 128 heads, 178-191 us (0.83 PFLOP/s); 16 of 16-32k, 64 heads, 84-91
// us (5.0-5.4 TB/s); one of 200,003, 32 heads, 52 us (6.1 TB/s from the first tile to the
// last).  Past 64 heads the groups are whole ones of 64: 65 heads take what 128 do (64
// sequences of 513-8192: 64 heads 71 us, 65 101, 96 103, 128 104).
// Issued from code that the compiler does not know to be a warp's, every instruction
// takes 64 clocks (the first of these 316 us then, 286 with that mended alone).
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa_decode.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kLatRope = 64;      // shared key values of a row
constexpr int kLatTile = 64;      // positions of a tile
constexpr int kLatWarps = 12;
constexpr int kLatSoftmax = 256;  // softmax threads: two warpgroups
constexpr int kLatThreads = kLatWarps * 32;
constexpr int kLatSmem = 232448;  // what a CTA may have
constexpr int kLatMisc = 2048;    // barriers and exchange
constexpr int kLatMaxLen = 1 << 24;  // positions (a CTA's whole sequence is a wait, below)
// Sequences are not cut where each has a range of its own and the longest is at most
// this many tiles above an even share: cutting costs a range the write of its partial
// results and all the joining launch.  Cut against whole, in us, of sequences of 8
// tiles: 4 of 64 heads (a share of 1 tile) 13.4 and 17.3, 20 (2) 16.3 and 17.4, 70 (4)
// 27.8 and 19.4, 64 of 128 heads (7) 33.7 and 21.8; of 12 tiles: 60 of 16 heads (5)
// 21.5 and 22.3, 140 (12) 33.2 and 27.3.
constexpr int kLatWhole = 5;

struct DecodeLatentParams {
    uint16_t *out;
    const uint16_t *pool;
    const int32_t *tables;
    const int32_t *lens;
    float *part_o;   // [ranges][groups][2][NH][RANK]
    float *part_ml;  // [ranges][groups][2][NH][2]: maximum (base 2), sum
    int4 *plan;      // [ranges]: sequence whose pieces begin in the range and go on, or -1
    int num_blocks, max_blocks, max_len, num_seqs, num_heads, log2_block;
    int ranges, groups;
    int whole;       // range b is sequence b, whatever the lengths
    float scale_log2;
    int *err;
};

template <int RANK, int NH>
struct LatShape {
    static constexpr int SLABS = RANK / 64 + 1;    // the last one rotary
    static constexpr int PAIRS = RANK / 128;
    static constexpr int Q_SLAB = NH * 128;
    static constexpr int GROUP = SLABS * 1024;     // 8 rows of all slabs
    static constexpr int UNIT = 2 * GROUP;         // 16 rows
    static constexpr int TILE = 4 * UNIT;
    static constexpr int P_BYTES = NH * 128;
    static constexpr int P_BUFS = RANK == 512 && NH == 64 ? 1 : 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + SLABS * Q_SLAB;
    static constexpr int OFF_RING = OFF_P + P_BUFS * P_BYTES;
    static constexpr int STAGES = (kLatSmem - 1024 - kLatMisc - OFF_RING) / TILE;
    static constexpr int OFF_MISC = OFF_RING + STAGES * TILE;
    static constexpr int SMEM_BYTES = OFF_MISC + kLatMisc + 1024;  // + slack to align the base
    static constexpr int S_COL = PAIRS * NH;       // TMEM: O first, then two S buffers
    // barriers
    static constexpr int FULL = 0, EMPTY = STAGES, Q_FULL = EMPTY + 4 * STAGES, Q_FREE = Q_FULL + 1,
                         S_FULL = Q_FREE + 1, S_FREE = S_FULL + 2, P_FULL = S_FREE + 2,
                         PV_DONE = P_FULL + 2, O_FREE = PV_DONE + 2, VOTE = O_FREE + 1,
                         DRAIN = VOTE + 1, BARS = DRAIN + 2;
    // behind the barriers: TMEM address, abort flag, scan scratch, sums; then the heads'
    // factors and two halves' maxima
    static constexpr int OFF_WORDS = OFF_MISC + 512, OFF_ALPHA = OFF_MISC + 1024;
    static_assert(BARS * 8 <= 512 && 3 * NH * 4 <= 1024, "misc");
    static_assert(STAGES >= 2 && S_COL + 2 * kLatTile <= 512, "rings, TMEM");
    static_assert(OFF_P % 1024 == 0 && OFF_RING % 1024 == 0 && SMEM_BYTES <= kLatSmem, "layout");
    // q.K reads 64 rows of A whatever NH: past a slab's own rows it meets other
    // operands, whose products end in lanes that nothing reads
    static_assert(OFF_P - Q_SLAB + 64 * 128 <= OFF_MISC, "A rows in shared memory");
};

// Length of a sequence, clamped to what the launch and the table cover.
__device__ __forceinline__ int latent_len(const DecodeLatentParams &p, int L, bool report) {
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

// The pieces of a range, in order: every role walks them by itself, the next
// sequence's length on its way meanwhile; by whole warps.
struct LatWalk {
    const DecodeLatentParams &p;
    int seq, tile, left;
    int len, n;    // of the current piece: the sequence's length, tiles
    bool more;     // the sequence goes on behind the range
    int ahead;     // length of the sequence after the current piece's
    __device__ __forceinline__ LatWalk(const DecodeLatentParams &prm, int s, int t, int l)
        : p(prm), seq(s), tile(t), left(l), ahead(s < prm.num_seqs ? prm.lens[s] : 0) {}
    __device__ __forceinline__ bool next() {  // the current piece's data, false at the end
        if (left <= 0 || seq >= p.num_seqs) return false;
        // (a shuffle's result is known to be the warp's: what follows from it stays in
        // uniform registers)
        len = __shfl_sync(kFullMask, latent_len(p, ahead, false), 0);
        if (seq + 1 < p.num_seqs) ahead = p.lens[seq + 1];
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

// Named barrier 1 over the softmax threads, true on all if any passed true.
__device__ __forceinline__ bool latent_bar_or(bool v) {
    int any;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.s32 pi, %1, 0;\n\t"
        "bar.red.or.pred po, 1, %2, pi;\n\t"
        "selp.s32 %0, 1, 0, po;\n\t}"
        : "=r"(any)
        : "r"((int)v), "n"(kLatSoftmax)
        : "memory");
    return any != 0;
}

// Largest (MAX) or smallest of 32 values, NaN left aside.
template <bool MAX>
__device__ __forceinline__ float top32(const float (&s)[32]) {
    float t[2] = {s[0], s[1]};
#pragma unroll
    for (int j = 2; j < 32; j += 2) {
        if constexpr (MAX) {
            if (j & 2) t[0] = max3(t[0], s[j], s[j + 1]);
            else t[1] = max3(t[1], s[j], s[j + 1]);
        } else {
            t[0] = fminf(t[0], s[j]);
            t[1] = fminf(t[1], s[j + 1]);
        }
    }
    return MAX ? fmaxf(t[0], t[1]) : fminf(t[0], t[1]);
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
    int *scan = words + 8;  // [kLatWarps] warp sums, then start sequence and tile
    float *alphas = reinterpret_cast<float *>(smem + S::OFF_ALPHA);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int group = blockIdx.x % p.groups, range = blockIdx.x / p.groups;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_rows);
        prefetch_tensormap(&map_q);
        for (int b = 0; b < S::BARS; ++b)
            mbar_init(&bar[b], (b >= S::S_FREE && b < S::PV_DONE) || b == S::O_FREE || b == S::VOTE
                                      ? kLatSoftmax / 32 : 1);
        *abort_flag = 0;
        words[4] = words[5] = 0;
        scan[kLatWarps] = p.num_seqs;
        scan[kLatWarps + 1] = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();

    // ---------------------------------------------------------- this CTA's range
    int seq0 = range, tile0 = 0, left;
    if (p.whole) {  // no sequence can be long enough to be cut
        left = latent_tiles(latent_len(p, p.lens[range], group == 0));
        tc_fence_before();
        __syncthreads();
    } else {
        int sum = 0, longest = 0, *longest_of = words + 32;
        for (int i = threadIdx.x; i < p.num_seqs; i += kLatThreads) {
            const int n = latent_tiles(latent_len(p, p.lens[i], blockIdx.x == 0));
            sum += n;
            longest = max(longest, n);
        }
        sum = __reduce_add_sync(kFullMask, sum);
        longest = __reduce_max_sync(kFullMask, longest);
        if (lane == 0) {
            scan[warp] = sum;
            longest_of[warp] = longest;
        }
        tc_fence_before();
        __syncthreads();
        int total = 0;
        longest = 0;
#pragma unroll
        for (int w = 0; w < kLatWarps; ++w) {
            total += scan[w];
            longest = max(longest, longest_of[w]);
        }
        const int per = (total + p.ranges - 1) / p.ranges;
        const bool whole = p.num_seqs <= p.ranges && longest <= per + kLatWhole;
        const int start = (int)min((int64_t)range * per, (int64_t)total);
        left = whole ? 0 : min(per, total - start);
        // the sequence and tile that the range begins with
        int before = 0;
        for (int base = 0; base < p.num_seqs && left > 0; base += kLatThreads) {
            const int i = base + (int)threadIdx.x;
            const int mine = i < p.num_seqs ? latent_tiles(latent_len(p, p.lens[i], false)) : 0;
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
                scan[kLatWarps] = i;
                scan[kLatWarps + 1] = start - first;
            }
            before += all;
            if (before > start) break;  // the same for all threads
        }
        __syncthreads();
        seq0 = scan[kLatWarps];
        tile0 = scan[kLatWarps + 1];
        if (whole && range < p.num_seqs) {
            seq0 = range;
            left = latent_tiles(latent_len(p, p.lens[range], false));
        }
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();  // the joining launch waits for this one's end by itself

    seq0 = __shfl_sync(kFullMask, seq0, 0);
    tile0 = __shfl_sync(kFullMask, tile0, 0);
    LatWalk walk(p, seq0, tile0, __shfl_sync(kFullMask, left, 0));
    bool ok = true;

    if (warp == 0) {
        // ---------------------------------------------------------- producer of rows
        // The table's entries of 32 units (8 tiles) are a warp's load, one window ahead
        // and the next sequence's first window with the current piece's; they are checked
        // when they come into use.
        const int log2_block = p.log2_block;
        auto entry = [&](int seq, int first, int u) -> int {
            const int64_t at = ((int64_t)first + u * kUnit) >> log2_block;
            return seq < p.num_seqs && at < p.max_blocks ? p.tables[(int64_t)seq * p.max_blocks + at] : 0;
        };
        auto unit_row = [&](int phys, int first, int u, int units) -> int {
            if (u >= units) return 0;
            if ((unsigned)phys >= (unsigned)p.num_blocks) {
                record_error(p.err, PA_ERR_BAD_INDEX);
                phys = 0;
            }
            return (phys << log2_block) + ((first + u * kUnit) & ((1 << log2_block) - 1));
        };
        // A unit's rows lie together: one prefetch brings them to L2, a tile before its
        // copy can go, or two where two CTAs read the same rows and wait for one another's.
        // (Farther ahead it only keeps the copies waiting: 16 sequences of 16-32k positions
        // 94 us without, 88, 90, 94 and 105 with one to four tiles; 128 heads of 513-8192
        // positions 219 without, 202, 188, 187 and 206.)
        const int far = p.groups > 1 ? 2 : 1;
        auto prefetch = [&](int row) {
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.pool + (int64_t)row * (RANK + kLatRope)),
                         "r"(kUnit * (RANK + kLatRope) * 2)
                         : "memory");
        };
        int st = 0, use = 0;
        int raw_first = entry(seq0, tile0 * kLatTile, lane);
        for (; ok && walk.next(); walk.advance()) {
            const int first = walk.tile * kLatTile;
            const int units = (min(walk.len - first, walk.n * kLatTile) + kUnit - 1) / kUnit;
            int raw = raw_first;
            int raw_next = units > 32 ? entry(walk.seq, first, 32 + lane) : 0;
            raw_first = entry(walk.seq + 1, 0, lane);
            if (walk.len == 0) continue;
            int rows_cur = unit_row(raw, first, lane, units), rows_next = 0;
            for (int t = 0; ok && t < walk.n; ++t) {
                if (t > 0 && (t & 7) == 0) rows_cur = rows_next;
                if ((t & 7) == 2 && 4 * (t - 2) + 32 < units) {
                    const int w = 4 * (t - 2) + 32;  // the next window's first unit
                    rows_next = unit_row(raw_next, first, w + lane, units);
                    raw_next = w + 32 < units ? entry(walk.seq, first, w + 32 + lane) : 0;
                }
                const int nu = min(units - 4 * t, 4);
                uint64_t *full = &bar[S::FULL + st];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int row = __shfl_sync(kFullMask, rows_cur, (t & 7) * 4 + u);
                    if (ok && use > 0)
                        ok = mbar_wait_or(&bar[S::EMPTY + 4 * st + u], (use - 1) & 1, abort_flag);
                    ok = __all_sync(kFullMask, ok);
                    if (ok && u < nu && elect_one()) {
                        if (u == 0) mbar_arrive_expect_tx(full, nu * S::UNIT);
                        tma_load_4d(smem + S::OFF_RING + st * S::TILE + u * S::UNIT, &map_rows, 0, 0, 0,
                                    row >> 3, full);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (++st == S::STAGES) st = 0, ++use;
                const int u = 4 * (t + far) + (lane & 3);
                const int r_cur = __shfl_sync(kFullMask, rows_cur, u & 31);
                const int r_next = __shfl_sync(kFullMask, rows_next, u & 31);
                if (lane < 4 && u < units) prefetch((u >> 5) == (t >> 3) ? r_cur : r_next);
            }
        }
        // every copy has landed before shared memory goes (a stage's last use)
        for (int i = 0; i < S::STAGES; ++i) {
            const int uses = use + (i < st);
            if (uses > 0) (void)mbar_wait(&bar[S::FULL + i], (uses - 1) & 1);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- q.K^T
        constexpr uint32_t idesc = f16_idesc(BF16, false, false, 64, kLatTile);
        const uint32_t base = smem_addr(smem);
        const uint64_t q_desc = sw128_desc(base + S::OFF_Q, 16, 1024);
        const uint64_t k_desc = sw128_desc(base + S::OFF_RING, 16, S::GROUP);
        int st = 0, use = 0, g = 0, piece = 0;
        for (; walk.next(); walk.advance()) {
            if (walk.len == 0) continue;
            mbar_wait_flow(&bar[S::Q_FULL], piece & 1, flag);
            for (int t = 0; t < walk.n; ++t, ++g) {
                const int b = g & 1;
                if (g >= 2) mbar_wait_flow(&bar[S::S_FREE + b], ((g >> 1) - 1) & 1, flag);
                mbar_wait_flow(&bar[S::FULL + st], use & 1, flag);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t k = k_desc + st * (S::TILE >> 4);
#pragma unroll
                    for (int i = 0; i < S::SLABS; ++i)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc_mma(tmem + S::S_COL + kLatTile * b, q_desc + ((i * S::Q_SLAB + ks * 32) >> 4),
                                   k + ((i * 1024 + ks * 32) >> 4), idesc, i > 0 || ks > 0);
                    if (t + 1 == walk.n) tc_commit(&bar[S::Q_FREE]);
                    tc_commit(&bar[S::S_FULL + b]);
                }
                __syncwarp();
                if (++st == S::STAGES) st = 0, ++use;
            }
            ++piece;
        }
        if (elect_one()) tc_commit(&bar[S::DRAIN]);
        (void)mbar_wait(&bar[S::DRAIN], 0);
        __syncwarp();
    } else if (warp == 10) {
        // ---------------------------------------------------------- P.V
        constexpr uint32_t idesc = f16_idesc(BF16, true, false, 128, NH);
        const uint32_t base = smem_addr(smem);
        const uint64_t p_desc = sw128_desc(base + S::OFF_P, 16, 1024);
        const uint64_t v_desc = sw128_desc(base + S::OFF_RING, 1024, S::GROUP);
        int st = 0, use = 0, g = 0, piece = 0;
        for (; walk.next(); walk.advance()) {
            if (walk.len == 0) continue;
            if (piece > 0) mbar_wait_flow(&bar[S::O_FREE], (piece - 1) & 1, flag);
            for (int t = 0; t < walk.n; ++t, ++g) {
                const int pb = g % S::P_BUFS;
                mbar_wait_flow(&bar[S::FULL + st], use & 1, flag);  // long since, as S came of it
                mbar_wait_flow(&bar[S::P_FULL + pb], (g / S::P_BUFS) & 1, flag);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t w = p_desc + pb * (S::P_BYTES >> 4);
                    const uint64_t v = v_desc + st * (S::TILE >> 4);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
#pragma unroll
                        for (int j = 0; j < S::PAIRS; ++j)
                            tc_mma(tmem + j * NH, v + ((u * S::UNIT + j * 2048) >> 4), w + u * 2, idesc,
                                   t > 0 || u > 0);
                        tc_commit(&bar[S::EMPTY + 4 * st + u]);
                    }
                    tc_commit(&bar[S::PV_DONE + pb]);
                }
                __syncwarp();
                if (++st == S::STAGES) st = 0, ++use;
            }
            ++piece;
        }
        if (elect_one()) tc_commit(&bar[S::DRAIN + 1]);
        (void)mbar_wait(&bar[S::DRAIN + 1], 0);
        __syncwarp();
    } else if (warp == 11) {
        // ---------------------------------------------------------- Q
        int piece = 0;
        for (; ok && walk.next(); walk.advance()) {
            if (walk.len == 0) continue;
            if (piece > 0) ok = mbar_wait_or(&bar[S::Q_FREE], (piece - 1) & 1, abort_flag);
            ok = __all_sync(kFullMask, ok);
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&bar[S::Q_FULL], S::SLABS * S::Q_SLAB);
                // rows past the last sequence read as zero, other heads' rows as they are
                for (int i = 0; i < S::SLABS; ++i)
                    tma_load_2d(smem + S::OFF_Q + i * S::Q_SLAB, &map_q, 64 * i,
                                walk.seq * p.num_heads + group * NH, &bar[S::Q_FULL]);
            }
            __syncwarp();
            ++piece;
        }
        if (piece > 0) (void)mbar_wait(&bar[S::Q_FULL], (piece - 1) & 1);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax / epilogue
        const int half = (warp - 2) >> 2;
        const int quad = warp & 3;                 // TMEM lanes this warp may access
        const int row = quad * 16 + lane;          // head of lanes 0-15 (M = 64: 16 lanes a quadrant)
        const int tid = threadIdx.x - 64;
        const int heads = min(NH, p.num_heads - group * NH);
        const bool mine = lane < 16 && row < heads;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        float *maxima = alphas + NH;               // [half][NH]
        float *sums = reinterpret_cast<float *>(words + 64);  // the second half's, at a piece's end
        constexpr int kPos = kLatTile / 2;         // positions of a half
        constexpr int kCols = S::PAIRS * NH / 2;   // O columns of a half
        // f16 weights as 2^7 of themselves: at most 2^15 with the lag of the maximum, and
        // normal down to 2^-21 of the largest
        constexpr float kLift = BF16 ? 0.f : 7.f;
        int g = 0, votes = 0;
        volatile int *asked = words + 4;           // by the parity of votes
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
                for (int h = half; h < heads; h += 2)
#pragma unroll
                    for (int j = 0; j < S::PAIRS; ++j) p.out[(out_row + h) * RANK + 128 * j + dim] = 0;
                continue;
            }
            float m_run = -INFINITY, l_run = 0.f;
            for (int t = 0; t < walk.n; ++t, ++g) {
                const int b = g & 1;
                bool fine = mbar_wait_or(&bar[S::S_FULL + b], (g >> 1) & 1, abort_flag);
                fine = __all_sync(kFullMask, fine);
                tc_fence_after();
                float s[kPos];
                tmem_ld32(tmem + lanes + S::S_COL + kLatTile * b + kPos * half, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[S::S_FREE + b]);
                const int valid = min(walk.len - (walk.tile + t) * kLatTile, kLatTile);
                const float sc = p.scale_log2;
                if (valid < kLatTile) {
#pragma unroll
                    for (int j = 0; j < kPos; ++j)  // NaN-safe select
                        s[j] = kPos * half + j < valid ? s[j] : sc > 0.f ? -INFINITY : INFINITY;
                }
                float mx = (sc > 0.f ? top32<true>(s) : top32<false>(s)) * sc;
                uint32_t w[kPos / 2];
                auto weigh = [&]() -> float {  // the weights' sum
                    const float from = (m_run == -INFINITY ? 0.f : m_run) - kLift;
                    const float2 sc2 = make_float2(sc, sc), from2 = make_float2(-from, -from);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int j = 0; j < kPos / 2; ++j) {
                        const float2 x = __ffma2_rn(make_float2(s[2 * j], s[2 * j + 1]), sc2, from2);
                        const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                        w[j] = narrow2<BF16>(e.x, e.y);
                    }
                    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                };
                // The first tile sets the maximum; later ones move it where a half asks for
                // it.  The weights by the old one are on their way while the warps vote.
                bool any = true;
                float sum = 0.f;
                if (t > 0) {
                    const bool ask = __any_sync(kFullMask, (mine && mx > m_run + kLazyRescale) || !fine);
                    if (lane == 0) {
                        if (ask) asked[votes & 1] = 1;
                        mbar_arrive(&bar[S::VOTE]);
                    }
                    sum = weigh();
                    fine = mbar_wait_or(&bar[S::VOTE], votes & 1, abort_flag) && fine;
                    fine = __all_sync(kFullMask, fine);
                    any = asked[votes & 1] != 0;
                    ++votes;
                }
                // (a vote that ran out is everyone's: the next wait for S ends all)
                if (any) {
                    if (mine) maxima[half * NH + row] = mx;
                    if (latent_bar_or(!fine)) {  // all end together
                        ok = false;
                        break;
                    }
                    if (mine) mx = fmaxf(mx, maxima[(1 - half) * NH + row]);
                    float alpha = 1.f;
                    if (mx > m_run + kLazyRescale) {
                        alpha = fast_exp2(m_run - mx);  // 0 from an empty maximum
                        m_run = mx;
                        l_run *= alpha;
                    }
                    if (t > 0) {
                        if (mine && half == 0) alphas[row] = alpha;
                        if (tid == 0) asked[(votes - 1) & 1] = 0;  // everyone has read it
                        fine = pv_done(g - 1);  // O at rest
                        if (latent_bar_or(!fine)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = kCols * half; c < kCols * (half + 1); c += 16) {
                            float o[16];
                            tmem_load16(tmem + lanes + c, o);
                            const float4 *a = reinterpret_cast<const float4 *>(alphas + c % NH);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 f = a[i];
                                o[4 * i] *= f.x, o[4 * i + 1] *= f.y;
                                o[4 * i + 2] *= f.z, o[4 * i + 3] *= f.w;
                            }
                            tmem_store16(tmem + lanes + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                if (any) sum = weigh();
                l_run += sum;
                if (g >= S::P_BUFS) fine = fine && pv_done(g - S::P_BUFS);  // P's buffer is free
                if (valid < kLatTile) {
                    // rows past the length: P is 0 there, and V must be finite
                    fine = fine && mbar_wait_or(&bar[S::FULL + g % S::STAGES], (g / S::STAGES) & 1, abort_flag);
                    uint8_t *tile = smem + S::OFF_RING + (g % S::STAGES) * S::TILE;
                    for (int i = tid; i < (kLatTile - valid) * (RANK / 8); i += kLatSoftmax) {
                        const int r = valid + i / (RANK / 8), c = i % (RANK / 8);
                        *reinterpret_cast<uint4 *>(tile + (r >> 3) * S::GROUP + (c >> 3) * 1024 +
                                                   (r & 7) * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (!fine) *abort_flag = 1;  // the next wait for S ends all
                if (mine) {
                    uint8_t *to = smem + S::OFF_P + (g % S::P_BUFS) * S::P_BYTES + (row >> 3) * 1024 +
                                  (row & 7) * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(to + (((4 * half + j) ^ (row & 7)) << 4)) =
                            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[S::P_FULL + g % S::P_BUFS]);
            }
            if (!ok) break;
            if (mine && half == 1) sums[row] = l_run;
            if (latent_bar_or(!pv_done(g - 1))) {
                ok = false;
                break;
            }
            if (mine && half == 0) l_run += sums[row];
            tc_fence_after();
            const bool whole = walk.tile == 0 && !walk.more;
            if (whole) {
                if (mine && half == 0) alphas[row] = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : l_run;
                latent_bar_or(false);
                auto put = [&](auto all) {  // all: every head of the group is there
#pragma unroll 1
                    for (int c = kCols * half; c < kCols * (half + 1); c += 16) {
                        float o[16];
                        tmem_load16(tmem + lanes + c, o);
                        const int h0 = c % NH, j = c / NH;
                        uint16_t *to = p.out + (out_row + h0) * RANK + 128 * j + dim;
                        const float4 *a = reinterpret_cast<const float4 *>(alphas + h0);
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 f = a[i / 4];
                            if (all.value || h0 + i < heads) to[i * RANK] = narrow1<BF16>(o[i] * f.x);
                            if (all.value || h0 + i + 1 < heads) to[(i + 1) * RANK] = narrow1<BF16>(o[i + 1] * f.y);
                            if (all.value || h0 + i + 2 < heads) to[(i + 2) * RANK] = narrow1<BF16>(o[i + 2] * f.z);
                            if (all.value || h0 + i + 3 < heads) to[(i + 3) * RANK] = narrow1<BF16>(o[i + 3] * f.w);
                        }
                    }
                };
                if (heads == NH)
                    put(std::true_type());
                else
                    put(std::false_type());
            } else {
                const int cut = walk.seq == seq0 && walk.tile == tile0 ? 0 : 1;
                const int64_t slot = ((int64_t)range * p.groups + group) * 2 + cut;
                if (walk.more && walk.tile == 0) {
                    const int rest = latent_tiles(walk.len) - walk.n;
                    plan = make_int4(walk.seq, cut, rest, 0);
                }
                if (mine && half == 0) {
                    p.part_ml[(slot * NH + row) * 2] = m_run;
                    p.part_ml[(slot * NH + row) * 2 + 1] = l_run;
                }
                float *part = p.part_o + slot * NH * RANK + dim;
#pragma unroll 1
                for (int c = kCols * half; c < kCols * (half + 1); c += 16) {
                    float o[16];
                    tmem_load16(tmem + lanes + c, o);
                    const int h0 = c % NH, j = c / NH;
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(h0 + i) * RANK + 128 * j] = o[i];  // heads that are not there too
                }
            }
            tc_fence_before();
            latent_bar_or(false);  // O, the factors and the sums have been read
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

// Joins the pieces of the sequences that ranges cut:
//   M = max m_i;  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i
// A unit of work is a head of such a sequence, or a part of its values; a warp takes
// whole units, or some warps of a block share one's pieces, as there are many units
// or few: one wave of blocks, each of which lists the cut sequences for itself.
// (A block a range and head instead, most of them with nothing to join, took longer
// than the joining: 128 sequences of 513 to 8,192 positions and 128 heads 227 us a
// call, 198 with this.)
constexpr int kLatJoinWarps = 8, kLatJoinThreads = kLatJoinWarps * 32;
constexpr int kLatMaxRanges = kLatJoinThreads;

// A warp's share of one unit: OWN float4 a lane from chunk `first` on of the head's
// values, of pieces part, part + share, ...  The first sixteen loads go out before the
// weights are known.
template <int OWN, int NH, int RANK, typename SlotOf>
__device__ __forceinline__ void latent_join(const DecodeLatentParams &p, float4 (&acc)[RANK / 128],
                                            float *weight, int n, int row, int first, int part,
                                            int share, SlotOf slot_of) {
    constexpr int BATCH = 16 / OWN;
    const int lane = threadIdx.x & 31;
    float4 v[BATCH][OWN];
    auto load = [&](int i0) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int i = i0 + b * share;
#pragma unroll
            for (int k = 0; k < OWN; ++k)
                v[b][k] = i < n ? reinterpret_cast<const float4 *>(
                                      p.part_o + (slot_of(i) * NH + row) * RANK)[32 * (first + k) + lane]
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    load(part);
    float2 ml[kLatMaxRanges / 32];
    float M = -INFINITY, total = 0.f;
#pragma unroll
    for (int j = 0; j < kLatMaxRanges / 32; ++j) {
        const int i = lane + 32 * j;
        ml[j] = i < n ? *reinterpret_cast<const float2 *>(p.part_ml + (slot_of(i) * NH + row) * 2)
                      : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, ml[j].x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
#pragma unroll
    for (int j = 0; j < kLatMaxRanges / 32; ++j) {
        const float w = ml[j].x == -INFINITY ? 0.f : fast_exp2(ml[j].x - M);
        weight[lane + 32 * j] = w;
        total += w * ml[j].y;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    const float inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
    __syncwarp();
    for (int i0 = part; i0 < n; i0 += BATCH * share) {
        if (i0 > part) load(i0);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int i = i0 + b * share;
            if (i < n) {
                const float w = weight[i] * inv;
#pragma unroll
                for (int k = 0; k < OWN; ++k) {
                    acc[k].x += w * v[b][k].x, acc[k].y += w * v[b][k].y;
                    acc[k].z += w * v[b][k].z, acc[k].w += w * v[b][k].w;
                }
            }
        }
    }
}

template <bool BF16, int RANK, int NH>
__global__ void __launch_bounds__(kLatJoinThreads) latent_join_kernel(
    const __grid_constant__ DecodeLatentParams p) {
    constexpr int CHUNKS = RANK / 128;  // float4 a lane for all of a head's values
    __shared__ int4 plans[kLatMaxRanges];  // sequence, cut, further pieces, range
    __shared__ int counts[kLatJoinWarps], most[kLatJoinWarps];
    __shared__ float weights[kLatJoinWarps][kLatMaxRanges];
    __shared__ float4 sums[kLatJoinWarps][CHUNKS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    int4 plan = make_int4(-1, 0, 0, 0);
    if (threadIdx.x < p.ranges) plan = p.plan[threadIdx.x];
    plan.w = threadIdx.x;
    const unsigned live = __ballot_sync(kFullMask, plan.x >= 0);
    const int deep = __reduce_max_sync(kFullMask, plan.x >= 0 ? plan.z + 1 : 0);
    if (lane == 0) {
        counts[warp] = __popc(live);
        most[warp] = deep;
    }
    __syncthreads();
    int at = 0, cut = 0, pieces = 0;
#pragma unroll
    for (int w = 0; w < kLatJoinWarps; ++w) {
        if (w < warp) at += counts[w];
        cut += counts[w];
        pieces = max(pieces, most[w]);
    }
    if (plan.x >= 0) plans[at + __popc(live & ((1u << lane) - 1))] = plan;
    __syncthreads();
    const int items = cut * p.num_heads, warps = gridDim.x * kLatJoinWarps;
    int split = 1, share = 1;  // parts of a head's values, warps a unit
    while (split < CHUNKS && items * split * 2 <= warps) split *= 2;
    while (share < kLatJoinWarps && share * 2 <= pieces && items * split * share * 2 <= warps) share *= 2;
    const int own = CHUNKS / split, units = items * split, per = kLatJoinWarps / share;
    const int part = warp % share;
    for (int base = blockIdx.x * per; base < units; base += gridDim.x * per) {
        const int unit = base + warp / share;
        float4 acc[CHUNKS];
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int item = unit / split, first = (unit % split) * own;
        const int h = item % p.num_heads, group = h / NH, row = h % NH;
        if (unit < units) {
            plan = plans[item / p.num_heads];
            auto slot_of = [&](int i) -> int64_t {
                return ((int64_t)(plan.w + i) * p.groups + group) * 2 + (i == 0 ? plan.y : 0);
            };
            if (own == 1)
                latent_join<1, NH, RANK>(p, acc, weights[warp], plan.z + 1, row, first, part, share, slot_of);
            else if (own == 2)
                latent_join<2, NH, RANK>(p, acc, weights[warp], plan.z + 1, row, first, part, share, slot_of);
            else
                latent_join<CHUNKS, NH, RANK>(p, acc, weights[warp], plan.z + 1, row, first, part, share,
                                              slot_of);
        }
        if (share > 1) {
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) sums[warp][k][lane] = acc[k];
            __syncthreads();
            if (part == 0) {
                for (int w = 1; w < share; ++w)
#pragma unroll
                    for (int k = 0; k < CHUNKS; ++k) {
                        const float4 v = sums[warp + w][k][lane];
                        acc[k].x += v.x, acc[k].y += v.y, acc[k].z += v.z, acc[k].w += v.w;
                    }
            }
            __syncthreads();
        }
        if (part == 0 && unit < units) {
            uint2 *to = reinterpret_cast<uint2 *>(p.out + ((int64_t)plan.x * p.num_heads + h) * RANK) +
                        32 * first + lane;
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k)
                if (k < own)
                    to[32 * k] = make_uint2(narrow2<BF16>(acc[k].x, acc[k].y), narrow2<BF16>(acc[k].z, acc[k].w));
        }
        __syncwarp();
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
    if (c.ranges > kLatMaxRanges) c.ranges = kLatMaxRanges;
    const int tiles = (max_seq_len + kLatTile - 1) / kLatTile;
    c.whole = num_seqs <= c.ranges && tiles <= kLatWhole + 1;  // an even share is a tile at least
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
    // positions that a sequence is taken to have at most
    const int64_t cover = (int64_t)max_blocks_per_seq * block_size;
    const int64_t longest = max_seq_len < cover ? max_seq_len : cover;
    if ((int64_t)num_blocks * block_size >= 1ll << 31 || cover >= 1ll << 31 ||
        (longest / kLatTile + 1) * num_seqs >= 1ll << 31)
        return PA_ERR_INVALID;
    // a CTA may have a whole sequence, and its next queries wait for the end of it: well
    // within the limit of a wait (64 positions take about 1.7 us)
    if (longest > kLatMaxLen) return PA_ERR_INVALID;
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
    p.pool = static_cast<const uint16_t *>(pool);
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
    p.scale_log2 = latent_scale(scale);
    const bool bf16 = dtype == PA_BF16;
    const LatentKernels k = rank == 512 ? (bf16 ? latent_kernels<true, 512>(c.nh) : latent_kernels<false, 512>(c.nh))
                                        : (bf16 ? latent_kernels<true, 256>(c.nh) : latent_kernels<false, 256>(c.nh));
    CUtensorMap map_rows, map_q;
    const int64_t row = rank + kLatRope;
    const int64_t qdims[2] = {row, (int64_t)num_seqs * num_heads}, step[1] = {row};
    const int64_t dims[4] = {64, 8, row / 64, (int64_t)num_blocks * block_size / 8};
    const int64_t steps[3] = {row, 64, 8 * row};
    const int box[4] = {64, 8, (int)(row / 64), kUnit / 8}, qbox[2] = {64, c.nh};
    if (!boxed_tensor_map(&map_rows, pool, 4, dims, steps, box, bf16) ||
        !boxed_tensor_map(&map_q, q, 2, qdims, step, qbox, bf16) ||
        !ensure_smem_attr(reinterpret_cast<const void *>(k.decode), k.smem))
        return PA_ERR_CUDA;
    if (launch_pdl(k.decode, dim3((unsigned)(c.ranges * c.groups)), dim3(kLatThreads), (size_t)k.smem,
                   as_stream(stream), p, map_rows, map_q) != cudaSuccess)
        return PA_ERR_CUDA;
    if (!c.whole &&
        launch_pdl(k.join, dim3((unsigned)(2 * sms)), dim3(kLatJoinThreads), 0,
                   as_stream(stream), p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
