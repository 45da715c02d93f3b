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
// Roles (11 warps): 0 producer (TMA); 1 issues every product (and owns TMEM);
// 2-5 softmax and epilogue of tile A, 6-9 of tile B: thread r of four warps owns
// row r (TMEM lane r), so maxima and sums need no exchange; 10 fetches the CTA's
// next work.  The products of a tile are issued in the order q.K(t), P.V(t),
// q.K(t + 1): S(t + 1) may take P(t)'s place, and once it is there, O is at rest for
// the lazy rescale.
//
// The launch has a block for every (256 queries, head, sequence) up to the longest
// sequence; or, where most of these would have no queries, for every piece of work that
// the numbers of tokens and sequences allow, which the fetching warp finds from the
// sequences' starts.  A CTA that runs takes over blocks that have not been launched yet
// (clusterlaunchcontrol), so the next work's queries and keys load, and its first
// products run, while the softmax of the last ends.  Where there are few blocks and many
// keys, a cluster shares a block's keys instead and joins its sums through distributed
// shared memory.
//
// What bounds it.  128 keys of one tile are 12 instructions of 64 clocks and 16 of 32,
// 1,280 clocks of the tensor pipe; their softmax, 128 exponentials a thread, runs under
// the other tile's.  2 x 2-4k queries behind 6-12k keys, 32 heads: 810-1,050 us, 1.2-1.55
// PFLOP/s, 70-92% of a library product's sustained rate at the power limit; 16 prompts of
// 31-2,048 tokens, 16 heads: 120-126 us, 0.87 PFLOP/s: half-masked tiles (15% of the work),
// the ends of pieces of work (a tile's last softmax, its output and the next one's first
// in turn), and the launch's end.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa_decode.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kPreRope = 64, kPreNope = 128, kPreValue = 128;
constexpr int kPreRows = 128;   // query rows of a tile
constexpr int kPreKeys = 128;   // keys of a tile
constexpr int kPreSlab = kPreKeys * 128;
constexpr int kPreSlots = 8;    // slabs of the ring
constexpr int kPreWarps = 11;
constexpr int kPreThreads = kPreWarps * 32;
constexpr int kPreOffRing = 2 * 3 * kPreSlab;
constexpr int kPreOffBar = kPreOffRing + kPreSlots * kPreSlab;
constexpr int kPreSmem = kPreOffBar + 1024 + 1024;  // + slack to align the base to 1 KiB
constexpr int kPreColS = 0, kPreColO = 256;        // TMEM columns: S_A S_B O_A O_B
// Up to so many (key, head) pairs the longest tiles of all heads go first, past them
// those of each head in turn, so that a head's tiles read its keys from L2 together.
// By length against by head, in us: one sequence of 8,192, 16 heads (131,000 pairs) 254 and 336; 16 ragged prompts, 16
// heads (266,000) 143 and 167; 8 pieces behind a context, 8 heads (394,000) 353 and 368;
// 4, 16 heads (674,000) 702 and 725; 64 ragged prompts, 4 heads (789,000) 810 and 810; 8
// pieces, 16 heads (892,000) 983 and 950, 32 heads (1,792,000) 2,072 and 1,938.  One long
// sequence gains for longer: 32,768, 32 heads (1,049,000) 6,745 and 7,403.
constexpr int kPreByLength = 400000;
// 256 queries meet 2^24 keys in about 0.3 s; the next work's queries and the fetching
// warp wait for the end of one such piece, which a wait's limit has to cover.
constexpr int kPreMaxKeys = 1 << 24;
// A work's keys are shared out over up to eight CTAs, at least kPreSplitTiles tiles
// each, as far as one wave holds them (1 query behind 8,000 keys, 4 heads: 89 us whole,
// 22 with eight; 300 behind 6,000 twice, 8 heads: 72 and 31 with four), and over two
// where there is about a wave of work, up to a fifth more, and sequences are long
// enough to even it out (in pieces of work and tiles of keys: 126 of 125 214 us whole,
// 118 in two; 160 of 63 180 and 157; 128 of 63 111 and 95; but 128 of 32 61 and 70, 224
// of 47 130 and 148, 240 of 47 115 and 128).
constexpr int kPreMaxSplit = 8, kPreSplitTiles = 4, kPreSplitLong = 40;
constexpr int kPreQueue = 3;                       // work in hand: being done and fetched
// Blocks of a launch at most; past them a block stands for several pieces of work in a
// row.  It bounds the blocks without work that a CTA takes over in a row (6,900 of 152)
// while its other roles wait.
constexpr int kPreBlocks = 1 << 20;
// A block for every (256 queries, head, sequence) while these are up to so many times
// the pieces of work that there can be: a piece is found faster so, but a block without
// queries costs its CTA about a microsecond.  16 heads, so and found from the starts:
// 255 sequences of 30-70 tokens 100 us and 105, one of 8,192 241 and 254, 16 of 31-2,048
// (1.6 times as many) 119 and 121, but 157 and 121 with a bound on lengths eight times
// as large; 255 of 30-70 and one of 8,192 (25 times) 496 and 315.
constexpr int kPreSparse = 2;
constexpr int kPreChunk = 256;                     // sequences that the fetching warp holds
static_assert(kPreSmem <= 232448, "shared memory");

// K and V of a tile are awaited as a whole: group 2 t is K's slabs, 2 t + 1 V's.  At
// most four groups lie in the ring.
constexpr int kPreGroups = 4;

enum PreBar { kPreFull = 0, kPreEmpty = kPreGroups, kPreQFull = kPreEmpty + kPreSlots,
              kPreQFree = kPreQFull + 2, kPreSFull = kPreQFree + 2, kPrePReady = kPreSFull + 2,
              kPreODone = kPrePReady + 2, kPreOFree = kPreODone + 2, kPreWorkFull = kPreOFree + 2,
              kPreWorkFree = kPreWorkFull + kPreQueue, kPreClaim = kPreWorkFree + kPreQueue,
              kPreDrain, kPreBars };
constexpr int kPreOffWork = kPreOffBar + 512;      // the queue, then the claim's answer
constexpr int kPreOffClaim = kPreOffWork + kPreQueue * 32;
constexpr int kPreOffWords = kPreOffClaim + 16;    // TMEM address, abort flag
static_assert(kPreBars * 8 <= 512 && kPreOffWords + 8 <= kPreOffBar + 1024, "barriers");

// 256 queries of a head of a sequence.
struct PreWork {
    int q0, n_q, k0, n_k;  // the sequence's tokens; n_q < 0: no more work
    int head, first;       // first query in the sequence
    int from, upto;        // key tiles
};

struct PrefillLatentParams {
    uint16_t *out;
    const int32_t *q_starts, *k_starts;
    int total_q, total_k, max_q, num_heads, causal;
    int wide;       // out lies on a 32-byte boundary
    int num_seqs;
    int per;        // pieces of work a block; 0: a block is (256 queries, head, sequence)
    int split;      // CTAs of a cluster that share a work's keys
    int by_length;  // order of work: grid (heads, sequences, tiles) instead of (tiles, heads, sequences)
    float scale_log2;
    int *err;
};

// Keys that rows [first + 128 x, + 128) of a sequence meet, in tiles of the work's.
__device__ __forceinline__ int prefill_tiles(const PreWork &w, int x, int causal) {
    const int a = w.first + x * kPreRows, b = min(a + kPreRows, w.n_q);
    if (a >= w.n_q) return 0;
    const int keys = causal ? min(w.n_k - w.n_q + b, w.n_k) : w.n_k;
    const int end = keys > 0 ? (keys + kPreKeys - 1) / kPreKeys : 0;
    return max(min(end, w.upto) - w.from, 0);
}

// A sequence's tokens; false: it has none, or its starts are bad.
__device__ __forceinline__ bool prefill_sequence(const PrefillLatentParams &p, int seq, PreWork &w, bool report) {
    const int q0 = p.q_starts[seq], q1 = p.q_starts[seq + 1], k0 = p.k_starts[seq], k1 = p.k_starts[seq + 1];
    const bool good = q0 >= 0 && q1 >= q0 && q1 - q0 <= p.max_q && q1 <= p.total_q && k0 >= 0 && k1 >= k0 &&
                      k1 <= p.total_k;
    if (!good && report) record_error(p.err, PA_ERR_BAD_INDEX);
    w.q0 = q0, w.n_q = q1 - q0, w.k0 = k0, w.n_k = k1 - k0;
    return good && q1 > q0;
}

// Where most blocks of (256 queries, head, sequence) would be empty: the pieces of work
// in their order, walked by a whole warp that holds the tiles of a chunk of sequences
// (32 k + lane in tiles[k]).  A chunk's follow the last one's.  Within a chunk the order
// is that of the blocks: by length, the longest sequences' last tiles of all heads first
// (tiles down, then sequences, then heads); or sequence by sequence, of each head in
// turn, the last tile first.
struct PreList {
    static constexpr int ROWS = kPreChunk / 32;
    const PrefillLatentParams &p;
    const int lane;
    int base;                   // the chunk's first sequence
    int tiles[ROWS];            // of 256 queries
    unsigned marks[ROWS];       // by length: lanes that reach `level`; else the row's tiles up to a lane
    int total, top;             // tiles of the chunk; of its longest sequence
    int level, above, there;    // by length: tiles past `level`, and on it
    int64_t before;             // pieces of work in earlier chunks

    __device__ __forceinline__ PreList(const PrefillLatentParams &prm, int l) : p(prm), lane(l) {}

    __device__ __forceinline__ void restart() {
        before = 0;
        load(0);
    }

    __device__ __forceinline__ void set_level(int l, int past) {
        level = l;
        above = past;
        there = 0;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            marks[k] = __ballot_sync(kFullMask, tiles[k] > level);
            there += __popc(marks[k]);
        }
    }

    // Sequences [first, first + kPreChunk).  A bad one has no work.
    __device__ __forceinline__ void load(int first) {
        base = first;
        int sum = 0, longest = 0;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int s = first + 32 * k + lane;
            PreWork w;
            tiles[k] = 0;
            if (s < p.num_seqs && prefill_sequence(p, s, w, true))
                tiles[k] = (int)(((unsigned)w.n_q + 2 * kPreRows - 1) / (2 * kPreRows));
            sum += tiles[k];
            longest = max(longest, tiles[k]);
        }
        total = __reduce_add_sync(kFullMask, sum);
        top = __reduce_max_sync(kFullMask, longest);
        if (p.by_length) {
            set_level(top - 1, 0);
        } else {
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                int upto = tiles[k];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(kFullMask, upto, o);
                    if (lane >= o) upto += v;
                }
                marks[k] = upto;
            }
        }
    }

    // Piece of work `item`; false: there are not so many.
    __device__ __forceinline__ bool find(int64_t item, PreWork &w) {
        const unsigned heads = p.num_heads;
        if (item < before) restart();
        while (item >= before + (int64_t)total * heads) {
            if (base + kPreChunk >= p.num_seqs) return false;
            before += (int64_t)total * heads;
            load(base + kPreChunk);
        }
        // (a chunk's pieces are fewer than 2^31: their outputs lie in memory)
        unsigned r = (unsigned)(item - before);
        int row = 0, mine, tile;
        if (p.by_length) {
            w.head = (int)(r % heads);
            r /= heads;
            if ((int)r < above) set_level(top - 1, 0);
            while ((int)r >= above + there) set_level(level - 1, above + there);
            tile = level;
            r -= above;  // the r-th of the sequences that reach it
            unsigned mask = marks[0];
#pragma unroll
            for (int k = 1; k < ROWS; ++k)
                if (r >= (unsigned)__popc(mask) && row == k - 1) {
                    r -= __popc(mask);
                    mask = marks[k];
                    row = k;
                }
            mine = __ffs(__ballot_sync(kFullMask, (mask >> lane & 1) &&
                                                      __popc(mask & ((1u << lane) - 1)) == (int)r)) - 1;
        } else {
            unsigned upto = marks[0], n = tiles[0];
#pragma unroll
            for (int k = 1; k < ROWS; ++k) {
                const unsigned all = __shfl_sync(kFullMask, upto, 31) * heads;
                if (r >= all && row == k - 1) {
                    r -= all;
                    upto = marks[k], n = tiles[k];
                    row = k;
                }
            }
            mine = __ffs(__ballot_sync(kFullMask, upto * heads > r)) - 1;
            n = __shfl_sync(kFullMask, n, mine);
            r -= (__shfl_sync(kFullMask, upto, mine) - n) * heads;
            w.head = (int)(r / n);
            tile = (int)(n - 1 - r % n);
        }
        w.first = tile * 2 * kPreRows;
        return prefill_sequence(p, base + 32 * row + mine, w, false);
    }
};

// Largest (MAX) or smallest of 128 values, NaN left aside.
template <bool MAX>
__device__ __forceinline__ float top128(const float (&s)[kPreKeys]) {
    float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int j = 4; j < kPreKeys; j += 2) {
        float &m = t[(j >> 1) & 3];
        m = MAX ? max3(m, s[j], s[j + 1]) : fminf(fminf(m, s[j]), s[j + 1]);
    }
    return MAX ? fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) : fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
}

// 32 bytes, in one store where the address allows it (a thread stores its own row, so
// a store of a warp touches 32 lines however short it is).
__device__ __forceinline__ void store32(uint16_t *to, const uint32_t *y, int wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(y[0]),
                     "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(to)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4 *>(to)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

// The CTAs of a cluster have had shares of one work's keys: their sums meet through
// distributed shared memory.  M = max m_c, out = sum 2^(m_c - M) O_c / sum 2^(m_c - M) l_c.
// Each CTA weighs its O rows and sends them to the CTA that owns the row, which adds
// them up.  Every product and copy has ended, so the shared memory is free: the rows'
// slots lie first in it, [tile][sender][owned row][128 + 4].
template <bool BF16>
__device__ __forceinline__ void prefill_join(const PrefillLatentParams &p, const PreWork &w, uint8_t *smem,
                                          uint32_t tmem, int warp, int lane, float m_run, float l_run) {
    constexpr int kStep = kPreValue + 4;
    constexpr int kSlots = 2 * kPreRows;  // C senders of 128 / C rows of either tile
    static_assert(kSlots * (kStep + 1) * 4 + 2 * kPreRows * 8 <= kPreOffBar, "shared memory");
    float *slots = reinterpret_cast<float *>(smem);
    float2 *ml = reinterpret_cast<float2 *>(slots + kSlots * kStep);  // [tile][row]
    float *weights = reinterpret_cast<float *>(ml + 2 * kPreRows);          // [tile][owned row][sender]
    const int C = p.split, R = kPreRows / C, rank = (int)cluster_ctarank();
    const bool softmax = warp >= 2 && warp < 10;
    const int x = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;
    if (softmax) ml[x * kPreRows + r] = make_float2(l_run == 0.f ? -INFINITY : m_run, l_run);
    __syncwarp();
    cluster_sync();
    if (softmax) {
        float M = -INFINITY, L = 0.f, own = 0.f;
        const uint32_t at = smem_addr(ml + x * kPreRows + r);
        for (int c = 0; c < C; ++c) M = fmaxf(M, ld_cluster_f32(map_cluster(at, c)));
        auto factor = [&](int c) -> float {
            const float m = ld_cluster_f32(map_cluster(at, c));
            return m == -INFINITY ? 0.f : fast_exp2(m - M);
        };
        for (int c = 0; c < C; ++c) L += factor(c) * ld_cluster_f32(map_cluster(at + 4, c));
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int owner = r / R, slot = r % R;
        for (int c = 0; c < C; ++c) {
            const float f = factor(c) * inv;
            if (c == rank) own = f;
            if (owner == rank) weights[(x * R + slot) * C + c] = f;
        }
        const uint32_t to = map_cluster(smem_addr(slots + ((x * C + rank) * R + slot) * kStep), owner);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + kPreColO + 128 * x + 32 * c, o);
            if (own != 0.f) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    st_cluster_f4(to + (32 * c + 4 * i) * 4,
                                  make_float4(o[4 * i] * own, o[4 * i + 1] * own, o[4 * i + 2] * own,
                                              o[4 * i + 3] * own));
            }
        }
    }
    __syncwarp();
    cluster_sync();
    if (softmax) {
        for (int i = r; i < R * (kPreValue / 8); i += kPreRows) {
            const int slot = i / (kPreValue / 8), d = i % (kPreValue / 8) * 8;
            const int row = w.first + x * kPreRows + rank * R + slot;
            if (row >= w.n_q) continue;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            for (int c = 0; c < C; ++c) {
                if (weights[(x * R + slot) * C + c] == 0.f) continue;  // nothing was sent
                const float4 *v = reinterpret_cast<const float4 *>(slots + ((x * C + c) * R + slot) * kStep + d);
                a.x += v[0].x, a.y += v[0].y, a.z += v[0].z, a.w += v[0].w;
                b.x += v[1].x, b.y += v[1].y, b.z += v[1].z, b.w += v[1].w;
            }
            *reinterpret_cast<uint4 *>(p.out + ((int64_t)(w.q0 + row) * p.num_heads + w.head) * kPreValue + d) =
                make_uint4(narrow2<BF16>(a.x, a.y), narrow2<BF16>(a.z, a.w), narrow2<BF16>(b.x, b.y),
                           narrow2<BF16>(b.z, b.w));
        }
    }
}

// SPLIT: the CTAs of a cluster share one block's keys, and take over no others.
template <bool BF16, bool SPLIT>
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
    int4 *queue = reinterpret_cast<int4 *>(smem + kPreOffWork);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kPreOffWords);
    int *flag = reinterpret_cast<int *>(smem + kPreOffWords + 4);
    volatile int *abort_flag = flag;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int split = SPLIT ? p.split : 1;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        prefetch_tensormap(&map_pe);
        for (int b = 0; b < kPreBars; ++b) {
            const bool softmax = (b >= kPrePReady && b < kPreODone) || (b >= kPreOFree && b < kPreWorkFull);
            const bool work = b >= kPreWorkFree && b < kPreClaim;
            mbar_init(&bar[b], softmax ? 4 : work ? 10 : 1);  // ten warps end a turn
        }
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
    pdl_wait();
    pdl_trigger();
    bool ok = true;
    float m_of = -INFINITY, l_of = 0.f;  // a softmax thread's row, for the cluster
    // The work of turn i, once it is there (roles take it in turns 0, 1, ...).
    auto read_work = [&](int turn) -> PreWork {
        const int4 a = queue[2 * (turn % kPreQueue)], b = queue[2 * (turn % kPreQueue) + 1];
        return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    };
    auto work_full = [&](int turn) -> uint64_t * { return &bar[kPreWorkFull + turn % kPreQueue]; };
    auto work_free = [&](int turn) -> uint64_t * { return &bar[kPreWorkFree + turn % kPreQueue]; };

    if (warp == 10) {
        // ---------------------------------------------------------- next work
        // by lane 0 where a block is (256 queries, head, sequence), by the warp where the
        // pieces of work are listed
        auto fetch = [&](auto is_listed) {
            constexpr bool LISTED = is_listed.value;
            auto agreed = [](bool v) -> bool {
                if constexpr (LISTED) v = __all_sync(kFullMask, v);
                return v;
            };
            int x = blockIdx.x / split, y = blockIdx.y, z = blockIdx.z, claims = 0;
            // a block that has not been launched yet becomes this CTA's; false: none is left
            auto claim = [&]() -> bool {
                if (lane == 0) {
                    fence_async_smem();  // the last answer has been read
                    mbar_arrive_expect_tx(&bar[kPreClaim], 16);
                    asm volatile(
                        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
                        "[%0], [%1];" ::"r"(smem_addr(smem + kPreOffClaim)), "r"(smem_addr(&bar[kPreClaim]))
                        : "memory");
                }
                if constexpr (LISTED) __syncwarp();
                ok = agreed(mbar_wait(&bar[kPreClaim], claims++ & 1));
                if (!ok) return false;
                uint32_t got;
                asm volatile(
                    "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
                    "ld.shared.b128 a, [%4];\n\t"
                    "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
                    "selp.u32 %0, 1, 0, p;\n\t"
                    "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
                    "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 "
                    "{%1, %2, %3, _}, a;\n\t}"
                    : "=&r"(got), "=&r"(x), "=&r"(y), "=&r"(z)
                    : "r"(smem_addr(smem + kPreOffClaim))
                    : "memory");
                if constexpr (LISTED) __syncwarp();  // before the next answer
                return got != 0;
            };
            PreList list(p, lane);
            int64_t item = 0, end = 1;
            if constexpr (LISTED) {
                item = (int64_t)x * p.per;
                end = item + p.per;
                list.restart();
            }
            // Of listed pieces, the CTA that has the first block goes on behind the last one: it
            // looks at every sequence's starts, and where some decrease, which makes a bad
            // sequence, those behind may have more queries together than the host counts.
            bool first = LISTED && x == 0, left = !SPLIT;
            for (int turn = 0;; ++turn) {
                if (turn >= kPreQueue) {
                    ok = agreed(mbar_wait_or(work_free(turn), (turn / kPreQueue - 1) & 1, abort_flag));
                    if (!ok) break;
                }
                PreWork w;
                bool found = false;
                while (!found) {
                    if (item == end) {
                        if (!left) break;
                        left = claim();  // if not, no more claims
                        if (left) {
                            item = LISTED ? (int64_t)x * p.per : 0;
                            end = LISTED ? item + p.per : 1;
                            first |= LISTED && x == 0;
                        } else if (first && ok) {
                            item = (int64_t)gridDim.x * p.per;
                            end = 1ll << 62;
                        } else {
                            break;
                        }
                    }
                    w.from = 0, w.upto = 0x7fffffff;
                    if constexpr (LISTED) {
                        found = list.find(item, w);
                        item = found ? item + 1 : end;
                    } else {
                        // the longest tiles of causal sequences come first: of each head in turn,
                        // or of all
                        const int last = (int)(p.by_length ? gridDim.z : gridDim.x / split) - 1;
                        w.first = (last - (p.by_length ? z : x)) * 2 * kPreRows;
                        w.head = p.by_length ? x : y;
                        found = prefill_sequence(p, p.by_length ? y : z, w, w.head == 0 && w.first == 0) &&
                                w.first < w.n_q;
                        item = end;
                    }
                    if (!found && !agreed(!*abort_flag)) break;
                }
                if (!found) w = {0, -1, 0, 0, 0, 0, 0, 0};  // no more work
                if constexpr (SPLIT) {  // this CTA's share of the keys
                    const int all = max(prefill_tiles(w, 0, p.causal), prefill_tiles(w, 1, p.causal));
                    const int per = (all + split - 1) / split;
                    w.from = per * (int)cluster_ctarank();
                    w.upto = w.from + per;
                }
                if (lane == 0) {
                    queue[2 * (turn % kPreQueue)] = make_int4(w.q0, w.n_q, w.k0, w.n_k);
                    queue[2 * (turn % kPreQueue) + 1] = make_int4(w.head, w.first, w.from, w.upto);
                    mbar_arrive(work_full(turn));
                }
                if (!found) break;
            }
        };
        if (!SPLIT && p.per > 0)
            fetch(std::bool_constant<!SPLIT>());
        else if (lane == 0)
            fetch(std::false_type());
        __syncwarp();
    } else if (warp == 0) {
        // ---------------------------------------------------------- producer
        if (lane == 0) {
            int u = 0, group = 0, loaded[2] = {0, 0};  // slabs, groups of them; queries of either tile
            uint64_t *full = nullptr;
            for (int turn = 0; ok; ++turn) {
                ok = mbar_wait_or(work_full(turn), (turn / kPreQueue) & 1, abort_flag);
                if (!ok) break;
                const PreWork w = read_work(turn);
                if (w.n_q < 0) break;
                const int tiles0 = prefill_tiles(w, 0, p.causal), tiles1 = prefill_tiles(w, 1, p.causal);
                const int end = u + 5 * max(tiles0, tiles1);
                auto load_q = [&](int x, int &count) -> bool {
                    if (count > 0 && !mbar_wait_or(&bar[kPreQFree + x], (count - 1) & 1, abort_flag))
                        return false;
                    ++count;
                    mbar_arrive_expect_tx(&bar[kPreQFull + x], 3 * kPreSlab);
                    for (int i = 0; i < 3; ++i)
                        tma_load_3d(smem + (3 * x + i) * kPreSlab, &map_q, 64 * i,
                                    w.q0 + w.first + x * kPreRows, w.head, &bar[kPreQFull + x]);
                    return true;
                };
                // Slab i of a tile: the keys' own values (two), the shared ones, V (two).  K's
                // three and V's two are awaited as one, on the barrier of the first.
                auto load = [&](int i, int key) -> bool {
                    const int slot = u % kPreSlots, use = u / kPreSlots;
                    if (use > 0 && !mbar_wait_or(&bar[kPreEmpty + slot], (use - 1) & 1, abort_flag))
                        return false;
                    uint8_t *to = smem + kPreOffRing + slot * kPreSlab;
                    if (i == 0 || i == 3) {
                        full = &bar[kPreFull + group % kPreGroups];
                        ++group;
                        mbar_arrive_expect_tx(full, (i == 0 ? 3 : 2) * kPreSlab);
                    }
                    if (i == 2)
                        tma_load_2d(to, &map_pe, 0, key, full);
                    else
                        tma_load_3d(to, i < 2 ? &map_k : &map_v, 64 * (i < 2 ? i : i - 3), key, w.head, full);
                    ++u;
                    return true;
                };
                if (tiles0 > 0) ok = load_q(0, loaded[0]);
                const int key0 = w.k0 + w.from * kPreKeys;
                for (int key = key0; ok && u < end; key += kPreKeys)
                    for (int i = 0; ok && i < 5; ++i) {
                        if (i == 3 && key == key0 && tiles1 > 0) ok = load_q(1, loaded[1]);
                        ok = ok && load(i, key);
                    }
                mbar_arrive(work_free(turn));
            }
            // every copy has landed before shared memory goes (each barrier's last use)
            for (int s = max(0, group - kPreGroups); s < group; ++s)
                (void)mbar_wait(&bar[kPreFull + s % kPreGroups], (s / kPreGroups) & 1);
            if (loaded[0] > 0) (void)mbar_wait(&bar[kPreQFull], (loaded[0] - 1) & 1);
            if (loaded[1] > 0) (void)mbar_wait(&bar[kPreQFull + 1], (loaded[1] - 1) & 1);
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
        int at[2] = {0, 0}, works[2] = {0, 0};  // P.V steps and pieces of work of either tile
        struct Turn {
            int turn, tiles0, tiles1, most, tile;  // most -1: no more work; tile: counted over all work
        };
        auto landed = [&](int group) {
            mbar_wait_flow(&bar[kPreFull + group % kPreGroups], (group / kPreGroups) & 1, flag);
        };
        // (a slab's first user waits for it; tile B uses it last where it reaches that far)
        auto issue_qk = [&](int x, const Turn &w, int t) {
            if (t == 0) mbar_wait_flow(&bar[kPreQFull + x], works[x] & 1, flag);
            if (x == 0 || t >= w.tiles0) landed(2 * (w.tile + t));
            const bool last = x == 1 || t >= w.tiles1;
            const bool done = t + 1 == (x ? w.tiles1 : w.tiles0);
            const int u = 5 * (w.tile + t);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int slot = (u + i) % kPreSlots;
                    const uint64_t q = q_desc + ((3 * x + i) * kPreSlab >> 4);
                    const uint64_t k = k_desc + slot * (kPreSlab >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma(tmem + kPreColS + 128 * x, q + ks * 2, k + ks * 2, idesc_qk, i > 0 || ks > 0);
                    if (last) tc_commit(&bar[kPreEmpty + slot]);
                }
                tc_commit(&bar[kPreSFull + x]);
                if (done) tc_commit(&bar[kPreQFree + x]);
            }
            __syncwarp();
        };
        auto issue_pv = [&](int x, const Turn &w, int t) {
            // O has been read where it begins anew
            if (t == 0 && works[x] > 0) mbar_wait_flow(&bar[kPreOFree + x], (works[x] - 1) & 1, flag);
            if (x == 0 || t >= w.tiles0) landed(2 * (w.tile + t) + 1);
            mbar_wait_flow(&bar[kPrePReady + x], at[x] & 1, flag);
            ++at[x];
            const bool last = x == 1 || t >= w.tiles1;
            const bool done = t + 1 == (x ? w.tiles1 : w.tiles0);
            const int u = 5 * (w.tile + t) + 3;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int slot = (u + i) % kPreSlots;
                    const uint64_t v = v_desc + slot * (kPreSlab >> 4);
#pragma unroll
                    for (int ks = 0; ks < kPreKeys / 16; ++ks)
                        tc_mma_ts(tmem + kPreColO + 128 * x + 64 * i, tmem + kPreColS + 128 * x + 8 * ks,
                                  v + ks * (2048 >> 4), idesc_pv, t > 0 || ks > 0);
                    if (last) tc_commit(&bar[kPreEmpty + slot]);
                }
                if (done) tc_commit(&bar[kPreODone + x]);
            }
            __syncwarp();
            if (done) ++works[x];
        };
        // The work of a turn, and the first one from there on that has keys (or the end).
        auto look = [&](int turn, int tile) -> Turn {
            mbar_wait_flow(work_full(turn), (turn / kPreQueue) & 1, flag);
            const PreWork w = read_work(turn);
            if (__any_sync(kFullMask, *abort_flag || w.n_q < 0)) return {turn, 0, 0, -1, tile};
            // by shuffles: values that the compiler knows to be the warp's
            const int tiles0 = __shfl_sync(kFullMask, prefill_tiles(w, 0, p.causal), 0);
            const int tiles1 = __shfl_sync(kFullMask, prefill_tiles(w, 1, p.causal), 0);
            return {turn, tiles0, tiles1, max(tiles0, tiles1), tile};
        };
        auto release = [&](int turn) {
            if (elect_one()) mbar_arrive(work_free(turn));
            __syncwarp();
        };
        auto keyed = [&](int turn, int tile) -> Turn {
            for (;; ++turn) {
                const Turn w = look(turn, tile);
                if (w.most != 0) return w;
                release(turn);
            }
        };
        auto start = [&](const Turn &w) {
            if (w.tiles0 > 0) issue_qk(0, w, 0);
            if (w.tiles1 > 0) issue_qk(1, w, 0);
        };
        Turn w = keyed(0, 0);
        start(w);
        while (w.most > 0) {
            for (int t = 0; t + 1 < w.most; ++t) {
                if (t < w.tiles0) issue_pv(0, w, t);
                if (t + 1 < w.tiles0) issue_qk(0, w, t + 1);
                if (t < w.tiles1) issue_pv(1, w, t);
                if (t + 1 < w.tiles1) issue_qk(1, w, t + 1);
            }
            // Every q.K of this work is issued: the next one's first may go before the other
            // tile's last P.V, as they need no slab but the two of V beside their own three.
            // No work past the next is looked at while this one's turn is held: the queue's
            // fourth turn waits for the release of its first.
            const int t = w.most - 1;
            if (t < w.tiles0) issue_pv(0, w, t);
            const Turn n = look(w.turn + 1, w.tile + w.most);
            if (n.tiles0 > 0) issue_qk(0, n, 0);
            if (t < w.tiles1) issue_pv(1, w, t);
            if (n.tiles1 > 0) issue_qk(1, n, 0);
            release(w.turn);
            w = n;
            if (w.most == 0) {  // without keys, and no turn held
                release(w.turn);
                w = keyed(w.turn + 1, w.tile);
                start(w);
            }
        }
        if (elect_one()) tc_commit(&bar[kPreDrain]);
        (void)mbar_wait(&bar[kPreDrain], 0);
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax / epilogue
        const int x = (warp - 2) >> 2;
        const int quad = warp & 3, r = quad * 32 + lane;  // TMEM lane = row of the tile
        const uint32_t s_at = tmem + ((uint32_t)(quad * 32) << 16) + kPreColS + 128 * x;
        const uint32_t o_at = tmem + ((uint32_t)(quad * 32) << 16) + kPreColO + 128 * x;
        // f16 weights as 2^7 of themselves: at most 2^15 with the lag of the maximum, and
        // normal down to 2^-21 of the largest
        constexpr float kLift = BF16 ? 0.f : 7.f;
        const float sc = p.scale_log2;
        int steps = 0, works = 0, tile = 0;
        for (int turn = 0; ok; ++turn) {
            ok = __all_sync(kFullMask, mbar_wait_or(work_full(turn), (turn / kPreQueue) & 1, abort_flag));
            if (!ok) break;
            const PreWork w = read_work(turn);
            if (w.n_q < 0) break;
            const int tiles0 = prefill_tiles(w, 0, p.causal), tiles1 = prefill_tiles(w, 1, p.causal);
            const int tiles = x ? tiles1 : tiles0;
            const int row = w.first + x * kPreRows + r;  // query in the sequence
            // keys below the limit are met; all of the warp's rows meet those below `clear`,
            // none those from `reach` on
            const int limit = p.causal ? min(w.n_k - w.n_q + 1 + row, w.n_k) : w.n_k;
            const int clear = __shfl_sync(kFullMask, limit, 0), reach = __shfl_sync(kFullMask, limit, 31);
            float m_run = -INFINITY, l_run = 0.f;
            for (int t = 0; t < tiles; ++t, ++steps) {
                ok = __all_sync(kFullMask, mbar_wait_or(&bar[kPreSFull + x], steps & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                float s[kPreKeys];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, s + 32 * c);
                const int here = (w.from + t) * kPreKeys;
                if (here + kPreKeys > clear) {
                    const float none = sc > 0.f ? -INFINITY : INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (here + 32 * c + 32 > clear) {
#pragma unroll
                            for (int j = 32 * c; j < 32 * c + 32; ++j)  // NaN-safe select
                                s[j] = here + j < limit ? s[j] : none;
                        }
                }
                const float mx = (sc > 0.f ? top128<true>(s) : top128<false>(s)) * sc;
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
                const float2 sc2 = make_float2(sc, sc), from2 = make_float2(-from, -from);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float o[16];
                    if (here + 32 * c < reach) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int k = 32 * c + 2 * j;
                            const float2 y = __ffma2_rn(make_float2(s[k], s[k + 1]), sc2, from2);
                            const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                            sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                            o[j] = __uint_as_float(narrow2<BF16>(e.x, e.y));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = 0.f;
                    }
                    tmem_store16(s_at + 16 * c, o);
                }
                l_run += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
                if (here + kPreKeys > w.n_k && (x == 0 || t >= tiles0)) {
                    // rows past the sequence's keys: P is 0 there, and V must be finite.  Tile
                    // B's product follows A's, so the first tile to reach them clears them.
                    const int group = 2 * (tile + t) + 1;
                    if (!mbar_wait_or(&bar[kPreFull + group % kPreGroups], (group / kPreGroups) & 1, abort_flag))
                        *abort_flag = 1;  // the next wait for S ends all
                    for (int i = 0; i < 2; ++i) {
                        const int slot = (5 * (tile + t) + 3 + i) % kPreSlots;
                        uint4 *z = reinterpret_cast<uint4 *>(smem + kPreOffRing + slot * kPreSlab);
                        for (int k = (w.n_k - here) * 8 + r; k < kPreKeys * 8; k += 128)
                            z[k] = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kPrePReady + x]);
            }
            if (ok && tiles > 0)
                ok = __all_sync(kFullMask, mbar_wait_or(&bar[kPreODone + x], works & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            if constexpr (SPLIT) {  // one piece of work, joined below
                m_of = m_run;
                l_of = l_run;
                break;
            }
            const float inv = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : l_run;
            uint16_t *to = p.out + ((int64_t)(w.q0 + row) * p.num_heads + w.head) * kPreValue;
            // O into registers first: the next work's products may take its place
            uint32_t y[kPreValue / 2];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float o[32];
                tmem_ld32(o_at + 32 * c, o);  // (nothing of use where no key was met)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[16 * c + i] = l_run == 0.f ? 0u : narrow2<BF16>(o[2 * i] * inv, o[2 * i + 1] * inv);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (tiles > 0) mbar_arrive(&bar[kPreOFree + x]);
                mbar_arrive(work_free(turn));
            }
            if (row < w.n_q) {
#pragma unroll
                for (int c = 0; c < 8; ++c) store32(to + 16 * c, y + 8 * c, p.wide);
            }
            works += tiles > 0;
            tile += max(tiles0, tiles1);
        }
    }
    if (!ok) *abort_flag = 1;
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_error(p.err, PA_ERR_DEVICE_TIMEOUT);
    if constexpr (SPLIT) {
        tc_fence_after();
        const PreWork w = read_work(0);
        if (w.n_q >= 0)  // the same for the cluster
            prefill_join<BF16>(p, w, smem, tmem, warp, lane, m_of, l_of);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Clusters of c CTAs that the current device holds at once (0 if the query fails),
// kept by device, size and type.
static int prefill_clusters(bool bf16, int c) {
    static std::atomic<int> known[128][kPreMaxSplit + 1][2];  // one more than the number, or 0
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
    std::atomic<int> &slot = known[dev][c][bf16];
    if (const int n = slot.load()) return n - 1;
    const void *kern = bf16 ? reinterpret_cast<const void *>(prefill_latent_kernel<true, true>)
                            : reinterpret_cast<const void *>(prefill_latent_kernel<false, true>);
    if (!ensure_smem_attr(kern, kPreSmem)) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(kPreThreads);
    cfg.dynamicSmemBytes = kPreSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
    slot.store(n + 1);
    return n;
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
        num_heads > 1024 || num_seqs > 65535 || total_k > kPreMaxKeys || !std::isfinite(scale) ||
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
    if (max_q_len > total_q) max_q_len = total_q;  // no sequence has more
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
    p.num_seqs = num_seqs;
    p.causal = causal != 0;
    p.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    p.scale_log2 = latent_scale(scale);
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
    const int64_t tiles = ((int64_t)max_q_len + 2 * kPreRows - 1) / (2 * kPreRows);
    const int64_t works = tiles * num_heads * num_seqs;  // pieces of work at most
    // few pieces of work with many keys each: clusters that share the keys of one
    const int64_t key_tiles = ((int64_t)total_k / num_seqs + kPreKeys - 1) / kPreKeys;
    p.split = 1;
    for (int c = kPreMaxSplit; c > 1 && p.split == 1; c /= 2)
        if (key_tiles >= c * kPreSplitTiles && works <= sm_count() / c && works <= prefill_clusters(bf16, c))
            p.split = c;
    if (p.split == 1 && 5 * works <= 6 * sm_count() && key_tiles >= kPreSplitLong) p.split = 2;
    p.by_length = p.split == 1 && (int64_t)total_k * num_heads <= kPreByLength;
    dim3 grid = p.by_length ? dim3((unsigned)num_heads, (unsigned)num_seqs, (unsigned)tiles)
                            : dim3((unsigned)(tiles * p.split), (unsigned)num_heads, (unsigned)num_seqs);
    // Sequences one behind the other have a piece of work of a head for each that has a
    // query, and one for every 256 queries beside those.
    const int64_t some = num_seqs < total_q ? num_seqs : total_q;
    const int64_t count = (some + (total_q - some) / (2 * kPreRows)) * num_heads;
    if (p.split == 1 && (works > kPreSparse * count || works > kPreBlocks || (p.by_length && tiles > 65535))) {
        const int64_t most = works < count ? works : count;
        p.per = (int)((most + kPreBlocks - 1) / kPreBlocks);
        grid = dim3((unsigned)((most + p.per - 1) / p.per));
    }
    auto kern = p.split > 1 ? (bf16 ? prefill_latent_kernel<true, true> : prefill_latent_kernel<false, true>)
                            : (bf16 ? prefill_latent_kernel<true, false> : prefill_latent_kernel<false, false>);
    if (!ensure_smem_attr(reinterpret_cast<const void *>(kern), kPreSmem)) return PA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kPreThreads);
    cfg.dynamicSmemBytes = kPreSmem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, p, map_q, map_k, map_v, map_pe) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
