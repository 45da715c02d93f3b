// Decode attention over 4-bit pools (pa_decode_int4).
//
// For a KV head with G <= 8 query heads, position p's key is m_p + s_p n_p
// with codes n in 0 .. 15, so
//   q . k_p = s_p (q . n_p) + m_p sum(q)
//   out     = sum_p (P_p s'_p) n'_p + sum_p P_p m'_p
// and only the products with the codes touch every element: they go to the
// matrix unit (mma.sync m16n8k16, f16 operands, fp32 sums), scales and minima
// are applied to the 16 x 8 score tile and to the weights.
//
// Codes become f16 operands by masking alone.  A half with the bits 0x000n is
// the subnormal n 2^-24, exactly, and 0x00n0 is 16 n 2^-24; so of a word w of
// eight codes, w & 0x000f000f, w & 0x00f000f0 and the same of w >> 8 are four
// operand pairs (elements e and e + 4): five instructions for eight elements,
// nothing stored.  The factor 16 is taken out of q (keys) or of the finished
// sums (values), the factor 2^-24 likewise.  Keys: rows of the A operand are
// positions, q is B (8 columns: the heads).  Values: A's rows are dimensions,
// its columns positions, so two positions' words are interleaved by halves
// (two byte permutes for 16 codes) before the same masks; B is the weights,
// which the transposing register exchange movmatrix brings from the score
// tile's layout.  The weights P s' are split into two f16 terms (22 bits).  f16's
// grid ends at 2^-24, so a power of two that each warp keeps for each head, like
// the running maximum, brings the largest product P s' to 2^6 .. 2^15: the grid is
// then 2^-30 of it or finer.  (It goes by the products and not by the scales s'
// alone, and falls when the maximum moves: a row of large values that has no weight
// must not push the others onto the grid.)  The matrix
// unit cuts sums off instead of rounding them, and sums of codes would all be of
// one sign: every other 16 positions enter as -P s' times 15 - n (a mask with an
// exclusive or), which leaves 15 s' for their minimum to take over and keeps the
// sums about zero.  (Without it a mean over 120,000 positions in one warp's sum
// was off by 9e-2 of itself; with it by 2.0e-4, which is f16's own rounding.)  What
// is left of the cut-off sums is about 2^-21 of the largest |v|, several times an fp32
// sum's error and a fortieth of half a step of a bf16 output of 20,000 positions: 1.2%
// of the outputs round to the other side than the exact value, 0.2% of an fp32 sum's.
//
// Why not tcgen05: its operands come from shared or tensor memory, where codes
// would have to be stored again as 8- or 16-bit values, two to four times the
// bytes that were read, and its smallest tile is 64 rows of a CTA-wide
// pipeline; with 8 columns 16 positions cost a warp 24 MMAs here (16 with up to
// four heads), and the masks feed them from the registers the loads filled.
//
// Bounds: 136 bytes a position and KV head (D = 128).  256 sequences of 32 + 8
// heads and 513 to 8192 positions: 219 us, 5.6 TB/s, 83% of the copy rate; 16 of
// 64 + 8 heads and 16,385 to 32,768: 94 to 97 us, 66%; one of 200,003: 47 us, 68%.
// The first without its arithmetic takes 191 us.  No pipe is full (ALU 53%, issue 51%,
// matrix unit 25% of cycles; eight heads: 49, 49 and 36%), but neither fewer
// instructions (12 of 240 for 16 positions: 1%) nor more warps (five or six CTAs an
// SM with the queries in shared memory: 12 to 39% slower) nor the next keys'
// products beside this step's values (4 to 7% slower) bring them together better.
// Taking the weights' scale from the products, which are held across the check,
// costs nothing against one taken from the scales (218 us for 219; the variants of
// five to eight heads of 128 spill 24 bytes by it, 94.6 us for 94.0);
// products formed anew after the check 224, a check of their own 224.
//
// A warp works alone: every fourth 32 positions of the CTA's piece, its own
// ring of stages filled by bulk copies of whole records, its own running
// maximum and sums; the four warps merge at the end through shared memory.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "pa_decode.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

// The parameters the decodes share (the pools are those of the records; the
// counters, flags and the fused write are not used), and:
struct Int4Params : DecodeParams {
    int balanced;  // balanced ranges: groups of CTAs in the first wave (0: chunks)
    int bundle;    // heads of a group
};

constexpr int kInt4Warps = 4;
constexpr int kInt4MaxG = 8;
constexpr int kInt4Step = 32;  // positions a warp takes at a time: two score tiles
// A column's factor fe = 2^(7 - ve) keeps its products P s' fe below this (f16 ends at
// 65504), ve at least kInt4LeastExponent (fe in fp32).
constexpr float kInt4Product = 32768.f;
constexpr int kInt4LeastExponent = -119;

template <int D>
struct Int4Shape {
    static constexpr int HALF = kInt4Step * (D / 2 + 4);  // a step's K (or V) records
    static constexpr int STAGE = 2 * HALF;
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int RING = STAGES * STAGE;           // a warp's
    static constexpr int BARS = kInt4Warps * RING;        // offset of the mbarriers
    static constexpr int SMEM_BYTES = BARS + kInt4Warps * STAGES * 8;
    static_assert(kInt4Warps * kInt4MaxG * (D + 2) * 4 <= BARS, "the merge reuses the rings");
};

// D += A B: A 16 x 16 f16 (row-major fragments), B 16 x 8 f16, D 16 x 8 fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8 x 8 matrix of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ve of a factor 2^(7 - ve).
__device__ __forceinline__ int int4_weight_exponent(float fe) {
    return 7 + 127 - (int)(__float_as_uint(fe) >> 23);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) { return narrow2<false>(a, b); }

// Balanced ranges (automatic partitions).  The heads go in bundles of up to 8:
// as many consecutive CTAs, a group, take the same positions of a bundle's heads
// at about the same time, so that the records of a block, which lie together, are
// read together (a small gain: 93.8 -> 93.3 us for 16 long sequences).  The work is
// one line of units of 128 positions, sequence by sequence and bundle by bundle;
// group c takes the units from bound(c) to bound(c + 1), moved to the next head's
// border where that is at most `slack` units away, so that no head is cut for a
// sliver.  Every CTA works the line out from the lengths (one load and a scan),
// whatever they are.  A first wave of groups takes equal large shares; a second,
// of smaller shares, is started as the first ends, which the SMs do not do
// together (equal shares in one wave alone ended between 138 and 222 us).  The
// partials of heads that bounds cut are merged by a second kernel.

// A group's range: units [unit, end) of the line.  Its next unit is unit `at`
// of the n units of bundle `bundle` of sequence seq.
struct Int4Range {
    int wave;          // groups of the first wave
    int share, small;  // units of a share in the first wave, in the second
    int slack;
    int unit, end;
    int seq, bundle, at, n;
};

// A piece of work: `count` positions of a head from `start` on (-1: none
// left), its partial's slot and the head's number of partials.
struct Int4Piece {
    int seq, kvh, start, count;
    int slot, nparts;
};

constexpr int kInt4Unit = kInt4Step * kInt4Warps;  // positions
// Longest heads that one CTA each takes whole, of few and of many (sequence, KV
// head) pairs.  Single pass against balanced ranges in us, of lengths that are all
// the longest / spread from half of it on / log-normal about a tenth of it (x 2: 14
// query heads of 64, x 8: 32 of 128, f16; 1024 heads and more than that stay faster
// in one pass further on, to 4096 for even lengths):
//            longest 1024                    2048                      2304
//    8 x 2   9 9 / 9 10 / 9 11       14 10 / 14 11 / 14 13     15 11 / 15 11 / 15 11
//    8 x 8   10 10 / 10 12 / 10 13   16 13 / 16 13 / 16 15     18 14 / 17 14 / 17 13
//   16 x 8   10 12 / 10 14 / 10 15   16 17 / 16 16 / 16 16     18 20 / 17 16 / 17 15
//   64 x 2   9 11 / 9 13 / 9 16      14 14 / 14 14 / 14 15     16 16 / 16 15 / 16 14
//  128 x 2   12 14 / 12 14 / 10 16   18 20 / 17 18 / 15 16     20 22 / 19 18 / 17 15
//   64 x 8   21 27 / 19 25 / 12 19   35 39 / 32 34 / 19 19     38 42 / 35 37 / 22 19
//  128 x 8   37 40 / 35 36 / 19 22   60 65 / 54 55 / 28 29     65 71 / 61 59 / 33 28
//  256 x 8   60 72 / 52 61 / 25 34   103 122 / 86 98 / 38 43   114 132 / 95 106 / 40 44
constexpr int kInt4SinglePass = 1024, kInt4SinglePassMany = 2048;
constexpr int kInt4ManyHeads = 128;
constexpr int kInt4MinShare = 4;                   // units: smaller shares cost more than they save
constexpr int kInt4MinSlack = 2;
// A second wave pays where its shares are still long next to a CTA's start (2 us
// to its first copies): 256 sequences (115 units a slot) 236 -> 216 us with it,
// 16 long ones (40 units) 94 -> 98.
constexpr int kInt4SecondWave = 64;  // units a slot from which on there is one,
constexpr int kInt4SecondPart = 5;   //   with a fifth of the work,
constexpr int kInt4SecondCtas = 2;   //   in twice as many groups
constexpr int kInt4BalancedSeqs = 1024;  // sequences

__device__ __forceinline__ int int4_units(const Int4Params &p, int seq) {
    return (item_len(p, seq, false) + kInt4Unit - 1) / kInt4Unit;
}

// The last bound at or before unit u of the line.
__device__ __forceinline__ int int4_bound_before(const Int4Range &r, int u) {
    const int large = r.wave * r.share;
    return u < large ? u / r.share : r.wave + (u - large) / r.small;
}

// Pieces that bounds cut the heads of the range's present bundle into, and the first bound
// inside it: those past its first slack units and before its last.
__device__ __forceinline__ int int4_parts(const Int4Range &r, int *first) {
    const int a = r.unit - r.at, b = a + r.n;  // the bundle on the line
    *first = int4_bound_before(r, a + r.slack) + 1;
    const int last = b <= r.slack ? -1 : int4_bound_before(r, b - r.slack - 1);
    return max(last - *first + 1, 0) + 1;
}

// The range of group `group` of ngroups, or (group < 0) the place of the index-th
// bundle of the batch, with n = 0 for one without positions.  Called by all T
// threads of the block; ends synchronised.
template <int T>
__device__ __forceinline__ void int4_plan(const Int4Params &p, int ngroups, int group, int index,
                                          Int4Range *range) {
    const int wave = p.balanced;
    __shared__ int sums[T / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int per = (p.num_seqs + T - 1) / T;
    const int s0 = min(tid * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
    int mine = 0;
    for (int s = s0; s < s1; ++s) mine += int4_units(p, s);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sums[tid >> 5] = incl;
    __syncthreads();
    int before = incl - mine, all = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
        if (w < (tid >> 5)) before += sums[w];
        all += sums[w];
    }
    const int H = p.num_kv_heads / p.bundle, total = all * H;
    // the second wave gets a part of the work if its shares are worth their CTAs
    int share = max((total + wave - 1) / wave, kInt4MinShare), small = share;
    if (ngroups > wave && share >= kInt4SecondWave) {
        share -= share / kInt4SecondPart;
        small = max((total - wave * share + ngroups - wave - 1) / (ngroups - wave), kInt4MinShare);
    }
    const int slack = max(small / 8, kInt4MinSlack);
    if (group < 0) {
        const int seq = index / H;
        if (seq >= s0 && seq < s1) {
            int base = before;
            for (int s = s0; s < seq; ++s) base += int4_units(p, s);
            range->seq = seq;
            range->bundle = index - seq * H;
            range->at = 0;
            range->n = int4_units(p, seq);
            range->unit = base * H + range->bundle * range->n;
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int c = group + b;
            const int u = min(c < wave ? c * share : wave * share + (c - wave) * small, total);
            if (u == total) {
                if (tid == 0) {
                    if (b == 0) range->unit = total;
                    range->end = total;
                }
            } else if (u >= before * H && u < (before + mine) * H) {  // in this thread's sequences
                int base = before * H, seq = s0, n = int4_units(p, s0);
                while (u >= base + n * H) {
                    base += n * H;
                    n = int4_units(p, ++seq);
                }
                const int bundle = (u - base) / n;
                int at = u - base - bundle * n;
                if (at <= slack)
                    at = 0;
                else if (n - at <= slack)
                    at = n;
                if (b == 0) {
                    range->seq = seq;
                    range->bundle = bundle;
                    range->at = at;
                    range->n = n;
                    range->unit = base + bundle * n + at;
                } else {
                    range->end = base + bundle * n + at;
                }
            }
        }
    }
    if (tid == 0) {
        range->wave = wave;
        range->share = share;
        range->small = small;
        range->slack = slack;
    }
    __syncthreads();
}

// The next piece of the range (one thread).
__device__ __forceinline__ void int4_next_piece(const Int4Params &p, Int4Range *range,
                                             Int4Piece *piece) {
    Int4Range &r = *range;
    if (r.unit >= r.end) {
        piece->count = -1;
        return;
    }
    if (r.at == r.n) {  // the next bundle with anything in it
        r.at = 0;
        if (++r.bundle == p.num_kv_heads / p.bundle) {
            r.bundle = 0;
            do r.n = int4_units(p, ++r.seq);
            while (r.n == 0);
        }
    }
    const int units = min(r.n - r.at, r.end - r.unit);
    piece->seq = r.seq;
    piece->kvh = r.bundle * p.bundle + (int)blockIdx.x % p.bundle;
    piece->start = r.at * kInt4Unit;
    piece->count = min(item_len(p, r.seq, false), (r.at + units) * kInt4Unit) - piece->start;
    piece->slot = 2 * (int)blockIdx.x + (r.at == 0 ? 1 : 0);
    int first;
    piece->nparts = int4_parts(r, &first);
    r.unit += units;
    r.at += units;
}

// Partials, m, l [slot][8] and O [slot][G][D].  Balanced ranges: a CTA leaves at
// most two, of the head its range starts inside of (slot 2 blockIdx.x) and of the
// one it ends inside of, if that one starts in it (the slot after).  Chunks: chunk
// c of a head has slot head * num_partitions + c.
//
// The merge: out = sum_k w_k O_k / sum_k w_k, w_k = l_k 2^(m_k - max m), over the
// n partials of every head that was cut.  Few heads (kMergeHeads, many partials
// each): a block a query head, its threads four dimensions each of every
// SLICES-th partial.  Many heads: a block a bound and head of the bundle
// (kMergeBounds; at work if that bound is the first inside the head) or a block a
// head (kMergeChunks), its threads four dimensions each of all partials of one or
// two query heads.  A thread has eight partials' loads in flight and keeps its own
// running maximum, so nothing waits for the maxima first.
enum Int4MergeKind { kMergeHeads, kMergeBounds, kMergeChunks };
__host__ __device__ constexpr int int4_merge_threads(Int4MergeKind kind) {
    return kind == kMergeHeads ? 512 : 128;
}

template <bool BF16, int D, Int4MergeKind KIND>
__global__ void __launch_bounds__(int4_merge_threads(KIND))
    int4_merge_kernel(const Int4Params p, int ngroups) {
    constexpr bool HEADS = KIND == kMergeHeads;
    constexpr int T = int4_merge_threads(KIND);
    constexpr int ITEMS = D / 4, ROWS = T / ITEMS, SLICES = HEADS ? ROWS : 1;
    __shared__ Int4Range range;
    __shared__ float4 sums[HEADS ? T : 1];
    __shared__ float tops[ROWS], totals[ROWS];
    const int item = threadIdx.x % ITEMS, row = threadIdx.x / ITEMS;
    // the first partial's slot and those from one to the next of the rest, the
    // number of partials, and the head
    int64_t slot0 = 0, slot1 = 0;
    int stride1 = 1, n = 0, seq, kvh;
    if constexpr (KIND == kMergeChunks) {
        pdl_wait();
        seq = blockIdx.x / p.num_kv_heads;
        kvh = blockIdx.x % p.num_kv_heads;
        const int L = item_len(p, seq, false);
        n = L == 0 ? 0 : (L - 1) / p.partition_tokens + 1;
        slot0 = (int64_t)blockIdx.x * p.num_partitions;
        slot1 = slot0 + 1;
        if (n <= 1) return;  // written by the decode itself
    } else {
        // the decode kernel began after all work before it was done, so the
        // lengths are there
        const int in_bundle = (int)blockIdx.x % p.bundle, index = (int)blockIdx.x / p.bundle;
        int4_plan<T>(p, ngroups, HEADS ? -1 : index + 1, index, &range);
        int first = 0;
        const bool mine = (HEADS ? range.n > 0 : range.unit < range.end && range.at > 0 &&
                                                     range.at < range.n) &&
                          (n = int4_parts(range, &first)) > 1 && (HEADS || first == index + 1);
        pdl_wait();
        if (!mine) return;
        slot0 = 2 * ((int64_t)(first - 1) * p.bundle + in_bundle) + 1;
        stride1 = 2 * p.bundle;
        slot1 = slot0 - 1 + stride1;
        seq = range.seq;
        kvh = range.bundle * p.bundle + in_bundle;
    }
    auto slot = [&](int k) { return k == 0 ? slot0 : slot1 + (int64_t)(k - 1) * stride1; };
    for (int g = HEADS ? blockIdx.y : row; g < p.group; g += ROWS) {
        const float4 *rows = reinterpret_cast<const float4 *>(p.part_o) + g * ITEMS + item;
        const int64_t stride = (int64_t)p.group * ITEMS;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f, M = -INFINITY;
        for (int k0 = HEADS ? row : 0; k0 < n; k0 += 8 * SLICES) {
            float4 v[8];
            float m[8], l[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t s = slot(min(k0 + j * SLICES, n - 1));
                v[j] = __ldcg(rows + s * stride);
                m[j] = __ldcg(p.part_m + s * kInt4MaxG + g);
                l[j] = __ldcg(p.part_l + s * kInt4MaxG + g);
            }
            float top = M;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, m[j]);
            const float f = fast_exp2(M - top);
            M = top;
            total *= f;
            o.x *= f;
            o.y *= f;
            o.z *= f;
            o.w *= f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (k0 + j * SLICES >= n) break;
                const float w = l[j] * fast_exp2(m[j] - M);
                total += w;
                o.x += w * v[j].x;
                o.y += w * v[j].y;
                o.z += w * v[j].z;
                o.w += w * v[j].w;
            }
        }
        if constexpr (HEADS) {
            sums[threadIdx.x] = o;
            if (item == 0) {
                tops[row] = M;
                totals[row] = total;
            }
            __syncthreads();
            if (row > 0) return;
            float top = M;
#pragma unroll
            for (int s = 1; s < SLICES; ++s) top = fmaxf(top, tops[s]);
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            total = 0.f;
#pragma unroll
            for (int s = 0; s < SLICES; ++s) {
                const float f = fast_exp2(tops[s] - top);  // a slice without partials: 0
                const float4 v = sums[s * ITEMS + item];
                total += f * totals[s];
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
            }
        }
        const float f = 1.f / total;
        uint16_t *out = static_cast<uint16_t *>(p.out) +
                        ((int64_t)seq * p.num_q_heads + kvh * p.group + g) * D;
        reinterpret_cast<uint2 *>(out)[item] =
            make_uint2(narrow2<BF16>(o.x * f, o.y * f), narrow2<BF16>(o.z * f, o.w * f));
        if constexpr (HEADS) return;
    }
}

template <bool BF16, int D, int B, bool H4>
__global__ void __launch_bounds__(32 * kInt4Warps, 4) decode_int4_kernel(
    const __grid_constant__ Int4Params p) {
    using S = Int4Shape<D>;
    constexpr int KW = D / 32;  // words of a key row a lane holds (8 codes each)
    constexpr int VW = D / 64;  // words of a value row a lane holds
    extern __shared__ __align__(16) uint8_t smem[];
    if (threadIdx.x % 32 == 0) {
        for (int i = 0; i < S::STAGES; ++i)
            mbar_init(reinterpret_cast<uint64_t *>(smem + S::BARS) + threadIdx.x / 32 * S::STAGES + i, 1);
        mbar_init_fence();
    }
    __syncwarp();
    pdl_wait();
    int stage = 0;        // of the warp's next step
    uint32_t parity = 0;
    bool arrived = true;

    // The CTA's pieces of work: one chunk of one head (partition_tokens given),
    // or every piece of its balanced range.  What only the ends of a piece need
    // waits in shared memory.
    __shared__ Int4Range range;
    __shared__ Int4Piece piece;
    if (p.balanced) {
        pdl_trigger();  // the merge kernel may work out its plan
        int4_plan<32 * kInt4Warps>(p, gridDim.x / p.bundle, blockIdx.x / p.bundle, 0, &range);
    } else {
        int chunk, kvh, seq;
        if (p.compact) {
            if (!compact_item(p, blockIdx.x, &seq, &chunk, &kvh)) return;
        } else {
            chunk = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
        }
        if (threadIdx.x == 0) {
            const int P = p.partition_tokens;
            const int L = item_len(p, seq, chunk == 0 && kvh == 0);
            piece.seq = seq;
            piece.kvh = kvh;
            piece.start = chunk * P;
            const int left = L - chunk * P;
            piece.count = left > 0 ? min(left, P) : L == 0 && chunk == 0 ? 0 : -1;
            piece.nparts = L == 0 ? 1 : (L - 1) / P + 1;
        }
        __syncthreads();
        if (piece.count < 0) return;
    }
    for (;;) {
    if (p.balanced) {
        if (threadIdx.x == 0) int4_next_piece(p, &range, &piece);
        __syncthreads();
        if (piece.count < 0) break;
    }
    // Taken anew for every piece, so that what follows from them is not kept in
    // registers from one piece to the next.
    int tid = threadIdx.x;
    asm volatile("" : "+r"(tid));
    const int warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, t = lane & 3;  // fragment row (or column) and quad lane
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::BARS) + warp * S::STAGES;
    const int G = p.group;
    const int seq = piece.seq, kvh = piece.kvh, start = piece.start, count = piece.count;
    if (count == 0) {  // a sequence without tokens (chunk 0 of it)
        uint16_t *out = static_cast<uint16_t *>(p.out) + ((int64_t)seq * p.num_q_heads + kvh * G) * D;
        for (int i = threadIdx.x; i < G * D; i += blockDim.x) out[i] = 0;
        return;
    }
    const int nsteps = (count + kInt4Step - 1) / kInt4Step;
    const int my_steps = (nsteps - warp + kInt4Warps - 1) / kInt4Warps;

    // -------------------------------------------------------------- loads
    // A step is one or two whole records of K and as many of V, each a bulk
    // copy issued by a lane of its own; lane 2 e + (0 K, 1 V) takes block e.
    constexpr int E = kInt4Step / B;  // blocks of a step
    constexpr int REC = int4_record_bytes<D>(B);
    uint8_t *ring = smem + warp * S::RING;
    const uint32_t block_stride = (uint32_t)p.num_kv_heads * REC;
    const uint8_t *mine = reinterpret_cast<const uint8_t *>(lane & 1 ? p.v_pool : p.k_pool) +
                          (int64_t)kvh * REC;
    const uint32_t to = (lane & 1) * S::HALF + (lane >> 1) * REC;
    const int32_t *table = seq_table(p, seq) + start / B;
    // block ids of this warp's steps, a lane each, 32 at a time; -1 past the end
    auto window = [&](int w) -> int {
        const int i = 32 * w + lane;
        const int b = (warp + kInt4Warps * (i / E)) * E + i % E;
        if (b >= (count + B - 1) / B) return -1;
        const int phys = table[b];
        if ((unsigned)phys < (unsigned)p.num_blocks) return phys;
        record_error(p.err, PA_ERR_BAD_INDEX);
        return 0;
    };
    int cur = window(0), nxt = 0;
    auto issue = [&](int k, int stage) {
        if (k >= my_steps) return;
        const int i = k * E;
        if ((i & 31) == 0) {
            if (i) cur = nxt;
            nxt = window((i >> 5) + 1);
        }
        const int phys = __shfl_sync(kFullMask, cur, (i + (lane >> 1)) & 31);
        // (every lane is past its reads of this stage: the ballot, and the
        // barrier before the copies)
        const bool copies = lane < 2 * E && phys >= 0;
        const int n = __popc(__ballot_sync(kFullMask, copies));
        if (lane == 0) mbar_arrive_expect_tx(&bars[stage], (uint32_t)(n * REC));
        __syncwarp();
        if (copies)
            bulk_copy_g2s(ring + stage * S::STAGE + to, mine + (uint64_t)(uint32_t)phys * block_stride,
                          REC, &bars[stage]);
    };
#pragma unroll
    for (int k = 0; k < S::STAGES - 1; ++k)
        issue(k, stage + k < S::STAGES ? stage + k : stage + k - S::STAGES);

    // ------------------------------------------------------------ queries
    // B fragments: column r is head r (H4, at most four heads: r mod 4), this
    // lane's elements are those of its key words.  2^kq brings the head's
    // largest |q| below 2^15; elements that meet codes in the high four bits
    // are divided by 16.  What takes scores back, 2^(24 - kq) scale, may pass
    // fp32's range while they do not (|q| of 2^100 and keys of 2^-100): a warp with
    // a head of such a size forms them, and keeps M, in units of 2^64 (full batch 218
    // -> 222 us, long and one long within 1%; a factor in every step the same).
    uint32_t qf[KW][4];
    float cs[2], qs[2];  // of the score tile's columns 2t, 2t + 1
    int careful;  // steps that take the branch below in any case: the first, or all
    {
        const int head = H4 ? r & 3 : r;
        float x[KW][8];
        float top = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (head < G)
                raw = *reinterpret_cast<const uint4 *>(
                    p.q + ((int64_t)seq * p.num_q_heads + kvh * G + head) * D + (t * KW + j) * 8);
            widen8<BF16>(raw, x[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                top = fmaxf(top, fabsf(x[j][i]));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        const int e = (int)(__float_as_uint(top) >> 23) - 127;  // top < 2^(e + 1)
        const int es = (int)(__float_as_uint(fabsf(p.scale_log2)) >> 23) - 127;
        const bool big = __any_sync(kFullMask, e + max(es, 0) > 80);
        careful = big ? INT_MAX : 1;
        const float unit = big ? 0x1p-64f : 1.f;
        const int kq = min(14 - e, 127);  // -113 .. 127
        const float even = pow2i(kq), odd = pow2i(kq - 4);
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(x[j][i], unit, sum);
        sum += __shfl_xor_sync(kFullMask, sum, 1);
        sum += __shfl_xor_sync(kFullMask, sum, 2);
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = i & 1 ? odd : even;
                qf[j][i] = half2_bits(x[j][i] * f, x[j][i + 4] * f);
            }
        const int back = 24 - kq, half = back >> 1;  // -103 .. 137, in two steps
        const float c = p.scale_log2 * unit * pow2i(half) * pow2i(back - half);
        const float s = sum * p.scale_log2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            cs[h] = __shfl_sync(kFullMask, c, 4 * (2 * t + h));
            qs[h] = __shfl_sync(kFullMask, s, 4 * (2 * t + h));
        }
    }

    // ---------------------------------------------------------- main loop
    // O[a][...]: of this lane's D/8 dimensions, 2a, and 2a + 1 16 times with 2a
    // added, columns 2t and 2t + 1, in units of 2^-24 / fe of the column.
    float O[4 * VW][4];
#pragma unroll
    for (int a = 0; a < 4 * VW; ++a) O[a][0] = O[a][1] = O[a][2] = O[a][3] = 0.f;
    // pm: sum of P times what the rows' codes are counted from
    float M[2] = {0.f, 0.f}, l[2] = {0.f, 0.f}, pm[2] = {0.f, 0.f};
    float fe[2] = {1.f, 1.f};  // the weights are P s' fe (the first step sets it)
    // Fragment row r is position pr of its half tile: pairs of rows (r, r + 1)
    // and rows of equal t differ in parity, so that neither the key loads (two
    // rows a quarter warp) nor the value loads (four rows a half warp) meet in
    // a bank more than they must.
    const int pr = r ^ ((r >> 1) & 1);
    constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u, kByte = 0x00ff00ffu;
    // offsets of position `pos` of a step in its half of a stage
    constexpr int U = B == 32 ? 16 * (D / 2) : REC;       // 16 positions on
    constexpr int PU = B == 32 ? 16 * 4 : REC;            // the same for the (s, m) pairs
    const int koff = pr * (D / 2) + t * (4 * KW);
    const int poff = B * (D / 2) + pr * 4;
    const int voff = S::HALF + (2 * t) * (D / 2) + r * (4 * VW);
    const int vx = (t & 1) * (D / 2);  // positions 2t, 2t + 1 change places where t is odd
#pragma unroll 1
    for (int k = 0; k < my_steps; ++k) {
        arrived = __all_sync(kFullMask, mbar_wait(&bars[stage], parity));
        if (!arrived) break;
        const uint8_t *tile = ring + stage * S::STAGE;
        issue(k + S::STAGES - 1, stage == 0 ? S::STAGES - 1 : stage - 1);
        if (++stage == S::STAGES) {
            stage = 0;
            parity ^= 1;
        }

        // scores less the running maximum, base 2: s[u] is (position pr, columns
        // 2t, 2t + 1), (position 8 + pr, the same) of the u-th 16 positions
        float s[2][4], sv[2][2], mv[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t w[2][KW];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *src = tile + koff + u * U + 8 * h * (D / 2);
                if constexpr (KW == 4) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(src);
                    w[h][0] = a.x; w[h][1] = a.y; w[h][2] = a.z; w[h][3] = a.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2 *>(src);
                    w[h][0] = a.x; w[h][1] = a.y;
                }
            }
            float c[4];
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const uint32_t a0 = w[0][j] & kLo, a1 = w[1][j] & kLo;
                const uint32_t a2 = w[0][j] & kHi, a3 = w[1][j] & kHi;
                if (j == 0)
                    mma_f16_zero(c, a0, a1, a2, a3, qf[j][0], qf[j][1]);
                else
                    mma_f16(c, a0, a1, a2, a3, qf[j][0], qf[j][1]);
                const uint32_t u0 = w[0][j] >> 8, u1 = w[1][j] >> 8;
                mma_f16(c, u0 & kLo, u1 & kLo, u0 & kHi, u1 & kHi, qf[j][2], qf[j][3]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *par = tile + poff + u * PU + 8 * h * 4;
                const uint32_t pk = *reinterpret_cast<const uint32_t *>(par);
                const uint32_t pv = *reinterpret_cast<const uint32_t *>(par + S::HALF);
                const float sk = from16<BF16>(pk & 0xffffu), mk = from16<BF16>(pk >> 16);
                sv[u][h] = from16<BF16>(pv & 0xffffu);
                mv[u][h] = from16<BF16>(pv >> 16);
                if (u == 1) mv[u][h] = fmaf(15.f, sv[u][h], mv[u][h]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    s[u][2 * h + i] = fmaf(c[2 * h + i], sk * cs[i], fmaf(mk, qs[i], -M[i]));
            }
        }
        const int left = count - (warp + kInt4Warps * k) * kInt4Step;
        if (left < kInt4Step) {  // slots past the end hold anything
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (16 * u + 8 * h + pr >= left) {
                        s[u][2 * h] = s[u][2 * h + 1] = -INFINITY;
                        sv[u][h] = mv[u][h] = 0.f;
                    }
        }

        // The weights P and their products with the scales of V.  The running
        // maximum moves only when a score passes it by more than kLazyRescale, a
        // column's fe only when a product passes kInt4Product (and both with the
        // first step).
        float P[2][4], x[2][4];
        float top = 0.f, mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                P[u][i] = fast_exp2(s[u][i]);
                x[u][i] = P[u][i] * (sv[u][i >> 1] * fe[i & 1]);
                top = fmaxf(top, fabsf(x[u][i]));
                mx = fmaxf(mx, s[u][i]);
            }
        if (__any_sync(kFullMask, mx > kLazyRescale || top > kInt4Product || k < careful)) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (careful > 1) {  // scores in units of 2^64
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        s[u][i] *= 0x1p64f;
                        s[u][2 + i] *= 0x1p64f;
                    }
                }
                float up = fmaxf(fmaxf(s[0][i], s[0][2 + i]), fmaxf(s[1][i], s[1][2 + i]));
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) up = fmaxf(up, __shfl_xor_sync(kFullMask, up, o));
                if (k > 0) up = fmaxf(up, 0.f);
                M[i] = fmaf(up, careful > 1 ? 0x1p-64f : 1.f, M[i]);
                f[i] = k == 0 ? 0.f : fast_exp2(-up);  // nothing summed yet
                l[i] *= f[i];
                pm[i] *= f[i];
                // the column's largest product now, below 2^e
                float most = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[u][2 * h + i] -= up;
                        P[u][2 * h + i] = fast_exp2(s[u][2 * h + i]);
                        x[u][2 * h + i] = P[u][2 * h + i] * sv[u][h];
                        most = fmaxf(most, fabsf(x[u][2 * h + i]));
                    }
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1)
                    most = fmaxf(most, __shfl_xor_sync(kFullMask, most, o));
                int e = (int)(__float_as_uint(most) >> 23) - 126;
                // that of the sums so far, which have shrunk by 2^up: below 2^(ve - up)
                const int ve = int4_weight_exponent(fe[i]);
                if (k > 0) e = max(e, ve - (int)fminf(up, 512.f));
                e = min(max(e, kInt4LeastExponent), 127);
                f[i] *= pow2i(max(min(ve - e, 126), -126));
                fe[i] = pow2i(7 - e);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    x[u][i] *= fe[i];
                    x[u][2 + i] *= fe[i];
                }
            }
#pragma unroll
            for (int a = 0; a < 4 * VW; ++a) {
                O[a][0] *= f[0];
                O[a][1] *= f[1];
                O[a][2] *= f[0];
                O[a][3] *= f[1];
            }
        }

#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // the weights' sums, and the two f16 terms of P s' fe, transposed
            // to B fragments (rows: positions, columns: heads; H4: the second
            // terms of heads 0 .. 3 are columns 4 .. 7)
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = P[u][2 * h], p1 = P[u][2 * h + 1];
                l[0] += p0;
                l[1] += p1;
                pm[0] = fmaf(p0, mv[u][h], pm[0]);
                pm[1] = fmaf(p1, mv[u][h], pm[1]);
                const float x0 = u == 0 ? x[u][2 * h] : -x[u][2 * h];
                const float x1 = u == 0 ? x[u][2 * h + 1] : -x[u][2 * h + 1];
                const uint32_t hi = half2_bits(x0, x1);
                const float2 y = widen2<false>(hi);
                const uint32_t lo = half2_bits(x0 - y.x, x1 - y.y);
                if constexpr (H4) {
                    bh[h] = transpose8(t < 2 ? hi : lo);
                } else {
                    bh[h] = transpose8(hi);
                    bl[h] = transpose8(lo);
                }
            }

            // O += V^T (P s')
            uint32_t v[4][VW];  // of B fragment rows 2t, 2t + 1, 8 + 2t, 9 + 2t
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *src = tile + voff + u * U + 8 * (i >> 1) * (D / 2) +
                                     (i & 1 ? D / 2 - vx : vx);
                if constexpr (VW == 2) {
                    const uint2 a = *reinterpret_cast<const uint2 *>(src);
                    v[i][0] = a.x;
                    v[i][1] = a.y;
                } else {
                    v[i][0] = *reinterpret_cast<const uint32_t *>(src);
                }
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // codes 0 .. 3 and 4 .. 7 of the words
                    const uint32_t sel = half ? 0x7632u : 0x5410u;
                    const uint32_t x = __byte_perm(v[0][j], v[1][j], sel);
                    const uint32_t y = __byte_perm(v[2][j], v[3][j], sel);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        // a whole byte, 16 n(odd) + n(even), and its low half; of
                        // the second 16 positions both from 255 and 15 down
                        const uint32_t nb = u == 0 ? 0u : kByte, nl = u == 0 ? 0u : kLo;
                        const uint32_t xb = q ? __byte_perm(x, 0u, 0x4341) ^ nb : (x & kByte) ^ nb;
                        const uint32_t yb = q ? __byte_perm(y, 0u, 0x4341) ^ nb : (y & kByte) ^ nb;
                        const uint32_t xl = q ? xb & kLo : (x & kLo) ^ nl;
                        const uint32_t yl = q ? yb & kLo : (y & kLo) ^ nl;
                        float(&acc)[4] = O[4 * j + 2 * half + q];
                        mma_f16(acc, xl, xb, yl, yb, bh[0], bh[1]);
                        if constexpr (!H4) mma_f16(acc, xl, xb, yl, yb, bl[0], bl[1]);
                    }
                }
            }
        }
    }

    // -------------------------------------------------------------- merge
    if (!arrived && lane == 0) {
        // A bounded wait ran out: let copies still in flight land (bounded
        // again) before the shared memory goes; the output is then unspecified.
        // There is no further piece: its waits would run out one after the other.
        record_error(p.err, PA_ERR_DEVICE_TIMEOUT);
        range.end = 0;
        for (int i = 0; i < S::STAGES; ++i) (void)mbar_wait(&bars[i], i >= stage ? parity : parity ^ 1);
    }
    __syncwarp();
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFullMask, l[h], o);
            pm[h] += __shfl_xor_sync(kFullMask, pm[h], o);
        }
    if constexpr (H4) {  // the two terms' sums
#pragma unroll
        for (int a = 0; a < 4 * VW; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) O[a][i] += __shfl_xor_sync(kFullMask, O[a][i], 2);
    }
    __syncthreads();  // the rings are done with
    float *red = reinterpret_cast<float *>(smem);  // [W][8][D]
    float *red_m = red + kInt4Warps * kInt4MaxG * D, *red_l = red_m + kInt4Warps * kInt4MaxG;
    if (!H4 || t < 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float unit = pow2i(int4_weight_exponent(fe[h]));
            const int g = warp * kInt4MaxG + 2 * t + h;
            float2 *dst = reinterpret_cast<float2 *>(red + g * D + r * (8 * VW));
#pragma unroll
            for (int a = 0; a < 4 * VW; ++a)  // 2^24 / fe = 2^17 unit
                dst[a] = make_float2(fmaf(O[a][h] * 0x1p17f, unit, pm[h]),
                                     fmaf((O[a][2 + h] - O[a][h]) * 0x1p13f, unit, pm[h]));
            if (r == 0) {
                red_m[g] = my_steps > 0 ? M[h] * (careful > 1 ? 0x1p64f : 1.f) : -INFINITY;
                red_l[g] = l[h];
            }
        }
    }
    __syncthreads();
    const int nparts = piece.nparts;
    const int64_t slot = p.balanced ? piece.slot
                                    : ((int64_t)seq * p.num_kv_heads + kvh) * p.num_partitions +
                                          start / p.partition_tokens;
    uint16_t *out = static_cast<uint16_t *>(p.out) + ((int64_t)seq * p.num_q_heads + kvh * G) * D;
    for (int i = threadIdx.x; i < G * (D / 2); i += blockDim.x) {
        const int g = i / (D / 2), x0 = i % (D / 2) * 2;
        float M = -INFINITY;
        for (int w = 0; w < kInt4Warps; ++w) M = fmaxf(M, red_m[w * kInt4MaxG + g]);
        float lsum = 0.f, o0 = 0.f, o1 = 0.f;
        for (int w = 0; w < kInt4Warps; ++w) {
            const int at = w * kInt4MaxG + g;
            // a warp without tiles has l = 0; one of NaN scores alone, l = NaN
            const float f = red_l[at] == 0.f ? 0.f : fast_exp2(red_m[at] - M);
            lsum += f * red_l[at];
            o0 += f * red[at * D + x0];
            o1 += f * red[at * D + x0 + 1];
        }
        const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
        if (M == -INFINITY) M = 0.f;  // NaN scores alone: l = NaN counts
        if (nparts == 1) {
            *reinterpret_cast<uint32_t *>(out + g * D + x0) = narrow2<BF16>(o0 * inv, o1 * inv);
        } else {
            if (x0 == 0) {
                p.part_m[slot * kInt4MaxG + g] = M;
                p.part_l[slot * kInt4MaxG + g] = lsum;
            }
            *reinterpret_cast<float2 *>(p.part_o + (slot * G + g) * D + x0) =
                make_float2(o0 * inv, o1 * inv);
        }
    }
    if (!p.balanced) break;
    // the next piece's copies write where this one's sums stand
    __syncthreads();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }  // pieces
    if (!p.balanced) return;
    // every sequence's length is reported on by one CTA, which also writes the
    // rows of those without tokens
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
        if (item_len(p, s, threadIdx.x == 0) > 0) continue;
        uint32_t *row = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) +
                                                     (int64_t)s * p.num_q_heads * D);
        for (int i = threadIdx.x; i < p.num_q_heads * (D / 2); i += blockDim.x) row[i] = 0;
    }
}

// ------------------------------------------------------------------ host side
using Int4Kernel = void (*)(const Int4Params);
using Int4Merge = void (*)(const Int4Params, int);

template <bool BF16, int D>
static Int4Kernel int4_variant(int block_size, bool h4) {
    if (block_size == 16)
        return h4 ? decode_int4_kernel<BF16, D, 16, true> : decode_int4_kernel<BF16, D, 16, false>;
    return h4 ? decode_int4_kernel<BF16, D, 32, true> : decode_int4_kernel<BF16, D, 32, false>;
}

static Int4Kernel pick_int4(bool bf16, int D, int block_size, int group, int *smem) {
    const bool h4 = group <= 4;
    *smem = D == 64 ? Int4Shape<64>::SMEM_BYTES : Int4Shape<128>::SMEM_BYTES;
    if (D == 64)
        return bf16 ? int4_variant<true, 64>(block_size, h4) : int4_variant<false, 64>(block_size, h4);
    return bf16 ? int4_variant<true, 128>(block_size, h4) : int4_variant<false, 128>(block_size, h4);
}

template <bool BF16, int D>
static Int4Merge merge_variant(Int4MergeKind kind) {
    return kind == kMergeHeads    ? int4_merge_kernel<BF16, D, kMergeHeads>
           : kind == kMergeBounds ? int4_merge_kernel<BF16, D, kMergeBounds>
                                  : int4_merge_kernel<BF16, D, kMergeChunks>;
}

static Int4Merge pick_merge(bool bf16, int D, Int4MergeKind kind) {
    if (D == 64) return bf16 ? merge_variant<true, 64>(kind) : merge_variant<false, 64>(kind);
    return bf16 ? merge_variant<true, 128>(kind) : merge_variant<false, 128>(kind);
}

// Resident CTAs per SM; asked of the runtime once per variant and device.
static int int4_ctas_per_sm(bool bf16, int head_dim, int block_size, int group) {
    static std::mutex mu;
    static int known[128][16] = {};
    int smem = 0, n = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 1;
    int &slot = known[dev][8 * bf16 + 4 * (head_dim == 64) + 2 * (block_size == 32) + (group > 4)];
    std::lock_guard<std::mutex> lock(mu);
    if (slot > 0) return slot;
    Int4Kernel k = pick_int4(bf16, head_dim, block_size, group, &smem);
    if (!ensure_smem_attr(reinterpret_cast<const void *>(k), smem)) return 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, 32 * kInt4Warps, smem) != cudaSuccess)
        return 1;
    return slot = n > 0 ? n : 1;
}

// Heads of a bundle: the largest divisor of num_kv_heads up to 8.
static int int4_bundle(int num_kv_heads) {
    int b = num_kv_heads < 8 ? num_kv_heads : 8;
    while (num_kv_heads % b) --b;
    return b;
}

// How a call is cut, and its workspace.
struct Int4Cut {
    int ctas = 0;    // balanced ranges: CTAs of the launch (0: chunks)
    int wave = 0;    //   groups of its first wave
    int bundle = 1;  //   heads of a group
    int P = -1;      // chunks: positions of one, or -1 for single pass
    int chunks = 1;  //   of the longest sequence
    size_t l_off = 0, o_off = 0, bytes = 0;
};

// Checks the shapes and chooses.  Automatic: single pass for short heads, else
// balanced ranges, or up to eight chunks for more sequences than a CTA should scan
// the lengths of.
static pa_status int4_cut(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                          int block_size, int max_seq_len, int partition_tokens, pa_dtype dtype,
                          Int4Cut *c) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_seq_len < 0)
        return PA_ERR_INVALID;
    if (num_seqs > 65535 || num_kv_heads > 65535) return PA_ERR_INVALID;  // grid y and z
    if ((int64_t)num_seqs * num_q_heads > 0x7fffffff) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_INVALID;
    if (num_q_heads % num_kv_heads) return PA_ERR_INVALID;
    const int G = num_q_heads / num_kv_heads;
    if (G > kInt4MaxG || (head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if (partition_tokens < -1 || (partition_tokens > 0 && partition_tokens % block_size))
        return PA_ERR_INVALID;
    *c = {};
    if (num_seqs == 0) return PA_OK;
    int64_t slots = 0;
    const int whole = (int64_t)num_seqs * num_kv_heads >= kInt4ManyHeads ? kInt4SinglePassMany
                                                                         : kInt4SinglePass;
    if (partition_tokens == 0 && max_seq_len > whole) {
        c->bundle = int4_bundle(num_kv_heads);
        const int64_t units = (int64_t)num_seqs * (num_kv_heads / c->bundle) *
                              (((int64_t)max_seq_len + kInt4Unit - 1) / kInt4Unit);
        if (num_seqs <= kInt4BalancedSeqs && units < (1 << 30)) {
            const int64_t shares = (units + kInt4MinShare - 1) / kInt4MinShare;
            int64_t wave = (int64_t)sm_count() *
                           int4_ctas_per_sm(dtype == PA_BF16, head_dim, block_size, G) / c->bundle;
            if (wave < 1) wave = 1;
            const bool second = units >= wave * kInt4SecondWave;
            if (shares < wave) wave = shares;
            c->wave = (int)wave;
            c->ctas = (int)wave * c->bundle * (second ? 1 + kInt4SecondCtas : 1);
            slots = 2ll * c->ctas;
        } else {
            partition_tokens = (int)(((int64_t)max_seq_len + 7) / 8);
            if (partition_tokens < 4096) partition_tokens = 4096;
            partition_tokens = (partition_tokens + 31) / 32 * 32;
        }
    }
    if (partition_tokens > 0 && max_seq_len > partition_tokens) {
        c->P = partition_tokens;
        c->chunks = (int)(((int64_t)max_seq_len + partition_tokens - 1) / partition_tokens);
        slots = (int64_t)num_seqs * num_kv_heads * c->chunks;
    }
    auto align256 = [](size_t x) { return (x + 255) & ~size_t(255); };
    if (slots) {
        c->l_off = align256((size_t)slots * kInt4MaxG * sizeof(float));
        c->o_off = 2 * c->l_off;
        c->bytes = c->o_off + align256((size_t)slots * G * head_dim * sizeof(float));
    }
    return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_decode_int4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, int max_seq_len, int partition_tokens,
                                     pa_dtype dtype) {
    Int4Cut c;
    if (int4_cut(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                 partition_tokens, dtype, &c) != PA_OK)
        return 0;
    return c.bytes;
}

pa_status pa_decode_int4(void *out, const void *q, const void *k_pool, const void *v_pool,
                         int num_blocks, const int32_t *block_tables, int max_blocks_per_seq,
                         const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_q_heads,
                         int num_kv_heads, int head_dim, int block_size, float scale,
                         int partition_tokens, void *workspace, size_t workspace_bytes,
                         pa_dtype dtype, void *stream) {
    Int4Cut c;
    const pa_status st = int4_cut(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                  max_seq_len, partition_tokens, dtype, &c);
    if (st != PA_OK) return st;
    if (num_blocks <= 0 || max_blocks_per_seq < 0 || !std::isfinite(scale)) return PA_ERR_INVALID;
    // Positions are ints: a table's must be, and a sequence's (by its table and
    // max_seq_len) at most a single pass's.
    const int64_t table = (int64_t)max_blocks_per_seq * block_size;
    if (table > 0x7fffffff || (table > kSinglePassTokens && max_seq_len > kSinglePassTokens))
        return PA_ERR_INVALID;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !aligned16(out) ||
        !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool))
        return PA_ERR_INVALID;
    if (c.bytes && (!workspace || workspace_bytes < c.bytes ||
                    (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return PA_ERR_INVALID;
    const bool bf16 = dtype == PA_BF16;
    Int4Params p;
    std::memset(&p, 0, sizeof p);
    p.out = out;
    p.q = static_cast<const uint16_t *>(q);
    p.k_pool = static_cast<const uint16_t *>(k_pool);
    p.v_pool = static_cast<const uint16_t *>(v_pool);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.block_size = block_size;
    p.log2_block = block_size == 16 ? 4 : 5;
    p.scale_log2 = scale * kLog2e;
    p.partition_tokens = c.P > 0 ? c.P : kSinglePassTokens;
    p.num_partitions = c.chunks;
    p.balanced = c.wave;
    p.bundle = c.bundle;
    if (c.bytes) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        p.part_m = reinterpret_cast<float *>(ws);
        p.part_l = reinterpret_cast<float *>(ws + c.l_off);
        p.part_o = reinterpret_cast<float *>(ws + c.o_off);
    }
    p.err = error_word();
    if (!p.err) return PA_ERR_CUDA;

    int smem = 0;
    Int4Kernel k = pick_int4(bf16, head_dim, block_size, p.group, &smem);
    if (!ensure_smem_attr(reinterpret_cast<const void *>(k), smem)) return PA_ERR_CUDA;
    const int64_t heads = (int64_t)num_seqs * num_kv_heads;
    dim3 grid((unsigned)c.ctas);
    if (!c.ctas) {
        // small batches: only the chunks that exist, the short last ones at the end
        if (num_seqs <= kCompactMaxSeqs && heads * c.chunks < (1ll << 31)) p.compact = 2;
        grid = decode_grid(p, c.chunks, num_kv_heads, num_seqs);
    }
    cudaStream_t s = as_stream(stream);
    if (launch_pdl(k, grid, dim3(32 * kInt4Warps), (size_t)smem, s, p) != cudaSuccess)
        return PA_ERR_CUDA;
    if (c.ctas > c.bundle || c.P > 0) {
        // a head cut into 8 partials or more on average: a block a query head
        const Int4MergeKind kind = c.P > 0                ? kMergeChunks
                                   : 8 * heads <= c.ctas ? kMergeHeads
                                                          : kMergeBounds;
        const dim3 blocks = kind == kMergeChunks  ? dim3((unsigned)heads)
                            : kind == kMergeHeads ? dim3((unsigned)heads, (unsigned)p.group)
                                                  : dim3((unsigned)(c.ctas - c.bundle));
        if (launch_pdl(pick_merge(bf16, head_dim, kind), blocks, dim3(int4_merge_threads(kind)), 0, s,
                       p, c.ctas / c.bundle) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
