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
// tile's layout.  The weights P s' are split into two f16 terms (22 bits) and
// scaled by a power of two kept, like the running maximum, per warp.
//
// Why not tcgen05: its A operand comes from shared memory, where codes would
// have to be stored again as 8- or 16-bit values, four to eight times the
// bytes that were read, and its smallest tile is 64 rows of a CTA-wide
// pipeline; with 8 columns a position costs a warp one MMA here (K and V
// together two), and the masks feed it from the registers the loads filled.
//
// A warp works alone: its own tiles of 16 positions (every fourth of the
// CTA's chunk), its own ring of stages filled by cp.async, its own running
// maximum and sums; the four warps merge at the end through shared memory.
// Long sequences are split over CTAs and combined as in the other decodes.
#include <cstdint>

#include "pa_decode.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kInt4Warps = 4;
constexpr int kInt4MaxG = 8;

template <int D>
struct Int4Shape {
    static constexpr int CODES = kUnit * D / 2;             // bytes of a tile's codes
    static constexpr int STAGE = 2 * CODES + 2 * kUnit * 4; // K codes, V codes, K and V (s, m)
    static constexpr int STAGES = D == 128 ? 4 : 6;
    static constexpr int RING = STAGES * STAGE;             // a warp's
    static constexpr int RED_BYTES = kInt4Warps * kInt4MaxG * (D + 2) * 4;
    static constexpr int SMEM_BYTES = kInt4Warps * RING > RED_BYTES ? kInt4Warps * RING : RED_BYTES;
};

// D += A B: A 16 x 16 f16 (row-major fragments), B 16 x 8 f16, D 16 x 8 fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t half2_bits(float a, float b) { return narrow2<false>(a, b); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kInt4Warps, 4) decode_int4_kernel(const DecodeParams p) {
    using S = Int4Shape<D>;
    constexpr int KW = D / 32;  // words of a key row a lane holds (32 D / 128 codes)
    constexpr int VW = D / 64;  // words of a value row a lane holds
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, t = lane & 3;  // fragment row (or column) and quad lane
    pdl_wait();
    int chunk, kvh, seq;
    if (p.compact) {
        if (!compact_item(p, blockIdx.x, &seq, &chunk, &kvh)) return;
    } else {
        chunk = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
    }
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
    const int end = L - start < P ? L : start + P;
    const int ntiles = (end - start + kUnit - 1) / kUnit;
    const int my_tiles = (ntiles - warp + kInt4Warps - 1) / kInt4Warps;

    // -------------------------------------------------------------- loads
    uint8_t *ring = smem + warp * S::RING;
    const int rec_bytes = int4_record_bytes<D>(p.block_size);
    const uint8_t *kpool = reinterpret_cast<const uint8_t *>(p.k_pool);
    const uint8_t *vpool = reinterpret_cast<const uint8_t *>(p.v_pool);
    const int32_t *table = seq_table(p, seq);
    // block ids of this warp's tiles, 32 tiles at a time, a lane each
    auto window = [&](int w) -> int {
        const int kt = warp + kInt4Warps * (32 * w + lane);
        if (kt >= ntiles) return 0;
        const int phys = table[(start + kt * kUnit) >> p.log2_block];
        if ((unsigned)phys < (unsigned)p.num_blocks) return phys;
        record_error(p.err, PA_ERR_BAD_INDEX);
        return 0;
    };
    int cur = window(0), nxt = 0;
    auto issue = [&](int k, int stage) {
        if (k < my_tiles) {
            if ((k & 31) == 0) {
                if (k) cur = nxt;
                nxt = window((k >> 5) + 1);
            }
            const int phys = __shfl_sync(kFullMask, cur, k & 31);
            const int row = (start + (warp + kInt4Warps * k) * kUnit) & (p.block_size - 1);
            const int64_t rec = ((int64_t)phys * p.num_kv_heads + kvh) * rec_bytes;
            const int codes = row * (D / 2), params = p.block_size * (D / 2) + row * 4;
            uint8_t *dst = ring + stage * S::STAGE;
#pragma unroll
            for (int i = 0; i < S::CODES / 512; ++i) {
                const int b = i * 512 + lane * 16;
                cp_async16_cg(dst + b, kpool + rec + codes + b);
                cp_async16_cg(dst + S::CODES + b, vpool + rec + codes + b);
            }
            if (lane < 8)
                cp_async16_cg(dst + 2 * S::CODES + lane * 16,
                              (lane < 4 ? kpool : vpool) + rec + params + (lane & 3) * 16);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < S::STAGES - 1; ++k) issue(k, k);

    // ------------------------------------------------------------ queries
    // B fragments: column r is head r, this lane's elements are those of its
    // key words.  2^kq brings the head's largest |q| below 2^15; elements
    // that meet codes in the high four bits are divided by 16.
    uint32_t qf[KW][4];
    float cs[2], qs[2];  // of the score tile's columns 2t, 2t + 1
    {
        float x[KW][8];
        float top = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (r < G)
                raw = *reinterpret_cast<const uint4 *>(
                    p.q + ((int64_t)seq * p.num_q_heads + kvh * G + r) * D + (t * KW + j) * 8);
            widen8<BF16>(raw, x[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                top = fmaxf(top, fabsf(x[j][i]));
                sum += x[j][i];
            }
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            sum += __shfl_xor_sync(kFullMask, sum, o);
        }
        int kq = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
        kq = kq > 100 ? 100 : kq < -100 ? -100 : kq;
        const float even = pow2i(kq), odd = pow2i(kq - 4);
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = i & 1 ? odd : even;
                qf[j][i] = half2_bits(x[j][i] * f, x[j][i + 4] * f);
            }
        const float c = p.scale_log2 * pow2i(24 - kq), s = sum * p.scale_log2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            cs[h] = __shfl_sync(kFullMask, c, 4 * (2 * t + h));
            qs[h] = __shfl_sync(kFullMask, s, 4 * (2 * t + h));
        }
    }

    // ---------------------------------------------------------- main loop
    // O[a][...]: dimensions 2a and 2a + 1 of this lane's D/8, heads 2t and
    // 2t + 1, in units of 2^-24 / fe (odd dimensions 16 times that).
    float O[4 * VW][4];
#pragma unroll
    for (int a = 0; a < 4 * VW; ++a) O[a][0] = O[a][1] = O[a][2] = O[a][3] = 0.f;
    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, pm[2] = {0.f, 0.f};
    int ve = -110;                  // scales of V seen so far are below 2^ve
    float fe = pow2i(7 - ve);       // weights are P s' fe, at most 2^8 2^7
    // Fragment row r is position pr of its half tile: pairs of rows (r, r + 1)
    // and rows of equal t differ in parity, so that neither the key loads (two
    // rows a quarter warp) nor the value loads (four rows a half warp) meet in
    // a bank more than they must.
    const int pr = r ^ ((r >> 1) & 1);
    const int pv[2] = {(2 * t) ^ (t & 1), (2 * t + 1) ^ (t & 1)};
    constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;
    int stage = 0;
    for (int k = 0; k < my_tiles; ++k) {
        cp_async_wait<S::STAGES - 2>();
        __syncwarp();
        issue(k + S::STAGES - 1, stage == 0 ? S::STAGES - 1 : stage - 1);
        const uint8_t *tile = ring + stage * S::STAGE;
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;

        // scores: two chains of MMAs over the dimensions
        uint32_t w0[KW], w1[KW];
        if constexpr (KW == 4) {
            const uint4 a = *reinterpret_cast<const uint4 *>(tile + pr * 64 + t * 16);
            const uint4 b = *reinterpret_cast<const uint4 *>(tile + (8 + pr) * 64 + t * 16);
            w0[0] = a.x; w0[1] = a.y; w0[2] = a.z; w0[3] = a.w;
            w1[0] = b.x; w1[1] = b.y; w1[2] = b.z; w1[3] = b.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(tile + pr * 32 + t * 8);
            const uint2 b = *reinterpret_cast<const uint2 *>(tile + (8 + pr) * 32 + t * 8);
            w0[0] = a.x; w0[1] = a.y;
            w1[0] = b.x; w1[1] = b.y;
        }
        const uint32_t *par = reinterpret_cast<const uint32_t *>(tile + 2 * S::CODES);
        const uint32_t pk0 = par[pr], pk1 = par[8 + pr], pv0 = par[16 + pr], pv1 = par[24 + pr];
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            mma_f16(c0, w0[j] & kLo, w1[j] & kLo, w0[j] & kHi, w1[j] & kHi, qf[j][0], qf[j][1]);
            const uint32_t u0 = w0[j] >> 8, u1 = w1[j] >> 8;
            mma_f16(c1, u0 & kLo, u1 & kLo, u0 & kHi, u1 & kHi, qf[j][2], qf[j][3]);
        }
        const float sk0 = from16<BF16>(pk0 & 0xffffu), mk0 = from16<BF16>(pk0 >> 16);
        const float sk1 = from16<BF16>(pk1 & 0xffffu), mk1 = from16<BF16>(pk1 >> 16);
        float sv0 = from16<BF16>(pv0 & 0xffffu), mv0 = from16<BF16>(pv0 >> 16);
        float sv1 = from16<BF16>(pv1 & 0xffffu), mv1 = from16<BF16>(pv1 >> 16);
        float s[4];  // (position pr, heads 2t, 2t + 1), (position 8 + pr, the same), base 2
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = fmaf(c0[h] + c1[h], sk0 * cs[h], mk0 * qs[h]);
            s[2 + h] = fmaf(c0[2 + h] + c1[2 + h], sk1 * cs[h], mk1 * qs[h]);
        }
        const int left = end - start - (warp + kInt4Warps * k) * kUnit;
        if (left < kUnit) {  // slots past the end hold anything
            if (pr >= left) s[0] = s[1] = -INFINITY, sv0 = mv0 = 0.f;
            if (8 + pr >= left) s[2] = s[3] = -INFINITY, sv1 = mv1 = 0.f;
        }

        // The running maximum moves only when a score passes it by more than
        // kLazyRescale, the running scale when one passes it.
        const float sv = fmaxf(sv0, sv1);
        const bool moves = fmaxf(s[0], s[2]) > M[0] + kLazyRescale ||
                           fmaxf(s[1], s[3]) > M[1] + kLazyRescale || sv * fe > 128.f;
        if (__any_sync(kFullMask, moves)) {
            float top = sv, mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(kFullMask, mx[0], o));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(kFullMask, mx[1], o));
            }
            int e = (int)(__float_as_uint(top) >> 23) - 126;  // top < 2^e
            e = e > 127 ? 127 : e < ve ? ve : e;
            const float shrink = pow2i(ve - e < -126 ? -126 : ve - e);
            ve = e;
            fe = pow2i(7 - ve);
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float m = fmaxf(M[h], mx[h]);
                f[h] = m == -INFINITY ? 1.f : fast_exp2(M[h] - m);
                M[h] = m;
                l[h] *= f[h];
                pm[h] *= f[h];
                f[h] *= shrink;
            }
#pragma unroll
            for (int a = 0; a < 4 * VW; ++a) {
                O[a][0] *= f[0];
                O[a][1] *= f[1];
                O[a][2] *= f[0];
                O[a][3] *= f[1];
            }
        }

        // weights, their sums, and the two f16 terms of P s' fe, transposed to
        // B fragments (rows: positions, columns: heads)
        uint32_t bh[2], bl[2];
        {
            const float g0 = sv0 * fe, g1 = sv1 * fe;
            const float p0 = fast_exp2(s[0] - M[0]), p1 = fast_exp2(s[1] - M[1]);
            const float p2 = fast_exp2(s[2] - M[0]), p3 = fast_exp2(s[3] - M[1]);
            l[0] += p0 + p2;
            l[1] += p1 + p3;
            pm[0] = fmaf(p0, mv0, fmaf(p2, mv1, pm[0]));
            pm[1] = fmaf(p1, mv0, fmaf(p3, mv1, pm[1]));
            const float x0 = p0 * g0, x1 = p1 * g0, x2 = p2 * g1, x3 = p3 * g1;
            const uint32_t h0 = half2_bits(x0, x1), h1 = half2_bits(x2, x3);
            const float2 y0 = widen2<false>(h0), y1 = widen2<false>(h1);
            bh[0] = transpose8(h0);
            bh[1] = transpose8(h1);
            bl[0] = transpose8(half2_bits(x0 - y0.x, x1 - y0.y));
            bl[1] = transpose8(half2_bits(x2 - y1.x, x3 - y1.y));
        }

        // O += V^T (P s')
        const uint8_t *vt = tile + S::CODES + r * (4 * VW);
        uint32_t v[4][VW];  // positions pv[0], pv[1], 8 + pv[0], 8 + pv[1]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *src = vt + ((i >> 1) * 8 + pv[i & 1]) * (D / 2);
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
                uint32_t x = __byte_perm(v[0][j], v[1][j], sel);
                uint32_t y = __byte_perm(v[2][j], v[3][j], sel);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float(&acc)[4] = O[4 * j + 2 * half + q];
                    const uint32_t a0 = x & kLo, a1 = x & kHi, a2 = y & kLo, a3 = y & kHi;
                    mma_f16(acc, a0, a1, a2, a3, bh[0], bh[1]);
                    mma_f16(acc, a0, a1, a2, a3, bl[0], bl[1]);
                    x >>= 8;
                    y >>= 8;
                }
            }
        }
    }

    // -------------------------------------------------------------- merge
    pdl_trigger();
    cp_async_wait<0>();
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFullMask, l[h], o);
            pm[h] += __shfl_xor_sync(kFullMask, pm[h], o);
        }
    __syncthreads();  // the rings are done with
    float *red = reinterpret_cast<float *>(smem);  // [W][8][D]
    float *red_m = red + kInt4Warps * kInt4MaxG * D, *red_l = red_m + kInt4Warps * kInt4MaxG;
    {
        const float unit = pow2i(ve);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int g = warp * kInt4MaxG + 2 * t + h;
            float2 *dst = reinterpret_cast<float2 *>(red + g * D + r * (8 * VW));
#pragma unroll
            for (int a = 0; a < 4 * VW; ++a)  // 2^24 / fe = 2^(17 + ve)
                dst[a] = make_float2(fmaf(O[a][h] * 0x1p17f, unit, pm[h]),
                                     fmaf(O[a][2 + h] * 0x1p13f, unit, pm[h]));
            if (r == 0) {
                red_m[g] = M[h];
                red_l[g] = l[h];
            }
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
            // a warp without tiles has l = 0; one of NaN scores alone, l = NaN
            const float f = red_l[at] == 0.f ? 0.f : fast_exp2(red_m[at] - M);
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
                p.part_m[row] = M == -INFINITY ? 0.f : M;  // NaN scores alone: l = NaN counts
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
    DecodeParams p = prm;
    if (p.compact) p.compact = 2;  // full chunks first, the short last ones at the end
    const dim3 grid = decode_grid(p, num_partitions, num_kv_heads, num_seqs);
    if (launch_pdl(k, grid, dim3(32 * kInt4Warps), (size_t)smem, stream, p) != cudaSuccess)
        return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
