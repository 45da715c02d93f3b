// 4-bit KV rows: the record layout, the quantiser and the read-back, shared
// by the cache write and read, the fused norm-rotation-write and the decode.
//
// A row of D 16-bit values is held as codes n in 0 .. 15 with a scale s and a
// minimum m of its own (of the 16-bit type): it stands for m + s n.  The
// record of a (block, KV head) is [B][D/2] bytes of codes, element 2i in the
// low half of byte i, then B pairs (s, m).
#pragma once

#include "pa_common.cuh"

namespace pa {

template <int D>
__host__ __device__ constexpr int int4_record_bytes(int block_size) {
    return block_size * (D / 2 + 4);
}

// Bits of the 16-bit value nearest to x.
template <bool BF16>
__device__ __forceinline__ uint32_t bits16(float x) {
    return BF16 ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x))
                : (uint32_t)__half_as_ushort(__float2half_rn(x));
}

template <bool BF16>
__device__ __forceinline__ float from16(uint32_t b) {
    return BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
}

// 8 16-bit values as fp32.
template <bool BF16>
__device__ __forceinline__ void widen8(uint4 v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = widen2<BF16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The smaller (larger) of two pairs of 16-bit values, NaN if either is.
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A row's share of one lane: W words of 8 codes, and the row's scale and
// minimum as 16-bit values (s in the low half).
template <int W>
struct Int4Row {
    uint32_t codes[W];  // element e of word w in bits [4e, 4e + 4)
    uint32_t params;
};

// The 8 values that codes with (s, m) stand for, as 16-bit values: fl(m + s n)
// (s n is exact) rounded to nearest even, saturating at the largest finite
// value; NaN where s is NaN.
template <bool BF16>
__device__ __forceinline__ uint4 read8_int4(uint32_t codes, uint32_t params) {
    constexpr float top = BF16 ? 3.38953138925e38f : 65504.f;
    const float2 sm = widen2<BF16>(params);
    const float s = sm.x, m = sm.y;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // 0x4b000000 | n is 2^23 + n
        const uint32_t n = i == 0 ? codes & 15u : (codes >> (4 * i)) & 15u;
        y[i] = fmaf(s, __uint_as_float(0x4b000000u | n) - 8388608.f, m);
    }
    if (fabsf(m) > top || !(fmaf(s, 15.f, m) <= top)) {  // rare; keeps NaN
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(y[i]) > top) y[i] = copysignf(top, y[i]);
    }
    return make_uint4(narrow2<BF16>(y[0], y[1]), narrow2<BF16>(y[2], y[3]),
                      narrow2<BF16>(y[4], y[5]), narrow2<BF16>(y[6], y[7]));
}

// Quantise a row held by LANES consecutive lanes (aligned to LANES), 8 W
// elements raw (16-bit) a lane; every lane of the warp calls it.
//
// s is the smallest 16-bit value with 15 s >= span = fl(max - min): the
// nearest one to span / 15, or the next one up (15 s is exact in fp32: 11 + 4
// bits).  Codes are the integers nearest to a / s, a = fl(x - m), ties to
// even.  The quotient t' = t + (a - t s) / s, with the remainder exact by FMA, is
// Markstein's correction of a product with the reciprocal (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): a tie, which is a quotient fp32 holds exactly, is met exactly, and
// adding 1.5 * 2^23 rounds it to even.  A quotient next to a tie may round onto
// it; the remainder a - n s, exact there, then passes s / 2 and the lane's
// elements are taken again with that comparison.  With OUT, y receives the values the codes stand for, as
// read8_int4 gives them.
template <bool BF16, int LANES, int W, bool OUT>
__device__ __forceinline__ Int4Row<W> quantise_row_int4(const uint4 (&raw)[W], uint4 *y) {
    // minimum and maximum on packed pairs; a lane's as (min, -max), so that one
    // shuffle and one minimum a step reduce both
    uint32_t mn = raw[0].x, mx = raw[0].x;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const uint32_t v[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int i = w == 0 ? 1 : 0; i < 4; ++i) {
            mn = min2<BF16>(mn, v[i]);
            mx = max2<BF16>(mx, v[i]);
        }
    }
    mx ^= 0x80008000u;
    uint32_t ends = min2<BF16>(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1)
        ends = min2<BF16>(ends, __shfl_xor_sync(kFullMask, ends, o));
    const float2 e = widen2<BF16>(ends);
    const float lo = e.x + 0.f;  // -0 becomes +0
    Int4Row<W> r;
    const float span = (0.f - e.y) - lo;  // never -0
    if (!(span < INFINITY)) {  // a NaN, an infinity or past fp32: the same in every lane of the row
#pragma unroll
        for (int w = 0; w < W; ++w) {
            r.codes[w] = 0u;
            if (OUT) y[w] = read8_int4<BF16>(0u, BF16 ? 0x7fc07fc0u : 0x7e007e00u);
        }
        r.params = BF16 ? 0x7fc07fc0u : 0x7e007e00u;
        return r;
    }
    uint32_t sb = bits16<BF16>(__fdiv_rn(span, 15.f));
    float s = from16<BF16>(sb);
    if (15.f * s < span) s = from16<BF16>(++sb);
    r.params = sb | (bits16<BF16>(lo) << 16);
    // (span = 0: s = 0, 1 / s infinite and every quotient NaN; redone below)
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the integer
    const float h = 0.5f * s, inv = __frcp_rn(s);
    float off = s < 0x1p-100f ? INFINITY : 0.f;  // 1 / s may pass fp32's range (bf16 only)
    const float2 inv2 = make_float2(inv, inv), s2 = make_float2(s, s), lo2 = make_float2(lo, lo);
    const float2 magic2 = make_float2(kMagic, kMagic);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const uint32_t word[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
        uint32_t out[4];
        // sum of (kMagic's bits + n_i) 16^i, modulo 2^32
        uint32_t codes = 0u;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const float2 x = widen2<BF16>(word[i]);
            const float2 a = __fadd2_rn(x, make_float2(-lo, -lo));
            float2 q = __fmul2_rn(a, inv2);
            q = __ffma2_rn(__ffma2_rn(make_float2(-q.x, -q.y), s2, a), inv2, q);
            const float2 u = __fadd2_rn(q, magic2);
            const float2 n = __fadd2_rn(u, make_float2(-kMagic, -kMagic));
            const float2 d = __ffma2_rn(n, make_float2(-s, -s), a);
            off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
            codes = codes * 16u + __float_as_uint(u.y);
            codes = codes * 16u + __float_as_uint(u.x);
            if (OUT) {
                const float2 v = __ffma2_rn(n, s2, lo2);
                out[i] = narrow2<BF16>(v.x, v.y);
            }
        }
        r.codes[w] = codes - 0x4b400000u * 0x11111111u;
        if (OUT) y[w] = make_uint4(out[0], out[1], out[2], out[3]);
    }
    // values that could pass the largest finite one are taken again too
    bool again = OUT && !(fmaf(s, 15.f, lo) <= (BF16 ? 3.38953138925e38f : 65504.f));
    if (off > h) {
        again = true;
#pragma unroll 1
        for (int w = 0; w < W; ++w) {
            uint4 v = raw[0];
#pragma unroll
            for (int j = 1; j < W; ++j)
                if (w == j) v = raw[j];
            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
            uint32_t codes = 0u;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint32_t pair = i < 4 ? (i < 2 ? word[0] : word[1]) : (i < 6 ? word[2] : word[3]);
                const float a = from16<BF16>(i & 1 ? pair >> 16 : pair & 0xffffu) - lo;
                float n = s > 0.f ? rintf(__fdiv_rn(a, s)) : 0.f;
                const float d = fmaf(-n, s, a);
                if (d > h) n += 1.f;
                if (d < -h) n -= 1.f;
                codes |= (uint32_t)fminf(fmaxf(n, 0.f), 15.f) << (4 * i);
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (w == j) r.codes[j] = codes;
        }
    }
    if (OUT && again) {
#pragma unroll
        for (int w = 0; w < W; ++w) y[w] = read8_int4<BF16>(r.codes[w], r.params);
    }
    return r;
}

}  // namespace pa
