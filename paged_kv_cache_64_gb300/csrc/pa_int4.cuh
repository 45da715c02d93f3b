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

struct Int4Row {
    uint32_t codes;   // this lane's 8 codes, element e in bits [4e, 4e + 4)
    uint32_t params;  // the row's s (low half) and m as 16-bit values
};

// Quantise a row held by LANES consecutive lanes (aligned to LANES), 8
// elements x (exactly 16-bit values) a lane; every lane of the warp calls it.
//
// s is the smallest 16-bit value with 15 s >= span = fl(max - min): the
// nearest one to span / 15, or the next one up (15 s is exact in fp32: 11 + 4
// bits).  Codes are the integers nearest to a / s, a = fl(x - m), ties to
// even.  The quotient t' = t + (a - t s) / s is the correctly rounded one (a
// Newton step with an exact FMA remainder), so a tie, which is a quotient
// fp32 holds exactly, is met exactly, and adding 1.5 * 2^23 rounds it to
// even.  A quotient next to a tie may round onto it; the remainder a - n s,
// exact there, then passes s / 2 and the element is taken again with that
// comparison.
template <bool BF16, int LANES>
__device__ __forceinline__ Int4Row quantise_row_int4(const float *x) {
    float lo = x[0], hi = x[0];
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        fine &= fabsf(x[i]) < INFINITY;
    }
    if (!fine) hi = INFINITY, lo = 0.f;
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFullMask, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFullMask, hi, o));
    }
    Int4Row r;
    const float span = hi - lo;
    if (!(span < INFINITY)) {  // the same in every lane of the row
        r.codes = 0u;
        r.params = BF16 ? 0x7fc07fc0u : 0x7e007e00u;
        return r;
    }
    lo += 0.f;  // -0 becomes +0
    uint32_t sb = bits16<BF16>(__fdiv_rn(span, 15.f));
    float s = from16<BF16>(sb);
    if (15.f * s < span) s = from16<BF16>(++sb);
    r.params = sb | (bits16<BF16>(lo) << 16);
    if (span == 0.f) {
        r.codes = 0u;
        return r;
    }
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the integer
    const float h = 0.5f * s, inv = __frcp_rn(s);
    const bool tiny = s < 0x1p-100f;      // 1 / s may pass fp32's range (bf16 only)
    float off = 0.f;
    uint32_t codes = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = x[i] - lo;
        float t = a * inv;
        t = fmaf(fmaf(-t, s, a), inv, t);
        const float u = t + kMagic;
        off = fmaxf(off, fabsf(fmaf(kMagic - u, s, a)));
        codes += (__float_as_uint(u) & 15u) << (4 * i);
    }
    if (tiny || off > h) {
        codes = 0u;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i == j) a = x[j] - lo;
            float n = rintf(__fdiv_rn(a, s));
            const float d = fmaf(-n, s, a);
            if (d > h) n += 1.f;
            if (d < -h) n -= 1.f;
            codes |= (uint32_t)fminf(fmaxf(n, 0.f), 15.f) << (4 * i);
        }
    }
    r.codes = codes;
    return r;
}

// The 8 values that codes with (s, m) stand for, as 16-bit values: fl(m + s n)
// (s n is exact) rounded to nearest even, saturating at the largest finite
// value; NaN where s is NaN.
template <bool BF16>
__device__ __forceinline__ uint4 read8_int4(uint32_t codes, uint32_t params) {
    const float top = BF16 ? 3.38953138925e38f : 65504.f;
    const float s = from16<BF16>(params & 0xffffu), m = from16<BF16>(params >> 16);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float n = (float)((codes >> (8 * i + 4 * j)) & 15u);
            const float y = fmaf(s, n, m);
            v[j] = fabsf(y) > top ? copysignf(top, y) : y;  // keeps NaN
        }
        w[i] = narrow2<BF16>(v[0], v[1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace pa
