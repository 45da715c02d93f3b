// Host-side helpers shared by the translation units of the library.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"

namespace pa {

// Device address of the current device's error word (a file-scope __device__
// int in pa_cache.cu), looked up once per device.  nullptr on failure.
int *error_word();

// Number of SMs of the current device (cached per device); 0 on failure.
int sm_count();

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per (kernel, device).
bool ensure_smem_attr(const void *kernel, int bytes);

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

// scale * log2(e) in fp32, kept from 0: a masked position's infinity times it stays
// infinite.  The smallest fp32 number in its place makes less than 5e-7 of any score.
inline float latent_scale(float scale) {
    const float x = (float)((double)scale * 1.4426950408889634);
    return x == 0.f ? 1.401298464324817e-45f : x;  // 2^-149
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pa
