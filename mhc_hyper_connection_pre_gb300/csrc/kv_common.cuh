// kv_common.cuh -- device helpers shared by the kv kernels (sm_103a).
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_index.cuh"

namespace mhc {
namespace kv {

// Device status word of a translation unit: a bad index.  Read and cleared by
// mhc_device_status().
constexpr unsigned int kIndexError = 2u;

// The sequence that token t belongs to: the last b with cu[b] <= t.  Called
// by a whole warp with the same t; 32 probes a round, so two rounds up to
// 1024 sequences.  Any cu gives some b in [0, B).
__device__ __forceinline__ int seq_of(const Seqs& s, int t, int lane) {
    if (!s.cu) return t;
    int lo = 0, hi = s.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int probe = lo + (lane + 1) * step;
        const bool below = probe < hi && __ldg(s.cu + probe) <= t;
        const int up = lo + step * __popc(__ballot_sync(0xffffffffu, below));
        lo = up;
        hi = hi < up + step ? hi : up + step;
    }
    return lo;
}

// Four e4m3 numbers of x[at .. at + 3], to nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x4(const float (&x)[8], int at) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[at], x[at + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[at + 2], x[at + 3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Two e4m3 numbers as two f16 (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

}  // namespace kv
}  // namespace mhc
