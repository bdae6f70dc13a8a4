// kv_attend.cuh -- what the kernels of mhc_kv_attend share: their arguments,
// the table of sequences from which blocks find their part of the work, the
// parts that cut tiles leave behind, and the tensor maps of the cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_common.cuh"
#include "sm100.cuh"

namespace mhc {
namespace kv {

constexpr int kTable = 256;                   // sequences of a block's table
constexpr float kLift = 10.0f;                // weights are 2^10 times the softmax's numerators
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What a block left unfinished: slot 1 a tile that it began, slot 0 one that
// it went on with.
struct PartDesc {
    int valid, last;                          // last: the tile ends here
    int begin, first_row, rows, head;         // rows of the tile
    int pad[2];
};

struct AttendArgs {
    Seqs seqs;
    Cut cut;
    const float* k_scale;
    const float* v_scale;
    const uint16_t* q;
    int64_t q_stride;
    float scale_log2;                         // softmax_scale * log2(e)
    uint16_t* out;
    float* lse;
    float* part;                              // [blocks][2][tile_rows][D + 2]: maximum, sum, the weighted values
    PartDesc* desc;                           // [blocks][2]
};

struct Table {
    SeqInfo info[kTable];
    int64_t prefix[kTable];
    int64_t warp_sum[kTable / 32];
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) { return f16x2_of_e4m3x2((uint16_t)(w & 0xffffu)); }
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) { return f16x2_of_e4m3x2((uint16_t)(w >> 16)); }

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Bytes of w that are e4m3's NaN, as 0x80 in each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Asynchronous 4-byte copy into shared memory, and an arrival on an mbarrier
// once this thread's copies so far have landed.
__device__ __forceinline__ void copy_async4(void* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// What the first threads of the first block check of the call as a whole.
__device__ __forceinline__ void check_offsets(const AttendArgs& a) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.seqs.cu && (a.seqs.cu[0] != 0 || a.seqs.cu[a.seqs.B] != a.seqs.T))
        atomicOr(&g_device_status, kIndexError);
}

// The barrier of the whole block; unlike __syncthreads, it may be met in
// different places of the code.
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 0;" ::: "memory"); }

// Fills the table with sequences base .. base + kTable - 1 and the running sum
// of their units; returns the units of them all.  Whole block, of at least
// kTable threads.
__device__ inline int64_t fill_table(const AttendArgs& a, Table& tab, int base) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int64_t mine = 0, run = 0;
    if (tid < kTable) {
        SeqInfo info{0, 0, 0, 0};
        if (base + tid < a.seqs.B) {
            const Span sp = span_of(a.seqs, base + tid);
            if (sp.bad) atomicOr(&g_device_status, kIndexError);
            info = info_of(sp, a.cut.group);
            mine = units_of_seq(info, a.cut);
        }
        tab.info[tid] = info;
        run = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
        }
        if (lane == 31) tab.warp_sum[warp] = run;
    }
    block_sync();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kTable / 32; ++w) {
        const int64_t s = tab.warp_sum[w];
        if (w < warp) before += s;
        total += s;
    }
    if (tid < kTable) tab.prefix[tid] = before + run - mine;
    block_sync();
    return total;
}

__device__ __forceinline__ void segment_keys(const Walk& w, const SeqInfo* info, const Cut& cut, int& key0, int& keys) {
    const int all = keys_of_tile(info[w.b], cut, w.tile), end = (w.first + w.count) * cut.unit;
    key0 = w.first * cut.unit;
    keys = end < all ? end : all;
}

// Row `row` of a sequence (new token row / group, query head row % group of
// the key/value head): its place in out and lse.
__device__ __forceinline__ int64_t place_of(const AttendArgs& a, int begin, int row, int head) {
    return (int64_t)(begin + row / a.cut.group) * (a.cut.heads * a.cut.group) + head * a.cut.group + row % a.cut.group;
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : kLn2 * (m - kLift + __log2f(l));
}

using PFN_encodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline PFN_encodeTiled encode_fn() {
    static const PFN_encodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_encodeTiled>(p) : nullptr;
    }();
    return fn;
}

// Codes as [num_pages * heads][page_tokens][D] bytes, in boxes of up to
// `tokens` tokens, each token's row in the swizzle of its length (D bytes).
inline bool encode_codes(CUtensorMap* map, const uint8_t* codes, int64_t blocks, int page_tokens, int D, int tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)page_tokens, (cuuint64_t)blocks};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * page_tokens};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)(page_tokens < tokens ? page_tokens : tokens), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode_fn() &&
           encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kv
}  // namespace mhc
