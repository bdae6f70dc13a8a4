// kv_attend.cuh -- what the kernels of mhc_kv_attend share: their arguments,
// how a warp or block finds its part of the work, the parts that cut tiles
// leave behind, and the tensor maps of the cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_common.cuh"
#include "sm100.cuh"

namespace mhc {
namespace kv {

constexpr float kLift = 10.0f;                // weights are 2^10 times the softmax's numerators
constexpr float kGrow = 5.0f;                   // the maximum follows when it has grown by more (in powers of two)
constexpr float kPartsLog2 = 12.0f;             // a tile has fewer than 2^12 parts; the join divides their weights by it
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The value scale that a tile's values are held relative to, from the largest
// one: at least the smallest normal number, so that its reciprocal is finite.
// Zero if all are.
__device__ __forceinline__ float value_unit(float most) { return most > 0.0f ? fmaxf(most, 1.17549435e-38f) : 0.0f; }

// A part of a tile that a share has left in the workspace.
struct PartDesc {
    int parts, owner;                         // as the segment's; parts 0: nothing here
    Segment seg;
};

struct AttendArgs {
    Seqs seqs;
    Cut cut;
    int shares;
    const float* k_scale;
    const float* v_scale;
    const uint16_t* q;
    int64_t q_stride;
    float scale_log2;                         // softmax_scale * log2(e)
    uint16_t* out;
    float* lse;
    float* part;                              // [shares][2]: mean of the values [rows][D], log2 of the weights' sum [rows]
    PartDesc* desc;                           // [shares][2]
};

// Part `slot` of a share: 1 of the tile that it began (it is the owner), 0 of one that it went on with.
__device__ __forceinline__ float* part_of(const AttendArgs& a, int share, int slot, int D) {
    return a.part + (((int64_t)share * 2 + slot) * (D + 1) << a.cut.tile_log2);
}

constexpr int kSegments = 32;                 // that the tensor-memory kernel plans at a time

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// To within a step or two of fp32, for normal numbers.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// The warp that runs it.
struct ThisWarp {
    int lane;
    __device__ __forceinline__ bool first() const { return lane == 0; }
    __device__ __forceinline__ bool any(bool x) const { return __any_sync(0xffffffffu, x); }
    __device__ __forceinline__ void sync() const { __syncwarp(); }
};

// Finds sequence b for a plan.
struct Lookup {
    const AttendArgs& a;
    __device__ __forceinline__ int count() const { return a.seqs.B; }
    __device__ __forceinline__ SeqInfo operator()(int b) const { return info_of(span_of(a.seqs, b < a.seqs.B ? b : a.seqs.B - 1)); }
};

__device__ __forceinline__ int64_t sum_upto(int64_t x, int lane) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += up;
    }
    return x;
}

// With more than 32 sequences a 32nd of them is this many.
__device__ __forceinline__ int each_of(const AttendArgs& a) { return a.seqs.B <= 32 ? 1 : (a.seqs.B + 31) / 32; }

// More sequences than this are counted by all warps of a block together.  In the
// one-token kernel, 1 head, up to 100 keys: 200 sequences take 17.4 us, with each
// warp by itself 17.1; 300: 17.3 and 19.0; 1024: 21 and 27.
constexpr int kTogether = 256;

// Units of the sequences of 32nd i, by one warp.
__device__ inline void count_units(const AttendArgs& a, int i, int lane, int64_t& units) {
    const Lookup look{a};
    const int each = each_of(a), end = (i + 1) * each < a.seqs.B ? (i + 1) * each : a.seqs.B;
    int64_t n = 0;
#pragma unroll 1
    for (int b = i * each + lane; b < end; b += 32) n += units_of_seq(look(b), a.cut);
#pragma unroll 1
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) units = n;
}

// Finds a share of the line and starts its plan; the line's shares in `shares`.
// One warp, which counts the units of all sequences: up to 32 of them a lane
// each, beyond that a 32nd of them each (or takes the counts of count_units) and
// then the ones of the 32nd in which the share begins.  No block-wide step, and
// each length is loaded once or twice: what a decode step's latency consists of
// is loads that wait for one another.
__device__ inline void find_share(const AttendArgs& a, int share, Plan& p, Shares& shares, int lane,
                                  const int64_t* counted = nullptr) {
    const Lookup look{a};
    const int each = each_of(a), first = lane * each;
    const int end = first + each < a.seqs.B ? first + each : a.seqs.B;
    SeqInfo info{0, 0, 0};
    int64_t mine = 0;
    if (counted) {
        mine = counted[lane];
    } else {
#pragma unroll 4
        for (int i = first; i < end; ++i) {
            info = look(i);
            mine += units_of_seq(info, a.cut);
        }
    }
    int64_t upto = sum_upto(mine, lane);
    const Shares sh = shares_of(__shfl_sync(0xffffffffu, upto, 31), a.shares);
    if (lane == 0) shares = sh;
    const int64_t from = share_start(sh, share), left = share_start(sh, share + 1) - from;
    int at = __ffs(__ballot_sync(0xffffffffu, upto > from)) - 1, b = at;
    int64_t before = __shfl_sync(0xffffffffu, upto - mine, at & 31);
    if (each > 1 && left > 0) {               // inside the 32nd, 32 sequences at a time
        const int stop = at * each + each < a.seqs.B ? at * each + each : a.seqs.B;
#pragma unroll 1
        for (b = at * each; b < stop; b += 32) {
            info = b + lane < stop ? look(b + lane) : SeqInfo{0, 0, 0};
            mine = units_of_seq(info, a.cut);
            upto = before + sum_upto(mine, lane);
            const uint32_t beyond = __ballot_sync(0xffffffffu, upto > from);
            if (beyond) {
                at = __ffs(beyond) - 1;
                before = __shfl_sync(0xffffffffu, upto - mine, at);
                b += at;
                break;
            }
            before = __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    info.begin = __shfl_sync(0xffffffffu, info.begin, at & 31);
    info.tokens = __shfl_sync(0xffffffffu, info.tokens, at & 31);
    info.before = __shfl_sync(0xffffffffu, info.before, at & 31);
    if (lane == 0) {
        p.w.left = 0;
        if (left > 0) {
            p.b = b;
            p.info = info;
            p.at = from;
            walk_enter(p.w, info, a.cut, from - before, left);
        }
    }
    __syncwarp();
}

// Reports lengths and offsets that had to be cut to what the arrays hold: every
// share's warp looks at some of them when it has nothing else to do.
__device__ inline void check_sequences(const AttendArgs& a, int share, int lane) {
    bool bad = share == 0 && lane == 0 && a.seqs.cu && (a.seqs.cu[0] != 0 || a.seqs.cu[a.seqs.B] != a.seqs.T);
#pragma unroll 1
    for (int i = share * 32 + lane; i < a.seqs.B; i += a.shares * 32) bad = bad || span_of(a.seqs, i).bad;
    if (bad) atomicOr(&g_device_status, kIndexError);
}

// mbar_wait for loops that have to fit the instruction cache: a few
// instructions.  A wait that gives up only sets `abort`; report_abort tells the
// host at the kernel's end.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
    const uint32_t at = smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < kSpinLimit; ++i) {
        if (mbar_try_wait(at, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    return false;
}
__device__ __forceinline__ void report_abort(volatile int* abort) {
    if (*abort) atomicOr(&g_device_status, kDeviceTimeout);
}

// The barrier of the whole block; unlike __syncthreads, it may be met in
// different places of the code.
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 0;" ::: "memory"); }

// Row r of a segment's tile: its place in out and lse.
__device__ __forceinline__ int64_t place_of(const AttendArgs& a, const Segment& s, int r) {
    int token, in_group;
    row_of(s, a.cut, r, token, in_group);
    return (int64_t)token * (a.cut.heads * a.cut.group) + s.head * a.cut.group + in_group;
}

// The logit (in powers of two) that has a weight of one: kLift below the maximum
// m, or less where fp32's steps are larger, but never more, as weights have to
// stay within f16.
__device__ __forceinline__ float zero_of(float m) { return m == -INFINITY ? 0.0f : __fadd_ru(m, -kLift); }

// The logarithm, in powers of two, of the numerators' sum: the maximum m and
// the sum l of 2^(logit - zero_of(m)).  m comes in last, so that a small result
// is not rounded in steps of the lift's size.
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.0f ? -INFINITY : m + (lg2(l * exp2f(-kLift)) + (kLift - (m - zero_of(m))));
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
