// kv_append.cu -- rotation of the new tokens' queries and keys, and the write
// of keys and values into the paged e4m3 cache (mhc_kv_append).
//
// What bounds it: each input number is read once and each output written
// once, a few operations a number, so memory for long prompts and the launch
// with its chain of dependent loads (sequence, length, page, scale) for a
// decode step.  The work of one page, head and tensor (k or v) belongs to one
// group of threads, because the scale needs the largest magnitude of all of
// the page's new numbers before the first of them can be rounded.  The group
// reads its numbers twice, the second time from the L1 cache: held in registers
// between the passes they left half as many threads on an SM, and the loads of
// a long prompt took 1.5 times as long.  16384 tokens of 40 query and 8 key
// heads take 82 us: 445 MB at 5.4 TB/s (the queries alone 6.0 TB/s).  The forms
// for many tokens that rotate spill 56 to 84 bytes a thread at the 64 registers
// of four blocks an SM: cos, sin and both numbers of eight pairs are alive at once
// beside the next step's loads.
#include <cuda_runtime.h>

#include "kv_common.cuh"

namespace mhc {
namespace kv {

static __device__ unsigned int g_append_status = 0;

struct AppendArgs {
    Seqs seqs;
    uint8_t* code[2];                 // k, v
    float* scale[2];
    const uint16_t* x[2];
    int64_t x_stride[2];
    int heads;
    const uint16_t* q;
    uint16_t* q_out;
    int64_t q_stride, q_out_stride;
    int q_heads;
    const float* cos;
    const float* sin;
    int rope_rows, R;                 // R == 0: no rotation
    int window;                       // tokens whose runs one group takes
    int windows;                      // ceil(T / window)
    int kv_blocks;                    // blocks [0, kv_blocks) append, the rest rotate q
    int q_steps;                      // head steps of one warp in the q part
};

enum Mode { kPlain, kHalves, kPairs };        // no rotation; pairs (i, i + R/2); pairs (2i, 2i + 1)

// A thread takes 16 numbers of a head: two chunks of 8 that hold both numbers
// of its pairs, so that nothing is exchanged between threads and each cos and
// sin is loaded once.  Thread p of a head's D/16 turns pairs 8p .. 8p + 7 if the
// rotation has so many.
struct Chunks {
    int a, b;                                 // first numbers of the two chunks
    bool turned;
};

template <int kMode>
__device__ __forceinline__ Chunks chunks_of(int R, int p) {
    const bool turned = kMode != kPlain && 16 * p < R;
    if (kMode == kHalves && turned) return Chunks{8 * p, 8 * p + R / 2, true};
    return Chunks{16 * p, 16 * p + 8, turned};        // with halves: what is left after the rotated numbers
}

struct Raw {                                  // the 16 numbers as stored
    uint4 a, b;
};

struct Turn {                                 // cos and sin of the eight pairs
    float c[8], s[8];
};

__device__ __forceinline__ void load_turn(const AppendArgs& a, int pos, int p, Turn& w) {
    const size_t at = (size_t)pos * (a.R / 2) + 8 * p;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(a.cos + at + j));
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.sin + at + j));
        w.c[j] = u.x; w.c[j + 1] = u.y; w.c[j + 2] = u.z; w.c[j + 3] = u.w;
        w.s[j] = v.x; w.s[j + 1] = v.y; w.s[j + 2] = v.z; w.s[j + 3] = v.w;
    }
}

// Every product and sum is rounded to fp32 (no fused multiply-add), as the
// header states it: the result does not depend on who computes it.
template <int kMode>
__device__ __forceinline__ void rotate(const Turn& w, float (&x)[8], float (&y)[8]) {
    auto turn = [](float& u, float& v, float c, float s) {
        const float p = u, q = v;
        u = __fsub_rn(__fmul_rn(p, c), __fmul_rn(q, s));
        v = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p, s));
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (kMode == kHalves) turn(x[j], y[j], w.c[j], w.s[j]);
        else if (j < 4) turn(x[2 * j], x[2 * j + 1], w.c[j], w.s[j]);
        else turn(y[2 * j - 8], y[2 * j - 7], w.c[j], w.s[j]);
    }
}

// The smallest power of two 2^e with a <= 448 * 2^e = 1.75 * 2^(8+e), e at
// least -116 (so that the smallest step, 2^-9 * 2^e, is a normal fp32
// number).  a is finite.
__device__ __forceinline__ float scale_for(float a) {
    const uint32_t u = __float_as_uint(a);
    int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -116 ? -116 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

template <int GT>
__device__ __forceinline__ void group_sync(int group) {
    if constexpr (GT > 32) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(GT) : "memory");
    else __syncwarp();
}

// Largest of the group's values, for all of its threads; a barrier of the group.
template <int GT>
__device__ __forceinline__ float group_max(float v, int group, float* red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (GT > 32) {
        constexpr int W = GT / 32;
        const int w = (threadIdx.x % GT) / 32;
        group_sync<GT>(group);        // the last call's readers are done
        if (threadIdx.x % 32 == 0) red[group * W + w] = v;
        group_sync<GT>(group);
        v = red[group * W];
#pragma unroll
        for (int i = 1; i < W; ++i) v = fmaxf(v, red[group * W + i]);
    } else {
        __syncwarp();
    }
    return v;
}

// GT threads take one (window, head, k or v), the loads of kAhead steps under
// way together.
template <int D, int GT, int kMode, int kAhead>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const AppendArgs a) {
    constexpr int kBlock = 256, kGroups = kBlock / GT;
    constexpr int kLanes = D / 16, kRows = GT / kLanes;               // threads of a head; rows of one step
    __shared__ float red[kBlock / 32];
    const int lane = threadIdx.x % 32;
    const Chunks at = chunks_of<kMode>(a.R, lane % kLanes);
    auto load = [&](const uint16_t* head) {
        return Raw{*reinterpret_cast<const uint4*>(head + at.a), *reinterpret_cast<const uint4*>(head + at.b)};
    };
    const uint4 none = make_uint4(0, 0, 0, 0);

    if ((int)blockIdx.x >= a.kv_blocks) {             // queries: a warp takes one token and some of its heads
        constexpr int kHeads = 32 / kLanes;           // heads of one step
        const int steps = (a.q_heads + kHeads - 1) / kHeads;
        const uint32_t parts = (steps + a.q_steps - 1) / a.q_steps;
        const uint32_t w = (blockIdx.x - a.kv_blocks) * (kBlock / 32) + threadIdx.x / 32;
        const int t = (int)(w / parts), part = (int)(w % parts);
        if (t >= a.seqs.T) return;
        const int first = part * a.q_steps * kHeads;
        const int end = a.q_heads < first + a.q_steps * kHeads ? a.q_heads : first + a.q_steps * kHeads;
        const uint16_t* src = a.q + t * a.q_stride;
        uint16_t* dst = a.q_out + t * a.q_out_stride;
        auto fetch = [&](int h) { return h < end ? load(src + h * D) : Raw{none, none}; };
        int h = first + lane / kLanes;
        Raw raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = fetch(h + i * kHeads);      // these loads do not wait for the position
        const int b = seq_of(a.seqs, t, lane);
        const int pos = pos_of(span_of(a.seqs, b), t);
        const bool turned = at.turned && pos >= 0 && pos < a.rope_rows;       // beyond: reported by the append part
        Turn turn;
        if (turned) load_turn(a, pos, lane % kLanes, turn);
#pragma unroll 1
        for (int base = first; base < end; base += kAhead * kHeads) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (turned) {
                    float x[8], y[8];
                    unpack8(raw[i].a, x);
                    unpack8(raw[i].b, y);
                    rotate<kMode>(turn, x, y);
                    raw[i] = Raw{pack8(x), pack8(y)};
                }
                if (h < end) {
                    *reinterpret_cast<uint4*>(dst + h * D + at.a) = raw[i].a;
                    *reinterpret_cast<uint4*>(dst + h * D + at.b) = raw[i].b;
                }
                raw[i] = fetch(h + kAhead * kHeads);
                h += kHeads;
            }
        }
        return;
    }

    const int group = threadIdx.x / GT, id = threadIdx.x % GT;
    const uint32_t item = blockIdx.x * kGroups + group, pair = item / a.heads;
    const int head = (int)(item % a.heads), kv = (int)(pair & 1), win = (int)(pair >> 1);
    if (win >= a.windows) return;
    const int64_t next = (int64_t)(win + 1) * a.window;
    const int t1 = (int)(next < a.seqs.T ? next : a.seqs.T);
    const int r0 = id / kLanes;
    const uint16_t* src = a.x[kv] + head * D;
    // the other offsets are looked at by the tokens that they are those of
    if (item == 0 && id == 0 && a.seqs.cu && (a.seqs.cu[0] != 0 || a.seqs.cu[a.seqs.B] != a.seqs.T))
        atomicOr(&g_append_status, kIndexError);

#pragma unroll 1
    for (int t = win * a.window; t < t1;) {
        const int b = seq_of(a.seqs, t, lane);
        const Span sp = span_of(a.seqs, b);
        if (sp.bad && id == 0) atomicOr(&g_append_status, kIndexError);
        if (t < sp.begin || t >= sp.end) {            // cu_q out of order
            if (id == 0) atomicOr(&g_append_status, kIndexError);
            ++t;
            continue;
        }
        const Run run = run_at(a.seqs, sp, t);
        const int t0 = t;
        t = run.next;
        if (!starts_run(sp, run, t0)) continue;
        int n = run.n;
        if (kMode != kPlain) {                        // positions beyond the tables: k and v are left out alike
            const int rows = a.rope_rows - run.pos;
            if (rows < n) n = rows < 0 ? 0 : rows;
        }
        Raw raw[kAhead];
        auto fetch_all = [&](int r) {                 // rows past the run: zeros
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                raw[i] = r + i * kRows < n ? load(src + (int64_t)(t0 + r + i * kRows) * a.x_stride[kv]) : Raw{none, none};
        };
        // f(r, the 16 numbers of row r) for every row of this thread.  The first rows are in `raw`.
        auto each = [&](auto&& f) {
#pragma unroll 1
            for (int base = 0; base < n; base += kAhead * kRows) {
                if (base) fetch_all(base + r0);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int r = base + i * kRows + r0;
                    if (r >= n) break;
                    float x[8], y[8];
                    unpack8(raw[i].a, x);
                    unpack8(raw[i].b, y);
                    if (kMode != kPlain && kv == 0 && at.turned) {
                        Turn turn;
                        load_turn(a, run.pos + r, lane % kLanes, turn);
                        rotate<kMode>(turn, x, y);
                    }
                    f(r, x, y);
                }
            }
        };
        fetch_all(r0);                                // under way before the page, and its scale, are known
        const int page = page_of(a.seqs, b, run.pos);
        if ((page < 0 || n < run.n) && id == 0) atomicOr(&g_append_status, kIndexError);
        if (page < 0 || n == 0) continue;

        float* scale_at = a.scale[kv] + (int64_t)page * a.heads + head;
        uint8_t* code = a.code[kv] + (((int64_t)page * a.heads + head) * D << a.seqs.page_log2);
        const float old = run.slot ? *scale_at : 0.0f;
        float top = 0.0f;
        each([&](int, const float(&x)[8], const float(&y)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                top = finite(x[j]) ? fmaxf(top, fabsf(x[j])) : top;
                top = finite(y[j]) ? fmaxf(top, fabsf(y[j])) : top;
            }
        });
        top = group_max<GT>(top, group, red);
        const float need = scale_for(top), scale = run.slot ? fmaxf(old, need) : need;
        const float per = 1.0f / scale;               // scales are powers of two: x * per is x / scale
        if (id == 0) *scale_at = scale;               // every thread has read it: group_max was a barrier
        if (n > kAhead * kRows) fetch_all(r0);
        each([&](int r, float(&x)[8], float(&y)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = finite(x[j]) ? x[j] * per : __int_as_float(0x7fc00000);
                y[j] = finite(y[j]) ? y[j] * per : __int_as_float(0x7fc00000);
            }
            uint8_t* to = code + (run.slot + r) * D;
            *reinterpret_cast<uint2*>(to + at.a) = make_uint2(e4m3x4(x, 0), e4m3x4(x, 4));
            *reinterpret_cast<uint2*>(to + at.b) = make_uint2(e4m3x4(y, 0), e4m3x4(y, 4));
        });
        if (run.slot && scale != old) {               // the scale grew: round the page's earlier slots once more
            const float by = old / scale;
#pragma unroll 1
            for (int i = id; i < run.slot * (D / 8); i += GT) {
                uint2* old_at = reinterpret_cast<uint2*>(code) + i;
                const uint2 v = *old_at;
                float y[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t h = f16x2_of_e4m3x2((uint16_t)((j < 2 ? v.x : v.y) >> (16 * (j & 1))));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    y[2 * j] = f.x * by;
                    y[2 * j + 1] = f.y * by;
                }
                *old_at = make_uint2(e4m3x4(y, 0), e4m3x4(y, 4));
            }
        }
    }
}

template <int D, int GT, int kMode, int kAhead>
static cudaError_t launch_mode(AppendArgs& a, cudaStream_t stream) {
    constexpr int kBlock = 256;
    const int64_t items = (int64_t)a.windows * a.heads * 2;
    const int64_t kv_blocks = (items + kBlock / GT - 1) / (kBlock / GT);
    int64_t q_blocks = 0;
    if (a.q) {
        const int heads = 32 / (D / 16), steps = (a.q_heads + heads - 1) / heads;
        const int64_t warps = (int64_t)a.seqs.T * ((steps + a.q_steps - 1) / a.q_steps);
        if (warps > 0x7fffffff) return cudaErrorInvalidValue;
        q_blocks = (warps + kBlock / 32 - 1) / (kBlock / 32);
    }
    if (items > 0x7fffffff || kv_blocks + q_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    a.kv_blocks = (int)kv_blocks;
    kv_append_kernel<D, GT, kMode, kAhead><<<(unsigned)(kv_blocks + q_blocks), kBlock, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D, int GT, int kAhead>
static cudaError_t launch_append(AppendArgs& a, int interleaved, cudaStream_t stream) {
    if (a.R == 0) return launch_mode<D, GT, kPlain, kAhead>(a, stream);
    return interleaved ? launch_mode<D, GT, kPairs, kAhead>(a, stream) : launch_mode<D, GT, kHalves, kAhead>(a, stream);
}

cudaError_t launch_kv_append(const Seqs& seqs, uint8_t* k_code, uint8_t* v_code, float* k_scale, float* v_scale,
                             int heads, int head_dim, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                             int64_t v_stride, const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                             int64_t q_out_stride, const float* cos, const float* sin, int rope_rows, int R,
                             int interleaved, cudaStream_t stream) {
    AppendArgs a;
    a.seqs = seqs;
    a.code[0] = k_code; a.code[1] = v_code;
    a.scale[0] = k_scale; a.scale[1] = v_scale;
    a.x[0] = k; a.x[1] = v;
    a.x_stride[0] = k_stride; a.x_stride[1] = v_stride;
    a.heads = heads;
    a.q = q; a.q_out = q_out;
    a.q_stride = q_stride; a.q_out_stride = q_out_stride;
    a.q_heads = q_heads;
    a.cos = cos; a.sin = sin;
    a.rope_rows = rope_rows; a.R = R;
    // Few new tokens a sequence on average: a warp for each token that may start a
    // run.  Many: one to four warps for each window of as many tokens as a page
    // has.  Like tile_rows for attend, this takes the sequences to be alike: a
    // window of single tokens is as many runs one after the other.  A prompt of
    // 2048 tokens beside 127 single ones takes 118 us (40 / 8 heads of 128; 14.5 and
    // 3.7 in calls of their own), one of 1000 beside 255, a warp a page, 27.5
    // (11.4 and 5.0).
    const bool few = seqs.T < 8 * (int64_t)seqs.B;
    a.window = few ? 1 : 1 << seqs.page_log2;
    a.windows = (seqs.T + a.window - 1) / a.window;
    // With few tokens a warp takes one step of a token's heads, else all of
    // them, so that the position is found and its row of cos and sin read once.
    a.q_steps = seqs.T < 2048 ? 1 : 1 << 20;
    if (few)
        return head_dim == 64 ? launch_append<64, 32, 1>(a, interleaved, stream)
                              : launch_append<128, 32, 1>(a, interleaved, stream);
    switch ((head_dim << seqs.page_log2) / 128) {     // a page is 8 steps of its group, or fewer
        case 128: return launch_append<128, 128, 2>(a, interleaved, stream);
        case 64: return head_dim == 64 ? launch_append<64, 64, 2>(a, interleaved, stream)
                                       : launch_append<128, 64, 2>(a, interleaved, stream);
        default: return head_dim == 64 ? launch_append<64, 32, 2>(a, interleaved, stream)
                                       : launch_append<128, 32, 2>(a, interleaved, stream);
    }
}

cudaError_t read_append_status(unsigned int* status) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_status, sizeof v);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_append_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace kv
}  // namespace mhc
