// kv_attend.cu -- causal attention of the new tokens over the paged e4m3
// cache (mhc_kv_attend).
//
// One warp takes one new token and query head and walks over the keys it
// sees, 32 at a time: each lane forms one key's product with the query, the
// running maximum and sum of the softmax are kept in fp32, and each lane
// collects its share of the head's dimensions over the 32 values.
#include <cuda_runtime.h>

#include "kv_common.cuh"

namespace mhc {
namespace kv {

static __device__ unsigned int g_attend_status = 0;

struct AttendArgs {
    Seqs seqs;
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int heads, group;                 // key/value heads; query heads of each
    const uint16_t* q;
    int64_t q_stride;
    float softmax_scale;
    uint16_t* out;
    float* lse;
};

template <int D>
__global__ void __launch_bounds__(128) kv_attend_rows_kernel(const AttendArgs a) {
    constexpr int kDims = D / 32;
    __shared__ float qs[4][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int q_heads = a.heads * a.group;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= (int64_t)a.seqs.T * q_heads) return;
    const int t = (int)(row / q_heads), hq = (int)(row % q_heads), h = hq / a.group;
    const int b = seq_of(a.seqs, t, lane);
    const Span sp = span_of(a.seqs, b);
    const bool in = t >= sp.begin && t < sp.end;
    if ((sp.bad || !in) && lane == 0) atomicOr(&g_attend_status, kIndexError);
    const int keys = in ? sp.before + (t - sp.begin) + 1 : 0;

    for (int i = lane; i < D; i += 32) {
        const uint32_t w = a.q[t * a.q_stride + hq * D + i];
        qs[warp][i] = bf16lo(w);
    }
    __syncwarp();
    float m = -INFINITY, l = 0.0f, o[kDims] = {};
    for (int base = 0; base < keys; base += 32) {
        const int key = base + lane;
        const int page = key < keys ? page_of(a.seqs, b, key) : -1;
        if (key < keys && page < 0) atomicOr(&g_attend_status, kIndexError);
        const int64_t block = (int64_t)page * a.heads + h;
        const int64_t at = (block * a.seqs.page_tokens + key % a.seqs.page_tokens) * D;
        float s = -INFINITY, vs = 0.0f;
        if (page >= 0) {
            float dot = 0.0f;
            for (int i = 0; i < D; i += 16) {
                const uint4 w = *reinterpret_cast<const uint4*>(a.k + at + i);
                const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t f = f16x2_of_e4m3x2((uint16_t)(word[j / 2] >> (16 * (j & 1))));
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f));
                    dot = fmaf(qs[warp][i + 2 * j], x.x, dot);
                    dot = fmaf(qs[warp][i + 2 * j + 1], x.y, dot);
                }
            }
            s = dot * a.k_scale[block] * a.softmax_scale;
            vs = a.v_scale[block];
        }
        float top = s;
#pragma unroll
        for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        top = fmaxf(top, m);
        const float zero = top == -INFINITY ? 0.0f : top;
        const float p = expf(s - zero), keep = expf(m - zero);
        float sum = p;
#pragma unroll
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        l = l * keep + sum;
        m = top;
#pragma unroll
        for (int d = 0; d < kDims; ++d) o[d] *= keep;
        for (int j = 0; j < 32 && base + j < keys; ++j) {
            const int64_t from = __shfl_sync(0xffffffffu, at, j);
            const float w = __shfl_sync(0xffffffffu, p * vs, j);
            if (__shfl_sync(0xffffffffu, page, j) < 0) continue;
            const uint8_t* v = a.v + from + lane * kDims;
#pragma unroll
            for (int d = 0; d < kDims; d += 2) {
                const uint32_t f = f16x2_of_e4m3x2(*reinterpret_cast<const uint16_t*>(v + d));
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f));
                o[d] = fmaf(w, x.x, o[d]);
                o[d + 1] = fmaf(w, x.y, o[d + 1]);
            }
        }
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < kDims; d += 2)
        *reinterpret_cast<uint32_t*>(a.out + row * D + lane * kDims + d) = pack_bf16x2(o[d] * r, o[d + 1] * r);
    if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

cudaError_t launch_kv_attend(const Seqs& seqs, const uint8_t* k, const uint8_t* v, const float* k_scale,
                             const float* v_scale, int heads, int head_dim, const uint16_t* q, int64_t q_stride,
                             int q_heads, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                             int num_sms, cudaStream_t stream) {
    const AttendArgs a{seqs, k, v, k_scale, v_scale, heads, q_heads / heads, q, q_stride, softmax_scale, out, lse};
    const int64_t blocks = ((int64_t)seqs.T * q_heads + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (head_dim == 64) kv_attend_rows_kernel<64><<<(unsigned)blocks, 128, 0, stream>>>(a);
    else kv_attend_rows_kernel<128><<<(unsigned)blocks, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

size_t kv_attend_workspace(int heads, int head_dim, int q_heads, int64_t B, int64_t T, int num_sms) { return 0; }

cudaError_t read_attend_status(unsigned int* status) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attend_status, sizeof v);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_attend_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace kv
}  // namespace mhc
