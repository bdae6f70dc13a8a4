// kv_abi.cu -- the C entry points of the paged 8-bit key/value cache (declared
// in include/mhc_kv.h): host-side argument checks and the launches.
#include "../../include/mhc_kv.h"

#include <cuda_runtime.h>

#include <algorithm>

#include "kv_index.cuh"

namespace mhc {
int kv_num_sms();                     // of the current device, 0 on error (mhc_abi.cu)
namespace kv {
cudaError_t launch_kv_append(const Seqs& seqs, uint8_t* k_code, uint8_t* v_code, float* k_scale, float* v_scale,
                             int heads, int head_dim, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                             int64_t v_stride, const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                             int64_t q_out_stride, const float* cos, const float* sin, int rope_rows, int R,
                             int interleaved, cudaStream_t stream);
cudaError_t launch_kv_attend(const Seqs& seqs, const uint8_t* k, const uint8_t* v, const float* k_scale,
                             const float* v_scale, int heads, int head_dim, const uint16_t* q, int64_t q_stride,
                             int q_heads, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                             int num_sms, cudaStream_t stream);
size_t kv_attend_workspace(int heads, int head_dim, int q_heads, int64_t B, int64_t T, int num_sms);
}  // namespace kv
}  // namespace mhc

namespace {

using mhc::kv::Seqs;

constexpr int64_t kMaxTokens = (int64_t)1 << 30;     // of a call, and of a table row: positions stay in 32 bits

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t rows, width, stride;
};

// Whether two sets of rows share a byte.  Rows with one common stride (slices
// of one buffer) are compared column by column, others by their whole spans.
bool meet(const Rows& a, const Rows& b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const int64_t a0 = (int64_t)reinterpret_cast<uintptr_t>(a.p), b0 = (int64_t)reinterpret_cast<uintptr_t>(b.p);
    const int64_t a1 = a0 + (a.rows - 1) * a.stride + a.width, b1 = b0 + (b.rows - 1) * b.stride + b.width;
    if (a0 >= b1 || b0 >= a1) return false;
    if (a.stride != b.stride || a.rows == 1 || b.rows == 1) return true;
    const int64_t s = a.stride, d = ((b0 - a0) % s + s) % s;   // b's first column from a's
    return d < a.width || d + b.width > s;
}

Rows dense(const void* p, int64_t bytes) { return Rows{p, 1, bytes, bytes}; }

// The checks that both calls share.
mhc_status check_common(const mhc_kv_cache* c, int64_t table_width, int64_t B, int64_t T, const int32_t* cu_q) {
    if (!c || T < 0 || B < 0) return MHC_ERR_INVALID_ARGUMENT;
    if (c->heads < 1 || c->num_pages < 1 || table_width < 1 || c->page_tokens < 1 || c->head_dim < 1)
        return MHC_ERR_INVALID_ARGUMENT;
    if (c->head_dim != 64 && c->head_dim != 128) return MHC_ERR_UNSUPPORTED;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return MHC_ERR_UNSUPPORTED;
    if (c->num_pages > 0x7fffffff / c->heads || T > kMaxTokens || B > kMaxTokens ||
        table_width > kMaxTokens / c->page_tokens)
        return MHC_ERR_UNSUPPORTED;
    if (!cu_q && B != T) return MHC_ERR_INVALID_ARGUMENT;
    if (T > 0 && B == 0) return MHC_ERR_INVALID_ARGUMENT;
    return MHC_OK;
}

mhc_status check_arrays(const mhc_kv_cache* c, const int32_t* block_table, const int32_t* seq_lens,
                        const int32_t* cu_q) {
    for (const void* p : {(const void*)c->k, (const void*)c->v})
        if (!p || !aligned(p, 16)) return MHC_ERR_INVALID_ARGUMENT;
    for (const void* p : {(const void*)c->k_scale, (const void*)c->v_scale, (const void*)block_table,
                          (const void*)seq_lens})
        if (!p || !aligned(p, 4)) return MHC_ERR_INVALID_ARGUMENT;
    if (cu_q && !aligned(cu_q, 4)) return MHC_ERR_INVALID_ARGUMENT;
    return MHC_OK;
}

bool rows_ok(const void* p, int64_t stride, int64_t width) {
    return p && aligned(p, 16) && stride >= width && stride % 8 == 0 && stride < ((int64_t)1 << 31);
}

Seqs seqs_of(const mhc_kv_cache* c, const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
             const int32_t* cu_q, int64_t B, int64_t T) {
    int log2 = 4;                                        // page_tokens is a power of two from 16 on (check_common)
    while ((1 << log2) < c->page_tokens) ++log2;
    return Seqs{block_table, seq_lens, cu_q, (int)table_width, (int)B, (int)T, log2, (int)c->num_pages};
}

}  // namespace

extern "C" {

mhc_status mhc_kv_append(const mhc_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                         int64_t q_out_stride, const float* cos, const float* sin, int64_t rope_rows, int rotary_dim,
                         int interleaved, const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                         const int32_t* cu_q, int64_t B, int64_t T, void* stream) {
    mhc_status st = check_common(cache, table_width, B, T, cu_q);
    if (st != MHC_OK) return st;
    if (rotary_dim < 0 || (!cos) != (!sin) || rope_rows < 0 || (q && q_heads < 1) || (!q) != (!q_out))
        return MHC_ERR_INVALID_ARGUMENT;
    if (rotary_dim > cache->head_dim || rotary_dim % 16 != 0 || rope_rows > kMaxTokens) return MHC_ERR_UNSUPPORTED;
    if (T == 0) return MHC_OK;
    st = check_arrays(cache, block_table, seq_lens, cu_q);
    if (st != MHC_OK) return st;
    const int64_t row = (int64_t)cache->heads * cache->head_dim;
    if (!rows_ok(k, k_stride, row) || !rows_ok(v, v_stride, row)) return MHC_ERR_INVALID_ARGUMENT;
    const int64_t q_row = q ? (int64_t)q_heads * cache->head_dim : 0;
    if (q && (!rows_ok(q, q_stride, q_row) || !rows_ok(q_out, q_out_stride, q_row))) return MHC_ERR_INVALID_ARGUMENT;
    const bool turn = cos && rotary_dim > 0;
    if (turn && (!aligned(cos, 16) || !aligned(sin, 16))) return MHC_ERR_INVALID_ARGUMENT;
    const int64_t codes = cache->num_pages * row * cache->page_tokens, scales = cache->num_pages * cache->heads * 4;
    const Rows outs[] = {dense(cache->k, codes), dense(cache->v, codes), dense(cache->k_scale, scales),
                         dense(cache->v_scale, scales), {q_out, T, q_row * 2, q_out_stride * 2}};
    const int64_t table = turn ? rope_rows * (rotary_dim / 2) * 4 : 0;
    const Rows ins[] = {{k, T, row * 2, k_stride * 2}, {v, T, row * 2, v_stride * 2}, dense(cos, table),
                        dense(sin, table), dense(block_table, B * table_width * 4), dense(seq_lens, B * 4),
                        dense(cu_q, (B + 1) * 4), {q, T, q_row * 2, q_stride * 2}};
    for (const Rows& o : outs) {
        for (const Rows& i : ins) {
            const bool in_place = o.p == q_out && i.p == q && q == q_out && q_stride == q_out_stride;
            if (!in_place && meet(o, i)) return MHC_ERR_INVALID_ARGUMENT;
        }
        for (const Rows& o2 : outs)
            if (&o != &o2 && meet(o, o2)) return MHC_ERR_INVALID_ARGUMENT;
    }
    if (mhc::kv_num_sms() <= 0) return MHC_ERR_CUDA;
    const cudaError_t e = mhc::kv::launch_kv_append(
        seqs_of(cache, block_table, table_width, seq_lens, cu_q, B, T), cache->k, cache->v, cache->k_scale,
        cache->v_scale, cache->heads, cache->head_dim, k, k_stride, v, v_stride, q, q_stride, q ? q_heads : 0, q_out,
        q_out_stride, cos, sin, (int)rope_rows, turn ? rotary_dim : 0, interleaved ? 1 : 0,
        static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

size_t mhc_kv_attend_workspace_bytes(const mhc_kv_cache* cache, int q_heads, int64_t B, int64_t T) {
    if (!cache || cache->heads < 1 || q_heads < 1 || q_heads % cache->heads != 0 || T <= 0 || B <= 0) return 0;
    const int sms = mhc::kv_num_sms();
    return sms > 0 ? mhc::kv::kv_attend_workspace(cache->heads, cache->head_dim, q_heads, B, T, sms) : 0;
}

mhc_status mhc_kv_attend(const mhc_kv_cache* cache, const uint16_t* q, int64_t q_stride, int q_heads,
                         const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                         const int32_t* cu_q, int64_t B, int64_t T, float softmax_scale, uint16_t* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
    mhc_status st = check_common(cache, table_width, B, T, cu_q);
    if (st != MHC_OK) return st;
    if (q_heads < 1 || q_heads % cache->heads != 0 || !(softmax_scale >= 0.f) || softmax_scale > 3.0e38f)
        return MHC_ERR_INVALID_ARGUMENT;
    if (q_heads / cache->heads > 128) return MHC_ERR_UNSUPPORTED;
    if (T == 0) return MHC_OK;
    st = check_arrays(cache, block_table, seq_lens, cu_q);
    if (st != MHC_OK) return st;
    const int64_t row = (int64_t)q_heads * cache->head_dim;
    if (T > (((int64_t)1 << 31) - 1) / q_heads) return MHC_ERR_UNSUPPORTED;
    if (!rows_ok(q, q_stride, row) || !out || !aligned(out, 16) || (lse && !aligned(lse, 16)))
        return MHC_ERR_INVALID_ARGUMENT;
    const int64_t codes = cache->num_pages * cache->heads * cache->page_tokens * cache->head_dim;
    const int64_t scales = cache->num_pages * cache->heads * 4;
    const Rows outs[] = {dense(out, T * row * 2), dense(lse, T * (int64_t)q_heads * 4),
                         dense(workspace, (int64_t)std::min<size_t>(workspace_bytes, (size_t)1 << 62))};
    const Rows ins[] = {{q, T, row * 2, q_stride * 2}, dense(cache->k, codes), dense(cache->v, codes),
                        dense(cache->k_scale, scales), dense(cache->v_scale, scales),
                        dense(block_table, B * table_width * 4), dense(seq_lens, B * 4), dense(cu_q, (B + 1) * 4)};
    for (const Rows& o : outs) {
        for (const Rows& i : ins)
            if (meet(o, i)) return MHC_ERR_INVALID_ARGUMENT;
        for (const Rows& o2 : outs)
            if (&o != &o2 && meet(o, o2)) return MHC_ERR_INVALID_ARGUMENT;
    }
    const int sms = mhc::kv_num_sms();
    if (sms <= 0) return MHC_ERR_CUDA;
    const size_t need = mhc::kv::kv_attend_workspace(cache->heads, cache->head_dim, q_heads, B, T, sms);
    if (workspace_bytes < need || (need && (!workspace || !aligned(workspace, 256)))) return MHC_ERR_INVALID_ARGUMENT;
    const cudaError_t e = mhc::kv::launch_kv_attend(
        seqs_of(cache, block_table, table_width, seq_lens, cu_q, B, T), cache->k, cache->v, cache->k_scale,
        cache->v_scale, cache->heads, cache->head_dim, q, q_stride, q_heads, softmax_scale, out, lse, workspace, sms,
        static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

}  // extern "C"
