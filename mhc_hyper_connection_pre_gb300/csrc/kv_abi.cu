// kv_abi.cu -- the C entry points of the paged 8-bit key/value cache (declared
// in include/mhc_kv.h): host-side argument checks and the launches.
#include "../../include/mhc_kv.h"

#include <cuda_runtime.h>

#include <algorithm>

#include "kv_index.cuh"
#include "kv_pages.cuh"

namespace mhc {
int kv_num_sms();                     // of the current device, 0 on error (mhc_abi.cu)
namespace kv {
cudaError_t launch_kv_append(const Seqs& seqs, uint8_t* k_code, uint8_t* v_code, float* k_scale, float* v_scale,
                             int heads, int head_dim, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                             int64_t v_stride, const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                             int64_t q_out_stride, const uint16_t* q_norm, int64_t q_norm_stride,
                             const uint16_t* k_norm, int64_t k_norm_stride, float norm_eps, const float* cos,
                             const float* sin, int rope_rows, int R, int interleaved, cudaStream_t stream);
cudaError_t launch_kv_attend(const Seqs& seqs, const uint8_t* k, const uint8_t* v, const float* k_scale,
                             const float* v_scale, int heads, int head_dim, const uint16_t* q, int64_t q_stride,
                             int q_heads, float softmax_scale, int window, int sinks, uint16_t* out, float* lse,
                             void* workspace, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_fork(const mhc_kv_cache* caches, int num_caches, const ForkIn& a, void* workspace, int num_sms,
                           cudaStream_t stream);
cudaError_t launch_kv_compact(const mhc_kv_cache* caches, int num_caches, const PagesIn& p, int32_t* top, void* workspace,
                              int num_sms, cudaStream_t stream);
size_t kv_fork_workspace(int64_t num_pages, int64_t width, int64_t B);
size_t kv_compact_workspace(int64_t num_pages, int64_t B);
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

// The least epsilon of a norm: squares that fp32 loses are far below it.
constexpr float kLeastEps = 1e-20f;

bool norm_ok(const uint16_t* w, int64_t stride, int head_dim) {
    return aligned(w, 16) && (stride == 0 || (stride >= head_dim && stride % 8 == 0 && stride < ((int64_t)1 << 31)));
}

Rows norm_rows(const uint16_t* w, int64_t stride, int heads, int head_dim) {
    return Rows{w, stride ? heads : 1, head_dim * 2, stride ? stride * 2 : head_dim * 2};
}

Seqs seqs_of(const mhc_kv_cache* c, const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
             const int32_t* cu_q, int64_t B, int64_t T) {
    int log2 = 4;                                        // page_tokens is a power of two from 16 on (check_common)
    while ((1 << log2) < c->page_tokens) ++log2;
    return Seqs{block_table, seq_lens, cu_q, (int)table_width, (int)B, (int)T, log2, (int)c->num_pages};
}

// The bytes of an array that a call writes (out) or reads.
struct Extent {
    uintptr_t begin, end;
    bool out;
};

constexpr int kMaxCaches = 512;

// Caches that share page numbers, and the calls' other arrays: n filled of all, which has 4 * kMaxCaches more places.
// Whether an array that is written overlaps another one.
bool overlap(const mhc_kv_cache* caches, int num_caches, Extent* all, int n) {
    for (int i = 0; i < num_caches; ++i) {
        const mhc_kv_cache& c = caches[i];
        const int64_t scales = c.num_pages * c.heads * 4, codes = c.num_pages * c.heads * c.page_tokens * c.head_dim;
        for (const void* p : {(const void*)c.k, (const void*)c.v}) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            all[n++] = Extent{at, at + (uintptr_t)codes, true};
        }
        for (const void* p : {(const void*)c.k_scale, (const void*)c.v_scale}) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            all[n++] = Extent{at, at + (uintptr_t)scales, true};
        }
    }
    std::sort(all, all + n, [](const Extent& a, const Extent& b) { return a.begin < b.begin; });
    uintptr_t written = 0, read = 0;                     // up to where arrays before this one reach
    for (int i = 0; i < n; ++i) {
        if (all[i].begin == all[i].end) continue;
        if (all[i].begin < written || (all[i].out && all[i].begin < read)) return true;
        (all[i].out ? written : read) = std::max(all[i].out ? written : read, all[i].end);
    }
    return false;
}

Extent extent(const void* p, int64_t bytes, bool out) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return Extent{at, p ? at + (uintptr_t)bytes : at, out};
}

bool pages_sizes_ok(int64_t num_pages, int64_t width, int64_t B) {
    return num_pages >= 1 && width >= 1 && B >= 0 && num_pages <= kMaxTokens && width <= kMaxTokens && B <= kMaxTokens &&
           B * (width + 1) < kMaxTokens;
}

// What mhc_kv_fork and mhc_kv_compact share of their checks.
mhc_status check_pages(const mhc_kv_cache* caches, int num_caches, const int32_t* block_table, int64_t table_width,
                       const int32_t* seq_lens, int64_t B_in, int64_t B, const uint8_t* held, const int32_t* table_out) {
    if (!caches || num_caches < 1 || B_in < 0 || B < 0) return MHC_ERR_INVALID_ARGUMENT;
    if (num_caches > kMaxCaches) return MHC_ERR_UNSUPPORTED;
    int64_t heads = 0;
    for (int i = 0; i < num_caches; ++i) {
        const mhc_status st = check_common(caches + i, table_width, 0, 0, nullptr);
        if (st != MHC_OK) return st;
        if (caches[i].num_pages != caches[0].num_pages || caches[i].page_tokens != caches[0].page_tokens)
            return MHC_ERR_INVALID_ARGUMENT;
        heads += caches[i].heads;
    }
    if (heads >= 1 << 28 || !pages_sizes_ok(caches[0].num_pages, table_width, B) ||
        !pages_sizes_ok(caches[0].num_pages, table_width, B_in))
        return MHC_ERR_UNSUPPORTED;
    if (B == 0) return MHC_OK;
    for (int i = 0; i < num_caches; ++i) {
        for (const void* p : {(const void*)caches[i].k, (const void*)caches[i].v})
            if (!p || !aligned(p, 16)) return MHC_ERR_INVALID_ARGUMENT;
        for (const void* p : {(const void*)caches[i].k_scale, (const void*)caches[i].v_scale})
            if (!p || !aligned(p, 4)) return MHC_ERR_INVALID_ARGUMENT;
    }
    for (const void* p : {(const void*)block_table, (const void*)seq_lens})
        if ((B_in > 0 && !p) || !aligned(p, 4)) return MHC_ERR_INVALID_ARGUMENT;
    if (!aligned(held, 4) || !table_out || !aligned(table_out, 4)) return MHC_ERR_INVALID_ARGUMENT;
    return MHC_OK;
}

mhc::kv::PagesIn pages_of(const mhc_kv_cache* c, const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                          int64_t B_in, int64_t B, const uint8_t* held, int32_t* table_out) {
    int log2 = 4;
    while ((1 << log2) < c->page_tokens) ++log2;
    return mhc::kv::PagesIn{block_table, seq_lens, held, table_out, (int)table_width, (int)B_in, (int)B, log2,
                            (int)c->num_pages};
}

// Both attention calls; window 0: none.
mhc_status attend(const mhc_kv_cache* cache, const uint16_t* q, int64_t q_stride, int q_heads,
                  const int32_t* block_table, int64_t table_width, const int32_t* seq_lens, const int32_t* cu_q,
                  int64_t B, int64_t T, float softmax_scale, int64_t window, int64_t sinks, uint16_t* out, float* lse,
                  void* workspace, size_t workspace_bytes, void* stream);

}  // namespace

extern "C" {

mhc_status mhc_kv_append_norm(const mhc_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                              int64_t q_out_stride, const uint16_t* q_norm, int64_t q_norm_stride,
                              const uint16_t* k_norm, int64_t k_norm_stride, float norm_eps, const float* cos,
                              const float* sin, int64_t rope_rows, int rotary_dim, int interleaved,
                              const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                              const int32_t* cu_q, int64_t B, int64_t T, void* stream) {
    mhc_status st = check_common(cache, table_width, B, T, cu_q);
    if (st != MHC_OK) return st;
    if (rotary_dim < 0 || (!cos) != (!sin) || rope_rows < 0 || (q && q_heads < 1) || (!q) != (!q_out))
        return MHC_ERR_INVALID_ARGUMENT;
    if ((q_norm || k_norm) && !(norm_eps >= kLeastEps && norm_eps <= 3.0e38f)) return MHC_ERR_INVALID_ARGUMENT;
    if (rotary_dim > cache->head_dim || rotary_dim % 16 != 0 || rope_rows > kMaxTokens) return MHC_ERR_UNSUPPORTED;
    if (T == 0) return MHC_OK;                           // an array of no queries may be a null pointer
    if (q_norm && !q) return MHC_ERR_INVALID_ARGUMENT;
    st = check_arrays(cache, block_table, seq_lens, cu_q);
    if (st != MHC_OK) return st;
    const int64_t row = (int64_t)cache->heads * cache->head_dim;
    if (!rows_ok(k, k_stride, row) || !rows_ok(v, v_stride, row)) return MHC_ERR_INVALID_ARGUMENT;
    const int64_t q_row = q ? (int64_t)q_heads * cache->head_dim : 0;
    if (q && (!rows_ok(q, q_stride, q_row) || !rows_ok(q_out, q_out_stride, q_row))) return MHC_ERR_INVALID_ARGUMENT;
    if ((q_norm && !norm_ok(q_norm, q_norm_stride, cache->head_dim)) ||
        (k_norm && !norm_ok(k_norm, k_norm_stride, cache->head_dim)))
        return MHC_ERR_INVALID_ARGUMENT;
    const bool turn = cos && rotary_dim > 0;
    if (turn && (!aligned(cos, 16) || !aligned(sin, 16))) return MHC_ERR_INVALID_ARGUMENT;
    const int64_t codes = cache->num_pages * row * cache->page_tokens, scales = cache->num_pages * cache->heads * 4;
    const Rows outs[] = {dense(cache->k, codes), dense(cache->v, codes), dense(cache->k_scale, scales),
                         dense(cache->v_scale, scales), {q_out, T, q_row * 2, q_out_stride * 2}};
    const int64_t table = turn ? rope_rows * (rotary_dim / 2) * 4 : 0;
    const Rows ins[] = {{q, T, q_row * 2, q_stride * 2}, {k, T, row * 2, k_stride * 2}, {v, T, row * 2, v_stride * 2},
                        dense(cos, table), dense(sin, table), dense(block_table, B * table_width * 4),
                        dense(seq_lens, B * 4), dense(cu_q, (B + 1) * 4),
                        norm_rows(q_norm, q_norm_stride, q_heads, cache->head_dim),
                        norm_rows(k_norm, k_norm_stride, cache->heads, cache->head_dim)};
    for (const Rows& o : outs) {
        for (const Rows& i : ins) {
            const bool in_place = &o == outs + 4 && &i == ins && q == q_out && q_stride == q_out_stride;
            if (!in_place && meet(o, i)) return MHC_ERR_INVALID_ARGUMENT;
        }
        for (const Rows& o2 : outs)
            if (&o != &o2 && meet(o, o2)) return MHC_ERR_INVALID_ARGUMENT;
    }
    if (mhc::kv_num_sms() <= 0) return MHC_ERR_CUDA;
    const cudaError_t e = mhc::kv::launch_kv_append(
        seqs_of(cache, block_table, table_width, seq_lens, cu_q, B, T), cache->k, cache->v, cache->k_scale,
        cache->v_scale, cache->heads, cache->head_dim, k, k_stride, v, v_stride, q, q_stride, q ? q_heads : 0, q_out,
        q_out_stride, q_norm, q_norm_stride, k_norm, k_norm_stride, norm_eps, cos, sin, (int)rope_rows,
        turn ? rotary_dim : 0, interleaved ? 1 : 0, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

mhc_status mhc_kv_append(const mhc_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                         int64_t q_out_stride, const float* cos, const float* sin, int64_t rope_rows, int rotary_dim,
                         int interleaved, const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                         const int32_t* cu_q, int64_t B, int64_t T, void* stream) {
    return mhc_kv_append_norm(cache, k, k_stride, v, v_stride, q, q_stride, q_heads, q_out, q_out_stride, nullptr, 0,
                              nullptr, 0, 0.f, cos, sin, rope_rows, rotary_dim, interleaved, block_table, table_width,
                              seq_lens, cu_q, B, T, stream);
}

size_t mhc_kv_attend_workspace_bytes(const mhc_kv_cache* cache, int q_heads, int64_t B, int64_t T) {
    if (!cache || cache->heads < 1 || q_heads < 1 || q_heads % cache->heads != 0 || T <= 0 || B <= 0) return 0;
    const int sms = mhc::kv_num_sms();
    return sms > 0 ? mhc::kv::kv_attend_workspace(cache->heads, cache->head_dim, q_heads, B, T, sms) : 0;
}

mhc_status mhc_kv_attend_window(const mhc_kv_cache* cache, const uint16_t* q, int64_t q_stride, int q_heads,
                                const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                                const int32_t* cu_q, int64_t B, int64_t T, float softmax_scale, int64_t window,
                                int64_t sinks, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (window < 1 || sinks < 0) return MHC_ERR_INVALID_ARGUMENT;
    return attend(cache, q, q_stride, q_heads, block_table, table_width, seq_lens, cu_q, B, T, softmax_scale, window,
                  sinks, out, lse, workspace, workspace_bytes, stream);
}

mhc_status mhc_kv_attend(const mhc_kv_cache* cache, const uint16_t* q, int64_t q_stride, int q_heads,
                         const int32_t* block_table, int64_t table_width, const int32_t* seq_lens,
                         const int32_t* cu_q, int64_t B, int64_t T, float softmax_scale, uint16_t* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
    return attend(cache, q, q_stride, q_heads, block_table, table_width, seq_lens, cu_q, B, T, softmax_scale, 0, 0, out,
                  lse, workspace, workspace_bytes, stream);
}

size_t mhc_kv_fork_workspace_bytes(int64_t num_pages, int64_t table_width, int64_t B) {
    return pages_sizes_ok(num_pages, table_width, B) ? mhc::kv::kv_fork_workspace(num_pages, table_width, B) : 0;
}

size_t mhc_kv_compact_workspace_bytes(int64_t num_pages, int64_t B) {
    return pages_sizes_ok(num_pages, 1, B) ? mhc::kv::kv_compact_workspace(num_pages, B) : 0;
}

mhc_status mhc_kv_fork(const mhc_kv_cache* caches, int num_caches, const int32_t* block_table, int64_t table_width,
                       const int32_t* seq_lens, int64_t B_in, const int32_t* parents, int64_t B, const int32_t* room,
                       int64_t room_all, const uint8_t* held, int64_t window, int64_t sinks, int32_t* block_table_out,
                       int32_t* seq_lens_out, void* workspace, size_t workspace_bytes, void* stream) {
    mhc_status st = check_pages(caches, num_caches, block_table, table_width, seq_lens, B_in, B, held, block_table_out);
    if (st != MHC_OK) return st;
    if (room_all < 0 || window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return MHC_ERR_INVALID_ARGUMENT;
    if (B == 0) return MHC_OK;                           // an array of no parents may be a null pointer, too
    if ((!parents && B != B_in) || !aligned(parents, 4) || !aligned(room, 4) || !seq_lens_out || !aligned(seq_lens_out, 4))
        return MHC_ERR_INVALID_ARGUMENT;
    const size_t need = mhc::kv::kv_fork_workspace(caches->num_pages, table_width, B);
    if (workspace_bytes < need || !workspace || !aligned(workspace, 256)) return MHC_ERR_INVALID_ARGUMENT;
    Extent all[9 + 4 * kMaxCaches];
    int n = 0;
    if (parents || block_table_out != block_table) all[n++] = extent(block_table, B_in * table_width * 4, false);
    if (parents || seq_lens_out != seq_lens) all[n++] = extent(seq_lens, B_in * 4, false);
    all[n++] = extent(parents, B * 4, false);
    all[n++] = extent(room, B * 4, false);
    all[n++] = extent(held, caches->num_pages, false);
    all[n++] = extent(block_table_out, B * table_width * 4, true);
    all[n++] = extent(seq_lens_out, B * 4, true);
    all[n++] = extent(workspace, (int64_t)need, true);
    if (overlap(caches, num_caches, all, n)) return MHC_ERR_INVALID_ARGUMENT;
    const int sms = mhc::kv_num_sms();
    if (sms <= 0) return MHC_ERR_CUDA;
    mhc::kv::ForkIn a;
    a.p = pages_of(caches, block_table, table_width, seq_lens, B_in, B, held, block_table_out);
    a.parents = parents;
    a.room = room;
    a.room_all = (int)std::min(room_all, kMaxTokens);
    a.window = (int)std::min(window, kMaxTokens);
    a.sinks = (int)std::min(sinks, kMaxTokens);
    a.lens_out = seq_lens_out;
    return mhc::kv::launch_kv_fork(caches, num_caches, a, workspace, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MHC_OK
               : MHC_ERR_CUDA;
}

mhc_status mhc_kv_compact(const mhc_kv_cache* caches, int num_caches, const int32_t* block_table, int64_t table_width,
                          const int32_t* seq_lens, int64_t B, const uint8_t* held, int32_t* block_table_out,
                          int32_t* pages, void* workspace, size_t workspace_bytes, void* stream) {
    mhc_status st = check_pages(caches, num_caches, block_table, table_width, seq_lens, B, B > 0 ? B : 1,
                                held, B ? block_table_out : pages);
    if (st != MHC_OK) return st;
    if (!pages || !aligned(pages, 4)) return MHC_ERR_INVALID_ARGUMENT;
    const size_t need = mhc::kv::kv_compact_workspace(caches->num_pages, B);
    if (workspace_bytes < need || !workspace || !aligned(workspace, 256)) return MHC_ERR_INVALID_ARGUMENT;
    Extent all[9 + 4 * kMaxCaches];
    int n = 0;
    if (block_table_out != block_table) all[n++] = extent(block_table, B * table_width * 4, false);
    all[n++] = extent(seq_lens, B * 4, false);
    all[n++] = extent(held, caches->num_pages, false);
    all[n++] = extent(block_table_out, B * table_width * 4, true);
    all[n++] = extent(pages, 4, true);
    all[n++] = extent(workspace, (int64_t)need, true);
    if (overlap(caches, num_caches, all, n)) return MHC_ERR_INVALID_ARGUMENT;
    const int sms = mhc::kv_num_sms();
    if (sms <= 0) return MHC_ERR_CUDA;
    const mhc::kv::PagesIn p = pages_of(caches, block_table, table_width, seq_lens, B, B, held, block_table_out);
    return mhc::kv::launch_kv_compact(caches, num_caches, p, pages, workspace, sms, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MHC_OK
               : MHC_ERR_CUDA;
}

}  // extern "C"

namespace {

mhc_status attend(const mhc_kv_cache* cache, const uint16_t* q, int64_t q_stride, int q_heads,
                  const int32_t* block_table, int64_t table_width, const int32_t* seq_lens, const int32_t* cu_q,
                  int64_t B, int64_t T, float softmax_scale, int64_t window, int64_t sinks, uint16_t* out, float* lse,
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
    // a window, or first tokens, of as many as the table can hold hide nothing
    const int64_t most = table_width * cache->page_tokens;
    const bool binds = window > 0 && window < most && sinks < most;
    const cudaError_t e = mhc::kv::launch_kv_attend(
        seqs_of(cache, block_table, table_width, seq_lens, cu_q, B, T), cache->k, cache->v, cache->k_scale,
        cache->v_scale, cache->heads, cache->head_dim, q, q_stride, q_heads, softmax_scale, binds ? (int)window : 0,
        binds ? (int)std::min(sinks, kMaxTokens) : 0, out, lse, workspace, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

}  // namespace
