// kv_pages.cu -- the pages of the next step (mhc_kv_fork) and moving the pages in
// use to the lowest numbers (mhc_kv_compact): one block plans (kv_pages.cuh), a further
// launch copies; the rows of large tables are all SMs' work before that.
//
// What bounds it: planning reads and writes the tables once, a few hundred KB at
// most; its time is a chain of dependent loads (parent, length, entry), of barriers,
// and one block's instructions.  A cluster of eight blocks that met in global memory was slower
// at every size: 256 rows of 47 entries 22.5 us when one block took 15.4 (12.3 since); 2048 rows of 128 169 and 90.
// Copying is memory: every byte of the copied slots is read and written once, 16 bytes a lane,
// by warps that take one page, head and tensor of one layer at a time.
#include "../../include/mhc_kv.h"

#include <cuda_runtime.h>

#include <algorithm>

#include "kv_common.cuh"
#include "kv_pages.cuh"
#include "sm100.cuh"

namespace mhc {
namespace kv {

static __device__ unsigned int g_pages_status = 0;

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;    // of the block that plans
constexpr int kRowThreads = 256;              // of a block that takes rows of large tables

// Caches that one launch copies: the layers that share page numbers.
constexpr int kMaxSet = 64;
struct CacheSet {
    uint8_t* code[kMaxSet][2];                // k, v
    float* scale[kMaxSet][2];
    int heads[kMaxSet], dim[kMaxSet];
    int first[kMaxSet + 1];                   // of a page's pieces those of cache i begin here, k's and then as many of v
    int count;
};

struct TeamScratch {
    int64_t sums[kWarps];
    int64_t all;
};

// The threads of the one block that plans.  kOwn: the pages' bits are in shared memory for certain.
template <bool kOwn>
struct BlockTeam {
    int rank, size;
    TeamScratch* scratch;
    bool own_bits;                            // they are

    __device__ __forceinline__ void sync() const { __syncthreads(); }
    __device__ __forceinline__ int64_t scan(int64_t x, int64_t& total) const {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        int64_t upto = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += up;
        }
        if (lane == 31) scratch->sums[warp] = upto;
        __syncthreads();
        if (warp == 0) {
            const int64_t own = scratch->sums[lane];
            int64_t y = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += up;
            }
            scratch->sums[lane] = y - own;
            if (lane == 31) scratch->all = y;
        }
        __syncthreads();
        const int64_t before = scratch->sums[warp] + upto - x;
        total = scratch->all;
        __syncthreads();
        return before;
    }
    template <class T>
    __device__ __forceinline__ T load(const T* p) const {
        return *const_cast<const volatile T*>(p);
    }
    __device__ __forceinline__ void store(int32_t* p, int32_t x) const { *const_cast<volatile int32_t*>(p) = x; }
    __device__ __forceinline__ void set_bit(uint32_t* bits, int page) const {
        if (kOwn || own_bits)
            asm volatile("{ .reg .pred p; setp.ge.s32 p, %2, 0; @p red.shared.or.b32 [%0], %1; }" ::"r"(
                             smem_u32(bits) + (page >> 5) * 4),
                         "r"(1u << (page & 31)), "r"(page)
                         : "memory");
        else if (page >= 0) atomicOr(bits + (page >> 5), 1u << (page & 31));
    }
    __device__ __forceinline__ void lower(int32_t* p, int32_t x) const { atomicMin(p, x); }
    __device__ __forceinline__ void raise(int32_t* p, int32_t x) const { atomicMax(p, x); }
    __device__ __forceinline__ void report(unsigned int x) const { atomicOr(&g_pages_status, x); }
};

// All threads of a grid, which meet nowhere.
struct GridTeam {
    int rank, size;
    __device__ __forceinline__ void store(int32_t* p, int32_t x) const { *const_cast<volatile int32_t*>(p) = x; }
    __device__ __forceinline__ void set_bit(uint32_t* bits, int page) const {
        if (page >= 0) atomicOr(bits + (page >> 5), 1u << (page & 31));
    }
    __device__ __forceinline__ void report(unsigned int x) const { atomicOr(&g_pages_status, x); }
};
__device__ __forceinline__ GridTeam this_grid() {
    return GridTeam{(int)(blockIdx.x * kRowThreads + threadIdx.x), (int)(gridDim.x * kRowThreads)};
}

// Shared memory of a block that plans alone, handed out as far as it goes; what
// does not fit stays in the workspace.
constexpr int kOwnBytes = 200 * 1024;
struct Own {
    uint8_t* at;
    int left;
    template <class T>
    __host__ __device__ void take(T*& p, int64_t n) {
        const int64_t bytes = (n * (int64_t)sizeof(T) + 15) / 16 * 16;
        if (bytes > left) return;
        if (at) {
            p = reinterpret_cast<T*>(at);
            at += bytes;
        }
        left -= (int)bytes;
    }
};
// `rows`: what the rows' own kernel does not fill.
__host__ __device__ void take_own(ForkSpace& s, const ForkIn& a, Own& own, bool rows) {
    own.take(s.bits, words_of(a.p.num_pages));
    if (!rows) return;
    own.take(s.place, a.p.B);
    own.take(s.first, a.p.B);
    own.take(s.keeper, a.p.num_pages);
}
__host__ __device__ void take_own(CompactSpace& s, const PagesIn& p, Own& own, bool rows) {
    own.take(s.bits, words_of(p.num_pages));
    if (!rows) return;
    own.take(s.held, words_of(p.num_pages));
    own.take(s.entries, p.B);
    own.take(s.moved, p.num_pages);
    own.take(s.hole, p.num_pages);
    own.take(s.mover, p.num_pages);
}
template <class Space, class In>
int own_bytes(Space s, const In& in, bool rows) {
    Own own{nullptr, kOwnBytes};
    take_own(s, in, own, rows);
    return kOwnBytes - own.left;
}

// kRows: the block takes the rows as well.  Else the bits of their pages are in s.bits.
template <bool kRows>
__global__ void __launch_bounds__(kThreads, 1) kv_fork_kernel(const ForkIn a, ForkSpace s) {
    extern __shared__ __align__(16) uint8_t own_memory[];
    __shared__ TeamScratch scratch;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the copies wait for this kernel's end
    const uint32_t* const marked = s.bits;
    Own own{own_memory, kOwnBytes};
    take_own(s, a, own, kRows);
    BlockTeam<kRows> team{(int)threadIdx.x, kThreads, &scratch, s.bits != marked};
    if constexpr (kRows) plan_fork(team, a, s);
    else fork_rest(team, a, s, marked);
}

template <bool kRows>
__global__ void __launch_bounds__(kThreads, 1) kv_compact_kernel(const PagesIn p, int32_t* top, CompactSpace s) {
    extern __shared__ __align__(16) uint8_t own_memory[];
    __shared__ TeamScratch scratch;
    if constexpr (kRows) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t* const marked = s.bits;
    Own own{own_memory, kOwnBytes};
    take_own(s, p, own, kRows);
    BlockTeam<kRows> team{(int)threadIdx.x, kThreads, &scratch, s.bits != marked};
    if constexpr (kRows) plan_compact(team, p, top, s);
    else compact_moves(team, p, top, s, marked);
}

__global__ void __launch_bounds__(kRowThreads) kv_fork_rows_kernel(const ForkIn a, const ForkSpace s) {
    fork_rows(this_grid(), a, s);
}
__global__ void __launch_bounds__(kRowThreads) kv_compact_rows_kernel(const PagesIn p, const CompactSpace s) {
    compact_rows(this_grid(), p, s);
}
__global__ void __launch_bounds__(kRowThreads) kv_compact_rename_kernel(const PagesIn p, const CompactSpace s) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const GridTeam team = this_grid();
    compact_rename(team, p, s, [&](int b) {
        const int64_t n = p.lens[b], cap = (int64_t)p.width << p.page_log2;      // bad ones are reported already
        return pages_for(n < 0 ? 0 : (n > cap ? cap : n), p.page_log2);
    });
}

// One warp takes a piece at a time: of a part-filled page one head of k or v, whose filled slots lie
// together; of a whole page (kWhole) up to kChunk bytes of k or v, all heads lying together.
constexpr int kChunk = 16384;

template <bool kWhole>
__global__ void __launch_bounds__(256) kv_copy_kernel(const __grid_constant__ CacheSet set, const PageCopy* copies,
                                                      const int32_t* count, int page_log2) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, per = set.first[set.count];
    const int64_t items = (int64_t)*count * per;
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; item < items; item += (int64_t)gridDim.x * 8) {
        const int64_t pair = divide(item, per);
        const int piece = (int)(item - pair * per);
        const PageCopy c = copies[pair];
        if (c.to < 0) continue;                       // there was no page
        int lo = 0, hi = set.count;                   // the cache that the piece is of
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (set.first[mid] <= piece) lo = mid;
            else hi = mid;
        }
        const int heads = set.heads[lo], dim = set.dim[lo], in_cache = piece - set.first[lo];
        const int of_kv = (set.first[lo + 1] - set.first[lo]) / 2, kv = in_cache >= of_kv, at = in_cache - (kv ? of_kv : 0);
        float* const scale = set.scale[lo][kv];
        const int64_t from = (int64_t)c.from * heads, to = (int64_t)c.to * heads;     // first heads of the pages
        int64_t off;                                  // of the piece in its page, bytes
        int n;                                        // 16 bytes each
        if constexpr (kWhole) {
            off = (int64_t)at * kChunk;
            const int64_t left = ((int64_t)heads * dim << page_log2) - off;
            n = (int)(left < kChunk ? left : kChunk) / 16;
            if (at == 0)
                for (int h = lane; h < heads; h += 32) scale[to + h] = scale[from + h];
        } else {
            off = (int64_t)at * dim << page_log2;
            n = c.slots * dim / 16;
            if (lane == 0) scale[to + at] = scale[from + at];
        }
        const uint4* src = reinterpret_cast<const uint4*>(set.code[lo][kv] + ((from * dim) << page_log2) + off);
        uint4* dst = reinterpret_cast<uint4*>(set.code[lo][kv] + ((to * dim) << page_log2) + off);
#pragma unroll 1
        for (int i = lane; i < n; i += 128) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 32 * j < n) v[j] = src[i + 32 * j];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 32 * j < n) dst[i + 32 * j] = v[j];
        }
    }
}

// The workspace's arrays, one after the other, 256-byte aligned; base null: their size alone.
struct Arena {
    uint8_t* base;
    size_t used = 0;
    template <class T>
    T* take(int64_t n) {
        const size_t at = used;
        used += ((size_t)n * sizeof(T) + 255) / 256 * 256;
        return base ? reinterpret_cast<T*>(base + at) : nullptr;
    }
};

size_t lay_out(ForkSpace& s, void* base, int64_t num_pages, int64_t width, int64_t B) {
    Arena m{static_cast<uint8_t*>(base)};
    const int64_t most = B * (width + 1);
    s.count = m.take<int32_t>(1);
    s.bits = m.take<uint32_t>(words_of((int)num_pages));
    s.place = m.take<Place>(B);
    s.first = m.take<int32_t>(B);
    s.keeper = m.take<int32_t>(num_pages);
    s.given = m.take<int32_t>(most < num_pages ? most : num_pages);
    s.copies = m.take<PageCopy>(B);
    return m.used;
}

size_t lay_out(CompactSpace& s, void* base, int64_t num_pages, int64_t B) {
    Arena m{static_cast<uint8_t*>(base)};
    s.count = m.take<int32_t>(1);
    s.mark = m.take<int32_t>(2);
    s.entries = m.take<int32_t>(B);
    s.bits = m.take<uint32_t>(words_of((int)num_pages));
    s.held = m.take<uint32_t>(words_of((int)num_pages));
    s.mover = m.take<int32_t>(num_pages);
    s.hole = m.take<int32_t>(num_pages);
    s.moved = m.take<int32_t>(num_pages);
    s.copies = m.take<PageCopy>(num_pages);
    return m.used;
}

// Whether one block takes the rows too: fewer launches to wait for, but one SM's instructions.  fork | compact, one
// block and apart, us, pages of 16 tokens, 64 dims: 64 rows of 32 entries 12.9, 18.0 | 15.0, 24.7; 256 of 64 17.4, 19.6 | 28.1,
// 38.8; 512 of 64 23.6, 23.2 | 47.4, 48.5; 1024 of 64 34.9, 25.8 | 90.1, 68.8; 4096 of 128 185, 49.6 | 635, 319.
bool few_rows(const PagesIn& p) { return (int64_t)p.B * p.width <= 32768 && p.num_pages <= 1 << 20; }

// The function's attribute is the most that any call uses: a call on another thread may set it in between.
template <class Kernel, class... Args>
cudaError_t launch_plan(Kernel kernel, int bytes, cudaStream_t stream, Args... args) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOwnBytes);
    if (e != cudaSuccess) return e;
    kernel<<<1, kThreads, bytes, stream>>>(args...);
    return cudaGetLastError();
}

template <class Kernel, class... Args>
cudaError_t launch_rows(Kernel kernel, const PagesIn& p, int num_sms, cudaStream_t stream, Args... args) {
    const int64_t blocks = ((int64_t)p.B * p.width + 16 * kRowThreads - 1) / (16 * kRowThreads);    // 16 entries a thread
    kernel<<<(unsigned)std::min<int64_t>(std::max<int64_t>(blocks, 1), 4 * num_sms), kRowThreads, 0, stream>>>(args...);
    return cudaGetLastError();
}

// `most`: copies that there may be.
template <bool kWhole>
cudaError_t launch_copies(const mhc_kv_cache* caches, int n, const PageCopy* copies, const int32_t* count, int64_t most,
                          int page_log2, int num_sms, cudaStream_t stream) {
    for (int begin = 0; begin < n; begin += kMaxSet) {
        CacheSet set;
        set.count = n - begin < kMaxSet ? n - begin : kMaxSet;
        int pieces = 0;
        for (int i = 0; i < set.count; ++i) {
            const mhc_kv_cache& c = caches[begin + i];
            set.code[i][0] = c.k; set.code[i][1] = c.v;
            set.scale[i][0] = c.k_scale; set.scale[i][1] = c.v_scale;
            set.heads[i] = c.heads;
            set.dim[i] = c.head_dim;
            set.first[i] = pieces;
            const int64_t page = (int64_t)c.heads * c.head_dim << page_log2;
            pieces += 2 * (kWhole ? (int)((page + kChunk - 1) / kChunk) : c.heads);
        }
        set.first[set.count] = pieces;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = begin == 0 ? 1 : 0;    // a further launch waits for the one before, and so for the plan
        const int64_t blocks = (most * pieces + 7) / 8;
        cfg.gridDim = dim3((unsigned)(blocks < 8 * num_sms ? blocks : 8 * num_sms), 1, 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = stream;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_copy_kernel<kWhole>, set, copies, count, page_log2);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t kv_fork_workspace(int64_t num_pages, int64_t width, int64_t B) {
    ForkSpace s;
    return lay_out(s, nullptr, num_pages, width, B);
}

size_t kv_compact_workspace(int64_t num_pages, int64_t B) {
    CompactSpace s;
    return lay_out(s, nullptr, num_pages, B);
}

cudaError_t launch_kv_fork(const mhc_kv_cache* caches, int num_caches, const ForkIn& a, void* workspace, int num_sms,
                           cudaStream_t stream) {
    ForkSpace s;
    lay_out(s, workspace, a.p.num_pages, a.p.width, a.p.B);
    cudaError_t e;
    if (few_rows(a.p)) {
        e = launch_plan(kv_fork_kernel<true>, own_bytes(s, a, true), stream, a, s);
    } else {
        e = cudaMemsetAsync(s.bits, 0, (size_t)words_of(a.p.num_pages) * 4, stream);
        if (e == cudaSuccess) e = launch_rows(kv_fork_rows_kernel, a.p, num_sms, stream, a, s);
        if (e == cudaSuccess) e = launch_plan(kv_fork_kernel<false>, own_bytes(s, a, false), stream, a, s);
    }
    return e == cudaSuccess ? launch_copies<false>(caches, num_caches, s.copies, s.count, a.p.B, a.p.page_log2, num_sms, stream) : e;
}

cudaError_t launch_kv_compact(const mhc_kv_cache* caches, int num_caches, const PagesIn& p, int32_t* top, void* workspace,
                              int num_sms, cudaStream_t stream) {
    CompactSpace s;
    lay_out(s, workspace, p.num_pages, p.B);
    cudaError_t e;
    if (few_rows(p)) {
        e = launch_plan(kv_compact_kernel<true>, own_bytes(s, p, true), stream, p, top, s);
    } else {
        e = cudaMemsetAsync(s.bits, 0, (size_t)words_of(p.num_pages) * 4, stream);
        if (e == cudaSuccess) e = launch_rows(kv_compact_rows_kernel, p, num_sms, stream, p, s);
        if (e == cudaSuccess) e = launch_plan(kv_compact_kernel<false>, own_bytes(s, p, false), stream, p, top, s);
        if (e == cudaSuccess) e = launch_rows(kv_compact_rename_kernel, p, num_sms, stream, p, s);
    }
    // half of the pages at most move
    const int64_t most = p.num_pages / 2 + 1;
    return e == cudaSuccess ? launch_copies<true>(caches, num_caches, s.copies, s.count, most, p.page_log2, num_sms, stream) : e;
}

// One query reports one thing: that pages ran out stays where a bad index, or what `other` says, comes first.
cudaError_t read_pages_status(unsigned int* status, bool other) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_pages_status, sizeof v);
    const unsigned int keep = other || (v & kBadIndex) ? v & kPagesError : 0;
    if (e == cudaSuccess && v != keep) e = cudaMemcpyToSymbol(g_pages_status, &keep, sizeof keep);
    *status = v;
    return e;
}

}  // namespace kv
}  // namespace mhc
