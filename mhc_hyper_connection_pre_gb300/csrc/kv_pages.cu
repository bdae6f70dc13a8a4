// kv_pages.cu -- the pages of the next step (mhc_kv_fork) and moving the pages in
// use to the lowest numbers (mhc_kv_compact): one launch that plans, by the
// threads of one block or of one cluster (kv_pages.cuh), and one that copies.
//
// What bounds it: planning reads and writes the tables once, a few hundred KB at
// most; its time is a chain of dependent loads (parent, length, entry) and of
// barriers, whose number is fixed.  Copying is memory: every byte of the copied
// slots is read and written once, 16 bytes a lane, by warps that take one page,
// head and tensor of one layer at a time.
#include "../../include/mhc_kv.h"

#include <cuda_runtime.h>

#include "kv_common.cuh"
#include "kv_pages.cuh"
#include "sm100.cuh"

namespace mhc {
namespace kv {

static __device__ unsigned int g_pages_status = 0;

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCluster = 8;                   // blocks of the large team

// Caches that one launch copies: the layers that share page numbers.
constexpr int kMaxSet = 64;
struct CacheSet {
    uint8_t* code[kMaxSet][2];                // k, v
    float* scale[kMaxSet][2];
    int heads[kMaxSet], dim[kMaxSet];
    int first[kMaxSet + 1];                   // of a page's pieces (one head of k or v): those of cache i begin here
    int count;
};

struct TeamScratch {
    int64_t sums[kWarps];
    int64_t all;
};

// One block, or (kOne false) the blocks of one cluster, which meet in global memory.
template <bool kOne>
struct GpuTeam {
    int rank, size;
    TeamScratch* scratch;
    int64_t* totals;                          // [2][kCluster] in the workspace
    int scans;

    __device__ __forceinline__ void sync() const {
        __syncwarp();
        if constexpr (kOne) {
            __syncthreads();
        } else {
            cluster_arrive_release();
            cluster_wait_acquire();
        }
    }
    __device__ __forceinline__ int64_t scan(int64_t x, int64_t& total) {
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
        int64_t before = scratch->sums[warp] + upto - x;
        total = scratch->all;
        if constexpr (kOne) {
            __syncthreads();
        } else {
            int64_t* of_blocks = totals + (scans++ & 1) * kCluster;
            const int block = (int)cluster_ctarank(), blocks = (int)ncluster_x();
            if (threadIdx.x == 0) of_blocks[block] = total;
            sync();
            total = 0;
            for (int i = 0; i < blocks; ++i) {
                const int64_t n = load(of_blocks + i);
                before += i < block ? n : 0;
                total += n;
            }
        }
        return before;
    }
    template <class T>
    __device__ __forceinline__ T load(const T* p) const {
        return *const_cast<const volatile T*>(p);
    }
    __device__ __forceinline__ void store(int32_t* p, int32_t x) const { *const_cast<volatile int32_t*>(p) = x; }
    // Of the pages' bits, which one block has in shared memory.
    __device__ __forceinline__ void set_bits(uint32_t* p, uint32_t x) const {
        if constexpr (kOne) asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(smem_u32(p)), "r"(x) : "memory");
        else atomicOr(p, x);
    }
    __device__ __forceinline__ void lower(int32_t* p, int32_t x) const { atomicMin(p, x); }
    __device__ __forceinline__ void raise(int32_t* p, int32_t x) const { atomicMax(p, x); }
    __device__ __forceinline__ void report(unsigned int x) const { atomicOr(&g_pages_status, x); }
};

template <bool kOne>
__device__ __forceinline__ GpuTeam<kOne> this_team(TeamScratch* scratch, int64_t* totals) {
    const int block = kOne ? 0 : (int)cluster_ctarank(), blocks = kOne ? 1 : (int)ncluster_x();
    return GpuTeam<kOne>{block * kThreads + (int)threadIdx.x, blocks * kThreads, scratch, totals, 0};
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
__host__ __device__ void take_own(ForkSpace& s, const ForkIn& a, Own& own) {
    own.take(s.bits, words_of(a.p.num_pages));
    own.take(s.place, a.p.B);
    own.take(s.first, a.p.B);
    own.take(s.keeper, a.p.num_pages);
}
__host__ __device__ void take_own(CompactSpace& s, const PagesIn& p, Own& own) {
    own.take(s.bits, words_of(p.num_pages));
    own.take(s.entries, p.B);
    own.take(s.moved, p.num_pages);
    own.take(s.hole, p.num_pages);
    own.take(s.mover, p.num_pages);
}
template <class Space, class In>
int own_bytes(Space s, const In& in) {
    Own own{nullptr, kOwnBytes};
    take_own(s, in, own);
    return kOwnBytes - own.left;
}

template <bool kOne>
__global__ void __launch_bounds__(kThreads, 1) kv_fork_kernel(const ForkIn a, ForkSpace s, int64_t* totals) {
    extern __shared__ __align__(16) uint8_t own_memory[];
    __shared__ TeamScratch scratch;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the copies wait for this kernel's end
    if constexpr (kOne) {
        Own own{own_memory, kOwnBytes};
        take_own(s, a, own);
    }
    GpuTeam<kOne> team = this_team<kOne>(&scratch, totals);
    plan_fork(team, a, s);
}

template <bool kOne>
__global__ void __launch_bounds__(kThreads, 1) kv_compact_kernel(const PagesIn p, int32_t* top, CompactSpace s, int64_t* totals) {
    extern __shared__ __align__(16) uint8_t own_memory[];
    __shared__ TeamScratch scratch;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (kOne) {
        Own own{own_memory, kOwnBytes};
        take_own(s, p, own);
    }
    GpuTeam<kOne> team = this_team<kOne>(&scratch, totals);
    plan_compact(team, p, top, s);
}

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
        const int heads = set.heads[lo], in_cache = piece - set.first[lo], kv = in_cache >= heads, head = in_cache - (kv ? heads : 0);
        const int64_t from = (int64_t)c.from * heads + head, to = (int64_t)c.to * heads + head;
        const int dim = set.dim[lo], n = c.slots * dim / 16;
        const uint4* src = reinterpret_cast<const uint4*>(set.code[lo][kv] + ((from * dim) << page_log2));
        uint4* dst = reinterpret_cast<uint4*>(set.code[lo][kv] + ((to * dim) << page_log2));
        if (lane == 0) set.scale[lo][kv][to] = set.scale[lo][kv][from];
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

size_t lay_out(ForkSpace& s, int64_t*& totals, void* base, int64_t num_pages, int64_t width, int64_t B) {
    Arena m{static_cast<uint8_t*>(base)};
    const int64_t most = B * (width + 1);
    totals = m.take<int64_t>(2 * kCluster);
    s.count = m.take<int32_t>(1);
    s.bits = m.take<uint32_t>(words_of((int)num_pages));
    s.place = m.take<Place>(B);
    s.first = m.take<int32_t>(B);
    s.keeper = m.take<int32_t>(num_pages);
    s.given = m.take<int32_t>(most < num_pages ? most : num_pages);
    s.copies = m.take<PageCopy>(B);
    return m.used;
}

size_t lay_out(CompactSpace& s, int64_t*& totals, void* base, int64_t num_pages, int64_t B) {
    Arena m{static_cast<uint8_t*>(base)};
    totals = m.take<int64_t>(2 * kCluster);
    s.count = m.take<int32_t>(1);
    s.mark = m.take<int32_t>(2);
    s.entries = m.take<int32_t>(B);
    s.bits = m.take<uint32_t>(words_of((int)num_pages));
    s.mover = m.take<int32_t>(num_pages);
    s.hole = m.take<int32_t>(num_pages);
    s.moved = m.take<int32_t>(num_pages);
    s.copies = m.take<PageCopy>(num_pages);
    return m.used;
}

// Whether one block plans: its barriers are short, but it has one SM's loads.
bool one_block(const PagesIn& p) { return (int64_t)p.B * p.width <= 65536 && p.num_pages <= 1 << 20; }

template <class Kernel, class... Args>
cudaError_t launch_plan(Kernel kernel, bool one, int bytes, cudaStream_t stream, Args... args) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = one ? 1 : kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(one ? 1 : kCluster, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// `most`: copies that there may be.
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
            pieces += 2 * c.heads;
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
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_copy_kernel, set, copies, count, page_log2);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t kv_fork_workspace(int64_t num_pages, int64_t width, int64_t B) {
    ForkSpace s;
    int64_t* totals;
    return lay_out(s, totals, nullptr, num_pages, width, B);
}

size_t kv_compact_workspace(int64_t num_pages, int64_t B) {
    CompactSpace s;
    int64_t* totals;
    return lay_out(s, totals, nullptr, num_pages, B);
}

cudaError_t launch_kv_fork(const mhc_kv_cache* caches, int num_caches, const ForkIn& a, void* workspace, int num_sms,
                           cudaStream_t stream) {
    ForkSpace s;
    int64_t* totals;
    lay_out(s, totals, workspace, a.p.num_pages, a.p.width, a.p.B);
    const bool one = one_block(a.p);
    const cudaError_t e = one ? launch_plan(kv_fork_kernel<true>, one, own_bytes(s, a), stream, a, s, totals)
                              : launch_plan(kv_fork_kernel<false>, one, 0, stream, a, s, totals);
    return e == cudaSuccess ? launch_copies(caches, num_caches, s.copies, s.count, a.p.B, a.p.page_log2, num_sms, stream) : e;
}

cudaError_t launch_kv_compact(const mhc_kv_cache* caches, int num_caches, const PagesIn& p, int32_t* top, void* workspace,
                              int num_sms, cudaStream_t stream) {
    CompactSpace s;
    int64_t* totals;
    lay_out(s, totals, workspace, p.num_pages, p.B);
    const bool one = one_block(p);
    const cudaError_t e = one ? launch_plan(kv_compact_kernel<true>, one, own_bytes(s, p), stream, p, top, s, totals)
                              : launch_plan(kv_compact_kernel<false>, one, 0, stream, p, top, s, totals);
    // half of the pages at most move
    const int64_t most = p.num_pages / 2 + 1;
    return e == cudaSuccess ? launch_copies(caches, num_caches, s.copies, s.count, most, p.page_log2, num_sms, stream) : e;
}

cudaError_t read_pages_status(unsigned int* status) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_pages_status, sizeof v);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_pages_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace kv
}  // namespace mhc
