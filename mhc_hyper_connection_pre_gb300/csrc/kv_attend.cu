// kv_attend.cu -- causal attention of the new tokens over the paged e4m3
// cache (mhc_kv_attend), for few rows a sequence: decoding.
//
// Mathematics.  The rows of a tile are the new tokens and query heads that
// share a key/value head (8 or 16 of them).  A warp takes 32 keys at a time
// and forms S^T = K Q^T (keys x rows) and O^T += V^T P^T (dims x rows) with
// m16n8k16 matrix instructions in f16 with fp32 sums, so that the few rows
// fill the 8-wide side and none of the 16-wide side is padding.  e4m3 becomes
// f16 exactly; a query row becomes f16 after a division by a power of two that
// puts its largest element into [2^7, 2^8), which loses nothing of bf16's 8
// bits down to 2^-21 of the largest.  The softmax keeps a running maximum and
// sum for each row in fp32, in powers of two.  The weights are rounded to f16
// for the second product (2^-11 of each, well below the output's own bf16
// rounding) after a factor of 2^10 that keeps small weights out of f16's
// subnormal range.  A page's value scale multiplies the weights, relative to
// the largest scale met so far, so that they stay below 2^10.
//
// What bounds it: the cache is read once, 2 * head_dim bytes a key and head
// for 4 * head_dim * group operations, far below the matrix rate for groups up
// to 16: HBM.  So every warp runs on its own, with its own ring of TMA loads
// (24 KB, 192 KB in flight on an SM) and its own part of the keys, and the
// warps of a block meet only when a segment ends.  All blocks take equally
// many units of 64 keys whatever the lengths are (kv_index.cuh); what a border
// cuts is left as partial sums in the workspace and joined by a second, small
// kernel.
#include "kv_attend.cuh"

namespace mhc {
namespace kv {

namespace {

constexpr int kSub = 32;                      // keys of one load of one warp
constexpr int kPass = 64;                     // dims that warps exchange at a time
constexpr int kPitch = kPass + 8;             // floats; conflict-free for the fragments' order
constexpr int kUnitLog2 = 6;                  // units of 64 keys

template <int D, int NB>
struct Shape {
    static constexpr int kWarps = NB == 1 ? (D == 128 ? 12 : 16) : (D == 128 ? 8 : 12);   // as the registers allow
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStage = kSub * D * 2;               // K and V of one load
    static constexpr int kStages = (D == 128 ? 192 : 160) * 1024 / (kWarps * kStage);     // of one warp's ring
};

struct __align__(16) Meta {                   // of one load
    float scale[4];                           // k of keys 0-15, k of 16-31, v, v; read only where there is a page
    int page[2];                              // -1: no such page
    int pad[2];
};

template <int D, int NB>
struct __align__(1024) Smem {
    static constexpr int kWarps = Shape<D, NB>::kWarps, kStages = Shape<D, NB>::kStages;
    uint8_t ring[kWarps][kStages * Shape<D, NB>::kStage];
    float pass[kWarps][8][kPitch];
    float ml[kWarps][8][2];
    Meta meta[kWarps][kStages];
    Segment segs[kSegments];
    int count;                                // of segs
    uint64_t full[kWarps][kStages];
    int abort;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The loads of one warp, in order: the 32-key pieces of each segment that are
// this warp's (every kWarps-th from the warp-th on).
struct Loads {
    int seg;                                  // index of the segment
    int key, keys;                            // the piece's first key, the segment's last key + 1
};

__device__ __forceinline__ void loads_settle(Loads& l, const Segment* segs, int count, const Cut& cut, int warp) {
    while (l.key >= l.keys) {                 // on to a segment that has a piece for this warp
        if (++l.seg >= count) return;
        keys_of(segs[l.seg], cut, l.key, l.keys);
        l.key += warp * kSub;
    }
}

// Word x of the dims that row group g holds of key r's values.
template <int D>
__device__ __forceinline__ uint32_t value_word(uint32_t vs, int r, int g, int x) {
    const uint32_t at = D == 128 ? r * 128 + ((g ^ (r & 7)) << 4) : r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8;
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(vs + at + 4 * x));
    return v;
}

// The 32 keys of one piece against the tile's rows.
template <int D, int NB>
struct Acc {
    float o[D / 16][NB][4];
    float m[NB][2], l[NB][2];                 // of rows 2t, 2t + 1 of each block of 8; l: this thread's share
    float ref;                                // the value scale that o is in units of
};

template <int D, int NB, bool kFull>
__device__ __forceinline__ void piece(uint32_t ks, uint32_t vs, const Meta& meta, const uint32_t (&q)[NB][D / 8],
                                      const float (&f)[NB][2], const int (&lim)[NB][2], int key0, int keys, int lane,
                                      Acc<D, NB>& acc) {
    const int g = lane / 4, t = lane % 4;
    float s[2][NB][4];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mb][nb][i] = 0.0f;
        const int r = mb * 16 + g;
        if constexpr (D == 128) {             // 128-byte swizzle: 16-byte chunk c of row r lies at c ^ (r & 7)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t at = ks + r * 128 + (((2 * t + j) ^ g) << 4);
                const uint4 u = lds128(at), v = lds128(at + 8 * 128);
                const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = cvt_lo(a[i]), a1 = cvt_lo(b[i]), a2 = cvt_hi(a[i]), a3 = cvt_hi(b[i]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        mma_f16(s[mb][nb], a0, a1, a2, a3, q[nb][8 * j + 2 * i], q[nb][8 * j + 2 * i + 1]);
                }
            }
        } else {                              // 64-byte swizzle: chunk c of row r lies at c ^ ((r >> 1) & 3)
            const uint32_t at = ks + r * 64 + ((t ^ ((g >> 1) & 3)) << 4);
            const uint4 u = lds128(at), v = lds128(at + 8 * 64);
            const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = cvt_lo(a[i]), a1 = cvt_lo(b[i]), a2 = cvt_hi(a[i]), a3 = cvt_hi(b[i]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_f16(s[mb][nb], a0, a1, a2, a3, q[nb][2 * i], q[nb][2 * i + 1]);
            }
        }
    }

    // logits in powers of two, masks, the running maximum
    const float k0 = meta.scale[0], k1 = meta.scale[1];
    const bool has0 = kFull || meta.page[0] >= 0, has1 = kFull || meta.page[1] >= 0;
    float keep[NB][2];
    bool same = true;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float f0 = f[nb][e] * k0, f1 = f[nb][e] * k1;
            float x[4] = {s[0][nb][e] * f0, s[0][nb][e + 2] * f0, s[1][nb][e] * f1, s[1][nb][e + 2] * f1};
            if (!kFull) {
                const int n = lim[nb][e] - key0;      // keys of this piece that the row sees
                x[0] = has0 && g < n ? x[0] : -INFINITY;
                x[1] = has0 && g + 8 < n ? x[1] : -INFINITY;
                x[2] = has1 && g + 16 < n ? x[2] : -INFINITY;
                x[3] = has1 && g + 24 < n ? x[3] : -INFINITY;
            }
            float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float old = acc.m[nb][e], now = fmaxf(old, top);
            const float zero = now == -INFINITY ? 0.0f : now - kLift;
            keep[nb][e] = old == now ? 1.0f : ex2(old - now);
            same = same && old == now;
            acc.m[nb][e] = now;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = ex2(x[i] - zero);
                sum += x[i];
            }
            acc.l[nb][e] = acc.l[nb][e] * keep[nb][e] + sum;
            s[0][nb][e] = x[0]; s[0][nb][e + 2] = x[1]; s[1][nb][e] = x[2]; s[1][nb][e + 2] = x[3];
        }
    }

    // value scales relative to the largest so far
    const float v0 = has0 ? meta.scale[2] : 0.0f, v1 = has1 ? meta.scale[3] : 0.0f;   // no page: no weight either
    const float most = fmaxf(v0, v1);
    float shrink = 1.0f;
    if (most > acc.ref) {                     // the same for the whole warp
        shrink = acc.ref / most;
        acc.ref = most;
        same = false;
    }
    if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const float x = keep[nb][0] * shrink, y = keep[nb][1] * shrink;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                acc.o[j][nb][0] *= x;
                acc.o[j][nb][1] *= y;
                acc.o[j][nb][2] *= x;
                acc.o[j][nb][3] *= y;
            }
        }
    }
    const float inv = acc.ref > 0.0f ? 1.0f / acc.ref : 0.0f;
    const float w0 = v0 * inv, w1 = v1 * inv;

    constexpr int kVW = D / 32;               // words of a key's values that a thread holds (4 dims each)
    uint32_t nans = 0;
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        const float w = mb ? w1 : w0;
        uint32_t b[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            b[nb][0] = transpose8x8(pack_f16x2(s[mb][nb][0] * w, s[mb][nb][1] * w));
            b[nb][1] = transpose8x8(pack_f16x2(s[mb][nb][2] * w, s[mb][nb][3] * w));
        }
        uint32_t v[4][kVW];                   // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = mb * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
            if constexpr (D == 128) {
                const uint4 u = lds128(vs + r * 128 + ((g ^ (r & 7)) << 4));
                v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
            } else {
                const uint2 u = lds64(vs + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
                v[i][0] = u.x; v[i][1] = u.y;
            }
        }
        if (!kFull) {
            // Keys that no row of the tile sees count as zeros, whatever their
            // bytes are.  NaN among the others must reach only the rows that
            // see its key, but 0 * NaN is NaN: it is taken out here and put
            // back into those rows below.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = mb * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
                const uint32_t use = (mb ? has1 : has0) && key0 + r < keys ? 0xffffffffu : 0u;
#pragma unroll
                for (int x = 0; x < kVW; ++x) {
                    const uint32_t n = nan_bytes(v[i][x]) & use;
                    nans |= n;
                    v[i][x] &= use & ~((n >> 7) * 0xffu);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < kVW; ++x) {
            const uint32_t lo = __byte_perm(v[0][x], v[1][x], 0x5140), hi = __byte_perm(v[0][x], v[1][x], 0x7362);
            const uint32_t lo8 = __byte_perm(v[2][x], v[3][x], 0x5140), hi8 = __byte_perm(v[2][x], v[3][x], 0x7362);
            const uint32_t a[2][4] = {{cvt_lo(lo), cvt_hi(lo), cvt_lo(lo8), cvt_hi(lo8)},
                                      {cvt_lo(hi), cvt_hi(hi), cvt_lo(hi8), cvt_hi(hi8)}};
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    mma_f16(acc.o[2 * x + y][nb], a[y][0], a[y][1], a[y][2], a[y][3], b[nb][0], b[nb][1]);
        }
    }
    if (!kFull && __any_sync(0xffffffffu, nans != 0)) {
#pragma unroll 1
        for (int r = 0; r < kSub && key0 + r < keys; ++r) {
            if (!(r < 16 ? has0 : has1)) continue;
            uint32_t v[kVW];                  // this thread's dims of key r
#pragma unroll
            for (int x = 0; x < kVW; ++x) v[x] = nan_bytes(value_word<D>(vs, r, g, x));
#pragma unroll
            for (int x = 0; x < kVW * 4; ++x)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if ((v[x / 4] >> (8 * (x % 4))) & 0x80u && key0 + r < lim[nb][e])
                            acc.o[x / 2][nb][2 * (x & 1) + e] = __int_as_float(0x7fc00000);
        }
    }
}

// Dim of position p of the order in which the fragments hold a head's dims:
// block j = p / 16 of O^T, its row group g = p / 2 % 8, first or second.
template <int D>
__device__ __forceinline__ int dim_of(int p) {
    return (D / 8) * ((p / 2) % 8) + 2 * (p / 16) + (p & 1);
}

// One tile's row r goes out: o[0..3] are positions p .. p + 3 (unnormalised),
// m and l the row's maximum and sum.
template <int D>
__device__ __forceinline__ void write_row(const AttendArgs& a, int begin, int row, int head, int p, const float4& o,
                                          float m, float l) {
    const int64_t at = place_of(a, begin, row, head);
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* out = a.out + at * D;
    *reinterpret_cast<uint32_t*>(out + dim_of<D>(p)) = pack_bf16x2(o.x * r, o.y * r);
    *reinterpret_cast<uint32_t*>(out + dim_of<D>(p + 2)) = pack_bf16x2(o.z * r, o.w * r);
    if (p == 0 && a.lse) a.lse[at] = lse_of(m, l);
}

template <int D, int NB>
__global__ void __launch_bounds__(Shape<D, NB>::kThreads, 1)
    kv_attend_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const AttendArgs a) {
    constexpr int kWarps = Shape<D, NB>::kWarps, kStages = Shape<D, NB>::kStages, kStage = Shape<D, NB>::kStage;
    constexpr int kRows = 8 * NB;
    extern __shared__ uint8_t raw[];
    Smem<D, NB>& sm = *reinterpret_cast<Smem<D, NB>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel waits for this one's end
    if (tid == 0) sm.abort = 0;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[warp][i], 1 + 4);   // lane 0 and the four scales
        fence_mbar_init_cluster();
    }
    if (tid == 0) a.desc[blockIdx.x].parts = 0;

    Planner plan;                             // of the first warp
    uint32_t issued = 0, waited = 0;          // loads of this warp
    for (bool begun = false;; begun = true) {
        if (warp == 0) {
            if (!begun) plan.begin(a, lane);
            const int n = plan.next(a, sm.segs, lane);
            if (lane == 0) sm.count = n;
        }
        __syncthreads();
        const int count = sm.count;
        if (count == 0) break;

        Loads ld{-1, 0, 0};
        loads_settle(ld, sm.segs, count, a.cut, warp);
        int page[2] = {-1, -1};
        auto find_pages = [&] {               // of the next load; used only when it is issued
            if (ld.seg >= count) return;
            const int32_t* row = a.seqs.table + (int64_t)sm.segs[ld.seg].b * a.seqs.width;
            page[0] = __ldg(row + (ld.key >> a.seqs.page_log2));
            page[1] = ld.key + 16 < ld.keys ? __ldg(row + ((ld.key + 16) >> a.seqs.page_log2)) : -1;
        };
        auto issue = [&] {
            if (ld.seg >= count || *(volatile int*)&sm.abort) return;
            const int st = issued % kStages;
            const int slot = ld.key & ((1 << a.seqs.page_log2) - 1), head = sm.segs[ld.seg].head;
            const bool ok0 = page[0] >= 0 && page[0] < a.seqs.num_pages;
            const bool ok1 = page[1] >= 0 && page[1] < a.seqs.num_pages;
            const bool two = ld.key + 16 < ld.keys;
            if ((!ok0 || (two && !ok1)) && lane == 0) atomicOr(&g_device_status, kIndexError);
            uint64_t* bar = &sm.full[warp][st];
            Meta& meta = sm.meta[warp][st];
            if (lane < 4) {
                const int mb = lane & 1;
                if (mb ? ok1 : ok0) {
                    const float* src = (lane < 2 ? a.k_scale : a.v_scale) + (int64_t)page[mb] * a.cut.heads + head;
                    copy_async4(&meta.scale[lane], src);
                }
                arrive_after_copies(bar);
            }
            if (lane == 0) {
                uint8_t* dst = sm.ring[warp] + st * kStage;
                meta.page[0] = ok0 ? page[0] : -1;
                meta.page[1] = ok1 ? page[1] : -1;
                if (a.seqs.page_log2 >= 5) {            // both halves lie in one page
                    mbar_arrive_expect_tx(bar, ok0 ? kStage : 0);
                    if (ok0) {
                        const int block = page[0] * a.cut.heads + head;
                        tma_load_3d(dst, &k_map, 0, slot, block, bar);
                        tma_load_3d(dst + kStage / 2, &v_map, 0, slot, block, bar);
                    }
                } else {
                    mbar_arrive_expect_tx(bar, (ok0 ? kStage / 2 : 0) + (ok1 ? kStage / 2 : 0));
                    if (ok0) {
                        const int block = page[0] * a.cut.heads + head;
                        tma_load_3d(dst, &k_map, 0, 0, block, bar);
                        tma_load_3d(dst + kStage / 2, &v_map, 0, 0, block, bar);
                    }
                    if (ok1) {
                        const int block = page[1] * a.cut.heads + head;
                        tma_load_3d(dst + kStage / 4, &k_map, 0, 0, block, bar);
                        tma_load_3d(dst + kStage / 2 + kStage / 4, &v_map, 0, 0, block, bar);
                    }
                }
            }
            ++issued;
            ld.key += kWarps * kSub;
            loads_settle(ld, sm.segs, count, a.cut, warp);
            find_pages();
        };
        find_pages();
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) issue();

        for (int index = 0; index < count; ++index) {
            const Segment seg = sm.segs[index];
            const SeqInfo info = seg.info;
            int key0, keys;
            keys_of(seg, a.cut, key0, keys);
            const int first_row = seg.tile * kRows;
            const int rows = info.rows - first_row < kRows ? info.rows - first_row : kRows;

            // queries: thread (g, t) holds row g's dims [t D/4, (t + 1) D/4) of each block of 8 rows
            uint32_t q[NB][D / 8];
            float f[NB][2];
            int lim[NB][2];
            Acc<D, NB> acc;
            acc.ref = 0.0f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int row = nb * 8 + g;
                uint4 u[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; ++i) u[i] = make_uint4(0, 0, 0, 0);
                if (row < rows) {
                    const int r = first_row + row, token = info.begin + r / a.cut.group;
                    const int head = seg.head * a.cut.group + r % a.cut.group;
                    const uint4* src =
                        reinterpret_cast<const uint4*>(a.q + token * a.q_stride + head * D + t * (D / 4));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) u[i] = __ldg(src + i);
                }
                float x[D / 4], top = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float y[8];
                    unpack8(u[i], y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[8 * i + j] = y[j];
                        top = fmaxf(top, fabsf(y[j]));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = 134 - (int)(__float_as_uint(top) >> 23);      // 7 - floor(log2(top))
                e = e < -120 ? -120 : (e > 120 ? 120 : e);
                const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) q[nb][i] = pack_f16x2(x[2 * i] * up, x[2 * i + 1] * up);
                const float back = down * a.scale_log2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = nb * 8 + 2 * t + i;
                    f[nb][i] = __shfl_sync(0xffffffffu, back, (2 * t + i) * 4);
                    lim[nb][i] = c < rows ? keys_of_row(info, a.cut, first_row + c) : 0;
                    acc.m[nb][i] = -INFINITY;
                    acc.l[nb][i] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc.o[j][nb][i] = 0.0f;
            }
            const int all_see = keys_of_row(info, a.cut, first_row);  // keys that every row sees

            for (int key = key0 + warp * kSub; key < keys; key += kWarps * kSub) {
                const int st = waited % kStages;
                if (waited == issued) break;  // after a wait that gave up
                const bool ok = wait_for(&sm.full[warp][st], (waited / kStages) & 1, &sm.abort);
                ++waited;
                if (!ok) break;
                const uint32_t base_addr = smem_u32(sm.ring[warp] + st * kStage);
                const Meta& meta = sm.meta[warp][st];
                const bool full = key + kSub <= all_see && meta.page[0] >= 0 && meta.page[1] >= 0;
                if (full)
                    piece<D, NB, true>(base_addr, base_addr + kStage / 2, meta, q, f, lim, key, keys, lane, acc);
                else
                    piece<D, NB, false>(base_addr, base_addr + kStage / 2, meta, q, f, lim, key, keys, lane, acc);
                __syncwarp();                 // every lane has read the stage
                issue();
            }

            // the warps' sums of this segment, joined
            const bool whole = seg.first == 0 && seg.count == seg.units;
            const int slot = seg.first == 0 ? 1 : 0;
            float* part = part_of(a, blockIdx.x, slot, D);
            if (!whole && slot && tid == 0)
                a.desc[blockIdx.x] = PartDesc{seg.parts, info.begin, first_row, rows, seg.head, {}};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = acc.l[nb][e];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    if (g == 0) {
                        sm.ml[warp][2 * t + e][0] = acc.m[nb][e];
                        sm.ml[warp][2 * t + e][1] = l;
                    }
                }
#pragma unroll
                for (int pass = 0; pass < D / kPass; ++pass) {
#pragma unroll
                    for (int j = 0; j < kPass / 16; ++j) {
                        const float(&o)[4] = acc.o[pass * (kPass / 16) + j][nb];
                        float* at = &sm.pass[warp][2 * t][j * 16 + 2 * g];
                        *reinterpret_cast<float2*>(at) = make_float2(o[0] * acc.ref, o[2] * acc.ref);
                        *reinterpret_cast<float2*>(at + kPitch) = make_float2(o[1] * acc.ref, o[3] * acc.ref);
                    }
                    __syncthreads();
                    const int row = tid / 16, p = (tid % 16) * 4;     // 8 rows x 16 threads: half of the block
                    if (tid < 128) {
                        float m = -INFINITY;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.ml[w][row][0]);
                        const float zero = m == -INFINITY ? 0.0f : m;
                        float l = 0.0f;
                        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            const float x = ex2(sm.ml[w][row][0] - zero);
                            const float4 y = *reinterpret_cast<const float4*>(&sm.pass[w][row][p]);
                            l = fmaf(x, sm.ml[w][row][1], l);
                            o.x = fmaf(x, y.x, o.x);
                            o.y = fmaf(x, y.y, o.y);
                            o.z = fmaf(x, y.z, o.z);
                            o.w = fmaf(x, y.w, o.w);
                        }
                        const int r = nb * 8 + row, at = pass * kPass + p;
                        if (r < rows) {
                            if (whole) {
                                write_row<D>(a, info.begin, first_row + r, seg.head, at, o, m, l);
                            } else {
                                float* dst = part + r * D;
                                *reinterpret_cast<float2*>(dst + dim_of<D>(at)) = make_float2(o.x, o.y);
                                *reinterpret_cast<float2*>(dst + dim_of<D>(at + 2)) = make_float2(o.z, o.w);
                                if (at == 0)
                                    *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(m, l);
                            }
                        }
                    }
                    __syncthreads();
                }
            }
        }
        __syncthreads();                      // before the next segments are planned
    }
    // after a wait that gave up: the loads still under way
    for (; waited != issued; ++waited) mbar_wait_drain(&sm.full[warp][waited % kStages], (waited / kStages) & 1);
}

// Joins the parts of the tile that block blockIdx.x of the attention began
// and did not finish: its slot 1, then slot 0 of the blocks after it.  A row is
// D / 4 lanes' work: first a lane for each part finds the parts' weights, then
// each lane adds up its four dims.  Every load but the first depends on nothing
// that came before it.
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const AttendArgs a) {
    constexpr int kLanes = D / 4, kRows = 256 / kLanes;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const PartDesc d = a.desc[c];
    if (d.parts == 0) return;
    const int lane = threadIdx.x % kLanes;
    const int64_t next = 2 * (int64_t)a.cut.tile_rows * (D + 2);      // from a block's part to the next block's
    const float* first = part_of(a, c, 1, D);
    const float* rest = part_of(a, c + 1, 0, D) - next;               // part k, k > 0, at rest + k * next
    const int ml = a.cut.tile_rows * D;
    for (int r0 = blockIdx.y * kRows; r0 < d.rows; r0 += gridDim.y * kRows) {
        const int row = r0 + threadIdx.x / kLanes, r = row < d.rows ? row : d.rows - 1;   // whole warps shuffle
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int base = 0; base < d.parts; base += kLanes) {
            const int n = d.parts - base < kLanes ? d.parts - base : kLanes, k = base + lane;
            float2 mine = make_float2(-INFINITY, 0.0f);
            if (lane < n) mine = *reinterpret_cast<const float2*>((k ? rest + k * next : first) + ml + 2 * r);
            float now = mine.x;
#pragma unroll
            for (int i = kLanes / 2; i; i >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, i));
            now = fmaxf(now, m);
            const float zero = now == -INFINITY ? 0.0f : now, keep = ex2(m - zero);
            const float w = ex2(mine.x - zero);
            float sum = w * mine.y;
#pragma unroll
            for (int i = kLanes / 2; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            l = fmaf(l, keep, sum);
            o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
            m = now;
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float x = __shfl_sync(0xffffffffu, w, i, kLanes);
                const float4 y =
                    reinterpret_cast<const float4*>((base + i ? rest + (base + i) * next : first) + r * D)[lane];
                o.x = fmaf(x, y.x, o.x);
                o.y = fmaf(x, y.y, o.y);
                o.z = fmaf(x, y.z, o.z);
                o.w = fmaf(x, y.w, o.w);
            }
        }
        if (row >= d.rows) continue;
        const int64_t to = place_of(a, d.begin, d.first_row + r, d.head);
        const float y = l == 0.0f ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint2*>(a.out + to * D + 4 * lane) =
            make_uint2(pack_bf16x2(o.x * y, o.y * y), pack_bf16x2(o.z * y, o.w * y));
        if (lane == 0 && a.lse) a.lse[to] = lse_of(m, l);
    }
}

// Rows of a tile.  Up to 16 rows a sequence: one tile of 8 or 16 for the warps
// of this file; more: the tensor-memory kernel's 256.
int tile_rows(int group, int64_t B, int64_t T) { return T * group > 16 * B ? 256 : (T * group > 8 * B ? 16 : 8); }

size_t part_bytes(int rows, int D, int blocks) { return ((size_t)blocks * 2 * rows * (D + 2) * 4 + 255) / 256 * 256; }

template <int D, int NB>
cudaError_t launch(const CUtensorMap& k_map, const CUtensorMap& v_map, const AttendArgs& a, int blocks,
                   cudaStream_t stream) {
    const int bytes = (int)sizeof(Smem<D, NB>) + 1024;
    // an attribute of the function on the current device: set on every call, which keeps no state here
    const cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kv_attend_kernel<D, NB><<<blocks, Shape<D, NB>::kThreads, bytes, stream>>>(k_map, v_map, a);
    return cudaGetLastError();
}

cudaError_t launch_join(const AttendArgs& a, int head_dim, int blocks, cudaStream_t stream) {
    if (blocks < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(blocks - 1, a.cut.tile_rows > 16 ? 8 : 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, head_dim == 64 ? kv_join_kernel<64> : kv_join_kernel<128>, a);
}

}  // namespace

cudaError_t launch_kv_attend_tc(const AttendArgs& a, const uint8_t* k, const uint8_t* v, int head_dim, int blocks,
                                cudaStream_t stream);

size_t kv_attend_workspace(int heads, int head_dim, int q_heads, int64_t B, int64_t T, int num_sms) {
    return part_bytes(tile_rows(q_heads / heads, B, T), head_dim, num_sms) + (size_t)num_sms * sizeof(PartDesc);
}

cudaError_t launch_kv_attend(const Seqs& seqs, const uint8_t* k, const uint8_t* v, const float* k_scale,
                             const float* v_scale, int heads, int head_dim, const uint16_t* q, int64_t q_stride,
                             int q_heads, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                             int num_sms, cudaStream_t stream) {
    AttendArgs a;
    const int rows = tile_rows(q_heads / heads, seqs.B, seqs.T);
    a.seqs = seqs;
    a.cut = Cut{heads, q_heads / heads, rows, rows == 256 ? kUnitLog2 + 1 : kUnitLog2};
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.q = q;
    a.q_stride = q_stride;
    a.scale_log2 = softmax_scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.part = static_cast<float*>(workspace);
    a.desc = reinterpret_cast<PartDesc*>(static_cast<uint8_t*>(workspace) + part_bytes(rows, head_dim, num_sms));
    cudaError_t e;
    if (rows == 256) {
        e = launch_kv_attend_tc(a, k, v, head_dim, num_sms, stream);
    } else {
        CUtensorMap k_map, v_map;
        const int64_t pages = (int64_t)seqs.num_pages * heads;
        if (!encode_codes(&k_map, k, pages, 1 << seqs.page_log2, head_dim, kSub) ||
            !encode_codes(&v_map, v, pages, 1 << seqs.page_log2, head_dim, kSub))
            return cudaErrorInvalidValue;
        if (rows == 8)
            e = head_dim == 64 ? launch<64, 1>(k_map, v_map, a, num_sms, stream)
                               : launch<128, 1>(k_map, v_map, a, num_sms, stream);
        else
            e = head_dim == 64 ? launch<64, 2>(k_map, v_map, a, num_sms, stream)
                               : launch<128, 2>(k_map, v_map, a, num_sms, stream);
    }
    return e == cudaSuccess ? launch_join(a, head_dim, num_sms, stream) : e;
}

cudaError_t read_attend_status(unsigned int* status) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof v);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace kv
}  // namespace mhc
