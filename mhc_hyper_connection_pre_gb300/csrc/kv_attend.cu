// kv_attend.cu -- causal attention of the new tokens over the paged e4m3
// cache (mhc_kv_attend), for few rows a sequence (see tile_rows): decoding.
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
// subnormal range.  The maximum follows only when a logit is more than 2^5 above
// it, so weights reach 2^15; logits are rounded before the maximum is taken off,
// so that this holds for sharp ones too.  A page's value scale multiplies the
// weights, relative to the largest scale met so far, so that they get no larger
// (a weight in f16's subnormal range is off by 2^-35 of the row's largest).
//
// What bounds it: the cache is read once, 2 * head_dim bytes a key and head
// for 4 * head_dim * group operations, far below the matrix rate for groups up
// to 16: HBM, as long as the conversion keeps up.  Every warp runs on its own:
// it has its own equal share of all units of 32 keys, whatever the lengths are
// (kv_index.cuh), its own ring of TMA loads, 192 KB in flight on an SM together,
// and it meets no other warp.  A block-wide join of the warps at each tile's
// end cost 10 us a tile and more in barriers and idle warps.  Tiles that a
// border between shares cuts are left as partial sums in the workspace and
// joined by a second kernel.
#include "kv_attend.cuh"

namespace mhc {
namespace kv {

namespace {

constexpr int kSub = 32;                      // keys of one load of one warp
constexpr int kQueue = 8;                     // segments that a warp's loads may be ahead of its products
constexpr int kUnitLog2 = 5;                  // units of 32 keys, one load

template <int D, int NB>
struct Shape {
    static constexpr int kWarps = NB == 1 ? (D == 128 ? 12 : 16) : (D == 128 ? 8 : 12);   // as the registers allow
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStage = kSub * D * 2;               // K and V of one load
    static constexpr int kStages = 192 * 1024 / (kWarps * kStage);     // of one warp's ring
};

struct __align__(16) Meta {                   // of one load
    float scale[4];                           // k of keys 0-15, k of 16-31, v, v; read only where there is a page
    int block[2];                             // -1: no such page
    int pad[2];
};

template <int D, int NB>
struct __align__(1024) Smem {
    static constexpr int kWarps = Shape<D, NB>::kWarps, kStages = Shape<D, NB>::kStages;
    uint8_t ring[kWarps][kStages * Shape<D, NB>::kStage];
    Meta meta[kWarps][kStages];
    Segment queue[kWarps][kQueue];
    Plan plan[kWarps];
    Shares shares[kWarps];
    int64_t counted[32];
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
    float ref, inv;                           // the value scale that o is in units of, and one over it
};

// `full`: every row sees all of them.  One copy of the code for both cases, as a
// second one would fall out of the instruction cache between its rare uses.
template <int D, int NB>
__device__ __forceinline__ void piece(bool full, uint32_t ks, uint32_t vs, const Meta& meta, const uint32_t (&q)[NB][D / 8],
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

    // Logits in powers of two and masks.  The running maximum follows only when a
    // logit is more than 2^5 above it (weights reach 2^15 then, within f16), so
    // that the rows' maxima are seldom brought together across the lanes.
    const float k0 = meta.scale[0], k1 = meta.scale[1];
    const bool has0 = meta.block[0] >= 0, has1 = meta.block[1] >= 0;
    bool grow = false;
    float top[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float f0 = f[nb][e] * k0, f1 = f[nb][e] * k1;
            float x[4] = {s[0][nb][e] * f0, s[0][nb][e + 2] * f0, s[1][nb][e] * f1, s[1][nb][e + 2] * f1};
            if (!full) {
                const int n = lim[nb][e] - key0 - g;      // of this thread's keys g, g + 8, .. the row sees those below n
                const int n0 = has0 ? n : 0, n1 = has1 ? n : 0;
                x[0] = n0 > 0 ? x[0] : -INFINITY;
                x[1] = n0 > 8 ? x[1] : -INFINITY;
                x[2] = n1 > 16 ? x[2] : -INFINITY;
                x[3] = n1 > 24 ? x[3] : -INFINITY;
            }
            top[nb][e] = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            grow = grow || top[nb][e] - acc.m[nb][e] > kGrow;
            s[0][nb][e] = x[0]; s[0][nb][e + 2] = x[1]; s[1][nb][e] = x[2]; s[1][nb][e + 2] = x[3];
        }
    }

    // value scales relative to the largest so far
    const float v0 = has0 ? meta.scale[2] : 0.0f, v1 = has1 ? meta.scale[3] : 0.0f;   // no page: no weight either
    const float most = fmaxf(v0, v1);
    grow = __any_sync(0xffffffffu, grow);
    if (grow || most > acc.ref) {             // the same for the whole warp
        float shrink = 1.0f;
        if (most > acc.ref) {
            const float now = value_unit(most);
            acc.inv = __frcp_rn(now);
            shrink = acc.ref * acc.inv;
            acc.ref = now;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float now = top[nb][e];
                now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 4));
                now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
                now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
                const float old = acc.m[nb][e];
                now = fmaxf(old, now);
                keep[e] = old == now ? 1.0f : ex2(old - now);
                acc.m[nb][e] = now;
                acc.l[nb][e] *= keep[e];
                keep[e] *= shrink;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc.o[j][nb][i] *= keep[i & 1];
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float zero = zero_of(acc.m[nb][e]);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float& x = s[i / 2][nb][e + 2 * (i & 1)];
                x = ex2(__fsub_rn(x, zero));      // of the rounded logit, as the maximum is
                sum += x;
            }
            acc.l[nb][e] += sum;
        }
    }
    const float w0 = v0 * acc.inv, w1 = v1 * acc.inv;

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
        if (!full) {
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
    if (!full && __any_sync(0xffffffffu, nans != 0)) {
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

// The plan's segment into the queue.  A call of its own: it is rare, and its
// code does not belong between the loads'.
__device__ __noinline__ bool push_segment(const AttendArgs& a, Plan& plan, const Shares& shares, Segment& to) {
    return plan_next(plan, Lookup{a}, a.cut, shares, to);
}

template <int D, int NB>
__global__ void __launch_bounds__(Shape<D, NB>::kThreads, 1)
    kv_attend_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const __grid_constant__ AttendArgs a) {
    constexpr int kStages = Shape<D, NB>::kStages, kStage = Shape<D, NB>::kStage;
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
    __syncthreads();

    // neighbouring shares go to different SMs, so that few units still spread over all of them
    const int share = warp * gridDim.x + blockIdx.x;
    if (lane < 2) a.desc[2 * share + lane].parts = 0;
    Plan& plan = sm.plan[warp];
    const bool together = a.seqs.B > kTogether;
    if (together) {
#pragma unroll 1
        for (int i = warp; i < 32; i += Shape<D, NB>::kWarps) count_units(a, i, lane, sm.counted[i]);
        __syncthreads();
    }
    find_share(a, share, plan, sm.shares[warp], lane, together ? sm.counted : nullptr);

    int flight = 0, from = 0;                 // loads under way; the stage of the first
    uint32_t phase = 0;                       // of that stage
    uint32_t pushed = 0, popped = 0;          // segments
    int key = 0, keys = 0, head = 0;          // of the next load: its first key, its segment's last key + 1 and head
    int b = 0;
    bool over = false;                        // the plan has no more segments
    int blocks[2], ahead = 32;                // page and head of both halves of 32 loads, one in each lane (-1: no page);
                                              // the next load's lane

    // On to the next load; false: there is none, or none before a segment of the queue is done.
    auto settle = [&] {
        while (key >= keys) {
            if (over || pushed - popped == kQueue) return false;
            Segment& s = sm.queue[warp][pushed % kQueue];
            // none: the share is done, or what is left of it are a tile's extra units
            if (!found_for_all(ThisWarp{lane}, [&] { return plan.w.left > 0 && push_segment(a, plan, sm.shares[warp], s); })) {
                over = true;
                return false;
            }
            ++pushed;
            key = s.key0;
            keys = s.keys;
            head = s.head;
            b = s.b;
            ahead = 32;
        }
        if (ahead == 32) {
            const int32_t* row = a.seqs.table + (int64_t)b * a.seqs.width;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = key + kSub * lane + 16 * i;
                const int page = k < keys ? __ldg(row + (k >> a.seqs.page_log2)) : -1;
                const bool ok = page >= 0 && page < a.seqs.num_pages;
                if (k < keys && !ok) atomicOr(&g_device_status, kIndexError);
                blocks[i] = ok ? page * a.cut.heads + head : -1;
            }
            ahead = 0;
        }
        return true;
    };
    bool more = settle();
    auto issue = [&] {
        const int st = from + flight < kStages ? from + flight : from + flight - kStages;
        const int block0 = __shfl_sync(0xffffffffu, blocks[0], ahead), block1 = __shfl_sync(0xffffffffu, blocks[1], ahead);
        const bool ok0 = block0 >= 0, ok1 = block1 >= 0;
        ++ahead;
        uint64_t* bar = &sm.full[warp][st];
        Meta& meta = sm.meta[warp][st];
        if (lane < 4) {
            const int block = lane & 1 ? block1 : block0;
            if (block >= 0) copy_async4(&meta.scale[lane], (lane < 2 ? a.k_scale : a.v_scale) + block);
            arrive_after_copies(bar);
        }
        if (lane == 0) {
            uint8_t* dst = sm.ring[warp] + st * kStage;
            meta.block[0] = block0;
            meta.block[1] = block1;
            if (a.seqs.page_log2 >= 5) {      // both halves lie in one page
                const int slot = key & ((1 << a.seqs.page_log2) - 1);
                mbar_arrive_expect_tx(bar, ok0 ? kStage : 0);
                if (ok0) {
                    tma_load_3d(dst, &k_map, 0, slot, block0, bar);
                    tma_load_3d(dst + kStage / 2, &v_map, 0, slot, block0, bar);
                }
            } else {
                mbar_arrive_expect_tx(bar, (ok0 ? kStage / 2 : 0) + (ok1 ? kStage / 2 : 0));
                if (ok0) {
                    tma_load_3d(dst, &k_map, 0, 0, block0, bar);
                    tma_load_3d(dst + kStage / 2, &v_map, 0, 0, block0, bar);
                }
                if (ok1) {
                    tma_load_3d(dst + kStage / 4, &k_map, 0, 0, block1, bar);
                    tma_load_3d(dst + kStage / 2 + kStage / 4, &v_map, 0, 0, block1, bar);
                }
            }
        }
        ++flight;
        key += kSub;
        more = settle();
    };

    // One turn: the loads that there is room for, then a piece of the segment
    // under way, or the beginning or end of one.  So each part of the code is
    // there once, and the loop stays in the instruction cache.
    uint32_t q[NB][D / 8];
    float f[NB][2];
    int lim[NB][2], all_see = 0;
    Acc<D, NB> acc;
    int at = 0, end = 0;                      // the next piece's first key, the segment's last + 1
    bool open = false;                        // a segment is under way
#pragma unroll 1
    for (;;) {
        while (flight < kStages) {
            if (!more) more = settle();
            if (!more) break;
            issue();
        }
        if (!open) {
            if (popped == pushed) break;
            const Segment& seg = sm.queue[warp][popped % kQueue];
            at = seg.key0;
            end = seg.keys;
            open = true;
            // queries: thread (g, t) holds row g's dims [t D/4, (t + 1) D/4) of each block of 8 rows
            acc.ref = acc.inv = 0.0f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int r = nb * 8 + g;
                uint4 u[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; ++i) u[i] = make_uint4(0, 0, 0, 0);
                if (r < seg.rows) {
                    int token, in_group;
                    row_of(seg, a.cut, r, token, in_group);
                    const uint4* src = reinterpret_cast<const uint4*>(
                        a.q + token * a.q_stride + (seg.head * a.cut.group + in_group) * D + t * (D / 4));
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
                // a row with an infinity is NaN where it sees a key, whatever its products are
                const float back = top == INFINITY ? __int_as_float(0x7fc00000) : down * a.scale_log2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = nb * 8 + 2 * t + i;
                    f[nb][i] = __shfl_sync(0xffffffffu, back, (2 * t + i) * 4);
                    lim[nb][i] = c < seg.rows ? keys_of_row(seg, a.cut, c) : 0;
                    acc.m[nb][i] = -INFINITY;
                    acc.l[nb][i] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc.o[j][nb][i] = 0.0f;
            }
            all_see = keys_of_row(seg, a.cut, 0);           // keys that every row sees
        }
        if (at < end) {
            const int st = from;
            const bool ok = __all_sync(0xffffffffu, wait_for(&sm.full[warp][st], phase, &sm.abort));
            if (!ok) break;
            --flight;
            from = from + 1 == kStages ? 0 : from + 1;
            phase ^= from == 0;
            const uint32_t base_addr = smem_u32(sm.ring[warp] + st * kStage);
            const Meta& meta = sm.meta[warp][st];
            const bool full = at + kSub <= all_see && meta.block[0] >= 0 && meta.block[1] >= 0;
            piece<D, NB>(full, base_addr, base_addr + kStage / 2, meta, q, f, lim, at, end, lane, acc);
            __syncwarp();                     // every lane has read the stage
            at += kSub;
            continue;
        }
        open = false;

        // the rows go out, or to the workspace: thread (g, t) has D/8 dims of rows 2t and 2t + 1
        const Segment& seg = sm.queue[warp][popped % kQueue];
        const bool whole = seg.parts == 1;
        const int slot = seg.owner == share ? 1 : 0;
        float* part = part_of(a, share, slot, D);
        if (!whole && lane == 0) a.desc[2 * share + slot] = PartDesc{seg.parts, seg.owner, seg};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = acc.l[nb][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const float m = acc.m[nb][e];
                const int r = nb * 8 + 2 * t + e;
                if (r >= seg.rows) continue;
                // one after the other: their product may be too small for fp32
                const float by = l == 0.0f ? 0.0f : rcp(l);
                float y[D / 8];
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    y[2 * j] = acc.o[j][nb][e] * by * acc.ref;
                    y[2 * j + 1] = acc.o[j][nb][e + 2] * by * acc.ref;
                }
                if (whole) {
                    const int64_t to = place_of(a, seg, r);
                    uint4* out = reinterpret_cast<uint4*>(a.out + to * D + g * (D / 8));
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
                        out[j] = make_uint4(pack_bf16x2(y[8 * j], y[8 * j + 1]), pack_bf16x2(y[8 * j + 2], y[8 * j + 3]),
                                            pack_bf16x2(y[8 * j + 4], y[8 * j + 5]), pack_bf16x2(y[8 * j + 6], y[8 * j + 7]));
                    if (g == 0 && a.lse) a.lse[to] = kLn2 * log_sum(m, l);
                } else {
                    float4* out = reinterpret_cast<float4*>(part + r * D + g * (D / 8));
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) out[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                    if (g == 0) part[kRows * D + r] = log_sum(m, l);
                }
            }
        }
        __syncwarp();                         // every lane has read the segment
        ++popped;
    }
    check_sequences(a, share, lane);
    if (lane == 0) report_abort(&sm.abort);
    // after a wait that gave up: the loads still under way
    for (; flight; --flight) {
        mbar_wait_drain(&sm.full[warp][from], phase);
        from = from + 1 == kStages ? 0 : from + 1;
        phase ^= from == 0;
    }
}

// Of the largest part's logarithm m and the sum l of 2^(part's - m - kPartsLog2).
__device__ __forceinline__ float join_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : kLn2 * (m + lg2(l * exp2f(kPartsLog2)));
}

// Joins the tiles that borders between shares have cut.  A part holds its own
// keys' mean of the values, not their sum, and its weight is held to add up to
// one at most with the others', so that values up to fp32's largest stay in
// range.  A tile's parts are
// slot 1 of the share that began it (its owner) and slot 0 of the shares after
// it.  Each share has a warp for either slot (or gridDim.y of them).  A tile's
// warps divide its rows; from kMany parts on, a long sequence, the blocks whose
// shares are all slot 0 of it do (there are kMany / 8 - 1 at least), and a
// block's warps divide a row's parts.  What bounds it is the number of
// instructions a row where there are few parts, so that they are loaded four at
// a time, and the loads' latency where there are many: 16 at a time, two rounds
// for the 228 parts of a whole GPU over eight heads.  Measured with blocks from
// 16 parts on: one sequence of 1001 keys 14.3 us, 12.4 from 64 on.
template <int D, int kAhead>
__global__ void __launch_bounds__(256, kAhead == 4 ? 4 : 2) kv_join_kernel(const AttendArgs a) {
    constexpr int kSome = 16, kMany = 64, kDims = D / 32;
    __shared__ float sum_o[8][D];
    __shared__ float2 sum_ml[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, share = blockIdx.x * 8 + warp;
    if (share >= a.shares) return;
    const int64_t next = (int64_t)(2 * (D + 1)) << a.cut.tile_log2;      // from a share's part to the next share's
    const PartDesc& d = a.desc[2 * share + blockIdx.z];
    const int parts = d.parts;
    if (parts == 0) return;
    const Segment seg = d.seg;
    const float* first = part_of(a, d.owner, 1, D);
    const float* sums = (D << a.cut.tile_log2) + first;              // weights of the first part
    const int64_t to_rest = part_of(a, d.owner + 1, 0, D) - next - first;   // part k, k > 0, is k * next further
    if (parts < kSome) {                      // a warp takes a row; four parts at a time, all their loads at once
#pragma unroll 1
        for (int r = share - d.owner + parts * blockIdx.y; r < seg.rows; r += parts * gridDim.y) {
            float m = -INFINITY, l = 0.0f, o[kDims] = {};
#pragma unroll 1
            for (int base = 0; base < parts; base += 4) {
                float w[4], y[4][kDims];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = base + i;
                    const int64_t off = k ? to_rest + k * next : 0;
                    w[i] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < kDims; ++c) y[i][c] = 0.0f;
                    if (k < parts) {
                        w[i] = sums[off + r];
                        const float* src = first + off + r * D + lane * kDims;
                        if constexpr (D == 128) {
                            const float4 v = *reinterpret_cast<const float4*>(src);
                            y[i][0] = v.x; y[i][1] = v.y; y[i][2] = v.z; y[i][3] = v.w;
                        } else {
                            const float2 v = *reinterpret_cast<const float2*>(src);
                            y[i][0] = v.x; y[i][1] = v.y;
                        }
                    }
                }
                const float now = fmaxf(fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])), m);
                const float zero = now == -INFINITY ? 0.0f : now, keep = ex2(m - zero);
                m = now;
                l *= keep;
#pragma unroll
                for (int c = 0; c < kDims; ++c) o[c] *= keep;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = ex2(w[i] - zero - kPartsLog2);
                    l += x;
#pragma unroll
                    for (int c = 0; c < kDims; ++c) o[c] = fmaf(x, y[i][c], o[c]);
                }
            }
            const int64_t to = place_of(a, seg, r);
            const float by = l == 0.0f ? 0.0f : rcp(l);
            uint32_t* out = reinterpret_cast<uint32_t*>(a.out + to * D + lane * kDims);
            if constexpr (D == 128)
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(o[0] * by, o[1] * by), pack_bf16x2(o[2] * by, o[3] * by));
            else
                *out = pack_bf16x2(o[0] * by, o[1] * by);
            if (lane == 0 && a.lse) a.lse[to] = join_lse(m, l);
        }
        return;
    }

    int r = share - d.owner + parts * blockIdx.y, step = parts * gridDim.y, k0 = 0, k1 = parts;
    if (parts >= kMany) {
        const int begin = blockIdx.x * 8, end = d.owner + parts;     // the block's shares; the tile's
        if (begin <= d.owner || begin + 8 > end) return;             // the same for the whole block
        const int at = (d.owner + 8) / 8, blocks = end / 8 - at;     // of this tile
        r = blockIdx.x - at + blocks * blockIdx.y;
        step = blocks * gridDim.y;
        const int per = (parts + 7) / 8;
        k0 = warp * per;
        k1 = k0 + per < parts ? k0 + per : parts;
    }
#pragma unroll 1
    for (; r < seg.rows; r += step) {
        float m = -INFINITY, l = 0.0f, o[kDims] = {};
#pragma unroll 1
        for (int base = k0; base < k1; base += kAhead) {             // the loads of kAhead parts at once
            float y[kAhead][kDims];
            float w = -INFINITY;
            if (lane < kAhead && base + lane < k1) w = sums[(base + lane ? to_rest + (base + lane) * next : 0) + r];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = base + i;
#pragma unroll
                for (int c = 0; c < kDims; ++c) y[i][c] = 0.0f;
                if (k < k1) {
                    const float* src = first + (k ? to_rest + k * next : 0) + r * D + lane * kDims;
                    if constexpr (D == 128) {
                        const float4 v = *reinterpret_cast<const float4*>(src);
                        y[i][0] = v.x; y[i][1] = v.y; y[i][2] = v.z; y[i][3] = v.w;
                    } else {
                        const float2 v = *reinterpret_cast<const float2*>(src);
                        y[i][0] = v.x; y[i][1] = v.y;
                    }
                }
            }
            float now = w;
#pragma unroll
            for (int i = kAhead / 2; i; i >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, i));
            now = fmaxf(__shfl_sync(0xffffffffu, now, 0), m);
            const float zero = now == -INFINITY ? 0.0f : now, keep = ex2(m - zero);
            w = ex2(w - zero - kPartsLog2);
            float all = w;
#pragma unroll
            for (int i = kAhead / 2; i; i >>= 1) all += __shfl_xor_sync(0xffffffffu, all, i);
            l = fmaf(l, keep, __shfl_sync(0xffffffffu, all, 0));
            m = now;
#pragma unroll
            for (int c = 0; c < kDims; ++c) o[c] *= keep;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float x = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
                for (int c = 0; c < kDims; ++c) o[c] = fmaf(x, y[i][c], o[c]);
            }
        }
        if (parts < kMany) {
            const int64_t to = place_of(a, seg, r);
            const float by = l == 0.0f ? 0.0f : rcp(l);
            uint32_t* out = reinterpret_cast<uint32_t*>(a.out + to * D + lane * kDims);
            out[0] = pack_bf16x2(o[0] * by, o[1] * by);
            if constexpr (D == 128) out[1] = pack_bf16x2(o[2] * by, o[3] * by);
            if (lane == 0 && a.lse) a.lse[to] = join_lse(m, l);
            continue;
        }
#pragma unroll
        for (int c = 0; c < kDims; ++c) sum_o[warp][lane * kDims + c] = o[c];
        if (lane == 0) sum_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (threadIdx.x < D / 2) {                                   // two dims a thread
            float top = -INFINITY, total = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) top = fmaxf(top, sum_ml[w].x);
            const float zero = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float by = ex2(sum_ml[w].x - zero);
                const float2 v = *reinterpret_cast<const float2*>(&sum_o[w][2 * threadIdx.x]);
                total = fmaf(by, sum_ml[w].y, total);
                x = fmaf(by, v.x, x);
                y = fmaf(by, v.y, y);
            }
            const int64_t to = place_of(a, seg, r);
            const float by = total == 0.0f ? 0.0f : rcp(total);
            reinterpret_cast<uint32_t*>(a.out + to * D)[threadIdx.x] = pack_bf16x2(x * by, y * by);
            if (threadIdx.x == 0 && a.lse) a.lse[to] = join_lse(top, total);
        }
        __syncthreads();
    }
}

// Rows of a tile: 8 or 16 for the warps of this file, 256 for the
// tensor-memory kernel, whose tiles cost more beside their keys.  On average B
// sequences have T * group / B rows, and a tile reads all their keys.  The rule
// takes the sequences to be alike.  Where they are not, one kernel runs for all of
// them all the same: a prompt of 2048 tokens over 4096 keys beside 127 tokens over
// 4000 keys takes 559 us (40 / 8 heads of 128; 137 and 177 in calls of their own),
// a prompt of 2700 beside 512 tokens over 1000 keys, here in tiles of 16 rows, 740
// (108 and 192), a prompt of 1000 in a batch of 256 places without other tokens 140
// (40 in a batch of one).  Measured on batches of like sequences
// (us; 8 key heads; 256 sequences of up to 300 keys | 64 of up to 2000 | 64 of
// 4096 | 1 of 32768):
//    rows   head_dim 128: 16, 256                           head_dim 64: 16, 256
//      16     -    |    -    | 108, 172 | 27, 37               -   |    -   |  75, 128 | 23, 29
//      24  67, 124 | 59, 73  | 196, 173 | 37, 37            41, 90 | 42, 56 | 129, 128 | 29, 29
//      32  75, 126 | 72, 79  | 196, 174 | 38, 37            46, 90 | 48, 58 | 130, 129 | 29, 29
//      44  93, 125 | 85, 78  |                              56, 93 | 58, 56 |
//      48     -    |    -    | 284, 175 | 52, 38               -   |    -   | 184, 130 | 35, 29
// Of the tiles of 8 and 16: up to 8 rows 104, 105 | 65, 72 for 64 sequences of 4096.
int tile_rows(int group, int64_t B, int64_t T) { return T * group > 32 * B ? 256 : (T * group > 8 * B ? 16 : 8); }

// Shares of the work: warps, or the tensor-memory kernel's blocks.  Fewer than
// 2^kPartsLog2 up to 256 SMs.
int shares_of(int rows, int D, int num_sms) {
    if (rows == 256) return num_sms;
    if (D == 64) return num_sms * (rows == 8 ? Shape<64, 1>::kWarps : Shape<64, 2>::kWarps);
    return num_sms * (rows == 8 ? Shape<128, 1>::kWarps : Shape<128, 2>::kWarps);
}

size_t part_bytes(int rows, int D, int shares) { return ((size_t)shares * 2 * rows * (D + 1) * 4 + 255) / 256 * 256; }

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

cudaError_t launch_join(const AttendArgs& a, int head_dim, cudaStream_t stream) {
    if (a.shares < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // With many parts a tile, as far as the host can tell, 16 of them at a time (1 sequence of 20000 keys, 80 rows, 4 heads:
    // 27.3 us, with 4 at a time 31.4); else 4, and twice the warps on an SM (drafted tokens 35.7 us, with 16 at a time 37.8).
    const int64_t rows = ((int64_t)a.seqs.T * a.cut.group) >> a.cut.tile_log2;
    const bool many = a.shares >= 16 * a.cut.heads * (rows > a.seqs.B ? rows : a.seqs.B);
    auto kernel = many ? (head_dim == 64 ? kv_join_kernel<64, 16> : kv_join_kernel<128, 16>)
                       : (head_dim == 64 ? kv_join_kernel<64, 4> : kv_join_kernel<128, 4>);
    cfg.gridDim = dim3((a.shares + 7) / 8, a.cut.tile_log2 > 4 ? 32 : 1, 2);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_attend_tc(const AttendArgs& a, const uint8_t* k, const uint8_t* v, int head_dim, int blocks,
                                cudaStream_t stream);

size_t kv_attend_workspace(int heads, int head_dim, int q_heads, int64_t B, int64_t T, int num_sms) {
    const int rows = tile_rows(q_heads / heads, B, T), shares = shares_of(rows, head_dim, num_sms);
    return part_bytes(rows, head_dim, shares) + (size_t)shares * 2 * sizeof(PartDesc);
}

cudaError_t launch_kv_attend(const Seqs& seqs, const uint8_t* k, const uint8_t* v, const float* k_scale,
                             const float* v_scale, int heads, int head_dim, const uint16_t* q, int64_t q_stride,
                             int q_heads, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                             int num_sms, cudaStream_t stream) {
    AttendArgs a;
    const int group = q_heads / heads, rows = tile_rows(group, seqs.B, seqs.T);
    a.seqs = seqs;
    // What a tile costs beside its keys, in units.  Tensor-memory kernel: 2, 3, 4, 6, 8 took 660, 560, 515, 522, 532 us
    // for a prompt of 8192 tokens (4 heads of 128, 8 rows each), with heads of 64 458, 425, 430, 438, 446.  Warps: 0, 1, 2,
    // 3, 4, 6 took 39.5, 33.4, 31.6, 31.6, 31.7, 31.6 us for 256 sequences up to 300 keys, 700 short ones 47.5, 41.2,
    // 39.7, 39.6, 40.0, 41.7.
    const int extra = rows == 256 && head_dim == 128 ? 4 : 3;
    a.cut = rows == 256 ? make_cut(heads, group, 8, 7, extra) : make_cut(heads, group, rows == 8 ? 3 : 4, kUnitLog2, extra);
    a.shares = shares_of(rows, head_dim, num_sms);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.q = q;
    a.q_stride = q_stride;
    a.scale_log2 = softmax_scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.part = static_cast<float*>(workspace);
    a.desc = reinterpret_cast<PartDesc*>(static_cast<uint8_t*>(workspace) + part_bytes(rows, head_dim, a.shares));
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
    return e == cudaSuccess ? launch_join(a, head_dim, stream) : e;
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
