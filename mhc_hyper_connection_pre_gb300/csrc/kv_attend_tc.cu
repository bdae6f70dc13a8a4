// kv_attend_tc.cu -- causal attention over the paged e4m3 cache
// (mhc_kv_attend) for many rows a sequence: prompts, chunks of prompts, and
// drafted tokens with many query heads to a key head.
//
// Mathematics.  A block takes 256 rows (new tokens x query heads of one
// key/value head) as two tiles of 128 and walks over the keys 64 at a time:
// S = Q K^T and O += P V on the tensor cores (tcgen05), the softmax between
// them with one thread a row.
//   * K is used as it is stored: S is an 8-bit product.  A query row, divided
//     by a power of two so that its largest element lies in [128, 256), is the
//     sum of two 8-bit numbers an element, hi in e4m3 and lo in e5m2.  What hi
//     leaves of bf16's 8 bits is 0 to 8 of their last place, which e5m2's 3
//     bits hold, down to 2^-14 of the row's largest element (hi's smallest
//     normal number); below that what is lost is at most 2^-13, 2^-20 of the
//     largest.  (lo in e4m3 lost up to 2^-17 of it, from 2^-10 on.)  S = hi K +
//     lo K costs as much tensor time as one f16 product and needs no conversion
//     of K.
//   * V becomes f16 on the way (times its page's scale over the largest scale of
//     the segment, times 2^7: exactly for scales that are powers of two, down to
//     f16's 2^-24, with one rounding for others), because the weights need more
//     than e4m3's 4 bits: they are f16, 2^10 times the softmax's numerators, so
//     that small weights stay out of f16's subnormals.
//   * The running maximum follows only when it has grown by more than 2^5
//     (weights then reach 2^15, within f16), so that O, in tensor memory, is
//     rescaled rarely; sums are fp32 and of the unrounded weights.  Logits are
//     rounded before the maximum is taken off, so that this bound holds however
//     large fp32's steps are at the logits' size.
//
// Up to 128 rows are one tile; both of a block's tiles then take it, each half
// of every load's keys, and their results are joined as the rows go out: 48 rows
// of 64 sequences of 4096 keys, 8 heads, took 231 us with one tile and 203 with
// both (head_dim 128; now 172), 191 and 146 (64; now 130).
//
// What bounds it: 4 * 128 * 64 * head_dim operations for 64 keys and 128 rows on
// the tensor cores against 128 * 64 exponentials and the conversion of V.  Each
// tile's S has two buffers in tensor memory, so that the next step's products
// run during the softmax of this one; the two tiles share loads and conversion.
// With one buffer (128 keys a step) each softmax waited for P V and Q K^T of its
// own tile: 1272 us for a chunk of 4096 tokens over 16384 keys, 40 heads; now
// 920.  A step of both tiles takes about 1900 cycles at head_dim 128.  At the
// tensor cores' rate its products are 1024, which is what their counter shows
// (50% of the time).  S keeps them for longer than that: one product of 64 keys
// by 32 dims is 32 cycles, but reads 4 KB of queries and 2 KB of keys from shared
// memory, 48 cycles at 128 bytes a cycle, so that all products are 1280.  The
// tensor warps' instructions between the products (waits and addresses, 10
// cycles each among the softmax's) and the softmax's own chain take the rest,
// about evenly.  A tile's queries, its first and last steps and
// its rows' way out take 8000 (head_dim 64) to 14,000 cycles on top, which
// bounds short prompts.
//
// With a window (mhc_kv_attend_window) a tile walks over the keys that its rows see, and only
// the steps at either end of the windows are masked: a chunk of 4096 tokens, window 4096, 342 us,
// 1.04 PFLOP/s.
//
// Warps 0-3 and 4-7: softmax of the two tiles; 8-11: V to f16; 12: TMA loads;
// 13 and 15: the tensor instructions of the two tiles; 14: planning.  The
// softmax gets 168 registers a thread and the others 88 of the 128 that 16
// warps start with.
#include "kv_attend.cuh"

namespace mhc {
namespace kv {

namespace {

constexpr int kThreads = 16 * 32;
constexpr int kTile = 128;                    // rows of one tile, and keys of one load
constexpr int kStep = 64;                     // keys of one step
constexpr int kPair = 2 * kTile;              // rows of a block's work
constexpr int kKStages = 3, kVStages = 2;
constexpr int kMetas = 2 * kKStages;          // the softmax reads a load's key scales after its stage is free
constexpr float kVLift = 128.0f;              // V in f16 is 2^7 times code * scale / largest scale
constexpr int kHighEnd = 1024;                // a stretch of kv_index.cuh's Ends is no longer: 256 tokens and two loads
constexpr int kSegs = 4;                      // segments whose value scale and NaNs are kept: the converter runs two ahead

struct __align__(16) Meta {                   // of one load: the scales of each 16 keys, which of them have a page
    float scale[8];
    uint32_t valid;
    int pad[3];
};

template <int D, class Seg>
struct __align__(1024) Smem {
    uint8_t q[2][2][kTile * D];               // tile, hi / lo (e4m3, e5m2)
    uint8_t k[kKStages][kTile * D];
    uint8_t v[kVStages][kTile * D];           // as stored
    uint8_t v16[2][kTile * D * 2];            // f16: 64 dims of every key, then the next 64
    Seg segs[kSegments];
    Plan plan;
    Shares shares;
    int64_t counted[32];
    int count;                                // of segs
    Meta k_meta[kMetas];
    Meta v_meta[kVStages];
    int nan_key[kSegs][D];                    // of the keys that not every row sees: the first with NaN in each dim; with a
                                              // window a bit for each that has NaN, from kHighEnd on those at the windows' ends
    int has_nan[kSegs];
    float ref[kSegs];                         // largest value scale of the segment
    float red[4];
    float2 half[kTile];                       // maximum and sum of a row's odd halves
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t v16_full[2], v16_empty[2], q_full[2], s_full[2][2], p_full[2][2], o_done[2], o_full[2], half_full, half_read, done;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 8-bit numbers, both from shared memory; f16 x f16 with A in tensor memory.
__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t e5m2x4(const float (&x)[8], int at) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[at], x[at + 1]), __NV_SATFINITE, __NV_E5M2);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[at + 2], x[at + 3]), __NV_SATFINITE, __NV_E5M2);
    return lo | (hi << 16);
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Byte offset of 16-byte chunk c of row r in a swizzled tile of rows of D bytes
// (D = 128: 128-byte swizzle, 64: 64-byte), as TMA writes it.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// Columns of tensor memory: S of the two tiles, two buffers each (P takes the
// first half of its S), then O.
__device__ __forceinline__ uint32_t col_s(int x, int buffer) { return x * 2 * kStep + buffer * kStep; }
template <int D>
__device__ __forceinline__ uint32_t col_o(int x) {
    return 4 * kStep + x * D;
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// Ring position of the n-th use of a ring of N stages.
template <int N>
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == N) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// The bits of keys at .. at + 31 of a step that the row sees: those before the
// n-th, in blocks of 16 that have a page.
// (With a window: those from n - window on, or below `sinks` of the step.)
__device__ __forceinline__ uint32_t seen_bits(int at, int n, uint32_t valid) {
    const int k = n - at;
    const uint32_t v = valid >> (at / 16);
    const uint32_t pages = ((v & 1) ? 0xffffu : 0u) | ((v & 2) ? 0xffff0000u : 0u);
    return k <= 0 ? 0u : (k >= 32 ? pages : pages & ((1u << k) - 1));
}

__device__ __forceinline__ uint32_t bits_below(int k) { return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1); }
__device__ __forceinline__ uint32_t window_bits(int at, int n, int window, int sinks) {
    return ~bits_below(n - window - at) | bits_below(sinks - at);
}

// The factor that makes a row's products with 16 keys logits in powers of two.
// Above zero, so that what is hidden stays minus infinity (a scale of zero
// makes logits of 1e-30 instead).
__device__ __forceinline__ float factor(const Meta& meta, int block, float f) {
    return fmaxf(f * meta.scale[block], 1e-37f);
}

// 32 products of a row as logits in powers of two, each rounded, as the maximum
// is: one operation for product and difference would leave an exponent's
// argument above the maximum's by a rounding, and of sharp logits that may be
// any size.
__device__ __forceinline__ void logits(uint32_t (&s)[32], int at, const Meta& meta, float f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float x = factor(meta, at / 16 + h, f);
        const f32x2 xx = make_f32x2(x, x);
#pragma unroll
        for (int i = 16 * h; i < 16 * h + 16; i += 2) {
            float a, b;
            split_f32x2(mul_rn2(make_f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), xx), a, b);
            s[i] = __float_as_uint(a);
            s[i + 1] = __float_as_uint(b);
        }
    }
}

// The largest of 32 logits, from the products: scales are not negative, and
// rounding keeps the order.  (From the logits, after their products, it took the
// chunk of the header from 918 to 943 us, as it then waits for them; this way 920.)
__device__ __forceinline__ float row_max(const uint32_t (&s)[32], int at, const Meta& meta, float f) {
    float top = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float m = __uint_as_float(s[16 * h]);
#pragma unroll
        for (int i = 1; i < 16; ++i) m = fmaxf(m, __uint_as_float(s[16 * h + i]));
        top = fmaxf(top, __fmul_rn(m, factor(meta, at / 16 + h, f)));
    }
    return top;
}

// 32 weights of a row, as 16 pairs of f16, added to the row's two sums.
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint32_t (&p)[16], float zero, f32x2& sum) {
    const f32x2 z = make_f32x2(-zero, -zero);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float a, b;
        split_f32x2(add_rn2(make_f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), z), a, b);
        a = ex2(a);
        b = ex2(b);
        sum = add_rn2(sum, make_f32x2(a, b));
        p[i / 2] = pack_f16x2(a, b);
    }
}

// The power of two, within 2^+-120, that brings a row's largest magnitude to [128, 256).
__device__ __forceinline__ float power_up(float top) {
    int e = 134 - (int)(__float_as_uint(top) >> 23);              // 7 - floor(log2(top))
    e = e < -120 ? -120 : (e > 120 ? 120 : e);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// Steps of a tile for so many keys.  `split`: up to 128 rows, which both tiles
// take, the first the even and the second the odd 64 keys of each load.
__device__ __forceinline__ int steps_of(bool split, int keys) {
    return split ? (keys + kTile - 1) / kTile : (keys + kStep - 1) / kStep;
}

// NaN for 32 dims (from c * 32 on) of the row that sees the segment's keys up to the n-th, where a
// value among those that not every row sees is NaN.  Rare, so the codes of the keys that have NaN are read once
// more: which rows see which keys differs at both ends of a window, and would need a set of keys for each dim.
// 512 tokens of 40 / 8 heads of 128 over 5000 keys, window 4096: 69 us without NaN, 88 with one value at the windows'
// end; 5381 with all of the segment's codes read again.
template <int D, class C>
__device__ __noinline__ void nan_dims(const AttendArgs<C>& a, const WindowSegment& s, const int* marks, int c, int n,
                                      uint32_t& mask) {
    const int log2 = a.seqs.page_log2;
    const int32_t* row = a.seqs.table + (int64_t)s.b * a.seqs.width;
    const Ends ends = ends_of(s, a.cut);
    mask = 0;
#pragma unroll 1
    for (int w = 0; w < 2 * kHighEnd / 32; ++w)
#pragma unroll 1
        for (uint32_t left = marks[w]; left; left &= left - 1) {
            const int bit = 32 * w + __ffs(left) - 1, key = bit < kHighEnd ? ends.low + bit : ends.high + bit - kHighEnd;
            const int place = place_of_key(s, key), page = __ldg(row + (place >> log2));
            if (page < 0 || page >= a.seqs.num_pages) continue;
            const uint8_t* from =
                a.cut.v + ((((int64_t)page * a.cut.heads + s.head) << log2) + (place & ((1 << log2) - 1))) * D + c * 32;
            uint32_t found = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = nan_bytes(__ldg(reinterpret_cast<const uint32_t*>(from) + i)) >> 7;
                found |= ((x & 1) | (x >> 7 & 2) | (x >> 14 & 4) | (x >> 21 & 8)) << (4 * i);
            }
            if (key_seen(key, n, a.cut)) mask |= found;
        }
}

template <int D, class C>
__device__ __forceinline__ void put_nans(const AttendArgs<C>& a, const WindowSegment& s, const int* marks, int c, int n,
                                         uint32_t (&o)[32]) {
    static_assert(2 * kHighEnd <= 32 * D, "a bit for each key of both ends");
    uint32_t mask;
    nan_dims<D>(a, s, marks, c, n, mask);
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if ((mask >> i) & 1) o[i] = 0x7fc00000u;
}

template <int D, class C>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attend_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                        const AttendArgs<C> a) {
    extern __shared__ uint8_t raw[];
    using Seg = typename SegmentOf<C::kWindow>::type;
    using Shared = Smem<D, Seg>;
    Shared& sm = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kStep >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel waits for this one's end
    if (tid == 0) {
        sm.abort = 0;
        for (int i = 0; i < kKStages; ++i) mbar_init(&sm.k_full[i], 1 + 8), mbar_init(&sm.k_empty[i], 2);
        for (int i = 0; i < kVStages; ++i) mbar_init(&sm.v_full[i], 1 + 8), mbar_init(&sm.v_empty[i], 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.v16_full[i], 4);
            mbar_init(&sm.v16_empty[i], 2);
            mbar_init(&sm.q_full[i], 4);
            for (int b = 0; b < 2; ++b) mbar_init(&sm.s_full[i][b], 1), mbar_init(&sm.p_full[i][b], 4);
            mbar_init(&sm.o_done[i], 1);
            mbar_init(&sm.o_full[i], 1);
        }
        mbar_init(&sm.half_full, 4);
        mbar_init(&sm.half_read, 4);
        mbar_init(&sm.done, 2);
        fence_mbar_init_cluster();
    }
    if (warp == 13) tmem_alloc(&sm.tmem, 512);
    if (tid < 2) a.desc[2 * blockIdx.x + tid].parts = 0;
    const bool together = a.seqs.B > kTogether;
    if (together) {
#pragma unroll 1
        for (int i = warp; i < 32; i += kThreads / 32) count_units(a, i, lane, sm.counted[i]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    // Runs a role over this block's segments, kSegments at a time; `plan` finds
    // them (warp 14).
    auto each_segments = [&](auto&& plan, auto&& role) {
#pragma unroll 1
        for (;;) {
            plan();
            block_sync();
            if (sm.count == 0) break;
            role();
            __syncwarp();
            block_sync();                     // before the next segments are planned
        }
    };
    const auto others = [] {};

    // counters of each role, over all segments
    Ring<kKStages> kr;
    Ring<kMetas> mr;
    Ring<kVStages> vr;
    Ring<2> v16r;
    uint32_t segs = 0;                        // segments with keys
    uint32_t phases = 0;                      // of a tile's s_full or p_full: a bit for each buffer
    uint32_t products = 0, halves = 0;        // P V of a softmax warp's tile so far; segments in halves
    bool unread = false;                      // tile 0 may still read this tile's last O
    uint32_t k_loads = 0, v_loads = 0;

    if (warp < 8) {
        // ------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        each_segments(others, [&] {
            const int x = warp / 4, in_tile = (warp % 4) * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(warp % 4) << 21);
            bool ok = true;
            for (int index = 0; ok && index < sm.count; ++index) {
                const Seg seg = sm.segs[index];
                const int rows = seg.rows;
                const bool split = rows <= kTile;
                const int mine = split ? in_tile : x * kTile + in_tile;              // of the block's rows
                const int key0 = seg.key0, keys = seg.keys;
                const int steps = steps_of(split, keys - key0);      // 0: a tile without keys
                float f = 0.0f, m = -INFINITY, l = 0.0f;
                int lim = 0;
                if (steps > 0) {
                    // the warp's 32 query rows as hi + lo: D / 8 lanes to a row, so that the loads
                    // are whole lines (a thread to a row took 7400 to 12,600 cycles at head_dim
                    // 128, this takes 6000 to 7700)
                    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = 4;
                    const int sub = lane / kLanes, part8 = lane % kLanes;
                    const int in_rows = rows - (mine - lane);     // of the warp's 32, those that there are
                    int64_t off = 0;
                    if (mine < rows) {
                        int token, in_group;
                        row_of(seg, a.cut, mine, token, in_group);
                        lim = keys_of_row(seg, a.cut, mine);
                        off = token * a.q_stride + (seg.head * a.cut.group + in_group) * D;
                    }
                    auto load = [&](int r) {
                        const int64_t from = __shfl_sync(0xffffffffu, off, r & 31) + part8 * 8;
                        return r < in_rows && r < 32 ? __ldg(reinterpret_cast<const uint4*>(a.q + from))
                                                     : make_uint4(0, 0, 0, 0);
                    };
                    const uint32_t hi_at = smem_u32(sm.q[x][0]), lo_at = smem_u32(sm.q[x][1]);
                    float my_top = 0.0f;
                    uint4 u[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) u[k] = load(k * kRows + sub);
#pragma unroll 1
                    for (int r0 = 0; r0 < 32; r0 += kAhead * kRows) {
                        uint4 now[kAhead];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            now[k] = u[k];
                            u[k] = load(r0 + (kAhead + k) * kRows + sub);
                        }
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const int r = r0 + k * kRows + sub;
                            float y[8], z[8], top = 0.0f;
                            unpack8(now[k], y);
#pragma unroll
                            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
#pragma unroll
                            for (int o = kLanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            const float up = power_up(top);
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] *= up;
                            const uint32_t hi[2] = {e4m3x4(y, 0), e4m3x4(y, 4)};
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                const uint32_t b = i % 4 ? cvt_hi(hi[i / 4]) : cvt_lo(hi[i / 4]);
                                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&b));
                                z[i] = y[i] - back.x;
                                z[i + 1] = y[i + 1] - back.y;
                            }
                            const uint32_t to = chunk_at<D>(in_tile - lane + r, part8 / 2) + (part8 & 1) * 8;
                            sts64(hi_at + to, hi[0], hi[1]);
                            sts64(lo_at + to, e5m2x4(z, 0), e5m2x4(z, 4));
                            const float t = __shfl_sync(0xffffffffu, top, (lane % kRows) * kLanes);
                            if (lane - lane % kRows == r - sub) my_top = t;
                        }
                    }
                    f = a.scale_log2 * __uint_as_float(0x7f000000u - __float_as_uint(power_up(my_top)));
                    // e4m3 has no infinity: such a row is NaN, if it sees a key
                    if (my_top == INFINITY && lim > 0) l = __int_as_float(0x7fc00000);
                    fence_proxy_async_smem();
                    if (unread) {             // the last segment's reads of O come before this one's products
                        ok = __all_sync(0xffffffffu, wait_for(&sm.half_read, (halves - 1) & 1, &sm.abort));
                        if (!ok) break;
                        unread = false;
                        tc_fence_after();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.q_full[x]);
                }

                const int all_see = keys_of_row(seg, a.cut, split ? 0 : x * kTile);
                [[maybe_unused]] int last_sees = 0;
                if constexpr (C::kWindow)
                    last_sees = keys_of_row(seg, a.cut, split || rows < (x + 1) * kTile ? rows - 1 : (x + 1) * kTile - 1);
                for (int j = 0; j < steps; ++j) {
                    const int buffer = j & 1, half = kStep * (split ? x : buffer);   // of the load
                    ok = __all_sync(0xffffffffu, wait_for(&sm.s_full[x][buffer], (phases >> buffer) & 1, &sm.abort));
                    if (!ok) break;
                    phases ^= 1u << buffer;
                    tc_fence_after();
                    const Meta& meta = sm.k_meta[mr.stage];
                    const int key = key0 + (split ? j * kTile : (j & ~1) * kStep) + half;
                    const int n = lim - key;  // keys of this step that the row sees
                    const uint32_t valid = meta.valid >> (half / 16);
                    const uint32_t from = lanes + col_s(x, buffer);
                    // the row's 64 products: their largest, the logits, the weights and their sum
                    uint32_t s[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_ld32(from + c * 32, s[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_regs_ready(s[c]);
                    bool part = key + kStep > all_see || (valid & 0xfu) != 0xfu;
                    if constexpr (C::kWindow) part = part || !keys_all_seen(key, kStep, all_see, last_sees, a.cut);
                    if (part) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t bits = seen_bits(c * 32, n, valid);
                            if constexpr (C::kWindow) bits &= window_bits(c * 32, n, a.cut.window, a.cut.sinks - key);
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[c][i] = (bits >> i) & 1 ? s[c][i] : 0xff800000u;
                        }
                    }
                    const float top = fmaxf(row_max(s[0], half, meta, f), row_max(s[1], half + 32, meta, f));
#pragma unroll
                    for (int c = 0; c < 2; ++c) logits(s[c], half + c * 32, meta, f);
                    const bool grow = top - m > kGrow;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float keep = grow ? ex2(m - top) : 1.0f;
                        m = grow ? top : m;
                        l *= keep;
                        // after the last step's P V; the one before it is done, as S of this step came after
                        // it, so that the phase's parity tells
                        if (j > 0) {
                            ok = __all_sync(0xffffffffu, wait_for(&sm.o_done[x], (products + j - 1) & 1, &sm.abort));
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(lanes + col_o<D>(x) + c * 32, o);
                                tmem_wait_ld();
                                tmem_regs_ready(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                                tmem_st32(lanes + col_o<D>(x) + c * 32, o);
                            }
                        }
                    }
                    const float zero = zero_of(m);
                    f32x2 sum = make_f32x2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t p[16];
                        weights(s[c], p, zero, sum);
                        tmem_st16(from + c * 16, p);
                    }
                    float sum0, sum1;
                    split_f32x2(sum, sum0, sum1);
                    l += sum0 + sum1;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[x][buffer]);
                    if (split || buffer || j + 1 == steps) mr.next();
                }
                if (!ok) break;
                if (steps > 0) {
                    products += steps - 1;    // the last one completes o_full
                    ok = __all_sync(0xffffffffu, wait_for(&sm.o_full[x], segs & 1, &sm.abort));
                    if (!ok) break;
                    tc_fence_after();
                }
                // tile 0 brings the halves of the keys together
                const bool join = split && steps > 0;
                float own = 1.0f, other = 0.0f;       // weights of the two O
                if (join) {
                    if (x == 1) {
                        sm.half[in_tile] = make_float2(m, l);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.half_full);
                        unread = true;
                    } else {
                        ok = __all_sync(0xffffffffu, wait_for(&sm.half_full, halves & 1, &sm.abort));
                        if (!ok) break;
                        tc_fence_after();
                        const float2 ml = sm.half[in_tile];
                        const float top = fmaxf(m, ml.x), zero = top == -INFINITY ? 0.0f : top;
                        own = ex2(m - zero);
                        other = ex2(ml.x - zero);
                        m = top;
                        l = l * own + ml.y * other;
                    }
                    ++halves;
                }
                if (split && x == 1) {
                    segs += steps > 0;
                    continue;
                }

                // the rows go out
                const bool whole = seg.parts == 1;
                const int slot = seg.owner == blockIdx.x ? 1 : 0;
                if (!whole && tid == 0) a.desc[2 * blockIdx.x + slot] = PartDesc{seg.parts, seg.owner, seg};
                const int64_t at = mine < rows ? place_of(a, seg, mine) : 0;
                float* part = part_of(a, blockIdx.x, slot, D);
                const int kept = segs % kSegs;
                const float unit = steps > 0 ? sm.ref[kept] * (1.0f / kVLift) : 0.0f;
                const float by = l == 0.0f ? 0.0f : rcp(l);     // apart from the unit: their product may be too
                                                                    // small for fp32
                const bool nans = steps > 0 && sm.has_nan[kept];
                own *= by;
                other *= by;
                // Rows go out by way of shared memory, 128 bytes of each of the warp's 32 at a time, so that
                // the stores are whole lines.  The queries' place is free, and its rows are this warp's.
                uint64_t to = 0;
                if (mine < rows) {
                    to = whole ? reinterpret_cast<uint64_t>(a.out + at * D) : reinterpret_cast<uint64_t>(part + mine * D);
                    if (whole && a.lse) a.lse[at] = kLn2 * log_sum(m, l);
                    if (!whole) part[kPair * D + mine] = log_sum(m, l);
                }
                auto staged = [&](int r, int c) {             // 16-byte chunk c of row r of the warp
                    const uint32_t row = D == 128 ? smem_u32(sm.q[x][0]) + (warp % 4) * 4096 + r * 128
                                                  : smem_u32(sm.q[x][r / 16]) + (warp % 4) * 2048 + (r % 16) * 128;
                    return row + ((c ^ (r & 7)) << 4);
                };
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (steps > 0) {
                        tmem_ld32(lanes + col_o<D>(x) + c * 32, o);
                        tmem_wait_ld();
                        tmem_regs_ready(o);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = steps > 0 ? __float_as_uint(__uint_as_float(o[i]) * own) : 0u;
                    if (join) {
                        uint32_t o1[32];
                        tmem_ld32(lanes + col_o<D>(1) + c * 32, o1);
                        tmem_wait_ld();
                        tmem_regs_ready(o1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), other, __uint_as_float(o[i])));
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * unit);
                    if constexpr (C::kWindow) {
                        if (nans) put_nans<D>(a, sm.segs[index], sm.nan_key[kept], c, lim, o);
                    } else if (nans) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (sm.nan_key[kept][c * 32 + i] < lim) o[i] = 0x7fc00000u;
                    }
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(o[8 * i + k]);
                            sts128(staged(lane, (c & 1) * 4 + i), pack8(y));
                        }
                        if (!(c & 1)) continue;
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sts128(staged(lane, i), make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int r = lane / 8; r < 32; r += 4) {
                        const uint64_t row = __shfl_sync(0xffffffffu, to, r);
                        const uint4 v = lds128(staged(r, lane % 8));
                        if (row) *reinterpret_cast<uint4*>(row + lane % 8 * 16) = v;
                    }
                    __syncwarp();
                    if (to) to += 128;
                }
                if (join) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.half_read);
                }
                segs += steps > 0;
            }
        });
    } else if (warp < 12) {
        // ------------------------------------------------- values to f16
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        each_segments(others, [&] {
            const int id = tid - 256;         // this thread's key of a step
            bool ok = true;                   // after a wait that gave up all go on to the barriers, without work
            for (int index = 0; index < sm.count; ++index) {
                const Seg seg = sm.segs[index];
                const int key0 = seg.key0, keys = seg.keys;
                if (keys <= key0) continue;
                const int slot = segs++ % kSegs, log2 = a.seqs.page_log2;
                const int32_t* row = a.seqs.table + (int64_t)seg.b * a.seqs.width;
                float most = 0.0f;
                for (int i = (key0 >> log2) + id; i << log2 < keys; i += 128) {
                    int at = i;
                    if constexpr (C::kWindow) {
                        const int place = place_of_key(seg, i << log2);
                        if (!page_seen(place, first_seen(seg, a.cut), a.cut.sinks, log2)) continue;
                        at = place >> log2;
                    }
                    const int page = __ldg(row + at);
                    if (page >= 0 && page < a.seqs.num_pages)
                        most = fmaxf(most, __ldg(a.v_scale + (int64_t)page * a.cut.heads + seg.head));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (lane == 0) sm.red[warp - 8] = most;
                for (int i = id; i < D; i += 128) sm.nan_key[slot][i] = C::kWindow ? 0 : 0x7fffffff;
                if (id == 0) sm.has_nan[slot] = 0;
                named_bar_sync(1, 128);
                most = value_unit(fmaxf(fmaxf(sm.red[0], sm.red[1]), fmaxf(sm.red[2], sm.red[3])));
                if (id == 0) sm.ref[slot] = most;
                named_bar_sync(1, 128);
                const float per = most > 0.0f ? __frcp_rn(most) : 0.0f;
                const int all_see = keys_of_row(seg, a.cut, 0);
                // whether every row sees `count` keys from `key` on
                auto all = [&](int key, int count) {
                    if constexpr (C::kWindow)
                        return keys_all_seen(key, count, all_see, keys_of_row(seg, a.cut, seg.rows - 1), a.cut);
                    else return key + count <= all_see;
                };
                for (int key = key0; ok && key < keys; key += kTile) {
                    ok = __all_sync(0xffffffffu, wait_for(&sm.v_full[vr.stage], vr.phase, &sm.abort)) &&
                         __all_sync(0xffffffffu, wait_for(&sm.v16_empty[v16r.stage], v16r.phase ^ 1, &sm.abort));
                    if (!ok) break;
                    const Meta& meta = sm.v_meta[vr.stage];
                    const uint32_t src = smem_u32(sm.v[vr.stage]), dst = smem_u32(sm.v16[v16r.stage]);
                    const bool use = ((meta.valid >> (id / 16)) & 1) && key + id < keys;
                    const float ratio = use ? meta.scale[id / 16] * per * kVLift : 0.0f;
                    // 64 dims of a key are one 128-byte row, swizzled; the next 64 dims follow all keys
                    auto put = [&](int c, const uint32_t (&h)[8]) {
                        const uint32_t to_row = dst + (c / 4) * (kTile * 128) + id * 128;
                        const int c16 = (2 * c) % 8;
                        sts128(to_row + ((c16 ^ (id & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                        sts128(to_row + (((c16 + 1) ^ (id & 7)) << 4), make_uint4(h[4], h[5], h[6], h[7]));
                    };
                    // a power of two, as mhc_kv_append writes them: exact, or one rounding in f16's subnormals
                    const bool exact = (__float_as_uint(ratio) & 0x7fffffu) == 0 && ratio >= 5.9604645e-8f;
                    if (__all_sync(0xffffffffu, exact && all(key, kTile))) {
                        const uint32_t times = pack_f16x2(ratio, ratio);
#pragma unroll 1
                        for (int c0 = 0; c0 < D / 16; c0 += 4) {
                            uint4 u[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) u[i] = lds128(src + chunk_at<D>(id, c0 + i));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                                uint32_t h[8];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    h[2 * k] = mul_f16x2(cvt_lo(w[k]), times);
                                    h[2 * k + 1] = mul_f16x2(cvt_hi(w[k]), times);
                                }
                                put(c0 + i, h);
                            }
                        }
                    } else {                  // any scales, and keys that not every row sees
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            const uint4 u = lds128(src + chunk_at<D>(id, c));
                            uint32_t w[4] = {u.x, u.y, u.z, u.w}, h[8];
                            if (!use) w[0] = w[1] = w[2] = w[3] = 0;
                            if (!all(key + id, 1)) {
                                // NaN must reach only the rows that see this key, but 0 * NaN is
                                // NaN: it is taken out here and put back as the rows go out
                                uint32_t any = 0;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t n = nan_bytes(w[k]);
                                    any |= n;
                                    w[k] &= ~((n >> 7) * 0xffu);
                                }
                                if (any) {
                                    sm.has_nan[slot] = 1;
                                    if constexpr (C::kWindow) {
                                        const Ends ends = ends_of(seg, a.cut);
                                        const int k = key + id, bit = k < ends.low_end && k >= ends.low ? k - ends.low
                                                                                                        : kHighEnd + k - ends.high;
                                        atomicOr(&sm.nan_key[slot][bit >> 5], 1 << (bit & 31));
                                    } else {
#pragma unroll 1
                                        for (int b = 0; b < 16; ++b)
                                            if ((sm.v[vr.stage][chunk_at<D>(id, c) + b] & 0x7f) == 0x7f)
                                                atomicMin(&sm.nan_key[slot][16 * c + b], key + id);
                                    }
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t x = k % 2 ? cvt_hi(w[k / 2]) : cvt_lo(w[k / 2]);
                                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x));
                                h[k] = pack_f16x2(y.x * ratio, y.y * ratio);
                            }
                            put(c, h);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.v16_full[v16r.stage]);
                        mbar_arrive(&sm.v_empty[vr.stage]);
                    }
                    vr.next();
                    v16r.next();
                }
            }
        });
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 12) {
            // ----------------------------------------------------------- TMA
            each_segments(others, [&] {
                const int log2 = a.seqs.page_log2, per_box = 1 << (log2 - 4);
                bool ok = true;
                for (int index = 0; ok && index < sm.count; ++index) {
                    const Seg seg = sm.segs[index];
                    const int key0 = seg.key0, keys = seg.keys;
                    const int32_t* row = a.seqs.table + (int64_t)seg.b * a.seqs.width;
                    // this lane's 16 keys of a step: whether their page is looked at, and which it is
                    auto looked = [&](int key) {
                        bool look = lane < 8 && key + 16 * lane < keys;
                        if constexpr (C::kWindow)
                            look = look && page_seen(place_of_key(seg, key + 16 * lane), first_seen(seg, a.cut),
                                                     a.cut.sinks, log2);
                        return look;
                    };
                    auto page_at = [&](int key) {
                        int place = key + 16 * lane;
                        if constexpr (C::kWindow) place = place_of_key(seg, place);
                        return looked(key) ? __ldg(row + (place >> log2)) : -1;
                    };
                    int page = page_at(key0);
                    for (int key = key0; key < keys; key += kTile) {
                        const int ahead = page_at(key + kTile);
                        const bool has = page >= 0 && page < a.seqs.num_pages;
                        if (looked(key) && !has) atomicOr(&g_device_status, kIndexError);
                        const uint32_t valid = __ballot_sync(0xffffffffu, lane < 8 && has);
                        const bool box = lane < 8 && has && (lane & (per_box - 1)) == 0;
                        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box)) * D << log2;
                        const int block = has ? page * a.cut.heads + seg.head : 0;

                        ok = __all_sync(0xffffffffu, wait_for(&sm.k_empty[kr.stage], kr.phase ^ 1, &sm.abort));
                        if (!ok) break;
                        if (lane == 0) {
                            sm.k_meta[mr.stage].valid = valid;
                            mbar_arrive_expect_tx(&sm.k_full[kr.stage], bytes);
                        }
                        __syncwarp();
                        if (lane < 8) {
                            if (has) copy_async4(&sm.k_meta[mr.stage].scale[lane], a.k_scale + block);
                            arrive_after_copies(&sm.k_full[kr.stage]);
                        }
                        if (box) tma_load_3d(sm.k[kr.stage] + lane * 16 * D, &k_map, 0, 0, block, &sm.k_full[kr.stage]);
                        ++k_loads;
                        ok = __all_sync(0xffffffffu, wait_for(&sm.v_empty[vr.stage], vr.phase ^ 1, &sm.abort));
                        if (!ok) break;
                        if (lane == 0) {
                            sm.v_meta[vr.stage].valid = valid;
                            mbar_arrive_expect_tx(&sm.v_full[vr.stage], bytes);
                        }
                        __syncwarp();
                        if (lane < 8) {
                            if (has) copy_async4(&sm.v_meta[vr.stage].scale[lane], a.v_scale + block);
                            arrive_after_copies(&sm.v_full[vr.stage]);
                        }
                        if (box) tma_load_3d(sm.v[vr.stage] + lane * 16 * D, &v_map, 0, 0, block, &sm.v_full[vr.stage]);
                        ++v_loads;
                        kr.next();
                        mr.next();
                        vr.next();
                        page = ahead;
                    }
                }
            });
        } else if (warp != 14) {
            // ------------------------------- tensor instructions of one tile
            // The whole warp runs the loop, so that the addresses stay in uniform
            // registers, and one elected lane issues.  A warp for each tile: the
            // issue of a step's twelve products takes longer than the products.
            const int x = warp == 13 ? 0 : 1;
            const uint64_t q_desc[2] = {smem_desc(smem_u32(sm.q[x][0]), 16, D * 8, D == 128 ? 2 : 4),
                                        smem_desc(smem_u32(sm.q[x][1]), 16, D * 8, D == 128 ? 2 : 4)};
            const uint64_t k_desc = smem_desc(smem_u32(sm.k[0]), 16, D * 8, D == 128 ? 2 : 4);
            // values: dims contiguous ("MN-major"); 64 dims a 128-byte row, 8 keys an atom, 64 further dims 16 KB on
            const uint64_t v_desc = smem_desc(smem_u32(sm.v16[0]), kTile * 128, 1024, 2);
            const uint32_t s_col = tmem + col_s(x, 0), o_col = tmem + col_o<D>(x);
            each_segments(others, [&] {
                const int segments = __shfl_sync(0xffffffffu, sm.count, 0);
                bool ok = true;
#pragma unroll 1
                for (int index = 0; ok && index < segments; ++index) {
                    const bool split = __shfl_sync(0xffffffffu, sm.segs[index].rows, 0) <= kTile;
                    const int steps =
                        steps_of(split, __shfl_sync(0xffffffffu, sm.segs[index].keys - sm.segs[index].key0, 0));
                    if (steps <= 0) continue;
                    // O with the weights of step j, then S of step j + 2 into their buffer
#pragma unroll 1
                    for (int j = -2; j < steps; ++j) {
                        const int buffer = j & 1, next = j + 2;
                        const bool has_o = j >= 0, has_s = next < steps;
                        const int half = split ? x : buffer;          // of the load
                        const bool last_o = has_o && (split || buffer || j + 1 == steps);     // the last use of its load
                        const bool last_s = has_s && (split || buffer || next + 1 == steps);
                        // first what is there already, as a rule, then the weights: nothing else lies between
                        // them and the products
                        if (has_s && (split || buffer == 0)) ok = wait_for(&sm.k_full[kr.stage], kr.phase, &sm.abort);
                        if (next == 0) ok = ok && wait_for(&sm.q_full[x], segs & 1, &sm.abort);
                        if (has_o && (split || buffer == 0)) ok = ok && wait_for(&sm.v16_full[v16r.stage], v16r.phase, &sm.abort);
                        const uint64_t vd = v_desc + v16r.stage * (kTile * D * 2 / 16) + half * (kStep * 128 / 16);
                        const uint64_t kd = k_desc + kr.stage * (kTile * D / 16) + half * (kStep * D / 16);
                        if (has_o) ok = ok && wait_for(&sm.p_full[x][buffer], (phases >> buffer) & 1, &sm.abort);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            if (has_o) {
#pragma unroll
                                for (int i = 0; i < kStep / 16; ++i)
                                    mma_f16_ts(o_col, s_col + buffer * kStep + 8 * i, vd + 128 * i, kIdescO, j > 0 || i > 0);
                                mma_commit(j + 1 < steps ? &sm.o_done[x] : &sm.o_full[x]);
                            }
                            if (has_s) {      // 64 of the load's keys
#pragma unroll
                                for (int h = 0; h < 2; ++h)
#pragma unroll
                                    for (int i = 0; i < D / 32; ++i)
                                        mma_8bit(s_col + buffer * kStep, q_desc[h] + 2 * i, kd + 2 * i,
                                                 kIdescS | (uint32_t)h << 7, h + i > 0);      // A: e4m3, e5m2
                                mma_commit(&sm.s_full[x][buffer]);
                            }
                            if (last_o) mma_commit(&sm.v16_empty[v16r.stage]);
                            if (last_s) mma_commit(&sm.k_empty[kr.stage]);
                        }
                        __syncwarp();
                        if (has_o) phases ^= 1u << buffer;
                        if (last_o) v16r.next();
                        if (last_s) kr.next();
                    }
                    ++segs;
                }
            });
        } else {
            // ------------------------------------------------------ planning
            find_share(a, blockIdx.x, sm.plan, sm.shares, lane, together ? sm.counted : nullptr);
            each_segments(
                [&] {
                    if (lane == 0) {
                        int n = 0;
#pragma unroll 1
                        while (n < kSegments && plan_next(sm.plan, Lookup<C>{a}, a.cut, sm.shares, sm.segs[n])) ++n;
                        sm.count = n;
                    }
                },
                others);
            check_sequences(a, blockIdx.x, lane);
        }
    }

    // Everything asynchronous has ended before the block does: the products by
    // their last commit, and, after a wait that gave up, the loads under way.
    if (warp == 13 || warp == 15) {
        if (elect_one()) mma_commit(&sm.done);
        mbar_wait_drain(&sm.done, 0);
    }
    if (warp == 12 && lane == 0 && sm.abort) {
        for (uint32_t i = k_loads > kKStages ? k_loads - kKStages : 0; i < k_loads; ++i)
            mbar_wait_drain(&sm.k_full[i % kKStages], (i / kKStages) & 1);
        for (uint32_t i = v_loads > kVStages ? v_loads - kVStages : 0; i < v_loads; ++i)
            mbar_wait_drain(&sm.v_full[i % kVStages], (i / kVStages) & 1);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13) tmem_dealloc(tmem, 512);
    if (tid == 0) report_abort(&sm.abort);
}

template <int D, class C>
cudaError_t launch(const AttendArgs<C>& a, const uint8_t* k, const uint8_t* v, int blocks, cudaStream_t stream) {
    CUtensorMap k_map, v_map;
    const int64_t pages = (int64_t)a.seqs.num_pages * a.cut.heads;
    if (!encode_codes(&k_map, k, pages, 1 << a.seqs.page_log2, D, kTile) ||
        !encode_codes(&v_map, v, pages, 1 << a.seqs.page_log2, D, kTile))
        return cudaErrorInvalidValue;
    using Shared = Smem<D, typename SegmentOf<C::kWindow>::type>;
    const int bytes = (int)sizeof(Shared) + 1024;
    static_assert(sizeof(Shared) + 1024 <= 227 * 1024, "shared memory of a block");
    const cudaError_t e = cudaFuncSetAttribute(kv_attend_tc_kernel<D, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kv_attend_tc_kernel<D, C><<<blocks, kThreads, bytes, stream>>>(k_map, v_map, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attend_tc(const AttendArgs<Cut>& a, const uint8_t* k, const uint8_t* v, int head_dim, int blocks,
                                cudaStream_t stream) {
    return head_dim == 64 ? launch<64>(a, k, v, blocks, stream) : launch<128>(a, k, v, blocks, stream);
}

cudaError_t launch_kv_attend_tc(const AttendArgs<WindowWork>& a, const uint8_t* k, const uint8_t* v, int head_dim,
                                int blocks, cudaStream_t stream) {
    return head_dim == 64 ? launch<64>(a, k, v, blocks, stream) : launch<128>(a, k, v, blocks, stream);
}

cudaError_t read_attend_tc_status(unsigned int* status) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof v);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace kv
}  // namespace mhc
