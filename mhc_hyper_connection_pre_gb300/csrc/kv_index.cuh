// kv_index.cuh -- where the new tokens of a call lie in the paged cache: the
// index arithmetic of the kv kernels, free of device code so that it can be
// compiled and checked on the host as well.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MHC_HD __host__ __device__ __forceinline__
#else
#define MHC_HD inline
#endif

namespace mhc {
namespace kv {

// A call's lengths and pages, as given (unchecked device data).
struct Seqs {
    const int32_t* table;   // [B][width]
    const int32_t* lens;    // [B]
    const int32_t* cu;      // [B + 1] or null: one token each
    int width;              // pages of a table row
    int B, T;
    int page_tokens;
    int num_pages;
};

// Sequence b's new tokens [begin, end), its length with them, and how many
// keys precede the first new token (negative: that many new tokens have no
// place).  Everything is clamped to what the call's arrays hold, whatever the
// device data say; `bad` is set when a clamp changed something.
struct Span {
    int begin, end, len, before;
    bool bad;
};

MHC_HD int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

MHC_HD Span span_of(const Seqs& s, int b) {
    Span r;
    const int cap = s.width * s.page_tokens;      // at most 2^30 (checked on the host)
    int begin, end;
    if (s.cu) {
        const int c0 = s.cu[b], c1 = s.cu[b + 1];
        begin = clampi(c0, 0, s.T);
        end = clampi(c1, begin, s.T);
        r.bad = begin != c0 || end != c1;
    } else {
        begin = b;
        end = b + 1;
        r.bad = false;
    }
    const int n = s.lens[b];
    r.len = clampi(n, 0, cap);
    r.bad = r.bad || r.len != n;
    r.begin = begin;
    r.end = end;
    r.before = r.len - (end - begin);
    return r;
}

// Page holding position pos of sequence b (pos < width * page_tokens), or -1.
MHC_HD int page_of(const Seqs& s, int b, int pos) {
    const int p = s.table[(int64_t)b * s.width + pos / s.page_tokens];
    return p >= 0 && p < s.num_pages ? p : -1;
}

// The new tokens of one page, from token t on: slot..slot + n - 1 of that
// page.  n == 0: token t has no place (next: the first that may have one).
struct Run {
    int pos, slot, n, next;
};

MHC_HD Run run_at(const Seqs& s, const Span& sp, int t) {
    Run r;
    r.pos = sp.before + (t - sp.begin);
    if (r.pos < 0) {
        const int first = sp.begin - sp.before;   // the token at position 0
        r.n = 0;
        r.slot = 0;
        r.next = first < sp.end ? first : sp.end;
        return r;
    }
    r.slot = r.pos % s.page_tokens;
    const int room = s.page_tokens - r.slot, left = sp.end - t;
    r.n = room < left ? room : left;
    r.next = t + r.n;
    return r;
}

// Whether a run starts at token t (the first of its sequence in its page).
MHC_HD bool starts_run(const Span& sp, const Run& r, int t) {
    return r.n > 0 && (t == sp.begin || r.slot == 0);
}

}  // namespace kv
}  // namespace mhc
