// kv_index.cuh -- where the new tokens of a call lie in the paged cache: the
// index arithmetic of the kv kernels, free of device code so that it can be
// compiled and checked on the host as well.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MHC_HD __host__ __device__ __forceinline__
#define MHC_ROLLED _Pragma("unroll 1")      // a loop that is rare and must not fill the instruction cache
#else
#define MHC_HD inline
#define MHC_ROLLED
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
    int page_log2;          // tokens of a page: 2^page_log2
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
    const int cap = s.width << s.page_log2;       // at most 2^30 (checked on the host)
    int begin, end;
    if (s.cu) {
        const int c0 = s.cu[b], c1 = s.cu[b + 1];
        begin = clampi(c0, 0, s.T);
        end = clampi(c1, begin, s.T);
        r.bad = begin != c0 || end != c1;
        if (r.bad) end = begin;                   // cut short, its tokens would get the positions of others
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

// Page holding position pos of sequence b (pos < width * tokens of a page), or -1.
MHC_HD int page_of(const Seqs& s, int b, int pos) {
    const int p = s.table[(int64_t)b * s.width + (pos >> s.page_log2)];
    return p >= 0 && p < s.num_pages ? p : -1;
}

// Position of new token t, or -1: not one of the sequence's, or one without a
// place.  A span that had to be clamped has no places: its positions would be
// those of other tokens.
MHC_HD int pos_of(const Span& sp, int t) {
    if (sp.bad || t < sp.begin || t >= sp.end) return -1;
    const int pos = sp.before + (t - sp.begin);
    return pos < 0 ? -1 : pos;
}

// The new tokens of one page, from the sequence's token t on: slot..slot + n - 1
// of that page.  n == 0: token t has no place (next: the first that may have one).
struct Run {
    int pos, slot, n, next;
};

MHC_HD Run run_at(const Seqs& s, const Span& sp, int t) {
    Run r;
    r.pos = pos_of(sp, t);
    if (sp.bad) {
        r.slot = r.n = 0;
        r.next = sp.end;
        return r;
    }
    if (r.pos < 0) {
        const int first = sp.begin - sp.before;   // the token at position 0
        r.n = 0;
        r.slot = 0;
        r.next = first < sp.end ? first : sp.end;
        return r;
    }
    r.slot = r.pos & ((1 << s.page_log2) - 1);
    const int room = (1 << s.page_log2) - r.slot, left = sp.end - t;
    r.n = room < left ? room : left;
    r.next = t + r.n;
    return r;
}

// Whether a run starts at token t (the first of its sequence in its page).
MHC_HD bool starts_run(const Span& sp, const Run& r, int t) {
    return r.n > 0 && (t == sp.begin || r.slot == 0);
}

// ---------------------------------------------------------------------------
// How mhc_kv_attend's work is cut.  The rows of one sequence and key/value head
// are its new tokens times the `group` query heads that share the head, row r
// being token r / group, query head r % group of it; a tile is 2^tile_log2 of
// them.  A tile's keys are cut in units of 2^unit_log2; a tile without keys
// still is one unit (its rows have to be written), and what a tile costs beside
// its keys (its queries, its rows' way out) counts as `extra` units.  All units of all tiles, ordered by
// sequence, tile, head and key, form one line that the takers (warps or blocks)
// share evenly whatever the lengths are, and a tile cut by a border is joined
// afterwards.

// One sequence as the walk needs it.
struct SeqInfo {
    int begin;              // first new token
    int tokens;             // new tokens
    int before;             // keys before them
};

// The cut's sizes; what would be divisions by the group is worked out once.
struct Cut {
    int heads, group;
    int tile_log2, unit_log2;
    int extra;              // units that a tile counts for beside those of its keys
    int group_inv;          // 65536 / group + 1: x / group is x * group_inv >> 16 for x up to 384
    int step_tokens, step_rem;  // rows of a tile / group and % group
};

MHC_HD Cut make_cut(int heads, int group, int tile_log2, int unit_log2, int extra) {
    const int rows = 1 << tile_log2;
    return Cut{heads, group, tile_log2, unit_log2, extra, 65536 / group + 1, rows / group, rows % group};
}

MHC_HD SeqInfo info_of(const Span& sp) {
    SeqInfo r;
    r.begin = sp.begin;
    r.tokens = sp.end - sp.begin;
    r.before = sp.before;
    return r;
}

MHC_HD int tiles_of(const SeqInfo& s, const Cut& c) {
    return (s.tokens * c.group + (1 << c.tile_log2) - 1) >> c.tile_log2;
}

// Units of a tile: those of its keys, at least one, and the extra ones, which come first.
MHC_HD int units_of(int keys, const Cut& c) {
    const int n = (keys + (1 << c.unit_log2) - 1) >> c.unit_log2;
    return (n < 1 ? 1 : n) + c.extra;
}

// The tiles of a sequence one after the other.
struct Tiles {
    int tile, units;
    int token, rem;         // of its row 0: new token of the sequence, query head of the group
    int rows, keys;         // keys: the most that any of its rows sees
};

MHC_HD void tiles_measure(Tiles& t, const SeqInfo& s, const Cut& c) {
    const int left = s.tokens * c.group - (t.tile << c.tile_log2);
    t.rows = left < 1 << c.tile_log2 ? left : 1 << c.tile_log2;
    const int n = s.before + t.token + ((t.rem + t.rows - 1) * c.group_inv >> 16) + 1;    // its last row's
    t.keys = n < 0 ? 0 : n;
    t.units = units_of(t.keys, c);
}

MHC_HD void tiles_start(Tiles& t, const SeqInfo& s, const Cut& c) {
    t.tile = t.token = t.rem = 0;
    tiles_measure(t, s, c);
}

MHC_HD void tiles_next(Tiles& t, const SeqInfo& s, const Cut& c) {
    ++t.tile;
    t.token += c.step_tokens;
    t.rem += c.step_rem;
    if (t.rem >= c.group) {
        t.rem -= c.group;
        ++t.token;
    }
    tiles_measure(t, s, c);
}

// Units of all tiles and heads of a sequence.
MHC_HD int64_t units_of_seq(const SeqInfo& s, const Cut& c) {
    const int tiles = tiles_of(s, c);
    if (tiles == 0) return 0;
    int64_t n = 0;
    Tiles t;
    tiles_start(t, s, c);
    MHC_ROLLED
    for (int i = 0; i < tiles; ++i) {
        n += t.units;
        if (i + 1 < tiles) tiles_next(t, s, c);
    }
    return n * c.heads;
}

// The line's equal shares; with fewer units than takers the first `total` take
// one each, so that the takers of a tile always follow one another.
struct Shares {
    int64_t total, each, extra;      // units of the line; of a share; how many first shares take one more
};

MHC_HD int64_t divide(int64_t a, int64_t b) {      // in 32 bits where they hold
    return (a | b) >> 31 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

MHC_HD Shares shares_of(int64_t total, int n) {
    Shares s;
    s.total = total;
    s.each = divide(total, n);
    s.extra = total - s.each * n;
    return s;
}

// The first unit of share c.
MHC_HD int64_t share_start(const Shares& s, int c) { return s.each * c + (c < s.extra ? c : s.extra); }

// The share that unit u of the line is in.
MHC_HD int share_at(const Shares& s, int64_t u) {
    const int64_t longer = s.extra * (s.each + 1);
    return (int)(u < longer ? divide(u, s.each + 1) : s.extra + divide(u - longer, s.each));
}

// A segment: the units of one tile and head that one share has.
struct Segment {
    int b, head;            // sequence, key/value head
    int token, rem;         // row 0 of the tile: new token, query head of the group
    int rows;               // of the tile
    int see;                // keys before that token
    int key0, keys;         // the segment's keys [key0, keys); none where the tile sees none
    int parts, owner;       // shares that the tile's units lie in, the first of them
};

// Row r of a segment's tile.
MHC_HD void row_of(const Segment& s, const Cut& c, int r, int& token, int& in_group) {
    const int x = s.rem + r, n = x * c.group_inv >> 16;
    token = s.token + n;
    in_group = x - n * c.group;
}

// How many keys that row sees.
MHC_HD int keys_of_row(const Segment& s, const Cut& c, int r) {
    const int n = s.see + ((s.rem + r) * c.group_inv >> 16) + 1;
    return n < 0 ? 0 : n;
}

// A walk over a share's segments.
struct Walk {
    Tiles t;
    int head, first, count;
    int64_t left;           // units of the share from this segment on; 0: the walk is over
};

MHC_HD void walk_cut(Walk& w) {
    const int rest = w.t.units - w.first;
    w.count = w.left < rest ? (int)w.left : rest;
}

// Enters a sequence (with new tokens) at unit r of its part of the line, with
// `left` units of the share to go.
MHC_HD void walk_enter(Walk& w, const SeqInfo& s, const Cut& c, int64_t r, int64_t left) {
    w.left = left;
    tiles_start(w.t, s, c);
    MHC_ROLLED
    while (r >= (int64_t)w.t.units * c.heads) {
        r -= (int64_t)w.t.units * c.heads;
        tiles_next(w.t, s, c);
    }
    w.head = (int)divide(r, w.t.units);
    w.first = (int)(r - (int64_t)w.head * w.t.units);
    walk_cut(w);
}

// The next segment; false where the sequence is done (then the caller enters
// the next one with new tokens, if w.left > 0).
MHC_HD bool walk_next(Walk& w, const SeqInfo& s, const Cut& c) {
    w.left -= w.count;
    if (w.left <= 0) return false;
    w.first = 0;
    if (++w.head == c.heads) {
        w.head = 0;
        if (w.t.tile + 1 == tiles_of(s, c)) return false;
        tiles_next(w.t, s, c);
    }
    walk_cut(w);
    return true;
}

// A share's plan: the walk, the sequence it is in and the line's unit that its
// segment starts at.
struct Plan {
    Walk w;
    SeqInfo info;
    int b;
    int64_t at;
};

// The plan's next segment, if it has one: a part of a share that has only
// extra units of a tile is none.  look(b) finds sequence b.
template <class Look>
MHC_HD bool plan_next(Plan& p, const Look& look, const Cut& c, const Shares& shares, Segment& s) {
    MHC_ROLLED
    while (p.w.left > 0) {
        const int end = p.w.first + p.w.count - c.extra;     // of the tile's key units
        const bool some = end > 0;
        if (some) {
            const int first = p.w.first > c.extra ? p.w.first - c.extra : 0;
            s.b = p.b;
            s.head = p.w.head;
            s.token = p.info.begin + p.w.t.token;
            s.rem = p.w.t.rem;
            s.rows = p.w.t.rows;
            s.see = p.info.before + p.w.t.token;
            s.key0 = first << c.unit_log2;
            s.keys = end << c.unit_log2 < p.w.t.keys ? end << c.unit_log2 : p.w.t.keys;
            if (first == 0 && end == p.w.t.units - c.extra) {
                s.parts = 1;
                s.owner = 0;
            } else {
                const int64_t begin = p.at - p.w.first;      // of the tile
                s.owner = share_at(shares, begin + c.extra);
                s.parts = share_at(shares, begin + p.w.t.units - 1) - s.owner + 1;
            }
        }
        p.at += p.w.count;
        if (!walk_next(p.w, p.info, c) && p.w.left > 0) {
            MHC_ROLLED
            do p.info = look(++p.b);
            while (p.info.tokens == 0 && p.b + 1 < look.count());
            if (p.info.tokens > 0) walk_enter(p.w, p.info, c, 0, p.w.left);
            else p.w.left = 0;               // lengths that changed since they were counted
        }
        if (some) return true;
    }
    return false;
}

// A segment that one lane of a warp finds, for all of its lanes: find() writes it
// into the warp's queue and says whether there was one.  The vote brings the
// lanes together but orders no memory, so a barrier follows before anybody reads
// the segment.  The plan is the one lane's alone.
template <class Warp, class Find>
MHC_HD bool found_for_all(const Warp& warp, Find&& find) {
    const bool found = warp.any(warp.first() && find());
    warp.sync();
    return found;
}

}  // namespace kv
}  // namespace mhc
