// kv_pages.cuh -- which pages the next step's tables name (mhc_kv_fork), and
// which pages move where when a cache is compacted (mhc_kv_compact): the
// planning of both calls, written for a team of threads and free of device code,
// so that it can be compiled and checked on the host, under a race detector too.
//
// A team T has `rank` of `size` threads (a power of two for what needs barriers), sync(), a barrier after
// which all see what each has written, scan(x, total), the sum of x over the ranks
// below and over all (a collective that ends in a barrier), load, set_bit (of a page, none
// for -1), lower and raise, which may meet one another on one word, and report.
//
// The rows of large tables are the work of all SMs (the _rows functions, by any
// number of threads that meet nowhere, between a call's other parts); of small ones, one block does
// all.  Nothing is kept between calls: a page is in use if the tables name it or `held`
// says so, and the pages that are handed out are the lowest others, in the order of
// the places and their entries.  So the results do not depend on the team.
#pragma once

#include "kv_index.cuh"

#ifdef __CUDACC__
#define MHC_UNROLLED _Pragma("unroll")
#else
#define MHC_UNROLLED
#endif

namespace mhc {
namespace kv {

constexpr unsigned int kPagesError = 4u;      // of a status word: no free page left
constexpr unsigned int kBadIndex = 2u;        // kIndexError
constexpr int kNobody = 0x7fffffff;

// A page whose first `slots` slots are to be copied, and where to.
struct PageCopy {
    int32_t from, to, slots;
};

// What both calls are given.
struct PagesIn {
    const int32_t* table;                     // [B_in][width]
    const int32_t* lens;                      // [B_in]
    const uint8_t* held;                      // [num_pages] or null
    int32_t* out;                             // [B][width]
    int width, B_in, B;
    int page_log2, num_pages;
};

// A place of the batch: where the row begins that it goes on with, its tokens, the
// first of its full pages that stay (after those of the first tokens), the page that
// is part-filled (-1: none).
struct alignas(16) Place {
    int32_t row, len, low, tail;
};

struct ForkIn {
    PagesIn p;
    const int32_t* parents;                   // [B] or null: b goes on with b
    const int32_t* room;                      // [B] or null: room_all
    int room_all;
    int window, sinks;                        // window 0: none
    int32_t* lens_out;                        // [B]
};

// The planning's scratch, in shared or global memory.  bits: a bit for each page.
struct ForkSpace {
    uint32_t* bits;
    Place* place;                             // [B]
    int32_t* first;                           // [B]: first of the pages that a place is given, times 2, and whether it copies
    int32_t* keeper;                          // [num_pages], written where it is read
    int32_t* given;                           // pages handed out, in order; as many as may be asked for
    PageCopy* copies;                         // [B]
    int32_t* count;                           // of copies
};

struct CompactSpace {
    uint32_t *bits, *held;                    // a bit for each page, in use and held
    int32_t* entries;                         // [B]: of each row, those that name its pages
    int32_t *mover, *hole, *moved;            // [num_pages]: used pages by rank; free places by rank; where a page is now
    PageCopy* copies;                         // [num_pages]
    int32_t* count;                           // of copies
    int32_t* mark;                            // [2]: how many used pages stay, the first page that may have moved
};

MHC_HD int pages_for(int64_t tokens, int page_log2) { return (int)((tokens + ((int64_t)1 << page_log2) - 1) >> page_log2); }

MHC_HD int words_of(int num_pages) { return (num_pages + 31) / 32; }

// The pages in pieces that the threads divide: 8 of them where each thread gets few, so that none goes over
// 32 bits one by one while the others wait, else whole words.
struct Pieces {
    int log2, count, num_pages;
    MHC_HD int first(int64_t c) const { return (int)(c << log2); }
    MHC_HD uint32_t real(int64_t c) const {
        const int n = num_pages - first(c);
        return n >= 32 ? (log2 == 5 ? 0xffffffffu : 0xffu) : ((1u << n) - 1) & (log2 == 5 ? 0xffffffffu : 0xffu);
    }
    MHC_HD uint32_t bits(uint32_t word, int64_t c) const { return word >> (first(c) & 31); }   // `real` of it count
    MHC_HD int word(int64_t c) const { return first(c) >> 5; }
};
MHC_HD Pieces pieces_of(int num_pages, int threads) {
    const int log2 = num_pages <= 64 * (int64_t)threads ? 3 : 5;
    return Pieces{log2, (int)(((int64_t)num_pages + (1 << log2) - 1) >> log2), num_pages};
}

MHC_HD uint32_t held_word(const uint8_t* held, int num_pages, int w) {
    uint32_t bits = 0;
    if (!held) return bits;
    if (num_pages - 32 * w >= 32) {           // 4-byte aligned
        const uint32_t* from = reinterpret_cast<const uint32_t*>(held) + 8 * (int64_t)w;
        MHC_UNROLLED
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = from[i];
            const uint32_t y = ((x & 0xff) ? 1u : 0u) | ((x & 0xff00) ? 2u : 0u) | ((x & 0xff0000) ? 4u : 0u) |
                               ((x & 0xff000000) ? 8u : 0u);
            bits |= y << (4 * i);
        }
        return bits;
    }
    for (int i = 0; 32 * w + i < num_pages; ++i) bits |= held[32 * (int64_t)w + i] ? 1u << i : 0u;
    return bits;
}

MHC_HD int ones(uint32_t x) {
#ifdef __CUDA_ARCH__
    return __popc(x);
#else
    return __builtin_popcount(x);
#endif
}
MHC_HD int lowest(uint32_t x) {
#ifdef __CUDA_ARCH__
    return __ffs(x) - 1;
#else
    return __builtin_ctz(x);
#endif
}
MHC_HD int highest(uint32_t x) {
#ifdef __CUDA_ARCH__
    return 31 - __clz(x);
#else
    return 31 - __builtin_clz(x);
#endif
}

// The entries of a row that are pages of its own: those below `early` and from `low` on, up to `end`; `base`
// is where the row begins.  Entry `skip` is left alone (-1: none).
struct RowPages {
    int32_t base, end, low, early, skip;
};

// use(b, i, page) for every entry of `rows` rows: the page that `from` has there, -1 for an entry that is not of
// the row's own (pages(b) says which are) or no page's number; numbers that are neither a page nor
// -1 are reported.  A thread takes four entries side by side of four rows, whose
// loads are under way together.  Half of the time is one block's instructions, so what
// is a row's is worked out once, and offsets are 32 bits (checked on the host).
template <class Team, class Pages, class Use>
MHC_HD void each_entry(const Team& t, int rows, int width, const int32_t* from, int num_pages, Pages&& pages, Use&& use) {
    constexpr int kRows = 4, kWide = 4;
    int log2 = 0;
    while ((2 << log2) <= t.size && (kWide << log2) < width) ++log2;
    const int lanes = 1 << log2, at_once = t.size >> log2, lane = t.rank & (lanes - 1);
    if (t.rank >> log2 >= at_once) return;    // threads left over, where a row's do not divide a grid's: an entry is one thread's alone
    bool bad = false;
    MHC_ROLLED
    for (int b0 = t.rank >> log2; b0 < rows; b0 += kRows * at_once)
        MHC_ROLLED
        for (int i0 = kWide * lane; i0 < width; i0 += kWide * lanes) {
            int32_t v[kRows][kWide], skip[kRows];
            MHC_UNROLLED
            for (int j = 0; j < kRows; ++j) {
                const int b = b0 + j * at_once;
                const RowPages r = b < rows ? pages(b) : RowPages{0, 0, 0, 0, -1};
                skip[j] = r.skip;
                MHC_UNROLLED
                for (int k = 0; k < kWide; ++k) {
                    const int i = i0 + k;
                    v[j][k] = i < r.end && (i >= r.low || i < r.early) ? from[r.base + i] : -1;
                }
            }
            MHC_UNROLLED
            for (int j = 0; j < kRows; ++j) {
                const int b = b0 + j * at_once;
                if (b >= rows) continue;
                MHC_UNROLLED
                for (int k = 0; k < kWide; ++k) {
                    const bool ok = (uint32_t)v[j][k] < (uint32_t)num_pages;
                    bad = bad || (!ok && v[j][k] != -1);
                    if (i0 + k < width && i0 + k != skip[j]) use(b, i0 + k, ok ? v[j][k] : -1);
                }
            }
        }
    if (bad) t.report(kBadIndex);
}

// A rank's part of n things in a row.
template <class Team>
MHC_HD void part_of_all(const Team& t, int64_t n, int64_t& begin, int64_t& end) {
    const int64_t each = (n + t.size - 1) / t.size;
    begin = each * t.rank < n ? each * t.rank : n;
    end = begin + each < n ? begin + each : n;
}

// An entry as a page, or -1; anything but a page's number or -1 is reported.
template <class Team>
MHC_HD int checked_page(const Team& t, int p, int num_pages) {
    if (p >= 0 && p < num_pages) return p;
    if (p != -1) t.report(kBadIndex);
    return -1;
}

// A length as the nearest one that a row of the table can hold.
template <class Team>
MHC_HD int checked_tokens(const Team& t, int64_t n, int cap) {
    const int64_t m = n < 0 ? 0 : (n > cap ? cap : n);
    if (m != n) t.report(kBadIndex);
    return (int)m;
}

// The first page of the window of the next token after n: with no window the first of all.
MHC_HD int first_page(int n, int window, int page_log2) {
    const int first = n - window + 1;
    return window == 0 || first < 0 ? 0 : first >> page_log2;
}

// Place b of the batch, without its part-filled page.
template <class Team>
MHC_HD Place place_of(const Team& t, const ForkIn& a, int b) {
    int from = a.parents ? a.parents[b] : b;
    if (from < -1 || from >= a.p.B_in) {
        t.report(kBadIndex);
        from = -1;
    }
    const int n = from < 0 ? 0 : checked_tokens(t, a.p.lens[from], a.p.width << a.p.page_log2);
    return Place{from * a.p.width, n, first_page(n, a.window, a.p.page_log2), -1};
}

// Every place: whom it goes on with, its tokens, its part-filled page.
template <class Team>
MHC_HD void fork_places(const Team& t, const ForkIn& a, const ForkSpace& s) {
    const int log2 = a.p.page_log2;
    for (int b = t.rank; b < a.p.B; b += t.size) {
        Place x = place_of(t, a, b);
        if (x.len & ((1 << log2) - 1)) x.tail = checked_page(t, a.p.table[x.row + (x.len >> log2)], a.p.num_pages);
        s.place[b] = x;
        if (x.tail >= 0) t.store(s.keeper + x.tail, kNobody);
    }
}

// Full pages are shared, those of the first tokens and of the window.  place(b): whom place b goes on with.
// The entry after the full pages is fork_rest's to write: others may still read it, where tables are written in place.
template <class Team, class PlaceOf>
MHC_HD void fork_entries(const Team& t, const ForkIn& a, const ForkSpace& s, PlaceOf&& place) {
    const PagesIn& p = a.p;
    const int early = pages_for(a.sinks, p.page_log2);
    each_entry(
        t, p.B, p.width, p.table, p.num_pages,
        [&](int b) {
            const Place x = place(b);
            const int full = x.len >> p.page_log2;
            return RowPages{x.row, full, x.low, early, full};
        },
        [&](int b, int i, int32_t page) {
            t.set_bit(s.bits, page);
            p.out[b * p.width + i] = page;
        });
}

// The rows of large tables; no bit is set before.
template <class Team>
MHC_HD void fork_rows(const Team& t, const ForkIn& a, const ForkSpace& s) {
    fork_places(t, a, s);
    fork_entries(t, a, s, [&](int b) { return place_of(t, a, b); });
}

// The rest, once the rows' full pages are marked.  `marked`: those and the pages that are held, where they are not
// in s.bits yet.
template <class Team>
MHC_HD void fork_rest(Team& t, const ForkIn& a, const ForkSpace& s, const uint32_t* marked = nullptr) {
    const PagesIn& p = a.p;
    const int log2 = p.page_log2, P = 1 << log2, cap = p.width << log2, words = words_of(p.num_pages);
    if (marked)
        for (int w = t.rank; w < words; w += t.size) s.bits[w] = marked[w] | held_word(p.held, p.num_pages, w);
    for (int b = t.rank; b < p.B; b += t.size)
        if (s.place[b].tail >= 0) t.lower(s.keeper + s.place[b].tail, b);
    t.sync();

    // A part-filled page stays with the first place that goes on with it, unless somebody else
    // has it too: as a full page, or held.  What a place is given: a page for its copy, and those of
    // its further tokens.
    int64_t begin, end, mine = 0, total;
    part_of_all(t, p.B, begin, end);
    auto copied = [&](int b) {                // before any bit of a part-filled page is set, but for those that
        const int last = s.place[b].tail;     // their keepers set: nobody else asks for these
        if (last < 0) return false;
        return t.load(s.keeper + last) != b || (t.load(s.bits + (last >> 5)) >> (last & 31) & 1);
    };
    for (int64_t b = begin; b < end; ++b) {
        const int n = s.place[b].len, last = s.place[b].tail;
        const int64_t asked = a.room ? a.room[b] : a.room_all;
        const int now = pages_for(n, log2);
        const int then = pages_for(checked_tokens(t, n + (asked < 0 ? -1 - (int64_t)n : asked), cap), log2);
        const bool copy = copied((int)b);
        s.first[b] = copy ? 1 : 0;            // for now: whether it copies
        mine += (then > now ? then - now : 0) + (copy ? ((int64_t)1 << 32) + 1 : 0);
        if (!copy) {
            t.set_bit(s.bits, last);
            if (n < cap) p.out[b * p.width + (n >> log2)] = last;
        }
    }
    int64_t before = t.scan(mine, total);
    const int64_t wanted = total & 0xffffffff;
    if (t.rank == 0) *s.count = (int32_t)(total >> 32);
    for (int64_t b = begin; b < end; ++b) {
        const int n = s.place[b].len;
        const int64_t asked = a.room ? a.room[b] : a.room_all;
        const int64_t to = (int64_t)n + (asked < 0 ? 0 : asked);
        const int now = pages_for(n, log2), then = pages_for(to < cap ? to : cap, log2);
        const bool copy = s.first[b];
        if (copy) s.copies[before >> 32] = PageCopy{s.place[b].tail, (int32_t)b, n & (P - 1)};    // `to` follows below
        s.first[b] = (int32_t)(before & 0xffffffff) << 1 | (copy ? 1 : 0);
        before += (then > now ? then - now : 0) + (copy ? ((int64_t)1 << 32) + 1 : 0);
        a.lens_out[b] = n;
    }

    // the lowest free pages
    const Pieces pieces = pieces_of(p.num_pages, t.size);
    auto free_in = [&](int64_t c) { return ~pieces.bits(t.load(s.bits + pieces.word(c)), c) & pieces.real(c); };
    part_of_all(t, pieces.count, begin, end);
    mine = 0;
    for (int64_t c = begin; c < end; ++c) mine += ones(free_in(c));
    int64_t k = t.scan(mine, total);
    for (int64_t c = begin; c < end && k < wanted; ++c)
        for (uint32_t left = free_in(c); left && k < wanted; left &= left - 1) s.given[k++] = pieces.first(c) + lowest(left);
    if (t.rank == 0 && total < wanted) t.report(kPagesError);
    t.sync();

    // and the entries that get them
    for (int i = t.rank; i < *s.count; i += t.size) {
        const int b = s.copies[i].to, at = s.first[b] >> 1;
        const int page = at < total ? s.given[at] : -1;
        s.copies[i].to = page;
        p.out[b * p.width + (s.place[b].len >> log2)] = page;
    }
    // a thread a place where each gets a few pages at most, as far as the call tells
    const int lanes = t.size < 32 || (!a.room && a.room_all <= 4 * P) ? 1 : 32;
    for (int b = t.rank / lanes; b < p.B; b += t.size / lanes) {
        const int n = s.place[b].len;
        const int64_t asked = a.room ? a.room[b] : a.room_all, to = (int64_t)n + (asked < 0 ? 0 : asked);
        const int now = pages_for(n, log2), then = pages_for(to < cap ? to : cap, log2);
        const int at = (s.first[b] >> 1) + (s.first[b] & 1) - now;
        for (int i = now + t.rank % lanes; i < then; i += lanes)
            p.out[b * p.width + i] = at + i < total ? s.given[at + i] : -1;
    }
}

template <class Team>
MHC_HD void plan_fork(Team& t, const ForkIn& a, const ForkSpace& s) {
    fork_places(t, a, s);
    for (int w = t.rank; w < words_of(a.p.num_pages); w += t.size) s.bits[w] = held_word(a.p.held, a.p.num_pages, w);
    t.sync();
    fork_entries(t, a, s, [&](int b) { return s.place[b]; });
    fork_rest(t, a, s);
}

// What is in use and not held goes to the lowest numbers that are not held: the pages there that are
// free ("holes") take the used ones above, in order.
template <class Team, class Entries, class Use>
MHC_HD void compact_entries(const Team& t, const PagesIn& p, Entries&& entries, Use&& use) {
    each_entry(t, p.B, p.width, p.table, p.num_pages, [&](int b) { return RowPages{b * p.width, entries(b), 0, 0, -1}; }, use);
}

// Marks the pages that the rows name; no bit is set before.
template <class Team>
MHC_HD void compact_rows(const Team& t, const PagesIn& p, const CompactSpace& s) {
    compact_entries(
        t, p, [&](int b) { return pages_for(checked_tokens(t, p.lens[b], p.width << p.page_log2), p.page_log2); },
        [&](int, int, int32_t page) { t.set_bit(s.bits, page); });
}

// The new rows, with the pages that moved in their new places.
template <class Team, class Entries>
MHC_HD void compact_rename(const Team& t, const PagesIn& p, const CompactSpace& s, Entries&& entries) {
    const int from = s.mark[1];
    compact_entries(t, p, entries, [&](int b, int i, int32_t x) {
        if (x >= from && !(p.held && p.held[x])) x = s.moved[x];
        p.out[b * p.width + i] = x;
    });
}

// Which pages move where, once those in use are marked (in `marked`, or in s.bits).
template <class Team>
MHC_HD void compact_moves(Team& t, const PagesIn& p, int32_t* top, const CompactSpace& s, const uint32_t* marked = nullptr) {
    const int log2 = p.page_log2, words = words_of(p.num_pages);
    if (marked)
        for (int w = t.rank; w < words; w += t.size) {
            s.bits[w] = marked[w];
            s.held[w] = held_word(p.held, p.num_pages, w);
        }
    if (t.rank == 0) t.store(top, 0);
    t.sync();
    const Pieces pieces = pieces_of(p.num_pages, t.size);
    auto held_in = [&](int64_t c) { return pieces.bits(s.held[pieces.word(c)], c) & pieces.real(c); };
    auto used_in = [&](int64_t c) { return pieces.bits(s.bits[pieces.word(c)], c) & pieces.real(c); };
    int64_t begin, end, mine = 0, total;      // in 32 bits each: used pages, and pages, that are not held
    part_of_all(t, pieces.count, begin, end);
    for (int64_t c = begin; c < end; ++c) {
        const uint32_t loose = pieces.real(c) & ~held_in(c);
        mine += (int64_t)ones(used_in(c) & loose) << 32 | ones(loose);
    }
    const int64_t before = t.scan(mine, total);
    const int used = (int)(total >> 32);
    int l = (int)(before >> 32), r = (int)(before & 0xffffffff), last = -1;
    for (int64_t c = begin; c < end; ++c) {
        const uint32_t held = held_in(c), loose = pieces.real(c) & ~held, in_use = used_in(c) & loose;
        const int count = ones(loose), first = pieces.first(c);
        uint32_t goal = 0;                    // the piece's pages among the lowest `used`
        if (r + count <= used) {
            goal = loose;
        } else if (r < used) {
            uint32_t rest = loose;
            for (int i = r; i < used; ++i, rest &= rest - 1) goal |= rest & (0u - rest);
        }
        const uint32_t beyond = loose & ~goal;
        if (beyond && r + ones(goal) == used) {       // the first page beyond them
            s.mark[0] = l + ones(in_use & goal);
            s.mark[1] = first + lowest(beyond);
        }
        int hole = r - l, rank = l + ones(in_use & goal);
        for (uint32_t x = goal & ~in_use; x; x &= x - 1) s.hole[hole++] = first + lowest(x);
        for (uint32_t x = in_use & ~goal; x; x &= x - 1) s.mover[rank++] = first + lowest(x);
        if (goal | held) last = first + highest(goal | held);
        l += ones(in_use);
        r += count;
    }
    if (last >= 0) t.raise(top, last + 1);
    if (t.rank == 0 && used == (int)(total & 0xffffffff)) {          // every page that is not held is used
        s.mark[0] = used;
        s.mark[1] = p.num_pages;
    }
    t.sync();

    const int stay = s.mark[0], moves = used - stay, from = s.mark[1];
    if (t.rank == 0) *s.count = moves;
    for (int k = t.rank; k < moves; k += t.size) {
        const int page = s.mover[stay + k];
        s.moved[page] = s.hole[k];
        s.copies[k] = PageCopy{page, s.hole[k], 1 << log2};
    }
}

template <class Team>
MHC_HD void plan_compact(Team& t, const PagesIn& p, int32_t* top, const CompactSpace& s) {
    for (int w = t.rank; w < words_of(p.num_pages); w += t.size) {
        s.bits[w] = 0;
        s.held[w] = held_word(p.held, p.num_pages, w);
    }
    for (int b = t.rank; b < p.B; b += t.size)
        s.entries[b] = pages_for(checked_tokens(t, p.lens[b], p.width << p.page_log2), p.page_log2);
    t.sync();
    compact_entries(t, p, [&](int b) { return s.entries[b]; }, [&](int, int, int32_t page) { t.set_bit(s.bits, page); });
    compact_moves(t, p, top, s);
    t.sync();
    compact_rename(t, p, s, [&](int b) { return s.entries[b]; });
}

}  // namespace kv
}  // namespace mhc
