// A window's ends in the tensor-memory kernel's segments, compiled for the host by test_kv_edges_cpu.py.
#include "kv_window_shim.cpp"

// Walks every share's segments; returns how many keys are in both or in neither of a segment's ends though the rows
// differ in whether they see them, or are in one though they do not differ.
// longest: keys of the longest end.
extern "C" int64_t kv_window_ends(const int32_t* lens, const int32_t* cu, int width, int B, int T, int log2, int heads,
                                  int group, int unit_log2, int extra, int window, int sinks, int n, int32_t* longest,
                                  int32_t* segments) {
    const Seqs s{nullptr, lens, cu, width, B, T, log2, 1};
    WindowCut c;
    static_cast<Cut&>(c) = make_cut(heads, group, 8, unit_log2, extra);
    c.window = window;
    c.sinks = sinks;
    c.load_log2 = 7;
    int64_t total = 0, wrong = 0;
    for (int b = 0; b < B; ++b) total += units_of_seq(info_of(span_of(s, b)), c);
    const Shares shares = shares_of(total, n);
    *longest = *segments = 0;
    for (int share = 0; share < n; ++share) {
        const int64_t from = share_start(shares, share), left = share_start(shares, share + 1) - from;
        if (left <= 0) continue;
        int64_t before = 0;
        Plan p;
        for (p.b = 0;; ++p.b) {
            p.info = info_of(span_of(s, p.b));
            const int64_t u = units_of_seq(p.info, c);
            if (from < before + u) break;
            before += u;
        }
        p.at = from;
        walk_enter(p.w, p.info, c, from - before, left);
        WindowSegment g;
        while (plan_next(p, Look{s}, c, shares, g)) {
            ++*segments;
            const Ends e = ends_of(g, c);
            if (e.low_end - e.low > *longest) *longest = e.low_end - e.low;
            if (e.high_end - e.high > *longest) *longest = e.high_end - e.high;
            const int n0 = keys_of_row(g, c, 0), n1 = keys_of_row(g, c, g.rows - 1);
            for (int key = g.key0; key < g.keys; ++key) {
                const int in = (key >= e.low && key < e.low_end) + (key >= e.high && key < e.high_end);
                wrong += in != !keys_all_seen(key, 1, n0, n1, c);
            }
        }
    }
    return wrong;
}
