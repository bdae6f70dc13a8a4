// How attention with a window is cut, compiled for the host by test_kv_more_cpu.py.
#include "../mhc_hyper_connection_pre_gb300/csrc/kv_index.cuh"

using namespace mhc::kv;

struct Look {
    const Seqs& s;
    int count() const { return s.B; }
    SeqInfo operator()(int b) const { return info_of(span_of(s, b)); }
};

extern "C" {

// Walks every share's segments.  seen[row][place] counts how often a row (token * q_heads + head * group + in_group)
// meets a key that it sees; looked[b][page] whether the page of a key's place is looked at.  Returns the number of
// contradictions: a key that is seen of a page that is not looked at, a run of keys that counts as seen by all rows of
// the tile but is not, a segment that is not of whole units, more keys than there are.  total: units of the line.
int64_t kv_window_walk(const int32_t* lens, const int32_t* cu, int width, int B, int T, int log2, int heads, int group,
                       int tile_log2, int unit_log2, int extra, int window, int sinks, int n, uint8_t* seen,
                       uint8_t* looked, int64_t* total, int32_t* longest) {
    const Seqs s{nullptr, lens, cu, width, B, T, log2, 1};
    WindowCut c;
    static_cast<Cut&>(c) = make_cut(heads, group, tile_log2, unit_log2, extra);
    c.window = window;
    c.sinks = sinks;
    c.load_log2 = unit_log2 > 7 ? 7 : unit_log2;
    const int cap = width << log2, unit = 1 << c.load_log2;
    *total = 0;
    for (int b = 0; b < B; ++b) *total += units_of_seq(info_of(span_of(s, b)), c);
    if (n == 0) return 0;                                       // the units alone
    const Shares shares = shares_of(*total, n);
    int64_t wrong = 0;
    *longest = 0;
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
            const int first = first_seen(g, c), n0 = keys_of_row(g, c, 0), n1 = keys_of_row(g, c, g.rows - 1);
            wrong += g.key0 % unit != 0 || g.skip % unit != 0 || g.skip_at % unit != 0 || g.skip < 0 || g.keys > n1;
            if (g.keys - g.key0 > *longest) *longest = g.keys - g.key0;
            for (int key = g.key0; key < g.keys; ++key) {
                const int place = place_of_key(g, key);
                if (place < 0 || place >= cap) {
                    ++wrong;
                    continue;
                }
                const bool look = page_seen(place, first, sinks, log2);
                if (look) looked[(int64_t)g.b * width + (place >> log2)] = 1;
                bool all[3];
                const int counts[3] = {1, 32, 64};
                for (int i = 0; i < 3; ++i) all[i] = keys_all_seen(key, counts[i], n0, n1, c);
                for (int r = 0; r < g.rows; ++r) {
                    int token, in_group;
                    row_of(g, c, r, token, in_group);
                    const int limit = keys_of_row(g, c, r);
                    const bool sees = key_seen(key, limit, c);
                    if (sees) {
                        wrong += !look;
                        ++seen[((int64_t)token * heads * group + g.head * group + in_group) * cap + place];
                    }
                    for (int i = 0; i < 3; ++i)
                        for (int k = 0; all[i] && k < counts[i]; ++k) wrong += !key_seen(key + k, limit, c);
                }
            }
        }
    }
    return wrong;
}

}
