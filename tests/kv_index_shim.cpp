// The kv kernels' index arithmetic, compiled for the host by test_kv_cpu.py.
#include "../mhc_hyper_connection_pre_gb300/csrc/kv_index.cuh"

using namespace mhc::kv;

static Seqs make(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P, int pages) {
    int log2 = 0;
    while ((1 << log2) < P) ++log2;
    return Seqs{table, lens, cu, width, B, T, log2, pages};
}

struct Look {
    const Seqs& s;
    int count() const { return s.B; }
    SeqInfo operator()(int b) const { return info_of(span_of(s, b)); }
};

extern "C" {

// The runs that an append writes: for each token t, what a thread group that
// meets t does.  out[t] = {starts, pos, slot, n, next, page, bad}.
void kv_runs(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P, int pages,
             const int32_t* seq, int32_t* out) {
    const Seqs s = make(table, lens, cu, width, B, T, P, pages);
    for (int t = 0; t < T; ++t) {
        const Span sp = span_of(s, seq[t]);
        int32_t* o = out + 7 * t;
        for (int i = 0; i < 7; ++i) o[i] = 0;
        o[6] = sp.bad;
        if (t < sp.begin || t >= sp.end) {
            o[4] = t + 1;
            o[6] = 1;
            continue;
        }
        const Run r = run_at(s, sp, t);
        o[0] = starts_run(sp, r, t);
        o[1] = r.pos;
        o[2] = r.slot;
        o[3] = r.n;
        o[4] = r.next;
        o[5] = o[0] ? page_of(s, seq[t], r.pos) : -1;
    }
}

// The position that each token's query is rotated by, -1: none.
void kv_positions(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P, int pages,
                  const int32_t* seq, int32_t* out) {
    const Seqs s = make(table, lens, cu, width, B, T, P, pages);
    for (int t = 0; t < T; ++t) out[t] = pos_of(span_of(s, seq[t]), t);
}

// The segments of share `share` of `n`: out[i] = {sequence, first token, query
// head of its first row, rows, head, first key, last key + 1, shares of the
// tile, the first of them, keys that the first and the last row see}.  Returns
// how many, or -1 if there are more than `most`; total: units of the line.
int kv_segments(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P,
                int pages, int heads, int group, int tile_log2, int unit_log2, int extra, int share, int n, int32_t* out,
                int most, int64_t* total) {
    const Seqs s = make(table, lens, cu, width, B, T, P, pages);
    const Cut c = make_cut(heads, group, tile_log2, unit_log2, extra);
    *total = 0;
    for (int b = 0; b < B; ++b) *total += units_of_seq(info_of(span_of(s, b)), c);
    const Shares shares = shares_of(*total, n);
    const int64_t from = share_start(shares, share), left = share_start(shares, share + 1) - from;
    if (left <= 0) return 0;
    int64_t seen = 0;
    Plan p;
    for (p.b = 0;; ++p.b) {
        p.info = info_of(span_of(s, p.b));
        const int64_t u = units_of_seq(p.info, c);
        if (from < seen + u) break;
        seen += u;
    }
    p.at = from;
    walk_enter(p.w, p.info, c, from - seen, left);
    int found = 0;
    Segment g;
    while (plan_next(p, Look{s}, c, shares, g)) {
        if (found == most) return -1;
        const int32_t o[] = {g.b, g.token, g.rem, g.rows, g.head, g.key0, g.keys, g.parts, g.owner,
                             keys_of_row(g, c, 0), keys_of_row(g, c, g.rows - 1)};
        for (int i = 0; i < 11; ++i) out[11 * found + i] = o[i];
        ++found;
    }
    return found;
}

// Token and query head of every row of a segment's tile.
void kv_rows(int token, int rem, int rows, int group, int32_t* out) {
    const Cut c = make_cut(1, group, 8, 5, 0);
    const Segment g{0, 0, token, rem, rows, 0, 0, 0, 1, 0};
    for (int r = 0; r < rows; ++r) row_of(g, c, r, out[2 * r], out[2 * r + 1]);
}

}
