// The kv kernels' index arithmetic, compiled for the host by test_kv_cpu.py.
#include "../mhc_hyper_connection_pre_gb300/csrc/kv_index.cuh"

using namespace mhc::kv;

static Seqs make(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P, int pages) {
    int log2 = 0;
    while ((1 << log2) < P) ++log2;
    return Seqs{table, lens, cu, width, B, T, log2, pages};
}

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

// The segments of block `block` of `blocks`: out[i] = {sequence, tile, head,
// first unit, units, units of the tile, first key, last key + 1, blocks from here on}.  Returns how
// many, or -1 if there are more than `most`; total: units of the whole line.
int kv_segments(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P,
                int pages, int heads, int group, int tile_rows, int unit_log2, int block, int blocks, int32_t* out,
                int most, int64_t* total) {
    const Seqs s = make(table, lens, cu, width, B, T, P, pages);
    const Cut c{heads, group, tile_rows, unit_log2};
    *total = 0;
    for (int b = 0; b < B; ++b) *total += units_of_seq(info_of(span_of(s, b), group), c);
    int64_t from, to, seen = 0;
    share_of(*total, block, blocks, from, to);
    int n = 0, b = 0;
    for (; b < B; ++b) {
        const int64_t u = units_of_seq(info_of(span_of(s, b), group), c);
        if (from < seen + u) break;
        seen += u;
    }
    int64_t left = to - from, r = from - seen;
    for (; left > 0; ++b) {
        const SeqInfo info = info_of(span_of(s, b), group);
        if (info.rows == 0) continue;
        Walk w;
        walk_enter(w, info, c, r, left);
        r = 0;
        do {
            if (n == most) return -1;
            const Segment g{b, info, w.t.tile, w.head, w.first, w.count, w.t.units,
                            blocks_beyond(*total, block, blocks, w.t.units - w.first - w.count) + 1};
            int32_t* o = out + 9 * n++;
            o[0] = b;
            o[1] = g.tile;
            o[2] = g.head;
            o[3] = g.first;
            o[4] = g.count;
            o[5] = g.units;
            keys_of(g, c, o[6], o[7]);
            o[8] = g.parts;
        } while (walk_next(w, info, c));
        left = w.left;
    }
    return n;
}

}
