// The kv kernels' index arithmetic, compiled for the host by test_kv_cpu.py.
#include "../mhc_hyper_connection_pre_gb300/csrc/kv_index.cuh"

using namespace mhc::kv;

static Seqs make(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P, int pages) {
    return Seqs{table, lens, cu, width, B, T, P, pages};
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

// The segments of block `block` of `blocks`, table by table as the kernel
// walks them: out[i] = {sequence, tile, head, first unit, units, units of the
// tile}.  Returns how many, or -1 if there are more than `most`; total: units
// of the whole line.
int kv_segments(const int32_t* table, const int32_t* lens, const int32_t* cu, int width, int B, int T, int P,
                int pages, int heads, int group, int tile_rows, int unit, int table_size, int block, int blocks, int32_t* out,
                int most, int64_t* total) {
    const Seqs s = make(table, lens, cu, width, B, T, P, pages);
    const Cut c{heads, group, tile_rows, unit};
    *total = 0;
    for (int b = 0; b < B; ++b) *total += units_of_seq(info_of(span_of(s, b), group), c);
    int64_t from, to;
    share_of(*total, block, blocks, from, to);
    int64_t seen = 0;
    int n = 0;
    SeqInfo* info = new SeqInfo[table_size];
    int64_t* prefix = new int64_t[table_size];
    for (int base = 0; base < B; base += table_size) {
        int64_t here = 0;
        for (int i = 0; i < table_size; ++i) {
            info[i] = base + i < B ? info_of(span_of(s, base + i), group) : SeqInfo{0, 0, 0, 0};
            prefix[i] = here;
            here += units_of_seq(info[i], c);
        }
        const int64_t lo = (from > seen ? from : seen) - seen, hi = (to < seen + here ? to : seen + here) - seen;
        seen += here;
        if (hi <= lo) continue;
        Walk w;
        for (walk_start(w, info, prefix, table_size, c, lo, hi - lo); w.left > 0; walk_next(w, info, c)) {
            if (n == most) { n = -1; break; }
            int32_t* o = out + 6 * n++;
            o[0] = base + w.b;
            o[1] = w.tile;
            o[2] = w.head;
            o[3] = w.first;
            o[4] = w.count;
            o[5] = w.units;
        }
        if (n < 0) break;
    }
    delete[] info;
    delete[] prefix;
    return n;
}

}
