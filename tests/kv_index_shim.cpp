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

}
