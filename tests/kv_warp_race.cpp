// The hand-over of a share's segments inside a warp, compiled for the host by
// test_kv_cpu.py with a race detector: the lanes are threads, and a vote
// synchronises them without ordering their memory, as the hardware's may.
#include "../mhc_hyper_connection_pre_gb300/csrc/kv_index.cuh"

#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

using namespace mhc::kv;

constexpr int kLanes = 8, kSlots = 8;

// A barrier of the lanes; `order` says whether it orders their memory.
struct Lanes {
    std::atomic<int> count{0}, turn{0}, votes[2] = {{0}, {0}};
    void meet(std::memory_order arrive, std::memory_order leave) {
        const int now = turn.load(std::memory_order_relaxed);
        if (count.fetch_add(1, arrive) + 1 == kLanes) {
            count.store(0, std::memory_order_relaxed);
            turn.store(now + 1, arrive == std::memory_order_relaxed ? arrive : std::memory_order_release);
        } else {
            while (turn.load(leave) == now) std::this_thread::yield();
        }
    }
};

struct HostWarp {
    Lanes& lanes;
    int lane;
    mutable int round = 0;
    bool first() const { return lane == 0; }
    bool any(bool x) const {
        std::atomic<int>& v = lanes.votes[round++ & 1];
        if (x) v.fetch_add(1, std::memory_order_relaxed);
        lanes.meet(std::memory_order_relaxed, std::memory_order_relaxed);
        const bool r = v.load(std::memory_order_relaxed) > 0;
        lanes.meet(std::memory_order_relaxed, std::memory_order_relaxed);
        if (lane == 0) v.store(0, std::memory_order_relaxed);      // two rounds before its next use
        return r;
    }
    void sync() const { lanes.meet(std::memory_order_acq_rel, std::memory_order_acquire); }
};

struct Look {
    const std::vector<SeqInfo>& seqs;
    int count() const { return (int)seqs.size(); }
    SeqInfo operator()(int b) const { return seqs[b]; }
};

int main() {
    const std::vector<SeqInfo> seqs = {{0, 3, 100}, {3, 1, 0}, {4, 0, 0}, {4, 40, 900}, {44, 1, 63}};
    const Cut cut = make_cut(2, 5, 4, 5, 3);
    int64_t total = 0;
    for (const SeqInfo& s : seqs) total += units_of_seq(s, cut);
    const Shares shares = shares_of(total, 1);
    Plan plan;
    plan.b = 0;
    plan.info = seqs[0];
    plan.at = 0;
    walk_enter(plan.w, plan.info, cut, 0, total);
    Segment queue[kSlots];
    Lanes lanes;
    int64_t seen[kLanes];
    std::vector<std::thread> threads;
    for (int lane = 0; lane < kLanes; ++lane)
        threads.emplace_back([&, lane] {
            const HostWarp warp{lanes, lane};
            const Look look{seqs};
            int64_t sum = 0;
            for (int n = 0;; ++n) {
                if (n && n % kSlots == 0) warp.sync();             // a segment is done with before its slot is used again
                Segment& s = queue[n % kSlots];
                if (!found_for_all(warp, [&] { return plan.w.left > 0 && plan_next(plan, look, cut, shares, s); })) break;
                sum = sum * 31 + s.b + s.head + s.token + s.key0 + s.keys + s.rows;
            }
            seen[lane] = sum;
        });
    for (std::thread& t : threads) t.join();
    for (int64_t s : seen)
        if (s != seen[0]) return 1;
    std::printf("%lld\n", (long long)seen[0]);
    return seen[0] == 0;
}
