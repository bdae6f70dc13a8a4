// The planning of mhc_kv_fork and mhc_kv_compact, compiled for the host by
// test_kv_more_cpu.py, by as many threads as the input asks for, with the address
// and the thread sanitizer.  Reads cases as numbers from the standard input until
// it ends, and writes each one's outputs as a line of numbers.
#include "../mhc_hyper_connection_pre_gb300/csrc/kv_pages.cuh"

#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>

using namespace mhc::kv;

struct Meeting {
    int size;
    std::mutex m;
    std::condition_variable cv;
    int waiting = 0, turn = 0;
    std::vector<int64_t> parts;
    unsigned int status = 0;
    void meet() {
        std::unique_lock<std::mutex> lock(m);
        const int now = turn;
        if (++waiting == size) {
            waiting = 0;
            ++turn;
            cv.notify_all();
        } else {
            cv.wait(lock, [&] { return turn != now; });
        }
    }
};

struct HostTeam {
    int rank, size;
    Meeting* all;
    void sync() const { all->meet(); }
    int64_t scan(int64_t x, int64_t& total) const {
        all->parts[rank] = x;
        sync();
        int64_t before = 0;
        total = 0;
        for (int i = 0; i < size; ++i) {
            before += i < rank ? all->parts[i] : 0;
            total += all->parts[i];
        }
        sync();
        return before;
    }
    template <class T>
    T load(const T* p) const { return __atomic_load_n(p, __ATOMIC_RELAXED); }
    void store(int32_t* p, int32_t x) const { __atomic_store_n(p, x, __ATOMIC_RELAXED); }
    void set_bit(uint32_t* bits, int page) const {
        if (page >= 0) __atomic_fetch_or(bits + page / 32, 1u << page % 32, __ATOMIC_RELAXED);
    }
    void lower(int32_t* p, int32_t x) const {
        for (int32_t v = load(p); x < v && !__atomic_compare_exchange_n(p, &v, x, true, __ATOMIC_RELAXED, __ATOMIC_RELAXED);) {}
    }
    void raise(int32_t* p, int32_t x) const {
        for (int32_t v = load(p); x > v && !__atomic_compare_exchange_n(p, &v, x, true, __ATOMIC_RELAXED, __ATOMIC_RELAXED);) {}
    }
    void report(unsigned int x) const { __atomic_fetch_or(&all->status, x, __ATOMIC_RELAXED); }
};

template <class F>
unsigned int run(int size, F&& f) {
    Meeting all;
    all.size = size;
    all.parts.resize(size);
    std::vector<std::thread> threads;
    for (int r = 0; r < size; ++r)
        threads.emplace_back([&, r] {
            HostTeam t{r, size, &all};
            f(t);
        });
    for (std::thread& t : threads) t.join();
    return all.status;
}

static int64_t number() {
    long long x;
    if (std::scanf("%lld", &x) != 1) std::exit(0);
    return x;
}

template <class T>
std::vector<T> numbers(int64_t n) {
    std::vector<T> v(n);
    for (T& x : v) x = (T)number();
    return v;
}

template <class T>
std::vector<T> scratch(int64_t n) {           // contents on entry do not matter
    std::vector<T> v(n);
    for (size_t i = 0; i < v.size() * sizeof(T); ++i) reinterpret_cast<uint8_t*>(v.data())[i] = 0x5a;
    return v;
}

template <class T>
const T* given(const std::vector<T>& v) { return v.empty() ? nullptr : v.data(); }

static void print(const int32_t* p, int64_t n) {
    for (int64_t i = 0; i < n; ++i) std::printf("%d ", p[i]);
}

int main() {
    for (;;) {
        const bool fork = number() == 0;
        const int size = (int)number(), width = (int)number(), B_in = (int)number(), B = (int)number();
        const int log2 = (int)number(), pages = (int)number();
        const bool in_place = number(), has_held = number(), rows_apart = number();
        std::vector<int32_t> table = numbers<int32_t>((int64_t)B_in * width), lens = numbers<int32_t>(B_in);
        const std::vector<uint8_t> held = numbers<uint8_t>(has_held ? pages : 0);
        std::vector<int32_t> table_out = scratch<int32_t>((int64_t)B * width), lens_out = scratch<int32_t>(B);
        std::vector<uint32_t> bits = scratch<uint32_t>(words_of(pages));
        const PagesIn p{table.data(), lens.data(), given(held), in_place ? table.data() : table_out.data(), width, B_in, B,
                        log2, pages};
        int32_t count = 0x5a5a5a5a, top = 0x5a5a5a5a;
        unsigned int status;
        std::vector<PageCopy> copies;
        if (fork) {
            const bool has_parents = number(), has_room = number();
            const std::vector<int32_t> parents = numbers<int32_t>(has_parents ? B : 0), room = numbers<int32_t>(has_room ? B : 0);
            const int room_all = (int)number(), window = (int)number(), sinks = (int)number();
            const int64_t most = (int64_t)B * (width + 1);
            std::vector<Place> place = scratch<Place>(B);
            std::vector<int32_t> first = scratch<int32_t>(B), keeper = scratch<int32_t>(pages),
                                 out = scratch<int32_t>(most < pages ? most : pages);
            copies = scratch<PageCopy>(B);
            const ForkIn a{p, given(parents), given(room), room_all, window, sinks, in_place ? lens.data() : lens_out.data()};
            const ForkSpace s{bits.data(), place.data(), first.data(), keeper.data(), out.data(),
                              copies.data(), &count};
            if (rows_apart) {
                std::vector<uint32_t> own = scratch<uint32_t>(words_of(pages));
                for (uint32_t& w : bits) w = 0;
                ForkSpace rest = s;
                rest.bits = own.data();
                status = run(size, [&](HostTeam& t) { fork_rows(t, a, s); });
                status |= run(size, [&](HostTeam& t) { fork_rest(t, a, rest, s.bits); });
            } else {
                status = run(size, [&](HostTeam& t) { plan_fork(t, a, s); });
            }
            print(in_place ? lens.data() : lens_out.data(), B);
        } else {
            std::vector<int32_t> mover = scratch<int32_t>(pages), hole = scratch<int32_t>(pages), moved = scratch<int32_t>(pages),
                                 mark = scratch<int32_t>(2), entries = scratch<int32_t>(B);
            copies = scratch<PageCopy>(pages);
            std::vector<uint32_t> held_bits = scratch<uint32_t>(words_of(pages));
            const CompactSpace s{bits.data(), held_bits.data(), entries.data(), mover.data(), hole.data(), moved.data(), copies.data(), &count, mark.data()};
            if (rows_apart) {
                std::vector<uint32_t> own = scratch<uint32_t>(words_of(pages));
                for (uint32_t& w : bits) w = 0;
                CompactSpace moves = s;
                moves.bits = own.data();
                status = run(size, [&](HostTeam& t) { compact_rows(t, p, s); });
                status |= run(size, [&](HostTeam& t) { compact_moves(t, p, &top, moves, s.bits); });
                status |= run(size, [&](HostTeam& t) {
                    compact_rename(t, p, s, [&](int b) {
                        const int64_t n = lens[b], cap = (int64_t)width << log2;
                        return pages_for(n < 0 ? 0 : (n > cap ? cap : n), log2);
                    });
                });
            } else {
                status = run(size, [&](HostTeam& t) { plan_compact(t, p, &top, s); });
            }
            std::printf("%d ", top);
        }
        print(in_place ? table.data() : table_out.data(), (int64_t)B * width);
        std::printf("%u %d ", status, count);
        for (int i = 0; i < count; ++i) std::printf("%d %d %d ", copies.at(i).from, copies.at(i).to, copies.at(i).slots);
        std::printf("\n");
    }
}
