// The rows of large tables (kv_pages.cuh), written in place by teams of any number of threads that
// meet nowhere, compiled for the host by test_kv_edges_cpu.py with the thread sanitizer.  Reads cases as numbers from
// the standard input until it ends, and writes each one's outputs as a line of numbers, as kv_pages_shim.cpp does.
#define main pages_main
#include "kv_pages_shim.cpp"
#undef main

int main() {
    for (;;) {
        const bool fork = number() == 0;
        const int size = (int)number(), width = (int)number(), B = (int)number(), log2 = (int)number(), pages = (int)number();
        std::vector<int32_t> table = numbers<int32_t>((int64_t)B * width), lens = numbers<int32_t>(B);
        std::vector<uint32_t> bits(words_of(pages)), own = scratch<uint32_t>(words_of(pages));
        const PagesIn p{table.data(), lens.data(), nullptr, table.data(), width, B, B, log2, pages};
        const int planners = 8;                   // a power of two, unlike the rows' threads
        int32_t count = 0, top = 0;
        unsigned int status;
        std::vector<PageCopy> copies;
        if (fork) {
            const int room = (int)number(), window = (int)number(), sinks = (int)number();
            const int64_t most = (int64_t)B * (width + 1);
            std::vector<Place> place = scratch<Place>(B);
            std::vector<int32_t> first = scratch<int32_t>(B), keeper = scratch<int32_t>(pages),
                                 out = scratch<int32_t>(most < pages ? most : pages);
            copies = scratch<PageCopy>(B);
            const ForkIn a{p, nullptr, nullptr, room, window, sinks, lens.data()};
            const ForkSpace s{bits.data(), place.data(), first.data(), keeper.data(), out.data(), copies.data(), &count};
            ForkSpace rest = s;
            rest.bits = own.data();
            status = run(size, [&](HostTeam& t) { fork_rows(t, a, s); });
            status |= run(planners, [&](HostTeam& t) { fork_rest(t, a, rest, s.bits); });
            print(lens.data(), B);
        } else {
            std::vector<int32_t> mover = scratch<int32_t>(pages), hole = scratch<int32_t>(pages), moved = scratch<int32_t>(pages),
                                 mark = scratch<int32_t>(2), entries = scratch<int32_t>(B);
            std::vector<uint32_t> held_bits = scratch<uint32_t>(words_of(pages));
            copies = scratch<PageCopy>(pages);
            const CompactSpace s{bits.data(), held_bits.data(), entries.data(), mover.data(), hole.data(), moved.data(),
                                 copies.data(), &count, mark.data()};
            CompactSpace moves = s;
            moves.bits = own.data();
            status = run(size, [&](HostTeam& t) { compact_rows(t, p, s); });
            status |= run(planners, [&](HostTeam& t) { compact_moves(t, p, &top, moves, s.bits); });
            status |= run(size, [&](HostTeam& t) {
                compact_rename(t, p, s, [&](int b) { return pages_for(lens[b], log2); });
            });
            std::printf("%d ", top);
        }
        print(table.data(), (int64_t)B * width);
        std::printf("%u %d ", status, count);
        for (int i = 0; i < count; ++i) std::printf("%d %d %d ", copies.at(i).from, copies.at(i).to, copies.at(i).slots);
        std::printf("\n");
    }
}
