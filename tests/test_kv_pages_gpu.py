"""GPU checks of mhc_kv_fork and mhc_kv_compact against their definitions, and
of a decoding loop over shared pages."""
import random
import threading

import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from mhc_hyper_connection_pre_gb300.graphs import SeamGraph
from test_kv_more_cpu import plan_compact, plan_fork

pytestmark = pytest.mark.gpu

INDEX_ERROR, PAGES_ERROR = 5, 6


@pytest.fixture(autouse=True)
def _status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mhc.load_library()
    assert mhc.device_status() == 0
    yield
    assert mhc.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def caches_of(shapes, pages, P, seed):
    """A cache of random bytes for each (heads, dim)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for H, D in shapes:
        c = mhc.kv_cache(pages, H, P, D)
        for n in ("k", "v"):
            c[n].view(torch.uint8).copy_(torch.randint(0, 256, c[n].shape, generator=g, device="cuda", dtype=torch.uint8))
            c[n + "_scale"].copy_(torch.rand(pages, H, generator=g, device="cuda"))
        out.append(c)
    return out


def bytes_of(caches):
    return [{n: t.view(torch.uint8).clone() if n in "kv" else t.clone() for n, t in c.items()} for c in caches]


def check_copies(caches, before, copies):
    """The caches are what they were, but for the copied slots and their pages' scales."""
    for c, was in zip(caches, before):
        want = {n: t.clone() for n, t in was.items()}
        for a, b, slots in copies:
            if b >= 0:
                for n in ("k", "v"):
                    want[n][b, :, :slots] = was[n][a, :, :slots]
                    want[n + "_scale"][b] = was[n + "_scale"][a]
        for n, t in c.items():
            assert torch.equal(t.view(torch.uint8) if n in "kv" else t, want[n]), n


def batch(r, B, width, pages, P, shared=0.5):
    """Lengths and tables of a batch, pages shared from the front by some, entries past the lengths anything."""
    lens = [r.choice([0, r.randint(0, width * P), r.randint(0, width * P), P]) for _ in range(B)]
    order = iter(r.sample(range(pages), min(pages, sum(-(-n // P) for n in lens))))
    table = [[next(order) if i * P < n else r.choice([-1, -7, 10 ** 9]) for i in range(width)] for n in lens]
    for b in range(1, B):
        if r.random() < shared:
            a = r.randrange(b)
            lens[b], table[b] = lens[a], list(table[a])
    return lens, table


SHAPES = [[(2, 64)], [(1, 128), (3, 64), (2, 128)], [(8, 128)] * 2]

FORKS = [
    # places, width, pages, P, parents, room, window, sinks, held
    (1, 1, 3, 16, False, 1, 0, 0, False),
    (7, 5, 60, 16, True, 0, 0, 0, True),
    (40, 3, 200, 64, True, 1, 0, 0, False),
    (33, 9, 400, 32, False, [0, 5, 70], 0, 0, True),
    (64, 12, 1500, 128, True, 300, 0, 0, False),
    (100, 30, 5000, 16, True, 1, 100, 20, True),
    (5, 200, 1400, 16, False, 1, 1, 0, False),
    (700, 120, 60000, 16, True, 1, 0, 0, True),               # a cluster plans
    (520, 130, 40000, 32, False, 40, 500, 33, False),
]


@pytest.mark.parametrize("case", range(len(FORKS)))
def test_fork_is_its_definition(case):
    B, width, pages, P, with_parents, room, window, sinks, with_held = FORKS[case]
    r = random.Random(case)
    lens, table = batch(r, B, width, pages, P)
    parents = [r.randint(-1, B - 1) for _ in range(B + r.choice([0, 3]))] if with_parents else None
    places = B if parents is None else len(parents)
    room = [min(r.choice(room), width * P - (lens[b] if parents is None else 0)) for b in range(places)] if isinstance(room, list) else room
    held = [r.random() < 0.1 for _ in range(pages)] if with_held else None
    if not isinstance(room, list):                             # lengths that leave the room that is asked for
        lens = [min(n, width * P - room) for n in lens]
    caches = caches_of(SHAPES[case % 3], pages, P, case)
    before = bytes_of(caches)
    got = mhc.kv_fork(caches, _i32(table), _i32(lens), None if parents is None else _i32(parents),
                      room=_i32(room) if isinstance(room, list) else room, window=window or None, sinks=sinks,
                      held=None if held is None else torch.tensor(held, device="cuda"))
    out, n, copies, status = plan_fork(table, lens, pages, P.bit_length() - 1, parents, room, window, sinks, held)
    assert mhc.device_status() == {0: 0, 4: PAGES_ERROR}[status]
    assert got["block_table"].tolist() == out and got["seq_lens"].tolist() == n
    check_copies(caches, before, copies)


COMPACTS = [
    # places, width, pages, P, held
    (1, 1, 3, 16, False), (7, 5, 60, 16, True), (40, 3, 250, 64, False), (24, 44, 3000, 16, True), (100, 30, 5000, 16, True),
    (700, 120, 90000, 16, True), (530, 130, 80000, 16, False), (3, 4, 12, 128, False),
]


@pytest.mark.parametrize("case", range(len(COMPACTS)))
def test_compact_is_its_definition(case):
    B, width, pages, P, with_held = COMPACTS[case]
    r = random.Random(50 + case)
    lens, table = batch(r, B, width, pages, P, shared=0.2)
    for row in table:                                          # some pages were let go
        for i in range(width):
            if r.random() < 0.1:
                row[i] = -1
    held = [r.random() < 0.1 for _ in range(pages)] if with_held else None
    caches = caches_of(SHAPES[case % 3], pages, P, case)
    before = bytes_of(caches)
    got = mhc.kv_compact(caches, _i32(table), _i32(lens), held=None if held is None else torch.tensor(held, device="cuda"))
    out, top, copies, status = plan_compact(table, lens, pages, P.bit_length() - 1, held)
    assert status == 0 and got["pages"].shape == () and got["pages"].item() == top
    assert got["block_table"].tolist() == out
    check_copies(caches, before, copies)


def test_many_caches_of_different_heads():
    """More than one launch of copies: 70 caches."""
    r = random.Random(3)
    lens, table = batch(r, 9, 4, 90, 16)
    parents = [r.randint(0, 8) for _ in range(20)]
    caches = caches_of([(1 + i % 3, 64 if i % 2 else 128) for i in range(70)], 90, 16, 4)
    before = bytes_of(caches)
    got = mhc.kv_fork(tuple(caches), _i32(table), _i32(lens), _i32(parents))
    out, n, copies, _ = plan_fork(table, lens, 90, 4, parents, 0, 0, 0, None)
    assert got["block_table"].tolist() == out and copies
    check_copies(caches, before, copies)
    table, before = got["block_table"].tolist(), bytes_of(caches)
    got = mhc.kv_compact(caches, got["block_table"], got["seq_lens"])
    out, top, copies, _ = plan_compact(table, n, 90, 4, None)
    assert got["block_table"].tolist() == out and got["pages"].item() == top and copies
    check_copies(caches, before, copies)


def test_one_cache_alone_and_outputs_given():
    """A single cache instead of a sequence; in place; outputs of the caller."""
    r = random.Random(5)
    lens, table = batch(r, 6, 4, 40, 16, shared=0)
    lens = [min(n, 60) for n in lens]
    (c,) = caches_of([(2, 64)], 40, 16, 5)
    expect = mhc.kv_fork(c, _i32(table), _i32(lens), room=3)
    t, n = _i32(table), _i32(lens)
    got = mhc.kv_fork([c], t, n, room=3, out={"block_table": t, "seq_lens": n})
    assert got["block_table"] is t and got["seq_lens"] is n
    assert torch.equal(t, expect["block_table"]) and torch.equal(n, expect["seq_lens"])
    a = mhc.kv_compact(caches_of([(2, 64)], 40, 16, 5), t, n)
    pages = torch.empty((), dtype=torch.int32, device="cuda")
    b = mhc.kv_compact(c, t, n, out={"block_table": t, "pages": pages})
    assert b["block_table"] is t and b["pages"] is pages
    assert torch.equal(t, a["block_table"]) and torch.equal(pages, a["pages"])


def test_large_tables_in_place():
    """Tables whose rows have kernels of their own, written over themselves: as into new ones."""
    r = random.Random(15)
    lens, table = batch(r, 300, 130, 30000, 16, shared=0.3)
    lens = [min(n, 129 * 16) for n in lens]
    a, b = caches_of([(1, 64)], 30000, 16, 15), caches_of([(1, 64)], 30000, 16, 15)
    expect = mhc.kv_fork(a, _i32(table), _i32(lens), room=9, window=700, sinks=20)
    t, n = _i32(table), _i32(lens)
    mhc.kv_fork(b, t, n, room=9, window=700, sinks=20, out={"block_table": t, "seq_lens": n})
    assert torch.equal(t, expect["block_table"]) and torch.equal(n, expect["seq_lens"])
    moved = mhc.kv_compact(a, expect["block_table"], n)
    got = mhc.kv_compact(b, t, n, out={"block_table": t})
    assert torch.equal(t, moved["block_table"]) and torch.equal(got["pages"], moved["pages"])
    for x, y in zip(bytes_of(a), bytes_of(b)):
        assert all(torch.equal(x[k], y[k]) for k in x)


def test_running_out_of_pages_is_reported():
    (c,) = caches_of([(1, 64)], 4, 16, 6)
    table, lens = _i32([[0, 1, 2, -1, -1], [3, -1, -1, -1, -1]]), _i32([48, 16])
    got = mhc.kv_fork(c, table, lens, room=1)
    assert mhc.device_status() == PAGES_ERROR
    assert got["block_table"].tolist() == [[0, 1, 2, -1, -1], [3, -1, -1, -1, -1]]
    got = mhc.kv_fork(c, table, lens, _i32([1, 1]), room=1)                        # the first one's pages are free now
    assert got["block_table"].tolist() == [[3, 0, -1, -1, -1], [3, 1, -1, -1, -1]]
    before = bytes_of([c])
    got = mhc.kv_fork(c, _i32([[0, 1, 2, 3]]), _i32([63]), _i32([0, 0]))           # nothing to copy to
    assert mhc.device_status() == PAGES_ERROR
    assert got["block_table"].tolist() == [[0, 1, 2, 3], [0, 1, 2, -1]]
    check_copies([c], before, [])


def test_bad_indices():
    (c,) = caches_of([(1, 64)], 6, 16, 7)
    table = [[0, 6, 1], [2, -2, -1], [-1, 2147483647, 4]]
    for lens, parents, room in (([40, 16, 48], None, 0), ([-1, 49, 2147483647], None, 0), ([16, 16, 16], [0, 3, -2], 0),
                                ([16, 16, 16], None, [5, -1, 2147483647])):
        before = bytes_of([c])
        got = mhc.kv_fork(c, _i32(table), _i32(lens), None if parents is None else _i32(parents),
                          room=_i32(room) if isinstance(room, list) else room)
        out, n, copies, status = plan_fork(table, lens, 6, 4, parents, room, 0, 0, None)
        assert mhc.device_status() == INDEX_ERROR and status & 2
        assert got["block_table"].tolist() == out and got["seq_lens"].tolist() == n
        check_copies([c], before, copies)
    got = mhc.kv_compact(c, _i32(table), _i32([48, -5, 2147483647]))
    out, top, _, status = plan_compact(table, [48, -5, 2147483647], 6, 4, None)
    assert mhc.device_status() == INDEX_ERROR and status == 2
    assert got["block_table"].tolist() == out and got["pages"].item() == top


def test_no_places_and_no_pages_in_use():
    (c,) = caches_of([(1, 64)], 6, 16, 8)
    none, no_rows = _i32([]), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    got = mhc.kv_fork(c, no_rows, none)
    assert got["block_table"].shape == (0, 3) and got["seq_lens"].shape == (0,)
    got = mhc.kv_fork(c, no_rows, none, _i32([-1, -1]), room=17)                   # a first batch
    assert got["block_table"].tolist() == [[0, 1, -1], [2, 3, -1]] and got["seq_lens"].tolist() == [0, 0]
    held = torch.tensor([False, True, False, False, False, False], device="cuda")
    assert mhc.kv_compact(c, no_rows, none)["pages"].item() == 0
    assert mhc.kv_compact(c, no_rows, none, held=held)["pages"].item() == 2
    assert mhc.kv_compact(c, _i32([[5]]), _i32([0]))["pages"].item() == 0


def test_held_as_bytes_of_any_value():
    (c,) = caches_of([(1, 64)], 37, 16, 9)
    held = torch.zeros(37, dtype=torch.uint8, device="cuda")
    held[[0, 2, 35, 36]] = torch.tensor([1, 128, 255, 2], dtype=torch.uint8, device="cuda")
    got = mhc.kv_fork(c, _i32([[0, -1, -1]]), _i32([5]), _i32([0, -1]), room=30, held=held)
    assert got["block_table"].tolist() == [[1, 3, 4], [5, 6, -1]]                  # 0 is held: copied


def test_far_pages():
    """Pages that begin beyond 2^32 bytes are copied and moved."""
    H, P, D = 8, 128, 128
    pages = (1 << 32) // (H * P * D) + 40
    c = mhc.kv_cache(pages, H, P, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    bits = torch.randint(0, 256, (2, H, P, D), generator=g, device="cuda", dtype=torch.uint8)
    for n in ("k", "v"):
        c[n].view(torch.uint8)[pages - 2:] = bits if n == "k" else bits.flip(0)
        c[n + "_scale"][pages - 2:] = 3.0
    held = torch.zeros(pages, dtype=torch.bool, device="cuda")
    held[:pages - 10] = True
    got = mhc.kv_fork(c, _i32([[pages - 2, pages - 1]]), _i32([200]), _i32([0, 0]), held=held)
    assert got["block_table"].tolist() == [[pages - 2, pages - 1], [pages - 2, pages - 10]]
    assert torch.equal(c["k"].view(torch.uint8)[pages - 10, :, :72], bits[1, :, :72])
    assert torch.equal(c["v"].view(torch.uint8)[pages - 10, :, :72], bits[0, :, :72])
    assert (c["k"].view(torch.uint8)[pages - 10, :, 72:] == 0).all() and (c["v_scale"][pages - 10] == 3).all()
    got = mhc.kv_compact(c, _i32([[pages - 2, pages - 1]]), _i32([200]))
    assert got["block_table"].tolist() == [[0, 1]] and got["pages"].item() == 2
    assert torch.equal(c["k"].view(torch.uint8)[:2], bits) and torch.equal(c["v"].view(torch.uint8)[:2], bits.flip(0))
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("pages", [1_100_000, 1_700_000])
def test_many_pages(pages):
    """More pages than one block takes beside the rows, and than its shared memory has bits for."""
    r = random.Random(pages)
    B, width = 20, 12
    lens = [r.randint(0, width * 16 - 20) for _ in range(B)]
    pick = r.sample(range(pages), B * width)
    table = [[pick[b * width + i] if i * 16 < n else -1 for i in range(width)] for b, n in enumerate(lens)]
    parents = [r.randint(-1, B - 1) for _ in range(2 * B)]
    hold = set(range(300)) | set(range(pages - 70, pages - 10)) | set(r.sample(pick, 9))
    held = torch.zeros(pages, dtype=torch.bool, device="cuda")
    held[list(hold)] = True
    flags = held.tolist()
    c = mhc.kv_cache(pages, 1, 16, 64)
    for n in ("k", "v"):
        c[n].view(torch.uint8)[pick] = torch.randint(0, 256, (len(pick), 1, 16, 64), device="cuda", dtype=torch.uint8)
    got = mhc.kv_fork(c, _i32(table), _i32(lens), _i32(parents), room=20, held=held)
    out, n, copies, status = plan_fork(table, lens, pages, 4, parents, 20, 0, 0, flags)
    assert status == 0 and copies
    assert got["block_table"].tolist() == out and got["seq_lens"].tolist() == n
    for a, b, slots in copies:
        assert torch.equal(c["k"].view(torch.uint8)[b, 0, :slots], c["k"].view(torch.uint8)[a, 0, :slots])
    got = mhc.kv_compact(c, _i32(table), _i32(lens), held=held)
    out, top, copies, _ = plan_compact(table, lens, pages, 4, flags)
    assert got["block_table"].tolist() == out and got["pages"].item() == top and copies
    for a, b, _ in copies:
        assert torch.equal(c["v"].view(torch.uint8)[b], c["v"].view(torch.uint8)[a])
    none, no_rows = _i32([]), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    assert mhc.kv_compact(c, no_rows, none, held=held)["pages"].item() == pages - 10
    del c
    torch.cuda.empty_cache()


def test_stream_graph_and_workspace():
    """On another stream, with a workspace of any contents, and captured and replayed: the same."""
    r = random.Random(12)
    lens, table = batch(r, 30, 9, 400, 16)
    parents = _i32([r.randint(-1, 29) for _ in range(30)])
    t, n = _i32(table), _i32(lens)
    a, b = caches_of([(2, 64), (1, 128)], 400, 16, 12), caches_of([(2, 64), (1, 128)], 400, 16, 12)
    expect = mhc.kv_fork(a, t, n, parents, room=1)
    moved = mhc.kv_compact(a, expect["block_table"], expect["seq_lens"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = mhc.kv_fork(b, t, n, parents, room=1, stream=st)
    again = mhc.kv_compact(b, got["block_table"], got["seq_lens"], stream=st)
    st.synchronize()
    for x, y in ((expect, got), (moved, again)):
        assert all(torch.equal(x[k], y[k]) for k in x)
    for x, y in zip(bytes_of(a), bytes_of(b)):
        assert all(torch.equal(x[k], y[k]) for k in x)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for fill in (0xFF, 0x7F, 0):
        ws.fill_(fill)
        got = mhc.kv_fork(b, t, n, parents, room=1, workspace=ws)
        assert all(torch.equal(expect[k], got[k]) for k in got)
        ws.fill_(fill)
        again = mhc.kv_compact(b, got["block_table"], got["seq_lens"], workspace=ws)
        assert all(torch.equal(moved[k], again[k]) for k in again)
    out = {"block_table": torch.zeros_like(expect["block_table"]), "seq_lens": torch.zeros_like(expect["seq_lens"])}
    fin = {"block_table": torch.zeros_like(out["block_table"]), "pages": torch.zeros((), dtype=torch.int32, device="cuda")}
    def calls(stream=None):
        mhc.kv_fork(b, t, n, parents, room=1, out=out, stream=stream)
        mhc.kv_compact(b, out["block_table"], out["seq_lens"], out=fin, stream=stream)
    graphs = [SeamGraph(calls, st), SeamGraph(calls, st, early_launch=True)]
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            calls()
        graphs.append(graph)
    for graph in graphs + graphs:
        for x in (*out.values(), *fin.values()):
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        mhc.kv_fork(a, t, n, parents, room=1)                   # the stream's own workspace meanwhile
        torch.cuda.synchronize()
        assert all(torch.equal(expect[k], out[k]) for k in out) and all(torch.equal(moved[k], fin[k]) for k in fin)


def test_two_streams_at_once():
    """Calls on two streams, each with tables and caches of its own, small and large: as one after the other."""
    r = random.Random(16)
    sets = []
    for B, width, pages in ((40, 9, 500), (400, 90, 40000)):
        lens, table = batch(r, B, width, pages, 16)
        lens = [min(n, width * 16 - 1) for n in lens]
        parents = _i32([r.randint(-1, B - 1) for _ in range(B)])
        c = caches_of([(2, 64)], pages, 16, 16)
        expect = mhc.kv_fork(c, _i32(table), _i32(lens), parents, room=1)
        moved = mhc.kv_compact(c, expect["block_table"], expect["seq_lens"])
        sets.append((c, _i32(table), _i32(lens), parents, expect, moved, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for c, t, n, parents, _, _, st in sets:
            f = mhc.kv_fork(c, t, n, parents, room=1, stream=st)
            got.append((f, mhc.kv_compact(c, f["block_table"], f["seq_lens"], stream=st)))
    torch.cuda.synchronize()
    for i, (f, m) in enumerate(got):
        expect, moved = sets[i % 2][4:6]
        assert all(torch.equal(f[k], expect[k]) for k in f) and all(torch.equal(m[k], moved[k]) for k in m)


def test_two_threads_at_once():
    """C calls of two host threads, each of its own sizes: none refuses the other's shared memory."""
    lib = mhc.load_library()
    failed = []

    def calls(B, width, pages):
        c = caches_of([(1, 64)], pages, 16, B)[0]
        cache = mhc.kv._Cache(*(c[k].data_ptr() for k in ("k", "v", "k_scale", "v_scale")), pages, 1, 16, 64)
        table, lens = _i32([[b * width + i for i in range(width)] for b in range(B)]), _i32([width * 16 - 1] * B)
        top = torch.zeros(1, dtype=torch.int32, device="cuda")
        need = max(lib.mhc_kv_fork_workspace_bytes(pages, width, B), lib.mhc_kv_compact_workspace_bytes(pages, B))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        t, n = table.data_ptr(), lens.data_ptr()

        def run():
            for _ in range(1000):
                got = [lib.mhc_kv_fork(cache, 1, t, width, n, B, None, B, None, 1, None, 0, 0, t, n, ws.data_ptr(), need,
                                       st.cuda_stream),
                       lib.mhc_kv_compact(cache, 1, t, width, n, B, None, t, top.data_ptr(), ws.data_ptr(), need,
                                          st.cuda_stream)]
                if any(got):
                    failed.append(got)
            st.synchronize()
        return run, lambda: (table.tolist(), lens.tolist(), top.item())

    sides = [calls(4, 3, 12), calls(60, 50, 20000)]
    expect = [state() for _, state in sides]
    threads = [threading.Thread(target=run) for run, _ in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[:3]
    for (_, state), (table, lens, _), top in zip(sides, expect, (12, 3000)):
        assert state() == (table, lens, top)


def test_refusals():
    r = random.Random(13)
    lens, table = batch(r, 4, 3, 30, 16)
    a, b = caches_of([(2, 64)] * 2, 30, 16, 13)
    t, n = _i32(table), _i32(lens)
    before = bytes_of([a, b])

    def refused(error, call=mhc.kv_fork, caches=(a, b), t=t, n=n, status=None, **kw):
        with pytest.raises(error) as e:
            call(caches, t, n, **kw)
        assert status is None or e.value.status == status
    for call in (mhc.kv_fork, mhc.kv_compact):
        refused(ValueError, call, caches=())
        refused(TypeError, call, caches=(a, 3))
        refused(TypeError, call, caches=3)
        refused(ValueError, call, caches=(a, {"k": a["k"]}))
        refused(ValueError, call, caches=(a, mhc.kv_cache(31, 2, 16, 64)))
        refused(ValueError, call, caches=(a, mhc.kv_cache(30, 2, 32, 64)))
        refused(ValueError, call, caches=(a, mhc.kv_cache(30, 2, 16, 64, device="cpu")))
        refused(mhc.MhcError, call, caches=(a, a), status=1)                        # one cache twice
        refused(mhc.MhcError, call, caches=(a, dict(b, v=a["v"])), status=1)
        refused(ValueError, call, n=n[:3])
        refused(TypeError, call, t=t.long())
        refused(ValueError, call, t=t.cpu())
        refused(ValueError, call, held=torch.zeros(29, dtype=torch.bool, device="cuda"))
        refused(TypeError, call, held=torch.zeros(30, device="cuda"))
        refused(mhc.MhcError, call, held=torch.zeros(31, dtype=torch.bool, device="cuda")[1:], status=1)
        refused(mhc.MhcError, call, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), status=1)
        refused(ValueError, call, out={"block_table": t[:3]})
        refused(mhc.MhcError, call, out={"block_table": a["k_scale"].view(torch.int32).flatten()[:12].view(4, 3)}, status=1)
    p = _i32([0, 1, 2, 3])
    refused(mhc.MhcError, parents=p, out={"block_table": t}, status=1)              # in place, with parents
    refused(mhc.MhcError, parents=p, out={"seq_lens": p}, status=1)
    refused(mhc.MhcError, out={"seq_lens": t.flatten()[:4]}, status=1)
    refused(ValueError, parents=p[None])
    refused(TypeError, parents=p.long())
    refused(ValueError, parents=p, out={"seq_lens": n[:3]})
    refused(mhc.MhcError, room=-1, status=1)
    refused(TypeError, room=1.5)
    refused(ValueError, room=p[:3])
    refused(ValueError, window=0)
    refused(ValueError, sinks=3)
    refused(mhc.MhcError, window=3, sinks=-1, status=1)
    for x, y in zip(before, bytes_of([a, b])):
        assert all(torch.equal(x[k], y[k]) for k in x)


# --------------------------------------------------------------- together ---

def test_example_with_a_window():
    """examples/attention_decode.py with a window shorter than the prompts: token by token from a replayed graph, with
    pages handed out and let go in it, and at once; the same keys, with scales that grew differently (e4m3's half
    step, 2^-4, on either side)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_decode.py")
    spec = importlib.util.spec_from_file_location("attention_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    stepped, at_once = (t.double() for t in m.run(window=40, sinks=3))
    whole = m.run()[1].double()
    assert (stepped - at_once).norm() <= 2 * 2.0 ** -4 * at_once.norm()
    assert not torch.equal(whole, at_once)                     # the window hides something


@pytest.mark.parametrize("D,P,H,Hq,window,sinks,seed", [(128, 16, 2, 10, None, 0, 0), (64, 16, 1, 4, 40, 5, 1),
                                                        (128, 32, 2, 8, 20, 0, 2), (64, 64, 3, 3, 100, 70, 3)])
def test_decoding_over_shared_pages(D, P, H, Hq, window, sinks, seed):
    """Prompts, then steps in which places follow others, begin and end, over
    two layers in one pool of pages, compacted now and then; beside it caches
    in which every place has pages of its own, copied whole when it follows
    another.  The same keys, so the same outputs to the bit."""
    r, layers, width = random.Random(seed), 2, 24
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, pages = 6, 6 * 24 + 9
    pool = [mhc.kv_cache(pages, H, P, D) for _ in range(layers)]
    own = [mhc.kv_cache(B * width, H, P, D) for _ in range(layers)]
    own_table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    norms = [(1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).bfloat16() for _ in range(layers)]
    angle = torch.rand(width * P, D // 2, generator=g, device="cuda") * 6.3
    cos, sin = angle.cos(), angle.sin()
    held = torch.zeros(pages, dtype=torch.bool, device="cuda")
    held[[3, 50]] = True                                       # somebody else's
    for c in pool:
        for n in ("k", "v"):
            c[n].view(torch.uint8).fill_(0x7F)                 # what nothing was written to is NaN

    def layer(cache, table, lens, cu, qkv, norm):
        q, k, v = qkv.split([Hq, H, H], dim=1)
        q = mhc.kv_append(cache, k, v, table, lens, cu, q=q, cos=cos, sin=sin, q_norm=norm[0], k_norm=norm[1])
        return mhc.kv_attend(q, cache, table, lens, cu, window=window, sinks=sinks, return_lse=True)

    def step(table, lens, counts):
        """New tokens for every place; returns the lengths with them."""
        now = [n + m for n, m in zip(lens, counts)]
        cu = [0]
        for m in counts:
            cu.append(cu[-1] + m)
        for i in range(layers):
            qkv = torch.randn(cu[-1], Hq + 2 * H, D, generator=g, device="cuda").bfloat16()
            a = layer(pool[i], table, _i32(now), _i32(cu), qkv, norms[i])
            b = layer(own[i], own_table, _i32(now), _i32(cu), qkv, norms[i])
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
            assert a["out"].isfinite().all()
        return now

    counts = [r.randint(1, 3 * P) for _ in range(B)]
    got = mhc.kv_fork(pool, torch.empty(0, width, dtype=torch.int32, device="cuda"), _i32([]), _i32([-1] * B),
                      room=_i32(counts), held=held, window=window, sinks=sinks)
    lens, table = step(got["block_table"], [0] * B, counts), got["block_table"]
    for i in range(40):
        parents = [r.choice([b, b, b, r.randrange(B), -1]) for b in range(B)]
        counts = [r.choice([1, 1, 3]) if p >= 0 else r.randint(1, 2 * P) for p in parents]
        got = mhc.kv_fork(pool, table, _i32(lens), _i32(parents), room=_i32(counts), held=held, window=window, sinks=sinks)
        table, before = got["block_table"], lens
        lens = [before[p] if p >= 0 else 0 for p in parents]
        assert got["seq_lens"].tolist() == lens
        follow = torch.tensor([max(p, 0) for p in parents], device="cuda")
        for c in own:
            for n in ("k", "v"):
                x, s = c[n].view(torch.uint8), c[n + "_scale"]
                x.copy_(x.view(B, width, H, P, D)[follow].reshape(x.shape))
                s.copy_(s.view(B, width, H)[follow].reshape(s.shape))
        lens = step(table, lens, counts)
        if i % 7 == 3:
            got = mhc.kv_compact(pool, table, _i32(lens), held=held)
            table = got["block_table"]
            used = {x for row, n in zip(table.tolist(), lens) for x in row[:-(-n // P)] if x >= 0}
            assert got["pages"].item() == 1 + max(used | {3, 50}) and not used & {3, 50}
        assert max(lens) + 3 <= width * P
