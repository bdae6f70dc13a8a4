"""Host-only checks of the paged cache's further calls: what the C entry
points refuse (no call here gets as far as a launch), and the index arithmetic
of windows and pages compiled for the host."""
import ctypes
import math
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from mhc_hyper_connection_pre_gb300 import build as mbuild
from mhc_hyper_connection_pre_gb300 import kv as kvmod

OK, INVALID, UNSUPPORTED, CUDA_ERR = 0, 1, 2, 3
HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 0x10000000000     # never dereferenced
ROW = (40 + 16) * 128
QKV = FAKE + (4 << 32)
NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(), reason="a well-formed call would be launched")


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mhc.load_library()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE + (1 << 32), k_scale=FAKE + (2 << 32), v_scale=FAKE + (3 << 32), num_pages=100, heads=8,
             page_tokens=64, head_dim=128)
    a.update(kw)
    return kvmod._Cache(*a.values())


# -------------------------------------------------------------------- norms ---

def _append_norm(lib, cache=None, **kw):
    a = dict(k=QKV + 40 * 256, k_stride=ROW, v=QKV + 48 * 256, v_stride=ROW, q=QKV, q_stride=ROW, q_heads=40,
             q_out=FAKE + (5 << 32), q_out_stride=40 * 128, q_norm=FAKE + (12 << 32), q_norm_stride=0,
             k_norm=FAKE + (13 << 32), k_norm_stride=128, eps=1e-6, cos=FAKE + (6 << 32), sin=FAKE + (7 << 32),
             rope_rows=1000, rotary_dim=128, interleaved=0, table=FAKE + (8 << 32), width=10, lens=FAKE + (9 << 32),
             cu=None, B=16, T=16, stream=None)
    a.update(kw)
    return lib.mhc_kv_append_norm(cache if cache is not None else _cache(), *a.values())


NORMS = [
    (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=1e-21), INVALID), (dict(eps=math.inf), INVALID),
    (dict(eps=math.nan), INVALID), (dict(q_norm=FAKE + (12 << 32) + 8), INVALID),
    (dict(k_norm=FAKE + (13 << 32) + 2), INVALID), (dict(q_norm_stride=120), INVALID),
    (dict(k_norm_stride=132), INVALID), (dict(k_norm_stride=-128), INVALID), (dict(k_norm_stride=1 << 31), INVALID),
    (dict(q=None, q_out=None), INVALID),                           # q_norm without q
    (dict(q_norm=FAKE + (5 << 32)), INVALID),                      # weights that the call writes over
    (dict(k_norm=FAKE + (2 << 32)), INVALID), (dict(k_norm=FAKE + 4096), INVALID),
    (dict(q_norm=FAKE + (5 << 32) - 39 * 256, q_norm_stride=128), INVALID),    # the last head's
    (dict(k=None), INVALID), (dict(T=17), INVALID), (dict(rotary_dim=24), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(T=0, B=0, k=None, q=None, q_out=None, q_norm=None, cu=FAKE), OK),
]


@pytest.mark.parametrize("case", range(len(NORMS)))
def test_append_norm_refuses(lib, case):
    kw, status = NORMS[case]
    assert _append_norm(lib, **kw) == status


@NO_DEVICE
def test_append_norm_passes_the_checks(lib):
    """With no device in the process well-formed calls end as MHC_ERR_CUDA."""
    assert _append_norm(lib) == CUDA_ERR
    assert _append_norm(lib, q_norm=None) == CUDA_ERR
    assert _append_norm(lib, k_norm=None) == CUDA_ERR
    assert _append_norm(lib, q=None, q_out=None, q_norm=None) == CUDA_ERR
    assert _append_norm(lib, q_norm=None, k_norm=None, eps=0.0) == CUDA_ERR       # no norm: eps is not read
    assert _append_norm(lib, q_norm=FAKE + (5 << 32) - 40 * 256, q_norm_stride=128) == CUDA_ERR      # just before q_out


@pytest.mark.parametrize("call", ["k", "v"])
def test_queries_in_place_are_not_keys_or_values_too(lib, call):
    """q_out may be q, but then no other input may lie there."""
    assert _append_norm(lib, q_out=QKV, q_out_stride=ROW, q_norm=None, k_norm=None, **{call: QKV}) == INVALID


# ------------------------------------------------------------------ windows ---

def _attend_window(lib, cache=None, **kw):
    a = dict(q=QKV, q_stride=ROW, q_heads=40, table=FAKE + (8 << 32), width=10, lens=FAKE + (9 << 32), cu=None, B=16,
             T=16, scale=0.1, window=100, sinks=4, out=FAKE + (5 << 32), lse=FAKE + (6 << 32), ws=FAKE + (10 << 32),
             ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.mhc_kv_attend_window(cache if cache is not None else _cache(), *a.values())


WINDOWS = [
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(window=-(1 << 63)), INVALID),
    (dict(q_heads=41), INVALID), (dict(scale=-1.0), INVALID), (dict(out=QKV + 256), INVALID), (dict(T=17), INVALID),
    (dict(table=None), INVALID), (dict(lens=FAKE + (9 << 32) + 2), INVALID), (dict(q_heads=8 * 129, q_stride=1 << 20), UNSUPPORTED),
    (dict(T=0, B=0, q=None, out=None, cu=FAKE), OK), (dict(T=0, B=0, q=None, out=None, cu=FAKE, window=0), INVALID),
]


@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_attend_window_refuses(lib, case):
    kw, status = WINDOWS[case]
    assert _attend_window(lib, **kw) == status


@NO_DEVICE
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (640, 0), (1 << 62, 1 << 62), (1, 1 << 62)])
def test_attend_window_passes_the_checks(lib, window, sinks):
    assert _attend_window(lib, window=window, sinks=sinks) == CUDA_ERR


def test_binding_refuses_windows(lib):
    cache = mhc.kv_cache(3, 2, 16, 64, device="cpu")
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):                                # not on a CUDA device
        mhc.kv_attend(x, cache, table, lens, window=4)


@pytest.fixture(scope="module")
def window_shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv") / "libkvwindow.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-shared",
                    "-fPIC", "-x", "c++", os.path.join(HERE, "kv_window_shim.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.kv_window_walk.restype = ctypes.c_int64
    return lib


def _ptr(x):
    return None if x is None else x.ctypes.data_as(ctypes.c_void_p)


def _walk(shim, lens, counts, log2, heads, group, tile_log2, unit_log2, extra, window, sinks, n):
    B, width = len(lens), max(1, (max(lens) + (1 << log2) - 1) >> log2)
    cu = np.cumsum([0] + counts).astype(np.int32)
    T, cap = int(cu[-1]), width << log2
    seen = np.zeros((T * heads * group, cap), np.uint8)
    looked, total, longest = np.zeros((B, width), np.uint8), ctypes.c_int64(0), ctypes.c_int32(0)
    lens_a = np.array(lens, np.int32)
    wrong = shim.kv_window_walk(_ptr(lens_a), _ptr(cu), width, B, T, log2, heads, group, tile_log2, unit_log2, extra, window,
                                sinks, n, _ptr(seen), _ptr(looked), ctypes.byref(total), ctypes.byref(longest))
    return wrong, seen.reshape(T, heads * group, cap), looked, total.value, cu


@pytest.mark.parametrize("seed", range(60))
def test_every_row_meets_the_keys_that_it_sees_once(window_shim, seed):
    """Over all shares a row meets each key of its window and of the first
    ones once and no other, and the pages that are looked at are those of
    which some new token sees a key."""
    r = random.Random(seed)
    log2, B = r.choice([4, 5, 6, 7]), r.randint(1, 5)
    heads, group = r.choice([1, 2]), r.choice([1, 1, 2, 3, 5])
    tile_log2, unit_log2 = r.choice([(3, 5), (4, 5), (8, 7), (8, 30)])
    counts = [r.choice([0, 1, 1, r.randint(0, 20), r.randint(0, 300 // group)]) for _ in range(B)]
    lens = [r.choice([0, n, max(0, n - 2), n + r.randint(0, 900)]) for n in counts]
    if not any(counts):
        counts[0] = 1
    window, sinks = r.choice([1, 2, 17, 64, 128, r.randint(1, 700)]), r.choice([0, 0, 1, 4, 31, 32, 33, 130, r.randint(0, 500)])
    wrong, seen, looked, total, cu = _walk(window_shim, lens, counts, log2, heads, group, tile_log2, unit_log2,
                                           0 if unit_log2 == 30 else r.choice([0, 3, 4]), window, sinks, r.choice([1, 7, 152, 500]))
    assert wrong == 0
    for b, n in enumerate(counts):
        pages = set()
        for i in range(n):
            p = lens[b] - n + i
            want = np.zeros(seen.shape[2], np.uint8)
            for j in range(max(0, p + 1)):
                if j > p - window or j < sinks:
                    want[j] = 1
                    pages.add(j >> log2)
            assert (seen[cu[b] + i] == want).all(), (b, i, p)
        assert set(np.flatnonzero(looked[b]).tolist()) == pages


def test_a_window_bounds_the_work(window_shim):
    """Units follow the window, not the sequence: 100 tokens, then one, of a sequence of 100,000."""
    args = (7, 1, 1, 8, 7, 0)
    assert _walk(window_shim, [100000], [1], *args, 1, 0, 1)[3] == 1
    assert _walk(window_shim, [100000], [1], *args, 256, 4, 1)[3] <= 4
    assert _walk(window_shim, [20000], [100], *args, 512, 130, 1)[3] <= 2 + 6


def test_largest_windows_and_positions(window_shim):
    """Windows, first keys and lengths up to 2^30 stay in range (the sanitizer ends a walk that does not)."""
    lens, cu = np.array([1 << 30], np.int32), np.array([0, 1], np.int32)
    one = np.zeros(1, np.uint8)
    total, longest = ctypes.c_int64(0), ctypes.c_int32(0)
    for window, sinks in ((1 << 30, 1 << 30), (1, 1 << 30), (1 << 30, 0)):
        window_shim.kv_window_walk(_ptr(lens), _ptr(cu), 1 << 23, 1, 1, 7, 1, 1, 8, 7, 4, window, sinks, 0, _ptr(one),
                                   _ptr(one), ctypes.byref(total), ctypes.byref(longest))
        assert total.value == (1 << 23) + 4


# -------------------------------------------------------------------- pages ---

def plan_fork(table, lens, pages, log2, parents, room, window, sinks, held):
    """mhc_kv_fork's definition: (table, lens, copies, status), one place and entry after the other."""
    P, width, cap = 1 << log2, len(table[0]) if table else 0, (len(table[0]) if table else 0) << log2
    status = 0

    def page(x):
        nonlocal status
        if 0 <= x < pages:
            return x
        status |= 2 if x != -1 else 0
        return -1
    B = len(lens) if parents is None else len(parents)
    out, n, source = [[-1] * width for _ in range(B)], [], []
    for b in range(B):
        a = b if parents is None else parents[b]
        if not -1 <= a < len(lens):
            status, a = status | 2, -1
        m = lens[a] if a >= 0 else 0
        if not 0 <= m <= cap:
            status, m = status | 2, min(max(m, 0), cap)
        n.append(m)
        source.append(a)
    for b in range(B):
        for i in range(n[b] >> log2):
            if window == 0 or i * P < sinks or (i + 1) * P > n[b] - window + 1:
                out[b][i] = page(table[source[b]][i])
    shared = {x for row in out for x in row if x >= 0} | {x for x in range(pages) if held and held[x]}
    keep, asks = set(), []
    for b in range(B):
        last = page(table[source[b]][n[b] >> log2]) if n[b] % P else -1
        if last >= 0:
            if last in shared or last in keep:
                asks.append((b, n[b] >> log2, last))
            else:
                keep.add(last)
                out[b][n[b] >> log2] = last
        more = room[b] if isinstance(room, list) else room
        if more < 0 or n[b] + more > cap:
            status, more = status | 2, min(max(more, 0), cap - n[b])
        asks += [(b, i, -1) for i in range(-(-n[b] // P), -(-(n[b] + more) // P))]
    free = [x for x in range(pages) if x not in shared and x not in keep]
    copies = []
    for k, (b, i, last) in enumerate(asks):
        out[b][i] = free[k] if k < len(free) else -1
        if last >= 0:
            copies.append((last, out[b][i], n[b] % P))
    return out, n, copies, status | (4 if len(asks) > len(free) else 0)


def plan_compact(table, lens, pages, log2, held):
    """mhc_kv_compact's definition: (table, pages, copies, status)."""
    width = len(table[0]) if table else 0
    cap, status = width << log2, 0
    out, used = [[-1] * width for _ in lens], set()
    for b, m in enumerate(lens):
        if not 0 <= m <= cap:
            status, m = status | 2, min(max(m, 0), cap)
        for i in range(-(-m >> log2) if m % (1 << log2) == 0 else (m >> log2) + 1):
            x = table[b][i]
            if 0 <= x < pages:
                out[b][i] = x
                used.add(x)
            elif x != -1:
                status |= 2
    stay = {x for x in range(pages) if held and held[x]}
    loose = sorted(used - stay)
    goal = [x for x in range(pages) if x not in stay][:len(loose)]
    moves = dict(zip([x for x in loose if x not in set(goal)], [x for x in goal if x not in used]))
    out = [[moves.get(x, x) for x in row] for row in out]
    return out, 1 + max([-1, *goal, *stay]), [(a, b, 1 << log2) for a, b in moves.items()], status


@pytest.fixture(scope="module")
def pages_exe(tmp_path_factory):
    """The planning with the address and with the thread sanitizer."""
    at = tmp_path_factory.mktemp("pages")
    for kind in ("address,undefined", "thread"):
        subprocess.run(["g++", "-O1", "-g", "-std=c++17", f"-fsanitize={kind}", "-fno-sanitize-recover=all",
                        os.path.join(HERE, "kv_pages_shim.cpp"), "-o", str(at / kind[:6]), "-pthread"], check=True)
    return at


def _flat(x):
    return [v for row in x for v in (row if isinstance(row, (list, tuple)) else [row])]


def _planned(exe, cases):
    """Runs cases (their numbers) through an executable; the lines of numbers that it writes."""
    text = "\n".join(" ".join(str(int(v)) for v in c) for c in cases)
    r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    lines = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
    assert len(lines) == len(cases)
    return lines


def _tables(r, wild):
    """A batch as a few steps leave it: pages shared from the front, part-filled ones too, some let go."""
    log2, B, width = r.choice([4, 4, 5, 7]), r.choice([1, 1, 2, 5, 17, 40]), r.choice([1, 2, 5, 9, 40])
    P, pages = 1 << log2, r.choice([1, 31, 32, 33, 64, 100, 500])
    lens = [r.choice([0, r.randint(0, width * P), r.randint(0, width * P), width * P, P]) for _ in range(B)]
    lens = [min(n, width * P) for n in lens]
    table = [[r.randrange(pages) for _ in range(width)] for _ in range(B)]
    for b in range(1, B):
        if r.random() < 0.4:                                     # shares its front with another
            a, k = r.randrange(b), r.randint(0, width)
            table[b][:k] = table[a][:k]
            if r.random() < 0.5:
                lens[b] = lens[a]
    for row in table:
        for i in range(width):
            if r.random() < 0.1:
                row[i] = -1
            if wild and r.random() < 0.1:
                row[i] = r.choice([pages, -2, 2147483647, -2147483648])
    if wild:
        lens = [r.choice([n, n, n, -1, width * P + 1, 2147483647, -2147483648]) for n in lens]
    held = [r.choice([0, 0, 0, 1, 255]) for _ in range(pages)] if r.random() < 0.5 else None
    return log2, P, pages, width, lens, table, held


def _fork_case(r, size, wild):
    log2, P, pages, width, lens, table, held = _tables(r, wild)
    B_in, parents = len(lens), None
    if r.random() < 0.7:
        parents = [r.randint(-1, B_in - 1) for _ in range(r.choice([1, B_in, 3 * B_in]))]
        if wild:
            parents = [r.choice([p, p, B_in, -2, 2147483647, -2147483648]) for p in parents]
    B = B_in if parents is None else len(parents)
    room = r.choice([0, 1, r.randint(0, 3 * P), None])
    if room is None:
        room = [r.choice([0, 1, r.randint(0, 2 * P)]) for _ in range(B)]
        if wild:
            room = [r.choice([x, -1, 2147483647, -2147483648]) for x in room]
    window = r.choice([0, 0, 1, r.randint(1, width * P)])
    sinks = r.choice([0, r.randint(0, 3 * P)]) if window else 0
    in_place = parents is None and r.random() < 0.5
    numbers = [0, size, width, B_in, B, log2, pages, in_place, held is not None, r.random() < 0.5, *_flat(table), *lens, *(held or []),
               parents is not None, isinstance(room, list), *(parents or []), *(room if isinstance(room, list) else []),
               0 if isinstance(room, list) else room, window, sinks]
    out, n, copies, status = plan_fork(table, lens, pages, log2, parents, room, window, sinks, held)
    return numbers, [*n, *_flat(out), status, len(copies), *_flat(copies)]


def _compact_case(r, size, wild):
    log2, P, pages, width, lens, table, held = _tables(r, wild)
    B = len(lens)
    numbers = [1, size, width, B, B, log2, pages, r.random() < 0.5, held is not None, r.random() < 0.5,
               *_flat(table), *lens, *(held or [])]
    out, top, copies, status = plan_compact(table, lens, pages, log2, held)
    return numbers, [top, *_flat(out), status, len(copies), *_flat(copies)]


@pytest.mark.parametrize("make", [_fork_case, _compact_case])
@pytest.mark.parametrize("wild", [False, True])
def test_pages_are_planned_as_defined(pages_exe, make, wild):
    """One to 64 threads, the rows with the rest or apart: the definition's tables, lengths, copies and reports, whatever the arrays hold, inside
    the arrays (a sanitizer ends the program otherwise)."""
    r = random.Random(7 + wild)
    cases = [make(r, r.choice([1, 2, 8, 64]), wild) for _ in range(250)]
    got = _planned(pages_exe / "addres", [c for c, _ in cases])
    for (_, want), line in zip(cases, got):
        if line != want:
            at = next(i for i, (x, y) in enumerate(zip(line, want)) if x != y)
            raise AssertionError((at, line[at:at + 9], want[at:at + 9]))


@pytest.mark.parametrize("make", [_fork_case, _compact_case])
def test_pages_are_planned_without_races(pages_exe, make):
    r = random.Random(11)
    cases = [make(r, r.choice([2, 4, 16]), r.random() < 0.3) for _ in range(60)]
    got = _planned(pages_exe / "thread", [c for c, _ in cases])
    assert got == [want for _, want in cases]


TABLE, LENS, OUT, OUT_LENS = (FAKE + (i << 32) for i in (20, 21, 22, 23))


def _layers(n=2, **kw):
    at = lambda i: {k: FAKE + ((30 + 4 * i + j) << 32) for j, k in enumerate(("k", "v", "k_scale", "v_scale"))}  # noqa: E731
    return (kvmod._Cache * n)(*[_cache(**{**at(i), **(kw if i == n - 1 else {})}) for i in range(n)])


def _fork(lib, caches=None, **kw):
    a = dict(num=2, table=TABLE, width=10, lens=LENS, B_in=16, parents=FAKE + (24 << 32), B=20, room=FAKE + (25 << 32),
             room_all=0, held=FAKE + (26 << 32), window=0, sinks=0, out=OUT, out_lens=OUT_LENS, ws=FAKE + (27 << 32),
             ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.mhc_kv_fork(caches if caches is not None else _layers(), *a.values())


def _compact(lib, caches=None, **kw):
    a = dict(num=2, table=TABLE, width=10, lens=LENS, B=16, held=FAKE + (26 << 32), out=OUT, pages=OUT_LENS,
             ws=FAKE + (27 << 32), ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.mhc_kv_compact(caches if caches is not None else _layers(), *a.values())


PAGES = [
    (dict(num=0), {}, INVALID), (dict(num=513), {}, UNSUPPORTED), (dict(width=0), {}, INVALID), (dict(B=-1), {}, INVALID),
    (dict(table=None), {}, INVALID), (dict(lens=None), {}, INVALID), (dict(table=TABLE + 2), {}, INVALID),
    (dict(lens=LENS + 1), {}, INVALID), (dict(held=FAKE + (26 << 32) + 1), {}, INVALID), (dict(out=None), {}, INVALID),
    (dict(out=OUT + 2), {}, INVALID), (dict(ws=None), {}, INVALID), (dict(ws=FAKE + (27 << 32) + 128), {}, INVALID),
    (dict(ws_bytes=256), {}, INVALID), (dict(width=1 << 26, B=16), {}, UNSUPPORTED),
    ({}, dict(num_pages=101), INVALID), ({}, dict(page_tokens=32), INVALID), ({}, dict(page_tokens=8), UNSUPPORTED),
    ({}, dict(head_dim=96), UNSUPPORTED), ({}, dict(heads=0), INVALID), ({}, dict(k=None), INVALID),
    ({}, dict(v=FAKE + (40 << 32) + 8), INVALID), ({}, dict(v_scale=FAKE + (41 << 32) + 2), INVALID),
    ({}, dict(k=FAKE + (31 << 32) + 16), INVALID),                 # in the first cache's values
    ({}, dict(k_scale=FAKE + (32 << 32)), INVALID),                # the first cache's scales
    (dict(out=TABLE + 4), {}, INVALID), (dict(out=LENS), {}, INVALID), (dict(out=FAKE + (30 << 32) + 64), {}, INVALID),
    (dict(ws=OUT), {}, INVALID), (dict(held=OUT), {}, INVALID), (dict(lens=FAKE + (27 << 32)), {}, INVALID),
    (dict(lens=FAKE + (32 << 32) + 100), {}, INVALID),
]


@pytest.mark.parametrize("call", [_fork, _compact])
@pytest.mark.parametrize("case", range(len(PAGES)))
def test_calls_on_pages_refuse(lib, call, case):
    kw, c, status = PAGES[case]
    assert call(lib, _layers(**c), **kw) == status


def test_fork_and_compact_refuse(lib):
    assert _fork(lib, parents=None) == INVALID                     # 16 places become 20 of their own
    assert _fork(lib, room_all=-1) == INVALID
    assert _fork(lib, window=-1) == INVALID
    assert _fork(lib, sinks=-1, window=2) == INVALID
    assert _fork(lib, sinks=1) == INVALID
    assert _fork(lib, B_in=-1) == INVALID
    assert _fork(lib, out_lens=None) == INVALID
    assert _fork(lib, out_lens=OUT) == INVALID
    assert _fork(lib, parents=FAKE + (24 << 32) + 2) == INVALID
    assert _fork(lib, room=FAKE + (25 << 32) + 2) == INVALID
    assert _fork(lib, out=TABLE) == INVALID                        # in place, with parents
    assert _fork(lib, out_lens=LENS) == INVALID
    assert _fork(lib, out_lens=FAKE + (24 << 32)) == INVALID
    assert _compact(lib, pages=None) == INVALID
    assert _compact(lib, pages=OUT_LENS + 2) == INVALID
    assert _compact(lib, pages=OUT + 4) == INVALID
    assert _compact(lib, pages=LENS + 4) == INVALID
    assert lib.mhc_kv_fork(None, *[0] * 18) == INVALID and lib.mhc_kv_compact(None, *[0] * 11) == INVALID
    assert _fork(lib, B_in=0, B=0, parents=None) == OK
    for f, sizes in ((lib.mhc_kv_fork_workspace_bytes, [(0, 1, 1), (1, 0, 1), (1, 1, -1), ((1 << 30) + 1, 1, 1), (1, 1 << 29, 2)]),
                     (lib.mhc_kv_compact_workspace_bytes, [(0, 1), (-1, 1), ((1 << 30) + 1, 1), (1, -1)])):
        assert all(f(*s) == 0 for s in sizes)
    assert lib.mhc_kv_fork_workspace_bytes(1000, 10, 20) > 4 * 1000 and lib.mhc_kv_compact_workspace_bytes(1000, 9) > 24 * 1000


@NO_DEVICE
def test_calls_on_pages_pass_the_checks(lib):
    assert _fork(lib) == CUDA_ERR
    assert _fork(lib, window=100, sinks=4, held=None, room=None, room_all=1 << 40) == CUDA_ERR
    assert _fork(lib, B_in=0, table=None, lens=None) == CUDA_ERR                   # a first batch
    assert _fork(lib, parents=None, B=16, out=TABLE, out_lens=LENS) == CUDA_ERR    # in place
    assert _fork(lib, _layers(1), num=1) == CUDA_ERR
    assert _fork(lib, _layers(heads=2, head_dim=64)) == CUDA_ERR                   # layers of different heads
    assert _compact(lib) == CUDA_ERR
    assert _compact(lib, out=TABLE) == CUDA_ERR
    assert _compact(lib, B=0, table=None, lens=None, out=None) == CUDA_ERR
    assert _fork(lib, ws_bytes=lib.mhc_kv_fork_workspace_bytes(100, 10, 20)) == CUDA_ERR
    assert _compact(lib, ws_bytes=lib.mhc_kv_compact_workspace_bytes(100, 16)) == CUDA_ERR
    assert _fork(lib, ws_bytes=lib.mhc_kv_fork_workspace_bytes(100, 10, 20) - 1) == INVALID


def test_status_string_of_pages_that_ran_out(lib):
    assert lib.mhc_status_string(6).decode().startswith("MHC_ERR_PAGES")
