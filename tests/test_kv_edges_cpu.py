"""Host-only checks of calls of the paged cache at their edges."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from test_kv_more_cpu import (CUDA_ERR, FAKE, HERE, INVALID, NO_DEVICE, OK, _append_norm, _flat, _fork, _planned, _ptr, lib,  # noqa: F401
                              plan_compact, plan_fork)             # (lib is a fixture)


def test_a_batch_that_has_ended(lib):
    """No places go on: an array of no parents is a null pointer, which is not "every place goes on with itself"."""
    assert _fork(lib, B=0, parents=None) == OK                     # 16 places before
    assert _fork(lib, B=0, parents=None, room=None, out=None, out_lens=None) == OK
    assert _fork(lib, B=0) == OK
    assert _fork(lib, B=0, parents=None, room_all=-1) == INVALID
    assert _fork(lib, B=1, parents=None) == INVALID


@NO_DEVICE
def test_batches_that_go_on_pass_the_checks(lib):
    assert _fork(lib, B=16, parents=None) == CUDA_ERR
    assert _fork(lib, B=1) == CUDA_ERR


def test_norms_of_no_tokens(lib):
    """A step without new tokens: its queries' array may be a null pointer, with norms as without."""
    for q_norm in (None, FAKE + (12 << 32)):
        assert _append_norm(lib, T=0, B=0, k=None, v=None, q=None, q_out=None, q_norm=q_norm) == OK
        assert _append_norm(lib, T=0, B=3, cu=FAKE, k=None, v=None, q=None, q_out=None, q_norm=q_norm) == OK
    assert _append_norm(lib, q=None, q_out=None) == INVALID        # keys alone have no queries to norm


@pytest.fixture(scope="module")
def rows_exe(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("rows") / "rows")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=thread", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "kv_rows_shim.cpp"), "-o", exe, "-pthread"], check=True)
    return exe


@pytest.mark.parametrize("make", ["fork", "compact"])
def test_rows_in_place_by_any_number_of_threads(rows_exe, make):
    """As many threads as a grid has, which is no power of two and no multiple of a wide row's threads: each
    entry is one thread's alone (the thread sanitizer ends the program otherwise), and the definition's."""
    r, cases = random.Random(17), []
    for size in (3, 5, 6, 11, 12, 20, 24, 44):
        for width in (1, 9, 40, 150):
            log2, B = 4, r.choice([1, 2, 5, 9, 13])
            pages = B * width + 7
            order = r.sample(range(pages), B * width)
            table = [[x if r.random() < 0.9 else -1 for x in order[b * width:(b + 1) * width]] for b in range(B)]
            lens = [r.choice([0, width << log2, r.randint(0, width << log2)]) for _ in range(B)]
            head = [0 if make == "fork" else 1, size, width, B, log2, pages, *_flat(table), *lens]
            if make == "fork":
                room, window = r.choice([0, 1, 30]), r.choice([0, 1, 100])
                sinks = r.choice([0, 20]) if window else 0
                out, n, copies, status = plan_fork(table, lens, pages, log2, None, room, window, sinks, None)
                cases.append((head + [room, window, sinks], [*n, *_flat(out), status, len(copies), *_flat(copies)]))
            else:
                out, top, copies, status = plan_compact(table, lens, pages, log2, None)
                cases.append((head, [top, *_flat(out), status, len(copies), *_flat(copies)]))
    got = _planned(rows_exe, [c for c, _ in cases])
    assert got == [want for _, want in cases]


@pytest.fixture(scope="module")
def ends_shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ends") / "libkvends.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-shared",
                    "-fPIC", "-x", "c++", os.path.join(HERE, "kv_ends_shim.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.kv_window_ends.restype = ctypes.c_int64
    return lib


@pytest.mark.parametrize("seed", range(80))
def test_ends_of_windows_are_short(ends_shim, seed):
    """The keys that not every row of a tile sees lie in two stretches, neither longer than its tokens and two loads of
    128, whatever the window: what is done again for a value that is NaN does not grow with it."""
    r = random.Random(seed)
    log2, B, group = r.choice([4, 5, 6, 7]), r.randint(1, 3), r.choice([1, 1, 2, 3, 5, 40])
    counts = [r.choice([1, r.randint(1, 20), r.randint(1, 700 // group)]) for _ in range(B)]
    lens = [r.choice([0, n, max(0, n - 2), n + r.randint(0, 9000)]) for n in counts]
    window, sinks = r.choice([1, 17, 128, 300, r.randint(1, 7000)]), r.choice([0, 1, 4, 127, 128, 129, r.randint(0, 5000)])
    width, cu = max(1, (max(lens) + (1 << log2) - 1) >> log2), np.cumsum([0] + counts).astype(np.int32)
    longest, segments = ctypes.c_int32(0), ctypes.c_int32(0)
    unit, extra, shares = r.choice([(7, 4, 152), (7, 3, 7), (30, 0, 152), (30, 0, 1)])
    wrong = ends_shim.kv_window_ends(_ptr(np.array(lens, np.int32)), _ptr(cu), width, B, int(cu[-1]), log2, r.choice([1, 2]), group,
                                     unit, extra, window, sinks, shares, ctypes.byref(longest), ctypes.byref(segments))
    assert wrong == 0 and segments.value > 0
    assert longest.value <= -(-256 // group) + 1 + 256
