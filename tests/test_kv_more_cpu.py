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
    tile_log2, unit_log2 = r.choice([(3, 5), (4, 5), (8, 7)])
    counts = [r.choice([0, 1, 1, r.randint(0, 20), r.randint(0, 300 // group)]) for _ in range(B)]
    lens = [r.choice([0, n, max(0, n - 2), n + r.randint(0, 900)]) for n in counts]
    if not any(counts):
        counts[0] = 1
    window, sinks = r.choice([1, 2, 17, 64, 128, r.randint(1, 700)]), r.choice([0, 0, 1, 4, 31, 32, 33, 130, r.randint(0, 500)])
    wrong, seen, looked, total, cu = _walk(window_shim, lens, counts, log2, heads, group, tile_log2, unit_log2,
                                           r.choice([0, 3, 4]), window, sinks, r.choice([1, 7, 152, 500]))
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
