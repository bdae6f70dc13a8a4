"""Host-only checks of the paged key/value cache: argument checks of the C
entry points (no call here gets as far as a launch), the binding's refusals,
and the kernels' index arithmetic compiled for the host."""
import ctypes
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


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mhc.load_library()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE + (1 << 32), k_scale=FAKE + (2 << 32), v_scale=FAKE + (3 << 32), num_pages=100, heads=8,
             page_tokens=64, head_dim=128)
    a.update(kw)
    return kvmod._Cache(*a.values())


ROW = (40 + 16) * 128
QKV = FAKE + (4 << 32)


def _append(lib, cache=None, **kw):
    a = dict(k=QKV + 40 * 256, k_stride=ROW, v=QKV + 48 * 256, v_stride=ROW, q=QKV, q_stride=ROW, q_heads=40,
             q_out=FAKE + (5 << 32), q_out_stride=40 * 128, cos=FAKE + (6 << 32), sin=FAKE + (7 << 32), rope_rows=1000,
             rotary_dim=128, interleaved=0, table=FAKE + (8 << 32), width=10, lens=FAKE + (9 << 32), cu=None, B=16,
             T=16, stream=None)
    a.update(kw)
    return lib.mhc_kv_append(cache if cache is not None else _cache(), *a.values())


def _attend(lib, cache=None, **kw):
    a = dict(q=QKV, q_stride=ROW, q_heads=40, table=FAKE + (8 << 32), width=10, lens=FAKE + (9 << 32), cu=None, B=16,
             T=16, scale=0.1, out=FAKE + (5 << 32), lse=FAKE + (6 << 32), ws=FAKE + (10 << 32), ws_bytes=1 << 30,
             stream=None)
    a.update(kw)
    return lib.mhc_kv_attend(cache if cache is not None else _cache(), *a.values())


COMMON = [
    (dict(T=-1), {}, INVALID), (dict(B=-1), {}, INVALID), (dict(width=0), {}, INVALID),
    (dict(T=17), {}, INVALID),                                      # no cu_q: one token each
    (dict(B=0, cu=FAKE + (11 << 32)), {}, INVALID),
    ({}, dict(heads=0), INVALID), ({}, dict(num_pages=0), INVALID), ({}, dict(head_dim=96), UNSUPPORTED),
    ({}, dict(head_dim=256), UNSUPPORTED), ({}, dict(page_tokens=48), UNSUPPORTED),
    ({}, dict(page_tokens=8), UNSUPPORTED), ({}, dict(num_pages=1 << 30), UNSUPPORTED),
    (dict(width=1 << 26), {}, UNSUPPORTED), (dict(T=1 << 31, B=1 << 31), {}, UNSUPPORTED),
    ({}, dict(k=None), INVALID), ({}, dict(v=FAKE + (1 << 32) + 8), INVALID), ({}, dict(k_scale=None), INVALID),
    ({}, dict(v_scale=FAKE + (3 << 32) + 2), INVALID), (dict(table=None), {}, INVALID), (dict(lens=None), {}, INVALID),
    (dict(cu=FAKE + (11 << 32) + 2), {}, INVALID), (dict(q=QKV + 2), {}, INVALID), (dict(q_stride=ROW + 4), {}, INVALID),
    (dict(q_stride=40 * 128 - 8), {}, INVALID),
]


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("case", range(len(COMMON)))
def test_both_calls_refuse(lib, call, case):
    kw, c, status = COMMON[case]
    assert call(lib, _cache(**c), **kw) == status


def test_append_refuses(lib):
    assert _append(lib, k=None) == INVALID
    assert _append(lib, v=QKV + 48 * 256 + 4) == INVALID
    assert _append(lib, k_stride=8) == INVALID
    assert _append(lib, q=None) == INVALID                         # q_out without q
    assert _append(lib, q_out=None) == INVALID
    assert _append(lib, q_heads=0) == INVALID
    assert _append(lib, cos=None) == INVALID
    assert _append(lib, sin=FAKE + (7 << 32) + 4) == INVALID
    assert _append(lib, rotary_dim=-16) == INVALID
    assert _append(lib, rotary_dim=24) == UNSUPPORTED
    assert _append(lib, rotary_dim=144) == UNSUPPORTED
    assert _append(lib, q_out=QKV + 40 * 256, q_out_stride=ROW) == INVALID       # onto k's columns
    assert _append(lib, q_out=QKV + 256, q_out_stride=ROW) == INVALID            # q shifted by a head
    assert _append(lib, q_out=QKV, q_out_stride=40 * 128) == INVALID             # q's place, another stride
    assert _append(lib, q_out=FAKE + 256) == INVALID                             # inside the cache
    assert _append(lib, _cache(v=FAKE + 64)) == INVALID                          # k and v overlap
    assert _append(lib, _cache(k_scale=FAKE + 64)) == INVALID
    assert _append(lib, k=FAKE + 128) == INVALID                                 # reads the cache it writes
    assert _append(lib, T=0, B=0, k=None, q=None, q_out=None, cu=FAKE) == OK


def test_attend_refuses(lib):
    assert _attend(lib, q_heads=41) == INVALID
    assert _attend(lib, q_heads=0) == INVALID
    assert _attend(lib, _cache(heads=1), q_heads=129, q_stride=129 * 128) == UNSUPPORTED
    assert _attend(lib, scale=-1.0) == INVALID
    assert _attend(lib, scale=float("nan")) == INVALID
    assert _attend(lib, scale=float("inf")) == INVALID
    assert _attend(lib, out=None) == INVALID
    assert _attend(lib, out=QKV + 256) == INVALID
    assert _attend(lib, out=FAKE + 256) == INVALID
    assert _attend(lib, lse=FAKE + (5 << 32) + 64) == INVALID
    assert _attend(lib, lse=FAKE + (6 << 32) + 4) == INVALID
    assert _attend(lib, ws=FAKE + (5 << 32)) == INVALID
    assert _attend(lib, T=0, B=0, q=None, out=None, cu=FAKE) == OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="a well-formed call would be launched")
def test_well_formed_calls_pass_the_checks(lib):
    """With no device in the process they end as MHC_ERR_CUDA."""
    assert _append(lib) == CUDA_ERR
    assert _append(lib, q=None, q_out=None, cos=None, sin=None) == CUDA_ERR
    assert _append(lib, q_out=QKV, q_out_stride=ROW) == CUDA_ERR                  # in place
    assert _append(lib, q_out=QKV + ROW * 2 * 16, q_out_stride=ROW) == CUDA_ERR   # just behind
    assert _append(lib, T=40, cu=FAKE + (11 << 32)) == CUDA_ERR
    assert _attend(lib) == CUDA_ERR
    assert _attend(lib, lse=None) == CUDA_ERR
    c = _cache()
    assert lib.mhc_kv_attend_workspace_bytes(c, 40, 16, 16) == 0                  # sized on a device
    assert lib.mhc_kv_attend_workspace_bytes(c, 41, 16, 16) == 0


def test_status_string_of_a_bad_index(lib):
    assert lib.mhc_status_string(5).decode().startswith("MHC_ERR_INDEX")


def _cpu_cache(H=2, P=16, D=64, pages=3):
    return mhc.kv_cache(pages, H, P, D, device="cpu")


def test_binding_refuses(lib):
    c = _cpu_cache()
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):                                # not on a CUDA device
        mhc.kv_append(c, x, x, table, lens)
    with pytest.raises(ValueError):
        mhc.kv_attend(x, c, table, lens)
    with pytest.raises(ValueError):
        mhc.kv_attend(x, dict(c, v=c["v"][:2]), table, lens)
    with pytest.raises(ValueError):
        mhc.kv_attend(x, dict(c, k_scale=c["k_scale"][:2]), table, lens)
    with pytest.raises(TypeError):
        mhc.kv_attend(x, dict(c, v_scale=None), table, lens)
    with pytest.raises(TypeError):
        mhc.kv_append(dict(c, k=None), x, x, table, lens)


# ---------------------------------------------------------- index arithmetic ---

@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv") / "libkvshim.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-shared",
                    "-fPIC", "-x", "c++", os.path.join(HERE, "kv_index_shim.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def _i32(x):
    return np.ascontiguousarray(np.array(x, dtype=np.int32))


def _ptr(x):
    return None if x is None else x.ctypes.data_as(ctypes.c_void_p)


def _seq_of(cu, T, B):
    """The kernels' search: the last b with cu[b] <= t, for ascending cu."""
    return _i32([t if cu is None else max(b for b in range(B) if cu[b] <= t) for t in range(T)])


@pytest.mark.parametrize("seed", range(20))
def test_runs_cover_every_new_token_once(shim, seed):
    r = random.Random(seed)
    P, B = r.choice([16, 32, 64, 128]), r.randint(1, 9)
    counts = [r.choice([0, 1, 1, 2, r.randint(0, 300)]) for _ in range(B)]
    lens = [max(0, n + r.choice([0, r.randint(0, 200), -1])) for n in counts]
    width = max(1, -(-max(lens) // P))
    table = _i32([[100 * b + i for i in range(width)] for b in range(B)])
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    T = cu[-1]
    if T == 0:
        return
    seq = _seq_of(cu, T, B)
    out = np.zeros((T, 7), dtype=np.int32)
    lens_a, cu_a = _i32(lens), _i32(cu)
    shim.kv_runs(_ptr(table), _ptr(lens_a), _ptr(cu_a), width, B, T, P, 100 * B, _ptr(seq), _ptr(out))
    for window in (1, P):
        writer = [0] * T
        for w in range(0, T, window):
            t, end = w, min(T, w + window)
            while t < end:
                starts, pos, slot, n, nxt, page, bad = out[t]
                assert not bad and t < nxt <= T
                if starts:
                    b = seq[t]
                    assert page == 100 * b + pos // P and slot == pos % P and slot + n <= P
                    for i in range(n):
                        writer[t + i] += 1
                        assert lens[b] - (cu[b + 1] - (t + i)) == pos + i
                t = nxt
        for t in range(T):
            b = seq[t]
            assert writer[t] == (1 if lens[b] - (cu[b + 1] - t) >= 0 else 0)


@pytest.mark.parametrize("seed", range(30))
def test_runs_stay_inside_whatever_the_arrays_hold(shim, seed):
    r = random.Random(1000 + seed)
    wild = lambda: r.choice([0, 1, -1, 5, 17, 2147483647, -2147483648, r.randint(-300, 300)])  # noqa: E731
    P, B, T, width, pages = r.choice([16, 128]), r.randint(1, 6), r.randint(1, 50), r.randint(1, 4), 7
    table = _i32([[wild() for _ in range(width)] for _ in range(B)])
    lens, cu = _i32([wild() for _ in range(B)]), _i32([wild() for _ in range(B + 1)])
    seq = _i32([r.randrange(B) for _ in range(T)])
    out = np.zeros((T, 7), dtype=np.int32)
    shim.kv_runs(_ptr(table), _ptr(lens), _ptr(cu), width, B, T, P, pages, _ptr(seq), _ptr(out))
    for t in range(T):
        starts, pos, slot, n, nxt, page, bad = out[t]
        assert nxt > t and nxt <= T
        if starts:
            assert 0 <= slot and n >= 1 and slot + n <= P and t + n <= T and pos + n <= width * P
            assert -1 <= page < pages


def _segments(shim, lens, cu, T, B, width, heads, group, rows, shares, unit=32, extra=0):
    """Every share's segments, in order, and the number of units."""
    pages = _i32(np.zeros((B, width)))
    out, total, got = np.zeros((20000, 11), dtype=np.int32), ctypes.c_int64(0), []
    for c in range(shares):
        n = shim.kv_segments(_ptr(pages), _ptr(lens), _ptr(cu), width, B, T, 16, 1, heads, group, rows.bit_length() - 1,
                             unit.bit_length() - 1, extra, c, shares, _ptr(out), 20000, ctypes.byref(total))
        assert n >= 0
        got.append(out[:n].tolist())
    return got, total.value


@pytest.mark.parametrize("seed", range(25))
def test_shares_have_every_unit_once(shim, seed):
    """The shares' segments are all units of all tiles, each once and in
    order; every tile has a unit, no share is more than a unit longer than
    another (a tile's extra units counted), and a tile's parts know of one another."""
    r = random.Random(50 + seed)
    B, shares, P, unit = r.choice([1, 3, 17, 40]), r.choice([1, 7, 152, 1000]), 16, r.choice([32, 128])
    heads, group, rows = r.choice([1, 2, 8]), r.choice([1, 3, 5, 16, 128]), r.choice([8, 16, 256])
    extra = r.choice([0, 1, 2, 5])
    counts = [r.choice([0, 1, 1, r.randint(0, 40), r.randint(0, 300 // group + 1)]) for _ in range(B)]
    lens = [r.choice([0, n, n + r.randint(0, 3000)]) for n in counts]
    if not any(counts):
        counts[0] = 1
    width = max(1, -(-max(lens) // P))
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    got, total = _segments(shim, _i32(lens), _i32(cu), cu[-1], B, width, heads, group, rows, shares, unit, extra)
    expect, tiles = [], 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        for i in range(-(-m * group // rows)):
            end = min((i + 1) * rows, m * group)
            sees = [max(0, n - m + x // group + 1) for x in (i * rows, end - 1)]
            tile = (b, cu[b] + i * rows // group, i * rows % group, end - i * rows)
            units = max(1, -(-sees[1] // unit))
            tiles += heads
            for h in range(heads):
                expect += [(*tile, h, *sees, u * unit, min((u + 1) * unit, sees[1])) for u in range(units)]
    flat, sizes, owners = [], [], {}
    for c, segs in enumerate(got):
        sizes.append(0)
        for b, t, rem, n, h, k0, k1, parts, owner, see0, see1 in segs:
            units = max(1, -(-(k1 - k0) // unit))
            sizes[-1] += units
            flat += [(b, t, rem, n, h, see0, see1, k0 + u * unit, min(k0 + (u + 1) * unit, k1)) for u in range(units)]
            owners.setdefault((b, t, rem, h), []).append((c, parts, owner))
    assert flat == expect and total == len(expect) + extra * tiles
    each = total // shares
    assert max(sizes) <= each + 1 and not any(sizes[total:])
    if extra == 0:
        assert min(sizes) >= each
    for of in owners.values():
        assert [c for c, _, _ in of] == list(range(of[0][0], of[0][0] + len(of)))
        for _, parts, owner in of:
            assert parts == len(of) and (parts == 1 or owner == of[0][0])
    for c, segs in enumerate(got):                     # at most one tile begun and left, one gone on with
        cut = [(owner == c) for *_, parts, owner, _, _ in segs if parts > 1]
        assert cut.count(True) <= 1 and cut.count(False) <= 1


@pytest.mark.parametrize("group", range(1, 129))
def test_rows_of_a_tile(shim, group):
    out = np.zeros((256, 2), dtype=np.int32)
    for rem in {0, 1 % group, group // 2, group - 1}:
        shim.kv_rows(7, rem, 256, group, _ptr(out))
        assert out.tolist() == [[7 + (rem + r) // group, (rem + r) % group] for r in range(256)]


@pytest.mark.parametrize("seed", range(25))
def test_segments_stay_inside_whatever_the_arrays_hold(shim, seed):
    r = random.Random(2000 + seed)
    wild = lambda: r.choice([0, 1, -1, 5, 17, 2147483647, -2147483648, r.randint(-300, 300)])  # noqa: E731
    B, T, width, heads, group, rows = r.randint(1, 9), r.randint(1, 30), r.randint(1, 40), 2, 3, 16
    lens, cu = _i32([wild() for _ in range(B)]), _i32([wild() for _ in range(B + 1)])
    got, total = _segments(shim, lens, cu, T, B, width, heads, group, rows, 5)
    assert sum(max(1, -(-(s[6] - s[5]) // 32)) for c in got for s in c) == total
    for c in got:
        for b, t, rem, n, h, k0, k1, parts, owner, see0, see1 in c:
            assert 0 <= b < B and 0 <= h < heads and 0 <= t and 1 <= n <= rows and t + (rem + n - 1) // group < T
            assert 0 <= k0 and k1 <= width * 16 and see1 <= width * 16 and 1 <= parts <= 5 and 0 <= owner < 5


@pytest.mark.parametrize("length,new", [(49, 1), (60, 20), (49, 48), (2147483647, 3), (-1, 1), (-2147483648, 20)])
def test_a_bad_length_has_no_places(shim, length, new):
    """Of a sequence longer than its table, or shorter than empty, nothing is
    written and no query is rotated; its neighbours have their places."""
    P, width, B, lens = 16, 3, 3, [20, length, 48]
    cu = [0, 5, 5 + new, 9 + new]
    T = cu[-1]
    seq, out, pos = _seq_of(cu, T, B), np.zeros((T, 7), dtype=np.int32), np.zeros(T, dtype=np.int32)
    table, lens_a, cu_a = _i32([[10 * b + i for i in range(width)] for b in range(B)]), _i32(lens), _i32(cu)
    shim.kv_runs(_ptr(table), _ptr(lens_a), _ptr(cu_a), width, B, T, P, 40, _ptr(seq), _ptr(out))
    shim.kv_positions(_ptr(table), _ptr(lens_a), _ptr(cu_a), width, B, T, P, 40, _ptr(seq), _ptr(pos))
    for t in range(T):
        starts, _, _, n, nxt, _, bad = out[t]
        assert t < nxt <= cu[seq[t] + 1] and bool(bad) == (seq[t] == 1)
        assert (pos[t] == -1 and not starts and n == 0) if bad else pos[t] == lens[seq[t]] - cu[seq[t] + 1] + t
    assert [bool(out[t][0]) for t in range(5)] == [True, True, False, False, False]       # positions 15 | 16 .. 19
    assert out[5 + new][0]


@pytest.mark.parametrize("cu,good", [([0, 2, 9, 9], [0]), ([-3, 2, 4, 4], [1]), ([0, 2, 4, 5], [0, 1]), ([0, 3, 1, 4], [0, 2])])
def test_bad_offsets_leave_their_sequence_out(shim, cu, good):
    T, B, width, heads, group = 4, 3, 3, 2, 5
    lens, cu_a = _i32([40, 45, 20]), _i32(cu)
    got, _ = _segments(shim, lens, cu_a, T, B, width, heads, group, 8, 7)
    rows = {(b, h): 0 for b in good for h in range(heads)}
    for b, t, rem, n, h, k0, k1, parts, owner, see0, see1 in (s for c in got for s in c):
        assert b in good and cu[b] <= t and see1 <= lens[b]
        rows[b, h] += n if k0 == 0 else 0
    assert all(n == (cu[b + 1] - cu[b]) * group for (b, _), n in rows.items())


def test_a_warps_segments_are_handed_over_in_order(tmp_path):
    """One lane plans, all lanes read: no data race where a vote orders no memory (a race ends the program with 66)."""
    exe = str(tmp_path / "race")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=thread", os.path.join(HERE, "kv_warp_race.cpp"), "-o", exe,
                    "-pthread"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_a_stream_of_another_device_is_refused(lib):
    """The calls run on the given stream or not at all: not on the current stream of the cache's device instead."""
    class Other:
        device, cuda_stream = torch.device("cuda", 1), 0
    c = _cpu_cache()
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="stream"):
        mhc.kv_append(c, x, x, table, lens, stream=Other())
    with pytest.raises(ValueError, match="stream"):
        mhc.kv_attend(x, c, table, lens, stream=Other())
    with pytest.raises(ValueError, match="stream"):
        mhc.kv_workspace_for(c, 2, 1, 1, Other())


def test_the_binding_is_built_anew_for_another_pytorch(tmp_path, monkeypatch):
    """An object compiled for another PyTorch or interpreter is not linked, however new it is."""
    ran = []

    def run(cmd, what):
        ran.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(mbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(mbuild, "BINDING", str(tmp_path / "_mhc_kv.so"))
    monkeypatch.setattr(mbuild, "_run", run)

    def built():
        ran.clear()
        mbuild._link_binding(mbuild._compile_binding())
        return len(ran)
    assert built() == 2 and built() == 0
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert built() == 2 and built() == 0
    monkeypatch.setattr(mbuild.sys, "version", "another interpreter")
    assert built() == 2 and built() == 0


def test_status_string_of_an_unsupported_shape(lib):
    """It names the cache's limits as well as the seam's."""
    text = lib.mhc_status_string(2).decode()
    assert all(w in text for w in ("C a multiple of 8", "head_dim", "page_tokens", "rotary_dim", "query heads"))
