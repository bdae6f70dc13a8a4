"""GPU checks of calls of the paged cache at their edges."""
import random

import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from kv_reference import check_append
from test_kv_more_cpu import plan_compact, plan_fork
from test_kv_window_gpu import attend, check, make, of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mhc.load_library()
    assert mhc.device_status() == 0
    yield
    assert mhc.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_fork_of_a_batch_that_has_ended():
    """Nobody goes on: empty tables, the caches as they were; and a batch may begin after it."""
    cache = mhc.kv_cache(4, 1, 16, 64)
    got = mhc.kv_fork(cache, _i32([[0, 1], [2, -1]]), _i32([20, 3]), _i32([]), room=1)
    assert got["block_table"].shape == (0, 2) and got["seq_lens"].shape == (0,)
    got = mhc.kv_fork(cache, got["block_table"], got["seq_lens"], _i32([]), room=_i32([]))
    assert got["block_table"].shape == (0, 2)
    got = mhc.kv_fork(cache, got["block_table"], got["seq_lens"], _i32([-1]), room=17)
    assert got["block_table"].tolist() == [[0, 1]] and got["seq_lens"].tolist() == [0]
    assert not cache["k"].view(torch.uint8).any()


@pytest.mark.parametrize("where", ["nowhere", "fork", "attend"])
def test_pages_that_ran_out_are_reported_after_a_bad_index(where):
    """Both between two queries: the first tells of the index, the next of the pages, the third of nothing."""
    cache = mhc.kv_cache(2, 1, 16, 64)
    bad = where == "fork"                              # a full page that is none, and no place for a further token
    got = mhc.kv_fork(cache, _i32([[0, -1], [1, 77 if bad else -1]]), _i32([16, 32 if bad else 16]), _i32([0, 0, 1]), room=1)
    assert got["block_table"].tolist() == [[0, -1], [0, -1], [1, -1]]
    if where == "attend":
        mhc.kv_attend(torch.zeros(1, 1, 64, device="cuda").bfloat16(), cache, _i32([[5]]), _i32([3]))
    assert [mhc.device_status() for _ in range(3)] == ([6, 0, 0] if where == "nowhere" else [5, 6, 0])


def test_a_step_without_new_tokens():
    """Three sequences of which none has a new token: empty queries back, the cache as it was."""
    cache = mhc.kv_cache(3, 2, 16, 64)
    w = torch.ones(64, device="cuda").bfloat16()
    x = torch.zeros(0, 8, 64, device="cuda").bfloat16()
    table, lens, cu = _i32([[0], [1], [2]]), _i32([3, 0, 16]), _i32([0, 0, 0, 0])
    for norms in ({}, {"k_norm": w}, {"q_norm": w}, {"q_norm": w.expand(4, 64), "k_norm": w.expand(2, 64)}):
        q = mhc.kv_append(cache, x[:, 4:6], x[:, 6:], table, lens, cu, q=x[:, :4], **norms)
        assert q.shape == (0, 4, 64)
        got = mhc.kv_attend(q, cache, table, lens, cu, window=4, return_lse=True)
        assert got["out"].shape == (0, 4, 64) and got["lse"].shape == (0, 4)
    assert not cache["k"].view(torch.uint8).any() and not cache["v_scale"].any()


@pytest.mark.parametrize("B,width", [(5, 8192), (9, 5000), (11, 3001)])
def test_wide_tables_in_place(B, width):
    """Rows whose threads do not divide the grid's, written in place: the definition's tables."""
    P, pages = 16, B * width + 50
    r = random.Random(width)
    order = r.sample(range(pages), B * width)
    lens = [r.randint(0, width * P - 20) if b else width * P - 20 for b in range(B)]
    table = [[order[b * width + i] if i * P < lens[b] and r.random() < 0.95 else -1 for i in range(width)] for b in range(B)]
    cache = mhc.kv_cache(pages, 1, P, 64)
    at, n = _i32(table), _i32(lens)
    out, want, _, _ = plan_fork(table, lens, pages, 4, None, 17, 3000, 40, None)
    mhc.kv_fork(cache, at, n, room=17, window=3000, sinks=40, out={"block_table": at, "seq_lens": n})
    assert at.tolist() == out and n.tolist() == want
    at, n = _i32(table), _i32(lens)
    out, top, _, _ = plan_compact(table, lens, pages, 4, None)
    got = mhc.kv_compact(cache, at, n, out={"block_table": at, "pages": _i32(0)})
    assert got["block_table"].tolist() == out and got["pages"].item() == top


def us(made, windowed=True):
    """The least time of a few calls."""
    q, cache, rows, lens, cu, window, sinks = made
    args, best = (q, cache, _i32(rows), _i32(lens), None if cu is None else _i32(cu)), 1e9
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        mhc.kv_attend(*args, **({"window": window, "sinks": sinks} if windowed else {}))
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


WIDE = [
    # D, P, H, Hq, new tokens, lengths, window, sinks
    (128, 64, 2, 10, [300], [5000], 4096, 40), (64, 16, 1, 1, [600], [5000], 3000, 0), (64, 128, 2, 16, [20, 90], [4100, 6000], 4096, 500),
    (128, 32, 1, 40, [30], [9000], 8000, 129),
]


@pytest.mark.parametrize("case", WIDE)
def test_nan_values_in_wide_windows(case):
    """NaN at both ends of windows of thousands of keys, in the middle and among the first: NaN in those dims of the rows that
    see them, no other number changes; and a call with one takes about as long as one without."""
    D, P, H, Hq, counts, lens, window, sinks = case
    made, clean = make(case, 500), make(case, 500)
    q, cache, rows, _, cu, _, _ = made
    put = []
    for b, (m, n) in enumerate(zip(counts, lens)):
        for j in {0, sinks, n - m - window, n - m - window + 1, n - m - window + 2, n - window - m // 2, n - window, n - 1500, n - m,
                  n - m // 2, n - 2, n - 1}:
            if 0 <= j < n and rows[b][j // P] >= 0:
                d = (7 * j + 3) % D
                for k, c in enumerate((cache, clean[1])):
                    c["v"].view(torch.uint8)[rows[b][j // P], j % H, j % P, d] = 0x38 if k else (0x7F if j % 2 else 0xFF)
                put.append((b, j, j % H, d))
    got, expect = attend(made), attend(clean)
    check(expect, *of(clean))
    nan, G = torch.zeros_like(got["out"], dtype=torch.bool), Hq // H
    for b, j, h, d in put:
        for t in range(cu[b], cu[b + 1]):
            p = lens[b] - (cu[b + 1] - t)
            if j <= p and (j > p - window or j < sinks):
                nan[t, h * G:(h + 1) * G, d] = True
    assert nan.any() and not nan.all(-1).any()
    assert torch.equal(got["out"].isnan(), nan)
    assert torch.equal(got["out"][~nan], expect["out"][~nan]) and torch.equal(got["lse"], expect["lse"])
    with_nan, without = us(made), us(clean)
    assert with_nan < 3 * without + 100, (with_nan, without)


def test_ends_full_of_nan():
    """Every value a window's ends hold is NaN: NaN in every row that sees one of them, whose number is the definition's."""
    case = (64, 32, 1, 5, [200], [3000], 700, 10)
    D, P, H, Hq, counts, lens, window, sinks = case
    made, clean = make(case, 510), make(case, 510)
    q, cache, rows, _, cu, _, _ = made
    m, n = counts[0], lens[0]
    where = [*range(n - m - window, n - m - window + 120), *range(n - 60, n)]
    for j in where:
        for k, c in enumerate((cache, clean[1])):
            c["v"].view(torch.uint8)[rows[0][j // P], :, j % P] = 0x38 if k else 0x7F
    got, expect = attend(made), attend(clean)
    see = torch.tensor([any(j <= p and j > p - window for j in where) for p in range(n - m, n)], device="cuda")
    assert see.any() and not see.all()
    assert got["out"][see].isnan().all() and torch.equal(got["out"][~see], expect["out"][~see])
    assert torch.equal(got["lse"], expect["lse"])


@pytest.mark.parametrize("tokens,short,window", [(1, 127, 2048), (1, 127, 16384), (1, 99, 8192), (51, 15, 4096)])
def test_one_long_sequence_in_a_wide_window(tokens, short, window):
    """One long sequence beside short ones: a window saves work, so the call takes no longer than without one (to a
    fifth and 10 us); and the long sequence's rows are the definition's."""
    counts, lens = None if tokens == 1 else [tokens] * (short + 1), [20000] + [500] * short
    made = make((128, 64, 2, 10, counts, lens, window, 4), 520)
    q, cache, rows, _, cu, _, _ = made
    rows = [r + [-1] * 100 for r in rows]                              # a table that has room for longer ones
    every = [[max(x, 0) for x in r] for r in rows]
    got = attend((q, cache, rows, lens, cu, window, 4))
    n = 1 if cu is None else tokens
    check({k: t[:n] for k, t in got.items()}, q[:n], cache, rows[:1], lens[:1], None if cu is None else cu[:2], 128 ** -0.5, window, 4)
    # heads as a model has them, for the time
    wide = mhc.kv_cache(cache["k"].shape[0], 8, 64, 128)
    x = torch.randn(q.shape[0], 40, 128, device="cuda").bfloat16()
    with_window, without = us((x, wide, rows, lens, cu, window, 4)), us((x, wide, every, lens, cu, None, 0), False)
    assert with_window < 1.2 * without + 10, (with_window, without)


def append_us(counts, D, P, normed):
    """An append of 40 query and 8 key/value heads, held to its definition without norms; the least time of a few calls."""
    B, T, H, Hq = len(counts), sum(counts), 8, 40
    width = -(-(max(counts) + 40) // P)
    cache = mhc.kv_cache(B * width, H, P, D)
    g = torch.Generator(device="cuda").manual_seed(T)
    rows = torch.randperm(B * width, generator=g, device="cuda").view(B, width).tolist()
    lens, cu = [n + 7 * i % 40 for i, n in enumerate(counts)], [0]
    for n in counts:
        cu.append(cu[-1] + n)
    x = torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda").bfloat16()
    q, k, v = x.split([Hq, H, H], dim=1)
    angles = torch.rand(width * P, D // 2, generator=g, device="cuda") * 6
    w = torch.ones(D, device="cuda").bfloat16()
    norms = {"q_norm": w, "k_norm": w} if normed else {}
    args, out = (cache, k, v, _i32(rows), _i32(lens), _i32(cu)), torch.empty(T, Hq, D, device="cuda").bfloat16()
    before, best, cos, sin = {n: t.cpu() for n, t in cache.items()}, 1e9, angles.cos(), angles.sin()
    for i in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        mhc.kv_append(*args, q=q, cos=cos, sin=sin, q_out=out, **norms)
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
        if i == 0 and not normed:
            check_append(before, {n: t.cpu() for n, t in cache.items()}, k.cpu(), v.cpu(), rows, lens, cu, cos.cpu(),
                         sin.cpu(), q=q.cpu(), q_out=out.cpu())
    return best


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("D,P", [(128, 128), (128, 64), (64, 128), (64, 32)])
def test_appends_of_8_to_20_tokens_a_sequence(D, P, normed):
    """A prompt beside single tokens, and a few tokens of one sequence, 8 to 20 a sequence on average: as long as the
    prompt and the single tokens would take in calls of their own, or as some more tokens, to half as much and 5 us."""
    n = 150 if P > 64 else 70
    apart = append_us([n], D, P, normed) + append_us([1] * 7, D, P, normed)
    assert append_us([n] + [1] * 7, D, P, normed) < 1.5 * apart + 5
    assert append_us([min(16, P // 2 - 1)], D, P, normed) < 1.5 * append_us([40], D, P, normed) + 5
