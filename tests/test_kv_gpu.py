"""GPU checks of the paged 8-bit key/value cache: mhc_kv_append and
mhc_kv_attend, through the binding, against plain 64-bit forms."""
import math

import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from mhc_hyper_connection_pre_gb300.graphs import SeamGraph
from kv_reference import attend, check_append, check_attend, e4m3_round

pytestmark = pytest.mark.gpu

INDEX_ERROR = 5


@pytest.fixture(autouse=True)
def _status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mhc.load_library()
    assert mhc.device_status() == 0
    yield
    assert mhc.device_status() == 0


def _cpu(d):
    return {k: v.cpu() for k, v in d.items()}


def _tables(lens, P, seed, extra=2, width=None):
    """A table of distinct pages in random order, unused entries out of range."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // P) for n in lens]
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=g).tolist()
    width = width or max(1, max(used))
    rows, at = [], 0
    for n in used:
        rows.append(order[at:at + n] + [-7] * (width - n))
        at += n
    return rows, pages


def _random_cache(pages, H, P, D, seed, powers=True):
    """A cache as appended normal values leave it; every slot filled."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = mhc.kv_cache(pages, H, P, D)
    for n in ("k", "v"):
        x = torch.randn(pages, H, P, D, generator=g, device="cuda").clamp(-6, 6) * 64
        cache[n].copy_(x.to(torch.float8_e4m3fn))
        s = torch.randint(-8, -4, (pages, H), generator=g, device="cuda").float().exp2()
        if not powers:
            s = s * (1 + torch.rand(pages, H, generator=g, device="cuda"))
        cache[n + "_scale"].copy_(s)
    return cache


def _spoil_unused(cache, rows, lens, P):
    """NaN codes in every slot past a sequence's end."""
    for r, n in zip(rows, lens):
        if n % P:
            for c in ("k", "v"):
                cache[c].view(torch.uint8)[r[n // P], :, n % P:] = 0x7F


def _cu(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append ---

APPENDS = [
    # D, P, H, Hq, new tokens of each sequence (None: one each), lengths, R, interleaved, fused
    (128, 64, 8, 40, None, [1], 128, False, True),
    (128, 64, 8, 40, None, [64, 65, 1, 130, 0, 63], 128, False, True),
    (128, 16, 2, 2, [3, 0, 17, 1], [3, 5, 40, 33], 64, True, False),
    (64, 16, 3, 9, [16, 1, 15], [16, 17, 47], 64, False, True),
    (64, 32, 1, 5, [100], [101], 32, True, True),
    (64, 128, 2, 16, [300, 5], [301, 6], 16, False, False),
    (128, 128, 4, 4, [257, 128, 1], [300, 128, 129], 128, True, True),
    (128, 32, 2, 8, [5, 4], [3, 4], 128, False, True),        # more new tokens than the sequence has places for
    (64, 64, 4, 8, [70], [200], 0, False, False),
    (128, 16, 1, 1, [1] * 45 + [2], [20] * 46, 128, False, True),
    (64, 16, 1, 1, [2] * 70, list(range(2, 72)), 64, True, False),
]


def _append_inputs(T, H, Hq, D, R, fused, seed, width):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        rows = torch.randn(T, (Hq + 2 * H) * D, generator=g, device="cuda").bfloat16()
        q = rows[:, :Hq * D].unflatten(1, (Hq, D))
        k = rows[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        v = rows[:, (Hq + H) * D:].unflatten(1, (H, D))
    else:
        q, k, v = (torch.randn(T, n, D, generator=g, device="cuda").bfloat16() for n in (Hq, H, H))
    cos = sin = None
    if R:
        angle = torch.rand(width, R // 2, generator=g, device="cuda") * 6.3
        cos, sin = angle.cos(), angle.sin()
    return q, k, v, cos, sin


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_is_its_definition(case):
    D, P, H, Hq, counts, lens, R, inter, fused = APPENDS[case]
    rows, pages = _tables(lens, P, case)
    cu = None if counts is None else _cu(counts)
    T = len(lens) if counts is None else cu[-1]
    cache = _random_cache(pages, H, P, D, case)
    for n in ("k", "v"):
        cache[n + "_scale"] *= 2.0 ** -3                       # old scales that some appends outgrow
    q, k, v, cos, sin = _append_inputs(T, H, Hq, D, R, fused, case, max(lens) + 1)
    before = _cpu({n: t.clone() for n, t in cache.items()})
    q_out = mhc.kv_append(cache, k, v, _i32(rows), _i32(lens), None if cu is None else _i32(cu), q=q, cos=cos,
                          sin=sin, interleaved=inter)
    table = _cpu({"k": k, "v": v, "q": q, "o": q_out})
    check_append(before, _cpu(cache), table["k"], table["v"], rows, lens, cu, None if cos is None else cos.cpu(),
                 None if sin is None else sin.cpu(), inter, table["q"], table["o"])


def test_append_without_queries_and_in_place():
    D, P, H, lens = 128, 16, 2, [5, 40, 17]
    rows, pages = _tables(lens, P, 3)
    q, k, v, cos, sin = _append_inputs(3, H, 4, D, D, True, 3, 64)
    a, b = _random_cache(pages, H, P, D, 3), _random_cache(pages, H, P, D, 3)
    expect = mhc.kv_append(a, k, v, _i32(rows), _i32(lens), q=q, cos=cos, sin=sin).clone()
    assert mhc.kv_append(b, k, v, _i32(rows), _i32(lens), cos=cos, sin=sin) is None
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8))
    got = mhc.kv_append(a, k, v, _i32(rows), _i32(lens), q=q, cos=cos, sin=sin, q_out=q)
    assert got is q and torch.equal(q, expect)
    for n in a:                                                # appending the same tokens again changes nothing
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8))


def test_append_token_by_token_and_at_once():
    """A prompt appended at once and token by token: the same scales, and the
    same numbers where growing scales did not push them into e4m3's subnormals."""
    D, P, H, n = 64, 16, 2, 50
    rows, pages = _tables([n], P, 5)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(n, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    k *= torch.logspace(-2, 2, n, base=2, device="cuda")[:, None, None].bfloat16()
    whole, steps = mhc.kv_cache(pages, H, P, D), mhc.kv_cache(pages, H, P, D)
    mhc.kv_append(whole, k, v, _i32(rows), _i32([n]), _i32([0, n]))
    for t in range(n):
        mhc.kv_append(steps, k[t:t + 1], v[t:t + 1], _i32(rows), _i32([t + 1]))
    for c in ("k", "v"):
        assert torch.equal(whole[c + "_scale"], steps[c + "_scale"])
        x, y = whole[c].float(), steps[c].float()
        assert torch.equal(x[x.abs() >= 2.0 ** -6], y[x.abs() >= 2.0 ** -6])
        assert ((x - y).abs() <= 2.0 ** -9).all()


def test_append_special_numbers():
    """Infinities and NaN are stored as NaN and do not move the scale; zeros
    and the smallest numbers take the smallest scale."""
    D, P, H = 64, 16, 1
    k = torch.zeros(6, H, D, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    k[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3.0])
    k[1, 0, :3] = torch.tensor([448.0, 450.0, -1e-3])
    k[2, 0, 0] = 2.0 ** -130
    k[4, 0, 0] = 3.3e38
    v[3, 0, 0] = -448.0 * 2 ** 5
    lens = [1] * 6
    rows, pages = _tables(lens, P, 1)
    cache = _random_cache(pages, H, P, D, 1)
    before = _cpu({n: t.clone() for n, t in cache.items()})
    mhc.kv_append(cache, k, v, _i32(rows), _i32(lens))
    after = _cpu(cache)
    check_append(before, after, k.cpu(), v.cpu(), rows, lens, None)
    p = [r[0] for r in rows]
    assert after["k"][p[0], 0, 0, :3].double().isnan().all() and after["k_scale"][p[0], 0] == 2.0 ** -7
    assert after["k_scale"][p[1], 0] == 2.0 and after["k_scale"][p[3], 0] == 2.0 ** -116
    assert after["v_scale"][p[3], 0] == 2.0 ** 5


def test_append_bad_indices_touch_nothing():
    """Pages out of range, lengths past the table and positions past the
    rotation's tables: the tokens concerned are left out, the others are not."""
    D, P, H = 128, 16, 2
    lens = [5, 20, 33, 4, 10]
    rows, pages = _tables(lens, P, 9)
    bad = [list(r) for r in rows]
    bad[1][1], bad[2][2] = pages, -1
    q, k, v, cos, sin = _append_inputs(5, H, 2, D, D, True, 9, 40)
    cache, expect = _random_cache(pages, H, P, D, 9), _random_cache(pages, H, P, D, 9)
    mhc.kv_append(cache, k, v, _i32(bad), _i32(lens), q=q, cos=cos, sin=sin)
    assert mhc.device_status() == INDEX_ERROR
    keep = [0, 3, 4]
    mhc.kv_append(expect, k[keep], v[keep], _i32([rows[i] for i in keep]), _i32([lens[i] for i in keep]), cos=cos,
                  sin=sin)
    for n in cache:
        assert torch.equal(cache[n].view(torch.uint8), expect[n].view(torch.uint8))
    cache = _random_cache(pages, H, P, D, 9)
    before = {n: t.clone() for n, t in cache.items()}
    mhc.kv_append(cache, k, v, _i32(rows), _i32(lens), cos=cos[:2], sin=sin[:2])          # no row for any position
    assert mhc.device_status() == INDEX_ERROR
    for n in cache:
        assert torch.equal(cache[n].view(torch.uint8), before[n].view(torch.uint8))
    mhc.kv_append(cache, k, v, _i32(rows), _i32([0] * 5), _i32([0, 9, -4, 900, 2, 5]))    # offsets out of order
    assert mhc.device_status() == INDEX_ERROR


# ------------------------------------------------------------------ attend ---

ATTENDS = [
    # D, P, H, Hq, new tokens (None: one each), lengths
    (128, 64, 8, 40, None, [1]),
    (128, 64, 8, 40, None, [1000]),
    (128, 64, 2, 2, None, [1, 63, 64, 65, 0, 127, 128, 129, 500]),
    (64, 16, 4, 16, None, [15, 16, 17, 31, 32, 33, 0, 0, 257]),
    (64, 32, 1, 7, None, [2049, 3, 900]),
    (128, 128, 1, 16, None, [4097, 1]),
    (128, 16, 3, 9, [4, 1, 3, 0, 2], [40, 1, 3, 17, 300]),
    (128, 32, 2, 32, [4, 4, 4], [100, 4, 2]),                # rows without keys
    (64, 64, 2, 2, [70, 1], [70, 900]),
    (64, 16, 2, 10, [33], [50]),
    (128, 64, 1, 5, [150, 40], [150, 300]),
    (128, 128, 2, 6, [129, 64], [200, 64]),
    (64, 128, 1, 1, [260], [260]),
    (128, 16, 1, 128, [3], [90]),
    (64, 32, 1, 64, None, [77, 5]),
    (128, 64, 1, 40, [65, 0, 200], [65, 10, 190]),
    (64, 32, 2, 32, [2, 2], [300, 2]),                       # 32 and 33 rows, 16 and 17 rows
    (64, 32, 1, 11, [3, 3], [300, 1000]),
    (128, 32, 1, 8, [2, 2], [300, 2]),
    (128, 32, 1, 17, None, [1000, 30, 0]),
    (128, 16, 2, 64, [4, 3], [5000, 130]),                   # 128 and 129 rows, long
    (64, 64, 1, 43, [3, 3], [3001, 64]),
    (128, 32, 1, 33, None, [1000, 30, 0]),                   # one row more than the one-token kernel takes
    (128, 64, 2, 64, None, [700, 64]),
]


def _attend(case, seed, scale=None, powers=True, fill=None, **kw):
    D, P, H, Hq, counts, lens = case
    rows, pages = _tables(lens, P, seed)
    cu = None if counts is None else _cu(counts)
    T = len(lens) if counts is None else cu[-1]
    cache = _random_cache(pages, H, P, D, seed, powers)
    _spoil_unused(cache, rows, lens, P)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(T, Hq + 2, D, generator=g, device="cuda").bfloat16()[:, 1:-1]         # rows with a stride
    if fill:
        fill(q, cache, rows)
    got = mhc.kv_attend(q, cache, _i32(rows), _i32(lens), None if cu is None else _i32(cu), softmax_scale=scale,
                        return_lse=True, **kw)
    return got, (q, cache, rows, lens, cu, D ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("case", range(len(ATTENDS)))
def test_attend_is_its_definition(case):
    got, of = _attend(ATTENDS[case], case)
    check_attend(got, *of)


@pytest.mark.parametrize("case", [1, 3, 6, 10, 15])
@pytest.mark.parametrize("scale", [0.0, 1.5])
def test_attend_flat_and_sharp(case, scale):
    """A scale of zero (the mean of the values) and one that leaves one key;
    page scales that are no powers of two."""
    got, of = _attend(ATTENDS[case], 100 + case, scale, powers=False)
    check_attend(got, *of)


@pytest.mark.parametrize("case", [6, 7, 8, 10, 15])
def test_attend_later_keys_stay_out(case):
    """NaN and the largest numbers in keys and values after a token's position
    (later tokens of its own sequence) do not reach its row."""
    D, P, H, Hq, counts, lens = ATTENDS[case]

    def fill(q, cache, rows):
        for b, (n, m) in enumerate(zip(lens, counts)):
            if m >= 2 and n >= 2:
                for c in ("k", "v"):
                    cache[c].view(torch.uint8)[rows[b][(n - 1) // P], :, (n - 1) % P] = 0x7F
                    cache[c].view(torch.uint8)[rows[b][(n - 2) // P], :, (n - 2) % P, ::3] = 0x7E
    got, (q, cache, rows, _, cu, scale) = _attend(ATTENDS[case], 200 + case, fill=fill)
    clean = {n: t.clone() for n, t in cache.items()}
    for b, (n, m) in enumerate(zip(lens, counts)):
        if m >= 2 and n >= 2:
            for c in ("k", "v"):
                clean[c].view(torch.uint8)[rows[b][(n - 1) // P], :, (n - 1) % P] = 0x38
    last = [cu[b + 1] - 1 for b, (n, m) in enumerate(zip(lens, counts)) if m >= 2 and n >= 2]
    keep = [t for t in range(cu[-1]) if t not in last]
    ref = mhc.kv_attend(q, clean, _i32(rows), _i32(lens), _i32(cu), return_lse=True)
    check_attend(ref, q, clean, rows, lens, cu, scale)
    for n in ("out", "lse"):
        assert torch.equal(got[n][keep], ref[n][keep])
        assert got[n][last].isnan().all()


def test_attend_nan_query_stays_in_its_row():
    got, of = _attend(ATTENDS[6], 300, fill=lambda q, c, r: q[2, 1, :2].fill_(math.nan))
    assert got["out"][2, 1].isnan().all() and got["lse"][2, 1].isnan()
    got["out"][2, 1], of[0][2, 1] = 0, 0
    assert not got["out"].isnan().any()


def test_attend_large_and_small_queries():
    def fill(q, cache, rows):
        q[0] *= 2.0 ** 40
        q[1] *= 2.0 ** -60
        q[2, :, ::2] *= 2.0 ** -20
        q[3] = 0
    got, of = _attend((128, 32, 2, 8, None, [70, 70, 70, 70]), 400, fill=fill)
    check_attend(got, *of)


@pytest.mark.parametrize("case", [1, 2, 4, 6, 8, 11])
def test_attend_is_deterministic(case):
    a, of = _attend(ATTENDS[case], case)
    b, _ = _attend(ATTENDS[case], case)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_attend_long_context():
    got, of = _attend((128, 64, 1, 5, None, [40000, 3]), 1)
    check_attend(got, *of)


@pytest.mark.parametrize("case", [(64, 64, 1, 7, None, [40000]), (128, 32, 1, 17, None, [30001, 5]),
                                  (64, 16, 1, 40, [7], [30000]), (128, 128, 4, 44, None, [20000]), (128, 32, 1, 34, None, [30001, 5]),
                                 
                                  (64, 32, 2, 16, [2], [9000])])
def test_attend_few_long_sequences(case):
    """Tiles whose parts come from many shares of the work, in each kernel."""
    got, of = _attend(case, 3)
    check_attend(got, *of)


def test_attend_many_sequences():
    lens = [(i * 37) % 200 for i in range(700)]
    got, of = _attend((64, 16, 1, 2, None, lens), 2)
    check_attend(got, *of)


@pytest.mark.parametrize("B", [33, 257, 1500])
@pytest.mark.parametrize("Hq", [2, 16, 48])
def test_attend_many_short_sequences(B, Hq):
    """More sequences than a warp has lanes, counted by a warp and by a block; some empty."""
    lens = [(i * 29) % 40 for i in range(B)]
    got, of = _attend((64, 16, 1, Hq, None, lens), 5)
    check_attend(got, *of)


def test_attend_many_short_drafts():
    """More than 256 sequences in the tensor-memory kernel, ragged, some empty."""
    counts = [(i * 7) % 5 for i in range(400)]
    lens = [(i * 29) % 40 if n else 0 for i, n in enumerate(counts)]
    got, of = _attend((128, 16, 1, 12, counts, lens), 8)
    check_attend(got, *of)


def test_attend_bad_length_among_many():
    """The last of many sequences is looked at as well."""
    lens = [3] * 900
    rows, pages = _tables(lens, 16, 6)
    cache = _random_cache(pages, 1, 16, 64, 6)
    q = torch.randn(900, 2, 64, device="cuda").bfloat16()
    mhc.kv_attend(q, cache, _i32(rows), _i32(lens[:-1] + [17]))
    assert mhc.device_status() == INDEX_ERROR
    mhc.kv_attend(q.repeat(1, 20, 1), cache, _i32(rows), _i32(lens[:-1] + [-1]))
    assert mhc.device_status() == INDEX_ERROR


def test_attend_and_append_far_pages():
    """A cache whose last pages start beyond 2^32 bytes."""
    D, P, H = 128, 128, 8
    pages = (1 << 32) // (D * P * H) + 40
    cache = mhc.kv_cache(pages, H, P, D)
    small = _random_cache(3, H, P, D, 7)
    far = [pages - 1, pages - 20, pages - 7]
    for n in cache:
        for i, p in enumerate(far):
            cache[n][p].copy_(small[n][i])
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (torch.randn(2, h, D, generator=g, device="cuda").bfloat16() for h in (16, H, H))
    lens = [130, 100]
    near_rows, far_rows = [[0, 1], [2, 0]], [[far[0], far[1]], [far[2], far[0]]]
    for c, r in ((cache, far_rows), (small, near_rows)):
        mhc.kv_append(c, k, v, _i32(r), _i32(lens))
    for n in cache:
        for i, p in enumerate(far):
            assert torch.equal(cache[n][p].view(torch.uint8), small[n][i].view(torch.uint8))
    a = mhc.kv_attend(q, cache, _i32(far_rows), _i32(lens), return_lse=True)
    b = mhc.kv_attend(q, small, _i32(near_rows), _i32(lens), return_lse=True)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    del cache
    torch.cuda.empty_cache()


def test_attend_bad_pages_are_left_out():
    """Page numbers out of range hide their keys, and a length past the table
    is cut to it; the other sequences are as ever."""
    D, P, H, Hq = 128, 16, 2, 8
    lens = [40, 50, 20]
    rows, pages = _tables(lens, P, 11, width=4)
    cache = _random_cache(pages, H, P, D, 11)
    q = torch.randn(3, Hq, D, device="cuda").bfloat16()
    good = mhc.kv_attend(q, cache, _i32(rows), _i32(lens), return_lse=True)
    bad = [list(r) for r in rows]
    bad[1][1] = pages + 5
    got = mhc.kv_attend(q, cache, _i32(bad), _i32(lens), return_lse=True)
    assert mhc.device_status() == INDEX_ERROR
    for n in got:
        assert torch.equal(got[n][[0, 2]], good[n][[0, 2]])
    assert got["out"][1].isfinite().all() and (got["lse"][1] < good["lse"][1]).all()
    bad = [list(r) for r in rows]
    bad[0] = [-1, pages, 1 << 30, -(1 << 31)]
    got = mhc.kv_attend(q, cache, _i32(bad), _i32(lens), return_lse=True)
    assert mhc.device_status() == INDEX_ERROR
    assert (got["out"][0] == 0).all() and (got["lse"][0] == -math.inf).all()
    got = mhc.kv_attend(q, cache, _i32(rows), _i32([40, 50, -3]), return_lse=True)
    assert mhc.device_status() == INDEX_ERROR
    assert (got["out"][2] == 0).all() and torch.equal(got["out"][:2], good["out"][:2])
    full = [r if i != 2 else r[:2] + rows[0][:2] for i, r in enumerate(rows)]
    cut = mhc.kv_attend(q, cache, _i32(full), _i32([40, 50, 64]))
    got = mhc.kv_attend(q, cache, _i32(full), _i32([40, 50, 2000000000]))
    assert mhc.device_status() == INDEX_ERROR
    assert torch.equal(got["out"], cut["out"])
    mhc.kv_attend(q, cache, _i32(rows), _i32(lens), _i32([0, 5, 1, 3]))                     # offsets out of order
    assert mhc.device_status() == INDEX_ERROR


# ------------------------------------------------- streams, graphs, chain ---

def test_other_stream_and_graph_replay():
    """Both calls on a stream of their own, captured and replayed: the same
    bits as on the current stream."""
    D, P, H, Hq = 128, 64, 2, 10
    lens = [100, 64, 1]
    rows, pages = _tables(lens, P, 21)
    q, k, v, cos, sin = _append_inputs(3, H, Hq, D, D, True, 21, 128)
    table, n = _i32(rows), _i32(lens)
    a, b = _random_cache(pages, H, P, D, 21), _random_cache(pages, H, P, D, 21)
    qa = mhc.kv_append(a, k, v, table, n, q=q, cos=cos, sin=sin)
    oa = mhc.kv_attend(qa, a, table, n, return_lse=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    qb = mhc.kv_append(b, k, v, table, n, q=q, cos=cos, sin=sin, stream=st)
    ob = mhc.kv_attend(qb, b, table, n, return_lse=True, stream=st)
    st.synchronize()
    for x in ("out", "lse"):
        assert torch.equal(oa[x], ob[x])
    out, lse, qo = torch.zeros_like(oa["out"]), torch.zeros_like(oa["lse"]), torch.empty_like(qa)
    ws = mhc.kv_workspace_for(b, Hq, 3, 3, st)

    def step(s):
        mhc.kv_append(b, k, v, table, n, q=q, cos=cos, sin=sin, q_out=qo, stream=s)
        mhc.kv_attend(qo, b, table, n, out=out, lse=lse, workspace=ws, stream=s)
    for early in (False, True):
        graph = SeamGraph(step, st, early_launch=early)
        for _ in range(3):
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, oa["out"]) and torch.equal(lse, oa["lse"])


def test_workspace_contents_do_not_matter():
    case = (128, 64, 1, 5, None, [5000, 10])
    a, (q, cache, rows, lens, _, _) = _attend(case, 31)
    ws = mhc.kv_workspace_for(cache, 5, 2, 2)
    if ws is not None:
        for fill in (0xFF, 0x7F, 0):
            ws.fill_(fill)
            b = mhc.kv_attend(q, cache, _i32(rows), _i32(lens), return_lse=True, workspace=ws)
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_binding_refuses():
    """Nothing is launched for tensors that are not what the calls take."""
    D, P, H, Hq, T = 64, 16, 2, 4, 3
    c = _random_cache(4, H, P, D, 1)
    before = {n: t.clone() for n, t in c.items()}
    q, k, v, cos, sin = _append_inputs(T, H, Hq, D, D, False, 1, 64)
    table, lens = _i32([[0], [1], [2]]), _i32([1, 2, 3])

    def both(error, cache=c, q=q, k=k, v=v, table=table, lens=lens, cu=None, **kw):
        with pytest.raises(error):
            mhc.kv_append(cache, k, v, table, lens, cu, q=q, cos=cos, sin=sin)
        with pytest.raises(error):
            mhc.kv_attend(q, cache, table, lens, cu)

    for n in c:
        both(ValueError, dict(c, **{n: c[n].cpu()}))
        both(TypeError, dict(c, **{n: c[n].view(torch.uint8) if n in "kv" else c[n].double()}))
        both(TypeError, dict(c, **{n: None}))
    both(ValueError, dict(c, v=c["v"][:3]))
    both(ValueError, dict(c, k_scale=c["k_scale"].t().contiguous()))
    both(ValueError, dict(c, k=c["k"].transpose(1, 2).contiguous().transpose(1, 2)))
    both(TypeError, q=q.half(), k=k.half())
    both(ValueError, q=q.cpu(), k=k.cpu())
    both(ValueError, q=q[0], k=k[0])
    both(ValueError, q=q[:, :, :32], k=k[:, :, :32])
    both(ValueError, q=q[:, ::2], k=torch.cat([k, k], 1)[:, ::2])
    both(ValueError, q=q[:2], k=k[:2], v=v[:2])                    # without cu_q one token for each sequence
    both(TypeError, table=table.long())
    both(ValueError, table=table[:2])
    both(ValueError, lens=lens.cpu())
    both(ValueError, cu=_i32([0, 3]))
    both(TypeError, cu=_i32([0, 1, 2, 3]).long())
    with pytest.raises(ValueError):
        mhc.kv_append(c, k, v[:, :1], table, lens)
    with pytest.raises(ValueError):
        mhc.kv_append(c, k, v, table, lens, cos=cos)
    with pytest.raises(ValueError):
        mhc.kv_append(c, k, v, table, lens, cos=cos, sin=sin[:3])
    with pytest.raises(ValueError):
        mhc.kv_append(c, k, v, table, lens, q_out=q)
    with pytest.raises(mhc.MhcError) as e:
        mhc.kv_append(c, k, v, table, lens, cos=cos[:, :5].contiguous(), sin=sin[:, :5].contiguous())
    assert e.value.status == 2
    with pytest.raises(mhc.MhcError):
        mhc.kv_append(c, k, v, table, lens, q=q, q_out=k.expand(T, H, D).repeat(1, 2, 1)[:, :Hq].as_strided((T, Hq, D), (0, D, 1)))
    with pytest.raises(mhc.MhcError) as e:
        mhc.kv_attend(q[:, :3], c, table, lens)                     # three query heads over two key heads
    assert e.value.status == 1
    for bad in (dict(out=q[:2]), dict(lse=torch.empty(T, Hq + 1, device="cuda")), dict(out=torch.empty_like(q).cpu())):
        with pytest.raises(ValueError):
            mhc.kv_attend(q, c, table, lens, **bad)
    with pytest.raises(mhc.MhcError):
        mhc.kv_attend(q, c, table, lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mhc.MhcError):
        mhc.kv_attend(q, c, table, lens, out=q)
    for n in c:
        assert torch.equal(c[n].view(torch.uint8), before[n].view(torch.uint8))


def test_no_tokens():
    cache = mhc.kv_cache(2, 2, 16, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert mhc.kv_append(cache, none, none, _i32([[0]]), _i32([5]), _i32([0, 0])) is None
    assert mhc.kv_attend(none, cache, _i32([[0]]), _i32([5]), _i32([0, 0]))["out"].shape == (0, 2, 64)


def test_e4m3_rounding_of_the_reference_is_the_format():
    x = torch.linspace(-448, 448, 40001)
    x = torch.cat([x, x * 2.0 ** -14])
    assert torch.equal(e4m3_round(x.double()), x.to(torch.float8_e4m3fn).double())


def test_example_prompt_then_tokens():
    """The attention sublayer of examples/: prompts and then single tokens from a replayed graph, against all
    tokens in one call.  The two write the same keys and values with scales that grew differently, so each side
    is off by at most e4m3's half step (2^-4 of a value); the streams carry the rest unchanged."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_decode.py")
    spec = importlib.util.spec_from_file_location("attention_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    stepped, at_once = (t.double() for t in m.run())
    assert stepped.shape == at_once.shape == (3, 4, 4, 5120)
    assert (stepped - at_once).norm() <= 2 * 2.0 ** -4 * at_once.norm()
    for i in range(4):                                   # and no step is another's
        assert (stepped[:, i] - at_once[:, i]).norm() <= 2 * 2.0 ** -4 * at_once[:, i].norm()


# ------------------------------------------------------- bad device data ---

@pytest.mark.parametrize("counts", [None, [20, 7, 1]])
@pytest.mark.parametrize("length", [49, 60, 2147483647, -1, -2147483648])
def test_append_past_the_table_writes_nothing(length, counts):
    """A sequence longer than its table, or shorter than empty: its tokens
    are left out, as nothing says where they belong, so its pages keep their
    bytes and its queries are copied; the other sequences are appended."""
    D, P, H, Hq, lens = 64, 16, 2, 4, [48, 30, 5]
    rows, pages = _tables(lens, P, 13)
    cu = _cu(counts or [1, 1, 1])
    q, k, v, cos, sin = _append_inputs(cu[-1], H, Hq, D, D, True, 13, 64)
    got, expect = _random_cache(pages, H, P, D, 13), _random_cache(pages, H, P, D, 13)
    n, own = cu[1], lambda t: t[cu[1]:]
    q_out = mhc.kv_append(got, k, v, _i32(rows), _i32([length, 30, 5]), None if counts is None else _i32(cu), q=q,
                          cos=cos, sin=sin)
    assert mhc.device_status() == INDEX_ERROR
    q_own = mhc.kv_append(expect, own(k), own(v), _i32(rows[1:]), _i32([30, 5]), _i32([c - n for c in cu[1:]]),
                          q=own(q), cos=cos, sin=sin)
    for x in got:
        assert torch.equal(got[x].view(torch.uint8), expect[x].view(torch.uint8)), x
    assert torch.equal(q_out[:n], q[:n]) and torch.equal(q_out[n:], q_own)


@pytest.mark.parametrize("cu", [[0, 2, 4, 5], [0, 2, 4, 3], [1, 2, 4, 4], [-1, 2, 4, 4]])
def test_append_reports_offsets_that_miss_the_tokens(cu):
    """Also where the offset is that of a sequence without any of the call's tokens."""
    rows, pages = _tables([10, 11, 12], 16, 16)
    x = torch.ones(4, 1, 64, device="cuda").bfloat16()
    mhc.kv_append(mhc.kv_cache(pages, 1, 16, 64), x, x, _i32(rows), _i32([10, 11, 12]), _i32(cu))
    assert mhc.device_status() == INDEX_ERROR


@pytest.mark.parametrize("cu,good", [([0, 2, 9, 9], (0, 0, 2)), ([-3, 2, 4, 4], (1, 2, 4)),
                                     ([0, 2, 4, 5], (0, 0, 2))])
@pytest.mark.parametrize("Hq", [2, 80])
def test_offsets_out_of_range_leave_their_sequences_out(cu, good, Hq):
    """Offsets beyond the tokens or below zero do not say which positions a
    sequence's tokens have: they are not written to the cache and
    not attended to; a sequence with good offsets is."""
    D, P, H, T, lens = 128, 16, 2, 4, [40, 45, 20]
    rows, pages = _tables(lens, P, 14)
    q, k, v, cos, sin = _append_inputs(T, H, Hq, D, D, True, 14, 64)
    got, expect = _random_cache(pages, H, P, D, 14), _random_cache(pages, H, P, D, 14)
    b, begin, end = good
    at = slice(begin, end)
    q_out = mhc.kv_append(got, k, v, _i32(rows), _i32(lens), _i32(cu), q=q, cos=cos, sin=sin)
    assert mhc.device_status() == INDEX_ERROR
    q_good = mhc.kv_append(expect, k[at], v[at], _i32([rows[b]]), _i32([lens[b]]), _i32([0, end - begin]), q=q[at],
                           cos=cos, sin=sin)
    whole = {i for c, d in zip(cu, cu[1:]) if 0 <= c <= d <= T for i in range(c, d)}
    if whole == set(range(begin, end)):
        for x in got:
            assert torch.equal(got[x].view(torch.uint8), expect[x].view(torch.uint8)), x
    assert torch.equal(q_out[at], q_good)
    out, lse = torch.full((T, Hq, D), 7.0, device="cuda").bfloat16(), torch.full((T, Hq), 7.0, device="cuda")
    mhc.kv_attend(q_out, expect, _i32(rows), _i32(lens), _i32(cu), out=out, lse=lse)
    assert mhc.device_status() == INDEX_ERROR
    check_attend({"out": out[at], "lse": lse[at]}, q_good, expect, [rows[b]], [lens[b]], [0, end - begin], D ** -0.5)
    rest = [i for i in range(T) if i not in whole]
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()


# ---------------------------------------------------- workspaces of graphs ---

class _GraphCase:
    """Decode attention of a few sequences, and a call that needs a larger workspace."""

    def __init__(self):
        D, P, H, self.Hq, lens = 128, 64, 2, 10, [2000, 64, 700]
        rows, pages = _tables(lens, P, 41)
        self.cache, self.table, self.lens = _random_cache(pages, H, P, D, 41), _i32(rows), _i32(lens)
        g = torch.Generator(device="cuda").manual_seed(42)
        self.q = torch.randn(3, self.Hq, D, generator=g, device="cuda").bfloat16()
        self.out, self.lse = torch.empty_like(self.q), torch.empty(3, self.Hq, device="cuda")
        self.many = torch.randn(600, self.Hq, D, generator=g, device="cuda").bfloat16()
        self.cu = _i32([0, 500, 550, 600])
        self.expect = mhc.kv_attend(self.q, self.cache, self.table, self.lens, return_lse=True)
        torch.cuda.synchronize()

    def call(self, stream=None):
        mhc.kv_attend(self.q, self.cache, self.table, self.lens, out=self.out, lse=self.lse, stream=stream)

    def larger(self, stream=None):
        return mhc.kv_attend(self.many, self.cache, self.table, self.lens, self.cu, stream=stream)

    def workspace(self, stream=None):
        return mhc.kv_workspace_for(self.cache, self.Hq, 3, 3, stream)

    def check(self):
        torch.cuda.synchronize()
        assert torch.equal(self.out, self.expect["out"]) and torch.equal(self.lse, self.expect["lse"])
        self.out.zero_()
        self.lse.zero_()


def _blocks_of_others(nbytes, stream, n=6):
    """What somebody else allocates on the stream, in the sizes that a workspace may have left free."""
    with torch.cuda.stream(stream):
        return [torch.full((nbytes,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(n)]


def _capture(case, stream, kind):
    if kind == "seam":
        graph = SeamGraph(case.call, stream)
        return graph, graph.replay
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        case.call()
    return graph, graph.replay


@pytest.mark.parametrize("kind", ["torch", "seam"])
@pytest.mark.parametrize("warm", [True, False])
def test_graph_keeps_its_workspace(kind, warm):
    """Captured with the default workspace, after a call on the stream or as
    the first one; then larger calls on it, and others' tensors in whatever
    memory that set free: replays still give the outputs and touch nobody's."""
    case, st = _GraphCase(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    if warm:
        case.call(st)
        case.check()
    size = case.workspace(torch.cuda.current_stream()).numel()
    graph, replay = _capture(case, st, kind)
    others = _blocks_of_others(size, st)
    case.larger(st)
    others += _blocks_of_others(size, st)
    for _ in range(3):
        with torch.cuda.stream(st):
            replay()
        case.check()
        case.larger(st)
        others += _blocks_of_others(size, st, 2)
    torch.cuda.synchronize()
    assert all((o == 0x5A).all() for o in others)
    del graph, replay


def test_captures_have_workspaces_of_their_own():
    """Two captures on one stream and the stream's own calls: three buffers; the calls of one capture share theirs."""
    case, st = _GraphCase(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    case.call(st)
    torch.cuda.synchronize()
    own, seen, graphs = case.workspace(st).data_ptr(), [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            first = case.workspace()
            case.call()
            assert case.workspace().data_ptr() == first.data_ptr()
        seen.append(first.data_ptr())
        del first
        graphs.append(graph)
    assert len({own, *seen}) == 3 and case.workspace(st).data_ptr() == own
    for graph in graphs:
        graph.replay()
        case.check()


@pytest.mark.parametrize("kind", ["torch", "seam"])
def test_workspace_ends_with_its_graph(kind):
    """Graphs made and dropped do not add up; one that lives keeps its own."""
    import gc
    case, st = _GraphCase(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    case.call(st)
    kept, replay = _capture(case, st, kind)
    torch.cuda.synchronize()
    case.call(st)
    size, before = case.workspace(st).numel(), torch.cuda.memory_allocated()
    for _ in range(12):
        graph, again = _capture(case, st, kind)
        again()
        torch.cuda.synchronize()
        del graph, again
        gc.collect()
    case.call(st)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= before + 2 * size       # the last one may not be back yet
    with torch.cuda.stream(st):
        replay()
    case.check()


# ------------------------------------------------------ infinite queries ---

@pytest.mark.parametrize("Hq", [2, 40])
def test_attend_infinite_queries_without_keys(Hq):
    """Rows that see no key are zero and minus infinity, whatever their queries hold, in each kernel."""
    def fill(q, cache, rows):
        q[0], q[1, :, 5], q[2, 0], q[2, 1, ::2] = math.inf, -math.inf, math.nan, math.inf
    got, of = _attend((128, 16, 1, Hq, [6, 4], [3, 40]), 500, fill=fill)
    assert (got["out"][:3] == 0).all() and (got["lse"][:3] == -math.inf).all()
    got["out"][:3], of[0][:3] = 0, 0
    check_attend(got, *of)


@pytest.mark.parametrize("Hq", [2, 40])
@pytest.mark.parametrize("n", [1, 70, 5000])
def test_attend_infinite_query_is_nan(Hq, n):
    """A query with an infinity that sees a key gives NaN in each kernel, also where every product is minus infinity."""
    def fill(q, cache, rows):
        cache["k"].view(torch.uint8)[:, :, :, 0] = 0x38        # one
        q[0, 0] = 1.0
        q[0, 0, 0] = -math.inf
    got, of = _attend((64, 16, 1, Hq, None, [n]), 510, fill=fill)
    assert got["out"][0, 0].isnan().all() and got["lse"][0, 0].isnan()
    got["out"][0, 0], got["lse"][0, 0], of[0][0, 0] = 0, 0, 0
    assert not got["out"].isnan().any() and not got["lse"].isnan().any()


# ----------------------------------------------------------- value scales ---

SCALES = {
    "zero": [0.0], "one zero": [0.0, 1.0], "subnormal": [2.0 ** -140], "subnormal, then normal": [2.0 ** -149, 2.0 ** -3],
    "reciprocal at the border": [2.0 ** -128, 2.0 ** -127, 2.0 ** -122], "smallest of append": [2.0 ** -116],
    "far apart": [1.0, 2.0 ** -20], "far apart, no powers": [1.3 * 2.0 ** -20, 1.7],
}


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("case", [(128, 16, 2, 4, None, [70, 30]), (64, 16, 2, 32, None, [3000]), (128, 16, 1, 5, [30], [400]),
                                  (64, 32, 1, 40, [3, 7], [3001, 100]), (128, 32, 1, 50, [3], [5000])])
def test_attend_value_scales(kind, case):
    """Any finite value scales that are not negative, page after page.

    Beside the usual bounds: bf16's step in its subnormal range is 2^-133,
    half of that for the output's rounding and the rest for fp32's subnormals
    before it."""
    D, P, H, Hq, counts, lens = case

    def fill(q, cache, rows):
        for r in rows:
            for i, p in enumerate(r):
                if p >= 0:
                    cache["v_scale"][p] = SCALES[kind][i % len(SCALES[kind])]
    got, of = _attend(case, 600, fill=fill)
    out, lse, tol, tol_lse = attend(*of)
    assert out.isfinite().all()
    o, l = got["out"].double(), got["lse"].double()
    bad = ~((o - out).abs() <= tol + 2.0 ** -133)
    assert not bad.any(), (int(bad.sum()), o[bad][:4].tolist(), out[bad][:4].tolist())
    assert ((l - lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("kind", [[2.0 ** 115], [2.0 ** 100, 2.0 ** 115], [2.0 ** -3, 2.0 ** 115], [1.7 * 2.0 ** 114]])
@pytest.mark.parametrize("case", [(128, 16, 2, 4, None, [70, 30]), (64, 16, 2, 32, None, [3000]), (128, 16, 1, 5, [30], [400]),
                                  (64, 32, 1, 40, [3, 7], [3001, 100]), (128, 32, 1, 50, [3], [5000]),
                                  (64, 64, 1, 7, None, [40000])])
def test_attend_largest_values(kind, case):
    """Values near bf16's largest, whose sums are beyond fp32, from few and
    from many shares of the work: the output is their mean and so finite."""
    D, P, H, Hq, counts, lens = case

    def fill(q, cache, rows):
        for r in rows:
            for i, p in enumerate(r):
                if p >= 0:
                    cache["v_scale"][p] = kind[i % len(kind)]
    got, of = _attend(case, 610, fill=fill)
    check_attend(got, *of)
    assert got["out"].isfinite().all()


@pytest.mark.parametrize("case", [(128, 16, 2, 4, None, [70, 30]), (64, 16, 2, 32, None, [3000]), (128, 16, 1, 5, [30], [400]),
                                  (64, 32, 1, 40, [3, 7], [3001, 100]), (128, 32, 1, 50, [3], [5000])])
@pytest.mark.parametrize("apart", [12, 20, 28])
def test_attend_small_values_beside_unseen_large_ones(apart, case):
    """Pages whose values are smaller by 2^apart have all of the weight: each
    key may add 2^-26 times the largest value scale to the usual bounds (a
    weight below f16's normal numbers is off by 2^-35 of one, a code is at
    most 448)."""
    D, P, H, Hq, counts, lens = case

    def fill(q, cache, rows):
        q.fill_(1.0)
        for r, n in zip(rows, lens):
            for i, p in enumerate(r):
                if p >= 0 and i % 3 == 1:
                    cache["v_scale"][p], cache["k_scale"][p] = 1.0, 1.0
                    cache["k"].view(torch.uint8)[p] = 0xC8             # -4: logits of -256 and less
                elif p >= 0:
                    cache["v_scale"][p], cache["k_scale"][p] = 2.0 ** -apart, 2.0 ** -8
            if n % P:
                for c in ("k", "v"):
                    cache[c].view(torch.uint8)[r[n // P], :, n % P:] = 0x7F
    got, of = _attend(case, 620, fill=fill)
    out, lse, tol, tol_lse = attend(*of)
    o, l = got["out"].double(), got["lse"].double()
    assert ((o - out).abs() <= tol + max(lens) * 2.0 ** -26).all()
    assert ((l - lse).abs() <= tol_lse).all()


# ---------------------------------------------------------- mixed batches ---

@pytest.mark.parametrize("D,P,H,Hq,prompt,tokens", [(128, 64, 2, 10, 300, 40), (64, 16, 1, 8, 700, 7), (128, 16, 2, 4, 90, 300),
                                                    (64, 32, 2, 2, 257, 100)])
def test_prompt_beside_tokens(D, P, H, Hq, prompt, tokens):
    """A prompt's chunk and many single tokens in one call, some places empty:
    appended and attended to as in calls of their own."""
    counts = [1] * tokens
    counts[tokens // 2] = prompt
    lens = [max(n, (i * 37) % 150) for i, n in enumerate(counts)]
    lens[tokens // 2] += 100
    lens[0] = counts[0] = 0
    rows, pages = _tables(lens, P, 15)
    cu = _cu(counts)
    q, k, v, cos, sin = _append_inputs(cu[-1], H, Hq, D, D, True, 15, max(lens))
    cache = _random_cache(pages, H, P, D, 15)
    before = _cpu({n: t.clone() for n, t in cache.items()})
    q_out = mhc.kv_append(cache, k, v, _i32(rows), _i32(lens), _i32(cu), q=q, cos=cos, sin=sin)
    check_append(before, _cpu(cache), k.cpu(), v.cpu(), rows, lens, cu, cos.cpu(), sin.cpu(), False, q.cpu(), q_out.cpu())
    got = mhc.kv_attend(q_out, cache, _i32(rows), _i32(lens), _i32(cu), return_lse=True)
    check_attend(got, q_out, cache, rows, lens, cu, D ** -0.5)


# ------------------------------------------------------------ sharp softmax ---

@pytest.mark.parametrize("case", [(64, 16, 1, 3, None, [70, 900]), (128, 64, 2, 4, None, [5000]), (64, 32, 2, 32, None, [300, 64]),
                                  (128, 16, 1, 16, None, [2000]), (64, 32, 1, 40, [3, 7], [3001, 100]),
                                  (128, 32, 2, 10, [200, 9], [400, 30])])
@pytest.mark.parametrize("scale,q_log2,k_log2", [(None, 0, 20), (1e7, 0, 0), (1e18, 0, 0), (None, 40, 0), (1e7, 20, -20), (3.0, 0, 60)])
def test_attend_sharp_logits(case, scale, q_log2, k_log2):
    """Logits of 2^23 to 2^70, where one step of fp32 is a logit's whole
    difference: the key with the largest, or, within a few steps of fp32 of
    it, a mean of such keys."""
    D, P, H, Hq, counts, lens = case

    def fill(q, cache, rows):
        q *= 2.0 ** q_log2
        cache["k_scale"].mul_(2.0 ** (k_log2 + 4))
    got, (q, cache, rows, lens, cu, s) = _attend(case, 630, scale, fill=fill)
    assert got["out"].isfinite().all()
    check_attend(got, q, cache, rows, lens, cu, float(torch.tensor(s, dtype=torch.float32)))
    T, G = q.shape[0], Hq // H
    clear = 0
    for b, (n, t0, t1) in enumerate(zip(lens, cu or range(T), cu[1:] if cu else range(1, T + 1))):
        pages = torch.tensor(rows[b][:-(-n // P)], device="cuda")
        for t in range(t0, t1):
            for h in range(Hq):
                k, v = (cache[c][pages, h // G].double().mul(cache[c + "_scale"][pages, h // G].double()[:, None, None])
                        .reshape(-1, D)[:n - (t1 - 1 - t)] for c in ("k", "v"))
                x = k @ q[t, h].double() * s
                two = x.topk(min(2, len(x))).values
                off = 2.0 ** -18 * (k.abs() @ q[t, h].double().abs() * s).max()
                if len(two) == 1 or two[0] - two[1] > 2 * off + 40:             # beyond rounding: the one key's values
                    clear += 1
                    assert ((got["out"][t, h].double() - v[x.argmax()]).abs() <= 2.0 ** -8 * v[x.argmax()].abs()).all()
    assert clear > 0
