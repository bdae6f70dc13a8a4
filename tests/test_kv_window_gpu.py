"""GPU checks of mhc_kv_attend_window: a sliding window and first keys that
stay visible, through the binding, against a plain 64-bit form."""
import math

import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from kv_reference import dequantised, spans

pytestmark = pytest.mark.gpu

INDEX_ERROR = 5


@pytest.fixture(autouse=True)
def _status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mhc.load_library()
    assert mhc.device_status() == 0
    yield
    assert mhc.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sees(p, n, window, sinks):
    """Mask over n keys of those that the token at position p sees."""
    j = torch.arange(n, device="cuda")
    return (j <= p) & ((j > p - window) | (j < sinks))


def pages_seen(counts, lens, P, window, sinks):
    """For each sequence the pages of which a new token sees a key, from the definition."""
    got = []
    for m, n in zip(counts, lens):
        s = set()
        for p in range(max(0, n - m), n):
            for i in range(p // P + 1):
                if i * P < sinks or (i + 1) * P > p - window + 1:
                    s.add(i)
        got.append(s)
    return got


def reference(q, cache, rows, lens, cu, scale, window, sinks):
    """out, lse in 64 bits and the bounds of their errors, which are those of
    kv_reference.attend: 2^-8 |out| + (2^-10 + 2^-18 S) A, with A the weighted sum
    of |v| and S the largest sum of |q_i k_i| * scale over the row's keys; and for
    each key 2^-26 of the largest value scale, as the header states it: a weight
    below f16's normal numbers is off by 2^-35 of the row's largest, a code is
    at most 448 < 2^9."""
    T, Hq, D = q.shape
    H, P = cache["k"].shape[1:3]
    G = Hq // H
    K, V = dequantised(cache, "k"), dequantised(cache, "v")
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, r0, r1, first in spans(lens, cu, T):
        n = lens[b]
        if n == 0 or r1 == r0:
            continue
        for t in range(r0, r1):
            p = first + t - r0
            if p < 0:
                continue
            j = sees(p, n, window, sinks).nonzero()[:, 0]
            page = torch.tensor(rows[b], device="cuda")[j // P]
            x = q[t].double().view(H, G, D)
            k, v = K[page, :, j % P].transpose(0, 1), V[page, :, j % P].transpose(0, 1)      # [H, keys, D]
            s = x @ k.transpose(1, 2) * scale
            S = (x.abs() @ k.abs().transpose(1, 2) * scale).amax(-1)
            l = torch.logsumexp(s, -1)
            w = (s - l[..., None]).exp()
            o, A = w @ v, w @ v.abs()
            out[t], lse[t] = o.reshape(Hq, D), l.reshape(Hq)
            far = len(j) * 2.0 ** -26 * cache["v_scale"][page].double().amax(0)[:, None, None]
            tol[t] = (2.0 ** -8 * o.abs() + (2.0 ** -10 + 2.0 ** -18 * S[..., None]) * A + far).reshape(Hq, D)
            tol_lse[t] = (2.0 ** -20 * (S + 1 + l.abs())).reshape(Hq)
    return out, lse, tol, tol_lse


def check(got, *of):
    out, lse, tol, tol_lse = reference(*of)
    o, l = got["out"].double(), got["lse"].double()
    bad = ~(((o - out).abs() <= tol) | (o.isnan() & out.isnan()))
    assert not bad.any(), (bad.nonzero()[:4].tolist(), o[bad][:4].tolist(), out[bad][:4].tolist())
    ok = ((l - lse).abs() <= tol_lse) | (l == lse) | (l.isnan() & lse.isnan())
    assert ok.all(), ((~ok).nonzero()[:4].tolist(), l[~ok][:4].tolist(), lse[~ok][:4].tolist())


def make(case, seed, absent=-1, powers=True):
    """Cache, tables and queries.  Pages that no new token sees are absent
    (``absent`` in the table); slots past the sequences' ends and keys that no
    token sees, in pages that some do, are NaN."""
    D, P, H, Hq, counts, lens, window, sinks = case
    counts_ = counts or [1] * len(lens)
    seen = pages_seen(counts_, lens, P, window, sinks)
    width = max(1, max(-(-n // P) for n in lens))
    total = sum(len(s) for s in seen) + 2
    order = iter(torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist())
    rows = [[next(order) if i in s else absent for i in range(width)] for s in seen]
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = mhc.kv_cache(total, H, P, D)
    for n in ("k", "v"):
        cache[n].copy_((torch.randn(total, H, P, D, generator=g, device="cuda").clamp(-6, 6) * 64).to(torch.float8_e4m3fn))
        s = torch.randint(-8, -4, (total, H), generator=g, device="cuda").float().exp2()
        cache[n + "_scale"].copy_(s if powers else s * (1 + torch.rand(total, H, generator=g, device="cuda")))
    for row, there, m, n in zip(rows, seen, counts_, lens):
        use = torch.zeros(width * P, dtype=torch.bool, device="cuda")
        first = max(0, n - m)
        if n > first:
            use[:n] |= torch.arange(n, device="cuda") < min(sinks, n)
            use[max(0, first - window + 1):n] = True
        for i, page in enumerate(row):
            if i in there:
                for c in ("k", "v"):
                    cache[c].view(torch.uint8)[page, :, ~use[i * P:(i + 1) * P]] = 0x7F
    cu = None
    if counts is not None:
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
    T = len(lens) if cu is None else cu[-1]
    q = torch.randn(T, Hq + 2, D, generator=g, device="cuda").bfloat16()[:, 1:-1]         # rows with a stride
    return q, cache, rows, lens, cu, window, sinks


def attend(made, scale=None, **kw):
    q, cache, rows, lens, cu, window, sinks = made
    return mhc.kv_attend(q, cache, _i32(rows), _i32(lens), None if cu is None else _i32(cu), softmax_scale=scale,
                         window=window, sinks=sinks, return_lse=True, **kw)


def of(made, scale=None):
    q, cache, rows, lens, cu, window, sinks = made
    return q, cache, rows, lens, cu, q.shape[2] ** -0.5 if scale is None else scale, window, sinks


CASES = [
    # D, P, H, Hq, new tokens (None: one each), lengths, window, sinks
    (128, 64, 8, 40, None, [1], 1, 0),
    (128, 64, 8, 40, None, [1000], 100, 4),
    (128, 64, 2, 2, None, [1, 63, 64, 65, 0, 127, 128, 129, 500], 64, 0),
    (64, 16, 4, 16, None, [15, 16, 17, 31, 32, 33, 0, 0, 257], 17, 3),
    (64, 32, 1, 7, None, [2049, 3, 900], 500, 40),
    (128, 128, 1, 16, None, [4097, 1], 1000, 129),
    (128, 32, 2, 8, None, [700, 33, 5000], 1, 0),                      # every token itself alone
    (128, 32, 2, 8, None, [700, 33, 5000], 1, 1),
    (64, 16, 2, 4, None, [900, 40], 3, 700),                           # more first keys than the window
    (128, 16, 3, 9, [4, 1, 3, 0, 2], [40, 1, 3, 17, 300], 5, 2),
    (128, 32, 2, 32, [4, 4, 4], [100, 4, 2], 20, 0),                   # rows without keys
    (64, 64, 2, 2, [70, 1], [70, 900], 33, 5),
    (64, 16, 2, 10, [33], [50], 7, 1),
    (128, 64, 1, 5, [150, 40], [150, 3000], 64, 0),
    (128, 128, 2, 6, [129, 64], [200, 6400], 200, 16),
    (64, 128, 1, 1, [260], [260], 1, 0),
    (64, 128, 1, 1, [300], [2000], 100, 0),
    (128, 16, 1, 128, [3], [90], 30, 4),
    (128, 64, 1, 40, [65, 0, 200], [65, 10, 1900], 128, 128),
    (64, 32, 1, 64, None, [77, 5, 5000], 300, 33),
    (128, 16, 2, 64, [4, 3], [5000, 130], 777, 20),                    # 128 and 129 rows, long
    (64, 64, 1, 43, [3, 3], [3001, 64], 1024, 0),
    (64, 16, 1, 2, [600], [1000], 450, 17),
    (128, 64, 2, 10, [700], [5000], 1024, 4),
    (128, 64, 2, 80, None, [700, 33, 1, 0], 8, 2),                     # many rows, few keys: the one-token kernel
    (64, 16, 1, 60, None, [300, 64, 41], 40, 5),
    (128, 32, 1, 22, [4, 2, 0], [300, 2, 77], 60, 0),
    (128, 64, 2, 80, None, [1700, 33, 1, 0], 300, 2),                  # and many keys: the other
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend_window_is_its_definition(case):
    made = make(CASES[case], case)
    check(attend(made), *of(made))


@pytest.mark.parametrize("case", [1, 3, 8, 9, 13, 18])
@pytest.mark.parametrize("scale", [0.0, 1.5])
def test_flat_and_sharp(case, scale):
    made = make(CASES[case], 100 + case, powers=False)
    check(attend(made, scale), *of(made, scale))


@pytest.mark.parametrize("absent", [-1, 1 << 30, -(1 << 31), 0])
@pytest.mark.parametrize("case", [1, 4, 5, 14, 18])
def test_absent_pages_are_not_looked_at(case, absent):
    """Whatever their place in the table holds, somebody else's page among it: same bits, nothing reported."""
    a, b = make(CASES[case], 200 + case), make(CASES[case], 200 + case, absent)
    x, y = attend(a), attend(b)
    assert torch.equal(x["out"], y["out"]) and torch.equal(x["lse"], y["lse"])


@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if CASES[c][4] or max(CASES[c][5]) < 1200])
def test_wide_windows_are_the_call_without_one(case):
    """A window, or first keys, of all there are: the bits of the call without a window."""
    D, P, H, Hq, counts, lens, _, _ = CASES[case]
    for window, sinks in ((1 << 40, 0), (1, 1 << 40), (max(lens) + P, 3)):
        made = make((D, P, H, Hq, counts, lens, window, sinks), 300 + case)
        q, cache, rows, lens, cu, _, _ = made
        plain = mhc.kv_attend(q, cache, _i32(rows), _i32(lens), None if cu is None else _i32(cu), return_lse=True)
        got = attend(made)
        assert torch.equal(got["out"], plain["out"]) and torch.equal(got["lse"], plain["lse"])


@pytest.mark.parametrize("case", [(128, 64, 2, 4, None, [300, 70], 128, 0), (128, 64, 1, 40, [30], [400], 256, 0),
                                  (64, 16, 1, 64, [5, 3], [333, 60], 250, 7)])
def test_windows_just_longer_than_the_sequence(case):
    """Wide enough for the lengths, not for the table: through the window's kernels, to the definition without one."""
    D, P, H, Hq, counts, lens, window, sinks = case
    made = make((D, P, H, Hq, counts, lens, max(lens), sinks), 320)
    q, cache, rows, lens, cu, w, s = made
    rows = [r + [-1] * 9 for r in rows]                                # a wider table
    check(attend((q, cache, rows, lens, cu, w, s)), *of((q, cache, rows, lens, cu, 1 << 20, 0)))


NANS = [(128, 16, 2, 4, [40, 3], [90, 60], 20, 3), (64, 16, 1, 40, [20, 2], [200, 77], 33, 5), (128, 64, 1, 5, [90], [300], 100, 0),
        (64, 32, 1, 2, [300], [700], 64, 40), (128, 32, 1, 48, [9], [200], 4, 2), (64, 64, 2, 2, [6], [150], 3, 0)]


@pytest.mark.parametrize("case", NANS)
def test_nan_values_reach_the_rows_that_see_them(case):
    """NaN in a few dims of values at both ends of the windows and among the
    first keys: NaN in those dims of the rows that see them, no other number changes."""
    D, P, H, Hq, counts, lens, window, sinks = case
    made, clean = make(case, 400), make(case, 400)
    q, cache, rows, _, cu, _, _ = made
    put = []
    for b, (m, n) in enumerate(zip(counts, lens)):
        for j in {0, sinks - 1, sinks, n - m - window, n - m - window + 1, n - m - window + 3, n - m, n - m // 2, n - 2, n - 1,
                  n - window, n - m + 1 - window + m // 2}:
            if 0 <= j < n and rows[b][j // P] >= 0:
                d = (7 * j + 3) % D
                for k, c in enumerate((cache, clean[1])):
                    c["v"].view(torch.uint8)[rows[b][j // P], j % H, j % P, d] = 0x38 if k else (0x7F if j % 2 else 0xFF)
                put.append((b, j, j % H, d))
    got, expect = attend(made), attend(clean)
    check(expect, *of(clean))
    nan = torch.zeros_like(got["out"], dtype=torch.bool)
    G = Hq // H
    for b, j, h, d in put:
        for t in range(cu[b], cu[b + 1]):
            p = lens[b] - (cu[b + 1] - t)
            if p >= 0 and j <= p and (j > p - window or j < sinks):
                nan[t, h * G:(h + 1) * G, d] = True
    assert nan.any() and not nan.all(-1).any()
    assert torch.equal(got["out"].isnan(), nan)
    assert torch.equal(got["out"][~nan], expect["out"][~nan]) and torch.equal(got["lse"], expect["lse"])


@pytest.mark.parametrize("case", NANS[:3])
def test_nan_keys_stay_with_the_rows_that_see_them(case):
    """A key that is NaN is one in every product: rows that see it are NaN, the others as without it."""
    D, P, H, Hq, counts, lens, window, sinks = case
    made, clean = make(case, 420), make(case, 420)
    q, cache, rows, _, cu, _, _ = made
    n, m = lens[0], counts[0]
    j = n - m - window + 1 + m // 2                                   # the windows of the first half of the tokens
    cache["k"].view(torch.uint8)[rows[0][j // P], :, j % P] = 0x7F
    clean[1]["k"].view(torch.uint8)[rows[0][j // P], :, j % P] = 0x38
    got, expect = attend(made), attend(clean)
    see = [t for t in range(m) if n - m + t - window < j <= n - m + t]
    rest = [t for t in range(cu[-1]) if t not in see]
    assert 0 < len(see) < m
    assert got["out"][see].isnan().all() and got["lse"][see].isnan().all()
    assert torch.equal(got["out"][rest], expect["out"][rest]) and torch.equal(got["lse"][rest], expect["lse"][rest])


def test_infinite_queries():
    for Hq in (2, 40):
        made = make((128, 16, 1, Hq, [6, 4], [3, 400], 50, 3), 430)
        made[0][0], made[0][7, 0, 5] = math.inf, -math.inf
        got = attend(made)
        assert (got["out"][:3] == 0).all() and (got["lse"][:3] == -math.inf).all()       # rows without keys
        assert got["out"][7, 0].isnan().all() and got["lse"][7, 0].isnan()
        got["out"][7, 0], got["lse"][7, 0], made[0][7, 0], made[0][:3] = 0, 0, 0, 0
        assert got["out"].isfinite().all()


@pytest.mark.parametrize("case", [1, 4, 9, 14, 19, 22])
def test_deterministic(case):
    a, b = attend(make(CASES[case], case)), attend(make(CASES[case], case))
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("case", [(128, 64, 1, 5, None, [131071, 40000, 3], 4096, 4), (64, 32, 2, 66, [2], [30001], 5000, 4),
                                  (64, 64, 1, 7, None, [60000], 20000, 300)])
def test_long_contexts(case):
    made = make(case, 440)
    check(attend(made), *of(made))


@pytest.mark.parametrize("Hq,window", [(2, 40), (16, 40), (48, 40), (48, 500)])
@pytest.mark.parametrize("B", [33, 300])
def test_many_sequences(B, Hq, window):
    made = make((64, 16, 1, Hq, None, [(i * 29) % (5 * window) for i in range(B)], window, 5), 450)
    check(attend(made), *of(made))


def test_bad_pages_that_are_seen_are_reported():
    made = make((128, 16, 2, 8, None, [400, 300, 90], 50, 3), 460)
    q, cache, rows, lens, cu, w, s = made
    good = attend(made)
    for Hq in (8, 80):
        bad = [list(r) for r in rows]
        bad[1][299 // 16] = cache["k"].shape[0]
        x = q if Hq == 8 else q.repeat(1, 10, 1)
        got = attend((x, cache, bad, lens, cu, w, s))
        assert mhc.device_status() == INDEX_ERROR
        bad[1][299 // 16] = rows[1][299 // 16]
        bad[0][0] = -1                                                 # of the first keys
        attend((x, cache, bad, lens, cu, w, s))
        assert mhc.device_status() == INDEX_ERROR
        if Hq == 8:
            assert torch.equal(got["out"][[0, 2]], good["out"][[0, 2]]) and got["out"].isfinite().all()
        attend((x, cache, rows, [400, 300, 1 << 20], cu, w, s))        # a length past the table
        assert mhc.device_status() == INDEX_ERROR


def test_other_stream_graph_and_workspace():
    """On a stream of its own, captured and replayed, with a workspace of any contents: the same bits."""
    made = make((128, 64, 2, 10, None, [3000, 64, 1], 700, 4), 470)
    q, cache, rows, lens, cu, w, s = made
    table, n = _i32(rows), _i32(lens)
    a = attend(made)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = mhc.kv_attend(q, cache, table, n, window=w, sinks=s, return_lse=True, stream=st)
    st.synchronize()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    ws = mhc.kv_workspace_for(cache, 10, 3, 3)
    for fill in (0xFF, 0x7F, 0):
        ws.fill_(fill)
        b = attend(made, workspace=ws)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    out, lse = torch.zeros_like(a["out"]), torch.zeros_like(a["lse"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        mhc.kv_attend(q, cache, table, n, window=w, sinks=s, out=out, lse=lse)
    for _ in range(2):
        out.zero_()
        attend(made)                                                   # the stream's own workspace meanwhile
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], out) and torch.equal(a["lse"], lse)


def test_refusals():
    made = make((64, 16, 2, 4, None, [30], 8, 2), 480)
    q, cache, rows, lens, _, _, _ = made
    for kw, error in ((dict(window=0), mhc.MhcError), (dict(window=-3), mhc.MhcError), (dict(window=4, sinks=-1), mhc.MhcError),
                      (dict(sinks=4), ValueError), (dict(window=2.5), TypeError), (dict(window=4, sinks=None), TypeError)):
        with pytest.raises(error):
            mhc.kv_attend(q, cache, _i32(rows), _i32(lens), **kw)
