"""GPU checks of mhc_kv_append_norm: norms of queries and keys, head by head,
before the rotation and in the same call."""
import math

import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc
from kv_reference import e4m3_round, need, rotated, spans

pytestmark = pytest.mark.gpu

INDEX_ERROR = 5
# A normed number's error, relative: 8 pairs of products and 3 sums of positive terms (19 roundings of 2^-24, halved by
# the root), the mean's (1, halved), the reciprocal root (2 steps, 4 x 2^-24) and two products: below 16 x 2^-24.
NORM_ERR = 2.0 ** -20


@pytest.fixture(autouse=True)
def _status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mhc.load_library()
    assert mhc.device_status() == 0
    yield
    assert mhc.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bytes(cache):
    return {n: t.clone().view(torch.uint8) for n, t in cache.items()}


def normed(x, weight, eps):
    """x [T, heads, D] in 64 bits, from the definition; weight None: as it is."""
    x = x.double()
    if weight is None:
        return x
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def check(before, after, q, k, v, q_out, q_norm, k_norm, eps, rows, lens, cu, cos, sin, inter):
    """Hold the call to its definition (CPU tensors).

    Normed and rotated numbers are off by NORM_ERR of their terms (none without
    a norm) and 3 * 2^-24 of them (see kv_reference.check_append); q_out is rounded
    to bf16 (2^-8), a code to e4m3 (2^-4 of its value, or 2^-10 scale steps)."""
    P, T = before["k"].shape[2], k.shape[0]
    nq, nk = (None if q is None else normed(q, q_norm, eps)), normed(k, k_norm, eps)
    eq, ek = (0.0 if n is None else NORM_ERR for n in (q_norm, k_norm))
    touched = torch.zeros(before["k"].shape[0], P, dtype=torch.bool)
    for b, r0, r1, first in spans(lens, cu, T):
        t = r0
        while t < r1:
            pos = first + t - r0
            if pos < 0:
                if q is not None:
                    assert torch.equal(q_out[t].view(torch.int16), q[t].view(torch.int16))
                t += 1
                continue
            page, slot = rows[b][pos // P], pos % P
            n = min(P - slot, r1 - t)
            for name in ("k", "v"):
                y, a = zip(*(rotated(nk[t + i], pos + i, cos, sin, inter) if name == "k"
                             else (v[t + i].double(), v[t + i].double().abs()) for i in range(n)))
                y, a = torch.stack(y, 1), torch.stack(a, 1)                 # [heads, n, D]
                err = ((ek + 3 * 2.0 ** -24) * a if name == "k" else torch.zeros_like(a)).nan_to_num(0, 0, 0)
                scale = after[name + "_scale"][page].double()
                for h in range(y.shape[0]):
                    top = torch.where(y[h].isfinite(), y[h].abs(), 0.0).max().item()
                    slack = err[h].max().item()
                    old = before[name + "_scale"][page, h].double().item() if slot else 0.0
                    allowed = {max(old, need(max(0.0, top + s))) for s in (-slack, 0.0, slack)}
                    assert scale[h].item() in allowed, (name, page, h, scale[h].item(), allowed)
                    if slot:
                        was = before[name][page, h, :slot].double()
                        keep = was if old == scale[h] else e4m3_round(was * (old / scale[h]))
                        now = after[name][page, h, :slot].double()
                        assert ((now == keep) | (now.isnan() & keep.isnan())).all()
                e, got = y / scale[:, None, None], after[name][page, :, slot:slot + n].double()
                half = torch.maximum(2.0 ** -4 * e.abs(), torch.full_like(e, 2.0 ** -10)) + err / scale[:, None, None]
                ok = ((got - e).abs() <= half) | (got.isnan() & ~e.isfinite())
                if name == "v":
                    exact = e4m3_round(e)
                    ok = (got == exact) | (got.isnan() & exact.isnan())
                assert ok.all(), (name, page)
            touched[page, slot:slot + n] = True
            if q is not None:
                for i in range(n):
                    y, a = rotated(nq[t + i], pos + i, cos, sin, inter)
                    o = q_out[t + i].double()
                    ok = ((o - y).abs() <= 2.0 ** -8 * y.abs() + 1.01 * (eq + 3 * 2.0 ** -24) * a) | (o.isnan() & y.isnan())
                    assert ok.all(), (t + i, (o - y).abs().max())
            t += n
    for name in ("k", "v"):                       # slots after the new ones and pages without any keep their bytes
        fresh = ~touched & ~(touched.flip(1).cumsum(1).flip(1) > 0)
        a, w = after[name].view(torch.uint8).transpose(1, 2), before[name].view(torch.uint8).transpose(1, 2)
        assert torch.equal(a[fresh], w[fresh])


# D, P, H, Hq, new tokens of each sequence (None: one each), lengths, R, interleaved, norms, weights for each head
CASES = [
    (128, 64, 8, 40, None, [1], 128, False, "qk", False),
    (128, 64, 8, 40, None, [64, 65, 1, 130, 0, 63], 128, False, "qk", False),
    (128, 16, 2, 2, [3, 0, 17, 1], [3, 5, 40, 33], 64, True, "qk", True),
    (64, 16, 3, 9, [16, 1, 15], [16, 17, 47], 64, False, "qk", True),
    (64, 32, 1, 5, [100], [101], 32, True, "k", False),
    (64, 128, 2, 16, [300, 5], [301, 6], 16, False, "q", True),
    (128, 128, 4, 4, [257, 128, 1], [300, 128, 129], 128, True, "qk", False),
    (128, 32, 2, 8, [5, 4], [3, 4], 128, False, "qk", True),              # more new tokens than places
    (64, 64, 4, 8, [70], [200], 0, False, "qk", False),
    (128, 16, 1, 1, [1] * 45 + [2], [20] * 46, 128, False, "qk", False),
    (64, 16, 1, 1, [2] * 70, list(range(2, 72)), 64, True, "k", True),
    (128, 64, 2, 6, [2500], [2533], 128, False, "qk", True),              # from 2048 tokens a warp takes all heads
]


def _make(case, seed):
    D, P, H, Hq, counts, lens, R, inter, norms, each = CASES[case] if isinstance(case, int) else case
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu = [0]
    for n in counts or [1] * len(lens):
        cu.append(cu[-1] + n)
    T = cu[-1]
    used = [-(-n // P) for n in lens]
    order = torch.randperm(sum(used) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
    rows, at = [], 0
    for n in used:
        rows.append(order[at:at + n] + [-7] * (max(1, max(used)) - n))
        at += n
    cache = mhc.kv_cache(len(order), H, P, D)
    for n in ("k", "v"):
        cache[n].copy_((torch.randn(cache[n].shape, generator=g, device="cuda") * 64).to(torch.float8_e4m3fn))
        cache[n + "_scale"].copy_(torch.randint(-12, -6, cache[n + "_scale"].shape, generator=g, device="cuda").float().exp2())
    x = torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda")
    x *= torch.rand(T, Hq + 2 * H, 1, generator=g, device="cuda").mul(16).sub(8).exp2()          # every head its own size
    q, k, v = x.bfloat16().split([Hq, H, H], dim=1)
    cos = sin = None
    if R:
        angle = torch.rand(max(lens) + 1, R // 2, generator=g, device="cuda") * 6.3
        cos, sin = angle.cos(), angle.sin()

    def weight(heads, on):
        shape = (heads, D) if each else (D,)
        return (1 + 0.3 * torch.randn(shape, generator=g, device="cuda")).bfloat16() if on else None
    return dict(cache=cache, k=k, v=v, rows=rows, lens=lens, cu=None if counts is None else cu, q=q, cos=cos, sin=sin,
                inter=inter, q_norm=weight(Hq, "q" in norms), k_norm=weight(H, "k" in norms))


def _run(m, eps=1e-6, **kw):
    a = dict(q=m["q"], cos=m["cos"], sin=m["sin"], interleaved=m["inter"], q_norm=m["q_norm"], k_norm=m["k_norm"], norm_eps=eps)
    a.update(kw)
    return mhc.kv_append(m["cache"], m["k"], m["v"], _i32(m["rows"]), _i32(m["lens"]),
                         None if m["cu"] is None else _i32(m["cu"]), **a)


def _check(m, before, q_out, eps=1e-6):
    c = lambda t: None if t is None else t.cpu()  # noqa: E731
    check(before, {n: t.cpu() for n, t in m["cache"].items()}, c(m["q"]), c(m["k"]), c(m["v"]), c(q_out), c(m["q_norm"]),
          c(m["k_norm"]), eps, m["rows"], m["lens"], m["cu"], c(m["cos"]), c(m["sin"]), m["inter"])


def _before(m):
    return {n: t.cpu() for n, t in m["cache"].items()}


@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_norm_is_its_definition(case):
    m = _make(case, case)
    before = _before(m)
    _check(m, before, _run(m))


@pytest.mark.parametrize("eps", [1e-20, 1e-5, 0.5, 1e6])
def test_epsilons(eps):
    m = _make(2, 50)
    before = _before(m)
    _check(m, before, _run(m, eps), eps)


@pytest.mark.parametrize("case", [1, 4, 7])
def test_large_small_and_zero_heads(case):
    """Squares beyond fp32's largest and below its smallest number, and heads of zeros."""
    m = _make(case, 60 + case)
    for i, by in enumerate([2.0 ** 100, 2.0 ** 64, 2.0 ** -70, 0.0, 1.0, 2.0 ** 119]):
        for n in ("q", "k"):
            x = m[n]
            if i < x.shape[0]:
                x[i] *= by / x[i].float().abs().amax().clamp(min=1e-30).log2().floor().exp2()
    before = _before(m)
    _check(m, before, _run(m))


def test_infinities_and_nan():
    """A head that holds one gives what the formula gives: NaN for NaN, and
    beside an infinity zeros, with NaN in its place.  Other heads do not."""
    m = _make((128, 16, 2, 4, None, [5, 17, 30], 0, False, "qk", False), 70)
    for n in ("q", "k"):
        m[n][0, 0, 3], m[n][1, 1, 7], m[n][2, 0, 0] = math.inf, math.nan, -math.inf
    before = _before(m)
    out = _run(m)
    _check(m, before, out)
    assert out[0, 0, 3].isnan() and (out[0, 0, :3] == 0).all() and out[1, 1].isnan().all()
    assert out[1, 0].isfinite().all() and out[0, 1:].isfinite().all()


def test_without_norm_weights_it_is_the_plain_call():
    a, b = _make(3, 80), _make(3, 80)
    qa, qb = _run(a, q_norm=None, k_norm=None), _run(b, q_norm=None, k_norm=None, norm_eps=0.0)
    assert torch.equal(qa, qb)
    for n, t in _bytes(a["cache"]).items():
        assert torch.equal(t, b["cache"][n].view(torch.uint8))


def test_weights_of_one_head_expanded_strided_and_shared():
    """[D], [heads, D] of equal rows, an expanded view and rows with a stride: the same bits."""
    D = 64
    w = (1 + 0.2 * torch.randn(D, device="cuda")).bfloat16()
    outs = []
    for form in (lambda h: w, lambda h: w.repeat(h, 1), lambda h: w.expand(h, D),
                 lambda h: torch.cat([w.repeat(h, 1), torch.zeros(h, 8, device="cuda").bfloat16()], 1)[:, :D]):
        m = _make((D, 16, 2, 6, [20, 3], [25, 30], D, False, "qk", False), 90)
        m["q_norm"], m["k_norm"] = form(6), form(2)
        outs.append((_run(m), _bytes(m["cache"])))
    for q, c in outs[1:]:
        assert torch.equal(q, outs[0][0])
        assert all(torch.equal(c[n], outs[0][1][n]) for n in c)


def test_in_place_on_a_stream_and_in_a_graph():
    m, e = _make(1, 95), _make(1, 95)
    expect = _run(e)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    table, lens, q0 = _i32(m["rows"]), _i32(m["lens"]), m["q"].clone()
    qo = torch.empty_like(q0)

    def call(stream=None):
        mhc.kv_append(m["cache"], m["k"], m["v"], table, lens, q=m["q"], cos=m["cos"], sin=m["sin"], q_norm=m["q_norm"],
                      k_norm=m["k_norm"], q_out=qo, stream=stream)
    torch.cuda.synchronize()
    call(st)
    st.synchronize()
    assert torch.equal(qo, expect)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for _ in range(2):
        qo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, expect)
    for n, t in _bytes(m["cache"]).items():
        assert torch.equal(t, e["cache"][n].view(torch.uint8))
    got = _run(m, q_out=m["q"])                                # queries in place
    assert got is m["q"] and torch.equal(got, expect)


def test_bad_indices_leave_rows_and_pages_alone():
    m = _make((128, 16, 2, 4, [3, 4, 2], [9, 20, 18], 128, False, "qk", False), 97)
    before = _bytes(m["cache"])
    m["lens"] = [9, 999, 18]
    out = _run(m)
    assert mhc.device_status() == INDEX_ERROR
    assert torch.equal(out[3:7], m["q"][3:7])                  # neither normed nor rotated
    after = _bytes(m["cache"])
    for p in m["rows"][1]:
        if p >= 0:
            assert all(torch.equal(after[n][p], before[n][p]) for n in after)


@pytest.mark.parametrize("counts,lens", [(None, [5, 40, 17]), ([30, 20], [50, 25])])
def test_positions_beyond_the_rotation_are_left_alone(counts, lens):
    """Their tokens are not written, and their queries neither normed nor rotated."""
    m = _make((64, 16, 2, 4, counts, lens, 64, False, "qk", False), 99)
    before = _bytes(m["cache"])
    rows = 18                                                  # positions that the tables have
    out = _run(m, cos=m["cos"][:rows].contiguous(), sin=m["sin"][:rows].contiguous())
    assert mhc.device_status() == INDEX_ERROR
    after = _bytes(m["cache"])
    for b, t0, t1, first in spans(lens, m["cu"], m["k"].shape[0]):
        for t in range(t0, t1):
            p = first + t - t0
            assert torch.equal(out[t], m["q"][t]) == (p >= rows)
            page, slot = m["rows"][b][p // 16], p % 16
            assert torch.equal(after["v"][page, :, slot], before["v"][page, :, slot]) == (p >= rows)


def test_refusals():
    m = _make((64, 16, 2, 4, None, [3, 4], 64, False, "qk", True), 98)
    before = _bytes(m["cache"])

    def refused(error, status=None, **kw):
        with pytest.raises(error) as e:
            _run(m, **kw)
        assert status is None or e.value.status == status
    refused(ValueError, q=None)                                # q_norm without q
    refused(ValueError, q_norm=m["q_norm"][:3])
    refused(ValueError, q_norm=m["q_norm"][:, :32])
    refused(ValueError, k_norm=m["k_norm"].cpu())
    refused(TypeError, k_norm=m["k_norm"].float())
    refused(TypeError, k_norm=3.0)
    refused(ValueError, k_norm=m["k_norm"].t().contiguous().t())
    refused(ValueError, q_norm=m["q_norm"][None])
    for eps in (0.0, -1e-6, 1e-21, math.inf, math.nan):
        refused(mhc.MhcError, 1, norm_eps=eps)
    refused(mhc.MhcError, 1, k_norm=torch.ones(65, device="cuda").bfloat16()[1:])        # not 16-byte aligned
    refused(mhc.MhcError, 1, q_norm=torch.ones(4, 68, device="cuda").bfloat16()[:, :64])  # stride no multiple of 8
    refused(mhc.MhcError, 1, k_norm=m["q"][0, :2], q_out=m["q"])                         # weights that the call writes over
    for n, t in _bytes(m["cache"]).items():
        assert torch.equal(t, before[n])
