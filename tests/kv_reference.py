"""Plain 64-bit forms of mhc_kv_append and mhc_kv_attend, written from their
definitions in include/mhc_kv.h, one sequence, head and page at a time."""
import math

import torch

E4M3_MAX = 448.0


def e4m3_round(x):
    """Nearest e4m3 number (ties to even) of float64 x with |x| <= 464: three
    bits after the leading one, exponents from -6; NaN where x is not finite."""
    _, e = torch.frexp(x.abs())
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    y = torch.round(x / step) * step
    return torch.where(x.isfinite(), y, math.nan)


def need(amax):
    """Smallest 2^e with amax <= 448 * 2^e, e >= -116, of a Python float."""
    e = -116
    if amax > 0:
        e = max(e, math.frexp(amax / E4M3_MAX)[1] - 1)
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def spans(seq_lens, cu_q, T):
    """(sequence, its first row, position of that row) of a call."""
    B = len(seq_lens)
    cu = cu_q if cu_q is not None else list(range(B + 1))
    return [(b, cu[b], cu[b + 1], seq_lens[b] - (cu[b + 1] - cu[b])) for b in range(B)]


def rotated(x, pos, cos, sin, interleaved):
    """x [heads, D] float64 of the token at pos, and the size of the terms
    that each element is the sum of."""
    if cos is None or pos < 0:
        return x.clone(), x.abs()
    half = cos.shape[1]
    c, s = cos[pos].double(), sin[pos].double()
    y, a = x.clone(), x.abs()
    for i in range(half):
        p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, p] = x[:, p] * c[i] - x[:, r] * s[i]
        y[:, r] = x[:, r] * c[i] + x[:, p] * s[i]
        a[:, p] = (x[:, p] * c[i]).abs() + (x[:, r] * s[i]).abs()
        a[:, r] = (x[:, r] * c[i]).abs() + (x[:, p] * s[i]).abs()
    return y, a


def dequantised(cache, name):
    return cache[name].double() * cache[name + "_scale"].double()[:, :, None, None]


def check_append(before, after, k, v, block_table, seq_lens, cu_q, cos=None, sin=None, interleaved=False, q=None,
                 q_out=None):
    """Hold a cache after the call (CPU tensors) to its definition.

    Bounds, from the roundings: a rotated number is a difference of two fp32
    products, so off by at most 3 * 2^-24 of its terms; a code is off by half
    a step, 2^-4 of its value (or half the subnormal step, 2^-10); q_out by
    2^-8 of its value.  v is not rotated, so its codes and scales are exact.
    """
    T = k.shape[0]
    P = before["k"].shape[2]
    expect = {n: before[n].double() for n in ("k", "v")}
    scale = {n: before[n + "_scale"].double().clone() for n in ("k", "v")}
    touched = torch.zeros(before["k"].shape[0], P, dtype=torch.bool)
    off = torch.zeros_like(expect["k"])                 # by how much k's numbers may be off before rounding
    for b, r0, r1, first in spans(seq_lens, cu_q, T):
        t = r0
        while t < r1:
            pos = first + t - r0
            if pos < 0:
                if q is not None:
                    assert torch.equal(q_out[t].view(torch.int16), q[t].view(torch.int16))
                t += 1
                continue
            page, slot = block_table[b][pos // P], pos % P
            n = min(P - slot, r1 - t)
            for name, src in (("k", k), ("v", v)):
                rows, terms = [], []
                for i in range(n):
                    x = src[t + i].double()
                    y, a = rotated(x, pos + i, cos, sin, interleaved) if name == "k" else (x, x.abs())
                    rows.append(y)
                    terms.append(a)
                y, a = torch.stack(rows, 1), torch.stack(terms, 1)     # [heads, n, D]
                err = 3 * 2.0 ** -24 * a if name == "k" and cos is not None else torch.zeros_like(a)
                got = after[name + "_scale"][page].double()
                for h in range(y.shape[0]):
                    m = torch.where(y[h].isfinite(), y[h].abs(), 0.0)
                    top = m.max().item()
                    slack = err[h].max().item() if name == "k" else 0.0
                    slack = slack if math.isfinite(slack) else 0.0
                    old = scale[name][page, h].item() if slot else 0.0
                    allowed = {max(old, need(top)), max(old, need(max(0.0, top - slack))), max(old, need(top + slack))}
                    assert got[h].item() in allowed, (name, page, h, got[h].item(), allowed)
                    if slot:
                        keep = expect[name][page, h, :slot] * (old / got[h])
                        expect[name][page, h, :slot] = keep if got[h] == old else e4m3_round(keep)
                    scale[name][page, h] = got[h]
                expect[name][page, :, slot:slot + n] = y / got[:, None, None]
                if name == "k":
                    off[page, :, slot:slot + n] = err / got[:, None, None]
            touched[page, slot:slot + n] = True
            if q is not None:
                for i in range(n):
                    y, a = rotated(q[t + i].double(), pos + i, cos, sin, interleaved)
                    d = (q_out[t + i].double() - y).abs()
                    assert (d <= 2.0 ** -8 * y.abs() + 3 * 2.0 ** -24 * a).all()
            t += n
    for name in ("k", "v"):
        assert torch.equal(after[name + "_scale"].double(), scale[name])
        got = after[name].double()
        stay = ~touched[:, None, :, None].expand_as(got)
        same = (got == expect[name]) | (got.isnan() & expect[name].isnan())
        assert same[stay].all(), name                   # older slots, re-rounded or not, and unused ones
        new = ~stay
        e = expect[name][new]
        exact = e4m3_round(e)
        if name == "v":
            ok = (got[new] == exact) | (got[new].isnan() & exact.isnan())
        else:
            half = torch.maximum(2.0 ** -4 * e.abs(), torch.full_like(e, 2.0 ** -10))
            ok = ((got[new] - e).abs() <= half + off[new]) | (got[new].isnan() & exact.isnan())
        assert ok.all(), name


def attend(q, cache, block_table, seq_lens, cu_q, softmax_scale):
    """out, lse in float64, and the bounds of their errors.

    The kernels hold logits and sums in fp32 and the weights exp(s - max) in
    f16 or better.  With S the largest sum of |q_i k_i| * softmax_scale of a
    row, a logit is off by 2^-20 S at most (128 terms of 2^-24, the scales and
    the exponential's argument); a weight by twice that and f16's 2^-11
    (relative); the sums' own roundings are below 2^-14 of what they add up.
    With A = sum_j p_j |v_j|: |out error| <= 2^-8 |out| + (2^-10 + 2^-18 S) A.
    """
    T, Hq, D = q.shape
    H, P = cache["k"].shape[1:3]
    G = Hq // H
    K, V = dequantised(cache, "k"), dequantised(cache, "v")
    dev = q.device
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    for b, r0, r1, first in spans(seq_lens, cu_q, T):
        n = seq_lens[b]
        if n == 0 or r1 == r0:
            continue
        pages = torch.tensor(block_table[b][:-(-n // P)], device=dev)
        for h in range(H):
            k, v = K[pages, h].reshape(-1, D)[:n], V[pages, h].reshape(-1, D)[:n]
            for t in range(r0, r1):
                keys = first + t - r0 + 1
                if keys <= 0:
                    continue
                x = q[t, h * G:(h + 1) * G].double()
                s = x @ k[:keys].T * softmax_scale
                S = (x.abs() @ k[:keys].abs().T * softmax_scale).amax(1)
                l = torch.logsumexp(s, 1)
                p = (s - l[:, None]).exp()
                o = p @ v[:keys]
                A = p @ v[:keys].abs()
                out[t, h * G:(h + 1) * G], lse[t, h * G:(h + 1) * G] = o, l
                tol[t, h * G:(h + 1) * G] = 2.0 ** -8 * o.abs() + (2.0 ** -10 + 2.0 ** -18 * S[:, None]) * A
                tol_lse[t, h * G:(h + 1) * G] = 2.0 ** -20 * (S + 1 + l.abs())
    return out, lse, tol, tol_lse


def check_attend(got, q, cache, block_table, seq_lens, cu_q, softmax_scale):
    out, lse, tol, tol_lse = attend(q, cache, block_table, seq_lens, cu_q, softmax_scale)
    o = got["out"].double()
    bad = ~(((o - out).abs() <= tol) | (o.isnan() & out.isnan()))
    assert not bad.any(), (bad.nonzero()[:4].tolist(), o[bad][:4].tolist(), out[bad][:4].tolist())
    if "lse" in got:
        l = got["lse"].double()
        ok = ((l - lse).abs() <= tol_lse) | (l == lse) | (l.isnan() & lse.isnan())
        assert ok.all(), ((~ok).nonzero()[:4].tolist(), l[~ok][:4].tolist(), lse[~ok][:4].tolist())
