"""The operators of a decode step's attention sublayer, as cases to be measured.

Between a seam's pre block and its post block a decoder runs the attention
sublayer.  Two operators carry it next to the projections:

  append  rotates the new tokens' queries and keys by their positions and
          writes keys and values into a paged cache held in 8 bits (e4m3, one
          scale for each page and head);
  attend  is the causal attention of the new tokens over that cache.

``run`` computes them in plain torch operations, or, with ``own`` set, calls
``kv_append`` and ``kv_attend`` of this package.

The cache of one layer is k and v [pages, Hkv, P, D] in e4m3, k_scale and
v_scale [pages, Hkv] fp32.  Sequence b holds its token at position i in page
table[b, i // P], slot i % P.  cu_q [B + 1] says which of the T new tokens
belong to which sequence, lens [B] how many tokens a sequence has with them:
its new tokens take the last positions.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -116            # smallest exponent of a scale: 2**-116 times e4m3's smallest step is a normal fp32


def listed():
    """Head layouts: 40 query heads of 128 make this repository's hidden size
    of 5120; the others are generic.  Token counts run from one to the
    repository's prefill of 16384."""
    return [
        # one user, one token: the launch is what counts
        dict(name="append one token", op="append", B=1, q=1, L=1001, ragged=False, Hq=40, Hkv=8, D=128, P=64,
             R=128, pairs=False, fused=True),
        # a full decode batch, sequences of every length
        dict(name="append decode batch", op="append", B=256, q=1, L=200, ragged=True, Hq=40, Hkv=8, D=128, P=64,
             R=128, pairs=False, fused=True),
        # several prompts at once, odd lengths, half of each head rotated in neighbouring pairs
        dict(name="append prompts", op="append", B=7, q=1500, L=1777, ragged=True, Hq=32, Hkv=4, D=64, P=16,
             R=32, pairs=True, fused=False),
        # one long prompt
        dict(name="append long prompt", op="append", B=1, q=16384, L=16384, ragged=False, Hq=40, Hkv=8, D=128, P=64,
             R=128, pairs=False, fused=True),
        # one user early in a conversation
        dict(name="attend one token", op="attend", B=1, q=1, L=1001, ragged=False, Hq=40, Hkv=8, D=128, P=64),
        # one user with a long document
        dict(name="attend long context", op="attend", B=1, q=1, L=131071, ragged=False, Hq=40, Hkv=8, D=128, P=64),
        # a decode batch of ragged lengths with unused places
        dict(name="attend decode batch", op="attend", B=128, q=1, L=8192, ragged=True, Hq=40, Hkv=8, D=128, P=64),
        # no shared heads, small pages
        dict(name="attend unshared heads", op="attend", B=48, q=1, L=4000, ragged=True, Hq=16, Hkv=16, D=64, P=16),
        # drafted tokens to be verified, many queries to one key head
        dict(name="attend drafted tokens", op="attend", B=32, q=4, L=6000, ragged=True, Hq=32, Hkv=2, D=128, P=32),
        # prompts of odd lengths that begin a conversation
        dict(name="attend prompts", op="attend", B=5, q=1100, L=1100, ragged=True, Hq=32, Hkv=4, D=64, P=32),
        # a chunk of a long prompt after what is cached of it
        dict(name="attend prompt chunk", op="attend", B=1, q=4096, L=16384, ragged=False, Hq=40, Hkv=8, D=128, P=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """Serving traffic over the same ranges: one to 256 sequences, one token
    to long prompts, contexts up to 131071, groups of 1 to 16 query heads."""
    D, P = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * Hkv <= 64])
    c = dict(op=rng.choice(["append", "attend", "attend"]), Hq=G * Hkv, Hkv=Hkv, D=D, P=P, ragged=rng.random() < 0.7)
    kind = rng.choice(["tokens", "tokens", "drafts", "prompts"])
    if kind == "tokens":
        c["B"], c["q"] = _log(rng, 1, 256), 1
    elif kind == "drafts":
        c["B"], c["q"] = _log(rng, 1, 128), rng.randint(2, 16)
    else:
        c["B"] = _log(rng, 1, 8)
        c["q"] = _log(rng, 17, 4096 // c["B"])
    row = Hkv * D * 2                                # bytes a cached token takes
    if c["op"] == "append":
        c["L"] = c["q"] + _log(rng, 1, 300) - 1
        c["R"] = rng.choice([D, D, D // 2, 0])
        c["pairs"], c["fused"] = rng.random() < 0.3, rng.random() < 0.6
    else:
        most = min(131071, int(2e9) // (row * c["B"]))          # 2 GB of cache
        most = min(most, int(1.5e11) // (c["Hq"] * D * c["q"] * c["B"]))   # and less work than the listed chunk
        c["L"] = max(c["q"], _log(rng, 1, max(1, most)))
    return c


def _lengths(case):
    """New tokens and whole lengths of the sequences: the same for every seed."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    q, lens = [], []
    for b in range(case["B"]):
        n, total = case["q"], case["L"]
        if case["ragged"] and b:
            n = max(1, n - r.randint(0, n // 2))
            total = max(n, int(total * r.uniform(0.1, 1.0)))
            if r.random() < 0.03:                    # a place of the batch that nobody uses; a batch
                total = 0                            # of single queries has a row for it all the same
                n = 1 if case["op"] == "attend" and case["q"] == 1 else 0
        q.append(n)
        lens.append(total)
    return q, lens


def _single(case):
    """Whether every sequence has exactly one new token (cu_q is then left out)."""
    return case["q"] == 1 and all(n == 1 for n in _lengths(case)[0])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    q_lens, lens = _lengths(case)
    B, Hq, Hkv, D, P = (case[k] for k in ("B", "Hq", "Hkv", "D", "P"))
    T = sum(q_lens)
    need = [-(-n // P) for n in lens]
    width, pages = max(1, max(need)), sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [order[-1]] * (width - n))
        at += n
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s = {"case": dict(case), "T": T,
         "table": torch.tensor(rows, dtype=torch.int32, device=dev),
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "cu_q": None if _single(case) else torch.tensor(cu, dtype=torch.int32, device=dev)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)

    def codes():
        # what appending normal values leaves: the largest of a page is near 4, so values reach 256
        # times a scale of 2**-6; slots that nothing was written to hold any byte, NaN's among them
        out = torch.empty(pages, Hkv, P, D, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (Hkv * P * D))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            x = torch.randn(n, Hkv, P, D, generator=g, device=dev).clamp_(-6.5, 6.5)
            out[i:i + n] = (x * 64.0).to(torch.float8_e4m3fn).view(torch.uint8)
        for b, n in enumerate(lens):
            if n % P and b < 64:
                out[rows[b][n // P], :, n % P:] = 0x7F
        return out.view(torch.float8_e4m3fn)

    def scales():
        return torch.full((pages, Hkv), 2.0 ** -6, dtype=torch.float32, device=dev)

    s["cache"] = {"k": codes(), "v": codes(), "k_scale": scales(), "v_scale": scales()}
    if case["op"] == "append":
        if case["fused"]:          # the three are slices of one projection's rows
            rowsqkv = normal(T, (Hq + 2 * Hkv) * D)
            s["q"] = rowsqkv[:, :Hq * D].unflatten(1, (Hq, D))
            s["k"] = rowsqkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
            s["v"] = rowsqkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        else:
            s["q"], s["k"], s["v"] = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
        R = case["R"]
        s["cos"] = s["sin"] = None
        if R:
            places = torch.arange(width * P, dtype=torch.float64, device=dev)
            rate = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device=dev) * 2 / R)
            angle = places[:, None] * rate
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    else:
        s["q"] = normal(T, Hq, D)
        # kinds of scales that a cache has after real use: every page and head its own
        for n in ("k_scale", "v_scale"):
            s["cache"][n] *= 2.0 ** torch.randint(-2, 2, (pages, Hkv), generator=g, device=dev).float()
    return s


# ------------------------------------------------------------- plain form ---

def _places(s):
    """Sequence, position and whether it is one of its sequence's, of each new token."""
    T, lens = s["T"], s["lens"].long()
    t = torch.arange(T, device=lens.device)
    if s["cu_q"] is None:
        b, left = t, torch.ones_like(t)
    else:
        cu = s["cu_q"].long()
        b = torch.searchsorted(cu, t, right=True) - 1
        left = cu[b + 1] - t
    return b, lens[b] - left


def _turn(x, cos, sin, pairs):
    """The rotation, each product rounded to fp32 before the sum."""
    R = 2 * cos.shape[-1]
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    c, d = a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]
    y = torch.stack((c, d), -1).flatten(-2) if pairs else torch.cat((c, d), -1)
    return torch.cat((y, x[..., R:]), -1)


def _plain_append(s):
    case, cache = s["case"], s["cache"]
    P = case["P"]
    b, pos = _places(s)
    page, slot = s["table"][b, pos // P].long(), pos % P
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos], s["sin"][pos]
        q, k = _turn(q, cos, sin, case["pairs"]), _turn(k, cos, sin, case["pairs"])
    pages = cache["k"].shape[0]
    first = torch.full((pages,), P, dtype=torch.int64, device=q.device).scatter_reduce(0, page, slot, "amin")
    out = {"q": q.to(torch.bfloat16)}
    for name, x in (("k", k), ("v", v)):
        codes, scale = cache[name], cache[name + "_scale"]
        top = torch.where(x.isfinite(), x, 0.0).abs().amax(-1)
        top = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand_as(top), top, "amax")
        m, e = torch.frexp(top)
        e = torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8), MIN_EXP).clamp(min=MIN_EXP)
        asked = torch.ldexp(torch.ones_like(top), e)
        old = torch.where(first[:, None] == 0, 0.0, scale)
        new = torch.where(first[:, None] < P, torch.maximum(old, asked), scale)
        kept = codes.float() * (scale / new)[:, :, None, None]
        before = torch.arange(P, device=q.device) < torch.where(first < P, first, 0)[:, None]
        codes = torch.where(before[:, None, :, None], kept.to(torch.float8_e4m3fn).view(torch.uint8),
                            codes.view(torch.uint8))
        x = torch.where(x.isfinite(), x / new[page][:, :, None], math.nan).to(torch.float8_e4m3fn)
        codes[page, :, slot] = x.view(torch.uint8)
        out[name], out[name + "_scale"] = codes.view(torch.float8_e4m3fn), new
    return out


def _plain_attend(s):
    case, cache, table = s["case"], s["cache"], s["table"].long()
    B, Hq, Hkv, D, P = (case[k] for k in ("B", "Hq", "Hkv", "D", "P"))
    G, n, width = Hq // Hkv, case["q"], table.shape[1]
    b, pos = _places(s)
    t = torch.arange(s["T"], device=pos.device)
    j = t - (t if s["cu_q"] is None else s["cu_q"].long()[b])
    rows = torch.zeros(B, n, Hq, D, device=pos.device)
    rows[b, j] = s["q"].float()
    at = torch.full((B, n), -1, dtype=torch.int64, device=pos.device)
    at[b, j] = pos
    rows = rows.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    seen = torch.arange(width * P, device=pos.device) <= at[:, :, None]              # [B, n, keys]
    used = torch.arange(width * P, device=pos.device) < s["lens"][:, None]           # [B, keys]

    def whole(name):
        x = cache[name][table].float() * cache[name + "_scale"][table][..., None, None]
        x = x.transpose(1, 2).reshape(B, Hkv, width * P, D)
        return torch.where(used[:, None, :, None], x, 0.0)

    w = (rows @ whole("k").transpose(2, 3)).view(B, Hkv, G, n, width * P)
    w *= 1.0 / math.sqrt(D)
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w -= torch.where(top == -math.inf, 0.0, top)
    w.exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, Hkv, G * n, width * P) @ whole("v")).view(B, Hkv, G, n, D)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D), lse.permute(0, 3, 1, 2).reshape(B, n, Hq)
    return {"out": o[b, j].to(torch.bfloat16), "lse": lse[b, j]}


def run(state):
    s = state
    if own:
        import mhc_hyper_connection_pre_gb300 as mhc
        if s["case"]["op"] == "append":
            q = mhc.kv_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cu_q"], q=s["q"], cos=s["cos"],
                              sin=s["sin"], interleaved=s["case"]["pairs"])
            return {"q": q, **s["cache"]}
        return mhc.kv_attend(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], return_lse=True)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attend(s)


def work(case):
    q_lens, lens = _lengths(case)
    Hq, Hkv, D, P = (case[k] for k in ("Hq", "Hkv", "D", "P"))
    T = sum(q_lens)
    if case["op"] == "append":
        pages = sum(-(-n // P) - (n - m) // P for m, n in zip(q_lens, lens) if m)
        R = case["R"]
        return {"bytes": T * (Hkv * D * 2 * 3 + Hq * D * 4) + T * R * 4 + pages * Hkv * 16,
                "flops": T * (Hq + Hkv) * R * 3}
    seen = sum(m * n - m * (m - 1) // 2 for m, n in zip(q_lens, lens) if n)
    return {"bytes": T * Hq * (D * 4 + 4) + sum(lens) * Hkv * D * 2 + sum(-(-n // P) for n in lens) * Hkv * 8,
            "flops": 4 * seen * Hq * D}


# --------------------------------------------------------- 64-bit results ---

def _round_e4m3(x):
    """Nearest e4m3 number, ties to even, of |x| <= 448 (from the format: 3 bits after the point, exponents from -6)."""
    _, e = torch.frexp(x.abs())
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    case, P, R = s["case"], s["case"]["P"], s["case"]["R"]
    q_lens, lens = _lengths(case)
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(q_lens, lens)]).to(s["q"].device)
    out = {}

    def turned(x):
        x = x.double()
        if not R:
            return x
        z = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) if case["pairs"] else torch.complex(x[..., :R // 2], x[..., R // 2:R])
        z = z * torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
        y = torch.view_as_real(z).flatten(-2) if case["pairs"] else torch.cat((z.real, z.imag), -1)
        return torch.cat((y, x[..., R:]), -1)

    out["q"] = turned(s["q"])
    table = s["table"].tolist()
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        codes, scale = s["cache"][name].double(), s["cache"][name + "_scale"].double()
        t = 0
        for b, (m, n) in enumerate(zip(q_lens, lens)):
            at = n - m
            while at < n:
                page, slot = table[b][at // P], at % P
                take = min(P - slot, n - at)
                new = x[t:t + take].transpose(0, 1)                       # [Hkv, take, D]
                need = torch.exp2(torch.ceil(torch.log2(new.abs().amax((1, 2)) / E4M3_MAX))).clamp(min=2.0 ** MIN_EXP)
                had = scale[page] if slot else torch.zeros_like(need)
                now = torch.maximum(had, need)
                if slot:
                    codes[page, :, :slot] = _round_e4m3(codes[page, :, :slot] * (had / now)[:, None, None])
                codes[page, :, slot:slot + take] = _round_e4m3(new / now[:, None, None])
                scale[page] = now
                at, t = at + take, t + take
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_attend(s):
    case, cache = s["case"], s["cache"]
    Hq, Hkv, D, P = (case[k] for k in ("Hq", "Hkv", "D", "P"))
    G = Hq // Hkv
    q_lens, lens = _lengths(case)
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (m, n) in enumerate(zip(q_lens, lens)):
        if m and n:
            used = s["table"][b, :-(-n // P)].long()
            for h in range(Hkv):
                k, v = ((cache[c][used, h].double() * cache[c + "_scale"][used, h].double()[:, None, None]).reshape(-1, D)[:n]
                        for c in ("k", "v"))
                for lo in range(0, m, 1024):
                    hi = min(m, lo + 1024)
                    x = torch.einsum("tgd,kd->gtk", s["q"][t + lo:t + hi, h * G:(h + 1) * G].double(), k) / D ** 0.5
                    hidden = torch.arange(n, device="cuda") > torch.arange(n - m + lo, n - m + hi, device="cuda")[:, None]
                    x[:, hidden] = -math.inf
                    l = torch.logsumexp(x, -1)
                    lse[t + lo:t + hi, h * G:(h + 1) * G] = l.T
                    out[t + lo:t + hi, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", (x - l[..., None]).exp(), v)
        t += m
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
