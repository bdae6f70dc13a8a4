"""More operators of the attention sublayer's paged cache, as cases to be measured.

  append   the new tokens' queries and keys are normed head by head and
           rotated, keys and values are written into the paged 8-bit cache;
  attend   causal attention of the new tokens over that cache with a sliding
           window and a few first tokens that stay visible;
  fork     the pages of the next step: every place of the batch goes on with
           the tokens of some place, sharing full pages and copying a
           part-filled last one, and gets pages for its next tokens;
  compact  the pages in use move to the lowest numbers.

``run`` computes them in plain torch operations, or, with ``own`` set, calls
``kv_append``, ``kv_attend``, ``kv_fork`` and ``kv_compact`` of this package.

The cache of one layer is k and v [pages, Hkv, P, D] in e4m3, k_scale and
v_scale [pages, Hkv] fp32; the layers of a model share page numbers.  Sequence
b holds its token at position i in page table[b, i // P], slot i % P; an entry
of -1 is a page that it no longer has.  cu_q [B + 1] says which of the T new
tokens belong to which sequence, lens [B] how many tokens a sequence has.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -116            # smallest exponent of a scale: 2**-116 times e4m3's smallest step is a normal fp32
EPS = 1e-6


def listed():
    """Head layouts: 40 query heads of 128 make this repository's hidden size
    of 5120; the others are generic.  Token counts run from one to the
    repository's prefill of 16384."""
    return [
        # one user, one token: the launch is what counts
        dict(name="append normed token", op="append", B=1, q=1, L=1001, ragged=False, Hq=40, Hkv=8, D=128, P=64,
             R=128, pairs=False, fused=True, each_head=False),
        # several prompts at once, odd lengths, a weight for every head, half of each head rotated in neighbouring pairs
        dict(name="append normed prompts", op="append", B=7, q=1500, L=1777, ragged=True, Hq=32, Hkv=4, D=64, P=16,
             R=32, pairs=True, fused=False, each_head=True),
        # one long prompt
        dict(name="append normed long prompt", op="append", B=1, q=16384, L=16384, ragged=False, Hq=40, Hkv=8, D=128,
             P=64, R=128, pairs=False, fused=True, each_head=False),
        # one user with a long document, of which a window and the first tokens are seen
        dict(name="attend window token", op="attend", B=1, q=1, L=131071, W=4096, S=4, ragged=False, Hq=40, Hkv=8,
             D=128, P=64),
        # a decode batch of ragged lengths, shorter and longer than the window, with unused places
        dict(name="attend window decode batch", op="attend", B=128, q=1, L=8192, W=1024, S=4, ragged=True, Hq=40,
             Hkv=8, D=128, P=64),
        # drafted tokens to be verified, heads that are not shared, small pages, a border inside a page
        dict(name="attend window drafted tokens", op="attend", B=48, q=3, L=4000, W=500, S=17, ragged=True, Hq=16,
             Hkv=16, D=64, P=16),
        # a chunk of a long prompt after what is cached of it
        dict(name="attend window prompt chunk", op="attend", B=1, q=4096, L=16384, W=4096, S=128, ragged=False, Hq=40,
             Hkv=8, D=128, P=64),
        # between two decode steps: some sequences need a page, some have one that left the window
        dict(name="fork decode step", op="fork", B=256, L=3001, groups=0, room=1, W=1024, S=4, layers=4, held=0.0,
             Hkv=8, D=128, P=64),
        # beams of several users after a step's choices
        dict(name="fork beams", op="fork", B=64, L=2000, groups=8, room=1, W=0, S=0, layers=4, held=0.1, Hkv=8, D=128,
             P=64),
        # many answers to be sampled for a few prompts, with pages for their first tokens
        dict(name="fork prompts", op="fork", B=512, L=1777, groups=512, room=100, W=0, S=0, layers=8, held=0.0, Hkv=8,
             D=128, P=64),
        # a small cache after some sequences have ended
        dict(name="compact small cache", op="compact", B=24, L=700, used=0.5, layers=2, held=0.05, Hkv=4, D=64, P=16),
        # a large one
        dict(name="compact large cache", op="compact", B=100, L=6000, used=0.6, layers=4, held=0.02, Hkv=8, D=128,
             P=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """Serving traffic over the same ranges: one to 512 sequences, one token
    to long prompts, contexts up to 131071, windows from a few tokens on,
    groups of 1 to 16 query heads, up to 8 layers."""
    D, P = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    op = rng.choice(["append", "attend", "attend", "fork", "compact"])
    c = dict(op=op, Hkv=Hkv, D=D, P=P)
    token = Hkv * D * 2                              # bytes that a cached token takes in a layer
    if op in ("append", "attend"):
        G = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * Hkv <= 64])
        c["Hq"], c["ragged"] = G * Hkv, rng.random() < 0.7
        kind = rng.choice(["tokens", "tokens", "drafts", "prompts"])
        if kind == "tokens":
            c["B"], c["q"] = _log(rng, 1, 256), 1
        elif kind == "drafts":
            c["B"], c["q"] = _log(rng, 1, 128), rng.randint(2, 16)
        else:
            c["B"] = _log(rng, 1, 8)
            c["q"] = _log(rng, 17, 4096 // c["B"])
    if op == "append":
        c["L"] = c["q"] + _log(rng, 1, 300) - 1
        c["R"] = rng.choice([D, D, D // 2, 0])
        c["pairs"], c["fused"], c["each_head"] = rng.random() < 0.3, rng.random() < 0.6, rng.random() < 0.3
    elif op == "attend":
        most = min(8192, int(2.5e8) // (token * c["B"]), int(8e10) // (c["Hq"] * D * c["q"] * c["B"]) - 300)
        c["W"] = _log(rng, 1, max(16, most))         # less work than the listed chunk
        c["S"] = rng.choice([0, 1, 4, rng.randint(1, 300)])
        c["L"] = max(c["q"], _log(rng, 1, 131071))
    elif op == "fork":
        c["B"] = _log(rng, 1, 512)
        c["L"] = _log(rng, 1, max(1, min(4000, int(5e8) // (token * c["B"]))))
        c["groups"] = rng.choice([0, rng.randint(1, c["B"]), c["B"]])
        c["room"] = rng.choice([0, 1, 1, rng.randint(1, 300)])
        c["W"] = rng.choice([0, 0, _log(rng, 1, 2000)])
        c["S"] = rng.randint(0, 40) if c["W"] else 0
        c["layers"], c["held"] = rng.randint(1, 8), rng.choice([0.0, 0.1])
    else:
        c["B"] = _log(rng, 1, 256)
        c["L"] = _log(rng, 1, max(1, min(20000, int(8e8) // (token * c["B"]))))
        c["used"], c["held"] = rng.uniform(0.2, 1.0), rng.choice([0.0, 0.05])
        c["layers"] = rng.randint(1, 4)
    return c


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """New tokens and whole lengths of the sequences: the same for every seed."""
    r = _rng(case)
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


def _kept(n, first, P, S):
    """Whether each page of n tokens holds one that a token sees whose window begins at `first`."""
    return [i * P < S or (i + 1) * P > first for i in range(-(-n // P))]


def _tokens(case):
    """fork, compact: the sequences' lengths, the same for every seed; the first is the longest."""
    r = _rng(case)
    return [case["L"] if b == 0 else (0 if r.random() < 0.03 else max(1, int(case["L"] * r.uniform(0.1, 1.0))))
            for b in range(case["B"])]


def _parents(case):
    """fork: which place each place goes on with; None: itself, all of them."""
    r, B, n = _rng(case), case["B"], case["groups"]
    if n == 0:
        return None
    size = max(2, B // n) if n < B else max(2, B // 8)      # beams of a user, or answers to a prompt
    if n < B:
        return [-1 if r.random() < 0.03 else min(B - 1, b // size * size + r.randrange(size)) for b in range(B)]
    return [b // size * size for b in range(B)]


def _draws(case, g, dev):
    """Sources of random bf16 numbers and of codes for a cache."""
    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)

    def codes(*shape):
        # what appending normal values leaves: the largest of a page is near 4, so values reach 256
        # times a scale of 2**-6
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
        flat = out.flatten()
        for i in range(0, flat.numel(), 1 << 26):
            x = torch.randn(min(1 << 26, flat.numel() - i), generator=g, device=dev).clamp_(-6.5, 6.5)
            flat[i:i + x.numel()] = (x * 64.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return out

    def scales(*shape):                    # each page and head its own
        return 2.0 ** torch.randint(-8, -4, shape, generator=g, device=dev).float()

    return normal, codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    normal, codes, scales = _draws(case, g, dev)
    Hkv, D, P = (case[k] for k in ("Hkv", "D", "P"))
    if case["op"] in ("fork", "compact"):
        return _prepare_pages(case, g, dev, codes, scales)
    q_lens, lens = _lengths(case)
    B, Hq, T = case["B"], case["Hq"], sum(q_lens)
    # with a window the pages that no new token sees are gone
    kept = [_kept(n, n - m - case["W"] + 1, P, case["S"]) if "W" in case else [True] * -(-n // P)
            for m, n in zip(q_lens, lens)]
    width, pages = max(1, max(len(k) for k in kept)), sum(sum(k) for k in kept) + 3
    order = iter(torch.randperm(pages, generator=g, device=dev).tolist())
    rows = [[next(order) if x else -1 for x in k] + [0] * (width - len(k)) for k in kept]
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s = {"case": dict(case), "T": T,
         "table": torch.tensor(rows, dtype=torch.int32, device=dev),
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "cu_q": None if _single(case) else torch.tensor(cu, dtype=torch.int32, device=dev)}
    s["cache"] = {"k": codes(pages, Hkv, P, D), "v": codes(pages, Hkv, P, D)}
    for b, n in enumerate(lens):           # slots that nothing was written to hold any byte, NaN's among them
        if n % P and b < 64:
            for name in ("k", "v"):
                s["cache"][name][rows[b][n // P], :, n % P:] = 0x7F
    s["cache"] = {n: x.view(torch.float8_e4m3fn) for n, x in s["cache"].items()}
    s["cache"].update(k_scale=scales(pages, Hkv), v_scale=scales(pages, Hkv))
    if case["op"] == "attend":
        s["q"] = normal(T, Hq, D)
        return s
    # projections of a residual stream: every head its own size
    size = 2.0 ** (torch.rand(Hq + 2 * Hkv, generator=g, device=dev) * 6 - 2)
    x = (normal(T, Hq + 2 * Hkv, D) * size[:, None]).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = x.split([Hq, Hkv, Hkv], dim=1)          # slices of one projection's rows
    if not case["fused"]:
        s["q"], s["k"], s["v"] = s["q"].contiguous(), s["k"].contiguous(), s["v"].contiguous()
    for name, heads in (("q_norm", Hq), ("k_norm", Hkv)):
        s[name] = (1 + 0.2 * normal(*([heads, D] if case["each_head"] else [D]))).to(torch.bfloat16)
    R = case["R"]
    s["cos"] = s["sin"] = None
    if R:
        places = torch.arange(width * P, dtype=torch.float64, device=dev)
        rate = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device=dev) * 2 / R)
        angle = places[:, None] * rate
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    return s


def _prepare_pages(case, g, dev, codes, scales):
    """The caches of all layers, as views of one buffer each for k, v and
    their scales, and the tables over them."""
    Hkv, D, P, B = (case[k] for k in ("Hkv", "D", "P", "B"))
    lens = _tokens(case)
    first = [n - case["W"] if case.get("W") else 0 for n in lens]    # the last token's window
    kept = [_kept(n, f, P, case.get("S", 0)) for n, f in zip(lens, first)]
    in_use = sum(sum(k) for k in kept)
    width = max(len(k) for k in kept) + -(-case.get("room", 0) // P)
    if case["op"] == "fork":
        need = B * (1 + -(-case["room"] // P))
        pages = int((in_use + need) * (1 + case["held"])) + 8
    else:
        pages = int(in_use / case["used"] * (1 + case["held"])) + 8
    order = torch.randperm(pages, generator=g, device=dev).tolist()
    it = iter(order)
    rows = [[next(it) if x else -1 for x in k] + [-1] * (width - len(k)) for k in kept]
    held = torch.zeros(pages, dtype=torch.bool, device=dev)
    spare = list(it)
    held[spare[:int(case["held"] * len(spare))]] = True              # kept for somebody outside of these tables
    s = {"case": dict(case), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "table": torch.tensor(rows, dtype=torch.int32, device=dev), "held": held if case["held"] else None}
    layers = case["layers"]
    s["all"] = {n: codes(layers, pages, Hkv, P, D).view(torch.float8_e4m3fn) for n in ("k", "v")}
    s["all"].update({n: scales(layers, pages, Hkv) for n in ("k_scale", "v_scale")})
    s["caches"] = [{n: x[i] for n, x in s["all"].items()} for i in range(layers)]
    if case["op"] == "fork":
        parents = _parents(case)
        s["parents"] = None if parents is None else torch.tensor(parents, dtype=torch.int32, device=dev)
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


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _turn(x, cos, sin, pairs):
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    c, d = a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]
    y = torch.stack((c, d), -1).flatten(-2) if pairs else torch.cat((c, d), -1)
    return torch.cat((y, x[..., R:]), -1)


def _plain_append(s):
    case, cache = s["case"], s["cache"]
    P = case["P"]
    b, pos = _places(s)
    page, slot = s["table"][b, pos // P].long(), pos % P
    q, k, v = _normed(s["q"], s["q_norm"]), _normed(s["k"], s["k_norm"]), s["v"].float()
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
        asked = ((e + 127) << 23).int().view(torch.float32)              # 2**e, to the bit
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
    """Over the keys that some new token of the sequence sees: the first ones,
    then those from its first new token's window on."""
    case, cache, table = s["case"], s["cache"], s["table"].long()
    B, Hq, Hkv, D, P, W, S = (case[k] for k in ("B", "Hq", "Hkv", "D", "P", "W", "S"))
    G, n, width = Hq // Hkv, case["q"], table.shape[1]
    b, pos = _places(s)
    dev = pos.device
    t = torch.arange(s["T"], device=dev)
    j = t - (t if s["cu_q"] is None else s["cu_q"].long()[b])
    rows = torch.zeros(B, n, Hq, D, device=dev)
    rows[b, j] = s["q"].float()
    at = torch.full((B, n), -1, dtype=torch.int64, device=dev)
    at[b, j] = pos
    rows = rows.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    first, last = min(S, width * P), min(W + n - 1, width * P)       # keys of either kind
    early = torch.arange(first, device=dev).expand(B, first)
    late = s["lens"].long()[:, None] - last + torch.arange(last, device=dev)
    key = torch.cat((early, torch.where(late >= S, late, -1)), 1)    # [B, keys], -1: none
    p = at[:, :, None]
    seen = (key >= 0)[:, None] & (key[:, None] <= p) & ((key[:, None] > p - W) | (key < S)[:, None])
    used = seen.any(1)
    page, slot = table.gather(1, key.clamp(min=0) // P).clamp(min=0), key.clamp(min=0) % P

    def whole(name):
        x = cache[name].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()      # [B, keys, Hkv, D]
        x = x * cache[name + "_scale"][page][..., None]
        return torch.where(used[:, :, None, None], x, 0.0).transpose(1, 2)

    w = (rows @ whole("k").transpose(2, 3)).view(B, Hkv, G, n, -1)
    w *= 1.0 / math.sqrt(D)
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w -= torch.where(top == -math.inf, 0.0, top)
    w.exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, Hkv, G * n, -1) @ whole("v")).view(B, Hkv, G, n, D)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D), lse.permute(0, 3, 1, 2).reshape(B, n, Hq)
    return {"out": o[b, j].to(torch.bfloat16), "lse": lse[b, j]}


def _plain_fork(s):
    case, P, W, S = s["case"], s["case"]["P"], s["case"]["W"], s["case"]["S"]
    table, lens = s["table"].long(), s["lens"].long()
    pages, width, dev = s["all"]["k"].shape[1], table.shape[1], table.device
    if s["parents"] is not None:
        a = s["parents"].long()
        table, lens = table[a.clamp(min=0)], torch.where(a >= 0, lens[a.clamp(min=0)], 0)
    place, entry = torch.arange(len(lens), device=dev), torch.arange(width, device=dev)
    full, tail = lens // P, lens % P
    kept = (entry < full[:, None]) & (table >= 0)
    if W:                                     # what the next token sees
        kept &= (entry * P < S) | ((entry + 1) * P > (lens - W + 1)[:, None])
    out = torch.where(kept, table, -1)
    used = torch.zeros(pages, dtype=torch.bool, device=dev) if s["held"] is None else s["held"].clone()
    used[table[kept]] = True
    last = table.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    has = (tail > 0) & (last >= 0)
    # a part-filled page stays with the first place that goes on with it, unless somebody else has it too
    keeper = torch.full((pages,), len(lens), dtype=torch.int64, device=dev).scatter_reduce(0, last[has], place[has], "amin")
    keeps = has & ~used[last.clamp(min=0)] & (keeper[last.clamp(min=0)] == place)
    used[last[keeps]] = True
    copied = has & ~keeps
    now, then = -(-lens // P), -(-(lens + case["room"]) // P)
    wants = then - now + copied
    rank = wants.cumsum(0) - wants
    free = (~used).nonzero()[:, 0]
    free = torch.cat((free, torch.full((int(width),), -1, dtype=torch.int64, device=dev)))
    out[place[keeps], full[keeps]] = last[keeps]
    to, src, n = free[rank[copied]], last[copied], tail[copied]
    out[place[copied], full[copied]] = to
    new = (entry >= now[:, None]) & (entry < then[:, None])
    out = torch.where(new, free[((rank + copied - now)[:, None] + entry).clamp(0, len(free) - 1)], out)
    filled = (torch.arange(P, device=dev) < n[:, None])[:, None, :, None]
    every = s["all"]
    for name in ("k", "v"):
        x = every[name].view(torch.uint8)
        x[:, to] = torch.where(filled, x[:, src], x[:, to])
        every[name + "_scale"][:, to] = every[name + "_scale"][:, src]
    return {"block_table": out.int(), "seq_lens": lens.int(), **every}


def _plain_compact(s):
    P, every = s["case"]["P"], s["all"]
    table, lens = s["table"].long(), s["lens"].long()
    pages, width, dev = every["k"].shape[1], table.shape[1], table.device
    named = (torch.arange(width, device=dev) < -(-lens // P)[:, None]) & (table >= 0)
    used = torch.zeros(pages, dtype=torch.bool, device=dev)
    used[table[named]] = True
    held = torch.zeros_like(used) if s["held"] is None else s["held"]
    loose = used & ~held
    goal = ~held & ((~held).cumsum(0) <= loose.sum())
    src, to = (loose & ~goal).nonzero()[:, 0], (goal & ~loose).nonzero()[:, 0]
    new = torch.arange(pages, device=dev)
    new[src] = to
    for name in ("k", "v"):
        x = every[name].view(torch.uint8)
        x[:, to] = x[:, src]
        every[name + "_scale"][:, to] = every[name + "_scale"][:, src]
    taken = torch.where(goal | held, torch.arange(1, pages + 1, device=dev), 0).amax()
    return {"block_table": torch.where(named, new[table.clamp(min=0)], -1).int(), "pages": taken.int(), **every}


def run(state):
    s = state
    case, op = s["case"], s["case"]["op"]
    if own:
        import mhc_hyper_connection_pre_gb300 as mhc
        if op == "append":
            q = mhc.kv_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cu_q"], q=s["q"], cos=s["cos"],
                              sin=s["sin"], interleaved=case["pairs"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                              norm_eps=EPS)
            return {"q": q, **s["cache"]}
        if op == "attend":
            return mhc.kv_attend(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], window=case["W"],
                                 sinks=case["S"], return_lse=True)
        if op == "fork":
            got = mhc.kv_fork(s["caches"], s["table"], s["lens"], s["parents"], room=case["room"],
                              window=case["W"] or None, sinks=case["S"], held=s["held"])
        else:
            got = mhc.kv_compact(s["caches"], s["table"], s["lens"], held=s["held"])
        return {**got, **s["all"]}
    if op == "append":
        return _plain_append(s)
    return _plain_attend(s) if op == "attend" else _plain_fork(s) if op == "fork" else _plain_compact(s)


def _seen(m, n, W, S):
    """Keys that each of the m last of n tokens sees, summed up; and that any of them sees."""
    if n == 0:
        return 0, 0
    pairs = 0
    for p in range(n - m, n):
        first = max(0, p - W + 1)
        pairs += p + 1 - first + min(S, first)
    first = max(0, n - m - W + 1)
    return pairs, n - first + min(S, first)


def work(case):
    Hkv, D, P = (case[k] for k in ("Hkv", "D", "P"))
    if case["op"] in ("append", "attend"):
        q_lens, lens = _lengths(case)
        Hq, T = case["Hq"], sum(q_lens)
    if case["op"] == "append":
        pages = sum(-(-n // P) - (n - m) // P for m, n in zip(q_lens, lens) if m)
        R = case["R"]
        return {"bytes": T * (Hkv * D * 2 * 3 + Hq * D * 4) + T * R * 4 + pages * Hkv * 16,
                "flops": T * (Hq + Hkv) * (R * 3 + D * 4)}
    if case["op"] == "attend":
        each = [_seen(m, n, case["W"], case["S"]) for m, n in zip(q_lens, lens)]
        any_sees = sum(k for _, k in each)
        return {"bytes": T * Hq * (D * 4 + 4) + any_sees * Hkv * D * 2 + -(-any_sees // P) * Hkv * 8,
                "flops": 4 * sum(p for p, _ in each) * Hq * D}
    lens, layers = _tokens(case), case["layers"]
    if case["op"] == "fork":
        parents = _parents(case) or list(range(case["B"]))
        rows = sum(-(-lens[a] // P) for a in parents if a >= 0)
        ahead = sum(-(-(lens[a] if a >= 0 else 0) // P) for a in parents) + case["B"] * -(-case["room"] // P)
        met, copied, slots = set(), 0, 0
        for a in parents:
            if a >= 0 and lens[a] % P:
                copied, slots = (copied + 1, slots + lens[a] % P) if a in met else (copied, slots)
                met.add(a)
        return {"bytes": 4 * (rows + ahead + 3 * case["B"]) + layers * Hkv * (slots * D * 4 + copied * 16), "flops": 0}
    in_use = sum(-(-n // P) for n in lens)
    pages = int(in_use / case["used"] * (1 + case["held"])) + 8
    moved = int(in_use * max(0.0, 1 - in_use / pages))                # as pages are named at random
    return {"bytes": 8 * in_use + layers * Hkv * moved * (P * D * 4 + 16), "flops": 0}


# --------------------------------------------------------- 64-bit results ---

def _two(e):
    """2**e, to the bit."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """Nearest e4m3 number, ties to even, of |x| <= 448 (from the format: 3 bits after the point, exponents from -6)."""
    _, e = torch.frexp(x.abs())
    step = _two((e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    case, P, R = s["case"], s["case"]["P"], s["case"]["R"]
    q_lens, lens = _lengths(case)
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(q_lens, lens)]).to(s["q"].device)
    out = {}

    def turned(x, weight):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt() * weight.double()
        if not R:
            return x
        z = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) if case["pairs"] else torch.complex(x[..., :R // 2], x[..., R // 2:R])
        z = z * torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
        y = torch.view_as_real(z).flatten(-2) if case["pairs"] else torch.cat((z.real, z.imag), -1)
        return torch.cat((y, x[..., R:]), -1)

    out["q"] = turned(s["q"], s["q_norm"])
    table = s["table"].tolist()
    for name, x in (("k", turned(s["k"], s["k_norm"])), ("v", s["v"].double())):
        codes, scale = s["cache"][name].double(), s["cache"][name + "_scale"].double()
        t = 0
        for b, (m, n) in enumerate(zip(q_lens, lens)):
            at = n - m
            while at < n:
                page, slot = table[b][at // P], at % P
                take = min(P - slot, n - at)
                new = x[t:t + take].transpose(0, 1)                       # [Hkv, take, D]
                part, e = torch.frexp(new.abs().amax((1, 2)) / E4M3_MAX)  # the smallest power of two that is no less
                need = torch.where(part > 0, _two(torch.where(part == 0.5, e - 1, e)), 0.0).clamp(min=2.0 ** MIN_EXP)
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
    Hq, Hkv, D, P, W, S = (case[k] for k in ("Hq", "Hkv", "D", "P", "W", "S"))
    G = Hq // Hkv
    q_lens, lens = _lengths(case)
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (m, n) in enumerate(zip(q_lens, lens)):
        for lo in range(0, m if n else 0, 1024):
            hi = min(m, lo + 1024)
            p = torch.arange(n - m + lo, n - m + hi, device="cuda")
            start = max(0, n - m + lo - W + 1)                            # of the first token's window
            key = torch.cat((torch.arange(min(S, start), device="cuda"), torch.arange(start, n - m + hi, device="cuda")))
            page, slot = s["table"][b].long()[key // P], key % P
            hidden = (key > p[:, None]) | ((key <= p[:, None] - W) & (key >= S))
            for h in range(Hkv):
                k, v = (cache[c].view(torch.uint8)[page, h, slot].view(torch.float8_e4m3fn).double()
                        * cache[c + "_scale"][page, h].double()[:, None] for c in ("k", "v"))
                x = torch.einsum("tgd,kd->gtk", s["q"][t + lo:t + hi, h * G:(h + 1) * G].double(), k) / D ** 0.5
                x[:, hidden] = -math.inf
                l = torch.logsumexp(x, -1)
                lse[t + lo:t + hi, h * G:(h + 1) * G] = l.T
                out[t + lo:t + hi, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", (x - l[..., None]).exp(), v)
        t += m
    return {"out": out, "lse": lse}


def _moved(s, src, to, slots):
    """The caches after slots[i] slots of page src[i] have been written to page to[i]."""
    every = {n: x.clone() for n, x in s["all"].items()}
    for a, b, n in zip(src, to, slots):
        for name in ("k", "v"):
            every[name][:, b, :, :n] = s["all"][name][:, a, :, :n]
            every[name + "_scale"][:, b] = s["all"][name + "_scale"][:, a]
    return every


def _exact_fork(s):
    case, P, W, S = s["case"], s["case"]["P"], s["case"]["W"], s["case"]["S"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    parents = list(range(len(lens))) if s["parents"] is None else s["parents"].tolist()
    width, pages = s["table"].shape[1], s["all"]["k"].shape[1]
    taken = set() if s["held"] is None else set(s["held"].nonzero()[:, 0].tolist())
    n = [lens[a] if a >= 0 else 0 for a in parents]
    out = [[-1] * width for _ in parents]
    for b, a in enumerate(parents):
        for i in range(n[b] // P):
            if not W or i * P < S or (i + 1) * P > n[b] - W + 1:
                out[b][i] = table[a][i]
    shared = taken | {p for row in out for p in row if p >= 0}
    asks, keep = [], set()
    for b, a in enumerate(parents):
        i, last = n[b] // P, -1
        if n[b] % P and table[a][i] >= 0:
            last = table[a][i]
            if last in shared or last in keep:
                asks.append((b, i, last, n[b] % P))
            else:
                keep.add(last)
                out[b][i] = last
        asks += [(b, i, -1, 0) for i in range(-(-n[b] // P), -(-(n[b] + case["room"]) // P))]
    free = iter(p for p in range(pages) if p not in shared and p not in keep)
    copies = []
    for b, i, last, slots in asks:
        out[b][i] = next(free, -1)
        if last >= 0 and out[b][i] >= 0:
            copies.append((last, out[b][i], slots))
    every = _moved(s, *zip(*copies)) if copies else s["all"]
    return {"block_table": torch.tensor(out, dtype=torch.int32), "seq_lens": torch.tensor(n, dtype=torch.int32), **every}


def _exact_compact(s):
    P, table, lens = s["case"]["P"], s["table"].tolist(), s["lens"].tolist()
    held = set() if s["held"] is None else set(s["held"].nonzero()[:, 0].tolist())
    pages = s["all"]["k"].shape[1]
    used = {p for row, n in zip(table, lens) for p in row[:-(-n // P)] if p >= 0} - held
    goal = [p for p in range(pages) if p not in held][:len(used)]
    to = [p for p in goal if p not in used]
    src = sorted(used - set(goal))
    new = dict(zip(src, to))
    out = [[new.get(p, p) if i < -(-n // P) else -1 for i, p in enumerate(row)] for row, n in zip(table, lens)]
    every = _moved(s, src, to, [P] * len(src))
    return {"block_table": torch.tensor(out, dtype=torch.int32),
            "pages": torch.tensor(1 + max([-1, *goal, *held]), dtype=torch.int32), **every}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)
