"""The operators of a decode step's attention over a paged key-value cache, as cases to be timed and compared.

Three families, which a serving program calls one after the other in every step:

* ``plan``    pages for the step's new tokens from a ring of free pages: block tables, the new tokens' cache slots
              and positions, new lengths; the pages of requests that have ended go back to the ring;
* ``append``  rotary embedding of the new queries and keys, the new keys and values written to their cache slots,
              in bf16 or in e4m3 with one fp32 scale per token and head;
* ``attn``    attention of one new token per request over its pages (grouped query heads, an optional window of
              the last tokens), with the logarithm of each row's softmax sum.

A cache holds ``[pages, page, heads, dim]`` keys and the same of values, as a view of ``[pages, heads, page, dim]``
where ``heads_first`` is true; the scales of an e4m3 cache are ``[pages, heads, page]``.
"""
import math

import torch

own = False

BF16, F32, E4M3, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
E4M3_MAX = 448.0
MIN_AMAX = 1e-12          # a row whose largest magnitude is below this is scaled as if it were this
THETA = 10000.0
ENDED = -1                # in a request's count of new tokens: it has ended


# ------------------------------------------------------------------ the cases
def _plan(B, held, new, page, ended=0.0):
    """Requests that hold up to `held` tokens; `new` = 1: one token each, more: prompts of up to `new` tokens."""
    return {"op": "plan", "B": B, "held": held, "new": new, "page": page, "ended": ended}


def _append(T, Hq, Hkv, D, R, page, cache="bf16", interleaved=False, heads_first=False, padded=0.0):
    return {"op": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "page": page, "cache": cache,
            "interleaved": interleaved, "heads_first": heads_first, "padded": padded}


def _attn(B, longest, Hkv, G, D, page, cache="bf16", heads_first=False, window=0, ragged=True, empty=False):
    return {"op": "attn", "B": B, "longest": longest, "Hkv": Hkv, "G": G, "D": D, "page": page, "cache": cache,
            "heads_first": heads_first, "window": window, "ragged": ragged, "empty": empty}


def listed():
    return [
        # the step of a full batch: one token each, a few requests have ended
        dict(_plan(256, 8192, 1, 16, 0.03), name="plan_step"),
        # a step that admits prompts
        dict(_plan(61, 0, 2048, 16), name="plan_prompts"),
        # one generated token: latency
        dict(_append(1, 32, 8, 128, 128, 16), name="append_token"),
        # a padded batch of generated tokens into an 8-bit cache
        dict(_append(61, 64, 8, 128, 64, 64, "e4m3", padded=0.1), name="append_batch_e4m3"),
        # the rows of long prompts: memory bandwidth
        dict(_append(16384, 32, 8, 128, 128, 16, interleaved=True), name="append_prompt"),
        # one request, a short conversation: latency
        dict(_attn(1, 777, 8, 4, 128, 16), name="attn_one_short"),
        # one request with a long document: the split over the length
        dict(_attn(1, 131071, 8, 4, 128, 16), name="attn_one_long"),
        # a batch of conversations of very different lengths
        dict(_attn(64, 16384, 8, 4, 128, 16), name="attn_batch"),
        # many short requests, some slots empty, an 8-bit cache
        dict(_attn(256, 2048, 8, 8, 128, 32, "e4m3", empty=True), name="attn_many_e4m3"),
        # a few long requests over an 8-bit cache with heads first
        dict(_attn(4, 65536, 8, 8, 128, 64, "e4m3", heads_first=True, ragged=False), name="attn_long_e4m3"),
        # one key head for all query heads, wide heads
        dict(_attn(32, 8192, 1, 16, 256, 16), name="attn_one_head_256"),
        # as many key heads as query heads, a window of the last tokens
        dict(_attn(16, 8192, 16, 1, 64, 64, heads_first=True, window=1024), name="attn_window_64"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attn", "attn", "attn", "attn"])
    page = rng.choice([16, 16, 32, 64, 128, 24])
    if op == "plan":
        B = _log(rng, 1, 1024)
        if rng.random() < 0.5:
            return _plan(B, _log(rng, 1, 8192), 1, page, rng.choice([0.0, 0.05, 0.2]))
        return _plan(B, _log(rng, 1, 1024), _log(rng, 2, max(2, min(8192, 131072 // B))), page, rng.choice([0.0, 0.1]))
    cache = rng.choice(["bf16", "bf16", "e4m3"])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 2, 4, 4, 5, 8, 16])
    if op == "append":
        T = _log(rng, 1, max(1, min(16384, 16384 * 48 * 128 // ((G + 2) * Hkv * D))))
        return _append(T, Hkv * G, Hkv, D, rng.choice([D, D, D // 32 * 16]), page, cache, rng.random() < 0.5,
                       rng.random() < 0.5, rng.choice([0.0, 0.0, 0.2]))
    longest = _log(rng, 1, 131072)
    B = _log(rng, 1, 256)
    while B > 1 and B * longest * Hkv * D > 64 * 16384 * 8 * 128:
        B = (B + 1) // 2
    return _attn(B, longest, Hkv, G, D, page, cache, rng.random() < 0.5, rng.choice([0, 0, 0, 128, 4095]),
                 rng.random() < 0.7, rng.random() < 0.3)


def _lengths(case):
    """The batch's lengths, before a seed shuffles them."""
    B, longest = case["B"], case["longest"]
    n = [max(1, longest * (i + 1) // B) if case["ragged"] else longest for i in range(B)]
    return [0 if case["empty"] and i % 7 == 3 else v for i, v in enumerate(n)]


def _new_tokens(case):
    """The requests' new tokens, before a seed shuffles them: one in eight has none."""
    B, new = case["B"], case["new"]
    ended = [case["ended"] and i % max(1, round(1 / case["ended"])) == 5 for i in range(B)]
    return [ENDED if ended[i] else 0 if i % 8 == 7 else max(1, new * (i + 1) // B) for i in range(B)]


# ------------------------------------------------------------------ what a user has in hand
_handle = None


def _library():
    """One handle, which a program opens once."""
    global _handle
    if _handle is None:
        from consumer_movement_gemm_gb300 import tovl
        _handle = tovl.Handle(0)
    return _handle


def _shuffled(values, g, dev):
    t = torch.tensor(values, dtype=I32, device=dev)
    return t[torch.randperm(len(values), generator=g, device=dev)]


def _empty_cache(s, case, pages, dev):
    """Keys and values of `pages` pages, and scales where they are held in 8 bits."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    shape = (pages, Hkv, page, D) if case["heads_first"] else (pages, page, Hkv, D)
    dt = BF16 if case["cache"] == "bf16" else E4M3
    for n in ("k", "v"):
        t = torch.empty(shape, dtype=dt, device=dev)
        s[n + "_cache"] = t.transpose(1, 2) if case["heads_first"] else t
        s[n + "_scale"] = None if dt is BF16 else torch.empty(pages, Hkv, page, dtype=F32, device=dev)


def _fill_cache(s, g, dev):
    """What earlier steps wrote: normal keys and values; in 8 bits they use the range that their scales give."""
    for n in ("k", "v"):
        t = s[n + "_cache"]
        for at in range(0, len(t), 4096):
            part = t[at:at + 4096]
            x = torch.randn(part.shape, generator=g, device=dev, dtype=BF16)
            part.copy_(x if t.dtype is BF16 else x.float().mul_(E4M3_MAX / 4).clamp_(-E4M3_MAX, E4M3_MAX))
        if s[n + "_scale"] is not None:
            s[n + "_scale"].uniform_(0.5, 2.0, generator=g).mul_(4 / E4M3_MAX)


def _own_cache(s):
    from consumer_movement_gemm_gb300 import tovl
    s["lib"] = _library()
    s["cache_"] = tovl.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    s["stream"] = torch.cuda.current_stream(dev).cuda_stream
    page = case["page"]
    if case["op"] == "plan":
        B = case["B"]
        add = _new_tokens(case)
        s["add"] = _shuffled(add, g, dev)
        s["length"] = (torch.rand(B, generator=g, device=dev) * (case["held"] + 1)).to(I32)
        s["cap"] = -(-sum(max(0, a) for a in add) // 8) * 8 + 8
        W = -(-(case["held"] + max(1, case["new"])) // page) + 1
        have = (s["length"].long() + page - 1) // page
        pages = B * W
        order = torch.randperm(pages, generator=g, device=dev).to(I32)
        held = torch.arange(W, device=dev)[None] < have[:, None]
        s["table"] = torch.where(held, order.view(B, W), -1)
        # the pages that no request holds, from somewhere in the ring on
        free = (B * W - have.sum()).to(I32)
        head = torch.randint(0, pages, (), generator=g, device=dev, dtype=I32)
        rank = torch.argsort(held.flatten().to(torch.int8), stable=True)       # free ones first
        s["ring"] = torch.where(torch.arange(pages, device=dev) < free, order[rank], -1).roll(int(head))
        s["state"] = torch.stack([head, free, torch.zeros_like(free), torch.zeros_like(free)])
        if own:
            s["lib"] = _library()
            s["length_out"], s["state_out"] = torch.empty_like(s["length"]), torch.empty_like(s["state"])
            s["slots"] = torch.empty(s["cap"], dtype=I32, device=dev)
            s["positions"] = torch.empty(s["cap"], dtype=I32, device=dev)
            s["starts"] = torch.empty(B + 1, dtype=I32, device=dev)
    elif case["op"] == "append":
        T, Hq, Hkv, D, R = (case[n] for n in ("T", "Hq", "Hkv", "D", "R"))
        # rows of one projection: queries, keys, values
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=dev, dtype=BF16)
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        farthest = 32768
        angle = torch.arange(farthest, device=dev, dtype=torch.float64)[:, None] * THETA ** (
            -torch.arange(R // 2, device=dev, dtype=torch.float64) * 2 / max(1, R))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(F32)
        s["positions"] = torch.randint(0, farthest, (T,), generator=g, device=dev, dtype=I32)
        pages = -(-T // page) + 3
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].to(I32)
        if case["padded"]:      # rows behind the step's tokens
            s["slots"][max(1, T - int(T * case["padded"])):] = -1
        _empty_cache(s, case, pages, dev)
        _fill_cache(s, g, dev)
        if own:
            _own_cache(s)
            s["q_out"] = torch.empty(T, Hq, D, dtype=BF16, device=dev)
    else:
        B, Hkv, G, D = (case[n] for n in ("B", "Hkv", "G", "D"))
        s["length"] = _shuffled(_lengths(case), g, dev)
        W = -(-case["longest"] // page)
        have = (s["length"].long() + page - 1) // page
        pages = sum(-(-v // page) for v in _lengths(case)) + 2
        order = torch.randperm(pages, generator=g, device=dev).to(I32)
        col = torch.arange(W, device=dev)[None]
        first = (have.cumsum(0) - have)[:, None]
        s["table"] = torch.where(col < have[:, None], order[(first + col).clamp_max(pages - 1)], -1)
        s["q"] = torch.randn(B, Hkv * G, D, generator=g, device=dev).mul_(2).to(BF16)
        _empty_cache(s, case, pages, dev)
        _fill_cache(s, g, dev)
        if own:
            _own_cache(s)
            s["out"] = torch.empty(B, Hkv * G, D, dtype=BF16, device=dev)
            s["lse"] = torch.empty(B, Hkv * G, dtype=F32, device=dev)
            s["workspace"] = torch.empty(_library().attn_decode_workspace(Hkv * G, Hkv, D), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_plan(s):
    s["lib"].page_plan(s["length"], s["add"], s["table"], s["ring"], s["state"], s["page"], s["length_out"], s["state_out"],
                       s["slots"], s["positions"], s["starts"], stream=s["stream"])
    return {"length": s["length_out"], "state": s["state_out"], "table": s["table"], "ring": s["ring"], "slots": s["slots"],
            "positions": s["positions"], "starts": s["starts"]}


def _own_append(s):
    s["lib"].rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["cache_"], s["q_out"],
                         interleaved=s["interleaved"], stream=s["stream"])
    return _cache_out(s, {"q": s["q_out"]})


def _own_attn(s):
    s["lib"].attn_decode(s["q"], s["cache_"], s["table"], s["length"], s["D"] ** -0.5, s["out"], s["workspace"],
                         window=s["window"], lse=s["lse"], stream=s["stream"])
    return {"out": s["out"], "lse": s["lse"]}


def _cache_out(s, r):
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if s[n] is not None:
            r[n] = s[n]
    return r


def _plain_plan(s):
    """Pages are taken from the ring's head in the order of the requests; those of ended requests go behind its tail."""
    dev, page, n, cap = s["add"].device, s["page"], len(s["ring"]), s["cap"]
    length, ended = s["length"].long(), s["add"] == ENDED
    add = s["add"].long().clamp_min(0)
    have = (length + page - 1) // page
    need = torch.where(ended, have, (length + add + page - 1) // page)
    take_end, tok_end = (need - have).cumsum(0), add.cumsum(0)
    take_at, tok_at = take_end - (need - have), tok_end - add
    head, free = s["state"][0].long(), s["state"][1].long()
    W = s["table"].shape[1]
    col = torch.arange(W, device=dev)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    taken = s["ring"][(head + take_at[:, None] + col - have[:, None]) % n]
    s["table"].copy_(torch.where(fresh, taken, s["table"]))
    i = torch.arange(cap, device=dev)
    b = torch.searchsorted(tok_end, i, right=True).clamp_max(len(add) - 1)
    real = i < tok_end[-1]
    at = length[b] + i - tok_at[b]
    slot = s["table"][b, (at // page).clamp(0, W - 1)].long() * page + at % page
    back = torch.where(ended, have, 0)
    back_end = back.cumsum(0)
    o = (torch.arange(n, device=dev) - head - free) % n
    rb = torch.searchsorted(back_end, o, right=True).clamp_max(len(add) - 1)
    page_back = s["table"][rb, (o - back_end[rb] + back[rb]).clamp(0, W - 1)]
    s["ring"].copy_(torch.where(o < back_end[-1], page_back, s["ring"]))
    zero = torch.zeros_like(head)
    return {"length": torch.where(ended, 0, length + add).to(I32),
            "state": torch.stack([(head + take_end[-1]) % n, free - take_end[-1] + back_end[-1], tok_end[-1], zero]).to(I32),
            "table": s["table"], "ring": s["ring"], "slots": torch.where(real, slot, -1).to(I32),
            "positions": torch.where(real, at, 0).to(I32), "starts": torch.cat([zero[None], tok_end]).to(I32)}


def _rotated(x, cs, R, interleaved):
    x = x.float()
    if R == 0:
        return x
    c, sn = cs[:, None, : R // 2], cs[:, None, R // 2:]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., : R // 2], x[..., R // 2: R])
    ra, rb = a * c - b * sn, b * c + a * sn
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., R:]], -1)


def _plain_append(s):
    """A slot of -1: the row is behind the step's tokens, and nothing of it goes to the cache."""
    cs = s["cos_sin"][s["positions"].long()]
    real = s["slots"] >= 0
    slot = torch.where(real, s["slots"], s["slots"][0]).long()      # (the first row's again: it writes the same)
    at, off = slot // s["page"], slot % s["page"]
    rows = {"k": _rotated(s["k"], cs, s["R"], s["interleaved"]), "v": s["v"].float()}
    for n, x in rows.items():
        x = torch.where(real[:, None, None], x, x[:1])
        if s["cache"] == "e4m3":
            scale = x.abs().amax(2).clamp_min(MIN_AMAX) / E4M3_MAX
            s[n + "_scale"][at, :, off] = scale
            x = (x / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
            s[n + "_cache"].view(torch.uint8)[at, off] = x.to(E4M3).view(torch.uint8)
        else:
            s[n + "_cache"][at, off] = x.to(BF16)
    return _cache_out(s, {"q": _rotated(s["q"], cs, s["R"], s["interleaved"]).to(BF16)})


def _plain_attn(s):
    B, Hkv, G, D, page = (s[n] for n in ("B", "Hkv", "G", "D", "page"))
    at = s["table"].clamp_min(0).long()
    L = at.shape[1] * page

    def rows(n):
        x = s[n + "_cache"]
        x = x[at].float() if x.dtype is BF16 else x.view(torch.uint8)[at].view(E4M3).float()
        if s[n + "_scale"] is not None:
            x = x * s[n + "_scale"][at].transpose(2, 3)[..., None]
        return x.reshape(B, L, Hkv, D)

    length = s["length"][:, None]
    pos = torch.arange(L, device=at.device)[None]
    seen = pos < length
    if s["window"]:
        seen &= pos >= length - s["window"]
    k = rows("k").permute(0, 2, 3, 1)
    z = (s["q"].float().view(B, Hkv, G, D) @ k) * D ** -0.5
    z = torch.where(seen[:, None, None], z, -torch.inf)
    m = z.amax(3, keepdim=True).clamp_min(-3e38)        # (no token: nothing but -inf)
    p = torch.exp(z - m)
    del k
    total = p.sum(3, keepdim=True)
    out = (p @ rows("v").permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1)
    lse = torch.where(total > 0, m + torch.log(total), -torch.inf)
    return {"out": out.view(B, Hkv * G, D).to(BF16), "lse": lse.view(B, Hkv * G)}


_plain = {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}
_own = {"plan": _own_plan, "append": _own_append, "attn": _own_attn}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    page = case["page"]
    if case["op"] == "plan":
        B = case["B"]
        tokens = sum(max(0, a) for a in _new_tokens(case))
        # lengths and counts read, lengths and starts written; per token a slot and a position; per page taken two words
        return {"bytes": 16 * B + 8 * tokens + 8 * (tokens // page + 1) + 32, "flops": 4 * B + 8 * tokens}
    each = 2 if case["cache"] == "bf16" else 1 + 4 / case["D"]
    if case["op"] == "append":
        T, Hq, Hkv, D, R = (case[n] for n in ("T", "Hq", "Hkv", "D", "R"))
        real = T - (int(T * case["padded"]) if case["padded"] else 0)
        return {"bytes": T * Hq * D * 4 + real * 2 * Hkv * D * (2 + each) + 4 * R * min(T, 32768) + 8 * T,
                "flops": 3 * T * (Hq + Hkv) * R}
    B, Hkv, G, D = (case[n] for n in ("B", "Hkv", "G", "D"))
    n = [min(v, case["window"]) if case["window"] else v for v in _lengths(case)]
    pages = sum(-(-v // page) for v in n)
    return {"bytes": sum(n) * Hkv * D * 2 * each + 4 * pages + B * (4 + Hkv * G * (4 * D + 4)),
            "flops": 4 * sum(n) * Hkv * G * D}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    W64 = torch.float64
    if case["op"] == "plan":
        return None          # (whole numbers only)
    if case["op"] == "append":
        R, half = case["R"], case["R"] // 2
        cs = s["cos_sin"][s["positions"].long()].to(W64)

        def turn(x):
            y = x.to(W64).clone()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                u, w = x[..., a].to(W64), x[..., b].to(W64)
                y[..., a] = u * cs[:, i, None] - w * cs[:, half + i, None]
                y[..., b] = u * cs[:, half + i, None] + w * cs[:, i, None]
            return y

        out = {"q": turn(s["q"])}
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot = s["slots"][keep].long()
        at, off = torch.div(slot, case["page"], rounding_mode="floor"), slot.remainder(case["page"])
        for n, x in (("k", turn(s["k"])), ("v", s["v"].to(W64))):
            x, c = x[keep], s[n + "_cache"].to(W64)
            if case["cache"] == "e4m3":
                top = torch.clamp(x.abs().max(2).values, min=MIN_AMAX) / E4M3_MAX
                scale = s[n + "_scale"].to(W64)
                scale[at, :, off] = top
                out[n + "_scale"] = scale
                x = x / top[:, :, None]
            c[at, off] = x
            out[n + "_cache"] = c
        return out
    B, Hkv, G, D, page = (case[n] for n in ("B", "Hkv", "G", "D", "page"))
    if sum(_lengths(case)) * Hkv * (G + 2) * D > 3 << 31:
        return None
    out = torch.zeros(B, Hkv * G, D, dtype=W64, device=s["q"].device)
    lse = torch.full((B, Hkv * G), -torch.inf, dtype=W64, device=s["q"].device)
    for b, n in enumerate(s["length"].tolist()):
        if n == 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        t = torch.arange(first, n, device=s["q"].device)
        at, off = s["table"][b].long()[torch.div(t, page, rounding_mode="floor")], t.remainder(page)
        for h in range(Hkv):
            kv = []
            for m in ("k", "v"):
                x = s[m + "_cache"]
                x = (x[at, off, h] if x.dtype is BF16 else x.view(torch.uint8)[at, off, h].view(E4M3)).to(W64)
                kv.append(x if s[m + "_scale"] is None else x * s[m + "_scale"][at, h, off].to(W64)[:, None])
            z = s["q"][b, h * G:(h + 1) * G].to(W64) @ kv[0].T / math.sqrt(D)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
            out[b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ kv[1]
    return {"out": out, "lse": lse}
