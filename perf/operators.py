"""The operators of a decode step around the experts, as cases to be timed and compared.

Four families, which one step of a served mixture-of-experts model calls one after the other:

* ``norm``   residual addition + root-mean-square norm, with a bf16 output and an e4m3 output that has one
             fp32 scale per group of columns;
* ``route``  router logits -> the k experts of each token and their gate weights;
* ``moe``    the whole gated expert layer for up to 64 tokens, bf16 or 4-bit expert weights;
* ``matvec`` few rows times one 4-bit weight matrix (a dense projection or a shared expert beside the layer).

Packed 4-bit weights, ``[.., K/8, N]`` 32-bit words: a word holds rows 8r .. 8r+7 of one column, row 8r+2i in
bits 4i .. 4i+3 and row 8r+2i+1 in bits 16+4i .. 16+4i+3; weight = (nibble - zero) * scale, with one bf16 scale
(and one zero of 8 bits; 8 where there are none) per column and group of rows.
"""
import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_AMAX = 1e-12          # a group whose largest magnitude is below this is scaled as if it were this
EPS = 1e-5
MAX_TOKENS = 64
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)   # bit position of row 8r + i in a packed word


# ------------------------------------------------------------------ the cases
def _norm(T, H, group, residual="bf16"):
    return {"op": "norm", "T": T, "H": H, "group": group, "residual": residual}


def _route(T, E, k, dtype="f32", renorm=True, masked=0.0):
    return {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "renorm": renorm, "masked": masked}


def _moe(T, E, k, H, I, weights="bf16", group=0, zeros=False, absent=0.0):
    return {"op": "moe", "T": T, "E": E, "k": k, "H": H, "I": I, "weights": weights, "group": group, "zeros": zeros,
            "absent": absent}


def _matvec(T, K, N, group, zeros=False, x="bf16"):
    return {"op": "matvec", "T": T, "K": K, "N": N, "group": group, "zeros": zeros, "x": x}


def listed():
    return [
        # one generated token: nothing but latency
        dict(_norm(1, 4096, 128), name="norm_token"),
        # a batch of generated tokens beside a running prompt, residual stream kept in 32 bits
        dict(_norm(333, 7168, 128, "f32"), name="norm_batch"),
        # the rows of long prompts: memory bandwidth
        dict(_norm(16384, 7168, 128), name="norm_prompt"),
        # the router of one generated token
        dict(_route(1, 32, 4), name="route_token"),
        # the routing of long prompts over many experts, some of them masked out; bf16 logits tie
        dict(_route(65536, 256, 8, "bf16", True, 0.05), name="route_prompt"),
        # one generated token, two of eight experts
        dict(_moe(1, 8, 2, 4096, 2048), name="moe_token"),
        # a small batch over 32 experts: most experts see one to three rows
        dict(_moe(13, 32, 4, 7168, 2048), name="moe_batch"),
        # the largest batch that the decode form takes: every expert is read
        dict(_moe(64, 32, 4, 7168, 2048), name="moe_full"),
        # the same two with 4-bit experts
        dict(_moe(1, 32, 4, 7168, 2048, "q4", 128), name="moe_q4_token"),
        dict(_moe(24, 8, 2, 4096, 2048, "q4", 64, True), name="moe_q4_batch"),
        # a dense projection of one token
        dict(_matvec(1, 4096, 4096, 128), name="matvec_token"),
        # a wide projection of a batch whose rows come in 8 bits from the norm
        dict(_matvec(16, 7168, 32768, 128, True, "e4m3"), name="matvec_batch"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "route", "moe", "moe", "moe", "matvec", "matvec"])
    if op == "norm":
        H = _log(rng, 64, 8192)
        T = _log(rng, 1, min(65536, 16384 * 7168 // H))
        return _norm(T, H, rng.choice([32, 64, 128, 0]), rng.choice(["bf16", "f32", "none"]))
    if op == "route":
        E = _log(rng, 2, 384)
        T = _log(rng, 1, min(65536, 65536 * 256 // E))
        return _route(T, E, rng.randint(1, min(16, E)), rng.choice(["f32", "bf16"]), rng.random() < 0.7,
                      rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "moe":
        weights = rng.choice(["bf16", "q4"])
        group = rng.choice([32, 64, 128]) if weights == "q4" else 0
        step = group or 8
        E = _log(rng, 2, 64)
        H = _log(rng, 256, 7168) // step * step
        I = _log(rng, 128, 4096) // step * step
        while E * H * I > 32 * 7168 * 2048:
            E //= 2
        return _moe(_log(rng, 1, MAX_TOKENS), E, rng.randint(1, min(8, E)), H, I, weights, group,
                    weights == "q4" and rng.random() < 0.5, rng.choice([0.0, 0.0, 0.25]))
    group = rng.choice([32, 64, 128])
    K = _log(rng, 256, 8192) // group * group
    N = _log(rng, 128, 32768) // 16 * 16
    return _matvec(_log(rng, 1, MAX_TOKENS), K, N, group, rng.random() < 0.5, rng.choice(["bf16", "bf16", "e4m3"]))


# ------------------------------------------------------------------ what a user has in hand
def _packed(g, dev, experts, K, N, group, zeros):
    """Nibbles around the middle of their range, as quantised weights have, and the scales that give W a
    deviation of about 1/sqrt(K)."""
    words = lambda: torch.randint(-2**31, 2**31 - 1, (experts, K // 8, N), generator=g, device=dev, dtype=torch.int32)  # noqa: E731
    q = (words() & 0x77777777) + (words() & 0x77777777) + (words() & 0x11111111)
    s = (torch.rand(experts, K // group, N, generator=g, device=dev) + 0.5) * (0.3 / K ** 0.5)
    z = torch.randint(6, 10, (experts, K // group, N), generator=g, device=dev, dtype=torch.uint8) if zeros else None
    return q, s.to(BF16), z


def _normal(g, dev, shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=dev, dtype=BF16).mul_(scale)


_handle = None


def _library():
    """One handle and its stream, which a program opens once."""
    global _handle
    if _handle is None:
        from consumer_movement_gemm_gb300 import tovl
        _handle = tovl.Handle(0)
    return _handle


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    s["stream"] = torch.cuda.current_stream(dev).cuda_stream
    if op == "norm":
        T, H, group = case["T"], case["H"], case["group"]
        s["x"] = _normal(g, dev, (T, H))
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = torch.randn(T, H, generator=g, device=dev).mul_(3).to(BF16 if case["residual"] == "bf16" else F32)
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device=dev)).to(BF16)
        groups = -(-H // group) if group else 1
        if own:
            s["residual_out"] = None if s["residual"] is None else torch.empty_like(s["residual"])
            s["out"] = torch.empty(T, H, dtype=BF16, device=dev)
            s["q"] = torch.empty(T, H, dtype=E4M3, device=dev)
            s["scale"] = torch.empty(T, groups, dtype=F32, device=dev)
    elif op == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn(T, E, generator=g, device=dev).mul_(2)
        if case["masked"]:
            logits[torch.rand(T, E, generator=g, device=dev) < case["masked"]] = float("-inf")
        s["logits"] = logits.to(BF16 if case["dtype"] == "bf16" else F32)
        if own:
            s["topk"] = torch.empty(T, case["k"], dtype=torch.int32, device=dev)
            s["gate_w"] = torch.empty(T, case["k"], dtype=F32, device=dev)
    elif op == "moe":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = _normal(g, dev, (T, H))
        s["topk"] = torch.rand(T, E, generator=g, device=dev).argsort(1)[:, :k].to(torch.int32).contiguous()
        if case["absent"]:   # pairs whose expert lives elsewhere
            s["topk"][torch.rand(T, k, generator=g, device=dev) < case["absent"]] = -1
        s["gate_w"] = torch.softmax(torch.randn(T, k, generator=g, device=dev), 1)
        if case["weights"] == "bf16":
            s["w13"] = _normal(g, dev, (E, H, 2 * I), H ** -0.5)
            s["w2"] = _normal(g, dev, (E, I, H), I ** -0.5)
        else:
            s["w13"] = _packed(g, dev, E, H, 2 * I, case["group"], case["zeros"])
            s["w2"] = _packed(g, dev, E, I, H, case["group"], case["zeros"])
        if own:
            s["out"] = torch.empty(T, H, dtype=BF16, device=dev)
            s["workspace"] = torch.empty(_library().moe_decode_workspace(T, k, H, I), dtype=torch.uint8, device=dev)
    else:
        T, K, N = case["T"], case["K"], case["N"]
        s["x"], s["x_scale"] = _normal(g, dev, (T, K)), None
        if case["x"] == "e4m3":
            s["x"] = (torch.randn(T, K, generator=g, device=dev) * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
            s["x_scale"] = (torch.rand(T, -(-K // 128), generator=g, device=dev) + 0.5) * 0.01
        q, sc, z = _packed(g, dev, 1, K, N, case["group"], case["zeros"])
        s["wq"], s["w_scale"], s["w_zero"] = q[0], sc[0], None if z is None else z[0]
        if own:
            s["out"] = torch.empty(T, N, dtype=BF16, device=dev)
            s["workspace"] = torch.empty(_library().matvec_q4_workspace(T, N), dtype=torch.uint8, device=dev)
    if own:
        s["lib"] = _library()
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_norm(s):
    s["lib"].add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], out=s["out"],
                         q=s["q"], q_scale=s["scale"], group=s["group"], stream=s["stream"])
    r = {"out": s["out"], "q": s["q"], "scale": s["scale"]}
    if s["residual"] is not None:
        r["residual"] = s["residual_out"]
    return r


def _own_route(s):
    s["lib"].route_topk(s["logits"], s["topk"], s["gate_w"], renormalize=s["renorm"], stream=s["stream"])
    return {"topk": s["topk"], "gate_w": s["gate_w"]}


def _own_moe(s):
    if s["weights"] == "bf16":
        s["lib"].moe_decode(s["x"], s["topk"], s["gate_w"], s["w13"], s["w2"], s["out"], s["workspace"], stream=s["stream"])
    else:
        s["lib"].moe_decode_q4(s["x"], s["topk"], s["gate_w"], s["w13"], s["w2"], s["group"], s["out"], s["workspace"],
                               stream=s["stream"])
    return s["out"]


def _own_matvec(s):
    s["lib"].matvec_q4(s["x"], s["wq"], s["w_scale"], s["group"], s["out"], s["workspace"], zero=s["w_zero"],
                       x_scale=s["x_scale"], stream=s["stream"])
    return s["out"]


def _groups(y, group, fill):
    """[T, H] as [T, groups, group], the last group filled up."""
    T, H = y.shape
    group = group or H
    n = -(-H // group)
    return torch.nn.functional.pad(y, (0, n * group - H), value=fill).view(T, n, group)


def _plain_norm(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    yg = _groups(y, s["group"], 0.0)
    scale = yg.abs().amax(2).clamp_min(MIN_AMAX) / E4M3_MAX
    q = (yg / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(len(y), -1)[:, : y.shape[1]].to(E4M3)
    out = {"out": y.to(BF16), "q": q, "scale": scale}
    if s["residual"] is not None:
        out["residual"] = r.to(s["residual"].dtype)
    return out


def _plain_route(s):
    """An expert whose logit is -inf or NaN is never chosen; slots left over hold expert -1 with weight 0."""
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -torch.inf, l)
    top, idx = torch.sort(l, dim=1, descending=True, stable=True)   # equal logits: the lowest index first
    top, idx = top[:, : s["k"]], idx[:, : s["k"]]
    m = top[:, :1]
    e = lambda v: torch.where(v == -torch.inf, 0.0, torch.where(v == m, 1.0, torch.exp(v - m)))  # noqa: E731
    p = e(top)
    total = (p if s["renorm"] else e(l)).sum(1, keepdim=True)
    w = torch.where(p > 0, p / total, 0.0)
    return {"topk": torch.where(top == -torch.inf, -1, idx).to(torch.int32), "gate_w": w}


def _weights(w, group, ids=None):
    """Expert matrices in 32 bits, all of them or those of `ids`."""
    if isinstance(w, torch.Tensor):
        return (w if ids is None else w[ids]).float()
    q, sc, z = w if ids is None else (t if t is None else t[ids] for t in w)
    at = torch.tensor(SHIFTS, dtype=torch.int32, device=q.device)[:, None]
    v = (q[:, :, None, :] >> at) & 15
    v = v.view(q.shape[0], -1, group, q.shape[2]).float()
    v = (v - (8.0 if z is None else z.float()[:, :, None, :])) * sc.float()[:, :, None, :]
    return v.view(q.shape[0], -1, q.shape[2])


def _plain_moe(s):
    x, topk, gate, E, I = s["x"].float(), s["topk"].long(), s["gate_w"], s["E"], s["I"]
    T, k = topk.shape
    gate = torch.where(topk < 0, 0.0, gate)
    topk = topk.clamp_min(0)
    if T * k < E:       # few pairs: each with its expert's matrices
        ids, rows = topk.flatten(), x.repeat_interleave(k, 0)[:, None, :]
    else:               # every token through every expert
        ids, rows = None, x[None]
        gate = torch.zeros(T, E, device=x.device).scatter_add_(1, topk, gate)
    a = rows @ _weights(s["w13"], s["group"], ids)
    g, u = a[..., :I], a[..., I:]
    y = (g / (1 + torch.exp(-g)) * u) @ _weights(s["w2"], s["group"], ids)
    if ids is not None:
        y = y.view(T, k, -1)
        return (y * gate[:, :, None]).sum(1).to(BF16)
    return (y * gate.t()[:, :, None]).sum(0).to(BF16)


def _plain_matvec(s):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].repeat_interleave(128, 1)[:, : s["K"]]
    w = _weights((s["wq"][None], s["w_scale"][None], None if s["w_zero"] is None else s["w_zero"][None]), s["group"])[0]
    return (x @ w).to(BF16)


_plain = {"norm": _plain_norm, "route": _plain_route, "moe": _plain_moe, "matvec": _plain_matvec}
_own = {"norm": _own_norm, "route": _own_route, "moe": _own_moe, "matvec": _own_matvec}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        res = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
        groups = -(-H // case["group"]) if case["group"] else 1
        return {"bytes": T * H * (2 + 2 * res + 2 + 1) + 2 * H + 4 * T * groups, "flops": 8 * T * H}
    if op == "route":
        return {"bytes": T * case["E"] * (2 if case["dtype"] == "bf16" else 4) + 8 * T * case["k"], "flops": 3 * T * case["E"]}
    if op == "moe":
        E, k, H, I = (case[n] for n in ("E", "k", "H", "I"))
        here = k * (1 - case["absent"])
        read = E * (1 - (1 - here / E) ** T)          # experts that at least one token names
        each = 2.0
        if case["weights"] == "q4":
            each = 0.5 + (3 if case["zeros"] else 2) / case["group"]
        return {"bytes": read * 3 * H * I * each + T * (4 * H + 8 * k), "flops": 6 * T * here * H * I}
    K, N = case["K"], case["N"]
    each = 0.5 + (3 if case["zeros"] else 2) / case["group"]
    x = T * K * 2 if case["x"] == "bf16" else T * (K + 4 * -(-K // 128))
    return {"bytes": K * N * each + x + 2 * T * N, "flops": 2 * T * K * N}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        r = s["x"].to(D) + (0 if s["residual"] is None else s["residual"].to(D))
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / case["H"] + EPS) * s["weight"].to(D)
        scale, q = [], []
        for part in y.split(case["group"] or case["H"], 1):
            sc = torch.clamp(part.abs().max(1).values, min=MIN_AMAX) / E4M3_MAX
            scale.append(sc)
            q.append(part / sc[:, None])
        out = {"out": y, "q": torch.cat(q, 1), "scale": torch.stack(scale, 1)}
        if s["residual"] is not None:
            out["residual"] = r
        return out
    if case["op"] == "route":
        l = s["logits"].to(D)
        bad = torch.isnan(l) | (l == -torch.inf)
        p = torch.softmax(torch.where(bad, torch.full_like(l, -1e300), l), 1).masked_fill(bad, 0.0)
        left, got = l.masked_fill(bad, -torch.inf), []
        for _ in range(case["k"]):
            best = left.max(1, keepdim=True).values
            at = (left == best).to(torch.int8).argmax(1, keepdim=True)     # the first of the largest
            got.append(torch.where(best == -torch.inf, 0.0, p.gather(1, at)))
            left = left.scatter(1, at, -torch.inf)
        w = torch.cat(got, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        return {"topk": None, "gate_w": w}

    def matrix(w, e):
        if isinstance(w, torch.Tensor):
            return w[e].to(D)
        q, sc, z = w
        rows = torch.empty(q.shape[1] * 8, q.shape[2], dtype=D, device=q.device)
        for i in range(8):
            bit = 4 * (i // 2) + 16 * (i % 2)
            rows[i::8] = torch.bitwise_and(torch.bitwise_right_shift(q[e], bit), 15).to(D)
        zero = 8.0 if z is None else z[e].to(D).repeat_interleave(case["group"], 0)
        return (rows - zero) * sc[e].to(D).repeat_interleave(case["group"], 0)

    if case["op"] == "matvec":
        x = s["x"].to(D)
        if s["x_scale"] is not None:
            x = torch.cat([p * s["x_scale"][:, i:i + 1].to(D) for i, p in enumerate(x.split(128, 1))], 1)
        w = (s["wq"][None], s["w_scale"][None], None if s["w_zero"] is None else s["w_zero"][None])
        return x @ matrix(w, 0)
    I = case["I"]
    y = torch.zeros(case["T"], case["H"], dtype=D, device=s["x"].device)
    for e in range(case["E"]):
        t, j = torch.nonzero(s["topk"] == e, as_tuple=True)
        if len(t):
            a = s["x"][t].to(D) @ matrix(s["w13"], e)
            h = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]
            y.index_add_(0, t, (h @ matrix(s["w2"], e)) * s["gate_w"][t, j].to(D)[:, None])
    return y
