"""Decode-step operators at the edges of their kernels' variants, against plain 64-bit implementations.

The tolerances are those of test_gpu_decode.py, error bounds and not fits, with one of their own: with 4-bit
weights h, the activation between the two products, is fp16 times a power of two per 128 columns (2^126 at most),
which brings the largest of them to [2^14, 2^15).  Rounding to the nearest of 11 significant bits is 2^-11 of the
value at most, and below 2^-14 half of a unit of 2^-24, which is 2^-39 of the largest, or 2^-151 where the power
ends.  With bf16 weights h is two bf16 numbers, which leave 2^-16.
"""
import pytest
import torch

from consumer_movement_gemm_gb300 import tovl
from tests.test_gpu_decode import (BF16, D, DEV, E4M3, F32, U16, U32, bf16_experts, gen, guarded, h, packed, randn,  # noqa: F401
                                   routing, space, sum_bound, unpack, within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the expert layer
def moe_bound(x, topk, gate, W13, W2, quant):
    """out and the bound of its error, in 64 bits."""
    T, H = x.shape
    if quant:
        W13, W2 = unpack(*W13, quant), unpack(*W2, quant)
    I = W2.shape[1]
    out = torch.zeros(T, H, dtype=D, device=DEV)
    bound = torch.zeros(T, H, dtype=D, device=DEV)
    for e in torch.unique(topk[topk >= 0]).tolist():
        t, j = torch.nonzero(topk == e, as_tuple=True)
        a, b = x[t].to(D), W13[e].to(D)
        z, dz = a @ b, sum_bound(H, a.abs() @ b.abs())
        zg, zu, dg, du = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
        s = zg * torch.sigmoid(zg)
        hh = s * zu
        # |silu'| <= 1.1; exp and the division: 8 units
        dh = 1.1 * dg * zu.abs() + (s.abs() + 1.1 * dg) * du + (8 * U32 + (2.0 ** -11 if quant else 2.0 ** -16)) * hh.abs()
        if quant:
            top = torch.cat([p.abs().amax(1, keepdim=True).expand_as(p) for p in hh.split(128, 1)], 1)
            dh = dh + 2.0 ** -39 * top + 2.0 ** -151
        w2, w = W2[e].to(D), gate[t, j].to(D)[:, None]
        mag = (hh.abs() + dh) @ w2.abs()
        out.index_add_(0, t, (hh @ w2) * w)
        bound.index_add_(0, t, w.abs() * (dh @ w2.abs() + sum_bound(2 * I, mag)))
    return out, bound + U16 * out.abs() + 2.0 ** -133


def experts(g, E, H, I, quant, zeros=True):
    if quant:
        return packed(g, (E,), H, 2 * I, quant, zeros), packed(g, (E,), I, H, quant, zeros)
    return bf16_experts(g, E, H, I)


def run_moe(h, x, topk, gate, w, quant, out, ws, stream=None):  # noqa: F811
    if quant:
        h.moe_decode_q4(x, topk, gate, *w, quant, out, ws, stream=stream)
    else:
        h.moe_decode(x, topk, gate, *w, out, ws, stream=stream)


def absent(g, topk, share=0.25):
    topk[torch.rand(topk.shape, generator=g, device=DEV) < share] = -1
    return topk


# one pass of the small form takes up to 16 tokens, and up to 32 names are found by every warp by itself: both sides of
# either edge, more experts than one pass can name, and calls that end inside a pass
@pytest.mark.parametrize("T", [8, 9, 15, 16, 17, 20, 31, 32, 33])
@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("E", [4, 19, 62])
@pytest.mark.parametrize("quant", [None, 32])
def test_moe_of_few_names(h, T, k, E, quant):  # noqa: F811
    g = gen(T * 1000 + E * 10 + k)
    H, I = 160, 96
    topk, gate = routing(g, T, E, k)
    absent(g, topk)
    w = experts(g, E, H, I, quant)
    x = torch.full((T + 32, H), float("nan"), dtype=BF16, device=DEV)[:T]      # what lies behind the rows shows where it is used
    x.copy_(randn(g, T, H))
    want, bound = moe_bound(x, topk, gate, *w, quant)
    ws = space(h.moe_decode_workspace(T, k, H, I))
    for _ in range(2):
        out, intact = guarded(T, H)
        run_moe(h, x, topk, gate, w, quant, out, ws)
        assert h.sync_status() == 0
        within(out, want, bound, "out")
        assert intact()


@pytest.mark.parametrize("quant", [None, 64])
def test_moe_of_one_name_a_token(h, quant):  # noqa: F811
    """Top-1 routing: every token an expert of its own, more of them than a pass has tokens, in the two-kernel form."""
    g = gen(61)
    T, E, k, H, I = 32, 32, 1, 512, 256
    topk = torch.randperm(E, generator=g, device=DEV).to(torch.int32)[:, None].contiguous()
    gate = torch.rand(T, k, generator=g, device=DEV) + 0.5
    w, x = experts(g, E, H, I, quant), randn(g, T, H)
    out, ws = torch.empty(T, H, dtype=BF16, device=DEV), space(h.moe_decode_workspace(T, k, H, I))
    run_moe(h, x, topk, gate, w, quant, out, ws)
    assert h.sync_status() == 0
    within(out, *moe_bound(x, topk, gate, *w, quant), "out")


# ------------------------------------------------------------------ norm
# aligned rows a warp and a CTA each, two pieces a thread and more, rows off the boundaries, pairs and single elements
@pytest.mark.parametrize("H,pad", [(384, 0), (1024, 0), (2048, 0), (10240, 0), (20480, 0), (203, 0), (2051, 0), (9001, 0), (2050, 0), (514, 3)])
@pytest.mark.parametrize("group", [32, 128, 0])
def test_norm_rounds_the_quotient(h, H, pad, group):  # noqa: F811
    """Rows of +-1 with eps = 0 give y = +-weight exactly, the groups' largest make the scales small odd numbers, and the
    quotients lie half way between two e4m3 numbers or are such numbers: q is e4m3(y / scale), ties to even."""
    g = gen(H + group)
    T, n = 3, group or H
    pick = lambda values, size: torch.tensor(values, device=DEV)[torch.randint(len(values), (size,), generator=g, device=DEV)]  # noqa: E731
    # odd * 25 and odd * 29 have eight bits at most, as bf16 has; so has 448 * odd
    scale = pick([1.0, 3.0, 5.0, 7.0], -(-H // n))
    ratio = pick([25.0, 29.0, 17.0, 27.0, 16.0, 7.5], H) * torch.exp2(pick([0.0, 1.0, 2.0, 3.0, -5.0, -11.0], H))
    ratio[torch.arange(H, device=DEV) % n == 0] = 448
    ratio *= pick([1.0, -1.0], H)
    weight = (ratio * scale.repeat_interleave(n)[:H]).to(BF16)
    want = weight.to(D) / scale.repeat_interleave(n)[:H].to(D)
    assert torch.equal(want.float(), ratio)
    sign = pick([1.0, -1.0], T * H).view(T, H)
    x = torch.empty(T, H + pad, dtype=BF16, device=DEV)[:, :H]
    x.copy_(sign)
    q, got = torch.empty(T, H, dtype=E4M3, device=DEV), torch.empty(T, len(scale), device=DEV)
    h.add_rmsnorm(x, weight, 0.0, q=q, q_scale=got, group=group)
    assert h.sync_status() == 0
    assert torch.equal(got, scale.expand(T, -1))
    assert torch.equal(q.float(), (sign * ratio).to(E4M3).float())


# ------------------------------------------------------------------ packed weights
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_takes_any_finite_weights(h, group, zeros):  # noqa: F811
    """Columns of every magnitude that bf16 has, ranges over its largest number and below its normal ones."""
    g = gen(group)
    K, N = 256, 32
    top = torch.tensor([3e38, 1e38, 1e30, 1.0, 1e-20, 1e-29, 1e-30, 1e-32, 1e-36, 1e-38, 1e-39, 2.0 ** -130, 2.0 ** -132, 2.0 ** -133, 0.0, 3.3e38],
                       dtype=D, device=DEV).repeat(2)
    w = ((torch.rand(K, N, generator=g, device=DEV).to(D) * 2 - 1) * top).to(BF16)
    w[::group, :] = top.to(BF16)                       # the range is the column's: its ends in every group
    w[1::group, :16] = -top[:16].to(BF16)
    w[:, 16:] = w[:, 16:].abs()
    q, scale, zero = h.quantize_q4(w, group, zeros)
    assert h.sync_status() == 0
    parts = w.float().view(K // group, group, N)
    hi, lo = parts.amax(1).clamp_min(0), parts.amin(1).clamp_max(0)
    want = (hi / 2 - lo / 2) / 7.5 if zeros else torch.maximum(hi, -lo) / 7
    none = want.to(BF16) == 0                          # nothing that bf16 can tell from zero: zeros, under any scale
    assert torch.equal(scale, torch.where(none, 1.0, want).to(BF16))
    got = unpack(q, scale, zero, group)
    # half a level, with zeros half a level more, and what the rounded scale's 7 or 15 levels are short of the range;
    # dividing in fp32 may take a weight over the middle of two levels
    s = scale.to(D)
    bound = s * ((1.0 if zeros else 0.5) + 2.0 ** -18) + (15 if zeros else 7) * (s - want.to(D)).abs()
    within(got, w.to(D), torch.where(none, (hi - lo).to(D), bound).repeat_interleave(group, 0), "quantised weights")
    assert (got.view(K // group, group, N)[none[:, None, :].expand(-1, group, -1)] == 0).all()


# Tokens and layers (7 experts, 3 a token) of the two-kernel form and of the rings: their weights lie on both sides of the
# rule's limits.  The products of 4-bit weights likewise, by their matrix.
FORMS = [(20, 192, 128), (20, 2560, 1600)]
E7, K3 = 7, 3
PRODUCTS = [(512, 256), (8192, 8320)]


def layer(h, g, T, H, I, quant):  # noqa: F811
    topk, gate = routing(g, T, E7, K3)
    return topk, gate, experts(g, E7, H, I, quant), space(h.moe_decode_workspace(T, K3, H, I))


@pytest.mark.parametrize("T,H,I", FORMS)
@pytest.mark.parametrize("quant", [None, 64])
def test_moe_strided_rows_on_a_side_stream(h, T, H, I, quant):  # noqa: F811
    """Rows of x apart, rows of out that allow only single elements; the same bits on every call and any stream."""
    g = gen(H)
    topk, gate, w, ws = layer(h, g, T, H, I, quant)
    x = randn(g, T, H + 72)[:, 24:24 + H]
    want, bound = moe_bound(x, topk, gate, *w, quant)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = None
    for pad, stream in ((8, None), (1, None), (3, side), (8, side)):
        out, intact = guarded(T, H, pad=pad)
        torch.cuda.synchronize()
        run_moe(h, x, topk, gate, w, quant, out, ws, stream=stream)
        assert h.sync_status() == 0
        within(out, want, bound, "out")
        assert intact()
        first = out.clone() if first is None else first
        assert torch.equal(out, first)


@pytest.mark.parametrize("T,H,I", FORMS)
@pytest.mark.parametrize("quant", [None, 64])
def test_moe_takes_any_magnitude_in_either_form(h, T, H, I, quant):  # noqa: F811
    g = gen(H + 1)
    topk, gate, w, ws = layer(h, g, T, H, I, quant)
    size = torch.tensor([1e-18, 1e-6, 1.0, 1e3, 1e9, 1e15], device=DEV).repeat(4)[:T, None]
    x = (torch.randn(T, H, generator=g, device=DEV) * size).to(BF16)
    out = torch.empty(T, H, dtype=BF16, device=DEV)
    run_moe(h, x, topk, gate, w, quant, out, ws)
    assert h.sync_status() == 0
    within(out, *moe_bound(x, topk, gate, *w, quant), "out")


@pytest.mark.parametrize("T,H,I", FORMS + [(3, 192, 128)])
@pytest.mark.parametrize("quant", [None, 64])
@pytest.mark.parametrize("bad", [E7, -2, 2 ** 31 - 1, -2 ** 31])
def test_moe_refuses_ids_outside(h, T, H, I, quant, bad):  # noqa: F811
    """More and fewer than 32 names, in either form: nothing written, an error status, and the next call is right."""
    g = gen(H + 2)
    topk, gate, w, ws = layer(h, g, T, H, I, quant)
    x, out = randn(g, T, H), torch.full((T, H), 5.0, dtype=BF16, device=DEV)
    worse = topk.clone()
    worse[T - 1, 1] = bad
    run_moe(h, x, worse, gate, w, quant, out, ws)
    assert h.sync_status() == tovl.TOVL_ERR_INVALID
    assert (out == 5).all()
    run_moe(h, x, topk, gate, w, quant, out, ws)
    assert h.sync_status() == 0
    within(out, *moe_bound(x, topk, gate, *w, quant), "out")


# ------------------------------------------------------------------ 4-bit products
def product(h, g, T, K, N, e4m3):  # noqa: F811
    """Rows, their scales, a packed matrix, a workspace."""
    x, xs = randn(g, T, K), None
    if e4m3:
        x = (torch.randn(T, K, generator=g, device=DEV) * 100).clamp_(-448, 448).to(E4M3)
        xs = (torch.rand(T, -(-K // 128), generator=g, device=DEV) + 0.5) * 0.01
    return x, xs, packed(g, (), K, N, 64, True), space(h.matvec_q4_workspace(T, N))


def product_bound(x, xs, w):
    W, xd = unpack(*w, 64), x.float().to(D)
    if xs is not None:
        xd = xd * xs.to(D).repeat_interleave(128, 1)[:, :x.shape[1]]
    want = xd @ W
    return want, U16 * want.abs() + 2.0 ** -133 + sum_bound(x.shape[1] + x.shape[1] / 64 * 16, xd.abs() @ W.abs())


@pytest.mark.parametrize("K,N", PRODUCTS)
@pytest.mark.parametrize("e4m3", [False, True])
def test_matvec_strided_rows_on_a_side_stream(h, K, N, e4m3):  # noqa: F811
    g = gen(K + 3)
    T = 18
    x, xs, w, ws = product(h, g, T, K, N, e4m3)
    x = torch.cat([x, x[:, :96]], 1)[:, :K]              # rows K + 96 apart
    want, bound = product_bound(x, xs, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = None
    for pad, stream in ((8, None), (1, None), (3, side), (8, side)):
        out, intact = guarded(T, N, pad=pad)
        torch.cuda.synchronize()
        h.matvec_q4(x, w[0], w[1], 64, out, ws, zero=w[2], x_scale=xs, stream=stream)
        assert h.sync_status() == 0
        within(out, want, bound, "out")
        assert intact()
        first = out.clone() if first is None else first
        assert torch.equal(out, first)


# ------------------------------------------------------------------ together
class Jobs:
    """Layers and products of both forms and both weight types, on one workspace and one handle."""

    def __init__(self, h, g, rows):  # noqa: F811
        self.h, self.calls = h, []
        sizes = []
        for (_, H, I), T, quant in [(f, T, q) for f in FORMS for T in rows for q in (None, 64)]:
            topk, gate, w, ws = layer(h, g, T, H, I, quant)
            self.calls.append(("moe", randn(g, T, H), topk, gate, w, quant, torch.empty(T, H, dtype=BF16, device=DEV)))
            sizes.append(len(ws))
        for (K, N), T, e4m3 in [(p, T, e) for p in PRODUCTS for T in rows for e in (False, True)]:
            x, xs, w, ws = product(h, g, T, K, N, e4m3)
            self.calls.append(("product", x, xs, w, torch.empty(T, N, dtype=BF16, device=DEV)))
            sizes.append(len(ws))
        self.ws = space(max(sizes))
        order = torch.randperm(len(self.calls), generator=torch.Generator().manual_seed(3)).tolist()
        self.calls = [self.calls[i] for i in order]

    def run(self):
        for kind, *c in self.calls:
            if kind == "moe":
                x, topk, gate, w, quant, out = c
                run_moe(self.h, x, topk, gate, w, quant, out, self.ws)
            else:
                x, xs, w, out = c
                self.h.matvec_q4(x, w[0], w[1], 64, out, self.ws, zero=w[2], x_scale=xs)

    def new_rows(self, g):
        for kind, x, *c in self.calls:
            x.copy_(randn(g, *x.shape) if x.dtype is BF16 else randn(g, *x.shape, scale=100, dtype=F32).clamp_(-448, 448))
            if kind == "moe":
                c[0].copy_(routing(g, len(x), E7, K3)[0])

    def check(self):
        assert self.h.sync_status() == 0
        for kind, *c in self.calls:
            want, bound = moe_bound(*c[:3], *c[3], c[4]) if kind == "moe" else product_bound(*c[:3])
            within(c[-1], want, bound, kind)

    def outputs(self):
        return [c[-1] for c in self.calls]


def test_back_to_back_calls_of_both_forms(h):  # noqa: F811
    """Calls in a row without a synchronisation share the handle's counters and a workspace; the same bits every time."""
    jobs = Jobs(h, gen(71), (9, 24))
    jobs.run()
    jobs.check()
    first = [o.clone() for o in jobs.outputs()]
    for _ in range(5):
        for o in jobs.outputs():
            o.zero_()
        for _ in range(2):
            jobs.run()
        assert h.sync_status() == 0
        assert all(torch.equal(o, f) for o, f in zip(jobs.outputs(), first))


@pytest.mark.parametrize("option,value", [(None, None), (tovl.OPT_COOPERATIVE, 0), (tovl.OPT_PDL, 0)])
def test_a_decode_step_in_a_graph(option, value):
    """Norm, router, layers and products of both forms captured once and replayed on new inputs, also without the cooperative
    attribute and without programmatic launches."""
    g = gen(72)
    with tovl.Handle(0, max_rows=4096, max_pairs=4096) as h:  # noqa: F811
        if option is not None:
            h.set_option(option, value)
        jobs = Jobs(h, g, (12,))
        T, H, E, k = 12, 1280, 32, 4
        x, res, weight = randn(g, T, H), randn(g, T, H, dtype=F32), randn(g, H, scale=0.1) + 1
        ro, y = torch.empty_like(res), torch.empty_like(x)
        logits, topk, gate = randn(g, T, E, dtype=F32), torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)

        def step():
            h.add_rmsnorm(x, weight, 1e-5, residual=res, residual_out=ro, out=y)
            h.route_topk(logits, topk, gate)
            jobs.run()

        step()
        assert h.sync_status() == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for seed in (1, 2):
            g = gen(seed)
            x.copy_(randn(g, T, H)), res.copy_(randn(g, T, H, dtype=F32)), logits.copy_(randn(g, T, E, dtype=F32))
            jobs.new_rows(g)
            graph.replay()
            torch.cuda.synchronize()
            jobs.check()
            r = x.to(D) + res.to(D)
            want = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-5) * weight.to(D)
            within(y, want, (U16 + (H + 24) * U32) * want.abs(), "norm")
            p, ids = torch.softmax(logits.to(D), 1).topk(k)
            assert torch.equal(topk.long(), ids)
            p = p / p.sum(1, keepdim=True)
            # exp (2 units and the rounded difference of arguments below 20), a sum of four, one division
            within(gate, p, 32 * U32 * p, "gate_w")


# ------------------------------------------------------------------ sizes at the end of int
def test_route_and_norm_of_as_many_rows_as_there_can_be(h):  # noqa: F811
    """2^31 - 1 rows: neither the grid's size nor an offset wraps."""
    T = 2 ** 31 - 1
    logits = torch.zeros(T, 1, dtype=BF16, device=DEV)
    topk, gate = torch.full((T, 1), 7, dtype=torch.int32, device=DEV), torch.zeros(T, 1, device=DEV)
    h.route_topk(logits, topk, gate)
    assert h.sync_status() == 0
    assert int(topk.max()) == 0 and int(topk.min()) == 0 and float(gate.min()) == 1 and float(gate.max()) == 1
    del topk, gate
    x, out, weight = logits.fill_(2), torch.empty(T, 1, dtype=BF16, device=DEV), torch.full((1,), 3, dtype=BF16, device=DEV)
    h.add_rmsnorm(x, weight, 0.0, out=out)                # contiguous rows: pieces
    assert h.sync_status() == 0
    assert float(out.min()) == 3 and float(out.max()) == 3
    out.zero_()
    h.add_rmsnorm(x, torch.full((2,), 3, dtype=BF16, device=DEV)[1:], 0.0, out=out)       # a weight off the boundary: elements
    assert h.sync_status() == 0
    assert float(out.min()) == 3 and float(out.max()) == 3
    del x, out, logits
    torch.cuda.empty_cache()
