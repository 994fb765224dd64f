"""Decode-step operators against plain 64-bit implementations.

Tolerances are error bounds, not fits:
  * a product of n terms summed in fp32: the tensor core adds 16 products at a
    time and truncates, so at most n/16 additions (plus fewer than 64 between
    warps, groups and parts) each lose 2^-23 of a partial sum, which is at most
    the sum of the terms' magnitudes;
  * a result rounded to bf16: 2^-8 of itself at most (half a unit is 2^-9, and
    the error before it may move it across one boundary); below 2^-126 the unit
    is 2^-133 whatever the value;
  * e4m3: half a unit, 2^-4 of the value or 2^-10 among the subnormals.
"""
import math

import pytest
import torch

from consumer_movement_gemm_gb300 import tovl

pytestmark = pytest.mark.gpu

DEV = "cuda"
D = torch.float64
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U32 = 2.0 ** -23
U16 = 2.0 ** -8


@pytest.fixture(scope="module")
def h():
    from consumer_movement_gemm_gb300 import build
    build.build()
    with tovl.Handle(0, max_rows=4096, max_pairs=4096) as handle:
        yield handle


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def guarded(T, N, dtype=BF16, pad=16):
    """A [T, N] view inside a larger buffer of a known pattern, and a check that nothing around it changed."""
    buf = torch.full((T + 2, N + 2 * pad), 3.0, device=DEV).to(dtype)
    view = buf[1:T + 1, pad:pad + N]

    def intact():
        ring = buf.clone()
        ring[1:T + 1, pad:pad + N] = 3.0
        return bool((ring.float() == 3.0).all())

    return view, intact


def within(got, want, bound, what):
    err = (got.to(D) - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at "
                           f"{tuple(int(i) for i in bad.nonzero()[0])}: {got[bad][0].item()} for {want[bad][0].item()}")


def sum_bound(n, magnitude):
    return (n / 16 + 64) * U32 * magnitude


# ------------------------------------------------------------------ norm
def norm_reference(x, weight, eps, residual):
    r = x.to(D) + (0 if residual is None else residual.to(D))
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * weight.to(D)
    return r, y


def check_norm(x, weight, eps, residual, residual_out, out, q, scale, group):
    T, H = x.shape
    r, y = norm_reference(x, weight, eps, residual)
    # r once, the squares' sum ((H + 16) additions at most), rsqrt (2 units), two products
    rel = (H + 24) * U32
    if residual is not None:
        within(residual_out, r, (U16 if residual.dtype == BF16 else U32) * r.abs(), "residual_out")
    if out is not None:
        within(out, y, (U16 + rel) * y.abs(), "out")
    if q is not None:
        group = group or H
        for i, (part, qp) in enumerate(zip(y.split(group, 1), q.float().split(group, 1))):
            want = part.abs().amax(1).clamp_min(1e-12) / 448
            within(scale[:, i], want, (rel + 4 * U32) * want, "scale")
            v = part / want[:, None]
            within(qp, v, 2.0 ** -4 * v.abs().clamp_min(2.0 ** -6) + 448 * (rel + 8 * U32), "q")


@pytest.mark.parametrize("T,H", [(1, 1), (1, 8), (3, 7), (5, 100), (70, 64), (2, 1000), (17, 1024), (9, 1032), (2, 1130),
                                 (4, 4096), (3, 7168), (2, 8200), (2, 9001), (2, 16384), (1, 32766), (2, 32768)])
@pytest.mark.parametrize("group,residual", [(128, "bf16"), (64, "f32"), (32, "none"), (0, "bf16")])
def test_norm_matches_the_formula(h, T, H, group, residual):
    g = gen(T * 100003 + H)
    x, weight = randn(g, T, H), randn(g, H) + 1
    res = None if residual == "none" else randn(g, T, H, scale=3, dtype=BF16 if residual == "bf16" else F32)
    ro = None if res is None else torch.empty_like(res)
    out, q = torch.empty_like(x), torch.empty(T, H, dtype=E4M3, device=DEV)
    scale = torch.empty(T, -(-H // group) if group else 1, device=DEV)
    h.add_rmsnorm(x, weight, 1e-5, residual=res, residual_out=ro, out=out, q=q, q_scale=scale, group=group)
    assert h.sync_status() == 0
    check_norm(x, weight, 1e-5, res, ro, out, q, scale, group)


@pytest.mark.parametrize("H,off,pad", [(4096, 8, 8), (4096, 2, 6), (1000, 1, 7), (520, 3, 2), (40, 0, 24)])
def test_norm_strided_and_misaligned_rows(h, H, off, pad):
    g = gen(H + off)
    T = 6
    big = randn(g, T, off + H + pad)
    x = big[:, off:off + H]
    weight = randn(g, H + off)[off:]
    res = randn(g, T, off + H + pad)[:, off:off + H]
    ro, intact_ro = guarded(T, H, pad=off + 1)
    res2, _ = guarded(T, H, pad=off + 1)
    res2.copy_(res)
    out, intact = guarded(T, H, pad=off + 1)
    h.add_rmsnorm(x, weight, 1e-6, residual=res2, residual_out=ro, out=out)
    assert h.sync_status() == 0
    assert intact() and intact_ro()
    check_norm(x, weight, 1e-6, res2, ro, out, None, None, 0)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("H", [9, 15, 33, 121, 127, 249, 250, 257, 393, 777, 1002, 1017, 1018, 1019, 1023, 2049, 4089, 4111, 8177,
                               8185, 8186, 8191, 12001, 16377, 16379])
@pytest.mark.parametrize("group,residual", [(128, "bf16"), (64, "f32"), (32, "none"), (0, "f32")])
def test_norm_of_odd_rows(h, T, H, group, residual):
    """Rows off the 16-byte boundaries, contiguous (every tensor the same distance off) and with x alone strided."""
    g = gen(T * 100003 + H)
    weight = randn(g, H) + 1
    for pad in (0, 3):
        x = randn(g, T, H + pad)[:, :H]
        res = None if residual == "none" else randn(g, T, H, scale=3, dtype=BF16 if residual == "bf16" else F32)
        ro = None if res is None else torch.empty_like(res)
        out, q = torch.empty(T, H, dtype=BF16, device=DEV), torch.full((T * H + 8,), 99, dtype=torch.uint8, device=DEV)
        scale = torch.full((T, -(-H // group) if group else 1), float("nan"), device=DEV)
        h.add_rmsnorm(x, weight, 1e-5, residual=res, residual_out=ro, out=out, q=q[:T * H].view(E4M3).view(T, H), q_scale=scale,
                      group=group)
        assert h.sync_status() == 0
        check_norm(x, weight, 1e-5, res, ro, out, q[:T * H].view(E4M3).view(T, H), scale, group)
        assert (q[T * H:] == 99).all()
        if res is not None and pad == 0:          # in place: the same bits
            x2, res2 = x.clone(), res.clone()
            h.add_rmsnorm(x2, weight, 1e-5, residual=res2, residual_out=res2, out=x2)
            assert torch.equal(x2, out) and torch.equal(res2, ro)


@pytest.mark.parametrize("H,off", [(64, 1), (128, 7), (776, 3), (1024, 5), (2048, 1), (4104, 6), (8176, 3)])
@pytest.mark.parametrize("group,residual", [(128, "bf16"), (32, "f32"), (0, "none")])
def test_norm_rows_equally_far_from_a_boundary(h, H, off, group, residual):
    """Whole multiples of eight elements, every tensor `off` elements past a 16-byte boundary."""
    g = gen(H + off)
    T, ld = 5, H + 8

    def shifted(dtype, fill=None):
        t = torch.full((T * ld + 32,), 7.0 if fill is None else fill, dtype=dtype, device=DEV)
        return t, t[off:off + T * ld].view(T, ld)[:, :H]

    weight = randn(g, H) + 1
    _, x = shifted(BF16)
    x.copy_(randn(g, T, H))
    res = ro = None
    if residual != "none":
        dtype = BF16 if residual == "bf16" else F32
        _, res = shifted(dtype)
        res.copy_(randn(g, T, H, scale=3, dtype=dtype))
        ro_all, ro = shifted(dtype)
    out_all, out = shifted(BF16)
    q_all = torch.full((T * H + 32,), 99, dtype=torch.uint8, device=DEV)
    q = q_all[off:off + T * H].view(E4M3).view(T, H)
    scale = torch.full((T, -(-H // group) if group else 1), float("nan"), device=DEV)
    h.add_rmsnorm(x, weight, 1e-5, residual=res, residual_out=ro, out=out, q=q, q_scale=scale, group=group)
    assert h.sync_status() == 0
    check_norm(x, weight, 1e-5, res, ro, out, q, scale, group)
    out.fill_(7.0), q_all[off:off + T * H].fill_(99)
    assert (out_all == 7).all() and (q_all == 99).all()
    if ro is not None:
        ro.fill_(7.0)
        assert (ro_all == 7).all()


def test_norm_in_place_and_single_outputs(h):
    g = gen(5)
    x, weight, res = randn(g, 9, 768), randn(g, 768), randn(g, 9, 768)
    x0, res0 = x.clone(), res.clone()
    h.add_rmsnorm(x, weight, 1e-5, residual=res, residual_out=res, out=x)
    check_norm(x0, weight, 1e-5, res0, res, x, None, None, 0)
    q, scale = torch.empty(9, 768, dtype=E4M3, device=DEV), torch.empty(9, 6, device=DEV)
    h.add_rmsnorm(x0, weight, 1e-5, q=q, q_scale=scale)
    assert h.sync_status() == 0
    check_norm(x0, weight, 1e-5, None, None, None, q, scale, 128)


def test_norm_zeros_infinities_and_nan(h):
    T, H = 5, 300
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    x[1] = 1e-30                    # squares vanish; eps 0 would divide by zero
    x[2, 7] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1.0
    weight = torch.ones(H, dtype=BF16, device=DEV)
    out, q = torch.empty_like(x), torch.empty(T, H, dtype=E4M3, device=DEV)
    scale = torch.empty(T, 3, device=DEV)
    h.add_rmsnorm(x, weight, 1e-5, out=out, q=q, q_scale=scale)
    assert h.sync_status() == 0
    assert (out[0] == 0).all() and (q[0].float() == 0).all()
    assert torch.equal(scale[0], torch.full((3,), 1e-12, device=DEV) / 448)
    assert torch.isfinite(out[1].float()).all() and torch.isfinite(scale[1]).all()
    assert torch.isnan(out[2].float()).all() and torch.isnan(scale[2]).all() and torch.isnan(q[2].float()).all()
    # an infinite element: 0 for the finite ones, NaN for itself
    assert torch.isnan(out[3, 7].float()) and (out[3, :7] == 0).all() and torch.isnan(scale[3, 0]) and scale[3, 1] > 0
    assert ((out[4].float() - 1).abs() < 0.01).all()


# ------------------------------------------------------------------ route
def route_reference(logits, k, renorm):
    l = logits.to(D)
    l = torch.where(torch.isnan(l), -math.inf, l)
    T, E = l.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=D)
    for t, row in enumerate(l.cpu().tolist()):
        m = max(row)
        p = [0.0 if v == -math.inf else 1.0 if v == m else math.exp(v - m) for v in row]
        order = sorted((i for i in range(E) if row[i] != -math.inf), key=lambda i: (-row[i], i))[:k]
        total = sum(p[i] for i in order) if renorm else sum(p)
        for j, i in enumerate(order):
            ids[t, j], w[t, j] = i, p[i] / total
    return ids, w


def check_route(h, logits, k, renorm):
    T = logits.shape[0]
    topk = torch.full((T, k), 77, dtype=torch.int32, device=DEV)
    gate = torch.full((T, k), 77.0, device=DEV)
    h.route_topk(logits, topk, gate, renormalize=renorm)
    assert h.sync_status() == 0
    ids, w = route_reference(logits, k, renorm)
    assert torch.equal(topk.cpu(), ids)
    # exp (2 units and the rounded difference: at most 100 units of argument), the sum of up to 512, one division
    within(gate.cpu(), w, (512 + 128) * U32 * w + 1e-37, "gate_w")
    return topk, gate


@pytest.mark.parametrize("E", [1, 2, 7, 8, 9, 16, 24, 31, 32, 33, 64, 100, 128, 200, 256, 300, 384, 511, 512])
@pytest.mark.parametrize("dtype,k,renorm", [(F32, 4, True), (BF16, 8, False), (BF16, 1, True), (F32, 32, False)])
def test_route_matches_the_formula(h, E, dtype, k, renorm):
    check_route(h, randn(gen(E), 37, E, scale=2, dtype=dtype), k, renorm)


@pytest.mark.parametrize("E", [5, 32, 160, 256, 512])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_ties_masks_and_special_values(h, E, dtype):
    inf, low = float("inf"), torch.finfo(dtype).min
    rows = [torch.zeros(E), torch.full((E,), -inf), torch.full((E,), low), torch.full((E,), float("nan")),
            torch.full((E,), inf), torch.arange(E).float() // 3]
    one = torch.full((E,), -inf)
    one[E - 1] = low
    signed = torch.zeros(E)
    signed[::2] = -0.0
    mixed = torch.linspace(-5, 5, E)
    mixed[1::3], mixed[E // 2] = -inf, float("nan")
    top = torch.zeros(E)
    top[E // 3] = inf
    far = torch.full((E,), -1e30)
    far[0] = 1e30
    logits = torch.stack(rows + [one, signed, mixed, top, far, -mixed.nan_to_num(nan=0.0, neginf=9.0)]).to(dtype).to(DEV)
    for k, renorm in [(3, True), (8, False), (E if E <= 32 else 32, True)]:
        topk, gate = check_route(h, logits, k, renorm)
        assert (topk[1] == -1).all() and (gate[1] == 0).all() and (topk[3] == -1).all()
        n = min(k, E)
        assert topk[0, :n].tolist() == list(range(n)) and topk[7, :n].tolist() == list(range(n))


def test_route_strided_rows_and_every_row_of_many(h):
    g = gen(9)
    big = randn(g, 700, 75, scale=2, dtype=F32)
    check_route(h, big[:, 3:67], 6, True)
    check_route(h, big[:, 0:64].to(BF16), 6, False)


# ------------------------------------------------------------------ packed weights
def unpack(q, scale, zero, group):
    """The matrices that packed words stand for, in 64 bits."""
    lead, K8, N = q.shape[:-2], q.shape[-2], q.shape[-1]
    v = torch.empty(*lead, K8 * 8, N, dtype=D, device=q.device)
    for i in range(8):
        v[..., i::8, :] = ((q >> (4 * (i // 2) + 16 * (i % 2))) & 15).to(D)
    z = 8.0 if zero is None else zero.to(D).repeat_interleave(group, -2)
    return (v - z) * scale.to(D).repeat_interleave(group, -2)


def packed(g, lead, K, N, group, zeros):
    q = torch.randint(-2**31, 2**31 - 1, (*lead, K // 8, N), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    scale = (torch.rand(*lead, K // group, N, generator=g, device=DEV) + 0.5).mul_(0.3 / K ** 0.5).to(BF16)
    zero = torch.randint(0, 16, (*lead, K // group, N), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    return q, scale, zero


@pytest.mark.parametrize("lead,K,N,group", [((), 32, 16, 32), ((3,), 256, 80, 64), ((2,), 384, 304, 128)])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_is_the_nearest_level(h, lead, K, N, group, zeros):
    w = randn(gen(K + N), *lead, K, N)
    w[..., :group, 1] = 0
    w[..., :group, 2] = w[..., :group, 2].abs() + 1
    q, scale, zero = h.quantize_q4(w, group, zeros)
    assert h.sync_status() == 0
    got = unpack(q, scale, zero, group)
    s = scale.to(D).repeat_interleave(group, -2)
    # half a level inside the range; the range itself is short of the weights by the rounding of scale (2^-8 of 7 or
    # 15 levels) and, with zeros, by the rounding of zero (half a level)
    within(got, w.to(D), s * (1.1 if zeros else 0.5 + 7 * U16) + 1e-12, "quantised weights")
    assert (got[..., :group, 1] == 0).all()
    nib = torch.stack([(q >> (4 * i)) & 15 for i in range(8)])
    assert int(nib.max()) <= 15 and (zeros or int(nib.min()) >= 1)


# ------------------------------------------------------------------ matvec
def check_matvec(h, x, xs, w, group, out, workspace, intact=None, stream=None):
    q, scale, zero = w
    h.matvec_q4(x, q, scale, group, out, workspace, zero=zero, x_scale=xs, stream=stream)
    assert h.sync_status() == 0
    W = unpack(q, scale, zero, group)
    xd = x.float().to(D)
    if xs is not None:
        xd = xd * xs.to(D).repeat_interleave(128, 1)[:, :x.shape[1]]
    want = xd @ W
    bound = U16 * want.abs() + 2.0 ** -133 + sum_bound(x.shape[1] + x.shape[1] / group * 16, xd.abs() @ W.abs())
    within(out, want, bound, "out")
    assert intact is None or intact()


def space(n):
    return torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)     # any content


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64])
@pytest.mark.parametrize("K,N,group,zeros,kind", [(32, 16, 32, True, "bf16"), (416, 8, 32, False, "bf16"),
                                                  (1024, 144, 128, True, "e4m3"), (2112, 1040, 64, False, "bf16"),
                                                  (128, 4112, 128, True, "bf16"), (672, 72, 32, False, "e4m3")])
def test_matvec_matches_the_formula(h, T, K, N, group, zeros, kind):
    g = gen(T * 7 + K + N)
    xs = None
    if kind == "bf16":
        x = randn(g, T, K)
    else:
        x = randn(g, T, K, scale=100, dtype=F32).clamp_(-448, 448).to(E4M3)
        xs = (torch.rand(T, -(-K // 128), generator=g, device=DEV) + 0.5) * 0.01
    out, intact = guarded(T, N)
    check_matvec(h, x, xs, packed(g, (), K, N, group, zeros), group, out, space(h.matvec_q4_workspace(T, N)), intact)


def test_matvec_strided_rows_large_and_repeated(h):
    g = gen(21)
    K, N, T = 4096, 4096, 5
    x = randn(g, T, K + 64)[:, 8:8 + K]
    w = packed(g, (), K, N, 128, False)
    out, intact = guarded(T, N)
    ws = space(h.matvec_q4_workspace(T, N))
    check_matvec(h, x, None, w, 128, out, ws, intact)
    first = out.clone()
    for _ in range(5):       # the same bits every time
        out.zero_()
        h.matvec_q4(x, w[0], w[1], 128, out, ws)
        assert torch.equal(out, first)


def test_matvec_rows_do_not_touch_each_other(h):
    g = gen(22)
    K, N, T = 256, 64, 6
    w = packed(g, (), K, N, 64, False)
    x = randn(g, T, K)
    x[2, 5], x[4, 9] = float("inf"), float("nan")
    out = torch.empty(T, N, dtype=BF16, device=DEV)
    ws = space(h.matvec_q4_workspace(T, N))
    h.matvec_q4(x, w[0], w[1], 64, out, ws)
    assert torch.isnan(out[4].float()).all() and not torch.isfinite(out[2].float()).any()
    keep = [0, 1, 3, 5]
    check_matvec(h, x[keep], None, w, 64, torch.empty(4, N, dtype=BF16, device=DEV), ws)
    assert torch.isfinite(out[keep].float()).all()


def test_matvec_takes_any_magnitude(h):
    """bf16 rows of 1e-30 and 1e30, and rows whose elements span 2^40, inside the bound of the fp32 sums: the
    activations' 16-bit form inside the kernel has to carry its own exponent."""
    g = gen(24)
    K, N, T = 512, 96, 9
    x = randn(g, T, K, dtype=F32)
    x[0] *= 1e-30
    x[1] *= 1e30
    x[2, ::2] *= 2.0 ** -40
    x[3] *= torch.exp2(torch.randint(-60, 60, (K,), generator=g, device=DEV).float())
    x[4, :128], x[4, 128:256] = 0, x[4, 128:256] * 1e20
    x[5] = 2.0 ** -126
    x[6] = 3e38 * torch.sign(x[6])
    w = packed(g, (), K, N, 128, True)
    w = (w[0], (w[1].float() * 2.0 ** -8).to(BF16), w[2])
    check_matvec(h, x.to(BF16), None, w, 128, torch.empty(T, N, dtype=BF16, device=DEV), space(h.matvec_q4_workspace(T, N)))


@pytest.mark.parametrize("T,K,N,kind", [(3, 8192, 131072 + 16, "bf16"), (17, 8192, 131072, "e4m3")])
def test_matvec_large_enough_for_tickets(h, T, K, N, kind):
    """Over 3 MB of weights a CTA: most items are taken by ticket; the bits stay the same."""
    g = gen(T)
    xs = None
    if kind == "bf16":
        x = randn(g, T, K)
    else:
        x = randn(g, T, K, scale=100, dtype=F32).clamp_(-448, 448).to(E4M3)
        xs = (torch.rand(T, K // 128, generator=g, device=DEV) + 0.5) * 0.01
    w = packed(g, (), K, N, 128, kind == "bf16")
    out, ws = torch.empty(T, N, dtype=BF16, device=DEV), space(h.matvec_q4_workspace(T, N))
    check_matvec(h, x, xs, w, 128, out, ws)
    first = out.clone()
    for _ in range(3):
        out.zero_()
        h.matvec_q4(x, w[0], w[1], 128, out, ws, zero=w[2], x_scale=xs)
        assert torch.equal(out, first)


def matvec_inputs(g, T, K, kind):
    if kind == "bf16":
        return randn(g, T, K), None
    x = randn(g, T, K, scale=100, dtype=F32).clamp_(-448, 448).to(E4M3)
    return x, (torch.rand(T, -(-K // 128), generator=g, device=DEV) + 0.5) * 0.01


# both sides of 2^26 weights (counted once per 16 rows), where another kernel begins
@pytest.mark.parametrize("T,K,N,group,zeros,kind", [
    (2, 16416, 4112, 32, True, "bf16"), (8, 8192, 8184, 64, False, "bf16"), (8, 8192, 8192, 64, False, "bf16"),
    (9, 10240, 6560, 128, True, "e4m3"), (16, 16384, 4104, 32, False, "e4m3"), (17, 5888, 5712, 128, False, "e4m3"),
    (33, 4832, 4640, 32, True, "e4m3"), (48, 4800, 4672, 64, True, "bf16"), (64, 4160, 4104, 64, False, "bf16"),
    (64, 4096, 4080, 128, True, "bf16")])
def test_matvec_of_large_matrices(h, T, K, N, group, zeros, kind):
    g = gen(T + K + N)
    x, xs = matvec_inputs(g, T, K, kind)
    out, intact = guarded(T, N)
    check_matvec(h, x, xs, packed(g, (), K, N, group, zeros), group, out, space(h.matvec_q4_workspace(T, N)), intact)


# few columns (their rows are shared out to several CTAs) and many (smaller CTAs)
@pytest.mark.parametrize("K,N,group", [(28672, 16, 128), (16416, 48, 32), (4224, 1040, 64), (2176, 2432, 128), (512, 8208, 64),
                                       (160, 20000, 32)])
@pytest.mark.parametrize("T,kind", [(1, "bf16"), (7, "e4m3"), (12, "bf16"), (16, "e4m3"), (40, "bf16")])
def test_matvec_of_few_and_many_columns(h, K, N, group, T, kind):
    g = gen(T + K + N)
    x, xs = matvec_inputs(g, T, K, kind)
    out, intact = guarded(T, N)
    w = packed(g, (), K, N, group, T != 12)
    ws = space(h.matvec_q4_workspace(T, N))
    check_matvec(h, x, xs, w, group, out, ws, intact)
    first = out.clone()
    h.matvec_q4(x, w[0], w[1], group, out, ws, zero=w[2], x_scale=xs)
    assert torch.equal(out, first)


def test_matvec_of_large_matrices_takes_any_magnitude(h):
    g = gen(25)
    K, N, T = 4096, 4112, 64
    x = randn(g, T, K, dtype=F32)
    x *= torch.exp2(torch.randint(-100, 100, (T, 1), generator=g, device=DEV).float())
    x[3] *= torch.exp2(torch.randint(-20, 20, (K,), generator=g, device=DEV).float())
    x[5], x[6, :2048], x[7, 40], x[8, 41] = 0, 0, float("inf"), float("nan")
    w = packed(g, (), K, N, 128, True)
    w = (w[0], (w[1].float() * 2.0 ** -8).to(BF16), w[2])
    out, ws = torch.empty(T, N, dtype=BF16, device=DEV), space(h.matvec_q4_workspace(T, N))
    h.matvec_q4(x.to(BF16), w[0], w[1], 128, out, ws, zero=w[2])
    assert torch.isnan(out[8].float()).all() and not torch.isfinite(out[7].float()).any()
    keep = [i for i in range(T) if i not in (7, 8)]
    clean = x.clone()
    clean[7], clean[8] = 1, 1
    again = torch.empty_like(out)
    check_matvec(h, clean.to(BF16), None, w, 128, again, ws)
    assert torch.equal(out[keep], again[keep])


def test_norm_rows_feed_the_matvec(h):
    """The 8-bit rows and scales of the norm are the 8-bit rows and scales that the product takes."""
    g = gen(23)
    T, H, N = 11, 1280, 512
    x, weight = randn(g, T, H), randn(g, H)
    q, scale = torch.empty(T, H, dtype=E4M3, device=DEV), torch.empty(T, 10, device=DEV)
    h.add_rmsnorm(x, weight, 1e-5, q=q, q_scale=scale)
    check_matvec(h, q, scale, packed(g, (), H, N, 128, True), 128, torch.empty(T, N, dtype=BF16, device=DEV),
                 space(h.matvec_q4_workspace(T, N)))


# ------------------------------------------------------------------ the expert layer
def moe_reference(x, topk, gate, W13, W2):
    """out and the bound of its error, in 64 bits; W13 [E, H, 2I], W2 [E, I, H] (any type)."""
    T, H = x.shape
    I = W2.shape[1]
    out = torch.zeros(T, H, dtype=D, device=DEV)
    bound = torch.zeros(T, H, dtype=D, device=DEV)
    for e in torch.unique(topk[topk >= 0]).tolist():
        t, j = torch.nonzero(topk == e, as_tuple=True)
        a, b = x[t].to(D), W13[e].to(D)
        z = a @ b
        dz = sum_bound(H, a.abs() @ b.abs())
        zg, zu, dg, du = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
        s = zg * torch.sigmoid(zg)
        hh = s * zu
        # |silu'| <= 1.1; exp and the division: 8 units; the pair of bf16 parts leaves 2^-16
        dh = 1.1 * dg * zu.abs() + (s.abs() + 1.1 * dg) * du + (8 * U32 + 2.0 ** -16) * hh.abs()
        w2, w = W2[e].to(D), gate[t, j].to(D)[:, None]
        mag = (hh.abs() + dh) @ w2.abs()
        out.index_add_(0, t, (hh @ w2) * w)
        bound.index_add_(0, t, w.abs() * (dh @ w2.abs() + sum_bound(2 * I, mag)))
    return out, bound + U16 * out.abs()


def check_moe(h, x, topk, gate, W13, W2, quant=None, out=None, stream=None):
    """quant: group of packed W13 and W2."""
    T, H = x.shape
    I = W2.shape[1] if quant is None else W2[0].shape[1] * 8
    ws = space(h.moe_decode_workspace(T, topk.shape[1], H, I))
    out, intact = guarded(T, H) if out is None else (out, lambda: True)
    if quant is None:
        h.moe_decode(x, topk, gate, W13, W2, out, ws, stream=stream)
        want, bound = moe_reference(x, topk, gate, W13, W2)
    else:
        h.moe_decode_q4(x, topk, gate, W13, W2, quant, out, ws, stream=stream)
        want, bound = moe_reference(x, topk, gate, unpack(*W13, quant), unpack(*W2, quant))
    assert h.sync_status() == 0
    within(out, want, bound, "out")
    assert intact()
    return out


def routing(g, T, E, k):
    topk = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    return topk, torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)


def bf16_experts(g, E, H, I):
    return randn(g, E, H, 2 * I, scale=H ** -0.5), randn(g, E, I, H, scale=I ** -0.5)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 8, 8), (1, 2, 1, 64, 64), (1, 8, 2, 512, 256), (3, 8, 2, 512, 256),
                                       (5, 7, 3, 200, 72), (8, 4, 4, 1000, 328), (9, 4, 4, 136, 520), (17, 2, 2, 264, 128),
                                       (33, 3, 2, 256, 192), (64, 2, 2, 512, 136), (64, 16, 4, 328, 264), (64, 1, 1, 72, 2048),
                                       (13, 40, 16, 96, 40), (2, 512, 8, 64, 64), (1, 4, 2, 4096, 64), (1, 4, 2, 64, 4096),
                                       (21, 32, 4, 1024, 512)])
def test_moe_matches_the_formula(h, T, E, k, H, I):
    g = gen(T + E + H + I)
    topk, gate = routing(g, T, E, k)
    check_moe(h, randn(g, T, H), topk, gate, *bf16_experts(g, E, H, I))


@pytest.mark.parametrize("T,E,k,H,I,group,zeros", [(1, 1, 1, 32, 32, 32, True), (1, 4, 2, 256, 128, 128, False),
                                                   (4, 8, 2, 512, 384, 128, True), (16, 3, 2, 320, 192, 64, True),
                                                   (17, 2, 2, 160, 96, 32, False), (64, 2, 2, 256, 256, 64, False),
                                                   (50, 8, 4, 128, 640, 128, True), (2, 64, 8, 1024, 128, 32, True)])
def test_moe_q4_matches_the_formula(h, T, E, k, H, I, group, zeros):
    g = gen(T + E + H + I)
    topk, gate = routing(g, T, E, k)
    check_moe(h, randn(g, T, H), topk, gate, packed(g, (E,), H, 2 * I, group, zeros), packed(g, (E,), I, H, group, zeros),
              quant=group)


# both sides of the size where other kernels begin: 2^27 (4-bit 2^26) weights of the experts that up to 8 tokens name, else
# 2^25 of those that 16 name, once per 16
@pytest.mark.parametrize("T,E,k,H,I,group,zeros", [
    (1, 2, 1, 8192, 5464, 0, False), (1, 2, 1, 8192, 5456, 0, False), (8, 4, 4, 3592, 3120, 0, False), (7, 3, 2, 3592, 2088, 0, False), (9, 4, 4, 2056, 1368, 0, False),
    (17, 2, 2, 4096, 920, 0, False), (33, 3, 2, 2048, 744, 0, False), (40, 16, 2, 1032, 296, 0, False), (64, 2, 2, 1544, 912, 0, False),
    (64, 8, 2, 1024, 360, 0, False), (64, 8, 2, 1024, 336, 0, False),
    (1, 3, 2, 4096, 2752, 64, True), (1, 3, 2, 4096, 2688, 64, True), (8, 4, 4, 2176, 2688, 128, False), (15, 2, 2, 3200, 1792, 128, True),
    (17, 2, 2, 4064, 928, 32, False), (33, 3, 2, 2048, 768, 128, True), (48, 16, 4, 1024, 320, 64, False), (64, 8, 2, 1024, 352, 32, True)])
def test_moe_of_large_experts(h, T, E, k, H, I, group, zeros):
    g = gen(T + E + H + I)
    topk, gate = routing(g, T, E, k)
    if group:
        w = packed(g, (E,), H, 2 * I, group, zeros), packed(g, (E,), I, H, group, zeros)
    else:
        w = bf16_experts(g, E, H, I)
    check_moe(h, randn(g, T, H), topk, gate, *w, quant=group or None)


# few columns (their rows are shared out to several CTAs), many experts, one long axis
@pytest.mark.parametrize("T,E,k,H,I", [(1, 2, 1, 8192, 32), (3, 2, 1, 32, 8192), (2, 4, 2, 4128, 96), (8, 64, 16, 96, 64),
                                       (11, 512, 4, 64, 32), (1, 4, 4, 2112, 1056), (16, 3, 1, 704, 32)])
@pytest.mark.parametrize("quant", [None, 32])
def test_moe_of_few_columns(h, T, E, k, H, I, quant):
    g = gen(T + E + H + I)
    topk, gate = routing(g, T, E, k)
    w = bf16_experts(g, E, H, I) if quant is None else (packed(g, (E,), H, 2 * I, quant, True), packed(g, (E,), I, H, quant, True))
    x = randn(g, T, H)
    first = check_moe(h, x, topk, gate, *w, quant=quant).clone()
    assert torch.equal(check_moe(h, x, topk, gate, *w, quant=quant), first)


@pytest.mark.parametrize("T,H,I", [(20, 192, 128), (20, 2560, 1600)])
@pytest.mark.parametrize("quant", [None, 64])
def test_moe_special_cases_of_routing_and_values(h, T, H, I, quant):
    """Missing and repeated experts, tokens without any, infinities and NaN in tokens and in one expert's weights:
    small and large experts."""
    g = gen(37)
    E, k = 7, 3
    topk, gate = routing(g, T, E - 1, k)
    topk[torch.rand(T, k, generator=g, device=DEV) < 0.3] = -1
    topk[0], topk[1] = -1, 2
    topk[5, 1], gate[5, 1] = 6, 0.5               # expert 6 is token 5's alone
    gate[topk < 0] = float("nan")
    w = bf16_experts(g, E, H, I) if quant is None else (packed(g, (E,), H, 2 * I, quant, True), packed(g, (E,), I, H, quant, True))
    x = randn(g, T, H)
    clean = check_moe(h, x, topk, gate, *w, quant=quant).clone()
    assert (clean[0] == 0).all()
    # the same call (the order of the sums depends on which experts are named) with NaN and infinities in expert 6
    for m in w:
        (m if quant is None else m[1])[6] = float("nan")
    (w[0] if quant is None else w[0][1])[6, 0] = float("inf")
    x[9, 3], x[10, 0] = float("inf"), float("nan")
    out, ws = torch.empty_like(clean), space(h.moe_decode_workspace(T, k, H, I))
    if quant is None:
        h.moe_decode(x, topk, gate, *w, out, ws)
    else:
        h.moe_decode_q4(x, topk, gate, *w, quant, out, ws)
    assert h.sync_status() == 0
    hit = {5} | {t for t in (9, 10) if (topk[t] >= 0).any()}
    keep = [t for t in range(T) if t not in (5, 9, 10)]
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[sorted(hit)].float()).any()


@pytest.mark.parametrize("quant", [None, 64])
def test_moe_missing_and_repeated_experts(h, quant):
    g = gen(31)
    T, E, k, H, I = 20, 6, 3, 192, 128
    topk, gate = routing(g, T, E, k)
    topk[torch.rand(T, k, generator=g, device=DEV) < 0.4] = -1
    topk[0] = -1                                  # a token without experts
    topk[1] = 2                                   # one expert three times
    topk[2, 0], topk[2, 2] = 5, 5
    topk[3:9, 0] = 4
    gate[topk < 0] = float("nan")                 # never read
    w = bf16_experts(g, E, H, I) if quant is None else (packed(g, (E,), H, 2 * I, 64, False), packed(g, (E,), I, H, 64, True))
    if quant:
        w = (w[0][:2] + (torch.full_like(w[0][1], 8).to(torch.uint8),), w[1])
    out = check_moe(h, randn(g, T, H), topk, gate, *w, quant=quant)
    assert (out[0] == 0).all()
    topk.fill_(-1)                                # no token has an expert
    out = check_moe(h, randn(g, T, H), topk, gate, *w, quant=quant)
    assert (out == 0).all()


def test_moe_reads_only_what_it_uses(h):
    """Experts that no token names and rows past H or I hold NaN; a token's infinities stay its own."""
    g = gen(32)
    T, E, k, H, I = 9, 5, 2, 104, 88
    W13, W2 = bf16_experts(g, E, H, I)
    x = randn(g, T, H)
    topk = torch.tensor([[1, 3]] * T, dtype=torch.int32, device=DEV)
    gate = torch.full((T, k), 0.5, device=DEV)
    for e in (0, 2, 4):
        W13[e], W2[e] = float("nan"), float("nan")
    want = check_moe(h, x, topk, gate, W13, W2).clone()
    x2 = x.clone()
    x2[4, 3], x2[7, 0] = float("inf"), float("nan")
    out = torch.empty(T, H, dtype=BF16, device=DEV)
    h.moe_decode(x2, topk, gate, W13, W2, out, space(h.moe_decode_workspace(T, k, H, I)))
    assert h.sync_status() == 0
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(out[keep], want[keep])
    assert not torch.isfinite(out[[4, 7]].float()).any()


def test_moe_strided_rows_streams_and_repeats(h):
    g = gen(33)
    T, E, k, H, I = 12, 8, 2, 640, 320
    topk, gate = routing(g, T, E, k)
    W = bf16_experts(g, E, H, I)
    x = randn(g, T, H + 64)[:, 16:16 + H]
    first = check_moe(h, x, topk, gate, *W).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):       # the same bits every time, on any stream
        out = check_moe(h, x, topk, gate, *W, stream=side)
        assert torch.equal(out, first)


@pytest.mark.parametrize("T,E,k,H,I,quant", [(5, 8, 4, 4096, 4096, None), (40, 8, 2, 4096, 4104, None),
                                             (20, 16, 4, 7168, 4096, 128)])
def test_moe_large_enough_for_tickets(h, T, E, k, H, I, quant):
    """Over 3 MB of weights a CTA: most items are taken by ticket; the bits stay the same."""
    g = gen(T)
    topk, gate = routing(g, T, E, k)
    x = randn(g, T, H)
    if quant:
        w = packed(g, (E,), H, 2 * I, quant, True), packed(g, (E,), I, H, quant, True)
    else:
        w = bf16_experts(g, E, H, I)
    first = check_moe(h, x, topk, gate, *w, quant=quant).clone()
    ws, out = space(h.moe_decode_workspace(T, k, H, I)), torch.empty_like(first)
    for _ in range(3):
        out.zero_()
        if quant:
            h.moe_decode_q4(x, topk, gate, *w, quant, out, ws)
        else:
            h.moe_decode(x, topk, gate, *w, out, ws)
        assert torch.equal(out, first)
    assert h.sync_status() == 0


@pytest.mark.parametrize("quant", [None, 64])
def test_moe_takes_any_magnitude(h, quant):
    """Rows of x from 1e-18 to 1e15: gate and up values, h and the result stay inside the bound."""
    g = gen(36)
    T, E, k, H, I = 6, 3, 2, 256, 192
    topk, gate = routing(g, T, E, k)
    x = (torch.randn(T, H, generator=g, device=DEV) * torch.tensor([1e-18, 1e-6, 1.0, 1e3, 1e9, 1e15], device=DEV)[:, None]).to(BF16)
    w = bf16_experts(g, E, H, I) if quant is None else (packed(g, (E,), H, 2 * I, 64, True), packed(g, (E,), I, H, 64, True))
    check_moe(h, x, topk, gate, *w, quant=quant)


def test_moe_back_to_back_calls_of_other_shapes(h):
    """Calls in a row without a synchronisation share the handle's counters and a workspace."""
    g = gen(34)
    shapes = [(1, 4, 2, 256, 128), (30, 4, 2, 512, 264), (2, 16, 4, 128, 1024), (64, 2, 1, 264, 64)]
    jobs = []
    for T, E, k, H, I in shapes:
        topk, gate = routing(g, T, E, k)
        jobs.append((randn(g, T, H), topk, gate, *bf16_experts(g, E, H, I), torch.empty(T, H, dtype=BF16, device=DEV)))
    ws = space(max(h.moe_decode_workspace(T, k, H, I) for T, E, k, H, I in shapes))
    for _ in range(10):
        for x, topk, gate, W13, W2, out in jobs:
            h.moe_decode(x, topk, gate, W13, W2, out, ws)
    assert h.sync_status() == 0
    for x, topk, gate, W13, W2, out in jobs:
        want, bound = moe_reference(x, topk, gate, W13, W2)
        within(out, want, bound, "out")


def test_moe_in_a_graph(h):
    g = gen(35)
    T, E, k, H, I = 4, 8, 2, 256, 192
    topk, gate = routing(g, T, E, k)
    W13, W2 = bf16_experts(g, E, H, I)
    x, out = randn(g, T, H), torch.empty(T, H, dtype=BF16, device=DEV)
    ws = space(h.moe_decode_workspace(T, k, H, I))
    h.moe_decode(x, topk, gate, W13, W2, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.moe_decode(x, topk, gate, W13, W2, out, ws)
    for seed in (1, 2, 3):
        x.copy_(randn(gen(seed), T, H))
        topk.copy_(routing(gen(seed), T, E, k)[0])
        graph.replay()
        torch.cuda.synchronize()
        want, bound = moe_reference(x, topk, gate, W13, W2)
        within(out, want, bound, "out")
    assert h.sync_status() == 0


# ------------------------------------------------------------------ together
def test_decode_step(h):
    """norm -> router -> experts, the residual stream carried on."""
    g = gen(41)
    T, E, k, H, I = 7, 16, 4, 512, 256
    x, res, weight = randn(g, T, H), randn(g, T, H, dtype=F32), randn(g, H, scale=0.1) + 1
    Wr = randn(g, H, E, scale=H ** -0.5)
    W13, W2 = bf16_experts(g, E, H, I)
    ro, y = torch.empty_like(res), torch.empty_like(x)
    topk, gate = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    h.add_rmsnorm(x, weight, 1e-5, residual=res, residual_out=ro, out=y)
    logits = y @ Wr
    h.route_topk(logits, topk, gate)
    out = check_moe(h, y, topk, gate, W13, W2)
    assert torch.isfinite(out.float()).all() and torch.equal(torch.sort(topk, 1).values.diff(dim=1) > 0,
                                                            torch.ones(T, k - 1, dtype=torch.bool, device=DEV))


def test_the_example_runs():
    from examples import decode_step
    assert 0 < decode_step.main(5) < 0.3      # (4-bit experts are near the bf16 ones, and not they)


# ------------------------------------------------------------------ refusals
def test_device_errors_are_reported_and_cleared(h):
    g = gen(51)
    T, E, k, H, I = 3, 4, 2, 128, 64
    topk, gate = routing(g, T, E, k)
    W13, W2 = bf16_experts(g, E, H, I)
    x = randn(g, T, H)
    out = torch.full((T, H), 5.0, dtype=BF16, device=DEV)
    ws = space(h.moe_decode_workspace(T, k, H, I))
    for bad in (E, -2):
        worse = topk.clone()
        worse[1, 1] = bad
        h.moe_decode(x, worse, gate, W13, W2, out, ws)
        assert h.sync_status() == tovl.TOVL_ERR_INVALID
        assert (out == 5).all()
    check_moe(h, x, topk, gate, W13, W2)


def test_a_wait_that_runs_out_is_an_error_status():
    g = gen(52)
    T, E, k, H, I = 3, 4, 2, 128, 64
    topk, gate = routing(g, T, E, k)
    W13, W2 = bf16_experts(g, E, H, I)
    x, out = randn(g, T, H), torch.empty(T, H, dtype=BF16, device=DEV)
    with tovl.Handle(0, max_rows=4096, max_pairs=4096, wait_timeout_ns=5_000_000) as hh:
        ws = space(hh.moe_decode_workspace(T, k, H, I))
        hh.set_option(tovl.OPT_FAULT_GATE_OFFSET, 1)
        hh.moe_decode(x, topk, gate, W13, W2, out, ws)
        assert hh.sync_status() == tovl.TOVL_ERR_TIMEOUT
        hh.set_option(tovl.OPT_FAULT_GATE_OFFSET, 0)
        hh.set_option(5, 2_000_000_000)
        check_moe(hh, x, topk, gate, W13, W2)


def test_refusals(h):
    INV, UNS, OK = tovl.TOVL_ERR_INVALID, tovl.TOVL_ERR_UNSUPPORTED, tovl.TOVL_OK
    L = tovl.load()
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    p = buf.data_ptr()
    s = torch.cuda.current_stream().cuda_stream

    def norm(x=p, ldx=64, res=None, ro=None, rt=0, ldr=64, w=p, eps=1e-5, T=1, H=64, out=p, ldo=64, q=None, qs=None, group=0):
        return L.tovl_add_rmsnorm(h.h, x, ldx, res, ro, rt, ldr, w, eps, T, H, out, ldo, q, qs, group, s)

    assert norm(T=0, x=None, w=None) == OK
    for bad in (dict(T=-1), dict(H=0), dict(out=None), dict(q=p), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
                dict(ldx=63), dict(ldo=63), dict(x=p + 1), dict(res=p), dict(res=p, ro=p, rt=2), dict(res=p, ro=p, ldr=1),
                dict(res=p + 2, ro=p, rt=1), dict(w=None)):
        assert norm(**bad) == INV, bad
    assert norm(H=32769, ldx=32769, ldo=32769) == UNS and norm(q=p, qs=p, group=48) == UNS

    def route(x=p, ty=1, ld=8, T=1, E=8, k=2, ids=p, w=p):
        return L.tovl_route_topk(h.h, x, ty, ld, T, E, k, 1, ids, w, s)

    assert route(T=0, x=None, ids=None, w=None) == OK
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(ty=2), dict(x=None), dict(ld=7), dict(ids=None), dict(w=None),
                dict(x=p + 2), dict(ids=p + 1)):
        assert route(**bad) == INV, bad
    assert route(E=513, ld=513) == UNS and route(k=33) == UNS

    n = L.tovl_moe_decode_workspace(h.h, 2, 2, 64, 64)
    ws = space(n)

    def moe(x=p, ldx=64, T=2, H=64, ids=p, gw=p, k=2, E=2, a=p, b=p, I=64, out=p, ldo=64, w=ws.data_ptr(), nb=n):
        return L.tovl_moe_decode(h.h, x, ldx, T, H, ids, gw, k, E, a, b, I, out, ldo, w, nb, s)

    assert moe(T=0, x=None, ids=None, gw=None, out=None, w=None) == OK
    for bad in (dict(T=-1), dict(H=60), dict(I=4), dict(k=0), dict(E=0), dict(x=None), dict(ids=None), dict(gw=None),
                dict(a=None), dict(b=p + 8), dict(out=None), dict(w=None), dict(nb=n - 1), dict(ldx=56), dict(ldx=66),
                dict(ldo=63), dict(x=p + 2), dict(w=ws.data_ptr() + 16)):
        assert moe(**bad) == INV, bad
    for bad in (dict(T=65), dict(k=17), dict(E=513), dict(H=32776, ldx=32776, ldo=32776)):
        assert moe(**bad) == UNS, bad
    assert L.tovl_moe_decode_workspace(h.h, 65, 2, 64, 64) == -1 and L.tovl_moe_decode_workspace(None, 1, 1, 64, 64) == -1

    def moe4(H=64, I=64, group=64, z1=None, z2=None, q=p, sc=p):
        return L.tovl_moe_decode_q4(h.h, p, 64, 2, H, p, p, 2, 2, q, sc, z1, p, p, z2, group, I, p, 64, ws.data_ptr(), n, s)

    for bad in (dict(H=96), dict(I=32), dict(z1=p), dict(z2=p), dict(q=None), dict(sc=None), dict(q=p + 4), dict(sc=p + 2)):
        assert moe4(**bad) == INV, bad
    assert moe4(group=16) == UNS

    m = L.tovl_matvec_q4_workspace(h.h, 2, 64)
    ws2 = space(m)

    def mv(x=p, ty=0, xs=None, ldx=64, T=2, K=64, q=p, sc=p, z=None, group=64, N=64, out=p, ldo=64, w=ws2.data_ptr(), nb=m):
        return L.tovl_matvec_q4(h.h, x, ty, xs, ldx, T, K, q, sc, z, group, N, out, ldo, w, nb, s)

    assert mv(T=0, x=None, out=None, w=None) == OK
    for bad in (dict(T=-1), dict(K=96), dict(N=12), dict(N=72, ldo=72, z=p), dict(ty=1), dict(ty=2), dict(x=None), dict(q=None),
                dict(sc=None), dict(out=None), dict(w=None), dict(nb=m - 1), dict(ldx=60), dict(ldx=66), dict(ldo=60),
                dict(ty=2, xs=p, ldx=72)):
        assert mv(**bad) == INV, bad
    for bad in (dict(T=65), dict(group=256), dict(K=32832, ldx=32832)):
        assert mv(**bad) == UNS, bad

    def quant(W=p, K=64, N=64, group=64, q=p, sc=p, E=1):
        return L.tovl_quantize_q4(h.h, W, E, K, N, group, q, sc, None, s)

    for bad in (dict(W=None), dict(K=32), dict(N=4), dict(q=None), dict(sc=None), dict(E=0)):
        assert quant(**bad) == INV, bad
    assert quant(group=16) == UNS
    assert h.sync_status() == 0


def test_binding_checks_types_shapes_and_strides(h):
    x = torch.zeros(2, 64, dtype=BF16, device=DEV)
    w = torch.zeros(64, dtype=BF16, device=DEV)
    with pytest.raises(TypeError):
        h.add_rmsnorm(x.float(), w, 1e-5, out=x)
    with pytest.raises(TypeError):
        h.add_rmsnorm(x, w[:32], 1e-5, out=x)
    with pytest.raises(TypeError):
        h.add_rmsnorm(x, w, 1e-5, out=torch.zeros(64, 2, dtype=BF16, device=DEV).t())
    with pytest.raises(TypeError):
        h.add_rmsnorm(x, w, 1e-5, residual=x, residual_out=x.float(), out=x)
    with pytest.raises(TypeError):
        h.route_topk(x, torch.zeros(2, 2, dtype=torch.int64, device=DEV), torch.zeros(2, 2, device=DEV))
    topk, gate = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.zeros(2, 1, device=DEV)
    W13, W2 = torch.zeros(1, 64, 128, dtype=BF16, device=DEV), torch.zeros(1, 64, 64, dtype=BF16, device=DEV)
    ws = space(h.moe_decode_workspace(2, 1, 64, 64))
    with pytest.raises(TypeError):
        h.moe_decode(x, topk, gate.double(), W13, W2, x, ws)
    with pytest.raises(TypeError):
        h.moe_decode(x, topk, gate, W13.transpose(1, 2).contiguous().transpose(1, 2), W2, x, ws)
    with pytest.raises(tovl.TovlError):
        h.moe_decode(x, topk, gate, W13, W2, x, ws[:256])
    q, sc, _ = h.quantize_q4(W2[0], 32)
    with pytest.raises(TypeError):
        h.matvec_q4(x, q, sc, 64, x, ws)
    with pytest.raises(TypeError):
        h.matvec_q4(x.to(E4M3), q, sc, 32, x, ws)
