"""Edges of the paged attention step: what its header allows and the sizes of test_gpu_paged.py do not reach.

Tolerances are those of test_gpu_paged.py.
"""
import math

import pytest
import torch

from consumer_movement_gemm_gb300 import tovl
from tests.test_gpu_decode import BF16, D, DEV, U16, gen, h, randn, within  # noqa: F401
from tests.test_gpu_paged import NAN, Cache, attn_reference, filled, ints, space

pytestmark = pytest.mark.gpu


def attend(h, q, c, table, lens, scale=1.0):  # noqa: F811
    out, lse = torch.full_like(q, NAN), torch.full(q.shape[:2], NAN, device=DEV)
    ws = space(h.attn_decode_workspace(q.shape[1], c.k.shape[2], q.shape[2]))
    h.attn_decode(q, c.cache, table, ints(lens), scale, out, ws, lse=lse)
    assert h.sync_status() == 0
    return out, lse


# ------------------------------------------------------------------ scales of values
@pytest.mark.parametrize("power", [-149, -126, -120, -90, -60, -48, 100, 119])
@pytest.mark.parametrize("heads,G,dim,page", [(2, 4, 128, 16), (1, 12, 64, 20)])
def test_attn_values_of_any_scale(h, power, heads, G, dim, page):  # noqa: F811
    """All scales of a request 2^power, one scale in nine 2^-12 instead, and all but one token's."""
    g = gen(power + 200 + dim)
    lens = [4096, 4096, 700, 1]
    c, table, slots = filled(g, lens, heads, dim, page, "e4m3")
    for b, s in enumerate(slots):
        x = (randn(g, len(s), heads, dim).float() * 100).clamp(-448, 448)
        unit = torch.full((len(s), heads), 2.0 ** power, dtype=D, device=DEV).float()
        if b == 1:
            unit[::9] = 2.0 ** -12
        if b == 2:
            unit[350] = 2.0 ** -12
        c.put("v", s, x, unit)
    q = randn(g, len(lens), heads * G, dim, scale=2)
    q[:, ::2] *= 2.0 ** -6          # weights much alike, so that all of them count in the sum
    out, lse = attend(h, q, c, table, lens, dim ** -0.5)
    want, bound, wl, bl = attn_reference(q, c, slots, dim ** -0.5, 0)
    # a value whose weight times scale is below 2^-48 is off by 2^-73 of its element
    for b, s in enumerate(slots):
        bound[b] += 2.0 ** -73 * c.v.view(torch.uint8)[s // page, s % page].view(c.v.dtype).to(D).abs().sum(0).repeat_interleave(G, 0)
    within(lse, wl, bl, "lse")
    within(out, want, bound, "out")


def test_attn_values_of_zeros(h):  # noqa: F811
    """Scales of 0: zeros, and the lse of the keys."""
    g = gen(1)
    lens = [3000, 17]
    c, table, slots = filled(g, lens, 2, 64, 16, "e4m3")
    q = randn(g, 2, 8, 64, scale=2)
    q[:, ::2] *= 2.0 ** -6
    _, _, want, bound = attn_reference(q, c, slots, 0.125, 0)
    c.vs.zero_()
    c.v.view(torch.uint8).zero_()
    out, lse = attend(h, q, c, table, lens, 0.125)
    assert (out == 0).all()
    within(lse, want, bound, "lse")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("score", [2.0 ** 20, 2.0 ** 25, 2.0 ** 26, -2.0 ** 26])
def test_attn_large_scores(h, kind, score):  # noqa: F811
    """Equal scores: the mean of the values, whatever the scores; and one token's value."""
    g = gen(2)
    lens = [1, 600]
    c, table, slots = filled(g, lens, 1, 64, 16, kind)
    for s in slots:
        x = torch.zeros(len(s), 1, 64, device=DEV)
        x[:, :, 0] = 256
        c.put("k", s, x, torch.ones(len(s), 1, device=DEV))
    q = torch.zeros(2, 2, 64, dtype=BF16, device=DEV)
    q[:, :, 0] = 1
    out, _ = attend(h, q, c, table, lens, score / 256)
    for b, s in enumerate(slots):
        V = c.rows("v", s)[:, 0]
        # weights of 1 but for the row's scale and their own rounding; sums of 600
        near = V.abs().mean(0) * (2.0 ** -11 + 4 * 600 * 2.0 ** -23) + U16 * V.mean(0).abs()
        within(out[b], V.mean(0).expand(2, 64), near.expand(2, 64), f"request {b}")


# ------------------------------------------------------------------ joins
# every number of columns and of blocks of query heads; requests of which many are joined in one CTA, in many
@pytest.mark.parametrize("dim", [16, 64, 72, 80, 88, 96, 104, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("heads,G", [(3, 32), (1, 9), (2, 16), (4, 8), (8, 1)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_joins_write_every_column(h, dim, heads, G, kind):  # noqa: F811
    if kind == "e4m3" and dim % 16:
        dim += 8
    g = gen(dim * 100 + G)
    for lens in ([440] * 60, list(range(20, 700, 17)), [3000, 1000, 9000]):
        c, table, slots = filled(g, lens, heads, dim, 16, kind)
        q = randn(g, len(lens), heads * G, dim, scale=2)
        out, lse = attend(h, q, c, table, lens, dim ** -0.5)
        want, bound, wl, bl = attn_reference(q, c, slots, dim ** -0.5, 0)
        within(out, want, bound, f"out {lens[:2]}")
        within(lse, wl, bl, f"lse {lens[:2]}")


# ------------------------------------------------------------------ the limit on tiles
@pytest.mark.parametrize("heads", [1, 2])
def test_attn_more_tiles_than_a_call_takes(h, heads):  # noqa: F811
    """Requests of 2^31 - 64 tokens in one shared page, in tiles of 16: reported before a row is read."""
    page, B = 1 << 16, 20
    c = Cache(1, page, heads, 128, "bf16")
    table = torch.zeros(B, 1 << 15, dtype=torch.int32, device=DEV)
    q = torch.zeros(B, heads, 128, dtype=BF16, device=DEV)
    out = torch.full_like(q, 7)
    ws = space(h.attn_decode_workspace(heads, heads, 128))
    for lens in ([2 ** 31 - 64] * B, [0, 1] + [2 ** 31 - 100] * (B - 2)):
        assert sum(-(-n // 16) for n in lens) > 2 ** 31
        h.attn_decode(q, c.cache, table, ints(lens), 0.1, out, ws)
        assert h.sync_status() == tovl.TOVL_ERR_UNSUPPORTED
        assert (out == 7).all()
    # the next call is as ever
    c.k.zero_(), c.v.fill_(3)
    h.attn_decode(q, c.cache, table, ints([5] * B), 0.1, out, ws)
    assert h.sync_status() == 0 and (out == 3).all()


# ------------------------------------------------------------------ what lies around the outputs
# workspaces of warps, CTAs and groups of CTAs; heads side by side; two blocks of a wide head from one ring (bf16, more than
# 128 columns, 16 or 32 query heads); two blocks a warp; pages of 20 slots, copied row by row
@pytest.mark.parametrize("heads,G,dim,kind", [(1, 1, 16, "bf16"), (8, 4, 128, "bf16"), (2, 12, 64, "bf16"), (8, 4, 80, "bf16"), (4, 1, 96, "bf16"),
                                              (1, 8, 192, "bf16"), (1, 16, 256, "bf16"), (2, 32, 192, "bf16"), (1, 24, 256, "bf16"), (1, 5, 136, "bf16"),
                                              (16, 1, 64, "e4m3"), (8, 8, 128, "e4m3"), (2, 16, 128, "e4m3"), (8, 2, 48, "e4m3"), (1, 16, 192, "e4m3"),
                                              (1, 40, 256, "e4m3"), (2, 3, 240, "e4m3"), (8, 16, 96, "e4m3")])
@pytest.mark.parametrize("page", [16, 20])
def test_attn_writes_its_outputs_and_workspace_only(h, heads, G, dim, kind, page):  # noqa: F811
    g = gen(heads * 1000 + G + dim)
    n = h.attn_decode_workspace(heads * G, heads, dim)
    for lens in ([60000], [0, 1, 40], [3000, 0, 777, 9000], list(range(0, 900, 9))):
        B, Hq = len(lens), heads * G
        c, table, slots = filled(g, lens, heads, dim, page, kind)
        q = randn(g, B, Hq, dim, scale=2)
        around = torch.full((n + 8192,), 0xa5, dtype=torch.uint8, device=DEV)
        wide = torch.full((B + 2, Hq * dim + 32), 3.0, dtype=BF16, device=DEV)
        stats = torch.full((B * Hq + 64,), 5.0, device=DEV)
        out, lse = wide[1:B + 1, 16:16 + Hq * dim].view(B, Hq, dim), stats[32:32 + B * Hq].view(B, Hq)
        h.attn_decode(q, c.cache, table, ints(lens), dim ** -0.5, out, around[4096:4096 + n], lse=lse)
        assert h.sync_status() == 0
        want, bound, wl, bl = attn_reference(q, c, slots, dim ** -0.5, 0)
        within(out, want, bound, "out")
        within(torch.where(wl == -math.inf, 0, lse), torch.where(wl == -math.inf, 0, wl), bl, "lse")
        assert (around[:4096] == 0xa5).all() and (around[4096 + n:] == 0xa5).all(), "workspace"
        out.fill_(3)
        lse.fill_(5)
        assert (wide == 3).all() and (stats == 5).all()


# ------------------------------------------------------------------ roundings of an e4m3 cache
@pytest.mark.parametrize("heads,dim,T", [(2, 128, 9), (1, 80, 5), (8, 64, 2000)])
def test_append_quotients_round_to_even(h, heads, dim, T):  # noqa: F811
    """Rows whose quotients are exact ties (the largest 448 times a power of two, the others odd multiples of half a
    unit), and any others: the bytes of the fp32 quotient by the scale that was written."""
    g = gen(dim)
    # every number half way between two neighbours of e4m3, and its neighbours in bf16
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    half = (grid[1:] + grid[:-1]) / 2
    near = torch.cat([half, half * (1 - 2.0 ** -8), half * (1 + 2.0 ** -7)]).to(BF16).float()
    pool = torch.cat([near, -near]).to(DEV)
    x = pool[torch.randint(0, len(pool), (T, heads, dim), generator=g, device=DEV)].clamp(-448, 448)
    x[:, :, dim // 3] = 448
    x = x * torch.exp2(torch.randint(-20, 20, (T, heads, 1), generator=g, device=DEV).float())
    x[T // 2:] = torch.randn(T - T // 2, heads, dim, generator=g, device=DEV)
    x = x.to(BF16)
    page = 16
    c = Cache(-(-T // page), page, heads, dim, "e4m3")
    slots = torch.arange(T, device=DEV)
    h.rope_append(x, x, x, slots.to(torch.int32), slots.to(torch.int32), None, c.cache, torch.empty_like(x))
    assert h.sync_status() == 0
    for t, s in ((c.k, c.ks), (c.v, c.vs)):
        scale = s[slots // page, :, slots % page]
        top = x.float().abs().amax(2)
        assert torch.equal(scale, top / torch.full_like(top, 448))
        got = t.view(torch.uint8)[slots // page, slots % page].view(t.dtype).float()
        want = (x.float() / scale[:, :, None]).clamp(-448, 448).to(t.dtype).float()
        assert torch.equal(got, want)
        ties = (x[:T // 2].float() / scale[:T // 2, :, None]).abs()[..., None] == half.to(DEV)
        assert ties.any(3).float().mean() > 0.2
