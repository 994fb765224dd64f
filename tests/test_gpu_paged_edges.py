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
