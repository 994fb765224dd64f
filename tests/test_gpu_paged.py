"""The paged attention step (page plan, rotary embedding with cache writes, attention of one new token) against plain
64-bit implementations.

Tolerances are error bounds, not fits; U32, U16 and sum_bound are those of test_gpu_decode.py.
  * A score is a product of `dim` terms summed in fp32 (sum_bound) and three fp32 products; with an e4m3 cache a
    query below 2^-14 of its row's largest times 2^-15 is off by half a unit of fp16's subnormals, 2^-39 of the largest.
  * A weight is exp2 of a difference: an error d of the exponent is a relative error of about d of the weight, the
    exponent's own roundings are 2 units of its terms' magnitudes (scores, and up to 128 for scales and shift), exp2's
    error is 2 units.  All of a row's weights relative to their sum: twice the largest relative error.
  * Weights enter the second product with an error of 2^-15 of themselves (bf16 cache: the upper 8 bits and
    the rest, below 2^-7, rounded to bf16), or as fp16, 2^-11 of themselves and, of the
    largest weight times scale, 2^-25.
  * Sums over n tokens: sum_bound, and a factor of 2 units for each tile that moves the maximum: 4 sum_bound(n) in all.
"""
import math

import numpy as np
import pytest
import torch

from consumer_movement_gemm_gb300 import tovl
from tests.test_gpu_decode import BF16, D, DEV, E4M3, F32, U16, U32, gen, guarded, h, randn, sum_bound, within  # noqa: F401

pytestmark = pytest.mark.gpu
I32 = torch.int32
NAN = float("nan")


def ints(*v):
    return torch.tensor(v if len(v) > 1 or not isinstance(v[0], (list, np.ndarray)) else v[0], dtype=I32, device=DEV)


# ------------------------------------------------------------------ caches
class Cache:
    """A cache whose unused slots hold NaN, and its rows in 64 bits."""

    def __init__(self, pages, page, heads, dim, kind, layout="nhd"):
        dt = BF16 if kind == "bf16" else E4M3
        shape = {"nhd": (pages, page, heads, dim), "hnd": (pages, heads, page, dim), "both": (pages, 2, page, heads, dim),
                 "wide": (pages, page + 1, heads + 2, dim + 16)}[layout]

        def empty():
            return torch.full(shape, NAN, device=DEV).to(dt)
        if layout == "both":
            kv = empty()
            self.k, self.v = kv[:, 0], kv[:, 1]
        else:
            view = {"nhd": lambda t: t, "hnd": lambda t: t.transpose(1, 2), "wide": lambda t: t[:, :page, 1:-1, :dim]}[layout]
            self.k, self.v = view(empty()), view(empty())
        self.ks = self.vs = None
        if dt is E4M3:
            self.ks, self.vs = (torch.full((pages, heads, page), NAN, device=DEV) for _ in range(2))
        self.kind, self.page = kind, page
        self.cache = tovl.KVCache(self.k, self.v, self.ks, self.vs)

    def put(self, which, slots, rows, scale=None):
        """rows [n, heads, dim] (and scales [n, heads]) as they are"""
        t, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        at, off = slots.long() // self.page, slots.long() % self.page
        if self.kind == "bf16":
            t[at, off] = rows.to(BF16)
        else:
            t.view(torch.uint8)[at, off] = rows.to(E4M3).view(torch.uint8)
            s[at, :, off] = scale

    def rows(self, which, slots):
        """[n, heads, dim] in 64 bits"""
        t, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        at, off = slots.long() // self.page, slots.long() % self.page
        if self.kind == "bf16":
            return t[at, off].to(D)
        return t.view(torch.uint8)[at, off].view(E4M3).to(D) * s[at, :, off].to(D)[:, :, None]


def filled(g, lens, heads, dim, page, kind, layout="nhd", spare=2, spread=(0.5, 2.0)):
    """A cache with the requests' tokens in shuffled pages, their table (entries that are not used are -7) and slots."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    c = Cache(pages, page, heads, dim, kind, layout)
    order = torch.randperm(pages, generator=g, device=DEV).to(I32)
    table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=I32, device=DEV)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = torch.arange(n, device=DEV)
        slots.append(table[b].long()[t // page] * page + t % page if n else t)
    every = torch.cat(slots)
    if len(every):
        for which in ("k", "v"):
            x = torch.randn(len(every), heads, dim, generator=g, device=DEV)
            s = torch.rand(len(every), heads, generator=g, device=DEV) * (spread[1] - spread[0]) + spread[0]
            c.put(which, every, x if kind == "bf16" else (x * 100).clamp(-448, 448), s / 100)
    return c, table, slots


def attn_reference(q, c, slots, scale, window):
    """out, its bound, lse, its bound."""
    B, Hq, dim = q.shape
    heads = c.k.shape[2]
    G = Hq // heads
    out, ob = torch.zeros(B, Hq, dim, dtype=D, device=DEV), torch.zeros(B, Hq, dim, dtype=D, device=DEV)
    lse, lb = torch.full((B, Hq), -math.inf, dtype=D, device=DEV), torch.zeros(B, Hq, dtype=D, device=DEV)
    for b in range(B):
        s = slots[b][-window:] if window else slots[b]
        n = len(s)
        if n == 0:
            continue
        K, V = (c.rows(w, s).permute(1, 0, 2) for w in ("k", "v"))              # [heads, n, dim]
        x = q[b].to(D).view(heads, G, dim)
        z, mag = scale * (x @ K.mT), abs(scale) * (x.abs() @ K.abs().mT)
        dz = sum_bound(dim, mag) + 4 * U32 * z.abs()
        if c.kind != "bf16":
            dz = dz + abs(scale) * 2.0 ** -39 * x.abs().amax(2, keepdim=True) * K.abs().sum(2)[:, None]
        e = dz + 2 * U32 * (z.abs() + z.abs().amax(2, keepdim=True) + 128) + 4 * U32
        w = torch.softmax(z, 2)
        r = w @ V
        rel = 2.0 ** -15 if c.kind == "bf16" else 2.0 ** -11
        near = (w * (e + rel)) @ V.abs() + (w * e).sum(2, keepdim=True) * r.abs() + 4 * sum_bound(n, w @ V.abs() + r.abs())
        if c.kind != "bf16":
            unit = c.vs[s.long() // c.page, :, s.long() % c.page].to(D).T            # [heads, n]
            top = (w * unit[:, None]).amax(2, keepdim=True)
            near = near + 2.0 ** -25 * top * (V.abs() / unit[:, :, None]).sum(1)[:, None]
        out[b], ob[b] = r.reshape(Hq, dim), (near + U16 * r.abs() + 2.0 ** -133).reshape(Hq, dim)
        y = torch.logsumexp(z, 2)
        lse[b] = y.reshape(Hq)
        lb[b] = ((w * e).sum(2) + 4 * sum_bound(n, torch.ones_like(y)) + 4 * U32 * (y.abs() + 128)).reshape(Hq)
    return out, ob, lse, lb


def space(n):
    return torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)      # (any content)


def check_attn(h, q, c, table, lens, slots, scale, window, what=""):  # noqa: F811
    B, Hq, dim = q.shape
    out = torch.full_like(q, NAN)
    lse = torch.full((B, Hq), NAN, device=DEV)
    ws = space(h.attn_decode_workspace(Hq, c.k.shape[2], dim))
    h.attn_decode(q, c.cache, table, lens, scale, out, ws, window=window, lse=lse)
    assert h.sync_status() == 0
    want, bound, wl, bl = attn_reference(q, c, slots, scale, window)
    within(out, want, bound, "out " + what)
    none = wl == -math.inf
    assert torch.equal(lse == -math.inf, none), "lse of requests without tokens"
    within(torch.where(none, 0, lse), torch.where(none, 0, wl), bl, "lse " + what)
    return out, lse


LENGTHS = [[1], [2], [15, 16, 17], [31, 32, 33, 0, 1], [777], [0, 0], [130, 0, 4101, 1, 64, 600], [1] * 70,
           list(range(0, 200, 7))]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("heads,G", [(1, 1), (2, 4), (3, 8), (2, 16), (1, 9), (1, 40)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_matches_the_formula(h, lens, heads, G, kind):  # noqa: F811
    g = gen(len(lens) * 1000 + heads * 100 + G)
    c, table, slots = filled(g, lens, heads, 128, 16, kind)
    q = randn(g, len(lens), heads * G, 128, scale=2)
    check_attn(h, q, c, table, ints(lens), slots, 128 ** -0.5, 0)


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("page,layout", [(1, "nhd"), (5, "hnd"), (16, "both"), (24, "wide"), (64, "hnd"), (1000, "nhd")])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_head_sizes_pages_and_layouts(h, dim, page, layout, kind):  # noqa: F811
    g = gen(dim * 1000 + page)
    lens = [1, 40, 333, 0, 95]
    for heads, G in ((2, 3), (1, 12)):
        c, table, slots = filled(g, lens, heads, dim, page, kind, layout)
        q = randn(g, len(lens), heads * G, dim, scale=2)
        check_attn(h, q, c, table, ints(lens), slots, dim ** -0.5, 0, f"{heads} x {G}")


# blocks of 8 or 16 query heads of one key head: two, four or eight warps share a ring; three and five do not; pages of 20
# slots are copied row by row, without shared rings
@pytest.mark.parametrize("heads,G,dim", [(1, 32, 128), (2, 64, 128), (1, 128, 64), (1, 16, 256), (3, 32, 192), (1, 24, 256), (1, 72, 128),
                                         (2, 48, 128), (1, 30, 112)])
@pytest.mark.parametrize("page,window", [(16, 0), (64, 300), (20, 0)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_many_query_heads_a_key_head(h, heads, G, dim, page, window, kind):  # noqa: F811
    g = gen(G * 1000 + dim + page)
    for lens in ([1], [700, 0, 31, 16], [5000, 9000], [33] * 90):
        c, table, slots = filled(g, lens, heads, dim, page, kind)
        q = randn(g, len(lens), heads * G, dim, scale=2)
        check_attn(h, q, c, table, ints(lens), slots, dim ** -0.5, window, str(lens[:3]))


@pytest.mark.parametrize("dim", [8, 24, 72, 136, 200])
def test_attn_odd_head_sizes(h, dim):  # noqa: F811
    g = gen(dim)
    lens = [50, 3]
    c, table, slots = filled(g, lens, 2, dim, 16, "bf16")
    check_attn(h, randn(g, 2, 6, dim, scale=2), c, table, ints(lens), slots, dim ** -0.5, 0)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 128, 4095, 1 << 30])
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3", 64), ("bf16", 256)])
def test_attn_window(h, window, kind, dim):  # noqa: F811
    g = gen(window % 1000 + dim)
    lens = [0, 1, 16, 33, 129, 1000, 5000]
    c, table, slots = filled(g, lens, 2, dim, 16, kind)
    # pages before the window are not read: their entries may be anything
    for b, n in enumerate(lens):
        table[b, :max(0, n - window) // 16] = -9
    check_attn(h, randn(g, len(lens), 8, dim, scale=2), c, table, ints(lens), slots, dim ** -0.5, window)


@pytest.mark.parametrize("lens,heads,G,dim,kind", [(range(300, 1900, 50), 1, 16, 256, "bf16"), (range(100, 2100, 20), 2, 8, 128, "e4m3"),
                                                   ([16000], 1, 16, 128, "bf16"), ([9000, 8000, 100], 2, 4, 96, "bf16")],
                         ids=lambda v: str(v)[:12])
def test_attn_same_bits_whichever_cta_joins(h, lens, heads, G, dim, kind):  # noqa: F811
    """The order in which the CTAs of a segment finish differs from call to call, and with it how many are joined at once."""
    lens = list(lens)
    g = gen(sum(lens))
    c, table, slots = filled(g, lens, heads, dim, 16, kind)
    q = randn(g, len(lens), heads * G, dim, scale=2)
    first, lse = check_attn(h, q, c, table, ints(lens), slots, dim ** -0.5, 0)
    ws = torch.empty(h.attn_decode_workspace(heads * G, heads, dim), dtype=torch.uint8, device=DEV)
    out, stats = torch.empty_like(first), torch.empty_like(lse)
    for _ in range(50):
        h.attn_decode(q, c.cache, table, ints(lens), dim ** -0.5, out, ws, lse=stats)
        assert torch.equal(out, first) and torch.equal(stats, lse)


@pytest.mark.parametrize("lens,heads,G,dim,kind", [([70001], 1, 1, 128, "bf16"), ([70001], 1, 16, 128, "e4m3"), ([20000, 1, 50000], 4, 8, 64, "bf16"),
                                                   ([30011] * 3, 2, 5, 256, "e4m3"), ([9000] * 40, 1, 4, 80, "bf16"),
                                                   ([300] * 500, 2, 4, 128, "bf16"), ([17] * 3000, 1, 2, 64, "e4m3")],
                         ids=lambda v: str(v)[:12])
def test_attn_long_and_many(h, lens, heads, G, dim, kind):  # noqa: F811
    g = gen(sum(lens))
    c, table, slots = filled(g, lens, heads, dim, 32, kind)
    q = randn(g, len(lens), heads * G, dim, scale=2)
    out, lse = check_attn(h, q, c, table, ints(lens), slots, dim ** -0.5, 0)
    again, _ = check_attn(h, q, c, table, ints(lens), slots, dim ** -0.5, 0)
    assert torch.equal(out, again)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_extreme_scores_and_scales(h, kind):  # noqa: F811
    """Scores of hundreds in either order (the maximum moves in every tile, or never again), all scores equal, scales
    from 2^-40 to 2^100."""
    g = gen(5)
    n = 700
    c, table, slots = filled(g, [n] * 4, 1, 64, 16, kind)
    q = torch.zeros(4, 4, 64, device=DEV)
    q[:, :, 0] = 1
    for b in range(4):
        ramp = torch.arange(n, device=DEV).float() * (1 if b == 0 else -1 if b == 1 else 0)
        x = c.rows("k", slots[b]).float()
        x[:, 0, 0] = ramp
        if kind == "bf16":
            c.put("k", slots[b], x)
        else:
            c.put("k", slots[b], x.clamp(-448, 448), torch.full((n, 1), 0.01 if b == 3 else 2.0, device=DEV))
            if b >= 2:
                v = (c.rows("v", slots[b]) / c.vs[slots[b] // 16, :, slots[b] % 16].to(D)[:, :, None]).float()
                c.put("v", slots[b], v, torch.exp2(torch.randint(-40, 100 if b == 3 else -30, (n, 1), generator=g, device=DEV).float()))
    check_attn(h, q.to(BF16), c, table, ints([n] * 4), slots, 1.0, 0)


def test_attn_infinities_and_nan_show_where_they_are_seen(h):  # noqa: F811
    g = gen(6)
    lens = [100, 100, 100, 100]
    c, table, slots = filled(g, lens, 1, 64, 16, "bf16")
    q = randn(g, 4, 2, 64).abs()
    clean, _ = check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)
    c.k[slots[1][40] // 16, slots[1][40] % 16, 0, 3] = NAN            # a NaN key
    c.k[slots[2][40] // 16, slots[2][40] % 16] = -math.inf            # a key that is never chosen
    c.v[slots[3][40] // 16, slots[3][40] % 16, 0, 5] = math.inf       # an infinite value
    out = torch.empty_like(q)
    h.attn_decode(q, c.cache, table, ints(lens), 0.125, out, space(h.attn_decode_workspace(2, 1, 64)))
    assert torch.equal(out[0], clean[0])
    assert out[1].isnan().all()
    assert out[2].isfinite().all()
    assert (out[3, :, 5] == math.inf).all() and out[3, :, :5].isfinite().all()
    h.attn_decode(q, c.cache, table, ints([100, 100, 100, 40]), 0.125, out, space(h.attn_decode_workspace(2, 1, 64)), window=59)
    assert out[[0, 1, 2, 3]].isfinite().all()                         # none of the three is seen


def test_attn_strided_rows_streams_and_a_null_lse(h):  # noqa: F811
    g = gen(8)
    lens = [200, 0, 31]
    c, table, slots = filled(g, lens, 2, 64, 16, "bf16")
    wide = randn(g, 3, 6 * 64 + 128, scale=2)
    q = wide[:, 64:64 + 4 * 64].view(3, 4, 64)
    view, intact = guarded(3, 4 * 64)
    out = view.view(3, 4, 64)
    ws = space(h.attn_decode_workspace(4, 2, 64))
    big = torch.full((3, table.shape[1] + 5), -3, dtype=I32, device=DEV)
    big[:, 2:2 + table.shape[1]] = table
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens_dev = ints(lens)
    side.wait_stream(torch.cuda.current_stream())
    h.attn_decode(q, c.cache, big[:, 2:2 + table.shape[1]], lens_dev, 0.125, out, ws, stream=side)
    side.synchronize()
    assert h.sync_status() == 0 and intact()
    want, bound, _, _ = attn_reference(q, c, slots, 0.125, 0)
    within(out, want, bound, "out")


# heads whose rows are not whole 128-byte lines: two, four or eight neighbours go together
@pytest.mark.parametrize("heads,dim,kind", [(8, 80, "bf16"), (8, 80, "e4m3"), (16, 64, "e4m3"), (4, 96, "bf16"), (8, 48, "e4m3"), (6, 80, "bf16"),
                                            (8, 144, "bf16"), (8, 240, "e4m3"), (5, 64, "e4m3")])
@pytest.mark.parametrize("G", [1, 8])
def test_attn_heads_that_share_lines(h, heads, dim, kind, G):  # noqa: F811
    g = gen(heads * 1000 + dim + G)
    for lens in ([1], [3000, 0, 70, 900], [250] * 60, [9000]):
        c, table, slots = filled(g, lens, heads, dim, 16, kind)
        check_attn(h, randn(g, len(lens), heads * G, dim, scale=2), c, table, ints(lens), slots, dim ** -0.5, 0, str(lens[:3]))


@pytest.mark.parametrize("heads,G,dim,kind", [(1, 1, 128, "bf16"), (2, 4, 64, "e4m3"), (1, 16, 256, "bf16")])
def test_attn_every_length_of_one_request(h, heads, G, dim, kind):  # noqa: F811
    """One CTA a head, several, all of them, and groups of them: lengths at which the shares change."""
    g = gen(dim)
    most = 60000
    c, table, slots = filled(g, [most], heads, dim, 16, kind)
    q = randn(g, 1, heads * G, dim, scale=2)
    for n in (1, 16, 17, 32, 33, 191, 192, 193, 383, 385, 577, 1200, 1201, 3000, 4607, 4609, 9300, 9400, 20000, 29184, 29200, 58368, 58369, most):
        check_attn(h, q, c, table, ints([n]), [slots[0][:n]], dim ** -0.5, 0, str(n))


def test_attn_of_the_largest_batch(h):  # noqa: F811
    """One token each: the output is its value, and the lse its score."""
    g = gen(3)
    B = 65536
    c = Cache(B, 1, 1, 64, "bf16")
    c.put("k", torch.arange(B, device=DEV), randn(g, B, 1, 64))
    c.put("v", torch.arange(B, device=DEV), randn(g, B, 1, 64))
    table = torch.randperm(B, generator=g, device=DEV).to(I32)[:, None]
    lens = (torch.rand(B, generator=g, device=DEV) < 0.9).to(I32)
    q = randn(g, B, 2, 64)
    out, lse = torch.full_like(q, NAN), torch.full((B, 2), NAN, device=DEV)
    h.attn_decode(q, c.cache, table, lens, 0.125, out, space(h.attn_decode_workspace(2, 1, 64)), lse=lse)
    assert h.sync_status() == 0
    row = table[:, 0].long()
    v = torch.where(lens[:, None] > 0, c.v[row, 0, 0], 0)
    within(out, v[:, None].to(D).expand(B, 2, 64), 2.0 ** -14 * v.abs()[:, None].to(D), "out")      # (a bf16 number is its own nearest)
    z = 0.125 * (q.to(D) * c.k[row, 0].to(D)).sum(2)
    seen = lens[:, None].expand(B, 2) > 0
    assert torch.equal(lse == -math.inf, ~seen)
    within(lse[seen], z[seen], 64 * U32 * (q.to(D).abs() * c.k[row, 0].to(D).abs()).sum(2)[seen] + 4 * U32 * 128, "lse")


@pytest.mark.parametrize("kind,layout", [("bf16", "nhd"), ("e4m3", "hnd")])
def test_a_cache_beyond_32_bit_offsets(h, kind, layout):  # noqa: F811
    """Pages whose keys and values lie more than 2^32 bytes and elements from the first."""
    g = gen(4)
    heads, dim, page = 8, 128, 16
    pages = 300000 if kind == "bf16" else 350000
    assert pages * page * heads * dim > 2 ** 32
    dt = BF16 if kind == "bf16" else E4M3
    shape = (pages, page, heads, dim) if layout == "nhd" else (pages, heads, page, dim)
    c = Cache(1, page, heads, dim, kind, layout)
    c.k, c.v = (torch.empty(shape, dtype=dt, device=DEV) for _ in range(2))
    if layout == "hnd":
        c.k, c.v = c.k.transpose(1, 2), c.v.transpose(1, 2)
    if kind != "bf16":
        c.ks, c.vs = (torch.empty(pages, heads, page, device=DEV) for _ in range(2))
    c.cache = tovl.KVCache(c.k, c.v, c.ks, c.vs)
    n = 50
    table = ints([pages - 1, 0, pages - 2, pages // 2 + 7])[None]
    t = torch.arange(n, device=DEV)
    slots = table[0].long()[t // page] * page + t % page
    k, v = randn(g, n, heads, dim), randn(g, n, heads, dim)
    h.rope_append(randn(g, n, 2 * heads, dim), k, v, t.to(I32), slots.to(I32), None, c.cache, torch.empty(n, 2 * heads, dim, dtype=BF16, device=DEV))
    assert h.sync_status() == 0
    if kind == "bf16":
        assert torch.equal(c.rows("k", slots).to(BF16), k) and torch.equal(c.rows("v", slots).to(BF16), v)
    check_attn(h, randn(g, 1, 2 * heads, dim, scale=2), c, table, ints([n]), [slots], dim ** -0.5, 0)


def test_attn_scales_off_the_16_byte_boundaries(h):  # noqa: F811
    """Boxes need aligned scales; without them rows are copied one by one."""
    g = gen(7)
    lens = [100, 40]
    c, table, slots = filled(g, lens, 2, 64, 16, "e4m3")
    q = randn(g, 2, 8, 64, scale=2)
    out, _ = check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)

    def shifted(s):
        t = torch.full((s.numel() + 4,), NAN, device=DEV)
        t[1:1 + s.numel()] = s.flatten()
        return t[1:1 + s.numel()].view(s.shape)
    c.ks, c.vs = shifted(c.ks), shifted(c.vs)
    c.cache = tovl.KVCache(c.k, c.v, c.ks, c.vs)
    again, _ = check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)
    assert torch.equal(out, again)


def test_without_programmatic_launches(h):  # noqa: F811
    g = gen(8)
    lens = [100, 4000]
    c, table, slots = filled(g, lens, 2, 64, 16, "bf16")
    q = randn(g, 2, 8, 64, scale=2)
    out, _ = check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)
    h.set_option(tovl.OPT_PDL, 0)
    try:
        again, _ = check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)
        check_append(h, g, 5, 4, 2, 64, 64, 16, "bf16", "nhd", False)
        p = Plan(3, 4, 12, 8)
        dev = Planned(p)
        same_plan(p, dev, p.step([9, 0, 20], 40), dev.step(h, [9, 0, 20], 40))
    finally:
        h.set_option(tovl.OPT_PDL, 1)
    assert torch.equal(out, again)


def test_attn_lengths_near_the_largest_int(h):  # noqa: F811
    """A table of 2^31 tokens, all in one page: a window at the end of the longest request, and a length beyond it."""
    g = gen(10)
    page = 1 << 20
    c = Cache(1, page, 1, 16, "bf16")
    c.k.copy_(randn(g, *c.k.shape))
    c.v.copy_(randn(g, *c.v.shape))
    table = torch.zeros(1, 2048, dtype=I32, device=DEV)
    q = randn(g, 1, 2, 16)
    n = 2 ** 31 - 64
    slots = torch.arange(n - 100, n, device=DEV) % page
    check_attn(h, q, c, table, ints([n]), [slots], 0.25, 100)
    h.attn_decode(q, c.cache, table, ints([2 ** 31 - 1]), 0.25, torch.empty_like(q), space(h.attn_decode_workspace(2, 1, 16)), window=100)
    assert h.sync_status() == tovl.TOVL_ERR_INVALID


def test_attn_bad_pages_and_lengths_are_reported(h):  # noqa: F811
    """They are recognised on the device before an address is made of them."""
    g = gen(9)
    lens = [100, 100]
    c, table, slots = filled(g, lens, 1, 64, 16, "bf16")
    q = randn(g, 2, 2, 64)
    ws = space(h.attn_decode_workspace(2, 1, 64))
    clean, _ = check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)
    for page in (-1, c.k.shape[0], 1 << 30):
        bad = table.clone()
        bad[1, 3] = page
        out = torch.empty_like(q)
        h.attn_decode(q, c.cache, bad, ints(lens), 0.125, out, ws)
        assert h.sync_status() == tovl.TOVL_ERR_INVALID
        assert torch.equal(out[0], clean[0])
    for n in (-1, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        bad = table.clone()
        bad[1] = 0
        out = torch.empty_like(q)
        h.attn_decode(q, c.cache, bad, ints(100, n), 0.125, out, ws)
        assert h.sync_status() == tovl.TOVL_ERR_INVALID
        assert torch.equal(out[0], clean[0])
    check_attn(h, q, c, table, ints(lens), slots, 0.125, 0)


# ------------------------------------------------------------------ rotary embedding and cache writes
def turn(x, cs, rot, interleaved):
    x = x.to(D).clone()
    half = rot // 2
    c, s = cs[:, None, :half].to(D), cs[:, None, half:].to(D)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    u, w = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    mag = torch.zeros_like(x)
    mag[..., a], mag[..., b] = (u * c).abs() + (w * s).abs(), (w * c).abs() + (u * s).abs()
    return x, 2 * U32 * mag


def angles(far, rot):
    a = torch.arange(far, device=DEV, dtype=D)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=D) * 2 / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def check_append(h, g, T, Hq, heads, dim, rot, page, kind, layout, interleaved, in_place=False, far=500, grow=1.0):  # noqa: F811
    pages = -(-T // page) + 2
    c = Cache(pages, page, heads, dim, kind, layout)
    qkv = randn(g, T, (Hq + 2 * heads) * dim + 24, scale=grow)
    q, k, v = (qkv[:, a * dim:b * dim].view(T, b - a, dim) for a, b in ((0, Hq), (Hq, Hq + heads), (Hq + heads, Hq + 2 * heads)))
    q0 = q.clone()
    positions = torch.randint(0, far, (T,), generator=g, device=DEV).to(I32)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(I32)
    if T > 2:
        slots[T - T // 3:] = -1
        slots[0] = -1
    real = slots >= 0
    cs = angles(far, rot) if rot else None
    before = [t.clone().view(torch.uint8) for t in (c.k, c.v)]
    q_out = q if in_place else torch.full((T, Hq, dim), NAN, dtype=BF16, device=DEV)
    h.rope_append(q, k, v, positions, slots, cs, c.cache, q_out, interleaved=interleaved)
    assert h.sync_status() == 0
    table = cs[positions.long()] if rot else torch.zeros(T, 0, device=DEV)
    want, err = turn(q0, table, rot, interleaved)
    within(q_out, want, U16 * want.abs() + err + 2.0 ** -133, "q_out")
    at = slots[real].long()
    for n, (x, e) in (("k", turn(k, table, rot, interleaved)), ("v", (v.to(D), torch.zeros_like(v, dtype=D)))):
        x, e = x[real], e[real]
        if kind == "bf16":
            within(c.rows(n, at), x, U16 * x.abs() + e + 2.0 ** -133, n)
        else:
            s = (c.ks if n == "k" else c.vs)[at // page, :, at % page]
            top = x.abs().amax(2).clamp_min(1e-12) / 448
            within(s, top, 4 * U32 * top + e.amax(2) / 448, n + "_scale")
            y = (c.k if n == "k" else c.v).view(torch.uint8)[at // page, at % page].view(E4M3).to(D)
            z = x / top[:, :, None]
            within(y, z, 2.0 ** -4 * z.abs().clamp_min(2.0 ** -6) + 448 * 8 * U32 + (e + e.amax(2, keepdim=True)) / top[:, :, None], n)
    # other slots as they were
    for t, b in zip((c.k, c.v), before):
        t = t.clone()
        t.view(torch.uint8)[at // page, at % page] = b.view(*t.shape[:3], -1)[at // page, at % page]
        assert torch.equal(t.view(torch.uint8), b)
    for s in (c.ks, c.vs):
        if s is not None:
            other = s.clone()
            other[at // page, :, at % page] = NAN
            assert other.isnan().all()


@pytest.mark.parametrize("T", [1, 2, 5, 64, 301])
@pytest.mark.parametrize("Hq,heads,dim,rot", [(1, 1, 16, 16), (4, 2, 64, 32), (6, 2, 80, 80), (5, 1, 96, 48), (32, 8, 128, 128), (3, 3, 240, 16),
                                              (4, 1, 256, 256), (4, 2, 48, 0), (7, 1, 112, 64)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_matches_the_formula(h, T, Hq, heads, dim, rot, kind, interleaved):  # noqa: F811
    for page, layout in ((16, "nhd"), (7, "hnd")):
        check_append(h, gen(T * 1000 + dim + rot), T, Hq, heads, dim, rot, page, kind, layout, interleaved)


@pytest.mark.parametrize("dim,rot", [(8, 0), (24, 16), (72, 64), (136, 128)])
def test_append_odd_head_sizes(h, dim, rot):  # noqa: F811
    check_append(h, gen(dim), 9, 3, 2, dim, rot, 16, "bf16", "wide", False)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_many_rows_in_place_and_any_magnitude(h, kind):  # noqa: F811
    check_append(h, gen(1), 9001, 32, 8, 128, 128, 16, kind, "both", True, in_place=True)
    check_append(h, gen(2), 9001, 10, 2, 64, 64, 16, kind, "hnd", False)
    for grow in (2.0 ** -60, 2.0 ** 100):
        check_append(h, gen(3), 33, 4, 2, 64, 64, 16, kind, "nhd", False, grow=grow)


def test_append_nan_shows_in_the_scale(h):  # noqa: F811
    c = Cache(2, 16, 1, 64, "e4m3")
    x = torch.zeros(3, 1, 64, dtype=BF16, device=DEV)
    x[1, 0, 5] = NAN
    x[2, 0, 63] = -math.inf
    q_out = torch.empty_like(x)
    h.rope_append(x, x, x, ints(0, 0, 0), ints(0, 1, 2), None, c.cache, q_out)
    assert h.sync_status() == 0
    assert c.ks[0, 0, 0] == torch.tensor(1e-12) / 448 and c.ks[0, 0, 1].isnan() and c.vs[0, 0, 2] == math.inf
    assert torch.equal(q_out.isnan(), x.isnan())


def test_append_bad_slots_and_positions_are_reported(h):  # noqa: F811
    g = gen(4)
    c = Cache(2, 16, 1, 64, "bf16")
    x = randn(g, 2, 1, 64)
    cs = angles(50, 64)
    for slots, pos in (((-2, 3), (0, 0)), ((32, 3), (0, 0)), ((5, 3), (50, 0)), ((5, 3), (-1, 0)), ((2 ** 31 - 1, 3), (0, 0))):
        h.rope_append(x, x, x, ints(*pos), ints(*slots), cs, c.cache, torch.empty_like(x))
        assert h.sync_status() == tovl.TOVL_ERR_INVALID
        assert c.k[0, 3].isfinite().all() and int(c.k.isfinite().all(3).sum()) == 1
    h.rope_append(x, x, x, ints(70, 0), ints(-1, 3), cs, c.cache, torch.empty_like(x))   # of a token that is not written
    assert h.sync_status() == 0


# ------------------------------------------------------------------ page plan
class Plan:
    """The plan in plain Python."""

    def __init__(self, B, width, pages, page, head=0):
        self.B, self.width, self.pages, self.page = B, width, pages, page
        self.length, self.table = [0] * B, [[-5] * width for _ in range(B)]
        self.ring = [(i - head) % pages for i in range(pages)]
        self.head, self.free = head, pages

    def step(self, add, cap):
        """slots, positions, starts, state_out"""
        up = lambda n: -(-n // self.page)  # noqa: E731
        take = [up(n + a) - up(n) if a > 0 else 0 for n, a in zip(self.length, add)]
        none = [-1] * cap, [0] * cap, [0] * (self.B + 1)
        if sum(take) > self.free:
            return (*none, [self.head, self.free, 0, sum(take) - self.free])
        if sum(max(a, 0) for a in add) > cap or any(a < -1 or n + a > self.width * self.page for n, a in zip(self.length, add)):
            return (*none, [self.head, self.free, 0, -1])
        slots, positions, starts = [], [], [0]
        tail = (self.head + self.free) % self.pages
        for b, a in enumerate(add):
            if a < 0:
                for p in self.table[b][:up(self.length[b])]:
                    self.ring[tail] = p
                    tail = (tail + 1) % self.pages
                    self.free += 1
                self.length[b] = 0
            else:
                for i in range(take[b]):
                    self.table[b][up(self.length[b]) + i] = self.ring[self.head]
                    self.head = (self.head + 1) % self.pages
                    self.free -= 1
                for pos in range(self.length[b], self.length[b] + a):
                    slots.append(self.table[b][pos // self.page] * self.page + pos % self.page)
                    positions.append(pos)
                self.length[b] += a
            starts.append(len(slots))
        n = len(slots)
        return slots + [-1] * (cap - n), positions + [0] * (cap - n), starts, [self.head, self.free, n, 0]


class Planned:
    """The same on the device, in place."""

    def __init__(self, p):
        self.length, self.table = ints(p.length), ints(p.table) if p.B > 1 else ints(p.table[0])[None]
        self.ring, self.state, self.page = ints(p.ring), ints(p.head, p.free, 7, 7), p.page

    def step(self, h, add, cap, stream=None):  # noqa: F811
        out = [torch.full((n,), -77, dtype=I32, device=DEV) for n in (cap, cap, len(add) + 1)]
        h.page_plan(self.length, ints(add), self.table, self.ring, self.state, self.page, self.length, self.state, *out, stream=stream)
        return out


def same_plan(p, dev, want, got):
    for name, w, x in zip(("slots", "positions", "starts"), want, got):
        assert x.tolist() == w, name
    assert dev.state.tolist() == want[3], "state"
    assert dev.length.tolist() == p.length, "length"
    assert dev.table.tolist() == p.table, "table"
    assert dev.ring.tolist() == p.ring, "ring"


@pytest.mark.parametrize("B,page,pages,width", [(1, 16, 40, 30), (3, 1, 50, 20), (7, 16, 100, 40), (64, 5, 700, 30), (513, 16, 3000, 12),
                                                (4096, 8, 30000, 9)])
@pytest.mark.parametrize("room", [0, 9000])
def test_plan_follows_a_serving_run(h, B, page, pages, width, room):  # noqa: F811
    rng = np.random.default_rng(B + page)
    p = Plan(B, width, pages, page, head=pages // 3)
    dev = Planned(p)
    lacked = 0
    for step in range(12):
        add = []
        for n in p.length:
            left = width * page - n
            kind = rng.random()
            add.append(-1 if n and kind < 0.15 else 0 if kind < 0.25 else min(left, 1) if n and kind < 0.9
                       else int(rng.integers(0, min(left, 6 * page) + 1)))
        cap = sum(max(a, 0) for a in add) + room
        want = p.step(add, cap)
        got = dev.step(h, add, cap)
        assert h.sync_status() == 0
        same_plan(p, dev, want, got)
        lacked += want[3][3] > 0
        if want[3][3] > 0:      # the longest requests make room
            order = sorted(range(B), key=lambda b: -p.length[b])[: B // 2 + 1]
            add = [-1 if b in order and p.length[b] else 0 for b in range(B)]
            same_plan(p, dev, p.step(add, 8), dev.step(h, add, 8))


def test_plan_lacking_pages_and_impossible_counts_change_nothing(h):  # noqa: F811
    p = Plan(3, 4, 6, 8)
    dev = Planned(p)
    same_plan(p, dev, p.step([9, 0, 20], 40), dev.step(h, [9, 0, 20], 40))
    same_plan(p, dev, p.step([1, 17, 0], 40), dev.step(h, [1, 17, 0], 40))      # two pages lack
    assert h.sync_status() == 0
    for add, cap in (([0, -2, 0], 9), ([24, 0, 0], 40), ([5, 1, 1], 6), ([2 ** 31 - 1, 2 ** 31 - 1, 0], 9)):
        got = dev.step(h, add, cap)
        assert h.sync_status() == tovl.TOVL_ERR_INVALID
        same_plan(p, dev, ([-1] * cap, [0] * cap, [0] * 4, [p.head, p.free, 0, -1]), got)
    for state in ([6, 0, 0, 0], [-1, 3, 0, 0], [0, 7, 0, 0], [0, 6, 0, 0]):     # (the last: more free ones than are left, with an end)
        dev.state.copy_(ints(state))
        dev.step(h, [-1, 0, 0], 4)
        assert h.sync_status() == tovl.TOVL_ERR_INVALID
        assert dev.state.tolist() == [state[0], state[1], 0, -1] and dev.ring.tolist() == p.ring and dev.length.tolist() == p.length


def test_plan_of_long_prompts_and_separate_outputs(h):  # noqa: F811
    B, page = 5, 16
    p = Plan(B, 5000, 20000, page, head=19990)
    dev = Planned(p)
    add = [50000, 1, 0, 70001, 16]
    cap = sum(add) + 100
    length, state = dev.length.clone(), dev.state.clone()
    out = [torch.empty(n, dtype=I32, device=DEV) for n in (cap, cap, B + 1)]
    length_out, state_out = torch.empty_like(length), torch.empty_like(state)
    for _ in range(2):          # the inputs stay, so a repeated call gives the same
        h.page_plan(length, ints(add), dev.table, dev.ring, state, page, length_out, state_out, *out)
        assert h.sync_status() == 0
    assert length.tolist() == [0] * B and state.tolist()[:2] == [19990, 20000]
    want = p.step(add, cap)
    dev.length, dev.state = length_out, state_out
    same_plan(p, dev, want, out)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_run(h, kind, captured):  # noqa: F811
    """Prompts are admitted, then tokens generated step by step; every step's attention against all keys and values
    that went before it."""
    g = gen(11)
    B, Hq, heads, dim, page, pages, width, cap, far = 4, 8, 2, 64, 16, 64, 12, 128, 256
    c = Cache(pages, page, heads, dim, kind)
    p = Plan(B, width, pages, page)
    dev = Planned(p)
    cs = angles(far, dim)
    add = torch.zeros(B, dtype=I32, device=DEV)
    slots, positions, starts = (torch.zeros(n, dtype=I32, device=DEV) for n in (cap, cap, B + 1))
    qkv = torch.zeros(cap, (Hq + 2 * heads) * dim, dtype=BF16, device=DEV)
    q, k, v = (qkv[:, a * dim:b * dim].view(cap, b - a, dim) for a, b in ((0, Hq), (Hq, Hq + heads), (Hq + heads, Hq + 2 * heads)))
    q_out = torch.zeros(cap, Hq, dim, dtype=BF16, device=DEV)
    out, ws = torch.zeros(B, Hq, dim, dtype=BF16, device=DEV), space(h.attn_decode_workspace(Hq, heads, dim))

    def step():
        h.page_plan(dev.length, add, dev.table, dev.ring, dev.state, page, dev.length, dev.state, slots, positions, starts)
        h.rope_append(q, k, v, positions, slots, cs, c.cache, q_out)
        last = (starts[1:].long() - 1).clamp_min(0)
        h.attn_decode(q_out[last].contiguous(), c.cache, dev.table, dev.length, dim ** -0.5, out, ws)

    graph = None
    for i in range(8):
        count = [40, 1, 0, 33] if i == 0 else [1, 1, 5, 1] if i == 3 else [1, -1, 1, 1] if i == 5 else [1, 1, 1, 1]
        if i == 6:
            count[1] = 30
        add.copy_(ints(count))
        qkv.copy_(randn(g, *qkv.shape))
        if captured and graph is None and i == 1:
            keep = [t.clone() for t in (dev.length, dev.table, dev.ring, dev.state)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for t, s in zip((dev.length, dev.table, dev.ring, dev.state), keep):
                assert torch.equal(t, s)        # capturing runs nothing
        if graph is None:
            step()
        else:
            graph.replay()
        assert h.sync_status() == 0
        want = p.step(count, cap)
        same_plan(p, dev, want, (slots, positions, starts))
        # this step's rows are in the cache as the formula gives them
        n = want[3][2]
        rows, err = turn(k[:n], cs[positions[:n].long()], dim, False)
        if kind == "bf16":
            within(c.rows("k", slots[:n]), rows, U16 * rows.abs() + err, "keys")
        else:
            within(c.rows("k", slots[:n]), rows, 2.0 ** -4 * rows.abs() + 2.0 ** -10 * rows.abs().amax(2, keepdim=True) / 400 + err, "keys")
        live = [torch.tensor([p.table[b][t // page] * page + t % page for t in range(p.length[b])], device=DEV, dtype=torch.long) for b in range(B)]
        last = (starts[1:].long() - 1).clamp_min(0)
        want, bound, _, _ = attn_reference(q_out[last], c, live, dim ** -0.5, 0)
        within(out, want, bound, f"step {i}")


def test_two_handles_on_two_streams(h):  # noqa: F811
    """Calls that run at the same time have a handle and a workspace each."""
    g = gen(12)
    lens = [4000, 17, 900]
    c, table, slots = filled(g, lens, 2, 128, 16, "bf16")
    q = randn(g, 3, 8, 128, scale=2)
    want, bound, _, _ = attn_reference(q, c, slots, 128 ** -0.5, 0)
    with tovl.Handle(0) as other:
        jobs = []
        for handle in (h, other):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            jobs.append((handle, s, [torch.empty_like(q) for _ in range(20)], space(handle.attn_decode_workspace(8, 2, 128))))
        n = ints(lens)
        torch.cuda.synchronize()
        for i in range(20):
            for handle, s, outs, ws in jobs:
                handle.attn_decode(q, c.cache, table, n, 128 ** -0.5, outs[i], ws, stream=s)
        for handle, s, outs, ws in jobs:
            assert handle.sync_status() == 0
            within(outs[0], want, bound, "out")
            assert all(torch.equal(o, outs[0]) for o in outs)
        assert torch.equal(jobs[0][2][0], jobs[1][2][0])


def test_binding_refuses_wrong_tensors(h):  # noqa: F811
    g = gen(13)
    c, table, slots = filled(g, [20, 3], 2, 64, 16, "bf16")
    q, n, ws = randn(g, 2, 4, 64), ints(20, 3), space(h.attn_decode_workspace(4, 2, 64))
    out = torch.empty_like(q)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(length=n.long()),
                dict(length=ints(1, 2, 3)), dict(table=table.long()), dict(table=table[:1]), dict(out=out[:, :2]), dict(out=out.float()),
                dict(lse=torch.empty(2, 3, device=DEV)), dict(workspace=ws[::2])):
        a = dict(q=q, cache=c.cache, table=table, length=n, scale=0.125, out=out, workspace=ws)
        with pytest.raises(TypeError):
            h.attn_decode(**{**a, **bad})
    for bad in (dict(workspace=ws[:-1]), dict(workspace=ws[16:]), dict(window=-1), dict(out=out.view(-1)[:4 * 64 * 2].as_strided((2, 4, 64), (128, 64, 1)))):
        a = dict(q=q, cache=c.cache, table=table, length=n, scale=0.125, out=out, workspace=ws)
        with pytest.raises(tovl.TovlError):
            h.attn_decode(**{**a, **bad})
    with pytest.raises(tovl.TovlError):
        h.attn_decode(randn(g, 2, 3, 64), c.cache, table, n, 0.125, torch.empty(2, 3, 64, dtype=BF16, device=DEV), ws)
    k = torch.zeros(3, 16, 2, 64, dtype=BF16, device=DEV)
    s = torch.ones(3, 2, 16, device=DEV)
    e = k.to(E4M3)
    for bad in ((k, k.float()), (k, k[:2]), (k, k.transpose(1, 2).contiguous().transpose(1, 2)), (k, k, s, s), (e, e), (e, e, s, None),
                (e, e, s, s[:2]), (k[0], k[0]), (k.half(), k.half())):
        with pytest.raises(TypeError):
            tovl.KVCache(*bad)
    with pytest.raises(tovl.TovlError):
        h.attn_decode_workspace(3, 2, 64)
    assert h.sync_status() == 0
