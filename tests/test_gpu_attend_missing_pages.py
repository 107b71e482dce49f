"""mx_attend where the table names pages outside the cache: their tokens count as rows of zeros, whatever ran before."""
import pytest
import torch

from gpu_helpers import dev
from test_gpu_attend import SHAPES, Case, nan_rows
from test_gpu_attend_latent import case as latent_case
from test_gpu_attend_rows import SHAPES as ROWS_SHAPES
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = [("few", *s) for s in SHAPES] + [("many", *s) for s in ROWS_SHAPES] + [("latents", 16, 1, 512, True)]


def make(mx, kind, shape, lengths, counts, **kw):  # noqa: F811
    """counts: query tokens where rows are few; forty times as many where they are not."""
    if kind == "few":
        return Case(mx, lengths, counts, *shape, **kw)
    counts = [40 * n for n in counts]
    return latent_case(mx, lengths, counts, **kw) if kind == "latents" else Case(mx, lengths, counts, *shape, **kw)


def without(c, gone):
    """Pages gone[b] (columns of the table) of sequence b lie outside the cache, which counts as zeros."""
    rows, outside = c.rows, [c.cache.pages, -1, -2**31, 2**31 - 1, c.cache.pages + 5]
    for b, cols in gone.items():
        for i, col in enumerate(cols):
            assert col * c.page < c.lengths[b]
            c.table[b, col] = outside[i % len(outside)]

    def zeroed(name, b):
        x = rows(name, b)
        for col in gone.get(b, ()):
            x[col * c.page:(col + 1) * c.page] = 0
        return x
    c.rows = zeroed


def loud(mx, kind, shape, scale):  # noqa: F811
    """A call whose tiles have this scale everywhere, and leave it in shared memory; its results say nothing."""
    c = make(mx, kind, shape, [1500] * 40, [1] * 40, fill=scale)
    for t in (c.cache.k_scales, c.cache.v_scales):
        if t is not None:
            t.fill_(scale)
    return c


def reported(c):
    assert c.mx.mx_device_status(c.h) == c.mx.MX_ERR_INVALID_ARG


@pytest.mark.parametrize("kind,group,heads,d,shared", KINDS)
def test_missing_pages_are_zeros(mx, kind, group, heads, d, shared):  # noqa: F811
    """Behind calls with large and with small scales: all tokens of a row, of a tile, and some of them."""
    shape = (group, heads, d, shared)
    c = make(mx, kind, shape, [16, 130, 300, 700], [1, 1, 3, 2], page=16, seed=1)
    without(c, {0: [0], 1: [0, 1, 8], 2: range(8, 16), 3: [3, 20, 21, 40, 43]})
    for scale in (0xE3, 0x01):
        before = loud(mx, kind, shape, scale)
        for kw in (dict(), dict(window=100)):
            before.run()
            mx.mx_device_status(c.h)
            out, lse = c.run(lse=True, **kw)
            reported(c)
            c.check(out, lse, **kw)
        assert all(torch.equal(c.run(window=100), out) for _ in range(3))
        reported(c)


@pytest.mark.parametrize("kind,group,heads,d,shared", KINDS)
def test_missing_pages_beside_a_nan(mx, kind, group, heads, d, shared):  # noqa: F811
    """A NaN value that only some rows see, in a tile with missing pages, behind a call all of whose scales are NaN."""
    shape = (group, heads, d, shared)
    n = 5 if kind == "few" else 1
    c = make(mx, kind, shape, [130, 300], [n, n], page=16, seed=2)
    for b, tokens in ((0, [129]), (1, [299])):
        nan_rows(c, "k" if shared else "v", b, tokens, 1)
    without(c, {0: [0, 2, 5, 7], 1: [0, 1, 9, 12, 17]})
    before = loud(mx, kind, shape, 0xFF)
    for kw in (dict(), dict(window=200)):
        before.run()
        mx.mx_device_status(c.h)
        out = c.run(**kw)
        reported(c)
        c.check(out, **kw)


@pytest.mark.parametrize("group,heads,d,shared", [s for s in SHAPES if not s[3]])
def test_missing_pages_behind_tiles_with_large_scales(mx, group, heads, d, shared):  # noqa: F811
    """Few rows, all in one call: tokens whose values are large and whose weights are next to nothing come first, and pages are
    missing in the tiles that take their places in shared memory. So many equal sequences that a CTA has all their tiles."""
    c = Case(mx, [1280], [1], group, heads, d, shared, page=16, seed=3)
    g = torch.Generator(device=dev()).manual_seed(4)
    sign = torch.sign(torch.randn(d, generator=g, device=dev()))
    c.q = (sign + 0.1 * torch.randn(c.q.shape, generator=g, device=dev())).to(c.q.dtype)
    slots = torch.from_numpy(c.slots[0][:512]).to(dev())  # four tiles
    # scores of -90 and below (a weight of 2^-130), small enough for the rounding of their sums to say nothing
    k = (-{64: 16, 128: 8, 256: 8, 512: 4}[d] * sign).expand(512, heads, d).bfloat16().contiguous()
    v = (2.0**60 * torch.randn(512, heads, d, generator=g, device=dev())).bfloat16()
    mx.mx_cache_write(c.h, c.cache, slots, k, None if shared else v)
    without(c, {0: [c0 + i for c0 in range(32, 64, 8) for i in (0, 3, 6)]})
    b = 512 // heads
    every = mx.mx_attend(c.h, c.q.repeat(b, 1, 1), c.cache, c.table.repeat(b, 1), c.len_t.repeat(b))
    reported(c)
    results = torch.unique(every.float(), dim=0)  # runs are cut at different tiles
    assert len(results) < 256
    for out in results:
        c.check(out.to(c.q.dtype)[None])
