"""mx_attend of many query rows (prompts, drafts, wide groups) against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev
from test_gpu_attend import Case, nan_rows
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(4, 2, 128, False), (8, 1, 64, True), (1, 3, 64, False), (5, 1, 128, True), (2, 2, 256, False), (8, 1, 256, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_prompts(mx, group, heads, d, shared, dtype):  # noqa: F811
    """Prompts of ragged lengths: alone, behind a prefix, of one token, of none, longer than what is cached."""
    c = Case(mx, [130, 300, 1, 64, 257, 40, 0], [130, 129, 1, 0, 200, 45, 3], group, heads, d, shared, 48, dtype, seed=1)
    out, lse = c.run(lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_all_see_all(mx, group, heads, d, shared):  # noqa: F811
    c = Case(mx, [200, 129, 77], [70, 100, 64], group, heads, d, shared, 16, seed=2)
    for scale in (0.15, -0.1, 0.0):
        out, lse = c.run(lse=True, causal=False, scale=scale)
        c.check(out, lse, causal=False, scale=scale)


@pytest.mark.parametrize("window", [1, 40, 128, 1000])
@pytest.mark.parametrize("group,heads,d,shared", [(4, 2, 128, False), (2, 1, 256, False), (8, 1, 64, True)])
def test_windows(mx, group, heads, d, shared, window):  # noqa: F811
    c = Case(mx, [500, 90], [300, 90], group, heads, d, shared, 32, seed=3)
    out, lse = c.run(lse=True, window=window)
    c.check(out, lse, window=window)


@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_few_rows_of_long_contexts(mx, group, heads, d, shared):  # noqa: F811
    """Fewer blocks of rows than SMs: the tokens are split and joined."""
    n = 80 // group + 3
    c = Case(mx, [3001, 2000], [n, n], group, heads, d, shared, seed=4)
    out, lse = c.run(lse=True, q_offsets=None)
    c.check(out, lse)
    assert torch.equal(c.run(), out)


@pytest.mark.parametrize("sizes", [dict(q_size=2.0**-60), dict(q_size=30.0), dict(k_size=2.0**60, q_size=2.0**-60),
                                   dict(v_size=2.0**60), dict(v_size=2.0**-100), dict(k_size=2.0**-40, q_size=2.0**40)])
@pytest.mark.parametrize("group,heads,d", [(4, 1, 128), (2, 1, 256)])
def test_sizes_of_values(mx, group, heads, d, sizes):  # noqa: F811
    c = Case(mx, [300], [64], group, heads, d, False, seed=5, **sizes)
    c.check(c.run())


def test_growing_scores_and_values(mx):  # noqa: F811
    """Each tile's scores and values are larger than all before: references and sums are scaled anew."""
    c = Case(mx, [900], [70], 2, 1, 128, False, 16, seed=6)
    for b, slots in enumerate(c.slots):
        for t, s in enumerate(slots):
            for side in ("k_scales", "v_scales"):
                x = getattr(c.cache, side)
                x[s // 16, :, s % 16] += t // 128
    out, lse = c.run(lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("group,heads,d,shared", [(4, 2, 128, False), (4, 1, 128, True), (2, 1, 256, False), (8, 1, 64, True)])
def test_nan_reaches_the_rows_that_see_it(mx, group, heads, d, shared):  # noqa: F811
    n = 96 // group + 20
    for side in ("k",) if shared else ("k", "v"):
        for window, tokens in ((0, [n + 30]), (20, [37, n + 10])):
            c = Case(mx, [n + 36, 20], [n, 20], group, heads, d, shared, 16, seed=7)
            nan_rows(c, side, 0, tokens, 1)
            out, lse = c.run(window=window, lse=True)
            c.check(out, None, window=window)
            nan = torch.isnan(out[:n]).any(2).any(1)
            pos = torch.arange(36, n + 36, device=dev())
            want = torch.zeros_like(nan)
            for t in tokens:
                want |= (pos >= t) & ((pos < t + window) if window else True)
            assert want.any() and not want.all()
            assert torch.equal(nan, want) and not torch.isnan(out[n:]).any()
            if side == "k":
                assert torch.equal(torch.isnan(lse[:n]).all(1), want)


def test_nan_and_infinite_queries_stay_in_their_rows(mx):  # noqa: F811
    c = Case(mx, [200], [50], 4, 1, 128, False, seed=8)
    clean = c.run()
    c.q[0, 1, 7] = float("nan")
    c.q[40, 3, 9] = float("inf")
    out = c.run()
    bad = torch.zeros(50, 4, dtype=torch.bool, device=dev())
    bad[0, 1] = bad[40, 3] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def test_same_bits_in_graphs_and_on_streams(mx):  # noqa: F811
    for lengths, counts in (([700, 1300, 64], [300, 20, 64]), ([4000], [33])):
        c = Case(mx, lengths, counts, 4, 2, 128, False, seed=9)
        want = c.run()
        assert all(torch.equal(c.run(), want) for _ in range(5))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got, other = c.run(stream=side), c.run()
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                out = c.run()
            graphs.append((graph, out))
        for _, out in graphs:
            out.zero_()
        torch.cuda.synchronize()
        for stream, (graph, _) in zip((torch.cuda.Stream(), torch.cuda.Stream()), graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want) and all(torch.equal(out, want) for _, out in graphs)


def test_strides_and_untouched_rows(mx):  # noqa: F811
    c = Case(mx, [77, 130], [60, 70], 4, 2, 128, False, seed=10)
    want = c.run()
    room = torch.full((140, 11, 136), 3.0, dtype=torch.bfloat16, device=dev())
    out = room[:, 3:, :128]
    q = torch.cat([c.q, c.q[:10]]).transpose(0, 1).contiguous().transpose(0, 1)
    mx.mx_attend(c.h, q, c.cache, c.table, c.len_t, q_offsets=c.off_t, out=out)
    assert torch.equal(out[:130], want)
    assert (room[130:] == 3).all() and (room[:, :3] == 3).all() and (room[..., 128:] == 3).all()


def test_wrong_pages_and_offsets_are_reported(mx):  # noqa: F811
    c = Case(mx, [170, 140], [100, 90], 4, 1, 128, False, page=16, seed=11)
    mx.mx_device_status(c.h)
    want = c.run()
    assert mx.mx_device_status(c.h) == mx.MX_OK
    table = c.table.clone()
    table[1, 1] = c.cache.pages
    got = mx.mx_attend(c.h, c.q, c.cache, table, c.len_t, q_offsets=c.off_t)
    assert mx.mx_device_status(c.h) == mx.MX_ERR_INVALID_ARG
    assert torch.equal(got[:100], want[:100]) and torch.isfinite(got).all()
    for offsets in ([0, 100, 191], [0, 150, 90], [-1, 100, 190]):
        mx.mx_attend(c.h, c.q, c.cache, c.table, c.len_t, q_offsets=torch.tensor(offsets, dtype=torch.int32, device=dev()))
        assert mx.mx_device_status(c.h) == mx.MX_ERR_INVALID_ARG


def test_scores_of_any_size(mx):  # noqa: F811
    """Scores of 2^40 in steps of 2^18: a weight is 1 or 0, and the largest score's own has to be 1."""
    c = Case(mx, [140], [140], 2, 1, 64, False, seed=12, q_size=2.0**20, k_size=2.0**20)
    out = c.run(causal=False)
    k, v, q = c.rows("k", 0)[:, 0], c.rows("v", 0)[:, 0], c.q.double().cpu().numpy()
    for j in range(2):
        x = q[:, j] @ k.T
        top = np.sort(x, 1)
        sure = top[:, -1] - top[:, -2] > 2.0**24 * 64  # beyond any rounding of the scores
        assert sure.sum() > 100
        want = torch.from_numpy(v[x.argmax(1)]).bfloat16()
        assert torch.equal(out[:, j].cpu()[torch.from_numpy(sure)], want[torch.from_numpy(sure)])
