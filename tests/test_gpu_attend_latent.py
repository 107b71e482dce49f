"""mx_attend over latents of 512 dimensions (keys and values in one), many rows and room for long sequences."""
import pytest
import torch

from gpu_helpers import dev
from test_gpu_attend import Case, nan_rows
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu


def case(mx, lengths, counts, group=16, heads=1, **kw):  # noqa: F811
    """The sequences, and behind them one with so many queries that 128 rows or more come to each, in a wide table."""
    more = max(0, -(-128 * (len(lengths) + 1) // group) - sum(counts)) if sum(counts) * group < 128 * len(lengths) else 0
    c = Case(mx, lengths + [90] * (more > 0), counts + [more] * (more > 0), group, heads, 512, True, **kw)
    cols = 160 * 16 * 64 * 128 // (len(c.q) * group * c.page) + 1
    wide = torch.full((len(c.table), max(cols, c.table.shape[1])), -1, dtype=torch.int32, device=dev())
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,heads", [(16, 1), (9, 2), (20, 1), (48, 1)])
def test_equal_queries(mx, group, heads, dtype):  # noqa: F811
    lengths = [1, 16, 17, 127, 128, 129, 255, 300, 513]
    c = case(mx, lengths, [-(-128 // group)] * len(lengths), group, heads, dtype=dtype, page=48)
    out, lse = c.run(lse=True, q_offsets=None)
    c.check(out, lse)


@pytest.mark.parametrize("group,counts", [(16, [1, 1, 1, 1, 1]), (16, [2, 0, 2, 1, 3]), (16, [9, 64, 2, 0, 40]), (3, [70, 1, 4, 30, 11])])
def test_ragged_queries(mx, group, counts):  # noqa: F811
    """More queries than tokens, sequences without queries and without tokens, blocks cut anywhere."""
    c = case(mx, [40, 64, 0, 300, 150], counts, group, seed=1, page=16)
    out, lse = c.run(lse=True)
    c.check(out, lse)
    out = c.run(causal=False, scale=-0.02)
    c.check(out, causal=False, scale=-0.02)


@pytest.mark.parametrize("window", [1, 40, 128, 1000])
def test_windows(mx, window):  # noqa: F811
    c = case(mx, [700, 90, 300], [1, 1, 30], seed=2, page=32)
    out, lse = c.run(lse=True, window=window)
    c.check(out, lse, window=window)


@pytest.mark.parametrize("lengths,counts", [([9001], [1]), ([9001], [3]), ([3000, 2500], [4, 1]), ([1500], [400])])
def test_units_cut_between_runs(mx, lengths, counts):  # noqa: F811
    c = case(mx, lengths, counts, seed=3)
    out, lse = c.run(lse=True)
    c.check(out, lse)
    assert all(torch.equal(c.run(), out) for _ in range(3))


@pytest.mark.parametrize("sizes", [dict(q_size=2.0**-60), dict(q_size=30.0), dict(k_size=2.0**60, q_size=2.0**-60),
                                   dict(k_size=2.0**-100), dict(k_size=2.0**-40, q_size=2.0**40)])
def test_sizes_of_values(mx, sizes):  # noqa: F811
    c = case(mx, [300, 130], [1, 3], seed=4, **sizes)
    c.check(c.run())


def test_growing_scores_and_values(mx):  # noqa: F811
    c = case(mx, [900, 400], [1, 2], seed=5, page=16)
    for slots in c.slots:
        for t, s in enumerate(slots):
            c.cache.k_scales[s // 16, :, s % 16] += t // 128
    out, lse = c.run(lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("window,tokens", [(0, [50, 131]), (20, [3, 137])])
def test_nan_reaches_the_rows_that_see_it(mx, window, tokens):  # noqa: F811
    c = case(mx, [156, 20], [120, 20], seed=6, page=16)
    nan_rows(c, "k", 0, tokens, 3)
    out, lse = c.run(window=window, lse=True)
    c.check(out, None, window=window)
    pos = torch.arange(36, 156, device=dev())
    want = torch.zeros(120, dtype=torch.bool, device=dev())
    for t in tokens:
        want |= (pos >= t) & ((pos < t + window) if window else True)
    assert want.any() and not want.all()
    assert torch.equal(torch.isnan(out[:120]).all(2).all(1), want) and torch.equal(torch.isnan(lse[:120]).all(1), want)
    assert not torch.isnan(out[:120][~want]).any() and not torch.isnan(out[120:140]).any()


def test_nan_and_infinite_queries_stay_in_their_rows(mx):  # noqa: F811
    c = case(mx, [200], [5], seed=7)
    clean = c.run()
    c.q[0, 1, 7] = float("nan")
    c.q[4, 3, 9] = float("inf")
    out = c.run()
    bad = torch.zeros(len(c.q), 16, dtype=torch.bool, device=dev())
    bad[0, 1] = bad[4, 3] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def test_wrong_pages_are_reported(mx):  # noqa: F811
    c = case(mx, [170, 140], [2, 1], page=16, seed=8)
    mx.mx_device_status(c.h)
    want = c.run()
    assert mx.mx_device_status(c.h) == mx.MX_OK
    table = c.table.clone()
    table[1, 1] = c.cache.pages
    got = mx.mx_attend(c.h, c.q, c.cache, table, c.len_t, q_offsets=c.off_t)
    assert mx.mx_device_status(c.h) == mx.MX_ERR_INVALID_ARG
    assert torch.equal(got[:2], want[:2]) and torch.isfinite(got).all()


def test_same_bits_in_graphs_and_on_streams(mx):  # noqa: F811
    for lengths, counts in (([700, 1300, 64], [1, 1, 1]), ([2000, 900], [40, 3])):
        c = case(mx, lengths, counts, seed=9)
        want = c.run()
        assert all(torch.equal(c.run(), want) for _ in range(5))
        torch.cuda.synchronize()
        got, other = c.run(stream=torch.cuda.Stream()), c.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = c.run()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want) and torch.equal(out, want)
