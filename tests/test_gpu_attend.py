"""mx_attend against the definition in 64 bits, on the cache's decoded rows."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, handle
from oracle import attention as oa
from oracle import experts as oe
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu


class Case:
    """Sequences of the given cached lengths and query tokens, in a cache whose pages lie anywhere."""

    def __init__(self, mx, lengths, counts, group, heads, d, shared, page=64, dtype=torch.bfloat16, seed=0,  # noqa: F811
                 q_size=1.0, k_size=1.0, v_size=1.0, fill=0xFF):
        self.mx, self.h = mx, handle()
        self.lengths, self.counts, self.group, self.heads, self.d, self.page = lengths, counts, group, heads, d, page
        rng = np.random.default_rng(seed)
        held = [(n + page - 1) // page for n in lengths]
        pages, cols = sum(held) + 2, max(max(held), 1) + 1
        order = rng.permutation(pages)
        # what no row may see is NaN: slots without a token, pages without a sequence
        c = mx.MxCache.zeros(self.h, pages, page, heads, d, shared)
        for t in (c.k, c.k_scales, c.v, c.v_scales):
            if t is not None:
                t.fill_(fill)
        table = np.full((len(lengths), cols), -1, np.int32)
        g = torch.Generator(device=dev()).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
        at, slots = 0, []
        for b, n in enumerate(lengths):
            table[b, :held[b]] = order[at:at + held[b]]
            t = np.arange(n)
            slots.append(table[b].astype(np.int64)[t // page] * page + t % page)
            at += held[b]
        self.slots = slots
        every = torch.from_numpy(np.concatenate(slots)).to(dev())
        if len(every):
            rows = lambda size: (normal(len(every), heads, d) * size * torch.exp(0.7 * normal(len(every), heads, 1))).bfloat16()  # noqa: E731
            mx.mx_cache_write(self.h, c, every, rows(k_size), None if shared else rows(v_size))
        self.cache, self.table = c, torch.from_numpy(table).to(dev())
        self.len_t = torch.tensor(lengths, dtype=torch.int32, device=dev())
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.off_t = torch.from_numpy(self.offsets).to(dev())
        self.q = (normal(int(self.offsets[-1]), heads * group, d) * q_size).to(dtype)

    def run(self, **kw):
        kw.setdefault("q_offsets", self.off_t)
        return self.mx.mx_attend(self.h, self.q, self.cache, self.table, self.len_t, **kw)

    def rows(self, name, b):
        pool, scales = getattr(self.cache, name), getattr(self.cache, name + "_scales")
        page = self.page
        p, s = (np.stack([x.cpu().numpy()[i // page, :, i % page] for i in self.slots[b]]) for x in (pool, scales))
        return oe.decode_fp4(p, s)  # [n, heads, d]

    def check(self, got, lse=None, scale=None, causal=True, window=0):
        scale = self.d ** -0.5 if scale is None else scale
        half = torch.finfo(self.q.dtype).eps / 2
        q = self.q.double().cpu().numpy()
        got = got.double().cpu().numpy()
        for b, n in enumerate(self.lengths):
            rows = slice(self.offsets[b], self.offsets[b + 1])
            if self.counts[b] == 0:
                continue
            if n:
                k = self.rows("k", b)
                v = k if self.cache.v is None else self.rows("v", b)
            else:
                k = v = np.zeros((0, self.heads, self.d))
            pos = n - self.counts[b] + np.arange(self.counts[b])
            for j in range(self.heads * self.group):
                want, wl, size, reach = oa.attend(q[rows, j], k[:, j // self.group], v[:, j // self.group], scale, pos,
                                                  causal, window)
                # a score: float32 sums of d products and a few roundings more; its error e is the weight's
                # relative one, twice (the weight, and the sum of all). exp2 2^-21, the weight to 11 bits 2^-11;
                # weights below 2^-22 of the largest contribution lose more, 2^-33 of it each. The output's half step is
                # relative above the type's smallest normal number, and that of this number below it: 2^-25 in
                # fp16 (a value of 1.44e-7, of a token whose weight is 2^-24, comes as 2^-23)
                e = (self.d + 8) * 2.0**-23 * reach[:, None]
                tol = half * np.maximum(np.abs(want), torch.finfo(self.q.dtype).tiny) + size * (2.0**-11 + 2 * e + 2.0**-20) * (1 + half) + n * 2.0**-33 * np.nan_to_num(size).max(initial=0)
                err = np.abs(got[rows, j] - want)
                assert np.array_equal(np.isnan(want), np.isnan(got[rows, j]))
                assert (err <= tol)[~np.isnan(want)].all(), (b, j, float((err / np.maximum(tol, 1e-300)).max()))
                if lse is not None:
                    l = lse[rows, j].double().cpu().numpy()
                    seen = np.isfinite(wl)
                    assert (l[~seen] == -np.inf).all()
                    assert (np.abs(l[seen] - wl[seen]) <= e[seen, 0] + 2.0**-20 + 2.0**-22 * np.abs(wl[seen])).all()
        assert self.mx.mx_device_status(self.h) == self.mx.MX_OK


SHAPES = [(16, 1, 512, True), (16, 1, 512, False), (4, 2, 128, False), (1, 3, 64, False), (8, 2, 256, False),
          (5, 1, 64, True), (16, 1, 256, True), (7, 1, 128, True)]


@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_single_tokens(mx, group, heads, d, shared):  # noqa: F811
    lengths = [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300, 513]
    c = Case(mx, lengths, [1] * len(lengths), group, heads, d, shared)
    out, lse = c.run(lse=True, q_offsets=None)
    c.check(out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_ragged_queries(mx, group, heads, d, shared, page, dtype):  # noqa: F811
    """Several query tokens: the causal mask within a tile, sequences without queries, without tokens, and with
    more queries than tokens."""
    c = Case(mx, [40, 7, 0, 130, 5, 200, 3], [3, 7, 2, 0, 1, 37, 6], group, heads, d, shared, page, dtype, seed=1)
    out, lse = c.run(lse=True)
    c.check(out, lse)
    if group <= 8:
        out = c.run(causal=False, scale=0.2)
        c.check(out, causal=False, scale=0.2)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1000])
@pytest.mark.parametrize("group,heads,d,shared", [(16, 1, 512, True), (4, 2, 128, False), (8, 1, 64, True)])
def test_windows(mx, group, heads, d, shared, window):  # noqa: F811
    c = Case(mx, [300, 64, 65, 9, 0], [1, 1, 20, 9, 1], group, heads, d, shared, 32, seed=2)
    out, lse = c.run(lse=True, window=window)
    c.check(out, lse, window=window)


@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_long_contexts(mx, group, heads, d, shared):  # noqa: F811
    """One sequence over every CTA: its sums are joined."""
    c = Case(mx, [9001], [1], group, heads, d, shared, seed=3)
    out, lse = c.run(lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("sizes", [dict(q_size=2.0**-60), dict(q_size=30.0), dict(k_size=2.0**60, q_size=2.0**-60),
                                   dict(v_size=2.0**60), dict(v_size=2.0**-100), dict(k_size=2.0**-40, q_size=2.0**40)])
@pytest.mark.parametrize("group,heads,d", [(4, 2, 128), (16, 1, 512)])
def test_sizes_of_values(mx, group, heads, d, sizes):  # noqa: F811
    c = Case(mx, [200, 40], [1, 3], group, heads, d, False, seed=4, **sizes)
    c.check(c.run())


def nan_rows(c, side, b, tokens, block):
    """One 32-block of the given tokens becomes NaN, as the writer holds it."""
    codes, scales = getattr(c.cache, side), getattr(c.cache, side + "_scales")
    for t in tokens:
        s = int(c.slots[b][t])
        scales[s // c.page, :, s % c.page, block] = 0xFF
        codes[s // c.page, :, s % c.page, 16 * block:16 * block + 16] = 0


@pytest.mark.parametrize("group,heads,d,shared", [(4, 2, 128, False), (4, 1, 128, True), (8, 1, 512, True), (8, 1, 512, False),
                                                  (2, 2, 64, False)])
def test_nan_reaches_the_rows_that_see_it(mx, group, heads, d, shared):  # noqa: F811
    """Token 50 is seen by the last queries only, 3 by the earliest of a window."""
    for side in ("k",) if shared else ("k", "v"):
        for window, tokens in ((0, [50]), (20, [3, 37])):
            c = Case(mx, [56, 20], [20, 20], group, heads, d, shared, 16, seed=5)
            nan_rows(c, side, 0, tokens, 1)
            out, lse = c.run(window=window, lse=True)
            c.check(out, None, window=window)
            nan = torch.isnan(out[:20]).any(2).any(1)
            pos = torch.arange(36, 56, device=dev())
            want = torch.zeros_like(nan)
            for t in tokens:
                want |= (pos >= t) & ((pos < t + window) if window else True)
            assert torch.equal(nan, want) and not torch.isnan(out[20:]).any()
            if side == "k":
                assert torch.equal(torch.isnan(lse[:20]).all(1), want)


def test_nan_and_infinite_queries_stay_in_their_rows(mx):  # noqa: F811
    for group, heads, d, shared in [(4, 2, 128, False), (16, 1, 512, True)]:
        c = Case(mx, [100], [2], group, heads, d, shared, seed=6)
        clean = c.run()
        c.q[0, 1, 7] = float("nan")
        c.q[1, 3, 9] = float("inf")
        out = c.run()
        bad = torch.zeros(2, heads * group, dtype=torch.bool, device=dev())
        bad[0, 1] = bad[1, 3] = True
        assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def test_strides_and_untouched_rows(mx):  # noqa: F811
    """Queries within wider rows, heads first, an output with room around; rows that no sequence has stay."""
    c = Case(mx, [77, 130], [2, 3], 4, 2, 128, False, seed=7)
    want = c.run()
    wide = torch.zeros(9, 12, 128, dtype=torch.bfloat16, device=dev())
    wide[:5, 2:10] = c.q
    q = wide[:, 2:10]
    room = torch.full((9, 11, 136), 3.0, dtype=torch.bfloat16, device=dev())
    out = room[:, 3:, :128]
    got = mx.mx_attend(c.h, q, c.cache, c.table, c.len_t, q_offsets=c.off_t, out=out)
    assert got is out and torch.equal(out[:5], want)
    assert (room[5:] == 3).all() and (room[:, :3] == 3).all() and (room[..., 128:] == 3).all()
    first = torch.empty(8, 5, 128, dtype=torch.bfloat16, device=dev()).transpose(0, 1)
    heads_first = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(mx.mx_attend(c.h, heads_first, c.cache, c.table, c.len_t, q_offsets=c.off_t, out=first), want)
    # a table within a wider one
    table = torch.full((2, 9), 10**9, dtype=torch.int32, device=dev())
    table[:, 3:3 + c.table.shape[1]] = c.table
    assert torch.equal(mx.mx_attend(c.h, c.q, c.cache, table[:, 3:3 + c.table.shape[1]], c.len_t, q_offsets=c.off_t), want)


def test_wrong_pages_lengths_and_offsets_are_reported(mx):  # noqa: F811
    h = handle()
    mx.mx_device_status(h)
    c = Case(mx, [70, 40, 20], [1, 1, 1], 4, 2, 128, False, page=16, seed=8)
    want = c.run()
    assert mx.mx_device_status(h) == mx.MX_OK
    table = c.table.clone()
    table[1, 1] = c.cache.pages  # tokens 16 .. 31 of sequence 1 are gone
    got = mx.mx_attend(h, c.q, c.cache, table, c.len_t, q_offsets=c.off_t)
    assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and torch.isfinite(got).all() and not torch.equal(got[1], want[1])
    table[1, 1] = -5
    mx.mx_attend(h, c.q, c.cache, table, c.len_t, q_offsets=c.off_t)
    assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG
    for bad in (-1, c.table.shape[1] * 16 + 1):
        lengths = c.len_t.clone()
        lengths[2] = bad
        full = c.table.clone()
        full[2] = c.table[0, 0]
        got = mx.mx_attend(h, c.q, c.cache, full, lengths, q_offsets=c.off_t)
        assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG
        assert torch.equal(got[:2], want[:2]) and torch.isfinite(got).all()
        assert bad > 0 or (got[2] == 0).all()
    for offsets in ([0, 1, 2, 4], [0, 2, 1, 3], [-1, 1, 2, 3]):
        off = torch.tensor(offsets, dtype=torch.int32, device=dev())
        mx.mx_attend(h, c.q, c.cache, c.table, c.len_t, q_offsets=off)
        assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG


def test_same_bits_in_a_graph_and_on_another_stream(mx):  # noqa: F811
    for group, heads, d, shared in [(4, 2, 128, False), (16, 1, 512, True)]:
        c = Case(mx, [700, 1300, 64], [1, 2, 1], group, heads, d, shared, seed=9)
        want = c.run()
        assert all(torch.equal(c.run(), want) for _ in range(5))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = c.run(stream=side)
        other = c.run()  # at the same time: each call has its own workspace
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want)
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = c.run()
            graphs.append((graph, out))
        for graph, out in graphs:
            out.zero_()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for stream, (graph, _) in zip((a, b), graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs)
        # the same graph after the sequences have grown
        c.len_t -= 30
        graph, out = graphs[0]
        graph.replay()
        torch.cuda.synchronize()
        c.lengths = [n - 30 for n in c.lengths]
        c.slots = [s[:n] for s, n in zip(c.slots, c.lengths)]
        c.check(out)


def test_a_workspace_given(mx):  # noqa: F811
    c = Case(mx, [3000], [1], 16, 1, 512, True, seed=10)
    need = mx.mx_attend_bytes(c.h, 512, True)
    room = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=dev())
    assert torch.equal(c.run(workspace=room[:need]), c.run())
    assert (room[need:] == 0x5A).all()
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=room[:need - 16])


@pytest.mark.parametrize("kw", [dict(window=-1), dict(window=5, causal=False), dict(scale=float("nan")),
                                dict(scale=3e38)])
def test_calls_that_are_refused(mx, kw):  # noqa: F811
    c = Case(mx, [30], [1], 4, 2, 128, False)
    with pytest.raises(mx.MxError) as e:
        c.run(**kw)
    assert e.value.code == mx.MX_ERR_INVALID_ARG


def test_head_dimensions_that_are_not_taken(mx):  # noqa: F811
    h = handle()
    cache = mx.MxCache.zeros(h, 2, 16, 1, 96)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev())  # noqa: E731
    with pytest.raises(mx.MxError) as e:
        mx.mx_attend(h, torch.zeros(1, 2, 96, dtype=torch.bfloat16, device=dev()), cache, i(0).view(1, 1), i(5))
    assert e.value.code == mx.MX_ERR_UNSUPPORTED
