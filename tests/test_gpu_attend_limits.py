"""mx_attend where numbers get large: scores, windows, sequences, pools. Each of its kernels: few rows, many, latents."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, handle
from test_gpu_attend import Case
from test_gpu_attend_latent import case as latent_case
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = ["few 64", "few 128", "few 512", "few shared", "many 128", "many 256", "latents"]


def make(mx, kind, lengths, counts, **kw):  # noqa: F811
    """counts: query tokens where rows are few; a hundred times as many where they are not."""
    shape = {"few 64": (4, 1, 64, False), "few 128": (4, 2, 128, False), "few 512": (8, 1, 512, False), "few shared": (16, 1, 512, True),
             "many 128": (4, 1, 128, False), "many 256": (2, 1, 256, True)}
    if kind == "latents":
        return latent_case(mx, lengths, [10 * n for n in counts], **kw)
    return Case(mx, lengths, counts if kind[0] == "f" else [40 * n for n in counts], *shape[kind], **kw)


@pytest.mark.parametrize("kind", KINDS)
def test_scores_of_any_size(mx, kind):  # noqa: F811
    """Scores of 2^40 in steps of 2^18: a weight is 1 or 0, and the largest score's own is 1, whatever its values' scale."""
    c = make(mx, kind, [300], [3], seed=12, q_size=2.0**20, k_size=2.0**20)
    out = c.run(causal=False)
    q = c.q.double().cpu().numpy()
    seen = 0
    for j in range(c.heads * c.group):
        k = c.rows("k", 0)[:, j // c.group]
        v = k if c.cache.v is None else c.rows("v", 0)[:, j // c.group]
        n = c.counts[0]
        x = q[:n, j] @ k.T
        top = np.sort(x, 1)
        # twice what float32 sums of d products may be off by
        sure = top[:, -1] - top[:, -2] > 4 * (c.d + 8) * 2.0**-23 * (abs(q[:n, j]) @ abs(k).T).max(1)
        seen += sure.sum()
        want = torch.from_numpy(v[x.argmax(1)]).bfloat16()
        assert torch.equal(out[:n, j].cpu()[torch.from_numpy(sure)], want[torch.from_numpy(sure)])
    assert seen > 0.8 * c.counts[0] * c.heads * c.group


@pytest.mark.parametrize("kind", KINDS)
def test_scores_that_are_all_the_same(mx, kind):  # noqa: F811
    c = make(mx, kind, [300, 20], [2, 1], seed=13)
    out, lse = c.run(scale=0.0, lse=True)
    c.check(out, lse, scale=0.0)


@pytest.mark.parametrize("kind", KINDS)
def test_windows_longer_than_anything(mx, kind):  # noqa: F811
    c = make(mx, kind, [300, 20], [2, 3], seed=14)
    out, lse = c.run(window=2**31 - 1, lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("kind,b", [("few 64", 700), ("few shared", 300), ("many 128", 300), ("latents", 430)])
def test_many_sequences(mx, kind, b):  # noqa: F811
    """More than a CTA has threads: some without queries, some without tokens."""
    rng = np.random.default_rng(15)
    lengths = rng.integers(0, 40, b).tolist()
    c = make(mx, kind, lengths, [int(x) for x in rng.integers(0, 3, b)] if kind[0] == "f" else [1] * b, seed=15, page=16)
    out, lse = c.run(lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("heads,d,shared,group,tokens", [(8, 128, False, 2, 3), (8, 128, False, 2, 90), (1, 512, True, 16, 2),
                                                         (1, 512, True, 16, 90)])
def test_pools_beyond_32_bits(mx, heads, d, shared, group, tokens):  # noqa: F811
    """The same rows in pages of a small cache, and in the first and the last of one of 8 GiB of codes, give the same bits."""
    h, page, n = handle(), 256, 500
    g = torch.Generator(device=dev()).manual_seed(16)
    k, v, q = (torch.randn(s, generator=g, device=dev()).bfloat16() for s in ((n, heads, d), (n, heads, d), (tokens, heads * group, d)))
    outs = []
    cols = 3 * 160 * 64 * 128 // (tokens * group * page) + 2  # room enough for the latents' kernel
    for pages, first, second in ((3, 2, 1), (2**33 // (heads * page * d // 2) + 3, 0, -1)):
        second %= pages
        c = mx.MxCache.zeros(h, pages, page, heads, d, shared)
        at = torch.arange(n, device=dev())
        slots = torch.where(at < page, first * page + at, second * page + at - page)
        mx.mx_cache_write(h, c, slots, k, None if shared else v)
        table = torch.full((1, cols), -1, dtype=torch.int32, device=dev())
        table[0, 0], table[0, 1] = first, second
        outs.append(mx.mx_attend(h, q, c, table, torch.tensor([n], dtype=torch.int32, device=dev())))
        del c
        torch.cuda.empty_cache()
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
