"""mx_attend where one call has prompts and single tokens: each kernel takes the other's kind of rows. And negative scales."""
import pytest
import torch

from test_gpu_attend import SHAPES, Case
from test_gpu_attend_latent import case as latent_case
from test_gpu_attend_rows import SHAPES as ROWS_SHAPES
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu


def mixed(total, singles):
    """Single tokens around one prompt."""
    lengths = [1 + 37 * i % 400 for i in range(singles)]
    at = singles // 2
    return lengths[:at] + [total + 70] + lengths[at:], [1] * at + [total] + [1] * (singles - at)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_a_prompt_among_single_tokens(mx, group, heads, d, shared, window):  # noqa: F811
    """Few rows on average: the prompt goes along, 8 or 16 rows at a time."""
    singles = 21
    total = min(150, 39 * (singles + 1) // group - singles)  # less than 40 rows to each
    assert (total + singles) * group < 40 * (singles + 1)
    c = Case(mx, *mixed(total, singles), group, heads, d, shared, 32, seed=1)
    out, lse = c.run(lse=True, window=window)
    c.check(out, lse, window=window)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("group,heads,d,shared", ROWS_SHAPES)
def test_single_tokens_beside_a_prompt(mx, group, heads, d, shared, window):  # noqa: F811
    """Many rows on average: a single token has a block of rows to itself."""
    c = Case(mx, *mixed(9 * 64 // group + 64, 7), group, heads, d, shared, 32, seed=2)
    out, lse = c.run(lse=True, window=window)
    c.check(out, lse, window=window)


@pytest.mark.parametrize("window", [0, 50])
def test_single_tokens_beside_a_prompt_of_latents(mx, window):  # noqa: F811
    c = latent_case(mx, *mixed(120, 7), seed=3)
    out, lse = c.run(lse=True, window=window)
    c.check(out, lse, window=window)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("group,heads,d,shared", SHAPES)
def test_negative_scales_of_few_rows(mx, group, heads, d, shared, causal):  # noqa: F811
    c = Case(mx, [300, 17, 129], [1, 3, 2], group, heads, d, shared, seed=4)
    out, lse = c.run(lse=True, scale=-0.1, causal=causal)
    c.check(out, lse, scale=-0.1, causal=causal)


@pytest.mark.parametrize("group,heads,d,shared", ROWS_SHAPES)
def test_many_tiles_many_times(mx, group, heads, d, shared):  # noqa: F811
    """Tiles follow one another in the same stages, one of them where keys and values of 256 dimensions lie apart."""
    n = 2 * 256 // group
    c = Case(mx, [6000, 2500], [n, n], group, heads, d, shared, seed=5)
    for kw in (dict(), dict(q_offsets=None)):  # blocks, and so splits, are counted apart
        out, lse = c.run(lse=True, **kw)
        c.check(out, lse)
        for _ in range(40):
            again, sums = c.run(lse=True, **kw)
            assert torch.equal(again, out) and torch.equal(sums, lse)
