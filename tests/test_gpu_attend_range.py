"""mx_attend: which blocks count as zeros beside larger ones. Few rows: those below 2^-27 of their token's largest. Many rows
and latents: of the largest of the 128 tokens that are taken together, whether a row
sees them or not."""
import pytest
import torch

from test_gpu_attend import Case
from test_gpu_attend_latent import case as latent_case
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu
FEW = [(4, 2, 128, False), (2, 2, 64, False), (8, 1, 512, True), (2, 2, 256, False)]
MANY = [("many", 4, 1, 128, False), ("many", 8, 1, 64, True), ("many", 2, 1, 256, False), ("latents", 16, 1, 512, True)]


def even(c):
    """All blocks of the cache get one scale."""
    for t in (c.cache.k_scales, c.cache.v_scales):
        if t is not None:
            t.fill_(120)


def raise_scale(c, side, token, by, block=slice(None)):
    s = int(c.slots[0][token])
    getattr(c.cache, side + "_scales")[s // c.page, :, s % c.page, block] = 120 + by


def zero(c, side, change):
    """What the oracle takes for this side's rows of sequence 0."""
    rows = c.rows

    def changed(name, b):
        x = rows(name, b)
        if b == 0 and name == side:
            change(x)
        return x
    c.rows = changed


@pytest.mark.parametrize("group,heads,d,shared", FEW)
def test_few_rows_blocks_of_a_token(mx, group, heads, d, shared):  # noqa: F811
    """Scores stay small: raised keys are those of the first dimensions of 32, where queries are."""
    for side in ("k",) if shared else ("k", "v"):
        for by in (27, 28):
            c = Case(mx, [200], [2], group, heads, d, shared, seed=1)
            even(c)
            c.q[..., 32:64] *= 2.0**-27
            raise_scale(c, side, 150, by, 1)
            if by > 27:
                def change(x):
                    x[150, :, :32] = x[150, :, 64:] = 0
                zero(c, side, change)
            out, lse = c.run(lse=True)
            c.check(out, lse)


@pytest.mark.parametrize("group,heads,d,shared", FEW)
def test_few_rows_other_tokens_change_nothing(mx, group, heads, d, shared):  # noqa: F811
    c = Case(mx, [200], [2], group, heads, d, shared, seed=2)
    even(c)
    want = c.run()
    raise_scale(c, "k" if shared else "v", 199, 80)  # the last query sees it
    out = c.run()
    assert torch.equal(out[0], want[0])


@pytest.mark.parametrize("kind,group,heads,d,shared", MANY)
def test_many_rows_tokens_taken_together(mx, kind, group, heads, d, shared):  # noqa: F811
    """One token is larger, of the second 128. Queries are 60 to 199: some see none of these, some not this one. (Latents: a
    block is four queries, and has no tokens behind its last one's.)"""
    token = 131 if kind == "latents" else 190
    for side in ("k",) if shared else ("k", "v"):
        for by in (27, 28):
            c = latent_case(mx, [200], [140], seed=3) if kind == "latents" else Case(mx, [200], [140], group, heads, d, shared, seed=3)
            even(c)
            if side == "k":
                c.q[token - 60:140] = 0  # rows that see it: its score is not to be all that counts
            raise_scale(c, side, token, by)
            if by > 27:
                def change(x):
                    x[128:token] = x[token + 1:] = 0
                zero(c, side, change)
            out, lse = c.run(lse=True)
            c.check(out, lse)
