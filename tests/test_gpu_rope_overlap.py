"""mx_rope into memory beside x, and its refusal of memory that overlaps x without being x."""
import pytest
import torch

from gpu_helpers import dev, handle
from test_gpu_experts import mx  # noqa: F401
from test_gpu_rope import rows, steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [True, False])
def test_memory_that_overlaps(mx, interleaved):  # noqa: F811
    """Other heads of the same rows and rows in between are taken; any element in common is not, but for all of them."""
    h, t, heads, d, n = handle(), 5, 3, 32, 16
    cs, pos = mx.mx_rope_table(h, 50, n), torch.arange(t, device=dev())
    go = lambda x, out: mx.mx_rope(h, x, pos, cs, interleaved=interleaved, out=out)  # noqa: E731
    room = rows(5, 2 * t, 8, d, torch.bfloat16)
    tail = room.view(-1)[-2 * (t * heads * d):]
    flat = lambda at: tail[at:at + t * heads * d].view(t, heads, d)  # noqa: E731
    for x, out in ((room[:t, :heads], room[:t, heads:2 * heads]), (room[::2, :heads], room[1::2, :heads]),
                   (room[:t, :heads], room[t:, :heads]), (room[:t, ::2][:, :heads], room[:t, 1::2][:, :heads]),
                   (flat(0), flat(t * heads * d))):
        x, out = x.view(x.shape), out.view(out.shape)
        x.copy_(rows(6, t, heads, d, torch.bfloat16))
        want = steps(x.contiguous(), cs[pos], d - n, interleaved, False)
        assert torch.equal(go(x, out).cpu(), want)
    for x, out in ((room[:t, :heads], room[:t, 2:2 + heads]), (room[:t, :heads], room[1:1 + t, :heads]),
                   (room[1:1 + t, 1:1 + heads], room[:t, :heads]), (flat(0), flat(2)), (flat(d * heads), flat(0)),
                   (flat(0), flat(t * heads * d - 2))):
        before = room.clone()
        with pytest.raises(mx.MxError) as e:
            go(x, out)
        assert e.value.code == mx.MX_ERR_INVALID_ARG and torch.equal(room, before)
