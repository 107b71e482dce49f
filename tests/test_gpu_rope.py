"""mx_rope_table against the definition in 64 bits, mx_rope bit for bit against float32 steps."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, handle
from oracle import attention as oa
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("max_pos,d,kw", [
    (1, 2, {}), (3, 64, {}), (1000, 26, dict(magnitude=1.1)), (70, 512, dict(base=500000.0)), (513, 130, {}),
    (4097, 64, dict(scaling="linear", factor=8.0)),
    (200003, 64, dict(scaling="yarn", factor=40.0, original=4096, magnitude=1.37)),
    (9001, 96, dict(scaling="yarn", factor=4.0, original=2048, base=500000.0, beta_fast=16.0, beta_slow=2.0)),
])
def test_table(mx, max_pos, d, kw):  # noqa: F811
    h = handle()
    got = mx.mx_rope_table(h, max_pos, d, **kw).cpu().numpy()
    # the polynomials (2^-28) and the angle's rounding to 24 bits (at most pi / 4 2^-24), two more roundings of the
    # result (2^-24 each, times the magnitude), the 64-bit angle of a far position (2e5 2^-53): below 2^-22
    assert np.abs(got - oa.rope_table(max_pos, d, **kw)).max() <= 2.0**-22 * kw.get("magnitude", 1.0)
    out = torch.full((max_pos + 1, d), 7.0, device=dev())
    mx.mx_rope_table(h, max_pos, d, out=out[:max_pos], **kw)
    assert np.array_equal(out[:max_pos].cpu().numpy(), got) and (out[max_pos] == 7).all()


def rows(seed, t, heads, d, dtype):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randn(t, heads, d, generator=g, device=dev()).to(dtype)


def steps(x, cs, first, interleaved, inverse):
    """The oracle's rotation in float32, rounded to x's type."""
    y = oa.rope(x.float().cpu().numpy(), cs.cpu().numpy(), first, interleaved, inverse)
    return torch.from_numpy(y).to(x.dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,heads,d,d_rope,first", [
    (1, 16, 512, 64, 448), (5, 3, 96, 64, 0), (37, 7, 128, 128, 0), (9, 2, 40, 12, 20), (3, 1, 10, 6, 2), (2, 5, 2, 2, 0),
    (129, 33, 192, 64, 128), (700, 32, 512, 64, 448), (1100, 16, 128, 128, 0)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation(mx, t, heads, d, d_rope, first, interleaved, dtype):  # noqa: F811
    h, x = handle(), rows(t + d, t, heads, d, dtype)
    cs = mx.mx_rope_table(h, 300, d_rope)
    pos = torch.randint(0, 300, (t,), device=dev())
    for inverse in (False, True):
        want = steps(x, cs[pos], first, interleaved, inverse)
        got = mx.mx_rope(h, x, pos, cs, first=first, interleaved=interleaved, inverse=inverse)
        assert torch.equal(got.cpu(), want)
        y = x.clone()
        assert mx.mx_rope(h, y, pos, cs, first=first, interleaved=interleaved, inverse=inverse, out=y) is y
        assert torch.equal(y.cpu(), want)
    assert mx.mx_device_status(h) == mx.MX_OK


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("layout", ["part of wider rows", "heads first", "odd strides", "one element off"])
def test_strides(mx, layout, interleaved):  # noqa: F811
    h, t, heads, d, n = handle(), 11, 4, 48, 32
    cs, pos = mx.mx_rope_table(h, 50, n), torch.arange(t, device=dev())
    def view():
        if layout == "part of wider rows":
            return rows(1, t, heads + 3, d, torch.bfloat16)[:, 2:2 + heads]
        if layout == "heads first":
            return rows(1, heads, t, d, torch.bfloat16).transpose(0, 1)
        if layout == "odd strides":
            return rows(1, t, heads, d + 2, torch.bfloat16)[..., :d]
        return rows(1, t, heads, d + 8, torch.bfloat16)[..., 2:2 + d]
    x, out = view(), view()
    whole = out._base if out._base is not None else out
    before = whole.clone()
    want = steps(x.contiguous(), cs[pos], 16, interleaved, False)
    assert mx.mx_rope(h, x, pos, cs, first=16, interleaved=interleaved, out=out) is out
    assert torch.equal(out.cpu(), want)
    out.copy_(x)
    assert torch.equal(whole, before)  # nothing beside the heads was written


def test_odd_places(mx):  # noqa: F811
    """Halves may begin anywhere, pairs of neighbours at even places."""
    h, t = handle(), 6
    cs, pos = mx.mx_rope_table(h, 50, 10), torch.arange(t, device=dev())
    x = rows(4, t, 3, 27, torch.bfloat16)
    got = mx.mx_rope(h, x, pos, cs, first=7, interleaved=False)
    assert torch.equal(got.cpu(), steps(x, cs[pos], 7, False, False))
    with pytest.raises(mx.MxError) as e:
        mx.mx_rope(h, x, pos, cs, first=7, interleaved=True)
    assert e.value.code == mx.MX_ERR_UNSUPPORTED


def test_inverse_is_the_gradient(mx):  # noqa: F811
    h, t, d, n = handle(), 5, 24, 16
    cs, pos = mx.mx_rope_table(h, 50, n, magnitude=1.25), torch.arange(7, 7 + t, device=dev())
    x, w = rows(2, t, 2, d, torch.float32), rows(3, t, 2, d, torch.float32)
    for interleaved in (True, False):
        f = lambda y: (mx.mx_rope(h, y, pos, cs, interleaved=interleaved).double() * w.double()).sum().item()  # noqa: E731,B023
        grad = mx.mx_rope(h, w, pos, cs, interleaved=interleaved, inverse=True)
        for at in [(0, 0, 0), (1, 1, 8), (2, 0, 9), (4, 1, 23), (3, 0, 16)]:
            up, dn = x.clone(), x.clone()
            up[at] += 0.5
            dn[at] -= 0.5
            # linear: the difference is the gradient but for roundings of 2^-24 of a few values of size 4
            assert abs(f(up) - f(dn) - grad[at].item()) < 1e-5


def test_positions_outside_the_table(mx):  # noqa: F811
    h, x = handle(), rows(2, 4, 3, 64, torch.bfloat16)
    cs = mx.mx_rope_table(h, 20, 64)
    mx.mx_device_status(h)
    got = mx.mx_rope(h, x, torch.tensor([3, 20, -1, 19], device=dev()), cs)
    assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG
    assert torch.equal(got.cpu(), steps(x, cs[[3, 0, 0, 19]], 0, True, False))
    assert mx.mx_device_status(h) == mx.MX_OK


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=float("nan")), dict(scaling="linear", factor=0.5),
                                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original=9, beta_fast=0.5),
                                dict(scaling="yarn", factor=2.0, original=9, beta_slow=0.0), dict(magnitude=float("inf")),
                                dict(d_rope=514), dict(d_rope=7)])
def test_tables_that_are_refused(mx, kw):  # noqa: F811
    with pytest.raises(mx.MxError):
        mx.mx_rope_table(handle(), 9, **{**dict(d_rope=8), **kw})
