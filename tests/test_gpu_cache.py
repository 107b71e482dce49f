"""mx_cache_write and mx_cache_read bit for bit against the oracle's MXFP4 rows."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, handle
from oracle import experts as oe
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def normal(seed, *shape):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev())


def quantized(x):
    """(codes, scales, values) of [T, heads, d]."""
    t, heads, d = x.shape
    q, s, v = oe.quantize_fp4(x.double().cpu().numpy().reshape(t * heads, d))
    return q.reshape(t, heads, -1), s.reshape(t, heads, -1), v.reshape(t, heads, d)


def filled(mx, pages, page, heads, d, shared, fill=0xA5):  # noqa: F811
    c = mx.MxCache.zeros(handle(), pages, page, heads, d, shared)
    for t in (c.k, c.k_scales, c.v, c.v_scales):
        if t is not None:
            t.fill_(fill)
    return c


def rows_of(pool, slots):
    page = pool.shape[2]
    p = pool.cpu().numpy()
    return np.stack([p[s // page, :, s % page] for s in slots])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,heads,d,page,shared", [(1, 1, 512, 64, True), (5, 2, 128, 16, False), (70, 3, 64, 48, False),
                                                   (33, 1, 32, 16, False), (130, 8, 256, 256, True), (9, 1, 96, 32, False)])
def test_write_and_read(mx, t, heads, d, page, shared, dtype):  # noqa: F811
    h = handle()
    pages = (t + page - 1) // page + 3
    c = filled(mx, pages, page, heads, d, shared)
    before = {n: getattr(c, n).clone() for n in ("k", "k_scales")}
    slots = np.random.default_rng(t).permutation(pages * page)[:t]
    sl = torch.from_numpy(slots).to(dev())
    sides = {"k": (normal(t, t, heads, d) * 3).to(dtype)}
    if not shared:
        sides["v"] = (normal(t + 1, t, heads, d) * 0.01).to(dtype)
    values = dict(zip("kv", mx.mx_cache_write(h, c, sl, sides["k"], sides.get("v"), values=True)))
    back = {kind: dict(zip("kv", mx.mx_cache_read(h, c, sl, dtype=kind))) for kind in TYPES}
    for n, x in sides.items():
        q, s, v = quantized(x)
        assert np.array_equal(rows_of(getattr(c, n), slots), q)
        assert np.array_equal(rows_of(getattr(c, n + "_scales"), slots), s)
        assert np.array_equal(values[n].double().cpu().numpy(), v)
        for kind in TYPES:
            assert torch.equal(back[kind][n].cpu(), torch.from_numpy(v).to(kind))
    if shared:
        assert values["v"] is None and back[torch.float32]["v"] is None
    # the other slots are as they were
    keep = np.ones(pages * page, bool)
    keep[slots] = False
    for n, old in before.items():
        a, b = (p.transpose(1, 2).reshape(pages * page, -1)[torch.from_numpy(keep)] for p in (getattr(c, n).cpu(), old.cpu()))
        assert torch.equal(a, b)
    assert mx.mx_device_status(h) == mx.MX_OK


def test_many_rows(mx):  # noqa: F811
    """Enough rows that a thread takes two units, the last ones short of it."""
    h, t, heads, d, page = handle(), 8209, 8, 128, 64
    c = mx.MxCache.zeros(h, 131, page, heads, d)
    slots = torch.randperm(131 * page, device=dev())[:t]
    k, v = normal(1, t, heads, d).bfloat16(), normal(2, t, heads, d).bfloat16()
    kv, vv = mx.mx_cache_write(h, c, slots, k, v, values=True)
    for x, y, back in zip((k, v), (kv, vv), mx.mx_cache_read(h, c, slots)):
        q, s, want = mx.mx_quantize_rows_fp4(h, x.reshape(t * heads, d), swizzled=False, y=True)
        assert torch.equal(y.view(-1), want.view(-1)) and torch.equal(back.view(-1), want.view(-1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rows_that_begin_within_32_bytes(mx, dtype):  # noqa: F811
    h, t, heads, d, page = handle(), 37, 3, 96, 16
    c = mx.MxCache.zeros(h, 4, page, heads, d)
    slots = torch.randperm(4 * page, device=dev())[:t]
    k, v = (torch.empty(t * (heads * (d + 8) + 8) + 8, device=dev(), dtype=dtype)[8:].as_strided((t, heads, d), (heads * (d + 8) + 8, d + 8, 1))
            .copy_(normal(i, t, heads, d)) for i in (1, 2))
    outs = [torch.zeros(t * heads * d + 8, device=dev(), dtype=dtype)[(4 if dtype is torch.float32 else 8):][:t * heads * d].view(t, heads, d) for _ in range(2)]
    assert all(x.data_ptr() % 32 == 16 for x in outs)
    values = mx.mx_cache_write(h, c, slots, k, v, values=True)
    mx.mx_cache_read(h, c, slots, dtype=dtype, k=outs[0], v=outs[1])
    for x, y, back in zip((k, v), values, outs):
        want = mx.mx_quantize_rows_fp4(h, x.reshape(t * heads, d), swizzled=False, y=True)[2].view(t, heads, d)
        assert torch.equal(y, want) and torch.equal(back, want.to(dtype))


def test_special_blocks(mx):  # noqa: F811
    h, d = handle(), 128
    x = normal(3, 4, 1, d)
    x[0, 0, 5], x[0, 0, 40] = float("inf"), float("nan")
    x[1] = 0
    x[1, 0, 3] = -0.0
    x[2] *= 2.0**-130
    x[3] *= 2.0**100
    c = mx.MxCache.zeros(h, 1, 16, 1, d, shared=True)
    slots = torch.tensor([3, 0, 15, 7], device=dev())
    v, _ = mx.mx_cache_write(h, c, slots, x, values=True)
    q, s, want = quantized(x)
    assert np.array_equal(rows_of(c.k, slots.tolist()), q) and np.array_equal(rows_of(c.k_scales, slots.tolist()), s)
    assert np.array_equal(v.double().cpu().numpy(), want, equal_nan=True)
    back = mx.mx_cache_read(h, c, slots, dtype=torch.float32)[0]
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)
    assert torch.isnan(back[0, 0, :64]).all() and torch.signbit(back[1, 0, 3])
    # fp16: nearest, beyond its range infinite
    assert torch.equal(mx.mx_cache_read(h, c, slots, dtype=torch.float16)[0][1:].cpu(), torch.from_numpy(want[1:]).half())


def test_slots_left_out_and_out_of_range(mx):  # noqa: F811
    h, heads, d, page = handle(), 2, 64, 16
    mx.mx_device_status(h)
    c = filled(mx, 2, page, heads, d, False)
    k, v = normal(1, 5, heads, d).bfloat16(), normal(2, 5, heads, d).bfloat16()
    mx.mx_cache_write(h, c, torch.tensor([-1, 31, -(2**40), 0, -7], device=dev()), k, v)
    assert mx.mx_device_status(h) == mx.MX_OK
    q, s, _ = quantized(k)
    assert np.array_equal(rows_of(c.k, [31, 0]), q[[1, 3]])
    left = [i for i in range(32) if i not in (0, 31)]
    assert (rows_of(c.k, left) == 0xA5).all() and (rows_of(c.v_scales, left) == 0xA5).all()
    # beyond the cache: reported, the others written
    mx.mx_cache_write(h, c, torch.tensor([5, 32, 2**40, 2**32 + 3, 6], device=dev()), k, v)
    assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG
    assert np.array_equal(rows_of(c.k, [5, 6]), q[[0, 4]]) and (rows_of(c.k, [3, 4]) == 0xA5).all()
    out = torch.full((4, heads, d), 9.0, dtype=torch.bfloat16, device=dev())
    mx.mx_cache_read(h, c, torch.tensor([5, -1, 5, -3], device=dev()), k=out)
    assert mx.mx_device_status(h) == mx.MX_OK
    assert (out[[1, 3]] == 9).all() and torch.equal(out[0], out[2])  # a slot may be read twice
    mx.mx_cache_read(h, c, torch.tensor([32, 5, 2**32 + 5, 5], device=dev()), k=out.fill_(9))
    assert mx.mx_device_status(h) == mx.MX_ERR_INVALID_ARG
    assert (out[[0, 2]] == 9).all() and not (out[1] == 9).all()


def test_strided_rows_and_pages_apart(mx):  # noqa: F811
    h, t, heads, d, page = handle(), 21, 3, 64, 16
    # layers of one allocation, keys and values of a fused projection
    pools = [torch.full((4, 5, heads, page, n), 0xA5, dtype=torch.uint8, device=dev()) for n in (32, 2, 32, 2)]
    c = mx.MxCache(*(p[:, 2] for p in pools))
    wide = normal(5, t, 2 * heads + 4, d).bfloat16()
    k, v = wide[:, 4:4 + heads], wide[:, 4 + heads:]
    slots = torch.randperm(4 * page, device=dev())[:t]
    mx.mx_cache_write(h, c, slots, k, v)
    for x, back in zip((k, v), mx.mx_cache_read(h, c, slots, dtype=torch.float32)):
        assert np.array_equal(back.double().cpu().numpy(), quantized(x)[2])
    for p in pools:
        assert (p[:, [0, 1, 3, 4]] == 0xA5).all()


def test_rows_beyond_32_bits(mx):  # noqa: F811
    """A cache of more than 4 GiB of codes: byte offsets of the last pages do not fit in 32 bits."""
    h, heads, d, page = handle(), 8, 512, 256
    pages = 2**33 // (heads * page * d // 2) + 3
    c = mx.MxCache.zeros(h, pages, page, heads, d, shared=True)
    last = pages * page - 1
    slots = torch.tensor([last, 0, last // 2, last - page], device=dev())
    k = normal(8, 4, heads, d).bfloat16()
    mx.mx_cache_write(h, c, slots, k)
    assert np.array_equal(mx.mx_cache_read(h, c, slots, dtype=torch.float32)[0].double().cpu().numpy(), quantized(k)[2])
    assert int((c.k_scales.view(pages, -1) != 0).any(1).sum()) == len({s // page for s in slots.tolist()})
