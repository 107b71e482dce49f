"""The tensor checks of the rotary, cache and attention entry points, on the CPU: each case is right in
every respect but one; tensors that are right but in host memory fail the last check."""
import ctypes

import pytest
import torch

from test_experts_binding import bf16, f32, h, i32, mx, u8  # noqa: F401


def i64(*shape):
    return torch.zeros(shape, dtype=torch.int64)


def pools(d=128, heads=2, page=32, pages=5):
    return u8(pages, heads, page, d // 2), u8(pages, heads, page, d // 32)


def cache(mx, shared=False, **kw):  # noqa: F811
    return mx.MxCache(*pools(**kw), *(() if shared else pools(**kw)))


def table(mx):  # noqa: F811
    return mx.mx_rope_table, dict(max_pos=9, d_rope=64, out=f32(9, 64))


def rope(mx):  # noqa: F811
    return mx.mx_rope, dict(x=bf16(4, 3, 96), positions=i64(4), cos_sin=f32(9, 64), out=bf16(4, 3, 96))


def write(mx):  # noqa: F811
    return mx.mx_cache_write, dict(cache=cache(mx), slots=i64(4), k=bf16(4, 2, 128), v=bf16(4, 2, 128))


def read(mx):  # noqa: F811
    return mx.mx_cache_read, dict(cache=cache(mx), slots=i64(4), k=bf16(4, 2, 128), v=bf16(4, 2, 128))


def attend(mx):  # noqa: F811
    return mx.mx_attend, dict(q=bf16(6, 8, 128), cache=cache(mx), table=i32(3, 4), lengths=i32(3), q_offsets=i32(4),
                              out=bf16(6, 8, 128))


CASES = [
    (table, dict(scaling="cubic"), ValueError), (table, dict(max_pos=0), ValueError), (table, dict(d_rope=0), ValueError),
    (table, dict(out=f32(8, 64)), ValueError), (table, dict(out=bf16(9, 64)), TypeError),
    (rope, dict(x=bf16(4, 96)), ValueError), (rope, dict(x=u8(4, 3, 96)), TypeError),
    (rope, dict(x=bf16(4, 3, 192)[..., ::2]), ValueError), (rope, dict(positions=i32(4)), TypeError),
    (rope, dict(positions=i64(3)), ValueError), (rope, dict(cos_sin=f32(9, 98)), ValueError),
    (rope, dict(cos_sin=f32(9, 63)), ValueError), (rope, dict(cos_sin=f32(9, 128)[:, :64]), ValueError),
    (rope, dict(first=33), ValueError), (rope, dict(first=-2), ValueError), (rope, dict(out=f32(4, 3, 96)), TypeError),
    (rope, dict(out=bf16(4, 2, 96)), ValueError), (rope, dict(out=bf16(1, 3, 96).expand(4, 3, 96)), ValueError),
    (write, dict(k=bf16(4, 256)), ValueError), (write, dict(k=u8(4, 2, 128)), TypeError),
    (write, dict(k=bf16(4, 3, 128)), ValueError), (write, dict(k=bf16(4, 2, 132)[..., :128]), ValueError),
    (write, dict(v=None), ValueError), (write, dict(v=f32(4, 2, 128)), TypeError), (write, dict(v=bf16(3, 2, 128)), ValueError),
    (write, dict(slots=i32(4)), TypeError), (write, dict(slots=i64(3)), ValueError), (write, dict(slots=i64(8)[::2]), ValueError),
    (read, dict(slots=i64(2, 2)), ValueError), (read, dict(slots=i32(4)), TypeError), (read, dict(dtype=torch.int8), TypeError),
    (read, dict(k=bf16(4, 2, 64)), ValueError), (read, dict(v=f32(4, 2, 128)), TypeError),
    (read, dict(k=bf16(4, 128, 2)), ValueError),
    (attend, dict(q=bf16(6, 1024)), ValueError), (attend, dict(q=f32(6, 8, 128)), TypeError),
    (attend, dict(q=bf16(6, 7, 128)), ValueError), (attend, dict(q=bf16(6, 8, 64)), ValueError),
    (attend, dict(q=bf16(6, 8, 256)[..., ::2]), ValueError), (attend, dict(table=i32(12)), ValueError),
    (attend, dict(table=i64(3, 4)), TypeError), (attend, dict(table=i32(4, 3).t()), ValueError),
    (attend, dict(lengths=i32(2)), ValueError), (attend, dict(lengths=i64(3)), TypeError),
    (attend, dict(q_offsets=i32(3)), ValueError), (attend, dict(q=bf16(7, 8, 128), q_offsets=None, out=None), ValueError),
    (attend, dict(out=bf16(6, 8, 64)), ValueError), (attend, dict(out=torch.zeros(6, 8, 128).half()), TypeError),
    (attend, dict(out=bf16(1, 8, 128).expand(6, 8, 128)), ValueError),
    (attend, dict(out=bf16(6, 1, 128).expand(6, 8, 128)), ValueError),
    (attend, dict(workspace=f32(1 << 20)), TypeError), (attend, dict(window=2**32), ValueError),
    (attend, dict(window=-2**32), ValueError),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_one_wrong_argument(mx, h, i):  # noqa: F811
    make, wrong, exc = CASES[i]
    call, args = make(mx)
    with pytest.raises(exc) as e:
        call(h, **{**args, **wrong})
    assert "cuda:0" not in str(e.value)  # refused for what is wrong, before residency


@pytest.mark.parametrize("make", [table, rope, write, read, attend])
def test_host_tensors_fail_the_residency_check(mx, h, make):  # noqa: F811
    call, args = make(mx)
    with pytest.raises(ValueError, match="cuda:0"):
        call(h, **args)


def test_values_where_the_cache_has_none(mx, h):  # noqa: F811
    with pytest.raises(ValueError, match="no values"):
        mx.mx_cache_write(h, cache(mx, shared=True), i64(4), bf16(4, 2, 128), bf16(4, 2, 128))
    with pytest.raises(ValueError, match="no values"):
        mx.mx_cache_read(h, cache(mx, shared=True), i64(4), v=bf16(4, 2, 128))


@pytest.mark.parametrize("wrong", [dict(k=u8(5, 2, 32, 60)), dict(k=u8(5, 2, 24, 64)), dict(k=u8(5, 64, 64)), dict(k=None),
                                   dict(k_scales=u8(5, 2, 32, 3)), dict(v_scales=None), dict(v=u8(4, 2, 32, 64)),
                                   dict(k=u8(5, 32, 2, 64).transpose(1, 2)), dict(k=u8(1, 2, 32, 64).expand(5, 2, 32, 64)),
                                   dict(k=u8(5 * 4096 + 8)[8:].view(5, 2, 32, 64)), dict(k_scales=None)])
def test_pools_of_a_cache(mx, wrong):  # noqa: F811
    k, s = pools()
    with pytest.raises(ValueError):
        mx.MxCache(**{**dict(k=k, k_scales=s, v=k.clone(), v_scales=s.clone()), **wrong})


def test_pages_apart(mx):  # noqa: F811
    """Layers of one allocation: a page's neighbours belong to other layers."""
    k, s = u8(5, 7, 2, 32, 64), u8(5, 7, 2, 32, 4)
    c = mx.MxCache(k[:, 3], s[:, 3])
    assert c.info.k_stride == 7 * 4096 and c.info.k_scales_stride == 7 * 256


def test_null_handle(mx):  # noqa: F811
    lib, n = mx.load_library(), None
    bad, f = mx.MX_ERR_INVALID_ARG, ctypes.c_float(1)
    assert lib.mx_rope_table(n, 1, 2, 1e4, 0, 1.0, 0, 1.0, 1.0, f, n, n) == bad
    assert lib.mx_rope(n, 1, 1, 2, 0, 2, n, 2, 2, 0, n, n, 1, 1, 0, n, 2, 2, n) == bad
    assert lib.mx_cache_write(n, n, 1, n, n, 8, 8, n, 0, 0, 0, n, n, n) == bad
    assert lib.mx_cache_read(n, n, 1, n, 0, n, n, n) == bad
    assert lib.mx_attend_bytes(n, 128, 0) == 0
    assert lib.mx_attend(n, n, 1, 1, 1, n, 8, 8, 0, n, n, 1, 1, n, f, 1, 0, n, 8, 8, n, n, 0, n) == bad
