"""Plan queries of the products with MXFP4 weights (host only, no GPU), over rows, shapes and
both kinds of activations: what a launch reads and holds, as invariants of the plans."""
import itertools

import pytest

import mxfp8_block_scaled_06_gb300 as mx

MAX_SMEM = 232448
NS = [128, 256, 640, 1024, 2048, 2560, 4096, 5120, 8192]
KS = [128, 384, 1536, 2048, 5120, 8192, 10368, 16384]
ROWS = [1, 2, 15, 16, 17, 48, 49, 64, 65, 100, 128, 129, 200, 240, 256, 257, 300, 344, 384, 385, 500, 512, 513, 600, 640,
        641, 1000, 2048]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def plans(rows=ROWS):
    for m, n, k, fp4, pdl in itertools.product(rows, NS, KS, (False, True), (False, True)):
        yield (m, n, k, fp4, pdl), mx.mx_plan_gemm_fp4(m, n, k, fp4_activations=fp4, pdl=pdl)


def test_scale_tiles_read_are_those_of_the_rows():
    """The scales end with the last row's 128-row tile, however the rows are sliced."""
    wide = 0
    for case, p in plans():
        assert p["scale_tiles"] == (case[0] + 127) // 128, (case, p)
        wide += p["slices"] > 1 and p["rows"] == 256 and (case[0] - 1) % 256 < 128
    assert wide > 0  # slices of 256 rows of which the last has one tile only


def test_slices_take_all_rows():
    for case, p in plans():
        assert p["splits"] == 1 or p["slices"] * p["rows"] >= case[0] > (p["slices"] - 1) * p["rows"], (case, p)


def test_rejects_bad_arguments():
    for args in ((0, 256, 256), (1 << 25, 256, 256), (1, 200, 256), (1, 256, 200), (1, 0, 256)):
        with pytest.raises(mx.MxError):
            mx.mx_plan_gemm_fp4(*args)
    for kw in (dict(experts=-1), dict(experts=513), dict(sm_count=0)):
        with pytest.raises(mx.MxError):
            mx.mx_plan_gemm_fp4(1, 256, 256, **kw)


def test_every_plan_fits():
    for case, p in plans():
        assert p["smem"] <= MAX_SMEM and p["tmem_cols"] <= 512 and p["stages"] >= p["min_stages"], (case, p)


@pytest.mark.parametrize("fp4", [False, True])
def test_slices_of_128_rows_are_open_to_more_rows(fp4):
    """j slices of 128 rows cost what one costs against j times the columns (the same clusters):
    where that splits K, so does the product of 128 j rows."""
    for j, n, k in itertools.product((2, 3, 4, 5, 8), NS, KS):
        if mx.mx_plan_gemm_fp4(128, j * n, k, fp4_activations=fp4)["splits"] > 1:
            assert mx.mx_plan_gemm_fp4(128 * j, n, k, fp4_activations=fp4)["splits"] > 1, (j, n, k)


@pytest.mark.parametrize("n", [9856, 12288, 16384, 19456])
@pytest.mark.parametrize("m", [34, 48, 64])
def test_split_of_33_to_64_rows_follows_k(m, n):
    """Measured: whole K is faster up to 1024 elements (by 4 to 29 %), a split from 4096 (by 4 to 33 %)."""
    for k in (256, 512, 1024):
        assert mx.mx_plan_gemm_fp4(m, n, k)["splits"] == 1
    for k in (4096, 8192):
        assert mx.mx_plan_gemm_fp4(m, n, k)["splits"] > 1


@pytest.mark.parametrize("fp4", [False, True])
def test_whole_k_rings_are_long_enough(fp4):
    """Experts' and plain products: the ring has the stages that warps which take them in turn need (the
    stages left to others and one more: 5 of MXFP8 rows, 3 of MXFP4 where two warps load the scales),
    and what shares an SM fits its tensor memory."""
    for e, r, n, k in itertools.product((1, 2, 7, 64, 512), (1, 16, 63, 100, 700, 1024, 4099, 20818, 50000, 1 << 20),
                                        (128, 256, 640, 4096), (128, 640, 4096)):
        if e * n * k > 1 << 34:
            continue
        p = mx.mx_plan_gemm_fp4(r, n, k, experts=e, fp4_activations=fp4)
        two = p["mtile"] <= 64  # CTAs to an SM
        assert p["splits"] == 1 and p["mtile"] % 16 == 0 and p["mtile"] <= 224
        assert p["stages"] >= p["min_stages"] >= 3 and (two or fp4 or p["min_stages"] == 5), (e, r, n, k, p)
        assert p["smem"] <= (115712 if two else MAX_SMEM) and p["tmem_cols"] <= (256 if two else 512), (e, r, n, k, p)
