"""The longest page tables, without a GPU: positions stay within 31 bits after
rounding up to the kernels' units."""
import pytest
import torch

import weight_only_int4_pack_b200 as w4
from tests.test_kv_args import attn_call, batch, cache, rows_call
from weight_only_int4_pack_b200 import build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake addresses: only where nothing can be launched")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return w4.load()


@pytest.mark.parametrize("page,width,ok", [
    (16, (1 << 27) - 16, True), (16, (1 << 27) - 15, False), (16, (1 << 27) - 1, False),
    (48, ((1 << 31) - 256) // 48, True), (48, ((1 << 31) - 256) // 48 + 1, False),
    (65536, 32767, True), (65536, 32768, False)])
def test_table_width(lib, page, width, ok):
    c, b = cache(page_size=page), batch(table_width=width, table_stride=width)
    for status in (rows_call(lib, "w4kv_append", c=c, b=b), rows_call(lib, "w4kv_read", c=c, b=b),
                   attn_call(lib, c=c, b=b)):
        if ok:  # past the checks: no device to run on
            assert status == w4.W4_ERR_CUDA
        else:
            assert status == w4.W4_ERR_INVALID_ARG
            assert b"table_width" in lib.w4_last_error()


@pytest.mark.parametrize("kw", [dict(rows=1, krs=1, vrs=3), dict(rows=1, krs=-5, vrs=1 << 40)])
def test_stride_of_a_single_row(lib, kw):
    """A dimension of size one has any stride (torch gives such views)."""
    for name in ("w4kv_append", "w4kv_read"):
        assert rows_call(lib, name, **kw) == w4.W4_ERR_CUDA  # past the checks
    assert attn_call(lib, rows=1, qrs=kw["krs"], ors=kw["vrs"]) == w4.W4_ERR_CUDA


def test_stride_of_a_single_head(lib):
    c = cache(kv_heads=1)
    for name in ("w4kv_append", "w4kv_read"):
        assert rows_call(lib, name, c=c, krs=128, khs=1, vrs=128, vhs=-1) == w4.W4_ERR_CUDA
    assert attn_call(lib, c=c, heads=1, qrs=128, qhs=1, ors=128, ohs=2) == w4.W4_ERR_CUDA


@pytest.mark.parametrize("scale,ok", [(3e38, False), (-3e38, False), (2.3e38, True), (float("nan"), False), (0.0, True)])
def test_scale_in_base_two(lib, scale, ok):
    """A finite scale whose product with log2(e) is not would answer NaN."""
    assert attn_call(lib, scale=scale) == (w4.W4_ERR_CUDA if ok else w4.W4_ERR_INVALID_ARG)
