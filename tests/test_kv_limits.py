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
