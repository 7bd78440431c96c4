"""Refusals of the key/value cache's entry points, without a GPU: the C ABI
with fake, never-dereferenced addresses (in a process that sees no GPU, so
that a regression could not launch anything on them) and the Python binding
with tensors that are not on a device."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import weight_only_int4_pack_b200 as w4
from weight_only_int4_pack_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GPU_VISIBLE = torch.cuda.is_available()


@pytest.fixture(autouse=True)
def _no_visible_gpu(request):
    if GPU_VISIBLE and request.node.name != "test_module_in_a_process_without_gpu":
        pytest.skip("fake-address checks run in a child process without a visible GPU")


@pytest.mark.skipif(not GPU_VISIBLE, reason="runs in-process here: no GPU is visible")
def test_module_in_a_process_without_gpu():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return w4.load()


def cache(**kw):
    a = dict(k_codes=0x100000, k_scales=0x200000, v_codes=0x300000, v_scales=0x400000, num_pages=10,
             page_size=16, kv_heads=2, head_dim=128, fmt=w4.W4KV_INT8)
    a.update(kw)
    return w4._CCache(*a.values())


def batch(**kw):
    a = dict(page_table=0x500000, table_stride=4, table_width=4, kv_lens=0x600000, cu_rows=0x700000,
             batch=3)
    a.update(kw)
    return w4._CBatch(*a.values())


BAD_CACHE = [(dict(fmt=3), 1), (dict(fmt=-1), 1), (dict(num_pages=0), 1), (dict(num_pages=1 << 31), 1),
             (dict(kv_heads=0), 1), (dict(page_size=0), 1), (dict(head_dim=0), 1),
             (dict(k_codes=None), 1), (dict(v_codes=None), 1), (dict(k_scales=None), 1),
             (dict(v_scales=None), 1), (dict(page_size=8), 2), (dict(page_size=24), 2),
             (dict(page_size=1 << 17), 2),
             (dict(page_size=1 << 16, kv_heads=1 << 15), 2), (dict(head_dim=96), 2), (dict(head_dim=256), 2),
             (dict(k_codes=0x100008), 2), (dict(v_scales=0x400004), 2)]
BAD_BATCH = [(dict(batch=-1), 1), (dict(batch=(1 << 20) + 1), 1), (dict(page_table=None), 1),
             (dict(kv_lens=None), 1), (dict(cu_rows=None), 1), (dict(table_width=0), 1),
             (dict(table_width=1 << 28), 1), (dict(table_stride=-4), 1)]


def rows_call(lib, name, c=None, b=None, **kw):
    a = dict(K=0x800000, V=0x900000, xt=0, rows=5, krs=256, khs=128, vrs=256, vhs=128)
    a.update(kw)
    c, b = c or cache(), b or batch()
    return getattr(lib, name)(ctypes.byref(c), ctypes.byref(b), *a.values(), None)


def attn_call(lib, c=None, b=None, **kw):
    a = dict(Q=0x800000, xt=0, rows=5, heads=8, qrs=1024, qhs=128, O=0x900000, ors=1024, ohs=128,
             lse=None, max_rows=2, scale=0.1, causal=1, window=0, ws=0xA00000, wsb=1 << 40)
    a.update(kw)
    c, b = c or cache(), b or batch()
    return lib.w4kv_attention(ctypes.byref(c), ctypes.byref(b), *a.values(), None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(lib, kw, status):
    for name in ("w4kv_append", "w4kv_read"):
        assert rows_call(lib, name, c=cache(**kw)) == status
    assert attn_call(lib, c=cache(**kw)) == status
    assert lib.w4kv_attention_workspace_bytes(ctypes.byref(cache(**kw)), 1, 1, 1, 8) == 0


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_bad_batches(lib, kw, status):
    for name in ("w4kv_append", "w4kv_read"):
        assert rows_call(lib, name, b=batch(**kw)) == status
    assert attn_call(lib, b=batch(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(K=None), 1),
    (dict(V=None), 1), (dict(krs=-8), 1), (dict(khs=-8), 1), (dict(vrs=1 << 33), 1),
    (dict(K=0x800008), 2), (dict(krs=260), 2), (dict(vhs=132, vrs=512), 2),
    (dict(rows=0, K=None, V=None), 0),
])
def test_bad_rows(lib, kw, status):
    for name in ("w4kv_append", "w4kv_read"):
        assert rows_call(lib, name, **kw) == status


def test_empty_batch_is_nothing_to_do(lib):
    b = batch(batch=0, page_table=None, kv_lens=None, cu_rows=None)
    for name in ("w4kv_append", "w4kv_read"):
        assert rows_call(lib, name, b=b) == 0
    assert attn_call(lib, b=b) == 0


@pytest.mark.parametrize("kw", [dict(krs=128), dict(khs=64), dict(khs=0), dict(vrs=0),
                                dict(krs=128, khs=128 * 4)])
def test_overlapping_outputs(lib, kw):
    assert rows_call(lib, "w4kv_read", **kw) == 1
    assert b"overlap" in lib.w4_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(xt=3), 1), (dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=7), 1), (dict(max_rows=0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(window=-1), 1),
    (dict(window=4, causal=0), 1), (dict(Q=None), 1), (dict(O=None), 1), (dict(ohs=64), 1),
    (dict(ors=512), 1), (dict(O=0x900008), 2), (dict(qrs=1028), 2), (dict(lse=0x2), 2),
    (dict(rows=0, Q=None, O=None), 0),
    (dict(rows=1 << 29, max_rows=1 << 29, qrs=1024, ors=1024), 1),   # rows * heads / kv_heads
])
def test_bad_attention(lib, kw, status):
    assert attn_call(lib, **kw) == status


def test_null_structs(lib):
    c, b = ctypes.byref(cache()), ctypes.byref(batch())
    for x, y in ((None, b), (c, None)):
        assert lib.w4kv_append(x, y, 0x800000, 0x900000, 0, 5, 256, 128, 256, 128, None) == 1
        assert lib.w4kv_attention(x, y, 0x800000, 0, 5, 8, 1024, 128, 0x900000, 1024, 128, None, 2,
                                  0.1, 1, 0, 0xA00000, 1 << 40, None) == 1
    assert lib.w4kv_attention_workspace_bytes(None, 1, 1, 1, 8) == 0


def test_binding_refusals():
    z = torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    s = torch.zeros(2, 1, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        w4.W4KVCache(z, s, z, s, w4.W4KV_INT8)
    with pytest.raises(ValueError, match="fmt"):
        w4.W4KVCache(z, s, z, s, 5)
