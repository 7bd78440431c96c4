"""Calls of the key/value cache in an order or on a stream that decides: empty
batches before full ones, refusals before valid calls."""
import pytest
import torch

from tests import kv_reference as R
from tests.test_gpu_kv import close, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import weight_only_int4_pack_b200 as m
    m.load()
    m.w4_device_status()
    return m


@pytest.fixture(autouse=True)
def _clean_status(w4):
    yield
    assert w4.w4_device_status() == w4.W4_OK


@pytest.mark.parametrize("n,heads", [(7, 6), (111, 6)])
def test_empty_batch_then_one_sequence(w4, n, heads):
    """A call without sequences leaves nothing behind that a later one trips over."""
    p = R.Plain([300], R.INT8, 2, 64, 16, 1)
    cache, (table, lens, cu) = p.device(w4), p.batch([n])
    Q = rows((n, heads, 64), torch.float16, 1)
    w4.w4kv_attention(Q.cuda(), cache, table[:0], lens[:0], cu[:1])
    O = w4.w4kv_attention(Q.cuda(), cache, table, lens, cu)
    close(O, None, R.attention(p, Q, [n], 0.125))


def test_workspace_sizes_are_few(w4):
    """What is kept of the sizes of past calls does not grow without end."""
    p = R.Plain([4000], R.INT8, 1, 64, 16, 1)
    cache, (table, lens, cu) = p.device(w4), p.batch([1])
    Q = rows((700, 1, 64), torch.float16, 1).cuda()
    for n in range(1, 700):
        w4.w4kv_attention(Q[:n], cache, table, lens, cu)
    assert len(cache._need) <= 256


@pytest.mark.parametrize("n,heads", [(9, 10), (113, 10)])
def test_refused_cache_then_a_valid_one(w4, n, heads):
    """A refused page size does not reach the calls on a cache that differs in nothing else."""
    bad = w4.W4KVCache(*(torch.zeros(s, dtype=d, device="cuda") for s, d in
                         (((4, 2, 24, 64), torch.uint8), ((4, 2, 24), torch.float32)) * 2), w4.W4KV_INT8)
    p = R.Plain([300], R.INT8, 2, 64, 16, 1)
    cache, batch = p.device(w4), p.batch([n])
    Q = rows((n, heads, 64), torch.float16, 1)
    with pytest.raises(w4.W4Error, match="page_size"):
        w4.w4kv_attention(Q.cuda(), bad, *batch)
    close(w4.w4kv_attention(Q.cuda(), cache, *batch), None, R.attention(p, Q, [n], 0.125))
