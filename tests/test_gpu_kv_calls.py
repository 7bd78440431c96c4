"""Calls of the key/value cache in an order or on a stream that decides: empty
batches before full ones, refusals before valid calls, explicit streams."""
import threading

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


@pytest.mark.parametrize("what", ["attention", "lse", "read"])
def test_explicit_stream_takes_its_own_memory(w4, what):
    """Outputs of a call on another stream do not land in memory that the
    current stream still reads."""
    p = R.Plain([400], R.INT8, 2, 128, 16, 1)
    n, H = 300, 16
    Q = rows((n, H, 128), torch.float16, 1).cuda()
    cache, batch = p.device(w4), p.batch([n])
    shape = {"attention": (n, H, 128), "lse": (n, H), "read": (n, 2, 128)}[what]
    dtype = torch.float32 if what == "lse" else torch.float16
    s = torch.cuda.Stream()

    def call(stream):
        if what == "read":
            return w4.w4kv_read(cache, *batch, n, stream=stream)
        return w4.w4kv_attention(Q, cache, *batch, return_lse=what == "lse", stream=stream)

    call(None)
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.full(shape, 7, dtype=dtype, device="cuda") for _ in range(4)]
        torch.cuda._sleep(20_000_000)          # some milliseconds of the current stream
        kept = [x.clone() for x in old]        # reads `old` after them
        del old
        out = call(s)
        torch.cuda.synchronize()
        assert all((x == 7).all() for x in kept)
        del out


def test_calls_on_two_streams_at_once(w4):
    """Scratch space and outputs of calls in flight on different streams are apart."""
    p = R.Plain([4000, 900], R.E4M3, 2, 128, 16, 1)
    Q = rows((2 * 150, 8, 128), torch.bfloat16, 1).cuda()
    cache, batch = p.device(w4), p.batch([150, 150])
    want = w4.w4kv_attention(Q, cache, *batch, max_rows=150)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        outs = [w4.w4kv_attention(Q, cache, *batch, max_rows=150, stream=s) for s in streams + [None]]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_two_threads_at_once(w4):
    """Each thread fills its own batch description."""
    plans = [R.Plain([300 + 50 * i, 90], R.INT8, 2, 64, 16, i) for i in range(2)]
    Q = rows((2 * 5, 8, 64), torch.float16, 1).cuda()
    calls = [(p.device(w4), p.batch([5, 5])) for p in plans]
    want = [w4.w4kv_attention(Q, c, *b, max_rows=5) for c, b in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(200):
            if not torch.equal(w4.w4kv_attention(Q, calls[i][0], *calls[i][1], max_rows=5), want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_explicit_stream_inside_a_capture(w4):
    """A graph that forks to another stream for its call."""
    p = R.Plain([700, 90], R.INT8, 2, 64, 16, 1)
    n = 40
    Q = rows((2 * n, 8, 64), torch.float16, 1).cuda()
    cache, batch = p.device(w4), p.batch([n, n])
    want = w4.w4kv_attention(Q, cache, *batch, max_rows=n)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        O = w4.w4kv_attention(Q, cache, *batch, max_rows=n, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        y = O + 0
    for _ in range(3):
        O.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_stream_of_no_device_of_the_cache(w4):
    """A stream of another device is refused (one that says so: there may be one device only)."""
    class Foreign:
        cuda_stream, device = 0, torch.device("cuda", 7)
    p = R.Plain([20], R.INT8, 1, 64, 16, 1)
    Q = rows((1, 1, 64), torch.float16, 1).cuda()
    with pytest.raises(ValueError, match="stream"):
        w4.w4kv_attention(Q, p.device(w4), *p.batch([1]), stream=Foreign())


def test_single_rows_and_heads_of_any_stride(w4):
    """Dimensions of size one keep odd strides through torch's views."""
    D = 64
    p = R.Plain([40], R.INT8, 1, D, 16, 1)
    cache, batch = p.device(w4), p.batch([1])
    q = rows((1, 1, D), torch.float16, 3).cuda()
    odd = q.view(D, 1).T.unsqueeze(1)
    odd = odd.as_strided((1, 1, D), (1, 3, 1))
    assert torch.equal(w4.w4kv_attention(odd, cache, *batch), w4.w4kv_attention(q, cache, *batch))
    K, V = w4.w4kv_read(cache, *batch, 1)
    other = R.Plain([40], R.INT8, 1, D, 16, 9).device(w4)
    w4.w4kv_append(K.as_strided((1, 1, D), (5, 1, 1)), V, other, *batch)
    k, v = w4.w4kv_read(other, *batch, 1)
    again = R.Plain([40], R.INT8, 1, D, 16, 9).device(w4)
    w4.w4kv_append(K, V, again, *batch)
    assert all(torch.equal(a, b) for a, b in zip((k, v), w4.w4kv_read(again, *batch, 1)))
