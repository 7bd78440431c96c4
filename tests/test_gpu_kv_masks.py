"""Attention over the quantized cache where masks decide: rows that see
nothing, and whatever lies where a row does not look."""
import numpy as np
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


# ---- many items of a block without steps of their own -----------------------------------------

@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("n,H,Hk", [(200, 4, 4), (130, 8, 4), (70, 4, 4)])
def test_padded_sequences(w4, n, H, Hk, D):
    """Sequences of length zero, more of them than the GPU has blocks, before
    and after one with tokens: zeros, lse = -infinity, and no wait runs out."""
    for lens in ([0] * 300, [0] * 150 + [400] + [0] * 149, [3, 0, 0, 0, 0, 0] * 40):
        p = R.Plain(lens, R.INT8, Hk, D, 16, 1)
        T = n * len(lens)
        Q = rows((T, H, D), torch.float16, 5).cuda()
        O, lse = w4.w4kv_attention(Q, p.device(w4), *p.batch([n] * len(lens)), max_rows=n, return_lse=True)
        for b, length in enumerate(lens):
            own = slice(b * n + max(0, n - length), (b + 1) * n)
            blind = slice(b * n, own.start)
            assert (O[blind] == 0).all() and (lse[blind] == -torch.inf).all()
            if length:
                one = R.Plain([length], R.INT8, Hk, D, 16, 1)
                one.codes, one.words, one.pages = p.codes, p.words, p.pages
                one.table = p.table[b:b + 1]
                want = R.attention(one, Q[own].cpu(), [min(n, length)], D ** -0.5)
                close(O[own], lse[own], want, f"{lens[:3]} {b}")
                if b > 150:
                    break


def test_short_items_in_every_block(w4):
    """Items of one and two steps, whole and split row tiles mixed."""
    r = np.random.default_rng(4)
    n_rows = [int(x) for x in r.choice([1, 70, 128, 129, 140, 256, 257], 120)]
    lens = [int(x) for x in r.choice([0, 1, 5, 100, 127, 128, 129, 200, 256], 120)]
    p = R.Plain(lens, R.E4M3, 3, 64, 16, 2)
    T = sum(n_rows)
    Q = rows((T, 3, 64), torch.bfloat16, 6)
    for causal in (True, False):
        O, lse = w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch(n_rows), max_rows=257,
                                   causal=causal, return_lse=True)
        close(O, lse, R.attention(p, Q, n_rows, 0.125, causal), str(causal))
