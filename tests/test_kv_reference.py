"""The reference of the quantized key/value cache, pinned on the CPU without
itself: E4M3 against torch's type, INT8 against numpy's rounding at scale 1,
INT4 by brute force over its levels and by a hand-written word, attention
against a library softmax and by special cases."""
import numpy as np
import pytest
import torch

from tests import kv_reference as R


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.e4m3_table(), t)


def test_e4m3_codes_are_torchs():
    x = np.random.default_rng(0).standard_normal((400, 64)).astype(np.float32)
    x[:, 0] = 448.0  # scale 1
    x[0, 1:40] = np.linspace(0, 0.03, 39)  # subnormals
    code, word = R.quantize(x, R.E4M3)
    assert (word.view(np.float32) == 1).all()
    np.testing.assert_array_equal(code, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8))


def test_int8_codes_at_scale_one():
    x = np.random.default_rng(1).uniform(-127, 127, (50, 64)).astype(np.float32)
    x[:, 3] = -127
    x[:, 5] = np.arange(50) + 0.5  # ties
    code, word = R.quantize(x, R.INT8)
    assert (word.view(np.float32) == 1).all()
    np.testing.assert_array_equal(code.view(np.int8), np.rint(x))


def test_int4_word_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :8] = np.arange(8)       # s = 1, z = 0 with the largest 15
    x[0, 8] = 15
    code, word = R.quantize(x, R.INT4)
    assert word[0] == np.float32(1).view(np.uint32)
    # nibbles 0 .. 7 hold k = 0, 2, 4, 6, 1, 3, 5, 7
    assert code[0, :4].tobytes() == bytes([0x20, 0x64, 0x31, 0x75])
    x[0, 9] = -15                 # range 30: s = 2, z = rne(7.5) = 8
    code, word = R.quantize(x, R.INT4)
    assert word[0] == np.float32(2).view(np.uint32) | 8


@pytest.mark.parametrize("seed", range(3))
def test_int4_codes_are_nearest_levels(seed):
    x = (np.random.default_rng(seed).standard_normal((64, 128)) * 10.0 ** seed).astype(np.float32)
    code, word = R.quantize(x, R.INT4)
    v = R.values(code, word, R.INT4)
    s = (word & ~np.uint32(15)).view(np.float32).astype(np.float64)[:, None]
    z = (word & np.uint32(15))[:, None]
    levels = (np.arange(16) - z)[:, None, :] * s[:, :, None]
    best = np.abs(levels - x[:, :, None]).min(-1)
    assert (np.abs(v - x) <= best * (1 + 1e-6) + s * 1e-6).all()
    # the scale keeps 20 of its 24 bits, and zero is a level
    lo, hi = np.minimum(x.min(-1), 0), np.maximum(x.max(-1), 0)
    assert (np.abs(s[:, 0] * 15 / (hi - lo) - 1) <= 2.0 ** -20 + 2.0 ** -22).all()
    assert (z >= 0).all() and (z <= 15).all()


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_special_rows(fmt):
    x = np.zeros((5, 64), np.float32)
    x[1, 7] = np.inf
    x[2, 7] = np.nan
    x[3] = 1e-45   # the scale underflows to 0
    x[4] = 3.0     # a constant row keeps its value
    code, word = R.quantize(x, fmt)
    v = R.values(code, word, fmt)
    assert (v[0] == 0).all() and np.isnan(v[1:3]).all() and (v[3] == 0).all()
    np.testing.assert_allclose(v[4], 3.0, rtol=2.0 ** -19)
    if fmt == R.INT4:  # hi - lo overflows
        y = np.zeros((1, 64), np.float32)
        y[0, 0], y[0, 1] = 3e38, -3e38
        assert np.isnan(R.values(*R.quantize(y, fmt), fmt)).all()


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_attention_reference(causal, window):
    n_rows, H = [3, 0, 7, 1], 6
    p = R.Plain([20, 4, 7, 33], R.INT8, 2, 64, 16, 3)
    Q = torch.randn(11, H, 64, generator=torch.Generator().manual_seed(1)).half()
    O, lse, tol, _ = R.attention(p, Q, n_rows, 0.125, causal, window)
    t = 0
    for b, n in enumerate(n_rows):
        L = p.lens[b]
        k, v = (torch.from_numpy(R.values(*p.rows(i, b), p.fmt)).repeat_interleave(3, 1).transpose(0, 1)
                for i in range(2))
        mask = torch.ones(n, L, dtype=torch.bool)
        if causal:
            mask = mask.tril(L - n)
            if window:
                mask &= ~torch.ones(n, L, dtype=torch.bool).tril(L - n - window)
        q = Q[t:t + n].double().transpose(0, 1)
        if n:
            want = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=mask, scale=0.125)
            torch.testing.assert_close(O[t:t + n], want.transpose(0, 1), rtol=1e-10, atol=1e-12)
        t += n
    assert (tol > 0).all() and (tol < 0.05).all()
    p2 = R.Plain([2], R.INT8, 1, 64, 16, 4)
    O, lse, tol, _ = R.attention(p2, Q[:5, :1], [5], 0.125)  # rows before the first position
    assert (O[:3] == 0).all() and torch.isinf(lse[:3]).all() and (tol[:3] < 1e-8).all()
    torch.testing.assert_close(O[3, 0], torch.from_numpy(R.values(*p2.rows(1, 0, 0, 1), R.INT8))[0, 0])
