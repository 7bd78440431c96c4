"""The quantized paged key/value cache on the GPU: w4kv_append and w4kv_read
bit for bit, w4kv_attention within the tolerance that tests/kv_reference.py
derives, at the sizes, masks and inputs where each can go wrong."""
import numpy as np
import pytest
import torch

from tests import kv_reference as R

pytestmark = pytest.mark.gpu
DTYPES = (torch.float16, torch.bfloat16)


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


def rows(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def same_cache(dev_cache, p):
    for i, (c, s) in enumerate(((dev_cache.k_codes, dev_cache.k_scales),
                                (dev_cache.v_codes, dev_cache.v_scales))):
        np.testing.assert_array_equal(c.cpu().numpy(), p.codes[i])
        np.testing.assert_array_equal(s.cpu().numpy().view(np.uint32), p.words[i])


# ---- append ----------------------------------------------------------------------------------

def check_append(w4, p, n_rows, K, V, cache=None):
    """Appends on both sides and compares the whole cache, garbage included."""
    cache = cache or p.device(w4)
    w4.w4kv_append(K.cuda() if not K.is_cuda else K, V.cuda() if not V.is_cuda else V, cache,
                   *p.batch(n_rows))
    t = 0
    for b, n in enumerate(n_rows):
        for i, x in enumerate((K, V)):
            p.store(i, b, p.lens[b] - n, *R.quantize(x[t:t + n].float().cpu().numpy(), p.fmt))
        t += n
    same_cache(cache, p)
    return cache


@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_append_bits(w4, fmt, dtype, D):
    n_rows = [1, 0, 17, 5, 40]
    p = R.Plain([1, 9, 33, 5, 100], fmt, 3, D, 16, 1)
    K, V = (rows((63, 3, D), dtype, s, 2.0) for s in (1, 2))
    check_append(w4, p, n_rows, K, V)


@pytest.mark.parametrize("Hk,page,B", [(1, 16, 1), (8, 48, 40), (5, 256, 3), (33, 32, 2), (2, 16, 1500)])
def test_append_layouts(w4, Hk, page, B):
    r = np.random.default_rng(B)
    lens = list(r.integers(1, 60, B))
    n_rows = [int(r.integers(0, n + 1)) for n in lens]
    p = R.Plain(lens, R.INT4, Hk, 64, page, 5)
    K, V = (rows((sum(n_rows), Hk, 64), torch.float16, s) for s in (3, 4))
    check_append(w4, p, n_rows, K, V)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_append_edge_rows(w4, fmt, dtype):
    """Zeros, constants, one-sided rows, ties, extremes, subnormals, NaN, infinity."""
    D = 64
    big = torch.finfo(dtype).max
    x = rows((24, 1, D), dtype, 9).float()
    x[0] = 0
    x[1] = 3.0
    x[2] = -3.0
    x[3] = x[3].abs()
    x[4] = -x[4].abs()
    x[5, 0, 0] = float("inf")
    x[6, 0, 63] = float("-inf")
    x[7, 0, 31] = float("nan")
    x[8] = big
    x[9, 0, 0], x[9, 0, 1] = big, -big
    x[10] *= torch.finfo(dtype).tiny
    x[11] = torch.finfo(dtype).smallest_normal * 2.0 ** -4
    x[12, 0] = torch.arange(D).float() + 0.5
    x[12, 0, 63] = 127 if fmt == R.INT8 else 448 if fmt == R.E4M3 else 15
    x[13, 0] = torch.arange(D).float() / 4 - 8
    x[14] = -0.0
    x[15] = 0
    x[15, 0, 5] = 1e-7
    x[16, 0] = torch.arange(D).float() * 2.0 ** -9
    x[16, 0, 0] = 448
    p = R.Plain([24], fmt, 1, D, 16, 2)
    x = x.to(dtype)
    check_append(w4, p, [24], x, x.flip(0))


def test_append_values_near_rounding_borders(w4):
    """Every fp16 value against one largest value per row: the codes' borders."""
    allv = torch.arange(0x7C00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    for fmt, top in ((R.INT8, 93.5), (R.E4M3, 1.37), (R.INT4, 7.3)):
        v = allv[allv <= top]
        n = v.numel() // 126
        x = torch.zeros(n, 1, 128, dtype=torch.float16)
        x[:, 0, 1:127] = v[:n * 126].view(n, 126)
        x[:, 0, 0] = top
        p = R.Plain([n], fmt, 1, 128, 64, 1)
        check_append(w4, p, [n], x, -x)


@pytest.mark.parametrize("layout", ["fused", "heads first", "one row for all"])
def test_append_strides(w4, layout):
    T, Hk, D = 21, 4, 128
    if layout == "fused":
        qkv = rows((T, 3 * Hk, D), torch.float16, 1).cuda()
        K, V = qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
    elif layout == "heads first":
        K, V = (rows((Hk, T, D), torch.float16, s).cuda().transpose(0, 1) for s in (1, 2))
    else:
        K, V = (rows((1, 1, D), torch.float16, s).cuda().expand(T, Hk, D) for s in (1, 2))
    p = R.Plain([30], R.E4M3, Hk, D, 16, 1)
    check_append(w4, p, [T], K, V)


def test_append_rows_behind_the_last_sequence(w4):
    p = R.Plain([20, 9], R.INT8, 2, 64, 16, 1)
    K, V = (rows((64, 2, 64), torch.float16, s) for s in (1, 2))
    check_append(w4, p, [4, 2], K, V)  # rows 6 .. 63 belong to nobody


@pytest.mark.parametrize("what", ["page too large", "page negative", "table too narrow", "too many rows"])
def test_append_out_of_range(w4, what):
    """Rows that have no place are not stored and reported; the others are stored."""
    lens, n_rows = [40, 24], [40, 3]
    p = R.Plain(lens, R.INT8, 2, 64, 16, 1)
    K, V = (rows((43, 2, 64), torch.float16, s) for s in (1, 2))
    cache = p.device(w4)
    table, kv_lens, cu = p.batch(n_rows)
    skip = set()
    if what == "page too large":
        table[0, 1] = p.pages
        skip = set(range(16, 32))
    elif what == "page negative":
        table[0, 1] = -1
        skip = set(range(16, 32))
    elif what == "table too narrow":
        table = table[:, :2].contiguous()
        skip = set(range(32, 40))
    else:
        kv_lens[0] = 37  # 40 rows of 37 tokens: the first three are before the start
    w4.w4kv_append(K.cuda(), V.cuda(), cache, table, kv_lens, cu)
    for i, x in enumerate((K, V)):
        c, s = R.quantize(x.float().numpy(), p.fmt)
        if what == "too many rows":
            p.store(i, 0, 0, c[3:40], s[3:40])
        else:
            for j in range(40):
                if j not in skip:
                    p.store(i, 0, j, c[j:j + 1], s[j:j + 1])
        p.store(i, 1, 21, c[40:], s[40:])
    same_cache(cache, p)
    assert w4.w4_device_status() == w4.W4_ERR_BOUNDS


# ---- read ------------------------------------------------------------------------------------

@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_read_bits(w4, fmt, dtype, D):
    lens, n_rows = [50, 3, 17, 129], [50, 0, 4, 129]
    p = R.Plain(lens, fmt, 3, D, 48, 7)
    K, V = w4.w4kv_read(p.device(w4), *p.batch(n_rows), sum(n_rows), dtype=dtype)
    for i, got in enumerate((K, V)):
        want = torch.cat([R.read16(*p.rows(i, b, p.lens[b] - n), fmt, dtype)
                          for b, n in enumerate(n_rows)])
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


def test_read_every_code(w4):
    """Each code byte (E4M3's two NaN codes aside) and each pair of nibbles
    with each zero point, at scales that round and overflow fp16."""
    for fmt in R.FORMATS:
        p = R.Plain([256], fmt, 1, 128, 16, 1)
        c = np.arange(256, dtype=np.uint8)[:, None].repeat(p.codes[0].shape[-1], 1)
        if fmt == R.E4M3:
            c = np.where((c & 127) == 127, np.uint8(0), c)
        w = np.float32([1.0, 0.3, 700.0, 1e-6])[np.arange(256) % 4].view(np.uint32)
        w = (w & ~np.uint32(15)) | (np.arange(256) // 4 % 16).astype(np.uint32)
        for i in range(2):
            p.store(i, 0, 0, c[:, None], w[:, None])
        for dtype in DTYPES:
            got = w4.w4kv_read(p.device(w4), *p.batch([256]), 256, dtype=dtype)[0]
            want = R.read16(*p.rows(0, 0), fmt, dtype)
            assert torch.equal(got.cpu(), want)


def test_read_leaves_rows_behind_the_last_sequence(w4):
    p = R.Plain([20, 9], R.E4M3, 2, 64, 16, 1)
    out = tuple(torch.full((2, 40, 64), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
                for _ in range(2))  # heads first
    w4.w4kv_read(p.device(w4), *p.batch([20, 2]), 40, out=out)
    for i in range(2):
        want = torch.cat([R.read16(*p.rows(i, 0), p.fmt, torch.float16),
                          R.read16(*p.rows(i, 1, 7), p.fmt, torch.float16)])
        assert torch.equal(out[i][:22].cpu(), want)
        assert (out[i][22:] == 7).all()


def test_read_out_of_range_is_zero(w4):
    p = R.Plain([40], R.INT8, 2, 64, 16, 1)
    table, lens, cu = p.batch([40])
    table[0, 1] = p.pages + 5
    K, V = w4.w4kv_read(p.device(w4), table, lens, cu, 40)
    assert (K[16:32] == 0).all() and (V[16:32] == 0).all()
    want = R.read16(*p.rows(0, 0), p.fmt, torch.float16)
    assert torch.equal(K[:16].cpu(), want[:16]) and torch.equal(K[32:].cpu(), want[32:])
    assert w4.w4_device_status() == w4.W4_ERR_BOUNDS


# ---- attention -------------------------------------------------------------------------------

def close(O, lse, want, label=""):
    Ow, lw, tol, ltol = want
    o = O.detach().cpu().double()
    live = ~torch.isnan(tol)
    err = (o - Ow).abs()
    bad = live & ~(err <= tol)
    assert not bad.any(), f"{label}: {int(bad.sum())} of {int(live.sum())} off, worst " \
                          f"{float((err / tol.clamp(min=1e-30))[live].max()):.2f} of the tolerance"
    if lse is not None:
        l = lse.cpu().double()
        fin = torch.isfinite(lw)
        inf = torch.isinf(lw)
        assert torch.equal(l[inf], lw[inf])
        assert ((l[fin] - lw[fin]).abs() <= ltol[fin]).all(), label


def check_attention(w4, p, n_rows, H, dtype=torch.float16, seed=11, causal=True, window=0, scale=None,
                    q_scale=1.0, max_rows=None):
    T = sum(n_rows)
    Q = rows((T, H, p.D), dtype, seed, q_scale)
    scale = p.D ** -0.5 if scale is None else scale
    O, lse = w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch(n_rows), scale=scale, causal=causal,
                               window=window, return_lse=True,
                               max_rows=max(n_rows) if max_rows is None else max_rows)
    close(O, lse, R.attention(p, Q, n_rows, scale, causal, window), f"{n_rows} {H}")
    return Q, O


@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("n,H", [(1, 2), (1, 16), (1, 32), (3, 12), (9, 8), (70, 4)])
def test_attention_types(w4, fmt, dtype, D, n, H):
    p = R.Plain([n, 131, 300], fmt, 2, D, 16, 1)
    check_attention(w4, p, [n, n, n], H, dtype)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_lengths(w4, length, n):
    n = min(n, length)
    p = R.Plain([length], R.INT8, 1, 128, 32, length)
    check_attention(w4, p, [n], 4)


@pytest.mark.parametrize("page", [16, 48, 80, 256])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_attention_pages(w4, page, fmt):
    p = R.Plain([700, 31, 255], fmt, 2, 128, page, 3)
    check_attention(w4, p, [1, 1, 1], 8)
    check_attention(w4, p, [100, 31, 60], 6)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 16, 17, 40, 128, 200])
def test_attention_head_groups(w4, G):
    p = R.Plain([90, 150], R.INT4, 2, 64, 16, 4)
    check_attention(w4, p, [1, 1], 2 * G)
    check_attention(w4, p, [5, 2], 2 * G)


@pytest.mark.parametrize("n_rows", [[1, 300, 1, 0, 17], [0, 0, 5], [257, 2], [128, 129, 127], [2, 2, 2, 2]])
def test_attention_mixed_batches(w4, n_rows):
    r = np.random.default_rng(len(n_rows))
    lens = [n + int(r.integers(0, 400)) for n in n_rows]
    p = R.Plain(lens, R.E4M3, 2, 64, 16, 8)
    check_attention(w4, p, n_rows, 8, torch.bfloat16)
    check_attention(w4, p, n_rows, 2, max_rows=sum(n_rows) + 1000)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 129, 5000])
@pytest.mark.parametrize("n_rows", [[1, 1], [4, 4], [200, 60]])
def test_attention_windows(w4, n_rows, window):
    p = R.Plain([513, 64], R.INT8, 2, 64, 16, 2)
    check_attention(w4, p, n_rows, 4, window=window)


@pytest.mark.parametrize("n_rows", [[1, 1, 1], [6, 90, 300]])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_attention_not_causal(w4, fmt, n_rows):
    p = R.Plain([20, 200, 311], fmt, 2, 128, 32, 2)
    check_attention(w4, p, n_rows, 6, causal=False)


@pytest.mark.parametrize("n_rows", [[1, 1, 1], [40, 30, 300]])
def test_attention_rows_that_see_nothing(w4, n_rows):
    """Lengths of zero, and fewer tokens than rows: zeros and lse = -infinity."""
    p = R.Plain([0, 12, 100], R.INT8, 2, 64, 16, 2)
    for causal in (True, False):
        Q, O = check_attention(w4, p, n_rows, 4, causal=causal)
        assert (O[:n_rows[0]] == 0).all()


def test_attention_empty_batch_and_no_rows(w4):
    p = R.Plain([5], R.INT8, 1, 64, 16, 1)
    cache, (table, lens, cu) = p.device(w4), p.batch([0])
    Q = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    out = torch.full_like(Q, 3)
    w4.w4kv_attention(Q, cache, table, lens, cu, out=out)         # rows, but of no sequence
    w4.w4kv_attention(Q, cache, table[:0], lens[:0], cu[:1], out=out)
    assert (out == 3).all()
    assert w4.w4kv_attention(Q[:0], cache, table, lens, cu).shape == (0, 2, 64)


@pytest.mark.parametrize("n_rows,extra", [([3, 1], 5), ([1, 1], 1), ([150, 20], 100)])
def test_attention_rows_behind_the_last_sequence(w4, n_rows, extra):
    p = R.Plain([200, 50], R.INT4, 2, 64, 16, 1)
    T = sum(n_rows)
    Q = rows((T + extra, 4, 64), torch.float16, 1)
    Q[T:] = float("nan")
    out = torch.full((T + extra, 4, 64), 3.0, dtype=torch.float16, device="cuda")
    w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch(n_rows), out=out)
    close(out[:T], None, R.attention(p, Q[:T], n_rows, 0.125))
    assert (out[T:] == 3).all()


@pytest.mark.parametrize("n", [1, 40])
def test_attention_strides(w4, n):
    """Queries as a slice of a fused projection, outputs heads first."""
    p = R.Plain([100, 60], R.E4M3, 2, 128, 16, 1)
    qkv = rows((2 * n, 12, 128), torch.bfloat16, 5).cuda()
    Q = qkv[:, 2:10]
    out = torch.empty((8, 2 * n, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    w4.w4kv_attention(Q, p.device(w4), *p.batch([n, n]), out=out)
    close(out, None, R.attention(p, Q.cpu(), [n, n], 128 ** -0.5))
    one = rows((1, 1, 128), torch.bfloat16, 6).cuda().expand(2 * n, 8, 128)  # one query for all
    O = w4.w4kv_attention(one, p.device(w4), *p.batch([n, n]))
    close(O, None, R.attention(p, one.cpu(), [n, n], 128 ** -0.5))


@pytest.mark.parametrize("n_rows", [[1], [3], [150]])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_attention_non_finite_where_unseen(w4, fmt, n_rows):
    """A row with a NaN reaches the rows that see it and no others: later
    tokens of the chunk, tokens before the window, garbage behind the end (the
    test caches are full of it), and other heads."""
    n, L = n_rows[0], 300
    p = R.Plain([L], fmt, 2, 64, 16, 1)
    H = 4
    Q = rows((n, H, 64), torch.float16, 2)
    clean = p.device(w4)
    batch = p.batch(n_rows)
    for at, window in ((L - 1, 0), (10, 64)):
        want = w4.w4kv_attention(Q.cuda(), clean, *batch, window=window)
        bad = p.device(w4)
        pg, off = p.at(0, at)
        for s in (bad.k_scales, bad.v_scales):
            s[int(pg), 0, int(off)] = float("nan")
        got = w4.w4kv_attention(Q.cuda(), bad, *batch, window=window)
        pos = torch.arange(L - n, L)
        sees = (pos >= at) & (pos - (window or L + 1) < at)
        assert torch.equal(got[:, 2:], want[:, 2:])          # the other key/value head
        assert torch.isnan(got[sees.cuda(), :2]).all()
        assert torch.equal(got[~sees.cuda(), :2], want[~sees.cuda(), :2])


def test_attention_nan_query_stays_in_its_row(w4):
    for n in (3, 60):
        p = R.Plain([100], R.INT8, 1, 64, 16, 1)
        Q = rows((n, 2, 64), torch.bfloat16, 2)
        want = w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch([n]))
        Q[1, 0, 5] = float("nan")
        got = w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch([n]))
        assert torch.isnan(got[1, 0]).all()
        got[1, 0] = want[1, 0]
        assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("n", [1, 40])
def test_attention_extreme_values(w4, fmt, n):
    """Value rows whose sizes span far more than fp16's range, large and tiny
    queries, and one token that takes all the weight."""
    L = 260
    p = R.Plain([L], fmt, 1, 128, 16, 1, dtype=torch.bfloat16)
    r = np.random.default_rng(3)
    v = r.standard_normal((L, 1, 128)) * 10.0 ** r.uniform(-12, 12, (L, 1, 1))
    p.store(1, 0, 0, *R.quantize(v.astype(np.float32), fmt))
    check_attention(w4, p, [n], 2, torch.bfloat16)
    p.store(1, 0, 0, *R.quantize((v[:, :, ::-1] * 1e-25).astype(np.float32), fmt))
    check_attention(w4, p, [n], 2, torch.bfloat16)
    p = R.Plain([L], fmt, 1, 128, 16, 1, dtype=torch.bfloat16)
    check_attention(w4, p, [n], 2, torch.bfloat16, q_scale=1e-30)
    check_attention(w4, p, [n], 2, torch.bfloat16, q_scale=1e30, scale=1e-31)
    check_attention(w4, p, [n], 2, torch.bfloat16, q_scale=20.0)
    check_attention(w4, p, [n], 2, torch.float16, q_scale=2.0 ** -20, scale=2.0 ** 16)
    check_attention(w4, p, [n], 2, torch.float16, scale=-0.1)
    check_attention(w4, p, [n], 2, torch.float16, scale=0.0)


@pytest.mark.parametrize("n_rows,H", [([1, 1], 4), ([200, 5], 4)])
def test_attention_bad_pages(w4, n_rows, H):
    """Pages out of range count as unseen, and are reported."""
    p = R.Plain([400, 250], R.E4M3, 2, 64, 16, 1)
    table, lens, cu = p.batch(n_rows)
    unseen = []
    for b, pg, v in ((0, 2, p.pages), (0, 7, -1), (1, 0, 1 << 30)):
        table[b, pg] = v
        unseen += [(b, j) for j in range(16 * pg, 16 * pg + 16)]
    Q = rows((sum(n_rows), H, 64), torch.float16, 3)
    O, lse = w4.w4kv_attention(Q.cuda(), p.device(w4), table, lens, cu, return_lse=True)
    close(O, lse, R.attention(p, Q, n_rows, 0.125, unseen=unseen))
    assert w4.w4_device_status() == w4.W4_ERR_BOUNDS


@pytest.mark.parametrize("n_rows", [[1, 1], [100, 100]])
def test_attention_length_beyond_the_table(w4, n_rows):
    p = R.Plain([256, 130], R.INT8, 1, 64, 16, 1)
    table, lens, cu = p.batch(n_rows)
    Q = rows((sum(n_rows), 2, 64), torch.float16, 3)
    short = table[:, :10].contiguous()
    O, lse = w4.w4kv_attention(Q.cuda(), p.device(w4), short, lens, cu, return_lse=True)
    close(O, lse, R.attention(p, Q, n_rows, 0.125, unseen=[(0, j) for j in range(160, 256)]))
    assert w4.w4_device_status() == w4.W4_ERR_BOUNDS


@pytest.mark.parametrize("n,given", [(5, 2), (100, 60), (40, 1)])
def test_attention_more_rows_than_max_rows(w4, n, given):
    """The first max_rows rows are served, the others left, and it is reported."""
    p = R.Plain([200], R.INT8, 1, 64, 16, 1)
    Q = rows((n, 4, 64), torch.float16, 3)
    out = torch.full((n, 4, 64), 3.0, dtype=torch.float16, device="cuda")
    w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch([n]), max_rows=given, out=out)
    close(out[:given], None, tuple(x[:given] for x in R.attention(p, Q, [n], 0.125)))
    assert (out[given:] == 3).all()
    assert w4.w4_device_status() == w4.W4_ERR_BOUNDS


@pytest.mark.parametrize("n_rows", [[1] * 40, [60, 1, 200]])
def test_attention_repeats_bit_for_bit(w4, n_rows):
    r = np.random.default_rng(1)
    p = R.Plain([n + int(r.integers(0, 900)) for n in n_rows], R.INT8, 2, 128, 16, 1)
    Q = rows((sum(n_rows), 8, 128), torch.float16, 1).cuda()
    cache, batch = p.device(w4), p.batch(n_rows)
    first = w4.w4kv_attention(Q, cache, *batch)
    for _ in range(5):
        assert torch.equal(w4.w4kv_attention(Q, cache, *batch), first)


def test_attention_many_sequences(w4):
    """More sequences than a block has threads, with gaps."""
    r = np.random.default_rng(5)
    n_rows = [int(x) for x in r.integers(0, 4, 700)]
    p = R.Plain([n + int(x) for n, x in zip(n_rows, r.integers(0, 50, 700))], R.INT8, 1, 64, 16, 1)
    check_attention(w4, p, n_rows, 2)
    n_rows[333] = 30
    p = R.Plain([n + int(x) for n, x in zip(n_rows, r.integers(0, 50, 700))], R.INT8, 1, 64, 16, 1)
    check_attention(w4, p, n_rows, 2)


def test_workspace_argument(w4):
    p = R.Plain([3000], R.INT8, 2, 128, 16, 1)
    Q = rows((1, 8, 128), torch.float16, 1).cuda()
    cache, batch = p.device(w4), p.batch([1])
    want = w4.w4kv_attention(Q, cache, *batch, max_rows=1)
    need = w4.w4kv_attention_workspace_bytes(cache, 1, 1, 1, 8)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(w4.w4kv_attention(Q, cache, *batch, max_rows=1, workspace=ws[256:256 + need]), want)
    assert (ws[:256] == 255).all() and (ws[256 + need:] == 255).all()
    if need:
        with pytest.raises(w4.W4Error, match="workspace"):
            w4.w4kv_attention(Q, cache, *batch, max_rows=1, workspace=ws[:need - 256])


# ---- streams, graphs, the operators together --------------------------------------------------

def test_side_stream(w4):
    p = R.Plain([400, 90], R.INT8, 2, 128, 16, 1)
    Q = rows((2, 8, 128), torch.float16, 1).cuda()
    cache, batch = p.device(w4), p.batch([1, 1])
    want = w4.w4kv_attention(Q, cache, *batch)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w4.w4kv_attention(Q, cache, *batch, stream=s)
    K, V = w4.w4kv_read(cache, *batch, 2, stream=s)
    w4.w4kv_append(K, V, cache, *batch, stream=s)  # what it stands for is kept by a second pass
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1, 40])
def test_captured_graphs_follow_lengths(w4, n):
    """One graph serves changing lengths and pages; two graphs run at once."""
    lens = [300, 77]
    p = R.Plain(lens, R.E4M3, 2, 64, 16, 1)
    cache, (table, kv_lens, cu) = p.device(w4), p.batch([n, n])
    Q = rows((2 * n, 8, 64), torch.bfloat16, 1).cuda()
    w4.w4kv_attention(Q, cache, table, kv_lens, cu, max_rows=n)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w4.w4kv_attention(Q, cache, table, kv_lens, cu, max_rows=n))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for new in (lens, [299, 70], [n, 60], [250, 77]):
        kv_lens.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        p.lens = list(new)
        want = R.attention(p, Q.cpu(), [n, n], 0.125)
        close(outs[0], None, want, str(new))
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_layer_with_quantized_weights(w4, fmt):
    """The operators as they are used: a prompt in two chunks and three decode
    steps of two sequences through W4A16 projections, the cache and the
    attention; the cache's contents and the attention's outputs against the
    reference on the very projections' outputs."""
    H, Hk, D, C = 8, 2, 64, 512
    dt = torch.float16
    g = torch.Generator().manual_seed(4)
    Wqkv = (torch.randn(((H + 2 * Hk) * D, C), generator=g) * 0.05).to(dt).cuda()
    Wo = (torch.randn((C, H * D), generator=g) * 0.05).to(dt).cuda()
    qkv_w, o_w = w4.w4_quantize(Wqkv, sym=False), w4.w4_quantize(Wo, sym=False)
    cache = w4.w4kv_cache_empty(30, 16, Hk, D, fmt)
    p = R.Plain([0, 0], fmt, Hk, D, 16, 1, width=8)
    p.pages = 30
    p.codes = [c.cpu().numpy().copy() for c in (cache.k_codes, cache.v_codes)]
    p.words = [s.cpu().numpy().view(np.uint32).copy() for s in (cache.k_scales, cache.v_scales)]
    p.table = np.random.default_rng(2).permutation(30)[:16].reshape(2, 8).astype(np.int32)
    for n_rows in ([50, 7], [33, 60], [1, 1], [1, 1], [1, 1]):
        T = sum(n_rows)
        p.lens = [a + n for a, n in zip(p.lens, n_rows)]
        x = torch.randn((T, C), generator=g).to(dt).cuda()
        qkv = w4.w4a16_gemm(x, *qkv_w).view(T, H + 2 * Hk, D)
        batch = p.batch(n_rows)
        w4.w4kv_append(qkv[:, H:H + Hk], qkv[:, H + Hk:], cache, *batch)
        O = w4.w4kv_attention(qkv[:, :H], cache, *batch, max_rows=max(n_rows))
        y = w4.w4a16_gemm(O.view(T, H * D), *o_w)
        t = 0
        for b, n in enumerate(n_rows):
            for i, lo in enumerate((H, H + Hk)):
                p.store(i, b, p.lens[b] - n,
                        *R.quantize(qkv[t:t + n, lo:lo + Hk].float().cpu().numpy(), fmt))
            t += n
        same_cache(cache, p)
        close(O, None, R.attention(p, qkv[:, :H].cpu(), n_rows, D ** -0.5))
        assert torch.isfinite(y).all()


def test_offsets_beyond_32_bits(w4):
    """A cache of more than 2^32 code bytes: its last pages are written, read
    and attended to like the first."""
    Hk, D, page = 8, 128, 256
    per = Hk * page * D
    pages = (1 << 32) // per + 40
    codes = [torch.empty((pages, Hk, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty((pages, Hk, page), dtype=torch.float32, device="cuda") for _ in range(2)]
    cache = w4.W4KVCache(codes[0], scales[0], codes[1], scales[1], w4.W4KV_INT8)
    n = 600
    p = R.Plain([n], R.INT8, Hk, D, page, 1)
    K, V = (torch.from_numpy(p.kv[i][0]).half() for i in range(2))
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    w4.w4kv_append(K.cuda(), V.cuda(), cache, table, lens, cu)
    k, v = w4.w4kv_read(cache, table, lens, cu, n)
    assert torch.equal(k.cpu(), R.read16(*p.rows(0, 0), p.fmt, torch.float16))
    assert torch.equal(v.cpu(), R.read16(*p.rows(1, 0), p.fmt, torch.float16))
    for m in (1, 20):
        Q = rows((m, 16, D), torch.float16, 1)
        O = w4.w4kv_attention(Q.cuda(), cache, table, lens,
                              torch.tensor([0, m], dtype=torch.int32, device="cuda"))
        close(O, None, R.attention(p, Q, [m], D ** -0.5))


@pytest.mark.parametrize("seed", range(12))
def test_attention_random_calls(w4, seed):
    """Calls drawn over formats, types, layouts, lengths, masks and row counts."""
    r = np.random.default_rng(1000 + seed)
    fmt, D = int(r.integers(3)), int(r.choice([64, 128]))
    Hk, G = int(r.integers(1, 4)), int(r.choice([1, 2, 3, 5, 8, 11]))
    B = int(r.integers(1, 7))
    n_rows = [int(r.choice([0, 1, 1, 2, 7, 20, 90, 140])) for _ in range(B)]
    lens = [max(1, n + int(r.integers(-3, 500))) for n in n_rows]
    if sum(n_rows) == 0:
        n_rows[0] = 1
    causal = bool(r.random() < 0.8)
    window = int(r.integers(1, 300)) if causal and r.random() < 0.4 else 0
    dtype = DTYPES[int(r.integers(2))]
    p = R.Plain(lens, fmt, Hk, D, int(r.choice([16, 48, 64, 128])), seed, dtype=dtype)
    check_attention(w4, p, n_rows, Hk * G, dtype, seed, causal, window,
                    scale=float(r.choice([D ** -0.5, 0.02, 0.3])), q_scale=float(r.choice([1.0, 4.0])),
                    max_rows=max(n_rows) + int(r.integers(0, 100)))


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_attention_errors_are_small(w4, fmt):
    """fp16 decode steps: the error's norm is the output rounding's (2^-11 / sqrt 3
    of a value at most), to 1.3; chunks carry the weights' rounding too, to 1.8."""
    p = R.Plain([700, 300], fmt, 2, 128, 16, 5)
    for n_rows, limit in (([1, 1], 1.3), ([5, 4], 1.3), ([90, 70], 1.8)):
        Q = rows((sum(n_rows), 8, 128), torch.float16, 4)
        O = w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch(n_rows)).cpu().double()
        want = R.attention(p, Q, n_rows, 128 ** -0.5)[0]
        assert (O - want).norm() <= limit * 2.0 ** -11 / 3 ** 0.5 * want.norm()
