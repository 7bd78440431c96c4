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


# ---- what a row does not see has no influence, whatever it holds -------------------------------

def row_tolerance(p, Q, n_rows, scale, causal=True, window=0):
    """R.attention with the absolute term of the tolerance taken per row, over
    the tokens that this row sees.  A weight is fed as fp16(prob * s * 2^(133 - e)),
    e the exponent field of the largest scale that the row sees: below fp16's
    normal range it is off by at most 2^-25, so the token's part by
    2^-25 * code * 2^(e - 133) <= 2^-31 * largest code * largest scale; the token
    of the largest scale has an element of that size (INT8, E4M3) or of half of
    it (INT4: one of 15 units' ends is 7.5 or more from zero).  The sum of the
    probabilities that divides it is 1 at least."""
    O, lse, tol, ltol = R.attention(p, Q, n_rows, scale, causal, window)
    T, H, D = Q.shape
    G = H // p.Hk
    u = torch.finfo(Q.dtype).eps / 2
    t = 0
    for b, n in enumerate(n_rows):
        L = p.lens[b]
        k, v = (torch.from_numpy(R.values(*p.rows(i, b), p.fmt)) for i in range(2))
        q = Q[t:t + n].double()
        pos, col = torch.arange(L - n, L)[:, None], torch.arange(L)[None, :]
        seen = torch.ones((n, L), dtype=torch.bool)
        if causal:
            seen = col <= pos
            if window:
                seen &= col > pos - window
        for h in range(H):
            s = torch.where(seen, (q[:, h] @ k[:, h // G].T) * scale, -torch.inf)
            w = torch.softmax(s, -1)
            va = v[:, h // G].abs()
            sa = torch.where(seen, (q[:, h].abs() @ k[:, h // G].abs().T) * abs(scale), torch.zeros_like(s))
            smax = sa.amax(-1)
            d = 2 * (smax * (D + 8) * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -23 * smax * 1.4427) + (L + 8) * 2.0 ** -23
            vmax = torch.where(seen, va.amax(-1)[None, :], 0).amax(-1)
            lost = seen.sum(-1) * 2.0 ** (-30 if p.fmt == R.INT4 else -31) * vmax
            tol[t:t + n, h] = u * O[t:t + n, h].abs() + (1 + u) * (w @ va) * (2.0 ** -11 + d[:, None]) + lost[:, None]
        t += n
    return O, lse, tol, ltol


# (rows, query heads of two key/value heads): the row kernel's tiles of 8 and 16, several of
# those, one split row tile, two row tiles, several items
SHAPES = [(3, 2), (6, 4), (20, 4), (40, 4), (100, 4), (300, 4)]
COPIES = (1, 50)
UNSEEN = [(399, 0), (398, 0), (10, 64), (250, 100)]  # position of a token, window


def shared(p, n, copies):
    """The batch of `copies` sequences in the pages of one, so that a block walks several steps."""
    return (torch.from_numpy(p.table.repeat(copies, 0)).cuda(),
            torch.full((copies,), p.lens[0], dtype=torch.int32, device="cuda"),
            torch.arange(copies + 1, dtype=torch.int32, device="cuda") * n)


def close_copies(O, lse, want, copies):
    n = O.shape[0] // copies
    for i in range(copies):
        close(O[i * n:(i + 1) * n], lse[i * n:(i + 1) * n], want, f"copy {i}")


def token_rows(L, n, at, window):
    pos = torch.arange(L - n, L)
    return (pos >= at) & (pos - (window or L + 1) < at)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("n,H", SHAPES)
@pytest.mark.parametrize("copies", COPIES)
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_unseen_sizes(w4, fmt, copies, n, H, dtype):
    """A token with a key or a value of 1e30 leaves the rows that do not see it
    as they were, bit for bit."""
    L, D = 400, 64
    p = R.Plain([L], fmt, 2, D, 16, 1)
    Q = rows((n * copies, H, D), dtype, 2).cuda()
    batch = shared(p, n, copies)
    r = np.random.default_rng(5)
    for at, window in UNSEEN:
        want = w4.w4kv_attention(Q, p.device(w4), *batch, max_rows=n, window=window)
        sees = token_rows(L, n, at, window).cuda().repeat(copies)
        pg, off = (int(x) for x in p.at(0, at))
        for which in range(2):
            bad = p.device(w4)
            code, word = R.quantize((r.standard_normal((1, D)) * 1e30).astype(np.float32), fmt)
            c, s = ((bad.k_codes, bad.k_scales), (bad.v_codes, bad.v_scales))[which]
            c[pg, 0, off] = torch.from_numpy(code[0]).cuda()
            s[pg, 0, off] = float(word.view(np.float32)[0])
            got = w4.w4kv_attention(Q, bad, *batch, max_rows=n, window=window)
            assert torch.equal(got[:, H // 2:], want[:, H // 2:])
            assert torch.equal(got[~sees], want[~sees]), (at, window, which)


@pytest.mark.parametrize("copies", COPIES)
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("n,H", SHAPES)
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_value_sizes_per_row(w4, fmt, n, H, window, copies):
    """Values from 1e-12 to 1e12, growing along the sequence and at random:
    each row within the tolerance of what it sees itself."""
    L, D = 400, 64
    r = np.random.default_rng(3)
    for sizes in (np.linspace(-12, 12, L), np.linspace(12, -12, L), r.uniform(-12, 12, L)):
        p = R.Plain([L], fmt, 2, D, 16, 1, dtype=torch.bfloat16)
        v = r.standard_normal((L, 2, D)) * 10.0 ** sizes[:, None, None]
        p.store(1, 0, 0, *R.quantize(v.astype(np.float32), fmt))
        Q = rows((n, H, D), torch.bfloat16, 2)
        O, lse = w4.w4kv_attention(Q.cuda().repeat(copies, 1, 1), p.device(w4), *shared(p, n, copies),
                                   max_rows=n, window=window, return_lse=True)
        close_copies(O, lse, row_tolerance(p, Q, [n], D ** -0.5, True, window), copies)


@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("n,H", [(1, 2), (1, 16)] + SHAPES)
def test_nan_codes(w4, n, H, dtype, D):
    """E4M3's NaN codes: in a value they make that element of the rows that see
    it NaN, in a key all of those rows, and nothing else changes."""
    L = 400
    p = R.Plain([L], R.E4M3, 2, D, 16, 1)
    Q = rows((n, H, D), dtype, 2).cuda()
    batch = p.batch([n])
    for at, window in UNSEEN + [(L - n // 2 - 1, 0), (3, 0), (L - 1, 1), (L - n, 5)]:
        want = w4.w4kv_attention(Q, p.device(w4), *batch, window=window)
        sees = token_rows(L, n, at, window).cuda()
        pg, off = (int(x) for x in p.at(0, at))
        for dim, code in ((0, 0x7F), (D - 1, 0xFF), (D // 2 + 5, 0x7F)):
            bad = p.device(w4)
            bad.v_codes[pg, 0, off, dim] = code
            got = w4.w4kv_attention(Q, bad, *batch, window=window)
            assert torch.equal(got[~sees], want[~sees]), (at, window, dim)
            assert torch.isnan(got[sees, :H // 2, dim]).all(), (at, window, dim)
            got[sees, :H // 2, dim] = want[sees, :H // 2, dim]
            assert torch.equal(got, want), (at, window, dim)
        bad = p.device(w4)
        bad.k_codes[pg, 0, off, 7] = 0x7F
        got = w4.w4kv_attention(Q, bad, *batch, window=window)
        assert torch.isnan(got[sees, :H // 2]).all()
        got[sees, :H // 2] = want[sees, :H // 2]
        assert torch.equal(got, want), (at, window)


def test_nan_codes_in_long_and_cut_items(w4):
    """NaN codes in many places of a long sequence whose items several blocks share."""
    L, D, n, H = 3000, 128, 300, 2
    p = R.Plain([L] * 12, R.E4M3, 1, D, 16, 1)
    Q = rows((12 * n, H, D), torch.bfloat16, 2).cuda()
    batch = p.batch([n] * 12)
    r = np.random.default_rng(1)
    for window in (0, 200, 1000):
        want = w4.w4kv_attention(Q, p.device(w4), *batch, max_rows=n, window=window)
        bad = p.device(w4)
        nan = torch.zeros((12 * n, D), dtype=torch.bool)
        for at in list(r.integers(2600, L, 40)) + list(r.integers(1500, 2600, 10)):
            b, dim = int(r.integers(12)), int(r.integers(D))
            pg, off = (int(x) for x in p.at(b, int(at)))
            bad.v_codes[pg, 0, off, dim] = 0xFF
            nan[b * n:(b + 1) * n, dim] |= token_rows(L, n, int(at), window)
        got = w4.w4kv_attention(Q, bad, *batch, max_rows=n, window=window)
        nan = nan[:, None].expand(12 * n, H, D).cuda()
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("n,H", [(9, 22), (16, 16), (5, 16), (40, 22)])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_unseen_sizes_beside_wide_values(w4, fmt, n, H, D):
    """As test_unseen_sizes, where most weights are below fp16's normal range, so
    that any other reference of the value scales shows."""
    L, copies = 400, 30
    for seed in range(6):
        r = np.random.default_rng(seed)
        p = R.Plain([L], fmt, 2, D, 16, seed, dtype=torch.bfloat16)
        v = r.standard_normal((L, 2, D)) * 10.0 ** r.uniform(-5, 5, (L, 1, 1))
        p.store(1, 0, 0, *R.quantize(v.astype(np.float32), fmt))
        Q = rows((n * copies, H, D), torch.bfloat16, seed, 2.0).cuda()
        batch = shared(p, n, copies)
        want = w4.w4kv_attention(Q, p.device(w4), *batch, max_rows=n)
        for at in (L - n + 1, L - n // 2, L - 1):
            sees = token_rows(L, n, at, 0).cuda().repeat(copies)
            pg, off = (int(x) for x in p.at(0, at))
            bad = p.device(w4)
            bad.v_scales[pg, 0, off] = 1e30
            got = w4.w4kv_attention(Q, bad, *batch, max_rows=n)
            assert torch.equal(got[~sees], want[~sees]), (seed, at)


# ---- scores far below zero --------------------------------------------------------------------

@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("n,H,L", [(1, 2, 1), (1, 2, 300), (5, 8, 40), (90, 2, 200), (150, 4, 300)])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_scores_below_any_reference(w4, fmt, n, H, L, D):
    """Keys of 1e33, all alike and against the queries: the rows see their
    tokens, and weigh them alike."""
    p = R.Plain([L], fmt, 1, D, 16, 1, dtype=torch.bfloat16)
    key = np.full((L, 1, D), -1e33, np.float32)
    p.store(0, 0, 0, *R.quantize(key, fmt))
    Q = torch.ones((n, H, D), dtype=torch.bfloat16)
    O, lse = w4.w4kv_attention(Q.cuda(), p.device(w4), *p.batch([n]), return_lse=True)
    k = R.values(*p.rows(0, 0, 0, 1), fmt)[0, 0]
    v = torch.from_numpy(R.values(*p.rows(1, 0), fmt))[:, 0]
    u = 2.0 ** -8
    for i in range(n):
        seen = v[:L - n + i + 1]
        mean, size = seen.mean(0), seen.abs().mean(0)
        tol = u * mean.abs() + (1 + u) * size * (2.0 ** -11 + (L + 8) * 2.0 ** -23 + 2.0 ** -20)
        assert ((O[i].cpu().double() - mean).abs() <= tol + L * 2.0 ** -30 * seen.abs().max()).all()
    assert ((lse.cpu().double() / (k.sum() * D ** -0.5) - 1).abs() <= (D + 16) * 2.0 ** -23).all()


@pytest.mark.parametrize("size", [3e3, 1e5, 1e8, 1e20, 1e33])
@pytest.mark.parametrize("n,H", [(3, 2), (20, 4), (40, 4), (300, 4)])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_first_tokens_of_no_weight(w4, fmt, n, H, size):
    """Many first tokens with scores far below the others: they weigh nothing,
    and the others as if they were alone."""
    L, D, far = 900, 64, 500
    p = R.Plain([L], fmt, 2, D, 16, 1, dtype=torch.bfloat16)
    Q = rows((n, H, D), torch.bfloat16, 2)
    Q[..., :8] = Q[..., :8].abs() + 0.5
    key = np.zeros((far, 2, D), np.float32)
    key[..., :8] = -size
    p.store(0, 0, 0, *R.quantize(key, fmt))
    for copies in COPIES:
        O, lse = w4.w4kv_attention(Q.cuda().repeat(copies, 1, 1), p.device(w4), *shared(p, n, copies),
                                   max_rows=n, return_lse=True)
        close_copies(O, lse, R.attention(p, Q, [n], D ** -0.5, unseen=[(0, j) for j in range(far)]), copies)


# ---- windows that reach beyond every position ---------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 20, 2 ** 31, 2 ** 40])
@pytest.mark.parametrize("n", [3, 40, 150])
def test_windows_of_31_bits(w4, n, window):
    """The longest windows are none, for rows before the first position too."""
    p = R.Plain([2, n - 1, 200], R.INT8, 1, 64, 16, 1)
    Q = rows((3 * n, 2, 64), torch.float16, 3).cuda()
    batch = p.batch([n, n, n])
    want = w4.w4kv_attention(Q, p.device(w4), *batch)
    assert torch.equal(w4.w4kv_attention(Q, p.device(w4), *batch, window=window), want)


@pytest.mark.parametrize("near", [-200.0, 0.0, 100.0, 250.0])
@pytest.mark.parametrize("apart", [100, 128, 150, 300, 600, 1000, 1100])
@pytest.mark.parametrize("n,H", [(40, 4), (300, 4)])
def test_first_tokens_at_middle_distances(w4, n, H, apart, near):
    """As above where the distance leaves nothing of the first tokens (2^-126 and
    less), around the longest that the maximum moves by, with scores of any size."""
    L, D, far = 900, 64, 500
    p = R.Plain([L], R.INT8, 2, D, 16, 1, dtype=torch.bfloat16)
    Q = rows((n, H, D), torch.bfloat16, 2)
    Q[..., :8] = 1.0
    unit = 1 / (8 * D ** -0.5 * 1.4427)  # in the first 8 elements of a key: a score of 1 in base 2
    key = p.kv[0][0].copy()
    key[:, :, :8] = near * unit
    key[:far, :, 8:] = 0
    key[:far, :, :8] -= apart * unit
    p.store(0, 0, 0, *R.quantize(key, R.INT8))
    for copies in COPIES:
        O, lse = w4.w4kv_attention(Q.cuda().repeat(copies, 1, 1), p.device(w4), *shared(p, n, copies),
                                   max_rows=n, return_lse=True)
        close_copies(O, lse, R.attention(p, Q, [n], D ** -0.5, unseen=[(0, j) for j in range(far)]), copies)


@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("up", [12, 18, 22])
@pytest.mark.parametrize("n,H", [(3, 2), (40, 4), (300, 4)])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_weights_before_a_long_move(w4, fmt, n, H, up, D):
    """A token that weighs 2^-up of a later one of the same 128 keeps its part
    where the maximum moves by more than that, past fp16's range."""
    L = 900
    p = R.Plain([L], fmt, 2, D, 16, 1, dtype=torch.bfloat16)
    Q = rows((n, H, D), torch.bfloat16, 2)
    Q[..., :8] = 1.0
    unit = 1 / (8 * D ** -0.5 * 1.4427)  # in the first 8 elements of a key: a score of 1 in base 2
    key = np.zeros((L, 2, D), np.float32)
    key[600, :, :8] = 7 * unit
    key[630, :, :8] = (7 + up) * unit
    p.store(0, 0, 0, *R.quantize(key, fmt))
    value = np.zeros((L, 2, D), np.float32)
    value[600] = 1000 * np.random.default_rng(1).standard_normal((2, D))
    p.store(1, 0, 0, *R.quantize(value, fmt))
    for copies in COPIES:
        O, lse = w4.w4kv_attention(Q.cuda().repeat(copies, 1, 1), p.device(w4), *shared(p, n, copies),
                                   max_rows=n, return_lse=True)
        close_copies(O, lse, row_tolerance(p, Q, [n], D ** -0.5), copies)
