"""Plain reference of the quantized paged key/value cache, in numpy / torch
float64 on the CPU: row formats (include/w4kv.h), page lookup and attention.
Shares no code with the CUDA library.

Tolerance of the attention output, per element, u = eps / 2 of the output type:

    |O - O_ref| <= u * |O_ref|                               output rounding
                 + (1 + u) * A * (2^-11 + d)                 weights
                 + n * 2^-32 * vmax                          weights below fp16's range

A = sum_j p_j |v_j| (p normalized): every weight p_j * scale_j is rounded to
fp16 (half a step, 2^-11), and carries the error d of its probability,
numerator and denominator together:
    d = 2 * (smax * (D + 8) * 2^-24 + 2^-22 + 2^-24 * tmax) + (n + 8) * 2^-24
with smax = max_j scale * sum_d |q_d k_jd| (fp32 products and sums of D terms
plus the scale factors; the factor 2 for the sum's terms), tmax = the largest
|score| in base-2 units (rounding of the exponent's argument), 2^-22 for exp2,
(n + 8) * 2^-24 for the sums over n tokens.  Tensor cores may cut instead of
round a sum: the terms with 2^-24 are doubled.  The last term: a weight is
held relative to the largest value scale with 21 bits of range above fp16's
smallest normal number, so one below loses at most 2^-32 of it; vmax is the
largest |v|.  Queries enter as fp16 with their row scaled: elements below 2^-14
of the row's largest carry at most 2^-25 of it, inside (D + 8) * 2^-24 of smax
for the rows tested here (none has nearly all its weight in one element).
"""
from __future__ import annotations

import numpy as np
import torch

INT8, E4M3, INT4 = 0, 1, 2
FORMATS = (INT8, E4M3, INT4)
NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)


def e4m3_table() -> np.ndarray:
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e > 0, (1 + f / 8.0) * 2.0 ** (e - 7.0), f / 8.0 * 2.0 ** -6)
    t = np.where(c > 127, -mag, mag)
    t[(c & 127) == 127] = np.nan
    return t


def quantize(x: np.ndarray, fmt: int):
    """x float32 [..., D] -> (codes uint8 [..., row bytes], words uint32 [...])."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], np.float32(0), x)
    if fmt == INT4:
        with np.errstate(over="ignore"):
            lo, hi = np.minimum(x.min(-1), np.float32(0)), np.maximum(x.max(-1), np.float32(0))
            rng = hi - lo
        bad = bad | ~np.isfinite(rng)
        rng = np.where(bad, np.float32(0), rng)
        sb = ((rng / np.float32(15)).astype(np.float32).view(np.uint32) + 8) & ~np.uint32(15)
        s = sb.view(np.float32)
        ok = (s != 0) & ~bad
        safe = np.where(ok, s, np.float32(1))
        z = np.where(ok, np.rint(-lo / safe), np.float32(0)).astype(np.float32)
        u = np.rint((x / safe[..., None]).astype(np.float32) + z[..., None])
        u = np.where(ok[..., None], np.clip(u, 0, 15), 0).astype(np.uint32)
        u = u.reshape(u.shape[:-1] + (u.shape[-1] // 8, 8))
        w = np.zeros(u.shape[:-1], np.uint32)
        for i, k in enumerate(NIBBLE):
            w |= u[..., k] << np.uint32(4 * i)
        code = np.ascontiguousarray(w).astype("<u4").view(np.uint8)
        word = np.where(ok, sb | z.astype(np.uint32), np.uint32(0))
    else:
        amax = np.abs(x).max(-1)
        s = (amax / np.float32(127 if fmt == INT8 else 448)).astype(np.float32)
        ok = (s != 0) & ~bad
        y = (x / np.where(ok, s, np.float32(1))[..., None]).astype(np.float32)
        y = np.where(ok[..., None], y, np.float32(0))
        if fmt == INT8:
            code = np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
        else:
            a = np.minimum(np.abs(y).astype(np.float64), 448)
            _, e = np.frexp(a)
            step = np.ldexp(1.0, np.maximum(e, -5) - 4)
            v = np.minimum(np.rint(a / step) * step, 448)
            pos = e4m3_table()[:127]
            code = np.searchsorted(pos, v).astype(np.uint8)
            assert np.array_equal(pos[code], v)
            code = code | np.where(np.signbit(y), np.uint8(128), np.uint8(0))
        word = np.where(ok, s.view(np.uint32), np.uint32(0))
    word = np.where(bad, np.uint32(0x7FC00000), word).astype(np.uint32)
    return code, word


def values(code: np.ndarray, word: np.ndarray, fmt: int) -> np.ndarray:
    """float64 [..., D]: what the codes and scale words stand for."""
    if fmt == INT4:
        w = np.ascontiguousarray(code).view("<u4")
        u = np.stack([(w >> np.uint32(4 * NIBBLE.index(k))) & 15 for k in range(8)], -1)
        u = u.reshape(u.shape[:-2] + (u.shape[-2] * 8,)).astype(np.float64)
        s = (word & ~np.uint32(15)).view(np.float32).astype(np.float64)
        return (u - (word & np.uint32(15))[..., None]) * s[..., None]
    q = code.view(np.int8).astype(np.float64) if fmt == INT8 else e4m3_table()[code]
    return q * word.view(np.float32).astype(np.float64)[..., None]


def read16(code, word, fmt, dtype: torch.dtype) -> torch.Tensor:
    """fl16(fl32(q * s)) as w4kv_read gives it."""
    v = values(code, word, fmt)
    with np.errstate(over="ignore", invalid="ignore"):
        return torch.from_numpy(v.astype(np.float32)).to(dtype)


class Plain:
    """A cache on the host with its page table; the device copies are made by `to`."""

    def __init__(self, lens, fmt, Hk, D, page, seed, spare=2, dtype=torch.float16, width=None):
        r = np.random.default_rng(seed)
        self.lens, self.fmt, self.Hk, self.D, self.page = list(lens), fmt, Hk, D, page
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = r.permutation(self.pages)
        width = max([1] + need) if width is None else width
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        rb = D // 2 if fmt == INT4 else D
        # what no row fills is garbage: every byte, NaN codes and scales among it
        shape = (self.pages, Hk, page)
        self.codes = [r.integers(0, 256, shape + (rb,), dtype=np.uint8) for _ in range(2)]
        self.words = [np.full(shape, 0x7FC00001, np.uint32) for _ in range(2)]
        self.kv = [[], []]
        for b, n in enumerate(lens):
            for i in range(2):
                x = r.standard_normal((n, Hk, D)) * np.exp(0.5 * r.standard_normal((n, Hk, 1)))
                x = torch.from_numpy(x).to(dtype).float().numpy()
                self.kv[i].append(x)
                self.store(i, b, 0, *quantize(x, fmt))
        self.rng = r

    def at(self, b, pos):
        pos = np.asarray(pos)
        return self.table[b, pos // self.page], pos % self.page

    def store(self, i, b, start, code, word):
        pg, off = self.at(b, np.arange(start, start + code.shape[0]))
        self.codes[i][pg, :, off] = code
        self.words[i][pg, :, off] = word

    def rows(self, i, b, lo=0, hi=None):
        pg, off = self.at(b, np.arange(lo, self.lens[b] if hi is None else hi))
        return self.codes[i][pg, :, off], self.words[i][pg, :, off]

    def device(self, w4, dev="cuda"):
        t = [torch.from_numpy(c.copy()).to(dev) for c in self.codes]
        s = [torch.from_numpy(w.view(np.float32).copy()).to(dev) for w in self.words]
        return w4.W4KVCache(t[0], s[0], t[1], s[1], self.fmt)

    def batch(self, n_rows, dev="cuda"):
        cu = np.concatenate([[0], np.cumsum(n_rows)]).astype(np.int32)
        return (torch.from_numpy(self.table.copy()).to(dev),
                torch.tensor(self.lens, dtype=torch.int32, device=dev),
                torch.from_numpy(cu).to(dev))


def attention(p: Plain, Q: torch.Tensor, n_rows, scale, causal=True, window=0, unseen=()):
    """(O, lse, tolerance of O, tolerance of lse) in float64 for Q [T][H][D];
    `unseen` lists (sequence, position) pairs that count as unseen.  lse
    carries the error d of a score and of the sum, and its own rounding."""
    T, H, D = Q.shape
    G = H // p.Hk
    O = torch.full((T, H, D), float("nan"), dtype=torch.float64)
    tol = torch.full((T, H, D), float("nan"), dtype=torch.float64)
    lse = torch.full((T, H), float("nan"), dtype=torch.float64)
    ltol = torch.zeros((T, H), dtype=torch.float64)
    u = torch.finfo(Q.dtype).eps / 2
    t = 0
    for b, n in enumerate(n_rows):
        L = p.lens[b]
        k, v = (torch.from_numpy(values(*p.rows(i, b), p.fmt)) for i in range(2))
        q = Q[t:t + n].double().cpu()
        pos = torch.arange(L - n, L)[:, None]
        col = torch.arange(L)[None, :]
        seen = torch.ones((n, L), dtype=torch.bool)
        if causal:
            seen = col <= pos
            if window:
                seen &= col > pos - window
        for bb, j in unseen:
            if bb == b:
                seen[:, j] = False
        for h in range(H):
            kh, vh = k[:, h // G], v[:, h // G]
            s = (q[:, h] @ kh.T) * scale
            s = torch.where(seen, s, torch.full_like(s, -torch.inf))
            norm = torch.logsumexp(s, -1) if L else torch.full((n,), -torch.inf, dtype=torch.float64)
            w = torch.exp(s - torch.where(torch.isinf(norm), torch.zeros_like(norm), norm)[:, None])
            w = torch.where(seen, w, torch.zeros_like(w))
            vz = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))
            O[t:t + n, h] = w @ vz
            lse[t:t + n, h] = norm
            if L == 0:
                tol[t:t + n, h] = 0
                continue
            sa = torch.where(seen, (q[:, h].abs() @ kh.abs().T) * abs(scale), torch.zeros_like(s))
            smax = sa.amax(-1)
            d = 2 * (smax * (D + 8) * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -23 * smax * 1.4427) + \
                (L + 8) * 2.0 ** -23
            ltol[t:t + n, h] = d + 2.0 ** -22 * torch.nan_to_num(norm.abs(), posinf=0.0)
            A = w @ vz.abs()
            tol[t:t + n, h] = u * O[t:t + n, h].abs() + (1 + u) * A * (2.0 ** -11 + d[:, None]) + \
                L * 2.0 ** -32 * vz.abs().amax()
        t += n
    return O, lse, tol, ltol
