"""The quantized paged key/value cache: what its three operators compute, on
which sizes they are measured, and their plain forms.

A cache holds keys and values of many sequences in pages of `page` tokens.  A
row (one token of one key/value head, `dim` numbers) is kept in 8 or 4 bits
with one 32-bit scale word:

    int8   s = fl32(amax / 127),  q = clamp(rne(fl32(x / s)), -127, 127)
    e4m3   s = fl32(amax / 448),  q = the nearest E4M3 value of fl32(x / s)
    int4   lo = min(x, 0), hi = max(x, 0), s = fl32(fl32(hi - lo) / 15) rounded
           to a multiple of 16 of its own last places (ties up), the zero point
           z = rne(fl32(-lo / s)) in the four bits this frees,
           u = clamp(rne(fl32(fl32(x / s) + z)), 0, 15)

and stands for q * s, or (u - z) * s.  s = 0 stores zeros.  Codes are laid out
[pages][kv heads][page][dim bytes, or dim / 2 for int4], scale words
[pages][kv heads][page]; eight int4 codes k = 8j.. form the little-endian word
j whose nibble i holds k = 8j + (0, 2, 4, 6, 1, 3, 5, 7)[i].

Sequence b of a batch has kv_lens[b] tokens in the pages that row b of the
page table lists; the rows cu_rows[b] .. cu_rows[b + 1] of a call are its last
tokens.

    append   quantizes the call's keys and values into the pages; the pass
             reads the same rows back, as a program does that carries on with
             the values the cache stands for
    read     the values of whole sequences, rounded once to 16 bits
    attend   out = softmax(scale * q k^T) v of the call's query rows over the
             cached rows of their sequence, each row seeing the positions up to
             its own (or all), the last `window` of them where one is given;
             query head h reads key/value head h // (heads / kv_heads)
"""
import math
import random

import torch

own = False

FORMATS = ("int8", "e4m3", "int4")
NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)


def listed():
    return [
        # one decode step of a busy server: a token of each of 64 sequences
        dict(name="append, decode step of 64, int8", op="append", fmt="int8", dtype="fp16", heads=64,
             kv_heads=8, dim=128, page=16, batch=64, rows=1, rows_min=1, context=1000,
             context_min=1, fused=False, seed=1),
        # a prompt's chunk, keys and values as slices of the fused projection's output
        dict(name="append, chunk of 2048, int4", op="append", fmt="int4", dtype="bf16", heads=32,
             kv_heads=32, dim=128, page=64, batch=1, rows=2048, rows_min=2048, context=4096,
             context_min=4096, fused=True, seed=2),
        # several prompts of odd lengths at once
        dict(name="append, 16 prompts to 1021, e4m3", op="append", fmt="e4m3", dtype="bf16", heads=64,
             kv_heads=8, dim=128, page=32, batch=16, rows=1021, rows_min=17, context=1021,
             context_min=1021, fused=True, seed=3),
        # a short prefix taken out of the cache
        dict(name="read, one prefix of 129, int4", op="read", fmt="int4", dtype="fp16", heads=32,
             kv_heads=32, dim=128, page=16, batch=1, rows=129, rows_min=129, context=129,
             context_min=129, fused=False, seed=4),
        # sequences moved out of the cache, e.g. to another machine
        dict(name="read, 12 sequences to 8192, int8", op="read", fmt="int8", dtype="bf16", heads=64,
             kv_heads=8, dim=128, page=64, batch=12, rows=8192, rows_min=100, context=8192,
             context_min=8192, fused=False, seed=5),
        # a chat with one user: latency counts
        dict(name="attend, decode of 1 at 1000, int8", op="attend", fmt="int8", dtype="fp16", heads=32,
             kv_heads=32, dim=128, page=16, batch=1, rows=1, rows_min=1, context=1000,
             context_min=1000, causal=True, window=0, lse=False, seed=6),
        # ordinary serving of a model with as many key heads as query heads
        dict(name="attend, decode of 32 to 4096, int4", op="attend", fmt="int4", dtype="fp16",
             heads=32, kv_heads=32, dim=128, page=16, batch=32, rows=1, rows_min=1, context=4096,
             context_min=65, causal=True, window=0, lse=False, seed=7),
        # long contexts, grouped heads
        dict(name="attend, decode of 64 to 16384, e4m3", op="attend", fmt="e4m3", dtype="bf16",
             heads=64, kv_heads=8, dim=128, page=64, batch=64, rows=1, rows_min=1, context=16384,
             context_min=300, causal=True, window=0, lse=True, seed=8),
        # proposals of a draft model checked at once
        dict(name="attend, 5 proposals of 16 to 8000, int8", op="attend", fmt="int8", dtype="bf16",
             heads=64, kv_heads=8, dim=128, page=32, batch=16, rows=5, rows_min=1, context=8000,
             context_min=500, causal=True, window=0, lse=False, seed=9),
        # a prompt's chunk in the middle of a document
        dict(name="attend, chunk of 509 at 4096, int8", op="attend", fmt="int8", dtype="fp16",
             heads=32, kv_heads=32, dim=128, page=16, batch=1, rows=509, rows_min=509, context=4096,
             context_min=4096, causal=True, window=0, lse=False, seed=10),
        # the last chunk of a long document
        dict(name="attend, chunk of 2048 at 16384, e4m3", op="attend", fmt="e4m3", dtype="bf16",
             heads=64, kv_heads=8, dim=128, page=64, batch=1, rows=2048, rows_min=2048,
             context=16384, context_min=16384, causal=True, window=0, lse=False, seed=11),
        # chunks and single tokens in one batch, sliding window, small heads, an odd page
        dict(name="attend, mixed 24 to 300, window, int4", op="attend", fmt="int4", dtype="fp16",
             heads=28, kv_heads=4, dim=64, page=48, batch=24, rows=300, rows_min=1, context=3000,
             context_min=300, causal=True, window=1024, lse=True, seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    limit = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("append", "read", "attend", "attend", "attend"))
        c = dict(op=op, fmt=rng.choice(FORMATS), dtype=rng.choice(("fp16", "bf16")),
                 dim=rng.choice((64, 128, 128)), page=rng.choice((16, 32, 48, 64, 128, 256)),
                 kv_heads=rng.choice((1, 2, 4, 8, 8, 16, 32)), seed=rng.randrange(1 << 30))
        c["heads"] = c["kv_heads"] * rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 16))
        if c["heads"] > 64:
            continue
        c["context"] = _log(rng, 1, 16384)
        if op == "attend":
            shape = rng.choice(("decode", "decode", "proposals", "chunk", "mixed"))
            if shape == "decode":
                c["rows"], c["batch"] = 1, _log(rng, 1, 64)
            elif shape == "proposals":
                c["rows"], c["batch"] = rng.randint(2, 16), _log(rng, 1, 32)
            elif shape == "chunk":
                c["rows"], c["batch"] = _log(rng, 17, 2048), _log(rng, 1, 4)
            else:
                c["rows"], c["batch"] = _log(rng, 17, 512), _log(rng, 2, 32)
            c["rows_min"] = 1 if shape in ("mixed", "proposals") else c["rows"]
            c["causal"] = rng.random() < 0.85
            c["window"] = _log(rng, 16, 4096) if c["causal"] and rng.random() < 0.2 else 0
            c["lse"] = rng.random() < 0.3
        else:
            c["rows"], c["batch"] = _log(rng, 1, 8192), _log(rng, 1, 32)
            c["rows_min"] = rng.choice((1, c["rows"]))
            c["fused"] = op == "append" and rng.random() < 0.5
        c["context"] = max(c["context"], c["rows"])
        c["context_min"] = rng.randint(1, c["context"])
        w = work(c)
        if _cost(c) <= limit and w["bytes"] <= 2e9:
            return c


def _lengths(case):
    """(rows of the call, cached length) of each sequence."""
    rng = random.Random(case["seed"])
    out = []
    for _ in range(case["batch"]):
        n = rng.randint(case["rows_min"], case["rows"])
        out.append((n, max(n, rng.randint(case["context_min"], case["context"]))))
    if case["op"] == "read":  # whole sequences
        out = [(n, n) for n, _ in out]
    return out


def _visible(case, n, length):
    """Positions that the n rows of a sequence see, summed over the rows, and
    the cached positions that any of them sees."""
    if not case["causal"]:
        return n * length, length
    first = length - n  # position of the first row
    pairs, lo = 0, 0
    w = case["window"]
    if w:
        pairs = sum(min(first + i + 1, w) for i in range(n))
        lo = max(0, first + 1 - w)
    else:
        pairs = n * first + n * (n + 1) // 2
    return pairs, length - lo


def _row_bytes(case):
    return (case["dim"] // 2 if case["fmt"] == "int4" else case["dim"]) + 4


def work(case):
    lens = _lengths(case)
    total = sum(n for n, _ in lens)
    D, H, Hk = case["dim"], case["heads"], case["kv_heads"]
    meta = 4 * (2 * len(lens) + 1)
    if case["op"] == "attend":
        pairs = seen = pages = 0
        for n, length in lens:
            p, s = _visible(case, n, length)
            pairs, seen = pairs + p, seen + s
            pages += -(-s // case["page"])
        nbytes = 2 * seen * Hk * _row_bytes(case) + 2 * total * H * D * 2 + meta + 4 * pages
        if case["lse"]:
            nbytes += 4 * total * H
        return {"bytes": nbytes, "flops": 4 * D * H * pairs}
    rows = 2 * total * Hk
    meta += 4 * sum(-(-n // case["page"]) for n, _ in lens)
    if case["op"] == "append":  # 16-bit rows in, codes and scales out; then read back
        return {"bytes": rows * (2 * D + 2 * _row_bytes(case) + 2 * D) + 2 * meta,
                "flops": rows * D * 5}
    return {"bytes": rows * (_row_bytes(case) + 2 * D) + meta, "flops": rows * D}


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.6e15)


# ---- plain forms ------------------------------------------------------------------------------

def _quantize(x, fmt):
    """x [..., dim] float32 -> (code bytes, scale words)."""
    if fmt == "int4":
        lo = x.amin(-1).clamp(max=0.0)
        hi = x.amax(-1).clamp(min=0.0)
        # (a tensor as divisor: torch divides by a number through its reciprocal)
        bits = ((hi - lo) / torch.full_like(hi, 15.0)).view(torch.int32)
        s = ((bits + 8) & ~15).view(torch.float32)
        safe = torch.where(s == 0, torch.ones_like(s), s)
        z = torch.where(s == 0, torch.zeros_like(s), torch.round(-lo / safe).clamp(0, 15))
        u = torch.round(x / safe[..., None] + z[..., None]).clamp(0, 15)
        u = torch.where(s[..., None] == 0, torch.zeros_like(u), u).to(torch.uint8)
        u = u.unflatten(-1, (-1, 8))[..., NIBBLE].unflatten(-1, (4, 2))
        code = (u[..., 0] | (u[..., 1] << 4)).flatten(-2)
        return code, (s.view(torch.int32) | z.to(torch.int32)).view(torch.float32)
    amax = x.abs().amax(-1)
    s = amax / torch.full_like(amax, 127.0 if fmt == "int8" else 448.0)
    safe = torch.where(s == 0, torch.ones_like(s), s)
    q = torch.where(s[..., None] == 0, torch.zeros_like(x), x / safe[..., None])
    if fmt == "int8":
        return torch.round(q).clamp(-127, 127).to(torch.int8).view(torch.uint8), s
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _values(code, scale, fmt):
    """(code bytes [..., row bytes], scale words [...]) -> float32 [..., dim]."""
    if fmt == "int8":
        return code.view(torch.int8).float() * scale[..., None]
    if fmt == "e4m3":
        return code.view(torch.float8_e4m3fn).float() * scale[..., None]
    bits = scale.view(torch.int32)
    z = (bits & 15).float()[..., None]
    s = (bits & ~15).view(torch.float32)[..., None]
    nib = torch.stack((code & 15, code >> 4), -1).flatten(-2).unflatten(-1, (-1, 8))
    back = [NIBBLE.index(k) for k in range(8)]
    return (nib[..., back].flatten(-2).float() - z) * s


def _rows_of(st, b, lo, hi):
    """Page and offset in the page of positions lo .. hi of sequence b."""
    pos = torch.arange(lo, hi, device=st["table"].device)
    return st["table"][b, pos // st["page"]].long(), pos % st["page"]


def _gather(st, which, b, lo, hi):
    """float32 [kv heads][hi - lo][dim] of one sequence."""
    first, last = lo // st["page"], -(-hi // st["page"])
    pages = st["table"][b, first:last].long()
    v = _values(st[which][pages], st[which + "_scales"][pages], st["fmt"])
    v = v.transpose(0, 1).flatten(1, 2)
    return v[:, lo - first * st["page"]:hi - first * st["page"]]


def _plain_append(st):
    for which, x in (("k", st["K"]), ("v", st["V"])):
        code, scale = _quantize(x.float(), st["fmt"])
        t = 0
        for b, (n, length) in enumerate(st["lens"]):
            page, off = _rows_of(st, b, length - n, length)
            st[which][page, :, off] = code[t:t + n]
            st[which + "_scales"][page, :, off] = scale[t:t + n]
            t += n


def _plain_read(st):
    out = []
    for which in ("k", "v"):
        parts = []
        for b, (n, length) in enumerate(st["lens"]):
            page, off = _rows_of(st, b, length - n, length)
            parts.append(_values(st[which][page, :, off], st[which + "_scales"][page, :, off],
                                 st["fmt"]))
        out.append(torch.cat(parts).to(st["dtype"]))
    return out


def _plain_attend(st):
    case = st["case"]
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    Q = st["Q"]
    out = torch.empty(Q.shape, dtype=Q.dtype, device=Q.device)
    lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device)
    t = 0
    for b, (n, length) in enumerate(st["lens"]):
        lo = length - _visible(case, n, length)[1]
        k, v = _gather(st, "k", b, lo, length), _gather(st, "v", b, lo, length)
        mask = None
        if case["causal"]:
            pos = torch.arange(length - n, length, device=Q.device)[:, None]
            col = torch.arange(lo, length, device=Q.device)[None, :]
            mask = col > pos
            if case["window"]:
                mask = mask | (col <= pos - case["window"])
        # as many key/value heads at a time as their scores take up to 2 GB
        step = max(1, int(5e8 // (n * (H // Hk) * (length - lo))))
        for h in range(0, Hk, step):
            e = min(Hk, h + step)
            q = Q[t:t + n, h * (H // Hk):e * (H // Hk)].float()
            q = q.reshape(n, e - h, H // Hk, D).permute(1, 2, 0, 3)  # [kv][group][n][D]
            s = torch.matmul(q, k[h:e, None].transpose(-1, -2)) * st["scale"]
            if mask is not None:
                s = s.masked_fill(mask, float("-inf"))
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v[h:e, None]) / total
            cols = slice(h * (H // Hk), e * (H // Hk))
            out[t:t + n, cols] = o.permute(2, 0, 1, 3).reshape(n, -1, D).to(Q.dtype)
            lse[t:t + n, cols] = (m + torch.log(total))[..., 0].permute(2, 0, 1).reshape(n, -1)
        t += n
    return [out, lse] if case["lse"] else [out]


# ---- state ------------------------------------------------------------------------------------

def _keys(shape, gen, dev):
    """Rows with a few strong channels per head, as rotated keys have them."""
    x = torch.randn(shape, generator=gen, device=dev)
    Hk, D = shape[-2:] if len(shape) == 3 else (shape[1], shape[3])
    strong = torch.rand((Hk, D), generator=gen, device=dev) < 4 / 128
    f = torch.where(strong, 8.0, 1.0)
    return x * (f if len(shape) == 3 else f[:, None])


def _vals(shape, gen, dev):
    """Rows whose size differs from token to token."""
    x = torch.randn(shape, generator=gen, device=dev)
    return x * torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens = _lengths(case)
    fmt, page, D, Hk = case["fmt"], case["page"], case["dim"], case["kv_heads"]
    dtype = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
    need = [-(-length // page) for _, length in lens]
    pages, width = sum(need) + 3, max(need)
    st = dict(case=case, lens=lens, fmt=fmt, page=page, dtype=dtype)
    # pages in any order, as an allocator that serves many requests gives them
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st["table"] = table
    st["kv_lens"] = torch.tensor([length for _, length in lens], dtype=torch.int32, device=dev)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    st["cu_rows"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["rows"], st["max_rows"] = cu[-1], max(n for n, _ in lens)
    width = D // 2 if fmt == "int4" else D
    for which, make in (("k", _keys), ("v", _vals)):
        st[which] = torch.empty((pages, Hk, page, width), dtype=torch.uint8, device=dev)
        st[which + "_scales"] = torch.empty((pages, Hk, page), dtype=torch.float32, device=dev)
        step = max(1, (1 << 27) // (Hk * page * D))
        for p in range(0, pages, step):
            e = min(pages, p + step)
            x = make((e - p, Hk, page, D), gen, dev).to(dtype).float()
            st[which][p:e], st[which + "_scales"][p:e] = _quantize(x, fmt)
    T, H = cu[-1], case["heads"]
    if case["op"] == "append":
        if case["fused"]:  # slices of one projection's output, [T][(heads + 2 kv heads) * dim]
            qkv = torch.randn((T, H + 2 * Hk, D), generator=gen, device=dev).to(dtype)
            qkv[:, H:H + Hk] = _keys((T, Hk, D), gen, dev).to(dtype)
            qkv[:, H + Hk:] = _vals((T, Hk, D), gen, dev).to(dtype)
            st["K"], st["V"] = qkv[:, H:H + Hk], qkv[:, H + Hk:]
        else:
            st["K"] = _keys((T, Hk, D), gen, dev).to(dtype)
            st["V"] = _vals((T, Hk, D), gen, dev).to(dtype)
    if case["op"] == "attend":
        st["Q"] = torch.randn((T, H, D), generator=gen, device=dev).to(dtype)
        st["scale"] = D ** -0.5
    return st


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import weight_only_int4_pack_b200 as w4
        if "cache" not in st:
            st["cache"] = w4.W4KVCache(st["k"], st["k_scales"], st["v"], st["v_scales"],
                                       {"int8": w4.W4KV_INT8, "e4m3": w4.W4KV_E4M3,
                                        "int4": w4.W4KV_INT4}[st["fmt"]])
        batch = (st["cache"], st["table"], st["kv_lens"], st["cu_rows"])
        if op == "attend":
            case = st["case"]
            r = w4.w4kv_attention(st["Q"], *batch, max_rows=st["max_rows"], scale=st["scale"],
                                  causal=case["causal"], window=case["window"],
                                  return_lse=case["lse"])
            return list(r) if case["lse"] else [r]
        if op == "append":
            w4.w4kv_append(st["K"], st["V"], *batch)
        out = list(w4.w4kv_read(*batch, st["rows"], dtype=st["dtype"]))
    elif op == "attend":
        return _plain_attend(st)
    else:
        if op == "append":
            _plain_append(st)
        out = _plain_read(st)
    return out + [st["k_scales"], st["v_scales"]] if op == "append" else out


# ---- the definition in 64 bits -----------------------------------------------------------------

def _f32(x):
    return x.to(torch.float32).to(torch.float64)


def _exact_rows(x, fmt):
    """(values, scale words) that rows x (float64) are kept as.  The definition
    rounds the scale and the quotients to 32 bits; with 53 bits in between
    that rounding of a quotient is the correct one."""
    if fmt == "int4":
        lo = torch.minimum(x.min(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
        hi = torch.maximum(x.max(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
        s = _f32(_f32(hi - lo) / 15)
        mant, exp = torch.frexp(s)                    # s = mant * 2^exp, 1/2 <= mant < 1
        unit = torch.ldexp(torch.ones_like(s), exp - 20)  # 16 of the 24 bits' last places
        s = torch.floor(s / unit + 0.5) * unit
        full = torch.where(s > 0, s, torch.ones_like(s))
        z = torch.round(_f32(-lo / full)) * (s > 0)
        u = torch.round(_f32(_f32(x / full[..., None]) + z[..., None])).clamp(0, 15)
        word = s + z * torch.ldexp(torch.ones_like(s), torch.frexp(full)[1] - 24) * (s > 0)
        return (u - z[..., None]) * s[..., None], word
    top = 127 if fmt == "int8" else 448
    s = _f32(x.abs().max(-1).values / top)
    full = torch.where(s > 0, s, torch.ones_like(s))
    y = _f32(x / full[..., None]) * (s > 0)[..., None]
    if fmt == "int8":
        q = torch.round(y).clamp(-127, 127)
    else:  # 3 fraction bits, smallest exponent -6
        step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp(min=-5) - 4)
        q = (torch.round(y / step) * step).clamp(-448, 448)
    return q * s[..., None], s


def _exact_values(code, scale, fmt):
    c = code.to(torch.int64)
    bits = scale.view(torch.int32).to(torch.int64)
    if fmt == "int4":
        word = sum(c[..., i::4] << (8 * i) for i in range(4))
        u = torch.stack([(word >> (4 * NIBBLE.index(k))) & 15 for k in range(8)], -1).flatten(-2)
        s = (bits & ~15).to(torch.int32).view(torch.float32).double()
        return (u - (bits & 15)[..., None]).double() * s[..., None]
    if fmt == "int8":
        q = torch.where(c > 127, c - 256, c).double()
    else:
        e, f = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(e > 0, torch.ldexp(1 + f / 8, e - 7), f / 8 * 2.0 ** -6)
        q = torch.where(c > 127, -mag, mag)
    return q * scale.double()[..., None]


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["table"].device
    if case["op"] == "append":
        out = []
        for which, x in (("k", st["K"]), ("v", st["V"])):
            val, word = _exact_rows(x.double(), case["fmt"])
            out.append((val, word))
        words = []
        for which, (_, word) in zip(("k", "v"), out):
            w = st[which + "_scales"].double()
            t = 0
            for b, (n, length) in enumerate(st["lens"]):
                for i in range(0, n, 1 << 16):
                    p = torch.arange(length - n + i, min(length, length - n + i + (1 << 16)),
                                     device=dev)
                    page = st["table"][b].long()[torch.div(p, case["page"], rounding_mode="floor")]
                    w[page, :, p.remainder(case["page"])] = word[t + i:t + i + p.numel()]
                t += n
            words.append(w)
        return [out[0][0], out[1][0]] + words
    if case["op"] == "read":
        out = []
        for which in ("k", "v"):
            parts = []
            for b, (n, length) in enumerate(st["lens"]):
                pages = st["table"][b, :-(-length // case["page"])].long()
                x = _exact_values(st[which][pages], st[which + "_scales"][pages], case["fmt"])
                x = x.permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["dim"])
                parts.append(x[length - n:length])
            out.append(torch.cat(parts))
        return out
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk
    O = torch.zeros((st["rows"], H, D), dtype=torch.float64, device=dev)
    L = torch.zeros((st["rows"], H), dtype=torch.float64, device=dev)
    t = 0
    for b, (n, length) in enumerate(st["lens"]):
        pages = st["table"][b, :-(-length // case["page"])].long()
        for h in range(Hk):
            k, v = (_exact_values(st[w][pages, h], st[w + "_scales"][pages, h],
                                  case["fmt"]).reshape(-1, D)[:length] for w in ("k", "v"))
            chunk = max(1, int(2.5e8 // (G * length)))
            for i in range(0, n, chunk):
                m = min(chunk, n - i)
                q = st["Q"][t + i:t + i + m, h * G:(h + 1) * G].double()
                s = torch.einsum("igd,jd->igj", q, k) * st["scale"]
                if case["causal"]:
                    own_pos = (length - n + i + torch.arange(m, device=dev))[:, None, None]
                    j = torch.arange(length, device=dev)[None, None, :]
                    seen = j <= own_pos
                    if case["window"]:
                        seen = seen & (j > own_pos - case["window"])
                    s = torch.where(seen, s, torch.full((), -math.inf, dtype=s.dtype, device=dev))
                norm = torch.logsumexp(s, -1)
                O[t + i:t + i + m, h * G:(h + 1) * G] = torch.einsum(
                    "igj,jd->igd", torch.exp(s - norm[..., None]), v)
                L[t + i:t + i + m, h * G:(h + 1) * G] = norm
        t += n
    return [O, L] if case["lse"] else [O]
