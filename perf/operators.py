"""What the operators over paged KV caches are measured on: writing INT4 pages
and reading them back, decode attention over INT4 pages, and decode attention
with a sliding window and sinks over fp16, FP8 and INT4 pages.

With `own` false, run() computes an operator in its plain form (elementary
torch operations, 32 bits); with `own` true it makes the calls a user makes of
w4a16_decode_paged_gb300.api.

INT4 pages: a (page, kv head) slice is 1024 code bytes and 64 scale bytes.
value = q * s with q in [-7, 7], stored as the nibble q + 8, and s one byte per
32 dims of a row, the 8 bits below the sign of an fp16 number.  K codes are row
major; V codes alternate the 2-byte quads (4 dims) of a token pair's two rows.
"""
import math

import torch

own = False

PAGE = 16
D = 128
SLICE = 1088                 # bytes of an INT4 (page, kv head) slice
THETA = 1e6
WORKSPACE_BYTES = 16 << 20   # split-KV partial results: one block for every case


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, pages, batch, hq, hkv, ctx, lens="full", window=0, sinks=0, rows=0):
    c = dict(op=op, pages=pages, batch=batch, hq=hq, hkv=hkv, ctx=ctx, lens=lens, window=window, sinks=sinks,
             rows=rows)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's decode step: one token's K and V written, and read back
        _case("write b1", "write", "int4", 1, 28, 4, 512),
        # a decode batch: one token of each of 32 sequences of mixed lengths
        _case("write b32", "write", "int4", 32, 28, 4, 4096, "spread"),
        # a prompt of 2048 tokens written in one call, and the whole cache read back
        _case("write prompt 2048", "prompt", "int4", 1, 28, 4, 2048, rows=2048),
        # a cache read back whole (to hand it on): 4 sequences, odd lengths up to 8191
        _case("read b4 8191", "read", "int4", 4, 28, 4, 8191, "spread"),
        # the tiny layer: 7 query heads on one kv head, 37 tokens: latency alone
        _case("int4 b1 37", "decode", "int4", 1, 7, 1, 37),
        # one sequence of 512 tokens, the headline decode shape
        _case("int4 b1 512", "decode", "int4", 1, 28, 4, 512),
        # a decode batch's step: RoPE, the append and the attention over mixed lengths
        _case("int4 step b32", "step", "int4", 32, 28, 4, 4096, "spread"),
        # long contexts
        _case("int4 b4 32768", "decode", "int4", 4, 28, 4, 32768),
        # a window of 1024 tokens and 4 sinks in one long sequence, fp16 pages
        _case("window fp16 b1", "window", "fp16", 1, 28, 4, 32768, window=1024, sinks=4),
        # a decode batch with mixed lengths, some shorter than the window
        _case("window fp16 b32", "window", "fp16", 32, 28, 4, 4096, "spread", window=1000, sinks=17),
        # FP8 pages, every head with its own K and V
        _case("window fp8 b8", "window", "fp8", 8, 8, 8, 16384, window=4096, sinks=64),
        # INT4 pages, the long contexts' batch
        _case("window int4 b4", "window", "int4", 4, 28, 4, 32768, window=8192, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "prompt", "read", "decode", "decode", "step", "window", "window", "window"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    batch = _log(rng, 1, 32)
    # (token, kv head) pairs of the whole batch: no more than the largest listed case's
    most = {"prompt": 2048 * 4, "read": 4 * 8191 * 2}.get(op, 4 * 32768 * 4)
    if op == "prompt":
        batch = 1
    hkv = hkv if op != "prompt" else min(hkv, 4)
    hi = max(1, min(2048 if op == "prompt" else 32768, most // (batch * hkv)))
    ctx = _log(rng, 1, hi)
    lens = rng.choice(["full", "spread"]) if op != "prompt" else "full"
    window = sinks = 0
    pages = "int4"
    if op == "window":
        pages = rng.choice(["fp16", "fp8", "int4"])
        window, sinks = _log(rng, 1, ctx), rng.choice([0, 1, 4, 16, rng.randint(0, 100)])
    if op in ("write", "prompt"):
        g = min(g, 7)
    return _case("", op, pages, batch, g * hkv, hkv, ctx, lens, window, sinks, ctx if op == "prompt" else 0)


def _lens(case):
    b, n = case["batch"], case["ctx"]
    if case["lens"] == "full" or b == 1:
        return [n] * b
    return [1 + (i * (n - 1)) // (b - 1) for i in range(b)]


def _visible(case, n):
    if case["op"] != "window":
        return n
    return min(n, case["window"] + min(case["sinks"], max(0, n - case["window"])))


def work(case):
    b, hq, hkv, op = case["batch"], case["hq"], case["hkv"], case["op"]
    lens = _lens(case)
    row = 2 * D                                            # bytes of one fp16 head row
    kv = 2 * {"fp16": row, "fp8": D + 4, "int4": D // 2 + 4}[case["pages"]]   # K and V of one token and kv head
    new = (case["rows"] or b) if op in ("write", "prompt", "step") else 0
    tokens = sum(_visible(case, n) for n in lens)
    nbytes = 4 * b + 4 * sum(-(-n // PAGE) for n in lens)
    if op in ("write", "prompt"):
        # q in and out, k and v in, the codes out; the codes in again, k and v out
        return {"bytes": nbytes + new * (2 * hq * row + hkv * (2 * row + 2 * kv + 2 * row)), "flops": new * 6 * D * (hq + hkv)}
    if op == "read":
        return {"bytes": nbytes + tokens * hkv * (kv + 2 * row), "flops": tokens * hkv * 2 * D}
    nbytes += tokens * hkv * kv + 2 * b * hq * row
    if op == "step":
        nbytes += new * hkv * (2 * row + kv + 2 * row)
    return {"bytes": nbytes, "flops": 4 * tokens * hq * D}


# ---------------------------------------------------------------------------
# the INT4 format in elementary operations
# ---------------------------------------------------------------------------
def _scale_values(byte):
    """fp32 values of scale bytes: the 8 bits below an fp16's sign."""
    return (byte.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()


def _quantise(x):
    """Codes in [-7, 7] (fp32) and scale bytes (int32) of rows x [..., 128]."""
    g = x.float().unflatten(-1, (4, 32))
    amax = g.abs().amax(-1)
    r = amax / torch.full_like(amax, 7.0)                                       # rounded once, as a division
    big = ((r.view(torch.int32) + ((1 << 20) - 1)) >> 20) - ((127 - 15) << 3)   # 3 fraction bits, rounded up
    small = torch.ceil(r * 2.0 ** 17).to(torch.int32)                           # multiples of 2^-17
    byte = torch.where(r < 2.0 ** -14, small, big)
    s = _scale_values(byte).unsqueeze(-1)
    q = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(g))
    return q.flatten(-2), byte


def _row_bytes(q):
    """Two codes a byte, the even dim in the low nibble: [..., 64]."""
    u = (q + 8).to(torch.int32).unflatten(-1, (64, 2))
    return (u[..., 0] | (u[..., 1] << 4)).to(torch.uint8)


def _pack(q, byte, which):
    """Slices [..., 1088] of codes [..., 16, 128] and scale bytes [..., 16, 4]."""
    b, s = _row_bytes(q), byte.to(torch.uint8)
    if which == "v":
        b = b.unflatten(-1, (32, 2)).unflatten(-3, (8, 2)).transpose(-3, -2)
        s = s.unflatten(-2, (2, 4, 2)).movedim(-1, -4).transpose(-3, -2)
        n = 4
    else:
        s = s.unflatten(-2, (2, 8)).movedim(-3, -1)
        n = 3
    b = b.flatten(-4) if which == "v" else b.flatten(-2)
    return torch.cat([b, s.flatten(-n)], -1)


def _unpack(sl, which):
    """fp32 rows [..., 16, 128] of slices [..., 1088]."""
    b, s = sl[..., :1024], sl[..., 1024:]
    if which == "v":
        b = b.unflatten(-1, (8, 32, 2, 2)).transpose(-3, -2).flatten(-2).flatten(-3, -2)
        s = s.unflatten(-1, (4, 4, 2, 2)).transpose(-3, -2).movedim(-4, -1).flatten(-4, -2)
    else:
        b = b.unflatten(-1, (16, 64))
        s = s.unflatten(-1, (8, 4, 2)).movedim(-1, -3).flatten(-3, -2)
    q = torch.stack([b & 15, b >> 4], -1).flatten(-2).float() - 8.0
    return (q.unflatten(-1, (4, 32)) * _scale_values(s).unsqueeze(-1)).flatten(-2)


def _store_rows(pool, rows, page, slot, which):
    """Quantised rows [n, hkv, 128] into their slots of the INT4 pool."""
    q, byte = _quantise(rows)
    n, hkv = rows.shape[:2]
    dev = rows.device
    i, g = torch.arange(64, device=dev), torch.arange(4, device=dev)
    sl = slot[:, None]
    if which == "v":
        off = (sl // 2) * 128 + (i // 2) * 4 + (sl % 2) * 2 + i % 2
        soff = 1024 + g * 16 + ((sl % 8) // 2) * 4 + (sl // 8) * 2 + sl % 2
    else:
        off = sl * 64 + i
        soff = 1024 + (sl % 8) * 8 + g * 2 + sl // 8
    p, h = page[:, None, None], torch.arange(hkv, device=dev)[None, :, None]
    pool[p, h, off[:, None, :]] = _row_bytes(q)
    pool[p, h, soff[:, None, :]] = byte.to(torch.uint8)


def _rotate(x, pos, inv):
    """Rotate-half RoPE of x [n, heads, 128] at positions pos [n], fp32."""
    ang = pos.float()[:, None] * inv
    cs, sn = ang.cos()[:, None, :], ang.sin()[:, None, :]
    a, b = x.float().split(D // 2, -1)
    return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = "cuda"
    b, hq, hkv, ctx = case["batch"], case["hq"], case["hkv"], case["ctx"]
    lens = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    blocks = -(-ctx // PAGE)
    used = [-(-n // PAGE) for n in _lens(case)]
    total = sum(used) + 16                                     # some pages of the pool belong to nobody
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((b, blocks), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(used):                               # scattered pages, -1 past each sequence's last
        table[i, :n] = perm[at:at + n]
        at += n

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def cache(spread):
        x = (normal(total, hkv, PAGE, D) * spread).half()
        if case["pages"] == "fp16":
            return x, None
        if case["pages"] == "fp8":
            s = x.float().abs().amax(-1) / 448.0
            return (x.float() / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8), s
        which = "k" if spread is chan else "v"
        return torch.cat([_pack(*_quantise(x[i:i + 1024]), which) for i in range(0, total, 1024)]), None

    # keys have a few channels that are larger than the others
    chan = torch.where(torch.rand(D, generator=gen, device=dev) < 1 / 32, 3.0, 1.0)
    ones = torch.ones(D, device=dev)
    st = dict(case=case, lens=lens, table=table, blocks=blocks)
    st["k_pool"], st["k_scale"] = cache(chan)
    st["v_pool"], st["v_scale"] = cache(ones)
    n = case["rows"] or b
    qkv = torch.cat([normal(n, hq, D), normal(n, hkv, D) * chan, normal(n, hkv, D)], 1).half()
    if case["op"] == "step":
        st["qkv"] = qkv.flatten(1)
    else:
        st["q"], st["k"], st["v"] = (t.contiguous() for t in qkv.split([hq, hkv, hkv], 1))
    # a prompt's rows: the sequence's pages and the length after each of its tokens
    st["row_table"] = table.expand(n, blocks).contiguous() if case["rows"] else table
    st["row_lens"] = torch.arange(1, n + 1, dtype=torch.int32, device=dev) if case["rows"] else lens
    st["inv"] = torch.tensor([THETA ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device=dev).float()
    st["last"] = (lens - 1).contiguous()
    if case["op"] == "read":                                   # rows past a sequence's length stay as they are
        st["k_out"], st["v_out"] = (torch.zeros((b, ctx, hkv, D), dtype=torch.float16, device=dev) for _ in "kv")
    st["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from w4a16_decode_paged_gb300 import api
    c, op = st["case"], st["case"]["op"]
    kp, vp, table, lens = st["k_pool"], st["v_pool"], st["table"], st["lens"]
    if op in ("write", "prompt"):
        q = torch.empty_like(st["q"])
        api.kv_append_rope_int4(st["q"], st["k"], st["v"], kp, vp, st["row_table"], st["row_lens"], THETA, q_out=q)
        if op == "prompt":
            return (q,) + api.kv_read_int4(kp, vp, table, lens, c["rows"])
        return (q,) + api.kv_read_int4(kp, vp, table, lens, 1, starts=st["last"])
    if op == "read":
        return api.kv_read_int4(kp, vp, table, lens, c["ctx"], k_out=st["k_out"], v_out=st["v_out"])
    if op == "decode":
        return api.paged_gqa_decode_int4(st["q"], kp, vp, table, lens, c["ctx"], workspace=st["workspace"])
    if op == "step":
        out = api.paged_gqa_decode_int4(st["qkv"], kp, vp, table, lens, c["ctx"], workspace=st["workspace"],
                                        qkv_theta=THETA, n_q_heads=c["hq"])
        return (out,) + api.kv_read_int4(kp, vp, table, lens, 1, starts=st["last"])
    return api.paged_gqa_decode_window(st["q"], kp, vp, table, lens, c["ctx"], c["window"], c["sinks"],
                                       k_scale=st["k_scale"], v_scale=st["v_scale"], workspace=st["workspace"])


def _slots(table, pos):
    return table.gather(1, (pos // PAGE).long()[:, None])[:, 0].long(), (pos % PAGE).long()


def _cached(st, which):
    """fp32 rows [b, hkv, tokens, 128] of the whole cache, through the block table."""
    pool, scale, t = st[which + "_pool"], st[which + "_scale"], st["table"].clamp(min=0).long()
    if st["case"]["pages"] == "int4":
        x = _unpack(pool[t], which)
    elif st["case"]["pages"] == "fp8":
        x = pool[t].view(torch.float8_e4m3fn).float() * scale[t].unsqueeze(-1)
    else:
        x = pool[t].float()
    return x.transpose(1, 2).flatten(2, 3)


def _attend(st, q):
    c = st["case"]
    b, hq, hkv = c["batch"], c["hq"], c["hkv"]
    k, v = _cached(st, "k"), _cached(st, "v")
    t, n = torch.arange(k.shape[2], device=k.device), st["lens"][:, None]
    seen = t < n
    if c["op"] == "window":
        seen = seen & ((t < c["sinks"]) | (t >= n - c["window"]))
    s = torch.matmul(q.float().view(b, hkv, hq // hkv, D), k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (torch.matmul(p, v) / p.sum(-1, keepdim=True)).view(b, hq, D).half()


def _last_rows(st):
    """The newest token's K and V of each sequence, read back: [b, 1, hkv, 128]."""
    page, slot = _slots(st["table"], st["last"])
    i = torch.arange(len(page), device=page.device)
    return tuple(_unpack(st[w + "_pool"][page], w)[i, :, slot].unsqueeze(1).half() for w in "kv")


def _run_plain(st):
    c, op = st["case"], st["case"]["op"]
    if op in ("write", "prompt", "step"):
        if op == "step":
            q, k, v = st["qkv"].view(c["batch"], -1, D).split([c["hq"], c["hkv"], c["hkv"]], 1)
        else:
            q, k, v = st["q"], st["k"], st["v"]
        pos = st["row_lens"] - 1
        page, slot = _slots(st["row_table"], pos)
        q = _rotate(q, pos, st["inv"]).half()
        _store_rows(st["k_pool"], _rotate(k, pos, st["inv"]).half(), page, slot, "k")
        _store_rows(st["v_pool"], v, page, slot, "v")
        if op == "write":
            return (q,) + _last_rows(st)
        if op == "step":
            return (_attend(st, q),) + _last_rows(st)
    if op in ("prompt", "read"):
        live = (torch.arange(c["ctx"], device=st["lens"].device) < st["lens"][:, None])[:, :, None, None]
        rows = [(_cached(st, w).transpose(1, 2)[:, :c["ctx"]] * live).half() for w in "kv"]
        return (q, *rows) if op == "prompt" else tuple(rows)
    return _attend(st, st["q"])


# ---------------------------------------------------------------------------
# the same from the definition, in 64 bits
# ---------------------------------------------------------------------------
def _two(e):
    """2^e in 64 bits, e whole (ldexp goes through an inexact power)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_scale(amax):
    """Smallest m * 2^e >= amax / 7 with m < 16 whole and 2^e >= 2^-17."""
    seven = torch.full_like(amax, 7.0)
    _, e = torch.frexp(amax / seven)                           # f * 2^e, f in [1/2, 1)
    unit = _two((e - 4).clamp(min=-17))
    return torch.ceil(amax / (seven * unit)) * unit


def _exact_row(x):
    """The values that rows [..., 128] of fp16 numbers (in 64 bits) are kept as."""
    out = torch.empty_like(x)
    for g in range(0, D, 32):
        part = x[..., g:g + 32]
        s = _exact_scale(part.abs().max(-1, keepdim=True).values)
        out[..., g:g + 32] = torch.where(s > 0, torch.round(part / s.clamp(min=2.0 ** -17)).clamp(-7, 7) * s, 0.0)
    return out


def _exact_rotated(x, pos):
    # the angle is the fp32 product of the position and the fp32 inverse frequency
    inv = torch.tensor([THETA ** (-i / 64.0) for i in range(64)], dtype=torch.float64).float().to(x.device)
    ang = (pos.float().view(-1, 1) * inv.view(1, -1)).double().unsqueeze(1)
    lo, hi = x[..., :64].double(), x[..., 64:].double()
    c, s = torch.cos(ang), torch.sin(ang)
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=2)


def _exact_page(slices, which):
    """Rows [pages, hkv, 16, 128] in 64 bits, addressed byte by byte."""
    dev = slices.device
    t = torch.arange(PAGE, device=dev).view(-1, 1)
    d = torch.arange(D, device=dev).view(1, -1)
    if which == "k":
        code, scale = t * 64 + torch.div(d, 2, rounding_mode="floor"), 1024 + (t % 8) * 8 + torch.div(d, 32, rounding_mode="floor") * 2 + torch.div(t, 8, rounding_mode="floor")
    else:
        pair, quad = torch.div(t, 2, rounding_mode="floor"), torch.div(d, 4, rounding_mode="floor")
        code = pair * 128 + quad * 4 + (t % 2) * 2 + torch.div(d % 4, 2, rounding_mode="floor")
        scale = 1024 + torch.div(d, 32, rounding_mode="floor") * 16 + (pair % 4) * 4 + torch.div(t, 8, rounding_mode="floor") * 2 + t % 2
    raw = slices.to(torch.int64)
    nib = (raw[..., code] >> (4 * (d % 2))) % 16
    byte = raw[..., scale]
    e, m = byte >> 3, (byte & 7).double()
    s = torch.where(e > 0, 8.0 + m, m) * _two((e - 18).clamp(min=-17))
    return (nib - 8).double() * s


def _exact_cache(st, i, which, first, last):
    """K or V of sequence i, tokens [first, last), [hkv, n, 128] in 64 bits."""
    p0 = first // PAGE
    ids = st["table"][i, p0:-(-last // PAGE)].long()
    pool = st[which + "_pool"][ids]
    if st["case"]["pages"] == "int4":
        x = _exact_page(pool, which)
    elif st["case"]["pages"] == "fp8":
        x = pool.view(torch.float8_e4m3fn).double() * st[which + "_scale"][ids].double()[..., None]
    else:
        x = pool.double()
    x = x.permute(1, 0, 2, 3).reshape(st["case"]["hkv"], -1, D)
    return x[:, first - p0 * PAGE:last - p0 * PAGE]


def exact(case, seed):
    st = prepare(case, seed)
    op, b, hq, hkv = case["op"], case["batch"], case["hq"], case["hkv"]
    lens = [int(n) for n in st["lens"].tolist()]
    if op in ("write", "prompt", "step"):
        if op == "step":
            rows = st["qkv"].view(b, hq + 2 * hkv, D)
            q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            q, k, v = st["q"], st["k"], st["v"]
        pos = st["row_lens"] - 1
        q = _exact_rotated(q, pos)
        k, v = _exact_row(_exact_rotated(k, pos).half().double()), _exact_row(v.double())
        if op == "prompt":
            return (q, k.unsqueeze(0), v.unsqueeze(0))
        if op == "write":
            return (q, k.unsqueeze(1), v.unsqueeze(1))
        q = q.half().double()
    if op == "read":
        outs = []
        for w in "kv":
            x = torch.zeros((b, case["ctx"], hkv, D), dtype=torch.float64, device="cuda")
            for i, n in enumerate(lens):
                x[i, :n] = _exact_cache(st, i, w, 0, n).transpose(0, 1)
            outs.append(x)
        return tuple(outs)
    if op != "step":
        q = st["q"].double()
    out = torch.empty((b, hq, D), dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        cut = max(0, n - case["window"]) if op == "window" else 0
        spans = [(0, n)] if cut <= case["sinks"] else [(0, case["sinks"])] * (case["sinks"] > 0) + [(cut, n)]
        kk, vv = (torch.cat([_exact_cache(st, i, w, a, z) for a, z in spans], 1) for w in "kv")
        if op == "step":
            kk[:, -1], vv[:, -1] = k[i], v[i]
        for h in range(hkv):
            s = q[i, h * (hq // hkv):(h + 1) * (hq // hkv)] @ kk[h].T / math.sqrt(float(D))
            out[i, h * (hq // hkv):(h + 1) * (hq // hkv)] = torch.softmax(s, -1) @ vv[h]
    return (out, k.unsqueeze(1), v.unsqueeze(1)) if op == "step" else out
