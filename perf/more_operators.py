"""What the operators over MXFP4 matrices are measured on: quantising and reading
back, the product of fp16 activations with MXFP4 weights (one projection, and the
gated pair with SiLU), and the product of two MXFP4 operands.

With `own` false, run() computes an operator in its plain form (elementary torch
operations, 32 bits); with `own` true it makes the calls a user makes of
w4a16_decode_paged_gb300.api.

MXFP4: 4-bit codes (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6), 8 to a 32-bit word, the
lowest nibble first, int32 [rows][K/8]; one power of two 2^(byte - 127) per 32
consecutive elements of a row, in tiles uint8 [rows/128 rounded up][K/128][512]: byte
16 (r % 32) + 4 (r / 32) + j of a tile belongs to its row r and its j-th 32 elements.
"""
import math

import torch

own = False

WORKSPACE_BYTES = 32 << 20   # split-K partial sums: one block for every case


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, m, n, k, bias=False, residual=False):
    c = dict(op=op, m=m, n=n, k=k, bias=bias, residual=residual)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token's hidden state, quantised and read back: latency alone
        _case("quantise b1", "quantise", 1, 0, 3584),
        # the MLP activations of a decode batch, an odd number of rows
        _case("quantise 33 x 18944", "quantise", 33, 0, 18944),
        # the MLP activations of a prompt of 2048 tokens
        _case("quantise 2048 x 18944", "quantise", 2048, 0, 18944),
        # one token through the k projection (512 rows, a bias)
        _case("a16 b1 k", "a16", 1, 512, 3584, bias=True),
        # one token through the down projection, added to the residual stream
        _case("a16 b1 down", "a16", 1, 3584, 18944, residual=True),
        # one token through gate and up: the largest weights of a layer
        _case("a16 b1 gate|up", "silu", 1, 18944, 3584),
        # a few sequences through a tiny layer's projection, odd count
        _case("a16 b7 tiny", "a16", 7, 2432, 896),
        # a decode batch of 32 through gate and up
        _case("a16 b32 gate|up", "silu", 32, 18944, 3584),
        # a prompt of 2048 tokens through the o projection, added to the residual stream
        _case("a16 prompt 2048 o", "a16", 2048, 3584, 3584, residual=True),
        # a short prompt of 37 tokens in 4 bits through a tiny layer's projection
        _case("a4 37 tiny", "a4", 37, 2432, 896, bias=True),
        # a prompt of 512 tokens in 4 bits through gate
        _case("a4 512 gate", "a4", 512, 18944, 3584),
        # a prompt of 4096 tokens in 4 bits through down, added to the residual stream
        _case("a4 4096 down", "a4", 4096, 3584, 18944, residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "a16", "a16", "silu", "a4", "a4"])
    k = 128 * _log(rng, 1, 148)
    if op == "quantise":
        return _case("", op, _log(rng, 1, 2048), 0, k)
    # multiply-adds: no more than the listed cases of the operator
    most = {"a16": 2048 * 3584 * 3584, "silu": 64 * 18944 * 3584, "a4": 4096 * 3584 * 18944}[op]
    n = _log(rng, 1, 18944)
    m = _log(rng, 1, max(1, min(4096, most // (n * k))))
    plain = op == "silu"
    return _case("", op, m, n, k, bias=not plain and rng.random() < 0.5, residual=not plain and rng.random() < 0.5)


def work(case):
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    four = k // 2 + k // 32                                    # bytes of a row in MXFP4
    if op == "quantise":                                       # x in, codes and scales out, those in, values out
        return {"bytes": m * (2 * 2 * k + 2 * four), "flops": 2 * m * k}
    nbytes = 2 * m * k + 2 * m * n * (1 + case["residual"]) + 2 * n * case["bias"]
    mats = 2 if op == "silu" else 1
    if op == "a4":
        nbytes += 2 * m * four                                 # x's codes, written and read
    return {"bytes": nbytes + mats * n * four, "flops": 2 * mats * m * n * k}


# ---------------------------------------------------------------------------
# the format in elementary operations
# ---------------------------------------------------------------------------
def _pow2(byte):
    """fp32 powers of two of scale bytes 1..254 (int32), NaN for 255."""
    p = (byte << 23).view(torch.float32)
    return torch.where(byte == 255, torch.full_like(p, math.nan), p)


def _quantise(x):
    """Codes (int32, 0..15) [R][K] and scale bytes (int32) [R][K/32] of fp16 rows x."""
    g = x.float().unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=104)
    bad = ~torch.isfinite(amax)
    inv = ((254 - byte) << 23).view(torch.float32)
    a = (g * inv.unsqueeze(-1)).abs()                          # exact; borders: ties go to the even code
    mag = torch.zeros_like(a, dtype=torch.int32)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        mag += (a >= border) if up else (a > border)
    code = mag | (torch.signbit(g).to(torch.int32) << 3)
    code = torch.where(bad.unsqueeze(-1), torch.zeros_like(code), code)
    return code.flatten(-2), torch.where(bad, torch.full_like(byte, 255), byte)


def _pack(code):
    """Eight codes a word, the first in the lowest nibble: int32 [R][K/8]."""
    c = code.unflatten(-1, (-1, 8))
    w = c[..., 0].clone()
    for i in range(1, 8):
        w |= c[..., i] << (4 * i)
    return w


def _tiles(byte):
    """Scale bytes [R][K/32] in tiles of 128 rows and 128 elements."""
    r, kb = byte.shape
    t = -(-r // 128)
    full = torch.full((t * 128, kb), 127, dtype=torch.uint8, device=byte.device)
    full[:r] = byte.to(torch.uint8)
    return full.view(t, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).reshape(t, kb // 4, 512).contiguous()


def _untiled(tiles, rows):
    t, kt, _ = tiles.shape
    return tiles.view(t, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(t * 128, kt * 4)[:rows].to(torch.int32)


def _values(codes, tiles):
    """fp32 values [R][K] of packed codes and scale tiles."""
    nib = torch.stack([(codes >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    s = _pow2(_untiled(tiles, codes.shape[0]))
    return (lut[nib].unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    m, n, k = case["m"], case["n"], case["k"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    # activations have a few channels that are much larger than the others
    chan = torch.where(torch.rand(k, generator=gen, device="cuda") < 1 / 64, 8.0, 1.0)
    st = dict(case=case, x=(normal(m, k) * chan).half())
    mats = {"quantise": 0, "silu": 2}.get(case["op"], 1)
    st["w"] = []
    for _ in range(mats):                                      # rows of differing size, as trained weights have them
        row = torch.exp(0.3 * normal(n, 1)) / math.sqrt(k)
        st["w"].append((normal(n, k) * row).half())
    st["bias"] = (0.1 * normal(n)).half() if case["bias"] else None
    st["residual"] = normal(m, n).half() if case["residual"] else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    packed = []
    for w in st.pop("w"):
        parts = [_quantise(w[i:i + 4096]) for i in range(0, w.shape[0], 4096)]
        packed += [torch.cat([_pack(c) for c, _ in parts]), _tiles(torch.cat([b for _, b in parts]))]
    st["packed"] = packed
    st["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from w4a16_decode_paged_gb300 import api
    op = st["case"]["op"]
    if op == "quantise":
        return api.mxfp4_dequantize(*api.mxfp4_quantize(st["x"]))
    if op == "silu":
        return api.w4a16_gemm_silu_mul_mxfp4(st["x"], *st["packed"], workspace=st["workspace"])
    if op == "a16":
        return api.w4a16_gemm_mxfp4(st["x"], *st["packed"], bias=st["bias"], residual=st["residual"],
                                    workspace=st["workspace"])
    return api.w4a4_gemm_mxfp4(*api.mxfp4_quantize(st["x"]), *st["packed"], bias=st["bias"],
                               residual=st["residual"], workspace=st["workspace"])


def _read_back(x):
    code, byte = _quantise(x)
    return _values(_pack(code), _tiles(byte))


def _run_plain(st):
    op, p = st["case"]["op"], st["packed"]
    if op == "quantise":
        return _read_back(st["x"]).half()
    x = _read_back(st["x"]) if op == "a4" else st["x"].float()
    y = torch.matmul(x, _values(p[0], p[1]).T)
    if op == "silu":
        return (y / (1.0 + torch.exp(-y)) * torch.matmul(x, _values(p[2], p[3]).T)).half()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.half()


# ---------------------------------------------------------------------------
# the same from the definition, in 64 bits
# ---------------------------------------------------------------------------
def _exact_rounded(x):
    """What fp16 rows x [R][K] (in 64 bits) are kept as."""
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], 4096):
        g = x[:, j:j + 4096].unflatten(1, (-1, 32))
        a = g.abs().max(2, keepdim=True).values
        _, e = torch.frexp(a)                                  # f * 2^e, f in [1/2, 1)
        unit = torch.where(a > 0, (e - 3).double(), -23.0).clamp(min=-23.0)
        unit = ((unit.to(torch.int64) + 1023) << 52).view(torch.float64)
        v = (g / unit).abs()
        # steps of 1/2 below 2, of 1 below 4, of 2 above; round() sends ties to even
        r = torch.where(v < 2, torch.round(v * 2) / 2, torch.where(v < 4, torch.round(v), torch.round(v / 2) * 2))
        out[:, j:j + 4096] = (r.clamp(max=6.0) * unit * torch.sign(g)).flatten(1)
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    x = st["x"].double()
    if case["op"] in ("quantise", "a4"):
        x = _exact_rounded(x)
    if case["op"] == "quantise":
        return x
    y = [x @ _exact_rounded(w.double()).T for w in st["w"]]
    if case["op"] == "silu":
        return y[0] * torch.sigmoid(y[0]) * y[1]
    out = y[0]
    for name in ("bias", "residual"):
        if st[name] is not None:
            out = out + st[name].double()
    return out
