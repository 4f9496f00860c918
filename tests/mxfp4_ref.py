"""MXFP4 matrices in 64 bits, from the definition (no product code), and the
bounds that the tests hold the kernels to."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def quantise(x):
    """Codes (uint8, 0..15) [R][K] and scale bytes (uint8) [R][K/32] of rows x
    (fp16), by comparing every value with all eight magnitudes."""
    x = np.asarray(x, dtype=np.float64)
    r, k = x.shape
    g = x.reshape(r, k // 32, 32)
    finite = np.isfinite(g).all(-1)
    a = np.where(finite, np.abs(np.where(np.isfinite(g), g, 0)).max(-1), 0.0)
    e = np.where(a > 0, np.frexp(np.where(a > 0, a, 1.0))[1] - 3, -23)      # floor(log2 a) - 2
    e = np.maximum(e, -23)
    v = np.where(finite[..., None], np.abs(np.where(np.isfinite(g), g, 0)), 0.0) / np.exp2(e)[..., None]
    d = np.abs(np.minimum(v, 6.0)[..., None] - E2M1[:8])
    best = d.min(-1, keepdims=True)
    tied = d == best
    even = np.argmax(tied & (np.arange(8) % 2 == 0), -1)
    first = np.argmax(tied, -1)
    code = np.where(tied.sum(-1) > 1, even, first) | (np.signbit(g).astype(np.int64) << 3)
    code = np.where(finite[..., None], code, 0)
    byte = np.where(finite, e + 127, 255)
    return code.reshape(r, k).astype(np.uint8), byte.astype(np.uint8)


def values(code, byte):
    """64-bit values of codes [R][K] and scale bytes [R][K/32] (255: NaN)."""
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return E2M1[code] * np.repeat(s, 32, axis=1)


def pack(code):
    """uint32 words [R][K/8], the first code in the lowest nibble."""
    c = code.reshape(code.shape[0], -1, 8).astype(np.uint32)
    return np.bitwise_or.reduce(c << (4 * np.arange(8, dtype=np.uint32)), axis=-1)


def unpack(words):
    w = np.asarray(words).view(np.uint32)
    return ((w[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(w.shape[0], -1).astype(np.uint8)


def tiles(byte, fill=127):
    """Scale bytes in tiles, byte by byte from the layout's formula."""
    r, kb = byte.shape
    out = np.full((-(-r // 128), kb // 4, 512), fill, np.uint8)
    i, b = np.meshgrid(np.arange(r), np.arange(kb), indexing="ij")
    out[i // 128, b // 4, 16 * (i % 32) + 4 * (i % 128 // 32) + b % 4] = byte
    return out


def untiled(t, rows):
    i, b = np.meshgrid(np.arange(rows), np.arange(t.shape[1] * 4), indexing="ij")
    return t[i // 128, b // 4, 16 * (i % 32) + 4 * (i % 128 // 32) + b % 4]


def weights(rng, n, k, spread=0.3):
    """fp16 weight rows of differing size."""
    return (rng.standard_normal((n, k)) * np.exp(spread * rng.standard_normal((n, 1))) / np.sqrt(k)).astype(np.float16)


def half_step(v):
    """Half an fp16 step at |v| (64 bits): 2^-11 relative, 2^-25 at least."""
    return np.maximum(np.abs(v) * 2.0 ** -11, 2.0 ** -25)


def sum_error(absum, k):
    """Error of an fp32 sum of k exact products whose magnitudes sum to absum,
    added 16 at a time or more: each of the k / 16 additions, and of some 32 that
    join parts, is off by at most 2^-23 (a truncated addition) of a partial sum
    no larger than absum."""
    return (k / 16 + 32) * 2.0 ** -23 * absum


def check_product(got, x, w, bias=None, residual=None, what=""):
    """got fp16 [M][N] against x . w^T (+ bias) (+ residual), all 64 bits."""
    s, a = x @ w.T, np.abs(x) @ np.abs(w).T
    for t in (bias, residual):
        if t is not None:
            s, a = s + t, a + np.abs(t)
    _hold(got, s, sum_error(a, x.shape[1]), what)


def check_silu(got, x, g, u, what=""):
    """got fp16 [M][N] against silu(x . g^T) * (x . u^T).  |silu'| <= 1.1; the
    exponential, the division and the two products are each off by a few
    2^-24 of the value: 2^-21 covers them."""
    gs, us = x @ g.T, x @ u.T
    eg, eu = (sum_error(np.abs(x) @ np.abs(m).T, x.shape[1]) for m in (g, u))
    silu = gs / (1 + np.exp(-gs))
    y = silu * us
    _hold(got, y, 1.1 * eg * (np.abs(us) + eu) + np.abs(silu) * eu + 2.0 ** -21 * np.abs(y), what)


def _hold(got, ref, err, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - (err + half_step(np.abs(ref) + err))
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over.max() <= 0, f"{what}: {(over > 0).sum()} of {over.size} off, worst at {i}: {got[i]} for {ref[i]}"
    # over many outputs: a rounding to fp16 is spread over a step of 2^-10 of the
    # value at most, so its root mean square is at most 2^-10 / sqrt(12) of it
    if ref.size >= 4096:
        rms = np.sqrt(np.mean((got - ref) ** 2) / np.mean(ref ** 2))
        assert rms <= 2.0 ** -10 / np.sqrt(12) * 1.02, f"{what}: rms error {rms}"
