"""Plain numpy references for the INT4 pages and the windowed decode attention
(64 bits; the format is written out byte by byte from its description)."""
import math

import numpy as np

PAGE, D, SLICE = 16, 128, 1088


def scale_value(byte):
    """Value of a scale byte: 5 exponent and 3 fraction bits, fp16's bias."""
    byte = int(byte)
    e, m = byte >> 3, byte & 7
    if e == 31:
        return math.nan
    return m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18)


SCALES = np.array([scale_value(b) for b in range(256)])


def k_code(t, d):
    return 64 * t + d // 2


def v_code(t, d):
    return 128 * (t // 2) + 4 * (d // 4) + 2 * (t % 2) + (d % 4) // 2


def k_scale(t, c):
    return 1024 + 8 * (t % 8) + 2 * c + t // 8


def v_scale(t, c):
    return 1024 + 16 * c + 4 * ((t % 8) // 2) + 2 * (t // 8) + t % 2


def quantise_row(x):
    """(codes in [-7, 7], scale bytes) of one row of 128 fp16 values."""
    q, byte = np.zeros(D, np.int64), np.zeros(4, np.int64)
    for c in range(4):
        g = np.asarray(x[32 * c:32 * c + 32], np.float64)
        if not np.all(np.isfinite(g)):
            byte[c] = 0xFF
            continue
        amax = np.abs(g).max()
        byte[c] = int(np.argmax(7 * SCALES[:248] >= amax))       # the first that covers it
        s = SCALES[byte[c]]
        if s > 0:
            q[32 * c:32 * c + 32] = np.rint(g / s).astype(np.int64)
    return q, byte


def store_row(sl, t, q, byte, which):
    """Write one row into a slice (uint8 [1088])."""
    code, scale = (k_code, k_scale) if which == "k" else (v_code, v_scale)
    for d in range(D):
        i, sh = code(t, d), 4 * (d % 2)
        sl[i] = (int(sl[i]) & (0xF0 >> sh)) | (int(q[d] + 8) << sh)
    for c in range(4):
        sl[scale(t, c)] = byte[c]


def _tables():
    out = {}
    for which, code, scale in (("k", k_code, k_scale), ("v", v_code, v_scale)):
        ci = np.array([[code(t, d) for d in range(D)] for t in range(PAGE)])
        si = np.array([[scale(t, d // 32) for d in range(D)] for t in range(PAGE)])
        out[which] = ci, si
    return out


_AT = _tables()


def unpack(pool, which):
    """float64 rows [..., 16, 128] of slices uint8 [..., 1088]."""
    ci, si = _AT[which]
    q = ((pool[..., ci].astype(np.int64) >> (4 * (np.arange(D) % 2))) & 15) - 8
    return q * SCALES[pool[..., si]]


def random_pool(r, pages, Hkv, spread=1.0):
    """A pool as appends leave it: any code but -8, scales of values of about `spread`."""
    u = r.integers(1, 16, size=(pages, Hkv, 1024, 2), dtype=np.uint8)
    pool = np.empty((pages, Hkv, SLICE), np.uint8)
    pool[..., :1024] = u[..., 0] | (u[..., 1] << 4)
    e = int(math.floor(math.log2(spread / 4))) + 15
    pool[..., 1024:] = r.integers(8 * e, 8 * e + 12, size=(pages, Hkv, 64), dtype=np.uint8)
    return pool


def rope(x, pos, theta):
    """Rotate-half RoPE of x [heads, 128] at one position, 64 bits; the angle
    is the fp32 product of the position and the fp32 inverse frequency."""
    inv = np.array([theta ** (-2.0 * i / D) for i in range(D // 2)]).astype(np.float32)
    ang = (np.float32(pos) * inv).astype(np.float64)
    a, b = x[:, :64].astype(np.float64), x[:, 64:].astype(np.float64)
    return np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], 1)


def attend(q, k_of, v_of, bt, lens, scale, window=None, sinks=0):
    """(out, bound ingredients) of decode attention.  k_of / v_of(page) give the
    rows [Hkv, 16, 128] of a pool page in 64 bits.  Returns out [B, Hq, 128] and
    the weighted mean of |v| [B, Hq, 128] beside the largest |v| seen."""
    B, Hq, _ = q.shape
    out, mean, top = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), 0.0
    for b in range(B):
        L = int(lens[b])
        seen = [t for t in range(L) if window is None or t >= L - window or t < sinks]
        if not seen:
            continue
        pages = sorted({t // PAGE for t in seen})
        ks = {p: k_of(int(bt[b, p])) for p in pages}
        vs = {p: v_of(int(bt[b, p])) for p in pages}
        K = np.stack([ks[t // PAGE][:, t % PAGE] for t in seen])   # [n, Hkv, D]
        V = np.stack([vs[t // PAGE][:, t % PAGE] for t in seen])
        G = Hq // K.shape[1]
        for h in range(Hq):
            s = K[:, h // G] @ q[b, h].astype(np.float64) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h], mean[b, h] = p @ V[:, h // G], p @ np.abs(V[:, h // G])
        top = max(top, np.abs(V).max())
    return out, mean, top


def check_attention(got, ref, n, what=""):
    """|got - out| <= 2^-11 |out|                 the output's fp16 rounding
                    + 2^-11 mean(|v|)             P rounded to fp16
                    + 2^-11 mean(|v|)             the scores: 128 fp32 adds of at most 2^-23 each
                                                  on sums of |q k| scale log2(e) up to 32
                    + n 2^-22 max(|v|)            P below fp16's normal range (half a step of 2^-24;
                                                  FP8 pages fold a scale in, up to 8 times that)"""
    out, mean, top = ref
    got = np.asarray(got, np.float64)
    assert got.shape == out.shape and np.all(np.isfinite(got)), what
    bound = 2.0 ** -11 * np.abs(out) + 2.0 ** -10 * mean + n * 2.0 ** -22 * top + 1e-7
    err = np.abs(got - out)
    i = np.unravel_index(np.argmax(err - bound), err.shape)
    assert np.all(err <= bound), f"{what}: at {i} got {got[i]} expected {out[i]}, off {err[i]:.3g}, allowed {bound[i]:.3g}"
