"""Decode attention over one sequence in 64 bits, with a bound on a kernel's
error that follows from the weights of the tokens (kv4_ref.check_attention's
grows with the context alone), and pools of every kind made from given rows."""
import numpy as np

import kv4_ref as ref

D, PAGE = 128, 16


def attend(q, K, V, scale):
    """(out [Hq][D], weights [Hq][n]) of q [Hq][D] over rows K, V [n][Hkv][D]."""
    Hq, Hkv = q.shape[0], K.shape[1]
    out, w = np.empty((Hq, D)), np.empty((Hq, len(K)))
    for h in range(Hq):
        s = K[:, h * Hkv // Hq] @ q[h].astype(np.float64) * scale
        e = np.exp(s - s.max())
        w[h] = e / e.sum()
        out[h] = w[h] @ V[:, h * Hkv // Hq]
    return out, w


def bound(q, K, V, scale, out, w, v_scale=None):
    """What a kernel may be off by, element by element.  A kernel that takes P
    relative to its largest weight with the factor 2^13, rounds it to fp16 and
    multiplies into fp32 sums is off by

      2^-11 |out| + 2^-25          the output's rounding (half a step of fp16)
      2^-11 sum(w |v|)             P's rounding where it is a normal number
      2^-38 max(w) sum(|v|)        and below: half a step of 2^-24 of P, whose
                                   factor is 2^13 over a reference that is no
                                   more than the largest score
                                   (FP8: P carries the row scale, so this is
                                   max(w s) sum(|code|))
      2 e sum(w |v|)               e: the weights' relative error from the scores
                                   (128 adds in fp32, each off by 2^-23 of
                                   sum |q k| at most; the products with the
                                   scale and log2 e, 2^-22 of the score) and
                                   from exp2 (2^-20), twice: P and its sum
      (n / 16 + 64) 2^-23 sum(w |v|)   the fp32 sums over the pages and parts
    """
    Hq, Hkv = q.shape[0], K.shape[1]
    res = np.empty_like(out)
    for h in range(Hq):
        k, v = K[:, h * Hkv // Hq], np.abs(V[:, h * Hkv // Hq])
        qa = np.abs(q[h].astype(np.float64))
        mass = w[h] @ v
        e = 128 * 2.0 ** -23 * scale * (np.abs(k) @ qa).max() + 2.0 ** -22 * scale * np.abs(k @ q[h]).max() + 2.0 ** -20
        if v_scale is None:
            small = w[h].max() * v.sum(0)
        else:
            s = v_scale[:, h * Hkv // Hq].astype(np.float64)
            small = (w[h] * s).max() * (v / np.where(s > 0, s, 1)[:, None]).sum(0)
        res[h] = (2.0 ** -11 * np.abs(out[h]) + 2.0 ** -25 + 2.0 ** -38 * small +
                  (2.0 ** -11 + 2 * e + (len(K) / 16 + 64) * 2.0 ** -23) * mass)
    return res


def check(got, q, K, V, scale, v_scale=None, what=""):
    out, w = attend(q, K, V, scale)
    lim = bound(q, K, V, scale, out, w, v_scale)
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - out)
    i = np.unravel_index(np.argmax(err / lim), err.shape)
    assert np.all(err <= lim), f"{what}: at {i} got {got[i]} expected {out[i]}, off {err[i]:.3g}, allowed {lim[i]:.3g}"


class Rows:
    """Rows K, V [n][Hkv][D] in pages of a kind: `pools` (numpy, the arguments
    k_pool, v_pool and k_scale, v_scale), `bt` [1][pages], and the rows as the
    pages hold them, `K`, `V` (and FP8: `v_scale`, [n][Hkv])."""

    def __init__(self, r, kind, K, V):
        n, Hkv = K.shape[:2]
        used = (n + PAGE - 1) // PAGE
        total = used + 3
        self.bt = r.permutation(total)[:used].astype(np.int32)[None]
        self.kind, self.n, self.pools, self.v_scale = kind, n, {}, None
        for which, x in (("k", K), ("v", V)):
            pages = np.zeros((total, Hkv, PAGE, D))
            padded = np.concatenate([x, np.zeros((used * PAGE - n, Hkv, D))])
            pages[self.bt[0]] = padded.reshape(used, PAGE, Hkv, D).transpose(0, 2, 1, 3)
            vals, scale = getattr(self, "_" + kind)(which, pages)
            rows = lambda a: a[self.bt[0]].swapaxes(1, 2).reshape((used * PAGE, Hkv) + a.shape[3:])[:n]
            setattr(self, which.upper(), rows(vals))
            if which == "v" and scale is not None:
                self.v_scale = rows(scale)

    def _fp16(self, which, x):
        self.pools[which + "_pool"] = x.astype(np.float16)
        return x.astype(np.float16).astype(np.float64), None

    def _fp8(self, which, x):
        import torch
        scale = (np.abs(x).max(-1) / 448).astype(np.float32)
        codes = torch.from_numpy(x / np.where(scale > 0, scale, 1)[..., None]).float().to(torch.float8_e4m3fn)
        self.pools[which + "_pool"], self.pools[which + "_scale"] = codes.view(torch.uint8).numpy(), scale
        return codes.double().numpy() * scale.astype(np.float64)[..., None], scale

    def _int4(self, which, x):
        x = x.astype(np.float16).astype(np.float64)
        g = x.reshape(x.shape[:-1] + (4, 32))
        byte = np.searchsorted(7 * ref.SCALES[:248], np.abs(g).max(-1))
        s = ref.SCALES[byte][..., None]
        q = np.where(s > 0, np.rint(g / np.where(s > 0, s, 1)), 0).reshape(x.shape).astype(np.int64)
        pool = np.zeros(x.shape[:2] + (ref.SLICE,), np.uint8)
        code, scale = (ref.k_code, ref.k_scale) if which == "k" else (ref.v_code, ref.v_scale)
        t = np.arange(PAGE)
        pool[..., np.array([[code(i, d) for d in range(0, D, 2)] for i in t])] = (q[..., ::2] + 8) | ((q[..., 1::2] + 8) << 4)
        pool[..., np.array([[scale(i, c) for c in range(4)] for i in t])] = byte
        self.pools[which + "_pool"] = pool
        return ref.unpack(pool, which), None
