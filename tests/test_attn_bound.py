"""The bound that the attention tests over long contexts use, on the CPU: a
kernel's roundings stay inside it, a page that is lost or counted twice, or
small weights that are dropped, do not."""
import numpy as np
import pytest

import attn_bound as ab
import kv4_ref as ref


def one_hot_pages(r, n, Hkv):
    """Rows whose weights are near each other; V is one-hot, page p in dim p % 128."""
    K = r.standard_normal((n, Hkv, 128)) * 0.25
    V = np.zeros((n, Hkv, 128))
    t = np.arange(n)
    V[t, :, (t // 16) % 128] = 1.0
    return K, V


def dominant_tokens(r, n, Hkv, above, every):
    """Every so many tokens one that outweighs the others, and whose V is zero."""
    K = r.standard_normal((n, Hkv, 128)) * 0.3
    K[:, :, 0] = r.standard_normal((n, Hkv))
    K[::every] = 0.0
    K[::every, :, 0] = above
    V = 200.0 * (1.0 + 0.25 * r.standard_normal((n, Hkv, 128)))
    V[::every] = 0.0
    return K, V


def sink_queries(r, Hq):
    q = r.standard_normal((Hq, 128)) * 0.3
    q[:, 0] = np.linspace(0.8, 1.0, Hq)
    return q.astype(np.float16)


def emulate(q, K, V, scale, shift, keep=slice(None), dtype=np.float64):
    """One part of a kernel: P = 2^(shift) times the weight over the largest one,
    rounded to fp16."""
    out = np.empty((len(q), 128))
    for h in range(len(q)):
        s = K[:, h * K.shape[1] // len(q)] @ q[h].astype(np.float64) * scale
        p = np.exp(s - s.max())[keep] * 2.0 ** shift
        out[h] = p.astype(np.float16).astype(np.float64) @ V[keep][:, h * K.shape[1] // len(q)] / p.sum()
    return out.astype(np.float16)


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
def test_rows_are_what_their_pages_hold(kind):
    r = np.random.default_rng(1)
    K, V = r.standard_normal((2, 45, 3, 128))
    V[7] = 0
    x = ab.Rows(r, kind, K, V)
    step = {"fp16": 2.0 ** -11 * 5, "fp8": 2.0 ** -4 * 5, "int4": 5 / 7 * 0.6}[kind]
    for a, b in ((x.K, K), (x.V, V)):
        assert a.shape == b.shape and np.abs(a - b).max() <= step
    assert np.all(x.V[7] == 0)
    if kind == "int4":                                         # the format, byte by byte
        for t in (0, 17, 44):
            want = np.zeros(ref.SLICE, np.uint8)
            got = x.pools["v_pool"][x.bt[0, t // 16], 1]
            ref.store_row(want, t % 16, *ref.quantise_row(V[t, 1].astype(np.float16)), "v")
            assert np.array_equal(ref.unpack(want, "v")[t % 16], ref.unpack(got, "v")[t % 16])


@pytest.mark.parametrize("n", [9000, 32768])
def test_a_lost_or_doubled_page_shows(n):
    r = np.random.default_rng(n)
    K, V = one_hot_pages(r, n, 1)
    q = r.standard_normal((3, 128)).astype(np.float16)
    scale = 128 ** -0.5
    ab.check(emulate(q, K, V, scale, 13), q, K, V, scale)
    for page in (0, 5, n // 32, n // 16 - 1):
        t = np.arange(n)
        for keep in (t[t // 16 != page], np.concatenate([t, t[t // 16 == page]])):
            with pytest.raises(AssertionError):
                ab.check(emulate(q, K, V, scale, 13, keep), q, K, V, scale)


def test_small_weights_that_are_dropped_show():
    r = np.random.default_rng(3)
    K, V = dominant_tokens(r, 32768, 1, 18.0, 32768)
    q = sink_queries(r, 4)
    ab.check(emulate(q, K, V, 1.0, 13), q, K, V, 1.0)
    with pytest.raises(AssertionError):
        ab.check(emulate(q, K, V, 1.0, 0), q, K, V, 1.0)       # fp16's subnormal range
