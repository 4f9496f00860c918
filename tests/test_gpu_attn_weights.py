"""Windowed and INT4 decode attention where single tokens, small weights, small
values and large scores decide the result, against the 64-bit formula with the
bound of attn_bound.  GPU only (marked gpu)."""
import numpy as np
import pytest

import attn_bound as ab
import kv4_ref as ref
from gpu_util import to_dev, to_host
from test_attn_bound import dominant_tokens, one_hot_pages, sink_queries

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as _api
    from w4a16_decode_paged_gb300 import build
    build.build()
    return _api


def run(api, x, q, scale, others=()):
    """Attention of one sequence over x's pages; `others`: lengths of sequences
    beside it in the batch, over the same pages."""
    lens = np.array([x.n, *others], np.int32)
    dev = lambda a: to_dev(a, torch)
    out = api.paged_gqa_decode_window(dev(np.repeat(q[None], len(lens), 0)), **{k: dev(a) for k, a in x.pools.items()},
                                      block_table=dev(np.repeat(x.bt, len(lens), 0)), context_lens=dev(lens),
                                      max_context=16 * x.bt.shape[1], window=x.n, sinks=0, sm_scale=scale)
    return to_host(out)[0]


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("n,above,every", [(600, 17.0, 600), (5000, 14.0, 16), (5000, 16.0, 16), (32768, 18.0, 16),
                                           (32768, 19.0, 900)])
def test_small_weights_beside_tokens_without_a_value(api, kind, n, above, every):
    """The largest weights are tokens whose V is zero (one, or one in every page);
    the output is the sum of many weights of e^-14 and less of them."""
    r = np.random.default_rng(int(n + above))
    x = ab.Rows(r, kind, *dominant_tokens(r, n, 2, above, every))
    q = sink_queries(r, 14)
    ab.check(run(api, x, q, 1.0), q, x.K, x.V, 1.0, x.v_scale, f"{kind} {n}")


@pytest.mark.parametrize("size", [1e4, 1.0, 1e-2, 1e-3, 1e-4, 3e-6])
def test_fp8_values_of_any_size(api, size):
    """Row scales from 22 down to 7e-9; V with a mean, scores spread by a few units."""
    r = np.random.default_rng(11)
    n = 4096
    K = r.standard_normal((n, 2, D))
    V = size * (1.0 + 0.5 * r.standard_normal((n, 2, D)))
    x = ab.Rows(r, "fp8", K, V)
    q = (3.0 * r.standard_normal((14, D))).astype(np.float16)
    ab.check(run(api, x, q, D ** -0.5, [100, 37]), q, x.K, x.V, D ** -0.5, x.v_scale, f"V of about {size}")


@pytest.mark.parametrize("order", ["falling", "rising", "mixed", "against the weights", "zeros first"])
def test_fp8_row_scales_that_differ(api, order):
    """Rows whose sizes lie up to 2^40 apart in one sequence; what counts is their
    part of the output."""
    r = np.random.default_rng(12)
    n, Hkv = 3000, 2
    K = r.standard_normal((n, Hkv, D)) * 0.5
    e = np.linspace(8.0, -16.0, n)
    if order == "rising":
        e = -8.0 - e
    if order == "mixed":
        e = r.uniform(-16.0, 8.0, n)
    V = (1.0 + 0.5 * r.standard_normal((n, Hkv, D))) * 2.0 ** e[:, None, None]
    if order == "against the weights":                     # a score of 24 (log2) takes back a size of 2^-24
        K[:, :, 0] = (8.0 - e[:, None]) * np.log(2.0) * D ** 0.5 / 16
    if order == "zeros first":
        V[:2500] = 0.0
    x = ab.Rows(r, "fp8", K, V)
    q = r.standard_normal((6, D)).astype(np.float16)
    if order == "against the weights":
        q[:, 0] = 16.0
    ab.check(run(api, x, q, D ** -0.5), q, x.K, x.V, D ** -0.5, x.v_scale, order)


def test_fp8_without_any_value(api):
    r = np.random.default_rng(13)
    x = ab.Rows(r, "fp8", r.standard_normal((200, 1, D)), np.zeros((200, 1, D)))
    assert np.all(run(api, x, r.standard_normal((7, D)).astype(np.float16), 0.1) == 0)


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("most", [3.0, 300.0, 3000.0, 60000.0])
def test_scores_of_any_size(api, kind, most):
    """Keys and queries up to the ends of fp16: scores up to 5e8 (log2), their
    spacing in fp32 up to 32.  From 300 on one token's score, or three equal ones, are
    more than 700 above the others, so that the output is its V or their mean: off
    by the roundings of P and of the output, 2^-11 each.  (3: 8 and more above a
    thousand others, which count then: the general bound.)"""
    r = np.random.default_rng(14)
    n, Hkv, G = 1000, 2, 7
    K = np.zeros((n, Hkv, D))
    K[:, :, 0] = most * 0.8 * r.uniform(0.1, 1.0, (n, Hkv))
    top = [[613], [40, 333, 999]]
    for h in range(Hkv):
        K[top[h], h, 0] = most
    V = r.standard_normal((n, Hkv, D))
    x = ab.Rows(r, kind, K, V)
    q = np.zeros((Hkv * G, D), np.float16)
    q[:, 0] = np.maximum(most, 300.0) * np.linspace(0.5, 1.0, Hkv * G)
    got = run(api, x, q, D ** -0.5, [10]).astype(np.float64)
    if most < 300:
        return ab.check(got, q, x.K, x.V, D ** -0.5, x.v_scale)
    for h in range(Hkv * G):
        v = x.V[top[h // G], h // G]
        assert np.all(np.abs(got[h] - v.mean(0)) <= 2.0 ** -11 * (np.abs(v.mean(0)) + np.abs(v).mean(0)) + 1e-6), h


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("n,Hkv,others", [(32768, 1, ()), (32768, 4, ()), (32761, 4, (32768, 20011, 777)), (9000, 8, ()),
                                          (100003, 1, ()), (32768, 2, (5,) * 40)])
def test_every_page_counts_once(api, kind, n, Hkv, others):
    """Long contexts in up to 64 parts, near-equal weights, and a V that tells which
    page it came from: one-hot, page p in dim p % 128.  (A lost or doubled page of
    the 6252 moves its dim by a 49th or more; the bound is a 500th.)"""
    r = np.random.default_rng(n + Hkv)
    K, V = one_hot_pages(r, n, Hkv)
    x = ab.Rows(r, kind, K, V)
    G = 7 if Hkv <= 4 else 1
    q = r.standard_normal((G * Hkv, D)).astype(np.float16)
    ab.check(run(api, x, q, D ** -0.5, [min(m, n) for m in others]), q, x.K, x.V, D ** -0.5, x.v_scale, f"{kind} {n}")


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("n,window,sinks", [(32768, 20000, 300), (32768, 4096, 5), (40000, 33, 30000)])
def test_every_visible_page_counts_once(api, kind, n, window, sinks):
    r = np.random.default_rng(n + window)
    K, V = one_hot_pages(r, n, 2)
    x = ab.Rows(r, kind, K, V)
    q = r.standard_normal((10, D)).astype(np.float16)
    dev = lambda a: to_dev(a, torch)
    out = api.paged_gqa_decode_window(dev(q[None]), **{k: dev(a) for k, a in x.pools.items()}, block_table=dev(x.bt),
                                      context_lens=dev(np.array([n], np.int32)), max_context=n, window=window, sinks=sinks)
    t = np.arange(n)
    seen = (t < sinks) | (t >= n - window)
    ab.check(to_host(out)[0], q, x.K[seen], x.V[seen], D ** -0.5, None if x.v_scale is None else x.v_scale[seen])


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("n,Hkv,batch", [(6000, 8, 40), (20001, 4, 100)])
def test_more_pages_than_a_warp_lists_at_once(api, kind, n, Hkv, batch):
    """Batches with more (sequence, kv head) pairs than CTAs fit at once: a pair is one
    CTA's, and a warp's list of page ids (32 at a time) is filled again."""
    r = np.random.default_rng(n)
    x = ab.Rows(r, kind, *one_hot_pages(r, n, Hkv))
    q = r.standard_normal((2 * Hkv, D)).astype(np.float16)
    dev = lambda a: to_dev(a, torch)
    lens = np.full(batch, n, np.int32)
    out = api.paged_gqa_decode_window(dev(np.repeat(q[None], batch, 0)), **{k: dev(a) for k, a in x.pools.items()},
                                      block_table=dev(np.repeat(x.bt, batch, 0)), context_lens=dev(lens), max_context=n,
                                      window=n, sinks=0)
    for b in (0, batch // 2, batch - 1):
        ab.check(to_host(out)[b], q, x.K, x.V, D ** -0.5, x.v_scale, f"{kind} {b}")


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_visible_token_without_numbers(api, kind, which):
    """NaN in K makes its kv head's outputs NaN, NaN in V the dims it is in (INT4: the
    32 of its scale); the other outputs are the formula's."""
    r = np.random.default_rng(15)
    n, Hkv, t, h, d = 1500, 3, 777, 1, 40
    x = ab.Rows(r, kind, *r.standard_normal((2, n, Hkv, D)))
    page, slot = x.bt[0, t // 16], t % 16
    pool = x.pools[which + "_pool"]
    if kind == "int4":
        pool[page, h, (ref.k_scale if which == "k" else ref.v_scale)(slot, d // 32)] = 0xFF
    else:
        pool[page, h, slot, d] = np.nan if kind == "fp16" else 0x7F
    q = r.standard_normal((2 * Hkv, D)).astype(np.float16)
    got = run(api, x, q, D ** -0.5, [40, 2])
    nan = np.zeros((Hkv, 2, D), bool)
    nan[h, :, slice(None) if which == "k" else slice(32, 64) if kind == "int4" else d] = True
    nan = nan.reshape(2 * Hkv, D)
    assert np.array_equal(np.isnan(got), nan)
    out, w = ab.attend(q, x.K, x.V, D ** -0.5)
    assert np.all((np.abs(got - out) <= ab.bound(q, x.K, x.V, D ** -0.5, out, w, x.v_scale)) | nan)
