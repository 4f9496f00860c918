"""The prompt attention over INT4 pages, row by row: each row's output against
the 64-bit formula over the rows that the pages hold, with the query that the
layer computed.  GPU only (marked gpu)."""
import math

import numpy as np
import pytest

import attn_bound as ab
from gpu_util import to_dev, to_host
from w4a16_decode_paged_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as _api
    from w4a16_decode_paged_gb300 import build
    build.build()
    return _api


def _cfg(Hq, Hkv, **kw):
    return dict(dict(name="kv4-prompt", hidden=256, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D, inter=256, n_layers=1,
                     vocab=512, eps=1e-6, theta=1e6, bias=True, codes="symmetric", seed=1), **kw)


class Prompt:
    """One layer over INT4 pools whose first rows are K, V [cached][Hkv][D]; run()
    gives the rotated queries and the attention's rows of a prompt."""

    def __init__(self, api, cfg, K, V, T, seed, change=None):
        r = np.random.default_rng(seed)
        self.api, self.cfg, self.T = api, cfg, T
        Hkv, cached = cfg["n_kv_heads"], len(K)
        self.n = cached + T
        pad = lambda x: np.concatenate([x, np.zeros((T, Hkv, D))])
        rows = ab.Rows(r, "int4", pad(K), pad(V))
        for which, p in rows.pools.items():                       # past the cached rows: anything
            for page in rows.bt[0, (cached + 15) // 16:]:
                p[page] = r.integers(0, 256, p[page].shape)
        case = synth.model_case(cfg, lens=[0], pool_pages=8, seed=seed)
        if change:
            change(case)
        self.layer = api.device_layer(case["layers"][0], rows.pools["k_pool"], rows.pools["v_pool"])
        self.model = api.Model(cfg, [self.layer], embed=to_dev(case["embed"], torch), final_norm=to_dev(case["fnorm"], torch),
                               lm_head=to_dev(case["lm"], torch), max_batch=1, max_context=self.n + 16)
        self.bt = to_dev(rows.bt, torch)
        self.lens = torch.tensor([cached], dtype=torch.int32, device="cuda")

    def run(self, tokens):
        c, T = self.cfg, self.T
        need = int(self.api.load().w4a16_prefill_workspace_size(self.model._h, T, self.bt.shape[1]))
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.model.prefill(to_dev(np.asarray(tokens, np.int32), torch), self.bt, self.lens, workspace=ws)
        assert self.model.check_errors() == 0
        # the workspace starts with x, the normalised rows, q | k | v and the attention's rows
        nq, nqkv = c["n_q_heads"] * D, (c["n_q_heads"] + 2 * c["n_kv_heads"]) * D
        up = lambda n: (n + 255) // 256 * 256
        at = up(T * c["hidden"] * 2) + up(T * max(c["hidden"], c["inter"], nq) * 2)
        half = lambda o, n: ws[o:o + 2 * T * n].view(torch.float16).view(T, n)
        q = to_host(half(at, nqkv))[:, :nq].reshape(T, -1, D)
        out = to_host(half(at + up(T * nqkv * 2), nq)).reshape(T, -1, D)
        k, v = self.api.kv_read_int4(self.layer["k4"], self.layer["v4"], self.bt, self.lens, self.n)
        self.model.close()
        return q, out, to_host(k)[0].astype(np.float64), to_host(v)[0].astype(np.float64)


def _check_rows(q, out, K, V, rows):
    first = len(K) - len(q)
    for i in rows:
        n = first + i + 1
        ab.check(out[i], q[i], K[:n], V[:n], 1 / math.sqrt(D), what=f"row {i}")


@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (4, 2), (8, 2), (14, 2), (28, 4), (16, 2)])
@pytest.mark.parametrize("cached,T", [(0, 1), (0, 300), (21, 37), (33, 160)])
def test_rows_of_every_head_layout(api, Hq, Hkv, cached, T):
    r = np.random.default_rng(Hq + cached)
    K, V = r.standard_normal((2, cached, Hkv, D))
    p = Prompt(api, _cfg(Hq, Hkv), K, V, T, 40 + Hq + T)
    q, out, K, V = p.run(r.integers(0, 512, T))
    rows = sorted({*range(0, T, 1 if T < 50 else 7), *range(max(0, T - 20), T)})
    _check_rows(q, out, K, V, rows)


@pytest.mark.parametrize("above", [10.0, 14.0, 16.0])
def test_rows_with_small_weights_beside_tokens_without_a_value(api, above):
    """The largest weights of a cached context are tokens whose V is zero, one in
    every page; the rows' output is the sum of many weights of e^-10 and less of them."""
    r = np.random.default_rng(int(above))
    cached, T, Hq, Hkv = 4000, 20, 14, 2
    d = 63                                                       # dims 63 and 127 turn by 1.2e-6 a position
    K = r.standard_normal((cached, Hkv, D)) * 0.1
    K[:, :, d] = r.standard_normal((cached, Hkv)) * 0.5
    K[::16, :, d] = above
    V = 200.0 * (1.0 + 0.25 * r.standard_normal((cached, Hkv, D)))
    V[::16] = 0.0

    def change(case):                                            # q, k, v: their biases
        w = case["layers"][0]
        for n in ("sq", "sk", "sv"):
            w[n] = np.zeros_like(w[n])
        w["bq"] = (0.3 * r.standard_normal((Hq, D))).astype(np.float16)
        w["bq"][:, d] = D ** 0.5 * np.linspace(0.8, 1.0, Hq)
        w["bq"] = w["bq"].reshape(-1)
        w["bk"], w["bv"] = np.zeros_like(w["bk"]), np.zeros_like(w["bv"])
    p = Prompt(api, _cfg(Hq, Hkv), K, V, T, 60, change)
    q, out, K, V = p.run(r.integers(0, 512, T))
    _check_rows(q, out, K, V, range(T))


@pytest.mark.parametrize("Hq,Hkv,cached,at", [(14, 2, 0, 10), (8, 2, 5, 16), (7, 1, 16, 33), (3, 3, 0, 0)])
def test_rows_before_a_token_without_numbers(api, Hq, Hkv, cached, at):
    """A prompt token whose activations are NaN: the rows before it see nothing of it,
    to the bit; those from it on are NaN."""
    r = np.random.default_rng(cached + at)
    K, V = r.standard_normal((2, cached, Hkv, D))
    T, bad = 40, 500

    def change(case):
        case["embed"][bad] = np.nan
    tokens = r.integers(0, bad, T)
    clean = Prompt(api, _cfg(Hq, Hkv), K, V, T, 70, change).run(tokens)[1]
    tokens[at] = bad
    out = Prompt(api, _cfg(Hq, Hkv), K, V, T, 70, change).run(tokens)[1]
    assert np.all(np.isnan(out[at:]))
    assert np.all(np.isfinite(out[:at])) and np.array_equal(out[:at], clean[:at])


@pytest.mark.parametrize("at", [0, 13, 16, 38, 39])
def test_a_value_group_without_numbers(api, at):
    """A token whose V overflows in dims 32 .. 63 of one kv head: NaN there in the
    rows from it on, and nothing else."""
    Hq, Hkv, T, bad = 8, 2, 40, 500
    r = np.random.default_rng(at)

    def change(case):
        case["embed"][:, :128] = 0                               # (in dims 0 .. 127 this token alone is not zero)
        case["embed"][bad] = 0
        case["embed"][bad, 5] = 1
        w = case["layers"][0]
        w["sv"][32:64, 0] = 10000.0
        w["sv"][32:64, 1] = 0.0
    tokens = r.integers(0, bad, T)
    tokens[at] = bad
    q, out, K, V = Prompt(api, _cfg(Hq, Hkv), np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D)), T, 80, change).run(tokens)
    lost = np.zeros_like(V, bool)
    lost[at, 0, 32:64] = True
    assert np.array_equal(np.isnan(V), lost)
    V = np.where(lost, 0.0, V)
    for i in range(T):
        ref_, w = ab.attend(q[i], K[:i + 1], V[:i + 1], D ** -0.5)
        nan = np.zeros((Hq, D), bool)
        nan[:Hq // Hkv, 32:64] = i >= at
        assert np.array_equal(np.isnan(out[i]), nan), i
        lim = ab.bound(q[i], K[:i + 1], V[:i + 1], D ** -0.5, ref_, w)
        assert np.all((np.abs(out[i] - ref_) <= lim) | nan), i
