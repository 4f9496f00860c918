"""A model whose KV cache is INT4 pages: layers and steps against the library's
own calls on the same activations (bit for bit), prompt against token by token,
graphs and continuous batching.  GPU only (marked gpu)."""
import numpy as np
import pytest

import kv4_ref as ref
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


CFG = dict(synth.TINY_LAYER, n_layers=3, vocab=900, bias=True, codes="symmetric")


def _model(api, lens, gen, seed, max_context, max_batch=None, cfg=CFG, pool_pages=32):
    case = synth.model_case(cfg, lens=lens, gen_tokens=gen, pool_pages=pool_pages, seed=seed)
    r = np.random.default_rng(seed)
    Hkv = cfg["n_kv_heads"]
    dls = []
    for w in case["layers"]:
        kp, vp = ref.random_pool(r, pool_pages, Hkv), ref.random_pool(r, pool_pages, Hkv)
        for p in (kp, vp):                                    # past each sequence's tokens: no numbers
            for b, n in enumerate(lens):
                for t in range(int(n), int(n) + gen):
                    for c in range(4):
                        at = ref.k_scale if p is kp else ref.v_scale
                        p[case["bt"][b, t // 16], :, at(t % 16, c)] = 0xFF
        dls.append(api.device_layer(w, kp, vp))
    m = api.Model(cfg, dls, embed=to_dev(case["embed"], torch), final_norm=to_dev(case["fnorm"], torch),
                  lm_head=to_dev(case["lm"], torch), max_batch=max_batch or len(lens), max_context=max_context,
                  num_pages=pool_pages)
    return m, dls, case


@pytest.mark.parametrize("lens", [[37], [1, 16, 17, 40], [5, 30, 47, 2, 16, 31]])
def test_layer_is_the_library_calls(api, lens):
    """A layer's attention and its pools after it: those of the fused call on
    the layer's own q|k|v rows, bit for bit."""
    m, dls, case = _model(api, [n - 1 for n in lens], 2, 100 + len(lens), 64)
    B = len(lens)
    x = to_dev(synth.normal_fp16(np.random.default_rng(1), (B, CFG["hidden"])), torch)
    bt, ld = to_dev(case["bt"], torch), to_dev(np.asarray(lens, np.int32), torch)
    for l in range(2):
        before = dls[l]["k4"].clone(), dls[l]["v4"].clone()
        m.layer(l, x, bt, ld)
        qkv, att = m.activation("qkv", B), m.activation("attn", B)
        want = api.paged_gqa_decode_int4(qkv, *before, bt, ld, 16 * bt.shape[1], qkv_theta=CFG["theta"], n_q_heads=CFG["n_q_heads"])
        assert torch.equal(att, want.reshape(B, -1))
        assert torch.equal(dls[l]["k4"], before[0]) and torch.equal(dls[l]["v4"], before[1])
        assert bool(torch.isfinite(att).all())
    assert m.check_errors() == 0
    m.close()


def test_graph_steps_equal_plain_launches(api):
    logits, pools = [], []
    for graph in (True, False):
        m, dls, case = _model(api, [37, 15], 12, 7, 64)
        assert m.decode_path(1) == "kernels"
        tok, ld, bt = to_dev(case["tok"], torch), to_dev(case["lens"], torch), to_dev(case["bt"], torch)
        lg = torch.empty((2, CFG["vocab"]), dtype=torch.float16, device="cuda")
        for _ in range(10):
            m.decode_step(tok, tok, bt, ld, logits=lg, use_graph=graph)
        assert m.check_errors() == 0 and to_host(ld).tolist() == [47, 25]
        logits.append(lg.clone())
        pools.append([dl[n].clone() for dl in dls for n in ("k4", "v4")])
        m.close()
    assert torch.equal(*logits) and bool(torch.isfinite(logits[0]).all())
    assert all(torch.equal(a, b) for a, b in zip(*pools))


@pytest.mark.parametrize("cached,T", [(0, 37), (21, 16), (0, 1), (16, 50)])
def test_prompt_against_token_by_token(api, cached, T):
    """A prompt in one pass against decode steps over a copy of the same pools.
    The first layer's rows differ by the roundings of two kinds of projection
    (to fp16, 2^-11 of their size) and a code's step where one of them sits at a
    border; later layers and the logits by what those grow to."""
    prompt = synth.rng(50 + cached).integers(0, CFG["vocab"], size=T).astype(np.int32)
    got = []
    for whole in (True, False):
        m, dls, case = _model(api, [cached], T + 2, 300 + cached + T, cached + T + 16)
        ld, bt = to_dev(case["lens"], torch), to_dev(case["bt"], torch)
        lg = torch.empty((1, CFG["vocab"]), dtype=torch.float16, device="cuda")
        if whole:
            m.prefill(to_dev(prompt, torch), bt, ld, logits=lg)
        else:
            out = torch.empty(1, dtype=torch.int32, device="cuda")
            for t in prompt:
                m.decode_step(torch.tensor([t], dtype=torch.int32, device="cuda"), out, bt, ld, logits=lg)
        assert m.check_errors() == 0 and int(to_host(ld)[0]) == cached + T
        rows = [api.kv_read_int4(dl["k4"], dl["v4"], bt, ld, T, starts=torch.full_like(ld, cached)) for dl in dls]
        got.append((to_host(lg).astype(np.float64), [[to_host(x).astype(np.float64) for x in r] for r in rows]))
        m.close()
    (la, ra), (lb, rb) = got
    rms = lambda x: np.sqrt(np.mean(x ** 2))
    for which in range(2):
        a, b = ra[0][which], rb[0][which]
        assert np.mean(a != b) < 0.02 and rms(a - b) < 0.02 * rms(b)
    assert rms(la - lb) < 0.05 * rms(lb)


def test_prompt_attention_equals_the_decode_attention(api):
    """The last prompt row's attention of the last layer: the decode call's on
    the same rows, to the two kernels' roundings."""
    cfg = dict(CFG, n_layers=1)
    m, dls, case = _model(api, [0], 60, 11, 80, cfg=cfg)
    T = 53
    prompt = synth.rng(3).integers(0, cfg["vocab"], size=T).astype(np.int32)
    ld, bt = to_dev(case["lens"], torch), to_dev(case["bt"], torch)
    lg = torch.empty((1, cfg["vocab"]), dtype=torch.float16, device="cuda")
    m.prefill(to_dev(prompt, torch), bt, ld, logits=lg)
    pools = dls[0]["k4"].clone(), dls[0]["v4"].clone()
    # the last token again as a decode step over the prompt's pages: it writes the same slot
    ld2 = torch.full_like(ld, T - 1)
    lg2 = torch.empty_like(lg)
    m.decode_step(torch.tensor([prompt[-1]], dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"),
                  bt, ld2, logits=lg2)
    assert m.check_errors() == 0
    a, b = to_host(lg).astype(np.float64), to_host(lg2).astype(np.float64)
    assert np.sqrt(np.mean((a - b) ** 2)) < 0.02 * np.sqrt(np.mean(b ** 2))
    same = [float((x == y).float().mean()) for x, y in zip(pools, (dls[0]["k4"], dls[0]["v4"]))]
    assert min(same) > 0.99
    m.close()


def test_continuous_batching_over_int4_pools(api):
    """Sequences of mixed lengths through fewer slots: the tokens each gets alone."""
    cfg = dict(CFG, n_layers=2)
    rng = synth.rng(77)
    prompts = [rng.integers(0, cfg["vocab"], size=n).astype(np.int32) for n in (3, 17, 9, 30, 1)]

    def serve(which, slots):
        m, dls, case = _model(api, [0], 2, 20, 64, max_batch=slots, cfg=cfg, pool_pages=16)
        bat = api.Batcher(m, num_pages=16, max_batch=slots, max_blocks=4, max_context=64)
        ids = [bat.submit(prompts[i], 12) for i in which]
        for _ in range(400):
            if bat.step() == 0:
                break
        out = [bat.poll(i) for i in ids]
        assert all(done for _, done in out) and m.check_errors() == 0
        bat.close()
        m.close()
        return [t.tolist() for t, _ in out]

    together = serve(range(5), 2)
    assert all(len(t) == 12 for t in together)
    # one slot: the same batch size at every step, so the same kernels
    alone = [serve([i], 2)[0] for i in range(5)]
    agree = np.mean([a == b for a, b in zip(together, alone)])
    assert agree >= 0.6        # (batch sizes 1 and 2 round sums differently: near-ties may go the other way)


def test_create_refuses_mixed_pools(api):
    from w4a16_decode_paged_gb300._lib import W4A16Error
    case = synth.model_case(dict(CFG, n_layers=2), lens=[0], gen_tokens=2, pool_pages=8, seed=5)
    kp = np.zeros((8, 1, 1088), np.uint8)
    dls = [api.device_layer(w, kp, kp) for w in case["layers"]]
    dls[1] = api.device_layer(case["layers"][1], synth.host_pool(case, 1, "k"), synth.host_pool(case, 1, "v"))
    with pytest.raises(W4A16Error, match="every layer or none"):
        api.Model(dict(CFG, n_layers=2), dls, max_context=64, num_pages=8)
    with pytest.raises(ValueError, match="k_pool"):
        api.device_layer(case["layers"][0], np.zeros((8, 1, 1024), np.uint8), kp)
