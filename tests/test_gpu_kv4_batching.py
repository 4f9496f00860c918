"""Continuous batching over INT4 pools against each sequence with a filler beside
it: the batch size is two in every step that a sequence takes part in, so that its
tokens have to be equal, whichever sequences share the batch and whose pages it
was given.  GPU only (marked gpu)."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import to_dev
from w4a16_decode_paged_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [16, 8])
def test_sequences_get_the_tokens_each_gets_beside_a_filler(pages):
    from w4a16_decode_paged_gb300 import api, build
    build.build()
    cfg = dict(synth.TINY_LAYER, n_layers=2, vocab=900, bias=True, codes="symmetric")
    r = synth.rng(78)
    prompts = [r.integers(0, cfg["vocab"], size=n).astype(np.int32) for n in (3, 17, 9, 30, 1, 33, 20)]
    case = synth.model_case(cfg, lens=[0], pool_pages=8, seed=21)

    def serve(which):
        """Tokens of the prompts, and the steps with fewer than two sequences; the
        filler comes last and outlasts them."""
        rr = np.random.default_rng(22)
        dls = [api.device_layer(w, ref.random_pool(rr, pages, 1), ref.random_pool(rr, pages, 1)) for w in case["layers"]]
        m = api.Model(cfg, dls, embed=to_dev(case["embed"], torch), final_norm=to_dev(case["fnorm"], torch),
                      lm_head=to_dev(case["lm"], torch), max_batch=2, max_context=64, num_pages=pages)
        bat = api.Batcher(m, num_pages=pages, max_batch=2, max_blocks=4, max_context=64)
        ids = [bat.submit(prompts[i], 12) for i in which]
        bat.submit(np.array([7], np.int32), 60)
        for _ in range(400):
            running = any(not bat.poll(i)[1] for i in ids)
            n = bat.step()
            if n == 0:
                break
            assert n == 2 or not running
        out = [bat.poll(i) for i in ids]
        assert all(done and len(t) == 12 for t, done in out) and m.check_errors() == 0
        assert bat.stats()["preemptions"] == 0
        bat.close()
        m.close()
        return [t.tolist() for t, _ in out]

    together = serve(range(len(prompts)))
    assert together == [serve([i])[0] for i in range(len(prompts))]
    assert len({tuple(t) for t in together}) > 1
