"""The fused INT4 step past its bound on the context.  GPU only (marked gpu)."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import to_dev, to_host
from w4a16_decode_paged_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D, THETA = 128, 1e4


@pytest.mark.parametrize("lens", [[65], [200, 64, 1, 65], [90] * 40])
def test_a_row_past_the_bound_is_rotated_for_its_own_position(lens):
    """Its output: the attention of the query, rotated for position len - 1, over
    the first max_context tokens (to the bit, as for rows within the bound)."""
    from w4a16_decode_paged_gb300 import api, build
    build.build()
    r = np.random.default_rng(31)
    Hq, Hkv, mc = 14, 2, 64
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    pages = int(sum((n + 15) // 16 for n in lens)) + 2
    bt = synth.block_table(r, lens, pages)
    pools = [to_dev(ref.random_pool(r, pages, Hkv), torch) for _ in "kv"]
    qkv = to_dev(synth.normal_fp16(r, (B, (Hq + 2 * Hkv) * D)), torch)
    dbt, dl = to_dev(bt, torch), to_dev(lens, torch)
    q, k, v = (t.clone(memory_format=torch.contiguous_format) for t in qkv.view(B, -1, D).split([Hq, Hkv, Hkv], 1))
    mine = [p.clone() for p in pools]
    api.kv_append_rope_int4(q, k, v, *mine, dbt, dl, THETA)
    want = api.paged_gqa_decode_int4(q, *mine, dbt, dl, mc)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.paged_gqa_decode_int4(qkv, *pools, dbt, dl, mc, qkv_theta=THETA, n_q_heads=Hq, err_flag=err)
    assert int(err.item()) == 1
    assert np.array_equal(to_host(got), to_host(want))
