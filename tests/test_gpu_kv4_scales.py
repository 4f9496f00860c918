"""INT4 pages that hold every scale byte a page may hold, up to the largest (0xE7),
read back and attended to.  GPU only (marked gpu)."""
import numpy as np
import pytest

import attn_bound as ab
import kv4_ref as ref
from gpu_util import to_dev, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


def _pool(r, pages, Hkv, which, bytes_):
    """Any codes whose product with their scale is an fp16 number."""
    pool = np.zeros((pages, Hkv, ref.SLICE), np.uint8)
    pool[..., 1024:] = r.choice(bytes_, (pages, Hkv, 64))
    ci, si = ref._AT[which]
    s = ref.SCALES[pool[..., si]]
    most = np.minimum(7, np.floor(65504 / np.maximum(s, 2.0 ** -20))).astype(int)
    q = r.integers(-most, most + 1) + 8
    pool[..., ci[:, ::2]] = q[..., ::2] | (q[..., 1::2] << 4)
    return pool


def test_every_scale_reads_back():
    from w4a16_decode_paged_gb300 import api, build
    build.build()
    r = np.random.default_rng(1)
    pages, Hkv = 40, 2
    kp, vp = (_pool(r, pages, Hkv, w, np.arange(0xE8)) for w in "kv")
    bt = r.permutation(pages).astype(np.int32)[None]
    n = torch.tensor([pages * 16], dtype=torch.int32, device="cuda")
    got = api.kv_read_int4(to_dev(kp, torch), to_dev(vp, torch), to_dev(bt, torch), n, pages * 16)
    for x, pool, which in zip(got, (kp, vp), "kv"):
        want = ref.unpack(pool[bt[0]], which).transpose(0, 2, 1, 3).reshape(pages * 16, Hkv, D)
        assert np.array_equal(to_host(x)[0].astype(np.float64), want)


@pytest.mark.parametrize("low", [0xD8, 0xE0, 0xE7])
def test_attention_over_the_largest_scales(low):
    from w4a16_decode_paged_gb300 import api
    r = np.random.default_rng(low)
    pages, Hkv, n = 20, 2, 309
    kp, vp = (_pool(r, pages, Hkv, w, np.arange(low, 0xE8)) for w in "kv")
    bt = r.permutation(pages).astype(np.int32)[None]
    q = (r.standard_normal((10, D)) * 2.0 ** -12).astype(np.float16)
    K, V = (ref.unpack(p[bt[0]], w).transpose(0, 2, 1, 3).reshape(pages * 16, Hkv, D)[:n] for p, w in ((kp, "k"), (vp, "v")))
    out = api.paged_gqa_decode_int4(to_dev(q[None], torch), to_dev(kp, torch), to_dev(vp, torch), to_dev(bt, torch),
                                    torch.tensor([n], dtype=torch.int32, device="cuda"), pages * 16, sm_scale=0.1)
    ab.check(to_host(out)[0], q, K, V, 0.1)
