"""MXFP4 products of a few fp16 rows whose CTAs have more weight rows than they keep
sums of at once (32 groups of 16): several rounds, with and without clusters, against
64 bits on the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as a
    return a


def weights(api, gen, n, k):
    return api.mxfp4_quantize((torch.randn((n, k), generator=gen, device="cuda") / k ** 0.5).half())


def products(api, q, x):
    """x . W^T and |x| . |W|^T in 64 bits, some rows of W at a time."""
    s, a = [], []
    rows = 128 * max(1, (1 << 26) // (128 * x.shape[1]))
    for i in range(0, q[0].shape[0], rows):
        w = api.mxfp4_dequantize(q[0][i:i + rows], q[1][i // 128:(i + rows) // 128]).double()
        s.append(x @ w.T)
        a.append(x.abs() @ w.abs().T)
    return torch.cat(s, 1), torch.cat(a, 1)


def hold(y, want, err):
    over = (y.double() - want).abs() - err - ((want.abs() + err) * 2.0 ** -11).clamp(min=2.0 ** -25)
    assert bool(torch.isfinite(y).all()) and float(over.max()) <= 0


# (more than two rows of larger weights go to the tensor cores)
@pytest.mark.parametrize("n,k,m", [(n, k, m) for n, k, most in ((262144, 128, 4), (262139, 256, 4), (77840, 5120, 2),
                                                               (46000, 8704, 2)) for m in range(1, most + 1)] +
                         [(80000, 128, 5), (80000, 128, 8), (151936, 8192, 1)])
def test_rounds(api, n, k, m):
    gen = torch.Generator("cuda").manual_seed(n + m)
    x = torch.randn((m, k), generator=gen, device="cuda").half()
    q = weights(api, gen, n, k)
    bias = torch.randn(n, generator=gen, device="cuda").half()
    res = torch.randn((m, n), generator=gen, device="cuda").half()
    s, a = products(api, q, x.double())
    y = api.w4a16_gemm_mxfp4(x, *q)
    hold(y, s, ref.sum_error(a, k))
    for _ in range(5):
        assert torch.equal(api.w4a16_gemm_mxfp4(x, *q), y)
    z = res.clone()
    api.w4a16_gemm_mxfp4(x, *q, bias=bias, residual=z, out=z)
    t, b = s + bias.double() + res.double(), a + bias.double().abs() + res.double().abs()
    hold(z, t, ref.sum_error(b, k))


@pytest.mark.parametrize("n,k,m", [(40000, 128, 1), (40000, 384, 2), (29568, 8192, 1), (29561, 8192, 2), (100003, 128, 3)])
def test_rounds_of_a_gated_pair(api, n, k, m):
    gen = torch.Generator("cuda").manual_seed(n + m)
    x = torch.randn((m, k), generator=gen, device="cuda").half()
    g, u = weights(api, gen, n, k), weights(api, gen, n, k)
    (gs, ga), (us, ua) = products(api, g, x.double()), products(api, u, x.double())
    eg, eu = ref.sum_error(ga, k), ref.sum_error(ua, k)
    silu = gs * torch.sigmoid(gs)
    y = api.w4a16_gemm_silu_mul_mxfp4(x, *g, *u)
    hold(y, silu * us, 1.1 * eg * (us.abs() + eu) + silu.abs() * eu + 2.0 ** -21 * (silu * us).abs())
    for _ in range(5):
        assert torch.equal(api.w4a16_gemm_silu_mul_mxfp4(x, *g, *u), y)
