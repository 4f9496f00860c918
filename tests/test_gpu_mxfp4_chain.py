"""Layer after layer on a residual stream that is updated in place, each call started
under the one before it: the same bits as with the GPU waited for after every call.
(What a call reads, it and the call before it may have read in another state: the
stream's rows as residual, and through the same caches as x.)"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as a
    return a


def layers(api, h, i, count, gen):
    def w(n, k):
        return api.mxfp4_quantize((0.5 * torch.randn((n, k), generator=gen, device="cuda") / k ** 0.5).half())
    return [(w(i, h), w(i, h), w(h, i), w(h, h)) for _ in range(count)]


def chain(api, x, ws, space, four, after):
    """x through all layers, in place."""
    for gate, up, down, o in ws:
        t = api.w4a16_gemm_mxfp4(x, *o, workspace=space)
        after()
        api.w4a16_gemm_mxfp4(t, *o, residual=x, out=x, workspace=space)
        after()
        t = api.w4a16_gemm_silu_mul_mxfp4(x, *gate, *up, workspace=space)
        after()
        if four:
            q = api.mxfp4_quantize(t)
            after()
            api.w4a4_gemm_mxfp4(*q, *down, residual=x, out=x, workspace=space)
        else:
            api.w4a16_gemm_mxfp4(t, *down, residual=x, out=x, workspace=space)
        after()
    return x


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("m,h,i", [(1, 512, 1152), (1, 3584, 2432), (2, 896, 2432), (4, 512, 1152), (8, 896, 1152),
                                   (33, 512, 2432), (130, 896, 1152)])
def test_chain(api, m, h, i, four):
    gen = torch.Generator("cuda").manual_seed(m + h)
    ws = layers(api, h, i, 6, gen)
    space = api.mxfp4_workspace()
    x = torch.randn((m, h), generator=gen, device="cuda").half()
    want = chain(api, x.clone(), ws, space, four, torch.cuda.synchronize)
    assert bool(torch.isfinite(want).all())
    for _ in range(20):
        assert torch.equal(chain(api, x.clone(), ws, space, four, lambda: None), want)
    y = x.clone()
    chain(api, y, ws, space, four, lambda: None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(api, y, ws, space, four, lambda: None)
    for _ in range(20):
        y.copy_(x)
        graph.replay()
        assert torch.equal(y, want)
