"""Every way in which the MXFP4 tensor-core products deal their tiles: each tile shape
with one tile a CTA, with several (whose sums and buffers are used again), split along
K, and split behind whole ones; rows of y that start on 16 bytes and rows that do not;
with and without bias and residual.  The plan that a case is meant for is asserted, so
that a changed rule cannot drop it.  All outputs against 64 bits on the GPU."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

SMS = 152
A16, SILU, A4 = 0, 1, 2
FORMS = {"one": lambda w, s: 0 < w <= SMS and s == 0, "two": lambda w, s: SMS < w <= 2 * SMS and s == 0,
         "more": lambda w, s: w > 2 * SMS and s == 0, "split": lambda w, s: w == 0 and s > 0,
         "both": lambda w, s: w >= SMS and s > 0}


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as a
    return a


def plan(kind, m, n, k, space):
    from w4a16_decode_paged_gb300 import _lib
    p = (ctypes.c_int32 * 7)()
    assert _lib.load().w4a16_debug_mxfp4_plan(kind, m, k, n, space, 0, p) == 0
    return list(p)


def planned(kind, m, n, k, space, tile, form):
    p = plan(kind, m, n, k, space)
    assert p[0] == 1 and (p[1], p[2]) == tile and FORMS[form](p[3], p[4]), p
    return p


def matrix(api, gen, n, k):
    q = api.mxfp4_quantize((torch.randn((n, k), generator=gen, device="cuda") * torch.rand((n, 1), generator=gen, device="cuda")
                            / k ** 0.5).half())
    return q, api.mxfp4_dequantize(*q).double()


def activations(gen, m, k):
    x = torch.randn((m, k), generator=gen, device="cuda") * torch.where(
        torch.rand(k, generator=gen, device="cuda") < 1 / 64, 8.0, 1.0)
    return x.half()


def hold(y, want, err):
    over = (y.double() - want).abs() - err - ((want.abs() + err) * 2.0 ** -11).clamp(min=2.0 ** -25)
    assert bool(torch.isfinite(y).all()) and float(over.max()) <= 0


def check_all(call, gen, xv, wv, m, n, k, spaces):
    """call(bias, residual, out, workspace, err) with each of bias and residual, alone, together
    and in place, against xv . wv^T in 64 bits."""
    s, a = xv @ wv.T, xv.abs() @ wv.abs().T
    bias = torch.randn(n, generator=gen, device="cuda").half()
    res = torch.randn((m, n), generator=gen, device="cuda").half()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b, r = bias.double(), res.double()
    for space in spaces:
        for add in ((), (b,), (r,), (b, r)):
            y = torch.full((m, n), float("nan"), dtype=torch.float16, device="cuda")
            held = r if any(t is r for t in add) else None
            if held is not None and len(add) == 2:
                y = res.clone()
            call(bias if any(t is b for t in add) else None, None if held is None else y if len(add) == 2 else res, y,
                 space, err)
            want, mag = s, a
            for t in add:
                want, mag = want + t, mag + t.abs()
            hold(y, want, ref.sum_error(mag, k))
    assert int(err.item()) == 0


@pytest.mark.parametrize("tile,form,m,n,k", [
    ((256, 192), "one", 132, 21800, 384), ((256, 192), "one", 133, 21619, 384),
    ((256, 192), "two", 413, 24408, 384), ((256, 192), "two", 1055, 11027, 384),
    ((256, 192), "two", 397, 22739, 128), ((256, 192), "more", 915, 19720, 128), ((256, 192), "more", 930, 19667, 128),
    ((256, 192), "split", 4898, 160, 7168), ((256, 192), "split", 3605, 267, 6272),
    ((256, 192), "both", 1472, 5016, 6656), ((256, 192), "both", 2263, 3275, 6656),
    ((128, 256), "one", 1, 19568, 384), ((128, 256), "one", 1, 19475, 384),
    ((128, 256), "two", 261, 21072, 384), ((128, 256), "two", 258, 20251, 384),
    ((128, 256), "more", 520, 20384, 384), ((128, 256), "more", 551, 20699, 384), ((128, 256), "more", 536, 20171, 128),
    ((128, 256), "split", 1, 5016, 6784), ((128, 256), "split", 1, 3323, 10368),
    ((128, 256), "both", 129, 20048, 7680), ((128, 256), "both", 131, 19619, 6656),
    ((128, 192), "one", 1, 19544, 896), ((128, 192), "one", 1, 19651, 896),
    ((128, 192), "two", 2896, 2496, 384), ((128, 192), "two", 131, 19691, 1408),
    ((128, 192), "more", 4096, 3584, 1024), ((128, 192), "more", 409, 19627, 384), ((128, 192), "more", 408, 19675, 128),
    ((128, 192), "split", 1, 4952, 4864), ((128, 192), "split", 1, 4011, 5248),
    ((128, 192), "both", 4879, 928, 3712), ((128, 192), "both", 2264, 2059, 3712),
    ((128, 128), "one", 300, 5000, 896), ((128, 128), "one", 299, 4999, 896),
    ((128, 128), "two", 4875, 784, 384), ((128, 128), "two", 4936, 771, 384),
    ((128, 128), "more", 272, 15256, 384), ((128, 128), "more", 2050, 7001, 640), ((128, 128), "more", 561, 15395, 128),
    ((128, 128), "split", 1, 8, 2944), ((128, 128), "split", 1, 11, 2944),
    ((128, 128), "both", 1, 20008, 9216), ((128, 128), "both", 1, 19539, 9472)])
def test_a4_tiles(api, tile, form, m, n, k):
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    x = api.mxfp4_quantize(activations(gen, m, k))
    w, wv = matrix(api, gen, n, k)
    room = 64 << 20
    planned(A4, m, n, k, room, tile, form)
    spaces = [torch.zeros(room, dtype=torch.uint8, device="cuda")]
    if form in ("split", "both"):
        spaces.append(spaces[0][:0])                               # the same without room to split
        assert plan(A4, m, n, k, 0)[5] == 1
    check_all(lambda b, r, y, ws, e: api.w4a4_gemm_mxfp4(*x, *w, bias=b, residual=r, out=y, workspace=ws, err_flag=e), gen,
              api.mxfp4_dequantize(*x).double(), wv, m, n, k, spaces)


def test_a4_long_prompt(api):
    """4096 rows onto the residual stream: two tiles of 256 x 192 a CTA, 74 steps each."""
    m, n, k = 4096, 3584, 18944
    gen = torch.Generator("cuda").manual_seed(7)
    x = api.mxfp4_quantize(activations(gen, m, k))
    w, wv = matrix(api, gen, n, k)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    planned(A4, m, n, k, ws.numel(), (256, 192), "two")
    bias = torch.randn(n, generator=gen, device="cuda").half()
    res = torch.randn((m, n), generator=gen, device="cuda").half()
    y = api.w4a4_gemm_mxfp4(*x, *w, bias=bias, residual=res, workspace=ws)
    rows = torch.unique(torch.cat([torch.randint(0, m, (300,), generator=gen, device="cuda"),
                                   torch.tensor([0, 127, 128, 255, 256, 2047, 2048, 4095], device="cuda")]))
    xv = api.mxfp4_dequantize(*x)[rows].double()
    want = xv @ wv.T + bias.double() + res[rows].double()
    mag = xv.abs() @ wv.abs().T + bias.double().abs() + res[rows].double().abs()
    hold(y[rows], want, ref.sum_error(mag, k))


@pytest.mark.parametrize("tile,form,m,n,k", [
    ((32, 256), "both", 20, 40000, 1280), ((32, 256), "both", 20, 39997, 1280), ((32, 256), "two", 32, 60001, 384),
    ((64, 256), "both", 50, 42000, 2048), ((64, 256), "both", 33, 40003, 1280), ((64, 256), "two", 64, 60008, 384),
    ((128, 256), "both", 200, 20000, 1536), ((128, 256), "both", 129, 19999, 1536), ((128, 256), "more", 300, 40001, 256)])
def test_a16_tiles(api, tile, form, m, n, k):
    """Whole tiles followed by parts of split ones in the same CTA, whose first steps are
    expanded under the tile before."""
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    x = activations(gen, m, k)
    w, wv = matrix(api, gen, n, k)
    ws = api.mxfp4_workspace(m, k, n)
    assert (ws.numel() > 8192) == (form == "both")
    planned(A16, m, n, k, ws.numel(), tile, form)
    check_all(lambda b, r, y, ws, e: api.w4a16_gemm_mxfp4(x, *w, bias=b, residual=r, out=y, workspace=ws, err_flag=e), gen,
              x.double(), wv, m, n, k, [ws])


@pytest.mark.parametrize("tile,form,m,n,k", [
    ((32, 256), "both", 20, 40000, 1280), ((32, 256), "both", 20, 39997, 1280),
    ((64, 256), "both", 50, 42000, 2048), ((64, 256), "both", 50, 41999, 2048),
    ((128, 256), "both", 200, 20000, 1536), ((128, 256), "both", 200, 19999, 1536)])
def test_silu_tiles(api, tile, form, m, n, k):
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    x = activations(gen, m, k)
    (g, gv), (u, uv) = matrix(api, gen, n, k), matrix(api, gen, n, k)
    ws = api.mxfp4_workspace(m, k, n, "silu")
    planned(SILU, m, n, k, ws.numel(), tile, form)
    xv, err = x.double(), torch.zeros(1, dtype=torch.int32, device="cuda")
    gs, us = xv @ gv.T, xv @ uv.T
    eg, eu = (ref.sum_error(xv.abs() @ v.abs().T, k) for v in (gv, uv))
    silu = gs * torch.sigmoid(gs)
    y = api.w4a16_gemm_silu_mul_mxfp4(x, *g, *u, workspace=ws, err_flag=err)
    hold(y, silu * us, 1.1 * eg * (us.abs() + eu) + silu.abs() * eu + 2.0 ** -21 * (silu * us).abs())
    assert int(err.item()) == 0


def test_rounds_are_planned(api):
    """What the tests of several rounds of the stream kernel are meant for."""
    for kind, m, n, k, cluster in ((A16, 1, 262144, 128, False), (A16, 4, 262139, 256, False), (A16, 8, 80000, 128, False),
                                   (A16, 2, 77840, 5120, True), (A16, 1, 151936, 8192, True), (SILU, 1, 40000, 128, False),
                                   (SILU, 2, 40000, 384, False), (SILU, 1, 29568, 8192, True), (SILU, 2, 29561, 8192, True),
                                   (SILU, 3, 100003, 128, False)):
        p = plan(kind, m, n, k, 0)
        assert p[0] == 0 and p[4] >= 2 and (p[1] > 1) == cluster, (kind, m, n, k, p)
