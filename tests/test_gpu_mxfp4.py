"""MXFP4 matrices on the GPU: quantising and reading back bit for bit, the products
against the 64-bit formula at every kind of tile edge, scales, NaN, streams, graphs
and workspaces."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as a
    return a


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


def host(t):
    return t.cpu().numpy()


def matrix(code, byte):
    """An MXFP4 matrix on the GPU; bytes of rows past the last are NaN scales."""
    return dev(ref.pack(code)), dev(ref.tiles(byte, fill=255))


def random_matrix(rng, n, k):
    code, byte = ref.quantise(ref.weights(rng, n, k))
    return matrix(code, byte), ref.values(code, byte)


def activations(rng, m, k):
    x = rng.standard_normal((m, k)) * np.where(rng.random(k) < 1 / 64, 8.0, 1.0)
    return x.astype(np.float16)


# --------------------------------------------------------------------------- quantising
@pytest.mark.parametrize("m,k", [(1, 128), (1, 3584), (3, 256), (31, 896), (33, 384), (127, 640), (129, 2432), (300, 1152),
                                 (1025, 128)])
def test_quantise_and_read_back(api, m, k):
    rng = np.random.default_rng(m * 7 + k)
    x = activations(rng, m, k)
    x *= np.exp2(rng.integers(-24, 12, (m, k // 32))).repeat(32, 1).astype(np.float16)   # blocks of every size
    x[rng.random((m, k)) < 0.05] = 0
    c, s = api.mxfp4_quantize(dev(x))
    code, byte = ref.quantise(x)
    assert np.array_equal(ref.unpack(host(c)), code)
    assert np.array_equal(ref.untiled(host(s), m), byte)
    y = host(api.mxfp4_dequantize(c, s)).astype(np.float64)
    assert np.array_equal(y, ref.values(code, byte), equal_nan=True)


def test_quantise_every_fp16_number(api):
    """Each of the 65536 bit patterns as a block's largest, beside its halves."""
    bits = np.arange(65536, dtype=np.uint16).view(np.float16)
    x = np.zeros((65536, 128), np.float16)
    with np.errstate(all="ignore"):
        for j, f in enumerate((1, .5, .7, -.35, .2, -.125, .0625, .9)):
            x[:, j] = (bits.astype(np.float32) * f).astype(np.float16)
            x[:, 40 + j] = bits if j == 0 else 0
            x[:, 71 - j] = bits if j < 2 else 0
    c, s = api.mxfp4_quantize(dev(x))
    code, byte = ref.quantise(x)
    assert np.array_equal(ref.unpack(host(c)), code) and np.array_equal(ref.untiled(host(s), 65536), byte)
    y, want = host(api.mxfp4_dequantize(c, s)).astype(np.float64), ref.values(code, byte)
    assert np.array_equal(y, want, equal_nan=True) and np.isnan(want).any()


def test_quantise_leaves_the_rest_alone(api):
    m, k = 37, 256
    s = torch.full((1, 2, 512), 77, dtype=torch.uint8, device="cuda")
    x = activations(np.random.default_rng(1), m, k)
    api.mxfp4_quantize(dev(x), scales=s)
    t = host(s)
    rows = ref.untiled(t, 128)
    assert (rows[m:] == 77).all() and np.array_equal(rows[:m], ref.quantise(x)[1])


def test_read_back_of_any_scale_byte(api):
    """Every byte with every code, rounded to fp16 once."""
    byte = np.arange(256).repeat(4).reshape(256, 4).astype(np.uint8)
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 8))
    y = host(api.mxfp4_dequantize(*matrix(code, byte)))
    with np.errstate(over="ignore"):
        want = ref.values(code, byte).astype(np.float16)
    assert np.array_equal(y[1:], want[1:], equal_nan=True) and not y[0].any()


# --------------------------------------------------------------------------- products
SHAPES = [(1, 1, 128), (1, 512, 3584), (1, 513, 128), (2, 33, 256), (3, 127, 384), (4, 128, 896), (5, 129, 512), (6, 16, 1152),
          (7, 2432, 896), (8, 640, 2432), (9, 255, 640), (15, 31, 768), (16, 17, 1408), (17, 300, 256), (31, 1, 128),
          (32, 512, 1152), (33, 257, 384), (48, 96, 640), (63, 130, 256), (64, 64, 1024), (65, 200, 128), (96, 384, 896),
          (127, 129, 512), (128, 256, 384), (129, 127, 640), (191, 500, 256), (192, 128, 128), (193, 65, 1280),
          (255, 385, 384), (256, 256, 256), (257, 641, 128), (300, 1000, 384), (513, 130, 256), (1000, 7, 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_a16(api, m, n, k):
    rng = np.random.default_rng(m + 1000 * n + k)
    x, (w, wv) = activations(rng, m, k), random_matrix(rng, n, k)
    bias = (0.1 * rng.standard_normal(n)).astype(np.float16)
    res = rng.standard_normal((m, n)).astype(np.float16)
    xd = dev(x)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    y = api.w4a16_gemm_mxfp4(xd, *w, workspace=ws)
    ref.check_product(host(y), x.astype(np.float64), wv, what="plain")
    y = api.w4a16_gemm_mxfp4(xd, *w, bias=dev(bias), residual=dev(res), workspace=ws)
    ref.check_product(host(y), x.astype(np.float64), wv, bias.astype(np.float64), res.astype(np.float64), "bias, residual")
    # no room to split; the residual's own memory as the output
    y = dev(res)
    api.w4a16_gemm_mxfp4(xd, *w, residual=y, out=y, workspace=ws[:0])
    ref.check_product(host(y), x.astype(np.float64), wv, None, res.astype(np.float64), "in place, no workspace")
    assert not ws[:8192].any()


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_silu(api, m, n, k):
    rng = np.random.default_rng(m + 1000 * n + k + 1)
    x, (g, gv), (u, uv) = activations(rng, m, k), random_matrix(rng, n, k), random_matrix(rng, n, k)
    y = api.w4a16_gemm_silu_mul_mxfp4(dev(x), *g, *u)
    ref.check_silu(host(y), x.astype(np.float64), gv, uv)
    y = api.w4a16_gemm_silu_mul_mxfp4(dev(x), *g, *u, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    ref.check_silu(host(y), x.astype(np.float64), gv, uv, "no workspace")


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_a4(api, m, n, k):
    rng = np.random.default_rng(m + 1000 * n + k + 2)
    code, byte = ref.quantise(activations(rng, m, k))
    x, xv = matrix(code, byte), ref.values(code, byte)
    w, wv = random_matrix(rng, n, k)
    bias = (0.1 * rng.standard_normal(n)).astype(np.float16)
    res = rng.standard_normal((m, n)).astype(np.float16)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    ref.check_product(host(api.w4a4_gemm_mxfp4(*x, *w, workspace=ws)), xv, wv, what="plain")
    y = dev(res)
    api.w4a4_gemm_mxfp4(*x, *w, bias=dev(bias), residual=y, out=y, workspace=ws)
    ref.check_product(host(y), xv, wv, bias.astype(np.float64), res.astype(np.float64), "bias, residual in place")
    y = api.w4a4_gemm_mxfp4(*x, *w, workspace=ws[:256])
    ref.check_product(host(y), xv, wv, what="no workspace")
    assert not ws[:8192].any()


@pytest.mark.parametrize("m", [1, 4, 5, 8, 16, 32, 64, 128, 130])
@pytest.mark.parametrize("call", ["a16", "silu", "a4"])
def test_each_weight_meets_its_own_x(api, call, m):
    """x picks one element of each row of W (a one-hot x): codes and scales all
    different along K and N, results exact."""
    n, k = 272, 1280
    rng = np.random.default_rng(m)
    code = rng.integers(0, 16, (n, k)).astype(np.uint8)
    byte = rng.integers(117, 130, (n, k // 32)).astype(np.uint8)
    w, wv = matrix(code, byte), ref.values(code, byte)
    at = rng.integers(0, k, m)
    x = np.zeros((m, k), np.float16)
    x[np.arange(m), at] = 1
    if call == "a4":
        c, b = ref.quantise(x)
        got = host(api.w4a4_gemm_mxfp4(*matrix(c, b), *w))
    elif call == "a16":
        got = host(api.w4a16_gemm_mxfp4(dev(x), *w))
    else:
        one = matrix(np.full((n, k), 2, np.uint8), np.full((n, k // 32), 127, np.uint8))    # G = 1: silu(1) * u
        got = host(api.w4a16_gemm_silu_mul_mxfp4(dev(x), *one, *w)).astype(np.float64)
        s = 1 / (1 + np.exp(-1.0))
        assert (np.abs(got - s * wv[:, at].T) <= ref.half_step(s * wv[:, at].T) * (1 + 2.0 ** -10)).all()
        return
    assert np.array_equal(got.astype(np.float64), wv[:, at].T)


@pytest.mark.parametrize("m", [1, 7, 32, 130])
def test_scales_at_both_ends(api, m):
    """Weights from 2^-24 to 49152 beside one another: fp16's whole range."""
    rng = np.random.default_rng(3)
    n, k = 96, 256
    code = rng.integers(0, 16, (n, k)).astype(np.uint8)
    byte = rng.choice([104, 105, 113, 127, 139, 140], (n, k // 32)).astype(np.uint8)
    wv = ref.values(code, byte)
    x = (rng.standard_normal((m, k)) * 2.0 ** -14).astype(np.float16)
    ref.check_product(host(api.w4a16_gemm_mxfp4(dev(x), *matrix(code, byte))), x.astype(np.float64), wv)
    small = np.full((n, k // 32), 104, np.uint8)                      # all small: nothing is lost beside larger ones
    x = (rng.standard_normal((m, k)) * 1000).astype(np.float16)
    ref.check_product(host(api.w4a16_gemm_mxfp4(dev(x), *matrix(code, small))), x.astype(np.float64), ref.values(code, small))
    tiny = rng.integers(0, 104, (n, k // 32)).astype(np.uint8)        # such blocks count as themselves or as zero
    y = host(api.w4a16_gemm_mxfp4(dev(x), *matrix(code, tiny))).astype(np.float64)
    most = np.abs(x.astype(np.float64)) @ np.abs(ref.values(code, tiny)).T
    assert (np.abs(y) <= most * (1 + 2.0 ** -10) + 2.0 ** -24).all()
    y = host(api.w4a16_gemm_mxfp4(dev(x), *matrix(code & 8, tiny)))   # zero codes under any of them: zero
    assert not y.any()


@pytest.mark.parametrize("m", [1, 33, 200])
def test_a4_takes_any_scale(api, m):
    rng = np.random.default_rng(5)
    n, k = 130, 384
    cx, cw = rng.integers(0, 16, (m, k)).astype(np.uint8), rng.integers(0, 16, (n, k)).astype(np.uint8)
    # bytes far apart whose products are of ordinary size: each block's two bytes add up to about 254
    bx = np.tile(rng.integers(30, 225, k // 32), (m, 1)) + rng.integers(-2, 3, (m, k // 32))
    bw = 254 - np.tile(bx[:1], (n, 1)) + rng.integers(-2, 3, (n, k // 32))
    bx, bw = bx.astype(np.uint8), bw.astype(np.uint8)
    y = host(api.w4a4_gemm_mxfp4(*matrix(cx, bx), *matrix(cw, bw)))
    ref.check_product(y, ref.values(cx, bx), ref.values(cw, bw))


@pytest.mark.parametrize("m", [1, 5, 33, 200])
@pytest.mark.parametrize("call", ["a16", "silu", "a4"])
def test_nan_stays_in_its_row(api, call, m):
    rng = np.random.default_rng(9)
    n, k = 150, 512
    x = activations(rng, m, k)
    code, byte = ref.quantise(ref.weights(rng, n, k))
    code[code & 7 == 0] = 1                                          # no zero weight: inf * 0 would be NaN as well
    byte[17, 3] = 255
    x[m // 2, 100] = np.nan if m % 2 else np.inf
    w = matrix(code, byte)
    if call == "a4":
        y = api.w4a4_gemm_mxfp4(*api.mxfp4_quantize(dev(x)), *w)
    elif call == "a16":
        y = api.w4a16_gemm_mxfp4(dev(x), *w)
    else:
        y = api.w4a16_gemm_silu_mul_mxfp4(dev(x), *w, *w)
    fine = np.isfinite(host(y))
    want = np.ones((m, n), bool)
    want[m // 2], want[:, 17] = False, False
    if call == "silu" and m % 2 == 0:                                # silu(-inf) * -inf: 0 * inf, or inf: not finite either
        assert not fine[~want].any()
    assert np.array_equal(fine, want)
    assert np.isnan(host(y)[:, 17]).all()


# --------------------------------------------------------------------------- use
def _mlp(api, x, w, ws):
    """A decode MLP's projections in one run: quantised weights straight from the quantiser."""
    y = api.w4a16_gemm_silu_mul_mxfp4(x, *w["g"], *w["u"], workspace=ws)
    return api.w4a16_gemm_mxfp4(y, *w["d"], residual=x, workspace=ws)


@pytest.mark.parametrize("m", [1, 8, 40, 256])
def test_a_run_of_them_equals_its_parts(api, m):
    """Weights quantised on the GPU, read back, and used at once, the MLP in 16 and
    in 4 bits; captured and replayed with new inputs, it gives the same bits."""
    rng = np.random.default_rng(m)
    h, i = 512, 1152
    w = {p: ref.weights(rng, *s) for p, s in (("g", (i, h)), ("u", (i, h)), ("d", (h, i)))}
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    x = activations(rng, m, h)
    q, dw = {}, {p: dev(a) for p, a in w.items()}
    for p in w:
        q[p] = api.mxfp4_quantize(dw[p])
    xd = dev(x)
    q["d2"] = api.mxfp4_quantize(dw["d"])
    first = api.w4a16_gemm_mxfp4(dev(np.ones((m, i), np.float16)), *q["d2"], workspace=ws)   # right behind the quantiser
    vals = {p: host(api.mxfp4_dequantize(*q[p])).astype(np.float64) for p in w}
    for p in w:
        assert np.array_equal(vals[p], ref.values(*ref.quantise(w[p])))
    ref.check_product(host(first), np.ones((m, i)), vals["d"])
    y = api.w4a16_gemm_silu_mul_mxfp4(xd, *q["g"], *q["u"], workspace=ws)
    ref.check_silu(host(y), x.astype(np.float64), vals["g"], vals["u"])
    z = api.w4a16_gemm_mxfp4(y, *q["d"], residual=xd, workspace=ws)
    ref.check_product(host(z), host(y).astype(np.float64), vals["d"], None, x.astype(np.float64))
    y4 = api.mxfp4_quantize(y)
    z4 = api.w4a4_gemm_mxfp4(*y4, *q["d"], residual=xd, workspace=ws)
    ref.check_product(host(z4), host(api.mxfp4_dequantize(*y4)).astype(np.float64), vals["d"], None, x.astype(np.float64))

    def run():
        y = api.w4a16_gemm_silu_mul_mxfp4(xd, *q["g"], *q["u"], workspace=ws)
        return api.w4a16_gemm_mxfp4(y, *q["d"], residual=xd, workspace=ws), api.w4a4_gemm_mxfp4(
            *api.mxfp4_quantize(y), *q["d"], residual=xd, workspace=ws)
    assert torch.equal(run()[0], z) and torch.equal(run()[1], z4)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    x2 = dev(activations(rng, m, h))
    for new in (xd.clone(), x2, xd.clone()):
        xd.copy_(new)
        graph.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, run()))


@pytest.mark.parametrize("m", [1, 16, 100])
def test_on_another_stream(api, m):
    """A call given a stream works there, and so do the tensors it makes."""
    rng = np.random.default_rng(m)
    n, k = 300, 896
    x = activations(rng, m, k)
    w, wv = random_matrix(rng, n, k)
    xd, s = dev(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    y = api.w4a16_gemm_mxfp4(xd, *w, stream=s)
    q = api.mxfp4_quantize(xd, stream=s)
    y4 = api.w4a4_gemm_mxfp4(*q, *w, stream=s)
    xr = api.mxfp4_dequantize(*q, stream=s)
    ys = api.w4a16_gemm_silu_mul_mxfp4(xd, *w, *w, stream=s)
    s.synchronize()
    ref.check_product(host(y), x.astype(np.float64), wv)
    ref.check_product(host(y4), host(xr).astype(np.float64), wv)
    ref.check_silu(host(ys), x.astype(np.float64), wv, wv)


def test_two_calls_at_once_with_a_workspace_each(api):
    rng = np.random.default_rng(0)
    n, k = 384, 2432
    w, wv = random_matrix(rng, n, k)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [api.mxfp4_workspace(24, k, n) for _ in streams]
    xs = [activations(rng, 24, k) for _ in streams]
    xd = [dev(x) for x in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        ys = [api.w4a16_gemm_mxfp4(xd[i], *w, workspace=spaces[i], stream=streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        ref.check_product(host(y), x.astype(np.float64), wv)


def test_rows_past_the_last_are_left_alone(api):
    rng = np.random.default_rng(4)
    n, k = 131, 256
    w, _ = random_matrix(rng, n, k)
    for m in (1, 3, 6, 33, 129):
        buf = torch.full((m * n + 4096,), 7.0, dtype=torch.float16, device="cuda")
        y = buf[:m * n].view(m, n)
        x = dev(activations(rng, m, k))
        api.w4a16_gemm_mxfp4(x, *w, out=y)
        assert (buf[m * n:] == 7).all()
        api.w4a16_gemm_silu_mul_mxfp4(x, *w, *w, out=y)
        assert (buf[m * n:] == 7).all()
        api.w4a4_gemm_mxfp4(*api.mxfp4_quantize(x), *w, out=y)
        assert (buf[m * n:] == 7).all()


def test_same_bits_each_time(api):
    """Split sums are joined in one order."""
    rng = np.random.default_rng(8)
    for m, n, k in ((1, 512, 3584), (7, 256, 3584), (32, 384, 3584), (100, 256, 3584)):
        x, (w, _) = dev(activations(rng, m, k)), random_matrix(rng, n, k)
        ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        q = api.mxfp4_quantize(x)
        y, y4 = api.w4a16_gemm_mxfp4(x, *w, workspace=ws), api.w4a4_gemm_mxfp4(*q, *w, workspace=ws)
        for _ in range(20):
            assert torch.equal(api.w4a16_gemm_mxfp4(x, *w, workspace=ws), y)
            assert torch.equal(api.w4a4_gemm_mxfp4(*q, *w, workspace=ws), y4)


@pytest.mark.parametrize("call,m,n,k", [("a16", 1, 3584, 18944), ("a16", 32, 3584, 18944), ("silu", 1, 18944, 3584),
                                        ("silu", 32, 18944, 3584), ("a16", 2048, 3584, 3584), ("a4", 512, 18944, 3584),
                                        ("a4", 700, 3584, 18944)])
def test_full_size(api, call, m, n, k):
    """The projections of the model shape the benchmark runs, against 64 bits on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = (rnd(m, k) * torch.where(torch.rand(k, generator=gen, device="cuda") < 1 / 64, 8.0, 1.0)).half()
    ws = [(rnd(n, k) / k ** 0.5).half() for _ in range(2 if call == "silu" else 1)]
    q = [api.mxfp4_quantize(w) for w in ws]
    wv = [api.mxfp4_dequantize(*p).double() for p in q]
    if call == "silu":
        y = api.w4a16_gemm_silu_mul_mxfp4(x, *q[0], *q[1])
        g, u = x.double() @ wv[0].T, x.double() @ wv[1].T
        want = g * torch.sigmoid(g) * u
    else:
        xq = api.mxfp4_quantize(x)
        xv = api.mxfp4_dequantize(*xq) if call == "a4" else x
        y = api.w4a4_gemm_mxfp4(*xq, *q[0]) if call == "a4" else api.w4a16_gemm_mxfp4(x, *q[0])
        want = xv.double() @ wv[0].T
    rms = float(((y.double() - want) ** 2).mean().sqrt() / (want ** 2).mean().sqrt())
    assert rms <= 2.0 ** -10 / 12 ** 0.5 * 1.02, rms
    assert float(((y.double() - want).abs() / (want.abs() + float((want ** 2).mean().sqrt()))).max()) <= 2.0 ** -10


def test_workspace_of_any_contents(api):
    """Parts are written before they are read, and the block that the other split-K
    GEMMs keep their counters in is left alone: they share a workspace in turn."""
    rng = np.random.default_rng(2)
    m, n, k = 40, 512, 3584
    x, (w, wv) = activations(rng, m, k), random_matrix(rng, n, k)
    xd = dev(x)
    q = api.mxfp4_quantize(xd)
    assert api.mxfp4_workspace(m, k, n).numel() > 8192 and api.mxfp4_workspace(m, k, n, "a4").numel() > 8192
    for call, xv in (("a16", x.astype(np.float64)), ("a4", host(api.mxfp4_dequantize(*q)).astype(np.float64))):
        ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
        y = api.w4a16_gemm_mxfp4(xd, *w, workspace=ws) if call == "a16" else api.w4a4_gemm_mxfp4(*q, *w, workspace=ws)
        ref.check_product(host(y), xv, wv)
        assert (ws[:8192] == 255).all() and not (ws[8192:65536] == 255).all()
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    qw = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), device="cuda", dtype=torch.int32)
    sc = torch.full((n, k // 128), 0.01, dtype=torch.float16, device="cuda")
    want = api.w4a16_gemm(xd[:32], qw, sc)
    for _ in range(3):
        ref.check_product(host(api.w4a16_gemm_mxfp4(xd, *w, workspace=ws)), x.astype(np.float64), wv)
        assert torch.equal(api.w4a16_gemm(xd[:32].contiguous(), qw, sc, workspace=ws), want)


@pytest.mark.parametrize("m", [1, 6, 40])
def test_the_checked_path_is_the_native_one(api, m):
    """With a stream given the binding checks in Python, without one natively."""
    rng = np.random.default_rng(m)
    n, k = 150, 640
    x, (w, _), (u, _) = dev(activations(rng, m, k)), random_matrix(rng, n, k), random_matrix(rng, n, k)
    bias, res = dev(rng.standard_normal(n).astype(np.float16)), dev(rng.standard_normal((m, n)).astype(np.float16))
    ws, here = api.mxfp4_workspace(m, k, n), torch.cuda.current_stream()
    a, b = api.mxfp4_quantize(x), api.mxfp4_quantize(x, stream=here)
    assert torch.equal(a[0], b[0]) and torch.equal(api.mxfp4_dequantize(*a), api.mxfp4_dequantize(*b, stream=here))
    for args in (dict(), dict(bias=bias), dict(residual=res), dict(bias=bias, residual=res)):
        out = torch.empty((m, n), dtype=torch.float16, device="cuda")
        y = api.w4a16_gemm_mxfp4(x, *w, workspace=ws, **args)
        assert torch.equal(y, api.w4a16_gemm_mxfp4(x, *w, workspace=ws, stream=here, **args))
        assert api.w4a16_gemm_mxfp4(x, *w, workspace=ws, out=out, **args) is out and torch.equal(out, y)
        y = api.w4a4_gemm_mxfp4(*a, *w, workspace=ws, **args)
        assert torch.equal(y, api.w4a4_gemm_mxfp4(*a, *w, workspace=ws, stream=here, **args))
    y = api.w4a16_gemm_silu_mul_mxfp4(x, *w, *u, workspace=ws)
    assert torch.equal(y, api.w4a16_gemm_silu_mul_mxfp4(x, *w, *u, workspace=ws, stream=here))
    wu = (w[0].view(torch.uint32), w[1])
    assert torch.equal(api.w4a16_gemm_mxfp4(x, *wu, workspace=ws), api.w4a16_gemm_mxfp4(x, *w, workspace=ws))
    with pytest.raises(ValueError, match="codes"):
        api.w4a16_gemm_mxfp4(x, w[0][:, :-16].contiguous(), w[1], workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        api.w4a16_gemm_mxfp4(x, *w, workspace=ws.view(torch.int8))


def _close(y, xv, wv, k):
    """y against xv . wv^T in 64 bits on the GPU: the bounds of mxfp4_ref.check_product."""
    s, a = xv @ wv.T, xv.abs() @ wv.abs().T
    err = ref.sum_error(a, k)
    over = (y.double() - s).abs() - err - ((s.abs() + err) * 2.0 ** -11).clamp(min=2.0 ** -25)
    assert bool(torch.isfinite(y).all()) and float(over.max()) <= 0


@pytest.mark.parametrize("m", [1, 3, 4, 7, 20, 200])
def test_the_longest_k(api, m):
    rng = np.random.default_rng(m)
    n, k = 24, 131072
    x, (w, wv) = activations(rng, m, k), random_matrix(rng, n, k)
    xd, wv = dev(x), dev(wv)
    _close(api.w4a16_gemm_mxfp4(xd, *w), xd.double(), wv, k)
    q = api.mxfp4_quantize(xd)
    _close(api.w4a4_gemm_mxfp4(*q, *w), api.mxfp4_dequantize(*q).double(), wv, k)


def test_more_rows_than_a_grid_is_wide(api):
    rng = np.random.default_rng(6)
    m, n, k = 70001, 24, 128
    x, (w, wv), (u, uv) = activations(rng, m, k), random_matrix(rng, n, k), random_matrix(rng, n, k)
    xd, wv, uv = dev(x), dev(wv), dev(uv)
    q = api.mxfp4_quantize(xd)
    code, byte = ref.quantise(x[-500:])
    assert np.array_equal(host(api.mxfp4_dequantize(*q))[-500:].astype(np.float64), ref.values(code, byte))
    _close(api.w4a16_gemm_mxfp4(xd, *w), xd.double(), wv, k)
    _close(api.w4a4_gemm_mxfp4(*q, *w), api.mxfp4_dequantize(*q).double(), wv, k)
    y = api.w4a16_gemm_silu_mul_mxfp4(xd, *w, *u)
    ref.check_silu(host(y)[-500:], x[-500:].astype(np.float64), host(wv), host(uv))
    y = api.w4a16_gemm_mxfp4(api.mxfp4_dequantize(*w), *q)                # as many weight rows
    _close(y, wv, api.mxfp4_dequantize(*q).double(), k)
    for rows in (1, 6):
        y = api.w4a16_gemm_mxfp4(api.mxfp4_dequantize(*w)[:rows].contiguous(), *q)
        _close(y, wv[:rows], api.mxfp4_dequantize(*q).double(), k)


@pytest.mark.parametrize("k", [128, 256, 384, 640])
@pytest.mark.parametrize("m,n", [(20, 130001), (50, 130000), (200, 70001)])
def test_many_tiles_a_cta(api, m, n, k):
    """Tiles of one to five steps along K, several to a CTA, so that each begins under the one
    before: whole and split along K, and with SiLU."""
    rng = np.random.default_rng(m + n + k)
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    xd = dev(activations(rng, m, k))
    w = [api.mxfp4_quantize((0.3 * torch.randn(n, k, generator=gen, device="cuda")).half()) for _ in range(2)]
    wv = [api.mxfp4_dequantize(*m_).double() for m_ in w]
    for ws in (torch.empty(256, dtype=torch.uint8, device="cuda"), api.mxfp4_workspace(m, k, n)):
        y = torch.full((m, n), float("nan"), dtype=torch.float16, device="cuda")
        _close(api.w4a16_gemm_mxfp4(xd, *w[0], out=y, workspace=ws), xd.double(), wv[0], k)
    y = api.w4a16_gemm_silu_mul_mxfp4(xd, *w[0], *w[1], workspace=api.mxfp4_workspace(m, k, n, "silu"))
    for r in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        ref.check_silu(host(y[:, r]), host(xd).astype(np.float64), host(wv[0][r]), host(wv[1][r]))


@pytest.mark.parametrize("call", ["a16", "a4"])
def test_outputs_past_32_bits(api, call):
    """More than 2^31 outputs: the last rows are what they would be alone."""
    rng = np.random.default_rng(7)
    m, n, k = 66000, 33000, 128
    x, (w, wv) = activations(rng, m, k), random_matrix(rng, n, k)
    xd = dev(x)
    q = api.mxfp4_quantize(xd)
    xv = (xd if call == "a16" else api.mxfp4_dequantize(*q)).double()
    y = api.w4a16_gemm_mxfp4(xd, *w) if call == "a16" else api.w4a4_gemm_mxfp4(*q, *w)
    assert y.numel() > 2 ** 31
    for rows in (slice(0, 40), slice(32000, 32100), slice(65070, 65090), slice(m - 40, m)):
        _close(y[rows], xv[rows], dev(wv), k)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_sizes(api, seed):
    """Sizes over the whole range, with and without room to split, odd rows of y."""
    rng = np.random.default_rng(100 + seed)
    for _ in range(6):
        log = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))
        m, n, k = log(1, 1500), log(1, 4000), 128 * log(1, 40)
        if rng.random() < 0.5:
            n = -(-n // 8) * 8
        x, (w, wv) = activations(rng, m, k), random_matrix(rng, n, k)
        xd, wv = dev(x), dev(wv)
        ws = torch.zeros(int(rng.choice([256, 1 << 20, 64 << 20])), dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        _close(api.w4a16_gemm_mxfp4(xd, *w, workspace=ws, err_flag=err), xd.double(), wv, k)
        q = api.mxfp4_quantize(xd)
        _close(api.w4a4_gemm_mxfp4(*q, *w, workspace=ws, err_flag=err), api.mxfp4_dequantize(*q).double(), wv, k)
        res = dev(rng.standard_normal((m, n)).astype(np.float16))
        one = torch.cat([xd.double(), torch.ones((m, 1), device="cuda", dtype=torch.double)], 1)
        bias = dev(rng.standard_normal(n).astype(np.float16))
        y = api.w4a16_gemm_mxfp4(xd, *w, bias=bias, residual=res, workspace=ws, err_flag=err)
        s = one @ torch.cat([wv, bias.double()[:, None]], 1).T + res.double()
        a = xd.double().abs() @ wv.abs().T + bias.double().abs() + res.double().abs()
        e = ref.sum_error(a, k)
        assert bool(((y.double() - s).abs() <= e + ((s.abs() + e) * 2.0 ** -11).clamp(min=2.0 ** -25)).all())
        g = api.w4a16_gemm_silu_mul_mxfp4(xd, *w, *w, workspace=ws, err_flag=err)
        t = xd.double() @ wv.T
        e = ref.sum_error(xd.double().abs() @ wv.abs().T, k)
        want = t * torch.sigmoid(t) * t
        e = 1.1 * e * (t.abs() + e) + (t * torch.sigmoid(t)).abs() * e + 2.0 ** -21 * want.abs()
        assert bool(((g.double() - want).abs() <= e + ((want.abs() + e) * 2.0 ** -11).clamp(min=2.0 ** -25)).all())
        assert int(err.item()) == 0


@pytest.mark.parametrize("m", [1, 5, 12, 150])
def test_graphs_of_two_users(api, m):
    """Two graphs with a workspace each, replayed at once on two streams; one that has
    the workspace of a call that ran before it."""
    rng = np.random.default_rng(m)
    n, k = 256, 2432
    w, wv = random_matrix(rng, n, k)
    users = []
    for _ in range(2):
        x = dev(activations(rng, m, k))
        ws = api.mxfp4_workspace(m, k, n)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            api.w4a16_gemm_mxfp4(x, *w, workspace=ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = api.w4a16_gemm_mxfp4(x, *w, workspace=ws)
        users.append((x, s, g, y))
    for _ in range(30):
        for x, s, g, y in users:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x, s, g, y in users:
        ref.check_product(host(y), host(x).astype(np.float64), wv)
