"""The MXFP4 format and the calls' refusals (CPU): the reference quantiser against
hand-made values, the scale tiles, and what the binding and the library refuse
before anything reaches the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_ref as ref  # noqa: E402
from w4a16_decode_paged_gb300 import api  # noqa: E402


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 256 if name.endswith("_size") else 0
        return fn

    def products(self):
        return [c for c in self.calls if not c[0].endswith("_size")]


@pytest.fixture
def lib(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(api, "load", lambda: rec)
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    monkeypatch.setattr(api, "stream_handle", lambda stream=None: 0)
    return rec


def h(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def mx(rows, k):
    return torch.zeros((rows, k // 8), dtype=torch.int32), torch.zeros((-(-rows // 128), k // 128, 512), dtype=torch.uint8)


def _row(values):
    x = np.zeros((1, 128), np.float16)
    x[0, :len(values)] = values
    return x


def test_codes_by_hand():
    # largest 6: e = 0, every E2M1 number is its own code, borders go to the even code
    x = _row([0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, .2500001, -.25, -5])
    code, byte = ref.quantise(x)
    assert code[0, :20].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 9, 15, 0, 2, 2, 4, 4, 6, 6, 0, 8, 14]
    assert byte.tolist() == [[127, 104, 104, 104]]
    # 7.9 is under 8: still e = 0, and saturates at 6; 8 is e = 1: code 4
    assert ref.values(*ref.quantise(_row([7.9])))[0, 0] == 6 and ref.values(*ref.quantise(_row([8])))[0, 0] == 8
    # the smallest and the largest fp16 numbers
    code, byte = ref.quantise(_row([2.0 ** -24]))
    assert (code[0, 0], byte[0, 0]) == (1, 104)
    code, byte = ref.quantise(_row([65504]))
    assert (code[0, 0], byte[0, 0]) == (7, 140)
    code, byte = ref.quantise(_row([1, np.inf]))
    assert byte[0, 0] == 255 and not code[0, :32].any()


def test_every_value_is_an_fp16_number():
    for e in range(-23, 14):
        v = ref.E2M1 * 2.0 ** e
        assert (v.astype(np.float16).astype(np.float64) == v).all()


@pytest.mark.parametrize("rows,k", [(1, 128), (33, 256), (128, 384), (129, 128), (300, 896)])
def test_scale_tiles(rows, k):
    b = np.random.default_rng(rows).integers(0, 256, (rows, k // 32)).astype(np.uint8)
    t = api.mxfp4_tile_scales(torch.from_numpy(b))
    assert np.array_equal(t.numpy(), ref.tiles(b)) and t.is_contiguous()
    assert np.array_equal(api.mxfp4_untile_scales(t, rows).numpy(), b) and np.array_equal(ref.untiled(t.numpy(), rows), b)
    with pytest.raises(ValueError, match="tiles"):
        api.mxfp4_untile_scales(t, 128 * t.shape[0] + 1)
    with pytest.raises(ValueError, match="scales"):
        api.mxfp4_tile_scales(torch.from_numpy(b[:, :-1].copy()))


def test_pack_round_trip():
    code = np.random.default_rng(0).integers(0, 16, (5, 128)).astype(np.uint8)
    w = ref.pack(code)
    assert np.array_equal(ref.unpack(w), code) and (w[0, 0] & 15) == code[0, 0] and (w[0, 0] >> 28) == code[0, 7]


def test_calls_reach_the_library_with_their_sizes(lib):
    M, K, N = 5, 384, 130
    c, s = api.mxfp4_quantize(h(M, K))
    assert c.shape == (M, K // 8) and c.dtype == torch.int32 and s.shape == (1, K // 128, 512)
    assert lib.products()[-1][1][1:3] == (M, K)
    y = api.mxfp4_dequantize(c, s)
    assert y.shape == (M, K) and y.dtype == torch.float16
    w = mx(N, K)
    y = api.w4a16_gemm_mxfp4(h(M, K), *w, bias=h(N), residual=h(M, N))
    assert y.shape == (M, N) and y.dtype == torch.float16
    name, a = lib.products()[-1]
    assert name == "w4a16_gemm_mxfp4" and (a[1], a[2], a[5]) == (M, K, N)
    y = api.w4a16_gemm_silu_mul_mxfp4(h(M, K), *w, *mx(N, K))
    assert y.shape == (M, N)
    y = api.w4a4_gemm_mxfp4(c, s, *w, bias=h(N), residual=h(M, N), out=h(M, N))
    name, a = lib.products()[-1]
    assert name == "w4a4_gemm_mxfp4" and (a[2], a[3], a[6]) == (M, K, N)
    api.w4a16_gemm_mxfp4(h(M, K), w[0].view(torch.uint32), w[1])


@pytest.mark.parametrize("bad,what", [
    (dict(x=h(5, 320)), "x"),                       # K no multiple of 128
    (dict(x=h(5, 256)), "codes"),
    (dict(x=h(0, 384)), "x"),
    (dict(x=h(384, 5).t()), "x"),
    (dict(x=h(5 * 384)), "x"),
    (dict(x=None), "x"),
    (dict(x=torch.zeros(5, 384)), "x"),
    (dict(codes=mx(130, 256)[0]), "codes"),
    (dict(codes=torch.zeros((130, 48), dtype=torch.int64)), "codes"),
    (dict(codes=None), "codes"),
    (dict(scales=mx(128, 384)[1]), "scales"),
    (dict(scales=mx(130, 256)[1]), "scales"),
    (dict(scales=torch.zeros((130, 12), dtype=torch.uint8)), "scales"),
    (dict(scales=None), "scales"),
    (dict(bias=h(129)), "bias"),
    (dict(residual=h(130, 5)), "residual"),
    (dict(out=h(5, 131)), "out"),
    (dict(out=torch.zeros(5, 130)), "out"),
    (dict(workspace=torch.zeros(64)), "workspace"),
    (dict(err_flag=torch.zeros(0, dtype=torch.int32)), "err_flag"),
])
def test_product_refusals(lib, bad, what):
    c, s = mx(130, 384)
    args = dict(x=h(5, 384), codes=c, scales=s, bias=None, residual=None, out=None, workspace=None, err_flag=None)
    args.update(bad)
    with pytest.raises(ValueError, match=what):
        api.w4a16_gemm_mxfp4(**args)
    assert not lib.products()
    if "x" not in bad:                              # the other two products refuse the same
        with pytest.raises(ValueError, match=what):
            del args["x"]
            api.w4a4_gemm_mxfp4(*mx(5, 384), **args)
        for k in ("bias", "residual"):
            args.pop(k)
        if not {"bias", "residual"} & set(bad):
            args["codes_gate"], args["scales_gate"] = args.pop("codes"), args.pop("scales")
            with pytest.raises(ValueError, match=what):
                api.w4a16_gemm_silu_mul_mxfp4(h(5, 384), codes_up=c, scales_up=s, **args)
    assert not lib.products()


def test_more_refusals(lib):
    with pytest.raises(ValueError, match="up codes"):
        api.w4a16_gemm_silu_mul_mxfp4(h(2, 128), *mx(40, 128), *mx(41, 128))
    with pytest.raises(ValueError, match="up scales"):
        api.w4a16_gemm_silu_mul_mxfp4(h(2, 128), *mx(40, 128), mx(40, 128)[0], mx(140, 128)[1])
    with pytest.raises(ValueError, match="x_codes"):
        api.w4a4_gemm_mxfp4(torch.zeros((2, 15), dtype=torch.int32), mx(2, 128)[1], *mx(40, 128))
    with pytest.raises(ValueError, match="x_scales"):
        api.w4a4_gemm_mxfp4(mx(2, 128)[0], mx(200, 128)[1], *mx(40, 128))
    with pytest.raises(ValueError, match="codes"):
        api.mxfp4_quantize(h(2, 128), codes=torch.zeros((2, 17), dtype=torch.int32))
    with pytest.raises(ValueError, match="codes"):
        api.mxfp4_quantize(h(2, 128), codes=torch.zeros((2, 16)))
    with pytest.raises(ValueError, match="scales"):
        api.mxfp4_quantize(h(2, 128), scales=torch.zeros((1, 1, 511), dtype=torch.uint8))
    with pytest.raises(ValueError, match="K="):
        api.mxfp4_quantize(h(2, 64))
    with pytest.raises(ValueError, match="out"):
        api.mxfp4_dequantize(*mx(2, 128), out=h(2, 129))
    with pytest.raises(ValueError, match="kind"):
        api.mxfp4_workspace(1, 128, 1, "a8")
    assert not lib.products()


ALIGNED, MISALIGNED = 1 << 20, (1 << 20) + 64      # device addresses that nothing reads


def test_the_library_refuses_before_any_launch():
    from w4a16_decode_paged_gb300 import _lib, build
    build.build()
    L = _lib.load()
    A, B = ALIGNED, MISALIGNED
    assert L.mxfp4_quantize(None, 1, 128, A, A, None) == 1
    assert L.mxfp4_quantize(A, 0, 128, A, A, None) == 1
    assert L.mxfp4_quantize(A, 1, 96, A, A, None) == 3 and b"multiple of 128" in L.w4a16_last_error()
    assert L.mxfp4_quantize(A, 1, 131200, A, A, None) == 3
    assert L.mxfp4_quantize(A, 1048577, 128, A, A, None) == 3
    for i in range(3):
        p = [A, A, A]
        p[i] = B
        assert L.mxfp4_quantize(p[0], 1, 128, p[1], p[2], None) == 2
        assert L.mxfp4_dequantize(p[0], p[1], 1, 128, p[2], None) == 2
    assert L.mxfp4_dequantize(A, A, 1, 64, A, None) == 3 and L.mxfp4_dequantize(A, None, 1, 128, A, None) == 1

    def a16(x=A, M=1, K=128, c=A, s=A, N=8, bias=None, res=None, y=A, ws=None, wb=0):
        return L.w4a16_gemm_mxfp4(x, M, K, c, s, N, bias, res, y, ws, wb, None, None)

    def a4(xc=A, xs=A, M=1, K=128, c=A, s=A, N=8, bias=None, res=None, y=A, ws=None, wb=0):
        return L.w4a4_gemm_mxfp4(xc, xs, M, K, c, s, N, bias, res, y, ws, wb, None, None)

    def silu(x=A, M=1, K=128, c=A, s=A, c2=A, s2=A, N=8, y=A, ws=None, wb=0):
        return L.w4a16_gemm_silu_mul_mxfp4(x, M, K, c, s, c2, s2, N, y, ws, wb, None, None)

    for f in (a16, a4, silu):
        assert f(M=0) == 1 and f(N=0) == 1 and f(K=0) == 1 and f(c=None) == 1 and f(s=None) == 1 and f(y=None) == 1
        assert f(K=192) == 3 and f(K=131200) == 3 and f(M=1048577) == 3 and f(N=1048577) == 3
        assert f(c=B) == 2 and f(s=B) == 2 and f(y=B) == 2 and f(ws=B, wb=1 << 20) == 2
    for f in (a16, a4):
        assert f(bias=B) == 2 and f(res=B) == 2
    assert a16(x=None) == 1 and a16(x=B) == 2 and silu(x=B) == 2 and silu(c2=None) == 1 and silu(s2=B) == 2
    assert a4(xc=None) == 1 and a4(xs=None) == 1 and a4(xc=B) == 2 and a4(xs=B) == 2
    assert L.mxfp4_scales_size(129, 256) == 2 * 2 * 512 and L.mxfp4_scales_size(1, 100) == 0
