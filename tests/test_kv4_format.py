"""The INT4 page format (CPU): the numpy reference against the format's own
statements, and the refusals of the entry points through the ABI and the
binding (no kernel runs)."""
import numpy as np
import pytest

import kv4_ref as ref

torch = pytest.importorskip("torch")


def test_scales_are_the_top_bits_of_fp16():
    got = (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(got, ref.SCALES[:248]) and np.all(np.isnan(ref.SCALES[248:]))


def test_every_value_is_an_fp16_number():
    v = np.arange(-7, 8)[:, None] * ref.SCALES[None, :227]      # 227: the largest scale a finite row takes, 10240
    assert np.array_equal(v[np.abs(v) <= 65504], v[np.abs(v) <= 65504].astype(np.float16).astype(np.float64))
    # and so is a 64th of it, with the unpacking's biases (264, 72, 24 times s / 64)
    for f in (1, 264, 72, 24):
        w = ref.SCALES[:227] / 64 * f
        assert np.array_equal(w, w.astype(np.float16).astype(np.float64))
    w = v / 64
    assert np.array_equal(w, w.astype(np.float16).astype(np.float64))


def test_code_and_scale_bytes_do_not_overlap():
    for code, scale in ((ref.k_code, ref.k_scale), (ref.v_code, ref.v_scale)):
        nib = {(code(t, d), d % 2) for t in range(16) for d in range(128)}
        assert nib == {(i, e) for i in range(1024) for e in range(2)}
        assert {scale(t, c) for t in range(16) for c in range(4)} == set(range(1024, 1088))
        owner = {code(t, d): t for t in range(16) for d in range(128)}
        assert all(owner[code(t, d)] == t for t in range(16) for d in range(128))   # no byte of two tokens


@pytest.mark.parametrize("spread", [1.0, 1e-6, 3e-5, 100.0, 20000.0])
def test_quantiser_is_off_by_half_a_step_at_most(spread):
    r = np.random.default_rng(1)
    for _ in range(20):
        x = np.clip(r.standard_normal(128) * spread, -65504, 65504).astype(np.float16)
        q, byte = ref.quantise_row(x)
        s = np.repeat(ref.SCALES[byte], 32)
        assert np.all(np.abs(q) <= 7)
        assert np.all(np.abs(x.astype(np.float64) - q * s) <= s / 2)
        amax = np.abs(x.astype(np.float64)).reshape(4, 32).max(1)
        assert np.all(7 * ref.SCALES[byte] >= amax)
        assert np.all((byte == 0) | (7 * ref.SCALES[np.maximum(byte - 1, 0)] < amax))


def test_rows_round_trip_through_slices():
    r = np.random.default_rng(2)
    for which in "kv":
        sl = r.integers(0, 256, ref.SLICE).astype(np.uint8)
        rows = {}
        for t in r.permutation(16):
            x = r.standard_normal(128).astype(np.float16)
            q, byte = ref.quantise_row(x)
            ref.store_row(sl, t, q, byte, which)
            rows[t] = q * np.repeat(ref.SCALES[byte], 32)
        got = ref.unpack(sl, which)
        for t, want in rows.items():
            assert np.array_equal(got[t], want)


# ---- refusals through the C ABI: fake device addresses, never dereferenced ----
A, MIS = 1 << 20, (1 << 20) + 64


@pytest.fixture(scope="module")
def lib():
    from w4a16_decode_paged_gb300 import _lib, build
    build.build()
    return _lib.load()


def _append(lib, q=A, k=A, v=A, stride=0, q_out=None, kp=A, vp=A, pages=8, bt=A, mb=4, lens=A, B=2, Hq=7, Hkv=1, D=128,
            theta=1e6):
    return lib.kv_append_rope_int4(q, k, v, stride, q_out, kp, vp, pages, bt, mb, lens, B, Hq, Hkv, D, theta, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), 1), (dict(kp=None), 1), (dict(lens=None), 1), (dict(B=0), 1), (dict(pages=0), 1), (dict(mb=0), 1),
    (dict(D=64), 3), (dict(Hq=7, Hkv=2), 3), (dict(theta=0.0), 1), (dict(stride=900), 1), (dict(stride=-8), 1),
    (dict(stride=512), 1), (dict(q=MIS), 2), (dict(q_out=MIS), 2), (dict(vp=MIS), 2)])
def test_append_refusals(lib, bad, code):
    assert _append(lib, **bad) == code and lib.w4a16_last_error()


def _read(lib, kp=A, vp=A, pages=8, bt=A, mb=4, starts=None, lens=A, T=5, B=2, Hkv=1, D=128, ko=A, vo=A, clear=0):
    return lib.kv_read_int4(kp, vp, pages, bt, mb, starts, lens, T, B, Hkv, D, ko, vo, clear, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(kp=None), 1), (dict(vo=None), 1), (dict(T=0), 1), (dict(B=0), 1), (dict(Hkv=0), 1), (dict(clear=2), 1), (dict(D=96), 3),
    (dict(B=65536), 3), (dict(ko=MIS), 2), (dict(kp=MIS), 2)])
def test_read_refusals(lib, bad, code):
    assert _read(lib, **bad) == code and lib.w4a16_last_error()


def _attn(lib, form, q=A, qs=0, kp=A, vp=A, ks=A, vs=A, pages=8, bt=A, mb=4096, lens=A, mc=65536, window=60000, sinks=4, B=2,
          Hq=7, Hkv=1, D=128, theta=1e6, ws=A, wsb=1 << 30, out=A):
    head = (q, qs, kp, vp) + ((ks, vs) if form == "window_fp8" else ()) + (pages, bt, mb, lens, mc)
    head += (window, sinks) if "window" in form else ()
    head += (B, Hq, Hkv, D) + ((theta,) if "append" in form else ())
    return getattr(lib, "paged_gqa_decode_" + form if form else "paged_gqa_decode")(
        *head, 0.088, ws, wsb, out, None, None)


FORMS = ["int4", "rope_append_int4", "window", "window_fp8", "window_int4"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad,code", [
    (dict(q=None), 1), (dict(kp=None), 1), (dict(bt=None), 1), (dict(out=None), 1), (dict(B=0), 1), (dict(mc=0), 1),
    (dict(mc=65537), 3), (dict(D=64), 3), (dict(Hq=9), 3), (dict(Hq=7, Hkv=2), 3), (dict(B=(1 << 24) + 1), 3), (dict(qs=100), 1),
    (dict(qs=4097), 1), (dict(q=MIS), 2), (dict(vp=MIS), 2), (dict(out=MIS), 2), (dict(ws=None), 1),
    (dict(wsb=1000), 1), (dict(ws=MIS), 2)])
def test_attention_refusals(lib, form, bad, code):
    assert _attn(lib, form, **bad) == code and lib.w4a16_last_error()


@pytest.mark.parametrize("form,bad", [("window", dict(window=-1)), ("window_int4", dict(sinks=-1)),
                                      ("window_fp8", dict(ks=None)), ("rope_append_int4", dict(theta=-1.0)),
                                      ("rope_append_int4", dict(qs=8 * 128))])
def test_attention_refusals_of_one_form(lib, form, bad):
    assert _attn(lib, form, **bad) == 1


def test_workspace_size_grows_with_what_is_seen(lib):
    size = lib.paged_gqa_decode_window_workspace_size
    assert size(4, 28, 4, 32768, 32768, 0, 128) >= size(4, 28, 4, 32768, 1024, 4, 128) > 0
    assert size(0, 28, 4, 512, 512, 0, 128) == 0 and size(1, 28, 4, 512, -1, 0, 128) == 0
    # a sequence that one CTA covers needs no partials of its own kind, whatever its bound
    assert size(1, 7, 1, 16, 16, 0, 128) <= size(1, 7, 1, 1 << 20, 1 << 20, 0, 128)


@pytest.mark.parametrize("form", FORMS)
def test_attention_refuses_pages_past_32_bit_pitches(lib, form):
    # (a page of 2^20 fp16 heads is 2^32 bytes: the sizes pass every other check)
    assert _attn(lib, form, B=1, Hq=1 << 20, Hkv=1 << 20, mc=16, mb=1, window=16) == 3
    assert b"Hkv" in lib.w4a16_last_error()


def test_append_refuses_rows_past_32_bits(lib):
    assert _append(lib, Hq=(1 << 20) + 1, Hkv=1) == 3


@pytest.mark.parametrize("Hq,Hkv", [(28, 4), (7, 1), (8, 8), (6, 2), (64, 8)])
@pytest.mark.parametrize("mc", [16, 300, 5000, 32768])
def test_workspace_serves_smaller_calls(lib, Hq, Hkv, mc):
    """A workspace for a batch serves every smaller one: the size falls with none
    of the arguments.  The calls check it against their own need, which has to be
    met for every kind of page."""
    size = lib.paged_gqa_decode_window_workspace_size
    sizes = [size(B, Hq, Hkv, mc, mc, 0, 128) for B in (1, 2, 3, 19, 37, 38, 39, 40, 76, 152, 153, 304, 305, 5000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for B in (1, 38, 39, 146):
        by_mc = [size(B, Hq, Hkv, n, n, 0, 128) for n in (1, 16, 17, 200, 1000, mc, 40000)[:5]]
        assert by_mc == sorted(by_mc)
        by_window = [size(B, Hq, Hkv, mc, w, 4, 128) for w in (0, 1, 100, 1000, 10 ** 6)]
        assert by_window == sorted(by_window) and by_window[-1] <= max(size(B, Hq, Hkv, mc, mc, 0, 128), 16384)
        by_sinks = [size(B, Hq, Hkv, mc, 64, n, 128) for n in (0, 1, 100, 10 ** 6)]
        assert by_sinks == sorted(by_sinks)


# ---- the binding's checks ------------------------------------------------------
@pytest.fixture
def rec(monkeypatch):
    from w4a16_decode_paged_gb300 import api

    class Rec:
        calls = []

        def __getattr__(self, name):
            return lambda *a: (self.calls.append((name, a)), 0)[1]
    r = Rec()
    r.calls = []
    monkeypatch.setattr(api, "load", lambda: r)
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    monkeypatch.setattr(api, "stream_handle", lambda stream=None: 0)
    return api, r


def _h(*s):
    return torch.zeros(s, dtype=torch.float16)


def _base(B=2, Hq=7, Hkv=1, pages=8, mb=4):
    return dict(k_pool=torch.zeros((pages, Hkv, 1088), dtype=torch.uint8),
                v_pool=torch.zeros((pages, Hkv, 1088), dtype=torch.uint8),
                block_table=torch.zeros((B, mb), dtype=torch.int32), context_lens=torch.ones(B, dtype=torch.int32))


def test_binding_append(rec):
    api, r = rec
    api.kv_append_rope_int4(_h(2, 7, 128), _h(2, 1, 128), _h(2, 1, 128), **_base(), theta=1e6)
    qkv = _h(2, 9 * 128)
    v3 = qkv.view(2, 9, 128)
    api.kv_append_rope_int4(v3[:, :7], v3[:, 7:8], v3[:, 8:], **_base(), theta=1e6, row_stride=9 * 128)
    name, a = r.calls[-1]
    assert name == "kv_append_rope_int4" and a[3] == 9 * 128 and a[11:15] == (2, 7, 1, 128)
    n = len(r.calls)
    for bad, what in ((dict(q=_h(2, 7, 64)), "q"), (dict(k=_h(2, 2, 128)), "k: shape"), (dict(v=_h(3, 1, 128)), "v"),
                      (dict(q=v3[:, :7]), "q"), (dict(q_out=_h(2, 6, 128)), "q_out"),
                      (dict(k_pool=torch.zeros((8, 1, 1024), dtype=torch.uint8)), "k_pool"),
                      (dict(block_table=torch.zeros((2, 4), dtype=torch.int64)), "block_table"),
                      (dict(context_lens=torch.ones(3, dtype=torch.int32)), "context_lens"),
                      (dict(q=_h(2, 7, 128).transpose(0, 1).contiguous().transpose(0, 1)), "q")):
        args = dict(q=_h(2, 7, 128), k=_h(2, 1, 128), v=_h(2, 1, 128), theta=1e6, **_base())
        args.update(bad)
        with pytest.raises(ValueError, match=what):
            api.kv_append_rope_int4(**args)
    assert len(r.calls) == n


def test_binding_read(rec):
    api, r = rec
    k, v = api.kv_read_int4(**_base(), T=5)
    assert tuple(k.shape) == tuple(v.shape) == (2, 5, 1, 128)
    for bad, what in ((dict(T=0), "T="), (dict(starts=torch.zeros(3, dtype=torch.int32)), "starts"),
                      (dict(k_out=_h(2, 4, 1, 128), v_out=_h(2, 5, 1, 128)), "k_out"),
                      (dict(k_out=_h(2, 5, 1, 128), v_out=_h(2, 5, 1, 128).float()), "v_out"),
                      (dict(v_out=_h(2, 5, 1, 128)), "k_out is required")):
        with pytest.raises(ValueError, match=what):
            api.kv_read_int4(**{**_base(), "T": 5, **bad})


def test_binding_attention(rec):
    api, r = rec
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    out = api.paged_gqa_decode_int4(_h(2, 7, 128), **_base(), max_context=64, workspace=ws)
    assert tuple(out.shape) == (2, 7, 128) and r.calls[-1][0] == "paged_gqa_decode_int4"
    out = api.paged_gqa_decode_int4(_h(2, 9 * 128), **_base(), max_context=64, workspace=ws, qkv_theta=1e6, n_q_heads=7)
    assert r.calls[-1][0] == "paged_gqa_decode_rope_append_int4" and r.calls[-1][1][1] == 9 * 128
    for bad, what in ((dict(q=_h(2, 7, 64)), "q"), (dict(q=_h(2, 8 * 128), qkv_theta=1e6, n_q_heads=7), "qkv"),
                      (dict(q=_h(2, 9 * 128), qkv_theta=1e6), "n_q_heads"),
                      (dict(out=_h(2, 7, 127)), "out"), (dict(workspace=ws.float()), "workspace")):
        with pytest.raises(ValueError, match=what):
            api.paged_gqa_decode_int4(**{"q": _h(2, 7, 128), **_base(), "max_context": 64, "workspace": ws, **bad})


def test_binding_window_takes_every_kind_of_pool(rec):
    api, r = rec
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    b = _base()
    fp16 = dict(b, k_pool=_h(8, 1, 16, 128), v_pool=_h(8, 1, 16, 128))
    fp8 = dict(b, k_pool=torch.zeros((8, 1, 16, 128), dtype=torch.uint8),
               v_pool=torch.zeros((8, 1, 16, 128), dtype=torch.uint8), k_scale=torch.ones(8, 1, 16),
               v_scale=torch.ones(8, 1, 16))
    for pools, name in ((fp16, "paged_gqa_decode_window"), (fp8, "paged_gqa_decode_window_fp8"),
                        (b, "paged_gqa_decode_window_int4")):
        api.paged_gqa_decode_window(_h(2, 7, 128), **pools, max_context=64, window=1 << 40, sinks=3, workspace=ws)
        got, a = r.calls[-1]
        assert got == name and a[-12:-9] == (64, 3, 2)          # the window, cut to max_context; sinks; B
    for pools, bad, what in ((fp16, dict(window=-1), "window"), (fp16, dict(sinks=-2), "sinks"),
                             (fp8, dict(k_scale=None), "k_scale"), (fp8, dict(v_scale=torch.ones(8, 1, 15)), "v_scale"),
                             (dict(fp8, k_scale=None, v_scale=None), {}, "k_pool"),
                             (dict(b, k_pool=_h(8, 1, 16, 64), v_pool=_h(8, 1, 16, 64)), {}, "k_pool"),
                             (fp16, dict(q=_h(2, 7, 64)), "q")):
        with pytest.raises(ValueError, match=what):
            api.paged_gqa_decode_window(**{"q": _h(2, 7, 128), **pools, "max_context": 64, "window": 9, "workspace": ws,
                                           **bad})
