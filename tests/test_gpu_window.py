"""Decode attention with a sliding window and sinks over fp16, FP8 and INT4
pages, against the numpy reference.  GPU only (marked gpu)."""
import math

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


class Cache:
    """Pools of one kind with random values, as numpy arrays and values in 64 bits."""

    def __init__(self, r, kind, pages, Hkv):
        self.kind = kind
        if kind == "int4":
            self.k, self.v = ref.random_pool(r, pages, Hkv), ref.random_pool(r, pages, Hkv)
            self.scales = {}
        elif kind == "fp16":
            self.k, self.v = synth.kv_pool(r, pages, Hkv, D), synth.kv_pool(r, pages, Hkv, D)
            self.scales = {}
        else:
            self.k, self.v = (r.integers(0, 256, (pages, Hkv, 16, D)).astype(np.uint8) for _ in "kv")
            for c in (self.k, self.v):
                c[(c & 0x78) > 0x60] ^= 0x40                        # magnitudes up to 60: no NaN codes
            self.scales = dict(k_scale=r.uniform(0.02, 0.06, (pages, Hkv, 16)).astype(np.float32),
                               v_scale=r.uniform(0.02, 0.06, (pages, Hkv, 16)).astype(np.float32))

    def values(self, which, p):
        pool = getattr(self, which)[p]
        if self.kind == "int4":
            return ref.unpack(pool, which)
        if self.kind == "fp16":
            return pool.astype(np.float64)
        codes = torch.from_numpy(pool).view(torch.float8_e4m3fn).double().numpy()
        return codes * self.scales[which + "_scale"][p].astype(np.float64)[..., None]

    def poison(self, p, tokens):
        """What a masked token's bytes may hold: NaN and infinities."""
        for t in tokens:
            for which in "kv":
                pool = getattr(self, which)
                if self.kind == "int4":
                    at = ref.k_scale if which == "k" else ref.v_scale
                    for c in range(4):
                        pool[p, :, at(t, c)] = 0xFF
                elif self.kind == "fp16":
                    pool[p, :, t] = np.nan
                    pool[p, :, t, ::2] = np.inf
                else:
                    pool[p, :, t] = 0x7F
                    self.scales[which + "_scale"][p, :, t] = np.nan

    def dev(self):
        s = {n: to_dev(a, torch) for n, a in self.scales.items()}
        return dict(k_pool=to_dev(self.k, torch), v_pool=to_dev(self.v, torch), **s)


def _run(api, r, kind, G, Hkv, lens, window, sinks, max_context=None, release=True):
    lens = np.asarray(lens, np.int32)
    pages = int(sum((max(n, 0) + 15) // 16 for n in lens)) + 3
    bt = synth.block_table(r, np.maximum(lens, 0), pages)
    c = Cache(r, kind, pages, Hkv)
    want_bt = bt.copy()
    for b, n in enumerate(lens):
        for p in range((n + 15) // 16):
            masked = [t for t in range(16) if not (p * 16 + t < n and (p * 16 + t >= n - window or p * 16 + t < sinks))]
            c.poison(bt[b, p], masked)
            if release and len(masked) == 16:
                bt[b, p] = -1                                     # pages that nothing sees may be gone
    q = synth.normal_fp16(r, (len(lens), G * Hkv, D))
    mc = max_context or max(int(lens.max()), 1)
    need = (mc + 15) // 16
    if bt.shape[1] < need:
        bt = np.pad(bt, ((0, 0), (0, need - bt.shape[1])), constant_values=-1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_gqa_decode_window(to_dev(q, torch), **c.dev(), block_table=to_dev(bt, torch),
                                      context_lens=to_dev(lens, torch), max_context=mc, window=window, sinks=sinks,
                                      err_flag=err)
    assert int(err.item()) == 0
    want = ref.attend(q, lambda p: c.values("k", p), lambda p: c.values("v", p), want_bt, lens, 1 / math.sqrt(D), window,
                      sinks)
    ref.check_attention(to_host(out), want, int(lens.max()), f"{kind} window {window} sinks {sinks}")
    return to_host(out), q, c, bt, lens


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 1), (100, 4), (64, 16), (33, 17), (1000, 3), (1, 1), (5, 40),
                                          (2, 160)])
def test_window_and_sinks(api, kind, window, sinks):
    r = np.random.default_rng(window * 31 + sinks)
    _run(api, r, kind, 7, 2, [1, 15, 16, 17, 33, 150, 163], window, sinks)


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
@pytest.mark.parametrize("G,Hkv,lens,window,sinks", [(1, 8, [3000], 1024, 4), (8, 1, [2000, 5, 0, 1300], 1000, 20),
                                                     (3, 2, [700] * 5, 128, 0), (5, 1, [4097], 4096, 0),
                                                     (6, 4, [1025, 1024], 1024, 1)])
def test_head_layouts_and_longer_windows(api, kind, G, Hkv, lens, window, sinks):
    r = np.random.default_rng(G + 10 * Hkv)
    _run(api, r, kind, G, Hkv, lens, window, sinks)


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
def test_rows_that_see_nothing_give_zeros(api, kind):
    r = np.random.default_rng(5)
    out, *_ = _run(api, r, kind, 7, 1, [40, 0, 16, -7], 0, 0)
    assert np.all(out == 0)
    out, *_ = _run(api, r, kind, 7, 1, [40, 3, 0, 20], 0, 5)         # the sinks alone
    assert np.any(out[0] != 0) and np.all(out[2] == 0)


@pytest.mark.parametrize("first", [0, 2, 40])
def test_tokens_that_score_minus_infinity_weigh_nothing(api, first):
    """K rows with an infinity whose product is -inf, a page of them and more:
    pages that come first, pages between, and all but one token."""
    r = np.random.default_rng(6)
    G, L = 7, 700
    bt = synth.block_table(r, np.array([L], np.int32), 50)
    c = Cache(r, "fp16", 50, 1)
    q = np.abs(synth.normal_fp16(r, (1, G, D))) + np.float16(0.1)
    hidden = [0, 1, 2, 3, 4, 5, 6, 7, 20, 43] if first == 0 else [first] if first == 2 else list(range(43))
    for p in hidden:
        c.k[bt[0, p], :, :, 5] = -np.inf                           # every token of the page, all heads
    out = to_host(api.paged_gqa_decode_window(to_dev(q, torch), **c.dev(), block_table=to_dev(bt, torch),
                                              context_lens=to_dev(np.array([L], np.int32), torch), max_context=L,
                                              window=L, sinks=0))
    # the formula without those tokens: they weigh exp(-inf) = 0
    seen = [t for t in range(L) if t // 16 not in hidden]
    k = np.concatenate([c.values("k", bt[0, p])[0] for p in range((L + 15) // 16)])[seen]
    v = np.concatenate([c.values("v", bt[0, p])[0] for p in range((L + 15) // 16)])[seen]
    s = q[0].astype(np.float64) @ k.T / math.sqrt(D)
    e = np.exp(s - s.max(1, keepdims=True))
    p = e / e.sum(1, keepdims=True)
    ref.check_attention(out, ((p @ v)[None], (p @ np.abs(v))[None], np.abs(v).max()), L, "scores of -inf")


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
def test_a_call_on_a_given_stream_makes_its_tensors_there(api, kind):
    """The current stream is busy and its freed memory holds anything; the call on
    another stream, with no workspace and no output given, is done regardless."""
    r = np.random.default_rng(7)
    out, q, c, bt, lens = _run(api, r, kind, 7, 2, [3000, 400], 2500, 4)
    args = dict(c.dev(), block_table=to_dev(bt, torch), context_lens=to_dev(lens, torch), max_context=3000, window=2500,
                sinks=4)
    dq = to_dev(q, torch)
    torch.full((1 << 22,), 0x7F, dtype=torch.uint8, device="cuda")  # (freed at once)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    got = api.paged_gqa_decode_window(dq, **args, stream=side)
    side.synchronize()
    host = torch.empty(got.shape, dtype=got.dtype, pin_memory=True)
    with torch.cuda.stream(side):
        host.copy_(got, non_blocking=True)
    side.synchronize()
    assert np.array_equal(host.numpy(), out)
    torch.cuda.synchronize()


def test_one_workspace_serves_a_shrinking_batch(api):
    """38 sequences may be split into more parts than 39."""
    r = np.random.default_rng(8)
    n = api.load().paged_gqa_decode_window_workspace_size(39, 28, 4, 2000, 2000, 0, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    lens = np.full(39, 2000, np.int32)
    bt = np.stack([r.permutation(200)[:125] for _ in lens]).astype(np.int32)   # (pages shared between sequences)
    for kind in ("fp16", "fp8", "int4"):
        c = Cache(r, kind, 200, 4)
        q = synth.normal_fp16(r, (39, 28, D))
        want = ref.attend(q[:3], lambda p: c.values("k", p), lambda p: c.values("v", p), bt[:3], lens[:3], 1 / math.sqrt(D),
                          2000, 0)
        for B in (39, 38, 20, 3):
            out = api.paged_gqa_decode_window(to_dev(q[:B], torch), **c.dev(), block_table=to_dev(bt[:B], torch),
                                              context_lens=to_dev(lens[:B], torch), max_context=2000, window=2000,
                                              sinks=0, workspace=ws)
            ref.check_attention(to_host(out)[:3], want, 2000, f"{kind} B={B}")


def test_the_same_sequence_twice_in_a_batch(api):
    r = np.random.default_rng(9)
    _, q, c, bt, lens = _run(api, r, "int4", 7, 2, [1000], 1000, 0)
    want = ref.attend(q, lambda p: c.values("k", p), lambda p: c.values("v", p), bt, lens, 1 / math.sqrt(D))
    two = api.paged_gqa_decode_int4(to_dev(np.repeat(q, 2, 0), torch), c.dev()["k_pool"], c.dev()["v_pool"],
                                    to_dev(np.repeat(bt, 2, 0), torch), to_dev(np.repeat(lens, 2), torch), 1000)
    assert torch.equal(two[0], two[1])
    ref.check_attention(to_host(two)[:1], want, 1000, "the same sequence twice")


@pytest.mark.parametrize("kind", ["fp16", "fp8", "int4"])
def test_a_wide_window_is_plain_attention(api, kind):
    """Window and sinks that cover everything, however they do it: the same bits."""
    r = np.random.default_rng(6)
    out, q, c, bt, lens = _run(api, r, kind, 4, 2, [90, 513], 513, 0, release=False)
    for window, sinks in ((2 ** 31 - 1, 0), (400, 113), (1, 2 ** 31 - 1), (513, 513)):
        got = api.paged_gqa_decode_window(to_dev(q, torch), **c.dev(), block_table=to_dev(bt, torch),
                                          context_lens=to_dev(lens, torch), max_context=513, window=window, sinks=sinks)
        assert np.array_equal(to_host(got), out)
    if kind == "int4":
        got = api.paged_gqa_decode_int4(to_dev(q, torch), *(c.dev()[n] for n in ("k_pool", "v_pool")), to_dev(bt, torch),
                                        to_dev(lens, torch), 513)
        assert np.array_equal(to_host(got), out)


def test_agrees_with_the_plain_kernels(api):
    """fp16 and FP8 pages without a mask: the framework's plain attention, to
    the two kernels' own roundings (the bound of the reference, twice)."""
    for kind in ("fp16", "fp8"):
        r = np.random.default_rng(7)
        out, q, c, bt, lens = _run(api, r, kind, 7, 4, [512, 100], 512, 0, release=False)
        d = c.dev()
        # the plain kernels take no bytes past the length that are not numbers
        pools = {n: (t.nan_to_num(0.0, 0.0, 0.0) if t.dtype != torch.uint8 else t.where(t != 0x7F, torch.zeros_like(t)))
                 for n, t in d.items()}
        fn = api.paged_gqa_decode if kind == "fp16" else api.paged_gqa_decode_fp8
        got = fn(to_dev(q, torch), **pools, block_table=to_dev(bt, torch), context_lens=to_dev(lens, torch),
                 max_context=512)
        a, b = out.astype(np.float64), to_host(got).astype(np.float64)
        assert np.all(np.abs(a - b) <= 2.0 ** -9 * np.abs(b) + 2.0 ** -8)


def test_a_window_that_slides(api):
    """Decode steps of a sequence that outgrows its window: pages behind the
    window are taken away and written over, the sinks' stay."""
    r = np.random.default_rng(8)
    Hq, Hkv, window, sinks, theta = 7, 1, 40, 4, 1e6
    pool, pages_free = 8, list(range(8))
    kp, vp = (torch.full((pool, Hkv, 1088), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
    bt = torch.full((1, 16), -1, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    K, V = [], []
    for step in range(200):
        p = step // 16
        if step % 16 == 0:
            dead = [i for i in range(1, p) if (i + 1) * 16 <= step + 1 - window]
            for i in dead:
                if int(bt[0, i]) >= 0:
                    pages_free.append(int(bt[0, i]))
                    bt[0, i] = -1
            bt[0, p] = pages_free.pop(0)
        n += 1
        q, k, v = [to_dev(synth.normal_fp16(r, (1, h, D)), torch) for h in (Hq, Hkv, Hkv)]
        api.kv_append_rope_int4(q, k, v, kp, vp, bt, n, theta)
        kr, vr = api.kv_read_int4(kp, vp, bt, n, 1, starts=n - 1)
        K.append(to_host(kr)[0, 0])
        V.append(to_host(vr)[0, 0])
        out = api.paged_gqa_decode_window(q, kp, vp, bt, n, 256, window, sinks)
        if step % 7 == 0 or step > 190:
            pad = lambda x: np.concatenate([np.stack(x).astype(np.float64), np.zeros((-len(x) % 16, Hkv, D))]).reshape(
                -1, 16, Hkv, D).transpose(0, 2, 1, 3)
            kk, vv = pad(K), pad(V)
            want = ref.attend(to_host(q), lambda p: kk[p], lambda p: vv[p], np.arange(len(kk))[None], [step + 1],
                              1 / math.sqrt(D), window, sinks)
            ref.check_attention(to_host(out), want, step + 1, f"step {step}")


@pytest.mark.parametrize("kind", ["fp16", "fp8"])
def test_offsets_past_32_bits(api, kind):
    Hkv = 4
    pages = (2 ** 32) // (Hkv * 2048 * (2 if kind == "fp16" else 1)) + 40
    r = np.random.default_rng(9)
    c = Cache(r, kind, 3, Hkv)
    small = c.dev()
    big = {n: torch.empty((pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for n, t in small.items()}
    bt = np.array([[pages - 1, 2, pages - 5]], np.int32)
    for i, p in enumerate(bt[0]):
        for n in big:
            big[n][p] = small[n][i]
    lens = np.array([41], np.int32)
    q = synth.normal_fp16(r, (1, 28, D))
    out = api.paged_gqa_decode_window(to_dev(q, torch), **big, block_table=to_dev(bt, torch),
                                      context_lens=to_dev(lens, torch), max_context=48, window=20, sinks=3)
    want = ref.attend(q, lambda p: c.values("k", p), lambda p: c.values("v", p), np.arange(3)[None], lens, 1 / math.sqrt(D),
                      20, 3)
    ref.check_attention(to_host(out), want, 41)
