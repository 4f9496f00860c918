"""INT4 KV pages on the GPU against the numpy references: the quantised
append, the read back, decode attention over the pages, the fused form, and
the calls together.  GPU only (marked gpu)."""
import math

import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import to_dev, to_host
from w4a16_decode_paged_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
THETA = 1e6
D = 128


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as _api
    from w4a16_decode_paged_gb300 import build
    build.build()
    return _api


def dev(*arrs):
    return [to_dev(a, torch) for a in arrs]


def _table(r, lens, spare=3):
    pages = int(sum((max(int(n), 0) + 15) // 16 for n in lens)) + spare
    return synth.block_table(r, np.maximum(lens, 0), pages), pages


def _rows_of(pool, which, bt, lens):
    """Values of each sequence's newest row, [B][Hkv][128]."""
    return np.stack([ref.unpack(pool[bt[b, (n - 1) // 16]], which)[:, (n - 1) % 16] for b, n in enumerate(lens)])


def _scales_of(pool, which, bt, lens):
    at = ref.k_scale if which == "k" else ref.v_scale
    out = []
    for b, n in enumerate(lens):
        sl = pool[bt[b, (n - 1) // 16]]
        out.append(np.stack([ref.SCALES[sl[:, at((n - 1) % 16, c)]] for c in range(4)], 1).repeat(32, 1))
    return np.stack(out)


# ---- append ---------------------------------------------------------------------
@pytest.mark.parametrize("Hq,Hkv,lens", [(7, 1, [1]), (28, 4, [16, 17, 15, 1]), (8, 8, [33, 512]), (6, 2, list(range(1, 41)))])
def test_append(api, Hq, Hkv, lens):
    r = np.random.default_rng(100 + Hq + len(lens))
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    bt, pages = _table(r, lens)
    q, k, v = (synth.normal_fp16(r, (B, n, D)) * np.float16(2) for n in (Hq, Hkv, Hkv))
    kp, vp = (r.integers(0, 256, (pages, Hkv, 1088)).astype(np.uint8) for _ in "kv")
    dq, dk, dv, dkp, dvp, dbt, dl = dev(q, k, v, kp, vp, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = api.kv_append_rope_int4(dq, dk, dv, dkp, dvp, dbt, dl, THETA, q_out=torch.empty_like(dq), err_flag=err)
    assert int(err.item()) == 0 and np.array_equal(to_host(dq), q)
    gk, gv = to_host(dkp), to_host(dvp)
    # V: the reference's bytes, and no other byte of either pool moved
    want_v, want_k = vp.copy(), kp.copy()
    for b, n in enumerate(lens):
        for h in range(Hkv):
            p, t = bt[b, (n - 1) // 16], (n - 1) % 16
            ref.store_row(want_v[p, h], t, *ref.quantise_row(v[b, h]), "v")
            sl = want_k[p, h]
            for d in range(D):
                sl[ref.k_code(t, d)] = gk[p, h, ref.k_code(t, d)]
            for c in range(4):
                sl[ref.k_scale(t, c)] = gk[p, h, ref.k_scale(t, c)]
    assert np.array_equal(gv, want_v)
    assert np.array_equal(gk, want_k)
    # rotation: fp16 rounding (2^-11) plus fp32 sine, cosine, products and sum (under 2^-20 of the pair's size)
    rot_q = np.stack([ref.rope(q[b], n - 1, THETA) for b, n in enumerate(lens)])
    rot_k = np.stack([ref.rope(k[b], n - 1, THETA) for b, n in enumerate(lens)])
    size = lambda x: np.abs(x.astype(np.float64)).max()
    assert np.all(np.abs(to_host(qo) - rot_q) <= 2.0 ** -11 * np.abs(rot_q) + 2.0 ** -20 * size(q) + 2.0 ** -25)
    # K: within half a step of its scale of the rotated value, whose rounding comes on top
    val, s = _rows_of(gk, "k", bt, lens), _scales_of(gk, "k", bt, lens)
    slack = 2.0 ** -11 * np.abs(rot_k) + 2.0 ** -20 * size(k)
    assert np.all(np.abs(val - rot_k) <= s / 2 + slack)
    amax = np.abs(rot_k).reshape(B, Hkv, 4, 32).max(-1).repeat(32, -1)
    assert np.all(7 * s >= amax * (1 - 2.0 ** -10)) and np.all(s <= amax / 7 * 1.125 * (1 + 2.0 ** -10) + 2.0 ** -17)
    for b, n in enumerate(lens):                      # position 0 rotates by nothing: the reference's bytes
        if n == 1:
            for h in range(Hkv):
                qq, byte = ref.quantise_row(k[b, h])
                assert np.array_equal(val[b, h], qq * np.repeat(ref.SCALES[byte], 32))


def test_append_in_place_and_strided_rows_write_the_same_bytes(api):
    r = np.random.default_rng(7)
    lens = np.array([40, 3, 17], np.int32)
    Hq, Hkv, B = 14, 2, 3
    bt, pages = _table(r, lens)
    rows = synth.normal_fp16(r, (B, Hq + 2 * Hkv, D))
    outs = []
    for form in ("packed", "in place", "strided"):
        dr, dbt, dl = dev(rows, bt, lens)
        kp, vp = (torch.zeros((pages, Hkv, 1088), dtype=torch.uint8, device="cuda") for _ in "kv")
        q, k, v = dr[:, :Hq], dr[:, Hq:Hq + Hkv], dr[:, Hq + Hkv:]
        if form == "strided":
            got = api.kv_append_rope_int4(q, k, v, kp, vp, dbt, dl, THETA, row_stride=(Hq + 2 * Hkv) * D)
            assert np.array_equal(to_host(dr)[:, Hq:], rows[:, Hq:])        # k and v are only read
        else:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
            got = api.kv_append_rope_int4(q, k, v, kp, vp, dbt, dl, THETA,
                                          q_out=torch.empty_like(q) if form == "packed" else None)
        outs.append((to_host(got.contiguous()), to_host(kp), to_host(vp)))
    for o in outs[1:]:
        assert all(np.array_equal(x, y) for x, y in zip(outs[0], o))


def test_rotation_rounds_its_products_and_their_sum(api):
    """Bit for bit the rotation in single fp32 operations (each rounded once, with
    the same cosines and sines): what makes every call write the same bytes."""
    r = np.random.default_rng(12)
    n, Hq, Hkv = 4000, 28, 4
    q, k, v = (to_dev(synth.normal_fp16(r, (n, h, D)), torch) for h in (Hq, Hkv, Hkv))
    bt = torch.arange(n // 16, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()
    lens = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros((n // 16, Hkv, 1088), dtype=torch.uint8, device="cuda") for _ in "kv")
    inv = torch.tensor([THETA ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64).float().cuda()
    ang = (lens - 1).float()[:, None] * inv
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def rotate(x):
        a, b = x.float().split(D // 2, -1)
        ac, bs, bc, as_ = a * c, b * s, b * c, a * s
        return torch.cat([ac - bs, bc + as_], -1).half()
    out = api.kv_append_rope_int4(q, k, v, kp, vp, bt, lens, THETA, q_out=torch.empty_like(q))
    assert torch.equal(out, rotate(q))
    # a small batch's kernel: the same values as the prompt's
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    few = torch.tensor([0, 1, 17, 1999, 2000, 3999], device="cuda")
    out2 = api.kv_append_rope_int4(q[few], k[few], v[few], kp2, vp2, bt[few], lens[few], THETA,
                                   q_out=torch.empty_like(q[few]))
    assert torch.equal(out2, out[few])
    rows = [api.kv_read_int4(*pools, bt[few], lens[few], 1, starts=lens[few] - 1) for pools in ((kp, vp), (kp2, vp2))]
    assert torch.equal(rows[0][0], rows[1][0]) and torch.equal(rows[0][1], rows[1][1])


def test_append_of_extreme_rows(api):
    """Zeros, the largest and the smallest fp16 numbers, infinities and NaN:
    V is not rotated, so its bytes are the reference's."""
    r = np.random.default_rng(8)
    big, tiny = np.float16(65504), np.float16(2.0 ** -24)
    v = synth.normal_fp16(r, (8, 1, D))
    v[0] = 0
    v[1, 0, :32], v[1, 0, 40], v[1, 0, 70] = big, -big, tiny
    v[2] = np.where(r.random(D) < 0.5, tiny, -tiny)
    v[3, 0, 5], v[4, 0, 100], v[5, 0, 127] = np.inf, -np.inf, np.nan
    v[6] = (r.standard_normal(D) * 2.0 ** -15).astype(np.float16)
    v[7, 0, :32] = np.float16(7.0) * np.float16(0.25)            # amax = 7 s exactly
    lens = np.arange(1, 9, dtype=np.int32)
    bt = np.zeros((8, 1), np.int32)
    k = np.zeros_like(v)
    vp = np.zeros((1, 1, 1088), np.uint8)
    dq, dk, dv, dkp, dvp, dbt, dl = dev(np.zeros((8, 1, D), np.float16), k, v, vp, vp, bt, lens)
    api.kv_append_rope_int4(dq, dk, dv, dkp, dvp, dbt, dl, THETA)
    want = vp.copy()
    for b in range(8):
        ref.store_row(want[0, 0], b, *ref.quantise_row(v[b, 0]), "v")
    assert np.array_equal(to_host(dvp), want)
    _, back = api.kv_read_int4(dkp, dvp, dbt[:1].contiguous(), dl[7:].clone(), 8)
    got, val = to_host(back)[0, :, 0], ref.unpack(want, "v")[0, 0, :8]
    assert np.array_equal(got.astype(np.float64), val, equal_nan=True)
    assert np.isnan(got[3, :32]).all() and np.isfinite(got[3, 32:]).all()


def test_append_skips_bad_pages_and_empty_rows(api):
    r = np.random.default_rng(9)
    lens = np.array([5, 0, -3, 20, 33, 4], np.int32)
    bt = np.array([[0, 1], [1, 1], [1, 1], [2, 7], [3, 3], [-1, 0]], np.int32)   # 7: outside; 33 tokens: past the row; -1
    kp = r.integers(0, 256, (4, 2, 1088)).astype(np.uint8)
    q, k, v = (synth.normal_fp16(r, (6, n, D)) for n in (4, 2, 2))
    dq, dk, dv, dkp, dvp, dbt, dl = dev(q, k, v, kp, kp, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_append_rope_int4(dq, dk, dv, dkp, dvp, dbt, dl, THETA, err_flag=err)
    assert int(err.item()) == 1
    for got in (to_host(dkp), to_host(dvp)):
        assert np.any(got[0] != kp[0]) and np.array_equal(got[1:], kp[1:])
    assert np.array_equal(to_host(dq)[1:3], q[1:3])


def test_prompt_append_equals_token_by_token(api):
    """T rows of one sequence in one call (pages shared by neighbours) give the
    bytes of T calls."""
    r = np.random.default_rng(10)
    T, Hq, Hkv = 75, 7, 1
    bt, pages = _table(r, [T])
    q, k, v = (synth.normal_fp16(r, (T, n, D)) for n in (Hq, Hkv, Hkv))
    dq, dk, dv = dev(q, k, v)
    dbt = to_dev(np.repeat(bt, T, 0), torch)
    dl = torch.arange(1, T + 1, dtype=torch.int32, device="cuda")
    pools = [torch.zeros((pages, Hkv, 1088), dtype=torch.uint8, device="cuda") for _ in range(4)]
    q1 = api.kv_append_rope_int4(dq, dk, dv, pools[0], pools[1], dbt, dl, THETA, q_out=torch.empty_like(dq))
    for i in range(T):
        qi = dq[i:i + 1].clone()
        api.kv_append_rope_int4(qi, dk[i:i + 1].clone(), dv[i:i + 1].clone(), pools[2], pools[3], dbt[:1],
                                dl[i:i + 1].clone(), THETA)
        assert torch.equal(qi[0], q1[i])
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_long_prompt_append(api):
    """More rows than are appended one per CTA, an odd number of them, some of
    length 0 and one with a page outside the pool: the bytes of smaller calls."""
    r = np.random.default_rng(11)
    T, Hq, Hkv = 611, 6, 3
    bt, pages = _table(r, [T])
    q, k, v = dev(*(synth.normal_fp16(r, (T, n, D)) for n in (Hq, Hkv, Hkv)))
    table = np.repeat(bt, T, 0)
    table[100] = pages
    lens = np.arange(1, T + 1, dtype=np.int32)
    lens[[7, 200]] = 0
    dbt, dl = dev(table, lens)
    mark = torch.full_like(q, 5.0)
    pools = [torch.zeros((pages, Hkv, 1088), dtype=torch.uint8, device="cuda") for _ in range(4)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q1 = api.kv_append_rope_int4(q, k, v, pools[0], pools[1], dbt, dl, THETA, q_out=mark.clone(), err_flag=err)
    assert int(err.item()) == 1
    q2 = mark.clone()
    for i in range(0, T, 200):
        j = min(i + 200, T)
        part = [x[i:j].clone() for x in (q, k, v, dbt, dl)]
        q2[i:j] = api.kv_append_rope_int4(*part[:3], pools[2], pools[3], part[3], part[4], THETA, q_out=mark[i:j].clone())
    assert torch.equal(q1, q2) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert bool((q1[[7, 200]] == 5.0).all()) and not bool((q1[100] == 5.0).any())


# ---- read -----------------------------------------------------------------------
@pytest.mark.parametrize("Hkv,lens,T,starts", [
    (1, [1], 1, None), (4, [37, 16, 0], 40, None), (2, [100, 31, 250], 19, [3, 16, 240]), (8, [17, 64], 64, [-5, 63]),
    (3, [48, 48, 48, -2], 16, [16, 48, 2 ** 31 - 1, -2 ** 31]), (1, [2000], 2000, None)])
def test_read_back(api, Hkv, lens, T, starts):
    r = np.random.default_rng(200 + T)
    lens = np.asarray(lens, np.int32)
    bt, pages = _table(r, lens)
    kp, vp = (r.integers(0, 256, (pages, Hkv, 1088)).astype(np.uint8) for _ in "kv")
    for p in (kp, vp):
        p[..., 1024:] = r.integers(0, 227, p[..., 1024:].shape)
        p[:, :, 1030] = 0xFF                                     # a group that reads as NaN
    dkp, dvp, dbt, dl = dev(kp, vp, bt, lens)
    ds = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    mark = torch.full((len(lens), T, Hkv, D), 7.5, dtype=torch.float16, device="cuda")
    ko, vo = mark.clone(), mark.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_read_int4(dkp, dvp, dbt, dl, T, starts=ds, k_out=ko, v_out=vo, err_flag=err)
    assert int(err.item()) == 0
    for pool, out, which in ((kp, ko, "k"), (vp, vo, "v")):
        want = to_host(mark).astype(np.float64)
        rows = ref.unpack(pool, which)
        for b, n in enumerate(lens):
            for i in range(T):
                t = (starts[b] if starts else 0) + i
                if 0 <= t < n:
                    want[b, i] = rows[bt[b, t // 16], :, t % 16]
        with np.errstate(over="ignore"):
            want = want.astype(np.float16)                       # (a code of -8 at the largest scales passes 65504)
        assert np.array_equal(to_host(out), want, equal_nan=True), which
    # tensors that the call makes: zeros where the caller's were left alone
    held = [ko != 7.5, vo != 7.5]
    torch.full((4 * ko.numel(),), 3.0, dtype=torch.float16, device="cuda")       # (memory that held something)
    for got, given, h in zip(api.kv_read_int4(dkp, dvp, dbt, dl, T, starts=ds), (ko, vo), held):
        rows = h.any(-1, keepdim=True)
        assert torch.equal(got.nan_to_num(9.0), torch.where(rows, given, torch.zeros_like(given)).nan_to_num(9.0))


def test_read_reports_bad_pages_and_leaves_their_rows(api):
    kp = torch.zeros((2, 1, 1088), dtype=torch.uint8, device="cuda")
    bt = torch.tensor([[0, 5, -1, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    k = torch.full((1, 64, 1, D), 3.0, dtype=torch.float16, device="cuda")
    v = k.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_read_int4(kp, kp, bt, lens, 64, k_out=k, v_out=v, err_flag=err)
    assert int(err.item()) == 1
    for x in (k, v):
        assert torch.all(x[:, 16:48] == 3.0) and torch.all(x[:, :16] == 0) and torch.all(x[:, 48:] == 0)


# ---- attention --------------------------------------------------------------------
def _poison(pool, bt, lens):
    """Bytes past each sequence's length hold NaN scales and any codes."""
    for which, p in zip("kv", pool):
        at = ref.k_scale if which == "k" else ref.v_scale
        for b, n in enumerate(lens):
            if n > 0 and n % 16:
                for t in range(n % 16, 16):
                    for c in range(4):
                        p[bt[b, (n - 1) // 16], :, at(t, c)] = 0xFF


@pytest.mark.parametrize("G,Hkv,lens", [
    (7, 1, [37]), (7, 4, [512]), (1, 2, [1, 15, 16, 17, 31, 32, 33]), (8, 2, [0, 257, 1000, -4]), (3, 1, [300, 2]),
    (5, 3, [129, 128, 127]), (2, 8, [64, 4097]), (6, 1, [2049, 16]), (4, 2, [1] * 40)])
def test_attention(api, G, Hkv, lens):
    r = np.random.default_rng(300 + G + Hkv)
    lens = np.asarray(lens, np.int32)
    bt, pages = _table(r, lens)
    kp, vp = ref.random_pool(r, pages, Hkv), ref.random_pool(r, pages, Hkv)
    _poison((kp, vp), bt, lens)
    q = synth.normal_fp16(r, (len(lens), G * Hkv, D))
    mc = max(int(lens.max()), 1)
    bt = bt if bt.shape[1] * 16 >= mc else np.pad(bt, ((0, 0), (0, 1)), constant_values=-1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_gqa_decode_int4(*dev(q, kp, vp, bt, lens), max_context=mc, err_flag=err)
    assert int(err.item()) == 0
    want = ref.attend(q, lambda p: ref.unpack(kp[p], "k"), lambda p: ref.unpack(vp[p], "v"), bt, lens, 1 / math.sqrt(D))
    ref.check_attention(to_host(out), want, int(lens.max()), f"G={G}")
    assert np.all(to_host(out)[lens <= 0] == 0)


@pytest.mark.parametrize("B,Hkv,lens", [(300, 2, [33, 1, 0, 700]), (2100, 2, [17]), (5, 1, [9000, 10, 10, 10, 8000])])
def test_attention_shares_a_batch_out(api, B, Hkv, lens):
    """Batches that take several rounds of the prefix sum over the lengths,
    that have more pairs than tickets, that are very uneven."""
    r = np.random.default_rng(600 + B)
    lens = np.resize(np.asarray(lens, np.int32), B)
    bt, pages = _table(r, lens)
    kp, vp = ref.random_pool(r, pages, Hkv), ref.random_pool(r, pages, Hkv)
    q = synth.normal_fp16(r, (B, 3 * Hkv, D))
    mc = int(lens.max())
    out = to_host(api.paged_gqa_decode_int4(*dev(q, kp, vp, bt, lens), max_context=mc))
    some = list(range(min(B, 8))) + [B // 2, B - 2, B - 1]
    want = ref.attend(q[some], lambda p: ref.unpack(kp[p], "k"), lambda p: ref.unpack(vp[p], "v"), bt[some], lens[some],
                      1 / math.sqrt(D))
    ref.check_attention(out[some], want, mc)
    # every row alone gives what the batch gave, to the order of the sums
    for b in (1, B // 2 + 1):
        alone = to_host(api.paged_gqa_decode_int4(*dev(q[b:b + 1], kp, vp, bt[b:b + 1], lens[b:b + 1]), max_context=mc))
        assert np.abs(alone[0].astype(np.float64) - out[b].astype(np.float64)).max() <= 2.0 ** -8


@pytest.mark.parametrize("spread,qstd", [(2.0 ** -12, 1.0), (600.0, 0.004), (9000.0, 2.0 ** -12)])
def test_attention_keeps_its_range(api, spread, qstd):
    """Pages of very small and very large values."""
    r = np.random.default_rng(17)
    lens = np.array([70, 33], np.int32)
    bt, pages = _table(r, lens)
    kp, vp = ref.random_pool(r, pages, 2, spread), ref.random_pool(r, pages, 2, spread)
    q = synth.normal_fp16(r, (2, 8, D), std=qstd)
    out = api.paged_gqa_decode_int4(*dev(q, kp, vp, bt, lens), max_context=80, sm_scale=0.05)
    want = ref.attend(q, lambda p: ref.unpack(kp[p], "k"), lambda p: ref.unpack(vp[p], "v"), bt, lens, 0.05)
    ref.check_attention(to_host(out), want, 70, f"spread {spread}")


def test_attention_reports_long_lengths_and_bad_pages(api):
    r = np.random.default_rng(18)
    lens = np.array([100, 40], np.int32)
    bt, pages = _table(r, lens)
    kp, vp = ref.random_pool(r, pages, 1), ref.random_pool(r, pages, 1)
    q = synth.normal_fp16(r, (2, 7, D))
    k_of, v_of = lambda p: ref.unpack(kp[p], "k"), lambda p: ref.unpack(vp[p], "v")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_gqa_decode_int4(*dev(q, kp, vp, bt, lens), max_context=64, err_flag=err)
    assert int(err.item()) == 1                            # the first 64 of the 100 tokens
    ref.check_attention(to_host(out), ref.attend(q, k_of, v_of, bt, np.minimum(lens, 64), 1 / math.sqrt(D)), 64)
    bad = bt.copy()
    bad[0, 2], bad[1, 0] = pages, -1                       # skipped: the other tokens are attended to
    err.zero_()
    out = api.paged_gqa_decode_int4(*dev(q, kp, vp, bad, lens), max_context=112, err_flag=err)
    assert int(err.item()) == 1
    one = lambda b, keep: ref.attend(q[b:b + 1], k_of, v_of, bt[b:b + 1, keep], [len(keep) * 16 - (12 if b == 0 else 8)],
                                     1 / math.sqrt(D))
    ref.check_attention(to_host(out)[:1], one(0, [0, 1, 3, 4, 5, 6]), 100)
    ref.check_attention(to_host(out)[1:], one(1, [1, 2]), 40)


@pytest.mark.parametrize("Hq,Hkv,lens", [(7, 1, [1]), (28, 4, [16, 513, 1, 40]), (8, 8, [15, 33]), (15, 3, [1000, 128, 129])])
def test_fused_step_equals_append_then_attention(api, Hq, Hkv, lens):
    r = np.random.default_rng(400 + Hq)
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    bt, pages = _table(r, lens)
    kp, vp = ref.random_pool(r, pages, Hkv), ref.random_pool(r, pages, Hkv)
    _poison((kp, vp), bt, lens)
    qkv = synth.normal_fp16(r, (B, (Hq + 2 * Hkv) * D + 64))        # rows longer than q | k | v
    dqkv, dkp, dvp, dbt, dl = dev(qkv, kp, vp, bt, lens)
    kp2, vp2 = dkp.clone(), dvp.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_gqa_decode_int4(dqkv, dkp, dvp, dbt, dl, int(lens.max()), qkv_theta=THETA, n_q_heads=Hq, err_flag=err)
    assert int(err.item()) == 0 and np.array_equal(to_host(dqkv), qkv)
    rows = dqkv[:, :(Hq + 2 * Hkv) * D].reshape(B, Hq + 2 * Hkv, D)
    q, k, v = (t.contiguous() for t in rows.split([Hq, Hkv, Hkv], 1))
    api.kv_append_rope_int4(q, k, v, kp2, vp2, dbt, dl, THETA)
    assert torch.equal(dkp, kp2) and torch.equal(dvp, vp2)          # the same bytes, and nothing else
    two = api.paged_gqa_decode_int4(q, kp2, vp2, dbt, dl, int(lens.max()))
    assert torch.equal(out, two)
    gk, gv = to_host(kp2), to_host(vp2)
    want = ref.attend(to_host(q), lambda p: ref.unpack(gk[p], "k"), lambda p: ref.unpack(gv[p], "v"), bt, lens,
                      1 / math.sqrt(D))
    ref.check_attention(to_host(out), want, int(lens.max()))


def test_fused_step_past_the_bound_appends_nothing(api):
    r = np.random.default_rng(19)
    lens = np.array([65, 0, 20], np.int32)
    bt, pages = _table(r, [80, 16, 32])
    kp, vp = ref.random_pool(r, pages, 1), ref.random_pool(r, pages, 1)
    qkv = synth.normal_fp16(r, (3, 9 * D))
    dqkv, dkp, dvp, dbt, dl = dev(qkv, kp, vp, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_gqa_decode_int4(dqkv, dkp, dvp, dbt, dl, 64, qkv_theta=THETA, n_q_heads=7, err_flag=err)
    assert int(err.item()) == 1 and np.all(to_host(out)[1] == 0)
    changed = {int(p) for p in np.argwhere(np.any(to_host(dkp) != kp, axis=(1, 2)))[:, 0]}
    assert changed == {int(bt[2, 1])}


# ---- the calls together, streams, graphs, workspaces -------------------------------------
def test_a_sequence_from_prompt_to_decode(api):
    """A prompt written in one call, decode steps in the fused form, the cache
    read back: attention over the pages equals attention over the rows read."""
    r = np.random.default_rng(20)
    Hq, Hkv, T, steps = 14, 2, 45, 8
    bt, pages = _table(r, [T + steps])
    dbt = to_dev(bt, torch)
    kp, vp = (torch.full((pages, Hkv, 1088), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
    q, k, v = dev(*(synth.normal_fp16(r, (T, n, D)) for n in (Hq, Hkv, Hkv)))
    lens = torch.arange(1, T + 1, dtype=torch.int32, device="cuda")
    api.kv_append_rope_int4(q, k, v, kp, vp, dbt.expand(T, -1).contiguous(), lens, THETA)
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    for _ in range(steps):
        n += 1
        qkv = to_dev(synth.normal_fp16(r, (1, (Hq + 2 * Hkv) * D)), torch)
        out = api.paged_gqa_decode_int4(qkv, kp, vp, dbt, n, T + steps, qkv_theta=THETA, n_q_heads=Hq)
    kr, vr = api.kv_read_int4(kp, vp, dbt, n, T + steps)
    kr, vr = to_host(kr)[0].astype(np.float64), to_host(vr)[0].astype(np.float64)
    rot = ref.rope(to_host(qkv)[0, :Hq * D].reshape(Hq, D), T + steps - 1, THETA).astype(np.float16)[None]
    pad = lambda x: np.concatenate([x, np.zeros((-len(x) % 16, Hkv, D))]).reshape(-1, 16, Hkv, D).transpose(0, 2, 1, 3)
    kk, vv = pad(kr), pad(vr)
    want = ref.attend(rot, lambda p: kk[p], lambda p: vv[p], np.arange(len(kk))[None], [T + steps], 1 / math.sqrt(D))
    # (the rotation in 64 bits may round to the neighbouring fp16 number: 2^-10 |q| on a score)
    ref.check_attention(to_host(out), want, T + steps)


def test_captured_step_replays_on_new_data(api):
    r = np.random.default_rng(21)
    lens = np.array([200, 700], np.int32)
    bt, pages = _table(r, lens + 16)
    kp, vp = ref.random_pool(r, pages, 4), ref.random_pool(r, pages, 4)
    dkp, dvp, dbt, dl = dev(kp, vp, bt, lens)
    qkv = to_dev(synth.normal_fp16(r, (2, 36 * D)), torch)
    ws = torch.zeros(api.load().paged_gqa_decode_window_workspace_size(2, 28, 4, 800, 800, 0, 128), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((2, 28, D), dtype=torch.float16, device="cuda")
    call = lambda: api.paged_gqa_decode_int4(qkv, dkp, dvp, dbt, dl, 720, qkv_theta=THETA, n_q_heads=28, workspace=ws,
                                             out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for _ in range(3):
        dl += 1
        qkv.copy_(to_dev(synth.normal_fp16(r, (2, 36 * D)), torch))
        kp2, vp2 = dkp.clone(), dvp.clone()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        again = api.paged_gqa_decode_int4(qkv, kp2, vp2, dbt, dl, 720, qkv_theta=THETA, n_q_heads=28)
        assert torch.equal(got, again) and torch.equal(dkp, kp2) and torch.equal(dvp, vp2)


def test_one_workspace_serves_shapes_in_turn_and_results_repeat(api):
    r = np.random.default_rng(22)
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    first = {}
    for turn in range(2):
        for i, (Hkv, G, lens) in enumerate(((4, 7, [3000]), (1, 8, [5000, 16]), (2, 3, [1, 900, 44]), (8, 1, [2500] * 3))):
            rr = np.random.default_rng(50 + i)
            lens = np.asarray(lens, np.int32)
            bt, pages = _table(rr, lens)
            kp, vp = ref.random_pool(rr, pages, Hkv), ref.random_pool(rr, pages, Hkv)
            q = synth.normal_fp16(rr, (len(lens), G * Hkv, D))
            out = api.paged_gqa_decode_int4(*dev(q, kp, vp, bt, lens), max_context=int(lens.max()), workspace=ws)
            if turn == 0:
                first[i] = out
            else:
                assert torch.equal(first[i], out)
    assert int(ws[:16384].sum().item()) == 0               # the tickets are left at zero


def test_two_streams_with_their_own_workspaces(api):
    r = np.random.default_rng(23)
    lens = np.array([6000], np.int32)
    bt, pages = _table(r, lens)
    kp, vp, dbt, dl = dev(ref.random_pool(r, pages, 4), ref.random_pool(r, pages, 4), bt, lens)
    qs = [to_dev(synth.normal_fp16(r, (1, 28, D)), torch) for _ in range(2)]
    want = [api.paged_gqa_decode_int4(q, kp, vp, dbt, dl, 6000) for q in qs]
    n = api.load().paged_gqa_decode_window_workspace_size(1, 28, 4, 6000, 6000, 0, 128)
    wss = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for q, ws, o, s in zip(qs, wss, outs, streams):
            api.paged_gqa_decode_int4(q, kp, vp, dbt, dl, 6000, workspace=ws, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_offsets_past_32_bits(api):
    """A pool whose last pages lie beyond 4 GiB."""
    pages, Hkv = 1_000_100, 4
    r = np.random.default_rng(24)
    kp, vp = (torch.empty((pages, Hkv, 1088), dtype=torch.uint8, device="cuda") for _ in "kv")
    bt = np.array([[pages - 1, 3, pages - 2]], np.int32)
    small = ref.random_pool(r, 3, Hkv), ref.random_pool(r, 3, Hkv)
    for i, p in enumerate(bt[0]):
        kp[p], vp[p] = to_dev(small[0][i], torch), to_dev(small[1][i], torch)
    q, k, v = dev(*(synth.normal_fp16(r, (1, n, D)) for n in (28, Hkv, Hkv)))
    dbt, dl = dev(bt, np.array([40], np.int32))
    api.kv_append_rope_int4(q, k, v, kp, vp, dbt, dl, THETA)
    out = api.paged_gqa_decode_int4(q, kp, vp, dbt, dl, 48)
    kr, vr = api.kv_read_int4(kp, vp, dbt, dl, 40)
    got = [np.stack([to_host(x[p]) for p in bt[0]]) for x in (kp, vp)]
    K, V = ref.unpack(got[0], "k"), ref.unpack(got[1], "v")
    for x, y in ((kr, K), (vr, V)):
        assert np.array_equal(to_host(x)[0].astype(np.float64), y.transpose(0, 2, 1, 3).reshape(48, Hkv, D)[:40])
    want = ref.attend(to_host(q), lambda p: K[p], lambda p: V[p], np.arange(3)[None], [40], 1 / math.sqrt(D))
    ref.check_attention(to_host(out), want, 40)


# ---- the binding on CUDA tensors: the native marshalling and the checked path ------------
def test_checked_and_native_paths_agree(api):
    """A stream given by name takes the checked path, none the native one."""
    r = np.random.default_rng(30)
    lens = np.array([90, 17], np.int32)
    bt, pages = _table(r, lens)
    kp, vp, dbt, dl = dev(ref.random_pool(r, pages, 2), ref.random_pool(r, pages, 2), bt, lens)
    q, k, v = dev(*(synth.normal_fp16(r, (2, n, D)) for n in (14, 2, 2)))
    qkv = torch.cat([q, k, v], 1).reshape(2, -1).contiguous()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    here = torch.cuda.current_stream()
    calls = (lambda **a: (api.kv_append_rope_int4(q, k, v, kp, vp, dbt, dl, THETA, q_out=torch.empty_like(q), **a), kp, vp),
             lambda **a: api.kv_read_int4(kp, vp, dbt, dl, 33, starts=dl - 20, **a),
             lambda **a: (api.paged_gqa_decode_int4(q, kp, vp, dbt, dl, 96, workspace=ws, err_flag=err, **a),),
             lambda **a: (api.paged_gqa_decode_int4(qkv, kp, vp, dbt, dl, 96, workspace=ws, qkv_theta=THETA, n_q_heads=14,
                                                    **a), kp, vp),
             lambda **a: (api.paged_gqa_decode_window(q, kp, vp, dbt, dl, 96, 20, 3, workspace=ws, sm_scale=-0.1, **a),))
    for call in calls:
        a = [t.clone() for t in call()]
        assert all(torch.equal(x, y) for x, y in zip(a, call(stream=here)))


def test_refusals_on_cuda_tensors(api):
    from w4a16_decode_paged_gb300._lib import W4A16Error
    kp = torch.zeros((4, 2, 1088), dtype=torch.uint8, device="cuda")
    bt = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 14, D), dtype=torch.float16, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="q"):
        api.paged_gqa_decode_int4(q.float(), kp, kp, bt, n, 64, workspace=ws)
    with pytest.raises(ValueError, match="v_pool"):
        api.paged_gqa_decode_int4(q, kp, kp[:2], bt, n, 64, workspace=ws)
    with pytest.raises(ValueError, match="block_table"):
        api.paged_gqa_decode_int4(q, kp, kp, bt.cpu(), n, 64, workspace=ws)
    with pytest.raises(ValueError, match="out"):
        api.paged_gqa_decode_window(q, kp, kp, bt, n, 64, 3, workspace=ws, out=torch.empty((1, 14, D), device="cuda"))
    with pytest.raises(ValueError, match="window"):
        api.paged_gqa_decode_window(q, kp, kp, bt, n, 64, -3, workspace=ws)
    with pytest.raises(W4A16Error, match="max_context"):
        api.paged_gqa_decode_int4(q, kp, kp, bt, n, 65, workspace=ws)
    with pytest.raises(W4A16Error, match="Hq=13"):
        api.paged_gqa_decode_int4(q[:, :13].contiguous(), kp, kp, bt, n, 64, workspace=ws)
    with pytest.raises(W4A16Error, match="theta"):
        api.kv_append_rope_int4(q, q[:, :2].contiguous(), q[:, :2].contiguous(), kp, kp.clone(), bt, n, 0.0)
    with pytest.raises(ValueError, match="T=0"):
        api.kv_read_int4(kp, kp, bt, n, 0)
