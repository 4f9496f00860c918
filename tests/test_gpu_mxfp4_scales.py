"""What each scale byte of a weight means in the fp16 products, whatever the number of
rows: 104 to 140 (those that the quantiser writes) the block's values, fewer none, more
a block of NaN.  And what the 4-bit product makes of the smallest and largest bytes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 4, 5, 8, 9, 32, 33, 64, 65, 130]


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as a
    return a


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


def every_byte(rng, k, kt):
    """256 rows of weights; in row r the byte r for one of the blocks of tile kt, the others 127.
    The weights' bytes, their codes, and their values with the bytes' meaning."""
    code = rng.integers(0, 16, (256, k)).astype(np.uint8)
    byte = np.full((256, k // 32), 127, np.uint8)
    byte[np.arange(256), 4 * kt + np.arange(256) % 4] = np.arange(256)
    v = ref.values(code, np.where(byte < 104, 127, byte))
    v = np.where(np.repeat(byte < 104, 32, 1), 0.0, v)
    return code, byte, np.where(np.repeat(byte > 140, 32, 1), np.nan, v)


def hold(got, x, wv, what):
    fine = np.isfinite(wv).all(1)
    assert np.isnan(got[:, ~fine]).all(), what
    ref._hold(got[:, fine], x @ wv[fine].T, ref.sum_error(np.abs(x) @ np.abs(wv[fine]).T, x.shape[1]), what)


@pytest.mark.parametrize("k,kt", [(128, 0), (384, 1), (1280, 9)])
@pytest.mark.parametrize("m", ROWS)
def test_every_byte(api, m, k, kt):
    rng = np.random.default_rng(1000 * m + k)
    x = (rng.standard_normal((m, k)) * 2.0 ** -7).astype(np.float16)
    code, byte, wv = every_byte(rng, k, kt)
    y = api.w4a16_gemm_mxfp4(dev(x), dev(ref.pack(code)), dev(ref.tiles(byte)))
    hold(y.cpu().numpy().astype(np.float64), x.astype(np.float64), wv, f"{m} rows")


@pytest.mark.parametrize("m", ROWS)
def test_every_byte_of_a_gated_pair(api, m):
    rng = np.random.default_rng(m)
    k = 256
    x = (rng.standard_normal((m, k)) * 2.0 ** -7).astype(np.float16)
    code, byte, wv = every_byte(rng, k, 1)
    plain = np.full_like(byte, 122)
    pv = ref.values(code, plain)
    a, b = (dev(ref.pack(code)), dev(ref.tiles(byte))), (dev(ref.pack(code)), dev(ref.tiles(plain)))
    xs, some = x.astype(np.float64), np.isfinite(wv).all(1) & (byte.max(1) < 134)     # (outputs that fp16 holds)
    for gate, up, gv, uv in ((a, b, wv, pv), (b, a, pv, wv)):
        y = api.w4a16_gemm_silu_mul_mxfp4(dev(x), *gate, *up).cpu().numpy()
        assert np.isnan(y[:, 141:]).all()
        ref.check_silu(y[:, some], xs, gv[some], uv[some], f"{m} rows")


@pytest.mark.parametrize("m", [1, 130, 300])
def test_4_bit_product_of_zero_blocks_under_any_byte(api, m):
    """Blocks whose codes are zero count as zero under every byte but 255, byte 0 among them
    (what some quantisers write for them), on either side."""
    rng = np.random.default_rng(m)
    n, k = 256, 512
    cx, cw = rng.integers(0, 16, (m, k)).astype(np.uint8), rng.integers(0, 16, (n, k)).astype(np.uint8)
    bx, bw = np.full((m, k // 32), 126, np.uint8), np.full((n, k // 32), 125, np.uint8)
    cw[:, 64:96] &= 8                                          # zeros, of either sign
    bw[:, 2] = np.arange(n) % 255
    cx[:, 480:512] &= 8
    bx[:, 15] = np.arange(m) % 255
    y = api.w4a4_gemm_mxfp4(dev(ref.pack(cx)), dev(ref.tiles(bx)), dev(ref.pack(cw)), dev(ref.tiles(bw)))
    ref.check_product(y.cpu().numpy(), ref.values(cx, bx), ref.values(cw, bw))


@pytest.mark.parametrize("m", [1, 130])
def test_4_bit_product_of_the_smallest_and_largest_bytes(api, m):
    """Bytes 0 and 1 on one side, 254 and 253 on the other: 2^-127 and 2^-126 are what they stand for."""
    rng = np.random.default_rng(m)
    n, k = 130, 256
    cx, cw = rng.integers(0, 16, (m, k)).astype(np.uint8), rng.integers(0, 16, (n, k)).astype(np.uint8)
    bx = rng.choice([0, 1], (m, k // 32)).astype(np.uint8)
    bw = rng.choice([253, 254], (n, k // 32)).astype(np.uint8)
    flip = np.arange(k // 32) % 2 == 1                          # the large bytes on x's side
    bx[:, flip], bw[:, flip] = rng.choice([253, 254], (m, flip.sum())), rng.choice([0, 1], (n, flip.sum()))
    y = api.w4a4_gemm_mxfp4(dev(ref.pack(cx)), dev(ref.tiles(bx)), dev(ref.pack(cw)), dev(ref.tiles(bw)))
    ref.check_product(y.cpu().numpy(), ref.values(cx, bx), ref.values(cw, bw))
