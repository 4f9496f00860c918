"""Tensors that the MXFP4 calls make are seen by torch's modes, and filled where new
memory is to be, as those of torch's own calls are."""
import pytest

torch = pytest.importorskip("torch")

from torch.overrides import TorchFunctionMode  # noqa: E402
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from w4a16_decode_paged_gb300 import api as a
    return a


class Dispatched(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.made.append((out.dtype, tuple(out.shape)))
        return out


class Called(TorchFunctionMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in getattr(func, "__name__", ""):
            self.made.append((out.dtype, tuple(out.shape)))
        return out


def calls(api):
    """Each call, and what it makes."""
    m, n, k = 5, 40, 256
    x = torch.randn(m, k, device="cuda").half()
    w = api.mxfp4_quantize(torch.randn(n, k, device="cuda").half())
    q = api.mxfp4_quantize(x)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    y = (torch.float16, (m, n))
    return [(lambda: api.mxfp4_quantize(x), [(torch.int32, (m, k // 8)), (torch.uint8, (1, k // 128, 512))]),
            (lambda: api.mxfp4_dequantize(*q), [(torch.float16, (m, k))]),
            (lambda: api.w4a16_gemm_mxfp4(x, *w, workspace=ws), [y]),
            (lambda: api.w4a16_gemm_silu_mul_mxfp4(x, *w, *w, workspace=ws), [y]),
            (lambda: api.w4a4_gemm_mxfp4(*q, *w, workspace=ws), [y])]


@pytest.mark.parametrize("mode", [Dispatched, Called])
def test_modes_see_what_is_made(api, mode):
    for call, made in calls(api):
        want = call()
        with mode() as seen:
            got = call()
        assert seen.made == made
        for a, b in zip(want if isinstance(want, tuple) else (want,), got if isinstance(got, tuple) else (got,)):
            assert a.shape == b.shape and (a.dtype == torch.uint8 or torch.equal(a, b))   # (scale bytes past M are free)


def test_new_memory_is_filled_where_asked_for(api):
    x = torch.randn(5, 256, device="cuda").half()
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.utils.deterministic.fill_uninitialized_memory
        like = torch.empty(8, dtype=torch.uint8, device="cuda")[0]
        _, s = api.mxfp4_quantize(x)
    finally:
        torch.use_deterministic_algorithms(False)
    rows = api.mxfp4_untile_scales(s, 128)
    assert bool((rows[5:] == like).all())
