"""One workspace for every MXFP4 product (CPU): as large as any call's, and every call
splits with it as with any amount."""
import ctypes
import random

import pytest

torch = pytest.importorskip("torch")

SMS = 152


@pytest.fixture(scope="module")
def lib():
    from w4a16_decode_paged_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_it_is_enough_for_every_call(lib):
    rng, room = random.Random(5), lib.mxfp4_workspace_size()
    assert 8192 < room < 32 << 20
    wants = []
    for _ in range(5000):
        m, n, k = int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 18)), 128 * int(2 ** rng.uniform(0, 10))
        wants += [lib.w4a16_gemm_mxfp4_workspace_size(m, k, n, 0), lib.w4a16_gemm_mxfp4_workspace_size(m, k, n, 1),
                  lib.w4a4_gemm_mxfp4_workspace_size(m, k, n)]
        for kind in (0, 1, 2):
            plans = []
            for space in (room, 1 << 40):
                p = (ctypes.c_int32 * 7)()
                assert lib.w4a16_debug_mxfp4_plan(kind, m, k, n, space, SMS, p) == 0
                plans.append(list(p))
            assert plans[0] == plans[1], (kind, m, n, k)
    assert max(wants) <= room


def test_one_calls_size_is_not_anothers(lib):
    """One row of a projection wants none in fp16 and 28 parts in 4 bits."""
    assert lib.w4a16_gemm_mxfp4_workspace_size(1, 3584, 512, 0) == 0
    assert lib.w4a4_gemm_mxfp4_workspace_size(1, 3584, 512) > 1 << 20


def test_binding(lib):
    from w4a16_decode_paged_gb300 import api
    assert api.mxfp4_workspace(device="cpu").numel() == lib.mxfp4_workspace_size()
    assert api.mxfp4_workspace(1, 3584, 512, "a4", device="cpu").numel() == lib.w4a4_gemm_mxfp4_workspace_size(1, 3584, 512)
    assert not api.mxfp4_workspace(device="cpu").any()
    with pytest.raises(ValueError, match="all three"):
        api.mxfp4_workspace(1, 3584, device="cpu")
    with pytest.raises(ValueError, match="kind"):
        api.mxfp4_workspace(1, 3584, 512, "a8", device="cpu")
