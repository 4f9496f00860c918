"""How the MXFP4 products are dealt (CPU, for 152 SMs): tiles cover the output once,
parts are what the workspace holds, and less room means fewer parts."""
import ctypes
import random

import pytest

SMS = 152


@pytest.fixture(scope="module")
def lib():
    from w4a16_decode_paged_gb300 import _lib, build
    build.build()
    return _lib.load()


def plan(lib, kind, m, n, k, space):
    p = (ctypes.c_int32 * 7)()
    assert lib.w4a16_debug_mxfp4_plan(kind, m, k, n, space, SMS, p) == 0
    return list(p)


def sizes(count, seed):
    rng = random.Random(seed)
    for _ in range(count):
        yield tuple(int(2 ** rng.uniform(0, b)) for b in (13, 15, 7.5))


def test_tiles_and_workspace(lib):
    for m, n, kt in sizes(2000, 1):
        k = 128 * kt
        for kind in (0, 1, 2):
            need = lib.w4a4_gemm_mxfp4_workspace_size(m, k, n) if kind == 2 else \
                lib.w4a16_gemm_mxfp4_workspace_size(m, k, n, kind)
            if kind < 2 and plan(lib, kind, m, n, k, 0)[0] == 0:
                assert need == 0
                continue
            tm, tn, whole, split, parts, ctas = plan(lib, kind, m, n, k, need)[1:]
            wide = 128 if kind == 1 else tn
            assert whole + split == -(-m // tm) * -(-n // wide)
            assert need == (8192 + split * parts * tm * tn * 4 if parts > 1 else 0) and split * parts <= SMS
            assert ctas == min(SMS, whole + split * parts)
            # (the most that a call can want)
            assert plan(lib, kind, m, n, k, 1 << 40)[1:] == [tm, tn, whole, split, parts, ctas]
            assert plan(lib, kind, m, n, k, 0)[5] == 1
            if need:
                less = plan(lib, kind, m, n, k, need - 1)
                assert 8192 * (less[5] > 1) + less[4] * (less[5] if less[5] > 1 else 0) * less[1] * less[2] * 4 < need


def test_refusals(lib):
    p = (ctypes.c_int32 * 7)()
    assert lib.w4a16_debug_mxfp4_plan(3, 1, 128, 1, 0, SMS, p) == 1 and lib.w4a16_debug_mxfp4_plan(0, 1, 128, 1, 0, SMS, None) == 1
    for m, k, n in ((0, 128, 1), (1, 0, 1), (1, 192, 1), (1, 128, 0), (1048577, 128, 1), (1, 131200, 1), (1, 128, 1048577)):
        assert lib.w4a16_debug_mxfp4_plan(2, m, k, n, 0, SMS, p) == 3
    for kind in (0, 2):                                            # the largest sizes: 22 and 34 million tiles
        _, tm, tn, whole = plan(lib, kind, 1048576, 1048576, 131072, 0)[:4]
        assert whole == -(-1048576 // tm) * -(-1048576 // tn) < 2 ** 31
