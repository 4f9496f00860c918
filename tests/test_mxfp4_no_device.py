"""Without a GPU the MXFP4 calls return an error, as the others do (CPU: a process
that sees no device; nothing can be launched there)."""
import os
import subprocess
import sys

import pytest

CALL = """
from w4a16_decode_paged_gb300 import _lib
L, A = _lib.load(), 1 << 20
m, k, n = {sizes}
got = [L.w4a16_gemm_mxfp4(A, m, k, A, A, n, None, None, A, A, 1 << 20, None, None),
       L.w4a16_gemm_silu_mul_mxfp4(A, m, k, A, A, A, A, n, A, A, 1 << 20, None, None),
       L.w4a4_gemm_mxfp4(A, A, m, k, A, A, n, None, None, A, A, 1 << 20, None, None),
       L.mxfp4_quantize(A, m, k, A, A, None), L.mxfp4_dequantize(A, A, m, k, A, None)]
print(got, L.w4a16_last_error())
assert got == [4] * 5
"""


@pytest.fixture(scope="module", autouse=True)
def library():
    from w4a16_decode_paged_gb300 import build
    build.build()


@pytest.mark.parametrize("sizes", [(1, 128, 1), (1, 512, 640), (2, 18944, 3584), (4, 1024, 256), (8, 1024, 256), (40, 512, 300),
                                   (300, 1024, 2000)])
def test_no_device(sizes):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CALL.format(sizes=sizes)], cwd=root, capture_output=True, text=True,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
