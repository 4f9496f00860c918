"""The native argument marshalling (CPU): which file is loaded, and that neither
the library's build nor the calls need it."""
import os
import subprocess
import sys
import warnings

import pytest

torch = pytest.importorskip("torch")

from w4a16_decode_paged_gb300 import _lib, api, build  # noqa: E402


def test_its_file_is_named_for_the_interpreter_and_torch(monkeypatch):
    here = build.args_lib()
    assert sys.implementation.cache_tag in here and torch.__version__ in here
    folder = build._torch()[0]
    monkeypatch.setattr(build, "_torch", lambda: (folder, "9.9.9"))
    assert build.args_lib() != here and "9.9.9" in build.args_lib()
    monkeypatch.setattr(build, "_torch", lambda: (None, None))
    assert build.args_lib() is None


def test_the_library_is_built_without_torch_headers(monkeypatch, tmp_path, capfd):
    monkeypatch.setattr(build, "_torch", lambda: (str(tmp_path), "1.0"))       # a torch with no headers
    assert build.build_args(force=True) is None
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "headers" in capfd.readouterr().err
    monkeypatch.setattr(build, "_torch", lambda: (None, None))                 # no torch at all
    assert build.build_args(force=True) is None and build.build() == build.LIB


def test_a_module_that_does_not_compile_is_an_error_behind_the_library(monkeypatch, tmp_path):
    bad = tmp_path / "bad.cpp"
    bad.write_text("#error no\n")
    monkeypatch.setattr(build, "ARGS_SRC", str(bad))
    monkeypatch.setattr(build, "args_lib", lambda: str(tmp_path / "x.so"))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert os.path.exists(build.LIB)


@pytest.mark.parametrize("what", ["missing", "broken", "no torch"])
def test_calls_go_on_without_it(monkeypatch, tmp_path, what):
    build.build()
    path = tmp_path / "m.so"
    if what == "broken":
        path.write_bytes(b"no module")
    monkeypatch.setattr(build, "args_lib", lambda: None if what == "no torch" else str(path))
    monkeypatch.setattr(_lib, "_native", None)
    with pytest.warns(RuntimeWarning, match="slower"):
        assert _lib.native() is None
    with warnings.catch_warnings():                                            # said once
        warnings.simplefilter("error")
        assert _lib.native() is None
    calls = []

    class Rec:
        def __getattr__(self, name):
            return lambda *a: (calls.append(name), 0)[1]
    monkeypatch.setattr(api, "load", Rec)
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    monkeypatch.setattr(api, "_cuda", lambda t: True)
    monkeypatch.setattr(api, "stream_handle", lambda stream=None: 0)
    kp = torch.zeros((4, 1, 1088), dtype=torch.uint8)
    bt, n = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    api.kv_append_rope_int4(h(1, 7, 128), h(1, 1, 128), h(1, 1, 128), kp, kp.clone(), bt, n, 1e6)
    api.kv_read_int4(kp, kp, bt, n, 1)
    api.paged_gqa_decode_int4(h(1, 7, 128), kp, kp, bt, n, 64, workspace=ws)
    api.paged_gqa_decode_window(h(1, 7, 128), kp, kp, bt, n, 64, 5, workspace=ws)
    assert calls == ["kv_append_rope_int4", "kv_read_int4", "paged_gqa_decode_int4", "paged_gqa_decode_window_int4"]


def test_it_loads_here():
    build.build()
    code = "from w4a16_decode_paged_gb300 import _lib; m = _lib.native(); assert m is not None and m.append and m.read"
    subprocess.run([sys.executable, "-W", "error::RuntimeWarning", "-c", code], check=True, cwd=build.ROOT)
