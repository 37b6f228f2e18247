"""The host code of the vocabulary loss, the expert moves and the gradient norms
(validation, shapes, workspace sizes) under the address and undefined-behaviour
sanitizers, as tests/test_sanitizers.py runs the rest of the library."""
import importlib.util
import os

import pytest


def test_host_paths_under_address_and_ub_sanitizers(tmp_path):
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_sanitizers.py")
    spec = importlib.util.spec_from_file_location("sanitizer_runs", path)
    runs = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(runs)
    rt = runs._clang_asan_runtime()
    if rt is None:
        pytest.skip("clang AddressSanitizer runtime not found")
    from sparse_communication_adam_amd.build import build
    lib = build(sanitize=True, out=str(tmp_path / "libscape_asan.so"))
    out = runs._run(["tests/test_vocab_expert_abi.py"], runs._env(rt, SCAPE_LIB=lib))
    assert "passed" in out
