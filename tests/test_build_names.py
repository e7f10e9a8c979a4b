"""The compiled calls are bound to the torch and the Python they were built with: their file
says which, and another pair finds it stale."""
import os
import sysconfig

import torch

from mxfp4_quantized_gemm_token_gb300 import build


def test_another_torch_or_python_builds_its_own(monkeypatch):
    build.build()
    assert os.path.exists(build.CALLS) and not build._stale()
    here = build.CALLS
    for change in (lambda m: m.setattr(torch, "__version__", "1.0"),
                   lambda m: m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-99.so")):
        with monkeypatch.context() as m:
            change(m)
            assert build.calls_path() != here
            m.setattr(build, "CALLS", build.calls_path())
            assert build._stale()
