"""Calls whose tensors are not on the current device are refused on the host: the
library launches on the current one."""
import ctypes
import importlib.util
import shutil
from types import SimpleNamespace

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib, build

BF = torch.bfloat16


def on(index):
    return SimpleNamespace(is_cuda=True, device=torch.device("cuda", index),
                           get_device=lambda: index)


def test_other_devices_are_refused(monkeypatch):
    monkeypatch.setattr(mxq, "_current_device", lambda: 1)
    mxq._need_cuda(on(1), None, on(1))
    for tensors in ([on(0)], [on(1), on(0)], [None, on(2)]):
        with pytest.raises(ValueError, match="the current device is cuda:1"):
            mxq._need_cuda(*tensors)


def test_status_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(mxq, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: SimpleNamespace(device=torch.device("cuda", 0),
                                                            cuda_stream=0))
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        mxq.sync_status("cuda:0")


def compiled_calls(tmp_path, entry, current_device):
    """A copy of the compiled calls of its own, whose entry points are all `entry`, with a
    current device as told."""
    def tell(at):
        at[0] = current_device
        return 0

    device = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.POINTER(ctypes.c_int32))(tell)
    _lib.load_calls(torch._C._cuda_getCurrentRawStream)
    path = shutil.copy(build.CALLS, str(tmp_path / "_attn_calls.so"))
    spec = importlib.util.spec_from_file_location("_attn_calls", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    entries = [ctypes.cast(f, ctypes.c_void_p).value for f in [entry] * 5 + [device]]
    mod.connect(*entries, _lib.check, torch._C._cuda_getCurrentRawStream)
    mod.kept = entry, device
    return mod


@pytest.mark.gpu
@pytest.mark.parametrize("current", [0, 1])
def test_compiled_calls(tmp_path, current):
    """With entry points that only count, and a current device as told."""
    reached = []
    entry = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: reached.append(1) or 0)
    calls = compiled_calls(tmp_path, entry, current)
    d = "cuda:0"
    q, kv = torch.zeros(2, 4, 64, dtype=BF, device=d), torch.zeros(2, 2, 64, dtype=BF, device=d)
    cache = torch.zeros(3, 16, 2, 64, dtype=BF, device=d)
    n = torch.zeros(2, dtype=torch.int32, device=d)
    ws = torch.zeros(256, dtype=torch.uint8, device=d)
    slots = torch.zeros(2, dtype=torch.int64, device=d)
    table, cu = torch.zeros(2, 3, dtype=torch.int32, device=d), n.new_zeros(3)
    for call in (lambda: calls.append(kv, kv, cache, cache, slots, None, None, q, None, None, None,
                                      False),
                 lambda: calls.decode(q, cache, cache, table, n, None, 0, None, None, None, False,
                                      None, ws),
                 lambda: calls.prompt(q, kv, kv, cu, None, None, True, 0, None, False, None, ws)):
        reached.clear()
        if current == 0:
            call()
            assert len(reached) == 1
        else:
            with pytest.raises(ValueError, match="tensors are on cuda:0, the current device is"
                                                 " cuda:1"):
                call()
            assert not reached
