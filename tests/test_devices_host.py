"""CPU: the calls around the attention take tensors of the handle's device only, and
its current stream (stand-ins for tensors and for the library; no GPU)."""
import ctypes as C

import numpy as np
import pytest

from test_qkv_host import pa  # noqa: F401

HQ, HKV, N_POOL, MAX_PAGES, N = 4, 2, 6, 3, 5
HANDLE, DEVICE = 4096, 1


def on(device, dtype, *shape):
    """A tensor that says that it lies on this GPU."""
    import torch

    class OnGpu(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return device
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def tensors(device):
    import torch
    b, f, i8, i32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
    pool = (N_POOL, 16, HKV, 256)
    return dict(q=on(device, b, N, HQ, 256), k=on(device, b, N, HKV, 256), v=on(device, b, N, HKV, 256),
                qw=on(device, b, 256), kw=on(device, b, 256), pos=on(device, i32, N), bt=on(device, i32, N, MAX_PAGES),
                kp=on(device, i8, *pool), vp=on(device, i8, *pool), ks=on(device, f, *pool[:3]),
                vs=on(device, f, *pool[:3]), qo=on(device, b, N, HQ, 256), ko=on(device, b, N, HKV, 256))


def rope_call(pa, t):  # noqa: F811
    pa.pa_qk_norm_rope(C.c_void_p(HANDLE), t["q"], t["k"], t["qw"], t["kw"], 1e-6, pa.pa_rope(), t["pos"], t["qo"], t["ko"])


def append_call(pa, t):  # noqa: F811
    pa.pa_qkv_append(C.c_void_p(HANDLE), np.array([(0, 0, N, N)], np.int32), t["q"], t["k"], t["v"], t["qw"], t["kw"], 1e-6,
                     pa.pa_rope(), t["pos"], t["bt"], t["kp"], t["vp"], t["ks"], t["vs"], t["qo"])


def shared_call(pa, t):  # noqa: F811
    pa.pa_decode_shared(C.c_void_p(HANDLE), np.array([(0, 20, 1, 21)], np.int32), 16, t["q"], t["kp"], t["vp"], t["ks"],
                        t["vs"], t["bt"], 1, 0, 1.0, t["qo"])


CALLS = (("pa_qk_norm_rope", rope_call, "q k qw kw pos qo ko"),
         ("pa_qkv_append", append_call, "q k v qw kw pos bt kp vp ks vs qo"),
         ("pa_decode_shared", shared_call, "q kp vp ks vs bt qo"))


@pytest.mark.parametrize("name, call, used", CALLS, ids=[c[0] for c in CALLS])
def test_tensors_of_the_handles_device(pa, monkeypatch, name, call, used):  # noqa: F811
    calls, streams = [], []

    class Library:
        def __getattr__(self, attr):
            return lambda *args: calls.append((attr, args)) or 0
    monkeypatch.setattr(pa, "_lib", Library())
    monkeypatch.setitem(pa._geometry, HANDLE, (HQ, HKV, N_POOL, MAX_PAGES, DEVICE))
    monkeypatch.setattr(pa, "_torch_names", pa._torch()[:4] + (lambda index: streams.append(index) or 77,))
    call(pa, tensors(DEVICE))
    assert [c[0] for c in calls] == [name] and calls[0][1][-1] == 77 and streams == [DEVICE]
    other = tensors(0)
    for arg in used.split():
        with pytest.raises(ValueError, match="device 1, got 0"):
            call(pa, {**tensors(DEVICE), arg: other[arg]})
    assert len(calls) == 1


def test_device_of_no_handle(pa):  # noqa: F811
    assert pa.pa_device(None) == pa.pa_device(C.c_void_p()) == pa.pa_device(0) == -1
