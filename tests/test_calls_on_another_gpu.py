"""Calls whose tensors are on a GPU that is not the current one run on the tensors' GPU: it is the current one from
the first size asked of the library on, and the caller's again afterwards. On a machine without a GPU: tensors that
call themselves device tensors pass all checks and stop at the missing device, before any launch."""
import pytest
import torch

import fp8_group_quant_amd as fq
from test_mxfp4_kv4_abi import CALLS as NEW_CALLS
from test_serving_abi import EDEVICE, no_gpu
from test_serving_devices import attention, on_gpu

CALLS = dict(NEW_CALLS, attention=attention)


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs by name, the first of them current; the list of those that were current when the library was called."""
    state = dict(current=0, seen=[])

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *_):
            state["current"] = self.before

    class Library:
        def __init__(self, lib):
            self.lib = lib

        def __getattr__(self, name):
            if name not in ("fp8q_status_string", "fp8q_last_error"):
                state["seen"].append(state["current"])
            return getattr(self.lib, name)

    lib = Library(fq.load_library())
    monkeypatch.setattr(fq, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return state


@no_gpu
@pytest.mark.parametrize("stream", [0, None])
@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_gpu_becomes_the_current_one(gpus, name, stream):
    fn, kw = CALLS[name]()
    for index in (0, 1):
        gpus["seen"].clear()
        with pytest.raises(fq.Fp8qError) as e:
            fn(**{k: on_gpu(t.as_subclass(torch.Tensor), index) for k, t in kw.items()}, stream=stream)
        assert e.value.status == EDEVICE
        assert gpus["seen"] and set(gpus["seen"]) == {index} and gpus["current"] == 0


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_gpu_is_refused(gpus, name, monkeypatch):
    class Stream:
        device_index, cuda_stream = 1, 0

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    fn, kw = CALLS[name]()
    with pytest.raises(ValueError):
        fn(**kw, stream=Stream())
    with pytest.raises(fq.Fp8qError) as e:
        fn(**{k: on_gpu(t.as_subclass(torch.Tensor), 1) for k, t in kw.items()}, stream=Stream())
    assert e.value.status == EDEVICE and set(gpus["seen"]) == {1} and gpus["current"] == 0
