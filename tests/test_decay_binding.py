"""The decayed attention's and the beam search's wrappers call the library with the tensors' device current and that
device's stream, whichever device is current outside.  On the CPU: library, guard and streams are recorders."""
import contextlib

import pytest
import torch

import recurrent_state_02_gb300 as la
from recurrent_state_02_gb300 import _native
from test_binding_device import DEV, FakeTensor

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(params=[0, 1], ids=["other", "same"])
def calls(request, monkeypatch):
    """(entry point, device current during the call, its last argument) of every call; cuda:1 is current or not."""
    state, made = {"dev": request.param}, []

    @contextlib.contextmanager
    def guard(device):
        prev, state["dev"] = state["dev"], torch.device(device).index
        try:
            yield
        finally:
            state["dev"] = prev

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                made.append((name, state["dev"], args[-1]))
                return 0
            return fn

    monkeypatch.setattr(la, "_device_guard", guard)
    monkeypatch.setattr(la, "_stream", lambda device: 1000 + torch.device(device).index)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["dev"])
    monkeypatch.setattr(_native, "lib", lambda: Lib())
    monkeypatch.setattr(torch, "empty_like", lambda t: FakeTensor(t.shape, t.dtype, t.device))
    monkeypatch.setattr(torch, "empty", lambda shape, device=None, dtype=F32: FakeTensor(shape, dtype, torch.device(device)))
    return made


def test_wrappers_use_the_tensors_device(calls):
    B, K, H, T, r, dv, V = 2, 3, 4, 70, 128, 64, 500
    q, k, v = (FakeTensor((B, H, T, n), BF) for n in (r, r, dv))
    S, decay = FakeTensor((B, H, r, dv), F32), FakeTensor((H,), F32)
    la.decay_prefill(q, k, v, decay, S0=S)
    la.decay_backward(q, k, v, v, decay, S0=S, dS_T=S)
    la.decay_prefill_varlen(*(FakeTensor((T, H, n), BF) for n in (r, r, dv)), decay, FakeTensor((B + 1,), I32), S0=S)
    la.decay_decode_step(*(FakeTensor((B, H, 1, n), BF) for n in (r, r, dv)), decay, S)
    la.beam_select(FakeTensor((B, K, V), F32), FakeTensor((B, K), F32), done=FakeTensor((B, K), U8), eos=1)
    la.state_reorder(FakeTensor((B * K, H, r, dv), F32), FakeTensor((B, K), I32), z=FakeTensor((B * K, H, r), F32))
    la.decay_prefill_workspace_bytes(B, H, T, r, dv, device=DEV)
    la.decay_backward_workspace_bytes(B, H, T, r, dv, device=DEV)
    entries = {"la_decay_prefill", "la_decay_backward", "la_decay_prefill_varlen", "la_decay_decode_step", "la_beam_select",
               "la_state_reorder", "la_decay_prefill_workspace_bytes", "la_decay_backward_workspace_bytes"}
    assert {name for name, _, _ in calls} == entries
    for name, dev, last in calls:
        assert dev == 1, name
        assert name.endswith("bytes") or last == 1001, name


def test_tensors_on_two_devices_are_refused(calls):
    other = torch.device("cuda", 0)
    q, v, S = FakeTensor((1, 2, 4, 128), BF), FakeTensor((1, 2, 4, 64), BF), FakeTensor((1, 2, 128, 64), F32)
    with pytest.raises(ValueError):
        la.decay_prefill(q, FakeTensor(q.shape, BF, other), v, FakeTensor((2,), F32))
    with pytest.raises(ValueError):
        la.decay_prefill(q, q, v, FakeTensor((2,), F32, other))
    with pytest.raises(ValueError):
        la.decay_prefill(q, q, v, FakeTensor((2,), F32), S0=FakeTensor(S.shape, F32, other))
    with pytest.raises(ValueError):
        la.beam_select(FakeTensor((1, 2, 9), F32), FakeTensor((1, 2), F32, other))
    with pytest.raises(ValueError):
        la.state_reorder(S, FakeTensor((1, 1), I32, other))
    assert calls == []
