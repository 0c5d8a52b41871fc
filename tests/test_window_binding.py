"""The windowed call's autograd binding on the CPU: what it does before the library is called."""
import contextlib
import types

import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa


@pytest.mark.parametrize("mode", [torch.enable_grad, torch.no_grad, torch.inference_mode])
def test_cpu_leaves_are_refused_as_such(mode):
    """CPU tensors that require a gradient get the binding's message, in every mode."""
    x = [torch.zeros(3, 2, 64, dtype=torch.bfloat16, requires_grad=True) for _ in range(3)]
    off = torch.tensor([0, 3])
    with mode(), pytest.raises(ValueError, match="CUDA"):
        jfa.window_attention(*x, off, off, 2)
    with mode(), pytest.raises(ValueError, match="CUDA"):
        jfa.WindowAttention.apply(*x, off, off, 2)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_graph_no_check(mode, monkeypatch):
    """Without a graph no accumulator is looked for (in inference mode none can be)."""
    seen = []
    monkeypatch.setattr(jfa.jfa, "_check_capture", lambda *t: seen.append(t))
    monkeypatch.setattr(jfa.jfa, "jfa_window_forward", lambda q, *a: (q * 2, q, None))
    x = [torch.ones(3, 2, 64, requires_grad=True) for _ in range(3)]
    off = torch.tensor([0, 3])
    with mode():
        out = jfa.window_attention(*x, off, off)
    assert not seen and not out.requires_grad
    assert jfa.window_attention(*x, off, off).requires_grad and len(seen) == 1


def test_status_is_read_on_the_workspaces_device(monkeypatch):
    """The stream that is waited for is one of the device that the workspace, and so the call, is on."""
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    @contextlib.contextmanager
    def stream(s):
        with device(s.device):
            yield

    lib = types.SimpleNamespace(jfa_check_status=lambda ptr, handle: calls.append((ptr, handle, current[0])) or 0)
    monkeypatch.setattr(jfa.jfa, "load_library", lambda *a: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=1000 + current[0]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    ws = types.SimpleNamespace(device=torch.device("cuda", 1), data_ptr=lambda: 4096)
    assert jfa.jfa_check_status(ws) == 0 and calls == [(4096, 1001, 1)]
    side = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)
    assert jfa.jfa_check_status(ws, side) == 0 and calls[1] == (4096, 77, 1) and current == [0]
    with pytest.raises(ValueError, match="stream"):
        jfa.jfa_check_status(ws, types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=5))
