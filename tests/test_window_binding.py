"""The windowed call's autograd binding on the CPU: what it does before the library is called."""
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
