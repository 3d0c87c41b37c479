"""The block's operators without a GPU: layouts of results, workspaces' sizes
and launches' limits at unusual arguments."""
import ctypes

import numpy as np
import pytest

lact = pytest.importorskip("test_layers_amd.lact", reason="liblact.so not built")
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(2, 3, 5, 8), lambda: torch.zeros(2, 5, 3, 8).transpose(1, 2),
    lambda: torch.zeros(5, 2, 3, 32).permute(1, 2, 0, 3)[..., 8:16], lambda: torch.zeros(2, 3, 9, 8)[:, :, :5],
    lambda: torch.zeros(1, 1, 5, 8).expand(2, 3, 5, 8), lambda: torch.zeros(0, 3, 5, 8), lambda: torch.zeros(1, 1, 1, 8),
    lambda: torch.zeros(2, 5, 9, 8)[:, :, ::3].transpose(1, 2)])
def test_layouts_of_results_take_no_memory(make):
    """Planned on tensors without memory, as torch lays out a result like the input."""
    t = make()
    x = lact._like(t)
    want = torch.empty(t.shape) if 0 in t.stride() else torch.empty_like(t)
    assert x.device.type == "meta" and x.shape == t.shape and x.stride() == want.stride() and x.dtype == t.dtype
