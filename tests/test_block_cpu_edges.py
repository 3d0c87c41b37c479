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


def test_numbers_beyond_their_fields_are_refused():
    """ctypes would keep the low bits: 2^32 + 1 sequences as one."""
    a = dict(batch=1, heads=2, kv_heads=1, d=64, io_dtype=0, scale=0.125, q_len=4, k_len=4, window=0, sinks=0)
    assert lact._struct(lact.Attention, *a.values()).heads == 2
    for name in ("batch", "heads", "kv_heads", "d"):
        with pytest.raises(ValueError, match=name):
            lact._struct(lact.Attention, *dict(a, **{name: (1 << 32) + 1}).values())
    with pytest.raises(ValueError, match="cols"):
        lact._struct(lact.NormProblem, 1, (1 << 32) + 5, 0, 1e-6)
    with pytest.raises(ValueError, match="pairs"):
        lact._struct(lact.RotaryProblem, 1, 1, 0, 64, (1 << 32) + 4, 0, 0, 1.0, 4, 0)
    for n in (1 << 63, -(1 << 63) - 1, (1 << 64) + 5):
        with pytest.raises(ValueError, match="window"):
            lact._int(n, "window")
    assert lact._int(-(1 << 63), "start") == -(1 << 63) and lact._int(torch.tensor(7), "start") == 7
    q = torch.zeros(1, 2, 4, 64)
    for kw in (dict(window=(1 << 64) + 5), dict(sinks=1 << 64)):
        with pytest.raises(ValueError, match="64-bit"):
            lact.window_attention(q, q, q, **kw)
        with pytest.raises(ValueError, match="64-bit"):
            lact.window_attention_backward(q, q, q, q, q[..., 0], dO=q, **kw)
    with pytest.raises(ValueError, match="64-bit"):
        lact.rotary(q, freqs=torch.ones(4, dtype=torch.float64), start=1 << 63)
