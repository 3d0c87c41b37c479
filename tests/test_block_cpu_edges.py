"""The block's operators without a GPU: layouts of results, workspaces' sizes
and launches' limits at unusual arguments."""
import ctypes

import numpy as np
import pytest

import block_precision as BP
from oracle import lact_block as OB
from test_gpu_block import ATTENTION

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


def _back_ws(**kw):
    a = dict(batch=1, heads=8, kv_heads=8, d=128, io_dtype=lact.DTYPE_BF16, scale=0.1, q_len=32768, k_len=32768,
             window=128, sinks=4)
    a.update(kw)
    n = lact.lib().lact_window_attention_backward_workspace_size(ctypes.byref(lact.Attention(**a)))
    assert n > 0
    return n, 8 * a["batch"] * a["heads"] * a["q_len"] + 256   # all, and the rows' two statistics


@pytest.mark.parametrize("kw", [
    dict(sinks=32768), dict(sinks=1 << 40), dict(sinks=4096), dict(sinks=1024, window=1), dict(batch=64), dict(),
    dict(batch=8, heads=32, kv_heads=32, q_len=4096, k_len=4096), dict(sinks=32767), dict(window=0, sinks=9),
    dict(batch=8, heads=32, kv_heads=32, q_len=4096, k_len=4096, sinks=4096), dict(q_len=1 << 29, k_len=1 << 29),
    dict(batch=4096, heads=64, kv_heads=64, q_len=500, k_len=500, window=3)])
def test_workspace_of_the_backward_is_bounded(kw):
    """At most 512 + 256 jobs of sink tiles, each with dk and dv of 128 keys by
    d in fp32, beside the rows' statistics: whatever the sinks and the batch."""
    need, stats = _back_ws(**kw)
    assert need <= stats + 768 * 2 * 128 * 128 * 4 + 256
    if kw.get("sinks", 0) >= kw.get("k_len", 32768) or kw.get("window") == 0:
        assert need <= stats   # every row sees all keys before it: nothing to split


def test_a_long_row_of_few_sinks_is_still_split():
    assert _back_ws(sinks=4)[0] > _back_ws(sinks=0)[0] + 60 * 2 * 128 * 128 * 4 * 8


@pytest.mark.parametrize("dtype,d,at_once", [("F32", 8, 256), ("F32", 32, 256), ("F32", 64, 256), ("F32", 128, 256),
                                             ("BF16", 8, 512), ("BF16", 64, 512), ("BF16", 72, 256)])
def test_key_splits_fill_the_chip_once(dtype, d, at_once):
    """128 key heads' next tokens over long keys: as many splits as make one
    round of workgroups, by the LDS that a workgroup of the padded width takes."""
    a = lact.Attention(8, 16, 16, d, getattr(lact, "DTYPE_" + dtype), 0.1, 1, 1 << 20, 0, 0)
    need = lact.lib().lact_window_attention_workspace_size(ctypes.byref(a))
    assert need == 128 * (at_once // 128) * (d + 2) * 4   # a row's partial results and statistics, each a multiple of 256


FAKE = 1 << 20   # aligned, never dereferenced: every call here is refused first


def test_grids_beyond_a_launch_are_refused():
    """A launch ends at 2^32 - 1 threads, 2^24 - 1 workgroups of 256: what needs
    more is refused before any device work, not left to fail there."""
    U, L = lact.ERR_UNSUPPORTED, lact.lib()

    def st(heads, rows, d=8):
        return ctypes.byref(lact.Strides(heads * rows * d, rows * d, d))

    def attention(B, H, q_len, k_len, d=8, dtype=lact.DTYPE_BF16, kv=None, **kw):
        kv = kv or H
        p = lact.Attention(B, H, kv, d, dtype, 0.1, q_len, k_len, kw.get("window", 0), 0)
        a, b = st(H, q_len, d), st(kv, k_len, d)
        f = L.lact_window_attention_forward(ctypes.byref(p), FAKE, a, FAKE, b, FAKE, b, None, None, FAKE * 8, a, None,
                                            FAKE, 1 << 60, None)
        g = L.lact_window_attention_backward(ctypes.byref(p), FAKE, a, FAKE, b, FAKE, b, None, None, FAKE, a, FAKE,
                                             FAKE, a, FAKE * 8, a, FAKE * 9, b, FAKE * 10, b, FAKE, 1 << 60, None)
        return f, g

    assert attention(1 << 18, 1 << 6, 64, 64) == (U, U)            # 2^24 tiles of rows and of keys
    assert attention(1 << 18, 1 << 6, 1, 64)[0] == U               # 2^24 workgroups of few rows, 256 threads each
    assert attention(1 << 19, 1 << 6, 1, 64, 128, lact.DTYPE_F32)[0] == U   # 2^25, of 128 threads
    for B, T in ((1, 1 << 29), (1 << 24, 1)):
        p = lact.RotaryProblem(B, 1, 0, 8, 4, lact.DTYPE_BF16, 0, 1.0, T, 0)
        assert L.lact_rotary(ctypes.byref(p), FAKE, st(1, T), None, None, FAKE, None, FAKE * 8, st(1, T), None, None,
                             None) == U
    assert "more than a launch" in lact.last_error()


# ------------------------------------------------------------------ what fp32 results are held to
def _fp32_inputs(case):
    B, H, Hk, d, Lq, Lk = case[:6]
    rng = np.random.default_rng(sum(case[:8]))
    return [rng.standard_normal(s).astype(np.float32).astype(np.float64)
            for s in ((B, H, Lq, d), (B, Hk, Lk, d), (B, Hk, Lk, d), (B, H, Lq, d))]


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "x".join(str(x) for x in c[:8]))
def test_bounds_of_fp32_attention_tell_lesser_paths(case):
    """The bounds that fp32 results are held to pass the formulas themselves,
    and neither probabilities rounded to bf16's 8 bits nor scores from operands
    of 11 bits."""
    B, H, Hk, d, Lq, Lk, window, sinks, ql, kl = case
    q, k, v, g = _fp32_inputs(case)
    ref = OB.window_attention(q, k, v, window, sinks, 0.3, ql, kl, g)
    limits = BP.bounds(q, k, v, g, window, sinks, 0.3, ql, kl, ref)
    args = (q, k, v, g, window, sinks, 0.3, ql, kl)
    single, rms = BP.excess(BP.attention(*args), ref, limits)
    assert max([*single.values(), *rms.values(), 0]) < 0.01
    sees = [OB.visible(Lq if ql is None else ql[b], Lk if kl is None else kl[b], window, sinks).sum(1)
            for b in range(B)]
    if max((int(n.max()) for n in sees if n.size), default=0) < 2:
        return   # a probability of one is one in any number of bits
    for name, lesser in (("weights", dict(weight=lambda x: BP.rounded(x, 8))),
                         ("operands", dict(operand=lambda x: BP.rounded(x, 11)))):
        _, rms = BP.excess(BP.attention(*args, **lesser), ref, limits)
        assert min(rms.values()) > 5, (name, rms)
