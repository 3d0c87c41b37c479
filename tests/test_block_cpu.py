"""The operators around the fast-weight layer, without a GPU: the oracle
against differences and special cases, the host's frequency tables, and every
refusal of the C ABI and the binding (each before any device work)."""
import ctypes

import numpy as np
import pytest

from oracle import lact_block as OB

lact = pytest.importorskip("test_layers_amd.lact", reason="liblact.so not built")
torch = pytest.importorskip("torch")

FAKE = 1 << 20   # aligned, never dereferenced: every call here is refused first


# ------------------------------------------------------------------ oracle
def _attention_inputs(rng, B=2, H=4, Hk=2, d=8, Lq=7, Lk=9):
    return [rng.standard_normal(s) for s in ((B, H, Lq, d), (B, Hk, Lk, d), (B, Hk, Lk, d), (B, H, Lq, d))]


def test_visible_by_hand():
    see = OB.visible(3, 5, 2, 1)   # rows at positions 2, 3, 4
    assert see.tolist() == [[True, True, True, False, False], [True, False, True, True, False],
                            [True, False, False, True, True]]
    assert not OB.visible(4, 2, 3, 1)[:2].any()   # rows before the first key
    assert OB.visible(3, 3, 0, 0).tolist() == np.tril(np.ones((3, 3), bool)).tolist()


@pytest.mark.parametrize("window,sinks,lens", [(3, 2, None), (0, 0, None), (2, 0, ([7, 4], [9, 3]))])
def test_attention_gradients_against_differences(window, sinks, lens):
    rng = np.random.default_rng(5)
    q, k, v, g = _attention_inputs(rng)
    ql, kl = lens or (None, None)
    f = lambda q, k, v: (OB.window_attention(q, k, v, window, sinks, 0.4, ql, kl)["o"] * g).sum()
    out = OB.window_attention(q, k, v, window, sinks, 0.4, ql, kl, dO=g)
    for n, name in enumerate(("dq", "dk", "dv")):
        for _ in range(6):
            x = [q, k, v]
            t = rng.standard_normal(x[n].shape)
            e = 1e-5
            up, dn = list(x), list(x)
            up[n], dn[n] = x[n] + e * t, x[n] - e * t
            # central difference: error e^2 f''' / 6 and rounding 1e-16 |f| / e
            assert abs((f(*up) - f(*dn)) / (2 * e) - (out[name] * t).sum()) < 1e-7 * (1 + np.abs(t).sum())


def test_attention_special_cases():
    rng = np.random.default_rng(6)
    q, k, v, _ = _attention_inputs(rng, Lq=9)
    one = OB.window_attention(q, k, v, 1, 0, 0.3)
    assert np.allclose(one["o"], np.repeat(v, 2, axis=1))          # only itself
    empty = OB.window_attention(q, k[:, :, :4], v[:, :, :4], 3, 2, 0.3)
    assert (empty["o"][:, :, :5] == 0).all() and (empty["lse"][:, :, :5] == -np.inf).all()
    flat = OB.window_attention(0 * q, k, v, 0, 0, 0.3)
    assert np.allclose(flat["o"][0, 0, 8], v[0, 0].mean(0)) and np.allclose(flat["lse"][0, 0, 8], np.log(9))


def test_norm_and_rotary_gradients_against_differences():
    rng = np.random.default_rng(7)
    x, r, g = (rng.standard_normal((5, 11)) for _ in range(3))
    w = rng.standard_normal(11)
    f = lambda x, w: (OB.add_rmsnorm(x, w, r, 0.1)[0] * g).sum()
    dx, dw = OB.add_rmsnorm_backward(x + r, w, g, None, 0.1)
    e = 1e-6
    for _ in range(5):
        t, u = rng.standard_normal(x.shape), rng.standard_normal(11)
        assert abs((f(x + e * t, w) - f(x - e * t, w)) / (2 * e) - (dx * t).sum()) < 1e-7
        assert abs((f(x, w + e * u) - f(x, w - e * u)) / (2 * e) - (dw * u).sum()) < 1e-7
    y = rng.standard_normal((2, 3, 4, 10))
    pos = np.array([[0, 1, 5, 1000000], [3, 2, 1, 0]])
    fr = OB.frequencies(4, 10000.0)
    for il in (False, True):
        z = OB.rotary(y, pos, fr, il, 1.5)
        back = OB.rotary(z, pos, fr, il, 1.5, inverse=True)
        t = rng.standard_normal(y.shape)
        assert np.allclose((z * t).sum(), (y * OB.rotary(t, pos, fr, il, 1.5, inverse=True)).sum())   # the adjoint
        assert np.allclose(back[..., :8], 2.25 * y[..., :8]) and (back[..., 8:] == y[..., 8:]).all()


# ------------------------------------------------------------------ frequency tables
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, context=4096),
                                dict(scaling="yarn", factor=2.5, context=100, slow=0.0, fast=2.0)])
@pytest.mark.parametrize("pairs,base", [(1, 10000.0), (2, 500000.0), (64, 10000.0), (33, 1000.0)])
def test_frequencies(pairs, base, kw):
    f, m = lact.rotary_frequencies(pairs, base, device="cpu", **kw)
    assert f.dtype == torch.float64
    np.testing.assert_allclose(f.numpy(), OB.frequencies(pairs, base, **kw), rtol=1e-13)
    want = 0.1 * np.log(kw["factor"]) + 1 if kw.get("scaling") == "yarn" else 1.0
    assert abs(m - want) < 1e-6
    if kw.get("scaling") == "ntk" and pairs > 1:
        plain = OB.frequencies(pairs, base)
        assert f[0] == 1.0 and abs(f[-1] / plain[-1] * kw["factor"] - 1) < 1e-12


@pytest.mark.parametrize("args,kw", [((-1,), {}), ((4000,), {}), ((4, 1.0), {}), ((4, float("nan")), {}),
                                     ((4,), dict(scaling="linear", factor=0.5)),
                                     ((4,), dict(scaling="ntk", factor=float("inf"))),
                                     ((4,), dict(scaling="yarn", factor=2.0, context=0)),
                                     ((4,), dict(scaling="yarn", factor=2.0, context=9, slow=3.0, fast=3.0))])
def test_frequency_refusals(args, kw):
    with pytest.raises(lact.LactError) as e:
        lact.rotary_frequencies(*args, device="cpu", **kw)
    assert e.value.status == lact.ERR_INVALID_ARG


def test_unknown_scaling_is_refused():
    with pytest.raises(ValueError):
        lact.rotary_frequencies(4, scaling="cubic", device="cpu")


# ------------------------------------------------------------------ refusals of the C ABI
def _attn(**kw):
    base = dict(batch=2, heads=4, kv_heads=2, d=64, io_dtype=lact.DTYPE_BF16, scale=0.125, q_len=64, k_len=64,
                window=16, sinks=4)
    base.update(kw)
    return lact.Attention(**base)


def _st(b=4 * 64 * 64, h=64 * 64, l=64):
    return ctypes.byref(lact.Strides(b, h, l))


def _fwd(p=None, ws=FAKE, ws_bytes=1 << 40, lse=None, q_lens=None, k_lens=None, **over):
    a = {n: (FAKE, _st()) for n in "qkv"}
    a["o"] = (FAKE * 8, _st())
    a.update(over)
    return lact.lib().lact_window_attention_forward(None if p is None else ctypes.byref(p), *a["q"], *a["k"],
                                                    *a["v"], q_lens, k_lens, *a["o"], lse, ws, ws_bytes, None)


def _bwd(p=None, ws=FAKE, ws_bytes=1 << 40, lse=FAKE, **over):
    a = {n: (FAKE, _st()) for n in ("q", "k", "v", "o", "dO")}
    a.update({n: (FAKE * (8 + i), _st()) for i, n in enumerate(("dq", "dk", "dv"))})
    a.update(over)
    return lact.lib().lact_window_attention_backward(
        None if p is None else ctypes.byref(p), *a["q"], *a["k"], *a["v"], None, None, *a["o"], lse, *a["dO"],
        *a["dq"], *a["dk"], *a["dv"], ws, ws_bytes, None)


BAD_ATTENTION = [
    (dict(batch=-1), lact.ERR_INVALID_ARG), (dict(heads=0), lact.ERR_INVALID_ARG),
    (dict(kv_heads=0), lact.ERR_INVALID_ARG), (dict(heads=3), lact.ERR_INVALID_ARG),
    (dict(d=0), lact.ERR_UNSUPPORTED), (dict(d=12), lact.ERR_UNSUPPORTED), (dict(d=136), lact.ERR_UNSUPPORTED),
    (dict(io_dtype=2), lact.ERR_INVALID_ARG), (dict(scale=0.0), lact.ERR_INVALID_ARG),
    (dict(scale=-1.0), lact.ERR_INVALID_ARG), (dict(scale=float("nan")), lact.ERR_INVALID_ARG),
    (dict(scale=float("inf")), lact.ERR_INVALID_ARG), (dict(scale=1e-37), lact.ERR_INVALID_ARG), (dict(q_len=-1), lact.ERR_INVALID_ARG),
    (dict(k_len=1 << 30), lact.ERR_INVALID_ARG), (dict(window=-1), lact.ERR_INVALID_ARG),
    (dict(sinks=-1), lact.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", BAD_ATTENTION)
def test_attention_refuses_bad_problems(kw, code):
    p = _attn(**kw)
    assert _fwd(p) == code and lact.last_error()
    assert _bwd(p) == code
    for size in (lact.lib().lact_window_attention_workspace_size,
                 lact.lib().lact_window_attention_backward_workspace_size):
        assert size(ctypes.byref(p)) == 0 and lact.last_error()


def test_attention_refuses_bad_tensors():
    I = lact.ERR_INVALID_ARG
    assert _fwd(None) == I and _bwd(None) == I
    for n in ("q", "k", "v", "o"):
        assert _fwd(_attn(), **{n: (None, _st())}) == I and n in lact.last_error()
        assert _fwd(_attn(), **{n: (FAKE, None)}) == I
        assert _fwd(_attn(), **{n: (FAKE + 8, _st())}) == I           # not 16-byte aligned
        assert _fwd(_attn(), **{n: (FAKE, _st(l=68))}) == I           # rows not 16-byte aligned
        assert _fwd(_attn(), **{n: (FAKE, _st(h=-4096))}) == I
        assert _fwd(_attn(), **{n: (FAKE, _st(b=1 << 60))}) == I
    for n in ("dO", "dq", "dk", "dv"):
        assert _bwd(_attn(), **{n: (None, _st())}) == I and n in lact.last_error()
    assert _bwd(_attn(), lse=None) == I
    assert _fwd(_attn(), lse=FAKE + 2) == I
    assert _fwd(_attn(), q_lens=FAKE + 4) == I and _fwd(_attn(), k_lens=FAKE + 4) == I
    # outputs whose rows fall on one another
    for st in (_st(l=0), _st(h=0), _st(b=0), _st(l=56), _st(h=64)):
        assert _fwd(_attn(), o=(FAKE, st)) == I and "overlap" in lact.last_error()
        assert _bwd(_attn(), dk=(FAKE, st)) == I


def test_outputs_that_are_inputs_are_refused():
    I = lact.ERR_INVALID_ARG
    two, three, four = FAKE * 2, FAKE * 3, FAKE * 4
    for n in ("q", "k", "v"):
        assert _fwd(_attn(), **{n: (two, _st()), "o": (two, _st())}) == I and "output" in lact.last_error()
    apart = dict(dq=(two, _st()), dk=(three, _st()), dv=(four, _st()))
    for n in ("q", "k", "v", "o", "dO"):
        assert _bwd(_attn(), **apart, **{n: (three, _st())}) == I and "output" in lact.last_error()
    assert _bwd(_attn(), **dict(apart, dv=(two, _st()))) == I and "same" in lact.last_error()
    assert _rot(_rp(), qo=(two, _st()), ko=(two, _st())) == I
    assert _rot(_rp(), k=(two, _st()), qo=(two, _st()), ko=(three, _st())) == I
    assert _rot(_rp(), q=(two, _st()), qo=(three, _st()), ko=(two, _st())) == I


def test_attention_workspace_checks():
    p = _attn(heads=2, kv_heads=2, q_len=1, k_len=5000, window=0, batch=1)   # few rows, keys split
    need = lact.lib().lact_window_attention_workspace_size(ctypes.byref(p))
    assert need > 0
    assert _fwd(p, ws_bytes=need - 1) == lact.ERR_WORKSPACE_TOO_SMALL
    assert _fwd(p, ws=None) == lact.ERR_INVALID_ARG and _fwd(p, ws=FAKE + 16) == lact.ERR_INVALID_ARG
    p = _attn()
    need = lact.lib().lact_window_attention_backward_workspace_size(ctypes.byref(p))
    assert need >= 2 * 4 * 64 * 4
    assert _bwd(p, ws_bytes=need - 1) == lact.ERR_WORKSPACE_TOO_SMALL
    assert _bwd(p, ws=FAKE + 128) == lact.ERR_INVALID_ARG


def test_attention_refuses_grids_beyond_a_launch():
    p = _attn(batch=1 << 20, heads=1 << 12, kv_heads=1 << 12, q_len=64, k_len=64)
    big = _st(b=64 * 64, h=64 * 64 << 20, l=64)
    assert _fwd(p, q=(FAKE, big), k=(FAKE, big), v=(FAKE, big), o=(FAKE * 8, big)) == lact.ERR_UNSUPPORTED


def test_nothing_to_do_is_accepted():
    assert _fwd(_attn(batch=0), q=(None, None), k=(None, None), v=(None, None), o=(None, None), ws=None,
                ws_bytes=0) == lact.OK
    assert _fwd(_attn(q_len=0), q=(None, None), o=(None, None), ws=None, ws_bytes=0) == lact.OK


def _rot(p=None, freqs=FAKE, positions=None, **over):
    a = {n: (FAKE, _st()) for n in ("q", "k", "qo", "ko")}
    a.update(qo=(FAKE * 8, _st()), ko=(FAKE * 9, _st()))
    a.update(over)
    return lact.lib().lact_rotary(None if p is None else ctypes.byref(p), *a["q"], *a["k"], freqs, positions,
                                  *a["qo"], *a["ko"], None)


def _rp(**kw):
    base = dict(batch=2, heads=4, kv_heads=2, d=64, pairs=32, io_dtype=lact.DTYPE_BF16, flags=0, mscale=1.0,
                tokens=64, start=0)
    base.update(kw)
    return lact.RotaryProblem(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(heads=0), -1), (dict(kv_heads=-1), -1), (dict(d=0), -2), (dict(d=8200), -2),
    (dict(pairs=-1), -1), (dict(pairs=33), -1), (dict(io_dtype=9), -1), (dict(flags=4), -1),
    (dict(mscale=float("inf")), -1), (dict(tokens=-1), -1), (dict(tokens=1 << 30), -1),
])
def test_rotary_refuses_bad_problems(kw, code):
    assert _rot(_rp(**kw)) == code and lact.last_error()


def test_rotary_refuses_bad_tensors():
    I = lact.ERR_INVALID_ARG
    assert _rot(None) == I
    for n in ("q", "k", "qo", "ko"):
        assert _rot(_rp(), **{n: (None, _st())}) == I
        assert _rot(_rp(), **{n: (FAKE + 1, _st())}) == I
        assert _rot(_rp(), **{n: (FAKE, _st(b=-8))}) == I
    assert _rot(_rp(), freqs=None) == I and _rot(_rp(), freqs=FAKE + 4) == I
    assert _rot(_rp(), positions=FAKE + 4) == I
    assert _rot(_rp(), qo=(FAKE * 8, _st(l=60))) == I and "overlap" in lact.last_error()
    assert _rot(_rp(), qo=(FAKE, _st(b=5 * 64 * 64))) == I and "in place" in lact.last_error()


def _norm(p=None, x=(FAKE, 256), r=(FAKE, 256), w=FAKE, h=(FAKE * 2, 256), y=(FAKE * 3, 256), y8=(None, 0),
          scales=None):
    return lact.lib().lact_add_rmsnorm_forward(None if p is None else ctypes.byref(p), *x, *r, w, *h, *y, *y8,
                                               scales, None)


def _np(**kw):
    base = dict(rows=8, cols=256, io_dtype=lact.DTYPE_BF16, eps=1e-6)
    base.update(kw)
    return lact.NormProblem(**base)


@pytest.mark.parametrize("kw,code", [(dict(rows=-1), -1), (dict(cols=0), -2), (dict(cols=32769), -2),
                                     (dict(io_dtype=3), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1)])
def test_norm_refuses_bad_problems(kw, code):
    p = _np(**kw)
    assert _norm(p) == code
    assert lact.lib().lact_add_rmsnorm_backward(ctypes.byref(p), FAKE, 256, FAKE, FAKE, 256, None, 0, FAKE, 256,
                                                FAKE, FAKE, 1 << 40, None) == code
    assert lact.lib().lact_add_rmsnorm_backward_workspace_size(ctypes.byref(p)) == 0


def test_norm_refuses_bad_tensors():
    I = lact.ERR_INVALID_ARG
    assert _norm(None) == I
    for kw in (dict(x=(None, 256)), dict(x=(FAKE + 1, 256)), dict(x=(FAKE, 255)), dict(x=(FAKE, -256)),
               dict(r=(FAKE, 100)), dict(h=(FAKE * 2, 0)), dict(y=(FAKE * 3, 0)), dict(w=None), dict(w=FAKE + 2),
               dict(y=(None, 0)), dict(y8=(FAKE, 256)), dict(y8=(FAKE, 8), scales=FAKE),
               dict(h=(FAKE, 512)), dict(y=(FAKE, 512)), dict(y=(FAKE * 2, 256))):
        assert _norm(_np(), **kw) == I, kw
    p = _np(rows=800)
    back = lambda dx=(FAKE, 256), dw=FAKE, ws=FAKE, n=1 << 40, dy=(FAKE, 256): lact.lib().lact_add_rmsnorm_backward(
        ctypes.byref(p), FAKE * 2, 256, FAKE, *dy, None, 0, *dx, dw, ws, n, None)
    need = lact.lib().lact_add_rmsnorm_backward_workspace_size(ctypes.byref(p))
    assert back(n=need - 1) == lact.ERR_WORKSPACE_TOO_SMALL
    assert back(dx=(None, 256)) == I and back(dx=(FAKE, 0)) == I and back(dy=(None, 0)) == I
    assert back(ws=None) == I and back(dw=FAKE + 1) == I and back(dx=(FAKE, 300)) == I


def test_norm_outputs_that_are_inputs_are_refused():
    I = lact.ERR_INVALID_ARG
    five = FAKE * 5
    for kw in (dict(x=(five, 256)), dict(r=(five, 256)), dict(h=(five, 256)), dict(y=(five, 256)), dict(w=five)):
        assert _norm(_np(), y8=(five, 256), scales=FAKE * 6, **kw) == I, kw
        assert _norm(_np(), y8=(FAKE * 6, 256), scales=five, **kw) == I, kw
    assert _norm(_np(), y8=(five, 256), scales=five) == I
    assert _norm(_np(), w=FAKE * 2) == I and _norm(_np(), w=FAKE * 3) == I
    p = _np(rows=800)
    back = lambda dx, dw: lact.lib().lact_add_rmsnorm_backward(
        ctypes.byref(p), FAKE * 2, 256, FAKE * 3, FAKE * 4, 256, FAKE * 5, 256, dx, 256, dw, FAKE * 6, 1 << 40, None)
    assert back(FAKE * 3, FAKE) == I and back(FAKE, FAKE) == I
    assert all(back(FAKE, FAKE * n) == I for n in (2, 3, 4, 5))


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_host_tensors_and_shapes():
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError):
        lact.window_attention(q, q, q)
    with pytest.raises(ValueError):
        lact.window_attention(q[0], q[0], q[0])
    with pytest.raises(ValueError):
        lact.window_attention(q.half(), q.half(), q.half())
    with pytest.raises(ValueError):
        lact.rotary(q, freqs=torch.ones(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        lact.add_rmsnorm(torch.zeros(3, 8), torch.ones(8))
    with pytest.raises(ValueError):
        lact.add_rmsnorm(torch.zeros(3, 8), torch.ones(9))

