"""Window attention, rotary positions and add-and-norm on the GPU against the
fp64 oracle, at the sizes, masks, layouts and callers where they can go wrong.

Tolerances, with u the half step of the tensors' type (bf16 2^-8, fp32 2^-24):
a result x is rounded once (u |x|); for bf16 the kernels round probabilities
and their gradients once more before a product, which moves a sum by at most
u times the sum of magnitudes (the oracle's *_abs), and the backward reads the
forward's rounded o (the *_delta sums).  fp32 arithmetic: a score is a sum of d
products, off by (d + 2) 2^-24 of scale sum |q||k| (score_abs); with the
exponent's and the statistics' own roundings a probability is off by the
relative EPS below, and so is every sum of magnitudes, lengthened by the number
of its terms.
"""
import numpy as np
import pytest

from oracle import lact_block as OB

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def lact():
    from test_layers_amd import lact as L
    return L


def half_step(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(gen, shape, t, layout="heads"):
    if layout == "tokens":
        b, h, l, d = shape
        return torch.randn((b, l, h, d), generator=gen, device="cuda").to(t).transpose(1, 2)
    if layout == "wide":   # heads inside wider rows, tokens outermost
        b, h, l, d = shape
        return torch.randn((l, b, h, d + 24), generator=gen, device="cuda").to(t).permute(1, 2, 0, 3)[..., 8:8 + d]
    return torch.randn(shape, generator=gen, device="cuda").to(t)


def fp32_slack(ref, d, n, scale_abs=None):
    e = 2.0 ** -24
    s = ref["score_abs"]
    return e * (4 * (d + 2) * s + 8 * s + 2 * n + 64)


def check(name, got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape, name
    fine = np.isfinite(ref)
    assert (np.isfinite(got) == fine).all(), name
    assert (got[~fine] == ref[~fine]).all() or np.isnan(ref[~fine]).any(), name
    if not ref.size:
        return
    off = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) - tol, -1)
    worst = np.unravel_index(np.argmax(off), off.shape)
    assert off[worst] <= 0, f"{name}{worst}: {got[worst]} for {ref[worst]}, tolerance {np.broadcast_to(tol, off.shape)[worst]}"


def check_attention(ref, out, t, d, n, back):
    u = half_step(t)
    eps = fp32_slack(ref, d, n)
    extra = u if t == torch.bfloat16 else 0.0
    check("o", out["o"], ref["o"], u * np.abs(ref["o"]) + (extra * (1 + u) + eps) * ref["o_abs"] + 1e-30)
    if "lse" in out:
        check("lse", out["lse"], ref["lse"], eps + 2.0 ** -23 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0)))
    if back:
        for g in ("dq", "dk", "dv"):
            tol = u * np.abs(ref[g]) + (extra * (1 + u) + 2 * eps) * ref[g + "_abs"] + 1e-30
            if g != "dv":
                tol = tol + (u * (1 + 4 * u) * ref[g + "_delta"] if t == torch.bfloat16 else 2 * u * ref[g + "_delta"])
            check(g, out[g], ref[g], tol)


# batch, heads, kv_heads, d, q_len, k_len, window, sinks, q_lens, k_lens
ATTENTION = [
    (1, 1, 1, 64, 1, 1, 1, 0, None, None),
    (1, 1, 1, 8, 1, 5, 3, 1, None, None),
    (2, 4, 2, 64, 130, 130, 37, 5, [130, 71], [130, 71]),
    (1, 2, 1, 128, 257, 257, 64, 0, None, None),
    (2, 2, 2, 40, 70, 70, 0, 0, None, None),               # no window: causal
    (1, 2, 2, 64, 200, 200, 1, 0, None, None),             # only itself
    (1, 2, 1, 64, 200, 200, 1, 3, None, None),
    (1, 3, 3, 8, 40, 200, 16, 3, None, None),              # a chunk over a longer cache
    (1, 2, 2, 96, 300, 100, 50, 2, None, None),            # rows before the first key are empty
    (1, 2, 1, 72, 40, 0, 9, 2, None, None),                # no keys at all
    (2, 2, 1, 128, 1, 0, 9, 2, None, None),
    (4, 4, 2, 64, 150, 150, 40, 4, [150, 0, 1, 129], [150, 0, 1, 129]),
    (3, 4, 4, 120, 90, 140, 33, 4, [90, 60, 5], [140, 20, 5]),   # more rows than keys in one sequence
    (1, 4, 2, 64, 700, 700, 100, 150, None, None),         # sinks over more than one key tile
    (1, 2, 2, 128, 900, 900, 64, 4, None, None),           # rows far behind the sinks: split sums
    (2, 2, 1, 80, 1000, 1000, 130, 1, [1000, 300], [1000, 300]),
    (1, 2, 1, 64, 500, 500, 100000, 7, None, None),        # window and sinks beyond the sequence
    (1, 2, 1, 64, 300, 300, 20, 100000, None, None),
    (2, 8, 2, 128, 1, 500, 128, 4, None, [500, 77]),       # next tokens
    (3, 32, 1, 64, 1, 300, 0, 0, None, [300, 1, 0]),       # 32 rows, one key head
    (2, 4, 1, 72, 5, 900, 300, 10, None, [900, 3]),        # few tokens; a cache shorter than them
    (1, 8, 8, 128, 1, 3000, 2048, 4, None, None),          # split keys
    (3, 8, 2, 64, 8, 400, 50, 2, [8, 3, 0], [400, 399, 7]),
    (2, 6, 2, 104, 33, 65, 31, 3, None, None),             # one row more than the few-row kernel takes
    # several tiles of 32 rows over split keys; many query heads to a key head
    (1, 2, 2, 64, 100, 1700, 0, 0, None, None),
    (2, 6, 2, 72, 45, 2100, 1600, 5, [45, 20], [2100, 900]),
    (3, 4, 2, 128, 40, 1601, 1580, 40, [0, 40, 33], [1601, 30, 1600]),
    (2, 5, 1, 40, 67, 1900, 1700, 0, [67, 9], [1900, 4]),
    (3, 72, 2, 64, 1, 200, 77, 3, None, [200, 0, 5]),
    (1, 40, 1, 128, 7, 90, 50, 2, [6], [90]),
    # more than 256 tiles of 128 rows (keys): a wave for every 32 of them, and
    # tiles that all of a workgroup's rows see whole
    (4, 24, 24, 64, 700, 700, 400, 5, None, None),
    (3, 32, 16, 128, 600, 600, 330, 4, [600, 513, 100], [600, 513, 100]),
    (5, 24, 24, 40, 500, 640, 0, 0, None, None),
    (6, 26, 26, 72, 270, 270, 50, 130, None, None),
    (2, 64, 64, 64, 515, 515, 129, 64, [515, 300], [515, 400]),
    (40, 8, 4, 128, 130, 130, 1000, 0, None, None),
    (9, 64, 64, 40, 140, 140, 60, 3, None, None),          # more than 1024: the same in fp32
]


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "x".join(str(x) for x in c[:8]))
def test_attention(lact, case, t):
    B, H, Hk, d, Lq, Lk, window, sinks, ql, kl = case
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(sum(case[:8]))
    layout = ("heads", "tokens", "wide")[(Lq + Lk + d) % 3]
    q, k, v, g = (randn(gen, s, dt, layout) for s in ((B, H, Lq, d), (B, Hk, Lk, d), (B, Hk, Lk, d), (B, H, Lq, d)))
    lens = lambda x: None if x is None else torch.tensor(x, dtype=torch.int64, device="cuda")
    kw = dict(window=window, sinks=sinks, scale=0.3, q_lens=lens(ql), k_lens=lens(kl))
    print("attention", t, layout, case, flush=True)
    out = {}
    out["o"], out["lse"] = lact.window_attention(q, k, v, return_lse=True, **kw)
    torch.cuda.synchronize()
    out.update(lact.window_attention_backward(q, k, v, out["o"], out["lse"], dO=g, **kw))
    torch.cuda.synchronize()
    ref = OB.window_attention(f64(q), f64(k), f64(v), window, sinks, float(np.float32(0.3)), ql, kl, f64(g))
    check_attention(ref, out, dt, d, Lk + Lq * H, True)


def test_default_scale_and_layouts_of_results(lact):
    gen = torch.Generator("cuda").manual_seed(1)
    q = randn(gen, (2, 4, 65, 64), torch.float32, "tokens")
    k = randn(gen, (2, 2, 65, 64), torch.float32)
    o = lact.window_attention(q, k, k, window=9)
    assert o.stride() == q.stride()
    ref = OB.window_attention(f64(q), f64(k), f64(k), 9, 0, 0.125)
    check_attention(ref, {"o": o}, torch.float32, 64, 65, False)


def test_slices_of_a_joint_projection_and_expanded_inputs(lact):
    """q, k, v as column slices of one [B, L, (H + 2 Hk) d] tensor; then keys
    and values that one head, or one sequence, provides for all by stride 0."""
    gen = torch.Generator("cuda").manual_seed(2)
    B, L, H, Hk, d = 2, 150, 4, 2, 64
    x = torch.randn(B, L, (H + 2 * Hk) * d, generator=gen, device="cuda").bfloat16()
    q, k, v = (s.unflatten(-1, (-1, d)).transpose(1, 2) for s in x.split([H * d, Hk * d, Hk * d], -1))
    g = randn(gen, (B, H, L, d), torch.bfloat16)
    kw = dict(window=40, sinks=3)
    for kk, vv in ((k, v), (k[:, :1].expand(B, Hk, L, d), v[:1].expand(B, Hk, L, d))):
        o, lse = lact.window_attention(q, kk, vv, return_lse=True, **kw)
        out = dict(lact.window_attention_backward(q, kk, vv, o, lse, dO=g, **kw), o=o, lse=lse)
        ref = OB.window_attention(f64(q), f64(kk), f64(vv), 40, 3, 0.125, None, None, f64(g))
        check_attention(ref, out, torch.bfloat16, d, L + L * H, True)
    # a broadcast gradient, as a sum's
    g1 = torch.ones((), device="cuda").bfloat16().expand(B, H, L, d)
    with pytest.raises(ValueError):
        lact.window_attention_backward(q, k, v, o, lse, dO=g1, **kw)   # d itself has to be contiguous


def test_rows_behind_the_lengths_are_left(lact):
    gen = torch.Generator("cuda").manual_seed(3)
    q, k, v = (randn(gen, (3, 4, 200, 64), torch.bfloat16) for _ in range(3))
    lens = torch.tensor([200, 0, 77], device="cuda")
    for L, n in ((200, lens), (6, torch.tensor([6, 0, 3], device="cuda"))):
        o = torch.full((3, 4, L, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((3, 4, L), 7.0, device="cuda")
        qq = q[:, :, :L]
        # what lies behind the lengths is never read
        kk, vv, qn = k.clone(), v.clone(), qq.clone()
        for b in range(3):
            kk[b, :, lens[b]:] = float("nan")
            vv[b, :, lens[b]:] = float("inf")
            qn[b, :, n[b]:] = float("nan")
        lact.window_attention(qn, kk, vv, o, window=30, sinks=2, q_lens=n, k_lens=lens, lse=lse)
        g = torch.ones_like(qn)
        for b in range(3):
            g[b, :, n[b]:] = float("nan")
        out = lact.window_attention_backward(qn, kk, vv, o, lse, dO=g, window=30, sinks=2, q_lens=n, k_lens=lens)
        want, wlse = lact.window_attention(qq, k, v, window=30, sinks=2, q_lens=n, k_lens=lens, return_lse=True)
        for b in range(3):
            m = int(n[b])
            assert torch.equal(o[b, :, :m], want[b, :, :m]) and torch.equal(lse[b, :, :m], wlse[b, :, :m])
            assert (o[b, :, m:] == 7).all() and (lse[b, :, m:] == 7).all()
            assert (out["dq"][b, :, m:] == 0).all()
            assert (out["dk"][b, :, int(lens[b]):] == 0).all() and (out["dv"][b, :, int(lens[b]):] == 0).all()
        assert all(torch.isfinite(x).all() for x in out.values())


def test_lengths_beyond_the_arrays_are_clamped(lact):
    gen = torch.Generator("cuda").manual_seed(4)
    q, k, v = (randn(gen, (2, 2, 50, 64), torch.bfloat16) for _ in range(3))
    big = torch.tensor([1 << 40, -5], device="cuda")
    fit = torch.tensor([50, 0], device="cuda")
    for L in (50, 4):
        a = lact.window_attention(q[:, :, :L], k, v, window=9, sinks=1, q_lens=big, k_lens=big)
        b = lact.window_attention(q[:, :, :L], k, v, window=9, sinks=1, q_lens=fit.clamp(max=L), k_lens=fit)
        assert torch.equal(a, b)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("L,d", [(150, 64), (300, 128), (3, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_non_finite_token_reaches_only_rows_that_see_it(lact, t, L, d, bad):
    L_ = lact
    """Masked places hold anything: with one key and value spoilt, the rows
    that do not see it are right (those that met it only as a masked place may
    be summed in another order), and those that do see the value are not
    finite where it is.  Once for a few heads and once for the same repeated
    (stride 0) over a batch that fills the chip: other kernels."""
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(5)
    Lk = 300
    q, k, v = randn(gen, (1, 2, L, d), dt), randn(gen, (1, 1, Lk, d), dt), randn(gen, (1, 1, Lk, d), dt)
    kw = dict(window=37, sinks=2)
    ref = OB.window_attention(f64(q), f64(k), f64(v), 37, 2, d ** -0.5)
    see = OB.visible(L, Lk, 37, 2)
    class lact:   # noqa: N801  the binding, both ways
        @staticmethod
        def window_attention(*x, **kw):
            one = L_.window_attention(*x, **kw)
            many = L_.window_attention(*[t.expand((90,) + t.shape[1:]) for t in x], **kw)
            unseen_are_right(many[-1:], s)
            assert torch.equal(many[:1].isfinite(), many[-1:].isfinite())
            return one

    def unseen_are_right(o, s):
        part = {n: ref[n][:, :, ~s] for n in ("o", "o_abs")}
        part["score_abs"] = ref["score_abs"]
        check_attention(part, {"o": o[:, :, torch.from_numpy(~s).cuda()]}, dt, d, Lk, False)

    for j in (0, 5, Lk - L, Lk - 40, Lk - 2, Lk - 1):
        v2, k2 = v.clone(), k.clone()
        v2[0, 0, j, 3] = bad
        s = see[:, j]
        o = lact.window_attention(q, k, v2, **kw)
        unseen_are_right(o, s)
        others = [c for c in range(d) if c != 3]
        assert torch.isfinite(o[..., others]).all()
        if s.any():
            on = o[:, :, torch.from_numpy(s).cuda(), 3]
            assert not torch.isfinite(on).any()
            if bad == float("inf"):
                assert (on == bad).all()
        k2[0, 0, j] = float("nan")
        v2[0, 0, j] = bad
        unseen_are_right(lact.window_attention(q, k2, v2, **kw), s)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_non_finite_token_among_split_keys(lact, t, d):
    """As above where several tiles of 32 rows share the work on long keys."""
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(8)
    L, Lk = 70, 2000
    q, k, v = randn(gen, (1, 2, L, d), dt), randn(gen, (1, 1, Lk, d), dt), randn(gen, (1, 1, Lk, d), dt)
    kw = dict(window=1600, sinks=2)
    ref = OB.window_attention(f64(q), f64(k), f64(v), 1600, 2, d ** -0.5)
    see = OB.visible(L, Lk, 1600, 2)
    for j in (0, 5, Lk - L - 1600, Lk - 1630, Lk - L, Lk - 33, Lk - 1):
        for bad in (float("nan"), float("inf")):
            v2, k2 = v.clone(), k.clone()
            v2[0, 0, j, 3] = bad
            s = see[:, j]
            o = lact.window_attention(q, k, v2, **kw)
            k2[0, 0, j] = float("nan")
            o2 = lact.window_attention(q, k2, v2, **kw)
            for x in (o, o2):
                part = {n: ref[n][:, :, ~s] for n in ("o", "o_abs")}
                part["score_abs"] = ref["score_abs"]
                check_attention(part, {"o": x[:, :, torch.from_numpy(~s).cuda()]}, dt, d, Lk, False)
            assert torch.isfinite(o[..., [c for c in range(d) if c != 3]]).all()
            assert not torch.isfinite(o[:, :, torch.from_numpy(s).cuda(), 3]).any()


def test_no_rows_and_no_keys(lact):
    """Gradients over nothing are zeros, and nothing is written elsewhere."""
    for lq, lk in ((0, 50), (50, 0), (0, 0)):
        q, k = torch.randn(2, 4, lq, 64, device="cuda"), torch.randn(2, 2, lk, 64, device="cuda")
        o, lse = lact.window_attention(q, k, k, window=9, sinks=1, return_lse=True)
        assert o.shape == q.shape and (o == 0).all() and (lse == -float("inf")).all()
        g = lact.window_attention_backward(q, k, k, o, lse, dO=torch.randn_like(q), window=9, sinks=1)
        assert all((x == 0).all() for x in g.values()) and g["dk"].shape == k.shape and g["dq"].shape == q.shape
    e = torch.empty(0, 4, 10, 64, device="cuda")
    o, lse = lact.window_attention(e, e, e, return_lse=True)
    assert o.shape == e.shape and lact.window_attention_backward(e, e, e, o, lse, dO=e)["dq"].shape == e.shape


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("batch", [1, 80])
def test_non_finite_gradients_stay_with_what_they_reach(lact, t, batch):
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(6)
    L, d, j = 500, 64, 150
    q, k, v, g = (randn(gen, (1, 1, L, d), dt) for _ in range(4))
    kw = dict(window=20, sinks=2)
    L_ = lact
    class lact:   # noqa: N801  the same repeated over a batch (stride 0); its last sequence is looked at
        window_attention = staticmethod(L_.window_attention)

        @staticmethod
        def window_attention_backward(*x, dO, **kw):
            r = lambda t: t.expand((batch,) + t.shape[1:])
            y = [r(t) for t in x]
            y[4] = y[4].contiguous()
            return {n: t[-1:] for n, t in L_.window_attention_backward(*y, dO=r(dO), **kw).items()}
    o, lse = lact.window_attention(q, k, v, return_lse=True, **kw)
    ref = OB.window_attention(f64(q), f64(k), f64(v), 20, 2, 0.125, dO=f64(g))
    see = OB.visible(L, L, 20, 2)

    def right(name, got, keep):
        part = {n: ref[n][:, :, keep] for n in ref if n.startswith(name)}
        u, eps = half_step(dt), fp32_slack(ref, d, 2 * L)
        tol = u * np.abs(part[name]) + ((u * (1 + u) if t == "bf16" else 0) + 2 * eps) * part[name + "_abs"]
        if name != "dv":
            tol = tol + u * (1 + 4 * u) * (1 if t == "bf16" else 2) * part[name + "_delta"]
        check(name, got[:, :, torch.from_numpy(keep).cuda()], part[name], tol)

    g2, q2, k2, v2 = g.clone(), q.clone(), k.clone(), v.clone()
    g2[0, 0, j] = float("nan")     # row j's gradient: reaches row j and the keys it sees
    out = lact.window_attention_backward(q, k, v, o, lse, dO=g2, **kw)
    keys, others = see[j], np.arange(L) != j
    for n in ("dk", "dv"):
        right(n, out[n], ~keys)
        assert torch.isnan(out[n][:, :, torch.from_numpy(keys).cuda()]).all()
    right("dq", out["dq"], others)
    unseen = ~see[:, j]
    for x in (k2, v2):             # a key, then a value, that only some later rows see
        x[0, 0, j] = float("inf")
        right("dq", lact.window_attention_backward(q, k2, v2, o, lse, dO=g, **kw)["dq"], unseen)
        x.copy_(k if x is k2 else v)
    q2[0, 0, j] = float("nan")
    out = lact.window_attention_backward(q2, k, v, o, lse, dO=g, **kw)
    right("dk", out["dk"], ~keys)


def test_large_scores(lact):
    """Scores in the thousands: the maximum is subtracted before any exp, and
    a score more than 2^8 above the others takes all of the sum."""
    gen = torch.Generator("cuda").manual_seed(7)
    for L in (150, 4):
        q, k, v = (30 * randn(gen, (1, 2, n, 64), torch.float32) for n in (L, 150, 150))
        o, lse = lact.window_attention(q, k, v, window=60, sinks=1, return_lse=True)
        ref = OB.window_attention(f64(q), f64(k), f64(v), 60, 1, 0.125)
        check_attention(ref, {"o": o, "lse": lse}, torch.float32, 64, 150, False)


def test_a_cache_beyond_32_bit_offsets(lact):
    """The last rows of a cache of 2^24 + 600 tokens (4.3 GB of keys)."""
    S = (1 << 24) + 600
    k = torch.empty(1, 1, S, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    gen = torch.Generator("cuda").manual_seed(8)
    for x in (k, v):
        x[:, :, :3] = torch.randn(1, 1, 3, 128, generator=gen, device="cuda")
        x[:, :, -700:] = torch.randn(1, 1, 700, 128, generator=gen, device="cuda")
    for L in (1, 100):
        q = randn(gen, (1, 4, L, 128), torch.bfloat16)
        o = lact.window_attention(q, k, v, window=500, sinks=3)
        pick = lambda x: torch.cat([x[:, :, :3], x[:, :, -700:]], 2)
        # the 3 sinks in front of 700 keys, of which a window sees the last 500
        ref = OB.window_attention(f64(q), f64(pick(k)), f64(pick(v)), 500, 3, 128 ** -0.5)
        check_attention(ref, {"o": o}, torch.bfloat16, 128, 703, False)


def _graph(call, outs, warm=1):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(warm):
            call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [x.clone() for x in outs()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        for x in outs():
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs(), want):
            assert torch.equal(x, y), rep
        _ = float((outs()[0].float() * 2).sum())   # eager work between replays


@pytest.mark.parametrize("L", [1, 500])
def test_graph_replays_of_the_operators(lact, L):
    """A norm, rotary positions, attention and all their gradients in one
    captured graph, replayed with eager work between; every replay equals the
    eager call bit for bit (no atomics, nothing kept between calls)."""
    gen = torch.Generator("cuda").manual_seed(9)
    H, Hk, d, Lk = 4, 2, 64, 2000
    x = randn(gen, (1, L, H, d), torch.bfloat16).view(L, H * d)
    r, dy = torch.randn_like(x), torch.randn_like(x)
    w = torch.randn(H * d, device="cuda")
    k, v = randn(gen, (1, Hk, Lk, d), torch.bfloat16), randn(gen, (1, Hk, Lk, d), torch.bfloat16)
    fr, _ = lact.rotary_frequencies(32)
    s = {}

    def call():
        y, h = lact.add_rmsnorm(x, w, r)
        q = y.view(1, L, H, d).transpose(1, 2)
        qr, kr = lact.rotary(q, k[:, :, :L].contiguous() if False else None, freqs=fr, start=Lk - L), k
        o, lse = lact.window_attention(qr, kr, v, window=300, sinks=4, return_lse=True)
        g = lact.window_attention_backward(qr, kr, v, o, lse, dO=o, window=300, sinks=4)
        dq = lact.rotary_backward(g["dq"], freqs=fr, start=Lk - L)
        dx, dw = lact.add_rmsnorm_backward(h, w, dy=dq.transpose(1, 2).reshape(L, H * d), dh=dy)
        y8, sc, _ = lact.add_rmsnorm_quantised(x, w, r)
        for n, t in dict(o=o, lse=lse, dk=g["dk"], dv=g["dv"], dx=dx, dw=dw, sc=sc, y8=y8.view(torch.uint8)).items():
            s.setdefault(n, torch.empty_like(t)).copy_(t)

    _graph(call, lambda: list(s.values()))


def test_calls_on_streams(lact):
    """The stream argument: the call, its results and its workspace belong to
    that stream; two streams at once give what each alone gives."""
    gen = torch.Generator("cuda").manual_seed(10)
    sets = [[randn(gen, (2, 4, 600, 64), torch.bfloat16) for _ in range(4)] for _ in range(2)]
    kw = dict(window=100, sinks=4)
    want = []
    for q, k, v, g in sets:
        o, lse = lact.window_attention(q, k, v, return_lse=True, **kw)
        want.append((o, lse, lact.window_attention_backward(q, k, v, o, lse, dO=g, **kw)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for st, (q, k, v, g) in zip(streams, sets):
            o, lse = lact.window_attention(q, k, v, return_lse=True, stream=st, **kw)
            one = lact.window_attention(q[:, :, :1], k, v, stream=st, **kw)
            got.append((o, lse, lact.window_attention_backward(q, k, v, o, lse, dO=g, stream=st, **kw)))
            del one
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            assert all(torch.equal(a[2][n], b[2][n]) for n in a[2])


def test_binding_refusals_on_the_device(lact):
    q = torch.zeros(1, 2, 8, 64, device="cuda")
    with pytest.raises(ValueError):
        lact.window_attention(q, q[:, :, :, :32], q)
    with pytest.raises(ValueError):
        lact.window_attention(q, q, q[:, :, :4])
    with pytest.raises(ValueError):
        lact.window_attention(q, q, q.bfloat16())
    with pytest.raises(ValueError):
        lact.window_attention(q, q, q, q_lens=torch.ones(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        lact.window_attention(q, q, q, k_lens=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        lact.window_attention(q, q.cpu(), q)
    with pytest.raises(ValueError):
        lact.window_attention(q, q, q, workspace=torch.empty(8, dtype=torch.float32, device="cuda"))
    with pytest.raises(lact.LactError):
        lact.window_attention(q, q, q, o=torch.zeros(1, 1, 8, 64, device="cuda").expand(1, 2, 8, 64))
    with pytest.raises(lact.LactError):
        lact.window_attention(q[..., 1:57], q[..., :56], q[..., :56])   # rows start off 16 bytes
    with pytest.raises(ValueError):
        lact.rotary(q, freqs=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        lact.rotary(q, freqs=torch.ones(4, dtype=torch.float64, device="cuda"),
                    positions=torch.ones(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        lact.add_rmsnorm(torch.zeros(4, 8, device="cuda").t(), torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        lact.add_rmsnorm(torch.zeros(4, 8, device="cuda"), torch.ones(8, device="cuda").bfloat16())


# ------------------------------------------------------------------ rotary positions
# batch, heads, kv_heads, tokens, d, pairs
ROTARY = [(1, 1, 0, 1, 2, 1), (2, 4, 2, 37, 64, 32), (1, 3, 1, 130, 128, 64), (3, 2, 2, 5, 80, 16), (2, 5, 1, 9, 90, 21),
          (1, 2, 1, 17, 33, 7), (1, 4, 4, 300, 96, 0), (1, 1, 1, 3, 4096, 2048), (40, 8, 2, 1, 128, 64)]


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "x".join(map(str, c)))
def test_rotary(lact, case, interleaved, t):
    B, H, Hk, L, d, n = case
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(11)
    layout = ("heads", "tokens", "wide")[(L + d) % 3]
    q = randn(gen, (B, H, L, d), dt, layout)
    k = randn(gen, (B, Hk, L, d), dt, layout) if Hk else None
    scaled = dict(scaling="yarn", factor=4.0, context=4096) if d % 3 else {}
    fr, m = lact.rotary_frequencies(n, 10000.0, **scaled)
    pos = torch.randint(0, 1 << 20, (B, L), generator=gen, device="cuda")
    pos[0, 0] = (1 << 31) + 12345
    print("rotary", t, layout, case, interleaved, flush=True)
    for inverse in (False, True):
        call = lact.rotary_backward if inverse else lact.rotary
        for p in (pos, None):
            got = call(q, k, freqs=fr, positions=p, start=777, interleaved=interleaved, mscale=m)
            got = got if Hk else (got,)
            at = pos.cpu().numpy() if p is not None else np.broadcast_to(777 + np.arange(L), (B, L))
            for x, y in zip((q, k), got):
                ref = OB.rotary(f64(x), at, fr.cpu().numpy(), interleaved, float(np.float32(m)), inverse)
                u = half_step(dt)
                # a feature is x cos - y sin: its rounding; cos and sin, off by
                # the turn's rounding to fp32 (pi 2^-24) and the function's
                # (2^-22; for bf16 tensors the hardware's, 2^-16), and two products
                mag = np.abs(f64(x))
                pair = mag.copy()
                i, j = ((np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved
                        else (np.arange(n), np.arange(n, 2 * n)))
                pair[..., i] = pair[..., j] = m * (mag[..., i] + mag[..., j])
                pair[..., 2 * n:] = 0
                c = 2.0 ** -16 if t == "bf16" else 2.0 ** -21
                check("rotary", y, ref, u * np.abs(ref) + c * pair)


def test_rotary_in_place_and_round_trip(lact):
    gen = torch.Generator("cuda").manual_seed(12)
    q, k = randn(gen, (2, 4, 50, 64), torch.float32, "tokens"), randn(gen, (2, 2, 50, 64), torch.float32)
    fr, _ = lact.rotary_frequencies(24)
    qo, ko = lact.rotary(q, k, freqs=fr)
    q2, k2 = q.clone(), k.clone()
    assert qo.stride() == q.stride()
    a, b = lact.rotary(q2, k2, freqs=fr, q_out=q2, k_out=k2)
    assert a is q2 and b is k2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    lact.rotary_backward(q2, k2, freqs=fr, q_out=q2, k_out=k2)
    assert float((q2 - q).abs().max()) < 8 * 2.0 ** -21 * float(q.abs().max())
    # into a cache's slots
    cache = torch.zeros(2, 2, 200, 64, device="cuda")
    lact.rotary(q, k, freqs=fr, k_out=cache[:, :, 100:150])
    assert torch.equal(cache[:, :, 100:150], ko) and (cache[:, :, :100] == 0).all() and (cache[:, :, 150:] == 0).all()


def test_rotary_of_expanded_input_and_empty(lact):
    fr, _ = lact.rotary_frequencies(8)
    x = torch.randn(1, 1, 5, 16, device="cuda").expand(2, 3, 5, 16)
    y = lact.rotary(x, freqs=fr)
    assert y.is_contiguous() and all(torch.equal(y[b, h], y[0, 0]) for b in range(2) for h in range(3))
    assert lact.rotary(x[:, :, :0], freqs=fr).shape == (2, 3, 0, 16)
    assert lact.rotary(x[:0], x[:0], freqs=fr)[1].shape == (0, 3, 5, 16)


# ------------------------------------------------------------------ add and norm
NORM = [(1, 1), (3, 7), (5, 64), (2, 129), (1100, 200), (2000, 520), (1, 2048), (1500, 2048), (70, 2560), (9, 4099), (3, 8192),
        (2, 12288), (2, 32768), (1, 30001), (4200, 72)]


def _norm_inputs(rows, cols, dt, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device="cuda").to(dt)
    r = (3 * torch.randn(rows, cols, generator=gen, device="cuda")).to(dt)
    w = 1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")
    return gen, x, r, w


def _rms_tol(cols):
    # a sum of squares of one sign and a square root: cols / 2 half steps at the worst order, and a few
    return 2.0 ** -24 * (cols + 16)


def e4m3_error(y):
    """Half a step of an e4m3 number: 2^-4 of the value, 2^-10 below the smallest normal (2^-6)."""
    return np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", NORM)
def test_norm(lact, rows, cols, t):
    dt = DT[t]
    gen, x, r, w = _norm_inputs(rows, cols, dt, 13)
    u, e = half_step(dt), _rms_tol(cols)
    print("norm", t, rows, cols, flush=True)
    for res in (r, None):
        y, h = lact.add_rmsnorm(x, w, res, eps=1e-5)
        ry, rh = OB.add_rmsnorm(f64(x), f64(w), None if res is None else f64(res), float(np.float32(1e-5)))
        # the fp32 sum x + residual rounds where the exponents differ
        check("h", h, rh, u * np.abs(rh) + 2.0 ** -24 * np.abs(rh))
        check("y", y, ry, (u + e) * np.abs(ry) + 2.0 ** -24 * np.abs(ry))
        assert (h is x) == (res is None)
        yy = torch.empty_like(x)
        y8, sc, h8 = lact.add_rmsnorm_quantised(x, w, res, eps=1e-5, y=yy)
        assert torch.equal(yy, y) and torch.equal(h8, h)
        rq, rs = OB.quantise(ry)
        check("scales", sc, rs, (e + 2.0 ** -22) * rs)
        check("y8", y8, rq, e4m3_error(rq) * (1 + e) + (2 * e + 2.0 ** -21) * np.abs(rq))
    hh = f64(h)
    dy, dh = (torch.randn(rows, cols, generator=gen, device="cuda").to(dt) for _ in range(2))
    for other in (dh, None):
        dx, dw = lact.add_rmsnorm_backward(h, w, dy=dy, dh=other, eps=1e-5)
        rx, rw = OB.add_rmsnorm_backward(hh, f64(w), f64(dy), None if other is None else f64(other), float(np.float32(1e-5)))
        f = 1 / np.sqrt((hh ** 2).mean(-1, keepdims=True) + 1e-5)
        g = np.abs(f64(dy) * f64(w))
        mag = f * (g + np.abs(hh) * f * f * (g * np.abs(hh)).mean(-1, keepdims=True))
        check("dx", dx, rx, u * np.abs(rx) + (3 * e + 2.0 ** -21) * mag + 2.0 ** -23 * np.abs(rx))
        wmag = (np.abs(f64(dy)) * np.abs(hh) * f).sum(0)
        check("dw", dw, rw, 2.0 ** -24 * (rows + cols + 40) * wmag)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_norm_strides_and_in_place(lact, t):
    dt = DT[t]
    gen, x, r, w = _norm_inputs(50, 200, dt, 14)
    y, h = lact.add_rmsnorm(x, w, r)
    # rows inside wider ones, aligned to 16 bytes and not; a broadcast row
    for lo, wide in ((8, 256), (3, 231)):
        big = torch.zeros(3, 50, wide, dtype=dt, device="cuda")
        xs, rs, ys = (big[i, :, lo:lo + 200] for i in range(3))
        xs.copy_(x)
        rs.copy_(r)
        y8 = torch.zeros(50, wide, device="cuda").to(torch.float8_e4m3fn)
        yy, hh = lact.add_rmsnorm(xs, w, rs, y=ys)
        assert torch.equal(yy, y) and torch.equal(hh, h)
        assert (big[2, :, :lo] == 0).all() and (big[2, :, lo + 200:] == 0).all()
        a = lact.add_rmsnorm_quantised(xs, w, rs, y8=y8[:, lo:lo + 200])
        b = lact.add_rmsnorm_quantised(x, w, r)
        assert torch.equal(a[0].float(), b[0].float()) and torch.equal(a[1], b[1])
        assert (y8.float()[:, :lo] == 0).all() and (y8.float()[:, lo + 200:] == 0).all()
    one = lact.add_rmsnorm(x, w, r[:1].expand(50, 200))
    two = lact.add_rmsnorm(x, w, r[:1].expand(50, 200).contiguous())
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    # in place: the residual stream, and both
    x2, r2 = x.clone(), r.clone()
    lact.add_rmsnorm(x2, w, r2, y=x2, h=r2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    g = torch.randn(50, 200, generator=gen, device="cuda").to(dt)
    d1, w1 = lact.add_rmsnorm_backward(h, w, dy=g, dh=x)
    for name in ("dy", "dh"):
        a = {"dy": g.clone(), "dh": x.clone()}
        d2, w2 = lact.add_rmsnorm_backward(h, w, **a, dx=a[name])
        assert torch.equal(d1, d2) and torch.equal(w1, w2)
    x3 = x.view(5, 10, 200)
    y3, h3 = lact.add_rmsnorm(x3, w, r.view(5, 10, 200))
    assert torch.equal(y3.view(50, 200), y) and torch.equal(h3.view(50, 200), h)


def test_norm_zero_rows_and_empty(lact):
    w = torch.ones(300, device="cuda")
    z = torch.zeros(4, 300, device="cuda").bfloat16()
    y8, sc, h = lact.add_rmsnorm_quantised(z, w, z)
    assert (y8.float() == 0).all() and torch.isfinite(sc).all() and (sc > 0).all() and (h == 0).all()
    y, _ = lact.add_rmsnorm(z, w)
    assert (y == 0).all()
    e = z[:0]
    assert lact.add_rmsnorm(e, w, e)[0].shape == (0, 300)
    dx, dw = lact.add_rmsnorm_backward(e, w, dy=e)
    assert dx.shape == (0, 300) and (dw == 0).all()   # the sum over no rows


# ------------------------------------------------------------------ together
def test_block_forward_and_backward(lact):
    """A block as it is used: the residual's norm, one joint projection, rotary
    positions, window attention beside the fast-weight layer on the same q, k,
    v, and the gradients of all of it back to the block's inputs, in fp32
    against the oracles of each in fp64."""
    import oracle as O
    from oracle import lact_backward as OBW
    B, H, L, d, C = 1, 2, 200, 64, 96
    n, gen = B * H, torch.Generator("cuda").manual_seed(15)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, r, w, P = rn(B, L, C), rn(B, L, C), 1 + 0.1 * rn(C), rn(C, 3 * H * d) / C ** 0.5
    lr, W = torch.rand(n, L, 3, generator=gen, device="cuda") * 0.01, [rn(n, d, d) / d ** 0.5 for _ in range(3)]
    fr, _ = lact.rotary_frequencies(d // 2)
    y, h = lact.add_rmsnorm(x, w, r)
    q, k, v = ((y.view(L, C) @ P).view(B, L, 3, H, d).unbind(2))
    q, k, v = (t.transpose(1, 2) for t in (q, k, v))
    qr, kr = lact.rotary(q, k, freqs=fr)
    kw = dict(window=64, sinks=4)
    o, lse = lact.window_attention(qr, kr, v, return_lse=True, **kw)
    flat = lambda t: t.contiguous().view(n, L, d)
    fast = lact.layer_forward(flat(qr), flat(kr), flat(v), lr, None, *[t.clone() for t in W], chunk=50)
    out = o + fast.view(B, H, L, d)
    g = rn(B, H, L, d)
    ga = lact.window_attention_backward(qr, kr, v, o, lse, dO=g, **kw)
    gf = lact.layer_backward(flat(qr), flat(kr), flat(v), lr, None, *W, dO=flat(g), chunk=50)
    dqr, dkr, dv = (ga[t] + gf[t].view(B, H, L, d) for t in ("dq", "dk", "dv"))
    dq, dk = lact.rotary_backward(dqr, dkr, freqs=fr)
    dqkv = torch.stack([t.transpose(1, 2) for t in (dq, dk, dv)], 2).reshape(L, 3 * H * d)
    dx, dw = lact.add_rmsnorm_backward(h, w, dy=(dqkv @ P.t().contiguous()).view(B, L, C))
    # the oracle's
    ry, rh = OB.add_rmsnorm(f64(x), f64(w), f64(r))
    z = (ry[0] @ f64(P)).reshape(B, L, 3, H, d).transpose(2, 0, 3, 1, 4)
    pos = np.arange(L)[None]
    fn = fr.cpu().numpy()
    zq, zk, zv = OB.rotary(z[0], pos, fn), OB.rotary(z[1], pos, fn), z[2]
    ref = OB.window_attention(zq, zk, zv, 64, 4, d ** -0.5, dO=f64(g))
    ref_out = ref["o"].copy()
    bounds, flags = list(range(0, L, 50)) + [L], [3] * 4
    gl = OBW.layer_backward(zq[0], zk[0], zv[0], f64(lr), None, *[f64(t) for t in W], bounds, flags, 0, 0, f64(g)[0])
    for i in range(n):
        ref_out[0, i] += O.forward_instance(zq[0, i], zk[0, i], zv[0, i], f64(lr)[i], None, *[f64(t)[i] for t in W],
                                            bounds, flags, 0, 0)["o"]
    dz = np.stack([OB.rotary(ref["dq"] + gl["dq"][None], pos, fn, inverse=True),
                   OB.rotary(ref["dk"] + gl["dk"][None], pos, fn, inverse=True), ref["dv"] + gl["dv"][None]])
    rdy = dz.transpose(1, 3, 0, 2, 4).reshape(L, 3 * H * d) @ f64(P).T
    rdx, rdw = OB.add_rmsnorm_backward(rh, f64(w), rdy.reshape(B, L, C))
    # the layer's own gate for fp32 is 1e-4 of the largest value; the rest of the chain adds fp32 roundings
    for name, a, b in (("out", out, ref_out), ("dx", dx, rdx), ("dw", dw, rdw)):
        assert np.abs(f64(a) - b).max() <= 2e-4 * np.abs(b).max(), name


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_decoding_over_a_cache_equals_the_whole_sequence(lact, t):
    """Tokens one at a time and four at a time, written into a cache by rotary
    and read by attention: each row as in one call over the sequence (other
    tile order, so equal within the rounding, not bit for bit)."""
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(16)
    H, Hk, L, d = 4, 2, 150, 64
    q, k, v = (randn(gen, (1, h, L, d), dt) for h in (H, Hk, Hk))
    fr, _ = lact.rotary_frequencies(d // 2)
    kw = dict(window=50, sinks=3)
    qr, kr = lact.rotary(q, k, freqs=fr)
    ref = OB.window_attention(f64(qr), f64(kr), f64(v), 50, 3, 0.125)
    cache = torch.full((2, 1, Hk, L + 20, d), float("nan"), device="cuda").to(dt)
    rows = []
    for step in (1, 4):
        at, lens = 0, torch.zeros(1, dtype=torch.int64, device="cuda")
        rows = []
        while at < L:
            m = min(step, L - at)
            qs = lact.rotary(q[:, :, at:at + m], k[:, :, at:at + m], freqs=fr, start=at,
                             k_out=cache[0][:, :, at:at + m])[0]
            cache[1][:, :, at:at + m] = v[:, :, at:at + m]
            at += m
            lens.fill_(at)
            rows.append(lact.window_attention(qs, cache[0], cache[1], k_lens=lens, **kw))
        check_attention(ref, {"o": torch.cat(rows, 2)}, dt, d, L, False)
