"""The block's operators on the GPU where an input, a length or a caller is
unusual: values that are not finite or near the type's largest beside lengths,
parameters that a caller changes in place, views that grow from call to call.
Tolerances as in test_gpu_block."""
import numpy as np
import pytest

from oracle import lact_block as OB
from test_gpu_block import DT, _graph, check_attention, f64, half_step, randn

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def lact():
    from test_layers_amd import lact as L
    return L


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", [1, 400])
@pytest.mark.parametrize("n,sinks", [(237, 0), (237, 3), (20, 3)])
def test_gradients_behind_the_lengths_are_zero(lact, t, d, batch, n, sinks):
    """A NaN in a live row of dO or q, and a length that ends inside a group of
    32 keys: the keys behind it take part in the products as masked places,
    and their gradients are zeros all the same.  Once with two waves a tile,
    once (stride 0 over a batch) with one; in a sink tile too."""
    gen = torch.Generator("cuda").manual_seed(20)
    L, dt = 300, DT[t]
    one = [randn(gen, (1, 1, L, d), dt) for _ in range(4)]
    lens = torch.full((batch,), n, dtype=torch.int64, device="cuda")
    kw = dict(window=40, sinks=sinks, q_lens=lens, k_lens=lens)
    rep = lambda x: x.expand((batch,) + x.shape[1:])
    q, k, v, g = (rep(x) for x in one)
    o, lse = lact.window_attention(q, k, v, return_lse=True, **kw)
    see = OB.visible(n, n, 40, sinks)
    for row in (n - 1, n - 7):
        for spoilt in ("q", "dO"):
            q2, g2 = one[0].clone(), one[3].clone()
            (q2 if spoilt == "q" else g2)[0, 0, row, 5] = float("nan")
            out = lact.window_attention_backward(rep(q2), k, v, o, lse, dO=rep(g2), **kw)
            unseen = torch.from_numpy(~see[row]).cuda()
            for name in ("dk", "dv"):
                x = out[name]
                assert (x[:, :, n:] == 0).all(), (name, row, spoilt)
                assert torch.isfinite(x[:, :, :n][:, :, unseen]).all(), (name, row, spoilt)
                assert (x[0] == x[-1]).logical_or(x[0].isnan()).all()
            assert (out["dq"][:, :, n:] == 0).all()


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Lq,Lk", [(1, 150, 150), (200, 150, 150), (1, 3, 300), (1, 3, 4000), (300, 2, 300)])
@pytest.mark.parametrize("size", [2.0 ** 104, 2.0 ** 125, 2.0 ** 127])
def test_values_near_the_types_largest(lact, t, d, B, Lq, Lk, size):
    """An average of values is no larger than the largest of them, also where
    scores climb along the keys, so that sums are held relative to an earlier,
    smaller maximum (by up to 2^24), and several parts are joined."""
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(21)
    q, k, v = (randn(gen, (1, 1, n, d), dt) for n in (Lq, Lk, Lk))
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(Lk, device="cuda") / Lk * 1.7).to(dt)   # times 8: 2^19.6 in the exponential
    v = (torch.sign(v) * (1 + v.abs().clamp(max=3) / 4) * size).to(dt)   # up to 1.75 times the size
    rep = lambda x: x.expand((B,) + x.shape[1:])
    o = lact.window_attention(rep(q), rep(k), rep(v), scale=1.0)
    ref = OB.window_attention(f64(q), f64(k), f64(v), 0, 0, 1.0)
    check_attention(ref, {"o": o[-1:]}, dt, d, Lk, False)


def test_parameters_given_as_tensors_are_read_at_every_call(lact):
    """A position counter or a scale that the caller keeps in a tensor and
    changes in place: nothing of an earlier call's value is used."""
    q, w = torch.randn(1, 2, 40, 64, device="cuda"), torch.ones(64, device="cuda")
    fr, _ = lact.rotary_frequencies(32)
    o, lse = lact.window_attention(q, q, q, return_lse=True)
    flat = q.view(80, 64)
    calls = {
        "start": (3, 8, lambda x: lact.rotary(q, freqs=fr, start=x)),
        "start back": (3, 8, lambda x: lact.rotary_backward(q, freqs=fr, start=x)),
        "mscale": (0.5, 1.5, lambda x: lact.rotary(q, freqs=fr, mscale=x)),
        "scale": (0.1, 0.7, lambda x: lact.window_attention(q, q, q, scale=x)),
        "window": (2, 9, lambda x: lact.window_attention(q, q, q, window=x)),
        "sinks": (0, 9, lambda x: lact.window_attention(q, q, q, window=3, sinks=x)),
        "scale back": (0.1, 0.7, lambda x: lact.window_attention_backward(q, q, q, o, lse, dO=q, scale=x)["dk"]),
        "window back": (2, 9, lambda x: lact.window_attention_backward(q, q, q, o, lse, dO=q, window=x)["dk"]),
        "eps": (0.1, 0.9, lambda x: lact.add_rmsnorm(flat, w, eps=x)[0]),
        "eps 8": (0.1, 0.9, lambda x: lact.add_rmsnorm_quantised(flat, w, eps=x)[1]),
        "eps back": (0.1, 0.9, lambda x: lact.add_rmsnorm_backward(flat, w, dy=flat, eps=x)[0]),
    }
    for name, (first, then, call) in calls.items():
        # powers of two and whole numbers apart, a float32 tensor holds another value than the float
        x = torch.tensor(first)
        one = call(x)
        x.fill_(then)
        two = call(x)
        assert torch.equal(one, call(torch.tensor(first).item())), name
        assert torch.equal(two, call(torch.tensor(then).item())) and not torch.equal(one, two), name
    for kw in (dict(window=2.0), dict(sinks="4")):
        with pytest.raises(ValueError):
            lact.window_attention(q, q, q, **kw)
    with pytest.raises(ValueError):
        lact.rotary(q, freqs=fr, start=1.5)


def test_a_first_call_takes_no_memory_but_its_results(lact):
    """The next token over a view of a cache that grows from call to call: each
    shape is new to the binding, and none costs memory of the cache's size."""
    n = 1 << 20
    k = torch.zeros(1, 1, n, 128, dtype=torch.bfloat16, device="cuda")   # 256 MB
    q = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    fr, _ = lact.rotary_frequencies(64)
    for m in (n - 8, n):
        kk = k[:, :, :m]
        # results of [1, 2, 1, 128], and 256 splits' partial results of two rows
        for call, most in ((lambda: lact.window_attention(q, kk, kk, window=4096), 1 << 20),
                           (lambda: lact.rotary(kk, freqs=fr, q_out=kk), 0)):
            torch.cuda.synchronize()
            before = torch.cuda.memory_allocated()
            torch.cuda.reset_peak_memory_stats()
            call()
            assert torch.cuda.max_memory_allocated() - before <= most


def test_a_decoding_loop_plans_its_rotary_call_once(lact):
    """The start moves on at every step; the plan does not depend on it."""
    q, fr = torch.randn(1, 2, 1, 64, device="cuda"), lact.rotary_frequencies(32)[0]
    lact.rotary(q, freqs=fr)
    plans = dict(lact._PLANS)
    for start in (0, 1, 2, 700, 1 << 40):
        at = torch.full((1, 1), start, dtype=torch.int64, device="cuda")
        want = lact.rotary(q, freqs=fr, positions=at, start=3)   # positions given: the start is not looked at
        plans.update(lact._PLANS)
        assert torch.equal(lact.rotary(q, freqs=fr, start=start), want)
        assert lact._PLANS == plans


def test_a_norm_over_its_input_returns_no_h(lact):
    """y = x without a residual: x holds y afterwards, and no h is handed out
    that a backward pass would take for the norm's input."""
    x, w = torch.randn(5, 64, device="cuda"), 2 * torch.ones(64, device="cuda")
    want, _ = lact.add_rmsnorm(x, w)
    q8, sc, h = lact.add_rmsnorm_quantised(x, w)
    assert h is x
    for given in (None, torch.empty_like(x)):
        z = x.clone()
        y, h = lact.add_rmsnorm(z, w, y=z, h=given)
        assert y is z and torch.equal(z, want) and h is given
        z = x.clone()
        a, b, h = lact.add_rmsnorm_quantised(z, w, y=z, h=given)
        assert torch.equal(a.float(), q8.float()) and torch.equal(b, sc) and torch.equal(z, want) and h is given
        assert given is None or torch.equal(given, x)
    # with a residual h has a place of its own
    z = x.clone()
    y, h = lact.add_rmsnorm(z, w, z, y=z)
    assert torch.equal(h, x + x)
    e = x[:0]
    assert lact.add_rmsnorm(e, w)[1] is e


@pytest.mark.parametrize("window,sinks", [(0, 7), (20, 300), (20, 1 << 40), (300, 5), (1 << 40, 0)])
def test_limits_that_hide_nothing_are_no_limits(lact, window, sinks):
    """A window or sinks over all keys: the bits of plain causal attention, and of its gradients."""
    gen = torch.Generator("cuda").manual_seed(22)
    q, k, v, g = (randn(gen, (2, 4, 300, 64), torch.bfloat16) for _ in range(4))
    for rows in (300, 3):
        qq, gg = q[:, :, :rows], g[:, :, :rows]
        o, lse = lact.window_attention(qq, k, v, return_lse=True)
        out = lact.window_attention_backward(qq, k, v, o, lse, dO=gg)
        o2, lse2 = lact.window_attention(qq, k, v, return_lse=True, window=window, sinks=sinks)
        out2 = lact.window_attention_backward(qq, k, v, o2, lse2, dO=gg, window=window, sinks=sinks)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(out[n], out2[n]) for n in out)


# tiles of 128 rows and keys on both sides of every bound by which one wave or
# two take a tile, with lengths that leave some of them empty
# (batch, heads, kv_heads, d, tokens, window, lengths)
SHARED = [
    (1, 32, 32, 64, 500, 500, None), (1, 33, 33, 64, 500, 500, None), (1, 16, 16, 64, 1000, 300, None),
    (1, 81, 81, 64, 500, 250, None), (1, 96, 96, 64, 500, 100, None), (1, 97, 97, 64, 500, 100, None),
    (1, 32, 32, 72, 500, 100, None), (1, 33, 33, 72, 500, 100, None), (1, 57, 57, 128, 500, 100, None),
    (1, 80, 80, 72, 500, 100, None), (1, 81, 81, 72, 500, 100, None), (2, 40, 40, 128, 500, 251, None),
    (5, 32, 16, 64, 500, 100, [500, 1, 250, 0, 129]), (5, 32, 16, 96, 500, 100, [500, 1, 250, 0, 129]),
    (3, 40, 40, 64, 400, 50, [400, 100, 0]),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "x".join(str(x) for x in c[:6]))
def test_waves_that_share_tiles(lact, case):
    B, H, Hk, d, L, window, lens = case
    gen = torch.Generator("cuda").manual_seed(23)
    q, k, v, g = (randn(gen, s, torch.bfloat16) for s in ((B, H, L, d), (B, Hk, L, d), (B, Hk, L, d), (B, H, L, d)))
    n = None if lens is None else torch.tensor(lens, device="cuda")
    kw = dict(window=window, sinks=3, q_lens=n, k_lens=n)
    out = {}
    out["o"], out["lse"] = lact.window_attention(q, k, v, return_lse=True, **kw)
    out.update(lact.window_attention_backward(q, k, v, out["o"], out["lse"], dO=g, **kw))
    ref = OB.window_attention(f64(q), f64(k), f64(v), window, 3, float(np.float32(d ** -0.5)), lens, lens, f64(g))
    check_attention(ref, out, torch.bfloat16, d, 2 * L * H // Hk, True)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_sines_of_turns(lact, t):
    """A feature alone in its pair comes out as the sine and the cosine.  fp32:
    right to 8 half steps of its own size also next to a zero: 4 of the sine
    function (2 units in the last place), one each of mscale, the put-back
    rounding of the turn and the result, and a quarter of the turn in fp64
    (2^-50 of angle, for results from 2^-24 on).  bf16: one half step, and
    2^-22 of what the hardware's sine and the turn's rounding are off."""
    rng = np.random.default_rng(24)
    sign = lambda n: rng.choice([-1.0, 1.0], n)
    turns = np.concatenate([rng.random(4096) - 0.5, 2.0 ** -rng.uniform(1, 24, 2048) * sign(2048),
                            0.25 + 2.0 ** -rng.uniform(4, 24, 2048) * sign(2048),
                            0.5 + 2.0 ** -rng.uniform(4, 24, 2048) * sign(2048), 1e6 * rng.random(2048)])
    u, fr = half_step(DT[t]), torch.from_numpy(2 * np.pi * turns)
    for n in range(0, len(turns), 1024):
        f = fr[n:n + 1024].cuda()
        for interleaved in (False, True):
            for axis in (0, 1):
                q = torch.zeros(1, 1, 1, 2048, device="cuda", dtype=DT[t])
                (q[..., axis::2] if interleaved else q[..., axis * 1024:(axis + 1) * 1024]).fill_(1.0)
                y = f64(lact.rotary(q, freqs=f, start=1, interleaved=interleaved))[0, 0, 0]
                a, b = (y[::2], y[1::2]) if interleaved else (y[:1024], y[1024:])
                s, c = np.sin(f.cpu().numpy()), np.cos(f.cpu().numpy())
                for got, ref in ((a, -s if axis else c), (b, c if axis else s)):
                    tol = np.where(np.abs(ref) > 2.0 ** -24, 8 * u * np.abs(ref), 2.0 ** -24)
                    if t == "bf16":
                        tol = u * np.abs(ref) + 2.0 ** -22
                    off = np.abs(got - ref) - tol
                    i = np.argmax(off)
                    assert off[i] <= 0, (got[i], ref[i], f[i].item())


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("L,lens", [(1, [2000, 77]), (40, [40, 11]), (500, [500, 130])])
def test_graph_with_rotary_keys_and_lengths(lact, t, L, lens):
    """q and k turned in one call, k into a cache's slots, a padded batch and its
    gradients back through rotary, with a workspace of the caller's, captured:
    every replay is the eager call bit for bit, after the inputs changed too."""
    gen = torch.Generator("cuda").manual_seed(25)
    B, H, Hk, d, Lk, dt = 2, 4, 2, 64, 2000, DT[t]
    q, kn, vn, g = (randn(gen, (B, h, L, d), dt, "tokens") for h in (H, Hk, Hk, H))
    cache = [randn(gen, (B, Hk, Lk, d), dt) for _ in range(2)]
    kl = torch.tensor(lens if L == 1 else [Lk - L, Lk - L], device="cuda")
    ql = None if L == 1 else torch.tensor(lens, device="cuda")
    fr, _ = lact.rotary_frequencies(d // 2)
    pos = torch.arange(L, device="cuda").expand(B, L).contiguous() + 5
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    kw = dict(window=300, sinks=4, q_lens=ql, k_lens=kl)
    s = {}

    def call():
        slots = cache[0][:, :, Lk - L:]
        qr, kr = lact.rotary(q, kn, freqs=fr, positions=pos, k_out=slots)
        cache[1][:, :, Lk - L:].copy_(vn)
        o, lse = lact.window_attention(qr, *cache, return_lse=True, workspace=ws, **kw)
        out = lact.window_attention_backward(qr, *cache, o, lse, dO=g, workspace=ws, **kw)
        dq, dk = lact.rotary_backward(out["dq"], out["dk"][:, :, Lk - L:], freqs=fr, positions=pos)
        for n, x in dict(o=o, lse=lse, dq=dq, dk=dk, dv=out["dv"], cache=cache[0]).items():
            s.setdefault(n, torch.empty_like(x)).copy_(x)

    _graph(call, lambda: list(s.values()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for x in (q, kn, vn, g):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        kl.sub_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in s.items()}
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], s[n]) for n in s)
