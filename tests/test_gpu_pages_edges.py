"""Packed and paged attention where one call leaves the usual: rows that a bound
leaves out, in numbers; what lies around results and workspaces; tokens that are
not finite inside a packed batch.  Tolerances as in test_gpu_block."""
import time

import numpy as np
import pytest

from oracle import lact_block as OB
from oracle import lact_pages as OP
from test_gpu_block import DT, check_attention, f64
from test_gpu_pages import _cache, _paged_ref, rows, sums, whole

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def lact():
    from test_layers_amd import lact as L
    return L


# ------------------------------------------------------------------ rows behind `longest`
@pytest.mark.parametrize("B", [1, 5, 64, 65, 300, 20000])
def test_rows_that_the_bound_leaves_out_are_cleared(lact, B):
    """Few and many sequences, of which some are longer than `longest`: the rows behind it are zero,
    the others what they are without those rows."""
    rng = np.random.default_rng(B)
    gen = torch.Generator("cuda").manual_seed(B)
    longest, H, Hk, d = 3, 4, 2, 40
    lens = rng.integers(0, longest + 1, B)
    over = rng.choice(B, size=max(1, B // 50), replace=False)
    lens[over] = rng.integers(longest + 1, 90, len(over))
    lens[over[0]] = 2000
    off = np.array(sums(lens, 2))
    T = int(off[-1]) + 1
    kept = np.concatenate([np.arange(a, min(z, a + longest)) for a, z in zip(off[:-1], off[1:])]).astype(np.int64)
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    live[torch.from_numpy(kept).cuda()] = True
    q, g = (rows(gen, H, T, d, torch.bfloat16, "tokens") for _ in range(2))
    k, v = (rows(gen, Hk, T, d, torch.bfloat16, "heads") for _ in range(2))
    kw = dict(offsets=whole(off.tolist()), longest=longest)
    o, lse = lact.packed_attention(q, k, v, return_lse=True, **kw)
    grads = lact.packed_attention_backward(q, k, v, o, lse, dO=g, **kw)
    # the same without the rows that are left out
    at = torch.from_numpy(kept).cuda()
    short = dict(offsets=whole(sums(np.minimum(lens, longest))), longest=longest)
    qs, ks, vs, gs = (x[:, at] for x in (q, k, v, g))
    os, lses = lact.packed_attention(qs, ks, vs, return_lse=True, **short)
    want = dict(lact.packed_attention_backward(qs, ks, vs, os, lses, dO=gs, **short), o=os, lse=lses)
    for name, x in dict(grads, o=o, lse=lse).items():
        assert (x[:, ~live] == 0).all() and torch.equal(x[:, live], want[name]), name
    kp, vp, table = _cache(gen, [9] * 8, Hk, 16, d, torch.bfloat16, "heads")
    tab = whole(np.tile(table, (-(-B // 8), 1))[:B], torch.int32)
    p, plse = lact.paged_attention(q, kp, vp, table=tab, k_lens=whole([9] * B), return_lse=True, **kw)
    assert (p[:, ~live] == 0).all() and (plse[:, ~live] == 0).all() and (p[:, live] != 0).any()


def test_a_long_text_behind_the_bound_is_cleared_by_all(lact):
    """A bound far too small takes a fraction of a call's time more, not a thousand times (80 and 110 ms by one lane)."""
    T, H, longest = 8192, 32, 1024
    q = torch.randn(T, H, 128, device="cuda").bfloat16().transpose(0, 1)
    k = torch.randn(T, 8, 128, device="cuda").bfloat16().transpose(0, 1)
    kw = dict(offsets=whole([0, T]), longest=longest)
    o, lse = lact.packed_attention(q, k, k, return_lse=True, **kw)
    assert (o[:, longest:] == 0).all() and (lse[:, longest:] == 0).all()
    for call in (lambda: lact.packed_attention(q, k, k, **kw), lambda: lact.packed_attention_backward(q, k, k, o, lse, dO=q, **kw)):
        call()
        torch.cuda.synchronize()
        start = time.perf_counter()
        out = call()
        torch.cuda.synchronize()
        took = time.perf_counter() - start
        assert took < 0.02, f"{took * 1e3} ms"
    assert all((x[:, longest:] == 0).all() for x in out.values())


# ------------------------------------------------------------------ what is not finite, inside a packed batch
# heads, kv_heads, d, window, sinks, lengths, the spoilt sequence
SPOILT = [
    (4, 2, 64, 37, 5, [130, 200, 31], 1),
    (2, 2, 128, 64, 4, [40, 900, 100], 1),                # split sums of the sinks
    (2, 1, 40, 0, 0, [90] * 70, 33),                      # more sequences than a wave tries at once
    (8, 1, 128, 0, 0, [130, 1100, 3, 300], 1),            # a tile's rows in parts
    (3, 1, 64, 0, 0, [20, 1300], 1),
    (12, 2, 96, 333, 17, [200, 0, 1200, 383], 2),         # parts, and split sums of the sinks beside them
    (4, 1, 64, 256, 200, [31, 1500, 90], 1),
]


def _reached(H, Hk, T, a, see, what, hk, h, at):
    """What a spoilt element reaches: rows [H, T], their gradients' keys [Hk, T], by the definition."""
    rows_, keys = np.zeros((H, T), bool), np.zeros((Hk, T), bool)
    n, G = see.shape[0], H // Hk
    if what in ("k", "v"):
        rows_[hk * G : (hk + 1) * G, a : a + n] = see[:, at]
    else:
        rows_[h, a + at] = True
        hk = h // G
    keys[hk, a : a + n] = see[rows_[h, a : a + n]].any(0)
    return rows_, keys


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("case", SPOILT, ids=lambda c: "x".join(str(x) for x in c[:5]) + f"_{len(c[5])}")
@pytest.mark.parametrize("what,bad", [("q", float("nan")), ("k", float("nan")), ("v", float("nan")), ("v", float("inf")),
                                      ("dO", float("nan")), ("dO", float("-inf"))])
def test_what_is_not_finite_reaches_only_what_sees_it(lact, case, t, what, bad):
    """One spoilt element of a sequence between others: what the definition leads it to is not finite, all else is right."""
    H, Hk, d, window, sinks, lens, nth = case
    dt, T, off = DT[t], sum(lens), sums(lens)
    gen = torch.Generator("cuda").manual_seed(sum(case[:5]))
    x = {"q": rows(gen, H, T, d, dt, "tokens"), "k": rows(gen, Hk, T, d, dt, "heads"), "v": rows(gen, Hk, T, d, dt, "tokens"),
         "dO": rows(gen, H, T, d, dt, "wide")}
    kw = dict(window=window, sinks=sinks, offsets=whole(off), longest=max(lens))
    scale = float(np.float32(d ** -0.5))
    ref = OP.packed_attention(f64(x["q"]), f64(x["k"]), f64(x["v"]), off, window, sinks, scale, f64(x["dO"]))
    n, a = lens[nth], off[nth]
    see = OB.visible(n, n, window, sinks)
    hk, h, c = Hk - 1, H - 1, 5
    for at in (0, n // 2, n - 2):
        y = dict(x)
        y[what] = x[what].clone()
        y[what][hk if what in ("k", "v") else h, a + at, c] = bad
        o, lse = lact.packed_attention(y["q"], y["k"], y["v"], return_lse=True, **kw)
        out = dict(lact.packed_attention_backward(y["q"], y["k"], y["v"], o, lse, dO=y["dO"], **kw), o=o, lse=lse)
        torch.cuda.synchronize()
        rows_, keys = _reached(H, Hk, T, a, see, what, hk, h, at)
        none, col = np.zeros((1, 1, 1), bool), (np.arange(d) == c)[None, None]
        every, r, k = ~np.zeros((1, 1, 1), bool), rows_[..., None], keys[..., None]
        hit = {"o": {"q": r & every, "k": r & every, "v": r & col, "dO": none}[what],
               "lse": rows_ if what in ("q", "k") else none[0],
               "dq": r & every, "dk": k & every,
               "dv": {"q": k & every, "k": k & every, "v": none, "dO": k & col}[what]}
        for name, got in out.items():
            spoilt = torch.from_numpy(np.broadcast_to(hit[name], got.shape).copy()).cuda()
            assert (got.isfinite() == ~spoilt).all(), (name, at, int((got.isfinite() == spoilt).sum()))
            out[name] = torch.where(spoilt, torch.from_numpy(ref[name]).float().cuda(), got.float())
        check_attention(ref, out, dt, d, max(lens) * (1 + H // Hk), True)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(1, 900), (5, 900), (200, 900), (200, 3100)])
@pytest.mark.parametrize("what", ["q", "k"])
def test_a_row_or_key_in_pages_that_is_not_finite(lact, t, d, n, m, what):
    gen = torch.Generator("cuda").manual_seed(21)
    dt, page, window, sinks = DT[t], 24, 333, 3
    seqs = [(max(1, n // 2), m // 2), (n, m), (1, 40)]
    new, lens = [x for x, _ in seqs], [x for _, x in seqs]
    off = sums(new)
    q = rows(gen, 4, off[-1], d, dt, "tokens")
    kp, vp, table = _cache(gen, lens, 2, page, d, dt, "tokens")
    kw = dict(table=whole(table, torch.int32), offsets=whole(off), k_lens=whole(lens), longest=max(new), window=window,
              sinks=sinks)
    ref = _paged_ref(q, kp, vp, table, off, lens, window, sinks, float(np.float32(d ** -0.5)))
    see = OB.visible(n, m, window, sinks)
    for at in (0, n // 2, n - 1) if what == "q" else (1, m // 2, m - 100, m - 2):
        q2, k2 = q.clone(), kp.clone()
        rows_ = np.zeros((4, off[-1]), bool)
        if what == "q":
            q2[3, off[1] + at, 5] = float("nan")
            rows_[3, off[1] + at] = True
        else:
            k2[table[1, at // page], 1, at % page, 5] = float("nan")
            rows_[2:, off[1] : off[2]] = see[:, at]
        o, lse = lact.paged_attention(q2, k2, vp, return_lse=True, **kw)
        spoilt = torch.from_numpy(rows_).cuda()
        assert (lse.isfinite() == ~spoilt).all() and (o.isfinite() == ~spoilt[..., None]).all(), at
        put = lambda x, y, s: torch.where(s, torch.from_numpy(y).float().cuda(), x.float())
        check_attention(ref, {"o": put(o, ref["o"], spoilt[..., None]), "lse": put(lse, ref["lse"], spoilt)}, dt, d, m, False)


# ------------------------------------------------------------------ around results and workspaces
class Inside:
    """A tensor inside a larger one that is filled with a pattern around it."""

    def __init__(self, shape, dtype, fill, margin=4096):
        n = int(np.prod(shape))
        self.all = torch.full((n + 2 * margin,), fill, dtype=dtype, device="cuda")
        self.x, self.margin, self.fill = self.all[margin : margin + n].view(shape), margin, fill

    def kept(self):
        return bool((self.all[: self.margin] == self.fill).all()) and bool((self.all[-self.margin :] == self.fill).all())


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [20, 90, 300, 700])
def test_offsets_out_of_order_keep_to_results_and_workspaces(lact, B, t):
    """Offsets that jump about, also for more sequences than a workgroup sums itself: what
    lies around o, lse, the gradients and the workspaces stays."""
    dt, T, d, H, Hk = DT[t], 700, 64, 4, 2
    gen = torch.Generator("cuda").manual_seed(B)
    q, k = rows(gen, H, T, d, dt, "heads"), rows(gen, Hk, T, d, dt, "heads")
    kp, vp, table = _cache(gen, [70] * 90, Hk, 32, d, dt, "heads")
    tab = whole(np.tile(table, (-(-B // 90), 1))[:B], torch.int32)
    o, dq = (Inside((H, T, d), dt, 7.0) for _ in range(2))
    dk, dv = (Inside((Hk, T, d), dt, 7.0) for _ in range(2))
    lse = Inside((H, T), torch.float32, 7.0)
    G = lambda n: Inside((n,), torch.uint8, 77)
    for longest in (2, 300, T):
        jump = torch.randint(-10, T + 10, (B + 1,), generator=gen, device="cuda")
        near = torch.arange(B + 1, device="cuda") % 2 + 40   # the same row again and again
        for off in (jump, near):
            kw = dict(offsets=off, longest=longest, window=30, sinks=3)
            need = lact._packed_back_plan(q, k, k, off, longest, 30, 3, None, o.x, lse.x, q, (None,) * 3).need
            ws = G(-(-need // 256) * 256)
            lact.packed_attention(q, k, k, o.x, lse=lse.x, **kw)
            lact.packed_attention_backward(q, k, k, o.x, lse.x, dO=q, out=dict(dq=dq.x, dk=dk.x, dv=dv.x), workspace=ws.x, **kw)
            lens = whole([70] * B)
            need = lact._paged_plan(q, kp, vp, tab, off, lens, longest, None, 30, 3, None).need
            ws2 = G(-(-need // 256) * 256)
            lact.paged_attention(q, kp, vp, o.x, lse=lse.x, table=tab, k_lens=lens, workspace=ws2.x, **kw)
            torch.cuda.synchronize()
            assert all(x.kept() for x in (o, lse, dq, dk, dv, ws, ws2)), (longest, off is jump)
