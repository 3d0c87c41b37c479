"""Packed and paged attention, page slots and page writes on the GPU against the
fp64 oracle, at the lengths, pages, masks, layouts and callers where they can go
wrong.  Tolerances as in test_gpu_block; whole numbers and copies are equal.
"""
import numpy as np
import pytest

from oracle import lact_block as OB
from oracle import lact_pages as OP
from test_gpu_block import DT, _graph, check_attention, f64

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def lact():
    from test_layers_amd import lact as L
    return L


def whole(x, dtype=torch.int64):
    return torch.tensor(x, dtype=dtype, device="cuda")


def sums(lens, first=0):
    return [first + int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def rows(gen, heads, tokens, d, t, layout):
    """[heads, tokens, d] in one of three orders in memory."""
    if layout == "tokens":
        return torch.randn((tokens, heads, d), generator=gen, device="cuda").to(t).transpose(0, 1)
    if layout == "wide":
        return torch.randn((tokens, heads, d + 24), generator=gen, device="cuda").to(t).transpose(0, 1)[..., 8 : 8 + d]
    return torch.randn((heads, tokens, d), generator=gen, device="cuda").to(t)


# heads, kv_heads, d, window, sinks, lengths, token of the first, tokens behind the last
PACKED = [
    (1, 1, 64, 0, 0, [1], 0, 0),
    (2, 1, 8, 3, 1, [1, 1, 2, 0, 5], 0, 0),
    (4, 2, 64, 0, 0, [130, 1, 64, 128, 129], 0, 0),
    (4, 2, 64, 37, 5, [0, 0, 200, 31, 0], 3, 5),
    (2, 2, 128, 64, 0, [257, 100], 0, 0),
    (2, 1, 128, 0, 0, [300, 33, 32, 31], 7, 130),
    (3, 3, 40, 16, 3, [70] * 5, 0, 1),
    (6, 2, 72, 100, 150, [700, 90, 400], 0, 0),            # sinks over more than one key tile
    (2, 2, 128, 64, 4, [900, 40, 300], 0, 0),              # rows far behind the sinks: split sums
    (2, 1, 80, 130, 1, [1000, 0, 300, 129], 0, 9),
    (8, 1, 104, 1, 0, [90, 63], 0, 0),                     # only itself
    (4, 4, 64, 20, 100000, [150, 150], 0, 0),              # sinks beyond the sequences: no limit
    (16, 2, 64, 0, 0, [5] * 90, 0, 0),                     # more sequences than a wave tries at once
    (12, 12, 64, 200, 4, [3, 5, 0, 2] * 70 + [1000], 2, 0),
    (24, 24, 64, 400, 5, [700, 700, 650, 1, 700], 0, 0),   # whole tiles, one wave for 32 rows
    (32, 16, 128, 330, 4, [600, 513, 100, 700], 0, 40),
    (64, 64, 40, 0, 0, [515, 300, 131], 0, 0),
    (32, 8, 96, 0, 0, [260, 1290], 0, 0),
    # few key tiles with many rows, which are split: over heads, and beside sinks' own splits
    (8, 1, 128, 0, 0, [1500, 700, 3, 0, 130], 1, 2),
    (12, 2, 96, 333, 17, [1400, 383, 0, 200, 800], 0, 3),
    (4, 1, 64, 256, 200, [1900, 31, 900], 0, 0),
    (3, 1, 40, 0, 0, [2100], 0, 0),
]


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("case", PACKED, ids=lambda c: "x".join(str(x) for x in c[:5]) + f"_{len(c[5])}_{sum(c[5])}")
def test_packed(lact, case, t):
    H, Hk, d, window, sinks, lens, first, behind = case
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(sum(case[:5]))
    layout = ("heads", "tokens", "wide")[(sum(lens) + d) % 3]
    off = sums(lens, first)
    T = off[-1] + behind
    q, k, v, g = (rows(gen, h, T, d, dt, layout) for h in (H, Hk, Hk, H))
    print("packed", t, layout, case, flush=True)
    ref = OP.packed_attention(f64(q), f64(k), f64(v), off, window, sinks, float(np.float32(0.3)), f64(g))
    # what lies in no sequence is not used
    for x in (q, k, v, g):
        x[:, :first] = float("nan")
        x[:, off[-1]:] = float("inf")
    for longest in (None, max(lens)):
        kw = dict(window=window, sinks=sinks, scale=0.3, offsets=whole(off), longest=longest)
        out = {}
        out["o"], out["lse"] = lact.packed_attention(q, k, v, return_lse=True, **kw)
        torch.cuda.synchronize()
        assert out["o"].stride() == torch.empty_like(q).stride()
        out.update(lact.packed_attention_backward(q, k, v, out["o"], out["lse"], dO=g, **kw))
        torch.cuda.synchronize()
        check_attention(ref, out, dt, d, max(lens) * (1 + H // Hk), True)


def _cache(gen, lens, Hk, page, d, t, layout, spare=3):
    """Random pages for requests of these lengths: k_pages, v_pages, table (host).  Unused entries of
    the table lead nowhere, unused places hold NaN."""
    used = [-(-n // page) for n in lens]
    P, width = sum(used) + spare, max(used + [1]) + 2
    order = torch.randperm(P, generator=gen, device="cuda").tolist()
    table = np.full((len(lens), width), -1, np.int64)
    table[:, 1::2] = 2 ** 31 - 1
    shape = (P, page, Hk, d) if layout == "tokens" else (P, Hk, page, d)
    pools = []
    for _ in range(2):
        x = torch.randn(shape, generator=gen, device="cuda").to(t)
        pools.append(x.transpose(1, 2) if layout == "tokens" else x)
    live = torch.zeros(P, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        for i in range(used[b]):
            table[b, i] = order[at]
            live[order[at], : min(page, n - i * page)] = True
            at += 1
    for x in pools:
        x.masked_fill_(~live[:, None, :, None], float("nan"))
    return pools[0], pools[1], table


def _paged_ref(q, kp, vp, table, off, lens, window, sinks, scale):
    clean = lambda x: np.nan_to_num(f64(x))
    t = np.clip(table, 0, kp.shape[0] - 1)
    return OP.paged_attention(f64(q), clean(kp), clean(vp), t, off, lens, window, sinks, scale)


# heads, kv_heads, d, page, window, sinks, (new tokens, keys) of each sequence, token of the first, tokens behind
PAGED = [
    (1, 1, 64, 8, 0, 0, [(1, 1)], 0, 0),
    (2, 1, 8, 8, 3, 1, [(1, 5), (2, 2), (0, 7), (3, 1)], 1, 2),      # more rows than keys: rows that see nothing
    (4, 2, 64, 16, 0, 0, [(1, 500), (1, 33), (1, 0), (1, 64)], 0, 0),
    (8, 2, 128, 16, 128, 4, [(1, 500), (1, 77)], 0, 0),
    (32, 8, 128, 24, 0, 0, [(1, 300), (8, 301), (9, 100), (40, 40), (1, 1)], 2, 3),   # few and many rows together
    (32, 1, 64, 64, 0, 0, [(1, 300), (1, 1), (1, 0)], 0, 0),         # 32 rows, one key head
    (72, 2, 64, 40, 77, 3, [(1, 200), (1, 0), (1, 5), (4, 90)], 0, 0),
    (40, 1, 128, 16, 50, 2, [(7, 90)], 0, 0),
    (8, 8, 128, 16, 2048, 4, [(1, 3000)], 0, 0),                     # split keys
    (2, 2, 64, 128, 0, 0, [(100, 1700)], 0, 0),                      # several row tiles over split keys
    (6, 2, 72, 48, 1600, 5, [(45, 2100), (20, 900)], 0, 0),
    (4, 2, 128, 256, 1580, 40, [(0, 30), (40, 1601), (33, 1600)], 0, 0),
    (4, 4, 64, 8, 40, 4, [(150, 150), (0, 0), (1, 1), (129, 200)], 0, 0),
    (2, 2, 96, 16, 50, 2, [(300, 100)], 0, 0),
    (3, 3, 8, 32, 16, 3, [(40, 200), (200, 210)], 5, 0),
    (4, 1, 128, 32, 0, 0, [(700, 4200)], 0, 0),                      # a chunk over a long text: split keys
    (8, 2, 64, 16, 300, 8, [(600, 2700), (1, 2000), (2, 10)], 0, 1),
    (16, 16, 64, 64, 0, 0, [(513, 700), (1, 640), (600, 600)], 0, 0),
    (32, 8, 128, 128, 400, 130, [(520, 1500), (300, 900)], 0, 0),    # whole tiles, window and sinks
    (12, 4, 104, 72, 0, 0, [(3, 100)] * 70 + [(65, 65)], 0, 0),      # more sequences than a wave tries at once
    (8, 8, 40, 16, 9, 0, [(1, 3 + i) for i in range(130)], 0, 0),
]


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "x".join(str(x) for x in c[:6]) + f"_{len(c[6])}")
def test_paged(lact, case, t):
    H, Hk, d, page, window, sinks, seqs, first, behind = case
    dt = DT[t]
    gen = torch.Generator("cuda").manual_seed(sum(case[:6]))
    new, lens = [n for n, _ in seqs], [m for _, m in seqs]
    off = sums(new, first)
    T = off[-1] + behind
    layout = ("heads", "tokens", "wide")[(T + d) % 3]
    q = rows(gen, H, T, d, dt, layout)
    kp, vp, table = _cache(gen, lens, Hk, page, d, dt, "tokens" if (sum(lens) + page) % 2 else "heads")
    print("paged", t, layout, case, flush=True)
    ref = _paged_ref(q, kp, vp, table, off, lens, window, sinks, float(np.float32(0.3)))
    ref["o"][:, :first] = ref["o"][:, off[-1]:] = 0
    q[:, :first] = float("nan")
    for bounds in (dict(), dict(longest=max(new)), dict(longest=max(new), k_len=max(lens))):
        o, lse = lact.paged_attention(q, kp, vp, table=whole(table, torch.int32), offsets=whole(off), k_lens=whole(lens),
                                      window=window, sinks=sinks, scale=0.3, return_lse=True, **bounds)
        torch.cuda.synchronize()
        assert o.stride() == torch.empty_like(q).stride()
        check_attention(ref, {"o": o, "lse": lse}, dt, d, max(lens + [1]), False)


@pytest.mark.parametrize("longest", [1, 40, None])
def test_given_results_keep_what_is_no_sequences(lact, longest):
    gen = torch.Generator("cuda").manual_seed(1)
    n = 1 if longest == 1 else 40
    off, lens = [4, 4 + n, 4 + n, 5 + n], [90, 3, 50]
    T = 9 + n
    q = rows(gen, 4, T, 64, torch.bfloat16, "tokens")
    kp, vp, table = _cache(gen, lens, 2, 16, 64, torch.bfloat16, "heads")
    kw = dict(table=whole(table, torch.int32), offsets=whole(off), k_lens=whole(lens), longest=longest)
    want, wlse = lact.paged_attention(q, kp, vp, return_lse=True, **kw)
    idle = [i for i in range(T) if not 4 <= i < 5 + n]
    assert (want[:, idle] == 0).all() and (wlse[:, idle] == 0).all()
    o, lse = torch.full_like(q, 7.0), torch.full((4, T), 7.0, device="cuda")
    got = lact.paged_attention(q, kp, vp, o, lse=lse, return_lse=True, **kw)
    assert got[0] is o and got[1] is lse
    live = slice(4, 5 + n)
    assert torch.equal(o[:, live], want[:, live]) and torch.equal(lse[:, live], wlse[:, live])
    assert (o[:, idle] == 7).all() and (lse[:, idle] == 7).all()
    # one given, one not
    o2 = torch.full_like(q, 7.0)
    _, lse2 = lact.paged_attention(q, kp, vp, o2, return_lse=True, **kw)
    assert (o2[:, idle] == 7).all() and torch.equal(lse2, wlse)
    # packed: the same, and gradients are zero there
    kw = dict(offsets=whole(off), longest=longest, window=9, sinks=1)
    k = q[:2]
    want, wlse = lact.packed_attention(q, k, k, return_lse=True, **kw)
    assert (want[:, idle] == 0).all() and (wlse[:, idle] == 0).all()
    o.fill_(7.0)
    lse.fill_(7.0)
    lact.packed_attention(q, k, k, o, lse=lse, **kw)
    assert torch.equal(o[:, live], want[:, live]) and torch.equal(lse[:, live], wlse[:, live])
    assert (o[:, idle] == 7).all() and (lse[:, idle] == 7).all()
    out = {n: torch.full_like(x, 7.0) for n, x in (("dq", q), ("dk", k), ("dv", k))}
    got = lact.packed_attention_backward(q, k, k, o, lse, dO=q, out=out, **kw)
    other = lact.packed_attention_backward(q, k, k, o, lse, dO=q, **kw)
    for name, x in got.items():
        assert x is out[name] and (x[:, idle] == 0).all() and torch.equal(x, other[name])


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(1, 900), (5, 900), (200, 900), (200, 3100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_non_finite_token_reaches_only_rows_that_see_it(lact, t, d, n, m, bad):
    gen = torch.Generator("cuda").manual_seed(4)
    dt, page, window, sinks = DT[t], 24, 333, 3
    seqs = [(n, m), (max(1, n // 2), m // 2)]
    new, lens = [x for x, _ in seqs], [x for _, x in seqs]
    off = sums(new)
    q = rows(gen, 4, off[-1], d, dt, "tokens")
    kp, vp, table = _cache(gen, lens, 2, page, d, dt, "tokens")
    kw = dict(table=whole(table, torch.int32), offsets=whole(off), k_lens=whole(lens), longest=max(new), window=window,
              sinks=sinks)
    want = lact.paged_attention(q, kp, vp, **kw)
    ref = _paged_ref(q, kp, vp, table, off, lens, window, sinks, d ** -0.5)
    for j in (1, m // 2, m - 100, m - 2):   # a sink's key, one that few rows see or none
        v2 = vp.clone()
        v2[table[0, j // page], 1, j % page, 5] = bad
        got = lact.paged_attention(q, kp, v2, **kw)
        see = OB.visible(n, m, window, sinks)[:, j]
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[2:, : off[1], 5] = torch.from_numpy(see).cuda()
        assert (~torch.isfinite(got) == hit).all(), j
        o = torch.where(hit, want, got)
        check_attention(ref, {"o": o}, dt, d, m, False)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(3, 4000), (150, 150), (256, 4000)])
@pytest.mark.parametrize("size", [2.0 ** 104, 2.0 ** 127])
def test_values_near_the_types_largest(lact, t, d, n, m, size):
    """As for window attention: an average is no larger than the largest value,
    also where scores climb along split keys."""
    gen = torch.Generator("cuda").manual_seed(5)
    dt = DT[t]
    q = rows(gen, 1, n, d, dt, "heads")
    kp, vp, table = _cache(gen, [m], 1, 64, d, dt, "heads")
    q[..., 0] = 8.0
    climb = (torch.arange(m, device="cuda") / m * 1.7).to(dt)
    for i in range(-(-m // 64)):
        at, c = table[0, i], min(64, m - 64 * i)
        kp[at, 0, :c, 0] = climb[64 * i : 64 * i + c]
        x = vp[at, 0, :c]
        vp[at, 0, :c] = (torch.sign(x) * (1 + x.abs().clamp(max=3) / 4) * size).to(dt)
    ref = _paged_ref(q, kp, vp, table, [0, n], [m], 0, 0, 1.0)
    o = lact.paged_attention(q, kp, vp, table=whole(table, torch.int32), offsets=whole([0, n]), k_lens=whole([m]),
                             scale=1.0)
    check_attention(ref, {"o": o}, dt, d, m, False)


def test_numbers_on_the_device_are_cut_to_the_arrays(lact):
    """Lengths beyond the table, offsets out of order or range, bounds that are too small: cut, not followed."""
    gen = torch.Generator("cuda").manual_seed(6)
    q = rows(gen, 4, 60, 64, torch.float32, "heads")
    kp, vp, table = _cache(gen, [80, 70], 2, 16, 64, torch.float32, "heads")
    kp.nan_to_num_()
    vp.nan_to_num_()
    table = np.clip(table, 0, kp.shape[0] - 1)   # rows of the table: 7 pages, 112 keys
    tab, full = whole(table, torch.int32), 16 * table.shape[1]
    run = lambda off, lens, **kw: lact.paged_attention(q, kp, vp, table=tab, offsets=whole(off), k_lens=whole(lens), **kw)
    good = run([0, 20, 60], [full, 70])
    assert torch.equal(run([0, 20, 60], [1 << 40, 70]), good)
    assert torch.equal(run([-5, 20, 1 << 40], [full, 70]), good)
    assert torch.equal(run([0, 20, 60], [full, 70], longest=1 << 40, k_len=1 << 40), good)
    assert (run([0, 20, 20], [-3, 70]) == 0).all()
    back = run([0, 40, 20], [full, 70])     # the second sequence has no rows
    assert torch.equal(back[:, :40], run([0, 40, 60], [full, 70])[:, :40])
    ref = _paged_ref(q, kp, vp, table, [0, 20, 60], [50, 50], 0, 0, 0.125)
    check_attention(ref, {"o": run([0, 20, 60], [full, 70], k_len=50)}, torch.float32, 64, 112, False)
    k = q[:2]
    one = lact.packed_attention(q, k, k, offsets=whole([0, 20, 60]))
    assert torch.equal(lact.packed_attention(q, k, k, offsets=whole([-7, 20, 99])), one)
    got = lact.packed_attention(q, k, k, offsets=whole([0, 20, 60]), longest=30)
    assert torch.equal(got[:, :20], one[:, :20])
    check_attention(OP.packed_attention(f64(q), f64(k), f64(k), [0, 20, 50], 0, 0, 0.125), {"o": torch.cat(
        [got[:, :50], torch.zeros_like(got[:, 50:])], 1), }, torch.float32, 64, 60, False)


def test_offsets_out_of_order_stay_inside(lact):
    """Offsets that jump about: whatever they give, nothing outside the tensors is touched."""
    gen = torch.Generator("cuda").manual_seed(14)
    T, d = 4000, 64
    around = [torch.full((T + 200, h, d), 7.0, device="cuda", dtype=torch.bfloat16) for h in (4, 4, 2, 2)]
    o, dq, dk, dv = (x[100 : T + 100].transpose(0, 1) for x in around)
    q = rows(gen, 4, T, d, torch.bfloat16, "tokens")
    k = rows(gen, 2, T, d, torch.bfloat16, "tokens")
    kp, vp, table = _cache(gen, [900] * 90, 2, 32, d, torch.bfloat16, "heads")
    for B in (20, 90):
        # found by slots: one long sequence, then numbers in any order
        jump = torch.randint(-10, T + 10, (B - 1,), generator=gen, device="cuda").tolist()
        off = whole([0, 3000] + jump)
        _, lse = lact.packed_attention(q, k, k, o, offsets=off, longest=3000, return_lse=True)
        lact.packed_attention_backward(q, k, k, o, lse, dO=q, offsets=off, longest=3000, out=dict(dq=dq, dk=dk, dv=dv))
        lact.paged_attention(q, kp, vp, o, table=whole(table[:B], torch.int32), offsets=off, k_lens=whole([900] * B))
        torch.cuda.synchronize()
        assert all((x[:100] == 7).all() and (x[T + 100 :] == 7).all() for x in around)


@pytest.mark.parametrize("longest", [1, 30])
def test_rows_behind_the_longest_are_no_sequences(lact, longest):
    gen = torch.Generator("cuda").manual_seed(15)
    off, n = [3, 63, 64, 164], 170
    q, k = rows(gen, 4, n, 64, torch.float32, "heads"), rows(gen, 2, n, 64, torch.float32, "heads")
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, z in zip(off[:-1], off[1:]):
        live[a : min(z, a + longest)] = True
    kw = dict(offsets=whole(off), longest=longest)
    o, lse = lact.packed_attention(q, k, k, return_lse=True, **kw)
    g = lact.packed_attention_backward(q, k, k, o, lse, dO=q, **kw)
    kp, vp, table = _cache(gen, [70, 9, 200], 2, 8, 64, torch.float32, "tokens")
    p = lact.paged_attention(q, kp, vp, table=whole(table, torch.int32), k_lens=whole([70, 9, 200]), **kw)
    for x in (o, lse, p, *g.values()):
        assert (x[:, ~live] == 0).all() and x[:, live].any()
    given = torch.full_like(q, 7.0)
    lact.packed_attention(q, k, k, given, **kw)
    assert (given[:, ~live] == 7).all() and torch.equal(given[:, live], o[:, live])


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("seqs", [[(1, 1900), (1, 700)], [(90, 1900), (1, 700), (70, 90)]])
def test_pages_before_the_window_may_be_gone(lact, t, seqs):
    """Entries between the sinks and what the window of any row reaches lead nowhere, or to pages that hold NaN."""
    dt, window, sinks, page = DT[t], 200, 5, 16
    gen = torch.Generator("cuda").manual_seed(16)
    new, lens = [n for n, _ in seqs], [m for _, m in seqs]
    q = rows(gen, 4, sum(new), 64, dt, "tokens")
    kp, vp, table = _cache(gen, lens, 2, page, 64, dt, "heads", spare=8)
    used = {int(x) for b, m in enumerate(lens) for x in table[b, : -(-m // page)]}
    spare = [x for x in range(kp.shape[0]) if x not in used]
    kp[spare], vp[spare] = float("nan"), float("inf")
    kw = dict(offsets=whole(sums(new)), k_lens=whole(lens), window=window, sinks=sinks, longest=max(new))
    want = lact.paged_attention(q, kp, vp, table=whole(table, torch.int32), **kw)
    for b, (n, m) in enumerate(seqs):
        first, last = -(-sinks // page), max(0, m - n - window + 1) // page   # pages that no row sees
        for i in range(first, last):
            table[b, i] = (-1, 2 ** 31 - 1, -2 ** 31, spare[i % len(spare)])[i % 4]
    got = lact.paged_attention(q, kp, vp, table=whole(table, torch.int32), **kw)
    # a row that a NaN passed is summed again, in another order
    ref = _paged_ref(q, kp, vp, np.clip(table, 0, kp.shape[0] - 1), sums(new), lens, window, sinks, 0.125)
    check_attention(ref, {"o": got}, dt, 64, max(lens), False)
    assert torch.isfinite(got).all() and float((got - want).abs().max()) < 0.1


@pytest.mark.parametrize("t,d,B", [("bf16", 64, 300), ("fp32", 128, 200), ("bf16", 128, 700), ("fp32", 40, 257)])
@pytest.mark.parametrize("chunk", [0, 60])
def test_many_requests(lact, t, d, B, chunk):
    """More sequences than a workgroup sums in one round, and than it sums itself; some without rows or keys."""
    rng, dt = np.random.default_rng([B, chunk]), DT[t]
    gen = torch.Generator("cuda").manual_seed(17)
    new = [int(x) for x in rng.integers(0, 3, B)]
    if chunk:
        new[B // 2] = chunk
    lens = [int(x) for x in rng.integers(0, 200, B)]
    lens[B // 2], lens[3] = 900, 0
    q = rows(gen, 8, sum(new), d, dt, "tokens")
    kp, vp, table = _cache(gen, lens, 2, 16, d, dt, "tokens")
    kw = dict(table=whole(table, torch.int32), offsets=whole(sums(new)), k_lens=whole(lens), longest=max(new), window=150,
              sinks=3, scale=0.3)
    print("many", t, d, B, chunk, flush=True)
    ref = _paged_ref(q, kp, vp, table, sums(new), lens, 150, 3, float(np.float32(0.3)))
    for _ in range(2):
        o, lse = lact.paged_attention(q, kp, vp, return_lse=True, **kw)
        check_attention(ref, {"o": o, "lse": lse}, dt, d, 900, False)


def test_work_counted_in_several_tiles(lact):
    """A table so wide that the tiles it could hold pass 2^30: the same results."""
    gen = torch.Generator("cuda").manual_seed(18)
    B, page, width = 40, 65536, 16383
    kp, vp = (torch.randn(3, 1, page, 8, generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0], table[:, 1] = torch.arange(B, device="cuda") % 3, (torch.arange(B, device="cuda") + 1) % 3
    lens = [1, 31, 32, 33, 65536, 65537, 70000, 0] * 5
    q = rows(gen, 2, B, 8, torch.bfloat16, "heads")
    kw = dict(table=table, offsets=whole(list(range(B + 1))), k_lens=whole(lens), longest=1)
    ref = _paged_ref(q, kp, vp, table.cpu().numpy()[:, :2], list(range(B + 1)), lens, 0, 0, 8 ** -0.5)
    for bound in (None, 70000):
        check_attention(ref, {"o": lact.paged_attention(q, kp, vp, k_len=bound, **kw)}, torch.bfloat16, 8, 70000, False)


def test_a_cache_beyond_32_bit_offsets(lact):
    """Pages more than 4 GB apart, and rows of q and o."""
    gen = torch.Generator("cuda").manual_seed(7)
    P, Hk, page, d = 9000, 2, 256, 512        # 4.7 GB of pages of rows of 512, of which heads take 64
    pool = torch.zeros(P, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    kp = pool.transpose(1, 2)[..., 64:128]
    lens, new = [600, 300], [1, 70]
    table = np.array([[8999, 0, 8500], [4300, 8998, -1]])
    for at in (0, 4300, 8500, 8998, 8999):
        kp[at] = torch.randn((Hk, page, 64), generator=gen, device="cuda").bfloat16()
    q = torch.randn(71, 4, 64, generator=gen, device="cuda").bfloat16().transpose(0, 1)
    few = [0, 8500, 8998, 8999, 4300]
    small = kp[few].contiguous()
    for n in ([1, 1], new):
        off = sums(n)
        qq = q[:, : off[-1]]
        o = lact.paged_attention(qq, kp, kp, table=whole(table, torch.int32), offsets=whole(off), k_lens=whole(lens))
        ref = OP.paged_attention(f64(qq), f64(small), f64(small), np.array([[3, 0, 1], [4, 2, 0]]), off, lens, 0, 0, 0.125)
        check_attention(ref, {"o": o}, torch.bfloat16, 64, 600, False)
    x = torch.randn(3, Hk, 64, generator=gen, device="cuda").bfloat16().transpose(0, 1)
    vp = pool.transpose(1, 2)[..., 128:192]
    before = pool.float().sum(dtype=torch.float64)
    lact.page_write(x, x, kp, vp, slots=whole([8999 * 256 + 255, 8999 * 256, 5]))
    for s, i in ((8999 * 256 + 255, 0), (8999 * 256, 1), (5, 2)):
        assert torch.equal(kp[s // 256, :, s % 256], x[:, i]) and torch.equal(vp[s // 256, :, s % 256], x[:, i])
    assert torch.isfinite(before) and (pool[..., 192:] == 0).all() and (pool[..., :64] == 0).all()


# ------------------------------------------------------------------ slots and writes
def _slots_case(rng, B, T, page, width, short, idle):
    counts = rng.integers(0, 2, B) if idle else np.ones(B, np.int64)
    extra = max(0, T - int(counts.sum()))
    if extra and B:
        counts = counts + rng.multinomial(extra - extra // 5, rng.dirichlet(np.full(B, 0.3)))
    lens = rng.integers(0, max(1, width * page - 1), B)
    lens[rng.random(B) < 0.1] = 0
    if B:
        counts[0], lens[-1] = -3, -9
    table = np.full((B, width), -1, np.int64)
    held = -(-np.maximum(lens, 0) // page)
    for b in range(B):
        table[b, : held[b]] = rng.integers(0, 1 << 20, held[b])
    free = rng.permutation(5000)
    have = int(rng.integers(0, 30)) if short else 5000
    return [int(x) for x in lens], [int(x) for x in counts], table, [int(x) for x in free], have


@pytest.mark.parametrize("B,T,page,width", [(1, 1, 8, 4), (1, 50, 16, 3), (7, 30, 24, 5), (64, 64, 16, 20),
                                            (300, 2000, 8, 50), (1024, 8192, 16, 30), (1025, 1025, 16, 9),
                                            (1100, 9000, 64, 7), (65, 20001, 8, 300), (3000, 3500, 128, 2),
                                            (1024, 8193, 16, 30), (0, 5, 8, 3), (5, 0, 8, 3), (2049, 12000, 32, 0)])
@pytest.mark.parametrize("short,idle", [(False, False), (True, True)])
def test_slots(lact, B, T, page, width, short, idle):
    rng = np.random.default_rng([B, T, page, short])
    lens, counts, table, free, have = _slots_case(rng, B, T, page, width, short, idle)
    print("slots", B, T, page, width, short, flush=True)
    want, wtable = OP.page_slots(lens, counts, table, free, have, page, T)
    dev = lambda: (whole(lens), whole(counts), whole(table, torch.int32).reshape(B, width), whole(free, torch.int32),
                   whole([have]))
    args = dev()
    for _ in range(2):   # a call repeated gives the same
        got = lact.page_slots(*args, page=page, tokens=T)
        torch.cuda.synchronize()
        for n, x in want.items():
            assert got[n].tolist() == x, n
        assert args[2].tolist() == [[int(x) for x in r] for r in wtable]
    # results given, what is left in place of what was free
    args = dev()
    out = {n: torch.full_like(x, 77) for n, x in got.items()}
    out["left"][0] = have
    back = lact.page_slots(*args[:4], out["left"], page=page, tokens=T, out=out)
    assert back is out and all(torch.equal(out[n], got[n]) for n in got) and args[2].tolist() == [list(map(int, r)) for r in wtable]


def test_slots_of_unusual_numbers(lact):
    """Counts and lengths near the ends of their type, more rows than the step has, a table that lacks pages."""
    big = 1 << 62
    lens, counts = [big, 3, -big, 5, 0, 9], [5, big, 4, -big, 1, 1]
    table = [[0] * 4, [7, 1, 1, 1], [-1] * 4, [2] * 4, [-1] * 4, [3, -1, 6, 6]]
    for T in (0, 5, 6, 30, 9000):
        for have in (3, -4, 1 << 60):
            want, wtable = OP.page_slots(lens, counts, table, list(range(20, 30)), have, 8, T)
            tab = whole(table, torch.int32)
            got = lact.page_slots(whole(lens), whole(counts), tab, whole(list(range(20, 30)), torch.int32), whole([have]),
                                  page=8, tokens=T)
            assert all(got[n].tolist() == x for n, x in want.items()), (T, have)
            assert tab.tolist() == wtable


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("Hk,T,d,page,layout", [(1, 1, 8, 8, "heads"), (2, 33, 64, 16, "tokens"), (3, 130, 72, 24, "wide"),
                                                (8, 700, 128, 16, "tokens"), (5, 257, 1000, 8, "heads"),
                                                (8, 20000, 128, 64, "wide"), (64, 4100, 128, 256, "heads")])
def test_write(lact, Hk, T, d, page, layout, t):
    gen = torch.Generator("cuda").manual_seed(T)
    dt = DT[t]
    P = T // page + 2
    k, v = (rows(gen, Hk, T, d, dt, layout) for _ in range(2))
    kp = torch.randn(P, page, Hk, d, generator=gen, device="cuda").to(dt).transpose(1, 2)
    vp = torch.randn(P, Hk, page, d, generator=gen, device="cuda").to(dt)
    slots = torch.randperm(P * page, generator=gen, device="cuda")[:T]
    slots[::7] = -1
    if T > 4:
        slots[1], slots[2], slots[3] = P * page, 1 << 40, -(1 << 40)
    want = []
    for x, p in ((k, kp), (v, vp)):
        p = p.clone()
        live = (slots >= 0) & (slots < P * page)
        s = slots[live]
        p[s // page, :, s % page] = x[:, live].transpose(0, 1)
        want.append(p)
    print("write", t, Hk, T, d, page, layout, flush=True)
    got = lact.page_write(k, v, kp, vp, slots=slots)
    assert got[0] is kp and got[1] is vp
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_a_slot_given_twice_holds_one_of_its_rows(lact):
    k = torch.arange(6, device="cuda").float().view(1, 6, 1).expand(1, 6, 8).contiguous()
    pool = torch.zeros(2, 1, 8, 8, device="cuda"), torch.zeros(2, 1, 8, 8, device="cuda")
    lact.page_write(k, k, *pool, slots=whole([3, 9, 3, 9, 9, 3]))
    for p in pool:
        assert all(x in (0, 2, 5) for x in p[0, 0, 3].tolist()) and all(x in (1, 3, 4) for x in p[1, 0, 1].tolist())


# ------------------------------------------------------------------ callers
def _step(lact, s, x, counts, tokens, fr, kw):
    """One step of a server: places, positions, the cache, attention."""
    q, k, v = x
    at = lact.page_slots(s["lens"], counts, s["table"], s["free"], s["left"], page=s["page"], tokens=tokens)
    qr, kr = (r[0] for r in lact.rotary(q[None], k[None], freqs=fr, positions=at["positions"][None]))
    lact.page_write(kr, v, s["k"], s["v"], slots=at["slots"])
    o = lact.paged_attention(qr, s["k"], s["v"], table=s["table"], offsets=at["offsets"], k_lens=at["k_lens"], **kw)
    s["lens"].copy_(at["k_lens"])
    s["left"].copy_(at["left"])
    return o


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_a_server_steps_equal_whole_sequences(lact, t):
    """Prompts in chunks and next tokens of four requests, in steps of different
    mixtures, over one cache: each request's rows are those of its whole
    sequence; and the same sequences packed.  A request that ends gives its
    pages back, and another takes its place."""
    dt, H, Hk, d, page = DT[t], 8, 2, 64, 16
    gen = torch.Generator("cuda").manual_seed(8)
    fr, _ = lact.rotary_frequencies(d // 2)
    total = [300, 75, 1, 150]
    full = [[rows(gen, h, n, d, dt, "tokens") for h in (H, Hk, Hk)] for n in total]
    P = 40
    s = dict(lens=whole([0] * 4), table=torch.full((4, 24), -1, dtype=torch.int32, device="cuda"),
             free=torch.randperm(P, generator=gen, device="cuda").int(), left=whole([P, 0]), page=page,
             k=torch.full((P, page, Hk, d), float("nan"), device="cuda", dtype=dt).transpose(1, 2),
             v=torch.full((P, page, Hk, d), float("nan"), device="cuda", dtype=dt).transpose(1, 2))
    kw = dict(window=100, sinks=4, longest=128)
    steps = [[128, 75, 0, 20], [128, 0, 1, 1], [1, 0, 0, 64]] + [[1, 0, 0, 1]] * 42 + [[1, 0, 0, 23]]
    got, done = [[] for _ in total], [0] * 4
    for counts in steps:
        x = [torch.cat([full[b][i][:, done[b] : done[b] + c] for b, c in enumerate(counts)] +
                       [torch.zeros((full[0][i].shape[0], 3, d), device="cuda", dtype=dt)], 1) for i in range(3)]
        tokens = sum(counts) + 3   # a padded step
        o = _step(lact, s, x, whole(counts), tokens, fr, kw)
        assert (o[:, sum(counts):] == 0).all()
        at = 0
        for b, c in enumerate(counts):
            got[b].append(o[:, at : at + c])
            done[b] += c
            at += c
    assert done == total and s["left"][1] == 0 and s["lens"].tolist() == total
    off = whole(sums(total))
    q, k, v = (torch.cat([f[i] for f in full], 1) for i in range(3))
    pos = torch.cat([torch.arange(n, device="cuda") for n in total])[None]
    qr, kr = (r[0] for r in lact.rotary(q[None], k[None], freqs=fr, positions=pos))
    ref = OP.packed_attention(f64(qr), f64(kr), f64(v), sums(total), 100, 4, 0.125)
    check_attention(ref, {"o": torch.cat([x for g in got for x in g], 1)}, dt, d, 300, False)
    check_attention(ref, {"o": lact.packed_attention(qr, kr, v, offsets=off, longest=300, window=100, sinks=4)}, dt, d, 300,
                    False)
    # request 1 ends: its pages go back, by the caller, and a new one takes its row
    n = -(-75 // page)
    left = int(s["left"][0])
    s["free"][left : left + n] = s["table"][1, :n]
    s["left"][0] += n
    s["lens"][1] = 0
    s["table"][1] = -1
    x = [rows(gen, h, 90, d, dt, "tokens") for h in (H, Hk, Hk)]
    o = _step(lact, s, x, whole([0, 90, 0, 0]), 90, fr, kw)
    qr, kr = (r[0] for r in lact.rotary(x[0][None], x[1][None], freqs=fr))
    ref = OP.packed_attention(f64(qr), f64(kr), f64(x[2]), [0, 90], 100, 4, 0.125)
    check_attention(ref, {"o": o}, dt, d, 300, False)
    assert s["left"].tolist() == [P - 19 - 1 - 10 - 6, 0]


@pytest.mark.parametrize("counts", [[1, 1, 1], [1, 90, 3]])
def test_graph_of_a_servers_step(lact, counts):
    """A step captured once and replayed as the requests grow, against the same steps run eagerly."""
    H, Hk, d, page, T = 4, 2, 64, 16, 100
    gen = torch.Generator("cuda").manual_seed(9)
    fr, _ = lact.rotary_frequencies(d // 2)
    kw = dict(window=50, sinks=2, longest=max(counts + [2]))   # what any replay has

    def state():
        g = torch.Generator("cuda").manual_seed(10)
        P = 80
        pool = lambda: torch.randn(P, page, Hk, d, generator=g, device="cuda").bfloat16().transpose(1, 2)
        # lengths, pages held, and everything else free
        s = dict(lens=whole([200, 0, 33]), page=page, left=whole([P - 16, 0]), k=pool(), v=pool(),
                 free=torch.arange(P, device="cuda").int(), table=torch.full((3, 60), -1, dtype=torch.int32, device="cuda"))
        s["table"][0, :13] = torch.arange(64, 77).int()
        s["table"][2, :3] = torch.arange(77, 80).int()
        s["x"] = [torch.randn(T, h, d, generator=g, device="cuda").bfloat16().transpose(0, 1) for h in (H, Hk, Hk)]
        s["counts"] = whole(counts)
        s["o"] = torch.zeros(T, H, d, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
        return s

    def step(s):
        s["o"].copy_(_step(lact, s, s["x"], s["counts"], T, fr, kw))

    a, b = state(), state()
    step(a)   # warm
    a = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(a)
    torch.cuda.synchronize()
    for i in range(5):
        for s in (a, b):
            gen.manual_seed(100 + i)
            for x in s["x"]:
                x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        if i == 3:
            a["counts"].copy_(whole([0, 1, 2]))
            b["counts"].copy_(whole([0, 1, 2]))
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(a["o"], b["o"]) and torch.equal(a["lens"], b["lens"]) and torch.equal(a["left"], b["left"])
        assert torch.equal(a["table"], b["table"]) and torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])


@pytest.mark.parametrize("G", [1, 4])
def test_graph_of_a_training_step(lact, G):
    """Packed attention and its gradients from a graph, with other texts in other lengths from replay to replay."""
    T, Hk, d = 900, 2, 64
    gen = torch.Generator("cuda").manual_seed(11)
    x = [rows(gen, h, T, d, torch.bfloat16, "tokens") for h in (G * Hk, Hk, Hk, G * Hk)]
    off = whole([0, 400, 400, 900])
    kw = dict(window=70, sinks=3, longest=500)
    s = {}

    def call():
        q, k, v, g = x
        o, lse = lact.packed_attention(q, k, v, return_lse=True, offsets=off, **kw)
        out = dict(lact.packed_attention_backward(q, k, v, o, lse, dO=g, offsets=off, **kw), o=o, lse=lse)
        for n, t in out.items():
            s.setdefault(n, torch.empty_like(t)).copy_(t)

    _graph(call, lambda: list(s.values()))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lens in ([400, 0, 500], [10, 490, 100], [0, 0, 500], [500, 1, 300]):
        off.copy_(whole(sums(lens)))
        for t in x:
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in s.items()}
        call()
        assert all(torch.equal(got[n], s[n]) for n in s), lens


def test_calls_on_streams(lact):
    """Two streams at once, each with its own state, give what each alone gives."""
    gen = torch.Generator("cuda").manual_seed(12)
    fr, _ = lact.rotary_frequencies(32)
    sets = []
    for _ in range(2):
        kp, vp, table = _cache(gen, [900, 2500, 40], 2, 32, 64, torch.bfloat16, "tokens")
        q = rows(gen, 8, 122, 64, torch.bfloat16, "tokens")
        sets.append((q, kp, vp, dict(table=whole(table, torch.int32), offsets=whole([0, 1, 121, 122]),
                                     k_lens=whole([900, 2500, 40]))))
    k = [rows(gen, 2, 122, 64, torch.bfloat16, "heads") for _ in range(2)]
    off = whole([0, 50, 122])

    def one(i, st):
        q, kp, vp, kw = sets[i]
        o = lact.paged_attention(q, kp, vp, stream=st, longest=120, **kw)
        few = lact.paged_attention(q[:, :3], kp, vp, stream=st, longest=1, table=kw["table"], k_lens=kw["k_lens"],
                                   offsets=steps[i])
        p, lse = lact.packed_attention(q, k[i], k[i], offsets=off, return_lse=True, stream=st)
        g = lact.packed_attention_backward(q, k[i], k[i], p, lse, dO=q, offsets=off, stream=st)
        return [o, few, p, lse] + list(g.values())

    steps = [whole([0, 1, 2, 3]) for _ in range(2)]
    want = [one(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [one(i, st) for i, st in enumerate(streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    a = (whole([5, 0]), whole([2, 9]), torch.zeros(2, 3, dtype=torch.int32, device="cuda"),
         torch.arange(9, device="cuda").int(), whole([9]))
    want = lact.page_slots(*a, page=8, tokens=12)
    torch.cuda.synchronize()
    got = lact.page_slots(*a, page=8, tokens=12, stream=streams[0])
    pool = torch.zeros(9, 2, 8, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(9, 2, 8, 64, device="cuda",
                                                                                     dtype=torch.bfloat16)
    torch.cuda.synchronize()
    lact.page_write(k[0][:, :12], k[0][:, :12], *pool, slots=want["slots"], stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want) and pool[0].any()


def test_parameters_given_as_tensors_are_read_at_every_call(lact):
    gen = torch.Generator("cuda").manual_seed(13)
    q = rows(gen, 2, 60, 64, torch.float32, "heads")
    off = whole([0, 60])
    o, lse = lact.packed_attention(q, q, q, offsets=off, return_lse=True)
    kp, vp, table = _cache(gen, [60], 2, 8, 64, torch.float32, "heads")
    kw = dict(table=whole(table, torch.int32), offsets=off, k_lens=whole([60]))
    calls = {}
    for name, one, two in (("window", 2, 9), ("scale", 0.1, 0.7), ("longest", 20, 60)):
        calls[name] = (one, two, lambda x, n=name: lact.packed_attention(q, q, q, offsets=off, **{n: x}))
        if name != "longest":
            calls[name + " back"] = (one, two, lambda x, n=name: lact.packed_attention_backward(
                q, q, q, o, lse, dO=q, offsets=off, **{n: x})["dk"])
        calls[name + " paged"] = (one, two, lambda x, n=name: lact.paged_attention(q, kp, vp, **dict(kw, **{n: x})))
    calls["k_len"] = (20, 56, lambda x: lact.paged_attention(q, kp, vp, k_len=x, **kw))
    for name, (first, then, call) in calls.items():
        x = torch.tensor(first)
        one = call(x)
        x.fill_(then)
        two = call(x)
        part = slice(0, 20) if "longest" in name else slice(0, 60)   # rows behind `longest` are not looked at
        if name != "longest paged":   # there it moves the rows' positions
            assert torch.equal(one[:, part], call(torch.tensor(first).item())[:, part]), name
        assert torch.equal(two, call(torch.tensor(then).item())), name
        if "longest" not in name:
            assert not torch.equal(one, two), name


def test_binding_refusals_on_the_device(lact):
    q, off = torch.zeros(2, 8, 64, device="cuda"), whole([0, 8])
    pool, table, n = torch.zeros(3, 2, 8, 64, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda"), whole([8])
    paged = lambda q=q, k=pool, v=pool, **kw: lact.paged_attention(q, k, v, **dict(dict(table=table, offsets=off, k_lens=n), **kw))
    bad = [lambda: lact.packed_attention(q, q[:, :4], q, offsets=off), lambda: lact.packed_attention(q, q, q.bfloat16(), offsets=off),
           lambda: lact.packed_attention(q, q, q, offsets=off.int()), lambda: lact.packed_attention(q, q, q, offsets=off[:0]),
           lambda: lact.packed_attention(q, q, q, offsets=off.cpu()), lambda: lact.packed_attention(q, q, q, offsets=off, longest=-1),
           lambda: lact.packed_attention(q, q, q, q[:1], offsets=off), lambda: lact.packed_attention(q, q, q, offsets=off, lse=q[..., 0]),
           lambda: paged(k=pool[..., :32]), lambda: paged(v=pool[:2]), lambda: paged(k=pool.bfloat16()),
           lambda: paged(table=table.long()), lambda: paged(table=table[0]), lambda: paged(table=whole([[0, 0]] * 2, torch.int32)),
           lambda: paged(table=torch.zeros(1, 4, dtype=torch.int32, device="cuda")[:, ::2]),
           lambda: paged(k_lens=whole([8, 8])), lambda: paged(k_lens=n.int()), lambda: paged(k=pool.cpu()),
           lambda: paged(workspace=torch.empty(8, device="cuda")), lambda: paged(longest=-2),
           lambda: lact.page_write(q, q, pool, pool[:2], slots=whole([0] * 8)),
           lambda: lact.page_write(q, q[:, :4], pool, pool, slots=whole([0] * 8)),
           lambda: lact.page_write(q, q, pool, pool, slots=whole([0] * 7)),
           lambda: lact.page_write(q, q, pool, pool, slots=whole([0] * 8).int()),
           lambda: lact.page_slots(n, whole([1, 1]), table, table[0], n, page=8, tokens=4),
           lambda: lact.page_slots(n, n, table.long(), table[0], n, page=8, tokens=4),
           lambda: lact.page_slots(n, n, table, table[0], whole([1, 1, 1]), page=8, tokens=4),
           lambda: lact.page_slots(n.int(), n, table, table[0], n, page=8, tokens=4)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    refused = [lambda: lact.page_write(q, q, pool, pool, slots=whole([0] * 8)),          # one pool for both
               lambda: lact.page_slots(n, n, table, table[0], n, page=12, tokens=4),
               lambda: lact.packed_attention(q[..., 1:57], q[..., :56], q[..., :56], offsets=off),
               lambda: lact.packed_attention(q, q, q, q, offsets=off), lambda: paged(k=pool[:, :, :4], v=pool[:, :, :4]),
               lambda: lact.packed_attention(q, q, q, torch.zeros(1, 8, 64, device="cuda").expand(2, 8, 64), offsets=off)]
    for i, call in enumerate(refused):
        with pytest.raises(lact.LactError):
            call()
            print("not refused:", i)


def test_no_rows_no_keys_no_sequences(lact):
    q, pool = torch.randn(2, 4, 64, device="cuda"), torch.randn(3, 2, 8, 64, device="cuda")
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    o, lse = lact.packed_attention(q, q, q, offsets=whole([0]), return_lse=True)
    assert (o == 0).all() and (lse == 0).all()
    g = lact.packed_attention_backward(q, q, q, o, lse, dO=q, offsets=whole([0]))
    assert all((x == 0).all() for x in g.values())
    assert lact.packed_attention(q[:, :0], q[:, :0], q[:, :0], offsets=whole([0, 0])).shape == (2, 0, 64)
    assert (lact.paged_attention(q, pool, pool, table=none, offsets=whole([0]), k_lens=whole([])) == 0).all()
    kw = dict(offsets=whole([0, 4]), k_lens=whole([0]))
    for p, w in ((pool, 2), (pool, 0), (pool[:0], 2)):
        o, lse = lact.paged_attention(q, p, p, table=torch.zeros(1, w, dtype=torch.int32, device="cuda"), return_lse=True, **kw)
        assert (o == 0).all() and (lse == -float("inf")).all()
    assert lact.page_write(q[:, :0], q[:, :0], pool, pool.clone(), slots=whole([]))[0] is pool
