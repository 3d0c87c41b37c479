"""Packed and paged attention, page slots and page writes without a GPU: the
oracle on cases by hand, and every refusal of the C ABI and the binding (each
before any device work)."""
import ctypes

import numpy as np
import pytest

from oracle import lact_block as OB
from oracle import lact_pages as OP

lact = pytest.importorskip("test_layers_amd.lact", reason="liblact.so not built")
torch = pytest.importorskip("torch")

FAKE = 1 << 20   # aligned, never dereferenced: every call here is refused first
I, U = lact.ERR_INVALID_ARG, lact.ERR_UNSUPPORTED
R = ctypes.byref


# ------------------------------------------------------------------ oracle
def test_slots_by_hand():
    # pages of 8: 5 tokens and 4 more (one new page), 8 and 8 more (one), 0 and 3 more (one)
    out, table = OP.page_slots([5, 8, 0], [4, 8, 3], [[3, -1], [1, -1], [-1, -1]], [9, 7, 6, 2], 4, 8, 17)
    assert table == [[3, 2], [1, 6], [7, -1]]
    assert out["offsets"] == [0, 4, 12, 15] and out["k_lens"] == [9, 16, 3] and out["left"] == [1, 0]
    assert out["slots"] == [29, 30, 31, 16] + list(range(48, 56)) + [56, 57, 58] + [-1, -1]
    assert out["positions"] == [5, 6, 7, 8] + list(range(8, 16)) + [0, 1, 2] + [0, 0]


def test_slots_that_run_out_by_hand():
    # three pages are free: the second request, which asks for three more, and those behind it that ask get none
    out, table = OP.page_slots([0, 0, 7, 0], [8, 24, 1, 1], [[-1] * 3, [-1] * 3, [4, -1, -1], [-1] * 3], [5, 6, 8], 3,
                               8, 40)
    assert out["left"] == [2, 2] and out["k_lens"] == [8, 0, 8, 0]
    assert table == [[8, -1, -1], [-1] * 3, [4, -1, -1], [-1] * 3]
    assert out["slots"][:8] == list(range(64, 72)) and out["slots"][8:32] == [-1] * 24 and out["slots"][32:34] == [39, -1]
    # and one that is longer than its row of the table, whatever is free; the others are served
    out, table = OP.page_slots([15, 3], [2, 2], [[0, 1], [2, -1]], list(range(9)), 9, 8, 4)
    assert out["left"] == [9, 1] and out["slots"] == [-1, -1, 19, 20] and out["k_lens"] == [15, 5]


def test_packed_and_paged_oracles_agree_with_the_padded_one():
    rng = np.random.default_rng(3)
    lens, H, Hk, d, page = [5, 0, 9, 1], 4, 2, 8, 8
    off = np.concatenate([[2], 2 + np.cumsum(lens)])
    q, g = (rng.standard_normal((H, 20, d)) for _ in range(2))
    k, v = (rng.standard_normal((Hk, 20, d)) for _ in range(2))
    out = OP.packed_attention(q, k, v, off, 3, 1, 0.4, g)
    for b, n in enumerate(lens):
        cut = lambda x: x[None, :, off[b] : off[b] + n]
        one = OB.window_attention(cut(q), cut(k), cut(v), 3, 1, 0.4, dO=cut(g))
        for name in ("o", "dq", "dk", "dv", "lse"):
            assert np.array_equal(cut(out[name]), one[name])
    assert (out["dk"][:, :2] == 0).all() and (out["o"][:, 17:] == 0).all()
    table = np.array([[3, 1], [0, 0], [2, 5], [4, -1]])
    pool = [np.zeros((6, Hk, page, d)) for _ in range(2)]
    slots = [int(table[b][i // page]) * page + i % page for b, n in enumerate(lens) for i in range(n)]
    pool = [OP.page_write(x[:, 2:17], p, slots) for x, p in zip((k, v), pool)]
    paged = OP.paged_attention(q, *pool, table, off, lens, 3, 1, 0.4)
    assert np.array_equal(paged["o"], out["o"]) and np.array_equal(paged["lse"], out["lse"])


# ------------------------------------------------------------------ refusals of the C ABI
def _st(b=1 << 20, h=64, l=256):
    return R(lact.Strides(b, h, l))


def _packed(**kw):
    base = dict(batch=3, heads=4, kv_heads=2, d=64, io_dtype=lact.DTYPE_BF16, scale=0.125, tokens=200, longest=100,
                window=16, sinks=4, flags=0)
    base.update(kw)
    return lact.Packed(**base)


def _paged(**kw):
    base = dict(batch=3, heads=4, kv_heads=2, d=64, io_dtype=lact.DTYPE_BF16, scale=0.125, tokens=200, longest=100,
                k_len=500, window=16, sinks=4, pages=50, page=16, width=40, flags=0)
    base.update(kw)
    return lact.Paged(**base)


def _fwd(p, offsets=FAKE * 20, lse=None, **over):
    a = {n: (FAKE * i, _st()) for i, n in enumerate(("q", "k", "v", "o"), 1)}
    a.update(over)
    return lact.lib().lact_packed_attention_forward(None if p is None else R(p), *a["q"], *a["k"], *a["v"], offsets,
                                                    *a["o"], lse, None)


def _bwd(p, offsets=FAKE * 20, lse=FAKE * 21, ws=FAKE * 22, n=1 << 40, **over):
    a = {n: (FAKE * i, _st()) for i, n in enumerate(("q", "k", "v", "o", "dO", "dq", "dk", "dv"), 1)}
    a.update(over)
    return lact.lib().lact_packed_attention_backward(
        None if p is None else R(p), *a["q"], *a["k"], *a["v"], offsets, *a["o"], lse, *a["dO"], *a["dq"], *a["dk"],
        *a["dv"], ws, n, None)


def _pgd(p, offsets=FAKE * 20, k_lens=FAKE * 21, table=FAKE * 22, lse=None, ws=FAKE * 23, n=1 << 40, **over):
    a = {n: (FAKE * i, _st()) for i, n in enumerate(("q", "k", "v", "o"), 1)}
    a["k"] = (FAKE * 2, _st(16 * 256))
    a["v"] = (FAKE * 3, _st(16 * 256))
    a.update(over)
    return lact.lib().lact_paged_attention(None if p is None else R(p), *a["q"], *a["k"], *a["v"], offsets, k_lens,
                                           table, *a["o"], lse, ws, n, None)


BAD = [(dict(batch=-1), I), (dict(batch=(1 << 24) + 1), U), (dict(heads=0), I), (dict(kv_heads=0), I),
       (dict(heads=3), I), (dict(d=0), U), (dict(d=12), U), (dict(d=136), U), (dict(io_dtype=2), I),
       (dict(scale=0.0), I), (dict(scale=float("nan")), I), (dict(tokens=-1), I), (dict(tokens=1 << 30), I),
       (dict(longest=-1), I), (dict(longest=201), I), (dict(window=-1), I), (dict(sinks=-1), I), (dict(flags=2), I)]


@pytest.mark.parametrize("kw,code", BAD)
def test_bad_problems_are_refused(kw, code):
    p, g = _packed(**kw), _paged(**kw)
    assert _fwd(p) == code and lact.last_error()
    assert _bwd(p) == code and _pgd(g) == code and lact.last_error()
    assert lact.lib().lact_packed_attention_backward_workspace_size(R(p)) == 0
    assert lact.lib().lact_paged_attention_workspace_size(R(g)) == 0


@pytest.mark.parametrize("kw,code", [(dict(page=0), U), (dict(page=12), U), (dict(page=-8), U), (dict(page=65544), U),
                                     (dict(pages=-1), I), (dict(pages=1 << 27), I), (dict(width=-1), I),
                                     (dict(width=1 << 26), I), (dict(k_len=-1), I), (dict(k_len=641), I)])
def test_bad_pages_are_refused(kw, code):
    assert _pgd(_paged(**kw)) == code and lact.last_error()


def test_bad_tensors_are_refused():
    assert _fwd(None) == I and _bwd(None) == I and _pgd(None) == I
    for call, p in ((_fwd, _packed()), (_pgd, _paged())):
        for n in ("q", "k", "v", "o"):
            assert call(p, **{n: (None, _st())}) == I and call(p, **{n: (FAKE * 9, None)}) == I
            assert call(p, **{n: (FAKE * 9 + 8, _st())}) == I
            assert call(p, **{n: (FAKE * 9, _st(l=260))}) == I and call(p, **{n: (FAKE * 9, _st(h=-64))}) == I
        assert call(p, o=(FAKE * 9, _st(l=64))) == I and "overlap" in lact.last_error()
        assert call(p, offsets=None) == I and call(p, offsets=FAKE + 4) == I and call(p, lse=FAKE + 2) == I
        for n in ("q", "k", "v"):
            assert call(p, **{n: (FAKE * 9, _st(4096)), "o": (FAKE * 9, _st())}) == I and "output" in lact.last_error()
        assert call(p, offsets=FAKE * 4) == I
    assert _pgd(_paged(), k_lens=None) == I and _pgd(_paged(), k_lens=FAKE + 4) == I
    assert _pgd(_paged(), table=None) == I and _pgd(_paged(), table=FAKE + 2) == I
    for n in ("k_lens", "table"):
        assert _pgd(_paged(), **{n: FAKE * 4}) == I and "output" in lact.last_error()
    far = R(lact.Strides(1 << 40, 64, (1 << 26) + 8))   # elements of two bytes
    assert _pgd(_paged(), k=(FAKE * 9, far)) == U and _pgd(_paged(), v=(FAKE * 9, far)) == U
    for n in ("dO", "dq", "dk", "dv"):
        assert _bwd(_packed(), **{n: (None, _st())}) == I and n in lact.last_error()
    assert _bwd(_packed(), lse=None) == I
    assert _bwd(_packed(), dk=(FAKE * 6, _st())) == I and _bwd(_packed(), dv=(FAKE * 4, _st())) == I
    assert _bwd(_packed(), dk=(FAKE * 9, _st(h=0))) == I and "overlap" in lact.last_error()


def test_workspaces_are_checked():
    p = _packed()
    need = lact.lib().lact_packed_attention_backward_workspace_size(R(p))
    assert need >= 2 * 4 * 200 * 4
    assert _bwd(p, n=need - 1) == lact.ERR_WORKSPACE_TOO_SMALL
    assert _bwd(p, ws=None) == I and _bwd(p, ws=FAKE + 16) == I
    g = _paged(batch=1, tokens=1, longest=1, k_len=32768, width=2048, window=0)   # one row, keys split
    need = lact.lib().lact_paged_attention_workspace_size(R(g))
    assert need > 0
    assert _pgd(g, n=need - 1) == lact.ERR_WORKSPACE_TOO_SMALL and _pgd(g, ws=None) == I
    s = _slots(batch=5000)
    need = lact.lib().lact_page_slots_workspace_size(R(s))
    assert need >= 4 * 5000 and _slt(s, n=need - 1) == lact.ERR_WORKSPACE_TOO_SMALL and _slt(s, ws=None) == I


@pytest.mark.parametrize("kw", [dict(), dict(batch=1 << 20), dict(longest=1), dict(batch=1, longest=20000, tokens=20000),
                                dict(sinks=1 << 40), dict(sinks=4096, window=1), dict(io_dtype=0, d=128)])
def test_workspace_of_the_backward_is_bounded(kw):
    """Two statistics a row and head, and what the padded form allows sink tiles."""
    a = dict(batch=8, heads=8, kv_heads=8, d=128, tokens=32768, longest=32768, window=128, sinks=4)
    a.update(kw)
    need = lact.lib().lact_packed_attention_backward_workspace_size(R(_packed(**a)))
    stats = 8 * a["heads"] * a["tokens"] + 256
    assert stats - 512 <= need <= stats + 768 * 2 * 128 * 128 * 4 + 256


def _paged_ws(**kw):
    a = dict(heads=32, kv_heads=8, d=128, k_len=32768, pages=1 << 15, page=128, width=256, window=0)
    a.update(kw)
    return lact.lib().lact_paged_attention_workspace_size(R(_paged(**a)))


def test_workspace_of_paged_attention():
    """Few rows: two parts a wave, of at most 2048 waves and 32 rows; a chunk
    that fills half the chip: parts of its rows; no more, whatever the batch."""
    part = 130 * 4   # a row's result and two statistics
    for kw, rows in ((dict(batch=1, tokens=1, longest=1), 4), (dict(batch=96, tokens=96, longest=1), 4),
                     (dict(batch=300, tokens=2400, longest=8), 32), (dict(batch=1 << 20, tokens=1 << 20, longest=1), 4)):
        need = _paged_ws(**kw)
        assert 512 * part < need <= 2048 * 2 * rows * part + 8 * (kw["batch"] + 1) + 1024, kw
    assert _paged_ws(batch=1, tokens=256, longest=256) >= 2 * 256 * 32 * part
    assert _paged_ws(batch=1, tokens=4096, longest=4096) == 0
    assert _paged_ws(batch=0, tokens=1, longest=1) == 0 and _paged_ws(batch=4, tokens=64, longest=0) == 0


def test_grids_beyond_a_launch_are_refused():
    big = dict(tokens=(1 << 30) - 1, longest=(1 << 30) - 1, heads=128, kv_heads=128, d=8)
    st = _st(1 << 40, 8, 1024)
    assert _fwd(_packed(**big), q=(FAKE, st), k=(FAKE * 2, st), v=(FAKE * 3, st), o=(FAKE * 4, st)) == U
    assert "launch" in lact.last_error()
    huge = dict(batch=1 << 24, heads=64, kv_heads=64, d=8, tokens=1 << 24, longest=99)
    st = _st(1 << 40, 8, 512)
    assert _pgd(_paged(**huge), q=(FAKE, st), o=(FAKE * 4, st), k=(FAKE * 2, _st(1 << 20, 8, 512)),
                v=(FAKE * 3, _st(1 << 20, 8, 512))) == U and "launch" in lact.last_error()


def _slots(**kw):
    base = dict(batch=3, page=16, width=10, entries=50, tokens=100)
    base.update(kw)
    return lact.Slots(**base)


SLOT_ARGS = ("lens", "counts", "table", "free", "have", "offsets", "k_lens", "slots", "positions", "left")


def _slt(p, ws=FAKE * 23, n=1 << 40, **over):
    a = {x: FAKE * i for i, x in enumerate(SLOT_ARGS, 1)}
    a.update(over)
    return lact.lib().lact_page_slots(None if p is None else R(p), *[a[x] for x in SLOT_ARGS], ws, n, None)


@pytest.mark.parametrize("kw,code", [(dict(batch=-1), I), (dict(batch=(1 << 24) + 1), I), (dict(page=0), U),
                                     (dict(page=20), U), (dict(width=-1), I), (dict(width=1 << 26), I),
                                     (dict(entries=-1), I), (dict(entries=1 << 28), I), (dict(tokens=-1), I), (dict(tokens=1 << 30), I)])
def test_slots_refuse_bad_problems(kw, code):
    assert _slt(_slots(**kw)) == code and lact.last_error()
    assert lact.lib().lact_page_slots_workspace_size(R(_slots(**kw))) == 0


def test_slots_refuse_bad_arrays():
    assert _slt(None) == I
    for x in SLOT_ARGS:
        assert _slt(_slots(), **{x: None}) == I, x
        assert _slt(_slots(), **{x: FAKE * 30 + 2}) == I, x
    outs = ("table",) + SLOT_ARGS[5:]
    for o in outs:
        for i in ("lens", "counts", "free"):
            assert _slt(_slots(), **{o: FAKE * 30, i: FAKE * 30}) == I and "output" in lact.last_error()
        if o != "left":
            assert _slt(_slots(), **{o: FAKE * 30, "have": FAKE * 30}) == I
        for x in outs:
            assert x == o or _slt(_slots(), **{o: FAKE * 30, x: FAKE * 30}) == I


def _write(**kw):
    base = dict(kv_heads=4, d=64, io_dtype=lact.DTYPE_BF16, pages=10, page=16, tokens=30)
    base.update(kw)
    return lact.Write(**base)


def _wrt(p, slots=FAKE * 9, **over):
    a = {n: (FAKE * i, _st(16 * 256)) for i, n in enumerate(("k", "v", "kp", "vp"), 1)}
    a.update(over)
    return lact.lib().lact_page_write(None if p is None else R(p), *a["k"], *a["v"], slots, *a["kp"], *a["vp"], None)


@pytest.mark.parametrize("kw,code", [(dict(kv_heads=0), I), (dict(kv_heads=65537), I), (dict(d=0), U), (dict(d=12), U),
                                     (dict(d=8200), U), (dict(io_dtype=7), I), (dict(pages=-1), I),
                                     (dict(pages=1 << 27), I), (dict(page=10), U), (dict(tokens=-1), I),
                                     (dict(tokens=1 << 30), I)])
def test_writes_refuse_bad_problems(kw, code):
    assert _wrt(_write(**kw)) == code and lact.last_error()


def test_writes_refuse_bad_tensors():
    assert _wrt(None) == I and _wrt(_write(), slots=None) == I and _wrt(_write(), slots=FAKE + 4) == I
    for n in ("k", "v", "kp", "vp"):
        assert _wrt(_write(), **{n: (None, _st())}) == I and _wrt(_write(), **{n: (FAKE * 20, None)}) == I
        assert _wrt(_write(), **{n: (FAKE * 20 + 8, _st())}) == I and _wrt(_write(), **{n: (FAKE * 20, _st(l=-256))}) == I
    for n in ("kp", "vp"):
        assert _wrt(_write(), **{n: (FAKE * 20, _st(16 * 256, 64, 64))}) == I and "overlap" in lact.last_error()
        for x in ("k", "v"):
            assert _wrt(_write(), **{n: (FAKE * 20, _st(16 * 256)), x: (FAKE * 20, _st())}) == I
    assert _wrt(_write(), vp=(FAKE * 3, _st(16 * 256))) == I and "same" in lact.last_error()


def test_nothing_to_do_is_accepted():
    none = {n: (None, None) for n in ("q", "k", "v", "o")}
    assert _fwd(_packed(tokens=0, longest=0), offsets=None, **none) == lact.OK
    assert _bwd(_packed(tokens=0, longest=0), offsets=None, lse=None, ws=None, n=0, dO=(None, None), dq=(None, None),
                dk=(None, None), dv=(None, None), **none) == lact.OK
    assert _pgd(_paged(tokens=0, longest=0), offsets=None, k_lens=None, table=None, ws=None, n=0, **none) == lact.OK
    none = {n: (None, None) for n in ("k", "v", "kp", "vp")}
    assert _wrt(_write(tokens=0), slots=None, **none) == lact.OK and _wrt(_write(pages=0), slots=None, **none) == lact.OK


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_host_tensors_shapes_and_numbers():
    q, off = torch.zeros(2, 4, 64), torch.tensor([0, 4])
    pool, n = torch.zeros(3, 2, 8, 64), torch.tensor([4])
    table = torch.zeros(1, 2, dtype=torch.int32)
    paged = lambda **kw: lact.paged_attention(q, pool, pool, **dict(dict(table=table, offsets=off, k_lens=n), **kw))
    for call in (lambda: lact.packed_attention(q, q, q, offsets=off), lambda: paged(),
                 lambda: lact.packed_attention_backward(q, q, q, q, q[..., 0], dO=q, offsets=off),
                 lambda: lact.page_write(q, q, pool, pool, slots=torch.zeros(4, dtype=torch.int64)),
                 lambda: lact.page_slots(n, n, table, table[0], n, page=8, tokens=4),
                 lambda: lact.packed_attention(q[0], q, q, offsets=off), lambda: lact.packed_attention(q, q[0], q, offsets=off)):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(window=(1 << 64) + 5), dict(sinks=1 << 64), dict(longest=1 << 64), dict(window=2.5), dict(longest="3")):
        with pytest.raises(ValueError):
            lact.packed_attention(q, q, q, offsets=off, **kw)
        with pytest.raises(ValueError):
            paged(**kw)
    with pytest.raises(ValueError):
        paged(k_len=1.5)
    for kw in (dict(page=8.5, tokens=4), dict(page=8, tokens=-1), dict(page=8, tokens=1 << 64)):
        with pytest.raises(ValueError):
            lact.page_slots(n, n, table, table[0], n, **kw)
    for name in ("batch", "heads", "kv_heads", "d", "pages", "page", "width"):
        a = dict(batch=1, heads=2, kv_heads=1, d=64, io_dtype=0, scale=0.125, tokens=4, longest=4, k_len=4, window=0,
                 sinks=0, pages=3, page=8, width=2, flags=0)
        with pytest.raises(ValueError, match=name):
            lact._struct(lact.Paged, *dict(a, **{name: (1 << 32) + 8}).values())
