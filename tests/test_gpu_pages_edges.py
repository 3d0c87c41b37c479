"""Packed and paged attention where one call leaves the usual: rows that a bound
leaves out, in numbers."""
import time

import numpy as np
import pytest

from test_gpu_pages import _cache, rows, sums, whole

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
