"""fp32 attention on the GPU against its derived bounds (block_precision): no
element beyond its bound, and the root mean square of a result's error within
the size that independent roundings give it, which a path with operands or
probabilities of fewer bits exceeds (test_block_cpu_edges)."""
import numpy as np
import pytest

import block_precision as BP
from oracle import lact_block as OB
from test_gpu_block import ATTENTION, f64, randn

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "x".join(str(x) for x in c[:8]))
def test_fp32_attention(case):
    from test_layers_amd import lact
    B, H, Hk, d, Lq, Lk, window, sinks, ql, kl = case
    gen = torch.Generator("cuda").manual_seed(sum(case[:8]))
    q, k, v, g = (randn(gen, s, torch.float32) for s in ((B, H, Lq, d), (B, Hk, Lk, d), (B, Hk, Lk, d), (B, H, Lq, d)))
    lens = lambda x: None if x is None else torch.tensor(x, dtype=torch.int64, device="cuda")
    kw = dict(window=window, sinks=sinks, scale=0.3, q_lens=lens(ql), k_lens=lens(kl))
    print("attention", case, flush=True)
    out = {}
    out["o"], out["lse"] = lact.window_attention(q, k, v, return_lse=True, **kw)
    torch.cuda.synchronize()
    out.update(lact.window_attention_backward(q, k, v, out["o"], out["lse"], dO=g, **kw))
    scale = float(np.float32(0.3))
    ref = OB.window_attention(f64(q), f64(k), f64(v), window, sinks, scale, ql, kl, f64(g))
    limits = BP.bounds(f64(q), f64(k), f64(v), f64(g), window, sinks, scale, ql, kl, ref)
    single, rms = BP.excess({n: f64(x) for n, x in out.items()}, ref, limits)
    print({n: "%.3f" % x for n, x in single.items()}, {n: "%.3f" % x for n, x in rms.items()}, flush=True)
    assert max([0, *single.values()]) <= 1, single
    assert max([0, *rms.values()]) <= 1, rms
