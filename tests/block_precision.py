"""How far fp32 attention may be off its fp64 oracle, derived from its sums.

With u = 2^-24, S the largest scale sum_i |q_i k_i| among what a row sees, n
the keys that a row sees, m the rows (over all query heads of its key head)
that see a key:

- a score is a sum of d products: d u S; the factor scale log2(e) is rounded
  twice and the exponent once, 3 u S and, relative to a maximum that lags by up
  to 24, 24 ln 2 u < 17 u; the exponential is off by a unit in the last place,
  2 u, and so are the few factors of rescaling.  A probability's numerator is
  off by the relative e = u ((d + 5) S + 40), the other terms of its row by as
  much again through the sum that divides it;
- a sum of n terms is off by n u of their magnitudes: o by (2 e + 2 n u + 8 u)
  sum P |v|, and u |o|; lse by e + n u + 2 u |lse|;
- P in the backward is exp(s - lse), off by w = 2 e + 2 u (|lse| + n) + 8 u.
  dP = dO . v and D = dO . o are sums of d products, off by (d + 2) u of their
  magnitudes, and D has the error of o.  dS = P (dP - D) is off by
      w P |dP - D| + P ((d + 4) u (|dO| . |v| + |dO| . |o|) + |dO| . (error of o)),
  and dq, dk, dv are sums of n and m terms of these.

The bounds hold for every element.  Roundings are as good as independent,
though, and the operands here of random sign, so that what they amount to adds
up in squares: a sum of d products is off by sqrt(d) u times the root of the
sum of their squares, sums over keys and rows likewise, while what is common to
a row (its sum's error, D's) moves o and dq by its share of these results
themselves and of sum P k.  The root mean square of a result's error stays
below that of these sizes: `expected`.
"""
import numpy as np

from oracle import lact_block as OB

U = 2.0 ** -24


def _sequences(q, k, q_lens, k_lens):
    for b in range(q.shape[0]):
        ql = q.shape[2] if q_lens is None else int(q_lens[b])
        kl = k.shape[2] if k_lens is None else int(k_lens[b])
        for h in range(q.shape[1] if ql and kl else 0):
            yield b, h, h // (q.shape[1] // k.shape[1]), ql, kl


def _softmax(s, see):
    some = see.any(1, keepdims=True)
    s = np.where(see, s, -np.inf)
    p = np.exp(s - np.where(some, s.max(1, keepdims=True), 0.0))
    return p / np.where(some, p.sum(1, keepdims=True), 1.0)


def bounds(q, k, v, g, window, sinks, scale, q_lens, k_lens, ref):
    """({name: bound of every element}, {name: its expected size}) for o, lse,
    dq, dk, dv, with ref the oracle's results."""
    G, d = q.shape[1] // k.shape[1], float(q.shape[3])
    worst, expected = ({n: np.zeros(ref[n].shape) for n in ("o", "lse", "dq", "dk", "dv")} for _ in range(2))
    for b, h, hk, ql, kl in _sequences(q, k, q_lens, k_lens):
        see = OB.visible(ql, kl, window, sinks)
        qq, kk, vv, gg = q[b, h, :ql], k[b, hk, :kl], v[b, hk, :kl], g[b, h, :ql]
        o, dq = np.abs(ref["o"][b, h, :ql]), np.abs(ref["dq"][b, h, :ql])
        n, m = see.sum(1)[:, None], G * see.sum(0)[:, None]
        lse = np.abs(np.where(np.isfinite(ref["lse"][b, h, :ql]), ref["lse"][b, h, :ql], 0.0))[:, None]
        p = _softmax(scale * qq @ kk.T, see)
        ds = p * np.abs(gg @ vv.T - (gg * ref["o"][b, h, :ql]).sum(1, keepdims=True))
        # every element: sums of magnitudes
        qq, kk, vv, gg = np.abs(qq), np.abs(kk), np.abs(vv), np.abs(gg)
        e = U * ((d + 5) * np.where(see, scale * qq @ kk.T, 0.0).max(1, keepdims=True) + 40)
        worst["lse"][b, h, :ql] = (e + n * U + 2 * U * lse + 2.0 ** -149)[:, 0]
        eo = (2 * e + 2 * n * U + 8 * U) * (p @ vv) + U * o
        worst["o"][b, h, :ql] = eo + 2.0 ** -149
        w = 2 * e + 2 * U * (lse + n) + 8 * U
        eds = w * ds + p * ((d + 4) * U * (gg @ vv.T + (gg * o).sum(1, keepdims=True)) + (gg * eo).sum(1, keepdims=True))
        worst["dq"][b, h, :ql] = scale * ((eds + n * U * ds) @ kk) + 4 * U * dq + 2.0 ** -140
        worst["dk"][b, hk, :kl] += scale * ((eds.T + m * U * ds.T) @ qq)
        worst["dv"][b, hk, :kl] += ((w * p).T + m * U * p.T) @ gg
        # expected: in squares
        root = lambda x: np.sqrt(np.maximum(x, 0.0))
        q2, k2, v2, g2, n, m = qq ** 2, kk ** 2, vv ** 2, gg ** 2, root(n), root(m)
        e = U * (root(d + 5) * root(np.where(see, scale ** 2 * q2 @ k2.T, 0.0).max(1, keepdims=True)) + 40)
        expected["lse"][b, h, :ql] = (e + n * U + 2 * U * lse + 2.0 ** -149)[:, 0]
        eo = e * (root(p ** 2 @ v2) + o) + (2 * n + 8) * U * root(p ** 2 @ v2) + U * o
        expected["o"][b, h, :ql] = eo + 2.0 ** -149
        common = e + 2 * U * (lse + n) + 8 * U
        eD = root(d) * U * root((g2 * o ** 2).sum(1, keepdims=True)) + root((g2 * eo ** 2).sum(1, keepdims=True))
        edp = root(d + 4) * U * root(g2 @ v2.T)
        own = e * ds + p * edp
        expected["dq"][b, h, :ql] = (scale * root((own + n * U * ds) ** 2 @ k2) + (common + 4 * U) * dq +
                                     scale * eD * np.abs(p @ k[b, hk, :kl]) + 2.0 ** -140)
        all_ = own + common * ds + p * eD
        # squares, of which the roots are taken behind the last head
        expected["dk"][b, hk, :kl] += scale ** 2 * ((all_.T + m * U * ds.T) ** 2 @ q2)
        expected["dv"][b, hk, :kl] += (((e + common) * p).T + m * U * p.T) ** 2 @ g2
    for name in ("dk", "dv"):
        worst[name] += 4 * U * np.abs(ref[name]) + 2.0 ** -140
        expected[name] = np.sqrt(expected[name]) + 4 * U * np.abs(ref[name]) + 2.0 ** -140
    return worst, expected


def excess(out, ref, limits):
    """The largest ratio of an element's error to its bound, and that of the
    root mean square, by name."""
    single, rms = {}, {}
    for name, x in out.items():
        live = np.isfinite(ref[name])
        assert (x[~live] == ref[name][~live]).all(), name
        if live.any():
            off = np.abs(np.where(live, x, 0.0) - np.where(live, ref[name], 0.0))[live]
            worst, mean = (t[name][live] for t in limits)
            assert (off[worst == 0] == 0).all(), name
            single[name] = float((off / (worst + 1e-300)).max())
            rms[name] = float(np.sqrt((off ** 2).mean() / ((mean ** 2).mean() + 1e-300)))
    return single, rms


def rounded(x, bits):
    """x to `bits` significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(m, bits)), e - bits)


def attention(q, k, v, g, window, sinks, scale, q_lens, k_lens, operand=lambda x: x, weight=lambda x: x):
    """Attention and its gradients in fp64 with the scores' operands, or the
    probabilities and dS, rounded: what a lesser path computes."""
    out = {n: np.zeros(x.shape) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    for b, h, hk, ql, kl in _sequences(q, k, q_lens, k_lens):
        qq, kk, vv, gg = q[b, h, :ql], k[b, hk, :kl], v[b, hk, :kl], g[b, h, :ql]
        p = _softmax(scale * operand(qq) @ operand(kk).T, OB.visible(ql, kl, window, sinks))
        o = weight(p) @ vv
        ds = weight(p * (gg @ vv.T - (gg * o).sum(1, keepdims=True)))
        out["o"][b, h, :ql], out["dq"][b, h, :ql] = o, scale * ds @ kk
        out["dk"][b, hk, :kl] += scale * ds.T @ qq
        out["dv"][b, hk, :kl] += weight(p).T @ gg
    return out
