"""fp64 numpy oracle of the operators around the fast-weight layer: window
attention with sinks (forward, backward), rotary positions, and the residual's
addition with the root-mean-square norm.  Written from the definitions, one
head at a time; shares no code with the HIP library.

The attention functions also return what a rounding of the probabilities, of
their gradients or of o can move each result by (keys ending in "_abs"): the
same sums over magnitudes, from which a caller derives its tolerance.
"""
import numpy as np


def visible(q_len, k_len, window, sinks):
    """[q_len, k_len] mask: row r stands at p = k_len - q_len + r and sees
    j <= p among the last `window` (0: all) or the first `sinks` keys."""
    p = (k_len - q_len + np.arange(q_len))[:, None]
    j = np.arange(k_len)[None, :]
    near = np.ones((q_len, k_len), bool) if window == 0 else j > p - window
    return (j <= p) & (near | (j < sinks))


def _softmax(s, see):
    s = np.where(see, s, -np.inf)
    top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    z = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, np.where(np.isfinite(top), top, 0.0) + np.log(z), -np.inf)
    return e / np.where(z > 0, z, 1.0), lse[:, 0]


def window_attention(q, k, v, window, sinks, scale, q_lens=None, k_lens=None, dO=None):
    """q [B, H, Lq, d], k, v [B, Hk, Lk, d] (fp64).  Returns a dict: o, lse and,
    with dO, dq, dk, dv.  Places behind the lengths are zero."""
    B, H, Lq, d = q.shape
    G = H // k.shape[1]
    out = {"o": np.zeros(q.shape), "o_abs": np.zeros(q.shape), "lse": np.zeros((B, H, Lq))}
    # the largest scale * sum |q||k| of a visible pair: what a score's rounding is relative to
    out["score_abs"] = 0.0
    if dO is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            out[n], out[n + "_abs"], out[n + "_delta"] = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    for b in range(B):
        ql = Lq if q_lens is None else int(q_lens[b])
        kl = k.shape[2] if k_lens is None else int(k_lens[b])
        see = visible(ql, kl, window, sinks)
        for h in range(H):
            qq, kk, vv = q[b, h, :ql], k[b, h // G, :kl], v[b, h // G, :kl]
            if ql == 0:
                continue
            p, lse = _softmax(scale * qq @ kk.T, see)
            o = p @ vv
            out["o"][b, h, :ql], out["lse"][b, h, :ql] = o, lse
            oa = out["o_abs"][b, h, :ql] = p @ np.abs(vv)
            if see.any():
                out["score_abs"] = max(out["score_abs"], float((scale * np.abs(qq) @ np.abs(kk).T)[see].max()))
            if dO is None:
                continue
            g = dO[b, h, :ql]
            dp = g @ vv.T
            delta = (g * o).sum(1, keepdims=True)
            ds = p * (dp - delta)
            dsa = p * (np.abs(g) @ np.abs(vv).T + np.abs(g * o).sum(1, keepdims=True))
            # the rounding of o enters delta: at most |dO| (|o| + o_abs) half steps
            de = p * (np.abs(g) * (np.abs(o) + oa)).sum(1, keepdims=True)
            out["dq"][b, h, :ql] = scale * ds @ kk
            out["dk"][b, h // G, :kl] += scale * ds.T @ qq
            out["dv"][b, h // G, :kl] += p.T @ g
            out["dq_abs"][b, h, :ql] = scale * dsa @ np.abs(kk)
            out["dk_abs"][b, h // G, :kl] += scale * dsa.T @ np.abs(qq)
            out["dv_abs"][b, h // G, :kl] += p.T @ np.abs(g)
            out["dq_delta"][b, h, :ql] = scale * de @ np.abs(kk)
            out["dk_delta"][b, h // G, :kl] += scale * de.T @ np.abs(qq)
    return out


def rotary(x, positions, freqs, interleaved=False, mscale=1.0, inverse=False):
    """x [B, H, L, d], positions [B, L], freqs [pairs]; all fp64."""
    n = len(freqs)
    y = x.copy()
    a = positions[:, None, :, None].astype(np.float64) * freqs * (-1.0 if inverse else 1.0)
    c, s = mscale * np.cos(a), mscale * np.sin(a)
    i, j = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def frequencies(pairs, base, scaling="plain", factor=1.0, context=0, slow=1.0, fast=32.0):
    if scaling == "ntk" and pairs > 1:
        base = base * factor ** (pairs / (pairs - 1.0))
    f = base ** (-np.arange(pairs) / max(pairs, 1.0))
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        keep = np.clip((context * f / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    return f


def add_rmsnorm(x, weight, residual=None, eps=1e-6):
    h = x if residual is None else x + residual
    return h * weight / np.sqrt((h * h).mean(-1, keepdims=True) + eps), h


def quantise(y, group=128):
    """(y / scale, scale): one scale for each `group` columns, not yet rounded to 8 bits."""
    cols = y.shape[-1]
    g = -(-cols // group)
    pad = np.zeros(y.shape[:-1] + (g * group,))
    pad[..., :cols] = y
    s = np.maximum(np.abs(pad.reshape(y.shape[:-1] + (g, group))).max(-1), 2.0 ** -100) / 448.0
    return y / np.repeat(s, group, axis=-1)[..., :cols], s


def add_rmsnorm_backward(h, weight, dy, dh=None, eps=1e-6):
    f = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = dy * weight
    dx = f * (g - h * f * f * (g * h).mean(-1, keepdims=True))
    dw = (dy * h * f).reshape(-1, h.shape[-1]).sum(0)
    return dx + (0.0 if dh is None else dh), dw
