"""The operators of a block around the fast-weight layer, as measured work.

A large-chunk block runs window attention beside the fast-weight layer, turns
the positions of q and k into rotations, and normalises the residual stream in
front of both.  This file lists those operators' cases at real sizes, makes
their inputs, and states each operator twice: in elementary torch operations
(`run` with `own` false) and in 64 bits from the definition (`exact`).  With
`own` true `run` makes the calls of test_layers_amd.lact.

Window attention.  Row r of sequence b stands at position
p = k_len[b] - q_len[b] + r and sees the keys j <= p, j < k_len[b] that are
among its last `window` (j > p - window) or among the first `sinks`.
  s_j = scale q . k_j,  lse = log sum_j exp s_j,  o = sum_j exp(s_j - lse) v_j,
a row that sees nothing gives o = 0 and lse = -inf; rows behind q_len[b] are
not written (zero here).  Gradients: with P = exp(s - lse), D = dO . o,
  dv_j = sum_r P dO,  dS = P (dO . v_j - D),
  dq = scale sum_j dS k_j,  dk_j = scale sum_r dS q,
summed over the query heads that share a key head.

Rotary positions.  Pair i of the first 2 n features, (x_i, x_{i+n}) in the
half layout or (x_{2i}, x_{2i+1}) interleaved, turns by the angle
position * freq_i and is scaled by mscale; the other features pass through.
The backward turns the other way.

Add and norm.  h = x + residual, y = h w / sqrt(mean(h^2) + eps); h is
returned rounded to its type.  The 8-bit output holds y / s in e4m3 with
s = max(amax, 2^-100) / 448 for each row's groups of 128 columns.  Backward
from the stored h, g = w dy, xh = h / rms:
  dx = (g - xh mean(g xh)) / rms + dh,  dw = sum_rows dy xh.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    att = dict(op="attention", ragged=False, sinks=4, layout="tokens")
    rot = dict(op="rotary", mscale=1.0, scaled=False)
    nrm = dict(op="norm")
    return [
        # one user's next token: the smallest call, all latency
        dict(att, name="decode_one", mode="decode", type="bf16", batch=1, heads=16, kv_heads=16, d=64, q_len=1,
             k_len=32768, window=2048),
        # a serving batch's next tokens, four query heads to a cache head, sequences of every length
        dict(att, name="decode_batch", mode="decode", type="bf16", batch=96, heads=32, kv_heads=8, d=128, q_len=1,
             k_len=8192, window=4096, ragged=True, layout="heads"),
        # reading a 32K prompt
        dict(att, name="prefill_32k", mode="forward", type="bf16", batch=1, heads=32, kv_heads=8, d=128, q_len=32768,
             k_len=32768, window=2048),
        # a training step at the 32K language-model length, window of one 2K chunk
        dict(att, name="train_32k", mode="train", type="bf16", batch=1, heads=16, kv_heads=16, d=64, q_len=32768,
             k_len=32768, window=2048),
        # a padded batch of short texts, odd sizes
        dict(att, name="train_ragged", mode="train", type="bf16", batch=5, heads=12, kv_heads=4, d=96, q_len=1777,
             k_len=1777, window=333, sinks=17, ragged=True, layout="heads"),
        # the fp32 path: the tiny language-model workload's length
        dict(att, name="train_fp32", mode="train", type="fp32", batch=2, heads=8, kv_heads=8, d=64, q_len=1024,
             k_len=1024, window=256),
        # positions of a decoding batch, far out
        dict(rot, name="rotary_decode", mode="forward", type="bf16", batch=64, heads=32, kv_heads=8, length=1, d=128,
             pairs=64, interleaved=False, start=500000, layout="heads", scaled=True, mscale=1.1386),
        # q and k of a training step's 32K tokens
        dict(rot, name="rotary_32k", mode="forward", type="bf16", batch=1, heads=32, kv_heads=8, length=32768, d=128,
             pairs=64, interleaved=False, start=0, layout="tokens"),
        # gradients through interleaved pairs on part of an odd head, fp32
        dict(rot, name="rotary_back_part", mode="backward", type="fp32", batch=3, heads=9, kv_heads=3, length=1531,
             d=90, pairs=21, interleaved=True, start=7, layout="heads"),
        # a decoding batch's norm ahead of an 8-bit projection
        dict(nrm, name="norm_decode_8bit", mode="quantised", type="bf16", rows=64, cols=2560),
        # a prompt's norm, 8-bit output
        dict(nrm, name="norm_prefill_8bit", mode="quantised", type="bf16", rows=32768, cols=4096),
        # a training step's norm, forward and backward, width not a power of two
        dict(nrm, name="norm_train", mode="train", type="bf16", rows=32768, cols=1536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rotary", "norm"])
    if op == "norm":
        mode = rng.choice(["forward", "quantised", "train"])
        cols = _log(rng, 64, 12288)
        if rng.random() < 0.7:
            cols = (cols + 7) // 8 * 8
        rows = _log(rng, 1, min(65536, (1 << 27) // cols))
        return dict(op=op, mode=mode, type=rng.choice(["bf16", "bf16", "fp32"]), rows=rows, cols=cols)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 8])
    layout = rng.choice(["tokens", "heads"])
    if op == "rotary":
        d = rng.choice([64, 80, 96, 128, 2 * rng.randint(8, 64)])
        pairs = d // 2 if rng.random() < 0.5 else rng.randint(1, d // 2)
        batch = _log(rng, 1, 64)
        length = _log(rng, 1, min(32768, max(1, (1 << 25) // (batch * heads * d))))
        scaled = rng.random() < 0.4
        return dict(op=op, mode=rng.choice(["forward", "backward"]), type=rng.choice(["bf16", "bf16", "fp32"]),
                    batch=batch, heads=heads, kv_heads=kv_heads, length=length, d=d, pairs=pairs,
                    interleaved=rng.random() < 0.5, start=_log(rng, 1, 1000000) - 1, layout=layout, scaled=scaled,
                    mscale=1.1386 if scaled else 1.0)
    mode = rng.choice(["decode", "forward", "train"])
    kind = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 64, 128, 8 * rng.randint(2, 16)])
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, 4, 16, rng.randint(0, 100)])
    if mode == "decode":
        batch, q_len = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 4, 5])
        k_len = max(q_len, _log(rng, 1, min(65536, (1 << 28) // (batch * kv_heads * d))))
    else:
        most = (1 << 31 if kind == "bf16" else 1 << 28) // (8 if mode == "train" else 1)
        q_len = _log(rng, 2, 16384)
        while q_len * heads * min(q_len, window + sinks) > most or q_len * heads * d > 1 << 26:
            q_len = (q_len + 1) // 2
        k_len = q_len if rng.random() < 0.8 else q_len + rng.randint(0, 2000)
        batch = max(1, min(_log(rng, 1, 6), most // (q_len * heads * min(k_len, window + sinks))))
    return dict(op=op, mode=mode, type=kind, batch=batch, heads=heads, kv_heads=kv_heads, d=d, q_len=q_len,
                k_len=k_len, window=window, sinks=sinks, ragged=batch > 1 and rng.random() < 0.5, layout=layout)


def _lens(case):
    """Key and query lengths of each sequence: full, or spread over a quarter to all of the padded length."""
    b, k, q = case["batch"], case["k_len"], case["q_len"]
    if not case["ragged"]:
        return [k] * b, [q] * b
    ks = [k - (3 * k // 4) * ((5 * i + 2) % b) // b for i in range(b)]
    if case["mode"] == "decode":
        return ks, [q] * b
    return ks, [min(q, x) for x in ks]


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _heads(gen, case, heads, length, dtype):
    """[batch, heads, length, d]: stored head by head, or as a view of token-major memory."""
    b, d = case["batch"], case["d"]
    if case["layout"] == "tokens":
        return _normal(gen, (b, length, heads, d), dtype).transpose(1, 2)
    return _normal(gen, (b, heads, length, d), dtype)


def _frequencies(case):
    """base^(-i / pairs), for a context stretched eight-fold with a ramp between kept and divided frequencies."""
    n, base = case["pairs"], 10000.0
    f = [base ** (-i / n) for i in range(n)]
    if case["scaled"]:
        turns = lambda x: x * 8192 / (2 * math.pi)  # turns within the original context
        ramp = lambda x: min(1.0, max(0.0, (turns(x) - 1.0) / 31.0))
        f = [x * ramp(x) + x / 8.0 * (1.0 - ramp(x)) for x in f]
    return f


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]
    s = dict(case)
    if case["op"] == "attention":
        d, mode = case["d"], case["mode"]
        q = _heads(gen, case, case["heads"], case["q_len"], t)
        k = _heads(gen, case, case["kv_heads"], case["k_len"], t)
        v = _heads(gen, case, case["kv_heads"], case["k_len"], t)
        # the first tokens draw attention from everywhere
        lean = _normal(gen, (d,), t)
        k[:, :, : case["sinks"]] += lean
        q += lean / 4
        s.update(q=q, k=k, v=v, scale=1.0 / math.sqrt(d), q_lens=None, k_lens=None)
        if case["ragged"]:
            ks, qs = _lens(case)
            s["k_lens"] = torch.tensor(ks, dtype=torch.int64, device="cuda")
            s["q_lens"] = None if mode == "decode" else torch.tensor(qs, dtype=torch.int64, device="cuda")
        if mode == "train":
            s["do"] = _heads(gen, case, case["heads"], case["q_len"], t)
    elif case["op"] == "rotary":
        s["q"] = _heads(gen, case, case["heads"], case["length"], t)
        s["k"] = _heads(gen, case, case["kv_heads"], case["length"], t)
        s["freqs"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        step = torch.arange(case["length"], device="cuda", dtype=torch.int64)
        jump = torch.randint(0, 1000, (case["batch"], 1), generator=gen, device="cuda", dtype=torch.int64)
        s["positions"] = case["start"] + jump + step
    else:
        shape = (case["rows"], case["cols"])
        s["x"], s["residual"] = _normal(gen, shape, t), _normal(gen, shape, t) * 3
        s["weight"] = 1 + 0.2 * _normal(gen, shape[1:], torch.float32)
        if case["mode"] == "train":
            s["dy"], s["dh"] = _normal(gen, shape, t), _normal(gen, shape, t)
    return s


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    from test_layers_amd import lact

    if s["op"] == "attention":
        kw = dict(window=s["window"], sinks=s["sinks"], scale=s["scale"], q_lens=s["q_lens"], k_lens=s["k_lens"])
        if s["mode"] != "train":
            return {"o": lact.window_attention(s["q"], s["k"], s["v"], **kw)}
        o, lse = lact.window_attention(s["q"], s["k"], s["v"], return_lse=True, **kw)
        g = lact.window_attention_backward(s["q"], s["k"], s["v"], o, lse, dO=s["do"], **kw)
        return {"o": o, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    if s["op"] == "rotary":
        call = lact.rotary_backward if s["mode"] == "backward" else lact.rotary
        return call(s["q"], s["k"], freqs=s["freqs"], positions=s["positions"], interleaved=s["interleaved"],
                    mscale=s["mscale"])
    if s["mode"] == "quantised":
        y8, scales, h = lact.add_rmsnorm_quantised(s["x"], s["weight"], s["residual"], eps=EPS)
        return {"y8": y8, "scales": scales, "h": h}
    y, h = lact.add_rmsnorm(s["x"], s["weight"], s["residual"], eps=EPS)
    if s["mode"] == "forward":
        return {"y": y, "h": h}
    dx, dw = lact.add_rmsnorm_backward(h, s["weight"], dy=s["dy"], dh=s["dh"], eps=EPS)
    return {"y": y, "h": h, "dx": dx, "dw": dw}


# ------------------------------------------------------------------ the plain forms

def _plain_attention(s):
    """All query blocks at once: each block meets the sinks and the one stretch of keys its rows can reach."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    b, h, lq, d = q.shape
    hk, lk = k.shape[1], k.shape[2]
    g = h // hk
    n, sinks, dev = min(s["window"], 2048, lq), min(s["sinks"], lk), q.device
    nb = (lq + n - 1) // n
    reach = min(s["window"], lk + lq) + n - 1  # keys that a block's window can touch
    whole = lambda x, to: torch.full((b,), to, dtype=torch.int64, device=dev) if x is None else x
    kl, ql = whole(s["k_lens"], lk), whole(s["q_lens"], lq)
    row = torch.arange(nb * n, device=dev).view(1, nb, n)
    pos = (kl - ql).view(b, 1, 1) + row
    live = row < ql.view(b, 1, 1)
    at = pos[:, :, :1] + n - reach + torch.arange(reach, device=dev)  # [b, nb, reach]
    first = torch.arange(sinks, device=dev).expand(b, nb, sinks)
    key = torch.cat([first, at], 2).unsqueeze(2)  # [b, nb, 1, sinks + reach]
    p = pos.unsqueeze(3)
    near = key > p - s["window"]
    near[..., :sinks] = ~near[..., :sinks]  # a sink within the window is met there
    see = near & (key >= 0) & (key <= p) & (key < kl.view(b, 1, 1, 1)) & live.unsqueeze(3)
    place = key.squeeze(2).clamp(0, lk - 1)
    spot = (torch.arange(b, device=dev).view(b, 1, 1) * lk + place).reshape(-1)

    def keys(x):  # [b, hk, lk, d] -> [b, hk, nb, keys, d]
        x = x.transpose(1, 2).reshape(b * lk, hk * d)[spot]
        return x.view(b, nb, -1, hk, d).permute(0, 3, 1, 2, 4).contiguous()

    def rows(x):  # [b, h, lq, d] -> [b, hk, nb, g n, d]
        x = torch.nn.functional.pad(x, (0, 0, 0, nb * n - lq))
        return x.view(b, hk, g, nb, n, d).transpose(2, 3).reshape(b, hk, nb, g * n, d)

    def unrows(x):
        return x.view(b, hk, nb, g, n, d).transpose(2, 3).reshape(b, h, nb * n, d)[:, :, :lq]

    see = see.unsqueeze(1).unsqueeze(3)  # [b, 1, nb, 1, n, keys]
    kk, vv, qq = keys(k), keys(v), rows(q)
    sc = (qq @ kk.transpose(-1, -2).contiguous() * s["scale"]).view(b, hk, nb, g, n, -1)
    sc = torch.where(see, sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(sc - top)
    z = e.sum(-1, keepdim=True)
    pr = (e / torch.where(z == 0, 1.0, z)).view(b, hk, nb, g * n, -1)
    o = pr @ vv
    out = {"o": unrows(o).to(s["q"].dtype)}
    if s["mode"] != "train":
        return out
    lse = (top + torch.log(z)).view(b, hk, nb, g, n).transpose(2, 3).reshape(b, h, nb * n)[:, :, :lq]
    seen = torch.arange(lq, device=dev).view(1, 1, lq) < ql.view(b, 1, 1)
    out["lse"] = torch.where(seen, lse, 0.0)
    do = rows(torch.where(seen.unsqueeze(3), s["do"].float(), 0.0))
    ds = pr * (do @ vv.transpose(-1, -2).contiguous() - (do * o).sum(-1, keepdim=True)) * s["scale"]

    def back(x):  # the sum of what each key got in every block that met it
        x = x.permute(0, 2, 3, 1, 4).reshape(-1, hk * d)
        x = torch.zeros(b * lk, hk * d, device=dev).index_add_(0, spot, x)
        return x.view(b, lk, hk, d).transpose(1, 2)

    out["dq"] = unrows(ds @ kk).to(s["q"].dtype)
    out["dk"] = back(ds.transpose(-1, -2).contiguous() @ qq).to(s["k"].dtype)
    out["dv"] = back(pr.transpose(-1, -2).contiguous() @ do).to(s["v"].dtype)
    return out


def _plain_rotary(s):
    angle = s["positions"].double().unsqueeze(-1) * s["freqs"]  # [b, l, pairs], in 64 bits: positions are far
    turn = -angle if s["mode"] == "backward" else angle
    c = (torch.cos(turn) * s["mscale"]).float().unsqueeze(1)
    z = (torch.sin(turn) * s["mscale"]).float().unsqueeze(1)
    n = s["pairs"]

    def one(x):
        y = x.float()
        if s["interleaved"]:
            a, b = y[..., 0 : 2 * n : 2], y[..., 1 : 2 * n : 2]
            r = torch.stack([a * c - b * z, a * z + b * c], -1).flatten(-2)
        else:
            a, b = y[..., :n], y[..., n : 2 * n]
            r = torch.cat([a * c - b * z, a * z + b * c], -1)
        return torch.cat([r, y[..., 2 * n :]], -1).to(x.dtype)

    return one(s["q"]), one(s["k"])


def _plain_norm(s):
    t = s["x"].dtype
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    out = {"h": h.to(t)}
    if s["mode"] == "quantised":
        rows, cols = y.shape
        g = torch.nn.functional.pad(y, (0, -cols % GROUP)).view(rows, -1, GROUP)
        sc = g.abs().amax(-1).clamp(min=2.0 ** -100) / 448.0
        out["y8"] = (g / sc.unsqueeze(-1)).reshape(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
        out["scales"] = sc
        return out
    out["y"] = y.to(t)
    if s["mode"] == "train":
        h = out["h"].float()
        r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        xh, dy = h * r, s["dy"].float()
        g = dy * s["weight"]
        out["dx"] = ((g - xh * (g * xh).mean(-1, keepdim=True)) * r + s["dh"].float()).to(t)
        out["dw"] = (dy * xh).sum(0)
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"] == "attention":
        return _plain_attention(state)
    return _plain_rotary(state) if state["op"] == "rotary" else _plain_norm(state)


# ------------------------------------------------------------------ work

def _pairs(case):
    """(visible pairs of one head, keys that some row sees) summed over the batch."""
    pairs = keys = 0
    w, f = case["window"], case["sinks"]
    for kl, ql in zip(*_lens(case)):
        p0 = kl - ql
        # rows at p see min(w, p + 1) keys of the window and min(f, p + 1 - w) sinks outside it
        upto = lambda p, m: sum(range(1, min(m, p) + 1)) + max(0, p - m) * m  # sum of min(m, x) over x = 1 .. p
        for m, p, sign in ((w, p0 + ql, 1), (w, p0, -1), (f, p0 + ql - w, 1), (f, p0 - w, -1)):
            pairs += sign * (upto(p, m) if p > 0 else 0)
        low = max(0, p0 - w + 1)
        keys += kl - low + min(f, low)
    return pairs, keys


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "attention":
        pairs, keys = _pairs(case)
        h, hk, d = case["heads"], case["kv_heads"], case["d"]
        rows = sum(_lens(case)[1])
        byte = 2 * rows * h * d * size + 2 * keys * hk * d * size  # q, o; k, v
        flop = 4.0 * pairs * h * d
        if case["mode"] == "train":  # do, dq; dk, dv; lse; five products
            byte = byte * 2 + 4 * rows * h
            flop += 10.0 * pairs * h * d
        return {"bytes": byte, "flops": flop}
    if case["op"] == "rotary":
        vals = case["batch"] * case["length"] * (case["heads"] + case["kv_heads"]) * case["d"]
        return {"bytes": 2 * vals * size + 8 * case["batch"] * case["length"], "flops": 6.0 * vals}
    n = case["rows"] * case["cols"]
    byte = {"forward": 4 * size, "quantised": 3 * size + 1 + 4.0 / GROUP, "train": 7 * size}[case["mode"]] * n
    return {"bytes": byte + 4 * case["cols"] * (2 if case["mode"] == "train" else 1),
            "flops": (16.0 if case["mode"] == "train" else 6.0) * n}


# ------------------------------------------------------------------ 64 bits

def _exact_attention(case, s):
    """One sequence and head at a time, a stretch of rows against all keys."""
    b, h, lq, d = s["q"].shape
    g = h // case["kv_heads"]
    zero = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    out = {"o": zero(s["q"])}
    train = case["mode"] == "train"
    if train:
        out.update(lse=zero(s["q"][..., 0]), dq=zero(s["q"]), dk=zero(s["k"]), dv=zero(s["v"]))
    for i, (kl, ql) in enumerate(zip(*_lens(case))):
        j = torch.arange(kl, device="cuda")
        for a in range(h):
            k, v = s["k"][i, a // g, :kl].double(), s["v"][i, a // g, :kl].double()
            for lo in range(0, ql, 8192):
                hi = min(ql, lo + 8192)
                p = (kl - ql + torch.arange(lo, hi, device="cuda")).unsqueeze(1)
                hidden = (j > p) | ((j <= p - case["window"]) & (j >= case["sinks"]))
                q = s["q"][i, a, lo:hi].double()
                sc = (q @ k.T * case_scale(case)).masked_fill_(hidden, -math.inf)
                lse = torch.logsumexp(sc, 1, keepdim=True)
                pr = (sc - torch.where(lse == -math.inf, 0.0, lse)).exp_()
                o = pr @ v
                out["o"][i, a, lo:hi] = o
                if train:
                    do = s["do"][i, a, lo:hi].double()
                    out["lse"][i, a, lo:hi] = lse[:, 0]
                    out["dv"][i, a // g, :kl] += pr.T @ do
                    ds = (do @ v.T).sub_((do * o).sum(1, keepdim=True)).mul_(pr).mul_(case_scale(case))
                    out["dq"][i, a, lo:hi] = ds @ k
                    out["dk"][i, a // g, :kl] += ds.T @ q
    return out


def case_scale(case):
    return 1.0 / math.sqrt(case["d"])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        ks, qs = _lens(case)
        if sum(x * y for x, y in zip(ks, qs)) * case["heads"] > 1 << 36:
            return None
        return _exact_attention(case, s)
    if case["op"] == "rotary":
        n = case["pairs"]
        angle = s["positions"].double()[:, None, :, None] * s["freqs"] * (-1.0 if case["mode"] == "backward" else 1.0)
        turn = torch.polar(torch.full_like(angle, case["mscale"]), angle)

        def one(x):
            x = x.double()
            r, i = (x[..., : 2 * n].unflatten(-1, (n, 2)).unbind(-1) if case["interleaved"]
                    else x[..., : 2 * n].unflatten(-1, (2, n)).unbind(-2))
            w = torch.view_as_real(torch.complex(r, i) * turn)
            x[..., : 2 * n] = (w if case["interleaved"] else w.transpose(-1, -2)).flatten(-2)
            return x

        return one(s["q"].clone()), one(s["k"].clone())
    h, w = s["x"].double() + s["residual"].double(), s["weight"].double()
    out = {"h": h}
    y = w * h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    if case["mode"] == "quantised":
        cols = torch.arange(case["cols"], device="cuda") // GROUP
        amax = torch.zeros(case["rows"], int(cols[-1]) + 1, dtype=torch.float64, device="cuda")
        amax.scatter_reduce_(1, cols.expand_as(y), y.abs(), "amax")
        out["scales"] = amax.clamp(min=2.0 ** -100) / 448.0
        out["y8"] = y / out["scales"][:, cols]
        return out
    out["y"] = y
    if case["mode"] == "train":
        # the gradient is taken at the stored h: x + residual rounded to its type
        h = h.to(s["x"].dtype).double()
        rms = torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        dy = s["dy"].double()
        out["dw"] = (dy * h / rms).sum(0)
        inner = (dy * w * h).sum(1, keepdim=True)
        out["dx"] = dy * w / rms - h * inner / (case["cols"] * rms ** 3) + s["dh"].double()
    return out
