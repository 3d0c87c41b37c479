"""Attention of a server's and a trainer's batches, as measured work: requests
whose keys lie in pages, and texts packed one after another.

A server keeps the keys and values of many requests in pages of a common pool.
Each step it places the new tokens (page_slots), writes their k and v there
(page_write) and lets them attend over what their request has so far
(paged_attention): single next tokens, chunks of a prompt, or both in one
batch.  Prompts that start from nothing, and texts of a training step, are
packed into one row of tokens (packed_attention and its backward).  This file
lists those operators' cases at real sizes, makes their inputs, and states each
operator twice: in elementary torch operations (`run` with `own` false) and in
64 bits from the definition (`exact`).  With `own` true `run` makes the calls of
test_layers_amd.lact.

Slots.  Request b has lens[b] tokens in pages table[b][0 .. ceil(lens / page))
and gets counts[b] more, at rows offsets[b] .. offsets[b + 1] of the step's
`tokens` rows (the counts are cut where the rows end).  The pages it needs more
come off the end of free[0 .. free_count), request by request.  A request whose
pages do not fit its row of the table, or the pool once those before it took
theirs, gets none: its tokens have slot -1 and its k_lens stays.  Row r of a
served request has position lens[b] + r and slot table[b][position / page] page
+ position % page; rows of no request have slot -1 and position 0.

Write.  cache[slot] = k, v of each row whose slot is in the cache.

Attention.  Row r of a sequence with n rows and m keys stands at p = m - n + r
and sees the keys j <= p, j < m that are among its last `window` (j > p -
window; 0: all) or among the first `sinks`.
  s_j = scale q . k_j,  lse = log sum_j exp s_j,  o = sum_j exp(s_j - lse) v_j,
a row that sees nothing gives o = 0 and lse = -inf.  Packed: n = m.  Gradients:
with P = exp(s - lse), D = dO . o, dS = P (dO . v - D),
  dv_j = sum_r P dO,  dq = scale sum_j dS k_j,  dk_j = scale sum_r dS q,
summed over the query heads that share a key head.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    slot = dict(op="slots", short=False)
    write = dict(op="write", type="bf16", kv_heads=8, d=128, layout="tokens")
    paged = dict(op="paged", type="bf16", sinks=0, window=0, heads=32, kv_heads=8, d=128, layout="tokens")
    packed = dict(op="packed", type="bf16", sinks=0, window=0, heads=32, kv_heads=8, d=128, layout="tokens", empty=0)
    return [
        # where a decoding batch's next tokens go: all latency
        dict(slot, name="slots_decode", batch=64, tokens=64, chunks=0, k_len=8192, page=64),
        # a step of a thousand requests, prompts among them
        dict(slot, name="slots_prompts", batch=1024, tokens=32768, chunks=100, k_len=8192, page=16),
        # the k and v of a decoding batch
        dict(write, name="write_decode", tokens=64, page=64),
        # those of a step's prompts
        dict(write, name="write_prompt", tokens=32768, page=16),
        # one user's next token over a long text: the smallest attention call
        dict(paged, name="paged_one", batch=1, chunks=0, chunk=1, k_len=32768, page=64, heads=16, kv_heads=16, d=64,
             window=2048, sinks=4),
        # a serving batch's next tokens, requests of every length, small pages
        dict(paged, name="paged_decode", batch=96, chunks=0, chunk=1, k_len=8192, page=16),
        # a chunk of a long prompt over what came before
        dict(paged, name="paged_chunk", batch=1, chunks=1, chunk=2048, k_len=32768, page=128),
        # next tokens and chunks of prompts in one batch; pages of an odd size
        dict(paged, name="paged_mixed", batch=40, chunks=4, chunk=512, k_len=12000, page=48),
        # a few short prompts
        dict(packed, name="packed_short", mode="forward", batch=12, tokens=2000, layout="heads"),
        # prompts of up to 7K tokens, read at once
        dict(packed, name="packed_32k", mode="forward", batch=8, tokens=32768),
        # a training step over packed texts at the 32K language-model length, window of one 2K chunk
        dict(packed, name="packed_train", mode="train", batch=11, tokens=32768, heads=16, kv_heads=16, d=64,
             window=2048, sinks=4),
        # fp32, odd sizes, an empty text among them
        dict(packed, name="packed_train_fp32", mode="train", type="fp32", batch=6, tokens=4001, heads=12, kv_heads=4,
             d=96, window=333, sinks=17, layout="heads", empty=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "write", "paged", "paged", "packed", "packed"])
    page = rng.choice([16, 16, 32, 64, 128, 256, 8 * rng.randint(1, 40)])
    if op == "slots":
        batch = _log(rng, 1, 4096)
        tokens = max(batch, _log(rng, 1, 32768)) if rng.random() < 0.7 else batch
        return dict(op=op, batch=batch, tokens=tokens, chunks=0 if tokens == batch else _log(rng, 1, batch),
                    k_len=_log(rng, 1, 16384), page=page, short=rng.random() < 0.2)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 64, 128, 8 * rng.randint(2, 16)])
    kind = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    base = dict(op=op, type=kind, kv_heads=kv_heads, d=d, layout=rng.choice(["tokens", "heads"]))
    if op == "write":
        return dict(base, tokens=_log(rng, 1, (1 << 25) // (kv_heads * d)), page=page)
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 8])
    limited = rng.random() < 0.6
    base.update(heads=heads, window=_log(rng, 1, 4096) if limited else 0,
                sinks=rng.choice([0, 1, 4, 4, 16, rng.randint(0, 100)]) if limited else 0)
    reach = lambda n: min(n, base["window"] + base["sinks"]) if limited else n
    most = (1 << 36 if kind == "bf16" else 1 << 32) // (heads * d)  # pairs of all rows and what they may see
    if op == "paged":
        batch = _log(rng, 1, 96)
        k_len = _log(rng, 1, min(32768, (1 << 29) // (batch * kv_heads * d)))
        chunks = rng.choice([0, 0, min(batch, rng.randint(1, 4)), batch])
        chunk = 1 if chunks == 0 else min(k_len, _log(rng, 2, 2048))
        while chunk > 1 and chunks * chunk * reach(k_len) > most:
            chunk = (chunk + 1) // 2
        return dict(base, batch=batch, chunks=chunks, chunk=chunk, k_len=k_len, page=page)
    mode = rng.choice(["forward", "train"])
    batch = _log(rng, 1, 64)
    tokens = max(batch, _log(rng, 2, 32768))
    while tokens > batch and tokens * reach(2 * tokens // batch + 1) > most // (4 if mode == "train" else 1):
        tokens = max(batch, (tokens + 1) // 2)
    return dict(base, mode=mode, batch=batch, tokens=tokens, empty=rng.choice([0, 0, 1]) if batch > 1 else 0)


def _spread(total, n):
    """`total` in n parts of different sizes."""
    w = [10 + (61 * i + 13) % 97 for i in range(n)]
    parts = [total * x // sum(w) for x in w]
    parts[-1] += total - sum(parts)
    return parts


def _new(case):
    """New tokens of each request: `chunks` of them get several, spread among the others, which get one."""
    b, n = case["batch"], case["chunks"]
    at = {i * b // n for i in range(n)} if n else set()
    if case["op"] == "paged":
        return [case["chunk"] - (case["chunk"] * i // (2 * b) if n < b else 0) if i in at else 1 for i in range(b)]
    counts = [1] * b
    if n:
        for i, x in zip(sorted(at), _spread(case["tokens"] - b, len(at))):
            counts[i] += x
    return counts


def _keys(case):
    """Tokens of each request with its new ones: from a quarter of k_len up to all of it."""
    b, k = case["batch"], case["k_len"]
    return [max(n, k - k * ((61 * i + 13) % 97) // 130) for i, n in enumerate(_new(case))] if b > 1 else [k]


def _texts(case):
    n = case["batch"] - case["empty"]
    texts = _spread(case["tokens"], n)
    return texts[: n // 2] + [0] * case["empty"] + texts[n // 2 :]


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _heads(gen, case, heads, tokens):
    """[heads, tokens, d]: stored head by head, or as a view of token-major memory."""
    t = TYPES[case["type"]]
    if case["layout"] == "tokens":
        return _normal(gen, (tokens, heads, case["d"]), t).transpose(0, 1)
    return _normal(gen, (heads, tokens, case["d"]), t)


def _pool(gen, case, pages):
    """[pages, kv_heads, page, d] in the same two orders."""
    t, h, d = TYPES[case["type"]], case["kv_heads"], case["d"]
    if case["layout"] == "tokens":
        return _normal(gen, (pages, case["page"], h, d), t).transpose(1, 2)
    return _normal(gen, (pages, h, case["page"], d), t)


def _whole(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")


def _sums(counts):
    total = [0]
    for n in counts:
        total.append(total[-1] + n)
    return total


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "packed":
        q = _heads(gen, case, case["heads"], case["tokens"])
        k = _heads(gen, case, case["kv_heads"], case["tokens"])
        v = _heads(gen, case, case["kv_heads"], case["tokens"])
        texts = _texts(case)
        s.update(q=q, k=k, v=v, scale=1.0 / math.sqrt(case["d"]), offsets=_whole(_sums(texts)), longest=max(texts))
        if case["mode"] == "train":
            s["do"] = _heads(gen, case, case["heads"], case["tokens"])
        return s
    size = case["page"]
    if case["op"] == "write":
        pages = -(-case["tokens"] * 5 // (4 * size)) + 1
        s["k"], s["v"] = (_heads(gen, case, case["kv_heads"], case["tokens"]) for _ in range(2))
        s["k_pages"], s["v_pages"] = (_pool(gen, case, pages) for _ in range(2))
        # runs of a page's slots, pages in any order
        order = torch.randperm(pages, generator=gen, device="cuda")
        s["slots"] = (order.unsqueeze(1) * size + torch.arange(size, device="cuda")).flatten()[: case["tokens"]]
        return s
    counts, keys = _new(case), _keys(case)
    used = [-(-x // size) for x in keys]
    pages, width = sum(used) + len(used) // 4 + 1, max(used) + 2
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    if case["op"] == "slots":
        # the requests hold what they needed before this step; the rest is free
        held = [-(-(x - n) // size) for x, n in zip(keys, counts)]
        first = _sums(held)
        free = pages - first[-1]
        if case["short"]:
            free = min(free, (sum(used) - first[-1]) // 2)
        s.update(lens=_whole([x - n for x, n in zip(keys, counts)]), counts=_whole(counts),
                 free=order[first[-1] :].contiguous(), free_count=_whole([free]))
    else:
        held, first = used, _sums(used)
        s["q"] = _heads(gen, case, case["heads"], sum(counts))
        s["k_pages"], s["v_pages"] = (_pool(gen, case, pages) for _ in range(2))
        if case["sinks"]:
            # the first tokens draw attention from everywhere
            lean = _normal(gen, (case["d"],), TYPES[case["type"]])
            at = order[_whole([a for a, n in zip(first, used) if n])].long()
            s["k_pages"][at, :, : case["sinks"]] += lean
            s["q"] += lean / 4
        s.update(offsets=_whole(_sums(counts)), k_lens=_whole(keys), scale=1.0 / math.sqrt(case["d"]),
                 longest=max(counts), q_host=counts, k_host=keys)
    col = torch.arange(width, device="cuda")
    at = _whole(first[:-1]).unsqueeze(1) + col
    table = torch.where(col < _whole(held).unsqueeze(1), order[at.clamp(max=pages - 1)], -1)
    s["table"] = table.int().contiguous()
    return s


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    from test_layers_amd import lact

    if s["op"] == "slots":
        out = lact.page_slots(s["lens"], s["counts"], s["table"], s["free"], s["free_count"], page=s["page"],
                              tokens=s["tokens"])
        return dict(out, table=s["table"])
    if s["op"] == "write":
        return lact.page_write(s["k"], s["v"], s["k_pages"], s["v_pages"], slots=s["slots"])
    kw = dict(window=s["window"], sinks=s["sinks"], scale=s["scale"], offsets=s["offsets"], longest=s["longest"])
    if s["op"] == "paged":
        return {"o": lact.paged_attention(s["q"], s["k_pages"], s["v_pages"], table=s["table"], k_lens=s["k_lens"], **kw)}
    if s["mode"] == "forward":
        return {"o": lact.packed_attention(s["q"], s["k"], s["v"], **kw)}
    o, lse = lact.packed_attention(s["q"], s["k"], s["v"], return_lse=True, **kw)
    g = lact.packed_attention_backward(s["q"], s["k"], s["v"], o, lse, dO=s["do"], **kw)
    return {"o": o, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}


# ------------------------------------------------------------------ the plain forms

def _plain_slots(s):
    size, t, table = s["page"], s["tokens"], s["table"]
    width, dev = table.shape[1], table.device
    lens = s["lens"].clamp(min=0)
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    offsets = torch.cat([zero, s["counts"].clamp(0, t).cumsum(0).clamp(max=t)])
    count = offsets[1:] - offsets[:-1]
    held = (lens + size - 1) // size
    fits = lens + count <= width * size
    need = torch.where(fits, (lens + count + size - 1) // size - held, 0)
    upto = need.cumsum(0)
    good = fits & ((need == 0) | (upto <= s["free_count"]))
    need = torch.where(good, need, 0)
    k_lens = torch.where(good, lens + count, lens)
    # the new pages of request b are the need[b] before free_count - (upto[b] - need[b])
    col = torch.arange(width, device=dev)
    nth = col - held.unsqueeze(1)
    fresh = (nth >= 0) & (nth < need.unsqueeze(1))
    at = (s["free_count"] - 1 - (upto - need).unsqueeze(1) - nth).clamp(0, max(0, s["free"].numel() - 1))
    if s["free"].numel():
        table.copy_(torch.where(fresh, s["free"][at], table))
    row = torch.arange(t, device=dev)
    b = torch.searchsorted(offsets, row, right=True) - 1
    live = row < offsets[-1]
    b = torch.where(live, b, 0)
    position = torch.where(live, lens[b] + row - offsets[b], 0)
    page = table[b, (position // size).clamp(max=width - 1)].long()
    slots = torch.where(live & good[b] & (page >= 0), page * size + position % size, -1)
    left = torch.stack([s["free_count"][0] - need.sum(), (~good).sum()])
    return {"offsets": offsets, "k_lens": k_lens, "slots": slots, "positions": position, "left": left, "table": table}


def _plain_write(s):
    size = s["page"]
    for x, pool in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
        pool.transpose(1, 2)[s["slots"] // size, s["slots"] % size] = x.transpose(0, 1)
    return s["k_pages"], s["v_pages"]


def _softmax(s, sc, p, k0, m):
    """Probabilities and lse of scores [..., n, keys] whose first key is k0, for rows at positions p of sequences of m keys."""
    j = k0 + torch.arange(sc.shape[-1], device=sc.device)
    see = (j <= p.unsqueeze(-1)) & (j < m)
    if s["window"]:
        see &= (j > p.unsqueeze(-1) - s["window"]) | (j < s["sinks"])
    sc = torch.where(see, sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(sc - top)
    z = e.sum(-1, keepdim=True)
    return e / torch.where(z == 0, 1.0, z), (top + torch.log(z)).squeeze(-1)


def _blocks(s, n, m):
    """Blocks of rows of a sequence with the stretch of keys that they can reach; the sinks lie before it or inside."""
    step = 1024
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        first = max(0, m - n + lo - s["window"] + 1) if s["window"] else 0
        if first <= s["sinks"]:
            first = 0
        yield lo, hi, first, max(0, m - n + hi)


def _part(s, x, first, last):
    """Keys first .. last - 1 of [heads, keys, d], after those of the sinks."""
    return torch.cat([x[:, : s["sinks"]], x[:, first:last]], 1) if first else x[:, :last]


def _plain_sequence(s, q, k, v, do, out):
    """One sequence, q [h, n, d], k and v [hk, m, d]: a block of rows after another."""
    h, n, d = q.shape
    hk, m = k.shape[0], k.shape[1]
    k, v = k.float(), v.float()
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for lo, hi, first, last in _blocks(s, n, m):
        kk, vv = _part(s, k, first, last), _part(s, v, first, last)
        rows = lambda x: x[:, lo:hi].float().reshape(hk, -1, d)  # query heads of a key head together
        unrows = lambda x: x.view(h, hi - lo, -1)
        p = (m - n + torch.arange(lo, hi, device=q.device)).repeat(h // hk)
        qq = rows(q)
        sc = qq @ kk.transpose(-1, -2).contiguous() * s["scale"]
        if first:
            near = sc[..., s["sinks"] :]
            j = first + torch.arange(near.shape[-1], device=q.device)
            see = (j <= p.unsqueeze(-1)) & (j > p.unsqueeze(-1) - s["window"])
            sc = torch.cat([sc[..., : s["sinks"]], torch.where(see, near, -math.inf)], -1)
            top = sc.amax(-1, keepdim=True)
            e = torch.exp(sc - top)
            z = e.sum(-1, keepdim=True)
            pr, lse = e / z, (top + torch.log(z)).squeeze(-1)
        else:
            pr, lse = _softmax(s, sc, p, 0, m)
        o = pr @ vv
        out["o"][:, lo:hi] = unrows(o).to(q.dtype)
        if do is None:
            continue
        out["lse"][:, lo:hi] = unrows(lse).squeeze(-1)
        g = rows(do)
        ds = pr * (g @ vv.transpose(-1, -2).contiguous() - (g * o).sum(-1, keepdim=True)) * s["scale"]
        out["dq"][:, lo:hi] = unrows(ds @ kk).to(q.dtype)
        for to, a, x in ((dk, ds, qq), (dv, pr, g)):
            x = a.transpose(-1, -2).contiguous() @ x
            if first:
                to[:, : s["sinks"]] += x[:, : s["sinks"]]
                to[:, first:last] += x[:, s["sinks"] :]
            else:
                to[:, :last] += x
    if do is not None:
        out["dk"].copy_(dk)
        out["dv"].copy_(dv)


def _plain_packed(s):
    q, k, v = s["q"], s["k"], s["v"]
    out = {"o": torch.zeros_like(q)}
    if s["mode"] == "train":
        out.update(lse=torch.zeros(q.shape[:2], device=q.device), dq=torch.zeros_like(q), dk=torch.zeros_like(k),
                   dv=torch.zeros_like(v))
    at = 0
    for n in _texts(s):
        if n:
            cut = lambda x: x[:, at : at + n]
            do = cut(s["do"]) if s["mode"] == "train" else None
            _plain_sequence(s, cut(q), cut(k), cut(v), do, {name: cut(x) for name, x in out.items()})
        at += n
    return out


def _plain_paged(s):
    q, size = s["q"], s["page"]
    h, t, d = q.shape
    hk = s["kv_heads"]
    out = torch.zeros_like(q)
    if s["longest"] > 1:
        at = 0
        for i, (n, m) in enumerate(zip(s["q_host"], s["k_host"])):
            pages = s["table"][i, : -(-m // size)].long()
            kk, vv = (x[pages].transpose(0, 1).reshape(hk, -1, d)[:, :m] for x in (s["k_pages"], s["v_pages"]))
            _plain_sequence(s, q[:, at : at + n], kk, vv, None, {"o": out[:, at : at + n]})
            at += n
        return {"o": out}
    # one row each: all requests at once
    m = s["k_lens"]
    high = max(s["k_host"])
    low = max(0, min(s["k_host"]) - s["window"]) if s["window"] else 0
    key = torch.arange(low, high, device=q.device)
    if low <= s["sinks"]:
        key = torch.arange(high, device=q.device)
    else:
        key = torch.cat([torch.arange(s["sinks"], device=q.device), key])
    page = s["table"][:, key // size].long().clamp(min=0)
    kk, vv = (x.transpose(1, 2)[page, key % size].float().permute(0, 2, 1, 3).contiguous()
              for x in (s["k_pages"], s["v_pages"]))
    qq = q.float().transpose(0, 1).reshape(t, hk, h // hk, d)
    sc = qq @ kk.transpose(-1, -2).contiguous() * s["scale"]
    end = m.view(-1, 1)
    see = key < end
    if s["window"]:
        see = see & ((key >= end - s["window"]) | (key < s["sinks"]))
    sc = torch.where(see.view(t, 1, 1, -1), sc, -math.inf)
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = (e / e.sum(-1, keepdim=True)) @ vv
    out.copy_(o.reshape(t, h, d).transpose(0, 1))
    return {"o": out}


def run(state):
    if own:
        return _own(state)
    return {"slots": _plain_slots, "write": _plain_write, "paged": _plain_paged, "packed": _plain_packed}[state["op"]](state)


# ------------------------------------------------------------------ work

def _seen(case, n, m):
    """(visible pairs of one head, keys that some row sees) of a sequence of n rows and m keys."""
    w, f = case["window"] or m + 1, case["sinks"]
    p0 = m - n
    # rows at p see min(w, p + 1) keys of the window and min(f, p + 1 - w) sinks outside it
    upto = lambda p, most: (min(most, p) * (min(most, p) + 1) // 2 + max(0, p - most) * most) if p > 0 else 0
    pairs = upto(p0 + n, w) - upto(p0, w) + upto(p0 + n - w, f) - upto(p0 - w, f)
    low = max(0, p0 - w + 1)
    return pairs, m - low + min(f, low)


def work(case):
    if case["op"] == "slots":
        b, t = case["batch"], case["tokens"]
        fresh = sum(-(-m // case["page"]) - -(-(m - n) // case["page"]) for n, m in zip(_new(case), _keys(case)))
        # lens, counts; offsets, k_lens; slots, positions; entries read and written
        return {"bytes": 32.0 * b + 16.0 * t + 4.0 * b + 8.0 * fresh, "flops": 8.0 * t}
    size = 2 if case["type"] == "bf16" else 4
    hk, d = case["kv_heads"], case["d"]
    if case["op"] == "write":
        return {"bytes": case["tokens"] * (4.0 * hk * d * size + 8), "flops": 0.0}
    h = case["heads"]
    lens = list(zip(_new(case), _keys(case))) if case["op"] == "paged" else [(n, n) for n in _texts(case) if n]
    seen = [_seen(case, n, m) for n, m in lens]
    pairs, keys, rows = sum(x for x, _ in seen), sum(x for _, x in seen), sum(n for n, _ in lens)
    byte = 2.0 * rows * h * d * size + 2.0 * keys * hk * d * size
    flop = 4.0 * pairs * h * d
    if case["op"] == "packed" and case["mode"] == "train":
        byte = 2 * byte + 4 * rows * h
        flop += 10.0 * pairs * h * d
    return {"bytes": byte, "flops": flop}


# ------------------------------------------------------------------ 64 bits

def _exact_slots(s):
    """One request and token after another, on the host."""
    size, t = s["page"], s["tokens"]
    table, free = s["table"].tolist(), s["free"].tolist()
    have = s["free_count"].item()
    wanted = row = refused = taken = 0
    out = {"offsets": [0], "k_lens": [], "slots": [-1] * t, "positions": [0] * t}
    for b, (n, c) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
        c = min(c, t - row)
        pages = lambda x: -(-x // size)
        good = n + c <= len(table[b]) * size
        if good:
            more = pages(n + c) - pages(n)
            wanted += more
            good = more == 0 or wanted <= have
            if good:
                for i in range(pages(n), pages(n + c)):
                    table[b][i] = free[have - 1 - taken]
                    taken += 1
        for r in range(c):
            out["positions"][row + r] = n + r
            if good and table[b][(n + r) // size] >= 0:
                out["slots"][row + r] = table[b][(n + r) // size] * size + (n + r) % size
        refused += not good
        row += c
        out["offsets"].append(row)
        out["k_lens"].append(n + c if good else n)
    out["left"] = [have - taken, refused]
    return dict({name: _whole(x) for name, x in out.items()}, table=torch.tensor(table, dtype=torch.int32, device="cuda"))


def _exact_sequence(case, q, k, v, do, out, add):
    """One head and stretch of rows at a time, against all keys up to their last."""
    h, n, d = q.shape
    g, m, scale = h // k.shape[0], k.shape[1], 1.0 / math.sqrt(d)
    for a in range(h):
        for lo in range(0, n, 4096):
            hi = min(n, lo + 4096)
            p = (m - n + torch.arange(lo, hi, device="cuda")).unsqueeze(1)
            last = m - n + hi
            j = torch.arange(last, device="cuda")
            hidden = j > p
            if case["window"]:
                hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
            kk, vv, qq = k[a // g, :last].double(), v[a // g, :last].double(), q[a, lo:hi].double()
            sc = (qq @ kk.T).mul_(scale).masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(sc, 1, keepdim=True)
            pr = sc.sub_(lse).exp_()
            o = pr @ vv
            out["o"][a, lo:hi] = o
            if do is not None:
                gg = do[a, lo:hi].double()
                out["lse"][a, lo:hi] = lse[:, 0]
                add["dv"][a // g, :last] += pr.T @ gg
                ds = (gg @ vv.T).sub_((gg * o).sum(1, keepdim=True)).mul_(pr).mul_(scale)
                out["dq"][a, lo:hi] = ds @ kk
                add["dk"][a // g, :last] += ds.T @ qq


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "slots":
        return _exact_slots(s)
    zero = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    if case["op"] == "write":
        out = s["k_pages"].double(), s["v_pages"].double()
        at = torch.zeros(out[0].shape[0] * case["page"], dtype=torch.int64, device="cuda") - 1
        at[s["slots"]] = torch.arange(case["tokens"], device="cuda")  # the row that each place gets
        at = at.view(-1, 1, case["page"], 1)
        for x, pool in zip((s["k"], s["v"]), out):
            new = x.double()[:, at.flatten().clamp(min=0)].unflatten(1, (-1, case["page"])).transpose(0, 1)
            pool.copy_(torch.where(at >= 0, new, pool))
        return out
    q = s["q"]
    out = {"o": zero(q)}
    if case["op"] == "paged":
        lens = list(zip(_new(case), _keys(case)))
        if sum(n * m for n, m in lens) * case["heads"] > 1 << 36:
            return None
        row = 0
        for i, (n, m) in enumerate(lens):
            j = torch.arange(m, device="cuda")
            page = s["table"][i, j // case["page"]].long()
            k, v = (x[page, :, j % case["page"]].transpose(0, 1) for x in (s["k_pages"], s["v_pages"]))
            _exact_sequence(case, q[:, row : row + n], k, v, None, {"o": out["o"][:, row : row + n]}, None)
            row += n
        return out
    train = case["mode"] == "train"
    if train:
        out.update(lse=zero(q[..., 0]), dq=zero(q), dk=zero(s["k"]), dv=zero(s["v"]))
    row = 0
    for n in _texts(case):
        cut = lambda x: x[:, row : row + n]
        parts = {name: cut(x) for name, x in out.items()}
        _exact_sequence(case, cut(q), cut(s["k"]), cut(s["v"]), cut(s["do"]) if train else None, parts, parts)
        row += n
    return out
