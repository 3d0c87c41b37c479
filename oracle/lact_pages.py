"""fp64 numpy oracle of the operators on batches of sequences of different
lengths: packed and paged attention, the places of a step's new tokens, and
their copies into a paged cache.  Written from the definitions, one sequence
and token at a time; shares no code with the HIP library.
"""
import numpy as np

from oracle import lact_block as OB


def packed_attention(q, k, v, offsets, window, sinks, scale, dO=None):
    """q [H, T, d], k, v [Hk, T, d], sequences at tokens offsets[b] .. offsets[b + 1].
    Returns what lact_block.window_attention does, for [heads, tokens, d];
    tokens of no sequence are zero."""
    H, T, d = q.shape
    out = {"score_abs": 0.0}
    for a, z in zip(offsets[:-1], offsets[1:]):
        cut = lambda x: None if x is None else x[None, :, a:z]
        one = OB.window_attention(cut(q), cut(k), cut(v), window, sinks, scale, dO=cut(dO))
        out["score_abs"] = max(out["score_abs"], one.pop("score_abs"))
        for n, x in one.items():
            out.setdefault(n, np.zeros((x.shape[1], T) + x.shape[3:]))[:, a:z] = x[0]
    return out


def gather(pages, table, n):
    """The first n tokens [Hk, n, d] of a request out of pages [P, Hk, page, d]."""
    page = pages.shape[2]
    j = np.arange(n)
    return pages[np.asarray(table)[j // page], :, j % page].transpose(1, 0, 2)


def paged_attention(q, k_pages, v_pages, table, offsets, k_lens, window, sinks, scale):
    H, T, d = q.shape
    out = {"score_abs": 0.0, "o": np.zeros(q.shape), "o_abs": np.zeros(q.shape), "lse": np.zeros((H, T))}
    for b, (a, z) in enumerate(zip(offsets[:-1], offsets[1:])):
        k, v = (gather(x, table[b], int(k_lens[b])) for x in (k_pages, v_pages))
        one = OB.window_attention(q[None, :, a:z], k[None], v[None], window, sinks, scale)
        out["score_abs"] = max(out["score_abs"], one["score_abs"])
        for n in ("o", "o_abs", "lse"):
            out[n][:, a:z] = one[n][0]
    return out


def page_slots(lens, counts, table, free, have, page, tokens):
    """(dict of offsets, k_lens, slots, positions, left; the table with its new entries)"""
    table = [list(row) for row in table]
    out = {"offsets": [0], "k_lens": [], "slots": [-1] * tokens, "positions": [0] * tokens}
    have = max(0, min(have, len(free)))
    pages = lambda n: -(-n // page)
    row = asked = taken = refused = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        n, c = max(n, 0), min(max(c, 0), tokens - row)
        served = n + c <= len(table[b]) * page
        if served:
            need = pages(n + c) - pages(n)
            asked += need
            served = need == 0 or asked <= have
        if served:
            for i in range(pages(n), pages(n + c)):
                table[b][i] = free[have - 1 - taken]
                taken += 1
        for r in range(c):
            out["positions"][row + r] = n + r
            if served and table[b][(n + r) // page] >= 0:
                out["slots"][row + r] = table[b][(n + r) // page] * page + (n + r) % page
        refused += not served
        row += c
        out["offsets"].append(row)
        out["k_lens"].append(n + c if served else n)
    out["left"] = [have - taken, refused]
    return out, table


def page_write(x, pages, slots):
    """Rows of x [Hk, T, d] in their places of a copy of pages [P, Hk, page, d]."""
    pages = pages.copy()
    size = pages.shape[2]
    for t, s in enumerate(slots):
        if 0 <= s < pages.shape[0] * size:
            pages[s // size, :, s % size] = x[:, t]
    return pages
