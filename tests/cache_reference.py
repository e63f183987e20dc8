"""Drafted tokens and caches of bounded length, written plainly in 64 bits on the CPU
for the tests: trees, what their tokens see, the weight that tokens draw, the choice of
those that are kept."""

from __future__ import annotations

import math

import numpy as np

from tests.attention_reference import attention_slack


def random_tree(rng, n, roots=1):
    """Parents of n drafted tokens, the first `roots` of them roots."""
    return [-1 if i < roots else int(rng.integers(0, i)) for i in range(n)]


def ancestors(parents):
    """For each token the set of those that it descends from, itself among them, by its path."""
    out = []
    for i in range(len(parents)):
        path, at = set(), i
        while at >= 0:
            path.add(at)
            at = parents[at] if 0 <= parents[at] < at else -1
        out.append(path)
    return out


def words_of(sets, words):
    """int64 [tokens, words] of sets of bit numbers."""
    out = np.zeros((len(sets), words), dtype=np.uint64)
    for i, bits in enumerate(sets):
        for j in bits:
            if j < 64 * words:
                out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def visible(length, queries, i, bits=None, window=0):
    """The tokens that query i of a sequence sees, in their order: those before the queries and
    its bits' drafts, or without bits all up to its own place; the last `window` of them."""
    before = length - queries
    if bits is None:
        seen = list(range(0, max(0, before + i + 1)))
        return seen if not window else [t for t in seen if t > before + i - window]
    seen = list(range(0, max(0, before)))
    seen += [before + j for j in sorted(bits) if j < queries and before + j >= 0]
    return seen[-window:] if window else seen


def tree_attention(q, values, query_start, seq_lens, page_table, page, scale, bits=None, window=0,
                   max_seq_len=None, max_query_len=1 << 30, lse_in=None):
    """For q [tokens, q_heads, d], cache values [pages, 2, kv_heads, page, d] and bits (a set a
    token, or None): dict of out, lse [tokens, q_heads] and bounds on a kernel's errors in
    them, drawn [pages, kv_heads, page] with its bound (exp(score - lse), of lse_in where
    given), and which places the step's sequences hold (`held`, and `fresh` of its own tokens)."""
    T, hq, d = q.shape
    pages, _, kv = values.shape[:3]
    group = hq // kv
    r = dict(out=np.full((T, hq, d), np.nan), out_slack=np.zeros((T, hq, d)), lse=np.full((T, hq), np.nan),
             lse_slack=np.zeros((T, hq)), drawn=np.zeros((pages, kv, page)), drawn_slack=np.zeros((pages, kv, page)),
             held=np.zeros((pages, page), dtype=bool), fresh=np.zeros((pages, page), dtype=bool))
    for s in range(len(seq_lens)):
        first, queries = query_start[s], query_start[s + 1] - query_start[s]
        length = max(0, seq_lens[s] if max_seq_len is None else min(seq_lens[s], max_seq_len))
        if not 0 <= first < T or queries <= 0:
            continue
        for t in range(length):
            p = page_table[s][t // page]
            if 0 <= p < pages:
                r["held"][p, t % page] = True
                r["fresh"][p, t % page] = t >= length - queries
        rows = min(queries, max_query_len, T - first)
        for i in range(rows):
            seen = visible(length, queries, i, None if bits is None else bits[first + i], window)
            seen = [t for t in seen if 0 <= page_table[s][t // page] < pages]
            if not seen:
                r["out"][first + i], r["lse"][first + i] = 0.0, -math.inf
                continue
            at = np.array(seen)
            held, inside = np.asarray(page_table[s])[at // page], at % page
            for h in range(hq):
                with np.errstate(all="ignore"):
                    k, v = values[held, 0, h // group, inside], values[held, 1, h // group, inside]
                    score = scale * (k @ q[first + i, h])
                    top = score.max()
                    e = np.exp(score - top)
                    total = e.sum()
                    p = e / total
                    out, lse = p @ v, top + math.log(total) if total > 0 else math.nan
                    size = abs(scale) * np.abs(q[first + i, h]).max() * np.abs(k).sum(1).max()
                    r["out"][first + i, h], r["lse"][first + i, h] = out, lse
                    r["out_slack"][first + i, h] = attention_slack(out, p @ np.abs(v), size, d, len(seen),
                                                                   np.abs(score).max())
                    # scores of d products summed in fp32, the power's argument and the power in fp32,
                    # a sum over n in fp32, a logarithm of at most 2^32 and the steps back to base e
                    products = size * d * 2.0 ** -24
                    r["lse_slack"][first + i, h] = (products + (np.abs(score).max() + 1) * 2.0 ** -22 +
                                                    len(seen) * 2.0 ** -24 + (abs(lse) + 32) * 2.0 ** -22)
                    used = lse if lse_in is None else lse_in[first + i, h]
                    if used == -math.inf:
                        continue
                    w = np.exp(score - used)
                    # the argument's terms in fp32, the power, and a sum over at most all rows
                    off = products + (np.abs(score) + abs(used) + 1) * 2.0 ** -22 + rows * group * 2.0 ** -24
                    np.add.at(r["drawn"], (held, h // group, inside), w)
                    # (powers below fp32's normal numbers may be lost)
                    np.add.at(r["drawn_slack"], (held, h // group, inside), w * off * 1.01 + 2.0 ** -125)
    return r


def mass_after(mass, r):
    """The mass after a step that drew r's, and a bound on a kernel's error in it."""
    held, fresh = r["held"][:, None, :], r["fresh"][:, None, :]
    with np.errstate(all="ignore"):
        want = np.where(held, r["drawn"] + np.where(fresh, 0.0, mass), mass)
        return want, np.where(held, r["drawn_slack"] + 2.0 ** -23 * np.abs(want), 0.0)


def select(weights, n, sinks, recent, budget):
    """The numbers that one key head keeps of n tokens with these weights (floats), ascending."""
    if n <= budget:
        return list(range(n))
    always = set(range(sinks)) | set(range(n - recent, n))
    w = [-math.inf if math.isnan(x) else x for x in weights[:n]]
    others = sorted((t for t in range(n) if t not in always), key=lambda t: (-w[t], t))
    return sorted(list(always) + others[:budget - len(always)])


def by_place(cache, d, page):
    """The bytes of each place, [pages, 2, kv_heads, page, d / 2 + d / 32], of a cache's bytes."""
    codes = cache[..., :page * (d // 2)].reshape(*cache.shape[:3], page, d // 2)
    scales = cache[..., page * (d // 2):].reshape(*cache.shape[:3], d // 32, page)
    return np.concatenate([codes, scales.swapaxes(-1, -2)], axis=-1)


def compact(places, mass, kept, counts, first, table, dst_table):
    """(places, mass) after the moves: every place gets what its source held before."""
    pages, _, kv, page, _ = places.shape
    new_places, new_mass = places.copy(), mass.copy()
    dst = table if dst_table is None else dst_table
    for s in range(len(counts)):
        base = 0 if first is None else int(first[s])
        n = max(0, min(int(counts[s]), kept.shape[2]))
        if base < 0:
            continue
        for h in range(kv):
            k = kept[s, h if kept.shape[1] > 1 else 0, :n].astype(np.int64)
            j = np.arange(n)
            ok = (k >= 0) & (base + k < table.shape[1] * page) & (base + j < dst.shape[1] * page)
            if dst_table is None:
                ok &= k > j
            src, to = (base + k)[ok], (base + j)[ok]
            a, b = table[s, src // page], dst[s, to // page]
            there = (a >= 0) & (a < pages) & (b >= 0) & (b < pages)
            a, b, src, to = a[there], b[there], src[there] % page, to[there] % page
            new_places[b, :, h, to] = places[a, :, h, src]
            new_mass[b, h, to] = mass[a, h, src]
    return new_places, new_mass
