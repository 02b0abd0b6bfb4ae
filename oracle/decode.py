"""float64 definitions of the steps between a decoder's projections and its
next token: rotary positions, attention over a paged cache, beam selection,
and a cache's pages.

Plain definitions, written from the formulas; nothing here follows the order
or the tiling of the device code.  The pages' definition goes row by row, as
the header states it.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rotary_axes(sections, striped=False):
    """Axis of every frequency pair."""
    if not striped:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, got = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                got.append(a)
                left[a] -= 1
    return got


def rotary(x, positions, inv_freq, sections=None, adjacent=False, striped=False, scale=1.0):
    """x [tokens][heads][dim], positions [axes][tokens], inv_freq [pairs]."""
    x = np.asarray(x, dtype=np.float64)
    positions = np.atleast_2d(np.asarray(positions))
    pairs = len(inv_freq)
    axes = rotary_axes([pairs] if sections is None else sections, striped)
    out = x.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, pairs + i)
        angle = positions[axes[i]].astype(np.float64) * float(inv_freq[i])
        c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
    return out


# ---------------------------------------------------------------------------
# attention over a paged cache
# ---------------------------------------------------------------------------
def paged(pool, pages, length):
    """[length][heads][dim] of a sequence from a [pages][page_size][heads][dim]
    pool."""
    ps = pool.shape[1]
    return np.stack([pool[pages[i // ps], i % ps] for i in range(length)]) if length else pool[:0, 0]


def attention(q, k, v, scale, window=0, softcap=0.0):
    """One sequence: q [heads][dim], k, v [length][kv heads][dim].  Returns
    (out [heads][dim], lse [heads], z [heads][seen])."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, H, G = len(k), q.shape[0], q.shape[0] // k.shape[1]
    lo = max(0, n - window) if window else 0
    out, lse = np.zeros_like(q), np.full(H, -np.inf)
    zs = np.zeros((H, n - lo))
    for h in range(H):
        z = scale * (k[lo:, h // G] @ q[h])
        if softcap:
            z = softcap * np.tanh(z / softcap)
        zs[h] = z
        if len(z):
            m = z.max()
            p = np.exp(z - m)
            out[h] = p @ v[lo:, h // G] / p.sum()
            lse[h] = m + math.log(p.sum())
    return out, lse, zs


# ---------------------------------------------------------------------------
# beam selection
# ---------------------------------------------------------------------------
def beam_select(logits, scores, choices, finished=None, end_token=0):
    """logits [beams][vocab], scores [beams] -> (tokens, parents, scores) of the
    `choices` best, and the best score left out."""
    W, V = np.shape(logits)
    found = []
    for w in range(W):
        s = float(scores[w])
        if not math.isfinite(s):
            continue
        if finished is not None and finished[w]:
            found.append((-s, w, 0.0, end_token))
            continue
        x = np.asarray(logits[w], dtype=np.float64)
        x = np.where(np.isnan(x), -np.inf, x)
        m = x.max()
        if not np.isfinite(m):
            continue
        off = math.log(np.exp(x - m).sum())
        there = np.nonzero(x > -np.inf)[0]
        first = there[np.lexsort((there, -x[there]))][:choices + 1]   # of one beam no more can be chosen
        found += [(-(s + ((float(x[v]) - m) - off)), w, -float(x[v]), int(v)) for v in first]
    found.sort()
    best = found[:choices]
    fill = choices - len(best)
    return (np.array([c[3] for c in best] + [-1] * fill), np.array([c[1] for c in best] + [-1] * fill),
            np.array([-c[0] for c in best] + [-np.inf] * fill),
            -found[choices][0] if len(found) > choices else -np.inf)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def pages_fork(table, lengths, refs, page_size, parents=None, grow=None, max_grow=0, has_slots=True):
    """Row by row; returns a dict of the outputs (slots [rows][max_grow])."""
    rows, width = table.shape
    P = len(refs)
    parents = np.arange(rows) if parents is None else parents
    grow = np.zeros(rows, dtype=int) if grow is None else grow
    held = lambda n: -(-int(n) // page_size)  # noqa: E731
    size = [int(n) if 0 <= n <= width * page_size else 0 for n in lengths]
    refs = [int(r) for r in refs]
    lists, new_len = [], []
    for r in range(rows):
        p = int(parents[r])
        ok = 0 <= p < rows
        lists.append([int(i) for i in table[p, :held(size[p])]] if ok else [])
        new_len.append(size[p] if ok else 0)
    for r in range(rows):
        for i in lists[r]:
            if 0 <= i < P:
                refs[i] += 1
        for i in table[r, :held(size[r])]:
            if 0 <= i < P:
                refs[i] -= 1
    inherited = ([list(x) for x in lists], list(new_len), list(refs))
    bad = sum(1 for r in range(rows) if grow[r] < 0 or (has_slots and max_grow and grow[r] > max_grow)
              or new_len[r] + int(grow[r]) > width * page_size)
    missing, pairs, slots = 0, [], np.full((rows, max_grow), -1)
    if not bad:
        free = [i for i in range(P) if refs[i] <= 0]
        for r in range(rows):
            n, g = new_len[r], int(grow[r])
            last = lists[r][-1] if lists[r] else -1
            if g > 0 and n % page_size and 0 <= last < P and refs[last] > 1:
                if free:
                    to = free.pop(0)
                    pairs.append((last, to, n % page_size))
                    refs[last] -= 1
                    refs[to] = 1
                    lists[r][-1] = to
                else:
                    missing += 1
            for _ in range(held(n + g) - held(n)):
                if free:
                    to = free.pop(0)
                    refs[to] = 1
                    lists[r].append(to)
                else:
                    missing += 1
            for j in range(min(g, max_grow)):
                i = lists[r][(n + j) // page_size] if (n + j) // page_size < len(lists[r]) else -1
                slots[r, j] = i * page_size + (n + j) % page_size if 0 <= i < P else -1
            new_len[r] = n + g
    if bad or missing:
        lists, new_len, refs = inherited
        pairs, slots = [], np.full((rows, max_grow), -1)
    out = np.full((rows, width), -1)
    for r in range(rows):
        out[r, :len(lists[r])] = lists[r]
    listed = np.full((rows, 3), -1)
    if pairs:
        listed[:len(pairs)] = pairs
    return {"table": out, "lengths": np.array(new_len), "refs": np.array(refs), "slots": slots, "pairs": listed,
            "count": len(pairs), "status": (0 if bad else missing, bad)}


def pages_compact(table, lengths, refs, page_size):
    rows, width = table.shape
    P = len(refs)
    used = sum(1 for r in refs if r > 0)
    movers = [i for i in range(used, P) if refs[i] > 0]
    places = [i for i in range(used) if refs[i] <= 0]
    refs = [int(r) for r in refs]
    to = {}
    for a, b in zip(movers, places):
        to[a] = b
        refs[b], refs[a] = refs[a], 0
    out = np.full((rows, width), -1)
    for r in range(rows):
        n = lengths[r]
        for c in range(-(-int(n) // page_size) if 0 <= n <= width * page_size else 0):
            out[r, c] = to.get(int(table[r, c]), int(table[r, c]))
    pairs = np.full((P, 3), -1)
    for j, (a, b) in enumerate(zip(movers, places)):
        pairs[j] = (a, b, page_size)
    return {"table": out, "refs": np.array(refs), "pairs": pairs, "count": len(movers)}
