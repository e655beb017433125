"""CPU fp64 oracle of the decoding operators: rotary positions, the append to a paged
key-value cache, attention of one new token over it, eviction by accumulated weight.

TEST INFRASTRUCTURE ONLY, like xattn_oracle. Arrays are numpy; a cache is a plain dict
of arrays: k, v [P, Hkv, page, C] (fp64 values as stored), acc, ordinal [P, Hkv, page],
table [B, max_pages], lens [B], and k_scale, v_scale [Hkv] or None. Every function
walks sequences, heads and slots one by one, straight from the definitions:

- pair p of a row turns by pos[axis(p)] * inv_freq[p];
- slot s of sequence b lies in page table[b, s // page], row s % page;
- o = sum_s softmax_s(scale q . k_s) v_s over s < lens[b]; no slot: o = 0, lse = -inf;
- eviction keeps the safe slots (ordinal >= seen - recent or < sink) first, then the
  largest weights, ties to the lower slot; the i-th evicted slot below n takes the i-th
  kept slot from the end.
"""
from __future__ import annotations

import numpy as np

__all__ = ["rope", "cache_slot", "cache_append", "cache_rows", "decode_attention", "evict_kept",
           "cache_evict"]


def rope(x, pos, inv_freq, sections, interleaved=False, inverse=False):
    """x [B, H, M, C] fp64, pos [B, M, axes] -> the rotated rows, fp64."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    P = len(axis)
    for b in range(x.shape[0]):
        for p in range(P):
            angle = pos[b, :, axis[p]].astype(np.float64) * float(inv_freq[p])
            if inverse:
                angle = -angle
            i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + P)
            c, s = np.cos(angle), np.sin(angle)
            y[b, :, :, i] = x[b, :, :, i] * c - x[b, :, :, j] * s
            y[b, :, :, j] = x[b, :, :, j] * c + x[b, :, :, i] * s
    return y


def cache_slot(cache, b, s):
    """(page, row) of slot s of sequence b."""
    page = cache["k"].shape[2]
    return int(cache["table"][b, s // page]), s % page


def cache_append(cache, k, v, n_new, seen):
    """k, v [B, Hkv, T, C] fp64 into the last n_new[b] slots; returns a new cache whose k, v
    hold the unrounded stored values (x / scale, saturated at 448 for scaled pages)."""
    out = dict(cache, k=cache["k"].copy(), v=cache["v"].copy(), acc=cache["acc"].copy(),
               ordinal=cache["ordinal"].copy())
    for b in range(len(cache["lens"])):
        for t in range(int(n_new[b])):
            pg, row = cache_slot(cache, b, int(cache["lens"][b]) - int(n_new[b]) + t)
            for name, x in (("k", k), ("v", v)):
                y = x[b, :, t]
                sc = cache[name + "_scale"]
                if sc is not None:
                    y = np.clip(y / np.asarray(sc, np.float64)[:, None], -448, 448)
                out[name][pg, :, row] = y
            out["acc"][pg, :, row] = 0
            out["ordinal"][pg, :, row] = int(seen[b]) - int(n_new[b]) + t
    return out


def cache_rows(cache, name, b, h):
    """The rows in use of sequence b, kv head h: [lens[b], ...] as values."""
    rows = [cache[name][cache_slot(cache, b, s)[0], h, cache_slot(cache, b, s)[1]]
            for s in range(int(cache["lens"][b]))]
    x = np.array(rows, np.float64).reshape((len(rows),) + cache[name].shape[3:])
    sc = cache.get(name + "_scale")
    return x if sc is None else x * float(sc[h])


def decode_attention(q, cache, scale):
    """q [B, Hq, C] fp64 -> (o [B, Hq, C], lse [B, Hq], w): w[b][h] the weights of kv head
    h's slots, summed over its query heads."""
    B, Hq, C = q.shape
    Hkv = cache["k"].shape[1]
    o, lse = np.zeros((B, Hq, C)), np.full((B, Hq), -np.inf)
    w = [[np.zeros(int(cache["lens"][b])) for _ in range(Hkv)] for b in range(B)]
    for b in range(B):
        if cache["lens"][b] == 0:
            continue
        for kv in range(Hkv):
            k, v = cache_rows(cache, "k", b, kv), cache_rows(cache, "v", b, kv)
            for h in range(kv * Hq // Hkv, (kv + 1) * Hq // Hkv):
                x = scale * (k @ q[b, h])
                top = x.max()
                e = np.exp(x - top)
                lse[b, h] = top + np.log(e.sum())
                p = e / e.sum()
                o[b, h] = p @ v
                w[b][kv] += p
    return o, lse, w


def evict_kept(acc, ordinal, n, seen, recent, sink):
    """The slots that stay, as a set, of one row with len(acc) slots."""
    def order(s):
        safe = ordinal[s] >= seen - recent or ordinal[s] < sink
        a = np.inf if np.isnan(acc[s]) else acc[s]
        return (not safe, 0 if safe else -int(np.isnan(acc[s])), 0.0 if safe else -a, s)
    return set(sorted(range(len(acc)), key=order)[:n])


def cache_evict(cache, budget, recent, sink, seen):
    """The cache after eviction (lens clamped to budget)."""
    out = dict(cache, **{name: cache[name].copy() for name in ("k", "v", "acc", "ordinal")})
    for b in range(len(cache["lens"])):
        length = int(cache["lens"][b])
        n = min(length, budget)
        where = [cache_slot(cache, b, s) for s in range(length)]
        for h in range(cache["k"].shape[1]):
            kept = evict_kept([cache["acc"][pg, h, r] for pg, r in where],
                              [cache["ordinal"][pg, h, r] for pg, r in where], n, int(seen[b]),
                              recent, sink)
            holes = [s for s in range(n) if s not in kept]
            movers = sorted((s for s in kept if s >= n), reverse=True)
            assert len(holes) == len(movers)
            for to, frm in zip(holes, movers):
                for name in ("k", "v", "acc", "ordinal"):
                    out[name][where[to][0], h, where[to][1]] = cache[name][where[frm][0], h, where[frm][1]]
    out["lens"] = np.minimum(cache["lens"], budget)
    return out
