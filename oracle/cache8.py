"""The 8-bit block cache in double precision: append, attention, accumulated
weights and eviction, from their definitions, and attention over packed
sequences of different lengths.

TEST INFRASTRUCTURE ONLY (see the package docstring): the library never
imports this module.

A cache is a dict of numpy arrays: k, v uint8 e4m3 codes [P, Hkv, 64, d],
k_scale, v_scale float32 [P, Hkv], weight float32 [P, Hkv, 64]. A block table is
int [B, max_blocks]; entries outside [0, P) stand for no block. Every function
returns new arrays and leaves its arguments alone.

Pins: tests/test_oracle_cache8.py (a dense attention for one sequence in
order, brute force for the scale, sorting in Python for the eviction).
"""
import numpy as np

from .attention import forward
from .fp8 import e4m3_decode, e4m3_encode

BLOCK = 64


def power_scale(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s; 1 for 0."""
    if amax == 0:
        return 1.0
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def encode(x, s):
    """e4m3 codes of x / s; infinities held at 448, NaN kept (0x7F)."""
    y = np.asarray(x, np.float64) / s
    nan = np.isnan(y)
    y = np.clip(np.where(nan, 0.0, y), -448.0, 448.0).astype(np.float32)
    return np.where(nan, np.uint8(0x7F), e4m3_encode(y)).astype(np.uint8)


def _finite_max(x):
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    return a.max() if a.size else 0.0


def append(cache, k, v, cu, start, table):
    """k, v [Hkv, T, d] float values of the new tokens."""
    c = {n: x.copy() for n, x in cache.items()}
    P, Hkv = c["k_scale"].shape
    for b in range(len(start)):
        first = {}                                   # block index -> list of (slot, token)
        for i, tok in enumerate(range(cu[b], cu[b + 1])):
            pos = start[b] + i
            if pos < table.shape[1] * BLOCK:
                first.setdefault(pos // BLOCK, []).append((pos % BLOCK, tok))
        for blk, items in first.items():
            page = table[b, blk]
            if not 0 <= page < P:
                continue
            slots, toks = np.array([s for s, _ in items]), np.array([t for _, t in items])
            lo = slots[0]
            for h in range(Hkv):
                for name, x in (("k", k), ("v", v)):
                    new = np.asarray(x, np.float64)[h, toks]
                    amax = _finite_max(new)
                    old = float(c[name + "_scale"][page, h])
                    if lo == 0:
                        now = power_scale(amax)
                    else:
                        now = max(old, power_scale(amax)) if amax > 0 else old
                        if now != old:
                            held = e4m3_decode(c[name][page, h, :lo])
                            c[name][page, h, :lo] = encode(held * (old / now), 1.0)
                    c[name + "_scale"][page, h] = now
                    c[name][page, h, slots] = encode(new, now)
                if c.get("weight") is not None:
                    c["weight"][page, h, slots] = 0
    return c


def gather(cache, table_row, h, n):
    """K and V values [n, d] float64 of one sequence and head, and the
    positions that exist (a table entry outside the pool has no tokens)."""
    P = cache["k"].shape[0]
    pos = np.arange(n)
    page = np.asarray(table_row)[pos // BLOCK]
    there = (page >= 0) & (page < P)
    pos, page = pos[there], page[there]
    out = [e4m3_decode(cache[x][page, h, pos % BLOCK]) * cache[x + "_scale"][page, h][:, None].astype(np.float64)
           for x in ("k", "v")]
    return out[0], out[1], pos


def attend(cache, q, table, lengths, causal, scale):
    """O [B, Hq, Nq, d], LSE [B, Hq, Nq] and the summed probabilities as a list
    over sequences of [Hkv, positions] arrays."""
    B, Hq, Nq, d = q.shape
    Hkv = cache["k"].shape[1]
    G = Hq // Hkv
    O = np.zeros(q.shape)
    lse = np.full((B, Hq, Nq), -np.inf)
    sums = []
    for b in range(B):
        n = int(min(max(lengths[b], 0), table.shape[1] * BLOCK))
        w = np.zeros((Hkv, n))
        for h in range(Hkv):
            K, V, pos = gather(cache, table[b], h, n)
            for r in range(Nq):
                seen = pos <= r + n - Nq if causal else np.ones(len(pos), bool)
                if not seen.any():
                    continue
                for j in range(h * G, (h + 1) * G):
                    s = scale * (K[seen] @ q[b, j, r])
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    O[b, j, r] = p @ V[seen] / l
                    lse[b, j, r] = m + np.log(l)
                    w[h, pos[seen]] += p / l
        sums.append(w)
    return O, lse, sums


def add_weights(cache, sums, table, lengths, decay):
    """The weight pool after an attention with weights."""
    w = cache["weight"].astype(np.float64).copy()
    P = w.shape[0]
    for b, x in enumerate(sums):
        for i in range(x.shape[1]):
            page = table[b, i // BLOCK]
            if 0 <= page < P:
                old = decay * w[page, :, i % BLOCK] if decay else 0.0
                w[page, :, i % BLOCK] = old + x[:, i]
    return w


def choose(weights, keep, recent):
    """Positions kept of len(weights) tokens, ascending."""
    n = len(weights)
    if n <= keep:
        return list(range(n))
    old = n - recent
    key = [np.inf if np.isnan(x) else float(x) for x in weights[:old]]
    nan = [bool(np.isnan(x)) for x in weights[:old]]
    order = sorted(range(old), key=lambda i: (not nan[i], -key[i], i))
    return sorted(order[: keep - recent]) + list(range(old, n))


def evict(cache, table, lengths, keep, recent, to_table):
    c = {n: x.copy() for n, x in cache.items()}
    B = len(lengths)
    P, Hkv = c["k_scale"].shape
    kept = np.full((B, Hkv, keep), -1, np.int32)
    new = np.array([min(max(int(x), 0), table.shape[1] * BLOCK) for x in lengths])
    for b in range(B):
        n = new[b]
        for h in range(Hkv):
            page = table[b, np.arange(n) // BLOCK]
            ok = (page >= 0) & (page < P)
            slot = np.arange(n) % BLOCK
            w = np.where(ok, cache["weight"][np.where(ok, page, 0), h, slot], 0.0)
            pick = np.array(choose(w, keep, recent), int)
            kept[b, h, : len(pick)] = pick
            for j in range(0, len(pick), BLOCK):
                part, to = pick[j:j + BLOCK], to_table[b, j // BLOCK]
                if not 0 <= to < P:
                    continue
                m = len(part)
                for name in ("k", "v"):
                    src = np.where(ok[part], page[part], 0)
                    x = e4m3_decode(cache[name][src, h, slot[part]]) * cache[name + "_scale"][src, h][:, None].astype(np.float64)
                    x = np.where(ok[part][:, None], x, 0.0)
                    s = power_scale(_finite_max(x))
                    c[name][to, h, :m] = encode(x, s)
                    c[name + "_scale"][to, h] = s
                c["weight"][to, h, :m] = np.where(ok[part], w[part], 0.0)
    return c, np.minimum(new, keep).astype(np.int32), kept


def packed(q, k, v, cu, causal, scale):
    """O [Hq, T, d] and LSE [Hq, T] of sequences cu[s] .. cu[s + 1] - 1 of
    packed q [Hq, T, d], k, v [Hkv, T, d]; NaN in rows of no sequence."""
    O = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for a, e in zip(cu[:-1], cu[1:]):
        if e > a:
            o1, l1 = forward(q[None, :, a:e], k[None, :, a:e], v[None, :, a:e], causal, scale)
            O[:, a:e], lse[:, a:e] = o1[0], l1[0]
    return O, lse
