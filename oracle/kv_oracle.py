"""Per-head key-value caches: append, one-token attention and eviction by
accumulated attention weight, written out in numpy float64.

Keys and values are [pages, page_size, heads, d]; `table` is an [n_seq, max_pages]
page table or None (sequence b is page b).  The eight-KV-head cache is the
baseline of the DeepSeek-V4 book, Ch.8 "A Cost Model for Long Context"; the
eviction rule and the hole filling are this library's own.
"""
from __future__ import annotations

import numpy as np


def kv_place(table, page_size, b, s):
    """(page, row) of slot s of sequence b."""
    if table is None:
        return b, s
    return int(table[b, s // page_size]), s % page_size


def kv_rows(x, table, b, n):
    """Slots 0 .. n-1 of sequence b: [n, heads, d] float64."""
    out = np.zeros((n,) + x.shape[2:])
    for s in range(n):
        page, row = kv_place(table, x.shape[1], b, s)
        out[s] = x[page, row]
    return out


def kv_append(k, v, table, lens, k_new, v_new, start=None, weights=None, slot_pos=None, pos=None):
    """Returns copies (k, v, lens, weights, slot_pos) after the append."""
    k, v, lens = k.copy(), v.copy(), np.array(lens).copy()
    weights = None if weights is None else weights.copy()
    slot_pos = None if slot_pos is None else slot_pos.copy()
    room = (1 if table is None else table.shape[1]) * k.shape[1]
    for a in (weights, slot_pos):
        if a is not None:
            room = min(room, a.shape[-1])
    for b in range(len(lens)):
        first, end = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        n = int(lens[b])
        for i, t in enumerate(range(first, end)):
            if n + i >= room:
                break
            page, row = kv_place(table, k.shape[1], b, n + i)
            k[page, row], v[page, row] = k_new[t], v_new[t]
            if weights is not None:
                weights[b, :, n + i] = 0
            if slot_pos is not None:
                slot_pos[b, :, n + i] = pos[b] + i
        lens[b] = min(n + end - first, room)
    return k, v, lens, weights, slot_pos


def kv_attend(q, k, v, table, lens, scale, window=0, sink=None):
    """Returns out [B, H, d], lse [B, H], prob: a list of [H, n] per sequence
    (zero before the window)."""
    B, H, d = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    out, lse, prob = np.zeros((B, H, d)), np.full((B, H), -np.inf), []
    for b in range(B):
        n = int(lens[b])
        kb, vb = kv_rows(k, table, b, n), kv_rows(v, table, b, n)
        lo = max(0, n - window) if window else 0
        pb = np.zeros((H, n))
        for h in range(H):
            z = scale * (kb[lo:, h // G] @ q[b, h])
            terms = z if sink is None else np.append(z, sink[h])
            if terms.size:
                top = terms.max()
                lse[b, h] = top + np.log(np.exp(terms - top).sum())
                pb[h, lo:] = np.exp(z - lse[b, h])
                out[b, h] = pb[h, lo:] @ vb[lo:, h // G]
        prob.append(pb)
    return out, lse, prob


def kv_weigh(weights, prob, n_kv_heads):
    """weights [B, heads, slots] plus each slot's probabilities summed over the group."""
    out = np.array(weights, dtype=np.float64)
    for b, p in enumerate(prob):
        out[b, :, :p.shape[1]] += p.reshape(n_kv_heads, p.shape[0] // n_kv_heads, p.shape[1]).sum(1)
    return out


def kv_evict(k, v, table, lens, weights, slot_pos, pos, budget, recent, keep_first=0, max_len=None, inplace=False):
    """Returns copies (k, v, lens, weights, slot_pos, src); weights and positions
    from the old length on are zero, or in place as they were."""
    k, v = k.copy(), v.copy()
    B, heads, slots = weights.shape
    max_len = slots if max_len is None else max_len
    w_out, p_out = weights.copy(), slot_pos.copy()
    src = np.full((B, heads, budget), -1, dtype=np.int64)
    new = np.minimum(lens, budget)
    for b in range(B):
        n = int(lens[b])
        for h in range(heads):
            def better(j):   # sorts first what stays
                held = slot_pos[b, h, j] > int(pos[b]) - recent or slot_pos[b, h, j] < keep_first
                w = weights[b, h, j]
                if held:
                    return (0, 0.0, j)
                return (1, 0.0, j) if np.isnan(w) else (2, -float(w) if w != 0 else 0.0, j)
            stay = sorted(sorted(range(n), key=better)[:budget])
            came = dict((j, j) for j in stay if j < budget)
            holes = [j for j in range(int(new[b])) if j not in came]
            came.update(zip(holes, [j for j in stay if j >= budget]))
            end = n if inplace else max_len
            w_out[b, h, :end] = 0
            p_out[b, h, :end] = 0
            for to, j in came.items():
                w_out[b, h, to], p_out[b, h, to], src[b, h, to] = weights[b, h, j], slot_pos[b, h, j], j
                if to != j:
                    at, frm = kv_place(table, k.shape[1], b, to), kv_place(table, k.shape[1], b, j)
                    k[at[0], at[1], h], v[at[0], at[1], h] = k[frm[0], frm[1], h], v[frm[0], frm[1], h]
    return k, v, new, w_out, p_out, src
