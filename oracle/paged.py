"""Paged-cache bookkeeping, block bounds, block choice and plain decode attention (fp64, loops).

Definitions (R = reading where the pages are silent; the pages describe none of the addressing):
  slots     slot(b, h, t) = (block_table[b, t // B] * Hkv + h) * B + t % B
  growth    sequence b takes ceil((len + new) / B) - ceil(len / B) blocks, in the order of the
            sequences, from one free list; a sequence that does not fit is refused whole (R)
  bounds    the channel minimum and maximum of the keys of one block and KV head
  score     max over the query heads of the KV head of sum_c max(q_c lower_c, q_c upper_c), an upper
            bound of every key's inner product with the query
  choice    first n_first and last n_last blocks, the best others by (score descending, index
            ascending), listed in the order of the sequence
  attention o = softmax(scale q K^T) V; no tokens give 0 (R)

Pinned by tests/test_oracle_paged.py.
"""
from __future__ import annotations

import math

import numpy as np


def extend(table, lens, new, free, head, n_rows, n_kv, block, n_blocks):
    """Returns (table, lens, granted, head, row offsets, slots [n_rows * n_kv])."""
    table, lens = np.array(table), [max(int(x), 0) for x in lens]
    new = [max(int(x), 0) for x in new]
    most = table.shape[1] * block
    granted, offsets, wanted, taken = [], [0], 0, 0
    slots = np.full((n_rows, n_kv), -1, dtype=np.int64)
    for b, (n, m) in enumerate(zip(lens, new)):
        row = offsets[-1]
        offsets.append(row + m)
        if n + m > most or row + m > n_rows:
            granted.append(0)
            continue
        have, need = -(-n // block), -(-(n + m) // block) - -(-n // block)
        wanted += need
        if need > 0 and head + wanted > len(free):
            granted.append(0)
            continue
        table[b, have:have + need] = free[head + wanted - need:head + wanted]
        taken += need
        granted.append(m)
        for i in range(m):
            e = int(table[b, (n + i) // block])
            if 0 <= e < n_blocks:
                for h in range(n_kv):
                    slots[row + i, h] = (e * n_kv + h) * block + (n + i) % block
    return (table, np.array([n + g for n, g in zip(lens, granted)]), np.array(granted), head + taken, np.array(offsets),
            slots.reshape(-1))


def append(table, lens, granted, offsets, k, v, k_cache, v_cache, bounds, block):
    """Caches [n_blocks, n_kv, block, d] and bounds [n_blocks, n_kv, 2, d] after the append (copies)."""
    k_cache, v_cache, bounds = np.array(k_cache), np.array(v_cache), np.array(bounds)
    for b, (n, m) in enumerate(zip(lens, granted)):
        for i in range(m):
            t = n - m + i
            e = int(table[b][t // block])
            if not 0 <= e < k_cache.shape[0]:
                continue
            row = offsets[b] + i
            k_cache[e, :, t % block], v_cache[e, :, t % block] = k[row], v[row]
            if t % block == 0:
                bounds[e, :, 0], bounds[e, :, 1] = k[row], k[row]
            bounds[e, :, 0] = np.minimum(bounds[e, :, 0], k[row])
            bounds[e, :, 1] = np.maximum(bounds[e, :, 1], k[row])
    return k_cache, v_cache, bounds


def block_scores(table, lens, q, bounds, block):
    """[batch * n_kv, max_blocks]; -inf past the last block and for entries that name no block."""
    batch, width = np.shape(table)
    n_blocks, n_kv = bounds.shape[:2]
    group = q.shape[1] // n_kv
    out = np.full((batch * n_kv, width), -np.inf)
    for b in range(batch):
        for j in range(min(width, -(-max(int(lens[b]), 0) // block))):
            e = int(table[b][j])
            if not 0 <= e < n_blocks:
                continue
            for h in range(n_kv):
                x = q[b, h * group:(h + 1) * group]
                out[b * n_kv + h, j] = np.maximum(x * bounds[e, h, 0], x * bounds[e, h, 1]).sum(1).max()
    return out


def select(table, lens, scores, n_kv, block, n_blocks, keep, first, last):
    """Block table [batch * n_kv, keep] of one-head sequences and the tokens in it."""
    batch, width = np.shape(table)
    out = np.full((batch * n_kv, keep), -1, dtype=np.int64)
    held = np.zeros(batch * n_kv, dtype=np.int64)
    for r in range(batch * n_kv):
        b, h = divmod(r, n_kv)
        n_tok = min(max(int(lens[b]), 0), width * block)
        n = -(-n_tok // block)
        if n == 0:
            continue
        chosen = list(range(n))
        if n > keep:
            rest = sorted(range(first, n - last), key=lambda j: (-scores[r, j] if scores[r, j] == scores[r, j] else math.inf, j))
            chosen = sorted(list(range(first)) + list(range(n - last, n)) + rest[:keep - first - last])
        for i, j in enumerate(chosen):
            e = int(table[b][j])
            out[r, i] = e * n_kv + h if 0 <= e < n_blocks else -1
        held[r] = (len(chosen) - 1) * block + n_tok - (n - 1) * block
    return out, held


def attend(table, lens, q, k_cache, v_cache, block, scale=0.0):
    """[batch, n_q, d] from caches [n_blocks, n_kv, block, d]."""
    batch, n_q, d = q.shape
    n_blocks, n_kv = k_cache.shape[:2]
    group = n_q // n_kv
    scale = scale if scale != 0.0 else 1.0 / math.sqrt(d)
    out = np.zeros((batch, n_q, d))
    for b in range(batch):
        t = np.arange(max(int(lens[b]), 0))
        e = np.asarray(table[b], dtype=np.int64)[t // block]
        ok = (e >= 0) & (e < n_blocks)
        t, e = t[ok] % block, e[ok]
        if len(t) == 0:
            continue
        for hq in range(n_q):
            k, v = k_cache[e, hq // group, t], v_cache[e, hq // group, t]
            s = scale * (k @ q[b, hq])
            w = np.exp(s - s.max())
            out[b, hq] = (w / w.sum()) @ v
    return out
