"""fp64 CPU oracle of the operators that draft into, weigh, cut and close up
the paged cache.  TEST INFRASTRUCTURE ONLY, as the rest of this package.

  tree_mask     node i of a drafted tree sees itself and its ancestors
  tree_decode   every node sees the committed prefix and, among the drafted
                tokens, those of its mask row; softmax attention as `attend`
  attn_weights  w_j = decay w_j + sum over the query rows that see j of
                exp(scale q . C_j - lse)
  evict_select  the first `sink`, the last `recent` and the heaviest of the
                rest (ties: the lowest position; NaN: lightest), ascending
  compact       row at src[k] -> position base + k, in order
"""
from __future__ import annotations

import numpy as np

from .mla_decode import D_QK, D_V, PAGE, attend, bf16_to_f64, gather_rows, visible_len


def tree_mask(parents: np.ndarray, lens=None) -> np.ndarray:
    """Ancestor bits int64 [b, s, ceil(s / 64)] of parents int [b, s]."""
    b, s = parents.shape
    out = np.zeros((b, s, (s + 63) // 64), dtype=np.uint64)
    for r in range(b):
        n = s if lens is None else max(0, min(int(lens[r]), s))
        for i in range(n):
            j = i
            while True:
                out[r, i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
                p = int(parents[r, j])
                if not 0 <= p < j:
                    break
                j = p
    return out.view(np.int64)


def mask_bit(mask: np.ndarray, r: int, i: int, d: int) -> bool:
    return bool((int(mask[r, i, d // 64]) >> (d % 64)) & 1)


def tree_decode(wl, mask: np.ndarray, lens=None):
    """(O float64 [b, s, h, 512], lse float64 [b, s, h])."""
    b, s, h, _ = wl.q.shape
    O = np.zeros((b, s, h, D_V))
    L = np.full((b, s, h), -np.inf)
    for r in range(b):
        t = int(wl.seqlens[r])
        n = min(s, t) if lens is None else max(0, min(int(lens[r]), s, t))
        C = gather_rows(wl.pool, wl.block_table, r, t, wl.kv_scale)
        for i in range(n):
            seen = np.concatenate([np.arange(t - n), [t - n + d for d in range(n) if mask_bit(mask, r, i, d)]]).astype(int)
            O[r, i], L[r, i] = attend(bf16_to_f64(wl.q[r, i]), C[seen] if len(seen) else np.zeros((0, D_QK)),
                                      wl.softmax_scale)
    return O, L


def attn_weights(wl, lse: np.ndarray, decay: float, old: np.ndarray) -> np.ndarray:
    """float64 [b, max_pages * 64]; rows of lse = -inf add nothing."""
    b, s, h, _ = wl.q.shape
    w = old.astype(np.float64).copy()
    for r in range(b):
        t = int(wl.seqlens[r])
        C = gather_rows(wl.pool, wl.block_table, r, t, wl.kv_scale)
        new = np.zeros(t)
        for i in range(s):
            k = max(0, visible_len(t, s, i, wl.causal))
            adds = lse[r, i] != -np.inf
            x = wl.softmax_scale * (C[:k] @ bf16_to_f64(wl.q[r, i])[adds].T)
            new[:k] += np.exp(x - lse[r, i][adds].astype(np.float64)).sum(axis=1)
        w[r, :t] = (decay * w[r, :t] if decay != 0.0 else 0.0) + new
    return w


def evict_select(w: np.ndarray, seqlens, budget: int, sink: int, recent: int):
    """(kept int32 [b, budget] ascending then -1, lens int32 [b])."""
    b = w.shape[0]
    kept = np.full((b, budget), -1, dtype=np.int32)
    lens = np.zeros(b, dtype=np.int32)
    for r in range(b):
        t = max(0, min(int(seqlens[r]), w.shape[1]))
        if t <= budget:
            stay = list(range(t))
        else:
            mid = range(sink, t - recent)
            key = lambda j: (0, 0.0) if np.isnan(w[r, j]) else (1, float(w[r, j]))
            heavy = sorted(mid, key=lambda j: (tuple(-x for x in key(j)), j))[:budget - sink - recent]
            stay = sorted(list(range(sink)) + heavy + list(range(t - recent, t)))
        kept[r, :len(stay)] = stay
        lens[r] = len(stay)
    return kept, lens


def compact(pool, kv_scale, block_table, src, lens, base=None, weights=None):
    """The cache (torch, as the workload holds it) with every listed row moved;
    returns (pool, kv_scale, weights), copies."""
    fp8 = kv_scale is not None
    new, new_scale = pool.clone(), None if not fp8 else kv_scale.clone()
    new_w = None if weights is None else weights.copy()
    for r in range(len(lens)):
        for k in range(int(lens[r])):
            a, d = int(src[r, k]), k + (0 if base is None else int(base[r]))
            pa, ia, pd, id_ = int(block_table[r][a // PAGE]), a % PAGE, int(block_table[r][d // PAGE]), d % PAGE
            if fp8:
                lat = PAGE * D_V
                new[pd, id_ * D_V:(id_ + 1) * D_V] = pool[pa, ia * D_V:(ia + 1) * D_V]
                new[pd, lat + id_ * 128:lat + (id_ + 1) * 128] = pool[pa, lat + ia * 128:lat + (ia + 1) * 128]
                new_scale[pd, id_] = kv_scale[pa, ia]
            else:
                new[pd, id_] = pool[pa, ia]
            if new_w is not None:
                new_w[r, d] = weights[r, a]
    return new, new_scale, new_w
