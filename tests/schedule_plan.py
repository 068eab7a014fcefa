"""The split-KV schedule from its definition, in plain Python, and the test
library's host planner of the tree decode's, for the schedule tests.

Tiles of 128 rows lie end to end on a line, each as long as its pages and an
overhead (nothing where it walks no page).  Whole tiles go to the worker whose
even share of the line they begin in, if the longest worker is then within 12
units of that share; else the line is cut at the shares' ends, and an end
inside a tile's overhead moves to the tile's start.
"""
import ctypes

import numpy as np

import mla_latent_space_b200 as mla
from gpu_helpers import test_lib as library

BAD_SEQLEN = 2


def plan(seqlens, s_q, heads, max_pages, workers, overhead=2, causal=False, tree=False, draft_lens=None):
    """int32 words, laid out as mla_get_schedule writes them."""
    rows, cap, flag = s_q * heads, max_pages * 64, 0
    per_req = -(-rows // 128)
    pages = []
    for r, t in enumerate(int(x) for x in seqlens):
        if not 0 <= t <= cap:
            flag, t = BAD_SEQLEN, min(max(t, 0), cap)
        n = min(s_q, t)
        if tree and draft_lens is not None:
            if not 0 <= draft_lens[r] <= n:
                flag = BAD_SEQLEN
            n = min(max(int(draft_lens[r]), 0), n)
        for q in range(per_req):
            last = (min((q + 1) * 128, rows) - 1) // heads
            seen = max(0, t - s_q + last + 1) if causal else t
            pages.append(0 if tree and q * 128 // heads >= n else -(-seen // 64))
    cost = [p + overhead if p else 0 for p in pages]
    prefix = [int(x) for x in np.concatenate([[0], np.cumsum(cost)])]
    total, T = prefix[-1], len(pages)
    We = min(total, workers)
    share = lambda w: total * w // We
    head = np.zeros(16, dtype=np.int64)
    head[:6] = 0x4d4c4131, workers, T, per_req, total, 0
    head[6:12] = flag, len(seqlens), s_q, heads, int(causal), max_pages
    wk, tl = np.zeros((workers, 8), dtype=np.int64), np.zeros((T, 4), dtype=np.int64)
    tl[:, 0], tl[:, 1] = pages, prefix[:-1]
    wk[:, [0, 2]] = T
    first = [next((k for k in range(T) if prefix[k] >= share(w)), T) for w in range(We)] + [T]
    if We:
        longest = max(prefix[first[w + 1]] - prefix[first[w]] for w in range(We))
        even = -(-total // We)
        if tree:
            even = max(even, overhead + 1)
    if We and longest <= even + 12:
        for w in range(We):
            wk[w, 0], wk[w, 2] = first[w], first[w + 1]
        tl[:, 2] = [int(p > 0) for p in pages]
    else:
        start = []
        for w in range(We):
            k = max(k for k in range(T) if prefix[k] <= share(w))
            start.append((k, max(0, share(w) - prefix[k] - overhead)))
        start += [(T, 0)] * (workers + 1 - We)
        inside = [[w for w in range(We) if start[w][0] == k and start[w][1] > 0] for k in range(T)]
        slots = 0
        for k in range(T):
            tl[k, 2] = 1 + len(inside[k]) if pages[k] else 0
            tl[k, 3] = slots
            slots += int(tl[k, 2]) if tl[k, 2] > 1 else 0
        for w in range(workers):
            wk[w, :4] = start[w] + start[w + 1]
            if start[w][1] > 0:
                wk[w, 4] = inside[start[w][0]].index(w) + 1
        head[5] = slots
    return np.concatenate([head, wk.ravel(), tl.ravel()]).astype(np.int32)


def tree_host(shape, seqlens, draft_lens, n_sms):
    fn = library().mla_test_plan_tree_schedule_host
    fn.argtypes = [ctypes.POINTER(mla.mla_shape_t), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                   ctypes.c_size_t]
    fn.restype = ctypes.c_int
    sl = np.ascontiguousarray(seqlens, dtype=np.int32)
    dl = None if draft_lens is None else np.ascontiguousarray(draft_lens, dtype=np.int32)
    out = np.zeros(mla.mla_schedule_bytes(shape, n_sms) // 4, dtype=np.int32)
    assert fn(ctypes.byref(shape), sl.ctypes.data, None if dl is None else dl.ctypes.data, n_sms, out.ctypes.data,
              out.nbytes) == 0
    return out
