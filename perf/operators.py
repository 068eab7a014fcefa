"""Cases of the operators around a paged latent cache that drafts, verifies and evicts.

Four operators, over the paged cache of one latent row (512 latent + 64 RoPE values) per token:

  tree     attention of a tree of drafted tokens: every drafted node sees the whole committed prefix and, among the
           drafted tokens, the ones its mask row names (its ancestors and itself)
  weights  the attention weight that each cached token received from a step's query rows, accumulated over steps
  select   which tokens of each request stay: the first few, the last few, and the heaviest of the rest
  compact  the kept (or accepted) rows moved to the front of the request's own pages, in order

`run` computes them with elementary torch operations, or, where `own` is true, with the calls of the library.
"""
import math

import torch

own = False

PAGE, D_QK, D_V, D_ROPE = 64, 576, 512, 64
FP8_LATENT = PAGE * D_V                       # bytes of a page's e4m3 plane; its bf16 RoPE plane follows
SCALE = 1.0 / math.sqrt(192.0)
LOG_RANGE = {"tree": (64, 16384), "weights": (64, 32768), "select": (256, 131072), "compact": (256, 65536)}


def listed():
    return [
        # a small tree at a batch of two short requests, on one rank of a model split over its heads: launch latency
        dict(name="tree_tiny", op="tree", batch=2, heads=16, s_q=8, t_lo=200, t_hi=256, cache="bf16", ragged=False, parents=False),
        # a verification step on the same rank with a serving batch, trees of different sizes, the masks built from
        # the parents in the step itself
        dict(name="tree_rank", op="tree", batch=32, heads=16, s_q=24, t_lo=500, t_hi=8192, cache="bf16", ragged=True, parents=True),
        # the speculative workload with a tree in the place of its chain: all heads, 16 nodes a request
        dict(name="tree_spec", op="tree", batch=32, heads=128, s_q=16, t_lo=4096, t_hi=4096, cache="bf16", ragged=False, parents=False),
        # all heads over an 8-bit cache, an odd number of nodes, lengths that differ
        dict(name="tree_fp8", op="tree", batch=16, heads=128, s_q=13, t_lo=1000, t_hi=16384, cache="fp8", ragged=True, parents=False),
        # the weights of one decode step of the serving batch: every cached row is read once
        dict(name="weights_decode", op="weights", batch=64, heads=128, s_q=1, t_lo=4096, t_hi=4096, cache="bf16", causal=False, decay=0.9),
        # the same over a long 8-bit cache
        dict(name="weights_fp8", op="weights", batch=16, heads=128, s_q=1, t_lo=20000, t_hi=32768, cache="fp8", causal=False, decay=1.0),
        # the window of a prompt's last queries, by which a prompt's cache is cut before the first decode step
        dict(name="weights_window", op="weights", batch=4, heads=128, s_q=16, t_lo=1000, t_hi=16384, cache="bf16", causal=True, decay=0.0),
        # a serving batch that has reached its budget
        dict(name="select_batch", op="select", batch=64, t_lo=3000, t_hi=4096, budget=1024, sink=4, recent=64),
        # two long contexts cut to a sixteenth
        dict(name="select_long", op="select", batch=2, t_lo=100000, t_hi=131072, budget=8192, sink=4, recent=256),
        # half of every request's rows go, the rest close up; their weights go with them
        dict(name="compact_evict", op="compact", batch=64, t_lo=4000, t_hi=4096, rows=2048, cache="bf16", base=False, weights=True),
        # long 8-bit caches cut to a quarter
        dict(name="compact_fp8", op="compact", batch=4, t_lo=50000, t_hi=65536, rows=16384, cache="fp8", base=False, weights=False),
        # after a verification step: the accepted path of each request's tree closes up behind its prefix
        dict(name="compact_accept", op="compact", batch=32, t_lo=1000, t_hi=4096, rows=16, cache="bf16", base=True, weights=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "weights", "select", "compact"])
    lo, hi = LOG_RANGE[op]
    t_hi = _log_int(rng, lo, hi)
    t_lo = max(lo // 2, int(t_hi * rng.uniform(0.1, 1.0)))
    cache = rng.choice(["bf16", "fp8"])
    if op in ("tree", "weights"):
        heads = rng.choice([5, 16, 16, 32, 40, 64, 128, 128])
        s_q = _log_int(rng, 1, 64 if op == "tree" else 32)
        batch = _log_int(rng, 1, 64)
        rows = 32 * 16 * 128 * 4096 if op == "tree" else 4 * 16 * 128 * 16384
        batch = max(1, min(batch, rows // (s_q * heads * t_hi), 262144 // t_hi))     # neither dearer nor larger than listed
        if op == "tree":
            return dict(op=op, batch=batch, heads=heads, s_q=s_q, t_lo=max(t_lo, s_q), t_hi=max(t_hi, s_q), cache=cache,
                        ragged=rng.random() < 0.5, parents=rng.random() < 0.5)
        return dict(op=op, batch=batch, heads=heads, s_q=s_q, t_lo=max(t_lo, s_q), t_hi=max(t_hi, s_q), cache=cache,
                    causal=rng.random() < 0.5, decay=rng.choice([0.0, 0.5, 0.9, 1.0]))
    batch = max(1, min(_log_int(rng, 1, 128), 262144 // t_hi))
    if op == "select":
        budget = max(1, int(t_hi * rng.uniform(0.05, 1.1)))
        sink = min(budget, rng.choice([0, 1, 4, 16]))
        return dict(op=op, batch=batch, t_lo=t_lo, t_hi=t_hi, budget=budget, sink=sink,
                    recent=min(budget - sink, rng.choice([0, 1, 32, 100, 256])))
    base = rng.random() < 0.4
    rows = _log_int(rng, 2, 64) if base else max(1, int(t_lo * rng.uniform(0.05, 1.0)))
    return dict(op=op, batch=batch, t_lo=t_lo, t_hi=t_hi, rows=rows, cache=cache, base=base, weights=rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, g):
    """Lengths spread over [t_lo, t_hi] by their logarithm, the longest among them."""
    u = torch.rand(case["batch"], generator=g, device="cuda", dtype=torch.float64)
    t = torch.exp(math.log(case["t_lo"]) + u * (math.log(case["t_hi"]) - math.log(case["t_lo"]))).round()
    t[0] = case["t_hi"]
    return t.to(torch.int32)


def _cache(case, g, seqlens):
    """A pool of pages in random order; the slots behind a request's last token hold NaN, as freed pages may."""
    b, pages = case["batch"], (case["t_hi"] + PAGE - 1) // PAGE
    table = torch.randperm(b * pages, generator=g, device="cuda").to(torch.int32).view(b, pages)
    n = b * pages
    spare = torch.empty((n, PAGE), dtype=torch.bool, device="cuda")
    spare[table.long().view(-1)] = (torch.arange(pages * PAGE, device="cuda") >= seqlens[:, None]).view(n, PAGE)
    if case.get("cache", "bf16") == "bf16":
        pool = torch.empty((n, PAGE, D_QK), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        pool.masked_fill_(spare[:, :, None], float("nan"))
        return table, pool, None
    pool = torch.empty((n, FP8_LATENT + PAGE * D_ROPE * 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n, PAGE), dtype=torch.float32, device="cuda")
    step = 512
    for i in range(0, n, step):
        x = torch.empty((min(step, n - i), PAGE, D_QK), dtype=torch.float32, device="cuda").normal_(generator=g).bfloat16().float()
        s = x[:, :, :D_V].abs().amax(2) / 448.0
        lat = (x[:, :, :D_V] / s[:, :, None]).to(torch.float8_e4m3fn)
        bytes_ = lat.view(torch.uint8).masked_fill(spare[i:i + step, :, None], 0x7F)
        pool[i:i + step, :FP8_LATENT] = bytes_.reshape(-1, FP8_LATENT)
        pool[i:i + step, FP8_LATENT:] = x[:, :, D_V:].bfloat16().contiguous().view(torch.uint8).reshape(x.shape[0], -1)
        scale[i:i + step] = s
    return table, pool, scale


def _queries(case, g):
    shape = (case["batch"], case["s_q"], case["heads"], D_QK)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _parents(case, g):
    """Node i's parent: one of the nodes before it, or -1 (the committed prefix)."""
    i = torch.arange(case["s_q"], device="cuda")
    u = torch.rand((case["batch"], case["s_q"]), generator=g, device="cuda")
    return ((u * (i + 1)).floor().long() - 1).minimum(i - 1).to(torch.int32)


def _ancestors(parents):
    """bool [b, s, s]: whether node j is i or an ancestor of i."""
    s = parents.shape[1]
    eye = torch.eye(s, device=parents.device)
    step = (parents[:, :, None] == torch.arange(s, device=parents.device)).float()
    return torch.linalg.matrix_power(eye + step, s) > 0


def _pack(seen):
    """bool [b, s, s] -> int64 [b, s, ceil(s / 64)], bit j % 64 of word j // 64."""
    b, s, _ = seen.shape
    words = (s + 63) // 64
    bits = torch.nn.functional.pad(seen, (0, words * 64 - s)).view(b, s, words, 64)
    return (bits.long() << torch.arange(64, device=seen.device)).sum(3)


def prepare(case, seed):
    g = _gen(seed)
    op, b = case["op"], case["batch"]
    seqlens = _lengths(case, g)
    st = dict(case=case, seqlens=seqlens)
    if op == "select":
        T = (case["t_hi"] + PAGE - 1) // PAGE * PAGE
        # weights span many powers of two, and equal ones are common among the light tokens
        w = torch.exp(4.0 * torch.empty((b, T), device="cuda").normal_(generator=g) - 6.0)
        w = torch.where(w < 1e-3, torch.zeros_like(w), w)
        st.update(weights=w, kept=torch.empty((b, case["budget"]), dtype=torch.int32, device="cuda"),
                  kept_lens=torch.empty(b, dtype=torch.int32, device="cuda"))
    else:
        st["table"], st["pool"], st["scale"] = _cache(case, g, seqlens)
    if op in ("tree", "weights"):
        st["q"] = _queries(case, g)
        st["out_shape"] = (b, case["s_q"], case["heads"])
    if op == "tree":
        s = case["s_q"]
        st["parents"] = _parents(case, g)
        lens = torch.randint(0 if s > 1 else 1, s + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        st["draft_lens"] = torch.minimum(lens, seqlens) if case["ragged"] else None
        st["out"] = torch.empty((b, s, case["heads"], D_V), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((b, s, case["heads"]), dtype=torch.float32, device="cuda")
        st["mask"] = torch.zeros((b, s, (s + 63) // 64), dtype=torch.int64, device="cuda")
        if not case["parents"]:
            st["mask"].copy_(_pack(_ancestors(st["parents"]) & _within(st)[:, :, None]))
    if op == "weights":
        st["lse"] = torch.logsumexp(_scores(st), -1).view(st["out_shape"])
        st["weights"] = torch.rand((b, st["table"].shape[1] * PAGE), generator=g, device="cuda")
    if op == "compact":
        R = case["rows"]
        if case["base"]:       # a path of each request's last R tokens, at least one node of it
            n = torch.minimum(torch.randint(1, R + 1, (b,), generator=g, device="cuda"), seqlens.long())
            span = torch.minimum(torch.full_like(n, R), seqlens.long())
            first = seqlens.long() - span
        else:
            n = torch.minimum(torch.full((b,), R, device="cuda"), seqlens.long())
            span, first = seqlens.long(), torch.zeros_like(seqlens).long()
        key = torch.rand((b, case["t_hi"]), generator=g, device="cuda")
        key = torch.where(torch.arange(case["t_hi"], device="cuda") < span[:, None], key, key + 2.0)
        pick = key.argsort(1)[:, :R]
        pick = torch.where(torch.arange(pick.shape[1], device="cuda") < n[:, None], pick, torch.full_like(pick, 1 << 30))
        src = pick.sort(1).values + first[:, None]
        st["src"] = torch.where(src < (1 << 29), src, torch.full_like(src, -1)).to(torch.int32).contiguous()
        st["src_lens"] = n.to(torch.int32)
        st["base"] = first.to(torch.int32) if case["base"] else None
        st["weights"] = torch.rand((b, st["table"].shape[1] * PAGE), generator=g, device="cuda") if case["weights"] else None
    if own:
        import mla_latent_space_b200 as mla
        st["mla"] = mla
        if op != "select":
            st["shape"] = mla.make_shape(b, case.get("s_q", 1), case.get("heads", 1), st["table"].shape[1], st["pool"].shape[0],
                                         case["cache"], case.get("causal", False))
        if op == "tree":
            st["decoder"] = mla.TreeDecoder(st["shape"])
        if op == "weights":
            st["attn"] = mla.AttnWeights(st["shape"])
        if op == "compact":
            st["compactor"] = mla.CacheCompactor(st["shape"], st["src"].shape[1])
    return st


# ---- plain forms ------------------------------------------------------------

def _rows(st):
    """Every request's cached rows, fp32 [b, T, 576] (zeros behind the last token)."""
    table, pool = st["table"].long(), st["pool"]
    b = table.shape[0]
    if st["scale"] is None:
        x = pool[table].view(b, -1, D_QK).float()
    else:
        lat = pool[:, :FP8_LATENT].view(torch.float8_e4m3fn).view(-1, PAGE, D_V).float() * st["scale"][:, :, None]
        rope = pool[:, FP8_LATENT:].view(torch.bfloat16).view(-1, PAGE, D_ROPE).float()
        x = torch.cat([lat, rope], 2)[table].view(b, -1, D_QK)
    live = torch.arange(x.shape[1], device=x.device) < st["seqlens"][:, None]
    return x.masked_fill_(~live[:, :, None], 0.0)


def _draft_lens(st):
    n = st["draft_lens"]
    return torch.clamp(st["seqlens"], max=st["case"]["s_q"]) if n is None else n


def _within(st):
    """bool [b, s]: which node slots of each request hold a node."""
    return torch.arange(st["case"]["s_q"], device="cuda") < _draft_lens(st)[:, None]


def _seen(st, T):
    """bool [b, s, T]: which positions each query token sees."""
    case, t = st["case"], st["seqlens"][:, None, None]
    pos = torch.arange(T, device="cuda")
    if case["op"] == "weights":
        i = torch.arange(case["s_q"], device="cuda")[:, None]
        return pos < (t - case["s_q"] + i + 1 if case["causal"] else t + 0 * i)
    n = _draft_lens(st)[:, None, None]
    d = pos - (t - n)                                                  # the position's place among the drafted tokens
    dc = d.clamp(0, case["s_q"] - 1).expand(-1, case["s_q"], -1)
    bit = (st["mask"].gather(2, dc // 64) >> (dc % 64)) & 1
    return ((d < 0) | ((d < n) & (bit == 1))) & _within(st)[:, :, None]


def _scores(st, rows=None):
    """Scaled scores fp32 [b, s * h, T], minus infinity where a row does not see the position."""
    case = st["case"]
    rows = _rows(st) if rows is None else rows
    q = st["q"].view(case["batch"], -1, D_QK).float()
    x = torch.matmul(q, rows.transpose(1, 2)).mul_(SCALE)
    seen = _seen(st, rows.shape[1])
    x.view(case["batch"], case["s_q"], case["heads"], -1).masked_fill_(~seen[:, :, None], float("-inf"))
    return x


def _run_tree(st):
    case = st["case"]
    if case["parents"]:
        within = _within(st)
        st["mask"].copy_(_pack(_ancestors(st["parents"]) & within[:, :, None]))
    rows = _rows(st)
    x = _scores(st, rows)
    m = x.amax(2, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(2, keepdim=True)
    o = torch.matmul(p, rows[:, :, :D_V]) / torch.where(l > 0, l, torch.ones_like(l))
    st["out"].copy_(o.view(st["out"].shape))
    st["lse"].copy_((m + l.log()).view(st["lse"].shape))
    return {"out": st["out"], "lse": st["lse"], "mask": st["mask"]}


def _run_weights(st):
    case = st["case"]
    x = _scores(st).sub_(st["lse"].view(case["batch"], -1, 1)).exp_()
    new = x.sum(1)
    w = st["weights"]
    live = torch.arange(w.shape[1], device="cuda") < st["seqlens"][:, None]
    old = w * case["decay"] if case["decay"] != 0.0 else torch.zeros_like(w)
    w.copy_(torch.where(live, old + new, w))
    return w


def _run_select(st):
    case = st["case"]
    t, w, B = st["seqlens"][:, None].long(), st["weights"], case["budget"]
    pos = torch.arange(w.shape[1], device="cuda")
    key = torch.where((pos < case["sink"]) | (pos >= t - case["recent"]), torch.full_like(w, float("inf")), w)
    key = torch.where(pos < t, key, torch.full_like(w, float("-inf")))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices      # ties: the lowest position first
    B_ = min(B, w.shape[1])
    n = t.clamp(max=B)
    pick = torch.where(torch.arange(B_, device="cuda") < n, order[:, :B_], torch.full_like(order[:, :B_], 1 << 30))
    pick = torch.sort(pick, dim=1).values
    st["kept"].fill_(-1)
    st["kept"][:, :B_] = torch.where(pick < (1 << 30), pick, torch.full_like(pick, -1)).to(torch.int32)
    st["kept_lens"].copy_(n[:, 0])
    return {"kept": st["kept"], "lens": st["kept_lens"]}


def _run_compact(st):
    src, n = st["src"].long(), st["src_lens"].long()[:, None]
    k = torch.arange(src.shape[1], device="cuda")
    k = torch.minimum(k, n - 1)                                         # places behind the list repeat its last row
    src = src.gather(1, k)
    dst = k if st["base"] is None else k + st["base"].long()[:, None]
    table = st["table"].long()

    def slot(pos):
        return (table.gather(1, pos // PAGE) * PAGE + pos % PAGE).view(-1)

    a, d = slot(src), slot(dst)
    pool = st["pool"]
    if st["scale"] is None:
        flat = pool.view(-1, D_QK)
        flat[d] = flat[a]
    else:
        lat = pool[:, :FP8_LATENT].unflatten(1, (PAGE, D_V))
        rope = pool[:, FP8_LATENT:].unflatten(1, (PAGE, D_ROPE * 2))
        lat[d // PAGE, d % PAGE] = lat[a // PAGE, a % PAGE]
        rope[d // PAGE, d % PAGE] = rope[a // PAGE, a % PAGE]
        st["scale"].view(-1)[d] = st["scale"].view(-1)[a]
    if st["weights"] is not None:
        st["weights"].scatter_(1, dst, st["weights"].gather(1, src))
    return _pool_out(st)


def _pool_out(st):
    """The cache and what moves with it, 8-bit values as the values they stand for."""
    out = {}
    if st["scale"] is None:
        out["pool"] = st["pool"]
    else:
        out["latent"] = st["pool"][:, :FP8_LATENT].view(torch.float8_e4m3fn)
        out["rope"] = st["pool"][:, FP8_LATENT:].view(torch.bfloat16)
        out["scale"] = st["scale"]
    if st["weights"] is not None:
        out["weights"] = st["weights"]
    return out


# ---- the library's calls ----------------------------------------------------

def _own_tree(st):
    if st["case"]["parents"]:
        st["mla"].mla_tree_mask(st["parents"], st["mask"], draft_lens=st["draft_lens"])
    st["decoder"].decode(st["q"], st["pool"], st["table"], st["seqlens"], st["mask"], SCALE, st["out"], st["lse"],
                         draft_lens=st["draft_lens"], kv_scale=st["scale"])
    return {"out": st["out"], "lse": st["lse"], "mask": st["mask"]}


def _own_weights(st):
    st["attn"].accumulate(st["q"], st["pool"], st["table"], st["seqlens"], st["lse"], SCALE, st["case"]["decay"],
                          st["weights"], kv_scale=st["scale"])
    return st["weights"]


def _own_select(st):
    case = st["case"]
    st["mla"].mla_evict_select(st["weights"], st["seqlens"], case["budget"], case["sink"], case["recent"], st["kept"],
                               st["kept_lens"])
    return {"kept": st["kept"], "lens": st["kept_lens"]}


def _own_compact(st):
    st["compactor"].compact(st["pool"], st["table"], st["src"], st["src_lens"], base=st["base"], kv_scale=st["scale"],
                            weights=st["weights"])
    return _pool_out(st)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "weights": _own_weights, "select": _own_select, "compact": _own_compact}[op](state)
    return {"tree": _run_tree, "weights": _run_weights, "select": _run_select, "compact": _run_compact}[op](state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    b, row = case["batch"], 1152 if case.get("cache", "bf16") == "bf16" else 512 + 128 + 4
    # the mean of lengths spread by their logarithm
    lo, hi = case["t_lo"], case["t_hi"]
    mean = hi if hi == lo else (hi - lo) / math.log(hi / lo)
    tokens = b * mean
    if case["op"] == "tree":
        n = case["s_q"] * (0.5 if case["ragged"] else 1.0)
        rows = b * n * case["heads"]
        return {"bytes": rows * (D_QK + D_V) * 2 + rows * 4 + tokens * row, "flops": 2.0 * rows * mean * (D_QK + D_V)}
    if case["op"] == "weights":
        rows = b * case["s_q"] * case["heads"]
        return {"bytes": rows * D_QK * 2 + rows * 4 + tokens * (row + (8 if case["decay"] != 0.0 else 4)), "flops": 2.0 * rows * mean * D_QK}
    if case["op"] == "select":
        return {"bytes": tokens * 4 + b * (case["budget"] + 2) * 4, "flops": tokens}
    moved = b * (case["rows"] * 0.5 if case["base"] else min(case["rows"], mean))
    return {"bytes": moved * (2 * row + (8 if case["weights"] else 0) + 4), "flops": 0}


# ---- the definitions in 64 bits ---------------------------------------------

def _request_rows64(st, r):
    """Request r's cached rows in 64 bits, token by token through its page list."""
    t = int(st["seqlens"][r])
    pos = torch.arange(t, device="cuda")
    page, at = st["table"][r].long()[pos // PAGE], pos % PAGE
    if st["scale"] is None:
        return st["pool"][page, at].double()
    lat = st["pool"][:, :FP8_LATENT].reshape(-1, PAGE, D_V)[page, at].view(torch.float8_e4m3fn).float().double()
    rope = st["pool"][:, FP8_LATENT:].reshape(-1, PAGE, 2 * D_ROPE)[page, at].contiguous().view(torch.bfloat16).double()
    return torch.cat([lat * st["scale"][page, at].double()[:, None], rope], 1)


def _exact_tree(st):
    case, b, s, h = st["case"], st["case"]["batch"], st["case"]["s_q"], st["case"]["heads"]
    out = torch.zeros((b, s, h, D_V), dtype=torch.float64, device="cuda")
    lse = torch.full((b, s, h), float("-inf"), dtype=torch.float64, device="cuda")
    par, lens = st["parents"].tolist(), _draft_lens(st).tolist()
    for r in range(b):
        c, n = _request_rows64(st, r), lens[r]
        if n == 0:
            continue
        P = c.shape[0] - n
        see = torch.zeros((n, c.shape[0]), dtype=torch.bool)
        see[:, :P] = True
        for i in range(n):
            j = i
            while j >= 0:
                see[i, P + j] = True
                j = par[r][j]
        x = (st["q"][r, :n].double().view(n * h, D_QK) @ c.T).view(n, h, -1) * SCALE
        x = x.masked_fill(~see.cuda()[:, None], float("-inf"))
        lse[r, :n] = torch.logsumexp(x, 2)
        out[r, :n] = (torch.softmax(x, 2).view(n * h, -1) @ c[:, :D_V]).view(n, h, D_V)
    return {"out": out, "lse": lse, "mask": None}


def _exact_weights(st):
    case, s, h = st["case"], st["case"]["s_q"], st["case"]["heads"]
    w = st["weights"].double()
    for r in range(case["batch"]):
        c = _request_rows64(st, r)
        t = c.shape[0]
        new = torch.zeros(t, dtype=torch.float64, device="cuda")
        for i in range(s):
            k = max(0, t - s + i + 1) if case["causal"] else t
            x = st["q"][r, i].double() @ c[:k].T * SCALE
            new[:k] += torch.exp(x - st["lse"][r, i].double()[:, None]).sum(0)
        w[r, :t] = case["decay"] * w[r, :t] + new
    return w


def _exact_compact(st):
    table, pool = st["table"].cpu(), st["pool"].clone()
    scale = None if st["scale"] is None else st["scale"].clone()
    weights = None if st["weights"] is None else st["weights"].clone()
    lat, rope = st["pool"][:, :FP8_LATENT], st["pool"][:, FP8_LATENT:]
    for r in range(table.shape[0]):
        n = int(st["src_lens"][r])
        src = st["src"][r, :n].long().cpu()
        dst = torch.arange(n) + (0 if st["base"] is None else int(st["base"][r]))
        a, d = [(table[r].long()[x // PAGE].cuda(), (x % PAGE).cuda()) for x in (src, dst)]
        if scale is None:
            pool[d] = st["pool"][a]
        else:
            pool[:, :FP8_LATENT].unflatten(1, (PAGE, D_V))[d] = lat.unflatten(1, (PAGE, D_V))[a]
            pool[:, FP8_LATENT:].unflatten(1, (PAGE, 2 * D_ROPE))[d] = rope.unflatten(1, (PAGE, 2 * D_ROPE))[a]
            scale[d] = st["scale"][a]
        if weights is not None:
            weights[r, :n + int(dst[0]) if n else 0][dst[0]:] = st["weights"][r, src.cuda()]
    if scale is None:
        out = {"pool": pool}
    else:
        out = {"latent": pool[:, :FP8_LATENT].view(torch.float8_e4m3fn), "rope": pool[:, FP8_LATENT:].view(torch.bfloat16), "scale": scale}
    if weights is not None:
        out["weights"] = weights
    return out


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None
    st = prepare(case, seed)
    return {"tree": _exact_tree, "weights": _exact_weights, "compact": _exact_compact}[op](st)
