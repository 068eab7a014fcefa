"""The tree decode, the acceptance, the attention weights, the eviction and
the compaction in a row, as a serving loop runs them, on the GPU against the
fp64 oracle.
"""
import dataclasses

import numpy as np
import pytest
import torch

import mla_latent_space_b200 as mla
import mla_workloads as mw
import oracle
from gpu_helpers import assert_parity, compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_space_b200 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_draft_verify_accept_weigh_evict_decode(cache):
    b, h, s = 3, 128, 8
    wl = mw.make(b, s, h, [500, 77, 1300], seed=100, cache_dtype=cache, name="chain")
    par = np.array([[-1, 0, 0, 1, 1, 2, 3, 3], [-1, -1, 0, 1, 2, 2, 4, 5], [-1, 0, 1, 2, 3, 4, 5, 6]], dtype=np.int32)
    bt, sl = torch.from_numpy(wl.block_table).cuda(), torch.from_numpy(wl.seqlens).cuda()
    pool, sc = wl.pool.cuda(), None if wl.kv_scale is None else wl.kv_scale.cuda()
    q = wl.q.cuda()

    # verify the tree
    tree = mla.TreeDecoder(mla.make_shape(b, s, h, wl.max_pages, wl.num_pages, cache))
    mask = torch.empty((b, s, 1), dtype=torch.int64, device="cuda")
    out = torch.empty((b, s, h, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b, s, h), dtype=torch.float32, device="cuda")
    mla.mla_tree_mask(torch.from_numpy(par).cuda(), mask)
    tree.decode(q, pool, bt, sl, mask, wl.softmax_scale, out, lse, kv_scale=sc)
    O_ref, L_ref = oracle.tree_decode(wl, oracle.tree_mask(par))
    assert_parity(compare(out.float().cpu().numpy(), lse.cpu().numpy(), O_ref, L_ref), "tree")
    assert tree.status() == 0

    # accept one path of each: it closes up behind the prefix
    paths = [[0, 1, 3, 7], [1, 3], [0, 1, 2, 3, 4, 5, 6, 7]]
    base = wl.seqlens - s
    src, n = np.full((b, s), -1, dtype=np.int32), np.array([len(p) for p in paths], dtype=np.int32)
    for r, p in enumerate(paths):
        src[r, :len(p)] = base[r] + np.array(p)
    shape1 = mla.make_shape(b, 1, h, wl.max_pages, wl.num_pages, cache)
    accept = mla.CacheCompactor(shape1, s)
    accept.compact(pool, bt, torch.from_numpy(src).cuda(), torch.from_numpy(n).cuda(),
                   base=torch.from_numpy(base.astype(np.int32)).cuda(), kv_scale=sc)
    assert accept.status() == 0
    wl.pool, wl.kv_scale, _ = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, src, n, base)
    wl.seqlens = (base + n).astype(np.int32)
    sl.copy_(torch.from_numpy(wl.seqlens))

    # the accepted nodes' weights: their rows at the end of the step's, the others without an lse, in causal order
    q_acc = torch.zeros_like(wl.q)
    l_acc = np.full((b, s, h), -np.inf, dtype=np.float32)
    for r, p in enumerate(paths):
        q_acc[r, s - len(p):] = wl.q[r, p]
        l_acc[r, s - len(p):] = lse[r].cpu().numpy()[p]
    acc_wl = dataclasses.replace(wl, q=q_acc, causal=True)
    w = torch.zeros((b, wl.max_pages * 64), device="cuda")
    mla.AttnWeights(mla.make_shape(b, s, h, wl.max_pages, wl.num_pages, cache, True)).accumulate(
        q_acc.cuda(), pool, bt, sl, torch.from_numpy(l_acc).cuda(), wl.softmax_scale, 0.0, w, kv_scale=sc)
    ref = oracle.attn_weights(acc_wl, l_acc, 0.0, np.zeros((b, wl.max_pages * 64)))
    assert (np.abs(w.cpu().numpy() - ref) <= 5e-4 * ref).all()
    for r, p in enumerate(paths):                       # each row's weights sum to one, up to the decode's lse
        assert abs(w[r].double().sum().item() - h * len(p)) <= 1.5e-3 * h * len(p)

    # the next token decodes over the closed-up cache and leaves its weights
    wl.q, wl.s_q = wl.q[:, :1].contiguous(), 1
    q1 = wl.q.cuda()
    dec = mla.Decoder(shape1)
    out1 = torch.empty((b, 1, h, 512), dtype=torch.bfloat16, device="cuda")
    lse1 = torch.empty((b, 1, h), dtype=torch.float32, device="cuda")
    dec.schedule(sl)
    dec.decode(q1, pool, sc, bt, sl, wl.softmax_scale, out1, lse1)
    O_ref, L_ref = oracle.decode(wl)
    assert_parity(compare(out1.float().cpu().numpy(), lse1.cpu().numpy(), O_ref, L_ref), "accepted")
    w = torch.zeros((b, wl.max_pages * 64), device="cuda")
    acc = mla.AttnWeights(shape1)
    acc.accumulate(q1, pool, bt, sl, lse1, wl.softmax_scale, 1.0, w, kv_scale=sc)
    got = w.cpu().numpy().astype(np.float64)
    ref = oracle.attn_weights(wl, L_ref, 0.0, np.zeros_like(got))
    # 5e-4 of a weight from its own arithmetic (see the weights' tests), 1e-3 from the decode's lse
    assert (np.abs(got - ref) <= 1.5e-3 * ref).all()

    # cut every request to its budget: the kept list is the sparse decode's list
    budget = 64
    kept = torch.empty((b, budget), dtype=torch.int32, device="cuda")
    n_kept = torch.empty(b, dtype=torch.int32, device="cuda")
    mla.mla_evict_select(w, sl, budget, 4, 8, kept, n_kept)
    k_ref, n_ref = oracle.evict_select(w.cpu().numpy(), wl.seqlens, budget, 4, 8)
    assert np.array_equal(kept.cpu().numpy(), k_ref) and np.array_equal(n_kept.cpu().numpy(), n_ref)
    sparse = mla.SparseDecoder(shape1, budget)
    out_s, lse_s = torch.empty_like(out1), torch.empty_like(lse1)
    sparse.decode(q1, pool, bt, sl, kept.view(b, 1, budget), wl.softmax_scale, out_s, lse_s, kv_scale=sc)

    # close up and decode again: the same rows, now dense
    comp = mla.CacheCompactor(shape1, budget)
    comp.compact(pool, bt, kept, n_kept, kv_scale=sc, weights=w)
    assert comp.status() == 0
    dec.schedule(n_kept)
    dec.decode(q1, pool, sc, bt, n_kept, wl.softmax_scale, out1, lse1)
    wl.pool, wl.kv_scale, w_ref = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, k_ref, n_ref, None, got.astype(np.float32))
    wl.seqlens = n_ref
    O_ref, L_ref = oracle.decode(wl)
    assert_parity(compare(out1.float().cpu().numpy(), lse1.cpu().numpy(), O_ref, L_ref), "dense after eviction")
    assert_parity(compare(out_s.float().cpu().numpy(), lse_s.cpu().numpy(), O_ref, L_ref), "sparse before eviction")
    assert np.array_equal(w.cpu().numpy(), w_ref)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_pools_past_four_gigabytes(cache):
    # the workload's pages lie past the 2^32nd byte of the pool
    wl = mw.make(2, 4, 16, [300, 130], seed=101, cache_dtype=cache)
    far = (5 << 30) // (73728 if cache == "bf16" else 40960)
    pages = far + wl.num_pages
    pool = torch.zeros((pages,) + tuple(wl.pool.shape[1:]), dtype=wl.pool.dtype, device="cuda")
    pool[far:] = wl.pool.cuda()
    sc = None
    if wl.kv_scale is not None:
        sc = torch.ones((pages, 64), device="cuda")
        sc[far:] = wl.kv_scale.cuda()
    bt, sl, q = torch.from_numpy(wl.block_table + far).cuda(), torch.from_numpy(wl.seqlens).cuda(), wl.q.cuda()
    shape = mla.make_shape(2, 4, 16, wl.max_pages, pages, cache)
    mask = oracle.tree_mask(np.tile(np.array([-1, 0, 0, 1], dtype=np.int32), (2, 1)))
    out = torch.empty((2, 4, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4, 16), dtype=torch.float32, device="cuda")
    tree = mla.TreeDecoder(shape)
    tree.decode(q, pool, bt, sl, torch.from_numpy(mask).cuda(), wl.softmax_scale, out, lse, kv_scale=sc)
    O_ref, L_ref = oracle.tree_decode(wl, mask)
    assert_parity(compare(out.float().cpu().numpy(), lse.cpu().numpy(), O_ref, L_ref), "far tree")
    l_ref = oracle.decode(wl)[1].astype(np.float32)
    w = torch.zeros((2, wl.max_pages * 64), device="cuda")
    acc = mla.AttnWeights(shape)
    acc.accumulate(q, pool, bt, sl, torch.from_numpy(l_ref).cuda(), wl.softmax_scale, 0.0, w, kv_scale=sc)
    ref = oracle.attn_weights(wl, l_ref, 0.0, np.zeros((2, wl.max_pages * 64)))
    assert (np.abs(w.cpu().numpy() - ref) <= 5e-4 * ref).all()
    src = np.stack([np.arange(3, 103), np.arange(30, 130)]).astype(np.int32)
    comp = mla.CacheCompactor(shape, 100)
    comp.compact(pool, bt, torch.from_numpy(src).cuda(), torch.tensor([100, 100], dtype=torch.int32, device="cuda"), kv_scale=sc)
    p_ref, s_ref, _ = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, src, [100, 100])
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    assert torch.equal(bits(pool[far:].cpu()), bits(p_ref)) and not pool[:far].any()
    if sc is not None:
        assert torch.equal(sc[far:].cpu(), s_ref)
    assert tree.status() == 0 and acc.status() == 0 and comp.status() == 0


def test_a_loop_that_appends_weighs_and_evicts_follows_every_token_by_name():
    """Decode, weigh, append, cut, and again: each token's weight is that of the token, wherever its row lies by then.

    A term is within 3e-4 of itself given the lse (see the weights' tests), so a sum of them is; each step rounds the
    sum once more.
    """
    b, h, budget, cap, steps = 3, 16, 70, 96, 60
    wl = mw.make(b, 1, h, [cap] * b, seed=120)
    g = torch.Generator().manual_seed(121)
    pages = wl.max_pages
    bt, pool = torch.from_numpy(wl.block_table).cuda(), wl.pool.cuda()
    n = np.array([80, 33, 64])
    rows = [[wl.pool[wl.block_table[r, j // 64], j % 64].double().numpy() for j in range(n[r])] for r in range(b)]
    model = [[0.0] * n[r] for r in range(b)]            # by token, as rows
    w = torch.zeros((b, pages * 64), device="cuda")
    shape = mla.make_shape(b, 1, h, pages, wl.num_pages)
    dec, acc, comp = mla.Decoder(shape), mla.AttnWeights(shape), mla.CacheCompactor(shape, budget)
    kept = torch.empty((b, budget), dtype=torch.int32, device="cuda")
    n_kept = torch.empty(b, dtype=torch.int32, device="cuda")
    out = torch.empty((b, 1, h, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b, 1, h), device="cuda")
    evictions = stale = 0
    for step in range(steps):
        q = torch.randn((b, 1, h, 576), generator=g).bfloat16()
        sl = torch.from_numpy(n.astype(np.int32)).cuda()
        dec.schedule(sl)
        dec.decode(q.cuda(), pool, None, bt, sl, wl.softmax_scale, out, lse)
        acc.accumulate(q.cuda(), pool, bt, sl, lse, wl.softmax_scale, 0.9, w)
        got, l_now = w.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        for r in range(b):
            x = np.stack(rows[r]) @ q[r, 0].double().numpy().T * wl.softmax_scale
            new = np.exp(x - l_now[r, 0]).sum(1)
            model[r] = [0.9 * a + c for a, c in zip(model[r], new)]
            ref = np.array(model[r])
            assert (np.abs(got[r, :n[r]] - ref) <= (3e-4 + steps * 2.0 ** -23) * ref).all(), (step, r)
        if (n >= cap - 1).any():                        # cut all to the budget
            mla.mla_evict_select(w, sl, budget, 4, 16, kept, n_kept)
            k_ref, n_ref = oracle.evict_select(w.cpu().numpy(), n, budget, 4, 16)
            assert np.array_equal(kept.cpu().numpy(), k_ref) and np.array_equal(n_kept.cpu().numpy(), n_ref)
            comp.compact(pool, bt, kept, n_kept, weights=w)
            for r in range(b):
                rows[r] = [rows[r][j] for j in k_ref[r, :n_ref[r]]]
                model[r] = [model[r][j] for j in k_ref[r, :n_ref[r]]]
            n = n_ref.astype(np.int64)
            evictions += 1
        for r in range(b):                              # append a token: its row, and a weight of zero
            row = torch.randn(576, generator=g).bfloat16()
            pool[wl.block_table[r, n[r] // 64], n[r] % 64] = row.cuda()
            stale += int(w[r, n[r]] != 0)
            w[r, n[r]] = 0.0
            rows[r].append(row.double().numpy())
            model[r].append(0.0)
        n = n + 1
    assert evictions >= 2 and stale > 0                 # places were used again, with something in them
    assert dec.status() == 0 and acc.status() == 0 and comp.status() == 0
