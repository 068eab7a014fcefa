"""Calls of the operators around the cache at the edges of what their
documentation allows: batches of thousands, head counts on either side of a
tile, table entries that mean nothing, and all of them at once.
"""
import numpy as np
import pytest
import torch

import mla_latent_space_b200 as mla
import mla_workloads as mw
import oracle
from gpu_helpers import assert_parity, compare, shape_of, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_space_b200 import build
    build.build()
    assert torch.cuda.is_available()


def parents_of(b, s, seed):
    g = np.random.default_rng(seed)
    return np.stack([[int(g.integers(-1, i)) if i else -1 for i in range(s)] for _ in range(b)]).astype(np.int32)


def tree(wl, mask, lens=None):
    dev, dec = to_device(wl), mla.TreeDecoder(shape_of(wl))
    out = torch.full((wl.batch, wl.s_q, wl.num_heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((wl.batch, wl.s_q, wl.num_heads), float("nan"), device="cuda")
    dec.decode(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], torch.from_numpy(mask).cuda(), wl.softmax_scale,
               out, lse, draft_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"),
               kv_scale=dev["kv_scale"])
    assert dec.status() == 0
    O_ref, L_ref = oracle.tree_decode(wl, mask, lens)
    assert_parity(compare(out.float().cpu().numpy(), lse.cpu().numpy(), O_ref, L_ref), wl.name)


def weigh(wl, tol):
    """tol: see the weights' tests (3e-4 of a weight, 5e-4 with the 8-bit cache)."""
    dev, acc = to_device(wl), mla.AttnWeights(shape_of(wl))
    lse = oracle.decode(wl)[1].astype(np.float32)
    old = np.random.default_rng(1).random((wl.batch, wl.max_pages * 64), dtype=np.float32)
    w = torch.from_numpy(old).cuda()
    acc.accumulate(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], torch.from_numpy(lse).cuda(), wl.softmax_scale,
                   0.5, w, kv_scale=dev["kv_scale"])
    assert acc.status() == 0
    got, ref = w.cpu().numpy(), oracle.attn_weights(wl, lse, 0.5, old)
    assert (np.abs(got - ref) <= tol * ref).all()
    for r, t in enumerate(wl.seqlens):
        assert np.array_equal(got[r, t:], old[r, t:])


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("s,heads", [(3, 200), (2, 129), (130, 1), (1, 1), (5, 26), (128, 1), (129, 1)])
def test_trees_of_odd_head_counts(cache, s, heads):
    wl = mw.make(3, s, heads, [s, s + 63, s + 700], seed=s + heads, cache_dtype=cache, name="odd_heads")
    tree(wl, oracle.tree_mask(parents_of(3, s, seed=heads)))
    tree(wl, oracle.tree_mask(parents_of(3, s, seed=heads)), [s // 2, s, max(1, s // 3)])


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_thousands_of_requests(cache):
    b = 2500
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(0, 130, b)]
    wl = mw.make(b, 2, 3, lens, seed=140, cache_dtype=cache, causal=True, name="many")
    weigh(wl, 3e-4 if cache == "bf16" else 5e-4)
    wl.causal = False
    tree(wl, oracle.tree_mask(parents_of(b, 2, seed=141)))
    # a choice of 40, and their rows closed up
    w = np.random.default_rng(4).random((b, wl.max_pages * 64), dtype=np.float32)
    kept = torch.empty((b, 40), dtype=torch.int32, device="cuda")
    n = torch.empty(b, dtype=torch.int32, device="cuda")
    mla.mla_evict_select(torch.from_numpy(w).cuda(), torch.from_numpy(wl.seqlens).cuda(), 40, 2, 5, kept, n)
    k_ref, n_ref = oracle.evict_select(w, wl.seqlens, 40, 2, 5)
    assert np.array_equal(kept.cpu().numpy(), k_ref) and np.array_equal(n.cpu().numpy(), n_ref)
    dev, comp = to_device(wl), mla.CacheCompactor(shape_of(wl), 40)
    comp.compact(dev["pool"], dev["block_table"], kept, n, kv_scale=dev["kv_scale"])
    assert comp.status() == 0
    p_ref, s_ref, _ = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, k_ref, n_ref)
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    assert torch.equal(bits(dev["pool"].cpu()), bits(p_ref))
    assert s_ref is None or torch.equal(dev["kv_scale"].cpu(), s_ref)


def test_batches_past_sixteen_bits():
    # the choice and the compaction number their requests past 65535; the masks and the weights refuse that many
    b = 70001
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.rand((b, 64), generator=g, device="cuda")
    sl = torch.randint(0, 65, (b,), generator=g, device="cuda", dtype=torch.int32)
    kept = torch.empty((b, 7), dtype=torch.int32, device="cuda")
    n = torch.empty(b, dtype=torch.int32, device="cuda")
    mla.mla_evict_select(w, sl, 7, 1, 2, kept, n)
    key = torch.where(torch.arange(64, device="cuda") < sl[:, None], w, -1.0)
    at = torch.arange(64, device="cuda")
    key = torch.where(((at < 1) | (at >= sl[:, None] - 2)) & (at < sl[:, None]), 2.0, key)
    ref = key.sort(dim=1, descending=True, stable=True).indices[:, :7]
    ref = torch.where(torch.arange(7, device="cuda") < sl[:, None], ref, 1000).sort(1).values
    ref = torch.where(ref < 1000, ref, -1).to(torch.int32)
    assert torch.equal(kept, ref) and torch.equal(n, sl.clamp(max=7))
    sh = mla.make_shape(b, 1, 1, 1, 1100)
    pool = torch.randn((1100, 64, 576), generator=g, device="cuda").bfloat16()
    bt = torch.full((b, 1), 1099, dtype=torch.int32, device="cuda")     # a page that all but a few share: nothing moves there
    few = torch.arange(0, b, 64, device="cuda")
    bt[few, 0] = torch.arange(len(few), device="cuda", dtype=torch.int32)
    n_few = torch.zeros_like(n)
    n_few[few] = n[few]
    before = pool.clone()
    comp = mla.CacheCompactor(sh, 7)
    comp.compact(pool, bt, kept, n_few)
    assert comp.status() == 0
    for k in range(7):
        rows = few[n_few[few] > k]
        before[bt[rows, 0].long(), k] = before[bt[rows, 0].long(), kept[rows, k].long()]
    assert torch.equal(pool.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_table_entries_behind_the_length_are_not_read(cache):
    wl = mw.make(3, 4, 40, [64, 130, 700], seed=142, cache_dtype=cache, name="garbage")
    for r, t in enumerate(wl.seqlens):
        wl.block_table[r, (int(t) + 63) // 64:] = [2**31 - 1, -7, wl.num_pages][r]
    weigh(wl, 3e-4 if cache == "bf16" else 5e-4)
    tree(wl, oracle.tree_mask(parents_of(3, 4, seed=143)))
    src = np.stack([np.arange(3, 43), np.arange(60, 100), np.arange(650, 690)]).astype(np.int32)
    dev, comp = to_device(wl), mla.CacheCompactor(shape_of(wl), 40)
    comp.compact(dev["pool"], dev["block_table"], torch.from_numpy(src).cuda(),
                 torch.full((3,), 40, dtype=torch.int32, device="cuda"), kv_scale=dev["kv_scale"])
    assert comp.status() == 0
    p_ref, _, _ = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, src, [40] * 3)
    assert torch.equal(dev["pool"].cpu().view(torch.uint8), p_ref.view(torch.uint8))


def test_all_operators_at_once_on_four_streams():
    # a cooperative launch, clusters of two kinds and plain grids beside each other, each with buffers of its own
    wl = mw.make(4, 6, 128, [4000, 900, 64, 2500], seed=144, name="at_once")
    dev = to_device(wl)
    sh = shape_of(wl)
    mask = oracle.tree_mask(parents_of(4, 6, seed=145))
    mask_d = torch.from_numpy(mask).cuda()
    lse0 = oracle.decode(wl)[1].astype(np.float32)
    lse_d = torch.from_numpy(lse0).cuda()
    dec, acc, comp = mla.TreeDecoder(sh), mla.AttnWeights(sh), mla.CacheCompactor(sh, 2000)
    out = torch.empty((4, 6, 128, 512), dtype=torch.bfloat16, device="cuda")
    lse, w = torch.empty((4, 6, 128), device="cuda"), torch.zeros((4, wl.max_pages * 64), device="cuda")
    long_w = torch.rand((4, 40000), device="cuda")
    long_l = torch.full((4,), 40000, dtype=torch.int32, device="cuda")
    kept = torch.empty((4, 4000), dtype=torch.int32, device="cuda")
    n = torch.empty(4, dtype=torch.int32, device="cuda")
    g = np.random.default_rng(6)
    lens = np.minimum(2000, wl.seqlens // 2).astype(np.int32)
    src = np.full((4, 2000), -1, dtype=np.int32)
    for r in range(4):
        src[r, :lens[r]] = np.sort(g.permutation(int(wl.seqlens[r]))[:lens[r]])
    src_d, lens_d = torch.from_numpy(src).cuda(), torch.from_numpy(lens).cuda()
    pools = [dev["pool"].clone() for _ in range(20)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for k in range(20):
        dec.decode(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], mask_d, wl.softmax_scale, out, lse, stream=streams[0])
        acc.accumulate(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], lse_d, wl.softmax_scale, 0.0, w, stream=streams[1])
        mla.mla_evict_select(long_w, long_l, 4000, 4, 64, kept, n, stream=streams[2])
        comp.compact(pools[k], dev["block_table"], src_d, lens_d, stream=streams[3])
    torch.cuda.synchronize()
    assert dec.status() == 0 and acc.status() == 0 and comp.status() == 0
    O_ref, L_ref = oracle.tree_decode(wl, mask)
    assert_parity(compare(out.float().cpu().numpy(), lse.cpu().numpy(), O_ref, L_ref), "tree")
    ref = oracle.attn_weights(wl, lse0, 0.0, np.zeros((4, wl.max_pages * 64)))
    assert (np.abs(w.cpu().numpy() - ref) <= 3e-4 * ref).all()
    assert np.array_equal(kept.cpu().numpy(), oracle.evict_select(long_w.cpu().numpy(), [40000] * 4, 4000, 4, 64)[0])
    p_ref = oracle.compact(wl.pool, None, wl.block_table, src, lens)[0]
    assert all(torch.equal(p.cpu().view(torch.int16), p_ref.view(torch.int16)) for p in pools)
