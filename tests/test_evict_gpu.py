"""GPU tests of the eviction's choice (mla_evict_select) and of the cache
compaction (mla_cache_compact) through the C ABI against the oracle.  Both
are exact: positions are equal, moved rows are equal bit for bit.
"""
import numpy as np
import pytest
import torch

import mla_latent_space_b200 as mla
import mla_workloads as mw
import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_space_b200 import build
    build.build()
    assert torch.cuda.is_available()


def select(w, seqlens, budget, sink, recent):
    b = w.shape[0]
    kept = torch.full((b, budget), 77, dtype=torch.int32, device="cuda")
    lens = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_evict_select(torch.from_numpy(w).cuda(), torch.tensor(seqlens, dtype=torch.int32, device="cuda"), budget, sink,
                         recent, kept, lens, st)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), lens.cpu().numpy(), st.item()


def check_select(w, seqlens, budget, sink, recent):
    kept, lens, st = select(w, seqlens, budget, sink, recent)
    k_ref, l_ref = oracle.evict_select(w, seqlens, budget, sink, recent)
    assert st == 0
    assert np.array_equal(lens, l_ref) and np.array_equal(kept, k_ref)


def weights(b, T, seed, kind="heavy"):
    g = np.random.default_rng(seed)
    w = np.exp(4.0 * g.standard_normal((b, T)) - 6.0).astype(np.float32)
    if kind == "ties":
        w = g.integers(0, 3, (b, T)).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "close":                       # keys that differ in their low bits alone
        w = (1.0 + g.integers(0, 4096, (b, T)) * 2.0 ** -23).astype(np.float32)
    elif kind == "odd":
        flat = w.reshape(-1)
        special = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.0, 1e-42, -1e-42], dtype=np.float32)
        flat[:] = np.where(g.random(flat.size) < 0.5, special[g.integers(0, 8, flat.size)], flat)
        flat[::17] = np.float32(np.nan) * -1
    return w


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "close", "odd"])
@pytest.mark.parametrize("T,budget,sink,recent", [
    (64, 16, 4, 4), (257, 100, 0, 0), (1000, 999, 16, 100), (4096, 1024, 4, 64), (1025, 1, 0, 0), (1023, 1, 1, 0),
    (2048, 1, 0, 1), (333, 32, 16, 16), (5000, 4999, 0, 0)])
def test_select(kind, T, budget, sink, recent):
    w = weights(4, T, T + budget, kind)
    check_select(w, [T, T // 2, max(0, budget - 1), min(T, budget + 1)], budget, sink, recent)


@pytest.mark.parametrize("T,b", [(20000, 3), (70001, 2), (131072, 1), (300000, 1), (1000000, 1)])
def test_select_long(T, b):
    for kind in ("heavy", "ties", "close"):
        w = weights(b, T, T, kind)
        check_select(w, [T, T // 3, 5][:b], 4097, 4, 256)


def test_select_wide_batch_and_short_requests():
    b, T = 300, 130
    w = weights(b, T, 3)
    check_select(w, [(r * 7) % (T + 1) for r in range(b)], 20, 2, 5)


def test_select_large_batch_of_long_rows():
    b, T = 40, 49152                            # one CTA holds a whole long row
    w = weights(b, T, 6)
    w[::3] = weights(len(w[::3]), T, 7, "ties")
    check_select(w, [T - 3 * r for r in range(b)], 4000, 4, 100)


def test_select_budget_larger_than_the_row():
    check_select(weights(2, 64, 4), [64, 0], 200, 4, 8)


def test_select_does_not_read_behind_the_length_and_flags_bad_lengths():
    w = weights(3, 500, 5)
    k0, l0, _ = select(w, [300, 200, 100], 50, 4, 10)
    w2 = w.copy()
    for r, t in enumerate([300, 200, 100]):
        w2[r, t:] = np.inf
    k1, l1, st = select(w2, [300, 200, 100], 50, 4, 10)
    assert np.array_equal(k0, k1) and np.array_equal(l0, l1) and st == 0
    k2, l2, st = select(w, [501, -1, 100], 50, 4, 10)
    assert st != 0
    k_ref, l_ref = oracle.evict_select(w, [500, 0, 100], 50, 4, 10)
    assert np.array_equal(k2, k_ref) and np.array_equal(l2, l_ref)


def test_select_replays_from_a_graph_and_runs_on_two_streams():
    for T in (3000, 20000):                                             # one CTA a request, and a cluster
        ws = [weights(3, T, 60 + k) for k in range(3)]
        dev = torch.from_numpy(ws[0]).cuda()
        sl = torch.tensor([T, T // 2, 100], dtype=torch.int32, device="cuda")
        kept = [torch.empty((3, 500), dtype=torch.int32, device="cuda") for _ in range(2)]
        lens = [torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for k, s in zip(range(2), streams):
            mla.mla_evict_select(dev, sl, 500, 4, 64, kept[k], lens[k], stream=s)
        torch.cuda.synchronize()
        ref = oracle.evict_select(ws[0], [T, T // 2, 100], 500, 4, 64)
        assert all(np.array_equal(kept[k].cpu().numpy(), ref[0]) and np.array_equal(lens[k].cpu().numpy(), ref[1]) for k in range(2))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.mla_evict_select(dev, sl, 500, 4, 64, kept[0], lens[0])
        for w in ws[1:]:
            dev.copy_(torch.from_numpy(w))
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(kept[0].cpu().numpy(), oracle.evict_select(w, [T, T // 2, 100], 500, 4, 64)[0])


# ---- compaction -----------------------------------------------------------------

def lists(seqlens, rows, seed, base=None):
    g = np.random.default_rng(seed)
    b = len(seqlens)
    src, lens = np.full((b, rows), -1, dtype=np.int32), np.zeros(b, dtype=np.int32)
    for r, t in enumerate(seqlens):
        first = 0 if base is None else int(base[r])
        n = min(rows, int(t) - first)
        lens[r] = n
        src[r, :n] = first + np.sort(g.permutation(int(t) - first)[:n])
    return src, lens


def check_compact(wl, src, lens, base=None, with_weights=True, comp=None, stream=None):
    sh = mla.make_shape(wl.batch, 1, 1, wl.max_pages, wl.num_pages, wl.cache_dtype)
    comp = mla.CacheCompactor(sh, src.shape[1]) if comp is None else comp
    w = np.random.default_rng(1).random((wl.batch, wl.max_pages * 64), dtype=np.float32) if with_weights else None
    pool, sc = wl.pool.cuda(), None if wl.kv_scale is None else wl.kv_scale.cuda()
    wd = None if w is None else torch.from_numpy(w).cuda()
    comp.compact(pool, torch.from_numpy(wl.block_table).cuda(), torch.from_numpy(src).cuda(), torch.from_numpy(lens).cuda(),
                 base=None if base is None else torch.tensor(base, dtype=torch.int32, device="cuda"), kv_scale=sc, weights=wd)
    torch.cuda.synchronize()
    assert comp.status() == 0
    p_ref, s_ref, w_ref = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, src, lens, base, w)
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    assert torch.equal(bits(pool.cpu()), bits(p_ref))
    if sc is not None:
        assert torch.equal(sc.cpu().view(torch.int32), s_ref.view(torch.int32))
    if w is not None:
        assert np.array_equal(wd.cpu().numpy(), w_ref)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("seqlens,rows", [([1, 64, 700], 1), ([65, 0, 3], 3), ([130, 1000, 200], 129), ([4000, 2500, 64], 2048),
                                          ([900, 901, 31], 900), ([3000, 10, 2000], 33)])
def test_compact_of_kept_rows(cache, seqlens, rows):
    wl = mw.make(3, 1, 1, seqlens, seed=rows, cache_dtype=cache)
    src, lens = lists(seqlens, rows, seed=rows + 1)
    check_compact(wl, src, lens)
    check_compact(wl, src, lens, with_weights=False)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_compact_of_accepted_paths(cache):
    seqlens = [70, 200, 16, 4096]
    wl = mw.make(4, 1, 1, seqlens, seed=7, cache_dtype=cache)
    base = [t - 16 for t in seqlens]
    src, lens = lists(seqlens, 9, seed=8, base=base)
    lens[1] = 0
    check_compact(wl, src, lens, base)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_compact_when_every_destination_is_a_later_source(cache):
    # shifts by one row, by one page and by 63 rows: each row that is overwritten is itself moved
    for shift in (1, 63, 64, 65):
        t = 3001
        wl = mw.make(2, 1, 1, [t, t], seed=shift, cache_dtype=cache)
        src = np.tile(np.arange(shift, t, dtype=np.int32), (2, 1))
        check_compact(wl, src, np.array([t - shift, 17], dtype=np.int32))


def test_compact_of_an_unmoved_prefix_and_of_everything():
    wl = mw.make(2, 1, 1, [500, 500], seed=9)
    src = np.tile(np.arange(500, dtype=np.int32), (2, 1))
    src[0, 300:499] = np.arange(301, 500)
    check_compact(wl, src, np.array([499, 500], dtype=np.int32))


def test_compact_many_requests_again_and_again_through_one_workspace():
    g = np.random.default_rng(11)
    seqlens = [int(x) for x in g.integers(0, 1500, 40)]
    wl = mw.make(40, 1, 1, seqlens, seed=11)
    comp = mla.CacheCompactor(mla.make_shape(40, 1, 1, wl.max_pages, wl.num_pages), 700)
    for seed in range(4):
        src, lens = lists(seqlens, 700, seed=seed)
        check_compact(wl, src, lens, comp=comp)


def test_compact_with_a_shared_prefix_that_stays():
    # two requests list the same first pages; nothing moves there
    wl = mw.make(2, 1, 1, [1000, 900], seed=18)
    wl.block_table[1, :3] = wl.block_table[0, :3]
    src = np.full((2, 600), -1, dtype=np.int32)
    for r, t in enumerate((1000, 900)):
        src[r, :192] = np.arange(192)
        src[r, 192:600] = 192 + np.sort(np.random.default_rng(r).permutation(t - 192)[:408])
    check_compact(wl, src, np.array([600, 600], dtype=np.int32))


def test_compact_flags_bad_lists_and_touches_no_other_request():
    wl = mw.make(2, 1, 1, [300, 300], seed=12)
    good_src, good_lens = lists([300, 300], 100, seed=13)
    p_ref, _, _ = oracle.compact(wl.pool, None, wl.block_table, good_src, [0, 100])
    sh = mla.make_shape(2, 1, 1, wl.max_pages, wl.num_pages)

    def run(src, lens, base=None, table=None):
        comp = mla.CacheCompactor(sh, 100)
        pool = wl.pool.cuda()
        comp.compact(pool, torch.from_numpy(wl.block_table if table is None else table).cuda(), torch.from_numpy(src).cuda(),
                     torch.from_numpy(lens).cuda(), base=None if base is None else torch.tensor(base, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert comp.status() == -6 and comp.status() == 0              # read and cleared
        rows = pool.cpu().view(torch.int16)[wl.block_table[1]]
        assert torch.equal(rows, p_ref.view(torch.int16)[wl.block_table[1]])

    for k, v in ((50, -1), (50, 1 << 30), (50, 3), (99, wl.max_pages * 64)):
        src = good_src.copy()
        src[0, k] = v
        run(src, good_lens)
    src = good_src.copy()
    src[0, 40:60] = src[0, 40]                                          # repeated
    run(src, good_lens)
    run(good_src, np.array([101, 100], dtype=np.int32))
    run(good_src, np.array([-3, 100], dtype=np.int32))
    run(good_src, good_lens, base=[-1, 0])
    run(good_src, good_lens, base=[2**31 - 1, 0])
    table = wl.block_table.copy()
    table[0, 0] = wl.num_pages
    run(good_src, good_lens, table=table)


def test_compact_replays_from_a_graph_and_runs_on_two_streams():
    seqlens = [2000, 700]
    wl = mw.make(2, 1, 1, seqlens, seed=14)
    sh = mla.make_shape(2, 1, 1, wl.max_pages, wl.num_pages)
    comps = [mla.CacheCompactor(sh, 600) for _ in range(2)]
    src, lens = lists(seqlens, 600, seed=15)
    ref = oracle.compact(wl.pool, None, wl.block_table, src, lens)[0].view(torch.int16)
    pools = [wl.pool.cuda() for _ in range(2)]
    bt, s_d, l_d = torch.from_numpy(wl.block_table).cuda(), torch.from_numpy(src).cuda(), torch.from_numpy(lens).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for c, p, s in zip(comps, pools, streams):
        c.compact(p, bt, s_d, l_d, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(p.cpu().view(torch.int16), ref) for p in pools)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        comps[0].compact(pools[0], bt, s_d, l_d)
    for seed in (16, 17):
        src, lens = lists(seqlens, 600, seed=seed)
        s_d.copy_(torch.from_numpy(src))
        pools[0].copy_(wl.pool)
        g.replay()
        torch.cuda.synchronize()
        ref = oracle.compact(wl.pool, None, wl.block_table, src, lens)[0].view(torch.int16)
        assert torch.equal(pools[0].cpu().view(torch.int16), ref) and comps[0].status() == 0


def test_binding_checks():
    w = torch.zeros((2, 100), device="cuda")
    sl = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
    kept, lens = torch.zeros((2, 8), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mla.mla_evict_select(w, sl, 9, 0, 0, kept, lens)
    with pytest.raises(TypeError):
        mla.mla_evict_select(w.double(), sl, 8, 0, 0, kept, lens)
    with pytest.raises(mla.MLAError):
        mla.mla_evict_select(w, sl, 8, 5, 4, kept, lens)
    sh = mla.make_shape(2, 1, 1, 2, 4)
    with pytest.raises(mla.MLAError):
        mla.CacheCompactor(sh, 0)
    comp = mla.CacheCompactor(sh, 8)
    pool, bt = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        comp.compact(pool, bt, kept[:, :7], lens)
    with pytest.raises(ValueError):
        comp.compact(pool, bt, kept, lens, kv_scale=torch.zeros((4, 64), device="cuda"))


def moved(cache, pool, sc, w, bt, src, lens, base):
    """The same move by plain indexing on the device (every destination is written once)."""
    b, rows = src.shape
    k = torch.arange(rows, device="cuda")
    r, k = (k < lens[:, None]).nonzero(as_tuple=True)
    a, d = src[r, k].long(), k + (0 if base is None else base[r].long())
    at = lambda pos: (bt[r, pos // 64].long(), pos % 64)
    pool, sc, w = pool.clone(), None if sc is None else sc.clone(), w.clone()
    if cache == "bf16":
        pool[at(d)] = pool[at(a)]
    else:
        for plane in (pool[:, :32768].unflatten(1, (64, 512)), pool[:, 32768:].unflatten(1, (64, 128))):
            plane[at(d)] = plane[at(a)]
        sc[at(d)] = sc[at(a)]
    w[r, d] = w[r, a]
    return pool, sc, w


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("b,rows,t,kind", [
    (64, 2048, 2300, "shift"),      # 64 (FP8: 32) groups a request: seven (four) for each resident CTA
    (64, 4096, 4400, "shift"),
    (64, 4096, 8192, "random"),
    (1, 81920, 100000, "shift"),    # one long list: most groups wait
    (700, 130, 200, "shift"),       # more requests than resident CTAs, several groups each: a CTA's request changes
    (299, 200, 400, "random"),
])
def test_compact_in_many_rounds(cache, b, rows, t, kind):
    g = torch.Generator(device="cuda").manual_seed(rows + b)
    pages = (t + 63) // 64
    bt = torch.randperm(b * pages, generator=g, device="cuda").to(torch.int32).view(b, pages)
    if cache == "bf16":
        pool = torch.randint(-2**15, 2**15, (b * pages, 64, 576), generator=g, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        sc = None
    else:
        pool = torch.randint(0, 256, (b * pages, 40960), generator=g, dtype=torch.uint8, device="cuda")
        sc = torch.rand((b * pages, 64), generator=g, device="cuda")
    w = torch.rand((b, pages * 64), generator=g, device="cuda")
    if kind == "shift":             # each row that is overwritten is itself moved
        shift = torch.tensor([1, 31, 32, 33, 63, 64, 65, t - rows], device="cuda").repeat(b)[:b]
        src = torch.arange(rows, device="cuda") + shift.clamp(max=t - rows)[:, None]
    else:
        src = torch.rand((b, t), generator=g, device="cuda").argsort(1)[:, :rows].sort(1).values
    src = src.to(torch.int32).contiguous()
    comp = mla.CacheCompactor(mla.make_shape(b, 1, 1, pages, b * pages, cache), rows)
    bits = lambda x: x.view(torch.int16) if x.dtype == torch.bfloat16 else x
    for call in range(3):           # through one workspace
        lens = torch.full((b,), rows, dtype=torch.int32, device="cuda")
        if call > 0 and b > 1:
            lens = torch.randint(0, rows + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        p_ref, s_ref, w_ref = moved(cache, pool, sc, w, bt, src, lens, None)
        comp.compact(pool, bt, src, lens, kv_scale=sc, weights=w)
        assert comp.status() == 0
        assert torch.equal(bits(pool), bits(p_ref)) and torch.equal(w, w_ref)
        assert sc is None or torch.equal(sc, s_ref)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_a_compaction_whose_wait_runs_out_says_so_and_the_next_one_is_right(cache):
    """The test library's stalled call never says that a request's first group has been read: after 2 s the group
    that waits for it reports that, leaves its rows alone and the kernel ends."""
    import ctypes
    import time
    from gpu_helpers import test_lib
    fn = test_lib().mla_test_compact_stalled
    fn.argtypes, fn.restype = mla.lib().mla_cache_compact.argtypes, ctypes.c_int
    wl = mw.make(2, 1, 1, [300, 300], seed=19, cache_dtype=cache)
    src = np.full((2, 200), -1, dtype=np.int32)
    src[0] = np.arange(1, 201)                          # the second group's first row goes where the first group's last lay
    src[1, :10] = np.arange(50, 60)
    lens = np.array([200, 10], dtype=np.int32)
    comp = mla.CacheCompactor(mla.make_shape(2, 1, 1, wl.max_pages, wl.num_pages, cache), 200)
    pool, sc = wl.pool.cuda(), None if wl.kv_scale is None else wl.kv_scale.cuda()
    bt, s_d, l_d = torch.from_numpy(wl.block_table).cuda(), torch.from_numpy(src).cuda(), torch.from_numpy(lens).cuda()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert fn(ctypes.byref(comp.shape), pool.data_ptr(), None if sc is None else sc.data_ptr(), bt.data_ptr(), s_d.data_ptr(),
              l_d.data_ptr(), None, 200, None, comp.workspace.data_ptr(), comp.workspace.numel(),
              torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert 1.0 < time.perf_counter() - t0 < 30.0
    assert comp.status() == -5 and comp.status() == 0
    check_compact(wl, src, lens, comp=comp)             # the same workspace, a cache that has not moved
    check_compact(wl, src, lens, comp=comp)


@pytest.mark.parametrize("T,b", [(200, 5), (3000, 40), (20000, 9), (60000, 40), (400000, 2)])
def test_select_updates_the_lengths_in_place(T, b):
    # kept_lens may be seqlens: one CTA a request, clusters, and rows that are re-read
    w = weights(b, T, T + b)
    seqlens = [[T, T // 2, 60, 0, T - 1, -5, T + 9][r % 7] for r in range(b)]
    dev, sl = torch.from_numpy(w).cuda(), torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    kept = torch.full((b, 100), 77, dtype=torch.int32, device="cuda")
    mla.mla_evict_select(dev, sl, 100, 4, 16, kept, sl)
    k_ref, l_ref = oracle.evict_select(w, seqlens, 100, 4, 16)
    assert np.array_equal(sl.cpu().numpy(), l_ref) and np.array_equal(kept.cpu().numpy(), k_ref)


@pytest.mark.parametrize("b,T", [(2, 8900), (2, 9100), (33, 21000), (33, 21600), (32, 49152), (36, 49152), (37, 49152), (37, 49200)])
def test_select_on_either_side_of_the_choice_of_variant(b, T):
    w = weights(b, T, b + T)
    w[1::2] = weights(len(w[1::2]), T, b, "ties")
    check_select(w, [T - 5 * r for r in range(b)], 2000, 4, 100)
