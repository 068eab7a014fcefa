"""GPU parity of the tree decode (mla_tree_mask, mla_tree_decode_fwd through
the C ABI) against the fp64 oracle, at the decode's tolerances: O max|err| <=
2e-2 and relative L1 against the bf16-rounded oracle <= 1e-3; lse max|err| <=
1e-3.  Masks are compared bit by bit.
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


def run_tree(wl, mask, lens=None, dev=None, stream=None):
    dev = to_device(wl) if dev is None else dev
    dec = mla.TreeDecoder(shape_of(wl))
    out = torch.full((wl.batch, wl.s_q, wl.num_heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((wl.batch, wl.s_q, wl.num_heads), float("nan"), dtype=torch.float32, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    dec.decode(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], torch.from_numpy(mask).cuda(), wl.softmax_scale,
               out, lse, draft_lens=dl, kv_scale=dev["kv_scale"])
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy(), dec.status()


def check(wl, mask, lens=None):
    O, L, st = run_tree(wl, mask, lens)
    assert st == 0, mla.error_string(st)
    O_ref, L_ref = oracle.tree_decode(wl, mask, lens)
    assert_parity(compare(O, L, O_ref, L_ref), wl.name)
    return O, L


@pytest.mark.parametrize("b,s", [(1, 1), (3, 2), (2, 63), (2, 64), (3, 65), (1, 200), (70, 7), (1, 8192), (1, 8193)])
def test_tree_mask_bits(b, s):
    par = parents_of(b, s, seed=s)
    if s > 4:
        par[-1] = np.arange(-1, s - 1)                 # a chain: the deepest path
        par[0, s - 1] = s - 2
    lens = np.array([s - (r % 3) * (s // 4) for r in range(b)], dtype=np.int32)
    for ln in (None, lens):
        m = torch.full((b, s, (s + 63) // 64), -1, dtype=torch.int64, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_tree_mask(torch.from_numpy(par).cuda(), m, None if ln is None else torch.from_numpy(ln).cuda(), st)
        assert st.item() == 0
        got = m.cpu().numpy()
        if s <= 200:
            assert np.array_equal(got, oracle.tree_mask(par, ln))
        else:                                           # the chain, from its definition
            n = s if ln is None else int(ln[-1])
            bits = np.unpackbits(got[-1].view(np.uint8), axis=1, bitorder="little")[:, :s]
            assert np.array_equal(bits[:n], np.tri(s, dtype=np.uint8)[:n]) and not bits[n:].any()


def test_tree_mask_flags_bad_parents_and_counts():
    par = np.array([[-1, 0, 5, -2], [-1, 0, 1, 2], [-1, 1, 0, 0]], dtype=np.int32)
    for lens, bad in (([4, 4, 1], True), ([2, 4, 1], False), ([2, 5, 1], True), ([2, -1, 1], True)):
        m = torch.empty((3, 4, 1), dtype=torch.int64, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_tree_mask(torch.from_numpy(par).cuda(), m, torch.tensor(lens, dtype=torch.int32, device="cuda"), st)
        assert (st.item() != 0) == bad
        assert np.array_equal(m.cpu().numpy(), oracle.tree_mask(par, lens))


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("s,heads,lens_t", [
    (1, 128, [1, 64, 700]),            # one node: plain decode
    (8, 16, [8, 200, 256]),            # one tile a request; a request that is all tree
    (13, 128, [13, 77, 1000]),         # odd count, drafts that straddle a page
    (64, 5, [64, 65, 130]),            # a full mask word, a head count that divides nothing
    (65, 16, [70, 128, 300]),          # two mask words
    (150, 3, [150, 192, 1000]),        # three mask words, tiles that end inside a node
])
def test_tree_decode_parity(cache, s, heads, lens_t):
    wl = mw.make(3, s, heads, lens_t, seed=60 + s, cache_dtype=cache, name=f"tree_{cache}_{s}_{heads}")
    check(wl, oracle.tree_mask(parents_of(3, s, seed=61)))


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_jagged_batches_are_cut_and_joined(cache):
    # tiles cut into many pieces, whole ones and empty ones side by side
    lens_t = [6000, 64, 700, 1, 0, 2500, 130, 9000]
    wl = mw.make(8, 6, 40, lens_t, seed=78, cache_dtype=cache, name="jagged_tree")
    mask = oracle.tree_mask(parents_of(8, 6, seed=79))
    check(wl, mask, [6, 6, 2, 1, 0, 0, 5, 4])


def test_tree_of_a_chain_equals_the_causal_decode():
    wl = mw.make(2, 16, 128, [300, 4096], causal=True, seed=62, name="chain")
    mask = oracle.tree_mask(np.tile(np.arange(-1, 15, dtype=np.int32), (2, 1)))
    wl.causal = False
    O, L, st = run_tree(wl, mask)
    wl.causal = True
    O_ref, L_ref = oracle.decode(wl)
    assert st == 0
    assert_parity(compare(O, L, O_ref, L_ref), "chain")


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_ragged_trees_no_tree_no_tokens_and_rows_that_see_nothing(cache):
    # request 0: no node; 1: no cached token; 2: all tree, whose rows see nothing, one node, everything;
    # 3: bits past its nodes (must count for nothing); 4: a long prefix with every node slot in use
    wl = mw.make(5, 16, 16, [90, 0, 3, 133, 2000], seed=63, cache_dtype=cache, name="ragged_tree")
    lens = [0, 0, 3, 9, 16]
    mask = oracle.tree_mask(parents_of(5, 16, seed=64))
    mask[2, 0], mask[2, 1], mask[2, 2] = 0, 1, 7
    mask[3] = -1
    O, L = check(wl, mask, lens)
    assert np.isneginf(L[2, 0]).all() and (O[2, 0] == 0).all() and np.isneginf(L[0]).all() and np.isneginf(L[3, 9:]).all()


def test_without_counts_a_short_request_holds_as_many_nodes_as_tokens():
    wl = mw.make(3, 16, 40, [5, 16, 17], seed=74, name="short_tree")
    O, L = check(wl, oracle.tree_mask(np.tile(np.arange(-1, 15, dtype=np.int32), (3, 1))))
    assert np.isneginf(L[0, 5:]).all() and np.isfinite(L[0, :5]).all()


def test_two_calls_at_once_on_two_streams():
    wl = mw.make(3, 8, 64, [900, 65, 2000], seed=75)
    dev = to_device(wl)
    masks = [oracle.tree_mask(parents_of(3, 8, seed=s)) for s in (76, 77)]
    decs = [mla.TreeDecoder(shape_of(wl)) for _ in masks]
    md = [torch.from_numpy(m).cuda() for m in masks]
    outs = [torch.empty((3, 8, 64, 512), dtype=torch.bfloat16, device="cuda") for _ in masks]
    lses = [torch.empty((3, 8, 64), dtype=torch.float32, device="cuda") for _ in masks]
    streams = [torch.cuda.Stream() for _ in masks]
    torch.cuda.synchronize()
    for _ in range(4):
        for k in range(2):
            decs[k].decode(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], md[k], wl.softmax_scale, outs[k],
                           lses[k], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert decs[k].status() == 0
        O_ref, L_ref = oracle.tree_decode(wl, masks[k])
        assert_parity(compare(outs[k].float().cpu().numpy(), lses[k].cpu().numpy(), O_ref, L_ref), f"stream {k}")


def test_nodes_behind_the_last_page_are_not_read():
    # NaN behind every length and in RoPE columns of a node that nobody sees: no trace in the output
    wl = mw.make(2, 12, 128, [100, 75], seed=65, name="poison")
    for r, t in enumerate(wl.seqlens):
        wl.pool[wl.block_table[r, t // 64], t % 64:] = float("nan")
    mask = oracle.tree_mask(parents_of(2, 12, seed=66))
    mask &= ~np.int64(1 << 5)
    mask[:, 5] = 1
    pos = 100 - 12 + 5
    wl.pool[wl.block_table[0, pos // 64], pos % 64, 512:] = float("nan")
    O, L, st = run_tree(wl, mask)
    assert st == 0 and np.isfinite(O).all()
    wl.pool[wl.block_table[0, pos // 64], pos % 64, 512:] = 0
    O_ref, L_ref = oracle.tree_decode(wl, mask)
    assert_parity(compare(O, L, O_ref, L_ref), "poison")


def test_bad_counts_and_pages_are_flagged():
    wl = mw.make(2, 4, 16, [100, 3], seed=67)
    mask = oracle.tree_mask(parents_of(2, 4, seed=68))
    _, _, st = run_tree(wl, mask, [5, 2])
    assert st == -6
    O, L, st = run_tree(wl, mask, [-1, 4])              # clamped to 0 and to the request's 3 tokens
    assert st == -6
    O_ref, L_ref = oracle.tree_decode(wl, mask, [0, 3])
    assert_parity(compare(O, L, O_ref, L_ref), "clamped")
    wl.block_table[0, 1] = wl.num_pages
    _, _, st = run_tree(wl, mask, [4, 3])
    assert st == -6


def test_tree_decode_replays_from_a_graph_with_new_trees_and_lengths():
    wl = mw.make(3, 8, 16, [300, 500, 700], seed=69)
    dev, dec = to_device(wl), mla.TreeDecoder(shape_of(wl))
    out = torch.empty((3, 8, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 8, 16), dtype=torch.float32, device="cuda")
    par = torch.from_numpy(parents_of(3, 8, seed=70)).cuda()
    dl = torch.tensor([8, 8, 8], dtype=torch.int32, device="cuda")
    mask = torch.empty((3, 8, 1), dtype=torch.int64, device="cuda")

    def step():
        mla.mla_tree_mask(par, mask, dl)
        dec.decode(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], mask, wl.softmax_scale, out, lse, draft_lens=dl)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, t, n in ((71, [300, 100, 650], [8, 3, 0]), (72, [8, 500, 77], [8, 8, 5])):
        p = parents_of(3, 8, seed)
        par.copy_(torch.from_numpy(p))
        dl.copy_(torch.tensor(n))
        wl.seqlens = np.array(t, dtype=np.int32)
        dev["seqlens"].copy_(torch.from_numpy(wl.seqlens))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert dec.status() == 0
        m = oracle.tree_mask(p, n)
        assert np.array_equal(mask.cpu().numpy(), m)
        O_ref, L_ref = oracle.tree_decode(wl, m, n)
        assert_parity(compare(out.float().cpu().numpy(), lse.cpu().numpy(), O_ref, L_ref), f"replay {seed}")


def test_binding_checks():
    wl = mw.make(2, 4, 16, [100, 30], seed=73)
    dev, dec = to_device(wl), mla.TreeDecoder(shape_of(wl))
    out = torch.empty((2, 4, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4, 16), dtype=torch.float32, device="cuda")
    mask = torch.zeros((2, 4, 1), dtype=torch.int64, device="cuda")
    args = (dev["q"], dev["pool"], dev["block_table"], dev["seqlens"])
    with pytest.raises(TypeError):
        dec.decode(*args, mask.int(), 0.1, out, lse)
    with pytest.raises(ValueError):
        dec.decode(*args, mask[:, :3], 0.1, out, lse)
    with pytest.raises(ValueError):
        dec.decode(*args, mask, 0.1, out, lse, draft_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(mla.MLAError):
        mla.TreeDecoder(mla.make_shape(2, 4, 16, 2, 4, causal=True))


@pytest.mark.parametrize("what", ["count", "length"])
def test_status_stays_until_it_is_read_and_is_cleared_by_the_read(what):
    # several steps are enqueued before the host looks: a flag of one of them outlives the good steps behind it
    wl = mw.make(2, 4, 16, [100, 30], seed=110)
    dev, dec = to_device(wl), mla.TreeDecoder(shape_of(wl))
    mask = torch.from_numpy(oracle.tree_mask(parents_of(2, 4, seed=111))).cuda()
    out = torch.empty((2, 4, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4, 16), dtype=torch.float32, device="cuda")
    good = torch.tensor([4, 2], dtype=torch.int32, device="cuda")
    bad_count = torch.tensor([5, 2], dtype=torch.int32, device="cuda")
    bad_length = torch.tensor([wl.max_pages * 64 + 1, 30], dtype=torch.int32, device="cuda")

    def step(lens, seqlens):
        dec.decode(dev["q"], dev["pool"], dev["block_table"], seqlens, mask, wl.softmax_scale, out, lse, draft_lens=lens)
    step(good, dev["seqlens"])
    assert dec.status() == 0
    if what == "count":
        step(bad_count, dev["seqlens"])
    else:
        step(good, bad_length)
    step(good, dev["seqlens"])
    assert dec.status() == -6
    assert dec.status() == 0
    step(good, dev["seqlens"])
    assert dec.status() == 0


@pytest.mark.parametrize("b,s", [(1, 8193), (3, 8300), (2, 20000)])
def test_tree_mask_bits_of_large_trees(b, s):
    par = parents_of(b, s, seed=s)
    par[0, 5000:] = np.maximum(par[0, 5000:], np.arange(5000, s) - 40)     # deep: parents near their children
    par[-1, 70], par[-1, 100], par[-1, s - 1] = 70, -9, s                   # bad ones: -1
    lens = np.array([s - 33 * r for r in range(b)], dtype=np.int32)
    lens[-1] = s + 1 if b == 2 else lens[-1]                                # a count past the slots
    m = torch.full((b, s, (s + 63) // 64), -1, dtype=torch.int64, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_tree_mask(torch.from_numpy(par).cuda(), m, torch.from_numpy(lens).cuda(), st)
    got = m.cpu().numpy().view(np.uint64)
    assert st.item() != 0
    for r in range(b):
        ref = np.zeros_like(got[r])
        for i in range(min(s, int(lens[r]))):           # a row is its parent's and the node's own bit
            p = par[r, i]
            if 0 <= p < i:
                ref[i] = ref[p]
            ref[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        assert np.array_equal(got[r], ref)


def test_tree_mask_of_a_long_chain_takes_no_time_worth_mentioning():
    # time that grows as nodes x words (a walk of every path by every word would take seconds here)
    s = 131072
    par = torch.arange(-1, s - 1, dtype=torch.int32, device="cuda")[None]
    m = torch.full((1, s, s // 64), 77, dtype=torch.int64, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    mla.mla_tree_mask(par, m, None, st)
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) < 1000.0 and st.item() == 0
    w = torch.arange(s // 64, device="cuda")
    for i0 in range(0, s, 8192):
        n = (torch.arange(i0, i0 + 8192, device="cuda")[:, None] + 1 - 64 * w).clamp(0, 64)
        ref = torch.where(n == 64, -1, (1 << n.clamp(max=63)) - 1)
        assert torch.equal(m[0, i0:i0 + 8192], ref)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("b,s,heads,top", [(8, 6, 40, 9000), (40, 24, 16, 3000), (300, 3, 16, 500), (4000, 20, 16, 64),
                                           (26000, 1, 1, 128)])
def test_the_device_plans_what_the_host_plans(cache, b, s, heads, top):
    # the last two: more tiles than the default shared memory holds (about 6000), and more than any (about 25500)
    from schedule_plan import plan, tree_host
    g = np.random.default_rng(b)
    lengths = np.exp(g.uniform(0, np.log(top + 1), b)).astype(np.int32)
    lengths[0], lengths[-1] = top, 0
    counts = g.integers(0, s + 2, b).astype(np.int32)                  # some past what the length allows: flagged
    pages = -(-top // 64)
    sh = mla.make_shape(b, s, heads, pages, 4, cache)
    dec = mla.TreeDecoder(sh)
    q = torch.zeros((b, s, heads, 576), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda") if cache == "bf16" else \
        torch.zeros((4, 40960), dtype=torch.uint8, device="cuda")
    sc = None if cache == "bf16" else torch.ones((4, 64), device="cuda")
    bt = torch.zeros((b, pages), dtype=torch.int32, device="cuda")
    mask = torch.full((b, s, 1), -1, dtype=torch.int64, device="cuda")
    out = torch.empty((b, s, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b, s, heads), device="cuda")
    for dl in (counts, None):
        dec.decode(q, pool, bt, torch.from_numpy(lengths).cuda(), mask, 0.1, out, lse, kv_scale=sc,
                   draft_lens=None if dl is None else torch.from_numpy(dl).cuda())
        ref = tree_host(sh, lengths, dl, dec.n_sms)
        assert np.array_equal(dec.workspace[:ref.nbytes].cpu().numpy().view(np.int32), ref)
        assert (dec.status() == -6) == (ref[6] != 0) and (ref[6] != 0) == (dl is not None)
        n = np.minimum(lengths, s) if dl is None else np.clip(dl, 0, np.minimum(lengths, s))
        live = lse.isfinite().view(b, s, heads).all(2).sum(1).cpu().numpy()
        assert np.array_equal(live, n)
