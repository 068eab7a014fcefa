"""GPU parity of the attention weights (mla_attn_weights_fwd through the C
ABI) against the fp64 oracle.

Tolerance, from the arithmetic: a term is exp(x - lse) with x = scale q . C.
The tensor core adds 576 exact products in 36 steps into an fp32 accumulator
that may truncate: each step is off by at most 2^-23 of the largest partial
sum, which is at most A = scale sum|q_d C_d|.  With N(0, 1) values A is about
0.072 * 576 * 0.64 = 27 (at most 33 over these rows), so x is off by at most
36 * 2^-23 * 33 = 1.4e-4; the steps inside one instruction add no more than
the same again.  The FP8 cache's query parts lose at most 2^-19 of the row's
largest |q| (4.5) per value: 0.072 * 512 * 0.64 * 4.5 * 2^-19 = 2e-4 more.  A
term is off by that much relative to itself, exp2 and the fp32 sum by 2^-20:
3e-4 (BF16) and 5e-4 (FP8) of the new weight, and half an fp32 step per
rounding of the old one.
"""
import numpy as np
import pytest
import torch

import mla_latent_space_b200 as mla
import mla_workloads as mw
import oracle
from gpu_helpers import shape_of, to_device

pytestmark = pytest.mark.gpu

REL_NEW = {"bf16": 3e-4, "fp8": 5e-4}
EPS = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_space_b200 import build
    build.build()
    assert torch.cuda.is_available()


def old_weights(wl, seed=9):
    return np.random.default_rng(seed).random((wl.batch, wl.max_pages * 64), dtype=np.float32)


def run(wl, lse, decay, old, acc=None, dev=None):
    dev = to_device(wl) if dev is None else dev
    acc = mla.AttnWeights(shape_of(wl)) if acc is None else acc
    w = torch.from_numpy(old).cuda()
    acc.accumulate(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], torch.from_numpy(lse).cuda(), wl.softmax_scale,
                   decay, w, kv_scale=dev["kv_scale"])
    torch.cuda.synchronize()
    return w.cpu().numpy(), acc.status()


def assert_close(wl, got, lse, decay, old):
    ref = oracle.attn_weights(wl, lse, decay, old)
    new = oracle.attn_weights(wl, lse, 0.0, old)
    for r, t in enumerate(wl.seqlens):
        assert np.array_equal(got[r, t:], old[r, t:])                  # behind the last token: as it was
        tol = REL_NEW[wl.cache_dtype] * new[r, :t] + EPS * np.abs(ref[r, :t]) + 1e-30
        err = np.abs(got[r, :t] - ref[r, :t])
        assert (err <= tol).all(), (r, float((err / tol).max()))


def lse_of(wl):
    return oracle.decode(wl)[1].astype(np.float32)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("s,heads,lens,causal,decay", [
    (1, 128, [1, 64, 700], False, 0.9),
    (1, 16, [0, 63, 65], False, 0.0),
    (1, 5, [127, 128, 129], False, 1.0),
    (3, 40, [255, 256, 257], True, 0.5),        # 120 rows, less than one tile
    (4, 64, [1000, 2, 5], True, 0.9),           # 256 rows; a length below s_q
    (7, 40, [300, 1, 90], True, 1.0),           # 280 rows: a ragged second tile
    (16, 128, [900, 17, 400], True, 0.0),       # 2048 rows
    (2, 200, [513, 64, 1], False, -0.5),        # 400 rows
])
def test_weights_parity(cache, s, heads, lens, causal, decay):
    wl = mw.make(3, s, heads, lens, causal=causal, seed=80 + s, cache_dtype=cache)
    lse, old = lse_of(wl), old_weights(wl)
    got, st = run(wl, lse, decay, old)
    assert st == 0, mla.error_string(st)
    assert_close(wl, got, lse, decay, old)


def test_weights_over_many_units_and_repeated_calls_agree_bit_for_bit():
    # enough tokens that every worker gets several ranges; the sums' order is fixed
    wl = mw.make(9, 2, 128, [4000, 1, 0, 9000, 64, 300, 12000, 129, 2500], causal=True, seed=85)
    lse, old = lse_of(wl), old_weights(wl)
    acc, dev = mla.AttnWeights(shape_of(wl)), to_device(wl)
    a, st = run(wl, lse, 0.9, old, acc, dev)
    assert st == 0
    assert_close(wl, a, lse, 0.9, old)
    for _ in range(3):
        b, st = run(wl, lse, 0.9, old, acc, dev)
        assert st == 0 and np.array_equal(a, b)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("s,heads,lens", [(5, 120, [9000, 14000, 700]), (16, 128, [12000]), (11, 100, [3000, 9, 5000])])
def test_weights_when_groups_of_tiles_meet_in_the_workspace(cache, s, heads, lens):
    # few units and many rows: each unit's tiles are shared between pairs, in groups of several and of unequal size
    wl = mw.make(len(lens), s, heads, lens, causal=True, seed=92, cache_dtype=cache)
    lse, old = lse_of(wl), old_weights(wl)
    acc, dev = mla.AttnWeights(shape_of(wl)), to_device(wl)
    a, st = run(wl, lse, 0.75, old, acc, dev)
    assert st == 0
    assert_close(wl, a, lse, 0.75, old)
    b, st = run(wl, lse, 0.75, old, acc, dev)
    assert st == 0 and np.array_equal(a, b)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_rows_without_lse_add_nothing_and_nan_behind_the_length_stays_out(cache):
    wl = mw.make(2, 4, 40, [100, 70], seed=86, cache_dtype=cache)
    lse, old = lse_of(wl), old_weights(wl)
    lse[0, 1], lse[1, :, 7] = -np.inf, -np.inf
    wl.q[0, 1] = float("nan")                                          # a padded query token may hold anything
    wl.q[1, 2, 7] = float("inf")
    for r, t in enumerate(wl.seqlens):
        page = wl.block_table[r, t // 64]
        if cache == "bf16":
            wl.pool[page, t % 64:] = float("nan")
        else:
            wl.pool[page, (t % 64) * 512:64 * 512] = 0x7F
            wl.kv_scale[page, t % 64:] = float("nan")
    got, st = run(wl, lse, 0.5, old)
    assert st == 0
    ref_wl = mw.make(2, 4, 40, [100, 70], seed=86, cache_dtype=cache)
    assert_close(ref_wl, got, lse, 0.5, old)


def test_decay_zero_does_not_read_the_old_weights():
    wl = mw.make(2, 1, 16, [100, 70], seed=87)
    lse = lse_of(wl)
    old = np.full((2, wl.max_pages * 64), np.nan, dtype=np.float32)
    got, st = run(wl, lse, 0.0, old)
    assert st == 0
    ref = oracle.attn_weights(wl, lse, 0.0, np.zeros_like(old))
    for r, t in enumerate(wl.seqlens):
        assert np.isnan(got[r, t:]).all()
        assert np.abs(got[r, :t] - ref[r, :t]).max() <= 3e-4 * ref[r, :t].max()


def test_weights_of_a_step_sum_to_its_rows():
    wl = mw.make(2, 1, 128, [900, 333], seed=88)
    got, _ = run(wl, lse_of(wl), 0.0, old_weights(wl))
    for r, t in enumerate(wl.seqlens):
        assert abs(got[r, :t].astype(np.float64).sum() - 128) <= 128 * 3e-4


def test_bad_lengths_and_pages_are_flagged_and_receive_nothing():
    wl = mw.make(2, 1, 16, [200, 130], seed=89)
    lse, old = lse_of(wl), old_weights(wl)
    good, _ = run(wl, lse, 0.5, old)
    dev = to_device(wl)
    dev["block_table"][0, 1] = wl.num_pages
    got, st = run(wl, lse, 0.5, old, dev=dev)
    assert st == -6
    assert np.array_equal(got[0, 64:128], np.float32(0.5) * old[0, 64:128])
    keep = np.r_[0:64, 128:200]
    assert np.array_equal(got[0, keep], good[0, keep]) and np.array_equal(got[1], good[1])
    dev = to_device(wl)
    dev["block_table"][1, 0] = -1
    assert run(wl, lse, 0.5, old, dev=dev)[1] == -6
    dev = to_device(wl)
    dev["seqlens"][1] = -4
    got, st = run(wl, lse, 0.5, old, dev=dev)
    assert st == -6 and np.array_equal(got[1], old[1]) and np.array_equal(got[0], good[0])
    dev = to_device(wl)
    dev["seqlens"][0] = wl.max_pages * 64 + 1                          # clamped
    assert run(wl, lse, 0.5, old, dev=dev)[1] == -6


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_two_calls_at_once_and_a_replayed_graph(cache):
    wl = mw.make(4, 2, 64, [3000, 500, 64, 1], seed=90, cache_dtype=cache)
    lse, old = lse_of(wl), old_weights(wl)
    dev, accs = to_device(wl), [mla.AttnWeights(shape_of(wl)) for _ in range(2)]
    one, _ = run(wl, lse, 0.9, old, accs[0], dev)
    l_dev, ws = torch.from_numpy(lse).cuda(), [torch.from_numpy(old).cuda() for _ in range(2)]
    args = (dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], l_dev, wl.softmax_scale, 0.9)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for acc, w, s in zip(accs, ws, streams):
            acc.accumulate(*args, w, kv_scale=dev["kv_scale"], stream=s)
    torch.cuda.synchronize()
    two = [w.cpu().numpy() for w in ws]
    seq = old
    for _ in range(3):
        seq, _ = run(wl, lse, 0.9, seq, accs[0], dev)
    assert np.array_equal(two[0], seq) and np.array_equal(two[1], seq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        accs[0].accumulate(*args, ws[0], kv_scale=dev["kv_scale"])
    ws[0].copy_(torch.from_numpy(old))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(ws[0].cpu().numpy(), one) and accs[0].status() == 0
    dev["seqlens"][0] = 1234                                            # replays read the lengths anew
    wl.seqlens[0] = 1234
    ws[0].copy_(torch.from_numpy(old))
    g.replay()
    torch.cuda.synchronize()
    got = ws[0].cpu().numpy()
    assert np.array_equal(got[0, 1234:], old[0, 1234:]) and np.array_equal(got[:, :1234], one[:, :1234])


def test_infinite_lse_and_empty_batches():
    # lse = +inf is a weight of zero; a batch without tokens is no work
    wl = mw.make(2, 1, 16, [100, 70], seed=93)
    lse, old = lse_of(wl), old_weights(wl)
    lse[1] = np.inf
    got, st = run(wl, lse, 0.5, old)
    assert st == 0 and np.array_equal(got[1, :70], np.float32(0.5) * old[1, :70])
    dev = to_device(wl)
    dev["seqlens"].zero_()
    got, st = run(wl, lse, 0.5, old, dev=dev)
    assert st == 0 and np.array_equal(got, old)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable(cache):
    """The test library's stalled call makes the MMA issuers wait for what
    never comes: after 2 s the kernel reports it, drains and returns."""
    import ctypes
    import time
    from gpu_helpers import test_lib
    fn = test_lib().mla_test_attn_weights_stalled
    fn.argtypes, fn.restype = mla.lib().mla_attn_weights_fwd.argtypes, ctypes.c_int
    wl = mw.make(2, 2, 128, [3000, 100], seed=94, cache_dtype=cache)
    lse, old = lse_of(wl), old_weights(wl)
    dev, acc = to_device(wl), mla.AttnWeights(shape_of(wl))
    l_dev, w = torch.from_numpy(lse).cuda(), torch.from_numpy(old).cuda()
    ptr = lambda t: None if t is None else t.data_ptr()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rc = fn(ctypes.byref(acc.shape), ptr(dev["q"]), ptr(dev["pool"]), ptr(dev["kv_scale"]), ptr(dev["block_table"]),
            ptr(dev["seqlens"]), ptr(l_dev), wl.softmax_scale, 0.5, ptr(w), ptr(acc.workspace), acc.workspace.numel(),
            torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert 1.0 < time.perf_counter() - t0 < 30.0
    assert acc.status() == -5 and acc.status() == 0
    acc.workspace.zero_()                                               # as the header asks after a timeout
    got, st = run(wl, lse, 0.5, old, acc, dev)
    assert st == 0
    assert_close(wl, got, lse, 0.5, old)


def test_binding_checks():
    wl = mw.make(2, 1, 16, [100, 70], seed=91)
    dev, acc = to_device(wl), mla.AttnWeights(shape_of(wl))
    lse = torch.zeros((2, 1, 16), device="cuda")
    w = torch.zeros((2, wl.max_pages * 64), device="cuda")
    args = (dev["q"], dev["pool"], dev["block_table"], dev["seqlens"])
    with pytest.raises(ValueError):
        acc.accumulate(*args, lse, 0.1, 0.5, w[:, :-1])
    with pytest.raises(TypeError):
        acc.accumulate(*args, lse.double(), 0.1, 0.5, w)
    with pytest.raises(mla.MLAError):
        acc.accumulate(*args, lse, 0.1, float("nan"), w)


def test_scores_that_are_exact_give_weights_as_near_as_their_exponent():
    """Whole numbers whose products and sums the accumulator holds exactly: x = 576 - k, lse = 576, a weight of e^-k.

    The exponent x log2(e) - lse log2(e) is one fused multiply-add of the rounded scale and the rounded lse: off by
    at most 2^-24 (|x| + |lse|) log2(e) and half a step of the result, and a weight by ln 2 times that (1152 * 2^-24 =
    6.9e-5); exp2 and the sum of four equal terms by 2^-20 more.
    """
    wl = mw.make(1, 1, 4, [200], seed=112)
    wl.softmax_scale = 1.0
    wl.q[:] = 1.0
    k = np.arange(200) % 60
    rows = torch.ones((200, 576), dtype=torch.bfloat16)
    for j in range(200):
        rows[j, 7 * j % 500:7 * j % 500 + k[j]] = 0.0
    for j in range(200):
        wl.pool[wl.block_table[0, j // 64], j % 64] = rows[j]
    got, st = run(wl, np.full((1, 1, 4), 576.0, dtype=np.float32), 0.0, old_weights(wl))
    ref = 4.0 * np.exp(-k.astype(np.float64))
    assert st == 0
    assert (np.abs(got[0, :200] - ref) <= (1152 * 2.0 ** -24 + 2.0 ** -20) * ref).all()
