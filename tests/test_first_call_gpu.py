"""The operators around the cache in a fresh process: captured by a graph in
their first call, and called after a call that failed on the host.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import mla_latent_space_b200 as mla, mla_workloads as mw, oracle
from gpu_helpers import assert_parity, compare, to_device
"""

CAPTURED = """
cache = sys.argv[1]
wl = mw.make(3, 4, 16, [300, 64, 900], seed=130, cache_dtype=cache)
dev = to_device(wl)
par = np.tile(np.array([-1, 0, 0, 1], dtype=np.int32), (3, 1))
par_d = torch.from_numpy(par).cuda()
mask = torch.empty((3, 4, 1), dtype=torch.int64, device="cuda")
out = torch.empty((3, 4, 16, 512), dtype=torch.bfloat16, device="cuda")
lse = torch.empty((3, 4, 16), device="cuda")
sh = mla.make_shape(3, 4, 16, wl.max_pages, wl.num_pages, cache)
tree, acc, comp = mla.TreeDecoder(sh), mla.AttnWeights(sh), mla.CacheCompactor(sh, 60)
w = torch.zeros((3, wl.max_pages * 64), device="cuda")
long_w = torch.rand((3, 20000), device="cuda")
long_l = torch.tensor([20000, 50, 9000], dtype=torch.int32, device="cuda")
kept = torch.empty((3, 60), dtype=torch.int32, device="cuda")
n = torch.empty(3, dtype=torch.int32, device="cuda")
long_kept = torch.empty((3, 1000), dtype=torch.int32, device="cuda")
long_n = torch.empty(3, dtype=torch.int32, device="cuda")
pool, sc = dev["pool"].clone(), None if dev["kv_scale"] is None else dev["kv_scale"].clone()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    mla.mla_tree_mask(par_d, mask)
    tree.decode(dev["q"], pool, dev["block_table"], dev["seqlens"], mask, wl.softmax_scale, out, lse, kv_scale=sc)
    acc.accumulate(dev["q"], pool, dev["block_table"], dev["seqlens"], lse, wl.softmax_scale, 0.5, w, kv_scale=sc)
    mla.mla_evict_select(w, dev["seqlens"], 60, 4, 8, kept, n)
    mla.mla_evict_select(long_w, long_l, 1000, 4, 8, long_kept, long_n)
    comp.compact(pool, dev["block_table"], kept, n, kv_scale=sc, weights=w)
for _ in range(2):
    pool.copy_(dev["pool"])
    if sc is not None:
        sc.copy_(dev["kv_scale"])
    w.zero_()
    g.replay()
    torch.cuda.synchronize()
    m = oracle.tree_mask(par)
    assert np.array_equal(mask.cpu().numpy(), m)
    O_ref, L_ref = oracle.tree_decode(wl, m)
    assert_parity(compare(out.float().cpu().numpy(), lse.cpu().numpy(), O_ref, L_ref), "tree")
    before = torch.zeros_like(w)
    acc.accumulate(dev["q"], dev["pool"], dev["block_table"], dev["seqlens"], lse, wl.softmax_scale, 0.5, before,
                   kv_scale=dev["kv_scale"])
    ref = oracle.attn_weights(wl, lse.cpu().numpy(), 0.5, np.zeros((3, wl.max_pages * 64)))
    assert (np.abs(before.cpu().numpy() - ref) <= 5e-4 * ref).all()
    k_ref, n_ref = oracle.evict_select(before.cpu().numpy(), wl.seqlens, 60, 4, 8)
    assert np.array_equal(kept.cpu().numpy(), k_ref) and np.array_equal(n.cpu().numpy(), n_ref)
    k_ref, l_ref = oracle.evict_select(long_w.cpu().numpy(), [20000, 50, 9000], 1000, 4, 8)
    assert np.array_equal(long_kept.cpu().numpy(), k_ref) and np.array_equal(long_n.cpu().numpy(), l_ref)
    p_ref, s_ref, w_ref = oracle.compact(wl.pool, wl.kv_scale, wl.block_table, kept.cpu().numpy(), n_ref, None, before.cpu().numpy())
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    assert torch.equal(bits(pool.cpu()), bits(p_ref)) and np.array_equal(w.cpu().numpy(), w_ref)
    assert sc is None or torch.equal(sc.cpu(), s_ref)
    assert tree.status() == 0 and acc.status() == 0 and comp.status() == 0
print("done")
"""

AFTER_AN_ERROR = """
call = sys.argv[1]
sh = mla.make_shape(2, 1, 16, 2, 4)
comp = mla.CacheCompactor(sh, 8)
pool = torch.randn((4, 64, 576), device="cuda").bfloat16()
bt = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
sl = torch.tensor([100, 70], dtype=torch.int32, device="cuda")
q = torch.randn((2, 1, 16, 576), device="cuda").bfloat16()
out = torch.empty((2, 1, 16, 512), dtype=torch.bfloat16, device="cuda")
lse, w = torch.empty((2, 1, 16), device="cuda"), torch.zeros((2, 128), device="cuda")
kept, n = torch.zeros((2, 8), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
mask = torch.ones((2, 1, 1), dtype=torch.int64, device="cuda")
tree, acc, dec = mla.TreeDecoder(sh), mla.AttnWeights(sh), mla.Decoder(sh)
calls = dict(mask=lambda: mla.mla_tree_mask(torch.full((2, 1), -1, dtype=torch.int32, device="cuda"), mask),
             tree=lambda: tree.decode(q, pool, bt, sl, mask, 0.1, out, lse),
             weights=lambda: acc.accumulate(q, pool, bt, sl, lse, 0.1, 0.0, w),
             select=lambda: mla.mla_evict_select(w, sl, 8, 1, 1, kept, n),
             compact=lambda: comp.compact(pool, bt, kept, n),
             decode=lambda: (dec.schedule(sl), dec.decode(q, pool, None, bt, sl, 0.1, out, lse)),
             noalloc=lambda: mla.mla_decode_fwd_noalloc(sh, q, pool, None, bt, sl, 0.1, out, lse))
for f in calls.values():
    f()
torch.cuda.synchronize()
refused = False
s = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
try:
    with torch.cuda.graph(g, stream=s):
        try:
            comp.status()                   # it synchronises: a capture refuses that
        except mla.MLAError as e:
            refused = e.code == -4
except Exception:                           # the capture that refused it is void
    pass
assert refused
calls[call]()                               # the other call's error is not this one's
torch.cuda.synchronize()
assert comp.status() == 0 and tree.status() == 0 and acc.status() == 0
print("done")
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_space_b200 import build
    build.build()


def run(code, *args):
    r = subprocess.run([sys.executable, "-c", SETUP % (ROOT, os.path.join(ROOT, "tests")) + code, *args],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout[-500:] + r.stderr[-2000:]


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_first_calls_of_a_process_can_be_captured(cache):
    run(CAPTURED, cache)


@pytest.mark.parametrize("call", ["mask", "tree", "weights", "select", "compact", "decode", "noalloc"])
def test_a_call_does_not_report_another_calls_error(call):
    run(AFTER_AN_ERROR, call)
