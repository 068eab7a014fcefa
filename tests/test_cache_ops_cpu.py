"""Host-side checks of the tree decode, the attention weights, the eviction
and the compaction (no GPU): argument checks, workspace sizes, the schedule
of ragged trees, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import mla_latent_space_b200 as mla
import mla_workloads as mw
import oracle

FAKE = ctypes.c_void_p(1 << 20)     # never dereferenced: validation fails first


def off(n):
    return ctypes.c_void_p((1 << 20) + n)


def shape(**kw):
    base = dict(batch=2, s_q=8, num_heads=128, max_pages_per_seq=4, num_pages=8)
    base.update(kw)
    return mla.make_shape(**base)


def test_tree_workspace_and_argument_checks():
    L = mla.lib()
    nb = L.mla_tree_workspace_bytes(ctypes.byref(shape()), 148)
    assert nb >= mla.mla_schedule_bytes(shape(), 148) + mla.mla_workspace_bytes(shape(), 148)
    assert nb % 4 == 0
    assert L.mla_tree_workspace_bytes(ctypes.byref(shape(causal=True)), 148) == 0
    assert L.mla_tree_workspace_bytes(ctypes.byref(shape()), 0) == 0

    def call(sh=None, q=FAKE, kv=FAKE, sc=None, bt=FAKE, sl=FAKE, dl=None, mask=FAKE, scale=0.1, ws=FAKE, nb=1 << 40,
             out=FAKE, lse=FAKE):
        return L.mla_tree_decode_fwd(ctypes.byref(shape() if sh is None else sh), q, kv, sc, bt, sl, dl, mask, scale, ws,
                                     nb, out, lse, None)
    assert call(sh=shape(causal=True)) == -1
    for kw in (dict(mask=None), dict(mask=off(4)), dict(dl=off(2)), dict(ws=None), dict(ws=off(16))):
        assert call(**kw) == -1, kw
    bad = shape()
    bad.d_v = 128
    assert call(sh=bad) == -2
    assert L.mla_tree_get_device_status(ctypes.byref(shape()), 148, None, None, None) == -1


def test_tree_mask_argument_checks():
    L = mla.lib()

    def call(b=2, s=8, par=FAKE, dl=None, mask=FAKE, st=None):
        return L.mla_tree_mask(b, s, par, dl, mask, st, None)
    for kw in (dict(b=0), dict(s=0), dict(par=None), dict(mask=None), dict(par=off(2)), dict(mask=off(4)), dict(dl=off(1)),
               dict(st=off(2))):
        assert call(**kw) == -1, kw
    assert call(b=65536) == -2
    assert call(s=(1 << 20) + 1) == -2


def test_attn_weights_argument_checks():
    L = mla.lib()

    def call(sh=None, q=FAKE, kv=FAKE, sc=None, bt=FAKE, sl=FAKE, lse=FAKE, scale=0.1, decay=0.5, w=FAKE, ws=FAKE,
             nb=1 << 40):
        return L.mla_attn_weights_fwd(ctypes.byref(shape() if sh is None else sh), q, kv, sc, bt, sl, lse, scale, decay, w,
                                      ws, nb, None)
    for kw in (dict(q=None), dict(q=off(8)), dict(kv=off(128)), dict(bt=off(2)), dict(sl=None), dict(lse=off(2)), dict(w=None),
               dict(w=off(2)), dict(ws=None), dict(ws=off(16)), dict(scale=float("nan")), dict(decay=float("inf")),
               dict(sh=shape(cache_dtype="fp8"))):
        assert call(**kw) == -1, kw
    assert call(sh=shape(batch=65536, s_q=1, num_heads=1)) == -2
    assert call(sh=shape(batch=1, s_q=65535, num_heads=1)) == -2
    assert L.mla_attn_weights_workspace_bytes(ctypes.byref(shape(batch=1, s_q=65535, num_heads=1)), 148) == 0
    assert L.mla_attn_weights_workspace_bytes(ctypes.byref(shape()), 148) >= 256
    assert L.mla_attn_weights_workspace_bytes(ctypes.byref(shape()), 0) == 0
    assert L.mla_attn_weights_workspace_bytes(ctypes.byref(shape(batch=65536, s_q=1, num_heads=1)), 148) == 0
    # the workspace does not grow with the longest length a request may reach
    long_ = L.mla_attn_weights_workspace_bytes(ctypes.byref(shape(max_pages_per_seq=16384)), 148)
    assert long_ <= 64 << 20
    assert L.mla_attn_weights_get_device_status(None, None, None) == -1


def test_evict_select_argument_checks():
    L = mla.lib()

    def call(b=2, T=256, w=FAKE, sl=FAKE, budget=16, sink=4, recent=4, kept=FAKE, lens=FAKE, st=None):
        return L.mla_evict_select(b, T, w, sl, budget, sink, recent, kept, lens, st, None)
    for kw in (dict(b=0), dict(T=0), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=9, recent=8), dict(w=None),
               dict(sl=None), dict(kept=None), dict(lens=None), dict(w=off(2)), dict(kept=off(2)), dict(lens=off(1)),
               dict(st=off(2)), dict(sink=2**31 - 1, recent=2**31 - 1, budget=2**31 - 1)):
        assert call(**kw) == -1, kw
    assert call(T=(1 << 30) + 1) == -2
    assert call(budget=(1 << 30) + 1) == -2
    assert call(b=(1 << 24) + 1) == -2


def test_compact_argument_checks():
    L = mla.lib()

    def call(sh=None, kv=FAKE, sc=None, bt=FAKE, src=FAKE, sl=FAKE, base=None, rows=64, w=None, ws=FAKE, nb=1 << 40):
        return L.mla_cache_compact(ctypes.byref(shape() if sh is None else sh), kv, sc, bt, src, sl, base, rows, w, ws, nb, None)
    for kw in (dict(kv=None), dict(kv=off(128)), dict(bt=None), dict(src=None), dict(src=off(2)), dict(sl=None), dict(base=off(2)),
               dict(rows=0), dict(w=off(2)), dict(ws=None), dict(ws=off(16)), dict(sh=shape(cache_dtype="fp8"))):
        assert call(**kw) == -1, kw
    assert call(nb=8) == -3
    assert call(rows=(1 << 30) + 1) == -2
    assert L.mla_compact_workspace_bytes(ctypes.byref(shape()), 0) == 0
    assert L.mla_compact_workspace_bytes(ctypes.byref(shape()), 64) >= 256
    assert L.mla_compact_get_device_status(None, None, None) == -1


def test_binding_refuses_what_the_kernels_do_not_take(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = torch.zeros((2, 8), dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_tree_mask(t, torch.zeros((2, 8, 1), dtype=torch.int64))         # CPU tensors
    with pytest.raises(TypeError):
        mla.mla_tree_mask([0, 1], None)
    with pytest.raises(ValueError):
        mla.mla_evict_select(torch.zeros((2, 8)), t[:, 0], 4, 0, 0, t, t[:, 0])


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    class On(torch.Tensor):
        """A tensor that says it is on a GPU."""
        index = 0

        def get_device(self):
            return self.index

        @property
        def is_cuda(self):
            return True
    t = torch.zeros((2, 3)).as_subclass(On)
    mla._need_here(0, t, "t", torch.float32, (2, 3))
    with pytest.raises(ValueError, match="current device"):
        mla._need_here(1, t, "t", torch.float32, (2, 3))
    for dtype, shape, error in ((torch.int32, (2, 3), TypeError), (torch.float32, (3, 2), ValueError)):
        with pytest.raises(error):
            mla._need_here(0, t, "t", dtype, shape)


# ---- the oracle's own pins ----------------------------------------------------

def test_oracle_tree_mask_of_chain_star_and_bad_parents():
    chain = np.array([[-1, 0, 1, 2]])
    assert [int(x) for x in oracle.tree_mask(chain)[0, :, 0]] == [1, 3, 7, 15]
    star = np.array([[-1, 0, 0, 0]])
    assert [int(x) for x in oracle.tree_mask(star, [3])[0, :, 0]] == [1, 3, 5, 0]
    bad = np.array([[-1, 5, -7, 3]])                                            # a parent outside [-1, i) is -1
    assert [int(x) for x in oracle.tree_mask(bad)[0, :, 0]] == [1, 2, 4, 8]
    deep = np.arange(-1, 129)[None]                                             # words past the first
    m = oracle.tree_mask(deep).view(np.uint64)
    assert int(m[0, 129, 0]) == 2**64 - 1 and int(m[0, 129, 2]) == 3 and int(m[0, 5, 1]) == 0


def test_oracle_tree_of_a_chain_is_the_causal_decode():
    wl = mw.make(2, 5, 3, [7, 70], causal=True, seed=1)
    O, L = oracle.tree_decode(wl, oracle.tree_mask(np.tile(np.arange(-1, 4), (2, 1))))
    O_ref, L_ref = oracle.decode(wl)
    assert np.allclose(O, O_ref, atol=1e-12) and np.allclose(L, L_ref, atol=1e-12)


def test_oracle_weights_sum_to_the_number_of_rows():
    wl = mw.make(2, 2, 3, [9, 70], seed=2)
    _, lse = oracle.decode(wl)
    w = oracle.attn_weights(wl, lse, 0.0, np.full((2, wl.max_pages * 64), 7.0))
    for r, t in enumerate(wl.seqlens):
        assert abs(w[r, :t].sum() - 6.0) < 1e-12 and (w[r, t:] == 7.0).all()


def test_oracle_select_keeps_sink_recent_and_the_heaviest():
    w = np.array([[0.0, 5.0, 1.0, 1.0, np.nan, 1.0, 9.0, 0.0]])
    kept, n = oracle.evict_select(w, [8], 5, 1, 1)
    assert kept.tolist() == [[0, 1, 2, 6, 7]] and n.tolist() == [5]
    kept, n = oracle.evict_select(w, [3], 5, 1, 1)
    assert kept.tolist() == [[0, 1, 2, -1, -1]] and n.tolist() == [3]


def _schedule(parents_lens, seqlens, s_q, heads):
    # the host planner knows no trees: the device scheduler's page counts are checked on the GPU through the status
    return mla.mla_plan_schedule_host(mla.make_shape(len(seqlens), s_q, heads, 8, 8), torch.tensor(seqlens), 148)


def test_plain_schedule_is_unchanged_by_the_tree_fields():
    sc = _schedule(None, [100, 300], 16, 128)
    tiles = sc[16 + 74 * 8:].view(-1, 4)
    assert tiles[:16, 0].tolist() == [2] * 16 and tiles[16:32, 0].tolist() == [5] * 16


@pytest.mark.parametrize("cls", ["TreeDecoder", "AttnWeights", "CacheCompactor"])
def test_status_is_read_on_the_device_that_ran_the_calls(monkeypatch, cls):
    # on another device's stream the read would not wait for the calls
    class On(torch.Tensor):
        def get_device(self):
            return 1

        @property
        def is_cuda(self):
            return True
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mla, "_stream_of", lambda dev, stream: None)
    obj = getattr(mla, cls).__new__(getattr(mla, cls))
    obj.shape, obj.n_sms = shape(), 148
    obj.workspace = torch.zeros(256, dtype=torch.uint8).as_subclass(On)
    with pytest.raises(ValueError, match="current device"):
        obj.status()


def test_binding_does_not_let_a_count_wrap_to_32_bits(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mla, "_need_here", lambda *a: None)
    monkeypatch.setattr(mla, "_stream_of", lambda dev, stream: None)
    monkeypatch.setattr(mla, "lib", lambda real=mla.lib(): Passes(real))

    class Passes:
        """The library, but for the choice, which would take what reaches it."""
        def __init__(self, real):
            self.mla_error_string = real.mla_error_string
            self.mla_evict_select = lambda *a: 0
    w, n, kept = torch.zeros((2, 64)), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 16), dtype=torch.int32)
    mla.mla_evict_select(w, n, 16, 4, 4, kept, n)
    for sink, recent in ((2**32, 0), (4, 2**32 + 4), (-1, 0), (0, -2**32), (9, 8)):
        with pytest.raises(mla.MLAError):
            mla.mla_evict_select(w, n, 16, sink, recent, kept, n)
