"""The host planner, plain and for drafted trees, word by word against the
schedule's definition."""
import numpy as np
import pytest
import torch

import mla_latent_space_b200 as mla
from schedule_plan import plan, tree_host

SHAPES = [
    # s_q, heads, max_pages, lengths
    (1, 128, 64, [4096] * 64),                  # the headline batch: whole tiles
    (1, 128, 200, [12000, 64, 3, 0, 700]),      # jagged: cut tiles
    (16, 128, 8, [100, 300]),
    (16, 128, 64, [4096] * 8),
    (5, 40, 100, [6000, 1, 64, 65, 6400]),
    (24, 16, 128, [500, 8000, 77, 0, 1300, 24, 5]),
    (1, 1, 3, [1]),
    (8, 16, 16, [0, 0]),                        # no work
    (3, 7, 40, [-1, 2561, 100]),                # lengths out of range: clamped and flagged
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("s_q,heads,max_pages,lengths", SHAPES)
@pytest.mark.parametrize("n_sms", [148, 12])
def test_plain_schedule_is_its_definition(s_q, heads, max_pages, lengths, causal, n_sms):
    sh = mla.make_shape(len(lengths), s_q, heads, max_pages, 8, causal=causal)
    got = mla.mla_plan_schedule_host(sh, torch.tensor(lengths), n_sms).numpy()
    assert np.array_equal(got, plan(lengths, s_q, heads, max_pages, n_sms // 2, causal=causal))


@pytest.mark.parametrize("cache,overhead", [("bf16", 6), ("fp8", 14)])
@pytest.mark.parametrize("s_q,heads,max_pages,lengths", SHAPES)
@pytest.mark.parametrize("n_sms", [148, 12])
def test_tree_schedule_is_its_definition(s_q, heads, max_pages, lengths, cache, overhead, n_sms):
    sh = mla.make_shape(len(lengths), s_q, heads, max_pages, 8, cache)
    g = np.random.default_rng(s_q + heads)
    for counts in (None, [s_q] * len(lengths), g.integers(0, s_q + 1, len(lengths)), g.integers(-1, s_q + 2, len(lengths)),
                   [0] * len(lengths)):
        got = tree_host(sh, lengths, counts, n_sms)
        assert np.array_equal(got, plan(lengths, s_q, heads, max_pages, n_sms // 2, overhead, tree=True, draft_lens=counts))


def test_every_page_of_every_tile_is_some_workers():
    for cache in ("bf16", "fp8"):
        g = np.random.default_rng(5)
        for _ in range(20):
            b, s_q, heads = int(g.integers(1, 9)), int(g.integers(1, 30)), int(g.integers(1, 40))
            lengths = np.exp(g.uniform(0, 9, b)).astype(int)
            sc = tree_host(mla.make_shape(b, s_q, heads, 128, 8, cache), lengths, g.integers(0, s_q + 1, b), 148)
            wk, tl = sc[16:16 + 74 * 8].reshape(74, 8), sc[16 + 74 * 8:].reshape(-1, 4)
            walked, pieces = np.zeros(len(tl), dtype=int), [[] for _ in tl]
            for t0, p0, t1, p1, split in wk[:, :5]:
                for t in range(t0, min(t1 + 1, len(tl))):
                    a, e = p0 if t == t0 else 0, p1 if t == t1 else tl[t, 0]
                    if a < e:
                        walked[t] += e - a
                        pieces[t].append(split if t == t0 else 0)
            assert np.array_equal(walked, tl[:, 0])
            assert all(p == list(range(n)) for p, n in zip(pieces, tl[:, 2]))
            assert sc[5] == sum(n for n in tl[:, 2] if n > 1) <= 2 * 74
