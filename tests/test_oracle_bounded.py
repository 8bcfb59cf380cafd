"""Pins of the oracle's anchored attention, accumulated weights and eviction: torch's attention with an
explicit mask in fp64, closed forms, and brute force."""

import itertools

import numpy as np
import pytest
import torch

import oracle as O


def _qkv(rng, n, ctx, H_q, H_kv, d):
    return rng.standard_normal((n, H_q, d)), rng.standard_normal((ctx, H_kv, d)), rng.standard_normal((ctx, H_kv, d))


@pytest.mark.parametrize("ctx,n,window,anchors", [(1, 1, 1, 0), (1, 1, 4, 9), (30, 1, 5, 3), (30, 7, 5, 3), (30, 30, 1, 1),
                                                  (30, 30, 40, 2), (33, 9, 8, 25), (33, 9, 8, 40), (20, 4, 0, 3)])
def test_anchored_attention_equals_sdpa_with_a_mask(ctx, n, window, anchors):
    rng = np.random.default_rng(ctx * 100 + n)
    q, K, V = _qkv(rng, n, ctx, 6, 2, 8)
    out, mag = O.anchored_prefill(q, K, V, 0.3, window, anchors)
    t, p = np.arange(ctx)[None], np.arange(ctx - n, ctx)[:, None]
    see = (t <= p) & ((t < anchors) | (p - t < window) | (window == 0))
    assert np.array_equal(see, O.anchored_mask(ctx, n, window, anchors))
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, np.repeat(K, 3, 1), np.repeat(V, 3, 1)))
    ref = torch.nn.functional.scaled_dot_product_attention(tq[None], tk[None], tv[None], attn_mask=torch.from_numpy(see),
                                                           scale=0.3)[0].transpose(0, 1).numpy()
    assert np.abs(out - ref).max() < 1e-12
    assert np.all(mag >= np.abs(out) - 1e-12)
    one, _ = O.anchored_decode(q[-1], K, V, 0.3, window, anchors)
    assert np.allclose(one, out[-1], atol=1e-13)


def test_anchors_that_reach_the_window_are_full_attention():
    rng = np.random.default_rng(3)
    q, K, V = _qkv(rng, 1, 50, 4, 2, 8)
    full = O.decode_attention(q[0], K, V, 0.3)
    assert np.allclose(O.anchored_decode(q[0], K, V, 0.3, 20, 30)[0], full)
    assert not np.allclose(O.anchored_decode(q[0], K, V, 0.3, 20, 29)[0], full)
    assert np.allclose(O.anchored_decode(q[0], K, V, 0.3, 20, 0)[0], O.decode_attention(q[0], K, V, 0.3, 20))


def test_weights_sum_to_the_group_and_are_the_softmax():
    rng = np.random.default_rng(4)
    q, K, V = _qkv(rng, 1, 37, 6, 2, 8)
    out, mag, w = O.decode_weights(q[0], K, V, 0.3)
    assert np.allclose(w.sum(1), 3.0)
    assert np.allclose(out, O.decode_attention(q[0], K, V, 0.3))
    s = torch.softmax(torch.einsum("hd,thd->ht", torch.from_numpy(q[0]), torch.from_numpy(np.repeat(K, 3, 1))) * 0.3, -1)
    assert np.allclose(w, s.view(2, 3, 37).sum(1).numpy())
    _, _, lw = O.decode_weights(q[0], K, V, 0.3, lo=30)
    assert np.all(lw[:, :30] == 0) and np.allclose(lw.sum(1), 3.0)
    assert O.decode_weights(q[0], K[:0], V[:0], 0.3)[2].shape == (2, 0)


def test_evict_order_by_brute_force():
    # every assignment of three scores to five slots: what stays is protected or scores at least what goes
    for sc in itertools.product([0.0, 1.0, 2.0], repeat=5):
        order = O.evict_order(sc, np.arange(5), 1, 1).tolist()
        assert order[:2] == [0, 4]
        rest = order[2:]
        assert all(sc[a] > sc[b] or (sc[a] == sc[b] and a < b) for a, b in zip(rest, rest[1:]))


def test_evict_order_special_values_and_positions():
    sc = [np.nan, -np.inf, 0.0, np.inf, -0.0, 1.0]
    # no slot protected (the newest position is past all of them only through recent = 0)
    assert O.evict_order(sc, np.arange(6), 0, 0).tolist() == [3, 5, 2, 4, 1, 0]
    # positions, not slots, decide what is recent: slot 0 holds the newest token
    assert O.evict_order(sc, [9, 1, 2, 3, 4, 5], 0, 1)[0] == 0
    assert set(O.evict_order(sc, [9, 1, 2, 3, 8, 0], 2, 2)[:4].tolist()) == {0, 1, 4, 5}


@pytest.mark.parametrize("n,budget", [(0, 4), (1, 4), (4, 4), (5, 4), (40, 4), (40, 39), (40, 1)])
def test_evict_plan_keeps_the_budget_and_fills_every_hole(n, budget):
    rng = np.random.default_rng(n * 50 + budget)
    sc = rng.random(n)
    holes, movers = O.evict_plan(sc, np.arange(n), budget, min(1, budget), 0)
    left = min(n, budget)
    slots = list(range(left))
    for h, m in zip(holes, movers):
        slots[h] = m
    assert sorted(slots) == sorted(O.evict_order(sc, np.arange(n), min(1, budget), 0)[:left].tolist())
    assert all(h < left <= m for h, m in zip(holes, movers))


def test_evict_rows_moves_every_part_of_a_row():
    rng = np.random.default_rng(8)
    c = O.PagedKVCache(4, 2, 128, k_dtype="int4", v_dtype="int4", num_seqs=1)
    row = np.array([2, 0, 3])
    for p in range(40):
        c.append(0, row, p, *(rng.integers(0, 1 << 14, (2, 128)).astype(np.uint16) for _ in range(2)))
    K, V = c.gather(0, row, 40)
    O.evict_rows(c, row, 1, [3, 17], [33, 39])
    K2, V2 = c.gather(0, row, 40)
    for a, b in ((K, K2), (V, V2)):
        assert np.array_equal(b[3, 1], a[33, 1]) and np.array_equal(b[17, 1], a[39, 1])
        same = np.ones((40, 2), dtype=bool)
        same[3, 1] = same[17, 1] = False
        assert np.array_equal(a[same], b[same])


def test_slide_window_anchored_keeps_the_anchors_blocks():
    pool = O.BlockPool(10)
    row = np.array([pool.alloc() for _ in range(8)])
    before = row.copy()
    assert O.slide_window_anchored(pool, row, 120, 40, 17) == 3  # blocks 2, 3, 4 of the 5 before position 80
    assert np.array_equal(row[:2], before[:2]) and np.all(row[2:5] == -1) and np.array_equal(row[5:], before[5:])
    assert pool.num_free() == 5
    assert O.slide_window_anchored(pool, row, 120, 0, 17) == 0


def test_planted_mistakes_are_caught():
    rng = np.random.default_rng(9)
    q, K, V = _qkv(rng, 5, 40, 4, 2, 8)
    ref, _ = O.anchored_prefill(q, K, V, 0.5, 6, 3)
    for wrong in (O.anchored_mask(40, 5, 6, 4), O.anchored_mask(40, 5, 7, 3), O.anchored_mask(40, 5, 6, 0)):
        assert np.abs(O.masked_attention(q, K, V, 0.5, wrong)[0] - ref).max() > 1e-3
