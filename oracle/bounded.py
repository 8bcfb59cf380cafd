"""Oracle of the operators that keep a cache bounded: anchors beside a sliding window, accumulated
attention weights, and eviction by them.  Plain numpy in fp64; test infrastructure like the rest of
this package.

Sliding window: untitled KV-cache article at ldpk.cn/news/58971 §5.3.  First tokens: "KV Cache 的显存
账本：PagedAttention 与连续批处理" §七 (attention sinks).  Eviction of the positions that attention has
looked at least: ldpk §5.3.
"""

from __future__ import annotations

import numpy as np

from .paged_kv import BLOCK_SIZE, locate, softmax_weights, window_start

__all__ = ["anchored_mask", "masked_attention", "anchored_decode", "anchored_prefill", "gather_positions",
           "slide_window_anchored", "decode_weights", "evict_order", "evict_plan", "evict_rows"]


def anchored_mask(ctx: int, n: int, window: int, anchors: int) -> np.ndarray:
    """[n][ctx] truth values: which positions the queries at ctx - n .. ctx - 1 attend."""
    m = np.zeros((n, ctx), dtype=bool)
    for i in range(n):
        p = ctx - n + i
        m[i, window_start(p + 1, window):p + 1] = True
        m[i, :min(anchors, p + 1)] = True
    return m


def masked_attention(q, K, V, scale, mask):
    """softmax over the allowed positions, times V; q [n][H_q][d], K and V [ctx][H_kv][d], mask [n][ctx].
    Returns (out [n][H_q][d], magnitude [n][H_q][d]) where magnitude is the same average of |V|, which
    bounds what relative errors of the weights and of V do to the output."""
    q = np.asarray(q, dtype=np.float64)
    n, H_q, d = q.shape
    G = H_q // K.shape[1]
    out, mag = np.zeros((n, H_q, d)), np.zeros((n, H_q, d))
    for i in range(n):
        t = np.nonzero(mask[i])[0]
        if len(t) == 0:
            continue
        for h in range(H_q):
            w = softmax_weights(scale * (K[t, h // G] @ q[i, h]))
            out[i, h] = w @ V[t, h // G]
            mag[i, h] = w @ np.abs(V[t, h // G])
    return out, mag


def anchored_decode(q, K, V, scale, window, anchors):
    """Decode: q [H_q][d] at position ctx - 1; (out, magnitude) as masked_attention."""
    o, m = masked_attention(np.asarray(q)[None], K, V, scale, anchored_mask(K.shape[0], min(1, K.shape[0]), window, anchors)
                            if K.shape[0] else np.zeros((1, 0), dtype=bool))
    return o[0], m[0]


def anchored_prefill(q, K, V, scale, window, anchors):
    """Prefill of the last n positions: q [n][H_q][d]."""
    return masked_attention(q, K, V, scale, anchored_mask(K.shape[0], len(q), window, anchors))


def gather_positions(cache, seq, table_row, positions):
    """K and V rows of the given positions of a PagedKVCache; no other table entry is looked up."""
    K = np.zeros((len(positions), cache.num_kv_heads, cache.head_dim))
    V = np.zeros_like(K)
    for i, p in enumerate(positions):
        k, v = cache.gather(seq, table_row, int(p) + 1, int(p))
        K[i], V[i] = k[0], v[0]
    return K, V


def slide_window_anchored(pool, row, ctx: int, window: int, anchors: int) -> int:
    """Release the blocks wholly before the window, except those that hold a position below anchors."""
    kept = {}
    if window > 0:
        for lb in range(min(len(row), -(-anchors // BLOCK_SIZE))):
            kept[lb] = int(row[lb])
            row[lb] = -1
        freed = pool.slide_window(row, ctx, window)
        for lb, b in kept.items():
            row[lb] = b
        return freed
    return 0


def decode_weights(q, K, V, scale, lo=0):
    """Decode attention over positions lo .. ctx - 1 and each position's weight per KV head, the sum of
    the softmax weights of its G query heads: (out [H_q][d], magnitude [H_q][d], weights [H_kv][ctx])."""
    q = np.asarray(q, dtype=np.float64)
    ctx, H_kv, _ = K.shape
    H_q, d = q.shape
    G = H_q // H_kv
    out, mag, w = np.zeros((H_q, d)), np.zeros((H_q, d)), np.zeros((H_kv, ctx))
    if ctx > lo:
        for h in range(H_q):
            p = softmax_weights(scale * (K[lo:, h // G] @ q[h]))
            out[h], mag[h] = p @ V[lo:, h // G], p @ np.abs(V[lo:, h // G])
            w[h // G, lo:] += p
    return out, mag, w


def evict_order(scores, positions, anchors: int, recent: int) -> np.ndarray:
    """Slots of one (sequence, KV head) from the one kept first to the one evicted first: the protected
    ones (position below anchors, or among the last `recent` positions), then by score, NaN last; equal
    ones by slot."""
    scores, positions = np.asarray(scores, dtype=np.float64), np.asarray(positions, dtype=np.int64)
    newest = positions.max() if len(positions) else -1
    key = []
    for j in range(len(scores)):
        safe = positions[j] < anchors or positions[j] > newest - recent
        nan = np.isnan(scores[j])
        key.append((0 if safe else 1, 1 if nan and not safe else 0, 0.0 if nan or safe else -scores[j], j))
    return np.array([k[-1] for k in sorted(key)], dtype=np.int64)


def evict_plan(scores, positions, budget: int, anchors: int, recent: int):
    """(holes, movers) of one (sequence, KV head): the i-th evicted slot below the new length, and the
    i-th kept slot at or past it, which moves there."""
    n = len(scores)
    left = min(n, budget)
    keep = set(evict_order(scores, positions, anchors, recent)[:left].tolist())
    holes = [j for j in range(left) if j not in keep]
    movers = [j for j in range(left, n) if j in keep]
    assert len(holes) == len(movers)
    return holes, movers


def evict_rows(cache, table_row, head: int, holes, movers):
    """Move K and V rows (codes, parameters, scales) of one head of a PagedKVCache."""
    for dst, src in zip(holes, movers):
        d, s = locate(table_row, dst), locate(table_row, src)
        for a in (cache.k, cache.v, cache.k_params, cache.v_params, cache.k_tscale):
            if a is not None:
                a[d, head] = a[s, head]
