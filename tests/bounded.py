"""Helpers of the tests of the bounded-cache operators: tolerances and seeded cache states.

A state is the harness's workload (the same tokens in the GPU's cache and in the oracle's).  The slots
that the operator under test must not read are poisoned: their table entries are -1, or, where the block
is held for other positions, bf16 slots hold NaN.
"""

import numpy as np
import torch

import oracle as O
from paged_kv_cache_table_gb300 import native as N
from paged_kv_cache_table_gb300.workloads import make_workload

from harness import BF16_NAN, GpuState, OracleState

KINDS = {
    "bf16": dict(),
    "fp8": dict(quant=True),
    "fp8tok": dict(quant=True, kv="e4m3_tok"),
    "int4": dict(kv="int4"),
}


def tolerance(ref, mag, extra=0.0):
    """How far an attention output may be from the fp64 reference.

    The output is rounded to bf16 (2^-8 of its value).  The probabilities are rounded to bf16 (or fp16,
    finer) before P V, at most 2^-8 of each, so at most 2^-8 of the average of |V| (`mag`).  fp32 sums,
    exponentials and the offsets of 4-bit codes add less than 2^-10 of it.  fp16 probabilities below the
    normal range lose at most 2^-25 each against a sum of at least 1, under 1e-4 in all for the lengths
    and values tested.  `extra`: what rounding K and V themselves adds, as a share of mag."""
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10 + extra) * mag + 1e-4


def decoded_extra(q, K, scale):
    """`extra` of the calls that round K and V to bf16: V by 2^-8; K by 2^-8 of each element, so a score
    moves by at most d = 2^-8 scale max sum |q k|, a weight by a factor within e^(+-2 d)."""
    G = q.shape[1] // K.shape[1]
    d = 2.0 ** -8 * scale * max((np.abs(K[:, h // G]) @ np.abs(q[:, h]).T).max() for h in range(q.shape[1]))
    return 2.0 ** -8 + np.expm1(2 * d)


def assert_within(got, ref, tol, what):
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    over = np.abs(got - ref) - tol
    assert over.max(initial=-1.0) <= 0, f"{what}: {np.abs(got - ref).max():.3e} off, {over.max():.3e} over the bound"


def workload(kind, steps=1, sinks=0, **kw):
    base = dict(B=5, H_q=8, H_kv=4, D=128, steps=steps, num_sink=sinks)
    base.update(KINDS[kind])
    base.update(kw)
    return make_workload("8b", **base)


def states(w, window=0):
    g, o = GpuState(w), OracleState(w)
    g.desc.sliding_window = window
    return g, o


def poison(g, seq, positions):
    """NaN in the bf16 slots of the given positions of a sequence (nothing else may be read there)."""
    if g.w.k_dtype != "bf16":
        return
    slots = [int(g.tables[seq, p // 16]) * 16 + p % 16 for p in positions if g.tables[seq, p // 16] >= 0]
    if slots:
        idx = torch.tensor(slots, device=g.dev)
        for pool in (g.k, g.v):
            pool.view(torch.int16)[idx] = BF16_NAN


def gpu(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype)


def release(g, o, ctx, window, anchors):
    """The anchored release on both sides, the host's tables copied to the device."""
    _, freed = g.bm.slide_window(g.tables, np.asarray(ctx, dtype=np.int32), window, anchors)
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    assert freed == sum(O.slide_window_anchored(o.pool, o.tables[s], int(c), window, anchors) for s, c in enumerate(ctx))
    assert np.array_equal(g.tables, o.tables)


def decode_anchored(g, q, ctx, anchors, partition=0, ws_fill=0xFF, max_ctx=None):
    w = g.w
    max_ctx = int(max(ctx)) if max_ctx is None else max_ctx
    out = torch.full((w.B, w.H_q, w.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = N.pa_decode_anchored_workspace_size(g.desc, max_ctx, partition, anchors)
    assert n > 0
    ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda")
    N.pa_decode_attention_anchored(g.desc, out, q.cuda(), g.k, g.v, g.tables_dev, gpu(ctx), max_ctx, w.scale, partition,
                                   anchors, ws, n, g.err)
    return out


def decode_weights(g, q, ctx, scores_in, scores_out, partition=0, ws_fill=0xFF, max_ctx=None):
    """pa_decode_attention_weights; scores as fp32 device tensors [B][H_kv][stride] (scores_in may be None)."""
    w = g.w
    max_ctx = int(max(ctx)) if max_ctx is None else max_ctx
    out = torch.full((w.B, w.H_q, w.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = N.pa_decode_weights_workspace_size(g.desc, max_ctx, partition)
    assert n > 0
    ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda")
    N.pa_decode_attention_weights(g.desc, out, q.cuda(), g.k, g.v, g.tables_dev, gpu(ctx), max_ctx, w.scale, partition,
                                  scores_in, scores_out, scores_out.shape[2], ws, n, g.err)
    return out


def weight_tolerance(weights, base, q, K, scale, kmag=None):
    """How far accumulated fp32 weights may be off.  A score is a sum of D exact products in fp32, off by
    at most D 2^-23 of the sum of |q k|, and is scaled and rounded (2^-22 of it); a weight is off by twice
    that (its own score and the sum's) and by the exponentials', the sum's and the division's roundings,
    under 2^-19.  kmag: the largest |code| that 4-bit keys enter the products with, in place of |K|.
    The running score is rounded once or twice more."""
    G = q.shape[0] // K.shape[1]
    tol = np.zeros_like(weights)
    for h in range(K.shape[1]):
        a = np.abs(q[h * G:(h + 1) * G])
        mag = scale * (np.abs(K[:, h]) @ a.T if kmag is None else np.full((len(K), G), kmag) * a.sum(1))
        d = mag.max(initial=0.0) * (K.shape[2] + 4) * 2.0 ** -23
        tol[h] = weights[h] * (2 * d + 2.0 ** -19) + 2.0 ** -22 * np.abs(base[h] + weights[h]) + 1e-30
    return tol


def evict(g, ctx, scores_in, scores_out, pos_in, pos_out, budget, anchors, recent, max_ctx=None, ws_fill=0xFF):
    max_ctx = int(max(ctx)) if max_ctx is None else max_ctx
    n = N.pa_cache_evict_workspace_size(g.desc, max_ctx, budget)
    assert n > 0
    ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda")
    N.pa_cache_evict(g.desc, g.k, g.v, g.tables_dev, gpu(ctx), max_ctx, scores_in, scores_out, pos_in, pos_out,
                     scores_in.shape[2], budget, anchors, recent, ws, n, g.err)


def oracle_evict(o, ctx, scores, pos, stride, budget, anchors, recent):
    """The same on the oracle's cache; scores and pos [B][H_kv][stride] (pos may be None).  Returns the
    expected (scores_out, pos_out)."""
    B, H = scores.shape[:2]
    so, po = np.zeros((B, H, stride), np.float32), np.zeros((B, H, stride), np.int64)
    for s in range(B):
        n = int(ctx[s])
        left = min(n, budget)
        for h in range(H):
            sc = scores[s, h, :n]
            ps = np.arange(n) if pos is None else pos[s, h, :n].astype(np.int64)
            holes, movers = O.evict_plan(sc, ps, budget, anchors, recent)
            O.evict_rows(o.cache, o.tables[s], h, holes, movers)
            place = np.arange(left)
            place[holes] = movers
            so[s, h, :left], po[s, h, :left] = sc[place], ps[place]
            po[s, h, left:] = (ps.max() if n else -1) + 1 + np.arange(stride - left)
    return so, po
