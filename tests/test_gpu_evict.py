"""Eviction by accumulated weight on the GPU against the oracle, bit for bit, and the loop that uses it."""

import numpy as np
import pytest
import torch

import oracle as O
from paged_kv_cache_table_gb300 import native as N
from paged_kv_cache_table_gb300.workloads import bf16_bits

from bounded import (KINDS, assert_within, decode_weights, evict, gpu, oracle_evict, states, tolerance, weight_tolerance,
                     workload)
from harness import assert_pools_equal, to_f64

pytestmark = pytest.mark.gpu


def _scores(rng, shape, mode):
    if mode == "ties":  # few distinct values
        return rng.integers(0, 3, shape).astype(np.float32)
    if mode == "equal":
        return np.zeros(shape, np.float32)
    if mode == "special":
        x = rng.standard_normal(shape).astype(np.float32)
        x[rng.random(shape) < 0.2] = np.nan
        x[rng.random(shape) < 0.1] = np.inf
        x[rng.random(shape) < 0.1] = -np.inf
        x[rng.random(shape) < 0.1] = -0.0
        x[rng.random(shape) < 0.1] = 0.0
        return x
    if mode == "close":  # neighbours in the last bits
        return (1.0 + rng.integers(0, 40, shape) * 2.0 ** -23).astype(np.float32)
    return np.exp(2 * rng.standard_normal(shape)).astype(np.float32)


def _positions(rng, B, H, ctx, stride, anchors):
    """Slots in no order of position, as earlier evictions leave them."""
    pos = np.full((B, H, stride), -9, np.int32)
    for s in range(B):
        n = int(ctx[s])
        for h in range(H):
            p = rng.choice(3 * n + 1, n, replace=False)
            front = min(anchors, n)
            p[:front] = np.arange(front)
            p[front:] = anchors + rng.choice(3 * n + 1, n - front, replace=False)
            pos[s, h, :n] = p
    return pos


def _check(w, ctx, budget, anchors, recent, mode="spread", given=False, in_place=False, extra=5, seed=0):
    g, o = states(w)
    rng = np.random.default_rng(seed)
    stride = int(max(ctx)) + extra
    sc = _scores(rng, (w.B, w.H_kv, stride), mode)
    pos = _positions(rng, w.B, w.H_kv, ctx, stride, anchors) if given else None
    si = torch.from_numpy(sc).cuda()
    pi = torch.from_numpy(pos).cuda() if given else None
    so = si if in_place else torch.full_like(si, -5.0)
    po = pi if in_place and given else torch.full(si.shape, -5, dtype=torch.int32, device="cuda")
    evict(g, ctx, si, so, pi, po, budget, anchors, recent)
    assert g.err_bits() == 0
    es, ep = oracle_evict(o, ctx, sc, pos, stride, budget, anchors, recent)
    assert np.array_equal(so.cpu().numpy(), es, equal_nan=True)
    assert np.array_equal(po.cpu().numpy(), ep)
    if not in_place:
        assert np.array_equal(si.cpu().numpy(), sc, equal_nan=True)
    assert_pools_equal(g, o)
    return g, o


CTX = [0, 1, 30, 133, 400]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("mode", ["spread", "ties", "equal", "special", "close"])
@pytest.mark.parametrize("budget,anchors,recent", [(1, 0, 0), (1, 0, 1), (30, 4, 8), (31, 4, 27), (100, 0, 0), (100, 100, 0),
                                                   (399, 4, 60), (400, 4, 60)])
def test_selection(budget, anchors, recent, mode, given):
    w = workload("bf16", H_q=3, H_kv=3, D=64, ctx_list=CTX)
    _check(w, CTX, budget, anchors, recent, mode, given)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("sinks", [0, 4])
def test_cache_kinds(kind, sinks):
    for in_place in (False, True):
        _check(workload(kind, sinks=sinks, ctx_list=CTX), CTX, 60, 4, 20, given=True, in_place=in_place, seed=3)


@pytest.mark.parametrize("H,D", [(1, 64), (8, 128), (16, 64)])
def test_head_layouts(H, D):
    _check(workload("bf16", B=2, H_q=H, H_kv=H, D=D, ctx_list=[90, 301]), [90, 301], 64, 1, 16)


@pytest.mark.parametrize("n", [4096, 4097, 9000, 20000, 40000, 70000])
def test_clusters(n):
    # few and many slots for one CTA, then four and eight CTAs per (sequence, head)
    w = workload("bf16", B=2, H_q=1, H_kv=1, D=64, ctx_list=[n, 37])
    for mode in ("spread", "equal"):
        _check(w, [n, 37], n // 4, 4, n // 16, mode, in_place=mode == "equal")
    _check(w, [n, 37], n - 1, 0, 1, "ties", given=True)


@pytest.mark.parametrize("B", [2, 10])  # 32 pairs, and 160, more than the GPU has SMs
@pytest.mark.parametrize("n", [2048, 2049, 4096, 4101, 12345])
def test_threads_of_a_cta(n, B):
    ctx = [n] + [0, 1, 37, 100, 64, 65, 300, 2, 33][:B - 1]
    w = workload("bf16", B=B, H_q=16, H_kv=16, D=64, ctx_list=ctx)
    for mode in ("special", "close"):
        for budget, anchors, recent in ((n - 1, 4, 16), (n // 2, 0, 0), (33, 4, 1)):
            _check(w, ctx, budget, anchors, recent, mode, given=mode == "close", in_place=mode == "special")


@pytest.mark.parametrize("n,budget", [(500_001, 70_000), (1 << 21, 1 << 20)])
def test_more_slots_than_shared_memory_holds(n, budget):
    # eight CTAs with 40960 keys each hold 327,680 slots; the rest are ranked from memory
    anchors, recent = 4, 1000
    blocks = -(-n // 16)
    k = torch.randint(-30000, 30000, (blocks * 16, 1, 64), dtype=torch.int16, device="cuda")
    v = torch.randint(-30000, 30000, (blocks * 16, 1, 64), dtype=torch.int16, device="cuda")
    rng = np.random.default_rng(2)
    table = rng.permutation(blocks).astype(np.int32)
    desc = N.make_desc(1, 1, 1, 64, blocks, blocks)
    for given in (False, True):
        sc = rng.integers(0, 5000, n).astype(np.float32)
        pos = rng.permutation(2 * n)[:n].astype(np.int32) if given else np.arange(n, dtype=np.int32)
        order = np.lexsort((np.arange(n), -sc, ~((pos < anchors) | (pos > pos.max() - recent))))[:budget]
        keep = np.zeros(n, dtype=bool)
        keep[order] = True
        holes, movers = np.nonzero(~keep[:budget])[0], budget + np.nonzero(keep[budget:])[0]
        si = torch.from_numpy(sc).cuda()[None, None].contiguous()
        pi = torch.from_numpy(pos).cuda()[None, None].contiguous()
        k0, v0 = k.clone(), v.clone()
        ws = torch.empty(N.pa_cache_evict_workspace_size(desc, n, budget), dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        N.pa_cache_evict(desc, k, v, gpu(table), gpu([n]), n, si, si, pi if given else None, pi, n, budget, anchors,
                         recent, ws, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        place = np.arange(budget)
        place[holes] = movers
        assert np.array_equal(si.cpu().numpy()[0, 0, :budget], sc[place])
        assert np.all(si.cpu().numpy()[0, 0, budget:] == 0)
        assert np.array_equal(pi.cpu().numpy()[0, 0, :budget], pos[place])
        assert np.array_equal(pi.cpu().numpy()[0, 0, budget:], pos.max() + 1 + np.arange(n - budget))
        src = gpu(table[movers // 16].astype(np.int64) * 16 + movers % 16, torch.int64)
        dst = gpu(table[holes // 16].astype(np.int64) * 16 + holes % 16, torch.int64)
        k0[dst], v0[dst] = k0[src], v0[src]
        assert torch.equal(k, k0) and torch.equal(v, v0)


def test_repeated_positions_stay_in_bounds():
    # more protected slots than the budget, which positions given by mistake can make: budget slots stay
    w = workload("bf16", B=1, ctx_list=[200])
    g, _ = states(w)
    si = torch.rand(1, w.H_kv, 200, device="cuda")
    pi = torch.zeros(1, w.H_kv, 200, dtype=torch.int32, device="cuda")
    so, po = torch.empty_like(si), torch.empty_like(pi)
    evict(g, [200], si, so, pi, po, 50, 4, 40)
    assert g.err_bits() == 0
    assert torch.equal(so[..., :50], si[..., :50])  # all protected, all equal: the first 50 slots


def test_bad_tables_and_lengths():
    w = workload("bf16", B=5, H_q=2, H_kv=2, D=64, ctx_list=[100] * 5)
    g, o = states(w)
    g.tables[1, 0] = w.num_blocks  # under holes of sequence 1
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    before_k, before_v = g.k.clone(), g.v.clone()
    rng = np.random.default_rng(5)
    sc = _scores(rng, (5, 2, 112), "spread")
    si, so = torch.from_numpy(sc).cuda(), torch.full((5, 2, 112), -5.0, device="cuda")
    po = torch.full((5, 2, 112), -5, dtype=torch.int32, device="cuda")
    ctx = np.array([100, 100, 101, -1, 100])
    evict(g, ctx, si, so, None, po, 40, 4, 10, max_ctx=100)
    assert g.err_bits() == N.PA_EFLAG_BAD_BLOCK_ID | N.PA_EFLAG_CTX_OVERFLOW
    assert torch.all(so[2:4] == -5) and torch.all(po[2:4] == -5)
    for s in (2, 3):
        idx = torch.from_numpy((w.tables[s][:7, None].astype(np.int64) * 16 + np.arange(16)).reshape(-1)).cuda()
        assert torch.equal(g.k.view(torch.int16)[idx], before_k.view(torch.int16)[idx])
        assert torch.equal(g.v.view(torch.int16)[idx], before_v.view(torch.int16)[idx])
    es, ep = oracle_evict(o, [100, 100, 0, 0, 100], sc, None, 112, 40, 4, 10)
    for s in (0, 1, 4):
        assert np.array_equal(so[s].cpu().numpy(), es[s]) and np.array_equal(po[s].cpu().numpy(), ep[s])


def test_nothing_cached_and_nothing_to_evict():
    w = workload("bf16", B=3, H_q=2, H_kv=2, D=64, ctx_list=[0, 5, 40])
    for lens, max_ctx in (([0, 0, 0], 0), ([0, 5, 40], 40)):
        g, o = states(w)
        before = g.k.clone()
        si = torch.rand(3, 2, 48, device="cuda")
        so, po = torch.full_like(si, -5.0), torch.full((3, 2, 48), -5, dtype=torch.int32, device="cuda")
        evict(g, lens, si, so, None, po, 40, 4, 8, max_ctx=max_ctx)
        assert g.err_bits() == 0
        es, ep = oracle_evict(o, lens, si.cpu().numpy(), None, 48, 40, 4, 8)
        assert np.array_equal(so.cpu().numpy(), es) and np.array_equal(po.cpu().numpy(), ep)
        assert torch.equal(g.k.view(torch.int16), before.view(torch.int16))


def test_two_calls_at_once_with_their_own_workspaces():
    w = workload("bf16", B=2, H_q=2, H_kv=2, D=64, ctx_list=[9000, 5000])
    runs = []
    for seed in (1, 2):
        g, o = states(w)
        rng = np.random.default_rng(seed)
        sc = _scores(rng, (2, 2, 9000), "spread")
        n = N.pa_cache_evict_workspace_size(g.desc, 9000, 1000)
        runs.append(dict(g=g, o=o, sc=sc, si=torch.from_numpy(sc).cuda(), so=torch.zeros(2, 2, 9000, device="cuda"),
                         po=torch.zeros(2, 2, 9000, dtype=torch.int32, device="cuda"), ctx=gpu([9000, 5000]), n=n,
                         ws=torch.empty(n, dtype=torch.uint8, device="cuda"), s=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for r in runs:
            N.pa_cache_evict(r["g"].desc, r["g"].k, r["g"].v, r["g"].tables_dev, r["ctx"], 9000, r["si"], r["so"], None,
                             r["po"], 9000, 1000, 4, 100, r["ws"], r["n"], r["g"].err, r["s"])
    torch.cuda.synchronize()
    for r in runs:
        es, ep = oracle_evict(r["o"], [9000, 5000], r["sc"], None, 9000, 1000, 4, 100)
        assert np.array_equal(r["so"].cpu().numpy(), es) and np.array_equal(r["po"].cpu().numpy(), ep)
        assert_pools_equal(r["g"], r["o"])
        assert r["g"].err_bits() == 0


def test_replayed_from_a_graph_on_another_stream():
    w = workload("bf16", ctx_list=CTX)
    g, o = states(w)
    rng = np.random.default_rng(6)
    sc = _scores(rng, (w.B, w.H_kv, 400), "spread")
    si, so = torch.from_numpy(sc).cuda(), torch.zeros(w.B, w.H_kv, 400, device="cuda")
    po = torch.zeros(w.B, w.H_kv, 400, dtype=torch.int32, device="cuda")
    ctx = gpu([0, 0, 0, 0, 0])
    n = N.pa_cache_evict_workspace_size(g.desc, 400, 60)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call():
        N.pa_cache_evict(g.desc, g.k, g.v, g.tables_dev, ctx, 400, si, so, None, po, 400, 60, 4, 20, ws, n, g.err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    ctx.copy_(gpu(CTX))
    for _ in range(2):  # the same scores again give the same cache
        graph.replay()
        torch.cuda.synchronize()
    es, ep = oracle_evict(o, CTX, sc, None, 400, 60, 4, 20)
    assert np.array_equal(so.cpu().numpy(), es) and np.array_equal(po.cpu().numpy(), ep)
    assert_pools_equal(g, o)
    assert g.err_bits() == 0


@pytest.mark.parametrize("kind,sinks", [("bf16", 0), ("fp8", 4), ("fp8tok", 4), ("int4", 0)])
def test_bounded_decode_loop(kind, sinks):
    """A stream held at a budget: append, attend with weights, evict when full, release the blocks."""
    budget, slack, anchors, recent = 48, 16, 4, 12
    steps = 90
    w = workload(kind, B=3, sinks=sinks, ctx_list=[0, 40, 90], steps=steps)
    g, o = states(w)
    stride = w.max_blocks * 16
    length = w.ctx_old.astype(np.int32).copy()
    scores = torch.zeros(w.B, w.H_kv, stride, device="cuda")
    pos = torch.arange(stride, dtype=torch.int32, device="cuda").expand(w.B, w.H_kv, stride).contiguous()
    want_pos = pos.cpu().numpy().astype(np.int64)
    kmag = 144 * 1.0 if kind == "int4" else None
    for i in range(steps):
        g.prepare(length)
        o.prepare(length)
        g.append(w.k_new[i], w.v_new[i], length)
        o.append(w.k_new[i], w.v_new[i], length)
        length = length + 1
        base = scores.cpu().numpy().astype(np.float64)
        out = to_f64(decode_weights(g, w.q[i], length, scores, scores))
        got = scores.cpu().numpy().astype(np.float64)
        qv = O.bf16_bits_to_f64(bf16_bits(w.q[i]))
        for s in range(w.B):
            n = int(length[s])
            K, V = O.gather_positions(o.cache, s, o.tables[s], np.arange(n))
            ref, mag, wt = O.decode_weights(qv[s], K, V, w.scale)
            assert_within(out[s], ref, tolerance(ref, mag), f"{kind} step {i} sequence {s}")
            assert_within(got[s, :, :n], base[s, :, :n] + wt,
                          weight_tolerance(wt, base[s, :, :n], qv[s], K, w.scale, kmag), f"{kind} step {i} weights {s}")
            assert np.all(got[s, :, n:] == 0)
        if length.max() >= budget + slack:
            want_s, want_pos = oracle_evict(o, length, scores.cpu().numpy(), want_pos, stride, budget, anchors, recent)
            evict(g, length, scores, scores, pos, pos, budget, anchors, recent)
            assert np.array_equal(scores.cpu().numpy(), want_s)
            assert np.array_equal(pos.cpu().numpy(), want_pos)
            length = np.minimum(length, budget).astype(np.int32)
            first = -(-budget // 16)
            for s in range(w.B):
                g.bm.release(g.tables[s, first:], w.max_blocks - first)
                o.pool.release(o.tables[s, first:], w.max_blocks - first)
            g.tables_dev.copy_(torch.from_numpy(g.tables))
            # the newest tokens and the first are there, for every head
            seen = i + 1 + w.ctx_old
            for s in range(w.B):
                for h in range(w.H_kv):
                    held = set(want_pos[s, h, :length[s]].tolist())
                    assert set(range(min(anchors, length[s]))) <= held
                    if seen[s] > budget:
                        assert set(range(seen[s] - recent, seen[s])) <= held
        assert g.bm.num_free() == o.pool.num_free()
    assert g.err_bits() == 0
    assert_pools_equal(g, o)
