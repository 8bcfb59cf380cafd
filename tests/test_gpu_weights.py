"""Decode attention with accumulated attention weights on the GPU against the oracle."""

import numpy as np
import pytest
import torch

import oracle as O
from paged_kv_cache_table_gb300 import native as N
from paged_kv_cache_table_gb300.workloads import bf16_bits

from bounded import KINDS, assert_within, decode_weights, gpu, poison, states, tolerance, weight_tolerance, workload
from harness import to_f64

pytestmark = pytest.mark.gpu


def _check(g, o, q, ctx, window, got, base, scores, what, seqs=None):
    w = g.w
    qv = O.bf16_bits_to_f64(bf16_bits(q))
    out, got_s = to_f64(got), scores.cpu().numpy().astype(np.float64)
    for s in range(w.B) if seqs is None else seqs:
        c = int(ctx[s])
        lo = O.window_start(c, window)
        K, V = O.gather_positions(o.cache, s, o.tables[s], np.arange(lo, c))
        ref, mag, wt = O.decode_weights(qv[s], K, V, w.scale)
        assert_within(out[s], ref, tolerance(ref, mag), f"{what}: output of sequence {s}")
        kmag = None
        if w.k_dtype == "int4":  # codes enter as 128 + n < 144, times the group's scale
            kmag = 144 * float(O.bf16_bits_to_f64((o.cache.k_params & 0xFFFF).astype(np.uint16)[
                o.cache.k_params != 0xFFFFFFFF]).max())
        full = np.zeros((w.H_kv, c))
        full[:, lo:] = wt
        tol = np.zeros((w.H_kv, c))
        if c > lo:
            tol[:, lo:] = weight_tolerance(wt, base[s][:, lo:c], qv[s], K, w.scale, kmag)
        assert_within(got_s[s, :, :c], base[s][:, :c] + full, tol, f"{what}: weights of sequence {s}")
        assert np.array_equal(got_s[s, :, c:], np.full_like(got_s[s, :, c:], -5.0)), "entries past the context written"


def _run(w, window=0, partition=0, steps=None):
    g, o = states(w, window)
    stride = w.max_blocks * 16 + 3
    rng = np.random.default_rng(1)
    scores = torch.zeros(w.B, w.H_kv, stride, device="cuda")
    for i in range(w.steps):
        pos, ctx = w.positions(i), w.context_lens(i)
        g.prepare(pos)
        o.prepare(pos)
        g.append(w.k_new[i], w.v_new[i], pos)
        o.append(w.k_new[i], w.v_new[i], pos)
        for s, c in enumerate(ctx):
            poison(g, s, range(w.num_sink, max(0, int(c) - window)) if window else [])
        base = rng.random((w.B, w.H_kv, stride)).astype(np.float32)
        scores = torch.full((w.B, w.H_kv, stride), -5.0, device="cuda")
        out = decode_weights(g, w.q[i], ctx, torch.from_numpy(base).cuda(), scores, partition)
        _check(g, o, w.q[i], ctx, window, out, base.astype(np.float64), scores, f"{w.k_dtype} P {partition} step {i}")
    assert g.err_bits() == 0
    return g, o


@pytest.mark.parametrize("partition", [0, 16, 48, 1 << 20])
def test_partitions(partition):
    _run(workload("bf16", steps=3, ctx_list=[0, 1, 30, 133, 400]), partition=partition)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("sinks", [0, 4, 20])
def test_cache_kinds_and_sinks(kind, sinks):
    _run(workload(kind, steps=2, sinks=sinks, ctx_list=[2, 19, 47, 150, 333]))


@pytest.mark.parametrize("H_q,H_kv,D", [(5, 1, 64), (16, 2, 64), (1, 1, 64), (12, 4, 128), (8, 8, 128), (64, 8, 128),
                                        (32, 16, 64), (12, 2, 128), (14, 2, 64)])
def test_head_layouts(H_q, H_kv, D):
    w = workload("bf16", H_q=H_q, H_kv=H_kv, D=D, ctx_list=[3, 40, 77, 150, 260])
    _run(w)
    _run(w, partition=32)


def test_many_kv_heads_take_the_wide_blocks():
    _run(workload("fp8", H_q=32, H_kv=16, B=2, ctx_list=[77, 260]))


@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("window", [1, 17, 1000])
def test_window(window, sinks):
    _run(workload("fp8", sinks=sinks, steps=2, ctx_list=[0, 3, 30, 133, 400]), window=window)
    _run(workload("bf16", sinks=sinks, steps=2, ctx_list=[0, 3, 30, 133, 400]), window=window, partition=32)


def test_many_sequences_and_one_long_one():
    _run(workload("bf16", B=40, ctx_range=(1, 60)))
    _run(workload("bf16", B=2, ctx_list=[3000, 5]))


def test_more_sequences_than_the_balanced_split_takes():
    # over 2048 sequences: fixed partitions, one merge of many short rows
    w = workload("bf16", B=2100, H_q=2, H_kv=1, D=64, ctx_range=(1, 20))
    g, o = states(w)
    scores = torch.full((w.B, 1, 32), -5.0, device="cuda")
    out = decode_weights(g, w.q[0], w.ctx_old, None, scores)
    _check(g, o, w.q[0], w.ctx_old, 0, out, np.zeros((w.B, 1, 32)), scores, "2100 sequences", seqs=range(0, w.B, 17))
    assert g.err_bits() == 0


def test_nothing_cached():
    w = workload("bf16", B=3, ctx_list=[5, 17, 40])
    g, _ = states(w)
    scores = torch.full((3, w.H_kv, 8), -5.0, device="cuda")
    out = decode_weights(g, w.q[0], [0, 0, 0], None, scores, max_ctx=0)
    assert g.err_bits() == 0
    assert torch.all(out == 0) and torch.all(scores == -5.0)


def test_two_calls_at_once_with_their_own_workspaces():
    w = workload("fp8", sinks=4, ctx_list=[500, 40, 900, 150, 2600])
    g, o = states(w)
    n = N.pa_decode_weights_workspace_size(g.desc, 2600, 0)
    ctx, q = gpu(w.ctx_old), w.q[0].cuda()
    runs = [dict(out=torch.zeros((w.B, w.H_q, w.D), dtype=torch.bfloat16, device="cuda"),
                 sc=torch.full((w.B, w.H_kv, 2600), -5.0, device="cuda"),
                 ws=torch.empty(n, dtype=torch.uint8, device="cuda"), s=torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for r in runs:
            N.pa_decode_attention_weights(g.desc, r["out"], q, g.k, g.v, g.tables_dev, ctx, 2600, w.scale, 0, None, r["sc"],
                                          2600, r["ws"], n, g.err, r["s"])
    torch.cuda.synchronize()
    for r in runs:
        _check(g, o, w.q[0], w.ctx_old, 0, r["out"], np.zeros((w.B, w.H_kv, 2600)), r["sc"], "one of two")
    assert g.err_bits() == 0


def test_accumulation_in_place_and_from_nothing():
    w = workload("bf16", ctx_list=[4, 40, 90, 150, 260])
    g, o = states(w)
    ctx = w.ctx_old
    one = torch.full((w.B, w.H_kv, 300), -5.0, device="cuda")
    a = decode_weights(g, w.q[0], ctx, None, one)
    _check(g, o, w.q[0], ctx, 0, a, np.zeros((w.B, w.H_kv, 300)), one, "from nothing")
    twice = one.clone()
    b = decode_weights(g, w.q[0], ctx, twice, twice)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for s, c in enumerate(ctx):
        assert torch.equal(twice[s, :, :c], one[s, :, :c] * 2), "a second pass adds the same weights"
        assert torch.all(twice[s, :, c:] == -5.0)
    # the same bits whatever the workspace held, and the same output as the plain call within its bound
    again = torch.full_like(one, -5.0)
    decode_weights(g, w.q[0], ctx, None, again, ws_fill=0)
    assert torch.equal(again, one)


def test_bad_tables_and_lengths_leave_their_rows():
    w = workload("bf16", ctx_list=[100, 100, 100, 100, 0])
    g, o = states(w)
    g.tables[1, 3] = w.num_blocks
    g.tables[2, 6] = -1
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    ctx = w.ctx_old.copy()
    ctx[3] = 101
    base = torch.rand(w.B, w.H_kv, 128, device="cuda")
    for partition in (0, 16):
        scores = torch.full((w.B, w.H_kv, 128), -5.0, device="cuda")
        g.err.zero_()
        out = decode_weights(g, w.q[0], ctx, base, scores, partition, max_ctx=100)
        assert g.err_bits() == N.PA_EFLAG_BAD_BLOCK_ID | N.PA_EFLAG_CTX_OVERFLOW
        assert torch.all(out[1:] == 0) and torch.all(scores[1:] == -5.0)
        _check(g, o, w.q[0], ctx, 0, out, base.cpu().numpy().astype(np.float64), scores, "the good row", seqs=[0])


def test_replayed_from_a_graph_on_another_stream():
    w = workload("bf16", ctx_list=[5, 40, 90, 150, 300])
    g, o = states(w)
    ctx, q = gpu(w.ctx_old), w.q[0].cuda()
    out = torch.zeros((w.B, w.H_q, w.D), dtype=torch.bfloat16, device="cuda")
    scores = torch.full((w.B, w.H_kv, 320), -5.0, device="cuda")
    n = N.pa_decode_weights_workspace_size(g.desc, 300, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call():
        N.pa_decode_attention_weights(g.desc, out, q, g.k, g.v, g.tables_dev, ctx, 300, w.scale, 0, None, scores, 320, ws,
                                      n, g.err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for lens in ([5, 40, 90, 150, 300], [1, 0, 60, 20, 299]):
        ctx.copy_(gpu(lens))
        scores.fill_(-5.0)
        graph.replay()
        torch.cuda.synchronize()
        _check(g, o, w.q[0], lens, 0, out, np.zeros((w.B, w.H_kv, 320)), scores, f"replay at {lens}",
               seqs=[s for s in range(w.B) if lens[s]])
    assert g.err_bits() == 0
