"""Decode and prefill attention over a sliding window and the first tokens, on the GPU against the oracle."""

import numpy as np
import pytest
import torch

import oracle as O
from paged_kv_cache_table_gb300 import native as N
from paged_kv_cache_table_gb300.workloads import bf16_bits

from bounded import (assert_within, decode_anchored, decoded_extra, gpu, poison, release, states, tolerance, workload)
from harness import to_f64

pytestmark = pytest.mark.gpu


def _anchors_in_blocks(w, anchors):
    return anchors if anchors > w.num_sink else 0


def _poison_hole(g, ctx, window, anchors):
    """Positions between the anchors and the window of every sequence."""
    for s, c in enumerate(ctx):
        poison(g, s, range(max(anchors, g.w.num_sink), max(0, int(c) - window)))


def _ref_decode(o, w, q, ctx, window, anchors):
    qv = O.bf16_bits_to_f64(bf16_bits(q))
    ref, tol = np.zeros((w.B, w.H_q, w.D)), np.zeros((w.B, w.H_q, w.D))
    for s in range(w.B):
        c = int(ctx[s])
        if c == 0:
            continue
        see = np.nonzero(O.anchored_mask(c, 1, window, anchors)[0])[0]
        K, V = O.gather_positions(o.cache, s, o.tables[s], see)
        r, m = O.masked_attention(qv[s:s + 1], K, V, w.scale, np.ones((1, len(see)), dtype=bool))
        ref[s], tol[s] = r[0], tolerance(r[0], m[0])
    return ref, tol


def _decode_loop(w, window, anchors, partition):
    g, o = states(w, window)
    keep = _anchors_in_blocks(w, anchors)
    release(g, o, w.ctx_old, window, keep)
    for i in range(w.steps):
        pos, ctx = w.positions(i), w.context_lens(i)
        g.prepare(pos)
        o.prepare(pos)
        g.append(w.k_new[i], w.v_new[i], pos)
        o.append(w.k_new[i], w.v_new[i], pos)
        _poison_hole(g, ctx, window, anchors)
        out = to_f64(decode_anchored(g, w.q[i], ctx, anchors, partition))
        ref, tol = _ref_decode(o, w, w.q[i], ctx, window, anchors)
        assert_within(out, ref, tol, f"{w.k_dtype} W {window} A {anchors} P {partition} step {i}")
        release(g, o, ctx, window, keep)
        assert g.bm.num_free() == o.pool.num_free()
    assert g.err_bits() == 0


@pytest.mark.parametrize("partition", [0, 16, 48])
@pytest.mark.parametrize("window,anchors", [(1, 1), (16, 4), (40, 16), (40, 17), (37, 100), (100, 1000)])
def test_decode_loop(window, anchors, partition):
    _decode_loop(workload("bf16", steps=4, ctx_list=[0, 1, 30, 133, 400]), window, anchors, partition)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8tok", "int4"])
@pytest.mark.parametrize("sinks,anchors", [(0, 4), (4, 4), (4, 2), (4, 21), (20, 20), (20, 40), (4, 0)])
def test_decode_cache_kinds_and_sinks(kind, sinks, anchors):
    _decode_loop(workload(kind, steps=2, sinks=sinks, ctx_list=[2, 19, 47, 150, 333]), 45, anchors, 0)


@pytest.mark.parametrize("H_q,H_kv,D", [(5, 1, 64), (16, 2, 64), (12, 4, 128), (8, 8, 128), (64, 8, 128)])
def test_decode_head_layouts(H_q, H_kv, D):
    w = workload("bf16", H_q=H_q, H_kv=H_kv, D=D, ctx_list=[3, 40, 77, 150, 260])
    _decode_loop(w, 33, 5, 0)
    _decode_loop(w, 33, 5, 32)


def test_decode_anchor_and_window_in_one_block():
    # the window opens inside the block that ends the anchors: listed twice, nothing counted twice
    for ctx in range(30, 50):
        w = workload("bf16", B=1, ctx_list=[ctx])
        _decode_loop(w, 20, 6, 0)
        _decode_loop(w, 20, 6, 16)


@pytest.mark.parametrize("sinks,anchors", [(4, 4), (20, 20), (33, 20), (20, 21)])
def test_decode_window_reaching_the_sinks(sinks, anchors):
    # the window opens before, at and past the anchors and sinks; blocks of sinks alone are released
    w = workload("fp8", sinks=sinks, B=8, steps=6, ctx_list=[44, 48, 52, 59, 61, 64, 76, 92])
    _decode_loop(w, 45, anchors, 0)
    _decode_loop(w, 45, anchors, 32)


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_decode_sink_buffers_of_any_alignment(offset):
    w = workload("fp8", sinks=5, ctx_list=[2, 19, 47, 150, 333])
    g, o = states(w, 45)
    ctx = w.ctx_old
    want = decode_anchored(g, w.q[0], ctx, 5)
    for name in ("k_sink", "v_sink"):
        old = getattr(g, name)
        flat = torch.empty(old.numel() + 8, dtype=old.dtype, device="cuda")[offset:offset + old.numel()]
        flat.copy_(old.view(-1))
        setattr(g, name, flat)
        setattr(g.desc, name, flat.data_ptr())
    assert torch.equal(decode_anchored(g, w.q[0], ctx, 5).view(torch.int16), want.view(torch.int16))
    assert g.err_bits() == 0


def test_decode_without_anchors_is_the_window_bit_for_bit():
    w = workload("bf16", ctx_list=[0, 30, 80, 150, 333])
    g, _ = states(w, 45)
    ctx = w.ctx_old
    a = decode_anchored(g, w.q[0], ctx, 0)
    b = g.attend(w.q[0], ctx)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    g.desc.sliding_window = 0
    a = decode_anchored(g, w.q[0], ctx, 7)
    b = g.attend(w.q[0], ctx)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_decode_bad_tables_and_lengths_zero_their_rows_only():
    w = workload("bf16", ctx_list=[100, 100, 100, 100, 100])
    g, o = states(w, 20)
    g.tables[1, 0] = w.num_blocks       # the anchors' block
    g.tables[2, 6] = -1                 # the window's last block
    g.tables[3, 2] = -7                 # between the two: not read
    o.tables[3, 2] = -7
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    ctx = w.ctx_old.copy()
    ctx[4] = 101
    out = to_f64(decode_anchored(g, w.q[0], ctx, 4, max_ctx=100))
    assert g.err_bits() == N.PA_EFLAG_BAD_BLOCK_ID | N.PA_EFLAG_CTX_OVERFLOW
    assert np.all(out[[1, 2, 4]] == 0)
    ref, tol = _ref_decode(o, w, w.q[0], [100, 0, 0, 100, 0], 20, 4)
    assert_within(out[[0, 3]], ref[[0, 3]], tol[[0, 3]], "the other rows")


def test_decode_replayed_from_a_graph_on_another_stream():
    w = workload("bf16", ctx_list=[5, 40, 90, 150, 300])
    g, o = states(w, 40)
    ctx = gpu(w.ctx_old)
    q = w.q[0].cuda()
    out = torch.zeros((w.B, w.H_q, w.D), dtype=torch.bfloat16, device="cuda")
    n = N.pa_decode_anchored_workspace_size(g.desc, 300, 0, 4)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call():
        N.pa_decode_attention_anchored(g.desc, out, q, g.k, g.v, g.tables_dev, ctx, 300, w.scale, 0, 4, ws, n, g.err)

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
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = _ref_decode(o, w, w.q[0], lens, 40, 4)
        assert_within(to_f64(out), ref, tol, f"replay at {lens}")
    assert g.err_bits() == 0


# ------------------------------------------------------------------------------------------
# Prefill
# ------------------------------------------------------------------------------------------
def prefill(g, q, q_start, ctx, max_q, anchors, max_ctx=None, ws_fill=0xFF):
    w = g.w
    max_ctx = int(max(ctx)) if max_ctx is None else max_ctx
    out = torch.full((max(1, int(q_start[-1])) + 2, w.H_q, w.D), 7.0, dtype=torch.bfloat16, device="cuda")
    n = N.pa_prefill_anchored_workspace_size(g.desc, max_q, max_ctx, anchors)
    ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda") if n else None
    N.pa_prefill_attention_anchored(g.desc, out, q, g.k, g.v, g.tables_dev, gpu(q_start), gpu(ctx), max_q, max_ctx,
                                    w.scale, anchors, ws, n, g.err)
    torch.cuda.synchronize()
    assert torch.all(out[int(q_start[-1]):] == 7.0), "rows behind the last query were written"
    return to_f64(out[:int(q_start[-1])])


def _prefill_case(w, chunk, window, anchors, seed=0, max_q=None):
    g, o = states(w, window)
    ctx = w.ctx_old.astype(np.int64)
    n = np.minimum(chunk, ctx)
    release(g, o, ctx - n + 1, window, _anchors_in_blocks(w, anchors))
    _poison_hole(g, ctx - n + 1, window, anchors)
    q_start = np.concatenate([[0], np.cumsum(n)])
    gen = torch.Generator().manual_seed(seed + 77)
    q = torch.randn(max(1, int(q_start[-1])), w.H_q, w.D, generator=gen).to(torch.bfloat16)
    out = prefill(g, q.cuda(), q_start, ctx, int(n.max()) if max_q is None else max_q, anchors)
    assert g.err_bits() == 0
    decoded = w.k_dtype != "bf16" or w.num_sink > 0
    qv = O.bf16_bits_to_f64(bf16_bits(q))
    for s in range(w.B):
        if n[s] == 0:
            continue
        c, k = int(ctx[s]), int(n[s])
        mask = O.anchored_mask(c, k, window, anchors)
        see = np.nonzero(mask.any(0))[0]
        K, V = O.gather_positions(o.cache, s, o.tables[s], see)
        qs = qv[q_start[s]:q_start[s + 1]]
        ref, mag = O.masked_attention(qs, K, V, w.scale, mask[:, see])
        extra = decoded_extra(qs, K, w.scale) if decoded else 0.0
        assert_within(out[q_start[s]:q_start[s + 1]], ref, tolerance(ref, mag, extra),
                      f"{w.k_dtype} seq {s} ctx {c} chunk {k} W {window} A {anchors}")
    return g, o, q, q_start


@pytest.mark.parametrize("window,anchors", [(1, 1), (16, 4), (50, 16), (50, 17), (37, 100), (300, 3), (130, 130),
                                            (100, 1000)])
@pytest.mark.parametrize("H_q,H_kv,D", [(8, 4, 128), (6, 2, 64)])
def test_prefill(H_q, H_kv, D, window, anchors):
    w = workload("bf16", H_q=H_q, H_kv=H_kv, D=D, ctx_list=[1, 33, 140, 333, 515])
    _prefill_case(w, np.array([1, 33, 5, 200, 129]), window, anchors)


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 8, 128), (16, 2, 128), (12, 4, 128), (5, 1, 64)])
def test_prefill_head_layouts(H_q, H_kv, D):
    w = workload("bf16", H_q=H_q, H_kv=H_kv, D=D, B=3, ctx_list=[70, 400, 290])
    _prefill_case(w, np.array([70, 150, 1]), 60, 20)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8tok", "int4"])
@pytest.mark.parametrize("sinks,anchors", [(0, 4), (4, 4), (4, 2), (4, 21), (20, 40), (17, 0)])
def test_prefill_cache_kinds_and_sinks(kind, sinks, anchors):
    w = workload(kind, sinks=sinks, B=4, ctx_list=[3, 60, 150, 333])
    _prefill_case(w, np.array([3, 20, 1, 70]), 45, anchors)


@pytest.mark.parametrize("sinks,anchors", [(4, 4), (20, 20), (33, 20), (20, 21)])
@pytest.mark.parametrize("H_q,D", [(8, 128), (12, 128), (8, 64)])
def test_prefill_window_reaching_the_sinks(H_q, D, sinks, anchors):
    w = workload("bf16", sinks=sinks, H_q=H_q, D=D, B=8, ctx_list=[44, 48, 52, 60, 64, 66, 80, 96])
    _prefill_case(w, np.array([1, 2, 1, 3, 1, 1, 20, 30]), 45, anchors)


@pytest.mark.parametrize("sinks", [0, 5])
def test_prefill_scales_of_either_sign(sinks):
    # a head's scale that is not positive cannot be applied after a row's maximum: it stays with the values
    w = workload("fp8", sinks=sinks, B=3, ctx_list=[60, 150, 333])
    w.k_scales[1] *= -1
    w.v_scales[2] *= -1
    _prefill_case(w, np.array([20, 1, 70]), 45, 7)


def test_prefill_decoded_cache_of_head_dim_64():
    _prefill_case(workload("bf16", sinks=4, H_q=8, H_kv=2, D=64, B=3, ctx_list=[30, 150, 333]),
                  np.array([30, 20, 70]), 45, 21)


def test_prefill_window_edges_against_the_anchors():
    # windows that open inside, at, and just past the anchors' blocks, tile by tile
    for ctx in (150, 151, 160, 175):
        w = workload("bf16", B=1, ctx_list=[ctx])
        for anchors in (15, 16, 17, 33):
            _prefill_case(w, np.array([140]), 20, anchors)


def test_prefill_long_enough_for_many_tiles():
    w = workload("bf16", B=2, H_q=8, H_kv=1, ctx_list=[1500, 900])
    _prefill_case(w, np.array([300, 257]), 700, 200)


def test_prefill_without_anchors_is_the_window_bit_for_bit():
    for kind in ("bf16", "fp8"):
        w = workload(kind, sinks=0, B=3, ctx_list=[60, 150, 333])
        g, _ = states(w, 45)
        q_start = np.array([0, 20, 21, 91])
        q = torch.randn(91, w.H_q, w.D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
        a = prefill(g, q, q_start, w.ctx_old, 70, 0)
        out = torch.empty(91, w.H_q, w.D, dtype=torch.bfloat16, device="cuda")
        n = N.pa_prefill_workspace_size(g.desc, 333)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        N.pa_prefill_attention_ws(g.desc, out, q, g.k, g.v, g.tables_dev, gpu(q_start), gpu(w.ctx_old), 70, 333, w.scale,
                                  ws, n, g.err)
        assert np.array_equal(a, to_f64(out))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_prefill_bad_tables_and_lengths_zero_their_rows_only(kind):
    w = workload(kind, ctx_list=[100, 100, 100, 100, 100])
    g, _, q, q_start = _prefill_case(w, np.array([5, 5, 5, 5, 5]), 20, 4)
    good = prefill(g, q.cuda(), q_start, w.ctx_old, 5, 4)
    g.tables[1, 0] = w.num_blocks
    g.tables[2, 6] = -1
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    ctx = w.ctx_old.copy()
    ctx[4] = 4  # five queries of a sequence of four
    out = prefill(g, q.cuda(), q_start, ctx, 5, 4, max_ctx=100)
    assert g.err_bits() == N.PA_EFLAG_BAD_BLOCK_ID | N.PA_EFLAG_CTX_OVERFLOW
    assert np.all(out[5:15] == 0) and np.all(out[20:] == 0)
    assert np.array_equal(out[:5], good[:5]) and np.array_equal(out[15:20], good[15:20])


# Chunks with many rows run on the tensor-core kernel (over a decoded copy for caches that need one); the
# cases above have few rows and run on the warp-level kernels with their keys split.
WIDE_CTX, WIDE_CHUNK = [256, 300, 333, 258, 410, 277, 500, 301], np.array([256, 200, 256, 1, 255, 130, 256, 256])


def _wide(kind, sinks=0, **kw):
    return workload(kind, sinks=sinks, B=8, H_q=32, H_kv=8, ctx_list=WIDE_CTX, **kw)


def _copy_bytes(g, max_q, max_ctx, anchors, window):
    # the decoded copy: a dense table and, per sequence, the blocks that the chunk can attend
    mb = -(-max_ctx // 16)
    cap = min(mb, -(-min(anchors, max_ctx) // 16) + (window + max_q) // 16 + 2)
    return -(-g.w.B * mb * 4 // 256) * 256 + 2 * g.w.B * cap * 16 * g.w.H_kv * 128 * 2


@pytest.mark.parametrize("window,anchors", [(1, 1), (16, 4), (50, 16), (50, 17), (37, 100), (130, 130), (300, 3)])
def test_prefill_many_rows(window, anchors):
    _prefill_case(_wide("bf16"), WIDE_CHUNK, window, anchors)


@pytest.mark.parametrize("kind,sinks,anchors", [("bf16", 4, 4), ("bf16", 20, 40), ("fp8", 0, 4), ("fp8", 4, 4),
                                                ("fp8", 4, 21), ("fp8tok", 4, 4), ("int4", 0, 20)])
def test_prefill_many_rows_of_decoded_caches(kind, sinks, anchors):
    w = _wide(kind, sinks)
    g, _, _, _ = _prefill_case(w, WIDE_CHUNK, 45, anchors)
    assert N.pa_prefill_anchored_workspace_size(g.desc, 256, 500, anchors) == _copy_bytes(g, 256, 500, anchors, 45)


def test_prefill_many_rows_scales_of_either_sign():
    w = _wide("fp8", 5)
    w.k_scales[1] *= -1
    w.v_scales[2] *= -1
    _prefill_case(w, WIDE_CHUNK, 45, 7)


def test_prefill_many_rows_eight_heads_per_kv_head_and_one():
    for H_q, H_kv, chunk in ((64, 8, 100), (16, 16, 256)):
        w = workload("bf16", B=8, H_q=H_q, H_kv=H_kv, ctx_list=WIDE_CTX)
        _prefill_case(w, np.minimum(WIDE_CHUNK, chunk), 60, 20)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_prefill_many_rows_bad_tables_and_lengths(kind):
    w = _wide(kind)
    g, _, q, q_start = _prefill_case(w, WIDE_CHUNK, 20, 4)
    good = prefill(g, q.cuda(), q_start, w.ctx_old, 256, 4)
    g.tables[1, 0] = w.num_blocks           # the anchors' block
    g.tables[2, (333 - 1) // 16] = -1       # the last block
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    ctx = w.ctx_old.copy()
    ctx[4] = 254  # 255 queries of a sequence of 254
    out = prefill(g, q.cuda(), q_start, ctx, 256, 4, max_ctx=500)
    assert g.err_bits() == N.PA_EFLAG_BAD_BLOCK_ID | N.PA_EFLAG_CTX_OVERFLOW
    last = q_start[3] - 16  # sequence 2: every query tile whose keys include its last block
    assert np.all(out[q_start[1]:q_start[2]][100:] == 0) and np.all(out[last:q_start[3]] == 0)
    assert np.all(out[q_start[4]:q_start[5]] == 0)
    for s in (0, 3, 5, 6, 7):
        assert np.array_equal(out[q_start[s]:q_start[s + 1]], good[q_start[s]:q_start[s + 1]])


# Items of many key tiles that do not fill the last round of CTAs are cut in parts and joined.
def _parts_bytes(items):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 256 + -(-sms * 16 // 256) * 256 + min(8 * items, 2 * sms) * 2 * 128 * 130 * 4


@pytest.mark.parametrize("H_q,H_kv,chunk", [(8, 2, [300, 300]), (8, 2, [300, 1]), (2, 2, [257, 400]), (8, 8, [257, 400]),
                                            (4, 2, [130, 300]), (16, 2, [100, 77]), (4, 1, [64, 65]), (8, 2, [0, 250])])
@pytest.mark.parametrize("window,anchors", [(1000, 20), (1500, 3)])
def test_prefill_parts(H_q, H_kv, chunk, window, anchors):
    w = workload("bf16", B=2, H_q=H_q, H_kv=H_kv, ctx_list=[1533, 2301])
    g, _, _, _ = _prefill_case(w, np.array(chunk), window, anchors)
    items = 2 * H_kv * -(-max(chunk) // (256 * H_kv // H_q))
    if items >= 16:  # (fewer may run on the warp-level kernel, their keys split)
        assert N.pa_prefill_anchored_workspace_size(g.desc, max(chunk), 2301, anchors) == _parts_bytes(items)


def test_prefill_parts_after_whole_rounds():
    # 5 sequences' items fill one round and part of another; short sequences have items of few tiles
    w = workload("bf16", B=5, H_q=32, H_kv=8, ctx_list=[1500, 700, 1333, 260, 1801])
    _prefill_case(w, np.array([300, 300, 290, 260, 310]), 1000, 20)


def test_prefill_parts_of_few_tiles():
    # more parts than an item has tiles
    w = workload("bf16", B=2, H_q=8, H_kv=1, ctx_list=[2000, 140])
    _prefill_case(w, np.array([100, 140]), 1800, 20)


@pytest.mark.parametrize("kind,sinks,H_kv", [("bf16", 4, 2), ("fp8", 0, 2), ("fp8", 4, 2), ("fp8tok", 4, 4), ("int4", 0, 4)])
def test_prefill_parts_of_decoded_caches(kind, sinks, H_kv):
    w = workload(kind, sinks=sinks, B=2, H_q=4 * H_kv, H_kv=H_kv, ctx_list=[1533, 1301])
    if kind == "fp8":
        w.k_scales[1] *= -1
    g, _, _, _ = _prefill_case(w, np.array([300, 200]), 1000, 21)
    assert N.pa_prefill_anchored_workspace_size(g.desc, 300, 1533, 21) == \
        _copy_bytes(g, 300, 1533, 21, 1000) + _parts_bytes(2 * H_kv * 5)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_prefill_parts_bad_tables_and_lengths(kind):
    w = workload(kind, B=4, H_q=8, H_kv=2, ctx_list=[1533, 1301, 1400, 1200])
    chunk = np.array([300, 200, 128, 64])
    g, _, q, q_start = _prefill_case(w, chunk, 1000, 20)
    good = prefill(g, q.cuda(), q_start, w.ctx_old, 300, 20)
    g.tables[0, 0] = w.num_blocks           # the anchors' block
    g.tables[1, (1301 - 1) // 16] = -1      # the last block: the last query tile alone
    g.tables_dev.copy_(torch.from_numpy(g.tables))
    ctx = w.ctx_old.copy()
    ctx[2] = 127  # 128 queries of a sequence of 127
    out = prefill(g, q.cuda(), q_start, ctx, 300, 20, max_ctx=1533)
    assert g.err_bits() == N.PA_EFLAG_BAD_BLOCK_ID | N.PA_EFLAG_CTX_OVERFLOW
    assert np.all(out[:q_start[1]] == 0) and np.all(out[q_start[2] - 8:q_start[3]] == 0)
    first = slice(q_start[1], q_start[1] + 128)  # other cuts than before, so other roundings
    assert np.abs(out[first] - good[first]).max() < 2.0 ** -6 * np.abs(good[first]).max()
    rest = slice(q_start[3], q_start[4])
    assert np.abs(out[rest] - good[rest]).max() < 2.0 ** -6 * np.abs(good[rest]).max()


def test_prefill_parts_context_beyond_the_declared_one():
    w = workload("bf16", B=2, H_q=8, H_kv=2, ctx_list=[1533, 1301])
    g, _ = states(w, 1000)
    q = torch.randn(400, w.H_q, w.D, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    out = prefill(g, q, np.array([0, 200, 400]), w.ctx_old, 200, 20, max_ctx=1532)
    assert N.pa_prefill_anchored_workspace_size(g.desc, 200, 1532, 20) == _parts_bytes(2 * 2 * 4)
    assert g.err_bits() == N.PA_EFLAG_CTX_OVERFLOW
    assert np.all(out[:200] == 0) and np.all(np.abs(out[200:]).max(axis=(1, 2)) > 0)


def test_prefill_parts_replayed_with_other_lengths():
    w = workload("bf16", B=2, H_q=8, H_kv=2, ctx_list=[1533, 1301])
    g, o = states(w, 1000)
    q_start = np.array([0, 200, 330])
    q = torch.randn(330, w.H_q, w.D, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    out = torch.zeros(330, w.H_q, w.D, dtype=torch.bfloat16, device="cuda")
    n = N.pa_prefill_anchored_workspace_size(g.desc, 200, 1533, 20)
    ws, ctx, qd, qs = torch.empty(n, dtype=torch.uint8, device="cuda"), gpu(w.ctx_old), q.cuda(), gpu(q_start)

    def call():
        N.pa_prefill_attention_anchored(g.desc, out, qd, g.k, g.v, g.tables_dev, qs, ctx, 200, 1533, w.scale, 20, ws, n,
                                        g.err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
            call()
    torch.cuda.synchronize()
    qv = O.bf16_bits_to_f64(bf16_bits(q))
    for lens, starts in (([1533, 1301], [0, 200, 330]), ([200, 1290], [0, 200, 201]), ([1500, 1301], [0, 0, 130])):
        ctx.copy_(gpu(lens))
        qs.copy_(gpu(np.array(starts)))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for s, c in enumerate(lens):
            rows = slice(starts[s], starts[s + 1])
            if starts[s] == starts[s + 1]:
                continue
            mask = O.anchored_mask(c, starts[s + 1] - starts[s], 1000, 20)
            K, V = O.gather_positions(o.cache, s, o.tables[s], np.arange(c))
            ref, mag = O.masked_attention(qv[rows], K, V, w.scale, mask)
            assert_within(to_f64(out)[rows], ref, tolerance(ref, mag), f"replay at {lens}, sequence {s}")
    assert g.err_bits() == 0


def test_prefill_few_rows_over_a_long_window():
    # up to 32 shares of the keys, one of them empty, and sequences without keys in some
    for chunk, G in (([1, 3], 1), ([8, 2], 4), ([5, 7], 7)):
        w = workload("bf16", B=2, H_q=2 * G, H_kv=2, D=128 if G < 7 else 64, ctx_list=[3500, 40])
        _prefill_case(w, np.array(chunk), 3000, 130)
    w = workload("fp8", B=1, sinks=4, H_q=12, H_kv=4, ctx_list=[1900])
    _prefill_case(w, np.array([5]), 1500, 40)


def test_prefill_replayed_from_a_graph_on_another_stream():
    w = workload("bf16", B=3, ctx_list=[200, 333, 500])
    g, o = states(w, 100)
    q_start = np.array([0, 3, 4, 9])
    q = torch.randn(9, w.H_q, w.D, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    out = torch.zeros(9, w.H_q, w.D, dtype=torch.bfloat16, device="cuda")
    n = N.pa_prefill_anchored_workspace_size(g.desc, 5, 500, 20)
    assert n > 0  # keys split
    ws, ctx, qd, qs = torch.empty(n, dtype=torch.uint8, device="cuda"), gpu(w.ctx_old), q.cuda(), gpu(q_start)

    def call():
        N.pa_prefill_attention_anchored(g.desc, out, qd, g.k, g.v, g.tables_dev, qs, ctx, 5, 500, w.scale, 20, ws, n, g.err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    qv = O.bf16_bits_to_f64(bf16_bits(q))
    for lens in ([200, 333, 500], [3, 60, 499]):
        ctx.copy_(gpu(lens))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for s, c in enumerate(lens):
            rows = slice(q_start[s], q_start[s + 1])
            mask = O.anchored_mask(c, q_start[s + 1] - q_start[s], 100, 20)
            K, V = O.gather_positions(o.cache, s, o.tables[s], np.arange(c))
            ref, mag = O.masked_attention(qv[rows], K, V, w.scale, mask)
            assert_within(to_f64(out)[rows], ref, tolerance(ref, mag), f"replay at {lens}, sequence {s}")
    assert g.err_bits() == 0


def test_prefill_context_beyond_the_declared_one():
    w = workload("bf16", B=2, ctx_list=[400, 300])
    g, _ = states(w, 200)
    q = torch.randn(4, w.H_q, w.D, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    out = prefill(g, q, np.array([0, 2, 4]), w.ctx_old, 2, 20, max_ctx=399)
    assert N.pa_prefill_anchored_workspace_size(g.desc, 2, 399, 20) > 0
    assert g.err_bits() == N.PA_EFLAG_CTX_OVERFLOW
    assert np.all(out[:2] == 0) and np.all(np.abs(out[2:]).max(axis=(1, 2)) > 0)


def test_prefill_then_decode_over_released_blocks():
    """A stream: chunks and single tokens alternate, blocks leave the pool as the window slides."""
    window, anchors = 50, 4
    w = workload("bf16", B=2, ctx_list=[0, 0], steps=150)
    g, o = states(w, window)
    pos = 0
    i = 0
    for n in (30, 1, 1, 64, 1, 17, 1, 1, 30):
        for _ in range(n):
            p = np.array([pos, pos])
            g.prepare(p)
            o.prepare(p)
            g.append(w.k_new[i], w.v_new[i], p)
            o.append(w.k_new[i], w.v_new[i], p)
            pos, i = pos + 1, i + 1
        ctx = np.array([pos, pos])
        if n == 1:
            out = to_f64(decode_anchored(g, w.q[i - 1], ctx, anchors))
            ref, tol = _ref_decode(o, w, w.q[i - 1], ctx, window, anchors)
        else:
            q = w.q[i - n:i].transpose(0, 1).reshape(2 * n, w.H_q, w.D).contiguous()
            out = prefill(g, q.cuda(), [0, n, 2 * n], ctx, n, anchors)
            qv = O.bf16_bits_to_f64(bf16_bits(q))
            mask = O.anchored_mask(pos, n, window, anchors)
            see = np.nonzero(mask.any(0))[0]
            ref, tol = np.zeros(out.shape), np.zeros(out.shape)
            for s in range(2):
                K, V = O.gather_positions(o.cache, s, o.tables[s], see)
                r, m = O.masked_attention(qv[s * n:(s + 1) * n], K, V, w.scale, mask[:, see])
                ref[s * n:(s + 1) * n], tol[s * n:(s + 1) * n] = r, tolerance(r, m)
        assert_within(out, ref, tol, f"after {pos} tokens")
        release(g, o, ctx, window, anchors)
    assert g.err_bits() == 0
    held = 2 * sum(1 for b in range(-(-pos // 16)) if b == 0 or b >= (pos - window) // 16)
    assert g.bm.num_free() == w.num_blocks - held
