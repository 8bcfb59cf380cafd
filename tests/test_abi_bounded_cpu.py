"""Host checks of the bounded-cache calls: refusals before anything is enqueued, workspace sizes, and the
anchored window release against the oracle's pool."""

import numpy as np
import pytest

import oracle as O
from paged_kv_cache_table_gb300 import build as B
from paged_kv_cache_table_gb300 import native as N

FAKE = 1 << 20  # never dereferenced: every call below returns before launching


def _no_gpu():
    try:
        import torch
        return not torch.cuda.is_available()
    except ImportError:
        return True


# Calls with fake device addresses are made only where no GPU is visible: should a host check ever go
# missing, such a call must not reach a device.
host_only = pytest.mark.skipif(not _no_gpu(), reason="fake device addresses: run without a GPU")


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def _desc(**kw):
    base = dict(num_seqs=8, num_q_heads=32, num_kv_heads=8, head_dim=128, num_blocks=64, max_blocks_per_seq=100,
                sliding_window=256)
    base.update(kw)
    return N.make_desc(**base)


def _refused(call, good, bad):
    for kw, status in bad:
        with pytest.raises(N.PaError) as e:
            call(**dict(good, **kw))
        assert e.value.status == status, kw


QUANT = dict(k_dtype="e4m3", v_dtype="int8", k_scales=FAKE, v_scales=FAKE)


@host_only
def test_anchored_decode():
    d = _desc()
    need = N.pa_decode_anchored_workspace_size(d, 1600, 512, 20)
    # 512-token partitions of the window's 256 / 16 + 2 blocks and the anchors' two: one per sequence
    assert need == 256 + 8 * 1 * 32 * 132 * 4
    # 16-token ones; contexts too short for a window still have room for a block listed twice
    assert N.pa_decode_anchored_workspace_size(d, 1600, 16, 20) == 256 + 8 * 20 * 32 * 132 * 4
    assert N.pa_decode_anchored_workspace_size(d, 160, 16, 20) == 256 + 8 * 11 * 32 * 132 * 4
    for part in (16, 512):
        assert N.pa_decode_anchored_workspace_size(d, 1600, part, 0) == N.pa_decode_workspace_size(d, 1600, part)
        whole = _desc(sliding_window=0)
        assert N.pa_decode_anchored_workspace_size(whole, 1600, part, 9) == N.pa_decode_workspace_size(whole, 1600, part)
    assert N.pa_decode_anchored_workspace_size(d, 1600, 512, -1) == 0
    assert N.pa_decode_anchored_workspace_size(d, 1600, 24, 4) == 0
    assert N.pa_decode_anchored_workspace_size(d, 2 ** 31 - 1, 512, 2 ** 31 - 1) > 0

    def call(out=FAKE, q=FAKE, k=FAKE, ctx=FAKE, max_ctx=1600, scale=0.1, anchors=20, ws=FAKE, n=need, desc=d):
        N.pa_decode_attention_anchored(desc, out, q, k, FAKE, FAKE, ctx, max_ctx, scale, 512, anchors, ws, n, None, 0)

    _refused(call, {}, [
        (dict(anchors=-1), N.PA_ERR_INVALID_ARG), (dict(out=0), N.PA_ERR_INVALID_ARG), (dict(q=FAKE + 8), N.PA_ERR_INVALID_ARG),
        (dict(ctx=0), N.PA_ERR_INVALID_ARG), (dict(max_ctx=-1), N.PA_ERR_INVALID_ARG),
        (dict(scale=float("inf")), N.PA_ERR_INVALID_ARG), (dict(ws=FAKE + 16), N.PA_ERR_INVALID_ARG),
        (dict(n=need - 1), N.PA_ERR_WORKSPACE_TOO_SMALL), (dict(desc=_desc(head_dim=96)), N.PA_ERR_UNSUPPORTED)])
    call(desc=_desc(num_seqs=0))  # nothing to enqueue


@host_only
def test_anchored_prefill():
    # many rows, the tensor-core kernel: bf16 caches without sinks need no workspace
    assert N.pa_prefill_anchored_workspace_size(_desc(), 256, 1600, 4) == 0
    d = _desc(**QUANT)
    # a dense table of 100 entries a sequence and, per sequence, the blocks that 256 queries of a
    # 256-token window and 20 anchors can attend: 2 + (256 + 256) / 16 + 2
    def copy(blocks, mb):
        return (8 * mb * 4 + 255) // 256 * 256 + 2 * 8 * blocks * 16 * 8 * 128 * 2
    assert N.pa_prefill_anchored_workspace_size(d, 256, 1600, 20) == copy(36, 100)
    assert N.pa_prefill_anchored_workspace_size(d, 256, 400, 20) == copy(25, 25)  # never more than the context
    # few rows: a tile's keys split; per query row and share of the keys head_dim + 4 floats.  One query of
    # 8 x 8 KV heads is 64 CTAs over 2 + (256 + 1) / 16 + 2 = 20 blocks: three shares of at least 8 blocks
    assert N.pa_prefill_anchored_workspace_size(_desc(), 1, 1600, 20) == 8 * 1 * 32 * 3 * 132 * 4
    assert N.pa_prefill_anchored_workspace_size(_desc(head_dim=64), 1, 1600, 20) == 8 * 1 * 32 * 3 * 68 * 4
    assert N.pa_prefill_anchored_workspace_size(_desc(num_q_heads=24), 1, 1600, 20) == 8 * 1 * 24 * 3 * 132 * 4
    # without anchors or a window the call is pa_prefill_attention_ws
    whole = _desc(sliding_window=0, **QUANT)
    assert N.pa_prefill_anchored_workspace_size(whole, 64, 1600, 20) == N.pa_prefill_workspace_size(whole, 1600)
    assert N.pa_prefill_anchored_workspace_size(_desc(), 1, 1600, 0) == 0
    for bad in ((-1, 1600, 4), (64, -1, 4), (64, 1601, 4), (64, 1600, -1)):
        assert N.pa_prefill_anchored_workspace_size(d, *bad) == 0
    need = copy(36, 100)

    def call(out=FAKE, q_start=FAKE, max_q=256, max_ctx=1600, scale=0.1, anchors=20, ws=FAKE, n=need, desc=d):
        N.pa_prefill_attention_anchored(desc, out, FAKE, FAKE, FAKE, FAKE, q_start, FAKE, max_q, max_ctx, scale, anchors,
                                        ws, n, None, 0)

    _refused(call, {}, [
        (dict(anchors=-1), N.PA_ERR_INVALID_ARG), (dict(out=FAKE + 8), N.PA_ERR_INVALID_ARG),
        (dict(q_start=0), N.PA_ERR_INVALID_ARG), (dict(max_q=-1), N.PA_ERR_INVALID_ARG),
        (dict(max_ctx=1601), N.PA_ERR_INVALID_ARG), (dict(scale=0.0), N.PA_ERR_INVALID_ARG),
        (dict(scale=-0.1), N.PA_ERR_INVALID_ARG), (dict(scale=float("nan")), N.PA_ERR_INVALID_ARG),
        (dict(ws=0), N.PA_ERR_INVALID_ARG), (dict(ws=FAKE + 16), N.PA_ERR_INVALID_ARG),
        (dict(n=need - 1), N.PA_ERR_WORKSPACE_TOO_SMALL),
        (dict(max_q=1, desc=_desc(), n=1000), N.PA_ERR_WORKSPACE_TOO_SMALL),
        (dict(max_q=1, desc=_desc(), ws=0), N.PA_ERR_INVALID_ARG)])
    odd = _desc(num_sink=4, k_sink=FAKE + 8, v_sink=FAKE, **QUANT)
    _refused(call, dict(desc=odd, n=1 << 40), [(dict(), N.PA_ERR_INVALID_ARG)])  # sink rows are read 16 bytes at a time
    call(desc=_desc(num_seqs=0, **QUANT))
    call(max_q=0)


@host_only
def test_weights():
    d = _desc(sliding_window=0)
    for part in (0, 512) if not _no_gpu() else (512,):
        base = (N.pa_decode_workspace_size(d, 1000, part) + 255) // 256 * 256
        assert N.pa_decode_weights_workspace_size(d, 1000, part) == base + 8 * 8 * 1008 * 4 * 4
        odd = _desc(num_q_heads=40, sliding_window=0)  # five query heads a KV head: eight scores a position
        base = (N.pa_decode_workspace_size(odd, 1000, part) + 255) // 256 * 256
        assert N.pa_decode_weights_workspace_size(odd, 1000, part) == base + 8 * 8 * 1008 * 8 * 4
    assert N.pa_decode_weights_workspace_size(d, -1, 512) == 0
    assert N.pa_decode_weights_workspace_size(d, 2 ** 31 - 1, 512) == 0
    need = N.pa_decode_weights_workspace_size(d, 1000, 512)

    def call(out=FAKE, si=FAKE, so=FAKE, stride=1000, max_ctx=1000, scale=0.1, part=512, ws=FAKE, n=need, desc=d):
        N.pa_decode_attention_weights(desc, out, FAKE, FAKE, FAKE, FAKE, FAKE, max_ctx, scale, part, si, so, stride, ws, n,
                                      None, 0)

    _refused(call, {}, [
        (dict(so=0), N.PA_ERR_INVALID_ARG), (dict(so=FAKE + 2), N.PA_ERR_INVALID_ARG), (dict(si=FAKE + 1), N.PA_ERR_INVALID_ARG),
        (dict(stride=999), N.PA_ERR_INVALID_ARG), (dict(out=0), N.PA_ERR_INVALID_ARG), (dict(ws=0), N.PA_ERR_INVALID_ARG),
        (dict(ws=FAKE + 64), N.PA_ERR_INVALID_ARG), (dict(n=need - 1), N.PA_ERR_WORKSPACE_TOO_SMALL),
        (dict(part=24), N.PA_ERR_INVALID_ARG), (dict(scale=float("nan")), N.PA_ERR_INVALID_ARG),
        (dict(desc=_desc(block_size=32)), N.PA_ERR_UNSUPPORTED)])
    call(desc=_desc(num_seqs=0))


@host_only
def test_evict():
    d = _desc(sliding_window=0)
    # at most min(budget, context - budget) rows move per (sequence, KV head), 8 bytes for either end of
    # each, and a count per (sequence, KV head)
    for max_ctx, budget, rows in ((1000, 900, 100), (1000, 300, 300), (1000, 1000, 0), (0, 5, 0)):
        a = (64 * rows * 8 + 255) // 256 * 256
        assert N.pa_cache_evict_workspace_size(d, max_ctx, budget) == 2 * a + 256 + 256
    assert N.pa_cache_evict_workspace_size(d, 1000, 0) == 0 and N.pa_cache_evict_workspace_size(d, -1, 5) == 0
    need = N.pa_cache_evict_workspace_size(d, 1000, 900)

    def call(k=FAKE, v=FAKE, tables=FAKE, ctx=FAKE, max_ctx=1000, si=FAKE, so=FAKE, pi=FAKE, po=FAKE, stride=1000,
             budget=900, anchors=4, recent=100, ws=FAKE, n=need, desc=d):
        N.pa_cache_evict(desc, k, v, tables, ctx, max_ctx, si, so, pi, po, stride, budget, anchors, recent, ws, n, None, 0)

    inval = [dict(k=0), dict(v=FAKE + 8), dict(tables=0), dict(ctx=0), dict(si=0), dict(so=0), dict(po=0), dict(so=FAKE + 2),
             dict(pi=FAKE + 2), dict(po=FAKE + 1), dict(stride=999), dict(budget=0), dict(anchors=-1), dict(recent=-1),
             dict(anchors=801, recent=100), dict(recent=2 ** 31 - 1, anchors=900), dict(ws=0), dict(ws=FAKE + 16),
             dict(max_ctx=-1),
             dict(desc=_desc(sliding_window=0, num_sink=5, k_sink=FAKE, v_sink=FAKE))]  # anchors below the sinks
    _refused(call, {}, [(kw, N.PA_ERR_INVALID_ARG) for kw in inval] + [
        (dict(n=need - 1), N.PA_ERR_WORKSPACE_TOO_SMALL), (dict(desc=_desc()), N.PA_ERR_UNSUPPORTED),
        (dict(max_ctx=2 ** 21 + 1, stride=2 ** 22), N.PA_ERR_UNSUPPORTED),
        (dict(desc=_desc(sliding_window=0, head_dim=96)), N.PA_ERR_UNSUPPORTED)])
    call(desc=_desc(sliding_window=0, num_seqs=0))


@pytest.mark.parametrize("window,anchors", [(16, 4), (20, 16), (33, 17), (40, 100), (0, 4), (5, 0)])
def test_anchored_release_matches_the_oracle_pool(window, anchors):
    rng = np.random.default_rng(window * 7 + anchors)
    nb, S, M = 60, 3, 14
    bm, pool = N.BlockManager(nb), O.BlockPool(nb)
    tables = np.full((S, M), -1, np.int32)
    otab = tables.astype(np.int64)
    pos = np.zeros(S, np.int32)
    for _ in range(16 * M - 8):
        bm.prepare_step(tables, pos)
        for s in range(S):
            pool.prepare_append(otab[s], int(pos[s]))
        pos += 1
        if rng.random() < 0.1:
            s = int(rng.integers(S))
            got = bm.slide_window(tables[s:s + 1], pos[s:s + 1], window, anchors)[1]
            assert got == O.slide_window_anchored(pool, otab[s], int(pos[s]), window, anchors)
        assert np.array_equal(tables, otab) and bm.num_free() == pool.num_free()
    assert np.all(tables[:, :min(M, -(-anchors // 16))] >= 0)


def test_anchored_release_rejects_bad_arguments():
    bm = N.BlockManager(8)
    t = np.array([[0, 1, 2, 3]], np.int32)
    with pytest.raises(N.PaError):
        bm.slide_window(t, np.array([64], np.int32), 8, -1)
    with pytest.raises(N.PaError):  # blocks the pool does not hold
        bm.slide_window(t, np.array([64], np.int32), 8, 4)
    assert t.tolist() == [[0, 1, 2, 3]]
