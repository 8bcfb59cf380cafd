"""Cases of the operators that keep a KV cache bounded, and their plain forms.

Four operators over the paged cache (pool of 16-slot blocks, block tables, GQA):

  anchored   decode attention over a sliding window and the first tokens (anchors)
  prefill    the same for a chunk of new queries per sequence
  weights    decode attention that adds every position's softmax weight to an accumulated score
  evict      eviction of the positions with the least accumulated score, per sequence and KV head,
             the cache compacted in place

``run`` is one call of an operator: with ``own`` false in elementary torch operations in fp32,
with ``own`` true through the library.  ``exact`` computes the same from the definition in fp64.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
DEV = "cuda"


# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # four short chats, one of them at its first token: what a step costs when nothing is large
        dict(name="anchored tiny", op="anchored", kv="bf16", B=4, Hq=8, Hkv=2, D=64, ctx="1,17,100,256", window=64,
             anchors=4, sinks=0),
        # a batch of long streams, each of which attends its last 4096 tokens and its first four
        dict(name="anchored batch", op="anchored", kv="bf16", B=64, Hq=32, Hkv=8, D=128, ctx="4096:16384:1",
             window=4096, anchors=4, sinks=0),
        # an odd batch of very long streams over an 8-bit cache, the anchors kept in bf16 beside it
        dict(name="anchored 8-bit", op="anchored", kv="fp8", B=37, Hq=64, Hkv=8, D=128, ctx="1000:131072:2",
             window=2047, anchors=4, sinks=4),
        # a chunk of every prompt of a batch, most of them past their window
        dict(name="prefill chunk", op="prefill", kv="bf16", B=8, Hq=32, Hkv=8, D=128, ctx="512:16384:3",
             chunk="512:512:0", window=4096, anchors=4, sinks=0),
        # ragged prompts, an odd window, anchors over more than one block, eight query heads a KV head
        dict(name="prefill ragged", op="prefill", kv="bf16", B=6, Hq=64, Hkv=8, D=128, ctx="700:9000:4",
             chunk="1:700:5", window=1000, anchors=20, sinks=0),
        # chunks over an 8-bit cache with its anchors in bf16
        dict(name="prefill 8-bit", op="prefill", kv="fp8", B=4, Hq=32, Hkv=8, D=128, ctx="2000:9000:6",
             chunk="1000:1024:7", window=2048, anchors=4, sinks=4),
        dict(name="weights tiny", op="weights", kv="bf16", B=4, Hq=8, Hkv=2, D=64, ctx="1,17,100,256", sinks=0),
        # the batch of an 8B-class model that a server decodes
        dict(name="weights batch", op="weights", kv="bf16", B=64, Hq=32, Hkv=8, D=128, ctx="512:4096:8", sinks=0),
        # few very long contexts over an 8-bit cache
        dict(name="weights long", op="weights", kv="fp8", B=4, Hq=32, Hkv=8, D=128, ctx="131072:131072:0", sinks=4),
        # a cache held at 2048 tokens that has taken 64 new ones: the eviction of every 64th step
        dict(name="evict step", op="evict", B=64, Hkv=8, D=128, ctx="2112:2112:0", budget=2048, recent=256,
             anchors=4, evicted=4096),
        # the first eviction of prompts of many lengths, some within the budget
        dict(name="evict prompts", op="evict", B=16, Hkv=8, D=128, ctx="500:8192:9", budget=1024, recent=128,
             anchors=4, evicted=0),
        # very long prompts cut to a quarter
        dict(name="evict long", op="evict", B=4, Hkv=8, D=128, ctx="131072:131072:0", budget=32768, recent=4096,
             anchors=4, evicted=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["anchored", "prefill", "weights", "evict"])
    kv = rng.choice(["bf16", "bf16", "fp8", "fp8tok", "int4"])
    heads = [(32, 8, 128), (64, 8, 128), (8, 8, 128), (12, 4, 128)]
    if kv == "bf16":
        heads += [(8, 2, 64), (5, 1, 128), (14, 2, 64)]
    Hq, Hkv, D = rng.choice(heads)
    seed = rng.randrange(1 << 20)
    if op == "evict":
        B = _log(rng, 1, 64)
        cap = max(64, min(131072, 3200000 // (B * Hkv)))
        hi = _log(rng, 40, cap)
        budget = _log(rng, 20, hi)
        anchors = rng.choice([0, 1, 4, 16])
        recent = _log(rng, 1, max(1, budget - anchors))
        fresh = rng.random() < 0.5
        return dict(op=op, B=B, Hkv=Hkv, D=D, ctx="%d:%d:%d" % (max(1, hi // rng.choice([1, 2, 8])), hi, seed),
                    budget=budget, recent=min(recent, max(0, budget - anchors)), anchors=min(anchors, budget),
                    evicted=0 if fresh else _log(rng, 1, 100000))
    sinks = rng.choice([0, 0, 1, 4, 17])
    if op == "prefill":
        B = _log(rng, 1, 12)
        chunk = _log(rng, 1, max(2, 1900 // B))
        window = _log(rng, 1, 4096)
        anchors = rng.choice([sinks, 1, 4, 20, 130])
        hi = chunk + _log(rng, 1, 16384)
        return dict(op=op, kv=kv, B=B, Hq=Hq, Hkv=Hkv, D=D, ctx="%d:%d:%d" % (chunk, hi, seed),
                    chunk="%d:%d:%d" % (max(1, chunk // rng.choice([1, 3])), chunk, seed + 1), window=window,
                    anchors=anchors, sinks=sinks)
    B = _log(rng, 1, 100)
    if op == "anchored":
        window = _log(rng, 1, max(2, min(16384, 240000 // B)))
        anchors = rng.choice([sinks, 1, 4, 20, 130])
        hi = _log(rng, 1, 131072)
        return dict(op=op, kv=kv, B=B, Hq=Hq, Hkv=Hkv, D=D, ctx="%d:%d:%d" % (max(1, hi // 4), hi, seed),
                    window=window, anchors=anchors, sinks=sinks)
    hi = _log(rng, 1, max(2, min(131072, 240000 // B)))
    return dict(op=op, kv=kv, B=B, Hq=Hq, Hkv=Hkv, D=D, ctx="%d:%d:%d" % (max(1, hi // 4), hi, seed), sinks=sinks)


def _lens(text, n):
    """Lengths of n sequences: a list "1,17,100", or "low:high:seed" drawn uniformly."""
    if "," in text:
        return [int(x) for x in text.split(",")]
    lo, hi, seed = (int(x) for x in text.split(":"))
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(n)]


def _chunks(case):
    """(context lengths, new tokens) of a prefill case: every context holds its own chunk."""
    ctx, new = _lens(case["ctx"], case["B"]), _lens(case["chunk"], case["B"])
    return [max(c, n) for c, n in zip(ctx, new)], new


def _scale(case):
    return float(np.float32(1.0 / math.sqrt(case["D"])))  # as the call takes it, in fp32


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------
def _tables(kept, width, rng):
    """Block tables that hold the logical blocks `kept[s]` at random places of the pool, the rest
    released (-1); and the pool's size."""
    need = sum(len(k) for k in kept)
    blocks = need + need // 10 + 2
    place = rng.permutation(blocks).astype(np.int32)
    table = np.full((len(kept), width), -1, dtype=np.int32)
    at = 0
    for s, k in enumerate(kept):
        table[s, k] = place[at:at + len(k)]
        at += len(k)
    return torch.from_numpy(table).to(DEV), blocks


def _encode_int4(x, value):
    """Codes and parameter words of rows x [n][128]: per 32 dims a bf16 scale and a zero point."""
    g = x.float().view(-1, 4, 32)
    lo = g.amin(-1).clamp(max=0)
    s = ((g.amax(-1).clamp(min=0) - lo) / 15).to(torch.bfloat16)
    sf = s.float()
    z = torch.round(-lo / sf).clamp(0, 15)
    q = (torch.round(g / sf[..., None]) + z[..., None]).clamp(0, 15).to(torch.int32)
    prm = (s.view(torch.int16).to(torch.int32) & 0xFFFF) | (z.to(torch.int32) << 16)
    n = q.shape[0]
    if value:  # byte 8r + m: dims 16m + r (low) and 16m + r + 8 (high)
        d = q.view(n, 8, 2, 8)
        codes = (d[:, :, 0] | (d[:, :, 1] << 4)).transpose(1, 2).reshape(n, 64).to(torch.uint8)
    else:  # word 4c + g: dims 32g + 8c + i at bits 4i
        w = q.view(n, 4, 4, 8).to(torch.int64) << (4 * torch.arange(8, device=q.device))
        w = w.sum(-1).transpose(1, 2).reshape(n, 16)
        codes = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous().view(torch.uint8)
    return codes.reshape(-1), prm.contiguous().view(torch.uint8).reshape(-1)


def _pools(case, slots, gen):
    """K and V pools of `slots` slots in the case's cache type, with their per-head scales."""
    kv, H, D = case["kv"], case["Hkv"], case["D"]
    k = torch.randn(slots, H, D, generator=gen, device=DEV).to(torch.bfloat16)
    v = torch.randn(slots, H, D, generator=gen, device=DEV).to(torch.bfloat16)
    if kv == "bf16":
        return k, v, None, None
    if kv == "int4":
        return (torch.cat(_encode_int4(k.view(-1, D), False)), torch.cat(_encode_int4(v.view(-1, D), True)), None, None)
    kf, vf = k.float(), v.float()
    vs = vf.abs().amax((0, 2)) / 127
    v8 = torch.round(vf / vs[:, None]).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    if kv == "fp8":
        ks = kf.abs().amax((0, 2)) / 448
        return (kf / ks[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), v8, ks, vs
    row = kf.abs().amax(-1) / 448  # fp8tok: one scale a row, after the codes
    codes = (kf / row[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes.reshape(-1), row.contiguous().view(torch.uint8).reshape(-1)]), v8, None, vs


def _attention_inputs(case, seed):
    B, Hq, Hkv, D, sinks = case["B"], case["Hq"], case["Hkv"], case["D"], case["sinks"]
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    new = [1] * B
    if case["op"] == "prefill":
        ctx, new = _chunks(case)
    else:
        ctx = _lens(case["ctx"], B)
    width = (max(ctx) + BLOCK - 1) // BLOCK
    kept = []
    for c, n in zip(ctx, new):
        first = max(0, c - n - case["window"] + 1) if "window" in case else 0
        held = set(range(first // BLOCK, (c + BLOCK - 1) // BLOCK))
        if "anchors" in case:
            held |= set(range((min(case["anchors"], c) + BLOCK - 1) // BLOCK))
        kept.append(sorted(held))
    tables, blocks = _tables(kept, width, rng)
    k, v, ks, vs = _pools(case, blocks * BLOCK, gen)
    st = dict(case=case, k=k, v=v, ks=ks, vs=vs, tables=tables, blocks=blocks, scale=_scale(case), max_ctx=max(ctx),
              max_new=max(new), ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV))
    if sinks:
        st["k_sink"] = torch.randn(B, sinks, Hkv, D, generator=gen, device=DEV).to(torch.bfloat16)
        st["v_sink"] = torch.randn(B, sinks, Hkv, D, generator=gen, device=DEV).to(torch.bfloat16)
    # queries that look sharply at a few keys
    q = 1.5 * torch.randn(sum(new), Hq, D, generator=gen, device=DEV)
    st["q"] = q.to(torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    if case["op"] == "prefill":
        st["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(DEV)
    if case["op"] == "weights":
        # weights that a few earlier steps have left: some tokens hold most of them
        w = torch.exp(2 * torch.randn(B, Hkv, width * BLOCK, generator=gen, device=DEV))
        w = w * (0.5 * Hq / Hkv / st["ctx"].float())[:, None, None]
        live = torch.arange(width * BLOCK, device=DEV) < st["ctx"][:, None, None] - 1
        st["scores"] = torch.where(live, w, 0.0)
        st["scores_out"] = torch.zeros_like(st["scores"])
    return st


def _evict_inputs(case, seed):
    B, H, D, budget, recent, anchors = (case[x] for x in ("B", "Hkv", "D", "budget", "recent", "anchors"))
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = _lens(case["ctx"], B)
    width = (max(n) + BLOCK - 1) // BLOCK
    stride = width * BLOCK
    tables, blocks = _tables([list(range((c + BLOCK - 1) // BLOCK)) for c in n], width, rng)
    k = torch.randn(blocks * BLOCK, H, D, generator=gen, device=DEV).to(torch.bfloat16)
    v = torch.randn(blocks * BLOCK, H, D, generator=gen, device=DEV).to(torch.bfloat16)
    ctx = torch.tensor(n, dtype=torch.int32, device=DEV)
    slot = torch.arange(stride, device=DEV)
    live = slot < ctx[:, None, None]
    w = torch.exp(2 * torch.randn(B, H, stride, generator=gen, device=DEV))
    w = torch.where(torch.rand(B, H, stride, generator=gen, device=DEV) < 0.02, 0.0, w)  # some were never looked at
    st = dict(case=case, k=k, v=v, tables=tables, blocks=blocks, max_ctx=max(n), ctx=ctx, pos=None,
              scores=torch.where(live, w, 0.0).contiguous())
    if case["evicted"]:
        # earlier evictions left `budget` slots in no order of position, the anchors in front, and
        # the tokens since were appended behind them
        gone = case["evicted"]
        pool = torch.rand(B, H, stride, generator=gen, device=DEV)
        old = torch.minimum(ctx, torch.full_like(ctx, budget))[:, None, None]
        inner = (slot >= anchors) & (slot < old)
        # distinct positions: each slot's own plus a share of the evicted ones, then shuffled
        spread = slot + torch.div((slot - anchors) * gone, torch.clamp(old - anchors, min=1), rounding_mode="floor")
        pos = torch.where(inner, spread, torch.where(slot < old, slot, slot + gone)).to(torch.int64)
        order = torch.argsort(torch.where(inner, pool, torch.where(slot < anchors, slot - 1e6, slot + 1.0)), dim=-1)
        st["pos"] = pos.expand(B, H, stride).gather(-1, order).to(torch.int32).contiguous()
    st["scores_out"] = torch.zeros_like(st["scores"])
    st["pos_out"] = torch.zeros(B, H, stride, dtype=torch.int32, device=DEV)
    return st


def prepare(case, seed):
    st = _evict_inputs(case, seed) if case["op"] == "evict" else _attention_inputs(case, seed)
    if own:  # the descriptor and the workspace, which a program makes once
        import paged_kv_cache_table_gb300 as P

        dt = {"bf16": ("bf16", "bf16"), "fp8": ("e4m3", "int8"), "fp8tok": ("e4m3_tok", "int8"),
              "int4": ("int4", "int4")}[case.get("kv", "bf16")]
        desc = P.make_desc(case["B"], case.get("Hq", case["Hkv"]), case["Hkv"], case["D"], st["blocks"],
                           st["tables"].shape[1], dt[0], dt[1], st.get("ks"), st.get("vs"), st.get("k_sink"),
                           st.get("v_sink"), case.get("sinks", 0), sliding_window=case.get("window", 0))
        if case["op"] == "anchored":
            size = P.pa_decode_anchored_workspace_size(desc, st["max_ctx"], 0, case["anchors"])
        elif case["op"] == "prefill":
            size = P.pa_prefill_anchored_workspace_size(desc, st["max_new"], st["max_ctx"], case["anchors"])
        elif case["op"] == "weights":
            size = P.pa_decode_weights_workspace_size(desc, st["max_ctx"], 0)
        else:
            size = P.pa_cache_evict_workspace_size(desc, st["max_ctx"], case["budget"])
        st.update(P=P, desc=desc, ws=torch.empty(max(size, 256), dtype=torch.uint8, device=DEV))
    return st


# ------------------------------------------------------------------------------------------
# Plain forms
# ------------------------------------------------------------------------------------------
def _rows(st, index):
    """K and V rows (fp32) of the positions index [B][T] of every sequence, as the cache holds them."""
    case = st["case"]
    kv, H, D = case["kv"], case["Hkv"], case["D"]
    block = st["tables"].gather(1, index // BLOCK).long().clamp(min=0)
    slot = block * BLOCK + index % BLOCK
    n = st["blocks"] * BLOCK
    if kv == "bf16":
        k, v = st["k"][slot].float(), st["v"][slot].float()
    elif kv == "int4":
        split = n * H * 64
        kc = st["k"][:split].view(torch.int32).view(n, H, 4, 4)[slot]  # [.][c][g]
        vc = st["v"][:split].view(n, H, 8, 8)[slot].int()  # [.][r][m]
        kp = st["k"][split:].view(torch.int32).view(n, H, 4)[slot]
        vp = st["v"][split:].view(torch.int32).view(n, H, 4)[slot]
        bits = 4 * torch.arange(8, device=DEV, dtype=torch.int32)
        kq = ((kc[..., None] >> bits) & 15).transpose(-3, -2).reshape(*slot.shape, H, 4, 32)
        vq = torch.stack([vc & 15, vc >> 4], -1).permute(0, 1, 2, 4, 5, 3).reshape(*slot.shape, H, 4, 32)
        k = ((kq - ((kp >> 16) & 255)[..., None]).float() * (kp << 16).view(torch.float32)[..., None]).flatten(-2)
        v = ((vq - ((vp >> 16) & 255)[..., None]).float() * (vp << 16).view(torch.float32)[..., None]).flatten(-2)
    else:
        v = st["v"].view(n, H, D)[slot].view(torch.int8).float() * st["vs"][:, None]
        if kv == "fp8":
            k = st["k"].view(n, H, D)[slot].view(torch.float8_e4m3fn).float() * st["ks"][:, None]
        else:
            split = n * H * D
            k = st["k"][:split].view(n, H, D)[slot].view(torch.float8_e4m3fn).float()
            k = k * st["k"][split:].view(torch.float32).view(n, H)[slot][..., None]
    if case["sinks"]:
        seq = torch.arange(case["B"], device=DEV)[:, None]
        at = index.clamp(max=case["sinks"] - 1)
        front = (index < case["sinks"])[..., None, None]
        k = torch.where(front, st["k_sink"][seq, at].float(), k)
        v = torch.where(front, st["v_sink"][seq, at].float(), v)
    return k, v


def _attended(st, first):
    """Positions of every sequence from its first attended one, after its anchors: [B][T], and which are real."""
    ctx = st["ctx"].long()
    anchors = st["case"].get("anchors", 0)
    near = torch.minimum(torch.full_like(ctx, anchors), first)  # anchors before the window
    total = near + ctx - first
    t = torch.arange(int(anchors + st["span"]), device=DEV)[None]
    index = torch.where(t < near[:, None], t, t - near[:, None] + first[:, None])
    real = t < total[:, None]
    return torch.where(real, index, 0), real


def _plain_decode(st):
    case = st["case"]
    ctx = st["ctx"].long()
    window = case.get("window", 0) or st["max_ctx"]
    st["span"] = min(window, st["max_ctx"])
    index, real = _attended(st, (ctx - window).clamp(min=0))
    k, v = _rows(st, index)
    B, Hkv, G, D = case["B"], case["Hkv"], case["Hq"] // case["Hkv"], case["D"]
    q = st["q"].view(B, Hkv, G, D).float()
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]
    s = s.masked_fill(~real[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.transpose(1, 2)).reshape(B, case["Hq"], D).to(torch.bfloat16)
    return out, p.sum(2)


def _plain_prefill(st):
    case = st["case"]
    B, Hkv, G, D, W = case["B"], case["Hkv"], case["Hq"] // case["Hkv"], case["D"], case["window"]
    ctx, start = st["ctx"].long(), st["q_start"].long()
    new = start[1:] - start[:-1]
    st["span"] = min(st["max_ctx"], W + st["max_new"] - 1)
    index, real = _attended(st, (ctx - new - W + 1).clamp(min=0))
    k, v = _rows(st, index)
    r = torch.arange(st["max_new"], device=DEV)[None]
    mine = r < new[:, None]
    row = torch.where(mine, start[:-1, None] + r, 0)
    q = st["q"][row].view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).float().flatten(2, 3)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, G, -1, index.shape[1]).mul_(st["scale"])
    p = (ctx - new)[:, None] + r  # positions of the queries
    see = real[:, None] & (index[:, None] <= p[..., None])
    see = see & ((index[:, None] > p[..., None] - W) | (index[:, None] < case["anchors"]))
    see = see | ~mine[..., None]  # padding rows: anything finite
    s.masked_fill_(~see[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    s = s.div_(s.sum(-1, keepdim=True))
    o = torch.matmul(s.flatten(2, 3), v.transpose(1, 2)).view(B, Hkv, G, -1, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, -1, case["Hq"], D)[mine].to(torch.bfloat16)


def _plain_evict(st):
    case = st["case"]
    budget, recent, anchors = case["budget"], case["recent"], case["anchors"]
    ctx, scores = st["ctx"].long()[:, None, None], st["scores"]
    B, H, N = scores.shape
    slot = torch.arange(N, device=DEV).expand(B, H, N)
    live = slot < ctx
    pos = slot if st["pos"] is None else st["pos"].long()
    newest = torch.where(live, pos, -1).amax(-1, keepdim=True)
    rank_by = torch.where((pos < anchors) | (pos > newest - recent), math.inf, scores.double())
    rank_by = torch.where(live, rank_by, -math.inf)
    order = torch.sort(rank_by, dim=-1, descending=True, stable=True).indices
    left = torch.clamp(ctx, max=budget)
    keep = torch.zeros(B, H, N, dtype=torch.bool, device=DEV).scatter_(-1, order, slot < left)
    hole, mover = ~keep & (slot < left), keep & (slot >= left)
    to = torch.where(hole, hole.cumsum(-1) - 1, N)
    who = torch.zeros(B, H, N + 1, dtype=torch.int64, device=DEV)
    who.scatter_(-1, torch.where(mover, mover.cumsum(-1) - 1, N), slot)  # the i-th mover
    source = torch.where(hole, who.gather(-1, to), slot)
    inside = slot < left
    st["scores_out"] = torch.where(inside, scores.gather(-1, source), 0.0)
    st["pos_out"] = torch.where(inside, pos.gather(-1, source), newest + 1 + slot - left).int()
    b, h, j = torch.nonzero(hole, as_tuple=True)
    i = source[b, h, j]
    table = st["tables"].long()
    src, dst = table[b, i // BLOCK] * BLOCK + i % BLOCK, table[b, j // BLOCK] * BLOCK + j % BLOCK
    st["k"][dst, h] = st["k"][src, h]
    st["v"][dst, h] = st["v"][src, h]
    return st["k"], st["v"], st["scores_out"], st["pos_out"]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        P, desc = st["P"], st["desc"]
        if op == "anchored":
            P.pa_decode_attention_anchored(desc, st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"],
                                           st["max_ctx"], st["scale"], 0, case["anchors"], st["ws"])
            return st["out"]
        if op == "prefill":
            P.pa_prefill_attention_anchored(desc, st["out"], st["q"], st["k"], st["v"], st["tables"], st["q_start"],
                                            st["ctx"], st["max_new"], st["max_ctx"], st["scale"], case["anchors"],
                                            st["ws"])
            return st["out"]
        if op == "weights":
            P.pa_decode_attention_weights(desc, st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"],
                                          st["max_ctx"], st["scale"], 0, st["scores"], st["scores_out"],
                                          st["scores"].shape[2], st["ws"])
            return st["out"], st["scores_out"]
        P.pa_cache_evict(desc, st["k"], st["v"], st["tables"], st["ctx"], st["max_ctx"], st["scores"],
                         st["scores_out"], st["pos"], st["pos_out"], st["scores"].shape[2], case["budget"],
                         case["anchors"], case["recent"], st["ws"])
        return st["k"], st["v"], st["scores_out"], st["pos_out"]
    if op == "anchored":
        return _plain_decode(st)[0]
    if op == "prefill":
        return _plain_prefill(st)
    if op == "weights":
        out, w = _plain_decode(st)
        new = st["scores"].clone()
        new[:, :, :w.shape[2]] += w
        return out, new
    return _plain_evict(st)


# ------------------------------------------------------------------------------------------
# Work
# ------------------------------------------------------------------------------------------
def work(case):
    op, H, D = case["op"], case["Hkv"], case["D"]
    if op == "evict":
        total = 0
        n = _lens(case["ctx"], case["B"])
        stride = (max(n) + BLOCK - 1) // BLOCK * BLOCK
        for c in n:
            moved = 0.0
            if c > case["budget"]:
                # tokens kept in the slots past the budget: the protected ones there, and of the
                # others the share that is kept anywhere
                b, held = case["budget"], min(case["recent"], c - case["budget"])
                others = max(1, c - case["anchors"] - case["recent"])
                moved = held + (c - b - held) * max(0, b - case["anchors"] - case["recent"]) / others
            total += c * (8 if case["evicted"] else 4) + stride * 8 + moved * 2 * (2 * 2 * D)
        return {"bytes": int(total * H), "flops": 0}
    row = {"bf16": 4 * D, "fp8": 2 * D, "fp8tok": 2 * D + 4, "int4": 160}[case["kv"]]
    Hq, A, S = case["Hq"], case.get("anchors", 0), case["sinks"]
    if op == "prefill":
        keys = pairs = rows = 0
        for c, n in zip(*_chunks(case)):
            first = max(0, c - n - case["window"] + 1)
            keys += c - first + min(A, first)
            rows += n
            for p in range(c - n, c):
                lo = max(0, p - case["window"] + 1)
                pairs += p + 1 - lo + min(A, lo)
        return {"bytes": int(keys * H * row + rows * Hq * D * 4), "flops": int(4 * D * Hq * pairs)}
    read = flops = 0
    for c in _lens(case["ctx"], case["B"]):
        lo = max(0, c - case["window"]) if "window" in case else 0
        t = c - lo + min(A, lo)
        front = min(S, A, lo) + max(0, min(S, c) - lo)  # sink rows, in bf16
        read += ((t - front) * row + front * 4 * D) * H + Hq * D * 4
        flops += 4 * D * Hq * t
        if op == "weights":
            read += 8 * t * H
    return {"bytes": int(read), "flops": int(flops)}


# ------------------------------------------------------------------------------------------
# The definition, in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_cache(st, s, upto):
    """K and V [upto][H][D] of sequence s in fp64 (released positions: zeros)."""
    case = st["case"]
    kv, H, D, nb = case["kv"], case["Hkv"], case["D"], st["blocks"]
    row = st["tables"][s, :(upto + BLOCK - 1) // BLOCK].long()
    gone = (row < 0).repeat_interleave(BLOCK)[:upto]
    row = row.clamp(min=0)

    def blocks(flat, dtype, *shape):
        return flat.view(dtype).reshape(nb, BLOCK, *shape)[row].flatten(0, 1)[:upto]

    def signed8(codes):
        c = codes.double()
        return torch.where(c > 127, c - 256, c)

    def e4m3(codes):  # sign, four exponent bits of bias 7, three mantissa bits
        c = codes.int()
        e, m = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
        return torch.where(c > 127, -mag, mag)

    if kv == "bf16":
        k, v = blocks(st["k"], torch.bfloat16, H, D).double(), blocks(st["v"], torch.bfloat16, H, D).double()
    elif kv == "int4":
        cut = nb * BLOCK * H * 64
        out = []
        for t, pool in enumerate((st["k"], st["v"])):
            code = blocks(pool[:cut], torch.uint8, H, 64).long()
            prm = blocks(pool[cut:], torch.int32, H, 4).long()
            nib = torch.stack([code & 15, code >> 4], -1).flatten(-2)  # nibble x of the row
            d = torch.arange(128, device=DEV)
            if t == 0:  # nibble of dim d = 32g + 8c + i: word 4c + g, nibble i
                x = (4 * ((d % 32) // 8) + d // 32) * 8 + d % 8
            else:  # dim 16m + r (+ 8): byte 8r + m, low (high) nibble
                x = (8 * (d % 8) + d // 16) * 2 + (d % 16) // 8
            scale = torch.bitwise_left_shift(prm & 0xFFFF, 16).int().view(torch.float32).double()
            zero = ((prm >> 16) & 255).double()
            out.append((nib[..., x].double() - zero[..., d // 32]) * scale[..., d // 32])
        k, v = out
    else:
        v = signed8(blocks(st["v"], torch.uint8, H, D)) * st["vs"].double()[:, None]
        if kv == "fp8":
            k = e4m3(blocks(st["k"], torch.uint8, H, D)) * st["ks"].double()[:, None]
        else:
            cut = nb * BLOCK * H * D
            k = e4m3(blocks(st["k"][:cut], torch.uint8, H, D))
            k = k * blocks(st["k"][cut:], torch.float32, H).double()[..., None]
    k[gone], v[gone] = 0, 0
    n = min(case["sinks"], upto)
    if n:
        k[:n], v[:n] = st["k_sink"][s, :n].double(), st["v_sink"][s, :n].double()
    return k, v


def _exact_attention(case, seed):
    st = _attention_inputs(case, seed)
    Hkv, D, G = case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    scores = st["scores"].double() if case["op"] == "weights" else None
    start = st["q_start"].tolist() if case["op"] == "prefill" else list(range(case["B"] + 1))
    for s, c in enumerate(st["ctx"].tolist()):
        n = start[s + 1] - start[s]
        k, v = _exact_cache(st, s, c)
        t, p = torch.arange(c, device=DEV), torch.arange(c - n, c, device=DEV)[:, None]
        see = t <= p
        if "window" in case:
            see = see & ((p - t < case["window"]) | (t < case["anchors"]))
        some = see.any(0).nonzero()[:, 0]
        see, k, v = see[:, some], k[some], v[some]
        for h in range(Hkv):
            q = st["q"][start[s]:start[s + 1], h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,td->gnt", q, k[:, h]) * st["scale"]
            x = torch.where(see, x, -math.inf)
            w = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
            out[start[s]:start[s + 1], h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", w, v[:, h])
            if scores is not None:
                scores[s, h, some] += w.sum((0, 1))
    return out if scores is None else (out, scores)


def _exact_evict(case, seed):
    st = _evict_inputs(case, seed)
    budget, recent, anchors = case["budget"], case["recent"], case["anchors"]
    scores, table = st["scores"].cpu().numpy().astype(np.float64), st["tables"].cpu().numpy().astype(np.int64)
    B, H, N = scores.shape
    pos = np.broadcast_to(np.arange(N), scores.shape) if st["pos"] is None else st["pos"].cpu().numpy()
    new_scores, new_pos = np.zeros(scores.shape), np.zeros(scores.shape, dtype=np.int64)
    src, dst, head = [], [], []
    for s, n in enumerate(st["ctx"].tolist()):
        left = min(n, budget)
        for h in range(H):
            sc, po = scores[s, h, :n], pos[s, h, :n].astype(np.int64)
            last = po.max()
            safe = (po < anchors) | (po > last - recent)
            best = np.lexsort((np.arange(n), -sc, ~safe))[:left]  # safe ones, then by score, then by slot
            best = np.sort(best)
            holes, movers = np.setdiff1d(np.arange(left), best), best[best >= left]
            place = np.arange(left)
            place[holes] = movers
            new_scores[s, h, :left] = sc[place]
            new_pos[s, h, :left] = po[place]
            new_pos[s, h, left:] = last + 1 + np.arange(N - left)
            src.append(table[s, movers // BLOCK] * BLOCK + movers % BLOCK)
            dst.append(table[s, holes // BLOCK] * BLOCK + holes % BLOCK)
            head.append(np.full(len(holes), h))
    src, dst, head = (torch.from_numpy(np.concatenate(x)).to(DEV) for x in (src, dst, head))
    k, v = st["k"], st["v"]
    k[dst, head], v[dst, head] = k[src, head], v[src, head]
    return k, v, torch.from_numpy(new_scores), torch.from_numpy(new_pos.astype(np.int32))


def exact(case, seed):
    return _exact_evict(case, seed) if case["op"] == "evict" else _exact_attention(case, seed)
