// Eviction from the cache by accumulated attention weight.
//
// Untitled KV-cache article at ldpk.cn/news/58971 §5.3: a cache of bounded size keeps the positions
// that attention has looked at most, and the most recent ones; "KV Cache 的显存账本：PagedAttention 与
// 连续批处理" §七: the first tokens stay whatever their weight.  Per (sequence, KV head), with n slots in
// use and a budget b < n: the protected slots and the best-scored others, b in all, stay.
//
// Compaction fills holes instead of closing ranks: kept slots below b stay where they are, and the i-th
// evicted slot below b (a hole) receives the i-th kept slot at or past b (a mover).  Attention does not
// depend on the order of the slots, so this is enough; it moves at most n - b rows per head where an
// order-preserving compaction moves nearly b (64 new tokens over a budget of 2048: 64 rows, not ~2000),
// and since every source is at or past b and every destination below it, no row is read after it has
// been overwritten, in place or not.  The heads of a token part company: slot j of head h holds the
// token at position token_pos[s][h][j].
//
// Design (one launch).  A cluster of C CTAs takes one (sequence, KV head); a CTA owns a run of slots
// and a warp a run of those, in order, so that ranks in slot order need only ballots and prefix sums.
//  1. newest position (maximum over the slots), needed to know which slots are recent;
//  2. keys: the score as an order-preserving 32-bit integer (protected: all ones, NaN: 0) in shared
//     memory, as many as fit; the others are made again from the scores at each pass;
//  3. the b-th largest key by radix selection, digits of 11, 11 and 10 bits: shared-memory histograms,
//     summed over the cluster through distributed shared memory;
//  4. slots equal to it are kept in slot order up to the budget (ranks only when some must go);
//  5. holes and movers are counted and ranked; their physical slots go to two lists in the workspace;
//     the kept scores and positions are written, and those past the new length;
//  6. the cluster moves the listed rows, 16 bytes per thread and access.
// Everything is integer comparison and counting in a fixed order: the result does not depend on timing.

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvMaxCluster = 8;  // the portable cluster size
// slots per CTA that a cluster is made larger for
#ifndef PA_EVICT_SPAN
#define PA_EVICT_SPAN 4096
#endif
constexpr size_t kEvMaxKeyBytes = 192 * 1024;  // dynamic shared memory for keys, beside the histograms

struct EvictParams {
  int B, H, num_blocks, max_blocks, max_ctx, stride, budget, anchors, recent;
  int cluster, key_cap, max_moves;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* scores_in;
  float* scores_out;
  const int32_t* pos_in;  // or null: slot j holds position j
  int32_t* pos_out;
  int2* holes;   // [B * H][max_moves] (physical slot or -1, slot)
  int4* movers;  // [B * H][max_moves] (physical slot or -1, score bits, position, 0)
  // a (slot, head) row in 16-byte units: K codes, V codes, K parameters, V parameters (INT4)
  uint4* part[4];
  int units[4], total_units;
  float* token_scales;  // per-token K scales, or null
  int32_t* err;
};

__device__ __forceinline__ void cluster_sync_all(int cluster) {
  if (cluster > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
// The int at this CTA's shared address `p`, in CTA `rank` of the cluster.
__device__ __forceinline__ int remote_ld(const int* p, int rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return static_cast<int>(v);
}

__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 ranks as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix over the warps of a CTA and the CTAs before it of v (one value per warp, valid in
// lane 0); `total` receives the cluster's sum.  `tot` and `sh` are this quantity's own shared words.
__device__ __forceinline__ int warp_prefix(int v, int* sh, int* tot, int warp, int lane, int rank, int cluster,
                                           int* total) {
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kEvWarps; ++w) {
    before += w < warp ? sh[w] : 0;
    all += sh[w];
  }
  if (cluster > 1) {
    if (threadIdx.x == 0) *tot = all;
    cluster_sync_all(cluster);
    int sum = 0;
    for (int c = 0; c < cluster; ++c) {
      const int x = remote_ld(tot, c);
      before += c < rank ? x : 0;
      sum += x;
    }
    all = sum;
  }
  *total = all;
  return before;
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kEvBins], above_warp[kEvWarps];
  __shared__ int sh_warp[3][kEvWarps];
  __shared__ int sh_tot[3];
  __shared__ int sh_max, sh_digit, sh_rest, sh_count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.cluster, rank = C > 1 ? cluster_rank() : 0;
  const int pair = blockIdx.x / C, s = pair / p.H, h = pair - s * p.H;
  grid_dep_wait();  // the previous kernel of the stream may still be writing any input
  const int n = p.context_lens[s];
  if (n < 0 || n > p.max_ctx || static_cast<long long>(n) > static_cast<long long>(p.max_blocks) * PA_BLOCK_SIZE) {
    if (h == 0 && rank == 0 && tid == 0) set_error(p.err, PA_EFLAG_CTX_OVERFLOW);
    return;  // the whole cluster leaves together
  }
  const int left = min(n, p.budget);
  const size_t row = static_cast<size_t>(pair) * p.stride;
  const float* sc = p.scores_in + row;
  const int32_t* po = p.pos_in ? p.pos_in + row : nullptr;

  // this CTA's run of slots [a, b), this warp's [wa, wb), both multiples of 32 long but at the end
  const int per = ((n + C - 1) / C + 31) & ~31, a = min(n, rank * per), b = min(n, a + per);
  const int wper = ((per + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int wa = min(b, a + warp * wper), wb = min(b, wa + wper);

  // ---- 1. the newest position ----
  int newest = n - 1;
  if (po) {
    int mx = -1;
#pragma unroll 4
    for (int j = wa + lane; j < wb; j += 32) mx = max(mx, po[j]);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (tid == 0) sh_max = -1;
    __syncthreads();
    if (lane == 0) atomicMax(&sh_max, mx);
    cluster_sync_all(C);
    newest = sh_max;
    for (int c = 0; c < C && C > 1; ++c) newest = max(newest, remote_ld(&sh_max, c));
  }
  const long long recent_from = static_cast<long long>(newest) - p.recent;  // positions past it are recent

  auto make_key = [&](int j) -> uint32_t {
    const int pos = po ? po[j] : j;
    return (pos < p.anchors || pos > recent_from) ? 0xFFFFFFFFu : score_key(sc[j]);
  };
  auto key = [&](int j) -> uint32_t { return j - a < p.key_cap ? keys[j - a] : make_key(j); };

  uint32_t thr = 0;  // keys above it are kept, `need` of those equal to it too
  int need = n, eq_base = 0;
  bool rank_eq = false;
  if (n > p.budget) {
    // ---- 2. keys ----
#pragma unroll 4
    for (int j = wa + lane; j < wb; j += 32)
      if (j - a < p.key_cap) keys[j - a] = make_key(j);

    // ---- 3. the budget-th largest key ----
    uint32_t mask = 0;
    int rest = p.budget;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t k = j < wb ? key(j) : 0u;
        const bool in = j < wb && (k & mask) == thr;
        const uint32_t d = (k >> shift) & ((1u << bits) - 1u);
        // a warp whose keys share the digit adds once (scores that are all zero, or protected slots)
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (who == 0) continue;
        const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !in || d == d0)) {
          if (lane == 0) atomicAdd(&hist[d0], __popc(who));
        } else if (in) {
          atomicAdd(&hist[d], 1);
        }
      }
      cluster_sync_all(C);
      // thread i sums bins 4i .. 4i + 3 over the cluster, then the bins above them over the CTA
      int cnt[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cnt[e] = 0;
        if (C > 1) {
          for (int c = 0; c < C; ++c) cnt[e] += remote_ld(&hist[4 * tid + e], c);
        } else {
          cnt[e] = hist[4 * tid + e];
        }
      }
      const int mine = cnt[0] + cnt[1] + cnt[2] + cnt[3];
      int suffix = mine;  // over this thread and the lanes above it
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_down_sync(0xffffffffu, suffix, off);
        if (lane + off < 32) suffix += v;
      }
      if (lane == 0) above_warp[warp] = suffix;
      __syncthreads();
      int above = suffix - mine;
      for (int w = warp + 1; w < kEvWarps; ++w) above += above_warp[w];
#pragma unroll
      for (int e = 3; e >= 0; --e) {  // exactly one bin holds the rest-th largest
        if (above < rest && rest <= above + cnt[e]) {
          sh_digit = 4 * tid + e;
          sh_rest = rest - above;
          sh_count = cnt[e];
        }
        above += cnt[e];
      }
      cluster_sync_all(C);  // the digit is known, and no CTA still reads another's histogram
      thr |= static_cast<uint32_t>(sh_digit) << shift;
      mask |= ((1u << bits) - 1u) << shift;
      rest = sh_rest;
    }
    need = rest;
    rank_eq = sh_count > need;

    // ---- 4. ranks of the slots equal to the threshold, when not all of them stay ----
    if (rank_eq) {
      int cnt = 0, all;
      for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        cnt += __popc(__ballot_sync(0xffffffffu, j < wb && key(j) == thr));
      }
      eq_base = warp_prefix(cnt, sh_warp[0], &sh_tot[0], warp, lane, rank, C, &all);
    }
  }

  // ---- 5. holes and movers ----
  const unsigned below = (1u << lane) - 1u;
  int moves = 0, hole_base = 0, mover_base = 0;
  // kept slots of 32 at j0; `eq` counts the slots equal to the threshold before them
  auto keep_at = [&](int j0, int& eq) -> bool {
    const int j = j0 + lane;
    if (n <= p.budget) return j < wb;
    const uint32_t k = j < wb ? key(j) : 0u;
    const unsigned same = __ballot_sync(0xffffffffu, j < wb && k == thr);
    const bool keep = j < wb && (k > thr || (k == thr && (!rank_eq || eq + __popc(same & below) < need)));
    eq += __popc(same);
    return keep;
  };
  if (n > p.budget) {
    int hc = 0, mc = 0, eq = eq_base, all;
    for (int j0 = wa; j0 < wb; j0 += 32) {
      const bool keep = keep_at(j0, eq);
      const int j = j0 + lane;
      hc += __popc(__ballot_sync(0xffffffffu, j < wb && j < left && !keep));
      mc += __popc(__ballot_sync(0xffffffffu, j >= left && keep));
    }
    hole_base = warp_prefix(hc, sh_warp[1], &sh_tot[1], warp, lane, rank, C, &moves);
    mover_base = warp_prefix(mc, sh_warp[2], &sh_tot[2], warp, lane, rank, C, &all);
  }
  auto physical = [&](int j) -> int {
    const int e = p.block_tables[static_cast<size_t>(s) * p.max_blocks + j / PA_BLOCK_SIZE];
    if (e < 0 || e >= p.num_blocks) {
      set_error(p.err, PA_EFLAG_BAD_BLOCK_ID);
      return -1;
    }
    return e * PA_BLOCK_SIZE + j % PA_BLOCK_SIZE;
  };
  int2* holes = p.holes + static_cast<size_t>(pair) * p.max_moves;
  int4* movers = p.movers + static_cast<size_t>(pair) * p.max_moves;
  {
    int eq = eq_base;
    for (int j0 = wa; j0 < wb; j0 += 32) {
      const bool keep = keep_at(j0, eq);
      const int j = j0 + lane;
      const bool hole = j < wb && j < left && !keep, mover = j >= left && keep;
      const unsigned hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
      if (j < wb) {
        const float x = sc[j];
        const int pos = po ? po[j] : j;
        if (hole) holes[hole_base + __popc(hm & below)] = make_int2(physical(j), j);
        if (mover) movers[mover_base + __popc(mm & below)] = make_int4(physical(j), __float_as_int(x), pos, 0);
        if (j >= left) {
          p.scores_out[row + j] = 0.f;
          p.pos_out[row + j] = newest + 1 + (j - left);
        } else if (keep) {
          p.scores_out[row + j] = x;
          p.pos_out[row + j] = pos;
        }
      }
      hole_base += __popc(hm);
      mover_base += __popc(mm);
    }
  }
  for (int j = n + rank * kEvThreads + tid; j < p.stride; j += C * kEvThreads) {
    p.scores_out[row + j] = 0.f;
    p.pos_out[row + j] = newest + 1 + (j - left);
  }

  // ---- 6. move ----
  __threadfence();
  // every list entry of this (sequence, head) is written, and no CTA still reads another's shared memory
  cluster_sync_all(C);
  if (n <= p.budget) return;
  for (int i = rank * kEvThreads + tid; i < moves; i += C * kEvThreads) {
    const int2 d = holes[i];
    const int4 m = movers[i];
    p.scores_out[row + d.y] = __int_as_float(m.y);
    p.pos_out[row + d.y] = m.z;
    if (p.token_scales && d.x >= 0 && m.x >= 0)
      p.token_scales[static_cast<size_t>(d.x) * p.H + h] = p.token_scales[static_cast<size_t>(m.x) * p.H + h];
  }
  const long long all_units = static_cast<long long>(moves) * p.total_units;
  constexpr int kDepth = 4;  // loads in flight per thread
  for (long long u0 = static_cast<long long>(rank) * kEvThreads + tid; u0 < all_units;
       u0 += static_cast<long long>(C) * kEvThreads * kDepth) {
    uint4 v[kDepth];
    uint4* dst[kDepth];
#pragma unroll
    for (int e = 0; e < kDepth; ++e) {
      const long long u = u0 + static_cast<long long>(e) * C * kEvThreads;
      dst[e] = nullptr;
      if (u < all_units) {
        const int i = static_cast<int>(u / p.total_units);
        int r = static_cast<int>(u - static_cast<long long>(i) * p.total_units), t = 0;
        while (r >= p.units[t]) r -= p.units[t++];
        const int to = holes[i].x, from = movers[i].x;
        if (to >= 0 && from >= 0) {
          dst[e] = p.part[t] + (static_cast<size_t>(to) * p.H + h) * p.units[t] + r;
          v[e] = p.part[t][(static_cast<size_t>(from) * p.H + h) * p.units[t] + r];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kDepth; ++e)
      if (dst[e]) *dst[e] = v[e];
  }
}

int evict_max_moves(int max_ctx, int budget) { return std::max(0, std::min(budget, max_ctx - budget)); }

bool evict_layout(const pa_cache_desc* d, int max_ctx, int budget, size_t* movers_off, size_t* total) {
  if (validate_desc(d) != PA_OK || max_ctx < 0 || max_ctx > 0x7FFFFF00 || budget < 1) return false;
  const size_t rows = static_cast<size_t>(d->num_seqs) * d->num_kv_heads * evict_max_moves(max_ctx, budget);
  *movers_off = (rows * sizeof(int2) + 255) / 256 * 256;
  *total = *movers_off + rows * sizeof(int4) + 256;
  return true;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_cache_evict_workspace_size(const pa_cache_desc* desc, int max_context_len, int budget) {
  size_t off = 0, total = 0;
  return pa::evict_layout(desc, max_context_len, budget, &off, &total) ? total : 0;
}

extern "C" pa_status pa_cache_evict(const pa_cache_desc* desc, void* k_cache, void* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens, int max_context_len,
                                    const float* scores_in, float* scores_out, const int32_t* pos_in,
                                    int32_t* pos_out, int stride, int budget, int num_anchor, int num_recent,
                                    void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  const pa_status st = pa::validate_desc(desc);
  if (st != PA_OK) return st;
  if (desc->sliding_window > 0) return PA_ERR_UNSUPPORTED;  // a window counts slots in order of position
  size_t movers_off = 0, total = 0;
  if (!pa::evict_layout(desc, max_context_len, budget, &movers_off, &total)) return PA_ERR_INVALID_ARG;
  if (stride < max_context_len || num_recent < 0 || num_anchor < desc->num_sink ||
      static_cast<long long>(num_anchor) + num_recent > budget)
    return PA_ERR_INVALID_ARG;
  if (desc->num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !scores_in || !scores_out || !pos_out || !workspace)
    return PA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15u) ||
      ((reinterpret_cast<uintptr_t>(scores_in) | reinterpret_cast<uintptr_t>(scores_out) |
        reinterpret_cast<uintptr_t>(pos_in) | reinterpret_cast<uintptr_t>(pos_out)) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < total) return PA_ERR_WORKSPACE_TOO_SMALL;

  pa::EvictParams p = {};
  p.B = desc->num_seqs;
  p.H = desc->num_kv_heads;
  p.num_blocks = desc->num_blocks;
  p.max_blocks = desc->max_blocks_per_seq;
  p.max_ctx = max_context_len;
  p.stride = stride;
  p.budget = budget;
  p.anchors = num_anchor;
  p.recent = num_recent;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.scores_in = scores_in;
  p.scores_out = scores_out;
  p.pos_in = pos_in;
  p.pos_out = pos_out;
  p.max_moves = pa::evict_max_moves(max_context_len, budget);
  p.holes = static_cast<int2*>(workspace);
  p.movers = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + movers_off);
  p.err = err_flag;
  const bool int4 = pa::is_int4(desc);
  const int row16 = static_cast<int>((int4 ? pa::int4_code_row_bytes(desc)
                                           : static_cast<size_t>(desc->head_dim) * pa::dtype_bytes(desc->k_dtype)) / 16);
  p.part[0] = static_cast<uint4*>(k_cache);
  p.part[1] = static_cast<uint4*>(v_cache);
  p.units[0] = p.units[1] = row16;
  if (int4) {  // one 16-byte row of parameters per (slot, head)
    p.part[2] = p.part[0] + pa::int4_params_offset(desc) / 16;
    p.part[3] = p.part[1] + pa::int4_params_offset(desc) / 16;
    p.units[2] = p.units[3] = 1;
  }
  p.total_units = p.units[0] + p.units[1] + p.units[2] + p.units[3];
  if (pa::has_token_scales(desc))
    p.token_scales = reinterpret_cast<float*>(static_cast<uint8_t*>(k_cache) + pa::token_scales_offset(desc));

  // CTAs per (sequence, head): enough that each has a few thousand slots
  int C = 1;
  while (C < pa::kEvMaxCluster && (max_context_len + C - 1) / C > PA_EVICT_SPAN) C *= 2;
  const long long pairs = static_cast<long long>(p.B) * p.H;
  if (pairs * C > 0x7FFFFFFFLL) return PA_ERR_UNSUPPORTED;
  p.cluster = C;
  const size_t span = (static_cast<size_t>((max_context_len + C - 1) / C) + 31) / 32 * 32;
  const size_t key_bytes = std::min(pa::kEvMaxKeyBytes, std::max<size_t>(span, 32) * 4);
  p.key_cap = static_cast<int>(key_bytes / 4);
  if (!pa::ensure_dynamic_smem(reinterpret_cast<const void*>(pa::evict_kernel), key_bytes)) return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * C));
  cfg.blockDim = dim3(pa::kEvThreads);
  cfg.dynamicSmemBytes = key_bytes;
  cfg.stream = pa::as_stream(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pa::evict_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
