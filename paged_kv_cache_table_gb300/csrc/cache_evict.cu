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
// Design.  A cluster of C CTAs takes one (sequence, KV head); a CTA owns a run of slots and a warp a run
// of those, in order, so that ranks in slot order need only ballots and prefix sums.
//  1. newest position (maximum over the slots), needed to know which slots are recent;
//  2. keys: the score as an order-preserving 32-bit integer (protected: all ones, NaN: 0), kept in shared
//     memory, as many as fit; the others are made again at each pass;
//  3. the b-th largest key by radix selection, digits of 12, 10 and 10 bits: shared-memory histograms,
//     summed over the cluster through distributed shared memory, each CTA taking its share of the bins
//     (12 bits: the sign, the exponent and three bits of the mantissa spread accumulated weights, which
//     range over many octaves, over enough bins that the lanes of a warp seldom meet in one).  After the
//     first digit the keys that share it, a few of a hundred, are put in a list for the other two;
//  4. slots equal to it are kept in slot order up to the budget (ranks only when some must go); one word
//     of kept bits per 32 slots;
//  5. holes and movers are counted and ranked, one lane per word, and their physical slots go to two lists
//     (in the workspace, or with few slots in shared memory over the keys), one lane per slot, so that a
//     store writes consecutive entries; scores and positions of kept slots are copied (unless in place);
//  6. movers' scores and positions go to the holes, and the listed rows move, 16 bytes per lane: a lane's
//     part of a row (which tensor, which 16 bytes) is the same for every row, and a warp has several rows
//     in flight.  Where there are few CTAs and many rows, a second launch with as many CTAs as the GPU
//     holds moves them.
// Everything is integer comparison and counting in a fixed order: the result does not depend on timing.
//
// Measured, d 128 bf16, 8 KV heads: 64 sequences from 2112 slots to 2048 21.5 us (50 MB; bound by the CTA's
// dependent steps, not by bytes), 16 of 500..8192 to 1024 30.5 us, 4 of 131072 to 32768 188 us (882 MB:
// 130 us for the rows at 6.2 TB/s, 50 for the selection).

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kEvBins = 4096;
constexpr int kEvList = 1024;     // keys of the list after the first digit; more: all keys are gone over again
constexpr int kEvMaxCluster = 8;  // the portable cluster size
constexpr int kEvSmall = 4096;     // slots up to which a CTA keeps scores and positions in shared memory
constexpr int kEvMaxKeys = 40960;  // keys kept in shared memory otherwise
constexpr int kEvMaxContext = 1 << 21;  // so that every word of kept bits has its place in shared memory too

struct EvictParams {
  int B, H, num_blocks, max_blocks, max_ctx, stride, budget, anchors, recent;
  int cluster, cap, max_moves;
  int rows_apart;  // a second launch moves the rows
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* scores_in;
  float* scores_out;
  const int32_t* pos_in;  // or null: slot j holds position j
  int32_t* pos_out;
  int2* holes;   // [B * H][max_moves] (physical slot or -1, slot)
  int2* movers;  // the same
  int* counts;   // [B * H] rows to move (when a second launch moves them)
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
__device__ __forceinline__ void remote_st(int* p, int rank, int v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 ranks as +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Bits 0 .. n - 1, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); }

// Bins are scanned by the thread that holds kEvRun consecutive ones; bin b lies at (b % kEvRun) *
// kEvPitch + b / kEvRun, so that neither this scan (threads at consecutive words) nor neighbouring
// bins hit by a warp's atomics (kEvPitch is odd) meet in a bank.
constexpr int kEvRun = 16, kEvRuns = kEvBins / kEvRun, kEvPitch = kEvRuns + 1;
__device__ __forceinline__ int bin_at(int b) { return (b & (kEvRun - 1)) * kEvPitch + (b / kEvRun); }

template <int T>
struct EvictShared {
  alignas(16) int hist[kEvRun * kEvPitch];
  int runs[kEvRuns];  // keys in this CTA's share of the runs of bins, over the cluster
  uint32_t list[kEvList];
  int above_warp[T / 32];
  int warp[3][T / 32];
  int tot[3];
  int slice[kEvMaxCluster];  // keys counted in each CTA's share of the bins
  int max, run, above, digit, rest, count, listed;
};

// Sum over the warps of a CTA of v[w], and of those before (or, `after`, behind) this one; every lane.
template <int W>
__device__ __forceinline__ int warps_sum(const int* v, int* part, bool after) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = lane < W ? v[lane] : 0;
  *part = __reduce_add_sync(0xffffffffu, (after ? lane > warp : lane < warp) ? x : 0);
  return __reduce_add_sync(0xffffffffu, x);
}

// Exclusive prefix, over the warps of a CTA and the CTAs before it, of N quantities that lane 0 of each
// warp holds; total[] receives the cluster's sums.  sh.warp[q0 ..] and sh.tot[q0 ..] are theirs alone.
template <int T, int N>
__device__ __forceinline__ void warp_prefix(EvictShared<T>& sh, int q0, const int (&v)[N], int (&before)[N],
                                            int (&total)[N], int rank, int cluster) {
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int q = 0; q < N; ++q) sh.warp[q0 + q][warp] = v[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < N; ++q) total[q] = warps_sum<T / 32>(sh.warp[q0 + q], &before[q], false);
  if (cluster > 1) {
    if (threadIdx.x == 0) {
#pragma unroll
      for (int q = 0; q < N; ++q) sh.tot[q0 + q] = total[q];
    }
    cluster_sync_all(cluster);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      total[q] = 0;
      for (int c = 0; c < cluster; ++c) {
        const int x = remote_ld(&sh.tot[q0 + q], c);
        before[q] += c < rank ? x : 0;
        total[q] += x;
      }
    }
  }
}

// Rows of the lists of one (sequence, head) that warp `w` of `nw` moves: 16 bytes per lane and row, four
// rows in flight.  (Loading 32 list entries at once, one per lane, and shuffling them out was slower: 46
// against 38 us for the 128 pairs of up to 8192 slots.)
__device__ __forceinline__ void move_rows(const EvictParams& p, int h, const int2* holes, const int2* movers,
                                          int moves, int w, int nw) {
  const int lane = threadIdx.x & 31;
  // a lane's 16 bytes of every row it takes: tensor t, unit r of row `sub` of the warp's `group` rows
  const int group = 32 / p.total_units, sub = lane / p.total_units;
  int r = lane - sub * p.total_units, t = 0;
  while (t < 3 && r >= p.units[t]) r -= p.units[t++];
  uint4* base = p.part[t] + static_cast<size_t>(h) * p.units[t] + r;
  const size_t step = static_cast<size_t>(p.H) * p.units[t];  // from one slot's row of this head to the next's
  constexpr int kDepth = 4;
  const int stride_rows = nw * group;
  for (int i0 = w * group + sub; i0 < moves; i0 += stride_rows * kDepth) {
    uint4 v[kDepth];
    int to[kDepth], from[kDepth];
#pragma unroll
    for (int e = 0; e < kDepth; ++e) {
      const int i = i0 + e * stride_rows;
      const bool on = sub < group && i < moves;
      to[e] = on ? holes[i].x : -1;
      from[e] = on ? movers[i].x : -1;
    }
#pragma unroll
    for (int e = 0; e < kDepth; ++e)  // (negative: a table entry outside the pool)
      if (to[e] >= 0 && from[e] >= 0) v[e] = base[static_cast<size_t>(from[e]) * step];
#pragma unroll
    for (int e = 0; e < kDepth; ++e)
      if (to[e] >= 0 && from[e] >= 0) base[static_cast<size_t>(to[e]) * step] = v[e];
  }
  if (p.token_scales)
    for (int i = w * 32 + lane; i < moves; i += nw * 32) {
      const int to = holes[i].x, from = movers[i].x;
      if (to >= 0 && from >= 0)
        p.token_scales[static_cast<size_t>(to) * p.H + h] = p.token_scales[static_cast<size_t>(from) * p.H + h];
    }
}

// SMALL: one CTA per (sequence, head) with at most kEvSmall slots, which keeps scores and positions in
// shared memory, and later the lists.
template <int T, bool SMALL>
__global__ void __launch_bounds__(T, 1024 / T) evict_kernel(const EvictParams p) {
  constexpr int W = T / 32;  // warps
  // keys [cap] (SMALL: first the scores), SMALL: positions [cap], one word of kept slots per 32
  extern __shared__ uint32_t dyn[];
  __shared__ EvictShared<T> sh;
  uint32_t* kept = dyn + (SMALL ? 2 : 1) * p.cap;
  int* own_pos = reinterpret_cast<int*>(dyn + p.cap);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = SMALL ? 1 : p.cluster, rank = C > 1 ? cluster_rank() : 0;
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
  float* sc_out = p.scores_out + row;
  int32_t* po_out = p.pos_out + row;
  const int32_t* table = p.block_tables + static_cast<size_t>(s) * p.max_blocks;

  // this CTA's run of slots [a, b), this warp's [wa, wb), both multiples of 32 long but at the end
  const int per = ((n + C - 1) / C + 31) & ~31, a = min(n, rank * per), b = min(n, a + per);
  const int wper = ((per + W - 1) / W + 31) & ~31;
  const int wa = min(b, a + warp * wper), wb = min(b, wa + wper);

  // Scores and positions of slots below the new length, unless in place; holes among them are written
  // again in step 6.
  const bool sc_apart = sc_out != sc, po_apart = po_out != po;
  auto copy_out = [&](int j, float x, int pos) {
    if (j >= left) return;
    if (sc_apart) sc_out[j] = x;
    if (po_apart) po_out[j] = pos;
  };

  // ---- 1. the newest position (and, SMALL, the slots' scores and positions) ----
  int newest = n - 1;
  if (SMALL || po) {
    int mx = -1;
#pragma unroll 4
    for (int j = wa + lane; j < wb; j += 32) {
      const int x = po ? po[j] : j;
      if constexpr (SMALL) {
        const float y = sc[j];
        dyn[j - a] = __float_as_uint(y);
        own_pos[j - a] = x;
        copy_out(j, y, x);
      }
      mx = max(mx, x);
    }
    if (po) {
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (tid == 0) sh.max = -1;
      __syncthreads();
      if (lane == 0) atomicMax(&sh.max, mx);
      cluster_sync_all(C);
      newest = sh.max;
      for (int c = 0; c < C && C > 1; ++c) newest = max(newest, remote_ld(&sh.max, c));
    }
  }
  const int recent_from = newest - p.recent;  // positions past it are recent (newest >= -1: no overflow)

  auto key_of = [&](float x, int pos) -> uint32_t {
    return (pos < p.anchors || pos > recent_from) ? 0xFFFFFFFFu : score_key(x);
  };
  const bool full = SMALL || per <= p.cap;  // every key of this CTA is in shared memory
  auto key = [&](int j) -> uint32_t {
    return full || j - a < p.cap ? dyn[j - a] : key_of(sc[j], po ? po[j] : j);
  };

  // The lists.  SMALL: where the keys and positions were (at most n / 2 entries each, and nothing reads
  // keys or positions after the kept words are known), unless a second launch reads them.
  int2* holes = p.holes + static_cast<size_t>(pair) * p.max_moves;
  int2* movers = p.movers + static_cast<size_t>(pair) * p.max_moves;
  if (SMALL && !p.rows_apart) {
    holes = reinterpret_cast<int2*>(dyn);
    movers = reinterpret_cast<int2*>(own_pos);
  }

  uint32_t thr = 0;  // keys above it are kept, `need` of those equal to it too
  int need = n, moves = 0;
  if (n > p.budget) {
    // ---- 2, 3. the budget-th largest key ----
    uint32_t mask = 0;
    int rest = p.budget;
    bool listed = false;  // sh.list holds this CTA's keys that share the digits so far
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 20 : (pass == 1 ? 10 : 0), bits = pass == 0 ? 12 : 10;
      const int bins = 1 << bits;
      for (int i = tid; i < kEvRun * kEvPitch / 4; i += T) reinterpret_cast<int4*>(sh.hist)[i] = make_int4(0, 0, 0, 0);
      if (tid < kEvRuns) sh.runs[tid] = 0;
      if (tid == 0) sh.run = -1;
      __syncthreads();
      auto count = [&](bool in, uint32_t k) {  // every lane of the warp takes part
        const uint32_t d = (k >> shift) & static_cast<uint32_t>(bins - 1);
        // a warp whose keys share the digit adds once (scores that are all zero, recent slots)
        const uint32_t d0 = __shfl_sync(0xffffffffu, d, 0);
        if (__all_sync(0xffffffffu, in && d == d0)) {
          if (lane == 0) atomicAdd(&sh.hist[bin_at(d)], 32);
        } else if (in) {
          atomicAdd(&sh.hist[bin_at(d)], 1);
        }
      };
      if (pass == 0) {
        constexpr int kAhead = SMALL ? 2 : 8;  // slots per lane that are loaded together
        for (int g0 = wa; g0 < wb; g0 += 32 * kAhead) {
          uint32_t k[kAhead];
          float x[kAhead];
          int pos[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int j = g0 + 32 * i + lane;
            x[i] = j >= wb ? 0.f : (SMALL ? __uint_as_float(dyn[j - a]) : sc[j]);
            pos[i] = j >= wb ? 0 : (SMALL ? own_pos[j - a] : (po ? po[j] : j));
          }
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int j = g0 + 32 * i + lane;
            k[i] = key_of(x[i], pos[i]);
            if (!SMALL && j < wb) copy_out(j, x[i], pos[i]);
          }
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int j = g0 + 32 * i + lane;
            if (j < wb && (full || j - a < p.cap)) dyn[j - a] = k[i];
            count(j < wb, k[i]);
          }
        }
      } else if (listed) {
        for (int i0 = warp * 32; i0 < sh.listed; i0 += T) {
          const uint32_t k = i0 + lane < sh.listed ? sh.list[i0 + lane] : 0u;
          count(i0 + lane < sh.listed && (k & mask) == thr, k);
        }
      } else {
        for (int j0 = wa; j0 < wb; j0 += 32) {
          const uint32_t k = j0 + lane < wb ? key(j0 + lane) : 0u;
          count(j0 + lane < wb && (k & mask) == thr, k);
        }
      }
      cluster_sync_all(C);
      // this CTA's share of the runs of bins, nt of them, summed over the cluster: one thread per (CTA, run)
      const int nt = bins / kEvRun / C, first_run = rank * nt;
      int mine = 0, above, own;
      if (tid < nt * C) {
        const int c = tid / nt, run = tid - c * nt;
#pragma unroll
        for (int e = 0; e < kEvRun; ++e) {
          const int* at = &sh.hist[e * kEvPitch + first_run + run];
          mine += C > 1 ? remote_ld(at, c) : *at;
        }
        if (C > 1) atomicAdd(&sh.runs[run], mine);
      }
      if (C > 1) {
        __syncthreads();
        mine = tid < nt ? sh.runs[tid] : 0;
      }
      int suffix = mine;  // over this thread and the lanes above it
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_down_sync(0xffffffffu, suffix, off);
        if (lane + off < 32) suffix += v;
      }
      if (lane == 0) sh.above_warp[warp] = suffix;
      if (tid == 0 && pass == 0) sh.listed = 0;
      __syncthreads();
      own = warps_sum<W>(sh.above_warp, &above, true);
      above += suffix - mine;
      if (C > 1) {  // the shares above this CTA's
        if (tid < C) remote_st(&sh.slice[rank], tid, own);
        cluster_sync_all(C);
        for (int c = rank + 1; c < C; ++c) above += sh.slice[c];
      }
      if (above < rest && rest <= above + mine) {  // one thread of the cluster: the rest-th largest is in its run
        sh.run = first_run + tid;
        sh.above = above;
      }
      __syncthreads();
      if (warp == 0 && sh.run >= 0) {  // its bin: one lane each
        int cnt = 0;
        if (lane < kEvRun)
          for (int c = 0; c < C; ++c) {
            const int* at = &sh.hist[lane * kEvPitch + sh.run];
            cnt += C > 1 ? remote_ld(at, c) : *at;
          }
        int up = cnt;
#pragma unroll
        for (int off = 1; off < kEvRun; off <<= 1) {
          const int v = __shfl_down_sync(0xffffffffu, up, off);
          if (lane + off < 32) up += v;
        }
        up += sh.above - cnt;  // keys in the bins above
        if (up < rest && rest <= up + cnt) {
          for (int c = 0; c < C; ++c) {
            if (C > 1) {
              remote_st(&sh.digit, c, sh.run * kEvRun + lane);
              remote_st(&sh.rest, c, rest - up);
              remote_st(&sh.count, c, cnt);
            } else {
              sh.digit = sh.run * kEvRun + lane;
              sh.rest = rest - up;
              sh.count = cnt;
            }
          }
        }
      }
      cluster_sync_all(C);  // the digit is known, and no CTA still reads another's histogram
      const int own_count = sh.hist[bin_at(sh.digit)];  // this CTA's keys that share it
      thr |= static_cast<uint32_t>(sh.digit) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      rest = sh.rest;
      if (pass == 0 && own_count <= kEvList) {
        listed = true;
        for (int g0 = wa; g0 < wb; g0 += 128) {
          uint32_t k[4], m[4];
          int all = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = g0 + 32 * i + lane;
            k[i] = j < wb ? key(j) : 0u;
            m[i] = __ballot_sync(0xffffffffu, j < wb && (k[i] & mask) == thr);
            all += __popc(m[i]);
          }
          if (all == 0) continue;
          int at = lane == 0 ? atomicAdd(&sh.listed, all) : 0;
          at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((m[i] >> lane) & 1u) sh.list[at + __popc(m[i] & low_bits(lane))] = k[i];
            at += __popc(m[i]);
          }
        }
      }
      __syncthreads();  // the list is complete, and the histogram may be cleared
    }
    need = rest;

    // ---- 4. the kept slots ----
    uint32_t* words = kept + ((wa - a) >> 5);
    if (sh.count == need) {  // every slot equal to the threshold stays
      for (int g0 = wa; g0 < wb; g0 += 128) {
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = g0 + 32 * i + lane;
          m[i] = __ballot_sync(0xffffffffu, j < wb && key(j) >= thr);
        }
        if (lane < 4 && g0 + 32 * lane < wb)
          words[((g0 - wa) >> 5) + lane] = lane == 0 ? m[0] : (lane == 1 ? m[1] : (lane == 2 ? m[2] : m[3]));
      }
    } else {
      int cnt[1] = {0}, before[1], all[1];
      for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        cnt[0] += __popc(__ballot_sync(0xffffffffu, j < wb && key(j) == thr));
      }
      warp_prefix<T, 1>(sh, 0, cnt, before, all, rank, C);
      int eq = before[0];  // slots equal to the threshold so far
      for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t k = j < wb ? key(j) : 0u;
        const bool same = j < wb && k == thr;
        const uint32_t em = __ballot_sync(0xffffffffu, same);
        const uint32_t m = __ballot_sync(
            0xffffffffu, j < wb && (k > thr || (same && eq + __popc(em & low_bits(lane)) < need)));
        if (lane == 0) words[(j0 - wa) >> 5] = m;
        eq += __popc(em);
      }
    }
    __syncwarp();

    // ---- 5. holes and movers: counted, then ranked and listed, one lane per word ----
    const int nw = (wb - wa + 31) >> 5;
    int cnt[2] = {0, 0}, before[2], all[2];
    for (int i = lane; i < nw; i += 32) {
      const int j0 = wa + 32 * i;
      const uint32_t m = words[i], under = low_bits(left - j0);
      cnt[0] += __popc(low_bits(wb - j0) & under & ~m);
      cnt[1] += __popc(m & ~under);
    }
    cnt[0] = __reduce_add_sync(0xffffffffu, cnt[0]);
    cnt[1] = __reduce_add_sync(0xffffffffu, cnt[1]);
    warp_prefix<T, 2>(sh, 1, cnt, before, all, rank, C);
    moves = all[0];
    for (int i0 = 0; i0 < nw; i0 += 32) {
      const int j0 = wa + 32 * (i0 + lane);
      uint32_t hm = 0u, mm = 0u;
      if (i0 + lane < nw) {
        const uint32_t m = words[i0 + lane], under = low_bits(left - j0);
        hm = low_bits(wb - j0) & under & ~m;
        mm = m & ~under;
      }
      const int both = __popc(hm) | (__popc(mm) << 16);  // up to 1024 each over the warp
      int incl = both;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      const int sum = __shfl_sync(0xffffffffu, incl, 31);
      // the word's two blocks: first slot in the pool, or a negative number for an entry outside it
      int first[2] = {-64, -64};
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (((hm | mm) >> (16 * q)) & 0xFFFFu) {
          const int e = table[j0 / PA_BLOCK_SIZE + q];
          if (e >= 0 && e < p.num_blocks) first[q] = e * PA_BLOCK_SIZE;
          else set_error(p.err, PA_EFLAG_BAD_BLOCK_ID);
        }
      for (int i = 0; i < min(32, nw - i0); ++i) {
        const uint32_t hw = __shfl_sync(0xffffffffu, hm, i), mw = __shfl_sync(0xffffffffu, mm, i);
        const int at = __shfl_sync(0xffffffffu, incl - both, i);
        const int f0 = __shfl_sync(0xffffffffu, first[0], i), f1 = __shfl_sync(0xffffffffu, first[1], i);
        const int2 entry = make_int2((lane < 16 ? f0 : f1) + (lane & 15), wa + 32 * (i0 + i) + lane);
        if ((hw >> lane) & 1u) holes[before[0] + (at & 0xFFFF) + __popc(hw & low_bits(lane))] = entry;
        if ((mw >> lane) & 1u) movers[before[1] + (at >> 16) + __popc(mw & low_bits(lane))] = entry;
      }
      before[0] += sum & 0xFFFF;
      before[1] += sum >> 16;
    }
  }
  if (!SMALL && n <= p.budget)  // (else copied as the keys were made)
    for (int j = wa + lane; j < wb; j += 32) copy_out(j, sc[j], po ? po[j] : j);
  // Past the new length: at once when no mover is still to be read there.
  auto clear = [&] {
    for (int j = left + rank * T + tid; j < p.stride; j += C * T) {
      sc_out[j] = 0.f;
      po_out[j] = newest + 1 + (j - left);
    }
  };
  if (sc_apart && po_apart) clear();

  // ---- 6. move ----
  // every list entry of this (sequence, head) is written (the barrier orders the cluster's memory accesses),
  // and no CTA still reads another's shared memory
  cluster_sync_all(C);
  for (int i = rank * T + tid; i < moves; i += C * T) {
    const int to = holes[i].y, from = movers[i].y;
    sc_out[to] = sc[from];
    po_out[to] = po ? po[from] : from;
  }
  if (!p.rows_apart) {
    move_rows(p, h, holes, movers, moves, rank * W + warp, C * W);
  } else if (rank == 0 && tid == 0) {
    p.counts[pair] = moves;
  }
  if (!(sc_apart && po_apart)) {
    cluster_sync_all(C);  // in place, the movers' scores have been read before they are cleared
    clear();
  }
}

// The second launch: blockIdx.x of gridDim.x shares of the rows of (sequence, head) blockIdx.y.
__global__ void __launch_bounds__(256) evict_rows_kernel(const EvictParams p) {
  const int warp = threadIdx.x >> 5, share = blockIdx.x, shares = gridDim.x;
  const int pair = blockIdx.y + 65535 * blockIdx.z;
  if (pair >= p.B * p.H) return;
  grid_dep_wait();
  const int n = p.context_lens[pair / p.H];  // (a context out of range has no count)
  if (n <= p.budget || n > p.max_ctx || static_cast<long long>(n) > static_cast<long long>(p.max_blocks) * PA_BLOCK_SIZE)
    return;
  const size_t list = static_cast<size_t>(pair) * p.max_moves;
  move_rows(p, pair % p.H, p.holes + list, p.movers + list, min(p.counts[pair], p.max_moves), share * 8 + warp,
            shares * 8);
}

int evict_max_moves(int max_ctx, int budget) { return std::max(0, std::min(budget, max_ctx - budget)); }

bool evict_layout(const pa_cache_desc* d, int max_ctx, int budget, size_t* movers_off, size_t* total) {
  if (validate_desc(d) != PA_OK || max_ctx < 0 || budget < 1) return false;
  const size_t pairs = static_cast<size_t>(d->num_seqs) * d->num_kv_heads;
  const size_t rows = pairs * evict_max_moves(max_ctx, budget);
  *movers_off = (rows * sizeof(int2) + 255) / 256 * 256;
  *total = 2 * *movers_off + (pairs * sizeof(int) + 255) / 256 * 256 + 256;
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
  if (max_context_len > pa::kEvMaxContext) return PA_ERR_UNSUPPORTED;
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
  p.movers = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + movers_off);
  p.counts = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + 2 * movers_off);
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

  // CTAs per (sequence, head).  A cluster costs about 5 us in barriers, so one CTA takes 16384 slots alone:
  // 512 pairs of 2112 slots take 22 us with one CTA and 44 with two, 128 of 10000 25 us with one, 30 with
  // two and 29 with four, 32 of 10000 22, 22 and 20.  Above, a cluster grows to 8192 slots per CTA while the
  // CTAs about fit the GPU at once (two of 512 threads on an SM): 64 pairs of 32000 take 53, 40, 38 and 45 us
  // with one, two, four and eight, 128 of them 71, 66, 82 and 99; and while a CTA has more slots than shared
  // memory holds keys.
  const long long pairs = static_cast<long long>(p.B) * p.H, sms = std::max(1, pa::sm_count_current());
  int C = 1;
  while (max_context_len > 16384 && C < pa::kEvMaxCluster && max_context_len / C > 8192 &&
         (max_context_len / C > pa::kEvMaxKeys || pairs * 2 * C <= sms * 5 / 2))
    C *= 2;
  if (pairs * C > 0x7FFFFFFFLL) return PA_ERR_UNSUPPORTED;
  p.cluster = C;
  const size_t span = std::max<size_t>((static_cast<size_t>((max_context_len + C - 1) / C) + 31) / 32 * 32, 32);
  const bool small = C == 1 && span <= static_cast<size_t>(pa::kEvSmall);
  p.cap = static_cast<int>(small ? span : std::min<size_t>(span, pa::kEvMaxKeys));
  const size_t key_bytes = static_cast<size_t>(p.cap) * (small ? 8 : 4) + span / 8;
  // Where each CTA has an SM to itself it takes 1024 threads, from 2048 slots on: 16 pairs of 4096 slots take
  // 10.8 us with 1024 and 13.6 with 256, of 2048 both 9.2, of 1024 8.4 and 7.0; 128 of 10000 24.2 us and with
  // 512 24.6; 32 clusters of 32000 27.2 and 26.4.  In two waves they lose: 168 pairs of 1024 15.8 and 7.9.
  const bool wide = C == 1 && pairs <= sms && max_context_len > 2048;
  // A second launch for the rows when this one has too few warps to keep enough of them in flight.  Inline and
  // apart, 256 threads: 400 pairs from 2048 to 1024 47 and 53 us, from 4096 to 2048 108 and 97, 64 pairs from
  // 1000 to 900 8.4 and 9.6.  1024 threads: 8 pairs of 4096 slots 10.6 and 11.9 us for 64 moves, 12.0 and 11.5
  // for 256, 17.8 and 12.0 for 1024; 128 pairs 10.8 and 12.4, 12.4 and 14.0, 23.9 and 27.1.  512 threads lose
  // inline, and many moves go apart at any number of pairs: they may be all of one long sequence's.
  const int inline_moves = wide    ? (pairs * 3 > sms * 2 ? 1024 : 256)
                           : small ? (pairs < 3 * sms / 2 ? 256 : 1536)
                                   : 0;
  p.rows_apart = p.max_moves > inline_moves ? 1 : 0;
  auto kern = small ? (wide ? pa::evict_kernel<1024, true> : pa::evict_kernel<256, true>)
                    : (wide ? pa::evict_kernel<1024, false> : pa::evict_kernel<512, false>);
  if (!pa::ensure_dynamic_smem(reinterpret_cast<const void*>(kern), key_bytes)) return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * C));
  cfg.blockDim = dim3(wide ? 1024 : (small ? 256 : 512));
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
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return PA_ERR_CUDA;
  if (!p.rows_apart) return PA_OK;
  // the rows: eight CTAs per SM in all, none with less than a round of its warps' rows
  const long long round = 8LL * 4 * (32 / p.total_units);
  const long long shares = std::max(1LL, std::min(8 * sms / pairs, (p.max_moves + round - 1) / round));
  const dim3 rows(static_cast<unsigned>(shares), static_cast<unsigned>(std::min(pairs, 65535LL)),
                  static_cast<unsigned>((pairs + 65534) / 65535));
  return pa::launch_overlapped(pa::evict_rows_kernel, rows, dim3(256), 0, pa::as_stream(stream), p);
}
