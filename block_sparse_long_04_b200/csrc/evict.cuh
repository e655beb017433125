// Eviction from a paged key-value cache by accumulated attention weight.
//
// For one (sequence, kv head) row of `len` slots and a budget n < len, the n best slots
// stay: first the safe ones (ordinal >= seen - recent, or ordinal < sink), then by
// accumulated weight, descending; equal ones by slot, ascending. The kept slots end up
// in slots 0..n-1: a kept slot below n stays where it is, and the i-th evicted slot
// below n (ascending) takes the row of the i-th kept slot from the end. Sources lie at
// or above n and destinations below it, so the moves need no order among themselves, no
// second buffer, and touch only the rows that have to move (at a budget of half the
// cache a quarter of it, instead of nearly every kept row for a move that keeps the
// order). Attention does not depend on the order of the slots; the ordinals move along.
//
// Selection: a radix search for the n-th smallest key, 11 + 11 + 10 bits, where the key
// is the weight's order-preserving bit pattern, inverted (ascending key = descending
// weight), and 0 for a safe slot. One cluster of 1 to 8 CTAs per row: each CTA reads its
// part of the weights and ordinals once, keeps the keys in shared memory (if they fit),
// and adds the other CTAs' histograms through distributed shared memory. The last sweep
// writes the two lists of the moves. Everything is counted in integers: the result does
// not depend on the order of the atomics.
#pragma once
#include "common.cuh"
#include "rope_append.cuh"
#include "sm100.cuh"

namespace xattn {

constexpr int kEvThreads = 1024;
constexpr int kEvRounds = 4;           // quads of slots a thread has in flight
static_assert(kEvThreads == 1024, "32 warps: their sums are scanned by one warp");
constexpr int kEvBins = 2048;
constexpr int kEvMaxKeys = 40960;      // keys a CTA can hold in shared memory (160 KB)
constexpr int kEvMoveThreads = 256;
constexpr int kEvMoveUnroll = 4;       // moves of a thread in flight

struct EvictParams {
  CacheView cache;
  const int32_t* seen;       // [B] or null (lens)
  float* acc_out;
  int32_t* ord_out;
  int32_t* count;            // [rows] moves
  int32_t* hole;             // [rows, max_moves] pool rows the moves go to
  int32_t* mover;            // [rows, max_moves] pool rows they come from
  long long max_moves;
  int budget, recent, sink;
  int smem_keys;             // keys the launch has shared memory for
  int C, row_bytes_log2;
};

// ascending key = descending weight; every NaN ranks above +inf, -0 equals +0
__device__ __forceinline__ uint32_t evict_key(float w, int ordinal, int safe_from, int sink) {
  if (ordinal >= safe_from || ordinal < sink) return 0u;
  uint32_t u = __float_as_uint(w + 0.f);
  if (w != w) u = 0x7fc00000u;
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ~u;
}

__device__ __forceinline__ int2 ld_cluster_int2(const void* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(sm100::mapa_shared(p, rank)) : "memory");
  return v;
}

// Exclusive prefix of N ints over the block's threads (x, in place), and their totals.
template <int N>
__device__ __forceinline__ void block_prefix(int (&x)[N], int (&total)[N],
                                             int (*warp_sum)[kEvThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = x[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int up = __shfl_up_sync(0xffffffffu, s[i], o);
      if (lane >= o) s[i] += up;
    }
  __syncthreads();                      // warp_sum of an earlier call has been read
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) warp_sum[i][warp] = s[i];
  __syncthreads();
  // every warp scans the warps' sums for itself
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = warp_sum[i][lane];
    int w = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    total[i] = __shfl_sync(0xffffffffu, w, 31);
    x[i] = s[i] - x[i] + __shfl_sync(0xffffffffu, w - v, warp);
  }
}

__global__ void __launch_bounds__(kEvThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[2][kEvBins];
  __shared__ int warp_sum[kEvRounds][kEvThreads / 32];
  __shared__ __align__(8) int2 mine;        // this CTA's (below the cut, at the cut)
  // (digit, candidates before it, of these in this part, this part's with the digit)
  __shared__ int4 found;

  const int tid = threadIdx.x;
  grid_dependents_may_start();              // the moves wait for this grid's end themselves
  const int CL = gridDim.x;                 // the grid's x is one cluster
  const uint32_t rank = blockIdx.x;
  const int row = blockIdx.y, b = row / p.cache.Hkv, kvh = row - b * p.cache.Hkv;
  const int len = p.cache.length(b);
  const int n = p.budget;
  const bool copy_acc = p.acc_out != p.cache.acc, copy_ord = p.ord_out != p.cache.ordinal;
  if (tid == 0 && rank == 0 && !p.cache.length_valid(b)) raise_device_error(kErrInvalid);

  // this CTA's slots [lo, hi); parts are multiples of four slots, which never cross a page
  const int share = ((len + CL - 1) / CL + 3) & ~3;
  const int lo = min((int)rank * share, len), hi = min(lo + share, len);
  const int seen = p.seen != nullptr ? __ldg(p.seen + b) : len;
  const int safe_from = (long long)seen - p.recent < -2147483647ll ? -2147483647 : seen - p.recent;
  const bool cached = share <= p.smem_keys;

  // keys of slots s..s+3 (behind hi: the largest key, never wanted)
  auto keys_of = [&](int s, float4 w, int4 o) -> uint4 {
    uint4 k = make_uint4(~0u, ~0u, ~0u, ~0u);
    k.x = evict_key(w.x, o.x, safe_from, p.sink);
    if (s + 1 < hi) k.y = evict_key(w.y, o.y, safe_from, p.sink);
    if (s + 2 < hi) k.z = evict_key(w.z, o.z, safe_from, p.sink);
    if (s + 3 < hi) k.w = evict_key(w.w, o.w, safe_from, p.sink);
    return k;
  };
  auto load4 = [&](int s) -> uint4 {
    const long long at = p.cache.slot_index(b, kvh, s);
    if (at < 0) {
      raise_device_error(kErrInvalid);
      return make_uint4(~0u, ~0u, ~0u, ~0u);
    }
    return keys_of(s, *reinterpret_cast<const float4*>(p.cache.acc + at),
                   *reinterpret_cast<const int4*>(p.cache.ordinal + at));
  };
  auto key4 = [&](int s) -> uint4 {
    return cached ? *reinterpret_cast<const uint4*>(keys + (s - lo)) : load4(s);
  };

  uint32_t prefix = 0, mask = 0;
  int want = n;                             // slots still to keep among the candidates
  if (len > n) {
    int2 below = make_int2(0, 0);           // this part's slots below and at the cut
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const int bins = pass == 2 ? 1024 : 2048;
      int* h = hist[pass & 1];
      *reinterpret_cast<int2*>(&h[tid * 2]) = make_int2(0, 0);
      if (pass == 0 && cached) {
        // the only sweep over global memory: four quads of a thread in flight
        constexpr int U = kEvRounds;
        for (int s0 = lo + tid * 4; s0 < hi; s0 += kEvThreads * 4 * U) {
          long long at[U];
          float4 w[U];
          int4 o[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kEvThreads * 4;
            at[u] = s < hi ? p.cache.slot_index(b, kvh, s) : -2;
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (at[u] >= 0) {
              w[u] = *reinterpret_cast<const float4*>(p.cache.acc + at[u]);
              o[u] = *reinterpret_cast<const int4*>(p.cache.ordinal + at[u]);
            }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kEvThreads * 4;
            if (at[u] == -1) raise_device_error(kErrInvalid);
            if (at[u] != -2)
              *reinterpret_cast<uint4*>(keys + (s - lo)) =
                  at[u] >= 0 ? keys_of(s, w[u], o[u]) : make_uint4(~0u, ~0u, ~0u, ~0u);
          }
        }
      }
      __syncthreads();
      for (int s = lo + tid * 4; s < hi; s += kEvThreads * 4) {
        const uint4 k = key4(s);
        const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (s + e < hi && (kk[e] & mask) == prefix)
            atomicAdd(&h[(kk[e] >> shift) & (bins - 1)], 1);
      }
      // all CTAs' histograms; every CTA scans the sum, and its own, for itself
      int2 c = make_int2(0, 0);
      if (CL > 1) {
        sm100::cluster_sync();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (r < CL) {
            const int2 v = ld_cluster_int2(&h[tid * 2], r);
            c.x += v.x;
            c.y += v.y;
          }
        }
      } else {
        __syncthreads();
      }
      const int2 own = *reinterpret_cast<const int2*>(&h[tid * 2]);
      if (CL == 1) c = own;
      int before[2] = {c.x + c.y, own.x + own.y}, all[2];
      block_prefix(before, all, warp_sum);
      if (before[0] < want && want <= before[0] + c.x + c.y) {
        const bool second = want > before[0] + c.x;
        found = make_int4(tid * 2 + second, before[0] + (second ? c.x : 0),
                          before[1] + (second ? own.x : 0), second ? own.y : own.x);
      }
      __syncthreads();
      prefix |= (uint32_t)found.x << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      want -= found.y;
      below.x += found.z;                   // its candidates before the digit are below the cut
      below.y = found.w;
    }
    // slots below / at the cut in the parts before this one
    int2 ahead = make_int2(0, 0);
    if (CL > 1) {
      if (tid == 0) mine = below;
      sm100::cluster_sync();
      for (uint32_t r = 0; r < rank; ++r) {
        const int2 v = ld_cluster_int2(&mine, r);
        ahead.x += v.x;
        ahead.y += v.y;
      }
    }
    // The moves, in slot order: ahead = slots below / at the cut before this sweep. A
    // thread's quads lie kEvThreads * 4 slots apart; their counts (at most 4096 per round
    // and kind, 16 bits each) go through one scan.
    for (int s0 = lo; s0 < hi; s0 += kEvThreads * 4 * kEvRounds) {
      uint32_t kk[kEvRounds][4];
      int cnt[kEvRounds], sum[kEvRounds], at[kEvRounds];
      int mine_cnt[kEvRounds];
#pragma unroll
      for (int q = 0; q < kEvRounds; ++q) {
        const int s = s0 + q * kEvThreads * 4 + tid * 4;
        const uint4 k = s < hi ? key4(s) : make_uint4(~0u, ~0u, ~0u, ~0u);
        at[q] = s < hi ? (int)p.cache.slot_index(b, kvh, s) : -1;     // pool rows stay below 2^31
        kk[q][0] = k.x; kk[q][1] = k.y; kk[q][2] = k.z; kk[q][3] = k.w;
        cnt[q] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          cnt[q] += s + e < hi ? (kk[q][e] < prefix ? 0x10000 : (kk[q][e] == prefix ? 1 : 0)) : 0;
        mine_cnt[q] = cnt[q];
      }
      block_prefix(cnt, sum, warp_sum);
#pragma unroll
      for (int q = 0; q < kEvRounds; ++q) {
        const int s = s0 + q * kEvThreads * 4 + tid * 4;
        int lt = ahead.x + (cnt[q] >> 16), eq = ahead.y + (cnt[q] & 0xffff);
        float4 w;
        int4 o;
        const bool copies = mine_cnt[q] != 0 && s < n && at[q] >= 0;
        if (copies && copy_acc) w = *reinterpret_cast<const float4*>(p.cache.acc + at[q]);
        if (copies && copy_ord) o = *reinterpret_cast<const int4*>(p.cache.ordinal + at[q]);
        const float ww[4] = {w.x, w.y, w.z, w.w};
        const int oo[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int slot = s + e;
          if (slot < hi) {
            const bool below_cut = kk[q][e] < prefix, at_cut = kk[q][e] == prefix;
            const bool kept = below_cut || (at_cut && eq < want);
            const int kept_before = lt + min(eq, want);
            if (slot < n) {
              if (!kept) {
                p.hole[row * p.max_moves + (slot - kept_before)] = at[q] < 0 ? -1 : at[q] + e;
              } else if (at[q] >= 0) {
                if (copy_acc) p.acc_out[at[q] + e] = ww[e];
                if (copy_ord) p.ord_out[at[q] + e] = oo[e];
              }
            } else if (kept) {
              p.mover[row * p.max_moves + (n - 1 - kept_before)] = at[q] < 0 ? -1 : at[q] + e;
            }
            if (slot == n) p.count[row] = n - kept_before;
            lt += below_cut;
            eq += at_cut;
          }
        }
        ahead.x += sum[q] >> 16;
        ahead.y += sum[q] & 0xffff;
      }
    }
    if (CL > 1) sm100::cluster_sync();      // nobody leaves while its counts are being read
  } else {
    if (tid == 0 && rank == 0) p.count[row] = 0;
    if (copy_acc || copy_ord) {
      for (int s = lo + tid; s < hi; s += kEvThreads) {
        const long long at = p.cache.slot_index(b, kvh, s);
        if (at < 0) {
          raise_device_error(kErrInvalid);
          continue;
        }
        if (copy_acc) p.acc_out[at] = p.cache.acc[at];
        if (copy_ord) p.ord_out[at] = p.cache.ordinal[at];
      }
    }
  }
}

// A move's K row and V row: row_bytes / 16 threads with 16 bytes of each, kEvMoveUnroll
// moves of a thread in flight. The lists hold pool rows, so a move is two dependent
// loads deep (list, row). Launched as a programmatic dependent of the selection.
__global__ void __launch_bounds__(kEvMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int U = kEvMoveUnroll;
  grid_dependency_wait();
  const int row = blockIdx.y;
  const int count = p.count[row];
  const int lanes_log2 = p.row_bytes_log2 - 4;             // threads of a move
  const int t = threadIdx.x & ((1 << lanes_log2) - 1);
  const int m0 = (blockIdx.x * kEvMoveThreads + threadIdx.x) >> lanes_log2;
  const int step = (gridDim.x * kEvMoveThreads) >> lanes_log2;
  uint8_t* kp = static_cast<uint8_t*>(p.cache.k_pages) + t * 16;
  uint8_t* vp = static_cast<uint8_t*>(p.cache.v_pages) + t * 16;
  const int32_t* hole = p.hole + row * p.max_moves;
  const int32_t* mover = p.mover + row * p.max_moves;

  for (int m = m0; m < count; m += step * U) {
    long long to[U], from[U];
    uint4 k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      to[u] = m + u * step < count ? hole[m + u * step] : -1;
      from[u] = m + u * step < count ? mover[m + u * step] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0 && from[u] >= 0) {
        k[u] = *reinterpret_cast<const uint4*>(kp + (from[u] << p.row_bytes_log2));
        v[u] = *reinterpret_cast<const uint4*>(vp + (from[u] << p.row_bytes_log2));
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (to[u] < 0 || from[u] < 0) continue;
      *reinterpret_cast<uint4*>(kp + (to[u] << p.row_bytes_log2)) = k[u];
      *reinterpret_cast<uint4*>(vp + (to[u] << p.row_bytes_log2)) = v[u];
      if (t == 0) p.acc_out[to[u]] = p.cache.acc[from[u]];
      if (t == 1) p.ord_out[to[u]] = p.cache.ordinal[from[u]];
    }
  }
}

}  // namespace xattn
