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

constexpr int kEvThreads = 512;
constexpr int kEvBins = 2048;
constexpr int kEvMaxKeys = 40960;      // keys a CTA can hold in shared memory (160 KB)
constexpr int kEvMoveThreads = 256;

struct EvictParams {
  CacheView cache;
  const int32_t* seen;       // [B] or null (lens)
  float* acc_out;
  int32_t* ord_out;
  int32_t* count;            // [rows] moves
  int32_t* hole;             // [rows, max_moves]
  int32_t* mover;            // [rows, max_moves]
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

__device__ __forceinline__ int4 ld_cluster_int4(const void* p, uint32_t rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(sm100::mapa_shared(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ int2 ld_cluster_int2(const void* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(sm100::mapa_shared(p, rank)) : "memory");
  return v;
}

// exclusive prefix of a pair over the block's threads, and the pair's total
__device__ __forceinline__ int2 block_prefix2(int2 v, int2* warp_sum, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) { s.x += x; s.y += y; }
  }
  __syncthreads();                      // warp_sum of an earlier call has been read
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  int2 before = make_int2(s.x - v.x, s.y - v.y), all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kEvThreads / 32; ++w) {
    const int2 t = warp_sum[w];
    if (w < warp) { before.x += t.x; before.y += t.y; }
    all.x += t.x;
    all.y += t.y;
  }
  *total = all;
  return before;
}

__global__ void __launch_bounds__(kEvThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[2][kEvBins];
  __shared__ int2 warp_sum[kEvThreads / 32];
  __shared__ __align__(8) int2 mine;        // this CTA's (below the cut, at the cut)
  __shared__ int2 found;                    // (digit, candidates before it)

  const int tid = threadIdx.x;
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
  auto load4 = [&](int s) -> uint4 {
    uint4 k = make_uint4(~0u, ~0u, ~0u, ~0u);
    const long long at = p.cache.slot_index(b, kvh, s);
    if (at < 0) {
      raise_device_error(kErrInvalid);
      return k;
    }
    const float4 w = *reinterpret_cast<const float4*>(p.cache.acc + at);
    const int4 o = *reinterpret_cast<const int4*>(p.cache.ordinal + at);
    k.x = evict_key(w.x, o.x, safe_from, p.sink);
    if (s + 1 < hi) k.y = evict_key(w.y, o.y, safe_from, p.sink);
    if (s + 2 < hi) k.z = evict_key(w.z, o.z, safe_from, p.sink);
    if (s + 3 < hi) k.w = evict_key(w.w, o.w, safe_from, p.sink);
    return k;
  };
  auto key4 = [&](int s) -> uint4 {
    return cached ? *reinterpret_cast<const uint4*>(keys + (s - lo)) : load4(s);
  };

  uint32_t prefix = 0, mask = 0;
  int want = n;                             // slots still to keep among the candidates
  if (len > n) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const int bins = pass == 2 ? 1024 : 2048;
      int* h = hist[pass & 1];
      for (int i = tid; i < kEvBins; i += kEvThreads) h[i] = 0;
      __syncthreads();
      for (int s = lo + tid * 4; s < hi; s += kEvThreads * 4) {
        uint4 k;
        if (pass == 0) {
          k = load4(s);
          if (cached) *reinterpret_cast<uint4*>(keys + (s - lo)) = k;
        } else {
          k = key4(s);
        }
        const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (s + e < hi && (kk[e] & mask) == prefix)
            atomicAdd(&h[(kk[e] >> shift) & (bins - 1)], 1);
      }
      // all CTAs' histograms; every CTA scans the sum for itself
      int c[4] = {0, 0, 0, 0};
      if (CL > 1) {
        sm100::cluster_sync();
        for (int r = 0; r < CL; ++r) {
          const int4 v = ld_cluster_int4(&h[tid * 4], r);
          c[0] += v.x; c[1] += v.y; c[2] += v.z; c[3] += v.w;
        }
      } else {
        __syncthreads();
        const int4 v = *reinterpret_cast<const int4*>(&h[tid * 4]);
        c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
      }
      int2 all;
      int before = block_prefix2(make_int2(c[0] + c[1] + c[2] + c[3], 0), warp_sum, &all).x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (before < want && want <= before + c[e]) found = make_int2(tid * 4 + e, before);
        before += c[e];
      }
      __syncthreads();
      prefix |= (uint32_t)found.x << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      want -= found.y;
    }
    // slots below and at the cut in this CTA's part, then in the parts before it
    int2 below = make_int2(0, 0);
    for (int s = lo + tid * 4; s < hi; s += kEvThreads * 4) {
      const uint4 k = key4(s);
      const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        below.x += s + e < hi && kk[e] < prefix;
        below.y += s + e < hi && kk[e] == prefix;
      }
    }
    int2 all;
    block_prefix2(below, warp_sum, &all);
    if (tid == 0) mine = all;
    int2 ahead = make_int2(0, 0);
    if (CL > 1) {
      sm100::cluster_sync();
      for (uint32_t r = 0; r < rank; ++r) {
        const int2 v = ld_cluster_int2(&mine, r);
        ahead.x += v.x;
        ahead.y += v.y;
      }
    }
    // the moves, in slot order: ahead = slots below / at the cut before this sweep
    for (int s0 = lo; s0 < hi; s0 += kEvThreads * 4) {
      const int s = s0 + tid * 4;
      const uint4 k = s < hi ? key4(s) : make_uint4(0, 0, 0, 0);
      const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
      int2 here = make_int2(0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        here.x += s + e < hi && kk[e] < prefix;
        here.y += s + e < hi && kk[e] == prefix;
      }
      int2 round;
      int2 bef = block_prefix2(here, warp_sum, &round);
      bef.x += ahead.x;
      bef.y += ahead.y;
      long long at = -1;
      if (s < hi && s < n && (copy_acc || copy_ord)) at = p.cache.slot_index(b, kvh, s);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (s + e >= hi) break;
        const bool lt = kk[e] < prefix, eq = kk[e] == prefix;
        const bool kept = lt || (eq && bef.y < want);
        const int kept_before = bef.x + min(bef.y, want);
        if (s + e < n) {
          if (!kept) {
            p.hole[row * p.max_moves + (s + e - kept_before)] = s + e;
          } else if (at >= 0) {
            if (copy_acc) p.acc_out[at + e] = p.cache.acc[at + e];
            if (copy_ord) p.ord_out[at + e] = p.cache.ordinal[at + e];
          }
        } else if (kept) {
          p.mover[row * p.max_moves + (n - 1 - kept_before)] = s + e;
        }
        if (s + e == n) p.count[row] = n - kept_before;
        bef.x += lt;
        bef.y += eq;
      }
      ahead.x += round.x;
      ahead.y += round.y;
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

// One K row and one V row per move, 16 bytes per lane, kUnroll moves of a lane in flight.
__global__ void __launch_bounds__(kEvMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kUnroll = 4;
  const int row = blockIdx.y, b = row / p.cache.Hkv, kvh = row - b * p.cache.Hkv;
  const int count = p.count[row];
  const int lanes_log2 = p.row_bytes_log2 - 4;             // lanes of a row
  const int t = threadIdx.x & ((2 << lanes_log2) - 1);     // lane of a move: K row, then V row
  const int m0 = (blockIdx.x * kEvMoveThreads + threadIdx.x) >> (lanes_log2 + 1);
  const int step = (gridDim.x * kEvMoveThreads) >> (lanes_log2 + 1);
  uint8_t* pages = static_cast<uint8_t*>((t >> lanes_log2) ? p.cache.v_pages : p.cache.k_pages);
  const long long off = (long long)(t & ((1 << lanes_log2) - 1)) * 16;
  const int32_t* hole = p.hole + row * p.max_moves;
  const int32_t* mover = p.mover + row * p.max_moves;

  for (int m = m0; m < count; m += step * kUnroll) {
    long long to[kUnroll], from[kUnroll];
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      to[u] = from[u] = -1;
      if (m + u * step < count) {
        to[u] = p.cache.slot_index(b, kvh, hole[m + u * step]);
        from[u] = p.cache.slot_index(b, kvh, mover[m + u * step]);
      }
      if (to[u] < 0) from[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (from[u] >= 0)
        x[u] = *reinterpret_cast<const uint4*>(pages + (from[u] << p.row_bytes_log2) + off);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (from[u] < 0) continue;
      *reinterpret_cast<uint4*>(pages + (to[u] << p.row_bytes_log2) + off) = x[u];
      if (t == 0) p.acc_out[to[u]] = p.cache.acc[from[u]];
      if (t == 1) p.ord_out[to[u]] = p.cache.ordinal[from[u]];
    }
  }
}

}  // namespace xattn
