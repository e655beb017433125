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
// and adds the other CTAs' histograms through distributed shared memory. Inside a CTA
// every warp owns a run of neighbouring slots, so that the last step, which writes the two
// lists of the moves, needs one exchange of counts and then only ballots. The kernel is
// bound by latencies (a row is a few KB to 1 MB, and each of its ~20 dependent steps is a
// memory or barrier latency), not by bandwidth; its loops are kept short and rolled, since
// code that runs once per CTA is fetched once per CTA too. Everything is counted in
// integers: the result does not depend on the order of the atomics.
#pragma once
#include "common.cuh"
#include "rope_append.cuh"
#include "sm100.cuh"

namespace xattn {

constexpr int kEvThreads = 1024;
static_assert(kEvThreads == 1024, "32 warps: their sums are scanned by one warp");
constexpr int kEvBins = 2048;
constexpr int kEvMaxKeys = 40960;      // keys a CTA can hold in shared memory (160 KB)
constexpr int kEvMoveThreads = 256;
constexpr int kEvMoveUnroll = 2;       // moves of a thread in flight

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

// exclusive prefix of a pair over the lanes of a warp, and the pair's total
__device__ __forceinline__ int2 warp_prefix2(int2 v, int2* total) {
  const int lane = threadIdx.x & 31;
  int2 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) { s.x += x; s.y += y; }
  }
  *total = make_int2(__shfl_sync(0xffffffffu, s.x, 31), __shfl_sync(0xffffffffu, s.y, 31));
  return make_int2(s.x - v.x, s.y - v.y);
}
// exclusive prefix of a pair over the warps of the block, for every thread of the warp
__device__ __forceinline__ int2 before_this_warp(int2 warp_total, int2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();                      // sums of an earlier call have been read
  if (lane == 0) sums[warp] = warp_total;
  __syncthreads();
  int2 all;
  const int2 v = warp_prefix2(sums[lane], &all);
  return make_int2(__shfl_sync(0xffffffffu, v.x, warp), __shfl_sync(0xffffffffu, v.y, warp));
}

__global__ void __launch_bounds__(kEvThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[2][kEvBins];
  __shared__ int2 sums[kEvThreads / 32];
  __shared__ __align__(8) int2 mine;        // this CTA's (below the cut, at the cut)
  // (digit, candidates before it, of these in this part, this part's with the digit)
  __shared__ int4 found;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependents_may_start();              // the moves wait for this grid's end themselves
  const int CL = gridDim.x;                 // the grid's x is one cluster
  const uint32_t rank = blockIdx.x;
  const int row = blockIdx.y, b = row / p.cache.Hkv, kvh = row - b * p.cache.Hkv;
  const int len = p.cache.length(b);
  const int n = p.budget;
  const bool copy_acc = p.acc_out != p.cache.acc, copy_ord = p.ord_out != p.cache.ordinal;
  if (tid == 0 && rank == 0 && !p.cache.length_valid(b)) raise_device_error(kErrInvalid);

  // this CTA's slots, and of these this warp's, [lo, hi); shares are multiples of four
  // slots, which never cross a page
  const int share = ((len + CL - 1) / CL + 3) & ~3;
  const int first = min((int)rank * share, len), last = min(first + share, len);
  const int run = ((last - first + kEvThreads / 32 - 1) / (kEvThreads / 32) + 3) & ~3;
  const int lo = min(first + warp * run, last), hi = min(lo + run, last);

  if (len <= n) {                           // nothing goes
    if (tid == 0 && rank == 0) p.count[row] = 0;
    if (copy_acc || copy_ord) {
#pragma unroll 2
      for (int s = lo + lane; s < hi; s += 32) {
        const long long at = p.cache.slot_index(b, kvh, s);
        if (at < 0) {
          raise_device_error(kErrInvalid);
          continue;
        }
        if (copy_acc) p.acc_out[at] = p.cache.acc[at];
        if (copy_ord) p.ord_out[at] = p.cache.ordinal[at];
      }
    }
    return;
  }

  const int seen = p.seen != nullptr ? __ldg(p.seen + b) : len;
  const int safe_from = (long long)seen - p.recent < -2147483647ll ? -2147483647 : seen - p.recent;
  const bool cached = share <= p.smem_keys;
  uint32_t* mykeys = keys + (lo - first);   // of this warp's run
  auto load_key = [&](int s) -> uint32_t {
    const long long at = p.cache.slot_index(b, kvh, s);
    if (at < 0) {
      raise_device_error(kErrInvalid);
      return ~0u;                           // the largest key: never wanted before another
    }
    return evict_key(p.cache.acc[at], p.cache.ordinal[at], safe_from, p.sink);
  };
  auto key_of = [&](int s) -> uint32_t { return cached ? mykeys[s - lo] : load_key(s); };

  if (cached) {
    // the only sweep over global memory: four slots per lane and load, four loads in flight
    constexpr int U = 4;
    for (int s0 = lo + lane * 4; s0 < hi; s0 += 128 * U) {
      long long at[U];
      float4 w[U];
      int4 o[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        at[u] = s0 + u * 128 < hi ? p.cache.slot_index(b, kvh, s0 + u * 128) : -2;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at[u] >= 0) {
          w[u] = *reinterpret_cast<const float4*>(p.cache.acc + at[u]);
          o[u] = *reinterpret_cast<const int4*>(p.cache.ordinal + at[u]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u] == -2) continue;
        uint4 k = make_uint4(~0u, ~0u, ~0u, ~0u);
        if (at[u] >= 0)
          k = make_uint4(evict_key(w[u].x, o[u].x, safe_from, p.sink),
                         evict_key(w[u].y, o[u].y, safe_from, p.sink),
                         evict_key(w[u].z, o[u].z, safe_from, p.sink),
                         evict_key(w[u].w, o[u].w, safe_from, p.sink));
        else
          raise_device_error(kErrInvalid);
        // (slots from hi on: written, never read)
        *reinterpret_cast<uint4*>(mykeys + (s0 + u * 128 - lo)) = k;
      }
    }
    __syncwarp();
  }

  uint32_t prefix = 0, mask = 0;
  int want = n;                             // slots still to keep among the candidates
  int2 below = make_int2(0, 0);             // this part's slots below and at the cut
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bins = pass == 2 ? 1024 : 2048;
    int* h = hist[pass & 1];
    *reinterpret_cast<int2*>(&h[tid * 2]) = make_int2(0, 0);
    __syncthreads();
#pragma unroll 4
    for (int s = lo + lane; s < hi; s += 32) {
      const uint32_t k = key_of(s);
      if ((k & mask) == prefix) atomicAdd(&h[(k >> shift) & (bins - 1)], 1);
    }
    // all CTAs' histograms; every CTA scans the sum, and its own, for itself
    int2 c = make_int2(0, 0);
    if (CL > 1) {
      sm100::cluster_sync();
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < CL) {
          const int2 v = ld_cluster_int2(&h[tid * 2], r);
          c.x += v.x;
          c.y += v.y;
        }
    } else {
      __syncthreads();
    }
    const int2 own = *reinterpret_cast<const int2*>(&h[tid * 2]);
    if (CL == 1) c = own;
    int2 total;
    int2 before = warp_prefix2(make_int2(c.x + c.y, own.x + own.y), &total);
    const int2 ahead = before_this_warp(total, sums);
    before.x += ahead.x;
    before.y += ahead.y;
    if (before.x < want && want <= before.x + c.x + c.y) {
      const bool second = want > before.x + c.x;
      found = make_int4(tid * 2 + second, before.x + (second ? c.x : 0),
                        before.y + (second ? own.x : 0), second ? own.y : own.x);
    }
    __syncthreads();
    prefix |= (uint32_t)found.x << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    want -= found.y;
    below.x += found.z;                     // its candidates before the digit are below the cut
    below.y = found.w;
  }

  // slots below / at the cut in the parts before this one, then in the warps before this one
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
  int2 here = make_int2(0, 0);
#pragma unroll 4
  for (int s = lo + lane; s < hi; s += 32) {
    const uint32_t k = key_of(s);
    here.x += k < prefix;
    here.y += k == prefix;
  }
  here.x = __reduce_add_sync(0xffffffffu, here.x);
  here.y = __reduce_add_sync(0xffffffffu, here.y);
  const int2 warps = before_this_warp(here, sums);
  ahead.x += warps.x;
  ahead.y += warps.y;
  // the moves, in slot order
#pragma unroll 2
  for (int s0 = lo; s0 < hi; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < hi;
    const uint32_t k = in ? key_of(s) : ~0u;
    const int at = in ? (int)p.cache.slot_index(b, kvh, s) : -1;     // pool rows stay below 2^31
    const bool lt = in && k < prefix, eq = in && k == prefix;
    const unsigned mlt = __ballot_sync(0xffffffffu, lt), meq = __ballot_sync(0xffffffffu, eq);
    const unsigned lower = (1u << lane) - 1;
    const int lt_before = ahead.x + __popc(mlt & lower), eq_before = ahead.y + __popc(meq & lower);
    const bool kept = lt || (eq && eq_before < want);
    const int kept_before = lt_before + min(eq_before, want);
    if (in) {
      if (s < n) {
        if (!kept) {
          p.hole[row * p.max_moves + (s - kept_before)] = at;
        } else if (at >= 0) {
          if (copy_acc) p.acc_out[at] = p.cache.acc[at];
          if (copy_ord) p.ord_out[at] = p.cache.ordinal[at];
        }
      } else if (kept) {
        p.mover[row * p.max_moves + (n - 1 - kept_before)] = at;
      }
      if (s == n) p.count[row] = n - kept_before;
    }
    ahead.x += __popc(mlt);
    ahead.y += __popc(meq);
  }
  if (CL > 1) sm100::cluster_sync();        // nobody leaves while its counts are being read
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
