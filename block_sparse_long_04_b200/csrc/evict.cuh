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
// part of the weights and ordinals once, keeps the keys in shared memory (or, if those of the
// table's capacity do not fit, in the workspace: 128 rows of 4224 slots take 14.8 us in a
// table of 131088 slots, 13.8 in one of 4224),
// and adds the bins that hold anything to the first CTA's through distributed shared memory;
// that one finds the digit and the others read it. Inside a CTA
// every warp owns a run of neighbouring slots, so that the last step, which writes the two
// lists of the moves, needs one exchange of counts and then only ballots. The kernel is
// bound by latencies (a row is a few KB to 1 MB, and each of its ~20 dependent steps is a
// memory or barrier latency), not by bandwidth; its loops are kept short and rolled, since
// code that runs once per CTA is fetched once per CTA too. 8 rows of 131072 slots (64 CTAs)
// take 25 us of the call's 73, 128 rows of 4224 slots 12 of its 14. Everything is counted in
// integers: the result does not depend on the order of the atomics.
#pragma once
#include "common.cuh"
#include "rope_append.cuh"
#include "sm100.cuh"

namespace xattn {

constexpr int kEvThreads = 1024;
static_assert(kEvThreads == 1024, "32 warps: their sums are scanned by one warp");
constexpr int kEvBins = 2048;
constexpr int kEvMaxKeys = 40960;      // keys a CTA can hold in shared memory (with rows: 200 KB)
constexpr int kEvMoveThreads = 512;

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
  uint32_t* keys;            // [rows, cluster, evict_part_words] where shared memory holds them not
  int share;                 // most slots of a CTA, a multiple of 4
  int row_bytes_log2;        // of a K or V row
};

// Words of a CTA's part of the workspace: `share` (a multiple of 4) keys, a pool row for every
// fourth slot, and up to the next multiple of four words, because the keys are stored and
// loaded 16 bytes at a time and the parts lie one behind the other.
__host__ __device__ constexpr long long evict_part_words(int share) {
  return ((long long)share + share / 4 + 3) & ~3ll;
}

// ascending key = descending weight; every NaN ranks above +inf, -0 equals +0
__device__ __forceinline__ uint32_t evict_key(float w, int ordinal, int safe_from, int sink) {
  const uint32_t u = w == w ? __float_as_uint(w + 0.f) : 0x7fc00000u;
  const uint32_t key = (int)u < 0 ? u : u ^ 0x7fffffffu;
  return ordinal >= safe_from || ordinal < sink ? 0u : key;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void add_cluster(const int* p, int v, uint32_t rank) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(
                   sm100::mapa_shared(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ int2 ld_cluster_int2(const void* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(sm100::mapa_shared(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ int warp_prefix(int v, int* total) {     // exclusive
  const int lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += x;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  return s - v;
}
// Sum over the warps before this one, and over all, of one value per warp.
__device__ __forceinline__ int before_this_warp(int v, int* sums, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  const int x = sums[lane];
  *all = __reduce_add_sync(0xffffffffu, x);
  return __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
}

__global__ void __launch_bounds__(kEvThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t smem_keys[];
  __shared__ __align__(16) int hist[kEvBins];         // this CTA's
  __shared__ __align__(16) int total[2][kEvBins];     // the cluster's (rank 0), passes in turn
  __shared__ int sums[5][kEvThreads / 32];            // one row per use
  __shared__ __align__(8) int2 mine;        // this CTA's (below the cut, at the cut)
  __shared__ __align__(8) int2 found[3];    // pass's (digit, candidates before it)

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
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
#pragma unroll 1
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

  // (totals are cleared here for the first two passes, and for the third by the first, each
  // ahead of a cluster barrier that everybody who adds to them passes before)
  *reinterpret_cast<int2*>(&hist[tid * 2]) = make_int2(0, 0);
  *reinterpret_cast<int2*>(&total[0][tid * 2]) = make_int2(0, 0);
  *reinterpret_cast<int2*>(&total[1][tid * 2]) = make_int2(0, 0);
  if (CL > 1) cluster_arrive();

  const int seen = p.seen != nullptr ? p.seen[b] : len;
  const int safe_from = (long long)seen - p.recent < -2147483647ll ? -2147483647 : seen - p.recent;
  // keys of this warp's run, and the pool row of every fourth slot, in shared memory or in
  // the workspace: written and read by the warp alone
  uint32_t* part_keys = p.keys == nullptr
                            ? smem_keys
                            : p.keys + ((long long)row * CL + rank) * evict_part_words(p.share);
  uint32_t* mykeys = part_keys + (lo - first);
  int* myrows = reinterpret_cast<int*>(part_keys + p.share) + (lo - first) / 4;
  {
    // the only sweep over the cache: four slots per lane and load, U loads in flight
    constexpr int U = 4;
#pragma unroll 1
    for (int s0 = lo + lane * 4; s0 < hi; s0 += 128 * U) {
      int at[U];                            // (pool rows stay below 2^31)
      float4 w[U];
      int4 o[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        at[u] = s0 + u * 128 < hi ? (int)p.cache.slot_index(b, kvh, s0 + u * 128) : -1;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at[u] >= 0) {
          w[u] = *reinterpret_cast<const float4*>(p.cache.acc + at[u]);
          o[u] = *reinterpret_cast<const int4*>(p.cache.ordinal + at[u]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * 128;
        if (s >= hi) break;
        uint4 k;
        if (at[u] >= 0) {
          k = make_uint4(evict_key(w[u].x, o[u].x, safe_from, p.sink),
                         evict_key(w[u].y, o[u].y, safe_from, p.sink),
                         evict_key(w[u].z, o[u].z, safe_from, p.sink),
                         evict_key(w[u].w, o[u].w, safe_from, p.sink));
          // into other arrays: slots below n as they are; the moves overwrite the evicted ones
          if (s + 4 <= n) {
            if (copy_acc) *reinterpret_cast<float4*>(p.acc_out + at[u]) = w[u];
            if (copy_ord) *reinterpret_cast<int4*>(p.ord_out + at[u]) = o[u];
          } else if (s < n) {
#pragma unroll 1
            for (int e = 0; s + e < n; ++e) {
              if (copy_acc) p.acc_out[at[u] + e] = p.cache.acc[at[u] + e];
              if (copy_ord) p.ord_out[at[u] + e] = p.cache.ordinal[at[u] + e];
            }
          }
        } else {
          // A bad page's slots have no rows to give or to take. Below n they stay (as safe ones:
          // n slots cannot come before them), from n on they go (the slots below n, bad ones
          // among them, are enough). So neither list of the moves names one.
          raise_device_error(kErrInvalid);
          k = make_uint4(s < n ? 0u : ~0u, s + 1 < n ? 0u : ~0u, s + 2 < n ? 0u : ~0u, s + 3 < n ? 0u : ~0u);
        }
        *reinterpret_cast<uint4*>(mykeys + (s - lo)) = k;     // (from hi on: written, never read)
        myrows[(s - lo) / 4] = at[u];
      }
    }
    __syncwarp();
  }
  __syncthreads();                          // the histogram has been cleared
  if (CL > 1) cluster_wait();               // and the totals

  uint32_t prefix = 0, mask = 0;
  int want = n;                             // slots still to keep among the candidates
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bins = pass == 2 ? 1024 : 2048;
#pragma unroll 4
    for (int s = lo + lane; s < hi; s += 32) {
      const uint32_t k = mykeys[s - lo];
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    int2 c = *reinterpret_cast<const int2*>(&hist[tid * 2]);
    *reinterpret_cast<int2*>(&hist[tid * 2]) = make_int2(0, 0);
    if (CL > 1) {
      int* sum = &total[pass & 1][tid * 2];
      if (c.x) add_cluster(sum, c.x, 0);
      if (c.y) add_cluster(sum + 1, c.y, 0);
      sm100::cluster_sync();
      if (rank == 0) {
        c = *reinterpret_cast<const int2*>(sum);
        *reinterpret_cast<int2*>(sum) = make_int2(0, 0);
      }
    }
    if (rank == 0) {
      int in_warp, all;
      int before = warp_prefix(c.x + c.y, &in_warp);
      before += before_this_warp(in_warp, sums[pass], &all);
      if (before < want && want <= before + c.x + c.y) {
        const bool second = want > before + c.x;
        found[pass] = make_int2(tid * 2 + second, before + (second ? c.x : 0));
      }
    }
    int2 f;
    if (CL > 1) {
      sm100::cluster_sync();
      f = ld_cluster_int2(&found[pass], 0);
    } else {
      __syncthreads();
      f = found[pass];
    }
    prefix |= (uint32_t)f.x << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    want -= f.y;
  }

  // slots below / at the cut: this warp's, those of the warps and of the parts before it
  int2 here = make_int2(0, 0), ahead, part;
#pragma unroll 4
  for (int s = lo + lane; s < hi; s += 32) {
    const uint32_t k = mykeys[s - lo];
    here.x += k < prefix;
    here.y += k == prefix;
  }
  here.x = __reduce_add_sync(0xffffffffu, here.x);
  here.y = __reduce_add_sync(0xffffffffu, here.y);
  ahead.x = before_this_warp(here.x, sums[3], &part.x);
  ahead.y = before_this_warp(here.y, sums[4], &part.y);
  if (CL > 1) {
    if (tid == 0) mine = part;
    sm100::cluster_sync();
    for (uint32_t r = 0; r < rank; ++r) {
      const int2 v = ld_cluster_int2(&mine, r);
      ahead.x += v.x;
      ahead.y += v.y;
    }
  }
  // the moves, in slot order, four neighbouring slots per lane
  int32_t* hole = p.hole + row * p.max_moves;
  int32_t* mover = p.mover + row * p.max_moves;
#pragma unroll 1
  for (int s0 = lo; s0 < hi; s0 += 128) {
    const int s = s0 + lane * 4;
    uint4 k = make_uint4(~0u, ~0u, ~0u, ~0u);
    int at = 0;
    if (s < hi) {
      at = myrows[(s - lo) / 4];
      k = *reinterpret_cast<const uint4*>(mykeys + (s - lo));
      if (s + 1 >= hi) k.y = ~0u;            // (not below any cut)
      if (s + 2 >= hi) k.z = ~0u;
      if (s + 3 >= hi) k.w = ~0u;
    }
    // slots below the cut in the low half, at the cut in the high half: this lane's, then
    // those of the lanes before it (at most 128 each)
    const int live = min(max(hi - s, 0), 4);
    const bool lt[4] = {k.x < prefix, k.y < prefix, k.z < prefix, k.w < prefix};
    const bool eq[4] = {k.x == prefix && live > 0, k.y == prefix && live > 1,
                        k.z == prefix && live > 2, k.w == prefix && live > 3};
    int all;
    const int before = warp_prefix(lt[0] + lt[1] + lt[2] + lt[3] +
                                       ((eq[0] + eq[1] + eq[2] + eq[3]) << 16), &all);
    int eq_before = ahead.y + (before >> 16);
    const int kept_before = ahead.x + (before & 0xffff) + min(eq_before, want);
    ahead.x += all & 0xffff;
    ahead.y += all >> 16;
    bool kept[4] = {lt[0], lt[1], lt[2], lt[3]};
    if (all >> 16) {                         // of the slots at the cut the first `want` stay
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kept[e] |= eq[e] && eq_before < want;
        eq_before += eq[e];
      }
    }
    if (s + 4 <= n) {                        // slots below n: the evicted ones are holes
      int i = s - kept_before;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!kept[e] && s + e < hi) hole[i++] = at + e;
    } else if (s >= n) {                     // slots from n on: the kept ones move
      if (s == n && s < hi) p.count[row] = n - kept_before;
      int i = n - 1 - kept_before;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (kept[e]) mover[i--] = at + e;
    } else {                                 // the quad that holds n
#pragma unroll 1
      for (int e = 0, kb = kept_before; e < 4; ++e) {
        const bool stays = e == 0 ? kept[0] : (e == 1 ? kept[1] : (e == 2 ? kept[2] : kept[3]));
        if (s + e == n && s + e < hi) p.count[row] = n - kb;
        if (s + e < n && !stays && s + e < hi) hole[s + e - kb] = at + e;
        if (s + e >= n && stays) mover[n - 1 - kb] = at + e;
        kb += stays;
      }
    }
  }
  if (CL > 1) sm100::cluster_sync();        // nobody leaves while its counts are being read
}

// A move's K row and V row: row_bytes / 16 threads with 16 bytes of each. The lists hold
// pool rows, so a move is two dependent loads deep (list, row). Many warps with one move
// each in flight did better than fewer with two or four (51 against 60 us for the 32768
// moves of 8 rows each of a 128K cache cut to half: 0.27 GB read and written, 5.2 TB/s;
// rows of 256 bytes at random places do not reach the copy's 6.5).
__global__ void __launch_bounds__(kEvMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  grid_dependency_wait();
  const int row = blockIdx.y;
  const int count = p.count[row];
  const int lanes_log2 = p.row_bytes_log2 - 4;             // threads of a move
  const int t = threadIdx.x & ((1 << lanes_log2) - 1);
  const int step = (gridDim.x * kEvMoveThreads) >> lanes_log2;
  uint8_t* kp = static_cast<uint8_t*>(p.cache.k_pages) + t * 16;
  uint8_t* vp = static_cast<uint8_t*>(p.cache.v_pages) + t * 16;
  const int32_t* hole = p.hole + row * p.max_moves;
  const int32_t* mover = p.mover + row * p.max_moves;
  for (int m = (blockIdx.x * kEvMoveThreads + threadIdx.x) >> lanes_log2; m < count; m += step) {
    const long long to = hole[m], from = mover[m];
    const uint4 k = *reinterpret_cast<const uint4*>(kp + (from << p.row_bytes_log2));
    const uint4 v = *reinterpret_cast<const uint4*>(vp + (from << p.row_bytes_log2));
    *reinterpret_cast<uint4*>(kp + (to << p.row_bytes_log2)) = k;
    *reinterpret_cast<uint4*>(vp + (to << p.row_bytes_log2)) = v;
    if (t == 0) p.acc_out[to] = p.cache.acc[from];
    if (t == 1) p.ord_out[to] = p.cache.ordinal[from];
  }
}

}  // namespace xattn
