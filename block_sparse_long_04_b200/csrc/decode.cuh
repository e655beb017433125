// Attention of one new token per sequence over a paged key-value cache.
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j,  j over the slots < lens[b]
//
// Bound. A cached element is used for 2 flops per query head of its kv head: 4 to 16 flops per
// byte of bf16 pages, 8 to 32 of e4m3 pages at 4 to 16 heads. Up to 16 heads every cached byte
// is loaded once, and HBM sets the pace (for e4m3 with more than 8 heads, the instructions).
// Larger groups are items of 16 heads each, which load K and V again at other times:
// 32 heads per kv head take about twice, 128 eight times as long as 16. The kernel's task is to keep
// enough bytes in flight on every SM and to stay off everybody's critical path.
//
// Split. The tiles (64 or 128 keys) of all (sequence, kv head) items form one linear order,
// which is cut into equal shares, one per CTA: ragged batches and single long sequences
// load all SMs alike, and nothing has to be planned on the host. A CTA walks its share;
// where an item ends inside it, the partial (maximum, sum, unnormalised output) goes to
// the workspace. Items that one CTA covers alone are finished there, the others by
// decode_join_kernel. CTA c and item i meet in at most one segment, and along the linear
// order c + i grows, so c + i numbers the partials.
//
// One CTA (two or three per SM): warp 4 loads K and V tiles by TMA, one box per page part,
// into a ring of stages; warps 0-3 own a quarter of the tile's keys each and run
// independently (own reference, sum and output) until the item's end. The products use
// warp-level MMAs with the cache as the A operand: S^T = K Q^T and O^T = V^T P^T, 16 keys
// or columns by 8 heads, so the usual groups of 4 or 8 query heads fill the tile's N
// (a tcgen05 tile would need M = 128 rows of queries, or P^T written to shared memory and
// O^T read from TMEM between the steps; the tensor pipe is not what binds here). P turns
// from the accumulator's layout into the B operand's with movmatrix, in registers.
//
// Rounding. The weights enter P V as two 16-bit terms, p cut to its type and what that left (16
// bits together in bf16, 22 in f16), for one more MMA per tile; a single bf16 weight would add
// an error as large as the output's own rounding. e4m3 pages are widened to f16, which
// holds them exactly. q is scaled there by a power of two per head so that its largest
// element is in [1/2, 1]; below 2^-14 of that f16 loses bits, an error of 2^-25 of the
// largest element, less than the fp32 sums'. f16 weights end at 2^-25, too early for one
// reference per head: beside a slot that takes nearly all the weight, and whose value may be 0,
// the others would count in the sum and not in the output. So the reference follows the
// tiles down too, and a weight is off by at most 2^-26 of the largest among the keys that
// a warp takes together (32 neighbours at most), or by 2^-112 of the head's largest. (Tiles
// with references of their own, scaled into the head's output, would hold 2^-38 of the largest
// neighbour, and took 159 us instead of 136 for 32 sequences of 8192 slots with 16 heads per kv head.)
// Sums, logits and statistics are fp32, o is rounded once.
//
// Measured, whole calls, 32 query and 8 kv heads, C = 128 (a range is over several GPUs): one
// sequence of 131072 bf16 slots 85 to 88 us (0.54 GB, 6.1 to 6.3 TB/s), 32 ragged e4m3 sequences
// 95 us (0.59 GB, 6.1 TB/s), 8 of 32768 with weights 185 to 189 us (1.09 GB, 5.8 TB/s), one of 777
// slots 6.8 us. 16 heads per kv head: 90 us for the first case in bf16, 71 to 82 us in e4m3 (half the
// bytes). One kv head, 32 sequences of 32768 slots (0.54 GB in bf16, 0.27 in e4m3): 32 query heads
// 168 and 132 us, 128 query heads 620 and 500 us. What binds up to 8 heads is HBM; for e4m3 the
// widening (64 of some 260 instructions per 16 keys and warp) comes close.
//
// Keys behind the end of a sequence inside its last page are masked, and their V rows
// are zeroed in shared memory before use: 0 * NaN of a stale row would not be 0.
// Every wait is bounded (sm100::mbar_wait).
#pragma once
#include <cuda_fp16.h>
#include "common.cuh"
#include "rope_append.cuh"
#include "sm100.cuh"

namespace xattn {

constexpr int kDecThreads = 160;      // four MMA warps, one TMA warp
constexpr int kDecMaxCtas = 444;      // 148 SMs x 3
constexpr int kJoinThreads = 128;     // at least the largest C
constexpr int kDecMaxGroup = 128;     // query heads per kv head
// f16 weights of a tile (e4m3 pages): the largest lies between 2^kF16Low and 2^kF16High (65504
// is the type's end), 2^kF16Set where the reference has just moved. Sums of weights and
// outputs stay below 2^(kF16Span + 9 + 28): 448 at most, 2^28 keys of a warp.
constexpr float kF16Low = 2.f, kF16Set = 12.f, kF16High = 15.f, kF16Span = 88.f;
constexpr float kTinyScale = 1e-37f;  // a logit scale that underflows must not make NaN of -inf

struct DecodeParams {
  CacheView cache;
  const bf16* q;
  long long q_sb, q_sh;
  bf16* O;                 // [B, Hq, C]
  float* lse;              // [B, Hq] or null
  float* part_o;           // [partials][rows][C]
  float2* part_ml;         // [partials][rows] (maximum in log2 units, sum)
  int2* seg;               // [items] first and last CTA of the item
  float* logits;           // [B, Hq, capacity] in log2 units, or null
  float* acc_out;          // [num_pages, Hkv, page] or null
  int Hq, G, HT;           // query heads, per kv head, head tiles per kv head
  float scale_log2;
  const int32_t* n_new;    // [B] (IDLE kernels)

  // Slots of sequence b that are attended to: none without a new token. (Kernels of their own
  // for n_new, because a test of the pointer here cost 0.4 us of a short context's 6.8.)
  template <bool IDLE>
  __device__ __forceinline__ int length(int b) const {
    const int n = cache.length(b);
    return IDLE && n_new[b] != 1 ? 0 : n;
  }
  template <bool IDLE>
  __device__ __forceinline__ bool valid(int b) const {
    return cache.length_valid(b) && !(IDLE && (unsigned)n_new[b] > 1u);
  }
};

// Keys per tile: 64, or 128 where a 32 KB stage holds them: a warp then works on two
// independent sets of 16 keys, which hides the latencies of its chain (load, widen,
// product, maximum, exponential, product) and halves its overhead per key.
__host__ __device__ constexpr int dec_tile_keys(int C, bool fp8, int NT) {
  return NT == 1 && C * (fp8 ? 1 : 2) <= 128 ? 128 : 64;
}

template <int C, bool FP8, int NT>
struct Decode {
  static constexpr int kPerSm = NT == 1 ? 3 : 2;       // CTAs per SM (128 or 168 registers)
  static constexpr int kRow = C * (FP8 ? 1 : 2);
  static constexpr int kKeys = dec_tile_keys(C, FP8, NT);
  static constexpr int kSets = kKeys / 64;             // sets of 16 keys per warp
  static constexpr int kTile = kKeys * kRow;
  static constexpr int kStage = 2 * kTile;
  static constexpr int kFit = (NT == 1 ? 65536 : 98304) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kRows = 8 * NT;                 // heads of one item
  static constexpr int kXRow = C + 4;                  // fp32 output row, off the bank period
  static constexpr int kOffX = kStages * kStage;       // [2][8][kXRow]
  static constexpr int kOffMl = kOffX + 2 * 8 * kXRow * 4;
  static constexpr int kOffBar = kOffMl + 4 * kRows * 8;
  static constexpr int kSmem = kOffBar + 256 + 1024;   // + alignment slack
};

// ------------------------------------------------------------ the linear order
template <int KEYS, bool IDLE>
__device__ __forceinline__ int dec_tiles(const DecodeParams& p, int b) {
  return (p.length<IDLE>(b) + KEYS - 1) / KEYS;
}
// sum of the tiles of all sequences (one warp)
template <int KEYS, bool IDLE>
__device__ __forceinline__ long long dec_total(const DecodeParams& p, int lane) {
  long long n = 0;
  for (int b = lane; b < p.cache.B; b += 32) n += dec_tiles<KEYS, IDLE>(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// A place in the linear order: tile `tile` of `tiles` of head item `hk` of sequence b.
struct DecPos {
  int b, hk, tile, tiles;
};
// Place of linear tile t (0 <= t < total * per), `per` items per sequence (one warp).
template <int KEYS, bool IDLE>
__device__ __forceinline__ DecPos dec_find(const DecodeParams& dp, long long t, int per, int lane) {
  long long base = 0;
  for (int b0 = 0; b0 < dp.cache.B; b0 += 32) {
    const int n = b0 + lane < dp.cache.B ? dec_tiles<KEYS, IDLE>(dp, b0 + lane) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, (base + incl) * per > t);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      const long long before = base + __shfl_sync(0xffffffffu, incl - n, l);
      const int tiles = __shfl_sync(0xffffffffu, n, l);
      const long long rem = t - before * per;
      DecPos p;
      p.b = b0 + l;
      p.hk = (int)(rem / tiles);
      p.tile = (int)(rem - (long long)p.hk * tiles);
      p.tiles = tiles;
      return p;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  DecPos none = {0, 0, 0, 1};
  return none;
}
// the next item with a tile (there is one)
template <int KEYS, bool IDLE>
__device__ __forceinline__ void dec_next_item(const DecodeParams& dp, DecPos& p, int per) {
  p.tile = 0;
  if (++p.hk < per) return;
  p.hk = 0;
  do {
    ++p.b;
    p.tiles = p.b < dp.cache.B ? dec_tiles<KEYS, IDLE>(dp, p.b) : 1;
  } while (p.tiles == 0);
}

// ------------------------------------------------------------ warp-level MMA
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four e4m3 -> two f16x2, exact
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t x, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n" : "=r"(*lo), "=r"(*hi) : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two 16-bit pairs whose sums are (x, y), x and y >= 0. f16: rounded, and what that left. bf16:
// the next value below x, and what is left, which is never 0 or negative unless x is 0. Both
// are multiplied with the same value, and an infinite one (e4m3 has none) must stay that
// infinity: 0 * inf and inf - inf are NaN.
template <bool F16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t* hi, uint32_t* lo) {
  if (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    *hi = *reinterpret_cast<const uint32_t*>(&h);
    *lo = pack_f16x2(x - __low2float(h), y - __high2float(h));
  } else {
    const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
    const uint32_t hx = (ux - (ux != 0u)) & 0xffff0000u, hy = (uy - (uy != 0u)) & 0xffff0000u;
    *hi = __byte_perm(hx, hy, 0x7632);
    *lo = pack_bf16x2(x - __uint_as_float(hx), y - __uint_as_float(hy));
  }
}
// transposes an 8 x 8 matrix of 16-bit values (lane l: row l/4, columns 2(l%4), +1)
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void bar_mma_warps() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Cached rows are read once per call and head tile: first to leave L2, where the partials, logits and
// queries should stay (128K keys 86.6 -> 84.5 us, ragged e4m3 batch 103.3 -> 100.4 us).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint64_t* bar) {
  asm volatile(
      "{\n .reg .b64 once;\n createpolicy.fractional.L2::evict_first.b64 once, 1.0;\n"
      " cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], once;\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ split
template <int C, bool FP8, int NT, bool IDLE>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 3 : 2)
decode_split_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ DecodeParams p) {
  using L = Decode<C, FP8, NT>;
  using namespace sm100;
  constexpr int ST = L::kStages;
  constexpr int kSteps = C / 16;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* xo = reinterpret_cast<float*>(smem + L::kOffX);        // [2][8][kXRow]
  float2* xml = reinterpret_cast<float2*>(smem + L::kOffMl);    // [4][kRows]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty = full + ST;
  uint32_t* parts = reinterpret_cast<uint32_t*>(empty + ST);    // [ST] page parts that were loaded
  volatile int* abort_flag = reinterpret_cast<volatile int*>(parts + ST);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = p.cache.Hkv * p.HT;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  grid_dependency_wait();
  // every warp finds the CTA's share for itself
  const long long total = dec_total<L::kKeys, IDLE>(p, lane) * per;
  const long long n_cta = total < gridDim.x ? total : gridDim.x;
  if ((long long)blockIdx.x >= n_cta) return;
  const long long t0 = blockIdx.x * total / n_cta;
  const int mine = (int)((blockIdx.x + 1) * total / n_cta - t0);
  DecPos at = dec_find<L::kKeys, IDLE>(p, t0, per, lane);
  __syncthreads();

  // a page holds a tile (or two), or a tile spans several pages
  const int part_log2 = min(p.cache.page_log2, 6);     // keys of a page part (one TMA box)
  const int n_parts = L::kKeys >> part_log2;

  if (warp == 4) {
    // ------------------------------------------------------ TMA producer
    const uint32_t part_bytes = (uint32_t)L::kRow << part_log2;
    // lane l < n_parts looks up the page of part l, one tile ahead of its load
    auto page_of = [&](const DecPos& q) -> int {
      const int slot = q.tile * L::kKeys + (lane << part_log2);
      if (lane >= n_parts || slot >= p.length<IDLE>(q.b)) return -1;
      return p.cache.page_table[(long long)q.b * p.cache.max_pages + (slot >> p.cache.page_log2)];
    };
    auto advance = [&](DecPos& q) {
      if (++q.tile == q.tiles) dec_next_item<L::kKeys, IDLE>(p, q, per);
    };
    int pid = page_of(at);
    int n = 0;
    for (; n < mine; ++n) {
      const DecPos cur = at;
      const int st = n % ST;
      const int slot = cur.tile * L::kKeys + (lane << part_log2);
      const bool wanted = lane < n_parts && slot < p.length<IDLE>(cur.b);
      const bool good = wanted && pid >= 0 && pid < p.cache.num_pages;
      const int row = (((pid * p.cache.Hkv) + cur.hk / p.HT) << p.cache.page_log2) +
                      (slot & ((1 << p.cache.page_log2) - 1));
      if (wanted && !good) raise_device_error(kErrInvalid);
      int next_pid = -1;
      if (n + 1 < mine) {
        advance(at);
        next_pid = page_of(at);
      }
      if (n >= ST &&
          !__all_sync(0xffffffffu, mbar_wait(&empty[st], ((n / ST) - 1) & 1, abort_flag)))
        break;
      const unsigned loaded = __ballot_sync(0xffffffffu, good);
      if (lane == 0) {
        parts[st] = loaded;
        mbar_expect_tx(&full[st], 2 * part_bytes * __popc(loaded));
      }
      __syncwarp();
      if (good) {
        const uint32_t dst = smem_u32(smem + st * L::kStage) + lane * part_bytes;
        tma_load_3d(dst, &tmK, 0, row, 0, &full[st]);
        tma_load_3d(dst + L::kTile, &tmV, 0, row, 0, &full[st]);
      }
      pid = next_pid;
    }
    // every load issued must land before the CTA may exit
    volatile int no_abort = 0;
    for (int i = (n > ST ? n - ST : 0); i < n; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, &no_abort);
    return;
  }

  // ------------------------------------------------------------ MMA warps
  constexpr int SETS = L::kSets;
  const int hr = lane >> 2, i4 = lane & 3;     // MMA row (head), column group
  // this warp's sets of 16 keys: first key in the tile, page part, and place of the part's
  // rows in a stage
  int k0[SETS], part[SETS], r0[SETS];
  uint32_t part_off[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    k0[u] = (warp * SETS + u) * 16;
    part[u] = k0[u] >> part_log2;
    r0[u] = k0[u] & ((1 << part_log2) - 1);
    part_off[u] = (uint32_t)part[u] * ((uint32_t)L::kRow << part_log2);
  }
  // Shared-memory places (the TMA swizzle): 16-byte chunk c of row r of a part lies at chunk
  // place c ^ (r & 7) of its 128-byte row (bf16 rows of 128: in the second half's rows from
  // c = 8 on), or c ^ ((r / 2) & 3) of its 64-byte row.
  auto chunk = [&](uint32_t base, int r, int cb) -> uint32_t {
    if (L::kRow == 64) return base + r * 64 + ((cb ^ ((r >> 1) & 3)) << 4);
    const uint32_t half = (uint32_t)(cb >> 3) << (7 + part_log2);
    return base + half + r * 128 + (((cb & 7) ^ (r & 7)) << 4);
  };
  // ldmatrix reads chunks k and k+1 of a row, k even: with the row's chunk (lane bit) placed
  // once, the place of any k is one exclusive or away (rows begin at multiples of their size)
  const int row_a = (((lane >> 3) & 1) << 3) + (lane & 7);     // matrices: rows, then chunks
  const int row_v = FP8 ? row_a : ((lane >> 4) << 3) + (lane & 7);   // (bf16 V: chunks, rows)
  uint32_t off_k[SETS], off_v[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    off_k[u] = chunk(part_off[u], r0[u] + row_a, lane >> 4);
    off_v[u] = L::kTile + chunk(part_off[u], r0[u] + row_v, FP8 ? lane >> 4 : (lane >> 3) & 1);
  }
  const uint32_t half_off = 128u << part_log2;
  auto place = [&](uint32_t row_chunk, int k) -> uint32_t {    // k: a constant
    return (row_chunk ^ (uint32_t)((k & (L::kRow == 64 ? 3 : 7)) << 4)) + (k >= 8 ? half_off : 0u);
  };

  bool ok = true;
  int n = 0;
  while (n < mine) {
    const int len = p.length<IDLE>(at.b);
    const int kvh = at.hk / p.HT, ht = at.hk - kvh * p.HT;
    const int h0 = kvh * p.G + ht * 16;                     // first query head of the item
    const int heads = min(p.G - ht * 16, L::kRows);
    const int seg_tiles = min(at.tiles - at.tile, mine - n);
    const bool whole = seg_tiles == at.tiles;
    const int item = at.b * per + at.hk;
    // logits of this lane's stores: head 2 (lane % 4) + (bit of lane/4), plus 8 per head tile
    float* logits = p.logits + ((long long)at.b * p.Hq + h0 + i4 * 2 + (hr & 1)) * p.cache.capacity();

    // queries as the B operand: lane holds head lane/4 (of the 8 of head tile t)
    uint32_t qb[NT][kSteps][2];
    float mult[NT][2];       // from product to log2 units, for this lane's heads 2i, 2i+1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = hr + 8 * t;
      const bf16* q = p.q + (long long)at.b * p.q_sb + (long long)(h0 + h) * p.q_sh;
      if (!FP8) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          qb[t][s][0] = h < heads ? *reinterpret_cast<const uint32_t*>(q + s * 16 + i4 * 2) : 0u;
          qb[t][s][1] = h < heads ? *reinterpret_cast<const uint32_t*>(q + s * 16 + i4 * 2 + 8) : 0u;
        }
        mult[t][0] = mult[t][1] = fmaxf(p.scale_log2, kTinyScale);
      } else {
        // four neighbouring elements per lane and step: the order in which e4m3 pairs
        // come out of a widened key row
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const uint2 w = h < heads ? *reinterpret_cast<const uint2*>(q + s * 16 + i4 * 4) : make_uint2(0u, 0u);
          qb[t][s][0] = w.x;
          qb[t][s][1] = w.y;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top = fmax3(top, fabsf(__uint_as_float(qb[t][s][e] << 16)),
                        fabsf(__uint_as_float(qb[t][s][e] & 0xffff0000u)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e >= top; clamped so that 2^e and 2^-e are both normal
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 126, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int w = 0; w < 2; ++w)
            qb[t][s][w] = pack_f16x2(__uint_as_float(qb[t][s][w] << 16) * down,
                                     __uint_as_float(qb[t][s][w] & 0xffff0000u) * down);
        const float back = fmaxf(p.scale_log2 * p.cache.k_scale[kvh] *
                                     __uint_as_float((uint32_t)(127 + e) << 23), kTinyScale);
        mult[t][0] = __shfl_sync(0xffffffffu, back, i4 * 8);
        mult[t][1] = __shfl_sync(0xffffffffu, back, i4 * 8 + 4);
      }
    }

    // reference, sum of this lane's keys, and O^T (columns lane/4, +8 of each 16), per head
    float m[NT][2], l[NT][2], o[NT][kSteps][4];
    float peak[FP8 ? NT : 1][2];     // largest logit so far
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = kNegInf;
      if (FP8) peak[t][0] = peak[t][1] = kNegInf;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int c = 0; c < kSteps; ++c) o[t][c][0] = o[t][c][1] = o[t][c][2] = o[t][c][3] = 0.f;
    }

    for (int s = 0; s < seg_tiles; ++s, ++n) {
      const int st = n % ST;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (n / ST) & 1, abort_flag));
      if (!ok) continue;
      const int t_first = (at.tile + s) * L::kKeys;
      const uint32_t loaded = parts[st];
      int live[SETS], most = 0, least = 16;        // keys of a set that exist
#pragma unroll
      for (int u = 0; u < SETS; ++u) {
        live[u] = ((loaded >> part[u]) & 1) ? max(min(len - t_first - k0[u], 16), 0) : 0;
        most = max(most, live[u]);
        least = min(least, live[u]);
      }
      if (most > 0) {
        const uint32_t stage = smem_u32(smem + st * L::kStage);
        if (least < 16) {     // stale rows behind the sequence's end: V = 0
          constexpr int kCh = L::kRow / 16;
#pragma unroll
          for (int u = 0; u < SETS; ++u)
            for (int i = lane; i < (16 - live[u]) * kCh; i += 32) {
              const uint32_t a = chunk(stage + L::kTile + part_off[u], r0[u] + live[u] + i / kCh, i % kCh);
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(0) : "memory");
            }
          __syncwarp();
        }
        // S^T: rows keys, columns heads
        float sc[SETS][NT][4];
#pragma unroll
        for (int u = 0; u < SETS; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t) sc[u][t][0] = sc[u][t][1] = sc[u][t][2] = sc[u][t][3] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; k += FP8 ? 2 : 1) {
#pragma unroll
          for (int u = 0; u < SETS; ++u) {
            uint32_t r[4];
            ldsm4(r, place(stage + off_k[u], FP8 ? k : 2 * k));
            if (!FP8) {
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816<false>(sc[u][t], r, qb[t][k][0], qb[t][k][1]);
            } else {
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                uint32_t a[4];
                e4m3x4_to_f16x2(r[2 * v], &a[0], &a[2]);
                e4m3x4_to_f16x2(r[2 * v + 1], &a[1], &a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma16816<true>(sc[u][t], a, qb[t][k + v][0], qb[t][k + v][1]);
              }
            }
          }
        }
        // softmax over this warp's keys, base 2; value e: key lane/4 + 8 (e/2), head 2i + e%2
        uint32_t pb[SETS][NT][4];        // P^T as the B operand: rounded, remainder
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float x[SETS][4], mx[2] = {kNegInf, kNegInf};
#pragma unroll
          for (int u = 0; u < SETS; ++u) {
            if (least < 16) {       // (mult > 0, so a product of -inf stays -inf)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hr + 8 * (e >> 1) >= live[u]) sc[u][t][e] = kNegInf;
            }
            mx[0] = fmax3(mx[0], sc[u][t][0], sc[u][t][2]);
            mx[1] = fmax3(mx[1], sc[u][t][1], sc[u][t][3]);
            if (p.logits != nullptr) {
              // The four lanes of keys r..r+3 (r = 0 or 4) transpose their 4 x 4 values: lane
              // (half, d) gets the four keys r + 8 half .. of head 2i + d, one 16-byte store
              // in place of four of 4 bytes.
              const bool d1 = hr & 1, half1 = hr & 2;
              const float v0 = sc[u][t][0] * mult[t][0], v1 = sc[u][t][1] * mult[t][1];
              const float v2 = sc[u][t][2] * mult[t][0], v3 = sc[u][t][3] * mult[t][1];
              const float a0 = d1 ? v1 : v0, a1 = d1 ? v3 : v2;
              const float b0 = __shfl_xor_sync(0xffffffffu, d1 ? v0 : v1, 4);
              const float b1 = __shfl_xor_sync(0xffffffffu, d1 ? v2 : v3, 4);
              const float2 y0 = d1 ? make_float2(b0, a0) : make_float2(a0, b0);   // half 0
              const float2 y1 = d1 ? make_float2(b1, a1) : make_float2(a1, b1);   // half 1
              const float2 own = half1 ? y1 : y0;
              const float2 out = half1 ? y0 : y1;
              const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, out.x, 8),
                                             __shfl_xor_sync(0xffffffffu, out.y, 8));
              const int h = i4 * 2 + d1 + 8 * t, j = (hr & 4) + (half1 ? 8 : 0);
              // (slots of the quad behind the end lie inside the row, and are not read)
              if (h < heads && j < live[u])
                *reinterpret_cast<float4*>(logits + (long long)(8 * t) * p.cache.capacity() + t_first +
                                           k0[u] + j) =
                    half1 ? make_float4(got.x, got.y, own.x, own.y)
                          : make_float4(own.x, own.y, got.x, got.y);
            }
          }
#pragma unroll
          for (int d = 0; d < 2; ++d) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx[d] = fmaxf(mx[d], __shfl_xor_sync(0xffffffffu, mx[d], w));
            mx[d] *= mult[t][d];
          }
          // the reference moves only when a head's maximum has left a range around it, which
          // bounds the weights and makes a rescaling of O rare. bf16 weights: up when it has
          // been outgrown by 2^8. f16 weights: also down, so that those of this tile stay clear
          // of that type's lower end, but never 2^kF16Span below the largest maximum so far.
          bool move[2];
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            if (FP8) {
              peak[t][d] = fmaxf(peak[t][d], mx[d]);
              move[d] = fabsf(mx[d] - m[t][d] - 0.5f * (kF16Low + kF16High)) > 0.5f * (kF16High - kF16Low);
            } else {
              move[d] = mx[d] > m[t][d] + 8.f;
            }
          }
          if (__any_sync(0xffffffffu, move[0] || move[1])) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              float to = mx[d];
              if (FP8) {
                move[d] = move[d] && mx[d] > kNegInf;
                to = fmaxf(mx[d] - kF16Set, peak[t][d] - kF16Span);
              }
              const float f = move[d] ? ex2(m[t][d] - to) : 1.f;
              l[t][d] *= f;
#pragma unroll
              for (int c = 0; c < kSteps; ++c) {
                o[t][c][d] *= f;
                o[t][c][2 + d] *= f;
              }
              if (move[d]) m[t][d] = to;
            }
          }
          const float ref[2] = {m[t][0] == kNegInf ? 0.f : m[t][0], m[t][1] == kNegInf ? 0.f : m[t][1]};
#pragma unroll
          for (int u = 0; u < SETS; ++u) {
            // the product fused with the difference: one rounding ahead of the exponential
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][e] = ex2(fmaf(sc[u][t][e], mult[t][e & 1], -ref[e & 1]));
            l[t][0] += x[u][0] + x[u][2];
            l[t][1] += x[u][1] + x[u][3];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float y0 = x[u][2 * w], y1 = x[u][2 * w + 1];
              uint32_t hi, lo;
              split_pair<FP8>(y0, y1, &hi, &lo);
              pb[u][t][w] = transpose8x8(hi);
              pb[u][t][2 + w] = transpose8x8(lo);
            }
          }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < SETS; ++u) {
          if (!FP8) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              uint32_t a[4];
              ldsm4t(a, place(stage + off_v[u], 2 * k));
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<false>(o[t][k], a, pb[u][t][0], pb[u][t][1]);
                mma16816<false>(o[t][k], a, pb[u][t][2], pb[u][t][3]);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < kSteps; k += 2) {
              uint32_t r[4];
              ldsm4t(r, place(stage + off_v[u], k));
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                // a register holds columns (2n, 2n+1) of two keys: regroup by column; the
                // MMA's rows 0-7 take the even columns, rows 8-15 the odd ones
                uint32_t a[4];
                e4m3x4_to_f16x2(__byte_perm(r[2 * v], 0, 0x3120), &a[0], &a[1]);
                e4m3x4_to_f16x2(__byte_perm(r[2 * v + 1], 0, 0x3120), &a[2], &a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  mma16816<true>(o[t][k + v], a, pb[u][t][0], pb[u][t][1]);
                  mma16816<true>(o[t][k + v], a, pb[u][t][2], pb[u][t][3]);
                }
              }
            }
          }
        }
        // the zeroed rows were written through the generic proxy: order them before
        // the next TMA write to this stage
        if (least < 16) fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ------------------------------------------- the four warps' outputs join
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int d = 0; d < 2; ++d) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[t][d] += __shfl_xor_sync(0xffffffffu, l[t][d], w);
        if (hr == 0) xml[warp * L::kRows + 8 * t + 2 * i4 + d] = make_float2(m[t][d], l[t][d]);
      }
    bar_mma_warps();
    const long long slot = (long long)blockIdx.x + item;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // every warp's output against the largest reference, in two rounds through the two
      // buffers: warps 2 and 3 write, warps 0 and 1 add theirs
      float f[2];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        float all = kNegInf;
#pragma unroll
        for (int w = 0; w < 4; ++w) all = fmaxf(all, xml[w * L::kRows + 8 * t + 2 * i4 + d].x);
        f[d] = ex2(m[t][d] - (all == kNegInf ? 0.f : all));
      }
      // in the end 16 lanes per head write C/16 columns each; the statistics are read
      // before the rounds' barriers, behind which a faster warp may write the next item's
      const int row = tid >> 4, g = row + 8 * t, c0 = (tid & 15) * (C / 16);
      float top = kNegInf, sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, xml[w * L::kRows + g].x);
      const float ref = top == kNegInf ? 0.f : top;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 ml = xml[w * L::kRows + g];
        sum += ex2(ml.x - ref) * ml.y;
      }
      float* buf = xo + (warp & 1) * 8 * L::kXRow;
#pragma unroll
      for (int round = 0; round < 2; ++round) {
        if ((warp >> 1) == 1 - round) {
#pragma unroll
          for (int c = 0; c < kSteps; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // e4m3: rows 0-7 of the tile are its even columns, rows 8-15 the odd ones
              const int col = c * 16 + (FP8 ? 2 * hr + (e >> 1) : hr + 8 * (e >> 1));
              float* y = buf + (2 * i4 + (e & 1)) * L::kXRow + col;
              const float v = o[t][c][e] * f[e & 1];
              *y = round == 0 ? v : *y + v;
            }
        }
        bar_mma_warps();
      }
      if (g < heads) {
        const float vs = FP8 ? p.cache.v_scale[kvh] : 1.f;
        const float inv = whole ? vs / sum : vs;
        const float* x0 = xo + row * L::kXRow + c0;
        const float* x1 = x0 + 8 * L::kXRow;
        float y[C / 16];
#pragma unroll
        for (int c = 0; c < C / 16; c += 4) {
          const float4 a = *reinterpret_cast<const float4*>(x0 + c);
          const float4 b = *reinterpret_cast<const float4*>(x1 + c);
          y[c] = (a.x + b.x) * inv;
          y[c + 1] = (a.y + b.y) * inv;
          y[c + 2] = (a.z + b.z) * inv;
          y[c + 3] = (a.w + b.w) * inv;
        }
        if (sum == 0.f)          // no mass: o = 0
#pragma unroll
          for (int c = 0; c < C / 16; ++c) y[c] = 0.f;
        if (whole) {
          bf16* out = p.O + ((long long)at.b * p.Hq + h0 + g) * C + c0;
#pragma unroll
          for (int c = 0; c < C / 16; c += 4)
            *reinterpret_cast<uint2*>(out + c) =
                make_uint2(pack_bf16x2(y[c], y[c + 1]), pack_bf16x2(y[c + 2], y[c + 3]));
        } else {
          float* out = p.part_o + (slot * L::kRows + g) * C + c0;
#pragma unroll
          for (int c = 0; c < C / 16; c += 4)
            *reinterpret_cast<float4*>(out + c) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
        }
        if ((tid & 15) == 0) {
          p.part_ml[slot * L::kRows + g] = make_float2(top, sum);
          if (whole && p.lse != nullptr)
            p.lse[(long long)at.b * p.Hq + h0 + g] = sum == 0.f ? kNegInf : (ref + log2f(sum)) * kLn2;
        }
      }
      if (t + 1 < NT) bar_mma_warps();      // the buffers have been read
    }
    if (tid == 0) {
      if (at.tile == 0) p.seg[item].x = blockIdx.x;
      if (at.tile + seg_tiles == at.tiles) p.seg[item].y = blockIdx.x;
    }
    if (n < mine) dec_next_item<L::kKeys, IDLE>(p, at, per);
  }
}

// ------------------------------------------------------------------- join
// (maximum, sum) of one row over n partials, in log2 units, by one warp: the lanes read
// the partials side by side, so a row of many costs a few load latencies, not n.
__device__ __forceinline__ float2 dec_row_stat(const float2* ml, int rows, int n, int lane) {
  float top = kNegInf, sum = 0.f;       // of this lane's partials
#pragma unroll 2
  for (int s = lane; s < n; s += 32) {
    const float2 v = ml[(long long)s * rows];
    const float up = fmaxf(top, v.x), ref = up == kNegInf ? 0.f : up;
    sum = sum * ex2(top - ref) + v.y * ex2(v.x - ref);
    top = up;
  }
  float all = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
  const float ref = all == kNegInf ? 0.f : all;
  sum *= ex2(top - ref);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return make_float2(ref, sum);
}

// Blocks [0, B * Hq): output and lse of one query head from its partials. The others
// (weights): acc_out[slot] = acc[slot] + sum over the group's heads of the slot's softmax
// weight, from the logits of the split kernel and the joined statistics. Its time is a chain
// of latencies (segment, statistics and values, sum): each warp takes every fourth partial,
// a lane C/32 columns of it, and the values are loaded before the statistics that weigh them
// are known.
template <int C, bool IDLE>
__global__ void __launch_bounds__(kJoinThreads)
decode_join_kernel(const __grid_constant__ DecodeParams p, int rows, int heads_per_tile,
                   int weight_blocks) {
  constexpr int kVec = C / 32;
  __shared__ float red[kJoinThreads / 32][C];
  __shared__ float stat[kDecMaxGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hq = p.Hq, per = p.cache.Hkv * p.HT;
  const int n_join = p.cache.B * Hq;
  grid_dependency_wait();

  if ((int)blockIdx.x < n_join) {
    const int bh = blockIdx.x, b = bh / Hq, h = bh - b * Hq;
    const int kvh = h / p.G, g = h - kvh * p.G;
    const int item = b * per + kvh * p.HT + g / heads_per_tile;
    const int row = g % heads_per_tile;
    const int len = p.length<IDLE>(b);
    const int2 seg = p.seg[item];      // not written for a sequence without keys
    if (len == 0) {                    // no key: o = 0, lse = -inf
      if (tid < C) p.O[(long long)bh * C + tid] = __float2bfloat16(0.f);
      if (tid == 0) {
        if (p.lse != nullptr) p.lse[bh] = kNegInf;
        if (!p.valid<IDLE>(b)) raise_device_error(kErrInvalid);
      }
      return;
    }
    if (seg.x == seg.y) return;        // one CTA had the whole item and finished it
    const int n = seg.y - seg.x + 1;
    const float2* ml = p.part_ml + ((long long)seg.x + item) * rows + row;
    const float* po = p.part_o + (((long long)seg.x + item) * rows + row) * C + lane * kVec;
    const long long step = (long long)rows * C;
    struct alignas(kVec * 4) Vec { float x[kVec]; };
    constexpr int U = 4;
    Vec v[U];
    float m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = warp + 4 * u;
      m[u] = kNegInf;
      if (s < n) {
        v[u] = *reinterpret_cast<const Vec*>(po + s * step);
        m[u] = ml[(long long)s * rows].x;
      }
    }
    const float2 st = dec_row_stat(ml, rows, n, lane);       // every warp for itself
    float y[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) y[c] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (warp + 4 * u < n) {
        const float f = ex2(m[u] - st.x);
#pragma unroll
        for (int c = 0; c < kVec; ++c) y[c] += f * v[u].x[c];
      }
#pragma unroll 4
    for (int s = warp + 4 * U; s < n; s += 4) {
      const Vec w = *reinterpret_cast<const Vec*>(po + s * step);
      const float f = ex2(ml[(long long)s * rows].x - st.x);
#pragma unroll
      for (int c = 0; c < kVec; ++c) y[c] += f * w.x[c];
    }
#pragma unroll
    for (int c = 0; c < kVec; ++c) red[warp][lane * kVec + c] = y[c];
    __syncthreads();
    if (tid < C) {
      const float o = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
      p.O[(long long)bh * C + tid] = __float2bfloat16(st.y == 0.f ? 0.f : o / st.y);
      if (tid == 0 && p.lse != nullptr)
        p.lse[bh] = st.y == 0.f ? kNegInf : (st.x + log2f(st.y)) * kLn2;
    }
    return;
  }

  // ---------------------------------------------------------------- weights
  const int wb = blockIdx.x - n_join;
  const int pair = wb / weight_blocks, first = wb - pair * weight_blocks;
  const int b = pair / p.cache.Hkv, kvh = pair - b * p.cache.Hkv;
  const int len = p.length<IDLE>(b);
  if (first * (kJoinThreads * 4) >= len) return;
  const int cap = p.cache.capacity();
  const float* logits = p.logits + ((long long)b * Hq + kvh * p.G) * cap;
  // four neighbouring slots per thread (never across a page): 16-byte loads. The first kPre
  // heads' logits and the old weights are on their way one round ahead, the first round's
  // while the statistics are worked out.
  constexpr int kPre = 4;
  int j = (first * kJoinThreads + tid) * 4;
  long long at = -1;
  float4 old, x[kPre];
  auto load = [&]() {
    at = j < len ? p.cache.slot_index(b, kvh, j) : -1;
    if (at < 0) return;                // a bad page: the split kernel raised the error
    old = *reinterpret_cast<const float4*>(p.cache.acc + at);
#pragma unroll
    for (int g = 0; g < kPre; ++g)
      if (g < p.G) x[g] = *reinterpret_cast<const float4*>(logits + (long long)g * cap + j);
  };
  load();
  // base-2 log-sum-exp of every head of the group
  for (int g = warp; g < p.G; g += kJoinThreads / 32) {
    const int item = b * per + kvh * p.HT + g / heads_per_tile;
    const int2 seg = p.seg[item];
    const float2 st = dec_row_stat(p.part_ml + ((long long)seg.x + item) * rows + g % heads_per_tile,
                                   rows, seg.y - seg.x + 1, lane);
    // +inf: every weight of this head is 0 (it saw no mass)
    if (lane == 0) stat[g] = st.y == 0.f ? -kNegInf : st.x + log2f(st.y);
  }
  __syncthreads();
  while (j < len) {
    const int j_now = j;
    const long long at_now = at;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v, float l) {
      w.x += ex2(v.x - l);
      w.y += ex2(v.y - l);
      w.z += ex2(v.z - l);
      w.w += ex2(v.w - l);
    };
    if (at_now >= 0) {
#pragma unroll
      for (int g = 0; g < kPre; ++g)
        if (g < p.G) add(x[g], stat[g]);
#pragma unroll 2
      for (int g = kPre; g < p.G; ++g)
        add(*reinterpret_cast<const float4*>(logits + (long long)g * cap + j_now), stat[g]);
      w = make_float4(old.x + w.x, old.y + w.y, old.z + w.z, old.w + w.w);
    }
    j += weight_blocks * kJoinThreads * 4;
    load();
    if (at_now < 0) continue;
    if (j_now + 4 <= len) {
      *reinterpret_cast<float4*>(p.acc_out + at_now) = w;
    } else {                           // the slots behind the end stay as they were
      p.acc_out[at_now] = w.x;
      if (j_now + 1 < len) p.acc_out[at_now + 1] = w.y;
      if (j_now + 2 < len) p.acc_out[at_now + 2] = w.z;
    }
  }
}

}  // namespace xattn
