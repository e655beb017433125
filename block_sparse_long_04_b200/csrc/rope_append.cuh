// Rotary positions and the append to a paged key-value cache, one kernel.
//
// Rotation. Pair p of a row (elements p and p+P, or 2p and 2p+1) turns by
//   angle = pos[axis(p)] * inv_freq[p],
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin);
// the inverse (and the gradient) turns by -angle. The angle is formed in 64 bits and
// reduced to a fraction of a turn there: at position 262144 a 32-bit product would be
// off by up to 0.016 rad. From the reduced angle on, 32 bits are enough (error below
// 2^-22 rad), and the result is rounded once, to bf16 or to the cache's e4m3.
//
// The work is a copy: 4 bytes per element (bf16 in and out), so the bound is HBM. One
// CTA owns a tile of tokens of one sequence and ALL their heads: the sines of a token
// are computed once, into shared memory, and serve its Hq + Hkv heads (for 32 + 8 heads
// the 64-bit work is 1/40 per row). A row is C/16 threads, each with two 16-byte chunks
// (the two halves of its pairs when the pairs are split across the row). The rows of a
// sweep are a multiple of the tile's tokens, so a thread meets the same token and the same
// 8 pairs in every row: it takes their sines into registers once (from a table laid out so
// that neighbouring threads read neighbouring words), and its loop over the heads is a
// strided copy with 16 products in it, four rows in flight. What the loop must not hold is
// address arithmetic: with it, and the sines read per row, a 32K prompt of 32 + 8 heads
// took 180 us, 120 us with the sines in registers, 107 us so (0.67 GB, 6.2 TB/s; the
// 118784-token layer of 24 + 24 heads 437 us, 6.7 TB/s; 32K tokens of 8 heads into bf16 pages
// 44 us, 6.1 TB/s, into e4m3 pages 38 us, 5.3 TB/s; rotated with 32 query heads on the way 129 us
// into either). The e4m3 instance without rotation is held to 64 registers and spills 100 bytes
// of them. Two resident CTAs with four rows in flight and three with two measured
// alike, more CTAs slower.
//
// Append. Token t of sequence b goes to slot lens[b] - n_new[b] + t; its page and row
// are resolved once per token. A page id or slot out of range writes nothing and raises
// XATTN_EINVAL in the device error word.
#pragma once
#include <cuda_fp8.h>
#include "common.cuh"

namespace xattn {

constexpr int kErrInvalid = 1;      // XATTN_EINVAL, raised by kernels
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;  // tokens per CTA

// A paged cache as the kernels see it (see xattn_cache in the header).
struct CacheView {
  void* k_pages;
  void* v_pages;
  const float* k_scale;
  const float* v_scale;
  float* acc;
  int32_t* ordinal;
  const int32_t* page_table;
  const int32_t* lens;
  int B, Hkv, page_log2, num_pages, max_pages;

  __device__ __forceinline__ int capacity() const { return max_pages << page_log2; }
  // Plain loads throughout: the read-only path must not be used for what an earlier kernel
  // wrote while this one was already being set up (see grid_dependency_wait).
  __device__ __forceinline__ bool length_valid(int b) const {
    return lens[b] >= 0 && lens[b] <= capacity();
  }
  // slots of sequence b; 0 for a length that its table cannot hold
  __device__ __forceinline__ int length(int b) const {
    const int n = lens[b];
    return n <= capacity() ? max(n, 0) : 0;
  }
  // index of (slot, kv head) in a [num_pages, Hkv, page] pool, -1 for a bad page id;
  // the slot must lie in [0, capacity)
  __device__ __forceinline__ long long slot_index(int b, int kvh, int slot) const {
    const int pid = page_table[(long long)b * max_pages + (slot >> page_log2)];
    if (pid < 0 || pid >= num_pages) return -1;
    return ((((long long)pid * Hkv + kvh) << page_log2) + (slot & ((1 << page_log2) - 1)));
  }
};

// bf16 rows [B, heads, M, C] at element strides
struct HeadsView {
  bf16* data;
  long long sb, sh, sm;
  int heads;
};

struct RopeParams {
  HeadsView q, k, v, qo, ko;
  const int32_t* pos;       // [1 or B, M, axes]
  const double* inv_freq;   // [pairs]
  long long pos_sb;         // elements between sequences (0: shared)
  int axes, end0, end1, end2;   // pairs of axis a end at end_a
  int pairs, interleaved;
  float sign;               // -1: inverse
  CacheView cache;
  const int32_t* n_new;
  const int32_t* seen;
  int M, tokens_log2;
};

// y / scale for the e4m3 conversion. The quotient must be the correctly rounded one: where it
// falls on the middle between two e4m3 values, one unit too much or too little turns the
// result. With r = RN(1/d), q = RN(x r), the remainder q d - x is exact in one FMA and
// RN(q - remainder r) is the rounded quotient x / d (Markstein, IBM J. Res. Dev. 34, 1990),
// as long as nothing over- or underflows. So scale = d 2^k with d in [1, 2), and x = y 2^-k:
// what that overflows saturates anyway, what it underflows vanishes. (A division per
// element made the append of a 32K prompt a fifth ALU work, and its code ten times longer.)
struct E4m3Scale {
  float d, inv, pow;
};
__device__ __forceinline__ E4m3Scale e4m3_scale(float scale) {
  const int k = max((int)(__float_as_uint(scale) >> 23) - 127, -126);   // 2^k; subnormals: 2^-126
  // 2^-k: normal for k <= 126, and for k = 127 the subnormal 2^-127
  const float pow = k < 127 ? __uint_as_float((uint32_t)(127 - k) << 23) : __uint_as_float(0x00400000u);
  const float d = scale * pow;
  return {d, __frcp_rn(d), pow};
}
// 16 quotients as e4m3, two 8-byte chunks
__device__ __forceinline__ void pack_e4m3x16(const float* y, const E4m3Scale& s, uint2* out0, uint2* out1) {
  float q[16];
  float top = 0.f;
  const float2 inv = make_float2(s.inv, s.inv), d = make_float2(s.d, s.d);
  const float2 minus_inv = make_float2(-s.inv, -s.inv), pow = make_float2(s.pow, s.pow);
  const float2 zero = make_float2(-0.f, -0.f);      // x + -0 is x, of either sign
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 x = ffma2(make_float2(y[i], y[i + 1]), pow, zero);
    const float2 r = ffma2(x, inv, zero);
    const float2 e = ffma2(ffma2(r, d, make_float2(-x.x, -x.y)), minus_inv, r);
    q[i] = e.x;
    q[i + 1] = e.y;
    top = fmax3(top, fabsf(r.x), fabsf(r.y));
  }
  if (top >= 1024.f) {      // far beyond the largest, or infinite (no remainder): saturate
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float r = y[i] * s.pow * s.inv;
      q[i] = fabsf(r) >= 1024.f ? r : q[i];
    }
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  *out0 = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  *out1 = make_uint2(w[4] | (w[5] << 16), w[6] | (w[7] << 16));
}
__device__ __forceinline__ void unpack_bf16x8(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// How a thread's two chunks rotate.
struct RopeLane {
  int ca, cb;               // their indices in the row
  bool rot_a, rot_b;        // do they rotate
  bool interleaved;
};

// Rows of one tensor, one token, heads h, h + step, ... < heads: x and y point at this
// thread's first row, xs and ys are bytes from one of its rows to the next. FP8: y is e4m3.
template <int C, bool ROT, bool FP8>
__device__ __forceinline__ void rope_rows(const char* x, long long xs, char* y, long long ys, int h,
                                          int step, int heads, const RopeLane& t, const float2* w,
                                          const float* scales) {
  constexpr int U = 4;                       // rows in flight
  constexpr int kOut = FP8 ? 8 : 16;         // bytes of a stored chunk
  x += t.ca * 16;
  y += t.ca * kOut;
  const int bx = (t.cb - t.ca) * 16, by = (t.cb - t.ca) * kOut;
#pragma unroll 1
  for (; h < heads; h += U * step) {
    uint4 xa[U], xb[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * step < heads) {
        xa[u] = *reinterpret_cast<const uint4*>(x + u * xs);
        xb[u] = *reinterpret_cast<const uint4*>(x + u * xs + bx);
      }
    x += U * xs;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u * step >= heads) break;
      if (!FP8 && !ROT) {
        *reinterpret_cast<uint4*>(y) = xa[u];
        *reinterpret_cast<uint4*>(y + by) = xb[u];
      } else {
        float v[16];
        unpack_bf16x8(xa[u], v);
        unpack_bf16x8(xb[u], v + 8);
        if (ROT) {
          if (t.interleaved) {               // w is (1, 0) for a chunk that passes through
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x1 = v[2 * i], x2 = v[2 * i + 1];
              v[2 * i] = x1 * w[i].x - x2 * w[i].y;
              v[2 * i + 1] = x2 * w[i].x + x1 * w[i].y;
            }
          } else {                           // chunk cb holds the partners of chunk ca
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x1 = v[i], x2 = v[8 + i];
              v[i] = x1 * w[i].x - x2 * w[i].y;
              v[8 + i] = x2 * w[i].x + x1 * w[i].y;
            }
          }
        }
        if (FP8) {
          uint2 a, b;
          // what passes through is not turned by (1, 0): that would make NaN of infinities
          if (ROT && !t.rot_a) unpack_bf16x8(xa[u], v);
          if (ROT && !t.rot_b) unpack_bf16x8(xb[u], v + 8);
          pack_e4m3x16(v, e4m3_scale(scales[h + u * step]), &a, &b);
          *reinterpret_cast<uint2*>(y) = a;
          *reinterpret_cast<uint2*>(y + by) = b;
        } else {
          *reinterpret_cast<uint4*>(y) = t.rot_a ? pack_bf16x8(v) : xa[u];
          *reinterpret_cast<uint4*>(y + by) = t.rot_b ? pack_bf16x8(v + 8) : xb[u];
        }
      }
      y += ys;
    }
  }
}

// DST: where keys (and values) go. 0: dense rows ko, no values; 1: bf16 pages; 2: e4m3 pages.
template <int C, bool ROPE, int DST>
__global__ void __launch_bounds__(kRopeThreads, ROPE ? 2 : 4)
rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kTpr = C / 16;                  // threads per row
  constexpr int kRows = kRopeThreads / kTpr;    // rows per sweep of the CTA
  // (cos, sin) of token t's pairs: 8 pairs of a thread lie C/16 apart; 8 words between tokens
  // keep the tokens of a warp on different banks
  constexpr int kCsRow = C / 2 + 8;
  __shared__ float2 cs[ROPE ? kRopeMaxTokens * kCsRow : 1];
  __shared__ long long dst_row[kRopeMaxTokens];   // pool index at head 0, -1: none

  grid_dependency_wait();
  const int b = blockIdx.y, TT = 1 << p.tokens_log2;
  const int m0 = blockIdx.x << p.tokens_log2;
  const int tid = threadIdx.x;
  int n_tok = min(TT, p.M - m0);                // tokens of this tile

  if (DST != 0) {
    const int nn = p.n_new != nullptr ? p.n_new[b] : p.M;
    const int len = p.cache.lens[b];
    if (nn < 0 || nn > p.M || nn > len || len > p.cache.capacity()) {
      if (tid == 0) raise_device_error(kErrInvalid);
      return;
    }
    n_tok = min(n_tok, nn - m0);
    if (n_tok <= 0) return;
    if (tid < n_tok) {
      const long long r = p.cache.slot_index(b, 0, len - nn + m0 + tid);
      if (r < 0) raise_device_error(kErrInvalid);
      dst_row[tid] = r;
    }
    // new slots: no weight yet, and the token's index in its sequence
    if (p.cache.acc != nullptr || p.cache.ordinal != nullptr) {
      const int seen = p.seen != nullptr ? p.seen[b] : len;
      __syncthreads();
      for (int i = tid; i < p.cache.Hkv << p.tokens_log2; i += kRopeThreads) {
        const int t = i & (TT - 1);
        const long long r = t < n_tok ? dst_row[t] : -1;
        if (r < 0) continue;
        const long long at = r + ((long long)(i >> p.tokens_log2) << p.cache.page_log2);
        if (p.cache.acc != nullptr) p.cache.acc[at] = 0.f;
        if (p.cache.ordinal != nullptr) p.cache.ordinal[at] = seen - nn + m0 + t;
      }
    }
  }
  if (ROPE) {
    const int P = p.pairs;
    const int32_t* pos = p.pos + (long long)b * p.pos_sb + (long long)m0 * p.axes;
    for (int i = tid; i < n_tok * P; i += kRopeThreads) {
      const int t = i / P, pr = i - t * P;
      const int ax = (pr >= p.end0) + (pr >= p.end1) + (pr >= p.end2);
      // turns = pos * inv_freq / (2 pi), then its fraction in [-1/2, 1/2]
      const double turns = (double)pos[t * p.axes + ax] * p.inv_freq[pr] *
                           0.15915494309189533577;
      const float half_turns = (float)(2.0 * (turns - rint(turns)));
      float s, c;
      sincospif(half_turns, &s, &c);
      // pair pr belongs to chunk pr/4 (interleaved; thread chunk % kTpr, its first or second
      // one) or to thread pr/8
      const int at = p.interleaved ? ((pr >> 2) / kTpr * 4 + (pr & 3)) * kTpr + (pr >> 2) % kTpr
                                   : (pr & 7) * kTpr + (pr >> 3);
      cs[t * kCsRow + at] = make_float2(c, s * p.sign);
    }
  }
  __syncthreads();

  // this thread's row (token and first head) and its two chunks of every row
  const int lane_r = tid / kTpr, t8 = tid % kTpr;
  const int tok = lane_r & (TT - 1), h0 = lane_r >> p.tokens_log2, step = kRows >> p.tokens_log2;
  if (tok >= n_tok) return;
  const int rotated = ROPE ? 2 * p.pairs / 8 : 0;     // chunks that rotate (pairs % 8 == 0)
  RopeLane t;
  t.ca = t8;
  t.cb = t8 + kTpr;
  if (ROPE && !p.interleaved && rotated < C / 8) {
    const int hp = rotated / 2;
    if (t8 < hp) { t.ca = t8; t.cb = t8 + hp; }
    else { t.ca = rotated + 2 * (t8 - hp); t.cb = t.ca + 1; }
  }
  t.rot_a = t.ca < rotated;
  t.rot_b = t.cb < rotated;
  t.interleaved = ROPE && p.interleaved;
  float2 w[ROPE ? 8 : 1];
  if (ROPE) {
    const float2* row = cs + tok * kCsRow + t8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = (t.interleaved && i >= 4 ? t.rot_b : t.rot_a) ? row[i * kTpr] : make_float2(1.f, 0.f);
  }
  // this thread's first row of a strided tensor, and the bytes to its next one
  auto row_of = [&](const HeadsView& v) -> char* {
    return reinterpret_cast<char*>(v.data + (long long)b * v.sb + (long long)h0 * v.sh +
                                   (long long)(m0 + tok) * v.sm);
  };
  auto step_of = [&](const HeadsView& v) -> long long { return v.sh * step * 2; };
  if (ROPE)
    rope_rows<C, true, false>(row_of(p.q), step_of(p.q), row_of(p.qo), step_of(p.qo), h0, step,
                              p.q.heads, t, w, nullptr);
  if (DST == 0) {
    rope_rows<C, true, false>(row_of(p.k), step_of(p.k), row_of(p.ko), step_of(p.ko), h0, step,
                              p.k.heads, t, w, nullptr);
  } else {
    const long long r = dst_row[tok];
    if (r < 0) return;
    constexpr int kBytes = C * (DST == 1 ? 2 : 1);
    const long long at = (r + ((long long)h0 << p.cache.page_log2)) * kBytes;
    const long long ys = ((long long)step << p.cache.page_log2) * kBytes;
    rope_rows<C, ROPE, DST == 2>(row_of(p.k), step_of(p.k), static_cast<char*>(p.cache.k_pages) + at,
                                 ys, h0, step, p.k.heads, t, w, p.cache.k_scale);
    rope_rows<C, false, DST == 2>(row_of(p.v), step_of(p.v), static_cast<char*>(p.cache.v_pages) + at,
                                  ys, h0, step, p.v.heads, t, w, p.cache.v_scale);
  }
}

}  // namespace xattn
