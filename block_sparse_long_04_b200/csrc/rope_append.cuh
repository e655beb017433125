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
// that neighbouring threads read neighbouring words) and its loop over the heads holds
// nothing but loads, 16 products and stores, with kUnroll rows in flight.
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
  // length of sequence b, clamped to what its table can name
  __device__ __forceinline__ int length(int b) const {
    const int n = __ldg(lens + b);
    return n < 0 ? 0 : min(n, capacity());
  }
  __device__ __forceinline__ bool length_valid(int b) const {
    const int n = __ldg(lens + b);
    return n >= 0 && n <= capacity();
  }
  // index of (slot, kv head) in a [num_pages, Hkv, page] pool, -1 for a bad page id;
  // the slot must lie in [0, capacity)
  __device__ __forceinline__ long long slot_index(int b, int kvh, int slot) const {
    const int pid = __ldg(page_table + (long long)b * max_pages + (slot >> page_log2));
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
// result. With r = RN(1/scale), q = RN(y r), the remainder y - q scale is exact in one FMA
// and RN(q + remainder r) is the rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990),
// as long as nothing over- or underflows: for scales between 2^-60 and 2^60 that leaves
// quotients far outside e4m3's range, whose uncorrected q saturates (or vanishes) alike.
// Other scales take the division itself.
struct E4m3Scale {
  float scale, inv;
  bool plain;
};
__device__ __forceinline__ E4m3Scale e4m3_scale(float scale) {
  const bool plain = !(scale > 0x1p-60f && scale < 0x1p60f);
  return {scale, __frcp_rn(scale), plain};
}
__device__ __forceinline__ float e4m3_quotient(float y, const E4m3Scale& s) {
  if (s.plain) return __fdiv_rn(y, s.scale);
  const float q = y * s.inv;
  const float exact = fmaf(fmaf(-q, s.scale, y), s.inv, q);
  // q will do where it is zero (the correction would lose the sign of -0), beyond e4m3's
  // largest, infinite or NaN: one comparison of the bits of |q|, 1024.f = 0x44800000
  return (__float_as_uint(fabsf(q)) - 1u) < 0x447fffffu ? exact : q;
}
__device__ __forceinline__ uint2 pack_e4m3x8(const float* y, const E4m3Scale& s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(
        make_float2(e4m3_quotient(y[2 * i], s), e4m3_quotient(y[2 * i + 1], s)), __NV_SATFINITE,
        __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
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

// DST: where keys (and values) go. 0: dense rows ko, no values; 1: bf16 pages; 2: e4m3 pages.
template <int C, bool ROPE, int DST>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kTpr = C / 16;                  // threads per row
  constexpr int kRows = kRopeThreads / kTpr;    // rows per sweep of the CTA
  constexpr int kUnroll = 2;
  // (cos, sin) of token t's pairs: 8 pairs of a thread lie C/16 apart; 8 words between tokens
  // keep the tokens of a warp on different banks
  constexpr int kCsRow = C / 2 + 8;
  __shared__ float2 cs[ROPE ? kRopeMaxTokens * kCsRow : 1];
  __shared__ long long dst_row[kRopeMaxTokens];   // pool index at head 0, -1: none

  const int b = blockIdx.y, TT = 1 << p.tokens_log2;
  const int m0 = blockIdx.x << p.tokens_log2;
  const int tid = threadIdx.x;
  int n_tok = min(TT, p.M - m0);                // tokens of this tile
  int first_slot = 0;

  if (DST != 0) {
    int nn = p.M;
    if (p.n_new != nullptr) {
      const int want = __ldg(p.n_new + b);
      nn = min(max(want, 0), p.M);
      if (want != nn && tid == 0) raise_device_error(kErrInvalid);
    }
    n_tok = min(n_tok, nn - m0);
    if (n_tok <= 0) return;
    const int len = __ldg(p.cache.lens + b);
    first_slot = len - nn + m0;
    if (tid < n_tok) {
      const int slot = first_slot + tid;
      long long r = -1;
      if (len >= nn && len <= p.cache.capacity()) r = p.cache.slot_index(b, 0, slot);
      if (r < 0) raise_device_error(kErrInvalid);
      dst_row[tid] = r;
    }
    // new slots: no weight yet, and the token's index in its sequence
    if (p.cache.acc != nullptr || p.cache.ordinal != nullptr) {
      const int seen = p.seen != nullptr ? __ldg(p.seen + b) : len;
      __syncthreads();
      for (int i = tid; i < n_tok * p.cache.Hkv; i += kRopeThreads) {
        const int h = i / n_tok, t = i - h * n_tok;
        const long long r = dst_row[t];
        if (r < 0) continue;
        const long long at = r + ((long long)h << p.cache.page_log2);
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
      const double turns = (double)__ldg(pos + t * p.axes + ax) * __ldg(p.inv_freq + pr) *
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

  const int lane_r = tid / kTpr, t8 = tid % kTpr;
  const int rotated = ROPE ? 2 * p.pairs / 8 : 0;     // chunks that rotate (pairs % 8 == 0)
  // the two 8-element chunks of this thread
  int ca = t8, cb = t8 + kTpr;
  if (ROPE && !p.interleaved && rotated < C / 8) {
    const int hp = rotated / 2;
    if (t8 < hp) { ca = t8; cb = t8 + hp; }
    else { ca = rotated + 2 * (t8 - hp); cb = ca + 1; }
  }
  const bool rope_a = ca < rotated, rope_b = cb < rotated;
  float2 w[ROPE ? 8 : 1];
  if (ROPE) {
    // unused ones (chunks that pass through, tokens behind the tile's last) are never applied
    const float2* row = cs + (lane_r & (TT - 1)) * kCsRow + t8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = (p.interleaved ? (i < 4 ? rope_a : rope_b) : rope_a) ? row[i * kTpr] : make_float2(1.f, 0.f);
  }
  const int nq = p.q.heads, nk = p.k.heads, nv = DST != 0 ? p.v.heads : 0;
  const int rows = (nq + nk + nv) << p.tokens_log2;

  for (int r0 = lane_r; r0 < rows; r0 += kUnroll * kRows) {
    uint4 xa[kUnroll], xb[kUnroll];
    int head[kUnroll], tok[kUnroll];
    bool live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kRows;
      tok[u] = r & (TT - 1);
      head[u] = r >> p.tokens_log2;
      live[u] = r < rows && tok[u] < n_tok;
      if (live[u]) {
        const int h = head[u];
        const HeadsView& src = h < nq ? p.q : (h < nq + nk ? p.k : p.v);
        const int hh = h < nq ? h : (h < nq + nk ? h - nq : h - nq - nk);
        const bf16* x = src.data + (long long)b * src.sb + (long long)hh * src.sh +
                        (long long)(m0 + tok[u]) * src.sm;
        xa[u] = *reinterpret_cast<const uint4*>(x + ca * 8);
        xb[u] = *reinterpret_cast<const uint4*>(x + cb * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!live[u]) continue;
      const int h = head[u];
      const bool is_q = h < nq, is_v = h >= nq + nk;
      float a[8], c[8];
      const bool raw_copy = DST != 2 || is_q;     // bf16 out: an unrotated chunk stays as it is
      const bool rot_a = ROPE && !is_v && rope_a, rot_b = ROPE && !is_v && rope_b;
      if (rot_a || rot_b || !raw_copy) {
        unpack_bf16x8(xa[u], a);
        unpack_bf16x8(xb[u], c);
      }
      if (ROPE && !is_v) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a1 = a[2 * i], a2 = a[2 * i + 1], c1 = c[2 * i], c2 = c[2 * i + 1];
            a[2 * i] = a1 * w[i].x - a2 * w[i].y;
            a[2 * i + 1] = a2 * w[i].x + a1 * w[i].y;
            c[2 * i] = c1 * w[4 + i].x - c2 * w[4 + i].y;
            c[2 * i + 1] = c2 * w[4 + i].x + c1 * w[4 + i].y;
          }
        } else {                     // cb = ca + pairs/8 holds the partners
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x1 = a[i], x2 = c[i];
            a[i] = x1 * w[i].x - x2 * w[i].y;
            c[i] = x2 * w[i].x + x1 * w[i].y;
          }
        }
      }
      if (DST == 0 || is_q) {
        const HeadsView& dst = is_q ? p.qo : p.ko;
        const int hh = is_q ? h : h - nq;
        bf16* y = dst.data + (long long)b * dst.sb + (long long)hh * dst.sh +
                  (long long)(m0 + tok[u]) * dst.sm;
        *reinterpret_cast<uint4*>(y + ca * 8) = rot_a ? pack_bf16x8(a) : xa[u];
        *reinterpret_cast<uint4*>(y + cb * 8) = rot_b ? pack_bf16x8(c) : xb[u];
      } else {
        const int hh = is_v ? h - nq - nk : h - nq;
        const long long r = dst_row[tok[u]];
        if (r < 0) continue;
        const long long at = (r + ((long long)hh << p.cache.page_log2)) * C;
        void* pages = is_v ? p.cache.v_pages : p.cache.k_pages;
        if (DST == 1) {
          bf16* y = static_cast<bf16*>(pages) + at;
          *reinterpret_cast<uint4*>(y + ca * 8) = rot_a ? pack_bf16x8(a) : xa[u];
          *reinterpret_cast<uint4*>(y + cb * 8) = rot_b ? pack_bf16x8(c) : xb[u];
        } else {
          const E4m3Scale sc = e4m3_scale(__ldg((is_v ? p.cache.v_scale : p.cache.k_scale) + hh));
          uint8_t* y = static_cast<uint8_t*>(pages) + at;
          *reinterpret_cast<uint2*>(y + ca * 8) = pack_e4m3x8(a, sc);
          *reinterpret_cast<uint2*>(y + cb * 8) = pack_e4m3x8(c, sc);
        }
      }
    }
  }
}

}  // namespace xattn
