// Argument checks, workspace sizing and launches of the decoding operators (rotary
// positions, paged cache, decode attention, eviction). Included by xattn_api.cu, whose
// helpers it uses; the contract of every entry point is documented in include/xattn.h.
#pragma once
#include "decode.cuh"
#include "evict.cuh"
#include "rope_append.cuh"

namespace {

inline int ilog2(int v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

// Launches `kern` so that it may be set up before the kernel ahead of it in the stream has
// ended. Every kernel launched here begins with grid_dependency_wait(), which waits for
// that kernel (whatever it is) to complete; so stream order holds for all they read and
// write, and only the launch latency overlaps: about 1 us of a decoding step's 4 to 9 us
// per call. `cluster` CTAs along x form a cluster.
template <typename... P, typename... A>
int launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
           const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? launch_status() : XATTN_ECUDA;
}

bool page_supported(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// What every entry point asks of a cache. *empty: nothing to do (B or Hkv is 0).
int check_cache(const xattn_cache* c, bool* empty) {
  *empty = false;
  if (c == nullptr) return XATTN_EINVAL;
  if (c->B < 0 || c->Hkv < 0 || c->C <= 0 || c->page <= 0 || c->num_pages < 0 || c->max_pages < 0)
    return XATTN_EINVAL;
  if (c->kv_type != XATTN_KV_BF16 && c->kv_type != XATTN_KV_E4M3) return XATTN_EINVAL;
  if (c->C != 64 && c->C != 128) return XATTN_EUNSUPPORTED;
  if (!page_supported(c->page)) return XATTN_EUNSUPPORTED;
  if ((long long)c->max_pages * c->page > (1LL << 30)) return XATTN_EUNSUPPORTED;
  // rows of a pool are TMA coordinates
  if ((long long)c->num_pages * c->Hkv * c->page >= (1LL << 31)) return XATTN_EUNSUPPORTED;
  if ((long long)c->B * c->Hkv > 65535 || c->B > 65535) return XATTN_EUNSUPPORTED;
  if (c->B == 0 || c->Hkv == 0) {
    *empty = true;
    return XATTN_OK;
  }
  if (c->num_pages == 0 || c->max_pages == 0) return XATTN_EINVAL;
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->lens) return XATTN_EINVAL;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return XATTN_EINVAL;
  if (c->kv_type == XATTN_KV_E4M3 && (!c->k_scale || !c->v_scale)) return XATTN_EINVAL;
  if (!aligned16(c->acc) || !aligned16(c->ordinal)) return XATTN_EINVAL;
  return XATTN_OK;
}

CacheView view_of(const xattn_cache* c) {
  CacheView v;
  v.k_pages = c->k_pages;
  v.v_pages = c->v_pages;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.acc = c->acc;
  v.ordinal = c->ordinal;
  v.page_table = c->page_table;
  v.lens = c->lens;
  v.B = c->B;
  v.Hkv = c->Hkv;
  v.page_log2 = ilog2(c->page);
  v.num_pages = c->num_pages;
  v.max_pages = c->max_pages;
  return v;
}

// Rows [B, heads, M, C] at element strides: 16-byte vectors, and no two rows of an
// output may be the same one.
int check_heads(const xattn_heads* x, int B, int M, bool output) {
  if (x == nullptr || x->heads < 0) return XATTN_EINVAL;
  if (x->heads == 0 || B == 0 || M == 0) return XATTN_OK;
  if (x->data == nullptr || !aligned16(x->data)) return XATTN_EINVAL;
  if ((x->stride_b | x->stride_h | x->stride_m) % 8 != 0) return XATTN_EUNSUPPORTED;
  if (output && ((B > 1 && x->stride_b == 0) || (x->heads > 1 && x->stride_h == 0) ||
                 (M > 1 && x->stride_m == 0)))
    return XATTN_EINVAL;
  return XATTN_OK;
}

HeadsView view_of(const xattn_heads* x) {
  HeadsView v;
  v.data = x ? static_cast<bf16*>(x->data) : nullptr;
  v.sb = x ? x->stride_b : 0;
  v.sh = x ? x->stride_h : 0;
  v.sm = x ? x->stride_m : 0;
  v.heads = x ? x->heads : 0;
  return v;
}

int check_rotary(const xattn_rotary* r, int B, int M, int C) {
  if (r == nullptr) return XATTN_EINVAL;
  if (r->axes < 1 || r->axes > XATTN_ROPE_MAX_AXES) return XATTN_EINVAL;
  long long pairs = 0;
  for (int a = 0; a < r->axes; ++a) {
    if (r->sections[a] < 0) return XATTN_EINVAL;
    pairs += r->sections[a];
  }
  if (pairs == 0 || pairs > C / 2) return XATTN_EINVAL;
  if (pairs % 8 != 0) return XATTN_EUNSUPPORTED;
  if (r->pos_batch != 1 && r->pos_batch != B) return XATTN_EINVAL;
  if (B > 0 && M > 0 && (!r->pos || !r->inv_freq)) return XATTN_EINVAL;
  return XATTN_OK;
}

void set_rotary(RopeParams* p, const xattn_rotary* r, int M, bool inverse) {
  int end[XATTN_ROPE_MAX_AXES], n = 0;
  for (int a = 0; a < XATTN_ROPE_MAX_AXES; ++a) {
    if (a < r->axes) n += r->sections[a];
    // axes that do not exist begin behind the last pair
    end[a] = a + 1 < r->axes ? n : (1 << 30);
  }
  p->pos = r->pos;
  p->inv_freq = r->inv_freq;
  p->pos_sb = r->pos_batch == 1 ? 0 : (long long)M * r->axes;
  p->axes = r->axes;
  p->end0 = end[0];
  p->end1 = end[1];
  p->end2 = end[2];
  p->pairs = n;
  p->interleaved = r->interleaved ? 1 : 0;
  p->sign = inverse ? -1.f : 1.f;
}

template <int C>
int launch_rope_append(RopeParams& p, bool rope, int dst, int B, int M, cudaStream_t st) {
  // 16 tokens per CTA where that fills the GPU twice over, else 4, else 1
  p.M = M;
  p.tokens_log2 = 0;
  for (int l = 4; l > 0; l -= 2)
    if ((long long)B * ((M + (1 << l) - 1) >> l) >= 296) {
      p.tokens_log2 = l;
      break;
    }
  const dim3 grid((unsigned)((M + (1LL << p.tokens_log2) - 1) >> p.tokens_log2), (unsigned)B);
  auto kern = dst == 0 ? rope_append_kernel<C, true, 0>
              : dst == 1 ? (rope ? rope_append_kernel<C, true, 1> : rope_append_kernel<C, false, 1>)
                         : (rope ? rope_append_kernel<C, true, 2> : rope_append_kernel<C, false, 2>);
  return launch(kern, grid, kRopeThreads, 0, st, 1, p);
}

int append_common(const xattn_heads* Q, const xattn_heads* K, const xattn_heads* V,
                  const xattn_rotary* rot, const xattn_cache* cache, int T, const int32_t* n_new,
                  const int32_t* seen, const xattn_heads* Qo, void* stream) {
  bool empty;
  int rc = check_cache(cache, &empty);
  if (rc != XATTN_OK) return rc;
  if (T < 0) return XATTN_EINVAL;
  const int B = cache->B;
  if ((rc = check_heads(K, B, T, false)) != XATTN_OK) return rc;
  if ((rc = check_heads(V, B, T, false)) != XATTN_OK) return rc;
  if (K->heads != cache->Hkv || V->heads != cache->Hkv) return XATTN_EINVAL;
  if (rot != nullptr) {
    if ((rc = check_rotary(rot, B, T, cache->C)) != XATTN_OK) return rc;
    if ((rc = check_heads(Q, B, T, false)) != XATTN_OK) return rc;
    if ((rc = check_heads(Qo, B, T, true)) != XATTN_OK) return rc;
    if (Q->heads != Qo->heads || Q->heads > 65535) return XATTN_EINVAL;
  }
  if (empty || T == 0) return XATTN_OK;
  RopeParams p = {};
  p.q = view_of(Q);
  p.k = view_of(K);
  p.v = view_of(V);
  p.qo = view_of(Qo);
  if (rot != nullptr) set_rotary(&p, rot, T, false);
  p.cache = view_of(cache);
  p.n_new = n_new;
  p.seen = seen;
  const int dst = cache->kv_type == XATTN_KV_BF16 ? 1 : 2;
  if (cache->C == 64)
    return launch_rope_append<64>(p, rot != nullptr, dst, B, T, as_stream(stream));
  return launch_rope_append<128>(p, rot != nullptr, dst, B, T, as_stream(stream));
}

// ------------------------------------------------------------------ decode
struct DecodePlan {
  int NT, HT, rows;
  long long items, partials;
  size_t off_seg, off_o, off_logits, bytes;
};

DecodePlan decode_plan(const xattn_cache* c, int Hq, bool weights) {
  DecodePlan d;
  const int G = Hq / c->Hkv;
  d.NT = G <= 8 ? 1 : 2;
  d.HT = (G + 15) / 16;
  d.rows = 8 * d.NT;
  d.items = (long long)c->B * c->Hkv * d.HT;
  d.partials = d.items + kDecMaxCtas;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  d.off_seg = up((size_t)d.partials * d.rows * sizeof(float2));
  d.off_o = d.off_seg + up((size_t)d.items * sizeof(int2));
  d.off_logits = d.off_o + up((size_t)d.partials * d.rows * c->C * sizeof(float));
  d.bytes = d.off_logits;
  if (weights) d.bytes += up((size_t)c->B * Hq * c->max_pages * c->page * sizeof(float));
  return d;
}

int check_decode(const xattn_cache* c, int Hq, bool* empty) {
  const int rc = check_cache(c, empty);
  if (rc != XATTN_OK) return rc;
  if (Hq < 0) return XATTN_EINVAL;
  if (*empty) return c->Hkv == 0 && Hq > 0 ? XATTN_EINVAL : XATTN_OK;
  if (Hq % c->Hkv != 0) return XATTN_EINVAL;
  if (Hq / c->Hkv > kDecMaxGroup) return XATTN_EUNSUPPORTED;
  if (Hq == 0) *empty = true;
  return XATTN_OK;
}

// [rows, C] pool as a 3-D map: 128-byte (or whole) column groups of `part` rows, swizzled
// as the MMA warps' ldmatrix addresses expect.
bool make_pool_map(CUtensorMap* map, const void* base, uint64_t rows, int C, int part, bool fp8) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const int group = fp8 ? C : 64;
  const uint64_t row_bytes = (uint64_t)C * (fp8 ? 1 : 2);
  cuuint64_t dims[3] = {(cuuint64_t)group, rows, (cuuint64_t)(C / group)};
  cuuint64_t strides[2] = {row_bytes, 128};
  cuuint32_t box[3] = {(cuuint32_t)group, (cuuint32_t)part, (cuuint32_t)(C / group)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             fp8 && C == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int C, bool FP8, int NT>
int launch_decode_split(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p,
                        cudaStream_t st) {
  using L = Decode<C, FP8, NT>;
  static unsigned long long done[2] = {0, 0};
  const bool idle = p.n_new != nullptr;
  auto kern = idle ? decode_split_kernel<C, FP8, NT, true> : decode_split_kernel<C, FP8, NT, false>;
  if (ensure_smem_limit(kern, L::kSmem, &done[idle]) != XATTN_OK) return XATTN_ECUDA;
  return launch(kern, dim3(148 * L::kPerSm), kDecThreads, L::kSmem, st, 1, mk, mv, p);
}

template <int C>
int launch_decode(const xattn_cache* c, DecodeParams& p, const DecodePlan& d, cudaStream_t st) {
  const bool fp8 = c->kv_type == XATTN_KV_E4M3;
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)c->num_pages * c->Hkv * c->page;
  const int part = c->page < 64 ? c->page : 64;
  if (!make_pool_map(&mk, c->k_pages, rows, C, part, fp8) ||
      !make_pool_map(&mv, c->v_pages, rows, C, part, fp8))
    return XATTN_ECUDA;
  int rc;
  if (fp8)
    rc = d.NT == 1 ? launch_decode_split<C, true, 1>(mk, mv, p, st)
                   : launch_decode_split<C, true, 2>(mk, mv, p, st);
  else
    rc = d.NT == 1 ? launch_decode_split<C, false, 1>(mk, mv, p, st)
                   : launch_decode_split<C, false, 2>(mk, mv, p, st);
  if (rc != XATTN_OK) return rc;
  // weight blocks per (sequence, kv head): enough for the longest, or to fill the GPU
  long long wb = 0;
  if (p.acc_out != nullptr) {
    const long long pairs = (long long)c->B * c->Hkv;
    constexpr int kSlots = 4 * kJoinThreads;     // slots of a block's sweep
    wb = std::min<long long>(((long long)c->max_pages * c->page + kSlots - 1) / kSlots,
                             std::max<long long>(1, 148 * 16 / pairs));
  }
  const long long blocks = (long long)c->B * p.Hq + wb * c->B * c->Hkv;
  auto join = p.n_new != nullptr ? decode_join_kernel<C, true> : decode_join_kernel<C, false>;
  return launch(join, dim3((unsigned)blocks), kJoinThreads, 0, st, 1, p, d.rows, 8 * d.NT, (int)wb);
}

// ------------------------------------------------------------------ evict
struct EvictPlan {
  long long rows, max_moves;
  int cluster, share;           // CTAs per row, most slots of one
  bool in_smem;                 // a CTA's keys fit its shared memory
  size_t off_hole, off_mover, off_keys, bytes;
};

EvictPlan evict_plan(const xattn_cache* c, int budget) {
  EvictPlan e;
  const long long cap = (long long)c->max_pages * c->page;
  e.rows = (long long)c->B * c->Hkv;
  e.max_moves = std::max<long long>(0, std::min<long long>(budget, cap - budget));
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  e.off_hole = up((size_t)e.rows * sizeof(int32_t));
  e.off_mover = e.off_hole + up((size_t)(e.rows * e.max_moves) * sizeof(int32_t));
  e.off_keys = e.off_mover + up((size_t)(e.rows * e.max_moves) * sizeof(int32_t));
  // CTAs per row: more while the rows alone leave SMs idle and a part stays worth a
  // cluster barrier per pass. (8 is the portable most; 16 CTAs, of which few clusters fit
  // the GPU at once, took 91 us for the eviction of a 128K cache instead of 77.)
  e.cluster = 1;
  while (e.cluster < 8 && e.rows * e.cluster * 2 <= 148 && cap / (e.cluster * 2) >= 2048) e.cluster *= 2;
  e.share = (int)((((cap + e.cluster - 1) / e.cluster) + 3) & ~3ll);
  e.in_smem = e.share <= kEvMaxKeys;
  const size_t keys = (size_t)e.rows * e.cluster * evict_part_words(e.share);
  e.bytes = e.off_keys + (e.in_smem ? 0 : up(keys * sizeof(uint32_t)));
  return e;
}

}  // namespace

extern "C" {

int xattn_rope(const xattn_heads* Q, const xattn_heads* K, const xattn_rotary* rot, int inverse,
               int B, int M, int C, const xattn_heads* Qo, const xattn_heads* Ko, void* stream) {
  if (B < 0 || M < 0 || C <= 0) return XATTN_EINVAL;
  if (C != 64 && C != 128) return XATTN_EUNSUPPORTED;
  if (B > 65535) return XATTN_EUNSUPPORTED;
  int rc = check_rotary(rot, B, M, C);
  if (rc != XATTN_OK) return rc;
  if ((rc = check_heads(Q, B, M, false)) != XATTN_OK) return rc;
  if ((rc = check_heads(Qo, B, M, true)) != XATTN_OK) return rc;
  if (Q->heads != Qo->heads || Q->heads > 65535) return XATTN_EINVAL;
  if ((K == nullptr) != (Ko == nullptr)) return XATTN_EINVAL;
  if (K != nullptr) {
    if ((rc = check_heads(K, B, M, false)) != XATTN_OK) return rc;
    if ((rc = check_heads(Ko, B, M, true)) != XATTN_OK) return rc;
    if (K->heads != Ko->heads || K->heads > 65535) return XATTN_EINVAL;
  }
  if (B == 0 || M == 0 || (Q->heads == 0 && (K == nullptr || K->heads == 0))) return XATTN_OK;
  RopeParams p = {};
  p.q = view_of(Q);
  p.k = view_of(K);
  p.qo = view_of(Qo);
  p.ko = view_of(Ko);
  set_rotary(&p, rot, M, inverse != 0);
  if (C == 64) return launch_rope_append<64>(p, true, 0, B, M, as_stream(stream));
  return launch_rope_append<128>(p, true, 0, B, M, as_stream(stream));
}

int xattn_cache_append(const xattn_heads* K, const xattn_heads* V, const xattn_cache* cache, int T,
                       const int32_t* n_new, const int32_t* seen, void* stream) {
  return append_common(nullptr, K, V, nullptr, cache, T, n_new, seen, nullptr, stream);
}

int xattn_rope_append(const xattn_heads* Q, const xattn_heads* K, const xattn_heads* V,
                      const xattn_rotary* rot, const xattn_cache* cache, int T,
                      const int32_t* n_new, const int32_t* seen, const xattn_heads* Qo,
                      void* stream) {
  if (rot == nullptr) return XATTN_EINVAL;
  return append_common(Q, K, V, rot, cache, T, n_new, seen, Qo, stream);
}

size_t xattn_decode_workspace_size(const xattn_cache* cache, int Hq, int weights) {
  bool empty;
  if (check_decode(cache, Hq, &empty) != XATTN_OK || empty) return 0;
  return decode_plan(cache, Hq, weights != 0).bytes;
}

int xattn_decode_attn(const xattn_heads* Q, const xattn_cache* cache, float softmax_scale, void* O,
                      float* lse, float* acc_out, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return xattn_decode_attn_ex(Q, cache, nullptr, softmax_scale, O, lse, acc_out, workspace,
                              workspace_bytes, stream);
}

int xattn_decode_attn_ex(const xattn_heads* Q, const xattn_cache* cache, const int32_t* n_new,
                         float softmax_scale, void* O, float* lse, float* acc_out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (Q == nullptr) return XATTN_EINVAL;
  bool empty;
  int rc = check_decode(cache, Q->heads, &empty);
  if (rc != XATTN_OK) return rc;
  if ((rc = check_heads(Q, cache->B, 1, false)) != XATTN_OK) return rc;
  // (in log2 units, as the kernels take it, the scale must be finite too)
  if (!(softmax_scale > 0.f) || softmax_scale * kLog2e == __builtin_huge_valf()) return XATTN_EINVAL;
  if (empty) return XATTN_OK;
  if (!O || !aligned16(O) || !workspace || !aligned16(workspace)) return XATTN_EINVAL;
  if (acc_out != nullptr && (cache->acc == nullptr || !aligned16(acc_out))) return XATTN_EINVAL;
  const DecodePlan d = decode_plan(cache, Q->heads, acc_out != nullptr);
  if (workspace_bytes < d.bytes) return XATTN_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeParams p = {};
  p.cache = view_of(cache);
  p.q = static_cast<const bf16*>(Q->data);
  p.q_sb = Q->stride_b;
  p.q_sh = Q->stride_h;
  p.O = static_cast<bf16*>(O);
  p.lse = lse;
  p.part_ml = reinterpret_cast<float2*>(ws);
  p.seg = reinterpret_cast<int2*>(ws + d.off_seg);
  p.part_o = reinterpret_cast<float*>(ws + d.off_o);
  p.logits = acc_out != nullptr ? reinterpret_cast<float*>(ws + d.off_logits) : nullptr;
  p.acc_out = acc_out;
  p.Hq = Q->heads;
  p.G = Q->heads / cache->Hkv;
  p.HT = d.HT;
  p.scale_log2 = softmax_scale * kLog2e;
  p.n_new = n_new;
  if (cache->C == 64) return launch_decode<64>(cache, p, d, as_stream(stream));
  return launch_decode<128>(cache, p, d, as_stream(stream));
}

size_t xattn_cache_evict_workspace_size(const xattn_cache* cache, int budget) {
  bool empty;
  if (check_cache(cache, &empty) != XATTN_OK || empty || budget < 1) return 0;
  return evict_plan(cache, budget).bytes;
}

int xattn_cache_evict(const xattn_cache* cache, int budget, int recent, int sink,
                      const int32_t* seen, float* acc_out, int32_t* ord_out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  bool empty;
  int rc = check_cache(cache, &empty);
  if (rc != XATTN_OK) return rc;
  if (budget < 1 || recent < 0 || sink < 0 || (long long)recent + sink > budget)
    return XATTN_EINVAL;
  if (empty) return XATTN_OK;
  if (!cache->acc || !cache->ordinal || !acc_out || !ord_out || !workspace) return XATTN_EINVAL;
  if (!aligned16(acc_out) || !aligned16(ord_out) || !aligned16(workspace)) return XATTN_EINVAL;
  const EvictPlan e = evict_plan(cache, budget);
  if (workspace_bytes < e.bytes) return XATTN_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  EvictParams p = {};
  p.cache = view_of(cache);
  p.seen = seen;
  p.acc_out = acc_out;
  p.ord_out = ord_out;
  p.count = reinterpret_cast<int32_t*>(ws);
  p.hole = reinterpret_cast<int32_t*>(ws + e.off_hole);
  p.mover = reinterpret_cast<int32_t*>(ws + e.off_mover);
  p.max_moves = e.max_moves;
  p.budget = budget;
  p.recent = recent;
  p.sink = sink;
  p.row_bytes_log2 = ilog2(cache->C * (cache->kv_type == XATTN_KV_BF16 ? 2 : 1));
  p.keys = e.in_smem ? nullptr : reinterpret_cast<uint32_t*>(ws + e.off_keys);
  p.share = e.share;
  static unsigned long long done = 0;
  if (ensure_smem_limit(evict_select_kernel, kEvMaxKeys * 5, &done) != XATTN_OK) return XATTN_ECUDA;
  cudaStream_t st = as_stream(stream);
  rc = launch(evict_select_kernel, dim3(e.cluster, (unsigned)e.rows), kEvThreads,
              e.in_smem ? (size_t)e.share * 5 : 0, st, e.cluster, p);
  if (rc != XATTN_OK) return rc;
  if (e.max_moves == 0) return XATTN_OK;
  const int per_block = kEvMoveThreads >> (p.row_bytes_log2 - 4);     // moves of a sweep
  const long long most = (e.max_moves + per_block - 1) / per_block;
  const long long fill = std::max<long long>(1, 148 * 8 / e.rows);
  return launch(evict_move_kernel, dim3((unsigned)std::min(most, fill), (unsigned)e.rows),
                kEvMoveThreads, 0, st, 1, p);
}

}  // extern "C"
