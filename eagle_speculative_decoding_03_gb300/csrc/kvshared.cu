// Attention over keys that are not the rows' own sequence: cross attention, attention of
// requests behind a shared prefix, and the join of partial results.  See include/eagle_draft.h.
//
//   o_i = sum_j p_ij v_j with p_ij = 2^(s_ij - m_i) and l_i = sum_j p_ij over the keys j of part i
//   M = max m_i,  L = sum 2^(m_i - M) l_i,  out = sum 2^(m_i - M) o_i / L,  lse = ln 2 (M + log2 L)
//
// Partial results over disjoint keys (key ranges, the prefix and a request's own keys) are joined
// by that rule, in a fixed order.  The kernels over the keys are in kvattn.cu (by ranges), kvcross.cu and
// kvfew.cu (dealt out in line).
#include "kvline.cuh"

#include <algorithm>

using namespace eagle;

namespace {

constexpr int MG_THREADS = 256;

// ------------------------------------------------------------------ prefix and own keys
// WARPS warps per (row, query head), each a share of the ranges: the own keys' first, then the
// prefix's (`pre`, whose buffers lie behind them).  For prefixes cut by ranges: kvcross.cu joins in its
// own epilogue.  Starts while the ranges run and waits for them; the prefix's ranges run beside the own
// keys' (2 requests behind 700 keys: 17 us, 22 one after the other; 32 behind 8,192: 44, with the own keys dealt out
// in line ahead of the prefix in the wide kernel 58).  The two caches' value factors are applied after the division
// (as in kvattn.cu), so the sums of the two are kept apart.
template <int HD, int WARPS>
__global__ void __launch_bounds__(128) kv_shared_join(const KaArgs a, const KaArgs pre) {
  constexpr int E = HD / 32;
  __shared__ float s_o[4][2][HD], s_l[4];
  pdl_wait();                                // the ranges' results
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WARPS;
  const long long w = static_cast<long long>(blockIdx.x) * (4 / WARPS) + warp / WARPS;
  const int n = static_cast<int>(w / a.Hq), h = static_cast<int>(w - static_cast<long long>(n) * a.Hq);
  if (n >= a.N) return;
  const int b = row_owner(a.cu, a.B, n);
  if (b < 0) return;
  const int g = row_owner(pre.groups, pre.B, b);
  if (g < 0) {                               // (a request outside every group)
    if (lane == 0) atomicOr(a.err, DEVERR_PREFIX);
    return;
  }
  const Req rq = request(a, b), rp = request(pre, g);
  if (n < rq.row0 || n - rq.row0 >= rq.R || n < rp.row0 || n - rp.row0 >= rp.R) return;
  const int own = ranges_of(a, rq.len), used = own + ranges_of(pre, rp.len);
  const size_t at = static_cast<size_t>(n) * a.Hq + h, step = static_cast<size_t>(a.N) * a.Hq;
  auto place = [&](int s) { return (s < own ? s : a.splits + s - own) * step + at; };
  float M = -INFINITY;
  for (int s = lane; s < used; s += 32) M = max_nan(M, a.part_ml[place(s)].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, d));
  float o[2][E], L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[0][e] = o[1][e] = 0.f;
#pragma unroll 4
  for (int s = part; s < used; s += WARPS) {
    const float2 ml = a.part_ml[place(s)];
    if (ml.x == -INFINITY) continue;
    const float f = M == INFINITY ? (ml.x == INFINITY ? 1.f : 0.f) : exp2f(ml.x - M);
    L = fmaf(f, ml.y, L);
    const float* p = a.part_o + place(s) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (s < own) o[0][e] = add_weighted(o[0][e], f, p[e]);
      else o[1][e] = add_weighted(o[1][e], f, p[e]);
    }
  }
  if constexpr (WARPS > 1) {                 // (the CTA is one row's: it is here whole)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s_o[part][0][lane * E + e] = o[0][e];
      s_o[part][1][lane * E + e] = o[1][e];
    }
    if (lane == 0) s_l[part] = L;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int r = 1; r < WARPS; ++r) {
      L += s_l[r];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[0][e] += s_o[r][0][lane * E + e];
        o[1][e] += s_o[r][1][lane * E + e];
      }
    }
  }
  const bool none = L == 0.f;
  const float i0 = none ? 0.f : a.vg / L, i1 = none ? 0.f : pre.vg / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + n * a.out_ld + static_cast<long long>(h) * HD + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    dst[e / 2] = none ? 0u : pack_bf16(fmaf(o[0][e], i0, o[1][e] * i1), fmaf(o[0][e + 1], i0, o[1][e + 1] * i1));
  if (a.lse && lane == 0) a.lse[at] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int HD>
cudaError_t launch_join(const KaArgs& a, const KaArgs& pre, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.N) * a.Hq;
  return a.splits + pre.splits > 8 ? launch_after(true, dim3(static_cast<unsigned>(rows)), 128, 0, st, kv_shared_join<HD, 4>, a, pre)
                                   : launch_after(true, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, st, kv_shared_join<HD, 1>, a, pre);
}

// ------------------------------------------------------------------ merge
struct MgArgs {
  const void* outs[EAGLE_MAX_PARTS];
  const float* lses[EAGLE_MAX_PARTS];
  long long ld[EAGLE_MAX_PARTS];
  void* out;
  long long out_ld;
  float* lse;
  long long chunks;                          // N * H * hd / 8
  int parts, H, per;                         // per: chunks of 8 dims per row and head
};

template <typename T>
EAGLE_DEV void load8(const void* base, long long at, float* x) {
  if constexpr (sizeof(T) == 4) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 u = p[0], v = p[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
}

// A thread per 8 dims of a row and head: each value is read once, the parts' weights again by each of a
// head's threads (from L1).  Bound by the bytes: 4 fp32 parts of 8,191 rows and 32 heads of 128 take
// 92 us, 98% of the measured copy rate; one row is one launch, 3.4 us.
template <typename TI, typename TO>
__global__ void __launch_bounds__(MG_THREADS) attention_merge(const MgArgs a) {
  const long long x = static_cast<long long>(blockIdx.x) * MG_THREADS + threadIdx.x;
  if (x >= a.chunks) return;
  const long long nh = x / a.per;
  const int c = static_cast<int>(x - nh * a.per);
  const long long n = nh / a.H;
  const int h = static_cast<int>(nh - n * a.H);
  const long long at = (static_cast<long long>(h) * a.per + c) * 8;
  float M = -INFINITY;
  for (int i = 0; i < a.parts; ++i) M = max_nan(M, a.lses[i][nh]);
  float o[8] = {}, L = 0.f;
  for (int i = 0; i < a.parts; ++i) {
    const float l = a.lses[i][nh];
    if (l == -INFINITY) continue;
    const float f = M == INFINITY ? (l == INFINITY ? 1.f : 0.f) : expf(l - M);
    L += f;
    float y[8];
    load8<TI>(a.outs[i], n * a.ld[i] + at, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = add_weighted(o[e], f, y[e]);
  }
  const bool none = M == -INFINITY;
  const float inv = none ? 0.f : 1.f / L;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = none ? 0.f : o[e] * inv;
  if constexpr (sizeof(TO) == 4) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + n * a.out_ld + at);
    dst[0] = make_float4(o[0], o[1], o[2], o[3]);
    dst[1] = make_float4(o[4], o[5], o[6], o[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + n * a.out_ld + at) =
        make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
  }
  if (c == 0 && a.lse) a.lse[nh] = none ? -INFINITY : M == INFINITY ? M : M + logf(L);
}

bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether rows [N] of `width` bytes, `ld` bytes apart, from p may share memory with rows of q.
bool rows_meet(const void* p, long long p_ld, long long p_width, const void* q, long long q_ld, long long q_width, long long N) {
  const intptr_t a = reinterpret_cast<intptr_t>(p), b = reinterpret_cast<intptr_t>(q);
  if (a + (N - 1) * p_ld + p_width <= b || b + (N - 1) * q_ld + q_width <= a) return false;
  if (p_ld != q_ld) return true;
  const long long d = ((b - a) % p_ld + p_ld) % p_ld;   // q's rows begin d bytes behind p's
  return d < p_width || d + q_width > p_ld;
}

// What the entry points over a paged cache check alike.
eagle_status_t check_rows(const char* who, int Hkv, int hd, int B, int N, int Hq, const void* q, long long q_ld, const void* out,
                          long long out_ld, float scale) {
  const long long width = static_cast<long long>(Hq) * hd;
  if (B < 1 || N < 0) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need B >= 1 and N >= 0", who);
  if (Hq < 1 || Hq % Hkv || Hq / Hkv > KA_MAX_GROUP)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: n_heads must be 1..%d times n_kv_heads", who, KA_MAX_GROUP);
  if (!std::isfinite(scale) || scale < 0.f) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: scale must be finite and not negative", who);
  if (width >= 1ll << 31 || static_cast<long long>(N) * Hq > (1ll << 31) - 8 || Hkv > 65535)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: too many rows or heads for one launch", who);
  if (!q && !out) return EAGLE_OK;           // (a workspace query)
  if (q_ld < width || out_ld < width || q_ld % 8 || out_ld % 8 || !aligned(q) || !aligned(out))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned and not overlap", who);
  if (N && rows_meet(q, 2 * q_ld, 2 * width, out, 2 * out_ld, 2 * width, N))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: out may not overlap q (ranges and blocks read q at different times)", who);
  return EAGLE_OK;
}

// What a call writes beside out: lse and the workspace are its own.
eagle_status_t check_own(const char* who, int N, int Hq, int hd, const void* q, long long q_ld, const void* out, long long out_ld,
                         const float* lse, const void* workspace, int64_t need) {
  const long long width = 2ll * Hq * hd, q_bytes = 2ll * (N - 1) * q_ld + width, out_bytes = 2ll * (N - 1) * out_ld + width, lse_bytes = 4ll * N * Hq;
  auto meet = [](const void* a, long long na, const void* b, long long nb) { return rows_meet(a, na, na, b, nb, nb, 1); };
  if (lse && (meet(lse, lse_bytes, q, q_bytes) || meet(lse, lse_bytes, out, out_bytes)))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: lse overlaps q or out", who);
  if (need > 0 && (meet(workspace, need, q, q_bytes) || meet(workspace, need, out, out_bytes) || (lse && meet(workspace, need, lse, lse_bytes))))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: the workspace overlaps q, out or lse", who);
  return EAGLE_OK;
}

eagle_status_t check_extent(const char* who, int max_rows, int max_len) {
  if (max_rows < 1 || max_len < 1) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need max_rows and max_len >= 1", who);
  if (max_len > 1 << 30) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: max_len must be at most 2^30", who);
  return EAGLE_OK;
}

eagle_status_t check_plan(const char* who, int B, const KaPlan& p) {
  if (static_cast<long long>(B) * p.blocks > 65535)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: too many rows, heads or requests for one launch", who);
  return EAGLE_OK;
}

// The page maps of a bf16 pool.
eagle_status_t page_maps(const char* who, const eagle_kv_cache_t* c, CUtensorMap* tmk, CUtensorMap* tmv) {
  memset(tmk, 0, sizeof(*tmk));
  memset(tmv, 0, sizeof(*tmv));
  const long long blocks = static_cast<long long>(c->num_pages) * c->n_kv_heads;
  if (c->kind == EAGLE_CACHE_BF16 && (!make_page_map(tmk, c->k, c->head_dim, c->page_size, blocks) ||
                                      !make_page_map(tmv, c->v, c->head_dim, c->page_size, blocks)))
    return kv_fail(EAGLE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  return EAGLE_OK;
}

float log2_scale(float scale, int hd) {
  return std::min((scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(hd))) * 1.4426950408889634f, FLT_MAX);
}

// How a call over keys that all rows see is cut: by ranges, or dealt out in line over the SMs (WIDE, or FEW for
// at most KF_QV query vectors over bf16 pages; FEW also takes a step's own keys, of one row a request, which
// sees them all).
enum class Cutting { RANGES, WIDE, FEW };
struct CrossPlan {
  Cutting by;
  KaPlan ranges;
  KxPlan line;
  bool separate() const { return by == Cutting::RANGES && ranges.splits > 1 && !ranges.joined; }
  int64_t line_bytes() const { return by == Cutting::RANGES ? 0 : line.bytes; }
};
// alone: a cross call; else the prefix of a shared one.
CrossPlan cross_plan(const eagle_kv_cache_t* c, int G, int B, int N, int max_rows, int max_len, bool alone) {
  CrossPlan p;
  const int Hkv = c->n_kv_heads, hd = c->head_dim;
  const long long qv = static_cast<long long>(max_rows) * G;
  p.by = Cutting::RANGES;
  p.ranges = ka_plan(c->kind, Hkv, G, B, max_rows, max_len, alone);
  if (qv > KF_QV && kx_worth(c->kind, Hkv, G, B, N, max_rows, max_len)) p.by = Cutting::WIDE;
  if (alone && qv <= KF_QV && c->kind == EAGLE_CACHE_BF16 && kf_worth(Hkv, hd, static_cast<int>(qv), B, max_len, true)) p.by = Cutting::FEW;
  // (a launch by ranges has no room for more blocks)
  if (p.by == Cutting::RANGES && (qv > KF_QV || !alone) && static_cast<long long>(B) * p.ranges.blocks > 65535) p.by = Cutting::WIDE;
  if (p.by == Cutting::WIDE) p.line = kx_plan(c->kind, Hkv, hd, G, B, max_rows, max_len);
  if (p.by == Cutting::FEW) p.line = kf_plan(Hkv, hd, B, max_len);
  return p;
}
// The own keys of a shared call.
CrossPlan own_plan(const eagle_kv_cache_t* c, int G, const eagle_kv_attention_t* w) {
  CrossPlan p;
  const int Hkv = c->n_kv_heads, hd = c->head_dim;
  p.by = w->max_rows == 1 && !w->mask && c->kind == EAGLE_CACHE_BF16 && G <= KF_QV && kf_worth(Hkv, hd, G, w->B, w->max_len, false)
             ? Cutting::FEW : Cutting::RANGES;
  p.ranges = ka_plan(c->kind, Hkv, G, w->B, w->max_rows, w->max_len, false);
  if (p.by == Cutting::FEW) p.line = kf_plan(Hkv, hd, w->B, w->max_len);
  return p;
}

eagle_status_t check_cross(const char* who, const eagle_kv_cache_t* cache, const eagle_kv_cross_t* w, KvPool* pool, CrossPlan* p) {
  eagle_status_t r = kv_pool(cache, who, pool);
  if (r != EAGLE_OK) return r;
  if (!w) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null arguments", who);
  r = check_extent(who, w->max_rows, w->max_len);
  if (r == EAGLE_OK) r = check_rows(who, cache->n_kv_heads, cache->head_dim, w->B, w->N, w->n_heads, w->q, w->q_stride, w->out, w->out_stride, w->scale);
  if (r != EAGLE_OK) return r;
  *p = cross_plan(cache, w->n_heads / cache->n_kv_heads, w->B, w->N, w->max_rows, w->max_len, true);
  return p->by != Cutting::RANGES ? EAGLE_OK : check_plan(who, w->B, p->ranges);
}

int64_t cross_bytes(const eagle_kv_cross_t* w, int hd, const CrossPlan& p) {
  return p.line_bytes() + (p.separate() ? p.ranges.splits * ka_part_bytes(w->N, w->n_heads, hd) : 0);
}

// Ranges of partial results of a shared call: the own keys', then the prefix's.
int own_ranges(const CrossPlan& own) { return own.by == Cutting::RANGES ? own.ranges.splits : 1; }
int pre_ranges(const CrossPlan& pre) { return pre.by == Cutting::WIDE ? 0 : pre.ranges.splits; }
int64_t shared_bytes(const eagle_kv_attention_t* w, int hd, const CrossPlan& pre, const CrossPlan& own) {
  return pre.line_bytes() + own.line_bytes() + (own_ranges(own) + pre_ranges(pre)) * ka_part_bytes(w->N, w->n_heads, hd);
}

eagle_status_t check_shared(const char* who, const eagle_kv_cache_t* prefix, const eagle_kv_groups_t* g, const eagle_kv_cache_t* cache,
                            const eagle_kv_attention_t* w, KvPool* pre, KvPool* own, CrossPlan* pp, CrossPlan* po) {
  eagle_status_t r = kv_pool(prefix, who, pre);
  if (r == EAGLE_OK) r = kv_pool(cache, who, own);
  if (r != EAGLE_OK) return r;
  if (!g || !w) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null arguments", who);
  if (prefix->n_kv_heads != cache->n_kv_heads || prefix->head_dim != cache->head_dim)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: the two caches must have the same heads and head_dim", who);
  r = check_extent(who, g->max_rows, g->max_len);
  if (r == EAGLE_OK) r = check_extent(who, w->max_rows, w->max_len);
  if (r == EAGLE_OK) r = check_rows(who, cache->n_kv_heads, cache->head_dim, w->B, w->N, w->n_heads, w->q, w->q_stride, w->out, w->out_stride, w->scale);
  if (r != EAGLE_OK) return r;
  if (g->n_groups < 1) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need n_groups >= 1", who);
  if (w->mask && (w->mask_slots < 1 || w->mask_slots > 64 || w->max_rows > w->mask_slots))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: a mask needs max_rows <= mask_slots <= 64", who);
  const int G = w->n_heads / cache->n_kv_heads;
  *pp = cross_plan(prefix, G, g->n_groups, w->N, g->max_rows, g->max_len, false);
  *po = own_plan(cache, G, w);
  if (pp->by == Cutting::RANGES) r = check_plan(who, g->n_groups, pp->ranges);
  return r != EAGLE_OK || po->by != Cutting::RANGES ? r : check_plan(who, w->B, po->ranges);
}

}  // namespace

extern "C" int64_t eagle_kv_cross_attention_workspace(const eagle_kv_cache_t* cache, const eagle_kv_cross_t* w) {
  KvPool pool;
  CrossPlan p;
  if (check_cross("kv_cross_attention_workspace", cache, w, &pool, &p) != EAGLE_OK) return -1;
  return cross_bytes(w, cache->head_dim, p);
}

extern "C" eagle_status_t eagle_kv_cross_attention(const eagle_kv_cache_t* cache, const eagle_kv_cross_t* w, uint32_t* err_word,
                                                   void* stream) {
  const char* who = "kv_cross_attention";
  if (w && (!err_word || !w->cu_rows || !w->lens || !w->q || !w->out)) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  KaArgs a;
  memset(&a, 0, sizeof(a));
  CrossPlan p;
  eagle_status_t r = check_cross(who, cache, w, &a.pool, &p);
  if (r != EAGLE_OK) return r;
  const bool f4 = cache->kind == EAGLE_CACHE_F4, separate = p.separate();
  const int64_t need = cross_bytes(w, cache->head_dim, p);
  if (need > 0 && (!w->workspace || w->workspace_bytes < need || !aligned(w->workspace)))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: needs %lld bytes of workspace, 16-byte aligned", who, static_cast<long long>(need));
  if (w->N == 0) return EAGLE_OK;
  r = check_own(who, w->N, w->n_heads, cache->head_dim, w->q, w->q_stride, w->out, w->out_stride, w->lse, w->workspace, need);
  if (r != EAGLE_OK) return r;
  a.B = w->B;
  a.N = w->N;
  a.Hq = w->n_heads;
  a.G = w->n_heads / cache->n_kv_heads;
  a.g_inverse = static_cast<uint32_t>(std::min((1ull << 32) / a.G, (1ull << 32) - 1));
  a.max_rows = w->max_rows;
  a.max_len = w->max_len;
  a.cross = 1;
  a.parts = separate;
  a.cu = w->cu_rows;
  a.lens = w->lens;
  a.q = static_cast<const __nv_bfloat16*>(w->q);
  a.q_ld = w->q_stride;
  a.scale_log2 = log2_scale(w->scale, cache->head_dim);
  a.vg = f4 ? a.pool.vg : 1.f;
  a.out = static_cast<__nv_bfloat16*>(w->out);
  a.out_ld = w->out_stride;
  a.lse = w->lse;
  a.part_o = static_cast<float*>(w->workspace);
  if (separate) a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(p.ranges.splits) * w->N * w->n_heads * cache->head_dim);
  a.err = err_word;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tmk, tmv;
  r = page_maps(who, cache, &tmk, &tmv);
  if (r != EAGLE_OK) return r;
  float* parts = static_cast<float*>(w->workspace);
  cudaError_t e = p.by == Cutting::WIDE ? kx_launch(a, nullptr, f4, tmk, tmv, p.line, parts, st)
                  : p.by == Cutting::FEW ? kf_launch(&a, cache, p.line, parts, st)
                                         : ka_launch(&a, p.ranges, f4, tmk, tmv, st);
  if (e == cudaSuccess && separate) e = ka_combine(a, st);
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}

extern "C" int64_t eagle_kv_shared_attention_workspace(const eagle_kv_cache_t* prefix, const eagle_kv_groups_t* g,
                                                       const eagle_kv_cache_t* cache, const eagle_kv_attention_t* w) {
  KvPool pre, own;
  CrossPlan pp, po;
  if (check_shared("kv_shared_attention_workspace", prefix, g, cache, w, &pre, &own, &pp, &po) != EAGLE_OK) return -1;
  return shared_bytes(w, cache->head_dim, pp, po);
}

extern "C" eagle_status_t eagle_kv_shared_attention(const eagle_kv_cache_t* prefix, const eagle_kv_groups_t* g,
                                                    const eagle_kv_cache_t* cache, const eagle_kv_attention_t* w, uint32_t* err_word,
                                                    void* stream) {
  const char* who = "kv_shared_attention";
  if (g && w && (!err_word || !g->cu_groups || !g->lens || !w->cu_rows || !w->lens || !w->q || !w->out))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  KaArgs a, x;                               // the own keys, the prefix
  memset(&a, 0, sizeof(a));
  memset(&x, 0, sizeof(x));
  CrossPlan pp, po;
  eagle_status_t r = check_shared(who, prefix, g, cache, w, &x.pool, &a.pool, &pp, &po);
  if (r != EAGLE_OK) return r;
  const int hd = cache->head_dim;
  const int64_t need = shared_bytes(w, hd, pp, po);
  const int own = own_ranges(po), ranges = own + pre_ranges(pp);
  if (need > 0 && (!w->workspace || w->workspace_bytes < need || !aligned(w->workspace)))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: needs %lld bytes of workspace, 16-byte aligned", who, static_cast<long long>(need));
  if (w->N == 0) return EAGLE_OK;
  r = check_own(who, w->N, w->n_heads, hd, w->q, w->q_stride, w->out, w->out_stride, w->lse, w->workspace, need);
  if (r != EAGLE_OK) return r;
  const size_t outs = static_cast<size_t>(w->N) * w->n_heads;
  a.B = w->B;
  a.N = w->N;
  a.Hq = w->n_heads;
  a.G = w->n_heads / cache->n_kv_heads;
  a.g_inverse = static_cast<uint32_t>(std::min((1ull << 32) / a.G, (1ull << 32) - 1));
  a.max_rows = w->max_rows;
  a.max_len = w->max_len;
  a.S = w->mask_slots;
  a.parts = 1;
  a.cu = w->cu_rows;
  a.lens = w->lens;
  a.q = static_cast<const __nv_bfloat16*>(w->q);
  a.q_ld = w->q_stride;
  a.mask = w->mask;
  a.scale_log2 = log2_scale(w->scale, hd);
  a.vg = cache->kind == EAGLE_CACHE_F4 ? a.pool.vg : 1.f;
  a.out = static_cast<__nv_bfloat16*>(w->out);
  a.out_ld = w->out_stride;
  a.lse = w->lse;
  float* pre_parts = static_cast<float*>(w->workspace);   // (what is dealt in line first: it keeps 16-byte alignment)
  float* own_parts = pre_parts + pp.line_bytes() / 4;
  a.part_o = own_parts + po.line_bytes() / 4;
  a.part_ml = reinterpret_cast<float2*>(a.part_o + ranges * outs * hd);
  a.err = err_word;
  const KvPool pool = x.pool;
  x = a;
  x.pool = pool;
  x.B = g->n_groups;
  x.max_rows = g->max_rows;
  x.max_len = g->max_len;
  x.cross = 1;
  x.behind = 1;
  x.groups = g->cu_groups;
  x.requests = w->B;
  x.lens = g->lens;
  x.mask = nullptr;
  x.vg = prefix->kind == EAGLE_CACHE_F4 ? x.pool.vg : 1.f;
  x.part_o = a.part_o + own * outs * hd;
  x.part_ml = a.part_ml + own * outs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tmk, tmv, pmk, pmv;
  r = page_maps(who, cache, &tmk, &tmv);
  if (r == EAGLE_OK) r = page_maps(who, prefix, &pmk, &pmv);
  if (r != EAGLE_OK) return r;
  const bool pf4 = prefix->kind == EAGLE_CACHE_F4;
  cudaError_t e = po.by == Cutting::FEW ? kf_launch(&a, cache, po.line, own_parts, st)
                                        : ka_launch(&a, po.ranges, cache->kind == EAGLE_CACHE_F4, tmk, tmv, st);
  if (e == cudaSuccess && pp.by == Cutting::WIDE) {
    e = kx_launch(x, &a, pf4, pmk, pmv, pp.line, pre_parts, st);
  } else if (e == cudaSuccess) {
    e = ka_launch(&x, pp.ranges, pf4, pmk, pmv, st);
    if (e == cudaSuccess) e = hd == 64 ? launch_join<64>(a, x, st) : launch_join<128>(a, x, st);
  }
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}

extern "C" eagle_status_t eagle_attention_merge(const eagle_attention_parts_t* w, void* stream) {
  const char* who = "attention_merge";
  if (!w || !w->outs || !w->lses || !w->out) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (w->parts < 1 || w->parts > EAGLE_MAX_PARTS || w->N < 0 || w->H < 1)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need 1..%d parts, N >= 0 and H >= 1", who, EAGLE_MAX_PARTS);
  for (const int t : {w->dtype, w->out_dtype})
    if (t != EAGLE_DTYPE_F32 && t != EAGLE_DTYPE_BF16) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: unknown dtype %d", who, t);
  if (w->head_dim < 8 || w->head_dim > 256 || w->head_dim % 8)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of 8 up to 256, not %d", who, w->head_dim);
  const long long width = static_cast<long long>(w->H) * w->head_dim, nh = static_cast<long long>(w->N) * w->H;
  if (width >= 1ll << 31 || nh > (1ll << 31) - 8) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: too many rows or heads for one launch", who);
  const int in = w->dtype == EAGLE_DTYPE_F32 ? 4 : 2, outb = w->out_dtype == EAGLE_DTYPE_F32 ? 4 : 2;
  MgArgs a;
  memset(&a, 0, sizeof(a));
  if (w->out_stride < width || w->out_stride * outb % 16 || !aligned(w->out))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: out's rows must be 16-byte aligned and not overlap", who);
  const long long lse_bytes = 4 * nh;
  if (w->lse && w->N && rows_meet(w->lse, lse_bytes, lse_bytes, w->out, w->N * w->out_stride * outb, ((w->N - 1) * w->out_stride + width) * outb, 1))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: lse overlaps out", who);
  for (int i = 0; i < w->parts; ++i) {
    const long long ld = w->strides ? w->strides[i] : width;
    if (!w->outs[i] || !w->lses[i]) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null part", who);
    if (ld < width || ld * in % 16 || !aligned(w->outs[i]) || reinterpret_cast<uintptr_t>(w->lses[i]) % 4)
      return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: a part's rows must be 16-byte aligned and not overlap", who);
    const long long extent = ((w->N - 1) * ld + width) * in;
    const bool same = w->outs[i] == w->out && ld == w->out_stride && in == outb;
    if (w->N && !same && rows_meet(w->outs[i], ld * in, width * in, w->out, w->out_stride * outb, width * outb, w->N))
      return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: out overlaps a part (only the same rows may)", who);
    if (w->N && rows_meet(w->lses[i], lse_bytes, lse_bytes, w->out, w->N * w->out_stride * outb, ((w->N - 1) * w->out_stride + width) * outb, 1))
      return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: out overlaps a part's lse", who);
    if (w->N && w->lse && (rows_meet(w->lses[i], lse_bytes, lse_bytes, w->lse, lse_bytes, lse_bytes, 1) ||
                           rows_meet(w->outs[i], extent, extent, w->lse, lse_bytes, lse_bytes, 1)))
      return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: lse overlaps a part", who);
    a.outs[i] = w->outs[i];
    a.lses[i] = w->lses[i];
    a.ld[i] = ld;
  }
  if (w->N == 0) return EAGLE_OK;
  a.out = w->out;
  a.out_ld = w->out_stride;
  a.lse = w->lse;
  a.parts = w->parts;
  a.H = w->H;
  a.per = w->head_dim / 8;
  a.chunks = nh * a.per;
  const long long grid = (a.chunks + MG_THREADS - 1) / MG_THREADS;
  if (grid >= 1ll << 31) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: too many rows or heads for one launch", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>(grid);
  if (in == 4 && outb == 4) attention_merge<float, float><<<blocks, MG_THREADS, 0, st>>>(a);
  else if (in == 4) attention_merge<float, __nv_bfloat16><<<blocks, MG_THREADS, 0, st>>>(a);
  else if (outb == 4) attention_merge<__nv_bfloat16, float><<<blocks, MG_THREADS, 0, st>>>(a);
  else attention_merge<__nv_bfloat16, __nv_bfloat16><<<blocks, MG_THREADS, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}
