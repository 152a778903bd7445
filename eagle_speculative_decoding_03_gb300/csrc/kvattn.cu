// Attention of a step's rows over the caller's paged key / value cache (bf16 or 4-bit), with
// the tree mask of an emitted draft tree or causally.  See include/eagle_draft.h.
#include "kvcache.cuh"

#include <algorithm>
#include <cmath>

using namespace eagle;

namespace {

constexpr int KA_MAX_GROUP = 64;

struct KaArgs {
  KvPool pool;
  int B, N, Hq, max_rows, max_len, S;
  const int* cu;
  const int* lens;
  const __nv_bfloat16* q;
  long long q_ld;
  const unsigned char* mask;
  float scale;
  __nv_bfloat16* out;
  long long out_ld;
  float* lse;
  unsigned* err;
};

// One warp per (row, query head): a lane holds hd / 32 dims; one pass over the visible keys
// with the running maximum and sum.
template <int HD, int CACHE>
__global__ void __launch_bounds__(128) kv_attention_rows(const KaArgs a) {
  constexpr int E = HD / 32;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int n = w / a.Hq, h = w - n * a.Hq;
  if (n >= a.N) return;
  const int b = row_owner(a.cu, a.B, n);
  if (b < 0) return;
  const int i = n - __ldg(a.cu + b), R = __ldg(a.cu + b + 1) - __ldg(a.cu + b), ctx = __ldg(a.lens + b);
  if (i >= a.max_rows || ctx < 0 || ctx + R > a.max_len) {
    atomicOr(a.err, DEVERR_PREFIX);
    return;
  }
  const int kvh = h / (a.Hq / a.pool.Hkv);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[n * a.q_ld + static_cast<long long>(h) * HD + lane * E + e]) * a.scale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < ctx + R; ++t) {
    const int j = t - ctx;
    if (j >= 0) {
      const bool see = a.mask ? (j < a.S && i < a.S && a.mask[(static_cast<size_t>(b) * a.S + i) * a.S + j]) : j <= i;
      if (!see) continue;
    }
    const int page = kv_page(a.pool, b, t, a.err);
    float kx[E], vx[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane * E + e;
      kx[e] = vx[e] = 0.f;
      if (page < 0) continue;
      const size_t row = kv_row(a.pool, page, kvh, t);
      if (CACHE == EAGLE_CACHE_BF16) {
        kx[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.pool.k)[row * HD + d]);
        vx[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.pool.v)[row * HD + d]);
      } else {
        const int sh = 4 * (d & 1);
        kx[e] = e2m1_to_f32((static_cast<const uint8_t*>(a.pool.k)[row * (HD / 2) + d / 2] >> sh) & 15) *
                e4m3_to_f32(static_cast<const uint8_t*>(a.pool.ks)[row * (HD / 16) + d / 16]) * a.pool.kg;
        vx[e] = e2m1_to_f32((static_cast<const uint8_t*>(a.pool.v)[row * (HD / 2) + d / 2] >> sh) & 15) *
                e4m3_to_f32(static_cast<const uint8_t*>(a.pool.vs)[row * (HD / 16) + d / 16]) * a.pool.vg;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kx[e], s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    if (mn == -INFINITY) {
      if (s != s) l = s;
      continue;
    }
    const float f = expf(m - mn), p = expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * vx[e];
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[n * a.out_ld + static_cast<long long>(h) * HD + lane * E + e] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] / l);
  if (a.lse && lane == 0) a.lse[static_cast<size_t>(n) * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

eagle_status_t check_args(const eagle_kv_cache_t* c, const eagle_kv_attention_t* w, const char* who, KvPool* pool) {
  const eagle_status_t r = kv_pool(c, who, pool);
  if (r != EAGLE_OK) return r;
  if (!w) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null arguments", who);
  if (w->B < 1 || w->N < 0 || w->max_rows < 1 || w->max_len < 1)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need B, max_rows, max_len >= 1 and N >= 0", who);
  if (w->n_heads < 1 || w->n_heads % c->n_kv_heads || w->n_heads / c->n_kv_heads > KA_MAX_GROUP)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: n_heads must be 1..%d times n_kv_heads", who, KA_MAX_GROUP);
  if (w->mask && (w->mask_slots < 1 || w->mask_slots > 64 || w->max_rows > w->mask_slots))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: a mask needs max_rows <= mask_slots <= 64", who);
  if (!std::isfinite(w->scale) || w->scale < 0.f) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: scale must be finite and not negative", who);
  return EAGLE_OK;
}

}  // namespace

extern "C" int64_t eagle_kv_attention_workspace(const eagle_kv_cache_t* cache, const eagle_kv_attention_t* args) {
  KvPool p;
  if (check_args(cache, args, "kv_attention_workspace", &p) != EAGLE_OK) return -1;
  return 0;
}

extern "C" eagle_status_t eagle_kv_attention(const eagle_kv_cache_t* cache, const eagle_kv_attention_t* w, uint32_t* err_word,
                                             void* stream) {
  const char* who = "kv_attention";
  KaArgs a;
  const eagle_status_t r = check_args(cache, w, who, &a.pool);
  if (r != EAGLE_OK) return r;
  if (!err_word || !w->cu_rows || !w->lens || !w->q || !w->out) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  const int hd = cache->head_dim;
  const long long width = static_cast<long long>(w->n_heads) * hd;
  if (w->q_stride < width || w->out_stride < width || w->q_stride % 8 || w->out_stride % 8 ||
      reinterpret_cast<uintptr_t>(w->q) % 16 || reinterpret_cast<uintptr_t>(w->out) % 16)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned and not overlap", who);
  const int64_t need = eagle_kv_attention_workspace(cache, w);
  if (need > 0 && (!w->workspace || w->workspace_bytes < need || reinterpret_cast<uintptr_t>(w->workspace) % 16))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: needs %lld bytes of workspace, 16-byte aligned", who, static_cast<long long>(need));
  if (w->N == 0) return EAGLE_OK;
  a.B = w->B;
  a.N = w->N;
  a.Hq = w->n_heads;
  a.max_rows = w->max_rows;
  a.max_len = w->max_len;
  a.S = w->mask_slots;
  a.cu = w->cu_rows;
  a.lens = w->lens;
  a.q = static_cast<const __nv_bfloat16*>(w->q);
  a.q_ld = w->q_stride;
  a.mask = w->mask;
  a.scale = w->scale > 0.f ? w->scale : 1.0f / std::sqrt(static_cast<float>(hd));
  a.out = static_cast<__nv_bfloat16*>(w->out);
  a.out_ld = w->out_stride;
  a.lse = w->lse;
  a.err = err_word;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long ctas = (static_cast<long long>(w->N) * w->n_heads + 3) / 4;
  if (ctas > 0x7fffffff) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: too many rows", who);
  const dim3 grid(static_cast<unsigned>(ctas));
  const bool bf = cache->kind == EAGLE_CACHE_BF16;
  if (hd == 64 && bf) kv_attention_rows<64, EAGLE_CACHE_BF16><<<grid, 128, 0, st>>>(a);
  else if (hd == 64) kv_attention_rows<64, EAGLE_CACHE_F4><<<grid, 128, 0, st>>>(a);
  else if (bf) kv_attention_rows<128, EAGLE_CACHE_BF16><<<grid, 128, 0, st>>>(a);
  else kv_attention_rows<128, EAGLE_CACHE_F4><<<grid, 128, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}
