// The caller's paged key / value cache: rotary positions, appending a step's rows, gathering
// pages into the packed prefix, keeping an accepted path.  See include/eagle_draft.h.
#include "kvcache.cuh"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <type_traits>

namespace eagle {

eagle_status_t kv_fail(eagle_status_t st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

static bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

eagle_status_t kv_pool(const eagle_kv_cache_t* c, const char* who, KvPool* out) {
  if (!c) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null cache", who);
  if (c->kind != EAGLE_CACHE_BF16 && c->kind != EAGLE_CACHE_F4)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: unknown cache kind %d", who, c->kind);
  if (c->head_dim != 64 && c->head_dim != 128)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128, not %d", who, c->head_dim);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: page_size must be 16, 32, 64 or 128, not %d", who, c->page_size);
  if (c->n_kv_heads < 1 || c->num_pages < 1 || c->max_pages < 1)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: n_kv_heads, num_pages and max_pages must be at least 1", who);
  if (static_cast<long long>(c->num_pages) * c->n_kv_heads >= (1ll << 31) / c->page_size)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: num_pages * n_kv_heads * page_size must be below 2^31", who);
  const bool f4 = c->kind == EAGLE_CACHE_F4;
  if (!c->k || !c->v || !c->page_table || (f4 && (!c->k_scale || !c->v_scale)))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null cache pointer", who);
  if (!aligned16(c->k) || !aligned16(c->v) || (f4 && (!aligned16(c->k_scale) || !aligned16(c->v_scale))))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: cache pointers must be 16-byte aligned", who);
  if (f4 && !(c->k_global >= 1e-30f && c->v_global >= 1e-30f && c->k_global <= 1e30f && c->v_global <= 1e30f))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: k_global and v_global must lie in 1e-30 .. 1e30", who);
  out->k = c->k;
  out->v = c->v;
  out->ks = c->k_scale;
  out->vs = c->v_scale;
  out->kg = c->k_global;
  out->vg = c->v_global;
  out->table = c->page_table;
  out->max_pages = c->max_pages;
  out->num_pages = c->num_pages;
  out->Hkv = c->n_kv_heads;
  out->hd = c->head_dim;
  out->ps_log = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  return EAGLE_OK;
}

namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;
constexpr int RT_MAX_PAIRS = 128;            // rot_dim <= 256

// inv_freq as fractions of a turn in 64-bit fixed point, to the nearest: position * turn[i] mod 2^64
// is the angle's fraction of a turn, exact but for |position| 2^-65 turns.
struct RopeTab {
  unsigned long long turn[RT_MAX_PAIRS];
  int pairs;                                 // rot_dim / 2 (0: no rotation)
  int inter;
  float amp;
};

struct RotArgs {
  // source rows: queries (or eagle_rotary's x), keys, values
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  long long q_ld, k_ld, v_ld, qo_ld;         // row strides, elements
  int Hq, Hk, Hv;                            // heads of each part (0: absent)
  int N, hd;
  const int* positions;
  // append only
  int B;
  const int* cu;
  const int* lens;
  unsigned* err;
  KvPool pool;
  int rows_per_cta, slices;
};

// 8 consecutive values of a row as loaded: two 16-byte words of floats or one of bf16
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
EAGLE_DEV Raw8<T> load_raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    r.w[4 * i] = u.x;
    r.w[4 * i + 1] = u.y;
    r.w[4 * i + 2] = u.z;
    r.w[4 * i + 3] = u.w;
  }
  return r;
}
EAGLE_DEV void unpack8(const Raw8<float>& r, float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
}
EAGLE_DEV void unpack8(const Raw8<__nv_bfloat16>& r, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
EAGLE_DEV void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
EAGLE_DEV uint4 pack8(const float* x) { return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])); }
EAGLE_DEV void store8(__nv_bfloat16* p, const float* x) { *reinterpret_cast<uint4*>(p) = pack8(x); }

// Of the codes `less` and `more` on either side of `border` (in units of `unit`, whose product with it is
// exact) the one of x: nearest, the even code where x lies on it.
EAGLE_DEV uint32_t nearer(float x, uint32_t less, uint32_t more, float border, double unit) {
  const double m = static_cast<double>(border) * unit, v = static_cast<double>(x);
  return v > m || (v == m && (more & 1u) == 0u) ? more : less;
}
// 8 dims of a cached row in 4 bits; the 16-dim group's other half is in lane ^ 1.  `w` holds them
// as bf16: the scale and the codes depend on the stored precision alone and not on how the rotation
// was rounded.  Called by whole warps; `live` lanes store.
//
// Quotients are products with reciprocals (an IEEE division each took half the kernel's time), so one
// next to a border between two codes needs care.  With a power of two as global factor it is enough
// to round the quotient to fewer bits, so that one that lies on a border lies on it exactly:
//   scale: largest / (6 global) to 18 bits (Veltkamp's splitting; borders have 5);
//   code:  value / unit, off by less than 2^-19 up to 6, to multiples of 2^-18 (adding and taking
//          away 48; borders are multiples of 1/4, and a bf16 value over a 4-bit scale that is not
//          on one is 2^-11 or more away).
// With another factor a quotient may lie as close to a border as it likes.  Rounded like this it still
// never crosses one; where one meets a multiple of 1/4 (the scale's: where the codes of a little less
// and a little more differ) the warp compares its values with the borders themselves, whose products
// with the scale and the factor have at most 32 bits (exact in a double; rare, but for zeros and for a
// factor that is a simple multiple of a bf16 value).  POW2: both factors are powers of two; the two forms in one
// kernel cost append_prompt_f4's append 51 us where it takes 46, other factors take 49.
template <bool POW2>
EAGLE_DEV void store8_f4(uint8_t* code, uint8_t* scale, uint4 w, float global, float inv6, bool live, bool even) {
  float y[8];
  unpack8(Raw8<__nv_bfloat16>{{w.x, w.y, w.z, w.w}}, y);
  float top = max_nan(max_nan(max_nan(fabsf(y[0]), fabsf(y[1])), max_nan(fabsf(y[2]), fabsf(y[3]))),
                       max_nan(max_nan(fabsf(y[4]), fabsf(y[5])), max_nan(fabsf(y[6]), fabsf(y[7]))));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  if (__any_sync(0xffffffffu, top != top)) {   // NaN has no code: stored as 0
    top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = y[e] != y[e] ? 0.f : y[e];
      top = fmaxf(top, fabsf(y[e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  }
  float ratio = fminf(__fmul_rn(top, inv6), 1024.f);   // (past 448 the scale saturates)
  const float cut = __fmul_rn(ratio, 65.f);
  uint32_t s = f32_to_e4m3(__fsub_rn(cut, __fsub_rn(cut, ratio)));
  float unit = e4m3_to_f32(s) * global, inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(unit));
  if (!(unit > 0.f)) inv = 0.f;
  uint32_t q = 0, near = 0xFFFFu;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float r0 = __fmaf_rn(fabsf(y[e]), inv, 48.f), r1 = __fmaf_rn(fabsf(y[e + 1]), inv, 48.f);
    if (!POW2) near = min(near, min(__float_as_uint(r0) & 0xFFFFu, __float_as_uint(r1) & 0xFFFFu));   // (0: a multiple of 1/4)
    q |= e2m1x2(copysignf(__fadd_rn(r0, -48.f), y[e]), copysignf(__fadd_rn(r1, -48.f), y[e + 1])) << (4 * e);
  }
  if constexpr (!POW2) {
    const uint32_t less = f32_to_e4m3(ratio * (1.f - 0x1p-20f)), more = f32_to_e4m3(ratio * (1.f + 0x1p-20f));
    const bool pow2 = (__float_as_uint(global) & 0x7FFFFFu) == 0u;   // (of this tensor alone)
    if (__any_sync(0xffffffffu, !pow2 && (near == 0u || less != more))) {
      if (less != more) s = nearer(top, less, more, 0.5f * (e4m3_to_f32(less) + e4m3_to_f32(more)), 6.0 * static_cast<double>(global));
      const double step = static_cast<double>(e4m3_to_f32(s)) * static_cast<double>(global);
      unit = static_cast<float>(step);
      inv = unit > 0.f ? 1.f / unit : 0.f;
      q = 0;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {          // (one value at a time: the kernel holds this block eight times)
        const uint32_t pair = e & 4 ? (e & 2 ? w.w : w.z) : (e & 2 ? w.y : w.x);
        const float x = __uint_as_float(e & 1 ? pair & 0xFFFF0000u : pair << 16), mag = x == x ? fabsf(x) : 0.f, t = mag * inv;
        const uint32_t both = e2m1x2(t * (1.f - 0x1p-20f), t * (1.f + 0x1p-20f));
        uint32_t c = both & 15u;
        if (c != both >> 4) {
          const float2 f = e2m1_pair_f32(both);
          c = nearer(mag, c, both >> 4, 0.5f * (f.x + f.y), step);
        }
        q |= (x == x ? c | (__float_as_uint(x) >> 31) << 3 : 0u) << (4 * e);
      }
    }
  }
  if (!(unit > 0.f)) q = 0u;                 // (of a scale of 0 the codes are 0, not the codes of -0)
  if (live) {
    *reinterpret_cast<uint32_t*>(code) = q;
    if (even) *scale = static_cast<uint8_t>(s);
  }
}

// Rotates heads and (CACHE != 0) stores keys and values in their pages.  A lane holds 8
// consecutive dims of one head: hd / 8 lanes per head, as many whole heads per warp as fit; a
// half-layout pair's other dim comes from another lane of the head by a shuffle, so every load
// of a head precedes its stores (in place is safe).  The CTA computes the cos / sin of its rows
// once into shared memory; a warp keeps one row's in registers over all the heads it takes.
// CACHE: 0 eagle_rotary, else eagle_cache_kind_t.  Bound by bytes where there are many rows
// (8,191 x 64 fp32 heads: 85 us, 92% of the measured copy rate); with 4-bit stores by latency, of its
// loads and of the chain that finds a row's place, at 24 warps an SM (80 registers; issue in 0.56 of
// the cycles, loads the largest stall): 8,188 rows, 48 heads: 46 us, 26 of them its 176 MB.  POW2:
// the 4-bit cache's global factors are powers of two.
template <typename T, int CACHE, bool POW2>
__global__ void __launch_bounds__(RT_THREADS) rotate_kernel(const RotArgs a, const RopeTab rt) {
  __shared__ float2 cs[RT_WARPS][RT_MAX_PAIRS];
  __shared__ int s_page[RT_WARPS], s_tok[RT_WARPS], s_req[RT_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.rows_per_cta, row0 = blockIdx.x * rows;
  // many rows: they come into L2 while their places are found (a chain of five loads; without it
  // append_prompt_f4 took 61 us, now 55; eagle_rotary, which has no places to find, lost by it)
  if (CACHE != 0 && rows >= 4 && blockIdx.y == 0) {
    auto fetch = [&](const void* p, long long ld, int H) {
      const int lines = static_cast<int>((static_cast<long long>(H) * a.hd * sizeof(T) + 127) >> 7);
      for (int r = warp; r < rows && row0 + r < a.N; r += RT_WARPS)
        for (int i = lane; i < lines; i += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(static_cast<const T*>(p) + (row0 + r) * ld) + i * 128ll));
    };
    if (a.Hq) fetch(a.q, a.q_ld, a.Hq);
    fetch(a.k, a.k_ld, a.Hk);
    fetch(a.v, a.v_ld, a.Hv);
  }
  if (CACHE != 0 && tid < rows) {
    const int n = row0 + tid;
    const int b = n < a.N ? row_owner(a.cu, a.B, n) : -1;
    int page = -1, t = 0;
    if (b >= 0) {
      const int len = __ldg(a.lens + b);
      if (len >= 0) {                        // (rows behind a negative length are skipped; flagged below)
        t = static_cast<int>(static_cast<unsigned>(len) + static_cast<unsigned>(n - __ldg(a.cu + b)));   // (past 2^31: no page)
        page = kv_page(a.pool, b, t, a.err);
      }
    }
    s_req[tid] = b;
    s_page[tid] = page;
    s_tok[tid] = t;
  }
  // (the warps that find no places, while warp 0 does)
  if (CACHE != 0 && blockIdx.x == 0 && blockIdx.y == 0 && warp > 0) check_ranges(a.cu, a.lens, a.B, a.N, tid - 32, RT_THREADS - 32, a.err);
  for (int i = tid; i < rows * rt.pairs; i += RT_THREADS) {
    const int r = i / rt.pairs, j = i - r * rt.pairs;
    if (row0 + r < a.N) {
      const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(__ldg(a.positions + row0 + r))) * rt.turn[j];
      // the nearest quarter turn and what is left of it, at most an eighth: only that is rounded to fp32
      const unsigned long long up = ph + (1ull << 61);
      const long long left = static_cast<long long>(up & ((1ull << 62) - 1)) - (1ll << 61);
      float s, c;
      sincospif(__ll2float_rn(left) * 1.0842021724855044e-19f, &s, &c);   // half turns: 2^-63
      if ((up >> 62) & 1) {
        const float t = s;
        s = c;
        c = -t;
      }
      if (up >> 63) {
        s = -s;
        c = -c;
      }
      cs[r][j] = make_float2(c * rt.amp, s * rt.amp);
    }
  }
  __syncthreads();
  const int wpr = RT_WARPS / rows;           // warps per row
  const int r = warp / wpr, n = row0 + r;
  if (n >= a.N) return;
  if (CACHE != 0 && s_req[r] < 0) return;
  const int lph = a.hd >> 3, hpw = 32 / lph; // lanes per head, heads per warp
  const int sub = lane / lph, o = lane - sub * lph;
  const bool in_warp = sub < hpw;
  const int ro = rt.pairs >> 3;              // octets of one half of the rotated dims
  const bool rot = o < 2 * ro;
  // this lane's factors: y[e] = x[e] * c[e] + other[e] * s[e]
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
    if (rot) {
      const int j = rt.inter ? 4 * o + (e >> 1) : 8 * (o < ro ? o : o - ro) + e;
      const float2 f = cs[r][j];
      c[e] = f.x;
      s[e] = (rt.inter ? (e & 1) == 0 : o < ro) ? -f.y : f.y;
    }
  }
  const int other = rot && !rt.inter ? (o < ro ? lane + ro : lane - ro) : lane;
  const bool whole = 2 * rt.pairs == a.hd;   // every dim is rotated
  const int page = CACHE != 0 ? s_page[r] : -1;
  const size_t row0_of = CACHE != 0 && page >= 0 ? kv_row(a.pool, page, 0, s_tok[r]) : 0;   // head 0's pool row
  const int head_rows = CACHE != 0 ? 1 << a.pool.ps_log : 0;                                // from head to head
  const float inv6k = CACHE == EAGLE_CACHE_F4 ? __fdiv_rn(1.f, 6.f * a.pool.kg) : 0.f;
  const float inv6v = CACHE == EAGLE_CACHE_F4 ? __fdiv_rn(1.f, 6.f * a.pool.vg) : 0.f;
  // PART 0: rotated to q_out; 1: rotated to the keys' pages; 2: as they are to the values' pages
  auto put = [&](auto part, int h, bool live, const Raw8<T>& raw) {
    constexpr int PART = decltype(part)::value;
    float y[8];
    if constexpr (PART == 2) {
      unpack8(raw, y);
    } else {
      float x[8];
      unpack8(raw, x);
      if (rt.inter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e], c[e], x[e ^ 1] * s[e]);
      } else {
        Raw8<T> oth;
        float z[8];
#pragma unroll
        for (int e = 0; e < static_cast<int>(2 * sizeof(T)); ++e) oth.w[e] = __shfl_sync(0xffffffffu, raw.w[e], other);
        unpack8(oth, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e], c[e], z[e] * s[e]);
      }
      if (!whole && !rot) {                  // dims behind rot_dim: as they are
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
      }
    }
    if constexpr (PART == 0) {
      if (live) store8(static_cast<T*>(a.q_out) + n * a.qo_ld + (h * a.hd + 8 * o), y);
    } else if constexpr (CACHE == EAGLE_CACHE_BF16) {
      if (live && page >= 0)
        store8(static_cast<__nv_bfloat16*>(PART == 1 ? a.pool.k : a.pool.v) + (row0_of + static_cast<size_t>(h) * head_rows) * a.hd + 8 * o, y);
    } else if constexpr (CACHE == EAGLE_CACHE_F4) {
      const size_t row = row0_of + static_cast<size_t>(h) * head_rows;
      uint4 w;
      if constexpr (PART == 2 && sizeof(T) == 2) w = make_uint4(raw.w[0], raw.w[1], raw.w[2], raw.w[3]);
      else w = pack8(y);
      const float global = PART == 1 ? a.pool.kg : a.pool.vg;
      store8_f4<POW2>(static_cast<uint8_t*>(PART == 1 ? a.pool.k : a.pool.v) + row * (a.hd >> 1) + 4 * o,
                static_cast<uint8_t*>(PART == 1 ? a.pool.ks : a.pool.vs) + row * (a.hd >> 4) + (o >> 1), w, global,
                PART == 1 ? inv6k : inv6v, live && page >= 0, (o & 1) == 0);
    }
  };
  // A part's heads over the row's warps, HB steps of a warp in flight: their loads come before
  // the first store (which might alias them).  Each part starts behind the last one's warps.
  constexpr int HB = 4;
  const int warps = wpr * a.slices;
  int first = blockIdx.y * wpr + warp % wpr;
  auto part_of = [&](auto part, const void* src, long long ld, int H) {
    const T* p = static_cast<const T*>(src) + n * ld + 8 * o;
    const int steps = (H + hpw - 1) / hpw;   // of hpw heads
    for (int i0 = first; i0 < steps; i0 += HB * warps) {
      Raw8<T> raw[HB];
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        const int h = (i0 + i * warps) * hpw + sub;
#pragma unroll
        for (int e = 0; e < static_cast<int>(2 * sizeof(T)); ++e) raw[i].w[e] = 0u;
        if (in_warp && h < H) raw[i] = load_raw8(p + static_cast<long long>(h) * a.hd);
      }
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        const int h = (i0 + i * warps) * hpw + sub;
        if (i0 + i * warps < steps) put(part, h, in_warp && h < H, raw[i]);
      }
    }
    first = (first + warps - steps % warps) % warps;
  };
  if (a.Hq) part_of(std::integral_constant<int, 0>{}, a.q, a.q_ld, a.Hq);
  if constexpr (CACHE != 0) {
    part_of(std::integral_constant<int, 1>{}, a.k, a.k_ld, a.Hk);
    part_of(std::integral_constant<int, 2>{}, a.v, a.v_ld, a.Hv);
  }
}

// ------------------------------------------------------------------------- gather
constexpr int GA_THREADS = 256;
constexpr int GA_TOKENS = 16;
constexpr int GA_STEPS = 4;

struct GatherArgs {
  KvPool pool;
  int B, total;
  unsigned by_heads;                         // ceil(2^32 / Hkv): j / Hkv by a product, exact for j < 16 Hkv, Hkv < 2^14; 0 for one head
  const int* cu;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  unsigned* err;
};

// A CTA writes GA_TOKENS packed rows of K (blockIdx.y = 0) or V, 16 bytes per thread and step,
// consecutive threads consecutive bytes of the output; reads come in runs of one head's row.
// Loads of GA_STEPS steps are issued before the first store.  67,966 tokens of 8 heads out of 4
// bits: 58 us, 90% of the measured copy rate.
template <int HD, int CACHE>
__global__ void __launch_bounds__(GA_THREADS) gather_kernel(const GatherArgs a) {
  constexpr int OCT = HD / 8, ROWS = GA_THREADS / OCT;     // rows (token, head) a step covers
  __shared__ int s_page[GA_TOKENS], s_tok[GA_TOKENS];
  const int t0 = blockIdx.x * GA_TOKENS, tid = threadIdx.x;
  if (tid < GA_TOKENS) {
    const int n = t0 + tid;
    const int b = n < a.total ? row_owner(a.cu, a.B, n) : -1;
    int page = -2, t = 0;                    // -2: no request's row, left as it was
    if (b >= 0) {
      t = n - __ldg(a.cu + b);
      page = kv_page(a.pool, b, t, a.err);   // -1: zeros
    }
    s_page[tid] = page;
    s_tok[tid] = t;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid >= 32) check_ranges(a.cu, nullptr, a.B, a.total, tid - 32, GA_THREADS - 32, a.err);
  __syncthreads();
  const bool is_v = blockIdx.y != 0;
  const uint8_t* pool = static_cast<const uint8_t*>(is_v ? a.pool.v : a.pool.k);
  const uint8_t* scales = static_cast<const uint8_t*>(is_v ? a.pool.vs : a.pool.ks);
  const float global = is_v ? a.pool.vg : a.pool.kg;
  __nv_bfloat16* const out = is_v ? a.v_out : a.k_out;
  const int o = tid % OCT, n_rows = GA_TOKENS * a.pool.Hkv;
  for (int j0 = tid / OCT; j0 < n_rows; j0 += GA_STEPS * ROWS) {
    uint4 u[GA_STEPS];
    uint32_t sb[GA_STEPS];
    int page[GA_STEPS];
#pragma unroll
    for (int i = 0; i < GA_STEPS; ++i) {
      const int j = j0 + i * ROWS;
      u[i] = make_uint4(0u, 0u, 0u, 0u);
      sb[i] = 0u;
      page[i] = -2;
      if (j < n_rows) {
        const int tk = a.by_heads ? __umulhi(j, a.by_heads) : j, h = j - tk * a.pool.Hkv;
        page[i] = s_page[tk];
        if (page[i] >= 0) {
          const size_t row = kv_row(a.pool, page[i], h, s_tok[tk]);
          if (CACHE == EAGLE_CACHE_BF16) {
            u[i] = __ldg(reinterpret_cast<const uint4*>(pool + row * (HD * 2)) + o);
          } else {
            u[i].x = __ldg(reinterpret_cast<const uint32_t*>(pool + row * (HD / 2)) + o);
            sb[i] = __ldg(scales + row * (HD / 16) + (o >> 1));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < GA_STEPS; ++i) {
      if (page[i] == -2) continue;
      if (CACHE == EAGLE_CACHE_F4) {
        const uint32_t w = u[i].x;
        const float unit = e4m3_to_f32(sb[i]) * global;
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = e2m1_pair_f32(w >> (8 * e));
          x[2 * e] = f.x * unit;
          x[2 * e + 1] = f.y * unit;
        }
        u[i] = pack8(x);
      }
      *reinterpret_cast<uint4*>(out + (static_cast<size_t>(t0) * a.pool.Hkv + j0 + i * ROWS) * HD + 8 * o) = u[i];
    }
  }
}

// ------------------------------------------------------------------------- accept
constexpr int AK_MAX_CACHES = 64;

struct AcceptCaches {
  char* p[4 * AK_MAX_CACHES];                // k, v, k_scale, v_scale of every cache
};
struct KeepArgs {
  KvPool pool;                               // caches[0]'s shape and table
  int f4, B, S;
  const int* lens;
  const int* accept_len;
  const int* slots;
  int* new_lens;
  unsigned* err;
};

// Moves count rows of `bytes` per (head, row) in units of U: a thread owns a column (head,
// unit) and moves its units in list order, 8 reads in flight.  No place written is the source of
// a later move of the list, so only reads before writes matter, and those are one thread's own.
template <typename U>
EAGLE_DEV void move_rows(const KvPool& c, char* base, int bytes, int count, const int* src_page, const int* src_tok,
                         const int* dst_page, const int* dst_tok) {
  const int units = bytes / static_cast<int>(sizeof(U));
  for (int col = threadIdx.x; col < c.Hkv * units; col += blockDim.x) {
    const int h = col / units, u = col - h * units;
    for (int j0 = 0; j0 < count; j0 += 8) {
      U x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j0 + e < count && src_page[j0 + e] >= 0)
          x[e] = *(reinterpret_cast<const U*>(base + kv_row(c, src_page[j0 + e], h, src_tok[j0 + e]) * bytes) + u);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j0 + e < count && src_page[j0 + e] >= 0 && dst_page[j0 + e] >= 0)
          *(reinterpret_cast<U*>(base + kv_row(c, dst_page[j0 + e], h, dst_tok[j0 + e]) * bytes) + u) = x[e];
    }
  }
}

// One CTA per (request, cache, key / value).  32 trees of 49 slots in 16 layers: 11 us, 68% of the
// measured copy rate for the bytes that move.
__global__ void __launch_bounds__(256) keep_kernel(const KeepArgs a, const __grid_constant__ AcceptCaches caches) {
  __shared__ int src_page[64], src_tok[64], dst_page[64], dst_tok[64], s_end[2], s_run[2];
  const int b = blockIdx.x, tid = threadIdx.x;
  const int base = __ldg(a.lens + b), want = __ldg(a.accept_len + b);
  if (base < 0) {                            // no places: nothing moves, the length stays
    if (tid == 0) {
      atomicOr(a.err, DEVERR_PREFIX);
      if (a.new_lens != a.lens && blockIdx.y == 0 && blockIdx.z == 0) a.new_lens[b] = base;
    }
    return;
  }
  // The path: strictly ascending slots of the tree; anything else ends it.  So slot j >= j, and
  // move j writes place j + 1: the source of a later move only where the path starts with the
  // slots 0, 1, 2, ... (one that names the root).  That run is moved back to front.
  int n = min(max(want, 0), a.S - 1);
  bool wrong = false;
  int s = 0;
  if (tid < 64) {
    s = tid < n ? __ldg(a.slots + static_cast<size_t>(b) * a.S + tid) : 0;
    src_tok[tid] = s;
    s_end[tid >> 5] = s_run[tid >> 5] = 64;
  }
  __syncthreads();
  if (tid < 64) {
    wrong = tid < n && (s <= (tid ? src_tok[tid - 1] : -1) || s >= a.S);
    const unsigned bits = __ballot_sync(0xffffffffu, wrong);
    const unsigned off = __ballot_sync(0xffffffffu, s != tid);
    if ((tid & 31) == 0 && bits) s_end[tid >> 5] = tid + __ffs(bits) - 1;
    if ((tid & 31) == 0 && off) s_run[tid >> 5] = tid + __ffs(off) - 1;
  }
  __syncthreads();
  const int end = min(s_end[0], s_end[1]);
  if (tid == 0 && (want != n || end < n)) atomicOr(a.err, DEVERR_TOKEN);
  n = min(n, end);
  if (tid < n) {
    const int run = min(min(s_run[0], s_run[1]), n), i = tid < run ? run - 1 - tid : tid;
    src_tok[i] = base + s;
    dst_tok[i] = base + 1 + tid;
    src_page[i] = s == tid + 1 ? -1 : kv_page(a.pool, b, base + s, a.err);   // (already in place)
    dst_page[i] = kv_page(a.pool, b, base + 1 + tid, a.err);
  }
  // new_lens apart from lens: written here; in place, after every CTA has read lens
  if (tid == 0 && a.new_lens != a.lens && blockIdx.y == 0 && blockIdx.z == 0) a.new_lens[b] = base + 1 + n;
  __syncthreads();
  const int c = blockIdx.y, w = blockIdx.z;  // cache, 0 keys / 1 values
  if (a.f4) {
    move_rows<uint32_t>(a.pool, caches.p[4 * c + w], a.pool.hd >> 1, n, src_page, src_tok, dst_page, dst_tok);
    move_rows<uint32_t>(a.pool, caches.p[4 * c + 2 + w], a.pool.hd >> 4, n, src_page, src_tok, dst_page, dst_tok);
  } else {
    move_rows<uint4>(a.pool, caches.p[4 * c + w], a.pool.hd * 2, n, src_page, src_tok, dst_page, dst_tok);
  }
}

// The new lengths in place of the old (every CTA of the moves reads those).
__global__ void keep_lens_kernel(const KeepArgs a) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.B || a.lens[b] < 0) return;
  const int n = min(max(__ldg(a.accept_len + b), 0), a.S - 1);
  int prev = -1, j = 0;
  for (; j < n; ++j) {
    const int s = __ldg(a.slots + static_cast<size_t>(b) * a.S + j);
    if (s <= prev || s >= a.S) break;
    prev = s;
  }
  a.new_lens[b] = a.lens[b] + 1 + j;
}

constexpr double INV_2PI = 0.15915494309189535, INV_2PI_LOW = -9.839338337591243e-18;   // 1 / (2 pi) = their sum
eagle_status_t rope_table(const eagle_rope_t* r, int hd, const char* who, RopeTab* t) {
  memset(t, 0, sizeof(*t));
  if (!r) return EAGLE_OK;
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > hd || r->rot_dim > 2 * RT_MAX_PAIRS)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: rot_dim must be a multiple of 16 up to head_dim, not %d", who, r->rot_dim);
  if (r->interleaved != 0 && r->interleaved != 1) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", who);
  if (!r->inv_freq && !(r->theta > 0.0 && std::isfinite(r->theta)))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: theta must be finite and positive", who);
  if (!std::isfinite(r->amplitude)) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: amplitude must be finite", who);
  t->pairs = r->rot_dim / 2;
  t->inter = r->interleaved;
  t->amp = r->amplitude;
  for (int i = 0; i < t->pairs; ++i) {
    const double f = r->inv_freq ? r->inv_freq[i] : std::pow(r->theta, -2.0 * i / r->rot_dim);
    if (!std::isfinite(f) || f < 0.0 || f > 1e6) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: inv_freq must lie in [0, 1e6]", who);
    // f / (2 pi) to twice a double's bits, then its fraction to 64
    const double turns = f * INV_2PI, low = std::fma(f, INV_2PI_LOW, std::fma(f, INV_2PI, -turns));
    const double frac = std::ldexp(turns - std::floor(turns), 64);   // whole turns per position change nothing
    const double whole = std::floor(frac);
    t->turn[i] = static_cast<unsigned long long>(whole) + static_cast<unsigned long long>(std::llrint(frac - whole + std::ldexp(low, 64)));
  }
  return EAGLE_OK;
}

// Rows per CTA and head slices: the more rows, the fewer warps share one, and the more heads its
// cos / sin serve; few rows are spread over warps and CTAs so that each warp has few heads.  (At
// 8,000 rows rotary_prompt takes 85 us with 4 to a CTA, 87 with 8; append_prompt_f4 57 and 55.)
void rotate_shape(RotArgs* a) {
  const int heads = a->Hq + a->Hk + a->Hv, hpw = 32 / (a->hd / 8);
  const int iters = (heads + hpw - 1) / hpw;            // warp steps per row
  const int sms = std::max(1, num_sms());
  a->rows_per_cta = a->N >= (a->Hk ? 16 : 128) * sms ? 8 : a->N >= 4 * sms ? 4 : a->N >= 2 * sms ? 2 : 1;
  const int wpr = RT_WARPS / a->rows_per_cta;
  const long long ctas = (a->N + a->rows_per_cta - 1) / a->rows_per_cta;
  const int most = std::max(1, (iters + wpr - 1) / wpr);
  a->slices = static_cast<int>(std::min<long long>(most, std::max<long long>(1, 4ll * sms / std::max(1ll, ctas))));
}

template <int CACHE, bool POW2 = true>
eagle_status_t launch_rotate(RotArgs& a, const RopeTab& rt, int dtype, const char* who, cudaStream_t st) {
  rotate_shape(&a);
  const dim3 grid((a.N + a.rows_per_cta - 1) / a.rows_per_cta, a.slices);
  if (dtype == EAGLE_DTYPE_BF16) rotate_kernel<__nv_bfloat16, CACHE, POW2><<<grid, RT_THREADS, 0, st>>>(a, rt);
  else rotate_kernel<float, CACHE, POW2><<<grid, RT_THREADS, 0, st>>>(a, rt);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}

// a row array of the caller: 16-byte aligned base and row stride, rows that do not overlap
bool bad_rows(const void* p, long long ld, int H, int hd, int dtype) {
  const int es = dtype == EAGLE_DTYPE_BF16 ? 2 : 4;
  return !aligned16(p) || ld < static_cast<long long>(H) * hd || (ld * es) % 16;
}
// The kernels count rows, and the elements of one row, in 32 bits; a grid's last CTA looks at row
// numbers a few past the end.
constexpr int KV_MAX_ROWS = INT32_MAX - 64;
bool too_large(int N, long long heads, int hd) { return N > KV_MAX_ROWS || heads * hd > INT32_MAX; }

// A call that writes pages: keys, values and scales must be pools of their own.
bool shared_pools(const eagle_kv_cache_t& x, const eagle_kv_cache_t& y, bool same_cache) {
  if (x.k == y.v || x.v == y.k || (!same_cache && (x.k == y.k || x.v == y.v))) return true;
  if (x.kind != EAGLE_CACHE_F4) return false;
  return x.k_scale == y.v_scale || x.v_scale == y.k_scale ||
         (!same_cache && (x.k_scale == y.k_scale || x.v_scale == y.v_scale));
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" eagle_status_t eagle_rotary(int32_t dtype, const void* x, int64_t x_stride, int32_t N, int32_t H,
                                       int32_t head_dim, const int32_t* positions, const eagle_rope_t* rope, void* out,
                                       int64_t out_stride, void* stream) {
  const char* who = "rotary";
  if (!x || !positions || !rope || !out) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (dtype != EAGLE_DTYPE_F32 && dtype != EAGLE_DTYPE_BF16) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: unknown dtype", who);
  if (N < 0 || H < 1) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need N >= 0 and H >= 1", who);
  if (head_dim < 16 || head_dim > 256 || head_dim % 8)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of 8 in 16..256, not %d", who, head_dim);
  if (too_large(N, H, head_dim)) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: more than 2^31 - 65 rows, or 2^31 - 1 elements in one", who);
  if (bad_rows(x, x_stride, H, head_dim, dtype) || bad_rows(out, out_stride, H, head_dim, dtype))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned and not overlap", who);
  if (x == out && x_stride != out_stride) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: in place needs equal strides", who);
  RopeTab rt;
  const eagle_status_t r = rope_table(rope, head_dim, who, &rt);
  if (r != EAGLE_OK) return r;
  if (N == 0) return EAGLE_OK;
  RotArgs a;
  memset(&a, 0, sizeof(a));
  a.q = x;
  a.q_out = out;
  a.q_ld = x_stride;
  a.qo_ld = out_stride;
  a.Hq = H;
  a.N = N;
  a.hd = head_dim;
  a.positions = positions;
  return launch_rotate<0>(a, rt, dtype, who, static_cast<cudaStream_t>(stream));
}

extern "C" eagle_status_t eagle_kv_append(const eagle_kv_cache_t* cache, const eagle_kv_rows_t* w, const eagle_rope_t* rope,
                                          uint32_t* err_word, void* stream) {
  const char* who = "kv_append";
  RotArgs a;
  memset(&a, 0, sizeof(a));
  eagle_status_t r = kv_pool(cache, who, &a.pool);
  if (r != EAGLE_OK) return r;
  if (!w || !err_word || !w->cu_rows || !w->lens || !w->k || !w->v || (rope && !w->positions) || (w->q && !w->q_out))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (w->dtype != EAGLE_DTYPE_F32 && w->dtype != EAGLE_DTYPE_BF16) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: unknown dtype", who);
  if (w->B < 1 || w->N < 0 || (w->q && w->n_heads < 1)) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need B >= 1, N >= 0, n_heads >= 1", who);
  if (w->q && !rope) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: queries need a rope", who);
  const int hd = cache->head_dim, Hkv = cache->n_kv_heads;
  if (too_large(w->N, std::max(Hkv, w->q ? w->n_heads : 0), hd))
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: more than 2^31 - 65 rows, or 2^31 - 1 elements in one", who);
  if (bad_rows(w->k, w->k_stride, Hkv, hd, w->dtype) || bad_rows(w->v, w->v_stride, Hkv, hd, w->dtype) ||
      (w->q && (bad_rows(w->q, w->q_stride, w->n_heads, hd, w->dtype) || bad_rows(w->q_out, w->q_out_stride, w->n_heads, hd, w->dtype))))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned and not overlap", who);
  if (w->q && w->q == w->q_out && w->q_stride != w->q_out_stride)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: in place needs equal strides", who);
  RopeTab rt;
  if ((r = rope_table(rope, hd, who, &rt)) != EAGLE_OK) return r;
  if (w->N == 0) return EAGLE_OK;
  if (shared_pools(*cache, *cache, true)) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: keys and values share a pool", who);
  a.q = w->q;
  a.k = w->k;
  a.v = w->v;
  a.q_out = w->q_out;
  a.q_ld = w->q_stride;
  a.k_ld = w->k_stride;
  a.v_ld = w->v_stride;
  a.qo_ld = w->q_out_stride;
  a.Hq = w->q ? w->n_heads : 0;
  a.Hk = a.Hv = Hkv;
  a.N = w->N;
  a.hd = hd;
  a.positions = w->positions;
  a.B = w->B;
  a.cu = w->cu_rows;
  a.lens = w->lens;
  a.err = err_word;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->kind == EAGLE_CACHE_BF16) return launch_rotate<EAGLE_CACHE_BF16>(a, rt, w->dtype, who, st);
  int e;
  const bool pow2 = std::frexp(cache->k_global, &e) == 0.5f && std::frexp(cache->v_global, &e) == 0.5f;
  return pow2 ? launch_rotate<EAGLE_CACHE_F4>(a, rt, w->dtype, who, st) : launch_rotate<EAGLE_CACHE_F4, false>(a, rt, w->dtype, who, st);
}

extern "C" eagle_status_t eagle_kv_gather(const eagle_kv_cache_t* cache, int32_t B, const int32_t* cu_seqlens, int32_t total,
                                          void* k_out, void* v_out, uint32_t* err_word, void* stream) {
  const char* who = "kv_gather";
  GatherArgs a;
  const eagle_status_t r = kv_pool(cache, who, &a.pool);
  if (r != EAGLE_OK) return r;
  if (B < 1 || total < 0) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need B >= 1 and total >= 0", who);
  if (total > KV_MAX_ROWS) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: more than 2^31 - 65 rows", who);
  if (total == 0) return EAGLE_OK;
  if (!cu_seqlens || !k_out || !v_out || !err_word) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (k_out == v_out) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: k_out and v_out must be buffers of their own", who);
  if (!aligned16(k_out) || !aligned16(v_out)) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: outputs must be 16-byte aligned", who);
  a.B = B;
  a.total = total;
  a.cu = cu_seqlens;
  if (cache->n_kv_heads >= 1 << 14) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: more than 16383 heads", who);
  a.by_heads = cache->n_kv_heads > 1 ? static_cast<unsigned>(((1ull << 32) + cache->n_kv_heads - 1) / cache->n_kv_heads) : 0u;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.err = err_word;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(total) + GA_TOKENS - 1) / GA_TOKENS), 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->kind == EAGLE_CACHE_BF16;
  if (cache->head_dim == 64 && bf) gather_kernel<64, EAGLE_CACHE_BF16><<<grid, GA_THREADS, 0, st>>>(a);
  else if (cache->head_dim == 64) gather_kernel<64, EAGLE_CACHE_F4><<<grid, GA_THREADS, 0, st>>>(a);
  else if (bf) gather_kernel<128, EAGLE_CACHE_BF16><<<grid, GA_THREADS, 0, st>>>(a);
  else gather_kernel<128, EAGLE_CACHE_F4><<<grid, GA_THREADS, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}

extern "C" eagle_status_t eagle_kv_accept(const eagle_kv_cache_t* caches, int32_t n_caches, int32_t B, int32_t S,
                                          const int32_t* lens, const int32_t* accept_len, const int32_t* accept_slots,
                                          int32_t* new_lens, uint32_t* err_word, void* stream) {
  const char* who = "kv_accept";
  if (!caches || n_caches < 1 || n_caches > AK_MAX_CACHES)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need 1..%d caches", who, AK_MAX_CACHES);
  if (!lens || !accept_len || !accept_slots || !new_lens || !err_word)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (B < 1 || S < 1 || S > 64) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need B >= 1 and 1 <= S <= 64", who);
  KeepArgs a;
  AcceptCaches ac;
  memset(&ac, 0, sizeof(ac));
  for (int i = 0; i < n_caches; ++i) {
    KvPool p;
    const eagle_status_t r = kv_pool(caches + i, who, &p);
    if (r != EAGLE_OK) return r;
    const eagle_kv_cache_t &x = caches[i], &y = caches[0];
    if (x.kind != y.kind || x.n_kv_heads != y.n_kv_heads || x.head_dim != y.head_dim || x.page_size != y.page_size ||
        x.num_pages != y.num_pages || x.max_pages != y.max_pages || x.page_table != y.page_table)
      return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: the caches must share one shape and page table", who);
    for (int j = 0; j <= i; ++j)
      if (shared_pools(x, caches[j], j == i))
        return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: caches %d and %d share a pool", who, j, i);
    if (i == 0) a.pool = p;
    ac.p[4 * i] = static_cast<char*>(p.k);
    ac.p[4 * i + 1] = static_cast<char*>(p.v);
    ac.p[4 * i + 2] = static_cast<char*>(p.ks);
    ac.p[4 * i + 3] = static_cast<char*>(p.vs);
  }
  if (new_lens == accept_len || new_lens == accept_slots)   // (every CTA of a request reads the path)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: new_lens may be lens, but not the path", who);
  a.f4 = caches[0].kind == EAGLE_CACHE_F4;
  a.B = B;
  a.S = S;
  a.lens = lens;
  a.accept_len = accept_len;
  a.slots = accept_slots;
  a.new_lens = new_lens;
  a.err = err_word;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  keep_kernel<<<dim3(B, n_caches, 2), 256, 0, st>>>(a, ac);
  if (new_lens == lens) keep_lens_kernel<<<(B + 127) / 128, 128, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}
