// Device helpers and host checks shared by the paged-cache kernels (kvcache.cu, kvattn.cu).
#pragma once

#include "../../include/eagle_draft.h"
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace eagle {

constexpr unsigned DEVERR_PAGE = 0x10u;

// What a kernel needs of an eagle_kv_cache_t.
struct KvPool {
  void* k;
  void* v;
  void* ks;
  void* vs;
  float kg, vg;
  const int* table;
  int max_pages, num_pages, Hkv, hd;
  int ps_log;                 // page_size = 1 << ps_log
};

// Page of token t of request b, or -1 (and DEVERR_PAGE) when the table or the pool ends before it.
EAGLE_DEV int kv_page(const KvPool& c, int b, int t, unsigned* err) {
  const int i = t >> c.ps_log;
  int page = -1;
  if (t >= 0 && i < c.max_pages) page = __ldg(c.table + static_cast<size_t>(b) * c.max_pages + i);
  if (page < 0 || page >= c.num_pages) {
    atomicOr(err, DEVERR_PAGE);
    return -1;
  }
  return page;
}

// Index of (page, head, row)'s row in the pool, in rows of hd elements.
EAGLE_DEV size_t kv_row(const KvPool& c, int page, int head, int t) {
  return (((static_cast<size_t>(page) * c.Hkv + head) << c.ps_log) + (t & ((1 << c.ps_log) - 1)));
}

// Request that owns row n under cu [B + 1] (ascending), or -1 for a row outside every request.
EAGLE_DEV int row_owner(const int* cu, int B, int n) {
  if (n < __ldg(cu) || n >= __ldg(cu + B)) return -1;
  int lo = 0, hi = B;                       // cu[lo] <= n < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= n) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Flags ranges cu [B + 1] that descend or leave [0, n], and negative lengths (lens may be null).
// Thread `i` of `threads` (in one CTA of a grid: the word is the call's).
EAGLE_DEV void check_ranges(const int* cu, const int* lens, int B, int n, int i, int threads, unsigned* err) {
  bool bad = false;
  for (; i < B; i += threads) {
    const int c0 = __ldg(cu + i), c1 = __ldg(cu + i + 1);
    bad |= c0 < 0 || c1 < c0 || c1 > n || (lens && __ldg(lens + i) < 0);
  }
  if (bad) atomicOr(err, DEVERR_PREFIX);
}

// the larger of two, NaN if either is
EAGLE_DEV float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// two floats to a packed bf16 pair (the first in the low half)
EAGLE_DEV uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two floats to e2m1 codes in a byte (a in the low nibble), nearest, ties to even, saturating.
EAGLE_DEV uint32_t e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
EAGLE_DEV uint32_t f32_to_e4m3(float x) {
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}
EAGLE_DEV float e4m3_to_f32(uint32_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3)));
}
// The values of the two e2m1 codes in the low byte of w (low nibble first).
EAGLE_DEV float2 e2m1_pair_f32(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 t<4>;\n\tmov.b32 {t0, t1, t2, t3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t0;\n\t}" : "=r"(h) : "r"(w));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Checks a cache struct and fills the kernels' view; `who` names the entry point in messages.
eagle_status_t kv_pool(const eagle_kv_cache_t* cache, const char* who, KvPool* out);
// set_last_error with a format, returning `st`
eagle_status_t kv_fail(eagle_status_t st, const char* fmt, ...);

}  // namespace eagle
