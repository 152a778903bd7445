// Work dealt out in line (kvcross.cu, kvfew.cu): the tiles of all items of a call lie in one line, which
// is cut evenly over the CTAs, whatever the sequences' lengths.  An item that a cut divides leaves
// partial results, which a second kernel joins in the CTAs' order.
#pragma once

#include "kvattn.cuh"

namespace eagle {

// Waits of these kernels, bounded by the clock as mbar_wait's are (a poll may suspend the thread for as
// long as the hardware likes, so their number bounds nothing).  32 bits of it, read at every 256th poll: with
// 64, or with a loop of its own behind the first 256, cross_prompt's sizes took 239 and 255 us where 218.
// SLEEP: for roles that may wake up late.
static_assert(WAIT_LIMIT_CYCLES < 1ll << 32, "");
template <bool SLEEP = false>
EAGLE_DEV bool kx_wait(uint32_t bar, uint32_t parity, unsigned* err, volatile int* abort_flag, uint32_t limit = WAIT_LIMIT_CYCLES) {
  uint32_t since = 0;
#pragma unroll 1
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
    if (SLEEP) __nanosleep(32);
    if ((i & 255u) != 255u) continue;
    const uint32_t now = static_cast<uint32_t>(clock64());
    if (i == 255u) since = now;
    if (*abort_flag || now - since > limit) {
      if (!*abort_flag) atomicOr(err, DEVERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
EAGLE_DEV uint32_t ld_acquire_smem(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
EAGLE_DEV void st_release_smem(uint32_t addr, uint32_t x) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
// the same until the count at `addr` has passed n (counts wrap)
EAGLE_DEV bool kx_wait_past(uint32_t addr, uint32_t n, unsigned* err, volatile int* abort_flag, uint32_t limit = WAIT_LIMIT_CYCLES) {
  uint32_t since = 0;
#pragma unroll 1
  for (uint32_t i = 0; static_cast<int>(ld_acquire_smem(addr) - n) <= 0; ++i) {
    if ((i & 255u) != 255u) continue;
    const uint32_t now = static_cast<uint32_t>(clock64());
    if (i == 255u) since = now;
    if (*abort_flag || now - since > limit) {
      if (!*abort_flag) atomicOr(err, DEVERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// How a call's work lies in line: an item is a block of 2^QV_LOG query vectors of one sequence and KV
// head, a unit one tile of KEYS keys of it; per sequence b, KV heads x blocks x tiles (at least 1, to
// write the rows of a sequence without keys).
template <int QV_LOG, int KEYS>
struct Line {
  Req rq;
  int blocks, tiles;
  EAGLE_DEV Line(const KaArgs& a, int b) {
    rq = request(a, b);
    blocks = static_cast<int>((static_cast<long long>(rq.R) * a.G + (1 << QV_LOG) - 1) >> QV_LOG);
    tiles = max((rq.len + KEYS - 1) / KEYS, 1);
  }
  EAGLE_DEV long long units(const KaArgs& a) const { return static_cast<long long>(a.pool.Hkv) * blocks * tiles; }
};
// An item whose first part is CTA c's last segment, and the last CTA with a part of it (0: none).
// [CTAs], ahead of the parts.
struct Cut {
  int last, kvh, row0, v0, qv, slot, pad[2];
};
// Whether the swizzled tiles cannot lie at shared address `ring`.  The call is flagged, and this CTA's cut
// left empty: the join, which follows all the same, takes its places from there.
EAGLE_DEV bool misplaced(uint32_t ring, float* parts, unsigned* err) {
  if ((ring & 1023u) == 0) return false;
  atomicOr(err, DEVERR_TIMEOUT);
  reinterpret_cast<Cut*>(parts)[blockIdx.x].last = 0;
  return true;
}
// x / y (x >= 0, y > 0), by 32 bits where they do
static __device__ __noinline__ long long quotient64(long long x, long long y) { return x / y; }
EAGLE_DEV long long quotient(long long x, long long y) {
  return (x | y) >> 32 ? quotient64(x, y) : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}
// Units of the call, and of a CTA.  By a whole warp.
template <typename L>
EAGLE_DEV long long all_units(const KaArgs& a, int lane) {
  long long n = 0;
  if (a.groups && lane == 0 && (__ldg(a.groups) != 0 || __ldg(a.groups + a.B) != a.requests)) atomicOr(a.err, DEVERR_PREFIX);
#pragma unroll 1
  for (int b = lane; b < a.B; b += 32) n += L(a, b).units(a);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  return n;
}
EAGLE_DEV long long units_per_cta(long long all, int ctas, int least) { return max(quotient(all + ctas - 1, ctas), static_cast<long long>(least)); }
// The sequence that holds unit u, and u's place among its units.  By a whole warp.
template <typename L>
EAGLE_DEV int find_unit(const KaArgs& a, int lane, long long u, long long* rest) {
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const long long n = b0 + lane < a.B ? L(a, b0 + lane).units(a) : 0;
    long long upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, upto > u);
    if (past) {
      const int k = __ffs(past) - 1;
      *rest = u - __shfl_sync(0xffffffffu, upto - n, k);
      return b0 + k;
    }
    u -= __shfl_sync(0xffffffffu, upto, 31);
  }
  *rest = 0;
  return a.B;
}

// v / G of a query vector: the row's index
EAGLE_DEV int row_of(const KaArgs& a, int v) {
  int q = static_cast<int>(__umulhi(static_cast<uint32_t>(v), a.g_inverse));   // off by one at most
  const int r = v - q * a.G;
  q += r >= a.G ? 1 : r < 0 ? -1 : 0;
  return q;
}

// The pages of boxes of `rows` keys from `first` on, 32 at a time and the next 32 ahead (a page looked up
// when its copy is due costs the producer the lookup's latency with every tile).  By a whole warp.
struct Pages {
  int cur, next;
  EAGLE_DEV int load(const KaArgs& a, int b, int first, int len, int rows, int box) const {
    const long long k = first + static_cast<long long>(box) * rows;
    return k < len ? kv_page(a.pool, b, static_cast<int>(k), a.err) : -1;
  }
  EAGLE_DEV void open(const KaArgs& a, int b, int first, int len, int rows, int lane) { next = load(a, b, first, len, rows, lane); }
  // this lane's page for box0 + lane; box0 runs over the multiples of a power of two up to 32, in order
  EAGLE_DEV int get(const KaArgs& a, int b, int first, int len, int rows, int lane, int box0) {
    if ((box0 & 31) == 0) {
      cur = next;
      next = load(a, b, first, len, rows, box0 + 32 + lane);
    }
    return __shfl_sync(0xffffffffu, cur, (box0 + lane) & 31);
  }
};

// 2^(m - M) where m is a part's maximum and M the largest
EAGLE_DEV float part_factor(float m, float M) {
  return m == -INFINITY ? 0.f : M == INFINITY ? (m == INFINITY ? 1.f : 0.f) : exp2f(m - M);
}

// Launches a kernel, with `overlap` before the one ahead of it on the stream has ended.
template <typename K, typename... A>
cudaError_t launch_after(bool overlap, dim3 grid, int threads, size_t smem, cudaStream_t st, K kernel, const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  cfg.stream = st;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace eagle
