// The products of cross attention: many query vectors over all cached keys of a sequence (bf16 or
// 4-bit pages), the keys' tiles dealt out evenly to the SMs.  See kvattn.cu for the notation.
//
// An item is a block of query vectors (row * G + head) of one sequence and KV head, a unit of work
// one tile of 128 keys of an item.  The units of all items lie in one line, which is cut evenly:
// CTA c takes units [c per, (c + 1) per), whatever the sequences' lengths.  An item that a cut
// divides leaves partial results, which a second kernel joins in the CTAs' order.
//
// One CTA per SM: 256 query vectors as two TMEM tiles of 128, each with a softmax warpgroup and an
// MMA thread of its own.  S = Q K^T of 128 keys takes 128 columns, P replaces its first half, O
// takes hd columns.  While one tile's scores are in the softmax the tensor cores work for the other
// tile.  128 keys an instruction, because Q and K both come from shared memory: 128 x 128 x 16 reads
// 8 KB in the 64 cycles that it computes, which is all that shared memory gives (with 64 keys
// kv_attention_tc needs 48 cycles for 32 of work).  P V starts when the first half of P is there.
// An item of at most 128 vectors is taken by both groups, every other tile each, and the two states
// are joined in TMEM: one group alone would leave the tensor cores idle during its softmax.
//
// bf16 p (8 bits) against bf16 values, fp16 p (11 bits) against 4-bit ones; l sums the unrounded p.
// No key that a row does not see enters a product (rows behind the last key are loaded as zeros), so
// values that are not finite reach the rows that see them, and need no second pass.
#include "kvattn.cuh"

#include <algorithm>
#include <atomic>

using namespace eagle;

namespace {

constexpr int KX_QV = 256;                 // query vectors of a block
static_assert(KX_QV == 1 << 8, "Line divides by a shift");
constexpr int KX_DESCS = 4;                // segments in flight between the scheduler and the roles
constexpr int KX_MIN_UNITS = 3;            // units that are worth a CTA
// barriers (0), segments (640), exchange between warps (1024), score factors (3072, 4 bits)
__host__ __device__ constexpr uint32_t kx_misc(int cache) { return cache == EAGLE_CACHE_F4 ? 5120 : 3072; }
constexpr int KX_SOFTMAX = 512;            // softmax threads: two per query vector
// registers per thread of the 4-bit kernel's roles (the launch checks their sum)
constexpr int KX_REG_CTRL = 40, KX_REG_SOFTMAX = 88, KX_REG_CONV = 56;
constexpr int KX_JOIN_V = 32, KX_JOIN_WARPS = 8;

__host__ __device__ constexpr int kx_threads(int cache) { return 128 + KX_SOFTMAX + (cache == EAGLE_CACHE_F4 ? 256 : 0); }
// floats of a partial result: [hd / 4][256] float4 outputs, [256] (maximum, sum)
__host__ __device__ constexpr size_t kx_slot(int hd) { return static_cast<size_t>(KX_QV) * (hd + 2); }

// Part of an item: tiles [t0, t0 + T) of query vectors [v0, v0 + qv) of sequence b.
struct Seg {
  int valid, b, kvh, row0, len, v0, qv, t0, T, slot;   // slot: partial result, -1: the item is whole
  // both groups have the same vectors, every other tile each
  EAGLE_DEV bool both() const { return qv <= KA_QV; }
  EAGLE_DEV bool tiles_of(int g) const { return T > (both() ? g : 0); }
};

// How the units lie in line: per sequence b, KV heads x blocks x tiles (at least 1, to write the
// rows of a sequence without keys).
struct Line {
  Req rq;
  int blocks, tiles;
  EAGLE_DEV Line(const KaArgs& a, int b) {
    rq = request(a, b);
    blocks = static_cast<int>((static_cast<long long>(rq.R) * a.G + KX_QV - 1) >> 8);
    tiles = max((rq.len + KA_CH - 1) / KA_CH, 1);
  }
  EAGLE_DEV long long units(const KaArgs& a) const { return static_cast<long long>(a.pool.Hkv) * blocks * tiles; }
};
// x / y (x >= 0, y > 0), by 32 bits where they do
EAGLE_DEV long long quotient(long long x, long long y) {
  return (x | y) >> 32 ? x / y : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}
// Units of the call, and of a CTA.  By a whole warp.
EAGLE_DEV long long all_units(const KaArgs& a, int lane) {
  long long n = 0;
  if (a.groups && lane == 0 && (__ldg(a.groups) != 0 || __ldg(a.groups + a.B) != a.requests)) atomicOr(a.err, DEVERR_PREFIX);
  for (int b = lane; b < a.B; b += 32) n += Line(a, b).units(a);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  return n;
}
EAGLE_DEV long long units_per_cta(long long all, int ctas) { return max(quotient(all + ctas - 1, ctas), static_cast<long long>(KX_MIN_UNITS)); }
// The sequence that holds unit u, and u's place among its units.  By a whole warp.
EAGLE_DEV int find_unit(const KaArgs& a, int lane, long long u, long long* rest) {
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const long long n = b0 + lane < a.B ? Line(a, b0 + lane).units(a) : 0;
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

// The partial results of a row's own keys (shared attention), behind the prefix's.
struct Own {
  const KaArgs& a;
  size_t at;
  int used;                                // its key ranges (0: the row belongs to no request)
  EAGLE_DEV Own(const KaArgs& o, int n, int h) : a(o), at(static_cast<size_t>(n) * o.Hq + h), used(0) {
    if (n < 0) return;
    const int b = row_owner(o.cu, o.B, n);
    if (b < 0) return;
    const Req rq = request(o, b);
    if (n < rq.row0 || n - rq.row0 >= rq.R) return;
    used = min(o.splits, (rq.len + o.tiles_per_cta * KA_CH - 1) / (o.tiles_per_cta * KA_CH));
  }
  EAGLE_DEV size_t place(int s) const { return s * (static_cast<size_t>(a.N) * a.Hq) + at; }
  EAGLE_DEV float2 ml(int s) const { return a.part_ml[place(s)]; }
};
// 2^(m - M) where m is a part's maximum and M the largest
EAGLE_DEV float part_factor(float m, float M) {
  return m == -INFINITY ? 0.f : M == INFINITY ? (m == INFINITY ? 1.f : 0.f) : exp2f(m - M);
}
// x[0 .. 3] += f y, nothing of a part without weight (whatever it holds)
EAGLE_DEV void add_part(float* x, float f, float4 y) {
  if (f == 0.f) return;
  x[0] = fmaf(f, y.x, x[0]);
  x[1] = fmaf(f, y.y, x[1]);
  x[2] = fmaf(f, y.z, x[2]);
  x[3] = fmaf(f, y.w, x[3]);
}

// 32 scores x -> p = 2^(x rs - mb), packed two to a word (fp16 or bf16), their sum into p8; MORE: and the
// largest of them and of 32 others.  The pipes need 4 cycles a warp for each ex2 and 2 for each maximum,
// product, sum and conversion of a pair: in the order written (volatile), the products two pairs ahead
// of ex2, sums and conversions four behind, they overlap.
EAGLE_DEV void ordered_max3(float& m, float x, float y) { asm volatile("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x), "f"(y)); }
EAGLE_DEV void ordered_exp2(float& x) { asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x)); }
EAGLE_DEV void ordered_fma2(float& x, float& y, float a, float b) {
  asm volatile("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\tfma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
               : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
EAGLE_DEV void ordered_add2(float& x, float& y, float z, float w) {
  asm volatile("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
               : "+f"(x), "+f"(y) : "f"(z), "f"(w));
}
template <bool F16>
EAGLE_DEV float ordered_pack(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return __uint_as_float(r);
}
template <bool F16, bool MORE>
EAGLE_DEV float powers32(float* x, const float* others, float rs, float mb, float* p8, float* pk) {
  constexpr int AHEAD = 2, BEHIND = 4;
  float m[4] = {x[0], x[2], x[4], x[6]};
#pragma unroll
  for (int i = -AHEAD; i < 16 + BEHIND; ++i) {
    const int u = i + AHEAD, w = i - BEHIND;
    if (i >= 0 && i < 16) ordered_exp2(x[2 * i]);
    if (u < 16) {
      if (MORE) ordered_max3(m[u & 3], x[2 * u], x[2 * u + 1]);
      ordered_fma2(x[2 * u], x[2 * u + 1], rs, -mb);
    }
    if (i >= 0 && i < 16) {
      ordered_exp2(x[2 * i + 1]);
      if (MORE) ordered_max3(m[i & 3], others[2 * i], others[2 * i + 1]);
    }
    if (w >= 0) {
      ordered_add2(p8[(2 * w) & 7], p8[((2 * w) & 7) + 1], x[2 * w], x[2 * w + 1]);
      pk[w] = ordered_pack<F16>(x[2 * w], x[2 * w + 1]);
    }
  }
  return max_nan(max3_nan(m[0], m[1], m[2]), m[3]);
}

template <int HD, int CACHE>
__global__ void __launch_bounds__(kx_threads(CACHE), 1)
kv_cross_wide(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const KaArgs a, const KaArgs own,
              const int with_own, float* parts, const int NS) {
  constexpr bool F4 = CACHE == EAGLE_CACHE_F4;
  constexpr float LIFT = F4 ? 7.f : 0.f;     // fp16 p is held times 2^7 (as in kv_attention_tc)
  constexpr int THREADS = kx_threads(CACHE), CONV_WARP = 4 + KX_SOFTMAX / 32, CONV = THREADS - 32 * CONV_WARP;
  constexpr uint32_t ENTRY = ka_entry(HD), HALF = KA_CH * 128, RAW = ka_raw_bytes(HD), RAW_SCALES = HD / 2 * KA_CH;
  constexpr uint32_t T_O = 256;
  extern __shared__ __align__(1024) uint8_t kx_sm[];   // (no byte is left to align it by hand: ring, queries, misc take all)
  uint8_t* sm = kx_sm;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t ring_u = uniform(smem_u32(sm));
  const uint32_t q_u = ring_u + static_cast<uint32_t>(NS) * ENTRY;
  uint8_t* raw = sm + static_cast<uint32_t>(NS + 2) * ENTRY;
  uint8_t* misc = raw + (F4 ? KA_RAW * RAW : 0);
  const uint32_t misc_u = smem_u32(misc);
  // ring full / free, scores there, first / second part of p there, P V done, queries there, segment
  // done, raw tiles full / free, segments full / free, an item of both groups: states there / read,
  // the two warps of 32 vectors
  const uint32_t bar_kvf = misc_u, bar_kve = misc_u + 112, bar_sf = misc_u + 224, bar_pf = misc_u + 240, bar_pe = misc_u + 272,
                 bar_q = misc_u + 288, bar_fin = misc_u + 304, bar_rf = misc_u + 320, bar_re = misc_u + 344, bar_df = misc_u + 368,
                 bar_de = misc_u + 400, bar_x = misc_u + 432, bar_m = misc_u + 448;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 516);
  volatile uint32_t* raw_pages = reinterpret_cast<volatile uint32_t*>(misc + 520);
  Seg* segs = reinterpret_cast<Seg*>(misc + 640);

  pdl_trigger();
  if (ring_u & 1023u) {                      // (the swizzled tiles' alignment)
    if (tid == 0) atomicOr(a.err, DEVERR_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < KA_MAX_SLOTS; ++s) {
      mbar_init(bar_kvf + 8 * s, F4 ? CONV / 32 : 1);
      mbar_init(bar_kve + 8 * s, 2);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar_sf + 8 * g, 1);
      mbar_init(bar_pf + 16 * g, 8);
      mbar_init(bar_pf + 16 * g + 8, 8);
      mbar_init(bar_pe + 8 * g, 1);
      for (int w = 0; w < 4; ++w) mbar_init(bar_m + 32 * g + 8 * w, 2);
      mbar_init(bar_q + 8 * g, 8);
      mbar_init(bar_fin + 8 * g, 1);
      mbar_init(bar_x + 8 * g, KX_SOFTMAX / 32);
    }
    for (int s = 0; F4 && s < KA_RAW; ++s) {
      mbar_init(bar_rf + 8 * s, 1);
      mbar_init(bar_re + 8 * s, F4 ? CONV / 32 : 1);
    }
    for (int s = 0; s < KX_DESCS; ++s) {
      mbar_init(bar_df + 8 * s, 1);
      mbar_init(bar_de + 8 * s, 3 + KX_SOFTMAX / 32 + (F4 ? CONV / 32 : 0));
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  bool ok = true;
  RingPos dp{0, 0};                          // the segment in hand
  // the segment at `p`, for a whole warp or one thread
  auto segment = [&](const RingPos& p) {
    ok = mbar_wait_sleepy(bar_df + 8 * p.slot, p.turn, a.err, abort_flag);
    Seg s = segs[p.slot];
    if (!ok) s.valid = 0;
    return s;
  };

  if (warp < 4) {
    if constexpr (F4) set_regs_down<KX_REG_CTRL>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer: lane = page of the tile
      const uint64_t pol = policy_evict_normal();   // (the other blocks of the sequence read the keys too)
      const int ps = 1 << a.pool.ps_log, per = KA_CH >> a.pool.ps_log, slots = F4 ? KA_RAW : NS;
      RingPos rp{0, 0};
      int e = 0;
      for (;; dp.step(1, KX_DESCS)) {
        const Seg s = segment(dp);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok || !s.valid) break;
        const int end_page = s.len >> a.pool.ps_log, end_rows = F4 ? 0 : s.len & (ps - 1);
        int page = -1;
        for (int x = 0; x < 2 * s.T && ok; ++x, rp.step(1, slots)) {
          const int slot = rp.slot, pi = (s.t0 + (x >> 1)) * per + lane;
          if (!(x & 1)) {
            page = -1;
            if (lane < per && (pi << a.pool.ps_log) < s.len) page = kv_page(a.pool, s.b, pi << a.pool.ps_log, a.err);
          }
          const uint32_t bar = (F4 ? bar_rf : bar_kvf) + 8 * slot;
          if (e >= slots) ok = mbar_wait_sleepy((F4 ? bar_re : bar_kve) + 8 * slot, rp.turn ^ 1, a.err, abort_flag);
          else ++e;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (F4) {
            const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
            const uint32_t codes = static_cast<uint32_t>(ps) * (HD / 2), scales = static_cast<uint32_t>(ps) * (HD / 16);
            if (lane == 0) {
              raw_pages[slot] = have;
              mbar_arrive_expect_tx(bar, __popc(have) * (codes + scales));
            }
            __syncwarp();
            if (page >= 0) {
              const size_t row = kv_row(a.pool, page, s.kvh, 0);
              const uint32_t dst = smem_u32(raw + slot * RAW);
              bulk_load(dst + lane * codes, static_cast<const uint8_t*>(x & 1 ? a.pool.v : a.pool.k) + row * (HD / 2), codes, bar);
              bulk_load(dst + RAW_SCALES + lane * scales, static_cast<const uint8_t*>(x & 1 ? a.pool.vs : a.pool.ks) + row * (HD / 16), scales, bar);
            }
          } else {
            if (lane == 0) mbar_arrive_expect_tx(bar, ENTRY);
            __syncwarp();
            if (lane < per) {   // (a page that is not there reads as zeros: a block outside the map)
              const int blk = page >= 0 ? page * a.pool.Hkv + s.kvh : a.pool.num_pages * a.pool.Hkv;
              const uint32_t dst = ring_u + slot * ENTRY + lane * (ps * 128);
              const int row = pi == end_page && end_rows ? end_rows - ps : 0;
#pragma unroll
              for (int h = 0; h < HD / 64; ++h) tma_load_3d(dst + h * HALF, x & 1 ? &tmv : &tmk, 64 * h, row, blk, bar, pol);
            }
          }
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar_de + 8 * dp.slot);
      }
      if (!ok) {   // let copies already issued land before the CTA releases its shared memory
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ scheduler
      const long long all = all_units(a, lane), per = units_per_cta(all, gridDim.x);
      const long long begin = min(per * blockIdx.x, all), end = min(begin + per, all);
      long long u = begin, rest = 0;
      int b = u < end ? find_unit(a, lane, u, &rest) : 0;
      int n = 0;
      while (ok) {
        Seg s;
        s.valid = 0;
        if (u < end) {
          Line l(a, b);
          while (rest >= l.units(a)) {       // (the next sequence that has units)
            rest -= l.units(a);
            ++b;
            l = Line(a, b);
          }
          const long long item = quotient(rest, l.tiles);
          s.valid = 1;
          s.b = b;
          s.t0 = static_cast<int>(rest - item * l.tiles);
          s.kvh = static_cast<int>(quotient(item, l.blocks));
          s.row0 = l.rq.row0;
          s.len = l.rq.len;
          s.v0 = static_cast<int>(item - static_cast<long long>(s.kvh) * l.blocks) * KX_QV;
          s.qv = static_cast<int>(min(static_cast<long long>(l.rq.R) * a.G - s.v0, static_cast<long long>(KX_QV)));
          const int units = static_cast<int>(min(static_cast<long long>(l.tiles - s.t0), end - u));
          s.T = s.len > 0 ? units : 0;
          s.slot = units == l.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (u == begin ? 0 : 1);
          u += units;
          rest += units;
        }
        if (n >= KX_DESCS) ok = mbar_wait_sleepy(bar_de + 8 * dp.slot, dp.turn ^ 1, a.err, abort_flag);
        else ++n;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          segs[dp.slot] = s;
          mbar_arrive(bar_df + 8 * dp.slot);
        }
        __syncwarp();
        dp.step(1, KX_DESCS);
        if (!s.valid) break;
      }
      if (with_own) pdl_wait();              // (this kernel ends after the one before it)
    } else if (elect_one()) {
      // ------------------------------------------------------------ MMA issuer of group g
      const int g = warp - 2;
      const uint32_t id1 = F4 ? idesc_f16_f32(128, KA_CH) : idesc_bf16_f32(128, KA_CH);
      const uint32_t id2 = (F4 ? idesc_f16_f32(128, HD) : idesc_bf16_f32(128, HD)) | (1u << 16);   // B (values) MN-major
      const uint64_t dq = smem_desc_sw128(q_u + g * ENTRY);
      const uint32_t tS = tmem + 128 * g, tO = tmem + T_O + 128 * g;
      RingPos base{0, 0};                    // the segment's first entry
      uint32_t n = 0, other = 0, turn = 0;   // tiles of this group so far, of the other one; segments with a tile
      bool after_1 = false;                  // the last segment's last tile was group 1's
      for (;; dp.step(1, KX_DESCS)) {
        const Seg s = segment(dp);
        if (!ok || !s.valid) break;
        const bool both = s.both(), work = s.tiles_of(g);
        const int step = both ? 2 : 1;
        if (work) {
          ok = mbar_wait(bar_q + 8 * g, turn, a.err, abort_flag);
          turn ^= 1;
        }
        tc_fence_after();
        RingPos kp = base;
        if (both && g) kp.step(2, NS);
        for (int t = both ? g : 0; t < s.T && ok; t += step, ++n) {
          RingPos vp = kp;
          vp.step(1, NS);
          ok = mbar_wait(bar_kvf + 8 * kp.slot, kp.turn, a.err, abort_flag);
          // The groups take turns, in one order for the whole call: a tile's scores start when those of
          // the tile before, where that is the other group's, are there.  So one group's softmax falls on
          // the other's products; left to themselves they fall into step, both waiting for their softmax
          // at once.  (The other group's next scores come after this tile in the order, so the barrier
          // cannot be a turn ahead.)
          const uint32_t before = other + (both ? t >> 1 : t) + g - 1;
          if (g || t || after_1) ok = ok && mbar_wait(bar_sf + 8 * (g ^ 1), before & 1, a.err, abort_flag);
          if (n) ok = ok && mbar_wait(bar_pe + 8 * g, (n - 1) & 1, a.err, abort_flag);   // (P lies over S)
          if (!ok) break;
          tc_fence_after();
          const uint64_t dk = smem_desc_sw128(ring_u + kp.slot * ENTRY);
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const uint32_t ko = ((j >> 2) * HALF + (j & 3) * 32) >> 4;
            tc_mma_bf16(tS, dq + ko, dk + ko, id1, j > 0 ? 1u : 0u);
          }
          tc_commit(bar_sf + 8 * g);
          tc_commit(bar_kve + 8 * kp.slot);
          if (both) tc_commit(bar_kve + 8 * kp.slot);
          ok = mbar_wait(bar_kvf + 8 * vp.slot, vp.turn, a.err, abort_flag);
          const uint64_t dv = smem_desc_sw128_mn(ring_u + vp.slot * ENTRY, HALF, 1024);
          const bool first = t < step;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && mbar_wait(bar_pf + 16 * g + 8 * h, n & 1, a.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 4; ++x) {    // keys 16 j .. 16 j + 15: part h is 32 keys of each half
              const int j = 4 * (x >> 1) + 2 * h + (x & 1);
              tc_mma_bf16_ta(tO, tS + KA_H * (j >> 2) + 8 * (j & 3), dv + j * 128, id2, first && h == 0 && x == 0 ? 0u : 1u);
            }
          }
          if (!ok) break;
          tc_commit(bar_pe + 8 * g);
          tc_commit(bar_kve + 8 * vp.slot);
          if (both) tc_commit(bar_kve + 8 * vp.slot);
          kp.step(2, NS);
          if (both) kp.step(2, NS);
        }
        if (!ok) break;
        other += both ? (s.T + g) >> 1 : s.T;
        if (s.T > 0) after_1 = !both || (s.T & 1) == 0;
        if (work) tc_commit(bar_fin + 8 * g);
        const uint32_t at = base.slot + 2u * s.T;
        base.turn ^= (at / NS) & 1;
        base.slot = at % NS;
        mbar_arrive(bar_de + 8 * dp.slot);
      }
      if (!ok) {   // let MMAs already issued finish before TMEM is released
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
      }
    }
  } else if (warp >= CONV_WARP) {
    if constexpr (F4) {
      set_regs_down<KX_REG_CONV>();
      // ------------------------------ raw tiles -> fp16 tiles, as in kv_attention_tc
      constexpr int GR = HD / 16, IT = KA_CH * GR / CONV, RSTEP = CONV / GR;
      static_assert(RSTEP % 8 == 0, "the swizzle repeats every 8 rows");
      const int ct = tid - 32 * CONV_WARP, gidx = ct % GR, r0 = ct / GR, sw = gidx >> 2;
      RingPos rp{0, 0}, wp{0, 0};
      int done = 0;
      for (;; dp.step(1, KX_DESCS)) {
        const Seg s = segment(dp);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok || !s.valid) break;
        for (int e = 0; e < 2 * s.T; ++e, rp.step(1, NS), wp.step(1, KA_RAW)) {
          ok = mbar_wait_sleepy(bar_rf + 8 * wp.slot, wp.turn, a.err, abort_flag);
          const uint8_t* src = raw + wp.slot * RAW;
          const uint32_t have = raw_pages[wp.slot];
          const int k0 = (s.t0 + (e >> 1)) * KA_CH;
          uint2 code[IT];
          uint32_t scale[IT];
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const int r = r0 + i * RSTEP;
            code[i] = reinterpret_cast<const uint2*>(src + r * (HD / 2))[gidx];
            scale[i] = src[RAW_SCALES + r * GR + gidx];
          }
          if (k0 + KA_CH > s.len || have != (1u << (KA_CH >> a.pool.ps_log)) - 1u) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {     // rows behind the last key, and of pages that are not there: zeros
              const int r = r0 + i * RSTEP;
              if (k0 + r >= s.len || !((have >> (r >> a.pool.ps_log)) & 1u)) {
                code[i] = make_uint2(0u, 0u);
                scale[i] = 0u;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_re + 8 * wp.slot);
          if (done >= NS) ok = mbar_wait_sleepy(bar_kve + 8 * rp.slot, rp.turn ^ 1, a.err, abort_flag) && ok;
          else ++done;
          ok = !__any_sync(0xffffffffu, !ok);
          if (!ok) break;
          const uint32_t dst = ring_u + rp.slot * ENTRY + sw * HALF, c = 2 * (gidx & 3);
          const uint32_t d0 = dst + ka_sw(r0, c + sw), d1 = dst + ka_sw(r0, c + (sw ^ 1));
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const uint32_t f = scale_pair(scale[i]);
            uint32_t h[4];
            dequant8(sw ? code[i].y : code[i].x, f, h);
            st_smem16(d0 + i * (RSTEP * 128), h);
            dequant8(sw ? code[i].x : code[i].y, f, h);
            st_smem16(d1 + i * (RSTEP * 128), h);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_kvf + 8 * rp.slot);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar_de + 8 * dp.slot);
      }
    }
  } else {
    if constexpr (F4) set_regs_up<KX_REG_SOFTMAX>();
    // ------------------------------------------------------------ softmax of group g
    // Two threads per vector: half hf has columns [64 hf, 64 hf + 64) of the scores.  (Latencies of TMEM
    // and barriers of one warp fall on the ex2 of the other; one thread per vector takes 1530 cycles
    // from the scores to the last p.)
    const int g = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, quad = warp & 3, lv = 32 * quad + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t ts = tmem + lane_base + 128 * g + KA_H * hf, to = tmem + lane_base + T_O + 128 * g;
    const int ps = 1 << a.pool.ps_log;
    float2* states = reinterpret_cast<float2*>(misc + 1024);                  // [group][128]
    float* xch = reinterpret_cast<float*>(misc + 1024) + (4 * g + quad) * 64;   // the pair's [2][32], in the same place
    float* factors = reinterpret_cast<float*>(misc + 3072) + (4 * g + quad) * 32;
    const uint32_t bar_pair = bar_m + 32 * g + 8 * quad;
    uint32_t mturn = 0;
    auto pair_arrive = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_pair);
    };
    auto pair_wait = [&]() {
      ok = mbar_wait(bar_pair, mturn, a.err, abort_flag) && ok;
      mturn ^= 1;
    };
    // 16 of the pair's 32 vectors of a segment into the group's query tile, LR lanes a row (a lane a row
    // would touch 32 rows with every load: 4096 cycles a segment)
    auto stage = [&](const Seg& s) {
      constexpr int LR = HD / 8, ROWS = 32 / LR, N = 16 / ROWS;   // lanes a row, rows a load, loads
      const int v = s.v0 + lv + (s.both() ? 0 : KA_QV * g), c = lane % LR, i = v / a.G;
      const bool live = v - s.v0 < s.qv;
      const long long at = live ? (s.row0 + i) * a.q_ld + static_cast<long long>(s.kvh * a.G + v - i * a.G) * HD : -1;
      uint4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const long long from = __shfl_sync(0xffffffffu, at, 16 * hf + ROWS * k + lane / LR);
        x[k] = from >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + from) + c) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        const int r = 16 * hf + ROWS * k + lane / LR;
        if (F4) {   // fp16, times a power of two: the vector's largest magnitude lies in [2^14, 2^15)
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
          for (int d = 1; d < LR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
          int ex = static_cast<int>(top >> 7);
          ex = ex == 255 ? 127 : max(ex, 30);  // (infinities and NaN pass; tiny vectors)
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack_f16(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
          if (c == 0) factors[r] = finite_scale(a.scale_log2 * a.pool.kg * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23));
        }
        st_smem16(q_u + g * ENTRY + (c >> 3) * HALF + ka_sw(32 * quad + r, c & 7), w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q + 8 * g);
    };
    // the score factor of this thread's vector, once both warps have staged
    auto factor = [&]() {
      if (!F4) return a.scale_log2;
      pair_arrive();
      pair_wait();
      return factors[lane];
    };
    uint32_t n = 0, turn = 0, xturn = 0;     // tiles of this group so far; segments with a tile; items that both groups took
    bool waited = false;                     // for the own keys' results
    Seg s = segment(dp);
    if (__all_sync(0xffffffffu, ok && s.valid && s.tiles_of(g))) stage(s);
    while (__all_sync(0xffffffffu, ok && s.valid)) {
      const bool both = s.both(), work = s.tiles_of(g);
      const float rs = work ? factor() : 0.f;
      const int step = both ? 2 : 1;
      const bool idle = 32 * quad >= s.qv - (both ? 0 : KA_QV * g);   // a pair without vectors
      const int end_page = s.len >> a.pool.ps_log, end_rows = F4 ? 0 : s.len & (ps - 1);
      float m_run = -INFINITY, l_run = 0.f;
      for (int t = both ? g : 0; t < s.T; t += step, ++n) {
        ok = ok && mbar_wait(bar_sf + 8 * g, n & 1, a.err, abort_flag);
        tc_fence_after();
        if (!idle) {
          // The first 32 scores become p with the maximum so far, which mostly stays, while this tile's
          // is found; where that rose too far they are read again.
          float x[KA_H], p8[8], pk[16];
          for (bool again = false;;) {
            tmem_ld32(ts, x);
            tmem_ld32(ts + 32, x + 32);
            const int kt = (s.t0 + t) * KA_CH;
            tmem_wait_ld();
            if (kt + KA_CH > s.len) {        // columns without a key; the page that the keys end inside has its own at its end
              const int at = (end_page << a.pool.ps_log) - kt;
              Bits vis = bits_below(end_rows ? at + ps : s.len - kt);
              if (end_rows) {
                const Bits lo = bits_below(at), hi = bits_below(at + ps - end_rows);
                vis.lo &= lo.lo | ~hi.lo;
                vis.hi &= lo.hi | ~hi.hi;
              }
              const unsigned long long bits = hf ? vis.hi : vis.lo;
#pragma unroll
              for (int e = 0; e < KA_H; ++e) x[e] = (bits >> e) & 1ull ? x[e] : -INFINITY;
            }
            // (a row without a key so far takes the maximum as 0: every score is -inf, every p is 0)
            const float mb = (m_run == -INFINITY ? 0.f : m_run * rs) - LIFT;
#pragma unroll
            for (int e = 0; e < 8; ++e) p8[e] = 0.f;
            float mt = powers32<F4, true>(x, x + 32, rs, mb, p8, pk);
            if (again) break;
            xch[32 * hf + lane] = mt;        // (the other warp read the last tile's before P V, and so before these scores)
            pair_arrive();
            pair_wait();
            mt = max_nan(mt, xch[32 * (hf ^ 1) + lane]);
            const bool rose = mt != -INFINITY && (m_run == -INFINITY || (mt - m_run) * rs > KA_RESCALE);
            if (!__any_sync(0xffffffffu, rose)) break;
            const bool resc = rose && m_run != -INFINITY;
            const float f = resc ? fast_exp2((m_run - mt) * rs) : 1.f;
            if (rose) m_run = mt;
            if (__any_sync(0xffffffffu, resc)) {   // (the scores are there, so the P V before them is done)
#pragma unroll 1
              for (int c0 = 0; c0 < HD / 2; c0 += 16) {
                float z[16];
                tmem_ld16(to + hf * (HD / 2) + c0, z);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] *= f;
                tmem_st16(to + hf * (HD / 2) + c0, z);
              }
            }
            l_run *= f;
            again = true;
          }
          tmem_st16(ts, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_pf + 16 * g);
          powers32<F4, false>(x + 32, x, rs, (m_run == -INFINITY ? 0.f : m_run * rs) - LIFT, p8, pk);
          tmem_st16(ts + 16, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_pf + 16 * g + 8);
          l_run += ((p8[0] + p8[1]) + (p8[2] + p8[3])) + ((p8[4] + p8[5]) + (p8[6] + p8[7]));
        } else if (lane == 0) {
          mbar_arrive(bar_pf + 16 * g);
          mbar_arrive(bar_pf + 16 * g + 8);
        }
      }
      // ---- the next segment's queries, as soon as this one's are read (its last scores are there).
      // The barriers of queries and of the segment's end turn only in segments where the group has a
      // tile: each of their turns then waits for every warp to have seen the one before.
      RingPos np = dp;
      np.step(1, KX_DESCS);
      const bool so_far = ok;
      const Seg s2 = segment(np);
      ok = __all_sync(0xffffffffu, ok && so_far);
      if (ok && s2.valid && s2.tiles_of(g)) stage(s2);
      if (work) {
        ok = mbar_wait(bar_fin + 8 * g, turn, a.err, abort_flag) && ok;
        turn ^= 1;
      }
      tc_fence_after();
      // ---- this segment's result: half of the dims of state g, or a quarter of both groups' states
      const int v = s.v0 + lv + (both ? 0 : KA_QV * g), i = v / a.G, h = s.kvh * a.G + (v - i * a.G);
      const bool live = v - s.v0 < s.qv;
      if (!idle) {
        xch[32 * hf + lane] = l_run;
        pair_arrive();
        pair_wait();
        l_run += xch[32 * (hf ^ 1) + lane];
        pair_arrive();                       // (both have read)
        pair_wait();
      }
      float2 st[2] = {make_float2(l_run == 0.f ? -INFINITY : m_run * rs - LIFT, l_run), make_float2(-INFINITY, 0.f)};
      if (both) {
        if (hf == 0) states[128 * g + lv] = st[0];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_x);
        ok = mbar_wait(bar_x, xturn, a.err, abort_flag) && ok;
        tc_fence_after();
        st[0] = states[lv];
        st[1] = states[128 + lv];
      }
      const uint32_t o0 = tmem + lane_base + T_O + (both ? 0 : 128 * g), o1 = tmem + lane_base + T_O + 128;
      constexpr int CW = HD / 4, BW = CW / 4;  // dims of a chunk, of a block
      const int c_lo = both ? (2 * g + hf) * CW : 2 * hf * CW, c_hi = c_lo + (both ? CW : 2 * CW);
      float M = max_nan(st[0].x, st[1].x);
      const bool join = with_own && s.slot < 0;
      if (join && !waited) {
        pdl_wait();
        waited = true;
      }
      const int row = s.row0 + i;
      Own mine(own, live && join ? row : -1, h);
      for (int k = 0; k < mine.used; ++k) M = max_nan(M, mine.ml(k).x);
      const float f0 = part_factor(st[0].x, M), f1 = part_factor(st[1].x, M);
      float L = fmaf(f0, st[0].y, f1 * st[1].y);
      for (int k = 0; k < mine.used; ++k) {
        const float2 ml = mine.ml(k);
        const float f = part_factor(ml.x, M);
        if (f != 0.f) L = fmaf(f, ml.y, L);
      }
      const bool none = L == 0.f, writes = live && (!join || mine.used > 0);
      const float inv = s.slot >= 0 ? 1.f : none ? 0.f : a.vg / L, own_inv = none ? 0.f : own.vg / L;
      float* part = parts + (s.slot >= 0 ? static_cast<size_t>(s.slot) : 0) * kx_slot(HD);
      const int pv = v - s.v0;
      // Four lanes' rows in chunks of hd / 4 dims are turned so that four lanes hold one row: a store then
      // touches 8 rows instead of 32.
      const long long at = row * a.out_ld + static_cast<long long>(h) * HD;
      const int ranges = join ? __reduce_max_sync(0xffffffffu, mine.used) : 0;
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_hi; c0 += CW) {
        float x[CW];
        __syncwarp();
        if constexpr (CW == 32) tmem_ld32(o0 + c0, x);
        else tmem_ld16(o0 + c0, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < CW; ++e) x[e] = f0 == 0.f ? 0.f : f0 * x[e];
        if (both) {
          float y[CW];
          if constexpr (CW == 32) tmem_ld32(o1 + c0, y);
          else tmem_ld16(o1 + c0, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < CW; ++e) x[e] = f1 == 0.f ? x[e] : fmaf(f1, y[e], x[e]);
        }
        if (s.slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(part) + static_cast<size_t>(c0 / 4) * KX_QV + pv;
          if (writes) {
#pragma unroll
            for (int e = 0; e < CW / 4; ++e) dst[e * KX_QV] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
          continue;
        }
#pragma unroll
        for (int e = 0; e < CW; ++e) x[e] = none ? 0.f : x[e] * inv;
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (b & d) continue;
#pragma unroll
            for (int e = 0; e < BW; ++e) {
              float& lo = x[b * BW + e];
              float& hi = x[(b + d) * BW + e];
              const float got = __shfl_xor_sync(0xffffffffu, lane & d ? lo : hi, d);
              if (lane & d) lo = got;
              else hi = got;
            }
          }
#pragma unroll
        for (int r = 0; r < 4; ++r) {        // block r: lane's dims [c0 + BW (lane % 4), ...) of row (lane & ~3) + r
          const int from = (lane & ~3) + r;
          float* y = x + r * BW;
          const long long to_row = __shfl_sync(0xffffffffu, at, from);
          const bool put = __shfl_sync(0xffffffffu, static_cast<int>(writes), from) != 0;
          const int d0 = c0 + BW * (lane & 3);
          for (int k = 0; k < ranges; ++k) {
            float f = 0.f;
            if (k < mine.used) f = part_factor(mine.ml(k).x, M) * own_inv;
            f = __shfl_sync(0xffffffffu, f, from);
            const size_t place = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(mine.place(k)), from);
            const float4* src = reinterpret_cast<const float4*>(own.part_o + place * HD + d0);
            if (f != 0.f) {
#pragma unroll
              for (int e = 0; e < BW / 4; ++e) add_part(y + 4 * e, f, src[e]);
            }
          }
          if (!put) continue;
          if constexpr (BW == 8)
            *reinterpret_cast<uint4*>(a.out + to_row + d0) = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
          else *reinterpret_cast<uint2*>(a.out + to_row + d0) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        }
      }
      if (writes && hf == 0 && (!both || g == 0)) {
        if (s.slot >= 0) reinterpret_cast<float2*>(part + static_cast<size_t>(KX_QV) * HD)[pv] = make_float2(none ? -INFINITY : M, L);
        else if (a.lse) a.lse[static_cast<size_t>(row) * a.Hq + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
      if (both) {                            // (all have read O and the states before any goes on)
        __syncwarp();
        tc_fence_before();
        if (lane == 0) mbar_arrive(bar_x + 8);
        ok = mbar_wait(bar_x + 8, xturn, a.err, abort_flag) && ok;
        xturn ^= 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_de + 8 * dp.slot);
      dp = np;
      s = s2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the partial results of the items that the cuts divide: block x the item behind CTA x's
// units, if CTA x is the first with a part of it; 32 of its vectors (lanes), HD / 8 dims a warp.
template <int HD>
__global__ void __launch_bounds__(32 * KX_JOIN_WARPS) kv_cross_wide_join(const KaArgs a, const KaArgs own, const int with_own, const float* parts) {
  constexpr int E = HD / 4 / KX_JOIN_WARPS;  // float4s of a thread
  __shared__ Seg s_seg;
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  if (warp == 0) {
    Seg s;
    s.valid = 0;
    int last = 0;
    const long long all = all_units(a, lane), per = units_per_cta(all, gridDim.x), begin = per * c, end = begin + per;
    if (end < all) {
      long long rest;
      s.b = find_unit(a, lane, end - 1, &rest);
      const Line l(a, s.b);
      const long long item = quotient(rest, l.tiles), first = end - 1 - (rest - item * l.tiles), behind = first + l.tiles;
      if (behind > end && first >= begin) {
        s.valid = 1;
        s.kvh = static_cast<int>(quotient(item, l.blocks));
        s.row0 = l.rq.row0;
        s.v0 = static_cast<int>(item - static_cast<long long>(s.kvh) * l.blocks) * KX_QV;
        s.qv = static_cast<int>(min(static_cast<long long>(l.rq.R) * a.G - s.v0, static_cast<long long>(KX_QV)));
        s.slot = 2 * c + (first == begin ? 0 : 1);
        last = static_cast<int>(quotient(behind - 1, per));
      }
    }
    if (lane == 0) {
      s_seg = s;
      s_last = last;
    }
  }
  __syncthreads();
  const Seg s = s_seg;
  const int pv = KX_JOIN_V * blockIdx.y + lane, v = s.v0 + pv, last = s_last;
  pdl_wait();                                // the parts, and the own keys' results
  if (!s.valid || pv >= s.qv) return;
  const int i = v / a.G, h = s.kvh * a.G + (v - i * a.G);
  const size_t row = static_cast<size_t>(s.row0 + i);
  auto part = [&](int k) { return parts + static_cast<size_t>(k == c ? s.slot : 2 * k) * kx_slot(HD); };
  auto state = [&](int k) { return reinterpret_cast<const float2*>(part(k) + static_cast<size_t>(KX_QV) * HD)[pv]; };
  float M = -INFINITY;
#pragma unroll 4
  for (int k = c; k <= last; ++k) M = max_nan(M, state(k).x);
  const Own mine(own, with_own ? static_cast<int>(row) : -1, h);
  if (with_own && mine.used == 0) return;
  for (int k = 0; k < mine.used; ++k) M = max_nan(M, mine.ml(k).x);
  float x[4 * E] = {}, L = 0.f;
#pragma unroll 4
  for (int k = c; k <= last; ++k) {
    const float2 ml = state(k);
    const float f = part_factor(ml.x, M);
    if (f == 0.f) continue;
    L = fmaf(f, ml.y, L);
    const float4* src = reinterpret_cast<const float4*>(part(k)) + static_cast<size_t>(warp * E) * KX_QV + pv;
#pragma unroll
    for (int e = 0; e < E; ++e) add_part(x + 4 * e, f, src[e * KX_QV]);
  }
  float y[4 * E] = {};
  for (int k = 0; k < mine.used; ++k) {
    const float2 ml = mine.ml(k);
    const float f = part_factor(ml.x, M);
    if (f == 0.f) continue;
    L = fmaf(f, ml.y, L);
    const float4* src = reinterpret_cast<const float4*>(own.part_o + mine.place(k) * HD) + warp * E;
#pragma unroll
    for (int e = 0; e < E; ++e) add_part(y + 4 * e, f, src[e]);
  }
  const bool none = L == 0.f;
  const float inv = none ? 0.f : a.vg / L, own_inv = none ? 0.f : own.vg / L;
  uint2* dst = reinterpret_cast<uint2*>(a.out + row * a.out_ld + static_cast<long long>(h) * HD) + warp * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = none ? 0.f : with_own ? fmaf(x[4 * e + k], inv, y[4 * e + k] * own_inv) : x[4 * e + k] * inv;
    dst[e] = make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
  }
  if (warp == 0 && a.lse) a.lse[row * a.Hq + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

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

template <int HD, int CACHE>
cudaError_t launch_wide(const CUtensorMap& tmk, const CUtensorMap& tmv, const KaArgs& a, const KaArgs& own, int with_own, float* parts,
                        int ctas, cudaStream_t st) {
  static std::atomic<size_t> granted[64];    // shared memory per device, set on its first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  size_t cap = dev < 64 ? granted[dev].load() : 0;
  if (!cap) {
    e = allow_max_smem(reinterpret_cast<const void*>(kv_cross_wide<HD, CACHE>), &cap);
    if (e != cudaSuccess) return e;
    if (CACHE == EAGLE_CACHE_F4) {   // the roles' registers must fit what the launch gives, or they would wait for ever
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kv_cross_wide<HD, CACHE>);
      if (e != cudaSuccess) return e;
      const int need = 128 * KX_REG_CTRL + KX_SOFTMAX * KX_REG_SOFTMAX + 256 * KX_REG_CONV;
      if (fa.numRegs / 8 * 8 * kx_threads(CACHE) < need || fa.numRegs < KX_REG_CONV) return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) granted[dev].store(cap);
  }
  const size_t fixed = 2 * ka_entry(HD) + (CACHE == EAGLE_CACHE_F4 ? KA_RAW * ka_raw_bytes(HD) : 0) + kx_misc(CACHE);
  const int ns = std::min<int>(KA_MAX_SLOTS, static_cast<int>((cap - fixed) / ka_entry(HD)));
  if (cap < fixed || ns < 4) return cudaErrorInvalidConfiguration;   // (a shared item steps 4 entries)
  e = launch_after(with_own, dim3(ctas), kx_threads(CACHE), fixed + static_cast<size_t>(ns) * ka_entry(HD), st, kv_cross_wide<HD, CACHE>,
                   tmk, tmv, a, own, with_own, parts, ns);
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_after(true, dim3(ctas, KX_QV / KX_JOIN_V), 32 * KX_JOIN_WARPS, 0, st, kv_cross_wide_join<HD>, a, own, with_own,
                      static_cast<const float*>(parts));
}

}  // namespace

KxPlan eagle::kx_plan(int Hkv, int hd, int G, int B, int max_rows, int max_len) {
  const long long blocks = (static_cast<long long>(max_rows) * G + KX_QV - 1) / KX_QV, tiles = (static_cast<long long>(max_len) + KA_CH - 1) / KA_CH;
  const double units = static_cast<double>(B) * Hkv * blocks * tiles;
  const int sms = num_sms() > 0 ? num_sms() : 152;   // (152: without a device, a GB300's)
  KxPlan p;
  p.ctas = units / KX_MIN_UNITS < sms ? static_cast<int>(units / KX_MIN_UNITS) + 1 : sms;
  p.bytes = p.ctas == 1 ? 0 : 2ll * p.ctas * kx_slot(hd) * 4;
  return p;
}

cudaError_t eagle::kx_launch(const KaArgs& a, const KaArgs* own, bool f4, const CUtensorMap& tmk, const CUtensorMap& tmv, const KxPlan& p,
                             float* parts, cudaStream_t st) {
  KaArgs none;
  memset(&none, 0, sizeof(none));
  const KaArgs& o = own ? *own : none;
  if (a.pool.hd == 64)
    return f4 ? launch_wide<64, EAGLE_CACHE_F4>(tmk, tmv, a, o, own != nullptr, parts, p.ctas, st)
              : launch_wide<64, EAGLE_CACHE_BF16>(tmk, tmv, a, o, own != nullptr, parts, p.ctas, st);
  return f4 ? launch_wide<128, EAGLE_CACHE_F4>(tmk, tmv, a, o, own != nullptr, parts, p.ctas, st)
            : launch_wide<128, EAGLE_CACHE_BF16>(tmk, tmv, a, o, own != nullptr, parts, p.ctas, st);
}
