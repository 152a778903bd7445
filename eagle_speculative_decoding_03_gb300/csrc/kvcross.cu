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
constexpr int KX_DESCS = 4;                // segments in flight between the scheduler and the roles
constexpr int KX_MIN_UNITS = 3;            // units that are worth a CTA
constexpr uint32_t KX_MISC = 3072;         // barriers (0), segments (512), the states of an item that both groups take (1024)
// registers per thread of the 4-bit kernel's roles (the launch checks their sum)
constexpr int KX_REG_CTRL = 56, KX_REG_SOFTMAX = 144, KX_REG_CONV = 64;
constexpr int KX_JOIN_V = 32, KX_JOIN_WARPS = 8;

__host__ __device__ constexpr int kx_threads(int cache) { return 384 + (cache == EAGLE_CACHE_F4 ? 256 : 0); }
// floats of a partial result: [hd / 4][256] float4 outputs, [256] (maximum, sum)
__host__ __device__ constexpr size_t kx_slot(int hd) { return static_cast<size_t>(KX_QV) * (hd + 2); }

// Part of an item: tiles [t0, t0 + T) of query vectors [v0, v0 + qv) of sequence b.
struct Seg {
  int valid, b, kvh, row0, len, v0, qv, t0, T, slot;   // slot: partial result, -1: the item is whole
};

// How the units lie in line: per sequence b, KV heads x blocks x tiles (at least 1, to write the
// rows of a sequence without keys).
struct Line {
  Req rq;
  int blocks, tiles;
  EAGLE_DEV Line(const KaArgs& a, int b) {
    rq = request(a, b);
    blocks = (static_cast<long long>(rq.R) * a.G + KX_QV - 1) / KX_QV;
    tiles = max((rq.len + KA_CH - 1) / KA_CH, 1);
  }
  EAGLE_DEV long long units(const KaArgs& a) const { return static_cast<long long>(a.pool.Hkv) * blocks * tiles; }
};
// Units of the call, and of a CTA.  By a whole warp.
EAGLE_DEV long long all_units(const KaArgs& a, int lane) {
  long long n = 0;
  if (a.groups && lane == 0 && (__ldg(a.groups) != 0 || __ldg(a.groups + a.B) != a.requests)) atomicOr(a.err, DEVERR_PREFIX);
  for (int b = lane; b < a.B; b += 32) n += Line(a, b).units(a);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  return n;
}
EAGLE_DEV long long units_per_cta(long long all, int ctas) { return max((all + ctas - 1) / ctas, static_cast<long long>(KX_MIN_UNITS)); }
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

template <int HD, int CACHE>
__global__ void __launch_bounds__(kx_threads(CACHE), 1)
kv_cross_wide(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const KaArgs a, const KaArgs own,
              const int with_own, float* parts, const int NS) {
  constexpr bool F4 = CACHE == EAGLE_CACHE_F4;
  constexpr float LIFT = F4 ? 7.f : 0.f;     // fp16 p is held times 2^7 (as in kv_attention_tc)
  constexpr int THREADS = kx_threads(CACHE), CONV_WARP = 12, CONV = THREADS - 32 * CONV_WARP;
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
  // ring full / free, scores there, first / second half of p there, P V done, queries there, raw
  // tiles full / free, segments full / free, the two groups' states exchanged / read
  const uint32_t bar_kvf = misc_u, bar_kve = misc_u + 112, bar_sf = misc_u + 224, bar_pf = misc_u + 240, bar_pe = misc_u + 272,
                 bar_q = misc_u + 288, bar_fin = misc_u + 304, bar_rf = misc_u + 320, bar_re = misc_u + 344, bar_df = misc_u + 368,
                 bar_de = misc_u + 400, bar_x = misc_u + 432;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 448);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 452);
  volatile uint32_t* raw_pages = reinterpret_cast<volatile uint32_t*>(misc + 456);
  Seg* segs = reinterpret_cast<Seg*>(misc + 512);
  float2* states = reinterpret_cast<float2*>(misc + 1024);   // [2][128]

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
      mbar_init(bar_pf + 16 * g, 4);
      mbar_init(bar_pf + 16 * g + 8, 4);
      mbar_init(bar_pe + 8 * g, 1);
      mbar_init(bar_q + 8 * g, 4);
      mbar_init(bar_fin + 8 * g, 1);
      mbar_init(bar_x + 8 * g, 8);
    }
    for (int s = 0; F4 && s < KA_RAW; ++s) {
      mbar_init(bar_rf + 8 * s, 1);
      mbar_init(bar_re + 8 * s, F4 ? CONV / 32 : 1);
    }
    for (int s = 0; s < KX_DESCS; ++s) {
      mbar_init(bar_df + 8 * s, 1);
      mbar_init(bar_de + 8 * s, 3 + 8 + (F4 ? CONV / 32 : 0));
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
          const long long item = rest / l.tiles;
          s.valid = 1;
          s.b = b;
          s.t0 = static_cast<int>(rest - item * l.tiles);
          s.kvh = static_cast<int>(item / l.blocks);
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
      uint32_t n = 0, turn = 0;              // tiles of this group so far; segments
      for (;; dp.step(1, KX_DESCS), turn ^= 1) {
        const Seg s = segment(dp);
        if (!ok || !s.valid) break;
        const bool both = s.qv <= KA_QV;     // both groups have the same vectors, every other tile each
        const int step = both ? 2 : 1;
        ok = mbar_wait(bar_q + 8 * g, turn, a.err, abort_flag);
        tc_fence_after();
        RingPos kp = base;
        if (both && g) kp.step(2, NS);
        for (int t = both ? g : 0; t < s.T && ok; t += step, ++n) {
          RingPos vp = kp;
          vp.step(1, NS);
          ok = mbar_wait(bar_kvf + 8 * kp.slot, kp.turn, a.err, abort_flag);
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
            for (int j = 4 * h; j < 4 * h + 4; ++j) tc_mma_bf16_ta(tO, tS + 8 * j, dv + j * 128, id2, first && j == 0 ? 0u : 1u);
          }
          if (!ok) break;
          tc_commit(bar_pe + 8 * g);
          tc_commit(bar_kve + 8 * vp.slot);
          if (both) tc_commit(bar_kve + 8 * vp.slot);
          kp.step(2, NS);
          if (both) kp.step(2, NS);
        }
        if (!ok) break;
        tc_commit(bar_fin + 8 * g);
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
    const int g = (warp - 4) >> 2, lv = (tid - 128) & 127;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_base + 128 * g, to = tmem + lane_base + T_O + 128 * g;
    const int ps = 1 << a.pool.ps_log;
    // this thread's vector of a segment into the group's query tile; returns its score factor
    auto stage = [&](const Seg& s) {
      const int v = s.v0 + lv + (s.qv <= KA_QV ? 0 : KA_QV * g);
      const bool live = v - s.v0 < s.qv;
      float rs = a.scale_log2 * (F4 ? a.pool.kg : 1.f), up = 1.f;
      const int i = v / a.G;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (s.row0 + (live ? i : 0)) * a.q_ld +
                                                        static_cast<long long>(s.kvh * a.G + (live ? v - i * a.G : 0)) * HD);
      if (F4) {   // (a power of two, so that the largest magnitude lies in [2^14, 2^15))
        uint32_t top = 0;
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
          const uint4 x = __ldg(src + c);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
        int ex = static_cast<int>(top >> 7);
        ex = ex == 255 ? 127 : max(ex, 30);
        up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23);
        rs = finite_scale(rs * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23));
      }
#pragma unroll 1
      for (int c0 = 0; c0 < HD / 8; c0 += 4) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = live ? __ldg(src + c0 + c) : make_uint4(0u, 0u, 0u, 0u);
          w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
        }
        if (F4) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_f16(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) st_smem16(q_u + g * ENTRY + ((c0 + c) >> 3) * HALF + ka_sw(lv, (c0 + c) & 7), w + 4 * c);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q + 8 * g);
      return rs;
    };
    uint32_t n = 0, turn = 0, xturn = 0;     // tiles of this group so far; segments; items that both groups took
    bool waited = false;                     // for the own keys' results
    Seg s = segment(dp);
    float rs = 0.f;
    if (s.valid) rs = stage(s);
    while (__all_sync(0xffffffffu, ok && s.valid)) {
      const bool both = s.qv <= KA_QV;
      const int step = both ? 2 : 1;
      const bool idle = both && 32 * (warp & 3) >= s.qv;   // a warp without vectors
      const int end_page = s.len >> a.pool.ps_log, end_rows = F4 ? 0 : s.len & (ps - 1);
      float m_run = -INFINITY, l_run = 0.f;
      int t = both ? g : 0;
      for (; t < s.T; t += step, ++n) {
        ok = ok && mbar_wait(bar_sf + 8 * g, n & 1, a.err, abort_flag);
        tc_fence_after();
        if (!idle) {
          float x[64], y[32];
          tmem_ld32(ts, x);
          tmem_ld32(ts + 32, x + 32);
          tmem_ld32(ts + 64, y);
          const int kt = (s.t0 + t) * KA_CH;
          // the columns that hold keys; the page that the keys end inside has them at its end
          const bool whole = kt + KA_CH <= s.len;
          Bits vis{~0ull, ~0ull};
          if (!whole) {
            const int at = (end_page << a.pool.ps_log) - kt;
            vis = bits_below(end_rows ? at + ps : s.len - kt);
            if (end_rows) {
              const Bits lo = bits_below(at), hi = bits_below(at + ps - end_rows);
              vis.lo &= lo.lo | ~hi.lo;
              vis.hi &= lo.hi | ~hi.hi;
            }
          }
          auto hide = [&](float* f, unsigned bits) {
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = (bits >> e) & 1u ? f[e] : -INFINITY;
          };
          auto top32 = [&](const float* f, float m) {
            float m4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = max_nan(f[k], f[k + 4]);
#pragma unroll
            for (int e = 8; e < 32; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) m4[k] = max3_nan(m4[k], f[e + k], f[e + 4 + k]);
            return max_nan(max3_nan(m4[0], m4[1], m4[2]), max_nan(m4[3], m));
          };
          tmem_wait_ld();
          if (!whole) {
            hide(x, static_cast<unsigned>(vis.lo));
            hide(x + 32, static_cast<unsigned>(vis.lo >> 32));
            hide(y, static_cast<unsigned>(vis.hi));
          }
          float mt = top32(y, -INFINITY);
          tmem_ld32(ts + 96, y);
          mt = top32(x + 32, top32(x, mt));
          tmem_wait_ld();
          if (!whole) hide(y, static_cast<unsigned>(vis.hi >> 32));
          mt = top32(y, mt);
          float f = 1.f;
          bool resc = false;
          if (mt != -INFINITY) {
            if (m_run == -INFINITY) {
              m_run = mt;
            } else if ((mt - m_run) * rs > KA_RESCALE) {
              f = fast_exp2((m_run - mt) * rs);
              m_run = mt;
              resc = true;
            }
          }
          if (__any_sync(0xffffffffu, resc)) {   // (the scores are there, so the P V before them is done)
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
              float z[32];
              tmem_ld32(to + c0, z);
              tmem_wait_ld();
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(z[e] * f);
              tmem_st32(to + c0, w);
            }
          }
          l_run *= f;
          const float mb = (m_run == -INFINITY ? 0.f : m_run * rs) - LIFT;
          float p8[8] = {};
          // 32 scores -> p -> 16 packed columns
          auto turn32 = [&](float* z, uint32_t dst) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              fma2(z[e], z[e + 1], rs, -mb);
              z[e] = fast_exp2(z[e]);
              z[e + 1] = fast_exp2(z[e + 1]);
              add2(p8[e & 7], p8[(e & 7) + 1], z[e], z[e + 1]);
            }
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = __uint_as_float(F4 ? pack_f16(z[2 * e], z[2 * e + 1]) : pack_bf16(z[2 * e], z[2 * e + 1]));
            tmem_st16(dst, pk);
          };
          turn32(x, ts);
          turn32(x + 32, ts + 16);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_pf + 16 * g);
          tmem_ld32(ts + 64, x);
          turn32(y, ts + 48);
          tmem_wait_ld();
          if (!whole) hide(x, static_cast<unsigned>(vis.hi));
          turn32(x, ts + 32);
          tmem_wait_st();
          l_run += ((p8[0] + p8[1]) + (p8[2] + p8[3])) + ((p8[4] + p8[5]) + (p8[6] + p8[7]));
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_pf + 16 * g + 8);
        } else if (lane == 0) {
          mbar_arrive(bar_pf + 16 * g);
          mbar_arrive(bar_pf + 16 * g + 8);
        }
      }
      // ---- the next segment's queries, as soon as this one's are read (its last scores are there; a
      // group without a tile waits for its MMA thread, which would otherwise miss the barrier's turn)
      const bool early = s.T > (both ? g : 0);
      RingPos np = dp;
      np.step(1, KX_DESCS);
      float rs2 = 0.f;
      if (!early) ok = mbar_wait_sleepy(bar_fin + 8 * g, turn, a.err, abort_flag) && ok;
      const bool so_far = ok;
      const Seg s2 = segment(np);
      ok = __all_sync(0xffffffffu, ok && so_far);
      if (ok && s2.valid) rs2 = stage(s2);
      if (early) ok = mbar_wait(bar_fin + 8 * g, turn, a.err, abort_flag) && ok;
      turn ^= 1;
      tc_fence_after();
      // ---- this segment's result: of state g alone, or of both groups' (then half of the dims each)
      const int v = s.v0 + lv + (both ? 0 : KA_QV * g), i = v / a.G, h = s.kvh * a.G + (v - i * a.G);
      const bool live = v - s.v0 < s.qv;
      float2 st[2] = {make_float2(l_run == 0.f ? -INFINITY : m_run * rs - LIFT, l_run), make_float2(-INFINITY, 0.f)};
      if (both) {
        states[128 * g + lv] = st[0];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_x);
        ok = mbar_wait(bar_x, xturn, a.err, abort_flag) && ok;
        tc_fence_after();
        st[0] = states[lv];
        st[1] = states[128 + lv];
      }
      const uint32_t o0 = tmem + lane_base + T_O + (both ? 0 : 128 * g), o1 = tmem + lane_base + T_O + 128;
      const int c_lo = both ? g * (HD / 2) : 0, c_hi = both ? c_lo + HD / 2 : HD;
      float M = max_nan(st[0].x, st[1].x);
      const bool join = with_own && s.slot < 0;
      if (join && !waited) {
        pdl_wait();
        waited = true;
      }
      const size_t row = static_cast<size_t>(s.row0 + i);
      Own mine(own, live && join ? static_cast<int>(row) : -1, h);
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
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
        float x[32];
        __syncwarp();
        tmem_ld32(o0 + c0, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = f0 == 0.f ? 0.f : f0 * x[e];
        if (both) {
          float y[32];
          tmem_ld32(o1 + c0, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = f1 == 0.f ? x[e] : fmaf(f1, y[e], x[e]);
        }
        if (!writes) continue;
        if (s.slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(part) + static_cast<size_t>(c0 / 4) * KX_QV + pv;
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e * KX_QV] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          continue;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] *= inv;
        for (int k = 0; k < mine.used; ++k) {
          const float f = part_factor(mine.ml(k).x, M) * own_inv;
          const float4* src = reinterpret_cast<const float4*>(own.part_o + mine.place(k) * HD + c0);
#pragma unroll
          for (int e = 0; e < 8; ++e) add_part(x + 4 * e, f, src[e]);
        }
        uint4* dst = reinterpret_cast<uint4*>(a.out + row * a.out_ld + static_cast<long long>(h) * HD + c0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = none ? 0u : pack_bf16(x[8 * e + 2 * k], x[8 * e + 2 * k + 1]);
          dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (writes && (!both || g == 0)) {
        if (s.slot >= 0) reinterpret_cast<float2*>(part + static_cast<size_t>(KX_QV) * HD)[pv] = make_float2(none ? -INFINITY : M, L);
        else if (a.lse) a.lse[row * a.Hq + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
      if (both) {                            // (both have read O and the states before either goes on)
        __syncwarp();
        tc_fence_before();
        if (lane == 0) mbar_arrive(bar_x + 8);
        ok = mbar_wait(bar_x + 8, xturn, a.err, abort_flag) && ok;
        xturn ^= 1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_de + 8 * dp.slot);
      dp = np;
      s = s2;
      rs = rs2;
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
      const long long item = rest / l.tiles, first = end - 1 - (rest - item * l.tiles), behind = first + l.tiles;
      if (behind > end && first >= begin) {
        s.valid = 1;
        s.kvh = static_cast<int>(item / l.blocks);
        s.row0 = l.rq.row0;
        s.v0 = static_cast<int>(item - static_cast<long long>(s.kvh) * l.blocks) * KX_QV;
        s.qv = static_cast<int>(min(static_cast<long long>(l.rq.R) * a.G - s.v0, static_cast<long long>(KX_QV)));
        s.slot = 2 * c + (first == begin ? 0 : 1);
        last = static_cast<int>((behind - 1) / per);
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
      const int need = 128 * KX_REG_CTRL + 256 * KX_REG_SOFTMAX + 256 * KX_REG_CONV;
      if (fa.numRegs / 8 * 8 * kx_threads(CACHE) < need || fa.numRegs < KX_REG_CONV) return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) granted[dev].store(cap);
  }
  const size_t fixed = 2 * ka_entry(HD) + (CACHE == EAGLE_CACHE_F4 ? KA_RAW * ka_raw_bytes(HD) : 0) + KX_MISC;
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
