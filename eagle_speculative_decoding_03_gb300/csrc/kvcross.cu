// The products of cross attention: many query vectors over all cached keys of a sequence (bf16 or
// 4-bit pages), the keys' tiles dealt out evenly to the SMs.  See kvattn.cu for the notation and
// kvline.cuh for how the work is dealt out.
//
//   S = Q K^T, p = 2^(rs S - m), O += P V, l += sum p      over tiles of 128 keys (4 bits: 64)
//
// An item is a block of up to 256 query vectors (row * G + head) of one sequence and KV head, one CTA
// per SM.  Two TMEM tiles of 128 vectors, each with a softmax warpgroup (a thread per vector) and an
// MMA thread of its own, so that the tensor cores work for one while the other's scores are in the
// softmax.  Units of 64 keys, two score buffers a tile; P replaces S in place, O takes hd columns.
// An item of at most 128 vectors is taken by both groups, every other tile each, and the two states
// are joined in TMEM: one group alone would leave the tensor cores idle during its softmax.  The next
// item's queries are staged while the last unit of this one runs, and results are written while the
// copies and products of the next are under way.
//
// Bound by the tensor cores: a unit's Q K^T takes 48 cycles an instruction for 32 of work, because
// both operands come from shared memory; with P V that is 2560 cycles for 128 keys and 256 vectors,
// and 3050 are measured (2 prompts of 2,047 rows and 32 heads of 128 over 4,099 keys: 219 us with the
// join, 1,255 TFLOP/s, 67% of the measured rate).  128 keys an instruction would run at the full rate, but
// its scores leave room for one buffer a tile: 250 us.  4 bits: four warps convert what they copied, 64 keys an entry (a
// chunk of 1,688 rows of 32 heads over 16,001 keys 420 us, 1,070 TFLOP/s).
//
// bf16 p (8 bits) against bf16 values, fp16 p (11 bits) against 4-bit ones: the second product takes
// one type on both sides, and p in two parts takes kv_attention_tc 75 us of a tree where one takes 60;
// l sums the unrounded p.  Every row sees every key and rows behind the last key are loaded as zeros, so
// nothing that is not finite reaches a row that does not see it.  An infinite value times a p that fell to 0
// is NaN where the formula has infinity: sums that are NaN are looked up among the values (`infinities`;
// cross_prompt's sizes with one infinite dim 517 us where 204 without, with all of them 1,490).
#include "kvline.cuh"

#include <algorithm>
#include <atomic>

using namespace eagle;

namespace {

constexpr int KX_QV = 256;                 // query vectors of a block
constexpr int KX_DESCS = 4;                // segments in flight between the scheduler and the roles
constexpr int KX_MIN_KEYS = 384;           // keys of an item that are worth a CTA
constexpr int KX_MAX_RAW = 12;             // raw tiles of a 4-bit pool in flight
constexpr uint32_t KX_MISC = 3 << 10;         // barriers (0, 896), segments (736), states of an item that both groups take (1024)
constexpr uint32_t KX_FULL2 = 896;         // from a place's barrier for even turns of the ring to that for odd ones
constexpr int KX_SOFTMAX = 256;            // softmax threads: one per query vector
constexpr int KX_COPIERS = 4;              // loader warps
constexpr int KX_THREADS = 128 + KX_SOFTMAX + 32 * KX_COPIERS;   // control, softmax, loaders
// registers per thread: at the launch, and of the roles (the launch checks their sum).  What is left of an
// SM's holds a CTA of kv_few_join, which waits there when own keys go ahead of this kernel: at 128 a thread
// this one could only start where that had ended.
constexpr int KX_REGS = 112, KX_REG_CTRL = 48, KX_REG_SOFTMAX = 160, KX_REG_LOAD = 72;
constexpr int KX_JOIN_V = 32, KX_JOIN_WARPS = 8;

// floats of a partial result: [hd / 4][256] float4 outputs, [256] (maximum, sum)
__host__ __device__ constexpr size_t kx_slot(int hd) { return static_cast<size_t>(KX_QV) * (hd + 2); }

// Keys of a tile, a ring entry: two units of bf16 keys; one of 4-bit ones, whose converted tiles must be
// in order and four of which at a time left the groups of a shared item waiting for each other's values.
__host__ __device__ constexpr int kx_keys(int cache) { return cache == EAGLE_CACHE_F4 ? KA_H : KA_CH; }
__host__ __device__ constexpr uint32_t kx_entry(int hd, int cache) { return static_cast<uint32_t>(hd) * 2 * kx_keys(cache); }
__host__ __device__ constexpr uint32_t kx_raw_bytes(int hd) { return static_cast<uint32_t>(hd) / 2 * KA_H + hd / 16 * KA_H; }
template <int CACHE>
using KxLine = Line<8, kx_keys(CACHE)>;    // (blocks of KX_QV vectors)

EAGLE_DEV uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// A place in the ring of keys and values, and how often the ring has turned (mod 4).  Its places have two
// barriers each, for the odd and the even turns: a group that skips the other's tiles may come to a place
// while what is ahead of its entry is still being copied, and one barrier's parity would then read as done.
struct RingAt {
  int slot, turn;
  EAGLE_DEV void step(int n, int NS) {
    slot += n;
    if (slot >= NS) {
      slot -= NS;
      turn = (turn + 1) & 3;
    }
  }
  EAGLE_DEV uint32_t full(uint32_t bar) const { return bar + 8 * slot + (turn & 1) * KX_FULL2; }
  EAGLE_DEV uint32_t parity() const { return static_cast<uint32_t>(turn) >> 1; }
};

// Part of an item: tiles [t0, t0 + T) of query vectors [v0, v0 + qv) of sequence b.
struct Seg {
  int valid, b, kvh, row0, len, v0, qv, t0, T, slot;   // slot: partial result, -1: the item is whole
  // both groups have the same vectors, every other tile each
  EAGLE_DEV bool both() const { return qv <= KA_QV; }
  // units of 64 keys that group g has of it, UPT to a tile and `last` in the last one
  template <int UPT>
  EAGLE_DEV int units_of(int g, int last) const {
    if (T == 0) return 0;
    if (!both()) return UPT * (T - 1) + last;
    const int n = (T + 1 - g) >> 1;          // its tiles
    return n == 0 ? 0 : UPT * n - (((T - 1) & 1) == g ? UPT - last : 0);
  }
  EAGLE_DEV bool tiles_of(int g) const { return T > (both() ? g : 0); }
};

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
    used = ranges_of(o, rq.len);
  }
  EAGLE_DEV size_t place(int s) const { return s * (static_cast<size_t>(a.N) * a.Hq) + at; }
  EAGLE_DEV float2 ml(int s) const { return a.part_ml[place(s)]; }
};
EAGLE_DEV void add_part(float* x, float f, float4 y) {
  x[0] = add_weighted(x[0], f, y.x);
  x[1] = add_weighted(x[1], f, y.y);
  x[2] = add_weighted(x[2], f, y.z);
  x[3] = add_weighted(x[3], f, y.w);
}

// 64 scores x -> p = 2^(x rs - mb), packed two to a word (fp16 or bf16), their sum into p8, and the
// largest score.  The pipes need 4 cycles a warp for each ex2 and 2 for each maximum, product, sum and
// conversion of a pair: in the order written (volatile), the products two pairs ahead of ex2, sums and
// conversions four behind, they overlap.
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
template <bool F16>
EAGLE_DEV float powers64(float* x, float rs, float mb, float* p8, float* pk) {
  constexpr int AHEAD = 2, BEHIND = 4;
  float m[4] = {x[0], x[2], x[4], x[6]};
#pragma unroll
  for (int i = -AHEAD; i < 32 + BEHIND; ++i) {
    const int u = i + AHEAD, w = i - BEHIND;
    if (i >= 0 && i < 32) ordered_exp2(x[2 * i]);
    if (u < 32) {
      ordered_max3(m[u & 3], x[2 * u], x[2 * u + 1]);
      ordered_fma2(x[2 * u], x[2 * u + 1], rs, -mb);
    }
    if (i >= 0 && i < 32) ordered_exp2(x[2 * i + 1]);
    if (w >= 0) {
      ordered_add2(p8[(2 * w) & 7], p8[((2 * w) & 7) + 1], x[2 * w], x[2 * w + 1]);
      pk[w] = ordered_pack<F16>(x[2 * w], x[2 * w + 1]);
    }
  }
  return max_nan(max3_nan(m[0], m[1], m[2]), m[3]);
}

template <int HD, int CACHE, bool OWN>
__global__ void __maxnreg__(KX_REGS)
kv_cross_wide(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const KaArgs a, const KaArgs own,
              float* parts, const int NS, const int NR) {
  constexpr bool F4 = CACHE == EAGLE_CACHE_F4;
  constexpr float LIFT = F4 ? 7.f : 0.f;     // fp16 p is held times 2^7 (as in kv_attention_tc)
  constexpr int LOAD_WARP = 4 + KX_SOFTMAX / 32;
  constexpr int KEYS = kx_keys(CACHE), UPT = KEYS / KA_H;
  constexpr uint32_t ENTRY = kx_entry(HD, CACHE), HALF = KEYS * 128, RAW = kx_raw_bytes(HD), RAW_SCALES = HD / 2 * KEYS;
  constexpr uint32_t Q_TILE = ka_entry(HD), Q_HALF = KA_QV * 128;
  constexpr uint32_t T_O = 256;
  static_assert(736 + KX_DESCS * sizeof(Seg) <= KX_FULL2 && KX_FULL2 + 8 * KA_MAX_SLOTS <= 1024, "");
  extern __shared__ __align__(1024) uint8_t kx_sm[];   // (no byte is left to align it by hand: ring, queries, misc take all)
  uint8_t* sm = kx_sm;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t ring_u = uniform(smem_u32(sm));
  const uint32_t q_u = ring_u + static_cast<uint32_t>(NS) * ENTRY;
  uint8_t* raw = sm + static_cast<uint32_t>(NS) * ENTRY + 2 * Q_TILE;
  uint8_t* misc = raw + (F4 ? NR * RAW : 0);
  const uint32_t misc_u = smem_u32(misc);
  // ring full (even turns; odd ones at KX_FULL2) / free; per score buffer (group, 64 columns): scores there, p there, P V done; per group:
  // queries there, segment done; raw tiles full / free, segments full / free; an item of both groups:
  // states there / read; a loader's turn
  const uint32_t bar_kvf = misc_u, bar_kve = misc_u + 112, bar_sf = misc_u + 224, bar_pf = misc_u + 256, bar_pe = misc_u + 288,
                 bar_q = misc_u + 320, bar_fin = misc_u + 336, bar_df = misc_u + 352, bar_de = misc_u + 384, bar_x = misc_u + 416,
                 bar_rf = misc_u + 432, bar_re = misc_u + 528, bar_next = misc_u + 680;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 624);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 628);
  volatile uint32_t* raw_pages = reinterpret_cast<volatile uint32_t*>(misc + 632);
  const uint32_t placed_u = misc_u + 716;    // ring entries whose place the loaders have taken
  Seg* segs = reinterpret_cast<Seg*>(misc + 736);

  pdl_trigger();
  if (misplaced(ring_u, parts, a.err)) {
    if (OWN) pdl_wait();                     // (this kernel ends after the one before it)
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < KA_MAX_SLOTS; ++s) {
      mbar_init(bar_kvf + 8 * s, 1);
      mbar_init(bar_kvf + 8 * s + KX_FULL2, 1);
      mbar_init(bar_kve + 8 * s, 2);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(bar_sf + 8 * b, 1);
      mbar_init(bar_pf + 8 * b, 4);
      mbar_init(bar_pe + 8 * b, 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar_q + 8 * g, 4);
      mbar_init(bar_fin + 8 * g, 1);
      mbar_init(bar_x + 8 * g, KX_SOFTMAX / 32);
    }
    for (int s = 0; F4 && s < KX_MAX_RAW; ++s) {
      mbar_init(bar_rf + 8 * s, 1);
      mbar_init(bar_re + 8 * s, 1);
    }
    for (int t = 0; t < KX_COPIERS; ++t) mbar_init(bar_next + 8 * t, 1);
    for (int s = 0; s < KX_DESCS; ++s) {
      mbar_init(bar_df + 8 * s, 1);
      mbar_init(bar_de + 8 * s, 2 + KX_SOFTMAX / 32 + KX_COPIERS);
    }
    *abort_flag = 0;
    st_release_smem(placed_u, 0);
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
    ok = kx_wait<true>(bar_df + 8 * p.slot, p.turn, a.err, abort_flag);
    Seg s = segs[p.slot];
    if (!ok) s.valid = 0;
    return s;
  };

  // how many of a segment's last tile's two units hold columns of keys (the page that the keys end inside
  // has its rows at its end)
  auto last_units = [&](const Seg& s) {
    if (UPT == 1) return 1;
    const int ps = 1 << a.pool.ps_log, kt = (s.t0 + s.T - 1) * KEYS;
    const int columns = !(s.len & (ps - 1)) ? s.len : ((s.len >> a.pool.ps_log) + 1) << a.pool.ps_log;
    return columns - kt > KA_H ? 2 : 1;
  };

  if (warp < 4) {
    set_regs_down<KX_REG_CTRL>();
    if (warp == 1) {
      // ------------------------------------------------------------ scheduler
      const long long all = all_units<KxLine<CACHE>>(a, lane), per = units_per_cta(all, gridDim.x, KX_MIN_KEYS / KEYS);
      const long long begin = min(per * blockIdx.x, all), end = min(begin + per, all);
      long long u = begin, rest = 0;
      int b = u < end ? find_unit<KxLine<CACHE>>(a, lane, u, &rest) : 0;
      Cut cut;
      cut.last = 0;
      int n = 0;
#pragma unroll 1
      while (ok) {
        Seg s;
        s.valid = 0;
        if (u < end) {
          KxLine<CACHE> l(a, b);
#pragma unroll 1
          while (rest >= l.units(a)) {       // (the next sequence that has units)
            rest -= l.units(a);
            ++b;
            l = KxLine<CACHE>(a, b);
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
          // the queries on their way while the segments before are in work
#pragma unroll 1
          for (int x = lane; x < s.qv * (HD / 64); x += 32) {
            const int v = s.v0 + x / (HD / 64), i = row_of(a, v);
            const __nv_bfloat16* q = a.q + (s.row0 + i) * a.q_ld + static_cast<long long>(s.kvh * a.G + v - i * a.G) * HD + x % (HD / 64) * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          }
          if (s.t0 == 0 && units < l.tiles) cut = Cut{static_cast<int>(quotient(u + l.tiles - 1, per)), s.kvh, s.row0, s.v0, s.qv, s.slot};
          u += units;
          rest += units;
        }
        if (n >= KX_DESCS) ok = kx_wait<true>(bar_de + 8 * dp.slot, dp.turn ^ 1, a.err, abort_flag);
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
      if (lane == 0) reinterpret_cast<Cut*>(parts)[blockIdx.x] = cut;
      if (OWN) pdl_wait();                   // (this kernel ends after the one before it)
    } else if (warp >= 2 && elect_one()) {
      // ------------------------------------------------------------ MMA issuer of group g
      // One thread walks the group's units and issues; nothing in the loop divides or votes.
      const int g = warp - 2;
      const uint32_t id1 = F4 ? idesc_f16_f32(128, KA_H) : idesc_bf16_f32(128, KA_H);
      const uint32_t id2 = (F4 ? idesc_f16_f32(128, HD) : idesc_bf16_f32(128, HD)) | (1u << 16);   // B (values) MN-major
      const uint64_t dq = smem_desc_sw128(q_u + g * Q_TILE);
      const uint32_t tO = tmem + T_O + 128 * g;
      RingAt base{0, 0};                     // the segment's first entry
      uint32_t n = 0, turn = 0;              // units of this group so far; segments with a tile
      uint32_t first = 0;                    // the segment's first entry, counted from the start
      for (;; dp.step(1, KX_DESCS)) {
        const Seg s = segment(dp);
        if (!ok || !s.valid) break;
        const bool both = s.both(), work = s.tiles_of(g);
        if (work) {
          ok = kx_wait(bar_q + 8 * g, turn, a.err, abort_flag);
          turn ^= 1;
        }
        tc_fence_after();
        const int W = s.units_of<UPT>(g, last_units(s));
        RingAt kp = base;
        if (both && g) kp.step(2, NS);
        // The group's first entry is under way, so what was ahead of it in its place is through (in a run of
        // short items this group may have skipped any number).  From there on it waits for one of any NS
        // entries, which leaves its place's barriers two turns apart.
        if (work) ok = ok && kx_wait_past(placed_u, first + (both ? 2 * g : 0), a.err, abort_flag);
        RingAt vp = kp;
        vp.step(1, NS);
#pragma unroll 1
        for (int w = 0; w <= W && ok; ++w) {
          if (w < W) {
            // S = Q K^T of unit w, once P V of the unit before the last (same buffer) is done
            const uint32_t u = n + w, buf = 2 * g + (u & 1);
            if (UPT == 1 || !(w & 1)) ok = kx_wait(kp.full(bar_kvf), kp.parity(), a.err, abort_flag);
            ok = ok && kx_wait(bar_pe + 8 * buf, ((u >> 1) & 1) ^ 1, a.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + buf * KA_H;
            const uint64_t dk = smem_desc_sw128(ring_u + kp.slot * ENTRY + (UPT == 2 ? (w & 1) * (KA_H * 128) : 0));
#pragma unroll
            for (int j = 0; j < HD / 16; ++j) {
              const uint32_t qo = ((j >> 2) * Q_HALF + (j & 3) * 32) >> 4, ko = ((j >> 2) * HALF + (j & 3) * 32) >> 4;
              tc_mma_bf16(d, dq + qo, dk + ko, id1, j > 0 ? 1u : 0u);
            }
            tc_commit(bar_sf + 8 * buf);
            if (UPT == 1 || (w & 1) || w == W - 1) {
              tc_commit(bar_kve + 8 * kp.slot);
              if (both) tc_commit(bar_kve + 8 * kp.slot);
              kp.step(2, NS);
              if (both) kp.step(2, NS);
            }
          }
          if (w > 0) {   // O += P V of unit x
            const int x = w - 1;
            const uint32_t u = n + x, buf = 2 * g + (u & 1);
            if (UPT == 1 || !(x & 1)) ok = kx_wait(vp.full(bar_kvf), vp.parity(), a.err, abort_flag);
            ok = ok && kx_wait(bar_pf + 8 * buf, (u >> 1) & 1, a.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dv = smem_desc_sw128_mn(ring_u + vp.slot * ENTRY + (UPT == 2 ? (x & 1) * (KA_H * 128) : 0), HALF, 1024);
            const uint32_t tp = tmem + buf * KA_H;
#pragma unroll
            for (int j = 0; j < KA_H / 16; ++j) tc_mma_bf16_ta(tO, tp + 8 * j, dv + j * 128, id2, x > 0 || j > 0 ? 1u : 0u);
            tc_commit(bar_pe + 8 * buf);
            if (UPT == 1 || (x & 1) || x == W - 1) {
              tc_commit(bar_kve + 8 * vp.slot);
              if (both) tc_commit(bar_kve + 8 * vp.slot);
              vp.step(2, NS);
              if (both) vp.step(2, NS);
            }
          }
        }
        if (!ok) break;
        n += W;
        if (work) tc_commit(bar_fin + 8 * g);
        const uint32_t at = base.slot + 2u * s.T;
        base.turn = (base.turn + at / NS) & 3;
        base.slot = at % NS;
        first += 2u * s.T;
        mbar_arrive(bar_de + 8 * dp.slot);
      }
      if (!ok) {   // let MMAs already issued finish before TMEM is released
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
      }
    }
  } else if (warp >= LOAD_WARP) {
    // ------------------------------------------------------------ loaders
    // Four warps take the entries, keys and values of the tiles, in turn: one thread issues a copy in 200
    // cycles, and 128 keys take 8 to 32 of them.  4 bits: they convert what they copied; an entry's chain of
    // waits, loads, stores and the proxy fence takes 1000 cycles however many warps share it.
    set_regs_down<KX_REG_LOAD>();
    const int team = warp - LOAD_WARP;
    const int ps = 1 << a.pool.ps_log, box = min(ps, KEYS), per = KEYS / box, NT = F4 ? NR / KX_COPIERS : 1;   // raw tiles of a warp
    RingAt rp{0, 0};                                   // the warp's entry in the ring
    RingPos cp{0, 0}, wp{0, 0};                        // its raw tile to copy into, to convert
    rp.step(team, NS);
    uint32_t entries = 0, taken = 0;                   // of the segments before; by this warp
    for (;; dp.step(1, KX_DESCS)) {
      const Seg s = segment(dp);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || !s.valid) break;
      const int end_page = s.len >> a.pool.ps_log, end_rows = F4 ? 0 : s.len & (ps - 1);
      const int first = (team - static_cast<int>(entries)) & (KX_COPIERS - 1), E = 2 * s.T;
      entries += E;
      // box `lane` of the tile of entry e, one entry ahead
      auto lookup = [&](int e) {
        const int k = (s.t0 + (e >> 1)) * KEYS + lane * box;
        return e < E && lane < per && k < s.len ? kv_page(a.pool, s.b, k, a.err) : -1;
      };
      int page = lookup(first);
      // All that a copy takes is the same for the whole warp.
      auto copy = [&](int e, uint32_t bar, int slot) {
        const int now = page, tile = s.t0 + (e >> 1), v = e & 1;
        page = lookup(e + KX_COPIERS);
        if constexpr (F4) {
          const uint32_t have = __ballot_sync(0xffffffffu, now >= 0);
          const uint32_t codes = static_cast<uint32_t>(box) * (HD / 2), scales = static_cast<uint32_t>(box) * (HD / 16);
          if (elect_one()) {
            raw_pages[slot] = have;
            mbar_arrive_expect_tx(bar, __popc(have) * (codes + scales));
          }
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < per; ++i) {
            const int pg = __shfl_sync(0xffffffffu, now, i);
            const size_t row = kv_row(a.pool, pg, s.kvh, tile * KEYS + i * box);
            const uint32_t dst = smem_u32(raw) + slot * RAW;
            if (pg >= 0 && elect_one()) {
              bulk_load(dst + i * codes, static_cast<const uint8_t*>(v ? a.pool.v : a.pool.k) + row * (HD / 2), codes, bar);
              bulk_load(dst + RAW_SCALES + i * scales, static_cast<const uint8_t*>(v ? a.pool.vs : a.pool.ks) + row * (HD / 16), scales, bar);
            }
          }
        } else {
          const uint64_t pol = policy_evict_normal();  // (the other blocks of the sequence read the keys too)
          if (elect_one()) mbar_arrive_expect_tx(bar, ENTRY);
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < per; ++i) {              // (a page that is not there reads as zeros: a block outside the map)
            const int pg = __shfl_sync(0xffffffffu, now, i), pi = tile * per + i;
            const int blk = pg >= 0 ? pg * a.pool.Hkv + s.kvh : a.pool.num_pages * a.pool.Hkv;
            const int row = pi == end_page && end_rows ? end_rows - ps : 0;
            const uint32_t dst = ring_u + slot * ENTRY + i * (ps * 128);
            if (elect_one()) {
#pragma unroll
              for (int h = 0; h < HD / 64; ++h) tma_load_3d(dst + h * HALF, v ? &tmv : &tmk, 64 * h, row, blk, bar, pol);
            }
          }
        }
      };
      // Waits until the entry's place in the ring is free.  The loaders take their places in the entries'
      // order: one that was a whole turn of the ring ahead would take a barrier's turn before the last for
      // the last (the groups of a shared item free theirs in no order).
      auto place = [&]() {
        const uint32_t n = taken * KX_COPIERS + team;
        if (n) ok = kx_wait(bar_next + 8 * team, (team ? taken : taken - 1) & 1, a.err, abort_flag) && ok;
        if (n >= static_cast<uint32_t>(NS)) ok = ok && kx_wait(bar_kve + 8 * rp.slot, (rp.turn & 1) ^ 1, a.err, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
          if (ok) st_release_smem(placed_u, n + 1);
          mbar_arrive(bar_next + 8 * ((team + 1) % KX_COPIERS));
        }
      };
      if constexpr (!F4) {
#pragma unroll 1
        for (int e = first; e < E; e += KX_COPIERS, ++taken, rp.step(KX_COPIERS, NS)) {
          const int slot = uniform(rp.slot);
          place();
          if (!ok) break;
          copy(e, uniform(rp.full(bar_kvf)), slot);
        }
      } else {
        // raw tiles are copied NT entries ahead of their conversion: 16 dims per thread and step, 8 steps at once
        constexpr int GR = HD / 16, IT = KEYS * GR / 32, RSTEP = 32 / GR;
        static_assert(IT % 8 == 0 && (RSTEP == 8 || RSTEP == 4), "");
        const int gidx = lane % GR, r0 = lane / GR, sw = gidx >> 2, c = 2 * (gidx & 3), box_log = min(a.pool.ps_log, 6);
        int ahead = first;
        uint32_t copied = taken;
        auto fill = [&]() {
          const int slot = uniform(team * NT + cp.slot);
          if (copied >= static_cast<uint32_t>(NT)) ok = kx_wait(bar_re + 8 * slot, cp.turn ^ 1, a.err, abort_flag) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (ok) copy(ahead, bar_rf + 8 * slot, slot);
          ahead += KX_COPIERS;
          ++copied;
          cp.step(1, NT);
        };
        for (int i = 1; i < NT && ahead < E; ++i) fill();
#pragma unroll 1
        for (int e = first; e < E; e += KX_COPIERS, ++taken, rp.step(KX_COPIERS, NS), wp.step(1, NT)) {
          if (ahead < E) fill();
          const int rslot = team * NT + wp.slot;
          ok = kx_wait(bar_rf + 8 * rslot, wp.turn, a.err, abort_flag) && ok;
          const uint8_t* src = raw + rslot * RAW;
          const uint32_t have = raw_pages[rslot];
          const int k0 = (s.t0 + (e >> 1)) * KEYS;
          const bool whole = k0 + KEYS <= s.len && have == (1u << per) - 1u;
          place();
          if (!ok) break;
          const uint32_t dst = ring_u + rp.slot * ENTRY + sw * HALF;
#pragma unroll 1
          for (int i0 = 0; i0 < IT; i0 += 8) {
            uint2 code[8];
            uint32_t scale[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = r0 + (i0 + i) * RSTEP;
              code[i] = reinterpret_cast<const uint2*>(src + r * (HD / 2))[gidx];
              scale[i] = src[RAW_SCALES + r * GR + gidx];
            }
            if (!whole) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {    // rows behind the last key, and of pages that are not there: zeros
                const int r = r0 + (i0 + i) * RSTEP;
                if (k0 + r >= s.len || !((have >> (r >> box_log)) & 1u)) {
                  code[i] = make_uint2(0u, 0u);
                  scale[i] = 0u;
                }
              }
            }
            // (the two 64-dim halves share banks: the upper one stores its chunks in the other order)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = r0 + (i0 + i) * RSTEP;
              const uint32_t f = scale_pair(scale[i]);
              uint32_t h[4];
              dequant8(sw ? code[i].y : code[i].x, f, h);
              st_smem16(dst + ka_sw(r, c + sw), h);
              dequant8(sw ? code[i].x : code[i].y, f, h);
              st_smem16(dst + ka_sw(r, c + (sw ^ 1)), h);
            }
          }
          fence_proxy_async_smem();            // (raw tile and entry change hands between the proxies)
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_re + 8 * rslot);
            mbar_arrive(rp.full(bar_kvf));
          }
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_de + 8 * dp.slot);
    }
    if (!ok) {   // let copies already issued land before the CTA releases its shared memory
      const long long t0 = clock64();
      while (clock64() - t0 < 4000000) {
      }
    }
  } else {
    set_regs_up<KX_REG_SOFTMAX>();
    // ------------------------------------------------------------ softmax of group g
    const int g = (warp - 4) >> 2, quad = warp & 3, lv = 32 * quad + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t to = tmem + lane_base + T_O + 128 * g;
    const int ps = 1 << a.pool.ps_log;
    float2* states = reinterpret_cast<float2*>(misc + 1024);   // [group][128]
    // The warp's 32 vectors of a segment into the group's query tile, LR lanes a row (a lane a row would
    // touch 32 rows with every load: 4096 cycles a segment); returns the score factor of this thread's.
    auto stage = [&](const Seg& s) {
      constexpr int LR = HD / 8, ROWS = 32 / LR, N = 32 / ROWS;   // lanes a row, rows a load, loads
      const int v = s.v0 + lv + (s.both() ? 0 : KA_QV * g), c = lane % LR, i = row_of(a, v);
      const bool live = v - s.v0 < s.qv;
      const long long at = live ? (s.row0 + i) * a.q_ld + static_cast<long long>(s.kvh * a.G + v - i * a.G) * HD : -1;
      uint4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const long long from = __shfl_sync(0xffffffffu, at, ROWS * k + lane / LR);
        x[k] = from >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + from) + c) : make_uint4(0u, 0u, 0u, 0u);
      }
      int mine = 127;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
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
          const int theirs = __shfl_sync(0xffffffffu, ex, (lane % ROWS) * LR);
          if (lane / ROWS == k) mine = theirs;
        }
        const int r = 32 * quad + ROWS * k + lane / LR;
        st_smem16(q_u + g * Q_TILE + (c >> 3) * Q_HALF + ka_sw(r, c & 7), w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q + 8 * g);
      return F4 ? finite_scale(a.scale_log2 * a.pool.kg * __uint_as_float(static_cast<uint32_t>(mine - 14) << 23)) : a.scale_log2;
    };
    uint32_t n = 0, turn = 0, xturn = 0;     // units of this group so far; segments with a tile; items that both groups took
    bool waited = false;                     // for the own keys' results
    Seg s;
    s.valid = 0;
    bool both = false, work = false, idle = false;
    float m_run = -INFINITY, l_run = 0.f, rs = 0.f, rs2 = 0.f;
    for (RingPos np = dp;; np.step(1, KX_DESCS)) {
      // ---- the next segment's queries, as soon as this one's are read (its last scores are there).
      // The barriers of queries and of the segment's end turn only in segments where the group has a
      // tile: each of their turns then waits for every warp to have seen the one before.
      const bool so_far = ok;
      const Seg s2 = segment(np);
      ok = __all_sync(0xffffffffu, ok && so_far);
      if (ok && s2.valid && s2.tiles_of(g)) rs2 = stage(s2);
      if (s.valid) {
        // ---- this segment's result: state g, or half of the dims of both groups' states
        if (work) {
          ok = kx_wait(bar_fin + 8 * g, turn, a.err, abort_flag) && ok;
          turn ^= 1;
        }
        tc_fence_after();
        const int v = s.v0 + lv + (both ? 0 : KA_QV * g), i = row_of(a, v), h = s.kvh * a.G + (v - i * a.G);
        const bool live = v - s.v0 < s.qv;
        float2 st[2] = {make_float2(l_run == 0.f ? -INFINITY : m_run * rs - LIFT, l_run), make_float2(-INFINITY, 0.f)};
        if (both) {
          states[128 * g + lv] = st[0];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_x);
          ok = kx_wait(bar_x, xturn, a.err, abort_flag) && ok;
          tc_fence_after();
          st[0] = states[lv];
          st[1] = states[128 + lv];
        }
        const uint32_t o0 = tmem + lane_base + T_O + (both ? 0 : 128 * g), o1 = tmem + lane_base + T_O + 128;
        constexpr int CW = 32, BW = 8;         // dims of a chunk, of a block
        const int c_lo = both ? g * (HD / 2) : 0, c_hi = c_lo + (both ? HD / 2 : HD);
        float M = max_nan(st[0].x, st[1].x);
        const bool join = OWN && s.slot < 0;
        if (join && !waited) {
          pdl_wait();
          waited = true;
        }
        const int row = s.row0 + i;
        const Own mine(own, OWN && live && join ? row : -1, h);
#pragma unroll 1
        for (int k = 0; OWN && k < mine.used; ++k) M = max_nan(M, mine.ml(k).x);
        const float f0 = part_factor(st[0].x, M), f1 = part_factor(st[1].x, M);
        float L = fmaf(f0, st[0].y, f1 * st[1].y);
#pragma unroll 1
        for (int k = 0; OWN && k < mine.used; ++k) {
          const float2 ml = mine.ml(k);
          if (ml.x != -INFINITY) L = fmaf(part_factor(ml.x, M), ml.y, L);
        }
        const bool none = L == 0.f, writes = live && (!join || mine.used > 0);
        const float inv = s.slot >= 0 ? 1.f : none ? 0.f : a.vg / L, own_inv = !OWN || none ? 0.f : own.vg / L;
        float* part = parts + gridDim.x * (sizeof(Cut) / 4) + (s.slot >= 0 ? static_cast<size_t>(s.slot) : 0) * kx_slot(HD);
        const int pv = v - s.v0;
        // Four lanes' rows in chunks of 32 dims are turned so that four lanes hold one row: a store then
        // touches 8 rows instead of 32.
        const long long at = row * a.out_ld + static_cast<long long>(h) * HD;
        const int ranges = OWN && join ? __reduce_max_sync(0xffffffffu, mine.used) : 0;
        const float w0 = f0 * inv, w1 = f1 * inv;
        // (a state of no tile: its O was never written; one whose weight fell to 0 leaves what is not finite)
        const bool gone0 = __any_sync(0xffffffffu, w0 == 0.f), gone1 = __any_sync(0xffffffffu, w1 == 0.f);
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_hi; c0 += CW) {
          float x[CW];
          __syncwarp();
          tmem_ld32(o0 + c0, x);
          tmem_wait_ld();
          if (gone0) {
#pragma unroll
            for (int e = 0; e < CW; ++e) x[e] = st[0].x == -INFINITY ? 0.f : weighted(w0, x[e]);
          } else {
#pragma unroll
            for (int e = 0; e < CW; ++e) x[e] *= w0;
          }
          if (both) {
            float y[CW];
            tmem_ld32(o1 + c0, y);
            tmem_wait_ld();
            if (gone1) {
#pragma unroll
              for (int e = 0; e < CW; ++e) x[e] = st[1].x == -INFINITY ? x[e] : add_weighted(x[e], w1, y[e]);
            } else {
#pragma unroll
              for (int e = 0; e < CW; ++e) x[e] = fmaf(w1, y[e], x[e]);
            }
          }
          if constexpr (!F4) {                 // (of 4-bit values none is infinite)
            float2 z = make_float2(0.f, 0.f);  // (0 unless some sum is not finite)
#pragma unroll
            for (int e = 0; e < CW; e += 2) z = __ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(0.f, 0.f), z);
            const bool bad = live && isnan(z.x + z.y) && fabsf(L) < INFINITY;
            if (__any_sync(0xffffffffu, bad)) {
              float inf;
              infinities<HD, 1>(a.pool, s.b, s.kvh, s.t0 * KEYS, min((s.t0 + s.T) * KEYS, s.len), c0 + lane, &inf, lane, a.err);
#pragma unroll
              for (int e = 0; e < CW; ++e) {
                const float y = __shfl_sync(0xffffffffu, inf, e);
                if (bad && isnan(x[e]) && y != 0.f) x[e] = y;
              }
            }
          }
          if (s.slot >= 0) {
            float4* dst = reinterpret_cast<float4*>(part) + static_cast<size_t>(c0 / 4) * KX_QV + pv;
            if (writes) {
#pragma unroll
              for (int e = 0; e < CW / 4; ++e) dst[e * KX_QV] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
            continue;
          }
          // blocks of BW dims; with own keys' results to come as floats, else packed
          constexpr int WORDS = OWN ? BW : BW / 2;
          float z[4 * WORDS];
#pragma unroll
          for (int e = 0; e < 4 * WORDS; ++e) z[e] = OWN ? x[e] : __uint_as_float(pack_bf16(x[(2 * e) % CW], x[(2 * e + 1) % CW]));
#pragma unroll
          for (int d = 1; d < 4; d <<= 1)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (b & d) continue;
#pragma unroll
              for (int e = 0; e < WORDS; ++e) {
                float& lo = z[b * WORDS + e];
                float& hi = z[(b + d) * WORDS + e];
                const float got = __shfl_xor_sync(0xffffffffu, lane & d ? lo : hi, d);
                if (lane & d) lo = got;
                else hi = got;
              }
            }
#pragma unroll
          for (int r = 0; r < 4; ++r) {        // block r: lane's dims [c0 + BW (lane % 4), ...) of row (lane & ~3) + r
            const int from = (lane & ~3) + r;
            float* y = z + r * WORDS;
            const long long to_row = __shfl_sync(0xffffffffu, writes ? at : -1, from);
            const int d0 = c0 + BW * (lane & 3);
#pragma unroll 1
            for (int k = 0; OWN && k < ranges; ++k) {
              float f = 0.f;
              unsigned long long place = ~0ull;
              if (k < mine.used) {
                const float m = mine.ml(k).x;
                f = part_factor(m, M) * own_inv;
                if (m != -INFINITY) place = mine.place(k);
              }
              f = __shfl_sync(0xffffffffu, f, from);
              place = __shfl_sync(0xffffffffu, place, from);
              const float4* src = reinterpret_cast<const float4*>(own.part_o + place * HD + d0);
              if (place != ~0ull) {
#pragma unroll
                for (int e = 0; e < WORDS / 4; ++e) add_part(y + 4 * e, f, src[e]);
              }
            }
            if (to_row < 0) continue;
            uint32_t w[BW / 2];
#pragma unroll
            for (int e = 0; e < BW / 2; ++e) w[e] = OWN ? pack_bf16(y[(2 * e) % WORDS], y[(2 * e + 1) % WORDS]) : __float_as_uint(y[e % WORDS]);
            *reinterpret_cast<uint4*>(a.out + to_row + d0) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (writes && (!both || g == 0)) {
          if (s.slot >= 0) reinterpret_cast<float2*>(part + static_cast<size_t>(KX_QV) * HD)[pv] = make_float2(none ? -INFINITY : M, L);
          else if (a.lse) a.lse[static_cast<size_t>(row) * a.Hq + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        }
        if (both) {                            // (all have read O and the states before any goes on)
          __syncwarp();
          tc_fence_before();
          if (lane == 0) mbar_arrive(bar_x + 8);
          ok = kx_wait(bar_x + 8, xturn, a.err, abort_flag) && ok;
          xturn ^= 1;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_de + 8 * dp.slot);
      }
      if (!__all_sync(0xffffffffu, ok && s2.valid)) break;
      dp = np;
      s = s2;
      both = s.both();
      work = s.tiles_of(g);
      rs = rs2;
      idle = 32 * quad >= s.qv - (both ? 0 : KA_QV * g);   // a warp without vectors
      const int end_page = s.len >> a.pool.ps_log, end_rows = F4 ? 0 : s.len & (ps - 1);
      const int W = s.units_of<UPT>(g, last_units(s));
      m_run = -INFINITY;
      l_run = 0.f;
#pragma unroll 1
      for (int w = 0; w < W; ++w, ++n) {
        const uint32_t buf = 2 * g + (n & 1), ts = tmem + lane_base + buf * KA_H;
        ok = ok && kx_wait(bar_sf + 8 * buf, (n >> 1) & 1, a.err, abort_flag);
        tc_fence_after();
        if (!idle) {
          // The scores become p with the maximum so far, which mostly stays, while this unit's is found;
          // where that rose too far they are read again.
          const int own_tile = UPT == 2 ? w >> 1 : w, kt = (s.t0 + (both ? g + 2 * own_tile : own_tile)) * KEYS;   // the tile's first key
          float x[KA_H], p8[8], pk[32];
#pragma unroll 1
          for (bool again = false;;) {
            tmem_ld32(ts, x);
            tmem_ld32(ts + 32, x + 32);
            tmem_wait_ld();
            if (kt + KEYS > s.len) {         // columns without a key
              const int at = (end_page << a.pool.ps_log) - kt;
              Bits vis = bits_below(end_rows ? at + ps : s.len - kt);
              if (end_rows) {
                const Bits lo = bits_below(at), hi = bits_below(at + ps - end_rows);
                vis.lo &= lo.lo | ~hi.lo;
                vis.hi &= lo.hi | ~hi.hi;
              }
              const unsigned long long bits = UPT == 2 && (w & 1) ? vis.hi : vis.lo;
#pragma unroll
              for (int e = 0; e < KA_H; ++e) x[e] = (bits >> e) & 1ull ? x[e] : -INFINITY;
            }
            // (a row without a key so far takes the maximum as 0: every score is -inf, every p is 0)
            const float mb = (m_run == -INFINITY ? 0.f : m_run * rs) - LIFT;
#pragma unroll
            for (int e = 0; e < 8; ++e) p8[e] = 0.f;
            const float mt = powers64<F4>(x, rs, mb, p8, pk);
            const bool rose = !again && mt != -INFINITY && (m_run == -INFINITY || (mt - m_run) * rs > KA_RESCALE);
            if (!__any_sync(0xffffffffu, rose)) break;
            const bool resc = rose && m_run != -INFINITY;
            const float f = resc ? fast_exp2((m_run - mt) * rs) : 1.f;
            if (rose) m_run = mt;
            if (__any_sync(0xffffffffu, resc)) {
              // (the scores are there, so the P V of the units before the last is done; that one's is waited for)
              ok = ok && kx_wait(bar_pe + 8 * (buf ^ 1), ((n - 1) >> 1) & 1, a.err, abort_flag);
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < HD; c0 += 16) {
                float z[16];
                tmem_ld16(to + c0, z);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] *= f;
                tmem_st16(to + c0, z);
              }
            }
            l_run *= f;
            again = true;
          }
          tmem_st16(ts, pk);
          tmem_st16(ts + 16, pk + 16);
          l_run += ((p8[0] + p8[1]) + (p8[2] + p8[3])) + ((p8[4] + p8[5]) + (p8[6] + p8[7]));
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_pf + 8 * buf);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the partial results of the items that the cuts divide: block x the item whose first part is
// CTA x's; 32 of its vectors (lanes), HD / 8 dims a warp.
template <int HD>
__global__ void __launch_bounds__(32 * KX_JOIN_WARPS) kv_cross_wide_join(const KaArgs a, const KaArgs own, const int with_own, const float* parts) {
  constexpr int E = HD / 4 / KX_JOIN_WARPS;  // float4s of a thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  pdl_wait();                                // the parts, and the own keys' results
  const Cut s = reinterpret_cast<const Cut*>(parts)[c];
  const int pv = KX_JOIN_V * blockIdx.y + lane, v = s.v0 + pv, last = s.last;
  if (last == 0 || pv >= s.qv) return;
  parts += gridDim.x * (sizeof(Cut) / 4);
  const int i = row_of(a, v), h = s.kvh * a.G + (v - i * a.G);
  const size_t row = static_cast<size_t>(s.row0 + i);
  auto part = [&](int k) { return parts + static_cast<size_t>(k == c ? s.slot : 2 * k) * kx_slot(HD); };
  auto state = [&](int k) { return reinterpret_cast<const float2*>(part(k) + static_cast<size_t>(KX_QV) * HD)[pv]; };
  float M = -INFINITY;
#pragma unroll 4
  for (int k = c; k <= last; ++k) M = max_nan(M, state(k).x);
  const Own mine(own, with_own ? static_cast<int>(row) : -1, h);
  if (with_own && mine.used == 0) return;
#pragma unroll 1
  for (int k = 0; k < mine.used; ++k) M = max_nan(M, mine.ml(k).x);
  float x[4 * E] = {}, L = 0.f;
#pragma unroll 4
  for (int k = c; k <= last; ++k) {
    const float2 ml = state(k);
    if (ml.x == -INFINITY) continue;
    const float f = part_factor(ml.x, M);
    L = fmaf(f, ml.y, L);
    const float4* src = reinterpret_cast<const float4*>(part(k)) + static_cast<size_t>(warp * E) * KX_QV + pv;
#pragma unroll
    for (int e = 0; e < E; ++e) add_part(x + 4 * e, f, src[e * KX_QV]);
  }
  float y[4 * E] = {};
#pragma unroll 1
  for (int k = 0; k < mine.used; ++k) {
    const float2 ml = mine.ml(k);
    if (ml.x == -INFINITY) continue;
    const float f = part_factor(ml.x, M);
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

template <int HD, int CACHE, bool OWN>
cudaError_t launch_wide(const CUtensorMap& tmk, const CUtensorMap& tmv, const KaArgs& a, const KaArgs& own, float* parts,
                        int ctas, cudaStream_t st) {
  static std::atomic<size_t> granted[64];    // shared memory per device, set on its first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  size_t cap = dev < 64 ? granted[dev].load() : 0;
  if (!cap) {
    e = allow_max_smem(reinterpret_cast<const void*>(kv_cross_wide<HD, CACHE, OWN>), &cap);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;                   // the roles' registers must fit what the launch gives, or they would wait for ever
    e = cudaFuncGetAttributes(&fa, kv_cross_wide<HD, CACHE, OWN>);
    if (e != cudaSuccess) return e;
    const int need = 128 * KX_REG_CTRL + KX_SOFTMAX * KX_REG_SOFTMAX + 32 * KX_COPIERS * KX_REG_LOAD;
    if (fa.numRegs / 8 * 8 * KX_THREADS < need || fa.numRegs < KX_REG_LOAD) return cudaErrorInvalidConfiguration;
    if (dev < 64) granted[dev].store(cap);
  }
  constexpr bool F4 = CACHE == EAGLE_CACHE_F4;
  constexpr size_t fixed = 2 * ka_entry(HD) + KX_MISC, entry = kx_entry(HD, CACHE), raw = kx_raw_bytes(HD);
  const int ns = F4 ? (HD == 64 ? 12 : 7) : std::min<int>(KA_MAX_SLOTS, static_cast<int>((cap - fixed) / entry));
  if (cap < fixed + 4 * entry || ns < 4 || cap < fixed + ns * entry) return cudaErrorInvalidConfiguration;   // (a shared item's groups are 4 entries apart)
  const int nr = F4 ? std::min<int>(KX_MAX_RAW, static_cast<int>((cap - fixed - ns * entry) / raw)) : 0;
  if (F4 && nr < KX_COPIERS) return cudaErrorInvalidConfiguration;
  e = launch_after(OWN, dim3(ctas), KX_THREADS, fixed + ns * entry + nr * raw, st, kv_cross_wide<HD, CACHE, OWN>,
                   tmk, tmv, a, own, parts, ns, nr);
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_after(true, dim3(ctas, KX_QV / KX_JOIN_V), 32 * KX_JOIN_WARPS, 0, st, kv_cross_wide_join<HD>, a, own, OWN ? 1 : 0,
                      static_cast<const float*>(parts));
}

template <int HD>
cudaError_t launch_kind(const CUtensorMap& tmk, const CUtensorMap& tmv, const KaArgs& a, const KaArgs& own, bool with_own, bool f4, float* parts,
                        int ctas, cudaStream_t st) {
  if (f4) return with_own ? launch_wide<HD, EAGLE_CACHE_F4, true>(tmk, tmv, a, own, parts, ctas, st)
                          : launch_wide<HD, EAGLE_CACHE_F4, false>(tmk, tmv, a, own, parts, ctas, st);
  return with_own ? launch_wide<HD, EAGLE_CACHE_BF16, true>(tmk, tmv, a, own, parts, ctas, st)
                  : launch_wide<HD, EAGLE_CACHE_BF16, false>(tmk, tmv, a, own, parts, ctas, st);
}

}  // namespace

// Ranges (kv_attention_tc, kv_attention_step_f4) start sooner and need one launch where they join in a cluster;
// this kernel's shares are even whatever the lengths, but it starts and joins for 16 us and every short
// item costs it a queue's drain.  Measured over 700 sizes (both kinds, 64 and 128 dims, 12 to 4,096
// vectors, 1 to 128 sequences of 250 to 80,000 keys, equal and spread), of items of 2,432 keys and more:
//   up to 128 vectors: ranges, which over bf16 pages keep 16 bits of p where this kernel keeps 8 (and are
//     slower where few sequences meet 16 KV heads of 64 dims: 8 of 8,000 keys, 128 vectors 94 us, here 60)
//   bf16, more: here where a few sequences leave the SMs under one item each (4 of 5,000 to 35,000 keys, 8
//     heads, 256 vectors: 86 us, by ranges 98), or where a hundred tiles an SM outweigh the start
//     (prompts: 219, by ranges 229)
//   4 bits, more: 10 tiles an SM and more (the same 4 sequences: 90, by ranges 119)
// and ranges elsewhere (1 of 8,000 bf16 keys, 12 vectors: 18 us, here 31; 32 of 125 to 870: 25, here 61;
// 256 vectors: 38, here 72).  The mean loss to the faster of the two: up to 128 vectors 4.2% (bf16) and 3.3%,
// more 0.6% and 1.2%.
// A range's CTAs are launched for every block that the bounds allow; where the rows can fill one in 8 of
// them at most, as a prompt of 4,096 rows among 63 single tokens does, the empty ones cost more than the
// rest (1,000 keys, 8 heads: 285 us, here 143; 1,024 rows: 109, here 96; one in 5: 56, here 63).
bool eagle::kx_worth(int kind, int Hkv, int G, int B, long long N, int max_rows, int max_len) {
  const int sms = num_sms() > 0 ? num_sms() : 152;   // (152: without a device, a GB300's)
  const long long qv = static_cast<long long>(max_rows) * G, blocks = (qv + KX_QV - 1) / KX_QV;
  if (blocks > 1 && static_cast<double>(B) * static_cast<double>(blocks) > 8. * (static_cast<double>(N) * G / KX_QV + B)) return true;
  const double tiles = static_cast<double>((static_cast<long long>(max_len) + KA_CH - 1) / KA_CH);
  const double items = static_cast<double>(B) * Hkv * static_cast<double>(blocks) / sms, work = items * tiles;
  if (qv <= KA_QV || tiles < 20) return false;
  const bool few = B > 1 && items <= 1;      // (of several sequences, whose lengths may differ)
  if (kind == EAGLE_CACHE_F4) return work >= 10;
  return (few && work >= 10) || work >= 100;
}

KxPlan eagle::kx_plan(int kind, int Hkv, int hd, int G, int B, int max_rows, int max_len) {
  const long long blocks = (static_cast<long long>(max_rows) * G + KX_QV - 1) / KX_QV, tiles = (static_cast<long long>(max_len) + kx_keys(kind) - 1) / kx_keys(kind);
  const double units = static_cast<double>(B) * Hkv * blocks * tiles;
  const int sms = num_sms() > 0 ? num_sms() : 152;   // (152: without a device, a GB300's)
  KxPlan p;
  const double ctas = units / (KX_MIN_KEYS / kx_keys(kind));
  p.ctas = ctas < sms ? static_cast<int>(ctas) + 1 : sms;
  p.bytes = p.ctas * (static_cast<int64_t>(sizeof(Cut)) + (p.ctas == 1 ? 0 : 8ll * kx_slot(hd)));
  return p;
}

cudaError_t eagle::kx_launch(const KaArgs& a, const KaArgs* own, bool f4, const CUtensorMap& tmk, const CUtensorMap& tmv, const KxPlan& p,
                             float* parts, cudaStream_t st) {
  KaArgs none;
  memset(&none, 0, sizeof(none));
  const KaArgs& o = own ? *own : none;
  return a.pool.hd == 64 ? launch_kind<64>(tmk, tmv, a, o, own != nullptr, f4, parts, p.ctas, st)
                         : launch_kind<128>(tmk, tmv, a, o, own != nullptr, f4, parts, p.ctas, st);
}
