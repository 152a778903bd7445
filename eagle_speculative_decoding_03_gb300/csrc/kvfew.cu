// Attention of few query vectors (at most 8 a KV head: a token of each of 8 grouped heads) over bf16
// pages, every row seeing all its keys: cross attention's step, and a step's own keys behind a shared
// prefix.  Bound by the keys' bytes.  See kvattn.cu for the notation and kvline.cuh for how the work
// is dealt out.
//
// One CTA per SM.  Four warps walk the CTA's tiles of 64 keys, across items, and bring keys, values
// and (ahead of an item's first tile) its queries into a ring, so that the copies of the next item run
// while the last is finished.  Eight warps, two teams that take every other tile, 16 keys of it each:
//   S^T [16 keys x 8 vectors] = K Q^T        A = keys (ldmatrix), B = queries
//   O^T [16 dims x 8 vectors] += V^T P^T     A = values (ldmatrix, transposed), B = P (8 x 8 transposes)
// with a running maximum and sum a warp; their states meet in shared memory at the item's end, in warp
// order.  (kv_attention_tc spends 128 rows of MMA and a CTA's start and end on such an item.)
//
// 32 sequences of 300 to 3,000 keys, 16 heads of 64 (217 MB): 51 us with the join, 4.3 TB/s, 63% of
// the measured copy rate; the ranges of kv_attention_tc take 75.  What is over is the start (a CTA finds
// its place among the sequences, 3 us), the copies' first latency and the join's launch.  With little
// to read those count for more than even shares, see kf_worth.
//
// Rows behind the last key are cleared in the fragments (they may hold NaN).  For the second product p is
// held in two bf16 parts, 16 bits, as in kv_attention_tc's ranges, so that a request's result does not get
// coarser with the batch that it is in: 1.7e-3 of the output's norm from 64 bits, its own rounding, for
// 1.2 us of the 51 (one part: 2.2e-3).  l sums the unrounded p.
#include "kvline.cuh"

#include <algorithm>
#include <atomic>

using namespace eagle;

namespace {

constexpr int KF_KEYS = 64;                // keys of a tile
constexpr int KF_WARPS = 8;                // computing warps: two teams of four
constexpr int KF_LOADERS = 4;              // warps that bring the tiles: one thread issues a copy in 200 cycles (57 us of
                                           // the case above, of 8 KB boxes, with one warp)
constexpr int KF_THREADS = 32 * (KF_WARPS + KF_LOADERS);
constexpr int KF_MAX_STAGES = 12;
constexpr int KF_MIN_UNITS = 4;            // tiles that are worth a CTA
constexpr uint32_t KF_MISC = 1152;         // barriers (0), tiles' descriptors (256), maxima (640) and sums (896)
using KfLine = Line<3, KF_KEYS>;           // (blocks of KF_QV vectors: one)

__host__ __device__ constexpr uint32_t kf_half() { return KF_KEYS * 128; }
__host__ __device__ constexpr uint32_t kf_stage(int hd) { return 2 * KF_KEYS * hd * 2 + KF_QV * hd * 2; }   // keys, values; queries
__host__ __device__ constexpr uint32_t kf_kv(int hd) { return 2 * KF_KEYS * hd * 2; }
__host__ __device__ constexpr int kf_ld(int hd) { return hd + 4; }   // (the lanes of a fragment fall on different banks)
__host__ __device__ constexpr uint32_t kf_states(int hd) { return KF_WARPS * KF_QV * kf_ld(hd) * 4; }
// floats of a partial result: [8][hd] outputs, [8] (maximum, sum)
__host__ __device__ constexpr size_t kf_slot(int hd) { return static_cast<size_t>(KF_QV) * (hd + 2); }

// A tile in the ring, and its place in the CTA's part of an item.
enum : int { KF_FIRST = 1, KF_LAST = 2, KF_END = 4 };
struct Tile {
  int flags, keys, row0, kvh, qv, slot, b, k0;   // keys: of the tile (0 .. 64), from k0 on; slot: partial result, -1: the item is whole
};

EAGLE_DEV void ldmatrix4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
EAGLE_DEV void ldmatrix4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
EAGLE_DEV void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
EAGLE_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Writes vector v's dims d, d + 1 (and, with d = 0, its maximum and sum): sums y of parts scaled to M.
EAGLE_DEV void emit(const KaArgs& a, int row0, int kvh, int v, int d, int HD, float M, float L, float y0, float y1) {
  const int i = row_of(a, v), h = kvh * a.G + (v - i * a.G);
  const long long n = row0 + i;
  const size_t at = static_cast<size_t>(n) * a.Hq + h;
  const bool none = L == 0.f;
  if (a.parts) {
    if (!none) *reinterpret_cast<float2*>(a.part_o + at * HD + d) = make_float2(y0, y1);
    if (d == 0) a.part_ml[at] = make_float2(none ? -INFINITY : M, L);
  } else {
    const float inv = none ? 0.f : a.vg / L;
    *reinterpret_cast<uint32_t*>(a.out + n * a.out_ld + static_cast<long long>(h) * HD + d) = none ? 0u : pack_bf16(y0 * inv, y1 * inv);
    if (d == 0 && a.lse) a.lse[at] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

template <int HD>
__global__ void __launch_bounds__(KF_THREADS, 1)
kv_few(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const KaArgs a, float* parts, const int NS) {
  constexpr int KS = HD / 16;                // 16-dim steps
  constexpr uint32_t HALF = kf_half(), STAGE = kf_stage(HD), V_AT = KF_KEYS * HD * 2, Q_AT = kf_kv(HD);
  constexpr int LD = kf_ld(HD);
  extern __shared__ __align__(1024) uint8_t kf_sm[];
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, g = lane >> 2, c = lane & 3;
  // keys and values of all stages first (whole swizzle atoms), then their queries
  const uint32_t ring = smem_u32(kf_sm), queries = ring + static_cast<uint32_t>(NS) * kf_kv(HD);
  uint8_t* rest = kf_sm + static_cast<uint32_t>(NS) * STAGE;
  float* s_o = reinterpret_cast<float*>(rest);                       // [warp][8][LD]
  uint8_t* misc = rest + kf_states(HD);
  const uint32_t misc_u = smem_u32(misc), bar_full = misc_u, bar_free = misc_u + 96, bar_states = misc_u + 192, bar_read = misc_u + 200;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 208);
  Tile* tiles = reinterpret_cast<Tile*>(misc + 256);
  float* s_m = reinterpret_cast<float*>(misc + 640);                 // [warp][8]
  float* s_l = reinterpret_cast<float*>(misc + 896);
  pdl_trigger();
  if (misplaced(ring, parts, a.err)) return;
  if (tid == 0) {
    for (int s = 0; s < KF_MAX_STAGES; ++s) {
      mbar_init(bar_full + 8 * s, KF_LOADERS);
      mbar_init(bar_free + 8 * s, KF_WARPS);
    }
    mbar_init(bar_states, KF_WARPS);
    mbar_init(bar_read, KF_WARPS);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  bool ok = true;
  RingPos rp{0, 0};
  if (warp >= KF_WARPS) {
    // ------------------------------------------------------------ the tiles
    const int part = warp - KF_WARPS;        // of every tile's copies
    const uint64_t pol = policy_evict_first();
    const long long all = all_units<KfLine>(a, lane), per = units_per_cta(all, gridDim.x, KF_MIN_UNITS);
    const long long begin = min(per * blockIdx.x, all), end = min(begin + per, all);
    long long u = begin, rest_u = 0;
    int b = u < end ? find_unit<KfLine>(a, lane, u, &rest_u) : 0, pushed = 0;
    Cut cut;
    cut.last = 0;
    const int rows = min(1 << a.pool.ps_log, KF_KEYS), boxes = KF_KEYS / rows;
    const int copies = 2 * (HD / 64) * boxes;          // 2, 4, ... 16
    const uint32_t box_bytes = static_cast<uint32_t>(rows) * 128, mine = static_cast<uint32_t>((copies - part + KF_LOADERS - 1) / KF_LOADERS) * box_bytes;
    // waits for the stage at rp and announces its tile, of which this warp copies `bytes`
    auto push = [&](const Tile& t, uint32_t bytes) {
      if (pushed >= NS) ok = kx_wait(bar_free + 8 * rp.slot, rp.turn ^ 1, a.err, abort_flag);
      else ++pushed;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) {
        if (part == 0) tiles[rp.slot] = t;
        if (bytes) mbar_arrive_expect_tx(bar_full + 8 * rp.slot, bytes);
        else mbar_arrive(bar_full + 8 * rp.slot);
      }
      __syncwarp();
    };
    while (ok && u < end) {
      KfLine l(a, b);
      while (rest_u >= l.units(a)) {         // (the next sequence that has units)
        rest_u -= l.units(a);
        ++b;
        l = KfLine(a, b);
      }
      const int kvh = static_cast<int>(quotient(rest_u, l.tiles)), t0 = static_cast<int>(rest_u - static_cast<long long>(kvh) * l.tiles);
      const int n = static_cast<int>(min(static_cast<long long>(l.tiles - t0), end - u)), qv = l.rq.R * a.G;
      Tile t;
      t.b = b;
      t.row0 = l.rq.row0;
      t.kvh = kvh;
      t.qv = qv;
      t.slot = n == l.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (u == begin ? 0 : 1);
      if (t0 == 0 && n < l.tiles) cut = Cut{static_cast<int>(quotient(u + l.tiles - 1, per)), kvh, t.row0, 0, qv, t.slot};
      Pages pages;
      pages.open(a, b, t0 * KF_KEYS, l.rq.len, rows, lane);
#pragma unroll 1
      for (int x = 0; x < n && ok; ++x) {
        const int k0 = (t0 + x) * KF_KEYS, page = pages.get(a, b, t0 * KF_KEYS, l.rq.len, rows, lane, x * boxes);
        t.k0 = k0;
        t.keys = max(min(l.rq.len - k0, KF_KEYS), 0);
        t.flags = (x == 0 ? KF_FIRST : 0) | (x == n - 1 ? KF_LAST : 0);
        const bool data = t.keys > 0;
        push(t, (data ? mine : 0u) + (x == 0 && part == 0 ? static_cast<uint32_t>(qv) * HD * 2 : 0u));
        if (!ok) break;
        const uint32_t slot = uniform(rp.slot), bar = bar_full + 8 * slot, at = ring + slot * kf_kv(HD);
        // (all that a copy takes is the same for the whole warp)
#pragma unroll 1
        for (int i = part; i < copies && data; i += KF_LOADERS) {   // (a page that is not there reads as zeros: a block outside the map)
          const int v = i & 1, h = (i >> 1) & (HD / 64 - 1), bx = i / (2 * (HD / 64)), pg = __shfl_sync(0xffffffffu, page, bx);
          const int blk = pg >= 0 ? pg * a.pool.Hkv + kvh : a.pool.num_pages * a.pool.Hkv;
          const int row = (k0 + bx * rows) & ((1 << a.pool.ps_log) - 1);
          if (elect_one()) tma_load_3d(at + v * V_AT + h * HALF + bx * box_bytes, v ? &tmv : &tmk, 64 * h, row, blk, bar, pol);
        }
        if (x == 0 && part == 0 && lane >= 16 && lane - 16 < qv) {
          const int v = lane - 16, i = row_of(a, v);
          bulk_load(queries + (rp.slot * KF_QV + v) * HD * 2, a.q + (t.row0 + i) * a.q_ld + static_cast<long long>(kvh * a.G + v - i * a.G) * HD, HD * 2, bar);
        }
        rp.step(1, NS);
      }
      u += n;
      rest_u += n;
    }
    if (ok) {
      Tile t;
      t.flags = KF_END;
      push(t, 0);
    }
    if (part == 0 && lane == 0) reinterpret_cast<Cut*>(parts)[blockIdx.x] = cut;
    if (!ok) {   // let copies already issued land before the CTA releases its shared memory
      const long long t0 = clock64();
      while (clock64() - t0 < 4000000) {
      }
    }
    return;
  }
  parts += gridDim.x * (sizeof(Cut) / 4);
  const int team = warp >> 2, sub = 16 * (warp & 3);
  // rows and 16-byte chunks that this lane addresses: of keys (row k, dims), of values (transposed)
  const int k_row = sub + ((lane >> 3) & 1) * 8 + (lane & 7), k_chunk = lane >> 4;
  const int v_row = sub + (lane >> 4) * 8 + (lane & 7), v_chunk = (lane >> 3) & 1;
  uint32_t q[KS][2];
  float o[KS][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // log2 units; sums over this lane's keys
  uint32_t items = 0;
  int begin = 0;                             // the item's first key here
  for (uint32_t n = 0;; ++n, rp.step(1, NS)) {
    ok = kx_wait(bar_full + 8 * rp.slot, rp.turn, a.err, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const Tile t = tiles[rp.slot];
    if (t.flags & KF_END) break;
    const uint32_t at = ring + rp.slot * kf_kv(HD);
    if (t.flags & KF_FIRST) {
      // vector g's dims 16 s + 2 c, + 1, + 8, + 9 (of vectors that are not there: zeros)
      const uint32_t src = queries + (rp.slot * KF_QV + g) * HD * 2 + 4 * c;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(q[s][0]) : "r"(src + 32 * s) : "memory");
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(q[s][1]) : "r"(src + 32 * s + 16) : "memory");
        if (g >= t.qv) q[s][0] = q[s][1] = 0u;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[s][e] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
      begin = t.k0;
    }
    const int left = t.keys - sub;           // keys of this warp's 16
    if ((n & 1) == team && left > 0) {
      float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        uint32_t k[4];
        const int ch = 2 * i + k_chunk;
        ldmatrix4(k, at + (ch >> 3) * HALF + ka_sw(k_row, ch & 7));
        mma_bf16(i & 1 ? s2 : s, k, q[i][0], q[i][1]);
      }
      // s: key g, vectors 2c, 2c + 1; key g + 8
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = (s[e] + s2[e]) * a.scale_log2;
      if (left < 16) {
        if (g >= left) s[0] = s[1] = -INFINITY;
        if (g + 8 >= left) s[2] = s[3] = -INFINITY;
      }
      const float t0 = max_nan(s[0], s[2]), t1 = max_nan(s[1], s[3]);
      // the running maximum moves only when some score exceeds it by more than KA_RESCALE
      if (__any_sync(0xffffffffu, !(t0 <= m0 + KA_RESCALE) || !(t1 <= m1 + KA_RESCALE))) {
        float n0 = max_nan(t0, m0), n1 = max_nan(t1, m1);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          n0 = max_nan(n0, __shfl_xor_sync(0xffffffffu, n0, d));
          n1 = max_nan(n1, __shfl_xor_sync(0xffffffffu, n1, d));
        }
        if (n0 <= m0 + KA_RESCALE) n0 = m0;  // (no vector's bits depend on the others')
        if (n1 <= m1 + KA_RESCALE) n1 = m1;
        const float f0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f1;
          o[j][2] *= f0;
          o[j][3] *= f1;
        }
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;   // (nothing seen yet: every p is 0)
      uint32_t p[2], r[2];                   // rounded to bf16, and what that leaves
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = fast_exp2(s[2 * h] - b0), p1 = fast_exp2(s[2 * h + 1] - b1);
        l0 += p0;
        l1 += p1;
        const uint32_t hi = pack_bf16(p0, p1);
        p[h] = transpose8x8(hi);             // keys 2c, 2c + 1 (+ 8 h) of vector g
        r[h] = transpose8x8(pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u)));
      }
      // masks of the pairs of keys 2c, 2c + 1 and 8 + those that are there
      const uint32_t lo = (2 * c < left ? 0xFFFFu : 0u) | (2 * c + 1 < left ? 0xFFFF0000u : 0u);
      const uint32_t hi = (2 * c + 8 < left ? 0xFFFFu : 0u) | (2 * c + 9 < left ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        uint32_t v[4];
        const int ch = 2 * j + v_chunk;
        ldmatrix4_trans(v, at + V_AT + (ch >> 3) * HALF + ka_sw(v_row, ch & 7));
        if (left < 16) {
          v[0] &= lo;
          v[1] &= lo;
          v[2] &= hi;
          v[3] &= hi;
        }
        mma_bf16(o[j], v, p[0], p[1]);
        mma_bf16(o[j], v, r[0], r[1]);
      }
    }
    // (the stage's next copy is another proxy's write; keys and values went through products, queries may
    // still be on their way to the registers of the team whose turn it is not)
    if (t.flags & KF_FIRST) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_free + 8 * rp.slot);
    if (t.flags & KF_LAST) {
      // ---- the eight warps' states, in warp order
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      if (items) ok = kx_wait(bar_read, (items - 1) & 1, a.err, abort_flag);   // (the last item's are read)
      if (g == 0) {
        s_m[warp * KF_QV + 2 * c] = m0;
        s_m[warp * KF_QV + 2 * c + 1] = m1;
        s_l[warp * KF_QV + 2 * c] = l0;
        s_l[warp * KF_QV + 2 * c + 1] = l1;
      }
      float* mine = s_o + warp * KF_QV * LD;
#pragma unroll
      for (int j = 0; j < KS; ++j) {         // dims 16 j + g and + 8
        mine[2 * c * LD + 16 * j + g] = o[j][0];
        mine[(2 * c + 1) * LD + 16 * j + g] = o[j][1];
        mine[2 * c * LD + 16 * j + 8 + g] = o[j][2];
        mine[(2 * c + 1) * LD + 16 * j + 8 + g] = o[j][3];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_states);
      ok = kx_wait(bar_states, items & 1, a.err, abort_flag) && ok;
      // one (vector, pair of dims): the warps' states joined, and written
      auto join = [&](int v, int d, float& M, float& L, float& y0, float& y1) {
        M = -INFINITY;
        L = y0 = y1 = 0.f;
#pragma unroll
        for (int w = 0; w < KF_WARPS; ++w) M = max_nan(M, s_m[w * KF_QV + v]);
#pragma unroll
        for (int w = 0; w < KF_WARPS; ++w) {
          const float mw = s_m[w * KF_QV + v];
          if (mw == -INFINITY) continue;
          const float f = part_factor(mw, M);
          const float2 y = *reinterpret_cast<const float2*>(s_o + (w * KF_QV + v) * LD + d);
          L = fmaf(f, s_l[w * KF_QV + v], L);
          y0 = add_weighted(y0, f, y.x);
          y1 = add_weighted(y1, f, y.y);
        }
      };
      auto write = [&](int v, int d, float M, float L, float y0, float y1) {
        if (t.slot >= 0) {
          float* part = parts + static_cast<size_t>(t.slot) * kf_slot(HD);
          *reinterpret_cast<float2*>(part + v * HD + d) = make_float2(y0, y1);
          if (d == 0) reinterpret_cast<float2*>(part + KF_QV * HD)[v] = make_float2(L == 0.f ? -INFINITY : M, L);
        } else {
          emit(a, t.row0, t.kvh, v, d, HD, M, L, y0, y1);
        }
      };
      bool odd = false;                      // some sum is NaN where no p is
      for (int x = tid; x < t.qv * (HD / 2); x += 32 * KF_WARPS) {
        const int v = x / (HD / 2), d = 2 * (x - v * (HD / 2));
        float M, L, y0, y1;
        join(v, d, M, L, y0, y1);
        odd |= (isnan(y0) || isnan(y1)) && fabsf(L) < INFINITY;
        write(v, d, M, L, y0, y1);
      }
      // A p or a factor that fell to 0 makes NaN of an infinite value: such sums are written once more.  (No loop
      // over x around the lookup: with one the case above took 54.4 us, whether a lookup ran or not.)
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
        for (int i = 0; i < KF_QV * HD / 2 / (32 * KF_WARPS); ++i) {
          const int x = tid + 32 * KF_WARPS * i, v = x / (HD / 2), d = 2 * (x - v * (HD / 2));
          float M, L, y0, y1, z[2];
          infinities<HD, 2>(a.pool, t.b, t.kvh, begin, t.k0 + t.keys, d, z, lane, a.err);
          join(v, d, M, L, y0, y1);
          if (isnan(y0) && z[0] != 0.f) y0 = z[0];
          if (isnan(y1) && z[1] != 0.f) y1 = z[1];
          if (v < t.qv && fabsf(L) < INFINITY) write(v, d, M, L, y0, y1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_read);
      ++items;
    }
  }
}

// Joins the partial results of the items that the cuts divide: block x the item whose first part is CTA x's.
template <int HD>
__global__ void __launch_bounds__(256) kv_few_join(const KaArgs a, const float* parts) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x;
  const Cut s = reinterpret_cast<const Cut*>(parts)[c];
  if (s.last == 0) return;
  parts += gridDim.x * (sizeof(Cut) / 4);
  for (int x = threadIdx.x; x < s.qv * (HD / 2); x += 256) {
    const int v = x / (HD / 2), d = 2 * (x - v * (HD / 2));
    auto part = [&](int k) { return parts + static_cast<size_t>(k == c ? s.slot : 2 * k) * kf_slot(HD); };
    auto state = [&](int k) { return reinterpret_cast<const float2*>(part(k) + KF_QV * HD)[v]; };
    float M = -INFINITY, L = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 4
    for (int k = c; k <= s.last; ++k) M = max_nan(M, state(k).x);
#pragma unroll 4
    for (int k = c; k <= s.last; ++k) {
      const float2 ml = state(k), y = *reinterpret_cast<const float2*>(part(k) + v * HD + d);
      if (ml.x == -INFINITY) continue;
      const float f = part_factor(ml.x, M);
      L = fmaf(f, ml.y, L);
      y0 = add_weighted(y0, f, y.x);
      y1 = add_weighted(y1, f, y.y);
    }
    emit(a, s.row0, s.kvh, v, d, HD, M, L, y0, y1);
  }
}

template <int HD>
cudaError_t launch_few(const CUtensorMap& tmk, const CUtensorMap& tmv, const KaArgs& a, float* parts, int ctas, cudaStream_t st) {
  static std::atomic<size_t> granted[64];    // shared memory per device, set on its first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  size_t cap = dev < 64 ? granted[dev].load() : 0;
  if (!cap) {
    e = allow_max_smem(reinterpret_cast<const void*>(kv_few<HD>), &cap);
    if (e != cudaSuccess) return e;
    if (dev < 64) granted[dev].store(cap);
  }
  const size_t fixed = kf_states(HD) + KF_MISC;
  const int ns = std::min<int>(KF_MAX_STAGES, static_cast<int>((cap - fixed) / kf_stage(HD)));
  if (cap < fixed || ns < 2) return cudaErrorInvalidConfiguration;
  e = launch_after(false, dim3(ctas), KF_THREADS, fixed + static_cast<size_t>(ns) * kf_stage(HD), st, kv_few<HD>, tmk, tmv, a, parts, ns);
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_after(true, dim3(ctas), 256, 0, st, kv_few_join<HD>, a, static_cast<const float*>(parts));
}

}  // namespace

static double kf_units(int Hkv, int B, int max_len) {
  return static_cast<double>(B) * Hkv * ((static_cast<long long>(max_len) + KF_KEYS - 1) / KF_KEYS);
}
static int kf_sms() { return num_sms() > 0 ? num_sms() : 152; }   // (152: without a device, a GB300's)

// Where the SMs have so many tiles each that even shares count for more than an earlier start.  Measured for 1 to
// 128 sequences of 250 to 80,000 keys: 8 heads of 64, 16 of 2,000 keys a head: 16.8 us, by ranges 20.5 (23 tiles an SM), 32 of
// 300: 16.4, 17.2 (15), 8 of 500: 10.9, 11.0 (6); heads of 128, 4 vectors: 16 of 1,000: 21.5, 23.0 (24), 32 of
// 300: 20.8, 19.4 (15); 8 vectors, whose eight columns are all at work: 32 of 2,000: 55, 60 (93), 128 of 300: 68, 60
// (61).  A step's own keys behind a prefix go by ranges side by side with the prefix's otherwise: 64
// of 500: 69 us, here 75 (50), 256 of 1,000: 317, here 296 (404).
bool eagle::kf_worth(int Hkv, int hd, int qv, int B, int max_len, bool alone) {
  const double least = !alone ? 80. : hd == 64 ? 12. : qv <= 4 ? 20. : 90.;
  return kf_units(Hkv, B, max_len) >= least * kf_sms();
}

KxPlan eagle::kf_plan(int Hkv, int hd, int B, int max_len) {
  const double ctas = kf_units(Hkv, B, max_len) / KF_MIN_UNITS;
  KxPlan p;
  p.ctas = ctas < kf_sms() ? static_cast<int>(ctas) + 1 : kf_sms();
  p.bytes = p.ctas * (static_cast<int64_t>(sizeof(Cut)) + (p.ctas == 1 ? 0 : 8ll * kf_slot(hd)));
  return p;
}

cudaError_t eagle::kf_launch(KaArgs* a, const eagle_kv_cache_t* cache, const KxPlan& p, float* parts, cudaStream_t st) {
  CUtensorMap tmk, tmv;
  const long long blocks = static_cast<long long>(cache->num_pages) * cache->n_kv_heads;
  const int rows = std::min(cache->page_size, KF_KEYS);
  if (!make_page_map(&tmk, cache->k, cache->head_dim, cache->page_size, blocks, rows) ||
      !make_page_map(&tmv, cache->v, cache->head_dim, cache->page_size, blocks, rows))
    return cudaErrorInvalidValue;
  a->splits = 1;                             // (whoever joins the results further finds one range)
  a->tiles_per_cta = 1 << 20;
  a->least = 1;
  return a->pool.hd == 64 ? launch_few<64>(tmk, tmv, *a, parts, p.ctas, st) : launch_few<128>(tmk, tmv, *a, parts, p.ctas, st);
}
