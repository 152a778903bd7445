// Attention of a step's rows over the caller's paged key / value cache (bf16 or 4-bit), with
// the tree mask of an emitted draft tree or causally.  See include/eagle_draft.h.
//
//   s = scale q k,  p = 2^(log2e (s - m)),  l = sum p,  out = (sum p v) / l
//
// All query heads of a KV group and all rows of a request share one pass over the keys: the
// query vectors v = row * G + head of the group fill the 128 TMEM lanes of a tcgen05 tile (one
// or two tiles per CTA).  A CTA takes a range of the keys; the ranges of a request meet in a
// cluster or in a combine kernel (in rank order: deterministic).  Three kernels: tensor cores for
// any shape, mma.sync on 4-bit pages for up to 8 query vectors, and the combine kernel.
#include "kvcache.cuh"

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>

using namespace eagle;

namespace {

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B, f32 D, both K-major (as
// idesc_bf16_f32, whose operands are bf16).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 3-D map over a paged bf16 cache [pages * Hkv][page_size][hd]: boxes of one page's rows of one
// KV head x 64 dims, 128-byte swizzle; rows outside the page or the pool read as zeros.
bool make_page_map(CUtensorMap* tm, const void* pool, int hd, int page_size, long long blocks) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd) * 2, static_cast<cuuint64_t>(hd) * 2 * page_size};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(page_size), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int KA_MAX_GROUP = 64;
constexpr int KA_CH = 128;                 // keys per tile (a ring entry)
constexpr int KA_H = 64;                   // keys per unit of work (half a tile)
constexpr int KA_QV = 128;                 // query vectors per tile (TMEM lanes)
constexpr float KA_RESCALE = 8.0f;         // log2 units: the running maximum may lag by this much
constexpr uint32_t KA_MISC = 2048;         // barriers (0), tree mask rows (512), joined states' m and l (1024)
constexpr int KA_MAX_SLOTS = 14;
constexpr int KA_MAX_JOIN = 8;             // ranges that join in a cluster
constexpr int KA_FIXED = 12;              // a CTA's fixed cost in tiles
constexpr int KS_FIXED = 2;               // the same for the kernel for few query vectors

struct KaArgs {
  KvPool pool;
  int B, N, Hq, G, max_rows, max_len, S;
  int blocks;                              // query-vector blocks per request
  int tiles_per_cta, splits;
  int joined;                              // the ranges of a request are one cluster and join in it
  const int* cu;
  const int* lens;
  const __nv_bfloat16* q;
  long long q_ld;
  const unsigned char* mask;
  float scale_log2;                        // scale * log2(e)
  float vg;                                // the values' global factor (1 with bf16 pages)
  __nv_bfloat16* out;
  long long out_ld;
  float* lse;
  float* part_o;                           // [splits][N][Hq][hd] unnormalised outputs (splits > 1)
  float2* part_ml;                         // [splits][N][Hq] running maximum (log2 units) and sum
  unsigned* err;
};

// Request b's rows and keys, clamped to what the call allows.
struct Req {
  int row0, R, ctx, len;
};
EAGLE_DEV Req request(const KaArgs& a, int b) {
  Req r;
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), l = __ldg(a.lens + b);
  r.row0 = min(max(c0, 0), a.N);
  r.R = min(max(min(c1, a.N) - r.row0, 0), min(a.max_rows, a.max_len));
  r.ctx = min(max(l, 0), a.max_len - r.R);
  if (r.row0 != c0 || r.R != c1 - c0 || r.ctx != l) atomicOr(a.err, DEVERR_PREFIX);
  r.len = r.ctx + r.R;
  return r;
}

EAGLE_DEV void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the float at this CTA's shared address `p` in CTA `rank` of the cluster
EAGLE_DEV float remote(const float* p, int rank) {
  uint32_t a;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
EAGLE_DEV float4 remote4(const float* p, int rank) {
  uint32_t a;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// 128 bits of key visibility
struct Bits {
  unsigned long long lo, hi;
};
EAGLE_DEV Bits bits_below(int n) {         // bits [0, n)
  Bits r;
  r.lo = n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
  r.hi = n >= 128 ? ~0ull : n <= 64 ? 0ull : (1ull << (n - 64)) - 1ull;
  return r;
}
EAGLE_DEV Bits shift_up(unsigned long long m, int n) {   // m << n; n < 0: m >> -n
  Bits r{0ull, 0ull};
  if (n <= -64 || n >= 128) return r;
  if (n < 0) r.lo = m >> -n;
  else if (n == 0) r.lo = m;
  else if (n < 64) { r.lo = m << n; r.hi = m >> (64 - n); }
  else r.hi = m << (n - 64);
  return r;
}

// byte offset of 16-byte chunk c (0-7) of row r in a 128-byte-swizzled block of 128-byte rows
EAGLE_DEV uint32_t ka_sw(int r, int c) {
  return static_cast<uint32_t>((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}
EAGLE_DEV void st_smem16(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// the largest of three, NaN if any is: a NaN score must reach the output
EAGLE_DEV float max3_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// (x, y) * (a, a) + (b, b) and (x, y) + (z, w), two fp32 lanes an instruction
EAGLE_DEV void fma2(float& x, float& y, float a, float b) {
  const float2 r = __ffma2_rn(make_float2(x, y), make_float2(a, a), make_float2(b, b));
  x = r.x;
  y = r.y;
}
EAGLE_DEV void add2(float& x, float& y, float z, float w) {
  const float2 r = __fadd2_rn(make_float2(x, y), make_float2(z, w));
  x = r.x;
  y = r.y;
}
// `bytes` (a multiple of 16) of global memory into shared memory, completing on `bar`
EAGLE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
EAGLE_DEV uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// byte B of w, two e2m1 codes -> fp16 pair (low nibble in the low half)
template <int B>
EAGLE_DEV uint32_t e2m1_pair(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 t<4>;\n\tmov.b32 {t0, t1, t2, t3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t%2;\n\t}" : "=r"(r) : "r"(w), "n"(B));
  return r;
}
EAGLE_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 8 consecutive dims of a cached row: 4 code bytes and the pair of their scale -> 8 fp16 values (exact:
// a code has 2 significant bits and a scale 4; the range is 2^-10 .. 2688)
EAGLE_DEV uint32_t scale_pair(uint32_t scale) {
  uint32_t s;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(s) : "r"(scale * 0x101u));
  return s;
}
EAGLE_DEV void dequant8(uint32_t code, uint32_t s, uint32_t* h) {
  h[0] = mul_f16x2(e2m1_pair<0>(code), s);
  h[1] = mul_f16x2(e2m1_pair<1>(code), s);
  h[2] = mul_f16x2(e2m1_pair<2>(code), s);
  h[3] = mul_f16x2(e2m1_pair<3>(code), s);
}

// A vector's score factor, kept within the normal numbers: a factor that fell to 0 would make NaN of
// a masked score (-inf * 0), one that overflowed of a score of 0.
EAGLE_DEV float finite_scale(float x) { return fminf(fmaxf(x, FLT_MIN), FLT_MAX); }

// a warp-uniform value, in a form that lets the compiler keep what follows from it in uniform
// registers (the operands of tcgen05.mma)
EAGLE_DEV int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// A place in the ring of NS entries: slot and the parity of its turn.  (Stepped, not computed: a
// division by NS costs the MMA warp as much as it takes to issue a unit.)
struct RingPos {
  int slot, turn;
  EAGLE_DEV void step(int n, int NS) {
    slot += n;
    if (slot >= NS) {
      slot -= NS;
      turn ^= 1;
    }
  }
};
// one thread of a converged warp, the same one every time
EAGLE_DEV bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
template <int R>
EAGLE_DEV void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
EAGLE_DEV void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

// The tensor-core kernel.  HD 64 or 128; CACHE the cache kind; NB: query-vector tiles per CTA.
//
// Shared memory is a ring of entries, key tile and value tile in turn (128 rows of 128 bytes per
// 64 dims, 128-byte swizzle).  bf16 pages come by TMA, one box per page and 64 dims; 4-bit pages
// by bulk copies into a ring of raw tiles, which converter warps turn into fp16 tiles.  Q is the A operand of S = Q K^T, in TMEM
// (NB = 1) or shared memory (NB = 2, where S and O of two tiles take all 512 columns); P replaces
// S in TMEM as the A operand of O += P V.  Work goes in units of 64 keys, two S buffers per query
// tile: a unit's QK^T runs while the unit before it is in the softmax, so the softmax warps find
// their scores ready: 1650 cycles a unit and two query tiles, of which the tensor cores need 1280
// (48 for each of 16 QK^T instructions, whose operands both come from shared memory, 64 for each
// of 8 of P V).  One 128-key buffer per query tile, whose QK^T had to wait for the softmax and the
// P V of the same buffer, took 2080; two threads per vector instead of one, 1800.
//
// A page that the keys end inside is loaded from a negative row, so that the copy reads zeros
// and then the valid rows: memory behind the last key never enters a product (it may hold NaN,
// and 0 * NaN would reach O).  The columns of that page are shifted by as much.
//
// P is rounded for the second product: fp16 (11 bits) with 4-bit caches; with bf16 values it
// must be bf16, kept as hi + lo parts (two products) where one query tile leaves the kernel bound
// by bytes, and rounded to 8 bits where two tiles make it bound by the tensor cores: 8 trees of 61
// rows x 64 heads over 4,096 keys take 60 us, with both parts 75, a prompt of 4,096 rows 157 and
// 175; the output is 2.3e-3 of its norm from 64 bits, with both parts 1.7e-3, which is its own
// rounding to bf16.  l sums the unrounded p.
__host__ __device__ constexpr int ka_threads(int cache, int nb) { return 128 + 128 * nb + (cache == EAGLE_CACHE_F4 ? 256 : 0); }
// registers per thread of the 4-bit kernel's roles after they moved (the launch checks their sum)
constexpr int KA_REG_CTRL = 40;
__host__ __device__ constexpr int ka_reg_softmax(int nb) { return nb == 2 ? 136 : 152; }
__host__ __device__ constexpr int ka_reg_conv(int nb) { return nb == 2 ? 80 : 128; }
__host__ __device__ constexpr uint32_t ka_entry(int hd) { return static_cast<uint32_t>(hd) * 2 * KA_CH; }
// 4-bit caches: a ring of raw tiles (128 rows of codes, then their scales) behind the entries
constexpr int KA_RAW = 3;
__host__ __device__ constexpr uint32_t ka_raw_bytes(int hd) { return static_cast<uint32_t>(hd) / 2 * KA_CH + hd / 16 * KA_CH; }

// The keys of a range that one vector sees.
struct VisibleKeys {
  const KvPool& pool;
  int b, kvh, begin, end, ctx, row;
  bool tree;
  unsigned long long bits;                 // tree mask row
  EAGLE_DEV bool see(int k) const {
    const int j = k - ctx;
    return k < end && (j < 0 || (tree ? (bits >> j) & 1ull : j <= row));
  }
};
// sum p v over them by a warp, from bf16 pages: lane l takes dims [l hd / 32, (l + 1) hd / 32).  The rare
// path (non-finite values in the cache), bound by the latency of its loads: 0.9 us a vector and 8 keys
// (15 ms where a request of 61 rows x 64 heads holds an infinite value among 4,096 keys; a thread
// per vector took 277).
template <int HD>
EAGLE_DEV void visible_sum(const VisibleKeys& keys, const __nv_bfloat16* qp, float row_scale, float m, float* o, int lane, unsigned* err) {
  constexpr int E = HD / 32, KB = 8;       // keys in flight (of one page)
  auto load = [&](const __nv_bfloat16* p, float* x) {
    uint32_t w[E / 2];
    if constexpr (E == 4) {
      const uint2 t = *reinterpret_cast<const uint2*>(p + E * lane);
      w[0] = t.x;
      w[1] = t.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p + E * lane);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  };
  float q[E];
  load(qp, q);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  int page = -1;
  for (int k = keys.begin; k < keys.end; k += KB) {   // (begin is a multiple of the page size)
    if ((k & ((1 << keys.pool.ps_log) - 1)) == 0) page = kv_page(keys.pool, keys.b, k, err);
    if (page < 0) continue;                // (reads as zeros)
    const size_t at = kv_row(keys.pool, page, keys.kvh, k) * HD;
    float s[KB], kk[KB][E], vv[KB][E];
#pragma unroll
    for (int i = 0; i < KB; ++i) {         // (the page is there whole: rows nobody sees are read and dropped)
      load(static_cast<const __nv_bfloat16*>(keys.pool.k) + at + i * HD, kk[i]);
      load(static_cast<const __nv_bfloat16*>(keys.pool.v) + at + i * HD, vv[i]);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s[i] = fmaf(q[e], kk[i][e], s[i]);
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) s[i] = warp_sum(s[i]);
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      if (!keys.see(k + i)) continue;
      const float p = fast_exp2(fmaf(s[i], row_scale, -m * row_scale));
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(p, vv[i][e], o[e]);
    }
  }
}

template <int HD, int CACHE, int NB>
__global__ void __launch_bounds__(ka_threads(CACHE, NB), 1)
kv_attention_tc(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const KaArgs a, const int NS) {
  constexpr bool F4 = CACHE == EAGLE_CACHE_F4;
  constexpr bool HILO = !F4 && NB == 1;
  // fp16 p is held times 2^7 (below 2^15): its subnormal step is then 2^-31 of the largest p
  constexpr float LIFT = F4 ? 7.f : 0.f;
  constexpr int THREADS = ka_threads(CACHE, NB);
  constexpr int CONV_WARP = 4 + 4 * NB, CONV = THREADS - 32 * CONV_WARP;   // converter threads (F4)
  constexpr uint32_t ENTRY = ka_entry(HD), HALF = KA_CH * 128, RAW = ka_raw_bytes(HD), RAW_SCALES = HD / 2 * KA_CH;
  constexpr uint32_t T_O = 256, T_Q = 384;
  extern __shared__ uint8_t ka_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ka_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t ring_u = uniform(smem_u32(sm));
  const uint32_t q_u = ring_u + static_cast<uint32_t>(NS) * ENTRY;       // NB = 2: Q tiles
  uint8_t* raw = sm + static_cast<uint32_t>(NS) * ENTRY + (NB == 2 ? 2 * ENTRY : 0);   // F4: raw tiles
  uint8_t* misc = raw + (F4 ? KA_RAW * RAW : 0);
  const uint32_t misc_u = smem_u32(misc);
  const uint32_t bar_kvf = misc_u, bar_kve = misc_u + 112, bar_sf = misc_u + 224, bar_pf = misc_u + 256,
                 bar_pe = misc_u + 288, bar_q = misc_u + 320, bar_fin = misc_u + 336;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 344);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 348);
  const uint32_t bar_rf = misc_u + 352, bar_re = misc_u + 408;            // raw tiles full / free
  volatile uint32_t* raw_pages = reinterpret_cast<volatile uint32_t*>(misc + 464);   // pages each holds (bits)
  float* mcta = reinterpret_cast<float*>(misc + 1024);   // [128] joined: this CTA's maximum per vector, its sum
  float* lcta = mcta + KA_QV;
  float* state = reinterpret_cast<float*>(sm);           // [128][HD + 4] joined: its output (in the ring, at the end)
  constexpr int ST_LD = HD + 4;
  unsigned long long* rowbits = reinterpret_cast<unsigned long long*>(misc + 512);   // [64] tree mask rows

  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z / a.blocks, blk0 = blockIdx.z - b * a.blocks;
  pdl_trigger();                             // (the combine kernel may start and wait)
  Req rq = request(a, b);
  rq.row0 = uniform(rq.row0);
  rq.R = uniform(rq.R);
  rq.ctx = uniform(rq.ctx);
  rq.len = uniform(rq.len);
  const int v0 = blk0 * KA_QV * NB;
  const int qv = min(rq.R * a.G - v0, KA_QV * NB);
  if (qv <= 0) return;
  const int i_first = v0 / a.G, i_last = (v0 + qv - 1) / a.G;
  // keys this block can see, and this CTA's tiles of them
  const int seen = a.mask ? rq.len : min(rq.len, rq.ctx + i_last + 1);
  const int all_tiles = (seen + KA_CH - 1) / KA_CH;
  // (a cluster shares the tiles there are; separate ranges are cut by the call's bounds)
  const bool joined = NB == 1 && a.joined;
  const int per_cta = joined ? (all_tiles + a.splits - 1) / a.splits : a.tiles_per_cta;
  const int t_begin = split * per_cta;
  if (!joined && t_begin * KA_CH >= rq.len) return;  // (not a range of this request at all)
  const int T = max(0, min(all_tiles - t_begin, per_cta));
  const int nb = uniform(NB == 2 && qv > KA_QV ? 2 : 1);
  const int nq0 = min(4, (min(qv, KA_QV) + 31) / 32), nq1 = nb == 2 ? (qv - KA_QV + 31) / 32 : nq0;
  const int ps = 1 << a.pool.ps_log;
  // the page that the request's keys end inside: its rows sit at the end of the box (bf16)
  const int end_page = rq.len >> a.pool.ps_log, end_rows = F4 ? 0 : rq.len & (ps - 1);
  // units of 64 columns (none when this range lies behind what the block sees)
  const int columns = end_rows && (end_page << a.pool.ps_log) < seen ? (end_page + 1) << a.pool.ps_log : seen;
  const int W = uniform(min(2 * T, (columns - t_begin * KA_CH + KA_H - 1) / KA_H));

  if (tid == 0) {
    for (int s = 0; s < KA_MAX_SLOTS; ++s) {
      mbar_init(bar_kvf + 8 * s, F4 ? CONV / 32 : 1);
      mbar_init(bar_kve + 8 * s, nb);
    }
    for (int i = 0; i < 4; ++i) {              // query tile i >> 1, buffer i & 1
      mbar_init(bar_sf + 8 * i, 1);
      mbar_init(bar_pf + 8 * i, i < 2 ? nq0 : nq1);
      mbar_init(bar_pe + 8 * i, 1);
    }
    mbar_init(bar_fin, nb);
    mbar_init(bar_q, 4 * nb);
    for (int s = 0; F4 && s < KA_RAW; ++s) {
      mbar_init(bar_rf + 8 * s, 1);
      mbar_init(bar_re + 8 * s, F4 ? CONV / 32 : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // tree mask rows of this block's rows as 64-bit words
  if (a.mask) {
    for (int i = i_first + warp; i <= i_last; i += THREADS / 32) {
      const unsigned char* mrow = a.mask + (static_cast<size_t>(b) * a.S + i) * a.S;
      const unsigned lo = __ballot_sync(0xffffffffu, lane < rq.R && __ldg(mrow + min(lane, a.S - 1)) != 0);
      const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < rq.R && __ldg(mrow + min(lane + 32, a.S - 1)) != 0);
      if (lane == 0) rowbits[i - i_first] = lo | (static_cast<unsigned long long>(hi) << 32);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);

  auto box_row = [&](int pi) { return pi == end_page && end_rows ? end_rows - ps : 0; };

  // queries: thread = vector; bf16 as they are, or fp16 scaled by a power of two so that the
  // vector's largest magnitude lies in [2^14, 2^15) (8 significant bits always fit)
  float row_scale = a.scale_log2 * (F4 ? a.pool.kg : 1.f);
  if (warp >= 4 && warp < 4 + 4 * nb) {
    const int g = (warp - 4) >> 2, lv = tid - 128 - 128 * g, v = v0 + KA_QV * g + lv;
    const bool live = KA_QV * g + lv < qv;
    const uint4* src = nullptr;
    if (live) {
      const int i = v / a.G;
      src = reinterpret_cast<const uint4*>(a.q + (rq.row0 + i) * a.q_ld + static_cast<long long>(kvh * a.G + v - i * a.G) * HD);
    }
    float up = 1.f;
    if (F4 && live) {
      uint32_t top = 0;
#pragma unroll 4
      for (int c = 0; c < HD / 8; ++c) {
        const uint4 x = __ldg(src + c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      int ex = static_cast<int>(top >> 7);              // biased exponent of the largest magnitude
      ex = ex == 255 ? 127 : max(ex, 30);               // (infinities and NaN pass; tiny vectors)
      up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23);
      row_scale = finite_scale(row_scale * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23));
    }
#pragma unroll 1
    for (int c0 = 0; c0 < HD / 8; c0 += 4) {            // 32 dims: 16 packed columns
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
      if (NB == 1) {
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(w[e]);
        tmem_st16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + T_Q + 4 * c0, f);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          st_smem16(q_u + g * ENTRY + ((c0 + c) >> 3) * HALF + ka_sw(lv, (c0 + c) & 7), w + 4 * c);
      }
    }
    if (NB == 1) tmem_wait_st();
    else fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_q);       // (the producer's copies are under way meanwhile)
  }
  // Registers move from the control and converter warps to the softmax warps, whose threads hold
  // 64 scores (each role's branch opens with its share; the shares stay within what the launch
  // gave the CTA).
  constexpr bool MOVE = F4;
  bool ok = true;
  if (warp < 4) {
    if constexpr (MOVE) set_regs_down<KA_REG_CTRL>();
    // ------------------------------------------------------------ producer: lane = page of the tile
    if (warp == 0) {
      const uint64_t pol = policy_evict_first();
      const int per = KA_CH >> a.pool.ps_log;
      RingPos rp{0, 0};
      const int slots = F4 ? KA_RAW : NS;
      int page = -1;
      for (int e = 0; e < 2 * T; ++e, rp.step(1, slots)) {
        const int slot = rp.slot;
        const int pi = (t_begin + (e >> 1)) * per + lane;
        if (!(e & 1)) {   // the tile's keys and values are in the same pages
          page = -1;
          if (lane < per && (pi << a.pool.ps_log) < rq.len) page = kv_page(a.pool, b, pi << a.pool.ps_log, a.err);
        }
        const uint32_t bar = (F4 ? bar_rf : bar_kvf) + 8 * slot;
        if (e >= slots) ok = mbar_wait_sleepy((F4 ? bar_re : bar_kve) + 8 * slot, rp.turn ^ 1, a.err, abort_flag);
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
            const size_t row = kv_row(a.pool, page, kvh, 0);
            const uint32_t dst = smem_u32(raw + slot * RAW);
            bulk_load(dst + lane * codes, static_cast<const uint8_t*>(e & 1 ? a.pool.v : a.pool.k) + row * (HD / 2), codes, bar);
            bulk_load(dst + RAW_SCALES + lane * scales, static_cast<const uint8_t*>(e & 1 ? a.pool.vs : a.pool.ks) + row * (HD / 16), scales, bar);
          }
        } else {
          if (lane == 0) mbar_arrive_expect_tx(bar, ENTRY);
          __syncwarp();
          if (lane < per) {   // (a page that is not there reads as zeros: a block outside the map)
            const int blk = page >= 0 ? page * a.pool.Hkv + kvh : a.pool.num_pages * a.pool.Hkv;
            const uint32_t dst = ring_u + slot * ENTRY + lane * (ps * 128);
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) tma_load_3d(dst + h * HALF, e & 1 ? &tmv : &tmk, 64 * h, box_row(pi), blk, bar, pol);
          }
        }
      }
      if (!ok) {   // let copies already issued land before the CTA releases its shared memory
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
      }
    }
    // ------------------------------------------------------------ MMA issuer
    // One thread per query tile walks the units and issues; nothing in the loop divides or votes,
    // since every hundred cycles here are a hundred of the tensor cores' idle time.  (One thread
    // for both tiles: 1.26 us per 64 keys.)
    if (warp >= 2 && warp - 2 < nb && elect_one()) {
      const int g = warp - 2;
      const uint32_t id1 = F4 ? idesc_f16_f32(128, KA_H) : idesc_bf16_f32(128, KA_H);
      const uint32_t id2 = (F4 ? idesc_f16_f32(128, HD) : idesc_bf16_f32(128, HD)) | (1u << 16);   // B (values) MN-major
      const uint64_t dq = smem_desc_sw128(q_u + g * ENTRY);
      const uint32_t tO = tmem + T_O + 128 * g;
      ok = mbar_wait(bar_q, 0, a.err, abort_flag);
      tc_fence_after();
      RingPos kp{0, 0}, vp{1, 0};            // the key tile of unit w, the value tile of unit w - 1
      for (int w = 0; w <= W && ok; ++w) {
        if (w < W) {
          // S = Q K^T of unit w, once P V of unit w - 2 (same buffer) is done
          const int buf = 2 * g + (w & 1);
          if (!(w & 1)) ok = mbar_wait(bar_kvf + 8 * kp.slot, kp.turn, a.err, abort_flag);
          ok = ok && mbar_wait(bar_pe + 8 * buf, ((w >> 1) & 1) ^ 1, a.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * KA_H;
          const uint64_t dk = smem_desc_sw128(ring_u + kp.slot * ENTRY + (w & 1) * (KA_H * 128));
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const uint32_t ko = ((j >> 2) * HALF + (j & 3) * 32) >> 4;
            if (NB == 1) tc_mma_bf16_ta(d, tmem + T_Q + 8 * j, dk + ko, id1, j > 0 ? 1u : 0u);
            else tc_mma_bf16(d, dq + ko, dk + ko, id1, j > 0 ? 1u : 0u);
          }
          tc_commit(bar_sf + 8 * buf);
          if ((w & 1) || w == W - 1) {
            tc_commit(bar_kve + 8 * kp.slot);
            kp.step(2, NS);
          }
        }
        if (w > 0) {   // O += P V of unit x
          const int x = w - 1, buf = 2 * g + (x & 1);
          if (!(x & 1)) ok = mbar_wait(bar_kvf + 8 * vp.slot, vp.turn, a.err, abort_flag);
          ok = ok && mbar_wait(bar_pf + 8 * buf, (x >> 1) & 1, a.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = smem_desc_sw128_mn(ring_u + vp.slot * ENTRY + (x & 1) * (KA_H * 128), HALF, 1024);
          const uint32_t tp = tmem + buf * KA_H;
#pragma unroll
          for (int j = 0; j < KA_H / 16; ++j) {
            const uint32_t first = (x > 0 || j > 0) ? 1u : 0u;
            if (HILO) {   // keys [32 c, 32 c + 32): 16 hi columns at 32 c, 16 lo columns behind
              const uint32_t pa = tp + 32 * (j >> 1) + 8 * (j & 1);
              tc_mma_bf16_ta(tO, pa, dv + j * 128, id2, first);
              tc_mma_bf16_ta(tO, pa + 16, dv + j * 128, id2, 1u);
            } else {
              tc_mma_bf16_ta(tO, tp + 8 * j, dv + j * 128, id2, first);
            }
          }
          tc_commit(bar_pe + 8 * buf);
          if ((x & 1) || x == W - 1) {
            tc_commit(bar_kve + 8 * vp.slot);
            vp.step(2, NS);
          }
        }
      }
      if (!ok) {   // let MMAs already issued finish before TMEM is released
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
        }
      }
      // (a range behind all its block sees has no tile: nothing to commit, and nobody waits, so an
      // arrival could land after the CTA has left)
      if (T > 0) tc_commit(bar_fin);
    }
  } else if (warp >= CONV_WARP) {
    if constexpr (F4) {
    set_regs_down<ka_reg_conv(NB)>();
    // ------------------------------ raw tiles -> fp16 tiles: 16 dims per thread and step
    constexpr int GR = HD / 16;                        // scale groups per row
    constexpr int IT = KA_CH * GR / CONV;              // 16-dim groups per thread and entry
    constexpr int RSTEP = CONV / GR;
    static_assert(RSTEP % 8 == 0, "the swizzle repeats every 8 rows");
    const int ct = tid - 32 * CONV_WARP, gidx = ct % GR, r0 = ct / GR;
    const int sw = gidx >> 2;   // (the two 64-dim halves share banks: the upper one stores its chunks in the other order)
    RingPos rp{0, 0}, wp{0, 0};
    for (int e = 0; e < 2 * T; ++e, rp.step(1, NS), wp.step(1, KA_RAW)) {
      ok = mbar_wait_sleepy(bar_rf + 8 * wp.slot, wp.turn, a.err, abort_flag);
      const uint8_t* src = raw + wp.slot * RAW;
      const uint32_t have = raw_pages[wp.slot];
      const int k0 = (t_begin + (e >> 1)) * KA_CH;
      uint2 code[IT];
      uint32_t scale[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int r = r0 + i * RSTEP;
        code[i] = reinterpret_cast<const uint2*>(src + r * (HD / 2))[gidx];
        scale[i] = src[RAW_SCALES + r * GR + gidx];
      }
      if (k0 + KA_CH > rq.len || have != (1u << (KA_CH >> a.pool.ps_log)) - 1u) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {       // rows behind the last key, and of pages that are not there: zeros
          const int r = r0 + i * RSTEP;
          if (k0 + r >= rq.len || !((have >> (r >> a.pool.ps_log)) & 1u)) {
            code[i] = make_uint2(0u, 0u);
            scale[i] = 0u;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_re + 8 * wp.slot);
      if (e >= NS) ok = mbar_wait_sleepy(bar_kve + 8 * rp.slot, rp.turn ^ 1, a.err, abort_flag) && ok;
      if (__any_sync(0xffffffffu, !ok)) break;
      // (rows r0 + i RSTEP share their place in the swizzle: RSTEP is a multiple of 8)
      const uint32_t dst = ring_u + rp.slot * ENTRY + sw * HALF, c = 2 * (gidx & 3);
      const uint32_t d0 = dst + ka_sw(r0, c + sw), d1 = dst + ka_sw(r0, c + (sw ^ 1));
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const uint32_t s = scale_pair(scale[i]);
        uint32_t h[4];
        dequant8(sw ? code[i].y : code[i].x, s, h);
        st_smem16(d0 + i * (RSTEP * 128), h);
        dequant8(sw ? code[i].x : code[i].y, s, h);
        st_smem16(d1 + i * (RSTEP * 128), h);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_kvf + 8 * rp.slot);
    }
    }
  } else {
    if constexpr (MOVE) set_regs_up<ka_reg_softmax(NB)>();
    // ------------------------------------------------------------ softmax
    const int g = (warp - 4) >> 2, lv = tid - 128 - 128 * g, v = v0 + KA_QV * g + lv;
    const bool live = KA_QV * g + lv < qv;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int irow = live ? v / a.G : i_last;
    const unsigned long long tree_bits = a.mask && live ? rowbits[irow - i_first] : 0ull;
    const uint32_t tO = tmem + lane_base + T_O + 128 * g;
    float m_run = -INFINITY, l_run = 0.f;              // raw scores' maximum; sum of p
    if (g < nb && (warp & 3) < (g == 0 ? nq0 : nq1)) {
      for (int w = 0; w < W; ++w) {
        const int buf = 2 * g + (w & 1);
        ok = ok && mbar_wait(bar_sf + 8 * buf, (w >> 1) & 1, a.err, abort_flag);
        tc_fence_after();
        const uint32_t ts = tmem + lane_base + buf * KA_H;
        // the row's scores stay in registers from the maximum to the probabilities
        float s[KA_H];
        tmem_ld32(ts, s);
        tmem_ld32(ts + 32, s + 32);
        // columns this vector sees; keys k0, k0 + 1, ... but for the shifted last page
        const int k0 = t_begin * KA_CH + w * KA_H;
        const int kt = k0 & ~(KA_CH - 1), off = rq.ctx - kt;   // the tile; its column of the first own row
        unsigned long long vis = ~0ull;
        if (off < KA_CH) {
          Bits seen_cols;
          if (a.mask) {
            const Bits own = shift_up(tree_bits, off);
            seen_cols = bits_below(off);
            seen_cols.lo |= own.lo;
            seen_cols.hi |= own.hi;
          } else {
            seen_cols = bits_below(off + irow + 1);
          }
          const int at = (end_page << a.pool.ps_log) - kt, sh = ps - end_rows;   // the last page's first column
          if (end_rows && at >= 0 && at < KA_CH) {   // columns from `at` on move up by sh (1 .. 127)
            const Bits below = bits_below(at);
            const unsigned long long mlo = seen_cols.lo & ~below.lo, mhi = seen_cols.hi & ~below.hi;
            const unsigned long long ulo = sh < 64 ? mlo << sh : 0ull;
            const unsigned long long uhi = sh < 64 ? (mhi << sh) | (mlo >> (64 - sh)) : mlo << (sh - 64);
            seen_cols.lo = (seen_cols.lo & below.lo) | ulo;
            seen_cols.hi = (seen_cols.hi & below.hi) | uhi;
          }
          vis = w & 1 ? seen_cols.hi : seen_cols.lo;
        }
        tmem_wait_ld();
        if (vis != ~0ull) {
#pragma unroll
          for (int e = 0; e < KA_H; ++e) s[e] = (vis >> e) & 1ull ? s[e] : -INFINITY;
        }
        float m8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) m8[e] = max_nan(s[e], s[e + 8]);
#pragma unroll
        for (int e = 16; e < KA_H; e += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) m8[k] = max3_nan(m8[k], s[e + k], s[e + 8 + k]);
        const float mt = max_nan(max3_nan(max3_nan(m8[0], m8[1], m8[2]), m8[3], m8[4]), max3_nan(m8[5], m8[6], m8[7]));
        float f = 1.f;
        bool resc = false;
        if (mt != -INFINITY) {
          if (m_run == -INFINITY) {
            m_run = mt;
          } else if ((mt - m_run) * row_scale > KA_RESCALE) {
            f = fast_exp2((m_run - mt) * row_scale);
            m_run = mt;
            resc = true;
          }
        }
        if (__any_sync(0xffffffffu, resc)) {
          // rows whose maximum rose: scale them in O once the earlier P V are done
          ok = ok && mbar_wait(bar_pe + 8 * (buf ^ 1), ((w - 1) >> 1) & 1, a.err, abort_flag);
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < HD; c0 += 32) {
            float x[32];
            tmem_ld32(tO + c0, x);
            tmem_wait_ld();
            uint32_t y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(x[e] * f);
            tmem_st32(tO + c0, y);
          }
          tmem_wait_st();
        }
        l_run *= f;
        // a row without a key so far takes the maximum as 0: every score is -inf, every p is 0
        // (lanes past the last vector hold scores of 0 and are never read)
        const float mb = (m_run == -INFINITY ? 0.f : m_run * row_scale) - LIFT;
        float p8[8] = {};
#pragma unroll
        for (int c = 0; c < KA_H; c += 32) {
#pragma unroll
          for (int e = c; e < c + 32; e += 2) {
            fma2(s[e], s[e + 1], row_scale, -mb);
            s[e] = fast_exp2(s[e]);
            s[e + 1] = fast_exp2(s[e + 1]);
            add2(p8[e & 7], p8[(e & 7) + 1], s[e], s[e + 1]);
          }
          if (HILO) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 16; ++e) split2_packed(s[c + 2 * e], s[c + 2 * e + 1], pk[e], pk[16 + e]);
            tmem_st32(ts + c, pk);
          } else {
            float pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = __uint_as_float(F4 ? pack_f16(s[c + 2 * e], s[c + 2 * e + 1]) : pack_bf16(s[c + 2 * e], s[c + 2 * e + 1]));
            tmem_st16(ts + c / 2, pk);
          }
        }
        l_run += ((p8[0] + p8[1]) + (p8[2] + p8[3])) + ((p8[4] + p8[5]) + (p8[6] + p8[7]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_pf + 8 * buf);
      }
      // ---- this CTA's result of vector v
      if (T > 0) ok = mbar_wait_sleepy(bar_fin, 0, a.err, abort_flag) && ok;
      tc_fence_after();
      const int n = rq.row0 + irow, h = kvh * a.G + (v - irow * a.G);
      const size_t at = static_cast<size_t>(n) * a.Hq + h;
      const bool none = l_run == 0.f;
      const float inv = none ? 0.f : a.vg / l_run;
      // A non-finite V reaches vectors that have nothing of it: in a row that the step masks as 0 *
      // NaN, and with p in two parts the lower part (0 or negative) makes NaN of a visible infinity.
      // Such sums are formed again from the visible keys alone, a vector at a time by the whole warp
      // (unless the vector's own sum of p is NaN: then so is its output), and written once more.
      const bool recheck = !F4 && T > 0 && (HILO || (t_begin + T) * KA_CH > rq.ctx);
      for (bool again = false;; again = true) {
        float2 z0 = make_float2(0.f, 0.f), z1 = z0;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 32) {
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0.f;
          if (T > 0) {
            tmem_ld32(tO + c0, x);
            tmem_wait_ld();
          }
          if (!F4) {                           // (0 unless some sum is not finite)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              z0 = __ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(0.f, 0.f), z0);
              z1 = __ffma2_rn(make_float2(x[e + 2], x[e + 3]), make_float2(0.f, 0.f), z1);
            }
          }
          if (joined) {
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(state + lv * ST_LD + c0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
          } else if (live && a.splits > 1) {
            if (!none) {
              float4* dst = reinterpret_cast<float4*>(a.part_o + (static_cast<size_t>(split) * a.N * a.Hq + at) * HD + c0);
#pragma unroll
              for (int e = 0; e < 8; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
          } else if (live) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + n * a.out_ld + static_cast<long long>(h) * HD + c0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = none ? 0u : pack_bf16(x[8 * e + 2 * k] * inv, x[8 * e + 2 * k + 1] * inv);
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();                        // (the next TMEM load is the whole warp's)
        }
        if (again || !recheck) break;
        const bool bad = !((z0.x + z0.y) + (z1.x + z1.y) == 0.f);
        unsigned todo = __ballot_sync(0xffffffffu, bad && live && !none && l_run < INFINITY);
        if (!todo) break;
        for (; todo; todo &= todo - 1) {
          const int u = __ffs(todo) - 1, ui = __shfl_sync(0xffffffffu, irow, u);
          const VisibleKeys keys{a.pool, b, kvh, t_begin * KA_CH, min(rq.len, (t_begin + T) * KA_CH), rq.ctx, ui,
                                 a.mask != nullptr, __shfl_sync(0xffffffffu, tree_bits, u)};
          const __nv_bfloat16* qp = a.q + (rq.row0 + ui) * a.q_ld + static_cast<long long>(kvh * a.G + v - lane + u - ui * a.G) * HD;
          float o[HD / 32];
          visible_sum<HD>(keys, qp, row_scale, __shfl_sync(0xffffffffu, m_run, u), o, lane, a.err);
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 32) {   // (the other lanes' sums go back as they were)
            float x[32];
            __syncwarp();
            tmem_ld32(tO + c0, x);
            tmem_wait_ld();
            uint32_t y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float mine = __shfl_sync(0xffffffffu, o[(c0 + e) % (HD / 32)], (c0 + e) / (HD / 32));
              y[e] = __float_as_uint(lane == u ? mine : x[e]);
            }
            tmem_st32(tO + c0, y);
          }
          tmem_wait_st();
        }
      }
      if (live) {
        const float m2 = none ? -INFINITY : m_run * row_scale - LIFT;
        if (joined) {
          mcta[lv] = m2;
          lcta[lv] = l_run;
        } else if (a.splits > 1) a.part_ml[static_cast<size_t>(split) * a.N * a.Hq + at] = make_float2(m2, l_run);
        else if (a.lse) a.lse[at] = none ? -INFINITY : (m2 + log2f(l_run)) * 0.6931471805599453f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (joined) {   // the cluster's ranges, in rank order
    cluster_sync();
    for (int x = split * THREADS + tid; x < qv * (HD / 4); x += a.splits * THREADS) {
      const int v = x / (HD / 4), d = 4 * (x - v * (HD / 4));
      float m[KA_MAX_JOIN], M = -INFINITY;
#pragma unroll
      for (int r = 0; r < KA_MAX_JOIN; ++r) {
        m[r] = r < a.splits ? remote(mcta + v, r) : -INFINITY;
        M = max_nan(M, m[r]);
      }
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < KA_MAX_JOIN; ++r) {
        if (m[r] == -INFINITY) continue;     // (a range without a key of this vector)
        const float f = M == INFINITY ? (m[r] == INFINITY ? 1.f : 0.f) : exp2f(m[r] - M);
        const float4 y = remote4(state + v * ST_LD + d, r);
        L = fmaf(f, remote(lcta + v, r), L);
        o.x = fmaf(f, y.x, o.x);
        o.y = fmaf(f, y.y, o.y);
        o.z = fmaf(f, y.z, o.z);
        o.w = fmaf(f, y.w, o.w);
      }
      const bool none = L == 0.f;
      const float inv = none ? 0.f : a.vg / L;
      const int i = (v0 + v) / a.G, n = rq.row0 + i, h = kvh * a.G + (v0 + v - i * a.G);
      *reinterpret_cast<uint2*>(a.out + n * a.out_ld + static_cast<long long>(h) * HD + d) =
          none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      if (d == 0 && a.lse) a.lse[static_cast<size_t>(n) * a.Hq + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    cluster_sync();                          // (the others' shared memory stays until it is read)
  }
}

// ------------------------------------------------------------------ few query vectors, 4 bits
// Up to 8 query vectors per KV head (a token of each of 8 grouped heads).  The tensor-core kernel
// above spends 128 rows of MMA and a decoded copy of every key in shared memory on them; here the
// 4-bit keys go from their raw tiles to registers and mma.sync fragments:
//   S^T [16 keys x 8 vectors] = K Q^T        A = keys, B = queries
//   O^T [16 dims x 8 vectors] += V^T P^T     A = values, B = P (an 8 x 8 transpose of S^T's tile)
// Any order of the dims serves S as long as Q has the same, and any order serves O, so a lane takes
// the dims that lie together in memory: lane (g, c) = (lane / 4, lane % 4) holds dims
// [c hd / 4, (c + 1) hd / 4) of two keys of K, and dims [g hd / 8, (g + 1) hd / 8) of four keys of
// V.  A value pair of two keys is one byte of two codes (two bit operations on four pairs), one
// conversion and one product with the pair of scales.
// One warp copies raw tiles of 128 keys (18 KB at hd 128: codes and scales of K and V) into a ring
// by bulk copies; four warps take 32 keys of a tile each.  The bytes (144 per key and head of 128)
// would take 80 us at 32 requests of 14,700 keys on average and 8 heads, the copies alone take 94;
// it takes 130 (62% of the measured bandwidth): three computing warps a scheduler, each in order
// through load, scores, softmax and P V, issue in 0.59 of the cycles and mostly wait for fixed
// latencies.  Loading the fragments straight from global memory left too few bytes in flight (176
// us); eight warps of 16 keys took 152 us, with 3 CTAs per SM 197.
constexpr int KS_WARPS = 4;
constexpr int KS_KEYS = 32;                // keys of a warp's step
constexpr int KS_QV = 8;
constexpr int KS_CTAS = 3;                 // per SM
constexpr int KS_STAGES = 4;
__host__ __device__ constexpr uint32_t ks_stage(int hd) { return 2 * ka_raw_bytes(hd); }

EAGLE_DEV void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
EAGLE_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// two e4m3 bytes (low half of x) -> fp16 pair
EAGLE_DEV uint32_t e4m3_pair(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
template <int W>
EAGLE_DEV void load_words(uint32_t* d, const uint8_t* p) {
  if constexpr (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    d[0] = x.x; d[1] = x.y;
  } else {
    d[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int HD>
__global__ void __launch_bounds__(32 * KS_WARPS + 32, KS_CTAS) kv_attention_step_f4(const KaArgs a) {
  constexpr int KW = HD / 32, VW = HD / 64, ST = HD / 16;      // words of a lane's K row, V row; 16-dim steps
  constexpr uint32_t RAW = ka_raw_bytes(HD), SCALES = HD / 2 * KA_CH;   // a tensor's part of a stage; its scales
  extern __shared__ __align__(128) uint8_t ks_raw[];           // [KS_STAGES][K | V][codes | scales]
  __shared__ __align__(8) uint64_t s_full[KS_STAGES], s_free[KS_STAGES];
  __shared__ uint32_t s_pages[KS_STAGES];
  __shared__ int s_abort;
  __shared__ float s_m[KS_WARPS][KS_QV], s_l[KS_WARPS][KS_QV], s_jm[KS_QV], s_jl[KS_QV];
  __shared__ unsigned long long s_bits[KS_QV];
  float (*s_o)[HD][KS_QV] = reinterpret_cast<float (*)[HD][KS_QV]>(ks_raw);   // (after the last tile)
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_trigger();
  const Req rq = request(a, b);
  const int qv = rq.R * a.G;
  const int per_cta = a.joined ? ((rq.len + KA_CH - 1) / KA_CH + a.splits - 1) / a.splits : a.tiles_per_cta;
  const int kb = split * per_cta * KA_CH;
  if (qv <= 0 || (!a.joined && kb >= rq.len)) return;
  const int ke = min(rq.len, kb + per_cta * KA_CH);
  const int tiles = max(0, (ke - kb + KA_CH - 1) / KA_CH);
  if (tid == 0) {
    for (int i = 0; i < KS_STAGES; ++i) {
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(s_free + i), KS_WARPS);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  if (a.mask) {                              // the step's visibility per query vector
    for (int v = warp; v < qv; v += KS_WARPS + 1) {
      const unsigned char* mrow = a.mask + (static_cast<size_t>(b) * a.S + v / a.G) * a.S;
      const unsigned lo = __ballot_sync(0xffffffffu, lane < rq.R && __ldg(mrow + min(lane, a.S - 1)) != 0);
      if (lane == 0) s_bits[v] = lo;         // (at most 8 rows)
    }
  }
  __syncthreads();
  bool ok = true;
  if (warp == KS_WARPS) {
    // ------------------------------------------------------------ producer: lane = page of the tile
    const int ps = 1 << a.pool.ps_log, per = KA_CH >> a.pool.ps_log;
    const uint32_t codes = static_cast<uint32_t>(ps) * (HD / 2), scales = static_cast<uint32_t>(ps) * (HD / 16);
    RingPos rp{0, 0};
    for (int t = 0; t < tiles; ++t, rp.step(1, KS_STAGES)) {
      const int k = kb + t * KA_CH + (lane << a.pool.ps_log);
      int page = -1;
      if (lane < per && k < ke) page = kv_page(a.pool, b, k, a.err);
      if (t >= KS_STAGES) ok = mbar_wait_sleepy(smem_u32(s_free + rp.slot), rp.turn ^ 1, a.err, &s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t have = __ballot_sync(0xffffffffu, page >= 0), bar = smem_u32(s_full + rp.slot);
      if (lane == 0) {
        s_pages[rp.slot] = have;
        mbar_arrive_expect_tx(bar, __popc(have) * 2 * (codes + scales));
      }
      __syncwarp();
      if (page >= 0) {
        const size_t row = kv_row(a.pool, page, kvh, 0);
        const uint32_t dst = smem_u32(ks_raw) + rp.slot * ks_stage(HD) + lane * codes, dss = smem_u32(ks_raw) + rp.slot * ks_stage(HD) + SCALES + lane * scales;
        bulk_load(dst, static_cast<const uint8_t*>(a.pool.k) + row * (HD / 2), codes, bar);
        bulk_load(dss, static_cast<const uint8_t*>(a.pool.ks) + row * (HD / 16), scales, bar);
        bulk_load(dst + RAW, static_cast<const uint8_t*>(a.pool.v) + row * (HD / 2), codes, bar);
        bulk_load(dss + RAW, static_cast<const uint8_t*>(a.pool.vs) + row * (HD / 16), scales, bar);
      }
    }
    if (!ok) {   // let copies already issued land before the CTA releases its shared memory
      const long long t0 = clock64();
      while (clock64() - t0 < 4000000) {
      }
    }
  }

  float o[ST][4];
#pragma unroll
  for (int j = 0; j < ST; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // log2 units; sums over this lane's keys
  if (warp < KS_WARPS) {
  // this lane's part of query vector g as fp16, scaled by a power of two (as in the kernel above)
  uint32_t q[ST][2];
  float up_scale = 0.f;
  {
    const bool live = g < qv;
    const int i = g / a.G;
    const uint2* src = reinterpret_cast<const uint2*>(a.q + (rq.row0 + (live ? i : 0)) * a.q_ld +
                                                      static_cast<long long>(kvh * a.G + (live ? g - i * a.G : 0)) * HD + c * (HD / 4));
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      const uint2 x = live ? __ldg(src + s) : make_uint2(0u, 0u);
      q[s][0] = x.x;
      q[s][1] = x.y;
      top = max(max(top, max(x.x & 0x7fffu, (x.x >> 16) & 0x7fffu)), max(x.y & 0x7fffu, (x.y >> 16) & 0x7fffu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    int ex = static_cast<int>(top >> 7);
    ex = ex == 255 ? 127 : max(ex, 30);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23);
    up_scale = finite_scale(a.scale_log2 * a.pool.kg * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23));
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q[s][h] = pack_f16(__uint_as_float(q[s][h] << 16) * up, __uint_as_float(q[s][h] & 0xFFFF0000u) * up);
  }
  // score factors of vectors 2c and 2c + 1 (the columns this lane holds of S^T)
  const float sc0 = __shfl_sync(0xffffffffu, up_scale, 8 * c), sc1 = __shfl_sync(0xffffffffu, up_scale, 8 * c + 4);

  // Which key of a 16-key group is row k of the fragments: an order in which neighbouring rows of K
  // and the four rows of a V load fall on different banks as far as 64-byte rows can.
  const int kr = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;        // row g of K (and + 8)
  const int vr0 = c, vr1 = 4 + (c ^ 1);                        // rows 2c, 2c + 1 of V (and + 8)
  RingPos rp{0, 0};
  for (int t = 0; t < tiles; ++t, rp.step(1, KS_STAGES)) {
    const int k0 = kb + t * KA_CH + warp * KS_KEYS;
    ok = ok && mbar_wait(smem_u32(s_full + rp.slot), rp.turn, a.err, &s_abort);
    const uint8_t* st = ks_raw + rp.slot * ks_stage(HD);
    uint32_t kw[2][2][KW], kss[2][2], vw[2][4][VW], vss[2][4];
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      const int base = warp * KS_KEYS + 16 * gr;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = base + kr + 8 * h;
        load_words<KW>(kw[gr][h], st + r * (HD / 2) + c * (KW * 4));
        const uint8_t* sp = st + SCALES + r * (HD / 16) + c * (HD / 64);
        kss[gr][h] = HD == 128 ? *reinterpret_cast<const unsigned short*>(sp) : *sp;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = base + ((i & 1) ? vr1 : vr0) + 8 * (i >> 1);
        load_words<VW>(vw[gr][i], st + RAW + r * (HD / 2) + g * (VW * 4));
        vss[gr][i] = st[RAW + SCALES + r * (HD / 16) + (g * HD) / 128];
      }
    }
    // rows behind the last key, and of pages that are not there: zeros
    const uint32_t have = s_pages[rp.slot];
    if (k0 + KS_KEYS > ke || have != (1u << (KA_CH >> a.pool.ps_log)) - 1u) {
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        const bool page = (have >> ((warp * KS_KEYS + 16 * gr) >> a.pool.ps_log)) & 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!page || k0 + 16 * gr + kr + 8 * h >= ke) {
#pragma unroll
            for (int w = 0; w < KW; ++w) kw[gr][h][w] = 0u;
            kss[gr][h] = 0u;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!page || k0 + 16 * gr + ((i & 1) ? vr1 : vr0) + 8 * (i >> 1) >= ke) {
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[gr][i][w] = 0u;
            vss[gr][i] = 0u;
          }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(s_free + rp.slot));
    // ---- scores of 32 keys: s[gr] = {key g: vectors 2c, 2c + 1; key g + 8: the same}
    float s[2][4];
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[gr][e] = 0.f;
      uint32_t sk[2][2];                     // scale pairs per key and 16-dim group
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = e4m3_pair(kss[gr][h]);
        sk[h][0] = __byte_perm(x, x, 0x1010);
        sk[h][1] = HD == 128 ? __byte_perm(x, x, 0x3232) : sk[h][0];
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {         // 8 dims a word: two 16-dim steps of 4 dims a lane
        const uint32_t x = kw[gr][0][w], y = kw[gr][1][w], sx = sk[0][w / 2], sy = sk[1][w / 2];
        mma_f16(s[gr], mul_f16x2(e2m1_pair<0>(x), sx), mul_f16x2(e2m1_pair<0>(y), sy), mul_f16x2(e2m1_pair<1>(x), sx),
                mul_f16x2(e2m1_pair<1>(y), sy), q[2 * w][0], q[2 * w][1]);
        mma_f16(s[gr], mul_f16x2(e2m1_pair<2>(x), sx), mul_f16x2(e2m1_pair<2>(y), sy), mul_f16x2(e2m1_pair<3>(x), sx),
                mul_f16x2(e2m1_pair<3>(y), sy), q[2 * w + 1][0], q[2 * w + 1][1]);
      }
    }
    // ---- softmax in log2 units
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      s[gr][0] *= sc0;
      s[gr][1] *= sc1;
      s[gr][2] *= sc0;
      s[gr][3] *= sc1;
    }
    if (k0 + KS_KEYS > rq.ctx || k0 + KS_KEYS > ke) {   // the step's own rows, or past the range
#pragma unroll
      for (int gr = 0; gr < 2; ++gr)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = k0 + 16 * gr + kr + 8 * (e >> 1), v = 2 * c + (e & 1), j = key - rq.ctx;
          bool see = key < ke;
          if (j >= 0) see = see && v < qv && (a.mask ? (s_bits[v] >> j) & 1ull : j <= v / a.G);
          if (!see) s[gr][e] = -INFINITY;
        }
    }
    const float t0 = max_nan(max3_nan(s[0][0], s[0][2], s[1][0]), s[1][2]), t1 = max_nan(max3_nan(s[0][1], s[0][3], s[1][1]), s[1][3]);
    // the running maximum moves only when some score exceeds it by more than KA_RESCALE
    if (__any_sync(0xffffffffu, !(t0 <= m0 + KA_RESCALE) || !(t1 <= m1 + KA_RESCALE))) {
      float n0 = max_nan(t0, m0), n1 = max_nan(t1, m1);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        n0 = max_nan(n0, __shfl_xor_sync(0xffffffffu, n0, d));
        n1 = max_nan(n1, __shfl_xor_sync(0xffffffffu, n1, d));
      }
      const float f0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int j = 0; j < ST; ++j) {
        o[j][0] *= f0;
        o[j][1] *= f1;
        o[j][2] *= f0;
        o[j][3] *= f1;
      }
    }
    // p times 2^7 in fp16 (as above); a vector that sees nothing yet: maximum 0, every p 0
    const float b0 = (m0 == -INFINITY ? 0.f : m0) - 7.f, b1 = (m1 == -INFINITY ? 0.f : m1) - 7.f;
    uint32_t pb[2][2];
#pragma unroll
    for (int gr = 0; gr < 2; ++gr)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = fast_exp2(s[gr][2 * h] - b0), p1 = fast_exp2(s[gr][2 * h + 1] - b1);
        l0 += p0;
        l1 += p1;
        pb[gr][h] = transpose8x8(pack_f16(p0, p1));   // keys 2c, 2c + 1 (+ 8 h) of vector g
      }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      const uint32_t sa = e4m3_pair(vss[gr][0] | (vss[gr][1] << 8)), sb = e4m3_pair(vss[gr][2] | (vss[gr][3] << 8));
#pragma unroll
      for (int w = 0; w < VW; ++w) {         // 8 dims a word: 4 tiles of 2 dims a lane
        const uint32_t x0 = vw[gr][0][w], x1 = vw[gr][1][w], y0 = vw[gr][2][w], y1 = vw[gr][3][w];
        const uint32_t xe = (x0 & 0x0F0F0F0Fu) | ((x1 << 4) & 0xF0F0F0F0u), xo = ((x0 >> 4) & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u);
        const uint32_t ye = (y0 & 0x0F0F0F0Fu) | ((y1 << 4) & 0xF0F0F0F0u), yo = ((y0 >> 4) & 0x0F0F0F0Fu) | (y1 & 0xF0F0F0F0u);
        mma_f16(o[4 * w], mul_f16x2(e2m1_pair<0>(xe), sa), mul_f16x2(e2m1_pair<0>(xo), sa), mul_f16x2(e2m1_pair<0>(ye), sb),
                mul_f16x2(e2m1_pair<0>(yo), sb), pb[gr][0], pb[gr][1]);
        mma_f16(o[4 * w + 1], mul_f16x2(e2m1_pair<1>(xe), sa), mul_f16x2(e2m1_pair<1>(xo), sa), mul_f16x2(e2m1_pair<1>(ye), sb),
                mul_f16x2(e2m1_pair<1>(yo), sb), pb[gr][0], pb[gr][1]);
        mma_f16(o[4 * w + 2], mul_f16x2(e2m1_pair<2>(xe), sa), mul_f16x2(e2m1_pair<2>(xo), sa), mul_f16x2(e2m1_pair<2>(ye), sb),
                mul_f16x2(e2m1_pair<2>(yo), sb), pb[gr][0], pb[gr][1]);
        mma_f16(o[4 * w + 3], mul_f16x2(e2m1_pair<3>(xe), sa), mul_f16x2(e2m1_pair<3>(xo), sa), mul_f16x2(e2m1_pair<3>(ye), sb),
                mul_f16x2(e2m1_pair<3>(yo), sb), pb[gr][0], pb[gr][1]);
      }
    }
  }
  }
  __syncthreads();                           // every tile is read: the ring takes the states
  // ---- the four warps' states, in warp order
  if (warp < KS_WARPS) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  if (g == 0) {
    s_m[warp][2 * c] = m0;
    s_m[warp][2 * c + 1] = m1;
    s_l[warp][2 * c] = l0;
    s_l[warp][2 * c + 1] = l1;
  }
#pragma unroll
  for (int j = 0; j < ST; ++j) {             // tile j of a lane: dims g hd / 8 + 2 j and + 1
    const int d = g * (HD / 8) + 2 * j;
    s_o[warp][d][2 * c] = o[j][0];
    s_o[warp][d][2 * c + 1] = o[j][1];
    s_o[warp][d + 1][2 * c] = o[j][2];
    s_o[warp][d + 1][2 * c + 1] = o[j][3];
  }
  }
  __syncthreads();
  for (int x = tid; x < qv * (HD / 2); x += 32 * KS_WARPS + 32) {
    const int v = x / (HD / 2), d = 2 * (x - v * (HD / 2));
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < KS_WARPS; ++w) M = max_nan(M, s_m[w][v]);
    float L = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < KS_WARPS; ++w) {
      if (s_m[w][v] == -INFINITY) continue;
      const float f = fast_exp2(s_m[w][v] - M);
      L = fmaf(f, s_l[w][v], L);
      y0 = fmaf(f, s_o[w][d][v], y0);
      y1 = fmaf(f, s_o[w][d + 1][v], y1);
    }
    const int i = v / a.G;
    const size_t at = static_cast<size_t>(rq.row0 + i) * a.Hq + kvh * a.G + (v - i * a.G);
    const bool none = L == 0.f;
    const float m2 = none ? -INFINITY : M - 7.f;
    if (a.joined) {                          // (this thread alone reads these two places)
      s_o[0][d][v] = y0;
      s_o[0][d + 1][v] = y1;
      if (d == 0) {
        s_jm[v] = m2;
        s_jl[v] = L;
      }
    } else if (a.splits > 1) {
      if (!none)
        *reinterpret_cast<float2*>(a.part_o + (static_cast<size_t>(split) * a.N * a.Hq + at) * HD + d) =
            make_float2(y0, y1);
      if (d == 0) a.part_ml[static_cast<size_t>(split) * a.N * a.Hq + at] = make_float2(m2, L);
    } else {
      const float inv = none ? 0.f : a.vg / L;
      *reinterpret_cast<uint32_t*>(a.out + (rq.row0 + i) * a.out_ld + static_cast<long long>(kvh * a.G + v - i * a.G) * HD + d) =
          none ? 0u : pack_bf16(y0 * inv, y1 * inv);
      if (d == 0 && a.lse) a.lse[at] = none ? -INFINITY : (m2 + log2f(L)) * 0.6931471805599453f;
    }
  }
  if (a.joined) {   // the cluster's ranges, in rank order
    __syncthreads();
    cluster_sync();
    constexpr int THREADS = 32 * KS_WARPS + 32;
    for (int x = split * THREADS + tid; x < qv * (HD / 2); x += a.splits * THREADS) {
      const int v = x / (HD / 2), d = 2 * (x - v * (HD / 2));
      float m[KA_MAX_JOIN], M = -INFINITY;
#pragma unroll
      for (int r = 0; r < KA_MAX_JOIN; ++r) {
        m[r] = r < a.splits ? remote(s_jm + v, r) : -INFINITY;
        M = max_nan(M, m[r]);
      }
      float L = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int r = 0; r < KA_MAX_JOIN; ++r) {
        if (m[r] == -INFINITY) continue;
        const float f = exp2f(m[r] - M);
        L = fmaf(f, remote(s_jl + v, r), L);
        y0 = fmaf(f, remote(&s_o[0][d][v], r), y0);
        y1 = fmaf(f, remote(&s_o[0][d + 1][v], r), y1);
      }
      const bool none = L == 0.f;
      const float inv = none ? 0.f : a.vg / L;
      const int i = v / a.G, n = rq.row0 + i, h = kvh * a.G + (v - i * a.G);
      *reinterpret_cast<uint32_t*>(a.out + n * a.out_ld + static_cast<long long>(h) * HD + d) = none ? 0u : pack_bf16(y0 * inv, y1 * inv);
      if (d == 0 && a.lse) a.lse[static_cast<size_t>(n) * a.Hq + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    cluster_sync();                          // (the others' shared memory stays until it is read)
  }
}

// Joins the key ranges of a request: WARPS warps per (row, query head), each a share of the ranges,
// HD / 32 dims per lane.  (One warp walking 57 ranges of a few rows took 10 us on its own.)
template <int HD, int WARPS>
__global__ void __launch_bounds__(128) kv_attention_combine(const KaArgs a) {
  constexpr int E = HD / 32;
  __shared__ float s_o[4][HD], s_l[4];
  pdl_wait();                                // the ranges' results
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WARPS;
  const long long w = static_cast<long long>(blockIdx.x) * (4 / WARPS) + warp / WARPS;
  const int n = static_cast<int>(w / a.Hq), h = static_cast<int>(w - static_cast<long long>(n) * a.Hq);
  if (n >= a.N) return;
  const int b = row_owner(a.cu, a.B, n);
  if (b < 0) return;
  const Req rq = request(a, b);
  if (n - rq.row0 >= rq.R || n < rq.row0) return;
  const int used = min(a.splits, (rq.len + a.tiles_per_cta * KA_CH - 1) / (a.tiles_per_cta * KA_CH));
  const size_t at = static_cast<size_t>(n) * a.Hq + h, step = static_cast<size_t>(a.N) * a.Hq;
  float M = -INFINITY;
  for (int s = lane; s < used; s += 32) M = fmaxf(M, a.part_ml[s * step + at].x);
  M = warp_max(M);
  float o[E], L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int s = part; s < used; s += WARPS) {
    const float2 ml = a.part_ml[s * step + at];
    if (ml.x == -INFINITY) continue;
    const float f = M == INFINITY ? (ml.x == INFINITY ? 1.f : 0.f) : exp2f(ml.x - M);
    L = fmaf(f, ml.y, L);
    const float* p = a.part_o + (s * step + at) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(f, p[e], o[e]);
  }
  if constexpr (WARPS > 1) {                 // (the CTA is one row's: it is here whole)
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[part][lane * E + e] = o[e];
    if (lane == 0) s_l[part] = L;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int r = 1; r < WARPS; ++r) {
      L += s_l[r];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += s_o[r][lane * E + e];
    }
  }
  const bool none = L == 0.f;
  // (the values' global factor last: a range's sum, of p up to 2^15 times values up to 2688, has room
  // for none of 1e30)
  const float inv = none ? 0.f : a.vg / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + n * a.out_ld + static_cast<long long>(h) * HD + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = none ? 0u : pack_bf16(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[at] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// How a call is cut: query-vector tiles per CTA, blocks per request, key ranges.
struct Plan {
  bool step;                               // the kernel for few vectors of a 4-bit cache
  bool joined;                             // a request's ranges are a cluster
  int nb, blocks, tiles_per_cta, splits;
};
Plan plan(const eagle_kv_cache_t* c, const eagle_kv_attention_t* w) {
  Plan p;
  const long long qv = static_cast<long long>(w->max_rows) * (w->n_heads / c->n_kv_heads);
  p.step = c->kind == EAGLE_CACHE_F4 && qv <= KS_QV;
  p.nb = qv > KA_QV ? 2 : 1;
  p.blocks = static_cast<int>((qv + KA_QV * p.nb - 1) / (KA_QV * p.nb));
  const long long base = static_cast<long long>(w->B) * c->n_kv_heads * p.blocks;
  const long long tiles = (static_cast<long long>(w->max_len) + KA_CH - 1) / KA_CH;
  // Key ranges: the split that takes least, a CTA costing its tiles and `fixed` more
  // for its start and its result.  Up to 8 ranges join in a cluster where the device holds all
  // clusters at once (each within one of its groups of about 19 SMs); in several waves the ranges of
  // requests of different lengths keep each other waiting (150 us of attention_step_b32_f4 where
  // separate ranges take 131).  Others join in a second kernel, which costs `second` tiles and
  // another for every four ranges (attention_step_b1: 13.2 us, joined 12.2, and 8 us less host time).
  const long long per_sm = p.step ? KS_CTAS : 1, sms = num_sms() > 0 ? num_sms() : 152, slots = sms * per_sm;   // (152: without a device, a GB300's)
  const long long fixed = p.step ? KS_FIXED : KA_FIXED, second = p.step ? 3 : 4;
  long long per = tiles;
  double best = -1.;
  p.joined = false;
  const long long most = std::min(tiles, 8 * slots / base + 1);   // (beyond 8 waves more ranges only cost)
  // (only the n at which the tiles per range change: about twice the root of the tiles)
  for (long long n = 1, t = 0; n <= most; n = t > 1 ? (tiles + t - 2) / (t - 1) : most + 1) {
    t = (tiles + n - 1) / n;
    const long long ranges = (tiles + t - 1) / t;
    const bool join = ranges > 1 && ranges <= KA_MAX_JOIN && p.nb == 1 && base <= sms / 19 * (19 * per_sm / ranges);
    // the requests all as long as the bound, and (of several requests) of lengths spread below it:
    // then the longest CTA, or the work of the average request on all slots
    const double even = static_cast<double>((base * ranges + slots - 1) / slots * (t + fixed));
    const double spread = std::max<double>(t + fixed, base * (0.5 * tiles + fixed * 0.5 * (ranges + 1)) / slots);
    const double cost = (w->B > 1 ? 0.5 * (even + spread) : even) + (ranges == 1 || join ? 0. : second + 0.25 * ranges);
    if (best < 0 || cost < best) {
      best = cost;
      per = t;
      p.joined = join;
    }
  }
  p.tiles_per_cta = static_cast<int>(per);
  p.splits = static_cast<int>((tiles + per - 1) / per);
  return p;
}

eagle_status_t check_args(const eagle_kv_cache_t* c, const eagle_kv_attention_t* w, const char* who, KvPool* pool) {
  const eagle_status_t r = kv_pool(c, who, pool);
  if (r != EAGLE_OK) return r;
  if (!w) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null arguments", who);
  if (w->B < 1 || w->N < 0 || w->max_rows < 1 || w->max_len < 1)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: need B, max_rows, max_len >= 1 and N >= 0", who);
  if (w->max_len > 1 << 30) return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: max_len must be at most 2^30", who);
  if (w->n_heads < 1 || w->n_heads % c->n_kv_heads || w->n_heads / c->n_kv_heads > KA_MAX_GROUP)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: n_heads must be 1..%d times n_kv_heads", who, KA_MAX_GROUP);
  if (w->mask && (w->mask_slots < 1 || w->mask_slots > 64 || w->max_rows > w->mask_slots))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: a mask needs max_rows <= mask_slots <= 64", who);
  if (!std::isfinite(w->scale) || w->scale < 0.f) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: scale must be finite and not negative", who);
  return EAGLE_OK;
}

// The ranges of a request (grid x) as one cluster where they join in it.
template <typename... P, typename... A>
cudaError_t launch_ranges(const KaArgs& a, dim3 grid, int threads, size_t smem, cudaStream_t st, void (*kernel)(P...), const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.joined ? a.splits : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = a.joined ? 1 : 0;
  cfg.stream = st;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

template <int HD, int CACHE, int NB>
cudaError_t launch_tc(const CUtensorMap& tmk, const CUtensorMap& tmv, const KaArgs& a, cudaStream_t st) {
  static std::atomic<size_t> granted[64];   // shared memory per device, set on its first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  size_t cap = dev < 64 ? granted[dev].load() : 0;
  if (!cap) {
    e = allow_max_smem(reinterpret_cast<const void*>(kv_attention_tc<HD, CACHE, NB>), &cap);
    if (e != cudaSuccess) return e;
    if (CACHE == EAGLE_CACHE_F4) {   // the roles' registers must fit what the launch gives, or they would wait for ever
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kv_attention_tc<HD, CACHE, NB>);
      if (e != cudaSuccess) return e;
      const int need = 128 * KA_REG_CTRL + 128 * NB * ka_reg_softmax(NB) + 256 * ka_reg_conv(NB);
      if (fa.numRegs / 8 * 8 * ka_threads(CACHE, NB) < need || fa.numRegs < ka_reg_conv(NB)) return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) granted[dev].store(cap);
  }
  const size_t fixed = (NB == 2 ? 2 * ka_entry(HD) : 0) + (CACHE == EAGLE_CACHE_F4 ? KA_RAW * ka_raw_bytes(HD) : 0) + KA_MISC + 1024;
  const int ns = std::min<int>(KA_MAX_SLOTS, static_cast<int>((cap - fixed) / ka_entry(HD)));
  const size_t smem = fixed + static_cast<size_t>(ns) * ka_entry(HD);
  return launch_ranges(a, dim3(a.splits, a.pool.Hkv, a.B * a.blocks), ka_threads(CACHE, NB), smem, st,
                       kv_attention_tc<HD, CACHE, NB>, tmk, tmv, a, ns);
}

template <int HD>
cudaError_t launch_step(const KaArgs& a, cudaStream_t st) {
  constexpr size_t smem = static_cast<size_t>(KS_STAGES) * ks_stage(HD);
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load()) {
    e = cudaFuncSetAttribute(kv_attention_step_f4<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(1);
  }
  return launch_ranges(a, dim3(a.splits, a.pool.Hkv, a.B), 32 * KS_WARPS + 32, smem, st, kv_attention_step_f4<HD>, a);
}

template <int HD>
cudaError_t launch_all(const CUtensorMap& tmk, const CUtensorMap& tmv, const KaArgs& a, bool f4, const Plan& p, cudaStream_t st) {
  cudaError_t e;
  const int nb = p.nb;
  if (p.step) {
    e = launch_step<HD>(a, st);
  } else if (f4) e = nb == 2 ? launch_tc<HD, EAGLE_CACHE_F4, 2>(tmk, tmv, a, st) : launch_tc<HD, EAGLE_CACHE_F4, 1>(tmk, tmv, a, st);
  else e = nb == 2 ? launch_tc<HD, EAGLE_CACHE_BF16, 2>(tmk, tmv, a, st) : launch_tc<HD, EAGLE_CACHE_BF16, 1>(tmk, tmv, a, st);
  if (e != cudaSuccess || a.splits == 1 || a.joined) return e;
  const long long rows = static_cast<long long>(a.N) * a.Hq;
  const bool wide = a.splits > 8 && rows < 1ll << 31;   // (fewer ranges: a warp each row)
  // (starts while the ranges still run and waits for them: their results, and nothing before)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(static_cast<unsigned>(wide ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(128);
  return wide ? cudaLaunchKernelEx(&cfg, kv_attention_combine<HD, 4>, a) : cudaLaunchKernelEx(&cfg, kv_attention_combine<HD, 1>, a);
}

}  // namespace

static int64_t workspace_bytes(const eagle_kv_cache_t* cache, const eagle_kv_attention_t* args, const Plan& p) {
  if (p.splits == 1 || p.joined) return 0;
  return static_cast<int64_t>(p.splits) * args->N * args->n_heads * (4 * cache->head_dim + 8);
}

extern "C" int64_t eagle_kv_attention_workspace(const eagle_kv_cache_t* cache, const eagle_kv_attention_t* args) {
  KvPool pool;
  if (check_args(cache, args, "kv_attention_workspace", &pool) != EAGLE_OK) return -1;
  return workspace_bytes(cache, args, plan(cache, args));
}

extern "C" eagle_status_t eagle_kv_attention(const eagle_kv_cache_t* cache, const eagle_kv_attention_t* w, uint32_t* err_word,
                                             void* stream) {
  const char* who = "kv_attention";
  KaArgs a;
  memset(&a, 0, sizeof(a));
  const eagle_status_t r = check_args(cache, w, who, &a.pool);
  if (r != EAGLE_OK) return r;
  if (!err_word || !w->cu_rows || !w->lens || !w->q || !w->out) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  const int hd = cache->head_dim;
  const long long width = static_cast<long long>(w->n_heads) * hd;
  if (w->q_stride < width || w->out_stride < width || w->q_stride % 8 || w->out_stride % 8 ||
      reinterpret_cast<uintptr_t>(w->q) % 16 || reinterpret_cast<uintptr_t>(w->out) % 16)
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned and not overlap", who);
  if (w->q == w->out) return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: out may not be q (ranges and blocks read q at different times)", who);
  const Plan p = plan(cache, w);
  const int64_t need = workspace_bytes(cache, w, p);
  if (need > 0 && (!w->workspace || w->workspace_bytes < need || reinterpret_cast<uintptr_t>(w->workspace) % 16))
    return kv_fail(EAGLE_ERR_INVALID_ARG, "%s: needs %lld bytes of workspace, 16-byte aligned", who, static_cast<long long>(need));
  if (w->N == 0) return EAGLE_OK;
  const long long rows_heads = static_cast<long long>(w->N) * w->n_heads;
  if (rows_heads > (1ll << 31) - 8 || cache->n_kv_heads > 65535 || static_cast<long long>(w->B) * p.blocks > 65535)
    return kv_fail(EAGLE_ERR_UNSUPPORTED, "%s: too many rows, heads or requests for one launch", who);
  a.B = w->B;
  a.N = w->N;
  a.Hq = w->n_heads;
  a.G = w->n_heads / cache->n_kv_heads;
  a.max_rows = w->max_rows;
  a.max_len = w->max_len;
  a.S = w->mask_slots;
  a.blocks = p.blocks;
  a.tiles_per_cta = p.tiles_per_cta;
  a.splits = p.splits;
  a.joined = p.joined;
  a.cu = w->cu_rows;
  a.lens = w->lens;
  a.q = static_cast<const __nv_bfloat16*>(w->q);
  a.q_ld = w->q_stride;
  a.mask = w->mask;
  a.scale_log2 = std::min((w->scale > 0.f ? w->scale : 1.0f / std::sqrt(static_cast<float>(hd))) * 1.4426950408889634f, FLT_MAX);
  a.vg = cache->kind == EAGLE_CACHE_F4 ? a.pool.vg : 1.f;
  a.out = static_cast<__nv_bfloat16*>(w->out);
  a.out_ld = w->out_stride;
  a.lse = w->lse;
  a.part_o = static_cast<float*>(w->workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(p.splits) * w->N * w->n_heads * hd);
  a.err = err_word;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f4 = cache->kind == EAGLE_CACHE_F4;
  CUtensorMap tmk, tmv;
  memset(&tmk, 0, sizeof(tmk));
  memset(&tmv, 0, sizeof(tmv));
  const long long blocks = static_cast<long long>(cache->num_pages) * cache->n_kv_heads;
  if (!f4 && (!make_page_map(&tmk, cache->k, hd, cache->page_size, blocks) || !make_page_map(&tmv, cache->v, hd, cache->page_size, blocks)))
    return kv_fail(EAGLE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", who);
  const cudaError_t e = hd == 64 ? launch_all<64>(tmk, tmv, a, f4, p, st) : launch_all<128>(tmk, tmv, a, f4, p, st);
  return e == cudaSuccess ? EAGLE_OK : kv_fail(EAGLE_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
}
