// What the attention kernels over paged caches share (kvattn.cu, kvcross.cu, kvshared.cu): a
// call's arguments, its rows and keys, how it is cut into key ranges, small device helpers.
#pragma once

#include "kvcache.cuh"

#include <cfloat>
#include <cmath>
#include <cstring>

namespace eagle {

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B, f32 D, both K-major (as
// idesc_bf16_f32, whose operands are bf16).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 3-D map over a paged bf16 cache [pages * Hkv][page_size][hd]: boxes of `rows` rows (0: all) of a page
// of one KV head x 64 dims, 128-byte swizzle; rows outside the page or the pool read as zeros.
inline bool make_page_map(CUtensorMap* tm, const void* pool, int hd, int page_size, long long blocks, int rows = 0) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd) * 2, static_cast<cuuint64_t>(hd) * 2 * page_size};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows ? rows : page_size), 1};
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

// registers per thread of the 4-bit kernel's roles after they moved (the launch checks their sum)
constexpr int KA_REG_CTRL = 40;
__host__ __device__ constexpr int ka_reg_softmax(int nb) { return nb == 2 ? 136 : 152; }
__host__ __device__ constexpr int ka_reg_conv(int nb) { return nb == 2 ? 80 : 128; }
__host__ __device__ constexpr uint32_t ka_entry(int hd) { return static_cast<uint32_t>(hd) * 2 * KA_CH; }
// 4-bit caches: a ring of raw tiles (128 rows of codes, then their scales) behind the entries
constexpr int KA_RAW = 3;
__host__ __device__ constexpr uint32_t ka_raw_bytes(int hd) { return static_cast<uint32_t>(hd) / 2 * KA_CH + hd / 16 * KA_CH; }

struct KaArgs {
  KvPool pool;
  int B, N, Hq, G, max_rows, max_len, S;
  uint32_t g_inverse;                      // 2^32 / G (kvcross.cu)
  int blocks;                              // query-vector blocks per request
  int tiles_per_cta, splits, least;        // a range's tiles at most, ranges, and its tiles at least (range_tiles)
  int joined;                              // the ranges of a request are one cluster and join in it
  int parts;                               // results go to part_o / part_ml: of several ranges, or to be joined with others
  int behind;                              // starts before the kernel ahead of it has ended, and ends after it
  int cross;                               // the rows are no keys of the cache: each sees lens[b] keys, all of them
  const int* groups;                       // [B + 1] or null: item b's rows are those of requests groups[b] .. groups[b + 1] - 1
  int requests;                            // (of this many)
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
  float* part_o;                           // [splits][N][Hq][hd] unnormalised outputs (parts)
  float2* part_ml;                         // [splits][N][Hq] running maximum (log2 units) and sum
  unsigned* err;
};

// Request b's rows and keys, clamped to what the call allows.  (cross: the keys are `ctx` alone.)
struct Req {
  int row0, R, ctx, len;
};
EAGLE_DEV Req request(const KaArgs& a, int b) {
  Req r;
  int i0 = b, i1 = b + 1;
  if (a.groups) {                          // (a group that descends or leaves the requests has no rows past them)
    const int g0 = __ldg(a.groups + b), g1 = __ldg(a.groups + b + 1);
    i0 = min(max(g0, 0), a.requests);
    i1 = min(max(g1, i0), a.requests);
    if (i0 != g0 || i1 != g1) atomicOr(a.err, DEVERR_PREFIX);
  }
  const int c0 = __ldg(a.cu + i0), c1 = __ldg(a.cu + i1), l = __ldg(a.lens + b);
  r.row0 = min(max(c0, 0), a.N);
  r.R = min(max(min(c1, a.N) - r.row0, 0), a.cross ? a.max_rows : min(a.max_rows, a.max_len));
  r.ctx = min(max(l, 0), a.cross ? a.max_len : a.max_len - r.R);
  if (r.row0 != c0 || r.R != c1 - c0 || r.ctx != l) atomicOr(a.err, DEVERR_PREFIX);
  r.len = a.cross ? r.ctx : r.ctx + r.R;
  return r;
}

// Tiles of a range of a sequence of `len` keys, and how many ranges it has.  The bound's ranges are shared out
// over the keys that there are: calls bounded by a cache's capacity would otherwise leave them to the
// first few CTAs, and the longest of mixed lengths decide (4 rows of 8 KV heads over 32,000 keys of at most
// 512,000: 239 us, now 33; 4 sequences of 5,000 to 35,000 keys 83, now 68).
EAGLE_DEV int range_tiles(const KaArgs& a, int len) {
  return min(a.tiles_per_cta, max(((len + KA_CH - 1) / KA_CH + a.splits - 1) / a.splits, a.least));
}
EAGLE_DEV int ranges_of(const KaArgs& a, int len) {
  const int keys = range_tiles(a, len) * KA_CH;
  return min(a.splits, (len + keys - 1) / keys);
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

// f y, x + f y of a part with a weight.  In 32 bits f may have fallen to 0: what is not finite in y stays
// all the same, so that no infinity or NaN depends on how the keys were cut into parts.
EAGLE_DEV float weighted(float f, float y) { return f != 0.f ? f * y : fabsf(y) < INFINITY ? 0.f : y; }
EAGLE_DEV float add_weighted(float x, float f, float y) { return f != 0.f ? fmaf(f, y, x) : fabsf(y) < INFINITY ? x : x + y; }

// The sum of what is not finite among the values of keys [begin, end), all of which the row sees: lane by
// lane of E dims from d on, bf16 pages: 0, an infinity, or NaN.  For sums p v that came out as NaN where no p is: a p
// that fell to 0, or the lower part of one in two parts, makes NaN of an infinity that the formula keeps.  A key
// that is not finite itself has a weight of 0 there (its score is -infinity; any other would have made
// the row's sum of p NaN), and 0 times infinity is NaN.  By a whole warp; begin a multiple of 16.  The rare
// path, bound by the latency of its loads: 0.05 us a key.
template <int HD, int E>
EAGLE_DEV void infinities(const KvPool& pool, int b, int kvh, int begin, int end, int d, float* r, int lane, unsigned* err) {
  constexpr int KB = 16;                   // keys in flight (of one page)
  const auto* kp = static_cast<const __nv_bfloat16*>(pool.k);
  const auto* vp = static_cast<const __nv_bfloat16*>(pool.v);
  auto value = [&](size_t row, int e) { return static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(vp + row * HD + d) + e)); };
#pragma unroll
  for (int e = 0; e < E; ++e) r[e] = 0.f;
#pragma unroll 1
  for (int k = begin; k < end; k += KB) {
    const int page = kv_page(pool, b, k, err);
    if (page < 0) continue;                // (reads as zeros)
    const size_t row = kv_row(pool, page, kvh, k);
    uint32_t top = 0;                      // (the page is there whole: rows behind `end` are read and dropped)
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) top = max(top, value(row + i, e) & 0x7fffu);
    if (!__any_sync(0xffffffffu, top >= 0x7f80u)) continue;
#pragma unroll 1
    for (int i = 0; i < KB && k + i < end; ++i) {
      bool odd = false;                    // the key's own dims
#pragma unroll
      for (int x = 0; x < HD / 32; ++x)
        odd |= (__ldg(reinterpret_cast<const unsigned short*>(kp + (row + i) * HD) + x * 32 + lane) & 0x7f80u) == 0x7f80u;
      odd = __any_sync(0xffffffffu, odd);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t v = value(row + i, e);
        if ((v & 0x7f80u) == 0x7f80u) r[e] += odd ? __uint_as_float(0x7fc00000u) : __uint_as_float(v << 16);
      }
    }
  }
}

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

// How a call is cut: query-vector tiles per CTA, blocks per request, key ranges.
struct KaPlan {
  bool step;                               // the kernel for few vectors of a 4-bit cache
  bool joined;                             // a request's ranges are a cluster
  int nb, blocks, tiles_per_cta, splits, least;
};
// Cuts B requests (or groups) of up to max_rows rows of G heads per KV head over up to max_len keys.
// may_join: a cluster may write the results; otherwise every range leaves a partial result.
KaPlan ka_plan(int kind, int Hkv, int G, int B, int max_rows, int max_len, bool may_join);
// Launches the ranges of a call (without the join of separate ranges), and that join.  The plan's
// members of `a` are filled in here.
cudaError_t ka_launch(KaArgs* a, const KaPlan& p, bool f4, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t st);
cudaError_t ka_combine(const KaArgs& a, cudaStream_t st);
// Bytes of one range's partial results.
inline int64_t ka_part_bytes(long long N, int Hq, int hd) { return N * Hq * (4ll * hd + 8); }

// The same for many query vectors of cross attention (kvcross.cu): its CTAs, and the bytes of
// workspace (`parts`) for items that they divide.  `own`: partial results of the rows' own keys, of a
// kernel launched before on the same stream, to be joined.
struct KxPlan {
  int ctas;
  int64_t bytes;
};
KxPlan kx_plan(int kind, int Hkv, int hd, int G, int B, int max_rows, int max_len);
cudaError_t kx_launch(const KaArgs& a, const KaArgs* own, bool f4, const CUtensorMap& tmk, const CUtensorMap& tmv, const KxPlan& p,
                      float* parts, cudaStream_t st);
// Whether it takes less time than ranges, for up to max_rows rows of G heads a KV head and sequence, N in all.
bool kx_worth(int kind, int Hkv, int G, int B, long long N, int max_rows, int max_len);

// The same for few query vectors (kvfew.cu: at most KF_QV a KV head and request, bf16 pages, every row
// sees all its keys).  Writes out and lse, or with a.parts the one partial result of every row; the
// plan's members of `a` are filled in here.
constexpr int KF_QV = 8;
KxPlan kf_plan(int Hkv, int hd, int B, int max_len);
bool kf_worth(int Hkv, int hd, int qv, int B, int max_len, bool alone);   // alone: no other keys are joined to them
cudaError_t kf_launch(KaArgs* a, const eagle_kv_cache_t* cache, const KxPlan& p, float* parts, cudaStream_t st);

// The ranges of a request (grid x) as one cluster where they join in it.
template <typename... P, typename... A>
cudaError_t launch_ranges(const KaArgs& a, dim3 grid, int threads, size_t smem, cudaStream_t st, void (*kernel)(P...), const A&... args) {
  cudaLaunchAttribute attr[1];
  if (a.behind) {                          // (never joined: its results go to another join)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.joined ? a.splits : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = a.behind || a.joined ? 1 : 0;
  cfg.stream = st;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace eagle
