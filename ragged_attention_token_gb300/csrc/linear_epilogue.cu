// Linear layer with its whole epilogue: c = act(a W^T + bias) + residual over
// the T = cu_seqlens[B] packed rows (T read on the device), a [cap, K] and
// W [N, K] both K-major.
//
// In 8 bits (e4m3): c = act(a_scale w_scale (a W^T) + bias) + residual, a scale for each row of a and of W, applied to the
// fp32 sums.  The kernels are the same, with K counted in bytes.  On a cool card, by graphs of calls: 12608 rows of 768 -> 2304
// 23 to 24 us, in fp32 33, 8192 of 4096 -> 16384 299 to 306 us (3600 to 3680 TFLOP/s), 4 of 4096 -> 4096 4.6 us; calls one by one
// under load 24 to 25, 347 to 361 (3050 to 3170) and 7 to 8.
//
// Three kernels, by the rows that a can hold.
//
// linear_pair_kernel: tcgen05 on pairs of SMs (cta_group::2).  A pair owns a
// tile of 256 rows x LN columns (LN = 256, 128 or 64): each CTA holds 128 of the rows
// and half of the W rows, and the pair's one product per 16-wide K step reads
// both halves, so an SM's shared memory serves 8 KB of operands per 256 x 256 x 16
// product instead of the 12 KB of a 128 x 256 x 16 one on a single SM, half as
// much per multiply-add: on one SM shared memory bandwidth holds the products
// at two thirds of the tensor rate.  Persistent, per CTA: warp 0 streams K
// chunks of 64 (16 + 16 KB) through a six-stage TMA ring, both CTAs' copies counted
// on the leader's barrier; one thread of the leader's warp 1 issues the products into one of
// two 256-column TMEM accumulators, so the next tile's products run while warps 2-9 of both
// CTAs drain the last one: bias, activation and residual in fp32, one
// rounding, through 4 KB of shared memory per warp to whole 128-byte row
// pieces.  LN is chosen on the device, where T is known: the width whose
// rounds over the pairs take the least time, the last round cut finer where it leaves pairs idle.
//
// linear_mid_kernel: tens to hundreds of rows (a token of each sequence of a large
// batch), or few outputs over a long K, by the rule at launch_typed.  The work is
// still the read of W, so W is the product's M operand (128 of its rows by up to 256
// rows of a): with a as the M operand its 128 rows are read from shared memory for
// every 64 columns of W, 320 cycles for each 8 KB of W a pair streams (64 x 4096 x
// 4096: 16.6 us, here 11.2).  A cluster of up to 8 CTAs shares K of a tile, TMA rings of 192 KB keeping W on
// its way, and joins the sums through distributed shared memory.
//
// linear_few_kernel: a handful of rows (one token of each sequence).  The work
// is one read of W, so W goes in 16-byte chunks into the mma.sync operands of the
// lane that copied them, eight warps splitting K of 16 W rows, the sums joined
// in shared memory.  The K order inside a 32-wide step is the one in which the 16-byte
// loads arrive, the same for both operands (a dot product does not mind).
//
// Every wait is bounded; a CTA that gives up tells its peer or its cluster, records
// RRA_DEVERR_WAIT_TIMEOUT, lets copies and products in flight land, frees its
// TMEM and returns; what its tile lacks then is not written.
#include <cuda_fp8.h>

#include <mutex>

#include "block.cuh"
#include "f32x2.cuh"
#include "tc_ptx.cuh"

namespace rra {
namespace {

constexpr int LM = 128;                                  // rows of a CTA's half tile
constexpr int LN_MAX = 256;                              // columns of a tile
// K per stage: one 128-byte swizzled row (64 elements, in 8 bits 128).  In bytes, the 8-bit layer (rra_linear_scaled) is the
// 16-bit one: a product reads 32 bytes of each row either way, so all of the shapes and rules here hold for it too.
template <typename Tin> constexpr int LK = 128 / static_cast<int>(sizeof(Tin));
template <typename Tin> constexpr bool SCALED = sizeof(Tin) == 1;   // rows and columns carry scales
constexpr int L_MAX_STAGES = 9;                          // ring: 6 stages at LN = 256, 8 at 128, 9 at 64
constexpr int L_EPI_WARPS = 8;                           // warps 2-9
constexpr int L_THREADS = 64 + 32 * L_EPI_WARPS;
constexpr uint32_t L_A_BYTES = LM * 128;
constexpr uint32_t L_RING_BYTES = 6 * (L_A_BYTES + LN_MAX / 2 * 128);   // 192 KB
constexpr uint32_t L_OUT_BYTES = 32 * 128;               // output staging of one epilogue warp
constexpr uint32_t L_OFF_OUT = L_RING_BYTES;
constexpr uint32_t L_OFF_BAR = L_OFF_OUT + L_EPI_WARPS * L_OUT_BYTES;
constexpr uint32_t LB_FULL = 0;                          // [stages] (the leader's: both CTAs' copies)
constexpr uint32_t LB_EMPTY = 80;                        // [stages] (each CTA's own)
constexpr uint32_t LB_ACC_FULL = 160;                    // [2] (each CTA's own)
constexpr uint32_t LB_ACC_EMPTY = 176;                   // [2] (the leader's: one arrival per epilogue warp of both)
constexpr uint32_t LW_TMEM = 192, LW_ABORT = 196;
constexpr uint32_t L_SMEM = L_OFF_BAR + 256;
constexpr uint32_t L_TMEM_COLS = 512;
// fp32 outputs: the tensor cores' additions truncate, which after K = 8192 has
// cost 1e-5 of the sum, so a tile is computed in parts of 8 chunks (K = 512),
// added in registers by the epilogue warps (which hold 128 columns of a tile):
// 7e-7.  16-bit outputs are rounded at 2^-9 and keep one sum.
constexpr int L_PART = 8, LN_PARTS = 128;

// --------------------------------------------------------- pair-of-CTAs PTX

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// The address of this shared-memory location in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Both operands K-major, fp32 sums.  E4M3 is format 0 of its kind, as F16 is of its own.
template <typename Tin>
__device__ __forceinline__ uint32_t idesc_in(int M, int N) {
  if constexpr (SCALED<Tin>) return idesc_f16(0u, 0, M, N);
  else return idesc_f16(IsBf16<Tin>::value, 0, M, N);
}
// Arrives on `bar` of both CTAs once every product issued so far has completed.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Arrival on a barrier of the pair's leader.  It publishes no memory: what it
// orders are this warp's TMEM reads, which have completed (tcgen05.wait::ld and the fence
// before it), so it is relaxed: a release waited for the warp's global stores, 1800 cycles a tile.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// ------------------------------------------------------------------ epilogue

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2f_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-x): relative to its value within a few 2^-23 for x >= 0 and (4 + 1.2 |x|) 2^-23 below (__expf is off by
// 2 + 1.17 |x| units in the last place); 0 below about -87.3, where the reciprocal of 1 + e^-x would be subnormal.
__device__ __forceinline__ float fast_sigmoid(float x) { return fast_rcp(1.f + __expf(-x)); }
// x/2 (1 + erf(x / sqrt 2)) of two values, by Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26: erfc(z) = (a1 t + ... + a5 t^5) e^{-z^2}, t = 1 / (1 + p z),
// z >= 0, within 1.5e-7 (absolute; in fp32 the result is off by up to 6e-7 |x|, 1e-7 |x| below -3).  With h = erfc(|x| / sqrt 2) / 2 the result is
// x (1/2 + copysign(1/2 - h, x)).  (With erff the epilogue of a K = 384 layer took
// 2.5 times as long as its products.)
__device__ __forceinline__ void act_gelu2(float& x, float& y) {
  auto both = [](float c) { return pair_f2(c, c); };
  const uint64_t v = pair_f2(x, y), z = pair_f2(fabsf(x), fabsf(y));
  const float2 d = halves_f2(fma_pair(z, both(0.3275911f * 0.70710678118654752f), both(1.f)));
  const uint64_t t = pair_f2(fast_rcp(d.x), fast_rcp(d.y));
  uint64_t q = fma_pair(t, both(0.5f * 1.061405429f), both(-0.5f * 1.453152027f));
  q = fma_pair(q, t, both(0.5f * 1.421413741f));
  q = fma_pair(q, t, both(-0.5f * 0.284496736f));
  q = fma_pair(q, t, both(0.5f * 0.254829592f));
  q = mul_pair(q, t);
  const float2 e = halves_f2(mul_pair(mul_pair(v, v), both(-0.5f * 1.4426950408889634f)));   // e^{-x^2 / 2} in base 2
  const float2 r = halves_f2(fma_pair(q, pair_f2(-exp2f_approx(e.x), -exp2f_approx(e.y)), both(0.5f)));
  const float2 o = halves_f2(mul_pair(v, pair_f2(0.5f + copysignf(r.x, x), 0.5f + copysignf(r.y, y))));
  x = o.x;
  y = o.y;
}
// (1 + tanh u) / 2 = 1 / (1 + e^{-2u}).
__device__ __forceinline__ float act_gelu_tanh(float x) {
  return x * fast_sigmoid(1.5957691216057308f * fmaf(0.044715f * x * x, x, x));
}
__device__ __forceinline__ float act_silu(float x) { return x * fast_sigmoid(x); }

template <int E>
__device__ __forceinline__ void activate(float (&v)[E], int act) {
  if (act == RRA_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
  } else if (act == RRA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < E; i += 2) act_gelu2(v[i], v[E > 1 ? i + 1 : i]);
  } else if (act == RRA_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = act_gelu_tanh(v[i]);
  } else if (act == RRA_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = act_silu(v[i]);
  }
}

// A 16-byte chunk of outputs as floats, and back (one rounding).
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void add(float* v, uint4 x) {
    v[0] += __uint_as_float(x.x);
    v[1] += __uint_as_float(x.y);
    v[2] += __uint_as_float(x.z);
    v[3] += __uint_as_float(x.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <> struct Chunk<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void add(float* v, uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] += __uint_as_float(w[i] << 16);
      v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Chunk<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void add(float* v, uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] += f.x;
      v[2 * i + 1] += f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 t = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The 8-bit epilogue.  The products of a tile take half the time there, and with a row a lane every lane needs every column's
// scale and bias: 32 reads of shared memory for 64 columns, beside the staging, held a tile of small K at 3.5 us.
// 32 rows (this warp's lanes of TMEM) by C columns as fragments: v[C / 2 h + 4 n + e] is row g + 16 h + 8 (e >> 1), column
// 8 n + 2 q + (e & 1), g = lane / 4, q = lane % 4.  A lane so meets C / 4 columns instead of C, in
// neighbouring pairs, which one instruction scales: 2.3 us a tile (sixteen warps with rows of 64 bytes 3.0).
template <int C>
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&v)[C]) {
  static_assert(C == 32 || C == 64, "four or eight groups of 8 columns");
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t* x = r + h * (C / 2);
    const uint32_t at = taddr + (static_cast<uint32_t>(16 * h) << 16);
#pragma unroll
    for (int k = 0; k < C / 32; ++k, x += 16)
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
            "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
          : "r"(at + 32 * k)
          : "memory");
  }
  // The wait is tied to the registers, so that no use of them is scheduled before it.
#pragma unroll
  for (int i = 0; i < C; i += 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]),
                   "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]), "+r"(r[i + 12]),
                   "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15])
                 :
                 : "memory");
}
// Two neighbouring outputs: added to floats from memory's form, and rounded to it.
__device__ __forceinline__ void add_two(float& x, float& y, uint32_t at, float) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  x += v.x;
  y += v.y;
}
__device__ __forceinline__ void add_two(float& x, float& y, uint32_t at, __nv_bfloat16) {
  const uint32_t w = ld_shared_u32(at);
  x += __uint_as_float(w << 16);
  y += __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void add_two(float& x, float& y, uint32_t at, __half) {
  const uint32_t w = ld_shared_u32(at);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  x += f.x;
  y += f.y;
}
__device__ __forceinline__ void put_two(uint32_t at, float x, float y, float) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void put_two(uint32_t at, float x, float y, __nv_bfloat16) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
  st_shared_u32(at, *reinterpret_cast<const uint32_t*>(&t));
}
__device__ __forceinline__ void put_two(uint32_t at, float x, float y, __half) {
  const __half2 t = __floats2half2_rn(x, y);
  st_shared_u32(at, *reinterpret_cast<const uint32_t*>(&t));
}

// How the T x N outputs are cut into tiles: `wide` tiles of ln columns in whole
// rounds over the pairs, then those of the last round cut f ways (1, 2 or 4) where that
// round has pairs to spare.
struct Tiling {
  int ln, f, mt, nt;
  long long wide, all, cost;
};

// The cut whose rounds take least: a tile of n columns costs 64 + n/4, the shared
// memory its products read (per 16-wide step 4 KB of a and n/64 KB of W).
__host__ __device__ __forceinline__ Tiling make_tiling(int T, int N, int pairs, int most) {
  Tiling best{};
  long long least = -1;
  const int mt = (T + 2 * LM - 1) / (2 * LM);
  for (int ln = most; ln >= 64; ln /= 2) {
    const int nt = (N + ln - 1) / ln;
    const long long tiles = static_cast<long long>(mt) * nt, rounds = tiles / pairs, rem = tiles - rounds * pairs;
    int f = 1;
    while (rounds > 0 && ln / f > 64 && 2 * f * rem <= pairs) f *= 2;
    const long long cost = rounds * (64 + ln / 4) + (rem > 0 ? 64 + ln / f / 4 : 0);
    if (least < 0 || cost < least) {
      least = cost;
      best.cost = cost;
      best.ln = ln;
      best.f = f;
      best.mt = mt;
      best.nt = nt;
      best.wide = f > 1 ? rounds * pairs : tiles;
      best.all = best.wide + (tiles - best.wide) * f;
    }
  }
  return best;
}

// Tile t of the grid of mt x nt: bands of 8 row tiles, column by column within
// a band, so that the pairs at work together share their rows of a and of W
// (8 x 9.5 tiles at 76 pairs).  With whole rows of tiles in order, every
// row tile read all of W again: 8192 x 4096 x 16384 took 780 us under load.
constexpr int L_BAND = 8;
__device__ __forceinline__ void tile_at(long long t, int mt, int nt, int& m, int& n) {
  const unsigned per = static_cast<unsigned>(L_BAND) * static_cast<unsigned>(nt);   // below 2^21
  const int band = t < (1LL << 32) ? static_cast<int>(static_cast<unsigned>(t) / per) : static_cast<int>(t / per);
  const int rows = min(L_BAND, mt - band * L_BAND);
  const int r = static_cast<int>(t - static_cast<long long>(band) * L_BAND * nt);
  m = band * L_BAND + r % rows;
  n = r / rows;
}

// Piece t of the work: its row tile, first column and width (a width of 0: past N).
__device__ __forceinline__ void piece_at(const Tiling& g, long long t, int N, int& m, int& n0, int& width) {
  int n;
  if (t < g.wide) {
    tile_at(t, g.mt, g.nt, m, n);
    n0 = n * g.ln;
    width = g.ln;
  } else {
    const long long q = t - g.wide;
    tile_at(g.wide + q / g.f, g.mt, g.nt, m, n);
    width = g.ln / g.f;
    n0 = n * g.ln + static_cast<int>(q % g.f) * width;
    if (n0 >= N) width = 0;
  }
}

// PARTS: fp32 outputs of K above one part.  A kernel of its own: the registers of the sums cost the
// one-part epilogue half its speed (SiLU on 7078 rows of 512 -> 3600: 78.9 against 39.5 us).
// LIMIT: the instantiation of launches made with a wait limit set (rra_set_wait_limit).
template <typename Tin, typename Tout, bool PARTS, bool LIMIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(L_THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w128,
                       const __grid_constant__ CUtensorMap map_w64, const __grid_constant__ CUtensorMap map_w32,
                       const LinearEpiArgs a, int act) {
  static_assert(!PARTS || sizeof(Tout) == 4, "16-bit outputs keep one sum");
  extern __shared__ __align__(1024) uint8_t smem_linear[];
  const uint32_t base = smem_u32(smem_linear);
  const uint32_t bars = base + L_OFF_BAR;
  auto bar = [&](uint32_t kind, uint32_t i) { return bars + kind + 8 * i; };
  const uint32_t abort_flag = bars + LW_ABORT;
  const volatile uint32_t* tmem_ptr = reinterpret_cast<const volatile uint32_t*>(smem_linear + L_OFF_BAR + LW_TMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bars + LW_TMEM),
                 "r"(L_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int s = 0; s < L_MAX_STAGES; ++s) {
      mbar_init(bar(LB_FULL, s), 1);
      mbar_init(bar(LB_EMPTY, s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(LB_ACC_FULL, b), 1);
      mbar_init(bar(LB_ACC_EMPTY, b), 2 * L_EPI_WARPS);
    }
    st_shared_u32(abort_flag, 0u);
    fence_barrier_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_w128);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                                    // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  dependent_launch();
  const int T = a.cu[a.B];
  bool bad = false;
  if (T < 0 || T > a.cap) {
    if (blockIdx.x == 0 && tid == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
  } else {
    const int pairs = static_cast<int>(gridDim.x) / 2, pair = static_cast<int>(blockIdx.x) / 2;
    const int kchunks = (a.K + LK<Tin> - 1) / LK<Tin>;
    const int parts = PARTS ? (kchunks + L_PART - 1) / L_PART : 1;
    const Tiling g = make_tiling(T, a.N, pairs, PARTS ? LN_PARTS : LN_MAX);
    const uint32_t stage_bytes = L_A_BYTES + static_cast<uint32_t>(g.ln / 2) * 128u;   // A rows, then W rows
    const uint32_t stages = L_RING_BYTES / stage_bytes;
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      uint32_t s = 0, lap = 0;                           // ring position: stage and times round
      if (elect_one()) {
        for (long long t = pair; t < g.all && !bad; t += pairs) {
          int m0, n0, width;
          piece_at(g, t, a.N, m0, n0, width);
          if (width == 0) continue;
          m0 = m0 * 2 * LM + static_cast<int>(rank) * LM;
          n0 += static_cast<int>(rank) * (width / 2);
          const CUtensorMap* mw = width == 256 ? &map_w128 : (width == 128 ? &map_w64 : &map_w32);
          const uint32_t bytes = 2 * (L_A_BYTES + static_cast<uint32_t>(width / 2) * 128u);
          for (int kc = 0; kc < kchunks; ++kc) {
            if (lap > 0 && !mbar_wait_limited<LIMIT>(bar(LB_EMPTY, s), (lap - 1) & 1, abort_flag, a.wait_limit)) {
              bad = true;
              break;
            }
            if (rank == 0) mbar_expect_tx(bar(LB_FULL, s), bytes);
            const uint32_t full = map_rank(bar(LB_FULL, s), 0), dst = base + s * stage_bytes;
            tma_load_2d_pair(dst, &map_a, kc * LK<Tin>, m0, full);       // rows past cap, columns past K: zeros
            tma_load_2d_pair(dst + L_A_BYTES, mw, kc * LK<Tin>, n0, full);
            if (++s == stages) {
              s = 0;
              ++lap;
            }
          }
        }
      }
      bad = __any_sync(0xffffffffu, bad);
    } else if (warp == 1) {
      // ------------------------------------------------------------ products
      if (rank == 0 && elect_one()) {
        const uint64_t da0 = sdesc(base, 16, 1024), dw0 = sdesc(base + L_A_BYTES, 16, 1024);
        uint32_t s = 0, lap = 0, i = 0;
        for (long long t = pair; t < g.all && !bad; t += pairs) {
          int m0, n0, width;
          piece_at(g, t, a.N, m0, n0, width);
          if (width == 0) continue;
          const uint32_t idesc = idesc_in<Tin>(2 * LM, width);
          for (int part = 0; part < parts && !bad; ++part, ++i) {
            const uint32_t b = i & 1;
            if (i >= 2 && !mbar_wait_limited<LIMIT>(bar(LB_ACC_EMPTY, b), ((i >> 1) - 1) & 1, abort_flag, a.wait_limit)) {
              bad = true;
              break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + b * LN_MAX;
            const int k_from = part * L_PART, k_to = PARTS ? min(kchunks, k_from + L_PART) : kchunks;
            for (int kc = k_from; kc < k_to; ++kc) {
              if (!mbar_wait_limited<LIMIT>(bar(LB_FULL, s), lap & 1, abort_flag, a.wait_limit)) {
                bad = true;
                break;
              }
              tc_fence_after();
              const uint64_t off = s * (stage_bytes >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t add = (kc > k_from || kk > 0) ? 1u : 0u;
                if constexpr (SCALED<Tin>) umma_f8_pair(acc, da0 + off + 2 * kk, dw0 + off + 2 * kk, idesc, add);
                else umma_f16_pair(acc, da0 + off + 2 * kk, dw0 + off + 2 * kk, idesc, add);
              }
              umma_commit_pair(bar(LB_EMPTY, s));
              if (++s == stages) {
                s = 0;
                ++lap;
              }
            }
            if (!bad) umma_commit_pair(bar(LB_ACC_FULL, b));
          }
        }
      }
      bad = __any_sync(0xffffffffu, bad);
    } else {
      // ------------------------------------------------------------ epilogue
      using Ch = Chunk<Tout>;
      constexpr int CHUNKS = 8;
      constexpr int CPP = CHUNKS * Ch::N;                // columns of a 128-byte piece
      constexpr int GROUPS = L_EPI_WARPS / 4;
      const int quad = warp & 3, group = (warp - 2) >> 2; // TMEM lane quadrant; which pieces
      const uint32_t stg = base + L_OFF_OUT + static_cast<uint32_t>(warp - 2) * L_OUT_BYTES;
      // Chunk k of row r of the staging, turned by the row so that neither rows nor columns of chunks meet a bank twice.
      auto staged = [&](int r, int k) { return stg + r * 128 + ((k ^ (r & 7)) << 4); };
      const uint32_t acc_empty[2] = {map_rank(bar(LB_ACC_EMPTY, 0), 0), map_rank(bar(LB_ACC_EMPTY, 1), 0)};
      uint32_t i = 0;
      // This lane's columns of the bias of piece p (of the tile at column n0): lane, and lane + 32 of a 64-column piece.
      float bias0 = 0.f, bias1 = 0.f, ws0 = 0.f, ws1 = 0.f;   // ws: those columns' scales
      float row_scale[4] = {}, next_scale = 0.f;         // of this lane's rows in fragments: g, g + 8, g + 16, g + 24; of row `lane` of the next tile
      auto load_bias = [&](int col0) {
        if (col0 >= a.N) return;
        const int c0 = min(col0 + lane, a.N - 1), c1 = min(col0 + 32 + lane, a.N - 1);
        if constexpr (SCALED<Tin>) {
          ws0 = a.w_scale[c0];
          if (CPP > 32) ws1 = a.w_scale[c1];
        }
        if (a.bias == nullptr) return;
        bias0 = a.bias[c0];
        if (CPP > 32) bias1 = a.bias[c1];
      };
      // The next piece of work with columns, found and its scales asked for while this one is drained.
      int m0 = 0, n0 = 0, width = 0, next_m0 = 0, next_n0 = 0, next_width = 0;
      auto find_next = [&](long long& t) {
        next_width = 0;
        for (; t < g.all && next_width == 0; t += pairs) piece_at(g, t, a.N, next_m0, next_n0, next_width);
        if (next_width > 0) next_m0 = next_m0 * 2 * LM + static_cast<int>(rank) * LM + quad * 32;
      };
      auto ask_next = [&]() {
        if (next_width == 0) return;
        load_bias(next_n0 + group * CPP);
        if constexpr (SCALED<Tin>)
          if (next_m0 < T) next_scale = a.a_scale[min(next_m0 + lane, T - 1)];
      };
      long long t_next = pair;
      find_next(t_next);
      ask_next();
      while (next_width > 0) {
        m0 = next_m0;
        n0 = next_n0;
        width = next_width;
        find_next(t_next);
        if constexpr (SCALED<Tin>) {
#pragma unroll
          for (int r = 0; r < 4; ++r) row_scale[r] = __shfl_sync(0xffffffffu, next_scale, (lane >> 2) + 8 * r);
        }
        const int cols = m0 < T ? min(width, a.N - n0) : 0; // columns of the tile to be written by this warp's rows
        // The tile's partial products, into registers: the sum of those before the last, fp32 outputs only.
        constexpr int SUMS = PARTS ? LN_PARTS / CPP / GROUPS : 1;
        float sum[SUMS][CPP] = {};
        for (int part = 0; part + 1 < parts && !bad; ++part, ++i) {
          if (!mbar_wait_limited<LIMIT>(bar(LB_ACC_FULL, i & 1), (i >> 1) & 1, abort_flag, a.wait_limit)) bad = true;
          bad = __any_sync(0xffffffffu, bad);
          if (bad) break;
          tc_fence_after();
          if constexpr (PARTS) {
#pragma unroll
            for (int y = 0; y < SUMS; ++y) {
              if ((group + GROUPS * y) * CPP < cols) {
                float v[CPP];
                const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (i & 1) * LN_MAX + (group + GROUPS * y) * CPP;
                if constexpr (SCALED<Tin>) tmem_ld_fragments<CPP>(at, v);
                else tmem_ld32(at, v);
#pragma unroll
                for (int k = 0; k < CPP; ++k) sum[y][k] += v[k];
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty[i & 1]);
        }
        if (bad) break;
        const uint32_t b = i & 1;
        if (!mbar_wait_limited<LIMIT>(bar(LB_ACC_FULL, b), (i >> 1) & 1, abort_flag, a.wait_limit)) bad = true;
        bad = __any_sync(0xffffffffu, bad);
        if (bad) break;
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(b) * LN_MAX;
        const int cc = lane & (CHUNKS - 1);              // this lane's 16-byte chunk of a row piece
        auto row_of = [&](int r) { return (32 / CHUNKS) * r + lane / CHUNKS; };
        // Piece p in fragments (8 bits); PARTS: v holds the sum of the parts before the last.
        auto piece_scaled = [&](int p, auto& v) {
          constexpr int E = static_cast<int>(sizeof(Tout)), ROW = 16 * CHUNKS;
          const int col0 = n0 + p * CPP, g = lane >> 2, q = lane & 3;
          const bool col_ok = col0 + cc * Ch::N < a.N;
          uint4 res[CHUNKS];
          if (a.residual != nullptr) {
            const Tout* from = static_cast<const Tout*>(a.residual) + (col_ok ? col0 + cc * Ch::N : 0);
#pragma unroll
            for (int r = 0; r < CHUNKS; ++r)
              res[r] = *reinterpret_cast<const uint4*>(from + static_cast<size_t>(min(m0 + row_of(r), T - 1)) * a.N);
          }
          // Scales and bias from a column per lane to the lanes that have it in their fragments.
          st_shared_u32(stg + lane * 4, __float_as_uint(ws0));
          st_shared_u32(stg + 256 + lane * 4, __float_as_uint(bias0));
          if (CPP > 32) {
            st_shared_u32(stg + 128 + lane * 4, __float_as_uint(ws1));
            st_shared_u32(stg + 384 + lane * 4, __float_as_uint(bias1));
          }
          const bool more = (p + GROUPS) * CPP < cols;
          if (more) load_bias(n0 + (p + GROUPS) * CPP);
          else ask_next();
          if constexpr (PARTS) {
            float last[CPP];
            tmem_ld_fragments<CPP>(taddr + p * CPP, last);
#pragma unroll
            for (int k = 0; k < CPP; ++k) v[k] += last[k];
          } else {
            tmem_ld_fragments<CPP>(taddr + p * CPP, v);
          }
          tc_fence_before();
          __syncwarp();
          if (!more && lane == 0) mbar_arrive_cluster(acc_empty[b]);   // this warp's share of the accumulator is in registers
          const uint32_t at_col = stg + 8 * q;
#pragma unroll
          for (int n = 0; n < CPP / 8; ++n) {
            uint64_t w, bb;
            asm volatile("ld.shared.b64 %0, [%1];" : "=l"(w) : "r"(at_col + 32 * n) : "memory");
            asm volatile("ld.shared.b64 %0, [%1];" : "=l"(bb) : "r"(at_col + 256 + 32 * n) : "memory");
#pragma unroll
            for (int r = 0; r < 4; ++r) {                // row g + 8 r
              float* x = v + (r >> 1) * (CPP / 2) + 4 * n + 2 * (r & 1);
              const float2 y = halves_f2(fma_pair(mul_pair(pair_f2(x[0], x[1]), w), pair_f2(row_scale[r], row_scale[r]), bb));
              x[0] = y.x;
              x[1] = y.y;
            }
          }
          __syncwarp();
          if (act != RRA_ACT_NONE) activate(v, act);
          // Fragment (r, n)'s place in the staging: rows 8 apart are turned alike, so the places of a chunk differ by 8 rows.
          uint32_t place[CPP / 8];
#pragma unroll
          for (int n = 0; n < CPP / 8; ++n) {
            const int byte = (8 * n + 2 * q) * E;
            place[n] = stg + g * ROW + (((byte >> 4) ^ g) << 4) + (byte & 15);
          }
          if (a.residual != nullptr) {
#pragma unroll
            for (int r = 0; r < CHUNKS; ++r) st_shared_v4(staged(row_of(r), cc), res[r].x, res[r].y, res[r].z, res[r].w);
            __syncwarp();
#pragma unroll
            for (int n = 0; n < CPP / 8; ++n) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float* x = v + (r >> 1) * (CPP / 2) + 4 * n + 2 * (r & 1);
                add_two(x[0], x[1], place[n] + 8 * r * ROW, Tout());
              }
            }
          }
#pragma unroll
          for (int n = 0; n < CPP / 8; ++n) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float* x = v + (r >> 1) * (CPP / 2) + 4 * n + 2 * (r & 1);
              put_two(place[n] + 8 * r * ROW, x[0], x[1], Tout());
            }
          }
          __syncwarp();
          Tout* to = static_cast<Tout*>(a.c) + static_cast<size_t>(m0 + lane / CHUNKS) * a.N + col0 + cc * Ch::N;
          const size_t down = static_cast<size_t>(32 / CHUNKS) * a.N;
#pragma unroll
          for (int r = 0; r < CHUNKS; ++r) {
            const uint4 w = ld_shared_v4(staged(row_of(r), cc));
            if (col_ok && m0 + row_of(r) < T) *reinterpret_cast<uint4*>(to) = w;
            to += down;
          }
          __syncwarp();                                  // read back before the next piece is written
        };
        // Piece p; PARTS: v holds the sum of the parts before the last.
        auto piece = [&](int p, auto& v) {
          const int col0 = n0 + p * CPP;
          const bool col_ok = col0 + cc * Ch::N < a.N;   // N is a multiple of 8: chunks are whole
          auto at = [&](int r) { return static_cast<size_t>(m0 + r) * a.N + col0 + cc * Ch::N; };
          uint4 res[CHUNKS];
          auto fetch_residual = [&]() {
            if (a.residual == nullptr) return;
            // Past T or N: some element that is in use, for outputs that are not stored.
            const Tout* from = static_cast<const Tout*>(a.residual) + (col_ok ? col0 + cc * Ch::N : 0);
#pragma unroll
            for (int r = 0; r < CHUNKS; ++r)
              res[r] = *reinterpret_cast<const uint4*>(from + static_cast<size_t>(min(m0 + row_of(r), T - 1)) * a.N);
          };
          if constexpr (PARTS) {
            float last[CPP];
            tmem_ld32(taddr + p * CPP, last);
#pragma unroll
            for (int k = 0; k < CPP; ++k) v[k] += last[k];
            fetch_residual();                            // behind the sums: the registers
          } else {
            fetch_residual();
#pragma unroll
            for (int q = 0; q < CPP / 32; ++q) tmem_ld32(taddr + p * CPP + q * 32, v + q * 32);
          }
          if ((p + GROUPS) * CPP >= cols) {
            // This warp's share of the accumulator is in registers: the products of tile i + 2 may overwrite it.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty[b]);
          }
          if (a.bias != nullptr) {
            // From a column per lane to every lane through the staging rows (16
            // broadcast loads from global memory came one after another: 3600 cycles a piece).
            st_shared_u32(stg + lane * 4, __float_as_uint(bias0));
            if (CPP > 32) st_shared_u32(stg + 128 + lane * 4, __float_as_uint(bias1));
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CPP / 4; ++j) {
              const uint4 bb = ld_shared_v4(stg + 16 * j);
              v[4 * j] += __uint_as_float(bb.x);
              v[4 * j + 1] += __uint_as_float(bb.y);
              v[4 * j + 2] += __uint_as_float(bb.z);
              v[4 * j + 3] += __uint_as_float(bb.w);
            }
            __syncwarp();
          }
          if ((p + GROUPS) * CPP < cols) load_bias(n0 + (p + GROUPS) * CPP);
          else ask_next();
          activate(v, act);
          if (a.residual != nullptr) {
            // The residual turns from row pieces into rows through the staging rows.
#pragma unroll
            for (int r = 0; r < CHUNKS; ++r) st_shared_v4(staged(row_of(r), cc), res[r].x, res[r].y, res[r].z, res[r].w);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) Ch::add(v + j * Ch::N, ld_shared_v4(staged(lane, j)));
          }
#pragma unroll
          for (int j = 0; j < CHUNKS; ++j) {
            const uint4 w = Ch::pack(v + j * Ch::N);
            st_shared_v4(staged(lane, j), w.x, w.y, w.z, w.w);
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < CHUNKS; ++r) {
            const int rr = row_of(r);
            const uint4 w = ld_shared_v4(staged(rr, cc));
            if (col_ok && m0 + rr < T) *reinterpret_cast<uint4*>(static_cast<Tout*>(a.c) + at(rr)) = w;
          }
          __syncwarp();                                  // read back before the next piece is written
        };
        if constexpr (PARTS) {
#pragma unroll
          for (int y = 0; y < SUMS; ++y)
            if ((group + GROUPS * y) * CPP < cols) {
              if constexpr (SCALED<Tin>) piece_scaled(group + GROUPS * y, sum[y]);
              else piece(group + GROUPS * y, sum[y]);
            }
        } else {
#pragma unroll 1
          for (int p = group; p * CPP < cols; p += GROUPS) {
            float v[CPP];
            if constexpr (SCALED<Tin>) piece_scaled(p, v);
            else piece(p, v);
          }
        }
        if (group * CPP >= cols) {                       // no piece for this warp
          if (lane == 0) mbar_arrive_cluster(acc_empty[b]);
          ask_next();
        }
        ++i;
      }
    }
    if (bad && lane == 0) {
      st_shared_u32(abort_flag, 1u);
      st_cluster_u32(map_rank(abort_flag, rank ^ 1u), 1u);
      record_error(a.err, RRA_DEVERR_WAIT_TIMEOUT);
    }
  }

  // Teardown: after an abort, copies and products still in flight get a
  // bounded grace period (~1 ms) to land before the TMEM is released.
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && ld_shared_volatile_u32(abort_flag) != 0u) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000LL) {
    }
  }
  __syncthreads();
  cluster_sync_all();                                    // the peer's copies, arrivals and products are done too
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L_TMEM_COLS) : "memory");
}

// ------------------------------------------------------------- medium rows

constexpr int M_ROWS = 256;                              // most rows of a in a tile
constexpr int M_SPLIT = 8;                               // most CTAs of a cluster
constexpr int M_THREADS = 320;                           // warp 0 loads, warp 1 products, warps 2-9 epilogue
constexpr int M_MAX_STAGES = 9;
template <bool HALF> constexpr uint32_t M_RING_BYTES = (HALF ? 96 : 192) * 1024;   // 3 (HALF) or 4 to 9 stages; then the partial sums
constexpr uint32_t M_W_BYTES = 128 * 128;
template <bool HALF> constexpr uint32_t M_OFF_BAR = M_RING_BYTES<HALF>;
constexpr uint32_t MB_FULL = 0, MB_EMPTY = 8 * M_MAX_STAGES, MB_DONE = 16 * M_MAX_STAGES;
constexpr uint32_t MW_TMEM = MB_DONE + 8, MW_ABORT = MW_TMEM + 4;
constexpr uint32_t MB_ACC_FULL = MW_ABORT + 4, MB_ACC_EMPTY = MB_ACC_FULL + 32;   // [4] each, fp32 outputs
static_assert(MB_ACC_FULL % 8 == 0 && MB_ACC_EMPTY + 32 <= 256, "barriers behind the ring");
template <bool HALF> constexpr uint32_t M_SMEM = M_OFF_BAR<HALF> + 256;
// Accumulators of 128 (or 256) columns that share K.  fp32 outputs (see L_PART): parts of 8 chunks take them in turn, and
// the epilogue warps add each finished part to their sums in registers while the next ones run (256 rows of 16384 -> 4096
// 37.5 us; 16-bit outputs 37.2).  16-bit outputs: one part of K each, added at the end.
template <bool HALF> constexpr int M_TMEM_COLS = HALF ? 256 : 512;

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr));
  return v;
}

// Four neighbouring outputs: + residual, one rounding.
__device__ __forceinline__ void finish4(float* c, const float* residual, float4 v) {
  if (residual != nullptr) {
    const float4 r = *reinterpret_cast<const float4*>(residual);
    v = make_float4(v.x + r.x, v.y + r.y, v.z + r.z, v.w + r.w);
  }
  *reinterpret_cast<float4*>(c) = v;
}
template <typename T>
__device__ __forceinline__ void finish4(T* c, const T* residual, float4 v) {
  float x[8] = {v.x, v.y, v.z, v.w, 0.f, 0.f, 0.f, 0.f};
  if (residual != nullptr) {
    const uint2 r = *reinterpret_cast<const uint2*>(residual);
    Chunk<T>::add(x, make_uint4(r.x, r.y, 0u, 0u));
  }
  const uint4 w = Chunk<T>::pack(x);
  *reinterpret_cast<uint2*>(c) = make_uint2(w.x, w.y);
}

// One cluster: `row_step` rows by 128 columns of c; its CTAs share K.  D[n, t] = sum_k W[n, k] a[t, k].
// HALF: two CTAs an SM, for up to 128 rows.
template <typename Tin, typename Tout, bool LIMIT, bool HALF>
__global__ void __launch_bounds__(M_THREADS, HALF ? 2 : 1)
    linear_mid_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                      const LinearEpiArgs a, int act, int splits, int row_step) {
  constexpr bool PARTS = sizeof(Tout) == 4;
  extern __shared__ __align__(1024) uint8_t smem_mid[];
  const uint32_t base = smem_u32(smem_mid), bars = base + M_OFF_BAR<HALF>;
  auto bar = [&](uint32_t kind, uint32_t i) { return bars + kind + 8 * i; };
  const uint32_t abort_flag = bars + MW_ABORT;
  const volatile uint32_t* tmem_ptr = reinterpret_cast<const volatile uint32_t*>(smem_mid + M_OFF_BAR<HALF> + MW_TMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % splits, tile = static_cast<int>(blockIdx.x) / splits;
  const int ntiles = (a.N + 127) / 128, n0 = tile % ntiles * 128, t0 = tile / ntiles * row_step;
  if (warp == 1) {
    tmem_alloc(bars + MW_TMEM, M_TMEM_COLS<HALF>);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < M_MAX_STAGES; ++s) {
      mbar_init(bar(MB_FULL, s), 1);
      mbar_init(bar(MB_EMPTY, s), 1);
    }
    mbar_init(bar(MB_DONE, 0), 1);
    if constexpr (PARTS) {
      for (int i = 0; i < 4; ++i) {
        mbar_init(bar(MB_ACC_FULL, i), 1);
        mbar_init(bar(MB_ACC_EMPTY, i), M_THREADS / 32 - 2);
      }
    }
    st_shared_u32(abort_flag, 0u);
    fence_barrier_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_w);
  }
  tc_fence_before();
  __syncthreads();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");   // this CTA's words are set; waited for ahead of the join
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  dependent_launch();
  const int T = a.cu[a.B];
  const bool valid = T >= 0 && T <= a.cap;
  if (!valid && blockIdx.x == 0 && tid == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
  const int rows = valid ? max(0, min(T - t0, row_step)) : 0, boxes = (rows + 31) / 32, cols = (rows + 15) & ~15;
  const uint32_t stage_bytes = M_W_BYTES + static_cast<uint32_t>(boxes) * 4096u;
  const uint32_t stages = min(static_cast<uint32_t>(M_MAX_STAGES), M_RING_BYTES<HALF> / stage_bytes);
  const int kchunks = (a.K + LK<Tin> - 1) / LK<Tin>;
  const int k_from = static_cast<int>(static_cast<long long>(kchunks) * rank / splits);
  const int k_to = rows > 0 ? static_cast<int>(static_cast<long long>(kchunks) * (rank + 1) / splits) : k_from;
  const int part_cols = cols > 128 ? 256 : 128;
  const int slots = M_TMEM_COLS<HALF> / part_cols, wanted = max(1, (k_to - k_from + L_PART - 1) / L_PART);
  const int parts = PARTS ? wanted : min(slots, wanted);
  const int per_part = (k_to - k_from + parts - 1) / parts;
  bool bad = false;
  if (warp == 0) {
    // -------------------------------------------------------------- loads
    if (elect_one()) {
      uint32_t s = 0, lap = 0;
      for (int kc = k_from; kc < k_to; ++kc) {
        if (lap > 0 && !mbar_wait_limited<LIMIT>(bar(MB_EMPTY, s), (lap - 1) & 1, abort_flag, a.wait_limit)) {
          bad = true;
          break;
        }
        const uint32_t dst = base + s * stage_bytes;
        mbar_expect_tx(bar(MB_FULL, s), stage_bytes);
        tma_load_2d(dst, &map_w, kc * LK<Tin>, n0, bar(MB_FULL, s));          // rows past N, columns past K: zeros
        for (int b = 0; b < boxes; ++b) tma_load_2d(dst + M_W_BYTES + b * 4096, &map_a, kc * LK<Tin>, t0 + 32 * b, bar(MB_FULL, s));
        if (++s == stages) {
          s = 0;
          ++lap;
        }
      }
    }
    bad = __any_sync(0xffffffffu, bad);
  } else if (warp == 1) {
    // ----------------------------------------------------------- products
    if (elect_one()) {
      const uint32_t idesc = idesc_in<Tin>(128, cols);
      const uint64_t dw0 = sdesc(base, 16, 1024), dx0 = sdesc(base + M_W_BYTES, 16, 1024);
      uint32_t s = 0, lap = 0;
      int slot = 0, turn = 0, at = 0;                    // accumulator, times round them, chunks of its part so far
      for (int kc = k_from; kc < k_to; ++kc) {
        if (!mbar_wait_limited<LIMIT>(bar(MB_FULL, s), lap & 1, abort_flag, a.wait_limit)) {
          bad = true;
          break;
        }
        if (PARTS && at == 0 && turn > 0 && !mbar_wait_limited<LIMIT>(bar(MB_ACC_EMPTY, slot), (turn - 1) & 1, abort_flag, a.wait_limit)) {
          bad = true;
          break;
        }
        tc_fence_after();
        const uint64_t off = s * (stage_bytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t add = (at > 0 || kk > 0) ? 1u : 0u;
          if constexpr (SCALED<Tin>) umma_f8(tmem + slot * part_cols, dw0 + off + 2 * kk, dx0 + off + 2 * kk, idesc, add);
          else umma_f16(tmem + slot * part_cols, dw0 + off + 2 * kk, dx0 + off + 2 * kk, idesc, add);
        }
        umma_commit(bar(MB_EMPTY, s));
        if (++at == per_part || kc + 1 == k_to) {
          if (PARTS) umma_commit(bar(MB_ACC_FULL, slot));
          at = 0;
          if (++slot == slots) {
            slot = 0;
            ++turn;
          }
        }
        if (++s == stages) {
          s = 0;
          ++lap;
        }
      }
      if (!bad) umma_commit(bar(MB_DONE, 0));
    }
    bad = __any_sync(0xffffffffu, bad);
  }
  // fp32: this warp's share of each part, as it finishes, into sums: rows of W by lane, 16 rows of a at 32 y.
  constexpr int MOST = HALF ? M_ROWS / 2 : M_ROWS;       // rows of a tile (sums for 256 spilled in the form of two CTAs an SM)
  float sum[PARTS ? MOST / 32 : 1][16] = {};
  const int half16 = ((warp - 2) >> 2) * 16;
  if (PARTS && warp >= 2) {
    const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half16;
    int slot = 0, turn = 0;
    for (int k = k_from; k < k_to; k += per_part) {
      if (!mbar_wait_limited<LIMIT>(bar(MB_ACC_FULL, slot), turn & 1, abort_flag, a.wait_limit)) bad = true;
      bad = __any_sync(0xffffffffu, bad);
      if (bad) break;
      tc_fence_after();
#pragma unroll
      for (int y = 0; y < MOST / 32; ++y) {
        if (half16 + 32 * y < cols) {
          float x[16];
          tmem_ld16(at + slot * part_cols + 32 * y, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[PARTS ? y : 0][i] += x[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(MB_ACC_EMPTY, slot));
      if (++slot == slots) {
        slot = 0;
        ++turn;
      }
    }
  }
  // Every warp: the products are done (and with them every copy has been read).
  if (!bad && !mbar_wait_limited<LIMIT>(bar(MB_DONE, 0), 0, abort_flag, a.wait_limit)) bad = true;
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) {
    st_shared_u32(abort_flag, 1u);
    record_error(a.err, RRA_DEVERR_WAIT_TIMEOUT);
  }
  __syncthreads();
  const bool aborted = ld_shared_volatile_u32(abort_flag) != 0u;
  if (aborted && tid == 0) {
    const long long t0 = clock64();                      // copies and products still in flight land
    while (clock64() - t0 < 2000000LL) {
    }
  }
  __syncthreads();
  if constexpr (SCALED<Tin>) {
    if (splits == 1) {
      // A tile of one CTA has no sums to join: from the accumulators to c, a column a lane, 16 rows at a time, not by way
      // of the ring (64 rows of 4096 -> 16384: 17.5 -> 16.3 us, with a residual and SiLU 21.1 -> 18.5).
      if (warp >= 2 && !aborted) {
        tc_fence_after();
        const int quad = warp & 3, n = n0 + quad * 32 + lane;
        const bool in = n < a.N;
        const float ws = in ? a.w_scale[n] : 0.f, bias = in && a.bias != nullptr ? a.bias[n] : 0.f;
#pragma unroll
        for (int y = 0; y < MOST / 32; ++y) {
          const int j = half16 + 32 * y;
          if (j < rows) {                                // (of the warp: TMEM is read by all of its lanes)
            const float sa = a.a_scale[t0 + min(j + (lane & 15), rows - 1)];
            float v[16];
            if constexpr (PARTS) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = sum[y][i];
            } else {
              tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + j, v);
              for (int p = 1; p < parts && p * per_part < k_to - k_from; ++p) {
                float x[16];
                tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + p * part_cols + j, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] += x[i];
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], __shfl_sync(0xffffffffu, sa, i) * ws, bias);
            activate(v, act);
            const size_t at = static_cast<size_t>(t0 + j) * a.N + n;
            if (a.residual != nullptr) {                 // (all 16 loads before the first store: c may be the residual)
              Tout x[16] = {};
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (in && j + i < rows) x[i] = static_cast<const Tout*>(a.residual)[at + static_cast<size_t>(i) * a.N];
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += static_cast<float>(x[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (in && j + i < rows) static_cast<Tout*>(a.c)[at + static_cast<size_t>(i) * a.N] = static_cast<Tout>(v[i]);
          }
        }
        tc_fence_before();
      }
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      __syncthreads();
      tc_fence_after();
      if (warp == 1) tmem_dealloc(tmem, M_TMEM_COLS<HALF>);
      return;
    }
  }
  // Partial sums [row of a][128] over the ring.
  if (warp >= 2 && !aborted && k_from < k_to) {
    tc_fence_after();
    const int quad = warp & 3, n = quad * 32 + lane;
    if constexpr (PARTS) {
#pragma unroll
      for (int y = 0; y < MOST / 32; ++y) {
        if (half16 + 32 * y < cols) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            st_shared_u32(base + static_cast<uint32_t>((half16 + 32 * y + i) * 128 + n) * 4u, __float_as_uint(sum[y][i]));
        }
      }
    }
    for (int j = half16; !PARTS && j < cols; j += 32) {
      float v[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + j, v);
      for (int p = 1; p < parts && p * per_part < k_to - k_from; ++p) {
        float x[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + p * part_cols + j, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += x[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) st_shared_u32(base + static_cast<uint32_t>((j + i) * 128 + n) * 4u, __float_as_uint(v[i]));
    }
    tc_fence_before();
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (aborted && tid < splits) st_cluster_u32(map_rank(abort_flag, static_cast<uint32_t>(tid)), 1u);
  __syncwarp();
  cluster_sync_all();
  // Four neighbouring outputs a thread, two such at a time, the cluster's rows
  // shared out, sums in rank order.  Where a CTA gave up, its ring holds no sums: the tile is not written.
  const int step = splits * M_THREADS;
  const bool gave_up = ld_shared_volatile_u32(abort_flag) != 0u;
  for (int e0 = rank * M_THREADS + tid; !gave_up && e0 < rows * 32; e0 += 2 * step) {
    float4 y[2][M_SPLIT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = min(e0 + u * step, rows * 32 - 1);
      const uint32_t at = base + static_cast<uint32_t>((e >> 5) * 128 + 4 * (e & 31)) * 4u;
#pragma unroll
      for (int p = 0; p < M_SPLIT; ++p)
        if (p < splits) y[u][p] = ld_cluster4(map_rank(at, static_cast<uint32_t>(p)));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = e0 + u * step, t = e >> 5, n = n0 + 4 * (e & 31);
      if (e >= rows * 32 || n >= a.N) continue;          // N is a multiple of 8: whole quads
      float v[4] = {y[u][0].x, y[u][0].y, y[u][0].z, y[u][0].w};
#pragma unroll
      for (int p = 1; p < M_SPLIT; ++p) {
        if (p < splits) {
          v[0] += y[u][p].x;
          v[1] += y[u][p].y;
          v[2] += y[u][p].z;
          v[3] += y[u][p].w;
        }
      }
      if constexpr (SCALED<Tin>) {
        const float4 ws = *reinterpret_cast<const float4*>(a.w_scale + n);
        const float sa = a.a_scale[t0 + t];
        v[0] *= sa * ws.x;
        v[1] *= sa * ws.y;
        v[2] *= sa * ws.z;
        v[3] *= sa * ws.w;
      }
      if (a.bias != nullptr) {
        const float4 b = *reinterpret_cast<const float4*>(a.bias + n);
        v[0] += b.x;
        v[1] += b.y;
        v[2] += b.z;
        v[3] += b.w;
      }
      activate(v, act);
      const size_t o = static_cast<size_t>(t0 + t) * a.N + n;
      finish4(static_cast<Tout*>(a.c) + o, a.residual != nullptr ? static_cast<const Tout*>(a.residual) + o : nullptr,
              make_float4(v[0], v[1], v[2], v[3]));
    }
  }
  cluster_sync_all();                                    // no CTA leaves while another may still read its sums
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, M_TMEM_COLS<HALF>);
}

// ------------------------------------------------------------------ few rows

constexpr int FEW_WARPS = 8, FEW_PART = 4;
// Steps of 32 in K in flight per warp: about 96 KB a CTA, two CTAs an SM.
template <int NT> struct FewCfg {
  static constexpr int U = NT == 1 ? 8 : (NT == 2 ? 6 : 4);
  static constexpr int SMEM = U * (2 + NT) * FEW_WARPS * 32 * 16;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_fp8_e4m3) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// NT: groups of 8 rows of a.  One CTA: 16 columns of c.
template <typename Tin, typename Tout, int NT>
__global__ void __launch_bounds__(32 * FEW_WARPS) linear_few_kernel(const LinearEpiArgs a, int act) {
  constexpr int U = FewCfg<NT>::U;
  __shared__ float part[FEW_WARPS][16][NT * 8 + 1];
  extern __shared__ __align__(16) uint8_t smem_few[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int n0 = static_cast<int>(blockIdx.x) * 16;
  dependent_launch();
  // Needed at the end only: rows of a from T to cap are multiplied too (each gives its
  // own outputs, which are not stored), so that no copy waits for T.
  const int T = a.cu[a.B];
  const Tin* W = static_cast<const Tin*>(a.w);
  const Tin* X = static_cast<const Tin*>(a.a);
  // Rows past N repeat the last one, rows past cap are zeros: their results are not stored.
  const Tin* w0 = W + static_cast<size_t>(min(n0 + g, a.N - 1)) * a.K;
  const Tin* w1 = W + static_cast<size_t>(min(n0 + g + 8, a.N - 1)) * a.K;
  const Tin* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = X + static_cast<size_t>(min(8 * t + g, a.cap - 1)) * a.K;
  // Sums of the products, in parts of FEW_PART steps (see L_PART) added up in sum.
  float d[NT][4], sum[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int j = 0; j < 4; ++j) d[t][j] = sum[t][j] = 0.f;
  }
  // Steps of 64 bytes in K (32 elements, 64 in 8 bits), taken by the warps in turn.  Each lane copies its own
  // chunks into its own slots of shared memory and reads them back, U steps
  // later: no other lane waits for them, and the copies in flight need no
  // registers (as register loads the compiler kept one step in flight).
  const uint32_t slot = smem_u32(smem_few) + static_cast<uint32_t>(threadIdx.x) * 16u;
  auto chunk = [&](int u, int j) { return slot + static_cast<uint32_t>((u * (2 + NT) + j) * FEW_WARPS * 32) * 16u; };
  // A warp takes pairs of steps (whole 128-byte lines of W), starting at a
  // place that differs from CTA to CTA: all CTAs read the same rows of a, and
  // in step they would all ask one L2 line at a time.
  constexpr int E16 = 16 / static_cast<int>(sizeof(Tin));   // elements of a 16-byte chunk
  const int units = (a.K + LK<Tin> - 1) / LK<Tin>, mine = 2 * ((units - warp + FEW_WARPS - 1) / FEW_WARPS);
  const int turn = mine > 0 ? 2 * (static_cast<int>(blockIdx.x) % (mine / 2)) : 0;
  auto k_of = [&](int i) {
    int j = i + turn;
    if (j >= mine) j -= mine;
    return (warp + (j >> 1) * FEW_WARPS) * LK<Tin> + (j & 1) * (LK<Tin> / 2) + q * E16;
  };
  auto fetch = [&](int i, int u) {
    // K is a multiple of 16 bytes: chunks are whole; past K the last one is copied and counts as zero.
    const int k = min(k_of(i), a.K - E16);
    cp_async16(chunk(u, 0), w0 + k);
    cp_async16(chunk(u, 1), w1 + k);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (8 * t + g < a.cap) cp_async16(chunk(u, 2 + t), x[t] + k);
  };
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (i < mine) fetch(i, i);
    cp_async_commit();
  }
  int u = 0;
  for (int i = 0; i < mine; ++i) {
    cp_async_wait<U - 1>();
    const bool in = k_of(i) < a.K;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4 va = in ? ld_shared_v4(chunk(u, 0)) : z, vb = in ? ld_shared_v4(chunk(u, 1)) : z;
    uint4 vx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) vx[t] = in && 8 * t + g < a.cap ? ld_shared_v4(chunk(u, 2 + t)) : z;
    if (i + U < mine) fetch(i + U, u);
    cp_async_commit();
    if (++u == U) u = 0;
    const uint32_t lo[4] = {va.x, vb.x, va.y, vb.y}, hi[4] = {va.z, vb.z, va.w, vb.w};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mma_16816(d[t], lo, vx[t].x, vx[t].y, Tin());
      mma_16816(d[t], hi, vx[t].z, vx[t].w, Tin());
    }
    if (i % FEW_PART == FEW_PART - 1 || i + 1 == mine) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[t][j] += d[t][j];
          d[t][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    part[warp][g][8 * t + 2 * q] = sum[t][0];
    part[warp][g][8 * t + 2 * q + 1] = sum[t][1];
    part[warp][g + 8][8 * t + 2 * q] = sum[t][2];
    part[warp][g + 8][8 * t + 2 * q + 1] = sum[t][3];
  }
  __syncthreads();
  if (T < 0 || T > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
    return;
  }
  for (int e = threadIdx.x; e < 16 * NT * 8; e += 32 * FEW_WARPS) {
    const int j = e & 15, t = e >> 4, n = n0 + j;
    if (t >= T || n >= a.N) continue;
    float v[1] = {0.f};
#pragma unroll
    for (int w = 0; w < FEW_WARPS; ++w) v[0] += part[w][j][t];
    if constexpr (SCALED<Tin>) v[0] *= a.a_scale[t] * a.w_scale[n];
    if (a.bias != nullptr) v[0] += a.bias[n];
    activate(v, act);
    const size_t at = static_cast<size_t>(t) * a.N + n;
    if (a.residual != nullptr) v[0] += static_cast<float>(static_cast<const Tout*>(a.residual)[at]);
    static_cast<Tout*>(a.c)[at] = static_cast<Tout>(v[0]);
  }
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 linear_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D map over a row-major [rows, K] matrix: box = 128 bytes of columns x box_rows rows,
// 128-byte swizzle (the canonical K-major operand layout).
template <typename Tin>
cudaError_t make_map_2d(CUtensorMap* map, const void* ptr, long long rows, int K, uint32_t box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * sizeof(Tin)};
  cuuint32_t box[2] = {LK<Tin>, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if constexpr (!SCALED<Tin>)
    type = IsBf16<Tin>::value == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUresult r = linear_encode_fn()(map, type, 2,
                                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launched as a programmatic dependent: the set-up overlaps the tail of the
// kernel before it in the stream, whose completion the kernels wait for
// before touching global memory.
cudaLaunchConfig_t dependent_config(cudaLaunchAttribute* attr, int grid, int threads, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Once per device and kernel (the template arguments name the kernel; NT: groups of rows, or below 0 the kernel's variant): its dynamic shared memory.
template <typename Tin, typename Tout, int NT, typename K>
cudaError_t allow_smem(K kernel, int bytes) {
  constexpr int kMaxDevices = 64;
  static bool attr_set[kMaxDevices] = {};
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(m);
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  return cudaSuccess;
}

template <typename Tin, typename Tout, bool PARTS, bool LIMIT>
cudaError_t launch_pair(const LinearEpiArgs& a, int act, int num_sms, cudaStream_t stream) {
  if (linear_encode_fn() == nullptr) return cudaErrorNotSupported;
  auto kernel = linear_pair_kernel<Tin, Tout, PARTS, LIMIT>;
  cudaError_t e = allow_smem<Tin, Tout, -1 - PARTS - 2 * LIMIT>(kernel, L_SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap ma, mw[3];
  if ((e = make_map_2d<Tin>(&ma, a.a, a.cap, a.K, LM)) != cudaSuccess) return e;
  for (int i = 0; i < 3; ++i)
    if ((e = make_map_2d<Tin>(&mw[i], a.w, a.N, a.K, 128u >> i)) != cudaSuccess) return e;
  const long long most = ((a.cap + 2LL * LM - 1) / (2 * LM)) * ((a.N + 63LL) / 64);   // tiles if every row is in use
  const int pairs = static_cast<int>(most < num_sms / 2 ? most : num_sms / 2);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = dependent_config(&attr, 2 * (pairs > 0 ? pairs : 1), L_THREADS, L_SMEM, stream);
  return cudaLaunchKernelEx(&cfg, kernel, ma, mw[0], mw[1], mw[2], a, act);
}

// How linear_mid_kernel cuts its work: tiles of row_step rows by 128 columns, K of each split while the clusters run
// at once (of 152 SMs clusters of 4 find room on 144, of 8 on 120) and each CTA keeps two chunks of 64; and about what it takes, in cycles: per step of 16 in K 64 +
// rows/2 for the shared memory that the products read, and some 36 a row for joining the sums.
struct MidCut {
  int splits, row_step;
  long long ctas, cycles;
};
MidCut cut_mid(const LinearEpiArgs& a, int kchunks, int num_sms) {
  MidCut m;
  const long long row_tiles = (a.cap - 1LL) / M_ROWS + 1, tiles = row_tiles * ((a.N + 127) / 128);
  m.row_step = static_cast<int>((a.cap + row_tiles - 1) / row_tiles + 15) & ~15;
  m.splits = 1;
  const int at_once[] = {num_sms, num_sms * 18 / 19, num_sms * 15 / 19};  // clusters of 2, 4, 8
  for (const int room : at_once)
    if (m.splits < M_SPLIT && 2 * m.splits * tiles <= room && kchunks >= 4 * m.splits) m.splits *= 2;
  m.ctas = tiles * m.splits;
  m.cycles = (4LL * ((kchunks + m.splits - 1) / m.splits) * (64 + m.row_step / 2) + 36 * m.row_step) *
             ((m.ctas + num_sms - 1) / num_sms);
  return m;
}

template <typename Tin, typename Tout, bool LIMIT, bool HALF>
cudaError_t launch_mid(const LinearEpiArgs& a, int act, const MidCut& cut, cudaStream_t stream) {
  if (linear_encode_fn() == nullptr) return cudaErrorNotSupported;
  auto kernel = linear_mid_kernel<Tin, Tout, LIMIT, HALF>;
  cudaError_t e = allow_smem<Tin, Tout, -5 - LIMIT - 2 * HALF>(kernel, M_SMEM<HALF>);
  if (e != cudaSuccess) return e;
  CUtensorMap ma, mw;
  if ((e = make_map_2d<Tin>(&ma, a.a, a.cap, a.K, 32)) != cudaSuccess) return e;
  if ((e = make_map_2d<Tin>(&mw, a.w, a.N, a.K, 128)) != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = dependent_config(attr, static_cast<int>(cut.ctas), M_THREADS, M_SMEM<HALF>, stream);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cut.splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mw, a, act, cut.splits, cut.row_step);
}

template <typename Tin, typename Tout, int NT>
cudaError_t launch_few(const LinearEpiArgs& a, int act, cudaStream_t stream) {
  auto kernel = linear_few_kernel<Tin, Tout, NT>;
  if (cudaError_t e = allow_smem<Tin, Tout, NT>(kernel, FewCfg<NT>::SMEM); e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      dependent_config(&attr, (a.N + 15) / 16, 32 * FEW_WARPS, FewCfg<NT>::SMEM, stream);
  return cudaLaunchKernelEx(&cfg, kernel, a, act);
}

template <typename Tin, typename Tout, bool LIMIT>
cudaError_t launch_tiles(const LinearEpiArgs& a, int act, int num_sms, cudaStream_t stream) {
  // The way that takes less, by the shared memory that the products read in turn (make_tiling's cost for pairs).
  // 4096 x 4096: 64 rows 11.2 us with W as the M operand against 16.6, 200 rows 15.6 / 16.1, 256 rows 17.4 / 16.3; 768 x
  // 2304: 64 rows 5.8 / 6.1, 128 rows 7.0 / 6.2; 16384 x 4096: 256 rows 36.7 / 48.3; 7440 x 72: 392 rows 12.4 / 23.8.
  // (Only where all of its clusters run at once: further rounds repeat a cluster's set-up.)
  const int kchunks = (a.K + LK<Tin> - 1) / LK<Tin>;
  const MidCut cut = cut_mid(a, kchunks, num_sms);
  const long long there = 4 * make_tiling(a.cap, a.N, num_sms / 2, LN_MAX).cost * kchunks;
  if (cut.cycles < there && (cut.ctas <= num_sms || a.cap <= M_ROWS)) {
    // In 8 bits, where several rounds of CTAs take turns on an SM, two at a time hide each other's set-up and output: 64 rows of
    // 4096 -> 32768 26.0 us against 31.9, in fp32 26.6 / 32.2 and with SiLU and a residual 29.4 / 37.1; 24 rows of 4096 -> 65536 46.7 /
    // 57.6, in fp32 47.5 / 58.3 (in one round one at a time: -> 16384 16.3, two 18.3).
    if constexpr (SCALED<Tin>)
      if (cut.ctas > num_sms && cut.row_step <= 128) return launch_mid<Tin, Tout, LIMIT, true>(a, act, cut, stream);
    return launch_mid<Tin, Tout, LIMIT, false>(a, act, cut, stream);
  }
  if constexpr (sizeof(Tout) == 4)
    if (kchunks > L_PART) return launch_pair<Tin, Tout, true, LIMIT>(a, act, num_sms, stream);
  return launch_pair<Tin, Tout, false, LIMIT>(a, act, num_sms, stream);
}

template <typename Tin, typename Tout>
cudaError_t launch_typed(const LinearEpiArgs& a, int act, int num_sms, cudaStream_t stream) {
  // In 8 bits W goes as the M operand too where 16 columns a CTA make more than 5 CTAs an SM, whose set-up in rounds then
  // outweighs that of the larger tiles (by columns / with W as the M operand, us; 8 rows of 1024 -> 8192 3.9 / 5.3, -> 12288
  // 5.3 / 5.2, -> 16384 6.7 / 5.4, -> 65536 29.6 / 17.8; of 4096 -> 9728 10.7 / 11.4, -> 16384 15.9 / 14.8; one row of 128 -> 16384
  // 5.1 / 5.5), and for 9 to 16 rows, which read as many bytes of a as of W, where W has more than 24 MB (16 rows of 4096
  // -> 9728 12.4 / 11.4, -> 4096 5.9 / 6.2).
  const bool by_columns = !SCALED<Tin> || (a.N <= 80LL * num_sms && (a.cap <= 8 || static_cast<long long>(a.N) * a.K <= 24LL << 20));
  if (a.cap <= 8 && by_columns) return launch_few<Tin, Tout, 1>(a, act, stream);
  if (a.cap <= 16 && by_columns) return launch_few<Tin, Tout, 2>(a, act, stream);
  return a.wait_limit > 0 ? launch_tiles<Tin, Tout, true>(a, act, num_sms, stream)
                          : launch_tiles<Tin, Tout, false>(a, act, num_sms, stream);
}

template <typename Tin>
cudaError_t launch_in(const LinearEpiArgs& a, rra_dtype out, int act, int num_sms, cudaStream_t stream) {
  if (out == RRA_BF16) return launch_typed<Tin, __nv_bfloat16>(a, act, num_sms, stream);
  if (out == RRA_F16) return launch_typed<Tin, __half>(a, act, num_sms, stream);
  return launch_typed<Tin, float>(a, act, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear_epilogue(const LinearEpiArgs& a, rra_dtype in, rra_dtype out, rra_activation act,
                                   int num_sms, cudaStream_t stream) {
  return in == RRA_BF16 ? launch_in<__nv_bfloat16>(a, out, act, num_sms, stream)
                        : launch_in<__half>(a, out, act, num_sms, stream);
}

cudaError_t launch_linear_scaled(const LinearEpiArgs& a, rra_dtype out, rra_activation act, int num_sms, cudaStream_t stream) {
  return launch_in<__nv_fp8_e4m3>(a, out, act, num_sms, stream);
}

}  // namespace rra
