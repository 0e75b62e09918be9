// Norms of queries and keys for each head, their rotation, and the write into
// a cache, in one pass over the tokens' head rows.
//
// For a head row x: inv = rsqrt(mean x^2 + eps) (1 without a norm), then for a
// pair (a, b) of the rotation: out_a = inv (x_a w_a cos - x_b w_b sin), out_b = inv (x_a w_a
// sin + x_b w_b cos).  With the weights and the rotation's scale folded into
// two coefficients per element, P (of the element) and Q (of its partner), a
// row costs one product and one multiply-add an element, two elements to an instruction.
//
// What bounds it is memory: each element is read once and written once.  A lane holds
// two chunks of 8 neighbouring elements (16-byte loads and stores) that are each
// other's partners in the half layout, so no element crosses lanes; a head row is 8
// (d = 128) or 4 (d = 64) lanes.  A warp takes a run of one token's heads, which share
// sines and cosines; several rows a lane are loaded before the first is used.  16411 tokens of
// 32 + 8 heads, d = 128: 59 us, 5.7 TB/s (one row at a time 80 us).
//
// Angles.  positions reach 2^24 and inv_freq is fp32, so an fp32 product loses
// the angle; it is reduced in turns instead: inv_freq / 2 pi as an unevaluated
// sum of two floats (Dekker's product, by fma), times the position (exact in
// fp32 below 2^24) again as two floats, minus the nearest integer.  The
// remainder in [-1/2, 1/2] turns is good to about 2^-24 of a turn.
#include "block.cuh"
#include "f32x2.cuh"

namespace rra {
namespace {

constexpr int R_WARPS = 4;       // of a CTA
// Rows a lane loads ahead, and CTAs an SM holds.
template <int D> struct RopeCfg {
  static constexpr int UNROLL = D == 128 ? 4 : 2, CTAS = D == 128 ? 4 : 5;
};

// cos and sin of pos * f.
__device__ __forceinline__ void rotation(float pos, float f, float& c, float& s) {
  constexpr double kTurn = 0.15915494309189533577;   // 1 / 2 pi
  constexpr float kHi = static_cast<float>(kTurn), kLo = static_cast<float>(kTurn - static_cast<double>(kHi));
  const float hi = f * kHi, lo = fmaf(f, kHi, -hi) + f * kLo;
  const float p = pos * hi, e = fmaf(pos, hi, -p) + pos * lo;
  const float r = (p - rintf(p)) + e;
  sincospif(2.f * r, &s, &c);
}

__device__ __forceinline__ uint64_t to_f2(uint32_t w, __nv_bfloat16) {
  return pair_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint64_t to_f2(uint32_t w, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair_f2(f.x, f.y);
}
__device__ __forceinline__ uint32_t from_f2(uint64_t v, __nv_bfloat16) {
  const float2 f = halves_f2(v);
  const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t from_f2(uint64_t v, __half) {
  const float2 f = halves_f2(v);
  const __half2 t = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ void load_weights(const float* w, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(w), y = reinterpret_cast<const float4*>(w)[1];
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

// A token's warps-full of heads are numbered queries, keys, values; a job is
// `iters` of them in a row, `jobs` of them a token.
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * R_WARPS, RopeCfg<D>::CTAS) qk_norm_rope_kernel(const NormRopeArgs a, int iters, int jobs) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;    // lanes of a head row, heads of a warp
  constexpr int U = RopeCfg<D>::UNROLL;
  const int lane = threadIdx.x & 31, p = lane % LPH, sub = lane / LPH;
  dependent_launch();
  const int rows_used = a.cu[a.B];
  if (rows_used < 0 || rows_used > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
    return;
  }
  // The lane's two chunks.  Half layout: elements 8p .. of the first half and
  // of the second; interleaved, and behind the rotated part: neighbours.
  const int half = a.rot / 2;
  const bool turned = 16 * p < a.rot, all_turned = a.rot == D;
  const int c0 = INTERLEAVED || !turned ? 16 * p : 8 * p, c1 = INTERLEAVED || !turned ? c0 + 8 : c0 + half;
  auto partner_of = [](const uint64_t (&v)[8], int j) {
    if constexpr (!INTERLEAVED) return v[j ^ 4];
    const float2 f = halves_f2(v[j]);
    return pair_f2(f.y, f.x);
  };
  const int full_q = (a.Hq + HPW - 1) / HPW, full_k = (a.Hkv + HPW - 1) / HPW;
  const int ends[3] = {full_q, full_q + full_k, full_q + 2 * full_k};
  const long long all = static_cast<long long>(rows_used) * jobs, step = static_cast<long long>(gridDim.x) * R_WARPS;
  for (long long job = static_cast<long long>(blockIdx.x) * R_WARPS + (threadIdx.x >> 5); job < all; job += step) {
    const long long t = job / jobs;
    const int from = static_cast<int>(job % jobs) * iters;
    const int to = min(from + iters, ends[a.v_out != nullptr ? 2 : 1]);
    auto input = [&](int kind) {
      return kind == 0 ? static_cast<const T*>(a.q) + t * a.q_stride
                       : (kind == 1 ? static_cast<const T*>(a.k) + t * a.k_stride
                                    : static_cast<const T*>(a.v) + t * a.v_stride);
    };
    // The lane's next rows: `left` warps-full to do, `lane_heads` of them with a head for this lane.
    uint4 x[U][2];
    auto fetch = [&](const T* src, int left, int lane_heads) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u < left && u < lane_heads) {
          x[u][0] = *reinterpret_cast<const uint4*>(src + u * HPW * D + c0);
          x[u][1] = *reinterpret_cast<const uint4*>(src + u * HPW * D + c1);
        } else {
          x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    auto heads_of_lane = [&](int heads, int h0) { return (heads - h0 + HPW - 1) / HPW; };
    {
      // The job's first rows, on their way while its angles are computed.
      const int kind = from < ends[0] ? 0 : (from < ends[1] ? 1 : 2), g = from - (kind == 0 ? 0 : ends[kind - 1]);
      fetch(input(kind) + (g * HPW + sub) * D, to - from, heads_of_lane(kind == 0 ? a.Hq : a.Hkv, g * HPW + sub));
    }
    int pos = 0;
    if (a.positions != nullptr) {
      pos = a.positions[t];
      if (pos < 0 || pos >= (1 << 24)) {
        if (lane == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
        continue;
      }
    }
    long long row = t;
    if (a.kv_rows != nullptr && to > full_q) {
      row = a.kv_rows[t];
      if (row < 0 || row >= a.kv_out_rows) {
        if (lane == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
        row = -1;                                             // the token's queries are still written
      }
    }
    // Sines and cosines of the token, once for all its heads: the lane's 8
    // angles 8p .. 8p + 7, of which each of the warp's heads computes a share.
    constexpr int OWN = 8 / HPW;
    float cs[8], sn[8];
    if (a.rot > 0 && from < ends[1]) {
      float oc[OWN], os[OWN];
#pragma unroll
      for (int j = 0; j < OWN; ++j) {
        oc[j] = 1.f;
        os[j] = 0.f;
        if (turned) rotation(static_cast<float>(pos), a.inv_freq[8 * p + sub * OWN + j], oc[j], os[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cs[j] = __shfl_sync(0xffffffffu, oc[j % OWN], (j / OWN) * LPH + p) * a.rope_scale;
        sn[j] = __shfl_sync(0xffffffffu, os[j % OWN], (j / OWN) * LPH + p) * a.rope_scale;
      }
    }
    // Coefficients of the 8 pairs of neighbouring elements, chunk c0 and then
    // chunk c1, for queries or for keys.
    uint64_t P[8], Q[8];
    bool normed = false;
    auto coefficients = [&](const float* weight) {
      normed = weight != nullptr;
      float w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = 1.f;
      if (normed) {
        load_weights(weight + c0, w);
        load_weights(weight + c1, w + 8);
      }
      if (!turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          P[j] = pair_f2(w[2 * j], w[2 * j + 1]);
          Q[j] = 0ull;
        }
      } else if constexpr (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          P[j] = pair_f2(w[2 * j] * cs[j], w[2 * j + 1] * cs[j]);
          Q[j] = pair_f2(-w[2 * j + 1] * sn[j], w[2 * j] * sn[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 2 * j;
          P[j] = pair_f2(w[e] * cs[e], w[e + 1] * cs[e + 1]);
          Q[j] = pair_f2(-w[8 + e] * sn[e], -w[9 + e] * sn[e + 1]);
          P[4 + j] = pair_f2(w[8 + e] * cs[e], w[9 + e] * cs[e + 1]);
          Q[4 + j] = pair_f2(w[e] * sn[e], w[e + 1] * sn[e + 1]);
        }
      }
    };
    // One head row, in the lane's two chunks.
    auto turn = [&](uint4 (&x)[2]) {
      const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
      uint32_t y[8];
      uint64_t v[8];
      float inv = 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = to_f2(w[j], T());
      if (normed) {
        uint64_t s0 = mul_pair(v[0], v[0]), s1 = mul_pair(v[1], v[1]);
#pragma unroll
        for (int j = 2; j < 8; j += 2) {
          s0 = fma_pair(v[j], v[j], s0);
          s1 = fma_pair(v[j + 1], v[j + 1], s1);
        }
        const float2 a0 = halves_f2(s0), a1 = halves_f2(s1);
        float ss = (a0.x + a0.y) + (a1.x + a1.y);
#pragma unroll
        for (int m = LPH / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
      }
      const uint64_t inv2 = pair_f2(inv, inv);
      if (all_turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = from_f2(mul_pair(fma_pair(partner_of(v, j), Q[j], mul_pair(v[j], P[j])), inv2), T());
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint64_t z = mul_pair(v[j], P[j]);
          if (turned) z = fma_pair(partner_of(v, j), Q[j], z);   // (not 0 * partner: it may be infinite)
          y[j] = from_f2(mul_pair(z, inv2), T());
        }
      }
      x[0] = make_uint4(y[0], y[1], y[2], y[3]);
      x[1] = make_uint4(y[4], y[5], y[6], y[7]);
    };
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {                    // queries, keys, values
      const int g0 = kind == 0 ? 0 : ends[kind - 1];
      const int g_from = max(from, g0) - g0, g_to = min(to, ends[kind]) - g0;
      if (g_from >= g_to || (kind > 0 && row < 0)) continue;
      const int heads = kind == 0 ? a.Hq : a.Hkv, h0 = g_from * HPW + sub;
      const T* src = input(kind) + h0 * D;
      T* dst = (kind == 0 ? static_cast<T*>(a.q_out) + t * a.q_out_stride
                          : (kind == 1 ? static_cast<T*>(a.k_out) + row * a.k_out_stride
                                       : static_cast<T*>(a.v_out) + row * a.v_out_stride)) + h0 * D;
      if (kind < 2) coefficients(kind == 0 ? a.q_weight : a.k_weight);
      int left = g_to - g_from, lane_heads = heads_of_lane(heads, h0);
      bool fetched = g0 + g_from == from;                     // (the job's first rows)
#pragma unroll 1
      for (; left > 0; left -= U, lane_heads -= U, src += U * HPW * D, dst += U * HPW * D) {
        if (!fetched) fetch(src, left, lane_heads);
        fetched = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= left) break;                               // warp-uniform
          if (kind < 2) turn(x[u]);
          if (u < lane_heads) {
            *reinterpret_cast<uint4*>(dst + u * HPW * D + c0) = x[u][0];
            *reinterpret_cast<uint4*>(dst + u * HPW * D + c1) = x[u][1];
          }
        }
      }
    }
  }
}

template <typename T, int D, bool INTERLEAVED>
cudaError_t launch_layout(const NormRopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int HPW = 32 / (D / 16);
  // Few tokens: a job for every warp-full of heads, so that all SMs take
  // part; many: whole tokens, so that sines and cosines serve all their heads.
  const int full_q = (a.Hq + HPW - 1) / HPW, full_k = (a.Hkv + HPW - 1) / HPW;
  const int full = full_q + (a.v_out != nullptr ? 2 : 1) * full_k;
  const long long even = static_cast<long long>(a.cap) * full / (static_cast<long long>(num_sms) * 16);
  const int iters = static_cast<int>(even < 1 ? 1 : (even > full ? full : even)), jobs = (full + iters - 1) / iters;
  const long long ctas = (static_cast<long long>(a.cap) * jobs + R_WARPS - 1) / R_WARPS, most = 64LL * num_sms;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
  cfg.blockDim = dim3(32 * R_WARPS);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, D, INTERLEAVED>, a, iters, jobs);
}

template <typename T, int D>
cudaError_t launch_d(const NormRopeArgs& a, bool interleaved, int num_sms, cudaStream_t stream) {
  return interleaved ? launch_layout<T, D, true>(a, num_sms, stream) : launch_layout<T, D, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int d, rra_dtype dt, bool interleaved, int num_sms,
                                cudaStream_t stream) {
  if (dt == RRA_BF16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, interleaved, num_sms, stream)
                   : launch_d<__nv_bfloat16, 128>(a, interleaved, num_sms, stream);
  return d == 64 ? launch_d<__half, 64>(a, interleaved, num_sms, stream)
                 : launch_d<__half, 128>(a, interleaved, num_sms, stream);
}

}  // namespace rra
