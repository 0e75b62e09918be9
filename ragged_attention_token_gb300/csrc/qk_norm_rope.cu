// Norms of queries and keys for each head, their rotation, and the write into
// a cache, in one pass: one warp per (token, head row).
//
// Angles.  positions reach 2^24 and inv_freq is fp32, so an fp32 product loses
// the angle; it is reduced in turns instead: inv_freq / 2 pi as an unevaluated
// sum of two floats (Dekker's product, by fma), times the position (exact in
// fp32 below 2^24) again as two floats, minus the nearest integer.  The
// remainder in [-1/2, 1/2] turns is good to about 2^-24 of a turn.
#include "common.cuh"

namespace rra {
namespace {

// cos and sin of pos * f.
__device__ __forceinline__ void rotation(float pos, float f, float& c, float& s) {
  constexpr double kTurn = 0.15915494309189533577;   // 1 / 2 pi
  constexpr float kHi = static_cast<float>(kTurn), kLo = static_cast<float>(kTurn - static_cast<double>(kHi));
  const float hi = f * kHi, lo = fmaf(f, kHi, -hi) + f * kLo;
  const float p = pos * hi, e = fmaf(pos, hi, -p) + pos * lo;
  const float r = (p - rintf(p)) + e;
  sincospif(2.f * r, &s, &c);
}

template <typename T, int D, bool INTERLEAVED>
__global__ void qk_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int E = D / 32;
  __shared__ float rowbuf[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T_rows = a.cu[a.B];
  if (T_rows < 0 || T_rows > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
    return;
  }
  const int heads = a.Hq + a.Hkv + (a.v_out != nullptr ? a.Hkv : 0);
  const long long w = static_cast<long long>(blockIdx.x) * 4 + warp;
  const int t = static_cast<int>(w / heads), hh = static_cast<int>(w % heads);
  if (t >= T_rows) return;
  int pos = 0;
  if (a.positions != nullptr) {
    pos = a.positions[t];
    if (pos < 0 || pos >= (1 << 24)) {
      if (lane == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
      return;
    }
  }
  const T* src;
  T* dst;
  const float* weight = nullptr;
  if (hh < a.Hq) {
    src = static_cast<const T*>(a.q) + t * a.q_stride + hh * D;
    dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + hh * D;
    weight = a.q_weight;
  } else {
    long long row = t;
    if (a.kv_rows != nullptr) {
      row = a.kv_rows[t];
      if (row < 0 || row >= a.kv_out_rows) {
        if (lane == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
        return;
      }
    }
    const bool is_k = hh < a.Hq + a.Hkv;
    const int h = hh - a.Hq - (is_k ? 0 : a.Hkv);
    src = is_k ? static_cast<const T*>(a.k) + t * a.k_stride + h * D : static_cast<const T*>(a.v) + t * a.v_stride + h * D;
    dst = is_k ? static_cast<T*>(a.k_out) + row * a.k_out_stride + h * D
               : static_cast<T*>(a.v_out) + row * a.v_out_stride + h * D;
    weight = a.k_weight;
    if (!is_k) {
      for (int e = 0; e < E; ++e) dst[lane + 32 * e] = src[lane + 32 * e];
      return;
    }
  }
  float x[E], ss = 0.f;
  for (int e = 0; e < E; ++e) {
    x[e] = static_cast<float>(src[lane + 32 * e]);
    ss = fmaf(x[e], x[e], ss);
  }
  for (int m = 16; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const float inv = weight != nullptr ? rsqrtf(ss / D + a.eps) : 1.f;
  for (int e = 0; e < E; ++e) rowbuf[warp][lane + 32 * e] = x[e] * inv * (weight != nullptr ? weight[lane + 32 * e] : 1.f);
  __syncwarp();
  for (int e = 0; e < E; ++e) {
    const int i = lane + 32 * e;
    float y = rowbuf[warp][i];
    if (i < a.rot) {
      const int half = a.rot / 2;
      const int f = INTERLEAVED ? i / 2 : i % half;
      const bool second = INTERLEAVED ? (i & 1) : i >= half;
      const float other = rowbuf[warp][INTERLEAVED ? (i ^ 1) : (second ? i - half : i + half)];
      float c, s;
      rotation(static_cast<float>(pos), a.inv_freq[f], c, s);
      y = a.rope_scale * (second ? other * s + y * c : y * c - other * s);
    }
    dst[i] = T(y);
  }
}

template <typename T, int D>
cudaError_t launch_d(const NormRopeArgs& a, bool interleaved, cudaStream_t stream) {
  const long long heads = a.Hq + a.Hkv + (a.v_out != nullptr ? a.Hkv : 0);
  const unsigned grid = static_cast<unsigned>((heads * a.cap + 3) / 4);
  if (interleaved) qk_norm_rope_kernel<T, D, true><<<grid, 128, 0, stream>>>(a);
  else qk_norm_rope_kernel<T, D, false><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int d, rra_dtype dt, bool interleaved, int num_sms,
                                cudaStream_t stream) {
  if (dt == RRA_BF16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, interleaved, stream) : launch_d<__nv_bfloat16, 128>(a, interleaved, stream);
  return d == 64 ? launch_d<__half, 64>(a, interleaved, stream) : launch_d<__half, 128>(a, interleaved, stream);
}

}  // namespace rra
