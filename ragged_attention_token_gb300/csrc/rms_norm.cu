// Root-mean-square norm of packed rows with the residual's addition, and an
// output in 16 bits, or in 8 bits (e4m3) with one scale a row.
//
// For row t < T = cu_seqlens[B], in fp32:
//   r = x + residual;  sum = r (rounded to the residual's type);
//   y = r rsqrt(mean(r^2) + eps) weight;
//   16 bits: y rounded;  8 bits: scale = max(max |y| / 448, 2^-100), q = y / scale rounded (448 is e4m3's largest).
//
// What bounds it is the one read of x and the residual and the one write of the
// sum and y: a row stays in the registers of the threads that loaded it (up
// to four chunks of 8 elements each) from the loads to the stores, through the
// sum of squares and, in 8 bits, the largest |y|.  Rows are short against what an SM
// keeps in flight, so that many rows at once (a warp, or a CTA of 64 to 1024
// threads, per row) hide each other's two reductions.
//
// |y| is compared as unsigned integers, which order like the values and put NaN on
// top: a NaN anywhere in a row makes its scale NaN, never a plausible number.
#include <cuda_fp8.h>

#include "block.cuh"
#include "f32x2.cuh"

namespace rra {
namespace {

constexpr int NV = 4;                        // chunks of 8 elements a thread holds
constexpr int N_WARP_ROWS = 4;               // rows of a CTA where a warp has a row
constexpr float N_LEAST = 7.888609052210118e-31f;   // 2^-100: a row of zeros, and rows whose scale would be subnormal

// 8 neighbouring elements as floats, and back (one rounding).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 t = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float add_over_warp(float v) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}

// WARP: a warp has a row, N_WARP_ROWS rows a CTA; else the CTA has one.
template <typename T, typename Tr, typename Ty, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * N_WARP_ROWS : 1024) rms_norm_kernel(const NormRowsArgs a) {
  constexpr bool EIGHT = sizeof(Ty) == 1;
  __shared__ float part[32];
  __shared__ uint32_t part_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = WARP ? 32 : static_cast<int>(blockDim.x), at = WARP ? lane : static_cast<int>(threadIdx.x);
  const int t = WARP ? static_cast<int>(blockIdx.x) * N_WARP_ROWS + warp : static_cast<int>(blockIdx.x);
  start_dependent();
  const int rows = a.cu[a.B];
  if (rows < 0 || rows > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
    return;
  }
  if (t >= rows) return;                     // a whole warp, and without WARP a whole CTA
  const int chunks = a.N / 8;
  const long long row = static_cast<long long>(t) * a.N;
  const T* x = static_cast<const T*>(a.x) + row;
  const Tr* res = a.residual != nullptr ? static_cast<const Tr*>(a.residual) + row : nullptr;
  float r[NV][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = at + i * threads;
    if (c < chunks) load8(x + 8 * c, r[i]);
  }
  if (res != nullptr) {
    float s[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at + i * threads;
      if (c < chunks) load8(res + 8 * c, s[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at + i * threads;
      if (c < chunks) {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i][k] += s[i][k];
        store8(static_cast<Tr*>(a.sum) + row + 8 * c, r[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (at + i * threads < chunks) {
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(r[i][k], r[i][k], ss);
    }
  }
  ss = add_over_warp(ss);
  if constexpr (!WARP) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = add_over_warp(lane < threads / 32 ? part[lane] : 0.f);
  }
  const float inv = rsqrtf(ss / static_cast<float>(a.N) + a.eps);
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = at + i * threads;
    if (c < chunks) {
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (a.weight != nullptr) load8(a.weight + 8 * c, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[i][k] *= inv * w[k];
        if constexpr (EIGHT) top = max(top, __float_as_uint(r[i][k]) & 0x7fffffffu);
      }
      if constexpr (!EIGHT) store8(static_cast<Ty*>(a.y) + row + 8 * c, r[i]);
    }
  }
  if constexpr (EIGHT) {
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (!WARP) {
      if (lane == 0) part_max[warp] = top;
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, lane < threads / 32 ? part_max[lane] : 0u);
    }
    float scale = __fdiv_rn(__uint_as_float(top), 448.f);
    if (scale < N_LEAST) scale = N_LEAST;    // NaN stays
    if (at == 0) a.scale[t] = scale;
    const float f = __fdiv_rn(1.f, scale);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at + i * threads;
      if (c < chunks) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // y / scale: the product with the reciprocal, put right by its remainder (a quotient next to the middle
          // of two values in 8 bits falls to the wrong side half as often).
          const float v = r[i][k] * f;
          r[i][k] = fmaf(fmaf(-v, scale, r[i][k]), f, v);
        }
        store8(static_cast<Ty*>(a.y) + row + 8 * c, r[i]);
      }
    }
  }
}

template <typename T, typename Tr, typename Ty>
cudaError_t launch_typed(const NormRowsArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = a.N / 8;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (chunks <= 32 * NV) {
    cfg.gridDim = dim3(static_cast<unsigned>((a.cap - 1) / N_WARP_ROWS + 1));
    cfg.blockDim = dim3(32 * N_WARP_ROWS);
    return cudaLaunchKernelEx(&cfg, rms_norm_kernel<T, Tr, Ty, true>, a);
  }
  int threads = 64;
  while (threads * NV < chunks) threads *= 2;
  (void)num_sms;
  cfg.gridDim = dim3(static_cast<unsigned>(a.cap));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  return cudaLaunchKernelEx(&cfg, rms_norm_kernel<T, Tr, Ty, false>, a);
}

template <typename T>
cudaError_t launch_in(const NormRowsArgs& a, rra_dtype residual, bool eight_bits, int num_sms, cudaStream_t stream) {
  if (residual == RRA_F32)
    return eight_bits ? launch_typed<T, float, __nv_fp8_e4m3>(a, num_sms, stream) : launch_typed<T, float, T>(a, num_sms, stream);
  return eight_bits ? launch_typed<T, T, __nv_fp8_e4m3>(a, num_sms, stream) : launch_typed<T, T, T>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const NormRowsArgs& a, rra_dtype dt, rra_dtype residual, bool eight_bits, int num_sms,
                            cudaStream_t stream) {
  return dt == RRA_BF16 ? launch_in<__nv_bfloat16>(a, residual, eight_bits, num_sms, stream)
                        : launch_in<__half>(a, residual, eight_bits, num_sms, stream);
}

}  // namespace rra
