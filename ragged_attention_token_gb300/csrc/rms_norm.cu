// Root-mean-square norm of packed rows with the residual's addition, and an
// output in 16 bits, or in 8 bits (e4m3) with one scale a row.
//
// For row t < T = cu_seqlens[B], in fp32:
//   r = x + residual;  sum = r (rounded to the residual's type);
//   y = r rsqrt(mean(r^2) + eps) weight;
//   16 bits: y rounded;  8 bits: scale = max(max |y| / 448, 2^-100), q = y / scale rounded (448 is e4m3's largest).
//
// What bounds it is the one read of x and the residual and the one write of the sum and y: a row stays in registers from
// the loads to the stores, through the sum of squares and, in 8 bits, the largest |y|.  A row is as many warps' as give each
// thread one to four chunks of 8 elements, several short rows to a CTA, and a thread's chunks of its next row are on
// their way while it works on this one: 16411 x 4096 with residual to 8 bits (471 MB) in 71.9 us, 6.5 TB/s.  (A CTA a row, of
// which the SMs start about one in a nanosecond, took 80 to 106 us, and 29 to 101 us for 100000 rows of 256.)
//
// |y| is compared as unsigned integers, which order like the values and put NaN on
// top: a NaN anywhere in a row makes its scale NaN, never a plausible number.
#include <cuda_fp8.h>

#include <mutex>

#include "block.cuh"
#include "f32x2.cuh"

namespace rra {
namespace {

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

// A chunk of 8 elements as it lies in memory.
template <typename T> struct Raw {
  uint4 v[sizeof(T) * 8 / 16];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) v[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const { load8(reinterpret_cast<const T*>(v), f); }
};

// A row is `warps` warps', `at` the thread's place among them, NV chunks a thread; barrier `id` is theirs.
// (MOST: threads of a CTA.  Past 16384 elements the registers have no room for the next row's chunks.)
template <typename T, typename Tr, typename Ty, bool RES, int NV, int MOST>
__global__ void __launch_bounds__(MOST) rms_norm_kernel(const NormRowsArgs a, int warps) {
  constexpr bool EIGHT = sizeof(Ty) == 1, AHEAD = NV < 4;
  __shared__ float part[32];
  __shared__ uint32_t part_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int of_cta = warp / warps, first = of_cta * warps, at = static_cast<int>(threadIdx.x) - 32 * first, threads = 32 * warps;
  const int per_cta = static_cast<int>(blockDim.x) / threads;
  const long long stride = static_cast<long long>(gridDim.x) * per_cta;
  long long t = static_cast<long long>(blockIdx.x) * per_cta + of_cta;
  const int chunks = a.N / 8;
  auto join = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + of_cta), "r"(threads) : "memory"); };
  Raw<T> x[NV];
  Raw<Tr> s[RES ? NV : 1];
  auto fetch_chunk = [&](long long row, int i, int c) {
    x[i].load(static_cast<const T*>(a.x) + row * a.N + 8 * c);
    if constexpr (RES) s[i].load(static_cast<const Tr*>(a.residual) + row * a.N + 8 * c);
  };
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at + i * threads;
      if (c < chunks) fetch_chunk(row, i, c);
    }
  };
  start_dependent();
  const int rows = a.cu[a.B];
  // The first row is asked for ahead of the count's arrival: rows up to cap are there to be read.
  if (AHEAD && t < a.cap) fetch(t);
  if (rows < 0 || rows > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
    return;
  }
  for (; t < rows; t += stride) {            // all of a row's warps go round together
    float r[NV][8], ss = 0.f;
    const long long row = t * a.N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at + i * threads;
      if (c < chunks) {
        if (!AHEAD) fetch_chunk(t, i, c);
        x[i].floats(r[i]);
        if constexpr (RES) {
          float f[8];
          s[i].floats(f);
#pragma unroll
          for (int k = 0; k < 8; ++k) r[i][k] += f[k];
        }
      }
    }
    if (AHEAD && t + stride < rows) fetch(t + stride);   // in flight through the rest
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at + i * threads;
      if (c < chunks) {
        if constexpr (RES) store8(static_cast<Tr*>(a.sum) + row + 8 * c, r[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(r[i][k], r[i][k], ss);
      }
    }
    ss = add_over_warp(ss);
    if (warps > 1) {
      if (lane == 0) part[warp] = ss;
      join();
      ss = add_over_warp(lane < warps ? part[first + lane] : 0.f);
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
      if (warps > 1) {
        if (lane == 0) part_max[warp] = top;
        join();                              // (and the sums are read before the next row's)
        top = __reduce_max_sync(0xffffffffu, lane < warps ? part_max[first + lane] : 0u);
      }
      float scale = __fdiv_rn(__uint_as_float(top), 448.f);
      if (scale < N_LEAST) scale = N_LEAST;  // NaN stays
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
    } else if (warps > 1) {
      join();                                // the sums are read before the next row's are written
    }
  }
}

// CTAs of `threads` threads of this kernel that an SM holds (asked once per device and size).
template <typename T, typename Tr, typename Ty, bool RES, int NV, int MOST>
cudaError_t resident(int threads, int* ctas) {
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices][33] = {};
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(m);
  int& n = known[dev][threads / 32];
  if (n == 0 && (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, rms_norm_kernel<T, Tr, Ty, RES, NV, MOST>, threads, 0)) != cudaSuccess) {
    n = 0;
    return e;
  }
  *ctas = n > 0 ? n : 1;
  return cudaSuccess;
}

template <typename T, typename Tr, typename Ty, bool RES, int NV, int MOST>
cudaError_t launch_nv(const NormRowsArgs& a, int num_sms, cudaStream_t stream) {
  const int warps = (a.N / 8 + 32 * NV - 1) / (32 * NV);
  const int per_cta = warps >= 8 ? 1 : 8 / warps, threads = 32 * warps * per_cta;
  int ctas = 0;
  if (cudaError_t e = resident<T, Tr, Ty, RES, NV, MOST>(threads, &ctas); e != cudaSuccess) return e;
  // Where the next row is not asked for ahead, CTAs that wait for room do as much.
  const long long all = (a.cap - 1LL) / per_cta + 1, room = NV < 4 ? static_cast<long long>(ctas) * num_sms : all;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(all < room ? all : room));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rms_norm_kernel<T, Tr, Ty, RES, NV, MOST>, a, warps);
}

template <typename T, typename Tr, typename Ty, bool RES>
cudaError_t launch_typed(const NormRowsArgs& a, int num_sms, cudaStream_t stream) {
  // Few rows: as many threads a row as there are chunks, for the shortest way through one.  Many: two chunks a thread
  // (three to 768 elements, where a warp then has a row and needs no barrier) keep more bytes on the way for each barrier.
  // One chunk against that: 512 x 4096 with residual to 8 bits 4.0 / 4.8 us, 16411 x 4096 79.5 / 71.9 us, 2049 x 5120 17.7 /
  // 15.8, 12608 x 768 in fp16 10.2 / 8.6 (two 9.0).
  // With a residual and 8 bits a bound of 80 registers a thread serves best (2 chunks: 5120 at 2049 rows 15.7 -> 15.4, 4096 x 12288
  // 62.8 -> 59.0, with the residual in fp32 112.9 -> 93.4; without a residual 16.2 -> 16.6 and 39.1 -> 40.3).  Past 6144 elements two
  // chunks let an SM hold two rows' threads: 4096 x 8192 43.8 -> 38.9, 16411 x 8192 165 -> 140 (a residual in fp32 has no
  // room for that: 63.8 -> 65.5).
  constexpr int WIDE = RES && sizeof(Ty) == 1 ? 768 : 512;
  if (a.N > 16384) return launch_nv<T, Tr, Ty, RES, 4, 1024>(a, num_sms, stream);
  if (WIDE == 768 && a.N > 8192 && a.N <= 12288) return launch_nv<T, Tr, Ty, RES, 2, WIDE>(a, num_sms, stream);
  if (a.N > 8192 || (sizeof(Tr) == 2 && a.N > 6144 && a.cap >= 2 * num_sms)) return launch_nv<T, Tr, Ty, RES, 2, 1024>(a, num_sms, stream);
  if (a.N > 256 && a.N <= 6144 && a.cap >= 8 * num_sms) {
    if (a.N > 512 && a.N <= 768) return launch_nv<T, Tr, Ty, RES, 3, 256>(a, num_sms, stream);
    if (a.N <= 4096) return launch_nv<T, Tr, Ty, RES, 2, 256>(a, num_sms, stream);
    return launch_nv<T, Tr, Ty, RES, 2, WIDE>(a, num_sms, stream);
  }
  if (a.N <= 2048) return launch_nv<T, Tr, Ty, RES, 1, 256>(a, num_sms, stream);
  return launch_nv<T, Tr, Ty, RES, 1, 1024>(a, num_sms, stream);
}

template <typename T>
cudaError_t launch_in(const NormRowsArgs& a, rra_dtype residual, bool eight_bits, int num_sms, cudaStream_t stream) {
  if (a.residual == nullptr)
    return eight_bits ? launch_typed<T, T, __nv_fp8_e4m3, false>(a, num_sms, stream) : launch_typed<T, T, T, false>(a, num_sms, stream);
  if (residual == RRA_F32)
    return eight_bits ? launch_typed<T, float, __nv_fp8_e4m3, true>(a, num_sms, stream) : launch_typed<T, float, T, true>(a, num_sms, stream);
  return eight_bits ? launch_typed<T, T, __nv_fp8_e4m3, true>(a, num_sms, stream) : launch_typed<T, T, T, true>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const NormRowsArgs& a, rra_dtype dt, rra_dtype residual, bool eight_bits, int num_sms, cudaStream_t stream) {
  return dt == RRA_BF16 ? launch_in<__nv_bfloat16>(a, residual, eight_bits, num_sms, stream)
                        : launch_in<__half>(a, residual, eight_bits, num_sms, stream);
}

}  // namespace rra
