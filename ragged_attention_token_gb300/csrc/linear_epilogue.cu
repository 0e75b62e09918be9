// Linear layer with bias, activation and residual: 32 x 32 output tiles,
// operands staged in shared memory as fp32, one output element per thread.
#include "common.cuh"

namespace rra {
namespace {

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case RRA_ACT_RELU: return x < 0.f ? 0.f : x;
    case RRA_ACT_GELU: return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    case RRA_ACT_GELU_TANH: return 0.5f * x * (1.f + tanhf(0.79788456080286536f * (x + 0.044715f * x * x * x)));
    case RRA_ACT_SILU: return x / (1.f + expf(-x));
    default: return x;
  }
}

template <typename Tin, typename Tout>
__global__ void linear_epilogue_kernel(const LinearEpiArgs a, int act) {
  __shared__ float sa[32][33], sw[32][33];
  const int T = a.cu[a.B];
  const int t0 = blockIdx.y * 32, n0 = blockIdx.x * 32, x = threadIdx.x, y = threadIdx.y;
  if (T < 0 || T > a.cap) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && x == 0 && y == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
    return;
  }
  if (t0 >= T) return;
  const Tin* pa = static_cast<const Tin*>(a.a);
  const Tin* pw = static_cast<const Tin*>(a.w);
  float acc = 0.f;
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    const int k = k0 + x;
    sa[y][x] = (t0 + y < T && k < a.K) ? static_cast<float>(pa[static_cast<size_t>(t0 + y) * a.K + k]) : 0.f;
    sw[y][x] = (n0 + y < a.N && k < a.K) ? static_cast<float>(pw[static_cast<size_t>(n0 + y) * a.K + k]) : 0.f;
    __syncthreads();
    for (int j = 0; j < 32; ++j) acc = fmaf(sa[y][j], sw[x][j], acc);
    __syncthreads();
  }
  const int t = t0 + y, n = n0 + x;
  if (t >= T || n >= a.N) return;
  if (a.bias != nullptr) acc += a.bias[n];
  acc = activate(acc, act);
  const size_t at = static_cast<size_t>(t) * a.N + n;
  if (a.residual != nullptr) acc += static_cast<float>(static_cast<const Tout*>(a.residual)[at]);
  static_cast<Tout*>(a.c)[at] = Tout(acc);
}

template <typename Tin>
cudaError_t launch_in(const LinearEpiArgs& a, rra_dtype out, int act, cudaStream_t stream) {
  const dim3 grid((a.N + 31) / 32, (a.cap + 31) / 32), block(32, 32);
  if (out == RRA_BF16) linear_epilogue_kernel<Tin, __nv_bfloat16><<<grid, block, 0, stream>>>(a, act);
  else if (out == RRA_F16) linear_epilogue_kernel<Tin, __half><<<grid, block, 0, stream>>>(a, act);
  else linear_epilogue_kernel<Tin, float><<<grid, block, 0, stream>>>(a, act);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_epilogue(const LinearEpiArgs& a, rra_dtype in, rra_dtype out, rra_activation act,
                                   int num_sms, cudaStream_t stream) {
  return in == RRA_BF16 ? launch_in<__nv_bfloat16>(a, out, act, stream) : launch_in<__half>(a, out, act, stream);
}

}  // namespace rra
