// Attention over packed prompts.  One warp per (row, query head): lanes hold
// d/32 elements each, a running maximum and sum over the keys.
#include "common.cuh"

namespace rra {
namespace {

template <typename T> __device__ __forceinline__ float to_f(T x) { return static_cast<float>(x); }

template <typename T, int D>
__global__ void attend_prompt_kernel(const PromptArgs a) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y % a.Hq, b = blockIdx.y / a.Hq;
  const int s0 = a.cu[b], n = a.cu[b + 1] - s0;
  if (n < 0 || n > a.max_seqlen || s0 < 0 || s0 > a.cap - n) {
    if (threadIdx.x == 0)
      record_error(a.err, n < 0 ? RRA_DEVERR_SEQ_NEGATIVE
                                : (n > a.max_seqlen ? RRA_DEVERR_SEQ_TOO_LONG : RRA_DEVERR_INDEX_RANGE));
    return;
  }
  const int i = blockIdx.x * 4 + warp;
  if (i >= n) return;
  const int hk = h / (a.Hq / a.Hkv);
  const T* q = static_cast<const T*>(a.q) + static_cast<long long>(s0 + i) * a.q_stride + h * D + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f(q[e]);
    o[e] = 0.f;
  }
  const int keys = a.causal ? i + 1 : n;
  for (int j = 0; j < keys; ++j) {
    const T* k = static_cast<const T*>(a.k) + static_cast<long long>(s0 + j) * a.k_stride + hk * D + lane * E;
    const T* v = static_cast<const T*>(a.v) + static_cast<long long>(s0 + j) * a.v_stride + hk * D + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += qv[e] * to_f(k[e]);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float c = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * c + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * to_f(v[e]);
  }
  T* out = static_cast<T*>(a.o) + (static_cast<long long>(s0 + i) * a.Hq + h) * D + lane * E;
  for (int e = 0; e < E; ++e) out[e] = T(l > 0.f ? o[e] / l : (l == 0.f ? 0.f : l));
}

template <typename T>
cudaError_t launch_d(const PromptArgs& a, int d, cudaStream_t stream) {
  const dim3 grid((a.max_seqlen + 3) / 4, a.B * a.Hq);
  if (d == 64) attend_prompt_kernel<T, 64><<<grid, 128, 0, stream>>>(a);
  else attend_prompt_kernel<T, 128><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_prompt(const PromptArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream) {
  return dt == RRA_BF16 ? launch_d<__nv_bfloat16>(a, d, stream) : launch_d<__half>(a, d, stream);
}

}  // namespace rra
