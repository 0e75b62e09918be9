// Attention of the newest tokens of each sequence over a padded cache.
// One warp per (row, query head): lanes hold d/32 elements each, a running
// maximum and sum over the keys.
#include "common.cuh"

namespace rra {
namespace {

template <typename T> __device__ __forceinline__ float to_f(T x) { return static_cast<float>(x); }

template <typename T, int D>
__global__ void attend_cache_kernel(const CacheArgs a) {
  constexpr int E = D / 32;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(a.B) * a.nq;
  if (w >= rows * a.Hq) return;
  const int h = static_cast<int>(w % a.Hq);
  const long long r = w / a.Hq;
  const int b = static_cast<int>(r / a.nq), i = static_cast<int>(r % a.nq);
  const int len = a.kv_len[b];
  if (len < 0 || len > a.cap) {
    if (lane == 0) record_error(a.err, len < 0 ? RRA_DEVERR_SEQ_NEGATIVE : RRA_DEVERR_SEQ_TOO_LONG);
    return;
  }
  const int n = len - (a.nq - 1 - i);
  const int hk = h / (a.Hq / a.Hkv);
  const T* q = static_cast<const T*>(a.q) + r * a.q_stride + h * D + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f(q[e]);
    o[e] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    const long long off = ((static_cast<long long>(b) * a.cap + j) * a.Hkv + hk) * D + lane * E;
    const T* k = static_cast<const T*>(a.k) + off;
    const T* v = static_cast<const T*>(a.v) + off;
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
  T* out = static_cast<T*>(a.o) + (r * a.Hq + h) * D + lane * E;
  for (int e = 0; e < E; ++e) out[e] = T(l > 0.f ? o[e] / l : (l == 0.f ? 0.f : l));
}

template <typename T>
cudaError_t launch_d(const CacheArgs& a, int d, cudaStream_t stream) {
  const long long warps = static_cast<long long>(a.B) * a.nq * a.Hq;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  if (d == 64) attend_cache_kernel<T, 64><<<grid, 128, 0, stream>>>(a);
  else attend_cache_kernel<T, 128><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_cache(const CacheArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream) {
  return dt == RRA_BF16 ? launch_d<__nv_bfloat16>(a, d, stream) : launch_d<__half>(a, d, stream);
}

}  // namespace rra
