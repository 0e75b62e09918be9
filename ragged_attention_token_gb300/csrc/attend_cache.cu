// Attention of the newest nq tokens of each sequence over a padded cache
// [B, cap, Hkv, d] (one token each: a decoding step).
//
// For row (token i, query head h) of a sequence of kv_len keys, over the keys
// j < kv_len - (nq - 1 - i): o = sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m),
// s_j = <q, k_j>, c = scale log2 e.
//
// What bounds it is the one read of the cache: a key and value row of d
// elements is used by the few rows of its head group only.  So a unit is
// (sequence, key/value head, 16 rows of its nq * Hq/Hkv), the rows filling one mma.sync
// tile; its keys are dealt out in chunks of 16 to the warps of a cluster of CTAs.
// Every warp runs on its own: cp.async copies of its next chunks into its own
// ring (24 KB, so two CTAs keep 192 KB in flight on an SM), S = Q K^T, a running
// reference and sum per row, O += P V, no barrier until its keys are
// done.  Then the partial results of all warps of the cluster are joined through
// distributed shared memory, each CTA a share of the output: one launch, no
// workspace, and an order of additions that does not depend on timing.
//
// The reference of a row moves only when a maximum exceeds it by more than 8
// (log2 units); weights are rounded to the input type for the second product
// (relative 2^-8 in bf16, 2^-11 in fp16, where a factor 2^7 that cancels keeps them
// out of the subnormal range), their sum is taken unrounded in fp32.
// Rows of the cache from kv_len on are not read: the copies fill their places with zeros.
#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "softmax_tc.cuh"

namespace rra {
namespace {

constexpr int CK = 16;                      // keys of a chunk
constexpr int C_WARPS = 4;
constexpr int C_ROWS = 16;                  // rows of a unit
constexpr int C_RING = 24 * 1024;           // bytes of a warp's ring
constexpr int C_MAX_SPLIT = 16;             // CTAs of a cluster
constexpr float C_MOVE = 8.f;

template <int D>
struct CacheCfg {
  static constexpr int TILE = CK * D * 2;                 // K (or V) of a chunk
  static constexpr int STAGES = C_RING / (2 * TILE);      // 3 at d = 128, 6 at d = 64
  // Partial results of a warp, over its ring once its keys are done: O [16][D], then m [16], l [16] (fp32).
  static constexpr int PART = (C_ROWS * D + 2 * C_ROWS) * 4;
  static constexpr int SMEM = C_WARPS * C_RING;
  static_assert(PART <= C_RING, "partial results live in the ring");
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
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16-byte copy global -> shared, zeros when `bytes` is 0 (the source is then not read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * C_WARPS, 2) attend_cache_kernel(const CacheArgs a, int nsplit, int row_blocks) {
  using C = CacheCfg<D>;
  constexpr bool BF = IsBf16<T>::value == 1;
  extern __shared__ __align__(128) uint8_t smem_cache[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % nsplit;         // = the CTA's rank in its cluster
  const int unit = static_cast<int>(blockIdx.x) / nsplit;
  const int rb = unit % row_blocks, hk = unit / row_blocks % a.Hkv, b = unit / row_blocks / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int rows = min(C_ROWS, a.nq * G - rb * C_ROWS);            // row r: token r / G, head hk * G + r % G (r from rb * 16)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = __ldg(a.kv_len + b);
  const bool valid = len >= 0 && len <= a.cap;
  if (!valid && split == 0 && rb == 0 && hk == 0 && threadIdx.x == 0)
    record_error(a.err, len < 0 ? RRA_DEVERR_SEQ_NEGATIVE : RRA_DEVERR_SEQ_TOO_LONG);
  const uint32_t ring = smem_u32(smem_cache) + static_cast<uint32_t>(warp) * C_RING;

  // Keys that row r of the unit sees: its first `sees(r)` ones (not above zero: none).
  auto sees = [&](int r) { return len - (a.nq - 1 - (rb * C_ROWS + r) / G); };
  const int keys = valid ? max(0, sees(rows - 1)) : 0;
  const int chunks = (keys + CK - 1) / CK, stride = nsplit * C_WARPS, first = split * C_WARPS + warp;
  const int mine = first < chunks ? (chunks - first + stride - 1) / stride : 0;

  // Copies of this warp's i-th chunk into stage s, 16-byte pieces, 128-byte
  // groups of pieces rotated by the row so that ldmatrix meets no bank twice.
  auto piece = [&](int row, int c) { return static_cast<uint32_t>(row * (D * 2) + (((c & ~7) | ((c ^ row) & 7)) << 4)); };
  const long long row_elems = static_cast<long long>(a.Hkv) * D;
  const long long base = (static_cast<long long>(b) * a.cap) * row_elems + hk * D;
  auto fetch = [&](int i, int s) {
    const int k0 = (first + i * stride) * CK;
    const uint32_t dk = ring + static_cast<uint32_t>(s) * (2 * C::TILE), dv = dk + C::TILE;
#pragma unroll
    for (int p = 0; p < CK * D / 8 / 32; ++p) {
      const int x = p * 32 + lane, row = x / (D / 8), c = x % (D / 8);
      const bool in = k0 + row < keys;
      const long long off = base + (in ? k0 + row : 0) * row_elems + c * 8;
      cp_async16_or_zero(dk + piece(row, c), static_cast<const T*>(a.k) + off, in ? 16 : 0);
      cp_async16_or_zero(dv + piece(row, c), static_cast<const T*>(a.v) + off, in ? 16 : 0);
    }
  };
#pragma unroll
  for (int s = 0; s < C::STAGES; ++s) {
    if (s < mine) fetch(s, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // Q as operand A: rows g and g + 8 of the unit, rows past its end as zeros.
  uint32_t qf[D / 16][4];
  int lim[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = g + 8 * x, rr = rb * C_ROWS + r;
    lim[x] = r < rows ? sees(r) : 0;
    const T* src = static_cast<const T*>(a.q) + (static_cast<long long>(b) * a.nq + (r < rows ? rr / G : 0)) * a.q_stride +
                   (hk * G + (r < rows ? rr % G : 0)) * D + 2 * q;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qf[kk][x] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * kk) : 0u;
      qf[kk][2 + x] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8) : 0u;
    }
  }
  float o[D / 8][4], m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

  int s = 0;
  for (int i = 0; i < mine; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 1) : "memory");
    __syncwarp();
    const uint32_t sk = ring + static_cast<uint32_t>(s) * (2 * C::TILE), sv = sk + C::TILE;
    const int k0 = (first + i * stride) * CK;
    // S: 16 rows x 16 keys.
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      // Matrices: keys 0-7 and 8-15, each with the step's first and last 8 elements.
      uint32_t r[4];
      ldmatrix4<false>(r, sk + piece((lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
      mma_16816(sc[0], qf[kk], r[0], r[1], T());
      mma_16816(sc[1], qf[kk], r[2], r[3], T());
    }
    uint32_t pf[4];
    float alpha[2] = {1.f, 1.f};
    bool moved = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // Row g + 8x: keys 2q, 2q + 1, 8 + 2q, 9 + 2q of the chunk.
      float t[4] = {sc[0][2 * x], sc[0][2 * x + 1], sc[1][2 * x], sc[1][2 * x + 1]};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        t[e] = k0 + 2 * q + (e & 1) + 8 * (e >> 1) < lim[x] ? t[e] * a.scale_log2 : -INFINITY;
      float mx = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (mx > m_ref[x] + C_MOVE) {
        alpha[x] = fast_exp2(m_ref[x] - mx);
        m_ref[x] = mx;
        l_run[x] *= alpha[x];
        moved = true;
      }
      // A row that has seen only -inf scores keeps its reference at -inf: weights 0.
      const float mu = (m_ref[x] == -INFINITY ? 0.f : m_ref[x]) - (BF ? 0.f : 7.f);
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = fast_exp2(t[e] - mu);
        l_run[x] += p[e];
      }
      if constexpr (BF) {
        pf[x] = pack2<__nv_bfloat162>(p[0], p[1]);
        pf[2 + x] = pack2<__nv_bfloat162>(p[2], p[3]);
      } else {
        pf[x] = pack2<__half2>(p[0], p[1]);
        pf[2 + x] = pack2<__half2>(p[2], p[3]);
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= alpha[0];
        o[n][1] *= alpha[0];
        o[n][2] *= alpha[1];
        o[n][3] *= alpha[1];
      }
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      // Matrices (transposed): keys 0-7 and 8-15 of elements 16n .. 16n + 7, then of the next 8.
      uint32_t r[4];
      ldmatrix4<true>(r, sv + piece((lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
      mma_16816(o[2 * n], pf, r[0], r[1], T());
      mma_16816(o[2 * n + 1], pf, r[2], r[3], T());
    }
    __syncwarp();                           // the chunk is read before its stage is filled again
    if (i + C::STAGES < mine) fetch(i + C::STAGES, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++s == C::STAGES) s = 0;
  }

  // This warp's partial result, over its ring.
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem_cache + warp * C_RING);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], 1);
    l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], 2);
    const int r = g + 8 * x;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(part + r * D + 8 * n + 2 * q) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
    if (q == 0) {
      part[C_ROWS * D + r] = m_ref[x];
      part[C_ROWS * D + C_ROWS + r] = l_run[x];
    }
  }
  if (nsplit > 1) asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
  else __syncthreads();

  // The cluster's CTAs take pairs of output elements in turn; each pair reads
  // all partial results in the same order.
  const uint32_t part0 = smem_u32(smem_cache);
  for (int e = split * blockDim.x + threadIdx.x; valid && e < rows * (D / 2); e += nsplit * blockDim.x) {
    const int r = e / (D / 2), c = 2 * (e % (D / 2));
    float top = -INFINITY;
    for (int p = 0; p < stride; ++p) {
      const uint32_t at = map_rank(part0 + static_cast<uint32_t>(p % C_WARPS) * C_RING, static_cast<uint32_t>(p / C_WARPS));
      top = fmaxf(top, ld_cluster_f32(at + 4u * static_cast<uint32_t>(C_ROWS * D + r)));
    }
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, y0 = 0.f, y1 = 0.f;
    for (int p = 0; p < stride; ++p) {
      const uint32_t at = map_rank(part0 + static_cast<uint32_t>(p % C_WARPS) * C_RING, static_cast<uint32_t>(p / C_WARPS));
      const float w = fast_exp2(ld_cluster_f32(at + 4u * static_cast<uint32_t>(C_ROWS * D + r)) - ref);
      sum = fmaf(w, ld_cluster_f32(at + 4u * static_cast<uint32_t>(C_ROWS * D + C_ROWS + r)), sum);
      y0 = fmaf(w, ld_cluster_f32(at + 4u * static_cast<uint32_t>(r * D + c)), y0);
      y1 = fmaf(w, ld_cluster_f32(at + 4u * static_cast<uint32_t>(r * D + c + 1)), y1);
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int rr = rb * C_ROWS + r;
    T* out = static_cast<T*>(a.o) + ((static_cast<long long>(b) * a.nq + rr / G) * a.Hq + hk * G + rr % G) * D + c;
    const uint32_t w = BF ? pack2<__nv_bfloat162>(y0 * inv, y1 * inv) : pack2<__half2>(y0 * inv, y1 * inv);
    *reinterpret_cast<uint32_t*>(out) = w;
  }
  // No CTA leaves while another may still read its partial results.
  if (nsplit > 1) asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

template <typename T, int D>
cudaError_t launch_d(const CacheArgs& a, int num_sms, cudaStream_t stream) {
  using C = CacheCfg<D>;
  auto kernel = attend_cache_kernel<T, D>;
  constexpr int kMaxDevices = 64;
  static int max_split[kMaxDevices] = {};                 // 0: not yet set up
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(32 * C_WARPS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  int most;
  {
    std::lock_guard<std::mutex> lock(m);
    if (max_split[dev] == 0) {
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
      // Clusters of 16 where the device takes them, else of 8 (which every device of this kind does).
      int clusters = 0;
      attr[0].val.clusterDim.x = C_MAX_SPLIT;
      cfg.gridDim = dim3(C_MAX_SPLIT);
      cfg.numAttrs = 1;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        clusters = 0;
      }
      max_split[dev] = clusters > 0 ? C_MAX_SPLIT : C_MAX_SPLIT / 2;
    }
    most = max_split[dev];
  }
  const int row_blocks = (a.nq * (a.Hq / a.Hkv) + C_ROWS - 1) / C_ROWS;
  const long long units = static_cast<long long>(a.B) * a.Hkv * row_blocks;
  // Split until the CTAs fill the SMs four times over (two at a time), so that
  // sequences of very different lengths even out, but leave a warp four chunks.
  int nsplit = 1;
  while (nsplit < most && units * nsplit < 8LL * num_sms && (a.cap + CK - 1) / CK >= 2 * nsplit * C_WARPS * 4) nsplit *= 2;
  if (units * nsplit >= (1LL << 31)) return cudaErrorInvalidValue;
  attr[0].val.clusterDim.x = static_cast<unsigned>(nsplit);
  cfg.gridDim = dim3(static_cast<unsigned>(units * nsplit));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, nsplit, row_blocks);
}

}  // namespace

cudaError_t launch_attend_cache(const CacheArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream) {
  if (dt == RRA_BF16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, num_sms, stream) : launch_d<__nv_bfloat16, 128>(a, num_sms, stream);
  return d == 64 ? launch_d<__half, 64>(a, num_sms, stream) : launch_d<__half, 128>(a, num_sms, stream);
}

}  // namespace rra
