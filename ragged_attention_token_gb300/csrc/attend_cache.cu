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

#include "block.cuh"
#include "rows_mma.cuh"
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
  static constexpr int CTA_PART = C_RING / 2;             // the CTA's joined result, behind warp 0's
  static constexpr int SMEM = C_WARPS * C_RING;
  static_assert(PART <= CTA_PART, "both lie in warp 0's ring");
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * C_WARPS, 2)
    attend_cache_kernel(const CacheArgs a, int cluster, int min_chunks, int row_blocks) {
  using C = CacheCfg<D>;
  constexpr bool BF = IsBf16<T>::value == 1;
  extern __shared__ __align__(128) uint8_t smem_cache[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % cluster;        // = the CTA's rank in its cluster
  const int unit = static_cast<int>(blockIdx.x) / cluster;
  const int rb = unit % row_blocks, hk = unit / row_blocks % a.Hkv, b = unit / row_blocks / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int rows = min(C_ROWS, a.nq * G - rb * C_ROWS);            // row r: token r / G, head hk * G + r % G (r from rb * 16)
  dependent_launch();
  const int len = a.kv_len[b];
  const bool valid = len >= 0 && len <= a.cap;
  if (!valid && split == 0 && rb == 0 && hk == 0 && threadIdx.x == 0)
    record_error(a.err, len < 0 ? RRA_DEVERR_SEQ_NEGATIVE : RRA_DEVERR_SEQ_TOO_LONG);
  const uint32_t ring = smem_u32(smem_cache) + static_cast<uint32_t>(warp) * C_RING;

  // Keys that row r of the unit sees: its first `sees(r)` ones (not above zero: none).
  auto sees = [&](int r) { return len - (a.nq - 1 - (rb * C_ROWS + r) / G); };
  const int keys = valid ? max(0, sees(rows - 1)) : 0;
  const int chunks = (keys + CK - 1) / CK;
  // The CTAs that share the keys: no more than give each warp its min_chunks
  // (the host knows only the cache's capacity); the others of the cluster leave.
  const int nsplit = min(cluster, max(1, chunks / (C_WARPS * min_chunks)));
  if (split >= nsplit) return;
  const int stride = nsplit * C_WARPS, first = split * C_WARPS + warp;
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
  __syncthreads();

  // Four neighbouring outputs of row r as T.
  auto store = [&](int r, int c, float4 y, float sum) {
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int rr = rb * C_ROWS + r;
    T* out = static_cast<T*>(a.o) + ((static_cast<long long>(b) * a.nq + rr / G) * a.Hq + hk * G + rr % G) * D + c;
    uint2 w;
    w.x = BF ? pack2<__nv_bfloat162>(y.x * inv, y.y * inv) : pack2<__half2>(y.x * inv, y.y * inv);
    w.y = BF ? pack2<__nv_bfloat162>(y.z * inv, y.w * inv) : pack2<__half2>(y.z * inv, y.w * inv);
    *reinterpret_cast<uint2*>(out) = w;
  };
  constexpr int QUADS = D / 4;
  // The CTA's warps joined: O, reference and sum of each row.
  float* joined = reinterpret_cast<float*>(smem_cache + C::CTA_PART);
  for (int e = threadIdx.x; valid && e < rows * QUADS; e += 32 * C_WARPS) {
    const int r = e / QUADS, c = 4 * (e % QUADS);
    float m[C_WARPS], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < C_WARPS; ++w) {
      m[w] = reinterpret_cast<const float*>(smem_cache + w * C_RING)[C_ROWS * D + r];
      top = fmaxf(top, m[w]);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C_WARPS; ++w) {
      const float* p = reinterpret_cast<const float*>(smem_cache + w * C_RING);
      const float f = fast_exp2(m[w] - ref);
      const float4 v = *reinterpret_cast<const float4*>(p + r * D + c);
      sum = fmaf(f, p[C_ROWS * D + C_ROWS + r], sum);
      y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
    }
    if (nsplit == 1) {
      store(r, c, y, sum);
    } else {
      *reinterpret_cast<float4*>(joined + r * D + c) = y;
      if (c == 0) {
        joined[C_ROWS * D + r] = top;
        joined[C_ROWS * D + C_ROWS + r] = sum;
      }
    }
  }
  if (nsplit == 1) return;
  cluster_sync_all();                       // (a CTA that left counts as arrived)
  // The cluster's CTAs joined, each CTA a share of the outputs, in rank order.
  const uint32_t mine_at = smem_u32(joined);
  for (int e = split * 32 * C_WARPS + threadIdx.x; valid && e < rows * QUADS; e += nsplit * 32 * C_WARPS) {
    const int r = e / QUADS, c = 4 * (e % QUADS);
    float m[C_MAX_SPLIT], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int p = 0; p < C_MAX_SPLIT; ++p) {
      m[p] = p < nsplit ? ld_cluster(map_rank(mine_at, p) + 4u * static_cast<uint32_t>(C_ROWS * D + r)) : -INFINITY;
    }
#pragma unroll
    for (int p = 0; p < C_MAX_SPLIT; ++p) top = fmaxf(top, m[p]);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < nsplit; ++p) {
      const uint32_t at = map_rank(mine_at, p);
      const float4 v = ld_cluster4(at + 4u * static_cast<uint32_t>(r * D + c));
      const float lp = ld_cluster(at + 4u * static_cast<uint32_t>(C_ROWS * D + C_ROWS + r));
      const float f = fast_exp2(ld_cluster(at + 4u * static_cast<uint32_t>(C_ROWS * D + r)) - ref);
      sum = fmaf(f, lp, sum);
      y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
    }
    store(r, c, y, sum);
  }
  cluster_sync_all();                       // no CTA leaves while another may still read its result
}

// The CTAs a cluster may have here, 16 or 8 (set up once per device and kernel).
template <typename T, int D>
cudaError_t cluster_limit(int* most) {
  using C = CacheCfg<D>;
  auto kernel = attend_cache_kernel<T, D>;
  constexpr int kMaxDevices = 64;
  static int limit[kMaxDevices] = {};
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(m);
  if (limit[dev] == 0) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    int clusters = 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C_MAX_SPLIT;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(C_MAX_SPLIT);
    cfg.blockDim = dim3(32 * C_WARPS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      clusters = 0;
    }
    limit[dev] = clusters > 0 ? C_MAX_SPLIT : C_MAX_SPLIT / 2;
  }
  *most = limit[dev];
  return cudaSuccess;
}

template <typename T, int D>
cudaError_t launch_d(const CacheArgs& a, int num_sms, cudaStream_t stream) {
  const int row_blocks = (a.nq * (a.Hq / a.Hkv) + C_ROWS - 1) / C_ROWS;
  const long long units = static_cast<long long>(a.B) * a.Hkv * row_blocks;
  int most = 0;
  cudaError_t e = cluster_limit<T, D>(&most);
  if (e != cudaSuccess) return e;
  // Few units: split them until the CTAs fill the SMs once (two at a time),
  // leaving a warp four chunks.  A second round of such small CTAs costs more than
  // it evens out (4 x 4096 keys, 8 heads: 8 CTAs a unit 11.5 us, 16 25.7 us).  Units
  // that nearly fill them over a long cache: up to four CTAs with at least 32 chunks a
  // warp even out sequences of different lengths (32 x up to 16384 keys, 8 heads: 1 CTA
  // a unit 167 us, 4 155 us, 16 216 us).  More units are not split: lengths that are alike or spread evenly even out
  // by themselves (48 x 1000 keys, 12 heads, in a cache of 32768: 1 CTA a unit 26 us, 2 40 us; 40 x 1 to 16384 keys, 8 heads,
  // 226 to 231 us in any order, 203 for the bytes), a few long ones among short ones do not (2 x 16384 among 38 x 100 120 us, 22).
  const int chunks = (a.cap - 1) / CK + 1;
  int cluster = 1, min_chunks = 4;
  while (2 * cluster <= most && units * 2 * cluster <= 2LL * num_sms && chunks >= 2 * cluster * C_WARPS * min_chunks)
    cluster *= 2;
  while (cluster < 4 && units <= 2LL * num_sms && chunks >= 2 * cluster * C_WARPS * 32) {
    cluster *= 2;
    min_chunks = 32;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
  cfg.blockDim = dim3(32 * C_WARPS);
  cfg.dynamicSmemBytes = CacheCfg<D>::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, attend_cache_kernel<T, D>, a, cluster, min_chunks, row_blocks);
}

}  // namespace

cudaError_t launch_attend_cache(const CacheArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream) {
  if (dt == RRA_BF16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, num_sms, stream) : launch_d<__nv_bfloat16, 128>(a, num_sms, stream);
  return d == 64 ? launch_d<__half, 64>(a, num_sms, stream) : launch_d<__half, 128>(a, num_sms, stream);
}

}  // namespace rra
