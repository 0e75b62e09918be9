// Attention of the new tokens of each sequence over a cache in pages.
//
// Sequence b has n new tokens, packed rows cu_seqlens[b] .. cu_seqlens[b+1] of q, and kv_len[b] keys in the
// cache, the new tokens' own among them, the last ones: key j is row j % page of page
// table[b][j / page].  Row i (query head h) sees the keys j < kv_len - (n - 1 - i):
//   o = sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m),  s_j = <q, k_j>, c = scale log2 e.
//
// paged_few_kernel: few rows a sequence (a decoding step).  The one read of the cache bounds it: a key
// and value row is used by the rows of its head group only.  So a unit is (sequence, key/value head, 16
// of its n * Hq/Hkv rows), the rows filling one mma.sync tile; its keys are dealt out in chunks of 16,
// which lie in one page, to the warps of a cluster of CTAs.  Every warp runs on its own: cp.async copies
// of its next chunks into its own ring (24 KB, so two CTAs keep 192 KB in flight on an SM), the page of
// each looked up one chunk ahead, S = Q K^T, a running reference and sum per row, O += P V.  Then the
// partial results of all warps are joined through distributed shared memory, each CTA a share of the output.
//
// (4 x 4096 keys, 8 of 32 heads, d = 128: 18 us.)
//
// paged_chunk_kernel: tiles of 128 rows on tcgen05, the rows of a tile the G query heads of one key/value head for
// 128 / G tokens, so that a K/V byte read serves all of them.  A CTA has one tile at a time, and an SM two CTAs: while one's
// softmax runs the tensor core works for the other.  Warps of a CTA: 0-3 softmax, a row a thread; 4 loads (the Q tile, then K
// and V blocks of 128 keys through a ring of 64 KB, by copies of as many rows as lie together in a page); 5 products (S = Q K^T,
// O += P V, P read from TMEM); 6 zeroes the V rows behind a sequence's end.
//
// All tiles' key blocks laid end to end are cut into equal shares, one a CTA (each finds its own two cuts from cu_seqlens and
// kv_len), so that contexts of all lengths, chunks and single tokens fill the SMs evenly: a tile cut between CTAs leaves
// each part's sums, reference and normaliser in the workspace, and paged_join_kernel joins them.  32 contexts of 1 to 16384 keys, 8
// of 32 heads, d = 128: 163 to 167 us (1.06 GB, 6.4 to 6.5 TB/s); 2048 new tokens on 16384 keys 378 us cool (515 GFLOP: 1360 TFLOP/s; the
// tensor pipe is active 66 % of the time), 402 to 408 under load (1270); 2 contexts of 16384 keys among 38 of 100 35 us.  What holds
// the chunk is the chain S, softmax, P V of a block, which two CTAs overlap only in part, and at d = 128 a ring of one K and one V
// block, so that a K block is asked for when S of the one before is done (the two were not separated): blocks of 64 keys with two S in turn, so that the softmax
// never waits for a product, took 451 us (each block's own costs twice as often), a share of the exponentials by polynomials
// 404 and more (the unit for them is a third in use here).
//
// In both, the reference of a row moves only when a maximum exceeds it by more than 8 (log2 units), the sum of the
// weights is taken unrounded in fp32, and in fp16 a factor 2^7 that cancels keeps the weights out of the subnormal range.
// For few rows a weight enters the second product as two 16-bit values, the second what the first's rounding leaves: the read
// of the cache bounds that kernel, and the products are no more than 6 % of it (4 x 4096 keys 17.3 -> 17.8 us, four short contexts
// 4.6 -> 4.8, 16 x 4096 of one head 14.5 -> 15.4).  Tiles round it once (relative 2^-8 in bf16, 2^-11 in fp16), which takes
// an output's error from 0.0017 to 0.0023 of its size, its own rounding to bf16 among both: two products took 516 us instead of
// 380 for 2048 tokens on 16384 keys, 102 instead of 82 for a mixed batch, 170 instead of 163 for next tokens of 32 contexts (d = 64
// 121 instead of 92).
// What a page holds from kv_len on reaches no output.
#include <algorithm>
#include <climits>
#include <mutex>

#include "block.cuh"
#include "rows_mma.cuh"
#include "softmax_tc.cuh"
#include "tc_ptx.cuh"
#include "tile_softmax.cuh"

namespace rra {
namespace {

// Sequence b's rows of q and keys; `valid` false: none of its rows are written.
struct PagedSeq {
  int s0, n, len;
  bool valid;
  __device__ PagedSeq(const PagedArgs& a, int b, bool record) {
    s0 = a.cu[b];
    n = a.cu[b + 1] - s0;
    len = a.kv_len[b];
    int code = RRA_DEVERR_NONE;
    if (n < 0 || len < 0) code = RRA_DEVERR_SEQ_NEGATIVE;
    else if (n > a.bound_new || len > a.max_kv) code = RRA_DEVERR_SEQ_TOO_LONG;
    else if (s0 < 0 || s0 > a.cap - n) code = RRA_DEVERR_INDEX_RANGE;
    valid = code == RRA_DEVERR_NONE;
    if (!valid && record) record_error(a.err, code);
  }
};

// ------------------------------------------------------------------ few rows

constexpr int CK = 16;                      // keys of a chunk
constexpr int C_WARPS = 4;
constexpr int C_ROWS = 16;                  // rows of a unit
constexpr int C_RING = 24 * 1024;           // bytes of a warp's ring
constexpr int C_MAX_SPLIT = 16;             // CTAs of a cluster
constexpr float C_MOVE = 8.f;

template <int D>
struct FewCfg {
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
    paged_few_kernel(const PagedArgs a, int cluster, int min_chunks, int row_blocks) {
  using C = FewCfg<D>;
  constexpr bool BF = IsBf16<T>::value == 1;
  extern __shared__ __align__(128) uint8_t smem_few[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int split = static_cast<int>(blockIdx.x) % cluster;        // = the CTA's rank in its cluster
  const int unit = static_cast<int>(blockIdx.x) / cluster;
  const int rb = unit % row_blocks, hk = unit / row_blocks % a.Hkv, b = unit / row_blocks / a.Hkv;
  const int G = a.Hq / a.Hkv;
  start_dependent();
  const PagedSeq sq(a, b, split == 0 && rb == 0 && hk == 0 && threadIdx.x == 0);
  const int rows = sq.valid ? min(C_ROWS, sq.n * G - rb * C_ROWS) : 0;   // row r: token r / G, head hk * G + r % G (r from rb * 16)
  if (rows <= 0) return;                                           // the whole cluster
  const uint32_t ring = smem_u32(smem_few) + static_cast<uint32_t>(warp) * C_RING;

  // Keys that row r of the unit sees: its first `sees(r)` ones (not above zero: none).
  auto sees = [&](int r) { return sq.len - (sq.n - 1 - (rb * C_ROWS + r) / G); };
  const int keys = max(0, sees(rows - 1));
  const int chunks = (keys + CK - 1) / CK;
  // The CTAs that share the keys: no more than give each warp its min_chunks
  // (the host knows only a bound); the others of the cluster leave.
  const int nsplit = min(cluster, max(1, chunks / (C_WARPS * min_chunks)));
  if (split >= nsplit) return;
  const int stride = nsplit * C_WARPS, first = split * C_WARPS + warp;
  const int mine = first < chunks ? (chunks - first + stride - 1) / stride : 0;

  // Page of this warp's i-th chunk.
  const int32_t* table = a.table + static_cast<long long>(b) * a.table_width;
  auto page_of = [&](int i) { return i < mine ? table[(first + i * stride) * CK / a.page] : 0; };
  // Copies of this warp's i-th chunk, which lies in page `id`, into stage s, 16-byte pieces, 128-byte
  // groups of pieces rotated by the row so that ldmatrix meets no bank twice.
  auto piece = [&](int row, int c) { return static_cast<uint32_t>(row * (D * 2) + (((c & ~7) | ((c ^ row) & 7)) << 4)); };
  const long long row_elems = static_cast<long long>(a.Hkv) * D;
  auto fetch = [&](int i, int s, int id) {
    if (id < 0 || id >= a.num_pages) {
      if (lane == 0) record_error(a.err, RRA_DEVERR_INDEX_RANGE);
      id = 0;
    }
    const int k0 = (first + i * stride) * CK;
    const long long base = id * a.page_stride + (k0 % a.page) * row_elems + hk * D;
    const uint32_t dk = ring + static_cast<uint32_t>(s) * (2 * C::TILE), dv = dk + C::TILE;
#pragma unroll
    for (int p = 0; p < CK * D / 8 / 32; ++p) {
      const int x = p * 32 + lane, row = x / (D / 8), c = x % (D / 8);
      const bool in = k0 + row < keys;
      const long long off = base + (in ? row : 0) * row_elems + c * 8;
      cp_async16_or_zero(dk + piece(row, c), static_cast<const T*>(a.k) + off, in ? 16 : 0);
      cp_async16_or_zero(dv + piece(row, c), static_cast<const T*>(a.v) + off, in ? 16 : 0);
    }
  };
  {
    int ids[C::STAGES];
#pragma unroll
    for (int s = 0; s < C::STAGES; ++s) ids[s] = page_of(s);
#pragma unroll
    for (int s = 0; s < C::STAGES; ++s) {
      if (s < mine) fetch(s, s, ids[s]);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  int next_id = page_of(C::STAGES);

  // Q as operand A: rows g and g + 8 of the unit, rows past its end as zeros.
  uint32_t qf[D / 16][4];
  int lim[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = g + 8 * x, rr = rb * C_ROWS + r;
    lim[x] = r < rows ? sees(r) : 0;
    const T* src = static_cast<const T*>(a.q) + (static_cast<long long>(sq.s0) + (r < rows ? rr / G : 0)) * a.q_stride +
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
    uint32_t pf[4], pl[4];                  // the weights, and what their rounding leaves
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
      split2<BF>(p[0], p[1], pf[x], pl[x]);
      split2<BF>(p[2], p[3], pf[2 + x], pl[2 + x]);
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
      mma_16816(o[2 * n], pl, r[0], r[1], T());
      mma_16816(o[2 * n + 1], pl, r[2], r[3], T());
    }
    __syncwarp();                           // the chunk is read before its stage is filled again
    if (i + C::STAGES < mine) fetch(i + C::STAGES, s, next_id);
    next_id = page_of(i + C::STAGES + 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++s == C::STAGES) s = 0;
  }

  // This warp's partial result, over its ring.
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem_few + warp * C_RING);
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
    T* out = static_cast<T*>(a.o) + ((static_cast<long long>(sq.s0) + rr / G) * a.Hq + hk * G + rr % G) * D + c;
    uint2 w;
    w.x = BF ? pack2<__nv_bfloat162>(y.x * inv, y.y * inv) : pack2<__half2>(y.x * inv, y.y * inv);
    w.y = BF ? pack2<__nv_bfloat162>(y.z * inv, y.w * inv) : pack2<__half2>(y.z * inv, y.w * inv);
    *reinterpret_cast<uint2*>(out) = w;
  };
  constexpr int QUADS = D / 4;
  // The CTA's warps joined: O, reference and sum of each row.
  float* joined = reinterpret_cast<float*>(smem_few + C::CTA_PART);
  for (int e = threadIdx.x; e < rows * QUADS; e += 32 * C_WARPS) {
    const int r = e / QUADS, c = 4 * (e % QUADS);
    float m[C_WARPS], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < C_WARPS; ++w) {
      m[w] = reinterpret_cast<const float*>(smem_few + w * C_RING)[C_ROWS * D + r];
      top = fmaxf(top, m[w]);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C_WARPS; ++w) {
      const float* p = reinterpret_cast<const float*>(smem_few + w * C_RING);
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
  for (int e = split * 32 * C_WARPS + threadIdx.x; e < rows * QUADS; e += nsplit * 32 * C_WARPS) {
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

// Clusters of 2, 4, 8 and 16 CTAs that run at once here (asked once per device and kernel; 152 SMs: 152, 74, 36, 14).
template <typename T, int D>
cudaError_t clusters_at_once(int (&most)[4]) {
  using C = FewCfg<D>;
  auto kernel = paged_few_kernel<T, D>;
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices][4] = {};
  static bool asked[kMaxDevices] = {};
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(m);
  if (!asked[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    const bool wide = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int i = 0; i < 4; ++i) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2u << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.gridDim = dim3(2u << i);
      cfg.blockDim = dim3(32 * C_WARPS);
      cfg.dynamicSmemBytes = C::SMEM;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if ((i == 3 && !wide) || cudaOccupancyMaxActiveClusters(&known[dev][i], kernel, &cfg) != cudaSuccess) known[dev][i] = 0;
    }
    (void)cudaGetLastError();
    asked[dev] = true;
  }
  for (int i = 0; i < 4; ++i) most[i] = known[dev][i];
  return cudaSuccess;
}

// CTAs of a unit's cluster: as many as run at once (a second round of such small CTAs costs more than it evens out: 16 contexts of
// 4096 keys, one head, in clusters of 16 21.7 us, of 8 14.7) and leave a warp C_LEAST chunks.
constexpr int C_LEAST = 4;
inline int few_cluster(long long units, int chunks, const int (&at_once)[4]) {
  int c = 1;
  for (int i = 0; i < 4 && units <= at_once[i] && chunks >= 2 * c * C_WARPS * C_LEAST; ++i) c *= 2;
  return c;
}

template <typename T, int D>
cudaError_t launch_few(const PagedArgs& a, cudaStream_t stream, int* launches) {
  const int row_blocks = (a.max_new * (a.Hq / a.Hkv) + C_ROWS - 1) / C_ROWS;
  const long long units = static_cast<long long>(a.B) * a.Hkv * row_blocks;
  int at_once[4];
  cudaError_t e = clusters_at_once<T, D>(at_once);
  if (e != cudaSuccess) return e;
  const int cluster = few_cluster(units, (a.max_kv - 1) / CK + 1, at_once);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
  cfg.blockDim = dim3(32 * C_WARPS);
  cfg.dynamicSmemBytes = FewCfg<D>::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, paged_few_kernel<T, D>, a, cluster, C_LEAST, row_blocks)) != cudaSuccess) return e;
  *launches += 1;
  return cudaSuccess;
}

// -------------------------------------------------------------------- chunks

constexpr int PG_THREADS = 256;              // warps 0-3 softmax, 4 loads, 5 products, 6 tails, 7 lends its registers
constexpr int PG_LOAD_WARP = 4, PG_MMA_WARP = 5, PG_TAIL_WARP = 6;
// Two CTAs an SM: 128 registers a thread at launch, 184 for the softmax warps (a row's 128 scores stay in registers), 72 for the others.
constexpr int PG_REGS_SOFTMAX = 184, PG_REGS_OTHER = 72;
static_assert(PG_REGS_SOFTMAX + PG_REGS_OTHER <= 2 * 128, "register split exceeds the launch's registers");
constexpr uint32_t PG_TMEM_COLS = 256;
constexpr uint32_t PG_SUB = PT * 128;        // one 64-element column group of a tile: 128 rows x 128 B
constexpr long long PG_UNIT_WAIT_CYCLES = 1LL << 36;   // a wait that lasts a whole piece (the warp for the tails)
constexpr int PG_MAX_CTAS = 320;             // two an SM, up to 160 SMs
// In blocks: what a unit costs beside its blocks; the least share of a CTA; no piece is cut shorter than PG_SNAP - PG_START.  (5 tokens on
// 2048 keys 15 us, with 2, 6 and 4 17.5; a mixed batch 82 / 84.)
constexpr int PG_START = 1, PG_SHARE = 2, PG_SNAP = 2;

template <int D>
struct PagedCfg {
  static constexpr uint32_t TILE = (D / 64) * PG_SUB;             // the Q tile, a K block or a V block
  static constexpr int SLOTS = D == 128 ? 2 : 4;                  // K/V ring: 64 KB
  static constexpr uint32_t OFF_KV = TILE;
  static constexpr uint32_t OFF_OUT = OFF_KV + SLOTS * TILE;      // output staging, 4 KB a softmax warp
  static constexpr uint32_t OFF_BAR = OFF_OUT + 4 * 4096;
  static constexpr uint32_t SMEM = OFF_BAR + 512;
  static_assert(SMEM <= 113 * 1024, "two CTAs an SM");
  // TMEM columns: S, O; P over S, or, where there is room (d = 64), beside it: then the next S need not wait for this P V.
  static constexpr bool OWN_P = D == 64;
  static constexpr uint32_t T_S = 0, T_O = PT, T_P = OWN_P ? T_O + D : T_S;
};

// Barrier and word offsets from OFF_BAR.
constexpr uint32_t GB_KV_FULL = 0;      // [4]
constexpr uint32_t GB_KV_EMPTY = 32;    // [4]
constexpr uint32_t GB_Q_FULL = 64, GB_Q_EMPTY = 72;
constexpr uint32_t GB_S_FULL = 80;      // S product done
constexpr uint32_t GB_S_READ = 88;      // the scores are in registers (one arrival per softmax warp; own P)
constexpr uint32_t GB_P_READY = 96;     // P written (one arrival per softmax warp)
constexpr uint32_t GB_PV_DONE = 104;    // P V product done
constexpr uint32_t GB_U_FULL = 112;     // [2] piece descriptor written
constexpr uint32_t GB_U_EMPTY = 128;    // [2] piece finished (softmax, product and tail warps)
constexpr uint32_t GB_TAIL = 144;       // [2] a V block's tail to zero; zeroed
constexpr uint32_t GB_DRAIN = 160;
constexpr uint32_t GW_TMEM = 168, GW_ABORT = 172;
constexpr uint32_t G_DESC = 192;        // [2] x 48 bytes
constexpr uint32_t G_PLAN = 288;        // the CTA's first piece and its end, 40 bytes each
constexpr uint32_t G_SCAN = 368;        // [8] x 8 bytes, one a warp

// What a CTA does at a time: key blocks b0 .. b1 of a unit of up to 128 rows (tokens q0 .. of a sequence times the G heads of
// key/value head hk).  slot < 0: the unit's only piece, whose rows are written out; else where its sums go.
struct PagedPiece {
  int s0, n, len, q0, hk, b, b0, b1, slot;
};

// The workspace: sums of pieces of units that several CTAs share, and who joins them.
struct PagedSpace {
  int* state;       // [2 PG_MAX_CTAS][4]: 1 where a warp's rows of a slot are written
  int* join;        // [PG_MAX_CTAS][8]: pieces of the unit that this CTA begins and others finish (0: none), s0 + q0, tokens, hk
  float2* ml;       // [2 PG_MAX_CTAS][rows]: reference and sum of a row
  float* o;         // [2 PG_MAX_CTAS][D / 4][rows][4]
  int rows;
};
__host__ __device__ inline int paged_space_rows(int max_new, int G) {
  const long long r = static_cast<long long>(max_new) * G;
  return r >= PT ? PT : (static_cast<int>(r) + 31) & ~31;
}
constexpr size_t PG_OFF_JOIN = 2 * PG_MAX_CTAS * 4 * 4, PG_OFF_ML = PG_OFF_JOIN + PG_MAX_CTAS * 8 * 4;
inline size_t paged_space_bytes(int rows, int d) {
  return PG_OFF_ML + static_cast<size_t>(2 * PG_MAX_CTAS) * rows * (8 + static_cast<size_t>(d) * 4);
}
__device__ inline PagedSpace paged_space(void* p, int rows) {
  uint8_t* w = static_cast<uint8_t*>(p);
  PagedSpace s;
  s.state = reinterpret_cast<int*>(w);
  s.join = reinterpret_cast<int*>(w + PG_OFF_JOIN);
  s.ml = reinterpret_cast<float2*>(w + PG_OFF_ML);
  s.o = reinterpret_cast<float*>(w + PG_OFF_ML + static_cast<size_t>(2 * PG_MAX_CTAS) * rows * 8);
  s.rows = rows;
  return s;
}

// Key blocks that the unit of tokens q0 .. q0 + tokens of a sequence sees.
__device__ __forceinline__ int paged_blocks(int n, int len, int q0, int tokens) {
  const int sees = len - n + min(n, q0 + tokens);
  return sees <= 0 ? 0 : (sees + PT - 1) / PT;
}
// The work of one key/value head of a sequence: its units' blocks, and PG_START for each.
__device__ __forceinline__ long long paged_work(int n, int len, int tokens) {
  long long w = 0;
  for (int q0 = 0; q0 < n; q0 += tokens) w += PG_START + paged_blocks(n, len, q0, tokens);
  return w;
}

// Where a cut falls: unit (b, hk, q0) and the work of the unit ahead of the cut (after snapping to the unit's
// ends); the unit starts at work `start` of all.
struct PagedCut {
  int b, hk, q0, off;
  int s0, n, len;                            // of sequence b
  long long start;
};
static_assert(2 * sizeof(PagedCut) <= G_SCAN - G_PLAN, "the plan's place");

// The cut after snapping, as work of its unit of w: one nearer an end than PG_SNAP falls on it, so that the piece ahead of a cut has
// PG_SNAP - PG_START blocks at least and the one behind it PG_SNAP.
__device__ __forceinline__ int paged_snap(int off, int w) {
  if (w - off < PG_SNAP && 2 * off >= w) return w;
  if (off < PG_SNAP) return 0;
  return w - off < PG_SNAP ? w : off;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

template <typename T, int D, bool LIMIT>
__global__ void __launch_bounds__(PG_THREADS, 2)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PagedArgs a, int box_rows, int space_rows) {
  using C = PagedCfg<D>;
  constexpr bool BF = IsBf16<T>::value == 1;
  extern __shared__ __align__(1024) uint8_t smem_paged[];   // the swizzled tiles start 1024-byte aligned
  const uint32_t base = smem_u32(smem_paged), bars = base + C::OFF_BAR;
  auto s_kv = [&](int i) { return base + C::OFF_KV + static_cast<uint32_t>(i) * C::TILE; };
  const uint32_t abort_flag = bars + GW_ABORT;
  const volatile uint32_t* tmem_ptr = reinterpret_cast<const volatile uint32_t*>(smem_paged + C::OFF_BAR + GW_TMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv, tokens = PT / G;               // of a unit
  const PagedSpace space = paged_space(a.space, space_rows);

  if (warp == PG_MMA_WARP) {
    tmem_alloc(bars + GW_TMEM, PG_TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(bars + GB_KV_FULL + 8 * i, 1);
      mbar_init(bars + GB_KV_EMPTY + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + GB_U_FULL + 8 * i, 1);
      mbar_init(bars + GB_U_EMPTY + 8 * i, 6);
      mbar_init(bars + GB_TAIL + 8 * i, 1);
    }
    mbar_init(bars + GB_Q_FULL, 1);
    mbar_init(bars + GB_Q_EMPTY, 1);
    mbar_init(bars + GB_S_FULL, 1);
    mbar_init(bars + GB_S_READ, 4);
    mbar_init(bars + GB_P_READY, 4);
    mbar_init(bars + GB_PV_DONE, 1);
    mbar_init(bars + GB_DRAIN, 1);
    st_shared_u32(abort_flag, 0u);
    fence_barrier_init();
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  start_dependent();

  // ------------------------------------------------------------------ plan
  // All units in order (sequence, key/value head, tokens) laid end to end, in work; CTA c of `active` takes its
  // share, cut between two blocks of a unit where need be.  Every CTA finds its own two cuts.
  const int me = static_cast<int>(blockIdx.x);
  long long* scan = reinterpret_cast<long long*>(smem_paged + C::OFF_BAR + G_SCAN);
  auto block_sum = [&](long long v, long long& before) {     // inclusive prefix by thread in `before`; returns the total
    long long x = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, k);
      if (lane >= k) x += y;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    long long sum = 0, ahead = 0;
#pragma unroll
    for (int w = 0; w < PG_THREADS / 32; ++w) {
      if (w == warp) ahead = sum;
      sum += scan[w];
    }
    before = ahead + x;
    return sum;
  };
  auto work_of = [&](int b, bool record) -> long long {
    if (b >= a.B) return 0;
    const PagedSeq sq(a, b, record);
    return sq.valid ? paged_work(sq.n, sq.len, tokens) * a.Hkv : 0;
  };
  long long total = 0, upto = 0, mine = work_of(tid, me == 0);
  total = block_sum(mine, upto);
  for (int b0 = PG_THREADS; b0 < a.B; b0 += PG_THREADS) {
    long long x;
    total += block_sum(work_of(b0 + tid, me == 0), x);
  }
  const long long active = min(static_cast<long long>(gridDim.x), max(1LL, total / PG_SHARE));
  const long long from = total * me / active, to = total * (me + 1) / active;
  PagedCut* plan = reinterpret_cast<PagedCut*>(smem_paged + C::OFF_BAR + G_PLAN);   // [2]: from, to
  if (tid < 2) {
    plan[tid].b = a.B;                                       // the end of all
    plan[tid].off = 0;
  }
  __syncthreads();
  if (me < active && total > 0) {
    long long done = 0;
    for (int b0 = 0; b0 < a.B; b0 += PG_THREADS) {
      long long in = mine, incl = upto;
      if (b0 > 0) {
        in = work_of(b0 + tid, false);
      }
      long long sum = b0 > 0 || a.B > PG_THREADS ? block_sum(in, incl) : total;
      const long long seq_from = done + incl - in;
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        const long long x = e == 0 ? from : to;
        if (in > 0 && x >= seq_from && x < seq_from + in) {
          const int b = b0 + tid;
          const PagedSeq sq(a, b, false);
          const long long per = in / a.Hkv;
          PagedCut c;
          c.b = b;
          c.s0 = sq.s0;
          c.n = sq.n;
          c.len = sq.len;
          c.hk = static_cast<int>((x - seq_from) / per);
          long long at = seq_from + c.hk * per;
          c.q0 = 0;
          int w = PG_START + paged_blocks(sq.n, sq.len, 0, tokens);
          while (x >= at + w) {
            at += w;
            c.q0 += tokens;
            w = PG_START + paged_blocks(sq.n, sq.len, c.q0, tokens);
          }
          c.off = paged_snap(static_cast<int>(x - at), w);
          c.start = at;
          plan[e] = c;
        }
      }
      done += sum;
    }
  }
  if (tid < 8) {
    if (tid == 0) space.join[me * 8] = 0;
    space.state[me * 8 + tid] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  bool bad = false;
  // A bounded wait; every lane of the warp leaves with the same `bad`.
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (!mbar_wait_limited<LIMIT>(b, parity, abort_flag, a.wait_limit)) bad = true;
    bad = __any_sync(0xffffffffu, bad);
    return !bad;
  };
  auto read_piece = [&](int i) {
    const uint32_t d = bars + G_DESC + 48u * static_cast<uint32_t>(i & 1);
    PagedPiece u;
    u.s0 = static_cast<int>(ld_shared_u32(d));
    u.n = static_cast<int>(ld_shared_u32(d + 4));
    u.len = static_cast<int>(ld_shared_u32(d + 8));
    u.q0 = static_cast<int>(ld_shared_u32(d + 12));
    u.hk = static_cast<int>(ld_shared_u32(d + 16));
    u.b0 = static_cast<int>(ld_shared_u32(d + 20));
    u.b1 = static_cast<int>(ld_shared_u32(d + 24));
    u.slot = static_cast<int>(ld_shared_u32(d + 28));
    return u;
  };
  // The last block of a sequence that a piece reads, and the V rows behind its end in the product's last step of 16 (0: none).
  auto pad_of = [&](const PagedPiece& u) { return u.b1 * PT >= u.len ? -u.len & 15 : 0; };

  if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PG_REGS_OTHER));
    if (warp == PG_LOAD_WARP) {
      // ------------------------------------------------------------ loads
      PagedCut cut = plan[0];
      const PagedCut end = plan[1];
      uint32_t it = 0;
      const int boxes = PT / box_rows, box = lane % boxes, half = lane / boxes;   // lanes of half >= D / 64 copy nothing
      // The cut's unit may lie behind it (snapped to the unit's end).
      for (int i = 0, nq = 0; !bad;) {
        PagedPiece u;
        u.s0 = -1;
        bool more = cut.b < a.B && !(cut.b == end.b && cut.hk == end.hk && cut.q0 == end.q0 && cut.off >= end.off);
        if (more && (cut.b > end.b || (cut.b == end.b && (cut.hk > end.hk || (cut.hk == end.hk && cut.q0 > end.q0))))) more = false;
        if (more) {
          if (cut.q0 >= cut.n) {                             // to the next head, or the next sequence with rows
            cut.q0 = 0;
            cut.off = 0;
            if (++cut.hk == a.Hkv) {
              cut.hk = 0;
              for (++cut.b; cut.b < a.B; cut.b += 32) {
                const PagedSeq sq(a, min(cut.b + lane, a.B - 1), false);
                const unsigned live = __ballot_sync(0xffffffffu, cut.b + lane < a.B && sq.valid && sq.n > 0);
                if (live == 0u) continue;
                const int src = __ffs(live) - 1;
                cut.b += src;
                cut.s0 = __shfl_sync(0xffffffffu, sq.s0, src);
                cut.n = __shfl_sync(0xffffffffu, sq.n, src);
                cut.len = __shfl_sync(0xffffffffu, sq.len, src);
                break;
              }
            }
            continue;
          }
          const int nb = paged_blocks(cut.n, cut.len, cut.q0, tokens), w = PG_START + nb;
          const bool last = cut.b == end.b && cut.hk == end.hk && cut.q0 == end.q0;
          const int off1 = last ? end.off : w;
          u.s0 = cut.s0;
          u.n = cut.n;
          u.len = cut.len;
          u.q0 = cut.q0;
          u.hk = cut.hk;
          u.b = cut.b;
          u.b0 = max(0, cut.off - PG_START);
          u.b1 = max(0, off1 - PG_START);
          u.slot = cut.off > 0 ? 2 * me : (off1 < w ? 2 * me + 1 : -1);
          if (u.slot == 2 * me + 1 && lane == 0) {
            // The unit goes on in the next CTAs, up to the last whose share begins inside it; its pieces are joined in
            // their order.
            long long c = min(active - 1, (end.start + w) * active / total + 1);
            for (; c > me + 1; --c) {
              const long long x = total * c / active - end.start;
              if (x < w && paged_snap(static_cast<int>(x), w) != w) break;
            }
            const int pieces = static_cast<int>(c - me) + 1;
            int* j = space.join + me * 8;
            j[1] = cut.s0 + cut.q0;
            j[2] = min(tokens, cut.n - cut.q0);
            j[3] = cut.hk;
            j[0] = pieces;
          }
          const bool skip = cut.off >= w;                    // the cut lies at the unit's end
          cut.off = 0;
          cut.q0 += tokens;
          if (skip) continue;
        }
        if (i >= 2 && !wait(bars + GB_U_EMPTY + 8 * (i & 1), ((i >> 1) - 1) & 1)) break;
        if (lane == 0) {
          const uint32_t d = bars + G_DESC + 48u * static_cast<uint32_t>(i & 1);
          st_shared_u32(d, static_cast<uint32_t>(u.s0));
          if (more) {
            st_shared_u32(d + 4, static_cast<uint32_t>(u.n));
            st_shared_u32(d + 8, static_cast<uint32_t>(u.len));
            st_shared_u32(d + 12, static_cast<uint32_t>(u.q0));
            st_shared_u32(d + 16, static_cast<uint32_t>(u.hk));
            st_shared_u32(d + 20, static_cast<uint32_t>(u.b0));
            st_shared_u32(d + 24, static_cast<uint32_t>(u.b1));
            st_shared_u32(d + 28, static_cast<uint32_t>(u.slot));
          }
          mbar_arrive(bars + GB_U_FULL + 8 * (i & 1));
        }
        __syncwarp();
        ++i;
        if (!more) break;
        if (u.b0 == u.b1) continue;                          // no keys: zeros are written
        const int32_t* table = a.table + static_cast<long long>(u.b) * a.table_width;
        const int key0 = box * box_rows;                     // of this lane's box in a block
        auto page_of = [&](int j) {
          const long long key = static_cast<long long>(j) * PT + key0;
          return half < D / 64 && j < u.b1 && key < u.len ? table[key / a.page] : 0;
        };
        int id = page_of(u.b0);
        if (nq > 0 && !wait(bars + GB_Q_EMPTY, (nq - 1) & 1)) break;
        ++nq;
        if (lane == 0) {
          mbar_expect_tx(bars + GB_Q_FULL, static_cast<uint32_t>(G * tokens) * 128u * (D / 64));
          for (int g = 0; g < D / 64; ++g)
            tma_load_3d(base + g * PG_SUB, &map_q, 64 * g, u.hk * G, u.s0 + u.q0, bars + GB_Q_FULL);
        }
        for (int j = u.b0; j < u.b1 && !bad; ++j) {
          if (id < 0 || id >= a.num_pages) {
            record_error(a.err, RRA_DEVERR_INDEX_RANGE);
            id = 0;
          }
          const int keys = min(PT, u.len - j * PT), used = (keys + box_rows - 1) / box_rows;
          const int row = static_cast<int>((static_cast<long long>(j) * PT + key0) % a.page);
          for (int kv = 0; kv < 2; ++kv) {
            const int s = static_cast<int>(it % C::SLOTS);
            const uint32_t full = bars + GB_KV_FULL + 8 * s;
            if (it >= C::SLOTS && !wait(bars + GB_KV_EMPTY + 8 * s, (it / C::SLOTS - 1) & 1)) break;
            ++it;
            if (lane == 0) mbar_expect_tx(full, static_cast<uint32_t>(used * box_rows) * 128u * (D / 64));
            __syncwarp();
            if (half < D / 64 && box < used)
              tma_load_4d(s_kv(s) + half * PG_SUB + key0 * 128, kv == 0 ? &map_k : &map_v, 64 * half, u.hk, row, id, full);
            __syncwarp();
          }
          id = page_of(j + 1);
        }
      }
    } else if (warp == PG_TAIL_WARP) {
      // ------------------------------------------------------------ tails
      // V rows [keys, 16 ceil(keys / 16)) of a sequence's last block: zeros, whatever the page holds there.  The product
      // thread hands the block over once it has landed and gets it back before its P V.
      uint32_t kv0 = 0, done = 0;
      for (int i = 0;; ++i) {
        if (!mbar_wait_limited<LIMIT, PG_UNIT_WAIT_CYCLES>(bars + GB_U_FULL + 8 * (i & 1), (i >> 1) & 1, abort_flag, a.unit_wait_limit))
          bad = true;
        bad = __any_sync(0xffffffffu, bad);
        if (bad) break;
        const PagedPiece u = read_piece(i);
        if (u.s0 < 0) break;
        const int pad = u.b0 < u.b1 ? pad_of(u) : 0;
        kv0 += 2 * static_cast<uint32_t>(u.b1 - u.b0);
        if (pad > 0) {
          if (!mbar_wait_limited<LIMIT, PG_UNIT_WAIT_CYCLES>(bars + GB_TAIL, done & 1, abort_flag, a.unit_wait_limit)) bad = true;
          bad = __any_sync(0xffffffffu, bad);
          if (bad) break;
          ++done;
          const uint32_t sv = s_kv(static_cast<int>((kv0 - 1) % C::SLOTS)) + static_cast<uint32_t>(u.len - (u.b1 - 1) * PT) * 128u;
          for (int z = lane; z < pad * 8 * (D / 64); z += 32) {
            const int g = z / (pad * 8), r = z % (pad * 8);
            st_shared_v4(sv + g * PG_SUB + r * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) {
          if (pad > 0) mbar_arrive(bars + GB_TAIL + 8);
          mbar_arrive(bars + GB_U_EMPTY + 8 * (i & 1));
        }
      }
    } else if (warp == PG_MMA_WARP) {
      // ------------------------------------------------------------ products
      if (elect_one()) {
        auto wait1 = [&](uint32_t b, uint32_t parity) {
          if (!mbar_wait_limited<LIMIT>(b, parity, abort_flag, a.wait_limit)) bad = true;
          return !bad;
        };
        const uint32_t idesc_s = idesc_f16(BF ? 1u : 0u, 0, PT, PT);
        const uint32_t idesc_pv = idesc_f16(BF ? 1u : 0u, 1, PT, D);
        const uint64_t dq = sdesc(base, 16, 1024), dk0 = sdesc(s_kv(0), 16, 1024), dv0 = sdesc(s_kv(0), PG_SUB, 1024);
        uint32_t it = 0, ns = 0, npv = 0, ntail = 0, nq = 0;   // ring, S, P V, tails and Q tiles so far
        auto slot_full = [&](uint32_t idx) {
          return wait1(bars + GB_KV_FULL + 8 * (idx % C::SLOTS), (idx / C::SLOTS) & 1);
        };
        // S with the K block at ring index idx, once S's columns are free: P V done with the P over them, or (own P) the scores read.
        auto next_s = [&](uint32_t idx, bool last) {
          if (!slot_full(idx)) return false;
          const uint32_t n = C::OWN_P ? ns : npv;
          if (n > 0 && !wait1(bars + (C::OWN_P ? GB_S_READ : GB_PV_DONE), (n - 1) & 1)) return false;
          ++ns;
          tc_fence_after();
          const uint64_t dk = dk0 + (idx % C::SLOTS) * (C::TILE >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * PG_SUB + (kk % 4) * 32) >> 4;
            umma_f16(tmem + C::T_S, dq + off, dk + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(bars + GB_S_FULL);
          umma_commit(bars + GB_KV_EMPTY + 8 * (idx % C::SLOTS));
          if (last) umma_commit(bars + GB_Q_EMPTY);
          return true;
        };
        for (int i = 0; !bad; ++i) {
          if (!wait1(bars + GB_U_FULL + 8 * (i & 1), (i >> 1) & 1)) break;
          const PagedPiece u = read_piece(i);
          if (u.s0 < 0) break;
          const int count = u.b1 - u.b0;
          if (count > 0) {
            if (!wait1(bars + GB_Q_FULL, nq & 1)) break;
            ++nq;
            if (!next_s(it, count == 1)) break;
            for (int j = 0; j < count && !bad; ++j) {
              const uint32_t vi = it + 2 * j + 1;
              if (!slot_full(vi)) break;
              const int keys = min(PT, u.len - (u.b0 + j) * PT), ksteps = (keys + 15) / 16;
              if (keys & 15) {
                mbar_arrive(bars + GB_TAIL);
                if (!wait1(bars + GB_TAIL + 8, ntail & 1)) break;
                ++ntail;
              }
              if (C::OWN_P && j + 1 < count && !next_s(vi + 1, j + 2 == count)) break;
              if (!wait1(bars + GB_P_READY, npv & 1)) break;
              ++npv;
              tc_fence_after();
              const uint64_t dv = dv0 + (vi % C::SLOTS) * (C::TILE >> 4);
#pragma unroll
              for (int kk = 0; kk < PT / 16; ++kk) {
                if (kk < ksteps)
                  umma_f16_tmem_a(tmem + C::T_O, tmem + C::T_P + kk * 8, dv + kk * (2048 >> 4), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
              }
              umma_commit(bars + GB_PV_DONE);
              umma_commit(bars + GB_KV_EMPTY + 8 * (vi % C::SLOTS));
              if (!C::OWN_P && j + 1 < count && !next_s(vi + 1, j + 2 == count)) break;
            }
            it += 2 * static_cast<uint32_t>(count);
          }
          if (bad) break;
          mbar_arrive(bars + GB_U_EMPTY + 8 * (i & 1));
        }
        if (!bad) {
          umma_commit(bars + GB_DRAIN);
          wait1(bars + GB_DRAIN, 0);
        }
      }
      bad = __any_sync(0xffffffffu, bad);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PG_REGS_SOFTMAX));
    const int row = tid;
    const uint32_t recip = (65536u + G - 1) / G;             // x / G for x < 128
    const int tok = static_cast<int>((row * recip) >> 16);   // the row's token; tok >= tokens: none
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::T_S, tO = tmem + lane_off + C::T_O, tP = tmem + lane_off + C::T_P;
    const uint32_t stg = base + C::OFF_OUT + static_cast<uint32_t>(warp) * 4096u;
    uint32_t count = 0;                                      // blocks so far
    for (int i = 0;; ++i) {
      if (!wait(bars + GB_U_FULL + 8 * (i & 1), (i >> 1) & 1)) break;
      const PagedPiece u = read_piece(i);
      if (u.s0 < 0) break;
      const int rows = min(tokens, u.n - u.q0) * G;          // of the unit
      const int sees = row < rows ? u.len - u.n + 1 + u.q0 + tok : 0;
      const int clear = (u.len - u.n + 1 + u.q0) / PT;       // blocks that every row sees whole (0 where that is negative)
      float m_ref = -INFINITY, l_run = 0.f;
      for (int j = u.b0; j < u.b1; ++j) {
        if (!wait(bars + GB_S_FULL, count & 1)) break;
        tc_fence_after();
        float s[PT], mx;
        if (j < clear) mx = prompt_scores<false>(tS, PT, s);
        else mx = prompt_scores<true>(tS, sees - j * PT, s);
        if constexpr (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + GB_S_READ);
          // P and O are free once the P V product before this one is done.
          if (count > 0 && !wait(bars + GB_PV_DONE, (count - 1) & 1)) break;
          tc_fence_after();
        }
        ++count;
        const float x = mx * a.scale_log2;
        const bool move = x > m_ref + P_MOVE;
        if (__any_sync(0xffffffffu, move)) {
          const float alpha = move ? fast_exp2(m_ref - x) : 1.f;
          if (move) m_ref = x;
          l_run *= alpha;
          if (j > u.b0) prompt_rescale<D>(tO, alpha);
        }
        l_run += prompt_weights<BF>(tP, s, a.scale_log2, m_ref);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + GB_P_READY);
      }
      if (bad) break;
      if (u.b1 > u.b0) {
        if (!wait(bars + GB_PV_DONE, (count - 1) & 1)) break;
        tc_fence_after();
      }
      if (u.slot >= 0) {
        // Sums of a piece: row by lane, 16 bytes each, so that a warp writes 512 bytes at a time.
        const bool in = row < rows;
        if (in) space.ml[static_cast<size_t>(u.slot) * space.rows + row] = make_float2(m_ref, l_run);
        float* to_o = space.o + (static_cast<size_t>(u.slot) * (D / 4) * space.rows + row) * 4;
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
          float o[32];
          tmem_ld32(tO + 32 * g, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (in) *reinterpret_cast<float4*>(to_o + static_cast<size_t>(8 * g + k) * space.rows * 4) = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        if (lane == 0) space.state[u.slot * 4 + warp] = 1;
      } else {
        const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
        // 64 columns at a time through the warp's 4 KB of staging (rows of 128 bytes, 16-byte chunks swizzled): whole
        // row pieces leave, four to an instruction.
        T* out = static_cast<T*>(a.o) + (static_cast<long long>(u.s0 + u.q0) * a.Hq + u.hk * G) * D;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          float o[64];
          if (u.b1 > u.b0) {
            tmem_ld32_nowait(tO + 64 * g, o);
            tmem_ld32_nowait(tO + 64 * g + 32, o + 32);
            tmem_wait_ld32(o);
            tmem_wait_ld32(o + 32);
          } else {
#pragma unroll
            for (int k = 0; k < 64; ++k) o[k] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pack2<Tout2<T>>(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
            st_shared_v4(stg + lane * 128 + ((k ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = 4 * k + (lane >> 3), cc = lane & 7, r = warp * 32 + rr;
            const uint4 v = ld_shared_v4(stg + rr * 128 + ((cc ^ (rr & 7)) << 4));
            const int t = static_cast<int>((r * recip) >> 16);
            if (r < rows) *reinterpret_cast<uint4*>(out + (static_cast<long long>(t) * a.Hq + (r - t * G)) * D + 64 * g + 8 * cc) = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + GB_U_EMPTY + 8 * (i & 1));
    }
  }
  if (bad && lane == 0) {
    st_shared_u32(abort_flag, 1u);
    record_error(a.err, RRA_DEVERR_WAIT_TIMEOUT);
  }

  // Teardown: after an abort, copies and products still in flight get a
  // bounded grace period (~1 ms) to land before the TMEM is released.
  tc_fence_before();
  __syncthreads();
  if (warp == PG_MMA_WARP) {
    if (lane == 0 && ld_shared_volatile_u32(abort_flag) != 0u) {
      const long long t0 = clock64();
      while (clock64() - t0 < 2000000LL) {
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, PG_TMEM_COLS);
  }
}

// Up to 16 rows of a head group go as rows of a warp's tile where that takes less by this estimate, in us: the bytes within the
// bounds at 6.2 TB/s, with 6 for the rest, or the chain of a warp's chunks; as tiles of 128 rows the bytes and 11, in
// even shares.  (Next tokens, 32 / 8 heads, d = 128, few rows / tiles: 4 x 1024 keys 8.4 / 12.7, 4 x 8192 27.6 / 31.4, 32 x 2048
// 43.7 / 53.7, 1 x 16384 23.5 / 22.3, 1 x 32768 39.7 / 33.1; 8 x 4096, 12 heads, d = 64 27.6 / 27.7; few rows 0.4 to 0.8 more since their
// weights have two parts, which changes no choice here.)  The clusters that run at once are written out, those of 152 SMs: the
// workspace is sized by this rule too, where there may be no device to ask (the launch asks it, and fits its clusters to the answer).  A chain of over 40 us is a
// matter of lengths that are alike: 2 contexts of 16384 keys among 38 of 100 187 / 35.  Nor has a grid more than 2^31 - 1 units.
bool paged_by_chunks(int B, int max_new, int max_kv, int Hkv, int G, int d) {
  if (G > PT) return false;
  if (static_cast<long long>(max_new) * G > C_ROWS || static_cast<long long>(B) * Hkv > INT_MAX) return true;
  constexpr int at_once[4] = {152, 74, 36, 14};
  const int chunks = (max_kv - 1) / CK + 1, per_unit = C_WARPS * few_cluster(static_cast<long long>(B) * Hkv, chunks, at_once);
  const double chain = ((chunks - 1) / per_unit + 1) * (d == 128 ? 1.0 : 0.7);
  const double bytes = static_cast<double>(B) * max_kv * Hkv * d * 4 / 6.2e6;
  return chain > 40 || std::max(bytes, chain) + 6 > bytes + 11;
}

// Joins the pieces of the unit that CTA blockIdx.x began and the CTAs behind it went on with: 8 neighbouring columns of a row at
// a time.  Where the pieces are many, eight lanes share them (every eighth each), so that no chain of loads is as long as
// they are; where they are few, a lane has them all, all of their loads at once, and a warp reads 512 bytes at a time.  The
// order of additions is that of the pieces by lane, then of the lanes.
constexpr int PJ_THREADS = 256, PJ_SPLIT = 8, PJ_FEW = 4;
template <typename T, int D, int LANES>
__device__ __forceinline__ void paged_join(const PagedArgs& a, const PagedSpace& space, const int4 j) {
  constexpr bool BF = IsBf16<T>::value == 1;
  const int me = static_cast<int>(blockIdx.x), pieces = j.x, G = a.Hq / a.Hkv, rows = j.z * G, hk = j.w;
  const int l = static_cast<int>(threadIdx.x) % LANES;
  auto slot_of = [&](int p) { return static_cast<size_t>(p == 0 ? 2 * me + 1 : 2 * (me + p)); };
  constexpr int PER_WARP = 32 / LANES, PER_CTA = PJ_THREADS / LANES;
  constexpr int AT_ONCE = LANES == 1 ? PJ_FEW : 2;             // pieces of a lane on their way together
  const int items = rows * (D / 8);
  // Whole warps go round together: their items may end before the round does.
  for (int e0 = static_cast<int>(blockIdx.y) * PER_CTA + static_cast<int>(threadIdx.x) / 32 * PER_WARP; e0 < items; e0 += PER_CTA * PJ_SPLIT) {
    const int e = min(e0 + static_cast<int>(threadIdx.x) % 32 / LANES, items - 1);
    const int c = e / rows, row = e - c * rows;
    float m = -INFINITY, sum = 0.f, y[8] = {};   // this lane's pieces so far, against reference m
    bool whole = true;                       // a CTA that gave up a wait has written no sums
    for (int p0 = l; p0 < pieces; p0 += AT_ONCE * LANES) {
      float2 ml[AT_ONCE];
      float4 u[AT_ONCE], v[AT_ONCE];
      float top = m;
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        u[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int p = p0 + i * LANES;
        if (p < pieces) {
          const size_t s = slot_of(p);
          const float* o = space.o + ((s * (D / 4) + 2 * c) * space.rows + row) * 4;
          whole = whole && space.state[s * 4 + (row >> 5)] == 1;
          ml[i] = space.ml[s * space.rows + row];
          u[i] = *reinterpret_cast<const float4*>(o);
          v[i] = *reinterpret_cast<const float4*>(o + static_cast<size_t>(space.rows) * 4);
        }
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) top = fmaxf(top, ml[i].x);
      const float ref = top == -INFINITY ? 0.f : top, old = fast_exp2(m - ref);
      m = top;
      sum *= old;
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= old;
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        if (p0 + i * LANES >= pieces) continue;
        const float f = fast_exp2(ml[i].x - ref);
        sum = fmaf(f, ml[i].y, sum);
        y[0] = fmaf(f, u[i].x, y[0]);
        y[1] = fmaf(f, u[i].y, y[1]);
        y[2] = fmaf(f, u[i].z, y[2]);
        y[3] = fmaf(f, u[i].w, y[3]);
        y[4] = fmaf(f, v[i].x, y[4]);
        y[5] = fmaf(f, v[i].y, y[5]);
        y[6] = fmaf(f, v[i].z, y[6]);
        y[7] = fmaf(f, v[i].w, y[7]);
      }
    }
    if constexpr (LANES > 1) {
      float top = m;
#pragma unroll
      for (int k = 1; k < LANES; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float f = fast_exp2(m - (top == -INFINITY ? 0.f : top));
      sum *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= f;
#pragma unroll
      for (int k = 1; k < LANES; k <<= 1) {
        whole = __shfl_xor_sync(0xffffffffu, static_cast<int>(whole), k) != 0 && whole;
        sum += __shfl_xor_sync(0xffffffffu, sum, k);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += __shfl_xor_sync(0xffffffffu, y[i], k);
      }
    }
    if (l != 0 || !whole) continue;
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = BF ? pack2<__nv_bfloat162>(y[2 * i] * inv, y[2 * i + 1] * inv) : pack2<__half2>(y[2 * i] * inv, y[2 * i + 1] * inv);
    const int t = row / G;
    T* out = static_cast<T*>(a.o) + ((static_cast<long long>(j.y) + t) * a.Hq + hk * G + (row - t * G)) * D + 8 * c;
    *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename T, int D>
__global__ void __launch_bounds__(PJ_THREADS) paged_join_kernel(const PagedArgs a, int space_rows) {
  start_dependent();
  const PagedSpace space = paged_space(a.space, space_rows);
  const int4 j = *reinterpret_cast<const int4*>(space.join + blockIdx.x * 8);   // pieces, first row of q, tokens, hk
  if (j.x > PJ_FEW) paged_join<T, D, 8>(a, space, j);
  else if (j.x > 1) paged_join<T, D, 1>(a, space, j);
}

PFN_cuTensorMapEncodeTiled_v12000 paged_encode_fn() {
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

// Row tensors [rows, H, d] (box: `tokens` rows of G heads) and pools [pages, page, Hkv, d] (box: rows of a page of one head), 64
// elements wide, 128-byte swizzle.  L2 takes in what is asked for: 256 bytes of a row at d = 128, 128 at d = 64, where more would be the
// next head's, which another CTA reads at another time (32 contexts of 1 to 16384 keys, d = 64: 98 us against 117).
cudaError_t encode(CUtensorMap* map, const void* ptr, bool bf16, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = paged_encode_fn()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                       static_cast<cuuint32_t>(rank), const_cast<void*>(ptr), dims, strides, box, estr,
                                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                       dims[0] == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t make_map_q(CUtensorMap* map, const PagedArgs& a, int D, bool bf16) {
  const int G = a.Hq / a.Hkv;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.cap)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(a.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(PT / G)};
  return encode(map, a.q, bf16, 3, dims, strides, box);
}
cudaError_t make_map_pages(CUtensorMap* map, const void* ptr, const PagedArgs& a, int D, bool bf16, int box_rows) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(a.page),
                              static_cast<cuuint64_t>(a.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(a.Hkv) * D * 2,
                                 static_cast<cuuint64_t>(a.page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1};
  return encode(map, ptr, bf16, 4, dims, strides, box);
}

template <typename T, int D, bool LIMIT>
cudaError_t launch_chunk(const PagedArgs& a, int num_sms, cudaStream_t stream, int* launches) {
  using C = PagedCfg<D>;
  if (paged_encode_fn() == nullptr) return cudaErrorNotSupported;
  auto kernel = paged_chunk_kernel<T, D, LIMIT>;
  constexpr int kMaxDevices = 64;
  static bool attr_set[kMaxDevices] = {};
  static std::mutex m;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(m);
    if (!attr_set[dev]) {
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  const bool bf16 = IsBf16<T>::value == 1;
  int box_rows = PT;                         // of a copy: the largest power of two that divides the page, up to a block
  while (a.page % box_rows != 0) box_rows /= 2;
  CUtensorMap mq, mk, mv;
  if ((e = make_map_q(&mq, a, D, bf16)) != cudaSuccess) return e;
  if ((e = make_map_pages(&mk, a.k, a, D, bf16, box_rows)) != cudaSuccess) return e;
  if ((e = make_map_pages(&mv, a.v, a, D, bf16, box_rows)) != cudaSuccess) return e;
  const int G = a.Hq / a.Hkv, tokens = PT / G, rows = paged_space_rows(a.max_new, G);
  // No more CTAs than the bounds leave work for.
  const long long units = std::min(static_cast<long long>(a.B) * ((a.max_new - 1) / tokens + 1), a.cap / tokens + static_cast<long long>(a.B)) * a.Hkv;
  const long long share = units * (PG_START + (a.max_kv - 1) / PT + 1) / PG_SHARE + 1;
  const int grid = static_cast<int>(std::min<long long>(share, std::min(2 * num_sms, PG_MAX_CTAS)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(PG_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, a, box_rows, rows)) != cudaSuccess) return e;
  *launches += 1;
  if (grid == 1 || PG_START + (a.max_kv - 1) / PT + 1 < 2 * PG_SNAP) return cudaSuccess;   // no unit is cut
  cfg.gridDim = dim3(static_cast<unsigned>(grid), PJ_SPLIT);
  cfg.blockDim = dim3(PJ_THREADS);
  cfg.dynamicSmemBytes = 0;
  if ((e = cudaLaunchKernelEx(&cfg, paged_join_kernel<T, D>, a, rows)) != cudaSuccess) return e;
  *launches += 1;
  return cudaSuccess;
}

template <typename T, int D>
cudaError_t launch_d(PagedArgs a, int num_sms, cudaStream_t stream, int* launches) {
  if (!paged_by_chunks(a.B, a.max_new, a.max_kv, a.Hkv, a.Hq / a.Hkv, D)) return launch_few<T, D>(a, stream, launches);
  const long long each = std::min(a.wait_limit > 0 ? a.wait_limit : WAIT_LIMIT_CYCLES, 1LL << 38);
  a.unit_wait_limit = each * (1 + a.max_kv / PT);            // at most 2^38 x 2^23
  return a.wait_limit > 0 ? launch_chunk<T, D, true>(a, num_sms, stream, launches) : launch_chunk<T, D, false>(a, num_sms, stream, launches);
}

}  // namespace

size_t attend_paged_space(int B, int max_new, int max_kv, int Hkv, int G, int d) {
  return paged_by_chunks(B, max_new, max_kv, Hkv, G, d) ? paged_space_bytes(paged_space_rows(max_new, G), d) : 0;
}

cudaError_t launch_attend_paged(const PagedArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream, int* launches) {
  if (dt == RRA_BF16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, num_sms, stream, launches) : launch_d<__nv_bfloat16, 128>(a, num_sms, stream, launches);
  return d == 64 ? launch_d<__half, 64>(a, num_sms, stream, launches) : launch_d<__half, 128>(a, num_sms, stream, launches);
}

}  // namespace rra
