// The softmax of a tile of 128 rows against a block of 128 keys, a row a thread, as the tcgen05 kernels of
// attend_prompt and attend_paged share it: scores from TMEM, weights back to it.
#pragma once

#include "block.cuh"
#include "softmax_tc.cuh"
#include "tc_ptx.cuh"

namespace rra {

constexpr int PT = 128;                      // rows of a tile, keys of a block
constexpr float P_MOVE = 8.f;                // log2 units by which a maximum may exceed the reference

// The row's 128 scores into registers (columns from `lim` on invisible when
// MASK) and their maximum.
template <bool MASK>
__device__ __forceinline__ float prompt_scores(uint32_t tS, int lim, float (&s)[PT]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) tmem_ld32_nowait(tS + 32 * g, s + 32 * g);
#pragma unroll
  for (int g = 0; g < 4; ++g) tmem_wait_ld32(s + 32 * g);
  if constexpr (MASK) {
    // By groups of 32 columns: those that every lane sees are left as they are
    // (on the diagonal a warp's rows end in one group).
    const int least = __reduce_min_sync(0xffffffffu, lim);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (least < 32 * g + 32) {
#pragma unroll
        for (int i = 32 * g; i < 32 * g + 32; ++i) s[i] = i < lim ? s[i] : -INFINITY;
      }
    }
  }
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < PT; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mx[k] = max3f(mx[k], s[i + 2 * k], s[i + 2 * k + 1]);
  }
  return max3f(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
}

// The row's D columns of O times alpha.
template <int D>
__device__ __forceinline__ void prompt_rescale(uint32_t tO, float alpha) {
#pragma unroll
  for (int g = 0; g < D / 16; ++g) {
    float o[16];
    tmem_ld16(tO + 16 * g, o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= alpha;
    tmem_st8(tO + 16 * g, reinterpret_cast<const uint32_t*>(o));
    tmem_st8(tO + 16 * g + 8, reinterpret_cast<const uint32_t*>(o) + 8);
  }
}

// The weights of the row's scores to tP, two per TMEM column, against the
// reference m_ref; returns their sum.
template <bool BF>
__device__ __forceinline__ float prompt_weights(uint32_t tP, const float (&s)[PT], float c2, float m_ref) {
  // A row that has seen only -inf scores keeps its reference at -inf: weights 0.
  const float mu = (m_ref == -INFINITY ? 0.f : m_ref) - (BF ? 0.f : 7.f);
  const uint64_t c2x2 = pack_f2(c2, c2), nm2 = pack_f2(-mu, -mu);
  uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
  for (int g = 0; g < PT / 16; ++g) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = 16 * g + 2 * i;
      float x0, x1;
      unpack_f2(fma_f2(pack_f2(s[col], s[col + 1]), c2x2, nm2), x0, x1);
      const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
      acc[i & 1] = add_f2(acc[i & 1], pack_f2(p0, p1));
      if constexpr (BF) w[i] = pack2<__nv_bfloat162>(p0, p1);
      else w[i] = pack2<__half2>(p0, p1);
    }
    tmem_st8(tP + 8 * g, w);
  }
  float a0, a1;
  unpack_f2(add_f2(acc[0], acc[1]), a0, a1);
  return a0 + a1;
}

}  // namespace rra
