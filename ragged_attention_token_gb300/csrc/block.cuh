// What the block operators' kernels and their launches share.  A header of its own: bench.py ties the image attention's
// recorded DRAM bytes to a hash of that kernel's source and headers, which this one does not belong to.
#pragma once

#include "tc_ptx.cuh"

namespace rra {

// For kernels launched as programmatic dependents: lets the next kernel of the
// stream start its set-up as soon as every CTA of this one is running, then waits for the
// kernels before it, which precedes every access to global memory.  Every CTA
// calls it, so that no kernel completes before those it depends on.
// The kernels run while those before them may still write what they read behind the wait, so they read it by ordinary loads:
// __ldg is for memory that nothing writes as long as the kernel lives, and the compiler may move it ahead of the wait.
__device__ __forceinline__ void dependent_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The same for the kernels of the norm of rows and of the paged cache.
__device__ __forceinline__ void start_dependent() { dependent_launch(); }

// A bounded wait: by the default bound, or, in the kernels for launches made with a limit set (rra_set_wait_limit), by
// that one, polling, so that a bound below the hardware's suspension of a wait holds too.
template <bool LIMIT, long long DEFAULT = WAIT_LIMIT_CYCLES>
__device__ __forceinline__ bool mbar_wait_limited(uint32_t bar, uint32_t parity, uint32_t abort_flag, long long limit) {
  if constexpr (!LIMIT) return mbar_wait_or_abort(bar, parity, abort_flag, DEFAULT);
  const long long t0 = clock64();
  while (!mbar_test_wait(bar, parity)) {
    if (ld_shared_volatile_u32(abort_flag) != 0u || clock64() - t0 > limit) return false;
  }
  return true;
}

// Linear layer with its epilogue: c = act(a W^T + bias) + residual for the T = cu[B] rows; in 8 bits the products are
// scaled first: a_scale[t] w_scale[n] (a W^T).
struct LinearEpiArgs {
  const int32_t* cu;
  int B, cap, K, N;
  const void* a;
  const void* w;
  const float* a_scale;    // [cap], 8-bit operands only
  const float* w_scale;    // [N]
  const float* bias;       // [N] or null
  const void* residual;    // [cap, N] of the output type, or null; may be c
  void* c;
  int32_t* err;
  long long wait_limit;    // clock cycles one on-chip wait may take before giving up (0: the default)
};
cudaError_t launch_linear_epilogue(const LinearEpiArgs& a, rra_dtype in, rra_dtype out, rra_activation act,
                                   int num_sms, cudaStream_t stream);
cudaError_t launch_linear_scaled(const LinearEpiArgs& a, rra_dtype out, rra_activation act, int num_sms,
                                 cudaStream_t stream);

// Norm of rows: r = x (+ residual), sum = r, y = r rsqrt(mean r^2 + eps) (weight), in 16 bits or in 8 with a scale a row.
struct NormRowsArgs {
  const void* x;
  const void* residual;    // [cap, N] or null
  void* sum;               // [cap, N] of the residual's type; may be it
  const float* weight;     // [N] or null
  float eps;
  const int32_t* cu;
  int B, cap, N;
  void* y;
  float* scale;            // [cap], 8-bit outputs only
  int32_t* err;
};
cudaError_t launch_rms_norm(const NormRowsArgs& a, rra_dtype dt, rra_dtype residual, bool eight_bits, int num_sms,
                            cudaStream_t stream);

// Norm + rotation of query and key heads (+ copy of values); strides in elements.
struct NormRopeArgs {
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;             // v_out null: no values
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride, v_out_stride;
  const int32_t* positions;
  const int32_t* cu;
  const int32_t* kv_rows;                  // null: row t
  long long kv_out_rows;
  int B, cap, Hq, Hkv;
  const float *q_weight, *k_weight, *inv_freq;
  float eps, rope_scale;
  int rot;
  int32_t* err;
};
cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int d, rra_dtype dt, bool interleaved, int num_sms,
                                cudaStream_t stream);

// Attention over packed prompts / of new tokens over a padded cache.
struct PromptArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between rows
  const int32_t* cu;
  int B, cap, max_seqlen, Hq, Hkv;
  float scale_log2;
  int causal;
  void* o;
  int32_t* err;
  long long wait_limit;                    // as above
  long long unit_wait_limit;               // the same for one that lasts a whole unit (set by the launch)
};
cudaError_t launch_attend_prompt(const PromptArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream);

struct CacheArgs {
  const void *q, *k, *v;
  long long q_stride;
  const int32_t* kv_len;
  int B, nq, cap, Hq, Hkv;
  float scale_log2;
  void* o;
  int32_t* err;
};
cudaError_t launch_attend_cache(const CacheArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream);

// Attention of the new tokens of each sequence over a paged cache.
struct PagedArgs {
  const void *q, *k, *v;
  long long q_stride, page_stride;         // elements between rows of q, between pages of k and of v
  const int32_t* table;                    // [B, table_width]
  const int32_t* kv_len;
  const int32_t* cu;
  int B, cap, max_new, max_kv, num_pages, page, table_width, Hq, Hkv;   // max_new: no more than cap
  int bound_new;                           // max_new as the caller gave it
  float scale_log2;
  void* o;
  int32_t* err;
  long long wait_limit;
  void* space;                             // workspace of attend_paged_space() bytes (0: not used)
  long long unit_wait_limit;               // set by the launch
};
size_t attend_paged_space(int B, int max_new, int max_kv, int Hkv, int G, int d);
cudaError_t launch_attend_paged(const PagedArgs& a, int d, rra_dtype dt, int num_sms, cudaStream_t stream, int* launches);

}  // namespace rra
