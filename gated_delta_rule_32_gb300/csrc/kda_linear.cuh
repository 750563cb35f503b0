// kda_linear.cuh -- what the kernels of linear attention with a decay for
// each head share: the arguments and a sequence's rows.
#pragma once

#include "kda_common.cuh"

namespace kda_linear {

// Rows (tokens) are `*_stride` elements apart, heads and channels of a row
// contiguous; out is contiguous.  Head h of v, out and the states reads head
// h / (H / HK) of q and k.
struct LinearArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float* decay;    // log-decays: [rows, decay_stride], or [H] with a stride of 0
  int64_t decay_stride;
  const float* init;     // [N, H, dk, dv], may be null
  void* out;             // [rows, H, dv]
  float* final_state;    // [N, H, dk, dv], may be null or init
  const int32_t* cu;     // device, may be null (dense: sequence n has rows n T .. n T + T - 1)
  int32_t* status;       // device, may be null
  int N, T, H, HK, dk, dv;
  float scale;
};

__device__ __forceinline__ void report(int32_t* status, kda_status s) {
  if (status) atomicExch(status, (int32_t)s);
}

// First row and length of sequence n; false (and a report) where the packed
// offsets are not 0 .. T non-decreasing, so that no access leaves the rows.
__device__ __forceinline__ bool span(const LinearArgs& p, int n, int64_t& row, int& len) {
  if (!p.cu) {
    row = (int64_t)n * p.T;
    len = p.T;
    return true;
  }
  const int a = p.cu[n], b = p.cu[n + 1];
  if (a < 0 || b < a || b > p.T || (n == 0 && a != 0)) {
    report(p.status, KDA_ERR_BAD_SEQLENS);
    return false;
  }
  row = a;
  len = b - a;
  return true;
}

// A log-decay as the operator takes it: at most 0 (a NaN stays one).
__device__ __forceinline__ float clamp_decay(float a) { return a > 0.0f ? 0.0f : a; }

// Whether a token forgets what is before it: e^-104 is below half of the least fp32 number, so
// the factor is 0.  The state is then dropped, not multiplied: it may hold anything.  (Factors
// that only come to 0 together, over many tokens, are products: a NaN stays.)
__device__ __forceinline__ bool forgets(float a) { return a < -104.0f; }

}  // namespace kda_linear

kda_status kda_launch_linear_rec(const kda_linear::LinearArgs& p, kda_dtype dtype,
                                 cudaStream_t stream);

// The tensor-core kernels (kda_linear_tile.cu): what they serve, the scratch
// that they need for these sizes, and the launch (with rows to work on).
bool kda_linear_tile_ok(int dk, int dv, kda_dtype dtype);
size_t kda_linear_tile_workspace(int N, int T, int H, int dk, int dv, bool packed);
kda_status kda_launch_linear_tile(const kda_linear::LinearArgs& p, void* workspace,
                                  cudaStream_t stream);
