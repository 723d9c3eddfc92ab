// delta.cuh -- arguments and small helpers of the gated delta rule's kernels.
#pragma once

#include "mixer.cuh"

namespace redlite {

struct DeltaArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const float *g, *beta;  // [rows, n_v]
  const int32_t *cu, *slots;
  int n_seqs, n_tokens, n_k, n_v, dk, dv;
  float scale, qk_eps;
  const float *state_in;
  float *state_out;
  int64_t n_slots;
  void *out;
  uint8_t *ws;
  int32_t *status;
};

// The slot of sequence `seq`, or -1: out of range, or named by an earlier
// sequence of the call (whose state it is then).  Every thread of the block
// calls it; sequences in front of this one are looked through together.
__device__ __forceinline__ int64_t delta_slot(const DeltaArgs &a, int seq) {
  if (!a.slots) return seq;  // n_slots >= n_seqs is checked on the host
  const int64_t slot = __ldg(a.slots + seq);
  int twice = 0;
  for (int s = threadIdx.x; s < seq; s += blockDim.x) twice |= __ldg(a.slots + s) == slot;
  twice = __syncthreads_or(twice);
  if (slot >= 0 && slot < a.n_slots && !twice) return slot;
  if (threadIdx.x == 0) set_status(a.status, REDLITE_STATUS_BAD_SLOT);
  return -1;
}

// Log decays below -1e6 are taken as -1e6 (both decays are 0 in fp32), so
// that differences of their sums stay exact enough: 64 of them in fp64 leave
// 2^-27.  NaN passes.
__device__ __forceinline__ float delta_clamp_g(float g) { return g < -1e6f ? -1e6f : (g > 1e6f ? 1e6f : g); }

int delta_check(int32_t dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                int64_t v_stride, const float *g, const float *beta, int32_t n_seqs, int64_t rows, int32_t n_k,
                int32_t n_v, int32_t dk, int32_t dv, float scale, const float *state_in, const float *state_out,
                const int32_t *slots, int64_t n_slots, const void *out, int64_t out_stride);

}  // namespace redlite
