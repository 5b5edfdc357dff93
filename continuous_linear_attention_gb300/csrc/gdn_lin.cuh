// Decayed linear attention: parameters and helpers shared by its kernels.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

// What the kernels of one gdn_lin_varlen_forward get, by value.
struct LinParams {
  const void *q, *k, *v;  // rows of H, Hkv and Hkv heads of d elements
  void* out;
  long long ldq, ldk, ldv, ldo;  // row pitches, elements
  const int32_t* cu;
  const int32_t* blk;
  const uint8_t* has_past;
  const float* log_decay;  // [H]
  float scale;
  unsigned char* layer_base;
  size_t stride;
  int T, N, H, group;  // group = H / Hkv
  int num_blocks, hint;
  int listed;   // the scheduler has run: take the sequences from its list
  int late;     // (recurrent kernel) launched behind the chunk kernel
  WorkArea work;
};

// e^x as a pair whose sum is it to about 2^-24 |x| relative, so that a state
// multiplied by the pair at every step keeps its decay over many steps: near
// x = 0 the rounding of e^x itself (2^-25) would add up over 1 / |x| steps to
// far more than the state's own rounding.
struct DecayPair {
  float hi, lo;
};
__device__ __forceinline__ DecayPair decay_pair(float x) {
  DecayPair d;
  if (x > -0.5f && x < 0.5f) {
    const float m = expm1f(x);
    d.hi = 1.f + m;
    d.lo = (1.f - d.hi) + m;
  } else {
    d.hi = expf(x);
    d.lo = 0.f;
  }
  return d;
}
// A head's log decay, with -inf (no memory at all) as a finite number, so
// that zero steps of it are no decay.
__device__ __forceinline__ float finite_decay(float g) { return g == -INFINITY ? -1e30f : g; }

// Validates the batch and lists the sequences: dec[] those of at most
// short_max tokens, pre[] the longer ones.
cudaError_t launch_lin_schedule(const LinParams& p, int short_max, cudaStream_t s);
// The token-serial kernel over the scheduler's dec[] list (p.listed) or over
// all N sequences, which it then validates itself.
cudaError_t launch_lin_recurrent(const LinParams& p, int d, int act, int max_items, cudaStream_t s);

}  // namespace gdn
