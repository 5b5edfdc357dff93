// Decayed linear attention: parameters and helpers shared by its kernels.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr int kLinChunk = 128;  // tokens per chunk of the chunked form
constexpr int kLinSlices = 4;   // parts of 32 columns of a head's state (d = 128)
// Sequences of up to this many tokens take the recurrent form.  (Times, here as
// in the other files of these operators: whole calls among others, their inputs
// out of cache.)  64 sequences of 32 heads: 91 us of 16 tokens (chunked form
// 118), 101 of 18 (118), 111 of 20 (119), 121 of 22 (120).  Where all its CTAs
// run at once the recurrent form is ahead for longer: four sequences of 40 heads
// 19.3 us of 28 tokens (19.3), 21.3 of 32 (19.8), one of 64 heads 12.4 of 32
// (15.1), 17.2 of 48 (15.3); and longer still with an SM for each: one sequence
// of 16 heads 11.7 us of 64 tokens (15.2), 16.4 of 96 (15.4).  (The lengths were
// chosen when the chunked form was a little cheaper: they lie somewhat below
// where the forms meet now.)
constexpr int kLinShort = 18, kLinShortFew = 32, kLinShortLone = 64;

// Header words of a layer's work area in these forwards (besides kErr, kNDec
// and kNPre): the segments of the long sequences, longest first.
enum LinCnt : int {
  kLinStateItems = 4,  // segments of the split sequences (the first ones)
  kLinHead = 5,        // work counter of the output pass
  kLinItems = 6,       // all segments
  kLinStateHead = 7,   // work counter of the state pass
  kLinSplit = 8,       // sequences of more than one segment
  kLinSegChunks = 9,   // chunks per segment of those
  kLinBad = 10,        // something has been left to the token-serial kernel
};

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
  int d, chunk;        // head size; tokens per chunk that the scheduler counts in
  int num_blocks, hint;
  int listed;   // the scheduler has run: take the sequences from its list
  int late;     // (recurrent kernel) launched behind the chunk kernel
  WorkArea work;
  // states of the split sequences' segments [slots][d][d] (nullptr: never
  // split), and the chunked form's marks for what is left to the token-serial
  // kernel [index in the list of long sequences][H][kLinSlices]
  float* seg_states;
  int seg_slots;
  unsigned char* bad;
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
// x, or the largest number of its sign where it is infinite: what the pair's
// second number multiplies, since a zero or negative one times an infinity
// would make NaN of a state that the recurrence leaves infinite.
__device__ __forceinline__ float bounded(float x) {
  float r;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(3.402823466e38f));
  return r;
}
// Pairs of fp32 in one 64-bit register: packed arithmetic (one instruction per
// pair).
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unf2(F2 v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ F2 bounded(F2 v) {
  float x, y;
  unf2(v, x, y);
  return f2(bounded(x), bounded(y));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A head's log decay, with -inf (no memory at all) as a finite number, so
// that zero steps of it are no decay.
__device__ __forceinline__ float finite_decay(float g) { return g == -INFINITY ? -1e30f : g; }

// Validates the batch and lists the sequences: dec[] those of at most
// short_max tokens, pre[] the longer ones, longest first, with their segments
// (pre_cp[]: segments before entry k).
cudaError_t launch_lin_schedule(const LinParams& p, int short_max, int num_sms, cudaStream_t s);
// The token-serial kernel over the scheduler's dec[] list (p.listed) or over
// all N sequences, which it then validates itself; behind the chunked form
// (p.late) also over what that has marked.
cudaError_t launch_lin_recurrent(const LinParams& p, int d, int act, int max_items, cudaStream_t s);
// The states at the segments' starts from the segments' own.
cudaError_t launch_lin_segments(const LinParams& p, int num_sms, cudaStream_t s);
// The whole forward in the token-serial form with long sequences cut into
// segments: scheduler, state pass, segment states, output pass.
cudaError_t launch_lin_serial_split(const LinParams& p, int act, int num_sms, cudaStream_t s);
// The chunked form over pre[] (d = 128, bf16); may_split: with the state pass
// that split sequences need.
bool lin_chunk_supported(int d, int act);
cudaError_t launch_lin_chunk(const LinParams& p, bool may_split, int num_sms, cudaStream_t s);

}  // namespace gdn
