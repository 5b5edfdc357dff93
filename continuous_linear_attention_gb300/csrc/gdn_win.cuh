// Windowed attention: parameters and helpers shared by its kernels.
#pragma once

#include "gdn_seqs.cuh"

namespace gdn {

// What the kernels of one gdn_win_varlen_forward get, by value.
struct WinParams {
  Batch batch;
  const void *q, *k, *v;  // rows of H, Hkv and Hkv heads of d elements
  void* out;
  long long ldq, ldk, ldv, ldo;  // row pitches, elements
  float scale;
  unsigned char* layer_base;
  size_t stride;
  int H, Hkv, group, d;  // group = H / Hkv
  int window, sinks;
  int report;  // this kernel raises the batch's flags
};

// Where a block keeps position j: the first `sinks` ones at their own index,
// the others in a ring behind them.
__device__ __forceinline__ int slot_of(const WinParams& p, int j) {
  return j < p.sinks ? j : p.sinks + (j - p.sinks) % p.window;
}
// A block's keys (part 0) or values (part 1) of kv head h: [sinks + window][d].
template <typename T>
__device__ __forceinline__ T* ring_of(const WinParams& p, int blk, int part, int h) {
  return reinterpret_cast<T*>(p.layer_base + (size_t)blk * p.stride) +
         (size_t)(part * p.Hkv + h) * (p.sinks + p.window) * p.d;
}
// Whether position pos sees position j.
__device__ __forceinline__ bool sees(const WinParams& p, int pos, int j) {
  return j <= pos && (j > pos - p.window || j < p.sinks);
}

// Work memory of a pool for the forms below: arrival counters of split windows,
// the units that the tensor-core form leaves (the header's kWorkHead counts
// them, its kItemHeadC the units claimed), partial results of split windows.
constexpr size_t kWinCounterBytes = 4096;
constexpr int kWinLeft = 16384;
constexpr size_t kWinListBytes = kWinLeft * sizeof(int32_t);

// The form for any type and shape, over the sequences of the given pieces; with
// left, over the units that the tensor-core form has left, in its pieces.
cudaError_t launch_win_rows(const WinParams& p, int act, const Pieces& of, int max_pieces, int sms,
                            const void* room, bool left, cudaStream_t s);
// The new keys and values of those sequences into their blocks, behind it.
cudaError_t launch_win_append(const WinParams& p, int act, const Pieces& of, int max_pieces, int sms,
                              cudaStream_t s);
// The form for few tokens (gdn_win_short.cu), which appends by itself: up to
// win_short_tokens(group) tokens per sequence (0: none); room: work memory of
// the pool, win_short_room bytes, zeroed once.
bool win_short_supported(int d, int act);
int win_short_tokens(int group);
size_t win_short_room(int sms, int d);
// late: right behind launch_win_tc, beside its last units.
cudaError_t launch_win_short(const WinParams& p, const Pieces& of, int max_items, int sms, bool late,
                             void* room, cudaStream_t s);

// The form for prompts (gdn_win_tc.cu): pieces of win_tc_tokens(group) tokens.
bool win_tc_supported(int d, int act, int group);
int win_tc_tokens(int group);
cudaError_t launch_win_tc(const WinParams& p, const Pieces& of, int max_pieces, int sms, void* room,
                          cudaStream_t s);

}  // namespace gdn
