// The pool handle of the C ABI (host side), shared by the translation units
// that implement its entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

struct gdn_pool {
  int num_blocks, num_layers, Hk, Hv, dk, dv, K, act;
  size_t stride, conv_off, rec_off, total;
  unsigned char* base;
  bool owns;
  int device, sms;  // and its streaming multiprocessors
  int32_t* work;  // num_layers * WorkArea::words(num_blocks) words
  cudaEvent_t ev_before, ev_after;  // optional timing events (caller-owned)
  // prefill scratch: chunk-major tiles of the split prefill path (gated delta
  // net pools, capacity in 64-token chunks) or the fp16 conv output of the
  // chunked scan (Mamba2 pools, capacity in tokens); allocated stream-ordered
  unsigned char* scr;
  size_t scr_bytes;
  bool scr_grow;  // false: never allocated; the fused chunked kernel is used
  int last_path;  // GDN_PREFILL_* of the last forward
  // 0: gated delta net pool (conv + recurrent state); 1: Mamba2 pool (conv +
  // SSM state [H][P][N] at rec_off), with its dimensions; 2: decayed linear
  // attention pool (state [Hv][dk][dv] at 0, no conv state)
  int kind;
  int ssd_H, ssd_P, ssd_N, ssd_G;
  int32_t* blk_work;  // work area of the block operations (gdn::BlockWork)
  // decayed linear attention pools: states between the segments of a split
  // prompt, fp32 [lin_slots][dk][dv] (gdn_lin_chunk.cu), or NULL
  float* lin_states;
  int lin_slots;
};

namespace gdn {
// Fills in the pool's device, memory and work area for its dimensions, stride
// and total, and zeroes them (synchronously).  On an error nothing stays
// allocated.
int pool_allocate(gdn_pool* p, void* device_mem);
}  // namespace gdn
