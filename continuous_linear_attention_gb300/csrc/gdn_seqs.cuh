// The sequences of a packed batch as the selective scan's and the windowed
// attention's kernels take them: checked as the pool's contract demands, and
// listed with a prefix of their pieces of work.  A call of up to
// kSelfPlan sequences is listed by every CTA for itself, in shared memory (one
// launch less); a larger one by plan_kernel, into the layer's work area.  Single
// tokens, 256 of them the first way and 257 the second: windowed attention (window
// 64, 2 kv heads) 16.0 and 17.1 us, the convolution (1,024 channels) 7.5 and 9.3, the
// scan (1,024 x 16) 12.3 and 14.0.
#pragma once

#include "gdn_internal.cuh"
#include "gdn_ptx.cuh"

namespace gdn {

constexpr int kSelfPlan = 256;

struct Batch {
  const int32_t* cu;
  const int32_t* blk;
  const uint8_t* has_past;  // or
  const int32_t* past_len;  // tokens before the call (windowed attention)
  int N, T, num_blocks, hint;
  int listed;  // plan_kernel has run
  WorkArea work;
};

// Which sequences a kernel takes, in pieces of how many tokens.
struct Pieces {
  int least, most;  // lengths
  int tokens;       // of a piece
  __host__ __device__ int of(int len) const {
    return len < least || len > most ? 0 : (len - 1) / tokens + 1;
  }
};

struct SeqList {
  const int32_t* items;  // sequences with pieces
  const int32_t* first;  // first[i]: pieces before items[i]; first[n]: all
  int n, total;
};

constexpr int kPlanSlots = 2 * kSelfPlan;  // of the hash table that finds blocks named twice

struct PlanSmem {
  int32_t lo[kSelfPlan + 1], blk[kSelfPlan], past[kSelfPlan], len[kSelfPlan], upto[kSelfPlan], items[kSelfPlan], first[kSelfPlan + 1];
  int32_t named[kPlanSlots];  // a block index, kPlanTwice with it where two sequences name it
  int32_t runs[kSelfPlan / 32], run_pieces[kSelfPlan / 32];
  unsigned flags;
  int longest, tokens;  // (longest, tokens: of the sequences with pieces)
};
constexpr int kPlanTwice = 0x40000000;  // (block indices are below 2^30)

// What is wrong with a sequence of len tokens by itself, as GDN_FLAG_* (0:
// nothing; a padding entry or an empty sequence has nothing wrong either).
__device__ __forceinline__ unsigned sequence_flags(const Batch& b, int past, int len, int blk) {
  if (blk < 0 || len == 0) return 0u;
  if (blk >= b.num_blocks) return GDN_FLAG_BLOCK_RANGE;
  if (blk == 0) return GDN_FLAG_TRASH_WRITE;
  if (b.hint > 0 && len > b.hint) return GDN_FLAG_HINT;
  if (b.past_len && (past < 0 || past > 0x7fffffff - len)) return GDN_FLAG_RANGE;
  return 0u;
}

// Every thread of the CTA (whole warps): the list of a call of up to kSelfPlan
// sequences, in order of their indices, or, kSort and no more than 32 of them,
// longest first (of equals the lower index first).  raise: this CTA reports what
// is wrong.  A block named by two sequences with tokens leaves both out.  size:
// called with the longest one and the sum of their lengths, says how many tokens a
// piece has.  Nothing here is unrolled: a kernel's first instructions are fetched
// as they are met, and that is most of the time this takes (2.5 us unrolled).
template <bool kSort, typename Size>
__device__ inline SeqList plan_self(const Batch& b, Pieces pieces, PlanSmem& sm, bool raise, Size size) {
  const int tid = threadIdx.x, threads = blockDim.x, N = b.N, lane = tid & 31, warps = threads >> 5;
  if (tid == 0) {
    sm.flags = 0u;
    sm.longest = sm.tokens = 0;
    sm.lo[N] = b.cu[N];
  }
#pragma unroll 1
  for (int i = tid; i < N; i += threads) {
    sm.lo[i] = b.cu[i];
    sm.blk[i] = b.blk[i];
    sm.past[i] = b.past_len ? b.past_len[i] : 0;
  }
#pragma unroll 1
  for (int i = tid; i < kPlanSlots; i += threads) sm.named[i] = -1;
  __syncthreads();
  auto slot_of = [](int blk) { return (int)((unsigned)blk * 2654435761u >> 23); };
  static_assert(kPlanSlots == 512, "nine bits of the hash");
  int bad = tid == 0 && (sm.lo[0] != 0 || sm.lo[N] != b.T);
#pragma unroll 1
  for (int i = tid; i < N; i += threads) {
    const int lo = sm.lo[i], hi = sm.lo[i + 1], blk = sm.blk[i];
    bad |= hi < lo;
    if (hi <= lo || blk <= 0 || blk >= b.num_blocks) continue;
#pragma unroll 1
    for (int at = slot_of(blk);; at = (at + 1) % kPlanSlots) {  // (half of the slots stay empty)
      const int was = atomicCAS(&sm.named[at], -1, blk);
      if (was == -1) break;
      if ((was & ~kPlanTwice) == blk) {
        atomicOr(&sm.named[at], kPlanTwice);
        break;
      }
    }
  }
  SeqList list = {sm.items, sm.first, 0, 0};
  if (__syncthreads_or(bad)) {
    if (raise && tid == 0) atomicOr((unsigned*)&b.work.header()[kErr], GDN_FLAG_SEQLENS);
    return list;
  }
#pragma unroll 1
  for (int i = tid; i < N; i += threads) {
    int len = sm.lo[i + 1] - sm.lo[i];
    const int blk = sm.blk[i];
    unsigned flags = sequence_flags(b, sm.past[i], len, blk);
    if (len > 0 && blk > 0 && blk < b.num_blocks) {
      int at = slot_of(blk);
#pragma unroll 1
      while ((sm.named[at] & ~kPlanTwice) != blk) at = (at + 1) % kPlanSlots;
      if (sm.named[at] & kPlanTwice) flags = GDN_FLAG_DUPLICATE;
    }
    if (flags && raise) atomicOr(&sm.flags, flags);
    if (flags || blk < 0 || len < pieces.least || len > pieces.most) len = 0;  // nothing to do here
    sm.len[i] = len;
    if (kSort && len > 0) {
      atomicMax(&sm.longest, len);
      atomicAdd(&sm.tokens, len);
    }
  }
  __syncthreads();
  if (raise && tid == 0 && sm.flags) atomicOr((unsigned*)&b.work.header()[kErr], sm.flags);
  pieces.tokens = size(sm.longest, sm.tokens);
  // the entries and pieces of each run of 32 sequences, with those of each before it
#pragma unroll 1
  for (int run = tid >> 5; run * 32 < N; run += warps) {
    const int i = run * 32 + lane, len = i < N ? sm.len[i] : 0;
    const int count = len > 0 ? (len - 1) / pieces.tokens + 1 : 0;
    int upto = count;
#pragma unroll 1
    for (int w = 1; w < 32; w <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, w);
      if (lane >= w) upto += x;
    }
    const unsigned mask = __ballot_sync(0xffffffffu, len > 0);
    if (i < N) sm.upto[i] = upto - count;
    if (lane == 31) {
      sm.runs[run] = __popc(mask);
      sm.run_pieces[run] = upto;
    }
  }
  __syncthreads();
  int all = 0, all_pieces = 0;
#pragma unroll 1
  for (int run = 0; run * 32 < N; ++run) {
    if (run % warps == tid >> 5) {
      const int i = run * 32 + lane;
      const bool mine = i < N && sm.len[i] > 0;
      const unsigned mask = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const int at = all + __popc(mask & ((1u << lane) - 1u));
        sm.items[at] = i;
        sm.first[at] = all_pieces + sm.upto[i];
      }
    }
    all += sm.runs[run];
    all_pieces += sm.run_pieces[run];
  }
  if (tid == 0) sm.first[all] = all_pieces;
  __syncthreads();
  if (kSort && all <= 32 && all > 1) {
    if (tid < 32) {
      const int mine = tid < all ? sm.items[tid] : -1, len = tid < all ? sm.len[mine] : 0;
      const int count = tid < all ? sm.first[tid + 1] - sm.first[tid] : 0;
      int rank = 0, ahead = 0;
#pragma unroll 1
      for (int j = 0; j < all; ++j) {
        const int lj = __shfl_sync(0xffffffffu, len, j), cj = __shfl_sync(0xffffffffu, count, j);
        if (lj > len || (lj == len && j < tid)) {
          ++rank;
          ahead += cj;
        }
      }
      __syncwarp();
      if (tid < all) {
        sm.items[rank] = mine;
        sm.first[rank] = ahead;
      }
    }
    __syncthreads();
  }
  list.n = all;
  list.total = all_pieces;
  return list;
}
__device__ inline SeqList plan_self(const Batch& b, const Pieces& pieces, PlanSmem& sm, bool raise) {
  return plan_self<false>(b, pieces, sm, raise, [&](int, int) { return pieces.tokens; });
}

// plan_kernel's list of the sequences with pieces (the others are in dec(),
// hdr[kNDec] of them).
__device__ inline SeqList listed_long(const Batch& b) {
  const int32_t* hdr = b.work.header();
  return {b.work.pre(), b.work.pre_cp(), hdr[kNPre], hdr[kPreChunks]};
}

// The list entry that piece u belongs to.
__device__ __forceinline__ int entry_of(const SeqList& list, int u) {
  if (list.total == list.n) return u;  // a piece each
  int lo = 0, hi = list.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.first[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A call's sequences of pieces.least to pieces.most tokens into pre() and
// pre_cp(), the others that have tokens into dec(), in order of their indices.
cudaError_t launch_plan(const Batch& b, const Pieces& pieces, cudaStream_t s);

}  // namespace gdn
