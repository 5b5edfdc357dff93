// The list of a large batch's sequences (gdn_seqs.cuh): one CTA, four barriers
// per 1,024 sequences.
#include "gdn_cta.cuh"
#include "gdn_seqs.cuh"

namespace gdn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kSmemCounts = 8192;  // pools whose block-use counts fit into shared memory

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Batch b, Pieces pieces) {
  __shared__ int32_t s_counts[kSmemCounts];
  __shared__ int warp_sums[32];
  __shared__ unsigned s_flags;
  const int tid = threadIdx.x, N = b.N, nb = b.num_blocks;
  pdl_wait_then_release();
  int32_t* hdr = b.work.header();
  int32_t* uses = nb <= kSmemCounts ? s_counts : b.work.blk_count();
  if (tid == 0) s_flags = 0u;
  for (int i = tid; i < nb; i += kPlanThreads) uses[i] = 0;
  int bad = tid == 0 && (b.cu[0] != 0 || b.cu[N] != b.T);
  for (int i = tid; i < N; i += kPlanThreads) bad |= b.cu[i + 1] < b.cu[i];
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr((unsigned*)&hdr[kErr], GDN_FLAG_SEQLENS);
      hdr[kNDec] = hdr[kNPre] = hdr[kPreChunks] = 0;
    }
    return;
  }
  for (int i = tid; i < N; i += kPlanThreads) {
    const int blk = b.blk[i];
    if (blk > 0 && blk < nb && b.cu[i + 1] > b.cu[i]) atomicAdd(&uses[blk], 1);
  }
  __syncthreads();
  int n_long = 0, n_rest = 0, before = 0;  // so far
  for (int i0 = 0; i0 < N; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int len = 0, mine = 0;
    if (i < N) {
      len = b.cu[i + 1] - b.cu[i];
      const int blk = b.blk[i];
      unsigned flags = sequence_flags(b, b.past_len ? b.past_len[i] : 0, len, blk);
      if (len > 0 && blk > 0 && blk < nb && atomicAdd(&uses[blk], 0) > 1) flags = GDN_FLAG_DUPLICATE;
      if (flags) atomicOr(&s_flags, flags);
      if (flags || blk < 0) len = 0;
      mine = len > 0 ? pieces.of(len) : 0;
    }
    const bool rest = mine == 0 && len > 0;
    int total;
    const int at = n_long + cta_scan(mine > 0, &total, warp_sums);
    n_long += total;
    const int other = n_rest + cta_scan(rest, &total, warp_sums);
    n_rest += total;
    const int first = before + cta_scan(mine, &total, warp_sums);
    before += total;
    if (mine > 0) {
      b.work.pre()[at] = i;
      b.work.pre_cp()[at] = first;
    } else if (rest) {
      b.work.dec()[other] = i;
    }
  }
  __syncthreads();
  if (tid == 0) {
    b.work.pre_cp()[n_long] = before;
    hdr[kNPre] = n_long;
    hdr[kNDec] = n_rest;
    hdr[kPreChunks] = before;
    if (s_flags) atomicOr((unsigned*)&hdr[kErr], s_flags);
  }
}

}  // namespace

cudaError_t launch_plan(const Batch& b, const Pieces& pieces, cudaStream_t s) {
  return launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, b, pieces);
}

}  // namespace gdn
