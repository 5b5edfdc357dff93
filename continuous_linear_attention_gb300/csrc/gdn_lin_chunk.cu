// Chunked form of decayed linear attention for prompts (d = 128, bf16): the
// recurrence S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over chunks
// of 128 tokens.  With S0 the state at a chunk's start, n its valid tokens and
// i, j = 0 .. n-1 in the chunk,
//   P[i][j] = scale e^{g (i-j)} (q_i . k_j)  for j <= i, else 0
//   o_i     = scale e^{g (i+1)} S0^T q_i + sum_j P[i][j] v_j
//   S_n     = e^{g n} S0 + sum_j e^{g (n-1-j)} k_j v_j^T
// so a (sequence, head) chain is four 128^3 products per chunk, and all but
// the first term of each line does not depend on the chunks before.
//
// Bytes bound it: q, k, v and o are 128 KB per chunk and head (2.9 us of one
// SM's share of HBM); the products, the state's in three terms, are six 128^3
// (1.9 us of one SM's tensor rate at the measured peak).
//
// One CTA per SM, chains claimed from a counter, longest first.  Roles, each
// a loop over the CTA's chunks that meets the others at mbarriers only:
//   producer  one thread: TMA loads of a chunk's q, k, v tiles, two stages
//   MMA 1     one thread: P = Q K^T, O = Q S0, O += P V
//   MMA 2     one thread: U = sum of the decayed v k^T, in halves of 64 tokens
//   store     one thread: the staged output tile to global memory by TMA
//   O warps   P with its decay -> bf16 A operand; O <- e^{g(i+1)} O; output
//   V warps   e^{g(n-1-j)} v_j -> A operand of U, rows past the chunk's end
//             zeroed, and the check for values that are not finite
//   S warps   the state, fp32 in registers (thread v holds S[.][v]): to bf16
//             as operand of O, S <- e^{g n} S + U
//
// Precision.  P and S0 enter as bf16 operands (their partners are bf16, and
// one MMA takes one type): each is off by 2^-9 rms like the output's own
// rounding, which they follow.  The state is an output in fp32 and carried
// over the whole prompt, so its update is not rounded: a decayed v has 8 + 24
// significant bits and goes in as three bf16 terms (hi, mid, lo: 24 bits), the
// smallest first, and U is added to S in fp32 registers with a decay pair
// (see decay_pair).  Accumulating into S itself in tensor memory would add a
// rounding of S at each of 24 MMA steps per chunk.
//
// A non-finite k or v in a chunk would reach rows of earlier tokens through
// 0 * inf in the masked products; such a chain is left to the token-serial
// kernel (its block keeps the old state, see the redo below).
//
// Few long chains: when the longest chain is far above an SM's share, the
// scheduler cuts long sequences into segments.  A first launch of this kernel
// (kState) computes every segment's own state from k and v alone, a small
// kernel turns those into the states at the segments' starts, and the output
// pass then runs all segments at once; k and v are read twice.
#include <cuda.h>

#include "gdn_lin.cuh"
#include "gdn_ptx.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int D = 128;
constexpr int CH = kLinChunk;  // 128
constexpr int kThreads = 512;  // O, V and S warps (4 each), then four single-thread warps
constexpr int kStages = 2;
constexpr uint32_t TILE = 32768, BOX = 16384;  // a [128][128] bf16 tile: two 64-column boxes
constexpr uint32_t ST_Q = 0, ST_K = TILE, ST_V = 2 * TILE, ST_BYTES = 3 * TILE;
constexpr uint32_t OFF_S = kStages * ST_BYTES;  // S0 as B operand: [v][k], two 64-k blocks
// tensor memory columns: P fp32 (bf16 over its first half), O, U, then the
// three terms of 64 decayed v rows (32 columns each)
constexpr uint32_t TM_P = 0, TM_O = 128, TM_U = 256, TM_V = 384, TM_COLS = 512;

enum Flag : int {
  kFirst = 1,   // first chunk of its chain (or segment)
  kLast = 2,    // last one
  kEnd = 4,     // no more chunks
  kNoU = 8,     // the state after this chunk is not needed
  kFinal = 16,  // the chain's end: its state goes to the pool block
};
struct Desc {
  int row, n, h, flags;
  int entry;            // index in the scheduler's list of long sequences
  int slot;             // segment state slot, or -1
  long long rblk, wblk;  // blocks read (0: zeros) and written
};

struct Ctl {
  Desc desc[kStages];
  uint64_t full[kStages], empty[kStages], zeroed[kStages], staged[kStages];
  uint64_t p_full, pb_full, qs_full, o_scaled, o_full, o_free, s_ready;
  uint64_t v_full, v_free, u_full, u_free;
  uint32_t bad[kStages][4];
  uint32_t tmem;
};
constexpr uint32_t OFF_CTL = OFF_S + TILE;
constexpr uint32_t SMEM_BYTES = OFF_CTL + sizeof(Ctl);
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");

// A warp's bounded wait: false for all lanes if any gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One arrival for a warp whose lanes' earlier accesses it orders.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, int c0, int r0, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(r0), "r"(smem_u32(src))
               : "memory");
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  return tc::pack2(lo, hi, (__nv_bfloat16*)nullptr);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool kState>
__global__ void __launch_bounds__(kThreads, 1)
lin_chunk_kernel(LinParams p, const __grid_constant__ CUtensorMap tq,
                 const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ CUtensorMap to) {
  extern __shared__ __align__(1024) unsigned char sm[];
  Ctl& ctl = *reinterpret_cast<Ctl*>(sm + OFF_CTL);
  pdl_wait_then_release();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* hdr = p.work.header();
  const int n_units = (kState ? hdr[kLinStateItems] : hdr[kLinItems]) * p.H;
  if ((int)blockIdx.x >= n_units) return;
  const uint32_t sbase = smem_u32(sm);
  if ((sbase & 1023u) != 0) {  // the operand tiles' swizzle counts on it
    if (tid == 0) atomicOr((unsigned*)&hdr[kErr], GDN_FLAG_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&ctl.full[b], 1);
      // V warps, S warps, MMA 2 (and MMA 1, store)
      mbar_init(&ctl.empty[b], kState ? 9 : 11);
      mbar_init(&ctl.zeroed[b], 4);
      mbar_init(&ctl.staged[b], 4);
    }
    mbar_init(&ctl.p_full, 1);
    mbar_init(&ctl.pb_full, 4);
    mbar_init(&ctl.qs_full, 1);
    mbar_init(&ctl.o_scaled, 4);
    mbar_init(&ctl.o_full, 1);
    mbar_init(&ctl.o_free, 4);
    mbar_init(&ctl.s_ready, 4);
    mbar_init(&ctl.v_full, 4);
    mbar_init(&ctl.v_free, 1);
    mbar_init(&ctl.u_full, 1);
    mbar_init(&ctl.u_free, 4);
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&ctl.tmem, TM_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem;
  bool dead = false;

  if (warp < 4) {
    // ============================== O warps ===============================
    regs_dec<112>();
    if (!kState) {
      const int i = tid;                               // row of the chunk, TMEM lane
      const uint32_t tl = (uint32_t)(warp * 32) << 16;
      int h = -1;
      float tab = 0.f, after = 0.f;   // e^{g lane}; scale e^{g (i+1)}
      float base[4];                  // scale e^{g (i - 32 jb - 31)} per block left of the diagonal
      float col[32];                  // e^{g (31 - jj)}
      for (int c = 0;; ++c) {
        const int b = c & 1;
        const uint32_t ph = (uint32_t)(c & 1);
        if (!warp_wait(&ctl.full[b], (c >> 1) & 1)) { dead = true; break; }
        const Desc d = ctl.desc[b];
        if (d.flags & kEnd) break;
        if (d.h != h) {
          h = d.h;
          const float g = finite_decay(p.log_decay[h]);
          tab = expf(g * (float)lane);
          after = p.scale * expf(g * (float)(i + 1));
#pragma unroll
          for (int jb = 0; jb < 4; ++jb)
            base[jb] = jb < warp ? p.scale * expf(g * (float)(i - 32 * jb - 31)) : 0.f;
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) col[jj] = __shfl_sync(0xffffffffu, tab, 31 - jj);
        }
        // ---- P: decay and mask, to bf16 over its own columns (block jb's 16
        // land on fp32 columns read before)
        if (!warp_wait(&ctl.p_full, ph)) { dead = true; break; }
        tc::fence_after_sync();
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          uint32_t w[16];
          if (jb <= warp) {
            float x[32];
            tc::tmem_ld32(tmem + tl + TM_P + jb * 32, x);
            tc::tmem_wait_ld();
            if (jb < warp) {
#pragma unroll
              for (int jj = 0; jj < 32; ++jj) x[jj] *= base[jb] * col[jj];
            } else {
#pragma unroll
              for (int jj = 0; jj < 32; ++jj) {
                const float f = __shfl_sync(0xffffffffu, tab, lane - jj) * p.scale;
                x[jj] = jj <= lane ? x[jj] * f : 0.f;
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = bf2(x[2 * e], x[2 * e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0u;
          }
          tc::tmem_st16u(tmem + tl + TM_P + jb * 16, w);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&ctl.pb_full);
        // ---- O = Q S0 times its row's decay
        if (!warp_wait(&ctl.qs_full, ph)) { dead = true; break; }
        tc::fence_after_sync();
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          float x[32];
          tc::tmem_ld32(tmem + tl + TM_O + jb * 32, x);
          tc::tmem_wait_ld();
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) x[jj] *= after;
          tc::tmem_st32(tmem + tl + TM_O + jb * 32, x);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&ctl.o_scaled);
        // ---- the chunk's outputs: staged over the q tile (its products are
        // done), or, past a sequence's end, the valid rows straight out
        if (!warp_wait(&ctl.o_full, ph)) { dead = true; break; }
        tc::fence_after_sync();
        unsigned char* stage = sm + b * ST_BYTES + ST_Q;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) +
                              (size_t)(d.row + i) * p.ldo + (size_t)d.h * D;
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          float x[32];
          tc::tmem_ld32(tmem + tl + TM_O + jb * 32, x);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w;
            w.x = bf2(x[8 * e], x[8 * e + 1]);
            w.y = bf2(x[8 * e + 2], x[8 * e + 3]);
            w.z = bf2(x[8 * e + 4], x[8 * e + 5]);
            w.w = bf2(x[8 * e + 6], x[8 * e + 7]);
            if (d.n == CH)
              *reinterpret_cast<uint4*>(stage + (jb >> 1) * BOX +
                                        tc::sw128_offset(i, (jb & 1) * 32 + 8 * e)) = w;
            else if (i < d.n)
              *reinterpret_cast<uint4*>(orow + jb * 32 + 8 * e) = w;
          }
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        warp_arrive(&ctl.o_free);
        if (lane == 0) arrive(&ctl.staged[b]);
      }
    }
  } else if (warp < 8) {
    // ============================== V warps ===============================
    regs_dec<112>();
    const int v = tid - 128;
    const uint32_t tl = (uint32_t)((warp - 4) * 32) << 16;
    // byte of element v in row t of a V tile: (t >> 3) KiB, then off[t & 7]
    uint32_t off[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      off[r] = (uint32_t)(v >> 6) * BOX + r * 128 + ((((v & 63) >> 3) ^ r) << 4) + (v & 7) * 2;
    int h = -1, halves = 0;
    float g = 0.f, w4[4];
    int w_n = 0;
    for (int c = 0;; ++c) {
      const int b = c & 1;
      if (!warp_wait(&ctl.full[b], (c >> 1) & 1)) { dead = true; break; }
      const Desc d = ctl.desc[b];
      if (d.flags & kEnd) break;
      unsigned char* kt = sm + b * ST_BYTES + ST_K;
      unsigned char* vt = sm + b * ST_BYTES + ST_V;
      // ---- k and v of the chunk: all finite?  Thread: 16-byte pieces of
      // both; x * 0 is NaN for what is not
      {
        __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
        const __nv_bfloat162 zero = acc;
#pragma unroll 4
        for (int e = v; e < 2 * 128 * 8; e += 128) {
          const int row = (e >> 3) & 127;
          if (row < d.n) {
            const uint32_t at = (uint32_t)(e >> 10) * BOX + row * 128 + (e & 7) * 16;
            const uint4 x = *reinterpret_cast<const uint4*>(kt + at);
            const uint4 y = *reinterpret_cast<const uint4*>(vt + at);
            const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int q = 0; q < 8; ++q)
              acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[q]), zero, acc);
          }
        }
        const float2 f = __bfloat1622float2(acc);
        const bool bad = __any_sync(0xffffffffu, !(f.x == 0.f && f.y == 0.f));
        if (lane == 0) {
          ctl.bad[b][warp - 4] = bad;
          if (bad) {
            p.bad[(size_t)d.entry * p.H + d.h] = 1;
            hdr[kLinBad] = 1;
          }
        }
      }
      // ---- rows past the sequence are another's: zeros, so that they add
      // nothing (their weights are zero, but 0 * inf is not)
      if (d.n < CH) {
        for (int e = v; e < 2 * 128 * 8; e += 128) {
          const int row = (e >> 3) & 127;
          if (row >= d.n) {
            const uint32_t at = (uint32_t)(e >> 10) * BOX + row * 128 + (e & 7) * 16;
            *reinterpret_cast<uint4*>(kt + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(vt + at) = make_uint4(0, 0, 0, 0);
          }
        }
        tc::fence_proxy_async_smem();
      }
      warp_arrive(&ctl.zeroed[b]);
      if (!(d.flags & kNoU)) {
        if (d.h != h || d.n != w_n) {
          if (d.h != h) g = finite_decay(p.log_decay[d.h]);
          h = d.h;
          w_n = d.n;
          // lane l: e^{g (n-1-j)} of tokens j = 4 l .. 4 l + 3, 0 past the end
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int back = w_n - 1 - (4 * lane + e);
            w4[e] = back >= 0 ? expf(g * (float)back) : 0.f;
          }
        }
        const int nh = d.n > 64 ? 2 : 1;
        for (int hf = 0; hf < nh; ++hf, ++halves) {
          if (halves > 0 && !warp_wait(&ctl.v_free, (halves - 1) & 1)) { dead = true; break; }
          tc::fence_after_sync();
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // 32 tokens: 16 columns of each term
            uint32_t hi[16], mid[16], lo[16];
            const int t0 = hf * 64 + q * 32;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int t = 2 * e;
              const unsigned char* at = vt + (t0 + t) / 8 * 1024;
              // rows past n read as zero from other warps' stores or as the
              // neighbour's bits from before them: the weight decides
              float f0 = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at + off[t & 7]) << 16);
              float f1 = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at + off[(t + 1) & 7]) << 16);
              const float wa = __shfl_sync(0xffffffffu, w4[t & 3], (t0 + t) >> 2);
              const float wb = __shfl_sync(0xffffffffu, w4[(t + 1) & 3], (t0 + t) >> 2);
              f0 = t0 + t < d.n ? f0 * wa : 0.f;
              f1 = t0 + t + 1 < d.n ? f1 * wb : 0.f;
              hi[e] = bf2(f0, f1);
              f0 -= bf_lo(hi[e]);
              f1 -= bf_hi(hi[e]);
              mid[e] = bf2(f0, f1);
              f0 -= bf_lo(mid[e]);
              f1 -= bf_hi(mid[e]);
              lo[e] = bf2(f0, f1);
            }
            tc::tmem_st16u(tmem + tl + TM_V + q * 16, hi);
            tc::tmem_st16u(tmem + tl + TM_V + 32 + q * 16, mid);
            tc::tmem_st16u(tmem + tl + TM_V + 64 + q * 16, lo);
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          warp_arrive(&ctl.v_full);
        }
        if (dead) break;
      }
      warp_arrive(&ctl.empty[b]);
    }
  } else if (warp < 12) {
    // ============================== S warps ===============================
    regs_inc<200>();
    const int v = tid - 256;
    const uint32_t tl = (uint32_t)((warp - 8) * 32) << 16;
    float S[D];
    bool bad = false;
    int ups = 0;  // updates so far
    for (int c = 0;; ++c) {
      const int b = c & 1;
      if (!warp_wait(&ctl.full[b], (c >> 1) & 1)) { dead = true; break; }
      const Desc d = ctl.desc[b];
      if (d.flags & kEnd) break;
      if (d.flags & kFirst) {
        bad = false;
        const float* src = nullptr;
        if (!kState) {
          if (d.slot >= 0)
            src = p.seg_states + (size_t)d.slot * D * D;
          else if (d.rblk != 0)
            src = reinterpret_cast<const float*>(p.layer_base + (size_t)d.rblk * p.stride) +
                  (size_t)d.h * D * D;
        }
#pragma unroll
        for (int k = 0; k < D; ++k) S[k] = src ? src[(size_t)k * D + v] : 0.f;
      }
      if (!kState) {
        // ---- S0 as the B operand [v][k] of O = Q S0
        if (c > 0 && !warp_wait(&ctl.qs_full, (c - 1) & 1)) { dead = true; break; }
#pragma unroll
        for (int k = 0; k < D; k += 8)
          tc::sw128_store8<__nv_bfloat16>(sm + OFF_S + (k >> 6) * BOX, v, k & 63, S + k);
        tc::fence_proxy_async_smem();
        warp_arrive(&ctl.s_ready);
      }
      if (!(d.flags & kNoU)) {
        const DecayPair a = decay_pair(finite_decay(p.log_decay[d.h]) * (float)d.n);
        if (!warp_wait(&ctl.u_full, ups & 1)) { dead = true; break; }
        ++ups;
        tc::fence_after_sync();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          float x[32];
          tc::tmem_ld32(tmem + tl + TM_U + kb * 32, x);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            S[kb * 32 + e] = fmaf(a.hi, S[kb * 32 + e], fmaf(a.lo, S[kb * 32 + e], x[e]));
        }
        tc::fence_before_sync();
        warp_arrive(&ctl.u_free);
      }
      bad |= (ctl.bad[b][0] | ctl.bad[b][1] | ctl.bad[b][2] | ctl.bad[b][3]) != 0;
      if (d.flags & kLast) {
        float* dst = nullptr;
        if (kState) {
          dst = p.seg_states + (size_t)d.slot * D * D;
        } else if ((d.flags & kFinal) && !bad &&
                   (d.slot < 0 || !p.bad[(size_t)d.entry * p.H + d.h])) {
          // (an earlier segment's mark is the state pass's, which has ended)
          dst = reinterpret_cast<float*>(p.layer_base + (size_t)d.wblk * p.stride) +
                (size_t)d.h * D * D;
        }
        if (dst) {
#pragma unroll
          for (int k = 0; k < D; ++k) dst[(size_t)k * D + v] = S[k];
        }
      }
      warp_arrive(&ctl.empty[b]);
    }
  } else {
    regs_dec<80>();
    if (warp == 12 && lane == 0) {
      // ============================== producer ==============================
      int c = 0;
      for (bool end = false; !end && !dead;) {
        const int u = atomicAdd(&hdr[kState ? kLinStateHead : kLinHead], 1);
        end = u >= n_units;
        int s = 0, h = 0, e = 0, seg = 0, c0 = 0, c1 = 1, L = 0, nseg = 1;
        if (!end) {
          const int item = u / p.H;
          h = u % p.H;
          const int32_t* first = p.work.pre_cp();  // first[k]: segments before entry k
          int lo = 0, hi = hdr[kNPre] - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= item) lo = mid; else hi = mid - 1;
          }
          e = lo;
          s = p.work.pre()[e];
          seg = item - first[e];
          nseg = first[e + 1] - first[e];
          L = p.cu[s + 1] - p.cu[s];
          const int nch = (L + CH - 1) / CH;
          const int per = nseg > 1 ? hdr[kLinSegChunks] : nch;
          c0 = seg * per;
          c1 = min(nch, c0 + per);
          // the last segment's own state is not needed by any other
          if (kState && seg == nseg - 1) continue;
        }
        const int hk = h / p.group;
        for (int k = c0; k < c1; ++k, ++c) {
          const int b = c & 1;
          if (c >= kStages && !mbar_wait_bounded(&ctl.empty[b], ((c >> 1) - 1) & 1)) {
            dead = true;
            break;
          }
          Desc d;
          d.row = end ? 0 : p.cu[s] + k * CH;
          d.n = end ? 0 : min(CH, L - k * CH);
          d.h = h;
          d.entry = e;
          d.slot = nseg > 1 ? (p.work.pre_cp()[e] + seg) * p.H + h : -1;
          d.wblk = end ? 0 : p.blk[s];
          d.rblk = !end && p.has_past[s] ? d.wblk : 0;
          d.flags = end ? kEnd
                        : (k == c0 ? kFirst : 0) | (k == c1 - 1 ? kLast : 0) |
                              (seg == nseg - 1 ? kFinal : 0) |
                              (!kState && k == c1 - 1 && seg < nseg - 1 ? kNoU : 0);
          ctl.desc[b] = d;
          if (end) {
            arrive(&ctl.full[b]);
            break;
          }
          unsigned char* st = sm + b * ST_BYTES;
          mbar_arrive_expect_tx(&ctl.full[b], kState ? 2 * TILE : 3 * TILE);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            tma_load_2d(st + ST_K + x * BOX, &tk, hk * D + x * 64, d.row, &ctl.full[b]);
            if (!kState) tma_load_2d(st + ST_Q + x * BOX, &tq, h * D + x * 64, d.row, &ctl.full[b]);
            tma_load_2d(st + ST_V + x * BOX, &tv, hk * D + x * 64, d.row, &ctl.full[b]);
          }
        }
      }
      if (dead) {
        // the loads already issued land before the CTA ends
        for (int k = c > kStages ? c - kStages : 0; k < c; ++k)
          mbar_wait_bounded(&ctl.full[k & 1], (k >> 1) & 1);
      }
    } else if (warp == 13 && lane == 0 && !kState) {
      // ============================== MMA 1 =================================
      constexpr uint32_t kId = tc::idesc_bf16_f32(128, 128);
      constexpr uint32_t kIdMN = tc::idesc_bf16_f32(128, 128, false, true);
      for (int c = 0;; ++c) {
        const int b = c & 1;
        const uint32_t ph = (uint32_t)(c & 1), st = sbase + b * ST_BYTES;
        if (!mbar_wait_bounded(&ctl.full[b], (c >> 1) & 1)) { dead = true; break; }
        if (ctl.desc[b].flags & kEnd) break;
        // P = Q K^T, once the last chunk's P V has read P
        if (c > 0 && !mbar_wait_bounded(&ctl.o_full, ph ^ 1)) { dead = true; break; }
        tc::fence_after_sync();
        tc::mma_op(tmem + TM_P, tc::Opnd{st + ST_Q, BOX, false}, tc::Opnd{st + ST_K, BOX, false}, 8,
                   kId, false);
        tc::commit(&ctl.p_full);
        // O = Q S0
        if (!mbar_wait_bounded(&ctl.s_ready, ph) ||
            (c > 0 && !mbar_wait_bounded(&ctl.o_free, ph ^ 1))) {
          dead = true;
          break;
        }
        tc::fence_after_sync();
        tc::mma_op(tmem + TM_O, tc::Opnd{st + ST_Q, BOX, false}, tc::Opnd{sbase + OFF_S, BOX, false},
                   8, kId, false);
        tc::commit(&ctl.qs_full);
        // O += P V
        if (!mbar_wait_bounded(&ctl.zeroed[b], (c >> 1) & 1) || !mbar_wait_bounded(&ctl.pb_full, ph) ||
            !mbar_wait_bounded(&ctl.o_scaled, ph)) {
          dead = true;
          break;
        }
        tc::fence_after_sync();
        tc::mma_op_ts(tmem + TM_O, tmem + TM_P, tc::Opnd{st + ST_V, BOX, true}, 8, kIdMN, true);
        tc::commit(&ctl.o_full);
        tc::commit(&ctl.empty[b]);
      }
    } else if (warp == 14 && lane == 0) {
      // ============================== MMA 2 =================================
      constexpr uint32_t kIdMN = tc::idesc_bf16_f32(128, 128, false, true);
      int halves = 0, ups = 0;
      for (int c = 0; !dead; ++c) {
        const int b = c & 1;
        const uint32_t kt = sbase + b * ST_BYTES + ST_K;
        if (!mbar_wait_bounded(&ctl.full[b], (c >> 1) & 1)) { dead = true; break; }
        const int flags = ctl.desc[b].flags, n = ctl.desc[b].n;
        if (flags & kEnd) break;
        if (flags & kNoU) {
          arrive(&ctl.empty[b]);
          continue;
        }
        if (ups > 0 && !mbar_wait_bounded(&ctl.u_free, (ups - 1) & 1)) { dead = true; break; }
        const int nh = n > 64 ? 2 : 1;
        for (int hf = 0; hf < nh; ++hf, ++halves) {
          if (!mbar_wait_bounded(&ctl.v_full, halves & 1)) { dead = true; break; }
          tc::fence_after_sync();
          // U (+)= (lo + mid + hi) K over 64 tokens, the smallest term first
#pragma unroll
          for (int term = 2; term >= 0; --term)
            tc::mma_op_ts(tmem + TM_U, tmem + TM_V + term * 32,
                          tc::Opnd{kt + (uint32_t)hf * 8192u, BOX, true}, 4, kIdMN,
                          hf > 0 || term < 2);
          tc::commit(&ctl.v_free);
        }
        if (dead) break;
        ++ups;
        tc::commit(&ctl.u_full);
        tc::commit(&ctl.empty[b]);
      }
    } else if (warp == 15 && lane == 0 && !kState) {
      // ============================== store =================================
      for (int c = 0;; ++c) {
        const int b = c & 1;
        if (!mbar_wait_bounded(&ctl.full[b], (c >> 1) & 1)) { dead = true; break; }
        const Desc d = ctl.desc[b];
        if (d.flags & kEnd) break;
        if (!mbar_wait_bounded(&ctl.staged[b], (c >> 1) & 1)) { dead = true; break; }
        if (d.n == CH) {
          const unsigned char* st = sm + b * ST_BYTES + ST_Q;
          tma_store_2d(&to, d.h * D, d.row, st);
          tma_store_2d(&to, d.h * D + 64, d.row, st + BOX);
          bulk_commit();
          bulk_wait_read_all();
        }
        arrive(&ctl.empty[b]);
      }
      bulk_wait_all();
    }
    __syncwarp();
  }
  if (dead && lane == 0) atomicOr((unsigned*)&hdr[kErr], GDN_FLAG_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, TM_COLS);
}

// The states at the segments' starts, from the segments' own: in place,
// Z[0] <- S0, Z[i] <- e^{g n} Z[i-1] + (the old Z[i-1]) with n tokens per
// segment.  One float4 of one head's state per thread.
__global__ void __launch_bounds__(256) lin_segments_kernel(LinParams p) {
  pdl_wait_then_release();
  const int32_t* hdr = p.work.header();
  const int n_split = hdr[kLinSplit];
  constexpr int kParts = D * D / 4 / 256;
  const int n_units = n_split * p.H * kParts;
  for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
    const int part = u % kParts, h = (u / kParts) % p.H, e = u / (kParts * p.H);
    const int s = p.work.pre()[e], blk = p.blk[s];
    const int first = p.work.pre_cp()[e], nseg = p.work.pre_cp()[e + 1] - first;
    const size_t at = (size_t)part * 256 + threadIdx.x;
    const DecayPair a =
        decay_pair(finite_decay(p.log_decay[h]) * (float)(hdr[kLinSegChunks] * CH));
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.has_past[s])
      S = reinterpret_cast<const float4*>(p.layer_base + (size_t)blk * p.stride)[(size_t)h * D * D / 4 + at];
    float4* z = reinterpret_cast<float4*>(p.seg_states) + ((size_t)first * p.H + h) * (D * D / 4) + at;
    const size_t step = (size_t)p.H * (D * D / 4);
    for (int i = 0; i < nseg; ++i, z += step) {
      const float4 own = i < nseg - 1 ? *z : S;
      *z = S;
      S.x = fmaf(a.hi, S.x, fmaf(a.lo, S.x, own.x));
      S.y = fmaf(a.hi, S.y, fmaf(a.lo, S.y, own.y));
      S.z = fmaf(a.hi, S.z, fmaf(a.lo, S.z, own.z));
      S.w = fmaf(a.hi, S.w, fmaf(a.lo, S.w, own.w));
    }
  }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

// Tensor map of `rows` rows of `cols` bf16 at a pitch of ld elements, in
// boxes of 64 columns x 128 rows, 128-byte swizzled, zero fill past the end.
cudaError_t rows_map(CUtensorMap* m, const void* base, int rows, long long cols, long long ld) {
  static EncodeFn encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    encode = reinterpret_cast<EncodeFn>(fn);
  }
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)CH}, estr[2] = {1, 1};
  const CUresult r =
      encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

bool lin_chunk_supported(int d, int act) { return d == D && act == GDN_BF16; }

cudaError_t launch_lin_chunk(const LinParams& p, bool may_split, int num_sms, cudaStream_t s) {
  CUtensorMap tq, tk, tv, to;
  const long long qc = (long long)p.H * D, kc = (long long)(p.H / p.group) * D;
  cudaError_t e = rows_map(&tq, p.q, p.T, qc, p.ldq);
  if (e == cudaSuccess) e = rows_map(&tk, p.k, p.T, kc, p.ldk);
  if (e == cudaSuccess) e = rows_map(&tv, p.v, p.T, kc, p.ldv);
  if (e == cudaSuccess) e = rows_map(&to, p.out, p.T, qc, p.ldo);
  if (e != cudaSuccess) return e;
  for (int state = may_split ? 1 : 0; state >= 0; --state) {
    auto kern = state ? lin_chunk_kernel<true> : lin_chunk_kernel<false>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e == cudaSuccess)
      e = launch_pdl(kern, dim3(num_sms), dim3(kThreads), SMEM_BYTES, s, p, tq, tk, tv, to);
    if (e == cudaSuccess && state)
      e = launch_pdl(lin_segments_kernel, dim3(4 * num_sms), dim3(256), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
