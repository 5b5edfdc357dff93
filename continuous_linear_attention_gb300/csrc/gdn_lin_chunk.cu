// Chunked form of decayed linear attention for prompts (d = 128, bf16): the
// recurrence S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over chunks
// of 128 tokens.  With S0 the state at a chunk's start, n its valid tokens and
// i, j = 0 .. n-1 in the chunk,
//   P[i][j] = scale e^{g (i-j)} (q_i . k_j)  for j <= i, else 0
//   o_i     = scale e^{g (i+1)} S0^T q_i + sum_j P[i][j] v_j
//   S_n     = e^{g n} S0 + sum_j e^{g (n-1-j)} k_j v_j^T
// so a (sequence, head) chain is four 128^3 products per chunk, and all but
// the first term of each line does not depend on the chunks before.  No weight
// is a growing power that another one takes back, so any decay will do.
//
// Bytes are its floor: q, k, v and o are 128 KB per chunk and head (2.9 us of
// one SM's share of HBM); the products, P V and Q S0 in two terms and the
// state's in four, are nine 128^3 (2.9 us of one SM's tensor rate at the
// measured peak).  Measured: 4.7 us per chunk with all SMs busy (15,843 tokens
// x 64 heads in 252 us, 4.3 TB/s; the loads and stores of this pipeline alone
// take 177).  What bounds it is the O warps' chain through a chunk: P's
// conversion, the scaling of Q S0, P V and the output one after the other.
//
// One CTA per SM, chains claimed from a counter, longest first.  Roles, each
// a loop over the CTA's chunks that meets the others at mbarriers only:
//   producer  one thread: TMA loads of a chunk's q, k, v tiles, two stages; k and
//             v as soon as their products are done, q when its tile has been
//             stored as output (2% faster than all three at once)
//   MMA 1     one warp: P = Q K^T, O = Q S0, then O += P V in two halves of 64
//             columns, so that the O warps' work on one half runs beside it
//   MMA 2     one warp: U = sum of the decayed v k^T, 32 tokens at a time
//   store     one thread: the staged output tile to global memory by TMA
//   O warps   P with its decay -> bf16 A operand; O <- scale e^{g(i+1)} O; output
//   V warps   e^{g(n-1-j)} v_j -> A operand of U, rows past the chunk's end
//             zeroed
//   S warps   the state, fp32 in registers (thread v holds S[.][v]): its bf16
//             terms in turn as operand of O, S <- e^{g n} S + U
//
// Precision.  The partners of P and S0 are bf16, and one MMA takes one type:
// both enter as two bf16 terms, exact to 2^-16, which leaves the output's own
// rounding the only one that counts, as in the recurrent form (rel. L2 1.7e-3;
// one term each made it 2.3e-3, in 217 us for the call above).  The state is
// an output in fp32 and carried over the whole prompt, so its update takes
// more: a decayed v has 8 + 24 significant bits and goes in as four bf16 terms.
// With the weight as
// wh + wm + wl (8 bits each), v wh is its bf16 rounding plus a remainder that
// an fma gives exactly and that is a bf16 again, v wm likewise, and v wl joins
// the last remainder (2^-18 of the whole, off by 2^-27): five packed bf16
// instructions for two elements, where splitting the fp32 product took twelve.
// The terms enter the smallest first, and U is added to S in fp32 registers
// with a decay pair (see decay_pair).  Accumulating into S itself in tensor
// memory would add a rounding of S at each of 32 MMA steps per chunk.
//
// A non-finite v reaches its column of earlier tokens' rows through 0 * inf in
// the masked products.  It also makes that column of the state non-finite for
// good, which is seen at the chain's end: those columns are left to the
// token-serial kernel, and their block keeps the old state until then.  A
// non-finite q or k reaches only its own row and the later ones, as it should:
// P's mask selects, it does not multiply.
//
// Weights.  P's weights scale e^{g (i-j)} are a head's table in shared memory,
// four loaded at a time; made of two factors, one of them by a shuffle per
// element, they took 3,400 cycles a chunk of the O warps instead of 2,200.
//
// Few long chains: where it is cheaper (see the scheduler), long sequences are
// cut into segments.  A first launch of this kernel
// (kState) computes every segment's own state from k and v alone, a small
// kernel turns those into the states at the segments' starts, and the output
// pass then runs all segments at once; k and v are read twice (32,768 tokens x 16
// heads 196 us, of one head 45 us; unsplit 990 and 880).
#include <cuda.h>

#include "gdn_lin.cuh"
#include "gdn_ptx.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int D = 128;
constexpr int CH = kLinChunk;  // 128
constexpr int kThreads = 768;  // O, V and S warps (8, 8, 4), producer, MMA 1, MMA 2, store
constexpr int kOWarps = 8, kVWarps = 8, kSWarp = 16, kCtlWarp = 20;
constexpr uint32_t TILE = 32768, BOX = 16384;  // a [128][128] bf16 tile: two 64-column boxes
// stages of a chunk's q, k and v (three of k and v for the state pass), then
// S0 as B operand, one bf16 term at a time: [v][k], two 64-k blocks
constexpr int kMaxStages = 3;
constexpr uint32_t OFF_S = 6 * TILE;
// Stage of a role's current chunk and the parity of its pass over the stages.
template <int kStages>
struct Pos {
  int b = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++b == kStages) {
      b = 0;
      ph ^= 1;
    }
  }
};
// tensor memory columns: P fp32 (per 32 columns then the two bf16 terms, 16 columns
// each), O, U, then the four terms of 32 decayed v rows, twice: per 16 rows 8
// columns of each term
constexpr uint32_t TM_P = 0, TM_O = 128, TM_U = 256, TM_V = 384, TM_COLS = 512;
constexpr int QT = 32;  // tokens per step of U
constexpr int kTerms = 4;
// the state pass has no P and O: two buffers for U and four for the decayed v
constexpr uint32_t TM_U1 = 0, TM_V1 = 128;

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
  int rblk, wblk;       // blocks read (0: zeros) and written
};

// A head's weights scale e^{g m}, 0 <= m < 128, by falling m and then zeros:
// copy r begins with the r-th, so that a thread reads four from any place on
// as one 16-byte load, and the copies lie a quarter of the banks apart.
constexpr int kWeights = 160, kWeightCopy = kWeights + 8;
struct Ctl {
  Desc desc[kMaxStages];
  uint64_t full[kMaxStages], kv_free[kMaxStages], q_free[kMaxStages], zeroed[kMaxStages], staged[kMaxStages];
  uint64_t p_full, pb_full, qs_full, o_scaled, o_full[2], o_free, s_ready, s_read;
  uint64_t v_full[4], v_free[4], u_full[2], u_free[2];
  uint64_t w_ready;
  uint32_t tmem;
  alignas(16) float weight[3 * kWeightCopy + kWeights];
};
constexpr uint32_t OFF_CTL = OFF_S + TILE;
constexpr uint32_t SMEM_BYTES = OFF_CTL + sizeof(Ctl);
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");

// A bounded wait.  The first test has no suspend time, which would add 30
// cycles to a wait whose phase is complete (55).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0 || mbar_wait_bounded(bar, parity);
}
// The same for a warp: false for all lanes if any gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_for(bar, parity));
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
__device__ __forceinline__ uint32_t bf2(F2 v) {
  float x, y;
  unf2(v, x, y);
  return bf2(x, y);
}
// The two bf16 of a word as fp32.
__device__ __forceinline__ F2 widen(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// A pair as two bf16 terms.  The first one of an infinity is the largest number,
// so that the second one and their sum are that infinity and not NaN.  (Volatile:
// computed again for the second term, where keeping 64 first ones would spill.)
__device__ __forceinline__ uint32_t term1(F2 v) {
  float x, y;
  unf2(v, x, y);
  uint32_t r;
  asm volatile("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t term2(F2 v) { return bf2(fma2(widen(term1(v)), f2(-1.f, -1.f), v)); }
// Four transposed 8 x 8 matrices of 16-bit elements: lane l gives the address
// of row l % 8 of matrix l / 8 and gets of each matrix column l / 4, rows
// 2 (l % 4) and the next.
__device__ __forceinline__ void ldmatrix4_t(const void* at, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(at))
               : "memory");
}
// Four pairs of such fragments as words of 16 tensor memory lanes x 32 columns:
// words 4 i and 4 i + 1 are lanes l / 4 and l / 4 + 8 of column 8 i + l % 4,
// words 4 i + 2 and 4 i + 3 of column 8 i + 4 + l % 4.
__device__ __forceinline__ void tmem_st_frag4(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Packed bf16 products, each rounded once.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// a b - c
__device__ __forceinline__ uint32_t hfms2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("{\n\t.reg .b32 m;\n\tneg.bf16x2 m, %3;\n\tfma.rn.bf16x2 %0, %1, %2, m;\n\t}"
      : "=r"(r)
      : "r"(a), "r"(b), "r"(c));
  return r;
}
// MMA issue.  A whole warp runs the issuing loop, so that descriptors and
// addresses stay in uniform registers, and one elected lane issues: with a
// lone thread every operand had to be moved there, 110 cycles per MMA, which
// bound the kernel.  Descriptors differ in their low word only: K-major
// operands advance by 32 bytes per 16 elements (two blocks of 64, BOX apart),
// MN-major ones by 16 rows of 128 bytes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | ((BOX >> 4) << 16);
}
// the high word of both: groups of 8 rows 1024 bytes apart, 128-byte swizzle
constexpr uint64_t kDescHi = ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
__host__ __device__ constexpr uint32_t step_k(int s) { return (uint32_t)(s >> 2) * (BOX >> 4) + (uint32_t)(s & 3) * 2u; }
constexpr uint32_t kStepMN = 2048u >> 4;

template <bool kState>
__global__ void __launch_bounds__(kThreads, 1)
lin_chunk_kernel(LinParams p, const __grid_constant__ CUtensorMap tq,
                 const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ CUtensorMap to) {
  constexpr int kStages = kState ? 3 : 2;
  constexpr uint32_t ST_Q = 0, ST_K = kState ? 0 : TILE, ST_V = ST_K + TILE, ST_BYTES = ST_V + TILE;
  static_assert(kStages * ST_BYTES == OFF_S && kStages <= kMaxStages, "stages fill their room");
  extern __shared__ __align__(1024) unsigned char sm[];
  Ctl& ctl = *reinterpret_cast<Ctl*>(sm + OFF_CTL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int32_t* hdr = p.work.header();
  const uint32_t sbase = smem_u32(sm);
  if (tid == 0) {
    for (int b = 0; b < kStages; ++b) {
      // of the k and v tiles, and of the q tile and the descriptor
      mbar_init(&ctl.full[b], kState ? 1 : 2);
      mbar_init(&ctl.kv_free[b], kVWarps + (kState ? 1 : 2));  // V warps, MMA 2 (and 1)
      mbar_init(&ctl.q_free[b], 4 + (kState ? 0 : 1));         // S warps (and the store)
      mbar_init(&ctl.zeroed[b], kVWarps);
      mbar_init(&ctl.staged[b], kOWarps);
    }
    mbar_init(&ctl.w_ready, kOWarps);
    mbar_init(&ctl.p_full, 1);
    mbar_init(&ctl.pb_full, kOWarps);
    mbar_init(&ctl.qs_full, 1);
    mbar_init(&ctl.o_scaled, kOWarps);
    mbar_init(&ctl.o_full[0], 1);
    mbar_init(&ctl.o_full[1], 1);
    mbar_init(&ctl.o_free, kOWarps);
    mbar_init(&ctl.s_ready, 4);
    mbar_init(&ctl.s_read, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.u_full[b], 1);
      mbar_init(&ctl.u_free[b], 4);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&ctl.v_full[b], kVWarps);
      mbar_init(&ctl.v_free[b], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&ctl.tmem, TM_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem;
  // (up to here beside the kernel before this one)
  pdl_wait_then_release();
  const int n_units = (kState ? hdr[kLinStateItems] : hdr[kLinItems]) * p.H;
  const bool aligned = (sbase & 1023u) == 0;  // the operand tiles' swizzle counts on it
  if (!aligned && tid == 0) atomicOr((unsigned*)&hdr[kErr], GDN_FLAG_TIMEOUT);
  if ((int)blockIdx.x >= n_units || !aligned) {
    if (warp == 0) tc::tmem_dealloc(tmem, TM_COLS);
    return;
  }
  bool dead = false;
  // buffers of U and of the decayed v: their number (a power of two, by its
  // logarithm) and tensor memory columns
  constexpr int kULog = kState ? 1 : 0, kVLog = kState ? 2 : 1;
  auto u_col = [](int b) { return b == 0 ? TM_U : TM_U1; };
  auto v_col = [](int b) { return (b < 2 ? TM_V : TM_V1) + (uint32_t)(b & 1) * (16 * kTerms); };

  // registers a thread, of 80 at launch: O as launched, V 48, S 184, the others 40
  if (warp < kOWarps) {
    // ============================== O warps ===============================
    // Warps w and w + 4 have rows 32 w .. 32 w + 31 of the chunk (TMEM lanes)
    // and columns 0 .. 63 or 64 .. 127 of P and O.
    const int rw = warp & 3, hf = warp >> 2;
    const int i = rw * 32 + lane;
    const uint32_t tl = (uint32_t)(rw * 32) << 16;
    int h = -1;
    uint32_t heads = 0;
    float after = 0.f;  // scale e^{g (i+1)}
    Pos<kStages> pos;
    for (int c = 0; !kState; ++c, pos.next()) {
      const int b = pos.b;
      const uint32_t ph = (uint32_t)(c & 1);
      if (!warp_wait(&ctl.full[b], pos.ph)) { dead = true; break; }
      if (ctl.desc[b].flags & kEnd) break;
      const int row = ctl.desc[b].row, n = ctl.desc[b].n;
      if (ctl.desc[b].h != h) {
        h = ctl.desc[b].h;
        const float g = finite_decay(p.log_decay[h]);
        after = p.scale * expf(g * (float)(i + 1));
        // the last head's weights have been used
        if (c > 0 && !warp_wait(&ctl.pb_full, ph ^ 1)) { dead = true; break; }
        for (int e = tid; e < 4 * kWeights; e += 32 * kOWarps) {
          const int copy = e / kWeights, at = e % kWeights, m = CH - 1 - at - copy;
          ctl.weight[copy * kWeightCopy + at] = m >= 0 ? p.scale * expf(g * (float)m) : 0.f;
        }
        warp_arrive(&ctl.w_ready);
        if (!warp_wait(&ctl.w_ready, heads)) { dead = true; break; }
        heads ^= 1;
      }
      // ---- P: decay and mask, each block of 32 columns to its two bf16 terms
      // in place, 16 columns each
      if (!warp_wait(&ctl.p_full, ph)) { dead = true; break; }
      tc::fence_after_sync();
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        const int jb = 2 * hf + u;
        const uint32_t at = tmem + tl + TM_P + jb * 32;
        if (jb > rw) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0u;
          tc::tmem_st16u(at, w);
          tc::tmem_st16u(at + 16, w);
        } else {
          float x[32];
          F2 y[16];
          tc::tmem_ld32(at, x);
          const bool diagonal = jb == rw;
          const float* wt = ctl.weight + (~lane & 3) * kWeightCopy + (CH - 4 - (i & ~3) + 32 * jb);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(wt + e);
            y[e / 2] = mul2(f2(x[e], x[e + 1]), f2(f.x, f.y));
            y[e / 2 + 1] = mul2(f2(x[e + 2], x[e + 3]), f2(f.z, f.w));
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = t == 0 ? term1(y[e]) : term2(y[e]);
            if (diagonal) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[e] = lane > 2 * e ? w[e] : lane == 2 * e ? w[e] & 0xffffu : 0u;
            }
            tc::tmem_st16u(at + 16 * t, w);
          }
        }
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      warp_arrive(&ctl.pb_full);
      // ---- O = Q S0 times its row's decay
      if (!warp_wait(&ctl.qs_full, ph)) { dead = true; break; }
      tc::fence_after_sync();
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        float x[32];
        const uint32_t at = tmem + tl + TM_O + hf * 64 + u * 32;
        tc::tmem_ld32(at, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] *= after;
        tc::tmem_st32(at, x);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      warp_arrive(&ctl.o_scaled);
      // ---- the chunk's outputs: staged over the q tile (its products are
      // done), or, past a sequence's end, the valid rows straight out
      if (!warp_wait(&ctl.o_full[hf], ph)) { dead = true; break; }
      tc::fence_after_sync();
      unsigned char* stage = sm + b * ST_BYTES + ST_Q + hf * BOX;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + (size_t)(row + i) * p.ldo +
                            (size_t)h * D + hf * 64;
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        float x[32];
        tc::tmem_ld32(tmem + tl + TM_O + hf * 64 + u * 32, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 w;
          w.x = bf2(x[8 * e], x[8 * e + 1]);
          w.y = bf2(x[8 * e + 2], x[8 * e + 3]);
          w.z = bf2(x[8 * e + 4], x[8 * e + 5]);
          w.w = bf2(x[8 * e + 6], x[8 * e + 7]);
          if (n == CH)
            *reinterpret_cast<uint4*>(stage + tc::sw128_offset(i, u * 32 + 8 * e)) = w;
          else if (i < n)
            *reinterpret_cast<uint4*>(orow + u * 32 + 8 * e) = w;
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      warp_arrive(&ctl.o_free);
      if (lane == 0) arrive(&ctl.staged[b]);
    }
  } else if (warp < kSWarp) {
    // ============================== V warps ===============================
    // Warps w and w + 4 make the operand rows (TMEM lanes) 32 w .. 32 w + 31 =
    // elements v, each of 16 of a step's 32 tokens, as transposed 8 x 8
    // fragments: this lane gets tokens 2 (lane % 4) and the next of each 8,
    // elements lane / 4 of each 8.  (With one warp per sub-partition these
    // dependent chains took 4,800 of a chunk's 8,400 cycles.)
    regs_dec<48>();
    const int vw = warp & 3, half = (warp >> 2) & 1;
    const uint32_t tl = (uint32_t)(vw * 32) << 16;
    const int mr = lane & 7, mt = lane >> 4, mv = (lane >> 3) & 1;  // matrix row, token and element half
    const uint32_t off = (uint32_t)(vw >> 1) * BOX + (mt * 8 + mr) * 128 +
                         ((((vw & 1) * 4 + mv) ^ mr) << 4);
    const int tl0 = 2 * (lane & 3);  // this lane's first token of each 8
    int h = -1, w_n = -1, steps = 0;
    // the weights' three bf16 terms of tokens 2 lane and 2 lane + 1 (wa), and
    // 64 more (wb)
    uint32_t wa[3] = {0, 0, 0}, wb[3] = {0, 0, 0};
    Pos<kStages> pos;
    for (int c = 0;; ++c, pos.next()) {
      const int b = pos.b;
      if (!warp_wait(&ctl.full[b], pos.ph)) { dead = true; break; }
      const Desc d = ctl.desc[b];
      if (d.flags & kEnd) break;
      unsigned char* kt = sm + b * ST_BYTES + ST_K;
      unsigned char* vt = sm + b * ST_BYTES + ST_V;
      const bool full = d.n == CH;
      // ---- rows past the sequence are another's: zeros, so that they add
      // nothing (their weights are zero, but 0 * inf is not)
      if (!full) {
        for (int e = tid - 32 * kOWarps; e < 2 * 128 * 8; e += 32 * kVWarps) {
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
      if (d.h != h || d.n != w_n) {
        h = d.h;
        w_n = d.n;
        const float g = finite_decay(p.log_decay[h]);
        const F2 minus = f2(-1.f, -1.f);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int back = w_n - 1 - 64 * u - 2 * lane;  // tokens behind the first of the pair
          F2 w = f2(back >= 0 ? expf(g * (float)back) : 0.f,
                    back >= 1 ? expf(g * (float)(back - 1)) : 0.f);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t r = bf2(w);
            w = fma2(widen(r), minus, w);
            (u ? wb : wa)[k] = r;
          }
        }
      }
      const int nq = (d.n + QT - 1) / QT;
      for (int q = 0; q < nq; ++q) {
        const int buf = steps & ((1 << kVLog) - 1);
        if (!(d.flags & kNoU)) {
          if ((steps >> kVLog) > 0 && !warp_wait(&ctl.v_free[buf], ((steps >> kVLog) - 1) & 1)) {
            dead = true;
            break;
          }
          tc::fence_after_sync();
        }
        const int t0 = q * QT + 16 * half;
        uint32_t x[8];
        ldmatrix4_t(vt + t0 * 128 + off, x);
        ldmatrix4_t(vt + t0 * 128 + (off ^ 32u), x + 4);
        // the weights of this lane's tokens in each 8
        uint32_t w[2][3];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int from = ((t0 & 63) >> 1) + 4 * m + (lane & 3);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            w[m][k] = __shfl_sync(0xffffffffu, t0 < 64 ? wa[k] : wb[k], from);
        }
        if (!full) {
          // rows past n read as zeros or, before another warp's stores, as the
          // neighbour's bits
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int left = d.n - (t0 + 8 * m + tl0);
            const uint32_t keep = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
            x[2 * m] &= keep;
            x[2 * m + 1] &= keep;
            x[2 * m + 4] &= keep;
            x[2 * m + 5] &= keep;
          }
        }
        // the products' four terms, 16 elements v at a time
        const uint32_t at = tmem + tl + v_col(buf) + half * (8 * kTerms);
#pragma unroll
        for (int v2 = 0; v2 < 2; ++v2) {
          uint32_t t[kTerms][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t y = x[4 * v2 + e];
            const uint32_t* wt = w[e >> 1];
            t[0][e] = hmul2(y, wt[0]);
            t[1][e] = hfms2(y, wt[0], t[0][e]);
            t[2][e] = hmul2(y, wt[1]);
            t[3][e] = hfma2(y, wt[2], hfms2(y, wt[1], t[2][e]));
          }
          if (!(d.flags & kNoU)) tmem_st_frag4(at + v2 * (16u << 16), t[0]);
        }
        if (!(d.flags & kNoU)) {
          tc::tmem_wait_st();
          tc::fence_before_sync();
          warp_arrive(&ctl.v_full[buf]);
          ++steps;
        }
      }
      if (dead) break;
      warp_arrive(&ctl.kv_free[b]);
    }
  } else if (warp < kCtlWarp) {
    // ============================== S warps ===============================
    regs_inc<184>();
    const int v = tid - 32 * kSWarp;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    F2 S[D / 2];  // S[k][v], k = 2 i, 2 i + 1
    int ups = 0;  // updates so far
    Pos<kStages> pos;
    for (int c = 0;; ++c, pos.next()) {
      const int b = pos.b;
      if (!warp_wait(&ctl.full[b], pos.ph)) { dead = true; break; }
      const Desc d = ctl.desc[b];
      if (d.flags & kEnd) break;
      if (d.flags & kFirst) {
        const float* src = nullptr;
        if (!kState) {
          if (d.slot >= 0)
            src = p.seg_states + (size_t)d.slot * D * D;
          else if (d.rblk != 0)
            src = reinterpret_cast<const float*>(p.layer_base + (size_t)d.rblk * p.stride) +
                  (size_t)d.h * D * D;
        }
        if (src) {
#pragma unroll
          for (int k = 0; k < D; k += 2) S[k / 2] = f2(src[(size_t)k * D + v], src[(size_t)(k + 1) * D + v]);
        } else {
#pragma unroll
          for (int k = 0; k < D / 2; ++k) S[k] = 0;
        }
      }
      if (!kState) {
        // ---- S0 as the B operand [v][k] of O = Q S0: its first bf16 term, then,
        // once that has been read, the second one in its place
        if (c > 0 && !warp_wait(&ctl.qs_full, (c - 1) & 1)) { dead = true; break; }
        auto put = [&](auto term) {
#pragma unroll
          for (int k = 0; k < D; k += 8) {
            uint4 w;
            w.x = term(S[k / 2]);
            w.y = term(S[k / 2 + 1]);
            w.z = term(S[k / 2 + 2]);
            w.w = term(S[k / 2 + 3]);
            *reinterpret_cast<uint4*>(sm + OFF_S + (k >> 6) * BOX + tc::sw128_offset(v, k & 63)) = w;
          }
          tc::fence_proxy_async_smem();
          warp_arrive(&ctl.s_ready);
        };
        put([](F2 s) { return term1(s); });
        if (!warp_wait(&ctl.s_read, c & 1)) { dead = true; break; }
        put([](F2 s) { return term2(s); });
      }
      if (!(d.flags & kNoU)) {
        const DecayPair a = decay_pair(finite_decay(p.log_decay[d.h]) * (float)d.n);
        const F2 ahi = f2(a.hi, a.hi), alo = f2(a.lo, a.lo);
        const int ub = ups & ((1 << kULog) - 1);
        if (!warp_wait(&ctl.u_full[ub], (ups >> kULog) & 1)) { dead = true; break; }
        ++ups;
        tc::fence_after_sync();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          float x[32];
          tc::tmem_ld32(tmem + tl + u_col(ub) + kb * 32, x);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            F2& s = S[kb * 16 + e];
            s = fma2(ahi, s, fma2(alo, s, f2(x[2 * e], x[2 * e + 1])));
          }
        }
        tc::fence_before_sync();
        warp_arrive(&ctl.u_free[ub]);
      }
      if (d.flags & kLast) {
        float* dst = nullptr;
        if (kState) {
          dst = p.seg_states + (size_t)d.slot * D * D;
        } else if (d.flags & kFinal) {
          // a v that is not finite has made its column of S so, in this or an
          // earlier segment: this warp's 32 columns of the chain are left to
          // the token-serial kernel
          F2 acc = 0;
#pragma unroll
          for (int k = 0; k < D / 2; ++k) acc = fma2(S[k], 0, acc);
          float x, y;
          unf2(acc, x, y);
          if (__any_sync(0xffffffffu, !(x + y == 0.f))) {
            if (lane == 0) {
              p.bad[((size_t)d.entry * p.H + d.h) * kLinSlices + (warp & 3)] = 1;
              hdr[kLinBad] = 1;
            }
          } else {
            dst = reinterpret_cast<float*>(p.layer_base + (size_t)d.wblk * p.stride) +
                  (size_t)d.h * D * D;
          }
        }
        if (dst) {
#pragma unroll
          for (int k = 0; k < D; k += 2) {
            float x, y;
            unf2(S[k / 2], x, y);
            dst[(size_t)k * D + v] = x;
            dst[(size_t)(k + 1) * D + v] = y;
          }
        }
      }
      warp_arrive(&ctl.q_free[b]);
    }
  } else {
    regs_dec<40>();
    if (warp == kCtlWarp && lane == 0) {
      // ============================== producer ==============================
      int c = 0;
      Pos<kStages> pos;
      auto load_kv = [&](unsigned char* st, int hk, int row, uint64_t* bar) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          tma_load_2d(st + ST_K + x * BOX, &tk, hk * D + x * 64, row, bar);
          tma_load_2d(st + ST_V + x * BOX, &tv, hk * D + x * 64, row, bar);
        }
      };
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
        for (int k = c0; k < c1; ++k, ++c, pos.next()) {
          const int b = pos.b;
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
          unsigned char* st = sm + b * ST_BYTES;
          // k and v over the last ones' while their outputs are still written, then
          // (all roles have read the last descriptor) q
          if (c >= kStages && !wait_for(&ctl.kv_free[b], pos.ph ^ 1)) { dead = true; break; }
          if (!kState && !end) {
            mbar_arrive_expect_tx(&ctl.full[b], 2 * TILE);
            load_kv(st, hk, d.row, &ctl.full[b]);
          }
          if (c >= kStages && !wait_for(&ctl.q_free[b], pos.ph ^ 1)) {
            dead = true;
            ++c;
            break;
          }
          ctl.desc[b] = d;
          if (end) {
            arrive(&ctl.full[b]);
            if (!kState) arrive(&ctl.full[b]);
            break;
          }
          if (kState) {
            mbar_arrive_expect_tx(&ctl.full[b], 2 * TILE);
            load_kv(st, hk, d.row, &ctl.full[b]);
          } else {
            mbar_arrive_expect_tx(&ctl.full[b], TILE);
#pragma unroll
            for (int x = 0; x < 2; ++x)
              tma_load_2d(st + ST_Q + x * BOX, &tq, h * D + x * 64, d.row, &ctl.full[b]);
          }
        }
      }
      if (dead) {
        // the loads already issued land before the CTA ends
        for (int k = c > kStages ? c - kStages : 0; k < c; ++k)
          wait_for(&ctl.full[k % kStages], (uint32_t)(k / kStages) & 1);
      }
    } else if (warp == kCtlWarp + 1 && !kState) {
      // ============================== MMA 1 =================================
      constexpr uint32_t kId = tc::idesc_bf16_f32(128, 128);
      constexpr uint32_t kIdMN = tc::idesc_bf16_f32(128, 64, false, true);
      const uint32_t s_lo = desc_k(sbase + OFF_S);
      const bool one = elect_one();
      Pos<kStages> pos;
      for (int c = 0;; ++c, pos.next()) {
        const int b = pos.b;
        const uint32_t ph = (uint32_t)(c & 1), st = sbase + b * ST_BYTES;
        if (!warp_wait(&ctl.full[b], pos.ph)) { dead = true; break; }
        if (ctl.desc[b].flags & kEnd) break;
        const uint32_t q_lo = desc_k(st + ST_Q), k_lo = desc_k(st + ST_K), v_lo = desc_mn(st + ST_V);
        // P = Q K^T, once the last chunk's P V has read P
        if (c > 0 && !warp_wait(&ctl.o_full[1], ph ^ 1)) { dead = true; break; }
        tc::fence_after_sync();
        if (one) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            tc::mma_bf16(tmem + TM_P, kDescHi | (q_lo + step_k(t)), kDescHi | (k_lo + step_k(t)), kId, t > 0);
          tc::commit(&ctl.p_full);
        }
        __syncwarp();
        // O = Q S0, of S0's two terms in turn
        if (c > 0 && !warp_wait(&ctl.o_free, ph ^ 1)) { dead = true; break; }
        for (uint32_t term = 0; term < 2; ++term) {
          if (!warp_wait(&ctl.s_ready, term)) { dead = true; break; }
          tc::fence_after_sync();
          if (one) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
              tc::mma_bf16(tmem + TM_O, kDescHi | (q_lo + step_k(t)), kDescHi | (s_lo + step_k(t)), kId,
                           t > 0 || term > 0);
            tc::commit(term == 0 ? &ctl.s_read : &ctl.qs_full);
          }
          __syncwarp();
        }
        if (dead) break;
        // O += P V, of P's two terms: 16 tokens' are 8 columns of each
        if (!warp_wait(&ctl.zeroed[b], pos.ph) || !warp_wait(&ctl.pb_full, ph) ||
            !warp_wait(&ctl.o_scaled, ph)) {
          dead = true;
          break;
        }
        tc::fence_after_sync();
        if (one) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int t = 0; t < 16; ++t)
              tc::mma_ts(tmem + TM_O + hf * 64, tmem + TM_P + (t >> 2) * 32 + (t & 3) * 8,
                         kDescHi | (v_lo + hf * (BOX >> 4) + ((t >> 2) * 2 + (t & 1)) * kStepMN), kIdMN, 1u);
            tc::commit(&ctl.o_full[hf]);
          }
          tc::commit(&ctl.kv_free[b]);
        }
        __syncwarp();
      }
    } else if (warp == kCtlWarp + 2) {
      // ============================== MMA 2 =================================
      constexpr uint32_t kIdMN = tc::idesc_bf16_f32(128, 128, false, true);
      const bool one = elect_one();
      int steps = 0, ups = 0;
      Pos<kStages> pos;
      for (int c = 0; !dead; ++c, pos.next()) {
        const int b = pos.b;
        const uint32_t k_lo = desc_mn(sbase + b * ST_BYTES + ST_K);
        if (!warp_wait(&ctl.full[b], pos.ph)) { dead = true; break; }
        const int flags = ctl.desc[b].flags, n = ctl.desc[b].n;
        if (flags & kEnd) break;
        if (flags & kNoU) {
          warp_arrive(&ctl.kv_free[b]);
          continue;
        }
        const int ub = ups & ((1 << kULog) - 1);
        if ((ups >> kULog) > 0 && !warp_wait(&ctl.u_free[ub], ((ups >> kULog) - 1) & 1)) {
          dead = true;
          break;
        }
        const int nq = (n + QT - 1) / QT;
        for (int q = 0; q < nq; ++q, ++steps) {
          const int buf = steps & ((1 << kVLog) - 1);
          if (!warp_wait(&ctl.v_full[buf], (steps >> kVLog) & 1)) { dead = true; break; }
          tc::fence_after_sync();
          // U (+)= the decayed v's terms times K over 32 tokens, the smallest first
          if (one) {
#pragma unroll
            for (int k = 0; k < 2 * kTerms; ++k)
              tc::mma_ts(tmem + u_col(ub), tmem + v_col(buf) + ((k & 1) * kTerms + kTerms - 1 - k / 2) * 8,
                         kDescHi | (k_lo + (2 * q + (k & 1)) * kStepMN), kIdMN, q > 0 || k > 0);
            tc::commit(&ctl.v_free[buf]);
          }
          __syncwarp();
        }
        if (dead) break;
        ++ups;
        if (one) {
          tc::commit(&ctl.u_full[ub]);
          tc::commit(&ctl.kv_free[b]);
        }
        __syncwarp();
      }
    } else if (warp == kCtlWarp + 3 && lane == 0 && !kState) {
      // ============================== store =================================
      Pos<kStages> pos;
      for (int c = 0;; ++c, pos.next()) {
        const int b = pos.b;
        if (!wait_for(&ctl.full[b], pos.ph)) { dead = true; break; }
        const Desc d = ctl.desc[b];
        if (d.flags & kEnd) break;
        if (!wait_for(&ctl.staged[b], pos.ph)) { dead = true; break; }
        if (d.n == CH) {
          const unsigned char* st = sm + b * ST_BYTES + ST_Q;
          tma_store_2d(&to, d.h * D, d.row, st);
          tma_store_2d(&to, d.h * D + 64, d.row, st + BOX);
          bulk_commit();
          bulk_wait_read_all();
        }
        arrive(&ctl.q_free[b]);
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

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

// Tensor map of `rows` rows of `cols` bf16 at a pitch of ld elements, in
// boxes of 64 columns x 128 rows, 128-byte swizzled, zero fill past the end.
cudaError_t rows_map(CUtensorMap* m, const void* base, int rows, long long cols, long long ld) {
  static const EncodeFn encode = [] {  // (set once, whichever threads come first)
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(fn) : nullptr;
  }();
  if (!encode) return cudaErrorNotSupported;
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
      e = launch_lin_segments(p, num_sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
