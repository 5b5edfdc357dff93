// Windowed attention for prompts: bf16, d = 64 or 128, on the tensor cores.
//
// A unit is one kv head of 2 * (128 / group) consecutive tokens of a sequence:
// two tiles, A and B, of up to 128 rows (queries of consecutive tokens, the heads
// that share the kv head next to each other), which read the same keys: the
// first tokens and the window of the first query up to the last query.  The keys
// lie in up to five runs (in the block: the sinks, and the ring in two parts; in
// the call's rows: the sinks, and the window), which are cut into segments of 16
// rows, eight to a tile of 128 keys, so that a tile is full wherever the runs
// begin and end.  With X in {A, B}, per tile of keys:
//   S_X = Q_X K^T                   (128 x 128, tensor memory)
//   P_X = 2^(scale log2 e S - m_X)  (bf16, over S), l_X += its row sums (fp32)
//   O_X += P_X V                    (128 x d, tensor memory)
// m_X is a row's maximum so far, or up to 2^8 below it: only a larger step scales
// O_X and l_X (in exact arithmetic m_X does not matter; in fp32 a weight up to
// 2^8 costs no precision either).
//
// Floor: the products, 4 d per pair of query and key (128 keys against two tiles
// 2,048 cycles; their exponentials, at the 32 a clock and SM that were measured,
// 1,024).  The two tiles alternate: the softmax of one beside the products of the
// other.  15,843 tokens x 32 heads (8 kv heads) x 128, window 1,024, the append
// with it: 201 to 203 us, 985 to 993 TFLOP/s; tensor pipe 51%, the exponentials'
// 28%: neither is full.  What is left is latency: a softmax of 128 keys takes some
// 1,500 clocks from its scores to its weights, by one thread a row, and the products
// of its tile wait for it; and some 5,000 clocks where a unit ends and the next one
// begins.
//
// One CTA per SM.  Roles:
//   softmax A, B  four warps each, a thread per row: S from tensor memory, P back
//                 to it, in the end the output
//   MMA A, B      a warp each: P V of a tile and S of the next one, in turns, so
//                 that the tiles do not fall into step: the softmax of one runs
//                 beside the products of the other (one warp for both leaves some
//                 500 cycles between them; without turns they start together, and
//                 the products wait for both softmaxes)
//   producer      one warp: TMA loads, and what the others need to know of a tile
//   check         one warp: zeros over the values behind a run's end (its last box of
//                 16 rows holds what follows in memory: other slots, another block,
//                 another sequence's tokens), and whether a value is not finite in a
//                 tile of which some row does not see all.  0 times it would reach
//                 that row; such a unit is left to the form for any shape, which runs
//                 behind this kernel over the list of them.
// P is rounded to bf16, 2^-8 relative at most, as the product's operand (its sum is
// not): outputs are off by 2.1e-3 to 2.3e-3 (2-norm), by 1.7e-3 where only they
// themselves are rounded.  A second term of P would be a third product as large as
// each of the two, and 128 more columns of tensor memory, of which none are free.
#include <cuda.h>

#include <cstddef>
#include <type_traits>

#include "gdn_lin.cuh"
#include "gdn_ptx.cuh"
#include "gdn_tc.cuh"
#include "gdn_win.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 384;  // softmax A and B (4 warps each), MMA A and B, producer, check
constexpr int kMmaWarp = 8, kLoadWarp = 10;
constexpr int kTile = 128, kSeg = 16, kSegs = kTile / kSeg;
constexpr int kRing = 16;      // descriptions of tiles
constexpr float kSlack = 8.f;  // how far m may be below the maximum (powers of two)
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // of tile A; B's 128 columns behind

// One tile of keys, as the producer describes it.
struct Tile {
  int flags, segs;
  int pos[kSegs], n[kSegs];  // first position of a segment and how many keys it has
  // the unit
  int row, pos0, tokens, hk, number;  // first packed row, its position, tokens
  int odd;                       // (check warps) a value is not finite
};
enum : int {
  kFirst = 1,   // first tile of its unit
  kLast = 2,
  kEnd = 4,     // no more tiles
  kHasB = 8,    // the unit has rows in tile B
  kPartly = 16, // some row does not see some key
  kTails = 32,  // a segment has less than 16 keys
};

// A run of keys: consecutive rows of the ring or of the call's tokens.
struct Run {
  int pos, n, row, ring;
};

template <int D>
struct TcSmem {
  static constexpr uint32_t kOperand = 128u * D * 2;  // a tile of Q, K or V: blocks of 64 columns
  static constexpr int kStages = D == 128 ? 2 : 4;    // of K and of V
  unsigned char q[2][kOperand];
  unsigned char k[kStages][kOperand], v[kStages][kOperand];
  unsigned char out[8][32 * 64];  // a softmax warp's 32 columns of output
  Tile tile[kRing];
  Run run[5];   // (producer) the unit's
  int seg0[5];  // and the first segment of each
  uint64_t described[kRing], checked[kRing], read[kRing];
  uint64_t q_full[2], q_free[2], k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
  uint64_t v_clean[kStages];  // (check warp) nothing but values of the segments' keys, and zeros
  uint64_t s_full[2], p_full[2], o_full[2], turn[2];
  uint32_t tmem;
  PlanSmem plan;
};

struct TcMaps {
  CUtensorMap q;                   // [T][H][d], boxes of a tile's rows x 64 columns
  CUtensorMap ring128, ring16;     // the layer's blocks as rows of d
  CUtensorMap k128, k16, v128, v16;  // [T][Hkv d]
};

// A bounded wait of a warp.  The first test has no suspend time, which would add
// to a wait whose phase is complete.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok != 0)) return true;
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int c0, int c1, int c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 16 consecutive tensor memory columns of this thread's lane, as they are.
__device__ __forceinline__ void tmem_ld16u(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// K-major operands advance by 32 bytes per 16 elements, blocks of 64 by 16 KB.
__host__ __device__ constexpr uint32_t step_k(int s) {
  return (uint32_t)(s >> 2) * (16384u >> 4) + (uint32_t)(s & 3) * 2u;
}

// Ring position of a role: its stage and the parity of its pass.
template <int kN>
struct Pos {
  int at = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++at == kN) {
      at = 0;
      ph ^= 1;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
win_tc_kernel(WinParams p, Pieces pieces, int32_t* left, const __grid_constant__ TcMaps maps) {
  using Smem = TcSmem<D>;
  constexpr int kStages = Smem::kStages, kBlocks = D / 64;
  constexpr uint32_t kBox = 128 * 128;  // bytes of a block of 64 columns x 128 rows
  extern __shared__ __align__(1024) unsigned char tc_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(tc_smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.described[i], 1);
      mbar_init(&sm.checked[i], 1);
      mbar_init(&sm.read[i], 8);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_free[i], 2);  // MMA A and B
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_clean[i], 1);
      mbar_init(&sm.v_free[i], 3);  // and check
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.q_full[x], 1);
      mbar_init(&sm.q_free[x], 1);
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x], 4);
      mbar_init(&sm.o_full[x], 1);
      mbar_init(&sm.turn[x], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&sm.tmem, TM_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  pdl_wait_then_release();
  const Batch& b = p.batch;
  const SeqList list = b.listed ? listed_long(b) : plan_self(b, pieces, sm.plan, p.report && blockIdx.x == 0);
  const int units = list.total * p.Hkv;
  const int tile_tokens = pieces.tokens / 2;
  const uint32_t sbase = smem_u32(tc_smem);
  const bool aligned = (sbase & 1023u) == 0;  // the operand tiles' swizzle counts on it
  bool dead = !aligned;

  // registers a thread, of 168 at launch: softmax 208, the others 88
  if (warp < 8) {
    // ============================== softmax ===============================
    regs_inc<208>();
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;  // tile, and row of it
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;      // this warp's tensor memory lanes
    const uint32_t ts = tmem + TM_S + 128u * x + lanes, to = tmem + TM_O + 128u * x + lanes;
    // (a negative scale: the product takes -Q; it is not 0, so that -inf stays -inf)
    const float to2 = fabsf(p.scale * kLog2e);
    // (a quotient by p.group of less than 128 rows: exact)
    const uint32_t over_group = (65536u + p.group - 1) / p.group;
    const int token = (int)((uint32_t)row * over_group >> 16);
    Pos<kRing> at;
    uint32_t turn = 0, unit = 0;  // parities of s_full, and of o_full
    float top = -INFINITY, sum = 0.f;
    bool odd = false;
    while (!dead) {
      if (!wait_for(&sm.described[at.at], at.ph)) { dead = true; break; }
      const Tile& tile = sm.tile[at.at];
      const int flags = tile.flags;
      if (flags & kEnd) break;
      if (x == 1 && !(flags & kHasB)) {
        warp_arrive(&sm.read[at.at]);
        at.next();
        continue;
      }
      if (flags & kFirst) {
        top = -INFINITY;
        sum = 0.f;
        odd = false;
      }
      const int pos = tile.pos0 + x * tile_tokens + token;
      if (!wait_for(&sm.s_full[x], turn)) { dead = true; break; }
      turn ^= 1;
      tc::fence_after_sync();
      if (flags & kPartly) {
        // what this row does not see: -inf in the scores' place.  (Rolled loops here, in
        // the scaling and in the output: code that runs once or twice a unit is fetched
        // anew each time, at some 6 cycles an instruction.)
#pragma unroll 1
        for (int i = 0; i < kSegs; ++i) {
          const int p0 = tile.pos[i], n = i < tile.segs ? tile.n[i] : 0;
          const int upto = min(n, max(0, pos - p0 + 1));              // not behind the row
          const int from = min(16, max(0, pos - p.window - p0 + 1));  // in the window
          const int sink = min(16, max(0, p.sinks - p0));             // or one of the first
          const uint32_t seen = ((1u << upto) - 1u) & (~((1u << from) - 1u) | ((1u << sink) - 1u));
          if (__all_sync(0xffffffffu, seen == 0xffffu)) continue;
          uint32_t w[kSeg];
          tmem_ld16u(ts + kSeg * i, w);
          tc::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < kSeg; ++k) w[k] = seen >> k & 1 ? w[k] : 0xff800000u;
          tc::tmem_st16u(ts + kSeg * i, w);
        }
        tc::tmem_wait_st();
      }
      float v[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(ts + 32 * c, v + 32 * c);
      tc::tmem_wait_ld();
      float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < 124; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = max3(m4[k], v[i + k], v[i + 4 + k]);
      const float high = fmaxf(max3(m4[0], m4[1], v[124]), max3(m4[2], m4[3], fmaxf(v[125], fmaxf(v[126], v[127])))) * to2;
      const bool more = high > top + kSlack;  // (the first one that is not -inf as well)
      if (__any_sync(0xffffffffu, more)) {
        // (a row without a larger step stays as it is: its rounding is its own)
        const float f = more ? ex2(top - high) : 1.f;
        top = more ? high : top;
        sum *= f;
        if (!(flags & kFirst)) {
          // (S_X full: all products before it are done, P V of the last tile among them)
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tc::tmem_ld32(to + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f;
            tc::tmem_st32(to + c, o);
          }
        }
      }
      const float base = top == -INFINITY ? 0.f : top;
      const F2 scale2 = f2(to2, to2), base2 = f2(-base, -base);
      F2 sum2[2] = {0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float e0, e1;
          unf2(fma2(f2(v[32 * c + i], v[32 * c + i + 1]), scale2, base2), e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          sum2[i >> 1 & 1] = add2(sum2[i >> 1 & 1], f2(e0, e1));
          w[i / 2] = tc::pack2(e0, e1, (__nv_bfloat16*)nullptr);
        }
        tc::tmem_st16u(ts + 16 * c, w);  // (over scores that are read)
      }
      float s0, s1, s2, s3;
      unf2(sum2[0], s0, s1);
      unf2(sum2[1], s2, s3);
      sum += (s0 + s1) + (s2 + s3);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      warp_arrive(&sm.p_full[x]);
      if (flags & kPartly) {
        if (!wait_for(&sm.checked[at.at], at.ph)) { dead = true; break; }
        odd |= tile.odd != 0;
      }
      if (flags & kLast) {
        const int tokens = min(tile_tokens, tile.tokens - x * tile_tokens);
        const int rows = tile_tokens * p.group;
        const int out_row = tile.row + x * tile_tokens, hk = tile.hk, number = tile.number;
        if (!wait_for(&sm.o_full[x], unit)) { dead = true; break; }
        unit ^= 1;
        tc::fence_after_sync();
        const float inv = 1.f / sum;
        // 32 columns at a time through shared memory, so that four lanes write 64 bytes
        // of a row (a lane per row writes 32 rows' 16 bytes at once: 5,000 cycles)
        unsigned char* room = sm.out[warp];
        __nv_bfloat16* dst[4];  // of rows 8 i + lane / 4 of the warp; nullptr: nothing to write
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int of = (warp & 3) * 32 + 8 * i + (lane >> 2), t = (int)((uint32_t)of * over_group >> 16);
          dst[i] = t < tokens && of < rows && !odd
                       ? static_cast<__nv_bfloat16*>(p.out) + (size_t)(out_row + t) * p.ldo +
                             (size_t)(hk * p.group + of - t * p.group) * D + 8 * (lane & 3)
                       : nullptr;
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tc::tmem_ld32(to + c, o);
          tc::tmem_wait_ld();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 y;
            y.x = tc::pack2(o[8 * i] * inv, o[8 * i + 1] * inv, (__nv_bfloat16*)nullptr);
            y.y = tc::pack2(o[8 * i + 2] * inv, o[8 * i + 3] * inv, (__nv_bfloat16*)nullptr);
            y.z = tc::pack2(o[8 * i + 4] * inv, o[8 * i + 5] * inv, (__nv_bfloat16*)nullptr);
            y.w = tc::pack2(o[8 * i + 6] * inv, o[8 * i + 7] * inv, (__nv_bfloat16*)nullptr);
            *reinterpret_cast<uint4*>(room + lane * 64 + ((i ^ (lane >> 1)) & 3) * 16) = y;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            const uint4 y = *reinterpret_cast<const uint4*>(room + r * 64 + (((lane & 3) ^ (r >> 1)) & 3) * 16);
            if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + c) = y;
          }
        }
        if (odd && tid == 0) {
          const int i = atomicAdd(&b.work.header()[kWorkHead], 1);
          if (i < kWinLeft) left[i] = number;
        }
      }
      warp_arrive(&sm.read[at.at]);
      at.next();
    }
  } else {
    regs_dec<88>();
    if (warp < kLoadWarp) {
      // ================================ MMA =================================
      // One elected lane of a warp that runs all of it issues.  (The empty asm keeps
      // the descriptors from being made ahead, all of them, and spilled.)
      constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, 128-byte swizzle
      auto desc = [](uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; };
      const uint32_t q_lo = (sbase + (uint32_t)offsetof(Smem, q)) >> 4 | 1u << 16;
      const uint32_t k_lo = (sbase + (uint32_t)offsetof(Smem, k)) >> 4 | 1u << 16;
      const uint32_t v_lo = (sbase + (uint32_t)offsetof(Smem, v)) >> 4 | (kBox >> 4) << 16;
      const bool one = elect_one();
      auto commit = [&](uint64_t* bar) {
        if (one) tc::commit(bar);
        __syncwarp();
      };
      auto role = [&](auto xc) {
        constexpr int x = decltype(xc)::value;
        Pos<kRing> at;
        Pos<kStages> ks, vs;
        uint32_t q_ph = 0, p_ph = 0, turn = 0;
        // (A begins)
        auto my_turn = [&]() {
          if (!wait_for(&sm.turn[x], x == 0 ? turn ^ 1 : turn)) dead = true;
          turn ^= 1;
        };
        auto your_turn = [&]() {
          if (lane == 0) arrive(&sm.turn[x ^ 1]);
          __syncwarp();
        };
        int flags = kEnd, segs = 0;
        auto described = [&](int& flags, int& segs) {
          if (!wait_for(&sm.described[at.at], at.ph)) {
            dead = true;
            return;
          }
          flags = __shfl_sync(0xffffffffu, sm.tile[at.at].flags, 0);
          segs = __shfl_sync(0xffffffffu, sm.tile[at.at].segs, 0);
        };
        // does this warp have rows in the unit
        auto mine = [&](int flags) { return x == 0 || (flags & kHasB) != 0; };
        // S = Q K^T of a tile (always of 128 keys: scores behind the last one are masked)
        const uint32_t id_s = tc::idesc_bf16_f32(128, 128) | (p.scale < 0.f ? 1u << 13 : 0u);  // (bit 13: -A)
        auto scores = [&]() {
          if (one) {
            uint32_t q0 = q_lo + x * (Smem::kOperand >> 4), k0 = k_lo + (uint32_t)ks.at * (Smem::kOperand >> 4);
            asm volatile("" : "+r"(q0), "+r"(k0));
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              tc::mma_bf16(tmem + TM_S + 128u * x, desc(q0 + step_k(s)), desc(k0 + step_k(s)), id_s, s > 0);
            tc::commit(&sm.s_full[x]);
          }
          __syncwarp();
        };
        // and behind them
        auto begun = [&](int flags) {
          if (one) {
            tc::commit(&sm.k_free[ks.at]);
            if (flags & kLast) tc::commit(&sm.q_free[x]);
          }
          __syncwarp();
          ks.next();
        };
        auto keys = [&](int flags) {
          if (flags & kFirst) {
            if (!wait_for(&sm.q_full[x], q_ph)) dead = true;
            q_ph ^= 1;
          }
          if (dead || !wait_for(&sm.k_full[ks.at], ks.ph)) dead = true;
        };
        // a tile without rows of this warp (not before its stages are full: one arrival
        // for each of their fills)
        auto pass = [&](uint64_t* full, uint64_t* free, uint32_t ph) {
          if (!wait_for(full, ph)) {
            dead = true;
            return;
          }
          if (lane == 0) arrive(free);
          __syncwarp();
        };
        // O += P V
        auto values = [&](int segs, bool first) {
          constexpr uint32_t id = tc::idesc_bf16_f32(128, D, false, true);
          if (one) {
            uint32_t v0 = v_lo + (uint32_t)vs.at * (Smem::kOperand >> 4);
            asm volatile("" : "+r"(v0));
#pragma unroll
            for (int s = 0; s < kSegs; ++s)
              if (s < segs)
                tc::mma_ts(tmem + TM_O + 128u * x, tmem + TM_S + 128u * x + 8u * s,
                           desc(v0 + (uint32_t)s * (2048u >> 4)), id, !first || s > 0);
          }
          __syncwarp();
        };
        // a unit's first scores: no turn, as the products of the unit before are behind
        auto begin = [&](int flags) {
          if (!mine(flags)) {
            pass(&sm.k_full[ks.at], &sm.k_free[ks.at], ks.ph);
            ks.next();
            return;
          }
          keys(flags);
          if (dead) return;
          tc::fence_after_sync();
          scores();
          begun(flags);
        };
        described(flags, segs);
        if (!dead && !(flags & kEnd)) begin(flags);
        while (!dead && !(flags & kEnd)) {
          at.next();
          int next = kEnd, next_segs = 0;
          described(next, next_segs);
          if (dead) break;
          // all that the turn needs first: within it the products follow one another
          const bool more = !(next & (kEnd | kFirst));  // (then of this unit, and of this warp's rows as well)
          if (mine(flags)) {
            if (more) keys(next);
            uint64_t* v_there = flags & kTails ? &sm.v_clean[vs.at] : &sm.v_full[vs.at];
            if (dead || !wait_for(v_there, vs.ph) || !wait_for(&sm.p_full[x], p_ph)) { dead = true; break; }
            p_ph ^= 1;
            my_turn();
            if (dead) break;
            tc::fence_after_sync();
            values(segs, (flags & kFirst) != 0);
            if (flags & kLast) commit(&sm.o_full[x]);
            if (more) scores();
            your_turn();
            commit(&sm.v_free[vs.at]);
            if (more) begun(next);
          } else {
            my_turn();
            if (!dead) your_turn();
            if (!dead) pass(&sm.v_full[vs.at], &sm.v_free[vs.at], vs.ph);
            if (!dead && more) begin(next);
            if (dead) break;
          }
          vs.next();
          if (!more && !(next & kEnd)) begin(next);
          flags = next;
          segs = next_segs;
        }
      };
      if (warp == kMmaWarp) role(std::integral_constant<int, 0>());
      else role(std::integral_constant<int, 1>());
    } else if (warp == kLoadWarp) {
      // ============================== producer ==============================
      Pos<kRing> at;
      Pos<kStages> st;
      uint32_t q_ph = 0;
      int loads = 0;
      const int total = p.sinks + p.window;
      const int rows_of = (int)(p.stride / (D * 2));  // rows of a block
      // a unit's sequence is looked up while the one before it is loaded
      int t0 = 0, row0 = 0, len = 0, past = 0, blk = 0;
      auto look_up = [&](int u) {
        const int piece = (units - 1 - u) / p.Hkv, e = entry_of(list, piece), s = list.items[e];
        t0 = (piece - list.first[e]) * pieces.tokens;
        row0 = b.cu[s];
        len = b.cu[s + 1];
        past = b.past_len[s];
        blk = b.blk[s];
      };
      // units from the last to the first (the first ones of a prompt see fewer keys than
      // the others) and, behind a CTA's first one, claimed from a counter that
      // win_append_kernel sets back: prompts of 16 Ki tokens 225 us by a fixed stride, 206 so
      auto claim = [&]() {
        int u = 0;
        if (lane == 0) u = atomicAdd(&b.work.header()[kItemHeadC], 1);
        return (int)gridDim.x + __shfl_sync(0xffffffffu, u, 0);
      };
      int next_u = blockIdx.x;
      if (next_u < units) look_up(next_u);
      while (next_u < units && !dead) {
        const int u = units - 1 - next_u, hk = u % p.Hkv;
        len -= row0;
        const int tokens = min(pieces.tokens, len - t0);
        const int p0 = past + t0, p1 = p0 + tokens;
        const bool has_b = tokens > tile_tokens;
        const int row_first_q = row0 + t0;
        // the runs of keys, in order of their positions
        const int lo = max(0, p0 - p.window + 1), before = min(p.sinks, lo);
        const int block_row = blk * rows_of + hk * total;
        __syncwarp();
        int n_segs = 0;
        {
          auto put = [&](int i, int pos, int n, int row, int ring) {
            if (lane == 0) {
              sm.run[i] = {pos, n, row, ring};
              sm.seg0[i] = n_segs;
            }
            n_segs += (n + kSeg - 1) / kSeg;
          };
          const int sinks = min(before, past), old = max(0, min(past, p1) - lo), slot = slot_of(p, lo);
          const int straight = min(old, total - slot), fresh = max(lo, past);
          put(0, 0, sinks, block_row, 1);
          put(1, sinks, before - sinks, row0 + (sinks - past), 0);
          put(2, lo, straight, block_row + slot, 1);
          put(3, lo + straight, old - straight, block_row + p.sinks, 1);
          put(4, fresh, p1 - fresh, row0 + (fresh - past), 0);
        }
        __syncwarp();
        const int n_tiles = (n_segs + kSegs - 1) / kSegs;
        for (int j = 0; j < n_tiles && !dead; ++j) {
          const int segs = min(kSegs, n_segs - j * kSegs);
          // segment lane % 8 of the tile
          const int seg = j * kSegs + (lane & 7);
          int r = 0;
#pragma unroll
          for (int i = 1; i < 5; ++i) r += seg >= sm.seg0[i];
          const Run mine = sm.run[r];
          const int in = (seg - sm.seg0[r]) * kSeg;
          const bool there = (lane & 7) < segs;
          const int pos = mine.pos + in, n = there ? min(kSeg, mine.n - in) : 0, row = mine.row + in;
          // every row sees a key that is not behind the first one and in the last one's window
          const bool all = there && n == kSeg && pos + kSeg - 1 <= p0 &&
                           (pos > p1 - 1 - p.window || pos + kSeg <= p.sinks);
          const bool full = __all_sync(0xffffffffu, all) && segs == kSegs;
          const bool tails = __any_sync(0xffffffffu, there && n < kSeg);
          // one box where all rows of the tile lie behind one another
          const int row_first = __shfl_sync(0xffffffffu, row, 0), ring_first = __shfl_sync(0xffffffffu, mine.ring, 0);
          const bool one = segs == kSegs &&
                           __all_sync(0xffffffffu, row == row_first + kSeg * (lane & 7) && mine.ring == ring_first);
          // (described kRing tiles ago, and read by all softmax warps)
          if (!wait_for(&sm.read[at.at], at.ph ^ 1)) { dead = true; break; }
          Tile& tile = sm.tile[at.at];
          if (lane < kSegs) {
            tile.pos[lane] = pos;
            tile.n[lane] = n;
          }
          if (lane == 0) {
            tile.flags = (j == 0 ? kFirst : 0) | (j == n_tiles - 1 ? kLast : 0) | (has_b ? kHasB : 0) |
                         (full ? 0 : kPartly) | (tails ? kTails : 0);
            tile.segs = segs;
            tile.row = row_first_q;
            tile.pos0 = p0;
            tile.tokens = tokens;
            tile.hk = hk;
            tile.number = u;
            tile.odd = 0;
          }
          warp_arrive(&sm.described[at.at]);
          at.next();
          if (j == 0) {
            for (int x = 0; x < (has_b ? 2 : 1); ++x) {
              // (B's turns differ from A's: each counts its own)
              const uint32_t ph = q_ph >> x & 1;
              if (!wait_for(&sm.q_free[x], ph ^ 1)) { dead = true; break; }
              q_ph ^= 1u << x;
              if (lane == 0) {
                mbar_arrive_expect_tx(&sm.q_full[x], (uint32_t)tile_tokens * p.group * D * 2);
#pragma unroll
                for (int h = 0; h < kBlocks; ++h)
                  tma_load_3d(sm.q[x] + h * kBox, &maps.q, 64 * h, hk * p.group, row_first_q + x * tile_tokens,
                              &sm.q_full[x]);
              }
              __syncwarp();
            }
            if (dead) break;
          }
          // keys, then values: a lane per segment and block, or two boxes
          for (int part = 0; part < 2; ++part) {
            uint64_t* full_bar = part ? &sm.v_full[st.at] : &sm.k_full[st.at];
            unsigned char* dst = part ? sm.v[st.at] : sm.k[st.at];
            if (!wait_for(part ? &sm.v_free[st.at] : &sm.k_free[st.at], st.ph ^ 1)) { dead = true; break; }
            if (lane == 0) mbar_arrive_expect_tx(full_bar, (uint32_t)segs * kSeg * D * 2);
            __syncwarp();
            const int shift = mine.ring && part ? p.Hkv * total : 0;  // the values' rows in a block
            const int h = one ? lane : lane >> 3;
            if (h < kBlocks && (one || there)) {
              const void* map = one ? (mine.ring ? &maps.ring128 : part ? &maps.v128 : &maps.k128)
                                    : (mine.ring ? &maps.ring16 : part ? &maps.v16 : &maps.k16);
              const int col = (mine.ring ? 0 : hk * D) + 64 * h;
              const uint32_t to = (uint32_t)h * kBox + (one ? 0u : (uint32_t)(lane & 7) * (kSeg * 128u));
              tma_load_2d(dst + to, map, col, (one ? row_first : row) + shift, full_bar);
            }
            __syncwarp();
          }
          ++loads;
          st.next();
          if (j == min(1, n_tiles - 1)) {  // (with the copies of two tiles on their way)
            next_u = claim();
            if (next_u < units) look_up(next_u);
          }
        }
      }
      if (!dead) {
        if (wait_for(&sm.read[at.at], at.ph ^ 1)) {
          if (lane == 0) sm.tile[at.at].flags = kEnd;
          warp_arrive(&sm.described[at.at]);
        } else {
          dead = true;
        }
      } else {
        // what is on its way lands before the CTA ends
        for (int i = max(0, loads - kStages); i < loads; ++i) {
          mbar_wait_bounded(&sm.k_full[i % kStages], (uint32_t)(i / kStages) & 1u);
          mbar_wait_bounded(&sm.v_full[i % kStages], (uint32_t)(i / kStages) & 1u);
        }
      }
    } else {
      // =============================== check ================================
      Pos<kRing> at;
      Pos<kStages> vs;
      while (!dead) {
        if (!wait_for(&sm.described[at.at], at.ph)) { dead = true; break; }
        Tile& tile = sm.tile[at.at];
        const int flags = tile.flags;
        if (flags & kEnd) break;
        const int n = lane < tile.segs ? tile.n[lane & 7] : kSeg;
        if (!wait_for(&sm.v_full[vs.at], vs.ph)) { dead = true; break; }
        unsigned char* values = sm.v[vs.at] + (lane & 7) * 16;  // (8 lanes a row)
        for (unsigned tails = __ballot_sync(0xffffffffu, n < kSeg); tails; tails &= tails - 1) {
          const int i = __ffs(tails) - 1;
#pragma unroll 1
          for (int r = kSeg * i + __shfl_sync(0xffffffffu, n, i) + (lane >> 3); r < kSeg * (i + 1); r += 4)
#pragma unroll
            for (int h = 0; h < kBlocks; ++h)
              *reinterpret_cast<uint4*>(values + h * kBox + r * 128) = make_uint4(0, 0, 0, 0);
        }
        if (flags & kTails) tc::fence_proxy_async_smem();
        warp_arrive(&sm.v_clean[vs.at]);
        if (flags & kPartly) {
          // 16 bytes of 4 rows at a time; 0 times a value that is not finite is NaN.  (The stage
          // is not free before this is done: with the exponents compared, five instructions
          // for two values, the prompts took 5% longer.)
          const int rows = tile.segs * kSeg;
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
#pragma unroll 4
          for (int r = lane >> 3; r < rows; r += 4)
#pragma unroll
            for (int h = 0; h < kBlocks; ++h) {
              const uint4 x4 = *reinterpret_cast<const uint4*>(values + h * kBox + r * 128);
              const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
              for (int c = 0; c < 4; ++c)
                sum[c] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[c]), zero, sum[c]);
            }
          const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
          const bool odd = !(__low2float(all) == 0.f && __high2float(all) == 0.f);
          if (__any_sync(0xffffffffu, odd) && lane == 0) tile.odd = 1;
        }
        warp_arrive(&sm.checked[at.at]);
        warp_arrive(&sm.v_free[vs.at]);
        vs.next();
        at.next();
      }
    }
  }
  if (dead && lane == 0) atomicOr((unsigned*)&b.work.header()[kErr], GDN_FLAG_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, TM_COLS);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

// Tensor map of bf16, 128-byte swizzled, zero fill past the end.
cudaError_t encode_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box) {
  static const EncodeFn encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(fn) : nullptr;
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t rows_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld,
                     int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return encode_map(m, base, 2, dims, strides, box);
}

template <int D>
cudaError_t launch_tc(const WinParams& p, const Pieces& of, int ctas, int32_t* left, cudaStream_t s) {
  TcMaps maps;
  const long long kc = (long long)p.Hkv * D, ring_rows = (long long)(p.stride / (D * 2)) * p.batch.num_blocks;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.H, (cuuint64_t)p.batch.T};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.ldq * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(of.tokens / 2)};
  cudaError_t e = encode_map(&maps.q, p.q, 3, dims, strides, box);
  if (e == cudaSuccess) e = rows_map(&maps.ring128, p.layer_base, ring_rows, D, D, kTile);
  if (e == cudaSuccess) e = rows_map(&maps.ring16, p.layer_base, ring_rows, D, D, kSeg);
  if (e == cudaSuccess) e = rows_map(&maps.k128, p.k, p.batch.T, kc, p.ldk, kTile);
  if (e == cudaSuccess) e = rows_map(&maps.k16, p.k, p.batch.T, kc, p.ldk, kSeg);
  if (e == cudaSuccess) e = rows_map(&maps.v128, p.v, p.batch.T, kc, p.ldv, kTile);
  if (e == cudaSuccess) e = rows_map(&maps.v16, p.v, p.batch.T, kc, p.ldv, kSeg);
  if (e != cudaSuccess) return e;
  auto kern = win_tc_kernel<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(TcSmem<D>));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), sizeof(TcSmem<D>), s, p, of, left, maps);
}

}  // namespace

bool win_tc_supported(int d, int act, int group) {
  return act == GDN_BF16 && (d == 64 || d == 128) && group <= kTile;
}

int win_tc_tokens(int group) { return 2 * (kTile / group); }

cudaError_t launch_win_tc(const WinParams& p, const Pieces& of, int max_pieces, int sms, void* room,
                          cudaStream_t s) {
  int32_t* left = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(room) + kWinCounterBytes);
  const long long units = (long long)max_pieces * p.Hkv;
  const int ctas = (int)(units < sms ? units : sms);
  return p.d == 64 ? launch_tc<64>(p, of, ctas, left, s) : launch_tc<128>(p, of, ctas, left, s);
}

}  // namespace gdn
