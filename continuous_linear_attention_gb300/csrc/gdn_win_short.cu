// Windowed attention for few tokens per sequence (single tokens, drafted ones,
// short prompts): bf16, d = 64 or 128, up to kMaxRows rows (tokens times query
// heads that share a kv head).
//
// Bound by HBM: a kv head's window streams in once for all of those rows.  A
// block keeps it as one contiguous run of slots, whatever the positions in them:
// the softmax does not depend on the keys' order, and slots that a row does not
// see are masked by their position.  A producer warp brings it into a ring of
// stages of 64 slots, keys and values, with bulk copies of 16 KB (d = 128), the
// new tokens as last stages, a copy per row; four consumer warps work on 16 keys
// each, or, with more than 8 rows, on a part of the rows and more keys.  What
// counts is the bytes on their way: 256 single tokens x 8 kv heads x 1,028 slots
// take 192 us (5.64 TB/s), with a consumer that issues the copies 221, with stages of 32
// slots 258, with a ring of 8 KB stages for each warp 203 (three of them) and 248
// (two).
// S^T = K Q^T and O^T += V^T P^T are m16n8k16 products (8 rows are their
// narrow side) of fragments read from shared memory as they lie: the products'
// inner index may be in any order that is the same for both sides, so a lane
// takes 16 bytes of a key's channels at once, and the output's channels in any
// order as well, so it takes 8 channels of a value at once and pairs keys in
// registers.  With 8 rows the legacy tensor instruction is at a tenth of its rate
// here, and tcgen05's least tile, 64 rows, would be mostly padding.
//
// P enters its product as two bf16 terms, exact to 2^-16, so that an output is off
// by its own rounding alone (with one term by 1.3 times that; the products have
// room for it beside the copies).
//
// Few sequences: a window is cut into parts for several CTAs; each leaves its
// maximum, sum and output, and the last one to finish joins them, in order.
#include <cuda_runtime.h>

#include <type_traits>

#include "gdn_win.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = 64;     // per stage
constexpr int kWarps = 4;     // consumers
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxRows = 8 * kWarps;

template <int D>
struct ShortSmem {
  static constexpr int kStages = 3 * (128 / D);  // 96 KB; two CTAs per SM
  __nv_bfloat16 kv[kStages][2][kKeys][D];
  float meet[kWarps][8][32];  // the warps' parts of an output, 32 columns at a time
  uint64_t full[kStages], empty[kStages];
  float top[kWarps][8], sum[kWarps][8];
  int last;
  PlanSmem plan;
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The 8 x 8 matrix of 16-bit elements whose row lane / 4 this lane has two of, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// The consumer warps' barrier.
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A unit: one kv head of one sequence, and a part of its stages.
struct Unit {
  int s, hk, part;
  int row0, len, past, blk;
  int slots;        // of the block that hold a position
  int ring_stages;  // behind them those of the new tokens
  int first, end;   // stages of this part
};

__device__ __forceinline__ Unit unit_of(const WinParams& p, const SeqList& list, const PlanSmem* plan,
                                        int u, int parts) {
  Unit w;
  w.part = u % parts;
  w.hk = u / parts % p.Hkv;
  w.s = list.items[u / (parts * p.Hkv)];
  const Batch& b = p.batch;
  w.row0 = plan ? plan->lo[w.s] : b.cu[w.s];
  w.len = (plan ? plan->lo[w.s + 1] : b.cu[w.s + 1]) - w.row0;
  w.blk = plan ? plan->blk[w.s] : b.blk[w.s];
  w.past = plan ? plan->past[w.s] : b.past_len[w.s];
  w.slots = min(w.past, p.sinks + p.window);
  w.ring_stages = (w.slots + kKeys - 1) / kKeys;
  const int all = w.ring_stages + (w.len + kKeys - 1) / kKeys;
  w.first = 0;
  w.end = all;
  if (parts > 1) {
    w.first = (int)((long long)all * w.part / parts);
    w.end = (int)((long long)all * (w.part + 1) / parts);
  }
  return w;
}

// What a CTA leaves of a part: per row its maximum (of scores in powers of
// two), sum and output, not divided.
template <int D>
__host__ __device__ constexpr size_t part_floats() {
  return (size_t)kMaxRows * (D + 2);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
win_short_kernel(WinParams p, Pieces pieces, int parts, int late, int32_t* arrived, float* left) {
  constexpr int kChunks = D / 32;  // 16-byte chunks per lane of a row of q or k
  constexpr int kHalves = D / 64;  // column halves of the output
  constexpr int kStages = ShortSmem<D>::kStages;
  extern __shared__ __align__(128) unsigned char short_smem[];
  ShortSmem<D>& sm = *reinterpret_cast<ShortSmem<D>*>(short_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
    }
    fence_mbar_init();
  }
  // late: launched behind the prompts' kernel, whose SMs it takes as they come free
  // without waiting for it (other sequences, other blocks; the inputs and the list are
  // there, as that kernel releases after its own wait); it waits before it ends.
  if (late)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else
    pdl_wait_then_release();
  const Batch& b = p.batch;
  SeqList list;
  const PlanSmem* plan = nullptr;
  if (b.listed) {
    list.items = b.work.dec();
    list.n = b.work.header()[kNDec];
  } else {
    list = plan_self(b, pieces, sm.plan, p.report && blockIdx.x == 0);
    plan = &sm.plan;
  }
  __syncthreads();
  const int units = list.n * p.Hkv * parts;
  bool dead = false;  // a wait of this warp gave up: no more waiting, the barriers are kept
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (dead || __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity))) return;
    dead = true;
    if (lane == 0) atomicOr((unsigned*)&b.work.header()[kErr], GDN_FLAG_TIMEOUT);
  };
  int slot = 0;  // the stage's place in the ring, and its round
  uint32_t phase = 0;
  auto next_stage = [&]() {
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1;
    }
  };

  if (warp == kWarps) {
    // the producer
    uint32_t fills = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit w = unit_of(p, list, plan, u, parts);
      const __nv_bfloat16* rk = ring_of<__nv_bfloat16>(p, w.blk, 0, w.hk);
      const __nv_bfloat16* rv = ring_of<__nv_bfloat16>(p, w.blk, 1, w.hk);
      for (int st = w.first; st < w.end; ++st) {
        wait(&sm.empty[slot], phase ^ 1);
        if (dead) break;
        uint64_t* full = &sm.full[slot];
        if (st < w.ring_stages) {
          if (lane == 0) {
            const uint32_t bytes = (uint32_t)min(kKeys, w.slots - st * kKeys) * D * 2;
            mbar_arrive_expect_tx(full, 2 * bytes);
            bulk_g2s(&sm.kv[slot][0][0][0], rk + (size_t)st * kKeys * D, bytes, full);
            bulk_g2s(&sm.kv[slot][1][0][0], rv + (size_t)st * kKeys * D, bytes, full);
          }
        } else {
          const int i0 = (st - w.ring_stages) * kKeys, n = min(kKeys, w.len - i0);
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)n * D * 4);
          __syncwarp();
          for (int i = lane; i < 2 * n; i += 32) {
            const int part = i & 1, r = i >> 1;
            const size_t row = w.row0 + i0 + r;
            bulk_g2s(&sm.kv[slot][part][r][0],
                     part ? static_cast<const __nv_bfloat16*>(p.v) + row * p.ldv + (size_t)w.hk * D
                          : static_cast<const __nv_bfloat16*>(p.k) + row * p.ldk + (size_t)w.hk * D,
                     D * 2, full);
          }
        }
        ++fills;
        next_stage();
      }
      if (dead) break;
    }
    // (where a wait gave up, what is on its way lands before the CTA ends)
    if (dead)
      for (uint32_t i = fills > kStages ? fills - kStages : 0; i < fills; ++i)
        mbar_wait_bounded(&sm.full[i % kStages], i / kStages & 1);
    if (late) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  // a consumer
  const int g = lane >> 2, t = lane & 3;
  const float to2 = p.scale * kLog2e;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_of(p, list, plan, u, parts);
    const int rows = w.len * p.group, tiles = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    const int mine = warp % tiles * 8;                      // this warp's first row
    const int sharing = kWarps / tiles, my = warp / tiles;  // the warps that share its keys
    // q of row g; the positions of rows 2t and 2t + 1, whose scores and outputs
    // this lane has, and of row g, whose weights it hands to the product
    auto token_of = [&](int row) { return row < rows ? row / p.group : 0; };
    uint32_t q[kChunks][4];
    int pos[2], pos_g;
    {
      const int row = mine + g, token = token_of(row);
      const int head = w.hk * p.group + (row < rows ? row - token * p.group : 0);
      pos_g = w.past + token;
#pragma unroll
      for (int r = 0; r < 2; ++r) pos[r] = w.past + token_of(mine + 2 * t + r);
      const __nv_bfloat16* src =
          static_cast<const __nv_bfloat16*>(p.q) + (size_t)(w.row0 + token) * p.ldq + (size_t)head * D;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < rows) x = *reinterpret_cast<const uint4*>(src + 32 * i + 8 * t);
        q[i][0] = x.x; q[i][1] = x.y; q[i][2] = x.z; q[i][3] = x.w;
      }
    }
    // slots that not every row sees: two runs
    const int total = p.sinks + p.window, p_last = w.past + w.len - 1;
    int m0, m1, n0, n1;
    if (w.past >= total) {  // the oldest len ones of the ring
      m0 = slot_of(p, w.past);
      m1 = m0 + min(w.len, p.window);
      n0 = p.sinks;
      n1 = p.sinks + max(0, m1 - total);
    } else {  // what is not there yet, and what the last row has left behind
      m0 = w.past;
      m1 = 0x7fffffff;
      n0 = p.sinks;
      n1 = p_last - p.window + 1;
    }
    // o[4 h + j]: channels 64 h + 8 g + 2 j (and + 1: elements 2 and 3) of rows 2t, 2t + 1
    float o[4 * kHalves][4];
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4 * kHalves; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[j][c] = 0.f;

    // 16 keys, from row k0 of the stage on; base0: the first one's index among the
    // block's slots or (fresh) the new tokens; n of them are there.  Partly: some row
    // may not see some of them.
    auto group = [&](auto partly_c, bool fresh, int k0, int base0, int n) {
      constexpr bool kPartly = decltype(partly_c)::value;
      // scores of keys g and g + 8 and rows 2t, 2t + 1, in two chains of products
      float sc[4] = {0.f, 0.f, 0.f, 0.f}, more[4] = {0.f, 0.f, 0.f, 0.f};
      const __nv_bfloat16* kr = &sm.kv[slot][0][k0 + g][8 * t];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(kr + 32 * i);
        const uint4 y = *reinterpret_cast<const uint4*>(kr + 8 * D + 32 * i);
        const uint32_t lo[4] = {x.x, y.x, x.y, y.y}, hi[4] = {x.z, y.z, x.w, y.w};
        mma16816(sc, lo, q[i][0], q[i][1]);
        mma16816(more, hi, q[i][2], q[i][3]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) sc[c] += more[c];
      // values of keys 2t, 2t + 1, 2t + 8, 2t + 9, channels 8 g .. of each half
      auto key_of = [&](int i) { return 2 * t + (i & 1) + 8 * (i >> 1); };
      auto value = [&](int i, int h) {
        return *reinterpret_cast<const uint4*>(&sm.kv[slot][1][k0 + key_of(i)][64 * h + 8 * g]);
      };
      // the position of a key that is there
      auto position = [&](int key) {
        const int sl = base0 + key;
        return fresh ? w.past + sl : sl < p.sinks ? sl : sl + (w.past - 1 - sl) / p.window * p.window;
      };
      unsigned seen = 0xfu;  // bit c: score c counts
      bool split = false;    // a value that is not finite, which not every row may see
      if constexpr (kPartly) {
        seen = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (g + 8 * k >= n) continue;
          const int j = position(g + 8 * k);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (sees(p, pos[r], j)) seen |= 1u << (2 * k + r);
        }
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (key_of(i) >= n) continue;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const uint4 x4 = value(i, h);
            const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
            // an exponent of all ones
#pragma unroll
            for (int c = 0; c < 4; ++c)
              odd |= (x[c] & 0x7f80u) == 0x7f80u || (x[c] & 0x7f800000u) == 0x7f800000u;
          }
        }
        split = __any_sync(0xffffffffu, odd);
      }
      // the softmax's next maximum
      float high[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float& x = sc[2 * k + r];
          x = !kPartly || (seen >> (2 * k + r) & 1) ? x * to2 : -INFINITY;
        }
        high[r] = fmaxf(sc[r], sc[2 + r]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], d));
      }
      if (__any_sync(0xffffffffu, high[0] > top[0] || high[1] > top[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float now = fmaxf(top[r], high[r]);
          const float f = now == -INFINITY ? 1.f : ex2(top[r] - now);
          top[r] = now;
          sum[r] *= f;
#pragma unroll
          for (int j = 0; j < 4 * kHalves; ++j) {
            o[j][r] *= f;
            o[j][2 + r] *= f;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // (nothing but -inf so far: any number in the maximum's place)
        const float base = top[r] == -INFINITY ? 0.f : top[r];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float& x = sc[2 * k + r];
          x = ex2(x - base);
          if (kPartly && !(seen >> (2 * k + r) & 1)) x = 0.f;
          sum[r] += x;
        }
      }
      // The weights as the product takes them: keys 2t .., row g; two bf16 terms each,
      // the first one cut off, so that the second is not negative, and not zero where
      // the weight is not: an infinite value stays infinite.
      auto rest = [](float x) {
        return x > 0.f ? fmaxf(x - __uint_as_float(__float_as_uint(x) & 0xffff0000u), 1.2e-38f) : x;
      };
      const uint32_t b0 = transpose8x8(__byte_perm(__float_as_uint(sc[0]), __float_as_uint(sc[1]), 0x7632));
      const uint32_t b1 = transpose8x8(__byte_perm(__float_as_uint(sc[2]), __float_as_uint(sc[3]), 0x7632));
      const uint32_t c0 = transpose8x8(pack(rest(sc[0]), rest(sc[1])));
      const uint32_t c1 = transpose8x8(pack(rest(sc[2]), rest(sc[3])));
      // one half's products; mask: the keys that count
      auto products = [&](int h, unsigned mask, auto&& each) {
        uint32_t x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 v = value(i, h);
          if (kPartly && !(mask >> i & 1)) v = make_uint4(0, 0, 0, 0);
          x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {__byte_perm(x[0][j], x[1][j], 0x5410), __byte_perm(x[0][j], x[1][j], 0x7632),
                                 __byte_perm(x[2][j], x[3][j], 0x5410), __byte_perm(x[2][j], x[3][j], 0x7632)};
          each(4 * h + j, a);
        }
      };
      if (!kPartly || !split) {
        unsigned there = 0;  // (what lies behind the last key may be anything)
        if constexpr (kPartly) {
#pragma unroll
          for (int i = 0; i < 4; ++i) there |= (key_of(i) < n ? 1u : 0u) << i;
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          products(h, there, [&](int j, const uint32_t* a) {
            mma16816(o[j], a, c0, c1);
            mma16816(o[j], a, b0, b1);
          });
      } else if constexpr (kPartly) {
        // token by token: its rows' weights alone, on the values that it sees, so that
        // what a row does not see does not reach it (0 times NaN would)
        const int lo = __reduce_min_sync(0xffffffffu, pos_g), hi = __reduce_max_sync(0xffffffffu, pos_g);
#pragma unroll 1
        for (int at = lo; at <= hi; ++at) {
          unsigned mask = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key_of(i) < n && sees(p, at, position(key_of(i)))) mask |= 1u << i;
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            products(h, mask, [&](int j, const uint32_t* a) {
              float c[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(c, a, pos_g == at ? c0 : 0u, pos_g == at ? c1 : 0u);
              mma16816(c, a, pos_g == at ? b0 : 0u, pos_g == at ? b1 : 0u);
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (pos[r] == at) {
                  o[j][r] += c[r];
                  o[j][2 + r] += c[2 + r];
                }
            });
        }
      }
    };
    for (int st = w.first; st < w.end; ++st) {
      const bool fresh = st >= w.ring_stages;
      const int first = (fresh ? st - w.ring_stages : st) * kKeys;
      const int n = min(kKeys, (fresh ? w.len : w.slots) - first);
      wait(&sm.full[slot], phase);
      for (int k0 = my * 16; k0 < n; k0 += 16 * sharing) {
        const int base0 = first + k0;
        if (fresh || n - k0 < 16 || (base0 < m1 && base0 + 16 > m0) || (base0 < n1 && base0 + 16 > n0))
          group(std::true_type(), fresh, k0, base0, n - k0);
        else
          group(std::false_type(), false, k0, base0, 16);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[slot]);
      next_stage();
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
      if (g == 0) {
        sm.top[warp][2 * t + r] = top[r];
        sm.sum[warp][2 * t + r] = sum[r];
      }
    }
    const int unit = u / parts;  // whose parts meet
    float* mine_left = left + (size_t)u * part_floats<D>();
    // (a half's 64 channels in two rounds: those of lanes g < 4, then the others')
#pragma unroll
    for (int h = 0; h < D / 32; ++h) {
      if (g >> 2 == (h & 1)) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 4; j += 2)
            *reinterpret_cast<float4*>(&sm.meet[warp][2 * t + r][8 * (g & 3) + 2 * j]) =
                make_float4(o[h / 2 * 4 + j][r], o[h / 2 * 4 + j][2 + r], o[h / 2 * 4 + j + 1][r],
                            o[h / 2 * 4 + j + 1][2 + r]);
      }
      consumer_sync();
      // four columns of a row at a time
      for (int i = tid; i < rows * 8; i += 32 * kWarps) {
        const int row = i / 8, c = i % 8 * 4, tile = row / 8, r = row % 8;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < sharing; ++k) m = fmaxf(m, sm.top[tile + k * tiles][r]);
        const float base = m == -INFINITY ? 0.f : m;
        for (int k = 0; k < sharing; ++k) {
          const int wk = tile + k * tiles;
          const float f = ex2(sm.top[wk][r] - base);
          const float4 x = *reinterpret_cast<const float4*>(&sm.meet[wk][r][c]);
          l = fmaf(sm.sum[wk][r], f, l);
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
        if (parts == 1) {
          const int token = row / p.group, head = w.hk * p.group + row % p.group;
          const float inv = 1.f / l;
          const uint2 y = make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)(w.row0 + token) * p.ldo +
                                    (size_t)head * D + 32 * h + c) = y;
        } else {
          *reinterpret_cast<float4*>(mine_left + (size_t)row * D + 32 * h + c) = acc;
          if (h == 0 && c == 0) {
            mine_left[(size_t)kMaxRows * D + 2 * row] = m;
            mine_left[(size_t)kMaxRows * D + 2 * row + 1] = l;
          }
        }
      }
      consumer_sync();  // the room is free again, and (the last time) all stages are read
    }
    bool last = true;
    if (parts > 1) {
      __threadfence();
      consumer_sync();
      if (tid == 0) {
        sm.last = atomicAdd(&arrived[unit], 1) == parts - 1;
        if (sm.last) arrived[unit] = 0;  // for the next call
        __threadfence();
      }
      consumer_sync();
      last = sm.last;
    }
    if (!last) continue;
    if (parts > 1) {
      const float* all = left + (size_t)unit * parts * part_floats<D>();
      for (int i = tid; i < rows * (D / 4); i += 32 * kWarps) {
        const int row = i / (D / 4), c = i % (D / 4) * 4;
        float m = -INFINITY, l = 0.f;
#pragma unroll 8
        for (int k = 0; k < parts; ++k)
          m = fmaxf(m, __ldcg(all + k * part_floats<D>() + (size_t)kMaxRows * D + 2 * row));
        const float base = m == -INFINITY ? 0.f : m;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < parts; ++k) {
          const float* from = all + k * part_floats<D>();
          const float f = ex2(__ldcg(from + (size_t)kMaxRows * D + 2 * row) - base);
          const float4 x = __ldcg(reinterpret_cast<const float4*>(from + (size_t)row * D + c));
          l = fmaf(__ldcg(from + (size_t)kMaxRows * D + 2 * row + 1), f, l);
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
        const int token = row / p.group, head = w.hk * p.group + row % p.group;
        const float inv = 1.f / l;
        uint2 y = make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)(w.row0 + token) * p.ldo +
                                  (size_t)head * D + c) = y;
      }
    }
    // the new keys and values into the block: all of this kv head's window has been read
    for (int i = tid; i < 2 * w.len * (D / 8); i += 32 * kWarps) {
      const int part = i / (w.len * (D / 8)), x = i % (w.len * (D / 8)), tok = x / (D / 8), c = x % (D / 8) * 8;
      const int j = w.past + tok;
      if (j >= p.sinks && tok < w.len - p.window) continue;  // out of every later window
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(part ? p.v : p.k) +
                                 (size_t)(w.row0 + tok) * (part ? p.ldv : p.ldk) + (size_t)w.hk * D + c;
      *reinterpret_cast<uint4*>(ring_of<__nv_bfloat16>(p, w.blk, part, w.hk) + (size_t)slot_of(p, j) * D + c) =
          *reinterpret_cast<const uint4*>(src);
    }
  }
  if (late) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D>
cudaError_t launch_short(const WinParams& p, const Pieces& of, int parts, int ctas, bool late, void* room,
                         cudaStream_t s) {
  auto kern = win_short_kernel<D>;
  const size_t smem = sizeof(ShortSmem<D>);
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int32_t* arrived = static_cast<int32_t*>(room);
  float* left = reinterpret_cast<float*>(static_cast<unsigned char*>(room) + kWinCounterBytes + kWinListBytes);
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, s, p, of, parts, (int)late, arrived, left);
}

}  // namespace

bool win_short_supported(int d, int act) { return act == GDN_BF16 && (d == 64 || d == 128); }

int win_short_tokens(int group) { return group <= kMaxRows ? kMaxRows / group : 0; }

size_t win_short_room(int sms, int d) {
  return kWinCounterBytes + kWinListBytes + (size_t)2 * sms * (d == 64 ? part_floats<64>() : part_floats<128>()) * sizeof(float);
}

cudaError_t launch_win_short(const WinParams& p, const Pieces& of, int max_items, int sms, bool late,
                             void* room, cudaStream_t s) {
  // Where the kv heads of all sequences leave CTAs idle, their windows are cut into
  // parts of two stages at least.
  const long long heads = (long long)max_items * p.Hkv;
  const int stages = (p.sinks + p.window + kKeys - 1) / kKeys + 1, side = 2 * sms;
  int parts = 1;
  if (heads > 0 && heads < side && heads * sizeof(int32_t) <= kWinCounterBytes) parts = (int)(side / heads);
  if (parts > (stages + 1) / 2) parts = (stages + 1) / 2;
  const long long units = heads * parts;
  const int ctas = (int)(units < side ? (units > 0 ? units : 1) : side);
  return p.d == 64 ? launch_short<64>(p, of, parts, ctas, late, room, s)
                   : launch_short<128>(p, of, parts, ctas, late, room, s);
}

}  // namespace gdn
