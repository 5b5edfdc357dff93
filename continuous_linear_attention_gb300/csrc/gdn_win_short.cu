// Windowed attention for few tokens per sequence (single tokens, drafted ones,
// short prompts): bf16, d = 64 or 128, up to kMaxRows rows (tokens times query
// heads that share a kv head).
//
// Bound by HBM: a kv head's window streams in once for all of those rows.  A
// block keeps it as one contiguous run of slots, cut into groups of 16,
// whatever the positions in them: the softmax does not depend on the keys'
// order, and slots that a row does not see are masked by their position.  The
// new tokens come as last groups.  Each of a CTA's four warps works on groups of
// its own, with a ring of stages of its own that it fills itself with bulk
// copies: no warp waits for another before the end of a unit (a ring that the
// warps share takes 221 us for 256 single tokens x 8 kv heads x 1,028 slots, and
// 361 with a warp for the copies alone, whose share of the registers makes the
// others spill; this form TIME_256).  With more than 16 rows the warps take
// different rows, and a group is read by several of them, out of L2.
// S = Q K^T and O += P V are m16n8k16 products of fragments read from shared
// memory as they lie: the products' inner index may be in any order that is the
// same for both sides, so a lane takes 16 bytes of a key's channels at once, and
// the output's columns in any order as well, so it takes 8 channels of a value at
// once and pairs keys in registers.  At m = 16 the legacy tensor instruction is at
// a tenth of its rate here, and tcgen05's least tile, 64 rows, would be mostly
// padding.
//
// P is rounded to bf16 as the product's operand (its sum is not): an output's
// error is 2^-9 / sqrt(3) relative to the root of the sum of its squared terms, on top
// of its own rounding by about as much.
//
// Few sequences: a window is cut into parts for several CTAs; each leaves its
// maximum, sum and output, and the last one to finish joins them, in order.
#include <cuda_runtime.h>

#include <type_traits>

#include "gdn_win.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = 16;     // per group
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxRows = 16 * kWarps;

template <int D>
struct ShortSmem {
  static constexpr int kStages = D == 64 ? 6 : 3;  // 24 KB per warp; two CTAs per SM
  __nv_bfloat16 kv[kWarps][kStages][2][kKeys][D];
  float meet[kWarps][16][32];  // the warps' parts of an output, 32 columns at a time
  uint64_t full[kWarps][kStages];
  float top[kWarps][16], sum[kWarps][16];
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
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// A unit: one kv head of one sequence, and a part of its groups of keys.
struct Unit {
  int s, hk, part;
  int row0, len, past, blk;
  int slots;        // of the block that hold a position
  int ring_groups;  // behind them those of the new tokens
  int first, end;   // groups of this part
  int tiles;        // of 16 rows
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
  w.past = b.past_len[w.s];
  w.slots = min(w.past, p.sinks + p.window);
  w.ring_groups = (w.slots + kKeys - 1) / kKeys;
  const int all = w.ring_groups + (w.len + kKeys - 1) / kKeys;
  w.first = (int)((long long)all * w.part / parts);
  w.end = (int)((long long)all * (w.part + 1) / parts);
  const int rows = w.len * p.group;
  w.tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
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
win_short_kernel(WinParams p, Pieces pieces, int parts, int32_t* arrived, float* left) {
  constexpr int kChunks = D / 32;  // 16-byte chunks per lane of a row of q or k
  constexpr int kHalves = D / 64;  // column halves of the output
  constexpr int kStages = ShortSmem<D>::kStages;
  extern __shared__ __align__(128) unsigned char short_smem[];
  ShortSmem<D>& sm = *reinterpret_cast<ShortSmem<D>*>(short_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kWarps * kStages) {
    mbar_init(&sm.full[0][0] + tid, 1);
    fence_mbar_init();
  }
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
  auto& ring = sm.kv[warp];

  // This warp's groups are on their way kStages ahead, across the units' borders.
  uint32_t fill = 0, take = 0, fill_slot = 0, slot = 0, phase = 0;
  int fill_u = blockIdx.x, fill_g = 0;
  Unit fw;
  fw.end = 0;
  auto fill_unit = [&]() {
    if (fill_u >= units) return;
    fw = unit_of(p, list, plan, fill_u, parts);
    fill_g = fw.first + warp / fw.tiles;
  };
  fill_unit();
  auto bring = [&]() {
    while (fill < take + kStages && fill_u < units) {
      if (fill_g >= fw.end) {
        fill_u += gridDim.x;
        fill_unit();
        continue;
      }
      if (!dead) {
        uint64_t* full = &sm.full[warp][fill_slot];
        if (fill_g < fw.ring_groups) {
          if (lane == 0) {
            const uint32_t bytes = (uint32_t)min(kKeys, fw.slots - fill_g * kKeys) * D * 2;
            mbar_arrive_expect_tx(full, 2 * bytes);
            bulk_g2s(&ring[fill_slot][0][0][0],
                     ring_of<__nv_bfloat16>(p, fw.blk, 0, fw.hk) + (size_t)fill_g * kKeys * D, bytes, full);
            bulk_g2s(&ring[fill_slot][1][0][0],
                     ring_of<__nv_bfloat16>(p, fw.blk, 1, fw.hk) + (size_t)fill_g * kKeys * D, bytes, full);
          }
        } else {
          // a copy per row
          const int i0 = (fill_g - fw.ring_groups) * kKeys, n = min(kKeys, fw.len - i0);
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)n * D * 4);
          __syncwarp();
          const int part = lane >> 4, i = lane & 15;
          const size_t row = fw.row0 + i0 + i;
          if (i < n)
            bulk_g2s(&ring[fill_slot][part][i][0],
                     part ? static_cast<const __nv_bfloat16*>(p.v) + row * p.ldv + (size_t)fw.hk * D
                          : static_cast<const __nv_bfloat16*>(p.k) + row * p.ldk + (size_t)fw.hk * D,
                     D * 2, full);
        }
      }
      ++fill;
      if (++fill_slot == kStages) fill_slot = 0;
      fill_g += kWarps / fw.tiles;
    }
  };
  bring();

  const int g = lane >> 2, t = lane & 3;
  const float to2 = p.scale * kLog2e;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_of(p, list, plan, u, parts);
    const int rows = w.len * p.group, tiles = w.tiles;
    const int mine = warp % tiles;  // this warp's tile of 16 rows
    const int sharing = kWarps / tiles;  // warps that work on its keys
    // rows g and g + 8 of the tile: their tokens and q
    uint32_t q[kChunks][2][4];
    int pos[2];
    bool live[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = mine * 16 + g + 8 * r;
      live[r] = row < rows;
      const int token = live[r] ? row / p.group : 0, head = w.hk * p.group + (live[r] ? row % p.group : 0);
      pos[r] = w.past + token;
      const __nv_bfloat16* src =
          static_cast<const __nv_bfloat16*>(p.q) + (size_t)(w.row0 + token) * p.ldq + (size_t)head * D;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live[r]) x = *reinterpret_cast<const uint4*>(src + 32 * i + 8 * t);
        q[i][r][0] = x.x; q[i][r][1] = x.y; q[i][r][2] = x.z; q[i][r][3] = x.w;
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
    float o[kHalves][8][4];
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[h][j][c] = 0.f;

    int gr = w.first + warp / tiles;
    // A group's keys.  partly: some row may not see some of them.
    auto group = [&](auto partly_c, bool fresh, int base0, int n) {
      constexpr bool kPartly = decltype(partly_c)::value;
      // scores of 16 keys
      float sc[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[h][c] = 0.f;
        const __nv_bfloat16* kr = &ring[slot][0][8 * h + g][8 * t];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(kr + 32 * i);
          const uint32_t lo[4] = {q[i][0][0], q[i][1][0], q[i][0][1], q[i][1][1]};
          const uint32_t hi[4] = {q[i][0][2], q[i][1][2], q[i][0][3], q[i][1][3]};
          mma16816(sc[h], lo, x.x, x.y);
          mma16816(sc[h], hi, x.z, x.w);
        }
      }
      // this lane's keys' values: 2t, 2t+1, 2t+8, 2t+9, channels 8g .. of each half
      auto key_of = [&](int i) { return 2 * t + (i & 1) + 8 * (i >> 1); };
      auto value = [&](int i, int h) {
        return *reinterpret_cast<const uint4*>(&ring[slot][1][key_of(i)][64 * h + 8 * g]);
      };
      // position of key i (only of one that is there)
      auto position = [&](int i) {
        const int sl = base0 + key_of(i);
        return fresh ? w.past + sl : sl < p.sinks ? sl : sl + (w.past - 1 - sl) / p.window * p.window;
      };
      unsigned seen = 0xffu;  // bit 2 i + r: row r sees key i
      bool split = false;     // a value that is not finite, which not every row sees
      if constexpr (kPartly) {
        seen = 0;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (key_of(i) >= n) continue;
          const int j = position(i);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (sees(p, pos[r], j)) seen |= 1u << (2 * i + r);
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
      float high[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float& x = sc[i >> 1][2 * r + (i & 1)];
          x = !kPartly || (seen >> (2 * i + r) & 1) ? x * to2 : -INFINITY;
          high[r] = fmaxf(high[r], x);
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 1));
        high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 2));
      }
      if (__any_sync(0xffffffffu, high[0] > top[0] || high[1] > top[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float now = fmaxf(top[r], high[r]);
          const float f = now == -INFINITY ? 1.f : ex2(top[r] - now);
          top[r] = now;
          sum[r] *= f;
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[h][j][2 * r] *= f;
              o[h][j][2 * r + 1] *= f;
            }
        }
      }
      float wt[4][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = top[r] == -INFINITY ? 0.f : top[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = ex2(sc[i >> 1][2 * r + (i & 1)] - base);
          wt[i][r] = !kPartly || (seen >> (2 * i + r) & 1) ? e : 0.f;
          sum[r] += wt[i][r];
        }
      }
      const uint32_t a[4] = {pack(wt[0][0], wt[1][0]), pack(wt[0][1], wt[1][1]),
                             pack(wt[2][0], wt[3][0]), pack(wt[2][1], wt[3][1])};
      if (!kPartly || !split) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          uint32_t x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 v = value(i, h);
            // (what lies behind the last key may be anything)
            if (kPartly && key_of(i) >= n) v = make_uint4(0, 0, 0, 0);
            x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t pick = j & 1 ? 0x7632u : 0x5410u;
            mma16816(o[h][j], a, __byte_perm(x[0][j >> 1], x[1][j >> 1], pick),
                     __byte_perm(x[2][j >> 1], x[3][j >> 1], pick));
          }
        }
      } else {
        // token by token: its rows' weights alone, on the values that it sees, so that
        // what a row does not see does not reach it (0 times NaN would)
        const int lo = __reduce_min_sync(0xffffffffu, live[0] ? pos[0] : 0x7fffffff);
        const int hi = __reduce_max_sync(0xffffffffu, max(live[0] ? pos[0] : 0, live[1] ? pos[1] : 0));
#pragma unroll 1
        for (int at = lo; at <= hi; ++at) {
          unsigned mask = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key_of(i) < n && sees(p, at, position(i))) mask |= 1u << i;
          const uint32_t at4[4] = {pos[0] == at ? a[0] : 0u, pos[1] == at ? a[1] : 0u,
                                   pos[0] == at ? a[2] : 0u, pos[1] == at ? a[3] : 0u};
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            uint32_t x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 v = value(i, h);
              if (!(mask >> i & 1)) v = make_uint4(0, 0, 0, 0);
              x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t pick = j & 1 ? 0x7632u : 0x5410u;
              float c[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(c, at4, __byte_perm(x[0][j >> 1], x[1][j >> 1], pick),
                       __byte_perm(x[2][j >> 1], x[3][j >> 1], pick));
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (pos[r] == at) {
                  o[h][j][2 * r] += c[2 * r];
                  o[h][j][2 * r + 1] += c[2 * r + 1];
                }
            }
          }
        }
      }
    };
    for (; gr < w.end; gr += sharing) {
      const bool fresh = gr >= w.ring_groups;
      // the group's first key, among the block's slots or the new tokens
      const int base0 = (fresh ? gr - w.ring_groups : gr) * kKeys;
      const int n = min(kKeys, (fresh ? w.len : w.slots) - base0);
      wait(&sm.full[warp][slot], phase);
      if (fresh || n < kKeys || (base0 < m1 && base0 + 16 > m0) || (base0 < n1 && base0 + 16 > n0))
        group(std::true_type(), fresh, base0, n);
      else
        group(std::false_type(), false, base0, n);
      __syncwarp();  // the stage is read: bring() may fill it
      ++take;
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
      bring();
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    }
    if (t == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sm.top[warp][g + 8 * r] = top[r];
        sm.sum[warp][g + 8 * r] = sum[r];
      }
    }
    const int unit = u / parts;  // whose parts meet
    float* mine_left = left + (size_t)u * part_floats<D>();
    // (this lane's columns of a half are 16 t .. + 15: lanes 0 and 1, then 2 and 3, put theirs down)
#pragma unroll
    for (int h = 0; h < D / 32; ++h) {
      if (t >> 1 == (h & 1)) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; j += 4)
              *reinterpret_cast<float4*>(&sm.meet[warp][g + 8 * r][16 * (t & 1) + 8 * c + j]) =
                  make_float4(o[h / 2][j][2 * r + c], o[h / 2][j + 1][2 * r + c],
                              o[h / 2][j + 2][2 * r + c], o[h / 2][j + 3][2 * r + c]);
      }
      __syncthreads();
      // four columns of a row at a time
      for (int i = tid; i < rows * 8; i += kThreads) {
        const int row = i / 8, c = i % 8 * 4, tile = row >> 4, r = row & 15;
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
      __syncthreads();  // the room is free again, and (the last time) all groups are read
    }
    bool last = true;
    if (parts > 1) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        sm.last = atomicAdd(&arrived[unit], 1) == parts - 1;
        if (sm.last) arrived[unit] = 0;  // for the next call
        __threadfence();
      }
      __syncthreads();
      last = sm.last;
    }
    if (!last) continue;
    if (parts > 1) {
      const float* all = left + (size_t)unit * parts * part_floats<D>();
      for (int i = tid; i < rows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), c = i % (D / 4) * 4;
        float m = -INFINITY, l = 0.f;
        for (int k = 0; k < parts; ++k)
          m = fmaxf(m, __ldcg(all + k * part_floats<D>() + (size_t)kMaxRows * D + 2 * row));
        const float base = m == -INFINITY ? 0.f : m;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
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
    for (int i = tid; i < 2 * w.len * (D / 8); i += kThreads) {
      const int part = i / (w.len * (D / 8)), x = i % (w.len * (D / 8)), tok = x / (D / 8), c = x % (D / 8) * 8;
      const int j = w.past + tok;
      if (j >= p.sinks && tok < w.len - p.window) continue;  // out of every later window
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(part ? p.v : p.k) +
                                 (size_t)(w.row0 + tok) * (part ? p.ldv : p.ldk) + (size_t)w.hk * D + c;
      *reinterpret_cast<uint4*>(ring_of<__nv_bfloat16>(p, w.blk, part, w.hk) + (size_t)slot_of(p, j) * D + c) =
          *reinterpret_cast<const uint4*>(src);
    }
  }  // (where a wait gave up, what is on its way lands before the CTA ends)
  if (dead)
    for (uint32_t i = fill > kStages ? fill - kStages : 0; i < fill; ++i)
      mbar_wait_bounded(&sm.full[warp][i % kStages], i / kStages & 1);
}

template <int D>
cudaError_t launch_short(const WinParams& p, const Pieces& of, int parts, int ctas, void* room,
                         cudaStream_t s) {
  auto kern = win_short_kernel<D>;
  const size_t smem = sizeof(ShortSmem<D>);
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int32_t* arrived = static_cast<int32_t*>(room);
  float* left = reinterpret_cast<float*>(static_cast<unsigned char*>(room) + kWinCounterBytes);
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, s, p, of, parts, arrived, left);
}

}  // namespace

bool win_short_supported(int d, int act) { return act == GDN_BF16 && (d == 64 || d == 128); }

int win_short_tokens(int group) { return group <= kMaxRows ? kMaxRows / group : 0; }

size_t win_short_room(int sms, int d) {
  return kWinCounterBytes + (size_t)2 * sms * (d == 64 ? part_floats<64>() : part_floats<128>()) * sizeof(float);
}

cudaError_t launch_win_short(const WinParams& p, const Pieces& of, int max_items, int sms, void* room,
                             cudaStream_t s) {
  // Where the kv heads of all sequences leave CTAs idle, their windows are cut into
  // parts of two groups per warp at least.
  const long long heads = (long long)max_items * p.Hkv;
  const int groups = (p.sinks + p.window + kKeys - 1) / kKeys + 1;
  int parts = heads > 0 && heads < 2 * sms && heads * sizeof(int32_t) <= kWinCounterBytes ? (int)(2 * sms / heads) : 1;
  if (parts > (groups + 7) / 8) parts = (groups + 7) / 8;
  const long long units = heads * parts;
  const int ctas = (int)(units < 2 * sms ? (units > 0 ? units : 1) : 2 * sms);
  return p.d == 64 ? launch_short<64>(p, of, parts, ctas, room, s)
                   : launch_short<128>(p, of, parts, ctas, room, s);
}

}  // namespace gdn
