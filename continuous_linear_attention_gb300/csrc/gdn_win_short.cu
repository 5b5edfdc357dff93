// Windowed attention for few tokens per sequence (single tokens, drafted ones,
// short prompts): bf16, d = 64 or 128, up to kMaxRows rows (tokens times query
// heads that share a kv head).
//
// Bound by HBM: a kv head's window streams in once for all of those rows.  A
// block keeps it as one contiguous run of slots, so bulk copies bring it into a
// ring of stages, kKeys slots of keys and values at a
// time, whatever the positions in them: the softmax does not depend on the
// keys' order, and slots that a row does not see are masked by their position.
// The new tokens come as a last stage, a copy per row.  Four warps work on
// 16 keys each (or, with more than 16 rows, on a part of the rows and
// more keys): S = Q K^T and O += P V as m16n8k16 products of fragments read
// from shared memory as they lie: the products' inner index may be in any order
// that is the same for both sides, so a lane takes 16 consecutive channels'
// bytes of a key at once, and the output's columns in any order as well, so it
// takes 8 channels of a value at once and pairs keys in registers.  At m = 16
// the legacy tensor instruction is at a tenth of its rate here, and tcgen05's
// least tile, 64 rows, would be mostly padding.
//
// P is rounded to bf16 as the product's operand (its sum is not): an output's
// error is 2^-9 / sqrt(3) relative to the root of the sum of its squared terms, on top
// of its own rounding by about as much.
//
// Few sequences: a window is cut into parts for several CTAs; each leaves its
// maximum, sum and output, and the last one to finish joins them, in order.
#include <cuda_runtime.h>

#include "gdn_win.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = 64;     // per stage
constexpr int kStages = 3;    // per CTA, two CTAs per SM
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxRows = 16 * kWarps;

template <int D>
struct ShortSmem {
  __nv_bfloat16 kv[kStages][2][kKeys][D];
  uint64_t full[kStages], empty[kStages];
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
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A unit: one kv head of one sequence, and a part of its stages.
struct Unit {
  int s, hk, part;
  int row0, len, past, blk;
  int slots;          // of the block that hold a position
  int first, end;     // stages of this part (the last of all is the new tokens)
  int ring_stages;
};

__device__ __forceinline__ Unit unit_of(const WinParams& p, const SeqList& list, int u, int parts) {
  Unit w;
  w.part = u % parts;
  w.hk = u / parts % p.Hkv;
  w.s = list.items[u / (parts * p.Hkv)];
  const Batch& b = p.batch;
  w.row0 = b.cu[w.s];
  w.len = b.cu[w.s + 1] - w.row0;
  w.past = b.past_len[w.s];
  w.blk = b.blk[w.s];
  w.slots = min(w.past, p.sinks + p.window);
  w.ring_stages = (w.slots + kKeys - 1) / kKeys;
  const int all = w.ring_stages + 1;
  w.first = (int)((long long)all * w.part / parts);
  w.end = (int)((long long)all * (w.part + 1) / parts);
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
  pdl_wait_then_release();
  const Batch& b = p.batch;
  SeqList list;
  if (b.listed) {
    list.items = b.work.dec();
    list.n = b.work.header()[kNDec];
    __syncthreads();
  } else {
    list = plan_self(b, pieces, sm.plan, p.report && blockIdx.x == 0);
    __syncthreads();
  }
  const int units = list.n * p.Hkv * parts;
  bool dead = false;  // a wait of this warp gave up: no more waiting, the barriers are kept
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (dead || __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity))) return;
    dead = true;
    if (lane == 0) atomicOr((unsigned*)&b.work.header()[kErr], GDN_FLAG_TIMEOUT);
  };

  // Warp 0 brings the stages in: all of the first ones, and, whenever it has
  // done with a stage, the one that takes the place of the stage before that (the
  // other warps have left it long ago).  A dedicated warp would cost more: its
  // share of the registers makes the others spill (361 us for 256 single tokens
  // x 8 kv heads x 1,028 slots; TIME_256 like this).
  uint32_t fill = 0;
  int fill_u = blockIdx.x, fill_st = 0;
  Unit fw;
  if (warp == 0 && fill_u < units) {
    fw = unit_of(p, list, fill_u, parts);
    fill_st = fw.first;
  }
  auto bring = [&](uint32_t upto) {
    while (fill < upto && fill_u < units) {
      if (fill_st >= fw.end) {
        fill_u += gridDim.x;
        if (fill_u >= units) return;
        fw = unit_of(p, list, fill_u, parts);
        fill_st = fw.first;
        continue;
      }
      const int slot = fill % kStages, st = fill_st;
      wait(&sm.empty[slot], (fill / kStages & 1) ^ 1);
      if (!dead) {
        if (st < fw.ring_stages) {
          if (lane == 0) {
            const uint32_t bytes = (uint32_t)min(kKeys, fw.slots - st * kKeys) * D * 2;
            mbar_arrive_expect_tx(&sm.full[slot], 2 * bytes);
            bulk_g2s(&sm.kv[slot][0][0][0],
                     ring_of<__nv_bfloat16>(p, fw.blk, 0, fw.hk) + (size_t)st * kKeys * D, bytes,
                     &sm.full[slot]);
            bulk_g2s(&sm.kv[slot][1][0][0],
                     ring_of<__nv_bfloat16>(p, fw.blk, 1, fw.hk) + (size_t)st * kKeys * D, bytes,
                     &sm.full[slot]);
          }
        } else {
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], (uint32_t)fw.len * D * 4);
          __syncwarp();
          for (int i = lane; i < fw.len; i += 32) {
            const size_t row = fw.row0 + i;
            bulk_g2s(&sm.kv[slot][0][i][0],
                     static_cast<const __nv_bfloat16*>(p.k) + row * p.ldk + (size_t)fw.hk * D, D * 2,
                     &sm.full[slot]);
            bulk_g2s(&sm.kv[slot][1][i][0],
                     static_cast<const __nv_bfloat16*>(p.v) + row * p.ldv + (size_t)fw.hk * D, D * 2,
                     &sm.full[slot]);
          }
        }
      }
      ++fill;
      ++fill_st;
    }
  };
  if (warp == 0) bring(kStages);

  const int g = lane >> 2, t = lane & 3;
  const float to2 = p.scale * kLog2e;
  uint32_t take = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_of(p, list, u, parts);
    const int rows = w.len * p.group;
    const int tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    const int mine = warp % tiles;                        // this warp's tile of 16 rows
    const int sharing = kWarps / tiles, my = warp / tiles;  // the warps that share its keys
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

    for (int st = w.first; st < w.end; ++st, ++take) {
      const int slot = take % kStages;
      const bool fresh = st == w.ring_stages;
      const int n = fresh ? w.len : min(kKeys, w.slots - st * kKeys);
      wait(&sm.full[slot], take / kStages & 1);
      for (int k0 = my * 16; k0 < n; k0 += 16 * sharing) {
        // scores of 16 keys
        float sc[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[h][c] = 0.f;
          const __nv_bfloat16* kr = &sm.kv[slot][0][k0 + 8 * h + g][8 * t];
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
        auto key_of = [&](int i) { return k0 + 2 * t + (i & 1) + 8 * (i >> 1); };
        auto value = [&](int i, int h) {
          return *reinterpret_cast<const uint4*>(&sm.kv[slot][1][key_of(i)][64 * h + 8 * g]);
        };
        // position of key i (only of one that is there)
        auto position = [&](int i) {
          const int key = key_of(i), sl = st * kKeys + key;
          return fresh ? w.past + key : sl < p.sinks ? sl : sl + (w.past - 1 - sl) / p.window * p.window;
        };
        const int s0 = st * kKeys + k0;
        const bool partly = fresh || k0 + 16 > n || (s0 < m1 && s0 + 16 > m0) || (s0 < n1 && s0 + 16 > n0);
        unsigned seen = 0xffu;  // bit 2 i + r: row r sees key i
        bool split = false;     // a value that is not finite, which not every row sees
        if (partly) {
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
            x = seen >> (2 * i + r) & 1 ? x * to2 : -INFINITY;
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
            wt[i][r] = seen >> (2 * i + r) & 1 ? e : 0.f;
            sum[r] += wt[i][r];
          }
        }
        const uint32_t a[4] = {pack(wt[0][0], wt[1][0]), pack(wt[0][1], wt[1][1]),
                               pack(wt[2][0], wt[3][0]), pack(wt[2][1], wt[3][1])};
        if (!split) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            uint32_t x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 v = value(i, h);
              // (what lies behind the last key may be anything)
              if (partly && key_of(i) >= n) v = make_uint4(0, 0, 0, 0);
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
      }
      if (st + 1 < w.end) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[slot]);
        if (warp == 0) bring(take + kStages);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    }
    // The warps' parts meet in the last stage's memory (which only then goes back
    // to the producer); a part without a stage has none, and leaves nothing.
    const bool some = w.end > w.first;
    const int slot = (take + kStages - 1) % kStages;
    float* meet = reinterpret_cast<float*>(&sm.kv[slot][0][0][0]);  // [warp][16][D]
    static_assert(sizeof(sm.kv[0]) >= sizeof(float) * kWarps * 16 * D, "room for the parts");
    __syncthreads();
    if (some) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float* row = meet + ((size_t)warp * 16 + g + 8 * r) * D;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; j += 4)
              *reinterpret_cast<float4*>(row + 64 * h + 16 * t + 8 * c + j) =
                  make_float4(o[h][j][2 * r + c], o[h][j + 1][2 * r + c], o[h][j + 2][2 * r + c],
                              o[h][j + 3][2 * r + c]);
        if (t == 0) {
          sm.top[warp][g + 8 * r] = top[r];
          sm.sum[warp][g + 8 * r] = sum[r];
        }
      }
    }
    __syncthreads();
    const int unit = u / parts;  // whose parts meet
    float* mine_left = left + (size_t)u * part_floats<D>();
    // four columns of a row at a time
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), c = i % (D / 4) * 4, tile = row >> 4, r = row & 15;
      float m = -INFINITY, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (some) {
        for (int k = 0; k < sharing; ++k) m = fmaxf(m, sm.top[tile + k * tiles][r]);
        const float base = m == -INFINITY ? 0.f : m;
        for (int k = 0; k < sharing; ++k) {
          const int wk = tile + k * tiles;
          const float f = ex2(sm.top[wk][r] - base);
          const float4 x = *reinterpret_cast<const float4*>(meet + ((size_t)wk * 16 + r) * D + c);
          l = fmaf(sm.sum[wk][r], f, l);
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
      }
      if (parts == 1) {
        const int token = row / p.group, head = w.hk * p.group + row % p.group;
        const float inv = 1.f / l;
        uint2 y = make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)(w.row0 + token) * p.ldo +
                                  (size_t)head * D + c) = y;
      } else {
        *reinterpret_cast<float4*>(mine_left + (size_t)row * D + c) = acc;
        if (c == 0) {
          mine_left[(size_t)kMaxRows * D + 2 * row] = m;
          mine_left[(size_t)kMaxRows * D + 2 * row + 1] = l;
        }
      }
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
    // (the stage's memory is read: the copies to come are ordered behind the writes above)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (parts == 1) __syncthreads();
    __syncwarp();
    if (some && lane == 0) mbar_arrive(&sm.empty[slot]);
    if (warp == 0) bring(take + kStages);
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
  if (warp == 0 && dead)
    for (uint32_t i = fill > kStages ? fill - kStages : 0; i < fill; ++i)
      mbar_wait_bounded(&sm.full[i % kStages], i / kStages & 1);
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
  // parts of two stages at least.
  const long long heads = (long long)max_items * p.Hkv;
  const int stages = (p.sinks + p.window + kKeys - 1) / kKeys + 1;
  int parts = heads > 0 && heads < 2 * sms && heads * sizeof(int32_t) <= kWinCounterBytes ? (int)(2 * sms / heads) : 1;
  if (parts > (stages + 1) / 2) parts = (stages + 1) / 2;
  const long long units = heads * parts;
  const int ctas = (int)(units < 2 * sms ? (units > 0 ? units : 1) : 2 * sms);
  return p.d == 64 ? launch_short<64>(p, of, parts, ctas, room, s)
                   : launch_short<128>(p, of, parts, ctas, room, s);
}

}  // namespace gdn
