// Causal attention with a sliding window and a few first tokens that stay
// visible, over a packed batch, continued from each request's keys and values
// in its block of a paged pool (the windowed layers beside the linear ones in
// hybrid models: their cache has a fixed size per request, as a linear layer's
// state has).  Position p of a request sees j <= p with j > p - window or
// j < sinks:
//   o_p = sum_j w_j v_j / sum_j w_j,   w_j = e^{scale q_p k_j - m_p}
// A block holds the keys and the values of the first `sinks` positions and of
// a ring of the last `window` ones, per kv head.
//
// This file: the form for any type and shape, the append of the new keys and
// values, and the C entry points.
#include <cuda_runtime.h>

#include <cmath>
#include <new>
#include <type_traits>

#include "gdn_cta.cuh"
#include "gdn_lin.cuh"
#include "gdn_pool.cuh"
#include "gdn_win.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// --- any type and shape ------------------------------------------------------
// A CTA takes kRows rows of one kv head (queries of consecutive tokens, the
// heads that share the kv head next to each other) and walks the keys in tiles
// of kKeys, with the running maximum and sum of the softmax: fp32 throughout.
// Bound by latency (a tile's loads, products and softmax follow one another) and,
// with many CTAs, by its 131,072 multiply-adds a tile (d = 64) at 128 a clock: six
// sequences of 1,554 tokens x 12 heads of d = 64 in fp32, window 200, 68.6 us (82
// with a row's maximum and sum by shuffles, row after row, and each masked weight
// looked at in the products).  Tensor cores would round the operands to less than
// fp32.
constexpr int kRowThreads = 128;
constexpr int kRows = 32, kKeys = 32;

template <int D>
struct RowSmem {
  float q[kRows][D + 4], k[kKeys][D + 4], v[kKeys][D + 4];
  float p[kKeys][kRows + 4];  // the weights (below 0: a masked value must not be touched)
  const void *from_k[kKeys], *from_v[kKeys];  // where a tile's rows lie
  float sum[kRows], shrink[kRows];
  PlanSmem plan;
};

// Tokens t0 .. t0 + tokens - 1 of sequence s (or, with more than kRows heads to a
// kv head, part `sub` of one token's heads).
template <typename T, int D>
__device__ void rows_of(const WinParams& p, RowSmem<D>& sm, int s, int t0, int tokens, int hk, int sub) {
  const Batch& b = p.batch;
  const int row0 = b.cu[s], past = b.past_len[s], blk = b.blk[s];
  const int per = min(kRows, p.group - sub * kRows);  // heads of a token here
  const int rows = p.group > kRows ? per : tokens * p.group;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* ring_k = ring_of<T>(p, blk, 0, hk);
  const T* ring_v = ring_of<T>(p, blk, 1, hk);
  auto head = [&](int r) { return hk * p.group + sub * kRows + r % per; };
  // four channels of a row
  auto four = [](const T* p4) {
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4*>(p4);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(p4);
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                         __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    }
  };
  constexpr int kVecs = D / 4;
  for (int i = tid; i < kRows * kVecs; i += kRowThreads) {
    const int r = i / kVecs, c = i % kVecs * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = four(static_cast<const T*>(p.q) + (size_t)(row0 + t0 + r / per) * p.ldq + (size_t)head(r) * D + c);
    *reinterpret_cast<float4*>(&sm.q[r][c]) = x;
  }
  // of the warp's 8 rows: the maximum so far, and each lane's part of the sum
  float top[8], sum[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    top[r] = -INFINITY;
    sum[r] = 0.f;
  }
  // the positions that any row sees: sinks before the window's first, then those
  const int p0 = past + t0, p1 = p0 + tokens;
  const int lo = max(0, p0 - p.window + 1), before = min(p.sinks, lo), n_keys = before + p1 - lo;
  auto position = [&](int i) { return i < before ? i : lo + i - before; };
  // each thread's part of the output: 4 rows, D/16 columns side by side
  constexpr int kCols = D / 16;
  const int or0 = tid / 16 * 4, oc = tid % 16 * kCols;
  F2 acc[4][kCols / 2];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) acc[r][c] = 0ull;
  const float to2 = p.scale * kLog2e;
  for (int k0 = 0; k0 < n_keys; k0 += kKeys) {
    const int n = min(kKeys, n_keys - k0);
    __syncthreads();  // the last tile is read
    if (tid < n) {
      const int j = position(k0 + tid);
      if (j < past) {
        const size_t at = (size_t)slot_of(p, j) * D;
        sm.from_k[tid] = ring_k + at;
        sm.from_v[tid] = ring_v + at;
      } else {
        const size_t row = row0 + (j - past);
        sm.from_k[tid] = static_cast<const T*>(p.k) + row * p.ldk + (size_t)hk * D;
        sm.from_v[tid] = static_cast<const T*>(p.v) + row * p.ldv + (size_t)hk * D;
      }
    }
    __syncthreads();
    bool odd = false;
#pragma unroll 4
    for (int i = tid; i < n * kVecs; i += kRowThreads) {
      const int r = i / kVecs, c = i % kVecs * 4;
      const float4 x = four(static_cast<const T*>(sm.from_k[r]) + c), y = four(static_cast<const T*>(sm.from_v[r]) + c);
      *reinterpret_cast<float4*>(&sm.k[r][c]) = x;
      *reinterpret_cast<float4*>(&sm.v[r][c]) = y;
      odd |= !(fabsf(y.x) + fabsf(y.y) + fabsf(y.z) + fabsf(y.w) < INFINITY);
    }
    // whether every row sees every key of the tile
    const int first = position(k0), last = position(k0 + n - 1);
    const bool all = rows == kRows && n == kKeys && last <= p0 &&
                     (first > p1 - 1 - p.window || last < p.sinks);
    // (finite values, or all seen: 0 is a masked one's weight)
    const bool plain = !__syncthreads_or(odd) || all;
    // scores: a warp has 8 rows, a lane one key
    const int j = lane < n ? position(k0 + lane) : 0;
    float sc[8];
    {
      F2 even[8];  // (sums over even and odd channels)
#pragma unroll
      for (int r = 0; r < 8; ++r) even[r] = 0ull;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {  // (lanes behind the last key: anything)
        const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(&sm.k[lane][c]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(&sm.q[warp * 8 + r][c]);
          even[r] = fma2(qq.x, kk.x, fma2(qq.y, kk.y, even[r]));
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float x, y;
        unf2(even[r], x, y);
        sc[r] = x + y;
      }
    }
    float most[8];
    unsigned unseen = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int row = warp * 8 + r;
      const bool seen = all || (row < rows && lane < n && sees(p, p0 + row / per, j));
      if (!seen) unseen |= 1u << r;
      most[r] = sc[r] = seen ? sc[r] * to2 : -INFINITY;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(most[r]));
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float to = fmaxf(top[r], most[r]);
      // (nothing but -inf so far: any number in the maximum's place)
      const float base = to == -INFINITY ? 0.f : to;
      const float shrink = exp2f(top[r] - base);
      const bool seen = !(unseen >> r & 1);
      const float w = seen ? exp2f(sc[r] - base) : 0.f;
      sum[r] = fmaf(sum[r], shrink, w);
      top[r] = to;
      sm.p[lane][warp * 8 + r] = seen || plain ? w : -1.f;
      if (lane == 0) sm.shrink[warp * 8 + r] = shrink;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = sm.shrink[or0 + r];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) acc[r][c] = mul2(acc[r][c], f2(f, f));
    }
    auto values = [&](auto all_c) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float4 w4 = *reinterpret_cast<const float4*>(&sm.p[i][or0]);
        const float w[4] = {w4.x, w4.y, w4.z, w4.w};
        F2 vv[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) vv[c] = *reinterpret_cast<const F2*>(&sm.v[i][oc + 2 * c]);
        // (a masked value is not touched: it may be infinite or NaN)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c)
            if (decltype(all_c)::value || !(w[r] < 0.f)) acc[r][c] = fma2(f2(w[r], w[r]), vv[c], acc[r][c]);
      }
    };
    if (plain) values(std::true_type());
    else values(std::false_type());
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], w);
    if (lane == 0) sm.sum[warp * 8 + r] = sum[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = or0 + r;
    if (row >= rows) continue;
    const float inv = 1.f / sm.sum[row];
    T* o = static_cast<T*>(p.out) + (size_t)(row0 + t0 + row / per) * p.ldo + (size_t)head(row) * D;
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) {
      float x, y;
      unf2(acc[r][c], x, y);
      o[oc + 2 * c] = from_f32<T>(x * inv);
      o[oc + 2 * c + 1] = from_f32<T>(y * inv);
    }
  }
}

// left: over the units in the list, pieces of the tensor-core form (p.group is at
// most its tile's 128 rows).
template <typename T, int D, bool kLeft>
__global__ void __launch_bounds__(kRowThreads, 5) win_rows_kernel(WinParams p, Pieces pieces, const int32_t* left) {
  extern __shared__ __align__(16) unsigned char row_smem[];
  RowSmem<D>& sm = *reinterpret_cast<RowSmem<D>*>(row_smem);
  pdl_wait_then_release();
  const Batch& b = p.batch;
  int n_left = 0;
  if (kLeft) {
    n_left = b.work.header()[kWorkHead];
    if (n_left == 0) return;
  }
  const SeqList list = b.listed ? listed_long(b)
                                : plan_self(b, pieces, sm.plan, p.report && blockIdx.x == 0);
  const int subs = (p.group + kRows - 1) / kRows;  // parts of a token's heads
  const int step = subs > 1 ? 1 : kRows / p.group;  // tokens at a time
  auto unit = [&](int piece, int hk, int sub) {
    const int e = entry_of(list, piece), s = list.items[e];
    const int t0 = (piece - list.first[e]) * pieces.tokens;
    const int end = min(t0 + pieces.tokens, b.cu[s + 1] - b.cu[s]);
    for (int t = t0; t < end; t += step) {
      rows_of<T, D>(p, sm, s, t, min(step, end - t), hk, sub);
      __syncthreads();
    }
  };
  if (kLeft) {
    // (more than the list holds: all)
    const int n = n_left > kWinLeft ? list.total * p.Hkv : n_left;
    for (int i = blockIdx.x; i < n * subs; i += gridDim.x) {
      const int u = n_left > kWinLeft ? i / subs : left[i / subs];
      if (u < list.total * p.Hkv) unit(u / p.Hkv, u % p.Hkv, i % subs);
    }
  } else {
    const int sub = blockIdx.x % subs, hk = blockIdx.x / subs % p.Hkv, piece = blockIdx.x / (subs * p.Hkv);
    if (piece < list.total) unit(piece, hk, sub);
  }
}

// --- the new keys and values into the blocks ----------------------------------
// Behind the attention, which reads what they replace.
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;  // per piece

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) win_append_kernel(WinParams p, Pieces pieces) {
  __shared__ PlanSmem plan;
  pdl_wait_then_release();
  const Batch& b = p.batch;
  if (blockIdx.x == 0 && threadIdx.x == 0) {  // nothing is left, and no unit claimed
    b.work.header()[kWorkHead] = 0;
    b.work.header()[kItemHeadC] = 0;
  }
  const SeqList list = b.listed ? listed_long(b) : plan_self(b, pieces, plan, false);  // (reported before)
  const int row16 = p.Hkv * p.d * (int)sizeof(T) / 16, head16 = p.d * (int)sizeof(T) / 16;
  for (int piece = blockIdx.x; piece < list.total; piece += gridDim.x) {
    const int e = entry_of(list, piece), s = list.items[e];
    const int t0 = (piece - list.first[e]) * pieces.tokens;
    const int row0 = b.cu[s], len = b.cu[s + 1] - row0, past = b.past_len[s], blk = b.blk[s];
    const int n = min(pieces.tokens, len - t0);
    if (past + t0 >= p.sinks && t0 + n <= len - p.window) continue;  // out of every later window
    // a thread has 16 bytes of a row (keys, then values) and walks the tokens, the
    // reads of kAhead of them on their way together
    constexpr int kAhead = 8;
    for (int x = threadIdx.x; x < 2 * row16; x += kAppendThreads) {
      const int part = x >= row16, y = part ? x - row16 : x, hk = y / head16, c = y - hk * head16;
      const long long ld = part ? p.ldv : p.ldk;
      const T* src = static_cast<const T*>(part ? p.v : p.k) + (size_t)(row0 + t0) * ld + (size_t)hk * p.d;
      uint4* dst = reinterpret_cast<uint4*>(ring_of<T>(p, blk, part, hk)) + c;
      for (int i0 = 0; i0 < n; i0 += kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i0 + i < n) v[i] = reinterpret_cast<const uint4*>(src + (size_t)(i0 + i) * ld)[c];
        int slot = slot_of(p, past + t0 + i0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int t = t0 + i0 + i;
          // (what is out of every later window stays out)
          if (i0 + i < n && (past + t < p.sinks || t >= len - p.window)) dst[(size_t)slot * head16] = v[i];
          if (++slot == p.sinks + p.window) slot = p.sinks;
        }
      }
    }
  }
}

template <typename T, int D, bool kLeft>
cudaError_t launch_rows(const WinParams& p, const Pieces& of, unsigned ctas, const int32_t* left,
                        cudaStream_t s) {
  auto kern = win_rows_kernel<T, D, kLeft>;
  const size_t smem = sizeof(RowSmem<D>);
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kRowThreads), smem, s, p, of, left);
}

size_t roundup(size_t v, size_t m) { return (v + m - 1) / m * m; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

size_t win_stride(int Hkv, int d, int window, int sinks, int act, size_t align) {
  const size_t row = (size_t)d * (act == GDN_F32 ? 4 : 2);
  return roundup(2 * (size_t)Hkv * ((size_t)window + sinks) * row, align > 128 ? align : 128);
}

int check_win_dims(int num_blocks, int num_layers, int Hkv, int d, int window, int sinks, int act,
                   size_t align) {
  if (num_blocks < 2 || num_layers < 1) return GDN_ERR_RANGE;
  if (Hkv < 1 || Hkv > 1024 || (d != 32 && d != 64 && d != 128)) return GDN_ERR_DIMS;
  if (window < 1 || window > (1 << 20) || sinks < 0 || sinks > 4096) return GDN_ERR_DIMS;
  if (act != GDN_F32 && act != GDN_BF16) return GDN_ERR_DIMS;
  if (align != 0 && (align < 128 || (align & (align - 1)) != 0)) return GDN_ERR_DIMS;
  if ((long long)num_blocks * num_layers >= (1ll << 30)) return GDN_ERR_RANGE;
  // (a layer's rows of keys and values are counted in 32 bits)
  if ((double)num_blocks * win_stride(Hkv, d, window, sinks, act, align) / (d * (act == GDN_F32 ? 4 : 2)) > 2147483000.0)
    return GDN_ERR_RANGE;
  return GDN_OK;
}

}  // namespace

cudaError_t launch_win_rows(const WinParams& p, int act, const Pieces& of, int max_pieces, int sms,
                            const void* room, bool left, cudaStream_t s) {
  const int subs = (p.group + kRows - 1) / kRows;
  if (left) {  // (bf16, d = 64 or 128)
    const int32_t* list =
        reinterpret_cast<const int32_t*>(static_cast<const unsigned char*>(room) + kWinCounterBytes);
    return p.d == 64 ? launch_rows<__nv_bfloat16, 64, true>(p, of, 2 * sms, list, s)
                     : launch_rows<__nv_bfloat16, 128, true>(p, of, 2 * sms, list, s);
  }
  const unsigned ctas = (unsigned)max_pieces * subs * p.Hkv;
  if (act == GDN_F32)
    return p.d == 32   ? launch_rows<float, 32, false>(p, of, ctas, nullptr, s)
           : p.d == 64 ? launch_rows<float, 64, false>(p, of, ctas, nullptr, s)
                       : launch_rows<float, 128, false>(p, of, ctas, nullptr, s);
  return p.d == 32   ? launch_rows<__nv_bfloat16, 32, false>(p, of, ctas, nullptr, s)
         : p.d == 64 ? launch_rows<__nv_bfloat16, 64, false>(p, of, ctas, nullptr, s)
                     : launch_rows<__nv_bfloat16, 128, false>(p, of, ctas, nullptr, s);
}

cudaError_t launch_win_append(const WinParams& p, int act, const Pieces& of, int max_pieces, int sms,
                              cudaStream_t s) {
  // (eight to an SM list the batch twice as often: 1.5 us more)
  const int ctas = max_pieces < 4 * sms ? max_pieces : 4 * sms;
  auto kern = act == GDN_F32 ? win_append_kernel<float> : win_append_kernel<__nv_bfloat16>;
  return launch_pdl(kern, dim3(ctas), dim3(kAppendThreads), 0, s, p, of);
}

}  // namespace gdn

extern "C" {

int gdn_win_pool_layout_for(int num_blocks, int num_layers, int num_kv_heads, int d, int window,
                            int sinks, int act, size_t block_align, size_t* block_stride,
                            size_t* v_off, size_t* total_bytes) {
  const int st = gdn::check_win_dims(num_blocks, num_layers, num_kv_heads, d, window, sinks, act, block_align);
  if (st != GDN_OK) return st;
  const size_t stride = gdn::win_stride(num_kv_heads, d, window, sinks, act, block_align);
  if (block_stride) *block_stride = stride;
  if (v_off) *v_off = (size_t)num_kv_heads * ((size_t)window + sinks) * d * (act == GDN_F32 ? 4 : 2);
  if (total_bytes) *total_bytes = stride * (size_t)num_blocks * (size_t)num_layers;
  return GDN_OK;
}

int gdn_win_pool_create(gdn_pool_t** out, int num_blocks, int num_layers, int num_kv_heads, int d,
                        int window, int sinks, int act, size_t block_align, void* device_mem,
                        size_t device_bytes) {
  if (!out) return GDN_ERR_NULL;
  *out = nullptr;
  int st = gdn::check_win_dims(num_blocks, num_layers, num_kv_heads, d, window, sinks, act, block_align);
  if (st != GDN_OK) return st;
  const size_t stride = gdn::win_stride(num_kv_heads, d, window, sinks, act, block_align);
  const size_t total = stride * (size_t)num_blocks * (size_t)num_layers;
  if (device_mem) {
    if (device_bytes < total) return GDN_ERR_NOMEM;
    if (((uintptr_t)device_mem & 255u) != 0) return GDN_ERR_ALIGN;
  }
  gdn_pool* p = new (std::nothrow) gdn_pool();
  if (!p) return GDN_ERR_NOMEM;
  p->kind = 4;
  p->num_blocks = num_blocks;
  p->num_layers = num_layers;
  p->Hk = num_kv_heads;
  p->dk = p->dv = d;
  p->window = window;
  p->sinks = sinks;
  p->act = act;
  p->last_path = GDN_PREFILL_NONE;
  p->stride = stride;
  p->rec_off = (size_t)num_kv_heads * ((size_t)window + sinks) * d * (act == GDN_F32 ? 4 : 2);
  p->total = total;
  st = gdn::pool_allocate(p, device_mem);
  if (st != GDN_OK) {
    delete p;
    return st;
  }
  if (gdn::win_short_supported(d, act)) {
    const size_t room = gdn::win_short_room(p->sms, d);
    if (cudaMalloc(&p->win_parts, room) != cudaSuccess) {
      cudaGetLastError();
      p->win_parts = nullptr;
      gdn_state_pool_destroy(p);
      return GDN_ERR_NOMEM;
    }
    // the arrival counters
    if (cudaMemset(p->win_parts, 0, gdn::kWinCounterBytes) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
      cudaGetLastError();
      gdn_state_pool_destroy(p);
      return GDN_ERR_CUDA;
    }
  }
  *out = p;
  return GDN_OK;
}

int gdn_win_varlen_forward(gdn_pool_t* p, int layer, const void* q, const void* k, const void* v,
                           int64_t ldq, int64_t ldk, int64_t ldv, int num_heads,
                           const int32_t* cu_seqlens, const int32_t* state_block_idx,
                           const int32_t* past_lens, float scale, void* out, int64_t ldo, int T,
                           int N, int max_seqlen_hint, void* stream) {
  if (!p) return GDN_ERR_NULL;
  if (p->kind != 4) return GDN_ERR_DIMS;
  if (layer < 0 || layer >= p->num_layers || T < 0 || N < 0 || max_seqlen_hint < 0)
    return GDN_ERR_RANGE;
  if (num_heads < 1 || num_heads > 4096 || num_heads % p->Hk != 0) return GDN_ERR_DIMS;
  // (its product with log2 e, which the kernels scale by, is finite)
  if (!(fabsf(scale) <= 0x1p127f)) return GDN_ERR_RANGE;
  if (N == 0) return T == 0 ? GDN_OK : GDN_ERR_RANGE;
  if (!cu_seqlens || !state_block_idx || !past_lens) return GDN_ERR_NULL;
  if (T > 0 && (!q || !k || !v || !out)) return GDN_ERR_NULL;
  const int d = p->dk;
  const int per16 = p->act == GDN_F32 ? 4 : 8;
  if (T > 0) {
    if (!gdn::aligned16(q) || !gdn::aligned16(k) || !gdn::aligned16(v) || !gdn::aligned16(out) ||
        ldq % per16 != 0 || ldk % per16 != 0 || ldv % per16 != 0 || ldo % per16 != 0)
      return GDN_ERR_ALIGN;
    const int64_t qcols = (int64_t)num_heads * d, kcols = (int64_t)p->Hk * d;
    const int64_t most = (int64_t)1 << 38;
    if (ldq < qcols || ldo < qcols || ldk < kcols || ldv < kcols || ldq > most || ldk > most ||
        ldv > most || ldo > most)
      return GDN_ERR_RANGE;
  }
  int max_items = N < p->num_blocks - 1 ? N : p->num_blocks - 1;
  if (max_items > T) max_items = T;
  // (the grid: a CTA per token and 32 heads at most)
  if (((long long)T + max_items) * num_heads > 0x7fffffffll) return GDN_ERR_RANGE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  if (dev != p->device) return GDN_ERR_DEVICE;

  gdn::WinParams wp = {};
  gdn::Batch& b = wp.batch;
  b.cu = cu_seqlens;
  b.blk = state_block_idx;
  b.past_len = past_lens;
  b.N = N;
  b.T = T;
  b.num_blocks = p->num_blocks;
  b.hint = max_seqlen_hint;
  b.listed = N > gdn::kSelfPlan;
  b.work.base = p->work + (size_t)layer * gdn::WorkArea::words(p->num_blocks);
  b.work.num_blocks = p->num_blocks;
  wp.q = q;
  wp.k = k;
  wp.v = v;
  wp.out = out;
  wp.ldq = ldq;
  wp.ldk = ldk;
  wp.ldv = ldv;
  wp.ldo = ldo;
  wp.scale = scale;
  wp.layer_base = p->base + (size_t)layer * p->num_blocks * p->stride;
  wp.stride = p->stride;
  wp.H = num_heads;
  wp.Hkv = p->Hk;
  wp.group = num_heads / p->Hk;
  wp.d = d;
  wp.window = p->window;
  wp.sinks = p->sinks;
  wp.report = 1;

  cudaStream_t s = (cudaStream_t)stream;
  // few tokens in a form of their own, where there is one
  const int few = gdn::win_short_supported(d, p->act) ? gdn::win_short_tokens(wp.group) : 0;
  const bool may_long = few == 0 || (T > few && (max_seqlen_hint == 0 || max_seqlen_hint > few));
  // (a single sequence that no form may take: a kernel that looks at the batch)
  const bool may_short = few > 0 && !(N == 1 && T > few && may_long);
  // (in the prompts' form a masked score is -inf before it is scaled, and 0 times it NaN: a scale
  // near 0 goes to the form for any shape)
  const bool tc = T > 0 && gdn::win_tc_supported(d, p->act, wp.group) && fabsf(scale) >= 0x1p-100f;
  gdn::Pieces of = {few + 1, 0x7fffffff,
                    tc ? gdn::win_tc_tokens(wp.group) : wp.group < gdn::kRows ? gdn::kRows / wp.group : 1};
  const int max_long = max_items < T / (few + 1) ? max_items : T / (few + 1);
  auto most_pieces = [&](int tokens) {
    const int n = T / tokens + max_long;
    return n > 0 ? n : 1;  // (a kernel that looks at the batch)
  };
  p->last_path = !may_long || T < 2 || max_seqlen_hint == 1 ? GDN_PREFILL_NONE
                 : tc                                        ? GDN_PREFILL_FUSED
                                                             : GDN_PREFILL_SERIAL;
  if (b.listed && gdn::launch_plan(b, of, s) != cudaSuccess) return GDN_ERR_CUDA;
  if (p->ev_before && cudaEventRecord(p->ev_before, s) != cudaSuccess) return GDN_ERR_CUDA;
  const gdn::Pieces of_few = {1, few, 0x7fffffff};
  if (may_long && tc) {
    if (gdn::launch_win_tc(wp, of, most_pieces(of.tokens), p->sms, p->win_parts, s) != cudaSuccess)
      return GDN_ERR_CUDA;
    wp.report = 0;
  }
  auto behind = [&]() {
    // (behind the prompts' kernel, not behind what follows it)
    if (may_short) {
      const cudaError_t e = gdn::launch_win_short(wp, of_few, max_items, p->sms, may_long && tc, p->win_parts, s);
      if (e != cudaSuccess) return e;
      wp.report = 0;
    }
    if (!may_long) return cudaSuccess;
    const cudaError_t e = gdn::launch_win_rows(wp, p->act, of, most_pieces(of.tokens), p->sms, p->win_parts, tc, s);
    if (e != cudaSuccess) return e;
    if (!b.listed) of.tokens = gdn::kAppendTokens;
    return gdn::launch_win_append(wp, p->act, of, most_pieces(of.tokens), p->sms, s);
  };
  if (behind() != cudaSuccess) {
    // (what the append, which was not launched, would have set back for the next call)
    static_assert(gdn::kItemHeadC == gdn::kWorkHead + 2, "the claimed and the left units' counters");
    if (may_long && tc) cudaMemsetAsync(b.work.header() + gdn::kWorkHead, 0, 3 * sizeof(int32_t), s);
    return GDN_ERR_CUDA;
  }
  if (p->ev_after && cudaEventRecord(p->ev_after, s) != cudaSuccess) return GDN_ERR_CUDA;
  return GDN_OK;
}

}  // extern "C"
