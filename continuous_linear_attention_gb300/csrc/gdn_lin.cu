// Linear attention with one decay per head over a packed batch, continued
// from each request's state in a paged pool (the lightning / simple gated
// linear attention layers among the families the model support tracker
// lists):
//   S_t = e^{g_h} S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t
// with S [d_k][d_v] fp32 per request and head.
//
// This file: the recurrent form, the batch scheduler and the C entry points.
// The recurrent kernel is bound by HBM for single tokens: a head's state
// (64 KiB at d = 128) is read once and written once whatever the number of
// tokens.  A CTA owns 32 columns v of one head's state (the columns are
// independent of each other), every thread 4 columns of d/16 rows in registers;
// all of a CTA's state loads are issued before anything else, and six CTAs per
// SM keep about 100 KB of reads in flight: 256 requests x 32 heads 160 us,
// 6.78 TB/s (fp32 161; d = 64, 64 heads 86, 6.3 TB/s; d = 32, 128 heads 57, 4.9
// TB/s: 4 KB of state a CTA).  With more tokens the arithmetic (4 d^2 multiply-adds
// per token and head with the decay, in packed fp32) shares the time: 64
// requests of 4 tokens x 32 heads 49 us, 0.82 of the copy bandwidth (fp32 64;
// d = 64, 64 heads 37 and 39; d = 32, 128 heads 26 and 27).
#include <cuda_runtime.h>

#include <new>
#include <type_traits>

#include "gdn_cta.cuh"
#include "gdn_lin.cuh"
#include "gdn_pool.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

// --- recurrent form ----------------------------------------------------------
constexpr int kRecThreads = 128;
constexpr int kSlice = 32;                          // state columns per CTA
constexpr int kColT = kSlice / 4;                   // threads across the columns
constexpr int kRowT = kRecThreads / kColT;          // threads across the rows
constexpr int kTile = 16;                           // tokens staged at a time
// Calls of up to this many sequences check the batch in every CTA, while its
// state loads are in flight, which saves the scheduler's launch: 256 single
// tokens x 32 heads 160 us (163 with the scheduler), 512 x 16 heads 167 and 166,
// 1,024 358 and 328; 128 times four tokens x 16 heads 50 (52), 256 100 and 96.
constexpr int kSelfCheck = 256;
// groups of kRecThreads that work on segments side by side on an SM (their
// shared memory: 176 KB of fp32 at d = 128)
constexpr int kSerialPerSm = 4;

// kN consecutive elements (kN * sizeof(T) aligned): as they lie, and as fp32.
template <typename T, int kN>
struct Vec {
  static constexpr int kWords = kN * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ F2 pair(int i) const { return f2(at(i), at(i + 1)); }
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <typename T, int D, bool kOne>
struct RecSmem {
  T q[2][kTile][D], k[2][kTile][D], v[2][kTile][kSlice];
  float part[kTile][kRecThreads / 32][kSlice];
};
template <typename T, int D>
struct RecSmem<T, D, true> {
  float part[1][kRecThreads / 32][kSlice];
};

// Barrier of the kRecThreads threads that work on one unit: the CTA, or one of
// its groups.
template <bool kGroups>
__device__ __forceinline__ void unit_sync() {
  if constexpr (kGroups)
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.x / kRecThreads), "n"(kRecThreads) : "memory");
  else
    __syncthreads();
}

// Columns 32 slice .. of head h over len tokens from row row0: the state is
// read from src (unless zero: it starts at zeros), advanced and written to dst
// (nullptr: not), both the head's [D][D].  ok() is asked once all reads are on their way, and
// nothing is written where it says no.  kOne: len is at most 1.  kState: the
// state only, no outputs.
template <typename T, int D, bool kOne, bool kState, bool kGroups, typename Ok>
__device__ __forceinline__ void recurrent_body(const LinParams& p, RecSmem<T, D, kOne>& sm,
                                               int row0, int len, int h, int slice,
                                               bool zero, const float* src, float* dst, Ok ok) {
  constexpr int kRows = D / kRowT;      // state rows per thread
  const int tid = kGroups ? threadIdx.x % kRecThreads : threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = slice * kSlice + (tid % kColT) * 4;  // this thread's columns
  const int r0 = (tid / kColT) * kRows;               // and rows
  const size_t at = (size_t)r0 * D + c0;
  float4 read[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    read[i] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : *reinterpret_cast<const float4*>(src + at + (size_t)i * D);
  // rows in pairs, for packed arithmetic: S[i][c] is rows 2 i and 2 i + 1 of
  // column c (made of the reads when all others are on their way)
  F2 S[kRows / 2][4];
  const DecayPair a = decay_pair(finite_decay(p.log_decay[h]));
  const int hk = h / p.group;
  const T* q = static_cast<const T*>(p.q) + (size_t)row0 * p.ldq + (size_t)h * D;
  const T* k = static_cast<const T*>(p.k) + (size_t)row0 * p.ldk + (size_t)hk * D;
  const T* v = static_cast<const T*>(p.v) + (size_t)row0 * p.ldv + (size_t)hk * D +
               slice * kSlice;
  // One token: S <- e^g S + k v^T, and this thread's part of S^T q.  The rest of
  // the decay, a.lo, is added for a whole tile at its first token (rest: that
  // many times a.lo), which saves a quarter of the arithmetic: the tile's own
  // tokens go without it until the next one (at most 15 times 2^-25, once), and
  // it is part of a sum that is rounded once, where a product with 1 + a.lo would
  // round it away.
  const F2 ahi = f2(a.hi, a.hi);
  auto rest_of = [&](int n) { return f2(a.lo * (float)n, a.lo * (float)n); };
  auto token = [&](const Vec<T, kRows>& qr, const Vec<T, kRows>& kr, const Vec<T, 4>& vc,
                   auto with_rest, F2 rest) {
    [[maybe_unused]] F2 o[4];
    F2 v2[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v2[c] = f2(vc.at(c), vc.at(c));
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      const F2 k2 = kr.pair(2 * i);
      [[maybe_unused]] const F2 q2 = kState ? 0 : qr.pair(2 * i);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        F2 t = mul2(k2, v2[c]);
        if constexpr (decltype(with_rest)::value) t = fma2(rest, bounded(S[i][c]), t);
        S[i][c] = t = fma2(ahi, S[i][c], t);
        if constexpr (!kState) o[c] = i == 0 ? mul2(q2, t) : fma2(q2, t, o[c]);
      }
    }
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (!kState) {
      float x, y;
      unf2(o[0], x, y); r.x = x + y;
      unf2(o[1], x, y); r.y = x + y;
      unf2(o[2], x, y); r.z = x + y;
      unf2(o[3], x, y); r.w = x + y;
    }
    return r;
  };
  // the sum over the warp's row groups
  auto across = [](float4 o) {
#pragma unroll
    for (int w = kColT; w < 32; w <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, w);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, w);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, w);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, w);
    }
    return o;
  };
  // a single token's q, k and v; with kOne before the checks, else (where they
  // would take registers from the longer sequences) behind them
  Vec<T, kRows> q0, k0;
  Vec<T, 4> v0;
  auto load_one = [&]() {
    if (len == 1) {
      if constexpr (!kState) q0.load(q + r0);
      k0.load(k + r0);
      v0.load(v + (tid % kColT) * 4);
    }
  };
  if constexpr (kOne) load_one();
  // stages tile t0 .. of the tokens in buffer b
  [[maybe_unused]] auto stage = [&](int t0, int b) {
    if constexpr (!kOne) {
      const int n = min(kTile, len - t0);
      constexpr int kRow16 = D * (int)sizeof(T) / 16, kSl16 = kSlice * (int)sizeof(T) / 16;
      constexpr int kPer = 16 / (int)sizeof(T);
      for (int i = tid; i < n * kRow16; i += kRecThreads) {
        const int t = i / kRow16, c = (i % kRow16) * kPer;
        if constexpr (!kState) cp_async16(&sm.q[b][t][c], q + (size_t)(t0 + t) * p.ldq + c);
        cp_async16(&sm.k[b][t][c], k + (size_t)(t0 + t) * p.ldk + c);
      }
      for (int i = tid; i < n * kSl16; i += kRecThreads) {
        const int t = i / kSl16, c = (i % kSl16) * kPer;
        cp_async16(&sm.v[b][t][c], v + (size_t)(t0 + t) * p.ldv + c);
      }
      cp_async_commit();
    }
  };
  if constexpr (!kOne) {
    if (len > 1) stage(0, 0);
  }
  const bool active = ok();
  if constexpr (!kOne) {
    // (what is left out has its first tile on the way: it lands before the CTA ends)
    if (!active) cp_async_wait<0>();
  }
  [[maybe_unused]] T* out =
      static_cast<T*>(p.out) + (size_t)row0 * p.ldo + (size_t)h * D + slice * kSlice;
  if constexpr (!kOne) load_one();
#pragma unroll
  for (int i = 0; i < kRows; i += 2) {
    S[i / 2][0] = f2(read[i].x, read[i + 1].x);
    S[i / 2][1] = f2(read[i].y, read[i + 1].y);
    S[i / 2][2] = f2(read[i].z, read[i + 1].z);
    S[i / 2][3] = f2(read[i].w, read[i + 1].w);
  }
  auto store = [&]() {
    if (!dst) return;
#pragma unroll
    for (int i = 0; i < kRows; i += 2) {
      float4 x, y;
      unf2(S[i / 2][0], x.x, y.x);
      unf2(S[i / 2][1], x.y, y.y);
      unf2(S[i / 2][2], x.z, y.z);
      unf2(S[i / 2][3], x.w, y.w);
      *reinterpret_cast<float4*>(dst + at + (size_t)i * D) = x;
      *reinterpret_cast<float4*>(dst + at + (size_t)(i + 1) * D) = y;
    }
  };
  if (active && len == 1) {
    const float4 mine = token(q0, k0, v0, std::true_type(), rest_of(1));
    store();
    if constexpr (!kState) {
      const float4 o = across(mine);
      if (lane < kColT) *reinterpret_cast<float4*>(&sm.part[0][warp][lane * 4]) = o;
      unit_sync<kGroups>();
      if (tid < kSlice) {
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < kRecThreads / 32; ++w) acc += sm.part[0][w][tid];
        out[tid] = from_f32<T>(acc * p.scale);
      }
    }
  } else if constexpr (!kOne) if (active && len > 1) {
    // tokens in tiles, staged one tile ahead
    constexpr int kBatch = D == 128 ? 2 : 4;
    for (int t0 = 0, b = 0; t0 < len; t0 += kTile, b ^= 1) {
      if (t0 + kTile < len) {
        stage(t0 + kTile, b ^ 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      unit_sync<kGroups>();  // the tile has landed, and the last one's sums are read
      const int n = min(kTile, len - t0);
      // kN tokens: their reads come first and their sums run side by side
      const F2 rest = rest_of(n);
      auto batch = [&](int t, auto count, auto first) {
        constexpr int kN = decltype(count)::value;
        Vec<T, kRows> qr[kN], kr[kN];
        Vec<T, 4> vc[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u) {
          if constexpr (!kState) qr[u].load(&sm.q[b][t + u][r0]);
          kr[u].load(&sm.k[b][t + u][r0]);
          vc[u].load(&sm.v[b][t + u][(tid % kColT) * 4]);
        }
        float4 o[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u) {
          if (u == 0) o[u] = token(qr[u], kr[u], vc[u], first, rest);
          else o[u] = token(qr[u], kr[u], vc[u], std::false_type(), rest);
        }
        if constexpr (!kState) {
#pragma unroll
          for (int u = 0; u < kN; ++u) o[u] = across(o[u]);
          if (lane < kColT) {
#pragma unroll
            for (int u = 0; u < kN; ++u)
              *reinterpret_cast<float4*>(&sm.part[t + u][warp][lane * 4]) = o[u];
          }
        }
      };
      int t = 1;
      if (n >= kBatch) {
        batch(0, std::integral_constant<int, kBatch>(), std::true_type());
        t = kBatch;
      } else {
        batch(0, std::integral_constant<int, 1>(), std::true_type());
      }
      for (; t + kBatch <= n; t += kBatch)
        batch(t, std::integral_constant<int, kBatch>(), std::false_type());
      for (; t < n; ++t) batch(t, std::integral_constant<int, 1>(), std::false_type());
      unit_sync<kGroups>();  // the tile's sums are there, and its buffer may be staged over
      if constexpr (!kState) {
        for (int i = tid; i < n * kSlice; i += kRecThreads) {
          const int t = i / kSlice, c = i % kSlice;
          float acc = 0.f;
#pragma unroll
          for (int w = 0; w < kRecThreads / 32; ++w) acc += sm.part[t][w][c];
          out[(size_t)(t0 + t) * p.ldo + c] = from_f32<T>(acc * p.scale);
        }
      }
    }
    store();
  }
}

// Sequence s, head h, columns 32 slice ..: its block's state advanced by all
// its tokens.  check: nothing has looked at the batch yet.
template <typename T, int D, bool kOne>
__device__ __forceinline__ void recurrent_unit(const LinParams& p, RecSmem<T, D, kOne>& sm, int s,
                                               int h, int slice, bool check) {
  const int tid = threadIdx.x;
  const int row0 = p.cu[s], len = p.cu[s + 1] - row0;
  const int blk = p.blk[s];
  // reads may be issued for what looks right here
  bool active = len > 0 && blk > 0 && blk < p.num_blocks;
  if (check)
    active = active && row0 >= 0 && len <= p.T && row0 <= p.T - len && (p.hint == 0 || len <= p.hint);
  float* state = active ? reinterpret_cast<float*>(p.layer_base + (size_t)blk * p.stride) +
                              (size_t)h * D * D
                        : nullptr;
  auto ok = [&]() {
    if (!check) return active;
    // the batch: cu_seqlens from 0 to T and never falling, no block named
    // twice by sequences with tokens
    int bad = 0, twice = 0;
#pragma unroll 1
    for (int i = tid; i < p.N; i += kRecThreads) {
      const int lo = p.cu[i], hi = p.cu[i + 1];
      bad |= hi < lo;
      twice |= i != s && hi > lo && p.blk[i] == blk;
    }
    if (tid == 0) bad |= p.cu[0] != 0 || p.cu[p.N] != p.T;
    bad = __syncthreads_or(bad);
    twice = __syncthreads_or(twice);
    unsigned flags = 0;
    if (bad) {
      flags = GDN_FLAG_SEQLENS;
    } else if (len > 0 && blk >= 0) {
      if (blk >= p.num_blocks) flags = GDN_FLAG_BLOCK_RANGE;
      else if (blk == 0) flags = GDN_FLAG_TRASH_WRITE;
      else if (twice) flags = GDN_FLAG_DUPLICATE;
      else if (p.hint > 0 && len > p.hint) flags = GDN_FLAG_HINT;
    }
    if (flags && tid == 0 && h == 0 && slice == 0) atomicOr((unsigned*)&p.work.header()[kErr], flags);
    return active && !flags;
  };
  recurrent_body<T, D, kOne, false, false>(p, sm, active ? row0 : 0, active ? len : 0, h, slice,
                                    !active || !p.has_past[s], state, state, ok);
}

// CTAs per SM, as many as the registers leave room for: state reads in flight.
// 64 requests of 4 tokens with five, six and seven, which spill the more: bf16,
// d = 128, 32 heads 54, 49 and 52 us, fp32 65, 64 and 71; d = 64, 64 heads 38,
// 37 and 35, fp32 40, 39 and 40; fp32, d = 32, 128 heads 29, 27 and 27.
constexpr int rec_ctas(int D, bool one) {
  return one && D < 128 ? 8 : 6;
}

template <typename T, int D, bool kOne>
__global__ void __launch_bounds__(kRecThreads, rec_ctas(D, kOne))
lin_recurrent_kernel(LinParams p) {
  constexpr int kSlices = D / kSlice;
  __shared__ __align__(16) RecSmem<T, D, kOne> sm;
  // late: launched behind the chunk kernel, whose idle SMs it takes without
  // waiting for it (other sequences, other blocks; the scheduler's lists are
  // there, as the chunk kernel releases after its own wait); before it ends it
  // waits, and computes what the chunk kernel has marked: columns whose blocks
  // still hold the old state.  A CTA keeps its place until then, so an SM that
  // comes free takes one round of units beside the last chains, and the rest
  // of the single tokens follow when the chunk kernel has ended.
  if (p.late)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else
    pdl_wait_then_release();
  const int slice = blockIdx.x % kSlices;
  const int h = (blockIdx.x / kSlices) % p.H;
  int s = blockIdx.x / (kSlices * p.H);
  const bool here = !p.listed || s < p.work.header()[kNDec];
  if (here) {
    if (p.listed) s = p.work.dec()[s];
    recurrent_unit<T, D, kOne>(p, sm, s, h, slice, !p.listed);
  }
  if constexpr (!kOne) {
    if (!p.late) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t* hdr = p.work.header();
    if (!hdr[kLinBad]) return;
    const long long n = (long long)hdr[kNPre] * p.H * kSlices;
    for (long long u = blockIdx.x; u < n; u += gridDim.x) {
      if (!p.bad[u]) continue;
      const long long chain = u / kSlices;
      __syncthreads();
      recurrent_unit<T, D, kOne>(p, sm, p.work.pre()[chain / p.H], (int)(chain % p.H),
                                 (int)(u % kSlices), false);
    }
  }
}

// The segments of long sequences: kState, each one's own state
// (from zeros; the last one's is not needed by any other) to its slot, else
// their outputs from the states at their starts, which lin_segments_kernel has
// left there, and the last one's final state to the block.  One CTA per SM, of
// kSerialPerSm groups that work by themselves.  The first units go to the CTAs'
// first groups and so on, which spreads them over the SMs (as CTAs of their
// own, several of the first ones shared an SM: twice the time of a call of few
// chains), the others are taken from a counter.
template <typename T, int D, bool kState>
__global__ void __launch_bounds__(kRecThreads* kSerialPerSm, 1) lin_rec_segments_kernel(LinParams p) {
  constexpr int kSlices = D / kSlice;
  extern __shared__ __align__(128) unsigned char rec_smem[];
  __shared__ int claimed[kSerialPerSm];
  const int group = threadIdx.x / kRecThreads;
  RecSmem<T, D, false>& sm = reinterpret_cast<RecSmem<T, D, false>*>(rec_smem)[group];
  pdl_wait_then_release();
  int32_t* hdr = p.work.header();
  const int32_t* first = p.work.pre_cp();  // first[k]: segments before entry k
  const int n_units = (kState ? hdr[kLinStateItems] : hdr[kLinItems]) * p.H * kSlices;
  const int per = hdr[kLinSegChunks], n_pre = hdr[kNPre], groups = gridDim.x * kSerialPerSm;
  for (int u = group * gridDim.x + blockIdx.x, next; u < n_units; u = next) {
    if (threadIdx.x % kRecThreads == 0)
      claimed[group] =
          n_units > groups ? groups + atomicAdd(&hdr[kState ? kLinStateHead : kLinHead], 1) : n_units;
    unit_sync<true>();
    next = claimed[group];
    const int slice = u % kSlices, h = (u / kSlices) % p.H, item = u / (kSlices * p.H);
    int lo = 0, hi = n_pre - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= item) lo = mid; else hi = mid - 1;
    }
    const int seg = item - first[lo], nseg = first[lo + 1] - first[lo], s = p.work.pre()[lo];
    const int row0 = p.cu[s], len = p.cu[s + 1] - row0;
    const int t0 = nseg > 1 ? seg * per * p.chunk : 0;
    const int n = nseg > 1 ? min(per * p.chunk, len - t0) : len;
    float* block = reinterpret_cast<float*>(p.layer_base + (size_t)p.blk[s] * p.stride) + (size_t)h * D * D;
    float* slot = p.seg_states + ((size_t)item * p.H + h) * D * D;
    const bool zero = kState || (nseg == 1 && !p.has_past[s]);
    float* dst = kState ? slot : seg == nseg - 1 ? block : nullptr;
    if (!(kState && seg == nseg - 1))
      recurrent_body<T, D, false, kState, true>(p, sm, row0 + t0, n, h, slice, zero,
                                                nseg > 1 ? slot : block, dst, [] { return true; });
    unit_sync<true>();
  }
}

// The states at the segments' starts, from the segments' own: in place,
// Z[0] <- S0, Z[i] <- e^{g n} Z[i-1] + (the old Z[i-1]) with n tokens per
// segment.  One element of one head's state per thread: a chain of as many
// steps as there are segments, whose reads are independent, so that many of
// them are in flight at a time.
__global__ void __launch_bounds__(256) lin_segments_kernel(LinParams p) {
  pdl_wait_then_release();
  const int32_t* hdr = p.work.header();
  const int n_split = hdr[kLinSplit];
  constexpr int kAhead = 32;
  const int words = p.d * p.d, parts = words / 256;
  const int n_units = n_split * p.H * parts;
  for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
    const int part = u % parts, h = (u / parts) % p.H, e = u / (parts * p.H);
    const int s = p.work.pre()[e], blk = p.blk[s];
    const int first = p.work.pre_cp()[e], nseg = p.work.pre_cp()[e + 1] - first;
    const size_t at = (size_t)part * 256 + threadIdx.x;
    const float g = finite_decay(p.log_decay[h]), one = decay_pair(g).hi;
    const DecayPair a = decay_pair(g * (float)(hdr[kLinSegChunks] * p.chunk));
    float S = 0.f;
    if (p.has_past[s])
      S = reinterpret_cast<const float*>(p.layer_base + (size_t)blk * p.stride)[(size_t)h * words + at];
    float* z = p.seg_states + ((size_t)first * p.H + h) * words + at;
    const size_t step = (size_t)p.H * words;
    for (int i0 = 0; i0 < nseg; i0 += kAhead) {
      float own[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)  // (the last segment's own state is not there)
        if (i0 + i < nseg - 1) own[i] = z[(i0 + i) * step];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i0 + i >= nseg) break;
        z[(i0 + i) * step] = S;
        // (an infinite state stays so over any number of decays that are not zero)
        S = fmaf(fabsf(S) <= 3.402823466e38f ? a.hi : one, S, fmaf(a.lo, bounded(S), own[i]));
      }
    }
  }
}

// --- scheduler ---------------------------------------------------------------
constexpr int kSchedThreads = 1024;

constexpr int kSortMax = 2048;     // long sequences that are put in order
constexpr int kSmemCounts = 4096;  // pools whose block-use counts fit into shared memory
constexpr int kLanes = 8;          // threads that weigh a length of segments together
// What the split of a call into segments is weighed by.  A round of segments of
// n chunks, one per SM, takes n + 1.5 in each of its two passes (both wait for
// first loads, and there are two launches more), all in chunks of a chain alone.
constexpr int kMinSegment = 2;
template <typename U>
__host__ __device__ constexpr U chunk_cost(U n, U rounds, int passes) {
  return rounds * (passes * n + (passes == 2 ? 3 : 0));
}
// The token-serial form's tiles of kTile tokens take the longer the more units
// share an SM: 1.5 us with one, 2.6 with four (bf16, d = 64), here 3 and one more
// for each; the second pass and its launches cost about 12 us.
constexpr int kMinSerial = 4, kSerialLaunch = 32;
template <typename U>
__host__ __device__ constexpr U serial_cost(U n, U per_sm, int passes) {
  return passes * n * (3 * ((per_sm + kSerialPerSm - 1) / kSerialPerSm) + per_sm) +
         (passes == 2 ? kSerialLaunch : 0);
}

// One CTA.  Checks the batch as the pool's contract demands, lists its
// sequences and cuts the long ones into segments (slices: the parts of a head's
// state that the token-serial form works on by themselves; 0: the chunked form).
__global__ void __launch_bounds__(kSchedThreads)
lin_schedule_kernel(LinParams p, int short_max, int num_sms, int slices) {
  __shared__ unsigned s_flags;
  __shared__ int s_dec, s_pre;
  __shared__ unsigned s_total;
  __shared__ unsigned long long s_best;
  // the long sequences and their chunks, as found and in order
  __shared__ int32_t found[kSortMax], chunks[kSortMax], in_order[kSortMax], counts[kSmemCounts];
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, N = p.N, nb = p.num_blocks;
  int32_t* hdr = p.work.header();
  int32_t* uses = nb <= kSmemCounts ? counts : p.work.blk_count();
  if (tid == 0) {
    s_flags = 0u;
    s_dec = s_pre = 0;
    s_total = 0;
    s_best = ~0ull << 31;  // (no segments)
  }
  if (uses == counts)
    for (int i = tid; i < nb; i += kSchedThreads) uses[i] = 0;
  pdl_wait_then_release();
  // a thread's first sequence is read once
  int cu0 = 0, cu1 = 0, blk0 = -1;
  if (tid < N) {
    cu0 = p.cu[tid];
    cu1 = p.cu[tid + 1];
    blk0 = p.blk[tid];
  }
  auto length = [&](int q) { return q == tid ? cu1 - cu0 : p.cu[q + 1] - p.cu[q]; };
  auto block = [&](int q) { return q == tid ? blk0 : p.blk[q]; };
  if (tid == 0) {
    hdr[kLinStateItems] = hdr[kLinHead] = hdr[kLinItems] = hdr[kLinStateHead] = 0;
    hdr[kLinSplit] = hdr[kLinSegChunks] = hdr[kLinBad] = 0;
  }
  if (uses != counts)
    for (int i = tid; i < nb; i += kSchedThreads) uses[i] = 0;
  int bad = (tid == 0 && cu0 != 0) || (tid == (N - 1) % kSchedThreads && p.cu[N] != p.T);
  for (int q = tid; q < N; q += kSchedThreads)  // (a difference could wrap)
    bad |= q == tid ? cu1 < cu0 : p.cu[q + 1] < p.cu[q];
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr((unsigned*)&hdr[kErr], GDN_FLAG_SEQLENS);
      hdr[kNDec] = hdr[kNPre] = 0;
    }
    return;
  }
  for (int s = tid; s < N; s += kSchedThreads) {
    const int b = block(s);
    if (b < 0 || length(s) == 0) continue;  // padding or empty
    if (b >= nb) atomicOr(&s_flags, GDN_FLAG_BLOCK_RANGE);
    else if (b == 0) atomicOr(&s_flags, GDN_FLAG_TRASH_WRITE);
    else atomicAdd(&uses[b], 1);
  }
  __syncthreads();
  int32_t *pre = p.work.pre(), *pre_tmp = p.work.pre_tmp(), *first = p.work.pre_cp();
  unsigned total = 0;  // chunks of the long sequences
  for (int s = tid; s < N; s += kSchedThreads) {
    const int b = block(s), len = length(s);
    if (b <= 0 || b >= nb || len == 0) continue;
    if (atomicAdd(&uses[b], 0) > 1) {
      atomicOr(&s_flags, GDN_FLAG_DUPLICATE);
    } else if (p.hint > 0 && len > p.hint) {
      atomicOr(&s_flags, GDN_FLAG_HINT);
    } else if (len <= short_max) {
      p.work.dec()[atomicAdd(&s_dec, 1)] = s;
    } else {
      const int k = atomicAdd(&s_pre, 1), c = (len - 1) / p.chunk + 1;
      pre_tmp[k] = s;
      if (k < kSortMax) {
        found[k] = s;
        chunks[k] = c;
      }
      total += c;
    }
  }
  total = __reduce_add_sync(0xffffffffu, total);
  if ((tid & 31) == 0 && total) atomicAdd(&s_total, total);
  __syncthreads();
  const int n_pre = s_pre;
  if (tid == 0) {
    if (s_flags) atomicOr((unsigned*)&hdr[kErr], s_flags);
    hdr[kNDec] = s_dec;
    hdr[kNPre] = n_pre;
  }
  if (n_pre == 0) return;
  static_assert(kLinSlices == 4, "a head's marks are a word");
  if (p.bad)
    for (long long i = tid; i < (long long)n_pre * p.H; i += kSchedThreads)
      reinterpret_cast<uint32_t*>(p.bad)[i] = 0u;
  const bool sorted = n_pre <= kSortMax;
  // longest first, ties by sequence (so that a call's order is always the same)
  for (int i = tid; i < n_pre; i += kSchedThreads) {
    if (sorted) {
      const int ci = chunks[i], si = found[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n_pre; ++j) rank += chunks[j] > ci || (chunks[j] == ci && found[j] < si);
      pre[rank] = si;
      in_order[rank] = ci;
    } else {
      pre[i] = pre_tmp[i];
    }
  }
  __syncthreads();
  auto chunks_of = [&](int k) {
    return sorted ? in_order[k] : (p.cu[pre[k] + 1] - p.cu[pre[k]] - 1) / p.chunk + 1;
  };
  // A chain is worked off in order by one SM (token-serial form: each of its
  // 32 columns by a group of an SM's threads), so that the call takes at least
  // the longest one.  Cut into segments, which are computed side by side, it
  // takes rounds of them over the SMs, each twice: first the segments' own
  // states, then the outputs from the states at their starts.  Lengths
  // around an SM's share of all chunks are weighed; the best counts if it
  // beats the whole sequences, and of equals the longest one (fewer states to
  // write and read).  Sequences longer than half a segment count as whole ones,
  // and shorter ones fill the gaps.
  int per = 0x7fffffff;
  if (p.seg_states && sorted) {
    // (32 bits hold all of this: q, k and v of that much work would not fit)
    const unsigned chains = p.H * (slices ? slices : 1);
    const unsigned share = (s_total * chains + num_sms - 1) / num_sms;
    const unsigned longest = chunks_of(0), least = slices ? kMinSerial : kMinSegment;
    auto cost = [&](unsigned items, unsigned n, int passes) {
      const unsigned per_sm = max((items * chains + num_sms - 1) / num_sms, (share - 1) / n + 1);
      return slices ? serial_cost(n, per_sm, passes) : chunk_cost(n, per_sm, passes);
    };
    int count = 0;
    for (int k = 0; k < n_pre; k += kSchedThreads)
      count += __syncthreads_count(k + tid < n_pre && in_order[k + tid] > longest / 2);
    const unsigned whole = cost(count, longest, 1);
    const unsigned lo = max(least, share / (slices ? 4 * kSerialPerSm : 4));
    const unsigned hi = min(longest, 2 * share + least);
    const unsigned n = lo + tid / kLanes * ((hi - min(hi, lo)) / (kSchedThreads / kLanes) + 1);
    unsigned items = 0, slots = 0;
    for (int k = tid % kLanes; n < hi && k < n_pre && in_order[k] > n / 2; k += kLanes) {
      const unsigned c = in_order[k];
      items += (c + n / 2) / n;
      if (c > n) slots += (c - 1) / n + 1;
    }
#pragma unroll
    for (int w = 1; w < kLanes; w <<= 1) {
      items += __shfl_xor_sync(0xffffffffu, items, w);
      slots += __shfl_xor_sync(0xffffffffu, slots, w);
    }
    if (tid % kLanes == 0 && n < hi && slots * p.H <= p.seg_slots) {
      const unsigned mine = cost(items, n, 2);
      if (mine < whole) atomicMin(&s_best, (unsigned long long)mine << 32 | (0x7fffffffu - n));
    }
    __syncthreads();
    per = 0x7fffffff - (int)(s_best & 0x7fffffffu);
  }
  int carry = 0, n_split = 0;
  if (n_pre <= 32) {  // one warp needs no barriers
    if (tid >= 32) return;
    const int segs = tid < n_pre ? (chunks_of(tid) - 1) / per + 1 : 0;
    int upto = segs;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int before = __shfl_up_sync(0xffffffffu, upto, w);
      if (tid >= w) upto += before;
    }
    if (tid < n_pre) first[tid] = upto - segs;
    if (tid == n_pre - 1) first[n_pre] = upto;
    carry = __shfl_sync(0xffffffffu, upto, 31);
    n_split = __popc(__ballot_sync(0xffffffffu, segs > 1));
    const int split_segs = __reduce_add_sync(0xffffffffu, segs > 1 ? segs : 0);
    if (tid == 0) hdr[kLinStateItems] = split_segs;
  } else {
    for (int k0 = 0; k0 < n_pre; k0 += kSchedThreads) {
      const int k = k0 + tid;
      const int segs = k < n_pre ? (chunks_of(k) - 1) / per + 1 : 0;
      n_split += __syncthreads_count(segs > 1);
      int total;
      const int before = carry + cta_scan(segs, &total, warp_sums);
      if (k < n_pre) {
        first[k] = before;
        if (k == n_pre - 1) first[n_pre] = before + segs;
        if (segs > 1) atomicAdd(&hdr[kLinStateItems], segs);
      }
      carry += total;
    }
  }
  if (tid == 0) {
    hdr[kLinItems] = carry;
    hdr[kLinSplit] = n_split;
    hdr[kLinSegChunks] = per;
  }
}

template <typename T, int D>
cudaError_t launch_rec(const LinParams& p, int max_items, cudaStream_t s) {
  const long long ctas = (long long)max_items * p.H * (D / kSlice);
  auto kern = p.hint == 1 ? lin_recurrent_kernel<T, D, true> : lin_recurrent_kernel<T, D, false>;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kRecThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_lin_recurrent(const LinParams& p, int d, int act, int max_items,
                                 cudaStream_t s) {
  if (max_items <= 0) return cudaSuccess;
  if (act == GDN_F32) {
    if (d == 32) return launch_rec<float, 32>(p, max_items, s);
    if (d == 64) return launch_rec<float, 64>(p, max_items, s);
    return launch_rec<float, 128>(p, max_items, s);
  }
  if (d == 32) return launch_rec<__nv_bfloat16, 32>(p, max_items, s);
  if (d == 64) return launch_rec<__nv_bfloat16, 64>(p, max_items, s);
  return launch_rec<__nv_bfloat16, 128>(p, max_items, s);
}

cudaError_t launch_lin_schedule(const LinParams& p, int short_max, int num_sms, cudaStream_t s) {
  return launch_pdl(lin_schedule_kernel, dim3(1), dim3(kSchedThreads), 0, s, p, short_max, num_sms, 0);
}

cudaError_t launch_lin_segments(const LinParams& p, int num_sms, cudaStream_t s) {
  return launch_pdl(lin_segments_kernel, dim3(4 * num_sms), dim3(256), 0, s, p);
}

cudaError_t launch_lin_serial_split(const LinParams& p, int act, int num_sms, cudaStream_t s) {
  const bool f32 = act == GDN_F32;
  const size_t smem = kSerialPerSm * (p.d == 32   ? f32 ? sizeof(RecSmem<float, 32, false>)
                                                        : sizeof(RecSmem<__nv_bfloat16, 32, false>)
                                      : p.d == 64 ? f32 ? sizeof(RecSmem<float, 64, false>)
                                                        : sizeof(RecSmem<__nv_bfloat16, 64, false>)
                                                  : sizeof(RecSmem<float, 128, false>));
  auto run = [&](auto state, auto out) {
    cudaError_t e = launch_pdl(lin_schedule_kernel, dim3(1), dim3(kSchedThreads), 0, s, p, 0, num_sms,
                               p.d / kSlice);
    const dim3 grid(num_sms), block(kRecThreads * kSerialPerSm);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(state, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(out, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_pdl(state, grid, block, smem, s, p);
    if (e == cudaSuccess) e = launch_lin_segments(p, num_sms, s);
    if (e == cudaSuccess) e = launch_pdl(out, grid, block, smem, s, p);
    return e;
  };
  if (p.d == 32)
    return f32 ? run(lin_rec_segments_kernel<float, 32, true>, lin_rec_segments_kernel<float, 32, false>)
               : run(lin_rec_segments_kernel<__nv_bfloat16, 32, true>,
                     lin_rec_segments_kernel<__nv_bfloat16, 32, false>);
  if (p.d == 64)
    return f32 ? run(lin_rec_segments_kernel<float, 64, true>, lin_rec_segments_kernel<float, 64, false>)
               : run(lin_rec_segments_kernel<__nv_bfloat16, 64, true>,
                     lin_rec_segments_kernel<__nv_bfloat16, 64, false>);
  return run(lin_rec_segments_kernel<float, 128, true>, lin_rec_segments_kernel<float, 128, false>);
}

namespace {

size_t roundup(size_t v, size_t m) { return (v + m - 1) / m * m; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int check_lin_dims(int num_blocks, int num_layers, int H, int d, int act, size_t align) {
  if (num_blocks < 2 || num_layers < 1) return GDN_ERR_RANGE;
  if (H < 1 || H > 4096 || (d != 32 && d != 64 && d != 128)) return GDN_ERR_DIMS;
  if (act != GDN_F32 && act != GDN_BF16) return GDN_ERR_DIMS;
  if (align != 0 && (align < 128 || (align & (align - 1)) != 0)) return GDN_ERR_DIMS;
  if ((long long)num_blocks * num_layers > (1ll << 30)) return GDN_ERR_RANGE;
  return GDN_OK;
}

// room for segments' states: 512 of d = 128 (three per SM), more smaller ones
constexpr size_t kSegBytes = 512 * 128 * 128 * sizeof(float);

size_t lin_stride(int H, int d, size_t align) {
  return roundup((size_t)H * d * d * sizeof(float), align > 128 ? align : 128);
}

}  // namespace
}  // namespace gdn

extern "C" {

int gdn_lin_pool_layout_for(int num_blocks, int num_layers, int num_heads, int d, int act,
                            size_t block_align, size_t* block_stride, size_t* total_bytes) {
  const int st = gdn::check_lin_dims(num_blocks, num_layers, num_heads, d, act, block_align);
  if (st != GDN_OK) return st;
  const size_t stride = gdn::lin_stride(num_heads, d, block_align);
  if (block_stride) *block_stride = stride;
  if (total_bytes) *total_bytes = stride * (size_t)num_blocks * (size_t)num_layers;
  return GDN_OK;
}

int gdn_lin_pool_create(gdn_pool_t** out, int num_blocks, int num_layers, int num_heads, int d,
                        int act, size_t block_align, void* device_mem, size_t device_bytes) {
  if (!out) return GDN_ERR_NULL;
  *out = nullptr;
  int st = gdn::check_lin_dims(num_blocks, num_layers, num_heads, d, act, block_align);
  if (st != GDN_OK) return st;
  const size_t stride = gdn::lin_stride(num_heads, d, block_align);
  const size_t total = stride * (size_t)num_blocks * (size_t)num_layers;
  if (device_mem) {
    if (device_bytes < total) return GDN_ERR_NOMEM;
    if (((uintptr_t)device_mem & 255u) != 0) return GDN_ERR_ALIGN;
  }
  gdn_pool* p = new (std::nothrow) gdn_pool();
  if (!p) return GDN_ERR_NOMEM;
  p->kind = 2;
  p->num_blocks = num_blocks;
  p->num_layers = num_layers;
  p->Hv = num_heads;
  p->dk = p->dv = d;
  p->act = act;
  p->last_path = GDN_PREFILL_NONE;
  p->stride = stride;
  p->total = total;
  st = gdn::pool_allocate(p, device_mem);
  if (st != GDN_OK) {
    delete p;
    return st;
  }
  // segment states, then the chunked form's marks
  p->lin_slots = (int)(gdn::kSegBytes / ((size_t)d * d * sizeof(float)));
  const size_t marks =
      gdn::lin_chunk_supported(d, act) ? (size_t)num_blocks * num_heads * gdn::kLinSlices : 0;
  if (cudaMalloc((void**)&p->lin_states, gdn::kSegBytes + marks) != cudaSuccess) {
    cudaGetLastError();
    p->lin_states = nullptr;
    gdn_state_pool_destroy(p);
    return GDN_ERR_NOMEM;
  }
  *out = p;
  return GDN_OK;
}

int gdn_lin_varlen_forward(gdn_pool_t* p, int layer, const void* q, const void* k, const void* v,
                           int64_t ldq, int64_t ldk, int64_t ldv, int num_kv_heads,
                           const int32_t* cu_seqlens, const int32_t* state_block_idx,
                           const uint8_t* has_past, const float* log_decay, float scale, void* out,
                           int64_t ldo, int T, int N, int max_seqlen_hint, void* stream) {
  if (!p) return GDN_ERR_NULL;
  if (p->kind != 2) return GDN_ERR_DIMS;
  if (layer < 0 || layer >= p->num_layers || T < 0 || N < 0 || max_seqlen_hint < 0)
    return GDN_ERR_RANGE;
  if (num_kv_heads < 1 || p->Hv % num_kv_heads != 0) return GDN_ERR_DIMS;
  if (N == 0) return T == 0 ? GDN_OK : GDN_ERR_RANGE;
  if (!cu_seqlens || !state_block_idx || !has_past || !log_decay) return GDN_ERR_NULL;
  if (T > 0 && (!q || !k || !v || !out)) return GDN_ERR_NULL;
  const int d = p->dk, H = p->Hv;
  const int per16 = p->act == GDN_F32 ? 4 : 8;
  if (T > 0) {
    if (!gdn::aligned16(q) || !gdn::aligned16(k) || !gdn::aligned16(v) || !gdn::aligned16(out) ||
        ldq % per16 != 0 || ldk % per16 != 0 || ldv % per16 != 0 || ldo % per16 != 0)
      return GDN_ERR_ALIGN;
    const int64_t qcols = (int64_t)H * d, kcols = (int64_t)num_kv_heads * d;
    const int64_t most = (int64_t)1 << 38;
    if (ldq < qcols || ldo < qcols || ldk < kcols || ldv < kcols || ldq > most || ldk > most ||
        ldv > most || ldo > most)
      return GDN_ERR_RANGE;
  }
  int max_items = N < p->num_blocks - 1 ? N : p->num_blocks - 1;
  if (max_items > T) max_items = T;
  if ((long long)(N <= gdn::kSelfCheck ? N : max_items) * H * (d / gdn::kSlice) > 0x7fffffffll)
    return GDN_ERR_RANGE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  if (dev != p->device) return GDN_ERR_DEVICE;

  gdn::LinParams lp = {};
  lp.q = q;
  lp.k = k;
  lp.v = v;
  lp.out = out;
  lp.ldq = ldq;
  lp.ldk = ldk;
  lp.ldv = ldv;
  lp.ldo = ldo;
  lp.cu = cu_seqlens;
  lp.blk = state_block_idx;
  lp.has_past = has_past;
  lp.log_decay = log_decay;
  lp.scale = scale;
  lp.layer_base = p->base + (size_t)layer * p->num_blocks * p->stride;
  lp.stride = p->stride;
  lp.T = T;
  lp.N = N;
  lp.H = H;
  lp.group = H / num_kv_heads;
  lp.num_blocks = p->num_blocks;
  lp.hint = max_seqlen_hint;
  lp.work.base = p->work + (size_t)layer * gdn::WorkArea::words(p->num_blocks);
  lp.work.num_blocks = p->num_blocks;

  cudaStream_t s = (cudaStream_t)stream;
  const int sms = p->sms;
  // prompts in the chunked form, where it has a kernel and the call room for one
  const long long units = (long long)N * H * gdn::kLinSlices;
  const int short_max = units <= sms       ? gdn::kLinShortLone
                        : units <= 5ll * sms ? gdn::kLinShortFew
                                             : gdn::kLinShort;
  int max_long = T / (short_max + 1);
  if (max_long > max_items) max_long = max_items;
  if (max_seqlen_hint > 0 && max_seqlen_hint <= short_max) max_long = 0;
  const bool chunked = max_long > 0 && gdn::lin_chunk_supported(d, p->act);
  p->last_path = chunked                             ? GDN_PREFILL_FUSED
                 : T > 1 && max_seqlen_hint != 1 ? GDN_PREFILL_SERIAL
                                                     : GDN_PREFILL_NONE;
  // the scheduler's rule for splitting (see there) on what the host knows: no
  // sequence is longer than T or the hint, and all tokens are some sequence's
  const long long longest = max_seqlen_hint > 0 && max_seqlen_hint < T ? max_seqlen_hint : T;
  lp.seg_slots = p->lin_slots;
  lp.d = d;
  lp.chunk = chunked ? gdn::kLinChunk : gdn::kTile;
  const long long steps = (longest - 1) / lp.chunk + 1;
  // (the least that two passes can cost: all SMs busy all the time)
  const long long work = (long long)(T / lp.chunk) * H * (chunked ? 1 : d / gdn::kSlice) / sms;
  long long whole, split;
  if (chunked) {
    whole = steps;
    split = gdn::chunk_cost(work > gdn::kMinSegment ? work : gdn::kMinSegment, 1ll, 2);
  } else {
    const long long per_sm = work > gdn::kSerialPerSm * gdn::kMinSerial ? gdn::kSerialPerSm : 1;
    whole = gdn::serial_cost(steps, 1ll, 1);
    split = gdn::serial_cost(per_sm > 1 ? work / per_sm : gdn::kMinSerial, per_sm, 2);
  }
  const bool may_split = T > 0 && whole > split;
  if (chunked) lp.bad = reinterpret_cast<unsigned char*>(p->lin_states) + gdn::kSegBytes;
  if (may_split) lp.seg_states = p->lin_states;
  if (!chunked && may_split) {
    if (p->ev_before && cudaEventRecord(p->ev_before, s) != cudaSuccess) return GDN_ERR_CUDA;
    if (gdn::launch_lin_serial_split(lp, p->act, sms, s) != cudaSuccess) return GDN_ERR_CUDA;
    if (p->ev_after && cudaEventRecord(p->ev_after, s) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  lp.listed = chunked || N > gdn::kSelfCheck;
  lp.late = chunked;
  if (lp.listed && gdn::launch_lin_schedule(lp, chunked ? short_max : INT32_MAX, sms, s) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (p->ev_before && cudaEventRecord(p->ev_before, s) != cudaSuccess) return GDN_ERR_CUDA;
  if (chunked && gdn::launch_lin_chunk(lp, may_split, sms, s) != cudaSuccess) return GDN_ERR_CUDA;
  if (gdn::launch_lin_recurrent(lp, d, p->act, lp.listed ? max_items : N, s) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (p->ev_after && cudaEventRecord(p->ev_after, s) != cudaSuccess) return GDN_ERR_CUDA;
  return GDN_OK;
}

}  // extern "C"
