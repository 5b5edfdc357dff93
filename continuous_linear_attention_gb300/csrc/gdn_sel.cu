// The selective state space mixer's two stateful operations over a packed
// batch, continued from each request's states in a paged pool (the mixers with
// one decay per channel and state entry among the hybrid families of the model
// support tracker): the short causal convolution with SiLU, and, behind the
// projections that make the time step, B and C of its output, the scan
//   dt = softplus(dt_raw + dt_bias),  A = -exp(A_log)
//   h_t[n] = e^{dt A[n]} h_{t-1}[n] + dt u_t B_t[n]        (per channel, fp32)
//   y_t = (sum_n h_t[n] C_t[n] + D u_t) * silu(z_t)
// A block holds the conv state [K-1][C] (activation dtype) and the state
// [C][N] fp32.
//
// This file: the kernels and the C entry points.
#include <cuda_runtime.h>

#include <new>

#include "gdn_cta.cuh"
#include "gdn_lin.cuh"
#include "gdn_pool.cuh"
#include "gdn_seqs.cuh"

namespace gdn {
namespace {

template <typename T>
struct Vec16 {  // 16 bytes of elements
  static constexpr int kN = 16 / (int)sizeof(T);
  uint4 w;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    else return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
};
template <typename T>
__device__ __forceinline__ Vec16<T> load16(const T* p) {
  Vec16<T> v;
  v.w = *reinterpret_cast<const uint4*>(p);
  return v;
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const float* f) {
  uint4 w;
  uint32_t* u = reinterpret_cast<uint32_t*>(&w);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p2 = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&p2);
    }
  }
  *reinterpret_cast<uint4*>(p) = w;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x for a decay (x <= 0).  Near 0, where a state keeps its value over many
// steps and a bias of the exponential adds up over as many (the hardware's is
// about 2^-27 there: 2e-5 of the state after 3,000 steps of 2^-13), from its
// series, rounded to nearest: its next term is 6e-10 at -1/64, where a state
// forgets fast enough for the bias (6e-7 of it).
constexpr float kNear = -0.015625f;
constexpr float kExp1 = 6.9314718e-1f, kExp2 = 2.4022651e-1f, kExp3 = 5.5504109e-2f;
__device__ __forceinline__ float decay2(float x) {
  const float p = fmaf(x, fmaf(x, fmaf(x, kExp3, kExp2), kExp1), 1.f);
  const float a = ex2(x);
  return x > kNear ? p : a;
}
__device__ __forceinline__ F2 decay2(F2 x) {
  const F2 p = fma2(x, fma2(x, fma2(x, f2(kExp3, kExp3), f2(kExp2, kExp2)), f2(kExp1, kExp1)), f2(1.f, 1.f));
  float x0, x1, p0, p1;
  unf2(x, x0, x1);
  unf2(p, p0, p1);
  const float a0 = ex2(x0), a1 = ex2(x1);
  return f2(x0 > kNear ? p0 : a0, x1 > kNear ? p1 : a1);
}

// softplus(x) = max(x, 0) + log(1 + t), t = e^-|x|, of two values: log(1 + t) / t on
// [0, 1] is the interpolating polynomial of degree 8 at the Chebyshev points, off by
// 2e-7 relative (a small softplus, a slow step, keeps its relative precision).
__device__ __constant__ const float kLogOnePlus[9] = {
    0.9999999403953552f,  -0.4999944567680359f,  0.3331812024116516f,
    -0.2483539879322052f, 0.19076880812644958f,  -0.13602247834205627f,
    0.0775160863995552f,  -0.029074065387248993f, 0.005126102361828089f};
__device__ __forceinline__ void softplus2(float& a, float& b) {
  const float ta = ex2(-fabsf(a) * kLog2e), tb = ex2(-fabsf(b) * kLog2e);
  const F2 t = f2(ta, tb);
  F2 q = f2(kLogOnePlus[8], kLogOnePlus[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) q = fma2(q, t, f2(kLogOnePlus[i], kLogOnePlus[i]));
  unf2(fma2(q, t, f2(fmaxf(a, 0.f), fmaxf(b, 0.f))), a, b);
}

// y / (1 + e^-y) of two values.
__device__ __forceinline__ F2 silu2(F2 y) {
  float a, b;
  unf2(mul2(y, f2(-kLog2e, -kLog2e)), a, b);
  a = 1.f + ex2(a);
  b = 1.f + ex2(b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return mul2(y, f2(a, b));
}

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

// --- convolution -------------------------------------------------------------
// Bound by HBM: each input is read once (the K-1 rows before a piece twice, out
// of L2) and each output written once.  A thread owns 16 bytes of channels and
// walks the tokens of a piece with the K-1 inputs before in registers.  15,843 tokens
// x 4,096 channels, K = 4: 49 us, 5.3 TB/s; issue slots at 54%, a third of them SiLU's.
constexpr int kConvThreads = 128;
constexpr int kConvTokens = 32;  // per piece
// Places of a thread for tokens on their way to it (1: single tokens only), in shared
// memory: as registers they leave an SM three CTAs (15,843 tokens x 4,096 channels 55.2 us,
// 49.0 us so; with 16 places 54.8).
constexpr int kConvAhead = 8;
constexpr int kConvCtas = 4;

struct ConvParams {
  Batch batch;
  const void* x;
  const void* w;     // [C][K]
  const void* bias;  // [C] or NULL
  void* out;
  long long ldx, ldo;
  unsigned char* layer_base;
  size_t stride;
  int C;
  int tx;  // threads across the channels (a power of two); the others take pieces
};

template <typename T, int K, int kAhead>
__global__ void __launch_bounds__(kConvThreads, kConvCtas) sel_conv_kernel(ConvParams p) {
  constexpr int kV = Vec16<T>::kN;
  __shared__ PlanSmem plan;
  __shared__ uint4 ring[kAhead > 1 ? kAhead : 1][kConvThreads];
  pdl_wait_then_release();
  const Batch& b = p.batch;
  const SeqList list = b.listed ? listed_long(b)
                                : plan_self(b, Pieces{1, 0x7fffffff, kConvTokens}, plan, blockIdx.x == 0);
  const int vecs = p.C / kV, ch_blocks = (vecs + p.tx - 1) / p.tx, rows = kConvThreads / p.tx;
  const int tx = threadIdx.x % p.tx, ty = threadIdx.x / p.tx;
  const long long units = (long long)((list.total + rows - 1) / rows) * ch_blocks;
  // (the grid is a multiple of ch_blocks, or all units: a CTA's channels stay the same)
  const int c0 = ((int)(blockIdx.x % ch_blocks) * p.tx + tx) * kV;
  if (c0 >= p.C) return;
  F2 w[K][kV / 2], bias[kV / 2];  // channels in pairs
  {
    const T* wp = static_cast<const T*>(p.w) + (size_t)c0 * K;
    float flat[K * kV];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const Vec16<T> v = load16(wp + i * kV);
#pragma unroll
      for (int j = 0; j < kV; ++j) flat[i * kV + j] = v.at(j);
    }
#pragma unroll
    for (int j = 0; j < kV; j += 2)
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][j / 2] = f2(flat[j * K + k], flat[(j + 1) * K + k]);
    Vec16<T> v;
    v.w = make_uint4(0, 0, 0, 0);
    if (p.bias) v = load16(static_cast<const T*>(p.bias) + c0);
#pragma unroll
    for (int j = 0; j < kV; j += 2) bias[j / 2] = f2(v.at(j), v.at(j + 1));
  }
  const int* lo = kAhead > 1 || b.listed ? b.cu : plan.lo;
  const int* blocks = kAhead > 1 || b.listed ? b.blk : plan.blk;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u / ch_blocks) * rows + ty;
    if (piece >= list.total) continue;
    const int e = entry_of(list, piece), s = list.items[e];
    const int at = (piece - list.first[e]) * kConvTokens;
    const int row0 = lo[s], len = lo[s + 1] - row0, n = min(kConvTokens, len - at);
    const T* x = static_cast<const T*>(p.x) + (size_t)row0 * p.ldx + c0;
    T* out = static_cast<T*>(p.out) + (size_t)row0 * p.ldo + c0;
    Vec16<T> win[K - 1];
    if (at == 0) {
      // the state, and (only this thread reads it) its new rows: the last K-1
      // inputs, former ones among them where the sequence is short
      T* st = reinterpret_cast<T*>(p.layer_base + (size_t)blocks[s] * p.stride) + c0;
      const bool past = b.has_past[s];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        win[j].w = make_uint4(0, 0, 0, 0);
        if (past) win[j] = load16(st + (size_t)j * p.C);
      }
      Vec16<T> next[K - 1];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = len - (K - 1) + j;
        if (t >= 0) {
          next[j] = load16(x + (size_t)t * p.ldx);
        } else {
          next[j] = win[K - 2];
#pragma unroll
          for (int i = 0; i < K - 1; ++i)
            if (i == t + K - 1) next[j] = win[i];
        }
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j) *reinterpret_cast<uint4*>(st + (size_t)j * p.C) = next[j].w;
    } else {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) win[j] = load16(x + (size_t)(at - (K - 1) + j) * p.ldx);
    }
    // the copies of kAhead - 1 tokens on their way to this thread's places in shared
    // memory, each to where the token before the last one lay
    auto ahead = [&](int t) {
      if (kAhead > 1 && t < n) cp_async16(&ring[t % kAhead][threadIdx.x], x + (size_t)(at + t) * p.ldx);
      cp_async_commit();
    };
    if (kAhead > 1)
#pragma unroll
      for (int i = 0; i < kAhead - 1; ++i) ahead(i);
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      Vec16<T> in[K];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) in[j] = win[j];
      if (kAhead > 1) {
        ahead(t + kAhead - 1);
        cp_async_wait<kAhead - 1>();
        in[K - 1].w = ring[t % kAhead][threadIdx.x];
      } else {
        in[K - 1] = load16(x + (size_t)(at + t) * p.ldx);
      }
      float y[kV];
#pragma unroll
      for (int j = 0; j < kV; j += 2) {
        F2 acc = bias[j / 2];
#pragma unroll
        for (int k = 0; k < K; ++k) acc = fma2(w[k][j / 2], f2(in[k].at(j), in[k].at(j + 1)), acc);
        unf2(silu2(acc), y[j], y[j + 1]);
      }
      store16(out + (size_t)(at + t) * p.ldo, y);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) win[j] = in[j + 1];
    }
  }
}

// --- scan --------------------------------------------------------------------
struct ScanParams {
  Batch batch;
  const void *u, *dt, *B, *C, *z;  // z may be NULL
  void* y;
  long long ldu, lddt, ldb, ldc, ldz, ldy;
  const float *A_log, *D, *dt_bias;  // D and dt_bias may be NULL
  unsigned char* layer_base;
  size_t stride, ssm_off;
  int channels;
  int report;  // this kernel raises the batch's flags
  // segments of long sequences: how many there is room for (0: none), the states at
  // their starts (first their own), their steps' sums
  int slots, sms;
  float *seg_states, *seg_sums;
};

// Single tokens: each state is read once and written once.  A thread has eight
// entries of a channel's state (with four, what is done once per channel, softplus
// above all, took most of the instructions: 52 us for 256 sequences x 4,096
// channels, now 29, 4.9 TB/s); a CTA keeps its channels and walks the sequences.
constexpr int kStepThreads = 256;
constexpr int kStepCtas = 4;  // per SM: reads in flight (5: 42 us, spilled; 3: 47)

template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads, kStepCtas) sel_step_kernel(ScanParams p) {
  constexpr int kLanes = N / 8;  // threads per channel
  __shared__ PlanSmem plan;
  pdl_wait_then_release();
  const Batch& b = p.batch;
  SeqList list;
  if (b.listed) {
    list.items = b.work.dec();
    list.n = b.work.header()[kNDec];
  } else {
    list = plan_self(b, Pieces{1, 1, 1}, plan, p.report && blockIdx.x == 0 && blockIdx.y == 0);
  }
  const int c = (blockIdx.x * kStepThreads + threadIdx.x) / kLanes, g = threadIdx.x % kLanes;
  const bool live = c < p.channels;
  const size_t at = (size_t)(live ? c : 0) * N + g * 8;
  F2 A[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 al = *reinterpret_cast<const float2*>(p.A_log + at + 2 * i);
    A[i] = f2(-expf(al.x) * kLog2e, -expf(al.y) * kLog2e);
  }
  const float bias = p.dt_bias && live ? p.dt_bias[c] : 0.f, skip = p.D && live ? p.D[c] : 0.f;
  const int* lo = b.listed ? b.cu : plan.lo;
  const int* blocks = b.listed ? b.blk : plan.blk;
  // eight elements, in pairs
  auto eight = [](const T* q, F2* f) {
    if constexpr (sizeof(T) == 4) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(q), w = *reinterpret_cast<const ulonglong2*>(q + 4);
      f[0] = v.x; f[1] = v.y; f[2] = w.x; f[3] = w.y;
    } else {
      const Vec16<T> v = load16(q);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = f2(v.at(2 * i), v.at(2 * i + 1));
    }
  };
  for (int i0 = blockIdx.y; i0 < list.n; i0 += gridDim.y) {
    const int s = list.items[i0];
    const size_t row = lo[s];
    // (read whether it counts or not: no wait for has_past)
    float* st = reinterpret_cast<float*>(p.layer_base + (size_t)blocks[s] * p.stride + p.ssm_off) + at;
    const ulonglong2 h01 = *reinterpret_cast<const ulonglong2*>(st), h23 = *reinterpret_cast<const ulonglong2*>(st + 4);
    F2 h[4] = {h01.x, h01.y, h23.x, h23.y}, B[4], C[4];
    const bool past = b.has_past[s];
    const int cc = live ? c : 0;
    const float u = to_f32(static_cast<const T*>(p.u)[row * p.ldu + cc]);
    float d = to_f32(static_cast<const T*>(p.dt)[row * p.lddt + cc]) + bias;
    const float z = p.z ? to_f32(static_cast<const T*>(p.z)[row * p.ldz + cc]) : 0.f;
    eight(static_cast<const T*>(p.B) + row * p.ldb + g * 8, B);
    eight(static_cast<const T*>(p.C) + row * p.ldc + g * 8, C);
    d = softplus_f32(d);
    const F2 dd = f2(d, d), du = f2(d * u, d * u);
    F2 part = 0ull;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fma2(past ? h[i] : 0ull, decay2(mul2(dd, A[i])), mul2(du, B[i]));
      part = fma2(h[i], C[i], part);
    }
    if (live) {
      *reinterpret_cast<ulonglong2*>(st) = make_ulonglong2(h[0], h[1]);
      *reinterpret_cast<ulonglong2*>(st + 4) = make_ulonglong2(h[2], h[3]);
    }
    float y, odd;
    unf2(part, y, odd);
    y += odd;
#pragma unroll
    for (int w = 1; w < kLanes; w <<= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
    if (live && g == 0) {
      y = fmaf(skip, u, y);
      if (p.z) y *= silu_f32(z);
      static_cast<T*>(p.y)[row * p.ldy + c] = from_f32<T>(y);
    }
  }
}

// Longer sequences: a CTA walks the tokens of one sequence, or of a segment of
// it, for kCB channels, kG threads per channel with N / kG states each in
// registers, a tile of kTT tokens at a time, the next one on its way.  Bound by
// issue slots, some 250 instructions per token and channel (N = 16) by the counter:
// per state two multiplications, the exponential with its series and its choice, two
// multiply-adds, in packed pairs 14 for two states, 112 in all; some 50 for softplus,
// SiLU and the tile's way through shared memory; and some 90 that each of a channel's
// lanes repeats (loads of the step, B and C, the step's pairs, the sums across
// lanes).  15,843 tokens x 4,096 channels: 575 to 608 us, issue slots at 74%.
//
// Long sequences of few channels are cut into segments: a first pass (kState)
// computes each segment's own state (from zeros) and its steps' sum, a small
// kernel the states at the segments' starts, h_start <- e^{A sum} h_start + own, and the
// output pass runs all segments side by side.  The work is 1.7 times as much, so
// that is done where otherwise too few CTAs run or one sequence is longer than an
// SM's share of all (segment_tokens; every kernel finds the same from the lengths).
// Only a batch that every CTA lists for itself is cut (up to kSelfPlan entries), and
// only where the room holds a segment for each entry besides: 32,768 tokens x 2,048
// channels, 800 us by themselves, are one piece beside 255 single tokens (3.1 ms) or
// 256 (2.3 ms).
constexpr int kScanThreads = 256;
constexpr int kTileTokens = 32;
constexpr int kSegmentBytes = 32 << 20;  // room for states between segments
constexpr int kSegmentsMax = 8192;       // (and for their steps' sums)

// Tokens per segment for a call whose longest sequence has `longest` and all
// together `tokens`, in ch_blocks CTAs each; slots: segments there is room for.
// In units of a token of one CTA where an SM is full: alone on an SM a CTA takes
// about two for a token; a segment's first loads, and the launches, cost as much
// as some 300.
__host__ __device__ inline int segment_tokens(int longest, long long tokens, int ch_blocks, int slots,
                                              int n, int sms) {
  const long long share = (tokens * ch_blocks + sms - 1) / sms;
  const long long whole = 2ll * longest > share ? 2ll * longest : share;
  // eight of them to an SM (with four, 32,768 tokens x 2,048 channels took 1.5 times as
  // long), and never more: the grid has room for so many
  long long seg = ((share + 7) / 8 + 31) / 32 * 32;
  if (seg < 64) seg = 64;
  const long long split = share * 7 / 4 + 2 * seg + 300;
  if (split >= whole || tokens / seg + n > slots) return 0x7fffffff;
  return (int)seg;
}

template <typename T, int N, int kG, bool kState>
struct ScanSmem {
  static constexpr int kCB = kScanThreads / kG;
  static constexpr int kTT = kTileTokens;
  static constexpr int kPad = kG > 1 ? 32 / kG : 0;  // the lanes of a channel write rows of y: apart by banks
  static constexpr int kOut = kState ? 1 : kTT;
  T u[2][kTT][kCB], dt[2][kTT][kCB], z[2][kOut][kCB];
  T B[2][kTT][N], C[2][kOut][N];
  alignas(16) float Bf[kTT][N], Cf[kOut][N];
  union {
    struct {
      alignas(16) float2 step[kTT][kCB];  // dt and dt u
      float y[kOut][kCB + kPad];
    };
    PlanSmem plan;  // (before the first tile's)
  };
};

template <typename T, int N, int kG, bool kState>
__global__ void __launch_bounds__(kScanThreads) sel_scan_kernel(ScanParams p) {
  using Smem = ScanSmem<T, N, kG, kState>;
  constexpr int kCB = Smem::kCB, kTT = Smem::kTT, kNS = N / kG, kPer = 16 / (int)sizeof(T);
  extern __shared__ __align__(16) unsigned char scan_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(scan_smem);
  pdl_wait_then_release();
  const Batch& b = p.batch;
  const int ch_blocks = (p.channels + kCB - 1) / kCB;
  int seg_tokens = 0x7fffffff;
  const SeqList list =
      b.listed ? listed_long(b)
               : plan_self<true>(b, Pieces{2, 0x7fffffff, 0x7fffffff}, sm.plan, p.report && blockIdx.x == 0,
                           [&](int longest, int tokens) {
                             if (p.slots > 0)
                               seg_tokens = segment_tokens(longest, tokens, ch_blocks, p.slots, b.N, p.sms);
                             return seg_tokens;
                           });
  if (kState && seg_tokens == 0x7fffffff) return;
  const int piece = blockIdx.x / ch_blocks;
  if (piece >= list.total) return;
  const int e = entry_of(list, piece), s = list.items[e];
  const int seg = piece - list.first[e], segs = list.first[e + 1] - list.first[e];
  if (kState && seg == segs - 1) return;  // (its own state is not needed by any other)
  const int cb = (int)(blockIdx.x % ch_blocks) * kCB;  // first channel
  const int t_first = segs > 1 ? seg * seg_tokens : 0;
  const int row0 = b.cu[s] + t_first;
  const int len = segs > 1 ? min(seg_tokens, b.cu[s + 1] - row0) : b.cu[s + 1] - row0;
  const int tid = threadIdx.x, c = tid / kG, g = tid % kG;
  const bool live = cb + c < p.channels;
  const int wide = min(kCB, p.channels - cb);
  __syncthreads();  // the plan is read

  auto stage = [&](int t0, int buf) {
    const int n = min(kTT, len - t0);
    constexpr int kRow = kCB / kPer, kStates = N / kPer;
    for (int i = tid; i < n * kRow; i += kScanThreads) {
      const int t = i / kRow, x = i % kRow * kPer;
      if (x >= wide) continue;
      const size_t row = row0 + t0 + t;
      cp_async16(&sm.u[buf][t][x], static_cast<const T*>(p.u) + row * p.ldu + cb + x);
      cp_async16(&sm.dt[buf][t][x], static_cast<const T*>(p.dt) + row * p.lddt + cb + x);
      if (!kState && p.z) cp_async16(&sm.z[buf][t][x], static_cast<const T*>(p.z) + row * p.ldz + cb + x);
    }
    for (int i = tid; i < n * kStates; i += kScanThreads) {
      const int t = i / kStates, x = i % kStates * kPer;
      const size_t row = row0 + t0 + t;
      cp_async16(&sm.B[buf][t][x], static_cast<const T*>(p.B) + row * p.ldb + x);
      if (!kState) cp_async16(&sm.C[buf][t][x], static_cast<const T*>(p.C) + row * p.ldc + x);
    }
    cp_async_commit();
  };
  stage(0, 0);

  const size_t at = (size_t)(live ? cb + c : 0) * N + g * kNS;
  float* st = reinterpret_cast<float*>(p.layer_base + (size_t)b.blk[s] * p.stride + p.ssm_off) + at;
  float* slot = p.seg_states + (size_t)piece * p.channels * N + at;
  const float* from = kState ? nullptr : segs > 1 ? slot : b.has_past[s] ? st : nullptr;
  F2 h[kNS / 2], A[kNS / 2];
#pragma unroll
  for (int i = 0; i < kNS / 2; ++i) {
    h[i] = from ? f2(from[2 * i], from[2 * i + 1]) : 0ull;
    A[i] = f2(-expf(p.A_log[at + 2 * i]) * kLog2e, -expf(p.A_log[at + 2 * i + 1]) * kLog2e);
  }
  // a thread's channels of a tile's other work: two of them, the same ones always
  // (a half of a 32-bit word of bf16 each)
  constexpr int kPairs = kCB / 2;
  const int xc = tid % kPairs * 2;
  const bool x_live = xc < wide;
  float bias[2] = {0.f, 0.f}, skip[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (p.dt_bias && x_live) bias[k] = p.dt_bias[cb + xc + k];
    if (p.D && x_live) skip[k] = p.D[cb + xc + k];
  }
  auto two = [](const T* q, float& a, float& b2) {
    if constexpr (sizeof(T) == 4) {
      const float2 v = *reinterpret_cast<const float2*>(q);
      a = v.x;
      b2 = v.y;
    } else {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(q);
      a = __uint_as_float(v << 16);
      b2 = __uint_as_float(v & 0xffff0000u);
    }
  };
  for (int t0 = 0, buf = 0; t0 < len; t0 += kTT, buf ^= 1) {
    const int n = min(kTT, len - t0);
    if (t0 + kTT < len) {
      stage(t0 + kTT, buf ^ 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();  // the tile has landed, and the last one's y is read
    // the time steps, and B and C in fp32
    for (int t = tid / kPairs; t < n; t += kScanThreads / kPairs) {
      if (!x_live) break;
      float d[2], u[2];
      two(&sm.dt[buf][t][xc], d[0], d[1]);
      two(&sm.u[buf][t][xc], u[0], u[1]);
      d[0] += bias[0];
      d[1] += bias[1];
      softplus2(d[0], d[1]);
      if (kState) {
        sum[0] += d[0];
        sum[1] += d[1];
      }
      *reinterpret_cast<float4*>(&sm.step[t][xc]) = make_float4(d[0], d[0] * u[0], d[1], d[1] * u[1]);
    }
    for (int i = 2 * tid; i < n * N; i += 2 * kScanThreads) {
      two(&sm.B[buf][0][0] + i, (&sm.Bf[0][0])[i], (&sm.Bf[0][0])[i + 1]);
      if (!kState) two(&sm.C[buf][0][0] + i, (&sm.Cf[0][0])[i], (&sm.Cf[0][0])[i + 1]);
    }
    __syncthreads();
    auto token = [&](int t) {
      const float2 d = sm.step[t][c];
      const F2 dd = f2(d.x, d.x), du = f2(d.y, d.y);
      [[maybe_unused]] F2 part = 0ull;
      if constexpr (kNS == 2) {
        h[0] = fma2(h[0], decay2(mul2(dd, A[0])), mul2(du, *reinterpret_cast<const F2*>(&sm.Bf[t][g * 2])));
        if constexpr (!kState) part = mul2(h[0], *reinterpret_cast<const F2*>(&sm.Cf[t][g * 2]));
      }
#pragma unroll
      for (int i = 0; i + 2 <= kNS / 2; i += 2) {
        const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(&sm.Bf[t][g * kNS + 2 * i]);
        h[i] = fma2(h[i], decay2(mul2(dd, A[i])), mul2(du, b2.x));
        h[i + 1] = fma2(h[i + 1], decay2(mul2(dd, A[i + 1])), mul2(du, b2.y));
        if constexpr (!kState) {
          const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(&sm.Cf[t][g * kNS + 2 * i]);
          part = i == 0 ? mul2(h[i], c2.x) : fma2(h[i], c2.x, part);
          part = fma2(h[i + 1], c2.y, part);
        }
      }
      float even = 0.f, odd = 0.f;
      if constexpr (!kState) unf2(part, even, odd);
      return even + odd;
    };
    // the sums over a channel's lanes: lane k ends up with token k's
    auto across = [&](float* part) {
#pragma unroll
      for (int w = kG / 2; w >= 1; w >>= 1) {
#pragma unroll
        for (int i = 0; i < w; ++i) {
          const bool up = g & w;
          const float send = up ? part[i] : part[i + w], keep = up ? part[i + w] : part[i];
          part[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
      }
      return part[0];
    };
    int t = 0;
    for (; t + kG <= n; t += kG) {
      float part[kG];
#pragma unroll
      for (int k = 0; k < kG; ++k) part[k] = token(t + k);
      if constexpr (!kState) sm.y[t + g][c] = across(part);
    }
    if (t < n) {
      float part[kG];
#pragma unroll
      for (int k = 0; k < kG; ++k) part[k] = t + k < n ? token(t + k) : 0.f;
      if constexpr (!kState) {
        const float y = across(part);
        if (t + g < n) sm.y[t + g][c] = y;
      }
    }
    __syncthreads();
    if constexpr (!kState) {
      for (int q = tid / kPairs; q < n; q += kScanThreads / kPairs) {
        if (!x_live) break;
        float u[2], y[2];
        two(&sm.u[buf][q][xc], u[0], u[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) y[k] = fmaf(skip[k], u[k], sm.y[q][xc + k]);
        if (p.z) {
          float z[2];
          two(&sm.z[buf][q][xc], z[0], z[1]);
          unf2(mul2(f2(y[0], y[1]), silu2(f2(z[0], z[1]))), y[0], y[1]);
        }
        T* out = static_cast<T*>(p.y) + (size_t)(row0 + t0 + q) * p.ldy + cb + xc;
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float2*>(out) = make_float2(y[0], y[1]);
        } else {
          *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(y[0], y[1]);
        }
      }
      __syncthreads();  // the buffer may be staged over
    }
  }
  if (live && (kState || seg == segs - 1)) {
    float* to = kState ? slot : st;
#pragma unroll
    for (int i = 0; i < kNS / 2; ++i) unf2(h[i], to[2 * i], to[2 * i + 1]);
  }
  if constexpr (kState) {
    // the steps' sums, over the threads that share a pair of channels
    __syncthreads();
    float2* room = &sm.step[0][0];
    room[tid] = make_float2(sum[0], sum[1]);
    __syncthreads();
    if (tid < kPairs && x_live) {
      float2 all = make_float2(0.f, 0.f);
      for (int i = tid; i < kScanThreads; i += kPairs) {
        all.x += room[i].x;
        all.y += room[i].y;
      }
      *reinterpret_cast<float2*>(p.seg_sums + (size_t)piece * p.channels + cb + xc) = all;
    }
  }
}

// The states at the segments' starts, in the place of their own ones: a thread
// per state entry, a chain of as many steps as there are segments.
template <int kCB>
__global__ void __launch_bounds__(256) sel_segments_kernel(ScanParams p, int n_states) {
  __shared__ PlanSmem plan;
  pdl_wait_then_release();
  const Batch& b = p.batch;
  int seg_tokens = 0x7fffffff;
  const SeqList list = plan_self<true>(b, Pieces{2, 0x7fffffff, 0x7fffffff}, plan, false, [&](int longest, int tokens) {
    return seg_tokens = segment_tokens(longest, tokens, (p.channels + kCB - 1) / kCB, p.slots, b.N, p.sms);
  });
  if (seg_tokens == 0x7fffffff) return;
  const int words = p.channels * n_states, parts = (words + 255) / 256;
  for (int u = blockIdx.x; u < list.n * parts; u += gridDim.x) {
    const int e = u / parts, at = u % parts * 256 + threadIdx.x;
    const int first = list.first[e], segs = list.first[e + 1] - first;
    if (segs < 2 || at >= words) continue;
    const int s = list.items[e], c = at / n_states;
    const float A = -expf(p.A_log[at]) * kLog2e;
    float h = b.has_past[s]
                  ? reinterpret_cast<const float*>(p.layer_base + (size_t)b.blk[s] * p.stride + p.ssm_off)[at]
                  : 0.f;
    constexpr int kAhead = 8;
    for (int i0 = 0; i0 < segs; i0 += kAhead) {
      float own[kAhead], sum[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < segs - 1) {  // (the last one's own state is not there)
          own[i] = p.seg_states[(size_t)(first + i0 + i) * words + at];
          sum[i] = p.seg_sums[(size_t)(first + i0 + i) * p.channels + c];
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i0 + i >= segs) break;
        p.seg_states[(size_t)(first + i0 + i) * words + at] = h;
        // (an infinite state stays infinite, as it does step by step, where the segment's decay
        // is too small for fp32: the least normal number in its place)
        const float x = sum[i] * A, decay = decay2(x);
        h = fmaf(h, isinf(h) && x > -INFINITY ? fmaxf(decay, 1.17549435e-38f) : decay, own[i]);
      }
    }
  }
}

template <typename T, int N, int kG, bool kState>
cudaError_t launch_scan_pass(const ScanParams& p, long long pieces, cudaStream_t s) {
  constexpr int kCB = kScanThreads / kG;
  auto kern = sel_scan_kernel<T, N, kG, kState>;
  const size_t smem = sizeof(ScanSmem<T, N, kG, kState>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(pieces * ((p.channels + kCB - 1) / kCB))), dim3(kScanThreads), smem,
                    s, p);
}

template <typename T, int N, int kG>
cudaError_t launch_scan(ScanParams p, int max_items, cudaStream_t s) {
  constexpr int kCB = kScanThreads / kG;
  const int ch_blocks = (p.channels + kCB - 1) / kCB;
  // What the segments' rule can say for any lengths that the call may have: none if
  // the longest possible one is not worth it.
  long long pieces = max_items;
  const Batch& b = p.batch;
  const int longest = b.hint > 0 && b.hint < b.T ? b.hint : b.T;
  if (b.listed || p.slots < 2 ||
      segment_tokens(longest, b.T, ch_blocks, 0x7fffffff, b.N, p.sms) == 0x7fffffff) {
    p.slots = 0;
  } else {
    pieces += 8ll * p.sms / ch_blocks + 1;  // (segments are an eighth of an SM's share at least)
    cudaError_t e = launch_scan_pass<T, N, kG, true>(p, pieces, s);
    if (e == cudaSuccess) {
      p.report = 0;
      e = launch_pdl(sel_segments_kernel<kCB>, dim3(4 * p.sms), dim3(256), 0, s, p, N);
    }
    if (e != cudaSuccess) return e;
  }
  return launch_scan_pass<T, N, kG, false>(p, pieces, s);
}

template <typename T, int N>
cudaError_t launch_step(const ScanParams& p, int max_items, int sms, cudaStream_t s) {
  const int per = kStepThreads / (N / 8), x = (p.channels + per - 1) / per;
  int y = (kStepCtas * sms + x - 1) / x;
  if (y > max_items) y = max_items;
  return launch_pdl(sel_step_kernel<T, N>, dim3(x, y), dim3(kStepThreads), 0, s, p);
}

template <typename T>
cudaError_t launch_scan_of(const ScanParams& p, int n, int max_long, int max_one, int sms,
                           cudaStream_t s) {
  ScanParams q = p;
  cudaError_t e = cudaSuccess;
  q.report = 1;
  if (max_long > 0) {
    // (whole sequences with two states to a thread, segments with four: 593 and 645 us
    // for 15,843 tokens x 4,096 channels, 922 and 806 (now 799) for 32,768 x 2,048)
    const Batch& b = q.batch;
    const int longest = b.hint > 0 && b.hint < b.T ? b.hint : b.T;
    const bool whole = b.listed || segment_tokens(longest, b.T, (q.channels + 63) / 64, q.slots, b.N, sms) == 0x7fffffff;
    e = n == 16   ? whole ? launch_scan<T, 16, 8>(q, max_long, s) : launch_scan<T, 16, 4>(q, max_long, s)
        : n == 32 ? launch_scan<T, 32, 4>(q, max_long, s)
                  : launch_scan<T, 64, 8>(q, max_long, s);
    q.report = 0;
  }
  if (max_one > 0 && e == cudaSuccess)
    e = n == 16   ? launch_step<T, 16>(q, max_one, sms, s)
        : n == 32 ? launch_step<T, 32>(q, max_one, sms, s)
                  : launch_step<T, 64>(q, max_one, sms, s);
  return e;
}

template <typename T>
cudaError_t launch_conv(const ConvParams& p, int K, unsigned ctas, cudaStream_t s) {
  auto kern = p.batch.hint == 1
                  ? K == 2 ? sel_conv_kernel<T, 2, 1> : K == 3 ? sel_conv_kernel<T, 3, 1> : sel_conv_kernel<T, 4, 1>
              : K == 2 ? sel_conv_kernel<T, 2, kConvAhead>
              : K == 3 ? sel_conv_kernel<T, 3, kConvAhead>
                       : sel_conv_kernel<T, 4, kConvAhead>;
  return launch_pdl(kern, dim3(ctas), dim3(kConvThreads), 0, s, p);
}

size_t roundup(size_t v, size_t m) { return (v + m - 1) / m * m; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int kMaxChannels = 65536;

int check_sel_dims(int num_blocks, int num_layers, int C, int N, int K, int act, size_t align) {
  if (num_blocks < 2 || num_layers < 1) return GDN_ERR_RANGE;
  if (C < 8 || C % 8 != 0 || C > kMaxChannels || (N != 16 && N != 32 && N != 64)) return GDN_ERR_DIMS;
  if (K < 2 || K > kMaxConvK) return GDN_ERR_DIMS;
  if (act != GDN_F32 && act != GDN_BF16) return GDN_ERR_DIMS;
  if (align != 0 && (align < 128 || (align & (align - 1)) != 0)) return GDN_ERR_DIMS;
  if ((long long)num_blocks * num_layers >= (1ll << 30)) return GDN_ERR_RANGE;
  return GDN_OK;
}

size_t sel_ssm_off(int C, int K, int act) {
  return roundup((size_t)(K - 1) * C * (act == GDN_F32 ? 4 : 2), 128);
}
size_t sel_stride(int C, int N, int K, int act, size_t align) {
  return roundup(sel_ssm_off(C, K, act) + (size_t)C * N * sizeof(float), align > 128 ? align : 128);
}

// What both forwards check, in the order of the other forwards' checks.
// *empty: nothing to do.
int check_sel_call(const gdn_pool_t* p, int layer, int T, int N, int hint, bool* empty) {
  *empty = false;
  if (!p) return GDN_ERR_NULL;
  if (p->kind != 3) return GDN_ERR_DIMS;
  if (layer < 0 || layer >= p->num_layers || T < 0 || N < 0 || hint < 0) return GDN_ERR_RANGE;
  if (N == 0) {
    *empty = true;
    return T == 0 ? GDN_OK : GDN_ERR_RANGE;
  }
  return GDN_OK;
}

// A row-wise tensor: [T] rows of cols elements, pitch ld.
int check_rows(const void* t, int64_t ld, int64_t cols, int act) {
  if (!aligned16(t) || ld % (act == GDN_F32 ? 4 : 8) != 0) return GDN_ERR_ALIGN;
  return ld < cols || ld > (int64_t)1 << 38 ? GDN_ERR_RANGE : GDN_OK;
}

Batch batch_of(gdn_pool_t* p, int layer, const int32_t* cu, const int32_t* blk,
               const uint8_t* has_past, int T, int N, int hint) {
  Batch b = {};
  b.cu = cu;
  b.blk = blk;
  b.has_past = has_past;
  b.N = N;
  b.T = T;
  b.num_blocks = p->num_blocks;
  b.hint = hint;
  b.listed = N > kSelfPlan;
  b.work.base = p->work + (size_t)layer * WorkArea::words(p->num_blocks);
  b.work.num_blocks = p->num_blocks;
  return b;
}

}  // namespace
}  // namespace gdn

extern "C" {

int gdn_sel_pool_layout_for(int num_blocks, int num_layers, int channels, int d_state, int conv_k,
                            int act, size_t block_align, size_t* block_stride, size_t* conv_off,
                            size_t* ssm_off, size_t* total_bytes) {
  const int st = gdn::check_sel_dims(num_blocks, num_layers, channels, d_state, conv_k, act, block_align);
  if (st != GDN_OK) return st;
  const size_t stride = gdn::sel_stride(channels, d_state, conv_k, act, block_align);
  if (block_stride) *block_stride = stride;
  if (conv_off) *conv_off = 0;
  if (ssm_off) *ssm_off = gdn::sel_ssm_off(channels, conv_k, act);
  if (total_bytes) *total_bytes = stride * (size_t)num_blocks * (size_t)num_layers;
  return GDN_OK;
}

int gdn_sel_pool_create(gdn_pool_t** out, int num_blocks, int num_layers, int channels, int d_state,
                        int conv_k, int act, size_t block_align, void* device_mem,
                        size_t device_bytes) {
  if (!out) return GDN_ERR_NULL;
  *out = nullptr;
  int st = gdn::check_sel_dims(num_blocks, num_layers, channels, d_state, conv_k, act, block_align);
  if (st != GDN_OK) return st;
  const size_t stride = gdn::sel_stride(channels, d_state, conv_k, act, block_align);
  const size_t total = stride * (size_t)num_blocks * (size_t)num_layers;
  if (device_mem) {
    if (device_bytes < total) return GDN_ERR_NOMEM;
    if (((uintptr_t)device_mem & 255u) != 0) return GDN_ERR_ALIGN;
  }
  gdn_pool* p = new (std::nothrow) gdn_pool();
  if (!p) return GDN_ERR_NOMEM;
  p->kind = 3;
  p->num_blocks = num_blocks;
  p->num_layers = num_layers;
  p->sel_C = channels;
  p->sel_N = d_state;
  p->K = conv_k;
  p->act = act;
  p->last_path = GDN_PREFILL_NONE;
  p->stride = stride;
  p->rec_off = gdn::sel_ssm_off(channels, conv_k, act);
  p->total = total;
  st = gdn::pool_allocate(p, device_mem);
  if (st != GDN_OK) {
    delete p;
    return st;
  }
  // states between segments, and their steps' sums (less than that again)
  if (cudaMalloc(&p->sel_room, gdn::kSegmentBytes + gdn::kSegmentBytes / 16) != cudaSuccess) {
    cudaGetLastError();
    p->sel_room = nullptr;
    gdn_state_pool_destroy(p);
    return GDN_ERR_NOMEM;
  }
  *out = p;
  return GDN_OK;
}

int gdn_sel_conv_varlen_forward(gdn_pool_t* p, int layer, const void* x, int64_t ldx,
                                const int32_t* cu_seqlens, const int32_t* state_block_idx,
                                const uint8_t* has_past, const void* conv_w, const void* conv_b,
                                void* out, int64_t ldo, int T, int N, int max_seqlen_hint,
                                void* stream) {
  bool empty;
  int st = gdn::check_sel_call(p, layer, T, N, max_seqlen_hint, &empty);
  if (st != GDN_OK || empty) return st;
  if (!cu_seqlens || !state_block_idx || !has_past || !conv_w || (T > 0 && (!x || !out)))
    return GDN_ERR_NULL;
  if (!gdn::aligned16(conv_w) || !gdn::aligned16(conv_b)) return GDN_ERR_ALIGN;
  if (T > 0) {
    st = gdn::check_rows(x, ldx, p->sel_C, p->act);
    if (st == GDN_OK) st = gdn::check_rows(out, ldo, p->sel_C, p->act);
    if (st != GDN_OK) return st;
  }
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  if (dev != p->device) return GDN_ERR_DEVICE;
  gdn::ConvParams cp = {};
  cp.batch = gdn::batch_of(p, layer, cu_seqlens, state_block_idx, has_past, T, N, max_seqlen_hint);
  cp.x = x;
  cp.w = conv_w;
  cp.bias = conv_b;
  cp.out = out;
  cp.ldx = ldx;
  cp.ldo = ldo;
  cp.layer_base = p->base + (size_t)layer * p->num_blocks * p->stride;
  cp.stride = p->stride;
  cp.C = p->sel_C;
  const int vecs = cp.C / (p->act == GDN_F32 ? 4 : 8);
  cp.tx = 1;
  while (cp.tx < vecs && cp.tx < gdn::kConvThreads) cp.tx *= 2;
  const int ch_blocks = (vecs + cp.tx - 1) / cp.tx, rows = gdn::kConvThreads / cp.tx;
  // pieces, at most: every sequence's last one, and the full ones
  long long pieces = (long long)T / gdn::kConvTokens + (N < T ? N : T);
  if (pieces < 1) pieces = 1;
  const long long units = (pieces + rows - 1) / rows * ch_blocks;
  // (CTAs per SM: for single tokens fewer, as each lists the batch first: 256 of them x
  // 4,096 channels 8.6 us with 4, 11.2 with 12; 15,843 tokens 51.4 with 4, 49.0 with 8,
  // 51.0 with 16)
  const int per_ch = (max_seqlen_hint == 1 ? 4 : 8) * p->sms / ch_blocks;
  long long ctas = (long long)(per_ch > 0 ? per_ch : 1) * ch_blocks;
  if (ctas > units) ctas = units;
  cudaStream_t s = (cudaStream_t)stream;
  if (cp.batch.listed &&
      gdn::launch_plan(cp.batch, gdn::Pieces{1, 0x7fffffff, gdn::kConvTokens}, s) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (p->ev_before && cudaEventRecord(p->ev_before, s) != cudaSuccess) return GDN_ERR_CUDA;
  const cudaError_t e = p->act == GDN_F32
                            ? gdn::launch_conv<float>(cp, p->K, (unsigned)ctas, s)
                            : gdn::launch_conv<__nv_bfloat16>(cp, p->K, (unsigned)ctas, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  if (p->ev_after && cudaEventRecord(p->ev_after, s) != cudaSuccess) return GDN_ERR_CUDA;
  return GDN_OK;
}

int gdn_sel_scan_varlen_forward(gdn_pool_t* p, int layer, const void* u, int64_t ldu, const void* dt,
                                int64_t lddt, const void* B, int64_t ldb, const void* C, int64_t ldc,
                                const void* z, int64_t ldz, const int32_t* cu_seqlens,
                                const int32_t* state_block_idx, const uint8_t* has_past,
                                const gdn_sel_weights_t* w, void* y, int64_t ldy, int T, int N,
                                int max_seqlen_hint, void* stream) {
  if (!w) return GDN_ERR_NULL;
  bool empty;
  int st = gdn::check_sel_call(p, layer, T, N, max_seqlen_hint, &empty);
  if (st != GDN_OK || empty) return st;
  if (!cu_seqlens || !state_block_idx || !has_past || !w->A_log ||
      (T > 0 && (!u || !dt || !B || !C || !y)))
    return GDN_ERR_NULL;
  if (!gdn::aligned16(w->A_log)) return GDN_ERR_ALIGN;
  if (T > 0) {
    const int chan = p->sel_C, n = p->sel_N;
    st = gdn::check_rows(u, ldu, chan, p->act);
    if (st == GDN_OK) st = gdn::check_rows(dt, lddt, chan, p->act);
    if (st == GDN_OK) st = gdn::check_rows(B, ldb, n, p->act);
    if (st == GDN_OK) st = gdn::check_rows(C, ldc, n, p->act);
    if (st == GDN_OK && z) st = gdn::check_rows(z, ldz, chan, p->act);
    if (st == GDN_OK) st = gdn::check_rows(y, ldy, chan, p->act);
    if (st != GDN_OK) return st;
  }
  // (the grid: a CTA per sequence and 8 channels, at most)
  if ((long long)N * (p->sel_C / 8) > 0x7fffffffll) return GDN_ERR_RANGE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  if (dev != p->device) return GDN_ERR_DEVICE;
  gdn::ScanParams sp = {};
  sp.batch = gdn::batch_of(p, layer, cu_seqlens, state_block_idx, has_past, T, N, max_seqlen_hint);
  sp.u = u;
  sp.dt = dt;
  sp.B = B;
  sp.C = C;
  sp.z = z;
  sp.y = y;
  sp.ldu = ldu;
  sp.lddt = lddt;
  sp.ldb = ldb;
  sp.ldc = ldc;
  sp.ldz = ldz;
  sp.ldy = ldy;
  sp.A_log = w->A_log;
  sp.D = w->D;
  sp.dt_bias = w->dt_bias;
  sp.layer_base = p->base + (size_t)layer * p->num_blocks * p->stride;
  sp.stride = p->stride;
  sp.ssm_off = p->rec_off;
  sp.channels = p->sel_C;
  sp.sms = p->sms;
  const size_t state_bytes = (size_t)p->sel_C * p->sel_N * sizeof(float);
  sp.slots = (int)(gdn::kSegmentBytes / state_bytes);
  if (sp.slots > gdn::kSegmentsMax) sp.slots = gdn::kSegmentsMax;
  sp.seg_states = static_cast<float*>(p->sel_room);
  sp.seg_sums = sp.seg_states + gdn::kSegmentBytes / sizeof(float);
  // what the call can hold: single tokens, and longer sequences
  int max_one = N < p->num_blocks - 1 ? N : p->num_blocks - 1;
  if (max_one > T) max_one = T;
  int max_long = max_one < T / 2 ? max_one : T / 2;
  if (max_seqlen_hint == 1) max_long = 0;
  if (N == 1 && T > 1) max_one = 0;
  if (max_one == 0 && max_long == 0) max_one = 1;  // (a kernel that looks at the batch)
  p->last_path = max_long > 0 ? GDN_PREFILL_SERIAL : GDN_PREFILL_NONE;
  cudaStream_t s = (cudaStream_t)stream;
  if (sp.batch.listed && gdn::launch_plan(sp.batch, gdn::Pieces{2, 0x7fffffff, 0x7fffffff}, s) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (p->ev_before && cudaEventRecord(p->ev_before, s) != cudaSuccess) return GDN_ERR_CUDA;
  const cudaError_t e =
      p->act == GDN_F32
          ? gdn::launch_scan_of<float>(sp, p->sel_N, max_long, max_one, p->sms, s)
          : gdn::launch_scan_of<__nv_bfloat16>(sp, p->sel_N, max_long, max_one, p->sms, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  if (p->ev_after && cudaEventRecord(p->ev_after, s) != cudaSuccess) return GDN_ERR_CUDA;
  return GDN_OK;
}

}  // extern "C"
