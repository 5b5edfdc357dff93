// Norms of queries and keys for each head with the position rotation in the
// same pass, as the attention layers beside the linear ones in hybrid models
// apply them before the attention (and as gdn_lin_varlen_forward's callers may):
//   y = x / sqrt(mean_c(x_c^2) + eps) * (w + weight_offset)   (where w is given)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin),  angle = position * inv_freq
// for channel pairs (c, c + rot/2), or (2c, 2c + 1) interleaved, of the first
// rot channels.
//
// Bound by HBM: each element is read once and written once.  A head's row is
// worked on by d/16 threads, each with the two runs of 8 channels whose halves
// belong together, so that the rotation needs no other thread; the sum of
// squares is the only thing that crosses lanes.  A warp takes as many tokens side
// by side as it has groups of d/16 threads and walks its share of their heads,
// over the next tokens' where the share is longer: every warp has the same work,
// and a token's sines and cosines are made once (CTAs of 32 whole tokens each came
// in 1.6 waves: 62 us).  The copies of the next rows are on their way meanwhile.
// 15,843 tokens x 40 heads x 128: 56.4 us, 5.75 TB/s.
#include <cuda_runtime.h>

#include <type_traits>

#include "gdn_cta.cuh"
#include "gdn_internal.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
// Places of a thread for rows on their way, and CTAs of an SM: 56.1 us with 4 and 2, 56.4
// with 3 and 2, 58.4 with 6 and 2, 62.1 with 4 and 3 (more warps are at more places of the
// memory at a time), 74 with 8 and 1.
constexpr int kRopeAhead = 4, kRopeCtas = 2;

struct RopeParams {
  const void *q, *k;
  void *q_out, *k_out;
  long long ldq, ldk, ldqo, ldko;  // row pitches, elements
  const int32_t* positions;        // [T]
  const float *q_weight, *k_weight;  // [d], or NULL: no norm
  const float* inv_freq;             // [rot / 2]
  float eps, offset;
  int T, H, Hkv, d, rot, interleaved;
  long long rows;  // of a warp: one head of its tokens each
  int per;         // rows a warp takes
};

// A run of 8 channels, as it lies.
template <typename T>
struct Run8 {
  uint4 w[sizeof(T) / 2];
  // the copy to this thread's places in shared memory, a row of them for 16 bytes
  static __device__ __forceinline__ void fetch(uint4 (*to)[kRopeThreads], const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&to[i][threadIdx.x])),
                   "l"(reinterpret_cast<const uint4*>(p) + i)
                   : "memory");
  }
  __device__ __forceinline__ void take(const uint4 (*from)[kRopeThreads]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = from[i][threadIdx.x];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
  }
};

// A frequency / 2 pi as a 64-bit fraction of a turn.  An angle is its product with the
// position modulo 2^64, off by 2^-32 of a turn at position 2^31 (an fp32 angle would be
// off by 0.06 at position 10^6).  1 / 2 pi enters in two doubles, so that the fraction is
// right to 2^-63 for frequencies up to 2^40 (in one, what is off by 2^-54 of the frequency
// grows with the position: 3e-4 at position 2^31 for a frequency of 1,000).
__device__ __forceinline__ unsigned long long turns_of(float frequency) {
  constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18, kOne = 18446744073709551616.0;
  const double f = fabs((double)frequency), high = f * kHigh;
  double low = fma(f, kLow, fma(f, kHigh, -high));  // f / 2 pi = high + low
  const double part = high - floor(high);
  low -= rint(low);
  if (!(part < 1.0)) return 0ull;  // (a frequency that is not finite)
  const unsigned long long turns = (unsigned long long)(part * kOne) + (unsigned long long)__double2ll_rn(low * kOne);
  return frequency < 0.f ? 0ull - turns : turns;
}

template <typename T, int D, bool kAny>
struct RopeSmem {
  static constexpr int kWords = sizeof(T) / 2;  // 16 bytes each, of a run
  uint4 ring[kRopeAhead][2 * kWords][kRopeThreads];
  unsigned long long turns[D / 2];  // turns_of each frequency
  float rows[kAny ? kRopeThreads * 16 : 1];
};

// kAny: a rotated half that is no multiple of 8 channels (and not interleaved),
// whose pairs lie in different threads' runs: they meet in shared memory.
template <typename T, int D, bool kAny>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(RopeParams p) {
  constexpr int kLanes = D / 16;  // threads per head
  constexpr int kAhead = kRopeAhead;
  extern __shared__ __align__(16) unsigned char rope_smem[];
  using Smem = RopeSmem<T, D, kAny>;
  constexpr int kWords = Smem::kWords;
  Smem& sm = *reinterpret_cast<Smem*>(rope_smem);
  pdl_wait_then_release();
  const int lane = threadIdx.x % kLanes;
  const int half = p.rot / 2;
  // this thread's two runs
  const bool apart = !kAny && !p.interleaved && lane < half / 8;  // those of a half and of the other
  const int ca = apart ? 8 * lane : 16 * lane, cb = apart ? ca + half : ca + 8;
  // the warp's rows: of kTokens tokens side by side, head by head
  constexpr int kTokens = 32 / kLanes;
  const int heads = p.H + p.Hkv, side = threadIdx.x % 32 / kLanes;
  const long long r0 = ((long long)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32) * p.per;
  const int n = (int)min((long long)p.per, max(0ll, p.rows - r0));
  long long token = r0 / heads * kTokens + side;
  int h = (int)(r0 % heads);
  // kAhead - 1 rows on their way (queries, then keys), each to where the one before the
  // last lay: the first ones while the angles are made
  long long token_in = token;
  int h_in = h, in = 0;
  auto ahead = [&]() {
    if (in < n) {
      if (token_in < p.T) {
        const T* src = h_in < p.H ? static_cast<const T*>(p.q) + token_in * p.ldq + (size_t)h_in * D
                                  : static_cast<const T*>(p.k) + token_in * p.ldk + (size_t)(h_in - p.H) * D;
        Run8<T>::fetch(sm.ring[in % kAhead], src + ca);
        Run8<T>::fetch(sm.ring[in % kAhead] + kWords, src + cb);
      }
      if (++h_in == heads) {
        h_in = 0;
        token_in += kTokens;
      }
    }
    ++in;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) ahead();
  int pos = token < p.T ? p.positions[token] : -1, pos_next = -1;
  if ((int)threadIdx.x < half) sm.turns[threadIdx.x] = turns_of(p.inv_freq[threadIdx.x]);
  __syncthreads();
  // the turns of a token's pairs, or (kAny) of their channels
  constexpr int kTurns = kAny ? 16 : 8;
  float co[kTurns], si[kTurns];
  auto turn = [&]() {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      co[i] = 1.f;
      si[i] = 0.f;
      int of = 8 * lane + i;  // the pair, in either order
      if (kAny) {
        of = ca + i;
        of = of < half ? of : of < 2 * half ? of - half : half;
      }
      if (pos >= 0 && of < half) {
        const unsigned long long a = sm.turns[of] * (unsigned long long)(unsigned)pos;
        sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &si[i], &co[i]);
      }
    }
  };
  // the lanes of one head: they come to its sum together or not at all
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const float* weight = nullptr;
  T* dst = nullptr;
  float wa[8], wb[8];
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    if (i == 0 || h == 0) {
      if (i > 0) pos = pos_next;
      turn();
      // (a position ahead of its token)
      pos_next = token + kTokens < p.T ? p.positions[token + kTokens] : -1;
    }
    if (i == 0 || h == 0 || h == p.H) {
      weight = h < p.H ? p.q_weight : p.k_weight;
      dst = h < p.H ? static_cast<T*>(p.q_out) + token * p.ldqo + (size_t)h * D
                    : static_cast<T*>(p.k_out) + token * p.ldko + (size_t)(h - p.H) * D;
      if (weight) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          wa[i] = weight[ca + i] + p.offset;
          wb[i] = weight[cb + i] + p.offset;
        }
      }
    }
    ahead();
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    // (the rows of no token, or of one without a position: not read and not written)
    if (pos >= 0) {
      Run8<T> ra, rb;
      ra.take(sm.ring[i % kAhead]);
      rb.take(sm.ring[i % kAhead] + kWords);
      float a[8], b[8];
      ra.get(a);
      rb.get(b);
      if (weight) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
        for (int w = 1; w < kLanes; w <<= 1) sum += __shfl_xor_sync(mask, sum, w);
        const float r = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] *= r * wa[i];
          b[i] *= r * wb[i];
        }
      }
      if constexpr (kAny) {
        float* row = sm.rows + threadIdx.x / kLanes * D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          row[ca + i] = a[i];
          row[cb + i] = b[i];
        }
        __syncwarp(mask);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = ca + i;
          float& x = i < 8 ? a[i] : b[i - 8];
          if (c < half) x = x * co[i] - row[c + half] * si[i];
          else if (c < 2 * half) x = x * co[i] + row[c - half] * si[i];
        }
        __syncwarp(mask);
      } else if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float x = a[i], y = b[i];
          a[i] = x * co[i / 2] - a[i + 1] * si[i / 2];
          a[i + 1] = a[i + 1] * co[i / 2] + x * si[i / 2];
          b[i] = y * co[4 + i / 2] - b[i + 1] * si[4 + i / 2];
          b[i + 1] = b[i + 1] * co[4 + i / 2] + y * si[4 + i / 2];
        }
      } else if (apart) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = a[i];
          a[i] = x * co[i] - b[i] * si[i];
          b[i] = b[i] * co[i] + x * si[i];
        }
      }
      Run8<T> oa, ob;
      oa.set(a);
      ob.set(b);
      oa.store(dst + ca);
      ob.store(dst + cb);
    }
    dst += D;
    if (++h == heads) {
      h = 0;
      token += kTokens;
    }
  }
}

template <typename T>
cudaError_t launch_rope(RopeParams& p, int sms, cudaStream_t s) {
  const int tokens = 32 / (p.d / 16);
  constexpr int kWarps = kRopeThreads / 32;
  p.rows = ((long long)p.T + tokens - 1) / tokens * (p.H + p.Hkv);
  // as many for a warp as leave every SM its CTAs
  const long long warps = (long long)sms * kRopeCtas * kWarps;
  p.per = (int)((p.rows + warps - 1) / warps);
  const long long ctas = (p.rows + (long long)p.per * kWarps - 1) / ((long long)p.per * kWarps);
  const bool any = !p.interleaved && p.rot % 16 != 0;
  auto go = [&](auto kern, size_t smem) {
    if (smem > 48 << 10) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, dim3((unsigned)ctas), dim3(kRopeThreads), smem, s, p);
  };
  auto of = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    return any ? go(rope_kernel<T, D, true>, sizeof(RopeSmem<T, D, true>))
               : go(rope_kernel<T, D, false>, sizeof(RopeSmem<T, D, false>));
  };
  return p.d == 32    ? of(std::integral_constant<int, 32>())
         : p.d == 64  ? of(std::integral_constant<int, 64>())
         : p.d == 128 ? of(std::integral_constant<int, 128>())
                      : of(std::integral_constant<int, 256>());
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace gdn

extern "C" int gdn_qk_norm_rope(const void* q, const void* k, int64_t ldq, int64_t ldk,
                                const int32_t* positions, const float* inv_freq, int rot,
                                int interleaved, const float* q_weight, const float* k_weight,
                                float weight_offset, float eps, int T, int H, int Hkv, int d, int act,
                                void* q_out, void* k_out, int64_t ldqo, int64_t ldko, void* stream) {
  if (T < 0 || !(eps >= 0.f)) return GDN_ERR_RANGE;
  if (H < 0 || Hkv < 0 || H + (int64_t)Hkv < 1 || H > 4096 || Hkv > 4096) return GDN_ERR_DIMS;
  if (d != 32 && d != 64 && d != 128 && d != 256) return GDN_ERR_DIMS;
  if (rot < 0 || rot > d || rot % 2 != 0) return GDN_ERR_DIMS;
  if (act != GDN_F32 && act != GDN_BF16) return GDN_ERR_DIMS;
  if (T == 0) return GDN_OK;
  if (!positions || (rot > 0 && !inv_freq) || (H > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)))
    return GDN_ERR_NULL;
  const int per16 = act == GDN_F32 ? 4 : 8;
  const int64_t most = (int64_t)1 << 38, qcols = (int64_t)H * d, kcols = (int64_t)Hkv * d;
  if (H > 0) {
    if (!gdn::aligned16(q) || !gdn::aligned16(q_out) || ldq % per16 != 0 || ldqo % per16 != 0)
      return GDN_ERR_ALIGN;
    if (ldq < qcols || ldqo < qcols || ldq > most || ldqo > most) return GDN_ERR_RANGE;
  }
  if (Hkv > 0) {
    if (!gdn::aligned16(k) || !gdn::aligned16(k_out) || ldk % per16 != 0 || ldko % per16 != 0)
      return GDN_ERR_ALIGN;
    if (ldk < kcols || ldko < kcols || ldk > most || ldko > most) return GDN_ERR_RANGE;
  }
  // (a warp's rows are counted in 32 bits)
  if ((long long)T * (H + Hkv) * (d / 16) / gdn::kRopeThreads >= 0x7fffffffll) return GDN_ERR_RANGE;
  gdn::RopeParams p = {};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldqo = ldqo;
  p.ldko = ldko;
  p.positions = positions;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.inv_freq = inv_freq;
  p.eps = eps;
  p.offset = weight_offset;
  p.T = T;
  p.H = H;
  p.Hkv = Hkv;
  p.d = d;
  p.rot = rot;
  p.interleaved = interleaved != 0;
  const int sms = gdn::num_sms();
  const cudaError_t e = act == GDN_F32 ? gdn::launch_rope<float>(p, sms, (cudaStream_t)stream)
                                       : gdn::launch_rope<__nv_bfloat16>(p, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
