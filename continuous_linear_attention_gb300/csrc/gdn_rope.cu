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
// squares is the only thing that crosses lanes.  A group of d/16 threads takes
// all heads of a token where there are tokens enough (the angle's sine and
// cosine are computed once per token), fewer where not.
// 15,843 tokens x 40 heads x 128: 64.5 us, 5.0 TB/s.
#include <cuda_runtime.h>

#include "gdn_cta.cuh"
#include "gdn_internal.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
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
  int per;     // heads a group takes
  int slices;  // groups a token takes
};

// A run of 8 channels, as it lies.
template <typename T>
struct Run8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
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

// kAny: a rotated half that is no multiple of 8 channels (and not interleaved),
// whose pairs lie in different threads' runs: they meet in shared memory.
template <typename T, int D, bool kAny>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(RopeParams p) {
  constexpr int kLanes = D / 16;  // threads per head
  constexpr int kAhead = sizeof(T) == 2 ? kRopeAhead : 2;  // heads whose reads are on their way together
  // inv_freq / 2 pi as 64-bit fractions of a turn: an angle is the product with
  // the position modulo 2^64, exact for any position (an fp32 angle at position
  // 10^6 would be off by 0.06)
  __shared__ unsigned long long turns[D / 2];
  __shared__ float rows[kAny ? kRopeThreads * 16 : 1];
  pdl_wait_then_release();
  const int half = p.rot / 2;
  if ((int)threadIdx.x < half) {
    double t = (double)p.inv_freq[threadIdx.x] * 0.15915494309189533577;
    t -= floor(t);
    turns[threadIdx.x] = t < 1.0 ? (unsigned long long)(t * 18446744073709551616.0) : 0ull;
  }
  __syncthreads();
  const int lane = threadIdx.x % kLanes;
  const long long group =
      ((long long)blockIdx.x * kRopeThreads + threadIdx.x) / kLanes;
  const long long token = group / p.slices;
  const int pos = token < p.T ? p.positions[token] : -1;
  const bool live = pos >= 0;  // (a group that is not lends its lanes to the sums)
  // this thread's two runs
  const bool apart = !kAny && !p.interleaved && lane < half / 8;  // those of a half and of the other
  const int ca = apart ? 8 * lane : 16 * lane, cb = apart ? ca + half : ca + 8;
  // the turns of their pairs, or (kAny) of their channels
  constexpr int kTurns = kAny ? 16 : 8;
  float co[kTurns], si[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    co[i] = 1.f;
    si[i] = 0.f;
    int of = 8 * lane + i;  // the pair, in either order
    if (kAny) {
      of = ca + i;
      of = of < half ? of : of < 2 * half ? of - half : half;
    }
    if (live && of < half) {
      const unsigned long long a = turns[of] * (unsigned long long)(unsigned)pos;
      sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &si[i], &co[i]);
    }
  }
  // the lanes of one head: they come to its sum together or not at all
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const int heads = p.H + p.Hkv;
  const int h0 = (int)(group % p.slices) * p.per, h1 = min(heads, h0 + p.per);
  // queries, then keys: their weights stay in registers
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = part ? max(h0, p.H) - p.H : h0, hi = part ? h1 - p.H : min(h1, p.H);
    if (lo >= hi) continue;  // (the same for all groups of a slice: a warp's may differ)
    const float* weight = part ? p.k_weight : p.q_weight;
    const T* src = static_cast<const T*>(part ? p.k : p.q) + token * (part ? p.ldk : p.ldq);
    T* dst = static_cast<T*>(part ? p.k_out : p.q_out) + token * (part ? p.ldko : p.ldqo);
    float wa[8], wb[8];
    if (weight) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wa[i] = weight[ca + i] + p.offset;
        wb[i] = weight[cb + i] + p.offset;
      }
    }
    for (int h = lo; h < hi; h += kAhead) {
      Run8<T> ra[kAhead], rb[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (live && h + u < hi) {
          ra[u].load(src + (size_t)(h + u) * D + ca);
          rb[u].load(src + (size_t)(h + u) * D + cb);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!live || h + u >= hi) continue;
        float a[8], b[8];
        ra[u].get(a);
        rb[u].get(b);
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
          float* row = rows + threadIdx.x / kLanes * D;
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
        oa.store(dst + (size_t)(h + u) * D + ca);
        ob.store(dst + (size_t)(h + u) * D + cb);
      }
    }
  }
}

template <typename T>
cudaError_t launch_rope(RopeParams& p, int sms, cudaStream_t s) {
  const int lanes = p.d / 16, heads = p.H + p.Hkv;
  // As many heads for a group as leave every SM 512 threads, and all of them
  // where that is so anyway.
  const long long want = (long long)sms * (kRopeThreads * kRopeCtas) / lanes;
  long long slices = (want + p.T - 1) / p.T;
  if (slices > heads) slices = heads;
  p.per = (int)((heads + slices - 1) / slices);
  p.slices = (heads + p.per - 1) / p.per;
  const long long groups = (long long)p.T * p.slices;
  const long long ctas = (groups * lanes + kRopeThreads - 1) / kRopeThreads;
  const bool any = !p.interleaved && p.rot % 16 != 0;
  auto kern = p.d == 32    ? any ? rope_kernel<T, 32, true> : rope_kernel<T, 32, false>
              : p.d == 64  ? any ? rope_kernel<T, 64, true> : rope_kernel<T, 64, false>
              : p.d == 128 ? any ? rope_kernel<T, 128, true> : rope_kernel<T, 128, false>
              : any        ? rope_kernel<T, 256, true>
                           : rope_kernel<T, 256, false>;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kRopeThreads), 0, s, p);
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
  // (groups of d/16 threads for up to 8,192 heads a token: the grid's size)
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
