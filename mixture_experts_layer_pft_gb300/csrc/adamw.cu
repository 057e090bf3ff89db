// One AdamW step over many tensors in one launch (per kAdamwMaxTensors tensors), states in 32 or 8 bits.
//
//   g' = g * grad_scale;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2;
//   p -= lr * (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)).
//
// A warp takes 256 consecutive elements of one tensor: the block of one scale of the 8-bit states.
// There m is kept in e4m3 (scale = amax / 2^8) and v in e5m2 (scale = amax / 2^15), both rounded up
// or down at random with the probability of what is cut off: with b2 = 0.999 a step moves v by about
// a thousandth, far below half of an 8-bit step, and rounding to nearest would leave it where it is.
// A positive v never rounds to zero, so that no later step divides a momentum by eps alone.  The
// update of p reads the states before they are rounded.  Every operation that decides a code is one
// correctly rounded fp32 operation (no contraction), so the codes follow from the formulas.
#include <cuda_fp8.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kOptBlock = 256;     // elements of one scale, handled by one warp
constexpr int kWarps = 8;
constexpr int kBlocksPerWarp = 4;
constexpr int kChunk = kOptBlock * kWarps * kBlocksPerWarp;  // elements of one thread block

template <int N>
struct AdamwArgs {
  AdamwTensor t[N];
  int first_chunk[N + 1];  // thread blocks before tensor i
  int n, first_tensor;
  const float* lr;
  const int* step;
  const float* grad_scale;
  int* status;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, log_beta1, log_beta2, eps;
  uint32_t seed_lo, seed_hi;
};

// Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1,
// 2, 3", 2011; 7 is the fewest rounds that pass that paper's tests).
__device__ __forceinline__ uint4 philox7(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint32_t h0 = __umulhi(c.x, 0xD2511F53u), l0 = c.x * 0xD2511F53u;
    const uint32_t h1 = __umulhi(c.z, 0xCD9E8D57u), l1 = c.z * 0xCD9E8D57u;
    c = make_uint4(h1 ^ c.y ^ k0, l1, h0 ^ c.w ^ k1, l0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The update of p needs no correctly rounded root or quotient: these are within 2 of the last bit, of a term that is
// a thousandth of p.
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x >= 0 to 23 - DROP mantissa bits, up with the probability of what is cut off (16 random bits);
// below `low`, the smallest normal value, on the fixed grid of [low, 2 low).
template <int DROP>
__device__ __forceinline__ float round_random(float x, uint32_t bits16, float low) {
  const bool small = x < low;
  uint32_t b = __float_as_uint(small ? __fadd_rn(x, low) : x);
  b = (b + ((bits16 << (DROP - 16)) | (1u << (DROP - 17)))) & ~((1u << DROP) - 1u);
  const float r = __uint_as_float(b);
  return small ? __fsub_rn(r, low) : r;
}

__device__ __forceinline__ void unpack4_fp8(uint32_t w, __nv_fp8_interpretation_t kind, float* f) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), kind)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), kind)));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
__device__ __forceinline__ uint32_t pack4_fp8(const float* f, __nv_fp8_interpretation_t kind) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, kind);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, kind);
  return lo | (hi << 16);
}
__device__ __forceinline__ float unpack1_fp8(unsigned char c, __nv_fp8_interpretation_t kind) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, kind)));
}

// Four consecutive elements, the last of a tensor one by one.
template <typename T>
__device__ __forceinline__ void get4(const T* p, long long e, long long n, float* f) {
  if (e + 4 <= n) {
    const float4 v = load4(p + e);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = e + i < n ? to_f(p[e + i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put4(T* p, long long e, long long n, const float* f) {
  if (e + 4 <= n) {
    store4(p + e, make_float4(f[0], f[1], f[2], f[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < n) p[e + i] = from_f<T>(f[i]);
  }
}
__device__ __forceinline__ void get4_fp8(const unsigned char* p, long long e, long long n, __nv_fp8_interpretation_t kind,
                                         float scale, float* f) {
  if (e + 4 <= n) {
    unpack4_fp8(*reinterpret_cast<const uint32_t*>(p + e), kind, f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = e + i < n ? unpack1_fp8(p[e + i], kind) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __fmul_rn(f[i], scale);
}
__device__ __forceinline__ void put4_fp8(unsigned char* p, long long e, long long n, __nv_fp8_interpretation_t kind,
                                         const float* f) {
  const uint32_t w = pack4_fp8(f, kind);
  if (e + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p + e) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < n) p[e + i] = (unsigned char)(w >> (8 * i));
  }
}

template <int N, bool Q8>
__global__ void __launch_bounds__(kWarps * 32) adamw_kernel(const __grid_constant__ AdamwArgs<N> a) {
  int lo = 0, hi = a.n - 1;  // the tensor of this thread block
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first_chunk[mid] <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamwTensor& q = a.t[lo];
  const long long n = q.numel;
  const int step = *a.step;
  if (step < 1) {
    if (threadIdx.x == 0) flag_status(a.status, MOE_STATUS_BAD_INDEX);
    return;
  }
  const float lr = *a.lr, gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  // 1 - b^t without cancellation
  const float rbc1 = -1.0f / expm1f((float)step * a.log_beta1), rbc2 = -1.0f / expm1f((float)step * a.log_beta2);
  const int lane = threadIdx.x % kWarp;
  const long long base = ((long long)blockIdx.x - a.first_chunk[lo]) * kChunk + (long long)(threadIdx.x / kWarp) * kBlocksPerWarp * kOptBlock;
  bool bad = false;
  for (int b = 0; b < kBlocksPerWarp; ++b) {
    const long long e0 = base + (long long)b * kOptBlock;
    if (e0 >= n) break;
    const long long block = e0 / kOptBlock;
    float m[8], v[8], amax_m = 0.f, amax_v = 0.f;
    const float ms = Q8 ? q.m_scale[block] : 1.f, vs = Q8 ? q.v_scale[block] : 1.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const long long e = e0 + half * 128 + lane * 4;
      float g[4], p[4];
      float* mm = m + half * 4;
      float* vv = v + half * 4;
      if (q.dtype == MOE_BF16) {
        get4(static_cast<const __nv_bfloat16*>(q.grad), e, n, g);
        get4(q.master, e, n, p);
      } else {
        get4(static_cast<const float*>(q.grad), e, n, g);
        get4(static_cast<const float*>(q.param), e, n, p);
      }
      if constexpr (Q8) {
        get4_fp8(static_cast<const unsigned char*>(q.m), e, n, __NV_E4M3, ms, mm);
        get4_fp8(static_cast<const unsigned char*>(q.v), e, n, __NV_E5M2, vs, vv);
      } else {
        get4(static_cast<const float*>(q.m), e, n, mm);
        get4(static_cast<const float*>(q.v), e, n, vv);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gi = __fmul_rn(g[i], gs), gg = __fmul_rn(gi, gi);
        if (!(gg <= FLT_MAX)) {  // not finite: this element stays as it is
          bad = true;
        } else {
          mm[i] = __fadd_rn(__fmul_rn(mm[i], a.beta1), __fmul_rn(gi, a.one_minus_beta1));
          vv[i] = __fadd_rn(__fmul_rn(vv[i], a.beta2), __fmul_rn(gg, a.one_minus_beta2));
          p[i] -= lr * (q.weight_decay * p[i] + __fdividef(mm[i] * rbc1, sqrt_approx(vv[i] * rbc2) + a.eps));
        }
        amax_m = fmaxf(amax_m, fabsf(mm[i]));
        amax_v = fmaxf(amax_v, vv[i]);
      }
      if (q.dtype == MOE_BF16) {
        put4(q.master, e, n, p);
        put4(static_cast<__nv_bfloat16*>(q.param), e, n, p);
      } else {
        put4(static_cast<float*>(q.param), e, n, p);
      }
      if constexpr (!Q8) {
        put4(static_cast<float*>(q.m), e, n, mm);
        put4(static_cast<float*>(q.v), e, n, vv);
      }
    }
    if constexpr (Q8) {
      const float new_ms = __fmul_rn(fmaxf(warp_max(amax_m), 0x1p-100f), 0x1p-8f);
      const float new_vs = __fmul_rn(fmaxf(warp_max(amax_v), 0x1p-100f), 0x1p-15f);
      const float rm = __frcp_rn(new_ms), rv = __frcp_rn(new_vs);
      if (lane == 0) {
        q.m_scale[block] = new_ms;
        q.v_scale[block] = new_vs;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const long long e = e0 + half * 128 + lane * 4;
        const unsigned long long four = (unsigned long long)e >> 2;
        const uint4 r4 = philox7(make_uint4((uint32_t)four, (uint32_t)(four >> 32), (uint32_t)(a.first_tensor + lo), (uint32_t)step),
                                 a.seed_lo, a.seed_hi);
        const uint32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
        float cm[4], cv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mi = m[half * 4 + i], vi = v[half * 4 + i];
          cm[i] = copysignf(round_random<20>(__fmul_rn(fabsf(mi), rm), r[i] & 0xffffu, 0x1p-6f), mi);
          cv[i] = round_random<21>(__fmul_rn(vi, rv), r[i] >> 16, 0x1p-14f);
          if (vi > 0.f && cv[i] == 0.f) cv[i] = 0x1p-16f;
        }
        put4_fp8(static_cast<unsigned char*>(q.m), e, n, __NV_E4M3, cm);
        put4_fp8(static_cast<unsigned char*>(q.v), e, n, __NV_E5M2, cv);
      }
    }
  }
  if (bad) flag_status(a.status, MOE_STATUS_NOT_FINITE);
}

template <int N>
void launch_some(const AdamwTensor* t, int n, int first_tensor, const AdamwScalars& c, cudaStream_t st) {
  AdamwArgs<N> a;
  long long chunks = 0;
  a.n = 0;
  for (int i = 0; i < n; ++i) {
    a.t[i] = t[i];
    a.first_chunk[i] = (int)chunks;
    chunks += (t[i].numel + kChunk - 1) / kChunk;
  }
  a.n = n;
  a.first_chunk[n] = (int)chunks;
  if (chunks == 0) return;
  a.first_tensor = first_tensor;
  a.lr = c.lr; a.step = c.step; a.grad_scale = c.grad_scale; a.status = c.status;
  a.beta1 = (float)c.beta1; a.one_minus_beta1 = (float)(1.0 - c.beta1);
  a.beta2 = (float)c.beta2; a.one_minus_beta2 = (float)(1.0 - c.beta2);
  a.log_beta1 = (float)c.log_beta1; a.log_beta2 = (float)c.log_beta2;
  a.eps = (float)c.eps;
  a.seed_lo = (uint32_t)c.seed; a.seed_hi = (uint32_t)(c.seed >> 32);
  if (c.q8) adamw_kernel<N, true><<<(unsigned)chunks, kWarps * 32, 0, st>>>(a);
  else adamw_kernel<N, false><<<(unsigned)chunks, kWarps * 32, 0, st>>>(a);
  count_launch(st);
}

}  // namespace

// At most kAdamwMaxTensors tensors, by launch argument (no table on the device, nothing to keep alive),
// in the smallest of three argument sizes (1.3, 7.4 and 29 KB; CUDA allows 32,764 bytes).
void launch_adamw(const AdamwTensor* t, int n, int first_tensor, const AdamwScalars& c, cudaStream_t st) {
  if (n <= 16) launch_some<16>(t, n, first_tensor, c, st);
  else if (n <= 96) launch_some<96>(t, n, first_tensor, c, st);
  else launch_some<kAdamwMaxTensors>(t, n, first_tensor, c, st);
}

}  // namespace moe
