// Add + RMSNorm before the layer: forward (with an optional 8-bit output) and backward.
//
//   s = round(x + residual);  rstd = 1 / sqrt(mean(s^2) + eps);  v = s * rstd * gamma;  y = round(v);
//   q = e4m3(v / scale), scale = max(amax(|v|), 2^-100) / 448 per row and 128 columns.
//   backward: g = dy * gamma, xh = s * rstd;
//   ds = round(ds_add + rstd * (g - xh * mean(g * xh)));  dgamma = sum_t dy * xh.
//
// A row stays in the registers of its `tpr` threads (16-byte vectors, at most kMaxVec a thread), so
// every array moves once.  Sums run in fp32 in a fixed order: no atomics, bitwise reproducible.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxVec = 4;       // 16-byte vectors of a row in one thread
constexpr int kQGroup = 128;     // columns per scale of the 8-bit output

struct NormGeom {
  int vpt, tpr, rpb;  // vectors a thread, threads a row, rows a block
};

NormGeom norm_geom(int nvec) {
  const int tpr = ((nvec + kMaxVec - 1) / kMaxVec + 31) / 32 * 32;
  const int rpb = tpr >= 256 ? 1 : 256 / tpr;
  return {kMaxVec, tpr, rpb};
}

// Sum over the `tpr` threads of a row, returned to all of them.  red: one float per warp.
__device__ __forceinline__ float row_sum(float v, float* red, int tpr) {
  v = warp_sum(v);
  if (tpr == kWarp) return v;
  const int warp = threadIdx.x / kWarp, wpr = tpr / kWarp, first = warp / wpr * wpr;
  if (threadIdx.x % kWarp == 0) red[warp] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < wpr; ++i) s += red[first + i];
  return s;
}

template <int VN>
__device__ __forceinline__ void store_q(unsigned char* q, const float* v, float inv) {
  uint32_t w[VN / 4];
#pragma unroll
  for (int i = 0; i < VN / 4; ++i) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  if constexpr (VN == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(q) = w[0];
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const T* x, const T* residual, const float* __restrict__ gamma,
                                                           float eps, int T_, int h, int tpr, int rpb, T* s, T* y,
                                                           unsigned char* __restrict__ q, float* __restrict__ q_scale,
                                                           float* __restrict__ rstd) {
  constexpr int VN = Vec<T>::N;
  __shared__ float red[32];
  const int lt = threadIdx.x % tpr;
  const int t = blockIdx.x * rpb + threadIdx.x / tpr;
  const int nvec = h / VN;
  const bool on = t < T_;
  const size_t row = (size_t)t * nvec;
  float f[VPT][VN];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
#pragma unroll
    for (int i = 0; i < VN; ++i) f[u][i] = 0.f;
    if (!on || v >= nvec) continue;
    unpack(reinterpret_cast<const uint4*>(x)[row + v], f[u], T());
    if (residual != nullptr) {
      float r[VN];
      unpack(reinterpret_cast<const uint4*>(residual)[row + v], r, T());
#pragma unroll
      for (int i = 0; i < VN; ++i) f[u][i] += r[i];
      const uint4 o = pack(f[u], T());
      reinterpret_cast<uint4*>(s)[row + v] = o;
      unpack(o, f[u], T());  // the norm is of the stored sum
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) ss = fmaf(f[u][i], f[u][i], ss);
  }
  ss = row_sum(ss, red, tpr);
  const float rs = 1.0f / sqrtf(ss / (float)h + eps);
  if (!on) return;
  if (rstd != nullptr && lt == 0) rstd[t] = rs;
  const int groups = (h + kQGroup - 1) / kQGroup;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    float amax = 0.f;
    if (v < nvec) {
#pragma unroll
      for (int i = 0; i < VN; i += 4) {
        const float4 g = load4(gamma + (size_t)v * VN + i);
        f[u][i] *= rs * g.x; f[u][i + 1] *= rs * g.y; f[u][i + 2] *= rs * g.z; f[u][i + 3] *= rs * g.w;
      }
#pragma unroll
      for (int i = 0; i < VN; ++i) amax = fmaxf(amax, fabsf(f[u][i]));
      if (y != nullptr) reinterpret_cast<uint4*>(y)[row + v] = pack(f[u], T());
    }
    if (q != nullptr) {
      // 128 columns are kQGroup / VN neighbouring lanes (tpr is a multiple of 32)
#pragma unroll
      for (int o = kQGroup / VN / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = fmaxf(amax, 0x1p-100f) / 448.0f;
      if (v < nvec) {
        if (v % (kQGroup / VN) == 0) q_scale[(size_t)t * groups + v / (kQGroup / VN)] = scale;
        store_q<VN>(q + (row + v) * VN, f[u], 1.0f / scale);
      }
    }
  }
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ s,
                                                               const float* __restrict__ gamma, const float* __restrict__ rstd,
                                                               const T* ds_add, int T_, int h, int tpr, int rpb, T* ds,
                                                               float* __restrict__ partial) {
  constexpr int VN = Vec<T>::N;
  __shared__ float red[2][32];
  const int lt = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const int nvec = h / VN;
  float dg[VPT][VN];
#pragma unroll
  for (int u = 0; u < VPT; ++u)
#pragma unroll
    for (int i = 0; i < VN; ++i) dg[u][i] = 0.f;
  int turn = 0;
  for (long long t0 = (long long)blockIdx.x * rpb; t0 < T_; t0 += (long long)gridDim.x * rpb, turn ^= 1) {
    const int t = (int)t0 + sub;
    const bool on = t < T_;
    const size_t row = (size_t)t * nvec;
    const float rs = on ? rstd[t] : 0.f;
    float xh[VPT][VN], g[VPT][VN];
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int v = lt + u * tpr;
      if (!on || v >= nvec) continue;
      float d[VN];
      unpack(reinterpret_cast<const uint4*>(dy)[row + v], d, T());
      unpack(reinterpret_cast<const uint4*>(s)[row + v], xh[u], T());
#pragma unroll
      for (int i = 0; i < VN; i += 4) {
        const float4 w = load4(gamma + (size_t)v * VN + i);
        g[u][i] = d[i] * w.x; g[u][i + 1] = d[i + 1] * w.y; g[u][i + 2] = d[i + 2] * w.z; g[u][i + 3] = d[i + 3] * w.w;
      }
#pragma unroll
      for (int i = 0; i < VN; ++i) {
        xh[u][i] *= rs;
        dg[u][i] = fmaf(d[i], xh[u][i], dg[u][i]);
        dot = fmaf(g[u][i], xh[u][i], dot);
      }
    }
    const float mean = row_sum(dot, red[turn], tpr) / (float)h;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int v = lt + u * tpr;
      if (!on || v >= nvec) continue;
      float o[VN];
      if (ds_add != nullptr) {
        unpack(reinterpret_cast<const uint4*>(ds_add)[row + v], o, T());
      } else {
#pragma unroll
        for (int i = 0; i < VN; ++i) o[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VN; ++i) o[i] = fmaf(rs, fmaf(-xh[u][i], mean, g[u][i]), o[i]);
      reinterpret_cast<uint4*>(ds)[row + v] = pack(o, T());
    }
  }
  float* p = partial + ((size_t)blockIdx.x * rpb + sub) * h;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    if (v >= nvec) continue;
#pragma unroll
    for (int i = 0; i < VN; i += 4)
      store4(p + (size_t)v * VN + i, make_float4(dg[u][i], dg[u][i + 1], dg[u][i + 2], dg[u][i + 3]));
  }
}

// dgamma[c] = sum over the `parts` partials, p ascending within each of 8 strips, strips ascending.
__global__ void __launch_bounds__(256) dgamma_kernel(const float* __restrict__ partial, int parts, int h,
                                                     float* __restrict__ dgamma) {
  __shared__ float red[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, strip = threadIdx.x / 32;
  float sum = 0.f;
  if (c < h)
    for (int p = strip; p < parts; p += 8) sum += partial[(size_t)p * h + c];
  red[strip][threadIdx.x % 32] = sum;
  __syncthreads();
  if (strip == 0 && c < h) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += red[i][threadIdx.x];
    dgamma[c] = sum;
  }
}

template <typename T>
void launch_fwd(const void* x, const void* residual, const float* gamma, float eps, int T_, int h, void* s, void* y,
                void* q, float* q_scale, float* rstd, cudaStream_t st) {
  const NormGeom g = norm_geom(h / Vec<T>::N);
  add_rmsnorm_kernel<T, kMaxVec><<<(T_ + g.rpb - 1) / g.rpb, g.tpr * g.rpb, 0, st>>>(
      static_cast<const T*>(x), static_cast<const T*>(residual), gamma, eps, T_, h, g.tpr, g.rpb, static_cast<T*>(s),
      static_cast<T*>(y), static_cast<unsigned char*>(q), q_scale, rstd);
  count_launch(st);
}

int bwd_blocks(int T_, int rpb) {
  const int need = (T_ + rpb - 1) / rpb, most = kNormMaxParts / rpb;
  return need < most ? need : most;
}

template <typename T>
void launch_bwd(const void* dy, const void* s, const float* gamma, const float* rstd, const void* ds_add, int T_, int h,
                void* ds, float* dgamma, float* partial, cudaStream_t st) {
  const NormGeom g = norm_geom(h / Vec<T>::N);
  const int blocks = bwd_blocks(T_, g.rpb);
  add_rmsnorm_bwd_kernel<T, kMaxVec><<<blocks, g.tpr * g.rpb, 0, st>>>(
      static_cast<const T*>(dy), static_cast<const T*>(s), gamma, rstd, static_cast<const T*>(ds_add), T_, h, g.tpr, g.rpb,
      static_cast<T*>(ds), partial);
  count_launch(st);
  dgamma_kernel<<<(h + 31) / 32, 256, 0, st>>>(partial, blocks * g.rpb, h, dgamma);
  count_launch(st);
}

}  // namespace

void launch_add_rmsnorm(int dtype, const void* x, const void* residual, const float* gamma, float eps, int T, int h, void* s,
                        void* y, void* q, float* q_scale, float* rstd, cudaStream_t st) {
  if (dtype == MOE_BF16) launch_fwd<__nv_bfloat16>(x, residual, gamma, eps, T, h, s, y, q, q_scale, rstd, st);
  else launch_fwd<float>(x, residual, gamma, eps, T, h, s, y, q, q_scale, rstd, st);
}

void launch_add_rmsnorm_bwd(int dtype, const void* dy, const void* s, const float* gamma, const float* rstd,
                            const void* ds_add, int T, int h, void* ds, float* dgamma, float* partial, cudaStream_t st) {
  if (dtype == MOE_BF16) launch_bwd<__nv_bfloat16>(dy, s, gamma, rstd, ds_add, T, h, ds, dgamma, partial, st);
  else launch_bwd<float>(dy, s, gamma, rstd, ds_add, T, h, ds, dgamma, partial, st);
}

}  // namespace moe
