// Routed experts over 4-bit weights, for the few tokens of a decode step, and the weights' quantisation.
//
//   W[n, i] = (nibble - 8) * scale[n, i / G];  a = silu(W1_e x) * (W3_e x);  y[t] = sum_j w_j W2_e a.
//
// With few rows an expert's product is bound by its weights' bytes, so each weight is read once for all
// rows of its expert, straight from HBM into the registers of the warp that uses it.  The product runs
// on the tensor cores with the outputs as M = 16 and the token rows as N = 8: the nibbles become bf16
// (128 + nibble by an OR into the mantissa, minus 136: exact), a group's sum is kept apart in fp32 and
// scaled once, so no weight is rounded.  fp32 activations go in as their three exact bf16 planes.
//
// A warp's step is 16 outputs x 128 inputs.  The sum over inputs may run in any order, so lane (g, q)
// takes for outputs g and g + 8 the G/4 consecutive inputs of each group that are contiguous in its
// 4-bit row: the weights need no other layout than [output][input / 2].
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;       // outputs of a thread block
constexpr int kStep = 128;      // inputs of a warp's step
constexpr int kRows = 8;        // token rows of one pass over the weights
constexpr int kList = 512;      // rows of an expert found in one scan

struct W4Mat {
  const unsigned char* q;
  const __nv_bfloat16* s;
};

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of w as two bf16: 128 + nibble has the nibble as its last mantissa bits.
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, int i) {
  const uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight consecutive activations as bf16 planes, in the order (0,4) (1,5) (2,6) (3,7) of nibble_pair.
template <typename X> struct Acts;
template <> struct Acts<__nv_bfloat16> {
  static constexpr int kPlanes = 1;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, uint32_t b[1][4]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    b[0][0] = __byte_perm(u.x, u.z, 0x5410); b[0][1] = __byte_perm(u.x, u.z, 0x7632);
    b[0][2] = __byte_perm(u.y, u.w, 0x5410); b[0][3] = __byte_perm(u.y, u.w, 0x7632);
  }
};
template <> struct Acts<float> {
  static constexpr int kPlanes = 3;
  static __device__ __forceinline__ void load(const float* p, uint32_t b[3][4]) {
    const float4 lo = __ldg(reinterpret_cast<const float4*>(p)), hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
    const float f[2][4] = {{lo.x, lo.y, lo.z, lo.w}, {hi.x, hi.y, hi.z, hi.w}};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v[3];
      split3_value(f[0][i], &v[0].x, &v[1].x, &v[2].x);
      split3_value(f[1][i], &v[0].y, &v[1].y, &v[2].y);
#pragma unroll
      for (int k = 0; k < 3; ++k) b[k][i] = *reinterpret_cast<uint32_t*>(&v[k]);
    }
  }
};
struct E4M3 { unsigned char v; };
template <> struct Acts<E4M3> {
  static constexpr int kPlanes = 1;
  static __device__ __forceinline__ void load(const E4M3* p, uint32_t b[1][4]) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // e4m3 values have 4 significant bits: exact in bf16
      const uint32_t two = ((u.x >> (8 * i)) & 0xffu) | (((u.y >> (8 * i)) & 0xffu) << 8);
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
      b[0][i] = pack_bf16x2(f.x, f.y);
    }
  }
};

// One step's weights of outputs `row` (this lane's g; g + 8 follows 8 rows later): 4 words each.
template <int G>
__device__ __forceinline__ void load_weights(const unsigned char* q, int K, int k0, int lane, uint32_t* w) {
  const int sub = lane % 4;
#pragma unroll
  for (int i = 0; i < kStep / G; ++i) {
    const int k = k0 + i * G + sub * (G / 4);
    const bool in = k < K;  // K is a multiple of 32, but a group may be cut short: G / 4 divides it
    const void* p = q + k / 2;
    if constexpr (G == 128) {
      const uint4 u = in ? __ldg(static_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (G == 64) {
      const uint2 u = in ? __ldg(static_cast<const uint2*>(p)) : make_uint2(0, 0);
      w[2 * i] = u.x; w[2 * i + 1] = u.y;
    } else {
      w[i] = in ? __ldg(static_cast<const uint32_t*>(p)) : 0u;
    }
  }
}

// acc[m] += the product of MATS matrices' 16 outputs with up to 8 rows, over this warp's steps.
// `x`: this lane's row (column lane / 4 of the product), null where there is none.  xs0, xs1: the
// activation scales of columns 2q and 2q + 1 (one per 128 inputs), or null.
template <typename X, int G, int MATS>
__device__ __forceinline__ void product(const W4Mat* mats, size_t out0, int K, const X* x, const float* xs0, const float* xs1,
                                        int warp, int lane, float acc[MATS][4]) {
  constexpr int P = Acts<X>::kPlanes;
  const int groups = (K + G - 1) / G;
  const size_t r0 = out0 + lane / 4, r1 = r0 + 8;
  for (int k0 = warp * kStep; k0 < K; k0 += kWarps * kStep) {
    uint32_t w[MATS][2][4];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      load_weights<G>(mats[m].q + r0 * (K / 2), K, k0, lane, w[m][0]);
      load_weights<G>(mats[m].q + r1 * (K / 2), K, k0, lane, w[m][1]);
    }
    const float s0 = xs0 != nullptr ? __ldg(xs0 + k0 / kStep) : 1.f, s1 = xs1 != nullptr ? __ldg(xs1 + k0 / kStep) : 1.f;
#pragma unroll
    for (int i = 0; i < kStep / G; ++i) {
      const int k = k0 + i * G;
      if (k >= K) break;
      float part[MATS][4];
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) part[m][c] = 0.f;
#pragma unroll
      for (int j = 0; j < G / 32; ++j) {
        const int kx = k + (lane % 4) * (G / 4) + j * 8;
        uint32_t b[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int c = 0; c < 4; ++c) b[p][c] = 0u;
        if (x != nullptr && kx < K) Acts<X>::load(x + kx, b);
        const int word = i * (G / 32) + j;
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t a[4] = {nibble_pair(w[m][0][word], 2 * half), nibble_pair(w[m][1][word], 2 * half),
                                   nibble_pair(w[m][0][word], 2 * half + 1), nibble_pair(w[m][1][word], 2 * half + 1)};
#pragma unroll
            for (int p = 0; p < P; ++p) mma_bf16(part[m], a, b[p][2 * half], b[p][2 * half + 1]);
          }
      }
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const float g0 = __bfloat162float(mats[m].s[r0 * groups + k / G]), g1 = __bfloat162float(mats[m].s[r1 * groups + k / G]);
        acc[m][0] = fmaf(part[m][0], g0 * s0, acc[m][0]);
        acc[m][1] = fmaf(part[m][1], g0 * s1, acc[m][1]);
        acc[m][2] = fmaf(part[m][2], g1 * s0, acc[m][2]);
        acc[m][3] = fmaf(part[m][3], g1 * s1, acc[m][3]);
      }
    }
  }
}

// The rows (t, j) of `e` from topk_idx[pos...], ascending, into list; returns the next position.
__device__ __forceinline__ int find_rows(const int* __restrict__ topk_idx, int rows, int e, int pos, int* list, int* counts,
                                         int* found) {
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  int n = 0;
  while (pos < rows && n <= kList - kWarps * kWarp) {
    const int r = pos + threadIdx.x;
    const bool hit = r < rows && __ldg(topk_idx + r) == e;
    const unsigned ballot = __ballot_sync(0xffffffffu, hit);
    __syncthreads();
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int before = n;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += counts[i];
      n += counts[i];
    }
    if (hit) list[before + __popc(ballot & ((1u << lane) - 1u))] = r;
    pos += kWarps * kWarp;
  }
  __syncthreads();
  *found = n;
  return pos;
}

struct W4Args {
  const void* x;
  const float* x_scale;
  const int* topk_idx;
  int rows, k, E, K, N;   // K inputs, N outputs
  W4Mat mat[2];
  void* out;              // gate/up: a [rows, N]; down: [rows, N] fp32
};

// GATEUP: out[r] = silu(W1 x[r / k]) * (W3 x[r / k]) in OUT; else out[r] = W2 x[r].
template <typename X, typename OUT, int G, bool GATEUP>
__global__ void __launch_bounds__(kWarps * 32) w4_kernel(const __grid_constant__ W4Args a) {
  constexpr int MATS = GATEUP ? 2 : 1;
  __shared__ int list[kList], counts[kWarps];
  __shared__ float red[kWarps][MATS][kTile][kRows + 1];
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const bool by_row = a.rows <= a.E;  // one slot a row (the first row of an expert does them all), or a slot an expert
  const int e = by_row ? __ldg(a.topk_idx + blockIdx.y) : (int)blockIdx.y;
  if ((unsigned)e >= (unsigned)a.E) return;  // flagged by the combine
  const size_t out0 = (size_t)e * a.N + blockIdx.x * kTile;
  bool leads = !by_row;
  for (int pos = 0; pos < a.rows;) {
    int n;
    pos = find_rows(a.topk_idx, a.rows, e, pos, list, counts, &n);
    if (!leads && list[0] != (int)blockIdx.y) return;  // the first scan finds this slot's own row at least
    leads = true;
    for (int first = 0; first < n; first += kRows) {
      const int col = first + lane / 4, c0 = first + (lane % 4) * 2;
      auto source = [&](int i) { return GATEUP ? list[i] / a.k : list[i]; };
      const X* x = col < n ? static_cast<const X*>(a.x) + (size_t)source(col) * a.K : nullptr;
      const float *xs0 = nullptr, *xs1 = nullptr;
      if (a.x_scale != nullptr) {
        const int xg = (a.K + kStep - 1) / kStep;
        if (c0 < n) xs0 = a.x_scale + (size_t)source(c0) * xg;
        if (c0 + 1 < n) xs1 = a.x_scale + (size_t)source(c0 + 1) * xg;
      }
      float acc[MATS][4];
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][c] = 0.f;
      product<X, G, MATS>(a.mat, out0, a.K, x, xs0, xs1, warp, lane, acc);
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[warp][m][lane / 4 + (c / 2) * 8][(lane % 4) * 2 + c % 2] = acc[m][c];
      __syncthreads();
      if (threadIdx.x < kTile * kRows) {
        const int o = threadIdx.x % kTile, c = threadIdx.x / kTile;
        if (first + c < n) {
          float v[MATS];
#pragma unroll
          for (int m = 0; m < MATS; ++m) {
            v[m] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v[m] += red[w][m][o][c];
          }
          const size_t at = (size_t)list[first + c] * a.N + blockIdx.x * kTile + o;
          if constexpr (GATEUP) static_cast<OUT*>(a.out)[at] = from_f<OUT>(v[0] * sigmoidf_(v[0]) * v[1]);
          else static_cast<OUT*>(a.out)[at] = from_f<OUT>(v[0]);
        }
      }
    }
    __syncthreads();
  }
}

// y[t] = sum_j topk_w[t,j] * rows[t*k+j], j ascending; a row of no expert counts as zeros.
template <typename T>
__global__ void __launch_bounds__(256) w4_combine_kernel(const float* __restrict__ rows, const int* __restrict__ topk_idx,
                                                         const float* __restrict__ topk_w, int k, int E, int h,
                                                         T* __restrict__ y, int* status) {
  const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= h) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < k; ++j) {
    const size_t r = (size_t)t * k + j;
    if ((unsigned)__ldg(topk_idx + r) >= (unsigned)E) {
      if (c == 0) flag_status(status, MOE_STATUS_BAD_INDEX);
      continue;
    }
    const float w = __ldg(topk_w + r);
    const float4 v = load4(rows + r * h + c);
    s.x = fmaf(w, v.x, s.x); s.y = fmaf(w, v.y, s.y); s.z = fmaf(w, v.z, s.z); s.w = fmaf(w, v.w, s.w);
  }
  store4(y + (size_t)t * h + c, s);
}

// W [E, K, N] -> q [E, N, K/2], scale [E, N, ceil(K/G)]: scale = bf16(amax / 7), nibble =
// clamp(rint(w / scale), -8, 7) + 8.  A block takes one group of inputs of 64 outputs.
template <typename T>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* __restrict__ W, int K, int N, int G,
                                                          unsigned char* __restrict__ q, __nv_bfloat16* __restrict__ scale) {
  __shared__ float tile[128][65];
  __shared__ float sc[64];
  const int n0 = blockIdx.x * 64, k0 = blockIdx.y * G, groups = gridDim.y;
  const size_t e = blockIdx.z;
  const int len = min(G, K - k0);
  for (int i = threadIdx.x; i < len * 64; i += 256) {
    const int k = i / 64, n = i % 64;
    tile[k][n] = n0 + n < N ? to_f(W[(e * K + k0 + k) * N + n0 + n]) : 0.f;
  }
  __syncthreads();
  if (threadIdx.x < 64 && n0 + threadIdx.x < N) {
    float amax = 0.f;
    for (int k = 0; k < len; ++k) amax = fmaxf(amax, fabsf(tile[k][threadIdx.x]));
    const __nv_bfloat16 s = __float2bfloat16_rn(amax / 7.0f);
    scale[(e * N + n0 + threadIdx.x) * groups + blockIdx.y] = s;
    sc[threadIdx.x] = __bfloat162float(s);
  }
  __syncthreads();
  const int half = len / 2;
  for (int i = threadIdx.x; i < half * 64; i += 256) {
    const int n = i / half, b = i % half;
    if (n0 + n >= N) continue;
    const float s = fmaxf(sc[n], 1e-30f);
    auto code = [&](float w) {
      const float z = rintf(w / s);
      return isnan(z) ? 8 : (int)fminf(fmaxf(z, -8.f), 7.f) + 8;
    };
    const int lo = code(tile[2 * b][n]), hi = code(tile[2 * b + 1][n]);
    q[(e * N + n0 + n) * (size_t)(K / 2) + k0 / 2 + b] = (unsigned char)(lo | (hi << 4));
  }
}

template <typename X, typename OUT, bool GATEUP>
void launch_product(const W4Args& a, int G, cudaStream_t st) {
  const dim3 grid(a.N / kTile, a.rows < a.E ? a.rows : a.E);
  if (G == 128) w4_kernel<X, OUT, 128, GATEUP><<<grid, kWarps * 32, 0, st>>>(a);
  else if (G == 64) w4_kernel<X, OUT, 64, GATEUP><<<grid, kWarps * 32, 0, st>>>(a);
  else w4_kernel<X, OUT, 32, GATEUP><<<grid, kWarps * 32, 0, st>>>(a);
  count_launch(st);
}

template <typename T>
void run(const W4Ffn& p, cudaStream_t st) {
  W4Args up{p.x, p.x_scale, p.topk_idx, p.T * p.k, p.k, p.E, p.h, p.f,
            {{static_cast<const unsigned char*>(p.W1q), static_cast<const __nv_bfloat16*>(p.W1s)},
             {static_cast<const unsigned char*>(p.W3q), static_cast<const __nv_bfloat16*>(p.W3s)}}, p.a};
  bool done = false;
  if constexpr (sizeof(T) == 2) {  // e4m3 activations come with bf16 outputs
    if ((done = p.x_scale != nullptr)) launch_product<E4M3, T, true>(up, p.group, st);
  }
  if (!done) launch_product<T, T, true>(up, p.group, st);
  W4Args down{p.a, nullptr, p.topk_idx, p.T * p.k, 1, p.E, p.f, p.h,
              {{static_cast<const unsigned char*>(p.W2q), static_cast<const __nv_bfloat16*>(p.W2s)}, {}}, p.rows};
  launch_product<T, float, false>(down, p.group, st);
  w4_combine_kernel<T><<<dim3(p.T, (p.h / 4 + 255) / 256), 256, 0, st>>>(p.rows, p.topk_idx, p.topk_w, p.k, p.E, p.h,
                                                                        static_cast<T*>(p.y), p.status);
  count_launch(st);
}

}  // namespace

void launch_expert_ffn_w4(int dtype, const W4Ffn& p, cudaStream_t st) {
  if (dtype == MOE_BF16) run<__nv_bfloat16>(p, st);
  else run<float>(p, st);
}

void launch_quantize_w4(int dtype, const void* W, int E, int K, int N, int group, void* q, void* scale, cudaStream_t st) {
  const dim3 grid((N + 63) / 64, (K + group - 1) / group, E);
  if (dtype == MOE_BF16)
    w4_quantize_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(W), K, N, group,
                                                          static_cast<unsigned char*>(q), static_cast<__nv_bfloat16*>(scale));
  else
    w4_quantize_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(W), K, N, group,
                                                    static_cast<unsigned char*>(q), static_cast<__nv_bfloat16*>(scale));
  count_launch(st);
}

}  // namespace moe
