// Add + RMSNorm before the layer: forward (with an optional 8-bit output) and backward.
//
//   s = round(x + residual);  rstd = 1 / sqrt(mean(s^2) + eps);  v = s * rstd * gamma;  y = round(v);
//   q = e4m3(v / scale), scale = max(amax(|v|), 2^-100) / 448 per row and 128 columns.
//   backward: g = dy * gamma, xh = s * rstd;
//   ds = round(ds_add + rstd * (g - xh * mean(g * xh)));  dgamma = sum_t dy * xh.
//
// Both are bound by HBM: every array moves once.  Forward: a row stays in the registers of its `tpr` threads (16-byte
// vectors, at most kMaxVec a thread).  4096 x 7168 bf16 with residual, y and q: 265 MB in 46 us, 85% of the measured copy
// rate (57 us where the loads of a row were mixed with its stores); one row: 4 us, all latency.  Backward: a ring of bulk
// copies, see there; the same rows with ds_add: 235 MB in 42 us (82%), dgamma's second kernel included.  Sums run in fp32
// in a fixed order: no atomics, bitwise reproducible.
#include <cuda_fp8.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kMaxVec = 4;       // 16-byte vectors of a row in one thread
constexpr int kQGroup = 128;     // columns per scale of the 8-bit output

constexpr int kRingMaxStages = 8;
constexpr int kRingThreads = 512;  // of a block, where several rows share one
constexpr int kRingBytes = 200 * 1024;

struct NormGeom {
  int tpr, rpb;  // threads a row, rows a block
};

NormGeom norm_geom(int nvec) {
  const int tpr = ((nvec + kMaxVec - 1) / kMaxVec + 31) / 32 * 32;
  const int rpb = tpr >= 256 ? 1 : 256 / tpr;
  return {tpr, rpb};
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
  // all of the thread's loads before the first store: x and residual may be s itself, so the compiler
  // keeps the order that is written here
  uint4 rx[VPT], rr[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    rx[u] = rr[u] = make_uint4(0, 0, 0, 0);
    if (on && v < nvec) {
      rx[u] = reinterpret_cast<const uint4*>(x)[row + v];
      if (residual != nullptr) rr[u] = reinterpret_cast<const uint4*>(residual)[row + v];
    }
  }
  float f[VPT][VN];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    unpack(rx[u], f[u], T());
    if (residual != nullptr) {
      float r[VN];
      unpack(rr[u], r, T());
#pragma unroll
      for (int i = 0; i < VN; ++i) f[u][i] += r[i];
      const uint4 o = pack(f[u], T());
      if (on && v < nvec) reinterpret_cast<uint4*>(s)[row + v] = o;
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
  // rstd in two factors, a power of two and one from [1, 2): s by the first is exact, and its product with gamma is at an end
  // of fp32 only where the output is
  const bool ordinary = rs > 0.f && rs <= FLT_MAX;
  const float power = ordinary ? __uint_as_float(__float_as_uint(rs) & 0x7f800000u) : 1.0f, rest = rs / power;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    float amax = 0.f;
    if (v < nvec) {
#pragma unroll
      for (int i = 0; i < VN; i += 4) {
        const float4 g = load4(gamma + (size_t)v * VN + i);
        f[u][i] = f[u][i] * power * g.x; f[u][i + 1] = f[u][i + 1] * power * g.y;
        f[u][i + 2] = f[u][i + 2] * power * g.z; f[u][i + 3] = f[u][i + 3] * power * g.w;
      }
#pragma unroll
      for (int i = 0; i < VN; ++i) amax = fmaxf(amax, fabsf(f[u][i]));
      if (y != nullptr) {
        float o[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) o[i] = f[u][i] * rest;
        reinterpret_cast<uint4*>(y)[row + v] = pack(o, T());
      }
    }
    if (q != nullptr) {
      // 128 columns are kQGroup / VN neighbouring lanes (tpr is a multiple of 32)
#pragma unroll
      for (int o = kQGroup / VN / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // `rest` cancels in y / scale: without it a code has two roundings less that may push it over a tie
      const float most = rest * amax, scale = fmaxf(most, 0x1p-100f) / 448.0f;
      const float inv = most >= 0x1p-100f ? 448.0f / amax : rest * (448.0f * 0x1p100f);
      if (v < nvec) {
        if (v % (kQGroup / VN) == 0) q_scale[(size_t)t * groups + v / (kQGroup / VN)] = scale;
        store_q<VN>(q + (row + v) * VN, f[u], inv);
      }
    }
  }
}

// The backward of rows that are too wide for two stages of the ring below (fp32 above 8,533 columns): a block takes
// every gridDim-th row into its registers.
template <int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_bwd_wide_kernel(const float* __restrict__ dy, const float* __restrict__ s,
                                                                    const float* __restrict__ gamma,
                                                                    const float* __restrict__ rstd, const float* ds_add, int T_,
                                                                    int h, float* ds, float* __restrict__ partial) {
  __shared__ float red[2][32];
  const int lt = threadIdx.x, tpr = blockDim.x, nvec = h / 4;
  float4 dg[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) dg[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  int turn = 0;
  for (int t = blockIdx.x; t < T_; t += gridDim.x, turn ^= 1) {
    const size_t row = (size_t)t * h;
    const float rs = rstd[t];
    float4 d[VPT], x[VPT];
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int v = lt + u * tpr;
      if (v >= nvec) continue;
      d[u] = load4(dy + row + v * 4);
      x[u] = load4(s + row + v * 4);
      const float4 w = load4(gamma + v * 4);
      x[u].x *= rs; x[u].y *= rs; x[u].z *= rs; x[u].w *= rs;
      const float4 p = make_float4(d[u].x * x[u].x, d[u].y * x[u].y, d[u].z * x[u].z, d[u].w * x[u].w);
      dg[u].x += p.x; dg[u].y += p.y; dg[u].z += p.z; dg[u].w += p.w;
      dot = fmaf(p.x, w.x, fmaf(p.y, w.y, fmaf(p.z, w.z, fmaf(p.w, w.w, dot))));
    }
    const float mean = row_sum(dot, red[turn], tpr) / (float)h;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int v = lt + u * tpr;
      if (v >= nvec) continue;
      const float4 w = load4(gamma + v * 4);
      float4 o = ds_add != nullptr ? load4(ds_add + row + v * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      o.x = fmaf(rs, fmaf(-x[u].x, mean, d[u].x * w.x), o.x);
      o.y = fmaf(rs, fmaf(-x[u].y, mean, d[u].y * w.y), o.y);
      o.z = fmaf(rs, fmaf(-x[u].z, mean, d[u].z * w.z), o.z);
      o.w = fmaf(rs, fmaf(-x[u].w, mean, d[u].w * w.w), o.w);
      store4(ds + row + v * 4, o);
    }
  }
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    if (v < nvec) store4(partial + (size_t)blockIdx.x * h + v * 4, dg[u]);
  }
}

// The backward over a ring of row groups in shared memory.  One block an SM; its thread 0 keeps `stages` groups of
// rows (dy, s, ds_add: each a contiguous piece of memory) under way as bulk copies, so that the reduction over a row
// and the stores never leave HBM idle, and no register waits for a load (a kernel that loads
// rows into registers took 147 us where this one takes 35).  16 elements of a row in a
// thread; gamma and the thread's columns of dgamma stay in registers over all rows.
template <typename T, int ELEMS, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) add_rmsnorm_bwd_ring_kernel(const T* dy, const T* s, const float* __restrict__ gamma,
                                                                       const float* __restrict__ rstd, const T* ds_add, int T_,
                                                                       int h, int tpr, int rpb, int stages, T* ds,
                                                                       float* __restrict__ partial, int* status) {
  constexpr int VN = Vec<T>::N, VPT = ELEMS / VN;
  extern __shared__ uint4 ring[];
  __shared__ float red[2][32];
  __shared__ uint64_t full[kRingMaxStages];
  __shared__ int give_up;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lt = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const int nvec = h / VN, arrays = ds_add != nullptr ? 3 : 2, slot = rpb * nvec;
  const long long step = (long long)gridDim.x * rpb, first = (long long)blockIdx.x * rpb;
  const int turns = (int)((T_ - first + step - 1) / step);
  auto issue = [&](int i, int slot_i) {
    const long long t0 = first + i * step;
    const uint32_t bytes = (uint32_t)(t0 + rpb <= T_ ? rpb : (int)(T_ - t0)) * (uint32_t)nvec * 16u;
    uint64_t* bar = &full[slot_i];
    uint4* to = ring + slot_i * 3 * slot;
    ptx::mbar_expect_tx(bar, bytes * arrays);
    ptx::bulk_load(ptx::smem_u32(to), reinterpret_cast<const uint4*>(dy) + t0 * nvec, bytes, bar);
    ptx::bulk_load(ptx::smem_u32(to + slot), reinterpret_cast<const uint4*>(s) + t0 * nvec, bytes, bar);
    if (arrays == 3) ptx::bulk_load(ptx::smem_u32(to + 2 * slot), reinterpret_cast<const uint4*>(ds_add) + t0 * nvec, bytes, bar);
  };
  if (threadIdx.x == 0) {
    give_up = 0;
    for (int i = 0; i < stages; ++i) ptx::mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < stages && i < turns; ++i) issue(i, i);
  }
  float w[VPT][VN], dg[VPT][VN];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
#pragma unroll
    for (int i = 0; i < VN; i += 4) {
      const float4 g = v < nvec ? load4(gamma + (size_t)v * VN + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[u][i] = g.x; w[u][i + 1] = g.y; w[u][i + 2] = g.z; w[u][i + 3] = g.w;
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) dg[u][i] = 0.f;
  }
  const float inv_h = 1.0f / (float)h;
  float rs_next = first + sub < T_ ? rstd[first + sub] : 0.f;
  __syncthreads();
  bool alive = true;
  const int warp = threadIdx.x / kWarp, wpr = tpr / kWarp, w0 = warp / wpr * wpr;
  long long t = first + sub;
  uint4* out = reinterpret_cast<uint4*>(ds) + t * nvec;
  int now = 0, before = stages - 1;  // the slots of this turn and the last
  uint32_t parity = 0;
  for (int i = 0; i < turns; ++i, t += step, out += step * nvec) {
    const bool on = t < T_;
    const float rs = rs_next;
    rs_next = t + step < T_ ? rstd[t + step] : 0.f;
    const uint4* in = ring + now * 3 * slot + sub * nvec;
    const bool ok = ptx::mbar_try_wait(&full[now], parity) || ptx::mbar_wait(&full[now], parity, &give_up, status, 0);
    uint4 rd[VPT], rx[VPT];
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int v = lt + u * tpr;
      rd[u] = rx[u] = make_uint4(0, 0, 0, 0);
      if (ok && on && v < nvec) {
        rd[u] = in[v];
        rx[u] = in[slot + v];
      }
      float d[VN], x[VN];
      unpack(rd[u], d, T());
      unpack(rx[u], x, T());
#pragma unroll
      for (int c = 0; c < VN; ++c) {
        const float dx = d[c] * (x[c] * rs);
        dg[u][c] += dx;
        dot = fmaf(dx, w[u][c], dot);
      }
    }
    dot = warp_sum(dot);
    if (threadIdx.x % kWarp == 0) red[i & 1][warp] = dot;
    // every thread is past the stage of turn i - 1 here: it may be filled again
    if (!__syncthreads_and(ok)) {
      alive = false;
      break;
    }
    if (threadIdx.x == 0 && i > 0 && i - 1 + stages < turns) issue(i - 1 + stages, before);
    if (wpr > 1) dot = warp_sum(threadIdx.x % kWarp < wpr ? red[i & 1][w0 + threadIdx.x % kWarp] : 0.f);
    const float mean = dot * inv_h;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int v = lt + u * tpr;
      if (!on || v >= nvec) continue;
      float d[VN], x[VN], o[VN];
      unpack(rd[u], d, T());
      unpack(rx[u], x, T());
      if (arrays == 3) {
        unpack(in[2 * slot + v], o, T());
      } else {
#pragma unroll
        for (int c = 0; c < VN; ++c) o[c] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < VN; ++c) o[c] = fmaf(rs, fmaf(-(x[c] * rs), mean, d[c] * w[u][c]), o[c]);
      out[v] = pack(o, T());
    }
    before = now;
    if (++now == stages) {
      now = 0;
      parity ^= 1;
    }
  }
  if (!alive) {  // copies may still be on their way into this block's shared memory: let them land
    const unsigned long long t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) {}
    return;
  }
  // one partial row of dgamma a block: the row groups' columns are added through shared memory
  float* sums = reinterpret_cast<float*>(ring);
  if (rpb > 1) __syncthreads();
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int v = lt + u * tpr;
    if (v >= nvec) continue;
    float* to = rpb > 1 ? sums + (size_t)sub * h : partial + (size_t)blockIdx.x * h;
#pragma unroll
    for (int i = 0; i < VN; i += 4)
      store4(to + (size_t)v * VN + i, make_float4(dg[u][i], dg[u][i + 1], dg[u][i + 2], dg[u][i + 3]));
  }
  if (rpb > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < h; c += blockDim.x) {
      float sum = sums[c];
      for (int r = 1; r < rpb; ++r) sum += sums[(size_t)r * h + c];
      partial[(size_t)blockIdx.x * h + c] = sum;
    }
  }
}

// dgamma[c] = sum over the `parts` partials: p ascending by 32 within each of 32 strips (at most ten loads of a thread, under
// way together), then the strips by halves.  8 strips took 5.3 us beside the Large layer's 35 us of rows.
__global__ void __launch_bounds__(1024) dgamma_kernel(const float* partial, int parts, int h, float* __restrict__ dgamma) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials
  const int lane = threadIdx.x % 32, strip = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  constexpr int MOST = (kNormMaxParts + 31) / 32;
  float v[MOST], sum = 0.f;
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int p = strip + 32 * i;
    v[i] = c < h && p < parts ? partial[(size_t)p * h + c] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) sum += v[i];
  red[strip][lane] = sum;
  __syncthreads();
  sum = warp_sum(red[lane][strip]);  // of column `strip`
  if (lane == 0 && blockIdx.x * 32 + strip < h) dgamma[blockIdx.x * 32 + strip] = sum;
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

// The ring needs two stages of a row group at least: rows up to 34,128 bytes (all of bf16's, fp32 up to 8,528 columns).
// Wider rows go through the kernel that loads them into registers.
template <typename T, int ELEMS, int MAXT>
int launch_ring(const void* dy, const void* s, const float* gamma, const float* rstd, const void* ds_add, int T_, int h,
                void* ds, float* dgamma, float* partial, int* status, cudaStream_t st) {
  const int tpr = ((h + ELEMS - 1) / ELEMS + 31) / 32 * 32, rpb = tpr >= kRingThreads ? 1 : kRingThreads / tpr;
  const int stage = 3 * rpb * h * (int)sizeof(T);
  int stages = kRingBytes / stage;
  if (stages > kRingMaxStages) stages = kRingMaxStages;
  const int need = (T_ + rpb - 1) / rpb, most = num_sms() < kNormMaxParts ? num_sms() : kNormMaxParts;
  // two turns of one block, whose sum is dgamma itself, are quicker than two blocks and a second kernel
  const int blocks = need <= 2 ? 1 : need < most ? need : most;
  if (blocks == 1) partial = dgamma;
  static bool ready[64] = {};  // per device: the attribute is set once
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    cudaFuncSetAttribute(add_rmsnorm_bwd_ring_kernel<T, ELEMS, MAXT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  add_rmsnorm_bwd_ring_kernel<T, ELEMS, MAXT><<<blocks, tpr * rpb, (size_t)stages * stage, st>>>(
      static_cast<const T*>(dy), static_cast<const T*>(s), gamma, rstd, static_cast<const T*>(ds_add), T_, h, tpr, rpb, stages,
      static_cast<T*>(ds), partial, status);
  return blocks;
}

template <typename T>
void launch_bwd(const void* dy, const void* s, const float* gamma, const float* rstd, const void* ds_add, int T_, int h,
                void* ds, float* dgamma, float* partial, int* status, cudaStream_t st) {
  int parts = 0;
  if (2 * 3 * h * (int)sizeof(T) <= kRingBytes) {
    parts = h <= 8192 ? launch_ring<T, 16, 512>(dy, s, gamma, rstd, ds_add, T_, h, ds, dgamma, partial, status, st)
                      : launch_ring<T, 16, 1024>(dy, s, gamma, rstd, ds_add, T_, h, ds, dgamma, partial, status, st);
  } else if constexpr (sizeof(T) == 4) {
    const NormGeom g = norm_geom(h / Vec<T>::N);  // a row a block at these widths
    parts = T_ < kNormMaxParts ? T_ : kNormMaxParts;
    add_rmsnorm_bwd_wide_kernel<kMaxVec><<<parts, g.tpr, 0, st>>>(
        static_cast<const float*>(dy), static_cast<const float*>(s), gamma, rstd, static_cast<const float*>(ds_add), T_, h,
        static_cast<float*>(ds), partial);
  }
  count_launch(st);
  if (parts == 1 && 2 * 3 * h * (int)sizeof(T) <= kRingBytes) return;  // the ring's one block wrote dgamma
  // may begin while the rows are still at work (it waits for them by itself): its launch costs no time of its own
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((h + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, dgamma_kernel, (const float*)partial, parts, h, dgamma);
  count_launch(st);
}

}  // namespace

void launch_add_rmsnorm(int dtype, const void* x, const void* residual, const float* gamma, float eps, int T, int h, void* s,
                        void* y, void* q, float* q_scale, float* rstd, cudaStream_t st) {
  if (dtype == MOE_BF16) launch_fwd<__nv_bfloat16>(x, residual, gamma, eps, T, h, s, y, q, q_scale, rstd, st);
  else launch_fwd<float>(x, residual, gamma, eps, T, h, s, y, q, q_scale, rstd, st);
}

void launch_add_rmsnorm_bwd(int dtype, const void* dy, const void* s, const float* gamma, const float* rstd,
                            const void* ds_add, int T, int h, void* ds, float* dgamma, float* partial, int* status,
                            cudaStream_t st) {
  if (dtype == MOE_BF16) launch_bwd<__nv_bfloat16>(dy, s, gamma, rstd, ds_add, T, h, ds, dgamma, partial, status, st);
  else launch_bwd<float>(dy, s, gamma, rstd, ds_add, T, h, ds, dgamma, partial, status, st);
}

}  // namespace moe
