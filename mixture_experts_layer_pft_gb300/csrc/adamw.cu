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
// update of p reads the states before they are rounded.
//
// Measured on the Small layer's 554 M parameters in bf16 with fp32 masters: 32-bit states 28 bytes an
// element in 2235 us (102% of the measured copy rate), 8-bit states 16 bytes in 1454 us (90%; some 80
// instructions an element and the conversions are the rest).  adamw_kernel's tensors come by launch
// argument: 57 small ones in one launch, 24 us with the host's part.
//
// Every operation that decides a code is one correctly rounded fp32 operation (no contraction), so the codes
// follow from the formulas.
#include <cuda_fp8.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kOptBlock = 256;     // elements of one scale, handled by one warp
constexpr int kWarps = 8;
constexpr int kBlocks8 = 5, kBlocks32 = 2;  // thread blocks an SM, 8- and 32-bit states

template <int N>
struct AdamwArgs {
  AdamwTensor t[N];
  int first_chunk[N + 1];  // thread blocks before tensor i
  int n, first_tensor, blocks_per_warp;
  const float* lr;
  const int* step;
  const float* grad_scale;
  int* status;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, log_beta1, log_beta2, eps;
  uint32_t key[14];  // Philox's round keys
};

// Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1,
// 2, 3", 2011; 7 is the fewest rounds that pass that paper's tests).  The round keys are the host's.
__device__ __forceinline__ uint4 philox7(uint4 c, const uint32_t* key) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const unsigned long long a = (unsigned long long)c.x * 0xD2511F53u, b = (unsigned long long)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ key[2 * r], (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ key[2 * r + 1], (uint32_t)a);
  }
  return c;
}

// The update of p needs no correctly rounded root or quotient: these are within 2 of the last bit, of a term that is
// a thousandth of p.
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The code (without sign) of x >= 0 in an 8-bit float of M mantissa bits and smallest normal value 2^LOW, rounded up with
// the probability of what is cut off: 16 random bits are added below the kept bits of the fp32 pattern, in which an
// overflowing mantissa carries into the exponent as it should.  Below 2^LOW the grid is that of [2^LOW, 2^(LOW+1)),
// where x is moved to for the sum.  The exponent fields differ by a constant.
template <int M, int LOW>
__device__ __forceinline__ uint32_t random_code(float x, uint32_t bits16) {
  constexpr int DROP = 23 - M;
  constexpr float kLow = LOW == -6 ? 0x1p-6f : 0x1p-14f;
  static_assert(LOW == -6 || LOW == -14, "e4m3 or e5m2");
  const bool small = x < kLow;
  if (small) x = __fadd_rn(x, kLow);
  const uint32_t bias = (uint32_t)(small ? 127 + LOW : 126 + LOW) << 23;
  return (__float_as_uint(x) + ((bits16 << (DROP - 16)) | (1u << (DROP - 17))) - bias) >> DROP;
}

// One warp's 256 elements as they lie in memory: elements 4 lane .. 4 lane + 3 of either half.
template <bool BF16, bool Q8>
struct Raw {
  float4 p[2];
  uint2 g16[2];
  float4 g32[2];
  uint32_t m8[2], v8[2];
  float4 m32[2], v32[2];
  float ms, vs;

  // the whole block is inside the tensor
  __device__ __forceinline__ void load(const AdamwTensor& q, long long e0, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long e = e0 + h * 128 + lane * 4;
      if constexpr (BF16) {
        g16[h] = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(q.grad) + e);
        p[h] = load4(q.master + e);
      } else {
        g32[h] = load4(static_cast<const float*>(q.grad) + e);
        p[h] = load4(static_cast<const float*>(q.param) + e);
      }
      if constexpr (Q8) {
        m8[h] = *reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(q.m) + e);
        v8[h] = *reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(q.v) + e);
      } else {
        m32[h] = load4(static_cast<const float*>(q.m) + e);
        v32[h] = load4(static_cast<const float*>(q.v) + e);
      }
    }
    if constexpr (Q8) {
      ms = q.m_scale[e0 / kOptBlock];
      vs = q.v_scale[e0 / kOptBlock];
    }
  }
  // the last block of a tensor: one by one, zeros beyond its end
  __device__ __forceinline__ void load_tail(const AdamwTensor& q, long long e0, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float pp[4], mm[4], vv[4], g[4];
      uint32_t gb[4], mc = 0, vc = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long e = e0 + h * 128 + lane * 4 + i;
        const bool in = e < q.numel;
        gb[i] = 0;
        g[i] = pp[i] = mm[i] = vv[i] = 0.f;
        if (!in) continue;
        if constexpr (BF16) {
          gb[i] = static_cast<const unsigned short*>(q.grad)[e];
          pp[i] = q.master[e];
        } else {
          g[i] = static_cast<const float*>(q.grad)[e];
          pp[i] = static_cast<const float*>(q.param)[e];
        }
        if constexpr (Q8) {
          mc |= (uint32_t)static_cast<const unsigned char*>(q.m)[e] << (8 * i);
          vc |= (uint32_t)static_cast<const unsigned char*>(q.v)[e] << (8 * i);
        } else {
          mm[i] = static_cast<const float*>(q.m)[e];
          vv[i] = static_cast<const float*>(q.v)[e];
        }
      }
      p[h] = make_float4(pp[0], pp[1], pp[2], pp[3]);
      g16[h] = make_uint2(gb[0] | (gb[1] << 16), gb[2] | (gb[3] << 16));
      g32[h] = make_float4(g[0], g[1], g[2], g[3]);
      m8[h] = mc;
      v8[h] = vc;
      m32[h] = make_float4(mm[0], mm[1], mm[2], mm[3]);
      v32[h] = make_float4(vv[0], vv[1], vv[2], vv[3]);
    }
    if constexpr (Q8) {
      ms = q.m_scale[e0 / kOptBlock];
      vs = q.v_scale[e0 / kOptBlock];
    }
  }
};

__device__ __forceinline__ void unpack4_fp8(uint32_t w, __nv_fp8_interpretation_t kind, float scale, float* f) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), kind)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), kind)));
  f[0] = __fmul_rn(a.x, scale); f[1] = __fmul_rn(a.y, scale);
  f[2] = __fmul_rn(b.x, scale); f[3] = __fmul_rn(b.y, scale);
}
__device__ __forceinline__ void unpack4(const float4& v, float* f) { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }

struct Factors {
  float lr, grad_scale, rbc1, rbc2;  // rbc: 1 / (1 - b^t)
  uint32_t tensor, step;
};

// Four codes as bytes, the first lowest.
__device__ __forceinline__ uint32_t four_bytes(const uint32_t* b) {
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// The step of one block, from its raw values.  FAST: the block is inside the tensor and every gradient is finite; where
// one turns out not to be (v is infinite or NaN then, and its pattern at or above infinity's), nothing is stored and the
// answer is false.  Without FAST every element is looked at by itself.
template <bool BF16, bool Q8, bool FAST, int N>
__device__ __forceinline__ bool update(const AdamwArgs<N>& a, const AdamwTensor& q, const Factors& c, const Raw<BF16, Q8>& r,
                                       long long e0, int lane) {
  float p[2][4], m[2][4], v[2][4];
  float amax_m = 0.f;
  uint32_t amax_v = 0;  // v >= 0: patterns are ordered as the values are
  bool bad = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float g[4];
    if constexpr (BF16) {
      g[0] = __uint_as_float(r.g16[h].x << 16); g[1] = __uint_as_float(r.g16[h].x & 0xffff0000u);
      g[2] = __uint_as_float(r.g16[h].y << 16); g[3] = __uint_as_float(r.g16[h].y & 0xffff0000u);
    } else {
      unpack4(r.g32[h], g);
    }
    unpack4(r.p[h], p[h]);
    if constexpr (Q8) {
      unpack4_fp8(r.m8[h], __NV_E4M3, r.ms, m[h]);
      unpack4_fp8(r.v8[h], __NV_E5M2, r.vs, v[h]);
    } else {
      unpack4(r.m32[h], m[h]);
      unpack4(r.v32[h], v[h]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gi = __fmul_rn(g[i], c.grad_scale), gg = __fmul_rn(gi, gi);
      if (FAST || gg <= FLT_MAX) {
        m[h][i] = __fadd_rn(__fmul_rn(m[h][i], a.beta1), __fmul_rn(gi, a.one_minus_beta1));
        v[h][i] = __fadd_rn(__fmul_rn(v[h][i], a.beta2), __fmul_rn(gg, a.one_minus_beta2));
        // v below the smallest normal number counts as that in the root
        const float u = m[h][i] * c.rbc1 * rcp_approx(sqrt_approx(fmaxf(v[h][i] * c.rbc2, FLT_MIN)) + a.eps);
        p[h][i] = fmaf(-c.lr, fmaf(q.weight_decay, p[h][i], u), p[h][i]);
      } else {
        bad = true;
      }
      amax_m = fmaxf(amax_m, fabsf(m[h][i]));
      amax_v = max(amax_v, __float_as_uint(v[h][i]));
    }
  }
  if constexpr (Q8) amax_v = __reduce_max_sync(0xffffffffu, amax_v);
  if constexpr (FAST) {
    if (__any_sync(0xffffffffu, amax_v >= 0x7f800000u)) return false;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long e = e0 + h * 128 + lane * 4;
    if constexpr (FAST) {
      const float4 o = make_float4(p[h][0], p[h][1], p[h][2], p[h][3]);
      if constexpr (BF16) {
        store4(q.master + e, o);
        store4(static_cast<__nv_bfloat16*>(q.param) + e, o);
      } else {
        store4(static_cast<float*>(q.param) + e, o);
      }
      if constexpr (!Q8) {
        store4(static_cast<float*>(q.m) + e, make_float4(m[h][0], m[h][1], m[h][2], m[h][3]));
        store4(static_cast<float*>(q.v) + e, make_float4(v[h][0], v[h][1], v[h][2], v[h][3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= q.numel) break;
        if constexpr (BF16) {
          q.master[e + i] = p[h][i];
          static_cast<__nv_bfloat16*>(q.param)[e + i] = __float2bfloat16_rn(p[h][i]);
        } else {
          static_cast<float*>(q.param)[e + i] = p[h][i];
        }
        if constexpr (!Q8) {
          static_cast<float*>(q.m)[e + i] = m[h][i];
          static_cast<float*>(q.v)[e + i] = v[h][i];
        }
      }
    }
  }
  if constexpr (Q8) {
    amax_m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax_m)));
    const float ms = __fmul_rn(fmaxf(amax_m, 0x1p-100f), 0x1p-8f);
    const float vs = __fmul_rn(fmaxf(__uint_as_float(amax_v), 0x1p-100f), 0x1p-15f);
    const float rm = __frcp_rn(ms), rv = __frcp_rn(vs);
    if (lane == 0) {
      q.m_scale[e0 / kOptBlock] = ms;
      q.v_scale[e0 / kOptBlock] = vs;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long e = e0 + h * 128 + lane * 4;
      const unsigned long long four = (unsigned long long)e >> 2;
      const uint4 w4 = philox7(make_uint4((uint32_t)four, (uint32_t)(four >> 32), c.tensor, c.step), a.key);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      uint32_t cm[4], cv[4], sign[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cm[i] = random_code<3, -6>(__fmul_rn(fabsf(m[h][i]), rm), w[i] & 0xffffu);
        cv[i] = random_code<2, -14>(__fmul_rn(v[h][i], rv), w[i] >> 16);
        if (v[h][i] > 0.f) cv[i] = max(cv[i], 1u);
        sign[i] = __float_as_uint(m[h][i]);
      }
      const uint32_t signs = __byte_perm(__byte_perm(sign[0], sign[1], 0x0073), __byte_perm(sign[2], sign[3], 0x0073), 0x5410);
      const uint32_t qm = four_bytes(cm) | (signs & 0x80808080u), qv = four_bytes(cv);
      unsigned char* to_m = static_cast<unsigned char*>(q.m) + e;
      unsigned char* to_v = static_cast<unsigned char*>(q.v) + e;
      if constexpr (FAST) {
        *reinterpret_cast<uint32_t*>(to_m) = qm;
        *reinterpret_cast<uint32_t*>(to_v) = qv;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (e + i >= q.numel) break;
          to_m[i] = (unsigned char)(qm >> (8 * i));
          to_v[i] = (unsigned char)(qv >> (8 * i));
        }
      }
    }
  }
  if (bad) flag_status(a.status, MOE_STATUS_NOT_FINITE);
  return true;
}

// One block by itself: the last of a tensor, or one with a gradient that is not finite.
template <bool BF16, bool Q8, int N>
__device__ __noinline__ void update_alone(const AdamwArgs<N>& a, const AdamwTensor& q, const Factors& c, long long e0, int lane) {
  Raw<BF16, Q8> r;
  r.load_tail(q, e0, lane);
  update<BF16, Q8, false, N>(a, q, c, r, e0, lane);
}

template <int N>
__device__ __forceinline__ Factors factors(const AdamwArgs<N>& a, int step, int tensor) {
  Factors c;
  c.lr = *a.lr;
  c.grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  c.rbc1 = -1.0f / expm1f((float)step * a.log_beta1);  // 1 - b^t without cancellation
  c.rbc2 = -1.0f / expm1f((float)step * a.log_beta2);
  c.tensor = (uint32_t)(a.first_tensor + tensor);
  c.step = (uint32_t)step;
  return c;
}

// A warp's `blocks` blocks.  With 32-bit states HBM is the bound and few warps an SM reach it when each loads a block
// ahead.  8-bit states are bound by some 80 instructions an element, which want warps to choose from: 40 an SM without a
// block ahead take 1454 us for the Small layer, 32 take 1497, 48 1529, 32 with a block ahead in registers 1581, 24 with two
// or three ahead in shared memory 1702.  (40 have 48 registers each and spill 176 bytes a thread; 48 spill more.)
template <bool BF16, bool Q8, int N>
__device__ __forceinline__ void run_warp(const AdamwArgs<N>& a, const AdamwTensor& q, int tensor, int step, long long base,
                                         int blocks, int lane) {
  const long long left = q.numel - base;
  const int full = left >= (long long)blocks * kOptBlock ? blocks : (int)(left / kOptBlock);
  Raw<BF16, Q8> r0;
  if (!Q8 && full > 0) r0.load(q, base, lane);
  const Factors c = factors(a, step, tensor);  // while the first block is on its way
  if constexpr (Q8) {
#pragma unroll 1
    for (int b = 0; b < full; ++b) {
      const long long e0 = base + (long long)b * kOptBlock;
      r0.load(q, e0, lane);
      if (!update<BF16, Q8, true, N>(a, q, c, r0, e0, lane)) update_alone<BF16, Q8, N>(a, q, c, e0, lane);
    }
  } else {
    Raw<BF16, Q8> r1;
#pragma unroll 1
    for (int b = 0; b < full; b += 2) {
      const long long e0 = base + (long long)b * kOptBlock;
      if (b + 1 < full) r1.load(q, e0 + kOptBlock, lane);
      if (!update<BF16, Q8, true, N>(a, q, c, r0, e0, lane)) update_alone<BF16, Q8, N>(a, q, c, e0, lane);
      if (b + 1 >= full) break;
      if (b + 2 < full) r0.load(q, e0 + 2 * kOptBlock, lane);
      if (!update<BF16, Q8, true, N>(a, q, c, r1, e0 + kOptBlock, lane)) update_alone<BF16, Q8, N>(a, q, c, e0 + kOptBlock, lane);
    }
  }
  if (full < blocks && left > (long long)full * kOptBlock)
    update_alone<BF16, Q8, N>(a, q, c, base + (long long)full * kOptBlock, lane);
}

template <int N, bool Q8>
__global__ void __launch_bounds__(kWarps * 32, Q8 ? kBlocks8 : kBlocks32) adamw_kernel(const __grid_constant__ AdamwArgs<N> a) {
  int lo = 0, hi = a.n - 1;  // the tensor of this thread block
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first_chunk[mid] <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamwTensor& q = a.t[lo];
  const int lane = threadIdx.x % kWarp;
  const long long warp = ((long long)blockIdx.x - a.first_chunk[lo]) * kWarps + threadIdx.x / kWarp;
  const long long base = warp * a.blocks_per_warp * kOptBlock;
  if (base >= q.numel) return;
  const int step = *a.step;
  if (step < 1) {
    if (lane == 0) flag_status(a.status, MOE_STATUS_BAD_INDEX);
    return;
  }
  if (q.dtype == MOE_BF16) run_warp<true, Q8, N>(a, q, lo, step, base, a.blocks_per_warp, lane);
  else run_warp<false, Q8, N>(a, q, lo, step, base, a.blocks_per_warp, lane);
}

template <int N>
void launch_some(const AdamwTensor* t, int n, int first_tensor, const AdamwScalars& c, cudaStream_t st) {
  AdamwArgs<N> a;
  // A warp's setup (its tensor, the bias corrections) costs about a block's work.  With 8-bit states, bound by the
  // instructions, 16 blocks share it (the Small layer: 4 blocks 1721 us, 8 1626, 16 1585, 32 1568); with 32-bit states,
  // bound by HBM, shorter runs keep its many streams closer together (4: 2244, 8: 2277, 16: 2286, 32: 2372).  Where
  // that leaves too few warps for the SMs, a warp takes fewer.  Long runs are then evened out to whole rounds of the
  // warps that the SMs hold, for a last round of a few warps takes as long as a full one (16.5 M parameters with 8-bit
  // states: 1.3 rounds of 8 blocks 63.5 us, one of 11 blocks 57.9).  Short ones are not: there more warps than one round
  // cover each other's setup (4.5 M parameters: 2 blocks 24.0 us, an even 3 25.0).
  long long all = 0, chunks = 0;
  for (int i = 0; i < n; ++i) all += (t[i].numel + kOptBlock - 1) / kOptBlock;
  a.blocks_per_warp = c.q8 ? 16 : 4;
  while (a.blocks_per_warp > 1 && all < (long long)num_sms() * 32 * a.blocks_per_warp) a.blocks_per_warp /= 2;
  if (a.blocks_per_warp >= 8) {
    const long long round = (long long)num_sms() * kWarps * kBlocks8, rounds = (all + 16 * round - 1) / (16 * round);
    a.blocks_per_warp = (int)((all + round * rounds - 1) / (round * rounds));
  }
  const long long chunk = (long long)kOptBlock * kWarps * a.blocks_per_warp;
  for (int i = 0; i < n; ++i) {
    a.t[i] = t[i];
    a.first_chunk[i] = (int)chunks;
    chunks += (t[i].numel + chunk - 1) / chunk;
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
  for (int r = 0; r < 7; ++r) {
    a.key[2 * r] = (uint32_t)c.seed + (uint32_t)r * 0x9E3779B9u;
    a.key[2 * r + 1] = (uint32_t)(c.seed >> 32) + (uint32_t)r * 0xBB67AE85u;
  }
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
