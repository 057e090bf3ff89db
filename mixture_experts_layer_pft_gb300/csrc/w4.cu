// Routed experts over 4-bit weights, for the few tokens of a decode step, and the weights' quantisation.
//
//   W[n, i] = (nibble - 8) * scale[n, i / G];  a = silu(W1_e x) * (W3_e x);  y[t] = sum_j w_j W2_e a.
//
// The floor is the active experts' bytes: 182 MB, 27 us, for one token of the Large layer (h 7168, f 2048, k 8 of 256).  What
// bounds the kernels instead is instructions and their latency: a byte of weights is two products, and turning nibbles into
// operands costs more than multiplying them.  Measured on this GPU, instructions a clock and SM: dp4a, LOP3, IMAD, I2F and bf16x2 FMA 1.9
// each, mma.sync bf16 16x8x16 0.50, mma.sync s8 16x8x32 0.06.  Two forms follow from that.
//
// "Few" (one token, or up to 8 and 12 rows, whose activations fit in shared memory): integers through dp4a, see below.
// Two launches: the first writes `a`, the second adds each token's outputs over its experts in registers; it starts early and has its
// first weights under way while the first still runs.  Large layer, one token in 8 bits: 52 us (51% of the floor's rate;
// tensor cores in this place 86 us).  Of a warp's 330 and 238 instructions a step of 16 outputs x 128 inputs (two matrices, one),
// some 208 and 112 are the products and their reads of shared memory; the rest converts x in every block, finds experts and
// addresses and copies.  2.4 are issued a clock and SM, and half of a warp's wait in the first kernel is for its next weights.
// Small layer (h 2048, f 1408, 6 of 64): 14 us, of which the launches, the chain from topk_idx to y and the host are most.
//
// "Many": tensor cores with 16 outputs as M and token rows as N.  A nibble n masked into the mantissa of an f16 1024 is
// 1024 + n, and n - 8 after a subtraction, exactly: eight nibbles are operands after nine instructions (in bf16 eleven).
// Activations go in as planes of f16 over one scale per row and step, which is a power of two: x in e4m3 and bf16 as one,
// exactly; x in fp32 as two, of 23 bits; `a` as one of 11 bits beside y's 8 in 16-bit layers, as two in fp32 ones (bf16
// planes take one more each).  Groups' sums are kept apart in fp32 and scaled once, so no weight is rounded.  An expert's
// rows come in units of 16 (fp32: 8); experts' output rows go to scratch, and a combine adds them.  64 tokens of the Medium
// layer (h 5120, f 1536, 6 of 128, skewed): 175 to 195 us against a floor of 36 (with bf16 operands 213); 13 fp32 tokens of
// the long-sequence layer (h f 2048, 2 of 128, groups of 32): 53 against 5 (70).  Unpacking for one or two tiles of rows,
// copies and the groups' scales, some 12 instructions a product at 2 a clock, as two blocks an SM do not cover their
// latencies, and five launches are the rest.
//
// Other operands: n alone is the subnormal f16 n 2^-24, with the 8 taken off where a group's sums start: five instructions,
// 155 to 163 us, but the tensor core aligns its products as if n were 1024, and what is lost of the sums (4e-6 of the
// outputs' norm) grows with the largest activation, also where it meets weights of zero.  e4m3 operands (n 2^-9, three
// instructions): 288 us, mma.sync does 0.28 of those a clock and SM once they change.  tcgen05 would want the unpacked
// weights in shared memory and its sums read back after each group, as a scale inside the operands would round them; it
// would pay from some 32 rows an expert on, and is not built.
//
// A warp's step is 16 outputs x 128 inputs.  The sum over inputs may run in any order, so lane (g, q) = (lane / 4, lane % 4)
// takes for outputs g and g + 8 the G/4 consecutive inputs of each group that are contiguous in its 4-bit row: the weights
// need no other layout than [output][input / 2].  Two nibbles of a word sit 16 bits apart as inputs i and i + 4, so for the
// tensor cores eight activations go in as (0,4) (1,5) (2,6) (3,7); planes are stored in that order.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;       // outputs of a warp
constexpr int kStep = 128;      // inputs of a warp's step
constexpr int kFewTokens = 8, kFewRows = 64, kSeveralRows = 12;
constexpr int kTurn = 4;         // steps between barriers of the many form
constexpr int kStages = 2;       // turns of activations in shared memory (three: the same)
// Rows of a unit of the many form.  With two planes a second tile of rows would take the registers that hide the latency
// (13 tokens of the long-sequence layer: 92 us).
template <int P> constexpr int kPass = P == 1 ? 16 : 8;
// Shared memory for the few form's activations.  One token may leave room for a single block of the second kernel on an SM (h
// 4096, 8 experts, f 5632: 85 us, the many form 119; f 7168: 103 and 142); several are left to the many form then (4 tokens of
// 3, h f 4096: 104 us, a block an SM 136).
template <int ROWS> constexpr int kFewBytes = (ROWS == 1 ? 200 : 100) * 1024;
constexpr int kFewSteps = 128;  // of a warp: kFewBytes / (128 inputs x 3.25 bytes) / 8, and one more an expert
static_assert(kFewBytes<1> / (kStep / 16 * 52) / kWarps + kFewRows <= kFewSteps, "a warp's list holds its steps");
// One token: blocks an SM of the first kernel, and steps of weights under way in a warp of either.  Large / Small layer, both
// kernels: 4, 1 and 4 52 / 16.3 us; 3, 1 and 4 60 / 16.6; 3, 2 and 4 63 / 16.7; 2, 2 and 4 58 / 16.6; 4, 1 and 2 52.5 / 17.7.
constexpr int kUpBlocks = 4, kUpAhead = 1, kDownAhead = 4;

struct W4Mat {
  const unsigned char* q;
  const __nv_bfloat16* s;
};

// Start of the dependent launch as soon as every block of this one runs; wait for the launch this one depends on.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct E4M3 { unsigned char v; };

// A lane's place in a matrix of one expert: byte offset of output g's row and this lane's quarter of a group, and offset of
// its scales; output g + 8 lies `q8` and `s8` further.  32 bits suffice for an expert's matrix.
template <int G>
struct LanePlace {
  uint32_t q, s, q8, s8;
  int k;  // first input of this lane in a step's first group
  __device__ __forceinline__ LanePlace(int out0, int K, int lane) {
    const uint32_t row = out0 + lane / 4, groups = (K + G - 1) / G;
    k = (lane % 4) * (G / 4);
    q = row * (uint32_t)(K / 2) + k / 2;
    s = row * groups;
    q8 = 8u * (uint32_t)(K / 2);
    s8 = 8u * groups;
  }
};

// Where the eight inputs number c of a step (16 of them) go: the word, and the lane quarter that reads it.
template <int G>
__device__ __forceinline__ void place_of(int c, int* word, int* quarter) {
  *word = c / (G / 8) * (G / 32) + c % (G / 32);
  *quarter = c % (G / 8) / (G / 32);
}

// ------------------------------------------------------------------------------------ few rows

// With one or two rows an expert the tensor cores would be fed mostly zeros, and the latency of their products is what
// takes the time.  Here the nibbles stay integers: 8 inputs' nibbles become two words of signed bytes 16 * (nibble - 8) in
// three instructions, and dp4a adds their products with the activations.  Those are integers
// too, of 24 bits as three signed bytes, with one fp32 scale per 16 inputs: an activation is off by at most 2^-24 of the
// largest of its 16, as much as an fp32 sum of the 16 may lose.  (Two bytes, 16 bits, took 47 us where three take 52, but
// an input 2000 times its neighbours left these four bits of their own: where its weights are small or zero, outputs were off by
// more than their type's rounding.)  Sums of 16 products are exact in 32 bits.
//
// Also measured for a token of the Large layer: bulk copies of the rows into shared memory (pieces of 512 bytes: 76 us, of
// 1024: 70, the copies are too small), and a warp along 1024 inputs of one output instead of 16 outputs x 128 (57 to 75).

struct FewArgs {
  const void* x;          // gate/up: [T, K] of X; down: nothing
  const float* x_scale;
  const int* topk_idx;
  const float* topk_w;
  int T, k, E, K, N;      // K inputs, N outputs
  W4Mat mat[2];
  unsigned char* bytes;   // `a` as integers: [T*k][f/16][3][16]
  float* scales;          // and its scales: [T*k][f/16]
  void* y;                // down: y [T, N]
  int* status;
};

// Rows of topk_idx that name expert e, as bits (at most 64 rows).
__device__ __forceinline__ unsigned long long rows_of(const int* __restrict__ topk_idx, int rows, int e, int lane) {
  const bool lo = lane < rows && __ldg(topk_idx + lane) == e;
  const bool hi = lane + 32 < rows && __ldg(topk_idx + lane + 32) == e;
  return (unsigned long long)__ballot_sync(0xffffffffu, lo) | ((unsigned long long)__ballot_sync(0xffffffffu, hi) << 32);
}
// Of a row mask, token t's bits, moved to bit 0.
__device__ __forceinline__ unsigned long long bits_of(unsigned long long mask, int t, int k) {
  return (mask >> (t * k)) & (k < 64 ? (1ull << k) - 1ull : ~0ull);
}

// The largest integer used, somewhat below three signed bytes 127, 127, 127 (a product with fp32's 24 bits may end a unit above).
constexpr int kPlanes = 3;
constexpr float kMostInt = 8355000.f;

// Scale of 16 values whose largest magnitude has the pattern `amax`, and its inverse.  Values that are no finite numbers
// make it NaN; below 2^-90 all count as zeros.  The scale carries the 1/16 of the weights' bytes.
__device__ __forceinline__ float int_scale(uint32_t amax, float* inverse) {
  const float m = __uint_as_float(amax);
  *inverse = m < 0x1p-90f || amax >= 0x7f800000u ? 0.f : kMostInt / m;
  return amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : m < 0x1p-90f ? 0.f : m * (1.0f / (16.0f * kMostInt));
}
// Byte planes of four integers, the highest first: a lower plane's bytes are the integers' own (read as signed they are up
// to 128 too small, which is added before the next shift).
__device__ __forceinline__ void int_planes(int q0, int q1, int q2, int q3, uint32_t* plane) {
  auto bytes = [](int x0, int x1, int x2, int x3, uint32_t from) {  // byte 0 or 1 of each
    return __byte_perm(__byte_perm(x0, x1, from), __byte_perm(x2, x3, from), 0x5410);
  };
  plane[2] = bytes(q0, q1, q2, q3, 0x0040);
  q0 = (q0 + 128) >> 8; q1 = (q1 + 128) >> 8; q2 = (q2 + 128) >> 8; q3 = (q3 + 128) >> 8;
  plane[1] = bytes(q0, q1, q2, q3, 0x0040);
  plane[0] = bytes(q0 + 128, q1 + 128, q2 + 128, q3 + 128, 0x0051);
}
// Place of input i of 16 in its 16 bytes: per 8 inputs the even ones, then the odd ones, as a word's nibbles lie.
__device__ __forceinline__ int byte_place(int i) { return (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3); }

// Sixteen consecutive activations as fp32.
__device__ __forceinline__ void load16(const float* p, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) unpack(__ldg(reinterpret_cast<const uint4*>(p) + i), f + 8 * i, __nv_bfloat16());
}
__device__ __forceinline__ void load16(const E4M3* p, float* f) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3)));
    f[2 * i] = v.x; f[2 * i + 1] = v.y;
  }
}

// Of a lane's inputs of a step, the sums for N outputs: w their words, g their groups' scales.  A lane has one scale for two
// words, with groups of 32 one a word.  bytes, scale: the row's in shared memory at the lane's first input k of the step (k / 16
// pieces from the row's start); rows are padded to whole steps with zeros.
template <int G, int N>
__device__ __forceinline__ void int_dots(const unsigned char* bytes, const float* scale, int k, const uint32_t* const* w,
                                         const __nv_bfloat16* const* g, float* sum) {
  constexpr int SCALES = G == 32 ? 4 : 2, WORDS = 4 / SCALES;
#pragma unroll
  for (int i = 0; i < SCALES; ++i) {
    const int block = G == 128 ? i : i * (G / 16);  // of one or two words
    uint32_t q[kPlanes][WORDS][2];
    const float s = scale[block];
#pragma unroll
    for (int p = 0; p < kPlanes; ++p) {
      const unsigned char* b = bytes + (block * kPlanes + p) * 16;
      if constexpr (G == 32) {
        const uint2 u = *reinterpret_cast<const uint2*>(b + (k & 8));
        q[p][0][0] = u.x; q[p][0][1] = u.y;
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(b);
        q[p][0][0] = u.x; q[p][0][1] = u.y; q[p][WORDS - 1][0] = u.z; q[p][WORDS - 1][1] = u.w;
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      int d[kPlanes];
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) d[p] = 0;
#pragma unroll
      for (int j = 0; j < WORDS; ++j) {
        // the signed bytes 16 (nibble - 8): even inputs, odd inputs
        const uint32_t word = w[n][i * WORDS + j];
        const int even = (int)(((word << 4) ^ 0x88888888u) & 0xf0f0f0f0u), odd = (int)((word ^ 0x88888888u) & 0xf0f0f0f0u);
#pragma unroll
        for (int p = 0; p < kPlanes; ++p) d[p] = __dp4a(odd, (int)q[p][j][1], __dp4a(even, (int)q[p][j][0], d[p]));
      }
      const float v = fmaf((float)(d[0] * 256 + d[1]), 256.f, (float)d[2]);
      if constexpr (G == 128) sum[n] = i == 0 ? v * s : fmaf(v, s, sum[n]);
      else sum[n] = fmaf(v * s, __bfloat162float(g[n][i]), i == 0 ? 0.f : sum[n]);
    }
  }
  if constexpr (G == 128) {
#pragma unroll
    for (int n = 0; n < N; ++n) sum[n] *= __bfloat162float(g[n][0]);
  }
}

// A lane's words and scales of a step, for outputs g and g + 8 of MATS matrices.
template <int G, int MATS>
struct IntWeights {
  uint32_t w[MATS][2][4] = {};
  __nv_bfloat16 s[MATS][2][kStep / G];

  // q, s: of output g at the lane's first input of the step; q8, s8: to output g + 8; k: that input
  __device__ __forceinline__ void load(const unsigned char* const* q, const __nv_bfloat16* const* sc, uint32_t q8, uint32_t s8, int k,
                                       int k0, int K) {
#pragma unroll
    for (int i = 0; i < kStep / G; ++i) {
      const bool in = k + i * G < K;  // K is a multiple of 32: of a lane's G / 4 inputs none or all are inside
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const unsigned char* p = q[m] + r * q8;
          if (in) {  // beyond K the words keep what they held: the activations there are zeros
            if constexpr (G == 128) {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
              w[m][r][0] = u.x; w[m][r][1] = u.y; w[m][r][2] = u.z; w[m][r][3] = u.w;
            } else if constexpr (G == 64) {
              const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + 32 * i));
              w[m][r][2 * i] = u.x; w[m][r][2 * i + 1] = u.y;
            } else {
              w[m][r][i] = __ldg(reinterpret_cast<const uint32_t*>(p + 16 * i));
            }
          }
          if (G == 128 || i == 0 || k0 + i * G < K) s[m][r][i] = sc[m][r * s8 + i];
          else s[m][r][i] = __float2bfloat16_rn(0.f);
        }
    }
  }
};

// `a` of 32 outputs of the slot's expert for the tokens that chose it: two tiles of outputs, the inputs' steps over four
// warps each.  One slot a row of topk_idx: the first row of an expert does them all.  ROWS: 1 for one token, else 8.
template <typename X, int G, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, ROWS == 1 ? kUpBlocks : 2) w4_few_up_kernel(const __grid_constant__ FewArgs a) {
  constexpr int AHEAD = kUpAhead, SPLIT = kWarps / 2;
  extern __shared__ uint4 acts[];  // bytes [row][8 S][3][16], then scales [row][8 S]
  __shared__ float red[kWarps][2][kTile][ROWS + (ROWS > 1)];
  __shared__ int token[kFewTokens];
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, tile = warp / SPLIT, part = warp % SPLIT;
  launch_dependents();
  const int rows = a.T * a.k, S = (a.K + kStep - 1) / kStep, blocks = S * 8;
  const int e = __ldg(a.topk_idx + blockIdx.y);
  if ((unsigned)e >= (unsigned)a.E) return;  // flagged by the second kernel
  const LanePlace<G> at((blockIdx.x * 2 + tile) * kTile, a.K, lane);
  const unsigned char* q[2];
  const __nv_bfloat16* sc[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    q[m] = a.mat[m].q + (size_t)e * a.N * (a.K / 2) + at.q + part * (kStep / 2);
    sc[m] = a.mat[m].s + (size_t)e * a.N * ((a.K + G - 1) / G) + at.s + part * (kStep / G);
  }
  int ahead = part;  // the next step to load
  IntWeights<G, 2> w[AHEAD];
  auto load = [&](IntWeights<G, 2>& to) {
    if (ahead < S) to.load(q, sc, at.q8, at.s8, ahead * kStep + at.k, ahead * kStep, a.K);
    ahead += SPLIT;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      q[m] += SPLIT * (kStep / 2);
      sc[m] += SPLIT * (kStep / G);
    }
  };
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) load(w[d]);
  unsigned long long mask = rows_of(a.topk_idx, rows, e, lane);
  if (__ffsll(mask) - 1 != (int)blockIdx.y) return;  // an earlier row's block does this expert
  const bool mine = lane < a.T && bits_of(mask, lane < a.T ? lane : 0, a.k) != 0;
  const unsigned chosen = __ballot_sync(0xffffffffu, mine);
  const int n = __popc(chosen);
  if (mine) token[__popc(chosen & ((1u << lane) - 1u))] = lane;  // every warp writes the same
  __syncwarp();
  float* scales = reinterpret_cast<float*>(acts + (size_t)n * blocks * kPlanes);
  for (int r = 0; r < n; ++r) {
    const X* x = static_cast<const X*>(a.x) + (size_t)token[r] * a.K;
    for (int i = threadIdx.x; i < blocks; i += kWarps * 32) {
      float f[16] = {}, inverse;
      if (i * 16 < a.K) load16(x + i * 16, f);
      uint32_t amax = 0;
#pragma unroll
      for (int c = 0; c < 16; ++c) amax = max(amax, __float_as_uint(f[c]) & 0x7fffffffu);
      float scale = int_scale(amax, &inverse);
      if constexpr (sizeof(X) == 1) scale *= __ldg(a.x_scale + (size_t)token[r] * S + i / 8);
      scales[r * blocks + i] = scale;
      uint32_t word[4][kPlanes];
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // of eight inputs the even ones, then the odd ones
        const float* v = f + c / 2 * 8 + (c & 1);
        int_planes(__float2int_rn(v[0] * inverse), __float2int_rn(v[2] * inverse), __float2int_rn(v[4] * inverse),
                   __float2int_rn(v[6] * inverse), word[c]);
      }
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) acts[(r * blocks + i) * kPlanes + p] = make_uint4(word[0][p], word[1][p], word[2][p], word[3][p]);
    }
  }
  __syncthreads();
  const unsigned char* bytes = reinterpret_cast<const unsigned char*>(acts) + (part * 8 + at.k / 16) * (16 * kPlanes);
  const float* scale = scales + part * 8 + at.k / 16;
  float acc[2][2][ROWS] = {};
  for (int s0 = part; s0 < S; s0 += SPLIT * AHEAD) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (s0 + d * SPLIT >= S) break;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (r >= n) break;
        const uint32_t* words[4] = {w[d].w[0][0], w[d].w[0][1], w[d].w[1][0], w[d].w[1][1]};
        const __nv_bfloat16* groups[4] = {w[d].s[0][0], w[d].s[0][1], w[d].s[1][0], w[d].s[1][1]};
        float sum[4];
        int_dots<G, 4>(bytes + r * blocks * (16 * kPlanes), scale + r * blocks, at.k, words, groups, sum);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int o = 0; o < 2; ++o) acc[m][o][r] += sum[m * 2 + o];
      }
      bytes += SPLIT * 8 * (16 * kPlanes);
      scale += SPLIT * 8;
      load(w[d]);
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float v = acc[m][o][r];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (lane % 4 == 0) red[warp][m][lane / 4 + o * 8][r] = v;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kTile * ROWS; i += kWarps * 32) {  // 16 threads a tile's row: whole warps
    const int o = i % kTile, t = i / kTile % 2, r = i / (2 * kTile);
    const bool on = r < n;
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int c = 0; c < SPLIT; ++c) v[m] += red[t * SPLIT + c][m][o][r];
    const float value = on ? v[0] * sigmoidf_(v[0]) * v[1] : 0.f;
    uint32_t amax = __float_as_uint(value) & 0x7fffffffu;
#pragma unroll
    for (int c = 8; c > 0; c >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, c));
    float inverse;
    const float sx = int_scale(amax, &inverse);
    if (on) {
      const size_t row = (size_t)token[r] * a.k + __ffsll(bits_of(mask, token[r], a.k)) - 1, block = row * (a.N / 16) + blockIdx.x * 2 + t;
      uint32_t plane[kPlanes];
      int_planes(__float2int_rn(value * inverse), 0, 0, 0, plane);
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) a.bytes[(block * kPlanes + p) * 16 + byte_place(o)] = (unsigned char)plane[p];
      if (o == 0) a.scales[block] = sx;
    }
  }
}

// y of 16 outputs for all tokens: the steps of all experts' products over the warps, each token's sum over its experts in
// registers.
template <typename T, int G, int ROWS, int BLOCKS>
__global__ void __launch_bounds__(kWarps * 32, BLOCKS) w4_few_down_kernel(const __grid_constant__ FewArgs a) {
  constexpr int AHEAD = kDownAhead;
  extern __shared__ uint4 acts[];  // `a`: bytes [row][8 S][3][16], then scales [row][8 S]
  __shared__ float red[kWarps][kTile][ROWS + (ROWS > 1)];
  __shared__ int expert[kFewRows], row[kFewRows][ROWS], idx[kFewRows];
  __shared__ float weight[kFewRows][ROWS];
  __shared__ unsigned lead[2];
  __shared__ unsigned short list[kWarps][kFewSteps];
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int rows = a.T * a.k, S = (a.K + kStep - 1) / kStep, blocks = S * 8;
  // the experts of these tokens, ascending, with each token's row of `a` and weight
  if (threadIdx.x < kFewRows) idx[threadIdx.x] = threadIdx.x < rows ? __ldg(a.topk_idx + threadIdx.x) : -1;
  __syncthreads();
  if (threadIdx.x < kFewRows) {
    const int e = idx[threadIdx.x];
    unsigned long long mask = 0, below = 0;
    for (int r = 0; r < rows; ++r) {
      mask |= (unsigned long long)(idx[r] == e) << r;
      below |= (unsigned long long)(idx[r] < e) << r;
    }
    const bool in = threadIdx.x < rows && (unsigned)e < (unsigned)a.E;
    if (threadIdx.x < rows && !in && blockIdx.x == 0) flag_status(a.status, MOE_STATUS_BAD_INDEX);
    const bool leads = in && __ffsll(mask) - 1 == (int)threadIdx.x;
    const unsigned ballot = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) lead[warp] = ballot;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (leads) {
      const int place = __popcll(below & (lead[0] | (unsigned long long)lead[1] << 32));
      expert[place] = e;
      for (int t = 0; t < ROWS; ++t) {
        unsigned long long mine = t < a.T ? bits_of(mask, t, a.k) : 0;
        row[place][t] = mine != 0 ? t * a.k + __ffsll(mine) - 1 : -1;
        float sum = 0.f;
        for (; mine != 0; mine &= mine - 1) sum += __ldg(a.topk_w + t * a.k + __ffsll(mine) - 1);
        weight[place][t] = sum;
      }
    }
  }
  __syncthreads();
  // Warp w takes the steps kb = w - e (mod 8) of expert e, so that a token's sum is the same whatever else is in the batch,
  // and experts whose steps are no multiple of 8 load the warps evenly.  Its list: (kb, number of the expert), experts in
  // order.  At most kFewSteps: the few form's rows x steps are bounded by their shared memory.
  const int experts = __popc(lead[0]) + __popc(lead[1]);
  int steps = 0;
  for (int l0 = 0; l0 < experts; l0 += kWarp) {
    const int l = l0 + lane, kb0 = l < experts ? (warp - expert[l]) & (kWarps - 1) : S;
    const int count = kb0 < S ? (S - kb0 + kWarps - 1) / kWarps : 0;
    int upto = count;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    for (int i = 0; i < count; ++i) list[warp][steps + upto - count + i] = (unsigned short)(l | (kb0 + i * kWarps) << 6);
    steps += __shfl_sync(0xffffffffu, upto, kWarp - 1);
  }
  __syncwarp();
  const LanePlace<G> at(blockIdx.x * kTile, a.K, lane);
  int ahead = 0;
  IntWeights<G, 1> w[AHEAD];
  auto load = [&](IntWeights<G, 1>& to) {
    if (ahead < steps) {
      const int l = list[warp][ahead] & 63, kb = list[warp][ahead] >> 6;
      const unsigned char* q = a.mat[0].q + (size_t)expert[l] * a.N * (a.K / 2) + at.q + kb * (kStep / 2);
      const __nv_bfloat16* sc = a.mat[0].s + (size_t)expert[l] * a.N * ((a.K + G - 1) / G) + at.s + kb * (kStep / G);
      to.load(&q, &sc, at.q8, at.s8, kb * kStep + at.k, kb * kStep, a.K);
    }
    ++ahead;
  };
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) load(w[d]);
  float* scales = reinterpret_cast<float*>(acts + (size_t)rows * blocks * kPlanes);
  if (a.K % kStep != 0) {  // the padding of a row's last step
    const int inside = a.K / 16, pad = blocks - inside;
    for (int i = threadIdx.x; i < rows * pad; i += kWarps * 32) {
      const int to = i / pad * blocks + inside + i % pad;
      scales[to] = 0.f;
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) acts[to * kPlanes + p] = make_uint4(0, 0, 0, 0);
    }
  }
  wait_dependency();  // `a` is read from here on; the weights above are nobody's output
  // copies alone, so that no thread waits for one before it starts the next
  for (int r = 0; r < rows; ++r) {
    const uint4* from = reinterpret_cast<const uint4*>(a.bytes) + (size_t)r * (a.K / 16) * kPlanes;
    for (int i = threadIdx.x; i < a.K / 16 * kPlanes; i += kWarps * 32)
      ptx::cp_async_16(ptx::smem_u32(acts + r * blocks * kPlanes + i), from + i, 16);
    const float* from_scale = a.scales + (size_t)r * (a.K / 16);
    for (int i = threadIdx.x; i < a.K / 16; i += kWarps * 32) ptx::cp_async_4(ptx::smem_u32(scales + r * blocks + i), from_scale + i);
  }
  ptx::cp_async_commit();
  ptx::cp_async_wait<0>();
  __syncthreads();
  float acc[2][ROWS] = {};
  for (int i0 = 0; i0 < steps; i0 += AHEAD) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (i0 + d >= steps) break;
      const int l = list[warp][i0 + d] & 63, block = (list[warp][i0 + d] >> 6) * 8 + at.k / 16;
#pragma unroll
      for (int t = 0; t < ROWS; ++t) {
        const int r = row[l][t];
        if (ROWS > 1 && r < 0) continue;
        const uint32_t* words[2] = {w[d].w[0][0], w[d].w[0][1]};
        const __nv_bfloat16* groups[2] = {w[d].s[0][0], w[d].s[0][1]};
        float sum[2];
        int_dots<G, 2>(reinterpret_cast<const unsigned char*>(acts) + (r * blocks + block) * (16 * kPlanes), scales + r * blocks + block,
                       at.k, words, groups, sum);
#pragma unroll
        for (int o = 0; o < 2; ++o) acc[o][t] = fmaf(sum[o], weight[l][t], acc[o][t]);
      }
      load(w[d]);
    }
  }
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
      float v = acc[o][t];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      if (lane % 4 == 0) red[warp][lane / 4 + o * 8][t] = v;
    }
  __syncthreads();
  if (threadIdx.x < kTile * ROWS) {
    const int o = threadIdx.x % kTile, t = threadIdx.x / kTile;
    if (t < a.T) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) v += red[q][o][t];
      static_cast<T*>(a.y)[(size_t)t * a.N + blockIdx.x * kTile + o] = from_f<T>(v);
    }
  }
}

// ------------------------------------------------------------------------------------ many rows

// The second nibble of a byte comes times 16 (16 (n - 8) is exact as well): the activations it meets, inputs 1, 3, 5, 7 of
// eight, are stored times 1/16.  f16 reaches from 2^15 down to steps of 2^-24: what is lost of an activation is below 2^-34
// of the largest of the row's 128.
//
// What the products work through: units of an expert and up to `pass` of its rows, and the rows by expert.
struct ManyPlan {
  int units, pad[3];
  int unit[1];  // units x (expert, first place in the rows' list, rows), then the list
};
__host__ __device__ __forceinline__ int most_units(int rows, int E, int pass) {  // an expert's last unit may be short
  return (rows < E ? rows : E) + rows / pass;
}

// One block makes the plan.  An expert's rows stay in their order: the place of a row decides whether it comes into a unit of
// one or of two tiles of rows, which add a group in different orders (many_step), so that it has to follow from topk_idx alone.
// Each warp counts, and then places, a stretch of the rows; it places 32 at a time by the lanes that name the same expert.
__device__ __forceinline__ void make_plan(const int* __restrict__ topk_idx, int rows, int E, int pass, ManyPlan* plan) {
  constexpr int ONCE = 4;  // turns of 32 rows whose loads are under way together
  __shared__ int start[1024];  // rows of an expert, then the place of its first
  // a warp's rows of an expert, then its next one's place among the expert's: 16 bits each, two to a word
  __shared__ uint32_t own_words[kWarps][512];
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  unsigned short* own = reinterpret_cast<unsigned short*>(own_words[warp]);
  const int stretch = (rows + kWarps * kWarp - 1) / (kWarps * kWarp) * kWarp, first = warp * stretch, last = min(first + stretch, rows);
  auto each_turn = [&](auto use) {  // use(row, its expert; below zero: none, those are flagged by the combine)
    for (int r0 = first; r0 < last; r0 += ONCE * kWarp) {
      int id[ONCE];
#pragma unroll
      for (int i = 0; i < ONCE; ++i) {
        const int r = r0 + i * kWarp + lane;
        id[i] = r < last ? __ldg(topk_idx + r) : -1;
      }
#pragma unroll
      for (int i = 0; i < ONCE; ++i)
        if (r0 + i * kWarp < last) use(r0 + i * kWarp + lane, (unsigned)id[i] < (unsigned)E ? id[i] : -1);
    }
  };
  for (int i = lane; i < (E + 1) / 2; i += kWarp) own_words[warp][i] = 0;
  __syncwarp();
  each_turn([&](int, int e) {
    if (e >= 0) atomicAdd(&own_words[warp][e / 2], 1u << (16 * (e & 1)));
  });
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kWarps * kWarp) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      unsigned short* of = reinterpret_cast<unsigned short*>(own_words[w]) + e;
      const int c = *of;
      *of = (unsigned short)before;
      before += c;
    }
    start[e] = before;
  }
  __syncthreads();
  if (warp == 0) {  // rows and units before each expert
    int before = 0, units = 0;
    for (int e0 = 0; e0 < E; e0 += kWarp) {
      const int e = e0 + lane, c = e < E ? start[e] : 0, u = (c + pass - 1) / pass;
      int cs = c, us = u;
#pragma unroll
      for (int o = 1; o < kWarp; o <<= 1) {
        const int cv = __shfl_up_sync(0xffffffffu, cs, o), uv = __shfl_up_sync(0xffffffffu, us, o);
        if (lane >= o) { cs += cv; us += uv; }
      }
      if (e < E) {
        start[e] = before + cs - c;
        for (int i = 0; i < u; ++i) {
          int* to = plan->unit + 3 * (units + us - u + i);
          to[0] = e;
          to[1] = before + cs - c + i * pass;
          to[2] = min(c - i * pass, pass);
        }
      }
      before += __shfl_sync(0xffffffffu, cs, kWarp - 1);
      units += __shfl_sync(0xffffffffu, us, kWarp - 1);
    }
    if (lane == 0) plan->units = units;
  }
  __syncthreads();
  int* list = plan->unit + 3 * most_units(rows, E, pass);
  each_turn([&](int r, int e) {
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & ((1u << lane) - 1u)), at = e >= 0 ? own[e] : 0;
    __syncwarp();
    if (e >= 0 && before == 0) own[e] = (unsigned short)(at + __popc(same));
    __syncwarp();
    if (e >= 0) list[start[e] + at + before] = r;
  });
}

// P planes of eight inputs each, in a word's order (0,4) (1,5) (2,6) (3,7).
struct HalfRows {
  uint4* plane;  // [rows][K / 8][P]
  float* scale;  // [rows][steps]
};
template <typename X> constexpr int kHalfPlanes = sizeof(X) == 4 ? 2 : 1;

__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 lo = *reinterpret_cast<const float4*>(p), hi = *(reinterpret_cast<const float4*>(p) + 1);
  f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w; f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  unpack(*reinterpret_cast<const uint4*>(p), f, __nv_bfloat16());
}
__device__ __forceinline__ void load8(const E4M3* p, float* f) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((i < 2 ? u.x : u.y) >> (16 * (i & 1))), __NV_E4M3)));
    f[2 * i] = v.x; f[2 * i + 1] = v.y;
  }
}

// Rows [rows, K] of x or `a` to P planes: 16 threads a row's step.  plan: block 0 makes it.
template <typename X, int P>
__global__ void __launch_bounds__(256) w4_planes_kernel(const X* x, const float* __restrict__ x_scale, int rows, int K, HalfRows out,
                                                        const int* __restrict__ topk_idx, int slots, int E, ManyPlan* plan) {
  launch_dependents();
  wait_dependency();
  if (plan != nullptr && blockIdx.x == 0) {
    make_plan(topk_idx, slots, E, kPass<P>, plan);
    return;
  }
  const int S = (K + kStep - 1) / kStep, block = blockIdx.x - (plan != nullptr ? 1 : 0);
  const long long place = (long long)block * 16 + threadIdx.x / 16;
  const int row = (int)(place / S), s = (int)(place % S), c = threadIdx.x % 16, k = s * kStep + c * 8;
  const bool in = row < rows && k < K;
  float v[8] = {}, scale = 0.f, inverse = 0.f;
  if (in) load8(x + (size_t)row * K + k, v);
  if constexpr (sizeof(X) == 1) {
    scale = in ? __ldg(x_scale + (size_t)row * S + s) * 0x1p-6f : 0.f;
    inverse = 0x1p6f;  // the largest is 448
  } else {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    // a power of two that brings the largest to 2^14 or more and below 2^15
    if (most >= 0x7f800000u) {
      scale = __uint_as_float(0x7fc00000u);
    } else if (__uint_as_float(most) >= 0x1p-90f) {
      const int e = (int)(most >> 23) - 127 - 14;
      scale = __uint_as_float((uint32_t)(127 + e) << 23);
      inverse = __uint_as_float((uint32_t)(127 - e) << 23);
    }
  }
  uint4 w[P];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // inputs i and i + 4
    const float at = i % 2 == 0 ? 1.f : 0.0625f;
    float lo = inverse == 0.f ? 0.f : v[i] * (inverse * at), hi = inverse == 0.f ? 0.f : v[i + 4] * (inverse * at);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const __half2 two = __floats2half2_rn(lo, hi);
      const float2 d = __half22float2(two);
      lo -= d.x;
      hi -= d.y;
      (&w[p].x)[i] = *reinterpret_cast<const uint32_t*>(&two);
    }
  }
  if (!in) return;
#pragma unroll
  for (int p = 0; p < P; ++p) out.plane[((size_t)row * K + k) / 8 * P + p] = w[p];
  if (c == 0) out.scale[(size_t)row * S + s] = scale;
}

struct ManyArgs {
  HalfRows x;
  const ManyPlan* plan;
  int rows, k, E, K, N;  // row r of topk_idx reads x's row r / k (gate/up) or r (down: k = 1)
  W4Mat mat[2];
  float* out;            // [rows, N]: a, or the outputs of the rows
};

// Shared memory of one stage: a turn's activations, [step][row tile][word][plane][lane], and their scales, [step][row].
template <int P> constexpr int kPlaneBytes = kTurn * (kPass<P> / 8) * 4 * P * 32 * 16;
template <int P> constexpr int kStageBytes = kPlaneBytes<P> + kTurn * kPass<P> * 4;

// The A operands of a word's two products, w0 of output g, w1 of output g + 8: n - 8 of the nibbles i and i + 4 as two f16
// (1024 + n has n as its last mantissa bits), and 16 (n - 8) of the next two.
__device__ __forceinline__ void unpack_word(uint32_t w0, uint32_t w1, uint32_t f[2][4]) {
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t n = (((i % 2 == 0 ? w0 : w1) >> (8 * half)) & (i < 2 ? 0x000f000fu : 0x00f000f0u)) | 0x64006400u;
      const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&n), __float2half2_rn(i < 2 ? 1032.f : 1152.f));
      f[half][i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

// A step of a warp: the weights w, once they are used `load` fetches the next into their place.  TILES tiles of 8 rows; one
// tile's sums go in two chains, of even and of odd words, so that a warp has four chains of products under way either way.
template <int P, int G, int TILES, typename LOAD>
__device__ __forceinline__ void many_step(IntWeights<G, 2>& w, const uint4* b, const float* scale, float (*acc)[kPass<P> / 8][4], LOAD load) {
  float2 of[TILES];  // the scales of two rows
#pragma unroll
  for (int u = 0; u < TILES; ++u) of[u] = *reinterpret_cast<const float2*>(scale + u * 8);
#pragma unroll
  for (int i = 0; i < kStep / G; ++i) {
    constexpr int CHAINS = TILES == 2 || G > 32 ? 2 : 1;
    float sum[2][CHAINS][4], low[2][CHAINS][4];  // low: of the second plane
#pragma unroll
    for (int u = 0; u < CHAINS; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[m][u][v] = low[m][u][v] = 0.f;
    float g[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int v = 0; v < 2; ++v) g[m][v] = __bfloat162float(w.s[m][v][i]);
#pragma unroll
    for (int j = i * (G / 32); j < (i + 1) * (G / 32); ++j) {
      uint32_t f[2][2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) unpack_word(w.w[m][0][j], w.w[m][1][j], f[m]);
#pragma unroll
      for (int u = 0; u < TILES; ++u) {
        const int chain = TILES == 2 ? u : j % CHAINS;
        const uint4 x = b[(u * 4 + j) * (P * 32)];
#pragma unroll
        for (int m = 0; m < 2; ++m) mma_f16(sum[m][chain], f[m][0], x.x, x.y);
#pragma unroll
        for (int m = 0; m < 2; ++m) mma_f16(sum[m][chain], f[m][1], x.z, x.w);
        if constexpr (P == 2) {
          const uint4 y = b[((u * 4 + j) * P + 1) * 32];
#pragma unroll
          for (int m = 0; m < 2; ++m) mma_f16(low[m][chain], f[m][0], y.x, y.y);
#pragma unroll
          for (int m = 0; m < 2; ++m) mma_f16(low[m][chain], f[m][1], y.z, y.w);
        }
      }
    }
    if (i == kStep / G - 1) load(w);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int u = 0; u < TILES; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float all = sum[m][u][v];
          if constexpr (P == 2) all += low[m][u][v];
          if constexpr (TILES < CHAINS) all += P == 2 ? sum[m][1][v] + low[m][1][v] : sum[m][1][v];
          acc[m][u][v] = fmaf(all, g[m][v / 2] * (v % 2 == 0 ? of[u].x : of[u].y), acc[m][u][v]);
        }
  }
}

// Blocks take turns at the items of a unit.  A warp has two tiles of 16 outputs, which share their activations: the same
// outputs of W1 and W3, or neighbours of W2.  SPLIT warps share a pair's steps, and add up at the end, so that there are
// more and shorter items: 1 from an item a block on (13 tokens of the Small layer, 1.3 to 1.8 items a block: 77 us, and with 2
// warps 80), 2 from a quarter on (64 tokens, 2 of 8 experts, h f 2048, 0.4 to 0.8: 60, with 1 69, with 4 70), else 4 (13
// fp32 tokens of the long-sequence layer, 0.2 to 0.3: 54, with 2 62, with 1 87).
template <int P, int G, bool GATEUP, int SPLIT>
__device__ __forceinline__ void many_items(const ManyArgs& a, unsigned char* stages, int* list, int* source) {
  constexpr int WIDE = kWarps / SPLIT, OUTS = WIDE * kTile * (GATEUP ? 1 : 2), GROUPS = kStep / G;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, tile = warp % WIDE, part = warp / WIDE;
  const int S = (a.K + kStep - 1) / kStep, turns = (S + kTurn - 1) / kTurn, groups = (a.K + G - 1) / G;
  const int across = (a.N + OUTS - 1) / OUTS, items = a.plan->units * across;
  const int* rows_by_expert = a.plan->unit + 3 * most_units(a.rows, a.E, kPass<P>);
  // an item's expert, number of rows and, in thread i, its i-th row: read an item ahead
  int e = 0, n = 0, r = 0;
  auto look = [&](int item) {
    if (item >= items) return;
    const int* unit = a.plan->unit + 3 * (item / across);
    e = unit[0];
    n = unit[2];
    r = threadIdx.x < n ? rows_by_expert[unit[1] + threadIdx.x] : 0;
  };
  look(blockIdx.x);
  const LanePlace<G> lanes(0, a.K, lane);  // strides, and this lane's place in the first tile
  // this thread's pieces of a turn's activations: the same eight inputs of rows APART apart
  constexpr int ROWS = kPass<P>, APART = kWarps * 2 / kTurn, FILLS = ROWS / APART;
  static_assert(FILLS * APART == ROWS && 8 % APART == 0, "the threads divide a turn evenly");
  static_assert(kTurn * ROWS <= kWarps * 32, "a thread copies one scale at most");
  const int c = threadIdx.x % (16 * kTurn), r0 = threadIdx.x / (16 * kTurn);
  int word, quarter;
  place_of<G>(c % 16, &word, &quarter);
  const uint32_t stage0 = ptx::smem_u32(stages), piece = ((c / 16 * (ROWS / 2) + word) * (P * 32) + r0 * 4 + quarter) * 16;
  const int c0 = (lane % 4) * 2;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    __syncthreads();  // the last item's list and sums have been read
    if (threadIdx.x < n) {
      list[threadIdx.x] = r;
      source[threadIdx.x] = r / a.k;
    }
    const int out0 = item % across * OUTS + tile * kTile * (GATEUP ? 1 : 2), rows = n;
    const bool live = out0 < a.N;  // N is a multiple of 32
    const size_t row0 = (size_t)e * a.N + (live ? out0 : 0);
    const unsigned char* q[2];
    const __nv_bfloat16* sc[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const size_t at = row0 + (GATEUP ? 0 : m * kTile);
      q[m] = a.mat[GATEUP ? m : 0].q + at * (a.K / 2) + lanes.q + part * (kStep / 2);
      sc[m] = a.mat[GATEUP ? m : 0].s + at * groups + lanes.s + part * GROUPS;
    }
    IntWeights<G, 2> w[2];
    int k0 = part * kStep;  // of the weights to load next
    auto load = [&](IntWeights<G, 2>& to) {
      if (k0 < a.K) to.load(q, sc, lanes.q8, lanes.s8, k0 + lanes.k, k0, a.K);
      k0 += SPLIT * kStep;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        q[m] += SPLIT * (kStep / 2);
        sc[m] += SPLIT * GROUPS;
      }
    };
    load(w[0]);
    load(w[1]);
    __syncthreads();
    look(item + gridDim.x);
    int from[FILLS];  // rows of x; below zero where there is none
#pragma unroll
    for (int i = 0; i < FILLS; ++i) from[i] = r0 + i * APART < rows ? source[r0 + i * APART] : -1;
    const int scale_step = threadIdx.x / ROWS;
    const int scale_from = scale_step < kTurn && threadIdx.x % ROWS < rows ? source[threadIdx.x % ROWS] : -1;
    auto fill = [&](int turn) {
      const uint32_t to = stage0 + turn % kStages * kStageBytes<P>;
#pragma unroll
      for (int i = 0; i < FILLS; ++i) {
        if (i * APART >= 8 && rows <= 8) break;  // a tile that no product reads
        const bool in = from[i] >= 0 && turn * kTurn * kStep + c * 8 < a.K;
        const uint4* x = a.x.plane + (in ? ((size_t)from[i] * (a.K / 8) + turn * (kTurn * 16) + c) * P : 0);
#pragma unroll
        for (int p = 0; p < P; ++p) ptx::cp_async_16(to + piece + (i * APART / 8 * 4 * P + p) * 512 + i * APART % 8 * 64, x + p, in ? 16u : 0u);
      }
      if (scale_step < kTurn) {
        const bool in = scale_from >= 0 && turn * kTurn + scale_step < S;
        ptx::cp_async_4(to + kPlaneBytes<P> + threadIdx.x * 4, a.x.scale + (in ? (size_t)scale_from * S + turn * kTurn + scale_step : 0),
                        in ? 4u : 0u);
      }
    };
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) {
      if (t < turns) fill(t);
      ptx::cp_async_commit();
    }
    float acc[2][ROWS / 8][4] = {};  // [tile of outputs][tile of rows]
    const int own = turns * kTurn / SPLIT;  // of a warp's steps, those beyond the inputs included
    int turn = 0;
    for (int o0 = 0; o0 < own; o0 += 2) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (o0 + d >= own) break;
        if ((o0 + d) * SPLIT % kTurn == 0) {
          ptx::cp_async_wait<kStages - 2>();
          __syncthreads();  // the turn's activations are there, and the stage before it has been read by all
          if (turn + kStages - 1 < turns) fill(turn + kStages - 1);
          ptx::cp_async_commit();
          ++turn;
        }
        const int s = (o0 + d) * SPLIT + part;
        if (s >= S) continue;
        const unsigned char* stage = stages + (turn - 1) % kStages * kStageBytes<P>;
        const uint4* b = reinterpret_cast<const uint4*>(stage) + s % kTurn * (ROWS / 2 * P * 32) + lane;
        const float* scale = reinterpret_cast<const float*>(stage + kPlaneBytes<P>) + s % kTurn * ROWS + c0;
        if (ROWS > 8 && rows > 8) many_step<P, G, ROWS / 8>(w[d], b, scale, acc, load);
        else many_step<P, G, 1>(w[d], b, scale, acc, load);
      }
    }
    ptx::cp_async_wait<0>();
    if constexpr (SPLIT > 1) {  // the parts' sums meet through shared memory: [value][warp][lane]
      constexpr int TILES = ROWS / 8;
      float* sums = reinterpret_cast<float*>(stages) + threadIdx.x;
      __syncthreads();
      if (part > 0) {
#pragma unroll
        for (int v = 0; v < TILES * 8; ++v) sums[v * kWarps * 32] = acc[v % 2][v / 2 % TILES][v / (2 * TILES)];
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int v = 0; v < TILES * 8; ++v)
#pragma unroll
          for (int i = 1; i < SPLIT; ++i) acc[v % 2][v / 2 % TILES][v / (2 * TILES)] += sums[(v * kWarps + i * WIDE) * 32];
      }
    }
    if (part == 0 && live) {
#pragma unroll
      for (int u = 0; u < ROWS / 8; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = u * 8 + c0 + v % 2, o = out0 + lane / 4 + v / 2 * 8;
          if (i >= rows) continue;
          float* to = a.out + (size_t)list[i] * a.N + o;
          if constexpr (GATEUP) {
            to[0] = acc[0][u][v] * sigmoidf_(acc[0][u][v]) * acc[1][u][v];
          } else {
            to[0] = acc[0][u][v];
            to[kTile] = acc[1][u][v];
          }
        }
    }
  }
}

template <int P, int G, bool GATEUP>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_many_kernel(const __grid_constant__ ManyArgs a) {
  extern __shared__ __align__(16) unsigned char stages[];
  __shared__ int list[kPass<P>], source[kPass<P>];
  launch_dependents();
  wait_dependency();
  constexpr int OUTS = kWarps * kTile * (GATEUP ? 1 : 2);
  const int items = a.plan->units * ((a.N + OUTS - 1) / OUTS), blocks = gridDim.x;
  const int split = items >= blocks ? 1 : 4 * items >= blocks ? 2 : 4;
  if (split == 1) many_items<P, G, GATEUP, 1>(a, stages, list, source);
  else if (split == 2) many_items<P, G, GATEUP, 2>(a, stages, list, source);
  else many_items<P, G, GATEUP, 4>(a, stages, list, source);
}

// y[t] = sum_j topk_w[t,j] * rows[t*k+j], j ascending; a row of no expert counts as zeros.  The choices do not wait for the
// products, and eight rows are under way at once (one after another they took 8 us for 64 tokens of the Medium layer).
template <typename T>
__global__ void __launch_bounds__(256) w4_combine_kernel(const float* rows, const int* __restrict__ topk_idx,
                                                         const float* __restrict__ topk_w, int k, int E, int h,
                                                         T* __restrict__ y, int* status) {
  constexpr int ONCE = 8;
  const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  const size_t r0 = (size_t)t * k;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < k; j0 += ONCE) {
    bool in[ONCE];
    float w[ONCE];
#pragma unroll
    for (int j = 0; j < ONCE; ++j) {
      in[j] = j0 + j < k && (unsigned)__ldg(topk_idx + r0 + j0 + j) < (unsigned)E;
      w[j] = j0 + j < k ? __ldg(topk_w + r0 + j0 + j) : 0.f;
      if (j0 + j < k && !in[j] && c == 0) flag_status(status, MOE_STATUS_BAD_INDEX);
    }
    if (j0 == 0) wait_dependency();
    if (c >= h) continue;
    float4 v[ONCE];
#pragma unroll
    for (int j = 0; j < ONCE; ++j)
      v[j] = in[j] ? *reinterpret_cast<const float4*>(rows + (r0 + j0 + j) * h + c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < ONCE; ++j) {
      if (!in[j]) continue;
      s.x = fmaf(w[j], v[j].x, s.x); s.y = fmaf(w[j], v[j].y, s.y); s.z = fmaf(w[j], v[j].z, s.z); s.w = fmaf(w[j], v[j].w, s.w);
    }
  }
  if (c < h) store4(y + (size_t)t * h + c, s);
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
    const float s = sc[n];
    auto code = [&](float w) {
      const float z = s == 0.f ? 0.f : rintf(w / s);
      return isnan(z) ? 8 : (int)fminf(fmaxf(z, -8.f), 7.f) + 8;
    };
    const int lo = code(tile[2 * b][n]), hi = code(tile[2 * b + 1][n]);
    q[(e * N + n0 + n) * (size_t)(K / 2) + k0 / 2 + b] = (unsigned char)(lo | (hi << 4));
  }
}

// A launch that may begin while the one before it on the stream still runs (the kernel waits for it by itself).
template <typename A>
void launch_early(void (*kernel)(A), dim3 grid, int threads, size_t bytes, cudaStream_t st, const A& args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, args);
  count_launch(st);
}

// Shared memory of `rows` rows of K activations in the few form.
size_t few_bytes(int rows, int K) {
  return (size_t)rows * ((K + kStep - 1) / kStep) * 8 * (16 * kPlanes + sizeof(float));
}

template <typename K>
void allow_shared(K kernel, int bytes, bool* ready) {  // per device: the attribute is set once
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
}

template <typename X, typename T, int G, int ROWS>
void few(const W4Ffn& p, cudaStream_t st) {
  unsigned char* bytes = static_cast<unsigned char*>(p.a);
  float* scales = reinterpret_cast<float*>(bytes + (size_t)p.T * p.k * p.f * kPlanes);
  const FewArgs up{p.x, p.x_scale, p.topk_idx, p.topk_w, p.T, p.k, p.E, p.h, p.f,
                   {{static_cast<const unsigned char*>(p.W1q), static_cast<const __nv_bfloat16*>(p.W1s)},
                    {static_cast<const unsigned char*>(p.W3q), static_cast<const __nv_bfloat16*>(p.W3s)}}, bytes, scales, nullptr, p.status};
  static bool ready[3][64] = {};
  allow_shared(w4_few_up_kernel<X, G, ROWS>, kFewBytes<ROWS>, ready[0]);
  w4_few_up_kernel<X, G, ROWS><<<dim3(p.f / (2 * kTile), p.T * p.k), kWarps * 32, few_bytes(p.T, p.h), st>>>(up);
  count_launch(st);
  const FewArgs down{nullptr, nullptr, p.topk_idx, p.topk_w, p.T, p.k, p.E, p.f, p.h,
                     {{static_cast<const unsigned char*>(p.W2q), static_cast<const __nv_bfloat16*>(p.W2s)}, {}}, bytes, scales, p.y, p.status};
  // One token's second kernel has 80 registers with three blocks an SM, and up to 120 with two.  A grid of more than two an SM
  // takes three rather than a second round (Large layer: 52 us for both kernels, with two 56; Medium: 30.5 and 32.3).  A smaller
  // one runs at once either way, and keeps more of its loads under way with two (Small layer: 13.9 us, with three 14.4; in
  // groups of 32, where three spill, 23.6 and 25.6; h 4096, f 1408, 6 experts: 21.7 and 24.0).
  const size_t shared = few_bytes(p.T * p.k, p.f);
  const int blocks = p.h / kTile;
  if (ROWS == 1 && blocks > 2 * num_sms()) {
    allow_shared(w4_few_down_kernel<T, G, ROWS, ROWS == 1 ? 3 : 2>, kFewBytes<ROWS>, ready[2]);
    launch_early(w4_few_down_kernel<T, G, ROWS, ROWS == 1 ? 3 : 2>, dim3(blocks), kWarps * 32, shared, st, down);
  } else {
    allow_shared(w4_few_down_kernel<T, G, ROWS, 2>, kFewBytes<ROWS>, ready[1]);
    launch_early(w4_few_down_kernel<T, G, ROWS, 2>, dim3(blocks), kWarps * 32, shared, st, down);
  }
}

template <typename T>
void combine(const W4Ffn& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.T, (p.h / 4 + 255) / 256);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, w4_combine_kernel<T>, (const float*)p.rows, p.topk_idx, p.topk_w, p.k, p.E, p.h, static_cast<T*>(p.y), p.status);
  count_launch(st);
}

// Planes and scales of [rows, K] at `to`.
template <int P>
HalfRows half_rows(void* to, size_t rows, int K) {
  unsigned char* b = static_cast<unsigned char*>(to);
  return {reinterpret_cast<uint4*>(b), reinterpret_cast<float*>(b + rows * K * 2 * P)};
}

template <typename X, int P>
void to_planes(const X* x, const float* x_scale, int rows, int K, const HalfRows& out, const W4Ffn& p, ManyPlan* plan, cudaStream_t st) {
  const long long steps = (long long)rows * ((K + kStep - 1) / kStep);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((steps + 15) / 16 + (plan != nullptr ? 1 : 0)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = plan != nullptr ? 0 : 1;  // the first launch follows whatever wrote x
  cudaLaunchKernelEx(&cfg, w4_planes_kernel<X, P>, x, x_scale, rows, K, out, p.topk_idx, p.T * p.k, p.E, plan);
  count_launch(st);
}

template <int P, int G, bool GATEUP>
void many_product(const ManyArgs& a, cudaStream_t st) {
  constexpr int stages = kStages * kStageBytes<P>, sums = kWarps * 16 * 32 * 4, bytes = stages > sums ? stages : sums;
  static bool ready[64] = {};
  allow_shared(w4_many_kernel<P, G, GATEUP>, bytes, ready);
  const long long items = (long long)most_units(a.rows, a.E, kPass<P>) * (a.N / kTile), blocks = 2ll * num_sms();
  launch_early(w4_many_kernel<P, G, GATEUP>, dim3((unsigned)(items < blocks ? items : blocks)), kWarps * 32, bytes, st, a);
}

template <typename X, typename T, int G>
void many(const W4Ffn& p, cudaStream_t st) {
  constexpr int P = kHalfPlanes<T>;
  const int rows = p.T * p.k;
  ManyPlan* plan = static_cast<ManyPlan*>(p.plan);
  const HalfRows x = half_rows<P>(p.x_planes, p.T, p.h), act = half_rows<P>(p.a_planes, rows, p.f);
  float* a = static_cast<float*>(p.a);
  to_planes<X, P>(static_cast<const X*>(p.x), p.x_scale, p.T, p.h, x, p, plan, st);
  const ManyArgs up{x, plan, rows, p.k, p.E, p.h, p.f,
                    {{static_cast<const unsigned char*>(p.W1q), static_cast<const __nv_bfloat16*>(p.W1s)},
                     {static_cast<const unsigned char*>(p.W3q), static_cast<const __nv_bfloat16*>(p.W3s)}}, a};
  many_product<P, G, true>(up, st);
  to_planes<float, P>(a, nullptr, rows, p.f, act, p, nullptr, st);
  const ManyArgs down{act, plan, rows, 1, p.E, p.f, p.h,
                      {{static_cast<const unsigned char*>(p.W2q), static_cast<const __nv_bfloat16*>(p.W2s)}, {}}, p.rows};
  many_product<P, G, false>(down, st);
  combine<T>(p, st);
}

template <typename X, typename T, int G>
void run_group(const W4Ffn& p, cudaStream_t st) {
  // Several tokens: the few form's second kernel does its rows one after another (8 rows of 2 tokens, h 1024, f 512: 12 us and
  // in the many form 17; 10 rows of the Small layer 33 and 35, 12 38 and 37; in fp32 12 rows 38 and 39; 18 rows, h 832, f 1408, 46
  // and 36).
  const size_t most = p.T == 1 ? kFewBytes<1> : kFewBytes<kFewTokens>;
  const bool is_few = p.T <= kFewTokens && p.T * p.k <= (p.T == 1 ? kFewRows : kSeveralRows) && few_bytes(p.T, p.h) <= most &&
                      few_bytes(p.T * p.k, p.f) <= most;
  if (!is_few) many<X, T, G>(p, st);
  else if (p.T == 1) few<X, T, G, 1>(p, st);
  else few<X, T, G, kFewTokens>(p, st);
}

template <typename X, typename T>
void run(const W4Ffn& p, cudaStream_t st) {
  if (p.group == 128) run_group<X, T, 128>(p, st);
  else if (p.group == 64) run_group<X, T, 64>(p, st);
  else run_group<X, T, 32>(p, st);
}

}  // namespace

size_t w4_scratch(int dtype, long long T, long long k, int h, int E, int f, W4Scratch* at) {
  auto round = [](size_t b) { return (b + 255) & ~size_t(255); };
  W4Scratch s;
  const size_t P = dtype == MOE_BF16 ? 1 : 2;
  auto planes = [=](size_t rows, int K) { return round(rows * K * 2 * P + rows * ((K + kStep - 1) / kStep) * sizeof(float)); };
  s.a = 0;
  s.rows = s.a + round((size_t)T * k * f * sizeof(float));
  s.x_planes = s.rows + round((size_t)T * k * h * sizeof(float));
  s.a_planes = s.x_planes + planes(T, h);
  s.plan = s.a_planes + planes(T * k, f);
  if (at != nullptr) *at = s;
  return s.plan + round(16 + sizeof(int) * (3 * (size_t)most_units((int)(T * k), E, P == 1 ? kPass<1> : kPass<2>) + T * k));
}

void launch_expert_ffn_w4(int dtype, const W4Ffn& p, cudaStream_t st) {
  if (dtype == MOE_F32) run<float, float>(p, st);
  else if (p.x_scale != nullptr) run<E4M3, __nv_bfloat16>(p, st);
  else run<__nv_bfloat16, __nv_bfloat16>(p, st);
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
