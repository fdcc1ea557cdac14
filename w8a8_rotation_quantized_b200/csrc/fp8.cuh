// 8-bit floating-point linear layer with one scale per block of 128: e4m3 codes,
// fp32 scales, activations in blocks of 1 x 128 (a token's 128 consecutive
// elements), weights in blocks of 128 x 128.
//
//   quantize   a = max |x| over the block; s = 0 where a = 0, else
//              max(RN(a / 448), 2^-126); q = e4m3_rne(RN(x * RN(1 / s))) (0 where
//              s = 0). The bound 2^-126 keeps 1 / s finite.
//   product    part_b = sum over the K block b of xq wq (tensor cores, fp32),
//              acc = sum_b part_b * RN(sx[b][m] * sw[n / 128][b]), fused
//              multiply-adds in fp32, b ascending (where the K axis is split over
//              CTAs: within each part, then the parts' sums in order); v = acc + bias;
//              y = bf16(v), bf16(silu(v_gate) v_up), or the latter quantized
//              again (1 x 128) straight from fp32.
//
// Layouts: xq [M, K], wq [N, K] row-major bytes; sx [ceil(K / 128), M] (the
// product's threads hold one row each, so a K block's scales of consecutive rows
// are one coalesced load); sw [ceil(N / 128), ceil(K / 128)].
//
// A NaN makes its block's scale and codes NaN, an infinity makes the scale
// infinite and its own code NaN, so the outputs that depend on either are NaN.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "gemm_sm100.cuh"
#include "nvfp4.cuh"
#include "ptx_sm100.cuh"

namespace h3q {

// max that returns NaN if either operand is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two e4m3 codes (round to nearest even, saturating): lo in bits 0-7, hi in bits 8-15.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  return f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(c, d) << 16);
}

// Scale of a block whose largest magnitude is a, and the factor that turns
// elements into code values.
__device__ __forceinline__ float fp8_scale(float a, float& inv) {
  const float s = a == 0.0f ? 0.0f : max_nan(__fdiv_rn(a, 448.0f), 0x1p-126f);
  inv = a == 0.0f ? 0.0f : __frcp_rn(s);
  return s;
}

// ---------------------------------------------------------------- quantize
// Eight consecutive elements as fp32.
__device__ __forceinline__ void fp8_load8(const __nv_bfloat16* p, float (&v)[8]) { load_bf16x8(p, v); }

__device__ __forceinline__ void fp8_load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ float fp8_absmax8(const float (&v)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
  return a;
}

__device__ __forceinline__ uint2 fp8_codes8(const float (&v)[8], float inv) {
  float2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(inv, inv));
  return make_uint2(f32x4_to_e4m3x4(t[0].x, t[0].y, t[1].x, t[1].y), f32x4_to_e4m3x4(t[2].x, t[2].y, t[3].x, t[3].y));
}

// Eight consecutive elements as loaded; the bits of the largest magnitude among them (of
// a bf16 pair's two halves, compared side by side), which max_bits combines and top turns
// into the magnitude; and their codes. A NaN wins.
template <typename T>
struct Fp8Chunk;

template <>
struct Fp8Chunk<__nv_bfloat16> {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float top(uint32_t bits) {
    return max_nan(__uint_as_float(bits << 16), __uint_as_float(bits & 0xFFFF0000u));
  }
  __device__ __forceinline__ uint32_t absmax() const {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max_bits(m, w[i] & 0x7FFF7FFFu);
    return m;
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return fp8_codes8(v, inv);
  }
};

template <>
struct Fp8Chunk<float> {
  float v[8] = {};
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float top(uint32_t bits) { return __uint_as_float(bits); }
  __device__ __forceinline__ uint32_t absmax() const { return __float_as_uint(fp8_absmax8(v)); }
  __device__ __forceinline__ uint2 codes(float inv) const { return fp8_codes8(v, inv); }
};

// 1 x 128 blocks. A CTA takes 32 rows x 256 columns, a warp four of the rows: sixteen
// lanes a block, eight elements each, all four loads in flight at once. The four rows'
// maxima are combined together, each exchange halving the rows a lane still carries, so
// that every lane ends with one of its block's four scales and divides once (five
// exchanges for four rows; with four each, and four divisions, the kernel was issue
// bound). The scales of the 32 rows leave together, a line for each of the two K blocks.
constexpr int kF8QuantRows = 32;

template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const T* __restrict__ x, int64_t M, int K, int KB,
                                                           uint8_t* __restrict__ codes, float* __restrict__ sx) {
  __shared__ float scales[2][kF8QuantRows];
  const int pairs = (KB + 1) >> 1;
  const int rb = blockIdx.x / pairs;
  const int kb = 2 * (blockIdx.x - rb * pairs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = kb * 128 + 8 * lane;
  const int64_t m0 = int64_t(rb) * kF8QuantRows;
  const int64_t first = (m0 + 4 * warp) * K + col;
  const int rows = col < K ? static_cast<int>(min(int64_t(4), M - m0 - 4 * warp)) : 0;  // of this warp, may be negative
  grid_dependents_start();
  grid_dependency_wait();
  Fp8Chunk<T> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < rows) v[i].load(x + first + int64_t(i) * K);
  uint32_t k[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) k[i] = v[i].absmax();
  auto exchange = [](uint32_t keep, uint32_t give, int mask) {
    return Fp8Chunk<T>::max_bits(keep, __shfl_xor_sync(0xFFFFFFFFu, give, mask));
  };
  const bool b3 = lane & 8, b2 = lane & 4;
  const uint32_t k0 = exchange(b3 ? k[2] : k[0], b3 ? k[0] : k[2], 8);  // row 0 or 2
  const uint32_t k1 = exchange(b3 ? k[3] : k[1], b3 ? k[1] : k[3], 8);  // row 1 or 3
  uint32_t top = exchange(b2 ? k1 : k0, b2 ? k0 : k1, 4);
  top = exchange(top, top, 2);
  top = exchange(top, top, 1);
  float inv;
  const float s = fp8_scale(Fp8Chunk<T>::top(top), inv);  // of row (lane >> 2) & 3
  if ((lane & 3) == 0) scales[lane >> 4][4 * warp + ((lane >> 2) & 3)] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float inv_i = __shfl_sync(0xFFFFFFFFu, inv, (lane & 16) | (4 * i));
    if (i < rows) *reinterpret_cast<uint2*>(codes + first + int64_t(i) * K) = v[i].codes(inv_i);
  }
  __syncthreads();
  if (warp < 2 && kb + warp < KB && m0 + lane < M) sx[int64_t(kb + warp) * M + m0 + lane] = scales[warp][lane];
}

// 128 x 128 blocks: one CTA of 256 threads per block; thread t holds the
// 8-element chunks t + 256 n (row (t + 256 n) / 16), n = 0..7.
template <typename T>
__global__ void __launch_bounds__(256) fp8_weight_kernel(const T* __restrict__ w, int64_t N, int K, int KB,
                                                         uint8_t* __restrict__ codes, float* __restrict__ sw) {
  __shared__ float warp_max[8];
  const int64_t nb = blockIdx.x / KB;
  const int kb = static_cast<int>(blockIdx.x - nb * KB);
  const int col = kb * 128 + 8 * (threadIdx.x & 15);
  float v[8][8];
  float a = 0.0f;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int64_t row = nb * 128 + (threadIdx.x >> 4) + 16 * n;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[n][i] = 0.0f;
    if (row < N && col < K) fp8_load8(w + row * K + col, v[n]);
  }
#pragma unroll
  for (int n = 0; n < 8; ++n) a = max_nan(a, fp8_absmax8(v[n]));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max_nan(a, warp_max[i]);
  float inv;
  const float s = fp8_scale(a, inv);
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int64_t row = nb * 128 + (threadIdx.x >> 4) + 16 * n;
    if (row < N && col < K) *reinterpret_cast<uint2*>(codes + row * K + col) = fp8_codes8(v[n], inv);
  }
  if (threadIdx.x == 0) sw[nb * KB + kb] = s;
}

// ---------------------------------------------------------------- product
// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 x e4m3 -> fp32, CTA pair.
__device__ __forceinline__ void mma_fp8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor for kind::f8f6f4: e4m3 A and B (format 0), fp32
// accumulator, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_fp8(uint32_t M, uint32_t N) {
  return (1u << 4)             // D format: f32
         | ((N >> 3) << 17)    // N / 8
         | ((M >> 4) << 24);   // M / 16
}

// tcgen05.wait::ld that the loaded registers depend on, so no use of them can be
// scheduled before it.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// silu(g) = g / (1 + e^-g) from the hardware's 2^x and reciprocal approximations, each
// brought near fp32's own rounding: the product g log2(e) keeps its rounding error, which
// enters as a factor 1 + lo ln 2, and the reciprocal takes one Newton step. What is left is
// the error of 2^x itself (two units of the last place), as in an fp32 evaluation. The
// error of a quantized output, which is that of codes on the other side of a border, halves
// (1.1e-4 to 5e-5 of its norm at 16384 x 5376 -> 14336) for 1% of that call's time. Below
// g = -87.3 the reciprocal leaves the normal range and the result is -0; silu is above
// -2^-119 there.
__device__ __forceinline__ float silu_approx(float g) {
  const float t = fminf(__fmul_rn(g, -1.44269504f), 126.0f);  // 2^t stays finite
  const float lo = __fmaf_rn(g, -1.92596299e-8f, __fmaf_rn(g, -1.44269504f, -t));
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = __fmaf_rn(e, fminf(__fmul_rn(lo, 0.693147181f), 1.0f), e);
  const float d = __fadd_rn(1.0f, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  r = __fmaf_rn(r, __fmaf_rn(-d, r, 1.0f), r);
  return __fmul_rn(g, r);
}

__device__ __forceinline__ uint4 f8_pack8(const float* a) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

// Adds eight bias values to acc[0 .. 7].
__device__ __forceinline__ void f8_bias8(float* acc, const __nv_bfloat16* bias) {
  float b[8];
  fp8_load8(bias, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], b[i]);
}

__device__ __forceinline__ void f8_bias32(float* acc, const __nv_bfloat16* bias) {
#pragma unroll
  for (int g = 0; g < 4; ++g) f8_bias8(acc + 8 * g, bias + 8 * g);
}

// tcgen05.alloc waits, without a limit, for columns that other CTAs of the SM hold, and a CTA
// of a cluster frees its own only with its peers: CTAs of two clusters (of two streams, say)
// that each held columns the other waits for would wait for ever. So every CTA of these
// products asks for at least the share of the SM's shared memory that its columns are of the
// SM's 512: CTAs that fit an SM together have their columns without a wait.
constexpr int kSmShared = 228 * 1024, kSmSharedPerCta = 1024;  // an SM's, and what it keeps for each CTA
__host__ __device__ constexpr int smem_for_tmem(int cols) { return cols * (kSmShared / 512) - kSmSharedPerCta; }

enum Fp8Epi : int { kF8BF16 = 0, kF8SwiGLU = 1, kF8SwiGLUQuant = 2 };

constexpr int64_t kF8MaxTiles = int64_t(1) << 23;  // output tiles of a call (the host refuses more)
constexpr int kF8Stages = 4;
// The two issuers take the K blocks in turn and each keeps its own stages: with an odd ring a
// stage would change hands, and the parity that its next owner waits for holds one round early.
static_assert(kF8Stages % 2 == 0, "a stage belongs to one issuer");
constexpr int kF8Warps = 16;                     // promotion warps
constexpr int kF8Threads = 32 * kF8Warps + 128;  // then operand and scale producers, two MMA issuers
constexpr int kF8Producer = kF8Warps, kF8Issuer = kF8Warps + 2;
constexpr int kF8StageBytes = kAStage + kBStage;
constexpr int kF8ScaleRing = 16;            // K blocks whose scales are in flight or waiting ...
constexpr int kF8ScaleGroup = 8;            // ... handed over in groups
constexpr int kF8ScaleGroups = kF8ScaleRing / kF8ScaleGroup;
constexpr int kF8ScaleSlot = 128 * 4 + 16;  // a K block's scales of the CTA's 128 rows, then of the two weight blocks
constexpr int kF8OutTile = 32 * 64;         // a warp's 32 output rows of 64 bytes
constexpr size_t kF8Smem = size_t(kF8Stages) * kF8StageBytes + kF8Warps * 2 * kF8OutTile + kF8ScaleRing * kF8ScaleSlot +
                           2 * 4 * 128 * 4 /*row maxima*/ + 256 /*barriers*/ + 1024 /*align*/;
static_assert(kF8Smem <= smem_for_tmem(kTmemCols), "shared memory of one CTA");
// Register split: the launch's 96 per thread, moved from the control warps to the
// ones that hold accumulators.
constexpr uint32_t kF8RegsCtl = 32, kF8RegsPromote = 112, kF8RegsLaunch = 96;
static_assert(128 * kF8RegsCtl + 32 * kF8Warps * kF8RegsPromote <= kF8Threads * kF8RegsLaunch, "register split");

struct Fp8Params {
  int M, N;                 // N: output columns (SwiGLU: F)
  int KB;                   // K blocks: ceil(K / 128)
  int num_m, num_n, num_tiles, group_m;
  float inv_per_group, inv_group_m;  // 1 / (group_m num_n), 1 / group_m
  int b_row_up;             // SwiGLU: first up row of the weight (= F)
  int last_nb;              // last row of sw
  const float* sx;          // [KB, M]
  const float* sw;          // [ceil(rows / 128), KB]
  const __nv_bfloat16* bias;  // nullable
  void* out;                // bf16 [M, N], or e4m3 codes
  float* sh;                // SwiGLUQuant: [F / 128, M]
  uint64_t wait_limit_ns;
  uint32_t missing_bytes;   // zero; bytes that every stage waits for in vain (test of the waits)
};

// acc += part * f, 32 columns, two multiply-adds an instruction: the same rate as single
// ones (664 against 712 cycles a K block) at half the issue slots, which the control warps
// need.
__device__ __forceinline__ void f8_promote(float (&acc)[32], const uint32_t (&r)[32], float f) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 t = __ffma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(f, f),
                                make_float2(acc[i], acc[i + 1]));
    acc[i] = t.x;
    acc[i + 1] = t.y;
  }
}

// Large products. CTA pairs, 256 x 256 output tiles, TMA ring and cta_group::2 MMAs as in
// the int8 GEMM. The tensor cores sum one K block of 128 at a time (four MMAs) into one of
// two 256-column buffers of tensor memory; sixteen promotion warps read each block's
// partial sums, multiply them by the block's scales and add them to fp32 accumulators in
// registers (64 columns of one row per thread) while the tensor cores fill the other
// buffer. Roles:
//   warps 0-15   promotion and output;
//   warp 16      operand tiles by TMA (both CTAs), warp 17 the block scales (cp.async, up
//                to sixteen blocks ahead), each a warp of its own, since the promotion
//                warps take the issue slots;
//   warps 18-19  MMA issue (leader CTA), one per buffer, so that each has two K blocks'
//                time for one.
// What bounds it: per SM and K block the MMAs take 512 cycles, reading the 128 KB of
// partial sums 256 and their multiply-adds 256 of the fp32 pipe, in parallel. Measured some
// 710 cycles a K block and 2300 an output tile between blocks (whole calls at zero operands
// and the full clock: 14 tiles of 42 blocks a pair 232 us, 19 of 112 793); the same kernel
// promoting once a tile (other results, for the comparison) takes 520. At random data the
// board's power limit sets in as well: 4096 x 5376 x 16128 takes 232 us at the full
// 1.965 GHz (zero operands), 289 alone with random ones and 340 back to back, at 1.4 GHz;
// 16384 x 14336 x 5376 0.79 ms, 1.07 and 1.24, at 1.2 to 1.3 GHz. A library product with
// one scale for the whole tensor, so without promotion, takes 186, 235 and 278 us in the
// first case, 0.72, 0.89 and 1.03 ms in the second: the promotion's cost, 10% to 25%.
// What counted on the way (16384 x 14336 x 5376, 3.0 ms at first): arrivals at
// the partner CTA without a cluster-scope release (-40%); control roles run by converged
// warps, their descriptors in uniform registers; scales fetched ahead instead of one block
// before (-15%); hardly any register spills (4 bytes in the bf16 form; addresses of shared
// memory as constants); the next block's scales and completion test fetched behind the
// release of this one (-15%). Halves of a block as MMAs of 128 columns ran slower (the A
// tile is read twice for the same work), and so did promotion by eight warps of 128
// columns each.
template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8Threads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmOut, const Fp8Params p) {
  constexpr bool kSwi = EPI != kF8BF16;
  // aligned by declaration, so that every address in it is a constant: the promotion
  // warps have no registers for pointers
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sA = smem;
  uint8_t* sB = smem + kF8Stages * kAStage;
  uint8_t* out_tiles = sB + kF8Stages * kBStage;        // [warp][2]
  uint8_t* scale_ring = out_tiles + kF8Warps * 2 * kF8OutTile;
  float* row_max = reinterpret_cast<float*>(scale_ring + kF8ScaleRing * kF8ScaleSlot);  // [tile parity][part][row]
  uint64_t* full = reinterpret_cast<uint64_t*>(row_max + 2 * 4 * 128);
  uint64_t* empty = full + kF8Stages;
  uint64_t* tfull = empty + kF8Stages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* rmax_bar = drain + 1;  // [quarter]: the four parts' row maxima are in shared memory
  uint64_t* sfull = rmax_bar + 4;   // [group % kF8ScaleGroups]: the group's scales are in shared memory
  uint64_t* sempty = sfull + 4;     // ... and have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp-uniform
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int KB = p.KB;
  const uint64_t limit = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kF8Stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kF8Warps);  // leader's: the promotion warps of both CTAs
    }
    mbar_init(drain, 2);  // the two issuers
    for (int i = 0; i < 4; ++i) {
      mbar_init(&rmax_bar[i], 4);
      mbar_init(&sfull[i], 32);  // every lane of the scale warp
      mbar_init(&sempty[i], kF8Warps);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kF8Producer && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmOut);
  }
  if (warp == kF8Issuer) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  grid_dependents_start();
  grid_dependency_wait();

  // Tiles run down groups of group_m row blocks, as in the int8 GEMM. The quotients come
  // from a product with the reciprocal and one correction, exact up to kF8MaxTiles: an
  // integer division here costs as much as half a K block.
  auto quotient = [](int n, int d, float inv) {
    int q = static_cast<int>(__fmul_rn(static_cast<float>(n), inv));
    const int r = n - q * d;
    q += r >= d ? 1 : (r < 0 ? -1 : 0);
    return q;
  };
  auto tile_at = [&](int tile, int& mb, int& nb) {
    const int per_group = p.group_m * p.num_n;
    const int gid = quotient(tile, per_group, p.inv_per_group);
    const int first_m = gid * p.group_m;
    const int gm = min(p.num_m - first_m, p.group_m);
    const int r = tile - gid * per_group;
    nb = quotient(r, gm, gm == p.group_m ? p.inv_group_m : __frcp_rn(static_cast<float>(gm)));
    mb = first_m + r - nb * gm;
  };

  if (warp >= kF8Warps) {
    regs_dec<kF8RegsCtl>();
    const int my_tiles = pair < p.num_tiles ? (p.num_tiles - pair + npairs - 1) / npairs : 0;
    const int total = my_tiles * KB;  // K blocks of all of this pair's tiles, in order
    if (warp == kF8Producer) {
      // ------------------------------------------------------------ operand tiles (both CTAs)
      const bool one = elect_one();
      const uint64_t pol = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int n = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < p.num_tiles; tile += npairs) {
        int mb, nb;
        tile_at(tile, mb, nb);
        const int a_row = mb * (2 * kBM) + static_cast<int>(rank) * kBM;
        const int b_row = kSwi ? (rank == 0 ? nb * 128 : p.b_row_up + nb * 128) : nb * kBN + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < KB; ++kb, ++n) {
          if (!mbar_wait_bounded_warp(&empty[stage], phase ^ 1u, limit, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full_leader = cluster_map(&full[stage], 0);
          if (one) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kF8StageBytes + p.missing_bytes);
            tma_load_2d_pair(sA + stage * kAStage, &tmA, full_leader, kb * kBK, a_row, pol);
            tma_load_2d_pair(sB + stage * kBStage, &tmB, full_leader, kb * kBK, b_row, pol);
          }
          if (++stage == kF8Stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (rank == 0) {
        // the last copies, which nobody else waits for where a role gave up (bounded, ignores
        // abort; after one wait that ran out they all have had their time)
        for (int m = n - 1; m >= 0 && m >= n - kF8Stages; --m)
          if (!mbar_wait_bounded(&full[m % kF8Stages], static_cast<uint32_t>((m / kF8Stages) & 1), limit, nullptr)) break;
      }
      // The issuers' last arrivals at this CTA's `empty`. They come from the leader, and neither
      // `tfull` nor `drain` says that they have landed here: a CTA that left earlier would have
      // them arrive in shared memory that is the next one's. Where a role gave up, this is also
      // the time in which the peer's copies land.
      for (int m = n - 1; m >= 0 && m >= n - kF8Stages; --m)
        if (!mbar_wait_bounded(&empty[m % kF8Stages], static_cast<uint32_t>((m / kF8Stages) & 1), limit, nullptr)) break;
    } else if (warp == kF8Producer + 1) {
      // ------------------------------------------------------------ scales (both CTAs)
      // Up to sixteen K blocks ahead: each lane copies four rows'
      // (zeros past the end of M), lanes 0 and 1 the two weight blocks'.
      int n = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < p.num_tiles; tile += npairs) {
        int mb, nb;
        tile_at(tile, mb, nb);
        const int row = mb * (2 * kBM) + static_cast<int>(rank) * kBM + lane;
        const float* sx = p.sx + row;
        const float* sw =
            p.sw + int64_t(kSwi ? ((lane & 1) ? p.b_row_up / 128 + nb : nb) : min(2 * nb + (lane & 1), p.last_nb)) * KB;
        for (int kb = 0; kb < KB; ++kb, ++n) {
          const int group = n / kF8ScaleGroup, slot = group & (kF8ScaleGroups - 1);
          if (n % kF8ScaleGroup == 0 &&
              !mbar_wait_bounded_warp(&sempty[slot], ((group / kF8ScaleGroups) & 1) ^ 1u, limit, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_u32(scale_ring) + (n & (kF8ScaleRing - 1)) * kF8ScaleSlot + lane * 4;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool in = row + 32 * j < p.M;
            cp_async4(dst + 128 * j, in ? sx + 32 * j : p.sx, in);
          }
          if (lane < 2) cp_async4(dst + 512, sw + kb, true);
          sx += p.M;
          if (n % kF8ScaleGroup == kF8ScaleGroup - 1) cp_async_arrive(&sfull[slot]);
        }
      }
      if (ok && n % kF8ScaleGroup != 0) cp_async_arrive(&sfull[n / kF8ScaleGroup & (kF8ScaleGroups - 1)]);
      cp_async_commit();
      cp_async_wait<0>();
    } else if (rank == 0) {
      // ------------------------------------------------------------ MMA issuers (leader only): one accumulator buffer each
      constexpr uint32_t idesc = idesc_fp8(2 * kBM, kBN);
      const bool one = elect_one();
      const int buf = warp - kF8Issuer;
      const uint32_t d = tmem + static_cast<uint32_t>(buf * kBN);
      const uint64_t ad0 = smem_desc_sw128(smem_u32(sA)), bd0 = smem_desc_sw128(smem_u32(sB));
      int stage = buf;
      uint32_t phase = 0, buf_phase = 0;
      for (int n = buf; n < total; n += 2) {
        if (!mbar_wait_bounded_warp(&full[stage], phase, limit, abort_flag) ||
            !mbar_wait_bounded_warp(&tempty[buf], buf_phase ^ 1u, limit, abort_flag))
          break;
        tc_fence_after();
        const uint64_t ad = ad0 + static_cast<uint32_t>(stage * (kAStage >> 4));
        const uint64_t bd = bd0 + static_cast<uint32_t>(stage * (kBStage >> 4));
        if (one) {
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k) mma_fp8_pair(d, ad + 2u * k, bd + 2u * k, idesc, k != 0 ? 1u : 0u);
          mma_commit_pair_both(&tfull[buf]);
          mma_commit_pair_both(&empty[stage]);
        }
        buf_phase ^= 1u;
        stage += 2;
        if (stage >= kF8Stages) {
          stage -= kF8Stages;
          phase ^= 1u;
        }
      }
      if (one) mma_commit_pair(cluster_map(drain, 0));
      mbar_wait_bounded(drain, 0, limit, nullptr);  // both issuers' MMAs are done
    }
  } else {
    regs_inc<kF8RegsPromote>();
    // -------------------------------------------------------------- promotion and epilogue (both CTAs)
    // Warps 0..15: warp w owns TMEM lanes 32*(w%4) .. +31 and, of each buffer, columns
    // [32 part, +32) and [128 + 32 part, +32), part = w/4: with SwiGLU gate and up.
    const int quarter = warp & 3;
    const int part = warp >> 2;
    const int row_in_cta = quarter * 32 + lane;
    const uint32_t tempty_leader = cluster_map(tempty, 0);
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(32 * part);
    uint8_t* out_tile = out_tiles + warp * 2 * kF8OutTile;
    const uint32_t my_scales = smem_u32(scale_ring) + row_in_cta * 4;
    const uint32_t block_scales = smem_u32(scale_ring) + 512;
    // What the next K block needs is fetched behind the release of this one: its scales,
    // and whether its products are there already (a wait costs some 200 cycles even when
    // it need not wait).
    const int total = pair < p.num_tiles ? (p.num_tiles - pair + npairs - 1) / npairs * KB : 0;
    int n = 0;  // K blocks so far: buffer n % 2, scale slot n % 16
    int iter = 0;
    bool ready = false;
    bool ok = total > 0 && mbar_wait_bounded_warp(&sfull[0], 0, p.wait_limit_ns, abort_flag);
    float sx_n = ok ? ld_shared_f32(my_scales) : 0.0f;
    float2 sw_n = ok ? ld_shared_f32x2(block_scales) : make_float2(0.0f, 0.0f);
    for (int tile = pair; ok && tile < p.num_tiles; tile += npairs, ++iter) {
      float acc[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
#pragma unroll 1
      for (int kb = 0; kb < KB; ++kb) {
        const float f0 = __fmul_rn(sx_n, sw_n.x), f1 = __fmul_rn(sx_n, sw_n.y);
        if (!__all_sync(0xFFFFFFFFu, ready) &&
            !mbar_wait_bounded_warp(&tfull[n & 1], (n >> 1) & 1, p.wait_limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tlane + static_cast<uint32_t>((n & 1) * kBN);
        uint32_t r[32];
        tmem_ld32(ta, r);
        tmem_ld_wait32(r);
        f8_promote(acc[0], r, f0);
        tmem_ld32(ta + 128, r);
        tmem_ld_wait32(r);
        tc_fence_before();
        if (lane == 0) mbar_arrive_remote(tempty_leader + (n & 1) * 8);  // the whole warp's loads are done
        ++n;
        const bool more = n < total;
        if (more && (n & (kF8ScaleGroup - 1)) == 0) {
          const int group = n / kF8ScaleGroup;
          __syncwarp();  // every lane has read the last group's scales
          if (lane == 0) mbar_arrive(&sempty[(group - 1) & (kF8ScaleGroups - 1)]);
          if (!mbar_wait_bounded_warp(&sfull[group & (kF8ScaleGroups - 1)], (group / kF8ScaleGroups) & 1,
                                      p.wait_limit_ns, abort_flag)) {
            ok = false;
            break;
          }
        }
        f8_promote(acc[1], r, f1);
        if (more) {
          const uint32_t slot = (n & (kF8ScaleRing - 1)) * kF8ScaleSlot;
          sx_n = ld_shared_f32(my_scales + slot);
          sw_n = ld_shared_f32x2(block_scales + slot);
          ready = mbar_test_wait(&tfull[n & 1], (n >> 1) & 1);
        }
      }
      if (!ok) break;
      int mb, nb;
      tile_at(tile, mb, nb);

      // Epilogue: 32 rows x 32 columns at a time through one of the warp's two
      // shared-memory tiles (in TMA's swizzle), which a TMA store takes away while the
      // next tile's K blocks are promoted.
      const int row0 = mb * (2 * kBM) + static_cast<int>(rank) * kBM + quarter * 32;
      bulk_wait_read<0>();  // lane 0's earlier stores have read their tiles
      __syncwarp();
      if constexpr (kSwi) {
        const int n0 = nb * 128 + 32 * part;  // first h column of this thread
        float amax = 0.0f;
        if (p.bias != nullptr) {
          f8_bias32(acc[0], p.bias + n0);
          f8_bias32(acc[1], p.bias + p.b_row_up + n0);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          acc[0][i] = __fmul_rn(silu_approx(acc[0][i]), acc[1][i]);
          if constexpr (EPI == kF8SwiGLUQuant) amax = max_nan(amax, fabsf(acc[0][i]));
        }
        if constexpr (EPI == kF8SwiGLUQuant) {
          // the row's 128 h columns are one scale block; its four parts sit in four warps
          float* maxima = row_max + (iter & 1) * 512 + row_in_cta;
          maxima[part * 128] = amax;
          __syncwarp();
          if (lane == 0) mbar_arrive(&rmax_bar[quarter]);
          if (!mbar_wait_bounded_warp(&rmax_bar[quarter], static_cast<uint32_t>(iter & 1), limit, abort_flag)) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) amax = max_nan(amax, maxima[i * 128]);
          float inv;
          const float s = fp8_scale(amax, inv);
          if (part == 0 && row0 + lane < p.M) p.sh[int64_t(nb) * p.M + row0 + lane] = s;
#pragma unroll
          for (int g = 0; g < 2; ++g) {  // 32 bytes a row, four rows to a 128-byte line
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* a = &acc[0][16 * g + 4 * i];
              w[i] = f32x4_to_e4m3x4(__fmul_rn(a[0], inv), __fmul_rn(a[1], inv), __fmul_rn(a[2], inv),
                                     __fmul_rn(a[3], inv));
            }
            *reinterpret_cast<uint4*>(out_tile + lane * 32 + ((g ^ (lane >> 2)) & 1) * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint4*>(out_tile + lane * 64 + ((g ^ (lane >> 1)) & 3) * 16) = f8_pack8(&acc[0][8 * g]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < p.M) {
          tma_store_2d(&tmOut, out_tile, n0, row0);
          bulk_commit();
        }
      } else {
        const int n0 = nb * kBN + 32 * part;  // and n0 + 128
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int n = n0 + 128 * pass + 8 * g;
            if (p.bias != nullptr && n < p.N) f8_bias8(&acc[pass][8 * g], p.bias + n);
            *reinterpret_cast<uint4*>(out_tile + pass * kF8OutTile + lane * 64 + ((g ^ (lane >> 1)) & 3) * 16) =
                f8_pack8(&acc[pass][8 * g]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < p.M) {
          if (n0 < p.N) tma_store_2d(&tmOut, out_tile, n0, row0);
          if (n0 + 128 < p.N) tma_store_2d(&tmOut, out_tile + kF8OutTile, n0 + 128, row0);
          bulk_commit();
        }
      }
    }
    bulk_wait_read<0>();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kF8Issuer) tmem_dealloc_pair(tmem, kTmemCols);
}

// ---------------------------------------------------------------- product, few tokens
// With few tokens the product is bound by reading the weight, so the weight is the
// MMA's M side: a CTA takes 128 weight rows (SwiGLU: 128 gate and the 128 matching up
// rows) and TM tokens (the N side), and where the row tiles do not fill the SMs a
// cluster of C CTAs splits the K axis of one tile. Every K block of 128 is summed into
// a tensor-memory buffer of its own and promoted into fp32 registers with its scales as
// in the large kernel (thread = weight row, register = token). The CTAs of a cluster
// then leave their partial sums in shared memory, and each adds up, in the order of the
// K axis, the tokens that fall to it and writes them out (a warp per token, four
// columns a lane), so the result does not depend on timing and nothing is kept in
// global memory.
// The tokens are shared out evenly over the tiles, and rows that do not exist are not
// loaded: the TMA would fill them with zeros, but is slow at it (one token, 5376 x 28672:
// 34.3 us with 15 such rows a load, 28.4 without). What their place in shared memory holds
// reaches only columns that are not written.
// (Tiles of 64 tokens, and of 128 with SwiGLU, spill 16 bytes of registers a thread.)
constexpr int kF8sMaxStages = 12;
constexpr int kF8sThreads = 384;  // eight promotion warps, operands, MMA, scales, one idle until the output
constexpr int kF8sScaleRing = 16;

template <int R, int TM>
struct Fp8Small {
  static constexpr int kStage = R * 128 * 128 + TM * 128;
  static constexpr int kCols = R * TM;                       // tensor-memory columns of one K block
  static constexpr int kHalf = kCols / 2;                    // columns of a promotion thread
  static constexpr int kBufs = kCols > 128 ? 2 : 4;
  static constexpr int kTmem = kCols * kBufs <= 64 ? 64 : kCols * kBufs <= 128 ? 128 : kCols * kBufs <= 256 ? 256 : 512;
  static constexpr int kPartials = R * TM * 128 * 4;
  static_assert(kPartials <= 3 * kStage, "the partial sums fit in the operand ring");
  static constexpr int kScaleSlot = TM * 4 + 16;
  static constexpr int kFixed = kF8sScaleRing * kScaleSlot + 512 /*barriers*/ + 1024 /*align*/;
};
// Nor does one of these CTAs, the smallest of three stages, fit beside a CTA of the other
// products whose clusters wait for all 512 columns.
static_assert(3 * Fp8Small<1, 16>::kStage + Fp8Small<1, 16>::kFixed + (kGemmSmem < kF4Smem ? kGemmSmem : kF4Smem) +
                      2 * kSmSharedPerCta > kSmShared, "tensor memory without a wait");

struct Fp8SmallParams {
  int M, N, KB;
  int num_m, num_n;    // token tiles, row tiles
  int stages, splits;  // ring depth; CTAs per cluster
  int x_rows;          // token rows of a tile: ceil(M / num_m), at most TM
  int up_row;          // SwiGLU: first up row of the weight (= F)
  int swiglu_rows;     // F / 128
  const float *sx, *sw;
  const __nv_bfloat16* bias;
  void* out;
  float* sh;
  uint64_t wait_limit_ns;
  uint32_t missing_bytes;   // zero; bytes that every stage waits for in vain (test of the waits)
};

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 x e4m3 -> fp32, one CTA.
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 8, 16 or 32 consecutive columns of the warp's lanes, and the wait that the loaded
// registers depend on.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }

__device__ __forceinline__ void tmem_ld_cols_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}

__device__ __forceinline__ void tmem_ld_cols_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])::"memory");
}

__device__ __forceinline__ void tmem_ld_cols_wait(uint32_t (&r)[32]) { tmem_ld_wait32(r); }

__device__ __forceinline__ float4 ld_shared_cluster_f32x4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int EPI, int TM>
__global__ void __launch_bounds__(kF8sThreads, (EPI == kF8BF16 ? TM : 2 * TM) <= 64 ? 2 : 1)
    gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                          const Fp8SmallParams p) {
  constexpr int R = EPI == kF8BF16 ? 1 : 2;
  using Cfg = Fp8Small<R, TM>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint8_t* ring = smem;  // [stage]: R weight tiles, then the token tile
  uint8_t* scale_ring = ring + S * Cfg::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_ring + kF8sScaleRing * Cfg::kScaleSlot);
  uint64_t* empty = full + kF8sMaxStages;
  uint64_t* tfull = empty + kF8sMaxStages;
  uint64_t* tempty = tfull + 4;
  uint64_t* sfull = tempty + 4;  // [group of four K blocks % 4]
  uint64_t* sempty = sfull + 4;
  uint64_t* drain = sempty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.splits;
  const int tile = blockIdx.x / p.splits;
  const int nt = tile / p.num_m, mt = tile - nt * p.num_m;
  const int kb0 = static_cast<int>(int64_t(p.KB) * rank / p.splits);
  const int nkb = static_cast<int>(int64_t(p.KB) * (rank + 1) / p.splits) - kb0;
  const uint64_t limit = p.wait_limit_ns;

  // The operand warp sets up the barriers and sends for the first stages at once, while
  // tensor memory is allocated.
  const bool one = elect_one();
  auto load_stage = [&](int stage, int i) {
    uint8_t* dst = ring + stage * Cfg::kStage;
    const uint64_t pol = policy_evict_normal();
    const int k = (kb0 + i) * 128;
    mbar_arrive_expect_tx(&full[stage], R * 128 * 128 + p.x_rows * 128 + p.missing_bytes);
    tma_load_2d(dst, &tmW, &full[stage], k, nt * 128, pol);
    if (R == 2) tma_load_2d(dst + 128 * 128, &tmW, &full[stage], k, p.up_row + nt * 128, pol);
    tma_load_2d(dst + R * 128 * 128, &tmX, &full[stage], k, mt * p.x_rows, pol);
  };
  if (warp == 8) {
    if (one) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmX);
      for (int s = 0; s < S; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      for (int b = 0; b < 4; ++b) {
        mbar_init(&tfull[b], 1);
        mbar_init(&tempty[b], 8);
        mbar_init(&sfull[b], 32);
        mbar_init(&sempty[b], 8);
      }
      mbar_init(drain, 1);
      *abort_flag = 0;
      fence_mbarrier_init();
    }
    grid_dependency_wait();
    if (one)
      for (int s = 0; s < min(S, nkb); ++s) load_stage(s, s);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  grid_dependents_start();
  grid_dependency_wait();

  if (warp == 8) {
    // ------------------------------------------------------------ operand tiles
    int stage = 0, i = min(S, nkb);  // the first round is on its way
    uint32_t phase = 0;
    for (; i < nkb; ++i) {
      if (!mbar_wait_bounded_warp(&empty[stage], phase, limit, abort_flag)) break;
      if (one) load_stage(stage, i);
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // the last copies, which nobody else waits for where a role gave up (bounded, ignores
    // abort; after one wait that ran out they all have had their time)
    for (int m = i - 1; m >= 0 && m >= i - S; --m)
      if (!mbar_wait_bounded(&full[m % S], static_cast<uint32_t>((m / S) & 1), limit, nullptr)) break;
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_fp8(128, TM);
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nkb; ++i) {
      const int b = i % Cfg::kBufs;
      if (!mbar_wait_bounded_warp(&full[stage], phase, limit, abort_flag) ||
          !mbar_wait_bounded_warp(&tempty[b], ((i / Cfg::kBufs) & 1) ^ 1u, limit, abort_flag))
        break;
      tc_fence_after();
      const uint32_t base = smem_u32(ring + stage * Cfg::kStage);
      const uint64_t xd = smem_desc_sw128(base + R * 128 * 128);
      if (one) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint64_t wd = smem_desc_sw128(base + r * 128 * 128);
          const uint32_t d = tmem + static_cast<uint32_t>(b * Cfg::kCols + r * TM);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_fp8(d, wd + 2u * k, xd + 2u * k, idesc, k != 0 ? 1u : 0u);
        }
        mma_commit(&tfull[b]);
        mma_commit(&empty[stage]);
      }
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (one) mma_commit(drain);
    mbar_wait_bounded(drain, 0, limit, nullptr);
  } else if (warp == 10) {
    // ------------------------------------------------------------ scales, handed over by fours
    bool ok = true;
    for (int i = 0; ok && i < nkb; ++i) {
      if ((i & 3) == 0 && !mbar_wait_bounded_warp(&sempty[(i >> 2) & 3], ((i >> 4) & 1) ^ 1u, limit, abort_flag)) {
        ok = false;
        break;
      }
      const uint32_t dst = smem_u32(scale_ring) + (i & (kF8sScaleRing - 1)) * Cfg::kScaleSlot;
      const int64_t kb = kb0 + i;
#pragma unroll
      for (int j = 0; j < (TM + 31) / 32; ++j) {
        const int m = 32 * j + lane;
        const bool in = m < p.x_rows && mt * p.x_rows + m < p.M;
        if (m < TM) cp_async4(dst + m * 4, in ? p.sx + kb * p.M + mt * p.x_rows + m : p.sx, in);
      }
      if (lane < R) cp_async4(dst + TM * 4 + lane * 4, p.sw + int64_t(nt + lane * p.swiglu_rows) * p.KB + kb, true);
      if ((i & 3) == 3 || i == nkb - 1) cp_async_arrive(&sfull[(i >> 2) & 3]);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp < 8) {
    // ------------------------------------------------------------ promotion: thread = weight row
    // Warps 0..7: TMEM lanes 32*(w%4) .. +31 and one half of the columns: with SwiGLU
    // gate or up, else half of the tokens.
    const int half = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    constexpr int kChunk = Cfg::kHalf % 32 == 0 ? 32 : Cfg::kHalf % 16 == 0 ? 16 : 8;
    float2 acc[Cfg::kHalf / 2];
#pragma unroll
    for (int m = 0; m < Cfg::kHalf / 2; ++m) acc[m] = make_float2(0.0f, 0.0f);
    const uint32_t tcol = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(half * Cfg::kHalf);
    const uint32_t sx_at = R == 2 ? 0 : half * Cfg::kHalf * 4, sw_at = TM * 4 + (R == 2 ? half * 4 : 0);
#pragma unroll 1
    for (int i = 0; i < nkb; ++i) {
      const int b = i % Cfg::kBufs;
      if ((i & 3) == 0 && !mbar_wait_bounded_warp(&sfull[(i >> 2) & 3], (i >> 4) & 1, limit, abort_flag)) break;
      const uint32_t slot = smem_u32(scale_ring) + (i & (kF8sScaleRing - 1)) * Cfg::kScaleSlot;
      const float swv = ld_shared_f32(slot + sw_at);
      if (!mbar_wait_bounded_warp(&tfull[b], (i / Cfg::kBufs) & 1, limit, abort_flag)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < Cfg::kHalf / kChunk; ++c) {
        uint32_t v[kChunk];
        tmem_ld_cols(tcol + static_cast<uint32_t>(b * Cfg::kCols + c * kChunk), v);
        tmem_ld_cols_wait(v);
        if (c == Cfg::kHalf / kChunk - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[b]);
        }
#pragma unroll
        for (int q = 0; q < kChunk / 4; ++q) {
          const float4 s = ld_shared_f32x4(slot + sx_at + (c * kChunk + 4 * q) * 4);
          float2* a = &acc[(c * kChunk + 4 * q) / 2];
          const float2 w2 = make_float2(swv, swv);
          a[0] = __ffma2_rn(make_float2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])),
                            __fmul2_rn(make_float2(s.x, s.y), w2), a[0]);
          a[1] = __ffma2_rn(make_float2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])),
                            __fmul2_rn(make_float2(s.z, s.w), w2), a[1]);
        }
      }
      if ((i & 3) == 3) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[(i >> 2) & 3]);
      }
    }
    // every K block has been read, so the operand ring is free: partial sums [column][row]
    named_barrier(1, 256);
    float* part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int m = 0; m < Cfg::kHalf / 2; ++m) {
      part[(half * Cfg::kHalf + 2 * m) * 128 + row] = acc[m].x;
      part[(half * Cfg::kHalf + 2 * m + 1) * 128 + row] = acc[m].y;
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();

  // ------------------------------------------------------------ sums over the cluster and output
  const int per = (p.x_rows + p.splits - 1) / p.splits;
  const int n = nt * 128 + 4 * lane;  // this lane's four columns (SwiGLU: of h)
  for (int m = rank * per + warp; m < min(rank * per + per, p.x_rows); m += kF8sThreads / 32) {
    const int row = mt * p.x_rows + m;
    if (row >= p.M) break;
    float4 v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t at = smem_u32(ring) + ((r * TM + m) * 128 + 4 * lane) * 4;
      v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int c = 0; c < p.splits; ++c) {
        float4 t;
        if (p.splits == 1) {
          t = ld_shared_f32x4(at);
        } else {
          uint32_t from;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(c));
          t = ld_shared_cluster_f32x4(from);
        }
        v[r] = make_float4(__fadd_rn(v[r].x, t.x), __fadd_rn(v[r].y, t.y), __fadd_rn(v[r].z, t.z),
                           __fadd_rn(v[r].w, t.w));
      }
      if (p.bias != nullptr && n < p.N) {
        const uint2 b = *reinterpret_cast<const uint2*>(p.bias + r * p.up_row + n);
        v[r].x = __fadd_rn(v[r].x, __uint_as_float(b.x << 16));
        v[r].y = __fadd_rn(v[r].y, __uint_as_float(b.x & 0xFFFF0000u));
        v[r].z = __fadd_rn(v[r].z, __uint_as_float(b.y << 16));
        v[r].w = __fadd_rn(v[r].w, __uint_as_float(b.y & 0xFFFF0000u));
      }
    }
    float4 h = v[0];
    if constexpr (R == 2) {
      h.x = __fmul_rn(silu_approx(h.x), v[R - 1].x);
      h.y = __fmul_rn(silu_approx(h.y), v[R - 1].y);
      h.z = __fmul_rn(silu_approx(h.z), v[R - 1].z);
      h.w = __fmul_rn(silu_approx(h.w), v[R - 1].w);
    }
    if constexpr (EPI == kF8SwiGLUQuant) {  // the warp holds one whole scale block
      float a = max_nan(max_nan(fabsf(h.x), fabsf(h.y)), max_nan(fabsf(h.z), fabsf(h.w)));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      float inv;
      const float s = fp8_scale(a, inv);
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + int64_t(row) * p.N + n) =
          f32x4_to_e4m3x4(__fmul_rn(h.x, inv), __fmul_rn(h.y, inv), __fmul_rn(h.z, inv), __fmul_rn(h.w, inv));
      if (lane == 0) p.sh[int64_t(nt) * p.M + row] = s;
    } else if (n < p.N) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + int64_t(row) * p.N + n) =
          make_uint2(pack_bf16x2(h.x, h.y), pack_bf16x2(h.z, h.w));
    }
  }
  cluster_sync_relaxed();  // the peers have read this CTA's sums
  if (warp == 9) tmem_dealloc(tmem, Cfg::kTmem);
}

}  // namespace h3q
