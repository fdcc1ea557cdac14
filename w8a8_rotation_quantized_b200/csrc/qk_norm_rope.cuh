// RMS norm of every query and key head and the rotation of positions, in one pass.
//   n = x * (1 / sqrt(mean(x^2) + eps)) * w      (fp32, over the head's D elements)
//   a' = a c - b s, b' = b c + a s               for each rotated pair (a, b)
// c, s: row position[t] of the caller's tables (fp32 [P, rot / 2]). Pairs are
// (i, i + rot/2), or (2 i, 2 i + 1) when interleaved; elements past rot are only
// normalised. Rounded to bf16 once, at the end.
//
// A head is read by a group of lanes, eight elements (16 bytes) each; a warp works on
// one token, so its lanes load the token's table row once for all of its heads.
// Each lane holds its elements until they are stored, and a group's loads come
// before its stores, so q_out and k_out may be q and k themselves.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace h3q {

struct QkParams {
  const __nv_bfloat16 *q, *k;     // [S, ldq], [S, ldk]
  __nv_bfloat16 *qo, *ko;         // [S, ldqo], [S, ldko]
  int64_t ldq, ldk, ldqo, ldko;
  const __nv_bfloat16 *wq, *wk;   // [D] or null
  const float *cos, *sin;         // [P, rot / 2]
  const int* pos;                 // [S] or null: token t is at position t
  int64_t S;
  int Hq, Hk, D, rot, P;
  float eps;
};

// G: lanes per head (a power of two, 8 G >= D).
template <int G, bool INTER>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkParams p) {
  constexpr int kHeads = 32 / G;  // heads a warp takes at once
  const int lane = threadIdx.x & 31;
  const int l = lane % G, sub = lane / G;
  const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
  const bool live = 8 * l < p.D;
  const bool turns = 8 * l < p.rot;
  const int half = p.rot >> 1;
  const int H = p.Hq + p.Hk;
  // half-split pairs: element i's partner sits rot / 2 away, in another lane
  const bool second = !INTER && 8 * l >= half;
  const int partner = INTER ? lane : (turns ? (second ? lane - half / 8 : lane + half / 8) : lane);
  const int pl = partner % G;
  for (int64_t t = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); t < p.S; t += warps) {
    float c[8], s[8];
    if (turns) {
      const int at = p.pos != nullptr ? p.pos[t] : static_cast<int>(t);
      const bool good = at >= 0 && at < p.P;
      const int64_t off = int64_t(good ? at : 0) * half;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = INTER ? 4 * l + i / 2 : (8 * l + i) - (second ? half : 0);
        c[i] = good ? __ldg(p.cos + off + j) : __int_as_float(0x7FC00000);
        s[i] = __ldg(p.sin + off + j);
        if (INTER ? !(i & 1) : !second) s[i] = -s[i];  // the pair's first element takes - b s
      }
    }
    for (int h0 = 0; h0 < H; h0 += kHeads) {
      const int h = h0 + sub;
      const bool is_q = h < p.Hq;
      const bool ok = live && h < H;
      const int64_t hc = int64_t(is_q ? h : h - p.Hq) * p.D + 8 * l;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (ok) raw = *reinterpret_cast<const uint4*>((is_q ? p.q + t * p.ldq : p.k + t * p.ldk) + hc);
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      float x[8], xp[8];
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        ss = __fmaf_rn(x[2 * i], x[2 * i], ss);
        ss = __fmaf_rn(x[2 * i + 1], x[2 * i + 1], ss);
        const uint32_t o = INTER ? w[i] : __shfl_sync(0xFFFFFFFFu, w[i], partner);
        xp[2 * i] = __uint_as_float(INTER ? o & 0xFFFF0000u : o << 16);
        xp[2 * i + 1] = __uint_as_float(INTER ? o << 16 : o & 0xFFFF0000u);
      }
#pragma unroll
      for (int o = 1; o < G; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(p.D)), p.eps)));
      if (ok) {
        const __nv_bfloat16* wt = is_q ? p.wq : p.wk;
        uint32_t out[4];
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float n = __fmul_rn(x[i], r);
          if (wt != nullptr) n = __fmul_rn(n, __bfloat162float(wt[8 * l + i]));
          if (turns) {
            float np = __fmul_rn(xp[i], r);
            if (wt != nullptr) np = __fmul_rn(np, __bfloat162float(wt[INTER ? 8 * l + (i ^ 1) : 8 * pl + i]));
            n = __fmaf_rn(n, c[i], __fmul_rn(np, s[i]));
          }
          y[i] = n;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
          out[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>((is_q ? p.qo + t * p.ldqo : p.ko + t * p.ldko) + hc) =
            make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
}

}  // namespace h3q
