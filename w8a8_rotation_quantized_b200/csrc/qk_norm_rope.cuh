// RMS norm of every query and key head and the rotation of positions, in one pass.
//   n = x * (1 / sqrt(mean(x^2) + eps)) * w      (fp32, over the head's D elements)
//   a' = a c - b s, b' = b c + a s               for each rotated pair (a, b)
// c, s: row position[t] of the caller's tables (fp32 [P, rot / 2]). Pairs are
// (i, i + rot/2), or (2 i, 2 i + 1) when interleaved; elements past rot are only
// normalised. Rounded to bf16 once, at the end.
//
// A head is read by a group of lanes, eight elements (16 bytes) each; a warp works on
// one token at a time, so its lanes load the token's table row once for all of its
// heads and fold the norm's weights into it: with C_i = w_i c_i and S_i = -+w_p s_i (p
// the partner of i), the result is (x_i r) C_i + (x_p r) S_i. The root comes before the
// weight, as in the formula: after it, a weight above one carried a large finite element
// to infinity, and where the sum of squares overflows (r = 0) that gave NaN for 0. It costs
// a multiplication for each pair of elements: 1% to 2% of the time with half-split pairs
// (4% to 6% where everything is in L2), nothing with interleaved ones, whose partner is in
// the same lane.
// Six heads a lane group are worked on while the next six load (two blocks an SM: 117 us
// at 84 heads of 128 over 16384 tokens, 115 interleaved or with the root last; with it last,
// eight at once without loads ahead 124, four 149, three or more blocks 120 to 135). Every
// element is read and written once and memory is the bound: 713 MB there, 93% of the
// measured copy rate. Few tokens are spread over more warps by splitting the heads.
//
// A head's loads come before its stores and no head reads another's elements, so q_out
// and k_out may be q and k themselves.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx_sm100.cuh"

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

// G: lanes per head (a power of two, 8 G >= D). Grid: x tokens (warps stride over
// them), y the part of the heads.
template <int G, bool INTER>
__global__ void __launch_bounds__(256, 2) qk_norm_rope_kernel(const QkParams p) {
  constexpr int kHeads = 32 / G;  // heads a warp step takes
  constexpr int kUnroll = 6;      // steps worked on, and as many in flight
  const int lane = threadIdx.x & 31;
  const int l = lane % G, sub = lane / G;
  const bool live = 8 * l < p.D;
  const bool turns = 8 * l < p.rot;
  const int half = p.rot >> 1;
  // half-split pairs: element i's partner sits rot / 2 away, in another lane
  const bool second = !INTER && 8 * l >= half;
  const int partner = INTER || !turns ? lane : (second ? lane - half / 8 : lane + half / 8);
  const float inv_d = __frcp_rn(static_cast<float>(p.D));
  const int steps_q = (p.Hq + kHeads - 1) / kHeads, steps_k = (p.Hk + kHeads - 1) / kHeads;
  const int per = (steps_q + steps_k + gridDim.y - 1) / gridDim.y;
  const int begin = blockIdx.y * per, end = min(begin + per, steps_q + steps_k);
  grid_dependents_start();
  grid_dependency_wait();
  const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
  for (int64_t t = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); t < p.S; t += warps) {
    float c[8], s[8];  // this token's table row for this lane's elements, s signed
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.0f, s[i] = 0.0f;
    if (turns) {
      const int at = p.pos != nullptr ? p.pos[t] : static_cast<int>(t);
      const bool good = at >= 0 && at < p.P;
      const int64_t off = int64_t(good ? at : 0) * half + (INTER ? 4 * l : 8 * l - (second ? half : 0));
      constexpr int kVec = INTER ? 1 : 2;  // 16-byte pieces of the row
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const float4 cv = reinterpret_cast<const float4*>(p.cos + off)[v];
        const float4 sv = reinterpret_cast<const float4*>(p.sin + off)[v];
        const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (INTER) {
            c[2 * i] = c[2 * i + 1] = cc[i];
            s[2 * i] = -ss[i];
            s[2 * i + 1] = ss[i];
          } else {
            c[4 * v + i] = cc[i];
            s[4 * v + i] = second ? ss[i] : -ss[i];
          }
        }
      }
      if (!good) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = __int_as_float(0x7FC00000);
      }
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int base = which ? steps_q : 0;
      const int lo = max(begin, base) - base, hi = min(end, base + (which ? steps_k : steps_q)) - base;
      if (lo >= hi) continue;
      const int H = which ? p.Hk : p.Hq;
      const __nv_bfloat16* wt = which ? p.wk : p.wq;
      const __nv_bfloat16* src = (which ? p.k + t * p.ldk : p.q + t * p.ldq) + 8 * l;
      __nv_bfloat16* dst = (which ? p.ko + t * p.ldko : p.qo + t * p.ldqo) + 8 * l;
      float2 cw[4], sw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cw[i] = make_float2(c[2 * i], c[2 * i + 1]);
        sw[i] = make_float2(s[2 * i], s[2 * i + 1]);
      }
      if (wt != nullptr && live) {
        float wi[8], wp[8];
        load_bf16x8(wt + 8 * l, wi);
        load_bf16x8(wt + 8 * (partner % G), wp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cw[i] = __fmul2_rn(cw[i], make_float2(wi[2 * i], wi[2 * i + 1]));
          if (turns) sw[i] = __fmul2_rn(sw[i], INTER ? make_float2(wp[2 * i + 1], wp[2 * i]) : make_float2(wp[2 * i], wp[2 * i + 1]));
        }
      }
      uint4 next[kUnroll];
      auto fetch = [&](int st) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = (st + u) * kHeads + sub;
          next[u] = make_uint4(0u, 0u, 0u, 0u);
          if (st + u < hi && live && h < H) next[u] = *reinterpret_cast<const uint4*>(src + int64_t(h) * p.D);
        }
      };
      fetch(lo);
      for (int st = lo; st < hi; st += kUnroll) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) raw[u] = next[u];
        if (st + kUnroll < hi) fetch(st + kUnroll);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (st + u >= hi) break;  // the same for the whole warp
          const int h = (st + u) * kHeads + sub;
          const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
          float2 x[4], y[4];
          float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            s2 = __ffma2_rn(x[i], x[i], s2);
          }
          float ss = s2.x + s2.y;
#pragma unroll
          for (int o = 1; o < G; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
          const float r = rsqrtf(__fmaf_rn(ss, inv_d, p.eps));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 r2 = make_float2(r, r), n = __fmul2_rn(x[i], r2);
            if constexpr (INTER) {
              y[i] = __fmul2_rn(n, cw[i]);
              if (turns) y[i] = __ffma2_rn(make_float2(n.y, n.x), sw[i], y[i]);  // else no partner: 0 times its infinity is not 0
            } else {  // past rot the partner is the element itself
              const uint32_t o = __shfl_sync(0xFFFFFFFFu, w[i], partner);
              const float2 np = __fmul2_rn(make_float2(__uint_as_float(o << 16), __uint_as_float(o & 0xFFFF0000u)), r2);
              y[i] = __ffma2_rn(n, cw[i], __fmul2_rn(np, sw[i]));
            }
          }
          if (live && h < H) {
            uint32_t out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(y[i].x, y[i].y);
              out[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(dst + int64_t(h) * p.D) = make_uint4(out[0], out[1], out[2], out[3]);
          }
        }
      }
    }
  }
}

}  // namespace h3q
