// qk_norm_rope.cu -- RMS norm of every query and key head with the position rotation in the same pass.
//
// For each head row x of D elements: y = x * rsqrt(mean(x^2) + eps) * w, then pair i of y at the token's position p,
// (a, b), becomes (a cos - b sin, b cos + a sin) with cos, sin from row p of the caller's fp32 tables; pairs are
// (i, i + D/2) or (2i, 2i + 1).  All in fp32, rounded to bf16 once at the end.
//
// What bounds it: HBM.  Every element is read once (2 bytes) and written once (2 bytes).  A lane holds 16 elements --
// eight whole pairs -- of a head, D/16 lanes a head, so the sum of squares takes three (two) shuffles and the
// rotation none.  A warp takes one token's heads four (eight) at a time: the table values of the token, twice the
// bytes of a head, are loaded once for all of them.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace attn {
namespace {

#ifndef ATTN_NORM_U
#define ATTN_NORM_U 4
#endif
#ifndef ATTN_NORM_MINB
#define ATTN_NORM_MINB 2
#endif
constexpr int kNormWarps = 8;

// STYLE 0: no rotation, 1: pairs (i, i + D/2), 2: pairs (2i, 2i + 1).
template <int D, int STYLE>
__global__ void __launch_bounds__(32 * kNormWarps, ATTN_NORM_MINB) qk_norm_rope_kernel(const QkNormRopeLaunch p, int chunks, int rounds) {
  constexpr int TPR = D / 16;    // lanes per head
  constexpr int HPW = 32 / TPR;  // heads per warp and round
  constexpr int U = ATTN_NORM_U;  // rounds in flight
  constexpr int OFF_B = STYLE == 1 ? D / 2 : 8;  // from a lane's first 8 elements to its other 8
  const int lane = threadIdx.x & 31;
  const long long job = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  const long long tok = job / chunks;
  if (tok >= (long long)p.B * p.L) return;
  const int chunk = (int)(job - tok * chunks);
  const int sub = lane % TPR, hw = lane / TPR;
  const int i0 = 8 * sub;                          // the lane's first pair
  const int d0 = STYLE == 1 ? 8 * sub : 16 * sub;  // its first element
  const long long sb = tok / p.L, st = tok - sb * p.L;
  const int pos = p.positions != nullptr ? p.positions[tok] : 0;
  const __nv_bfloat16* qrow = reinterpret_cast<const __nv_bfloat16*>(p.q) + sb * p.qs[0] + st * p.qs[1] + d0;
  const __nv_bfloat16* krow = reinterpret_cast<const __nv_bfloat16*>(p.k) + sb * p.ks[0] + st * p.ks[1] + d0;
  const int H = p.Hq + p.Hkv;
  const int r1 = min((chunk + 1) * rounds, (H + HPW - 1) / HPW);
  uint4 x[U][2];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (r0 + u) * HPW + hw;
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      if (r0 + u < r1 && h < H) {
        const __nv_bfloat16* src = h < p.Hq ? qrow + h * p.qs[2] : krow + (h - p.Hq) * p.ks[2];
        x[u][0] = *reinterpret_cast<const uint4*>(src);
        x[u][1] = *reinterpret_cast<const uint4*>(src + OFF_B);
      }
    }
  };
  int r0 = chunk * rounds;
  load(r0);  // while the position, and then the tables, are on their way
  if (pos < 0 || (STYLE != 0 && pos >= p.rope.max_pos)) {  // -1 pads; anything else out of range is an error
    if (pos != -1 && lane == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    return;
  }
  float c[8], s[8];
  if constexpr (STYLE != 0) {
    const float4* cr = reinterpret_cast<const float4*>(p.rope.cos + (size_t)pos * (D / 2) + i0);
    const float4* sr = reinterpret_cast<const float4*>(p.rope.sin + (size_t)pos * (D / 2) + i0);
    *reinterpret_cast<float4*>(c) = __ldg(cr);
    *reinterpret_cast<float4*>(c + 4) = __ldg(cr + 1);
    *reinterpret_cast<float4*>(s) = __ldg(sr);
    *reinterpret_cast<float4*>(s + 4) = __ldg(sr + 1);
  }
  __nv_bfloat16* qdst = reinterpret_cast<__nv_bfloat16*>(p.q_out) + sb * p.qos[0] + st * p.qos[1] + d0;
  __nv_bfloat16* kdst = reinterpret_cast<__nv_bfloat16*>(p.k_out) + sb * p.kos[0] + st * p.kos[1] + d0;
  const uint4* wq = reinterpret_cast<const uint4*>(
      p.q_weight != nullptr ? reinterpret_cast<const __nv_bfloat16*>(p.q_weight) + d0 : nullptr);
  const uint4* wk = reinterpret_cast<const uint4*>(
      p.k_weight != nullptr ? reinterpret_cast<const __nv_bfloat16*>(p.k_weight) + d0 : nullptr);
  while (true) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u >= r1) break;  // warp-uniform
      const int h = (r0 + u) * HPW + hw;
      float v[16];
      unpack8(x[u][0], *reinterpret_cast<float(*)[8]>(v));
      unpack8(x[u][1], *reinterpret_cast<float(*)[8]>(v + 8));
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
      for (int mask = 1; mask < TPR; mask <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, mask);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      const bool is_q = h < p.Hq;
      const uint4* wp = is_q ? wq : wk;  // (from L1: held in registers they would cost a quarter of the warps)
      if (wp != nullptr) {
        float w[16];
        unpack8(__ldg(wp), *reinterpret_cast<float(*)[8]>(w));
        unpack8(__ldg(wp + OFF_B / 8), *reinterpret_cast<float(*)[8]>(w + 8));
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= inv * w[j];
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= inv;
      }
      float y[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ia = STYLE == 1 ? j : 2 * j, ib = STYLE == 1 ? j + 8 : 2 * j + 1;
        if constexpr (STYLE != 0) {
          y[ia] = fmaf(v[ia], c[j], -v[ib] * s[j]);
          y[ib] = fmaf(v[ib], c[j], v[ia] * s[j]);
        } else {
          y[ia] = v[ia];
          y[ib] = v[ib];
        }
      }
      if (h < H) {
        __nv_bfloat16* dst = is_q ? qdst + h * p.qos[2] : kdst + (h - p.Hq) * p.kos[2];
        *reinterpret_cast<uint4*>(dst) = pack8(*reinterpret_cast<float(*)[8]>(y));
        *reinterpret_cast<uint4*>(dst + OFF_B) = pack8(*reinterpret_cast<float(*)[8]>(y + 8));
      }
    }
    r0 += U;
    if (r0 >= r1) break;
    load(r0);
  }
}

template <int D>
cudaError_t dispatch_style(const QkNormRopeLaunch& p) {
  constexpr int HPW = 32 / (D / 16);
  const long long tokens = (long long)p.B * p.L;
  const int all = (p.Hq + p.Hkv + HPW - 1) / HPW;  // rounds that cover a token's heads
  // One warp a token once the tokens give every SM's warps work; a round a warp below that (a decode step).
  const int rounds = tokens * all <= 32ll * 1024 ? 1 : all;
  const int chunks = (all + rounds - 1) / rounds;
  const long long blocks = (tokens * chunks + kNormWarps - 1) / kNormWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.rope.style == 1)
    qk_norm_rope_kernel<D, 1><<<(unsigned)blocks, 32 * kNormWarps, 0, p.stream>>>(p, chunks, rounds);
  else if (p.rope.style == 2)
    qk_norm_rope_kernel<D, 2><<<(unsigned)blocks, 32 * kNormWarps, 0, p.stream>>>(p, chunks, rounds);
  else
    qk_norm_rope_kernel<D, 0><<<(unsigned)blocks, 32 * kNormWarps, 0, p.stream>>>(p, chunks, rounds);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& p) {
  if ((long long)p.B * p.L == 0) return cudaSuccess;
  return p.D == 64 ? dispatch_style<64>(p) : dispatch_style<128>(p);
}

}  // namespace attn
