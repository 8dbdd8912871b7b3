// qk_norm_rope.cu -- RMS norm of every query and key head with the position rotation in the same pass.
//
// For each head row x of D elements: y = x * rsqrt(mean(x^2) + eps) * w, then pair i of y at the token's position p,
// (a, b), becomes (a cos - b sin, b cos + a sin) with cos, sin from row p of the caller's fp32 tables; pairs are
// (i, i + D/2) or (2i, 2i + 1).  All in fp32, rounded to bf16 once at the end.
//
// What bounds it: HBM.  Every element is read once (2 bytes) and written once (2 bytes).  A lane holds 16 elements --
// eight whole pairs -- of a head, D/16 lanes a head, so the sum of squares takes three (two) shuffles and the
// rotation none; a warp takes one token's heads four (eight) at a time, a round.  The table values of a token are twice the
// bytes of a head and come after its position, two round trips to memory, so a warp takes a run of tokens, as many as make
// one wave of the grid: it reads the run's positions at once, brings the next token's table rows into shared memory while
// it works on this one's, and loads a round's heads two rounds ahead, across tokens.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace attn {
namespace {

// 4 warps a block, 5 blocks an SM (96 registers, 20 warps), two rounds in flight: 65,536 tokens of 32 + 8 heads at D = 128
// take 218 us (6.2 TB/s, 0.91 of the copy bandwidth), 8,158 of 16 + 16 heads at D = 64 15.4 us; 16 warps an SM: 234 and
// 16.9 us (three or four rounds in flight: 229 to 242 us), 24 warps that spill: 231 and 18.8 us.  One round a lane and
// as many warps as fit, no runs of tokens: 306 and 18.9 us (table rows through L1 bound it).
constexpr int kNormWarps = 4;
constexpr int kNormBlocks = 5;

// A warp takes `tokens` tokens and `rounds` of each one's rounds; `chunks` warps share a token (1 unless tokens is 1).
struct NormShare {
  int tokens, rounds, chunks;
};

// STYLE 0: no rotation, 1: pairs (i, i + D/2), 2: pairs (2i, 2i + 1).
template <int D, int STYLE>
__global__ void __launch_bounds__(32 * kNormWarps, kNormBlocks)
    qk_norm_rope_kernel(const QkNormRopeLaunch p, const NormShare share) {
  constexpr int TPR = D / 16;    // lanes per head
  constexpr int HPW = 32 / TPR;  // heads per round
  constexpr int U = 2;           // rounds in flight
  constexpr int OFF_B = D / 2;   // from a lane's first 8 elements to its other 8 (whole sectors for a warp's accesses)
  __shared__ __align__(16) float tables[kNormWarps][2][STYLE != 0 ? D : 4];  // cos row, sin row of two tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long job = (long long)blockIdx.x * kNormWarps + warp;
  const long long t0 = share.chunks == 1 ? job * share.tokens : job / share.chunks;
  const long long left = (long long)p.B * p.L - t0;
  if (left <= 0) return;
  const int ntok = left < share.tokens ? (int)left : share.tokens;
  const int sub = lane % TPR;
  const int d0 = 8 * sub;  // the lane's first element
  const int H = p.Hq + p.Hkv;
  const int rbase = share.chunks == 1 ? 0 : (int)(job - t0 * share.chunks) * share.rounds;
  const int h0 = rbase * HPW + lane / TPR;
  const int rounds = min(share.rounds, (H + HPW - 1) / HPW - rbase);  // (>= 1)
  // lane i: the position of token t0 + i (-1 pads; anything else out of range is an error: its row is left alone)
  int pos_l = -1;
  if (lane < ntok) {
    pos_l = p.positions != nullptr ? p.positions[t0 + lane] : 0;
    if (pos_l < 0 || (STYLE != 0 && pos_l >= p.rope.max_pos)) {
      if (pos_l != -1) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
      pos_l = -1;
    }
  }
  // element offset of head h of token t0 + tk, from strides st
  auto row_at = [&](const long long (&st)[3], int tk, int h) -> long long {
    const long long t = t0 + tk;
    if (p.B == 1) return t * st[1] + h * st[2] + d0;
    const long long b = t / p.L;
    return b * st[0] + (t - b * p.L) * st[1] + h * st[2] + d0;
  };
  uint4 x[U][2];
  auto load = [&](int u, int tk, int r) {
    const int h = h0 + r * HPW;
    x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
    if (tk < ntok && r < rounds && h < H) {
      const __nv_bfloat16* src = h < p.Hq ? reinterpret_cast<const __nv_bfloat16*>(p.q) + row_at(p.qs, tk, h)
                                          : reinterpret_cast<const __nv_bfloat16*>(p.k) + row_at(p.ks, tk, h - p.Hq);
      x[u][0] = *reinterpret_cast<const uint4*>(src);
      x[u][1] = *reinterpret_cast<const uint4*>(src + OFF_B);
    }
  };
  // The table rows of token tk on their way to buffer tk & 1 (16 bytes a lane).
  auto fetch_tables = [&](int tk) {
    if constexpr (STYLE != 0) {
      const int pos = __shfl_sync(0xffffffffu, pos_l, tk & 31);
      if (tk < ntok && pos >= 0 && lane < D / 4) {
        const float* src = (lane < D / 8 ? p.rope.cos : p.rope.sin) + (size_t)pos * (D / 2) + 4 * (lane % (D / 8));
        cp_async16(&tables[warp][tk & 1][4 * lane], src);
      }
      cp_async_commit();
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, 0, u);
  fetch_tables(0);
  for (int tk = 0; tk < ntok; ++tk) {
    const bool live = __shfl_sync(0xffffffffu, pos_l, tk) >= 0;
    float c[8], s[8];
    if constexpr (STYLE != 0) {
      __syncwarp();  // the buffer's last readers are done
      fetch_tables(tk + 1);
      cp_async_wait<1>();
      __syncwarp();
      // the lane's eight pairs: 8 sub .., or four from each of its runs of elements
      constexpr int NEXT = STYLE == 1 ? 1 : D / 16;
      const float4* tab = reinterpret_cast<const float4*>(tables[warp][tk & 1] + (STYLE == 1 ? 8 : 4) * sub);
      *reinterpret_cast<float4*>(c) = tab[0];
      *reinterpret_cast<float4*>(c + 4) = tab[NEXT];
      *reinterpret_cast<float4*>(s) = tab[D / 8];
      *reinterpret_cast<float4*>(s + 4) = tab[D / 8 + NEXT];
    }
    for (int r0 = 0; r0 < rounds; r0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u;
        if (r >= rounds) break;  // warp-uniform
        const int h = h0 + r * HPW;
        float v[16];
        unpack8(x[u][0], *reinterpret_cast<float(*)[8]>(v));
        unpack8(x[u][1], *reinterpret_cast<float(*)[8]>(v + 8));
        if (r + U < rounds) load(u, tk, r + U); else load(u, tk + 1, u);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
        for (int mask = 1; mask < TPR; mask <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, mask);
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        const bool is_q = h < p.Hq;
        const __nv_bfloat16* weight = reinterpret_cast<const __nv_bfloat16*>(is_q ? p.q_weight : p.k_weight);
        if (weight != nullptr) {  // (from L1: held in registers they would cost a quarter of the warps)
          float w[16];
          unpack8(__ldg(reinterpret_cast<const uint4*>(weight + d0)), *reinterpret_cast<float(*)[8]>(w));
          unpack8(__ldg(reinterpret_cast<const uint4*>(weight + d0 + OFF_B)), *reinterpret_cast<float(*)[8]>(w + 8));
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] *= inv * w[j];
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] *= inv;
        }
        if constexpr (STYLE != 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int ia = STYLE == 1 ? j : 2 * j, ib = STYLE == 1 ? j + 8 : 2 * j + 1;
            const float a = v[ia], b = v[ib];
            v[ia] = fmaf(a, c[j], -b * s[j]);
            v[ib] = fmaf(b, c[j], a * s[j]);
          }
        }
        if (live && h < H) {
          __nv_bfloat16* dst = is_q ? reinterpret_cast<__nv_bfloat16*>(p.q_out) + row_at(p.qos, tk, h)
                                    : reinterpret_cast<__nv_bfloat16*>(p.k_out) + row_at(p.kos, tk, h - p.Hq);
          *reinterpret_cast<uint4*>(dst) = pack8(*reinterpret_cast<float(*)[8]>(v));
          *reinterpret_cast<uint4*>(dst + OFF_B) = pack8(*reinterpret_cast<float(*)[8]>(v + 8));
        }
      }
    }
  }
  if constexpr (STYLE != 0) cp_async_wait<0>();
}

template <int D>
cudaError_t dispatch_style(const QkNormRopeLaunch& p) {
  constexpr int HPW = 32 / (D / 16);
  const long long tokens = (long long)p.B * p.L;
  const int all = (p.Hq + p.Hkv + HPW - 1) / HPW;  // rounds that cover a token's heads
  const long long warps = (long long)kNormBlocks * kNormWarps * p.num_sms;
  const long long per = (tokens + warps - 1) / warps;
  NormShare share;
  share.tokens = (int)(per > 32 ? 32 : per);  // a lane holds a position
  const long long parts = share.tokens > 1 ? 1 : warps / tokens;  // few tokens (a decode step): several warps for each
  share.chunks = (int)(parts < 1 ? 1 : parts < all ? parts : all);
  share.rounds = (all + share.chunks - 1) / share.chunks;
  share.chunks = (all + share.rounds - 1) / share.rounds;
  const long long jobs = (tokens + share.tokens - 1) / share.tokens * share.chunks;
  const long long blocks = (jobs + kNormWarps - 1) / kNormWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.rope.style == 1)
    qk_norm_rope_kernel<D, 1><<<(unsigned)blocks, 32 * kNormWarps, 0, p.stream>>>(p, share);
  else if (p.rope.style == 2)
    qk_norm_rope_kernel<D, 2><<<(unsigned)blocks, 32 * kNormWarps, 0, p.stream>>>(p, share);
  else
    qk_norm_rope_kernel<D, 0><<<(unsigned)blocks, 32 * kNormWarps, 0, p.stream>>>(p, share);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& p) {
  if ((long long)p.B * p.L == 0) return cudaSuccess;
  return p.D == 64 ? dispatch_style<64>(p) : dispatch_style<128>(p);
}

}  // namespace attn
