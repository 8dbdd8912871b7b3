// kv_append_paged.cu -- rows of k and v into the pages of a bf16 cache, with the position rotation of k, and of q, on the way.
//
// Pair i of the first R dims of a head of k (and of q) at the token's position p, (a, b), becomes (a cos - b sin,
// b cos + a sin) with cos, sin from row p of the caller's fp32 tables [max_pos, R/2]; pairs are dims (i, i + R/2) or
// (2i, 2i + 1); the other dims, and v, are copied.  In fp32, rounded to bf16 once.
//
// What bounds it: HBM.  Every element is read once (2 bytes) and written once.  A lane holds two chunks of eight dims of a
// head -- eight whole pairs, or dims that are copied -- so that its eight pairs' table values stay in registers for all of
// a token's heads.  Table rows come after the position, two round trips to memory, so a warp takes a run of tokens, as many
// as make one wave of the grid, reads the run's positions and slots at once, brings the next token's table rows into shared
// memory while it works on this one's, and loads a round's heads two rounds ahead, across tokens.
// 65,536 tokens of 32 + 8 heads at D = 128 take 256 us (6.3 TB/s, 0.95 of the copy bandwidth), 8,158 of 16 + 16 heads at D = 64
// with half of each turned 19.7 us (5.1 TB/s), 8 tokens 2.4.  Six blocks an SM: 274 and 19.3 us; three rounds in flight: 259 and
// 20.2.
#include <cuda_bf16.h>

#include "common.cuh"
#include "intdiv.h"
#include "kernels.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kAppendBlocks = 5;

struct AppendArgs {
  KvAppendPagedLaunch p;
  FastDiv page;
  int tokens;  // of a warp
  int chunks;  // warps that share a token (1 unless tokens is 1)
  int rounds;  // of a token's rounds that a warp takes
};

// STYLE 0: no rotation, 1: pairs (i, i + R/2), 2: pairs (2i, 2i + 1).
template <int D, int STYLE>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendBlocks) kv_append_paged_kernel(const AppendArgs a) {
  constexpr int TPR = D / 16;    // lanes per head
  constexpr int HPW = 32 / TPR;  // heads per round
  constexpr int U = 2;           // rounds in flight
  const KvAppendPagedLaunch& p = a.p;
  __shared__ __align__(16) float tables[kAppendWarps][2][STYLE != 0 ? D : 4];  // cos row, sin row of two tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long job = (long long)blockIdx.x * kAppendWarps + warp;
  const long long t0 = a.chunks == 1 ? job * a.tokens : job / a.chunks;
  const long long left = (long long)p.T - t0;
  if (left <= 0) return;
  const int ntok = left < a.tokens ? (int)left : a.tokens;
  const int sub = lane % TPR;
  // the lane's chunks of eight dims
  int ca = sub, cb = sub + TPR;
  const int rot = p.rotary / 16;  // STYLE 1: lanes of a head that rotate
  if (STYLE == 1) {
    ca = sub < rot ? sub : rot + sub;
    cb = sub < rot ? sub + rot : TPR + sub;
  }
  const int da = 8 * ca, db = 8 * cb;
  const int H = p.Hq + 2 * p.Hkv;
  const int rbase = a.chunks == 1 ? 0 : (int)(job - t0 * a.chunks) * a.rounds;
  const int h0 = rbase * HPW + lane / TPR;
  const int rounds = min(a.rounds, (H + HPW - 1) / HPW - rbase);  // (>= 1)
  // lane i: position and slot of token t0 + i (-1: padding; anything else out of range is an error, and nothing is written)
  int pos_l = -1, slot_l = -1;
  if (lane < ntok) {
    pos_l = p.positions != nullptr ? p.positions[t0 + lane] : 0;
    slot_l = p.slots[t0 + lane];
    if (pos_l < 0 || (STYLE != 0 && pos_l >= p.rope.max_pos)) {
      if (pos_l != -1) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
      pos_l = -1;
    }
    if (slot_l < 0 || slot_l >= p.num_pages * p.page_size) {
      if (slot_l != -1) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
      slot_l = -1;
    }
    if (pos_l < 0) slot_l = -1;
  }
  uint4 x[U][2];
  auto load = [&](int u, int tk, int r) {
    const int h = h0 + r * HPW;
    x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
    if (tk < ntok && r < rounds && h < H) {
      const long long t = t0 + tk;
      const __nv_bfloat16* src;
      if (h < p.Hq)
        src = reinterpret_cast<const __nv_bfloat16*>(p.q) + t * p.qs[0] + h * p.qs[1];
      else if (h < p.Hq + p.Hkv)
        src = reinterpret_cast<const __nv_bfloat16*>(p.k) + t * p.ks[0] + (h - p.Hq) * p.ks[1];
      else
        src = reinterpret_cast<const __nv_bfloat16*>(p.v) + t * p.vs[0] + (h - p.Hq - p.Hkv) * p.vs[1];
      x[u][0] = *reinterpret_cast<const uint4*>(src + da);
      x[u][1] = *reinterpret_cast<const uint4*>(src + db);
    }
  };
  // The table rows of token tk on their way to buffer tk & 1 (16 bytes a lane).
  const int quads = p.rotary / 8;  // float4s of a row
  auto fetch_tables = [&](int tk) {
    if constexpr (STYLE != 0) {
      const int pos = __shfl_sync(0xffffffffu, pos_l, tk & 31);
      if (tk < ntok && pos >= 0 && lane < 2 * quads) {
        const bool second = lane >= quads;
        const int i = second ? lane - quads : lane;
        const float* src = (second ? p.rope.sin : p.rope.cos) + (size_t)pos * (p.rotary / 2) + 4 * i;
        cp_async16(&tables[warp][tk & 1][(second ? D / 2 : 0) + 4 * i], src);
      }
      cp_async_commit();
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, 0, u);
  fetch_tables(0);
  for (int tk = 0; tk < ntok; ++tk) {
    const bool live = __shfl_sync(0xffffffffu, pos_l, tk) >= 0;
    const int slot = __shfl_sync(0xffffffffu, slot_l, tk);
    const unsigned page = slot >= 0 ? a.page.div((unsigned)slot) : 0u;
    const int off = slot - (int)(page * a.page.d);
    // first element of this token's row of kv head 0 in the pools; a head is page_size * D further
    const long long cache = ((long long)page * p.Hkv * p.page_size + off) * D;
    float c[8], s[8];
    bool turn_a = false, turn_b = false;
    if constexpr (STYLE != 0) {
      __syncwarp();  // the buffer's last readers are done
      fetch_tables(tk + 1);
      cp_async_wait<1>();
      __syncwarp();
      const float* tab = tables[warp][tk & 1];
      if (STYLE == 1) {
        turn_a = turn_b = sub < rot;  // chunk ca with chunk cb: pairs 8 sub ..
      } else {
        turn_a = ca < 2 * rot;  // four pairs from each chunk: 4 ca .., 4 cb ..
        turn_b = cb < 2 * rot;
      }
      const int ia = STYLE == 1 ? 8 * sub : 4 * ca, ib = STYLE == 1 ? 8 * sub + 4 : 4 * cb;
      if (turn_a) {
        *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(tab + ia);
        *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(tab + D / 2 + ia);
      }
      if (turn_b) {
        *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(tab + ib);
        *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(tab + D / 2 + ib);
      }
    }
    for (int r0 = 0; r0 < rounds; r0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u;
        if (r >= rounds) break;  // warp-uniform
        const int h = h0 + r * HPW;
        uint4 y0 = x[u][0], y1 = x[u][1];
        if (r + U < rounds) load(u, tk, r + U); else load(u, tk + 1, u);
        if (h >= H || !live) continue;
        const bool is_v = h >= p.Hq + p.Hkv;
        if (STYLE != 0 && !is_v) {
          float va[8], vb[8];
          unpack8(y0, va);
          unpack8(y1, vb);
          if constexpr (STYLE == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float e = va[j], f = vb[j];
              va[j] = fmaf(e, c[j], -f * s[j]);
              vb[j] = fmaf(f, c[j], e * s[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float e = va[2 * j], f = va[2 * j + 1];
              va[2 * j] = fmaf(e, c[j], -f * s[j]);
              va[2 * j + 1] = fmaf(f, c[j], e * s[j]);
              e = vb[2 * j];
              f = vb[2 * j + 1];
              vb[2 * j] = fmaf(e, c[4 + j], -f * s[4 + j]);
              vb[2 * j + 1] = fmaf(f, c[4 + j], e * s[4 + j]);
            }
          }
          if (turn_a) y0 = pack8(va);  // (dims that do not turn keep their bits, NaN and infinities among them)
          if (turn_b) y1 = pack8(vb);
        }
        const long long t = t0 + tk;
        if (h < p.Hq) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.q_out) + t * p.qos[0] + h * p.qos[1];
          *reinterpret_cast<uint4*>(dst + da) = y0;
          *reinterpret_cast<uint4*>(dst + db) = y1;
        } else {
          const int hk = h - p.Hq - (is_v ? p.Hkv : 0);
          if (slot >= 0) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? p.vpages : p.kpages) + cache +
                                 (long long)hk * p.page_size * D;
            *reinterpret_cast<uint4*>(dst + da) = y0;
            *reinterpret_cast<uint4*>(dst + db) = y1;
          }
          if (!is_v && p.k_out != nullptr) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.k_out) + t * p.kos[0] + hk * p.kos[1];
            *reinterpret_cast<uint4*>(dst + da) = y0;
            *reinterpret_cast<uint4*>(dst + db) = y1;
          }
        }
      }
    }
  }
  if constexpr (STYLE != 0) cp_async_wait<0>();
}

template <int D>
cudaError_t dispatch_style(const KvAppendPagedLaunch& p) {
  constexpr int HPW = 32 / (D / 16);
  const int all = (p.Hq + 2 * p.Hkv + HPW - 1) / HPW;  // rounds that cover a token's heads
  const long long warps = (long long)kAppendBlocks * kAppendWarps * p.num_sms;
  const long long per = (p.T + warps - 1) / warps;
  AppendArgs a;
  a.p = p;
  a.page = make_fast_div((unsigned)p.page_size);
  a.tokens = (int)(per > 32 ? 32 : per);  // a lane holds a position
  const long long parts = a.tokens > 1 ? 1 : warps / p.T;  // few tokens (a decode step): several warps for each
  a.chunks = (int)(parts < 1 ? 1 : parts < all ? parts : all);
  a.rounds = (all + a.chunks - 1) / a.chunks;
  a.chunks = (all + a.rounds - 1) / a.rounds;
  const long long jobs = ((long long)p.T + a.tokens - 1) / a.tokens * a.chunks;
  const long long blocks = (jobs + kAppendWarps - 1) / kAppendWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.rotary == 0)
    kv_append_paged_kernel<D, 0><<<(unsigned)blocks, 32 * kAppendWarps, 0, p.stream>>>(a);
  else if (p.rope.style == 1)
    kv_append_paged_kernel<D, 1><<<(unsigned)blocks, 32 * kAppendWarps, 0, p.stream>>>(a);
  else
    kv_append_paged_kernel<D, 2><<<(unsigned)blocks, 32 * kAppendWarps, 0, p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_paged(const KvAppendPagedLaunch& p) {
  if (p.T == 0) return cudaSuccess;
  return p.D == 64 ? dispatch_style<64>(p) : dispatch_style<128>(p);
}

}  // namespace attn
