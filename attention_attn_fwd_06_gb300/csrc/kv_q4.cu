// kv_q4.cu -- writing rows into the 4-bit KV cache, and reading them back (layout: kv_q4.h).
//
// A group is 64 consecutive dims of one key's (value's) row.  With m = fp16(min x) and s = fp16((max x - min x) / 15)
// its codes are u = clamp(round((x - m) / s), 0, 15), ties to even, and a code reads back as s * u + m.  Scale and
// minimum are held in fp16: eleven bits, so that a code's step is off by 2^-12 at most against the step's half that
// the four bits themselves cost.  NaN is stored as 0, values beyond fp16's range as its largest.
//
// What bounds both: HBM.  Writing takes 2 bytes in and 0.5625 out per element, reading back the reverse.  A thread
// takes 16 dims (32 bytes of bf16, 8 bytes of codes), so four lanes hold a group and its extremes take two shuffles.
//
// The rounding is decided without a division: k = floor of the approximate quotient brackets it, and the sign of
// x - m - (k + 1/2) s, one fused multiply-add over an exact product, says whether k or k + 1 is nearer.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "kv_q4.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr float kF16Max = 65504.f;

template <int D>
__global__ void __launch_bounds__(256) kv_append_q4_kernel(const KvAppendQ4Launch p, long long threads) {
  constexpr int G = D / 64, TPR = D / 16;
  const long long tid = (long long)blockIdx.x * 256 + threadIdx.x;
  if (tid >= threads) return;  // whole rows: a multiple of TPR threads
  const int sub = (int)(tid % TPR);
  const long long row = tid / TPR;  // (token, K then V, head)
  const int heads2 = 2 * p.Hkv;
  const long long tok = row / heads2;
  const int hh = (int)(row - tok * heads2);
  const bool is_v = hh >= p.Hkv;
  const int h = is_v ? hh - p.Hkv : hh;
  const int slot = p.slots[tok];
  const bool live = slot >= 0 && slot < p.num_pages * p.page_size;
  if (!live && slot != -1 && sub == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
  const __nv_bfloat16* src = is_v ? reinterpret_cast<const __nv_bfloat16*>(p.v) + tok * p.vs[0] + h * p.vs[1]
                                  : reinterpret_cast<const __nv_bfloat16*>(p.k) + tok * p.ks[0] + h * p.ks[1];
  float x[16];
  unpack8(*reinterpret_cast<const uint4*>(src + 16 * sub), *reinterpret_cast<float(*)[8]>(x));
  unpack8(*reinterpret_cast<const uint4*>(src + 16 * sub + 8), *reinterpret_cast<float(*)[8]>(x + 8));
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    x[j] = x[j] == x[j] ? fminf(fmaxf(x[j], -kF16Max), kF16Max) : 0.f;
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
  const unsigned team = 0xfu << (threadIdx.x & 28);  // the group's four lanes (rows end on a multiple of four)
#pragma unroll
  for (int mask = 1; mask < 4; mask <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(team, lo, mask));
    hi = fmaxf(hi, __shfl_xor_sync(team, hi, mask));
  }
  if (!live) return;
  const __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f)), mh = __float2half_rn(lo);
  const float s = __half2float(sh), m = __half2float(mh);
  const float inv = s > 0.f ? 1.f / s : 0.f;
  unsigned w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float t = x[j] - m;
    const float k = fminf(fmaxf(floorf(t * inv), 0.f), 14.f);
    const float e = fmaf(-(k + 0.5f), s, t);
    const int ki = (int)k;
    const int u = ki + ((e > 0.f || (e == 0.f && (ki & 1))) ? 1 : 0);
    w[j / 8] |= (unsigned)u << (4 * (j % 8));
  }
  if (!(s > 0.f)) w[0] = w[1] = 0;
  const int page = slot / p.page_size, in_page = slot - page * p.page_size;
  const int tile = in_page / kTileKeys, key = in_page - tile * kTileKeys;
  uint8_t* dst = reinterpret_cast<uint8_t*>(p.pool) + kv_q4_tile_at(page, h, tile, p.Hkv, p.page_size / kTileKeys, D);
  const int g = sub / 4;
  *reinterpret_cast<uint2*>(dst + (is_v ? kv_q4_v_off(D) : 0) + (g * kTileKeys + key) * 32 + (sub % 4) * 8) =
      make_uint2(w[0], w[1]);
  if (sub % 4 == 0)
    *reinterpret_cast<__half2*>(dst + (is_v ? kv_q4_vp_off(D) : kv_q4_kp_off(D)) + (key * G + g) * 4) =
        __halves2half2(sh, mh);
}

__device__ __forceinline__ void codes_to_bf16(uint2 w, __half2 par, __nv_bfloat16* dst) {
  const float s = __low2float(par), m = __high2float(par);
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = fmaf(s, (float)(((j < 8 ? w.x : w.y) >> (4 * (j % 8))) & 15u), m);
  *reinterpret_cast<uint4*>(dst) = pack8(*reinterpret_cast<float(*)[8]>(x));
  *reinterpret_cast<uint4*>(dst + 8) = pack8(*reinterpret_cast<float(*)[8]>(x + 8));
}

template <int D>
__global__ void __launch_bounds__(256) kv_gather_q4_kernel(const KvGatherQ4Launch p, long long threads) {
  constexpr int G = D / 64, TPR = D / 16;
  const long long tid = (long long)blockIdx.x * 256 + threadIdx.x;
  if (tid >= threads) return;
  const int sub = (int)(tid % TPR);
  const long long row = tid / TPR;  // (token, head)
  const long long tok = row / p.Hkv;
  const int h = (int)(row - tok * p.Hkv);
  if (tok >= p.cu_k[p.B] || tok < p.cu_k[0]) return;  // rows of no sequence stay as they were
  int lo = 0, hi = p.B;  // the sequence with cu[s] <= tok < cu[s + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_k[mid] <= tok) lo = mid; else hi = mid;
  }
  const long long pos = tok - p.cu_k[lo] + (p.kv_starts != nullptr ? p.kv_starts[lo] : 0);
  const long long pg = pos >= 0 ? pos / p.page_size : -1;
  int page = -1;
  if (pg >= 0 && pg < p.max_pages) page = p.block_table[(size_t)lo * p.max_pages + pg];
  if (page < 0 || page >= p.num_pages) {  // the row stays as it was
    if (sub == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    return;
  }
  const int in_page = (int)(pos - pg * p.page_size);
  const int tile = in_page / kTileKeys, key = in_page - tile * kTileKeys;
  const uint8_t* src =
      reinterpret_cast<const uint8_t*>(p.pool) + kv_q4_tile_at(page, h, tile, p.Hkv, p.page_size / kTileKeys, D);
  const int g = sub / 4;
  const int code = (g * kTileKeys + key) * 32 + (sub % 4) * 8, par = (key * G + g) * 4;
  const uint2 wk = *reinterpret_cast<const uint2*>(src + code);
  const uint2 wv = *reinterpret_cast<const uint2*>(src + kv_q4_v_off(D) + code);
  const __half2 pk = *reinterpret_cast<const __half2*>(src + kv_q4_kp_off(D) + par);
  const __half2 pv = *reinterpret_cast<const __half2*>(src + kv_q4_vp_off(D) + par);
  const size_t at = (size_t)row * D + 16 * sub;
  codes_to_bf16(wk, pk, reinterpret_cast<__nv_bfloat16*>(p.k) + at);
  codes_to_bf16(wv, pv, reinterpret_cast<__nv_bfloat16*>(p.v) + at);
}

}  // namespace

cudaError_t launch_kv_append_q4(const KvAppendQ4Launch& p) {
  const long long threads = (long long)p.T * 2 * p.Hkv * (p.D / 16);
  if (threads == 0) return cudaSuccess;
  const long long blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.D == 64)
    kv_append_q4_kernel<64><<<(unsigned)blocks, 256, 0, p.stream>>>(p, threads);
  else
    kv_append_q4_kernel<128><<<(unsigned)blocks, 256, 0, p.stream>>>(p, threads);
  return cudaGetLastError();
}

cudaError_t launch_kv_gather_q4(const KvGatherQ4Launch& p) {
  const long long threads = (long long)p.total_k * p.Hkv * (p.D / 16);
  if (threads == 0) return cudaSuccess;
  const long long blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.D == 64)
    kv_gather_q4_kernel<64><<<(unsigned)blocks, 256, 0, p.stream>>>(p, threads);
  else
    kv_gather_q4_kernel<128><<<(unsigned)blocks, 256, 0, p.stream>>>(p, threads);
  return cudaGetLastError();
}

}  // namespace attn
