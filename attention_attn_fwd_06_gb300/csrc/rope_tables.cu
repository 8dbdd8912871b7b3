// rope_tables.cu -- rotary tables: row r holds cos and sin of (start + r) f_i for every pair i, times an amplitude.
//
// A pair's frequency comes in turns a position, as a 64-bit binary fraction F = round(2^64 f / 2 pi): the product with the
// position, modulo 2^64, is the angle's fraction of a turn without rounding, whatever the position, where a product in
// 32 bits would be off by 2^-4 of a radian at position 2^20 of a first pair (by 2^6 near 2^31) and one in 64-bit floats runs at
// a fiftieth of the rate.  F's own rounding moves the angle of position p by p 2^-65 turns, the host's 64-bit f by p 2^-51
// of its size.  The fraction's nearest quarter turn picks which of sin and cos is which, and its sign; the rest, at most an
// eighth of a turn, is rounded to fp32 (2^-24 of itself) before polynomials give its sine and cosine.
//
// What bounds it: the writes, 8 bytes a pair, and closely behind them the arithmetic.  131,072 rows of 64 pairs take 11.8 us (5.7
// TB/s; 10.1 at the copy bandwidth), 4096 rows 2.5.  CUDA's sincospif for a pair at a time and two conversions: 17.8 us; eight
// blocks an SM, of which five fit at once: 12.0 us, as many as fit at 32 registers 13.5.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kTableThreads = 256;
constexpr int kTableBlocks = 5;  // an SM
constexpr int kTablePairs = 4;  // of one row, a thread

struct TableArgs {
  float* cos;
  float* sin;
  int rows, start, pairs;
  int groups;     // pairs / kTablePairs
  int block_rows; // rows that a block's threads cover at once
  float amplitude;
  unsigned long long turn[kMaxRotaryPairs];
};

// Sine and cosine of half turns x in [-1/4, 1/4], two at a time: x (s0 + s1 z + s2 z^2 + s3 z^3) and 1 + c0 z + .. + c3 z^4
// with z = x^2, coefficients fitted by Lawson's reweighted least squares at 400 Chebyshev nodes of z (relative 3.2e-9 of
// the sine, 5.4e-11 of the cosine before rounding); in fp32 within 9.0e-8 and 5.8e-8 over 2,000,001 points.
__device__ __forceinline__ void sincos_half_turns(float2 x, float2& s, float2& c) {
  auto two = [](float v) { return make_float2(v, v); };
  const float2 z = __fmul2_rn(x, x);
  float2 p = __ffma2_rn(two(-0x1.2d92ep-1f), z, two(0x1.465e92p+1f));
  p = __ffma2_rn(p, z, two(-0x1.4abbb8p+2f));
  p = __ffma2_rn(p, z, two(0x1.921fb6p+1f));
  s = __fmul2_rn(p, x);
  float2 q = __ffma2_rn(two(0x1.d9f788p-3f), z, two(-0x1.55c664p+0f));
  q = __ffma2_rn(q, z, two(0x1.03c1dep+2f));
  q = __ffma2_rn(q, z, two(-0x1.3bd3ccp+2f));
  c = __ffma2_rn(q, z, two(1.f));
}

// `phase` / 2^64 turns as a quarter turn (its low two bits) and a rest of at most an eighth of a turn, in half turns: 32 of the
// rest's 62 bits (2^-35 of a turn), by one conversion.
__device__ __forceinline__ float split_phase(unsigned long long phase, unsigned& quarter) {
  const unsigned hi = (unsigned)(phase >> 32);
  quarter = (hi + (1u << 29)) >> 30;
  return (float)(int)__funnelshift_l((unsigned)phase, hi, 2) * 0x1p-33f;  // (the quarter's bits leave at the top)
}

__global__ void __launch_bounds__(kTableThreads, kTableBlocks) rope_tables_kernel(const TableArgs a) {
  const int r0 = threadIdx.x / a.groups, g = threadIdx.x - r0 * a.groups;
  if (r0 >= a.block_rows) return;
  unsigned long long f[kTablePairs], phase[kTablePairs], step[kTablePairs];
  const long long first = (long long)blockIdx.x * a.block_rows + r0;
  const long long stride = (long long)gridDim.x * a.block_rows;
#pragma unroll
  for (int j = 0; j < kTablePairs; ++j) {
    f[j] = a.turn[kTablePairs * g + j];
    phase[j] = f[j] * (unsigned long long)(a.start + first);
    step[j] = f[j] * (unsigned long long)stride;
  }
  for (long long r = first; r < a.rows; r += stride) {
    float s[kTablePairs], c[kTablePairs];
#pragma unroll
    for (int j = 0; j < kTablePairs; j += 2) {
      unsigned quarter[2];
      float2 x, ss, cc;
      x.x = split_phase(phase[j], quarter[0]);
      x.y = split_phase(phase[j + 1], quarter[1]);
      phase[j] += step[j];
      phase[j + 1] += step[j + 1];
      sincos_half_turns(x, ss, cc);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const unsigned t = quarter[k];
        const float sn = k ? ss.y : ss.x, cs = k ? cc.y : cc.x;
        const unsigned amp = __float_as_uint(a.amplitude);
        s[j + k] = ((t & 1) ? cs : sn) * __uint_as_float(amp ^ ((t & 2) << 30));
        c[j + k] = ((t & 1) ? sn : cs) * __uint_as_float(amp ^ (((t + 1) & 2) << 30));
      }
    }
    const size_t at = (size_t)r * a.pairs + kTablePairs * g;
    *reinterpret_cast<float4*>(a.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(a.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

}  // namespace

cudaError_t launch_rope_tables(const RopeTablesLaunch& p) {
  if (p.rows <= 0) return cudaSuccess;
  TableArgs a;
  a.cos = p.cos;
  a.sin = p.sin;
  a.rows = p.rows;
  a.start = p.start;
  a.pairs = p.pairs;
  a.groups = p.pairs / kTablePairs;
  a.block_rows = kTableThreads / a.groups;
  a.amplitude = p.amplitude;
  for (int i = 0; i < kMaxRotaryPairs; ++i) a.turn[i] = i < p.pairs ? p.turn[i] : 0;
  const long long need = ((long long)p.rows + a.block_rows - 1) / a.block_rows;
  const long long most = (long long)p.num_sms * kTableBlocks;
  rope_tables_kernel<<<(unsigned)(need < most ? need : most), kTableThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
