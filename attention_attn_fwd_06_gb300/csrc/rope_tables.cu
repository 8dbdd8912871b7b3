// rope_tables.cu -- rotary tables: row r holds cos and sin of (start + r) f_i for every pair i, times an amplitude.
//
// A pair's frequency comes in turns a position, as a 64-bit binary fraction F = round(2^64 f / 2 pi): the product with the
// position, modulo 2^64, is the angle's fraction of a turn without rounding, whatever the position, where a product in
// 32 bits would be off by whole radians (2^20 positions of a first pair: 2^-4 of a radian) and one in 64-bit floats runs at
// a fiftieth of the rate.  F's own rounding moves the angle of position p by p 2^-65 turns, the host's 64-bit f by p 2^-53
// of its size.  The fraction's nearest quarter turn picks which of sin and cos is which, and its sign; the rest, at most an
// eighth of a turn, is rounded to fp32 (2^-24 of itself) before its sine and cosine.
//
// What bounds it: the writes, 8 bytes a pair.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kTableThreads = 256;
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

// sin and cos of `phase` / 2^64 turns
__device__ __forceinline__ void sincos_turns(unsigned long long phase, float& s, float& c) {
  const unsigned quarter = (unsigned)((phase + (1ull << 61)) >> 62);
  const long long rest = (long long)(phase - ((unsigned long long)quarter << 62));  // in [-2^61, 2^61)
  // in half turns; the two halves' sum is rounded once (the low one's own rounding is 2^-24 of 2^-31 of an eighth turn)
  const float x = fmaf((float)(int)(rest >> 32), 0x1p-31f, (float)(unsigned)rest * 0x1p-63f);
  float ss, cc;
  sincospif(x, &ss, &cc);
  const bool swap = quarter & 1;
  const float a = swap ? cc : ss, b = swap ? ss : cc;
  s = (quarter & 2) ? -a : a;
  c = ((quarter + 1) & 2) ? -b : b;
}

__global__ void __launch_bounds__(kTableThreads) rope_tables_kernel(const TableArgs a) {
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
    for (int j = 0; j < kTablePairs; ++j) {
      sincos_turns(phase[j], s[j], c[j]);
      phase[j] += step[j];
    }
    const size_t at = (size_t)r * a.pairs + kTablePairs * g;
    const float m = a.amplitude;
    *reinterpret_cast<float4*>(a.cos + at) = make_float4(c[0] * m, c[1] * m, c[2] * m, c[3] * m);
    *reinterpret_cast<float4*>(a.sin + at) = make_float4(s[0] * m, s[1] * m, s[2] * m, s[3] * m);
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
  const long long most = (long long)p.num_sms * 8;
  rope_tables_kernel<<<(unsigned)(need < most ? need : most), kTableThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
