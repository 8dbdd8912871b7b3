// kv_q4.cu -- writing rows into the 4-bit KV cache, and reading them back (layout: kv_q4.h).
//
// A group is 64 consecutive dims of one key's (value's) row.  With m = fp16(min x) and s = fp16((max x - min x) / 15)
// its codes are u = clamp(round((x - m) / s), 0, 15), ties to even, and a code reads back as s * u + m.  Scale and
// minimum are held in fp16: eleven bits, so that each is off by 2^-11 of itself at most, against the half of a step that the
// four bits themselves cost.  Below 2^-14 fp16 has fewer bits: the scale of a group whose range is below 9.2e-4 is a multiple
// of 2^-24, and with a range below 4.5e-7 it is 0 and the minimum stands for all.  NaN is stored as 0, values beyond fp16's
// range as its largest.
//
// What bounds both: HBM, once the arithmetic is short.  Writing takes 2 bytes in and 0.5625 out per element, reading
// back the reverse.  A lane takes 16 dims (32 bytes of bf16, 8 bytes of codes) of one head's key and of its value, so four
// lanes hold a group, its extremes take two shuffles and the row's place is looked up once for both; as many warps as fit.
// 70k tokens of 8 heads at D = 128 take 66 us to write (5.6 TB/s) and 60 us to read back (6.2 TB/s).  Each lane's 32 bytes are
// one access where rows start on 32 bytes: as two of 16, each store fills half a sector, and reading back takes 73 us (a fill
// of 290 MB that way 76 against 42 us), writing 67 against 64 that day.  A key's or a value's dims a lane: 89 us to write; a
// warp for each token and two rounds of its heads in flight (with the slower codes of that day): 113 and 79 us; one wave of
// warps that walk runs of tokens: 124 and 111 us; warps of four tokens of one head: 65.7 and 59.4 us.
//
// Writing: extremes by packed bf16 min and max that pass NaN on; quotients correctly rounded, by a product with the
// rounded reciprocal and its residual's share (Markstein's theorem), so that a tie between two codes is seen as one; their
// rounding is that of an add of 1.5 2^23, whose low bits are the code (a conversion instruction runs at an eighth of the
// rate); all of it in packed pairs.  Issue-bound with floor, conversions and a decision by residual: 166 us, and 112 us with
// the residual only checked, which bf16's coarse values tie too often for.  A group whose codes or values leave
// their range (NaN, infinities, a scale of 0, a minimum that fp16 rounds) is decided code by code.
// Reading: a code masked in place in a 16-bit half is, as fp16, the subnormal u 2^-24 or u 2^-20, so the conversion to
// fp32 and one fused multiply-add with the scale make the value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "intdiv.h"
#include "kernels.h"
#include "kv_q4.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr float kF16Max = 65504.f;
constexpr int kKvThreads = 256;

// The codes of 16 dims, decided one by one (u_j = the nearest code, ties to even, in 0..15).
__device__ __noinline__ uint2 quantise_slow(uint4 w0, uint4 w1, float s, float m) {
  float x[16];
  unpack8(w0, *reinterpret_cast<float(*)[8]>(x));
  unpack8(w1, *reinterpret_cast<float(*)[8]>(x + 8));
  unsigned out[2] = {0, 0};
  if (!(s > 0.f)) return make_uint2(0, 0);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float v = x[j] == x[j] ? fminf(fmaxf(x[j], -kF16Max), kF16Max) : 0.f;
    const float t = v - m;
    const float b = t - v, rest = (v - (t - b)) + (-m - b);  // v - m = t + rest exactly (Knuth's two-sum)
    const float k = fminf(fmaxf(floorf(t / s), 0.f), 14.f);
    const float e = fmaf(-(k + 0.5f), s, t);  // above or below the border (16 bits, so t is not rounded across it), or on it:
    const int ki = (int)k;                    // then the rest decides, and where there is none the tie goes to the even code
    const bool up = e > 0.f || (e == 0.f && (rest > 0.f || (rest == 0.f && (ki & 1))));
    out[j / 8] |= (unsigned)(ki + (up ? 1 : 0)) << (4 * (j % 8));
  }
  return make_uint2(out[0], out[1]);
}

// Extremes of a group with NaN as 0 and values beyond fp16's range as its largest (one lane's 16 dims).
__device__ __noinline__ float2 extremes_slow(uint4 w0, uint4 w1) {
  float x[16];
  unpack8(w0, *reinterpret_cast<float(*)[8]>(x));
  unpack8(w1, *reinterpret_cast<float(*)[8]>(x + 8));
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float v = x[j] == x[j] ? fminf(fmaxf(x[j], -kF16Max), kF16Max) : 0.f;
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  return make_float2(lo, hi);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

struct Quantised {
  uint2 code;
  __half2 pair;  // scale, minimum
};

// One lane's 16 dims wa, wb of a group that the lanes of `team` hold.
__device__ __forceinline__ Quantised quantise(uint4 wa, uint4 wb, unsigned team) {
  const uint32_t q[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
  __nv_bfloat162 mn = as_bf162(q[0]), mx = mn;
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mn = __hmin2_nan(mn, as_bf162(q[j]));
    mx = __hmax2_nan(mx, as_bf162(q[j]));
  }
#pragma unroll
  for (int mask = 1; mask < 4; mask <<= 1) {
    mn = __hmin2_nan(mn, as_bf162(__shfl_xor_sync(team, bits_of(mn), mask)));
    mx = __hmax2_nan(mx, as_bf162(__shfl_xor_sync(team, bits_of(mx), mask)));
  }
  mn = __hmin2_nan(mn, __lowhigh2highlow(mn));
  mx = __hmax2_nan(mx, __lowhigh2highlow(mx));
  float lo = __low2float(mn), hi = __low2float(mx);
  bool odd = !(lo >= -kF16Max) || !(hi <= kF16Max);  // too large, or NaN: the same for the group's four lanes
  if (odd) {
    float2 ex = extremes_slow(wa, wb);
#pragma unroll
    for (int mask = 1; mask < 4; mask <<= 1) {
      ex.x = fminf(ex.x, __shfl_xor_sync(team, ex.x, mask));
      ex.y = fmaxf(ex.y, __shfl_xor_sync(team, ex.y, mask));
    }
    lo = ex.x;
    hi = ex.y;
  }
  // (hi - lo) / 15: a product, and its residual's share added (correctly rounded, as by Markstein's theorem)
  const float d = hi - lo;
  const float d0 = d * (1.f / 15.f);
  const __half sh = __float2half_rn(fmaf(fmaf(-15.f, d0, d), 1.f / 15.f, d0)), mh = __float2half_rn(lo);
  const float s = __half2float(sh), m = __half2float(mh);
  const float inv = __frcp_rn(s);
  // all quotients lie between those of lo and hi (infinite or NaN where s is 0)
  odd |= !((lo - m) * inv > -0.25f) || !((hi - m) * inv < 15.25f);
  constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, ties to even
  // x - m is rounded where |x| is below 2^-16 or |m| below 2^-12 of it, and may then seem to lie on a border (k + 0.5) s that
  // it only comes near: with a small x if -m / s is within 2^-12 of k + 0.5, with a small m if that is below 2^-8 s.  m / s in
  // units of 2^-10, as the low bits of a sum, tells both; only then (a group in 1000) are the dims looked through.  (All such
  // groups decided code by code: 78 us; the question not asked: 64.3 us, not 65.7.)
  constexpr uint32_t kZero = 0x46400000u;  // 1.5 2^13
  const uint32_t z = __float_as_uint(fmaf(m, inv, __uint_as_float(kZero)));
  if ((z & 0x3ffu) == 0x200u || z - kZero + 4u <= 8u) {
    odd |= m != 0.f && z - kZero + 4u <= 8u;
    const uint32_t small = __float_as_uint(fabsf(m) * 0x1p-15f) >> 16;  // as bf16 bits
#pragma unroll
    for (int j = 0; j < 8; ++j)  // 0 itself is exact
      odd |= (q[j] & 0x7fffu) - 1u < small || (q[j] >> 16 & 0x7fffu) - 1u < small;
  }
  const float2 m2 = make_float2(-m, -m), i2 = make_float2(inv, inv), s2 = make_float2(-s, -s);
  const float2 up = make_float2(kMagic, kMagic);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float2 x;
    bf16x2_to_f32(q[j], x.x, x.y);
    const float2 t = __fadd2_rn(x, m2);
    const float2 q0 = __fmul2_rn(t, i2);
    const float2 b = __fadd2_rn(__ffma2_rn(__ffma2_rn(q0, s2, t), i2, q0), up);
    c[j / 4] += (__float_as_uint(b.x) << (8 * (j % 4))) + (__float_as_uint(b.y) << (8 * (j % 4) + 4));
  }
  // the sums of the adds' exponent bits: sum of 0x4b400000 << 4 j, j = 0..7, modulo 2^32
  constexpr uint32_t kBias = 0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8) + (0x4b400000u << 12) +
                             (0x4b400000u << 16) + (0x4b400000u << 20) + (0x4b400000u << 24) + (0x4b400000u << 28);
  uint2 code = make_uint2(c[0] - kBias, c[1] - kBias);
  if (odd) code = quantise_slow(wa, wb, s, m);
  return {code, __halves2half2(sh, mh)};
}

// A lane: 16 dims of one (token, head)'s key and of its value.  WIDE: rows start on 32 bytes.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kKvThreads) kv_append_q4_kernel(const KvAppendQ4Launch p, const unsigned nrows,
                                                                  const FastDiv heads, const FastDiv page_keys) {
  constexpr int G = D / 64, TPR = D / 16;  // groups and lanes of a row
  const unsigned row = blockIdx.x * (kKvThreads / TPR) + threadIdx.x / TPR;  // (token, head)
  if (row >= nrows) return;  // whole groups of lanes
  const int sub = threadIdx.x % TPR;
  const unsigned tok = heads.div(row);
  const int h = (int)(row - tok * heads.d);
  const int slot = p.slots[tok];
  const uint4* ksrc = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.k) +
                                                     (long long)tok * p.ks[0] + h * p.ks[1] + 16 * sub);
  const uint4* vsrc = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.v) +
                                                     (long long)tok * p.vs[0] + h * p.vs[1] + 16 * sub);
  uint4 ka, kb, va, vb;
  if constexpr (WIDE) {
    ldg256(ksrc, ka, kb);
    ldg256(vsrc, va, vb);
  } else {
    ka = ksrc[0], kb = ksrc[1], va = vsrc[0], vb = vsrc[1];
  }
  const unsigned team = 0xfu << (threadIdx.x & 28);  // the group's four lanes
  const Quantised qk = quantise(ka, kb, team), qv = quantise(va, vb, team);
  if (slot < 0 || slot >= p.num_pages * p.page_size) {  // -1: not written; anything else is an error
    if (slot != -1 && sub == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    return;
  }
  const int page = (int)page_keys.div((unsigned)slot), in_page = slot - page * p.page_size;
  const int tile = in_page / kTileKeys, key = in_page % kTileKeys, g = sub / 4;
  uint8_t* const dst = reinterpret_cast<uint8_t*>(p.pool) + kv_q4_tile_at(page, h, tile, p.Hkv, p.page_size / kTileKeys, D);
  uint8_t* const code = dst + (g * kTileKeys + key) * 32 + (sub % 4) * 8;
  *reinterpret_cast<uint2*>(code) = qk.code;
  *reinterpret_cast<uint2*>(code + kv_q4_v_off(D)) = qv.code;
  if (sub % 4 == 0) {
    uint8_t* const pair = dst + kv_q4_kp_off(D) + (key * G + g) * 4;
    *reinterpret_cast<__half2*>(pair) = qk.pair;
    *reinterpret_cast<__half2*>(pair + kv_q4_vp_off(D) - kv_q4_kp_off(D)) = qv.pair;
  }
}

template <bool WIDE>
__device__ __forceinline__ void codes_to_bf16(uint2 w, uint32_t pair, __nv_bfloat16* dst) {
  const float2 sm = __half22float2(*reinterpret_cast<__half2*>(&pair));
  const float s24 = sm.x * 16777216.f, s20 = sm.x * 1048576.f;
  uint4 out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i ? w.y : w.x;
    float x[8];
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // dims n and n + 4 of the word
      const uint32_t h = (n < 2 ? v : v >> 8) & (n % 2 ? 0x00f000f0u : 0x000f000fu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[n] = fmaf(f.x, n % 2 ? s20 : s24, sm.y);
      x[n + 4] = fmaf(f.y, n % 2 ? s20 : s24, sm.y);
    }
    out[i] = pack8(x);
  }
  if constexpr (WIDE) {
    stg256(dst, out[0], out[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) = out[0];
    *reinterpret_cast<uint4*>(dst + 8) = out[1];
  }
}

// WIDE: k and v start on 32 bytes.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kKvThreads) kv_gather_q4_kernel(const KvGatherQ4Launch p, const unsigned nrows,
                                                                  const FastDiv heads, const FastDiv page_keys) {
  constexpr int G = D / 64, TPR = D / 16;
  const unsigned row = blockIdx.x * (kKvThreads / TPR) + threadIdx.x / TPR;  // (token, head)
  if (row >= nrows) return;
  const int sub = threadIdx.x % TPR;
  const int tok = (int)heads.div(row);
  const int h = (int)(row - (unsigned)tok * heads.d);
  int seq = 0;
  for (int n = p.B; n > 1;) {  // the last of the sequences that start at or before tok
    const int half = n / 2;
    if (p.cu_k[seq + half] <= tok) {
      seq += half;
      n -= half;
    } else {
      n = half;
    }
  }
  const int first = p.cu_k[seq];
  if (tok < first || tok >= p.cu_k[seq + 1]) return;  // rows of no sequence stay as they were
  const long long pos = (long long)tok - first + (p.kv_starts != nullptr ? p.kv_starts[seq] : 0);
  const int pg = pos >= 0 && pos <= 0x7fffffffLL ? (int)page_keys.div((unsigned)pos) : -1;
  int page = -1;
  if (pg >= 0 && pg < p.max_pages) page = p.block_table[(size_t)seq * p.max_pages + pg];
  if (page < 0 || page >= p.num_pages) {  // the row stays as it was
    if (sub == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    return;
  }
  const int in_page = (int)pos - pg * p.page_size;
  const int tile = in_page / kTileKeys, key = in_page % kTileKeys;
  const uint8_t* src =
      reinterpret_cast<const uint8_t*>(p.pool) + kv_q4_tile_at(page, h, tile, p.Hkv, p.page_size / kTileKeys, D);
  const int g = sub / 4;
  const int code = (g * kTileKeys + key) * 32 + (sub % 4) * 8, par = (key * G + g) * 4;
  const uint2 wk = *reinterpret_cast<const uint2*>(src + code);
  const uint2 wv = *reinterpret_cast<const uint2*>(src + kv_q4_v_off(D) + code);
  const uint32_t pk = *reinterpret_cast<const uint32_t*>(src + kv_q4_kp_off(D) + par);
  const uint32_t pv = *reinterpret_cast<const uint32_t*>(src + kv_q4_vp_off(D) + par);
  const size_t at = (size_t)row * D + 16 * sub;
  codes_to_bf16<WIDE>(wk, pk, reinterpret_cast<__nv_bfloat16*>(p.k) + at);
  codes_to_bf16<WIDE>(wv, pv, reinterpret_cast<__nv_bfloat16*>(p.v) + at);
}

// Blocks for `rows` rows of D elements; cudaErrorNotSupported past 2^31 rows (more than any GPU's memory).
cudaError_t kv_blocks(long long rows, int D, unsigned& blocks) {
  if (rows > 0x7fffffffLL) return cudaErrorNotSupported;
  const int per = kKvThreads / (D / 16);
  blocks = (unsigned)((rows + per - 1) / per);
  return cudaSuccess;
}

}  // namespace

namespace {

bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

template <int D>
void append(const KvAppendQ4Launch& p, unsigned rows, unsigned blocks) {
  const FastDiv heads = make_fast_div((unsigned)p.Hkv), page_keys = make_fast_div((unsigned)p.page_size);
  const bool wide = on32(p.k) && on32(p.v) && (p.ks[0] | p.ks[1] | p.vs[0] | p.vs[1]) % 16 == 0;
  if (wide)
    kv_append_q4_kernel<D, true><<<blocks, kKvThreads, 0, p.stream>>>(p, rows, heads, page_keys);
  else
    kv_append_q4_kernel<D, false><<<blocks, kKvThreads, 0, p.stream>>>(p, rows, heads, page_keys);
}

template <int D>
void gather(const KvGatherQ4Launch& p, unsigned rows, unsigned blocks) {
  const FastDiv heads = make_fast_div((unsigned)p.Hkv), page_keys = make_fast_div((unsigned)p.page_size);
  if (on32(p.k) && on32(p.v))
    kv_gather_q4_kernel<D, true><<<blocks, kKvThreads, 0, p.stream>>>(p, rows, heads, page_keys);
  else
    kv_gather_q4_kernel<D, false><<<blocks, kKvThreads, 0, p.stream>>>(p, rows, heads, page_keys);
}

}  // namespace

cudaError_t launch_kv_append_q4(const KvAppendQ4Launch& p) {
  const long long rows = (long long)p.T * p.Hkv;
  unsigned blocks;
  const cudaError_t e = kv_blocks(rows, p.D, blocks);
  if (e != cudaSuccess || blocks == 0) return e;
  if (p.D == 64)
    append<64>(p, (unsigned)rows, blocks);
  else
    append<128>(p, (unsigned)rows, blocks);
  return cudaGetLastError();
}

cudaError_t launch_kv_gather_q4(const KvGatherQ4Launch& p) {
  const long long rows = (long long)p.total_k * p.Hkv;
  unsigned blocks;
  const cudaError_t e = kv_blocks(rows, p.D, blocks);
  if (e != cudaSuccess || blocks == 0) return e;
  if (p.D == 64)
    gather<64>(p, (unsigned)rows, blocks);
  else
    gather<128>(p, (unsigned)rows, blocks);
  return cudaGetLastError();
}

}  // namespace attn
