// verify_drafts.cu -- which drafted tokens stand, and the token that follows them, from given random numbers.
//
// Sequence b has n drafted tokens x_0 .. x_{n-1}, drawn from q_0 .. q_{n-1}, and n + 1 rows p_0 .. p_n of the target's
// probabilities.  Draft i stands while u_i q_i(x_i) < p_i(x_i) (both sides exact: products of 24-bit numbers in 64-bit
// floats).  The token after the ones that stand has the weights max(p_r - q_r, 0), r being the refused draft, or p_n where
// all stand; it is the lowest j with w_0 + .. + w_j > u (w_0 + .. + w_{V-1}).  Accepting and then drawing so leaves a token
// distributed as p.
//
// The sums decide which token comes out, so they carry more than 32 bits: a lane adds fp32 terms into a pair of floats (a
// sum and the sum of its roundings, Knuth's two-sum), a difference p - q enters with its own rounding, and the lane's pairs of
// some 2048 tokens, lanes, warps and CTAs are joined as such pairs, 2^-47 each, in a fixed order: 2^-39 of the sum up to 2^20
// tokens, 2^-34 up to 2^30 (thousands of joins one after another), and the same bits every time.  (64-bit floats run at two
// adds a clock and SM: with the joins in them 8 sequences over 32,000 tokens took 20.5 us a call, 12 without.)
//
// What bounds it: for few sequences the chain of launch, drafts (1.4 us), the row (1.1), the exchange (0.7), the segment (0.6)
// and the token in it (2 us), by timer stamps of 8 sequences; for many, reading a row of p each, and of q where a draft is refused,
// beside that chain.  A cluster of CTAs takes a sequence: every CTA decides which drafts stand by itself, its warps sum a segment of the row each,
// the segments' sums go to every CTA of the cluster through distributed shared memory, and the CTA that holds the segment where
// the sum passes u's share reads that segment again (from L2), its warps a piece each, and finds the token.  CTAs of 8 warps at 48
// registers, so that five share an SM and one's chain runs beside another's reading.
// Measured (CUDA-graph replays over rotating inputs): 8 sequences of 4 drafts over 32,000 tokens 6.6 us; 64 of up to 8 over
// 131,072 16.2 us (a draft refused in half of them: 51.5 MB, 3.2 TB/s, 0.48 of the copy bandwidth); 37 without distributions over
// 50,001 in bf16, one element a load, 9.3 us.  Beside 6.3 / 15.9 / 8.9 us of the day: four CTAs an SM with twice the loads in
// flight 6.5 / 16.5 / 8.8 us, CTAs of 16 warps 7.6 / 21.2 / 11.5 us; sums element by element with every weight's check 8.0 / 29.2 /
// 12.0 us, loads behind their conditions besides 7.9 / 28.6 / 15.6.
#include <atomic>
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kVerifyWarps = 8;
constexpr int kVerifyMaxCluster = 16;
// Sixteen CTAs a sequence in place of eight where a row is this long and all sequences' CTAs still fit at four an SM: 2 sequences
// over 220,000 tokens 8.6 against 11.6 us, 32 over 131,072 11.4 against 13.4, 19 over them 9.0 against 10.3; below, the larger
// exchange costs more (8 over 32,000 7.0 against 6.5).
constexpr int kVerifyLongRow = 65536;
constexpr int kVerifySegments = kVerifyWarps * kVerifyMaxCluster;

template <typename T>
__device__ __forceinline__ float as_float(T x);
template <>
__device__ __forceinline__ float as_float<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// A sum and the sum of its roundings.
struct Sum {
  float s = 0.f, e = 0.f;
  // Knuth's two-sum of s and x; what it rounds off, and `rest`, go to e
  __device__ __forceinline__ void add(float x, float rest) {
    const float t = s + x;
    const float z = t - s;
    e += ((s - (t - z)) + (x - z)) + rest;
    s = t;
  }
  // the pair's sum in s, the rest in e (half an ulp of s at most)
  __device__ __forceinline__ void settle() {
    const float t = s + e;
    const float z = t - s;
    e = (s - (t - z)) + (e - z);
    s = t;
  }
  __device__ __forceinline__ void add(Sum o) {
    add(o.s, o.e);
    settle();
  }
};
__device__ __forceinline__ Sum plus(Sum a, Sum b) {
  a.add(b);
  return a;
}
// a > b, both settled (where the leading parts are near each other their difference is exact; where they are not it decides)
__device__ __forceinline__ bool above(Sum a, Sum b) { return (a.s - b.s) + (a.e - b.e) > 0.f; }
__device__ __forceinline__ bool positive(Sum a) { return a.s > 0.f; }
// u times a; NaN, which nothing is above, unless u < 1: added up otherwise, the weights short of the last ones may come out as their
// total or an ulp of the rests past it
__device__ __forceinline__ Sum share(float u, Sum a) {
  Sum r;
  r.s = u < 1.f ? u * a.s : NAN;
  r.e = fmaf(u, a.s, -r.s) + u * a.e;
  r.settle();
  return r;
}

__device__ __forceinline__ Sum shuffle(Sum v, int lane) {
  Sum r;
  r.s = __shfl_sync(0xffffffffu, v.s, lane);
  r.e = __shfl_sync(0xffffffffu, v.e, lane);
  return r;
}
__device__ __forceinline__ Sum warp_sum(Sum v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    Sum o;
    o.s = __shfl_xor_sync(0xffffffffu, v.s, m);
    o.e = __shfl_xor_sync(0xffffffffu, v.e, m);
    v = plus(v, o);
  }
  return v;
}
// Of the lanes below and this one's (incl), and of the lanes below (excl).
__device__ __forceinline__ void warp_scan(Sum v, Sum& incl, Sum& excl, int lane) {
  incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    Sum up;
    up.s = __shfl_up_sync(0xffffffffu, incl.s, off);
    up.e = __shfl_up_sync(0xffffffffu, incl.e, off);
    if (lane >= off) incl = plus(up, incl);
  }
  excl.s = __shfl_up_sync(0xffffffffu, incl.s, 1);
  excl.e = __shfl_up_sync(0xffffffffu, incl.e, 1);
  if (lane == 0) excl = Sum{};
}

// The row that the token is drawn from.
template <typename T>
struct Row {
  const T* p;
  const T* q;    // taken away; or null
  int skip;      // this token's weight is 0 (a refused draft without a distribution); or -1
  // Weight of token j with probabilities pj, qj: d, and what rounding took from it; whatever is not a positive finite number
  // counts as 0.
  __device__ __forceinline__ float weight(float pj, float qj, int j, float& rest) const {
    float d = pj - qj;
    rest = (pj - d) - qj;  // exact where pj >= qj
    if (!(d > 0.f && d < INFINITY) || j == skip) {
      d = 0.f;
      rest = 0.f;
    }
    return d;
  }
};

// Elements 16 bytes at a time, or one by one where rows do not start on 16 bytes.
template <typename T, bool VEC>
struct Access {
  static constexpr int N = VEC ? 16 / sizeof(T) : 1;
  struct Raw {
    uint32_t w[VEC ? 4 : 1];
  };
  // tokens j .. j + N - 1, all of them in the row
  static __device__ __forceinline__ Raw load(const T* row, int j) {
    Raw r;
    if constexpr (!VEC) {
      r.w[0] = __float_as_uint(as_float<T>(__ldg(row + j)));
    } else {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + j));
      r.w[0] = x.x;
      r.w[1] = x.y;
      r.w[2] = x.z;
      r.w[3] = x.w;
    }
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[N]) {
    if constexpr (VEC && sizeof(T) == 2) {
      unpack8(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r.w[i]);
    }
  }
  // of a row that may end among them: what lies past it is not read, and 0
  static __device__ __forceinline__ void load_to(const T* row, int j, int V, float (&v)[N]) {
    if (j + N <= V) {
      unpack(load(row, j), v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = j + i < V ? as_float<T>(__ldg(row + j + i)) : 0.f;
    }
  }
};

__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return __ffma2_rn(b, two(-1.f), a); }

// Two sums side by side (packed adds), of weights that are finite where positive: one that is not makes the sum so.
struct Sum2 {
  float2 s = make_float2(0.f, 0.f), e = make_float2(0.f, 0.f);
  // the weights max(p - q, 0)
  template <bool HAS_Q>
  __device__ __forceinline__ void add(float2 p, float2 q) {
    float2 d = p, rest = two(0.f);
    if constexpr (HAS_Q) {
      d = minus(p, q);
      rest = minus(minus(p, d), q);
      rest.x = d.x > 0.f ? rest.x : 0.f;
      rest.y = d.y > 0.f ? rest.y : 0.f;
    }
    d.x = fmaxf(d.x, 0.f);  // (0 for a NaN too)
    d.y = fmaxf(d.y, 0.f);
    const float2 t = __fadd2_rn(s, d);
    const float2 z = minus(t, s);
    float2 r = __fadd2_rn(minus(s, minus(t, z)), minus(d, z));
    if constexpr (HAS_Q) r = __fadd2_rn(r, rest);
    e = __fadd2_rn(e, r);
    s = t;
  }
  __device__ __forceinline__ Sum joined() const {
    Sum a, b;
    a.s = s.x;
    a.e = e.x;
    b.s = s.y;
    b.e = e.y;
    a.settle();
    a.add(b);
    return a;
  }
};

// Sum of the weights of tokens [lo, hi) (lo and hi - lo multiples of a warp's step, or hi == V) over this lane's elements, the
// positive ones taken to be finite.  A round's loads go out together: none waits behind a condition (in the last round those
// past the end read the first tokens again).  The roundings that a sum gathers (Sum2::e) are rounded themselves: 65,536 adds of
// 0.1 to one pair are off by 2^-22 of their sum, n alike ones by n^2 / 6 2^-48 at most, 2^-40.6 for the 32 of kSumTokens.  FAR, for
// segments of more: after so many a sum is joined to the lane's word of `far` (shared memory: two more registers here would spill)
// and starts again.  (64 sequences over 131,072 tokens, whose segments are no longer: 17.5 us a call with it, 17.2 without.)
constexpr int kSumTokens = 2048;
template <typename T, bool VEC, bool FAR, bool HAS_Q>
__device__ __forceinline__ Sum lane_sum_of(const Row<T>& row, int lo, int hi, int V, int lane, Sum* far) {
  using A = Access<T, VEC>;
  constexpr int STEP = 32 * A::N;
  constexpr int U = VEC ? 2 : 8;
  Sum2 s;
  const int whole = VEC && hi == V ? V - V % A::N : hi;  // end of the row's whole 16 bytes
  auto round = [&](int base, bool all) {
    typename A::Raw p[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int j = base + u * STEP + lane * A::N;
      if (!all && j >= whole) j = lo;
      p[u] = A::load(row.p, j);
      if constexpr (HAS_Q) q[u] = A::load(row.q, j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + u * STEP + lane * A::N;
      float pj[A::N + 1], qj[A::N + 1];
      A::unpack(p[u], *reinterpret_cast<float(*)[A::N]>(pj));
      if constexpr (HAS_Q) A::unpack(q[u], *reinterpret_cast<float(*)[A::N]>(qj));
      if (!all && j >= whole)
#pragma unroll
        for (int i = 0; i < A::N; ++i) pj[i] = 0.f, qj[i] = 0.f;
      if (!HAS_Q && (unsigned)row.skip - (unsigned)j < (unsigned)A::N)
#pragma unroll
        for (int i = 0; i < A::N; ++i)
          if (j + i == row.skip) pj[i] = 0.f;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < A::N; i += 2) s.add<HAS_Q>(make_float2(pj[i], pj[i + 1]), make_float2(qj[i], qj[i + 1]));
      } else if (u % 2 == 0) {
        pj[1] = 0.f;  // (paired below)
        p[u].w[0] = __float_as_uint(pj[0]);
        q[u].w[0] = HAS_Q ? __float_as_uint(qj[0]) : 0u;
      } else {
        s.add<HAS_Q>(make_float2(__uint_as_float(p[u - 1].w[0]), pj[0]),
                     make_float2(__uint_as_float(q[u - 1].w[0]), HAS_Q ? qj[0] : 0.f));
      }
    }
  };
  int base = lo;
  static_assert(kSumTokens % (U * STEP) == 0, "whole rounds");
  for (; base + U * STEP <= whole; base += U * STEP) {
    if (FAR && base != lo && (base - lo) % kSumTokens == 0) {
      Sum v = s.joined();
      if (base - lo > kSumTokens) v.add(far[threadIdx.x]);
      far[threadIdx.x] = v;
      s = Sum2{};
    }
    round(base, true);
  }
  if (base < whole) round(base, false);
  if (VEC && whole + lane < hi) {  // the row's last tokens, short of 16 bytes
    const int j = whole + lane;
    const float p = j == row.skip ? 0.f : as_float<T>(__ldg(row.p + j));
    s.add<HAS_Q>(make_float2(p, 0.f), make_float2(HAS_Q ? as_float<T>(__ldg(row.q + j)) : 0.f, 0.f));
  }
  Sum v = s.joined();
  if (FAR && base - lo > kSumTokens) v.add(far[threadIdx.x]);
  return v;
}
// The same with every weight looked at (rows with infinities).
template <typename T>
__device__ __noinline__ Sum lane_sum_careful(const Row<T> row, int lo, int hi, int lane) {
  Sum s;
  int n = 0;
  Sum far;
  for (int j = lo + lane; j < hi; j += 32) {
    float rest;
    const float w = row.weight(as_float<T>(__ldg(row.p + j)), row.q != nullptr ? as_float<T>(__ldg(row.q + j)) : 0.f, j, rest);
    s.add(w, rest);
    s.settle();
    if (++n % (kSumTokens / 32) == 0) {
      far.add(s);
      s = Sum{};
    }
  }
  s.add(far);
  return s;
}
// (No tokens: nothing.  A row's last tokens, short of 16 bytes, are those of the part that they end.)
template <typename T, bool VEC, bool FAR>
__device__ __forceinline__ Sum lane_sum(const Row<T>& row, int lo, int hi, int V, int lane, bool careful, Sum* far) {
  if (lo >= hi) return Sum{};
  if (careful) return lane_sum_careful<T>(row, lo, hi, lane);
  return row.q != nullptr ? lane_sum_of<T, VEC, FAR, true>(row, lo, hi, V, lane, far)
                          : lane_sum_of<T, VEC, FAR, false>(row, lo, hi, V, lane, far);
}

// Parts of a sum, PER a lane, one warp: their running sums.
template <int PER>
struct Parts {
  Sum v[PER], incl, excl;
  __device__ __forceinline__ Parts(const Sum* parts, int count, int lane) {
    Sum own;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = lane * PER + i < count ? parts[lane * PER + i] : Sum{};
      own.add(v[i]);
    }
    warp_scan(own, incl, excl, lane);
  }
  __device__ __forceinline__ Sum total() const { return shuffle(incl, 31); }
  // The first part, in order, at whose end the running sum (from `before`) passes `target`; where none does (u of 1 or more, or
  // NaN), the last one that holds weight; -1 if none holds any.  `before` becomes the sum before that part.
  __device__ __forceinline__ int pick(Sum target, Sum& before, int lane) const {
    Sum run = plus(before, excl), at_hit = run, at_last = run;
    int hit = -1, last = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const Sum end = plus(run, v[i]);
      if (positive(v[i])) {
        last = lane * PER + i;
        at_last = run;
        if (hit < 0 && above(end, target)) {
          hit = last;
          at_hit = run;
        }
      }
      run = end;
    }
    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), lasts = __ballot_sync(0xffffffffu, last >= 0);
    if (lasts == 0) return -1;
    const int src = hits != 0 ? __ffs(hits) - 1 : 31 - __clz(lasts);
    before = shuffle(hits != 0 ? at_hit : at_last, src);
    return __shfl_sync(0xffffffffu, hits != 0 ? hit : last, src);
  }
};

template <typename T, bool VEC, bool FAR>
__global__ void __launch_bounds__(32 * kVerifyWarps, 5) verify_drafts_kernel(const VerifyDraftsLaunch p, int segment) {
  namespace cg = cooperative_groups;
  using A = Access<T, VEC>;
  constexpr int STEP = 32 * A::N;
  __shared__ Sum sums[2][kVerifySegments];  // of all segments of the row, of one try and the next
  __shared__ Sum pieces[kVerifyWarps], s_before, s_target;
  __shared__ Sum far[FAR ? 32 * kVerifyWarps : 1];
  __shared__ int s_n, s_stand, s_row, s_seg;
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = p.K, V = p.V;
  cluster.barrier_arrive();  // (waited for before the first store into another CTA's shared memory: all have started)

  if (warp == 0) {
    // Which drafts stand.  The first 32 drafts and numbers are read beside the length, not after it.
    int n = K, row0 = 0;
    bool bad = false;
    int x = lane < K ? p.drafts[(long long)b * K + lane] : 0;
    float u = lane < K ? p.uniforms[(long long)b * (K + 1) + lane] : 0.f;
    if (p.cu != nullptr) {
      const int c0 = p.cu[b], c1 = p.cu[b + 1];
      bad = c0 < 0 || c1 < c0 || c1 > p.total || c1 - c0 > K + 1;
      n = bad ? -1 : c1 - c0 - 1;  // -1: no rows, nothing to draw from
      row0 = c0;
    } else if (p.draft_lens != nullptr) {
      n = p.draft_lens[b];
      if (n < 0 || n > K) {
        bad = true;
        n = n < 0 ? 0 : K;
      }
    }
    int stand = n < 0 ? 0 : n;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      if (i0 > 0 && i < n) {
        x = p.drafts[(long long)b * K + i];
        u = p.uniforms[(long long)b * (K + 1) + i];
      }
      bool ok = true;
      if (i < n) {
        ok = false;
        if (x < 0 || x >= V) {
          bad = true;
        } else {
          const T* pr = reinterpret_cast<const T*>(p.target) +
                        (p.cu != nullptr ? (long long)(row0 + i) * p.ts[1] : (long long)b * p.ts[0] + (long long)i * p.ts[1]);
          double qx = 1.0;
          if (p.draft != nullptr)
            qx = as_float<T>(__ldg(reinterpret_cast<const T*>(p.draft) + (long long)b * p.ds[0] + (long long)i * p.ds[1] + x));
          ok = (double)u * qx < (double)as_float<T>(__ldg(pr + x));
        }
      }
      const unsigned refused = __ballot_sync(0xffffffffu, !ok);
      if (refused != 0) {
        stand = i0 + __ffs(refused) - 1;
        break;
      }
    }
    if (bad && rank == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    if (lane == 0) {
      s_n = n;
      s_stand = stand;
      s_row = row0;
    }
  }
  __syncthreads();
  const int n = s_n, stand = s_stand;
  int* tokens = p.tokens + (long long)b * (K + 1);
  if (rank == 0) {
    for (int i = threadIdx.x; i <= K; i += blockDim.x)
      if (i != stand || n < 0) tokens[i] = i < stand ? p.drafts[(long long)b * K + i] : -1;
    if (threadIdx.x == 0) {
      p.accepted[b] = stand;
      if (p.keep_lens != nullptr) p.keep_lens[b] = p.kv_lens[b] - (n < 0 ? 0 : n - stand);
    }
  }
  cluster.barrier_wait();
  if (n < 0) return;  // (every CTA of the cluster)

  Row<T> row;
  row.p = reinterpret_cast<const T*>(p.target) +
          (p.cu != nullptr ? (long long)(s_row + stand) * p.ts[1] : (long long)b * p.ts[0] + (long long)stand * p.ts[1]);
  row.q = nullptr;
  row.skip = -1;
  if (stand < n) {
    if (p.draft != nullptr)
      row.q = reinterpret_cast<const T*>(p.draft) + (long long)b * p.ds[0] + (long long)stand * p.ds[1];
    else
      row.skip = p.drafts[(long long)b * K + stand];
  }
  const int count = size * kVerifyWarps;
  const int mine = rank * kVerifyWarps + warp;
  const float u = p.uniforms[(long long)b * (K + 1) + K];
  // Up to three tries: with weights taken to be finite; if their sum is not, with every one looked at; if there is none and
  // something was taken from p, with p itself (looked at again).
  int seg = -1;
  bool careful = false;
  for (int attempt = 0;; ++attempt) {
    const long long lo = (long long)mine * segment;
    Sum v = lane_sum<T, VEC, FAR>(row, (int)min(lo, (long long)V), (int)min(lo + segment, (long long)V), V, lane, careful, far);
    v = warp_sum(v);
    Sum* const parts = sums[attempt & 1];  // (the tries before the last one have been read: a cluster barrier lies between)
    if (lane < size) *cluster.map_shared_rank(&parts[mine], lane) = v;
    cluster.sync();
    if (warp == 0) {  // the total, and the segment, found by every CTA for itself
      const Parts<kVerifySegments / 32> all(parts, count, lane);
      const Sum total = all.total(), target = share(u, total);
      Sum before;
      int found = all.pick(target, before, lane);
      if (!(total.s < INFINITY)) found = -2;
      if (lane == 0) {
        s_seg = found;
        s_before = before;
        s_target = target;
      }
    }
    __syncthreads();
    seg = s_seg;
    if (seg == -2 && !careful) {
      careful = true;
    } else if (seg < 0 && (row.q != nullptr || row.skip >= 0)) {
      row.q = nullptr;  // p nowhere above q: p itself
      row.skip = -1;
      careful = true;
    } else {
      break;
    }
  }
  if (seg < 0) {  // no weight at all
    if (rank == 0 && threadIdx.x == 0) {
      tokens[stand] = -1;
      record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    }
    return;
  }
  if (seg / kVerifyWarps != rank) return;
  // the segment's pieces, one a warp
  const int first = seg * segment, end = (int)min((long long)first + segment, (long long)V);
  const int piece = ((segment + kVerifyWarps - 1) / kVerifyWarps + STEP - 1) / STEP * STEP;
  {
    const int lo = min(first + warp * piece, end);
    const Sum v = warp_sum(lane_sum<T, VEC, FAR>(row, lo, min(lo + piece, end), V, lane, careful, far));
    if (lane == 0) pieces[warp] = v;
  }
  __syncthreads();
  const Sum target = s_target;
  Sum base = s_before;
  int w = Parts<1>(pieces, kVerifyWarps, lane).pick(target, base, lane);
  if (w < 0) w = 0;  // (cannot be: the segment holds weight)
  if (warp != w) return;
  // a warp's step at a time; the step's sum in the order of tokens: lanes, then a lane's elements
  const int lo = min(first + w * piece, end), hi = min(lo + piece, end);
  int found = -1;
  for (int j0 = lo; j0 < hi; j0 += STEP) {
    const int j = j0 + lane * A::N;
    float pj[A::N] = {}, qj[A::N] = {};
    if (j < hi) {
      A::load_to(row.p, j, V, pj);
      if (row.q != nullptr) A::load_to(row.q, j, V, qj);
    }
    Sum part[A::N], own;
#pragma unroll
    for (int i = 0; i < A::N; ++i) {
      part[i].s = row.weight(pj[i], qj[i], j + i, part[i].e);
      own.add(part[i].s, part[i].e);
    }
    own.settle();
    Sum incl, excl;
    warp_scan(own, incl, excl, lane);
    int at = -1, last = -1;
    Sum run = plus(base, excl);
#pragma unroll
    for (int i = 0; i < A::N; ++i) {
      run.add(part[i]);
      if (positive(part[i])) {
        last = j + i;
        if (at < 0 && above(run, target)) at = j + i;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at >= 0), any = __ballot_sync(0xffffffffu, last >= 0);
    if (hit != 0) {
      found = __shfl_sync(0xffffffffu, at, __ffs(hit) - 1);
      break;
    }
    if (any != 0) found = __shfl_sync(0xffffffffu, last, 31 - __clz(any));
    base = plus(base, shuffle(incl, 31));
  }
  if (lane == 0) tokens[stand] = found;
}

template <typename T, bool VEC, bool FAR>
cudaError_t launch_t(const VerifyDraftsLaunch& p, int size, int segment) {
  // clusters of more than 8 CTAs are opted into, per device; host threads may be here at once
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(verify_drafts_kernel<T, VEC, FAR>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.B * (unsigned)size);
  cfg.blockDim = dim3(32 * kVerifyWarps);
  cfg.stream = p.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, VEC, FAR>, p, segment);
  return e != cudaSuccess ? (cudaGetLastError(), e) : e;  // (an error that is told does not wait for the next call)
}

template <typename T, bool VEC>
cudaError_t dispatch_far(const VerifyDraftsLaunch& p) {
  constexpr int STEP = 32 * Access<T, VEC>::N;
  int size = kVerifyMaxCluster;
  if (p.V < kVerifyLongRow || (long long)p.B * size > 4ll * p.num_sms) size /= 2;
  while (size > 1 && ((long long)p.V <= (long long)STEP * kVerifyWarps * (size / 2))) size /= 2;
  const long long warps = (long long)size * kVerifyWarps;
  const long long segment = (((long long)p.V + warps - 1) / warps + STEP - 1) / STEP * STEP;
  return segment > kSumTokens ? launch_t<T, VEC, true>(p, size, (int)segment) : launch_t<T, VEC, false>(p, size, (int)segment);
}

template <typename T>
cudaError_t dispatch_vec(const VerifyDraftsLaunch& p) {
  constexpr int N = 16 / sizeof(T);
  bool vec = reinterpret_cast<unsigned long long>(p.target) % 16 == 0 && p.ts[0] % N == 0 && p.ts[1] % N == 0;
  if (p.draft != nullptr)
    vec = vec && reinterpret_cast<unsigned long long>(p.draft) % 16 == 0 && p.ds[0] % N == 0 && p.ds[1] % N == 0;
  return vec ? dispatch_far<T, true>(p) : dispatch_far<T, false>(p);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyDraftsLaunch& p) {
  if (p.B == 0) return cudaSuccess;
  return p.f32 ? dispatch_vec<float>(p) : dispatch_vec<__nv_bfloat16>(p);
}

}  // namespace attn
