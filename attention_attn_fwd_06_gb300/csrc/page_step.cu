// page_step.cu -- page bookkeeping of a serving step: block tables and slot maps from request lengths, on the GPU.
//
// Row b of the block table holds a = kv_lens[b] keys on its first ceil(a / page_size) pages.  A step keeps the first
// c = keep_lens[b] of them (default: all) and adds n = new_lens[b] (default: 0).  With have = ceil(a / page_size) and
// need = ceil((c + n) / page_size) the row gives the pages need .. have-1 back or takes the pages have .. need-1;
// the pages it keeps stay where they are.  Free pages are a stack: pages come back in reverse row-major order and are
// taken in row-major order from the top, so dropping what a step added restores the stack exactly.  New token i of
// row b sits at position c + i, slot = page id * page_size + position % page_size.
//
// What bounds it: latency.  A decode step moves a few hundred bytes; 64k prompt tokens take 0.6 MB.  So everything
// is one launch of one thread-block cluster: every CTA reads all lengths and scans them in its own shared memory
// (three running sums: tokens, pages taken, pages given back), and a cluster barrier separates these reads from the
// in-place writes, which needs no scratch memory and no second launch.
#include <atomic>

#include "common.cuh"
#include "intdiv.h"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kPageThreads = 1024;  // at most; kPageThreadsSmall for a decode step
constexpr int kPageThreadsSmall = 256;

// All CTAs of the launch: what each has read comes before what any writes next.
__device__ __forceinline__ void launch_barrier() {
  if (gridDim.x == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// ceil(x / d) for x >= 0
__device__ __forceinline__ int pages_of(int x, const FastDiv& d) {
  const unsigned q = d.div((unsigned)x);
  return (int)(q + (q * d.d < (unsigned)x ? 1u : 0u));
}

// The largest b with sum[b] <= i, for 0 <= i < sum[B] (rows of no items are passed over).
__device__ __forceinline__ int row_of(const int* sum, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPageThreads) page_step_kernel(const PageStepLaunch p, const FastDiv page_keys) {
  extern __shared__ int page_smem[];
  const int B = p.B, ps = p.page_size;
  int* cu = page_smem;          // [B + 1] tokens before row b
  int* taken = cu + B + 1;      // [B + 1] pages taken before row b
  int* given = taken + B + 1;   // [B + 1] pages given back before row b
  int* kept = given + B + 1;    // [B] keys kept
  int* have = kept + B;         // [B] pages before the step
  int* need = have + B;         // [B] pages after it
  __shared__ int wsum[4][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int gtid = blockIdx.x * threads + tid, gthreads = gridDim.x * threads;
  const int count = *p.free_count;

  // ---- lengths and their running sums (every CTA: all rows) ----
  const long long cap = (long long)p.max_pages * ps;  // below 2^31
  const int per = (B + threads - 1) / threads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  unsigned s0 = 0;                       // the thread's tokens (modulo 2^32)
  int s1 = 0, s2 = 0;                    // pages taken, pages given back
  unsigned n_low = 0, n_high = 0;        // tokens again, in halves that cannot overflow
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int a = p.kv_lens[b];
    const int c = p.keep_lens != nullptr ? p.keep_lens[b] : a;
    const int n = p.new_lens != nullptr ? p.new_lens[b] : 0;
    const bool ok = a >= 0 && a <= cap && c >= 0 && c <= a && n >= 0 && n <= cap - c;
    bad |= ok ? 0 : 1;
    const int h = ok ? pages_of(a, page_keys) : 0, d = ok ? pages_of(c + n, page_keys) : 0;
    kept[b] = c;
    have[b] = h;
    need[b] = d;
    s0 += ok ? (unsigned)n : 0u;
    n_low += ok ? n & 0xffff : 0;
    n_high += ok ? n >> 16 : 0;
    s1 += max(d - h, 0);
    s2 += max(h - d, 0);
  }
  unsigned i0 = s0;
  int i1 = s1, i2 = s2;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned t0 = __shfl_up_sync(0xffffffffu, i0, off);
    const int t1 = __shfl_up_sync(0xffffffffu, i1, off), t2 = __shfl_up_sync(0xffffffffu, i2, off);
    if (lane >= off) {
      i0 += t0;
      i1 += t1;
      i2 += t2;
    }
  }
  n_low = __reduce_add_sync(0xffffffffu, n_low);
  n_high = __reduce_add_sync(0xffffffffu, n_high);
  if (lane == 31) {
    wsum[0][warp] = (int)n_low;
    wsum[1][warp] = (int)n_high;
    wsum[2][warp] = i1;
    wsum[3][warp] = i2;
  }
  bad = __syncthreads_or(bad);
  // lane w: warp w's sums; totals, and what comes before this warp
  int ws[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) ws[k] = lane < threads / 32 ? wsum[k][lane] : 0;
  const long long total = ((long long)__reduce_add_sync(0xffffffffu, (unsigned)ws[1]) << 16) +
                          __reduce_add_sync(0xffffffffu, (unsigned)ws[0]);
  const int ntaken = (int)__reduce_add_sync(0xffffffffu, (unsigned)ws[2]);
  const int ngiven = (int)__reduce_add_sync(0xffffffffu, (unsigned)ws[3]);
  const bool before = lane < warp;
  unsigned e0 = __reduce_add_sync(0xffffffffu, before ? ((unsigned)ws[1] << 16) + (unsigned)ws[0] : 0u) + i0 - s0;
  int e1 = (int)__reduce_add_sync(0xffffffffu, before ? (unsigned)ws[2] : 0u) + i1 - s1;
  int e2 = (int)__reduce_add_sync(0xffffffffu, before ? (unsigned)ws[3] : 0u) + i2 - s2;
  const bool listed = p.slots != nullptr || p.positions != nullptr;
  const bool wrong = bad || count < 0 || (long long)count + ngiven > p.num_pages || (listed && total > p.max_tokens) ||
                     total > 0x7fffffffLL;
  const bool refused = wrong || count + ngiven < ntaken;
  if (!refused) {
    for (int b = b0; b < b1; ++b) {  // the row's sums again, from what it kept
      cu[b] = (int)e0;  // (below 2^31 now, as the total is)
      taken[b] = e1;
      given[b] = e2;
      e0 += p.new_lens != nullptr ? (unsigned)p.new_lens[b] : 0u;
      e1 += max(need[b] - have[b], 0);
      e2 += max(have[b] - need[b], 0);
    }
    if (tid == 0) {
      cu[B] = (int)total;
      taken[B] = ntaken;
      given[B] = ngiven;
    }
  }
  __syncthreads();
  if (gridDim.x > 1) launch_barrier();  // every CTA has read the lengths and the count: they may change now

  if (refused) {  // nothing changes but the lists, which name no token
    if (gtid == 0) record_status(p.status, wrong ? ATTN_ERR_DEVICE_BOUNDS : ATTN_ERR_DEVICE_POOL);
    for (int i = gtid; i < p.max_tokens; i += gthreads) {
      if (p.slots != nullptr) p.slots[i] = -1;
      if (p.positions != nullptr) p.positions[i] = -1;
    }
    if (p.cu_new != nullptr)
      for (int b = gtid; b <= B; b += gthreads) p.cu_new[b] = 0;
    return;
  }

  // ---- pages given back, onto the stack ----
  for (int r = gtid; r < ngiven; r += gthreads) {
    const int b = row_of(given, B, r);
    int* entry = p.block_table + (size_t)b * p.max_pages + need[b] + (r - given[b]);
    const int id = *entry;
    if (id < 0 || id >= p.num_pages) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    p.free_pages[count + ngiven - 1 - r] = id;
    *entry = -1;
  }
  if (ngiven > 0) launch_barrier();  // (the same in every CTA) pages just given back can be taken below
  const int top = count + ngiven;

  // ---- pages taken, lengths, running sums ----
  for (int r = gtid; r < ntaken; r += gthreads) {
    const int b = row_of(taken, B, r);
    const int id = __ldcg(p.free_pages + top - 1 - r);
    if (id < 0 || id >= p.num_pages) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    p.block_table[(size_t)b * p.max_pages + have[b] + (r - taken[b])] = id;
  }
  for (int b = gtid; b < B; b += gthreads) {
    p.kv_lens[b] = kept[b] + cu[b + 1] - cu[b];
    if (p.cu_new != nullptr) p.cu_new[b] = cu[b];
  }
  if (gtid == 0) {
    *p.free_count = top - ntaken;
    if (p.cu_new != nullptr) p.cu_new[B] = (int)total;
  }

  // ---- the new tokens: four in a row for each thread, which mostly share one row and one page ----
  if (!listed) return;
  const bool vec = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
  // (from the last thread on: other warps than those that work on rows, when there are few of both)
  for (long long i4 = 4ll * (gthreads - 1 - gtid); i4 < p.max_tokens; i4 += 4ll * gthreads) {
    int slot[4], at[4];
    int b = i4 < total ? row_of(cu, B, (int)i4) : B;
    int pg = -1, id = -1, pgb = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long i = i4 + u;
      slot[u] = at[u] = -1;
      if (i < total) {
        while (cu[b + 1] <= (int)i) ++b;
        const int pos = kept[b] + ((int)i - cu[b]);
        const int q = (int)page_keys.div((unsigned)pos);
        if (q != pg || b != pgb) {
          pg = q;
          pgb = b;
          id = q < have[b] ? p.block_table[(size_t)b * p.max_pages + q]
                           : __ldcg(p.free_pages + top - 1 - (taken[b] + q - have[b]));
          if (id < 0 || id >= p.num_pages) {
            record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            id = -1;
          }
        }
        at[u] = pos;
        slot[u] = id < 0 ? -1 : id * ps + (pos - q * ps);
      }
    }
    if (vec && i4 + 4 <= p.max_tokens) {
      if (p.slots != nullptr) *reinterpret_cast<int4*>(p.slots + i4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (p.positions != nullptr) *reinterpret_cast<int4*>(p.positions + i4) = make_int4(at[0], at[1], at[2], at[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i4 + u < p.max_tokens) {
          if (p.slots != nullptr) p.slots[i4 + u] = slot[u];
          if (p.positions != nullptr) p.positions[i4 + u] = at[u];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_page_step(const PageStepLaunch& p) {
  // the shared-memory opt-in is per device; host threads may be here at once
  static std::atomic<bool> attr_set[64] = {};
  const size_t smem = ((size_t)6 * p.B + 3) * sizeof(int);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(page_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(((size_t)6 * kPageStepMaxRows + 3) * sizeof(int)));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  // One CTA until the tokens fill it, or the pages that may move where no list of tokens bounds them; then the largest
  // portable cluster.  (8 rows, a token each: 3.3 us a call with 256 threads, 5.9 us with 1024; 70k prompt tokens and their
  // release, 4.4k pages: 13.9 us with clusters for both calls, 19.5 us with one CTA for the release.)  What moves is known to
  // the device only, so a step with keep_lens goes by the table's width: 8 rows that take two tokens each and drop them again
  // take 6.8 us for both calls up to 4096 entries, 8.0 us above.
  const bool unbounded = p.keep_lens != nullptr || p.max_tokens == 0;
  const bool many = p.max_tokens > 2 * kPageThreads || (unbounded && (long long)p.B * p.max_pages > 4 * kPageThreads);
  cfg.gridDim = dim3(many ? 8 : 1);
  cfg.blockDim = dim3(many || p.B > kPageThreadsSmall || p.max_tokens > 4 * kPageThreadsSmall ? kPageThreads
                                                                                               : kPageThreadsSmall);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = p.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cfg.gridDim.x;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = many ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, page_step_kernel, p, make_fast_div((unsigned)p.page_size));
}

}  // namespace attn
