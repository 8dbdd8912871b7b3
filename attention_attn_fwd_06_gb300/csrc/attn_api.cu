// attn_api.cu -- the C ABI declared in include/attn.h.
//
// Host side only: argument validation (before anything touches the device),
// the sm_103 device check, the per-device split-KV workspace and status word,
// and the kernel launches.  No compute happens here and there is no CPU path.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/attn.h"
#include "kernels.h"
#include "kv_q4.h"

// Device status word: kernels record the first problem they see (a kv_len out
// of range, an expired pipeline wait); attn_get_device_status() reads and
// clears it.  Each device holds its own copy.
__device__ unsigned g_attn_device_status;

namespace {

constexpr int kMaxDevices = 64;
// Decode workspace layout: [counters: kDecodeCounterSlots x u32][part_o][part_ml].
// The counter area must be zero before the first call; the kernel leaves it zero.
constexpr size_t kCounterBytes = size_t(attn::kDecodeCounterSlots) * sizeof(unsigned);

struct DeviceState {
  bool probed = false;
  int support = ATTN_OK;  // ATTN_ERR_UNSUPPORTED when the device is not sm_103
  int num_sms = 0;
  unsigned* status = nullptr;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  void* ws_q4 = nullptr;  // attn_decode_q4's partials: all zeros between calls
  size_t ws_q4_bytes = 0;
  void* ws_paged = nullptr;  // attn_decode_multi_paged's counters and partials
  size_t ws_paged_bytes = 0;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

// Fixed split-KV scratch for attn_decode_noalloc: 4 MiB of fp32 partials per
// device, part of the library's device image (no runtime allocation).
constexpr size_t kNoAllocScratchBytes = size_t(4) << 20;
__device__ __align__(256) float g_noalloc_scratch[kNoAllocScratchBytes / sizeof(float)];
// Device address of g_noalloc_scratch per device (host code cannot use the
// symbol itself as a pointer), looked up on the first no-alloc call there.
float* g_noalloc_ptr[kMaxDevices] = {};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ATTN_FAULT_INJECT=skip_arrive (read at each decode and prefill call): CTA 0 of the kernel withholds one
// arrival -- decode a pipeline-slot release, prefill and multi-token decode a P-ready signal -- so a bounded
// wait runs out and ATTN_ERR_DEVICE_TIMEOUT is recorded: a test of the failure path on a real kernel that
// neither faults nor hangs the GPU.
int fault_skip_arrive() {
  const char* v = std::getenv("ATTN_FAULT_INJECT");
  return (v != nullptr && std::strcmp(v, "skip_arrive") == 0) ? 1 : 0;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Looks up (and on first use probes) the current device.  Caller holds g_mu.
int device_state_locked(DeviceState** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return ATTN_ERR_UNSUPPORTED;
  }
  DeviceState& s = g_dev[dev];
  if (!s.probed) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    s.support = (major == 10 && minor == 3) ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
    s.num_sms = sms;
    if (s.support == ATTN_OK) {
      if (cudaGetSymbolAddress(reinterpret_cast<void**>(&s.status), g_attn_device_status) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
      }
    }
    s.probed = true;
  }
  *out = &s;
  return s.support;
}

int map_cuda(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  if (e == cudaErrorNotSupported) return ATTN_ERR_UNSUPPORTED;
  return ATTN_ERR_CUDA;
}

// Ensures the workspace (ws, ws_bytes) holds `bytes`, its first `zeroed` bytes zero when it is made (on `stream`, whose
// next kernel uses it: streams made not to wait for the default stream would not wait for a memset there).  Refuses to
// allocate while the stream is being captured into a CUDA graph.  Caller holds g_mu.
int ensure_buffer_locked(void*& ws, size_t& ws_bytes, size_t bytes, size_t zeroed, cudaStream_t stream) {
  if (bytes <= ws_bytes) return ATTN_OK;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  if (cap != cudaStreamCaptureStatusNone) return ATTN_ERR_INVALID_ARG;
  if (ws != nullptr) {
    cudaFree(ws);  // synchronises the device: no earlier decode can still be using it
    ws = nullptr;
    ws_bytes = 0;
  }
  if (cudaMalloc(&ws, bytes) != cudaSuccess) {
    cudaGetLastError();
    ws = nullptr;
    return ATTN_ERR_CUDA;
  }
  if (cudaMemsetAsync(ws, 0, zeroed, stream) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(ws);
    ws = nullptr;
    return ATTN_ERR_CUDA;
  }
  ws_bytes = bytes;
  return ATTN_OK;
}

int ensure_workspace_locked(DeviceState& s, size_t bytes, cudaStream_t stream) {
  return ensure_buffer_locked(s.ws, s.ws_bytes, bytes, kCounterBytes, stream);  // counters start at zero
}

struct DecodeShape {
  int grid = 0;               // CTAs of the persistent launch
  size_t part_o_elems = 0;    // 2 * grid * GP * D
  size_t part_ml_elems = 0;   // 2 * grid * GP * 2
  size_t bytes = 0;           // counters + partials
};

// The stream-K split gives every CTA an equal slice of the key space and each
// CTA at most two partial rows, so the partial area depends on the grid, the
// heads per CTA and D -- not on the batch or the cache length.
DecodeShape decode_shape(int Hq, int Hkv, int D, int num_sms) {
  DecodeShape s;
  const int gp = attn::decode_heads_per_cta(Hq / Hkv);
  s.grid = attn::decode_grid(num_sms, Hq / Hkv);
  s.part_o_elems = (size_t)2 * s.grid * gp * D;
  s.part_ml_elems = (size_t)2 * s.grid * gp * 2;
  s.bytes = kCounterBytes + (s.part_o_elems + s.part_ml_elems) * sizeof(float);
  return s;
}

// Rows of per-row counters the decode kernel uses for these sizes.
long long decode_counter_rows(int B, int Hq, int Hkv) {
  const int group = Hq / Hkv;
  return (long long)B * Hkv * (group / attn::decode_heads_per_cta(group));
}

int validate_decode(const attn_decode_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->B < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->Lmax < 0 || p->D <= 0) return ATTN_ERR_INVALID_ARG;
  if (p->Hq % p->Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->out_dtype != ATTN_DTYPE_BF16 && p->out_dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (p->chunk < 0 || p->chunk > (1 << 20)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;  // NaN or infinite scale
  if (p->B == 0) return ATTN_OK;
  if (p->q == nullptr || p->kcache == nullptr || p->vcache == nullptr || p->kv_lens == nullptr ||
      p->out == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->kcache) || !aligned16(p->vcache) || !aligned16(p->out) ||
      !aligned4(p->kv_lens) || (p->lse != nullptr && !aligned4(p->lse)))
    return ATTN_ERR_ALIGNMENT;
  if (p->B > 65535 || p->Hkv > 65535 || (long long)p->B * p->Hq > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int validate_fwd(const attn_fwd_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->B < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->Lq < 0 || p->Lkv < 0 || p->D <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (p->Hq % p->Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->causal != 0 && p->causal != 1) return ATTN_ERR_INVALID_ARG;
  if (p->out_dtype != ATTN_DTYPE_BF16 && p->out_dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;  // NaN or infinite scale
  const bool varlen = p->cu_seqlens_q != nullptr || p->cu_seqlens_k != nullptr;
  if (varlen) {
    if (p->cu_seqlens_q == nullptr || p->cu_seqlens_k == nullptr) return ATTN_ERR_INVALID_ARG;
    if (p->total_q < 0 || p->total_k < 0) return ATTN_ERR_INVALID_ARG;
    if (!aligned4(p->cu_seqlens_q) || !aligned4(p->cu_seqlens_k)) return ATTN_ERR_ALIGNMENT;
  }
  if (p->B == 0 || p->Lq == 0 || (varlen && p->total_q == 0)) return ATTN_OK;
  const bool no_keys = varlen ? p->total_k == 0 : p->Lkv == 0;  // then k and v are never read
  if (p->q == nullptr || p->out == nullptr || (!no_keys && (p->k == nullptr || p->v == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->out) ||
      (p->lse != nullptr && !aligned4(p->lse)))
    return ATTN_ERR_ALIGNMENT;
  if (p->B > 65535 || (long long)p->B * p->Hq > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Checks a rotary-embedding argument whose largest position is max_needed - 1 (0: nothing rotated).
int validate_rope(const attn_rope& r, int D, long long max_needed) {
  if (r.style == ATTN_ROPE_NONE || r.cos == nullptr) return ATTN_OK;
  if (r.style != ATTN_ROPE_HALF && r.style != ATTN_ROPE_INTERLEAVED) return ATTN_ERR_INVALID_ARG;
  if (r.sin == nullptr || r.max_pos <= 0) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(r.cos) || !aligned16(r.sin)) return ATTN_ERR_ALIGNMENT;
  if (max_needed > r.max_pos) return ATTN_ERR_INVALID_ARG;
  if ((long long)r.max_pos * (D / 2) > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn::RopeArgs rope_args(const attn_rope& r) {
  attn::RopeArgs a{};
  if (r.style != ATTN_ROPE_NONE && r.cos != nullptr) {
    a.cos = r.cos;
    a.sin = r.sin;
    a.max_pos = r.max_pos;
    a.style = r.style;
  }
  return a;
}

// The current device's state, or why there is none.
int device_state(DeviceState** out) {
  std::lock_guard<std::mutex> lock(g_mu);
  return device_state_locked(out);
}

constexpr long long kIntMax = 0x7fffffffLL;

// Sizes of a 4-bit cache pool (page_size keys a page, in tiles of 16).
int validate_pool_q4(int Hkv, int D, int page_size, int num_pages) {
  if (Hkv <= 0 || D <= 0 || page_size < attn::kTileKeys || page_size > 65536 || page_size % attn::kTileKeys != 0 ||
      num_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if ((long long)num_pages * page_size > kIntMax || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Strides in elements of rows read or written 16 bytes at a time; that of an axis of one element says nothing and becomes 0.
bool take_strides8(const long long* stride, const int* extent, int n, long long* out) {
  bool ok = true;
  for (int i = 0; i < n; ++i) {
    out[i] = extent[i] > 1 ? stride[i] : 0;
    ok = ok && out[i] % 8 == 0;
  }
  return ok;
}

bool aligned128(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 127u) == 0; }

struct DecodeQ4Shape {
  size_t count_bytes = 0;
  size_t part_o_elems = 0;
  size_t bytes = 0;
};

// The counts and partials of any variant: sums, and for each of a CTA's warps that hold one every column's (max, sum).
DecodeQ4Shape decode_q4_shape(int D, int num_sms) {
  DecodeQ4Shape s;
  const size_t cols = attn::decode_q4_partials(num_sms);
  s.count_bytes = (attn::decode_q4_counts(num_sms) * sizeof(unsigned) + 127) / 128 * 128;
  s.part_o_elems = cols * D;
  s.bytes = s.count_bytes + cols * (D + attn::kDecodeQ4Owners * 2) * sizeof(float);
  return s;
}

int validate_decode_q4_heads(int Hq, int Hkv, int Lq, int D) {
  if (Hq <= 0 || Hkv <= 0 || Lq < 1 || D <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if ((long long)(Hq / Hkv) * Lq > 128) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Counters, then two partials (rows of O, and of maximum and sum) for each CTA.
struct DecodeMultiShape {
  size_t part_o_elems = 0;
  size_t bytes = 0;
};
DecodeMultiShape decode_multi_shape(long long rows, int D, int num_sms) {
  DecodeMultiShape s;
  const size_t slots = (size_t)2 * attn::decode_multi_grid(num_sms);
  s.part_o_elems = slots * (size_t)rows * D;
  s.bytes = kCounterBytes + (s.part_o_elems + slots * (size_t)rows * 2) * sizeof(float);
  return s;
}

// A workspace of attn_decode_multi_paged: the region of the kernel for few rows, all zeros between calls, sized for its
// largest call; behind it, for calls of more rows, decode_multi_shape's.  Calls of any sizes can so follow one another.
size_t decode_rows_region(int num_sms) {
  size_t most = 0;
  for (int D : {64, 128})
    for (int rows = 16; rows <= attn::decode_rows_max(D); rows *= 2)
      most = std::max(most, attn::decode_rows_shape(rows, D, num_sms).bytes);
  return most;
}
size_t decode_multi_paged_bytes(long long rows, int D, int num_sms) {
  if (rows <= attn::decode_rows_max(D)) return attn::decode_rows_shape((int)rows, D, num_sms).bytes;
  return decode_rows_region(num_sms) + decode_multi_shape(rows, D, num_sms).bytes;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

// base^(n / d), n and d whole.  The quotient's rounding would come out times ln(base) (2^-49.7 of a frequency with base 1e8 and 112
// dims, 2^-44.6 with 1e300); what it left over, which fma tells exactly, is put back.
double power(double base, double log_base, double n, double d) {
  const double e = n / d, v = std::pow(base, e);
  return std::isfinite(v) ? std::fma(v, std::fma(-e, d, n) / d * log_base, v) : v;
}

double rope_base(const attn_rope_tables_params& p) {
  const double R = p.rotary_dim;
  return p.scaling == ATTN_ROPE_SCALE_BASE ? p.base * power(p.factor, std::log(p.factor), R, R - 2) : p.base;
}

// Radians a position of every pair of a rotary table (attn_rope_tables), sizes checked.  base^(-2i / R) is a product of two of
// sixteen powers (64 calls of pow would take 1 us of a call).
void rope_frequencies(const attn_rope_tables_params& p, double* f) {
  const double R = p.rotary_dim, base = rope_base(p), log_base = std::log(base);
  const int pairs = p.rotary_dim / 2;
  double fine[8], coarse[8], a = 0.0, b = 1.0;
  for (int i = 0; i < 8; ++i) fine[i] = power(base, log_base, -2.0 * i, R);
  for (int i = 0; 8 * i < pairs; ++i) coarse[i] = power(base, log_base, -16.0 * i, R);
  if (p.scaling == ATTN_ROPE_SCALE_INDEX) {
    const double per = R / 2 / log_base;
    a = std::fmax(0.0, std::floor(per * std::log(p.context / (kTwoPi * p.high))));
    b = std::fmin(R - 1, std::ceil(per * std::log(p.context / (kTwoPi * p.low))));
  }
  for (int i = 0; i < pairs; ++i) {
    f[i] = coarse[i / 8] * fine[i % 8];
    if (p.scaling == ATTN_ROPE_SCALE_NONE || p.scaling == ATTN_ROPE_SCALE_BASE) continue;
    double keep = 0.0;  // the share of the pair's speed that stays as it is
    if (p.scaling == ATTN_ROPE_SCALE_TURNS)
      keep = (p.context * f[i] / kTwoPi - p.low) / (p.high - p.low);
    else if (p.scaling == ATTN_ROPE_SCALE_INDEX)
      keep = 1.0 - (i - a) / std::fmax(b - a, 0.001);
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    f[i] = f[i] * keep + f[i] * (1.0 - keep) / p.factor;
  }
}

bool is_empty_fwd(const attn_fwd_params* p) {
  const bool varlen = p->cu_seqlens_q != nullptr;
  return p->B == 0 || p->Lq == 0 || (varlen && p->total_q == 0);
}

}  // namespace

extern "C" {

int attn_version(void) { return 100; }

int attn_selftest_wait_timeout(unsigned int limit_us, void* stream) {
  if (limit_us < 1 || limit_us > 1000000) return ATTN_ERR_INVALID_ARG;
  DeviceState* s = nullptr;
  int st;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    st = device_state_locked(&s);
  }
  if (st != ATTN_OK) return st;
  return map_cuda(attn::launch_selftest_timeout((unsigned long long)limit_us * 1000ull, s->status,
                                                static_cast<cudaStream_t>(stream)));
}

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_INVALID_ARG: return "ATTN_ERR_INVALID_ARG";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
    case ATTN_ERR_ALIGNMENT: return "ATTN_ERR_ALIGNMENT";
    case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA";
    case ATTN_ERR_DEVICE_TIMEOUT: return "ATTN_ERR_DEVICE_TIMEOUT";
    case ATTN_ERR_DEVICE_BOUNDS: return "ATTN_ERR_DEVICE_BOUNDS";
    case ATTN_ERR_SCRATCH_TOO_SMALL: return "ATTN_ERR_SCRATCH_TOO_SMALL";
    case ATTN_ERR_DEVICE_POOL: return "ATTN_ERR_DEVICE_POOL";
    default: return "ATTN_STATUS_UNKNOWN";
  }
}

unsigned long long attn_decode_workspace_bytes(int B, int Hq, int Hkv, int Lmax, int D, int chunk) {
  attn_decode_params p = {};
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lmax = Lmax; p.D = D; p.chunk = chunk;
  p.q = p.kcache = p.vcache = reinterpret_cast<const void*>(16);
  p.kv_lens = reinterpret_cast<const int*>(16);
  p.out = reinterpret_cast<void*>(16);
  if (validate_decode(&p) != ATTN_OK || B == 0) return 0;
  if (2 + decode_counter_rows(B, Hq, Hkv) > attn::kDecodeCounterSlots) return 0;
  int sms = 0;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* s = nullptr;
    if (device_state_locked(&s) == ATTN_OK) sms = s->num_sms;
  }
  return decode_shape(Hq, Hkv, D, sms).bytes;
}

int attn_decode_ex(const attn_decode_params* p) {
  int st = validate_decode(p);
  if (st != ATTN_OK) return st;
  st = validate_rope(p->rope, p->D, p->Lmax);
  if (st != ATTN_OK) return st;
  if (p->B == 0) return ATTN_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  if (2 + decode_counter_rows(p->B, p->Hq, p->Hkv) > attn::kDecodeCounterSlots) return ATTN_ERR_UNSUPPORTED;
  const DecodeShape sh = decode_shape(p->Hq, p->Hkv, p->D, s->num_sms);
  st = ensure_workspace_locked(*s, sh.bytes, stream);
  if (st != ATTN_OK) return st;
  attn::DecodeLaunch L{};
  L.q = p->q;
  L.kcache = p->kcache;
  L.vcache = p->vcache;
  L.kv_lens = p->kv_lens;
  L.out = p->out;
  L.lse = p->lse;
  L.counters = static_cast<unsigned*>(s->ws);
  L.part_o = reinterpret_cast<float*>(static_cast<char*>(s->ws) + kCounterBytes);
  L.part_ml = L.part_o + sh.part_o_elems;
  L.B = p->B;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.Lmax = p->Lmax;
  L.D = p->D;
  L.min_keys = p->chunk > 0 ? p->chunk : 64;
  L.scale = p->scale;
  L.out_f32 = p->out_dtype == ATTN_DTYPE_F32;
  L.status = s->status;
  L.fault_skip_arrive = fault_skip_arrive();
  L.rope = rope_args(p->rope);
  L.stream = stream;
  return map_cuda(attn::launch_decode(L, s->num_sms));
}

int attn_decode_noalloc(const attn_decode_params* p) {
  int st = validate_decode(p);
  if (st != ATTN_OK) return st;
  st = validate_rope(p->rope, p->D, p->Lmax);
  if (st != ATTN_OK) return st;
  if (p->B == 0) return ATTN_OK;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  if (g_noalloc_ptr[dev] == nullptr) {
    // One-time set-up on this device (it is current).  Its memset and synchronise would invalidate a stream
    // capture in progress, so a first call made inside one is refused before anything touches the device.
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(static_cast<cudaStream_t>(p->stream), &cap) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    if (cap != cudaStreamCaptureStatusNone) return ATTN_ERR_INVALID_ARG;
    // Resolve the scratch array's device address.
    float* ptr = nullptr;
    if (cudaGetSymbolAddress(reinterpret_cast<void**>(&ptr), g_noalloc_scratch) != cudaSuccess || ptr == nullptr) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    // Its counter area must start at zero; the kernel keeps it zero afterwards.
    if (cudaMemset(ptr, 0, kCounterBytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    g_noalloc_ptr[dev] = ptr;
  }
  const DecodeShape sh = decode_shape(p->Hq, p->Hkv, p->D, s->num_sms);
  if (2 + decode_counter_rows(p->B, p->Hq, p->Hkv) > attn::kDecodeCounterSlots || sh.bytes > kNoAllocScratchBytes)
    return ATTN_ERR_SCRATCH_TOO_SMALL;
  attn::DecodeLaunch L{};
  L.q = p->q;
  L.kcache = p->kcache;
  L.vcache = p->vcache;
  L.kv_lens = p->kv_lens;
  L.out = p->out;
  L.lse = p->lse;
  L.counters = reinterpret_cast<unsigned*>(g_noalloc_ptr[dev]);
  L.part_o = g_noalloc_ptr[dev] + kCounterBytes / sizeof(float);
  L.part_ml = L.part_o + sh.part_o_elems;
  L.B = p->B;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.Lmax = p->Lmax;
  L.D = p->D;
  L.min_keys = p->chunk > 0 ? p->chunk : 64;
  L.scale = p->scale;
  L.out_f32 = p->out_dtype == ATTN_DTYPE_F32;
  L.status = s->status;
  L.fault_skip_arrive = fault_skip_arrive();
  L.rope = rope_args(p->rope);
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_decode(L, s->num_sms));
}

int attn_decode_paged(const attn_decode_paged_params* pp) {
  if (pp == nullptr) return ATTN_ERR_INVALID_ARG;
  if (pp->page_size < 8 || pp->page_size > 65536 || pp->max_pages < 1 || pp->num_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  const long long lmax = (long long)pp->max_pages * pp->page_size;
  if (lmax > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  // Validate everything else as the contiguous call does (same meaning of every other field).
  attn_decode_params p = {};
  p.q = pp->q;
  p.kcache = pp->kpages;
  p.vcache = pp->vpages;
  p.kv_lens = pp->kv_lens;
  p.out = pp->out;
  p.lse = pp->lse;
  p.B = pp->B;
  p.Hq = pp->Hq;
  p.Hkv = pp->Hkv;
  p.Lmax = (int)lmax;
  p.D = pp->D;
  p.scale = pp->scale;
  p.out_dtype = pp->out_dtype;
  p.chunk = pp->chunk;
  p.stream = pp->stream;
  p.rope = pp->rope;
  int st = validate_decode(&p);
  if (st != ATTN_OK) return st;
  st = validate_rope(p.rope, p.D, p.Lmax);
  if (st != ATTN_OK) return st;
  if (p.B == 0) return ATTN_OK;
  if (pp->block_table == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned4(pp->block_table)) return ATTN_ERR_ALIGNMENT;
  cudaStream_t stream = static_cast<cudaStream_t>(p.stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  if (2 + decode_counter_rows(p.B, p.Hq, p.Hkv) > attn::kDecodeCounterSlots) return ATTN_ERR_UNSUPPORTED;
  const DecodeShape sh = decode_shape(p.Hq, p.Hkv, p.D, s->num_sms);
  st = ensure_workspace_locked(*s, sh.bytes, stream);
  if (st != ATTN_OK) return st;
  attn::DecodeLaunch L{};
  L.q = p.q;
  L.kcache = p.kcache;
  L.vcache = p.vcache;
  L.block_table = pp->block_table;
  L.page_size = pp->page_size;
  L.max_pages = pp->max_pages;
  L.num_pages = pp->num_pages;
  L.kv_lens = p.kv_lens;
  L.out = p.out;
  L.lse = p.lse;
  L.counters = static_cast<unsigned*>(s->ws);
  L.part_o = reinterpret_cast<float*>(static_cast<char*>(s->ws) + kCounterBytes);
  L.part_ml = L.part_o + sh.part_o_elems;
  L.B = p.B;
  L.Hq = p.Hq;
  L.Hkv = p.Hkv;
  L.Lmax = p.Lmax;
  L.D = p.D;
  L.min_keys = p.chunk > 0 ? p.chunk : 64;
  L.scale = p.scale;
  L.out_f32 = p.out_dtype == ATTN_DTYPE_F32;
  L.status = s->status;
  L.fault_skip_arrive = fault_skip_arrive();
  L.rope = rope_args(p.rope);
  L.stream = stream;
  return map_cuda(attn::launch_decode(L, s->num_sms));
}

int attn_decode_multi(const attn_decode_multi_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->Lq < 1) return ATTN_ERR_INVALID_ARG;
  // Everything but q/out's token axis means what it means for attn_decode_ex.
  attn_decode_params d = {};
  d.q = p->q;
  d.kcache = p->kcache;
  d.vcache = p->vcache;
  d.kv_lens = p->kv_lens;
  d.out = p->out;
  d.lse = p->lse;
  d.B = p->B;
  d.Hq = p->Hq;
  d.Hkv = p->Hkv;
  d.Lmax = p->Lmax;
  d.D = p->D;
  d.scale = p->scale;
  d.out_dtype = p->out_dtype;
  d.stream = p->stream;
  int st = validate_decode(&d);
  if (st != ATTN_OK) return st;
  st = validate_rope(p->rope, p->D, p->Lmax);
  if (st != ATTN_OK) return st;
  if (p->B == 0) return ATTN_OK;
  const long long rows = (long long)(p->Hq / p->Hkv) * p->Lq;
  if (rows > 128) return ATTN_ERR_UNSUPPORTED;
  if ((long long)p->B * p->Hq * p->Lq > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (2 + (long long)p->B * p->Hkv > attn::kDecodeCounterSlots) return ATTN_ERR_UNSUPPORTED;
  cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  const DecodeMultiShape sh = decode_multi_shape(rows, p->D, s->num_sms);
  st = ensure_workspace_locked(*s, sh.bytes, stream);
  if (st != ATTN_OK) return st;
  attn::DecodeMultiLaunch L{};
  L.q = p->q;
  L.kcache = p->kcache;
  L.vcache = p->vcache;
  L.kv_lens = p->kv_lens;
  L.out = p->out;
  L.lse = p->lse;
  L.counters = static_cast<unsigned*>(s->ws);
  L.part_o = reinterpret_cast<float*>(static_cast<char*>(s->ws) + kCounterBytes);
  L.part_ml = L.part_o + sh.part_o_elems;
  L.B = p->B;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.Lq = p->Lq;
  L.Lmax = p->Lmax;
  L.D = p->D;
  L.scale = p->scale;
  L.out_f32 = p->out_dtype == ATTN_DTYPE_F32;
  L.num_sms = s->num_sms;
  L.status = s->status;
  L.rope = rope_args(p->rope);
  L.fault_skip_arrive = fault_skip_arrive();
  L.stream = stream;
  return map_cuda(attn::launch_decode_multi(L));
}

int attn_decode(const void* q, const void* kcache, const void* vcache, const int* kv_lens, void* out, float* lse,
                int B, int Hq, int Hkv, int Lmax, int D, float scale, void* stream) {
  attn_decode_params p = {};
  p.q = q;
  p.kcache = kcache;
  p.vcache = vcache;
  p.kv_lens = kv_lens;
  p.out = out;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Lmax = Lmax;
  p.D = D;
  p.scale = scale;
  p.out_dtype = ATTN_DTYPE_BF16;
  p.chunk = 0;
  p.stream = stream;
  return attn_decode_ex(&p);
}

int attn_fwd_ex(const attn_fwd_params* p) {
  int st = validate_fwd(p);
  if (st != ATTN_OK) return st;
  // positions reach Lkv - 1 (keys and the last query); a dense call with Lq > Lkv would place queries before 0
  st = validate_rope(p->rope, p->D, p->Lkv);
  if (st != ATTN_OK) return st;
  const bool rope_on = p->rope.style != ATTN_ROPE_NONE && p->rope.cos != nullptr;
  if (rope_on && p->cu_seqlens_q == nullptr && p->Lq > p->Lkv) return ATTN_ERR_INVALID_ARG;
  if (rope_on && p->rope.k_out != nullptr && !aligned16(p->rope.k_out)) return ATTN_ERR_ALIGNMENT;
  if (is_empty_fwd(p)) return ATTN_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
  DeviceState* s = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    st = device_state_locked(&s);
  }
  if (st != ATTN_OK) return st;
  const void* kk = p->k;
  const bool varlen = p->cu_seqlens_q != nullptr;
  const long long krows = varlen ? (long long)p->total_k * p->Hkv : (long long)p->B * p->Hkv * p->Lkv;
  const void* qq = p->q;
  const long long qrows = varlen ? (long long)p->total_q * p->Hq : (long long)p->B * p->Hq * p->Lq;
  if (rope_on && krows > 0) {
    // rotate the keys once (into k_out or the workspace) and the queries (into the workspace), then attend over
    // the rotated copies
    void* kdst = p->rope.k_out;
    void* qdst = nullptr;
    {
      const size_t kbytes = kdst == nullptr ? (size_t)krows * p->D * 2 : 0;
      std::lock_guard<std::mutex> lock(g_mu);
      st = ensure_workspace_locked(*s, kCounterBytes + kbytes + (size_t)qrows * p->D * 2, stream);
      if (st != ATTN_OK) return st;
      if (kdst == nullptr) kdst = static_cast<char*>(s->ws) + kCounterBytes;
      qdst = static_cast<char*>(s->ws) + kCounterBytes + kbytes;
    }
    attn::RopeRowsLaunch R{};
    R.src = p->k;
    R.dst = kdst;
    R.cu = varlen ? p->cu_seqlens_k : nullptr;
    R.B = p->B;
    R.H = p->Hkv;
    R.L = p->Lkv;
    R.D = p->D;
    R.total = p->total_k;
    R.rope = rope_args(p->rope);
    R.status = s->status;
    R.stream = stream;
    st = map_cuda(attn::launch_rope_rows(R));
    if (st != ATTN_OK) return st;
    kk = kdst;
    attn::RopeRowsLaunch Rq = R;  // query i of a sequence sits at i + Lkv - Lq
    Rq.src = p->q;
    Rq.dst = qdst;
    Rq.cu = varlen ? p->cu_seqlens_q : nullptr;
    Rq.cu_kv = varlen ? p->cu_seqlens_k : nullptr;
    Rq.H = p->Hq;
    Rq.L = p->Lq;
    Rq.total = p->total_q;
    Rq.pos_off = varlen ? 0 : p->Lkv - p->Lq;
    st = map_cuda(attn::launch_rope_rows(Rq));
    if (st != ATTN_OK) return st;
    qq = qdst;
  }
  attn::PrefillLaunch L{};
  L.q = qq;
  L.k = kk;
  L.v = p->v;
  L.out = p->out;
  L.lse = p->lse;
  L.B = p->B;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.Lq = p->Lq;
  L.Lkv = p->Lkv;
  L.D = p->D;
  L.scale = p->scale;
  L.causal = p->causal;
  L.out_f32 = p->out_dtype == ATTN_DTYPE_F32;
  L.cu_q = p->cu_seqlens_q;
  L.cu_k = p->cu_seqlens_k;
  L.total_q = p->total_q;
  L.total_k = p->total_k;
  L.num_sms = s->num_sms;
  L.status = s->status;
  L.fault_skip_arrive = fault_skip_arrive();
  L.stream = stream;
  return map_cuda(attn::launch_prefill(L));
}

int attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq, int Hkv, int Lq,
             int Lkv, int D, float scale, int causal, void* stream) {
  attn_fwd_params p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Lq = Lq;
  p.Lkv = Lkv;
  p.D = D;
  p.scale = scale;
  p.causal = causal;
  p.out_dtype = ATTN_DTYPE_BF16;
  p.stream = stream;
  return attn_fwd_ex(&p);
}

int attn_page_step(const attn_page_step_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->B < 0 || p->page_size < 1 || p->max_pages < 1 || p->num_pages < 1 || p->max_tokens < 0)
    return ATTN_ERR_INVALID_ARG;
  if (p->B > attn::kPageStepMaxRows || (long long)p->num_pages * p->page_size > kIntMax ||
      (long long)p->B * p->max_pages > kIntMax || (long long)p->max_pages * p->page_size > kIntMax)
    return ATTN_ERR_UNSUPPORTED;
  if (p->kv_lens == nullptr || p->block_table == nullptr || p->free_pages == nullptr || p->free_count == nullptr) {
    if (p->B > 0) return ATTN_ERR_INVALID_ARG;
  }
  if (!aligned4(p->kv_lens) || !aligned4(p->keep_lens) || !aligned4(p->new_lens) || !aligned4(p->block_table) ||
      !aligned4(p->free_pages) || !aligned4(p->free_count) || !aligned4(p->cu_new) || !aligned4(p->slots) ||
      !aligned4(p->positions))
    return ATTN_ERR_ALIGNMENT;
  if (p->B == 0) return ATTN_OK;
  DeviceState* s = nullptr;
  const int st = device_state(&s);
  if (st != ATTN_OK) return st;
  attn::PageStepLaunch L{};
  L.kv_lens = p->kv_lens;
  L.keep_lens = p->keep_lens;
  L.new_lens = p->new_lens;
  L.block_table = p->block_table;
  L.free_pages = p->free_pages;
  L.free_count = p->free_count;
  L.cu_new = p->cu_new;
  L.slots = p->slots;
  L.positions = p->positions;
  L.B = p->B;
  L.page_size = p->page_size;
  L.max_pages = p->max_pages;
  L.num_pages = p->num_pages;
  L.max_tokens = p->slots == nullptr && p->positions == nullptr ? 0 : p->max_tokens;
  L.status = s->status;
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_page_step(L));
}

int attn_qk_norm_rope(const attn_qk_norm_rope_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->B < 0 || p->L < 0 || p->Hq <= 0 || p->Hkv < 0 || p->D <= 0) return ATTN_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return ATTN_ERR_INVALID_ARG;
  const bool rope_on = p->rope.style != ATTN_ROPE_NONE && p->rope.cos != nullptr;
  int st = validate_rope(p->rope, p->D, 0);
  if (st != ATTN_OK) return st;
  if (p->B == 0 || p->L == 0) return ATTN_OK;
  if (p->q == nullptr || p->q_out == nullptr || (p->Hkv > 0 && (p->k == nullptr || p->k_out == nullptr)) ||
      (rope_on && p->positions == nullptr))
    return ATTN_ERR_INVALID_ARG;
  attn::QkNormRopeLaunch L{};
  const int q_extent[3] = {p->B, p->L, p->Hq}, k_extent[3] = {p->B, p->L, p->Hkv};
  if (!aligned16(p->q) || !aligned16(p->q_out) || !aligned16(p->q_weight) || !aligned16(p->k_weight) ||
      !aligned4(p->positions) || !take_strides8(p->q_stride, q_extent, 3, L.qs) ||
      !take_strides8(p->q_out_stride, q_extent, 3, L.qos))
    return ATTN_ERR_ALIGNMENT;
  if (p->Hkv > 0 && (!aligned16(p->k) || !aligned16(p->k_out) || !take_strides8(p->k_stride, k_extent, 3, L.ks) ||
                     !take_strides8(p->k_out_stride, k_extent, 3, L.kos)))
    return ATTN_ERR_ALIGNMENT;
  if ((long long)p->B * p->L > kIntMax || (long long)p->Hq + p->Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  DeviceState* s = nullptr;
  st = device_state(&s);
  if (st != ATTN_OK) return st;
  L.q = p->q;
  L.k = p->k;
  L.q_out = p->q_out;
  L.k_out = p->k_out;
  L.q_weight = p->q_weight;
  L.k_weight = p->k_weight;
  L.positions = p->positions;
  L.B = p->B;
  L.L = p->L;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.D = p->D;
  L.eps = p->eps;
  L.rope = rope_args(p->rope);
  L.status = s->status;
  L.stream = static_cast<cudaStream_t>(p->stream);
  L.num_sms = s->num_sms;
  return map_cuda(attn::launch_qk_norm_rope(L));
}

unsigned long long attn_kv_q4_page_bytes(int page_size, int Hkv, int D) {
  if (validate_pool_q4(Hkv, D, page_size, 1) != ATTN_OK) return 0;
  return (unsigned long long)(page_size / attn::kTileKeys) * Hkv * attn::kv_q4_tile_bytes(D);
}

int attn_kv_append_q4(const attn_kv_append_q4_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  int st = validate_pool_q4(p->Hkv, p->D, p->page_size, p->num_pages);
  if (st != ATTN_OK) return st;
  if (p->T < 0) return ATTN_ERR_INVALID_ARG;
  if (p->T == 0) return ATTN_OK;
  if (p->k == nullptr || p->v == nullptr || p->pool == nullptr || p->slots == nullptr) return ATTN_ERR_INVALID_ARG;
  attn::KvAppendQ4Launch L{};
  const int extent[2] = {p->T, p->Hkv};
  if (!aligned16(p->k) || !aligned16(p->v) || !aligned128(p->pool) || !aligned4(p->slots) ||
      !take_strides8(p->k_stride, extent, 2, L.ks) || !take_strides8(p->v_stride, extent, 2, L.vs))
    return ATTN_ERR_ALIGNMENT;
  DeviceState* s = nullptr;
  st = device_state(&s);
  if (st != ATTN_OK) return st;
  L.k = p->k;
  L.v = p->v;
  L.pool = p->pool;
  L.slots = p->slots;
  L.T = p->T;
  L.Hkv = p->Hkv;
  L.D = p->D;
  L.page_size = p->page_size;
  L.num_pages = p->num_pages;
  L.status = s->status;
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_kv_append_q4(L));
}

int attn_kv_gather_q4(const attn_kv_gather_q4_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  int st = validate_pool_q4(p->Hkv, p->D, p->page_size, p->num_pages);
  if (st != ATTN_OK) return st;
  if (p->B < 0 || p->max_pages < 1 || p->total_k < 0) return ATTN_ERR_INVALID_ARG;
  if ((long long)p->max_pages * p->page_size > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if (p->B == 0 || p->total_k == 0) return ATTN_OK;
  if (p->pool == nullptr || p->block_table == nullptr || p->cu_k == nullptr || p->k == nullptr || p->v == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned128(p->pool) || !aligned16(p->k) || !aligned16(p->v) || !aligned4(p->block_table) ||
      !aligned4(p->cu_k) || !aligned4(p->kv_starts))
    return ATTN_ERR_ALIGNMENT;
  DeviceState* s = nullptr;
  st = device_state(&s);
  if (st != ATTN_OK) return st;
  attn::KvGatherQ4Launch L{};
  L.pool = p->pool;
  L.block_table = p->block_table;
  L.cu_k = p->cu_k;
  L.kv_starts = p->kv_starts;
  L.k = p->k;
  L.v = p->v;
  L.B = p->B;
  L.Hkv = p->Hkv;
  L.D = p->D;
  L.page_size = p->page_size;
  L.max_pages = p->max_pages;
  L.num_pages = p->num_pages;
  L.total_k = p->total_k;
  L.status = s->status;
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_kv_gather_q4(L));
}

unsigned long long attn_decode_q4_workspace_bytes(int Hq, int Hkv, int Lq, int D) {
  if (validate_decode_q4_heads(Hq, Hkv, Lq, D) != ATTN_OK) return 0;
  DeviceState* s = nullptr;
  const int sms = device_state(&s) == ATTN_OK ? s->num_sms : 0;
  return decode_q4_shape(D, sms).bytes;
}

int attn_decode_q4(const attn_decode_q4_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  int st = validate_decode_q4_heads(p->Hq, p->Hkv, p->Lq, p->D);
  if (st != ATTN_OK) return st;
  st = validate_pool_q4(p->Hkv, p->D, p->page_size, p->num_pages);
  if (st != ATTN_OK) return st;
  if (p->B < 0 || p->max_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (p->out_dtype != ATTN_DTYPE_BF16 && p->out_dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (p->chunk < 0 || p->chunk > (1 << 20)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;
  if ((long long)p->max_pages * p->page_size > kIntMax - attn::kTileKeys) return ATTN_ERR_UNSUPPORTED;
  if (p->B == 0) return ATTN_OK;
  if (p->q == nullptr || p->pool == nullptr || p->block_table == nullptr || p->kv_lens == nullptr ||
      p->out == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned128(p->pool) || !aligned16(p->out) || !aligned16(p->workspace) ||
      !aligned4(p->block_table) || !aligned4(p->kv_lens) || !aligned4(p->lse))
    return ATTN_ERR_ALIGNMENT;
  if ((long long)p->B * p->Hq * p->Lq > kIntMax) return ATTN_ERR_UNSUPPORTED;
  cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  const DecodeQ4Shape sh = decode_q4_shape(p->D, s->num_sms);
  char* ws = static_cast<char*>(p->workspace);
  if (ws == nullptr) {
    // made for the larger D, so that it never has to grow under a graph that was captured with it
    const size_t bytes = decode_q4_shape(128, s->num_sms).bytes;
    st = ensure_buffer_locked(s->ws_q4, s->ws_q4_bytes, bytes, bytes, stream);
    if (st != ATTN_OK) return st;
    ws = static_cast<char*>(s->ws_q4);
  } else if (p->workspace_bytes < sh.bytes) {
    return ATTN_ERR_SCRATCH_TOO_SMALL;
  }
  attn::DecodeQ4Launch L{};
  L.q = p->q;
  L.pool = p->pool;
  L.block_table = p->block_table;
  L.kv_lens = p->kv_lens;
  L.out = p->out;
  L.lse = p->lse;
  L.counts = reinterpret_cast<unsigned*>(ws);
  L.part_o = reinterpret_cast<float*>(ws + sh.count_bytes);
  L.part_ml = L.part_o + sh.part_o_elems;
  L.B = p->B;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.Lq = p->Lq;
  L.D = p->D;
  L.page_size = p->page_size;
  L.max_pages = p->max_pages;
  L.num_pages = p->num_pages;
  L.min_tiles = p->chunk > 0 ? (p->chunk + attn::kTileKeys - 1) / attn::kTileKeys : 0;
  L.scale = p->scale;
  L.out_f32 = p->out_dtype == ATTN_DTYPE_F32;
  L.num_sms = s->num_sms;
  L.status = s->status;
  L.fault_skip_arrive = fault_skip_arrive();
  L.stream = stream;
  return map_cuda(attn::launch_decode_q4(L));
}

int attn_rope_tables(const attn_rope_tables_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->rows < 0 || p->start < 0 || p->rotary_dim <= 0) return ATTN_ERR_INVALID_ARG;
  if (p->scaling < ATTN_ROPE_SCALE_NONE || p->scaling > ATTN_ROPE_SCALE_INDEX) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->base) || p->base <= 1.0 || !std::isfinite((float)p->amplitude)) return ATTN_ERR_INVALID_ARG;
  if (p->scaling != ATTN_ROPE_SCALE_NONE && (!std::isfinite(p->factor) || p->factor <= 0.0)) return ATTN_ERR_INVALID_ARG;
  if ((p->scaling == ATTN_ROPE_SCALE_TURNS || p->scaling == ATTN_ROPE_SCALE_INDEX) &&
      !(std::isfinite(p->context) && p->context > 0.0 && p->low > 0.0 && p->high > p->low && std::isfinite(p->high)))
    return ATTN_ERR_INVALID_ARG;
  if (p->rotary_dim % 16 != 0 || p->rotary_dim > 2 * attn::kMaxRotaryPairs) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(rope_base(*p)) || rope_base(*p) <= 1.0) return ATTN_ERR_INVALID_ARG;
  if ((long long)p->start + p->rows > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if (p->rows == 0) return ATTN_OK;
  if (p->cos == nullptr || p->sin == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(p->cos) || !aligned16(p->sin)) return ATTN_ERR_ALIGNMENT;
  attn::RopeTablesLaunch L{};
  L.pairs = p->rotary_dim / 2;
  static_assert(attn::kMaxRotaryPairs <= 64, "rope_frequencies");
  double f[attn::kMaxRotaryPairs];
  rope_frequencies(*p, f);
  for (int i = 0; i < L.pairs; ++i) {
    const double turn = f[i] / kTwoPi;
    const double part = turn - std::floor(turn);  // whole turns a position say nothing (a factor below 1)
    if (!std::isfinite(part)) return ATTN_ERR_INVALID_ARG;
    L.turn[i] = part >= 0.5 ? (unsigned long long)((part - 0.5) * 0x1p64 + 0.5) + (1ull << 63)
                            : (unsigned long long)(part * 0x1p64 + 0.5);
  }
  DeviceState* s = nullptr;
  const int st = device_state(&s);
  if (st != ATTN_OK) return st;
  L.cos = p->cos;
  L.sin = p->sin;
  L.rows = p->rows;
  L.start = p->start;
  L.amplitude = (float)p->amplitude;
  L.num_sms = s->num_sms;
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_rope_tables(L));
}

int attn_kv_append_paged(const attn_kv_append_paged_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->T < 0 || p->Hq < 0 || p->Hkv <= 0 || p->D <= 0 || p->page_size < 1 || p->num_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return ATTN_ERR_UNSUPPORTED;
  const bool rope_on = p->rope.style != ATTN_ROPE_NONE && p->rope.cos != nullptr;
  int st = validate_rope(p->rope, rope_on ? p->rotary_dim : p->D, 0);
  if (st != ATTN_OK) return st;
  if (rope_on && p->rotary_dim <= 0) return ATTN_ERR_INVALID_ARG;
  if (rope_on && (p->rotary_dim % 16 != 0 || p->rotary_dim > p->D)) return ATTN_ERR_UNSUPPORTED;
  if ((p->q == nullptr) != (p->q_out == nullptr) || (p->q == nullptr) != (p->Hq == 0)) {
    if (p->T > 0) return ATTN_ERR_INVALID_ARG;
  }
  if (!rope_on && (p->q != nullptr || p->k_out != nullptr)) return ATTN_ERR_INVALID_ARG;
  if ((long long)p->num_pages * p->page_size > kIntMax || (long long)p->Hq + 2ll * p->Hkv > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (p->T == 0) return ATTN_OK;
  if (p->k == nullptr || p->v == nullptr || p->kpages == nullptr || p->vpages == nullptr || p->slots == nullptr ||
      (rope_on && p->positions == nullptr))
    return ATTN_ERR_INVALID_ARG;
  attn::KvAppendPagedLaunch L{};
  const int extent[2] = {p->T, p->Hkv}, q_extent[2] = {p->T, p->Hq};
  if (!aligned16(p->k) || !aligned16(p->v) || !aligned16(p->kpages) || !aligned16(p->vpages) || !aligned16(p->q) ||
      !aligned16(p->q_out) || !aligned16(p->k_out) || !aligned4(p->slots) || !aligned4(p->positions) ||
      !take_strides8(p->k_stride, extent, 2, L.ks) || !take_strides8(p->v_stride, extent, 2, L.vs))
    return ATTN_ERR_ALIGNMENT;
  if (p->q != nullptr && (!take_strides8(p->q_stride, q_extent, 2, L.qs) || !take_strides8(p->q_out_stride, q_extent, 2, L.qos)))
    return ATTN_ERR_ALIGNMENT;
  if (p->k_out != nullptr && !take_strides8(p->k_out_stride, extent, 2, L.kos)) return ATTN_ERR_ALIGNMENT;
  DeviceState* s = nullptr;
  st = device_state(&s);
  if (st != ATTN_OK) return st;
  L.k = p->k;
  L.v = p->v;
  L.q = p->q;
  L.kpages = p->kpages;
  L.vpages = p->vpages;
  L.q_out = p->q_out;
  L.k_out = p->k_out;
  L.slots = p->slots;
  L.positions = p->positions;
  L.T = p->T;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.D = p->D;
  L.page_size = p->page_size;
  L.num_pages = p->num_pages;
  L.rotary = rope_on ? p->rotary_dim : 0;
  L.rope = rope_args(p->rope);
  L.num_sms = s->num_sms;
  L.status = s->status;
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_kv_append_paged(L));
}

unsigned long long attn_decode_multi_paged_workspace_bytes(int Hq, int Hkv, int max_new, int D) {
  if (validate_decode_q4_heads(Hq, Hkv, max_new, D) != ATTN_OK) return 0;
  DeviceState* s = nullptr;
  const int sms = device_state(&s) == ATTN_OK ? s->num_sms : 152;
  return decode_multi_paged_bytes((long long)(Hq / Hkv) * max_new, D, sms);
}

int attn_decode_multi_paged(const attn_decode_multi_paged_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  int st = validate_decode_q4_heads(p->Hq, p->Hkv, p->max_new, p->D);  // (the same limits: 128 query rows a kv head)
  if (st != ATTN_OK) return st;
  if (p->B < 0 || p->T < 0 || p->page_size < 8 || p->page_size > 65536 || p->max_pages < 1 || p->num_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if (p->out_dtype != ATTN_DTYPE_BF16 && p->out_dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;
  if (p->page_size % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  // (a tile's keys past the last one stay countable: up to 127 more)
  if ((long long)p->max_pages * p->page_size > kIntMax - 128 || (long long)p->num_pages * p->Hkv > kIntMax ||
      (long long)p->T * p->Hq > kIntMax)
    return ATTN_ERR_UNSUPPORTED;
  if (p->B == 0 || p->T == 0) return ATTN_OK;
  if (p->q == nullptr || p->kpages == nullptr || p->vpages == nullptr || p->block_table == nullptr ||
      p->kv_lens == nullptr || p->cu_new == nullptr || p->out == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->kpages) || !aligned16(p->vpages) || !aligned16(p->out) ||
      !aligned16(p->workspace) || !aligned4(p->block_table) || !aligned4(p->kv_lens) || !aligned4(p->cu_new) ||
      !aligned4(p->lse))
    return ATTN_ERR_ALIGNMENT;
  if (2 + (long long)p->B * p->Hkv > attn::kDecodeCounterSlots) return ATTN_ERR_UNSUPPORTED;
  cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  const long long rows = (long long)(p->Hq / p->Hkv) * p->max_new;
  char* ws = static_cast<char*>(p->workspace);
  if (ws == nullptr) {
    // made for the largest call, so that it never has to grow under a graph that was captured with it
    const size_t bytes = decode_multi_paged_bytes(128, 128, s->num_sms);
    st = ensure_buffer_locked(s->ws_paged, s->ws_paged_bytes, bytes, bytes, stream);
    if (st != ATTN_OK) return st;
    ws = static_cast<char*>(s->ws_paged);
  } else if (p->workspace_bytes < decode_multi_paged_bytes(rows, p->D, s->num_sms)) {
    return ATTN_ERR_SCRATCH_TOO_SMALL;
  }
  attn::DecodeMultiLaunch L{};
  L.q = p->q;
  L.kcache = p->kpages;
  L.vcache = p->vpages;
  L.block_table = p->block_table;
  L.cu_new = p->cu_new;
  L.T = p->T;
  L.page_size = p->page_size;
  L.max_pages = p->max_pages;
  L.num_pages = p->num_pages;
  L.kv_lens = p->kv_lens;
  L.out = p->out;
  L.lse = p->lse;
  L.rows_ws = ws;
  L.B = p->B;
  L.Hq = p->Hq;
  L.Hkv = p->Hkv;
  L.Lq = p->max_new;
  L.Lmax = p->max_pages * p->page_size;
  L.D = p->D;
  L.scale = p->scale;
  L.out_f32 = p->out_dtype == ATTN_DTYPE_F32;
  L.num_sms = s->num_sms;
  L.status = s->status;
  L.fault_skip_arrive = fault_skip_arrive();
  L.stream = stream;
  if (rows <= attn::decode_rows_max(p->D)) return map_cuda(attn::launch_decode_rows(L));
  ws += decode_rows_region(s->num_sms);
  L.counters = reinterpret_cast<unsigned*>(ws);
  L.part_o = reinterpret_cast<float*>(ws + kCounterBytes);
  L.part_ml = L.part_o + decode_multi_shape(rows, p->D, s->num_sms).part_o_elems;
  return map_cuda(attn::launch_decode_multi(L));
}

int attn_verify_drafts(const attn_verify_drafts_params* p) {
  if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (p->B < 0 || p->K < 0 || p->V < 1 || (p->cu_target != nullptr && p->total < 0)) return ATTN_ERR_INVALID_ARG;
  if (p->dtype != ATTN_DTYPE_BF16 && p->dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (p->K >= (1 << 20) || p->V >= (1 << 30) || (long long)p->B * (p->K + 1) >= (1 << 28)) return ATTN_ERR_UNSUPPORTED;
  if (p->B == 0) return ATTN_OK;
  // (with cu_target and no rows at all no sequence has any, and the probabilities are never read)
  if ((p->target_probs == nullptr && (p->cu_target == nullptr || p->total > 0)) || p->uniforms == nullptr ||
      p->tokens == nullptr || p->accepted == nullptr || (p->K > 0 && p->draft_tokens == nullptr) ||
      (p->kv_lens == nullptr) != (p->keep_lens == nullptr))
    return ATTN_ERR_INVALID_ARG;
  const unsigned mask = p->dtype == ATTN_DTYPE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(p->target_probs) & mask) || (reinterpret_cast<uintptr_t>(p->draft_probs) & mask) ||
      !aligned4(p->draft_tokens) || !aligned4(p->uniforms) || !aligned4(p->cu_target) || !aligned4(p->draft_lens) ||
      !aligned4(p->kv_lens) || !aligned4(p->tokens) || !aligned4(p->accepted) || !aligned4(p->keep_lens))
    return ATTN_ERR_ALIGNMENT;
  DeviceState* s = nullptr;
  const int st = device_state(&s);
  if (st != ATTN_OK) return st;
  attn::VerifyDraftsLaunch L{};
  L.drafts = p->draft_tokens;
  L.target = p->target_probs;
  L.draft = p->K > 0 ? p->draft_probs : nullptr;
  L.uniforms = p->uniforms;
  L.cu = p->cu_target;
  L.draft_lens = p->cu_target == nullptr ? p->draft_lens : nullptr;
  L.kv_lens = p->kv_lens;
  L.tokens = p->tokens;
  L.accepted = p->accepted;
  L.keep_lens = p->keep_lens;
  L.B = p->B;
  L.K = p->K;
  L.V = p->V;
  L.total = p->total;
  L.f32 = p->dtype == ATTN_DTYPE_F32;
  // the strides of axes of one element say nothing
  L.ts[0] = p->cu_target == nullptr && p->B > 1 ? p->target_stride[0] : 0;
  L.ts[1] = (p->cu_target == nullptr ? p->K + 1 : p->total) > 1 ? p->target_stride[1] : 0;
  L.ds[0] = p->B > 1 ? p->draft_stride[0] : 0;
  L.ds[1] = p->K > 1 ? p->draft_stride[1] : 0;
  L.num_sms = s->num_sms;
  L.status = s->status;
  L.stream = static_cast<cudaStream_t>(p->stream);
  return map_cuda(attn::launch_verify_drafts(L));
}

int attn_get_device_status(void* stream) {
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* s = nullptr;
  int st = device_state_locked(&s);
  if (st != ATTN_OK) return st;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  unsigned v = 0;
  if (cudaMemcpy(&v, s->status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return ATTN_ERR_CUDA;
  const unsigned zero = 0;
  if (cudaMemcpy(s->status, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return ATTN_ERR_CUDA;
  if (v == ATTN_ERR_DEVICE_TIMEOUT) {
    // A decode that gave up part-way may have left its work counters armed, or partials unread: clear them, with no
    // decode of another stream on the device.
    int dev = -1;
    cudaGetDevice(&dev);
    cudaDeviceSynchronize();
    if (s->ws != nullptr) cudaMemset(s->ws, 0, kCounterBytes);
    if (s->ws_q4 != nullptr) cudaMemset(s->ws_q4, 0, s->ws_q4_bytes);
    if (s->ws_paged != nullptr) cudaMemset(s->ws_paged, 0, s->ws_paged_bytes);
    if (dev >= 0 && dev < kMaxDevices && g_noalloc_ptr[dev] != nullptr) cudaMemset(g_noalloc_ptr[dev], 0, kCounterBytes);
    cudaDeviceSynchronize();
    cudaGetLastError();
  }
  return static_cast<int>(v);
}

void attn_release_workspace(void) {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return;
  }
  DeviceState& s = g_dev[dev];
  if (s.ws != nullptr) cudaFree(s.ws);
  s.ws = nullptr;
  s.ws_bytes = 0;
  if (s.ws_q4 != nullptr) cudaFree(s.ws_q4);
  s.ws_q4 = nullptr;
  s.ws_q4_bytes = 0;
  if (s.ws_paged != nullptr) cudaFree(s.ws_paged);
  s.ws_paged = nullptr;
  s.ws_paged_bytes = 0;
}

}  // extern "C"
