// decode_q4.cu -- decode attention over the 4-bit paged KV cache (layout: kv_q4.h), one or several new tokens a
// sequence, split along the keys, with the log-sum-exp combine in the same launch.
//
// A cached row x of a group of 64 dims reads back as s u + m, u in 0..15.  So
//   q . k   = sum over groups of  s_k (q . u_k) + m_k (sum of q over the group)
//   sum p v = sum over keys of    (p s_v) u_v   + (sum of p m_v)
// and the matrix products run over the codes themselves: scales and minima are applied to scores and weights, once per
// key and group, not once per element.
//
// What bounds it: 0.5625 bytes an element and 4 heads an element leave 3.5 times fewer bytes than bf16 for the same
// arithmetic.  At the copy bandwidth an SM takes some 40 elements a clock; four heads' multiply-adds alone would
// exceed its fp32 units.  So products run on the tensor cores -- mma.sync m16n8k16 in fp16, whose A operand
// comes straight from registers: K^T and V^T tiles are 16 keys (dims) by 16, the 8 columns are the query rows of one
// kv head.  A tcgen05 product would need the unpacked tile written to shared or tensor memory first, four times the
// bytes of the codes, for an N of 8: 37 against 30 us for 32 query rows over 8 x 4096 keys.  (Over long caches those rows
// would gain by it, 179 against 214 us at 131k keys; this kernel has no such variant, and with 32 rows it takes longer than
// bf16 does: 218 us for 313,590 keys, attn_decode_multi 199.8 us for 327,680 of 3.6 times the bytes.)  mma.sync on 8-bit
// floats (codes are e4m3 as they are, q two terms) runs at fp16's rate and converts its operands on the way (72 against
// 65 us at 131k keys).
//  * Unpacking costs one mask per two elements: (w & 0x000f000f) is, as a pair of fp16, the subnormals u 2^-24, and
//    (w & 0x00f000f0) is u 2^-20, both exact; the factors go into q (2^10 and 2^6, q first scaled by a power of two
//    to a largest element in [16, 32), which is exact) and, for V, into the output.  One shift by 8 gives the
//    other two pairs of a word.  For V, whose pairs run along keys, a byte permute first joins two keys' halves.
//  * Scores come as S^T (keys by query rows), so a row's maximum is two registers and three shuffles for 32 keys,
//    and the weights turn into the second product's B operand by two 8x8 transposes (movmatrix).  With up to four query
//    rows each has two of the eight columns and a lane keeps one: half the softmax work of four columns left empty.
//  * Weights are p s_v 2^x rounded to fp16, each off by at most 2^-11 of itself: 2^-11 of the sum of |p s u| for O, in which
//    these terms and the p m cancel, against the output's own rounding, 2^-8 of what is left.  Each warp chooses x by the
//    largest scale s of the keys of a step (32, or 48 at D = 64): a weight stays below 2^15, and that scale times 2^x at 2^9 or
//    above, so that what falls below fp16's normal range is off by 2^-34 of that scale at most.  (Scales or-ed together in
//    place of their maximum gave x up to 14 too low, and 68.9 us over 131k keys with scales on both sides of 2, now 64.0.)
//    A call with fp32 output carries weights as two fp16 terms.  Maxima, sums,
//    the term in m_v and all accumulators are fp32.  The matrix unit truncates as it adds to an accumulator, one add for 16
//    keys: over a slice of 131,072 keys, 2048 adds a warp, that biases O by some 2^-13 of its terms' sum, below the 2^-11
//    that a weight's rounding is off by at most.  With fp32 output each tile's products start from zero and are added with
//    rounding (131k keys 71.1 against 66.3 us, 8 x 4096 14.3 against 13.9 us; 32 query rows over 131k 317 against 300 us).
// At long contexts the instructions bound it: 243 a tile of 16 keys at D = 128 (all that a launch executes over its tiles), 40
// of them masks and shifts for K, 48 with the byte permutes for V, at two clocks each (dropping either product's unpacking
// and matrix products reaches the 60 us that the copies alone take of the 64); over short ones the chain of a launch:
// lengths, split, block table and first
// copies (1.6 us), first data (4 us), a row's stages at 0.6 us each, exchange and merge (2 to 3 us).
// Measured (CUDA-graph replays over rotating pools, 32 query and 8 kv heads, D = 128): 4 sequences of 32k to 131k keys 64.1 us
// (5.6 TB/s, 0.83 of the copy bandwidth), 8 of 512 to 4096 keys 14.0 us, one of 4096 keys 11.4 us; 64 of up to 700 keys with
// 16 heads of D = 64 16.9 us; 8 tokens each over 8 x 4096 keys 30.3 us.  Two CTAs of seven consumer warps an SM: 70.3 /
// 15.0 / - / 22.0 us against 70.8 / 14.3 / - / 16.6 us that day; four tiles a warp and stage 70.5 / 16.7 / - / 19.1 us;
// four CTAs at 96 registers 86 / 18.9 us (spills).  At D = 64 two, three, four tiles a warp and stage: 16 heads over 4 x 16k to
// 64k keys 45.1, 37.9, 36.2 us, the 64 short sequences 16.0, 16.1, 18.3 us.
// The split is decode.cu's: persistent CTAs take equal slices of the tiles of all (sequence, kv head, row chunk) rows, a
// producer warp streams them with bulk copies (one copy per page and stage) into a shared-memory ring.  At a piece's
// end each warp sums a quarter of the accumulators over the warps; the pieces of a row split between CTAs are published and
// counted, and who counts the last one merges them, so no CTA depends on another that may not have started.  (One count and
// a fence for it: 21.4 against 16.1 us over the 64 short sequences; one flag a warp, released and acquired: 17.0 us, 16.0
// against 14.4 us over the 8: a release waits 2 to 4 us for its stores while the cache streams.  The CTA of the first piece
// waiting for the others' words, with no counts: 63.9 / 13.4 / 11.2 / 15.8 / 29.6 us for the list above, but CUDA does not
// promise that the CTAs it waits for start; tickets that make them run, slices dealt from the back: 70.3 / 14.1 / 14.1 / 16.9 /
// 31.8 us, a cooperative launch: 68.1 / 13.4 / 14.4 / 16.3 / 30.8 us.)
#include <cfloat>
#include <algorithm>
#include <cmath>
#include <cuda_fp16.h>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv_q4.h"
#include "rope.cuh"
#include "slice_map.h"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Tiles charged to every row for its piece-end work (8 x 4096 GQA / 64 short rows of D = 64: 8 tiles 15.4 / 22.9 us, 16
// 14.4 / 21.1, 32 14.5 / 22.0, with the merge of that day).
constexpr int kRowCostTiles = 16;
// From this many tiles a CTA at the caches' capacity on, 16 query rows a CTA (two CTAs an SM, each tile unpacked once for
// all 16) beat 8 (three): 32 rows over 131k keys 213 against 252 us; below, 8 rows win by their cheaper piece ends: 32
// rows over 8 x 4096 keys 29.4 against 31.1 us, 16 rows 18.7 against 24.3 us.  The lengths are on the device, so this reads the
// tables' width: over tables 32 times wider than 8 requests of 512 to 4096 keys need, 16 rows take 26.9 us (19.8 over tight
// ones), 32 rows 32.9 (28.8).
constexpr long long kWideTiles = 256;

// R4: groups of 4 query rows a CTA serves (1, 2 or 4).
template <int D, int R4>
struct Q4Cfg {
  static constexpr int G = D / 64;                      // scale groups of a row
  static constexpr int ROWS = 4 * R4;                   // query rows per CTA
  static constexpr int NT = (R4 + 1) / 2;               // column tiles of the second product
  static constexpr int NC = R4 == 1 ? 1 : 2;            // query rows a lane keeps of each
  static constexpr int NW = 4;                          // consumer warps
  static constexpr int KT = D == 64 ? 3 : 2;            // tiles of a stage per consumer warp
  static constexpr int ST = NW * KT;                    // tiles per stage
  static constexpr int TILE = kv_q4_tile_bytes(D);
  static constexpr int STAGE = ST * TILE;
  static constexpr int MINB = NT == 1 ? 3 : 2;          // resident CTAs per SM
  static constexpr int NS = D == 64 ? 5 : 4;            // ring stages
  static constexpr int THREADS = 32 * (NW + 1);
  static constexpr int LENS_CACHE = 512;                // kv_lens kept in shared memory for the walk
  static constexpr int OWN = kDecodeQ4Owners;           // warps that gather the accumulators at a piece's end,
  static constexpr int OW = 4 * G / OWN;                // each this many of a column group
  static constexpr int SCR_BYTES = OWN * (NW - 1) * NT * OW * 512;  // [owner][other warps][NT][OW][lane] float4
  static constexpr bool SCR_IN_STAGE = SCR_BYTES <= STAGE;  // the exchange takes the piece's last stage, or its own room
  static constexpr int OFF_SCR = NS * STAGE;
  static constexpr int OFF_BAR = OFF_SCR + (SCR_IN_STAGE ? 0 : SCR_BYTES);  // full[NS], empty[NS], told[NS]
  static constexpr int OFF_INFO = OFF_BAR + 3 * NS * 8;
  static constexpr int OFF_ML = OFF_INFO + NS * 32;     // (m, l) [NW][8 NT]
  static constexpr int OFF_LENS = OFF_ML + NW * 8 * NT * 8;
  static constexpr int OFF_MISC = OFF_LENS + LENS_CACHE * 4;
  static constexpr int SMEM = OFF_MISC + 16;
  static_assert(OWN == NW && 4 * G % OWN == 0, "every warp owns as many accumulators");
  static_assert(OFF_BAR % 16 == 0 && OFF_ML % 8 == 0, "aligned regions");
  static_assert(MINB * (SMEM + 1024) <= 228 * 1024, "MINB CTAs per SM");
  static_assert(ST <= 32, "a stage spans at most one page per lane");
};

// What the first stage of a row piece tells about the piece.
struct Q4PieceInfo {
  int b;       // sequence; -1 marks the end of the work
  int hg;      // kv head * chunks + chunk
  int tile0;   // the piece's first tile of the sequence
  int tiles;   // and their number
  int len;     // keys of the sequence
  int np;      // CTAs holding a piece of this row (0: no keys, 1: whole row here)
  int c_lo;    // the first of them
};

__device__ __forceinline__ int clamp_len(int len, int Lmax) { return len < 0 ? 0 : (len > Lmax ? Lmax : len); }

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t half2_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ float2 half2_floats(uint32_t w) { return __half22float2(as_half2(w)); }

constexpr uint32_t kLowNibble = 0x000f000fu, kHighNibble = 0x00f000f0u;

// WIDE: the weights of the second product as two fp16 terms (fp32 output).
template <int D, int R4, bool WIDE>
__global__ void __launch_bounds__(Q4Cfg<D, R4>::THREADS, Q4Cfg<D, R4>::MINB)
    decode_q4_kernel(const DecodeQ4Launch p, const int chunks, const int rows) {
  using C = Q4Cfg<D, R4>;
  constexpr int G = C::G, NT = C::NT, NC = C::NC;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NS;
  uint64_t* told = empty + C::NS;  // a piece's record is written (its data may still be on the way)
  Q4PieceInfo* info = reinterpret_cast<Q4PieceInfo*>(smem + C::OFF_INFO);
  float2* mlbuf = reinterpret_cast<float2*>(smem + C::OFF_ML);
  int* lens_s = reinterpret_cast<int*>(smem + C::OFF_LENS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Hg = p.Hkv * chunks;  // rows per sequence
  const int cta = blockIdx.x;
  const int Lmax = p.max_pages * p.page_size;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::NW);
      mbar_init(&told[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  const int len_first = (warp == C::NW && lane < p.B) ? p.kv_lens[lane] : 0;
  __syncthreads();

  if (warp == C::NW) {
    // ---------------- producer: walk this CTA's slice of the tiles ----------------
    long long tsum = 0;
    int nonempty = 0;
    for (int b = lane; b < p.B; b += 32) {
      const int raw = (b == lane) ? len_first : p.kv_lens[b];
      const int len = clamp_len(raw, Lmax);
      if (raw != len && cta == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
      if (b < C::LENS_CACHE) lens_s[b] = len;
      tsum += (len + kTileKeys - 1) / kTileKeys;
      nonempty += len > 0 ? 1 : 0;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      tsum += __shfl_xor_sync(0xffffffffu, tsum, off);
      nonempty += __shfl_xor_sync(0xffffffffu, nonempty, off);
    }
    __syncwarp();
    auto seq_len = [&](int b) -> int { return b < C::LENS_CACHE ? lens_s[b] : clamp_len(p.kv_lens[b], Lmax); };
    auto seq_tiles = [&](int b) -> int { return (seq_len(b) + kTileKeys - 1) / kTileKeys; };
    const long long W = tsum * Hg;
    // Slices of at least min_tiles tiles, but never fewer slices than rows with keys.  By default a slice's time is not
    // to fall far below the merge of the partials it makes: with T tiles a row in slices of s, both (T / s and s) are
    // alike at s ~ sqrt(T); 2 sqrt(T) measured best over one sequence of 4096 keys (11.8 us against 16.5 us with slices of
    // 4 tiles, sqrt(2 T) 11.2 us) and eight (14.1 against 14.4 us, 14.1 us).
    int min_tiles = p.min_tiles;
    if (min_tiles == 0) min_tiles = max(4, (int)(2.f * sqrtf(to_f32(W) / (float)max(1, nonempty * Hg))));
    long long geff = floor_div(W + min_tiles - 1, min_tiles);
    if (geff < (long long)nonempty * Hg) geff = (long long)nonempty * Hg;
    if (geff > (long long)gridDim.x) geff = gridDim.x;
    if (geff < 1) geff = 1;
    // Every row occupies [rs, rs + kRowCostTiles + tiles) of the cost space, its tiles last.
    const long long Wc = W + (long long)kRowCostTiles * nonempty * Hg;
    const SliceMap sm = make_slice_map(Wc, geff, C::MINB, gridDim.x);
    const long long lo = sm.start(cta);
    const long long hi = sm.start(cta + 1);

    int t = 0;  // stages issued
    bool ok = true;
    const uint64_t policy = l2_policy_evict_first();  // the cache is read once
    const int tpp = p.page_size / kTileKeys;
    int win_b = -1, win_base = 0, my_page = 0;  // lane i: block-table entry of page win_base + i of sequence win_b
    auto need_pages = [&](int b, int first, int last) {
      if (b == win_b && first >= win_base && last < win_base + 32) return;
      win_b = b;
      win_base = first;
      const int pg = first + lane;
      my_page = 0;
      if (pg < p.max_pages && (long long)pg * p.page_size < seq_len(b))
        my_page = p.block_table[(size_t)b * p.max_pages + pg];
    };
    // Tiles [t0, t0 + nt) of (b, hkv) to dst: lane j copies the part on the run's page first + j.
    auto copy_tiles = [&](int b, int hkv, int t0, int nt, uint8_t* dst, uint64_t* bar) {
      const int first = t0 / tpp, last = (t0 + nt - 1) / tpp;
      need_pages(b, first, last);
      const int pg = first + lane;
      int page = __shfl_sync(0xffffffffu, my_page, min(pg, last) - win_base);
      if (pg <= last) {
        if (page < 0 || page >= p.num_pages) {
          record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);  // out-of-pool page id: read page 0 instead
          page = 0;
        }
        const int tl = max(t0, pg * tpp), th = min(t0 + nt, (pg + 1) * tpp);
        bulk_g2s_hint(dst + (size_t)(tl - t0) * C::TILE,
                      reinterpret_cast<const uint8_t*>(p.pool) + kv_q4_tile_at(page, hkv, tl - pg * tpp, p.Hkv, tpp, D),
                      (uint32_t)(th - tl) * C::TILE, bar, policy);
      }
    };
    auto wait_empty = [&](int slot_r) -> bool {
      int okw = 1;
      if (lane == 0) okw = mbar_wait(&empty[slot_r], ((t / C::NS) - 1) & 1, p.status, abort_flag) ? 1 : 0;
      return __shfl_sync(0xffffffffu, okw, 0) != 0;
    };
    // Stream tiles [tb, te) of row (b, hg), whose tiles sit at cost positions [ks, ks + tiles); te == tb emits one
    // empty stage (a sequence with no keys).
    auto emit = [&](int b, int hg, int tb, int te, long long ks) -> bool {
      const int hkv = hg / chunks;
      const int n = te - tb;
      const int nst = n > 0 ? (n + C::ST - 1) / C::ST : 1;
      int np = 0, row_lo = 0;
      for (int u = 0; u < nst; ++u, ++t) {
        const int slot_r = t % C::NS;
        if (t >= C::NS && !wait_empty(slot_r)) return false;
        const int t0 = tb + u * C::ST;
        const int nt = n > 0 ? min(C::ST, te - t0) : 0;
        if (lane == 0) {
          if (nt > 0) mbar_expect_tx(&full[slot_r], (uint32_t)nt * C::TILE);
        }
        __syncwarp();
        if (nt > 0) copy_tiles(b, hkv, t0, nt, smem + slot_r * C::STAGE, &full[slot_r]);
        if (u == 0 && nt > 0) {
          // Which CTAs hold a piece of this row.
          const long long last = ks + seq_tiles(b) - 1;
          int c_lo = 0, c_hi = cta;
          for (int top = cta;; top -= 32) {  // c_lo: the largest c <= cta with start(c) <= ks
            const unsigned m = __ballot_sync(0xffffffffu, top - lane >= 0 && sm.starts_by(top - lane, ks));
            if (m) {
              c_lo = top - (__ffs(m) - 1);
              break;
            }
          }
          for (int bot = cta + 1;; bot += 32) {  // c_hi: the largest c with start(c) <= last
            const unsigned m = __ballot_sync(0xffffffffu, bot + lane >= sm.g || !sm.starts_by(bot + lane, last));
            if (m) {
              c_hi = bot + (__ffs(m) - 1) - 1;
              break;
            }
          }
          np = c_hi - c_lo + 1;
          row_lo = c_lo;
        }
        if (lane == 0) {
          if (u == 0) {
            Q4PieceInfo pi;
            pi.b = b;
            pi.hg = hg;
            pi.tile0 = tb;
            pi.tiles = n;
            pi.len = seq_len(b);
            pi.np = np;
            pi.c_lo = row_lo;
            info[slot_r] = pi;
          }
          mbar_arrive(&told[slot_r]);  // every stage, so that its phases run with the others'
          mbar_arrive(&full[slot_r]);
        }
      }
      return true;
    };

    if (lo < hi) {
      // the row whose cost interval holds position lo: sequences 32 at a time
      long long acc = 0;  // first cost position of sequence b
      int b = 0, nt = 0;
      int next_nt = lane < p.B ? seq_tiles(lane) : 0;
      for (int b32 = 0;; b32 += 32) {
        const int my_nt = next_nt;
        next_nt = b32 + 32 + lane < p.B ? seq_tiles(b32 + 32 + lane) : 0;  // (on its way, past the lengths kept here)
        const long long mine = my_nt > 0 ? Hg * ((long long)my_nt + kRowCostTiles) : 0;
        long long upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, acc + upto > lo);
        if (past != 0) {
          const int src = __ffs(past) - 1;
          acc += __shfl_sync(0xffffffffu, upto - mine, src);
          nt = __shfl_sync(0xffffffffu, my_nt, src);
          b = b32 + src;
          break;
        }
        acc += __shfl_sync(0xffffffffu, upto, 31);
      }
      long long rcost = (long long)nt + kRowCostTiles;
      int hg = (int)floor_div(lo - acc, rcost);
      long long rs = acc + (long long)hg * rcost;
      long long pos = lo;
      while (ok && pos < hi) {
        const long long ks = rs + kRowCostTiles;
        const long long a = max(pos, ks), e = min(hi, ks + nt);
        if (a < e) ok = emit(b, hg, (int)(a - ks), (int)(e - ks), ks);
        pos = rs + rcost;
        rs += rcost;
        if (++hg == Hg) {
          hg = 0;
          for (++b; b < p.B; ++b) {
            nt = seq_tiles(b);
            if (nt > 0) break;
          }
          rcost = (long long)nt + kRowCostTiles;
        }
      }
    }
    if (nonempty < p.B) {  // rows of sequences with no keys, one row per CTA in turn
      for (long long e = cta; ok && e < (long long)p.B * Hg; e += gridDim.x) {
        const int b = (int)floor_div(e, Hg);
        if (seq_len(b) == 0) ok = emit(b, (int)(e - (long long)b * Hg), 0, 0, 0);
      }
    }
    if (ok) {  // end-of-work marker
      const int slot_r = t % C::NS;
      if (t < C::NS || wait_empty(slot_r)) {
        if (lane == 0) {
          info[slot_r].b = -1;
          mbar_arrive(&told[slot_r]);
        }
      }
    }
    if (lane == 0 && *abort_flag) {
      // Let copies already in flight land before the CTA's shared memory is released.
      for (int u = (t > C::NS ? t - C::NS : 0); u < t; ++u)
        mbar_wait(&full[u % C::NS], (u / C::NS) & 1, p.status, nullptr);
    }
    return;
  }

  // ---------------- consumers ----------------
  constexpr int nct = C::NW * 32;
  const int g = lane >> 2, t4 = lane & 3;
  const int kg = g ^ ((g >> 2) & 1);             // key of the tile's score row g (row g + 8: kg + 8)
  const int kv0 = 2 * t4 + (t4 >> 1);            // keys of score rows 2 t4 and 2 t4 + 1: this order keeps
  const int kv1 = 2 * t4 + 1 - (t4 >> 1);        // the four lanes' 32-byte rows in different banks, for K and for V
  // The test hook withholds CTA 0's release of its second stage: the producer's bounded wait then runs out.
  int to_skip = p.fault_skip_arrive && cta == 0 ? 1 : -1;
  int slot = 0;
  uint32_t phase = 0;  // of the ring
  auto release = [&]() {
    if (lane == 0 && to_skip != 0) mbar_arrive(&empty[slot]);
    --to_skip;
    if (++slot == C::NS) {
      slot = 0;
      phase ^= 1;
    }
  };

  // A wait can run out in one warp and just succeed in another (not in lanes of one warp, which test in one instruction).  So
  // every warp takes part in two barriers for each record, the end's among them; the second tells whether any gave up.
  auto wait = [&](uint64_t* bar) -> bool { return mbar_wait(bar, phase, p.status, abort_flag); };
  auto leave = [&](bool gave_up) {
    named_bar_sync(1, nct);
    named_bar_any(1, nct, gave_up);
  };

  while (true) {
    if (!wait(&told[slot])) {
      leave(true);
      break;
    }
    const Q4PieceInfo si = info[slot];
    if (si.b < 0) {
      leave(false);
      break;
    }
    const int hkv = si.hg / chunks;
    const int row0 = (si.hg - hkv * chunks) * C::ROWS;  // first query row of the kv head this CTA serves
    const int len = si.len;
    // ---- q of the piece, as the first product's B operand: column 2 t + c of column tile nt is query row
    // 8 nt + 4 c + t (with up to 4 rows, row t twice), so that every lane's scores are of rows there are ----
    uint32_t qf[NT][4 * G][2];
    float f[NT][NC], qs[NT][G][NC];  // of row 8 nt + 4 c + t4: score factor (>= 0), q's sums
    int vis[NT][NC];                 // keys it sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + 8 * nt + (NC == 2 ? 4 * (g & 1) : 0) + (g >> 1);
      const __nv_bfloat16* qrow = reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                  (((size_t)si.b * p.Hkv + hkv) * rows + min(r, rows - 1)) * D;
      float v[G][16];
      float amax = 0.f;
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        const uint4* src = reinterpret_cast<const uint4*>(qrow + 64 * gg + 16 * t4);
        const uint4 w0 = __ldg(src), w1 = __ldg(src + 1);
        unpack8(w0, *reinterpret_cast<float(*)[8]>(v[gg]));
        unpack8(w1, *reinterpret_cast<float(*)[8]>(v[gg] + 8));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          v[gg][j] = r < rows ? v[gg][j] : 0.f;
          amax = fmaxf(amax, fabsf(v[gg][j]));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // e with 2^e <= amax < 2^(e+1); q 2^(4 - e) lies below 32 (elements 2^-25 of the largest and less lose bits)
      const int e = amax > 0.f ? max((int)(__float_as_uint(amax) >> 23) - 127, -100) : 0;
      const float up = copysignf(__uint_as_float((unsigned)(127 + 4 - e) << 23), p.scale);  // so that f >= 0
      const float fc = fabsf(p.scale) * kLog2e * __uint_as_float((unsigned)(127 - 4 + e) << 23) * 16384.f;
      float sum[G];
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        sum[gg] = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          v[gg][j] *= up;
          sum[gg] += v[gg][j];
        }
        sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], 1);
        sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], 2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float* x = v[gg] + 8 * j;
          qf[nt][4 * gg + 2 * j][0] = half2_bits(x[0] * 1024.f, x[4] * 1024.f);
          qf[nt][4 * gg + 2 * j][1] = half2_bits(x[1] * 64.f, x[5] * 64.f);
          qf[nt][4 * gg + 2 * j + 1][0] = half2_bits(x[2] * 1024.f, x[6] * 1024.f);
          qf[nt][4 * gg + 2 * j + 1][1] = half2_bits(x[3] * 64.f, x[7] * 64.f);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        f[nt][c] = __shfl_sync(0xffffffffu, fc, 8 * t4 + 4 * c);
#pragma unroll
        for (int gg = 0; gg < G; ++gg)
          qs[nt][gg][c] = __shfl_sync(0xffffffffu, sum[gg], 8 * t4 + 4 * c) * (1.f / 16384.f);
        vis[nt][c] = len - p.Lq + 1 + (row0 + 8 * nt + 4 * c + t4) % p.Lq;
      }
    }
    float o[4 * G][NT][4];   // O^T: dims 64 gg + 8 g + 2 mt (+1), rows 8 nt + t4 (+4)
    float z[G][NT][NC];      // this lane's share of sum p m_v
    float m[NT][NC], l[NT][NC];
    // Weights, their sums l and z, and O all carry the factor 2^wexp (2^30 until the first scales are seen).
    float wexp = 30.f;
    uint32_t wlimit, wlow;   // as fp16 bits: the largest scale that wexp allows, 2^(15 - wexp) or less, and the least
                             // largest scale of a step that it serves, 2^(9 - wexp) (weights below 2^9 in it rise again)
    float sub[NT][NC];       // wexp - max of a row
    auto set_wlimits = [&]() {
      const __half hi = __float2half_rz(ex2_approx(15.f - wexp) * 0.9990234375f), lo = __float2half_rz(ex2_approx(9.f - wexp));
      wlimit = *reinterpret_cast<const uint16_t*>(&hi);
      wlow = *reinterpret_cast<const uint16_t*>(&lo);
    };
    set_wlimits();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4 * G; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        m[nt][c] = -INFINITY;
        sub[nt][c] = wexp;
        l[nt][c] = 0.f;
#pragma unroll
        for (int gg = 0; gg < G; ++gg) z[gg][nt][c] = 0.f;
      }
    }
    const int all_see = len - p.Lq + 1;  // keys below it are seen by every column

    // The (scale, minimum) pairs of score rows g and g + 8, from the tile's pairs at `par`.
    auto load_pairs = [&](const uint8_t* par, uint32_t (&ra)[G], uint32_t (&rb)[G]) {
      if constexpr (G == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(par + kg * 8), b = *reinterpret_cast<const uint2*>(par + (kg + 8) * 8);
        ra[0] = a.x, ra[G - 1] = a.y, rb[0] = b.x, rb[G - 1] = b.y;
      } else {
        ra[0] = *reinterpret_cast<const uint32_t*>(par + kg * 4);
        rb[0] = *reinterpret_cast<const uint32_t*>(par + (kg + 8) * 4);
      }
    };
    // N tiles at `tp`, the first of which is tile `tile` of the sequence; EDGE: some column does not see all their keys.
    auto process = [&](const uint8_t* tp, int tile, auto n_c, auto edge_c) {
      constexpr int N = decltype(n_c)::value;
      constexpr bool EDGE = decltype(edge_c)::value;
      const int key0 = tile * kTileKeys;
      float x[N][NT][4];
      // scores; the products that wait on one another's sums alternate between the groups
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint8_t* tb = tp + i * C::TILE;
        uint2 wa[G], wb[G];
        float acc[G][NT][4];
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          wa[gg] = *reinterpret_cast<const uint2*>(tb + gg * 512 + kg * 32 + t4 * 8);
          wb[gg] = *reinterpret_cast<const uint2*>(tb + gg * 512 + (kg + 8) * 32 + t4 * 8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[gg][nt][0] = acc[gg][nt][1] = acc[gg][nt][2] = acc[gg][nt][3] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int gg = 0; gg < G; ++gg) {
            uint32_t a = j / 2 ? wa[gg].y : wa[gg].x, b = j / 2 ? wb[gg].y : wb[gg].x;
            if (j % 2) {
              a >>= 8;
              b >>= 8;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(acc[gg][nt], a & kLowNibble, b & kLowNibble, a & kHighNibble, b & kHighNibble,
                        qf[nt][4 * gg + j][0], qf[nt][4 * gg + j][1]);
          }
        uint32_t ra[G], rb[G];
        load_pairs(tb + kv_q4_kp_off(D), ra, rb);
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          const float2 pa = half2_floats(ra[gg]), pb = half2_floats(rb[gg]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float q = qs[nt][gg][c];
              x[i][nt][c] = fmaf(pa.x, acc[gg][nt][c], gg ? fmaf(pa.y, q, x[i][nt][c]) : pa.y * q);
              x[i][nt][2 + c] = fmaf(pb.x, acc[gg][nt][2 + c], gg ? fmaf(pb.y, q, x[i][nt][2 + c]) : pb.y * q);
            }
        }
      }
      // V's pairs (those of keys past the sequence's end are no data), and the lane's largest scale (the low halves).
      uint32_t va[N][G], vb[N][G];
      __half2 tops = __halves2half2(__half(0.f), __half(0.f));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        load_pairs(tp + i * C::TILE + kv_q4_vp_off(D), va[i], vb[i]);
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          if constexpr (EDGE) {
            const int k = key0 + i * kTileKeys + kg;
            if (k >= len) va[i][gg] = 0;
            if (k + 8 >= len) vb[i][gg] = 0;
          }
          tops = __hmax2(tops, __hmax2(__habs2(as_half2(va[i][gg])), __habs2(as_half2(vb[i][gg]))));
        }
      }
      uint32_t top = half2_word(tops) & 0x7fffu;  // (as fp16 bits, which order as the scales do)
      // row maxima (of x, or at an edge of the masked logits f x)
      float mx[NT][NC];
      const bool low = !__any_sync(0xffffffffu, top >= wlow);  // (the vote is every lane's, so apart from the next line)
      bool change = low | (top > wlimit);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float v = -INFINITY;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if constexpr (EDGE) {
              const int k = key0 + i * kTileKeys + kg;
              x[i][nt][c] = k < vis[nt][c] ? x[i][nt][c] * f[nt][c] : -INFINITY;
              x[i][nt][2 + c] = k + 8 < vis[nt][c] ? x[i][nt][2 + c] * f[nt][c] : -INFINITY;
            }
            v = max3f(v, x[i][nt][c], x[i][nt][2 + c]);
          }
#pragma unroll
          for (int mask = 4; mask < 32; mask <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, mask));
          mx[nt][c] = EDGE ? v : v * f[nt][c];
          change |= mx[nt][c] > m[nt][c];
        }
      // A maximum rises, or the weights' factor has to fall or may rise: rescale what is there.
      if (__any_sync(0xffffffffu, change)) {
        top = __reduce_max_sync(0xffffffffu, top);
        float ratio = 1.f;
        if (top > wlimit || (top < wlow && top > 0)) {  // 2^wexp times the largest scale (below 2^16): into [2^12, 2^13)
          const float we = (float)(12 - ((int)(__float_as_uint(fminf(half2_floats(top).x, 65504.f)) >> 23) - 127));
          ratio = ex2_approx(we - wexp);
          wexp = we;
          set_wlimits();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float mn = fmaxf(m[nt][c], mx[nt][c]);
            // (no key seen yet: all sums are 0)
            const float a = (m[nt][c] == -INFINITY ? 0.f : ex2_approx(m[nt][c] - mn)) * ratio;
            m[nt][c] = mn;
            sub[nt][c] = wexp - (mn == -INFINITY ? 0.f : mn);
            l[nt][c] *= a;
#pragma unroll
            for (int gg = 0; gg < G; ++gg) z[gg][nt][c] *= a;
#pragma unroll
            for (int i = 0; i < 4 * G; ++i) {
              o[i][nt][c] *= a;
              o[i][nt][2 + c] *= a;
              if (NC == 1 && WIDE) {  // the second column holds the weights' second term
                o[i][nt][1] *= a;
                o[i][nt][3] *= a;
              }
            }
          }
      }
      // the weights 2^(f x - max + wexp)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int k = c; k < 4; k += 2)
              x[i][nt][k] = EDGE ? ex2_approx(x[i][nt][k] + sub[nt][c]) : ex2_approx(fmaf(x[i][nt][k], f[nt][c], sub[nt][c]));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint8_t* tb = tp + i * C::TILE + kv_q4_v_off(D);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < NC; ++c) l[nt][c] += x[i][nt][c] + x[i][nt][2 + c];
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          uint32_t b0[NT], b1[NT];
          [[maybe_unused]] uint32_t c0[NT], c1[NT];
          const float2 sa = half2_floats(va[i][gg]), sb = half2_floats(vb[i][gg]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              z[gg][nt][c] = fmaf(x[i][nt][c], sa.y, fmaf(x[i][nt][2 + c], sb.y, z[gg][nt][c]));
            const float w0 = x[i][nt][0] * sa.x, w2 = x[i][nt][2] * sb.x;
            float w1 = 0.f, w3 = 0.f;
            if constexpr (NC == 2) {
              w1 = x[i][nt][1] * sa.x;
              w3 = x[i][nt][3] * sb.x;
            } else if constexpr (WIDE) {
              w1 = w0 - half2_floats(half2_bits(w0, 0.f)).x;
              w3 = w2 - half2_floats(half2_bits(w2, 0.f)).x;
            }
            const uint32_t h0 = half2_bits(w0, w1), h1 = half2_bits(w2, w3);
            b0[nt] = transpose8(h0);
            b1[nt] = transpose8(h1);
            if constexpr (WIDE && NC == 2) {
              const float2 r0 = half2_floats(h0), r1 = half2_floats(h1);
              c0[nt] = transpose8(half2_bits(w0 - r0.x, w1 - r0.y));
              c1[nt] = transpose8(half2_bits(w2 - r1.x, w3 - r1.y));
            }
          }
          const uint8_t* tv = tb + gg * 512 + g * 4;
          const uint32_t u0 = *reinterpret_cast<const uint32_t*>(tv + kv0 * 32);
          const uint32_t u1 = *reinterpret_cast<const uint32_t*>(tv + kv1 * 32);
          const uint32_t u8 = *reinterpret_cast<const uint32_t*>(tv + (kv0 + 8) * 32);
          const uint32_t u9 = *reinterpret_cast<const uint32_t*>(tv + (kv1 + 8) * 32);
          // two keys' halves in one word: dims 8 g .. 8 g + 3 of the group, then 8 g + 4 .. 8 g + 7
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            const unsigned sel = mt < 2 ? 0x5410u : 0x7632u;
            uint32_t a = __byte_perm(u0, u1, sel), b = __byte_perm(u8, u9, sel);
            if (mt & 1) {
              a >>= 8;
              b >>= 8;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float(&oo)[4] = o[4 * gg + mt][nt];
              if constexpr (WIDE) {  // a tile's products apart, then rounded adds (the matrix unit's own adds truncate)
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816(part, a & kLowNibble, a & kHighNibble, b & kLowNibble, b & kHighNibble, b0[nt], b1[nt]);
                if constexpr (NC == 2)
                  mma_16816(part, a & kLowNibble, a & kHighNibble, b & kLowNibble, b & kHighNibble, c0[nt], c1[nt]);
#pragma unroll
                for (int c = 0; c < 4; ++c) oo[c] += part[c];
              } else {
                mma_16816(oo, a & kLowNibble, a & kHighNibble, b & kLowNibble, b & kHighNibble, b0[nt], b1[nt]);
              }
            }
          }
        }
      }
    };

    bool alive = true;
    const int j0 = warp * C::KT;  // this warp's tiles of a stage
    const int last = si.tiles > 0 ? (si.tiles - 1) / C::ST : 0;  // the piece's last stage
    // stages whose tiles of this warp are all there and seen by every column
    const int whole = min(si.tiles, max(0, all_see) / kTileKeys - si.tile0) - j0 - C::KT;
    const int interior = whole < 0 ? 0 : whole / C::ST + 1;
    int stage = 0;
    for (; stage < interior; ++stage) {
      if (!wait(&full[slot])) {
        alive = false;
        break;
      }
      process(smem + slot * C::STAGE + j0 * C::TILE, 0, std::integral_constant<int, C::KT>{}, std::false_type{});
      __syncwarp();
      if (stage == last) break;  // its slot is released after the exchange below
      release();
    }
    for (; alive && stage <= last && !(stage == last && interior > last); ++stage) {
      if (!wait(&full[slot])) {
        alive = false;
        break;
      }
      const int first = stage * C::ST + j0;
      const int mine = min(si.tiles - first, C::KT);
      for (int i = 0; i < mine; ++i)
        process(smem + slot * C::STAGE + (j0 + i) * C::TILE, si.tile0 + first + i, std::integral_constant<int, 1>{},
                std::true_type{});
      __syncwarp();
      if (stage < last) release();
    }
    if (!alive) {
      leave(true);
      break;
    }

    // ---------------- end of a row piece: each warp gathers its share of the accumulators from all ----------------
    // Accumulators i = warp * OW .. + OW-1 of every column group are summed by `warp`, weighted by 2^(m_w - M), in warp
    // order (bitwise reproducible).  A row held by one CTA is written; otherwise the share is this CTA's partial.
    const float back = ex2_approx(-wexp);
    float own[NT][C::OW][4];
    float4* const scr = reinterpret_cast<float4*>(smem + (C::SCR_IN_STAGE ? slot * C::STAGE : C::OFF_SCR));
    named_bar_sync(1, nct);  // every warp is done with the stage and with the last piece's exchange
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float zz[G][2] = {}, ll[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        ll[c] = l[nt][c] * back;
#pragma unroll
        for (int gg = 0; gg < G; ++gg) zz[gg][c] = z[gg][nt][c] * back;
      }
#pragma unroll
      for (int mask = 4; mask < 32; mask <<= 1)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          ll[c] += __shfl_xor_sync(0xffffffffu, ll[c], mask);
#pragma unroll
          for (int gg = 0; gg < G; ++gg) zz[gg][c] += __shfl_xor_sync(0xffffffffu, zz[gg][c], mask);
        }
#pragma unroll
      for (int w = 0; w < C::OWN; ++w)
#pragma unroll
        for (int k = 0; k < C::OW; ++k) {
          const int i = w * C::OW + k;
          float(&oo)[4] = o[i][nt];
          if constexpr (NC == 1) {
            if constexpr (WIDE) {
              oo[0] += oo[1];
              oo[2] += oo[3];
            }
            oo[1] = oo[3] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) oo[c] = fmaf(oo[c], back * (c < 2 ? 16777216.f : 1048576.f), zz[i / 4][c & 1]);
          if (w == warp) {
#pragma unroll
            for (int c = 0; c < 4; ++c) own[nt][k][c] = oo[c];
          } else {
            const int from = warp < w ? warp : warp - 1;
            scr[(((w * (C::NW - 1) + from) * NT + nt) * C::OW + k) * 32 + lane] = make_float4(oo[0], oo[1], oo[2], oo[3]);
          }
        }
      if (g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          mlbuf[(warp * NT + nt) * 8 + 2 * t4 + c] = make_float2(c < NC ? m[nt][c < NC ? c : 0] : -INFINITY, ll[c]);
      }
    }
    if (named_bar_any(1, nct, false)) break;  // the sums of a warp that gave up are missing
    float M[NT][2], L[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float wt[C::NW][2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float2 ml[C::NW];
        M[nt][c] = -INFINITY;
        L[nt][c] = 0.f;
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
          ml[w] = mlbuf[(w * NT + nt) * 8 + 2 * t4 + c];
          M[nt][c] = fmaxf(M[nt][c], ml[w].x);
        }
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
          wt[w][c] = ml[w].x == -INFINITY ? 0.f : ex2_approx(ml[w].x - M[nt][c]);
          L[nt][c] = fmaf(wt[w][c], ml[w].y, L[nt][c]);
        }
      }
#pragma unroll
      for (int k = 0; k < C::OW; ++k) {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
          const int from = w < warp ? w : w - 1;
          float4 v = make_float4(own[nt][k][0], own[nt][k][1], own[nt][k][2], own[nt][k][3]);
          if (w != warp) v = scr[(((warp * (C::NW - 1) + from) * NT + nt) * C::OW + k) * 32 + lane];
          sum[0] = fmaf(wt[w][0], v.x, sum[0]);
          sum[1] = fmaf(wt[w][1], v.y, sum[1]);
          sum[2] = fmaf(wt[w][0], v.z, sum[2]);
          sum[3] = fmaf(wt[w][1], v.w, sum[3]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) own[nt][k][c] = sum[c];
      }
    }
    if constexpr (C::SCR_IN_STAGE) {
      fence_proxy_async_smem();  // the exchange comes before the copy that refills the slot
      __syncwarp();
    }
    release();
    const size_t orow0 = ((size_t)si.b * p.Hkv + hkv) * rows + row0;
    // The row's output from the sums `own`, M and L: two neighbouring dims of two rows for each accumulator.
    auto write_out = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int row = 8 * nt + 4 * c + t4;
          if (row0 + row >= rows) continue;
          const bool none = L[nt][c] == 0.f;  // a row that sees no key: O = 0, lse = -inf (a NaN query: L and O are NaN)
          const float inv = none ? 0.f : 1.f / L[nt][c];
          const size_t at = (orow0 + row) * D;
#pragma unroll
          for (int k = 0; k < C::OW; ++k) {
            const int i = warp * C::OW + k;
            const int d = 64 * (i / 4) + 8 * g + 2 * (i % 4);
            const float a = own[nt][k][c] * inv, b = own[nt][k][2 + c] * inv;
            if (p.out_f32)
              *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at + d) = make_float2(a, b);
            else
              *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at + d) = pack2_bf16(a, b);
          }
          if (warp == 0 && g == 0 && p.lse != nullptr)
            p.lse[orow0 + row] = none ? -INFINITY : (M[nt][c] + log2f(L[nt][c])) * kLn2;
        }
    };
    if (si.np <= 1) {
      write_out();
      continue;
    }
    // A row split between CTAs: each CTA publishes its piece and counts it, each warp its share, and the warp that counts the
    // last one merges them all: no CTA waits for another's work.  A CTA holds at most two such pieces, the first of its slice
    // (slot 2 cta) and the last (2 cta + 1, a row's first piece).  A partial's words are stored complemented over zeros, and no
    // sum has the bits ~0 (a NaN that arithmetic does not make), so a word that is not zero has arrived: no fence between
    // the words and the count, only a wait for what is on its way.  The merging warp zeroes what it has read, and the count.
    // Words of four: an accumulator's two dims of two rows; with one row a lane two accumulators, and the row's (m, l).
    constexpr int OV = NC == 1 ? (C::OW + 1) / 2 : C::OW;
    uint4* const part_o = reinterpret_cast<uint4*>(p.part_o);
    uint4* const part_ml = reinterpret_cast<uint4*>(p.part_ml);
    auto o_at = [&](int sl, int nt, int k) { return part_o + ((((size_t)sl * C::OWN + warp) * NT + nt) * OV + k) * 32 + lane; };
    auto ml_at = [&](int sl, int nt) { return part_ml + (((size_t)sl * C::OWN + warp) * NT + nt) * 4 + t4; };
    // value v of word k of column tile nt
    auto value = [&](int nt, int k, int v) -> float& {
      return NC == 1 ? own[nt][min(2 * k + v / 2, C::OW - 1)][2 * (v & 1)] : own[nt][k][v];
    };
    const int mine = 2 * cta + (cta == si.c_lo ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (row0 + 8 * nt + t4 >= rows) continue;
#pragma unroll
      for (int k = 0; k < OV; ++k)
        st_relaxed_gpu(o_at(mine, nt, k), make_uint4(~__float_as_uint(value(nt, k, 0)), ~__float_as_uint(value(nt, k, 1)),
                                                     ~__float_as_uint(value(nt, k, 2)), ~__float_as_uint(value(nt, k, 3))));
      if (g == 0)
        st_relaxed_gpu(ml_at(mine, nt), make_uint4(~__float_as_uint(M[nt][0]), ~__float_as_uint(L[nt][0]),
                                                   ~__float_as_uint(M[nt][1]), ~__float_as_uint(L[nt][1])));
    }
    unsigned* const count = p.counts + si.c_lo * C::OWN + warp;
    unsigned before = 0;
    __syncwarp();
    if (lane == 0) before = atomicAdd(count, 1u);
    if (__shfl_sync(0xffffffffu, before, 0) + 1 != (unsigned)si.np) continue;
    if (lane == 0) *count = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      M[nt][0] = M[nt][1] = -INFINITY;
      L[nt][0] = L[nt][1] = 0.f;
#pragma unroll
      for (int k = 0; k < C::OW; ++k) own[nt][k][0] = own[nt][k][1] = own[nt][k][2] = own[nt][k][3] = 0.f;
    }
    // Fold the partials in slice order with running maxima (a fixed order: bitwise reproducible), the loads of
    // up to N in flight at a time.
    auto fold = [&](int i, auto n_c) -> bool {
      constexpr int N = decltype(n_c)::value;
      auto slot_of = [&](int u) { return 2 * (si.c_lo + i + u) + (i + u == 0 ? 1 : 0); };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool have = row0 + 8 * nt + t4 < rows;
        uint4 ml[N], ov[N][OV];
        uint64_t since = 0;
        while (true) {
          uint32_t least = 1;
#pragma unroll
          for (int u = 0; u < N; ++u) {
            ml[u] = make_uint4(1, 1, 1, 1);
            if (have) ml[u] = ld_relaxed_gpu(ml_at(slot_of(u), nt));
#pragma unroll
            for (int k = 0; k < OV; ++k) {
              ov[u][k] = make_uint4(1, 1, 1, 1);
              if (have) ov[u][k] = ld_relaxed_gpu(o_at(slot_of(u), nt, k));
            }
          }
#pragma unroll
          for (int u = 0; u < N; ++u) {
            least = min(least, min(min(ml[u].x, ml[u].y), min(ml[u].z, ml[u].w)));
#pragma unroll
            for (int k = 0; k < OV; ++k)
              least = min(least, min(min(ov[u][k].x, ov[u][k].y), min(ov[u][k].z, ov[u][k].w)));
          }
          if (__all_sync(0xffffffffu, least != 0)) break;
          const uint64_t now = globaltimer_ns();
          if (since == 0) since = now;
          if (__any_sync(0xffffffffu, now - since > kWaitLimitNs)) {
            record_status(p.status, ATTN_ERR_DEVICE_TIMEOUT);
            return false;
          }
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const float mc[2] = {__uint_as_float(~ml[u].x), __uint_as_float(~ml[u].z)};
          const float lc[2] = {__uint_as_float(~ml[u].y), __uint_as_float(~ml[u].w)};
          float sc[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float mn = fmaxf(M[nt][c], mc[c]);
            sc[c] = M[nt][c] == -INFINITY ? 0.f : ex2_approx(M[nt][c] - mn);
            w[c] = mc[c] == -INFINITY ? 0.f : ex2_approx(mc[c] - mn);
            M[nt][c] = mn;
            L[nt][c] = fmaf(w[c], lc[c], L[nt][c] * sc[c]);
          }
#pragma unroll
          for (int k = 0; k < OV; ++k) {
            const uint32_t v[4] = {ov[u][k].x, ov[u][k].y, ov[u][k].z, ov[u][k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (NC == 1 && 2 * k + j / 2 >= C::OW) continue;
              const int c = NC == 1 ? 0 : j & 1;
              value(nt, k, j) = fmaf(w[c], __uint_as_float(~v[j]), value(nt, k, j) * sc[c]);
            }
          }
          if (have) {
            if (g == 0) st_relaxed_gpu(ml_at(slot_of(u), nt), make_uint4(0, 0, 0, 0));
#pragma unroll
            for (int k = 0; k < OV; ++k) st_relaxed_gpu(o_at(slot_of(u), nt, k), make_uint4(0, 0, 0, 0));
          }
        }
      }
      return true;
    };
    constexpr int N = 4;
    int i = 0;
    bool got = true;
    for (; got && i + N - 1 < si.np; i += N) got = fold(i, std::integral_constant<int, N>{});
    for (; got && i < si.np; ++i) got = fold(i, std::integral_constant<int, 1>{});
    if (got) write_out();
  }
}

template <int D, int R4, bool WIDE>
cudaError_t launch_one(const DecodeQ4Launch& p) {
  using C = Q4Cfg<D, R4>;
  static bool attr_set[64] = {};  // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(decode_q4_kernel<D, R4, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int rows = (p.Hq / p.Hkv) * p.Lq;
  decode_q4_kernel<D, R4, WIDE><<<C::MINB * p.num_sms, C::THREADS, C::SMEM, p.stream>>>(
      p, (rows + C::ROWS - 1) / C::ROWS, rows);
  return cudaGetLastError();
}

// Query rows a CTA serves: 4, 8, or 16 (kWideTiles).
int rows_per_cta(const DecodeQ4Launch& p) {
  const int rows = (p.Hq / p.Hkv) * p.Lq;
  if (rows <= 8) return rows <= 4 ? 4 : 8;
  const long long tiles = (long long)p.max_pages * (p.page_size / kTileKeys) * p.B * p.Hkv * ((rows + 15) / 16);
  return tiles >= kWideTiles * Q4Cfg<128, 4>::MINB * p.num_sms ? 16 : 8;
}

template <int D, bool WIDE>
cudaError_t launch_rows(const DecodeQ4Launch& p) {
  switch (rows_per_cta(p)) {
    case 4: return launch_one<D, 1, WIDE>(p);
    case 8: return launch_one<D, 2, WIDE>(p);
    default: return launch_one<D, 4, WIDE>(p);
  }
}

}  // namespace

size_t decode_q4_partials(int num_sms) {
  const int sms = num_sms > 0 ? num_sms : 152;
  return (size_t)2 * sms * std::max(8 * Q4Cfg<128, 2>::MINB, 16 * Q4Cfg<128, 4>::MINB);
}

size_t decode_q4_counts(int num_sms) {
  return (size_t)(num_sms > 0 ? num_sms : 152) * Q4Cfg<128, 2>::MINB * kDecodeQ4Owners;
}

cudaError_t launch_decode_q4(const DecodeQ4Launch& p) {
  if (p.D == 64) return p.out_f32 ? launch_rows<64, true>(p) : launch_rows<64, false>(p);
  return p.out_f32 ? launch_rows<128, true>(p) : launch_rows<128, false>(p);
}

}  // namespace attn
