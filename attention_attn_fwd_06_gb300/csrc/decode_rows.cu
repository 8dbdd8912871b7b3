// decode_rows.cu -- decode of a few new tokens of each sequence over a paged bf16 cache, for up to 32 query rows a kv head, 64
// of D = 64 (attn_decode_multi_paged; more rows take decode_multi.cu's tcgen05 tiles of 128).
//
// What it computes: token t of a sequence with n keys, nq of them its new tokens', sees keys 0 .. n - nq + t; softmax and the
// product with V in one pass over the keys with a running maximum and sum, pieces of a row joined by their log-sum-exp.
//
// What bounds it: HBM (each key and value is read once for all rows of its kv head), and over short caches the chain of a launch
// and of each row.  A tile of 128 tcgen05 rows is one CTA an SM, whose roles wait for one another tile by tile: 64 short
// sequences of 16 heads and a few tokens took 50.5 us there, 23.2 here.  Here two or three CTAs share an SM, and a warp takes 32
// keys by itself:
//  * mma.sync m16n8k16 (bf16): A is 16 query rows, kept in registers for a whole piece, B 16 dims of 8 keys by ldmatrix.  The
//    scores' accumulators are, packed to bf16, the second product's A operand as they stand; V comes by transposing ldmatrix.
//    Sixteen query rows cost 2 matrix instructions a key at D = 128 (the tensor pipe is a third busy with 32 rows at the copy
//    bandwidth; with 64 rows 428 us against the tcgen05 tiles' 282 over 4 x 32k to 131k keys, 39 against 31 over 8 x 4096).
//    At D = 64 a key costs half of that, and 33 to 64 rows (in brackets the tcgen05 tiles) of 8 kv heads took 10.6 us (12.9)
//    over 4 x 300 to 500 keys, 21.6 (21.7) over 8 x 512 to 4096, 89 (106) over 4 x 30k to 60k on 16-key pages, 45 (55) over
//    40 x 1000 to 3000 with 40 rows; only over large pages and long caches more, 137 (128) over 4 x 50k to 100k on 64-key pages.
//  * RT tiles of 16 rows: 4 / RT warps share a tile's keys, 32 after 32; a tile of no rows is passed over.
//  * The split is decode.cu's: persistent CTAs take equal slices of the stages (16 KB: 32 keys at D = 128, 64 at D = 64) of all
//    (sequence, kv head) rows, a row charged kRowCost stages beside its own.  A producer warp brings a stage with TMA boxes of
//    gcd(page_size, stage) rows, each in one page, a lane a box, into a ring in the 128-byte swizzle that keeps ldmatrix free
//    of bank conflicts.  Boxes past a sequence's last key are not loaded, and V's keys past it are masked to zero in registers.
//  * At a piece's end the warps of a tile join their sums through the piece's last stage, each a share of the columns; the
//    pieces of a row split between CTAs are published and counted, and who counts the last one merges them (the scheme of
//    decode_q4.cu: complemented words over zeros, no fences, no CTA waits for one that may not have started).
// Scores, maxima, sums and accumulators are fp32; weights are rounded to bf16 before the second product (2^-8 of themselves,
// as in decode_multi.cu), whose adds truncate: over a slice of 131,072 keys some 2^-13 of the terms' sum.
//
// Measured (CUDA-graph replays over rotating pools; 32 query and 8 kv heads, D = 128; in brackets the tcgen05 tiles): 8 sequences
// of 512 to 4096 keys on 16-key pages, 4 tokens each 21.6 us (25.7), 8 tokens 24.9 (27.1); 4 of 32k to 131k keys, 8 tokens
// 265 us, 6.8 TB/s, the copy bandwidth (270.6); 64 of 512 to 1536 keys, 8 tokens 50.8 (69.1); one token to 5 of 64 sequences
// of up to 700 keys with 16 heads of D = 64, 48-key pages 23.2 us (50.5).  At D = 128 4 to 24 bytes of registers spill, at D = 64 none.
// Of the 24.9 us, by timer stamps of an earlier form: 2.5 to the first copy, 0.9 until it lands, 12 of stream, 1 of exchange, 3.5
// (rows of 5 pieces) to 8 (of 10) of merge.  Six stages a CTA in place of five: 24.8 against 24.6, and 282 us over the long caches (the
// SMs nearer to memory run further ahead, and finish 4 % apart); three CTAs at D = 128: 32 to 38 and 370 to 440 us, at D = 64
// with 32 rows 36.1 against 32.3 us (64 sequences of 350 to 700 keys, 16 kv heads; with 16 rows 28.7 against 30.2); one CTA of
// eight warps with ten stages: 27 to 34 and 327 to 504 us (one producer warp's chain is the stream's bound); two producers
// for two CTAs: 25.7 and 278 us; a piece counted before it is published: 27.4 against 26.2 us that day; divisions in the
// producer's stage: 26.2, 59 against 51 us over the 64.  A CTA's last row merged through the idle ring, all of its pieces' words
// in flight at once: 24.1 against 24.6, but 18.0 against 16.8 us with 8 rows over one sequence of 4000 keys and 57.5 against 55.5 with 32
// rows of D = 64 over 64 of 3000: the words themselves are on their way when they are asked for.
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "intdiv.h"
#include "kernels.h"
#include "rope.cuh"
#include "slice_map.h"
#include "tcgen05.cuh"
#include "tmap.h"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowCost = 3;            // stages charged to a row for its piece-end work
constexpr float kRescale = 8.f;        // a row's reference rises when its maximum passes it by this (log2): weights up to 2^8

template <int D, int RT>
struct RowsCfg {
  static constexpr int NDB = D / 64;          // 64-column blocks
  static constexpr int SK = D == 128 ? 32 : 64;  // keys a stage
  static constexpr int NW = 4;                // consumer warps
  static constexpr int KW = NW / RT;          // of them on one row tile
  static constexpr int GS = SK / 32;          // groups of 32 keys a stage
  static constexpr int BLOCK = SK * 128;      // one column block of K (or V)
  static constexpr int HALF = NDB * BLOCK;    // K, then V
  static constexpr int STAGE = 2 * HALF;
  static constexpr int MINB = D == 64 && RT == 1 ? 3 : 2;
  static constexpr int NS = MINB == 2 ? 5 : 4;
  static constexpr int THREADS = 32 * (NW + 1);
  static constexpr int NT = D / 8;            // column tiles of O
  static constexpr int NTW = NT / KW;         // of them a warp's share at a piece's end
  static constexpr int SCR = RT * KW * (KW - 1) * NTW * 512;  // the exchange: [tile][owner][from][NTW][lane] float4
  static constexpr int ROUNDS = KW == 1 ? 1 : (SCR + STAGE - 1) / STAGE;  // through the piece's last stage
  static constexpr int NTR = NTW / ROUNDS;    // column tiles of a share exchanged a round
  static constexpr int LENS_CACHE = 512;
  static constexpr int OFF_BAR = NS * STAGE;  // full[NS], empty[NS], told[NS]
  static constexpr int OFF_INFO = OFF_BAR + 3 * NS * 8;
  static constexpr int OFF_ML = OFF_INFO + NS * 48;  // (m, l) [NW][16]
  static constexpr int OFF_LENS = OFF_ML + NW * 16 * 8;
  static constexpr int OFF_MISC = OFF_LENS + LENS_CACHE * 4;
  static constexpr int SMEM_USED = OFF_MISC + 16;
  static constexpr int SMEM = SMEM_USED + 1024;  // slack to align the ring to 1024
  static_assert(NTR * ROUNDS == NTW && SCR / ROUNDS <= STAGE, "the exchange takes the last stage");
  static_assert(SMEM <= 227 * 1024 && MINB * (SMEM + 1024) <= 228 * 1024, "MINB CTAs per SM");
};

struct RowsArgs {
  const void* q;       // bf16 [T, Hq, D]
  const int* block_table;
  const int* kv_lens;
  const int* cu_new;
  void* out;
  float* lse;
  unsigned* counts;    // [grid][NW]; zero between calls
  uint4* part_o;       // [2 grid][NW][NTW][32]; zero between calls
  uint4* part_ml;      // [2 grid][NW][8]; zero between calls
  int B, T, Hq, Hkv, GP, max_new, max_pages, num_pages, Lmax;
  int box_rows;
  FastDiv page;
  float c;             // scale * log2(e)
  int uniform;         // scale == 0
  int out_f32;
  unsigned* status;
  int fault_skip_arrive;
};

struct RowsPiece {
  int b;      // -1: the end of the work
  int hk;
  int unit0;  // first stage of the sequence in this piece
  int units;  // and their number
  int len;
  int np;     // CTAs holding a piece of this row (0: no keys, 1: whole row here)
  int c_lo;   // the first of them
  int q0, nq; // the sequence's rows of q
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int RT>
__global__ void __launch_bounds__(RowsCfg<D, RT>::THREADS, RowsCfg<D, RT>::MINB)
    decode_rows_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const RowsArgs a) {
  using C = RowsCfg<D, RT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NS;
  uint64_t* told = empty + C::NS;  // the record of piece i % NS is written (its data may still be on the way)
  RowsPiece* info = reinterpret_cast<RowsPiece*>(smem + C::OFF_INFO);
  float2* mlbuf = reinterpret_cast<float2*>(smem + C::OFF_ML);
  int* lens_s = reinterpret_cast<int*>(smem + C::OFF_LENS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const int Hkv = a.Hkv;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::NW);
      mbar_init(&told[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == C::NW) {
    // ---------------- producer: walk this CTA's slice of the stages ----------------
    if (lane == 0) {
      tc::tma_prefetch_desc(&tmk);
      tc::tma_prefetch_desc(&tmv);
    }
    // New tokens of sequence b: offsets that fall, leave [0, T] or give too many count as none.
    auto seq_new = [&](int b, int& q0, bool& bad) -> int {
      q0 = a.cu_new[b];
      const int q1 = a.cu_new[b + 1];
      bad = !(q0 >= 0 && q1 >= q0 && q1 <= a.T && q1 - q0 <= a.max_new);
      return bad ? 0 : q1 - q0;
    };
    // keys that sequence b has to look at (none without new tokens)
    auto load_len = [&](int b, bool flag) -> int {
      int q0;
      bool bad;
      const int raw = a.kv_lens[b];
      const int nq = seq_new(b, q0, bad);
      const int len = raw < 0 ? 0 : (raw > a.Lmax ? a.Lmax : raw);
      if ((bad || len != raw) && flag) record_status(a.status, ATTN_ERR_DEVICE_BOUNDS);
      return nq > 0 ? len : 0;
    };
    long long usum = 0;
    int nonempty = 0;
    for (int b = lane; b < a.B; b += 32) {
      const int len = load_len(b, cta == 0);
      if (b < C::LENS_CACHE) lens_s[b] = len;
      usum += (len + C::SK - 1) / C::SK;
      nonempty += len > 0 ? 1 : 0;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      usum += __shfl_xor_sync(0xffffffffu, usum, off);
      nonempty += __shfl_xor_sync(0xffffffffu, nonempty, off);
    }
    __syncwarp();
    auto seq_len = [&](int b) -> int { return b < C::LENS_CACHE ? lens_s[b] : load_len(b, false); };
    auto seq_units = [&](int b) -> int { return (seq_len(b) + C::SK - 1) / C::SK; };
    const long long W = usum * Hkv;
    // Slices of so many stages that a slice's time does not fall far below the merge of the partials it makes, but never
    // fewer slices than rows with keys.
    const int min_units = max(2, (int)sqrtf(to_f32(W) / (float)max(1, nonempty * Hkv)));
    long long geff = floor_div(W + min_units - 1, min_units);
    if (geff < (long long)nonempty * Hkv) geff = (long long)nonempty * Hkv;
    if (geff > (long long)gridDim.x) geff = gridDim.x;
    if (geff < 1) geff = 1;
    // Every row occupies [rs, rs + kRowCost + units) of the cost space, its stages last.
    const long long Wc = W + (long long)kRowCost * nonempty * Hkv;
    const SliceMap sm = make_slice_map(Wc, geff, 1, gridDim.x);
    const long long lo = sm.start(cta), hi = sm.start(cta + 1);

    int t = 0;  // stages issued
    int piece = 0;  // record of the next piece: at most NS are on the way, as each has a stage
    int slot = 0;
    uint32_t freed = 1;  // parity of the phase in which the slot's last stage was released
    bool ok = true;
    const uint64_t policy = l2_policy_evict_first();  // the cache is read once
    const int ps = (int)a.page.d;
    // Lane 8 w + i (w 0: K, 1: V) brings column block i % NDB of box i / NDB of every stage.  A stage's instructions are one warp's
    // chain, and a chain of each of an SM's CTAs has to keep up with its stream (1400 cycles a stage of two CTAs, stamps of an
    // earlier form 900 to 1350): no divisions in it, and each lane reads its box's block-table entry a stage ahead.
    const int which = lane >> 3, box = (lane & 7) / C::NDB, db = (lane & 7) % C::NDB;
    const bool has_box = lane < 16 && box * a.box_rows < C::SK;
    const int per_stage = C::SK / a.box_rows;
    const uint32_t box_bytes = (uint32_t)a.box_rows * (2 * 128 * C::NDB);
    const int step_pages = C::SK / ps, step_off = C::SK - step_pages * ps;  // a stage further
    const uint32_t dst0 = (uint32_t)(which * C::HALF + db * C::BLOCK + box * a.box_rows * 128);
    const void* const tm = which ? &tmv : &tmk;
    auto wait_empty = [&]() -> bool {
      return t < C::NS || mbar_wait_warp(&empty[slot], freed, a.status, abort_flag);
    };
    auto next_slot = [&]() {
      ++t;
      if (++slot == C::NS) {
        slot = 0;
        freed ^= 1;
      }
    };
    // Stream stages [ub, ue) of row (b, hk), whose stages sit at cost positions [ks, ..); ue == ub emits one empty stage (a
    // sequence of new tokens with no keys).
    auto emit = [&](int b, int hk, int ub, int ue, long long ks) -> bool {
      const int n = ue - ub, nst = n > 0 ? n : 1;
      const int len = seq_len(b);
      int np = 0, row_lo = 0;
      int q0;
      bool bad;
      const int nq = seq_new(b, q0, bad);  // (on its way beside the first copies)
      // the lane's box: its page and the row in it; the boxes that hold keys from this piece's start on
      const int key = ub * C::SK + box * a.box_rows;
      int pg = (int)a.page.div((unsigned)key);
      int off = key - pg * ps;
      int boxes = n > 0 ? (len - ub * C::SK + a.box_rows - 1) / a.box_rows : 0;
      const int* const row = a.block_table + (size_t)b * a.max_pages;
      const int pages = len > 0 ? (int)a.page.div((unsigned)(len - 1)) + 1 : 0;  // that hold keys: entries past them are not read
      int page = has_box && pg < pages ? __ldg(row + pg) : 0;
      for (int u = 0; u < nst; ++u, next_slot()) {
        if (!wait_empty()) return false;
        if (n > 0) {
          const int now = min(boxes, per_stage);
          boxes -= now;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)now * box_bytes);
          const bool mine = has_box && box < now;
          if (mine) {
            if (page < 0 || page >= a.num_pages) {
              record_status(a.status, ATTN_ERR_DEVICE_BOUNDS);  // out-of-pool page id: read page 0 instead
              page = 0;
            }
            tc::tma_load_3d_hint(smem + slot * C::STAGE + dst0, tm, db * 64, off, page * Hkv + hk, &full[slot], policy);
          }
          pg += step_pages;
          off += step_off;
          if (off >= ps) {
            off -= ps;
            ++pg;
          }
          page = has_box && pg < pages ? __ldg(row + pg) : 0;
        } else if (lane == 0) {
          mbar_arrive(&full[slot]);
        }
        if (u == 0 && n > 0) {
          // which CTAs hold a piece of this row
          const long long last = ks + seq_units(b) - 1;
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
        if (u == 0) {
          if (lane == 0) {
            RowsPiece pi;
            pi.b = b;
            pi.hk = hk;
            pi.unit0 = ub;
            pi.units = n;
            pi.len = len;
            pi.np = np;
            pi.c_lo = row_lo;
            pi.q0 = q0;
            pi.nq = nq;
            info[piece] = pi;
            mbar_arrive(&told[piece]);
          }
          if (++piece == C::NS) piece = 0;
        }
      }
      return true;
    };

    if (lo < hi) {
      // the row whose cost interval holds position lo: sequences 32 at a time
      long long acc = 0;  // first cost position of sequence b
      int b = 0, nu = 0;
      for (int b32 = 0;; b32 += 32) {
        const int my_nu = b32 + lane < a.B ? seq_units(b32 + lane) : 0;
        const long long mine = my_nu > 0 ? Hkv * ((long long)my_nu + kRowCost) : 0;
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
          nu = __shfl_sync(0xffffffffu, my_nu, src);
          b = b32 + src;
          break;
        }
        acc += __shfl_sync(0xffffffffu, upto, 31);
      }
      long long rcost = (long long)nu + kRowCost;
      int hk = (int)floor_div(lo - acc, rcost);
      long long rs = acc + (long long)hk * rcost;
      long long pos = lo;
      while (ok && pos < hi) {
        const long long ks = rs + kRowCost;
        const long long s = max(pos, ks), e = min(hi, ks + nu);
        if (s < e) ok = emit(b, hk, (int)(s - ks), (int)(e - ks), ks);
        pos = rs + rcost;
        rs += rcost;
        if (++hk == Hkv) {
          hk = 0;
          for (++b; b < a.B; ++b) {
            nu = seq_units(b);
            if (nu > 0) break;
          }
          rcost = (long long)nu + kRowCost;
        }
      }
    }
    if (nonempty < a.B) {  // rows of sequences with new tokens and no keys, one row per CTA in turn
      for (long long e = cta; ok && e < (long long)a.B * Hkv; e += gridDim.x) {
        const int b = (int)floor_div(e, Hkv);
        int q0;
        bool bad;
        if (seq_len(b) == 0 && seq_new(b, q0, bad) > 0) ok = emit(b, (int)(e - (long long)b * Hkv), 0, 0, 0);
      }
    }
    if (ok && wait_empty() && lane == 0) {  // end-of-work marker
      info[piece].b = -1;
      mbar_arrive(&told[piece]);
    }
    if (lane == 0 && *abort_flag) {
      // Let copies already in flight land before the CTA's shared memory is released.
      for (int u = (t > C::NS ? t - C::NS : 0); u < t; ++u)
        mbar_wait(&full[u % C::NS], (u / C::NS) & 1, a.status, nullptr);
    }
    return;
  }

  // ---------------- consumers ----------------
  constexpr int nct = C::NW * 32;
  const int g = lane >> 2, t4 = lane & 3;
  const int rt = warp / C::KW, kw = warp % C::KW;
  // The test hook withholds CTA 0's release of its second stage: the producer's bounded wait then runs out.
  int to_skip = a.fault_skip_arrive && cta == 0 ? 1 : -1;
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
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return mbar_wait_warp(bar, parity, a.status, abort_flag); };
  int piece = 0;  // the next record, and its phase
  uint32_t piece_phase = 0;
  // Addresses within a stage of the lane's rows for ldmatrix: K's matrices are (keys 0-7, 8-15) x (dims 0-7, 8-15) of a step of
  // 16 dims, V's (keys 0-7, 8-15) x (dims 0-7, 8-15) with keys first; chunks of 8 dims XOR-swizzled by the key's low bits.
  const int lk = lane & 7;
  const uint32_t k_row = (uint32_t)(((lane >> 4) * 8 + lk) * 128), v_row = (uint32_t)((((lane >> 3) & 1) * 8 + lk) * 128);
  const int k_half = (lane >> 3) & 1, v_half = lane >> 4;

  while (true) {
    // Every warp takes part in one vote for each record, the end's among them: a wait can run out in one warp and just succeed
    // in another.
    bool alive = wait(&told[piece], piece_phase);
    RowsPiece si;
    si.b = -1;
    if (alive) si = info[piece];
    if (++piece == C::NS) {
      piece = 0;
      piece_phase ^= 1;
    }
    float o[C::NT][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int valid = 0;  // rows of the tile that are tokens' (all tiles)
#pragma unroll
    for (int i = 0; i < C::NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    if (si.b >= 0) {
      valid = a.GP * si.nq;
      // q as the first product's A operand: rows g and g + 8 of the tile
      uint32_t qf[D / 16][4];
      int vis[2];  // keys that the lane's rows see
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = rt * 16 + g + 8 * c;
        const int tok = r / a.GP;
        vis[c] = r < valid ? si.len - si.nq + tok + 1 : 0;
        const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                   ((size_t)(si.q0 + tok) * a.Hq + si.hk * a.GP + (r - tok * a.GP)) * D + 2 * t4;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          qf[j][c] = r < valid ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * j)) : 0u;
          qf[j][2 + c] = r < valid ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * j + 8)) : 0u;
        }
      }
      const int all_see = si.len - si.nq + 1;  // keys below it are seen by every row
      // 32 keys from key0 on, at `base` (their rows of K's first block); EDGE: some row does not see all of them.
      auto process = [&](uint32_t base, int key0, auto edge_c) {
        constexpr bool EDGE = decltype(edge_c)::value;
        float s[4][4] = {};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const int ch = 2 * j + k_half;
          const uint32_t at = base + (ch >> 3) * C::BLOCK + k_row + (((ch & 7) ^ lk) << 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t kf[4];
            ldmatrix4(kf, at + h * 2048);
            mma_bf16(s[2 * h], qf[j], kf[0], kf[1]);
            mma_bf16(s[2 * h + 1], qf[j], kf[2], kf[3]);
          }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = a.uniform ? 0.f : s[i][e] * a.c;
            if constexpr (EDGE) x = key0 + 8 * i + 2 * t4 + (e & 1) < vis[e >> 1] ? x : -INFINITY;
            s[i][e] = x;
            mx[e >> 1] = fmaxf(mx[e >> 1], x);
          }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 1));
          mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kRescale || mx[1] > m[1] + kRescale)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (mx[c] > m[c] + kRescale) {
              const float alpha = ex2_approx(m[c] - mx[c]);  // (0 while nothing was seen)
              m[c] = mx[c];
              l[c] *= alpha;
#pragma unroll
              for (int i = 0; i < C::NT; ++i) {
                o[i][2 * c] *= alpha;
                o[i][2 * c + 1] *= alpha;
              }
            }
          }
        }
        const float sub[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        uint32_t p[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = ex2_approx(s[i][e] - sub[e >> 1]);
          l[0] += s[i][0] + s[i][1];
          l[1] += s[i][2] + s[i][3];
          p[i >> 1][2 * (i & 1)] = tc::pack_bf16x2(s[i][0], s[i][1]);
          p[i >> 1][2 * (i & 1) + 1] = tc::pack_bf16x2(s[i][2], s[i][3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of V's keys 2 t4, 2 t4 + 1 and those 8 on: past the end is no data
          if constexpr (EDGE) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k = key0 + 16 * h + 8 * i + 2 * t4;
              keep[i] = (k < si.len ? 0xffffu : 0u) | (k + 1 < si.len ? 0xffff0000u : 0u);
            }
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t vf[4];
            const int ch = 2 * j + v_half;
            ldmatrix4_trans(vf, base + C::HALF + (ch >> 3) * C::BLOCK + h * 2048 + v_row + (((ch & 7) ^ lk) << 4));
            if constexpr (EDGE) {
              vf[0] &= keep[0];
              vf[1] &= keep[1];
              vf[2] &= keep[0];
              vf[3] &= keep[1];
            }
            mma_bf16(o[2 * j], p[h], vf[0], vf[1]);
            mma_bf16(o[2 * j + 1], p[h], vf[2], vf[3]);
          }
        }
      };
      const int last = si.units > 0 ? si.units - 1 : 0;
      for (int u = 0;; ++u) {
        if (!wait(&full[slot], phase)) {
          alive = false;
          break;
        }
        if (u < si.units) {
          const uint32_t base = smem_u32(smem + slot * C::STAGE);
#pragma unroll
          for (int j = 0; j < C::GS; ++j) {
            if ((u * C::GS + j) % C::KW != kw) continue;
            const int key0 = (si.unit0 + u) * C::SK + 32 * j;
            if (rt * 16 >= valid) continue;  // (a tile of no rows)
            if (key0 + 32 <= all_see)
              process(base + 32 * j * 128, key0, std::false_type{});
            else if (key0 < si.len)
              process(base + 32 * j * 128, key0, std::true_type{});
          }
        }
        __syncwarp();
        if (u == last) break;  // its slot is released after the exchange below
        release();
      }
    }
    if (named_bar_any(1, nct, !alive)) break;  // (and every warp is done with the piece's last stage)
    if (si.b < 0) break;

    // ---------------- end of a row piece ----------------
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l[c] += __shfl_xor_sync(0xffffffffu, l[c], 1);
      l[c] += __shfl_xor_sync(0xffffffffu, l[c], 2);
      if (C::KW > 1 && t4 == 0) mlbuf[warp * 16 + g + 8 * c] = make_float2(m[c], l[c]);
    }
    // Column tiles kw NTW .. + NTW - 1 of this row tile are summed by this warp, weighted by 2^(m_w - M), in warp order (bitwise
    // reproducible).
    float own[C::NTW][4];
    float M[2], L[2];
    if constexpr (C::KW == 1) {  // a warp has all of its tile's keys
#pragma unroll
      for (int k = 0; k < C::NTW; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) own[k][e] = o[k][e];
      M[0] = m[0], M[1] = m[1], L[0] = l[0], L[1] = l[1];
    } else {
      float4* const scr = reinterpret_cast<float4*>(smem + slot * C::STAGE);
      auto at = [&](int owner, int from, int k) {
        return ((rt * C::KW + owner) * (C::KW - 1) + (from < owner ? from : from - 1)) * C::NTR + k;
      };
#pragma unroll
      for (int w = 0; w < C::KW; ++w)
        if (w == kw)
#pragma unroll
          for (int k = 0; k < C::NTW; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) own[k][e] = o[w * C::NTW + k][e];
      float wt[C::KW][2];
#pragma unroll
      for (int round = 0; round < C::ROUNDS; ++round) {
#pragma unroll
        for (int w = 0; w < C::KW; ++w) {
          if (w == kw) continue;
#pragma unroll
          for (int k = 0; k < C::NTR; ++k) {
            const float(&v)[4] = o[w * C::NTW + round * C::NTR + k];
            scr[at(w, kw, k) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        named_bar_sync(1, nct);
        if (round == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float2 ml[C::KW];
            M[c] = -INFINITY;
            L[c] = 0.f;
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
              ml[w] = mlbuf[(rt * C::KW + w) * 16 + g + 8 * c];
              M[c] = fmaxf(M[c], ml[w].x);
            }
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
              wt[w][c] = ml[w].x == -INFINITY ? 0.f : ex2_approx(ml[w].x - M[c]);
              L[c] = fmaf(wt[w][c], ml[w].y, L[c]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < C::NTR; ++k) {
          const int kk = round * C::NTR + k;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < C::KW; ++w) {
            float4 v = make_float4(own[kk][0], own[kk][1], own[kk][2], own[kk][3]);
            if (w != kw) v = scr[at(kw, w, k) * 32 + lane];
            sum[0] = fmaf(wt[w][0], v.x, sum[0]);
            sum[1] = fmaf(wt[w][0], v.y, sum[1]);
            sum[2] = fmaf(wt[w][1], v.z, sum[2]);
            sum[3] = fmaf(wt[w][1], v.w, sum[3]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) own[kk][e] = sum[e];
        }
        if (round + 1 < C::ROUNDS) named_bar_sync(1, nct);
      }
      named_bar_sync(1, nct);    // (m, l) and the last stage are read
      fence_proxy_async_smem();  // the exchange comes before the copy that refills the slot
      __syncwarp();
    }
    release();
    auto write_out = [&]() {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = rt * 16 + g + 8 * c;
        if (r >= valid) continue;
        const int tok = r / a.GP;
        const size_t row = (size_t)(si.q0 + tok) * a.Hq + si.hk * a.GP + (r - tok * a.GP);
        const bool none = L[c] == 0.f;  // a row that sees no key: O = 0, lse = -inf (a NaN query: L and O are NaN)
        const float inv = none ? 0.f : 1.f / L[c];
#pragma unroll
        for (int k = 0; k < C::NTW; ++k) {
          const size_t at = row * D + 8 * (kw * C::NTW + k) + 2 * t4;
          const float x = none ? 0.f : own[k][2 * c] * inv, y = none ? 0.f : own[k][2 * c + 1] * inv;
          if (a.out_f32)
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = make_float2(x, y);
          else
            *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) = tc::pack_bf16x2(x, y);
        }
        if (kw == 0 && t4 == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : (M[c] + log2f(L[c])) * kLn2;
      }
    };
    if (si.np <= 1) {
      write_out();
      continue;
    }
    // A row split between CTAs: each CTA publishes its piece and counts it, each warp its share, and the warp that counts the
    // last one merges them all.  A CTA holds at most two such pieces, the first of its slice (slot 2 cta) and the last (2 cta + 1,
    // a row's first piece).  A partial's words are stored complemented over zeros, and no sum has the bits ~0, so a word that is
    // not zero has arrived: no fence between the words and the count, only a wait for what is on its way.  The merging warp
    // zeroes what it has read, and the count.
    if (rt * 16 >= valid) continue;  // (a tile of no rows has nothing to tell: in every CTA alike)
    auto o_at = [&](int sl, int k) { return a.part_o + (((size_t)sl * C::NW + warp) * C::NTW + k) * 32 + lane; };
    auto ml_at = [&](int sl) { return a.part_ml + ((size_t)sl * C::NW + warp) * 8 + g; };
    const int mine = 2 * cta + (cta == si.c_lo ? 1 : 0);
#pragma unroll
    for (int k = 0; k < C::NTW; ++k)
      st_relaxed_gpu(o_at(mine, k), make_uint4(~__float_as_uint(own[k][0]), ~__float_as_uint(own[k][1]),
                                               ~__float_as_uint(own[k][2]), ~__float_as_uint(own[k][3])));
    if (t4 == 0)
      st_relaxed_gpu(ml_at(mine), make_uint4(~__float_as_uint(M[0]), ~__float_as_uint(L[0]), ~__float_as_uint(M[1]),
                                             ~__float_as_uint(L[1])));
    unsigned* const count = a.counts + si.c_lo * C::NW + warp;
    unsigned before = 0;
    __syncwarp();
    if (lane == 0) before = atomicAdd(count, 1u);
    if (__shfl_sync(0xffffffffu, before, 0) + 1 != (unsigned)si.np) continue;
    if (lane == 0) *count = 0;
    M[0] = M[1] = -INFINITY;
    L[0] = L[1] = 0.f;
#pragma unroll
    for (int k = 0; k < C::NTW; ++k) own[k][0] = own[k][1] = own[k][2] = own[k][3] = 0.f;
    // Fold the partials in slice order with running maxima (a fixed order: bitwise reproducible), N partials' loads in flight.
    auto fold = [&](int i, auto n_c) -> bool {
      constexpr int N = decltype(n_c)::value;
      auto slot_of = [&](int u) { return 2 * (si.c_lo + i + u) + (i + u == 0 ? 1 : 0); };
      uint4 ml[N], ov[N][C::NTW];
      uint64_t since = 0;
      while (true) {
        uint32_t least = 1;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          ml[u] = ld_relaxed_gpu(ml_at(slot_of(u)));
#pragma unroll
          for (int k = 0; k < C::NTW; ++k) ov[u][k] = ld_relaxed_gpu(o_at(slot_of(u), k));
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
          least = min(least, min(min(ml[u].x, ml[u].y), min(ml[u].z, ml[u].w)));
#pragma unroll
          for (int k = 0; k < C::NTW; ++k) least = min(least, min(min(ov[u][k].x, ov[u][k].y), min(ov[u][k].z, ov[u][k].w)));
        }
        if (__all_sync(0xffffffffu, least != 0)) break;
        const uint64_t now = globaltimer_ns();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, now - since > kWaitLimitNs)) {
          record_status(a.status, ATTN_ERR_DEVICE_TIMEOUT);
          return false;
        }
      }
      __syncwarp();  // every lane has read (m, l), which another zeroes
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const float mc[2] = {__uint_as_float(~ml[u].x), __uint_as_float(~ml[u].z)};
        const float lc[2] = {__uint_as_float(~ml[u].y), __uint_as_float(~ml[u].w)};
        float sc[2], w[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mn = fmaxf(M[c], mc[c]);
          sc[c] = M[c] == -INFINITY ? 0.f : ex2_approx(M[c] - mn);
          w[c] = mc[c] == -INFINITY ? 0.f : ex2_approx(mc[c] - mn);
          M[c] = mn;
          L[c] = fmaf(w[c], lc[c], L[c] * sc[c]);
        }
#pragma unroll
        for (int k = 0; k < C::NTW; ++k) {
          own[k][0] = fmaf(w[0], __uint_as_float(~ov[u][k].x), own[k][0] * sc[0]);
          own[k][1] = fmaf(w[0], __uint_as_float(~ov[u][k].y), own[k][1] * sc[0]);
          own[k][2] = fmaf(w[1], __uint_as_float(~ov[u][k].z), own[k][2] * sc[1]);
          own[k][3] = fmaf(w[1], __uint_as_float(~ov[u][k].w), own[k][3] * sc[1]);
          st_relaxed_gpu(o_at(slot_of(u), k), make_uint4(0, 0, 0, 0));
        }
        if (t4 == 0) st_relaxed_gpu(ml_at(slot_of(u)), make_uint4(0, 0, 0, 0));
      }
      return true;
    };
    constexpr int N = C::NTW <= 4 ? 4 : 2;
    int i = 0;
    bool got = true;
    for (; got && i + N - 1 < si.np; i += N) got = fold(i, std::integral_constant<int, N>{});
    for (; got && i < si.np; ++i) got = fold(i, std::integral_constant<int, 1>{});
    if (got) write_out();
  }
}

template <int D, int RT>
cudaError_t launch_one(const DecodeMultiLaunch& p) {
  using C = RowsCfg<D, RT>;
  static bool attr_set[64] = {};  // the shared-memory opt-in is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(decode_rows_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  RowsArgs a{};
  a.box_rows = C::SK;
  while (p.page_size % a.box_rows != 0) a.box_rows /= 2;  // gcd(page_size, SK), at least 8
  if (a.box_rows < 8) return cudaErrorInvalidValue;
  const uint64_t row_b = (uint64_t)D * 2, page_b = row_b * p.page_size, heads = (uint64_t)p.num_pages * p.Hkv;
  CUtensorMap tmk, tmv;
  if (!make_tmap_bf16_3d(&tmk, p.kcache, D, p.page_size, heads, row_b, page_b, 64, (uint32_t)a.box_rows, 1) ||
      !make_tmap_bf16_3d(&tmv, p.vcache, D, p.page_size, heads, row_b, page_b, 64, (uint32_t)a.box_rows, 1))
    return cudaErrorInvalidValue;
  const int grid = C::MINB * p.num_sms;
  a.q = p.q;
  a.block_table = p.block_table;
  a.kv_lens = p.kv_lens;
  a.cu_new = p.cu_new;
  a.out = p.out;
  a.lse = p.lse;
  const DecodeRowsShape sh = decode_rows_shape(16 * RT, D, p.num_sms);
  char* ws = static_cast<char*>(p.rows_ws);
  a.counts = reinterpret_cast<unsigned*>(ws);
  a.part_ml = reinterpret_cast<uint4*>(ws + sh.count_bytes);
  a.part_o = reinterpret_cast<uint4*>(ws + sh.count_bytes + sh.ml_bytes);
  a.B = p.B;
  a.T = p.T;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.GP = p.Hq / p.Hkv;
  a.max_new = p.Lq;
  a.max_pages = p.max_pages;
  a.num_pages = p.num_pages;
  a.Lmax = p.Lmax;
  a.page = make_fast_div((unsigned)p.page_size);
  a.uniform = p.scale == 0.f;
  a.c = p.scale * kLog2e;
  a.out_f32 = p.out_f32;
  a.status = p.status;
  a.fault_skip_arrive = p.fault_skip_arrive;
  decode_rows_kernel<D, RT><<<grid, C::THREADS, C::SMEM, p.stream>>>(tmk, tmv, a);
  return cudaGetLastError();
}

}  // namespace

DecodeRowsShape decode_rows_shape(int rows, int D, int num_sms) {
  const int tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const int per_sm = D == 128 ? RowsCfg<128, 1>::MINB : tiles == 1 ? RowsCfg<64, 1>::MINB : RowsCfg<64, 2>::MINB;
  const size_t grid = (size_t)(num_sms > 0 ? num_sms : 152) * per_sm;
  DecodeRowsShape s;
  s.count_bytes = (grid * 4 * sizeof(unsigned) + 127) / 128 * 128;
  s.ml_bytes = 2 * grid * 4 * 8 * sizeof(uint4);
  s.bytes = s.count_bytes + s.ml_bytes + 2 * grid * tiles * 16 * D * sizeof(float);
  return s;
}

cudaError_t launch_decode_rows(const DecodeMultiLaunch& p) {
  const int rows = p.Hq / p.Hkv * p.Lq;
  if (p.D == 64) return rows <= 16 ? launch_one<64, 1>(p) : rows <= 32 ? launch_one<64, 2>(p) : launch_one<64, 4>(p);
  return rows <= 16 ? launch_one<128, 1>(p) : launch_one<128, 2>(p);
}

}  // namespace attn
