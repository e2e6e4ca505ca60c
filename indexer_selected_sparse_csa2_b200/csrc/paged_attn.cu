// MLA attention of packed chunks of new tokens over a paged latent cache
// (csa_paged_attn_args in csa.h): causal, optional sliding window, sink and
// partial RoPE, FP8 or FP4 entries, one token per sequence up to whole prompts.
//
// A work item is 64 query rows (token, head) of one sequence, rows in (token,
// head) order, so any head count fills the tile; it runs over the 32-entry
// key tiles its rows see.  Per key tile, with K = V = the decoded entries:
//   S  = Q K^T    tcgen05.mma kind::f16, M = 128 TMEM lanes holding the 64
//                 rows twice (lane L: row L mod 64), N = 32 entries, K = 512.
//                 Channels 0..383 of Q are the A operand in TMEM, the last
//                 128 in shared memory.  The two copies let two pairs of
//                 softmax warps take turns: warps 0-1 even tiles, 2-3 odd ones.
//   O^T += V^T P^T  M = 128 latent channels (4 chunks), N = 64 rows, K = 32
//                 entries: 4 x 64 TMEM columns, where O (64 x 512) would take
//                 all 512.  The shared-memory tile of decoded entries is the
//                 K-major B operand of S and the MN-major A operand here.
// Online softmax in the exp2 domain; the running max moves only when a tile's
// max exceeds it by more than 8, and only then O^T is rescaled in TMEM.  P is
// held in fp16 times 2^6: at most 2^14, and weights down to 2^-31 of the max
// keep a value.
//
// Work split: the batch is a line on which an item of T key tiles takes
// kPgItemCost + T; CTA i takes the tiles on [iU/G, (i+1)U/G) of its length U,
// whatever the sequences' lengths, and computes where that is from the lengths
// on the device.  An item that ends up in several CTAs leaves (max, sum, O^T)
// partials in the workspace, at most two per CTA, which paged_attn_combine
// joins in CTA order; the result does not depend on timing.
//
// Warp roles: 0-3 softmax and output, 4-7 and 8-11 staging of Q and loading and
// decoding of even and odd tiles, 12 issues the S MMAs, 13 the PV MMAs.  Four
// entry tiles and P tiles are in flight: a tile's way (decode, S, softmax, PV)
// is several times longer than its share of the tensor pipe.
#include <climits>

#include "sm100.cuh"
#include "paged.cuh"
#include "rope.cuh"

namespace csa {

constexpr int kPgRows = 64;               // query rows per item
constexpr int kPgE = 32;                  // entries per key tile
constexpr int kPgBufs = 4;                // entry tiles (and P tiles) in the ring
constexpr int kPgDeqWarps = 8;            // two groups of 4: even and odd tiles
constexpr int kPgWarpS = 4 + kPgDeqWarps;
constexpr int kPgWarpPV = kPgWarpS + 1;
constexpr int kPgWarps = kPgWarpPV + 1;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgQTmemBlocks = 6;         // 64-channel blocks of Q in TMEM
constexpr int kPgQBlk = 128 * 128;        // shared Q block: 128 rows x 64 fp16
constexpr int kPgKVBlk = kPgE * 128;      // 64-channel block of an entry tile
constexpr int kPgKVBytes = 8 * kPgKVBlk;
constexpr int kPgPBytes = kPgRows * kPgE * 2;
constexpr uint32_t kPgSCol = 32 * kPgQTmemBlocks;   // two S tiles of 32 columns
constexpr uint32_t kPgOCol = 256;
constexpr uint32_t kPgTmemCols = 512;
static_assert(kPgSCol + 2 * kPgE <= kPgOCol, "TMEM map");
constexpr int kPgItemCost = 4;            // an item's own cost (Q, output) in key tiles
constexpr float kPgRescale = 8.0f;        // lazy-rescale threshold (exp2 units)
constexpr float kPgPExp = 6.0f;           // P carries a factor 2^6
constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgLn2 = 0.6931471805599453f;
constexpr int kPgMaxB = 65536;
constexpr size_t kPgSmemBytes = 1024 + 2 * kPgQBlk + kPgBufs * (kPgKVBytes + kPgPBytes) + 4096;
static_assert(kPgMaxB / 32 * 8 <= kPgBufs * kPgKVBytes, "the plan's group sums use the entry tiles");

static __device__ int g_pg_error;

// What a CTA left for the combine.
struct PgMeta {
  int64_t row0;      // leader: first output row (token * H + head) of its last item
  int32_t rows;      // leader: rows of that item; 0 = its last item is not split here
  int32_t cont;      // its first item began in an earlier CTA ...
  int32_t done;      // ... and ends here
  int32_t pad;
};

struct PgParams {
  csa_paged_attn_args a;
  float scale_log2;  // softmax_scale * log2(e), times the entries' staging factor
  float out_scale;   // inverse of the entries' staging factor
  float* part_o;     // [2 * gridDim.x][64][512] fp32
  float2* part_ml;   // [2 * gridDim.x][64] (max, sum)
  PgMeta* meta;      // [gridDim.x]
};

struct PgSmem {
  uint8_t* q;        // channels 384..511 of Q: 2 blocks of 128 rows
  uint8_t* kv;       // [kPgBufs] entry tiles
  uint8_t* p;        // [kPgBufs] P tiles
  float* mx;         // [2][64] tile maxima by tile parity
  float* alpha;      // [64] rescale factors
  float* lx;         // [2][64] sums over the even and the odd tiles
  float* scl;        // [64] output factors
  uint32_t* valid;   // [kPgBufs] entries present in a tile
  int64_t* start;    // this CTA's range: {its start inside its first item, length, sequence, item}
  uint64_t* bars;
  uint32_t* tmem_base;
};

CSA_DEV PgSmem carve_pg(uint8_t* raw) {
  PgSmem s;
  uint8_t* p = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  s.q = p; p += 2 * kPgQBlk;
  s.kv = p; p += kPgBufs * kPgKVBytes;
  s.p = p; p += kPgBufs * kPgPBytes;
  s.mx = reinterpret_cast<float*>(p); p += 4 * 64 * 4;
  s.alpha = reinterpret_cast<float*>(p); p += 64 * 4;
  s.lx = reinterpret_cast<float*>(p); p += 2 * 64 * 4;
  s.scl = reinterpret_cast<float*>(p); p += 64 * 4;
  s.bars = reinterpret_cast<uint64_t*>(p); p += 24 * 8;
  s.start = reinterpret_cast<int64_t*>(p); p += 4 * 8;
  s.valid = reinterpret_cast<uint32_t*>(p); p += 4 * 4;
  s.tmem_base = reinterpret_cast<uint32_t*>(p);
  return s;
}

CSA_DEV uint32_t pg_h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
CSA_DEV __half2 pg_u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
CSA_DEV float pg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bounded wait by a whole warp, the same answer in every lane.
CSA_DEV bool pg_wait_warp(uint64_t* bar, uint32_t parity, int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, &g_pg_error, code));
}

// MMAs with descriptors given by their low words (the high words are
// constants of the layout), so that an unrolled sequence costs one addition
// per operand; issued by one lane of a warp that runs its loops as a whole.
constexpr uint32_t kPgDescK = (1024u >> 4) | 1u << 14 | 2u << 29;    // K-major, 128-byte swizzle: high word
CSA_DEV uint32_t pg_desc_k(uint32_t smem_addr) { return (smem_addr >> 4) | 1u << 16; }
CSA_DEV uint32_t pg_desc_mn(uint32_t smem_addr, uint32_t lbo) { return (smem_addr >> 4) | (lbo >> 4) << 16; }
template <bool ACC>
CSA_DEV void pg_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}"
      ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kPgDescK), "n"(ACC ? 1 : 0) : "memory");
}
template <bool ACC>
CSA_DEV void pg_mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}"
      ::"r"(d), "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kPgDescK), "n"(ACC ? 1 : 0) : "memory");
}
// P rows are 64 bytes (32 fp16): 64-byte swizzle for that operand.
constexpr uint32_t kPgDescP = (512u >> 4) | 1u << 14 | 4u << 29;
template <bool ACC>
CSA_DEV void pg_mma_pv(uint32_t d, uint32_t v_lo, uint32_t p_lo, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}"
      ::"r"(d), "r"(v_lo), "r"(p_lo), "r"(idesc), "n"(kPgDescK), "n"(kPgDescP), "n"(ACC ? 1 : 0) : "memory");
}
CSA_DEV bool pg_elect() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}

// ------------------------------------------------------------- work items --
struct PgSeq {
  int n;        // new tokens
  int kv;       // cache length with them, >= 0
  int row0;     // first packed row
  int tiles;    // items of 64 (token, head) rows
};
CSA_DEV PgSeq pg_seq(const csa_paged_attn_args& a, int b) {
  PgSeq s;
  const int hi = (int)a.n_rows;
  s.row0 = min(max(a.kv.cu_q[b], 0), hi);
  s.n = min(max(a.kv.cu_q[b + 1], s.row0), hi) - s.row0;
  s.kv = max(a.kv.kv_len[b], 0);
  s.tiles = (int)(((int64_t)s.n * a.H + kPgRows - 1) / kPgRows);
  return s;
}
// Positions [k0, k1) that the rows of item j see (k1 = k0: none), before the
// rows' own masks.  Row r of the item is (token, head) row 64 j + r.
CSA_DEV void pg_item(const csa_paged_attn_args& a, const PgSeq& s, int j, int& k0, int& k1) {
  const int r0 = j * kPgRows, r1 = min(r0 + kPgRows, s.n * a.H) - 1;
  const int p0 = s.kv - s.n + r0 / a.H, p1 = s.kv - s.n + r1 / a.H;
  k1 = min(p1 + 1, a.kv.max_pages * a.kv.page_size);
  k0 = a.window ? max(0, p0 + 1 > a.window ? p0 + 1 - a.window : 0) : 0;
  if (k1 < k0) k1 = k0;
}
CSA_DEV int pg_tiles(int k0, int k1) { return (k1 - k0 + kPgE - 1) / kPgE; }

// The CTA's walk over its items.  An item of T key tiles spans kPgItemCost + T
// of the cost axis; the CTA takes the tiles whose place lies in its range.
struct PgWalk {
  int64_t left;    // cost left, from this item's start in the range on
  int b, j;        // sequence, item
  int at;          // where in the item the range starts
  PgSeq s;
  int k0, k1, total;   // the item's positions and key tiles
  int off, take;       // first key tile taken here, number taken
  CSA_DEV void item(const csa_paged_attn_args& a) {
    pg_item(a, s, j, k0, k1);
    total = pg_tiles(k0, k1);
    off = min(max(at - kPgItemCost, 0), total);
    take = (int)min((int64_t)total, max(at + left - kPgItemCost, (int64_t)0)) - off;
  }
  // does this CTA do anything for the item? (a tileless one belongs to the
  // CTA at its start)
  CSA_DEV bool mine() const { return take > 0 || (total == 0 && at == 0); }
  CSA_DEV void settle(const csa_paged_attn_args& a) {
    while (left > 0 && !mine()) step(a);
  }
  CSA_DEV void step(const csa_paged_attn_args& a) {
    left -= kPgItemCost + total - at;
    at = 0;
    if (left <= 0) return;
    if (++j >= s.tiles) {
      j = 0;
      do {
        if (++b >= a.kv.B) { left = 0; return; }
        s = pg_seq(a, b);
      } while (s.tiles == 0);
    }
    item(a);
  }
  CSA_DEV bool begin(const csa_paged_attn_args& a, const int64_t* start) {
    at = (int)start[0];
    left = start[1];
    b = (int)start[2];
    j = (int)start[3];
    if (left <= 0) return false;
    s = pg_seq(a, b);
    item(a);
    settle(a);
    return left > 0;
  }
  CSA_DEV bool next(const csa_paged_attn_args& a) {
    step(a);
    settle(a);
    return left > 0;
  }
};

CSA_DEV int64_t pg_warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Cost of sequences 32 g + lane (0 past the last).  Sequences with many
// items are summed by the whole warp.
CSA_DEV int64_t pg_group_cost(const csa_paged_attn_args& a, int g, int lane) {
  const int b = 32 * g + lane;
  PgSeq s{0, 0, 0, 0};
  if (b < a.kv.B) s = pg_seq(a, b);
  int64_t u = 0;
  if (s.tiles <= 4) {
    for (int j = 0; j < s.tiles; ++j) {
      int k0, k1;
      pg_item(a, s, j, k0, k1);
      u += kPgItemCost + pg_tiles(k0, k1);
    }
  }
  for (uint32_t big = __ballot_sync(0xffffffffu, s.tiles > 4); big; big &= big - 1) {
    const int l = __ffs(big) - 1;
    PgSeq q;
    q.n = __shfl_sync(0xffffffffu, s.n, l);
    q.kv = __shfl_sync(0xffffffffu, s.kv, l);
    q.row0 = 0;
    q.tiles = __shfl_sync(0xffffffffu, s.tiles, l);
    int64_t v = 0;
    for (int j = lane; j < q.tiles; j += 32) {
      int k0, k1;
      pg_item(a, q, j, k0, k1);
      v += kPgItemCost + pg_tiles(k0, k1);
    }
    v = pg_warp_sum64(v);
    if (lane == l) u = v;
  }
  return u;
}
// Lane whose value the running sum `at` (0 <= at < the warp's sum) falls in;
// `at` becomes the offset inside it.  v >= 0.
CSA_DEV int pg_locate(int64_t v, int64_t& at, int lane) {
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  const int l = __ffs(__ballot_sync(0xffffffffu, at < inc)) - 1;
  const int64_t before = __shfl_sync(0xffffffffu, inc - v, l < 0 ? 0 : l);
  at -= before;
  return l < 0 ? 0 : l;
}
// Finds the CTA's range of the cost axis; every warp of the CTA takes part.
CSA_DEV void pg_plan(const csa_paged_attn_args& a, const PgSmem& S, int warp, int lane) {
  int64_t* gsum = reinterpret_cast<int64_t*>(S.kv);
  const int groups = (a.kv.B + 31) / 32;
  for (int g = warp; g < groups; g += kPgWarps) {
    const int64_t u = pg_warp_sum64(pg_group_cost(a, g, lane));
    if (lane == 0) gsum[g] = u;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t total = 0;
    for (int g = lane; g < groups; g += 32) total += gsum[g];
    total = pg_warp_sum64(total);
    const int64_t G = min((int64_t)gridDim.x, (total + 1) / 2);
    int64_t u0 = 0, u1 = 0;
    if ((int64_t)blockIdx.x < G) {
      u0 = total * blockIdx.x / G;
      u1 = total * (blockIdx.x + 1) / G;
    }
    int64_t at = u0;
    int b = 0, j = 0;
    if (u1 > u0) {
      int base = 0;
      for (;; base += 32) {                                // the 32 groups
        const int64_t v = base + lane < groups ? gsum[base + lane] : 0;
        const int64_t sum = pg_warp_sum64(v);
        if (at < sum || base + 32 >= groups) {
          base += pg_locate(v, at, lane);
          break;
        }
        at -= sum;
      }
      const int64_t v = pg_group_cost(a, base, lane);     // the sequence
      b = 32 * base + pg_locate(v, at, lane);
      const PgSeq s = pg_seq(a, b);
      for (;; j += 32) {                                   // the item
        int64_t w = 0;
        if (j + lane < s.tiles) {
          int k0, k1;
          pg_item(a, s, j + lane, k0, k1);
          w = kPgItemCost + pg_tiles(k0, k1);
        }
        const int64_t sum = pg_warp_sum64(w);
        if (at < sum || j + 32 >= s.tiles) {
          j += pg_locate(w, at, lane);
          break;
        }
        at -= sum;
      }
    }
    if (lane == 0) {
      S.start[0] = at;
      S.start[1] = u1 - u0;
      S.start[2] = b;
      S.start[3] = j;
    }
  }
  __syncthreads();
}

// --------------------------------------------------------------- decoding --
// Operand channel order.  Inside every group of 8 channels the staged K, V
// and Q hold them in the order in which shifts and masks produce fp16 pairs
// from a word of codes: FP8 words of 4 codes give (0, 2), (1, 3); FP4 words
// of 8 codes give (0, 4), (1, 5), (2, 6), (3, 7).  S does not depend on the
// order, and the output undoes it.
template <bool FP4>
CSA_DEV int pg_channel(int pos) {   // channel at operand position pos
  return FP4 ? (pos & ~7) | ((pos & 7) >> 1) | ((pos & 1) << 2)
             : (pos & ~3) | ((pos & 3) >> 1) | ((pos & 1) << 1);
}
// 8 query channels as four operand words.
template <bool FP4>
CSA_DEV void pg_q_words(const float (&f)[8], uint32_t (&o)[4]) {
  if (FP4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = pg_h2u(__floats2half2_rn(f[k], f[k + 4]));
  } else {
    o[0] = pg_h2u(__floats2half2_rn(f[0], f[2]));
    o[1] = pg_h2u(__floats2half2_rn(f[1], f[3]));
    o[2] = pg_h2u(__floats2half2_rn(f[4], f[6]));
    o[3] = pg_h2u(__floats2half2_rn(f[5], f[7]));
  }
}
CSA_DEV void pg_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
// E4M3 codes in bytes 0 and 2 (and 1 and 3) of w as fp16 pairs E4M3 * 2^-8:
// exponent and mantissa move to bits 7..13, the sign to bit 15; subnormals
// land on subnormals, so every code is exact.
CSA_DEV uint32_t pg_e4m3_02(uint32_t w) { return ((w << 7) & 0x3F803F80u) | ((w << 8) & 0x80008000u); }
CSA_DEV uint32_t pg_e4m3_13(uint32_t w) { return ((w >> 1) & 0x3F803F80u) | (w & 0x80008000u); }
// 16 codes of one FP8 block half -> two 8-channel chunks of fp16 values
// (E4M3 * 2^-8) * f2, f2 = 2^(exponent byte - 119) twice, a power of two that
// fp16 holds (exponent bytes 105..134), or 0.
CSA_DEV void pg_decode_fp8(const uint4& v, uint32_t f2, uint4& c0, uint4& c1) {
  const __half2 f = pg_u2h(f2);
  c0 = make_uint4(pg_h2u(__hmul2(pg_u2h(pg_e4m3_02(v.x)), f)), pg_h2u(__hmul2(pg_u2h(pg_e4m3_13(v.x)), f)),
                  pg_h2u(__hmul2(pg_u2h(pg_e4m3_02(v.y)), f)), pg_h2u(__hmul2(pg_u2h(pg_e4m3_13(v.y)), f)));
  c1 = make_uint4(pg_h2u(__hmul2(pg_u2h(pg_e4m3_02(v.z)), f)), pg_h2u(__hmul2(pg_u2h(pg_e4m3_13(v.z)), f)),
                  pg_h2u(__hmul2(pg_u2h(pg_e4m3_02(v.w)), f)), pg_h2u(__hmul2(pg_u2h(pg_e4m3_13(v.w)), f)));
}
// Any exponent byte: fp32 product, rounded to fp16.
CSA_DEV void pg_decode_fp8_far(const uint4& v, int ex, uint4& c0, uint4& c1) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
  const float f = exp2f((float)(ex - 119));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = __half22float2(pg_u2h(pg_e4m3_02(w[k]))), b = __half22float2(pg_u2h(pg_e4m3_13(w[k])));
    o[2 * k] = pg_h2u(__floats2half2_rn(a.x * f, a.y * f));
    o[2 * k + 1] = pg_h2u(__floats2half2_rn(b.x * f, b.y * f));
  }
  c0 = make_uint4(o[0], o[1], o[2], o[3]);
  c1 = make_uint4(o[4], o[5], o[6], o[7]);
}
// One word of 8 FP4 codes with block scale s2 = (E4M3 scale) * 2^7 -> 8 fp16
// values E2M1 * s * 2^-7 (at most 6 significant bits and >= 2^-17: exact).
template <int kk>
CSA_DEV uint32_t pg_e2m1_pair(uint32_t w) {   // codes kk and kk + 4 as E2M1 * 2^-14
  const uint32_t mag = kk < 3 ? (w << (9 - 4 * kk)) : (w >> 3);
  const uint32_t sgn = w << (12 - 4 * kk);
  return (mag & 0x0E000E00u) | (sgn & 0x80008000u);
}
CSA_DEV uint4 pg_decode_fp4(uint32_t w, __half2 s2) {
  return make_uint4(pg_h2u(__hmul2(pg_u2h(pg_e2m1_pair<0>(w)), s2)), pg_h2u(__hmul2(pg_u2h(pg_e2m1_pair<1>(w)), s2)),
                    pg_h2u(__hmul2(pg_u2h(pg_e2m1_pair<2>(w)), s2)), pg_h2u(__hmul2(pg_u2h(pg_e2m1_pair<3>(w)), s2)));
}
CSA_DEV __half2 pg_fp4_scale(uint32_t code) {   // E4M3 scale * 2^7, twice
  return __hmul2(pg_u2h(pg_e4m3_02(code | (code << 16))), pg_u2h(0x78007800u));
}

// Stages half g of an item's 64 query rows: channels 192 g .. 192 g + 191 into
// TMEM (twice: lanes L and L + 64 hold row L), channels 384 + 64 g .. into
// shared block g.  Called by the 4 warps of decode group g; rows past the
// sequence are zero.  Loads are issued before the wait for the operand's last
// reader.
template <bool FP4, typename Wait>
CSA_DEV bool pg_stage_q(const csa_paged_attn_args& a, const PgWalk& w, uint8_t* qblk, uint32_t tbase, int warp, int lane, int g,
                        Wait wait) {
  const int n_rows = w.s.n * a.H - w.j * kPgRows;          // rows left in the sequence from this item on
  const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q);
  auto q_row = [&](int rr) -> const __nv_bfloat16* {
    const int ri = w.j * kPgRows + rr, tok = ri / a.H;
    return qb + (int64_t)(w.s.row0 + tok) * a.q_row_stride + (int64_t)(ri - tok * a.H) * a.q_head_stride;
  };
  const int wl = warp & 3, rr = (32 * wl + lane) & 63;
  const bool on = rr < n_rows;
  const uint4* src = reinterpret_cast<const uint4*>(q_row(on ? rr : 0)) + 24 * g;
  bool ok = true;
#pragma unroll 1
  for (int u = 0; u < 2; ++u) {                            // 48 columns: 96 channels
    uint4 v[12];
#pragma unroll
    for (int k = 0; k < 12; ++k) v[k] = on ? src[12 * u + k] : make_uint4(0, 0, 0, 0);
    if (u == 0) {
      ok = wait();
      if (!ok) break;
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      uint32_t o[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
        uint32_t ow[4];
        pg_bf16x8(v[4 * q + k], f);
        pg_q_words<FP4>(f, ow);
#pragma unroll
        for (int m = 0; m < 4; ++m) o[4 * k + m] = ow[m];
      }
      tmem_st16(tbase + ((uint32_t)(32 * wl) << 16) + 96u * g + 48u * u + 16u * q, o);
    }
  }
  if (ok) {
    const int st = 32 * wl + lane, c8 = st & 7;            // 128 threads: 16 rows x 8 chunks, 4 times
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (st >> 3) + 16 * k;
      v[k] = r < n_rows ? *reinterpret_cast<const uint4*>(q_row(r) + 384 + 64 * g + 8 * c8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (st >> 3) + 16 * k;
      float f[8];
      pg_bf16x8(v[k], f);
      if (a.rope_cs && g == 1 && r < n_rows) {             // channels 448 + 8 c8 ..
        const int tok = w.s.row0 + (w.j * kPgRows + r) / a.H;
        const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + (int64_t)tok * 64 + 8 * c8);
        const float4 ca = cs[0], cb = cs[1];
        float2 x;
        x = rope_fwd(f[0], f[1], ca.x, ca.y); f[0] = x.x; f[1] = x.y;
        x = rope_fwd(f[2], f[3], ca.z, ca.w); f[2] = x.x; f[3] = x.y;
        x = rope_fwd(f[4], f[5], cb.x, cb.y); f[4] = x.x; f[5] = x.y;
        x = rope_fwd(f[6], f[7], cb.z, cb.w); f[6] = x.x; f[7] = x.y;
      }
      uint32_t ow[4];
      pg_q_words<FP4>(f, ow);
      const uint4 o = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      *reinterpret_cast<uint4*>(qblk + sw128_offset_h(r, 8 * c8)) = o;
      *reinterpret_cast<uint4*>(qblk + sw128_offset_h(r + 64, 8 * c8)) = o;
    }
    tmem_wait_st();
    fence_proxy_async_smem();
    tc_fence_before();
  }
  __syncwarp();
  return ok;
}

// A position in the CTA's list of key tiles.
struct PgCursor {
  PgWalk w;
  int i;           // tile of the item
  bool live;
  CSA_DEV void begin(const csa_paged_attn_args& a, const int64_t* start, int skip) {
    live = w.begin(a, start);
    i = 0;
    advance(a, skip);
  }
  CSA_DEV void advance(const csa_paged_attn_args& a, int n) {
    i += n;
    while (live && i >= w.take) {
      i -= w.take;
      live = w.next(a);
    }
  }
};

template <bool FP4>
__global__ void __launch_bounds__(kPgThreads, 1) paged_attn_kernel(const __grid_constant__ PgParams p) {
  constexpr int kScaleOff = FP4 ? 256 : 512;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const PgSmem S = carve_pg(smem_raw);
  uint64_t* kv_full = S.bars + 0;    // [kPgBufs] tile decoded (4 warp arrivals)
  uint64_t* kv_free = S.bars + 4;    // [kPgBufs] PV done: entry tile and P tile reusable
  uint64_t* p_full = S.bars + 8;     // [kPgBufs] P written, O^T rescaled (2 warp arrivals)
  uint64_t* s_full = S.bars + 12;    // [2] S in TMEM
  uint64_t* s_free = S.bars + 14;    // [2] S read by the softmax (2 warp arrivals)
  uint64_t* q_full = S.bars + 16;    // an item's Q staged (8 warp arrivals)
  uint64_t* q_free = S.bars + 17;    // an item's last S done
  uint64_t* acc_done = S.bars + 18;  // an item's last PV done
  uint64_t* drain = S.bars + 19;     // [2] all MMAs of an issuer retired (teardown)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const csa_paged_attn_args& a = p.a;
  if (tid == 0) {
    for (int k = 0; k < kPgBufs; ++k) {
      mbar_init(kv_full + k, 4);
      mbar_init(kv_free + k, 1);
      mbar_init(p_full + k, 2);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(s_full + k, 1);
      mbar_init(s_free + k, 2);
      mbar_init(drain + k, 1);
    }
    mbar_init(q_full, kPgDeqWarps);
    mbar_init(q_free, 1);
    mbar_init(acc_done, 1);
    fence_mbar_init();
  }
  if (warp == kPgWarpS) tmem_alloc(S.tmem_base, kPgTmemCols);
  pdl_wait();
  pg_plan(a, S, warp, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *S.tmem_base;

  if (warp == kPgWarpS) {
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t idesc = idesc_make(kFmtF16, kFmtF16, 128, kPgE);
    const uint32_t qd = pg_desc_k(smem_u32(S.q)), kvd = pg_desc_k(smem_u32(S.kv));
    PgWalk w;
    uint32_t t = 0, seg = 0;
    bool ok = true;
    for (bool go = w.begin(a, S.start); go && ok; go = w.next(a)) {
      if (w.take == 0) continue;
      ok = pg_wait_warp(q_full, seg++ & 1u, kErrWaitTmaFull);
      for (int i = 0; i < w.take && ok; ++i, ++t) {
        const uint32_t bi = t % kPgBufs;
        ok = pg_wait_warp(kv_full + bi, (t / kPgBufs) & 1u, kErrWaitTmaFull);
        if (ok && t >= 2) ok = pg_wait_warp(s_free + (t & 1u), ((t >> 1) - 1) & 1u, kErrWaitAccEmpty);
        if (!ok) break;
        tc_fence_after();
        const uint32_t kd = kvd + bi * (kPgKVBytes >> 4), sd = tbase + kPgSCol + kPgE * (t & 1u);
        if (pg_elect()) {
          pg_mma_ts<false>(sd, tbase, kd, idesc);
#pragma unroll
          for (int ks = 1; ks < kD / 16; ++ks) {
            const uint32_t kb = ks >> 2, sub = ks & 3;
            const uint32_t bd = kd + kb * (kPgKVBlk >> 4) + sub * 2;
            if (kb < (uint32_t)kPgQTmemBlocks) pg_mma_ts<true>(sd, tbase + kb * 32 + sub * 8, bd, idesc);
            else pg_mma_ss<true>(sd, qd + (kb - kPgQTmemBlocks) * (kPgQBlk >> 4) + sub * 2, bd, idesc);
          }
          mma_commit(s_full + (t & 1u));
          if (i == w.take - 1) mma_commit(q_free);
        }
        __syncwarp();
      }
    }
    if (pg_elect()) {
      mma_commit(drain);
      mbar_wait(drain, 0u, &g_pg_error, kErrWaitAccFull);
    }
    __syncwarp();
  } else if (warp == kPgWarpPV) {
    // ----------------------------------------------------------- PV issuer
    constexpr uint32_t idesc = idesc_make_amn(kFmtF16, kFmtF16, 128, kPgRows);
    const uint32_t kvd = pg_desc_mn(smem_u32(S.kv), kPgKVBlk), pd = pg_desc_k(smem_u32(S.p));
    PgWalk w;
    uint32_t t = 0;
    bool ok = true;
    for (bool go = w.begin(a, S.start); go && ok; go = w.next(a)) {
      for (int i = 0; i < w.take; ++i, ++t) {
        const uint32_t bi = t % kPgBufs;
        ok = pg_wait_warp(p_full + bi, (t / kPgBufs) & 1u, kErrWaitAccFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t vd = kvd + bi * (kPgKVBytes >> 4), pb = pd + bi * (kPgPBytes >> 4);
        if (pg_elect()) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int ks = 0; ks < kPgE / 16; ++ks) {
              const uint32_t ad = vd + 2 * c * (kPgKVBlk >> 4) + ks * (2048 >> 4), bd = pb + ks * 2;
              if (ks == 0 && i == 0) pg_mma_pv<false>(tbase + kPgOCol + 64u * c, ad, bd, idesc);
              else pg_mma_pv<true>(tbase + kPgOCol + 64u * c, ad, bd, idesc);
            }
          }
          mma_commit(kv_free + bi);
          if (i == w.take - 1) mma_commit(acc_done);
        }
        __syncwarp();
      }
    }
    if (pg_elect()) {
      mma_commit(drain + 1);
      mbar_wait(drain + 1, 0u, &g_pg_error, kErrWaitAccFull);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------- entry loads and decoding
    // Group g (4 warps) takes the CTA's tiles of parity g, 8 entries a warp.
    const int wq = (warp - 4) & 3, g = (warp - 4) >> 2;
    PgCursor cu;                       // the tile whose page table values are fetched next
    cu.begin(a, S.start, g);
    // page id and entry number in the page of entry 8 wq + (lane & 7) of the
    // tile whose entries are loaded next
    int id = -1;
    uint32_t slot = 0;
    auto lookup = [&]() {
      id = -1;
      if (cu.live) {
        const int pos = cu.w.k0 + (cu.w.off + cu.i) * kPgE + 8 * wq + (lane & 7);
        if (pos < cu.w.k1) {
          const uint32_t pg = (uint32_t)pos / (uint32_t)a.kv.page_size;
          slot = (uint32_t)pos - pg * (uint32_t)a.kv.page_size;
          id = a.kv.block_table[(int64_t)cu.w.b * a.kv.table_stride + pg];
        }
      }
    };
    constexpr int kN = FP4 ? 4 : 8;    // 16-byte words per lane and tile
    uint4 r[kN];
    uint2 sc;
    uint32_t vb;                       // valid entries of this warp's 8
    // address of lane l's entry 8 wq + (l & 7); where there is none, the
    // cache's first entry: every load is issued, and the decoder writes zeros
    auto entry_ptr = [&](uint32_t& v) -> unsigned long long {
      const bool on = id >= 0 && id < a.kv.n_pages;
      v = __ballot_sync(0xffffffffu, on) & 0xFFu;
      return (unsigned long long)(a.kv.pages + (on ? (int64_t)id * a.kv.page_stride + (int64_t)slot * a.kv.row_stride : 0));
    };
    // FP8: word k is bytes [16 lane, 16 lane + 16) of entry k; FP4: bytes
    // [16 (lane & 15), ..) of entry 2k + (lane >> 4)
    auto load_word = [&](unsigned long long ptr, int k) -> uint4 {
      const unsigned long long q = __shfl_sync(0xffffffffu, ptr, FP4 ? 2 * k + (lane >> 4) : k);
      return ld_nc_v4(reinterpret_cast<const uint8_t*>(q) + 16 * (FP4 ? lane & 15 : lane));
    };
    // scales: lane 4e + w holds word w of entry e's scale bytes
    auto load_scales = [&](unsigned long long ptr) -> uint2 {
      const uint8_t* q = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, ptr, lane >> 2)) + kScaleOff;
      if (FP4) return *reinterpret_cast<const uint2*>(q + 8 * (lane & 3));
      return make_uint2(*reinterpret_cast<const uint32_t*>(q + 4 * (lane & 3)), 0);
    };
    lookup();
    {
      const unsigned long long ptr = entry_ptr(vb);
#pragma unroll
      for (int k = 0; k < kN; ++k) r[k] = load_word(ptr, k);
      sc = load_scales(ptr);
    }
    cu.advance(a, 2);
    lookup();
    PgWalk w;
    uint32_t t0 = 0, seg = 0;          // tiles before the item, items with tiles before it
    bool ok = true;
    for (bool go = w.begin(a, S.start); go && ok; go = w.next(a)) {
    if (w.take == 0) continue;
    ok = pg_stage_q<FP4>(a, w, S.q + g * kPgQBlk, tbase, warp, lane, g, [&]() {
      const bool k = seg == 0 || pg_wait_warp(q_free, (seg - 1) & 1u, kErrWaitSmemEmpty);
      tc_fence_after();
      return k;
    });
    if (!ok) break;
    if (lane == 0) mbar_arrive(q_full);
    ++seg;
    {
      // the next item's rows into L2 (an item's rows are contiguous when the
      // heads are): 128 bytes a thread and step, half a row's two lines a group
      PgWalk nx = w;
      if (nx.next(a) && nx.take > 0) {
        const int nr = min(nx.s.n * a.H - nx.j * kPgRows, kPgRows);
        for (int l = 32 * (warp & 3) + lane; l < 4 * nr; l += 128) {
          const int ri = nx.j * kPgRows + (l >> 2), tok = ri / a.H;
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(nx.s.row0 + tok) * a.q_row_stride +
                                   (int64_t)(ri - tok * a.H) * a.q_head_stride + 64 * (4 * g + (l & 3));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        }
      }
    }
    uint32_t t = t0 + ((t0 ^ (uint32_t)g) & 1u);
    t0 += (uint32_t)w.take;
    for (; t < t0; t += 2) {
      const uint32_t bi = t % kPgBufs;
      if (t >= kPgBufs && !pg_wait_warp(kv_free + bi, (t / kPgBufs - 1) & 1u, kErrWaitSmemEmpty)) {
        ok = false;
        break;
      }
      uint8_t* kt = S.kv + bi * kPgKVBytes;
      if (FP4) {
        const int l16 = lane & 15, kb = l16 >> 1;
        uint8_t* blk = kt + kb * kPgKVBlk;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const int e = 2 * k + (lane >> 4);
          const uint32_t sx = __shfl_sync(0xffffffffu, sc.x, 4 * e + (l16 >> 2));
          const uint32_t sy = __shfl_sync(0xffffffffu, sc.y, 4 * e + (l16 >> 2));
          uint32_t two = ((l16 & 2) ? sy : sx) >> (16 * (l16 & 1));
          if (!((vb >> e) & 1u)) two = 0;                  // no entry: zeros
          const __half2 sa = pg_fp4_scale(two & 0xFF), sb = pg_fp4_scale((two >> 8) & 0xFF);
          const uint4 c[4] = {pg_decode_fp4(r[k].x, sa), pg_decode_fp4(r[k].y, sa), pg_decode_fp4(r[k].z, sb),
                              pg_decode_fp4(r[k].w, sb)};
          // the four chunks in an order by block, so that 8 lanes' stores
          // meet 8 different 16-byte columns
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int cc = m ^ (kb & 3);
            const uint4 v = cc == 0 ? c[0] : cc == 1 ? c[1] : cc == 2 ? c[2] : c[3];
            *reinterpret_cast<uint4*>(blk + sw128_offset_h(8 * wq + e, 32 * (l16 & 1) + 8 * cc)) = v;
          }
        }
      } else {
        const int kb = lane >> 2, f = kb & 1;
        uint8_t* blk = kt + kb * kPgKVBlk;
        const bool on = (vb >> (lane >> 2)) & 1u;          // of the entry whose scales this lane holds
        // any block of the warp's entries with a scale that fp16 cannot hold?
        const bool far = on && __vcmpgtu4(__vsub4(sc.x, 0x69696969u), 0x1D1D1D1Du) != 0;
        const uint32_t ex4 = on ? sc.x - 0x68686868u : 0u; // exponent fields of the fp16 factors; 0: factor 0
        if (!__any_sync(0xffffffffu, far)) {
#pragma unroll
          for (int k = 0; k < kN; ++k) {
            const uint32_t fe = (__shfl_sync(0xffffffffu, ex4, 4 * k + (lane >> 3)) >> (8 * ((lane >> 1) & 3))) & 0xFFu;
            // odd blocks write their second chunk first, so that 8 lanes'
            // stores meet 8 different 16-byte columns
            uint4 c0, c1;
            pg_decode_fp8(f ? make_uint4(r[k].z, r[k].w, r[k].x, r[k].y) : r[k], fe * 0x04000400u, c0, c1);
            *reinterpret_cast<uint4*>(blk + sw128_offset_h(8 * wq + k, 16 * (lane & 3) + 8 * f)) = c0;
            *reinterpret_cast<uint4*>(blk + sw128_offset_h(8 * wq + k, 16 * (lane & 3) + 8 * (f ^ 1))) = c1;
          }
        } else {
#pragma unroll
          for (int k = 0; k < kN; ++k) {
            const uint32_t ex = (__shfl_sync(0xffffffffu, sc.x, 4 * k + (lane >> 3)) >> (8 * ((lane >> 1) & 3))) & 0xFFu;
            uint4 c0 = make_uint4(0, 0, 0, 0), c1 = c0;
            if ((vb >> k) & 1u) pg_decode_fp8_far(r[k], (int)ex, c0, c1);
            *reinterpret_cast<uint4*>(blk + sw128_offset_h(8 * wq + k, 16 * (lane & 3))) = c0;
            *reinterpret_cast<uint4*>(blk + sw128_offset_h(8 * wq + k, 16 * (lane & 3) + 8)) = c1;
          }
        }
      }
      if (lane == 0) reinterpret_cast<uint8_t*>(S.valid)[4 * bi + wq] = (uint8_t)vb;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(kv_full + bi);
      // the next tile's entries, all loads together (issued one by one between
      // the decodes, each decode waits for the load before it: loads share
      // their scoreboards), then the table values of the tile after it
      const unsigned long long ptr = entry_ptr(vb);
#pragma unroll
      for (int k = 0; k < kN; ++k) r[k] = load_word(ptr, k);
      sc = load_scales(ptr);
      cu.advance(a, 2);
      lookup();
    }
    }
  } else {
    // ------------------------------------------------------ softmax, output
    // Warps 0-1 take the CTA's even tiles, warps 2-3 the odd ones: while one
    // pair turns its S into P, the other reads the next S and finds its max.
    // All four meet once per tile, where the running max may move.
    const int rr = 32 * (warp & 1) + lane;     // row of the item
    const uint32_t grp = (uint32_t)warp >> 1;
    const uint32_t trow = tbase + ((uint32_t)(32 * warp) << 16);
    const float sc = p.scale_log2;
    PgWalk w;
    uint32_t t = 0, seg = 0;
    bool ok = true;
    int64_t meta_row0 = 0;
    int meta_rows = 0, meta_cont = 0, meta_done = 0;
    for (bool go = w.begin(a, S.start); go; go = w.next(a)) {
      const int nt = w.take;
      const int n_rows = w.s.n * a.H - w.j * kPgRows;
      const int ri = w.j * kPgRows + rr;
      // positions this row sees: (lo, hi]; none for rows past the sequence
      const int hi = rr < n_rows ? w.s.kv - w.s.n + ri / a.H : -1;
      const int lo = a.window && hi >= a.window ? hi - a.window : -1;
      float m_run = -INFINITY, l_run = 0.f;    // l_run: this pair's tiles
      for (int i = 0; i < nt; ++i, ++t) {
        const uint32_t bi = t % kPgBufs, si = t & 1u;
        const bool own = si == grp;
        uint32_t sv[32], mask = 0;
        float mt = -INFINITY;
        // a failed wait leaves `ok` false and skips the later waits; every
        // warp still passes the group's barriers once per tile
        if (own) {
          const int kb = w.k0 + (w.off + i) * kPgE;
          const int nh = hi - kb + 1, nl = lo - kb + 1;      // the row sees entries [nl, nh) of the tile
          mask = nh >= 32 ? 0xffffffffu : nh <= 0 ? 0u : (1u << nh) - 1u;
          mask &= nl <= 0 ? 0xffffffffu : nl >= 32 ? 0u : ~((1u << nl) - 1u);
          ok = ok && pg_wait_warp(s_full + si, (t >> 1) & 1u, kErrWaitAccFull);
          tc_fence_after();
          tmem_ld32(trow + kPgSCol + kPgE * si, sv);
          mask &= S.valid[bi];                 // written before the tile's S was issued
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + si);
          if (__all_sync(0xffffffffu, mask == 0xffffffffu)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) mt = fmaxf(mt, __uint_as_float(sv[k]));
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) mt = fmaxf(mt, ((mask >> k) & 1u) ? __uint_as_float(sv[k]) : -INFINITY);
          }
          if (mt != -INFINITY) mt *= sc;
          S.mx[64 * si + rr] = mt;
        }
        uint32_t over;
        asm volatile("{\n .reg .pred q, r;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred r, 1, 128, q;\n selp.u32 %0, 1, 0, r;\n}"
                     : "=r"(over) : "r"(mt > m_run + kPgRescale ? 1u : 0u) : "memory");
        if (over) {
          const float mm = S.mx[64 * si + rr];
          float alpha = 1.f;
          if (mm > m_run + kPgRescale) {
            alpha = m_run == -INFINITY ? 0.f : pg_ex2(m_run - mm);
            m_run = mm;
            l_run *= alpha;
          }
          if (i > 0) {
            if (own) S.alpha[rr] = alpha;
            named_bar(1, 128);
            // the PV before this tile's has retired (its tile's buffer is free)
            ok = ok && pg_wait_warp(kv_free + (t - 1) % kPgBufs, ((t - 1) / kPgBufs) & 1u, kErrWaitAccFull);
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {      // 16 rows at a time
              float al[16];
#pragma unroll
              for (int cc = 0; cc < 16; ++cc) al[cc] = S.alpha[16 * k + cc];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t ta = trow + kPgOCol + 64 * c + 16 * k;
                uint32_t o[16];
                tmem_ld16(ta, o);
                tmem_wait_ld();
#pragma unroll
                for (int cc = 0; cc < 16; ++cc) o[cc] = __float_as_uint(__uint_as_float(o[cc]) * al[cc]);
                tmem_st16(ta, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar(1, 128);                 // every quarter rescaled before this tile's PV
          }
        }
        if (own) {
          // this tile's P buffer is free: its entries were decoded after the
          // PV that read both last
          const float mref = m_run - kPgPExp;
          float l0 = 0.f, l1 = 0.f;
          uint8_t* pt = S.p + bi * kPgPBytes;
          const bool full = __all_sync(0xffffffffu, mask == 0xffffffffu);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e0 = 8 * c + 2 * k;
              float x0 = pg_ex2(fmaf(__uint_as_float(sv[e0]), sc, -mref));
              float x1 = pg_ex2(fmaf(__uint_as_float(sv[e0 + 1]), sc, -mref));
              if (!full) {
                x0 = ((mask >> e0) & 1u) ? x0 : 0.f;
                x1 = ((mask >> (e0 + 1)) & 1u) ? x1 : 0.f;
              }
              l0 += x0;
              l1 += x1;
              o[k] = pg_h2u(__floats2half2_rn(x0, x1));
            }
            *reinterpret_cast<uint4*>(pt + sw64_offset(rr, 16 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          l_run += l0 + l1;
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + bi);
        }
      }
      // ------------------------------------------------------------ output
      const bool whole = w.take == w.total;
      S.lx[64 * grp + rr] = l_run;
      named_bar(1, 128);
      const int64_t orow = (int64_t)w.s.row0 * a.H + w.j * kPgRows;
      const int slot = 2 * blockIdx.x + (w.off > 0 ? 0 : 1);
      if (grp == 0) {
        float l = l_run + S.lx[64 + rr];
        if (whole) {
          const float m0 = m_run - kPgPExp;
          float scl, M = m0, L = l;
          if (a.sink) {
            const float s0 = rr < n_rows ? a.sink[ri - ri / a.H * a.H] * kPgLog2e : -INFINITY;
            M = fmaxf(m0, s0);
            const float f = l > 0.f ? exp2f(m0 - M) : 0.f;
            L = l * f + (s0 == -INFINITY ? 0.f : exp2f(s0 - M));
            scl = l > 0.f ? p.out_scale * f / L : 0.f;
          } else {
            scl = l > 0.f ? p.out_scale / l : 0.f;
          }
          if (a.lse && rr < n_rows) a.lse[orow + rr] = L > 0.f ? (M + log2f(L)) * kPgLn2 : -INFINITY;
          S.scl[rr] = scl;
        } else {
          p.part_ml[slot * 64 + rr] = make_float2(m_run, l);
        }
      }
      named_bar(1, 128);
      // every PV of the item
      if (nt > 0) ok = ok && pg_wait_warp(acc_done, seg++ & 1u, kErrWaitAccFull);
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < 8; ++ch) {               // 128 channels x 32 rows at a time
        const int c = ch >> 1, k0 = 32 * (ch & 1);
        const int d = pg_channel<FP4>(128 * c + 32 * warp + lane);
        if (k0 >= n_rows) continue;
        uint32_t o[32];
        if (nt > 0 && ok) {
          tmem_ld32(trow + kPgOCol + 64 * c + k0, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (whole) {
          if (a.rope_cs && d >= kRopeStart) {          // whole warps: 32 channels from 448 or 480
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float v = __uint_as_float(o[k]);
              const float u = __shfl_xor_sync(0xffffffffu, v, 2);   // channel d ^ 1
              const int tok = w.s.row0 + (w.j * kPgRows + min(k0 + k, n_rows - 1)) / a.H;
              const float2 cs = *reinterpret_cast<const float2*>(a.rope_cs + (int64_t)tok * 64 + ((d - kRopeStart) & ~1));
              o[k] = __float_as_uint((d & 1) ? v * cs.x - u * cs.y : v * cs.x + u * cs.y);
            }
          }
          // rows k, k + 1: the lane of the even channel stores row k's pair of
          // channels, the lane of the odd one row k + 1's
          const int odd = d & 1;
          __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(a.out) + (orow + k0 + odd) * kD + (d & ~1);
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 f = *reinterpret_cast<const float2*>(S.scl + k0 + 2 * k);
            const float v0 = __uint_as_float(o[2 * k]) * f.x, v1 = __uint_as_float(o[2 * k + 1]) * f.y;
            const float u = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 2);
            const __nv_bfloat162 h = __floats2bfloat162_rn(odd ? u : v0, odd ? v1 : u);
            v[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (k0 + 32 <= n_rows) {
#pragma unroll
            for (int k = 0; k < 16; ++k) *reinterpret_cast<uint32_t*>(ob + 2 * k * kD) = v[k];
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k0 + 2 * k + odd < n_rows) *reinterpret_cast<uint32_t*>(ob + 2 * k * kD) = v[k];
          }
        } else {
          float* po = p.part_o + (int64_t)slot * (64 * kD) + k0 * kD + d;
          if (k0 + 32 <= n_rows) {
#pragma unroll
            for (int k = 0; k < 32; ++k) po[k * kD] = __uint_as_float(o[k]);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k0 + k < n_rows) po[k * kD] = __uint_as_float(o[k]);
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        if (w.off > 0) {
          meta_cont = 1;
          meta_done = w.off + w.take == w.total;
        } else {
          meta_rows = min(n_rows, kPgRows);
          meta_row0 = orow;
        }
      }
    }
    if (tid == 0) p.meta[blockIdx.x] = PgMeta{meta_row0, meta_rows, meta_cont, meta_done, 0};
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPgWarpS) {
    tc_fence_after();
    tmem_dealloc(tbase, kPgTmemCols);
  }
}

// Joins the partials of the items that several CTAs share.  CTA (i, r): row r
// of the item that CTA i of the attention began and did not finish; its
// partials are slot 2i + 1 and then slot 2k of k = i + 1, i + 2, ... up to
// the CTA that ends the item, added in that order.
__global__ void __launch_bounds__(128) paged_attn_combine_kernel(const __grid_constant__ PgParams p, int n_ctas) {
  pdl_enter();
  const csa_paged_attn_args& a = p.a;
  const int i = blockIdx.x, row = blockIdx.y, lane = threadIdx.x & 31;
  const PgMeta me = p.meta[i];
  if (row >= me.rows) return;
  int n = 1;                                   // partials
  for (int k0 = i + 1; k0 < n_ctas; k0 += 32) {
    const uint32_t end = __ballot_sync(0xffffffffu, k0 + lane < n_ctas && p.meta[k0 + lane].cont && p.meta[k0 + lane].done);
    if (end) {
      n = k0 - i + __ffs(end);
      break;
    }
    n = min(k0 + 32, n_ctas) - i;
  }
  auto slot = [&](int s) { return (int64_t)(s == 0 ? 2 * i + 1 : 2 * (i + s)); };
  const int64_t orow = me.row0 + row;
  const int head = (int)(orow % a.H);
  const float s0 = a.sink ? a.sink[head] * kPgLog2e : -INFINITY;
  float M = -INFINITY;
  for (int s = lane; s < n; s += 32) M = fmaxf(M, p.part_ml[slot(s) * 64 + row].x);
  M = warp_max(M);
  M = fmaxf(M - kPgPExp, s0);
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* po = p.part_o + (int64_t)row * kD + 4 * threadIdx.x;
  for (int sb = 0; sb < n; sb += 32) {
    float wt = 0.f;
    if (sb + lane < n) {
      const float2 ml = p.part_ml[slot(sb + lane) * 64 + row];
      wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - kPgPExp - M);
      L += wt * ml.y;
    }
    const int m = min(32, n - sb);
#pragma unroll 8
    for (int s = 0; s < m; ++s) {
      const float ws = __shfl_sync(0xffffffffu, wt, s);
      const float4 v = *reinterpret_cast<const float4*>(po + slot(sb + s) * (64 * kD));
      acc.x += ws * v.x; acc.y += ws * v.y; acc.z += ws * v.z; acc.w += ws * v.w;
    }
  }
  L = warp_sum(L);
  const bool any = L > 0.f;
  if (s0 != -INFINITY) L += exp2f(s0 - M);
  const float f = any ? p.out_scale / L : 0.f;
  if (threadIdx.x == 0 && a.lse) a.lse[orow] = L > 0.f ? (M + log2f(L)) * kPgLn2 : -INFINITY;
  const float* cs = a.rope_cs ? a.rope_cs + orow / a.H * 64 : nullptr;
  store_out4(a.out, true, orow * kD + 4 * threadIdx.x,
             rope_out4(make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f), cs, 4 * threadIdx.x));
}

// CTAs of a call: one per SM, fewer when the call cannot have that many tiles.
static int pg_grid(const csa_paged_attn_args* a) {
  const int64_t items = (a->n_rows * a->H + kPgRows - 1) / kPgRows + a->kv.B;
  const int64_t tiles = ((int64_t)a->kv.max_pages * a->kv.page_size + kPgE - 1) / kPgE;
  return items * tiles < kNumSMs ? (int)(items * tiles) : kNumSMs;
}
static size_t pg_al256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t paged_attn_ws_bytes(const csa_paged_attn_args* a) {
  const size_t g = (size_t)pg_grid(a);
  return pg_al256(g * sizeof(PgMeta)) + pg_al256(g * 2 * 64 * sizeof(float2)) + g * 2 * 64 * kD * sizeof(float);
}

cudaError_t launch_paged_attn(const csa_paged_attn_args* a, void* ws, cudaStream_t stream) {
  const bool fp4 = a->kv.fmt == CSA_FMT_FP4_E2M1_E4M3X16;
  static SmemAttrOnce attr4, attr8;
  const cudaError_t ea = fp4 ? attr4.set(paged_attn_kernel<true>, kPgSmemBytes) : attr8.set(paged_attn_kernel<false>, kPgSmemBytes);
  if (ea != cudaSuccess) return ea;
  const int g = pg_grid(a);
  PgParams p;
  p.a = *a;
  // FP4 entries are staged times 2^-7
  p.scale_log2 = a->softmax_scale * kPgLog2e * (fp4 ? 128.f : 1.f);
  p.out_scale = fp4 ? 128.f : 1.f;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.meta = reinterpret_cast<PgMeta*>(w);
  w += pg_al256((size_t)g * sizeof(PgMeta));
  p.part_ml = reinterpret_cast<float2*>(w);
  w += pg_al256((size_t)g * 2 * 64 * sizeof(float2));
  p.part_o = reinterpret_cast<float*>(w);
  {
    ProfScope ps(stream, "paged_attn");
    if (fp4) launch_k(paged_attn_kernel<true>, dim3(g), dim3(kPgThreads), kPgSmemBytes, stream, p);
    else launch_k(paged_attn_kernel<false>, dim3(g), dim3(kPgThreads), kPgSmemBytes, stream, p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(stream, "paged_attn_combine");
    launch_k(paged_attn_combine_kernel, dim3(g, 64), dim3(128), 0, stream, p, g);
  }
  note_launches(2);
  return cudaGetLastError();
}

int read_pg_error(bool clear) {
  int v = 0;
  cudaMemcpyFromSymbol(&v, g_pg_error, sizeof(int));
  if (clear && v) {
    int z = 0;
    cudaMemcpyToSymbol(g_pg_error, &z, sizeof(int));
  }
  return v;
}

}  // namespace csa
