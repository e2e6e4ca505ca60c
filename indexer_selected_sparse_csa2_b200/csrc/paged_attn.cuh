// Shared by the kernels of csa_paged_attn: the division of a batch into work
// items and of those among the parts of the grid, decoding of cache entries,
// staging of queries, tcgen05 operands.
//
// A work item is up to ROWS query rows (token, head) of one sequence, rows in
// (token, head) order, so any head count fills it; it runs over the key tiles
// of kPgTile entries that its rows see.
//
// Work split: the batch is a line on which an item of T key tiles takes
// kPgItemCost + T; part i of G (a CTA pair, or a CTA) takes the tiles on
// [iU/G, (i+1)U/G) of its length U, whatever the sequences' lengths, and
// computes where that is from the lengths on the device.  An item that ends up
// in several parts leaves (max, sum, O) partials in the workspace, at most two
// per part, which the combine joins in order; the result does not depend on
// timing.
//
// Online softmax in the exp2 domain; the running max moves only when a tile's
// max exceeds it by kPgRescale or more, and only then O is rescaled in TMEM.
// P is held in fp16 times 2^6: at most 2^14, and weights down to 2^-31 of the
// max keep a value.  One fp16 part, where csa_sparse_attn's kernels hold P in
// two: a second one doubles PV's MMAs (512 of a pair's 2050 cycles a tile).  The
// rounding, 2^-11 of a weight, is below the output's own to bf16 except where
// large values cancel: in channels of 20 times the others' size, rms 20, outputs
// were off by up to 0.0034 beside it, and 0.1 % of them by more than 0.001 +
// 0.002 |out|.  (Past 2^24 fp32 values are 2 and more apart, and 6 - max
// may round up to 8 - max: with less than kPgRescale between a logit and the
// running max that still stays below 2^13.)
#pragma once
#include <climits>

#include "sm100.cuh"
#include "paged.cuh"
#include "rope.cuh"

namespace csa {

// Entries per key tile, by an item's rows.
template <int ROWS>
constexpr int kPgTile = ROWS == 64 ? 32 : 64;
constexpr int kPgE = kPgTile<128>;
constexpr int kPgOwn = 32;                // ... decoded together
constexpr int kPgQTmemBlocks = 6;         // 64-channel blocks of Q in TMEM
// warps 0-3: softmax and output
constexpr int kPgWarpDec = 4;             // first decode warp (two groups of 4)
constexpr int kPgWarpS = 12;             // S issuer
constexpr int kPgWarpPV = 13;            // PV issuer
constexpr int kPgWarps = 14;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr uint32_t kPgSCol = 32 * kPgQTmemBlocks;   // S: 64 columns
constexpr uint32_t kPgOCol = 256;
constexpr uint32_t kPgTmemCols = 512;
static_assert(kPgSCol + kPgE <= kPgOCol, "TMEM map");
// An item's own cost (Q, first tile, output) in key tiles, by its rows.  Pairs: 8
// prompts of up to 2047 tokens take 748, 678, 696 and 715 us with 2, 4, 6 and 8.
// One CTA, tiles half as long: 64 sequences' tokens, 64 heads each, behind 1 to
// 8000 FP8 entries take 111, 102, 89, 81 and 79 us with 4, 6, 8, 12 and 16; 200
// sequences' tokens, 16 heads each, behind 1 to 2000 FP4 entries 96, 81, 73, 65
// and 67.  Batches of equal lengths take the same with each.
template <int ROWS>
constexpr int kPgItemCost = ROWS == 64 ? 12 : 4;
constexpr float kPgRescale = 8.0f;        // lazy-rescale threshold (exp2 units)
constexpr float kPgPExp = 6.0f;           // P carries a factor 2^6
constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgLn2 = 0.6931471805599453f;
constexpr int kPgMaxB = 65536;
constexpr int kPgKBlk = kPgOwn * 128;     // 64-channel block of a decoded tile of 32 entries
constexpr int kPgKBytes = 8 * kPgKBlk;

static __device__ int g_pg_error;

// What a part of the grid (a pair of CTAs, or one) left for the combine.
struct PgMeta {
  int64_t row0;      // leader: first output row (token * H + head) of its last item
  int32_t rows;      // leader: rows of that item; 0 = its last item is not split here
  int32_t cont;      // its first item began in an earlier part ...
  int32_t done;      // ... and ends here
  int32_t pad;
};

struct PgParams {
  csa_paged_attn_args a;
  float scale_log2;  // softmax_scale * log2(e)
  uint32_t page_inv, h_inv;   // pg_inv of page_size and H
  float* part_o;     // [2 * parts][rows of an item][512] fp32
  float2* part_ml;   // [2 * parts][rows of an item] (max, sum)
  int item_rows;     // query rows per item
  PgMeta* meta;      // [parts]
};

// 16 bytes of an entry.  AGAIN: other items will read them from L2; else they
// are read once.  (no_allocate in L1 marks a line as L2's first to evict: a
// third of the chunks' reads then went to HBM, 2.33 ms for 2.24.)
template <bool AGAIN>
CSA_DEV uint4 pg_ld_entry(const void* p) {
  uint4 r;
  if (AGAIN) asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  else asm volatile("ld.global.nc.L1::evict_first.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
CSA_DEV uint32_t pg_h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
CSA_DEV float pg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 logits times the scale, and minus the max, two an instruction (one fma for
// both would need as many).  The product is rounded before the difference is
// taken: a max is a rounded product too, and where logits pass 2^24 an fma's
// exact product may lie whole units from it, so that the largest weight left
// fp16's range or vanished.
CSA_DEV void pg_mul32(uint32_t (&s)[32], float f) {
#pragma unroll
  for (int k = 0; k < 32; k += 2)
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "+r"(s[k]), "+r"(s[k + 1]) : "f"(f));
}
CSA_DEV void pg_add32(uint32_t (&s)[32], float f) {
#pragma unroll
  for (int k = 0; k < 32; k += 2)
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "+r"(s[k]), "+r"(s[k + 1]) : "f"(f));
}

// Bounded wait by a whole warp, the same answer in every lane.
CSA_DEV bool pg_wait_warp(uint64_t* bar, uint32_t parity, int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, &g_pg_error, code));
}
// Bounded wait by a whole warp for a count in shared memory; giving up is no error.
CSA_DEV bool pg_wait_count(const volatile uint32_t* count, uint32_t n) {
  const uint64_t t0 = global_ns();
  bool there = *count >= n;
  while (!there && global_ns() - t0 <= kWaitNs) {
    __nanosleep(200);
    there = *count >= n;
  }
  return __all_sync(0xffffffffu, there);
}
// MMAs with descriptors given by their low words (the high word is a constant
// of the layout: 128-byte swizzle, 8-row groups 1024 bytes apart), so that an
// unrolled sequence costs one addition per operand; issued by one lane of a
// warp that runs its loops as a whole.
constexpr uint32_t kPgDesc = (1024u >> 4) | 1u << 14 | 2u << 29;
CSA_DEV uint32_t pg_desc_k(uint32_t smem_addr) { return (smem_addr >> 4) | 1u << 16; }
CSA_DEV uint32_t pg_desc_mn(uint32_t smem_addr, uint32_t lbo) { return (smem_addr >> 4) | (lbo >> 4) << 16; }
CSA_DEV bool pg_elect() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}

// n / d for 0 <= n < 2^31: the product with floor(2^32 / d) is at most one short
// (d = 1: with 2^32 - 1).
static uint32_t pg_inv(uint32_t d) { return d == 1 ? 0xffffffffu : (uint32_t)(((uint64_t)1 << 32) / d); }
CSA_DEV int pg_div(int n, int d, uint32_t inv, int& rem) {
  uint32_t q = __umulhi((uint32_t)n, inv), r = (uint32_t)n - q * (uint32_t)d;
  if (r >= (uint32_t)d) {
    ++q;
    r -= (uint32_t)d;
  }
  rem = (int)r;
  return (int)q;
}
CSA_DEV int pg_div(int n, int d, uint32_t inv) {
  int r;
  return pg_div(n, d, inv, r);
}

// ------------------------------------------------------------- work items --
struct PgSeq {
  int n;        // new tokens
  int kv;       // cache length with them, >= 0
  int row0;     // first packed row
  int tiles;    // items of ROWS (token, head) rows
};
template <int ROWS>
CSA_DEV PgSeq pg_seq(const csa_paged_attn_args& a, int b) {
  PgSeq s;
  const int hi = (int)a.n_rows;
  s.row0 = min(max(a.kv.cu_q[b], 0), hi);
  s.n = min(max(a.kv.cu_q[b + 1], s.row0), hi) - s.row0;
  s.kv = max(a.kv.kv_len[b], 0);
  s.tiles = (int)(((int64_t)s.n * a.H + ROWS - 1) / ROWS);
  return s;
}
// Positions [k0, k1) that the rows of item j see (k1 = k0: none), before the
// rows' own masks.  Row r of the item is (token, head) row ROWS j + r.
template <int ROWS>
CSA_DEV void pg_item(const PgParams& p, const PgSeq& s, int j, int& k0, int& k1) {
  const csa_paged_attn_args& a = p.a;
  const int r0 = j * ROWS, r1 = min(r0 + ROWS, s.n * a.H) - 1;
  const int p0 = s.kv - s.n + pg_div(r0, a.H, p.h_inv), p1 = s.kv - s.n + pg_div(r1, a.H, p.h_inv);
  k1 = min(p1 + 1, a.kv.max_pages * a.kv.page_size);
  k0 = a.window ? max(0, p0 + 1 > a.window ? p0 + 1 - a.window : 0) : 0;
  if (k1 < k0) k1 = k0;
}
template <int ROWS>
CSA_DEV int pg_tiles(int k0, int k1) { return (k1 - k0 + kPgTile<ROWS> - 1) / kPgTile<ROWS>; }

// A part's walk over its items.  An item of T key tiles spans kPgItemCost + T
// of the cost axis; the part takes the tiles whose place lies in its range.
template <int ROWS>
struct PgWalk {
  int64_t left;    // cost left, from this item's start in the range on
  int b, j;        // sequence, item
  int at;          // where in the item the range starts
  PgSeq s;
  int k0, k1, total;   // the item's positions and key tiles
  int off, take;       // first key tile taken here, number taken
  bool fresh;          // opened, not yet gone to an item
  CSA_DEV void item(const PgParams& p) {
    pg_item<ROWS>(p, s, j, k0, k1);
    total = pg_tiles<ROWS>(k0, k1);
    off = min(max(at - kPgItemCost<ROWS>, 0), total);
    take = (int)min((int64_t)total, max(at + left - kPgItemCost<ROWS>, (int64_t)0)) - off;
  }
  // does this part do anything for the item? (a tileless one belongs to the
  // part at its start)
  CSA_DEV bool mine() const { return take > 0 || (total == 0 && at == 0); }
  CSA_DEV void step(const PgParams& p) {
    left -= kPgItemCost<ROWS> + total - at;
    at = 0;
    if (left <= 0) return;
    if (++j >= s.tiles) {
      j = 0;
#pragma unroll 1
      do {
        if (++b >= p.a.kv.B) { left = 0; return; }
        s = pg_seq<ROWS>(p.a, b);
      } while (s.tiles == 0);
    }
    item(p);
  }
  CSA_DEV void open(const PgParams& p, const int64_t* start) {
    at = (int)start[0];
    left = start[1];
    b = (int)start[2];
    j = (int)start[3];
    s.n = (int)start[4];
    s.kv = (int)start[5];
    s.row0 = (int)start[6];
    s.tiles = (int)start[7];
    fresh = true;
    if (left > 0) item(p);
  }
  // To the first and to the next item that has something for this part.
  CSA_DEV bool begin(const PgParams& p, const int64_t* start) {
    open(p, start);
#pragma unroll 1
    while (left > 0 && !mine()) step(p);
    return left > 0;
  }
  CSA_DEV bool next(const PgParams& p) {
    step(p);
#pragma unroll 1
    while (left > 0 && !mine()) step(p);
    return left > 0;
  }
  // Both in one, behind open(): a loop over it holds step()'s code once where
  // begin() and next() hold it three times, which counts where a kernel is over
  // before its instructions have all been fetched (one token: 18.9 -> 18.0 us).
  CSA_DEV bool go(const PgParams& p) {
    bool skip = !fresh;
    fresh = false;
#pragma unroll 1
    while (left > 0) {
      if (!skip && mine()) return true;
      step(p);
      skip = false;
    }
    return false;
  }
};

CSA_DEV int64_t pg_warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Cost of sequences 32 g + lane (0 past the last).  Sequences with many
// items are summed by the whole warp.
template <int ROWS>
CSA_DEV int64_t pg_group_cost(const PgParams& p, int g, int lane) {
  const csa_paged_attn_args& a = p.a;
  const int b = 32 * g + lane;
  PgSeq s{0, 0, 0, 0};
  if (b < a.kv.B) s = pg_seq<ROWS>(a, b);
  int64_t u = 0;
  if (s.tiles <= 4) {
#pragma unroll 1
    for (int j = 0; j < s.tiles; ++j) {
      int k0, k1;
      pg_item<ROWS>(p, s, j, k0, k1);
      u += kPgItemCost<ROWS> + pg_tiles<ROWS>(k0, k1);
    }
  }
#pragma unroll 1
  for (uint32_t big = __ballot_sync(0xffffffffu, s.tiles > 4); big; big &= big - 1) {
    const int l = __ffs(big) - 1;
    PgSeq q;
    q.n = __shfl_sync(0xffffffffu, s.n, l);
    q.kv = __shfl_sync(0xffffffffu, s.kv, l);
    q.row0 = 0;
    q.tiles = __shfl_sync(0xffffffffu, s.tiles, l);
    int64_t v = 0;
#pragma unroll 1
    for (int j = lane; j < q.tiles; j += 32) {
      int k0, k1;
      pg_item<ROWS>(p, q, j, k0, k1);
      v += kPgItemCost<ROWS> + pg_tiles<ROWS>(k0, k1);
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
// Finds the range of the cost axis of part `part` of `parts`; every warp of a
// CTA takes part (both CTAs of a pair find the same).  `gsum` holds a number
// per 32 sequences.
template <int ROWS>
CSA_DEV void pg_plan(const PgParams& p, int64_t* gsum, int64_t* start, int part, int parts, int warp, int warps, int lane) {
  const csa_paged_attn_args& a = p.a;
  const int groups = (a.kv.B + 31) / 32;
  if (groups > 1) {
#pragma unroll 1
    for (int g = warp; g < groups; g += warps) {
      const int64_t u = pg_warp_sum64(pg_group_cost<ROWS>(p, g, lane));
      if (lane == 0) gsum[g] = u;
    }
    __syncthreads();
  }
  if (warp == 0) {
    int64_t total = 0, only = 0;               // only: of the one group's sequences
    if (groups > 1) {
#pragma unroll 1
      for (int g = lane; g < groups; g += 32) total += gsum[g];
    } else {
      total = only = pg_group_cost<ROWS>(p, 0, lane);
    }
    total = pg_warp_sum64(total);
    const int64_t G = min((int64_t)parts, (total + 1) / 2);
    int64_t u0 = 0, u1 = 0;
    if (part < G) {
      u0 = total * part / G;
      u1 = total * (part + 1) / G;
    }
    int64_t at = u0;
    int b = 0, j = 0;
    PgSeq s{0, 0, 0, 0};
    if (u1 > u0) {
      int base = 0;
#pragma unroll 1
      for (; groups > 1; base += 32) {                     // the 32 groups
        const int64_t v = base + lane < groups ? gsum[base + lane] : 0;
        const int64_t sum = pg_warp_sum64(v);
        if (at < sum || base + 32 >= groups) {
          base += pg_locate(v, at, lane);
          break;
        }
        at -= sum;
      }
      const int64_t v = groups > 1 ? pg_group_cost<ROWS>(p, base, lane) : only;   // the sequence
      b = 32 * base + pg_locate(v, at, lane);
      s = pg_seq<ROWS>(a, b);
#pragma unroll 1
      for (;; j += 32) {                                   // the item
        int64_t w = 0;
        if (j + lane < s.tiles) {
          int k0, k1;
          pg_item<ROWS>(p, s, j + lane, k0, k1);
          w = kPgItemCost<ROWS> + pg_tiles<ROWS>(k0, k1);
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
      start[0] = at;
      start[1] = u1 - u0;
      start[2] = b;
      start[3] = j;
      start[4] = s.n;
      start[5] = s.kv;
      start[6] = s.row0;
      start[7] = s.tiles;
    }
  }
  __syncthreads();
}

// --------------------------------------------------------------- decoding --
CSA_DEV void pg_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
CSA_DEV uint4 pg_f16x8(const float (&f)[8]) {
  return make_uint4(pg_h2u(__floats2half2_rn(f[0], f[1])), pg_h2u(__floats2half2_rn(f[2], f[3])),
                    pg_h2u(__floats2half2_rn(f[4], f[5])), pg_h2u(__floats2half2_rn(f[6], f[7])));
}
// The conversion instructions run at the rate of the ALU here (2 cycles a warp
// and scheduler, as LOP3 or HMUL2), so they beat decoding by shifts and masks
// (two of them and a shift against seven for 4 FP8 codes).
// 8 FP8 codes times f (a power of two, twice).
CSA_DEV uint4 pg_decode_fp8(uint32_t w0, uint32_t w1, __half2 f) {
  return make_uint4(pg_h2u(__hmul2(dec_e4m3x2(w0), f)), pg_h2u(__hmul2(dec_e4m3x2(w0 >> 16), f)),
                    pg_h2u(__hmul2(dec_e4m3x2(w1), f)), pg_h2u(__hmul2(dec_e4m3x2(w1 >> 16), f)));
}
// 2^(byte - 127) twice in fp16 (0 for byte 0, whose block decodes to less than
// half of fp16's smallest value).
CSA_DEV __half2 pg_fp8_scale(uint32_t byte) {
  const float f = __uint_as_float(byte << 23);
  return __floats2half2_rn(f, f);
}
// Exponent bytes that pg_fp8_scale does not hold exactly: 1..102 and 143..255.
CSA_DEV bool pg_fp8_far(uint32_t bytes) {
  return (__vcmpgtu4(__vsub4(bytes, 0x67676767u), 0x27272727u) & ~__vcmpeq4(bytes, 0u)) != 0u;
}
// ... for those: fp32 products, rounded to fp16.
CSA_DEV uint4 pg_decode_fp8_far(uint32_t w0, uint32_t w1, uint32_t byte) {
  const float s = exp2f((float)((int)byte - 127));
  const float2 a = __half22float2(dec_e4m3x2(w0)), b = __half22float2(dec_e4m3x2(w0 >> 16));
  const float2 c = __half22float2(dec_e4m3x2(w1)), d = __half22float2(dec_e4m3x2(w1 >> 16));
  const float f[8] = {a.x * s, a.y * s, b.x * s, b.y * s, c.x * s, c.y * s, d.x * s, d.y * s};
  return pg_f16x8(f);
}
// One word of 8 FP4 codes times the block scale s (twice): at most 6
// significant bits between 2^-10 and 2688, exact in fp16.
CSA_DEV uint4 pg_decode_fp4(uint32_t w, __half2 s) {
  return make_uint4(pg_h2u(__hmul2(dec_e2m1x2(w & 0xFF), s)), pg_h2u(__hmul2(dec_e2m1x2((w >> 8) & 0xFF), s)),
                    pg_h2u(__hmul2(dec_e2m1x2((w >> 16) & 0xFF), s)), pg_h2u(__hmul2(dec_e2m1x2(w >> 24), s)));
}
// w[m] becomes w[m ^ q] (q in 0..3).
CSA_DEV void pg_rotate(uint4& v, int q) {
  if (q & 1) v = make_uint4(v.y, v.x, v.w, v.z);
  if (q & 2) v = make_uint4(v.z, v.w, v.x, v.y);
}
// 32 FP4 codes and the block scales of their halves (E4M3 codes in bytes 0 and
// 1 of `two`) as four 8-channel chunks, chunk m ^ q at place m.
CSA_DEV void pg_decode_fp4x32(uint4 v, uint32_t two, int q, uint4 (&c)[4]) {
  const __half2 s = dec_e4m3x2((q & 2) ? __byte_perm(two, 0, 0x4401) : two);
  const __half2 sa = __low2half2(s), sb = __high2half2(s);
  pg_rotate(v, q);
  c[0] = pg_decode_fp4(v.x, sa);
  c[1] = pg_decode_fp4(v.y, sa);
  c[2] = pg_decode_fp4(v.z, sb);
  c[3] = pg_decode_fp4(v.w, sb);
}

// Stages channels 256 g .. of an item's query rows r0 .. r0 + on - 1 (of the
// sequence's (token, head) rows, whose first token is packed row row0), padded
// to 64 with zeros, by the 4 warps of decode group g: channels below 384 into
// TMEM (twice: lanes L and L + 64 hold row L), the last 128 into two shared
// blocks of 64 rows (TWICE: of 128, the rows twice), all as fp16.  The rows
// come as they are, by asynchronous copies of whole rows (a row a lane would
// touch 32 lines an instruction), into 32 KB of the group's that are free.
// pg_fetch_q issues the copies, pg_stage_q waits for them; after a failed wait
// (`ok` false) the warps only keep their barriers.
struct PgRowsIn {
  int row0, r0, on;
};
CSA_DEV void pg_cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
CSA_DEV void pg_fetch_q(const PgParams& p, const PgRowsIn& R, uint8_t* buf, int wl, int lane, int g) {
  const csa_paged_attn_args& a = p.a;
  const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q) + 256 * g + 8 * lane;
  int head, tok = pg_div(R.r0 + 16 * wl, a.H, p.h_inv, head) + R.row0;
  // [64 rows][512 bytes], 16-byte chunk c of row r at c ^ (r & 31)
  const uint32_t at = smem_u32(buf) + 16 * wl * 512;
#pragma unroll 4
  for (int k = 0; k < 16; ++k) {                           // the warp's 16 rows
    const bool on = 16 * wl + k < R.on;
    pg_cp_async16(at + k * 512 + 16 * (lane ^ ((16 * wl + k) & 31)),
                  on ? qb + (int64_t)tok * a.q_row_stride + (int64_t)head * a.q_head_stride : qb, on);
    if (++head == a.H) {
      head = 0;
      ++tok;
    }
  }
  cp_async_commit();
}
template <bool TWICE>
CSA_DEV void pg_stage_q(const PgParams& p, const PgRowsIn& R, const uint8_t* buf, uint8_t* q, uint32_t tbase, int wl, int lane,
                        int g, bool ok) {
  constexpr int kBlk = (TWICE ? 128 : 64) * 128;
  const csa_paged_attn_args& a = p.a;
  cp_async_wait_all();
  named_bar(4 + g, 128);
  if (ok) {
    const int rr = (32 * wl + lane) & 63;
    const uint8_t* from = buf + rr * 512;
#pragma unroll 2
    for (int c = 0; c < (g ? 16 : 32); c += 4) {           // 16 columns
      uint32_t o[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
        pg_bf16x8(*reinterpret_cast<const uint4*>(from + 16 * ((c + k) ^ (rr & 31))), f);
        const uint4 h = pg_f16x8(f);
        o[4 * k] = h.x;
        o[4 * k + 1] = h.y;
        o[4 * k + 2] = h.z;
        o[4 * k + 3] = h.w;
      }
      tmem_st16(tbase + ((uint32_t)(32 * wl) << 16) + 128u * g + 4u * c, o);
    }
    if (g == 1) {
#pragma unroll 2
      for (int k = 0; k < 8; ++k) {                        // 8 rows x 16 chunks of the last 128 channels
        const int r = 8 * k + 2 * wl + (lane >> 4), c = lane & 15;
        float f[8];
        pg_bf16x8(*reinterpret_cast<const uint4*>(buf + r * 512 + 16 * ((16 + c) ^ (r & 31))), f);
        if (a.rope_cs && c >= 8 && r < R.on) {             // channels 448 + 8 (c - 8) ..
          const int tok = R.row0 + pg_div(R.r0 + r, a.H, p.h_inv);
          const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + (int64_t)tok * 64 + 8 * (c - 8));
          const float4 ca = cs[0], cb = cs[1];
          float2 x;
          x = rope_fwd(f[0], f[1], ca.x, ca.y); f[0] = x.x; f[1] = x.y;
          x = rope_fwd(f[2], f[3], ca.z, ca.w); f[2] = x.x; f[3] = x.y;
          x = rope_fwd(f[4], f[5], cb.x, cb.y); f[4] = x.x; f[5] = x.y;
          x = rope_fwd(f[6], f[7], cb.z, cb.w); f[6] = x.x; f[7] = x.y;
        }
        uint8_t* to = q + (c >> 3) * kBlk + sw128_offset_h(r, 8 * (c & 7));
        const uint4 h = pg_f16x8(f);
        *reinterpret_cast<uint4*>(to) = h;
        if (TWICE) *reinterpret_cast<uint4*>(to + 64 * 128) = h;
      }
    }
    tmem_wait_st();
    fence_proxy_async_smem();
    tc_fence_before();
  }
  named_bar(4 + g, 128);                                   // `buf` is read
}

// A position in the part's list of key tiles.
template <int ROWS>
struct PgCursor {
  PgWalk<ROWS> w;
  int i;           // tile of the item
  bool live;
  CSA_DEV void begin(const PgParams& p, const int64_t* start, int skip) {
    live = w.begin(p, start);
    i = 0;
    advance(p, skip);
  }
  CSA_DEV void advance(const PgParams& p, int n) {
    i += n;
#pragma unroll 1
    while (live && i >= w.take) {
      i -= w.take;
      live = w.next(p);
    }
  }
};

}  // namespace csa
