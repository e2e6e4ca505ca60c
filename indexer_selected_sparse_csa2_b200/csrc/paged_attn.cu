// MLA attention of packed chunks of new tokens over a paged latent cache
// (csa_paged_attn_args in csa.h): causal, optional sliding window, sink and
// partial RoPE, FP8 or FP4 entries, one token per sequence up to whole prompts.
//
// A work item is up to 128 query rows (token, head) of one sequence, rows in
// (token, head) order, so any head count fills the tile; it runs over the
// 64-entry key tiles its rows see.  A cluster of two CTAs works on an item,
// each CTA on half of its rows, with tcgen05.mma cta_group::2 over both.  Per
// key tile, with K = V = the decoded entries:
//   S = Q K^T   M = 128 rows (64 per CTA), N = 64 entries (32 per CTA), K = 512.
//               A CTA decodes its 32 entries, all channels.  Its 64 rows of Q
//               are the A operand in TMEM for channels 0..383 (the hardware
//               reads them from lanes L and L + 64 alike: staged twice), in
//               shared memory for the last 128.
//   O += P V    M = 128 rows, N = 2 x 256 channels (128 per CTA each), K = 64
//               entries.  A CTA holds 256 channels of all 64 entries; it decodes
//               those of the other CTA's 32 too.
// TMEM per CTA: lane L is row L mod 64; lanes 64.. hold the second half of S's
// 64 columns and of each block of 256 channels: O takes 256 columns, S 2 x 32,
// Q 192: all 512.
//
// Why two CTAs: shared memory bounds this attention.  With O (64 x 512) of one
// CTA alone, an entry's 1 KB is written once and read twice for 64 rows; the
// pair reads half of it per CTA for 128 rows.  Single CTAs (paged_attn_one.cu)
// take 3.42 ms where the pairs take 2.30: their MMAs need 148 KB of shared-
// memory reads and writes per 64 x 32 tile, 84 KB per 64 x 32 here.
//
// Warp roles: 0-3 softmax and output; 4-7 and 8-11 staging of Q, and loading
// and decoding of even and odd tiles; 12 issues the S MMAs, 13 the PV MMAs (of
// CTA 0 for both).  In flight: two K tiles, three V tiles, two S and two P.
// Four V tiles leave the loads in flight too little of L1 (2.59 ms for 2.29
// then), two are too few for a tile's way of 6000 cycles (3.74 ms).  A second
// softmax warpgroup left 96 registers a thread, and with shared memory at its
// maximum a spilled register is a trip to L2.
//
// Measured: 4 x 512 new tokens x 64 heads behind up to 16384 FP8 entries 2.02
// ms alone (1090 TFLOP/s), 2.28 ms back to back (963); 8 prompts of up to 2047
// tokens x 32 heads 637 / 678 us (719 / 675 TFLOP/s); 4 x 1024 tokens, window
// 128, 206 us (1.89 TB/s of queries, entries and output).  A tile of 128 x 64
// takes about 2050 cycles: the tensor pipe is busy for half of them, shared
// memory for two thirds, instruction issue for 56 %.
#include "paged_attn.cuh"

namespace csa {

constexpr int kPgRows = 128;              // query rows per item (two CTAs)
constexpr int kPgHalf = 64;               // ... per CTA
constexpr int kPgKBufs = 2, kPgVBufs = 3; // K and V tiles in flight
constexpr int kPgQBlk = kPgHalf * 128;    // shared Q block: 64 rows x 64 fp16
constexpr int kPgVBlk = kPgE * 128;       // 64-channel block of a V tile
constexpr int kPgVBytes = 4 * kPgVBlk;
constexpr int kPgPBytes = kPgHalf * kPgE * 2;
constexpr size_t kPgOperandBytes = 2 * kPgQBlk + kPgKBufs * kPgKBytes + kPgVBufs * kPgVBytes + 2 * kPgPBytes;
constexpr size_t kPgSmemBytes = kPgOperandBytes + 2048;   // and the small arrays
static_assert(kPgSmemBytes <= 232448, "shared memory of a CTA");
static_assert(kPgMaxB / 32 * 8 <= kPgVBufs * kPgVBytes, "the plan's group sums use the V tiles");

struct PgSmem {
  uint8_t* q;        // channels 384..511 of Q: 2 blocks
  uint8_t* k;        // [kPgKBufs] own 32 entries, 8 blocks of 64 channels
  uint8_t* v;        // [kPgVBufs] all 64 entries, this CTA's 4 blocks
  uint8_t* p;        // [2] P tiles
  float* mx;         // [2][2][64] tile maxima by tile parity and entry half
  float* lx;         // [2][64] sums by entry half
  uint32_t* valid;   // [kPgVBufs][2] entries present, by entry half
  int64_t* start;    // the pair's range: {its start inside its first item, length, sequence, item, PgSeq}
  uint64_t* bars;
  uint32_t* tmem_base;
  volatile uint32_t* begun;   // items with tiles whose queries the decode warps have turned to
};

CSA_DEV PgSmem carve_pg(uint8_t* p) {
  PgSmem s;
  s.q = p; p += 2 * kPgQBlk;
  s.k = p; p += kPgKBufs * kPgKBytes;
  s.v = p; p += kPgVBufs * kPgVBytes;
  s.p = p; p += 2 * kPgPBytes;
  s.mx = reinterpret_cast<float*>(p); p += 4 * 64 * 4;
  s.lx = reinterpret_cast<float*>(p); p += 2 * 64 * 4;
  s.bars = reinterpret_cast<uint64_t*>(p); p += 24 * 8;
  s.start = reinterpret_cast<int64_t*>(p); p += 8 * 8;
  s.valid = reinterpret_cast<uint32_t*>(p); p += 2 * kPgVBufs * 4;
  s.tmem_base = reinterpret_cast<uint32_t*>(p); p += 4;
  s.begun = reinterpret_cast<uint32_t*>(p);
  return s;
}

// ------------------------------------------------- barriers across the pair --
// Arrival on CTA 0's barrier (`bar` is its address in the cluster's window).
// What it publishes lies in the arriving CTA's own shared memory or TMEM,
// where the pair's MMAs read it on the same SM.
CSA_DEV void pg_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrival on both CTAs' barriers once every MMA issued so far completes.
CSA_DEV void pg_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
CSA_DEV void pg_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n}"
      ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kPgDesc), "r"(acc) : "memory");
}
CSA_DEV void pg_mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n}"
      ::"r"(d), "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kPgDesc), "r"(acc) : "memory");
}
// Instruction descriptor with B MN-major (bit 16).
constexpr uint32_t kPgIdescS = (1u << 4) | ((uint32_t)(kPgE >> 3) << 17) | ((uint32_t)(kPgRows >> 4) << 24);
constexpr uint32_t kPgIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(256 >> 3) << 17) | ((uint32_t)(kPgRows >> 4) << 24);

// The rows of an item that CTA `rank` works on: its `per` rows from rank * per
// on, `per` a half of the item's rows rounded up, so a short item's output is
// shared out too.
struct PgRowsOf {
  int base, on;      // first row in the item, rows
  CSA_DEV PgRowsOf(const csa_paged_attn_args& a, const PgWalk<kPgRows>& w, uint32_t rank) {
    const int n = min(w.s.n * a.H - w.j * kPgRows, kPgRows), per = (n + 1) >> 1;
    base = (int)rank * per;
    on = min(per, n - base);
  }
};

template <bool FP4>
__global__ void __launch_bounds__(kPgThreads, 1) paged_attn_kernel(const __grid_constant__ PgParams p) {
  constexpr int kScaleOff = FP4 ? 256 : 512;
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const PgSmem S = carve_pg(smem_raw);
  // Waited on in CTA 0, whose warps issue for both; arrivals from both CTAs:
  uint64_t* k_full = S.bars + 0;     // [kPgKBufs] K tile decoded (8 warp arrivals)
  uint64_t* v_full = S.bars + 2;     // [kPgVBufs] V tile decoded (8)
  uint64_t* s_free = S.bars + 6;     // [2] S read by the softmax (8)
  uint64_t* p_full = S.bars + 8;     // [2] P written, O rescaled (8)
  uint64_t* q_full = S.bars + 10;    // an item's Q staged (16)
  // In both CTAs, by commits:
  uint64_t* k_free = S.bars + 11;    // [kPgKBufs] S done: K tile reusable
  uint64_t* v_free = S.bars + 13;    // [kPgVBufs] PV done: V tile (and P tile) reusable
  uint64_t* s_full = S.bars + 17;    // [2] S in TMEM
  uint64_t* q_free = S.bars + 19;    // an item's last S done
  uint64_t* acc_done = S.bars + 20;  // an item's last PV done
  uint64_t* drain = S.bars + 21;     // [2] all MMAs of an issuer retired (teardown)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const csa_paged_attn_args& a = p.a;
  if (tid == 0) {
    for (int k = 0; k < kPgVBufs; ++k) {
      mbar_init(v_full + k, 8);
      mbar_init(v_free + k, 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(k_full + k, 8);
      mbar_init(k_free + k, 1);
      mbar_init(s_full + k, 1);
      mbar_init(s_free + k, 8);
      mbar_init(p_full + k, 8);
      mbar_init(drain + k, 1);
    }
    mbar_init(q_full, 16);
    mbar_init(q_free, 1);
    mbar_init(acc_done, 1);
    fence_mbar_init();
    *S.begun = 1;
  }
  if (warp == kPgWarpS) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(S.tmem_base)), "r"(kPgTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pg_plan<kPgRows>(p, reinterpret_cast<int64_t*>(S.v), S.start, pair, pairs, warp, kPgWarps, lane);
  tc_fence_before();
  cluster_sync_all();                // barriers and TMEM of both CTAs are there
  tc_fence_after();
  const uint32_t tbase = *S.tmem_base;

  if (warp == kPgWarpS) {
    // ------------------------------------------------------------ S issuer
    if (rank == 0) {
      const uint32_t qd = pg_desc_k(smem_u32(S.q)), kd0 = pg_desc_k(smem_u32(S.k));
      PgWalk<kPgRows> w;
      uint32_t t = 0, seg = 0;
      bool ok = true;
      for (bool go = w.begin(p, S.start); go && ok; go = w.next(p)) {
        if (w.take == 0) continue;
        ok = pg_wait_warp(q_full, seg++ & 1u, kErrWaitTmaFull);
        for (int i = 0; i < w.take && ok; ++i, ++t) {
          const uint32_t si = t & 1u;
          if (t >= 2) ok = pg_wait_warp(s_free + si, ((t >> 1) - 1) & 1u, kErrWaitAccEmpty);
          ok = ok && pg_wait_warp(k_full + t % kPgKBufs, (t / kPgKBufs) & 1u, kErrWaitTmaFull);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kd = kd0 + (t % kPgKBufs) * (kPgKBytes >> 4), sd = tbase + kPgSCol + 32 * si;
          if (pg_elect()) {
            // rolled by 64-channel blocks: unrolled, 5 KB of instructions
            // missed the cache once a tile
            uint32_t bd = kd;
#pragma unroll 1
            for (uint32_t kb = 0; kb < (uint32_t)kPgQTmemBlocks; ++kb, bd += kPgKBlk >> 4) {
#pragma unroll
              for (uint32_t sub = 0; sub < 4; ++sub) pg_mma_ts(sd, tbase + kb * 32 + sub * 8, bd + sub * 2, kPgIdescS, kb | sub);
            }
#pragma unroll 1
            for (uint32_t kb = 0; kb < 8u - kPgQTmemBlocks; ++kb, bd += kPgKBlk >> 4) {
#pragma unroll
              for (uint32_t sub = 0; sub < 4; ++sub) pg_mma_ss(sd, qd + kb * (kPgQBlk >> 4) + sub * 2, bd + sub * 2, kPgIdescS, 1);
            }
            pg_commit(s_full + si);
            pg_commit(k_free + t % kPgKBufs);
            if (i == w.take - 1) pg_commit(q_free);
          }
          __syncwarp();
        }
      }
      if (pg_elect()) pg_commit(drain);
      __syncwarp();
    }
  } else if (warp == kPgWarpPV) {
    // ----------------------------------------------------------- PV issuer
    if (rank == 0) {
      const uint32_t vd0 = pg_desc_mn(smem_u32(S.v), kPgVBlk), pd0 = pg_desc_k(smem_u32(S.p));
      PgWalk<kPgRows> w;
      uint32_t t = 0;
      bool ok = true;
      for (bool go = w.begin(p, S.start); go && ok; go = w.next(p)) {
        for (int i = 0; i < w.take; ++i, ++t) {
          ok = pg_wait_warp(v_full + t % kPgVBufs, (t / kPgVBufs) & 1u, kErrWaitTmaFull);
          ok = ok && pg_wait_warp(p_full + (t & 1u), (t >> 1) & 1u, kErrWaitAccFull);
          if (!ok) break;
          tc_fence_after();
          const uint32_t vd = vd0 + (t % kPgVBufs) * (kPgVBytes >> 4), pd = pd0 + (t & 1u) * (kPgPBytes >> 4);
          if (pg_elect()) {
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
              for (int ks = 0; ks < kPgE / 16; ++ks) {
                const uint32_t bd = vd + 2 * nb * (kPgVBlk >> 4) + ks * (2048 >> 4), ad = pd + ks * 2;
                pg_mma_ss(tbase + kPgOCol + 128u * nb, ad, bd, kPgIdescO, ks | i);
              }
            }
            pg_commit(v_free + t % kPgVBufs);
            if (i == w.take - 1) pg_commit(acc_done);
          }
          __syncwarp();
        }
      }
      if (pg_elect()) pg_commit(drain + 1);
      __syncwarp();
    } else {
      // CTA 1's warp fetches an item's query rows, of both CTAs, into L2 once
      // the decode warps have turned to the item before.  It follows a count,
      // not a barrier's phase: nobody waits for this warp, so it may fall any
      // number of items behind; and a wait that gives up (an item may take as
      // long) ends the prefetching, not the result.
      PgWalk<kPgRows> w;
      uint32_t items = 0;                // with tiles, up to this one
      bool ok = true;
      for (bool go = w.begin(p, S.start); go && ok; go = w.next(p)) {
        if (w.take == 0) continue;
        if (items > 0) ok = pg_wait_count(S.begun, items);
        if (items++ > 0 && ok) {
          const int n = min(w.s.n * a.H - w.j * kPgRows, kPgRows);
          for (int l = lane; l < 8 * n; l += 32) {         // 128 bytes each
            int head;
            const int tok = pg_div(w.j * kPgRows + (l >> 3), a.H, p.h_inv, head);
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(w.s.row0 + tok) * a.q_row_stride +
                                     (int64_t)head * a.q_head_stride + 64 * (l & 7);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          }
        }
      }
    }
  } else if (warp >= kPgWarpDec) {
    // ---------------------------------------------- entry loads and decoding
    // Group g (4 warps) takes the pair's tiles of parity g.  A warp decodes 8
    // of this CTA's 32 entries, all channels, into K and (this CTA's 256
    // channels) V, and 8 of the other CTA's entries, those 256 channels, into
    // V.  (One CTA decoding for both, through distributed shared memory, spent
    // 3000 cycles a tile in the fence behind its remote stores.)
    const int wq = (warp - kPgWarpDec) & 3, g = (warp - kPgWarpDec) >> 2;
    // the first item's query rows come first: their way is the longest
    PgWalk<kPgRows> w;
    bool go = w.begin(p, S.start);
    while (go && w.take == 0) go = w.next(p);
    auto rows = [&]() {
      const PgRowsOf R(a, w, rank);
      return PgRowsIn{w.s.row0, w.j * kPgRows + R.base, R.on};
    };
    uint8_t* q_buf = S.k + g * kPgKBytes;                  // free between an item's last S and the next one's first tile
    if (go) pg_fetch_q(p, rows(), q_buf, wq, lane, g);
    PgCursor<kPgRows> cu;                       // the tile whose page table values are fetched next
    cu.begin(p, S.start, g);
    // page id and entry number in the page of entry 8 wq + (lane & 7), lanes
    // 8-15 (24-31) of the other CTA's half, of the tile whose entries are
    // loaded next
    const int e_at = kPgOwn * (int)(rank ^ (uint32_t)((lane >> 3) & 1)) + 8 * wq + (lane & 7);
    int id = -1;
    uint32_t slot = 0;
    auto lookup = [&]() {
      id = -1;
      if (cu.live) {
        const int pos = cu.w.k0 + (cu.w.off + cu.i) * kPgE + e_at;
        if (pos < cu.w.k1) {
          int rem;
          const int pg = pg_div(pos, a.kv.page_size, p.page_inv, rem);
          slot = (uint32_t)rem;
          id = a.kv.block_table[(int64_t)cu.w.b * a.kv.table_stride + pg];
        }
      }
    };
    // 16-byte words per lane and tile: kN of the own entries, kN / 2 of the
    // others
    constexpr int kN = FP4 ? 4 : 8;
    uint4 r[kN], x[kN / 2];
    uint2 sc, scx;
    uint32_t vb;                       // valid entries: 8 own, 8 of the other half
    auto at_lane = [&](unsigned long long ptr, int l) {
      return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, ptr, l));
    };
    // own entries.  FP8: word k is bytes [16 lane, ..) of entry k; FP4: bytes
    // [16 (lane & 15), ..) of entry 2k + (lane >> 4).  kb: the 64-channel block
    const int kb = FP4 ? (lane & 15) >> 1 : lane >> 2;
    // the other half's.  FP8: entry 2k + (lane >> 4), piece lane & 15 of 16
    // channels; FP4: entry 4k + (lane >> 3), piece lane & 7 of 32.  xb: the V
    // block, of channels 64 xc ..
    const int xb = FP4 ? (lane & 7) >> 1 : (lane & 15) >> 2;
    const int xc = (xb >> 1) * 4 + 2 * (int)rank + (xb & 1);
    const int x_off = FP4 ? 32 * xc + 16 * (lane & 1) : 64 * xc + 16 * (lane & 3);
    // All loads of a tile.  Where there is no entry, the cache's first one is
    // read instead, and the decoder writes zeros.
    auto load_tile = [&]() {
      const bool on = id >= 0 && id < a.kv.n_pages;
      vb = __ballot_sync(0xffffffffu, on) & 0xFFFFu;
      const unsigned long long ptr =
          (unsigned long long)(a.kv.pages + (on ? (int64_t)id * a.kv.page_stride + (int64_t)slot * a.kv.row_stride : 0));
      const uint8_t *q0, *q1;          // the entries whose scales this lane loads
      const int id0 = __shfl_sync(0xffffffffu, id, lane & 8);
      if (__all_sync(0xffffffffu, on && id == id0)) {
        // the usual case: a warp's 8 entries of either half lie in one page,
        // so their addresses need no exchange (a load behind each pair of
        // shuffles made these 14 loads take 2000 cycles)
        const int64_t rs = a.kv.row_stride;
        const uint8_t *p0 = at_lane(ptr, 0), *p1 = at_lane(ptr, 8);
        q0 = p0 + (lane >> 2) * rs;
        q1 = p1 + (lane >> 2) * rs;
        const uint8_t* o = p0 + (FP4 ? (lane >> 4) * rs + 16 * (lane & 15) : 16 * lane);
#pragma unroll
        for (int k = 0; k < kN; ++k, o += (FP4 ? 2 : 1) * rs) r[k] = pg_ld_entry<true>(o);
        o = p1 + (FP4 ? lane >> 3 : lane >> 4) * rs + x_off;
#pragma unroll
        for (int k = 0; k < kN / 2; ++k, o += (FP4 ? 4 : 2) * rs) x[k] = pg_ld_entry<true>(o);
      } else {
#pragma unroll
        for (int k = 0; k < kN; ++k)
          r[k] = pg_ld_entry<true>(at_lane(ptr, FP4 ? 2 * k + (lane >> 4) : k) + 16 * (FP4 ? lane & 15 : lane));
#pragma unroll
        for (int k = 0; k < kN / 2; ++k) x[k] = pg_ld_entry<true>(at_lane(ptr, 8 + (FP4 ? 4 * k + (lane >> 3) : 2 * k + (lane >> 4))) + x_off);
        q0 = at_lane(ptr, lane >> 2);
        q1 = at_lane(ptr, 8 + (lane >> 2));
      }
      // scales: lane 4e + w holds word w of entry e's scale bytes
      if (FP4) {
        sc = *reinterpret_cast<const uint2*>(q0 + kScaleOff + 8 * (lane & 3));
        scx = *reinterpret_cast<const uint2*>(q1 + kScaleOff + 8 * (lane & 3));
      } else {
        sc.x = *reinterpret_cast<const uint32_t*>(q0 + kScaleOff + 4 * (lane & 3));
        scx.x = *reinterpret_cast<const uint32_t*>(q1 + kScaleOff + 4 * (lane & 3));
      }
    };
    lookup();
    load_tile();
    cu.advance(p, 2);
    lookup();
    const bool v_own = (uint32_t)((kb >> 1) & 1) == rank;   // block kb belongs to this CTA's V
    const uint32_t k_at = smem_u32(S.k) + (uint32_t)kb * kPgKBlk;
    const uint32_t v_at = smem_u32(S.v) + (uint32_t)((kb >> 2) * 2 + (kb & 1)) * kPgVBlk + kPgOwn * 128 * rank;
    const uint32_t x_at = smem_u32(S.v) + (uint32_t)xb * kPgVBlk + kPgOwn * 128 * (rank ^ 1u);
    const uint32_t k_full_at = dsmem(k_full, 0), v_full_at = dsmem(v_full, 0), q_full_at = dsmem(q_full, 0);
    auto st16 = [](uint32_t at, const uint4& q) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
    };
    uint32_t t0 = 0, seg = 0;          // tiles before the item, items with tiles before it
    bool ok = true;
    // a failed wait leaves `ok` false and skips the later waits and all work;
    // every warp still passes its group's barriers once per item
    for (; go; go = w.next(p)) {
      if (w.take == 0) continue;
      const PgRowsIn R = rows();
      if (seg > 0) {
        ok = ok && pg_wait_warp(q_free, (seg - 1) & 1u, kErrWaitSmemEmpty);
        if (tid == 32 * kPgWarpDec) *S.begun = seg + 1;
        if (ok) pg_fetch_q(p, R, q_buf, wq, lane, g);
      }
      tc_fence_after();
      pg_stage_q<false>(p, R, q_buf, S.q, tbase, wq, lane, g, ok);
      if (ok && lane == 0) pg_arrive(q_full_at);
      ++seg;
      uint32_t t = t0 + ((t0 ^ (uint32_t)g) & 1u);
      t0 += (uint32_t)w.take;
      for (; t < t0; t += 2) {
        const uint32_t vi = t % kPgVBufs;
        if (ok && t >= kPgKBufs) ok = pg_wait_warp(k_free + t % kPgKBufs, (t / kPgKBufs - 1) & 1u, kErrWaitSmemEmpty);
        if (ok && t >= kPgVBufs) ok = pg_wait_warp(v_free + vi, (t / kPgVBufs - 1) & 1u, kErrWaitSmemEmpty);
        if (!ok) continue;
        const uint32_t kt = k_at + (t % kPgKBufs) * kPgKBytes, vt = v_at + vi * kPgVBytes, xt = x_at + vi * kPgVBytes;
        auto put = [&](int row, int c, const uint4& q) {    // 8 channels of an own entry
          const uint32_t o = sw128_offset_h(row, c);
          st16(kt + o, q);
          if (v_own) st16(vt + o, q);
        };
        // K is announced before the other half's V is decoded: S can start.
        auto announce = [&](uint32_t bar) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) pg_arrive(bar);
        };
        if (lane < 2) reinterpret_cast<uint8_t*>(S.valid)[8 * vi + 4 * (rank ^ (uint32_t)lane) + wq] = (uint8_t)(vb >> (8 * lane));
        // Stores go in an order by block, so that 8 lanes' stores meet 8
        // different 16-byte columns.
        if (FP4) {
          const int l16 = lane & 15;
#pragma unroll
          for (int k = 0; k < kN; ++k) {
            const int e = 2 * k + (lane >> 4);
            const uint32_t sx = __shfl_sync(0xffffffffu, sc.x, 4 * e + (l16 >> 2));
            const uint32_t sy = __shfl_sync(0xffffffffu, sc.y, 4 * e + (l16 >> 2));
            uint32_t two = ((l16 & 2) ? sy : sx) >> (16 * (l16 & 1));
            if (!((vb >> e) & 1u)) two = 0;                  // no entry: zeros
            uint4 c[4];
            pg_decode_fp4x32(r[k], two, kb & 3, c);
#pragma unroll
            for (int m = 0; m < 4; ++m) put(8 * wq + e, 32 * (l16 & 1) + 8 * (m ^ (kb & 3)), c[m]);
          }
          announce(k_full_at + 8 * (t % kPgKBufs));
#pragma unroll
          for (int k = 0; k < kN / 2; ++k) {
            // this lane's 32 channels: scale bytes 4 xc + 2 (lane & 1), + 1
            const int e = 4 * k + (lane >> 3);
            const uint32_t sx = __shfl_sync(0xffffffffu, scx.x, 4 * e + (xc >> 1));
            const uint32_t sy = __shfl_sync(0xffffffffu, scx.y, 4 * e + (xc >> 1));
            uint32_t two = ((xc & 1) ? sy : sx) >> (16 * (lane & 1));
            if (!((vb >> (8 + e)) & 1u)) two = 0;
            uint4 c[4];
            pg_decode_fp4x32(x[k], two, xb, c);
#pragma unroll
            for (int m = 0; m < 4; ++m) st16(xt + sw128_offset_h(8 * wq + e, 32 * (lane & 1) + 8 * (m ^ xb)), c[m]);
          }
        } else {
          const int f = kb & 1, fx = xb & 1;
          if (vb != 0xFFFFu) {                               // no entry: zeros
#pragma unroll
            for (int k = 0; k < kN; ++k)
              if (!((vb >> k) & 1u)) r[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < kN / 2; ++k)
              if (!((vb >> (8 + 2 * k + (lane >> 4))) & 1u)) x[k] = make_uint4(0, 0, 0, 0);
            if (!((vb >> (lane >> 2)) & 1u)) sc.x = 0;
            if (!((vb >> (8 + (lane >> 2))) & 1u)) scx.x = 0;
          }
          const int xs = xc >> 1, xsh = 8 * (2 * (xc & 1) + ((lane >> 1) & 1));   // word and byte of the piece's block
          const bool far = __any_sync(0xffffffffu, pg_fp8_far(sc.x) || pg_fp8_far(scx.x));
          if (!far) {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
              const __half2 m = pg_fp8_scale((__shfl_sync(0xffffffffu, sc.x, 4 * k + (lane >> 3)) >> (8 * ((lane >> 1) & 3))) & 0xFFu);
              if (f) r[k] = make_uint4(r[k].z, r[k].w, r[k].x, r[k].y);
              put(8 * wq + k, 16 * (lane & 3) + 8 * f, pg_decode_fp8(r[k].x, r[k].y, m));
              put(8 * wq + k, 16 * (lane & 3) + 8 * (f ^ 1), pg_decode_fp8(r[k].z, r[k].w, m));
            }
            announce(k_full_at + 8 * (t % kPgKBufs));
#pragma unroll
            for (int k = 0; k < kN / 2; ++k) {
              const int e = 2 * k + (lane >> 4);
              const __half2 m = pg_fp8_scale((__shfl_sync(0xffffffffu, scx.x, 4 * e + xs) >> xsh) & 0xFFu);
              if (fx) x[k] = make_uint4(x[k].z, x[k].w, x[k].x, x[k].y);
              st16(xt + sw128_offset_h(8 * wq + e, 16 * (lane & 3) + 8 * fx), pg_decode_fp8(x[k].x, x[k].y, m));
              st16(xt + sw128_offset_h(8 * wq + e, 16 * (lane & 3) + 8 * (fx ^ 1)), pg_decode_fp8(x[k].z, x[k].w, m));
            }
          } else {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
              const uint32_t m = (__shfl_sync(0xffffffffu, sc.x, 4 * k + (lane >> 3)) >> (8 * ((lane >> 1) & 3))) & 0xFFu;
              put(8 * wq + k, 16 * (lane & 3), pg_decode_fp8_far(r[k].x, r[k].y, m));
              put(8 * wq + k, 16 * (lane & 3) + 8, pg_decode_fp8_far(r[k].z, r[k].w, m));
            }
            announce(k_full_at + 8 * (t % kPgKBufs));
#pragma unroll
            for (int k = 0; k < kN / 2; ++k) {
              const int e = 2 * k + (lane >> 4);
              const uint32_t m = (__shfl_sync(0xffffffffu, scx.x, 4 * e + xs) >> xsh) & 0xFFu;
              st16(xt + sw128_offset_h(8 * wq + e, 16 * (lane & 3)), pg_decode_fp8_far(x[k].x, x[k].y, m));
              st16(xt + sw128_offset_h(8 * wq + e, 16 * (lane & 3) + 8), pg_decode_fp8_far(x[k].z, x[k].w, m));
            }
          }
        }
        announce(v_full_at + 8 * vi);
        // the next tile's entries, all loads together (issued one by one
        // between the decodes, each decode waits for the load before it: loads
        // share their scoreboards), then the table values of the tile after it
        load_tile();
        cu.advance(p, 2);
        lookup();
      }
    }
  } else {
    // ------------------------------------------------------ softmax, output
    const int q4 = warp, rr = 32 * (q4 & 1) + lane;          // TMEM lane quarter, row of this CTA
    const int half = q4 >> 1;                                // entries 32 half .. of a tile; channel half of a block
    const uint32_t trow = tbase + ((uint32_t)(32 * q4) << 16);
    const uint32_t s_free_at = dsmem(s_free, 0), p_full_at = dsmem(p_full, 0);
    PgWalk<kPgRows> w;
    uint32_t t = 0, seg = 0;
    bool ok = true;
    int64_t meta_row0 = 0;
    int meta_rows = 0, meta_cont = 0, meta_done = 0;
    for (bool go = w.begin(p, S.start); go; go = w.next(p)) {
      const int nt = w.take;
      const PgRowsOf R(a, w, rank);
      const int ri = w.j * kPgRows + R.base + rr;
      // positions this row sees: (lo, hi]; none for rows past the item's
      int head;
      const int tok = pg_div(ri, a.H, p.h_inv, head);
      const int hi = rr < R.on ? w.s.kv - w.s.n + tok : -1;
      const int lo = a.window && hi >= a.window ? hi - a.window : -1;
      float m_run = -INFINITY, l_run = 0.f;    // l_run: this lane's entry half
      for (int i = 0; i < nt; ++i, ++t) {
        const uint32_t si = t & 1u;
        const int kb = w.k0 + (w.off + i) * kPgE + 32 * half;
        const int nh = hi - kb + 1, nl = lo - kb + 1;        // the row sees entries [nl, nh) of this half
        uint32_t mask = nh >= 32 ? 0xffffffffu : nh <= 0 ? 0u : (1u << nh) - 1u;
        mask &= nl <= 0 ? 0xffffffffu : nl >= 32 ? 0u : ~((1u << nl) - 1u);
        // a failed wait leaves `ok` false and skips the later waits; every
        // warp still passes the group's barriers once per tile
        ok = ok && pg_wait_warp(s_full + si, (t >> 1) & 1u, kErrWaitAccFull);
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld32(trow + kPgSCol + 32 * si, sv);
        mask &= S.valid[2 * (t % kPgVBufs) + half];          // written before the tile's S was issued
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pg_arrive(s_free_at + 8 * si);
        // rounded before anything is subtracted (pg_mul32)
        pg_mul32(sv, p.scale_log2);
        if (!__all_sync(0xffffffffu, mask == 0xffffffffu)) {
#pragma unroll
          for (int k = 0; k < 32; ++k) sv[k] = ((mask >> k) & 1u) ? sv[k] : 0xff800000u;   // -inf
        }
        float m4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(__uint_as_float(sv[k]), __uint_as_float(sv[k + 4]));
#pragma unroll
        for (int k = 8; k < 32; ++k) m4[k & 3] = fmaxf(m4[k & 3], __uint_as_float(sv[k]));
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        S.mx[(2 * si + half) * 64 + rr] = mt;
        uint32_t over;
        // a row's two halves are lanes of warps w and w + 2: they meet here
        asm volatile("{\n .reg .pred q, r;\n setp.ne.u32 q, %2, 0;\n bar.red.or.pred r, %1, 64, q;\n selp.u32 %0, 1, 0, r;\n}"
                     : "=r"(over) : "r"(1 + (q4 & 1)), "r"(mt - m_run >= kPgRescale ? 1u : 0u) : "memory");
        if (over) {
          const float mm = fmaxf(mt, S.mx[(2 * si + (half ^ 1)) * 64 + rr]);
          float alpha = 1.f;
          if (mm - m_run >= kPgRescale) {
            alpha = m_run == -INFINITY ? 0.f : pg_ex2(m_run - mm);
            m_run = mm;
            l_run *= alpha;
          }
          if (i > 0) {
            // O of this lane's row, once the PV before this tile's has retired
            ok = ok && pg_wait_warp(v_free + (t - 1) % kPgVBufs, ((t - 1) / kPgVBufs) & 1u, kErrWaitAccFull);
            tc_fence_after();
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < 256; c += 32) {
                uint32_t o[32];
                tmem_ld32(trow + kPgOCol + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st16(trow + kPgOCol + c, *reinterpret_cast<uint32_t(*)[16]>(o));
                tmem_st16(trow + kPgOCol + c + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
              }
              tmem_wait_st();
            }
          }
        }
        // the P tile is free once the PV two tiles back has retired
        if (t >= 2) ok = ok && pg_wait_warp(v_free + (t - 2) % kPgVBufs, ((t - 2) / kPgVBufs) & 1u, kErrWaitSmemEmpty);
        // a row that has seen nothing yet: every logit here is -inf, and so is
        // its max; any finite reference gives the zeros it needs
        pg_add32(sv, m_run == -INFINITY ? 0.f : kPgPExp - m_run);
        float l0 = 0.f, l1 = 0.f;
        uint8_t* pt = S.p + si * kPgPBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e0 = 8 * c + 2 * k;
            const float x0 = pg_ex2(__uint_as_float(sv[e0]));
            const float x1 = pg_ex2(__uint_as_float(sv[e0 + 1]));
            l0 += x0;
            l1 += x1;
            o[k] = pg_h2u(__floats2half2_rn(x0, x1));
          }
          *reinterpret_cast<uint4*>(pt + sw128_offset_h(rr, 32 * half + 8 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        l_run += l0 + l1;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pg_arrive(p_full_at + 8 * si);
      }
      // ------------------------------------------------------------ output
      const bool whole = w.take == w.total;
      S.lx[half * 64 + rr] = l_run;
      named_bar(1 + (q4 & 1), 64);
      const float l = S.lx[rr] + S.lx[64 + rr];
      const int64_t orow = (int64_t)w.s.row0 * a.H + w.j * kPgRows + R.base;
      const int slot = 2 * pair + (w.off > 0 ? 0 : 1);
      float scl = 0.f;
      if (whole) {
        const float m0 = m_run - kPgPExp;
        float M = m0, L = l;
        if (a.sink) {
          const float s0 = rr < R.on ? a.sink[head] * kPgLog2e : -INFINITY;
          M = fmaxf(m0, s0);
          const float f = l > 0.f ? exp2f(m0 - M) : 0.f;
          L = l * f + (s0 == -INFINITY ? 0.f : exp2f(s0 - M));
          scl = l > 0.f ? f / L : 0.f;
        } else {
          scl = l > 0.f ? 1.f / l : 0.f;
        }
        if (warp < 2 && a.lse && rr < R.on) a.lse[orow + rr] = L > 0.f ? (M + log2f(L)) * kPgLn2 : -INFINITY;
      } else if (warp < 2 && rr < R.on) {
        p.part_ml[slot * kPgRows + R.base + rr] = make_float2(m_run, l);
      }
      named_bar(1 + (q4 & 1), 64);            // lx read
      // every PV of the item
      if (nt > 0) ok = ok && pg_wait_warp(acc_done, seg++ & 1u, kErrWaitAccFull);
      tc_fence_after();
      // this lane's row, channels 128 half .. + 127 of each 256
      const bool valid_o = nt > 0 && ok;
      const float2* cs = nullptr;
      if (whole && a.rope_cs && half == 1 && rr < R.on)
        cs = reinterpret_cast<const float2*>(a.rope_cs + (int64_t)(w.s.row0 + tok) * 64);
      // A lane's row goes through 128 bytes of the (free) P tiles, so that a
      // store instruction writes whole lines of four rows instead of a piece
      // of each of 32.  The warp's 4 KB are touched again by other warps' P
      // only behind the next tile's meeting of the row's two warps.
      uint8_t* st = S.p + half * kPgPBytes + (q4 & 1) * 4096;
      uint8_t* st_row = st + lane * 128;
      const int8_t sw = (int8_t)(lane & 7);
      const int rl = lane >> 3, cl = lane & 7;               // row of four, 16-byte chunk
      const uint8_t* ld_row = st + rl * 128;
      const int step = whole ? 64 : 32;                      // columns a pass: 128 bytes of bf16 or fp32
      uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(a.out) + orow * kD)
                           : reinterpret_cast<uint8_t*>(p.part_o + ((int64_t)slot * kPgRows + R.base) * kD);
      const int64_t row_bytes = whole ? kD * 2 : kD * 4;
      dst += (32 * (q4 & 1) + rl) * row_bytes + 16 * cl;
      const int rows_on = R.on - 32 * (q4 & 1) - rl;
#pragma unroll 1
      for (int c = 0; c < 256; c += step) {
        const int ch = c + 128 * half + (c < 128 ? 0 : 128); // first channel
        if (whole) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            if (valid_o) {
              tmem_ld32(trow + kPgOCol + c + 32 * h, o);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0u;
            }
            if (cs && c == 192) {                            // channels 448 + 32 h ..
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 z = cs[16 * h + k], f = rope_inv(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]), z.x, z.y);
                o[2 * k] = __float_as_uint(f.x);
                o[2 * k + 1] = __float_as_uint(f.y);
              }
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[2 * k]) * scl, __uint_as_float(o[2 * k + 1]) * scl);
              o[k] = *reinterpret_cast<const uint32_t*>(&b2);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(st_row + 16 * ((4 * h + k) ^ sw)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        } else {
          uint32_t o[32];
          if (valid_o) {
            tmem_ld32(trow + kPgOCol + c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(st_row + 16 * (k ^ sw)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        __syncwarp();
        uint8_t* to = dst + (int64_t)ch * (whole ? 2 : 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {                        // rows 4 k + rl of the warp's 32
          const uint4 v = *reinterpret_cast<const uint4*>(ld_row + 512 * k + 16 * (cl ^ ((4 * k + rl) & 7)));
          if (4 * k < rows_on) *reinterpret_cast<uint4*>(to + 4 * k * row_bytes) = v;
        }
        __syncwarp();
      }
      tc_fence_before();
      if (!whole) {
        if (w.off > 0) {
          meta_cont = 1;
          meta_done = w.off + w.take == w.total;
        } else {
          meta_rows = min(w.s.n * a.H - w.j * kPgRows, kPgRows);
          meta_row0 = orow - R.base;
        }
      }
    }
    if (tid == 0 && rank == 0) p.meta[pair] = PgMeta{meta_row0, meta_rows, meta_cont, meta_done, 0};
  }
  __syncthreads();
  if (warp == kPgWarpS) {
    // every MMA issued has retired, and every commit has arrived here, before
    // TMEM and shared memory go
    pg_wait_warp(drain, 0u, kErrWaitAccFull);
    pg_wait_warp(drain + 1, 0u, kErrWaitAccFull);
  }
  tc_fence_before();
  cluster_sync_all();                // no CTA leaves while the other may still reach into it
  if (warp == kPgWarpS) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kPgTmemCols) : "memory");
  }
}

// Joins the partials of the items that several parts of the grid share.  CTA
// (i, y): rows of the item that part i of the attention began and did not
// finish, 128 threads a row; its partials are slot 2i + 1 and then slot 2k of
// k = i + 1, i + 2, ... up to the part that ends the item, added in that order.
// Latency counts here: the records of the next 32 parts come with the first
// one, and the first partials are loaded before their weights are known.
constexpr int kPgCombRows = 4, kPgCombY = 16;   // rows of a CTA, CTAs of a part
__global__ void __launch_bounds__(128 * kPgCombRows) paged_attn_combine_kernel(const __grid_constant__ PgParams p, int n_parts) {
  pdl_enter();
  const csa_paged_attn_args& a = p.a;
  const int i = blockIdx.x, lane = threadIdx.x & 31, col = threadIdx.x & 127;
  const PgMeta me = p.meta[i];
  const PgMeta after = i + 1 + lane < n_parts ? p.meta[i + 1 + lane] : PgMeta{0, 0, 0, 0, 0};
  if ((int)blockIdx.y * kPgCombRows >= me.rows) return;
  uint32_t end = __ballot_sync(0xffffffffu, after.cont && after.done);
  int n = __ffs(end) + 1;                      // partials
  for (int k0 = i + 33; !end; k0 += 32) {
    const PgMeta mk = k0 + lane < n_parts ? p.meta[k0 + lane] : PgMeta{0, 0, 0, 1, 1};
    end = __ballot_sync(0xffffffffu, mk.cont && mk.done);
    n = min(k0 - i + __ffs(end), n_parts - i);
  }
  auto slot = [&](int s) { return (int64_t)(s == 0 ? 2 * i + 1 : 2 * (i + s)); };
  for (int row = blockIdx.y * kPgCombRows + (threadIdx.x >> 7); row < me.rows; row += kPgCombRows * kPgCombY) {
    const int64_t orow = me.row0 + row;
    const float* po = p.part_o + (int64_t)row * kD + 4 * col;
    constexpr int kR = 8;
    float4 v[kR];
#pragma unroll
    for (int s = 0; s < kR; ++s)
      v[s] = s < n ? *reinterpret_cast<const float4*>(po + slot(s) * (p.item_rows * kD)) : make_float4(0.f, 0.f, 0.f, 0.f);
    const int head = (int)(orow % a.H);
    const float s0 = a.sink ? a.sink[head] * kPgLog2e : -INFINITY;
    const float2 ml0 = lane < n ? p.part_ml[slot(lane) * p.item_rows + row] : make_float2(-INFINITY, 0.f);
    float M = ml0.x;
    for (int s = lane + 32; s < n; s += 32) M = fmaxf(M, p.part_ml[slot(s) * p.item_rows + row].x);
    M = warp_max(M);
    M = fmaxf(M - kPgPExp, s0);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int sb = 0; sb < n; sb += 32) {
      const float2 ml = sb == 0 ? ml0 : sb + lane < n ? p.part_ml[slot(sb + lane) * p.item_rows + row] : make_float2(-INFINITY, 0.f);
      const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - kPgPExp - M);
      L += wt * ml.y;
      for (int q = 0; q < 32 && sb + q < n; q += kR) {
        if (sb + q > 0) {
#pragma unroll
          for (int s = 0; s < kR; ++s)
            v[s] = sb + q + s < n ? *reinterpret_cast<const float4*>(po + slot(sb + q + s) * (p.item_rows * kD)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int s = 0; s < kR; ++s) {
          // a partial of weight 0 holds nothing (zeros past the last one)
          const float ws = __shfl_sync(0xffffffffu, wt, q + s);
          acc.x += ws * v[s].x; acc.y += ws * v[s].y; acc.z += ws * v[s].z; acc.w += ws * v[s].w;
        }
      }
    }
    L = warp_sum(L);
    const bool any = L > 0.f;
    if (s0 != -INFINITY) L += exp2f(s0 - M);
    const float f = any ? 1.f / L : 0.f;
    if (col == 0 && a.lse) a.lse[orow] = L > 0.f ? (M + log2f(L)) * kPgLn2 : -INFINITY;
    const float* cs = a.rope_cs ? a.rope_cs + orow / a.H * 64 : nullptr;
    store_out4(a.out, true, orow * kD + 4 * col,
               rope_out4(make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f), cs, 4 * col));
  }
}

// Which kernel a call takes: the one-CTA kernel where the sequences have 64
// rows or fewer on average, so that most items of 128 would be half empty.
// Pairs and single CTAs, back to back: 8 x 1 token x 64 heads behind up to
// 65536 FP8 entries 119 and 94 us; 32 x 1 token x 16 heads, FP4, 106 and 70 us;
// 16 x 1 token x 128 heads 117 and 144 us; 4 x 512 tokens x 64 heads 2.30 and
// 3.42 ms.  64 tokens x 64 heads behind 8000 entries beside a chunk of 512 tokens
// behind as many: 745 and 917 us, the two parts alone 126 + 608.  It is an
// average over what the host knows: 64 tokens of which two are one sequence's
// take 165 us on the pairs that they then get, 129 on single CTAs; that chunk,
// padded with 600 sequences without tokens, 800 us on single CTAs, 609 on pairs.
static bool pg_one(const csa_paged_attn_args* a) { return a->n_rows * a->H <= (int64_t)kPgRows / 2 * a->kv.B; }
// Parts of the grid (pairs, or CTAs): all SMs, fewer when the call cannot have
// two tiles for each.
static int pg_parts(const csa_paged_attn_args* a) {
  const bool one = pg_one(a);
  const int rows = one ? kPgRows / 2 : kPgRows, most = one ? kNumSMs : kNumSMs / 2;
  const int64_t items = (a->n_rows * a->H + rows - 1) / rows + a->kv.B;
  const int e = one ? kPgTile<kPgRows / 2> : kPgTile<kPgRows>;
  const int64_t tiles = ((int64_t)a->kv.max_pages * a->kv.page_size + e - 1) / e;
  const int64_t cost = items * (tiles + (one ? kPgItemCost<kPgRows / 2> : kPgItemCost<kPgRows>));
  return cost / 2 < most ? (int)((cost + 1) / 2) : most;
}
static size_t pg_al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Partials of 64 rows in the workspace: two per CTA of either kernel.  One
// bound for both that grows with the call, so that the workspace of a larger
// call serves a smaller one.
static size_t pg_slots(const csa_paged_attn_args* a) {
  const int64_t items = (a->n_rows * a->H + 63) / 64 + a->kv.B;
  const int64_t tiles = ((int64_t)a->kv.max_pages * a->kv.page_size + 31) / 32;
  const int64_t cost = items * (tiles + kPgItemCost<64>);
  return 2 * (size_t)(cost < kNumSMs ? cost : kNumSMs);
}

size_t paged_attn_ws_bytes(const csa_paged_attn_args* a) {
  const size_t n = pg_slots(a);
  return pg_al256(n / 2 * sizeof(PgMeta)) + pg_al256(n * 64 * sizeof(float2)) + n * 64 * kD * sizeof(float);
}

cudaError_t launch_paged_attn_one(const PgParams& p, int ctas, cudaStream_t stream);

static cudaError_t launch_pairs(const PgParams& p, int pairs, cudaStream_t stream) {
  const bool fp4 = p.a.kv.fmt == CSA_FMT_FP4_E2M1_E4M3X16;
  static SmemAttrOnce attr4, attr8;
  const cudaError_t e = fp4 ? attr4.set(paged_attn_kernel<true>, kPgSmemBytes) : attr8.set(paged_attn_kernel<false>, kPgSmemBytes);
  if (e != cudaSuccess) return e;
  ProfScope ps(stream, "paged_attn");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kPgThreads);
  cfg.dynamicSmemBytes = kPgSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return fp4 ? cudaLaunchKernelEx(&cfg, paged_attn_kernel<true>, p) : cudaLaunchKernelEx(&cfg, paged_attn_kernel<false>, p);
}

cudaError_t launch_paged_attn(const csa_paged_attn_args* a, void* ws, cudaStream_t stream) {
  const bool one = pg_one(a);
  const int g = pg_parts(a);
  const size_t n = pg_slots(a);
  PgParams p;
  p.a = *a;
  p.scale_log2 = a->softmax_scale * kPgLog2e;
  p.page_inv = pg_inv((uint32_t)a->kv.page_size);
  p.h_inv = pg_inv((uint32_t)a->H);
  p.item_rows = one ? kPgRows / 2 : kPgRows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.meta = reinterpret_cast<PgMeta*>(w);
  w += pg_al256(n / 2 * sizeof(PgMeta));
  p.part_ml = reinterpret_cast<float2*>(w);
  w += pg_al256(n * 64 * sizeof(float2));
  p.part_o = reinterpret_cast<float*>(w);
  cudaError_t e = one ? launch_paged_attn_one(p, g, stream) : launch_pairs(p, g, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(stream, "paged_attn_combine");
    launch_k(paged_attn_combine_kernel, dim3(g, kPgCombY), dim3(128 * kPgCombRows), 0, stream, p, g);
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
