// csa_paged_attn for short runs of rows: items of 64 query rows on one CTA
// each, where the pair kernel's items of 128 rows would stay half empty (a new
// token of 64 heads, or of 16, is one such item).
//
// Per key tile of 32 entries, K = V = the decoded entries:
//   S = Q K^T       M = 128 TMEM lanes holding the 64 rows twice (lane L: row L
//                   mod 64), N = 32 entries, K = 512.  Channels 0..383 of Q are
//                   the A operand in TMEM, the last 128 in shared memory.  The
//                   two copies let two pairs of softmax warps take turns.
//   O^T += V^T P^T  M = 128 channels (4 chunks), N = 64 rows, K = 32 entries: 4
//                   x 64 TMEM columns, where O (64 x 512) would take all 512.
// An entry is decoded once; its shared-memory copy is the K-major B operand of
// S and the MN-major A operand of O^T, where the pair kernel's CTAs keep two
// tiles and decode half of the other's channels as well.
//
// Bound: latency.  A tile takes 0.93 us (FP8, 64 heads; by the growth of the time
// with the length, 8 tokens behind 65536 and 131072 entries), 1700 to 1800 cycles,
// of which the tensor pipe needs 1090 (S 24 x 16 + 8 x 40, O^T 8 x 48) and shared
// memory 1190 (36 KB written, 112 KB read): with five tiles in flight, a tile's
// way (loads, decode, S, softmax, PV) is five times that long.  FP4 entries, with
// fewer bytes to load, take 0.88 us; 16 heads 0.82 and 0.79.  With tiles of 64
// entries, two and a half of them in flight, 64 entries took 3600 cycles.
// Measured: 8 x 1 token x 64 heads behind up to 65536 FP8 entries 93 us (2.1
// TB/s of entries, 510 TFLOP/s): 72 us of tiles, and 20 us of launches, plan, first
// tile, output and combine; 32 x 1 token x 16 heads behind up to 16384 FP4
// entries 70 us; one token behind 1000 entries 17 us.
#include "paged_attn.cuh"

namespace csa {

constexpr int kP1Rows = 64;
constexpr int kP1E = kPgTile<kP1Rows>;    // entries per key tile
// Warp roles are the pair kernel's, with a second S issuer: 12 and 14, for even
// and odd tiles.  A warp goes on behind a commit only when its MMAs are about
// done, so one alone issued a tile's S every 1630 cycles.  (In the pair kernel
// S would then delay PV: 2.36 ms for 2.11.)
constexpr int kP1Threads = kPgThreads + 32;
constexpr int kP1WarpS2 = kPgWarps;
constexpr int kP1Bufs = 5;                // tiles in flight
constexpr int kP1QBlk = 128 * 128;        // shared Q block: 128 rows x 64 fp16
constexpr int kP1PBytes = kP1Rows * kP1E * 2;
constexpr size_t kP1SmemBytes = 2 * kP1QBlk + kP1Bufs * (kPgKBytes + kP1PBytes) + 2048;
static_assert(kP1SmemBytes <= 232448, "shared memory of a CTA");
static_assert(kPgMaxB / 32 * 8 <= kP1Bufs * kPgKBytes, "the plan's group sums use the entry tiles");

struct P1Smem {
  uint8_t* q;        // channels 384..511 of Q: 2 blocks
  uint8_t* kv;       // [kP1Bufs] 32 entries, 8 blocks of 64 channels
  uint8_t* p;        // [kP1Bufs] P tiles
  float* mx;         // [2][64] tile maxima by tile parity
  float* lx;         // [2][64] sums over the even and the odd tiles
  float* alpha;      // [64] rescale factors
  float* scl;        // [64] output factors
  uint32_t* valid;   // [kP1Bufs] entries present
  int64_t* start;
  uint64_t* bars;
  uint32_t* tmem_base;
};

CSA_DEV P1Smem carve_p1(uint8_t* p) {
  P1Smem s;
  s.q = p; p += 2 * kP1QBlk;
  s.kv = p; p += kP1Bufs * kPgKBytes;
  s.p = p; p += kP1Bufs * kP1PBytes;
  s.mx = reinterpret_cast<float*>(p); p += 2 * 64 * 4;
  s.lx = reinterpret_cast<float*>(p); p += 2 * 64 * 4;
  s.alpha = reinterpret_cast<float*>(p); p += 64 * 4;
  s.scl = reinterpret_cast<float*>(p); p += 64 * 4;
  s.bars = reinterpret_cast<uint64_t*>(p); p += 26 * 8;
  s.start = reinterpret_cast<int64_t*>(p); p += 8 * 8;
  s.valid = reinterpret_cast<uint32_t*>(p); p += 8 * 4;
  s.tmem_base = reinterpret_cast<uint32_t*>(p);
  return s;
}

CSA_DEV void p1_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}"
      ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kPgDesc), "r"(acc) : "memory");
}
CSA_DEV void p1_mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}"
      ::"r"(d), "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kPgDesc), "r"(acc) : "memory");
}

// P rows are 64 bytes (32 fp16): 64-byte swizzle for that operand.
constexpr uint32_t kP1DescP = (512u >> 4) | 1u << 14 | 4u << 29;
CSA_DEV void p1_mma_pv(uint32_t d, uint32_t v_lo, uint32_t p_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}"
      ::"r"(d), "r"(v_lo), "r"(p_lo), "r"(idesc), "n"(kPgDesc), "n"(kP1DescP), "r"(acc) : "memory");
}

template <bool FP4>
__global__ void __launch_bounds__(kP1Threads, 1) paged_attn_one_kernel(const __grid_constant__ PgParams p) {
  constexpr int kScaleOff = FP4 ? 256 : 512;
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const P1Smem S = carve_p1(smem_raw);
  // tile t: buffer t % kP1Bufs, S tile t & 1
  uint64_t* kv_full = S.bars + 0;    // [kP1Bufs] decoded (4 warp arrivals)
  uint64_t* kv_free = S.bars + 5;    // [kP1Bufs] PV done: buffer and P tile reusable (commit)
  uint64_t* p_full = S.bars + 10;    // [kP1Bufs] P written, O^T rescaled (2)
  uint64_t* s_full = S.bars + 15;    // [2] S in TMEM (commit)
  uint64_t* s_free = S.bars + 17;    // [2] S read by the softmax (2)
  uint64_t* q_full = S.bars + 19;    // an item's Q staged (8)
  uint64_t* q_free = S.bars + 20;    // an item's S all done (2 commits)
  uint64_t* acc_done = S.bars + 21;  // an item's last PV done (commit)
  uint64_t* drain = S.bars + 22;     // [3] all MMAs of an issuer retired (teardown)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x, parts = gridDim.x;
  const csa_paged_attn_args& a = p.a;
  if (tid == 0) {
    for (int k = 0; k < kP1Bufs; ++k) {
      mbar_init(kv_full + k, 4);
      mbar_init(kv_free + k, 1);
      mbar_init(p_full + k, 2);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(s_full + k, 1);
      mbar_init(s_free + k, 2);
    }
    for (int k = 0; k < 3; ++k) mbar_init(drain + k, 1);
    mbar_init(q_full, 8);
    mbar_init(q_free, 2);
    mbar_init(acc_done, 1);
    fence_mbar_init();
  }
  if (warp == kPgWarpS) tmem_alloc(S.tmem_base, kPgTmemCols);
  pdl_wait();
  pg_plan<kP1Rows>(p, reinterpret_cast<int64_t*>(S.kv), S.start, part, parts, warp, kP1Threads / 32, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *S.tmem_base;

  if (warp == kPgWarpS || warp == kP1WarpS2) {
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t idesc = idesc_make(kFmtF16, kFmtF16, 128, kP1E);
    const uint32_t mine = warp == kPgWarpS ? 0u : 1u;        // parity of this issuer's tiles
    const uint32_t qd = pg_desc_k(smem_u32(S.q)), kd0 = pg_desc_k(smem_u32(S.kv));
    PgWalk<kP1Rows> w;
    uint32_t t0 = 0, seg = 0;
    bool ok = true;
    w.open(p, S.start);
#pragma unroll 1
    while (ok && w.go(p)) {
      if (w.take == 0) continue;
      ok = pg_wait_warp(q_full, seg++ & 1u, kErrWaitTmaFull);
      const uint32_t end = t0 + (uint32_t)w.take;
#pragma unroll 1
      for (uint32_t t = t0 + ((t0 ^ mine) & 1u); t < end && ok; t += 2) {
        const uint32_t si = mine, bi = t % kP1Bufs;
        if (t >= 2) ok = pg_wait_warp(s_free + si, ((t >> 1) - 1) & 1u, kErrWaitAccEmpty);
        ok = ok && pg_wait_warp(kv_full + bi, (t / kP1Bufs) & 1u, kErrWaitTmaFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t kd = kd0 + bi * (kPgKBytes >> 4), sd = tbase + kPgSCol + kP1E * si;
        if (pg_elect()) {
          // rolled by 64-channel blocks: unrolled, 5 KB of instructions
          // missed the cache once a tile
          uint32_t bd = kd;
#pragma unroll 1
          for (uint32_t kb = 0; kb < (uint32_t)kPgQTmemBlocks; ++kb, bd += kPgKBlk >> 4) {
#pragma unroll
            for (uint32_t sub = 0; sub < 4; ++sub) p1_mma_ts(sd, tbase + kb * 32 + sub * 8, bd + sub * 2, idesc, kb | sub);
          }
#pragma unroll 1
          for (uint32_t kb = 0; kb < 8u - kPgQTmemBlocks; ++kb, bd += kPgKBlk >> 4) {
#pragma unroll
            for (uint32_t sub = 0; sub < 4; ++sub) p1_mma_ss(sd, qd + kb * (kP1QBlk >> 4) + sub * 2, bd + sub * 2, idesc, 1);
          }
          mma_commit(s_full + si);
        }
        __syncwarp();
      }
      t0 = end;
      if (ok && pg_elect()) mma_commit(q_free);
      __syncwarp();
    }
    if (pg_elect()) mma_commit(drain + mine);
    __syncwarp();
  } else if (warp == kPgWarpPV) {
    // ----------------------------------------------------------- PV issuer
    constexpr uint32_t idesc = idesc_make_amn(kFmtF16, kFmtF16, 128, kP1Rows);
    const uint32_t vd0 = pg_desc_mn(smem_u32(S.kv), kPgKBlk), pd0 = pg_desc_k(smem_u32(S.p));
    PgWalk<kP1Rows> w;
    uint32_t t = 0;
    bool ok = true;
    w.open(p, S.start);
#pragma unroll 1
    while (ok && w.go(p)) {
#pragma unroll 1
      for (int i = 0; i < w.take; ++i, ++t) {
        const uint32_t bi = t % kP1Bufs;
        ok = pg_wait_warp(p_full + bi, (t / kP1Bufs) & 1u, kErrWaitAccFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t vd = vd0 + bi * (kPgKBytes >> 4), pd = pd0 + bi * (kP1PBytes >> 4);
        if (pg_elect()) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int ks = 0; ks < kP1E / 16; ++ks) {
              const uint32_t ad = vd + 2 * c * (kPgKBlk >> 4) + ks * (2048 >> 4), bd = pd + ks * 2;
              p1_mma_pv(tbase + kPgOCol + 64u * c, ad, bd, idesc, ks | i);
            }
          }
          mma_commit(kv_free + bi);
          if (i == w.take - 1) mma_commit(acc_done);
        }
        __syncwarp();
      }
    }
    if (pg_elect()) mma_commit(drain + 2);
    __syncwarp();
  } else if (warp >= kPgWarpDec) {
    // ---------------------------------------------- entry loads and decoding
    // Group g (4 warps) takes the CTA's tiles of parity g, 8 entries a warp.
    const int wq = (warp - kPgWarpDec) & 3, g = (warp - kPgWarpDec) >> 2;
    // the first item's query rows come first: their way is the longest
    PgWalk<kP1Rows> w;
    w.open(p, S.start);
    bool go = w.go(p);
#pragma unroll 1
    while (go && w.take == 0) go = w.go(p);
    auto rows = [&]() { return PgRowsIn{w.s.row0, w.j * kP1Rows, min(w.s.n * a.H - w.j * kP1Rows, kP1Rows)}; };
    if (go) pg_fetch_q(p, rows(), S.kv + g * kPgKBytes, wq, lane, g);
    PgCursor<kP1Rows> cu;              // the tile whose page table values are fetched next
    cu.begin(p, S.start, g);
    // page id and entry number in the page of entry 8 wq + (lane & 7) of the
    // tile whose entries are loaded next
    int id = -1;
    uint32_t slot = 0;
    auto lookup = [&]() {
      id = -1;
      if (cu.live) {
        const int pos = cu.w.k0 + (cu.w.off + cu.i) * kP1E + 8 * wq + (lane & 7);
        if (pos < cu.w.k1) {
          int rem;
          const int pg = pg_div(pos, a.kv.page_size, p.page_inv, rem);
          slot = (uint32_t)rem;
          id = a.kv.block_table[(int64_t)cu.w.b * a.kv.table_stride + pg];
        }
      }
    };
    constexpr int kN = FP4 ? 4 : 8;    // 16-byte words per lane and tile
    uint4 r[kN];
    uint2 sc;
    uint32_t vb;                       // valid entries of the warp's 8
    auto at_lane = [&](unsigned long long ptr, int l) {
      return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, ptr, l));
    };
    // FP8: word k is bytes [16 lane, ..) of entry k; FP4: bytes [16 (lane &
    // 15), ..) of entry 2k + (lane >> 4).  kb: the 64-channel block
    const int kb = FP4 ? (lane & 15) >> 1 : lane >> 2;
    // All loads of a tile.  Where there is no entry, the cache's first one is
    // read instead, and the decoder writes zeros.
    auto load_tile = [&]() {
      const bool on = id >= 0 && id < a.kv.n_pages;
      vb = __ballot_sync(0xffffffffu, on) & 0xFFu;
      const unsigned long long ptr =
          (unsigned long long)(a.kv.pages + (on ? (int64_t)id * a.kv.page_stride + (int64_t)slot * a.kv.row_stride : 0));
      const uint8_t* q0;               // the entry whose scales this lane loads
      const int id0 = __shfl_sync(0xffffffffu, id, 0);
      if (__all_sync(0xffffffffu, on && id == id0)) {
        // the usual case: the 8 entries lie in one page
        const int64_t rs = a.kv.row_stride;
        const uint8_t* p0 = at_lane(ptr, 0);
        q0 = p0 + (lane >> 2) * rs;
        const uint8_t* o = p0 + (FP4 ? (lane >> 4) * rs + 16 * (lane & 15) : 16 * lane);
#pragma unroll
        for (int k = 0; k < kN; ++k, o += (FP4 ? 2 : 1) * rs) r[k] = pg_ld_entry<false>(o);
      } else {
#pragma unroll
        for (int k = 0; k < kN; ++k)
          r[k] = pg_ld_entry<false>(at_lane(ptr, FP4 ? 2 * k + (lane >> 4) : k) + 16 * (FP4 ? lane & 15 : lane));
        q0 = at_lane(ptr, lane >> 2);
      }
      // scales: lane 4e + w holds word w of entry e's scale bytes
      if (FP4) sc = *reinterpret_cast<const uint2*>(q0 + kScaleOff + 8 * (lane & 3));
      else sc.x = *reinterpret_cast<const uint32_t*>(q0 + kScaleOff + 4 * (lane & 3));
    };
    lookup();
    load_tile();
    cu.advance(p, 2);
    lookup();
    const uint32_t kv_at = smem_u32(S.kv) + (uint32_t)kb * kPgKBlk;
    uint32_t t0 = 0, seg = 0;          // tiles before the item, items with tiles before it
    bool ok = true;
    // a failed wait leaves `ok` false and skips the later waits and all work;
    // every warp still passes its group's barriers once per item
#pragma unroll 1
    for (; go; go = w.go(p)) {
      if (w.take == 0) continue;
      const PgRowsIn R = rows();
      // the raw rows go through the buffer of the group's next tile
      uint32_t t = t0 + ((t0 ^ (uint32_t)g) & 1u);
      uint8_t* q_buf = S.kv + (t % kP1Bufs) * kPgKBytes;
      if (seg > 0) {
        ok = ok && pg_wait_warp(q_free, (seg - 1) & 1u, kErrWaitSmemEmpty);
        if (ok && t >= kP1Bufs) ok = pg_wait_warp(kv_free + t % kP1Bufs, (t / kP1Bufs - 1) & 1u, kErrWaitSmemEmpty);
        if (ok) pg_fetch_q(p, R, q_buf, wq, lane, g);
      }
      tc_fence_after();
      pg_stage_q<true>(p, R, q_buf, S.q, tbase, wq, lane, g, ok);
      if (ok && lane == 0) mbar_arrive(q_full);
      ++seg;
      t0 += (uint32_t)w.take;
#pragma unroll 1
      for (; t < t0; t += 2) {
        const uint32_t bi = t % kP1Bufs;
        if (ok && t >= kP1Bufs) ok = pg_wait_warp(kv_free + bi, (t / kP1Bufs - 1) & 1u, kErrWaitSmemEmpty);
        if (!ok) continue;
        const uint32_t kt = kv_at + bi * kPgKBytes;
        auto put = [&](int row, int c, const uint4& q) {    // 8 channels of an entry
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       ::"r"(kt + sw128_offset_h(row, c)), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
        };
        if (lane == 0) reinterpret_cast<uint8_t*>(S.valid)[4 * bi + wq] = (uint8_t)vb;
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
        } else {
          const int f = kb & 1;
          if (vb != 0xFFu) {                                 // no entry: zeros
#pragma unroll
            for (int k = 0; k < kN; ++k)
              if (!((vb >> k) & 1u)) r[k] = make_uint4(0, 0, 0, 0);
            if (!((vb >> (lane >> 2)) & 1u)) sc.x = 0;
          }
          if (!__any_sync(0xffffffffu, pg_fp8_far(sc.x))) {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
              const __half2 m = pg_fp8_scale((__shfl_sync(0xffffffffu, sc.x, 4 * k + (lane >> 3)) >> (8 * ((lane >> 1) & 3))) & 0xFFu);
              if (f) r[k] = make_uint4(r[k].z, r[k].w, r[k].x, r[k].y);
              put(8 * wq + k, 16 * (lane & 3) + 8 * f, pg_decode_fp8(r[k].x, r[k].y, m));
              put(8 * wq + k, 16 * (lane & 3) + 8 * (f ^ 1), pg_decode_fp8(r[k].z, r[k].w, m));
            }
          } else {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
              const uint32_t m = (__shfl_sync(0xffffffffu, sc.x, 4 * k + (lane >> 3)) >> (8 * ((lane >> 1) & 3))) & 0xFFu;
              put(8 * wq + k, 16 * (lane & 3), pg_decode_fp8_far(r[k].x, r[k].y, m));
              put(8 * wq + k, 16 * (lane & 3) + 8, pg_decode_fp8_far(r[k].z, r[k].w, m));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full + bi);
        // the next tile's entries, all loads together, then the table values
        // of the tile after it
        load_tile();
        cu.advance(p, 2);
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
    PgWalk<kP1Rows> w;
    uint32_t t = 0, seg = 0;
    bool ok = true;
    int64_t meta_row0 = 0;
    int meta_rows = 0, meta_cont = 0, meta_done = 0;
    w.open(p, S.start);
#pragma unroll 1
    while (w.go(p)) {
      const int nt = w.take, n_on = min(w.s.n * a.H - w.j * kP1Rows, kP1Rows);
      // positions this row sees: (lo, hi]; none for rows past the item's
      int head;
      const int tok = pg_div(w.j * kP1Rows + rr, a.H, p.h_inv, head);
      const int hi = rr < n_on ? w.s.kv - w.s.n + tok : -1;
      const int lo = a.window && hi >= a.window ? hi - a.window : -1;
      float m_run = -INFINITY, l_run = 0.f;    // l_run: this pair's tiles
#pragma unroll 1
      for (int i = 0; i < nt; ++i, ++t) {
        const uint32_t bi = t % kP1Bufs, si = t & 1u;
        const bool own = si == grp;
        uint32_t sv[32];
        float mt = -INFINITY;
        // a failed wait leaves `ok` false and skips the later waits; every
        // warp still passes the group's barriers once per tile
        if (own) {
          const int kb = w.k0 + (w.off + i) * kP1E;
          const int nh = hi - kb + 1, nl = lo - kb + 1;      // the row sees entries [nl, nh) of the tile
          uint32_t mask = nh >= 32 ? 0xffffffffu : nh <= 0 ? 0u : (1u << nh) - 1u;
          mask &= nl <= 0 ? 0xffffffffu : nl >= 32 ? 0u : ~((1u << nl) - 1u);
          ok = ok && pg_wait_warp(s_full + si, (t >> 1) & 1u, kErrWaitAccFull);
          tc_fence_after();
          tmem_ld32(trow + kPgSCol + kP1E * si, sv);
          mask &= S.valid[bi];                 // written before the tile's S was issued
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + si);
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
          mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          S.mx[64 * si + rr] = mt;
        }
        uint32_t over;
        asm volatile("{\n .reg .pred q, r;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred r, 1, 128, q;\n selp.u32 %0, 1, 0, r;\n}"
                     : "=r"(over) : "r"(mt - m_run >= kPgRescale ? 1u : 0u) : "memory");
        if (over) {
          const float mm = S.mx[64 * si + rr];
          float alpha = 1.f;
          if (mm - m_run >= kPgRescale) {
            alpha = m_run == -INFINITY ? 0.f : pg_ex2(m_run - mm);
            m_run = mm;
            l_run *= alpha;
          }
          if (i > 0) {
            if (own) S.alpha[rr] = alpha;
            named_bar(1, 128);
            // O^T (a row is a column of it, in all four warps' lanes), once the
            // PV before this tile's has retired
            ok = ok && pg_wait_warp(kv_free + (t - 1) % kP1Bufs, ((t - 1) / kP1Bufs) & 1u, kErrWaitAccFull);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 256; c += 16) {
              uint32_t o[16];
              tmem_ld16(trow + kPgOCol + c, o);
              tmem_wait_ld();
              const float4* al = reinterpret_cast<const float4*>(S.alpha + (c & 63));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 f = al[k];
                o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * f.x);
                o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * f.y);
                o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * f.z);
                o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * f.w);
              }
              tmem_st16(trow + kPgOCol + c, o);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar(1, 128);                 // every quarter rescaled before this tile's PV
          }
        }
        if (own) {
          // this tile's P buffer is free: its entries were decoded after the
          // PV that read both last.  A row that has seen nothing yet: every
          // logit here is -inf, and so is its max; any finite reference gives
          // the zeros it needs
          pg_add32(sv, m_run == -INFINITY ? 0.f : kPgPExp - m_run);
          float l0 = 0.f, l1 = 0.f;
          uint8_t* pt = S.p + bi * kP1PBytes;
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
      const int64_t orow = (int64_t)w.s.row0 * a.H + w.j * kP1Rows;
      const int slot = 2 * part + (w.off > 0 ? 0 : 1);
      if (grp == 0) {
        const float l = S.lx[rr] + S.lx[64 + rr];
        float scl = 1.f;
        if (whole) {
          const float m0 = m_run - kPgPExp;
          float M = m0, L = l;
          if (a.sink) {
            const float s0 = rr < n_on ? a.sink[head] * kPgLog2e : -INFINITY;
            M = fmaxf(m0, s0);
            const float f = l > 0.f ? exp2f(m0 - M) : 0.f;
            L = l * f + (s0 == -INFINITY ? 0.f : exp2f(s0 - M));
            scl = l > 0.f ? f / L : 0.f;
          } else {
            scl = l > 0.f ? 1.f / l : 0.f;
          }
          if (a.lse && rr < n_on) a.lse[orow + rr] = L > 0.f ? (M + log2f(L)) * kPgLn2 : -INFINITY;
        } else if (rr < n_on) {
          p.part_ml[slot * kP1Rows + rr] = make_float2(m_run, l);
        }
        S.scl[rr] = scl;
      }
      named_bar(1, 128);
      // every PV of the item
      if (nt > 0) ok = ok && pg_wait_warp(acc_done, seg++ & 1u, kErrWaitAccFull);
      tc_fence_after();
      const bool valid_o = nt > 0 && ok;
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {                    // rows (c & 32) .. of channels 2 c ..
        const int k0 = c & 32, ch = 2 * (c & ~63) + 32 * warp + lane;
        if (k0 >= n_on) continue;
        uint32_t o[32];
        if (valid_o) {
          tmem_ld32(trow + kPgOCol + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (!whole) {
          float* dst = p.part_o + ((int64_t)slot * kP1Rows + k0) * kD + ch;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k0 + k < n_on) dst[k * kD] = __uint_as_float(o[k]);
        } else {
          const bool rope = a.rope_cs && c >= 192 && warp >= 2;  // channels 448 ..: pairs in neighbouring lanes
          const int odd = lane & 1;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (orow + k0 + odd) * kD + (ch & ~1);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x[2] = {__uint_as_float(o[k]), __uint_as_float(o[k + 1])};
            if (rope) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float y = __shfl_xor_sync(0xffffffffu, x[u], 1);
                const int row = min(k0 + k + u, n_on - 1);
                const int tk = w.s.row0 + pg_div(w.j * kP1Rows + row, a.H, p.h_inv);
                const float2 z = *reinterpret_cast<const float2*>(a.rope_cs + (int64_t)tk * 64 + (ch & ~1) - 448);
                const float2 f = odd ? rope_inv(y, x[u], z.x, z.y) : rope_inv(x[u], y, z.x, z.y);
                x[u] = odd ? f.y : f.x;
              }
            }
            x[0] *= S.scl[k0 + k];
            x[1] *= S.scl[k0 + k + 1];
            // two channels of row k in even lanes, of row k + 1 in odd ones
            const float y = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], 1);
            const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(y, x[1]) : __floats2bfloat162_rn(x[0], y);
            if (k0 + k + odd < n_on) *reinterpret_cast<__nv_bfloat162*>(dst + k * kD) = v;
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        if (w.off > 0) {
          meta_cont = 1;
          meta_done = w.off + w.take == w.total;
        } else {
          meta_rows = n_on;
          meta_row0 = orow;
        }
      }
    }
    if (tid == 0) p.meta[part] = PgMeta{meta_row0, meta_rows, meta_cont, meta_done, 0};
  }
  __syncthreads();
  if (warp == kPgWarpS) {
    // every MMA issued has retired before TMEM and shared memory go
    pg_wait_warp(drain, 0u, kErrWaitAccFull);
    pg_wait_warp(drain + 1, 0u, kErrWaitAccFull);
    pg_wait_warp(drain + 2, 0u, kErrWaitAccFull);
    tc_fence_after();
    tmem_dealloc(tbase, kPgTmemCols);
  }
}

cudaError_t launch_paged_attn_one(const PgParams& p, int ctas, cudaStream_t stream) {
  const bool fp4 = p.a.kv.fmt == CSA_FMT_FP4_E2M1_E4M3X16;
  static SmemAttrOnce attr4, attr8;
  const cudaError_t e = fp4 ? attr4.set(paged_attn_one_kernel<true>, kP1SmemBytes) : attr8.set(paged_attn_one_kernel<false>, kP1SmemBytes);
  if (e != cudaSuccess) return e;
  ProfScope ps(stream, "paged_attn");
  if (fp4) launch_k(paged_attn_one_kernel<true>, dim3(ctas), dim3(kP1Threads), kP1SmemBytes, stream, p);
  else launch_k(paged_attn_one_kernel<false>, dim3(ctas), dim3(kP1Threads), kP1SmemBytes, stream, p);
  return cudaGetLastError();
}

int read_p1_error(bool clear) {
  int v = 0;
  cudaMemcpyFromSymbol(&v, g_pg_error, sizeof(int));
  if (clear && v) {
    int z = 0;
    cudaMemcpyToSymbol(g_pg_error, &z, sizeof(int));
  }
  return v;
}

}  // namespace csa
