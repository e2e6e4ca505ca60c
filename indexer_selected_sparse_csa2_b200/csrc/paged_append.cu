// Append of new latents to a paged cache (csa_paged_append_args in csa.h):
// RMS norm, partial RoPE and the cache-entry encoder in one pass.
//
// Bound by HBM (1 or 2 KB read, 528 or 288 B written per row) for prompts and
// by latency for a decode batch.  One warp per row, lane l on channels
// [16l, 16l + 16): the norm is one warp sum, the rotated channels 448..511
// are lanes 28-31's own pairs, and the encoder's blocks are lane-local or
// lane pairs.  A row's place takes a chain of four dependent loads (its
// sequence by a 32-way search of cu_q, the sequence's length, the page table),
// so for many rows a warp takes `ch` neighbouring ones, as many as give every
// warp that fits the SMs one such chunk: lane i looks up row i, and the rows'
// values and angles are loaded two rows ahead.
// Measured: 67,000 bf16 rows into FP8 entries 29.7 us (4.1 TB/s; 49 us with a
// search per row, 33-39 us with chunks of 16, 8 or 4 rows); instruction issue
// is then busy for two thirds of the time.  fp32 rows 34 us (4.8 TB/s), into FP4
// entries, with a division a value, 43 us (bf16) and 46 us.  32 rows 9.8 us.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "encode.cuh"
#include "paged.cuh"
#include "rope.cuh"

namespace csa {

template <int SRC, bool ONE>   // ONE: ch is 1
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ csa_paged_append_args a, int chunk) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  constexpr int kEsz = SRC == CSA_SRC_BF16 ? 2 : 4;
  constexpr int kV = SRC == CSA_SRC_BF16 ? 2 : 4;     // 16-byte words of a lane's 16 channels
  constexpr int kAhead = ONE ? 1 : 2;
  const int ch = ONE ? 1 : chunk;                     // 1..32
  const int cu_end = a.kv.cu_q[a.kv.B];
  const int64_t rows = min(a.n_rows, (int64_t)cu_end);
  const int cu_l = a.kv.B <= 32 && lane < a.kv.B ? a.kv.cu_q[lane] : INT_MAX;
  const int len_l = a.kv.B <= 32 && lane < a.kv.B ? a.kv.kv_len[lane] : 0;
  float w[16];
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const float4 v = a.weight ? *reinterpret_cast<const float4*>(a.weight + 16 * lane + k) : make_float4(1.f, 1.f, 1.f, 1.f);
    w[k] = v.x; w[k + 1] = v.y; w[k + 2] = v.z; w[k + 3] = v.w;
  }
  for (int64_t r0 = ch * ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)); r0 < rows; r0 += ch * warps) {
    uint4 raw[kAhead][kV], ang[kAhead];                // ang: a row's (cos, sin), 16 words over lanes 0-15
    auto load = [&](int i, uint4 (&v)[kV], uint4& cs) {
      const int64_t r = min(r0 + i, rows - 1);
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.src) + r * a.src_row_stride * kEsz) + kV * lane;
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] = ld_nc_v4(p + k);
      if (a.rope_cs && lane < 16) cs = ld_nc_v4(a.rope_cs + r * 64 + 4 * lane);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, raw[i], ang[i]);
    // entry of row r0 + lane (lanes < ch), nullptr where there is none
    uint8_t* mine = nullptr;
    const int64_t r = r0 + lane;
    if (a.kv.B <= 32) {
      // the whole batch's tables are in the lanes already
      int b = -1, end = 0, len = 0;
      if (ONE) {
        b = 31 - __clz(__ballot_sync(0xffffffffu, lane < a.kv.B && cu_l <= r0));
      } else {
        for (int j = 0; j < a.kv.B; ++j) b = __shfl_sync(0xffffffffu, cu_l, j) <= r ? j : b;
      }
      len = __shfl_sync(0xffffffffu, len_l, b & 31);
      end = __shfl_sync(0xffffffffu, cu_l, (b + 1) & 31);
      if (b + 1 == a.kv.B) end = cu_end;
      if (lane < ch && r < rows && b >= 0) mine = paged_entry(a.kv, b, (int64_t)len - end + r);
    } else {
      int b = max(paged_find_seq(a.kv.cu_q, a.kv.B, r0, lane), 0);   // -1: r0 lies before the first sequence
      if (lane < ch && r < rows && r >= a.kv.cu_q[0]) {
        while (b + 1 < a.kv.B && a.kv.cu_q[b + 1] <= r) ++b;
        mine = paged_entry(a.kv, b, (int64_t)a.kv.kv_len[b] - a.kv.cu_q[b + 1] + r);
      }
    }
    const int n = (int)min((int64_t)ch, rows - r0);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u;
        float x[16];
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          const uint32_t v[4] = {raw[u][k].x, raw[u][k].y, raw[u][k].z, raw[u][k].w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (SRC == CSA_SRC_BF16) {
              x[8 * k + 2 * m] = __uint_as_float(v[m] << 16);
              x[8 * k + 2 * m + 1] = __uint_as_float(v[m] & 0xffff0000u);
            } else {
              x[4 * k + m] = __uint_as_float(v[m]);
            }
          }
        }
        const uint4 cs = ang[u];
        if (i + kAhead < n) load(i + kAhead, raw[u], ang[u]);
        // i past the last row: lane i holds nullptr, as for a row without an entry
        uint8_t* dst = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)mine, i & 31));
        if (!dst) continue;                            // uniform
        if (a.norm) {
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < 16; ++k) ss = fmaf(x[k], x[k], ss);
          const float rs = rsqrtf(warp_sum(ss) * (1.f / kD) + a.eps);
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] *= rs * w[k];
        }
        if (a.rope_cs) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = (4 * (lane - kRopeStart / 16) + k) & 15;      // used by lanes 28-31
            const float c0 = __uint_as_float(__shfl_sync(0xffffffffu, cs.x, from)), s0 = __uint_as_float(__shfl_sync(0xffffffffu, cs.y, from));
            const float c1 = __uint_as_float(__shfl_sync(0xffffffffu, cs.z, from)), s1 = __uint_as_float(__shfl_sync(0xffffffffu, cs.w, from));
            if (lane >= kRopeStart / 16) {
              const float2 p = rope_fwd(x[4 * k], x[4 * k + 1], c0, s0), q = rope_fwd(x[4 * k + 2], x[4 * k + 3], c1, s1);
              x[4 * k] = p.x; x[4 * k + 1] = p.y; x[4 * k + 2] = q.x; x[4 * k + 3] = q.y;
            }
          }
        }
        __syncwarp();
        if (a.kv.fmt == CSA_FMT_FP4_E2M1_E4M3X16) encode_fp4_vals(x, lane, dst);
        else encode_fp8w_vals(x, lane, dst);
      }
    }
  }
}

template <int SRC>
static void launch_append_t(const csa_paged_append_args* a, cudaStream_t stream) {
  const int64_t warps = (int64_t)kNumSMs * 16;        // two CTAs an SM, by registers
  const int64_t ch = std::min<int64_t>((a->n_rows + warps - 1) / warps, 32);
  const int64_t g = std::min((a->n_rows + 8 * ch - 1) / (8 * ch), (int64_t)kNumSMs * 16);
  if (ch <= 1) launch_k(paged_append_kernel<SRC, true>, dim3((unsigned)g), dim3(256), 0, stream, *a, 1);
  else launch_k(paged_append_kernel<SRC, false>, dim3((unsigned)g), dim3(256), 0, stream, *a, (int)ch);
}

cudaError_t launch_paged_append(const csa_paged_append_args* a, cudaStream_t stream) {
  ProfScope ps(stream, "paged_append");
  if (a->src_dtype == CSA_SRC_BF16) launch_append_t<CSA_SRC_BF16>(a, stream);
  else launch_append_t<CSA_SRC_F32>(a, stream);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace csa
