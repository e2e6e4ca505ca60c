// Append of new latents to a paged cache (csa_paged_append_args in csa.h):
// RMS norm, partial RoPE and the cache-entry encoder in one pass.
//
// Bound by HBM (1 or 2 KB read, 528 or 288 B written per row) for prompts and
// by latency for a decode batch.  One warp per row, lane l on channels
// [16l, 16l + 16): the norm is one warp sum, the rotated channels 448..511
// are lanes 28-31's own pairs, and the encoder's blocks are lane-local or
// lane pairs.  The row's sequence comes from a 32-way search of cu_q, under
// the loads of the row.
#include "common.cuh"
#include "encode.cuh"
#include "paged.cuh"
#include "rope.cuh"

namespace csa {

template <int SRC>
__global__ void __launch_bounds__(256) paged_append_kernel(csa_paged_append_args a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  constexpr int kEsz = SRC == CSA_SRC_BF16 ? 2 : 4;
  const int64_t rows = min(a.n_rows, (int64_t)a.kv.cu_q[a.kv.B]);
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += warps) {
    float x[16];
    load16<SRC>(static_cast<const uint8_t*>(a.src) + r * a.src_row_stride * kEsz, lane, x);
    const int b = paged_find_seq(a.kv.cu_q, a.kv.B, r, lane);
    if (b < 0) continue;
    uint8_t* dst = paged_entry(a.kv, b, (int64_t)a.kv.kv_len[b] - a.kv.cu_q[b + 1] + r);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) ss = fmaf(x[k], x[k], ss);
      const float rs = rsqrtf(warp_sum(ss) * (1.f / kD) + a.eps);
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        const float4 w = a.weight ? *reinterpret_cast<const float4*>(a.weight + 16 * lane + k) : make_float4(1.f, 1.f, 1.f, 1.f);
        x[k] *= rs * w.x; x[k + 1] *= rs * w.y; x[k + 2] *= rs * w.z; x[k + 3] *= rs * w.w;
      }
    }
    if (a.rope_cs && lane >= kRopeStart / 16) {
      const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + r * 64 + 16 * (lane - kRopeStart / 16));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 c = cs[k];
        const float2 u = rope_fwd(x[4 * k], x[4 * k + 1], c.x, c.y), v = rope_fwd(x[4 * k + 2], x[4 * k + 3], c.z, c.w);
        x[4 * k] = u.x; x[4 * k + 1] = u.y; x[4 * k + 2] = v.x; x[4 * k + 3] = v.y;
      }
    }
    __syncwarp();
    if (!dst) continue;                      // uniform: every lane found the same entry
    if (a.kv.fmt == CSA_FMT_FP4_E2M1_E4M3X16) encode_fp4_vals(x, lane, dst);
    else encode_fp8w_vals(x, lane, dst);
  }
}

cudaError_t launch_paged_append(const csa_paged_append_args* a, cudaStream_t stream) {
  int64_t g = (a->n_rows + 7) / 8;
  if (g > (int64_t)kNumSMs * 8) g = (int64_t)kNumSMs * 8;
  ProfScope ps(stream, "paged_append");
  if (a->src_dtype == CSA_SRC_BF16) launch_k(paged_append_kernel<CSA_SRC_BF16>, dim3((unsigned)g), dim3(256), 0, stream, *a);
  else launch_k(paged_append_kernel<CSA_SRC_F32>, dim3((unsigned)g), dim3(256), 0, stream, *a);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace csa
