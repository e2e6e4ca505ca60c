// Residual addition + RMS norm of token rows, with an output in the rows'
// type and / or E4M3 codes with block scales (rules: csa_norm_args in csa.h).
//
// Bound by HBM: per channel the row (2 or 4 B), the residual in and out, and
// what is written; a row is read once and stays in registers between the sum
// of squares and the output.  A thread owns C chunks of 8 neighbouring
// channels, so a 32-channel scale block is 4 lanes and a 128-channel one 16
// lanes of one warp, and their maxima meet by shuffles.
//   dim <= 1024 : one warp per row (no shared memory, no barrier), 1 to 4 chunks
//                 a lane (544 channels with 3 instead of 4: 27.1 -> 23.8 us).
//   else        : one CTA of dim / (8 C) threads per row.
// CTAs stay for several rows and load the next one before they reduce this
// one, so that loads are in flight through the barrier and the stores (8192
// rows of 4096 bf16 channels with residual and UE8M0 codes: 48.9 -> 41.7 us).
// Measured: those rows 5.66 TB/s, 65537 fp32 rows of 512 channels 5.6 TB/s (48
// us); one row 6.2 us, a launch.
#include <algorithm>

#include "common.cuh"
#include "encode.cuh"

namespace csa {

struct NormParams {
  int64_t n_rows;
  int dim;
  int scale_kind;
  const void* x;
  const void* residual;
  void* residual_out;
  const float* weight;
  void* out;
  uint8_t* codes;
  void* scales;
  int64_t x_stride, residual_stride, residual_out_stride, out_stride, codes_stride, scales_stride;  // elements
  float eps;
};

// Streaming loads without the non-coherent path: residual_out and out may be
// x or residual themselves.
CSA_DEV uint4 ld_stream_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
CSA_DEV void unpack_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
CSA_DEV uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <int SRC>
CSA_DEV void store8(void* base, int64_t i, const float (&f)[8]) {
  if (SRC == CSA_SRC_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

// C chunks of 8 channels per thread; WARP_ROW: one warp per row, else one CTA.
template <int SRC, int C, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 256 : 512) rms_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kV = SRC == CSA_SRC_F32 ? 2 : 1;   // 16-byte words per chunk
  constexpr int kEsz = SRC == CSA_SRC_F32 ? 4 : 2;
  __shared__ float part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = WARP_ROW ? lane : threadIdx.x;     // thread within the row
  const int nt = WARP_ROW ? 32 : blockDim.x;
  const int chunks = p.dim >> 3;
  const int64_t row0 = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  const int64_t step = WARP_ROW ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  pdl_enter();
  const float inv_dim = 1.f / (float)p.dim;
  auto load_row = [&](int64_t r, uint4 (&xv)[C][kV], uint4 (&rv)[C][kV]) {
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + r * p.x_stride * kEsz;
    const uint8_t* rr = static_cast<const uint8_t*>(p.residual) + r * p.residual_stride * kEsz;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = t + c * nt;
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        xv[c][v] = ch < chunks ? ld_stream_v4(xr + (int64_t)ch * 8 * kEsz + 16 * v) : make_uint4(0, 0, 0, 0);
        if (p.residual) rv[c][v] = ch < chunks ? ld_stream_v4(rr + (int64_t)ch * 8 * kEsz + 16 * v) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  int flip = 0;
  uint4 xn[C][kV], rn[C][kV];
  if (row0 < p.n_rows) load_row(row0, xn, rn);
  for (int64_t r = row0; r < p.n_rows; r += step, flip ^= 1) {
    float s[C][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8];
      if (SRC == CSA_SRC_F32) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          s[c][4 * v] = __uint_as_float(xn[c][v].x); s[c][4 * v + 1] = __uint_as_float(xn[c][v].y);
          s[c][4 * v + 2] = __uint_as_float(xn[c][v].z); s[c][4 * v + 3] = __uint_as_float(xn[c][v].w);
          f[4 * v] = __uint_as_float(rn[c][v].x); f[4 * v + 1] = __uint_as_float(rn[c][v].y);
          f[4 * v + 2] = __uint_as_float(rn[c][v].z); f[4 * v + 3] = __uint_as_float(rn[c][v].w);
        }
      } else {
        unpack_bf16x8(xn[c][0], s[c]);
        unpack_bf16x8(rn[c][0], f);
      }
      if (p.residual) {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[c][k] += f[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(s[c][k], s[c][k], ss);
    }
    // the next row is another one, so an output over its own inputs is safe
    if (r + step < p.n_rows) load_row(r + step, xn, rn);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = t + c * nt;
      if (p.residual_out && ch < chunks) store8<SRC>(p.residual_out, r * p.residual_out_stride + 8 * ch, s[c]);
    }
    ss = warp_sum(ss);
    if (!WARP_ROW) {
      // two buffers in turn: a warp may reach the next row's sum while
      // another still reads this one's
      if (lane == 0) part[flip][warp] = ss;
      __syncthreads();
      ss = lane < (nt >> 5) ? part[flip][lane] : 0.f;
      ss = warp_sum(ss);
    }
    const float rs = rsqrtf(ss * inv_dim + p.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = t + c * nt;
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (p.weight && ch < chunks) {
        const float4 a = reinterpret_cast<const float4*>(p.weight)[2 * ch], b = reinterpret_cast<const float4*>(p.weight)[2 * ch + 1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
      }
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[c][k] = s[c][k] * rs * w[k];
        amax = fmaxf(amax, fabsf(s[c][k]));
      }
      if (p.out && ch < chunks) store8<SRC>(p.out, r * p.out_stride + 8 * ch, s[c]);
      if (!p.codes) continue;
      float inv = 1.f;
      if (p.scale_kind == CSA_SCALE_UE8M0X32) {
        // 4 lanes share a block; chunks past the row only meet one another
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = ue8m0_exponent(amax);
        inv = pow2f(-e);
        if ((lane & 3) == 0 && ch < chunks)
          static_cast<uint8_t*>(p.scales)[r * p.scales_stride + (ch >> 2)] = (uint8_t)(e + 127);
      } else if (p.scale_kind == CSA_SCALE_F32X128) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // at least 2^-126, whose reciprocal fp32 holds
        const float sc = amax > 0.f ? fmaxf(__fdiv_rn(amax, 448.f), 0x1p-126f) : 0.f;
        inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
        if ((lane & 15) == 0 && ch < chunks) static_cast<float*>(p.scales)[r * p.scales_stride + (ch >> 4)] = sc;
      }
      if (ch < chunks) {
        uint32_t o[2];
#pragma unroll
        for (int v = 0; v < 2; ++v)
          o[v] = (uint32_t)enc_e4m3x2(s[c][4 * v + 1] * inv, s[c][4 * v] * inv) |
                 ((uint32_t)enc_e4m3x2(s[c][4 * v + 3] * inv, s[c][4 * v + 2] * inv) << 16);
        *reinterpret_cast<uint2*>(p.codes + r * p.codes_stride + 8 * ch) = make_uint2(o[0], o[1]);
      }
    }
  }
}

template <int SRC, int C, bool WARP_ROW>
static void launch_norm_t(const NormParams& p, int threads, int64_t grid, cudaStream_t stream) {
  launch_k(rms_norm_kernel<SRC, C, WARP_ROW>, dim3((unsigned)grid), dim3(threads), 0, stream, p);
}

template <int SRC>
static void launch_norm_src(const NormParams& p, cudaStream_t stream) {
  const int chunks = p.dim >> 3;
  if (chunks <= 128) {
    const int64_t rows_cta = 8;
    int64_t g = (p.n_rows + rows_cta - 1) / rows_cta;
    if (g > (int64_t)kNumSMs * 6) g = (int64_t)kNumSMs * 6;
    // as many chunks a lane as the row needs
    switch ((chunks + 31) / 32) {
      case 1: launch_norm_t<SRC, 1, true>(p, 256, g, stream); break;
      case 2: launch_norm_t<SRC, 2, true>(p, 256, g, stream); break;
      case 3: launch_norm_t<SRC, 3, true>(p, 256, g, stream); break;
      default: launch_norm_t<SRC, 4, true>(p, 256, g, stream);
    }
    return;
  }
  const int C = chunks <= 1024 ? 2 : 4;                     // dim <= 16384: at most 512 threads
  const int threads = ((chunks + C - 1) / C + 31) / 32 * 32;
  const int64_t per_sm = std::max(1, (C == 2 && SRC == CSA_SRC_BF16 ? 1024 : 512) / threads);   // by registers
  const int64_t g = std::min(p.n_rows, kNumSMs * per_sm);
  if (C == 2) launch_norm_t<SRC, 2, false>(p, threads, g, stream);
  else launch_norm_t<SRC, 4, false>(p, threads, g, stream);
}

cudaError_t launch_rms_norm(const csa_norm_args* a, cudaStream_t stream) {
  NormParams p;
  p.n_rows = a->n_rows;
  p.dim = a->dim;
  p.scale_kind = a->scale_kind;
  p.x = a->x;
  p.residual = a->residual;
  p.residual_out = a->residual_out;
  p.weight = a->weight;
  p.out = a->out;
  p.codes = a->codes;
  p.scales = a->scales;
  p.x_stride = a->x_stride;
  p.residual_stride = a->residual_stride;
  p.residual_out_stride = a->residual_out_stride;
  p.out_stride = a->out_stride;
  p.codes_stride = a->codes_stride;
  p.scales_stride = a->scales_stride;
  p.eps = a->eps;
  ProfScope ps(stream, "rms_norm");
  if (a->dtype == CSA_SRC_BF16) launch_norm_src<CSA_SRC_BF16>(p, stream);
  else launch_norm_src<CSA_SRC_F32>(p, stream);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace csa
