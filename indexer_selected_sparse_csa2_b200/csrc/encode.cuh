// Row loaders and cache-entry encoders shared by the encoding kernels (rules:
// see csa_kv_format in csa.h).  One warp encodes one 512-channel entry; lane l
// owns channels [16l, 16l + 16): one FP4 scale block, or half an FP8 one.
#pragma once
#include "common.cuh"

namespace csa {

template <int SRC>  // 0 = fp32, 1 = bf16
CSA_DEV void load16(const void* row, int lane, float (&x)[16]) {
  if (SRC == 0) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + 16 * lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v = ld_nc_v4(p + i);
      x[4 * i + 0] = __uint_as_float(v.x);
      x[4 * i + 1] = __uint_as_float(v.y);
      x[4 * i + 2] = __uint_as_float(v.z);
      x[4 * i + 3] = __uint_as_float(v.w);
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + 16 * lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 v = ld_nc_v4(p + i);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[8 * i + 2 * k + 0] = __uint_as_float(w[k] << 16);          // bf16 -> fp32 is exact
        x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}

// Lane `lane` of a warp encodes channels [16 lane, 16 lane + 16) of one FP4
// entry (one scale block) from values in registers.  Called by all 32 lanes
// of a warp for one entry: the entry is written with 16-byte stores (each
// even lane stores its codes and its odd neighbour's, lanes 0 and 16 the 32
// scale bytes).
CSA_DEV void encode_fp4_vals(const float (&x)[16], int lane, uint8_t* out) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  const uint32_t s_code = enc_e4m3x2(0.f, __fdiv_rn(amax, 6.0f)) & 0xFF;
  const float s = dec_e4m3(s_code);
  uint32_t packed[2] = {0u, 0u};
  if (s != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // even channel in the low nibble
      uint32_t b = enc_e2m1x2(__fdiv_rn(x[2 * i + 1], s), __fdiv_rn(x[2 * i], s));
      packed[i >> 2] |= b << (8 * (i & 3));
    }
  }
  const uint32_t n0 = __shfl_xor_sync(0xffffffffu, packed[0], 1);
  const uint32_t n1 = __shfl_xor_sync(0xffffffffu, packed[1], 1);
  if ((lane & 1) == 0) *reinterpret_cast<uint4*>(out + 8 * lane) = make_uint4(packed[0], packed[1], n0, n1);
  // scale bytes: lane 4w gathers the word of lanes 4w .. 4w + 3, then lanes
  // 0 and 16 gather four words each
  uint32_t word = s_code;
  word |= __shfl_down_sync(0xffffffffu, s_code, 1) << 8;
  word |= __shfl_down_sync(0xffffffffu, s_code, 2) << 16;
  word |= __shfl_down_sync(0xffffffffu, s_code, 3) << 24;
  uint32_t w4[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w4[k] = __shfl_sync(0xffffffffu, word, (lane & 16) + 4 * k);
  if ((lane & 15) == 0) *reinterpret_cast<uint4*>(out + 256 + lane) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
}

// Smallest e with amax <= 448 * 2^e, clamped to [-127, 127]; amax == 0 -> -127.
// amax = (1 + m / 2^23) * 2^E for a normal fp32; 448 = 1.75 * 2^8, so the
// answer is E - 8 when the significand is at most 1.75 and E - 7 otherwise.
CSA_DEV int ue8m0_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int ef = (int)((u >> 23) & 0xFF);
  if (ef == 0) return -127;  // zero or subnormal: far below 448 * 2^-127
  const uint32_t m = u & 0x7FFFFFu;
  int e = (ef - 127) - 8 + (m > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// 2^k as an fp32 value for k in [-127, 127] (2^-127 is subnormal).
CSA_DEV float pow2f(int k) {
  return k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23) : __uint_as_float(1u << 22);
}

// Lane `lane` of a warp encodes channels [16 lane, 16 lane + 16) of one FP8
// window entry (half a scale block) from values in registers.  Called by all
// 32 lanes of a warp for one entry.
CSA_DEV void encode_fp8w_vals(const float (&x)[16], int lane, uint8_t* out) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));   // 32-channel block = lane pair
  const int e = ue8m0_exponent(amax);
  const float sc = pow2f(-e);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = enc_e4m3x2(x[4 * i + 1] * sc, x[4 * i + 0] * sc);
    uint32_t hi = enc_e4m3x2(x[4 * i + 3] * sc, x[4 * i + 2] * sc);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint4*>(out + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((lane & 1) == 0) out[512 + (lane >> 1)] = (uint8_t)(e + 127);
}

}  // namespace csa
