// ckpt8.cuh - arithmetic of the 8-bit activation checkpoint, and of MX blocks
// taken from fp32 values, shared by the norm and the checkpoint kernels.
//
// Checkpoint block: 32 consecutive elements of a row share one power of two
// 2^e, e the smallest with amax <= 127 * 2^e (clamped below at -127); the
// code is RN(x * 2^-e), a whole number in [-127, 127], so nothing saturates.
// The byte of the scale is e + 127.  All-zero block: byte 0.  A block that
// holds a NaN or an infinity: byte 0xFF, which loads as NaN everywhere.
// A loaded value code * 2^e has at most seven significant bits: exact in bf16
// (down to bf16's own subnormals).  Against E4M3 codes on the same blocks the
// linear codes keep about five times less error on normal data (0.75% against
// 2.6% of the standard deviation), which is why checkpoints use them: they
// feed no tensor core.
#pragma once

#include "common.cuh"

namespace mx {

// |x| as bits, so that the integer maximum orders NaN above infinity above
// every number.
MX_DEVINL uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Scale byte of a checkpoint block from the fp32 bits of its amax.
MX_DEVINL uint32_t ckpt8_scale(uint32_t amax) {
  const uint32_t E = amax >> 23, m = amax & 0x7FFFFFu;
  if (E == 0xFF) return 0xFF;
  const int s = (int)E - 6 + (m > 0x7E0000u ? 1 : 0);  // 127 = 1.984375 * 2^6
  return s < 0 ? 0u : (uint32_t)s;
}

// E8M0 byte of an MX block from the fp32 bits of its amax (the fp32 form of
// e8m0_from_amax_bits: 448 = 1.75 * 2^8).
MX_DEVINL uint32_t e8m0_from_amax_f32(uint32_t amax, uint32_t rceil) {
  const uint32_t E = amax >> 23, m = amax & 0x7FFFFFu;
  if (E == 0xFF) return 0xFF;
  const int s = (int)E - 8 + ((m > 0x600000u && rceil) ? 1 : 0);
  return s < 0 ? 0u : (uint32_t)s;
}

// 2^(127 - s): finite for every byte that a finite block gets (0 <= s <= 249).
MX_DEVINL float inv_pow2(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^(s - 127); NaN for 0xFF.
MX_DEVINL float pow2_of_byte(uint32_t s) {
  return __uint_as_float(s == 0xFF ? 0x7FC00000u : s ? s << 23 : 0x00400000u);
}

// Four codes RN(x * inv) in one word, element 0 in the lowest byte.  Adding
// 1.5 * 2^23 rounds the exact product once, to nearest even, into the low
// bits of the sum.
MX_DEVINL uint32_t ckpt8_codes4(float a, float b, float c, float d, float inv) {
  const float big = 12582912.0f;
  const uint32_t ua = __float_as_uint(__fmaf_rn(a, inv, big)), ub = __float_as_uint(__fmaf_rn(b, inv, big));
  const uint32_t uc = __float_as_uint(__fmaf_rn(c, inv, big)), ud = __float_as_uint(__fmaf_rn(d, inv, big));
  return __byte_perm(__byte_perm(ua, ub, 0x0040), __byte_perm(uc, ud, 0x0040), 0x5410);
}

// Four codes times the block's power of two.  A code's byte with its sign bit
// flipped is code + 128; placed in the low byte of 2^23 it reads as the fp32
// 2^23 + 128 + code.
MX_DEVINL void ckpt8_values4(uint32_t codes, float scale, float (&v)[4]) {
  const uint32_t u = codes ^ 0x80808080u;
  const float big = 8388736.0f;  // 2^23 + 128
  v[0] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650)), big), scale);
  v[1] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7651)), big), scale);
  v[2] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7652)), big), scale);
  v[3] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7653)), big), scale);
}

MX_DEVINL void values8(uint2 codes, float scale, float (&v)[8]) {
  float a[4], b[4];
  ckpt8_values4(codes.x, scale, a);
  ckpt8_values4(codes.y, scale, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
}

// Eight bf16 of a 16-byte vector as fp32, and back (one rounding each).
MX_DEVINL void unpack8(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
MX_DEVINL uint4 pack8(const float (&v)[8]) {
  return make_uint4(f2_to_bf16x2(f2_pack(v[0], v[1])), f2_to_bf16x2(f2_pack(v[2], v[3])),
                    f2_to_bf16x2(f2_pack(v[4], v[5])), f2_to_bf16x2(f2_pack(v[6], v[7])));
}

// amax (as bits) of a 32-element block held by four consecutive lanes, eight
// elements each.  All 32 lanes take part.
MX_DEVINL uint32_t block_amax(const float (&v)[8]) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(v[i]));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// This lane's eight checkpoint codes of such a block.
MX_DEVINL uint2 ckpt8_encode(const float (&v)[8], uint32_t s) {
  if (s == 0xFF) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = inv_pow2(s);
  return make_uint2(ckpt8_codes4(v[0], v[1], v[2], v[3], inv), ckpt8_codes4(v[4], v[5], v[6], v[7], inv));
}

// This lane's eight E4M3 codes of an MX block (scaling by a power of two is
// exact, so fp32 values round once; NaN and infinite blocks as in MX).
MX_DEVINL uint2 mx_encode(const float (&v)[8], uint32_t s) {
  if (s == 0xFF) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = inv_pow2(s);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = cvt_e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)) |
           (cvt_e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)) << 16);
  return make_uint2(w[0], w[1]);
}

// Reads of data that is used once, past L1.
MX_DEVINL uint4 ld_once(const uint4* p) { return __ldcs(p); }
MX_DEVINL uint2 ld_once(const uint2* p) { return __ldcs(p); }

}  // namespace mx
