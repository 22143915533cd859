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
#include "tile_quant.cuh"

namespace mx {

// Products and sums straight from the halves of packed bf16 pairs: the two
// elements of a times those of b in fp32 (exact), their squares added to c, and
// the two elements times a power of two plus c (one rounding).
MX_DEVINL f2 mul_bf16x2(uint32_t a, uint32_t b) {
  f2 r;
  asm("{\n .reg .b16 al, ah, bl, bh;\n mov.b32 {al, ah}, %2;\n mov.b32 {bl, bh}, %3;\n"
      " fma.rn.f32.bf16 %0, al, bl, 0f80000000;\n fma.rn.f32.bf16 %1, ah, bh, 0f80000000;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "r"(b));
  return r;
}
MX_DEVINL void sumsq_bf16x2(uint32_t a, f2& c) {
  asm("{\n .reg .b16 al, ah;\n mov.b32 {al, ah}, %2;\n"
      " fma.rn.f32.bf16 %0, al, al, %0;\n fma.rn.f32.bf16 %1, ah, ah, %1;\n}"
      : "+f"(c.x), "+f"(c.y)
      : "r"(a));
}
MX_DEVINL f2 scale_add_bf16x2(uint32_t a, uint16_t pow2, float c) {
  f2 r;
  asm("{\n .reg .b16 al, ah;\n mov.b32 {al, ah}, %2;\n"
      " fma.rn.f32.bf16 %0, al, %3, %4;\n fma.rn.f32.bf16 %1, ah, %3, %4;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(a), "h"(pow2), "f"(c));
  return r;
}

// max(|a|, |b|, |c|); NaN if one is.
MX_DEVINL float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
MX_DEVINL float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// E8M0 byte of an MX block from its amax (not negative; the fp32 form of
// e8m0_from_amax_bits: 448 = 1.75 * 2^8).
MX_DEVINL uint32_t e8m0_from_amax_f32(float amax_f, uint32_t rceil) {
  const uint32_t amax = __float_as_uint(amax_f);
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

// This lane's eight checkpoint codes RN(x * inv), inv a power of two, element
// 0 in the lowest byte.  Adding 1.5 * 2^23 rounds the exact product once, to
// nearest even, into the low bits of the sum.  (A NaN or infinite block has
// inv = infinity; its codes mean nothing.)
MX_DEVINL uint2 ckpt8_encode(const uint4& x, uint16_t inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 v = scale_add_bf16x2(w[i], inv, 12582912.0f);
    h[i] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x0040);
  }
  return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
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
MX_DEVINL uint4 pack8(const f2 (&v)[4]) {
  return make_uint4(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]), f2_to_bf16x2(v[2]), f2_to_bf16x2(v[3]));
}

// Checkpoint scales of two 32-element blocks, each held by four consecutive
// lanes, eight elements (a, b) each: block a's byte in the low half, b's in the
// high half.  The bf16 maxima of both travel in one word, and the rule
// max(((amax + 1) >> 7) - 6, 0) works on both halves at once (the + 1 carries
// into the exponent exactly for significands above 127/64).  All 32 lanes take part.
MX_DEVINL uint32_t ckpt8_block_scales(const uint4& a, const uint4& b) {
  const uint32_t ma = maxabs2(maxabs2(a.x, a.y), maxabs2(a.z, a.w));
  const uint32_t mb = maxabs2(maxabs2(b.x, b.y), maxabs2(b.z, b.w));
  uint32_t m = maxabs2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));
  m = maxabs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = maxabs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2)) & 0x7FFF7FFFu;
  uint32_t s = __viaddmax_s16x2(((m + 0x00010001u) >> 7) & 0x01FF01FFu, 0xFFFAFFFAu, 0u);
  const uint32_t bad = (m + 0x00800080u) & 0x80008000u;  // exponent field 255
  if (bad) s |= (bad >> 15) * 0xFFu;
  return s;
}
// 2^(127 - s) of both blocks, bf16 (+infinity for 0xFF).  Each half is 0x1FE - s,
// 0xFF or more, so that no half borrows from the other, and 0x1FF or less, so that
// none shifts into the other; the sign bit that this leaves is cleared.
MX_DEVINL uint32_t inv_pow2_bf16x2(uint32_t s2) { return ((0x01FE01FEu - s2) << 7) & 0x7FFF7FFFu; }

// This lane's eight E4M3 codes of an MX block with scale byte s (scaling by a
// power of two is exact, so fp32 values round once; a NaN or infinite block
// has a NaN for its inverse scale and every code 0x7F, as in MX).
MX_DEVINL uint2 mx_encode(const f2 (&v)[4], uint32_t s) {
  const f2 inv = f2_splat(s == 0xFF ? __uint_as_float(0x7FC00000u) : inv_pow2(s));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 t = f2_mul(v[i], inv);
    w[i] = cvt_e4m3x2(t.x, t.y);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));  // the shift is part of the conversion
}

// MX scale bytes of two blocks as above (fp32 values): low and high half.  Only
// max(((bits + up) >> 23) - 8, 0) of the maxima matters, with up = 0x1FFFFF
// (RCEIL: carries for significands above 1.75) or 0 (FLOOR), and it is
// monotone, so each lane's own value, 16 bits, is what the lanes exchange.  A
// lane that holds a NaN or an infinity gives 0x7FFF.
MX_DEVINL uint32_t mx_block_scales(const f2 (&a)[4], const f2 (&b)[4], uint32_t up) {
  auto key = [up](const f2 (&v)[4]) {
    float m = max3_abs(v[0].x, v[0].y, v[1].x);
    m = max3_abs(m, v[1].y, v[2].x);
    m = max3_abs(m, v[2].y, v[3].x);
    const uint32_t bits = __float_as_uint(max_abs(m, v[3].y));
    return bits >= 0x7F800000u ? 0x7FFFu : (bits + up) >> 23;
  };
  uint32_t k = __byte_perm(key(a), key(b), 0x5410);
  k = __vmaxs2(k, __shfl_xor_sync(0xFFFFFFFFu, k, 1));
  k = __vmaxs2(k, __shfl_xor_sync(0xFFFFFFFFu, k, 2));
  uint32_t s = __viaddmax_s16x2(k, 0xFFF8FFF8u, 0u);
  if (s & 0x7F007F00u) s |= ((s >> 8) & 0x00010001u) * 0xFFu;
  return s & 0x00FF00FFu;
}

// Reads of data that is used once, past L1.
MX_DEVINL uint4 ld_once(const uint4* p) { return __ldcs(p); }
MX_DEVINL uint2 ld_once(const uint2* p) { return __ldcs(p); }

}  // namespace mx
