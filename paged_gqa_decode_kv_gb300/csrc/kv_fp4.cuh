// kv_fp4.cuh -- the 4-bit cache: E2M1 codes with one E4M3 scale per token, KV
// head and 16 dims.  Layout, conversions and the parameter blocks, shared by
// the kernels that write, read back and attend to it.
//
// A tile (one block of bs tokens, one KV head) is bs / 16 groups of 1152
// bytes: 1024 of codes, then 128 of scales, 72 bytes a token.  A scale of its
// own for every 16 dims of a token means that appending a token never touches
// what is cached, and keeps E2M1's eight magnitudes near the values.
//
// K: token t's codes at t * 64, two dims a byte, its scales at 1024 + t * 8.
// V is kept as the p.v product takes it, four tokens of one dim in 16 bits, so
// that an attention warp expands a word of codes straight into operand
// registers whose halves are neighbouring tokens.  With t = 4 t4 + u and dim
// i = 16 g + 8 h + r the 16-bit word is at (g / 4) * 512 + (r * 4 + t4) * 16 +
// (g % 4) * 4 + h * 2, token u its nibble u, and the scale at 1024 + t4 * 32 +
// g * 4 + u.  (The lane that holds row r, tokens 4 t4 .. reads 16 bytes at
// lane * 16 of each half: no bank conflict.)
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_fp8b.cuh"

namespace pgd {

constexpr int kGroupTokens4 = 16;
constexpr int kGroupCodes4 = kGroupTokens4 * kHeadDim / 2;           // 1024
constexpr int kGroupBytes4 = kGroupCodes4 + kGroupTokens4 * kHeadDim / 16;  // 1152
constexpr float kE2M1Max = 6.f;

// Eight E2M1 codes as four pairs of halves, in the order of the nibbles.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two values as a byte of E2M1 codes (lo in the low nibble): rounded to
// nearest, ties to the even code, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ __half2 bits_half2(uint32_t w) {
  return *reinterpret_cast<const __half2 *>(&w);
}

// The most 16-token groups of a table row that T > 0 tokens in a row touch.
inline long long most_groups4(long long T, int bs, int MB) {
  const long long n = 1 + (T - 1 + kGroupTokens4 - 1) / kGroupTokens4;
  const long long all = (long long)MB * (bs / kGroupTokens4);
  return n < all ? n : all;
}

// Write and read-back of ranges of positions (kv_fp4.cu).
struct Kv4Params {
  const __nv_bfloat16 *k_new, *v_new;  // packed rows [N][n_kv][D] (write)
  __nv_bfloat16 *k_out, *v_out;        // packed rows [N][n_kv][D] (read)
  unsigned char *k_cache, *v_cache;
  float k_scale, v_scale;              // powers of two
  const int32_t *tables;               // [B][MB]
  const int32_t *pos;                  // [B]
  int pos_offset;                      // added to pos[b]
  const int32_t *starts;               // [B + 1], or null: T tokens each
  int B, T, N, n_kv, bs, MB, NB;
  int32_t *err;
};
cudaError_t kv_append_fp4_launch(const Kv4Params &p, cudaStream_t stream);
cudaError_t kv_read_fp4_launch(const Kv4Params &p, cudaStream_t stream);

// Decode attention over the 4-bit cache (attention_fp4.cu): the parameters of
// the other decode kernels; K's scale is part of a.qk_scale_log2.
struct Attn4Params {
  AttnParams a;
  float v_scale;
  int splits;          // parts of a unit, or 0: automatic,
  int resident;        // ... for this many CTAs at once,
  int least_steps;     // ... of so many steps at least
  int uneven;          // the units are so many that parts of one size do not fill these CTAs
  float inv_resident;  // 1 / resident
};
long long attention_fp4_grid(long long units, long long tokens, int sms);
cudaError_t attention_fp4_launch(const Attn4Params &p, int G, int bs, int grid, int sms,
                                 cudaStream_t stream);

}  // namespace pgd
