// kv_fp8b.cuh -- the block-scaled 8-bit cache: E4M3 codes with one fp32 scale
// per (block of tokens, KV head).  Layout, the scale rule and the parameter
// blocks, shared by the kernels that write, read back and attend to it.
//
// A tile (one block of bs tokens, one KV head) is bs x 128 codes as 8 x 16
// core matrices: code of slot s, dim i at (s / 8) * 1024 + (i / 16) * 128 +
// (s % 8) * 16 + i % 16.  Its value is E4M3(code) * scale[block][head].
//
// The writer's scales are powers of two.  For a floating-point code the
// spacing of the codes is relative, so a power of two costs no precision over
// max / 448 (it costs at most one binade of the subnormal end), and it buys
// exactness elsewhere: x / scale and a read-back are exact but for the E4M3
// rounding itself, and raising the scale of a block that already holds tokens
// only shifts its codes' exponents (a code loses bits only where it falls
// below E4M3's smallest normal, 2^-6 of the scale).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pgd_device.cuh"

namespace pgd {

constexpr int kGroupBytes8b = 8 * kHeadDim;  // 8 tokens of a tile
constexpr int kMinScaleExp = -100;           // a block of zeros (or nearly) takes 2^-100

// 2^e, e an integer in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The smallest integer e >= -100 with a <= top * 2^e, for a finite a >= 0 and
// top = (1 + top_mantissa / 2^23) * 2^top_exp: a's exponent less top's, one
// more where a's mantissa is the larger.  (Zeros and subnormal a take -100.)
__device__ __forceinline__ int scale_exponent(float a, int top_exp, uint32_t top_mantissa) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127 - top_exp + ((bits & 0x7fffffu) > top_mantissa ? 1 : 0);
  return max(e, kMinScaleExp);
}
// top = 448 = 1.75 * 2^8, E4M3's largest value.
__device__ __forceinline__ int scale_exponent_e4m3(float a) {
  return scale_exponent(a, 8, 0x600000u);
}
// top = 127 = 1.984375 * 2^6, int8's largest value.
__device__ __forceinline__ int scale_exponent_int8(float a) {
  return scale_exponent(a, 6, 0x7e0000u);
}

// Byte offset in a tile of dims 16 c .. 16 c + 15 of slot s.
__device__ __forceinline__ int code_offset8b(int s, int c) {
  return (s >> 3) * kGroupBytes8b + c * 128 + (s & 7) * 16;
}

__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float a, float b) {
  return (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint16_t v) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3));
}

// The tokens of one call over ranges of positions: sequence b's are rows
// [first row, first row + count) of the packed arrays, at positions[b] on.
struct TokenRange {
  long long row;  // first packed row
  int count;      // tokens (0: nothing to do, or a bad range)
  bool bad;       // the starts are out of order, out of the arrays or hold over T tokens
};
__device__ __forceinline__ TokenRange token_range(const int32_t *starts, int b, int T, int N) {
  TokenRange r;
  r.row = (long long)b * T;
  r.count = T;
  r.bad = false;
  if (starts) {
    const int s = __ldg(starts + b), e = __ldg(starts + b + 1);
    r.bad = s < 0 || e < s || e > N || e - s > T;
    r.row = s;
    r.count = r.bad ? 0 : e - s;
  }
  return r;
}

// The most blocks of a table row (MB of them) that T > 0 tokens in a row touch.
inline int most_blocks(int T, int bs, int MB) {
  const long long n = 1 + ((long long)T - 1 + bs - 1) / bs;
  return n < MB ? (int)n : MB;
}

// Write and read-back of ranges of positions (kv_fp8b.cu).
struct Kv8bParams {
  const __nv_bfloat16 *k_new, *v_new;  // packed rows [N][n_kv][D] (write)
  __nv_bfloat16 *k_out, *v_out;        // packed rows [N][n_kv][D] (read)
  unsigned char *k_cache, *v_cache;
  float *k_scales, *v_scales;          // [NB][n_kv]
  const int32_t *tables;               // [B][MB]
  const int32_t *pos;                  // [B]
  int pos_offset;                      // added to pos[b]
  const int32_t *starts;               // [B + 1], or null: T tokens each
  int B, T, N, n_kv, bs, MB, NB;
  int32_t *err;
};
cudaError_t kv_append_fp8b_launch(const Kv8bParams &p, cudaStream_t stream);
cudaError_t kv_read_fp8b_launch(const Kv8bParams &p, cudaStream_t stream);

// Decode attention over the block-scaled cache: the parameters of the other
// decode kernels and the scales, indexed by tile (block * n_kv + head).
struct Attn8bParams {
  AttnParams a;
  const float *k_scales;
  const float *v_scales;
};
cudaError_t attention_fp8b_launch(const Attn8bParams &p, int G, int bs, int grid,
                                  cudaStream_t stream);
int cluster_max_tokens();
cudaError_t cluster_attention_fp8b_launch(const Attn8bParams &p, int G, int bs,
                                          cudaStream_t stream);

// Key bounds of blocks and the selection of blocks by them (block_select.cu).
struct BoundsParams {
  signed char *bounds;            // [NB][n_kv][2][D]
  float *bound_scales;            // [NB][n_kv]
  const unsigned char *k_cache;   // bf16 tiles, or 8-bit tiles with k_scales
  const float *k_scales;          // [NB][n_kv], or null: bf16
  const int32_t *tables, *pos, *ctx;  // pos null: 0
  int B, T, n_kv, bs, MB, NB;
  int32_t *err;
};
cudaError_t block_bounds_launch(const BoundsParams &p, cudaStream_t stream);

struct SelectParams {
  int32_t *tiles;                 // [B][n_kv][W]
  int32_t *lens;                  // [B][n_kv]
  const __nv_bfloat16 *q;         // [B][n_q][D]
  const signed char *bounds;
  const float *bound_scales;
  const int32_t *tables, *ctx;
  int B, n_q, n_kv, bs, MB, NB, W, keep_first, keep_last;
  int32_t *err;
};
cudaError_t select_blocks_launch(const SelectParams &p, int G, cudaStream_t stream);
int select_max_blocks();

}  // namespace pgd
