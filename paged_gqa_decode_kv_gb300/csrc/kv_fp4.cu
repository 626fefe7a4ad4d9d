// kv_fp4.cu -- writing tokens into the 4-bit cache and reading ranges of it
// back (layout: kv_fp4.cuh).
//
// One warp per (sequence, group of 16 positions, KV head, K or V).  Lane l has
// dims 16 c .. 16 c + 15 (c = l % 8) of tokens l / 8, l / 8 + 4, ...: a lane's
// values of a token are one scale's, so nothing is exchanged to find it.
//
// Write.  With m = max |x| over the 16 values and S the call's scale (a power
// of two), s = E4M3(m / 6 / S) and code = E2M1(x / (s S)), both to nearest
// even, saturating.  The quotient is a product with the rounded inverse of
// s S, cut to 12 fraction bits before the conversion: the values at which a
// code changes, times s S, have at most 7 significant bits and x has 8, so an
// x that is not such a value is 2^-8 of it away, one that is comes out within
// 2^-22 and becomes the tie itself: every code is that of the exact quotient.
// V's nibbles of four tokens share a word: the codes pass through shared
// memory, and words with tokens that are not written keep their nibbles.
//
// Read.  E2M1 * E4M3 has 6 significant bits: exact in f16, and in bf16 times S.
//
// Both are bound by memory (2 + 0.56 bytes a value).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_fp4.cuh"

namespace pgd {
namespace {

constexpr int kWarps = 4;
constexpr int kRow = 80;  // bytes between tokens' codes in shared memory (64 and a pad)

// This warp's group: the tokens [t0, t1) of its 16, their packed row and place.
struct Group {
  bool some;
  int g, is_v, t0, t1;
  long long row0;  // packed row of token t0
  size_t at;       // byte of the group in its pool
};

__device__ __forceinline__ Group find_group(const Kv4Params &p, uint32_t groups) {
  Group it;
  it.some = false;
  const long long id = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool lane0 = (threadIdx.x & 31) == 0;
  const uint32_t heads = (uint32_t)p.n_kv;
  const long long per_b = (long long)groups * 2 * heads;
  if (id >= per_b * p.B) return it;
  const int b = (int)(id / per_b);
  uint32_t r = (uint32_t)(id % per_b);
  const uint32_t jrel = r / (2 * heads);
  r %= 2 * heads;
  it.is_v = (int)(r / heads);
  it.g = (int)(r % heads);
  const TokenRange t = token_range(p.starts, b, p.T, p.N);
  const bool first = jrel == 0 && r == 0 && lane0;
  if (t.bad) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return it;
  }
  if (t.count == 0) return it;
  const long long p0 = (long long)__ldg(p.pos + b) + p.pos_offset, p1 = p0 + t.count;
  if (p0 < 0 || p1 > (long long)p.MB * p.bs) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return it;
  }
  const long long base = (p0 / kGroupTokens4 + jrel) * kGroupTokens4;
  if (base >= p1) return it;
  const int blk = __ldg(p.tables + (size_t)b * p.MB + base / p.bs);
  if ((unsigned)blk >= (unsigned)p.NB) {
    if (r == 0 && lane0) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    return it;
  }
  it.t0 = (int)max(0ll, p0 - base);
  it.t1 = (int)min((long long)kGroupTokens4, p1 - base);
  it.row0 = t.row + (base + it.t0 - p0);
  it.at = (((size_t)blk * p.n_kv + it.g) * (p.bs / kGroupTokens4) +
           (size_t)(base % p.bs) / kGroupTokens4) * kGroupBytes4;
  it.some = true;
  return it;
}

__device__ __forceinline__ float to_twelve_bits(float y) {
  return __uint_as_float((__float_as_uint(y) + 0x400u) & 0xfffff800u);
}

// 16 bf16 values as codes (two words) and their scale's byte.
__device__ __forceinline__ uint2 quantise16(const uint4 (&x)[2], float scale, uint32_t &scale_code) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
  // (as bits: an infinity is above every number, a NaN above an infinity)
  const float m = __uint_as_float(max(top & 0xffffu, top >> 16) << 16);
  const float want = __fdiv_rn(m, kE2M1Max) * __frcp_rn(scale);
  scale_code = f32x2_to_e4m3x2(want, 0.f) & 0xffu;
  const float s = __half2float(__low2half(e4m3x2_to_half2((uint16_t)scale_code))) * scale;
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      b[k] = f32x2_to_e2m1x2(to_twelve_bits(bf16lo(w[4 * h + k]) * inv),
                             to_twelve_bits(bf16hi(w[4 * h + k]) * inv));
    c[h] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
  }
  return make_uint2(c[0], c[1]);
}

__device__ __forceinline__ void append_group(const Kv4Params &p, const Group &it,
                                             unsigned char *smem) {
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const size_t stride = (size_t)p.n_kv * (kHeadDim / 8);  // uint4s between tokens
  const uint4 *rows = reinterpret_cast<const uint4 *>(it.is_v ? p.v_new : p.k_new) +
                      ((size_t)it.row0 * p.n_kv + it.g) * (kHeadDim / 8) + 2 * c;
  unsigned char *dst = (it.is_v ? p.v_cache : p.k_cache) + it.at;
  const float scale = it.is_v ? p.v_scale : p.k_scale;
  uint4 x[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * i + r;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (t >= it.t0 && t < it.t1) {
      x[i][0] = __ldg(rows + (size_t)(t - it.t0) * stride);
      x[i][1] = __ldg(rows + (size_t)(t - it.t0) * stride + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * i + r;
    uint32_t sc;
    const uint2 codes = quantise16(x[i], scale, sc);
    const bool there = t >= it.t0 && t < it.t1;
    if (it.is_v) {
      *reinterpret_cast<uint2 *>(smem + t * kRow + c * 8) = codes;
      if (there) dst[kGroupCodes4 + i * 32 + c * 4 + r] = (unsigned char)sc;
    } else if (there) {
      *reinterpret_cast<uint2 *>(dst + t * 64 + c * 8) = codes;
      dst[kGroupCodes4 + t * 8 + c] = (unsigned char)sc;
    }
  }
  if (!it.is_v) return;
  __syncwarp();
  // Lane (row r of 8, tokens 4 t4 ..): the 16-bit words of dims 8 j + r.
  const int t4 = lane & 3, sh = (lane >> 2) * 4;
  uint32_t keep = 0;  // nibbles of a word that stay as they are
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (4 * t4 + u < it.t0 || 4 * t4 + u >= it.t1) keep |= 0xfu << (4 * u);
  if (keep == 0xffffu) return;
  keep |= keep << 16;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned char *src = smem + (4 * t4 + u) * kRow + h * 32;
      const uint4 a = *reinterpret_cast<const uint4 *>(src),
                  b = *reinterpret_cast<const uint4 *>(src + 16);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j >> 1] |= ((w[j] >> sh) & 0xfu) << (16 * (j & 1) + 4 * u);
    }
    uint4 *at = reinterpret_cast<uint4 *>(dst + h * 512 + lane * 16);
    if (keep) {
      const uint4 old = *at;
      o[0] = (o[0] & ~keep) | (old.x & keep);
      o[1] = (o[1] & ~keep) | (old.y & keep);
      o[2] = (o[2] & ~keep) | (old.z & keep);
      o[3] = (o[3] & ~keep) | (old.w & keep);
    }
    *at = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// 16 codes (in the order of the dims) times their scale, as bf16.
__device__ __forceinline__ void expand16(uint2 codes, uint32_t scale_code, float scale, uint4 *dst) {
  const __half2 s2 = e4m3x2_to_half2((uint16_t)(scale_code | (scale_code << 8)));
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t o[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t y[4];
    e2m1x8_to_half2x4(w[h], y);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(__hmul2(bits_half2(y[k]), s2));
      const __nv_bfloat162 z = __floats2bfloat162_rn(f.x * scale, f.y * scale);
      o[4 * h + k] = *reinterpret_cast<const uint32_t *>(&z);
    }
  }
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void read_group(const Kv4Params &p, const Group &it,
                                           unsigned char *smem) {
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const unsigned char *src = (it.is_v ? p.v_cache : p.k_cache) + it.at;
  const float scale = it.is_v ? p.v_scale : p.k_scale;
  uint4 *rows = reinterpret_cast<uint4 *>(it.is_v ? p.v_out : p.k_out) +
                ((size_t)it.row0 * p.n_kv + it.g) * (kHeadDim / 8) + 2 * c;
  const size_t stride = (size_t)p.n_kv * (kHeadDim / 8);
  uint2 codes[4];
  uint32_t sc[4];
  if (it.is_v) {
    const uint4 *at = reinterpret_cast<const uint4 *>(src) + lane;
    const uint4 a = __ldg(at), b = __ldg(at + 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = __ldg(src + kGroupCodes4 + i * 32 + c * 4 + r);
    *reinterpret_cast<uint4 *>(smem + lane * 16) = a;
    *reinterpret_cast<uint4 *>(smem + 512 + lane * 16) = b;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // dims 16 c + k and 16 c + 8 + k of tokens 4 i ..: the halves of a word
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(
            smem + (c >> 2) * 512 + (k * 4 + i) * 16 + (c & 3) * 4) >> (4 * r);
        lo |= (w & 0xfu) << (4 * k);
        hi |= ((w >> 16) & 0xfu) << (4 * k);
      }
      codes[i] = make_uint2(lo, hi);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      codes[i] = __ldg(reinterpret_cast<const uint2 *>(src + (4 * i + r) * 64 + c * 8));
      sc[i] = __ldg(src + kGroupCodes4 + (4 * i + r) * 8 + c);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * i + r;
    if (t >= it.t0 && t < it.t1)
      expand16(codes[i], sc[i], scale, rows + (size_t)(t - it.t0) * stride);
  }
}

template <bool WRITE>
__global__ void __launch_bounds__(kWarps * 32) ranges_fp4_kernel(const Kv4Params p,
                                                                uint32_t groups) {
  __shared__ __align__(16) unsigned char smem[kWarps][kGroupTokens4 * kRow];
  pdl_wait();
  pdl_launch_dependents();
  const Group it = find_group(p, groups);
  if (!it.some) return;
  if constexpr (WRITE)
    append_group(p, it, smem[threadIdx.x >> 5]);
  else
    read_group(p, it, smem[threadIdx.x >> 5]);
}

template <typename K>
cudaError_t launch(K kernel, const Kv4Params &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  const long long groups = most_groups4(p.T, p.bs, p.MB);
  const long long grid = (p.B * groups * 2 * p.n_kv + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, (uint32_t)groups);
}

}  // namespace

cudaError_t kv_append_fp4_launch(const Kv4Params &p, cudaStream_t stream) {
  return launch(ranges_fp4_kernel<true>, p, stream);
}

cudaError_t kv_read_fp4_launch(const Kv4Params &p, cudaStream_t stream) {
  return launch(ranges_fp4_kernel<false>, p, stream);
}

}  // namespace pgd
