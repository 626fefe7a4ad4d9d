// kv_fp4.cu -- writing tokens into the 4-bit cache and reading ranges of it
// back (layout: kv_fp4.cuh).
//
// A warp takes a group of 16 positions of a sequence and one or more of its items
// (KV heads of K, then of V).  Lane l has
// dims 16 c .. 16 c + 15 (c = l % 8) of tokens l / 8, l / 8 + 4, ...: a lane's
// values of a token are one scale's, so nothing is exchanged to find it.
//
// Write.  With m = max |x| over the 16 values and S the call's scale (a power
// of two), s = E4M3(m / 6 / S) and code = E2M1(x / (s S)), both to nearest
// even, saturating.  The quotient is a product with the rounded inverse of
// s S, rounded to a multiple of 2^-12 (by adding and taking off 1.5 * 2^11)
// before the conversion: the quotients at which a code changes are multiples of
// 1/4, and those times s S have at most 7 significant bits where x has 8, so an
// x that is not at such a quotient is 2^-8 of it away, 2^-10 at least, and one
// that is comes out within 2^-21 and becomes the tie itself: every code is that
// of the exact quotient.
// V's nibbles of four tokens share a word: two exchanges among the four lanes
// that hold them turn nibbles of a token's dims into nibbles of a dim's tokens,
// and the group passes through shared memory to leave in 16-byte pieces; words
// with tokens that are not written keep their nibbles.
//
// Read.  E2M1 * E4M3 has 6 significant bits: exact in f16, and in bf16 times S.
//
// The read is bound by memory (16 x 8192 tokens of 8 heads: 106 us, 2 + 0.56 bytes
// a value at the copy rate 102.7), the write by conversions beside it (58 % of the
// issue slots taken, the ALU pipe at 57 %, DRAM at 60 %): 48.6k ragged tokens in 49
// us, 38 at the copy rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_fp4.cuh"

namespace pgd {
namespace {

constexpr int kWarps = 4;
// Items a warp takes of a call of many: four when it writes (48.6k tokens of 8 heads:
// 49.1 us; two 51.2, eight 53.4), two when it reads (43.5; four 45.1).  More groups
// a warp were slower throughout (two: 54.9 and 44.9).
template <bool WRITE>
constexpr int kRun = WRITE ? 4 : 2;
// Bytes of a V group's codes in shared memory, 16 more after every 128 (so that
// the lanes' words fall into different banks).
constexpr int kImage = kGroupCodes4 + kGroupCodes4 / 8;
__device__ __forceinline__ int image_at(int byte) { return byte + (byte >> 7) * 16; }

// 16 codes of one token (16 dims) in each of four lanes l, l ^ 8, l ^ 16, l ^ 24
// (tokens u = l / 8) become 16 bits of each dim 4 a + u, a the 16-bit place, that
// hold the four tokens' codes; and the same again is the way back.
__device__ __forceinline__ uint32_t turn_nibbles(uint32_t w, int lane) {
  const uint32_t y = __shfl_xor_sync(kFullMask, w, 16);
  // bytes: dims 2, 3 of every four for the other lane's 0, 1
  w = __byte_perm(w, y, lane & 16 ? 0x3715 : 0x6240);
  const uint32_t z = __shfl_xor_sync(kFullMask, w, 8);
  const uint32_t keep = lane & 8 ? 0xf0f0f0f0u : 0x0f0f0f0fu;
  return (w & keep) | (__funnelshift_l(z, z, lane & 8 ? 28 : 4) & ~keep);
}

// This warp's work: the tokens [t0, t1) of a group of 16 of a sequence, for the
// items [r0, r1) of its 2 * n_kv (K heads, then V heads).
struct Group {
  int r0, r1, t0, t1;
  long long row0;  // packed row of token t0
  size_t at;       // byte of the group in head 0's tile
};

__device__ __forceinline__ Group find_group(const Kv4Params &p, uint32_t groups, uint32_t run,
                                            uint32_t runs) {
  Group it;
  it.r0 = it.r1 = 0;
  const long long warp = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool lane0 = (threadIdx.x & 31) == 0;
  const uint32_t items = 2 * (uint32_t)p.n_kv;
  const uint32_t per_b = groups * runs;  // (the host bounds B * groups * items by 2^32)
  if (warp >= (long long)per_b * p.B) return it;
  const uint32_t id = (uint32_t)warp;
  const int b = (int)(id / per_b);
  const uint32_t rest = id - (uint32_t)b * per_b, jrel = groups == 1 ? 0 : rest / runs;
  const uint32_t r0 = (rest - jrel * runs) * run;
  const int pos = __ldg(p.pos + b);  // (beside the starts)
  const TokenRange t = token_range(p.starts, b, p.T, p.N);
  const bool first = jrel == 0 && r0 == 0 && lane0;
  if (t.bad) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return it;
  }
  if (t.count == 0) return it;
  const long long p0 = (long long)pos + p.pos_offset, p1 = p0 + t.count;
  if (p0 < 0 || p1 > (long long)p.MB * p.bs) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return it;
  }
  const long long base = (p0 / kGroupTokens4 + jrel) * kGroupTokens4;
  if (base >= p1) return it;
  // (blocks of 16 or 32)
  const int lg_bs = p.bs == 32 ? 5 : 4, in_tile = p.bs / kGroupTokens4;
  const int blk = __ldg(p.tables + (size_t)b * p.MB + (base >> lg_bs));
  if ((unsigned)blk >= (unsigned)p.NB) {
    if (r0 == 0 && lane0) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    return it;
  }
  it.t0 = (int)max(0ll, p0 - base);
  it.t1 = (int)min((long long)kGroupTokens4, p1 - base);
  it.row0 = t.row + (base + it.t0 - p0);
  it.at = ((size_t)blk * p.n_kv * in_tile + ((size_t)base & (p.bs - 1)) / kGroupTokens4) *
          kGroupBytes4;
  it.r0 = (int)r0;
  it.r1 = (int)min(items, r0 + run);
  return it;
}

// Two quotients to a multiple of 2^-12, by paired instructions: issue slots are what
// the write is short of.  |x * inv| stays below 9 but where x is an infinity or its
// scale has saturated (a wanted scale just below 1.5 * 2^-9 becomes 2^-9, the smallest
// there is), so that the sum lies in [2^11, 2^12), whose numbers are 2^-12 apart; past
// it the code is 6 whatever the rounding.
__device__ __forceinline__ float2 quotients(float2 x, float inv) {
  constexpr float kCut = 0x1.8p11f;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\t"
      "mov.b64 c, {%4, %4};\n\tadd.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x.x), "+f"(x.y)
      : "f"(inv), "f"(kCut), "f"(-kCut));
  return x;
}

// 16 bf16 values as codes (two words) and their scale's byte.
__device__ __forceinline__ uint2 quantise16(const uint4 (&x)[2], float inv_scale,
                                            uint32_t &scale_code) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
  // (as bits: an infinity is above every number, a NaN above an infinity)
  const float m = __uint_as_float(max(top & 0xffffu, top >> 16) << 16);
  // m / 6 / S to 12 fraction bits, for the same reason as the quotients below
  const float sixth = m * (1.f / kE2M1Max) * inv_scale;
  float want = __uint_as_float((__float_as_uint(sixth) + 0x400u) & 0xfffff800u);
  if (!(m < __uint_as_float(0x7f800000u))) want = m;  // an infinity or a NaN as it is
  scale_code = f32x2_to_e4m3x2(want, 0.f) & 0xffu;
  const float s = __half2float(__low2half(e4m3x2_to_half2((uint16_t)scale_code)));
  const float inv = s > 0.f ? __fdividef(inv_scale, s) : 0.f;
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 y = quotients(make_float2(bf16lo(w[4 * h + k]), bf16hi(w[4 * h + k])), inv);
      b[k] = f32x2_to_e2m1x2(y.x, y.y);
    }
    c[h] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
  }
  return make_uint2(c[0], c[1]);
}

__device__ __forceinline__ void append_group(const Kv4Params &p, const Group &it, int item,
                                             unsigned char *smem) {
  const bool is_v = item >= p.n_kv;
  const int head = is_v ? item - p.n_kv : item;
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const size_t stride = (size_t)p.n_kv * (kHeadDim / 8);  // uint4s between tokens
  const uint4 *rows = reinterpret_cast<const uint4 *>(is_v ? p.v_new : p.k_new) +
                      ((size_t)it.row0 * p.n_kv + head) * (kHeadDim / 8) + 2 * c;
  unsigned char *dst = (is_v ? p.v_cache : p.k_cache) + it.at +
                             (size_t)head * (p.bs / kGroupTokens4) * kGroupBytes4;
  // (a power of two: its inverse is exact)
  const float inv_scale = __frcp_rn(is_v ? p.v_scale : p.k_scale);
  // V's words that keep nibbles: lane * 16 holds dims of row lane / 4, tokens 4 t4 ..
  const int t4 = lane & 3;
  uint32_t keep = 0;
  uint4 old[2];
  if (is_v) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (4 * t4 + u < it.t0 || 4 * t4 + u >= it.t1) keep |= 0x000f000fu << (4 * u);
    if (keep != 0 && keep != 0xffffffffu) {
      old[0] = *reinterpret_cast<const uint4 *>(dst + lane * 16);
      old[1] = *reinterpret_cast<const uint4 *>(dst + 512 + lane * 16);
    }
  }
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
    if (4 * i + 3 < it.t0 || 4 * i >= it.t1) continue;  // (none of these four)
    uint32_t sc;
    const uint2 codes = quantise16(x[i], inv_scale, sc);
    const bool there = t >= it.t0 && t < it.t1;
    if (is_v) {
      // dims 4 a + r of tokens 4 i ..: a = 0, 2 are words of row r, a = 1, 3 of r + 4
      const uint32_t lo = turn_nibbles(codes.x, lane), hi = turn_nibbles(codes.y, lane);
      const int at = (c >> 2) * 512 + (r * 4 + i) * 16 + (c & 3) * 4;
      *reinterpret_cast<uint32_t *>(smem + image_at(at)) = __byte_perm(lo, hi, 0x5410);
      *reinterpret_cast<uint32_t *>(smem + image_at(at + 256)) = __byte_perm(lo, hi, 0x7632);
      if (there) dst[kGroupCodes4 + i * 32 + c * 4 + r] = (unsigned char)sc;
    } else if (there) {
      *reinterpret_cast<uint2 *>(dst + t * 64 + c * 8) = codes;
      dst[kGroupCodes4 + t * 8 + c] = (unsigned char)sc;
    }
  }
  if (!is_v) return;
  __syncwarp();
  if (keep == 0xffffffffu) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 o = *reinterpret_cast<const uint4 *>(smem + image_at(h * 512 + lane * 16));
    uint4 *at = reinterpret_cast<uint4 *>(dst + h * 512 + lane * 16);
    if (keep) {
      o.x = (o.x & ~keep) | (old[h].x & keep);
      o.y = (o.y & ~keep) | (old[h].y & keep);
      o.z = (o.z & ~keep) | (old[h].z & keep);
      o.w = (o.w & ~keep) | (old[h].w & keep);
    }
    *at = o;
  }
}

// 16 codes (in the order of the dims) times their scale, as bf16.
__device__ __forceinline__ void expand16(uint2 codes, uint32_t scale_code, float scale, uint4 *dst) {
  // (a code times a scale, times a power of two: exact in fp32)
  const float f = __half2float(__low2half(e4m3x2_to_half2((uint16_t)scale_code))) * scale;
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t o[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t y[4];
    e2m1x8_to_half2x4(w[h], y);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(bits_half2(y[k]));
      const __nv_bfloat162 z = __floats2bfloat162_rn(v.x * f, v.y * f);
      o[4 * h + k] = *reinterpret_cast<const uint32_t *>(&z);
    }
  }
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void read_group(const Kv4Params &p, const Group &it, int item,
                                           unsigned char *smem) {
  const bool is_v = item >= p.n_kv;
  const int head = is_v ? item - p.n_kv : item;
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const unsigned char *src = (is_v ? p.v_cache : p.k_cache) + it.at +
                             (size_t)head * (p.bs / kGroupTokens4) * kGroupBytes4;
  const float scale = is_v ? p.v_scale : p.k_scale;
  uint4 *rows = reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out) +
                ((size_t)it.row0 * p.n_kv + head) * (kHeadDim / 8) + 2 * c;
  const size_t stride = (size_t)p.n_kv * (kHeadDim / 8);
  uint2 codes[4];
  uint32_t sc[4];
  if (is_v) {
    const uint4 *at = reinterpret_cast<const uint4 *>(src) + lane;
    const uint4 a = __ldg(at), b = __ldg(at + 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = __ldg(src + kGroupCodes4 + i * 32 + c * 4 + r);
    *reinterpret_cast<uint4 *>(smem + image_at(lane * 16)) = a;
    *reinterpret_cast<uint4 *>(smem + image_at(512 + lane * 16)) = b;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (c >> 2) * 512 + (r * 4 + i) * 16 + (c & 3) * 4;
      const uint32_t x = *reinterpret_cast<const uint32_t *>(smem + image_at(at)),
                     y = *reinterpret_cast<const uint32_t *>(smem + image_at(at + 256));
      codes[i] = make_uint2(turn_nibbles(__byte_perm(x, y, 0x5410), lane),
                            turn_nibbles(__byte_perm(x, y, 0x7632), lane));
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
__global__ void __launch_bounds__(kWarps * 32, WRITE ? 6 : 8)
    ranges_fp4_kernel(const Kv4Params p, uint32_t groups, uint32_t run, uint32_t runs) {
  __shared__ __align__(16) unsigned char smem[kWarps][kImage];
  pdl_wait();
  pdl_launch_dependents();
  const Group it = find_group(p, groups, run, runs);
#pragma unroll 1
  for (int r = it.r0; r < it.r1; ++r) {
    if constexpr (WRITE)
      append_group(p, it, r, smem[threadIdx.x >> 5]);
    else
      read_group(p, it, r, smem[threadIdx.x >> 5]);
    __syncwarp();  // (the group in shared memory has been read)
  }
}

template <bool WRITE>
cudaError_t launch(const Kv4Params &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  const long long groups = most_groups4(p.T, p.bs, p.MB);
  const uint32_t items = 2 * (uint32_t)p.n_kv;
  // one item a warp for few, several of many, which share the chain of loads
  // that finds the group
  const uint32_t run = p.B * groups * items > 16384 ? kRun<WRITE> : 1;
  const uint32_t runs = (items + run - 1) / run;
  const long long grid = (p.B * groups * runs + kWarps - 1) / kWarps;
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
  return cudaLaunchKernelEx(&cfg, ranges_fp4_kernel<WRITE>, p, (uint32_t)groups, run, runs);
}

}  // namespace

cudaError_t kv_append_fp4_launch(const Kv4Params &p, cudaStream_t stream) {
  return launch<true>(p, stream);
}

cudaError_t kv_read_fp4_launch(const Kv4Params &p, cudaStream_t stream) {
  return launch<false>(p, stream);
}

}  // namespace pgd
