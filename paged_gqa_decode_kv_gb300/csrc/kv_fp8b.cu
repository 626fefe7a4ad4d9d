// kv_fp8b.cu -- writing tokens into the block-scaled 8-bit cache and reading
// ranges of it back (layout and scale rule: kv_fp8b.cuh).
//
// One warp per (sequence, block, KV head, K or V).  Lane l holds dims
// 16 (l % 8) .. + 15 of slots l / 8, l / 8 + 4, ...: a row is 8 lanes x 32 B
// of bf16 and 8 x 16 B of codes, so both sides move in whole 16-byte vectors.
//
// Write: the rows are loaded into registers (all loads in flight together),
// their largest finite |x| gives the least power-of-two scale that holds
// them, and each value becomes E4M3(x / scale).  A block that a sequence has
// begun before (its first new slot is not slot 0) keeps the larger of its
// scale and that; where it grows, the earlier slots' codes are encoded again
// for the new scale.  The slots behind the last new token are not touched:
// they hold no token.  NaN is stored as NaN; an infinity saturates.
// Read: bf16(E4M3(code) * scale), one rounding (none for power-of-two scales).
//
// Both are bound by memory: 2 + 1 bytes per value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_fp8b.cuh"

namespace pgd {
namespace {

constexpr int kWarps = 4;

// The item of this warp: sequence, block of the sequence and the slots
// [s0, s1) of it that the call's tokens fill.  False: nothing to do.
struct Item {
  int b, g, is_v;
  int s0, s1;
  long long row0;  // packed row of slot s0
  size_t tile;
};
__device__ __forceinline__ bool find_item(const Kv8bParams &p, int bs, int JM, Item &it) {
  const long long id = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long per_b = (long long)JM * 2 * p.n_kv;
  if (id >= per_b * p.B) return false;
  it.b = (int)(id / per_b);
  int r = (int)(id % per_b);
  const int jrel = r / (2 * p.n_kv);
  r %= 2 * p.n_kv;
  it.is_v = r / p.n_kv;
  it.g = r % p.n_kv;
  const TokenRange t = token_range(p.starts, it.b, p.T, p.N);
  const bool first = jrel == 0 && it.g == 0 && it.is_v == 0 && lane == 0;
  if (t.bad) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return false;
  }
  if (t.count == 0) return false;
  const long long p0 = (long long)__ldg(p.pos + it.b) + p.pos_offset, p1 = p0 + t.count;
  if (p0 < 0 || p1 > (long long)p.MB * bs) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return false;
  }
  const long long j = p0 / bs + jrel;
  if (j * bs >= p1) return false;
  const int blk = __ldg(p.tables + (size_t)it.b * p.MB + j);
  if ((unsigned)blk >= (unsigned)p.NB) {
    if (it.g == 0 && it.is_v == 0 && lane == 0) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    return false;
  }
  it.s0 = (int)max(0ll, p0 - j * bs);
  it.s1 = (int)min((long long)bs, p1 - j * bs);
  it.row0 = t.row + (j * bs + it.s0 - p0);
  it.tile = (size_t)blk * p.n_kv + it.g;
  return true;
}

// The largest finite |x| of two bf16 pairs' worth of bits, as bf16 bits (a
// non-finite value counts as 0).
__device__ __forceinline__ uint32_t finite_abs(uint32_t w) {
  w &= 0x7fff7fffu;
  if ((w & 0xffffu) >= 0x7f80u) w &= 0xffff0000u;
  if ((w >> 16) >= 0x7f80u) w &= 0xffffu;
  return w;
}

template <int BS>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const Kv8bParams p, int JM) {
  constexpr int NI = BS / 4;
  pdl_wait();
  pdl_launch_dependents();
  Item it;
  if (!find_item(p, BS, JM, it)) return;
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const uint4 *src = reinterpret_cast<const uint4 *>(it.is_v ? p.v_new : p.k_new) + c * 2;
  unsigned char *tile = (it.is_v ? p.v_cache : p.k_cache) + it.tile * (size_t)(BS * kHeadDim);
  float *scale_at = (it.is_v ? p.v_scales : p.k_scales) + it.tile;
  uint4 x[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (s >= it.s0 && s < it.s1) {
      const uint4 *row = src + ((it.row0 + (s - it.s0)) * p.n_kv + it.g) * (kHeadDim / 8);
      x[i][0] = __ldg(row);
      x[i][1] = __ldg(row + 1);
    }
  }
  const float old = it.s0 > 0 ? *scale_at : 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top = __vmaxu2(top, finite_abs(x[i][h].x));
      top = __vmaxu2(top, finite_abs(x[i][h].y));
      top = __vmaxu2(top, finite_abs(x[i][h].z));
      top = __vmaxu2(top, finite_abs(x[i][h].w));
    }
  const uint32_t amax = __reduce_max_sync(kFullMask, max(top & 0xffffu, top >> 16));
  const float need = pow2f(scale_exponent_e4m3(__uint_as_float(amax << 16)));
  const float scale = it.s0 > 0 ? fmaxf(old, need) : need;
  // x / scale: exact as a product with the inverse where the scale is a power
  // of two (always, unless the caller filled in another one)
  const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
  const float inv = pow2 ? __uint_as_float(0x7f000000u - __float_as_uint(scale)) : 1.f;
  auto put = [&](int s, const float (&f)[16]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (uint32_t)f32x2_to_e4m3x2(f[4 * k], f[4 * k + 1]) |
             ((uint32_t)f32x2_to_e4m3x2(f[4 * k + 2], f[4 * k + 3]) << 16);
    *reinterpret_cast<uint4 *>(tile + code_offset8b(s, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    if (s < it.s0 || s >= it.s1) continue;
    float a[8], b[8], f[16];
    unpack8(x[i][0], a);
    unpack8(x[i][1], b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = pow2 ? a[k] * inv : __fdiv_rn(a[k], scale);
      f[8 + k] = pow2 ? b[k] * inv : __fdiv_rn(b[k], scale);
    }
    put(s, f);
  }
  if (it.s0 > 0 && scale != old) {
    const float ratio = __fdiv_rn(old, scale);
    for (int s = r; s < it.s0; s += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(tile + code_offset8b(s, c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float f[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 y = __half22float2(e4m3x2_to_half2((uint16_t)(w[k >> 1] >> ((k & 1) * 16))));
        f[2 * k] = y.x * ratio;
        f[2 * k + 1] = y.y * ratio;
      }
      put(s, f);
    }
  }
  if (lane == 0) *scale_at = scale;
}

template <int BS>
__global__ void __launch_bounds__(kWarps * 32) read_kernel(const Kv8bParams p, int JM) {
  constexpr int NI = BS / 4;
  pdl_wait();
  pdl_launch_dependents();
  Item it;
  if (!find_item(p, BS, JM, it)) return;
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const unsigned char *tile = (it.is_v ? p.v_cache : p.k_cache) + it.tile * (size_t)(BS * kHeadDim);
  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    x[i] = make_uint4(0, 0, 0, 0);
    if (s >= it.s0 && s < it.s1)
      x[i] = __ldg(reinterpret_cast<const uint4 *>(tile + code_offset8b(s, c)));
  }
  const float scale = __ldg((it.is_v ? p.v_scales : p.k_scales) + it.tile);
  uint4 *dst = reinterpret_cast<uint4 *>(it.is_v ? p.v_out : p.k_out) + c * 2;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    if (s < it.s0 || s >= it.s1) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 y = __half22float2(e4m3x2_to_half2((uint16_t)(w[k >> 1] >> ((k & 1) * 16))));
      const __nv_bfloat162 z = __floats2bfloat162_rn(y.x * scale, y.y * scale);
      o[k] = *reinterpret_cast<const uint32_t *>(&z);
    }
    uint4 *row = dst + ((it.row0 + (s - it.s0)) * p.n_kv + it.g) * (kHeadDim / 8);
    row[0] = make_uint4(o[0], o[1], o[2], o[3]);
    row[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Most blocks that T tokens of a sequence can touch, and the launch over them.
template <typename K>
cudaError_t launch(K kernel, const Kv8bParams &p, cudaStream_t stream) {
  const int JM = 1 + (p.T - 1 + p.bs - 1) / p.bs;
  const long long items = (long long)p.B * JM * p.n_kv * 2;
  const long long grid = (items + kWarps - 1) / kWarps;
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
  return cudaLaunchKernelEx(&cfg, kernel, p, JM);
}

}  // namespace

cudaError_t kv_append_fp8b_launch(const Kv8bParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  return p.bs == 16 ? launch(append_kernel<16>, p, stream) : launch(append_kernel<32>, p, stream);
}

cudaError_t kv_read_fp8b_launch(const Kv8bParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  return p.bs == 16 ? launch(read_kernel<16>, p, stream) : launch(read_kernel<32>, p, stream);
}

}  // namespace pgd
