// kv_fp8b.cu -- writing tokens into the block-scaled 8-bit cache and reading
// ranges of it back (layout and scale rule: kv_fp8b.cuh).
//
// One warp per (sequence, run of blocks, KV head, K or V), block by block,
// holding slots l / 8, l / 8 + 4, ... in lane l.
//
// Write: lane l has dims 8 c .. + 7 and 64 + 8 c .. + 7 (c = l % 8) of its
// slots, so that every load instruction reads four rows' halves of 128
// contiguous bytes.  The rows are loaded into registers (all loads in flight
// together), their largest finite |x| gives the least power-of-two scale that
// holds them, and each value becomes E4M3(x / scale): a product with the
// inverse, exact, in packed bf16.  A block that a sequence has begun before
// (its first new slot is not slot 0) keeps the larger of its scale and that;
// where it grows, the earlier slots' codes are encoded again for the new
// scale.  The slots behind the last new token are not touched: they hold no
// token.  NaN is stored as NaN; an infinity saturates.
// Read: lane l has dims 16 c .. + 15; bf16(E4M3(code) * scale): exact for
// power-of-two scales, else an fp32 product rounded to bf16 (two roundings, as
// a write with such a scale rounds an fp32 quotient to E4M3).
//
// Both are bound by memory: 2 + 1 bytes per value.  What is rare (values that
// are not finite, growing a begun block, a caller's scale that is no power of
// two) is out of line and works from memory, so that the common path stays
// short: with it inlined and unrolled the write stalled on instruction
// fetches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_fp8b.cuh"

namespace pgd {
namespace {

constexpr int kWarps = 4;

// The tokens of this warp: those of sequence b that fall into blocks j0 ..
// j0 + n - 1, KV head g, K or V.  n = 0: nothing to do.
struct Items {
  int b, g, is_v, n;
  long long j0;
  long long p0, p1;   // the sequence's positions [p0, p1)
  long long row0;     // packed row of position p0
  int ids;            // lane i: the id of block j0 + i
};
__device__ __forceinline__ Items find_items(const Kv8bParams &p, int bs, int runs, int run) {
  Items it;
  it.n = 0;
  const long long id = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long per_b = (long long)runs * 2 * p.n_kv;
  if (id >= per_b * p.B) return it;
  it.b = (int)(id / per_b);
  uint32_t r = (uint32_t)(id % per_b);  // (up to 2^32: the host bounds runs * n_kv by 2^31)
  const uint32_t heads = (uint32_t)p.n_kv;
  const int jrel = (int)(r / (2 * heads)) * run;
  r %= 2 * heads;
  it.is_v = (int)(r / heads);
  it.g = (int)(r % heads);
  const TokenRange t = token_range(p.starts, it.b, p.T, p.N);
  const bool first = jrel == 0 && it.g == 0 && it.is_v == 0 && lane == 0;
  if (t.bad) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return it;
  }
  if (t.count == 0) return it;
  it.p0 = (long long)__ldg(p.pos + it.b) + p.pos_offset;
  it.p1 = it.p0 + t.count;
  if (it.p0 < 0 || it.p1 > (long long)p.MB * bs) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return it;
  }
  it.row0 = t.row;
  it.j0 = it.p0 / bs + jrel;
  it.n = (int)max(0ll, min((long long)run, (it.p1 + bs - 1) / bs - it.j0));
  it.ids = lane < it.n ? __ldg(p.tables + (size_t)it.b * p.MB + it.j0 + lane) : 0;
  return it;
}

// Block i of the warp's: its tile, the slots [s0, s1) and the packed row of s0.
// False (and flagged): its id is bad.
struct Item {
  int s0, s1;
  long long row0;
  size_t tile;
};
__device__ __forceinline__ bool find_item(const Kv8bParams &p, int bs, const Items &its, int i,
                                          Item &it) {
  const int blk = __shfl_sync(kFullMask, its.ids, i);
  if ((unsigned)blk >= (unsigned)p.NB) {
    if (its.g == 0 && its.is_v == 0 && (threadIdx.x & 31) == 0)
      atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    return false;
  }
  const long long at = (its.j0 + i) * bs;
  it.s0 = (int)max(0ll, its.p0 - at);
  it.s1 = (int)min((long long)bs, its.p1 - at);
  it.row0 = its.row0 + (at + it.s0 - its.p0);
  it.tile = (size_t)blk * p.n_kv + its.g;
  return true;
}

// The 16 values of a lane (dims 16 c .. + 15 of a slot) as codes.
__device__ __forceinline__ void put16(unsigned char *at, const float (&f)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = (uint32_t)f32x2_to_e4m3x2(f[4 * k], f[4 * k + 1]) |
           ((uint32_t)f32x2_to_e4m3x2(f[4 * k + 2], f[4 * k + 3]) << 16);
  *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The warp's largest finite |x| over rows [row, row + n), as bf16 bits.
__device__ __noinline__ uint32_t finite_max(const __nv_bfloat16 *row, size_t stride, int n) {
  uint32_t top = 0;
  for (int i = threadIdx.x & 31; i < n * kHeadDim; i += 32) {
    const uint32_t a =
        __bfloat16_as_ushort(row[(size_t)(i / kHeadDim) * stride + i % kHeadDim]) & 0x7fffu;
    if (a < 0x7f80u) top = max(top, a);
  }
  return __reduce_max_sync(kFullMask, top);
}

// The codes of slots [0, s0) encoded again for a scale `ratio` times smaller
// relative to their values.
__device__ __noinline__ void rescale_codes(unsigned char *tile, int s0, float ratio) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  for (int s = lane >> 3; s < s0; s += 4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(tile + code_offset8b(s, c));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 y = __half22float2(e4m3x2_to_half2((uint16_t)(w[k >> 1] >> ((k & 1) * 16))));
      f[2 * k] = y.x * ratio;
      f[2 * k + 1] = y.y * ratio;
    }
    put16(tile + code_offset8b(s, c), f);
  }
}

// Rows [row, row + s1 - s0) into slots [s0, s1), divided by any scale.
__device__ __noinline__ void write_divided(unsigned char *tile, const __nv_bfloat16 *row,
                                           size_t stride, int s0, int s1, float scale) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  for (int s = s0 + (lane >> 3); s < s1; s += 4) {
    float f[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      f[k] = __fdiv_rn(__bfloat162float(row[(size_t)(s - s0) * stride + 16 * c + k]), scale);
    put16(tile + code_offset8b(s, c), f);
  }
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t w, __nv_bfloat162 m) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), m);
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <int BS>
__device__ __forceinline__ void append_tile(const Kv8bParams &p, const Items &its,
                                            const Item &it) {
  constexpr int NI = BS / 4;
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const size_t stride = (size_t)p.n_kv * kHeadDim;  // a packed row's
  const __nv_bfloat16 *rows = (its.is_v ? p.v_new : p.k_new) +
                              ((size_t)it.row0 * p.n_kv + its.g) * kHeadDim;  // slot s0's
  unsigned char *tile = (its.is_v ? p.v_cache : p.k_cache) + it.tile * (size_t)(BS * kHeadDim);
  float *scale_at = (its.is_v ? p.v_scales : p.k_scales) + it.tile;
  uint4 x[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (s >= it.s0 && s < it.s1) {
      const uint4 *at = reinterpret_cast<const uint4 *>(rows + (size_t)(s - it.s0) * stride) + c;
      x[i][0] = __ldg(at);
      x[i][1] = __ldg(at + 8);
    }
  }
  const float old = it.s0 > 0 ? *scale_at : 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top = __vmaxu2(top, x[i][h].x & 0x7fff7fffu);
      top = __vmaxu2(top, x[i][h].y & 0x7fff7fffu);
      top = __vmaxu2(top, x[i][h].z & 0x7fff7fffu);
      top = __vmaxu2(top, x[i][h].w & 0x7fff7fffu);
    }
  uint32_t amax = __reduce_max_sync(kFullMask, max(top & 0xffffu, top >> 16));
  if (amax >= 0x7f80u) amax = finite_max(rows, stride, it.s1 - it.s0);
  const float need = pow2f(scale_exponent_e4m3(__uint_as_float(amax << 16)));
  const float scale = it.s0 > 0 ? fmaxf(old, need) : need;
  if (it.s0 > 0 && scale != old) rescale_codes(tile, it.s0, __fdiv_rn(old, scale));
  __syncwarp();
  if (lane == 0) *scale_at = scale;
  // a power of two in the range of the writer's own: its inverse is a bf16
  // number and the products are exact (or so small that they are 0 in E4M3)
  const uint32_t bits = __float_as_uint(scale);
  if ((bits & 0x7fffffu) != 0 || scale < 0x1p-100f || scale > 0x1p120f) {
    write_divided(tile, rows, stride, it.s0, it.s1, scale);
    return;
  }
  const __nv_bfloat162 inv = __float2bfloat162_rn(__uint_as_float(0x7f000000u - bits));
  unsigned char *dst = tile + (c >> 1) * 128 + (c & 1) * 8;  // dims 8 c of slot 0
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    if (s < it.s0 || s >= it.s1) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v[4] = {x[i][h].x, x[i][h].y, x[i][h].z, x[i][h].w};
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t y = bf16x2_mul(v[k], inv);
        q[k] = f32x2_to_e4m3x2(bf16lo(y), bf16hi(y));
      }
      *reinterpret_cast<uint2 *>(dst + (s >> 3) * kGroupBytes8b + (s & 7) * 16 + h * 512) =
          make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    }
  }
}

template <int BS>
__device__ __forceinline__ void read_tile(const Kv8bParams &p, const Items &its, const Item &it) {
  constexpr int NI = BS / 4;
  const int lane = threadIdx.x & 31, c = lane & 7, r = lane >> 3;
  const unsigned char *tile = (its.is_v ? p.v_cache : p.k_cache) + it.tile * (size_t)(BS * kHeadDim);
  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int s = 4 * i + r;
    x[i] = make_uint4(0, 0, 0, 0);
    if (s >= it.s0 && s < it.s1)
      x[i] = __ldg(reinterpret_cast<const uint4 *>(tile + code_offset8b(s, c)));
  }
  const float scale = __ldg((its.is_v ? p.v_scales : p.k_scales) + it.tile);
  uint4 *dst = reinterpret_cast<uint4 *>(its.is_v ? p.v_out : p.k_out) + c * 2;
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
    uint4 *row = dst + ((it.row0 + (s - it.s0)) * p.n_kv + its.g) * (kHeadDim / 8);
    row[0] = make_uint4(o[0], o[1], o[2], o[3]);
    row[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int BS, bool WRITE>
__global__ void __launch_bounds__(kWarps * 32) ranges_kernel(const Kv8bParams p, int runs, int run) {
  pdl_wait();
  pdl_launch_dependents();
  const Items its = find_items(p, BS, runs, run);
#pragma unroll 1
  for (int i = 0; i < its.n; ++i) {
    Item it;
    if (!find_item(p, BS, its, i, it)) continue;
    if constexpr (WRITE)
      append_tile<BS>(p, its, it);
    else
      read_tile<BS>(p, its, it);
  }
}

// The launch over the most blocks that T tokens of a sequence can touch.  A
// writing warp takes one block of few (latency), four of many one after
// another, so that the chain of its first loads (range, position, block ids)
// is paid once for four tiles (56k tokens: 55.7 us, one by one 58.5).  Reading
// back is bound by the stores of twice the bytes it loads, and one block a
// warp spreads those best (16 x 8192 tokens: 130 us, four 137).
template <typename K>
cudaError_t launch(K kernel, const Kv8bParams &p, bool write, cudaStream_t stream) {
  const int JM = most_blocks(p.T, p.bs, p.MB);
  const int run = write && (long long)p.B * JM * p.n_kv * 2 > 16384 ? 4 : 1,
            runs = (JM + run - 1) / run;
  const long long items = (long long)p.B * runs * p.n_kv * 2;
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
  return cudaLaunchKernelEx(&cfg, kernel, p, runs, run);
}

}  // namespace

cudaError_t kv_append_fp8b_launch(const Kv8bParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  return p.bs == 16 ? launch(ranges_kernel<16, true>, p, true, stream)
                    : launch(ranges_kernel<32, true>, p, true, stream);
}

cudaError_t kv_read_fp8b_launch(const Kv8bParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  return p.bs == 16 ? launch(ranges_kernel<16, false>, p, false, stream)
                    : launch(ranges_kernel<32, false>, p, false, stream);
}

}  // namespace pgd
