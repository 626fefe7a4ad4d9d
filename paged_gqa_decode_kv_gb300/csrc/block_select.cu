// block_select.cu -- key bounds of cache blocks, and the selection of the
// blocks that a query's decode attention reads.
//
// Bounds.  Per tile (block, KV head): an int8 lower and upper bound of every
// key dim over the block's tokens, with one power-of-two scale s (the least
// with max |k| <= 127 s): lo_i = floor(min_t k_ti / s), hi_i = ceil(max_t
// k_ti / s).  So s lo_i <= k_ti <= s hi_i for every token, in 260 bytes
// against the tile's 4096 (bf16) or 2048 (8-bit) of keys at 16 tokens.
//
// Score.  With the query rounded to int8 (q'_h = rint(q_h / f_h), f_h the
// least power of two with max |q_h| <= 127 f_h),
//   score = s * max_h f_h * sum_i (max(q'_hi, 0) hi_i + min(q'_hi, 0) lo_i)
// over the heads h that share the KV head: an upper bound of every
// f_h q'_h . k_t in the block, so a block left out holds no key whose product
// with the rounded query exceeds the least selected score.  The sums are
// integers below 2^23 and the factors powers of two: every step is exact in
// fp32, no order of summation changes a score, and ties are real (the lower
// block wins).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_fp8b.cuh"

namespace pgd {
namespace {

constexpr int kBoundWarps = 4;

// One warp per tile to be updated.  bf16: lane = (16-byte chunk of 8 dims,
// half of each 8-token group); 8-bit: lane = (16-byte chunk of 16 dims,
// quarter).  Minimum and maximum over the lane's tokens in the storage's own
// precision (bf16, or f16 for widened codes: exact), then over the lanes that
// share the dims; fminf/fmaxf semantics, so a NaN among numbers is passed
// over.  Bound by the read of the keys.
template <int BS, bool FP8>
__global__ void __launch_bounds__(kBoundWarps * 32) bounds_kernel(const BoundsParams p, int JM) {
  pdl_wait();
  pdl_launch_dependents();
  const long long id = (long long)blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long per_b = (long long)JM * p.n_kv;
  if (id >= per_b * p.B) return;
  const int b = (int)(id / per_b), r = (int)(id % per_b);
  const int jrel = r / p.n_kv, g = r % p.n_kv;
  const int ctx = __ldg(p.ctx + b), p0 = p.pos ? __ldg(p.pos + b) : 0;
  const bool first = jrel == 0 && g == 0 && lane == 0;
  if (ctx < 0 || ctx > p.MB * BS) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
    return;
  }
  if (p0 < 0 || p0 > ctx || ctx - p0 > p.T) {
    if (first) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    return;
  }
  const int j = p0 / BS + jrel;
  if (p0 == ctx || j * BS >= ctx) return;
  const int blk = __ldg(p.tables + (size_t)b * p.MB + j);
  if ((unsigned)blk >= (unsigned)p.NB) {
    if (g == 0 && lane == 0) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    return;
  }
  const int valid = min(BS, ctx - j * BS);
  const size_t tile = (size_t)blk * p.n_kv + g;
  constexpr int ND = FP8 ? 16 : 8;  // dims of a lane
  float lo[ND], hi[ND];
  const float inf = __int_as_float(0x7f800000);
  if constexpr (FP8) {
    const int c = lane & 7, qt = lane >> 3;
    const unsigned char *base = p.k_cache + tile * (size_t)(BS * kHeadDim);
    uint4 x[BS / 4];
#pragma unroll
    for (int i = 0; i < BS / 4; ++i) {
      const int s = (i >> 1) * 8 + qt * 2 + (i & 1);
      x[i] = make_uint4(0, 0, 0, 0);
      if (s < valid) x[i] = __ldg(reinterpret_cast<const uint4 *>(base + code_offset8b(s, c)));
    }
    const float scale = __ldg(p.k_scales + tile);
    __half2 l[8], h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      l[k] = __half2half2(__ushort_as_half(0x7c00));
      h[k] = __half2half2(__ushort_as_half(0xfc00));
    }
#pragma unroll
    for (int i = 0; i < BS / 4; ++i) {
      const int s = (i >> 1) * 8 + qt * 2 + (i & 1);
      if (s < valid) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __half2 v = e4m3x2_to_half2((uint16_t)(w[k >> 1] >> ((k & 1) * 16)));
          l[k] = __hmin2(l[k], v);
          h[k] = __hmax2(h[k], v);
        }
      }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        l[k] = __hmin2(l[k], __shfl_xor_sync(kFullMask, l[k], o));
        h[k] = __hmax2(h[k], __shfl_xor_sync(kFullMask, h[k], o));
      }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 a = __half22float2(l[k]), bb = __half22float2(h[k]);
      lo[2 * k] = a.x * scale; lo[2 * k + 1] = a.y * scale;
      hi[2 * k] = bb.x * scale; hi[2 * k + 1] = bb.y * scale;
    }
  } else {
    const int c = lane & 15, half = lane >> 4;
    const uint4 *base = reinterpret_cast<const uint4 *>(p.k_cache) + tile * (size_t)(BS * 16);
    uint4 x[BS / 2];
#pragma unroll
    for (int i = 0; i < BS / 2; ++i) {
      const int s = (i >> 2) * 8 + half * 4 + (i & 3);
      x[i] = make_uint4(0, 0, 0, 0);
      if (s < valid) x[i] = __ldg(base + (s >> 3) * 128 + c * 8 + (s & 7));
    }
    __nv_bfloat162 l[4], h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l[k] = __bfloat162bfloat162(__ushort_as_bfloat16(0x7f80));
      h[k] = __bfloat162bfloat162(__ushort_as_bfloat16(0xff80));
    }
#pragma unroll
    for (int i = 0; i < BS / 2; ++i) {
      const int s = (i >> 2) * 8 + half * 4 + (i & 3);
      if (s < valid) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&w[k]);
          l[k] = __hmin2(l[k], v);
          h[k] = __hmax2(h[k], v);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l[k] = __hmin2(l[k], __shfl_xor_sync(kFullMask, l[k], 16));
      h[k] = __hmax2(h[k], __shfl_xor_sync(kFullMask, h[k], 16));
      const float2 a = __bfloat1622float2(l[k]), bb = __bfloat1622float2(h[k]);
      lo[2 * k] = a.x; lo[2 * k + 1] = a.y;
      hi[2 * k] = bb.x; hi[2 * k + 1] = bb.y;
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < ND; ++k) {
    const float m = fmaxf(fabsf(lo[k]), fabsf(hi[k]));
    amax = fmaxf(amax, m < inf ? m : 0.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
  const int e = scale_exponent_int8(amax);
  const float inv = pow2f(-e);
  const int part = FP8 ? lane >> 3 : lane >> 4;  // 0 writes the lower bounds, 1 the upper
  if (part < 2) {
    uint32_t w[ND / 4];
#pragma unroll
    for (int k = 0; k < ND / 4; ++k) {
      w[k] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = part ? ceilf(hi[4 * k + i] * inv) : floorf(lo[4 * k + i] * inv);
        const int n = (int)fminf(fmaxf(v, -127.f), 127.f);
        w[k] |= (uint32_t)(n & 0xff) << (8 * i);
      }
    }
    signed char *dst = p.bounds + tile * (2 * kHeadDim) + part * kHeadDim;
    if constexpr (FP8)
      *reinterpret_cast<uint4 *>(dst + (lane & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2 *>(dst + (lane & 15) * 8) = make_uint2(w[0], w[1]);
  }
  if (lane == 0) p.bound_scales[tile] = pow2f(e);
}

template <typename K, typename P, typename... A>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const P &p, A... more) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, more...);
}

// ------------------------------------------------------------------ selection
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;

// A float's bits as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, KV head).  Eight lanes score a block: lane i holds
// dims 16 i .. + 15 of both bounds (two 16-byte loads) and of the G rounded
// queries (positive and negative parts), four products of int8 per
// instruction.  The keys of the scores stay in shared memory; the W-th
// largest is found digit by digit (8 bits a pass, histogram of the keys that
// share the digits so far), then the selected blocks are written in order.
template <int G>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];  // [MB]
  __shared__ uint32_t hist[256];
  __shared__ int warp_sum[2][kSelWarps];
  __shared__ int digit_out[2];
  __shared__ __align__(16) signed char qpos[G][kHeadDim], qneg[G][kHeadDim];
  __shared__ float qf[G];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.n_kv, g = blockIdx.x % p.n_kv;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = __ldg(p.ctx + b);
  const int W = p.W;
  int32_t *tiles = p.tiles + (size_t)blockIdx.x * W;
  const int32_t *row = p.tables + (size_t)b * p.MB;
  if (ctx < 1 || ctx > p.MB * p.bs) {
    if (tid == 0 && g == 0) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
    for (int i = tid; i < W; i += kSelThreads) tiles[i] = -1;
    if (tid == 0) p.lens[blockIdx.x] = 0;
    return;
  }
  const int nblk = (ctx + p.bs - 1) / p.bs;
  const int tail = ctx - (nblk - 1) * p.bs;
  if (tid == 0) p.lens[blockIdx.x] = (min(nblk, W) - 1) * p.bs + tail;
  auto tile_of = [&](int j) {
    const int blk = __ldg(row + j);
    return (unsigned)blk < (unsigned)p.NB ? blk * p.n_kv + g : -1;
  };
  if (nblk <= W) {  // everything is selected
    for (int i = tid; i < W; i += kSelThreads) tiles[i] = i < nblk ? tile_of(i) : -1;
    return;
  }
  // The rounded queries: warp h takes head h (8 heads at most).
  if (warp < G) {
    const uint2 raw = __ldg(reinterpret_cast<const uint2 *>(
        p.q + ((size_t)b * p.n_q + g * G + warp) * kHeadDim) + lane);
    float f[4];
    unpack4(raw, f);
    float a = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
    const int e = scale_exponent_int8(fminf(a, 3.3895314e38f));
    const float inv = pow2f(-e);
    uint32_t wp = 0, wn = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = max(-127, min(127, __float2int_rn(f[i] * inv)));
      wp |= (uint32_t)(max(n, 0) & 0xff) << (8 * i);
      wn |= (uint32_t)(min(n, 0) & 0xff) << (8 * i);
    }
    reinterpret_cast<uint32_t *>(qpos[warp])[lane] = wp;
    reinterpret_cast<uint32_t *>(qneg[warp])[lane] = wn;
    if (lane == 0) qf[warp] = pow2f(e);
  }
  __syncthreads();
  {
    const int i8 = lane & 7;
    uint4 qp[G], qn[G];
    float f[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      qp[h] = *reinterpret_cast<const uint4 *>(&qpos[h][16 * i8]);
      qn[h] = *reinterpret_cast<const uint4 *>(&qneg[h][16 * i8]);
      f[h] = qf[h];
    }
    for (int j0 = 0; j0 < nblk; j0 += kSelThreads / 8) {
      const int j = j0 + (tid >> 3);
      int blk = -1;
      if (j < nblk) blk = __ldg(row + j);
      const bool there = (unsigned)blk < (unsigned)p.NB;
      const size_t tile = there ? (size_t)blk * p.n_kv + g : 0;
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      float s = 0.f;
      if (there) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds + tile * (2 * kHeadDim));
        lo = __ldg(src + i8);
        hi = __ldg(src + 8 + i8);
        s = __ldg(p.bound_scales + tile);
      }
      float best = -__int_as_float(0x7f800000);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        int d = 0;
        d = __dp4a((int)hi.x, (int)qp[h].x, d); d = __dp4a((int)hi.y, (int)qp[h].y, d);
        d = __dp4a((int)hi.z, (int)qp[h].z, d); d = __dp4a((int)hi.w, (int)qp[h].w, d);
        d = __dp4a((int)lo.x, (int)qn[h].x, d); d = __dp4a((int)lo.y, (int)qn[h].y, d);
        d = __dp4a((int)lo.z, (int)qn[h].z, d); d = __dp4a((int)lo.w, (int)qn[h].w, d);
        d += __shfl_xor_sync(kFullMask, d, 1);
        d += __shfl_xor_sync(kFullMask, d, 2);
        d += __shfl_xor_sync(kFullMask, d, 4);
        best = fmaxf(best, (float)d * f[h]);
      }
      if (i8 == 0 && j < nblk) {
        const bool kept = j < p.keep_first || j >= nblk - p.keep_last;
        keys[j] = kept ? 0xffffffffu : there ? order_key(best * s) : 0u;
      }
    }
  }
  // The W-th largest key, 8 bits at a time from the top; `need` of the keys
  // equal to the prefix so far remain to be taken.
  uint32_t prefix = 0;
  int need = W;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    hist[tid] = 0;  // (256 threads, 256 bins)
    __syncthreads();
    for (int j = tid; j < nblk; j += kSelThreads) {
      const uint32_t k = keys[j];
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    // count of keys in bins above this thread's: suffix sums
    const int bin = 255 - tid;
    int n = (int)hist[bin], sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFullMask, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[0][warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += warp_sum[0][w];
    if (sum >= need && sum - n < need) {
      digit_out[0] = bin;
      digit_out[1] = need - (sum - n);
    }
    __syncthreads();
    prefix |= (uint32_t)digit_out[0] << shift;
    need = digit_out[1];
  }
  // All keys above the prefix, and the first `need` equal to it, in order.
  int taken = 0, ties = 0;
  for (int j0 = 0; j0 < nblk; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t k = j < nblk ? keys[j] : 0u;
    const bool tie = j < nblk && k == prefix;
    const unsigned tb = __ballot_sync(kFullMask, tie);
    __syncthreads();
    if (lane == 0) warp_sum[0][warp] = __popc(tb);
    __syncthreads();
    int tpos = ties + __popc(tb & ((1u << lane) - 1u));
    int all = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) tpos += warp_sum[0][w];
      all += warp_sum[0][w];
    }
    ties += all;
    const bool sel = j < nblk && (k > prefix || (tie && tpos < need));
    const unsigned sb = __ballot_sync(kFullMask, sel);
    if (lane == 0) warp_sum[1][warp] = __popc(sb);
    __syncthreads();
    int spos = taken + __popc(sb & ((1u << lane) - 1u));
    all = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) spos += warp_sum[1][w];
      all += warp_sum[1][w];
    }
    taken += all;
    if (sel) tiles[spos] = tile_of(j);
  }
}

}  // namespace

cudaError_t block_bounds_launch(const BoundsParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  const int JM = 1 + (p.T - 1 + p.bs - 1) / p.bs;
  const long long items = (long long)p.B * JM * p.n_kv;
  const long long grid = (items + kBoundWarps - 1) / kBoundWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 gd((unsigned)grid);
  const int nt = kBoundWarps * 32;
  if (p.k_scales)
    return p.bs == 16 ? launch_pdl(bounds_kernel<16, true>, gd, nt, 0, stream, p, JM)
                      : launch_pdl(bounds_kernel<32, true>, gd, nt, 0, stream, p, JM);
  return p.bs == 16 ? launch_pdl(bounds_kernel<16, false>, gd, nt, 0, stream, p, JM)
                    : launch_pdl(bounds_kernel<32, false>, gd, nt, 0, stream, p, JM);
}

// Blocks of a sequence that the selection holds keys for (192 KiB of them).
int select_max_blocks() { return 49152; }

cudaError_t select_blocks_launch(const SelectParams &p, int G, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  const dim3 grid((unsigned)(p.B * p.n_kv));
  const size_t smem = (size_t)p.MB * 4;
  auto go = [&](auto kernel) {
    if (smem > 40 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(
          kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, select_max_blocks() * 4);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, grid, kSelThreads, smem, stream, p);
  };
  switch (G) {
    case 1: return go(select_kernel<1>);
    case 2: return go(select_kernel<2>);
    case 4: return go(select_kernel<4>);
    case 8: return go(select_kernel<8>);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pgd
