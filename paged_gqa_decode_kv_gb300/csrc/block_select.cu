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
// block wins).  Scores of one query and KV head are held as parts of 2^24 times
// its largest f_h, which keeps them in fp32's range whatever the query's and
// the keys' magnitude: |sum| 2^-24 < 2^-1, f_h / max f_h <= 1, 2^-100 <= s <= 2^122.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "cluster.cuh"
#include "kv_fp8b.cuh"
#include "select_range.cuh"

namespace pgd {
namespace {

constexpr int kBoundWarps = 4;
constexpr int kGridRows = 65535;  // of a launch

// Least (largest) of each of two packed numbers, passing over a NaN beside a
// number: f16 (widened 8-bit codes) or bf16.
template <bool FP8>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (FP8) {
    const __half2 r = __hmin2(*reinterpret_cast<const __half2 *>(&a),
                              *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
  } else {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
  }
}
template <bool FP8>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (FP8) {
    const __half2 r = __hmax2(*reinterpret_cast<const __half2 *>(&a),
                              *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
  } else {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
  }
}
template <bool FP8>
__device__ __forceinline__ float2 widen2(uint32_t a) {
  if constexpr (FP8) return __half22float2(*reinterpret_cast<const __half2 *>(&a));
  return make_float2(bf16lo(a), bf16hi(a));
}

// 16 bytes that this SM reads once, or zeros: past L1, whose lines a long stream
// would only churn.
// (Predicated in the text: a branch around each load would keep the loads of a
// sequence from being in flight together.)
__device__ __forceinline__ uint4 load_once(const uint4 *p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)there));
  return v;
}

// The bounds of one tile by one warp.  Lane l takes slots l % 4 and l % 4 + 4 of
// every 8-token group and the 16-byte chunks l / 4, l / 4 + 8, so that a load
// instruction reads whole 64-byte pieces.  Per chunk it keeps the least and the
// largest k of each dim in the storage's own precision (bf16, or f16 for
// widened codes: exact); the four lanes of a chunk then reduce the least and
// the negated largest by halves: a lane keeps one half of the values and sends
// the other, and ends with the lower bounds (l % 4 < 2) or the negated upper
// bounds of a few dims over all tokens.  Bound by the read of the keys (bf16)
// and by the ALU pipe (8-bit: 80 % busy with conversions and minima): 84k tokens
// of bf16 24.2 us, 115k of 8 bits and 10 heads 34.6.  (One slot a lane, eight lanes a chunk: 25.7 and 43.0, of which
// the minimum of -k instead of the maximum 0.6 and 2.9.)
template <int BS, bool FP8, bool STREAM>
__device__ __forceinline__ void tile_bounds(const BoundsParams &p, size_t tile, int valid,
                                            int lane) {
  constexpr int NT = BS / 4;             // tokens of a lane: its slot of every half group
  constexpr int NC = FP8 ? 1 : 2;        // chunks of a lane
  constexpr int ND2 = FP8 ? 8 : 4;       // pairs of dims in a chunk
  constexpr int NW = ND2 / 2;            // pairs of a chunk that a lane ends with
  constexpr uint32_t kSign = 0x80008000u, kInf = FP8 ? 0x7c007c00u : 0x7f807f80u;
  const int slot = lane & 3, cl = lane >> 2;
  // (chunks of a group are 8 slots x 16 bytes apart, groups follow each other)
  const uint4 *base = reinterpret_cast<const uint4 *>(p.k_cache) +
                      tile * (size_t)(BS * (FP8 ? 8 : 16)) + cl * 8 + slot;
  uint4 x[NT][NC];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint4 *at = base + (i >> 1) * (NC * 64) + c * 64 + (i & 1) * 4;
      const bool there = 4 * i + slot < valid;
      if constexpr (STREAM) {
        x[i][c] = load_once(at, there);
      } else {
        x[i][c] = make_uint4(0, 0, 0, 0);
        if (there) x[i][c] = __ldg(at);
      }
    }
  float scale = 1.f;
  if constexpr (FP8) scale = __ldg(p.k_scales + tile);
  uint32_t out[NC][NW];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t v[2 * ND2];  // least k of the chunk's pairs, then the largest, negated below
#pragma unroll
    for (int k = 0; k < 2 * ND2; ++k) v[k] = k < ND2 ? kInf : kInf | kSign;
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (4 * i + slot < valid) {
        const uint32_t w[4] = {x[i][c].x, x[i][c].y, x[i][c].z, x[i][c].w};
#pragma unroll
        for (int k = 0; k < ND2; ++k) {
          uint32_t y = w[FP8 ? k >> 1 : k];
          if constexpr (FP8) {
            const __half2 h = e4m3x2_to_half2((uint16_t)(y >> ((k & 1) * 16)));
            y = *reinterpret_cast<const uint32_t *>(&h);
          }
          v[k] = min2<FP8>(v[k], y);
          v[ND2 + k] = max2<FP8>(v[ND2 + k], y);
        }
      }
#pragma unroll
    for (int k = ND2; k < 2 * ND2; ++k) v[k] ^= kSign;
#pragma unroll
    for (int m = 2 * ND2, off = 2; off > 0; m >>= 1, off >>= 1) {
      const bool up = (slot & off) != 0;
#pragma unroll
      for (int k = 0; k < m / 2; ++k) {
        const uint32_t keep = up ? v[k + m / 2] : v[k], send = up ? v[k] : v[k + m / 2];
        v[k] = min2<FP8>(keep, __shfl_xor_sync(kFullMask, send, off));
      }
    }
#pragma unroll
    for (int k = 0; k < NW; ++k) out[c][k] = v[k];
  }
  // Largest finite bound, the scale, and this lane's bounds: dims
  // chunk * 2 ND2 + (slot % 2) * 2 NW .. of the lower or upper ones.
  const bool upper = slot >= 2;
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float2 y = widen2<FP8>(out[c][k]);
      const float a0 = fabsf(y.x * scale), a1 = fabsf(y.y * scale);
      amax = fmaxf(amax, fmaxf(a0 < INFINITY ? a0 : 0.f, a1 < INFINITY ? a1 : 0.f));
    }
  amax = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(amax)));
  const int e = scale_exponent_int8(amax);
  const float inv = pow2f(-e);
  signed char *dst = p.bounds + tile * (2 * kHeadDim) + (upper ? kHeadDim : 0) +
                     cl * 2 * ND2 + (slot & 1) * 2 * NW;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t w[NW / 2];
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float2 y = widen2<FP8>(out[c][k]);
      float f[2] = {y.x * scale, y.y * scale};
      if ((k & 1) == 0) w[k / 2] = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (floor of -max is -ceil(max))
        int n = (int)fminf(fmaxf(floorf(f[i] * inv), -127.f), 127.f);
        if (upper) n = -n;
        w[k / 2] |= (uint32_t)(n & 0xff) << (16 * (k & 1) + 8 * i);
      }
    }
    if constexpr (FP8)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t *>(dst + c * 16 * ND2) = w[0];
  }
  if (lane == 0) p.bound_scales[tile] = pow2f(e);
}

// One warp per run of up to 32 blocks of a (sequence, KV head).  STREAM: many
// tiles, read past L1 (20 prompts: 7 % faster; 48 x 8 tiles: 2.6 us, 2.2 through
// it).
template <int BS, bool FP8, bool STREAM>
__global__ void __launch_bounds__(kBoundWarps * 32)
bounds_kernel(const BoundsParams p, int runs, int run) {
  pdl_wait();
  pdl_launch_dependents();
  const int r = (int)blockIdx.x * kBoundWarps + (int)(threadIdx.x >> 5), b = (int)blockIdx.y;
  const int lane = threadIdx.x & 31;
  if (r >= runs * p.n_kv) return;
  const int jrel = r / p.n_kv * run, g = r % p.n_kv;
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
  const int j0 = p0 / BS + jrel, jend = p0 == ctx ? 0 : (ctx + BS - 1) / BS;
  const int n = min(run, jend - j0);
  const int mine = lane < n ? __ldg(p.tables + (size_t)b * p.MB + j0 + lane) : 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int blk = __shfl_sync(kFullMask, mine, i);
    if ((unsigned)blk < (unsigned)p.NB)
      tile_bounds<BS, FP8, STREAM>(p, (size_t)blk * p.n_kv + g, min(BS, ctx - (j0 + i) * BS), lane);
    else if (g == 0 && lane == 0)
      atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
  }
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
// (two CTAs an SM: 256 heads of 256 blocks take 8.5 us, with 512 threads 15.0)
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kLarge[2] = {16, 12};  // clusters past the portable 8

constexpr int kSMs = 152;          // of a GB300
// Dynamic shared memory that leaves an SM room for one CTA.
constexpr size_t kAloneBytes = 120 * 1024;
constexpr int kSliceKeys = 6144;   // keys of a CTA's slice at most (24 KiB)
constexpr int kBins = kRangeBins;
static_assert(kBins == kSelThreads, "a thread takes a bin");

// D += A B, m16n8k16, f16 operands, fp32 accumulation.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One cluster of C CTAs per (sequence, KV head), each CTA a contiguous slice
// of the blocks.
//
// 1. Scores: a [blocks][256] by [256][heads] product of integers.  A warp takes
//    16 blocks: lane (r, t) = (l / 4, l % 4) reads the 16-byte pieces t, t + 4,
//    ... of the bounds of blocks r and r + 8, all eight loads in flight.  The
//    product runs on the warp-level tensor instruction in f16: the byte b + 128
//    zero-extended to 16 bits is the f16 subnormal (b + 128) 2^-24, one byte
//    permutation for two values, and the query's integers are f16 numbers, so
//    each product and each sum (below 2^23, times 2^-24) is exact in fp32; the
//    accumulator starts at -128 sum_i r_hi to take the 128 off.  (Four int8
//    products an instruction on the CUDA cores took 12.8k cycles for 1024
//    blocks, three times the loads.  The operands come from registers, 16 rows
//    at a time from scattered blocks: the shared-memory operands of the
//    fifth-generation instruction would cost a pass through shared memory for
//    an eighth of its N.)
// 2. The least selected score, by 256-way refinement of the range [least,
//    largest] of the unforced keys: every CTA histograms its keys in the
//    range, sends the counts into every CTA's shared memory and, once all have
//    arrived, adds them up and keeps the bin that holds the wanted rank, until
//    the bin is one value or all its keys are wanted.  (Starting from the
//    range rather than from the keys' top byte, which is all but constant for
//    scores of one query, saves a pass and the contention on one bin.)  The
//    same histograms say how many blocks the slices before ours take, so the
//    places to write need no further exchange.
// 3. Every warp counts, then writes, its own part of the slice in order.
// 8 heads of 8192 blocks: 11.6 us, in clusters of 12; 7.8k of its 21k cycles go
// to the scores (29 bytes a cycle and SM; loads further ahead, and prefetches
// to L2, took longer), about 2k to each of three exchanges.  16 x 8 heads of 512
// blocks: 7.8 us, the scores at 5 TB/s.
template <int G, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p, int cluster) {
  const int C = CLUSTER ? cluster : 1;
  extern __shared__ uint32_t ids[];  // a slice: block ids, and behind them the keys
  __shared__ __align__(16) uint32_t hist[kBins];
  // by pass parity, every CTA's
  __shared__ __align__(16) uint16_t all_hist[2][CLUSTER ? kMaxCluster : 1][kBins];
  // (largest ~key and largest key of the unforced ones)
  __shared__ __align__(8) uint32_t all_range[CLUSTER ? kMaxCluster : 1][2];
  __shared__ uint64_t range_bar, hist_bar[2];  // the peers' ranges, counts (by pass parity)
  __shared__ uint32_t range[2];
  __shared__ int warp_cnt[2][kSelWarps];
  __shared__ int found[5];
  __shared__ __align__(16) uint32_t qh[8][kHeadDim / 2];  // rounded queries, f16 pairs
  __shared__ int qe[8];  // exponents of the queries' steps
  __shared__ float qbias[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = (int)blockIdx.x / C, rank = (int)blockIdx.x % C;
  const int b = unit / p.n_kv, g = unit % p.n_kv;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = __ldg(p.ctx + b);
  uint2 raw = make_uint2(0, 0);
  if (warp < G)
    raw = __ldg(reinterpret_cast<const uint2 *>(
                    p.q + ((size_t)b * p.n_q + g * G + warp) * kHeadDim) + lane);
  const int W = p.W;
  int32_t *tiles = p.tiles + (size_t)unit * W;
  const int32_t *row = p.tables + (size_t)b * p.MB;
  const int nthr = C * kSelThreads, me = rank * kSelThreads + tid;
  if (ctx < 1 || ctx > p.MB * p.bs) {
    if (me == 0) {
      if (g == 0) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
      p.lens[unit] = 0;
    }
    for (int i = me; i < W; i += nthr) tiles[i] = -1;
    return;
  }
  const int nblk = (ctx + p.bs - 1) / p.bs;
  if (me == 0) p.lens[unit] = (min(nblk, W) - 1) * p.bs + ctx - (nblk - 1) * p.bs;
  auto tile_of = [&](int blk) { return (unsigned)blk < (unsigned)p.NB ? blk * p.n_kv + g : -1; };
  if (nblk <= W) {  // everything is selected
    for (int i = me; i < W; i += nthr) tiles[i] = i < nblk ? tile_of(__ldg(row + i)) : -1;
    return;
  }
  // (every CTA of the cluster has started and has its barriers: waited for
  // before the first store into another's shared memory)
  if constexpr (CLUSTER) {
    if (tid == 0) {
      mbar_init(&range_bar, 1);
      mbar_init(&hist_bar[0], 1);
      mbar_init(&hist_bar[1], 1);
      mbar_init_fence();
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  const int per = (nblk + C - 1) / C;
  const int jlo = min(nblk, rank * per), n = min(nblk, jlo + per) - jlo;
  uint32_t *keys = ids + per;
  for (int i = tid; i < n; i += kSelThreads) {
    const uint32_t blk = (uint32_t)__ldg(row + jlo + i);
    ids[i] = blk;
  }
  hist[tid] = 0;
  if (tid < 2) range[tid] = 0;
  // The rounded queries: warp h takes head h (heads past G are zero).
  if (warp < 8) {
    float f[4];
    unpack4(raw, f);
    float a = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
    const int e = scale_exponent_int8(fminf(a, 3.3895314e38f));
    const float inv = pow2f(-e);
    int v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = max(-127, min(127, __float2int_rn(f[i] * inv)));
      sum += v[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 h = __floats2half2_rn((float)v[2 * i], (float)v[2 * i + 1]);
      qh[warp][2 * lane + i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    sum = __reduce_add_sync(kFullMask, sum);
    if (lane == 0) {
      qe[warp] = e;
      qbias[warp] = (float)(-128 * sum) * 0x1p-24f;
    }
  }
  __syncthreads();
  {
    // B fragments: head l / 4, the query's dims that meet bytes 64 c + 16 t +
    // 4 w of a block's bounds; the lower bounds (c < 2) take the negative part,
    // the upper the positive part.
    const int r = lane >> 2, t = lane & 3;
    uint32_t bq[2][4][2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) bq[c][w][i] = qh[r][(c * 64 + 16 * t + 4 * w) / 2 + i];
    auto part = [](uint32_t x, bool upper) {
      const __half2 h = *reinterpret_cast<const __half2 *>(&x), zero = __float2half2_rn(0.f);
      const __half2 y = upper ? __hmax2(h, zero) : __hmin2(h, zero);
      return *reinterpret_cast<const uint32_t *>(&y);
    };
    int top = qe[0];  // heads' steps are relative to the largest
#pragma unroll
    for (int h = 1; h < G; ++h) top = max(top, qe[h]);
    const float f0 = pow2f(max(qe[2 * t] - top, -126)), f1 = pow2f(max(qe[2 * t + 1] - top, -126));
    const float b0 = qbias[2 * t], b1 = qbias[2 * t + 1];
    uint32_t kmin = 0xffffffffu, kmax = 0;
    // 16 blocks' bounds and scales; the next ones are loaded before the last
    // ones are used
    struct Rows {
      uint4 x[2][4];
      float s[2];
      bool there[2];
    };
    auto load = [&](int i0, Rows &v) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = i0 + r + 8 * h;
        const uint32_t blk = i < n ? ids[i] : 0xffffffffu;
        v.there[h] = blk < (uint32_t)p.NB;
        v.s[h] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) v.x[h][c] = make_uint4(0, 0, 0, 0);
        if (v.there[h]) {
          const size_t tile = (size_t)blk * p.n_kv + g;
          const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds + tile * (2 * kHeadDim)) + t;
#pragma unroll
          for (int c = 0; c < 4; ++c) v.x[h][c] = __ldg(src + 4 * c);
          v.s[h] = __ldg(p.bound_scales + tile);
        }
      }
    };
    constexpr int kStep = kSelWarps * 16;
    Rows v, next;
    load(warp * 16, next);
#pragma unroll 1
    for (int i0 = warp * 16; i0 < n; i0 += kStep) {
      v = next;
      load(i0 + kStep, next);
      float d[4] = {b0, b1, b0, b1};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t u[2][4] = {{v.x[0][c].x, v.x[0][c].y, v.x[0][c].z, v.x[0][c].w},
                                  {v.x[1][c].x, v.x[1][c].y, v.x[1][c].z, v.x[1][c].w}};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t y0 = u[0][w] ^ 0x80808080u, y1 = u[1][w] ^ 0x80808080u;
          mma16816(d, __byte_perm(y0, 0, 0x4140), __byte_perm(y1, 0, 0x4140),
                   __byte_perm(y0, 0, 0x4342), __byte_perm(y1, 0, 0x4342),
                   part(bq[c & 1][w][0], c >= 2), part(bq[c & 1][w][1], c >= 2));
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float inf = __int_as_float(0x7f800000);
        float best = fmaxf(2 * t < G ? d[2 * h] * f0 : -inf,
                           2 * t + 1 < G ? d[2 * h + 1] * f1 : -inf);
        best = fmaxf(best, __shfl_xor_sync(kFullMask, best, 1));
        best = fmaxf(best, __shfl_xor_sync(kFullMask, best, 2));
        const int i = i0 + r + 8 * h, j = jlo + i;
        if (i < n && t == 0) {
          const bool forced = j < p.keep_first || j >= nblk - p.keep_last;
          // (the maximum: a score that is no number becomes the least)
          const uint32_t score =
              v.there[h] ? score_key(__float_as_uint(fmaxf(best * v.s[h], -3.4028235e38f))) : 0u;
          const uint32_t key = forced ? 0xffffffffu : score;
          if (!forced) {
            kmin = min(kmin, key);
            kmax = max(kmax, key);
          }
          keys[i] = key;
        }
      }
    }
    kmin = __reduce_min_sync(kFullMask, kmin);
    kmax = __reduce_max_sync(kFullMask, kmax);
    if (lane == 0) {
      atomicMax(&range[0], ~kmin);
      atomicMax(&range[1], kmax);
    }
  }
  __syncthreads();
  bool failed = false;  // a wait for the peers gave up: the CTA leaves at its next barrier
  auto sync_failed = [&] {
    if constexpr (CLUSTER) return __syncthreads_or(failed) != 0;
    __syncthreads();
    return false;
  };
  auto gave_up = [&] {
    if (tid == 0) atomicOr(p.err, PGD_DEVERR_TIMEOUT);
    wait_to_leave();
  };
  // `need` of the unforced keys in [lo, hi] remain to be taken, largest first
  // (there are more unforced blocks than that).
  uint32_t lo = range[0], hi = range[1];
  if constexpr (CLUSTER) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0) mbar_arrive_expect_tx(&range_bar, C * 8);
    if (tid < C) send8(all_range[rank], &range_bar, tid, lo, hi);
    failed = !wait_for_peers(&range_bar, 0);
    for (int r = 0; r < C; ++r) {
      lo = max(lo, all_range[r][0]);
      hi = max(hi, all_range[r][1]);
    }
  }
  lo = ~lo;
  int need = W - p.keep_first - p.keep_last;
  bool all = false;  // every key of [lo, hi] is wanted
  // In the slices before ours: forced blocks, unforced keys above hi, and keys
  // in [lo, hi] (read when this is the last range).
  const int forced = min(jlo, p.keep_first) + max(0, jlo - (nblk - p.keep_last));
  int before = forced, inside = jlo - forced;
  for (int pass = 0; pass < kRangePasses && need > 0 && !all && lo != hi; ++pass) {
    const int shift = range_shift(lo, hi);
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = keys[i];
      const int j = jlo + i;
      if (k >= lo && k <= hi && j >= p.keep_first && j < nblk - p.keep_last)
        atomicAdd(&hist[(k - lo) >> shift], 1u);
    }
    if (sync_failed()) return gave_up();
    if constexpr (CLUSTER) {
      // A warp sends all counts to one CTA, in 16 bits (a slice's fit), eight a
      // lane.  (This pass's half of all_hist was last read two passes ago,
      // before the barrier that every CTA has passed since.)
      for (int r = warp; r < C; r += kSelWarps) {
        const uint4 x = *reinterpret_cast<const uint4 *>(&hist[8 * lane]);
        const uint4 y = *reinterpret_cast<const uint4 *>(&hist[8 * lane + 4]);
        send16(&all_hist[pass & 1][rank][8 * lane], &hist_bar[pass & 1], r, x.x | x.y << 16,
               x.z | x.w << 16, y.x | y.y << 16, y.z | y.w << 16);
      }
      if (tid == 0)
        mbar_arrive_expect_tx(&hist_bar[pass & 1], C * (uint32_t)sizeof(all_hist[0][0]));
      failed = !wait_for_peers(&hist_bar[pass & 1], (uint32_t)(pass >> 1) & 1u);
    }
    const int bin = kBins - 1 - tid;
    // (two counts below 2^16: of all slices, and of the ones before ours)
    uint32_t cnt = 0;
    if constexpr (CLUSTER) {
      for (int r = 0; r < C; ++r)
        cnt += all_hist[pass & 1][r][bin] * (r < rank ? 0x10001u : 1u);
    } else {
      cnt = hist[bin];
    }
    uint32_t sum = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFullMask, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_cnt[0][warp] = (int)sum;
    if (sync_failed()) return gave_up();
    hist[bin] = 0;  // (every warp has read and sent it)
    for (int w = 0; w < warp; ++w) sum += (uint32_t)warp_cnt[0][w];
    const uint32_t over = sum - cnt;  // in higher bins
    const int n_over = (int)(over & 0xffffu), n_bin = (int)(cnt & 0xffffu);
    if (n_over < need && n_over + n_bin >= need) {  // this bin holds the need-th largest
      found[0] = bin;
      found[1] = need - n_over;
      found[2] = n_bin;
      found[3] = (int)(over >> 16);
      found[4] = (int)(cnt >> 16);
    }
    __syncthreads();
    need = found[1];
    all = found[2] == need;
    before += found[3];
    inside = found[4];
    narrow_range(lo, hi, (uint32_t)found[0], shift);
  }
  // Above: forced, or a key above hi, or in [lo, hi] where all are wanted.
  // Equal: the rest of [lo, hi], one value, the first `need` of which are taken.
  if (need == 0) {  // (nothing but the forced blocks)
    hi = lo = 0xffffffffu;
    inside = 0;
  }
  if (all) need = 0;
  auto above = [&](int i) {
    const int j = jlo + i;
    if (j < p.keep_first || j >= nblk - p.keep_last) return true;
    return all ? keys[i] >= lo : keys[i] > hi;
  };
  auto equal = [&](int i) {
    const int j = jlo + i;
    return !all && need > 0 && j >= p.keep_first && j < nblk - p.keep_last && keys[i] >= lo &&
           keys[i] <= hi;
  };
  const int pw = (n + kSelWarps - 1) / kSelWarps;
  const int w0 = min(n, warp * pw), w1 = min(n, w0 + pw);
  int n_above = 0, n_equal = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    n_above += __popc(__ballot_sync(kFullMask, in && above(i)));
    n_equal += __popc(__ballot_sync(kFullMask, in && equal(i)));
  }
  if (lane == 0) {
    warp_cnt[0][warp] = n_above;
    warp_cnt[1][warp] = n_equal;
  }
  if (sync_failed()) return gave_up();
  // Next output place, and equal keys still to be taken.
  if (!all) inside = min(inside, need);
  int at = before + inside, left = need - (all ? 0 : inside);
  for (int w = 0; w < warp; ++w) {
    const int take = min(warp_cnt[1][w], left);
    at += warp_cnt[0][w] + take;
    left -= take;
  }
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const bool a = in && above(i), e = in && equal(i);
    const unsigned below = (1u << lane) - 1u;
    const unsigned eb = __ballot_sync(kFullMask, e);
    const bool sel = a || (e && __popc(eb & below) < left);
    const unsigned sb = __ballot_sync(kFullMask, sel);
    const int place = at + __popc(sb & below);
    if (sel && place < W) tiles[place] = tile_of((int)ids[i]);
    at += __popc(sb);
    left -= min(left, __popc(eb));
  }
}

}  // namespace

template <bool FP8>
static cudaError_t bounds_form(const BoundsParams &p, dim3 grid, int runs, int run,
                               cudaStream_t stream) {
  constexpr int nt = kBoundWarps * 32;
  if (p.bs == 16)
    return run > 1 ? launch_pdl(bounds_kernel<16, FP8, true>, grid, nt, 0, stream, p, runs, run)
                   : launch_pdl(bounds_kernel<16, FP8, false>, grid, nt, 0, stream, p, runs, run);
  return run > 1 ? launch_pdl(bounds_kernel<32, FP8, true>, grid, nt, 0, stream, p, runs, run)
                 : launch_pdl(bounds_kernel<32, FP8, false>, grid, nt, 0, stream, p, runs, run);
}

cudaError_t block_bounds_launch(const BoundsParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  // Blocks a warp takes one after another: one for a few (latency), four for
  // many, so that the chain of a warp's first loads (lengths, then block ids)
  // is paid once for four tiles.
  const int JM = most_blocks(p.T, p.bs, p.MB);
  const int run = (long long)p.B * JM * p.n_kv > 16384 ? 4 : 1, runs = (JM + run - 1) / run;
  const long long grid = ((long long)runs * p.n_kv + kBoundWarps - 1) / kBoundWarps;
  if (grid * kBoundWarps > 0x7fffffffLL) return cudaErrorInvalidValue;
  // a grid row a sequence, as many of them as a grid has to a launch
  for (int b = 0; b < p.B; b += kGridRows) {
    BoundsParams part = p;
    part.B = std::min(kGridRows, p.B - b);
    part.tables += (size_t)b * p.MB;
    part.ctx += b;
    if (p.pos) part.pos += b;
    const dim3 gd((unsigned)grid, (unsigned)part.B);
    const cudaError_t e = p.k_scales ? bounds_form<true>(part, gd, runs, run, stream)
                                     : bounds_form<false>(part, gd, runs, run, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Blocks of a sequence that the selection holds keys for.
int select_max_blocks() { return 8 * kSliceKeys; }

// CTAs per (sequence, KV head): as many as fill the GPU once, but no more than
// leave each 128 blocks (fewer are not worth the cluster barriers), and at
// least as many as hold the keys.  Past the portable 8 a cluster takes most of
// a GPC, so only as many as are resident at once (`large`, asked for per
// device) run side by side: 8 heads of 8192 blocks took 13.9 us in clusters of
// 8, 12.7 in 12 and 20.5 in 16, of which 7 fit; 4 heads 14.8 in 8, 11.8 in 16.
static int select_cluster(int units, int MB, const int (&large)[2]) {
  for (int i = 0; i < 2; ++i)
    if (units <= large[i] && units * kLarge[i] <= kSMs && MB >= kLarge[i] * 128) return kLarge[i];
  int C = 1;
  while (C < 8 && units * C * 2 <= kSMs && MB >= C * 2 * 128) C *= 2;
  while (MB > C * kSliceKeys) C *= 2;
  return C;
}

static cudaLaunchAttribute cluster_of(int n) {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)n;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

// A kernel's limits raised on the current device.
template <class Kernel>
static cudaError_t raise_limits(Kernel kernel) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kAloneBytes);
  return e != cudaSuccess
             ? e
             : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <int G>
static cudaError_t launch_select(const SelectParams &p, cudaStream_t stream) {
  // Per device, once: both kernels' limits raised (bit 16), and the large
  // clusters that are resident at once (bits 0-7, 8-15).
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int state = dev >= 0 && dev < 64 ? known[dev].load() : 0;
  if (!state) {
    if ((e = raise_limits(select_kernel<G, true>)) != cudaSuccess) return e;
    if ((e = raise_limits(select_kernel<G, false>)) != cudaSuccess) return e;
    state = 1 << 16;
    for (int i = 0; i < 2; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)kLarge[i]);
      cfg.blockDim = dim3(kSelThreads);
      cfg.dynamicSmemBytes = kAloneBytes;
      cudaLaunchAttribute attr = cluster_of(kLarge[i]);
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, select_kernel<G, true>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      state |= n << (8 * i);
    }
    if (dev >= 0 && dev < 64) known[dev].store(state);
  }
  const int large[2] = {state & 255, state >> 8 & 255};
  const int units = p.B * p.n_kv, C = select_cluster(units, p.MB, large);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kSelThreads);
  // With no more CTAs than SMs each gets an SM to itself: behind an attention
  // call, whose CTAs leave one by one, two would crowd the first SMs to be free
  // (a sparse step of one 131072-token context: 31.5 us crowded, 27.3 apart).
  cfg.dynamicSmemBytes = units * C <= kSMs ? kAloneBytes : (size_t)((p.MB + C - 1) / C) * 8;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1] = cluster_of(C);
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return C > 1 ? cudaLaunchKernelEx(&cfg, select_kernel<G, true>, p, C)
               : cudaLaunchKernelEx(&cfg, select_kernel<G, false>, p, C);
}

cudaError_t select_blocks_launch(const SelectParams &p, int G, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  switch (G) {
    case 1: return launch_select<1>(p, stream);
    case 2: return launch_select<2>(p, stream);
    case 4: return launch_select<4>(p, stream);
    case 8: return launch_select<8>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pgd
