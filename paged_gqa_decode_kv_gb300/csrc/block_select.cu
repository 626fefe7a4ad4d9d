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

// Least of each of two packed numbers, passing over a NaN beside a number:
// f16 (widened 8-bit codes) or bf16.
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
__device__ __forceinline__ float2 widen2(uint32_t a) {
  if constexpr (FP8) return __half22float2(*reinterpret_cast<const __half2 *>(&a));
  return make_float2(bf16lo(a), bf16hi(a));
}

// The bounds of one tile by one warp.  Lane l takes slot l % 8 of every 8-token
// group and the 16-byte chunks l / 8, l / 8 + 4, ..., so that a load
// instruction reads 512 contiguous bytes.  Per chunk it keeps the least k and
// the least -k of each dim in the storage's own precision (bf16, or f16 for
// widened codes: exact); the eight lanes of a chunk then reduce them by
// halves: a lane keeps one half of the values and sends the other, and ends
// with the lower bounds (l % 8 < 4) or the negated upper bounds (l % 8 >= 4)
// of a few dims over all tokens.  Bound by the read of the keys.
template <int BS, bool FP8>
__device__ __forceinline__ void tile_bounds(const BoundsParams &p, size_t tile, int valid,
                                            int lane) {
  constexpr int NG = BS / 8;             // 8-token groups
  constexpr int NC = FP8 ? 2 : 4;        // chunks of a lane
  constexpr int ND2 = FP8 ? 8 : 4;       // pairs of dims in a chunk
  constexpr int NW = ND2 / 4;            // pairs of a chunk that a lane ends with
  constexpr uint32_t kSign = 0x80008000u, kInf = FP8 ? 0x7c007c00u : 0x7f807f80u;
  const int slot = lane & 7, cl = lane >> 3;
  // (chunks of a group are 8 slots x 16 bytes apart, groups follow each other)
  const uint4 *base = reinterpret_cast<const uint4 *>(p.k_cache) +
                      tile * (size_t)(BS * (FP8 ? 8 : 16)) + cl * 8 + slot;
  uint4 x[NG][NC];
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      x[i][c] = make_uint4(0, 0, 0, 0);
      if (8 * i + slot < valid) x[i][c] = __ldg(base + i * (NC * 32) + c * 32);
    }
  float scale = 1.f;
  if constexpr (FP8) scale = __ldg(p.k_scales + tile);
  uint32_t out[NC][NW];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t v[2 * ND2];  // least k of the chunk's pairs, then least -k
#pragma unroll
    for (int k = 0; k < 2 * ND2; ++k) v[k] = kInf;
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (8 * i + slot < valid) {
        const uint32_t w[4] = {x[i][c].x, x[i][c].y, x[i][c].z, x[i][c].w};
#pragma unroll
        for (int k = 0; k < ND2; ++k) {
          uint32_t y = w[FP8 ? k >> 1 : k];
          if constexpr (FP8) {
            const __half2 h = e4m3x2_to_half2((uint16_t)(y >> ((k & 1) * 16)));
            y = *reinterpret_cast<const uint32_t *>(&h);
          }
          v[k] = min2<FP8>(v[k], y);
          v[ND2 + k] = min2<FP8>(v[ND2 + k], y ^ kSign);
        }
      }
#pragma unroll
    for (int m = 2 * ND2, off = 4; off > 0; m >>= 1, off >>= 1) {
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
  // chunk * 2 ND2 + (slot % 4) * 2 NW .. of the lower or upper ones.
  const bool upper = slot >= 4;
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
                     cl * 2 * ND2 + (slot & 3) * 2 * NW;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float2 y = widen2<FP8>(out[c][k]);
      float f[2] = {y.x * scale, y.y * scale};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (floor of -max is -ceil(max))
        int n = (int)fminf(fmaxf(floorf(f[i] * inv), -127.f), 127.f);
        if (upper) n = -n;
        w |= (uint32_t)(n & 0xff) << (16 * k + 8 * i);
      }
    }
    if constexpr (FP8)
      *reinterpret_cast<uint32_t *>(dst + c * 8 * ND2) = w;
    else
      *reinterpret_cast<uint16_t *>(dst + c * 8 * ND2) = (uint16_t)w;
  }
  if (lane == 0) p.bound_scales[tile] = pow2f(e);
}

// One warp per run of up to 32 blocks of a (sequence, KV head).
template <int BS, bool FP8>
__global__ void __launch_bounds__(kBoundWarps * 32)
bounds_kernel(const BoundsParams p, int runs, int run) {
  pdl_wait();
  pdl_launch_dependents();
  const long long id = (long long)blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long per_b = (long long)runs * p.n_kv;
  if (id >= per_b * p.B) return;
  const int b = (int)(id / per_b), r = (int)(id % per_b);
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
      tile_bounds<BS, FP8>(p, (size_t)blk * p.n_kv + g, min(BS, ctx - (j0 + i) * BS), lane);
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
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kSliceKeys = 10240;  // keys of a CTA's slice (40 KiB)
constexpr int kUnroll = 4;  // blocks that a group of eight lanes has in flight

// A float's bits as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Barrier over the cluster's CTAs (shared-memory writes before it are visible
// to the peers' reads behind it), or over the one CTA.
__device__ __forceinline__ void sync_all(int C) {
  if (C > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
}
// A word of CTA `rank`'s shared memory, at the place `local` has in ours.
__device__ __forceinline__ uint32_t ld_peer(const uint32_t *local, int rank, int C) {
  if (C == 1) return *local;
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(remote)
               : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// One cluster of C CTAs per (sequence, KV head), each CTA a contiguous slice
// of the blocks.
// 1. Scores.  Eight lanes take a block: lane i holds dims 16 i .. + 15 of both
//    bounds (two 16-byte loads; a block's 256 bytes are two full lines) and of
//    the rounded queries' positive and negative parts, four int8 products an
//    instruction; a group has kUnroll blocks in flight.  The heads' sums are
//    reduced over the eight lanes by halves (a lane keeps one half of the
//    heads and sends the other).
// 2. The least selected score, by 256-way refinement of the range [least,
//    largest] of the unforced keys: every CTA histograms its keys in the
//    range, adds up all CTAs' histograms through distributed shared memory and
//    keeps the bin that holds the wanted rank, until the bin is one value or
//    all its keys are wanted.  (Starting from the range rather than from the
//    keys' top byte, which is all but constant for scores of one query, saves
//    a pass and the contention on one bin.)
// 3. Every warp counts, then writes, its own part of the slice in order.
template <int G>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p, int C) {
  extern __shared__ uint32_t keys[];  // a slice: block ids, then keys
  __shared__ uint32_t hist[3][256];   // a pass adds in one, zeroes the next's and leaves the
                                      // last's to peers that may still be reading it
  __shared__ uint32_t range[2];       // largest of ~key, largest key: unforced ones
  __shared__ uint32_t counts[2];      // this CTA's keys above the least, and equal to it
  __shared__ int warp_cnt[2][kSelWarps];
  __shared__ int found[3];
  __shared__ __align__(16) signed char qpos[G][kHeadDim], qneg[G][kHeadDim];
  __shared__ float qf[G];
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
  const int per = (nblk + C - 1) / C;
  const int jlo = min(nblk, rank * per), n = min(nblk, jlo + per) - jlo;
  for (int i = tid; i < n; i += kSelThreads) keys[i] = (uint32_t)__ldg(row + jlo + i);
  if (tid < 256) hist[0][tid] = 0;
  if (tid < 2) range[tid] = 0;
  // The rounded queries: warp h takes head h.
  if (warp < G) {
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
      const int v = max(-127, min(127, __float2int_rn(f[i] * inv)));
      wp |= (uint32_t)(max(v, 0) & 0xff) << (8 * i);
      wn |= (uint32_t)(min(v, 0) & 0xff) << (8 * i);
    }
    reinterpret_cast<uint32_t *>(qpos[warp])[lane] = wp;
    reinterpret_cast<uint32_t *>(qneg[warp])[lane] = wn;
    if (lane == 0) qf[warp] = pow2f(e);
  }
  __syncthreads();
  {
    const int i8 = lane & 7;
    uint4 qp[G], qn[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      qp[h] = *reinterpret_cast<const uint4 *>(&qpos[h][16 * i8]);
      qn[h] = *reinterpret_cast<const uint4 *>(&qneg[h][16 * i8]);
    }
    // after the reduction by halves lane i8 holds head i8 / (8 / G)
    const float f = qf[i8 / (8 / G)];
    uint32_t kmin = 0xffffffffu, kmax = 0;
    constexpr int kGroups = kSelThreads / 8;
    for (int i0 = 0; i0 < n; i0 += kGroups * kUnroll) {
      uint4 lo[kUnroll], hi[kUnroll];
      float s[kUnroll];
      bool there[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kGroups + (tid >> 3);
        const uint32_t blk = i < n ? keys[i] : 0xffffffffu;
        there[u] = blk < (uint32_t)p.NB;
        lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
        s[u] = 0.f;
        if (there[u]) {
          const size_t tile = (size_t)blk * p.n_kv + g;
          const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds + tile * (2 * kHeadDim));
          lo[u] = __ldg(src + i8);
          hi[u] = __ldg(src + 8 + i8);
          s[u] = __ldg(p.bound_scales + tile);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        int d[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          int x = 0;
          x = __dp4a((int)hi[u].x, (int)qp[h].x, x); x = __dp4a((int)hi[u].y, (int)qp[h].y, x);
          x = __dp4a((int)hi[u].z, (int)qp[h].z, x); x = __dp4a((int)hi[u].w, (int)qp[h].w, x);
          x = __dp4a((int)lo[u].x, (int)qn[h].x, x); x = __dp4a((int)lo[u].y, (int)qn[h].y, x);
          x = __dp4a((int)lo[u].z, (int)qn[h].z, x); x = __dp4a((int)lo[u].w, (int)qn[h].w, x);
          d[h] = x;
        }
        int off = 4;
#pragma unroll
        for (int m = G; m > 1; m >>= 1, off >>= 1) {
          const bool up = (i8 & off) != 0;
#pragma unroll
          for (int h = 0; h < m / 2; ++h) {
            const int keep = up ? d[h + m / 2] : d[h], send = up ? d[h] : d[h + m / 2];
            d[h] = keep + __shfl_xor_sync(kFullMask, send, off);
          }
        }
#pragma unroll
        for (int o = 4 / G; o > 0; o >>= 1) d[0] += __shfl_xor_sync(kFullMask, d[0], o);
        float best = (float)d[0] * f;
#pragma unroll
        for (int o = 4; o > 4 / G && o > 0; o >>= 1)
          best = fmaxf(best, __shfl_xor_sync(kFullMask, best, o));
        const int i = i0 + u * kGroups + (tid >> 3);
        if (i < n) {
          const int j = jlo + i;
          const bool forced = j < p.keep_first || j >= nblk - p.keep_last;
          const uint32_t key = forced ? 0xffffffffu : there[u] ? order_key(best * s[u]) : 0u;
          if (!forced) {
            kmin = min(kmin, key);
            kmax = max(kmax, key);
          }
          if (i8 == 0) keys[i] = key;
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
  sync_all(C);
  // `need` of the unforced keys in [lo, hi] remain to be taken, largest first
  // (there are more unforced blocks than that).
  uint32_t lo = 0, hi = 0;
  for (int r = 0; r < C; ++r) {
    lo = max(lo, ld_peer(&range[0], r, C));
    hi = max(hi, ld_peer(&range[1], r, C));
  }
  lo = ~lo;
  int need = W - p.keep_first - p.keep_last;
  bool all = false;  // every key of [lo, hi] is wanted
  for (int pass = 0; need > 0 && !all && lo != hi; ++pass) {
    uint32_t *h = hist[pass % 3];
    const int shift = max(0, 24 - __clz(hi - lo));
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = keys[i];
      const int j = jlo + i;
      if (k >= lo && k <= hi && j >= p.keep_first && j < nblk - p.keep_last)
        atomicAdd(&h[(k - lo) >> shift], 1u);
    }
    if (tid < 256) hist[(pass + 1) % 3][tid] = 0;
    sync_all(C);
    const int bin = 255 - tid;
    int cnt = 0, sum = 0;
    if (tid < 256) {
      for (int r = 0; r < C; ++r) cnt += (int)ld_peer(&h[bin], r, C);
      sum = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFullMask, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) warp_cnt[0][warp] = sum;
    }
    __syncthreads();
    if (tid < 256) {
      for (int w = 0; w < warp; ++w) sum += warp_cnt[0][w];
      if (sum >= need && sum - cnt < need) {  // this bin holds the need-th largest
        found[0] = bin;
        found[1] = need - (sum - cnt);
        found[2] = cnt;
      }
    }
    __syncthreads();
    need = found[1];
    all = found[2] == need;
    lo += (uint32_t)found[0] << shift;
    hi = min(hi, lo + ((1u << shift) - 1u));
  }
  // Above: forced, or a key above hi, or in [lo, hi] where all are wanted.
  // Equal: the rest of [lo, hi], one value, the first `need` of which are taken.
  if (need == 0) {
    hi = 0xffffffffu;  // (nothing but the forced blocks)
    lo = 0xffffffffu;
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
  __syncthreads();  // (warp_cnt was read by the last pass)
  if (lane == 0) {
    warp_cnt[0][warp] = n_above;
    warp_cnt[1][warp] = n_equal;
  }
  __syncthreads();
  if (tid == 0) {
    int a = 0, e = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      a += warp_cnt[0][w];
      e += warp_cnt[1][w];
    }
    counts[0] = (uint32_t)a;
    counts[1] = (uint32_t)e;
  }
  sync_all(C);
  int at = 0, left = need;  // next output place, equal keys still to be taken
  for (int r = 0; r < rank; ++r) {
    const int a = (int)ld_peer(&counts[0], r, C), e = (int)ld_peer(&counts[1], r, C);
    const int take = min(e, left);
    at += a + take;
    left -= take;
  }
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
    if (sel) tiles[at + __popc(sb & below)] = tile_of(__ldg(row + jlo + i));
    at += __popc(sb);
    left -= min(left, __popc(eb));
  }
  if (C > 1) sync_all(C);  // peers may still be reading this CTA's counts
}

}  // namespace

cudaError_t block_bounds_launch(const BoundsParams &p, cudaStream_t stream) {
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  // Blocks a warp takes one after another: one for a few (latency), four for
  // many, so that the chain of a warp's first loads (lengths, then block ids)
  // is paid once for four tiles.
  const int JM = 1 + (p.T - 1 + p.bs - 1) / p.bs;
  const int run = (long long)p.B * JM * p.n_kv > 16384 ? 4 : 1, runs = (JM + run - 1) / run;
  const long long items = (long long)p.B * runs * p.n_kv;
  const long long grid = (items + kBoundWarps - 1) / kBoundWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 gd((unsigned)grid);
  const int nt = kBoundWarps * 32;
  if (p.k_scales)
    return p.bs == 16 ? launch_pdl(bounds_kernel<16, true>, gd, nt, 0, stream, p, runs, run)
                      : launch_pdl(bounds_kernel<32, true>, gd, nt, 0, stream, p, runs, run);
  return p.bs == 16 ? launch_pdl(bounds_kernel<16, false>, gd, nt, 0, stream, p, runs, run)
                    : launch_pdl(bounds_kernel<32, false>, gd, nt, 0, stream, p, runs, run);
}

// Blocks of a sequence that the selection holds keys for.
int select_max_blocks() { return kMaxCluster * kSliceKeys; }

// CTAs per (sequence, KV head): as many as fill the GPU once, up to 8, but no
// more than leave each 128 blocks (fewer are not worth the cluster barriers),
// and at least as many as hold the keys.  (Clusters of 16 do not all find
// their place at once: 8 heads of 8192 blocks take 29.8 us in clusters of 16,
// 16.5 in 8, 21.5 in 4, 34.5 in 2.)
static int select_cluster(int units, int MB) {
  int C = 1;
  while (C < 8 && units * C * 2 <= 152 && MB >= C * 2 * 128) C *= 2;
  while (MB > C * kSliceKeys) C *= 2;
  return C;
}

cudaError_t select_blocks_launch(const SelectParams &p, int G, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  const int units = p.B * p.n_kv, C = select_cluster(units, p.MB);
  auto go = [&](auto kernel) {
    if (C > 8) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)((p.MB + C - 1) / C) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, C);
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
