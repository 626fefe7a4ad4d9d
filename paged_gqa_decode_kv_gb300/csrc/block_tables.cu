// block_tables.cu -- block tables, positions and slots of a step built on the
// GPU from the requests' lengths, and cut back.
//
// grow: row b takes need_b = ceil((len + new) / bs) - ceil(len / bs) blocks,
// one more where its last block is partly filled and shared (a private copy in
// its place).  The need is summed over the rows, the free bits are summed over
// the pool's words, and the i-th block needed is the i-th lowest free id: the
// outcome is a function of the state alone, whatever order blocks came back in.
// Every new token gets its slot (block * bs + offset) and its position.
//
// The rows and the pool's bits are a few kilobytes to 128 KiB; what bounds a
// step's call is a chain of dependent loads (length, last entry, its references)
// and barriers.  So one CTA takes three sums (blocks, tokens, free bits) in one
// scan and gives out blocks and slots from shared memory (64 requests: 3.2 us).
// Admissions (many tokens) and large pools take a cluster of CTAs that share
// the blocks to write, and a second launch over all SMs for the
// tokens' slots.  Nothing changes when the blocks do not suffice.
//
// trim: a CTA a row gives back the blocks behind the tokens that it keeps.
// Counts fall by atomics whose order does not matter; the row that takes the
// last reference sets the block's bit.  Many blocks' loads and atomics are in
// flight together, and blocks of one word of the pool's bits, as they are given
// out, go back in one operation (256 prompts grown and cut: 19.4 -> 17.7 us).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "block_tables.cuh"

namespace pgd {
namespace {

namespace cg = cooperative_groups;

// 16 CTAs of 512 threads where there is much to write (256 prompts, 36 thousand blocks
// of a pool of 240 thousand, with the cut behind it, which took 2 us more then: 19.3 us;
// 8 of 1024 21.8, 8 of 512 24.0, 16 of 1024 19.7).
constexpr int kCluster = 16, kClusterThreads = 512;
constexpr int kSlotThreads = 256;
// Up to this many token places, and blocks of a pool, one CTA does everything.
constexpr int kInlineTokens = 8192;
constexpr int kInlineBlocks = 1 << 18;
constexpr int kWords = 4;     // of the pool's bits a thread looks at
constexpr int kIds = 2048;   // new ids that it keeps in shared memory
constexpr int kMost = 1 << 30;  // sums end here: more than any pool or call has

// a, b from 0 to kMost (twice kMost is 2^31: added without a sign).
__device__ __forceinline__ int capped(int a, int b) {
  return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kMost);
}

// Inclusive sums of x over the CTA's NT threads, and the totals.
template <int NT, int N>
__device__ __forceinline__ void block_scan(int (&x)[N], int (*sums)[32], int (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int y = __shfl_up_sync(kFullMask, x[j], i);
      if (lane >= i) x[j] = capped(x[j], y);
    }
  if (lane == 31)
#pragma unroll
    for (int j = 0; j < N; ++j) sums[j][warp] = x[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    int w = lane < NT / 32 ? sums[j][lane] : 0;
#pragma unroll
    for (int i = 1; i < NT / 32; i <<= 1) {
      const int y = __shfl_up_sync(kFullMask, w, i);
      if (lane >= i) w = capped(w, y);
    }
    total[j] = __shfl_sync(kFullMask, w, NT / 32 - 1);
    const int before = __shfl_sync(kFullMask, w, max(warp - 1, 0));
    if (warp) x[j] = capped(x[j], before);
  }
}

// x / bs, rounded down and up (x >= 0): block sizes are powers of two as a rule.
__device__ __forceinline__ int blocks_down(int x, int bs, int lg) { return lg >= 0 ? x >> lg : x / bs; }
__device__ __forceinline__ int blocks_up(long long x, int bs, int lg) {
  return (int)(lg >= 0 ? (x + bs - 1) >> lg : (x + bs - 1) / bs);
}

// The last row whose start is at most n (starts[B] > n).
__device__ __forceinline__ int row_of(const int32_t *starts, int B, int n) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= n) lo = mid; else hi = mid;
  }
  return lo;
}

// Word w of the pool's bits; bits past the pool do not count.
__device__ __forceinline__ uint32_t free_word(const GrowParams &p, int w) {
  const uint32_t bits = p.free_bits[w];
  const int left = p.NB - w * 32;
  return left < 32 ? bits & ((1u << left) - 1u) : bits;
}

// The place of set bit n (from 0) of a word that has more than n.
__device__ __forceinline__ int nth_bit(uint32_t w, int n) {
  int at = 0;
#pragma unroll
  for (int width = 16; width; width >>= 1) {
    const int c = __popc(w & ((1u << width) - 1u));
    if (n >= c) {
      n -= c;
      w >>= width;
      at += width;
    }
  }
  return at;
}

// One CTA of NT threads, or (C > 1) a cluster of C.
template <int NT, int C>
__global__ void __launch_bounds__(NT) grow_tables_kernel(const GrowParams p) {
  extern __shared__ int32_t rows[];
  int32_t *off = rows;                 // [B + 1] blocks taken by the rows before
  int32_t *starts = off + p.B + 1;     // [B + 1] tokens of the rows before
  int32_t *lens = starts + p.B + 1;    // [B] the length, its top bit: last block copied
  int32_t *lasts = lens + p.B;         // [B] the last block (C = 1 and keep_lasts)
  __shared__ int sums[3][32];
  __shared__ int counts[C];            // free blocks of every CTA's share
  __shared__ int ids[C == 1 ? kIds : 1];
  __shared__ int upto[NT];             // a chunk of the pool: free blocks up to
  __shared__ __align__(16) uint32_t chunk[NT][kWords];  // and with a thread's words
  const int tid = threadIdx.x;
  const int rank = C > 1 ? (int)blockIdx.x : 0;
  const bool first = rank == 0;
  const int words = (p.NB - 1) / 32 + 1;
  const int row_per = (p.B + NT - 1) / NT;  // rows a thread, side by side
  // (every CTA of the cluster has started: waited for before the first store into
  // another's shared memory)
  if constexpr (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();

  int x[3] = {0, 0, 0};  // blocks needed, tokens, free blocks
  uint32_t bits[kWords];  // of a chunk of the pool
  if (C == 1) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = tid * kWords + i;
      bits[i] = w < words ? free_word(p, w) : 0u;
      x[2] += __popc(bits[i]);
    }
    for (int w = NT * kWords + tid; w < words; w += NT) x[2] += __popc(free_word(p, w));
  } else {
    for (int w = rank * NT + tid; w < words; w += C * NT)
      x[2] = capped(x[2], __popc(free_word(p, w)));
  }
  const int b0 = tid * row_per;
  for (int b = b0; b < min(p.B, b0 + row_per); ++b) {
    int need = 0, src = -1, last = -1;
    const int len = p.ctx[b];
    int add = p.new_tokens[b];
    if (len < 0 || add < 0 || (long long)len + add > (long long)p.MB * p.bs) {
      if (first) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
      add = 0;
    }
    if (add > 0) {
      const int at = blocks_up(len, p.bs, p.lg_bs);
      need = blocks_up((long long)len + add, p.bs, p.lg_bs) - at;
      if (len != at * (long long)p.bs) {
        last = p.tables[(size_t)b * p.MB + at - 1];
        if ((unsigned)last >= (unsigned)p.NB) {
          if (first) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
          need = add = 0;
        } else if (p.refs[last] > 1) {
          src = last;
          ++need;
        }
      }
    }
    off[b] = need;
    starts[b] = add;
    lens[b] = len & 0x7fffffff;
    if (src >= 0) lens[b] |= (int)0x80000000;
    if (p.keep_lasts) lasts[b] = last;
    if (first) {
      p.positions[b] = len;
      p.copy_src[b] = src;
      p.copy_dst[b] = -1;
    }
    x[0] = capped(x[0], min(need, kMost));
    x[1] = capped(x[1], min(add, kMost));
  }
  const int mine[3] = {x[0], x[1], x[2]};
  int total[3];
  block_scan<NT, 3>(x, sums, total);
  int free_blocks = total[2];
  if constexpr (C > 1) {
    // every CTA learns what the others counted; none changes anything before
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    if (tid < C) *cluster.map_shared_rank(counts + rank, tid) = total[2];
    cluster.sync();
    free_blocks = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) free_blocks = capped(free_blocks, counts[i]);
  }
  const int need = total[0], tokens = total[1];
  const bool fits = tokens <= p.N, done = fits && need <= free_blocks;
  if (first && tid == 0) {
    p.result[0] = done ? 0 : fits ? 1 : 2;
    p.result[1] = done ? need : 0;
    p.result[2] = done || !fits ? 0 : need - free_blocks;
    p.result[3] = done ? tokens : 0;
  }
  if (!done) {
    if (!first) return;
    if (tid == 0 && !fits) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    __syncthreads();
    for (int b = tid; b <= p.B; b += NT) {
      p.starts[b] = 0;
      if (b < p.B) p.copy_src[b] = -1;
    }
    if (C == 1)
      for (int n = tid; n < p.N; n += NT) {
        p.slots[n] = -1;
        p.token_positions[n] = 0;
      }
    return;
  }
  {  // counts to sums of the rows before
    int o = x[0] - mine[0], t = x[1] - mine[1];
    for (int b = b0; b < min(p.B, b0 + row_per); ++b) {
      const int n = off[b], m = starts[b];
      off[b] = o;
      starts[b] = t;
      o += n;
      t += m;
    }
    if (tid == 0) {
      off[p.B] = need;
      starts[p.B] = tokens;
    }
  }
  // (the first chunk of one CTA is summed already)
  if (C == 1 && words <= NT * kWords) {
    upto[tid] = x[2];
    *reinterpret_cast<uint4 *>(chunk[tid]) = make_uint4(bits[0], bits[1], bits[2], bits[3]);
  }
  __syncthreads();

  // The lowest free ids, in the order of the rows, by chunks of the pool that
  // every CTA sums for itself: the i-th free block of a chunk is found by
  // bisection, so that neighbouring threads write neighbouring entries and the
  // CTAs take equal shares wherever in the pool the free blocks lie.
  int before = 0;
  for (int c0 = 0; c0 < words && before < need; c0 += NT * kWords) {
    int n[1] = {0}, all[1] = {total[2]};
    if (C > 1 || c0 > 0)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int w = c0 + tid * kWords + i;
        bits[i] = w < words ? free_word(p, w) : 0u;
      }
#pragma unroll
    for (int i = 0; i < kWords; ++i) n[0] += __popc(bits[i]);
    const int had = n[0];
    if (C > 1 || words > NT * kWords) {
      __syncthreads();  // (the last chunk is done with)
      block_scan<NT, 1>(n, sums, all);
      upto[tid] = n[0];
      *reinterpret_cast<uint4 *>(chunk[tid]) = make_uint4(bits[0], bits[1], bits[2], bits[3]);
      if constexpr (C > 1)
        cg::this_cluster().sync();  // every CTA has read the chunk's bits
      else
        __syncthreads();
    } else {
      n[0] = x[2];
    }
    for (int k = rank * NT + tid; k < min(all[0], need - before); k += C * NT) {
      int lo = 0, hi = NT - 1;  // the first thread with upto > k
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > k) hi = mid; else lo = mid + 1;
      }
      int left = k - (lo ? upto[lo - 1] : 0), word = 0;
#pragma unroll
      for (int i = 0; i < kWords - 1; ++i) {
        const int m = __popc(chunk[lo][i]);
        if (word == i && left >= m) {
          left -= m;
          ++word;
        }
      }
      const int id = (c0 + lo * kWords + word) * 32 + nth_bit(chunk[lo][word], left);
      const int i = before + k, b = row_of(off, p.B, i), at = i - off[b];
      const int len = lens[b] & 0x7fffffff;
      const bool copied = lens[b] < 0;
      const int col = blocks_up(len, p.bs, p.lg_bs) - (copied ? 1 : 0);
      p.tables[(size_t)b * p.MB + col + at] = id;
      p.refs[id] = 1;
      if (C == 1 && i < kIds) ids[i] = id;
      if (at == 0 && copied) p.copy_dst[b] = id;
    }
    // the bits of what was taken: the lowest of this thread's
    int taken = min(had, need - before - (n[0] - had));
    if (taken > 0 && tid % C == rank)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int m = __popc(bits[i]), t = min(m, taken);
        if (t <= 0) continue;
        taken -= t;
        const uint32_t kept = t == m ? 0u : bits[i] & ~((1u << nth_bit(bits[i], t)) - 1u);
        p.free_bits[c0 + tid * kWords + i] = kept;
      }
    before += all[0];
  }
  if constexpr (C > 1) {
    cg::this_cluster().sync();
    if (!first) return;
  } else {
    __syncthreads();
  }
  for (int b = tid; b <= p.B; b += NT) {
    p.starts[b] = starts[b];
    if (b == p.B) break;
    if (starts[b + 1] > starts[b])
      p.ctx[b] = (lens[b] & 0x7fffffff) + (starts[b + 1] - starts[b]);
    if (lens[b] < 0) {
      const int src = p.copy_src[b];
      if (src >= 0 && atomicSub(p.refs + src, 1) == 1)
        atomicOr(p.free_bits + (src >> 5), 1u << (src & 31));
    }
  }
  if constexpr (C == 1)
    for (int n = tid; n < p.N; n += NT) {
      long long slot = -1;
      int pos = 0;
      if (n < tokens) {
        const int b = row_of(starts, p.B, n), len = lens[b] & 0x7fffffff;
        const int col = blocks_up(len, p.bs, p.lg_bs) - (lens[b] < 0 ? 1 : 0);
        pos = len + (n - starts[b]);
        const int j = blocks_down(pos, p.bs, p.lg_bs), i = off[b] + (j - col);
        int id;
        if (j >= col && i < kIds)
          id = ids[i];
        else if (j < col && p.keep_lasts)
          id = lasts[b];
        else
          id = p.tables[(size_t)b * p.MB + j];
        slot = (long long)id * p.bs + (pos - j * p.bs);
      }
      p.slots[n] = slot;
      p.token_positions[n] = pos;
    }
}

// Slots of many tokens: a warp takes 32 times kRun in a row and finds the first
// one's row of the table; the others walk on from there.
constexpr int kRun = 4;
__global__ void __launch_bounds__(kSlotThreads) place_tokens_kernel(const GrowParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int n0 = (blockIdx.x * (kSlotThreads / 32) + (threadIdx.x >> 5)) * 32 * kRun;
  if (n0 >= p.N) return;
  const int total = p.result[3];
  int b = n0 < total ? row_of(p.starts, p.B, n0) : 0;
  int j[kRun], at[kRun], entry[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int n = n0 + 32 * i + (threadIdx.x & 31);
    j[i] = -1;
    at[i] = 0;
    if (n < total) {
      while (p.starts[b + 1] <= n) ++b;
      at[i] = p.positions[b] + (n - p.starts[b]);
      j[i] = blocks_down(at[i], p.bs, p.lg_bs);
      entry[i] = p.tables[(size_t)b * p.MB + j[i]];
    }
  }
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int n = n0 + 32 * i + (threadIdx.x & 31);
    if (n >= p.N) break;
    p.slots[n] = j[i] < 0 ? -1 : (long long)entry[i] * p.bs + (at[i] - j[i] * p.bs);
    p.token_positions[n] = at[i];
  }
}

constexpr int kTrimThreads = 256, kTrimRun = 2;
// Up to so many blocks of a row go back one by one (64 requests grown and cut: 6.35 us,
// the other way 6.6).
constexpr int kFewBlocks = 8;

__global__ void __launch_bounds__(kTrimThreads) trim_tables_kernel(const TrimParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x;
  const int len = p.ctx[b], keep = __ldg(p.keep + b);
  if (len < 0 || (long long)len > (long long)p.MB * p.bs || keep < 0) {
    if (threadIdx.x == 0) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
    return;
  }
  if (keep >= len) return;
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) p.ctx[b] = keep;
  int32_t *row = p.tables + (size_t)b * p.MB;
  // (unsigned: a row may have 2^31 - 1 blocks, of one token, and a place behind the last wraps)
  const uint32_t j0 = (uint32_t)blocks_up(keep, p.bs, p.lg_bs),
                 j1 = (uint32_t)blocks_up(len, p.bs, p.lg_bs);
  if (j1 - j0 <= kFewBlocks) {
    const uint32_t j = j0 + threadIdx.x;
    if (j >= j1) return;
    const int id = row[j];
    row[j] = -1;
    const int had = (unsigned)id < (unsigned)p.NB ? atomicSub(p.refs + id, 1) : 0;
    if (had == 1) {
      atomicOr(p.free_bits + (id >> 5), 1u << (id & 31));
      return;
    }
    if (had > 1) return;
    if ((unsigned)id < (unsigned)p.NB) atomicAdd(p.refs + id, 1);  // not held: as it was
    atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    return;
  }
  for (uint32_t at = j0; at < j1; at += kTrimThreads * kTrimRun) {
    int id[kTrimRun], had[kTrimRun];
#pragma unroll
    for (int i = 0; i < kTrimRun; ++i) {
      const uint32_t j = at + i * kTrimThreads + threadIdx.x;
      id[i] = j < j1 ? row[j] : 0;
    }
#pragma unroll
    for (int i = 0; i < kTrimRun; ++i) {
      const uint32_t j = at + i * kTrimThreads + threadIdx.x;
      had[i] = 2;
      if (j >= j1) continue;
      row[j] = -1;
      if ((unsigned)id[i] < (unsigned)p.NB)
        had[i] = atomicSub(p.refs + id[i], 1);
      else
        atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    }
#pragma unroll
    for (int i = 0; i < kTrimRun; ++i) {
      if (had[i] < 1) {  // not held: as it was
        atomicAdd(p.refs + id[i], 1);
        atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
      }
      // blocks given out together lie together: their bits in one operation a word
      const int word = had[i] == 1 ? id[i] >> 5 : -1;
      if (__ballot_sync(kFullMask, word >= 0) == 0) continue;
      const uint32_t with = __match_any_sync(kFullMask, word);
      const uint32_t bits = __reduce_or_sync(with, 1u << (id[i] & 31));
      if (word >= 0 && (threadIdx.x & 31) == __ffs(with) - 1) atomicOr(p.free_bits + word, bits);
    }
  }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int grid, int threads, size_t smem, int cluster,
                   cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// -1: no power of two.
static int log2_of(int bs) { return (bs & (bs - 1)) ? -1 : __builtin_ctz((unsigned)bs); }

cudaError_t grow_tables_launch(const GrowParams &p_in, cudaStream_t stream) {
  GrowParams p = p_in;
  const bool one = p.N <= kInlineTokens && p.NB <= kInlineBlocks;
  p.keep_lasts = one && p.B <= 8192 ? 1 : 0;
  p.lg_bs = log2_of(p.bs);
  const size_t smem = ((size_t)p.B * (p.keep_lasts ? 4 : 3) + 2) * sizeof(int32_t);
  auto kernel = one ? grow_tables_kernel<512, 1> : grow_tables_kernel<kClusterThreads, kCluster>;
  if (!one) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (smem > 16 * 1024) {  // (more than 48 KB with the static part)
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(((size_t)kMaxGrowRows * 3 + 2) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  if (one) return launch(kernel, 1, 512, smem, 1, stream, p);
  const cudaError_t e = launch(kernel, kCluster, kClusterThreads, smem, kCluster, stream, p);
  if (e != cudaSuccess || p.N == 0) return e;
  const long long per = kSlotThreads * kRun;
  return launch(place_tokens_kernel, (int)((p.N + per - 1) / per), kSlotThreads, 0, 1, stream, p);
}

cudaError_t trim_tables_launch(const TrimParams &p_in, cudaStream_t stream) {
  TrimParams p = p_in;
  if (p.B == 0) return cudaSuccess;
  p.lg_bs = log2_of(p.bs);
  return launch(trim_tables_kernel, p.B, kTrimThreads, 0, 1, stream, p);
}

}  // namespace pgd
