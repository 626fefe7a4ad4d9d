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
// One CTA does the sums and the tables (the rows and the pool's bits are a few
// kilobytes to 128 KiB, and what bounds it is a chain of dependent loads); the
// tokens' slots follow in the same CTA while they are few, else in a second
// launch over all SMs, which finds a token's row by bisection of the starts.
// Nothing changes when the blocks do not suffice.
//
// trim: a warp a row gives back the blocks behind the tokens that it keeps.
// Counts fall by atomics whose order does not matter; the row that takes the
// last reference sets the block's bit.
#include <cuda_runtime.h>

#include "block_tables.cuh"

namespace pgd {
namespace {

constexpr int kGrowThreads = 1024;
constexpr int kGrowWarps = kGrowThreads / 32;
constexpr int kSlotThreads = 256;
// Up to this many token places are written by the CTA that builds the tables.
constexpr int kInlineTokens = 8192;

// Inclusive sum over the CTA, and the total.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *warp_sums, T &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const T y = __shfl_up_sync(kFullMask, x, i);
    if (lane >= i) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  T w = warp_sums[lane];
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const T y = __shfl_up_sync(kFullMask, w, i);
    if (lane >= i) w += y;
  }
  total = __shfl_sync(kFullMask, w, 31);
  if (warp) x += __shfl_sync(kFullMask, w, warp - 1);
  __syncthreads();  // warp_sums is free again
  return x;
}
static_assert(kGrowWarps == 32, "one lane a warp in block_scan");

// The row of token n: the last whose start is at most n (starts[B] > n).
__device__ __forceinline__ int row_of_token(const int32_t *starts, int B, int n) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= n) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void place_token(const GrowParams &p, const int32_t *starts, int n,
                                            int total) {
  long long slot = -1;
  int pos = 0;
  if (n < total) {
    const int b = row_of_token(starts, p.B, n);
    pos = p.positions[b] + (n - starts[b]);
    slot = (long long)p.tables[(size_t)b * p.MB + pos / p.bs] * p.bs + pos % p.bs;
  }
  p.slots[n] = slot;
  p.token_positions[n] = pos;
}

// Word w of the pool's bits; bits past the pool do not count.
__device__ __forceinline__ uint32_t free_word(const GrowParams &p, int w) {
  const uint32_t bits = p.free_bits[w];
  const int left = p.NB - w * 32;
  return left < 32 ? bits & ((1u << left) - 1u) : bits;
}

__global__ void __launch_bounds__(kGrowThreads) grow_tables_kernel(const GrowParams p) {
  extern __shared__ int32_t rows[];
  int32_t *off = rows;                 // [B + 1] blocks taken by the rows before
  int32_t *starts = rows + p.B + 1;    // [B + 1] tokens of the rows before
  int32_t *col = starts + p.B + 1;     // [B] the first table entry that changes
  __shared__ long long sums[kGrowWarps];
  __shared__ int isums[kGrowWarps];
  const int tid = threadIdx.x, words = (p.NB - 1) / 32 + 1;
  pdl_wait();
  pdl_launch_dependents();

  int mine = 0;
  for (int w = tid; w < words; w += kGrowThreads) mine += __popc(free_word(p, w));

  // What every row needs.
  long long blocks = 0, tokens = 0;
  for (int b0 = 0; b0 < p.B; b0 += kGrowThreads) {
    const int b = b0 + tid;
    int need = 0, add = 0, at = 0, src = -1, len = 0;
    if (b < p.B) {
      len = p.ctx[b];
      add = p.new_tokens[b];
      if (len < 0 || add < 0 || (long long)len + add > (long long)p.MB * p.bs) {
        atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
        add = 0;
      }
      if (add > 0) {
        at = (int)(((long long)len + p.bs - 1) / p.bs);
        need = (int)(((long long)len + add + p.bs - 1) / p.bs) - at;
        if (len % p.bs) {
          const int last = p.tables[(size_t)b * p.MB + at - 1];
          if ((unsigned)last >= (unsigned)p.NB) {
            atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
            need = add = 0;
          } else if (p.refs[last] > 1) {
            src = last;
            --at;
            ++need;
          }
        }
      }
    }
    long long n, m;
    const long long e = block_scan<long long>(need, sums, n);
    const long long f = block_scan<long long>(add, sums, m);
    if (b < p.B) {
      // (beyond int32 only where the call is refused below)
      off[b] = (int)(blocks + e - need);
      starts[b] = (int)(tokens + f - add);
      col[b] = at;
      p.positions[b] = len;
      p.copy_src[b] = src;
      p.copy_dst[b] = -1;
    }
    blocks += n;
    tokens += m;
  }
  int free_blocks;
  block_scan<int>(mine, isums, free_blocks);
  const bool fits = tokens <= p.N, done = fits && blocks <= free_blocks;
  if (tid == 0) {
    p.result[0] = done ? 0 : fits ? 1 : 2;
    p.result[1] = done ? (int)blocks : 0;
    p.result[2] = done || !fits ? 0 : (int)min(blocks - free_blocks, 0x7fffffffLL);
    p.result[3] = done ? (int)tokens : 0;
  }
  if (!done) {
    if (tid == 0 && !fits) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
    for (int b = tid; b <= p.B; b += kGrowThreads) {
      p.starts[b] = 0;
      if (b < p.B) p.copy_src[b] = -1;
    }
    if (p.N <= kInlineTokens)
      for (int n = tid; n < p.N; n += kGrowThreads) {
        p.slots[n] = -1;
        p.token_positions[n] = 0;
      }
    return;
  }
  const int need = (int)blocks, total = (int)tokens;
  if (tid == 0) {
    off[p.B] = need;
    starts[p.B] = total;
  }
  __syncthreads();

  // The lowest free ids, in the order of the rows.
  int before = 0;
  for (int w0 = 0; before < need; w0 += kGrowThreads) {
    const int w = w0 + tid;
    const uint32_t bits = w < words ? free_word(p, w) : 0u;
    int n;
    int i = before + block_scan<int>(__popc(bits), isums, n) - __popc(bits);
    before += n;
    if (bits && i < need) {
      int b = row_of_token(off, p.B, i);
      uint32_t left = bits;
      while (left && i < need) {
        while (off[b + 1] <= i) ++b;
        const int id = w * 32 + __ffs(left) - 1;
        left &= left - 1;
        const int k = i - off[b];
        p.tables[(size_t)b * p.MB + col[b] + k] = id;
        p.refs[id] = 1;
        if (k == 0 && p.copy_src[b] >= 0) p.copy_dst[b] = id;
        ++i;
      }
      p.free_bits[w] = left;
    }
  }
  __syncthreads();
  for (int b = tid; b <= p.B; b += kGrowThreads) {
    p.starts[b] = starts[b];
    if (b == p.B) break;
    p.ctx[b] = p.positions[b] + (starts[b + 1] - starts[b]);
    const int src = p.copy_src[b];
    if (src >= 0 && atomicSub(p.refs + src, 1) == 1)
      atomicOr(p.free_bits + (src >> 5), 1u << (src & 31));
  }
  if (p.N <= kInlineTokens)
    for (int n = tid; n < p.N; n += kGrowThreads) place_token(p, starts, n, total);
}

__global__ void __launch_bounds__(kSlotThreads) place_tokens_kernel(const GrowParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int n = blockIdx.x * kSlotThreads + threadIdx.x;
  if (n < p.N) place_token(p, p.starts, n, p.result[3]);
}

__global__ void __launch_bounds__(128) trim_tables_kernel(const TrimParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.B) return;
  const int len = p.ctx[b], keep = __ldg(p.keep + b);
  if (len < 0 || (long long)len > (long long)p.MB * p.bs || keep < 0) {
    if (lane == 0) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
    return;
  }
  if (keep >= len) return;
  int32_t *row = p.tables + (size_t)b * p.MB;
  const int j1 = (int)(((long long)len + p.bs - 1) / p.bs);
  for (int j = (int)(((long long)keep + p.bs - 1) / p.bs) + lane; j < j1; j += 32) {
    const int id = row[j];
    row[j] = -1;
    if ((unsigned)id >= (unsigned)p.NB) {
      atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
      continue;
    }
    const int had = atomicSub(p.refs + id, 1);
    if (had == 1) {
      atomicOr(p.free_bits + (id >> 5), 1u << (id & 31));
    } else if (had < 1) {  // not held: as it was
      atomicAdd(p.refs + id, 1);
      atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
    }
  }
  __syncwarp();
  if (lane == 0) p.ctx[b] = keep;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t stream,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t grow_tables_launch(const GrowParams &p, cudaStream_t stream) {
  const size_t smem = ((size_t)p.B * 3 + 2) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        grow_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)(((size_t)kMaxGrowRows * 3 + 2) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch(grow_tables_kernel, 1, kGrowThreads, smem, stream, p);
  if (e == cudaSuccess && p.N > kInlineTokens)
    e = launch(place_tokens_kernel, (int)(((long long)p.N + kSlotThreads - 1) / kSlotThreads),
               kSlotThreads, 0, stream, p);
  return e;
}

cudaError_t trim_tables_launch(const TrimParams &p, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  return launch(trim_tables_kernel, (p.B + 3) / 4, 128, 0, stream, p);
}

}  // namespace pgd
