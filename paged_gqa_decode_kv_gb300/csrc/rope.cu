// rope.cu -- rotary positions on rows of queries and keys, to rows or with K
// (and V beside it) into the paged bf16 cache.
//
//   (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a),  a = position * f_i
//
// for the pairs i of dims first .. first + rotary - 1: (i, i + rotary / 2) or
// (2 i, 2 i + 1); the other dims are copied.
//
// Angles.  In fp32 position * f loses the place in the circle as positions
// grow (2^-24 of 10^6 radians is 0.06).  Frequencies come as 64-bit fractions
// of a turn, so that position * f wraps modulo 2^64 to the fraction itself:
// one integer product, exact, for any int32 position.  What is left is within
// half a turn, where the fast sine and cosine are off by 2^-21: 2^12 times less
// than the rounding to bf16 that follows.
//
// Bound by memory: every row read and written once.  A thread takes 16 dims (8
// pairs) of one token, finds their cosines and sines itself and stays with them
// for head after head, two 16-byte vectors a head, four heads' loads in flight:
// no barrier, and nothing shared.  Few tokens' heads are spread over several
// threads.  (A kernel of its own for K and V whose stores were whole lines of the
// tiles, 8 tokens by 4 columns a warp, read its rows in pieces and was slower: 138
// against 129 us for 32 thousand tokens of 48 heads.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rope.cuh"

namespace pgd {
namespace {

constexpr int kThreads = 128;
constexpr int kInFlight = 4;  // heads
// Heads of a thread where tokens are many.  To rows 16 (43 thousand tokens of 40
// heads: 157.8 us, eight 164, all 159.8), into the cache eight (32 thousand tokens of
// 48: 128.8 at slots side by side, 16 134.0; 188.9 at slots anywhere, where every
// 16 bytes are a sector of their own, 16 219.2).
template <bool APPEND>
constexpr int kManyHeads = APPEND ? 8 : 16;

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 z = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&z);
}

// Cosines and sines of a thread's pairs; where its vectors lie in a row.
struct Pairs {
  float c[8], s[8];
  int v0, v1;
  bool rotary, known;  // known: c and s are found
};

// The angles of pairs 8 x .. 8 x + 7 of a token.
__device__ __forceinline__ void find_angles(const RopeParams &p, long long t, int x, Pairs &r) {
  const uint64_t pos = (uint64_t)(int64_t)__ldg(p.positions + t);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t part = pos * (uint64_t)__ldg(p.freq + 8 * x + i);
    const float half_turns = (float)(int32_t)(uint32_t)(part >> 32) * 0x1p-31f;
    float s, c;
    __sincosf(half_turns * 3.14159265358979f, &s, &c);
    r.c[i] = c * p.factor;
    r.s[i] = s * p.factor;
  }
}

template <bool INTERLEAVED>
__device__ __forceinline__ void turn(const Pairs &r, uint4 &a, uint4 &b) {
  float y[8], z[8];
  unpack8(a, y);
  unpack8(b, z);
  if (INTERLEAVED) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float u = y[k], w = y[k + 1], e = z[k], f = z[k + 1];
      y[k] = u * r.c[k / 2] - w * r.s[k / 2];
      y[k + 1] = w * r.c[k / 2] + u * r.s[k / 2];
      z[k] = e * r.c[4 + k / 2] - f * r.s[4 + k / 2];
      z[k + 1] = f * r.c[4 + k / 2] + e * r.s[4 + k / 2];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float u = y[k], w = z[k];
      y[k] = u * r.c[k] - w * r.s[k];
      z[k] = w * r.c[k] + u * r.s[k];
    }
  }
  a = make_uint4(pack(y[0], y[1]), pack(y[2], y[3]), pack(y[4], y[5]), pack(y[6], y[7]));
  b = make_uint4(pack(z[0], z[1]), pack(z[2], z[3]), pack(z[4], z[5]), pack(z[6], z[7]));
}

// n heads' rows from src to dst (16-byte vectors; `from` and `to` between
// heads, `step` between a row's vectors at dst).
template <bool INTERLEAVED>
__device__ __forceinline__ void rows(const RopeParams &p, long long t, Pairs &r, bool rotated,
                                     const uint4 *src, long long from, uint4 *dst, long long to,
                                     int step, int n) {
  if (!r.rotary && src == dst && from == to) return;  // in place: there already
  const int w0 = r.v0 * step, w1 = r.v1 * step;
#pragma unroll 1
  for (int h = 0; h < n; h += kInFlight) {
    uint4 a[kInFlight], b[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
      if (h + i < n) {
        a[i] = __ldcs(src + i * from + r.v0);
        b[i] = __ldcs(src + i * from + r.v1);
      }
    if (rotated && r.rotary && !r.known) {  // (beside the first loads)
      find_angles(p, t, threadIdx.x, r);
      r.known = true;
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
      if (h + i < n) {
        if (rotated && r.rotary) turn<INTERLEAVED>(r, a[i], b[i]);
        dst[i * to + w0] = a[i];
        dst[i * to + w1] = b[i];
      }
    src += kInFlight * from;
    dst += kInFlight * to;
  }
}

// Threads (columns of 16 dims, tokens); blockIdx.y: `share` heads of a token's.
template <bool APPEND, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int share) {
  pdl_wait();
  pdl_launch_dependents();
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.T) return;
  long long slot = 0;
  if (APPEND) {
    slot = __ldg(p.slots + t);
    if (slot < 0) return;
    if (slot >= (long long)p.NB * p.bs) {
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
      return;
    }
  }
  const int cols = p.rotary >> 4, x = threadIdx.x, lead = p.first >> 3;
  Pairs r;
  r.known = false;
  r.rotary = x < cols;
  if (r.rotary) {
    r.v0 = lead + (INTERLEAVED ? 2 * x : x);
    r.v1 = lead + (INTERLEAVED ? 2 * x + 1 : x + cols);
  } else {
    // the vectors outside the rotary part, two at a time
    const int i = 2 * (x - cols);
    r.v0 = i < lead ? i : i + 2 * cols;
    r.v1 = i + 1 < lead ? i + 1 : i + 1 + 2 * cols;
  }
  // heads [h0, h1) of q's, then k's, then (appended) v's
  const int h0 = blockIdx.y * share;
  const int h1 = min(h0 + share, p.n_q + (APPEND ? 2 : 1) * p.n_kv);
  if (h0 < p.n_q)
    rows<INTERLEAVED>(p, t, r, true,
                      reinterpret_cast<const uint4 *>(p.q + t * p.q_row + h0 * p.q_head),
                      p.q_head >> 3,
                      reinterpret_cast<uint4 *>(p.q_out + t * p.qo_row + h0 * p.qo_head),
                      p.qo_head >> 3, 1, min(h1, p.n_q) - h0);
  const int k0 = max(h0 - p.n_q, 0), k1 = min(h1 - p.n_q, p.n_kv);
  if (!APPEND) {
    if (k0 < k1)
      rows<INTERLEAVED>(p, t, r, true,
                        reinterpret_cast<const uint4 *>(p.k + t * p.k_row + k0 * p.k_head),
                        p.k_head >> 3,
                        reinterpret_cast<uint4 *>(p.k_out + t * p.ko_row + k0 * p.ko_head),
                        p.ko_head >> 3, 1, k1 - k0);
    return;
  }
  // 16-byte vector v of slot s of a tile: core matrix (s / 8, v), row s % 8
  const int lg_bs = p.bs == 32 ? 5 : 4;  // (blocks of 16 or 32)
  const long long blk = slot >> lg_bs;
  const int s = (int)slot & (p.bs - 1);
  const long long tile = p.bs * 16LL, at = (s >> 3) * 128 + (s & 7);
  if (k0 < k1)
    rows<INTERLEAVED>(p, t, r, true,
                      reinterpret_cast<const uint4 *>(p.k + t * p.k_row + k0 * p.k_head),
                      p.k_head >> 3,
                      reinterpret_cast<uint4 *>(p.k_cache) + (blk * p.n_kv + k0) * tile + at, tile,
                      8, k1 - k0);
  const int v0 = max(h0 - p.n_q - p.n_kv, 0), v1 = h1 - p.n_q - p.n_kv;
  if (v0 < v1)
    rows<INTERLEAVED>(p, t, r, false,
                      reinterpret_cast<const uint4 *>(p.v + t * p.v_row + v0 * p.v_head),
                      p.v_head >> 3,
                      reinterpret_cast<uint4 *>(p.v_cache) + (blk * p.n_kv + v0) * tile + at, tile,
                      8, v1 - v0);
}

template <bool APPEND, bool INTERLEAVED>
cudaError_t launch(const RopeParams &p, int sms, cudaStream_t stream) {
  const int cols = p.d >> 4, heads = p.n_q + (APPEND ? 2 : 1) * p.n_kv;
  const int y = std::max(1, std::min(kThreads / cols, p.T));
  const long long tiles = ((long long)p.T + y - 1) / y, threads = tiles * y * cols;
  // kManyHeads a thread where that makes four times the threads that are resident at
  // once, else as many threads as twice those (15 thousand tokens of 90 heads to rows:
  // 107 us, every thread all of them 112; 600 tokens of 72: 5.4 and, 16 a thread, 8.4)
  const long long want = std::max(1LL, (sms * 1024LL + threads - 1) / threads);
  constexpr int kMany = kManyHeads<APPEND>;
  const int share =
      threads * heads / kMany >= sms * 512LL * 4 ? kMany : (int)((heads + want - 1) / want);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)((heads + share - 1) / share));
  cfg.blockDim = dim3((unsigned)cols, (unsigned)y);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<APPEND, INTERLEAVED>, p, share);
}

}  // namespace

cudaError_t rope_launch(const RopeParams &p, int sms, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  if (p.k_cache)
    return p.interleaved ? launch<true, true>(p, sms, stream) : launch<true, false>(p, sms, stream);
  return p.interleaved ? launch<false, true>(p, sms, stream) : launch<false, false>(p, sms, stream);
}

}  // namespace pgd
