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
// one integer product, exact, for any int32 position.  Its upper 32 bits go to
// sincospi.
//
// Bound by memory: every row read and written once.  A CTA takes 1 or 4 tokens;
// its threads find one (token, pair) angle each, and then stay with 16 dims of
// a head (8 pairs, whose cosines and sines they load once) for every head in
// turn, two 16-byte vectors a head, four heads' loads in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rope.cuh"

namespace pgd {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;  // heads

// A head's row of one token: where from, where to (16-byte vectors).
struct Row {
  const uint4 *src;
  uint4 *dst;
  int step;  // vectors between the row's 16-byte vectors at dst (8 in a tile)
  bool rotated, there;
};

template <bool APPEND>
__device__ __forceinline__ Row row_of(const RopeParams &p, int t, int head, long long slot) {
  Row r;
  r.step = 1;
  r.there = true;
  r.rotated = true;
  if (head < p.n_q) {
    r.src = reinterpret_cast<const uint4 *>(p.q + t * p.q_row + head * p.q_head);
    r.dst = reinterpret_cast<uint4 *>(p.q_out + t * p.qo_row + head * p.qo_head);
    return r;
  }
  int g = head - p.n_q;
  const bool is_v = g >= p.n_kv;
  if (!APPEND) {
    r.there = !is_v;
    r.src = reinterpret_cast<const uint4 *>(p.k + t * p.k_row + g * p.k_head);
    r.dst = reinterpret_cast<uint4 *>(p.k_out + t * p.ko_row + g * p.ko_head);
    return r;
  }
  if (is_v) g -= p.n_kv;
  r.there = g < p.n_kv;
  r.rotated = !is_v;
  r.src = is_v ? reinterpret_cast<const uint4 *>(p.v + t * p.v_row + g * p.v_head)
               : reinterpret_cast<const uint4 *>(p.k + t * p.k_row + g * p.k_head);
  // 16-byte vector v of slot s: core matrix (s / 8, v), row s % 8
  const long long blk = slot / p.bs;
  const int s = (int)(slot % p.bs);
  r.dst = reinterpret_cast<uint4 *>(is_v ? p.v_cache : p.k_cache) +
          (blk * p.n_kv + g) * (long long)(p.bs * 16) + (s >> 3) * 128 + (s & 7);
  r.step = 8;
  return r;
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 z = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&z);
}

// TT tokens a CTA; blockDim (columns of 16 dims, heads at a time).
template <bool APPEND, int TT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  extern __shared__ __align__(16) float2 turn[];  // [TT][rotary / 2] (cos, sin)
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, n = blockDim.x * blockDim.y;
  const int pairs = p.rotary >> 1, t0 = blockIdx.x * TT;
  for (int i = tid; i < TT * pairs; i += n) {
    const int t = t0 + i / pairs, f = i % pairs;
    if (t < p.T) {
      const uint64_t part = (uint64_t)(int64_t)__ldg(p.positions + t) *
                            (uint64_t)__ldg(p.freq + f);
      const float half_turns = (float)(int32_t)(uint32_t)(part >> 32) * 0x1p-31f;
      float s, c;
      sincospif(half_turns, &s, &c);
      turn[i] = make_float2(c * p.factor, s * p.factor);
    }
  }
  __syncthreads();
  // This thread's 16 dims: column x of the rotary part, or of what is copied.
  const int cols = p.rotary >> 4, x = threadIdx.x;
  const bool rotary = x < cols;
  int v0, v1;  // its two vectors of a row
  if (rotary) {
    v0 = (p.first >> 3) + (p.interleaved ? 2 * x : x);
    v1 = (p.first >> 3) + (p.interleaved ? 2 * x + 1 : x + cols);
  } else {
    // the vectors outside the rotary part, two at a time
    const int i = 2 * (x - cols), lead = p.first >> 3;
    v0 = i < lead ? i : i + 2 * cols;
    v1 = i + 1 < lead ? i + 1 : i + 1 + 2 * cols;
  }
  const int heads = p.n_q + (APPEND ? 2 : 1) * p.n_kv;
#pragma unroll 1
  for (int j = 0; j < TT; ++j) {
    const int t = t0 + j;
    if (t >= p.T) break;
    long long slot = 0;
    if (APPEND) {
      slot = __ldg(p.slots + t);
      if (slot < 0) continue;
      if (slot >= (long long)p.NB * p.bs) {
        if (tid == 0) atomicOr(p.err, PGD_DEVERR_BAD_POSITION);
        continue;
      }
    }
    float c[8], s[8];
    if (rotary) {
      const float4 *at = reinterpret_cast<const float4 *>(turn + j * pairs + 8 * x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 y = at[i];
        c[2 * i] = y.x;
        s[2 * i] = y.y;
        c[2 * i + 1] = y.z;
        s[2 * i + 1] = y.w;
      }
    }
#pragma unroll 1
    for (int h0 = threadIdx.y; h0 < heads; h0 += kInFlight * blockDim.y) {
      uint4 a[kInFlight], b[kInFlight];
      Row r[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int h = h0 + i * blockDim.y;
        r[i] = row_of<APPEND>(p, t, h, slot);
        if (h >= heads) r[i].there = false;
        // (in place, what is not rotated is there already)
        if (!rotary && r[i].src == r[i].dst) r[i].there = false;
        if (r[i].there) {
          a[i] = r[i].src[v0];
          b[i] = r[i].src[v1];
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (!r[i].there) continue;
        if (rotary && r[i].rotated) {
          float y[8], z[8];
          unpack8(a[i], y);
          unpack8(b[i], z);
          if (p.interleaved) {
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              const float u = y[k], w = y[k + 1], e = z[k], f = z[k + 1];
              y[k] = u * c[k / 2] - w * s[k / 2];
              y[k + 1] = w * c[k / 2] + u * s[k / 2];
              z[k] = e * c[4 + k / 2] - f * s[4 + k / 2];
              z[k + 1] = f * c[4 + k / 2] + e * s[4 + k / 2];
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float u = y[k], w = z[k];
              y[k] = u * c[k] - w * s[k];
              z[k] = w * c[k] + u * s[k];
            }
          }
          a[i] = make_uint4(pack(y[0], y[1]), pack(y[2], y[3]), pack(y[4], y[5]),
                            pack(y[6], y[7]));
          b[i] = make_uint4(pack(z[0], z[1]), pack(z[2], z[3]), pack(z[4], z[5]),
                            pack(z[6], z[7]));
        }
        r[i].dst[v0 * r[i].step] = a[i];
        r[i].dst[v1 * r[i].step] = b[i];
      }
    }
  }
}

template <bool APPEND, int TT>
cudaError_t launch(const RopeParams &p, cudaStream_t stream) {
  const int cols = p.d >> 4;
  const int heads = p.n_q + (APPEND ? 2 : 1) * p.n_kv;
  int y = kThreads / cols;
  if (y > heads) y = heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + TT - 1) / TT));
  cfg.blockDim = dim3((unsigned)cols, (unsigned)y);
  cfg.dynamicSmemBytes = (size_t)TT * (p.rotary >> 1) * sizeof(float2);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<APPEND, TT>, p);
}

}  // namespace

cudaError_t rope_launch(const RopeParams &p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  const bool many = p.T > 1024;
  if (p.k_cache) return many ? launch<true, 4>(p, stream) : launch<true, 1>(p, stream);
  return many ? launch<false, 4>(p, stream) : launch<false, 1>(p, stream);
}

}  // namespace pgd
