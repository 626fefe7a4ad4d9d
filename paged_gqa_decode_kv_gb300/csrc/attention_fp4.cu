// attention_fp4.cu -- paged GQA decode attention over the 4-bit cache
// (kv_fp4.cuh).
//
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k_t) v_t,  t < ctx[b],
//   k_t, v_t = E2M1(code) * E4M3(scale of 16 dims) * (the call's scale)
//
// Arithmetic.  A product of a code and its scale has 6 significant bits and is
// exact in f16, so both contractions run on f16 operands with fp32
// accumulators, S^T = K Q^T and O^T = V^T P^T, 16 tokens (resp. 16 dims) by 8
// query heads.  A query is scaled by a power of two so that its largest element
// lies in [2^14, 2^15): f16 then holds every element to its last bf16 bit, or
// to 2^-39 of the largest.  A weight is 2^7 times 2^(score - reference), the
// reference moving when a score exceeds it by 2^8 (so it stays below f16's
// largest): rounded by 2^-11 of itself, and by 2^-32 of the largest where it
// is that small.  Scores, sums and outputs are fp32.
//
// Why operands in registers.  A scale of its own per token and 16 dims is not
// one that the tensor cores could apply between products, so codes have to be
// expanded.  The warp-level instruction takes them from the registers that the
// conversion leaves them in; for tcgen05 they would go back to shared or
// tensor memory, four times the bytes that came, and with at most 8 query
// heads to a KV head its rate is not needed: the expansion is what costs.
// Both layouts are made for it: every lane loads 16 bytes of codes whose
// expansion is its part of the operands of eight products.
//
// Copies.  Each warp has a ring of its own of 32-token steps, filled by
// 16-byte asynchronous copies and waited for by that warp alone: no barrier
// and no wait on another warp while a context is read.  (Bulk copies of whole
// tiles on barriers of the warp took 224 us where these took 213 on 64 ragged
// contexts with eight heads.)
//
// Split.  A unit (sequence, KV head) is cut into parts of nearly equal size, of
// at most the total over a number of CTAs that goes by the SMs: one part a CTA,
// four CTAs an SM side by side and the rest as those finish, so that one's start
// and end lie beside another's stream.  A CTA's warps take its steps in turn and
// merge their states in shared memory; parts of a unit go through the
// workspace, merged by the CTA that finishes last, in the order of the parts.
// Few units of long contexts take CTAs of 16 warps and one an SM: fewer parts to
// merge.  Where tables are short a unit has a CTA or a cluster of its own
// (shape_of).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "cluster.cuh"
#include "kv_fp4.cuh"

namespace pgd {
namespace {

constexpr int kStepTokens = 32;
constexpr int kStepBytes = 2 * 2 * kGroupBytes4;  // K and V of two groups
constexpr int kStages = 3;
constexpr int kHeads = 8;              // query heads a product takes
constexpr int kMergeRow = kHeadDim + 4;  // floats between heads when states are merged
// Units of no more steps than this are not cut: a part's way through the workspace
// takes longer than three steps of a warp (4 contexts of 217 tokens: 4.1 us whole,
// 5.8 in two parts; a step a warp of 16: 512 tokens of a wide table 5.4, 6.7 in two).
template <int W>
constexpr int kWholeSteps = W == 16 ? 16 : 12;
// Steps a warp from which three CTAs follow one another: fewer where the units are so
// many that one wave cannot be cut evenly (512 units of 1 to 8000 tokens: 60 us, from
// 40 steps 87; but 256 of 8192: 64 and 58), and none up to a unit for every fourth
// CTA (80 of 1 to 80000: 87, in one wave 78; 128 of 1 to 60000: 101 and 97, of 32768
// all: 103 and 105; but 256 of 1 to 40000: 111 and 150).
constexpr int kManySteps = 40, kManyUnits = 25;
constexpr float kMoveLog2 = 8.f;       // move the reference when exceeded by 2^8
constexpr float kUnitLog2 = 7.f;       // a weight of the reference is 2^7

// CTAs an SM: 16 warps with a ring each, as many as shared memory holds.
template <int W>
constexpr int kResident = 16 / W;
template <int W>
constexpr int ring_bytes() {
  return W * kStages * kStepBytes;
}
template <int W>
constexpr size_t smem_bytes() {
  return (size_t)ring_bytes<W>() + W * kHeads * 8 + 16;
}
static_assert(kHeads * kMergeRow * 4 <= kStages * kStepBytes, "a warp's state fits its ring");

// 16 bytes; read once, so the first to leave L2.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t times(uint32_t a, __half2 s) {
  return half2_bits(__hmul2(bits_half2(a), s));
}

// Steps of a sequence's units (0: a bad context).
__device__ __forceinline__ int unit_steps(const AttnParams &a, int BS, int b, int &ctx, bool tell) {
  ctx = __ldg(a.ctx + b);
  if (ctx < 1 || ctx > a.MB * BS) {
    if (tell) atomicOr(a.err, PGD_DEVERR_BAD_CONTEXT);
    return 0;
  }
  return (ctx - 1) / kStepTokens + 1;
}

// What a CTA does: steps [i0, i1) of a unit, which is one of its `parts` parts.
struct Part {
  bool some;
  int b, h, ctx, steps, parts;
  int i0, i1;
  int first;   // the CTA of (part 0, head 0) of this sequence
};

// How units are cut: into parts of at most `size` steps (to a millionth: every
// CTA computes the same, and never more than ceil(steps / size)), or into a given
// number.
template <int W>
struct Cut {
  int splits;
  float inverse;  // of the size, and 2^-20 less
  __device__ __forceinline__ int parts(int steps) const {
    if (splits) return min(splits, steps);
    if (steps <= kWholeSteps<W>) return steps > 0 ? 1 : 0;
    return max(1, (int)ceilf((float)steps * inverse));
  }
};
// The sizes to try, the smallest first, for `all` steps, and the most parts that
// there should be: as many as CTAs are resident at once, or three times as many
// where a CTA has much to do.  Rounding makes them more, by half a part a unit where
// lengths differ, by one at most: the next sizes are for half the units fewer and
// for all the units fewer, which is never too many.  (64 contexts of 128 to 32768
// tokens, 512 units: 203.9 us with the first size alone, 200.4; 256 of 1 to 8000: 39.1
// and 33.0.)  Three waves of very many units keep the first: 1024 of 1 to 8000
// tokens 114.3, with half of them fewer 116.5.
constexpr int kSizes = 3;
template <int W>
__device__ __forceinline__ Cut<W> choose_cut(const Attn4Params &p, int all, int k, int &limit) {
  const float x = (float)all;
  const int units = p.a.B * p.a.n_kv;
  limit = p.resident;
  float size = ceilf(x * p.inv_resident);
  const bool waves = p.uneven && size >= (float)(W * (2 * units > limit ? kManyUnits : kManySteps));
  if (waves) {
    limit *= 3;
    size = ceilf(size * (1.f / 3.f));
  }
  if (k > 0) {
    const int less = k == 1 || waves ? units / 2 : units;
    if (!waves || 2 * units <= limit)
      size = units < p.resident || waves ? ceilf(__fdividef(x, (float)(limit - less))) : x;
  }
  return {p.splits, __frcp_rn(fmaxf(size, (float)p.least_steps)) * (1.f - 0x1p-20f)};
}

__device__ __forceinline__ int inclusive_sum(int x, int lane) {
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(kFullMask, x, i);
    if (lane >= i) x += y;
  }
  return x;
}

// The sequence of CTA blockIdx.x's part, found by every warp for itself: a lane
// looks at R sequences.  False: there is none.
template <int R, int W>
__device__ __forceinline__ bool find_in_lanes(const Attn4Params &p, int BS, Part &r) {
  const AttnParams &a = p.a;
  const int lane = threadIdx.x & 31, cta = blockIdx.x;
  int ctx[R], steps[R], n[R], sum = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    ctx[i] = steps[i] = 0;
    if (lane * R + i < a.B) steps[i] = unit_steps(a, BS, lane * R + i, ctx[i], cta == 0);
    sum += steps[i];
  }
  const int all = __reduce_add_sync(kFullMask, sum) * a.n_kv;
  int mine, limit;
#pragma unroll 1
  for (int k = 0; k < kSizes; ++k) {
    const Cut<W> cut = choose_cut<W>(p, all, k, limit);
    mine = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) mine += n[i] = cut.parts(steps[i]);
    if (p.splits || __reduce_add_sync(kFullMask, mine) * a.n_kv <= limit) break;
  }
  const int upto = inclusive_sum(mine, lane) * a.n_kv;
  int at = upto - mine * a.n_kv;
  const uint32_t hit = __ballot_sync(kFullMask, at <= cta && cta < upto);
  if (!hit) return false;
  const int from = __ffs(hit) - 1;
  // (which of the lane's R it is matters in that lane alone)
  int pick = 0;
#pragma unroll
  for (int i = 0; i + 1 < R; ++i)
    if (pick == i && cta >= at + n[i] * a.n_kv) {
      at += n[i] * a.n_kv;
      ++pick;
    }
#pragma unroll
  for (int i = 1; i < R; ++i)
    if (pick == i) {
      ctx[0] = ctx[i];
      steps[0] = steps[i];
      n[0] = n[i];
    }
  r.b = from * R + __shfl_sync(kFullMask, pick, from);
  r.ctx = __shfl_sync(kFullMask, ctx[0], from);
  r.steps = __shfl_sync(kFullMask, steps[0], from);
  r.parts = __shfl_sync(kFullMask, n[0], from);
  r.first = __shfl_sync(kFullMask, at, from);
  return true;
}

// Finds CTA blockIdx.x's part.  Called by every thread: up to 128 sequences are
// looked at by every warp in its lanes, without a barrier; more by all threads, a
// run each.
template <int W>
__device__ __forceinline__ Part find_part(const Attn4Params &p, int BS) {
  __shared__ int sums[2][W], got[6];
  const AttnParams &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x;
  Part r;
  if (a.B <= 128) {
    r.some = a.B <= 32 ? find_in_lanes<1, W>(p, BS, r) : find_in_lanes<4, W>(p, BS, r);
    if (!r.some) return r;
  } else {
    const int run = (a.B + 32 * W - 1) / (32 * W);
    const int b0 = threadIdx.x * run, b1 = min(a.B, b0 + run);
    int ctx, sum = 0;
    for (int b = b0; b < b1; ++b) sum += unit_steps(a, BS, b, ctx, cta == 0);
    sum = __reduce_add_sync(kFullMask, sum);
    if (lane == 0) sums[0][warp] = sum;
    if (threadIdx.x == 0) got[5] = 0;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) all += sums[0][i];
    Cut<W> cut;
    int at, end, limit;
#pragma unroll 1
    for (int k = 0; k < kSizes; ++k) {
      cut = choose_cut<W>(p, all * a.n_kv, k, limit);
      int n = 0;
      for (int b = b0; b < b1; ++b) n += cut.parts(unit_steps(a, BS, b, ctx, cta == 0));
      const int upto = inclusive_sum(n, lane);
      int *const of_warps = sums[(k + 1) & 1];  // (the other is still being read)
      if (lane == 31) of_warps[warp] = upto;
      __syncthreads();
      int before = 0, total = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        total += of_warps[i];
        if (i < warp) before += of_warps[i];
      }
      end = (before + upto) * a.n_kv;
      at = end - n * a.n_kv;
      if (p.splits || total * a.n_kv <= limit) break;
    }
    if (at <= cta && cta < end)  // (one thread at most)
      for (int b = b0; b < b1; ++b) {
        const int steps = unit_steps(a, BS, b, ctx, cta == 0);
        const int parts = cut.parts(steps);
        end = at + parts * a.n_kv;
        if (cta < end) {
          got[0] = b;
          got[1] = ctx;
          got[2] = steps;
          got[3] = parts;
          got[4] = at;
          got[5] = 1;
          break;
        }
        at = end;
      }
    __syncthreads();
    r.some = got[5];
    if (!r.some) return r;
    r.b = got[0];
    r.ctx = got[1];
    r.steps = got[2];
    r.parts = got[3];
    r.first = got[4];
  }
  int part = 0;
  r.h = cta - r.first;
  if (r.parts > 1) {
    part = r.h / a.n_kv;
    r.h -= part * a.n_kv;
    const int q = r.steps / r.parts, left = r.steps - q * r.parts;
    r.i0 = part * q + min(part, left);
    r.i1 = r.i0 + q + (part < left ? 1 : 0);
  } else {
    r.i0 = 0;
    r.i1 = r.steps;
  }
  return r;
}

template <int BS, int W>
struct Worker {
  const Attn4Params &p;
  int lane, g, t4, warp;
  unsigned char *ring;  // this warp's
  uint32_t ring_at, rest_at;  // as shared addresses: its start, this lane's last piece
  uint64_t policy;
  const unsigned char *from_k, *from_v;  // the head's tile of block 0, this lane's first piece

  // Fragments and state.
  uint32_t qf[16];
  float f0, f1;      // factors of the products of heads 2 t4, 2 t4 + 1 (scores in log2)
  float m0, m1;      // references, as products
  float limit0, limit1;  // products at which they move
  float l0, l1;      // this lane's part of the sums
  float o[8][4];     // dims 16 i + g (+ 8) of those two heads
  uint32_t pf[2][2]; // weights of a step's tokens as operands

  __device__ __forceinline__ Worker(const Attn4Params &p_, unsigned char *smem) : p(p_) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    g = lane >> 2;
    t4 = lane & 3;
    ring = smem + warp * kStages * kStepBytes;
    ring_at = smem_addr(ring);
    rest_at = ring_at + (lane >> 3) * kGroupBytes4 + 1024 + (lane & 7) * 16;
    policy = l2_policy_evict_first();
  }

  // The query's loads: lane (g, t4) holds dims 32 t4 .. + 31 of head g.
  __device__ __forceinline__ void fetch_query(int b, int h, int G, uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (g < G)
        v[i] = __ldg(reinterpret_cast<const uint4 *>(
                         p.a.q + ((size_t)b * p.a.n_q + (size_t)h * G + g) * kHeadDim + 32 * t4) +
                     i);
    }
  }
  // As operand registers, in the order in which K's codes lie; the state of a
  // unit without tokens.
  __device__ __forceinline__ void start(const uint4 (&v)[4]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top = __vmaxu2(top, v[i].x & 0x7fff7fffu);
      top = __vmaxu2(top, v[i].y & 0x7fff7fffu);
      top = __vmaxu2(top, v[i].z & 0x7fff7fffu);
      top = __vmaxu2(top, v[i].w & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(kFullMask, top, 1));
    top = max(top, __shfl_xor_sync(kFullMask, top, 2));
    // the largest lies in [2^e, 2^(e + 1)); a query of next to nothing keeps 2^-100
    const int e = max((int)(top >> 7) - 127, -100);
    const float up = pow2f(14 - e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      unpack8(v[i], x);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        qf[4 * i + j] = half2_bits(__floats2half2_rn(x[2 * j] * up, x[2 * j + 1] * up));
    }
    // (never 0, which would make a masked score of minus infinity NaN, nor infinite,
    // which would a distance of 0)
    const float back = fminf(fmaxf(p.a.qk_scale_log2 * pow2f(e - 14), 0x1p-126f), 0x1p127f);
    f0 = __shfl_sync(kFullMask, back, 8 * t4);
    f1 = __shfl_sync(kFullMask, back, 8 * t4 + 4);
    m0 = m1 = limit0 = limit1 = __uint_as_float(0xff800000u);
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  }

  // Starts the copies of a step from its blocks' ids: of each of its four groups
  // (72 pieces of 16 bytes) two pieces a lane, and the last eight of all in one.
  __device__ __forceinline__ void load_step(int slot, int id0, int id1) {
    const uint32_t dst = ring_at + slot * kStepBytes + lane * 16;
    const uint32_t block = (uint32_t)p.a.n_kv * (BS / kGroupTokens4 * kGroupBytes4);
    const unsigned char *src[4];
    src[0] = from_k + (uint64_t)(uint32_t)id0 * block;
    src[2] = from_v + (uint64_t)(uint32_t)id0 * block;
    src[1] = BS == 32 ? src[0] + kGroupBytes4 : from_k + (uint64_t)(uint32_t)id1 * block;
    src[3] = BS == 32 ? src[2] + kGroupBytes4 : from_v + (uint64_t)(uint32_t)id1 * block;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      copy16(dst + i * kGroupBytes4, src[i], policy);
      copy16(dst + i * kGroupBytes4 + 512, src[i] + 512, policy);
    }
    const unsigned char *mine = lane < 16 ? (lane < 8 ? src[0] : src[1]) : (lane < 24 ? src[2] : src[3]);
    copy16(rest_at + slot * kStepBytes, mine + 1024 - (lane & 24) * 16, policy);
  }

  // Quarter w of the scores of a step, s += : both groups' 16 tokens by two of
  // the eight steps over the dims.
  struct Keys {
    uint4 a[2], b[2];        // codes of token rows g and g + 8 of the product
    __half2 sa[2], sb[2];    // their scales of this lane's 32 dims
  };
  __device__ __forceinline__ void load_keys(const unsigned char *st, Keys &x) {
    const int tok = 4 * (g >> 1) + (g & 1);  // row g; row g + 8 is tok + 2
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const unsigned char *k = st + sub * kGroupBytes4;
      x.a[sub] = *reinterpret_cast<const uint4 *>(k + tok * 64 + t4 * 16);
      x.b[sub] = *reinterpret_cast<const uint4 *>(k + tok * 64 + 128 + t4 * 16);
      x.sa[sub] = e4m3x2_to_half2(
          *reinterpret_cast<const uint16_t *>(k + kGroupCodes4 + tok * 8 + 2 * t4));
      x.sb[sub] = e4m3x2_to_half2(
          *reinterpret_cast<const uint16_t *>(k + kGroupCodes4 + tok * 8 + 16 + 2 * t4));
    }
  }
  template <int w>
  __device__ __forceinline__ void scores(const Keys &k, float (&s)[2][4]) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const uint32_t wa = w == 0 ? k.a[sub].x : w == 1 ? k.a[sub].y : w == 2 ? k.a[sub].z : k.a[sub].w;
      const uint32_t wb = w == 0 ? k.b[sub].x : w == 1 ? k.b[sub].y : w == 2 ? k.b[sub].z : k.b[sub].w;
      const __half2 fa = w < 2 ? __low2half2(k.sa[sub]) : __high2half2(k.sa[sub]);
      const __half2 fb = w < 2 ? __low2half2(k.sb[sub]) : __high2half2(k.sb[sub]);
      uint32_t x[4], y[4];
      e2m1x8_to_half2x4(wa, x);
      e2m1x8_to_half2x4(wb, y);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mma_16816(s[sub], times(x[2 * i], fa), times(y[2 * i], fb), times(x[2 * i + 1], fa),
                  times(y[2 * i + 1], fb), qf[4 * w + 2 * i], qf[4 * w + 2 * i + 1]);
    }
  }

  // V's scales as halves, each converted once: lane l those of tokens 4 (l / 8)
  // .. + 3 and group l % 8 of the 16, for all lanes that hold these tokens.  They
  // take the place of K's codes, which have been read.  Tokens behind the context
  // get zeros (they may hold NaN).
  __device__ __forceinline__ void spread_scales(unsigned char *st, int valid) const {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x = *reinterpret_cast<const uint32_t *>(st + (2 + i) * kGroupBytes4 + kGroupCodes4 +
                                                       lane * 4);
      if (valid < kStepTokens) {
        const int left = valid - 16 * i - 4 * (lane >> 3);  // tokens of this lane's four
        x = left <= 0 ? 0u : left < 4 ? x & ((1u << (8 * left)) - 1u) : x;
      }
      *reinterpret_cast<uint2 *>(st + i * 256 + lane * 8) =
          make_uint2(half2_bits(e4m3x2_to_half2((uint16_t)x)),
                     half2_bits(e4m3x2_to_half2((uint16_t)(x >> 16))));
    }
    __syncwarp();
  }

  // Quarter w of the outputs of a step: 64 dims of 16 tokens.
  template <int w>
  __device__ __forceinline__ void outputs(const unsigned char *st) {
    constexpr int sub = w >> 1, half = w & 1;
    const uint4 a = *reinterpret_cast<const uint4 *>(st + (2 + sub) * kGroupBytes4 + half * 512 +
                                                     lane * 16);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 c = *reinterpret_cast<const uint4 *>(st + sub * 256 + t4 * 64 + half * 32 + j * 16);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 s01 = bits_half2(i ? c.z : c.x), s23 = bits_half2(i ? c.w : c.y);
        uint32_t x[4];
        e2m1x8_to_half2x4(wa[2 * j + i], x);  // dim row g: tokens 0 1, 2 3; dim row g + 8
        mma_16816(o[4 * half + 2 * j + i], times(x[0], s01), times(x[2], s01), times(x[1], s23),
                  times(x[3], s23), pf[sub][0], pf[sub][1]);
      }
    }
  }

  // Weights from the products of a step with `valid` tokens.
  __device__ __forceinline__ void weights(float (&s)[2][4], int valid) {
    if (valid < kStepTokens) {
      const int tok = 4 * (g >> 1) + (g & 1);
      const float none = __uint_as_float(0xff800000u);
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        if (16 * sub + tok >= valid) s[sub][0] = s[sub][1] = none;
        if (16 * sub + tok + 2 >= valid) s[sub][2] = s[sub][3] = none;
      }
    }
    float x0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
    float x1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
    if (__any_sync(kFullMask, x0 > limit0 || x1 > limit1)) {
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(kFullMask, x0, i));
        x1 = fmaxf(x1, __shfl_xor_sync(kFullMask, x1, i));
      }
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float r0 = exp2_approx((m0 - n0) * f0), r1 = exp2_approx((m1 - n1) * f1);
      m0 = n0;
      m1 = n1;
      // (rounded down: no weight is above 2^15)
      limit0 = __fadd_rd(m0, __fdividef(kMoveLog2, f0));
      limit1 = __fadd_rd(m1, __fdividef(kMoveLog2, f1));
      l0 *= r0;
      l1 *= r1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] *= r0;
        o[i][1] *= r1;
        o[i][2] *= r0;
        o[i][3] *= r1;
      }
    }
    // The distance to the reference before the factor: the score of a large product
    // less that of the reference would keep nothing but their roundings.
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float w0 = exp2_approx(fmaf(s[sub][2 * i] - m0, f0, kUnitLog2)),
                    w1 = exp2_approx(fmaf(s[sub][2 * i + 1] - m1, f1, kUnitLog2));
        l0 += w0;
        l1 += w1;
        pf[sub][i] = transposed(half2_bits(__floats2half2_rn(w0, w1)));
      }
    }
  }

  // Steps i0 + warp, + W, ... below i1 of one unit.
  __device__ __forceinline__ void run(const Part &u, int G) {
    const int32_t *row = p.a.tables + (size_t)u.b * p.a.MB;
    const int nblk = (u.ctx - 1) / BS + 1;
    const int first = u.i0 + warp;
    const int n = first < u.i1 ? (u.i1 - first + W - 1) / W : 0;
    const size_t head = (size_t)u.h * (BS / kGroupTokens4 * kGroupBytes4) + lane * 16;
    from_k = p.a.k_cache + head;
    from_v = p.a.v_cache + head;
    // lane l: the ids of the warp's step 32 j + l; a bad id (flagged) and a block
    // that the context does not reach (its tokens are masked) read block 0
    int a0 = 0, a1 = 0;
    auto ids = [&](int k0) {
      const int t = first + (k0 + lane) * W;
      a0 = a1 = 0;
      if (k0 + lane < n) {
        if constexpr (BS == 32) {
          a0 = check(__ldg(row + t));
        } else {
          a0 = check(__ldg(row + 2 * t));
          if (2 * t + 1 < nblk) a1 = check(__ldg(row + 2 * t + 1));
        }
      }
    };
    auto issue = [&](int k, int slot) {
      if (k < n) {
        if ((k & 31) == 0) ids(k);
        load_step(slot, __shfl_sync(kFullMask, a0, k & 31),
                  BS == 32 ? 0 : __shfl_sync(kFullMask, a1, k & 31));
      }
      copies_commit();
    };
    // the query's loads before the copies, which they would queue behind
    uint4 q[4];
    fetch_query(u.b, u.h, G, q);
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k, k);
    start(q);
    int slot = 0;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      copies_wait<kStages - 2>();
      __syncwarp();  // every lane's copies have landed, and step k - 1 is read
      issue(k + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
      const int valid = min(kStepTokens, u.ctx - (first + k * W) * kStepTokens);
      unsigned char *st = ring + slot * kStepBytes;
      Keys x;
      load_keys(st, x);
      spread_scales(st, valid);
      float s[2][4] = {};
      scores<0>(x, s);
      scores<1>(x, s);
      scores<2>(x, s);
      scores<3>(x, s);
      weights(s, valid);
      outputs<0>(st);
      outputs<1>(st);
      outputs<2>(st);
      outputs<3>(st);
      if (++slot == kStages) slot = 0;
    }
    copies_wait<0>();
  }

  __device__ __forceinline__ int check(int id) {
    if ((unsigned)id < (unsigned)p.a.NB) return id;
    atomicOr(p.a.err, PGD_DEVERR_BAD_BLOCK_ID);
    return 0;
  }
};

// The states of a CTA's warps on one reference a head, in their rings.
template <int W>
struct Sums {
  const float *refs, *totals;  // [W][8]
  __device__ __forceinline__ float reference(int h) const {
    float M = refs[h];
#pragma unroll
    for (int j = 1; j < W; ++j) M = fmaxf(M, refs[j * kHeads + h]);
    return M;
  }
  // Outputs i, i + 1 of [G][128] (i even), and their head's sum.
  __device__ __forceinline__ float2 dims(const unsigned char *smem, int i, float &total) const {
    const float *src = reinterpret_cast<const float *>(smem) + (i >> 7) * kMergeRow + (i & 127);
    float2 acc = make_float2(0.f, 0.f);
    total = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float2 v = *reinterpret_cast<const float2 *>(src + j * (kStages * kStepBytes / 4));
      total += totals[j * kHeads + (i >> 7)];
      acc.x += v.x;
      acc.y += v.y;
    }
    return acc;
  }
};

// Called by every thread; refs: [2][W][8] floats.
template <int BS, int W>
__device__ __forceinline__ Sums<W> merge_warps(const Worker<BS, W> &w, float *refs) {
  float *totals = refs + W * kHeads;
  float l0 = w.l0, l1 = w.l1;
#pragma unroll
  for (int i = 4; i < 32; i <<= 1) {
    l0 += __shfl_xor_sync(kFullMask, l0, i);
    l1 += __shfl_xor_sync(kFullMask, l1, i);
  }
  const int mine_at = w.warp * kHeads + 2 * w.t4;
  // (in log2 from here on)
  const float m0 = w.m0 * w.f0, m1 = w.m1 * w.f1;
  if (w.g == 0) *reinterpret_cast<float2 *>(refs + mine_at) = make_float2(m0, m1);
  __syncthreads();  // the rings are done with, the references written
  float M0 = m0, M1 = m1;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 m = *reinterpret_cast<const float2 *>(refs + i * kHeads + 2 * w.t4);
    M0 = fmaxf(M0, m.x);
    M1 = fmaxf(M1, m.y);
  }
  const float none = __uint_as_float(0xff800000u);  // (a warp without steps has no weight)
  const float r0 = m0 == none ? 0.f : exp2_approx(m0 - M0);
  const float r1 = m1 == none ? 0.f : exp2_approx(m1 - M1);
  if (w.g == 0) *reinterpret_cast<float2 *>(totals + mine_at) = make_float2(l0 * r0, l1 * r1);
  float *mine = reinterpret_cast<float *>(w.ring) + 2 * w.t4 * kMergeRow + w.g;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mine[16 * i] = w.o[i][0] * r0;
    mine[16 * i + kMergeRow] = w.o[i][1] * r1;
    mine[16 * i + 8] = w.o[i][2] * r0;
    mine[16 * i + 8 + kMergeRow] = w.o[i][3] * r1;
  }
  __syncthreads();
  return {refs, totals};
}

__device__ __forceinline__ void store_row(__nv_bfloat16 *at, float4 v, float f) {
  const __nv_bfloat162 y0 = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 y1 = __floats2bfloat162_rn(v.z * f, v.w * f);
  *reinterpret_cast<uint2 *>(at) = make_uint2(*reinterpret_cast<const uint32_t *>(&y0),
                                              *reinterpret_cast<const uint32_t *>(&y1));
}

// A unit's parts, slots s0, s0 + n_kv, ..., to its G rows at `out`: a head by a
// warp, or by W / G of them that take the parts in turn.
template <int W>
__device__ __forceinline__ void merge_parts(const Attn4Params &p, int G, size_t s0, int parts,
                                            __nv_bfloat16 *out, unsigned char *smem) {
  const AttnParams &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sets = G < W ? W / G : 1;
  const int set = G < W ? warp / G : 0;  // (G is a power of two)
  float4 *sum = reinterpret_cast<float4 *>(smem);               // [W][32]
  float2 *states = reinterpret_cast<float2 *>(smem + W * 512);  // [W] (max, sum)
  constexpr int kBatch = 8;  // parts' loads in flight
  for (int h = G < W ? warp % G : warp; h < G; h += W) {
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + s0 * G + h;
    const float4 *o = reinterpret_cast<const float4 *>(a.part_o) + (s0 * G + h) * 32 + lane;
    float M = __uint_as_float(0xff800000u), L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = set; i0 < parts; i0 += kBatch * sets) {
      float2 s[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * sets;
        const size_t at = (size_t)i * a.n_kv * G;
        s[j] = make_float2(__uint_as_float(0xff800000u), 0.f);
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < parts) {
          s[j] = __ldcg(ml + at);
          v[j] = __ldcg(o + at * 32);
        }
      }
      float top = M;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) top = fmaxf(top, s[j].x);
      const float keep = exp2_approx(M - top);
      M = top;
      L *= keep;
      acc.x *= keep;
      acc.y *= keep;
      acc.z *= keep;
      acc.w *= keep;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float r = exp2_approx(s[j].x - M);
        L += s[j].y * r;
        acc.x += v[j].x * r;
        acc.y += v[j].y * r;
        acc.z += v[j].z * r;
        acc.w += v[j].w * r;
      }
    }
    if (sets == 1) {
      store_row(out + (size_t)h * kHeadDim + 4 * lane, acc, p.v_scale / L);
    } else {
      sum[warp * 32 + lane] = acc;
      if (lane == 0) states[warp] = make_float2(M, L);
    }
  }
  if (sets == 1) return;
  __syncthreads();
  if (warp < G) {
    float M = states[warp].x, L = 0.f;
    for (int i = 1; i < sets; ++i) M = fmaxf(M, states[i * G + warp].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < sets; ++i) {
      // (a set without parts has no weight)
      const float2 s = states[i * G + warp];
      const float r = exp2_approx(s.x - M);
      const float4 v = sum[(i * G + warp) * 32 + lane];
      L += s.y * r;
      acc.x += v.x * r;
      acc.y += v.y * r;
      acc.z += v.z * r;
      acc.w += v.w * r;
    }
    store_row(out + (size_t)warp * kHeadDim + 4 * lane, acc, p.v_scale / L);
  }
}

template <int BS, int W>
__global__ void __launch_bounds__(W * 32, kResident<W>)
    attention_fp4_kernel(const Attn4Params p, int G) {
  extern __shared__ __align__(128) unsigned char smem[];
  float *refs = reinterpret_cast<float *>(smem + ring_bytes<W>());  // [W][8] warps' references
  int *flag = reinterpret_cast<int *>(refs + 2 * W * kHeads);
  const int tid = threadIdx.x;
  const AttnParams &a = p.a;

  if (!a.wait_late) pdl_wait();
  pdl_launch_dependents();
  const Part u = find_part<W>(p, BS);
  if (a.wait_late) pdl_wait();
  if (!u.some) return;
  Worker<BS, W> w(p, smem);
  w.run(u, G);

  const Sums<W> sums = merge_warps(w, refs);
  const bool whole = u.parts == 1;
  const int unit = u.b * a.n_kv + u.h;
  const size_t slot = blockIdx.x;
  __nv_bfloat16 *out = a.out + ((size_t)u.b * a.n_q + (size_t)u.h * G) * kHeadDim;
  // two dims of a head a thread
  for (int i = 2 * tid; i < G * kHeadDim; i += 64 * W) {
    const int h = i >> 7;
    float L;
    const float2 acc = sums.dims(smem, i, L);
    if (whole) {
      const float inv = p.v_scale / L;
      *reinterpret_cast<__nv_bfloat162 *>(out + i) = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    } else {
      *reinterpret_cast<float2 *>(a.part_o + slot * G * kHeadDim + i) = acc;
      if ((i & 127) == 0) {
        const float M = sums.reference(h);
        *reinterpret_cast<float2 *>(a.part_ml + (slot * G + h) * 2) = make_float2(M, L);
      }
    }
  }
  if (whole) return;
  __syncthreads();
  if (tid == 0) {
    const int seen = atomic_add_acq_rel_gpu(a.counters + unit, 1);
    if (seen == u.parts - 1) a.counters[unit] = 0;
    *flag = seen == u.parts - 1;
  }
  __syncthreads();
  if (*flag) merge_parts<W>(p, G, (size_t)u.first + u.h, u.parts, out, smem);
}

// Units with CTAs of their own: a cluster of CL, each with an equal share of the
// unit's steps, or one of W warps.  Which unit and steps a CTA has follows from its
// place and one length: no scan of the lengths, nothing through the workspace.  The
// states of a cluster go to its CTAs' shared memory on their barriers, each CTA
// merging 128 / CL dims.
template <int BS, int CL, int W>
__global__ void __launch_bounds__(W * 32)
    attention_fp4_unit_kernel(const Attn4Params p, int G) {
  constexpr int kDims = kHeadDim / CL;
  extern __shared__ __align__(128) unsigned char smem[];
  float *refs = reinterpret_cast<float *>(smem + ring_bytes<W>());  // [2][W][8]
  __shared__ __align__(16) float in_o[CL][kHeads][kDims];
  __shared__ __align__(16) float2 in_ml[CL][kHeads];
  __shared__ __align__(8) uint64_t arrived;
  const AttnParams &a = p.a;
  const int tid = threadIdx.x, rank = blockIdx.x % CL;
  if (CL > 1 && tid == 0) {
    mbar_init(&arrived, 1);
    mbar_init_fence();
    mbar_arrive_expect_tx(&arrived, (uint32_t)(CL * G * (kDims * 4 + 8)));
  }
  // (every CTA of the cluster has its barrier: waited for before the first store)
  if (CL > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (!a.wait_late) pdl_wait();
  pdl_launch_dependents();
  Part u;
  u.b = blockIdx.y;
  u.h = blockIdx.x / CL;
  u.steps = unit_steps(a, BS, u.b, u.ctx, rank == 0 && u.h == 0);
  u.i0 = u.steps * rank / CL;
  u.i1 = u.steps * (rank + 1) / CL;
  if (a.wait_late) pdl_wait();
  if (u.steps == 0) {  // (a bad context: the whole cluster leaves)
    if (CL > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
  }
  Worker<BS, W> w(p, smem);
  w.run(u, G);
  const Sums<W> sums = merge_warps(w, refs);
  __nv_bfloat16 *out = a.out + ((size_t)u.b * a.n_q + (size_t)u.h * G) * kHeadDim;
  if constexpr (CL == 1) {
    for (int i = 2 * tid; i < G * kHeadDim; i += 64 * W) {
      float L;
      const float2 acc = sums.dims(smem, i, L);
      const float f = p.v_scale / L;
      *reinterpret_cast<__nv_bfloat162 *>(out + i) = __floats2bfloat162_rn(acc.x * f, acc.y * f);
    }
    return;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int i = 2 * tid; i < G * kHeadDim; i += 64 * W) {
    const int h = i >> 7, to = (i & 127) / kDims, d = i % kDims;
    float L;
    const float2 acc = sums.dims(smem, i, L);
    send8(&in_o[rank][h][d], &arrived, (uint32_t)to, __float_as_uint(acc.x),
          __float_as_uint(acc.y));
    if (d == 0)
      send8(&in_ml[rank][h], &arrived, (uint32_t)to, __float_as_uint(sums.reference(h)),
            __float_as_uint(L));
  }
  if (tid >= G * kDims) return;
  if (!peers_in_time(&arrived, 0, a.wait_limit_ns)) return leave_late(&arrived, 0, a.err);
  for (int i = tid; i < G * kDims; i += 32 * W) {
    const int h = i / kDims, d = i % kDims;
    float M = in_ml[0][h].x;
#pragma unroll
    for (int k = 1; k < CL; ++k) M = fmaxf(M, in_ml[k][h].x);
    float num = 0.f, L = 0.f;
#pragma unroll
    for (int k = 0; k < CL; ++k) {
      // (a CTA without steps has no weight)
      const float x = in_ml[k][h].x;
      const float r = x == __uint_as_float(0xff800000u) ? 0.f : exp2_approx(x - M);
      num = fmaf(r, in_o[k][h][d], num);
      L = fmaf(r, in_ml[k][h].y, L);
    }
    out[h * kHeadDim + rank * kDims + d] = __float2bfloat16_rn(num * (p.v_scale / L));
  }
}

template <int BS, int W>
cudaError_t launch_kernel(const Attn4Params &p, int G, int grid, cudaStream_t stream) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = attention_fp4_kernel<BS, W>;
  if (!set[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<W>());
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    set[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem_bytes<W>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, G);
}

template <int BS, int CL, int W>
cudaError_t launch_units_of(const Attn4Params &p, int G, cudaStream_t stream) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = attention_fp4_unit_kernel<BS, CL, W>;
  constexpr size_t smem = ring_bytes<W>() + 2 * W * kHeads * 4;
  if (!set[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && CL > 8)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    set[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.a.n_kv * CL), (unsigned)p.a.B);
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, G);
}

template <int CL, int W>
cudaError_t launch_units(const Attn4Params &p, int G, int bs, cudaStream_t stream) {
  return bs == 16 ? launch_units_of<16, CL, W>(p, G, stream)
                  : launch_units_of<32, CL, W>(p, G, stream);
}

}  // namespace

// Which units get CTAs of their own, by the tokens that the tables hold, or none
// (0): parts through the workspace.  Equal shares of short contexts are worth more
// than parts of equal size while all clusters run at once and are small (us,
// clusters / workspace):
//   16 CTAs  8 x 8192: 7.0 / 8.7, 8 x 4096: 5.0 / 6.5 (8 CTAs: 5.4); 8 x 16384: 11.0 / 9.6;
//            of 16 warps 1 x 16384: 7.6 / 9.9, 4 x 32768: 11.1 / 12.8, 6 x 16384: 7.2 / 9.3;
//            8 x 16384: 13.8 / 9.6 (not all at once), 1 x 65536: 16.4 / 13.2;
//   8 CTAs   1 x 512: 3.2 / 5.1, 32 x 1024: 5.2 / 6.8, 32 x 4096: 9.1 / 11.9,
//            32 x 8192: 14.0 / 16.2; 64 x 2048: 10.8 / 9.0; and where the rule takes the
//            slower one, 32 x 256: 4.5 / 4.2;
//   4 CTAs   100 x 1000: 6.3 / 9.4, 64 x 512: 4.6 / 5.8, 64 x 2048: 8.2 / 9.1;
//            64 x 128: 3.8 / 3.4, 112 x 2300: 15.9 / 14.0, 136 x 1000: 11.9 / 10.9.
// Where units are enough for the SMs, a CTA each takes less than parts of equal size
// as long as the longest context is not far from the mean (whole / workspace):
//   16 warps  136 x 500-1000: 7.8 / 10.9, 112 x 4096: 16.9 / 18.7, 152 x 1-4000: 15.9 / 15.4;
//             76 x 1-2500: 11.1 / 9.7, 100 x 1-3000: 12.7 / 11.1, 136 x 1-8000: 25.8 / 22.3;
//   8 warps   256 x 200-1000: 9.7 / 12.5, 304 x 1-2000: 16.0 / 18.5; 256 x 1-4000: 26.9 / 21.4,
//             304 x 2000-4000: 27.7 / 30.4;
//   4 warps   696 x 125-991: 16.3 / 18.6, 1024 x 1-2000: 36.7 / 39.4, 2048 x 1-2000: 60 / 71,
//             64 x 128: 2.9 / 3.4 (16 warps 3.8); 512 x 1-8000: 82 / 63;
//   2 warps (or 4)  1024 x 100-300: 11.6 (12.4), 4096 x 1-64: 14.9 (22.1); 512 x 100-200:
//             6.1 (5.8), 1024 x 100-600: 17.8 (16.7);
//   1 warp (or 2)   4096 x 1-64: 11.8 (14.9), 1024 x 1-20: 3.9 (4.8); 1024 x 30-100: 6.9 (6.6).
struct Shape {
  int ctas, warps;  // CTAs a unit, warps a CTA
};
static Shape shape_of(long long units, long long tokens, int splits, int sms) {
  if (splits > 1) return {0, 0};
  if (splits == 0 && units <= 6 && tokens > 8192 && tokens <= 32768) return {16, 16};
  if (splits == 0 && tokens <= 8192) {
    if (16 * units <= sms && tokens > 1024) return {16, 4};
    if (4 * units <= sms) return {8, 4};
    if (4 * units <= 3 * sms && tokens > 384 && units * tokens <= 1 << 17) return {4, 4};
  }
  const int most = 3 * units <= 2 * sms ? 384 : units > sms && units <= 2 * sms ? 2048 : 4096;
  if (splits == 0 && tokens > most) return {0, 0};
  if (tokens <= 384) return {1, units <= 4 * sms ? 4 : tokens <= 64 ? 1 : 2};
  return {1, units > 2 * sms ? 4 : units > sms ? 8 : 16};
}

// 4 warps a CTA, four CTAs an SM, or 16 and one: 16 for so few units that smaller
// parts are many to merge (one context of 131072 tokens, 8 units: 30.8 us, with 4
// warps 35; 1 unit of 65536: 16.2 and 37.9; but 32 units of 32768: 32 and 29.7).  A
// CTA of 16 warps a unit was 6 % faster for 128 units of 8192 tokens each (30.0 and
// 31.9), but 36 where 21.5 do for 1 to 8192 tokens.
static int warps_of(long long units) { return units <= 16 ? 16 : 4; }
static long long resident_ctas(int W, int sms) {
  return (W == 16 ? kResident<16> : kResident<4>) * (long long)sms;
}

// Steps of a part at least: two a warp.  Where so few units have all the CTAs more
// parts take longer to merge than they save (1 unit of 65536 tokens: 13.2 us, 16.2
// with 8 steps; but 8 of 1000 to 20000: 9.7 and 9.1).
static int least_steps(long long units) { return units <= 4 ? 32 : 8; }

// The most CTAs of an automatic call on tables of MB * bs = tokens.
long long attention_fp4_grid(long long units, long long tokens, int sms) {
  const long long steps = (tokens - 1) / kStepTokens + 1;
  const long long most = units * ((steps - 1) / least_steps(units) + 1);
  return std::min(most, units + 3 * resident_ctas(warps_of(units), sms));
}

cudaError_t attention_fp4_launch(const Attn4Params &p_in, int G, int bs, int grid, int sms,
                                 cudaStream_t stream) {
  Attn4Params p = p_in;
  const long long units = (long long)p.a.B * p.a.n_kv, tokens = (long long)p.a.MB * bs;
  switch (const Shape x = shape_of(units, tokens, p.splits, sms); 100 * x.ctas + x.warps) {
    case 1604: return launch_units<16, 4>(p, G, bs, stream);
    case 1616: return launch_units<16, 16>(p, G, bs, stream);
    case 804: return launch_units<8, 4>(p, G, bs, stream);
    case 404: return launch_units<4, 4>(p, G, bs, stream);
    case 116: return launch_units<1, 16>(p, G, bs, stream);
    case 108: return launch_units<1, 8>(p, G, bs, stream);
    case 104: return launch_units<1, 4>(p, G, bs, stream);
    case 102: return launch_units<1, 2>(p, G, bs, stream);
    case 101: return launch_units<1, 1>(p, G, bs, stream);
  }
  const int W = warps_of(units);
  p.resident = (int)resident_ctas(W, sms);
  p.least_steps = least_steps(units);
  p.inv_resident = 1.f / (float)p.resident;
  p.uneven = 4 * units > p.resident;
  if (W == 16)
    return bs == 16 ? launch_kernel<16, 16>(p, G, grid, stream)
                    : launch_kernel<32, 16>(p, G, grid, stream);
  return bs == 16 ? launch_kernel<16, 4>(p, G, grid, stream)
                  : launch_kernel<32, 4>(p, G, grid, stream);
}

}  // namespace pgd
