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
// and no wait on another warp while a context is read.
//
// Split.  The steps of all units (sequence, KV head) lie on one line, in that
// order, cut into equal parts, one a CTA.  A cut within `snap` steps of a
// unit's end moves there, so that units are not split for nothing.  A CTA's
// warps take its steps of a unit in turn and merge their states in shared
// memory; parts of a unit go through the workspace, merged by the CTA that
// finishes last, in the order of the parts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kv_fp4.cuh"

namespace pgd {
namespace {

constexpr int kStepTokens = 32;
constexpr int kStepBytes = 2 * 2 * kGroupBytes4;  // K and V of two groups
constexpr int kStages = 3;
constexpr int kHeads = 8;              // query heads a product takes
constexpr int kMergeRow = kHeadDim + 4;  // floats between heads when states are merged
constexpr float kMoveLog2 = 8.f;       // move the reference when exceeded by 2^8
constexpr float kUnitLog2 = 7.f;       // a weight of the reference is 2^7

template <int W>
constexpr int ring_bytes() {
  return W * kStages * kStepBytes;
}
template <int W>
constexpr size_t smem_bytes(int B) {
  return (size_t)ring_bytes<W>() + W * kHeads * 8 + 64 + (size_t)(B + 1) * 4;
}
static_assert(kHeads * kMergeRow * 4 <= kStages * kStepBytes, "a warp's state fits its ring");

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
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

// The line of steps: sequence b's units begin at pre[b], n_kv of them with
// (pre[b + 1] - pre[b]) / n_kv steps each.
struct Line {
  const int *pre;
  int B, n_kv, total;
};
struct Unit {
  int b, h, start, steps;  // start: on the line
};
// The unit of step x (0 <= x < total).
__device__ __forceinline__ Unit unit_at(const Line &l, int x) {
  int lo = 0, hi = l.B;  // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.pre[mid] <= x) lo = mid; else hi = mid;
  }
  Unit u;
  u.b = lo;
  u.steps = (l.pre[lo + 1] - l.pre[lo]) / l.n_kv;
  u.h = (x - l.pre[lo]) / u.steps;
  u.start = l.pre[lo] + u.h * u.steps;
  return u;
}

// Equal cuts: CTA c's part of the line before any moves.
struct Cuts {
  int n, q, r, snap;  // parts; r of them have q + 1 steps, the others q
  __device__ __forceinline__ int at(int c) const { return c * q + min(c, r); }
  // The least c with at(c) >= x.
  __device__ __forceinline__ int reach(int x) const {
    const int head = r * (q + 1);
    return x <= head ? (x + q) / (q + 1) : r + (x - head + q - 1) / q;
  }
};
__device__ __forceinline__ int cut(const Line &l, const Cuts &k, int c) {
  const int x = k.at(c);
  if (x >= l.total) return l.total;
  const Unit u = unit_at(l, x);
  if (x - u.start <= k.snap) return u.start;
  if (u.start + u.steps - x <= k.snap) return u.start + u.steps;
  return x;
}

template <int BS, int W>
struct Worker {
  const Attn4Params &p;
  int lane, g, t4, warp;
  unsigned char *ring;  // this warp's
  uint32_t ring_at;

  // Fragments and state.
  uint32_t qf[16];
  float f0, f1;      // factors of the scores of heads 2 t4, 2 t4 + 1 (log2 domain)
  float m0, m1;      // references
  float l0, l1;      // this lane's part of the sums
  float o[8][4];     // dims 16 i + g (+ 8) of those two heads

  __device__ __forceinline__ Worker(const Attn4Params &p_, unsigned char *smem) : p(p_) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    g = lane >> 2;
    t4 = lane & 3;
    ring = smem + warp * kStages * kStepBytes;
    ring_at = smem_addr(ring);
  }

  // The query as operand registers: lane (g, t4) holds dims 32 t4 .. + 31 of
  // head g, in the order in which K's codes lie.
  __device__ __forceinline__ void load_query(int b, int h, int G) {
    float x[32];
    uint32_t top = 0;
    if (g < G) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          p.a.q + ((size_t)b * p.a.n_q + (size_t)h * G + g) * kHeadDim + 32 * t4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = __ldg(src + i);
        float y[8];
        unpack8(v, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[8 * i + j] = y[j];
        top = __vmaxu2(top, v.x & 0x7fff7fffu);
        top = __vmaxu2(top, v.y & 0x7fff7fffu);
        top = __vmaxu2(top, v.z & 0x7fff7fffu);
        top = __vmaxu2(top, v.w & 0x7fff7fffu);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.f;
    }
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(kFullMask, top, 1));
    top = max(top, __shfl_xor_sync(kFullMask, top, 2));
    // the largest lies in [2^e, 2^(e + 1)); a query of next to nothing keeps 2^-100
    const int e = max((int)(top >> 7) - 127, -100);
    const float up = pow2f(14 - e);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      qf[i] = half2_bits(__floats2half2_rn(x[2 * i] * up, x[2 * i + 1] * up));
    const float back = p.a.qk_scale_log2 * pow2f(e - 14);
    f0 = __shfl_sync(kFullMask, back, 8 * t4);
    f1 = __shfl_sync(kFullMask, back, 8 * t4 + 4);
    m0 = m1 = __uint_as_float(0xff800000u);
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  }

  // Starts the copies of a step from its blocks' ids (-1: nothing, zeros).
  __device__ __forceinline__ void load_step(int slot, int id0, int id1, int h) {
    const uint32_t dst = ring_at + slot * kStepBytes + lane * 16;
    if constexpr (BS == 32) {
      const size_t at = ((size_t)max(id0, 0) * p.a.n_kv + h) * (2 * kGroupBytes4);
      const unsigned char *k = p.a.k_cache + at, *v = p.a.v_cache + at;
      const uint32_t n = id0 >= 0 ? 16u : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) copy16(dst + j * 512, k + lane * 16 + j * 512, n);
      // the fifth goes on from K (128 more bytes ... 144 pieces) to V
      copy16(dst + 4 * 512, lane < 16 ? k + lane * 16 + 2048 : v + (lane - 16) * 16, n);
#pragma unroll
      for (int j = 5; j < 9; ++j) copy16(dst + j * 512, v + (lane - 16) * 16 + (j - 4) * 512, n);
    } else {
      const size_t a0 = ((size_t)max(id0, 0) * p.a.n_kv + h) * kGroupBytes4;
      const size_t a1 = ((size_t)max(id1, 0) * p.a.n_kv + h) * kGroupBytes4;
      const unsigned char *k0 = p.a.k_cache + a0, *v0 = p.a.v_cache + a0;
      const unsigned char *k1 = p.a.k_cache + a1, *v1 = p.a.v_cache + a1;
      const uint32_t n0 = id0 >= 0 ? 16u : 0u, n1 = id1 >= 0 ? 16u : 0u;
      const int x = lane * 16;
      copy16(dst, k0 + x, n0);
      copy16(dst + 512, k0 + x + 512, n0);
      copy16(dst + 1024, lane < 8 ? k0 + x + 1024 : k1 + (x - 128), lane < 8 ? n0 : n1);
      copy16(dst + 1536, k1 + (x - 128) + 512, n1);
      copy16(dst + 2048, lane < 16 ? k1 + (x - 128) + 1024 : v0 + (x - 256), lane < 16 ? n1 : n0);
      copy16(dst + 2560, v0 + (x - 256) + 512, n0);
      copy16(dst + 3072, lane < 24 ? v0 + (x - 256) + 1024 : v1 + (x - 384), lane < 24 ? n0 : n1);
      copy16(dst + 3584, v1 + (x - 384) + 512, n1);
      copy16(dst + 4096, v1 + (x - 384) + 1024, n1);
    }
  }

  // One step of 32 tokens, `valid` of them (32 but at a context's end).
  __device__ __forceinline__ void compute(int slot, int valid) {
    unsigned char *st = ring + slot * kStepBytes;
    if (valid < kStepTokens) {
      // tokens behind the context: their V scales to zero (they may hold NaN)
      for (int i = lane; i < kStepTokens * 8; i += 32) {
        const int t = i >> 3, c = i & 7;
        if (t >= valid)
          st[2 * kGroupBytes4 + (t >> 4) * kGroupBytes4 + kGroupCodes4 + ((t & 15) >> 2) * 32 +
             c * 4 + (t & 3)] = 0;
      }
      __syncwarp();
    }
    const int tok = 4 * (g >> 1) + (g & 1);  // row g of the product; row g + 8 is tok + 2
    float s[2][4];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const unsigned char *k = st + sub * kGroupBytes4;
      const uint4 a = *reinterpret_cast<const uint4 *>(k + tok * 64 + t4 * 16);
      const uint4 b = *reinterpret_cast<const uint4 *>(k + tok * 64 + 128 + t4 * 16);
      const __half2 sa = e4m3x2_to_half2(
          *reinterpret_cast<const uint16_t *>(k + kGroupCodes4 + tok * 8 + 2 * t4));
      const __half2 sb = e4m3x2_to_half2(
          *reinterpret_cast<const uint16_t *>(k + kGroupCodes4 + tok * 8 + 16 + 2 * t4));
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
      s[sub][0] = s[sub][1] = s[sub][2] = s[sub][3] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const __half2 fa = w < 2 ? __low2half2(sa) : __high2half2(sa);
        const __half2 fb = w < 2 ? __low2half2(sb) : __high2half2(sb);
        uint32_t x[4], y[4];
        e2m1x8_to_half2x4(wa[w], x);
        e2m1x8_to_half2x4(wb[w], y);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_16816(s[sub], times(x[2 * i], fa), times(y[2 * i], fb), times(x[2 * i + 1], fa),
                    times(y[2 * i + 1], fb), qf[4 * w + 2 * i], qf[4 * w + 2 * i + 1]);
      }
    }
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      s[sub][0] *= f0;
      s[sub][1] *= f1;
      s[sub][2] *= f0;
      s[sub][3] *= f1;
    }
    if (valid < kStepTokens) {
      const float none = __uint_as_float(0xff800000u);
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        if (16 * sub + tok >= valid) s[sub][0] = s[sub][1] = none;
        if (16 * sub + tok + 2 >= valid) s[sub][2] = s[sub][3] = none;
      }
    }
    float x0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
    float x1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
    if (__any_sync(kFullMask, x0 > m0 + kMoveLog2 || x1 > m1 + kMoveLog2)) {
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(kFullMask, x0, i));
        x1 = fmaxf(x1, __shfl_xor_sync(kFullMask, x1, i));
      }
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float r0 = exp2_approx(m0 - n0), r1 = exp2_approx(m1 - n1);
      m0 = n0;
      m1 = n1;
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
    uint32_t pf[2][2];
    const float b0 = kUnitLog2 - m0, b1 = kUnitLog2 - m1;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float w0 = exp2_approx(s[sub][2 * i] + b0), w1 = exp2_approx(s[sub][2 * i + 1] + b1);
        l0 += w0;
        l1 += w1;
        pf[sub][i] = transposed(half2_bits(__floats2half2_rn(w0, w1)));
      }
    }
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const unsigned char *v = st + (2 + sub) * kGroupBytes4;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 a = *reinterpret_cast<const uint4 *>(v + half * 512 + lane * 16);
        const uint4 c = *reinterpret_cast<const uint4 *>(v + kGroupCodes4 + t4 * 32 + half * 16);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 s01 = e4m3x2_to_half2((uint16_t)wc[i]);
          const __half2 s23 = e4m3x2_to_half2((uint16_t)(wc[i] >> 16));
          uint32_t x[4];
          e2m1x8_to_half2x4(wa[i], x);  // dim row g: tokens 0 1, 2 3; dim row g + 8
          mma_16816(o[4 * half + i], times(x[0], s01), times(x[2], s01), times(x[1], s23),
                    times(x[3], s23), pf[sub][0], pf[sub][1]);
        }
      }
    }
  }

  // Steps i0 + warp, + W, ... below i1 of one unit.
  __device__ __forceinline__ void run(const Unit &u, int ctx, int i0, int i1) {
    const int32_t *row = p.a.tables + (size_t)u.b * p.a.MB;
    const int nblk = (ctx - 1) / BS + 1;
    const int first = i0 + warp;
    const int n = first < i1 ? (i1 - first + W - 1) / W : 0;
    int a0 = -1, a1 = -1;  // lane l: the ids of the warp's step 32 j + l
    auto ids = [&](int k0) {
      const int t = first + (k0 + lane) * W;
      a0 = a1 = -1;
      if (k0 + lane < n) {
        if constexpr (BS == 32) {
          a0 = check(__ldg(row + t));
        } else {
          a0 = check(__ldg(row + 2 * t));
          if (2 * t + 1 < nblk) a1 = check(__ldg(row + 2 * t + 1));
        }
      }
    };
    auto issue = [&](int k) {
      if (k < n) {
        if ((k & 31) == 0) ids(k);
        load_step(k % kStages, __shfl_sync(kFullMask, a0, k & 31),
                  BS == 32 ? -1 : __shfl_sync(kFullMask, a1, k & 31), u.h);
      }
      copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k);
    int slot = 0;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      copies_wait<kStages - 2>();
      __syncwarp();  // every lane's copies have landed, and step k - 1 is read
      issue(k + kStages - 1);
      compute(slot, min(kStepTokens, ctx - (first + k * W) * kStepTokens));
      slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    copies_wait<0>();
  }

  __device__ __forceinline__ int check(int id) {
    if ((unsigned)id < (unsigned)p.a.NB) return id;
    atomicOr(p.a.err, PGD_DEVERR_BAD_BLOCK_ID);
    return -1;
  }
};

template <int BS, int W>
__global__ void __launch_bounds__(W * 32, W == 4 ? 4 : 1)
    attention_fp4_kernel(const Attn4Params p, int G) {
  extern __shared__ __align__(16) unsigned char smem[];
  float2 *ml = reinterpret_cast<float2 *>(smem + ring_bytes<W>());  // [W][8] (max, sum)
  int *flag = reinterpret_cast<int *>(smem + ring_bytes<W>() + W * kHeads * 8);
  int *pre = flag + 16;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnParams &a = p.a;

  if (!a.wait_late) pdl_wait();
  pdl_launch_dependents();

  // The line: steps of every sequence's units, summed by warp 0.
  if (warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < a.B) {
        const int ctx = __ldg(a.ctx + b);
        if (ctx < 1 || ctx > a.MB * BS) {
          if (blockIdx.x == 0) atomicOr(a.err, PGD_DEVERR_BAD_CONTEXT);
        } else {
          n = ((ctx - 1) / kStepTokens + 1) * a.n_kv;
        }
      }
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int y = __shfl_up_sync(kFullMask, n, i);
        if (lane >= i) n += y;
      }
      if (b < a.B) pre[b + 1] = sum + n;
      sum += __shfl_sync(kFullMask, n, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
  const Line line = {pre, a.B, a.n_kv, pre[a.B]};
  Cuts k;
  k.n = max(1, min((int)gridDim.x, line.total / p.steps_per_cta));
  k.q = line.total / k.n;
  k.r = line.total % k.n;
  k.snap = a.auto_split ? min(k.q >> 3, 2 * W) : 0;
  const int cta = blockIdx.x;
  if (a.wait_late) pdl_wait();
  if (cta >= k.n || line.total == 0) return;

  const int end = cut(line, k, cta + 1);
  int x = cut(line, k, cta);
  Worker<BS, W> w(p, smem);
  while (x < end) {
    const Unit u = unit_at(line, x);
    const int i0 = x - u.start, i1 = min(u.steps, end - u.start);
    x = u.start + i1;
    const int ctx = __ldg(a.ctx + u.b);
    w.load_query(u.b, u.h, G);
    w.run(u, ctx, i0, i1);

    // ---- the warps' states, merged
    float l0 = w.l0, l1 = w.l1;
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) {
      l0 += __shfl_xor_sync(kFullMask, l0, i);
      l1 += __shfl_xor_sync(kFullMask, l1, i);
    }
    if (w.g == 0) {
      ml[warp * kHeads + 2 * w.t4] = make_float2(w.m0, l0);
      ml[warp * kHeads + 2 * w.t4 + 1] = make_float2(w.m1, l1);
    }
    __syncthreads();  // the rings are done with, the references written
    float M0 = w.m0, M1 = w.m1;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      M0 = fmaxf(M0, ml[i * kHeads + 2 * w.t4].x);
      M1 = fmaxf(M1, ml[i * kHeads + 2 * w.t4 + 1].x);
    }
    {
      const float r0 = exp2_approx(w.m0 - M0), r1 = exp2_approx(w.m1 - M1);
      float *mine = reinterpret_cast<float *>(w.ring) + 2 * w.t4 * kMergeRow + w.g;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mine[16 * i] = w.o[i][0] * r0;
        mine[16 * i + kMergeRow] = w.o[i][1] * r1;
        mine[16 * i + 8] = w.o[i][2] * r0;
        mine[16 * i + 8 + kMergeRow] = w.o[i][3] * r1;
      }
    }
    __syncthreads();
    const bool whole = i0 == 0 && i1 == u.steps;
    const int unit = u.b * a.n_kv + u.h;
    const size_t slot = (size_t)unit + cta;
    for (int h = warp; h < G; h += W) {
      float M = ml[h].x;
#pragma unroll
      for (int i = 1; i < W; ++i) M = fmaxf(M, ml[i * kHeads + h].x);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 s = ml[i * kHeads + h];
        L += s.y * exp2_approx(s.x - M);
        const float4 v = *reinterpret_cast<const float4 *>(
            smem + i * kStages * kStepBytes + (h * kMergeRow + 4 * lane) * 4);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      if (whole) {
        const float inv = p.v_scale / L;
        const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(a.out + ((size_t)u.b * a.n_q + (size_t)u.h * G + h) * kHeadDim +
                                   4 * lane) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&y0),
                       *reinterpret_cast<const uint32_t *>(&y1));
      } else {
        if (lane == 0) *reinterpret_cast<float2 *>(a.part_ml + (slot * G + h) * 2) = make_float2(M, L);
        *reinterpret_cast<float4 *>(a.part_o + (slot * G + h) * kHeadDim + 4 * lane) = acc;
      }
    }
    if (!whole) {
      // the parts of this unit: those of the CTAs first .. last
      const int c1 = k.reach(u.start + k.snap + 1);
      const int c2 = k.reach(u.start + u.steps - k.snap) - 1;
      const int first = c1 - 1, parts = c2 - first + 1;
      __syncthreads();
      if (tid == 0) {
        const int seen = atomic_add_acq_rel_gpu(a.counters + unit, 1);
        if (seen == parts - 1) a.counters[unit] = 0;
        *flag = seen == parts - 1;
      }
      __syncthreads();
      if (*flag) {
        __threadfence();
        const size_t s0 = (size_t)unit + first;
        for (int h = warp; h < G; h += W) {
          float M = __uint_as_float(0xff800000u);
          for (int i = lane; i < parts; i += 32)
            M = fmaxf(M, __ldcg(a.part_ml + ((s0 + i) * G + h) * 2));
#pragma unroll
          for (int i = 16; i; i >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, i));
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int i = 0; i < parts; ++i) {
            const float2 s = __ldcg(reinterpret_cast<const float2 *>(a.part_ml + ((s0 + i) * G + h) * 2));
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(
                a.part_o + ((s0 + i) * G + h) * kHeadDim + 4 * lane));
            const float r = exp2_approx(s.x - M);
            L += s.y * r;
            acc.x += v.x * r;
            acc.y += v.y * r;
            acc.z += v.z * r;
            acc.w += v.w * r;
          }
          const float inv = p.v_scale / L;
          const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
          const __nv_bfloat162 y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2 *>(a.out +
                                     ((size_t)u.b * a.n_q + (size_t)u.h * G + h) * kHeadDim +
                                     4 * lane) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&y0),
                         *reinterpret_cast<const uint32_t *>(&y1));
        }
      }
    }
    __syncthreads();  // rings, states and flag are free again
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
                             (int)smem_bytes<W>(PGD_MAX_BATCH));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    set[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem_bytes<W>(p.a.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, G);
}
static_assert(smem_bytes<4>(PGD_MAX_BATCH) <= 232448, "layout exceeds 227 KB");

}  // namespace

int attention_fp4_grid(long long units, int sms) { return 4 * sms; }

cudaError_t attention_fp4_launch(const Attn4Params &p_in, int G, int bs, int grid,
                                 cudaStream_t stream) {
  Attn4Params p = p_in;
  p.steps_per_cta = p.a.auto_split ? 4 : 1;
  return bs == 16 ? launch_kernel<16, 4>(p, G, grid, stream)
                  : launch_kernel<32, 4>(p, G, grid, stream);
}

}  // namespace pgd
