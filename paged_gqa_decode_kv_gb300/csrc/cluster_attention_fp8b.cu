// cluster_attention_fp8b.cu -- decode attention over the block-scaled 8-bit
// cache for short contexts, on the CUDA cores: one cluster of CTAs per
// (sequence, KV head), 8 of them up to 1024 tokens and 16 up to 2048.
//
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k_t) v_t,  t < ctx[b] <= 2048,
//   k_t = sk[tile] * E4M3(code), v_t = sv[tile] * E4M3(code)
//
// Such a call is bound by a chain of latencies, so the chain is short:
// - the context length, the table row (at most 128 blocks) and the query are
//   loaded side by side; then K and V codes and scales, all in flight together;
// - CTA r of a cluster takes the contiguous tokens [r ctx / C, (r + 1) ctx / C),
//   at most 128, in one piece: two threads a token for q.k (64 dims each), one
//   maximum and one sum per head; p.v with two dims a thread and every fourth
//   token, V's scale folded into the probability; fp32, exact exp2;
// - every CTA stores its maxima, sums and output dims into the shared memory of
//   the CTAs that write them, counted on a barrier of the receiver, and CTA r
//   merges the C states of its 128 / C dims by log-sum-exp from its own memory
//   (a cluster barrier instead takes 0.3 us more; reading the peers' states, a
//   second barrier before a CTA may exit and the latency of the loads).
// 8 heads x 2048 tokens, G = 4: 7.0 us (8.7 on the tensor cores; 4096 tokens
// in 16 CTAs of 512 threads: 13.2 against 11.2).
// 8 heads x 512 tokens, G = 4: 3.9 us (5.1 in pieces of 64 tokens with a table
// load behind the length and remote loads; 8.0 with eight threads a token, whose
// reads of the query met in the same banks).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cluster.cuh"
#include "kv_fp8b.cuh"

namespace pgd {
namespace cl8b {

constexpr int THREADS = 256;
constexpr int CH = 128;        // tokens of a CTA at most
constexpr int NTG = 4;         // token groups of p.v

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// CL: CTAs per (sequence, KV head), one cluster.
template <int G, int BS, int CL>
__global__ void __launch_bounds__(THREADS) cluster_attention_kernel(const Attn8bParams pp) {
  const AttnParams &p = pp.a;
  constexpr size_t TILE = (size_t)BS * kHeadDim;
  constexpr int NW = THREADS / 32;
  constexpr int MAXB = CL * CH / 16;  // blocks of a sequence (16 tokens each) at most
  constexpr int OD = kHeadDim / CL;   // output dims that a CTA merges
  // (two halves, 4 banks apart: a warp reads the same dims of both at once)
  __shared__ __align__(16) float qs[G][2][kHeadDim / 2 + 4];
  __shared__ __align__(16) unsigned char vs[CH][kHeadDim];  // V codes
  __shared__ float vsc[CH];                                 // their scales (0: no weight)
  __shared__ __align__(16) float ps[CH][G];                 // probability times V's scale
  __shared__ float red[2][NW][G];                           // per-warp maxima, sums
  __shared__ int tbl[MAXB];
  __shared__ float po[NTG][G][kHeadDim];                    // outputs of the token groups
  // written by the peers: maxima and sums, outputs
  __shared__ __align__(16) float2 in_ml[CL][G];
  __shared__ __align__(16) float in_o[CL][G][OD];
  __shared__ uint64_t arrived;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int unit = (int)blockIdx.x / CL;
  const int b = unit / p.n_kv, g = unit % p.n_kv;
  // (every CTA of the cluster has started and has its barrier: waited for before
  // the first store into another's shared memory)
  if (tid == 0) {
    mbar_init(&arrived, 1);
    mbar_init_fence();
    mbar_arrive_expect_tx(&arrived, sizeof(in_ml) + sizeof(in_o));
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = __ldg(p.ctx + b);
  const int32_t *trow = p.tables + (size_t)b * p.MB;
  if (tid < p.MB && tid < MAXB) tbl[tid] = __ldg(trow + tid);
  const uint4 *qsrc = reinterpret_cast<const uint4 *>(p.q + ((size_t)b * p.n_q + g * G) * kHeadDim);
  if (tid < G * 16) {
    float f[8];
    unpack8(__ldg(qsrc + tid), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) qs[tid / 16][(tid % 16) / 8][(tid % 8) * 8 + e] = f[e];
  }
  const bool ctx_ok = ctx >= 1 && ctx <= p.MB * BS;
  if (!ctx_ok && tid == 0 && rank == 0 && g == 0) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
  const int n = ctx_ok ? ctx : 0;
  const int t_lo = n * (int)rank / CL, nt = n * ((int)rank + 1) / CL - t_lo;
  __syncthreads();

  // K of token j (64 dims); V row 32 k + tid / 8, chunk tid % 8
  const int j = tid >> 1, hf = tid & 1;
  uint4 kr[4], vr[4];
  float ksc = 0.f, vscl = 0.f;
  const int kblk = j < nt ? tbl[(t_lo + j) / BS] : -1;
  const bool kval = (unsigned)kblk < (unsigned)p.NB;
  if (j < nt && !kval) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
#pragma unroll
  for (int k = 0; k < 4; ++k) kr[k] = make_uint4(0, 0, 0, 0);
  if (kval) {
    const size_t tile = (size_t)kblk * p.n_kv + g;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      kr[k] = __ldg(reinterpret_cast<const uint4 *>(
          p.k_cache + tile * TILE + code_offset8b((t_lo + j) % BS, 4 * hf + k)));
    ksc = __ldg(pp.k_scales + tile);
    if (hf == 0) vscl = __ldg(pp.v_scales + tile);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int jj = 32 * k + (tid >> 3), tv = t_lo + jj;
    vr[k] = make_uint4(0, 0, 0, 0);
    if (jj < nt) {
      const int blk = tbl[tv / BS];
      if ((unsigned)blk < (unsigned)p.NB)
        vr[k] = __ldg(reinterpret_cast<const uint4 *>(
            p.v_cache + ((size_t)blk * p.n_kv + g) * TILE + code_offset8b(tv % BS, tid & 7)));
    }
  }
  float s[G];
#pragma unroll
  for (int h = 0; h < G; ++h) s[h] = 0.f;
  if (warp * 16 < nt) {  // (the other warps have no token)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {kr[k].x, kr[k].y, kr[k].z, kr[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = __half22float2(e4m3x2_to_half2((uint16_t)w[e]));
        const float2 c = __half22float2(e4m3x2_to_half2((uint16_t)(w[e] >> 16)));
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float4 q4 = *reinterpret_cast<const float4 *>(&qs[h][hf][16 * k + 4 * e]);
          s[h] = fmaf(q4.x, a.x, s[h]);
          s[h] = fmaf(q4.y, a.y, s[h]);
          s[h] = fmaf(q4.z, c.x, s[h]);
          s[h] = fmaf(q4.w, c.y, s[h]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint4 *>(&vs[32 * k + (tid >> 3)][16 * (tid & 7)]) = vr[k];
  if (hf == 0) vsc[j] = vscl;
  // the CTA's maximum of each head, the probabilities, their sums
#pragma unroll
  for (int h = 0; h < G; ++h) {
    s[h] += __shfl_xor_sync(kFullMask, s[h], 1);
    s[h] = kval ? s[h] * ksc * p.qk_scale_log2 : -INFINITY;
    float m = s[h];
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    if (lane == 0) red[0][warp][h] = m;
  }
  __syncthreads();
  float mx[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    mx[h] = red[0][0][h];
#pragma unroll
    for (int w = 1; w < NW; ++w) mx[h] = fmaxf(mx[h], red[0][w][h]);
    const float e = s[h] == -INFINITY ? 0.f : exp2f(s[h] - mx[h]);
    if (hf == 0) ps[j][h] = e * vsc[j];
    float l = e;
#pragma unroll
    for (int o = 2; o < 32; o <<= 1) l += __shfl_xor_sync(kFullMask, l, o);
    if (lane == 0) red[1][warp][h] = l;
  }
  __syncthreads();
  // p.v: dims 2 d and 2 d + 1 over the tokens of group tg
  {
    const int d = tid & 63, tg = tid >> 6;
    float a0[G], a1[G];
#pragma unroll
    for (int h = 0; h < G; ++h) { a0[h] = 0.f; a1[h] = 0.f; }
#pragma unroll 4
    for (int jj = tg; jj < nt; jj += NTG) {
      const float2 v = __half22float2(
          e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(&vs[jj][2 * d])));
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float w = ps[jj][h];
        a0[h] = fmaf(w, v.x, a0[h]);
        a1[h] = fmaf(w, v.y, a1[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < G; ++h)
      *reinterpret_cast<float2 *>(&po[tg][h][2 * d]) = make_float2(a0[h], a1[h]);
  }
  __syncthreads();
  // This CTA's state to the CTAs that merge it.
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int i = tid; i < G * (kHeadDim / 4); i += THREADS) {
    const int h = i / (kHeadDim / 4), d = i % (kHeadDim / 4) * 4;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = __float_as_uint((po[0][h][d + k] + po[1][h][d + k]) +
                             (po[2][h][d + k] + po[3][h][d + k]));
    send16(&in_o[rank][h][d % OD], &arrived, (uint32_t)(d / OD), o[0], o[1], o[2], o[3]);
  }
  if (tid >= THREADS - CL * G) {
    const int i = THREADS - 1 - tid, h = i / CL, r = i % CL;
    float l = 0.f, m = red[0][0][h];
    for (int w = 0; w < NW; ++w) {
      l += red[1][w][h];
      m = fmaxf(m, red[0][w][h]);
    }
    send8(&in_ml[rank][h], &arrived, (uint32_t)r, __float_as_uint(m), __float_as_uint(l));
  }
  if (tid < OD * G) {
    const int h = tid / OD, d = tid % OD;
    if (!wait_for_peers(&arrived, 0)) {
      atomicOr(p.err, PGD_DEVERR_TIMEOUT);
      wait_to_leave();
      return;
    }
    float M = in_ml[0][h].x;
#pragma unroll
    for (int k = 1; k < CL; ++k) M = fmaxf(M, in_ml[k][h].x);
    float num = 0.f, den = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        const float w = in_ml[k][h].x == -INFINITY ? 0.f : exp2f(in_ml[k][h].x - M);
        num = fmaf(w, in_o[k][h][d], num);
        den = fmaf(w, in_ml[k][h].y, den);
      }
    }
    p.out[((size_t)b * p.n_q + g * G + h) * kHeadDim + rank * OD + d] =
        __float2bfloat16_rn(den != 0.f ? num / den : 0.f);
  }
}

template <class Kernel>
cudaError_t allow_large_clusters(Kernel kernel, volatile int (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = 1;
  return e;
}
cudaLaunchAttribute cluster_of(int n) {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)n;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

template <int G, int BS, int CL>
cudaError_t launch_cl(const Attn8bParams &p, cudaStream_t stream) {
  auto kernel = cluster_attention_kernel<G, BS, CL>;
  if (CL > 8) {
    static volatile int done[64] = {0};  // larger clusters allowed, per device
    const cudaError_t e = allow_large_clusters(kernel, done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.a.B * p.a.n_kv * CL));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0] = cluster_of(CL);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int G, int BS>
cudaError_t launch_g(const Attn8bParams &p, cudaStream_t stream) {
  return p.a.MB * BS <= 8 * CH ? launch_cl<G, BS, 8>(p, stream) : launch_cl<G, BS, 16>(p, stream);
}

template <int BS>
cudaError_t launch_bs(const Attn8bParams &p, int G, cudaStream_t stream) {
  switch (G) {
    case 1: return launch_g<1, BS>(p, stream);
    case 2: return launch_g<2, BS>(p, stream);
    case 4: return launch_g<4, BS>(p, stream);
    case 8: return launch_g<8, BS>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace cl8b

// Whether the current device places clusters of 16 (a slice of a GPU may not).
static bool clusters_of_16() {
  static volatile int known[64] = {0};  // per device: 1 no, 2 yes
  static volatile int done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (!known[dev]) {
    auto kernel = cl8b::cluster_attention_kernel<8, 16, 16>;  // the largest one
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(cl8b::THREADS);
    cudaLaunchAttribute attr = cl8b::cluster_of(16);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cl8b::allow_large_clusters(kernel, done) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[dev] = n > 0 ? 2 : 1;
  }
  return known[dev] == 2;
}

int cluster_max_tokens() { return (clusters_of_16() ? 16 : 8) * cl8b::CH; }

cudaError_t cluster_attention_fp8b_launch(const Attn8bParams &p, int G, int bs,
                                          cudaStream_t stream) {
  if (p.a.B * p.a.n_kv == 0) return cudaSuccess;
  if ((long long)p.a.MB * bs > 16 * cl8b::CH) return cudaErrorInvalidValue;
  return bs == 16   ? cl8b::launch_bs<16>(p, G, stream)
         : bs == 32 ? cl8b::launch_bs<32>(p, G, stream)
                    : cudaErrorInvalidValue;
}

}  // namespace pgd
