// cluster_attention_fp8b.cu -- decode attention over the block-scaled 8-bit
// cache on the CUDA cores, one cluster of 8 CTAs per (sequence, KV head).
//
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k_t) v_t,  t < ctx[b],
//   k_t = sk[tile] * E4M3(code), v_t = sv[tile] * E4M3(code)
//
// CTA r of a cluster takes the contiguous tokens [r ctx / 8, (r + 1) ctx / 8)
// in pieces of 64: two threads per token for q.k (64 dims each), an online
// softmax over the pieces (fp32, exact exp2), one thread per output dim for
// p.v from codes staged in shared memory.  The eight (max, sum, output)
// states are merged by log-sum-exp through distributed shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_fp8b.cuh"

namespace pgd {
namespace cl8b {

constexpr int CL = 8;         // CTAs per (sequence, KV head): one cluster
constexpr int CH = 64;        // tokens per piece
constexpr int THREADS = 128;  // = the head dim

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A load from CTA `rank`'s shared memory at the offset `local` has in ours.
__device__ __forceinline__ float ld_peer(const float *local, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

template <int G, int BS>
__global__ void __launch_bounds__(THREADS) cluster_attention_kernel(const Attn8bParams pp) {
  const AttnParams &p = pp.a;
  constexpr size_t TILE = (size_t)BS * kHeadDim;
  __shared__ __align__(16) float qs[G][kHeadDim];
  __shared__ __align__(16) unsigned char vs[CH][kHeadDim];  // V codes of a piece
  __shared__ float vsc[CH];                                 // their scales (0: no weight)
  __shared__ __align__(16) float ps[CH][G];                 // probabilities
  __shared__ float red[4][G];
  __shared__ float st_m[G], st_l[G], st_o[G][kHeadDim];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int unit = (int)blockIdx.x / CL;
  const int b = unit / p.n_kv, g = unit % p.n_kv;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = __ldg(p.ctx + b);
  const uint4 *qsrc = reinterpret_cast<const uint4 *>(p.q + ((size_t)b * p.n_q + g * G) * kHeadDim);
  for (int i = tid; i < G * 16; i += THREADS) {
    float f[8];
    unpack8(__ldg(qsrc + i), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) qs[i / 16][(i % 16) * 8 + e] = f[e];
  }
  const int32_t *trow = p.tables + (size_t)b * p.MB;
  const bool ctx_ok = ctx >= 1 && ctx <= p.MB * BS;
  if (!ctx_ok && tid == 0 && rank == 0 && g == 0) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
  const int n = ctx_ok ? ctx : 0;
  const int t_lo = (int)((long long)n * rank / CL), t_hi = (int)((long long)n * (rank + 1) / CL);
  __syncthreads();

  const int j = tid >> 1, hf = tid & 1;
  float m_run[G], l_run[G], o_acc[G];
#pragma unroll
  for (int h = 0; h < G; ++h) { m_run[h] = -INFINITY; l_run[h] = 0.f; o_acc[h] = 0.f; }
  bool bad = false;
  for (int tb = t_lo; tb < t_hi; tb += CH) {
    const int nt = min(CH, t_hi - tb);
    // K of token tb + j (this thread's 64 dims), V row 16 k + tid / 8, chunk tid % 8
    uint4 kr[4], vr[4];
    float ksc = 0.f, vscl = 0.f;
    const int t = tb + j;
    const int kblk = j < nt ? __ldg(trow + t / BS) : -1;
    const bool kval = (unsigned)kblk < (unsigned)p.NB;
    if (j < nt && !kval) bad = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) kr[k] = make_uint4(0, 0, 0, 0);
    if (kval) {
      const size_t tile = (size_t)kblk * p.n_kv + g;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        kr[k] = __ldg(reinterpret_cast<const uint4 *>(p.k_cache + tile * TILE +
                                                      code_offset8b(t % BS, 4 * hf + k)));
      ksc = __ldg(pp.k_scales + tile);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int jj = 16 * k + (tid >> 3), tv = tb + jj;
      vr[k] = make_uint4(0, 0, 0, 0);
      if (jj < nt) {
        const int blk = __ldg(trow + tv / BS);
        if ((unsigned)blk < (unsigned)p.NB)
          vr[k] = __ldg(reinterpret_cast<const uint4 *>(
              p.v_cache + ((size_t)blk * p.n_kv + g) * TILE + code_offset8b(tv % BS, tid & 7)));
      }
    }
    if (tid < nt) {
      const int blk = __ldg(trow + (tb + tid) / BS);
      if ((unsigned)blk < (unsigned)p.NB) vscl = __ldg(pp.v_scales + (size_t)blk * p.n_kv + g);
    }
    float s[G];
#pragma unroll
    for (int h = 0; h < G; ++h) s[h] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {kr[k].x, kr[k].y, kr[k].z, kr[k].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = __half22float2(e4m3x2_to_half2((uint16_t)(w[e >> 1] >> ((e & 1) * 16))));
        const int d = 64 * hf + 16 * k + 2 * e;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float2 q2 = *reinterpret_cast<const float2 *>(&qs[h][d]);
          s[h] = fmaf(q2.x, f.x, s[h]);
          s[h] = fmaf(q2.y, f.y, s[h]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4 *>(&vs[16 * k + (tid >> 3)][16 * (tid & 7)]) = vr[k];
    if (tid < CH) vsc[tid] = vscl;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      s[h] += __shfl_xor_sync(kFullMask, s[h], 1);
      s[h] = kval ? s[h] * ksc * p.qk_scale_log2 : -INFINITY;
      float m = s[h];
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
      if (lane == 0) red[warp][h] = m;
    }
    __syncthreads();
    float alpha[G], m_new[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float mc = fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h]));
      m_new[h] = fmaxf(m_run[h], mc);
      alpha[h] = m_run[h] == -INFINITY ? 0.f : exp2f(m_run[h] - m_new[h]);
      m_run[h] = m_new[h];
      if (hf == 0) ps[j][h] = s[h] == -INFINITY ? 0.f : exp2f(s[h] - m_new[h]);
    }
    __syncthreads();
    float acc[G], ls[G];
#pragma unroll
    for (int h = 0; h < G; ++h) { acc[h] = 0.f; ls[h] = 0.f; }
    for (int jj = 0; jj < nt; ++jj) {
      const __half hv = __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)vs[jj][tid], __NV_E4M3));
      const float v = __half2float(hv) * vsc[jj];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float pw = ps[jj][h];
        acc[h] = fmaf(pw, v, acc[h]);
        ls[h] += pw;
      }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      o_acc[h] = o_acc[h] * alpha[h] + acc[h];
      l_run[h] = l_run[h] * alpha[h] + ls[h];
    }
    __syncthreads();
  }
  if (bad) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
#pragma unroll
  for (int h = 0; h < G; ++h) st_o[h][tid] = o_acc[h];
  if (tid == 0) {
#pragma unroll
    for (int h = 0; h < G; ++h) { st_m[h] = m_run[h]; st_l[h] = l_run[h]; }
  }
  cluster_sync();
  if (tid < 16 * G) {
    const int h = tid / 16, d = (int)rank * 16 + (tid % 16);
    float mk[CL], lk[CL], ok[CL];
#pragma unroll
    for (int k = 0; k < CL; ++k) {
      mk[k] = ld_peer(&st_m[h], (uint32_t)k);
      lk[k] = ld_peer(&st_l[h], (uint32_t)k);
      ok[k] = ld_peer(&st_o[h][d], (uint32_t)k);
    }
    float M = mk[0];
#pragma unroll
    for (int k = 1; k < CL; ++k) M = fmaxf(M, mk[k]);
    float num = 0.f, den = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        const float w = mk[k] == -INFINITY ? 0.f : exp2f(mk[k] - M);
        num = fmaf(w, ok[k], num);
        den = fmaf(w, lk[k], den);
      }
    }
    p.out[((size_t)b * p.n_q + g * G + h) * kHeadDim + d] =
        __float2bfloat16_rn(den != 0.f ? num / den : 0.f);
  }
  cluster_sync();  // peers may still be reading this CTA's state
}

template <int G, int BS>
cudaError_t launch_g(const Attn8bParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.a.B * p.a.n_kv * CL));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cluster_attention_kernel<G, BS>, p);
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

cudaError_t cluster_attention_fp8b_launch(const Attn8bParams &p, int G, int bs,
                                          cudaStream_t stream) {
  if (p.a.B * p.a.n_kv == 0) return cudaSuccess;
  return bs == 16   ? cl8b::launch_bs<16>(p, G, stream)
         : bs == 32 ? cl8b::launch_bs<32>(p, G, stream)
                    : cudaErrorInvalidValue;
}

}  // namespace pgd
