// attention_fp8b.cu -- paged GQA decode attention over the block-scaled 8-bit
// cache (kv_fp8b.cuh) on the fifth-generation tensor cores, reading the codes
// as they lie: nothing is dequantised.
//
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k_t) v_t,  t < ctx[b],
//   k_t = sk[tile] * E4M3(code), v_t = sv[tile] * E4M3(code)
//
// The schedule (units, cost-balanced cuts over CTAs, last-arriver merge) and
// the bounded waits are those of attention_kernel.cuh, whose helpers this
// kernel uses; what differs is the arithmetic of a stage of 128 tokens, two
// E4M3 contractions with tokens on the M side (A) resp. the K side, fp32
// accumulators in tensor memory:
//   S^T[128 tok][16]   = Kc[128 tok][128 d]    . Q^T[128 d][16]
//   O^T[128 d][NP]    += Vc^T[128 d][128 tok]  . P^T[128 tok][NP]
//
// Scores.  Q carries each head as a high and a low E4M3 part (columns h and
// 8 + h), the bf16 query itself within 2^-17 of its largest element; the
// softmax adds the two columns and applies the query's and the block's scale.
//
// Probabilities.  An E4M3 number has four significant bits and no value
// between 0 and 2^-9, too few of either for a softmax weight.  But M = 128 by
// N = 16 leaves columns free, so a weight goes in as three E4M3 terms in three
// columns: x = hi + 2^-5 lo + 2^-10 lo2, each the rounding of what the terms
// before it leave, scaled up by 2^5.  A residual is at most 2^-4 of its term's
// binade, so three terms hold a weight to 2^-12 of itself, and to 2^-24 of
// the head's largest weight however small it is (hi alone ends at 2^-13).
// The epilogue adds the three columns.  (Two terms would hold 2^-8, but a
// context of 2^17 light tokens beside a heavy one needs the range: its weights
// are 2^-17 of the largest.)
//
// V's scale goes into the weight: x = 16 p sv.  So that x keeps its range
// whatever the blocks' scales, the running reference of a head is the maximum
// of log2(p sv) rather than of log2(p); the sum of p takes the same reference
// and stays exact in fp32, so outputs, partial states and their merge need no
// second one.  The reference moves when exceeded by 2^4: x <= 2^8, and 2^5
// times a residual of x stays within E4M3's 448.  Relative to it a sum of p is
// as large as 1 / sv: 2^100 for blocks of zeros.  Two references can lie further
// apart than the exponents of fp32 reach while both sums count alike, so a sum
// passes to another reference by two factors, each the root of the whole (an
// output, at most 2^8 times its tokens, has vanished where one factor does).
//
// Roles (512 threads): warps 0-3 and 12-15 softmax (thread t = token row t),
// 4 / 5 K / V producers, 6 q.k^T issuer, 7 p.v issuer, 8-11 query conversion,
// a segment ahead, and epilogue.  (The issuer's warp converting a query when its
// segment began held up the tensor cores: 51 contexts of 1800 tokens, G = 8:
// 51.8 us, 46.1 so.)  The two softmax groups take alternate stages, each with a
// reference, sums and an accumulator of its own that the epilogue merges: a
// stage's chain (barrier, tensor-memory load, vote, exponentials, conversions)
// is longer than the time HBM takes to deliver a stage, so one group alone sets
// the pace.  The K producer also fetches both scales of every block of a stage
// into a 16-stage ring by 4-byte asynchronous copies that count on the stage's
// own barrier, so no warp waits for a dependent load.
//
// Start.  What lies between the wait for the previous kernel and the first
// copy is on the path of every call (6 us of it at first), so it is kept to
// the context lengths, one scan, 32-bit arithmetic and the block ids, which
// are guessed and loaded beside the lengths; the query is converted beside the
// first copies.
#include <cuda.h>

#include <atomic>

#include "attention_kernel.cuh"
#include "kv_fp8b.cuh"

namespace pgd {
namespace tc8b {

using namespace tc;

// The launch's parameters: pools of 16-token tiles also as tensors of NB * n_kv
// rows (tiles) of 256 8-byte elements, read in boxes of one row.
struct Params {
  Attn8bParams q8;
  float split_root;  // parts of a split by its cost X: split_root * sqrt(X)
  float inv_units;   // 1 / (B * n_kv)
  float starts;      // B * n_kv * kSegCost
  CUtensorMap k_map, v_map;
};

constexpr int NTHREADS = 512;
constexpr int WARP_SM1 = 12;            // warps of the second softmax group
constexpr uint32_t TMEM_COLS8 = 256;   // S 4 x 16; O 2 x 2 x 32 from column 64
constexpr int GROUP = kGroupBytes8b;   // bytes of 8 tokens
constexpr int STAGE = TOK * kHeadDim;  // K (or V) codes of a stage
constexpr int NSK = 5, NSV = 5;        // ring depths (3, 4 and 6 stages: 350, 342, 351 us where 5
                                       // take 344 on 64 ragged contexts)
constexpr int NSR = 16;                // stages of scales
constexpr int Q_BYTES = NPAD * 128;    // 16 E4M3 rows as 8 x 16-byte core matrices
constexpr float kMoveLog2 = 4.f;       // move the reference when exceeded by 2^4
constexpr float kWeightUnit = 16.f;    // x = 16 p sv
constexpr float kTerm = 32.f;          // a term's residual is scaled by 2^5

// Columns of P and O: term i of head h in column i * TS + h.
template <int G> constexpr int TS = G <= 4 ? 4 : 8;
template <int G> constexpr int NP = G <= 4 ? 16 : 32;
constexpr int P_BYTES8 = TOK * 32;     // a P buffer (NP = 32; NP = 16 uses half)

constexpr int OFF_K = 0;
constexpr int OFF_V = OFF_K + NSK * STAGE;
constexpr int OFF_Q = OFF_V + NSV * STAGE;  // double buffered by segment parity
constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;  // double buffered by stage parity
constexpr int OFF_SC = OFF_P + 2 * P_BYTES8;           // f32 [NSR][2][8] (K, V) scales
constexpr int OFF_BAR = OFF_SC + NSR * 2 * 8 * 4;
constexpr int OFF_RED = OFF_BAR + 512;                 // f32 [group][2][4][8] warp maxima
constexpr int OFF_LRED = OFF_RED + 2 * 2 * 4 * 8 * 4;  // f32 [2][group][4][8] warp sums
constexpr int OFF_MREF = OFF_LRED + 2 * 2 * 4 * 8 * 4;  // f32 [2][group][8] references
constexpr int OFF_QS = OFF_MREF + 2 * 2 * 8 * 4;           // f32 [NQS][8] query scales
constexpr int NQS = 2;  // (by segment parity, like the queries)
constexpr int OFF_MISC = OFF_QS + NQS * 8 * 4;
constexpr int OFF_PRE = OFF_MISC + 256;                // int [B + 1]

constexpr size_t smem_size(int B) { return (size_t)SMEM_SLACK + OFF_PRE + (size_t)(B + 1) * 4; }
static_assert(smem_size(PGD_MAX_BATCH) <= 232448, "layout exceeds 227 KB");
static_assert((OFF_MISC + 24) % 8 == 0, "WaitCtl alignment");
// The scales and the invalid-block mask of stage s are written when it is
// armed, after the q.k^T of stage s - NSK has completed and so (S buffers)
// after the softmax has read those of stage s - NSK - NSB.
static_assert(NSR >= NSK + NSB && (NSR & (NSR - 1)) == 0, "scale and mask rings");
static_assert(40 + 4 * NSR <= 112 && OFF_MISC % 16 == 0, "misc layout");

// One CTA streams at most about 1/kShare of the HBM rate (128 of 152 CTAs take
// the whole of it: 0.58 us a stage).
constexpr float kShare = 126.f;
template <int BS> constexpr float kBlockBytes = 2.f * BS * kHeadDim;
constexpr int MERGE_U = 5;  // parts of a unit that a merging warp has in flight

// kind::f8f6f4, D f32, A and B E4M3, both MN-major, M = 128.
__host__ __device__ constexpr uint32_t idesc_pv(int n) {
  return (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(TOK >> 4) << 24);
}

// 4 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy4_async(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Four 2 KiB tiles into `dst`, one behind the other: rows t0 .. t3 of the pool
// as a two-dimensional tensor.  A row outside the pool arrives as zeros.
__device__ __forceinline__ void gather_tiles(void *dst, const CUtensorMap *map, int t0, int t1,
                                             int t2, int t3, uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(0), "r"(t0), "r"(t1), "r"(t2), "r"(t3), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
// Arrive on `bar` (one of its expected arrivals) once this thread's earlier
// asynchronous copies have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// The CTAs' parts of the cost space of attention_kernel.cuh, in 32 bits (the
// host refuses calls whose cost space does not fit): whole units, or parts of
// one size.
struct Cuts {
  int X, P, S;     // cost of all units, parts, cost of a part (but the last)
  bool units;      // part c = unit c
  const int *pre;  // cost of one head of the sequences before b
  int n_kv, ov;
};

struct Piece {  // blocks j0 .. j0 + n - 1 of the nblk of unit (b, g), at cost [ucs, uce)
  int b, g, j0, nblk, n, ucs, uce;
};

// A CTA's place in its part: what is left of it, and the last unit.
struct Walk {
  int x, end, b, g;
};
// Largest b with n_kv * pre[b] <= x.  Out of line: one copy for all roles.
__device__ __noinline__ int find_sequence(const int *pre, int n_kv, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (n_kv * pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// (g: one before the first unit)
__device__ __forceinline__ void walk_start(const Cuts &sc, int B, Walk &w) {
  w.x = (int)min((long long)sc.X, (long long)blockIdx.x * sc.S);
  w.end = (int)min((long long)sc.X, (long long)w.x + sc.S);
  if (w.x >= w.end) return;
  w.b = find_sequence(sc.pre, sc.n_kv, B, w.x);
  w.g = (w.x - sc.n_kv * sc.pre[w.b]) / (sc.pre[w.b + 1] - sc.pre[w.b]) - 1;
}
// Part c of a split into whole units: unit c, if it has blocks.
__device__ __forceinline__ bool whole_unit(const Cuts &sc, int b, Piece &sg) {
  const int c = (int)blockIdx.x;
  if (c >= sc.P) return false;
  sg.b = b;
  sg.g = c - b * sc.n_kv;
  const int cost = sc.pre[sg.b + 1] - sc.pre[sg.b];
  sg.j0 = 0;
  sg.nblk = sg.n = cost - sc.ov;
  sg.ucs = sc.n_kv * sc.pre[sg.b] + sg.g * cost;
  sg.uce = sg.ucs + cost;
  return cost > 0;
}
// The next segment.  (Inlined into every role, its state in registers: out of
// line the state went through local memory, 3000 cycles at every change of unit.)
__device__ __forceinline__ bool walk_next(const int *pre, int n_kv, int ov, int B, Walk &w,
                                          Piece &sg) {
#pragma unroll 1
  while (w.x < w.end) {
    if (++w.g == n_kv) {
      w.g = 0;
#pragma unroll 1
      do { ++w.b; } while (w.b < B - 1 && pre[w.b + 1] == pre[w.b]);
    }
    const int cost = pre[w.b + 1] - pre[w.b];
    const int ucs = n_kv * pre[w.b] + w.g * cost, uce = ucs + cost;
    const int e = min(w.end, uce);
    const int j0 = max(0, w.x - ucs - ov), j1 = max(0, e - ucs - ov);
    w.x = e;
    if (j1 > j0) {
      sg.b = w.b;
      sg.g = w.g;
      sg.j0 = j0;
      sg.nblk = cost - ov;
      sg.n = j1 - j0;
      sg.ucs = ucs;
      sg.uce = uce;
      return true;
    }
  }
  return false;
}
// Block ids of a segment: entries lane and 32 + lane of what is left of it.
struct Ids {
  int tab, tab_next;
};
__device__ __forceinline__ Ids load_ids(const AttnParams &p, const Piece &g, int lane) {
  const int32_t *trow = p.tables + (size_t)g.b * p.MB + g.j0;
  Ids a;
  a.tab = (lane < g.n) ? __ldg(trow + lane) : 0;
  a.tab_next = (32 + lane < g.n) ? __ldg(trow + 32 + lane) : 0;
  return a;
}

// One producer warp: walks the CTA's stages.  Tiles of 16 tokens come four at
// a time by two gathers a stage (a bulk copy a tile, one lane each, costs the
// warp about 100 cycles a copy: 1200 a stage of eight, as long as HBM takes to
// deliver it); in the place of absent blocks of a last stage and of blocks
// whose id is bad, tile 0 is read, and its rows take no weight.  Tiles of 32
// tokens come by a bulk copy each (a gather's rows end at 2 KiB: 4 KiB tiles
// in two halves took 343 us where whole ones take 335 on 64 ragged contexts).
// The K producer also copies the blocks' scales and records which blocks of a
// stage had an invalid id.  Block ids are loaded one step ahead; `ids` has
// those of the first segment.
template <int BS, bool IS_K>
__device__ __forceinline__ void produce(const Params &pr, const Cuts &sc, Walk w, Piece sg,
                                        bool have, Ids ids, unsigned char *smem, uint64_t *full,
                                        uint64_t *empty, volatile int *stage_mask,
                                        volatile int *abort_flag, uint64_t policy, int lane) {
  const Attn8bParams &pp = pr.q8;
  const AttnParams &p = pp.a;
  constexpr int SB = TOK / BS;
  constexpr int NS = IS_K ? NSK : NSV;
  constexpr bool GATHER = BS == 16;
  constexpr uint32_t TILE = BS * kHeadDim;
  const CUtensorMap *map = IS_K ? &pr.k_map : &pr.v_map;
  const unsigned char *cache = IS_K ? p.k_cache : p.v_cache;
  unsigned char *ring = smem + (IS_K ? OFF_K : OFF_V);
  const uint32_t sring = smem_addr(smem + OFF_SC);
  if (p.wait_late == 1) pdl_wait();  // the append has written the cache
  int s = 0, slot = 0;
  uint32_t phase = 1;  // (the ring starts empty)
  bool stop = false;
  while (have && !stop) {
    bool have_next = false;
    Piece nsg{};
    Ids next_ids{};
    const int32_t *trow = p.tables + (size_t)sg.b * p.MB + sg.j0;
    int tab = ids.tab, tab_next = ids.tab_next;
    int tchunk = 0;
    const int nstages = (sg.n + SB - 1) / SB;
    for (int st = 0; st < nstages; ++st, ++s) {
      const int first = st * SB;
      if ((first >> 5) != tchunk) {
        tchunk = first >> 5;
        tab = tab_next;
        const int j = (tchunk + 1) * 32 + lane;
        tab_next = (j < sg.n) ? __ldg(trow + j) : 0;
      }
      const int nb = min(SB, sg.n - first);
      const int blk = __shfl_sync(kFullMask, tab, (first & 31) + (lane & (SB - 1)));
      const bool ok = lane < nb && (unsigned)blk < (unsigned)p.NB;
      const unsigned okmask = __ballot_sync(kFullMask, ok);
      const int tile = ok ? blk * p.n_kv + sg.g : 0;
      unsigned char *dst = ring + (size_t)slot * STAGE;
      int rows[SB];
      if constexpr (GATHER) {
#pragma unroll
        for (int i = 0; i < SB; ++i) rows[i] = __shfl_sync(kFullMask, tile, i);
      }
      int go = 1;
      if (lane == 0) {
        wait_or_abort(&empty[slot], phase, abort_flag, p.err);
        go = *abort_flag ? 0 : 1;
        if (go) {
          if (IS_K) {
            const unsigned bad = ((1u << nb) - 1u) & ~okmask;
            stage_mask[s & (NSR - 1)] = (int)bad;
            if (bad) atomicOr(p.err, PGD_DEVERR_BAD_BLOCK_ID);
          }
          if constexpr (GATHER) {
            mbar_arrive_expect_tx(&full[slot], STAGE);
            gather_tiles(dst, map, rows[0], rows[1], rows[2], rows[3], &full[slot], policy);
            gather_tiles(dst + STAGE / 2, map, rows[SB - 4], rows[SB - 3], rows[SB - 2],
                         rows[SB - 1], &full[slot], policy);
          } else if (okmask) {
            mbar_arrive_expect_tx(&full[slot], (uint32_t)__popc(okmask) * TILE);
          } else {
            mbar_arrive(&full[slot]);
          }
        }
      }
      // (one decision for the warp: after a timeout nothing more is armed)
      if (!__shfl_sync(kFullMask, go, 0)) {
        stop = true;
        break;
      }
      if (!GATHER && ok)
        bulk_copy_g2s(dst + (size_t)lane * TILE, cache + (size_t)tile * TILE, TILE, &full[slot],
                      policy);
      if (IS_K) {
        if (ok) {
          const uint32_t at = sring + (uint32_t)(((s & (NSR - 1)) * 16 + lane) * 4);
          copy4_async(at, pp.k_scales + tile);
          copy4_async(at + 32, pp.v_scales + tile);
        }
        arrive_after_copies(&full[slot]);
      }
      if (st == 0) {  // the next segment's ids, once this one's copies have begun
        have_next = walk_next(sc.pre, sc.n_kv, sc.ov, p.B, w, nsg);
        if (have_next) next_ids = load_ids(p, nsg, lane);
      }
      if (++slot == NS) {
        slot = 0;
        phase ^= 1u;
      }
    }
    sg = nsg;
    ids = next_ids;
    have = have_next;
  }
  // no copy may still be landing when the CTA exits
  if (lane == 0) {
    for (int i = 1; i <= NS && i <= s; ++i) {
      const int last = s - i;
      if (!mbar_wait_bounded(&full[last % NS], (uint32_t)(last / NS) & 1u))
        atomicOr(p.err, PGD_DEVERR_TIMEOUT);
    }
  }
}

// A segment's query rows by the 128 epilogue threads: thread e takes 16 bytes
// (piece c of row r) and writes them as E4M3, high parts in rows 0-7 and low
// parts in rows 8-15 of the B operand, with one power-of-two scale a head.
template <int G>
__device__ __forceinline__ void convert_query(const AttnParams &p, const Piece &g,
                                              unsigned char *qdst, float *qscale, int e) {
  const int r = e >> 4, c = e & 15;
  uint4 q = make_uint4(0, 0, 0, 0);
  if (r < G)
    q = __ldg(reinterpret_cast<const uint4 *>(p.q + q_index(p, g.b, g.g, r) * kHeadDim + c * 8));
  float f[8];
  unpack8(q, f);
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
  // the scale 2^(x - 7), x the largest element's exponent: the elements
  // keep their bits and the largest lands in [128, 256)
  const int x = max((int)((__float_as_uint(a) >> 23) & 0xffu) - 127, -119);
  if (r < G) {
    uint2 hi, lo;
    q_hi_lo(q, pow2f(7 - x), hi, lo);
    const int off = (c >> 1) * 128 + (c & 1) * 8;
    *reinterpret_cast<uint2 *>(qdst + r * 16 + off) = hi;
    *reinterpret_cast<uint2 *>(qdst + 8 * 128 + r * 16 + off) = lo;
    if (c == 0) qscale[r] = pow2f(x - 7);
  }
  fence_proxy_async();
  __syncwarp();
}

// The root of the factor that takes a state from reference m to M >= m (0 for a
// state without a reference).
__device__ __forceinline__ float to_reference_root(float m, float M) {
  return m == -INFINITY ? 0.f : exp2_approx(0.5f * (m - M));
}

// A unit's partial states (unit, first part, parts) merged by log-sum-exp into
// its output rows by the whole CTA.  Warp w takes head w % G and every
// (16 / G)-th part: lane i holds the weight of its i-th part, four dims a lane,
// the loads of MERGE_U parts and of the weights in flight together; the warps'
// states then meet in shared memory.  (19 parts of 4 heads by a thread for each
// dim, which computes every weight itself: 4400 cycles.)
template <int G>
__device__ __forceinline__ void merge_unit(const AttnParams &p, const int4 &m, float *scratch,
                                           int tid) {
  constexpr int NG = NTHREADS / 32 / G;  // warps a head
  constexpr int ROW = kHeadDim + 4;      // a warp's outputs, maximum, sum
  const int lane = tid & 31, warp = tid >> 5, h = warp % G, first = warp / G;
  const size_t row0 = ((size_t)m.x + (size_t)m.y) * G + h;
  float M = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c0 = first; c0 < m.z; c0 += 32 * NG) {
    const int cnt = min(32, (m.z - c0 + NG - 1) / NG);
    float4 o[MERGE_U];
    auto load = [&](int j0) {
#pragma unroll
      for (int k = 0; k < MERGE_U; ++k) {
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + k < cnt)
          o[k] = __ldcg(reinterpret_cast<const float4 *>(
                            p.part_o + (row0 + (size_t)(c0 + NG * (j0 + k)) * G) * kHeadDim) +
                        lane);
      }
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < cnt)
      ml = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + row0 +
                  (size_t)(c0 + NG * lane) * G);
    load(0);
    float mx = ml.x;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, x));
    mx = fmaxf(mx, M);
    const float c_root = to_reference_root(M, mx), c = c_root * c_root;
    const float f_root = to_reference_root(ml.x, mx), f = f_root * f_root;
    float l = f_root * ml.y * f_root;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(kFullMask, l, x);
    L = fmaf(L * c_root, c_root, l);
    M = mx;
    O.x *= c, O.y *= c, O.z *= c, O.w *= c;
#pragma unroll 1
    for (int j0 = 0;;) {
#pragma unroll
      for (int k = 0; k < MERGE_U; ++k) {
        const float fk = __shfl_sync(kFullMask, f, j0 + k);  // (past cnt: o is 0)
        O.x = fmaf(fk, o[k].x, O.x);
        O.y = fmaf(fk, o[k].y, O.y);
        O.z = fmaf(fk, o[k].z, O.z);
        O.w = fmaf(fk, o[k].w, O.w);
      }
      if ((j0 += MERGE_U) >= cnt) break;
      load(j0);
    }
  }
  float *mine = scratch + warp * ROW;
  *reinterpret_cast<float4 *>(mine + 4 * lane) = O;
  if (lane == 0) {
    mine[kHeadDim] = M;
    mine[kHeadDim + 1] = L;
  }
  __syncthreads();
  const size_t obase = q_index(p, m.x / p.n_kv, m.x % p.n_kv, 0) * kHeadDim;
#pragma unroll
  for (int i = 0; i < (G * kHeadDim + NTHREADS - 1) / NTHREADS; ++i) {
    const int at = tid + i * NTHREADS;
    if (at >= G * kHeadDim) break;
    const float *s = scratch + at / kHeadDim * ROW;
    float mx = s[kHeadDim];
#pragma unroll
    for (int k = 1; k < NG; ++k) mx = fmaxf(mx, s[k * G * ROW + kHeadDim]);
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float *r = s + k * G * ROW;
      const float root = to_reference_root(r[kHeadDim], mx);
      den = fmaf(root * r[kHeadDim + 1], root, den);
      num = fmaf(root * root, r[at % kHeadDim], num);
    }
    p.out[obase + at] = __float2bfloat16_rn(num / den);
  }
}

template <int G, int BS>
__global__ void __launch_bounds__(NTHREADS, 1)
attention_fp8b_kernel(const __grid_constant__ Params pr) {
  const AttnParams &p = pr.q8.a;
  constexpr int SB = TOK / BS;
  constexpr int NCOL = NP<G>, TSTEP = TS<G>;
  constexpr int PROW = NCOL;             // bytes of a token's weights
  constexpr uint32_t PGRP = 8 * PROW;    // bytes of 8 tokens' weights
  constexpr uint32_t IDESC_QK = instr_desc_e4m3();
  constexpr uint32_t IDESC_PV = idesc_pv(NCOL);

  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + OFF_BAR);
  uint64_t *full_k = bars;              // [NSK]
  uint64_t *empty_k = full_k + NSK;     // [NSK]
  uint64_t *full_v = empty_k + NSK;     // [NSV]
  uint64_t *empty_v = full_v + NSV;     // [NSV]
  uint64_t *s_full = empty_v + NSV;     // [NSB]
  uint64_t *s_free = s_full + NSB;      // [NSB]
  uint64_t *m_ready = s_free + NSB;     // [NSB]
  uint64_t *p_full = m_ready + NSB;     // [2]
  uint64_t *p_free = p_full + 2;        // [2]
  uint64_t *o_full = p_free + 2;        // [2]
  uint64_t *o_free = o_full + 2;        // [2]
  uint64_t *done = o_free + 2;          // [2]
  uint64_t *seg_done = done + 2;        // [2]
  uint64_t *q_ready = seg_done + 2;     // [2]
  float *red = reinterpret_cast<float *>(smem + OFF_RED);
  float *lred = reinterpret_cast<float *>(smem + OFF_LRED);
  float *mref = reinterpret_cast<float *>(smem + OFF_MREF);
  float *qscale = reinterpret_cast<float *>(smem + OFF_QS);
  const float *scl = reinterpret_cast<const float *>(smem + OFF_SC);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
  int *n_merges = reinterpret_cast<int *>(smem + OFF_MISC + 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + OFF_MISC + 24);  // WaitCtl
  volatile int *stage_mask = reinterpret_cast<volatile int *>(smem + OFF_MISC + 40);  // [NSR]
  int *over_flag = reinterpret_cast<int *>(smem + OFF_MISC + 112);  // [group][2][4] votes
  int4 *merges = reinterpret_cast<int4 *>(smem + OFF_MISC + 176);  // [2] unit, first part, parts
  int2 *warp_sum = reinterpret_cast<int2 *>(smem + OFF_RED);  // (before the softmax)
  int *pre = reinterpret_cast<int *>(smem + OFF_PRE);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The next kernel of the stream may take this one's place CTA by CTA; like
  // this one it waits for its predecessor before it reads memory.
  pdl_launch_dependents();
  if (warp == 0) {
    // Arrivals a barrier expects, in the order of the arrays above: 33 = the
    // producer's and each lane's scale copies, 4 and 8 = softmax or epilogue
    // warps.
    constexpr int N_BARS = 2 * NSK + 2 * NSV + 3 * NSB + 7 * 2;
    static_assert(N_BARS * 8 <= 512, "barriers");
    for (int i = lane; i < N_BARS; i += 32) {
      constexpr int S0 = 2 * NSK + 2 * NSV, P0 = S0 + 3 * NSB;
      uint32_t n = 1;
      if (i < NSK) n = 1 + 32;                          // full_k
      else if (i >= S0 + NSB && i < S0 + 2 * NSB) n = 4;  // s_free
      else if (i >= P0 && i < P0 + 2) n = 4;            // p_full
      else if (i >= P0 + 6 && i < P0 + 8) n = 4;        // o_free
      else if (i >= P0 + 10 && i < P0 + 12) n = 8;      // seg_done
      else if (i >= P0 + 12) n = 4;                     // q_ready
      mbar_init(&bars[i], n);
    }
    mbar_init_fence();
    if (lane == 0) {
      *n_merges = 0;
      init_wait_ctl(smem + OFF_MISC + 24, p.wait_limit_ns);
    }
  }
  // Query rows and weight columns that belong to no head stay zero.
  {
    uint4 *z = reinterpret_cast<uint4 *>(smem + OFF_Q);
    for (int i = tid; i < (2 * Q_BYTES + 2 * P_BYTES8) / 16; i += NTHREADS)
      z[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
  }
  const int unit_b = (int)blockIdx.x / p.n_kv;  // CTA c's unit in a split into whole units
  uint64_t policy = 0;
  if (warp == WARP_KP || warp == WARP_VP) {
    policy = l2_policy_evict_first();
    if (BS == 16 && lane == 0)
      asm volatile("prefetch.tensormap [%0];" ::"l"(warp == WARP_KP ? &pr.k_map : &pr.v_map)
                   : "memory");
  }
  if (warp == WARP_QK) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(TMEM_COLS8)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Everything above touches only this CTA's own memory; what follows reads
  // the caller's.
  if (!p.wait_late) pdl_wait();
  // The producers' guess: CTA c streams unit c from its first block (so it
  // does with no more units than CTAs, unless the units are cut).
  int guess_b = -1;
  Ids guess{};
  if ((warp == WARP_KP || warp == WARP_VP) && unit_b < p.B) {
    guess_b = unit_b;
    const int32_t *trow = p.tables + (size_t)guess_b * p.MB;
    if (lane < p.MB) guess.tab = __ldg(trow + lane);
    if (32 + lane < p.MB) guess.tab_next = __ldg(trow + 32 + lane);
  }
  // Cost of every sequence's blocks and its prefix over the batch.
  const int max_tokens = p.MB * BS;
  auto cost_of = [&](int b, bool report) {
    const int c = __ldg(p.ctx + b);
    if (c >= 1 && c <= max_tokens) return (c + BS - 1) / BS + kSegCost<BS>;
    if (report) atomicOr(p.err, PGD_DEVERR_BAD_CONTEXT);
    return 0;
  };
  int longest = 0;
  if (p.B <= 32) {  // by every warp for itself: no barrier (0.4 us of every call)
    int upto = 0;
    if (lane < p.B) upto = longest = cost_of(lane, blockIdx.x == 0 && warp == 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += v;
    }
    longest = __reduce_max_sync(kFullMask, longest);
    if (lane < p.B) pre[lane + 1] = upto;
    if (lane == 0) pre[0] = 0;
    __syncwarp();
  } else {  // thread t takes `per` sequences from t * per
    const int per = (p.B + NTHREADS - 1) / NTHREADS;
    const int b_end = min(p.B, (tid + 1) * per);
    int sum = 0;
#pragma unroll 1
    for (int b = tid * per; b < b_end; ++b) {
      const int cost = cost_of(b, blockIdx.x == 0);
      sum += cost;
      longest = max(longest, cost);
      pre[b + 1] = sum;
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += v;
    }
    longest = __reduce_max_sync(kFullMask, longest);
    if (lane == 31) warp_sum[warp] = make_int2(upto, longest);
    __syncthreads();
    int before = upto - sum;
#pragma unroll
    for (int w = 0; w < NTHREADS / 32; ++w) {
      const int2 v = warp_sum[w];
      if (w < warp) before += v.x;
      longest = max(longest, v.y);
    }
#pragma unroll 1
    for (int b = tid * per; b < b_end; ++b) pre[b + 1] += before;
    if (tid == 0) pre[0] = 0;
    __syncthreads();
  }
  auto col_o = [&](int ob, int grp) { return tmem + 64u + (uint32_t)(ob * 2 + grp) * 32u; };

  // The split: whole units, or balanced cuts (the cost model of
  // attention_kernel.cuh with this cache's bytes per block).
  Cuts sc;
  sc.X = p.n_kv * pre[p.B];
  sc.pre = pre;
  sc.n_kv = p.n_kv;
  sc.ov = kSegCost<BS>;
  sc.P = min(sc.X, (int)gridDim.x);
  sc.units = false;
  if (p.auto_split && sc.X > 0) {
    // (approximate functions: the same in every thread, which is all it takes)
    const int U = p.B * p.n_kv;
    constexpr float m0 = (float)kMergeFixedBytes / kBlockBytes<BS>;
    constexpr float m1 = (float)kMergePartBytes / kBlockBytes<BS>;
    const float X = (float)sc.X;
    float root;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(X));
    const int P = max(1, min(sc.P, (int)(pr.split_root * root)));
    // (what HBM has to deliver is without the units' starts, and so is a CTA's
    // only unit, which begins as the call does)
    const float bytes = X - pr.starts;
    const float cost_cut = fmaxf(__fdividef(X, (float)P) * kShare, bytes) + m0 +
                           m1 * ceilf((float)P * pr.inv_units);
    sc.P = P;
    if (U <= (int)gridDim.x &&
        fmaxf(fmaf((float)longest, kShare, -kSegCost<BS> * kShare), bytes) <= cost_cut) {
      sc.units = true;
      sc.P = U;
    }
  }

  // Every role walks the same segments; the first is found once.
  Walk walk{};
  Piece sg{};
  bool have;
  if (sc.units) {
    have = whole_unit(sc, unit_b, sg);
  } else {
    sc.S = sc.P > 0 ? (sc.X - 1) / sc.P + 1 : 1;  // (X + P may not fit 32 bits)
    walk_start(sc, p.B, walk);
    have = walk_next(pre, sc.n_kv, sc.ov, p.B, walk, sg);
  }
  if ((warp == WARP_KP || warp == WARP_VP) && have && !(sg.b == guess_b && sg.j0 == 0))
    guess = load_ids(p, sg, lane);
  auto next = [&](Piece &g) { return walk_next(pre, sc.n_kv, sc.ov, p.B, walk, g); };

  if (warp == WARP_KP) {
    produce<BS, true>(pr, sc, walk, sg, have, guess, smem, full_k, empty_k, stage_mask,
                      abort_flag, policy, lane);
  } else if (warp == WARP_VP) {
    produce<BS, false>(pr, sc, walk, sg, have, guess, smem, full_v, empty_v, nullptr, abort_flag,
                       policy, lane);
  } else if (warp == WARP_QK) {
    // ------------------------------------------------------ q.k^T issuer
    if (lane == 0) {
      int s = 0, k = 0, slot = 0;
      uint32_t phase = 0;
      while (have) {
        const int nstages = (sg.n + SB - 1) / SB;
        wait_or_abort(&q_ready[k & 1], (uint32_t)(k >> 1) & 1u, abort_flag, p.err);
        const uint64_t qd =
            smem_desc(smem_addr(smem + OFF_Q + (k & 1) * Q_BYTES), 128, 1024, 0);
        for (int st = 0; st < nstages; ++st) {
          const int su = s + st, sb = su % NSB;
          wait_or_abort(&full_k[slot], phase, abort_flag, p.err);
          wait_or_abort(&s_free[sb], ((uint32_t)(su / NSB) & 1u) ^ 1u, abort_flag, p.err);
          tc_fence_after();
          if (!*abort_flag) {
            // K core matrices 128 B apart along d, token groups 1024 B apart;
            // a k-step of 32 dims moves K and Q by two core matrices
            const uint64_t kd = smem_desc(smem_addr(smem + OFF_K + slot * STAGE), 128, GROUP, 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_e4m3(tmem + col_s(sb), kd + (uint64_t)(kk * 16), qd + (uint64_t)(kk * 16),
                        IDESC_QK, kk > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[sb]);
          umma_commit(&empty_k[slot]);
          // the stage's invalid-block mask and scales, which full_k ordered
          // before this, and the query's scales, for the softmax
          mbar_arrive(&m_ready[sb]);
          if (++slot == NSK) {
            slot = 0;
            phase ^= 1u;
          }
        }
        s += nstages;
        ++k;
        have = next(sg);
      }
      if (s > 0) {
        umma_commit(&done[0]);
        mbar_wait_bounded(&done[0], 0);
      }
    }
  } else if (warp == WARP_PV) {
    // ------------------------------------------------------- p.v issuer
    if (lane == 0) {
      int s = 0, k = 0, slot = 0;
      uint32_t phase = 0;
      while (have) {
        const int nstages = (sg.n + SB - 1) / SB;
        const int ob = k & 1;
        for (int st = 0; st < nstages; ++st, ++s) {
          const int sb = s & 1;
          wait_or_abort(&p_full[sb], (uint32_t)(s >> 1) & 1u, abort_flag, p.err);
          wait_or_abort(&full_v[slot], phase, abort_flag, p.err);
          if (st == 0)
            wait_or_abort(&o_free[ob], ((uint32_t)(k >> 1) & 1u) ^ 1u, abort_flag, p.err);
          tc_fence_after();
          if (!*abort_flag) {
            // V: dims (M) 128 B apart in chunks of 16, token groups (K)
            // 1024 B apart; P: columns (N) 128 B apart in chunks of 16, token
            // groups PGRP apart; a k-step is 32 token rows
            const uint64_t vd = smem_desc(smem_addr(smem + OFF_V + slot * STAGE), GROUP, 128, 0);
            const uint64_t pd = smem_desc(smem_addr(smem + OFF_P + sb * P_BYTES8), PGRP, 128, 0);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
              umma_e4m3(col_o(ob, sb), vd + (uint64_t)(kt * (4 * GROUP / 16)),
                        pd + (uint64_t)(kt * (4 * PGRP / 16)), IDESC_PV,
                        (kt > 0 || st > 1) ? 1u : 0u);
          }
          umma_commit(&empty_v[slot]);
          umma_commit(&p_free[sb]);
          if (st + 1 == nstages) umma_commit(&o_full[ob]);
          if (++slot == NSV) {
            slot = 0;
            phase ^= 1u;
          }
        }
        ++k;
        have = next(sg);
      }
      if (s > 0) {
        umma_commit(&done[1]);
        mbar_wait_bounded(&done[1], 0);
      }
    }
  } else if (warp < 4 || warp >= WARP_SM1) {
    // ----------------------------------------------------------- softmax
    // Group grp takes the stages s with s % 2 == grp.
    const int grp = warp < 4 ? 0 : 1;
    const int t = tid & 127, gw = warp & 3;
    const uint32_t lane_base = (uint32_t)(gw * 32) << 16;
    constexpr int NCT = 128;
    float *gred = red + grp * 2 * 4 * 8;
    int *gvote = over_flag + grp * 2 * 4;
    const int tblk = t / BS;  // the stage's block of row t
    Piece nsg;
    int s = 0, k = 0, it = 0;  // s: the segment's first stage
    int ctx_b = have ? __ldg(p.ctx + sg.b) : 0;
    while (have) {
      const bool have_next = next(nsg);
      const int ctx_n = have_next ? __ldg(p.ctx + nsg.b) : 0;
      const int nstages = (sg.n + SB - 1) / SB;
      const int ob = k & 1;
      const int st0 = (s & 1) == grp ? 0 : 1;  // this group's first stage
      float m_ref[G], l_part[G], qsc[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m_ref[h] = -INFINITY;
        l_part[h] = 0.f;
        qsc[h] = 0.f;
      }
      for (int st = st0; st < nstages; st += 2, ++it) {
        const int su = s + st, sbu = su % NSB;
        wait_or_abort(&s_full[sbu], (uint32_t)(su / NSB) & 1u, abort_flag, p.err);
        wait_or_abort(&m_ready[sbu], (uint32_t)(su / NSB) & 1u, abort_flag, p.err);
        const int msk = stage_mask[su & (NSR - 1)];
        const int nb = min(SB, sg.n - st * SB);
        int nvalid = nb * BS;
        if (sg.j0 + st * SB + nb == sg.nblk) nvalid -= sg.nblk * BS - ctx_b;
        const bool valid = (t < nvalid) && !((msk >> tblk) & 1);
        const float ks = scl[(su & (NSR - 1)) * 16 + tblk];
        const float vs = scl[(su & (NSR - 1)) * 16 + 8 + tblk];
        if (st == st0) {
#pragma unroll
          for (int h = 0; h < G; ++h) qsc[h] = qscale[(k & (NQS - 1)) * 8 + h] * p.qk_scale_log2;
        }
        tc_fence_after();
        uint32_t sv[16];
        tmem_ld8_async(tmem + lane_base + col_s(sbu), sv);
        tmem_ld8_async(tmem + lane_base + col_s(sbu) + 8, sv + 8);
        tmem_wait8(sv);
        tmem_wait8(sv + 8);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[sbu]);
        // scores in log2 units, and with the V scale's logarithm the weights
        // that the reference bounds (a row that is not valid has w = -inf;
        // 2^-120 keeps the logarithm finite whatever the ring holds)
        const float lv = __log2f(fmaxf(vs, 0x1p-120f));
        float w[G];
#pragma unroll
        for (int h = 0; h < G; ++h)
          w[h] = valid ? (__uint_as_float(sv[h]) + __uint_as_float(sv[8 + h])) * (qsc[h] * ks)
                       : -INFINITY;
        const int rb = it & 1;
        bool move = true;  // (a segment's first stage always sets it)
        if (st > st0) {
          bool over = false;
#pragma unroll
          for (int h = 0; h < G; ++h) over |= w[h] + lv > m_ref[h] + kMoveLog2;
          const bool wover = __any_sync(kFullMask, over);
          if (lane == 0) gvote[rb * 4 + gw] = wover ? 1 : 0;
          named_barrier_sync(1 + 2 * grp, NCT);
          const int4 votes = *reinterpret_cast<const int4 *>(gvote + rb * 4);
          move = (votes.x | votes.y | votes.z | votes.w) != 0;
        }
        if (move) {
          float v2[G];
#pragma unroll
          for (int h = 0; h < G; ++h) v2[h] = w[h] + lv;
          const float wm = warp_reduce_heads<G, true>(v2, lane);
          constexpr int SH = 5 - kLog2<G>;
          if ((lane & ((1 << SH) - 1)) == 0) gred[(rb * 4 + gw) * 8 + (lane >> SH)] = wm;
          named_barrier_sync(1 + 2 * grp, NCT);
          float alpha[TSTEP];
#pragma unroll
          for (int h = 0; h < TSTEP; ++h) alpha[h] = 1.f;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float tm = fmaxf(fmaxf(gred[(rb * 4 + 0) * 8 + h], gred[(rb * 4 + 1) * 8 + h]),
                                   fmaxf(gred[(rb * 4 + 2) * 8 + h], gred[(rb * 4 + 3) * 8 + h]));
            const float mn = fmaxf(m_ref[h], tm);
            const float root = to_reference_root(m_ref[h], mn);
            alpha[h] = root * root;
            m_ref[h] = mn;
            l_part[h] = l_part[h] * root * root;
          }
          if (st > st0) {
            // (the group's last p.v was that of stage su - 2)
            wait_or_abort(&p_free[grp], (uint32_t)((su - 2) >> 1) & 1u, abort_flag, p.err);
            tc_fence_after();
#pragma unroll
            for (int c8 = 0; c8 < NCOL / 8; ++c8) {
              float ov[8];
              tmem_ld8(col_o(ob, grp) + lane_base + 8 * c8, ov);
#pragma unroll
              for (int i = 0; i < 8; ++i) ov[i] *= alpha[(8 * c8 + i) % TSTEP];
              tmem_st8(col_o(ob, grp) + lane_base + 8 * c8, ov);
            }
            tc_fence_before();
          }
        }
        // A weight's three terms, two heads a conversion.
        constexpr int HP = G == 1 ? 2 : G;
        uint32_t word[3][(TSTEP + 3) / 4];
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int j = 0; j < (TSTEP + 3) / 4; ++j) word[i][j] = 0;
        const float unit = vs * kWeightUnit;
#pragma unroll
        for (int h = 0; h < HP; h += 2) {
          float x0 = 0.f, x1 = 0.f;
          if (valid) {
            const float p0 = exp2_approx(w[h] - m_ref[h]);
            l_part[h] += p0;
            x0 = p0 * unit;
            if (h + 1 < G) {
              const float p1 = exp2_approx(w[h + 1 < G ? h + 1 : h] - m_ref[h + 1 < G ? h + 1 : h]);
              l_part[h + 1 < G ? h + 1 : h] += p1;
              x1 = p1 * unit;
            }
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint16_t c = e4m3x2(x0, x1);
            word[i][h >> 2] |= (uint32_t)c << ((h & 2) * 8);
            if (i < 2) {
              const float2 back = e4m3x2_to_float2(c);
              x0 = (x0 - back.x) * kTerm;
              x1 = (x1 - back.y) * kTerm;
            }
          }
        }
        wait_or_abort(&p_free[grp], ((uint32_t)(su >> 1) & 1u) ^ 1u, abort_flag, p.err);
        unsigned char *dst = smem + OFF_P + grp * P_BYTES8 + (t >> 3) * PGRP + (t & 7) * 16;
        if constexpr (TSTEP == 4) {
          *reinterpret_cast<uint4 *>(dst) = make_uint4(word[0][0], word[1][0], word[2][0], 0);
        } else {
          *reinterpret_cast<uint4 *>(dst) =
              make_uint4(word[0][0], word[0][1], word[1][0], word[1][1]);
          *reinterpret_cast<uint4 *>(dst + 128) = make_uint4(word[2][0], word[2][1], 0, 0);
        }
        if (!valid) {
          // rows that hold no token: their codes may be NaN
          const int vslot = su % NSV;
          wait_or_abort(&full_v[vslot], (uint32_t)(su / NSV) & 1u, abort_flag, p.err);
          uint4 *vrow = reinterpret_cast<uint4 *>(smem + OFF_V + vslot * STAGE +
                                                  (t >> 3) * GROUP + (t & 7) * 16);
#pragma unroll
          for (int c = 0; c < 8; ++c) vrow[c * 8] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[grp]);
      }
      s += nstages;
      // the group's references and per-warp sums, for the epilogue
      wait_or_abort(&o_free[ob], ((uint32_t)(k >> 1) & 1u) ^ 1u, abort_flag, p.err);
      {
        const float ws = warp_reduce_heads<G, false>(l_part, lane);
        constexpr int SH = 5 - kLog2<G>;
        if ((lane & ((1 << SH) - 1)) == 0)
          lred[((ob * 2 + grp) * 4 + gw) * 8 + (lane >> SH)] = ws;
      }
      if (t == 0) {
#pragma unroll
        for (int h = 0; h < G; ++h) mref[(ob * 2 + grp) * 8 + h] = m_ref[h];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_done[ob]);
      ++k;
      sg = nsg;
      ctx_b = ctx_n;
      have = have_next;
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int e = tid - 32 * WARP_EPI;  // head-dim row of O
    const int ew = warp - WARP_EPI;
    const uint32_t lane_base = (uint32_t)(ew * 32) << 16;
    constexpr int NET = 128;
    const int part = (int)blockIdx.x;
    // Query buffer k % 2 for segment k, one segment ahead: its last readers, the
    // MMAs of segment k - 2, were done before that segment's epilogue.
    auto convert = [&](const Piece &g, int k) {
      convert_query<G>(p, g, smem + OFF_Q + (k & 1) * Q_BYTES, qscale + (k & (NQS - 1)) * 8, e);
      if (lane == 0) mbar_arrive(&q_ready[k & 1]);
    };
    if (have) convert(sg, 0);
    int k = 0;
    while (have) {
      Piece nsg;
      const bool have_next = next(nsg);
      if (have_next) convert(nsg, k + 1);
      const int ob = k & 1;
      const int unit = sg.b * p.n_kv + sg.g;
      wait_or_abort(&seg_done[ob], (uint32_t)(k >> 1) & 1u, abort_flag, p.err);
      // the two softmax groups' states merged (a group without stages, or
      // with none of its rows valid, has the reference -inf and no weight; its
      // accumulator was perhaps never written)
      float Lsum[G], M[G], f0[G], f1[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float m0 = mref[ob * 16 + h], m1 = mref[ob * 16 + 8 + h];
        M[h] = fmaxf(m0, m1);
        // (as to_reference_root, by the full exponential: with the approximate one the
        // compiler's code for G = 8 took 338 us on 64 ragged contexts, so 329)
        const float r0 = m0 == -INFINITY ? 0.f : exp2f(0.5f * (m0 - M[h]));
        const float r1 = m1 == -INFINITY ? 0.f : exp2f(0.5f * (m1 - M[h]));
        f0[h] = r0 * r0;
        f1[h] = r1 * r1;
        const float *l0 = lred + ob * 64 + h, *l1 = l0 + 32;
        Lsum[h] = r0 * ((l0[0] + l0[8]) + (l0[16] + l0[24])) * r0 +
                  r1 * ((l1[0] + l1[8]) + (l1[16] + l1[24])) * r1;
      }
      wait_or_abort(&o_full[ob], (uint32_t)(k >> 1) & 1u, abort_flag, p.err);
      tc_fence_after();
      float ov[G];
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        float o[NCOL];
#pragma unroll
        for (int c8 = 0; c8 < (3 * TSTEP + 7) / 8; ++c8)
          tmem_ld8(col_o(ob, grp) + lane_base + 8 * c8,
                   *reinterpret_cast<float(*)[8]>(o + 8 * c8));
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float f = grp ? f1[h] : f0[h];
          const float x =
              fmaf(fmaf(o[2 * TSTEP + h], 1.f / kTerm, o[TSTEP + h]), 1.f / kTerm, o[h]);
          const float y = f != 0.f ? x * (f * (1.f / kWeightUnit)) : 0.f;
          ov[h] = grp ? ov[h] + y : y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[ob]);

      const bool whole = sg.j0 == 0 && sg.n == sg.nblk;
      const int c_first = sc.units ? part : (sg.ucs + sc.ov) / sc.S;
      const int c_last = sc.units ? part : (sg.uce - 1) / sc.S;
      const size_t obase = q_index(p, sg.b, sg.g, 0);
      if (whole) {
#pragma unroll
        for (int h = 0; h < G; ++h)
          p.out[(obase + h) * kHeadDim + e] = __float2bfloat16_rn(ov[h] / Lsum[h]);
      } else {
        const size_t srow = ((size_t)unit + (size_t)part) * G;
#pragma unroll
        for (int h = 0; h < G; ++h) p.part_o[(srow + h) * kHeadDim + e] = ov[h];
#pragma unroll
        for (int h = 0; h < G; ++h)
          if (e == h)
            *reinterpret_cast<float2 *>(p.part_ml + (srow + h) * 2) = make_float2(M[h], Lsum[h]);
        // Publish this part; the CTA of the unit's last part to arrive merges
        // them, once all its warps are done (a CTA's part holds at most two
        // cut units: its first and its last).  The barrier orders the 128
        // threads' stores before the atomic, whose release makes them visible
        // and whose acquire, in the last arriver, the other parts'.
        named_barrier_sync(2, NET);
        if (e == 0) {
          const int n_parts = c_last - c_first + 1;
          if (atomic_add_acq_rel_gpu(p.counters + unit, 1) == n_parts - 1) {
            atomicExch(p.counters + unit, 0);  // ready for the next call
            merges[*n_merges] = make_int4(unit, c_first, n_parts, 0);
            ++*n_merges;
          }
        }
      }
      ++k;
      sg = nsg;
      have = have_next;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (nothing lands in the K ring any more)
  for (int i = 0; i < *n_merges; ++i) {
    if (i) __syncthreads();
    merge_unit<G>(p, merges[i], reinterpret_cast<float *>(smem + OFF_K), tid);
  }
  if (warp == WARP_QK) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(TMEM_COLS8)
                 : "memory");
  }
}

// A pool as a tensor of tiles (see Params).
cudaError_t encode_map(CUtensorMap *map, const void *pool, long long tiles) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<Encode> encode{nullptr};
  Encode fn = encode.load();
  if (!fn) {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found);
    if (e != cudaSuccess) return e;
    if (!f || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    fn = reinterpret_cast<Encode>(f);
    encode.store(fn);
  }
  const cuuint64_t dims[2] = {256, (cuuint64_t)tiles};
  const cuuint64_t strides[1] = {16 * kHeadDim};
  const cuuint32_t box[2] = {256, 1}, steps[2] = {1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, const_cast<void *>(pool), dims, strides, box, steps,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int G, int BS>
cudaError_t launch_cfg(const Params &p, int grid, cudaStream_t stream) {
  static volatile int done[64] = {0};  // shared-memory limit raised, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(attention_fp8b_kernel<G, BS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_size(PGD_MAX_BATCH));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = smem_size(p.q8.a.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_fp8b_kernel<G, BS>, p);
}

}  // namespace tc8b

cudaError_t attention_fp8b_launch(const Attn8bParams &q8, int G, int bs, int grid,
                                  cudaStream_t stream) {
  tc8b::Params p = {};
  p.q8 = q8;
  const float units = (float)q8.a.B * (float)q8.a.n_kv;
  const float block = bs == 16 ? tc8b::kBlockBytes<16> : tc8b::kBlockBytes<32>;
  p.split_root = sqrtf(tc8b::kShare * units * block / (float)tc::kMergePartBytes);
  p.inv_units = 1.f / units;
  p.starts = units * (float)(bs == 16 ? tc::kSegCost<16> : tc::kSegCost<32>);
  if (bs == 16) {
    const long long tiles = (long long)q8.a.NB * q8.a.n_kv;
    cudaError_t e = tc8b::encode_map(&p.k_map, q8.a.k_cache, tiles);
    if (e == cudaSuccess) e = tc8b::encode_map(&p.v_map, q8.a.v_cache, tiles);
    if (e != cudaSuccess) return e;
  }
#define PGD_CASE(G_, BS_) \
  if (G == G_ && bs == BS_) return tc8b::launch_cfg<G_, BS_>(p, grid, stream);
  PGD_CASE(1, 16) PGD_CASE(2, 16) PGD_CASE(4, 16) PGD_CASE(8, 16)
  PGD_CASE(1, 32) PGD_CASE(2, 32) PGD_CASE(4, 32) PGD_CASE(8, 32)
#undef PGD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pgd
