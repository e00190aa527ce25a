// awq_moe.cuh — a whole mixture-of-experts layer for a few tokens (T <= 32), experts in packed
// 4-bit weights, in two kernels.
//
//   l_te = x_t . Wr_e              the top_k experts of token t by l (ties: lowest index)
//   p_te = exp(l_te - max) / sum   the sum over all experts, or over the chosen ones (renormalize)
//   h    = p_te * SiLU(x_t . Wg_e^T) * (x_t . Wu_e^T) [/ s_e]          (fp16)
//   y_t  = sum over the chosen e of h . Wd_e^T
//
// The layer is bound by the packed weights of the experts that are chosen at all (0.52 bytes per
// weight, each read once whatever the number of its tokens).
//
// awq_moe_route_kernel: clusters of 8 CTAs, 4 tokens each; the CTAs split the experts, rank 0
// gathers the logits through distributed shared memory and one warp per token picks its experts.
//
// awq_moe_experts_kernel: one CTA per SM, launched cooperatively. Phase 1 computes h for every
// (expert, 16 gate rows + their 16 up rows) unit, phase 2 the output tiles of 16 rows, summed over
// the experts; a grid-wide barrier lies between. A producer lane streams both phases' packed weights
// through one ring without waiting for the barrier, so phase 2's first weights arrive while phase 1
// ends. The consumer warps split a unit's group pairs and use the exact integer dequantization and
// warp MMAs of the decode kernel; activations are read through L1, the columns of an MMA being the
// expert's own tokens. Phase 2 adds an expert's columns to its tokens' places in the warp's record.
// h carries p: its fp16 rounding (2^-12 of each term on average) is the one the unfused layers make
// between their calls.
// Partial sums of the warps are added in warp order: results repeat bit for bit.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "awq_common.cuh"
#include "awq_gemv.cuh"

namespace awq {

constexpr int kMoeMaxTokens = 32;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int kRouteCluster = 8;
constexpr int kRouteTokens = 4;      // tokens per cluster
constexpr int kRouteWarps = 8;

// ---------------------------------------------------------------------------- routing
struct MoeRouteArgs {
  const __half* x;        // [T, K]
  const __half* router;   // [E, K]
  int* ids;               // [T, top]
  float* p;               // [T, top]
  unsigned* barrier;      // zeroed for the experts kernel
  int T, E, K, top, renorm;
};

__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(32 * kRouteWarps)
    awq_moe_route_kernel(const MoeRouteArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ float s_logits[kRouteTokens][kMoeMaxExperts];                                   // rank 0's is used
  __shared__ float s_part[kRouteWarps][kMoeMaxExperts / kRouteCluster][kRouteTokens];
  pdl_launch_dependents();
  pdl_wait();
  const int rank = static_cast<int>(cluster.block_rank());
  const int t0 = static_cast<int>(blockIdx.x) / kRouteCluster * kRouteTokens;
  const int nt = min(kRouteTokens, a.T - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 1 && threadIdx.x == 0) *a.barrier = 0u;
  // this CTA's experts; with few of them several warps split K
  const int epc = ceil_div(a.E, kRouteCluster), e0 = rank * epc;
  const int wpe = epc == 1 ? 8 : epc == 2 ? 4 : epc <= 4 ? 2 : 1;
  const int part = warp % wpe;
  const __half* xr[kRouteTokens];
#pragma unroll
  for (int t = 0; t < kRouteTokens; ++t) xr[t] = a.x + static_cast<size_t>(t0 + min(t, nt - 1)) * a.K;
  for (int le = warp / wpe; le < epc && e0 + le < a.E; le += kRouteWarps / wpe) {
    const __half* wr = a.router + static_cast<size_t>(e0 + le) * a.K;
    float acc[kRouteTokens] = {};
#pragma unroll 4
    for (int c = part * 32 + lane; c < a.K / 8; c += 32 * wpe) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(wr + c * 8));
      const uint32_t w4[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int t = 0; t < kRouteTokens; ++t) {
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(xr[t] + c * 8));
        const uint32_t x4[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 wf = half2_bits_to_float2(w4[j]), xf = half2_bits_to_float2(x4[j]);
          acc[t] = fmaf(wf.x, xf.x, acc[t]);
          acc[t] = fmaf(wf.y, xf.y, acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], o);
      if (lane == 0) s_part[part][le][t] = acc[t];
    }
  }
  __syncthreads();
  float* dst = cluster.map_shared_rank(&s_logits[0][0], 0);
  for (int i = threadIdx.x; i < epc * kRouteTokens; i += blockDim.x) {
    const int le = i / kRouteTokens, t = i % kRouteTokens;
    if (e0 + le >= a.E) continue;
    float v = 0.0f;
    for (int q = 0; q < wpe; ++q) v += s_part[q][le][t];
    dst[t * kMoeMaxExperts + e0 + le] = v;
  }
  cluster.sync();
  if (rank != 0 || warp >= nt) return;
  // one warp per token. Keys order by (logit, lowest index first); a NaN orders below every number and
  // a chosen expert's key is 0, so top_k distinct experts are found whatever the logits are.
  constexpr int kPer = kMoeMaxExperts / 32;
  unsigned long long key[kPer];
  float best = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0;
    if (e < a.E) {
      const float v = s_logits[warp][e];
      best = fmaxf(best, v);
      const uint32_t b = __float_as_uint(v);
      const uint32_t ord = v != v ? 0u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
      key[i] = (static_cast<unsigned long long>(ord) << 32) | static_cast<uint32_t>(~e);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i * 32 + lane < a.E) total += expf(s_logits[warp][i * 32 + lane] - best);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  float mine = 0.0f, chosen = 0.0f;   // lane k: the numerator of the k-th choice
  int mine_id = 0;
  for (int k = 0; k < a.top; ++k) {
    unsigned long long m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = key[i] > m ? key[i] : m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, m, o);
      m = other > m ? other : m;
    }
    const int e = static_cast<int>(~static_cast<uint32_t>(m));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] == m) key[i] = 0;
    const float v = expf(s_logits[warp][e] - best);
    chosen += v;
    if (lane == k) { mine = v; mine_id = e; }
  }
  if (lane < a.top) {
    a.ids[(t0 + warp) * a.top + lane] = mine_id;
    a.p[(t0 + warp) * a.top + lane] = __fdiv_rn(mine, a.renorm ? chosen : total);
  }
}

// ---------------------------------------------------------------------------- experts
struct MoeArgs {
  const __half* x;                             // [T, K]
  const uint8_t *gu_q, *gu_s, *gu_z;           // gate/up layers, packed layout v2, one after another
  const uint8_t *dn_q, *dn_s, *dn_z;           // down layers
  size_t gu_pairs, dn_pairs;                   // (tile, group pair) items of one expert's layer
  const float* h_scale;                        // [E, I] or null
  const int* ids;                              // [T, top]
  const float* p;
  __half* h;                                   // [T * top, I]
  __half* y;                                   // [T, K]
  unsigned* barrier;
  int T, E, K, I, top;
};

constexpr int kMoeCW = 16;                      // consumer warps
constexpr int kMoeThreads = 32 * (kMoeCW + 2);  // + producer, + epilogue
constexpr int kMoeStageItems = 16;              // (tile, group pair) items per ring stage, one per consumer warp
constexpr int kMoeOffS = kMoeStageItems * kPairCodeBytes;
constexpr int kMoeOffZ = kMoeOffS + kMoeStageItems * kPairScaleBytes;
constexpr int kMoeStage = kMoeOffZ + kMoeStageItems * kPairZeroBytes;   // 34048 bytes
static_assert(kMoeStage % 128 == 0, "ring stages stay aligned");

// MTT: 8-token tiles (T <= 8 MTT). A record is one warp's fp32 sums of one 16-row tile, [column][20]
// (20: rows padded so that the fragment stores hit distinct banks).
template <int MTT>
struct MoeCfg {
  static constexpr int kStages = MTT == 4 ? 3 : 4;
  static constexpr int kBlock = MTT == 1 ? 2 : 1;       // tiles per warp that share activation fragments
  static constexpr int kRec = 8 * MTT * 20;             // floats
  static constexpr int kBufs = MTT == 4 ? 1 : 2;        // record buffers (two tiles each)
  static constexpr int kRecBytes = kBufs * kMoeCW * 2 * kRec * 4;
  static constexpr int kBars = 2 * kStages + 2 * kBufs + 1;
};

// How a strip (one tile of one expert, Q group pairs along its K) is cut into stages. Up to 8 pairs:
// `strips` strips share a stage, `wide` warps each. More: `chunks` stages of up to `len` pairs.
struct MoeCut {
  int Q, wide, strips, chunks, len;
  __device__ explicit MoeCut(int q) : Q(q) {
    wide = q <= 1 ? 1 : q <= 2 ? 2 : q <= 4 ? 4 : q <= 8 ? 8 : 16;
    strips = kMoeStageItems / wide;
    chunks = (q + kMoeStageItems - 1) / kMoeStageItems;
    len = (q + chunks - 1) / chunks;
  }
};

// acc += S (sum x q) - S z (sum x) for the lane's four sums of one group (columns 2t, 2t+1 of rows r
// and r+8), two columns to an instruction. tq carries 2^-24 (rows r) and 2^-20 (rows r+8).
__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
}
__device__ __forceinline__ void moe_scale(float (&acc)[4], const float (&tq)[4], const float (&xs)[2], uint32_t sv, uint32_t zz) {
  const float2 sf = half2_bits_to_float2(sv);
  const float s_lo = sf.x * 16777216.0f, s_hi = sf.y * 1048576.0f;   // 2^24 and 2^20: exact
  const float z_lo = -sf.x * small_uint_to_float(zz & 0xFu), z_hi = -sf.y * small_uint_to_float(zz >> 4);
  float2 lo = make_float2(acc[0], acc[1]), hi = make_float2(acc[2], acc[3]);
  const float2 x2 = make_float2(xs[0], xs[1]);
  fma2(lo, make_float2(s_lo, s_lo), make_float2(tq[0], tq[1]));
  fma2(hi, make_float2(s_hi, s_hi), make_float2(tq[2], tq[3]));
  fma2(lo, make_float2(z_lo, z_lo), x2);
  fma2(hi, make_float2(z_hi, z_hi), x2);
  acc[0] = lo.x;
  acc[1] = lo.y;
  acc[2] = hi.x;
  acc[3] = hi.y;
}

// Sums of the activation fragments over a group, by an MMA whose A operand is all ones: lane (r, t)
// gets those of its accumulator columns 2t and 2t+1.
template <int MT>
__device__ __forceinline__ void moe_sums(float (&xs)[MT][2], const uint4 (&xv)[2][MT][2]) {
  const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    float d[4];
    mma_m16n8k16_f32_zero(d, ones, xv[0][j][0].x, xv[0][j][0].y);
    mma_m16n8k16_f32(d, ones, xv[0][j][0].z, xv[0][j][0].w);
    mma_m16n8k16_f32(d, ones, xv[0][j][1].x, xv[0][j][1].y);
    mma_m16n8k16_f32(d, ones, xv[0][j][1].z, xv[0][j][1].w);
    mma_m16n8k16_f32(d, ones, xv[1][j][0].x, xv[1][j][0].y);
    mma_m16n8k16_f32(d, ones, xv[1][j][0].z, xv[1][j][0].w);
    mma_m16n8k16_f32(d, ones, xv[1][j][1].x, xv[1][j][1].y);
    mma_m16n8k16_f32(d, ones, xv[1][j][1].z, xv[1][j][1].w);
    xs[j][0] = d[0];
    xs[j][1] = d[1];
  }
}

// acc += S (sum x q - z sum x) for one group. A code pair masked out of its word is a pair of fp16
// subnormals q 2^-24 (16 q 2^-24 in the odd nibbles, rows r+8): one AND makes an operand of the MMA,
// whose products are exact. The zero point costs no instruction per code: it enters once per group
// with the group's activation sum. 66 instructions per 2048 weights, where subtracting it from
// every code pair takes about 130 and made the integer pipe the bound.
template <int MT>
__device__ __forceinline__ void moe_group(float (&acc)[MT][4], const uint4& c0, const uint4& c1,
                                          const uint4 (&xv)[2][MT][2], const float (&xs)[MT][2], uint32_t sv, uint32_t zz) {
  float tq[MT][4];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const uint4& wv = kk ? c1 : c0;
#pragma unroll
    for (int s4 = 0; s4 < 4; ++s4) {
      const uint32_t q = (s4 == 0) ? wv.x : (s4 == 1) ? wv.y : (s4 == 2) ? wv.z : wv.w;
      const uint32_t q8 = q >> 8;
      const uint32_t a[4] = {q & 0x000F000Fu, q & 0x00F000F0u, q8 & 0x000F000Fu, q8 & 0x00F000F0u};
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const uint4& xq = xv[kk][j][s4 >> 1];
        const uint32_t b0 = (s4 & 1) ? xq.z : xq.x, b1 = (s4 & 1) ? xq.w : xq.y;
        if (kk == 0 && s4 == 0) mma_m16n8k16_f32_zero(tq[j], a, b0, b1);
        else mma_m16n8k16_f32(tq[j], a, b0, b1);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) moe_scale(acc[j], tq[j], xs[j], sv, zz);
}

// The activation fragments of one group pair for one 8-token tile, and their sums per group.
struct MoeFrag {
  uint4 v[2][2][2];   // [group][64-k tile][half]
  float s[2][2];      // [group][column 2t, 2t+1]
};

// One group pair with at most 8 tokens: the two groups' MMA chains run side by side.
__device__ __forceinline__ void moe_pair(float (&acc)[4], const uint4 (&w)[2][2], const MoeFrag& f, const uint32_t (&sv)[2],
                                         const uint32_t (&zz)[2]) {
  float tq[2][4];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint4& wv = w[g][kk];
        const uint32_t q = (s4 == 0) ? wv.x : (s4 == 1) ? wv.y : (s4 == 2) ? wv.z : wv.w;
        const uint32_t q8 = q >> 8;
        const uint32_t a[4] = {q & 0x000F000Fu, q & 0x00F000F0u, q8 & 0x000F000Fu, q8 & 0x00F000F0u};
        const uint4& xq = f.v[g][kk][s4 >> 1];
        const uint32_t b0 = (s4 & 1) ? xq.z : xq.x, b1 = (s4 & 1) ? xq.w : xq.y;
        if (kk == 0 && s4 == 0) mma_m16n8k16_f32_zero(tq[g], a, b0, b1);
        else mma_m16n8k16_f32(tq[g], a, b0, b1);
      }
#pragma unroll
  for (int g = 0; g < 2; ++g) moe_scale(acc, tq[g], f.s[g], sv[g], zz[g]);
}

// Bytes of the routing lists: expert counts, active experts, first slots (+1), assignment experts,
// slot tokens, slot weights.
__host__ __device__ inline int moe_list_bytes(int T, int E, int top) {
  const int n = T * top, act = n < E ? n : E;
  return (E + 2 * act + 1 + 3 * n) * 4;
}
template <int MT>
__host__ __device__ inline int moe_smem_bytes(int T, int E, int top) {
  using C = MoeCfg<MT>;
  return C::kStages * kMoeStage + C::kRecBytes + C::kBars * 8 + 8 + moe_list_bytes(T, E, top);
}
__device__ __forceinline__ uint4 ld_coherent_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int MTT>
__global__ void __launch_bounds__(kMoeThreads, 1) awq_moe_experts_kernel(const MoeArgs a) {
  using C = MoeCfg<MTT>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  float* rec = reinterpret_cast<float*>(smem + S * kMoeStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * kMoeStage + C::kRecBytes);
  uint64_t* empty = full + S;
  uint64_t* rfull = empty + S;                 // record buffers
  uint64_t* rempty = rfull + C::kBufs;
  uint64_t* go = rempty + C::kBufs;            // phase 2 may read h
  volatile int* s_abort = reinterpret_cast<volatile int*>(go + 1);
  int* s_active = const_cast<int*>(s_abort) + 1;
  const int n_assign = a.T * a.top;
  const int max_act = min(n_assign, a.E);
  int* l_count = s_active + 1;                 // [E]: counts, then the active index
  int* l_expert = l_count + a.E;               // [max_act]: expert of an active index
  int* l_first = l_expert + max_act;           // [max_act + 1]: its first slot
  int* l_ids = l_first + max_act + 1;          // [n_assign]
  int* l_token = l_ids + n_assign;             // [n_assign]: token of a slot
  float* l_p = reinterpret_cast<float*>(l_token + n_assign);   // [n_assign]: weight of a slot

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMoeCW);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&rfull[b], kMoeCW);
      mbar_init(&rempty[b], 1);
    }
    mbar_init(go, 1);
    *s_abort = 0;
    mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  const unsigned long long budget = g_wait_budget_ns;

  // ---- the experts that are chosen and their slots (token order)
  for (int i = threadIdx.x; i < a.E; i += kMoeThreads) l_count[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n_assign; i += kMoeThreads) {
    const int e = a.ids[i];
    l_ids[i] = e;
    atomicAdd(&l_count[e], 1);
  }
  __syncthreads();
  if (warp == 0) {
    int act = 0, slots = 0;
    for (int b = 0; b < a.E; b += 32) {
      const int e = b + lane, c = e < a.E ? l_count[e] : 0;
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, c > 0);
      int before = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      const int all = __shfl_sync(0xFFFFFFFFu, before, 31);
      const int idx = act + __popc(live & ((1u << lane) - 1));
      if (c > 0) {
        l_expert[idx] = e;
        l_first[idx] = slots + before - c;
      }
      if (e < a.E) l_count[e] = idx;
      act += __popc(live);
      slots += all;
    }
    if (lane == 0) {
      l_first[act] = slots;
      *s_active = act;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_assign; i += kMoeThreads) {
    const int e = l_ids[i], idx = l_count[e];
    int rank = 0;
    for (int j = 0; j < i; ++j) rank += l_ids[j] == e;
    const int slot = l_first[idx] + rank;
    l_token[slot] = i / a.top;
    l_p[slot] = a.p[i];
  }
  __syncthreads();

  // ---- this CTA's work. Phase 1: units (active expert, 16-row gate tile and its up tile). Phase 2:
  // 16-row output tiles, over all active experts. All roles walk the same stages in the same order.
  const int A = *s_active, P = a.I / 16;
  const int G1 = a.K / kGroup, G2 = a.I / kGroup;
  const MoeCut k1((G1 + 1) / 2), k2((G2 + 1) / 2);
  const int c0 = blockIdx.x, nc = gridDim.x;
  auto share = [&](int units, int c) { return static_cast<int>(static_cast<long long>(units) * c / nc); };
  const int u1a = share(A * P, c0), u1b = share(A * P, c0 + 1);
  const int u2a = share(a.K / 16, c0), u2b = share(a.K / 16, c0 + 1);
  constexpr int BL = C::kBlock;
  int slot = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++slot == S) { slot = 0; phase ^= 1; }
  };
  int ev = 0;                                  // record events so far
  auto buf_of = [&]() { return ev % C::kBufs; };
  auto buf_parity = [&]() { return static_cast<uint32_t>((ev / C::kBufs) & 1); };
  auto rec_of = [&](int w, int half) { return rec + ((buf_of() * kMoeCW + w) * 2 + half) * C::kRec; };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, s_abort, budget));
  };

  if (warp == kMoeCW) {
    // ---------------------------------------------------------------- producer lane
    if (lane != 0) return;
    int issued = 0;
    constexpr int kItem = kPairCodeBytes + kPairScaleBytes + kPairZeroBytes;
    uint8_t* sb = nullptr;
    auto open = [&](int items) -> bool {
      if (!mbar_wait_bounded(&empty[slot], phase ^ 1, s_abort, budget)) return false;
      sb = smem + slot * kMoeStage;
      mbar_arrive_expect_tx(&full[slot], items * kItem);
      return true;
    };
    // `n` items from (tile, pair) index tp of the packed layers into places at..at+n-1 of the stage
    auto copy = [&](int at, const uint8_t* q, const uint8_t* s, const uint8_t* z, size_t tp, int n, size_t total) {
      if (!AWQ_CHECK(n >= 1 && at >= 0 && at + n <= kMoeStageItems && tp + n <= total)) return;
      bulk_g2s(sb + at * kPairCodeBytes, q + tp * kPairCodeBytes, n * kPairCodeBytes, &full[slot]);
      bulk_g2s(sb + kMoeOffS + at * kPairScaleBytes, s + tp * kPairScaleBytes, n * kPairScaleBytes, &full[slot]);
      bulk_g2s(sb + kMoeOffZ + at * kPairZeroBytes, z + tp * kPairZeroBytes, n * kPairZeroBytes, &full[slot]);
    };
    auto close = [&]() {
      ++issued;
      advance();
    };
    const size_t gu_total = a.E * a.gu_pairs, dn_total = a.E * a.dn_pairs;
    auto produce = [&]() {
      for (int u = u1a; u < u1b;) {
        const int x = u / P, ja = u - x * P, jb = min(P, ja + u1b - u);
        const size_t base = static_cast<size_t>(l_expert[x]) * a.gu_pairs;
        if (k1.strips == 1) {
          for (int j0 = ja; j0 < jb; j0 += BL)
            for (int c = 0; c < k1.chunks; ++c) {
              const int p0 = c * k1.len, n = min(k1.len, k1.Q - p0);
              for (int b = 0; b < 2 * min(BL, jb - j0); ++b) {
                if (!open(n)) return;
                copy(0, a.gu_q, a.gu_s, a.gu_z, base + static_cast<size_t>((b & 1) * P + j0 + (b >> 1)) * k1.Q + p0, n, gu_total);
                close();
              }
            }
        } else {
          const int half = k1.strips / 2;
          for (int j0 = ja; j0 < jb; j0 += half) {
            const int n = min(half, jb - j0) * k1.Q;
            if (!open(2 * n)) return;
            for (int h = 0; h < 2; ++h)
              copy(h * half * k1.Q, a.gu_q, a.gu_s, a.gu_z, base + static_cast<size_t>(h * P + j0) * k1.Q, n, gu_total);
            close();
          }
        }
        u += jb - ja;
      }
      for (int t0 = u2a; t0 < u2b; t0 += BL)
        for (int x0 = 0; x0 < A; x0 += k2.strips) {
          const int m = min(k2.strips, A - x0);
          for (int c = 0; c < k2.chunks; ++c) {
            const int p0 = c * k2.len, n = min(k2.len, k2.Q - p0);
            for (int b = 0; b < min(BL, u2b - t0); ++b) {
              if (!open(m * n)) return;
              for (int i = 0; i < m; ++i)
                copy(i * n, a.dn_q, a.dn_s, a.dn_z,
                     static_cast<size_t>(l_expert[x0 + i]) * a.dn_pairs + static_cast<size_t>(t0 + b) * k2.Q + p0, n, dn_total);
              close();
            }
          }
        }
    };
    produce();
    // drain: every copy this thread issued has landed before the CTA may exit
    int never = 0;
    for (int i = max(0, issued - S); i < issued; ++i)
      mbar_wait_bounded(&full[i % S], static_cast<uint32_t>((i / S) & 1), &never, kDrainBudgetNs);
    return;
  }

  if (warp == kMoeCW + 1) {
    // ---------------------------------------------------------------- epilogue warp
    auto sum = [&](int half, int w0, int nw, int col, int row) {
      float v = 0.0f;
#pragma unroll 4
      for (int w = 0; w < nw; ++w) v += rec_of(w0 + w, half)[col * 20 + row];
      return v;
    };
    auto done = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&rempty[buf_of()]);
      ++ev;
    };
    bool ok = true;
    for (int u = u1a; ok && u < u1b;) {
      const int x = u / P, ja = u - x * P, jb = min(P, ja + u1b - u);
      const int first = l_first[x], cnt = l_first[x + 1] - first;
      const int per = k1.strips == 1 ? 1 : k1.strips / 2;               // units per event
      for (int j0 = ja; j0 < jb; j0 += per) {
        ok = warp_wait(&rfull[buf_of()], buf_parity());
        if (!ok) break;
        const int nu = min(per, jb - j0);
        for (int q = lane; q < 16 * nu * cnt; q += 32) {
          const int row = q & 15, i = (q >> 4) % nu, col = (q >> 4) / nu;
          const int i_row = 16 * (j0 + i) + row;
          if (!AWQ_CHECK(first + col < n_assign && i_row < a.I)) continue;
          const bool one = k1.strips == 1;
          const float g = one ? sum(0, 0, k1.len, col, row) : sum(0, i * k1.wide, k1.Q, col, row);
          const float v = one ? sum(1, 0, k1.len, col, row) : sum(0, (per + i) * k1.wide, k1.Q, col, row);
          float hv = silu_mul(g, v) * l_p[first + col];
          if (a.h_scale != nullptr) hv = __fdiv_rn(hv, __ldg(a.h_scale + static_cast<size_t>(l_expert[x]) * a.I + i_row));
          a.h[static_cast<size_t>(first + col) * a.I + i_row] = __float2half_rn(hv);
        }
        done();
      }
      u += jb - ja;
    }
    // grid-wide barrier: every CTA's h is written (release) and visible (acquire)
    __threadfence();
    __syncwarp();
    if (ok && lane == 0) {
      unsigned v;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(a.barrier) : "memory");
      const uint64_t t0 = globaltimer_ns();
      while (true) {
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.barrier) : "memory");
        if (v >= gridDim.x || *s_abort) break;
        if (globaltimer_ns() - t0 > budget) {
          *s_abort = 1;
          atomicOr(&g_dev_status, kDevStatusTimeout);
          break;
        }
      }
      if (*s_abort == 0) mbar_arrive(go);
    }
    for (int t0 = u2a; ok && t0 < u2b; t0 += BL) {
      ok = warp_wait(&rfull[buf_of()], buf_parity());
      if (!ok) break;
      const int rows = 16 * min(BL, u2b - t0);
      for (int q = lane; q < rows * a.T; q += 32) {
        const int row = q % rows, col = q / rows;
        if (!AWQ_CHECK(16 * t0 + row < a.K)) continue;
        a.y[static_cast<size_t>(col) * a.K + 16 * t0 + row] = __float2half_rn(sum(row >> 4, 0, kMoeCW, col, row & 15));
      }
      done();
    }
    return;
  }

  // ------------------------------------------------------------------ consumer warps
  const int r = lane >> 2, t = lane & 3;
  const uint8_t* sb = nullptr;
  auto take = [&]() -> bool {
    sb = smem + slot * kMoeStage;
    return warp_wait(&full[slot], phase);
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    advance();
  };
  auto rec_ready = [&]() { return warp_wait(&rempty[buf_of()], buf_parity() ^ 1); };
  auto rec_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&rfull[buf_of()]);
    ++ev;
  };
  // Fragments of an 8-token tile: `row` points at the lane's token (k 0), the group starts at k0.
  auto load8 = [&](uint4 (&v)[2][2], const __half* row, int k0) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      v[kk][0] = ld_coherent_v4(row + k0 + kk * 64 + 16 * t);
      v[kk][1] = ld_coherent_v4(row + k0 + kk * 64 + 16 * t + 8);
    }
  };
  auto load_frag = [&](MoeFrag& f, const __half* row, int pr, int G) {
    load8(f.v[0], row, pr * 256);
    if (2 * pr + 1 < G) {
      load8(f.v[1], row, pr * 256 + 128);
    } else {                                   // the padding group: its codes and scales are zero
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[1][i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
    }
  };
  auto sum_frag = [&](MoeFrag& f) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float d[4];
      const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
      mma_m16n8k16_f32_zero(d, ones, f.v[g][0][0].x, f.v[g][0][0].y);
      mma_m16n8k16_f32(d, ones, f.v[g][0][0].z, f.v[g][0][0].w);
      mma_m16n8k16_f32(d, ones, f.v[g][0][1].x, f.v[g][0][1].y);
      mma_m16n8k16_f32(d, ones, f.v[g][0][1].z, f.v[g][0][1].w);
      mma_m16n8k16_f32(d, ones, f.v[g][1][0].x, f.v[g][1][0].y);
      mma_m16n8k16_f32(d, ones, f.v[g][1][0].z, f.v[g][1][0].w);
      mma_m16n8k16_f32(d, ones, f.v[g][1][1].x, f.v[g][1][1].y);
      mma_m16n8k16_f32(d, ones, f.v[g][1][1].z, f.v[g][1][1].w);
      f.s[g][0] = d[0];
      f.s[g][1] = d[1];
    }
  };
  auto scale_of = [&](int item, int g) {
    return *reinterpret_cast<const uint32_t*>(sb + kMoeOffS + item * kPairScaleBytes + g * 32 + r * 4);
  };
  auto zero_of = [&](int item, int g) { return static_cast<uint32_t>(sb[kMoeOffZ + item * kPairZeroBytes + g * 8 + r]); };
  auto code_of = [&](int item, int g, int kk) {
    return *reinterpret_cast<const uint4*>(sb + item * kPairCodeBytes + g * 1024 + kk * 512 + lane * 16);
  };
  auto pair8 = [&](float (&acc)[4], const MoeFrag& f, int item) {
    const uint4 w[2][2] = {{code_of(item, 0, 0), code_of(item, 0, 1)}, {code_of(item, 1, 0), code_of(item, 1, 1)}};
    const uint32_t sv[2] = {scale_of(item, 0), scale_of(item, 1)}, zz[2] = {zero_of(item, 0), zero_of(item, 1)};
    moe_pair(acc, w, f, sv, zz);
  };
  // More than 8 tokens: 16 at a time, group by group; the fragments do not stay in registers.
  // `row_of(col)` is the lane's activation row for a column.
  auto pair_many = [&](float (&acc)[MTT][4], int item, int pr, int G, int cnt, auto row_of) {
    if constexpr (MTT > 1) {
#pragma unroll
      for (int b = 0; b < MTT / 2; ++b) {
        if (16 * b >= cnt) break;
        const __half* row[2] = {row_of(min(16 * b + r, cnt - 1)), row_of(min(16 * b + 8 + r, cnt - 1))};
#pragma unroll 1
        for (int g = 0; g < 2 && 2 * pr + g < G; ++g) {
          uint4 v[2][2][2];                    // [64-k tile][token tile][half]
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint4 one[2][2];
            load8(one, row[m], pr * 256 + g * 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i >> 1][m][i & 1] = one[i >> 1][i & 1];
          }
          float xs[2][2];
          moe_sums<2>(xs, v);
          moe_group<2>(reinterpret_cast<float(&)[2][4]>(acc[2 * b]), code_of(item, g, 0), code_of(item, g, 1), v, xs,
                       scale_of(item, g), zero_of(item, g));
        }
      }
    }
  };
  bool ok = true;

  // ---- phase 1
  {
    float acc[BL][2][MTT][4] = {};
    // this warp's sums of a tile become its record
    auto record = [&](float (&v)[MTT][4], int half, int cnt) {
      float* p = rec_of(warp, half);
#pragma unroll
      for (int m = 0; m < MTT; ++m)
        if (8 * m < cnt)
#pragma unroll
          for (int c = 0; c < 4; ++c) p[(8 * m + 2 * t + (c & 1)) * 20 + r + 8 * (c >> 1)] = v[m][c];
#pragma unroll
      for (int m = 0; m < MTT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[m][c] = 0.0f;
    };
    const int pl = warp % k1.wide, sub = warp / k1.wide;
    for (int u = u1a; ok && u < u1b;) {
      const int x = u / P, ja = u - x * P, jb = min(P, ja + u1b - u);
      const int first = l_first[x], cnt = l_first[x + 1] - first;
      auto row_of = [&](int col) { return a.x + static_cast<size_t>(l_token[first + col]) * a.K; };
      const __half* row8 = row_of(min(r, cnt - 1));
      // `many`: more than 8 tokens (separate code, so that its fragments and f do not share registers)
      auto expert = [&](auto many) {
        constexpr bool kMany = decltype(many)::value;
        MoeFrag f;
        if (k1.strips == 1) {
          for (int j0 = ja; ok && j0 < jb; j0 += BL) {
            const int nb = min(BL, jb - j0);
            for (int c = 0; ok && c < k1.chunks; ++c) {
              const int pr = c * k1.len + pl;
              const bool live = pl < min(k1.len, k1.Q - c * k1.len);
              if (!kMany && live && (k1.chunks > 1 || j0 == ja)) {   // one chunk: they last for the expert
                load_frag(f, row8, pr, G1);
                sum_frag(f);
              }
#pragma unroll
              for (int b = 0; b < 2 * BL; ++b) {
                if (b >= 2 * nb || !ok) break;
                ok = take();
                if (!ok) break;
                if (live) {
                  if constexpr (kMany) pair_many(acc[b >> 1][b & 1], pl, pr, G1, cnt, row_of);
                  else pair8(acc[b >> 1][b & 1][0], f, pl);
                }
                release();
                if (c == k1.chunks - 1) {
                  if ((b & 1) == 0) ok = rec_ready();
                  if (!ok) break;
                  record(acc[b >> 1][b & 1], b & 1, cnt);
                  if (b & 1) rec_done();
                }
              }
            }
          }
        } else {
          const int half = k1.strips / 2, i = sub % half;
          if (!kMany && pl < k1.Q) {
            load_frag(f, row8, pl, G1);
            sum_frag(f);
          }
          for (int j0 = ja; ok && j0 < jb; j0 += half) {
            ok = take();
            if (!ok) break;
            if (pl < k1.Q && j0 + i < jb) {
              if constexpr (kMany) pair_many(acc[0][0], sub * k1.Q + pl, pl, G1, cnt, row_of);
              else pair8(acc[0][0][0], f, sub * k1.Q + pl);
            }
            release();
            ok = rec_ready();
            if (!ok) break;
            record(acc[0][0], 0, cnt);
            rec_done();
          }
        }
      };
      if (MTT == 1 || cnt <= 8) expert(std::false_type{});
      else expert(std::bool_constant<(MTT > 1)>{});
      u += jb - ja;
    }
  }

  ok = ok && warp_wait(go, 0);

  // ---- phase 2: an expert's sums are added to its tokens' places in the warp's record
  {
    float acc[BL][MTT][4] = {};
    const int pl = warp % k2.wide, sub = warp / k2.wide;
    for (int t0 = u2a; ok && t0 < u2b; t0 += BL) {
      const int nb = min(BL, u2b - t0);
      ok = rec_ready();
      if (!ok) break;
      for (int b = 0; b < nb; ++b)
        for (int i = lane; i < a.T * 20; i += 32) rec_of(warp, b)[i] = 0.0f;
      __syncwarp();
      for (int x0 = 0; ok && x0 < A; x0 += k2.strips) {
        const int x = x0 + sub;
        const bool mine = x < A;
        const int first = mine ? l_first[x] : 0, cnt = mine ? l_first[x + 1] - first : 0;
        auto row_of = [&](int col) { return a.h + static_cast<size_t>(first + col) * a.I; };
        const __half* row8 = row_of(max(0, min(r, cnt - 1)));
        auto expert = [&](auto many) {
          constexpr bool kMany = decltype(many)::value;
          for (int c = 0; ok && c < k2.chunks; ++c) {
            const int n = min(k2.len, k2.Q - c * k2.len), pr = c * k2.len + pl;
            const bool live = mine && pl < n;
            MoeFrag f;
            if (!kMany && live) {
              load_frag(f, row8, pr, G2);
              sum_frag(f);
            }
#pragma unroll
            for (int b = 0; b < BL; ++b) {
              if (b >= nb || !ok) break;
              ok = take();
              if (!ok) break;
              if (live) {
                if constexpr (kMany) pair_many(acc[b], sub * n + pl, pr, G2, cnt, row_of);
                else pair8(acc[b][0], f, sub * n + pl);
              }
              release();
            }
          }
        };
        if (MTT == 1 || cnt <= 8) expert(std::false_type{});
        else expert(std::bool_constant<(MTT > 1)>{});
        if (!ok) break;
        if (mine && pl < k2.len) {
#pragma unroll
          for (int b = 0; b < BL; ++b) {
            if (b >= nb) break;
            float* p = rec_of(warp, b);
#pragma unroll
            for (int m = 0; m < MTT; ++m)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int col = 8 * m + 2 * t + c;
                if (col < cnt) {
                  float* pt = p + l_token[first + col] * 20 + r;
                  pt[0] += acc[b][m][c];
                  pt[8] += acc[b][m][c + 2];
                }
                acc[b][m][c] = acc[b][m][c + 2] = 0.0f;
              }
          }
        }
      }
      if (ok) rec_done();
    }
  }
}

}  // namespace awq
