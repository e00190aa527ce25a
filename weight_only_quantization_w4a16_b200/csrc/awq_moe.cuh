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
// expert's own tokens in phase 1 and all tokens in phase 2 (zero where a token did not choose the
// expert), so phase 2 sums over experts in its accumulators. h carries p: its fp16 rounding
// (2^-12 of each term on average) is the one the unfused layers make between their calls.
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

constexpr int kMoeCW = 8;                       // consumer warps
constexpr int kMoeThreads = 32 * (kMoeCW + 1);
constexpr int kMoeStageItems = 16;              // (tile, group pair) items per ring stage
constexpr int kMoeOffS = kMoeStageItems * kPairCodeBytes;
constexpr int kMoeOffZ = kMoeOffS + kMoeStageItems * kPairScaleBytes;
constexpr int kMoeStage = kMoeOffZ + kMoeStageItems * kPairZeroBytes;   // 34048 bytes
static_assert(kMoeStage % 128 == 0, "ring stages stay aligned");

// MT: 8-token tiles (T <= 8 MT). A record is one warp's fp32 sums of one 16-row tile, [column][20]
// (20: rows padded so that the fragment stores hit distinct banks).
template <int MT>
struct MoeCfg {
  static constexpr int kStages = 3;
  static constexpr int kRec = 8 * MT * 20;              // floats
  static constexpr int kBufs = MT == 1 ? 4 : 2;         // units whose records are held at a time
  static constexpr int kDone = kBufs / 2;               // units that may end within one stage
  static constexpr int kRecBytes = kBufs * kMoeCW * 2 * kRec * 4;
};

// Bytes of the routing lists: expert counts, active experts, first slots (+1), assignment experts,
// slot tokens, slot weights, and the 16-bit slot map.
__host__ __device__ inline int moe_list_bytes(int T, int E, int top) {
  const int n = T * top, act = n < E ? n : E;
  return (E + 2 * act + 1 + 3 * n) * 4 + act * T * 2;
}
template <int MT>
__host__ __device__ inline int moe_smem_bytes(int T, int E, int top) {
  using C = MoeCfg<MT>;
  return C::kStages * kMoeStage + C::kRecBytes + (2 * C::kStages + 1) * 8 + 8 + moe_list_bytes(T, E, top);
}
__device__ __forceinline__ uint4 ld_coherent_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
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
  uint64_t* cbar = empty + S;                  // the consumer warps' barrier
  volatile int* s_abort = reinterpret_cast<volatile int*>(cbar + 1);
  int* s_active = const_cast<int*>(s_abort) + 1;
  const int n_assign = a.T * a.top;
  const int max_act = min(n_assign, a.E);
  int* l_count = s_active + 1;                 // [E]: counts, then the active index
  int* l_expert = l_count + a.E;               // [max_act]: expert of an active index
  int* l_first = l_expert + max_act;           // [max_act + 1]: its first slot
  int* l_ids = l_first + max_act + 1;          // [n_assign]
  int* l_token = l_ids + n_assign;             // [n_assign]: token of a slot
  float* l_p = reinterpret_cast<float*>(l_token + n_assign);   // [n_assign]: weight of a slot
  int16_t* l_map = reinterpret_cast<int16_t*>(l_p + n_assign); // [max_act][T]: slot of (active index, token) or -1

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMoeCW);
    }
    mbar_init(cbar, kMoeCW);
    *s_abort = 0;
    mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  const unsigned long long budget = g_wait_budget_ns;

  // ---- the experts that are chosen, their slots (token order) and the slot of each (expert, token)
  for (int i = threadIdx.x; i < a.E; i += kMoeThreads) l_count[i] = 0;
  for (int i = threadIdx.x; i < max_act * a.T; i += kMoeThreads) l_map[i] = -1;
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
    l_map[idx * a.T + i / a.top] = static_cast<int16_t>(slot);
  }
  __syncthreads();

  // ---- this CTA's work. Phase 1: units are (active expert, 16-row gate tile + up tile), items its
  // group pairs. Phase 2: units are 16-row output tiles, items (active expert, group pair).
  const int A = *s_active, P = a.I / 16;
  const int G1 = a.K / kGroup, G2 = a.I / kGroup;
  const int Q1 = (G1 + 1) / 2, Q2 = (G2 + 1) / 2;        // group pairs along K and along I
  const int c0 = blockIdx.x, nc = gridDim.x;
  auto share = [&](int units, int c) { return static_cast<int>(static_cast<long long>(units) * c / nc); };
  const int u1a = share(A * P, c0), u1b = share(A * P, c0 + 1);
  const int u2a = share(a.K / 16, c0), u2b = share(a.K / 16, c0 + 1);
  const int ipu1 = Q1, ipu2 = A * Q2;                     // items per unit
  // a stage holds items of one phase, so many that at most kDone units end within it
  const int len1 = min(kMoeStageItems / 2, C::kDone * ipu1), len2 = min(kMoeStageItems, C::kDone * ipu2);
  const int n1 = (u1b - u1a) * ipu1, n2 = (u2b - u2a) * ipu2;

  if (warp == kMoeCW) {
    // ---------------------------------------------------------------- producer lane
    if (lane == 0) {
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      // `n` items from (tile, pair) index tp of the packed layers into places at..at+n-1 of the stage
      auto copy = [&](uint8_t* sb, int at, const uint8_t* q, const uint8_t* s, const uint8_t* z, size_t tp, int n,
                      size_t total, uint64_t* bar) {
        if (!AWQ_CHECK(n >= 1 && at >= 0 && at + n <= kMoeStageItems && tp + n <= total)) return;
        bulk_g2s(sb + at * kPairCodeBytes, q + tp * kPairCodeBytes, n * kPairCodeBytes, bar);
        bulk_g2s(sb + kMoeOffS + at * kPairScaleBytes, s + tp * kPairScaleBytes, n * kPairScaleBytes, bar);
        bulk_g2s(sb + kMoeOffZ + at * kPairZeroBytes, z + tp * kPairZeroBytes, n * kPairZeroBytes, bar);
      };
      constexpr int kItem = kPairCodeBytes + kPairScaleBytes + kPairZeroBytes;
      auto next = [&]() -> uint8_t* {
        if (!mbar_wait_bounded(&empty[slot], phase ^ 1, s_abort, budget)) return nullptr;
        return smem + slot * kMoeStage;
      };
      auto advance = [&]() {
        ++issued;
        if (++slot == S) { slot = 0; phase ^= 1; }
      };
      for (int i = 0; ok && i < n1; i += len1) {
        const int n = min(len1, n1 - i);
        uint8_t* sb = next();
        if (sb == nullptr) { ok = false; break; }
        mbar_arrive_expect_tx(&full[slot], 2 * n * kItem);
        for (int d = 0; d < n;) {                          // runs within one expert are contiguous
          const int u = u1a + (i + d) / ipu1, pr = (i + d) % ipu1;
          const int x = u / P, j = u - x * P;
          const int run = min(n - d, (P - j) * ipu1 - pr);
          const size_t base = static_cast<size_t>(l_expert[x]) * a.gu_pairs;
          copy(sb, d, a.gu_q, a.gu_s, a.gu_z, base + static_cast<size_t>(j) * Q1 + pr, run, a.E * a.gu_pairs, &full[slot]);
          copy(sb, kMoeStageItems / 2 + d, a.gu_q, a.gu_s, a.gu_z, base + static_cast<size_t>(P + j) * Q1 + pr, run,
               a.E * a.gu_pairs, &full[slot]);
          d += run;
        }
        advance();
      }
      for (int i = 0; ok && i < n2; i += len2) {
        const int n = min(len2, n2 - i);
        uint8_t* sb = next();
        if (sb == nullptr) { ok = false; break; }
        mbar_arrive_expect_tx(&full[slot], n * kItem);
        for (int d = 0; d < n;) {
          const int u = u2a + (i + d) / ipu2, r = (i + d) % ipu2;
          const int x = r / Q2, pr = r - x * Q2;
          const int run = min(n - d, Q2 - pr);
          copy(sb, d, a.dn_q, a.dn_s, a.dn_z,
               static_cast<size_t>(l_expert[x]) * a.dn_pairs + static_cast<size_t>(u) * Q2 + pr, run,
               a.E * a.dn_pairs, &full[slot]);
          d += run;
        }
        advance();
      }
      // drain: every copy this thread issued has landed before the CTA may exit
      int never = 0;
      for (int i = max(0, issued - S); i < issued; ++i)
        mbar_wait_bounded(&full[i % S], static_cast<uint32_t>((i / S) & 1), &never, kDrainBudgetNs);
    }
    return;
  }

  // ------------------------------------------------------------------ consumer warps
  const int r = lane >> 2, t = lane & 3;
  int slot = 0;
  uint32_t phase = 0;
  float acc[2][MTT][4];
  auto clear = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < MTT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[h][j][c] = 0.0f;
  };
  clear();
  auto rec_of = [&](int unit, int w, int half) { return rec + (((unit % C::kBufs) * kMoeCW + w) * 2 + half) * C::kRec; };
  // this warp's sums of `unit` become its record
  auto flush = [&](int unit, int halves) {
    for (int h = 0; h < halves; ++h) {
      float* p = rec_of(unit, warp, h);
#pragma unroll
      for (int j = 0; j < MTT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) p[(8 * j + 2 * t + (c & 1)) * 20 + r + 8 * (c >> 1)] = h ? acc[1][j][c] : acc[0][j][c];
    }
    clear();
  };
  auto sum_of = [&](int unit, int half, int col, int row) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeCW; ++w) v += rec_of(unit, w, half)[col * 20 + row];
    return v;
  };
  auto wait_full = [&]() -> bool {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[slot], phase, s_abort, budget));
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == S) { slot = 0; phase ^= 1; }
  };
  bool ok = true;
  // The consumer warps' barrier, bounded like every wait: false once any warp has given up.
  uint32_t cphase = 0;
  auto consumer_sync = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(cbar);
    const bool done = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(cbar, cphase, s_abort, budget));
    cphase ^= 1;
    return done;
  };

  // ---- phase 1
  {
    int cur = 0;                                           // the (relative) unit that acc holds
    for (int i = 0; ok && i < n1; i += len1) {
      const int n = min(len1, n1 - i);
      ok = wait_full();
      if (!ok) break;
      const uint8_t* sb = smem + slot * kMoeStage;
      if (warp < n) {
        const int u = (i + warp) / ipu1, pr = (i + warp) % ipu1;
        while (cur < u) flush(cur++, 2);
        const int x = (u1a + u) / P, first = l_first[x], cnt = l_first[x + 1] - first;
        auto item = [&](auto mt) {
          constexpr int MT = decltype(mt)::value;
          const __half* xr[MT];
#pragma unroll
          for (int j = 0; j < MT; ++j)
            xr[j] = a.x + static_cast<size_t>(l_token[first + min(8 * j + r, cnt - 1)]) * a.K + pr * 256 + 16 * t;
#pragma unroll
          for (int gg = 0; gg < 2; ++gg) {
            if (2 * pr + gg >= G1) break;
            uint4 xv[2][MT][2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int j = 0; j < MT; ++j) {
                xv[kk][j][0] = __ldg(reinterpret_cast<const uint4*>(xr[j] + gg * 128 + kk * 64));
                xv[kk][j][1] = __ldg(reinterpret_cast<const uint4*>(xr[j] + gg * 128 + kk * 64 + 8));
              }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int it = warp + h * (kMoeStageItems / 2);
              const uint8_t* cb = sb + it * kPairCodeBytes + gg * 1024 + lane * 16;
              const uint4 w0 = *reinterpret_cast<const uint4*>(cb);
              const uint4 w1 = *reinterpret_cast<const uint4*>(cb + 512);
              const uint32_t sv = *reinterpret_cast<const uint32_t*>(sb + kMoeOffS + it * kPairScaleBytes + gg * 32 + r * 4);
              const uint32_t zz = sb[kMoeOffZ + it * kPairZeroBytes + gg * 8 + r];
              gemv_group<MT>(reinterpret_cast<float(&)[MT][4]>(acc[h]), w0, w1, xv, sv, zz);
            }
          }
        };
        if (MTT == 1 || cnt <= 8) item(std::integral_constant<int, 1>{});
        else if (MTT == 2 || cnt <= 16) item(std::integral_constant<int, MTT < 2 ? 1 : 2>{});
        else item(std::integral_constant<int, MTT>{});
      }
      release();
      const int done0 = i / ipu1, done1 = (i + n) / ipu1;  // units that end within this stage
      if (done1 > done0) {
        while (cur < done1) flush(cur++, 2);
        ok = consumer_sync();
        if (!ok) break;
        for (int v = done0; v < done1; ++v) {
          const int x = (u1a + v) / P, j = (u1a + v) - x * P;
          const int first = l_first[x], cnt = l_first[x + 1] - first;
          for (int q = threadIdx.x; q < 16 * cnt; q += 32 * kMoeCW) {
            const int row = q & 15, col = q >> 4;
            if (!AWQ_CHECK(first + col < n_assign && 16 * j + row < a.I)) continue;
            float hv = silu_mul(sum_of(v, 0, col, row), sum_of(v, 1, col, row)) * l_p[first + col];
            if (a.h_scale != nullptr) hv = __fdiv_rn(hv, __ldg(a.h_scale + static_cast<size_t>(l_expert[x]) * a.I + 16 * j + row));
            a.h[static_cast<size_t>(first + col) * a.I + 16 * j + row] = __float2half_rn(hv);
          }
        }
      }
    }
  }

  // ---- grid-wide barrier: every CTA's h is written (release) and visible (acquire)
  __threadfence();
  ok = ok && consumer_sync();
  if (ok && threadIdx.x == 0) {
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
  }
  ok = ok && consumer_sync() && *s_abort == 0;

  // ---- phase 2
  {
    int cur = 0;
    clear();
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = 0; ok && i < n2; i += len2) {
      const int n = min(len2, n2 - i);
      ok = wait_full();
      if (!ok) break;
      const uint8_t* sb = smem + slot * kMoeStage;
      for (int it = warp; it < n; it += kMoeCW) {
        const int u = (i + it) / ipu2, q = (i + it) % ipu2;
        while (cur < u) flush(cur++, 1);
        const int x = q / Q2, pr = q - x * Q2;
        const __half* hr[MTT];
        bool mine[MTT][2];                                 // whether this lane's two columns chose the expert
#pragma unroll
        for (int j = 0; j < MTT; ++j) {
          const int s = 8 * j + r < a.T ? l_map[x * a.T + 8 * j + r] : -1;
          hr[j] = s >= 0 ? a.h + static_cast<size_t>(s) * a.I + pr * 256 + 16 * t : nullptr;
#pragma unroll
          for (int c = 0; c < 2; ++c) mine[j][c] = 8 * j + 2 * t + c < a.T && l_map[x * a.T + 8 * j + 2 * t + c] >= 0;
        }
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          if (2 * pr + gg >= G2) break;
          uint4 xv[2][MTT][2];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int j = 0; j < MTT; ++j) {
              xv[kk][j][0] = hr[j] != nullptr ? ld_coherent_v4(hr[j] + gg * 128 + kk * 64) : zero;
              xv[kk][j][1] = hr[j] != nullptr ? ld_coherent_v4(hr[j] + gg * 128 + kk * 64 + 8) : zero;
            }
          const uint8_t* cb = sb + it * kPairCodeBytes + gg * 1024 + lane * 16;
          const uint4 w0 = *reinterpret_cast<const uint4*>(cb);
          const uint4 w1 = *reinterpret_cast<const uint4*>(cb + 512);
          const uint32_t sv = *reinterpret_cast<const uint32_t*>(sb + kMoeOffS + it * kPairScaleBytes + gg * 32 + r * 4);
          const uint32_t zz = sb[kMoeOffZ + it * kPairZeroBytes + gg * 8 + r];
          float g[MTT][4] = {};
          gemv_group<MTT>(g, w0, w1, xv, sv, zz);
#pragma unroll
          for (int j = 0; j < MTT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (mine[j][c & 1]) acc[0][j][c] += g[j][c];
        }
      }
      release();
      const int done0 = i / ipu2, done1 = (i + n) / ipu2;
      if (done1 > done0) {
        while (cur < done1) flush(cur++, 1);
        ok = consumer_sync();
        if (!ok) break;
        for (int v = done0; v < done1; ++v)
          for (int q = threadIdx.x; q < 16 * a.T; q += 32 * kMoeCW) {
            const int row = q & 15, col = q >> 4;
            if (!AWQ_CHECK(16 * (u2a + v) + row < a.K)) continue;
            a.y[static_cast<size_t>(col) * a.K + 16 * (u2a + v) + row] = __float2half_rn(sum_of(v, 0, col, row));
          }
      }
    }
  }
}

}  // namespace awq
