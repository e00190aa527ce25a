// awq_moe.cuh — a whole mixture-of-experts layer for a few tokens (T <= 32), experts in packed
// 4-bit weights, in one kernel.
//
//   l_te = x_t . Wr_e              the top_k experts of token t by l (ties: lowest index)
//   p_te = exp(l_te - max) / sum   the sum over all experts, or over the chosen ones (renormalize)
//   h    = SiLU(x_t . Wg_e^T) * (x_t . Wu_e^T) [/ s_e]                 (fp32)
//   y_t  = sum over the chosen e of p_te * (h . Wd_e^T)
//
// The layer is bound by the packed weights of the experts that are chosen at all (0.52 bytes per
// weight). One CTA per SM, launched cooperatively, in four phases with a grid-wide barrier between:
//   0  the router's logits, a CTA per expert and up to 8 tokens; after the barrier every CTA picks all
//      tokens' experts itself and sorts the choices into blocks of at most 8 tokens of one expert;
//   1  h for every unit (block, 16 gate rows and their 16 up rows);
//   2  fp32 partial sums of y for every unit (block, part of K, two 16-row output tiles);
//   3  y, the partial sums added in a fixed order.
// In phases 1 and 2 the last units go to whoever is done first: SMs differ by up to 15% in the bandwidth
// they get. An expert with more than 8 tokens has several blocks, whose weights come from L2 after the
// first: each block's activation fragments then fit a warp's registers. Phase 2 goes through partial
// sums so that its units are as many and as small as phase 1's and a warp keeps its fragments along the
// tiles; summing all blocks of a tile in one CTA left it at 59% of the HBM rate.
//
// Per CTA: a producer lane streams both phases' packed weights through one ring of shared memory
// without waiting for the barrier, so phase 2's first weights arrive while phase 1 ends. A stage holds
// 16 (tile, group pair) items of each of two tiles, one of each for each of the 16 consumer warps, which so
// split the tiles' K. A warp's activation fragments stay in registers while it walks along the tiles of a
// block. Each warp leaves its sums of a tile in shared memory, and epilogue warps add them in warp order
// and apply SiLU (phase 1) or the weight p (phase 2): results repeat bit for bit. h stays in fp32 and enters
// phase 2 as 21-bit integers with a power of two per token and 256 values (MoeInts), so y's rounding is the
// only one to fp16.
//
// Measured (8 experts of 4096 x 14336, two per token): 1 token 54 us, of which 28 are the HBM time of the
// weights and 17 to 20 the router, three barriers (1.3 to 2 us each), the first and last stages and the
// integers of h; 8 tokens 144 (floor 96); 32 tokens 212 to 218 (floor 112), bound by the consumers'
// instructions, of which every block of 8 tokens has its own. 64 experts of 2048 x 1408, six per token, 5
// tokens: 46 (floor 17). A warp's integers of h take 1300 to 2000 cycles each time it comes to another block
// or part of K. (With h in fp16 the calls took 51, 138, 205 and 42 us, but its rounding doubled the output's
// squared error, and what lies below 2^-14 lost more, down to all of it.)
//
// The kernel neither starts before its predecessor has ended nor lets its successor start early: CTAs
// that wait for it could otherwise hold the registers that its own last CTAs need, and the barrier
// would never be complete.
#pragma once

#include <type_traits>

#include "awq_common.cuh"
#include "awq_gemm.cuh"

namespace awq {

constexpr int kMoeMaxTokens = 32;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;

struct MoeArgs {
  const __half* x;                             // [T, K]
  const __half* router;                        // [E, K]
  const uint8_t *gu_q, *gu_s, *gu_z;           // gate/up layers, packed layout v2, one after another
  const uint8_t *dn_q, *dn_s, *dn_z;           // down layers
  size_t gu_pairs, dn_pairs;                   // (tile, group pair) items of one expert's layer
  const float* h_scale;                        // [E, I] or null
  float* logits;                               // [T, E]
  float* h;                                    // [T * top, I]
  float* part;                                 // [T * top, chunks of I, K]
  __half* y;                                   // [T, K]
  int T, E, K, I, top, renorm;
};

constexpr int kMoeCW = 16;                      // consumer warps
constexpr int kMoeEpi = 3;                      // epilogue warps
constexpr int kMoeThreads = 32 * (kMoeCW + 1 + kMoeEpi);   // + producer
constexpr int kMoeStages = 2;
constexpr int kMoeTile = 16;                    // (tile, group pair) items of a stage's half, one per consumer warp
constexpr int kMoeOffS = 2 * kMoeTile * kPairCodeBytes;
constexpr int kMoeOffZ = kMoeOffS + 2 * kMoeTile * kPairScaleBytes;
constexpr int kMoeStage = kMoeOffZ + 2 * kMoeTile * kPairZeroBytes;     // 68096 bytes
static_assert(kMoeStage % 128 == 0, "ring stages stay aligned");

// A record is one warp's fp32 sums of one 16-row tile, [column][20] (20: rows padded so that the
// fragment stores hit distinct banks). A buffer holds two tiles' records of every warp.
constexpr int kMoeRec = 8 * 20;
constexpr int kMoeBufs = 2;
// Routing lists: the choices in (token, rank) order (expert, weight), whose place the blocks (expert,
// first slot; one more) take; then by slot the token, weight and expert; and the choices' slots.
__host__ __device__ inline int moe_list_ints(int T, int top) { return 6 * T * top + 1; }
__host__ __device__ inline int moe_smem_bytes(int T, int top) {
  return kMoeStages * kMoeStage + kMoeBufs * kMoeCW * 2 * kMoeRec * 4 + (kMoeStages + kMoeBufs) * 16 +
         (2 * kMoeStages + 2 * kMoeBufs + 2) * 8 + 8 + moe_list_ints(T, top) * 4;
}

// How a strip (one tile of one block, Q group pairs along its K) is cut into stages. Up to 8 pairs:
// 2^shift strips share a stage's half, `wide` warps each. More: `chunks` stages of up to `len` pairs.
struct MoeCut {
  int Q, wide, shift, strips, chunks, len;
  __host__ __device__ explicit MoeCut(int q) : Q(q) {
    shift = q <= 1 ? 4 : q <= 2 ? 3 : q <= 4 ? 2 : q <= 8 ? 1 : 0;
    strips = 1 << shift;
    wide = kMoeTile >> shift;
    chunks = (q + kMoeTile - 1) / kMoeTile;
    len = (q + chunks - 1) / chunks;
  }
};

// Arrivals at the grid-wide barriers since the library was loaded. Every CTA of a launch arrives at
// each barrier exactly once, also when it has given up a wait, so the count is a multiple of the grid
// size between barriers. One counter is enough: a CTA takes more than half of an SM's shared memory
// and the grid all SMs, so two launches never run at once as long as none of a launch's CTAs ends before
// all have arrived at its last barrier. Only a CTA that has given up a wait does: a launch on another
// stream may then start beside the ones that are late, count their arrivals as its own and pass a barrier
// early. Its results are undefined like the first one's (the header says so); its accesses stay in bounds,
// as the lists that it reads are its own CTA's, and later launches find a multiple of the grid size again.
__device__ unsigned long long g_moe_arrivals = 0;
static_assert(kMoeStages * kMoeStage > 114 * 1024, "two of these CTAs must not fit one SM");

// Tickets drawn for the units of phases 1 and 2 since the library was loaded. A launch reads the counts
// before its first barrier and draws after it, so all of its CTAs start from the same counts.
__device__ __align__(16) unsigned long long g_moe_tickets[2] = {0, 0};

// The arrival releases, at GPU scope, what the thread has written or seen synchronised from its CTA's
// other threads, and the wait acquires it, so a CTA barrier on either side completes the chain.
__device__ __forceinline__ unsigned long long moe_arrive() {
  unsigned long long old;
  asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(&g_moe_arrivals) : "memory");
  return old - old % gridDim.x + gridDim.x;    // the count at which the barrier is complete
}
__device__ __forceinline__ void moe_await(unsigned long long target, volatile int* abort, unsigned long long budget) {
  const uint64_t t0 = globaltimer_ns();
  while (!*abort) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(&g_moe_arrivals) : "memory");
    if (v >= target) return;
    if (globaltimer_ns() - t0 > budget) {
      *abort = 1;
      atomicOr(&g_dev_status, kDevStatusTimeout);
    }
  }
}

__device__ __forceinline__ uint4 ld_coherent_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// One warp picks a token's experts from its E <= 32 PER logits. `ord` orders the logits as integers; a
// NaN is 1, below every number, and a chosen expert (or none) 0, so that `top` distinct experts are
// found whatever the logits are.
template <int PER>
__device__ __forceinline__ void moe_pick(const float* logits, int E, int top, bool renorm, int* ids, float* p) {
  const int lane = threadIdx.x & 31;
  uint32_t ord[PER];
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    ord[i] = 0;
    l[i] = -INFINITY;
    if (e < E) asm volatile("ld.global.f32 %0, [%1];" : "=f"(l[i]) : "l"(logits + e));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t b = __float_as_uint(l[i]);
    if (i * 32 + lane < E) ord[i] = l[i] != l[i] ? 1u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  }
  float mine = 0.0f, best = 0.0f;              // lane k: the logit of the k-th choice
  int mine_id = 0;
  for (int k = 0; k < top; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = max(m, ord[i]);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    uint32_t e = 0xFFFFFFFFu;                  // the lowest index among the equal ones
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (ord[i] == m) e = i * 32 + lane;
    e = __reduce_min_sync(0xFFFFFFFFu, e);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane == static_cast<int>(e)) ord[i] = 0;
    const float v = m == 1u ? NAN : __uint_as_float((m & 0x80000000u) ? m ^ 0x80000000u : ~m);
    if (k == 0) best = v;                      // the largest logit (NaN if all are)
    if (lane == k) { mine = v; mine_id = static_cast<int>(e); }
  }
  const float num = lane < top ? expf(mine - best) : 0.0f;
  float total = num;
  if (!renorm) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane < E) total += expf(l[i] - best);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane < top) {
    ids[lane] = mine_id;
    p[lane] = __fdiv_rn(num, total);
  }
}

// acc += S (sum x q - z sum x) for the lane's four sums of one group (columns 2t, 2t+1 of rows r and
// r+8). tq carries 2^-24 in row r and 2^-20 in row r+8, and so does z as the bits of fp16 subnormals;
// acc keeps those factors until the epilogue.
__device__ __forceinline__ void moe_scale(float (&acc)[4], const float (&tq)[4], const float (&xs)[2], uint32_t sv, uint32_t zz) {
  const float2 s = half2_bits_to_float2(sv), z = half2_bits_to_float2((zz * 0x10001u) & 0x00F0000Fu);
  acc[0] = fmaf(s.x, fmaf(-z.x, xs[0], tq[0]), acc[0]);
  acc[1] = fmaf(s.x, fmaf(-z.x, xs[1], tq[1]), acc[1]);
  acc[2] = fmaf(s.y, fmaf(-z.y, xs[0], tq[2]), acc[2]);
  acc[3] = fmaf(s.y, fmaf(-z.y, xs[1], tq[3]), acc[3]);
}

// The activation fragments of one group pair for one 8-token tile, and their sums per group.
struct MoeFrag {
  uint4 v[2][2][2];   // [group][64-k tile][half]
  float s[2][2];      // [group][column 2t, 2t+1]
};

// The codes, scales and zero points of one item, in registers: the stage can be refilled while the
// products are computed.
struct MoeItem {
  uint4 w[2][2];      // [group][64-k tile]
  uint32_t s[2], z[2];
};

// acc += the item's products with the fragments. A code pair masked out of its word is a pair of fp16
// subnormals q 2^-24 (16 q 2^-24 in the odd nibbles, rows r+8): one AND makes an operand of the MMA, whose
// products are exact. The zero point costs no instruction per code, it enters once per group with the
// group's activation sum. The two groups' MMA chains run side by side.
__device__ __forceinline__ void moe_products(float (&acc)[4], const MoeItem& m, const MoeFrag& f) {
  float tq[2][4];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint4& wv = m.w[g][kk];
        const uint32_t q = (s4 == 0) ? wv.x : (s4 == 1) ? wv.y : (s4 == 2) ? wv.z : wv.w;
        const uint32_t q8 = q >> 8;
        const uint32_t a[4] = {q & 0x000F000Fu, q & 0x00F000F0u, q8 & 0x000F000Fu, q8 & 0x00F000F0u};
        const uint4& xq = f.v[g][kk][s4 >> 1];
        const uint32_t b0 = (s4 & 1) ? xq.z : xq.x, b1 = (s4 & 1) ? xq.w : xq.y;
        if (kk == 0 && s4 == 0) mma_m16n8k16_f32_zero(tq[g], a, b0, b1);
        else mma_m16n8k16_f32(tq[g], a, b0, b1);
      }
#pragma unroll
  for (int g = 0; g < 2; ++g) moe_scale(acc, tq[g], f.s[g], m.s[g], m.z[g]);
}

// h is fp32 and enters phase 2 as integers: a token's 256 values of a group pair are H / 2^(19 - e), e the
// exponent of the largest magnitude and H = rint(h 2^(19 - e)), |H| <= 2^20, so that each is off by at most
// 2^-20 of the largest. The sums of (q - z) H are exact: |sum| <= 15 * 128 * 2^20 < 2^31. H's three bytes
// are the operands of three products with the codes as bytes: mma.sync in 8-bit integers takes 32 k in the
// two cycles in which fp16 takes 16 (measured per SM), and the codes of 32 k four ANDs and two shifts, half
// of what fp16 operands take. h as a sum of two fp16 values needs two products of that kind and 32 registers
// more, which spill: 22% of the call at 8 tokens over fp16 alone (123 to 150 us), where the integers cost 6%
// (136 to 144).
struct MoeInts {
  uint32_t v[3][2][2][4];   // [byte of H, highest first][group][64-k tile][4 k]
  uint32_t s[2][2];         // sum of H: [group][column 2t, 2t+1]
  float inv[2];             // 2^(e - 19) of the columns; NaN where a value is not finite
};

// D = A . B + C, A unsigned bytes, B signed or unsigned bytes, int32.
template <bool SIGNED>
__device__ __forceinline__ void mma_m16n8k32_i32(uint32_t (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                                 const uint32_t (&c)[4]) {
  if (SIGNED)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

// acc += S sum (q - z) H of one group (w: its two 64-k tiles). A word's low nibbles are row r at k, k+2, k+1,
// k+3, its high nibbles row r + 8.
__device__ __forceinline__ void moe_int_products(float (&acc)[4], const uint4 (&w)[2], uint32_t sv, uint32_t zz, const MoeInts& f, int g) {
  uint32_t d[3][4] = {};
#pragma unroll
  for (int kt = 0; kt < 2; ++kt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t q0 = j ? w[kt].z : w[kt].x, q1 = j ? w[kt].w : w[kt].y;
      const uint32_t a[4] = {q0 & 0x0F0F0F0Fu, (q0 >> 4) & 0x0F0F0F0Fu, q1 & 0x0F0F0F0Fu, (q1 >> 4) & 0x0F0F0F0Fu};
      mma_m16n8k32_i32<true>(d[0], a, f.v[0][g][kt][2 * j], f.v[0][g][kt][2 * j + 1], d[0]);
      mma_m16n8k32_i32<false>(d[1], a, f.v[1][g][kt][2 * j], f.v[1][g][kt][2 * j + 1], d[1]);
      mma_m16n8k32_i32<false>(d[2], a, f.v[2][g][kt][2 * j], f.v[2][g][kt][2 * j + 1], d[2]);
    }
  const float2 sc = half2_bits_to_float2(sv);
#pragma unroll
  for (int j = 0; j < 4; ++j) {                // modulo 2^32 on the way, in range at the end
    const uint32_t z = j < 2 ? zz & 15u : zz >> 4;
    const uint32_t v = (((d[0][j] << 8) + d[1][j]) << 8) + d[2][j] - z * f.s[g][j & 1];
    acc[j] = fmaf(j < 2 ? sc.x : sc.y, static_cast<float>(static_cast<int>(v)), acc[j]);
  }
}

__global__ void __launch_bounds__(kMoeThreads, 1) awq_moe_kernel(const MoeArgs a) {
  constexpr int S = kMoeStages;
  extern __shared__ __align__(128) uint8_t smem[];
  float* rec = reinterpret_cast<float*>(smem + S * kMoeStage);
  // what a stage or a record holds: block, first unit, units (0: the phase ends), chunk of K
  int4* stage_of = reinterpret_cast<int4*>(rec + kMoeBufs * kMoeCW * 2 * kMoeRec);
  int4* event_of = stage_of + S;
  uint64_t* full = reinterpret_cast<uint64_t*>(event_of + kMoeBufs);
  uint64_t* empty = full + S;
  uint64_t* rfull = empty + S;                 // record buffers
  uint64_t* rempty = rfull + kMoeBufs;
  uint64_t* edone = rempty + kMoeBufs;         // this CTA's results of the phase are stored
  uint64_t* go = edone + 1;                    // everybody's are
  volatile int* s_abort = reinterpret_cast<volatile int*>(go + 1);
  const int n_assign = a.T * a.top;
  int* l_ids = const_cast<int*>(s_abort) + 2;
  float* l_pa = reinterpret_cast<float*>(l_ids + n_assign);
  int* l_expert = l_ids;
  int* l_first = l_ids + n_assign;
  int* l_token = l_first + n_assign + 1;
  float* l_p = reinterpret_cast<float*>(l_token + n_assign);
  int* l_slot = reinterpret_cast<int*>(l_p + n_assign);        // expert of a slot, times two, + 1 where a block starts
  int* l_of = l_slot + n_assign;               // slot of a choice

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMoeCW);
    }
    for (int b = 0; b < kMoeBufs; ++b) {
      mbar_init(&rfull[b], kMoeCW);
      mbar_init(&rempty[b], kMoeEpi);
    }
    mbar_init(edone, kMoeEpi);
    mbar_init(go, 1);
    *s_abort = 0;
    mbar_fence_init();
  }
  const unsigned long long budget = g_wait_budget_ns;
  const int c0 = blockIdx.x, nc = gridDim.x;

  // ---- phase 0: logits of NT tokens with one expert, the consumer warps splitting K; as few tokens at a
  // time as the CTAs allow
  unsigned long long tickets[2] = {0, 0};
  {
    if (threadIdx.x == 32 * kMoeCW)
      asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];"
                   : "=l"(tickets[0]), "=l"(tickets[1])
                   : "l"(&g_moe_tickets)
                   : "memory");
    float* part = rec;                         // [2][kMoeCW][8]
    auto logits = [&](auto n) {
      constexpr int NT = decltype(n)::value;
      const int tasks = a.E * ((a.T + NT - 1) / NT);
      for (int i = c0, it = 0; i < tasks; i += nc, it ^= 1) {
        const int e = i % a.E, t0 = i / a.E * NT;
        if (warp < kMoeCW) {
          const __half* wr = a.router + static_cast<size_t>(e) * a.K;
          float acc[NT] = {};
          for (int c = threadIdx.x; c < a.K / 8; c += 32 * kMoeCW) {
            const uint4 wv = __ldg(reinterpret_cast<const uint4*>(wr + c * 8));
            uint4 xv[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
              xv[t] = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(min(t0 + t, a.T - 1)) * a.K + c * 8));
            const uint32_t w4[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t x4[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 wf = half2_bits_to_float2(w4[j]), xf = half2_bits_to_float2(x4[j]);
                acc[t] = fmaf(wf.x, xf.x, acc[t]);
                acc[t] = fmaf(wf.y, xf.y, acc[t]);
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xFFFFFFFFu, acc[t], o);
            if (lane == 0) part[(it * kMoeCW + warp) * 8 + t] = acc[t];
          }
        }
        __syncthreads();
        if (threadIdx.x < NT && t0 + threadIdx.x < a.T) {
          float v = 0.0f;
          for (int w = 0; w < kMoeCW; ++w) v += part[(it * kMoeCW + w) * 8 + threadIdx.x];
          a.logits[static_cast<size_t>(t0 + threadIdx.x) * a.E + e] = v;
        }
      }
    };
    if (a.E * a.T <= nc) logits(std::integral_constant<int, 1>{});
    else if (a.E * ((a.T + 1) / 2) <= nc) logits(std::integral_constant<int, 2>{});
    else if (a.E * ((a.T + 3) / 4) <= nc) logits(std::integral_constant<int, 4>{});
    else logits(std::integral_constant<int, 8>{});
    __syncthreads();
    if (threadIdx.x == 0) moe_await(moe_arrive(), s_abort, budget);
    __syncthreads();
  }

  // ---- the choices, and the blocks: slots ordered by expert, then token
  for (int t = warp; t < a.T; t += kMoeThreads / 32) {
    const float* l = a.logits + static_cast<size_t>(t) * a.E;
    int* ids = l_ids + t * a.top;
    float* p = l_pa + t * a.top;
    if (a.E <= 32) moe_pick<1>(l, a.E, a.top, a.renorm != 0, ids, p);
    else if (a.E <= 128) moe_pick<4>(l, a.E, a.top, a.renorm != 0, ids, p);
    else moe_pick<kMoeMaxExperts / 32>(l, a.E, a.top, a.renorm != 0, ids, p);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_assign; i += kMoeThreads) {
    const int e = l_ids[i];
    int rank = 0, first = 0;
    for (int j = 0; j < n_assign; ++j) {
      const int o = l_ids[j];
      first += o < e;
      rank += o == e && j < i;
    }
    l_token[first + rank] = i / a.top;
    l_p[first + rank] = l_pa[i];
    l_slot[first + rank] = 2 * e + (rank % 8 == 0);
    l_of[i] = first + rank;
  }
  __syncthreads();
  int V = 0;                                   // blocks
  for (int b = 0; b < n_assign; b += 32) {     // every warp counts, one writes
    const int v = b + lane < n_assign ? l_slot[b + lane] : 0;
    const uint32_t starts = __ballot_sync(0xFFFFFFFFu, v & 1);
    if (warp == 0 && (v & 1)) {
      const int idx = V + __popc(starts & ((1u << lane) - 1));
      l_expert[idx] = v >> 1;
      l_first[idx] = b + lane;
    }
    V += __popc(starts);
  }
  if (threadIdx.x == 0) l_first[V] = n_assign;
  __syncthreads();

  // ---- phases 1 and 2. A unit is the items of two tiles, j and j + P (gate and up; the two halves of
  // y). In phase 2 every chunk of K has units of its own. The first units, all of them if they are few,
  // are divided evenly, and the last eighth of many is drawn. The producer leaves word of each stage's
  // content beside it, from which the others learn what to do.
  const MoeCut k1((a.K / kGroup + 1) / 2), k2((a.I / kGroup + 1) / 2);
  const uint32_t hint = brief_hint(budget);
  int slot = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++slot == S) { slot = 0; phase ^= 1; }
  };
  int rbuf = 0;                                // record buffer of the current event
  uint32_t rphase = 0;
  auto next_event = [&]() {
    if (++rbuf == kMoeBufs) { rbuf = 0; rphase ^= 1; }
  };
  auto rec_of = [&](int w, int half) { return rec + ((rbuf * kMoeCW + w) * 2 + half) * kMoeRec; };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, mbar_wait_brief(bar, parity, hint, s_abort, budget));
  };

  if (warp == kMoeCW) {
    // ---------------------------------------------------------------- producer lane
    if (lane != 0) return;
    int issued = 0;
    constexpr int kItem = kPairCodeBytes + kPairScaleBytes + kPairZeroBytes;
    auto produce = [&](bool second) -> bool {
      const MoeCut& k = second ? k2 : k1;
      const uint8_t *q = second ? a.dn_q : a.gu_q, *sc = second ? a.dn_s : a.gu_s, *z = second ? a.dn_z : a.gu_z;
      const size_t pairs = second ? a.dn_pairs : a.gu_pairs;
      const int P = second ? a.K / 32 : a.I / 16;
      auto stage = [&](int4 what) -> bool {
        if (!mbar_wait_brief(&empty[slot], phase ^ 1, hint, s_abort, budget)) return false;
        uint8_t* sb = smem + slot * kMoeStage;
        const int p0 = what.w * k.len, n = what.z * min(k.len, k.Q - p0);      // items of a half
        stage_of[slot] = what;
        mbar_arrive_expect_tx(&full[slot], 2 * n * kItem);
        if (n > 0 && AWQ_CHECK(what.x >= 0 && what.x < V && slot < S)) {
          size_t tp = static_cast<size_t>(l_expert[what.x]) * pairs + static_cast<size_t>(what.y) * k.Q + p0;
          for (int h = 0; h < 2; ++h) {
            if (AWQ_CHECK(n <= kMoeTile && tp + n <= a.E * pairs)) {
              bulk_g2s(sb + h * kMoeTile * kPairCodeBytes, q + tp * kPairCodeBytes, n * kPairCodeBytes, &full[slot]);
              bulk_g2s(sb + kMoeOffS + h * kMoeTile * kPairScaleBytes, sc + tp * kPairScaleBytes, n * kPairScaleBytes, &full[slot]);
              bulk_g2s(sb + kMoeOffZ + h * kMoeTile * kPairZeroBytes, z + tp * kPairZeroBytes, n * kPairZeroBytes, &full[slot]);
            }
            tp += static_cast<size_t>(P) * k.Q;
          }
        }
        ++issued;
        advance();
        return true;
      };
      auto units = [&](int u, int end) -> bool {
        while (u < end) {
          const int v = u / P, j = u - v * P;
          const int x = second ? v / k.chunks : v, n = min(k.strips, min(P - j, end - u));
          for (int c = second ? v - x * k.chunks : 0;; ++c) {
            if (!stage(make_int4(x, j, n, c))) return false;
            if (second || c + 1 == k.chunks) break;
          }
          u += n;
        }
        return true;
      };
      const int all = (second ? V * k.chunks : V) * P;
      const int even = all < 8 * nc * k.strips ? all : all - all / 8;
      if (!units(static_cast<int>(static_cast<long long>(even) * c0 / nc),
                 static_cast<int>(static_cast<long long>(even) * (c0 + 1) / nc)))
        return false;
      while (even < all) {                     // the ring holds several stages while a draw takes its time
        unsigned long long drawn;
        asm volatile("atom.add.relaxed.gpu.global.u64 %0, [%1], 1;" : "=l"(drawn) : "l"(&g_moe_tickets[second]) : "memory");
        const long long u = even + static_cast<long long>(drawn - (second ? tickets[1] : tickets[0])) * k.strips;
        if (u >= all) break;
        if (!units(static_cast<int>(u), static_cast<int>(min(u + k.strips, static_cast<long long>(all))))) return false;
      }
      return stage(make_int4(0, 0, 0, 0));     // the phase ends
    };
    if (produce(false)) produce(true);
    // drain: every copy this thread issued has landed before the CTA may exit
    int never = 0;
    for (int i = max(0, issued - S); i < issued; ++i)
      mbar_wait_bounded(&full[i % S], static_cast<uint32_t>((i / S) & 1), &never, kDrainBudgetNs);
    return;
  }

  if (warp > kMoeCW) {
    // ---------------------------------------------------------------- epilogue warps
    // the sum of the records of warps w0..w0+nw-1
    auto sum = [&](int half, int w0, int nw, int col, int row) {
      const float* p = rec_of(w0, half) + col * 20 + row;
      float v = 0.0f;
      if (nw == kMoeCW) {
#pragma unroll
        for (int w = 0; w < kMoeCW; ++w) v += p[w * 2 * kMoeRec];
      } else {
        for (int w = 0; w < nw; ++w) v += p[w * 2 * kMoeRec];
      }
      return v;
    };
    const int lane0 = 32 * (warp - kMoeCW - 1) + lane;
    bool ok = true;
    for (int ph = 0; ph < 2; ++ph) {
      while (ok) {
        ok = warp_wait(&rfull[rbuf], rphase);
        if (!ok) break;
        const int4 what = event_of[rbuf];
        const int x = what.x, nu = what.z;
        if (nu > 0) {
          const int first = l_first[x], cnt = l_first[x + 1] - first;
          if (ph == 0) {
            for (int q = lane0; q < (16 * cnt) << k1.shift; q += 32 * kMoeEpi) {
              const int row = q & 15, i = (q >> 4) & (k1.strips - 1), col = q >> (4 + k1.shift);
              const int i_row = 16 * (what.y + i) + row;
              if (i >= nu || !AWQ_CHECK(first + col < n_assign && i_row < a.I && i * k1.wide + k1.len <= kMoeCW)) continue;
              const float code = row < 8 ? 16777216.0f : 1048576.0f;           // the factors that the codes carry
              const float g = code * sum(0, i * k1.wide, k1.len, col, row), v = code * sum(1, i * k1.wide, k1.len, col, row);
              float hv = silu_mul(g, v);
              if (a.h_scale != nullptr) hv = __fdiv_rn(hv, __ldg(a.h_scale + static_cast<size_t>(l_expert[x]) * a.I + i_row));
              a.h[static_cast<size_t>(first + col) * a.I + i_row] = hv;
            }
          } else {
            const int nw = min(k2.len, k2.Q - what.w * k2.len);
            for (int q = lane0; q < (32 * cnt) << k2.shift; q += 32 * kMoeEpi) {
              const int row = q & 15, i = (q >> 4) & (k2.strips - 1), half = (q >> (4 + k2.shift)) & 1, col = q >> (5 + k2.shift);
              const int k = 16 * (half * (a.K / 32) + what.y + i) + row;
              if (i >= nu || !AWQ_CHECK(first + col < n_assign && k < a.K && i * k2.wide + nw <= kMoeCW && what.w < k2.chunks)) continue;
              a.part[(static_cast<size_t>(first + col) * k2.chunks + what.w) * a.K + k] =
                  l_p[first + col] * sum(half, i * k2.wide, nw, col, row);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rempty[rbuf]);
        next_event();
        if (nu == 0) break;
      }
      // the grid-wide barrier: every CTA's results are written and visible
      __syncwarp();
      if (lane == 0) mbar_arrive(edone);
      if (warp == kMoeCW + 1) {
        warp_wait(edone, ph);
        if (lane == 0) {
          moe_await(moe_arrive(), s_abort, budget);
          if (*s_abort == 0) mbar_arrive(go);
        }
        __syncwarp();   // the other lanes block here: polling ahead, they could keep lane 0 from its turn
      }
    }
    return;
  }

  // ------------------------------------------------------------------ consumer warps
  const int r = lane >> 2, t = lane & 3;
  // The fragments of pair `pr` for a block's tokens, and their sums; `row` is the lane's token.
  auto load_frag = [&](MoeFrag& f, const __half* row, int pr, int G) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          f.v[g][kk][i] = 2 * pr + g < G ? ld_coherent_v4(row + pr * 256 + g * 128 + kk * 64 + 16 * t + 8 * i)
                                         : make_uint4(0, 0, 0, 0);   // the padding group
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
  // The same of h; `row` is fp32.
  auto load_ints = [&](MoeInts& f, const float* row, int pr, int G) {
    float v[2][2][4][4];
    float top = 0.0f;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = 2 * pr + g < G ? ld_coherent_v4(row + pr * 256 + g * 128 + kk * 64 + 16 * t + 4 * i)
                                         : make_uint4(0, 0, 0, 0);   // the padding group
          v[g][kk][i][0] = __uint_as_float(w.x);
          v[g][kk][i][1] = __uint_as_float(w.y);
          v[g][kk][i][2] = __uint_as_float(w.z);
          v[g][kk][i][3] = __uint_as_float(w.w);
        }
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top = max_abs_nan(top, v[g][kk][i][0], v[g][kk][i][1]);
          top = max_abs_nan(top, v[g][kk][i][2], v[g][kk][i][3]);
        }
    const float other = __shfl_xor_sync(0xFFFFFFFFu, top, 1);
    top = max_abs_nan(top, other, other);
    const float others = __shfl_xor_sync(0xFFFFFFFFu, top, 2);               // the four lanes of a token
    const uint32_t bits = __float_as_uint(max_abs_nan(top, others, others)) & 0x7FFFFFFFu;
    const uint32_t e = max(bits >> 23, 27u);   // 127 more than the exponent; values below 2^-100 go by that one
    const float scale = __uint_as_float((273u - e) << 23);     // 2^(19 - exponent)
    const float inv = bits >= 0x7F800000u ? NAN : __uint_as_float((e - 19u) << 23);
    f.inv[0] = __shfl_sync(0xFFFFFFFFu, inv, 8 * t);
    f.inv[1] = __shfl_sync(0xFFFFFFFFu, inv, 8 * t + 4);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t sum = 0;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // 1.5 2^23 + H: H, rounded half to even, in the low bits; plus 64 in byte 2
          uint32_t n[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) n[c] = __float_as_uint(fmaf(v[g][kk][i][c], scale, 12582912.0f));
          sum += n[0] + n[1];
          sum += n[2] + n[3];
          const uint32_t p = __byte_perm(n[0], n[2], 0x5140), q = __byte_perm(n[1], n[3], 0x5140);   // in the codes' order
          const uint32_t hi = __byte_perm(__byte_perm(n[0], n[2], 0x0062), __byte_perm(n[1], n[3], 0x0062), 0x5410);
          f.v[0][g][kk][i] = (hi ^ 0x40404040u) | (~(hi << 1) & 0x80808080u);      // less 64, from 48..80
          f.v[1][g][kk][i] = __byte_perm(p, q, 0x7632);
          f.v[2][g][kk][i] = __byte_perm(p, q, 0x5410);
        }
      sum -= 32u * 0x4B400000u;
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      f.s[g][0] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t);
      f.s[g][1] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t + 4);
    }
  };
  // Waits for the stage that `slot` names; whether there is one, and in `what` its content.
  auto next_stage = [&](int4& what) -> bool {
    if (!warp_wait(&full[slot], phase)) return false;
    what = stage_of[slot];
    return true;
  };
  auto release_stage = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    advance();
  };
  auto put = [&](int half, float v0, float v1, float v2, float v3) {
    float* p = rec + rbuf * (kMoeCW * 2 * kMoeRec) + (2 * warp + half) * kMoeRec + 2 * t * 20 + r;
    p[0] = v0;
    p[20] = v1;
    p[8] = v2;
    p[28] = v3;
  };
  auto announce = [&](const int4& what) {
    if (threadIdx.x == 0) event_of[rbuf] = what;
    __syncwarp();
    if (lane == 0) mbar_arrive(&rfull[rbuf]);
    next_event();
  };
  // columns past a block's last token repeat it; they are never used
  auto slot_of = [&](int x) { return l_first[x] + min(r, l_first[x + 1] - l_first[x] - 1); };
  // whether a slot and a pair of groups lie inside the lists and the rows (bounds-checked builds)
  [[maybe_unused]] auto inside = [&](int s, int pr, const MoeCut& k) {
    return s >= 0 && s < n_assign && l_token[s] >= 0 && l_token[s] < a.T && pr >= 0 && pr < k.Q;
  };
  const uint8_t* const item0 = smem + lane * 16;
  auto load_item = [&](uint4 (&w)[2], uint32_t& sv, uint32_t& zz, const uint8_t* sb, int item, int h, int g) {
    const uint8_t* c = sb + (item + h * kMoeTile) * kPairCodeBytes + g * 1024;
    w[0] = *reinterpret_cast<const uint4*>(c);
    w[1] = *reinterpret_cast<const uint4*>(c + 512);
    sv = *reinterpret_cast<const uint32_t*>(sb + kMoeOffS + (item + h * kMoeTile) * kPairScaleBytes + g * 32 + (r - 4 * lane) * 4);
    zz = sb[kMoeOffZ + (item + h * kMoeTile) * kPairZeroBytes + g * 8 + r - 16 * lane];
  };
  auto phase1 = [&]() -> bool {
    const int pl = warp % k1.wide, sub = warp / k1.wide;
    const int item = sub * k1.Q + pl;          // of a stage with several strips, one after another
    float acc[2][4] = {};                      // the unit's two tiles
    MoeFrag f;
    int fx = -1, fc = 0;                       // block and chunk of the fragments
    bool mine = false;                         // whether the warp has a pair of the chunk
    while (true) {
      int4 what;
      if (!next_stage(what)) return false;
      if (what.z > 0) {
        if (what.x != fx || what.w != fc) {
          fx = what.x;
          fc = what.w;
          mine = pl < k1.len && fc * k1.len + pl < k1.Q;
          if (mine && AWQ_CHECK(inside(slot_of(fx), fc * k1.len + pl, k1)))
            load_frag(f, a.x + static_cast<size_t>(l_token[slot_of(fx)]) * a.K, fc * k1.len + pl, a.K / kGroup);
        }
        if (mine && sub < what.z && AWQ_CHECK(item < kMoeTile)) {
          const uint8_t* sb = item0 + slot * kMoeStage;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            MoeItem m;
#pragma unroll
            for (int g = 0; g < 2; ++g) load_item(m.w[g], m.s[g], m.z[g], sb, item, h, g);
            moe_products(acc[h], m, f);
          }
        }
      }
      release_stage();
      if (what.z > 0 && what.w != k1.chunks - 1) continue;   // the unit's sums go on
      if (!warp_wait(&rempty[rbuf], rphase ^ 1)) return false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        put(h, acc[h][0], acc[h][1], acc[h][2], acc[h][3]);
        acc[h][0] = acc[h][1] = acc[h][2] = acc[h][3] = 0.0f;
      }
      announce(what);
      if (what.z == 0) return warp_wait(go, 0);
    }
  };
  auto phase2 = [&]() -> bool {                // every stage completes its units
    const int pl = warp % k2.wide, sub = warp / k2.wide;
    const int item = sub * k2.Q + pl;
    MoeInts f;
    int fx = -1, fc = 0;
    bool mine = false;
    while (true) {
      int4 what;
      if (!next_stage(what)) return false;
      if (what.z > 0 && (what.x != fx || what.w != fc)) {
        fx = what.x;
        fc = what.w;
        mine = pl < k2.len && fc * k2.len + pl < k2.Q;
        if (mine && AWQ_CHECK(inside(slot_of(fx), fc * k2.len + pl, k2)))
          load_ints(f, a.h + static_cast<size_t>(slot_of(fx)) * a.I, fc * k2.len + pl, a.I / kGroup);
      }
      if (!warp_wait(&rempty[rbuf], rphase ^ 1)) return false;
      const bool has = mine && sub < what.z && AWQ_CHECK(item < kMoeTile);
      const uint8_t* sb = item0 + slot * kMoeStage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float acc[4] = {};
        if (has) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint4 w[2];
            uint32_t sv, zz;
            load_item(w, sv, zz, sb, item, h, g);
            moe_int_products(acc, w, sv, zz, f, g);
          }
          acc[0] *= f.inv[0];
          acc[1] *= f.inv[1];
          acc[2] *= f.inv[0];
          acc[3] *= f.inv[1];
        }
        put(h, acc[0], acc[1], acc[2], acc[3]);
      }
      release_stage();
      announce(what);
      if (what.z == 0) return warp_wait(go, 1);
    }
  };
  const bool ok = phase1() && phase2();

  // ---- phase 3: y, four values a thread; a token's partial sums in the order of its choices and of K
  if (!ok) return;
  const int quads = a.K / 4, terms = a.top * k2.chunks;
  for (int q = threadIdx.x * nc + c0; q < a.T * quads; q += nc * 32 * kMoeCW) {
    const int tok = q / quads, k4 = (q - tok * quads) * 4;
    const int* of = l_of + tok * a.top;
    float v[4] = {};
    for (int n = 0; n < terms; n += 4) {       // four loads under way
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = min(n + j, terms - 1) / k2.chunks, c = min(n + j, terms - 1) - i * k2.chunks;
        w[j] = AWQ_CHECK(of[i] >= 0 && of[i] < n_assign && c < k2.chunks && k4 + 4 <= a.K && tok < a.T)
                   ? ld_coherent_v4(a.part + (static_cast<size_t>(of[i]) * k2.chunks + c) * a.K + k4)
                   : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (n + j >= terms) break;
        v[0] += __uint_as_float(w[j].x);
        v[1] += __uint_as_float(w[j].y);
        v[2] += __uint_as_float(w[j].z);
        v[3] += __uint_as_float(w[j].w);
      }
    }
    const __half2 lo = __floats2half2_rn(v[0], v[1]), hi = __floats2half2_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(a.y + static_cast<size_t>(tok) * a.K + k4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

}  // namespace awq
