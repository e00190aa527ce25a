// awq_int8.cuh — linear layers in 8-bit integers: the row quantizer (per token, per output
// channel) and the int8 x int8 product on tcgen05 tensor cores.
//
//   step_r  = max_k |v_rk| / 127                     (fp32, IEEE division)
//   code_rk = rint(v_rk / step_r), -127..127         (IEEE quotient, half to even)
//   y_mn    = fp16(float(sum_k xq_mk wq_nk) * (sx_m * sw_n))
//
// with v = x, x' = fp16(x / s) or w' = fp16(W s), the activation and weight halves of the
// equivalent transform (CSDN "02.02 AWQ"). The sum of products is exact in int32 (K < 2^17).
#pragma once

#include "awq_common.cuh"

namespace awq {

// ---------------------------------------------------------------------------- row quantizer
// One CTA per row. A row that fits (K <= 8 VPT threads) stays in registers between the maximum and the
// codes, so it is read once: 3 bytes of traffic per value. The maximum is taken on the fp16 magnitude
// bits as integers: exact, and a NaN compares above every number, so it reaches the row's step instead
// of being dropped. The codes' IEEE quotients come from a reciprocal per row and two corrections on pairs
// of values (6 instructions a pair).
enum RowScale { kRowPlain = 0, kRowDivide = 1, kRowMultiply = 2 };

__device__ __forceinline__ float2 fma_rn2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul_rn2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
// RN(v / d) for two values, with minus_d = -d and r = RN(1 / d). The product v r is off by less than 1.5
// units in the last place and the first residual correction leaves an error just above half a unit; from
// such a quotient and a correctly rounded reciprocal the second gives RN(v / d) (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990). Exact as long as no step
// under- or overflows: v is 0 or a finite fp16 value, d a row's step.
__device__ __forceinline__ float2 div_rn2(float2 v, float2 minus_d, float2 r) {
  float2 q = mul_rn2(v, r);
  q = fma_rn2(fma_rn2(minus_d, q, v), r, q);
  return fma_rn2(fma_rn2(minus_d, q, v), r, q);
}

// fp16(v / s) or fp16(v * s) of eight values.
template <int MODE>
__device__ __forceinline__ uint4 row_scaled(uint4 v, const float* __restrict__ s, int k) {
  if (MODE == kRowPlain) return v;
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(s + k));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(s + k + 4));
  const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = half2_bits_to_float2(w[j]);
    const float a = MODE == kRowDivide ? __fdiv_rn(f.x, sc[2 * j]) : __fmul_rn(f.x, sc[2 * j]);
    const float b = MODE == kRowDivide ? __fdiv_rn(f.y, sc[2 * j + 1]) : __fmul_rn(f.y, sc[2 * j + 1]);
    const __half2 h = __floats2half2_rn(a, b);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t max_abs_bits(uint32_t m, const uint4& v) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// rint(RN(v / step)) for eight values, packed as int8; step is in [2^-24 / 127, 65504 / 127].
__device__ __forceinline__ uint2 row_codes(const uint4& v, float step, float r) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float2 md = make_float2(-step, -step), r2 = make_float2(r, r);
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = div_rn2(half2_bits_to_float2(w[j]), md, r2);
    // |a| <= 127 (1 + 2^-23): adding 1.5 2^23 rounds half to even and leaves the integer in the low byte
    q[2 * j] = __float_as_uint(a.x + 12582912.0f);
    q[2 * j + 1] = __float_as_uint(a.y + 12582912.0f);
  }
  const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  return make_uint2(lo, hi);
}

// VPT 8-value chunks per thread in registers; VPT = 0: any K, the row is read twice.
// kWeights: the packed output may be read early by a later linear call, so dependents are not
// launched before this kernel ends (the prefetch rule of awq_w8a8_linear).
template <int MODE, int VPT, bool kWeights>
__global__ void __launch_bounds__(1024) awq_quantize_rows_kernel(const __half* __restrict__ x,
                                                                const float* __restrict__ s, int K,
                                                                int8_t* __restrict__ q, float* __restrict__ step_out) {
  if (!kWeights) pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t s_max[32];
  const size_t row = blockIdx.x;
  const __half* xr = x + row * K;
  const int chunks = K / 8, tid = threadIdx.x, nthr = blockDim.x;
  auto inside = [&](int c) { return AWQ_CHECK(c >= 0 && 8 * c + 8 <= K && row < gridDim.x); };
  constexpr int V = VPT > 0 ? VPT : 1;
  uint4 v[V];
  uint32_t m = 0;
  if (VPT > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * nthr;
      v[i] = c < chunks && inside(c) ? ldg_stream_v4(xr + c * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * nthr;
      if (MODE != kRowPlain && c < chunks && inside(c)) v[i] = row_scaled<MODE>(v[i], s, c * 8);
      m = max_abs_bits(m, v[i]);
    }
  } else {
    for (int c = tid; c < chunks && inside(c); c += nthr)
      m = max_abs_bits(m, row_scaled<MODE>(__ldg(reinterpret_cast<const uint4*>(xr + c * 8)), s, c * 8));
  }
  m = __vmaxu2(m, (m >> 16) | (m << 16)) & 0xFFFFu;
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
  m = (tid & 31) < (nthr >> 5) ? s_max[tid & 31] : 0u;
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  const float amax = __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
  const float step = __fdiv_rn(amax, 127.0f);
  if (tid == 0) step_out[row] = step;
  const bool live = m != 0 && m < 0x7C00u;   // an all-zero row, or one with an infinity or NaN, has code 0 throughout
  const float r = live ? __frcp_rn(step) : 0.0f;
  int8_t* qr = q + row * K;
  auto store = [&](int c, const uint4& w) {
    const uint2 o = live ? row_codes(w, step, r) : make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(qr + c * 8) = o;
  };
  if (VPT > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * nthr;
      if (c < chunks && inside(c)) store(c, v[i]);
    }
  } else {
    for (int c = tid; c < chunks && inside(c); c += nthr)
      store(c, row_scaled<MODE>(__ldg(reinterpret_cast<const uint4*>(xr + c * 8)), s, c * 8));
  }
  if (kWeights) __threadfence();
}

// ---------------------------------------------------------------------------- int8 product
// The weights are the MMA's A operand (rows = output channels), the tokens its B operand (columns),
// so one kernel serves one token (BT = 16 columns) and a long prompt (BT = 256). Per CTA:
//   warp 0: producer — per 128-byte k block one TMA box of the tile's weight rows and one of BT token rows
//       (128-byte swizzle, zero fill past M, N and K) into a ring; the first ring pass of weights is
//       requested before the wait on the stream's predecessor;
//   warp 1: tcgen05.mma kind::i8, 128 x BT x 32 per instruction, int32 in tensor memory;
//   warps 2..: epilogue — tcgen05.ld, scales in fp32, fp16 stores, the channels of a warp side by side.
// A tile has 128 MT weight rows. ks > 1: the CTAs of a cluster split a tile's k blocks, and each adds
// the int32 partial sums (exact in any order) of its share of the token columns from distributed
// shared memory.
//
// Bound: up to 64 tokens by the weight bytes. Above, a 128-byte k block takes 390 cycles at 128 columns (32 KB
// of operands), 600 at 256 (48 KB, of which 512 cycles are the tensor pipe's) and 559 for two CTAs of 64
// columns on an SM (48 KB): 82 to 88 bytes per cycle into an SM in every form, which is what bounds them as
// far as these figures tell; the tensor pipe is 78% busy. Run without a pause, the power limit comes on top
// (4096 x 28672 x 4096: 337 us at first, 385 to 395 at the 1.4 GHz that it leaves). The issuing warps were the
// bound before: a wait, four MMAs and a commit took 728 cycles per k block, whatever BT, while a single lane
// ran them; 530 with a converged warp, elect.sync, a wait without the deadline code inside and descriptors in
// 32 bits; 390 when two blocks share a stage. A second producer warp for the tokens was slower: its barrier
// is one more wait for the MMA warp.
// Rows that do not start on 128-byte lines (K % 128 != 0) cost the copies two lines per row: 3 cycles
// per row and k block, which bounds 333 x 5001 x 4112.
struct Int8Args {
  const float* sx;
  const float* sw;
  __half* y;
  int M, N, K;
  int row_blocks, tok_tiles;   // tiles along N and M
  int ks;           // CTAs per tile (cluster size); > 1: one tile per cluster
  int stages, kpb;  // ring stages; 128-byte k blocks per stage
};

constexpr int kI8MaxStages = 16;
constexpr int kI8Bars = 2 * kI8MaxStages + 5;
constexpr int kI8SmemMax = 232448;
constexpr int kI8Fixed = kI8Bars * 8 + 16 + 1024;    // barriers, tensor-memory address, alignment slack

template <int BT, int MT>
struct Int8Cfg {
  // epilogue warps: one per tensor-memory lane quarter, two where a tile has many columns
  static constexpr int kEpi = BT >= 128 ? 8 : 4;
  static constexpr int kThreads = 32 * (2 + kEpi);
  static constexpr int kCols = BT / (kEpi / 4);              // token columns of an epilogue warp
  static constexpr int kSxBytes = kEpi * kCols * 4;          // their sx, a copy per warp
  static constexpr int kAcc = MT * BT;                       // accumulator columns
  static constexpr int kNAcc = 2 * kAcc <= 512 ? 2 : 1;      // two let an epilogue overlap the next tile
  static constexpr int kTmem = kNAcc * kAcc <= 32 ? 32 : kNAcc * kAcc;
  static_assert((kTmem & (kTmem - 1)) == 0 && kTmem <= 512, "tensor memory");
  static constexpr int kChunk = BT < 32 ? 16 : 32;           // accumulator columns per tcgen05.ld
};

// D[tmem] (+)= A . B^T, int8 inputs, int32 accumulate.
__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of tcgen05.mma kind::i8: signed A and B (K-major), int32 D, M x N.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[16]) { tmem_ld_32x32b_x16(taddr, v); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld_32x32b_x32(taddr, v); }

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t cluster_addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
__device__ __forceinline__ __half i8_out(int sum, float sx, float sw) {
  return __float2half_rn(static_cast<float>(sum) * (sx * sw));
}

// One lane of the converged warp. (Code behind elect.sync is known to have one thread, which the copy and
// MMA instructions need.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mbar_expect_tx_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

template <int BT, int MT>
__global__ void __launch_bounds__(Int8Cfg<BT, MT>::kThreads, 1)
    awq_w8a8_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                    const Int8Args a) {
  using C = Int8Cfg<BT, MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = a.stages, kpb = a.kpb;
  constexpr int kRows = 128 * MT, a_bytes = kRows * 128, b_bytes = BT * 128;   // one k block
  const int stage_bytes = kpb * (a_bytes + b_bytes);
  const int ring_bytes = S * stage_bytes;
  float* s_sx = reinterpret_cast<float*>(smem + ring_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ring_bytes + C::kSxBytes);
  uint64_t* empty = full + kI8MaxStages;
  uint64_t* accfull = empty + kI8MaxStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accfull + 4;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + kI8Bars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  // (the shuffle tells the compiler that a warp's index is the same in all of its lanes)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int ks = a.ks;
  const int rank = ks > 1 ? static_cast<int>(blockIdx.x) % ks : 0;
  const int KB = (a.K + 127) / 128;
  const int kb0 = static_cast<int>(static_cast<long long>(rank) * KB / ks);
  const int kb1 = static_cast<int>(static_cast<long long>(rank + 1) * KB / ks);
  const int ntiles = a.row_blocks * a.tok_tiles;
  const int tile0 = static_cast<int>(blockIdx.x) / ks;
  const int step = ks > 1 ? ntiles : static_cast<int>(gridDim.x);
  // Tiles in groups of up to 16 token tiles, token tile fastest within a group: concurrent CTAs share
  // few weight blocks and a set of token tiles that stays in L2.
  auto tile_at = [&](int t, int& rb, int& tt) {
    const int per_group = 16 * a.row_blocks;
    const int g = t / per_group, i = t - g * per_group;
    const int width = min(16, a.tok_tiles - 16 * g);
    rb = i / width;
    tt = 16 * g + i - rb * width;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], C::kEpi);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_x);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem_base = *s_tmem;
  const unsigned long long budget = g_wait_budget_ns;

  const uint32_t base = smem_u32(smem), full0 = smem_u32(full);
  const uint32_t hint = brief_hint(budget);
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, mbar_wait_brief(bar, parity, hint, s_abort, budget));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    auto issue_w = [&](int slot, int row, int kb, int n) {
      if (!AWQ_CHECK(slot >= 0 && slot < S && n >= 1 && n <= kpb && row >= 0 && row < a.N && kb >= kb0 && kb + n <= kb1)) return;
      const uint32_t dst = base + slot * stage_bytes, bar = full0 + 8 * slot;
      mbar_expect_tx_at(bar, static_cast<uint32_t>(n * (a_bytes + b_bytes)));
      for (int j = 0; j < n; ++j) tma_load_2d_at(dst + j * a_bytes, &tmap_w, (kb + j) * 128, row, bar);
    };
    auto issue_x = [&](int slot, int row, int kb, int n) {
      if (!AWQ_CHECK(slot >= 0 && slot < S && n >= 1 && n <= kpb && row >= 0 && row < a.M && kb >= kb0 && kb + n <= kb1)) return;
      const uint32_t dst = base + slot * stage_bytes + kpb * a_bytes, bar = full0 + 8 * slot;
      for (int j = 0; j < n; ++j) tma_load_2d_at(dst + j * b_bytes, &tmap_x, (kb + j) * 128, row, bar);
    };
    int rb, tt;
    // first ring pass of the first tile's weights before the wait on the predecessor
    int pre = 0;
    if (tile0 < ntiles) {
      tile_at(tile0, rb, tt);
      for (int kb = kb0; kb < kb1 && pre < S; kb += kpb, ++pre)
        if (elect_one()) issue_w(pre, rb * kRows, kb, min(kpb, kb1 - kb));
    }
    __syncwarp();
    pdl_wait();
    int slot = 0, n_issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = tile0; ok && t < ntiles; t += step) {
      tile_at(t, rb, tt);
      for (int kb = kb0; kb < kb1; kb += kpb) {
        const int n = min(kpb, kb1 - kb);
        if (n_issued >= pre && !warp_wait(&empty[slot], phase ^ 1)) { ok = false; break; }
        if (elect_one()) {
          if (n_issued >= pre) issue_w(slot, rb * kRows, kb, n);
          issue_x(slot, tt * BT, kb, n);
        }
        __syncwarp();
        ++n_issued;
        if (++slot == S) { slot = 0; phase ^= 1; }
      }
    }
    // drain: every copy this warp issued has landed before the CTA may exit
    int never = 0;
    if (lane == 0)
      for (int i = max(0, n_issued - S); i < n_issued; ++i)
        mbar_wait_bounded(&full[i % S], static_cast<uint32_t>((i / S) & 1), &never, kDrainBudgetNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    pdl_wait();                                // its waits' budget starts with the tokens' copies
    constexpr uint32_t idesc = idesc_s8_s32(128, BT);
    const uint64_t desc_hi = smem_desc_sw128(0) & ~0xFFFFFFFFull;
    const uint32_t desc_lo = static_cast<uint32_t>(smem_desc_sw128(base));
    int slot = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true, any = false;
    for (int t = tile0; ok && t < ntiles; t += step, ++it) {
      const int b = it % C::kNAcc;
      ok = warp_wait(&accempty[b], ((it / C::kNAcc) & 1) ^ 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::kAcc);
      for (int kb = kb0; kb < kb1; kb += kpb) {
        ok = warp_wait(&full[slot], phase);
        if (!ok) break;
        tc_fence_after();
        const int n = min(kpb, kb1 - kb);
        // descriptors count in 16 bytes; shared memory ends well below the 2^18 that their field holds
        const uint32_t da = desc_lo + ((slot * stage_bytes) >> 4), db = da + ((kpb * a_bytes) >> 4);
        if (elect_one()) {
          for (int j = 0; j < n; ++j) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int m = 0; m < MT; ++m)
                tc_mma_i8(d + m * BT, desc_hi | (da + ((j * a_bytes + m * 16384 + 32 * kk) >> 4)),
                          desc_hi | (db + ((j * b_bytes + 32 * kk) >> 4)), idesc, (kb != kb0 || j != 0 || kk != 0) ? 1u : 0u);
          }
          tc_commit(&empty[slot]);
        }
        __syncwarp();
        any = true;
        if (++slot == S) { slot = 0; phase ^= 1; }
      }
      if (ok && elect_one()) tc_commit(&accfull[b]);
      __syncwarp();
    }
    if (any) {
      int never = 0;
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      if (lane == 0) mbar_wait_bounded(drain, 0, &never, kDrainBudgetNs);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    pdl_wait();
    const int e = warp & 3;                    // tensor-memory lane quarter of this warp
    const int cw = (warp - 2) >> 2;            // its part of the token columns
    constexpr int CH = C::kChunk;
    float* my_sx = s_sx + (warp - 2) * C::kCols;
    // channels in pairs: with an even N, the lanes of a pair trade values of two tokens, so that each
    // stores both channels of one token in four bytes
    const bool paired = (a.N & 1) == 0;
    // whether an output lies inside y (bounds-checked builds)
    auto inside = [&](long long n, int tok) { return AWQ_CHECK(n >= 0 && n < a.N && tok >= 0 && tok < a.M); };
    bool ok = true;
    int it = 0;
    for (int t = tile0; ok && t < ntiles; t += step, ++it) {
      int rb, tt;
      tile_at(t, rb, tt);
      const int tok0 = tt * BT + cw * C::kCols;
      if (ks == 1) {
        __syncwarp();
        for (int i = lane; i < C::kCols; i += 32) my_sx[i] = tok0 + i < a.M ? __ldg(a.sx + tok0 + i) : 0.0f;
        __syncwarp();
      }
      const int b = it % C::kNAcc;
      ok = warp_wait(&accfull[b], (it / C::kNAcc) & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int lr = m * 128 + 32 * e + lane;              // row within the tile
        const long long n = static_cast<long long>(rb) * kRows + lr;
        const bool n_ok = n < a.N;
        const float sw = ks == 1 && n_ok ? __ldg(a.sw + n) : 0.0f;
#pragma unroll 1
        for (int c0 = 0; c0 < C::kCols; c0 += CH) {
          if (ks == 1 && tok0 + c0 >= a.M) break;
          uint32_t v[CH];
          tmem_ld_cols(tmem_base + (static_cast<uint32_t>(32 * e) << 16) +
                           static_cast<uint32_t>(b * C::kAcc + m * BT + cw * C::kCols + c0), v);
          tc_wait_ld();
          if (ks > 1) {                                      // the ring is idle: partial sums take its place
            int* part = reinterpret_cast<int*>(smem) + (m * BT + cw * C::kCols + c0) * 128 + 32 * e + lane;
            if (AWQ_CHECK(static_cast<int>(reinterpret_cast<uint8_t*>(part + (CH - 1) * 128 + 1) - smem) <= ring_bytes)) {
#pragma unroll
              for (int j = 0; j < CH; ++j) part[j * 128] = static_cast<int>(v[j]);
            }
            continue;
          }
          __half o[CH];
#pragma unroll
          for (int j = 0; j < CH; j += 4) {
            const float4 s4 = *reinterpret_cast<const float4*>(my_sx + c0 + j);
            o[j] = i8_out(static_cast<int>(v[j]), s4.x, sw);
            o[j + 1] = i8_out(static_cast<int>(v[j + 1]), s4.y, sw);
            o[j + 2] = i8_out(static_cast<int>(v[j + 2]), s4.z, sw);
            o[j + 3] = i8_out(static_cast<int>(v[j + 3]), s4.w, sw);
          }
          if (paired) {
            const int odd = lane & 1;
            __half* p = a.y + static_cast<size_t>(tok0 + c0 + odd) * a.N + (n - odd);
            const int left = a.M - (tok0 + c0 + odd);
#pragma unroll
            for (int j = 0; j < CH; j += 2) {
              const uint32_t own = (static_cast<uint32_t>(__half_as_ushort(o[j + 1])) << 16) | __half_as_ushort(o[j]);
              const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
              // even lanes: token j of both channels; odd lanes: token j + 1
              const uint32_t w = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
              if (n_ok && j < left && inside(n + 1 - odd, tok0 + c0 + j + odd)) *reinterpret_cast<uint32_t*>(p) = w;
              p += 2 * static_cast<size_t>(a.N);
            }
          } else if (n_ok) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
              if (tok0 + c0 + j < a.M && inside(n, tok0 + c0 + j)) a.y[static_cast<size_t>(tok0 + c0 + j) * a.N + n] = o[j];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty[b]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmem);
  }
  if (ks > 1) {
    cluster_arrive();
    cluster_wait();                                          // every CTA's partial sums are in its shared memory
    if (*s_abort == 0 && tile0 < ntiles) {
      int rb, tt;
      tile_at(tile0, rb, tt);
      const int c_lo = rank * BT / ks, c_hi = min((rank + 1) * BT / ks, a.M - tt * BT);
      const uint32_t base = smem_u32(smem);
      constexpr int quads = kRows / 4;
      for (int i = threadIdx.x; i < (c_hi - c_lo) * quads; i += C::kThreads) {
        const int c = c_lo + i / quads, lr = i % quads * 4;   // four rows of one column
        const long long n = static_cast<long long>(rb) * kRows + lr;
        const uint32_t off = base + (((lr >> 7) * BT + c) * 128 + (lr & 127)) * 4;
        if (!AWQ_CHECK(c >= 0 && tt * BT + c < a.M && off - base + 16 <= static_cast<uint32_t>(ring_bytes))) continue;
        int4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (r >= ks) break;
          uint32_t addr;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(off), "r"(r));
          v[r] = ld_cluster_v4(addr);
        }
        int sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (r >= ks) break;
          sum[0] += v[r].x;
          sum[1] += v[r].y;
          sum[2] += v[r].z;
          sum[3] += v[r].w;
        }
        const int tok = tt * BT + c;
        const float sx = __ldg(a.sx + tok);
        __half* p = a.y + static_cast<size_t>(tok) * a.N + n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < a.N) p[j] = i8_out(sum[j], sx, __ldg(a.sw + n + j));
      }
    }
    cluster_arrive();
    cluster_wait();                                          // no CTA exits while another reads its partial sums
  }
}

}  // namespace awq
