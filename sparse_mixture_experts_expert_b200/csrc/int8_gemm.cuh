// Grouped expert products in 8-bit integers on the 5th-generation tensor cores (tcgen05 kind::i8 + TMA), with one
// scale a token and one a channel:
//   out[rows of group g] = epilogue( A[rows of group g] . B_g^T ),   A [R, K] int8 codes, B_g int8 codes.
// The integer sums are exact (|code| <= 128, K <= 65536: below 2^31); the epilogue forms float(sum) s_row s_col.
//   gate/up (GLU): a tile holds the gate and the up slice of the same hidden columns side by side, and writes
//     h = act(g) u rounded once to bf16 (the layer's h has that type for every weight format, and it halves what the
//     two kernels around h move; the rounding is at most half a step of the 8-bit codes that h becomes next, for the
//     row's largest elements, and 2^-8 of the value for the others);
//   down (plain): writes y in bf16.
// ExpertMesh README (grouped routed-expert products of quantised weights in [expert, output, input] order).
//
// Structure as k_grouped_gemm: persistent CTAs; warps 0 and 2 feed A and B tiles of 128 bytes of K by TMA into a ring,
// warp 3 the channel scales; warp 1 issues tcgen05.mma (M = 128, or 256 over a CTA pair; four MMAs of K = 32 per
// stage); the epilogue drains one accumulator while the next one fills.  A k-step holds twice the inputs of a bf16 one
// for the same bytes and the same MMA time, so a tile's main loop takes half as long and the epilogue weighs twice as
// much: sixteen epilogue warps (four per TMEM quarter, each on a quarter of the columns) instead of four, arithmetic
// in packed fp32 pairs, and no access to global memory between a tile's MMAs and its stores.  Pair tiles store by TMA,
// others straight from the registers in whole 32-byte sectors.
// Measured (B200): one dense group of 8192 rows, 7168 -> 2 x 4096: 263 us, 3660 TOP/s.  16384 rows over 32 experts,
// GeGLU 768 -> 4096: gate/up 116 us (1780 TOP/s; 113 us with a tail formula two terms shorter), down 54 us (1890 TOP/s);
// on another GPU at 1.58 GHz 125 and 57 us, tensor pipe 50 and 54% busy, DRAM 31 and 39%.  There the groups cost the
// rest: a third of the 256-row tiles is nearly empty, and 300 MB of weights come from HBM (one dense group of that
// shape: 87 and 40 us).  Keeping the A tile in shared memory for four column tiles (half the operand bytes) left the
// gate/up kernel at 121 us against 118.
// 64 rows over 48 experts of 7168 x 2048: 159 and 85 us, the weights at 6.4 TB/s.
// Row tiles of at most 64 rows load them in boxes of 32, no more than the group has: with a handful of rows an expert
// (decode) the weights are then nearly all that moves.  Shared memory behind those rows holds whatever it held; integer
// products of it are finite and stay in rows that the epilogue does not store.  Fuller tiles take one box of 128 rows
// (four of 32 made the gate/up kernel above 30 us longer: the copy engine's work goes by the box).
#pragma once

#include "gemm_tc.cuh"
#include "int8_quant.cuh"

namespace moe {

struct I8Params {
  const int32_t* group_start;   // [n_groups] or nullptr (one group of R rows)
  const int32_t* group_rows;
  int n_groups;
  long long R;
  int K;                        // reduction length = bytes of a row
  int N;                        // output columns
  int up_row0;                  // GLU: first up row of B (= H)
  int b_rows;                   // rows of B per group (scales per group)
  const float* a_scale;         // [R]
  const float* b_scale;         // [n_groups, b_rows]
  __nv_bfloat16* out;           // [R, N]
  unsigned long long wait_limit_ns;
};

constexpr int kI8BK = 128;                      // codes per k-step: one 128-byte swizzle row
constexpr int kI8ABox = 32;                     // rows per A box of a tile of at most kI8Few rows, else kBM
constexpr int kI8Few = 64;
constexpr int kI8EpiWarps = 16;
constexpr int kI8ScaleBufs = 8;                 // tiles (or jobs) whose channel scales are in flight
constexpr int kI8Threads = (4 + kI8EpiWarps) * 32;

template <int BN, int CG>
struct I8Cfg {
  static constexpr int kABytes = kBM * kI8BK;
  static constexpr int kBBytes = (CG == 2 ? BN / 2 : BN) * kI8BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kOutBytes = CG == 2 ? kI8EpiWarps * 32 * 64 : 0;   // output staging: 2 KB per epilogue warp
  static constexpr int kBudget = 211 * 1024 - 1024 - kOutBytes;
  static constexpr int kStages = kBudget / kStageBytes > 8 ? 8 : kBudget / kStageBytes;
  static constexpr int kTmemCols = 2 * BN;      // two accumulators (128, 256 or 512 columns)
  static constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + kOutBytes;
};

// Instruction descriptor, kind::i8: D s32, A and B signed 8-bit, both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
  return (2u << 4)                       // D format: s32
         | (1u << 7)                     // A format: signed 8-bit
         | (1u << 10)                    // B format: signed 8-bit
         | ((uint32_t)(N >> 3) << 17)    // N / 8
         | ((uint32_t)(M >> 4) << 24);   // M / 16
}

// D[tmem] (+)= A[smem] * B[smem]^T by the lane with `lead` set.  The whole warp runs the code around it: descriptors
// and loop counters then stay in uniform registers, where tcgen05.mma takes them, which a branch on the lane prevents.
template <int CG>
__device__ __forceinline__ void tc_mma_i8(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}

// Arrive on the mbarrier (of both CTAs of a pair) when the lead lane's MMAs so far complete.
template <int CG>
__device__ __forceinline__ void tc_commit_i8(uint32_t lead, uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)0x3), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}

// mbar_wait by the whole warp; the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort,
                                               unsigned int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns, abort, site)) != 0;
}

// Warp index in a uniform register.
__device__ __forceinline__ int warp_id_uniform() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// One k-step: four MMAs of K = 32 over the 128-byte rows at the two shared addresses (1024-byte aligned).
template <int CG>
__device__ __forceinline__ void i8_mma_step(uint32_t lead, uint32_t d_tmem, uint32_t a_addr, uint32_t b_addr, uint32_t idesc,
                                            bool first) {
  const uint64_t a = smem_desc_k128(a_addr), b = smem_desc_k128(b_addr);   // + 2: 32 bytes on
  tc_mma_i8<CG>(lead, d_tmem, a, b, idesc, first ? 0u : 1u);
#pragma unroll
  for (int kk = 1; kk < kI8BK / 32; ++kk) tc_mma_i8<CG>(lead, d_tmem, a + 2 * kk, b + 2 * kk, idesc, 1u);
}

// Position in a ring of S stages: index, phase parity.
template <int S>
struct RingPos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == S) { stage = 0; phase ^= 1u; }
  }
};

// 16 bf16 values of a row: one 32-byte sector per lane in one store where the output lies on 32-byte boundaries
// (`wide`, the same for the whole output: its rows are multiples of 32 bytes), else two of 16 bytes.
__device__ __forceinline__ void st_row16(void* p, const uint32_t (&o)[8], bool wide) {
  if (!wide) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
               "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two columns of an accumulator, scaled: float(sum) * s_row * s_col.
__device__ __forceinline__ float2 i8_scaled(uint32_t v0, uint32_t v1, float row, float c0, float c1) {
  const float2 f = make_float2((float)(int)v0, (float)(int)v1);
  return __fmul2_rn(__fmul2_rn(f, make_float2(row, row)), make_float2(c0, c1));
}

// act(g) u of two columns, in packed fp32 pairs.  SiLU: g / (1 + exp(-g)).  GELU: g Phi(g) = max(g, 0) - |g| Q(|g|)
// with the normal tail Q; that form does not cancel for negative g.  Q(a) = exp(-a^2 / 2) t P(t), t = 1 / (1 + c a): P
// has degree 6 and c = 0.26374, fitted so that the largest relative error over 0 <= a <= 13.3 is least (5.2e-7 before,
// 1e-6 after the fp32 arithmetic; beyond, exp underflows).  The error is relative because a row whose gates all lie in
// the tail is lifted back to full size by its scale.  (Two terms fewer leave 2.7e-5.)
template <int MODE>
__device__ __forceinline__ float2 i8_glu2(float2 g, float2 u) {
  auto both = [](float c) { return make_float2(c, c); };
  if (MODE == kModeSwiGLU) {
    const float2 x = __fmul2_rn(g, both(-1.4426950408889634f));
    const float2 d = __fadd2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), both(1.0f));
    return __fmul2_rn(__fmul2_rn(g, make_float2(rcp_approx(d.x), rcp_approx(d.y))), u);
  }
  const float2 a = make_float2(fabsf(g.x), fabsf(g.y));
  const float2 d = __ffma2_rn(both(0.26374f), a, both(1.0f));
  const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  float2 poly = __ffma2_rn(t, both(-0.0696539249f), both(0.205525397f));
  poly = __ffma2_rn(t, poly, both(-0.078861467f));
  poly = __ffma2_rn(t, poly, both(0.150310451f));
  poly = __ffma2_rn(t, poly, both(0.0797937966f));
  poly = __ffma2_rn(t, poly, both(0.107823258f));
  poly = __ffma2_rn(t, poly, both(0.105062232f));
  const float2 x = __fmul2_rn(__fmul2_rn(g, g), both(-0.7213475204444817f));
  const float2 q = __fmul2_rn(__fmul2_rn(t, poly), make_float2(ex2_approx(x.x), ex2_approx(x.y)));
  return __fmul2_rn(__ffma2_rn(make_float2(-a.x, -a.y), q, make_float2(fmaxf(g.x, 0.f), fmaxf(g.y, 0.f))), u);
}

// Wait for the scale copies still in flight (the last kI8ScaleBufs of n): none may land after the CTA has ended.
__device__ __forceinline__ void i8_drain_scales(uint64_t* bar_sfull, long long n, uint64_t limit_ns, unsigned int site) {
  for (int i = 1; i <= kI8ScaleBufs && i <= n; ++i) {
    volatile int dummy = 0;
    mbar_wait(&bar_sfull[(int)((n - i) % kI8ScaleBufs)], (uint32_t)(((n - i) / kI8ScaleBufs) & 1), limit_ns, &dummy,
              site);
  }
}

// First row and number of rows of group g, kept inside [0, R).
__device__ __forceinline__ void i8_group(const I8Params& p, int g, int& start, int& rows) {
  if (p.group_rows == nullptr) {
    start = 0;
    rows = (int)p.R;
    return;
  }
  const int s = p.group_start[g];
  start = s;
  rows = (s < 0 || s >= p.R) ? 0 : (int)max(0ll, min((long long)p.group_rows[g], p.R - s));
}

// Row-tile table of the groups by one warp: prefix[g] = row tiles of TM rows before group g.
__device__ __forceinline__ void i8_group_table(const I8Params& p, int TM, int* prefix, int* gstart, int* grows) {
  const int G = p.group_rows == nullptr ? 1 : p.n_groups;
  const int lane = lane_id();
  const int per = (G + 31) / 32;
  const int g0 = min(G, lane * per), g1 = min(G, g0 + per);
  int local = 0;
  for (int g = g0; g < g1; ++g) {
    int s, r;
    i8_group(p, g, s, r);
    gstart[g] = s;
    grows[g] = r;
    local += (r + TM - 1) / TM;
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - local;
  for (int g = g0; g < g1; ++g) {
    prefix[g] = run;
    run += (grows[g] + TM - 1) / TM;
  }
  if (lane == 31) prefix[G] = incl;
}

// Last g with prefix[g] <= mt.
__device__ __forceinline__ int i8_find_group(const int* prefix, int G, int mt) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= mt) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int MODE, int BN, int CG>
__global__ void __launch_bounds__(kI8Threads, 1)
    k_int8_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmAFew,
                const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmOut, const I8Params p) {
  using Cfg = I8Cfg<BN, CG>;
  constexpr bool kGLU = MODE == kModeSwiGLU || MODE == kModeGeGLU;
  constexpr bool kPair = CG == 2;
  constexpr int OUTN = kGLU ? BN / 2 : BN;   // output columns per tile
  constexpr int TM = kBM * CG;               // rows per tile
  constexpr int S = Cfg::kStages;
  constexpr uint32_t IDESC = idesc_i8_s32(TM, BN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar_full[S], bar_empty[S], bar_tfull[2], bar_tempty[2], bar_final;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_prefix[kMaxGroupsSmem + 1];
  __shared__ int s_gstart[kMaxGroupsSmem];
  __shared__ int s_grows[kMaxGroupsSmem];
  constexpr int PARTS = OUTN >= 64 ? 4 : OUTN / 16;   // epilogue warps per TMEM quarter that have columns
  constexpr int CW = OUTN / PARTS;                    // output columns of such a warp, in chunks of 16
  // channel scales of the tiles in flight (gate, then up): copied in by the producer ahead of a tile's operands, so
  // that the epilogue never waits for global memory
  __shared__ __align__(16) float s_scale[kI8ScaleBufs][BN];
  __shared__ __align__(8) uint64_t bar_sfull[kI8ScaleBufs], bar_sempty[kI8ScaleBufs];

  const int warp = warp_id_uniform(), lane = lane_id();
  const int crank = kPair ? (int)cluster_ctarank() : 0;   // 0 = leader of the pair
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int n_units = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int n_tiles = (p.N + OUTN - 1) / OUTN;
  const int nk = (p.K + kI8BK - 1) / kI8BK;
  const int G = p.group_rows == nullptr ? 1 : p.n_groups;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&bar_full[s], 1); mbar_init(&bar_empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&bar_tfull[a], 1); mbar_init(&bar_tempty[a], CG * 4 * PARTS); }
    for (int b = 0; b < kI8ScaleBufs; ++b) { mbar_init(&bar_sfull[b], 1); mbar_init(&bar_sempty[b], 4 * PARTS); }
    mbar_init(&bar_final, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmAFew);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&s_tmem, Cfg::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&s_tmem, Cfg::kTmemCols);
      tmem_relinquish();
    }
  }
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  if (warp == 3) i8_group_table(p, TM, s_prefix, s_gstart, s_grows);
  tc_fence_before();
  if (kPair) cluster_sync_all();  // both CTAs' barriers initialised before any cross-CTA arrival
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;
  const long long total = (long long)s_prefix[G] * n_tiles;

  // group, this CTA's first row, rows left in the group from the tile's first row, first output column
  auto locate = [&](long long tile, int& g, int& row0, int& rows_left, int& n0) {
    const int mt = (int)(tile / n_tiles);
    n0 = (int)(tile - (long long)mt * n_tiles) * OUTN;
    g = i8_find_group(s_prefix, G, mt);
    const int m_tile = (mt - s_prefix[g]) * TM;
    row0 = s_gstart[g] + m_tile + crank * kBM;
    rows_left = s_grows[g] - m_tile;
  };
  // rows that a CTA with `rows` rows of its tile left loads
  auto loaded = [](int rows) {
    return rows <= 0 ? 0 : rows > kI8Few ? kBM : (rows + kI8ABox - 1) / kI8ABox * kI8ABox;
  };

  // The copies are dealt to three warps (A and the byte counts, B, channel scales): one thread's chain of waits and
  // copies, in an SM whose issue slots the epilogue fills, took longer per k-step than the MMAs.
  if (warp == 0) {
    // ------------------------------------------------ A tiles
    if (lane == 0) {
      RingPos<S> r;
      long long issued = 0;
      bool ok = true;
      const uint32_t fb0 = kPair ? mapa_shared(smem_u32(&bar_full[0]), 0) : 0;
      for (long long tile = unit; tile < total && ok && !s_abort; tile += n_units) {
        int g, row0, rows_left, n0;
        locate(tile, g, row0, rows_left, n0);
        const int na = loaded(rows_left - crank * kBM);
        const int na_all = kPair ? loaded(rows_left) + loaded(rows_left - kBM) : na;
        const uint32_t bytes = (uint32_t)(na_all * kI8BK + CG * Cfg::kBBytes);
        for (int k0 = 0; k0 < p.K; k0 += kI8BK) {
          uint8_t* a_s = smem + (size_t)r.stage * Cfg::kStageBytes;
          if (!(ok = mbar_wait(&bar_empty[r.stage], r.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0501))) break;
          // the leader's barrier counts the bytes of both CTAs of a pair
          if (crank == 0) mbar_arrive_expect_tx(&bar_full[r.stage], bytes);
          if (na == kBM) {
            if (kPair) tma_load_2d_pair(a_s, &tmA, fb0 + 8 * r.stage, k0, row0);
            else tma_load_2d(a_s, &tmA, &bar_full[r.stage], k0, row0);
          } else {
            for (int i = 0; i < na; i += kI8ABox) {
              if (kPair) tma_load_2d_pair(a_s + i * kI8BK, &tmAFew, fb0 + 8 * r.stage, k0, row0 + i);
              else tma_load_2d(a_s + i * kI8BK, &tmAFew, &bar_full[r.stage], k0, row0 + i);
            }
          }
          ++issued;
          r.next();
        }
      }
      // No copy may still be landing in shared memory when the CTA ends (in a pair the leader's barriers count
      // both CTAs' copies; the pair leaves together).
      if (crank == 0) {
        const int last = (int)(issued < S ? issued : (long long)S);
        for (int i = 1; i <= last; ++i) {
          const long long n = issued - i;
          volatile int dummy = 0;
          mbar_wait(&bar_full[(int)(n % S)], (uint32_t)((n / S) & 1), p.wait_limit_ns, &dummy, 0x0502);
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------ B tiles
    if (lane == 0) {
      RingPos<S> r;
      bool ok = true;
      const uint32_t fb0 = kPair ? mapa_shared(smem_u32(&bar_full[0]), 0) : 0;
      for (long long tile = unit; tile < total && ok && !s_abort; tile += n_units) {
        int g, row0, rows_left, n0;
        locate(tile, g, row0, rows_left, n0);
        const int brow = !kPair ? n0 : kGLU ? (crank == 0 ? n0 : p.up_row0 + n0) : n0 + crank * (BN / 2);
        for (int k0 = 0; k0 < p.K; k0 += kI8BK) {
          uint8_t* b_s = smem + (size_t)r.stage * Cfg::kStageBytes + Cfg::kABytes;
          if (!(ok = mbar_wait(&bar_empty[r.stage], r.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x050A))) break;
          if (kPair) {
            tma_load_3d_pair(b_s, &tmB, fb0 + 8 * r.stage, k0, brow, g);
          } else {
            tma_load_3d(b_s, &tmB, &bar_full[r.stage], k0, brow, g);
            if (kGLU)
              tma_load_3d(b_s + (BN / 2) * kI8BK, &tmB, &bar_full[r.stage], k0, p.up_row0 + n0, g);
          }
          r.next();
        }
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------ channel scales
    if (lane == 0) {
      RingPos<kI8ScaleBufs> r;
      long long issued = 0;
      for (long long tile = unit; tile < total && !s_abort; tile += n_units) {
        int g, row0, rows_left, n0;
        locate(tile, g, row0, rows_left, n0);
        if (!mbar_wait(&bar_sempty[r.stage], r.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0507)) break;
        const uint32_t n = (uint32_t)min(OUTN, p.N - n0) * 4;   // a multiple of 64 bytes
        const float* src = p.b_scale + (size_t)g * p.b_rows + n0;
        mbar_arrive_expect_tx(&bar_sfull[r.stage], kGLU ? 2 * n : n);
        bulk_load(&s_scale[r.stage][0], src, n, &bar_sfull[r.stage]);
        if (kGLU) bulk_load(&s_scale[r.stage][OUTN], src + p.up_row0, n, &bar_sfull[r.stage]);
        ++issued;
        r.next();
      }
      i8_drain_scales(bar_sfull, issued, p.wait_limit_ns, 0x0508);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (crank == 0) {
      RingPos<S> r;
      RingPos<2> acc;
      bool ok = true;
      const uint32_t lead = lane == 0, base = smem_u32(smem);
      for (long long tile = unit; tile < total && ok; tile += n_units) {
        if (!mbar_wait_warp(&bar_tempty[acc.stage], acc.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0503)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc.stage * BN);
        for (int kb = 0; kb < nk; ++kb) {
          if (!(ok = mbar_wait_warp(&bar_full[r.stage], r.phase, p.wait_limit_ns, &s_abort, 0x0504))) break;
          tc_fence_after();
          const uint32_t a_addr = base + (uint32_t)(r.stage * Cfg::kStageBytes);
          i8_mma_step<CG>(lead, d_tmem, a_addr, a_addr + Cfg::kABytes, IDESC, kb == 0);
          tc_commit_i8<CG>(lead, &bar_empty[r.stage]);
          r.next();
        }
        if (!ok) break;
        tc_commit_i8<CG>(lead, &bar_tfull[acc.stage]);
        acc.next();
      }
      // all issued MMAs complete before TMEM is released
      if (lane == 0) {
        if (kPair) tc_commit_pair(&bar_final);
        else tc_commit(&bar_final);
        volatile int dummy = 0;
        mbar_wait(&bar_final, 0, p.wait_limit_ns, &dummy, 0x0505);
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + 4 * PARTS) {
    // ------------------------------------------------ epilogue
    const int ew = warp - 4;
    const int q = warp & 3;                 // TMEM lane quarter: this warp's 32 accumulator rows
    const int c_base = (ew >> 2) * CW;      // this warp's first output column in the tile
    const int row = q * 32 + lane;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    long long n_tile = 0;
    int g, row0 = 0, rows_left = 0, n0 = 0;
    float sx = 0.f;                         // this lane's token scale, loaded a tile ahead
    auto fetch = [&](long long tile) {
      if (tile >= total) return;
      locate(tile, g, row0, rows_left, n0);
      sx = row < rows_left - crank * kBM ? p.a_scale[(long long)row0 + row] : 0.f;
    };
    fetch(unit);
    uint8_t* stg = smem + (size_t)S * Cfg::kStageBytes + (kPair ? ew * (32 * 64) : 0);
    for (long long tile = unit; tile < total && !s_abort; tile += n_units, ++n_tile) {
      const int nv = max(0, min(32, rows_left - crank * kBM - q * 32));   // rows of this warp
      const float sxc = sx;
      const long long o_row0 = (long long)row0 + q * 32;
      const int o_col0 = n0 + c_base;
      const int cols = p.N - o_col0;        // N is a multiple of 16: whole chunks
      fetch(tile + n_units);
      const int sb = (int)(n_tile % kI8ScaleBufs);
      if (!mbar_wait(&bar_sfull[sb], (uint32_t)((n_tile / kI8ScaleBufs) & 1), p.wait_limit_ns, &s_abort, 0x0509)) break;
      const float* scl = &s_scale[sb][c_base];
      if (!mbar_wait(&bar_tfull[acc], acc_phase, p.wait_limit_ns, &s_abort, 0x0506)) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + c_base);
      const bool some = nv > 0 && cols > 0;
      // A warp whose 32 rows all belong to the group sends them out by TMA, 32 columns at a time, through 2 KB of shared
      // memory (row = lane, 16-byte chunk c at c ^ ((lane >> 1) & 3)); else its lanes store their rows themselves.
      const bool by_tma = kPair && nv == 32;
      // chunks of 16 columns; the next chunk's loads are in flight while one is worked on
      uint32_t v[2][16], u[2][kGLU ? 16 : 1];
      if (some) {
        tmem_ld16(t_row, v[0]);
        if constexpr (kGLU) tmem_ld16(t_row + OUTN, u[0]);
      }
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += 16) {
        const int b = (c0 / 16) & 1;
        if (some) tmem_ld_wait();
        if (c0 + 16 < CW) {
          if (some) {
            tmem_ld16(t_row + c0 + 16, v[b ^ 1]);
            if constexpr (kGLU) tmem_ld16(t_row + OUTN + c0 + 16, u[b ^ 1]);
          }
        } else {   // the accumulator is drained: one arrival per epilogue warp (on the leader)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kPair) mbar_arrive_cluster(mapa_shared(smem_u32(&bar_tempty[acc]), 0));
            else mbar_arrive(&bar_tempty[acc]);
          }
        }
        if (!some) continue;
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 sg = *reinterpret_cast<const float4*>(scl + c0 + i);
          float2 f0 = i8_scaled(v[b][i], v[b][i + 1], sxc, sg.x, sg.y);
          float2 f1 = i8_scaled(v[b][i + 2], v[b][i + 3], sxc, sg.z, sg.w);
          if constexpr (kGLU) {
            const float4 su = *reinterpret_cast<const float4*>(scl + OUTN + c0 + i);
            f0 = i8_glu2<MODE>(f0, i8_scaled(u[b][i], u[b][i + 1], sxc, su.x, su.y));
            f1 = i8_glu2<MODE>(f1, i8_scaled(u[b][i + 2], u[b][i + 3], sxc, su.z, su.w));
          }
          o[i / 2] = pack_bf16x2(f0.x, f0.y);
          o[i / 2 + 1] = pack_bf16x2(f1.x, f1.y);
        }
        if (by_tma) {
          if (c0 % 32 == 0) {
            if (lane == 0) bulk_wait_read();   // the last store has left the staging rows
            __syncwarp();
          }
          uint4* r = reinterpret_cast<uint4*>(stg + lane * 64);
          const uint32_t c = (c0 / 8) & 3, x = (uint32_t)(lane >> 1) & 3u;
          r[c ^ x] = make_uint4(o[0], o[1], o[2], o[3]);
          r[(c + 1) ^ x] = make_uint4(o[4], o[5], o[6], o[7]);
          if (c0 % 32 == 16) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmOut, stg, o_col0 + c0 - 16, (int)o_row0);
              bulk_commit();
            }
          }
        } else if (lane < nv && c0 < cols) {
          st_row16(p.out + (o_row0 + lane) * p.N + o_col0 + c0, o, wide);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_sempty[sb]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (kPair && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  if (kPair) cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (kPair) tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

// Codes and scales of the rows that the groups hold (h between the two products); rows outside every group are not
// read.  A row per TPR threads, the filled rows dealt over a fixed grid.  Bound by HBM: 16384 rows of 4096 in 31 to 38
// us (201 MB).
template <int TPR, int NV>
__global__ void __launch_bounds__(256) k_quant_groups(const __nv_bfloat16* __restrict__ x, const I8Params p,
                                                      int8_t* __restrict__ q, float* __restrict__ scale) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  __shared__ int s_prefix[kMaxGroupsSmem + 1];
  __shared__ int s_gstart[kMaxGroupsSmem];
  __shared__ int s_grows[kMaxGroupsSmem];
  __shared__ uint32_t s_max[8];
  if (warp_id() == 0) i8_group_table(p, 1, s_prefix, s_gstart, s_grows);
  __syncthreads();
  const int K = p.K;
  const int total = s_prefix[p.n_groups];
  constexpr int RPC = 256 / TPR;   // rows per CTA and step
  const int sub = (int)threadIdx.x / TPR;
  for (long long i0 = (long long)blockIdx.x * RPC; i0 < total; i0 += (long long)gridDim.x * RPC) {
    const bool on = i0 + sub < total;
    const int i = (int)(on ? i0 + sub : i0);
    const int g = i8_find_group(s_prefix, p.n_groups, i);
    const size_t r = (size_t)(s_gstart[g] + i - s_prefix[g]);
    const float s = quant_row<TPR, NV>(x + r * K, K, on, s_max, [&](int c, uint2 v) {
      reinterpret_cast<uint2*>(q + r * K)[c] = v;
    });
    if (on && (int)threadIdx.x % TPR == 0) scale[r] = s;
  }
}

}  // namespace moe
