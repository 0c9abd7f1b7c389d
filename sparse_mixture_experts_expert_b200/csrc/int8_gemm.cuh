// Grouped expert products in 8-bit integers on the 5th-generation tensor cores (tcgen05 kind::i8 + TMA), with one
// scale a token and one a channel:
//   out[rows of group g] = epilogue( A[rows of group g] . B_g^T ),   A [R, K] int8 codes, B_g int8 codes.
// The integer sums are exact (|code| <= 128, K <= 65536: below 2^31); the epilogue forms float(sum) s_row s_col.
//   gate/up (GLU): a tile holds the gate and the up slice of the same hidden columns side by side, and writes
//     h = act(g) u rounded once to bf16 (the layer's h has that type for every weight format; the rounding is a
//     tenth of the step of the 8-bit codes that h becomes next);
//   down (plain): writes y in bf16.
// ExpertMesh README (grouped routed-expert products of quantised weights in [expert, output, input] order).
//
// Structure as k_grouped_gemm: persistent CTAs, warp 0 feeds A and B tiles of 128 bytes of K by TMA into a ring,
// warp 1 issues tcgen05.mma (M = 128, or 256 over a CTA pair; four MMAs of K = 32 per stage), and the epilogue drains
// one accumulator while the next one fills.  A k-step holds twice the inputs of a bf16 one for the same bytes and the
// same MMA time, so a tile's main loop takes half as long and the epilogue weighs twice as much: sixteen epilogue warps
// (four per TMEM quarter, each on a quarter of the columns) instead of four, and rows stored straight from the
// registers in whole 32-byte sectors instead of through shared memory.
// Row tiles of at most 64 rows load them in boxes of 32, no more than the group has: with a handful of rows an expert
// (decode) the weights are then nearly all that moves.  Shared memory behind those rows holds whatever it held; integer
// products of it are finite and stay in rows that the epilogue does not store.  Fuller tiles take one box of 128 rows
// (four of 32 made the gate/up kernel of 16384 rows, 768 -> 4096, 168 us instead of 138: the copy engine's work goes
// by the box).
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
constexpr int kI8Threads = (4 + kI8EpiWarps) * 32;

template <int BN, int CG>
struct I8Cfg {
  static constexpr int kABytes = kBM * kI8BK;
  static constexpr int kBBytes = (CG == 2 ? BN / 2 : BN) * kI8BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBudget = 215 * 1024 - 1024;
  static constexpr int kStages = kBudget / kStageBytes > 8 ? 8 : kBudget / kStageBytes;
  static constexpr int kTmemCols = 2 * BN;      // two accumulators (128, 256 or 512 columns)
  static constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes;
};

// Instruction descriptor, kind::i8: D s32, A and B signed 8-bit, both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
  return (2u << 4)                       // D format: s32
         | (1u << 7)                     // A format: signed 8-bit
         | (1u << 10)                    // B format: signed 8-bit
         | ((uint32_t)(N >> 3) << 17)    // N / 8
         | ((uint32_t)(M >> 4) << 24);   // M / 16
}

template <int CG>
__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

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
// act(g) with few instructions.  SiLU: g / (1 + exp(-g)).  GELU: g Phi(g) = max(g, 0) - |g| Q(|g|) with the normal
// tail Q(a) = erfc(a / sqrt 2) / 2 by Abramowitz & Stegun 7.1.26 (the factor 1/2 and the sqrt 2 folded into its
// coefficients); the tail form does not cancel for negative g.
template <int MODE>
__device__ __forceinline__ float i8_act(float g) {
  if (MODE == kModeSwiGLU) return g * rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * g));
  const float a = fabsf(g);
  const float t = rcp_approx(fmaf(0.3275911f * 0.7071067811865476f, a, 1.0f));
  const float poly = t * (0.5f * 0.254829592f +
                          t * (-0.5f * 0.284496736f +
                               t * (0.5f * 1.421413741f + t * (-0.5f * 1.453152027f + t * (0.5f * 1.061405429f)))));
  const float e = ex2_approx(-0.7213475204444817f * (g * g));
  return fmaf(-a, poly * e, fmaxf(g, 0.0f));
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
                const __grid_constant__ CUtensorMap tmB, const I8Params p) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
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
  __shared__ __align__(16) float s_scale[4 * PARTS][kGLU ? 2 * CW : CW];

  const int warp = warp_id(), lane = lane_id();
  const int crank = kPair ? (int)cluster_ctarank() : 0;   // 0 = leader of the pair
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int n_units = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int n_tiles = (p.N + OUTN - 1) / OUTN;
  const int nk = (p.K + kI8BK - 1) / kI8BK;
  const int G = p.group_rows == nullptr ? 1 : p.n_groups;

  if (warp == 2) i8_group_table(p, TM, s_prefix, s_gstart, s_grows);
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&bar_full[s], 1); mbar_init(&bar_empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&bar_tfull[a], 1); mbar_init(&bar_tempty[a], CG * 4 * PARTS); }
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

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    if (lane == 0) {
      for (long long tile = unit; tile < total && !s_abort; tile += n_units) {
        int g, row0, rows_left, n0;
        locate(tile, g, row0, rows_left, n0);
        const int na = loaded(rows_left - crank * kBM);
        const int na_all = kPair ? loaded(rows_left) + loaded(rows_left - kBM) : na;
        const uint32_t bytes = (uint32_t)(na_all * kI8BK + CG * Cfg::kBBytes);
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb) {
          uint8_t* a_s = smem + (size_t)stage * Cfg::kStageBytes;
          uint8_t* b_s = a_s + Cfg::kABytes;
          ok = mbar_wait(&bar_empty[stage], phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0501);
          if (!ok) break;
          // the leader's barrier counts the bytes of both CTAs of a pair
          if (crank == 0) mbar_arrive_expect_tx(&bar_full[stage], bytes);
          if (kPair) {
            const uint32_t fb = mapa_shared(smem_u32(&bar_full[stage]), 0);
            if (na == kBM) tma_load_2d_pair(a_s, &tmA, fb, kb * kI8BK, row0);
            else
              for (int i = 0; i < na; i += kI8ABox)
                tma_load_2d_pair(a_s + i * kI8BK, &tmAFew, fb, kb * kI8BK, row0 + i);
            const int brow = kGLU ? (crank == 0 ? n0 : p.up_row0 + n0) : n0 + crank * (BN / 2);
            tma_load_3d_pair(b_s, &tmB, fb, kb * kI8BK, brow, g);
          } else {
            if (na == kBM) tma_load_2d(a_s, &tmA, &bar_full[stage], kb * kI8BK, row0);
            else
              for (int i = 0; i < na; i += kI8ABox)
                tma_load_2d(a_s + i * kI8BK, &tmAFew, &bar_full[stage], kb * kI8BK, row0 + i);
            tma_load_3d(b_s, &tmB, &bar_full[stage], kb * kI8BK, n0, g);
            if (kGLU)
              tma_load_3d(b_s + (BN / 2) * kI8BK, &tmB, &bar_full[stage], kb * kI8BK, p.up_row0 + n0, g);
          }
          ++issued;
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
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
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0 && crank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      for (long long tile = unit; tile < total && !s_abort; tile += n_units) {
        if (!mbar_wait(&bar_tempty[acc], acc_phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0503)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&bar_full[stage], phase, p.wait_limit_ns, &s_abort, 0x0504)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + (size_t)stage * Cfg::kStageBytes);
          const uint32_t b_addr = a_addr + Cfg::kABytes;
#pragma unroll
          for (int kk = 0; kk < kI8BK / 32; ++kk)
            tc_mma_i8<CG>(d_tmem, smem_desc_k128(a_addr + kk * 32), smem_desc_k128(b_addr + kk * 32), IDESC,
                          (kb > 0 || kk > 0) ? 1u : 0u);
          if (kPair) tc_commit_pair_mc(&bar_empty[stage], 0x3);
          else tc_commit(&bar_empty[stage]);
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (kPair) tc_commit_pair_mc(&bar_tfull[acc], 0x3);
        else tc_commit(&bar_tfull[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      // all issued MMAs complete before TMEM is released
      if (kPair) tc_commit_pair(&bar_final);
      else tc_commit(&bar_final);
      volatile int dummy = 0;
      mbar_wait(&bar_final, 0, p.wait_limit_ns, &dummy, 0x0505);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + 4 * PARTS) {
    // ------------------------------------------------ epilogue
    const int ew = warp - 4;
    const int q = warp & 3;                 // TMEM lane quarter: this warp's 32 accumulator rows
    const int c_base = (ew >> 2) * CW;      // this warp's first output column in the tile
    float* scl = s_scale[ew];
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (long long tile = unit; tile < total && !s_abort; tile += n_units) {
      int g, row0, rows_left, n0;
      locate(tile, g, row0, rows_left, n0);
      const int row = q * 32 + lane;
      const bool live = row < rows_left - crank * kBM;
      // this warp's channel scales (gate, then up) and this lane's token scale, while the MMAs run
      {
        const float* bs = p.b_scale + (size_t)g * p.b_rows;
        for (int c = lane; c < CW; c += 32) {
          const int col = n0 + c_base + c;
          scl[c] = col < p.N ? bs[col] : 0.f;
          if (kGLU) scl[CW + c] = col < p.N ? bs[p.up_row0 + col] : 0.f;
        }
      }
      const float sx = live ? p.a_scale[(long long)row0 + row] : 0.f;
      __nv_bfloat16* out = p.out + ((long long)row0 + row) * p.N + n0 + c_base;
      const int cols = p.N - n0 - c_base;   // N is a multiple of 16: whole chunks
      __syncwarp();
      if (!mbar_wait(&bar_tfull[acc], acc_phase, p.wait_limit_ns, &s_abort, 0x0506)) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + c_base);
#pragma unroll
      for (int c0 = 0; c0 < CW; c0 += 16) {
        uint32_t v[16];
        uint32_t u[kGLU ? 16 : 1];
        tmem_ld16(t_row + c0, v);
        if constexpr (kGLU) tmem_ld16(t_row + OUTN + c0, u);
        tmem_ld_wait();
        if (c0 + 16 == CW) {   // the accumulator is drained: one arrival per epilogue warp (on the leader)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kPair) mbar_arrive_cluster(mapa_shared(smem_u32(&bar_tempty[acc]), 0));
            else mbar_arrive(&bar_tempty[acc]);
          }
        }
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 sg = *reinterpret_cast<const float4*>(scl + c0 + i);
          const float gs[4] = {sg.x, sg.y, sg.z, sg.w};
          float f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = (float)(int)v[i + j] * sx * gs[j];
          if constexpr (kGLU) {
            const float4 su = *reinterpret_cast<const float4*>(scl + CW + c0 + i);
            const float us[4] = {su.x, su.y, su.z, su.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = i8_act<MODE>(f[j]) * ((float)(int)u[i + j] * sx * us[j]);
          }
          o[i / 2] = pack_bf16x2(f[0], f[1]);
          o[i / 2 + 1] = pack_bf16x2(f[2], f[3]);
        }
        if (live && c0 < cols) st_row16(out + c0, o, wide);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
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
// read.  A row per TPR threads, the filled rows dealt over a fixed grid.
template <int TPR>
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
    const float s = quant_row<TPR>(x + r * K, K, on, s_max, [&](int c, uint2 v) {
      reinterpret_cast<uint2*>(q + r * K)[c] = v;
    });
    if (on && (int)threadIdx.x % TPR == 0) scale[r] = s;
  }
}

}  // namespace moe
