// Both 8-bit products of narrow experts (hidden H = 128 or 256) in one kernel: per row tile of one expert
//   gate/up  z = (x W13^T) s_x s_13,  h = bf16(act(g) u)         jobs of 128 hidden columns, reduction over d
//   codes    s_h = max|h| / 127, hq = rint(127 h / max|h|)       in shared memory, in the tcgen05 operand layout
//   down     y = (hq W2^T) s_h s_2                               jobs of 256 output columns, reduction over H
// with the results of k_int8_gemm / k_quant_groups / k_int8_gemm bit for bit (moe_expert_ffn_int8 in the header).
//
// Why: at H <= 256 the products are short (d = 768, H = 256: six and two 128-code steps a tile), so that three
// kernels spend their time on h: written as bf16, read and written as codes, read again.  Here a tile's h never
// leaves the SM: a thread holds its 32 columns of h per job in registers as bf16, the row's maximum joins the four
// threads that share a row through shared memory, and the codes (128 bytes a row per 128 columns) are the A operand
// of the down product as they lie.
//
// Order of work of one CTA (pair): gate/up of tile i + 1 before down of tile i.  The tensor core then has a tile's
// gate/up to do while the epilogue turns the tile before it into codes; h is double-buffered.  Jobs alternate between
// two TMEM accumulators of 256 columns, so an epilogue overlaps the next job's MMAs.  h of tile i is rewritten by the
// epilogue of tile i + 2's gate/up, whose accumulator is ready only after every MMA issued before it, down of tile i
// among them.  Roles as k_int8_gemm: warp 0 TMA, warp 1 MMA, warps 4-19 epilogue.
#pragma once

#include "int8_gemm.cuh"

namespace moe {

template <int H, int CG>
struct I8FusedCfg {
  static constexpr int kHBytes = (H / 128) * kBM * 128;              // one buffer of h codes: 16 KB per 128 columns
  static constexpr int kABytes = kBM * kI8BK;
  static constexpr int kBBytes = (CG == 2 ? 128 : 256) * kI8BK;      // a 256-row B box, half of it per CTA of a pair
  static constexpr int kSlotBytes = kABytes + kBBytes;
  static constexpr int kDownSteps = CG == 2 ? H / 128 : 1;           // down k-steps whose B boxes share a slot
  static constexpr int kBudget = 212 * 1024 - 1024 - 2 * kHBytes;
  static constexpr int kStages = kBudget / kSlotBytes > 8 ? 8 : kBudget / kSlotBytes;
  static constexpr size_t kSmemBytes = 1024 + 2 * (size_t)kHBytes + (size_t)kStages * kSlotBytes;
  static_assert(kStages >= 2 && kDownSteps * kBBytes <= kSlotBytes, "shared memory budget");
};

// p as k_int8_gemm's gate/up (K = d, N = d output columns of y, up_row0 = H, b_scale = s13, b_rows = 2H); s2 [n, d].
template <int MODE, int H, int CG>
__global__ void __launch_bounds__(kI8Threads, 1)
    k_int8_fused(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXFew,
                 const __grid_constant__ CUtensorMap tmW13, const __grid_constant__ CUtensorMap tmW2, const I8Params p,
                 const float* __restrict__ s2) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  using Cfg = I8FusedCfg<H, CG>;
  static_assert(H == 128 || H == 256, "fused expert hidden width");
  constexpr bool kPair = CG == 2;
  constexpr int TM = kBM * CG;
  constexpr int S = Cfg::kStages;
  constexpr int NGU = H / 128;                      // gate/up jobs per tile
  constexpr int NKD = H / kI8BK;                    // down k-steps
  constexpr uint32_t IDESC = idesc_i8_s32(TM, 256);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * Cfg::kHBytes;          // h codes: [2][128 columns][128 rows][128 B], swizzled
  __shared__ __align__(8) uint64_t bar_full[S], bar_empty[S], bar_tfull[2], bar_tempty[2], bar_hready[2], bar_final;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_prefix[kMaxGroupsSmem + 1];
  __shared__ int s_gstart[kMaxGroupsSmem];
  __shared__ int s_grows[kMaxGroupsSmem];
  __shared__ __align__(16) float s_scale[kI8EpiWarps][64];
  __shared__ uint32_t s_top[2][4][kBM];             // partial row maxima of h, by tile parity

  const int warp = warp_id(), lane = lane_id();
  const int crank = kPair ? (int)cluster_ctarank() : 0;   // 0 = leader of the pair
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int n_units = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int nk = (p.K + kI8BK - 1) / kI8BK;
  const int nd = (p.N + 255) / 256;                 // down jobs per tile
  const int G = p.group_rows == nullptr ? 1 : p.n_groups;

  if (warp == 2) i8_group_table(p, TM, s_prefix, s_gstart, s_grows);
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&bar_full[s], 1); mbar_init(&bar_empty[s], 1); }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar_tfull[a], 1);
      mbar_init(&bar_tempty[a], CG * kI8EpiWarps);
      mbar_init(&bar_hready[a], CG * kI8EpiWarps);
    }
    mbar_init(&bar_final, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmXFew);
    tma_prefetch_desc(&tmW13);
    tma_prefetch_desc(&tmW2);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&s_tmem, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&s_tmem, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (kPair) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;
  const int total = s_prefix[G];
  const int mine = total > unit ? (total - unit + n_units - 1) / n_units : 0;   // this unit's tiles

  auto locate = [&](int i, int& g, int& row0, int& rows_left) {   // the unit's i-th tile
    const int tile = unit + i * n_units;
    g = i8_find_group(s_prefix, G, tile);
    const int m_tile = (tile - s_prefix[g]) * TM;
    row0 = s_gstart[g] + m_tile + crank * kBM;
    rows_left = s_grows[g] - m_tile;
  };

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      auto loaded = [](int rows) {
        return rows <= 0 ? 0 : rows > kI8Few ? kBM : (rows + kI8ABox - 1) / kI8ABox * kI8ABox;
      };
      // waits for the slot and arms it; false when a wait gave up
      auto arm = [&](uint32_t bytes) {
        if (!mbar_wait(&bar_empty[stage], phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0601)) return false;
        if (crank == 0) mbar_arrive_expect_tx(&bar_full[stage], bytes);
        return true;
      };
      auto next = [&]() {
        ++issued;
        if (++stage == S) { stage = 0; phase ^= 1u; }
      };
      auto load_b = [&](uint8_t* dst, const CUtensorMap* map, int k0, int row, int g) {
        if (kPair) tma_load_3d_pair(dst, map, mapa_shared(smem_u32(&bar_full[stage]), 0), k0, row, g);
        else tma_load_3d(dst, map, &bar_full[stage], k0, row, g);
      };
      bool ok = true;
      for (int i = 0; i <= mine && ok && !s_abort; ++i) {
        int g, row0, rows_left;
        if (i < mine) {
          locate(i, g, row0, rows_left);
          const int na = loaded(rows_left - crank * kBM);
          const int na_all = kPair ? loaded(rows_left) + loaded(rows_left - kBM) : na;
          const uint32_t bytes = (uint32_t)(na_all * kI8BK + CG * Cfg::kBBytes);
          for (int job = 0; job < NGU && ok; ++job) {
            for (int kb = 0; kb < nk; ++kb) {
              if (!(ok = arm(bytes))) break;
              uint8_t* a_s = ring + (size_t)stage * Cfg::kSlotBytes;
              uint8_t* b_s = a_s + Cfg::kABytes;
              const CUtensorMap* mx = na == kBM ? &tmX : &tmXFew;
              const int step = na == kBM ? kBM : kI8ABox;
              for (int r = 0; r < na; r += step) {
                if (kPair)
                  tma_load_2d_pair(a_s + r * kI8BK, mx, mapa_shared(smem_u32(&bar_full[stage]), 0), kb * kI8BK,
                                   row0 + r);
                else
                  tma_load_2d(a_s + r * kI8BK, mx, &bar_full[stage], kb * kI8BK, row0 + r);
              }
              if (kPair) {
                load_b(b_s, &tmW13, kb * kI8BK, (crank == 0 ? 0 : H) + 128 * job, g);
              } else {
                load_b(b_s, &tmW13, kb * kI8BK, 128 * job, g);
                load_b(b_s + 128 * kI8BK, &tmW13, kb * kI8BK, H + 128 * job, g);
              }
              next();
            }
          }
        }
        if (i > 0 && ok) {
          locate(i - 1, g, row0, rows_left);
          for (int job = 0; job < nd && ok; ++job) {
            for (int kb = 0; kb < NKD; kb += Cfg::kDownSteps) {
              if (!(ok = arm((uint32_t)(CG * Cfg::kDownSteps * Cfg::kBBytes)))) break;
              uint8_t* b_s = ring + (size_t)stage * Cfg::kSlotBytes;
              for (int j = 0; j < Cfg::kDownSteps; ++j)
                load_b(b_s + j * Cfg::kBBytes, &tmW2, (kb + j) * kI8BK, 256 * job + 128 * crank, g);
              next();
            }
          }
        }
      }
      // no copy may still be landing in shared memory when the CTA ends
      if (crank == 0) {
        const int last = (int)(issued < S ? issued : (long long)S);
        for (int i = 1; i <= last; ++i) {
          const long long n = issued - i;
          volatile int dummy = 0;
          mbar_wait(&bar_full[(int)(n % S)], (uint32_t)((n / S) & 1), p.wait_limit_ns, &dummy, 0x0602);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader CTA)
    if (lane == 0 && crank == 0) {
      int stage = 0, slot = 0;
      uint32_t phase = 0, slot_phase = 0;
      const uint32_t h_addr = smem_u32(smem);
      auto mma128 = [&](uint32_t d_tmem, uint32_t a_addr, uint32_t b_addr, bool first) {
#pragma unroll
        for (int kk = 0; kk < kI8BK / 32; ++kk)
          tc_mma_i8<CG>(d_tmem, smem_desc_k128(a_addr + kk * 32), smem_desc_k128(b_addr + kk * 32), IDESC,
                        (!first || kk > 0) ? 1u : 0u);
      };
      auto acquire = [&]() {
        if (!mbar_wait(&bar_tempty[slot], slot_phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0603)) return false;
        tc_fence_after();
        return true;
      };
      auto full = [&]() {
        if (!mbar_wait(&bar_full[stage], phase, p.wait_limit_ns, &s_abort, 0x0605)) return false;
        tc_fence_after();
        return true;
      };
      auto release_stage = [&]() {
        if (kPair) tc_commit_pair_mc(&bar_empty[stage], 0x3);
        else tc_commit(&bar_empty[stage]);
        if (++stage == S) { stage = 0; phase ^= 1u; }
      };
      auto publish = [&]() {
        if (kPair) tc_commit_pair_mc(&bar_tfull[slot], 0x3);
        else tc_commit(&bar_tfull[slot]);
        if (++slot == 2) { slot = 0; slot_phase ^= 1u; }
      };
      bool ok = true;
      for (int i = 0; i <= mine && ok && !s_abort; ++i) {
        if (i < mine) {
          for (int job = 0; job < NGU && ok; ++job) {
            if (!(ok = acquire())) break;
            const uint32_t d_tmem = tmem_base + (uint32_t)(slot * 256);
            for (int kb = 0; kb < nk; ++kb) {
              if (!(ok = full())) break;
              const uint32_t a_addr = smem_u32(ring + (size_t)stage * Cfg::kSlotBytes);
              mma128(d_tmem, a_addr, a_addr + Cfg::kABytes, kb == 0);
              release_stage();
            }
            if (ok) publish();
          }
        }
        if (i > 0 && ok) {
          const int t = i - 1;
          // h codes of tile t, written by both CTAs' epilogues
          if (!(ok = mbar_wait_cluster(&bar_hready[t & 1], (uint32_t)((t >> 1) & 1), p.wait_limit_ns, &s_abort, 0x0604)))
            break;
          tc_fence_after();
          for (int job = 0; job < nd && ok; ++job) {
            if (!(ok = acquire())) break;
            const uint32_t d_tmem = tmem_base + (uint32_t)(slot * 256);
            for (int kb = 0; kb < NKD; kb += Cfg::kDownSteps) {
              if (!(ok = full())) break;
              const uint32_t b_addr = smem_u32(ring + (size_t)stage * Cfg::kSlotBytes);
#pragma unroll
              for (int j = 0; j < Cfg::kDownSteps; ++j)
                mma128(d_tmem, h_addr + (uint32_t)((t & 1) * Cfg::kHBytes + (kb + j) * (kBM * 128)),
                       b_addr + (uint32_t)(j * Cfg::kBBytes), kb + j == 0);
              release_stage();
            }
            if (ok) publish();
          }
        }
      }
      if (kPair) tc_commit_pair(&bar_final);
      else tc_commit(&bar_final);
      volatile int dummy = 0;
      mbar_wait(&bar_final, 0, p.wait_limit_ns, &dummy, 0x0606);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------ epilogue
    const int ew = warp - 4;
    const int q = warp & 3;                  // TMEM lane quarter
    const int part = ew >> 2;                // this warp's quarter of a job's columns
    const int row = q * 32 + lane;           // this thread's row of the tile
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    float* scl = s_scale[ew];
    int slot = 0;
    uint32_t slot_phase = 0;
    float hs = 0.f, hs_prev = 0.f;           // scale of this row's codes: the tile just encoded, the one before
    auto arrive = [&](uint64_t* bar) {       // one arrival per warp, on the leader's barrier
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
        else mbar_arrive(bar);
      }
    };
    bool ok = true;
    // after a wait that gave up the loop runs on without waits or stores, so that all 16 warps meet at the barrier
    for (int i = 0; i <= mine; ++i) {
      int g, row0, rows_left;
      if (i < mine) {
        locate(i, g, row0, rows_left);
        const bool live = row < rows_left - crank * kBM;
        const float sx = live ? p.a_scale[(long long)row0 + row] : 0.f;
        const float* s13 = p.b_scale + (size_t)g * (2 * H) + 32 * part + lane;
        uint32_t hv[NGU][16] = {};           // h, bf16 pairs: 32 columns per job
        uint32_t top = 0;                    // maximum of |h| as bf16 bits, per half word
#pragma unroll
        for (int job = 0; job < NGU; ++job) {
          if (!ok) break;
          __syncwarp();
          scl[lane] = s13[128 * job];
          scl[32 + lane] = s13[H + 128 * job];
          __syncwarp();
          if (!mbar_wait(&bar_tfull[slot], slot_phase, p.wait_limit_ns, &s_abort, 0x0607)) { ok = false; break; }
          tc_fence_after();
          const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * 256 + 32 * part);
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
            uint32_t v[16], u[16];
            tmem_ld16(t_row + c0, v);
            tmem_ld16(t_row + 128 + c0, u);
            tmem_ld_wait();
            if (c0 == 16) {
              tc_fence_before();
              arrive(&bar_tempty[slot]);
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 sg = *reinterpret_cast<const float4*>(scl + c0 + j);
              const float4 su = *reinterpret_cast<const float4*>(scl + 32 + c0 + j);
              const float gs[4] = {sg.x, sg.y, sg.z, sg.w}, us[4] = {su.x, su.y, su.z, su.w};
              float f[4];
#pragma unroll
              for (int l = 0; l < 4; ++l)
                f[l] = i8_act<MODE>((float)(int)v[j + l] * sx * gs[l]) * ((float)(int)u[j + l] * sx * us[l]);
              hv[job][(c0 + j) / 2] = pack_bf16x2(f[0], f[1]);
              hv[job][(c0 + j) / 2 + 1] = pack_bf16x2(f[2], f[3]);
              top = __vmaxu2(top, __vmaxu2(hv[job][(c0 + j) / 2] & 0x7FFF7FFFu,
                                           hv[job][(c0 + j) / 2 + 1] & 0x7FFF7FFFu));
            }
          }
          if (++slot == 2) { slot = 0; slot_phase ^= 1u; }
        }
        // the row's maximum over its four threads, then the codes into the operand layout: the row's 128 bytes of a
        // 128-column atom, 16-byte chunk c at position c ^ (row & 7)
        s_top[i & 1][part][row] = max(top << 16, top & 0xFFFF0000u);
        named_bar_sync(1, kI8EpiWarps * 32);
        uint32_t m = s_top[i & 1][0][row];
#pragma unroll
        for (int k = 1; k < 4; ++k) m = max(m, s_top[i & 1][k][row]);
        float r;
        hs_prev = hs;
        quant_scale(__uint_as_float(m), hs, r);
        uint8_t* h_row = smem + (size_t)(i & 1) * Cfg::kHBytes + (size_t)row * 128;
        const uint32_t sw = (uint32_t)(row & 7);
#pragma unroll
        for (int job = 0; job < NGU; ++job) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a = hv[job][8 * c + 2 * j], b = hv[job][8 * c + 2 * j + 1];
              o[j] = pack_codes(quant_code(bf16lo(a), r), quant_code(bf16hi(a), r), quant_code(bf16lo(b), r),
                                quant_code(bf16hi(b), r));
            }
            *reinterpret_cast<uint4*>(h_row + (size_t)job * (kBM * 128) + (((uint32_t)(2 * part + c) ^ sw) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        // publish to the tensor core (async proxy) and to the leader's MMA issuer
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (kPair) mbar_arrive_cluster_release(mapa_shared(smem_u32(&bar_hready[i & 1]), 0));
          else mbar_arrive(&bar_hready[i & 1]);
        }
      } else {
        hs_prev = hs;
      }
      if (i > 0 && ok) {
        locate(i - 1, g, row0, rows_left);
        const bool live = row < rows_left - crank * kBM;
        __nv_bfloat16* out = p.out + ((long long)row0 + row) * p.N + 64 * part;
        const float* s2g = s2 + (size_t)g * p.N + 64 * part;
        for (int job = 0; job < nd; ++job) {
          const int cols = p.N - 256 * job - 64 * part;   // a multiple of 16, may be <= 0
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 64; c += 32) scl[c + lane] = c + lane < cols ? s2g[256 * job + c + lane] : 0.f;
          __syncwarp();
          if (!mbar_wait(&bar_tfull[slot], slot_phase, p.wait_limit_ns, &s_abort, 0x0608)) { ok = false; break; }
          tc_fence_after();
          const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * 256 + 64 * part);
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(t_row + c0, v);
            tmem_ld_wait();
            if (c0 == 48) {
              tc_fence_before();
              arrive(&bar_tempty[slot]);
            }
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 sg = *reinterpret_cast<const float4*>(scl + c0 + j);
              o[j / 2] = pack_bf16x2((float)(int)v[j] * hs_prev * sg.x, (float)(int)v[j + 1] * hs_prev * sg.y);
              o[j / 2 + 1] = pack_bf16x2((float)(int)v[j + 2] * hs_prev * sg.z, (float)(int)v[j + 3] * hs_prev * sg.w);
            }
            if (live && c0 < cols) st_row16(out + 256 * job + c0, o, wide);
          }
          if (++slot == 2) { slot = 0; slot_phase ^= 1u; }
        }
      }
    }
  }
  tc_fence_before();
  if (kPair) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (kPair) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace moe
