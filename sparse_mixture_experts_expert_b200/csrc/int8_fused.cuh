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
// Order of work of one CTA (pair): the gate/up jobs of tile i + 1, the down jobs of tile i, the codes of tile i + 1 (for
// d = 768, H = 256: G0 G1 D0 D1 D2 C).  The tensor core has the next tile's gate/up to do while the epilogue makes the
// codes, and the epilogue has two finished gate/up accumulators when it is through with them.
// Jobs alternate between two TMEM accumulators of 256 columns, so an epilogue overlaps the next job's MMAs.  The codes
// of tile i + 1 replace those of tile i after the epilogue has seen tile i's last down accumulator, that is after every
// MMA that reads them.  The epilogue is what the kernel waits for, so it is kept lean: channel scales come by bulk
// copies of the producer, y leaves through shared memory by TMA (a warp's 32 rows x 32 columns at a time; stores from
// registers touch 32 lines each and held up the fence before the codes are published), and warps without rows skip
// the arithmetic.  Roles as k_int8_gemm: warps 0, 2, 3 copies, warp 1 MMA, warps 4-19 epilogue.
//
// Measured (B200), 131072 rows over 192 experts of 768 x 256: 98 us against 172 us for the three kernels (floors: 414 MB
// 64 us, 155 GOP 47 us).  Tensor pipe 39% busy, issue slots 51%, DRAM 46%: the waits of the MMA thread are about
// evenly on accumulators (the down epilogues), on operands and on its own issue.  Eight epilogue warps for each
// accumulator instead of sixteen for one at a time took 5 us more, prefetching the next tile into L2 33 us more.
#pragma once

#include "int8_gemm.cuh"

namespace moe {

template <int H, int CG>
struct I8FusedCfg {
  static constexpr int kHBytes = (H / 128) * kBM * 128;              // h codes: 16 KB per 128 columns
  static constexpr int kABytes = kBM * kI8BK;
  static constexpr int kBBytes = (CG == 2 ? 128 : 256) * kI8BK;      // a 256-row B box, half of it per CTA of a pair
  static constexpr int kSlotBytes = kABytes + kBBytes;
  static constexpr int kDownSteps = CG == 2 ? H / 128 : 1;           // down k-steps whose B boxes share a slot
  static constexpr int kOutBytes = CG == 2 ? kI8EpiWarps * 32 * 64 : 0;    // y staging: 2 KB per epilogue warp
  static constexpr int kBudget = 208 * 1024 - 1024 - kHBytes - kOutBytes;
  static constexpr int kStages = kBudget / kSlotBytes > 8 ? 8 : kBudget / kSlotBytes;
  static constexpr size_t kSmemBytes = 1024 + (size_t)kHBytes + kOutBytes + (size_t)kStages * kSlotBytes;
  static_assert(kStages >= 2 && kDownSteps * kBBytes <= kSlotBytes, "shared memory budget");
};

// p as k_int8_gemm's gate/up (K = d, N = d output columns of y, up_row0 = H, b_scale = s13, b_rows = 2H); s2 [n, d].
template <int MODE, int H, int CG>
__global__ void __launch_bounds__(kI8Threads, 1)
    k_int8_fused(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXFew,
                 const __grid_constant__ CUtensorMap tmW13, const __grid_constant__ CUtensorMap tmW2,
                 const __grid_constant__ CUtensorMap tmY, const I8Params p, const float* __restrict__ s2) {
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
  // h codes [128 columns][128 rows][128 B], y staging [16 warps][32 rows][64 B] (both swizzled), ring
  uint8_t* stage_y = smem + Cfg::kHBytes;
  uint8_t* ring = stage_y + Cfg::kOutBytes;
  __shared__ __align__(8) uint64_t bar_full[S], bar_empty[S], bar_tfull[2], bar_tempty[2], bar_final;
  // h codes written: by this CTA's epilogue warps, and (on the leader) by the pair's other CTA
  __shared__ __align__(8) uint64_t bar_hlocal, bar_hpeer;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_prefix[kMaxGroupsSmem + 1];
  __shared__ int s_gstart[kMaxGroupsSmem];
  __shared__ int s_grows[kMaxGroupsSmem];
  // channel scales of the jobs in flight (gate then up, or 256 of s2), copied in by the producer
  __shared__ __align__(16) float s_scale[kI8ScaleBufs][256];
  __shared__ __align__(8) uint64_t bar_sfull[kI8ScaleBufs], bar_sempty[kI8ScaleBufs];
  __shared__ uint32_t s_top[2][4][kBM];             // partial row maxima of h, by tile parity

  const int warp = warp_id_uniform(), lane = lane_id();
  const int crank = kPair ? (int)cluster_ctarank() : 0;   // 0 = leader of the pair
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int n_units = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int nk = (p.K + kI8BK - 1) / kI8BK;
  const int nd = (p.N + 255) / 256;                 // down jobs per tile
  const int G = p.group_rows == nullptr ? 1 : p.n_groups;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(&bar_full[s], 1); mbar_init(&bar_empty[s], 1); }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar_tfull[a], 1);
      mbar_init(&bar_tempty[a], CG * kI8EpiWarps);
    }
    mbar_init(&bar_hlocal, kI8EpiWarps);
    mbar_init(&bar_hpeer, 1);
    for (int b = 0; b < kI8ScaleBufs; ++b) { mbar_init(&bar_sfull[b], 1); mbar_init(&bar_sempty[b], kI8EpiWarps); }
    mbar_init(&bar_final, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmXFew);
    tma_prefetch_desc(&tmW13);
    tma_prefetch_desc(&tmW2);
    if (Cfg::kOutBytes > 0) tma_prefetch_desc(&tmY);
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
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  if (warp == 3) i8_group_table(p, TM, s_prefix, s_gstart, s_grows);
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

  // As in k_int8_gemm the copies are dealt to three warps.  Each walks the jobs in the same order.
  if (warp == 0) {
    // ------------------------------------------------ x tiles, and the byte counts of every slot
    if (lane == 0) {
      RingPos<S> r;
      long long issued = 0;
      bool ok = true;
      const uint32_t fb0 = kPair ? mapa_shared(smem_u32(&bar_full[0]), 0) : 0;
      auto loaded = [](int rows) {
        return rows <= 0 ? 0 : rows > kI8Few ? kBM : (rows + kI8ABox - 1) / kI8ABox * kI8ABox;
      };
      // waits for the slot and arms it; false when a wait gave up
      auto arm = [&](uint32_t bytes) {
        if (!mbar_wait(&bar_empty[r.stage], r.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0601)) return false;
        if (crank == 0) mbar_arrive_expect_tx(&bar_full[r.stage], bytes);
        return true;
      };
      for (int i = 0; i <= mine && ok && !s_abort; ++i) {
        int g, row0 = 0, rows_left = 0;
        if (i < mine) locate(i, g, row0, rows_left);
        const int na = loaded(rows_left - crank * kBM);
        const int na_all = kPair ? loaded(rows_left) + loaded(rows_left - kBM) : na;
        const uint32_t bytes = (uint32_t)(na_all * kI8BK + CG * Cfg::kBBytes);
        const CUtensorMap* mx = na == kBM ? &tmX : &tmXFew;
        const int step = na == kBM ? kBM : kI8ABox;
        for (int job = 0; i < mine && ok && job < NGU; ++job) {
          for (int k0 = 0; k0 < p.K; k0 += kI8BK) {
            if (!(ok = arm(bytes))) break;
            uint8_t* a_s = ring + (size_t)r.stage * Cfg::kSlotBytes;
            for (int n = 0; n < na; n += step) {
              if (kPair) tma_load_2d_pair(a_s + n * kI8BK, mx, fb0 + 8 * r.stage, k0, row0 + n);
              else tma_load_2d(a_s + n * kI8BK, mx, &bar_full[r.stage], k0, row0 + n);
            }
            ++issued;
            r.next();
          }
        }
        for (int n = 0; i > 0 && ok && n < nd * (NKD / Cfg::kDownSteps); ++n) {   // W2 alone
          if (!(ok = arm((uint32_t)(CG * Cfg::kDownSteps * Cfg::kBBytes)))) break;
          ++issued;
          r.next();
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
  } else if (warp == 2) {
    // ------------------------------------------------ weight tiles
    if (lane == 0) {
      RingPos<S> r;
      bool ok = true;
      const uint32_t fb0 = kPair ? mapa_shared(smem_u32(&bar_full[0]), 0) : 0;
      auto empty = [&]() { return mbar_wait(&bar_empty[r.stage], r.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x060E); };
      auto load_b = [&](uint8_t* dst, const CUtensorMap* map, int k0, int row, int g) {
        if (kPair) tma_load_3d_pair(dst, map, fb0 + 8 * r.stage, k0, row, g);
        else tma_load_3d(dst, map, &bar_full[r.stage], k0, row, g);
      };
      int g = 0, gd = 0;
      for (int i = 0; i <= mine && ok && !s_abort; ++i) {
        int row0, rows_left;
        gd = g;
        if (i < mine) locate(i, g, row0, rows_left);
        for (int job = 0; i < mine && ok && job < NGU; ++job) {
          for (int k0 = 0; k0 < p.K; k0 += kI8BK) {
            if (!(ok = empty())) break;
            uint8_t* b_s = ring + (size_t)r.stage * Cfg::kSlotBytes + Cfg::kABytes;
            if (kPair) {
              load_b(b_s, &tmW13, k0, (crank == 0 ? 0 : H) + 128 * job, g);
            } else {
              load_b(b_s, &tmW13, k0, 128 * job, g);
              load_b(b_s + 128 * kI8BK, &tmW13, k0, H + 128 * job, g);
            }
            r.next();
          }
        }
        for (int jd = 0; jd < nd && ok; ++jd) {
          for (int kb = 0; i > 0 && ok && kb < NKD; kb += Cfg::kDownSteps) {
            if (!(ok = empty())) break;
            uint8_t* b_s = ring + (size_t)r.stage * Cfg::kSlotBytes;
            for (int j = 0; j < Cfg::kDownSteps; ++j)
              load_b(b_s + j * Cfg::kBBytes, &tmW2, (kb + j) * kI8BK, 256 * jd + 128 * crank, gd);
            r.next();
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------ channel scales
    if (lane == 0) {
      RingPos<kI8ScaleBufs> r;
      long long issued = 0;
      bool ok = true;
      // a job's channel scales: n floats of a (and of b, behind 128 floats)
      auto load_scales = [&](const float* a, const float* b, int n) {
        if (!mbar_wait(&bar_sempty[r.stage], r.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0609)) return false;
        mbar_arrive_expect_tx(&bar_sfull[r.stage], (uint32_t)n * (b != nullptr ? 8u : 4u));
        bulk_load(&s_scale[r.stage][0], a, (uint32_t)n * 4, &bar_sfull[r.stage]);
        if (b != nullptr) bulk_load(&s_scale[r.stage][128], b, (uint32_t)n * 4, &bar_sfull[r.stage]);
        ++issued;
        r.next();
        return true;
      };
      int g = 0, gd = 0;
      for (int i = 0; i <= mine && ok && !s_abort; ++i) {
        int row0, rows_left;
        gd = g;
        if (i < mine) locate(i, g, row0, rows_left);
        for (int job = 0; i < mine && ok && job < NGU; ++job) {
          const float* s13 = p.b_scale + (size_t)g * (2 * H) + 128 * job;
          ok = load_scales(s13, s13 + H, 128);
        }
        for (int jd = 0; jd < nd && ok; ++jd) {
          if (i > 0) ok = load_scales(s2 + (size_t)gd * p.N + 256 * jd, nullptr, min(256, p.N - 256 * jd));
        }
      }
      i8_drain_scales(bar_sfull, issued, p.wait_limit_ns, 0x060A);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader CTA)
    if (crank == 0) {
      RingPos<S> r;
      RingPos<2> acc;
      const uint32_t lead = lane == 0, h_addr = smem_u32(smem), ring_addr = smem_u32(ring);
      auto acquire = [&]() {
        if (!mbar_wait_warp(&bar_tempty[acc.stage], acc.phase ^ 1u, p.wait_limit_ns, &s_abort, 0x0603)) return false;
        tc_fence_after();
        return true;
      };
      auto full = [&]() {
        if (!mbar_wait_warp(&bar_full[r.stage], r.phase, p.wait_limit_ns, &s_abort, 0x0605)) return false;
        tc_fence_after();
        return true;
      };
      auto release_stage = [&]() {
        tc_commit_i8<CG>(lead, &bar_empty[r.stage]);
        r.next();
      };
      auto publish = [&]() {
        tc_commit_i8<CG>(lead, &bar_tfull[acc.stage]);
        acc.next();
      };
      bool ok = true;
      for (int i = 0; i <= mine && ok; ++i) {
        for (int job = 0; i < mine && ok && job < NGU; ++job) {
          if (!(ok = acquire())) break;
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc.stage * 256);
          for (int kb = 0; kb < nk; ++kb) {
            if (!(ok = full())) break;
            const uint32_t a_addr = ring_addr + (uint32_t)(r.stage * Cfg::kSlotBytes);
            i8_mma_step<CG>(lead, d_tmem, a_addr, a_addr + Cfg::kABytes, IDESC, kb == 0);
            release_stage();
          }
          if (ok) publish();
        }
        if (i == 0 || !ok) continue;
        const uint32_t ph = (uint32_t)((i - 1) & 1);   // h codes of tile i - 1, written by both CTAs' epilogues
        ok = mbar_wait_warp(&bar_hlocal, ph, p.wait_limit_ns, &s_abort, 0x0604);
        if (kPair && ok)
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(&bar_hpeer, ph, p.wait_limit_ns, &s_abort, 0x060C)) != 0;
        tc_fence_after();
        for (int jd = 0; jd < nd && ok; ++jd) {
          if (!(ok = acquire())) break;
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc.stage * 256);
          for (int kb = 0; kb < NKD; kb += Cfg::kDownSteps) {
            if (!(ok = full())) break;
            const uint32_t b_addr = ring_addr + (uint32_t)(r.stage * Cfg::kSlotBytes);
#pragma unroll
            for (int j = 0; j < Cfg::kDownSteps; ++j)
              i8_mma_step<CG>(lead, d_tmem, h_addr + (uint32_t)((kb + j) * (kBM * 128)),
                              b_addr + (uint32_t)(j * Cfg::kBBytes), IDESC, kb + j == 0);
            release_stage();
          }
          if (ok) publish();
        }
      }
      if (lane == 0) {
        if (kPair) tc_commit_pair(&bar_final);
        else tc_commit(&bar_final);
        volatile int dummy = 0;
        mbar_wait(&bar_final, 0, p.wait_limit_ns, &dummy, 0x0606);
      }
    }
    // The other CTA of a pair passes its epilogue's "h ready" on to the leader.  A release at cluster scope took each
    // epilogue warp about 3500 cycles a tile while stores were under way; here nothing waits for it but the MMAs.
    if (kPair && lane == 0 && crank == 1) {
      for (int t = 0; t < mine; ++t) {
        if (!mbar_wait_cluster(&bar_hlocal, (uint32_t)(t & 1), p.wait_limit_ns, &s_abort, 0x060D)) break;
        mbar_arrive_cluster_release(mapa_shared(smem_u32(&bar_hpeer), 0));
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------ epilogue
    const int ew = warp - 4;
    const int q = warp & 3;                  // TMEM lane quarter
    const int part = ew >> 2;                // this warp's quarter of a job's columns
    const int row = q * 32 + lane;           // this thread's row of the tile
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    int slot = 0;
    uint32_t slot_phase = 0;
    long long n_job = 0;
    float hs = 0.f;                          // scale of this row's codes in the tile encoded last
    auto arrive = [&](uint64_t* bar) {       // one arrival per warp, on the leader's barrier
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
        else mbar_arrive(bar);
      }
    };
    bool ok = true;
    // the job's channel scales and accumulator
    auto job_ready = [&]() {
      const int k = (int)(n_job % kI8ScaleBufs);
      if (!mbar_wait(&bar_sfull[k], (uint32_t)((n_job / kI8ScaleBufs) & 1), p.wait_limit_ns, &s_abort, 0x060B)) return false;
      if (!mbar_wait(&bar_tfull[slot], slot_phase, p.wait_limit_ns, &s_abort, 0x0607)) return false;
      tc_fence_after();
      return true;
    };
    auto job_done = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_sempty[(int)(n_job % kI8ScaleBufs)]);
      ++n_job;
      if (++slot == 2) { slot = 0; slot_phase ^= 1u; }
    };
    // tile i's rows and this thread's token scale are fetched a tile ahead
    int g_n, row0_n = 0, left_n = 0, row0 = 0;
    float sx_n = 0.f;
    auto fetch = [&](int i) {
      left_n = 0;
      sx_n = 0.f;
      if (i >= mine) return;
      locate(i, g_n, row0_n, left_n);
      if (row < left_n - crank * kBM) sx_n = p.a_scale[(long long)row0_n + row];
    };
    fetch(0);
    uint8_t* my_y = stage_y + ew * (32 * 64);
    uint8_t* h_row = smem + (size_t)row * 128;
    const uint32_t sw = (uint32_t)(row & 7);
    int nv = 0;                              // rows of this warp in tile i
    for (int i = 0; i <= mine; ++i) {
      const int nv_d = nv;                   // and in tile i - 1
      const long long y_row0 = (long long)row0 + q * 32;
      const float hs_d = hs;                 // scale of this row's codes in tile i - 1
      row0 = row0_n;
      nv = max(0, min(32, left_n - crank * kBM - q * 32));
      const float sx = sx_n;
      fetch(i + 1);
      uint32_t hv[NGU][16];                  // h of tile i, bf16 pairs: 32 columns per job
      uint32_t top = 0;                      // maximum of |h| as bf16 bits, per half word
#pragma unroll
      for (int job = 0; job < NGU; ++job) {
        if (i == mine || !ok || !(ok = job_ready())) continue;
        const float* scl = &s_scale[(int)(n_job % kI8ScaleBufs)][32 * part];
        const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * 256 + 32 * part);
        if (nv == 0) {
          arrive(&bar_tempty[slot]);
          job_done();
          continue;
        }
        uint32_t v[2][16], u[2][16];
        tmem_ld16(t_row, v[0]);
        tmem_ld16(t_row + 128, u[0]);
#pragma unroll
        for (int c0 = 0; c0 < 32; c0 += 16) {
          tmem_ld_wait();
          if (c0 == 0) {
            tmem_ld16(t_row + 16, v[1]);
            tmem_ld16(t_row + 144, u[1]);
          } else {
            tc_fence_before();
            arrive(&bar_tempty[slot]);
          }
          const uint32_t* vc = v[c0 / 16];
          const uint32_t* uc = u[c0 / 16];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 sg = *reinterpret_cast<const float4*>(scl + c0 + j);
            const float4 su = *reinterpret_cast<const float4*>(scl + 128 + c0 + j);
            const float2 f0 = i8_glu2<MODE>(i8_scaled(vc[j], vc[j + 1], sx, sg.x, sg.y),
                                            i8_scaled(uc[j], uc[j + 1], sx, su.x, su.y));
            const float2 f1 = i8_glu2<MODE>(i8_scaled(vc[j + 2], vc[j + 3], sx, sg.z, sg.w),
                                            i8_scaled(uc[j + 2], uc[j + 3], sx, su.z, su.w));
            const uint32_t p0 = pack_bf16x2(f0.x, f0.y), p1 = pack_bf16x2(f1.x, f1.y);
            hv[job][(c0 + j) / 2] = p0;
            hv[job][(c0 + j) / 2 + 1] = p1;
            top = __vmaxu2(top, __vmaxu2(p0 & 0x7FFF7FFFu, p1 & 0x7FFF7FFFu));
          }
        }
        job_done();
      }
      for (int jd = 0; jd < nd; ++jd) {
        if (i == 0 || !ok || !(ok = job_ready())) continue;
        const int cols = p.N - 256 * jd - 64 * part;   // a multiple of 16, may be <= 0
        const float* scl = &s_scale[(int)(n_job % kI8ScaleBufs)][64 * part];
        const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * 256 + 64 * part);
        if (nv_d == 0 || cols <= 0) {
          arrive(&bar_tempty[slot]);
          job_done();
          continue;
        }
        const bool by_tma = kPair && nv_d == 32;       // a warp whose rows all belong to the group
        uint32_t v[2][16];
        tmem_ld16(t_row, v[0]);
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 16) {
          const uint32_t* vc = v[(c0 / 16) & 1];
          tmem_ld_wait();
          if (c0 < 48) {
            tmem_ld16(t_row + c0 + 16, v[((c0 / 16) & 1) ^ 1]);
          } else {
            tc_fence_before();
            arrive(&bar_tempty[slot]);
          }
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 sg = *reinterpret_cast<const float4*>(scl + c0 + j);
            const float2 f0 = i8_scaled(vc[j], vc[j + 1], hs_d, sg.x, sg.y);
            const float2 f1 = i8_scaled(vc[j + 2], vc[j + 3], hs_d, sg.z, sg.w);
            o[j / 2] = pack_bf16x2(f0.x, f0.y);
            o[j / 2 + 1] = pack_bf16x2(f1.x, f1.y);
          }
          if (by_tma) {   // 32 columns at a time: staging row = lane, 16-byte chunk c at c ^ ((lane >> 1) & 3)
            if (c0 % 32 == 0) {
              if (lane == 0) bulk_wait_read();         // the last store has left the staging rows
              __syncwarp();
            }
            uint4* r = reinterpret_cast<uint4*>(my_y + lane * 64);
            const uint32_t c = (c0 / 8) & 3, x = (uint32_t)(lane >> 1) & 3u;
            r[c ^ x] = make_uint4(o[0], o[1], o[2], o[3]);
            r[(c + 1) ^ x] = make_uint4(o[4], o[5], o[6], o[7]);
            if (c0 % 32 == 16) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmY, my_y, 256 * jd + 64 * part + c0 - 16, (int)y_row0);
                bulk_commit();
              }
            }
          } else if (lane < nv_d && c0 < cols) {
            st_row16(p.out + (y_row0 + lane) * p.N + 256 * jd + 64 * part + c0, o, wide);
          }
        }
        job_done();
      }
      if (i == mine) break;
      // codes of tile i: the row's maximum over its four threads, then the row's 128 bytes of a 128-column atom of the
      // operand layout, 16-byte chunk c at position c ^ (row & 7).  Every warp comes here, also after a wait that gave
      // up (it then waits for and stores nothing any more), so that the barrier is whole.
      s_top[i & 1][part][row] = max(top << 16, top & 0xFFFF0000u);
      named_bar_sync(1, kI8EpiWarps * 32);
      if (!ok) continue;
      if (nv > 0) {
        uint32_t m = s_top[i & 1][0][row];
#pragma unroll
        for (int k = 1; k < 4; ++k) m = max(m, s_top[i & 1][k][row]);
        float r;
        quant_scale(__uint_as_float(m), hs, r);
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
        fence_proxy_async_smem();   // the tensor core reads them through the async proxy
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_hlocal);
    }
    if (kPair && lane == 0) bulk_wait_all();
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
