// Gradients of the grouping and of the weighted combine as steps of their own, for experts that are not this
// library's (moe_backward holds them inside its chain).  With p_tj the grouped row of (token t, slot j), -1 when
// the capacity dropped it:
//   combine   out_t = sum_j w_tj y[p_tj] + ysh_t   ->   dy[p_tj] = w_tj dout_t,  dw_tj = <dout_t, y[p_tj]>,
//                                                       dysh = dout (no work)
//   dispatch  x_perm[p_tj] = x_t                   ->   dx_t = sum_j dx_perm[p_tj]
// (moe_stream.py ``out[mask] += w * expert_out``; ExpertMesh flowchart "Group activations by expert owner" and
// "Weighted top-k reduction".)  Every output row has one writer and every sum a fixed order: no atomics, and
// identical inputs give bit-identical outputs.  Both kernels move each row once and are bound by HBM.
#pragma once

#include "common.cuh"

namespace moe {

// A row index read from the caller's table is used only inside [0, R): anything else counts as dropped.
__device__ __forceinline__ int row_or_none(int p, int R) { return (unsigned)p < (unsigned)R ? p : -1; }

// Eight consecutive elements of a row, held in fp32.  bf16: one 16-byte access, fp32: two.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
  f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

constexpr int kPadRows = 64;   // padding rows that one CTA of k_combine_bwd clears

// W warps per token.  Each lane takes 16-byte column slices: it reads the slice of dout once, then for every slot
// reads the slice of y (the k loads are issued together), adds its part of <dout, y> and writes w dout.  The k dot
// products end in an xor tree over the lanes and, with W > 1, a sum over the warps in order.
// CTAs from tok_blocks on clear the rows of each group's slab that no slot fills (kept given, capacity cap).
// The bound on registers sets how many rows are in flight: 32768 tokens of width 768, top-4, 163968 rows take 83 us
// (6.1 TB/s) at five CTAs an SM, 94 us without the bound, 88 us at six, 99 us at seven (spills); loads and stores with
// streaming hints take 102 to 104 us.
template <int KMAX, int W>
__global__ void __launch_bounds__(256, KMAX <= 4 ? 5 : KMAX <= 8 ? 3 : 2) k_combine_bwd(const __nv_bfloat16* __restrict__ dout,
                                                     const __nv_bfloat16* __restrict__ y,
                                                     const int32_t* __restrict__ slot_pos, const float* __restrict__ w,
                                                     __nv_bfloat16* __restrict__ dy, float* __restrict__ dw, int T,
                                                     int d, int k, int R, unsigned tok_blocks,
                                                     const int32_t* __restrict__ kept, int cap) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  const int warp = warp_id(), lane = lane_id();
  if (blockIdx.x >= tok_blocks) {
    const unsigned per = (unsigned)((cap + kPadRows - 1) / kPadRows);
    const unsigned b = blockIdx.x - tok_blocks;
    const int e = (int)(b / per);
    const int first = min(max(kept[e], 0), cap) + (int)(b % per) * kPadRows;
    const int last = min(cap, first + kPadRows);
    for (int r = first + warp; r < last; r += 8) {
      uint4* row = reinterpret_cast<uint4*>(dy + ((size_t)e * cap + r) * d);
      for (int v = lane; v < (d >> 3); v += 32) row[v] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  __shared__ float part[W > 1 ? 8 : 1][KMAX];
  const long long t = (long long)blockIdx.x * (8 / W) + warp / W;
  if (t >= T) return;   // W > 1: one token per CTA, so the whole CTA leaves
  int p[KMAX];
  float g[KMAX], acc[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    p[j] = j < k ? row_or_none(slot_pos[t * k + j], R) : -1;
    g[j] = j < k ? w[t * k + j] : 0.f;
    acc[j] = 0.f;
  }
  const int nvec = d >> 3;
  for (int v = (warp % W) * 32 + lane; v < nvec; v += 32 * W) {
    float o[8];
    load8(dout + t * d + 8 * v, o);
    if (dw != nullptr) {
      uint4 u[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        u[j] = p[j] >= 0 ? *reinterpret_cast<const uint4*>(y + (size_t)p[j] * d + 8 * v) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        acc[j] = fmaf(o[0], bf16lo(u[j].x), acc[j]); acc[j] = fmaf(o[1], bf16hi(u[j].x), acc[j]);
        acc[j] = fmaf(o[2], bf16lo(u[j].y), acc[j]); acc[j] = fmaf(o[3], bf16hi(u[j].y), acc[j]);
        acc[j] = fmaf(o[4], bf16lo(u[j].z), acc[j]); acc[j] = fmaf(o[5], bf16hi(u[j].z), acc[j]);
        acc[j] = fmaf(o[6], bf16lo(u[j].w), acc[j]); acc[j] = fmaf(o[7], bf16hi(u[j].w), acc[j]);
      }
    }
    if (dy != nullptr) {
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (p[j] < 0) continue;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = g[j] * o[i];
        store8(dy + (size_t)p[j] * d + 8 * v, q);
      }
    }
  }
  if (dw == nullptr) return;
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], s);
    if (p[j] < 0) acc[j] = 0.f;   // also where dout is not finite
  }
  if (W == 1) {
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < k && lane == j) dw[t * k + j] = acc[j];
  } else {
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < KMAX; ++j) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) s += part[i][threadIdx.x];
      dw[t * k + threadIdx.x] = s;
    }
  }
}

// dx_t = sum over the kept slots of dx_perm rows (slot order, fp32), plus add_t when given; one thread per eight
// columns of a token, its k row loads issued together.  `add` may be dx itself: the thread reads its slice first.
// Bound by HBM: 32768 tokens of width 768, top-4, bf16 in 40.5 us (6.2 TB/s); 1500 of width 7168, top-8, fp32 with an
// addend in 66 us (6.5 TB/s).
template <int KMAX, typename TIn, typename TOut>
__global__ void __launch_bounds__(256) k_permute_bwd(const TIn* __restrict__ dx_perm,
                                                     const int32_t* __restrict__ slot_pos, const TOut* add, TOut* dx,
                                                     int T, int d, int k, int R) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int nvec = d >> 3;
  if (i >= (long long)T * nvec) return;
  const long long t = i / nvec;
  const int v = (int)(i - t * nvec);
  float f[KMAX][8];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const int p = j < k ? row_or_none(slot_pos[t * k + j], R) : -1;
    if (p >= 0) load8(dx_perm + (size_t)p * d + 8 * v, f[j]);
    else {
#pragma unroll
      for (int q = 0; q < 8; ++q) f[j][q] = 0.f;
    }
  }
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    acc[q] = f[0][q];
#pragma unroll
    for (int j = 1; j < KMAX; ++j) acc[q] += f[j][q];
  }
  if (add != nullptr) {
    float a[8];
    load8(add + t * d + 8 * v, a);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += a[q];
  }
  store8(dx + t * d + 8 * v, acc);
}

}  // namespace moe
