// Symmetric 8-bit quantisation of rows: one fp32 scale a row (a token of the activations, an output channel of the
// weights), the form the 8-bit integer expert products take (int8_gemm.cuh).  With m = max|x_r| of row r:
//   s_r = m / 127 (IEEE),   q = rint(127 x / m), ties to even, in [-127, 127],   x ~ q s_r.
// A row with m < 2^-119 (zeros among them) gets s = 0, q = 0, so that 127 / m stays finite.  A row that holds an
// infinity or a NaN gets that as its scale, so what is computed from it is not finite either.
//
// q is computed as fma(x, r, 1.5 2^23) with r = 127 / m rounded up: the sum's low byte is rint(x r).  For bf16 rows
// this is exactly rint(127 x / m).  r is less than 2^-23 of itself too large, which moves a quotient Q = 127 x / m by
// less than 2^-23 Q.  With x = X 2^a and m = M 2^(a + s), X and M integers below 256, Q's distance from a tie n + 1/2 is
// |254 X - (2n + 1) M 2^s| / (2 M 2^s): when it is not zero, at least 1 / (2 M 2^s) = Q / (254 X), about 2^-16 Q.  Of the
// ties, those with 127 / m a power of two are exact; in the others 127 divides 2n + 1, so |x| = m / 2, where the quotient
// 63.5 rounds to 64 and r >= 127 / m keeps it there.
// (For fp32 rows a quotient within 2^-16 of a tie may go either way.)
// The pass is bound by HBM: the row stays in registers between the maximum and the codes (131072 bf16 rows of 768: 48 us,
// 6.3 TB/s).
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kQuantTiny = 1.5046327690525280e-36f;   // 2^-119
constexpr int kQuantVec = 4;   // 8-element vectors a thread keeps between the two passes, unless more are asked for

// Eight elements as they lie in memory.
template <typename T> struct RawVec;
template <> struct RawVec<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  // maximum of |x| as bits: a NaN's exceed infinity's, infinity's every number's
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu),
                                __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? a.x : i < 4 ? a.y : i < 6 ? a.z : a.w;
    return (i & 1) ? bf16hi(w) : bf16lo(w);
  }
};
template <> struct RawVec<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ static uint32_t mag(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
  __device__ __forceinline__ uint32_t top() const {
    return max(max(max(mag(a.x), mag(a.y)), max(mag(a.z), mag(a.w))),
               max(max(mag(b.x), mag(b.y)), max(mag(b.z), mag(b.w))));
  }
  __device__ __forceinline__ float at(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
};

// Scale and multiplier of a row with maximum m.
__device__ __forceinline__ void quant_scale(float m, float& s, float& r) {
  if (m < kQuantTiny) {
    s = 0.f;
    r = 0.f;
  } else {
    s = __fdiv_rn(m, 127.0f);
    r = __fdiv_ru(127.0f, m);
  }
}

// rint(x r) in the low byte (|x r| <= 127 (1 + 2^-23)).
__device__ __forceinline__ uint32_t quant_code(float x, float r) { return __float_as_uint(fmaf(x, r, 12582912.0f)); }
__device__ __forceinline__ uint32_t pack_codes(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
  return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
}

template <typename T>
__device__ __forceinline__ uint2 quant_vec(const RawVec<T>& v, float r) {
  return make_uint2(pack_codes(quant_code(v.at(0), r), quant_code(v.at(1), r), quant_code(v.at(2), r),
                               quant_code(v.at(3), r)),
                    pack_codes(quant_code(v.at(4), r), quant_code(v.at(5), r), quant_code(v.at(6), r),
                               quant_code(v.at(7), r)));
}

// One row by TPR threads (8 or 32 lanes of a warp, or the CTA's 256): maximum, then codes handed to put(vector index,
// 8 codes); returns the scale.  Every thread of the warp (or CTA) takes part; with on == false it reads and puts
// nothing.  Rows longer than TPR * NV vectors are read a second time past that.
template <int TPR, int NV, typename T, typename Put>
__device__ __forceinline__ float quant_row(const T* __restrict__ x, int K, bool on, uint32_t* s_max, Put put) {
  const int nvec = on ? K >> 3 : 0;
  const int th = (int)threadIdx.x % TPR;
  RawVec<T> v[NV];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (th + i * TPR < nvec) v[i].load(x + 8 * (th + i * TPR));
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (th + i * TPR < nvec) m = max(m, v[i].top());
  for (int c = th + NV * TPR; c < nvec; c += TPR) {
    RawVec<T> u;
    u.load(x + 8 * c);
    m = max(m, u.top());
  }
  if (TPR == 8) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  } else {
    m = __reduce_max_sync(0xffffffffu, m);
  }
  if (TPR > 32) {
    if (lane_id() == 0) s_max[warp_id()] = m;
    __syncthreads();
    m = s_max[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) m = max(m, s_max[i]);
    __syncthreads();   // s_max may be rewritten for the next row
  }
  float s, r;
  quant_scale(__uint_as_float(m), s, r);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (th + i * TPR < nvec) put(th + i * TPR, quant_vec(v[i], r));
  for (int c = th + NV * TPR; c < nvec; c += TPR) {
    RawVec<T> u;
    u.load(x + 8 * c);
    put(c, quant_vec(u, r));
  }
  return s;
}

// Rows 0 .. rows-1 of x [rows, K], 256 / TPR rows per CTA.
template <int TPR, int NV, typename T>
__global__ void __launch_bounds__(256) k_quant_rows(const T* __restrict__ x, long long rows, int K,
                                                    int8_t* __restrict__ q, float* __restrict__ scale) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  __shared__ uint32_t s_max[8];
  const long long r = (long long)blockIdx.x * (256 / TPR) + (int)threadIdx.x / TPR;
  const bool on = r < rows;
  const float s = quant_row<TPR, NV>(x + r * K, K, on, s_max, [&](int c, uint2 v) {
    reinterpret_cast<uint2*>(q + r * K)[c] = v;
  });
  if (on && (int)threadIdx.x % TPR == 0) scale[r] = s;
}

// The dispatch: token t's row is read once, quantised, and its codes and scale written to the grouped row of each of
// its kept slots; with q_tok, also to row t there (the shared expert's input).
template <int TPR, int KMAX>
__global__ void __launch_bounds__(256) k_quant_slots(const __nv_bfloat16* __restrict__ x,
                                                     const int32_t* __restrict__ slot_pos, int T, int d, int k, int R,
                                                     int8_t* __restrict__ q, float* __restrict__ scale,
                                                     int8_t* __restrict__ q_tok, float* __restrict__ s_tok) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  __shared__ uint32_t s_max[8];
  const long long t = (long long)blockIdx.x * (256 / TPR) + (int)threadIdx.x / TPR;
  const bool on = t < T;
  int p[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    p[j] = on && j < k ? slot_pos[t * k + j] : -1;
    if ((unsigned)p[j] >= (unsigned)R) p[j] = -1;
  }
  const float s = quant_row<TPR, kQuantVec>(x + t * d, d, on, s_max, [&](int c, uint2 v) {
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (p[j] >= 0) reinterpret_cast<uint2*>(q + (size_t)p[j] * d)[c] = v;
    if (q_tok != nullptr) reinterpret_cast<uint2*>(q_tok + t * d)[c] = v;
  });
  if (on && (int)threadIdx.x % TPR == 0) {
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (p[j] >= 0) scale[p[j]] = s;
    if (q_tok != nullptr) s_tok[t] = s;
  }
}

// The whole of moe_permute_int8 for few (token, slot) pairs in one launch: counting, grouping and quantising.  Every CTA
// counts all T k pairs itself (shared-memory additions of ones: the sums do not depend on their order), the pairs of
// earlier CTAs' tokens apart, which gives its own tokens' first ranks without a pass over the GPU before; the ranks
// among its own 256 / TPR tokens come from comparing their pairs.  Then its tokens are quantised into their rows.  The
// results are those of k_chunk_hist, k_chunk_scan, k_scatter and k_quant_slots (four launches / one, us: 256 tokens,
// top-2, width 64: 7.3 / 3.8; 1024 tokens, top-4, width 768: 9.8 / 5.0; 1024 tokens, top-8, width 7168: 21.5 / 21.0).
constexpr int kSmallPairs = 4096;

template <int TPR, int KMAX>
__global__ void __launch_bounds__(256) k_permute_quant_small(const __nv_bfloat16* __restrict__ x,
                                                             const int32_t* __restrict__ topk_idx, int T, int d, int E,
                                                             int k, int cap, int32_t* __restrict__ slot_pos,
                                                             uint8_t* __restrict__ drop, int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ kept, int32_t* __restrict__ offsets,
                                                             int32_t* __restrict__ row_src, int8_t* __restrict__ q,
                                                             float* __restrict__ scale) {
  pdl_wait();  // inputs written by the previous kernel on the stream are visible past this point
  constexpr int TOK = 256 / TPR;
  __shared__ int s_cnt[512], s_before[512], s_off[513];
  __shared__ int s_exp[TOK * KMAX], s_slot[TOK * KMAX];
  __shared__ uint32_t s_max[8];
  const int tid = threadIdx.x, t0 = blockIdx.x * TOK;
  for (int e = tid; e < E; e += 256) s_cnt[e] = s_before[e] = 0;
  __syncthreads();
  for (int i = tid; i < T * k; i += 256) {
    const int e = topk_idx[i];
    if ((unsigned)e >= (unsigned)E) continue;
    atomicAdd(&s_cnt[e], 1);
    if (i < t0 * k) atomicAdd(&s_before[e], 1);
  }
  const int mine = min(TOK, T - t0) * k;   // this CTA's pairs
  for (int i = tid; i < mine; i += 256) s_exp[i] = topk_idx[t0 * k + i];
  __syncthreads();
  if (tid < 32) {   // first row of each group
    const int per = (E + 31) / 32, e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int local = 0;
    for (int e = e0; e < e1; ++e) local += cap > 0 ? cap : s_cnt[e];
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += v;
    }
    int run = incl - local;
    for (int e = e0; e < e1; ++e) {
      s_off[e] = run;
      run += cap > 0 ? cap : s_cnt[e];
    }
    if (tid == 31) s_off[E] = incl;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = tid; e < E; e += 256) {
      if (counts) counts[e] = s_cnt[e];
      kept[e] = cap > 0 ? min(cap, s_cnt[e]) : s_cnt[e];
      offsets[e] = s_off[e];
    }
    if (tid == 0) offsets[E] = s_off[E];
  }
  for (int i = tid; i < mine; i += 256) {
    const int e = s_exp[i];
    int pos = -1;
    if ((unsigned)e < (unsigned)E) {
      int rank = s_before[e];
      for (int o = 0; o < i; ++o) rank += s_exp[o] == e;
      if (cap == 0 || rank < cap) pos = s_off[e] + rank;
    }
    const int pair = t0 * k + i;
    s_slot[i] = pos;
    slot_pos[pair] = pos;
    if (drop) drop[pair] = pos < 0 ? 1 : 0;
    if (row_src && pos >= 0) row_src[pos] = pair;
  }
  __syncthreads();
  const int lt = tid / TPR;
  const bool on = t0 + lt < T;
  int p[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) p[j] = on && j < k ? s_slot[lt * k + j] : -1;
  const float s = quant_row<TPR, kQuantVec>(x + (size_t)(t0 + lt) * d, d, on, s_max, [&](int c, uint2 v) {
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (p[j] >= 0) reinterpret_cast<uint2*>(q + (size_t)p[j] * d)[c] = v;
  });
  if (on && tid % TPR == 0) {
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (p[j] >= 0) scale[p[j]] = s;
  }
}

}  // namespace moe
