// Attention with modified scores, a warp a row, straight from the formulas:
// each lane holds D / 32 elements of the row, a product is a warp sum, and only
// visible keys are ever read.  The tensor-core kernels call these for
// the rows whose results are not finite, where a 0 x NaN of a hidden key may have got in.
// Bound by the dependent chain of one warp sum a key: 0.58 us a key and row in a warp beside others (a whole causal
// forward of 2 x 32 heads x 4096 rows took 62 ms this way, against 0.55 ms on the tensor cores).
#pragma once

#include "mod_common.cuh"

namespace smx {

// D / 32 consecutive elements of a row, as fp32, in one access a lane
template <typename T, int N>
struct alignas(sizeof(T) * N) ModPiece {
  T e[N];
};
template <typename T, int D>
__device__ __forceinline__ void mod_row_load(const T* row, float (&f)[D / 32]) {
  using P = ModPiece<T, D / 32>;
  const P p = *(reinterpret_cast<const P*>(row) + (threadIdx.x & 31));
#pragma unroll
  for (int i = 0; i < D / 32; ++i) f[i] = Elem<T>::to_f32(p.e[i]);
}
template <typename T, int D>
__device__ __forceinline__ void mod_row_store(T* row, const float (&f)[D / 32]) {
  using P = ModPiece<T, D / 32>;
  P p;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p.e[i] = Elem<T>::from_f32(f[i]);
  *(reinterpret_cast<P*>(row) + (threadIdx.x & 31)) = p;
}
template <int N>
__device__ __forceinline__ float mod_dot(const float (&x)[N], const float (&y)[N]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = __fmaf_rn(x[i], y[i], s);
  return warp_sum(s);
}

// the warp's largest value (NaN operands are passed over)
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// One row's state over the visible keys of [j0, j1): m (base 2), l and this
// lane's part of the unnormalised o.
template <typename T, int D>
__device__ void mod_exact_row(const ModArgs& a, const T* qrow, const T* kh, const T* vh, const int32_t* kdoc,
                              const ModView& v, float slope2, int64_t j0, int64_t j1, float& m, float& l,
                              float (&o)[D / 32]) {
  constexpr int N = D / 32;
  float q[N];
  mod_row_load<T, D>(qrow, q);
  m = neg_inf();
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.0f;
  const int64_t end = j1 < v.lim ? j1 : v.lim;
  for (int64_t j = j0; j < end; ++j) {
    if (kdoc != nullptr && kdoc[j] != v.doc) continue;
    float k[N];
    mod_row_load<T, D>(kh + j * a.ks[2], k);
    float deriv;
    float y = mod_score(a, mod_dot(q, k), deriv);
    if (slope2 != 0.0f) y += mod_bias(slope2, v.pos, j);
    if (y == neg_inf()) continue;  // weight +0
    const float mn = fmaxf(m, y);
    const float al = m == neg_inf() ? 0.0f : ex2_full(m - mn);
    const float p = ex2_full(y - mn);  // NaN for a NaN or +inf score
    float vr[N];
    mod_row_load<T, D>(vh + j * a.vs[2], vr);
    l = __fmaf_rn(l, al, p);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = __fmaf_rn(p, vr[i], o[i] * al);
    m = mn;
    if (l != l) return;  // a NaN score: the whole row is NaN
  }
}

// LSE in natural units of a state; the empty row is -inf
__device__ __forceinline__ float mod_lse(float m, float l) {
  return l == 0.0f ? neg_inf() : __fmaf_rn(m, LN2, logf(l));
}

// P_ij from the row's LSE in base 2; 0 in rows whose LSE is -inf
__device__ __forceinline__ float mod_prob(float y, float lse2) {
  return lse2 == neg_inf() || y == neg_inf() ? 0.0f : ex2_full(y - lse2);
}

// dq of one row over its visible keys, and its D: do . o with o as it was rounded, corrected by r = sum P (dP - D) as
// the tensor-core kernel does (dq by -r sum P (1 - t^2) k).  A row without visible keys has D = 0, whatever do holds.
template <typename T, int D>
__device__ void mod_exact_dq_row(const ModArgs& a, const T* qrow, const T* dorow, const T* orow, const T* kh,
                                 const T* vh, const int32_t* kdoc, const ModView& v, float slope2, float lse2,
                                 float (&dq)[D / 32], float& delta) {
  constexpr int N = D / 32;
  float q[N], g[N], o[N], w[N], r = 0.0f;
  mod_row_load<T, D>(qrow, q);
  mod_row_load<T, D>(dorow, g);
  mod_row_load<T, D>(orow, o);
#pragma unroll
  for (int i = 0; i < N; ++i) dq[i] = w[i] = 0.0f;
  delta = 0.0f;
  if (v.lim <= 0 || lse2 == neg_inf()) return;
  delta = mod_dot(g, o);
  for (int64_t j = 0; j < v.lim; ++j) {
    if (kdoc != nullptr && kdoc[j] != v.doc) continue;
    float k[N], vr[N];
    mod_row_load<T, D>(kh + j * a.ks[2], k);
    mod_row_load<T, D>(vh + j * a.vs[2], vr);
    float deriv;
    float y = mod_score(a, mod_dot(q, k), deriv);
    if (slope2 != 0.0f) y += mod_bias(slope2, v.pos, j);
    const float p = mod_prob(y, lse2);
    const float dp = mod_dot(g, vr);
    if (p == 0.0f) continue;
    const float pv = p * (dp - delta), ds = pv * deriv, pw = p * deriv;
    r += pv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dq[i] = __fmaf_rn(ds, k[i], dq[i]);
      w[i] = __fmaf_rn(pw, k[i], w[i]);
    }
    if (ds != ds) break;  // NaN in all of dq, and in r
  }
#pragma unroll
  for (int i = 0; i < N; ++i) dq[i] = __fmaf_rn(-r, w[i], dq[i]);
  delta += r;
}

// dk and dv of key j of one query head, added to what the arrays hold, with the rows' D (delta); ends where all of them are NaN (as they
// are once a NaN row sees the key: nothing after it changes them)
template <typename T, int D>
__device__ void mod_exact_dkv_head(const ModArgs& a, const T* qh, const T* doh, const float* delta, const float* lse,
                                   const int64_t (&dos)[3], int b, int64_t j, int kdoc, float slope2,
                                   const float (&k)[D / 32], const float (&vr)[D / 32], float (&dk)[D / 32],
                                   float (&dv)[D / 32]) {
  constexpr int N = D / 32;
  for (int64_t i = 0; i < a.sq; ++i) {
    const ModView v = mod_view(a, b, i);
    if (j >= v.lim || v.doc != kdoc) continue;
    float q[N], g[N];
    mod_row_load<T, D>(qh + i * a.qs[2], q);
    mod_row_load<T, D>(doh + i * dos[2], g);
    float deriv;
    float y = mod_score(a, mod_dot(q, k), deriv);
    if (slope2 != 0.0f) y += mod_bias(slope2, v.pos, j);
    const float p = mod_prob(y, lse[i] * L2E_HI);
    const float ds = p == 0.0f ? 0.0f : p * (mod_dot(g, vr) - delta[i]) * deriv;
#pragma unroll
    for (int x = 0; x < N; ++x) {
      if (p != 0.0f) {
        dk[x] = __fmaf_rn(ds, q[x], dk[x]);
        dv[x] = __fmaf_rn(p, g[x], dv[x]);
      }
    }
    bool lost = true;
#pragma unroll
    for (int x = 0; x < N; ++x) lost = lost && dk[x] != dk[x] && dv[x] != dv[x];
    if (__all_sync(0xffffffffu, lost)) return;
  }
}

}  // namespace smx
