// Attention with modified scores: arguments, visibility and score arithmetic
// that its kernels share (capped scores, a bias that falls with the distance;
// causal, prefix, document and length masks; grouped heads; strided tensors).
// The running state is that of "Online stable softmax" ("Carry a weighted
// value numerator for attention").
//
// Scores are held in base-2 units: y = log2(e) s, so that a probability is one
// exp2.  Visible keys of a row are j < lim (causal limit, prefix and length
// folded into one bound) whose document is the row's.
#pragma once

#include "kernel_attention.cuh"
#include "smx_mod.h"

namespace smx {

// A call's kernels are launched with programmatic stream serialization: one may start while
// its predecessor drains (a shared prefix of 300 keys: 16.5 us without, 12.4 with; mod_trigger, at a kernel's start: its successor's CTAs take what room there is once
// all of its own run), and waits for the predecessor's end and its writes in mod_wait.  Every kernel calls
// mod_wait before it ends, so that an end is the end of all before it.
__device__ __forceinline__ void mod_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void mod_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A row's view of its keys.
struct ModView {
  int64_t pos;  // the query's position among the keys
  int64_t lim;  // keys j < lim may be visible
  int doc;      // its document (0 where there are none)
};

__device__ __forceinline__ int64_t mod_klen(const ModArgs& a, int b) {
  int64_t n = a.sk;
  if (a.k_len != nullptr) {
    const int64_t v = a.k_len[b];
    n = v < 0 ? 0 : (v < a.sk ? v : a.sk);
  }
  return n;
}
__device__ __forceinline__ int64_t mod_start(const ModArgs& a, int b) {
  if (a.at_end) return mod_klen(a, b) - a.sq;
  return a.q_start != nullptr ? (int64_t)a.q_start[b] : a.sk - a.sq;
}
// lim without the document: the keys that row i may see
__device__ __forceinline__ int64_t mod_limit(const ModArgs& a, int64_t pos, int64_t prefix, int64_t klen) {
  if (!a.causal) return klen;
  int64_t lim = pos + 1 > prefix ? pos + 1 : prefix;
  lim = lim < klen ? lim : klen;
  return lim > 0 ? lim : 0;
}
__device__ __forceinline__ int64_t mod_prefix(const ModArgs& a, int b) {
  return a.prefix_len != nullptr ? (int64_t)a.prefix_len[b] : 0;
}
__device__ __forceinline__ ModView mod_view(const ModArgs& a, int b, int64_t i) {
  ModView v;
  v.pos = mod_start(a, b) + i;
  v.lim = mod_limit(a, v.pos, mod_prefix(a, b), mod_klen(a, b));
  v.doc = 0;
  if (a.q_doc != nullptr) {
    v.doc = a.q_doc[(int64_t)b * a.sq + i];
    if (v.doc < 0) v.lim = 0;
  }
  return v;
}

// The capped score in base-2 units and its derivative factor 1 - t^2, from the
// raw product: t = tanh(acc c), c = scale / softcap.  tanhf keeps its relative
// accuracy where c acc is small, so the cap does not blur small scores.
__device__ __forceinline__ float mod_score(const ModArgs& a, float acc, float& deriv) {
  if (a.cap2 > 0.0f) {
    const float t = tanhf(acc * a.c);
    deriv = __fmaf_rn(-t, t, 1.0f);
    return a.cap2 * t;
  }
  deriv = 1.0f;
  return acc * a.c;
}

__device__ __forceinline__ float mod_bias(float slope2, int64_t pos, int64_t j) {
  const int64_t far = pos > j ? pos - j : j - pos;
  return -slope2 * (float)far;
}

// Which of N members of a block (of 64) share `doc`, out of `seen` (bit masks).  A warp
// collective: members are compared one by one only where the block holds several documents, or
// places without any, and some lane needs it.
template <int N = 64>
__device__ __forceinline__ uint64_t mod_doc_seen(uint64_t seen, int doc, int4 block, const int32_t* members) {
  if (doc < block.x || doc > block.y) seen = 0;
  const bool one_by_one = seen != 0 && (block.x != block.y || block.z != 0);
  if (__any_sync(0xffffffffu, one_by_one)) {
    uint64_t same = 0;
#pragma unroll 4
    for (int x = 0; x < N; x += 4) {
      const int4 d = *reinterpret_cast<const int4*>(members + x);
      same |= (uint64_t)((d.x == doc ? 1u : 0u) | (d.y == doc ? 2u : 0u) | (d.z == doc ? 4u : 0u) |
                         (d.w == doc ? 8u : 0u))
              << x;
    }
    if (one_by_one) seen &= same;
  }
  return seen;
}

// tanh(u) / u as polynomials in u^2 (least maximum relative error, fitted by weighted Chebyshev
// least squares): NEAR on |u| <= 0.375 (degree 3, the coefficients as written: 6e-8; 1.5e-7 in 32-bit arithmetic), else
// |u| <= 1 (degree 6: 1.8e-7; 2.7e-7 in 32-bit arithmetic, 4.6 times 2^-24).  Scores that a cap leaves nearly alone are
// the usual case; where some of a block pass |u| = 1 its exponentials and reciprocals make a forward 1.6 times as long
// (2 x 32 x 4096 x 128: 632 us within, 1010 beyond).
constexpr float TANH_NEAR = 0.375f;
template <bool NEAR>
struct TanhPoly;
template <>
struct TanhPoly<true> {
  static constexpr int N = 4;
  __device__ static constexpr float c(int i) {
    constexpr float v[4] = {0.9999999405367f, -0.3333197482105f, 0.1328450214143f, -0.0482722621716f};
    return v[i];
  }
};
template <>
struct TanhPoly<false> {
  static constexpr int N = 7;
  __device__ static constexpr float c(int i) {
    constexpr float v[7] = {0.9999999403954f, -0.3333283960819f, 0.1332520395517f, -0.0534570291638f,
                            0.0202899798751f, -0.0062033785507f, 0.0010410224785f};
    return v[i];
  }
};
// scale tanh over the whole range, 1 - 2 / (1 + e^(2u)): absolute error within 2^-22 scale
__device__ __forceinline__ float tanh_exp(float u, float scale = 1.0f) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_full(u * 2.8853900817779268f)));
  return __fmaf_rn(-2.0f * scale, r, scale);
}
// scale tanh(u) / u of a pair (the scale rides on the coefficients)
template <bool NEAR>
__device__ __forceinline__ unsigned long long tanh_ratio2(unsigned long long u, float scale) {
  using P = TanhPoly<NEAR>;
  const unsigned long long w = mul2(u, u);
  float c = P::c(P::N - 1) * scale;
  unsigned long long r = pk(c, c);
#pragma unroll
  for (int i = P::N - 2; i >= 0; --i) {
    c = P::c(i) * scale;
    r = fma2(r, w, pk(c, c));
  }
  return r;
}
__device__ __forceinline__ float tanh_score(float u) {
  return fabsf(u) <= 1.0f ? u * pk_lo(tanh_ratio2<false>(pk(u, u), 1.0f)) : tanh_exp(u);
}
// the forms a block's cap may take: the smallest range that holds all its arguments
enum : int { CAP_NEAR = 0, CAP_POLY = 1, CAP_EXP = 2 };

}  // namespace smx
