// Backward of the attention with modified scores on the 5th-generation tensor
// cores ("Softmax numerics architecture...", "The Jacobian, and the backward
// pass that never divides"): P is formed again from the scores and the row's LSE, then
//   dS = P (dP - D) (1 - t^2),  dP = do V^T,  D = do . o,
// and dq = scale dS K, dk = scale dS^T q, dv = P^T do.
//
// Two kernels of one shape (k_mod_backward, MODE): each CTA keeps 128 rows of one side
// as the lanes of tensor memory and streams the other side in blocks of 64
// columns, so every sum stays in one CTA's accumulators, in a fixed order, and
// nothing is added through memory:
//   MODE_DQ   lanes = queries, columns = keys:  X1 += P K,  X2 += dS K
//   MODE_DKV  lanes = keys, columns = queries of every head of the group:
//             X1 += P^T do (dv),  X2 += dS^T q (dk)
// Each block takes four products: S = A1 C1^T and dP = A2 C2^T (128 x 64 x D) from shared memory,
// X1 and X2 (128 x D x 64) with their A operand (P or dS in the input type) in tensor memory over
// the scores it came from.  Two groups of 256 row threads (two a lane, 32 columns each) take the blocks
// in turn, each with its own S and dP tile: while one turns scores into P, the other turns dP into dS, and
// the products run beside both, issued by two warps: X1(i), S(i+2) by one, X2(i), dP(i+2) by the other (a
// wait that is already satisfied costs an issuing warp some 130 cycles; one warp for all four left the tensor
// cores idle half of the time).  (One group on blocks of 128
// columns, its chain of load, exponentials, store and product in lockstep with the products, took 3400 cycles for
// 128 columns at D = 128 and nearly as many at D = 64, whether two or four threads shared a lane.)
//
// D: do . o uses o as it was rounded, which is what is left of the error of rows
// that attend to few keys (measured on such rows: 1.5 times the error of the result's own
// rounding).  MODE_DQ therefore sums r = sum_j P (dP - D~) = D - D~ in fp32, corrects its
// result by -r sum_j P k_j (X1, one product more) and leaves D~ + r for MODE_DKV, which runs after it.  (Hence o
// and the LSE have to be the forward's over these very keys: sum_j P = 1.)
//
// A lane whose result is not finite is computed again from the pairs that are visible
// (kernel_mod_exact.cuh).  Bound: at D = 128 the products, four a block (1280 tensor cycles, the 64-column ones at two
// thirds of the full rate; S and dP are formed in both kernels, and MODE_DQ's X1 is the correction's) beside the row
// threads (capped: tensor pipe busy 49 to 54 % of the time, issue slots 57, exp2 unit 14); at D = 64 the row threads
// (documents and bias: tensor pipe 24 %, issue slots 44).  16 heads x 8192 rows, causal, calls back to back: 699 us at
// D = 128 (983 TFLOP/s of the five products of the formulas), 619 us at D = 64; every key 1430 us;
// capped causal 885 (1000 where scores reach the cap), slopes 729; documents of 900 rows 201.
#pragma once

#include "kernel_mod_exact.cuh"
#include "kernel_mod_forward.cuh"

namespace smx {

enum : int { MODE_DQ = 0, MODE_DKV = 1 };

struct ModBwdKernelArgs {
  ModBwdArgs m;
  const float* lse2;     // [batch x hq][sq_pad] base-2 LSE; +inf where a row sees nothing
  float* delta;          // [batch x hq][sq_pad] D
  int64_t sq_pad;        // a multiple of 128
  int lane_tiles;        // 128-row tiles of the lanes' side
  const int2* range;     // documents: [batch][lane tiles] first and end block of 64 columns; or null
  const int4* cblock;    // documents: [batch][ncb] summaries of 64 columns (kernel_mod_docs.cuh)
  const int32_t* cdoc;   // documents: [batch][64 ncb] of the columns, -1 past the end
  int ncb;
  // few lane tiles: the columns of each in parts, whose X1, X2 and r are added up in order afterwards
  int parts;
  float* px1;          // [parts][batch x heads x lanes][D], or null (parts == 1)
  float* px2;
  float* pr;           // [parts][batch x heads x lanes]
  int* status;
  int64_t max_polls;
  int64_t probe_polls;
};

constexpr int MBW_ROWS = 512;                // row threads: two groups of two a lane
constexpr int MBW_GROUP = 256;
constexpr int MBW_MMA_WARP = 16, MBW_LOAD_WARP = 18;  // two issuing warps: S and X1, dP and X2
constexpr int MBW_THREADS = 608;
constexpr int MBW_NB = 64;                   // columns a block
constexpr int MBW_NST = 4;                   // stages: blocks i - 1 .. i + 2 are in use
constexpr int MBW_NBAR = 24;
template <int D>
struct MbwShape {
  static constexpr int TILE = 128 * D * 2;           // a tile of the lanes' side
  static constexpr int CT = MBW_NB * D * 2;          // a tile of the columns' side
  static constexpr int STAGE = 2 * CT;               // C1, C2
  static constexpr int STATS = MBW_NST * 2 * 256;    // (lse2, D) of a stage's 64 columns
  static constexpr int XCHG = 4 * 128 * 4 + 128 * 4;  // r of a lane's four threads, bad lanes
  static constexpr int SMEM = 1024 + 2 * TILE + MBW_NST * STAGE + STATS + XCHG + MBW_NBAR * 8 + 16;
};

// What a row thread knows of its lane and of the block's columns.
struct MbwCols {
  uint32_t seen;          // visible columns of its 32
  float d0;               // distance at column 0; falls (MODE_DQ) or rises by 1 a column
  float slope2;
  float lse2;             // MODE_DQ: the lane's
  uint32_t stats;         // MODE_DKV: shared address of the 32 columns' lse2
};

// P of the thread's 32 columns from the raw products y: p, and packed in the input type pk2.  With a cap p holds
// P (1 - t^2), all that dS needs; MODE_DQ's r = sum P (dP - D) takes the rest of P beside it: t2 keeps P t^2 2^14 as fp16
// pairs (in 32 bits they would take 16 registers more, which spill).  Off by 2^-11 of P t^2 and, scaled, never
// subnormal where it matters, they blur the correction of D alone, by 2^-11 sum P t^2 |dP - D|.  (dS itself takes no
// rounding but its own: with 1 - t^2 in fp16 it was off by sqrt 2 as much in fp16, with t^2 in fp16 by up to 149 times
// its bound where scores reach the cap.)
constexpr float MBW_T = 128.0f;  // MODE_DQ holds t times this, t^2 times its square
template <typename T, int MODE, bool CAP, bool BIAS, int FORM, bool BORDER, int LINE>
__device__ __forceinline__ void mbw_probs(float (&p)[32], const ModArgs& a, const MbwCols& q,
                                          uint32_t (&t2)[CAP && MODE == MODE_DQ ? 16 : 1], uint32_t (&pk2)[16]) {
  // LINE: 1 the distance falls (MODE_DQ) or rises along the columns, 0 it turns within them
  const float step = MODE == MODE_DQ ? -1.0f : 1.0f;
  const float st = -q.slope2 * step, base = -q.slope2 * q.d0;
  constexpr float TS = CAP && MODE == MODE_DQ ? MBW_T : 1.0f;
  const float k = a.cap2 * (1.0f / TS);
  const unsigned long long c2 = pk(a.c, a.c), k2 = pk(k, k), st2 = pk(2.0f * st, 2.0f * st);
  const unsigned long long nl = pk(-q.lse2, -q.lse2);
  unsigned long long line = 0;  // stepped, anew every 8 columns
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    unsigned long long sub = nl;
    if constexpr (MODE == MODE_DKV) {
      float l0, l1;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(l0), "=f"(l1) : "r"(q.stats + 4 * x));
      sub = pk(-l0, -l1);
    }
    const bool v0 = !BORDER || ((q.seen >> x) & 1u), v1 = !BORDER || ((q.seen >> (x + 1)) & 1u);
    unsigned long long e, tt = 0;
    if constexpr (CAP) {
      unsigned long long t;
      const unsigned long long u = mul2(pk(v0 ? p[x] : 0.0f, v1 ? p[x + 1] : 0.0f), c2);
      if constexpr (FORM == CAP_EXP)
        t = pk(tanh_exp(pk_lo(u), TS), tanh_exp(pk_hi(u), TS));
      else
        t = mul2(tanh_ratio2<FORM == CAP_NEAR>(u, TS), u);
      tt = mul2(t, t);
      e = fma2(t, k2, sub);
    } else {
      e = fma2(pk(p[x], p[x + 1]), c2, sub);
    }
    if constexpr (BIAS) {
      if constexpr (LINE != 0) {
        line = x % 8 == 0 ? pk(__fmaf_rn((float)x, st, base), __fmaf_rn((float)(x + 1), st, base)) : add2(line, st2);
        e = add2(e, line);
      } else {
        const float f0 = fabsf(q.d0 + step * (float)x), f1 = fabsf(q.d0 + step * (float)(x + 1));
        e = pk(__fmaf_rn(-q.slope2, f0, pk_lo(e)), __fmaf_rn(-q.slope2, f1, pk_hi(e)));
      }
    }
    float p0 = ex2_ftz(pk_lo(e)), p1 = ex2_ftz(pk_hi(e));
    if constexpr (BORDER) {
      p0 = v0 ? p0 : 0.0f;
      p1 = v1 ? p1 : 0.0f;
    }
    p[x] = p0;
    p[x + 1] = p1;
    if constexpr (!CAP) {
      pk2[x / 2] = pack2<T>(p0, p1);
    } else {
      constexpr float one = 1.0f / (TS * TS);
      const unsigned long long pp = pk(p0, p1), pd = mul2(pp, fma2(tt, pk(-one, -one), pk(1.0f, 1.0f)));
      p[x] = pk_lo(pd);
      p[x + 1] = pk_hi(pd);
      if constexpr (MODE == MODE_DKV) {
        pk2[x / 2] = pack2<T>(p0, p1);
      } else {
        // X1 takes P (1 - t^2): the correction it serves is one of dS
        pk2[x / 2] = pack2<T>(p[x], p[x + 1]);
        const unsigned long long rest = mul2(pp, tt);
        t2[x / 2] = pack2<__half>(pk_lo(rest), pk_hi(rest));
      }
    }
  }
}

template <typename T, int MODE, bool CAP, bool BIAS, int FORM, bool BORDER>
__device__ __forceinline__ void mbw_probs_line(float (&p)[32], const ModArgs& a, const MbwCols& q, int line,
                                               uint32_t (&t2)[CAP && MODE == MODE_DQ ? 16 : 1], uint32_t (&pk2)[16]) {
  if constexpr (!BIAS) {
    mbw_probs<T, MODE, CAP, BIAS, FORM, BORDER, 0>(p, a, q, t2, pk2);
  } else {
    // (a line that rises against the usual direction takes the general form)
    if (__builtin_expect(line > 0, 1))
      mbw_probs<T, MODE, CAP, BIAS, FORM, BORDER, 1>(p, a, q, t2, pk2);
    else
      mbw_probs<T, MODE, CAP, BIAS, FORM, BORDER, 0>(p, a, q, t2, pk2);
  }
}

// Scores to P, over the first 16 of the score columns they came from
template <typename T, int MODE, bool CAP, bool BIAS>
__device__ __forceinline__ void mbw_phase1(uint32_t ts, const ModArgs& a, const MbwCols& q, bool border, int line,
                                           float (&p)[32], uint32_t (&t2)[CAP && MODE == MODE_DQ ? 16 : 1]) {
  tc_ld32(ts, p);
  int form = CAP_EXP;
  if constexpr (CAP) {
    // the smallest range that holds the warp's arguments (what is hidden counts too: at worst a wider one is taken)
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) far = max3(far, fabsf(p[i]), fabsf(p[i + 1]));
    far *= a.c;
    form = __all_sync(0xffffffffu, far <= TANH_NEAR) ? CAP_NEAR : (__all_sync(0xffffffffu, far <= 1.0f) ? CAP_POLY : CAP_EXP);
  }
  uint32_t pk2[16];
  if (__builtin_expect(!border && (!CAP || form == CAP_NEAR), 1)) {
    mbw_probs_line<T, MODE, CAP, BIAS, CAP_NEAR, false>(p, a, q, line, t2, pk2);
  } else if (border) {
    if (CAP && form != CAP_EXP)
      mbw_probs_line<T, MODE, CAP, BIAS, CAP_POLY, true>(p, a, q, line, t2, pk2);
    else
      mbw_probs_line<T, MODE, CAP, BIAS, CAP_EXP, true>(p, a, q, line, t2, pk2);
  } else if (CAP && form == CAP_POLY) {
    mbw_probs_line<T, MODE, CAP, BIAS, CAP_POLY, false>(p, a, q, line, t2, pk2);
  } else if (CAP) {
    mbw_probs_line<T, MODE, CAP, BIAS, CAP_EXP, false>(p, a, q, line, t2, pk2);
  }
  tc_st16u(ts, pk2);
}

// dS = P (1 - t^2) (dP - D) over the first 16 columns of the dP it came from; MODE_DQ: r += P (dP - D)
template <typename T, int MODE, bool CAP>
__device__ __forceinline__ void mbw_phase2(uint32_t tdp, float delta, uint32_t stats, const float (&p)[32],
                                           const uint32_t (&t2)[CAP && MODE == MODE_DQ ? 16 : 1], float& r) {
  const unsigned long long nd = pk(-delta, -delta);
  unsigned long long acc[2] = {0ull, 0ull};
  float dp[32];
  uint32_t ds[16];
  tc_ld32(tdp, dp);
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    unsigned long long sub = nd;
    if constexpr (MODE == MODE_DKV) {
      float l0, l1;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(l0), "=f"(l1) : "r"(stats + 4 * x));
      sub = pk(-l0, -l1);
    }
    const unsigned long long v = add2(pk(dp[x], dp[x + 1]), sub), d = mul2(pk(p[x], p[x + 1]), v);
    if constexpr (CAP && MODE == MODE_DQ) {
      const float2 rest = __half22float2(*reinterpret_cast<const __half2*>(&t2[x / 2]));
      acc[0] = add2(acc[0], d);
      acc[1] = fma2(pk(rest.x, rest.y), v, acc[1]);
    } else if constexpr (MODE == MODE_DQ) {
      acc[(x >> 1) & 1] = fma2(pk(p[x], p[x + 1]), v, acc[(x >> 1) & 1]);
    }
    ds[x / 2] = pack2<T>(pk_lo(d), pk_hi(d));
  }
  tc_st16u(tdp, ds);
  if constexpr (MODE == MODE_DQ)
    r += __fmaf_rn(CAP ? 1.0f / (MBW_T * MBW_T) : 1.0f, pk_lo(acc[1]) + pk_hi(acc[1]), pk_lo(acc[0]) + pk_hi(acc[0]));
}

// 64 bytes (pkd) of each of a warp's 32 rows through its 2 KB of shared memory, so that the stores go out
// in 64-byte pieces of eight rows (row's base offset in `off`, < 0: not stored; c: the first column)
template <typename T>
__device__ __forceinline__ void mbw_store64b(uint32_t stg, const uint32_t (&pkd)[16], T* out, int64_t off, int c) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t addr = stg + (uint32_t)(lane * 64 + ((x ^ ((lane >> 1) & 3)) * 16));
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(pkd[4 * x]), "r"(pkd[4 * x + 1]),
                 "r"(pkd[4 * x + 2]), "r"(pkd[4 * x + 3])
                 : "memory");
  }
  __syncwarp();
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int rr = 8 * x + (lane >> 2), qq = lane & 3;
    const uint32_t addr = stg + (uint32_t)(rr * 64 + ((qq ^ ((rr >> 1) & 3)) * 16));
    uint4 val;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(val.x), "=r"(val.y), "=r"(val.z), "=r"(val.w)
                 : "r"(addr)
                 : "memory");
    const int64_t to = __shfl_sync(0xffffffffu, off, rr);
    if (to >= 0) *reinterpret_cast<uint4*>(out + to + c + qq * (16 / (int)sizeof(T))) = val;
  }
  __syncwarp();
}
// 32 columns in the output type, or as fp32 in two pieces
template <typename T>
__device__ __forceinline__ void mbw_store32(uint32_t stg, const float (&x)[32], T* out, int64_t off, int c) {
  uint32_t pkd[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) pkd[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  mbw_store64b(stg, pkd, out, off, c);
}
__device__ __forceinline__ void mbw_store32_f32(uint32_t stg, const float (&x)[32], float* out, int64_t off, int c) {
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
    uint32_t pkd[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) pkd[i] = __float_as_uint(x[h + i]);
    mbw_store64b(stg, pkd, out, off, c + h);
  }
}

// One lane again from its visible pairs, by a whole warp.
template <typename T, int D, int MODE>
__device__ __noinline__ void mbw_exact(const ModBwdKernelArgs& f, int b, int h, int64_t at, const T* q, const T* k,
                                       const T* v, const T* o, const float* lse, const T* d_o, T* out1, T* out2) {
  const ModArgs& a = f.m.a;
  constexpr int N = D / 32;
  if constexpr (MODE == MODE_DQ) {
    const int u = h / a.group;
    float acc[N], delta;
    mod_exact_dq_row<T, D>(a, q + b * a.qs[0] + h * a.qs[1] + at * a.qs[2],
                           d_o + b * f.m.dos[0] + h * f.m.dos[1] + at * f.m.dos[2],
                           o + b * a.os[0] + h * a.os[1] + at * a.os[2], k + b * a.ks[0] + u * a.ks[1],
                           v + b * a.vs[0] + u * a.vs[1], a.k_doc != nullptr ? a.k_doc + (int64_t)b * a.sk : nullptr,
                           mod_view(a, b, at), a.slopes != nullptr ? a.slopes[h] * L2E_HI : 0.0f,
                           lse[((int64_t)b * a.hq + h) * a.sq + at] * L2E_HI, acc, delta);
    // (the D that MODE_DKV reads: one NaN there would send all keys of its block here too)
    if ((threadIdx.x & 31) == 0) f.delta[((int64_t)b * a.hq + h) * f.sq_pad + at] = delta;
#pragma unroll
    for (int x = 0; x < N; ++x) acc[x] *= f.m.scale;
    mod_row_store<T, D>(out1 + b * f.m.dqs[0] + h * f.m.dqs[1] + at * f.m.dqs[2], acc);
  } else {
    const int u = h;
    float kr[N], vr[N], gk[N], gv[N];
    mod_row_load<T, D>(k + b * a.ks[0] + u * a.ks[1] + at * a.ks[2], kr);
    mod_row_load<T, D>(v + b * a.vs[0] + u * a.vs[1] + at * a.vs[2], vr);
#pragma unroll
    for (int x = 0; x < N; ++x) gk[x] = gv[x] = 0.0f;
    const int kdoc = a.k_doc != nullptr ? a.k_doc[(int64_t)b * a.sk + at] : 0;
    if (kdoc >= 0 && at < mod_klen(a, b))
      for (int hh = u * a.group; hh < (u + 1) * a.group; ++hh)
        mod_exact_dkv_head<T, D>(a, q + b * a.qs[0] + hh * a.qs[1], d_o + b * f.m.dos[0] + hh * f.m.dos[1],
                                 f.delta + ((int64_t)b * a.hq + hh) * f.sq_pad, lse + ((int64_t)b * a.hq + hh) * a.sq,
                                 f.m.dos, b, at,
                                 kdoc, a.slopes != nullptr ? a.slopes[hh] * L2E_HI : 0.0f, kr, vr, gk, gv);
#pragma unroll
    for (int x = 0; x < N; ++x) gk[x] *= f.m.scale;
    mod_row_store<T, D>(out2 + b * f.m.dks[0] + u * f.m.dks[1] + at * f.m.dks[2], gk);
    mod_row_store<T, D>(out1 + b * f.m.dvs[0] + u * f.m.dvs[1] + at * f.m.dvs[2], gv);
  }
}

// tm_a1, tm_a2: the lanes' side (q, do or k, v); tm_c1, tm_c2: the columns' (k, v or q, do).
// out1: dq (MODE_DQ) or dv; out2: dk.
template <typename T, int D, int MODE, bool CAP, bool BIAS>
__global__ void __launch_bounds__(MBW_THREADS, 1)
    k_mod_backward(const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                   const __grid_constant__ CUtensorMap tm_c1, const __grid_constant__ CUtensorMap tm_c2,
                   const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                   const T* __restrict__ o, const float* __restrict__ lse, const T* __restrict__ d_o, T* out1, T* out2,
                   const __grid_constant__ ModBwdKernelArgs f) {
  using S = MbwShape<D>;
  constexpr int NB = MBW_NB, NST = MBW_NST, TILE = S::TILE, CT = S::CT;
  // barriers: the lanes' tiles; C1 and C2 full, stage free, by stage; S, dP ready, by group; probe, end;
  // P and dS written, by group (a warp's arrival each).  Every hand-over is an mbarrier, whose waits are
  // bounded: after a wait ran out the sides may be out of step, and a named barrier would then never open
  constexpr int B_A = 0, B_C1 = 1, B_C2 = 5, B_FREE = 9, B_S = 13, B_DP = 15, B_PROBE = 17, B_END = 18, B_P = 19,
                B_DS = 21;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const ModArgs& a = f.m.a;
  // (a warp's number and the tensor memory's address by shuffle: values and branches that the compiler
  // knows to be the same in the whole warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t raw = tc_su32(smem_raw);
  const uint32_t pad = (1024 - (raw & 1023)) & 1023;
  uint8_t* base = smem_raw + pad;
  const uint32_t sA1 = tc_su32(base), sA2 = sA1 + TILE, sC = sA2 + TILE;  // stage s: C1 at sC + s STAGE, C2 behind
  const uint32_t sStats = sC + NST * S::STAGE;                            // stage s: lse2, D of 64 columns
  float* xchg = reinterpret_cast<float*>(base + 2 * TILE + NST * S::STAGE + S::STATS);
  int* flags = reinterpret_cast<int*>(xchg + 512);
  uint64_t* bars = reinterpret_cast<uint64_t*>(flags + 128);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + MBW_NBAR);
  const uint32_t bar0 = tc_su32(bars);
  auto bar = [bar0](int i) { return bar0 + 8u * (uint32_t)i; };

  mod_trigger();
  mod_wait();
  // this CTA's lanes: tile lt of (batch b, head); under a causal mask the longest tiles
  // come first (late queries, early keys)
  const int heads = MODE == MODE_DQ ? a.hq : a.hkv;
  const int part = (int)(blockIdx.x % (unsigned)f.parts);
  const unsigned unit = blockIdx.x / (unsigned)f.parts;
  const int bh = (int)(unit % (unsigned)(a.batch * heads)), order = (int)(unit / (unsigned)(a.batch * heads));
  const int lt = MODE == MODE_DQ && a.causal ? f.lane_tiles - 1 - order : order;
  const int b = bh / heads, head = bh - b * heads;
  const int u = MODE == MODE_DQ ? head / a.group : head;
  const int64_t l0 = (int64_t)lt * 128, lanes = MODE == MODE_DQ ? a.sq : a.sk;
  const int64_t start = mod_start(a, b), prefix = mod_prefix(a, b), klen = mod_klen(a, b);
  // blocks of 64 columns [c_lo, c_hi), the same for each head of the group
  int c_lo = 0, c_hi = 0;
  if (f.range != nullptr) {
    const int2 rg = f.range[(int64_t)b * f.lane_tiles + lt];
    c_lo = rg.x;
    c_hi = rg.y;
  } else if constexpr (MODE == MODE_DQ) {
    const int64_t last = l0 + 127 < a.sq - 1 ? l0 + 127 : a.sq - 1;
    c_hi = (int)((mod_limit(a, start + last, prefix, klen) + NB - 1) / NB);
  } else {
    // queries i >= l0 - start see the tile's first key (every query where it lies in the prefix)
    int64_t first = a.causal && l0 >= prefix ? l0 - start : 0;
    if (first < 0) first = 0;
    if (l0 < klen && first < a.sq) {
      c_lo = (int)(first / NB);
      c_hi = (int)((a.sq + NB - 1) / NB);
    }
  }
  const int per = c_hi - c_lo, ng = MODE == MODE_DQ ? 1 : a.group;
  // this part's blocks: n of them from first on
  const int share = (per * ng + f.parts - 1) / f.parts, first = part * share;
  const int n = __shfl_sync(0xffffffffu, per * ng - first < share ? (per * ng > first ? per * ng - first : 0) : share, 0);

  if (warp == MBW_MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_su32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < MBW_NBAR; ++i) mbar_init(bar(i), i >= B_P ? MBW_GROUP / 32 : ((i >= B_FREE && i < B_FREE + NST) || i == B_END ? 2 : 1));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 128) flags[tid] = 0;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // S and dP of group g at t_s + 64 g, t_dp + 64 g
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_x1 = tmem + 256, t_x2 = tmem + 256 + D;
  bool ok = true;
  auto wait_or_flag = [&](int i, uint32_t par) {
    if (!tc_wait(bar(i), par, f.max_polls, f.status)) {
      ok = false;
      atomicOr(f.status, DEV_TIMEOUT);
    }
  };
  if (f.probe_polls > 0 && tid == 0 && !tc_wait(bar(B_PROBE), 0u, f.probe_polls, f.status))
    atomicOr(f.status, DEV_TIMEOUT);

  if (warp == MBW_MMA_WARP || warp == MBW_MMA_WARP + 1) {
    // 0: S and X1; 1: dP and X2
    const int which = warp - MBW_MMA_WARP;
    const uint32_t id_s = tc_idesc<T>(128, NB), id_x = tc_idesc<T>(128, D, true);
    // one lane's products; the whole warp runs this code alike (tc_mma_one)
    const uint32_t one = tc_elect();
    // A C^T: D / 16 steps of K = 16, four a 64-element half
    auto issue_ab = [&](uint32_t td, uint32_t sa, uint32_t sc) {
      uint32_t da = tc_desc(sa), dc = tc_desc(sc);
#pragma unroll 1
      for (int h = 0; h < D / 64; ++h) {
#pragma unroll
        for (int st = 0; st < 4; ++st)
          tc_mma_one(one, td, da + (uint32_t)(2 * st), dc + (uint32_t)(2 * st), id_s, (uint32_t)(h + st));
        da += (128 * 128) >> 4;
        dc += (NB * 128) >> 4;
      }
    };
    auto stage = [&](int i) { return sC + (uint32_t)((i % NST) * S::STAGE); };
    const uint32_t sA = which ? sA2 : sA1, t_sc = which ? t_dp : t_s, tx = which ? t_x2 : t_x1;
    // S(i) or dP(i).  Keys behind the sequence weigh 0, but 0 x NaN is NaN: the columns' K and V rows there
    // become zero first.
    auto issue_scores = [&](int i) {
      const uint32_t tile = stage(i) + (uint32_t)(which * CT);
      if constexpr (MODE == MODE_DQ) {
        const int64_t j0 = (int64_t)(c_lo + first + i) * NB;
        if (__builtin_expect(j0 + NB > klen, 0)) {
          const int from = klen - j0 < 0 ? 0 : (int)(klen - j0);
          for (int x = lane; x < (NB - from) * (D / 8); x += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             tile + tc_off(from + x / (D / 8), (x % (D / 8)) * 8, NB)),
                         "r"(0)
                         : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
      }
      issue_ab(t_sc + (uint32_t)(64 * (i & 1)), sA, tile);
      tc_commit_one(one, bar((which ? B_DP : B_S) + (i & 1)));
    };
    if (n > 0) {
      wait_or_flag(B_A, 0u);
#pragma unroll 1
      for (int i = -2; i < n; ++i) {
        // block i + 2's C1 or C2 first: it is there long before the rows are done with block i
        if (i + 2 < n) wait_or_flag((which ? B_C2 : B_C1) + (i + 2) % NST, (uint32_t)(((i + 2) / NST) & 1));
        // X1 of MODE_DKV takes C2, which this warp's scores do not
        if (MODE == MODE_DKV && which == 0 && i >= 0) wait_or_flag(B_C2 + i % NST, (uint32_t)((i / NST) & 1));
        __syncwarp();
        if (i >= 0) {
          // P(i) or dS(i) is in tensor memory: X += it E, 4 steps of 16 columns (a thread's part starts at its
          // first score column); then the stage is free of this warp's products
          wait_or_flag((which ? B_DS : B_P) + (i & 1), (uint32_t)((i >> 1) & 1));
          __syncwarp();
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t tp = t_sc + (uint32_t)(64 * (i & 1));
          const uint32_t de = tc_desc_mn(stage(i) + (uint32_t)(MODE == MODE_DKV && !which ? CT : 0), (uint32_t)(NB * 128));
#pragma unroll
          for (int st = 0; st < NB / 16; ++st)
            tc_mma_ta_one(one, tx, tp + (uint32_t)((st >> 1) * 32 + (st & 1) * 8), de + (uint32_t)((st * 2048) >> 4), id_x,
                          (uint32_t)(i + st));
          tc_commit_one(one, bar(B_FREE + i % NST));
        }
        if (i + 2 < n) issue_scores(i + 2);
      }
      // every product has finished before the rows read X1, X2 (and before the
      // tensor memory is freed, also after a wait that ran out)
      tc_commit_one(one, bar(B_END));
      tc_wait_drain(bar(B_END), 0u);
      __syncwarp();
    }
  } else if (warp == MBW_LOAD_WARP) {
    if (lane == 0 && n > 0) {
      tma_prefetch_map(&tm_a1);
      tma_prefetch_map(&tm_a2);
      tma_prefetch_map(&tm_c1);
      tma_prefetch_map(&tm_c2);
      // the lanes' tiles in boxes of 64 rows
      auto load_a = [&](uint32_t dst, const CUtensorMap* map) {
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            tma_load_4d(dst + (uint32_t)(x * 128 * 128 + y * 64 * 128), map, x * 64, (int)l0 + 64 * y, head, b, bar(B_A));
      };
      int sent = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % NST;
        if (i >= NST && !tc_wait(bar(B_FREE + s), (uint32_t)((i / NST - 1) & 1), f.max_polls, f.status)) {
          ok = false;
          atomicOr(f.status, DEV_TIMEOUT);
          break;
        }
        const int g = (first + i) / per, ct = c_lo + first + i - g * per;
        const int ch = MODE == MODE_DQ ? u : u * a.group + g;
        const uint32_t c1 = sC + (uint32_t)(s * S::STAGE), st = sStats + (uint32_t)(s * 512);
        if (i == 0) {
          mbar_arrive_expect_tx(bar(B_A), (uint32_t)(2 * TILE));
          load_a(sA1, &tm_a1);
        }
        mbar_arrive_expect_tx(bar(B_C1 + s), (uint32_t)(CT + (MODE == MODE_DKV ? 512 : 0)));
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_4d(c1 + (uint32_t)(x * NB * 128), &tm_c1, x * 64, ct * NB, ch, b, bar(B_C1 + s));
        if constexpr (MODE == MODE_DKV) {
          const int64_t at = ((int64_t)b * a.hq + ch) * f.sq_pad + (int64_t)ct * NB;
          bulk_load_g2s(st, f.lse2 + at, 256u, bar(B_C1 + s));
          bulk_load_g2s(st + 256, f.delta + at, 256u, bar(B_C1 + s));
        }
        if (i == 0) load_a(sA2, &tm_a2);
        mbar_arrive_expect_tx(bar(B_C2 + s), (uint32_t)CT);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_4d(c1 + (uint32_t)(CT + x * NB * 128), &tm_c2, x * 64, ct * NB, ch, b, bar(B_C2 + s));
        sent = i + 1;
      }
      // every copy has landed before the CTA ends (already so on the normal path)
      for (int s = 0; s < NST && s < sent; ++s) {
        const int last = s + ((sent - 1 - s) / NST) * NST;
        tc_wait_drain(bar(B_C1 + s), (uint32_t)((last / NST) & 1));
        tc_wait_drain(bar(B_C2 + s), (uint32_t)((last / NST) & 1));
      }
      tc_wait_drain(bar(B_A), 0u);
    }
    __syncwarp();
  } else {
    // row threads: lane rt, blocks of group grp, columns 32 side ..
    const int grp = warp >> 3, side = (warp >> 2) & 1, rt = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = t_s + lane_off + (uint32_t)(64 * grp + 32 * side),
                   tdp = t_dp + lane_off + (uint32_t)(64 * grp + 32 * side);
    const int64_t at = l0 + rt;
    const bool in = at < lanes;
    const int64_t ac = in ? at : lanes - 1;
    // the lane's own constants: its limit among the columns and its document
    int lim = 0, doc = 0;      // MODE_DQ: keys below lim; MODE_DKV: queries from lim on
    int64_t pos = 0;
    float lse2 = 0.0f, delta = 0.0f, r = 0.0f;
    const int64_t row = ((int64_t)b * a.hq + head) * f.sq_pad + ac;
    if constexpr (MODE == MODE_DQ) {
      const ModView view = mod_view(a, b, ac);
      pos = view.pos;
      lim = in ? (int)view.lim : 0;
      doc = view.doc;
      lse2 = f.lse2[row];
      delta = f.delta[row];
    } else {
      doc = a.k_doc != nullptr ? a.k_doc[(int64_t)b * a.sk + ac] : 0;
      int64_t from = a.causal && ac >= prefix ? ac - start : 0;
      if (from < 0) from = 0;
      lim = in && ac < klen && doc >= 0 && from < a.sq ? (int)from : 0x7fffffff;
    }
    const int4* cblock = f.cblock != nullptr ? f.cblock + (int64_t)b * f.ncb : nullptr;
    const int32_t* cdoc = f.cdoc != nullptr ? f.cdoc + (int64_t)b * f.ncb * 64 : nullptr;
    for (int i = grp; i < n; i += 2) {
      const int g = MODE == MODE_DQ ? 0 : (first + i) / per, ct = c_lo + first + i - g * per;
      const int col0 = ct * NB + 32 * side;
      MbwCols cq;
      // visible columns
      if constexpr (MODE == MODE_DQ) {
        const int left = lim - col0;
        cq.seen = left >= 32 ? ~0u : (left <= 0 ? 0u : (~0u >> (32 - left)));
        cq.d0 = BIAS ? (float)(pos - col0) : 0.0f;
        cq.slope2 = BIAS ? a.slopes[head] * L2E_HI : 0.0f;
      } else {
        const int skip = lim == 0x7fffffff ? 32 : lim - col0;
        cq.seen = skip <= 0 ? ~0u : (skip >= 32 ? 0u : (~0u << skip));
        cq.d0 = BIAS ? (float)(start + col0 - ac) : 0.0f;
        cq.slope2 = BIAS ? a.slopes[u * a.group + g] * L2E_HI : 0.0f;
      }
      if (cblock != nullptr) {
        cq.seen = (uint32_t)mod_doc_seen<32>(cq.seen, doc, cblock[ct], cdoc + (int64_t)ct * 64 + 32 * side);
      }
      cq.lse2 = lse2;
      const uint32_t stats = sStats + (uint32_t)((i % NST) * 512 + 128 * side);
      cq.stats = stats;
      const bool border = __any_sync(0xffffffffu, cq.seen != ~0u);
      int line = 0;
      if constexpr (BIAS) {
        // distances >= 0 along the thread's columns, or wherever a key is visible
        const bool ahead =
            (MODE == MODE_DQ ? cq.d0 >= 31.0f : cq.d0 >= 0.0f) || (a.causal && a.prefix_len == nullptr);
        line = __all_sync(0xffffffffu, ahead) ? 1 : 0;
      }
      float p[32];
      uint32_t t2[CAP && MODE == MODE_DQ ? 16 : 1];
      wait_or_flag(B_S + grp, (uint32_t)((i >> 1) & 1));
      if constexpr (MODE == MODE_DKV) wait_or_flag(B_C1 + i % NST, (uint32_t)((i / NST) & 1));  // the statistics
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      mbw_phase1<T, MODE, CAP, BIAS>(ts, a, cq, border, line, p, t2);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_P + grp));
      wait_or_flag(B_DP + grp, (uint32_t)((i >> 1) & 1));
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      mbw_phase2<T, MODE, CAP>(tdp, delta, stats + 256, p, t2, r);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_DS + grp));
    }
    if (n > 0) wait_or_flag(B_END, 0u);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if constexpr (MODE == MODE_DQ) {
      // r over the lane's four threads; the corrected D for MODE_DKV
      xchg[(2 * grp + side) * 128 + rt] = r;
      asm volatile("barrier.sync.aligned 1, %0;" ::"n"(MBW_ROWS) : "memory");
      r = (xchg[rt] + xchg[128 + rt]) + (xchg[256 + rt] + xchg[384 + rt]);
      if (f.px1 == nullptr && tid < 128 && in) f.delta[row] = delta + r;
    }
    // a lane's threads share its columns, 32 each (D = 64: the first group alone); each warp stores
    // through 2 KB of the (now free) stages
    const uint32_t stg = sC + (uint32_t)(warp * 2048);
    const int col = (2 * grp + side) * 32;
    float chk = 0.0f;
    if (col < D) {
      float x1[32], x2[32];
      if (n > 0) {
        tc_ld32(t_x1 + lane_off + (uint32_t)col, x1);
        tc_ld32(t_x2 + lane_off + (uint32_t)col, x2);
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) x1[x] = x2[x] = 0.0f;
      }
      if (f.px1 != nullptr) {
        const int64_t prow = ((int64_t)part * a.batch * heads + bh) * lanes + at;
        mbw_store32_f32(stg, x1, f.px1, in ? prow * D : -1, col);
        mbw_store32_f32(stg, x2, f.px2, in ? prow * D : -1, col);
        if (MODE == MODE_DQ && tid < 128 && in) f.pr[prow] = r;
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if constexpr (MODE == MODE_DQ)
            x1[x] = __fmaf_rn(-r, x1[x], x2[x]) * f.m.scale;
          else
            x2[x] *= f.m.scale;
          chk = __fmaf_rn(x1[x], 0.0f, chk);
          if constexpr (MODE == MODE_DKV) chk = __fmaf_rn(x2[x], 0.0f, chk);
        }
        if constexpr (MODE == MODE_DQ) {
          mbw_store32(stg, x1, out1, in ? b * f.m.dqs[0] + head * f.m.dqs[1] + at * f.m.dqs[2] : -1, col);
        } else {
          mbw_store32(stg, x1, out1, in ? b * f.m.dvs[0] + head * f.m.dvs[1] + at * f.m.dvs[2] : -1, col);
          mbw_store32(stg, x2, out2, in ? b * f.m.dks[0] + head * f.m.dks[1] + at * f.m.dks[2] : -1, col);
        }
      }
    }
    // lanes whose result is not finite, again: after every thread's stores, a warp a lane
    if (in && n > 0 && chk != 0.0f) atomicOr(&flags[rt], 1);
    asm volatile("barrier.sync.aligned 1, %0;" ::"n"(MBW_ROWS) : "memory");
    for (int x = 0; x < 8; ++x) {
      const int bad = warp * 8 + x;
      if (flags[bad] != 0) mbw_exact<T, D, MODE>(f, b, head, l0 + bad, q, k, v, o, lse, d_o, out1, out2);
    }
  }
  if (!ok) atomicOr(f.status, DEV_TIMEOUT);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == MBW_MMA_WARP) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// The parts of each lane added up in their order: dq and the corrected D, or dk and dv.  A warp a lane;
// bound by reading the parts (mostly out of the L2).  Both kernels in parts took 52 us where whole columns took 110
// (1 x 8 heads x 1000 rows, D = 128), 280 against 427 (1 x 16 over 2 key heads x 4096).
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(128)
    k_mod_backward_sum(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                       const T* __restrict__ o, const float* __restrict__ lse, const T* __restrict__ d_o, T* out1,
                       T* out2, const __grid_constant__ ModBwdKernelArgs f) {
  mod_trigger();
  const ModArgs& a = f.m.a;
  const int heads = MODE == MODE_DQ ? a.hq : a.hkv, lane = threadIdx.x & 31;
  const int64_t lanes = MODE == MODE_DQ ? a.sq : a.sk, rows = (int64_t)a.batch * heads * lanes;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  mod_wait();
  if (row >= rows) return;
  constexpr int N = D / 32;
  const int64_t bh = row / lanes, at = row - bh * lanes;
  const int b = (int)(bh / heads), h = (int)(bh - (int64_t)b * heads);
  float x1[N], x2[N], r = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) x1[i] = x2[i] = 0.0f;
  for (int p = 0; p < f.parts; ++p) {
    float y1[N], y2[N];
    mod_row_load<float, D>(f.px1 + (p * rows + row) * D, y1);
    mod_row_load<float, D>(f.px2 + (p * rows + row) * D, y2);
    if constexpr (MODE == MODE_DQ) r += f.pr[p * rows + row];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x1[i] += y1[i];
      x2[i] += y2[i];
    }
  }
  float chk = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (MODE == MODE_DQ)
      x1[i] = __fmaf_rn(-r, x1[i], x2[i]) * f.m.scale;
    else
      x2[i] *= f.m.scale;
    chk = __fmaf_rn(x1[i], 0.0f, chk);
    if constexpr (MODE == MODE_DKV) chk = __fmaf_rn(x2[i], 0.0f, chk);
  }
  if (MODE == MODE_DQ && lane == 0) f.delta[bh * f.sq_pad + at] += r;
  if (__any_sync(0xffffffffu, chk != 0.0f)) {
    mbw_exact<T, D, MODE>(f, b, h, at, q, k, v, o, lse, d_o, out1, out2);
  } else if constexpr (MODE == MODE_DQ) {
    mod_row_store<T, D>(out1 + b * f.m.dqs[0] + h * f.m.dqs[1] + at * f.m.dqs[2], x1);
  } else {
    mod_row_store<T, D>(out1 + b * f.m.dvs[0] + h * f.m.dvs[1] + at * f.m.dvs[2], x1);
    mod_row_store<T, D>(out2 + b * f.m.dks[0] + h * f.m.dks[1] + at * f.m.dks[2], x2);
  }
}

// Base-2 LSE and D = do . o of every query row, padded to whole tiles of 128 (+inf and 0: such
// rows weigh nothing).  16 bytes a lane: D / 8 lanes a row, MBW_PRE rows' loads in flight a lane. Bound by
// reading o and do once.
constexpr int MBW_PRE = 4;
template <typename T, int D>
__global__ void __launch_bounds__(256)
    k_mod_backward_rows(const T* __restrict__ o, const T* __restrict__ d_o, const float* __restrict__ lse,
                        float* __restrict__ lse2, float* __restrict__ delta, int64_t sq_pad,
                        const __grid_constant__ ModBwdArgs m) {
  mod_trigger();
  const ModArgs& a = m.a;
  constexpr int L = D / 8, R = 256 / L;  // lanes a row, rows a pass of the CTA
  // a CTA's rows lie in one head: sq_pad is a multiple of 128 and R x MBW_PRE divides 128
  static_assert(128 % (R * MBW_PRE) == 0, "a CTA's rows share a head");
  const int64_t row0 = (int64_t)blockIdx.x * (R * MBW_PRE);
  const int64_t bh = row0 / sq_pad, i0 = row0 - bh * sq_pad;
  const int b = (int)(bh / a.hq), h = (int)(bh - (int64_t)b * a.hq);
  const int sub = threadIdx.x / L, c = (threadIdx.x % L) * 8;
  const T* ob = o + b * a.os[0] + h * a.os[1] + c;
  const T* gb = d_o + b * m.dos[0] + h * m.dos[1] + c;
  uint4 x[MBW_PRE], y[MBW_PRE];
#pragma unroll
  for (int p = 0; p < MBW_PRE; ++p) {
    const int64_t i = i0 + p * R + sub;
    x[p] = y[p] = make_uint4(0, 0, 0, 0);
    if (i < a.sq) {
      x[p] = *reinterpret_cast<const uint4*>(ob + i * a.os[2]);
      y[p] = *reinterpret_cast<const uint4*>(gb + i * m.dos[2]);
    }
  }
#pragma unroll
  for (int p = 0; p < MBW_PRE; ++p) {
    const int64_t i = i0 + p * R + sub;
    float u[8], v[8], dl = 0.0f;
    unpack16<T>(x[p], u);
    unpack16<T>(y[p], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) dl = __fmaf_rn(u[j], v[j], dl);
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) dl += __shfl_xor_sync(0xffffffffu, dl, off);
    if (threadIdx.x % L == 0) {
      const float l = i < a.sq ? lse[bh * a.sq + i] : neg_inf();
      const bool none = l == neg_inf();
      lse2[row0 + p * R + sub] = none ? pos_inf() : l * L2E_HI;
      delta[row0 + p * R + sub] = none ? 0.0f : dl;
    }
  }
  mod_wait();
}

}  // namespace smx
