// Attention with modified scores on the 5th-generation tensor cores: the
// running state (m, l, o) of "Online stable softmax" ("Carry a weighted value
// numerator for attention"), one query row a thread.
//
// The layout is that of the persistent two-tile kernel (kernel_attention_tma.cuh,
// whose comment gives the roles, the issue rounds and the reuse of barriers):
// a CTA an SM walks work items of 2 x 128 query rows over key blocks of 64; the two
// tiles' row warps turn scores into probabilities in tensor memory, one warp a tile issues
// its products, two warps fetch K, and Q and V, by tensor maps.  What differs:
//   - the rows hand a block over by an mbarrier, not a named barrier: a wait that runs out cannot
//     leave a warp behind at it;
//   - an item has a first key block (documents, parts of a split row) and
//     rows of one or of several query heads of a key head's group (pf > 1: the group's rows,
//     which lie behind each other, share the tile and each K and V fetch);
//   - the scores pass the cap and get the bias in registers, in base-2 units, before
//     the maximum; only blocks at a mask's border test keys one by one;
//   - a row's keys may be split over items (few rows, many keys): each part leaves its
//     unnormalised (m, l, o) in fp32 and k_mod_merge joins them in order;
//   - a row whose result is not finite is computed again from the keys it sees, behind the CTA's items
//     (mod_fix_items, kernel_mod_exact.cuh): a product's 0 x NaN from a key that the row does not see leaves no trace.
//
// Bound: at D = 128 the tensor cores (2 x 32 heads over 8 key heads x 4096 rows, calls back to back: 373 us, 1470
// TFLOP/s; causal 217); with a cap (631, causal 360), a bias (530, causal 340) or D = 64 (341) the row warps' chain: a
// block's load from tensor memory, maximum, exponentials, store and hand-over, two warps a scheduler.  No unit is full
// then: a causal capped forward has its tensor pipe busy 31 % of the time, its issue slots 47, exp2 unit 16, FMA pipe 20
// (ncu; the exp2 unit gives 32 a cycle an SM, so 128 x 64 scores take it 256 cycles).  The issuing and rare code is
// kept short: what the instruction cache loses between blocks or items is fetched anew (its hit rate is 89 to 97 %, and
// about one of a scheduler's warps waits for instructions; capped rows in two rolled passes with a maximum before the
// cap: 379 us where one unrolled pass took 415; an item's output in rolled loops and its decoding by 32-bit divisions:
// causal 211, before 234).
#pragma once

#include "kernel_attention_tma.cuh"
#include "kernel_mod_exact.cuh"

namespace smx {

struct ModFwdArgs {
  ModArgs a;
  int pf;            // query heads of a group whose rows share the tiles (1: none)
  int heads;         // batch x hq / pf
  int64_t rows;      // pf x sq
  int64_t nq;        // items of 256 rows a head
  uint32_t chunk;    // heads whose items are dealt together
  int splits;        // parts of a row's keys
  int64_t items;     // heads x nq x splits
  const int2* range;   // documents: [batch][row tiles of 128] first and end key block; or null
  const int4* kblock;  // documents: [batch][nkb] summaries of the key blocks (kernel_mod_docs.cuh)
  const int32_t* kdoc;  // documents: [batch][64 nkb], -1 past the keys
  int nkb, row_tiles;
  // rows of a shared prefix (req > 0): [request][group head][token] of one key head a tile head; every
  // key is visible.  own_len [req] (or null: own_sk) and own_sk: the requests' own keys, behind the prefix's
  int req, map_group, map_sq, map_hq;
  const int32_t* own_len;
  int64_t own_sk;
  int q_req;  // > 0: rows a request has in the query map, whose boxes are whole requests of one key head
  float* po;           // partial states: [part][all rows][D], or null (whole rows)
  float2* pml;         // [all rows][parts] (m, l)
  int parts;           // parts of a row in all
  int64_t all_rows;    // rows of the result, batch x heads x queries
  int split0;          // first part's place among the row's parts
  int* status;
  int64_t max_polls;
  int64_t probe_polls;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2_4d(const CUtensorMap* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};\n"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Work item w: its heads, rows and key blocks.
struct ModItem {
  int64_t head, r0;  // tile head and its first row
  int b, hp, u;      // batch, tile head within the batch, key head
  int first, n[2], nmax, split;
  __device__ __forceinline__ ModItem(int64_t w, const ModFwdArgs& f) {
    const ModArgs& a = f.a;
    // (32-bit divisions: fewer than 2^31 items; every role goes through this at each item)
    uint32_t x = (uint32_t)w;
    split = 0;
    if (f.splits > 1) {
      split = (int)(x % (uint32_t)f.splits);
      x /= (uint32_t)f.splits;
    }
    // chunks of heads; in a chunk every head's last rows first, then the rows before
    // them: under a causal mask the longest items come first, so that the last round's are short
    const uint32_t nq = (uint32_t)f.nq, h0 = x / (f.chunk * nq) * f.chunk;
    const uint32_t hn = min((uint32_t)f.heads - h0, f.chunk);
    x -= h0 * nq;
    const uint32_t qb = x / hn;
    head = h0 + (x - qb * hn);
    r0 = (int64_t)(a.causal ? nq - 1 - qb : qb) * 256;
    const uint32_t per = (uint32_t)(f.pf > 1 ? a.hq / f.pf : a.hq);
    b = (int)((uint32_t)head / per);
    hp = (int)((uint32_t)head - (uint32_t)b * per);
    u = f.pf > 1 ? hp * f.pf / a.group : hp / a.group;
    int lo[2], hi[2];
    const int64_t start = mod_start(a, b), prefix = mod_prefix(a, b), klen = mod_klen(a, b);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t f0 = r0 + t * 128;
      lo[t] = hi[t] = 0;
      if (f0 >= f.rows) continue;
      if (f.range != nullptr) {
        const int2 rg = f.range[(int64_t)b * f.row_tiles + f0 / 128];
        lo[t] = rg.x;
        hi[t] = rg.y;
      } else {
        // the row with the largest limit: the last query of the tile's rows
        const int64_t l0 = f0 + 127 < f.rows - 1 ? f0 + 127 : f.rows - 1;
        int64_t i = l0;
        if (f.pf > 1) {
          const uint32_t sq = (uint32_t)a.sq, g0 = (uint32_t)f0 / sq, g1 = (uint32_t)l0 / sq;
          i = g0 != g1 ? a.sq - 1 : l0 - (int64_t)g1 * sq;
        }
        const int64_t lim = f.req > 0 ? a.sk : mod_limit(a, start + i, prefix, klen);
        hi[t] = (int)((lim + 63) / 64);
      }
    }
    const int e0 = hi[0] > lo[0], e1 = hi[1] > lo[1];
    int from = e0 ? lo[0] : lo[1], to = hi[0] > hi[1] ? hi[0] : hi[1];
    if (e0 && e1 && lo[1] < from) from = lo[1];
    if (!e0 && !e1) to = from;
    if (f.splits > 1) {
      const int part = (to - from + f.splits - 1) / f.splits;
      from += split * part;
      to = from + part < to ? from + part : to;
    }
    first = from;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int end = hi[t] < to ? hi[t] : to;
      n[t] = hi[t] > lo[t] && end > from ? end - from : 0;
    }
    nmax = n[0] > n[1] ? n[0] : n[1];
  }
  __device__ __forceinline__ int nt(int t) const { return t ? n[1] : n[0]; }
};

// A row thread's constants for its item.
struct ModRowState {
  int lim;        // keys below it may be visible
  int doc;        // its document
  float slope2;   // base-2 slope
  int64_t pos;
};

// Row rt of an item's tile t: query i of head h, its place among all rows of the result, its query's offset.
// Rows past the end stand for the last row (in false: nothing of theirs is stored).
struct ModRowAt {
  bool in;
  int h;
  int64_t i, lse_at, qoff;
  ModRowState rs;
};
template <bool BIAS>
__device__ __forceinline__ ModRowAt mod_row_at(const ModFwdArgs& f, const ModItem& it, int t, int rt) {
  const ModArgs& a = f.a;
  ModRowAt x;
  const int64_t r = it.r0 + t * ATM_BM + rt;
  x.in = r < f.rows;
  const int64_t rc = x.in ? r : f.rows - 1;
  const int g = f.pf > 1 ? (int)((uint32_t)rc / (uint32_t)a.sq) : 0;
  x.i = rc - (int64_t)g * a.sq;
  x.h = it.hp * f.pf + g;
  x.lse_at = ((int64_t)it.b * a.hq + x.h) * a.sq + x.i;
  x.qoff = it.b * a.qs[0] + (int64_t)x.h * a.qs[1] + x.i * a.qs[2];
  if (f.req > 0) {
    const int per = f.map_group * f.map_sq, rq = (int)rc / per, rest = (int)rc - rq * per;
    const int hg = rest / f.map_sq, tok = rest - hg * f.map_sq, hh = it.u * f.map_group + hg;
    x.lse_at = ((int64_t)rq * f.map_hq + hh) * f.map_sq + tok;
    if (f.q_req) x.qoff = (int64_t)rq * a.qs[0] + (int64_t)hh * a.qs[1] + tok * a.qs[2];
    int64_t own = f.own_sk;
    if (f.own_len != nullptr) {
      const int64_t y = f.own_len[rq];
      own = y < 0 ? 0 : (y < own ? y : own);
    }
    x.rs.pos = a.sk + own - f.map_sq + tok;
    x.rs.lim = (int)a.sk;
    x.rs.doc = 0;
    x.rs.slope2 = BIAS ? a.slopes[hh] * L2E_HI : 0.0f;
  } else {
    const ModView view = mod_view(a, it.b, x.i);
    x.rs.pos = view.pos;
    x.rs.lim = (int)view.lim;
    x.rs.doc = view.doc;
    x.rs.slope2 = BIAS ? a.slopes[x.h] * L2E_HI : 0.0f;
  }
  return x;
}

// Keys of a block of 64 below the row's limit, as a bit mask.
__device__ __forceinline__ uint64_t mod_block_seen(const ModRowState& rs, int key0) {
  const int left = rs.lim - key0;
  return left >= 64 ? ~0ull : (left <= 0 ? 0ull : (~0ull >> (64 - left)));
}
__device__ __forceinline__ bool mod_bit(uint32_t s0, uint32_t s1, int i) { return ((i < 32 ? s0 : s1) >> (i & 31)) & 1u; }

// largest and smallest of a row's 64 scores (NaN passed over)
__device__ __forceinline__ float mod_max64(const float (&y)[64]) {
  float m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = fmaxf(y[2 * j], y[2 * j + 1]);
#pragma unroll
  for (int i = 8; i < 64; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = max3(m[j], y[i + 2 * j], y[i + 2 * j + 1]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
__device__ __forceinline__ float mod_min64(const float (&y)[64]) {
  float m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = fminf(y[2 * j], y[2 * j + 1]);
#pragma unroll
  for (int i = 8; i < 64; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = fmin3(m[j], y[i + 2 * j], y[i + 2 * j + 1]);
  return fminf(fminf(m[0], m[1]), fminf(m[2], m[3]));
}

// y = cap tanh(c y) in base 2
template <int FORM>
__device__ __forceinline__ void mod_cap64(float (&y)[64], const ModArgs& a) {
  const unsigned long long c2 = pk(a.c, a.c);
#pragma unroll
  for (int i = 0; i < 64; i += 2) {
    if constexpr (FORM == CAP_EXP) {
      y[i] = a.cap2 * tanh_exp(y[i] * a.c);
      y[i + 1] = a.cap2 * tanh_exp(y[i + 1] * a.c);
    } else {
      const unsigned long long u = mul2(pk(y[i], y[i + 1]), c2);
      const unsigned long long r = mul2(tanh_ratio2<FORM == CAP_NEAR>(u, a.cap2), u);
      y[i] = pk_lo(r);
      y[i + 1] = pk_hi(r);
    }
  }
}

// P of a row's 64 scores against the reference maximum: 2^(c y - m), or 2^(y - m) (DONE: the cap and the bias
// are in y already; what is hidden is -inf); packed in the input type; their sum returned.
template <typename T, bool DONE>
__device__ __forceinline__ float mod_exp64(const float (&y)[64], const ModArgs& a, float nsub, uint32_t (&pk2)[32]) {
  const unsigned long long c2 = pk(a.c, a.c), ns2 = pk(nsub, nsub);
  unsigned long long acc2[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 64; i += 2) {
    const unsigned long long y2 = pk(y[i], y[i + 1]), e = DONE ? add2(y2, ns2) : fma2(y2, c2, ns2);
    const float p0 = ex2_ftz(pk_lo(e)), p1 = ex2_ftz(pk_hi(e));
    acc2[(i >> 1) & 1] = add2(acc2[(i >> 1) & 1], pk(p0, p1));
    pk2[i / 2] = pack2<T>(p0, p1);
  }
  return (pk_lo(acc2[0]) + pk_hi(acc2[0])) + (pk_lo(acc2[1]) + pk_hi(acc2[1]));
}

// largest (smallest) of 32 scores (NaN passed over)
__device__ __forceinline__ float mod_max32(const float (&y)[32], float m) {
  float m2 = fmaxf(y[0], y[1]);
#pragma unroll
  for (int i = 2; i < 32; i += 4) {
    m = max3(m, y[i], y[i + 1]);
    if (i + 2 < 32) m2 = max3(m2, y[i + 2], y[i + 3]);
  }
  return fmaxf(m, m2);
}
__device__ __forceinline__ float mod_min32(const float (&y)[32], float m) {
  float m2 = fminf(y[0], y[1]);
#pragma unroll
  for (int i = 2; i < 32; i += 4) {
    m = fmin3(m, y[i], y[i + 1]);
    if (i + 2 < 32) m2 = fmin3(m2, y[i + 2], y[i + 3]);
  }
  return fminf(m, m2);
}

// 2^(x - m) of 32 scores, x = cap tanh(c y) (FORM), packed, and their sum; HIDE: what `seen` leaves out
// becomes 0.
template <typename T, int FORM, bool HIDE>
__device__ __forceinline__ float mod_exp32(const float (&y)[32], const ModArgs& a, float nsub, uint32_t seen,
                                           uint32_t (&pk2)[16]) {
  const unsigned long long c2 = pk(a.c, a.c), ns2 = pk(nsub, nsub);
  unsigned long long acc2[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    unsigned long long e;
    if constexpr (FORM == CAP_EXP) {
      e = pk(__fmaf_rn(a.cap2, tanh_exp(y[i] * a.c), nsub), __fmaf_rn(a.cap2, tanh_exp(y[i + 1] * a.c), nsub));
    } else {
      const unsigned long long u = mul2(pk(y[i], y[i + 1]), c2);
      e = fma2(tanh_ratio2<FORM == CAP_NEAR>(u, a.cap2), u, ns2);
    }
    float p0 = ex2_ftz(pk_lo(e)), p1 = ex2_ftz(pk_hi(e));
    if constexpr (HIDE) {
      p0 = (seen >> i) & 1u ? p0 : 0.0f;
      p1 = (seen >> (i + 1)) & 1u ? p1 : 0.0f;
    }
    acc2[(i >> 1) & 1] = add2(acc2[(i >> 1) & 1], pk(p0, p1));
    pk2[i / 2] = pack2<T>(p0, p1);
  }
  return (pk_lo(acc2[0]) + pk_hi(acc2[0])) + (pk_lo(acc2[1]) + pk_hi(acc2[1]));
}

// One key block of one row thread with a cap: the scores are read twice, 32 at a time, for their maximum and
// for the exponentials, in loops that stay rolled.  (Unrolled over 64 scores in registers the capped code
// overruns the instruction cache, which two warps an SM quarter, apart from each other, and the issuing warps
// share: a causal 2 x 32 x 4096 x 128 forward took 415 us, against 380.  With a bias instead of a cap the
// second reading and its bias cost more than that: 708 against 533 us without a mask.)
template <typename T, int D>
__device__ __forceinline__ void mod_rows_cap(uint32_t ts, uint32_t to, bool first, const ModArgs& a, uint64_t seen,
                                             bool border, float& m_ref, float& l, bool& ok, uint32_t o_bar,
                                             uint32_t o_par, int64_t max_polls, int* status) {
  float mx = neg_inf(), lo = pos_inf();
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float y[32];
    tc_ld32(ts + (uint32_t)(32 * h), y);
    if (__builtin_expect(border, 0)) {
      asm volatile("");
      const uint32_t bits = (uint32_t)(seen >> (32 * h));
      float z = lo;
#pragma unroll
      for (int i = 0; i < 32; ++i) z = fminf(z, (bits >> i) & 1u ? y[i] : pos_inf());
      lo = z;
#pragma unroll
      for (int i = 0; i < 32; ++i) y[i] = (bits >> i) & 1u ? y[i] : neg_inf();
    } else {
      lo = mod_min32(y, lo);
    }
    mx = mod_max32(y, mx);
  }
  const float far = fmaxf(mx, -lo) * a.c;
  const int form =
      __all_sync(0xffffffffu, far <= TANH_NEAR) ? CAP_NEAR : (__all_sync(0xffffffffu, far <= 1.0f) ? CAP_POLY : CAP_EXP);
  // (the cap is monotonic: the maximum is taken before it.  A visible product of -inf is a score of -cap: a row is
  // without a maximum only where it sees no key of the block)
  mx = seen == 0 ? neg_inf() : a.cap2 * tanh_score(mx * a.c);
  float alpha = 1.0f;
  if (mx > m_ref + 8.0f) {
    alpha = m_ref == neg_inf() ? 0.0f : ex2_full(m_ref - mx);
    m_ref = mx;
  }
  const float nsub = m_ref == neg_inf() ? 0.0f : -m_ref;
  float ps = 0.0f;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float y[32];
    uint32_t pk2[16];
    const uint32_t bits = (uint32_t)(seen >> (32 * h));
    tc_ld32(ts + (uint32_t)(32 * h), y);
    if (__builtin_expect(form == CAP_NEAR && !border, 1)) {
      ps += mod_exp32<T, CAP_NEAR, false>(y, a, nsub, bits, pk2);
    } else if (border) {
      if (form == CAP_EXP)
        ps += mod_exp32<T, CAP_EXP, true>(y, a, nsub, bits, pk2);
      else
        ps += mod_exp32<T, CAP_POLY, true>(y, a, nsub, bits, pk2);
    } else if (form == CAP_POLY) {
      ps += mod_exp32<T, CAP_POLY, false>(y, a, nsub, bits, pk2);
    } else {
      ps += mod_exp32<T, CAP_EXP, false>(y, a, nsub, bits, pk2);
    }
    // P over scores that are read: the first half's over its own, the second's behind it
    tc_st16u(ts + (uint32_t)(16 * h), pk2);
  }
  l = __fmaf_rn(l, alpha, ps);
  if (__builtin_expect(!first && __any_sync(0xffffffffu, alpha != 1.0f), 0)) {
    if (!tc_wait(o_bar, o_par, max_polls, status)) {
      ok = false;
      atomicOr(status, DEV_TIMEOUT);
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      float t16[16];
      tc_ld16(to + (uint32_t)c, t16);
#pragma unroll
      for (int i = 0; i < 16; ++i) t16[i] *= alpha;
      tc_st16(to + (uint32_t)c, t16);
    }
  }
}

// One key block of one row thread (as tc_rows_block, with the scores' changes):
// scores at ts, P over their first 32 columns, O at `to`.
template <typename T, int D, bool CAP, bool BIAS>
__device__ __forceinline__ void mod_rows_block(uint32_t ts, uint32_t to, bool first, const ModArgs& a,
                                               const ModRowState& rs, int key0, uint64_t seen, bool border,
                                               float& m_ref, float& l,
                                               bool& ok, uint32_t o_bar, uint32_t o_par, int64_t max_polls,
                                               int* status) {
  float y[64];
  tc_ld64(ts, y);
  const uint32_t s0 = (uint32_t)seen, s1 = (uint32_t)(seen >> 32);
  float mx = 0.0f;
  int form = CAP_EXP;
  // (the empty asm keeps the rare path a branch: as selects it would cost every block)
  if constexpr (!BIAS) {
    if (__builtin_expect(border, 0)) {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 64; ++i) y[i] = mod_bit(s0, s1, i) ? y[i] : neg_inf();
    }
    mx = mod_max64(y) * a.c;
  }
  if constexpr (CAP) {
    if (__builtin_expect(border, 0)) {
      // hidden places decide nothing about the cap's form
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 64; ++i) y[i] = mod_bit(s0, s1, i) ? y[i] : 0.0f;
    }
    const float far = fmaxf(mod_max64(y), -mod_min64(y)) * a.c;
    form = __all_sync(0xffffffffu, far <= TANH_NEAR) ? CAP_NEAR : (__all_sync(0xffffffffu, far <= 1.0f) ? CAP_POLY : CAP_EXP);
  }
  if constexpr (BIAS) {
    if constexpr (CAP) {
      if (form == CAP_NEAR)
        mod_cap64<CAP_NEAR>(y, a);
      else if (form == CAP_POLY)
        mod_cap64<CAP_POLY>(y, a);
      else
        mod_cap64<CAP_EXP>(y, a);
    }
    // -slope |pos - j|: one line along the block unless the row's position lies in it
    const float c = CAP ? 1.0f : a.c;
    const float d0 = (float)(rs.pos - key0);
    const bool before = d0 >= 63.0f || (a.causal && a.prefix_len == nullptr);  // every visible key is at or before pos
    if (__all_sync(0xffffffffu, before || d0 <= 0.0f)) {
      const float st = before ? rs.slope2 : -rs.slope2, base = before ? -rs.slope2 * d0 : rs.slope2 * d0;
      // (the line is stepped, anew every 8 keys: three additions' rounding at most)
      const unsigned long long c2 = pk(c, c), st2 = pk(2.0f * st, 2.0f * st);
#pragma unroll
      for (int h = 0; h < 64; h += 8) {
        unsigned long long line = pk(__fmaf_rn((float)h, st, base), __fmaf_rn((float)(h + 1), st, base));
#pragma unroll
        for (int i = h; i < h + 8; i += 2) {
          const unsigned long long r = fma2(pk(y[i], y[i + 1]), c2, line);
          y[i] = pk_lo(r);
          y[i + 1] = pk_hi(r);
          if (i + 2 < h + 8) line = add2(line, st2);
        }
      }
    } else {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 64; ++i) y[i] = __fmaf_rn(y[i], c, -rs.slope2 * fabsf(d0 - (float)i));
    }
    if (__builtin_expect(border, 0)) {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 64; ++i) y[i] = mod_bit(s0, s1, i) ? y[i] : neg_inf();
    }
    mx = mod_max64(y);
  }
  float alpha = 1.0f;
  if (mx > m_ref + 8.0f) {
    alpha = m_ref == neg_inf() ? 0.0f : ex2_full(m_ref - mx);
    m_ref = mx;
  }
  const float nsub = m_ref == neg_inf() ? 0.0f : -m_ref;
  uint32_t pk2[32];
  const float ps = mod_exp64<T, BIAS>(y, a, nsub, pk2);
  l = __fmaf_rn(l, alpha, ps);
  if (__builtin_expect(!first && __any_sync(0xffffffffu, alpha != 1.0f), 0)) {
    if (!tc_wait(o_bar, o_par, max_polls, status)) {
      ok = false;
      atomicOr(status, DEV_TIMEOUT);
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
    for (int c = 0; c < D; c += 16) {
      float t16[16];
      tc_ld16(to + (uint32_t)c, t16);
#pragma unroll
      for (int i = 0; i < 16; ++i) t16[i] *= alpha;
      tc_st16(to + (uint32_t)c, t16);
    }
  }
  tc_st32(ts, pk2);
}

// A warp's rows whose stored results are not finite, again from the keys they see (rare: a NaN or an infinity
// among the inputs): a walk over the CTA's items behind the last of them.  (Not within an item: a row takes 0.58 us a
// key, a warp's 32 rows over 11000 keys outlast the 200 ms after which the other warps' waits for it give up.)
template <typename T, int D, bool BIAS>
__device__ __noinline__ void mod_fix_items(const ModFwdArgs& f, int t, int rt, const T* q, const T* k, const T* v, T* o,
                                           float* lse) {
  const ModArgs& a = f.a;
  __syncwarp();  // the rows' stores, by other lanes
  for (int64_t kk = 0, w; (w = atm_item_of(kk, f.items)) >= 0; ++kk) {
    const ModItem it(w, f);
    if (it.nt(t) == 0) continue;
    const ModRowAt x = mod_row_at<BIAS>(f, it, t, rt);
    const int64_t ooff = it.b * a.os[0] + (int64_t)x.h * a.os[1] + x.i * a.os[2];
    const int64_t part = f.split0 + it.split, pat = part * f.all_rows + x.lse_at;
    bool lost = false;
    if (x.in && f.po != nullptr) {
      const float l = f.pml[x.lse_at * f.parts + part].y;
      lost = l != l;
      for (int c = 0; c < D && !lost; c += 4) {
        const float4 y = *reinterpret_cast<const float4*>(f.po + pat * D + c);
        const float chk = __fmaf_rn(y.x, 0.0f, __fmaf_rn(y.y, 0.0f, __fmaf_rn(y.z, 0.0f, y.w * 0.0f)));
        lost = chk != chk;
      }
    } else if (x.in) {
      for (int c = 0; c < D && !lost; c += 8) {
        float y[8], chk = 0.0f;
        unpack16<T>(*reinterpret_cast<const uint4*>(o + ooff + c), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) chk = __fmaf_rn(y[i], 0.0f, chk);
        lost = chk != chk;
      }
    }
    uint32_t bad = __ballot_sync(0xffffffffu, lost);
    while (bad != 0) {
      const int lane = __ffs(bad) - 1;
      bad &= bad - 1;
      ModView view;
      view.pos = __shfl_sync(0xffffffffu, x.rs.pos, lane);
      view.lim = __shfl_sync(0xffffffffu, x.rs.lim, lane);
      view.doc = __shfl_sync(0xffffffffu, x.rs.doc, lane);
      const float slope2 = __shfl_sync(0xffffffffu, x.rs.slope2, lane);
      const int64_t qo = __shfl_sync(0xffffffffu, x.qoff, lane), oo = __shfl_sync(0xffffffffu, ooff, lane);
      const int64_t la = __shfl_sync(0xffffffffu, x.lse_at, lane), pa = __shfl_sync(0xffffffffu, pat, lane);
      float m, l, acc[D / 32];
      mod_exact_row<T, D>(a, q + qo, k + it.b * a.ks[0] + it.u * a.ks[1], v + it.b * a.vs[0] + it.u * a.vs[1],
                          f.kdoc != nullptr ? f.kdoc + (int64_t)it.b * f.nkb * 64 : nullptr, view, slope2,
                          (int64_t)it.first * 64, ((int64_t)it.first + it.nmax) * 64, m, l, acc);
      if (f.po != nullptr) {
        mod_row_store<float, D>(f.po + pa * D, acc);
        if ((threadIdx.x & 31) == 0) f.pml[la * f.parts + part] = make_float2(m, l);
      } else {
        const float inv = l == 0.0f ? 0.0f : recip_refined(l);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= inv;
        mod_row_store<T, D>(o + oo, acc);
        if (lse != nullptr && (threadIdx.x & 31) == 0) lse[la] = mod_lse(m, l);
      }
    }
  }
}

template <typename T, int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(AtmShape<2>::BLOCK, 1)
    k_mod_forward(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const T* __restrict__ q, const T* __restrict__ k,
                  const T* __restrict__ v, T* __restrict__ o, float* __restrict__ lse,
                  const __grid_constant__ ModFwdArgs f) {
  static_assert(D == 64 || D == 128, "head dimension");
  constexpr int TILES = 2;
  using S = AtmShape<TILES>;
  constexpr int BM = ATM_BM, BN = ATM_BN, NK = S::NK, NV = S::NV;
  constexpr int QT = BM * D * 2;  // bytes of a Q tile
  constexpr int KT = BN * D * 2;  // bytes of a K or V stage
  // ... and P written, B_P + 2 t + (block & 1): the hand-over from a tile's rows to its issuing warp, an
  // arrival a warp.  (An mbarrier, whose waits are bounded: after a wait ran out rows and issuer may be
  // out of step, and a named barrier would then never open.)  The rows are at most one block ahead of the
  // issuer, so two barriers a tile keep the phases apart.
  constexpr int B_R = 0, B_KF = 32, B_VF = 36, B_Q = 40, B_PROBE = 41, B_DRAIN = 42, B_P = 44, NBAR = 48;
  static_assert(NK == 4 && NV == 4, "barrier layout");
  auto rnd = [](int t, int r) { return B_R + 16 * t + (r & 15); };
  auto rpar = [](int r) { return (uint32_t)((r >> 4) & 1); };
  extern __shared__ __align__(16) uint8_t smem_raw[];

  const ModArgs& a = f.a;
  // (a warp's number and the tensor memory's address by shuffle: values and branches that the compiler
  // knows to be the same in the whole warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t raw = tc_su32(smem_raw);
  const uint32_t pad = (1024 - (raw & 1023)) & 1023;
  uint8_t* base = smem_raw + pad;
  const uint32_t sQ = tc_su32(base), sK = sQ + TILES * QT, sV = sK + NK * KT, sO = sV + NV * KT;
  constexpr uint32_t AUX = NBAR * 8 + 4;
  static_assert(2 * AUX < 1024, "barriers fit the alignment slack");
  uint8_t* aux = pad >= AUX ? smem_raw : base + S::template tile_bytes<D>();
  uint64_t* bars = reinterpret_cast<uint64_t*>(aux);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBAR);
  const uint32_t bar0 = tc_su32(bars);
  auto bar = [bar0](int i) { return bar0 + 8u * (uint32_t)i; };

  mod_trigger();
  if (warp == S::ISSUE_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_su32(tmem_slot)),
                 "r"(S::TCOLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < NBAR; ++i) mbar_init(bar(i), i >= B_P ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  mod_wait();
  if (f.probe_polls > 0 && tid == 0 && !tc_wait(bar(B_PROBE), 0u, f.probe_polls, f.status))
    atomicOr(f.status, DEV_TIMEOUT);
  auto t_o = [tmem](int t) { return tmem + (uint32_t)(t * D); };
  auto t_s = [tmem](int t, int i) { return tmem + (uint32_t)(TILES * D + 128 * t + 64 * i); };
  bool ok = true;
  auto wait_or_flag = [&](uint32_t b_, uint32_t par) {
    if (!tc_wait(b_, par, f.max_polls, f.status)) {
      ok = false;
      atomicOr(f.status, DEV_TIMEOUT);
    }
  };
  // counters every role keeps alike over the CTA's items: rounds, blocks (and
  // K / V fetches), Q loads.  A tile takes part in every block of its item: where it has no keys of its own it
  // issues nothing, but still waits, commits and meets its rows, so that no role is ever two
  // phases of a barrier away from another.  (Rows that fill one tile leave the second out altogether.)
  int R0 = 0, J = 0, QC = 0;
  const int tiles = f.rows > BM ? 2 : 1;
  auto advance = [&](const ModItem& it) {
    R0 += it.nmax > 0 ? it.nmax + 2 : 0;
    J += it.nmax;
    QC += it.nmax > 0 ? 1 : 0;
  };

  if (warp >= S::ISSUE_WARP && warp < S::ISSUE_WARP + TILES) {
    // the issuing warp of tile t: the whole warp runs this code alike, lane 0's products (tc_mma_one)
    const int t = warp - S::ISSUE_WARP;
    const uint32_t one = tc_elect();
    const uint32_t id_s = tc_idesc<T>(BM, BN), id_o = tc_idesc<T>(BM, D, true);
    const uint32_t dq = tc_desc(sQ + (uint32_t)(t * QT));
    auto issue_s = [&](int g, int fe) {
      uint32_t da = dq, dk = tc_desc(sK + (uint32_t)((fe % NK) * KT));
      const uint32_t ts = t_s(t, g & 1);
#pragma unroll 1
      for (int h = 0; h < D / 64; ++h) {
#pragma unroll
        for (int st = 0; st < 4; ++st)
          tc_mma_one(one, ts, da + (uint32_t)(2 * st), dk + (uint32_t)(2 * st), id_s, (uint32_t)(h + st));
        da += (BM * 128) >> 4;
        dk += (BN * 128) >> 4;
      }
    };
    auto issue_pv = [&](int g, int fe, uint32_t more) {
      const uint32_t dv = tc_desc_mn(sV + (uint32_t)((fe % NV) * KT), (uint32_t)(BN * 128)), pb = t_s(t, g & 1);
#pragma unroll
      for (int s2 = 0; s2 < BN / 16; ++s2)
        tc_mma_ta_one(one, t_o(t), pb + (uint32_t)(s2 * 8), dv + (uint32_t)((s2 * 2048) >> 4), id_o,
                      s2 > 0 ? 1u : more);
    };
    for (int64_t kk = 0, w; (w = atm_item_of(kk, f.items)) >= 0; ++kk) {
      const ModItem it(w, f);
      const int n = __shfl_sync(0xffffffffu, it.nt(t), 0), nmax = __shfl_sync(0xffffffffu, t < tiles ? it.nmax : 0, 0),
                r0 = R0, g0 = J;
      const int64_t klen = f.req > 0 ? a.sk : mod_klen(a, it.b);
      const bool tail = ((int64_t)it.first + n) * BN > klen;  // the last block holds keys behind the length
      if (nmax > 0) {
        wait_or_flag(bar(B_Q), (uint32_t)(QC & 1));
#pragma unroll 1
        for (int r = 0; r < 2; ++r) {
          if (r < nmax) wait_or_flag(bar(B_KF + (J + r) % NK), (uint32_t)(((J + r) / NK) & 1));
          __syncwarp();
          if (r < n) issue_s(g0 + r, J + r);
          tc_commit_one(one, bar(rnd(t, r0 + r)));
        }
        for (int b = 0; b < nmax; ++b) {
          const int g = g0 + b;
          // V first: it is there long before the rows are done with the block (a satisfied wait costs some
          // 130 cycles; K's below is hidden behind O += P V)
          wait_or_flag(bar(B_VF + (J + b) % NV), (uint32_t)(((J + b) / NV) & 1));
          wait_or_flag(bar(B_P + 2 * t + (g & 1)), (uint32_t)((g >> 1) & 1));
          __syncwarp();
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (tail && b == n - 1) {
            // what lies behind the sequence's keys weighs 0, but 0 x NaN is NaN: those rows
            // of V become zero (both tiles' warps write the same zeros)
            const int from = klen - (int64_t)(it.first + b) * BN < 0 ? 0 : (int)(klen - (int64_t)(it.first + b) * BN);
            const uint32_t vb = sV + (uint32_t)(((J + b) % NV) * KT);
            for (int x = lane; x < (BN - from) * (D / 8); x += 32) {
              const int vr = from + x / (D / 8), vc = (x % (D / 8)) * 8;
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + tc_off(vr, vc, BN)), "r"(0)
                           : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          if (b < n) issue_pv(g, J + b, b > 0 ? 1u : 0u);
          if (b + 2 < nmax) {
            wait_or_flag(bar(B_KF + (J + b + 2) % NK), (uint32_t)(((J + b + 2) / NK) & 1));
            __syncwarp();
          }
          if (b + 2 < n) issue_s(g + 2, J + b + 2);
          tc_commit_one(one, bar(rnd(t, r0 + b + 2)));
        }
      }
      advance(it);
    }
    if (R0 > 0 && t < tiles) {
      tc_commit_one(one, bar(B_DRAIN + t));
      tc_wait_drain(bar(B_DRAIN + t), 0u);
    }
    __syncwarp();
  } else if (warp == S::KLOAD_WARP || warp == S::VLOAD_WARP) {
    // the stage fetchers: K, or Q and V
    const bool is_k = warp == S::KLOAD_WARP;
    const CUtensorMap* map = is_k ? &tm_k : &tm_v;
    const uint32_t stages = is_k ? sK : sV;
    const int full0 = is_k ? B_KF : B_VF;
    constexpr int NS = NK;
    int rec[2][NS];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < NS; ++i) rec[t][i] = -1;
    int qwait[2] = {-1, -1};
    if (lane == 0) {
      tma_prefetch_map(map);
      if (!is_k) tma_prefetch_map(&tm_q);
      for (int64_t kk = 0, w; (w = atm_item_of(kk, f.items)) >= 0; ++kk) {
        const ModItem it(w, f);
        const int64_t wn = atm_item_of(kk + 1, f.items);
        if (it.nmax > 0) {
          if (!is_k) {
#pragma unroll
            for (int t = 0; t < TILES; ++t)
              if (qwait[t] >= 0 && !tc_wait(bar(rnd(t, qwait[t])), rpar(qwait[t]), f.max_polls, f.status)) {
                ok = false;
                atomicOr(f.status, DEV_TIMEOUT);
              }
            mbar_arrive_expect_tx(bar(B_Q), (uint32_t)(TILES * QT));
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(sQ + (uint32_t)(t * QT + h * BM * 128), &tm_q, h * 64,
                            f.q_req ? 0 : (int)(it.r0 + t * BM), f.q_req ? (int)(it.r0 + t * BM) / f.q_req : it.hp,
                            f.q_req ? it.u : it.b, bar(B_Q));
#pragma unroll
            for (int t = 0; t < TILES; ++t)
              if (t < tiles) qwait[t] = R0 + it.nmax - 1;
          }
          const int pre_at = it.nmax > 8 ? it.nmax - 8 : 0;
          for (int j = 0; j < it.nmax; ++j) {
            if (j == pre_at && wn >= 0) {
              const ModItem nx(wn, f);
              for (int jj = 0; jj < NS && jj < nx.nmax; ++jj)
#pragma unroll
                for (int h = 0; h < D / 64; ++h) tma_prefetch_l2_4d(map, h * 64, (nx.first + jj) * BN, nx.u, nx.b);
              if (!is_k)
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    if (!f.q_req) tma_prefetch_l2_4d(&tm_q, h * 64, (int)(nx.r0 + t * BM), nx.hp, nx.b);
            }
            const int fe = J + j, s = fe % NS;
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              const int r = rec[t][0];
              if (r >= 0 && !atm_wait_lazy(bar(rnd(t, r)), rpar(r), f.max_polls, f.status)) {
                ok = false;
                atomicOr(f.status, DEV_TIMEOUT);
              }
            }
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
#pragma unroll
              for (int i = 0; i + 1 < NS; ++i) rec[t][i] = rec[t][i + 1];
              rec[t][NS - 1] = t < tiles ? R0 + (is_k ? j : j + 2) : -1;
            }
            mbar_arrive_expect_tx(bar(full0 + s), (uint32_t)KT);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(stages + (uint32_t)(s * KT + h * BN * 128), map, h * 64, (it.first + j) * BN, it.u, it.b,
                          bar(full0 + s));
          }
        }
        advance(it);
      }
      for (int s = 0; s < NS && s < J; ++s) {
        const int fl = s + ((J - 1 - s) / NS) * NS;  // the last fetch into stage s
        tc_wait_drain(bar(full0 + s), (uint32_t)((fl / NS) & 1));
      }
      if (!is_k && QC > 0) tc_wait_drain(bar(B_Q), (uint32_t)((QC - 1) & 1));
    }
    __syncwarp();
  } else {
    // row threads: tile t, TMEM lane rt of the tile
    const int t = tid >> 7, rt = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    bool redo = false;  // some row of the warp's items is not finite
    for (int64_t kk = 0, w; (w = atm_item_of(kk, f.items)) >= 0; ++kk) {
      const ModItem it(w, f);
      const int n = it.nt(t), nmax = t < tiles ? it.nmax : 0, r0 = R0, g0 = J;
      const ModRowAt at_row = mod_row_at<BIAS>(f, it, t, rt);
      const ModRowState& rs = at_row.rs;
      const bool in = at_row.in;
      const int64_t lse_at = at_row.lse_at;
      float m_ref = neg_inf(), l = 0.0f;
      const int4* kblock = f.kblock != nullptr ? f.kblock + (int64_t)it.b * f.nkb + it.first : nullptr;
      int4 docs = make_int4(0, 0, 0, 0);
      if (kblock != nullptr && n > 0) docs = kblock[0];
      const int32_t* kdoc = f.kdoc != nullptr ? f.kdoc + ((int64_t)it.b * f.nkb + it.first) * 64 : nullptr;
      for (int b = 0; b < n; ++b) {
        const int gg = g0 + b, rr = r0 + b;
        uint64_t seen = mod_block_seen(rs, (it.first + b) * BN);
        if (kblock != nullptr) {
          const int4 now = docs;
          if (b + 1 < n) docs = kblock[b + 1];  // a block ahead of its use
          seen = mod_doc_seen(seen, rs.doc, now, kdoc + b * 64);
        }
        const bool border = __any_sync(0xffffffffu, seen != ~0ull);
        if (!tc_wait(bar(rnd(t, rr)), rpar(rr), f.max_polls, f.status)) {
          ok = false;
          atomicOr(f.status, DEV_TIMEOUT);
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (CAP && !BIAS)
          mod_rows_cap<T, D>(t_s(t, gg & 1) + lane_off, t_o(t) + lane_off, b == 0, a, seen, border, m_ref, l, ok,
                             bar(rnd(t, rr + 1)), rpar(rr + 1), f.max_polls, f.status);
        else
          mod_rows_block<T, D, CAP, BIAS>(t_s(t, gg & 1) + lane_off, t_o(t) + lane_off, b == 0, a, rs,
                                          (it.first + b) * BN, seen, border, m_ref, l, ok, bar(rnd(t, rr + 1)),
                                          rpar(rr + 1), f.max_polls, f.status);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P + 2 * t + (gg & 1)));
      }
      // the tile's last O += P V: round n + 1; then the item's output, while
      // the other tile may still have blocks to go
      if (n > 0 && !tc_wait(bar(rnd(t, r0 + n + 1)), rpar(r0 + n + 1), f.max_polls, f.status)) {
        ok = false;
        atomicOr(f.status, DEV_TIMEOUT);
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // the item's output: whole rows normalised in the input type, or the
      // part's state in fp32.  chk stays 0 while every value is finite
      float chk = 0.0f;
      const int64_t ooff = it.b * a.os[0] + (int64_t)at_row.h * a.os[1] + at_row.i * a.os[2];
      if (f.po != nullptr) {
        const int64_t at = (int64_t)(f.split0 + it.split) * f.all_rows + lse_at;
        if (n > 0) {
          // 16 columns at a time through the warp's staging rows (64 bytes each), then eight rows' 64
          // bytes a store instruction
          const uint32_t stg = sO + (uint32_t)(warp * 2048);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float t16[16];
            tc_ld16(t_o(t) + lane_off + (uint32_t)c, t16);
#pragma unroll
            for (int x = 0; x < 16; ++x) chk = __fmaf_rn(t16[x], 0.0f, chk);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t addr = stg + (uint32_t)(lane * 64 + ((x ^ ((lane >> 1) & 3)) * 16));
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(t16[4 * x]),
                           "f"(t16[4 * x + 1]), "f"(t16[4 * x + 2]), "f"(t16[4 * x + 3])
                           : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int rr = 8 * x + (lane >> 2), qq = lane & 3;
              const uint32_t addr = stg + (uint32_t)(rr * 64 + ((qq ^ ((rr >> 1) & 3)) * 16));
              float4 val;
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(val.x), "=f"(val.y), "=f"(val.z), "=f"(val.w)
                           : "r"(addr)
                           : "memory");
              const int64_t to = __shfl_sync(0xffffffffu, at, rr);
              if (__shfl_sync(0xffffffffu, (int)in, rr))
                *reinterpret_cast<float4*>(f.po + to * D + c + qq * 4) = val;
            }
            __syncwarp();
          }
        }
        if (in) f.pml[lse_at * f.parts + f.split0 + it.split] = make_float2(m_ref, l);
      } else {
        const float inv = l == 0.0f ? 0.0f : recip_refined(l);
        const uint32_t stg = sO + (uint32_t)(warp * 2048);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t pkd[16];
#pragma unroll
          for (int hh = 0; hh < 32; hh += 16) {
            float t16[16];
            if (n > 0) {
              tc_ld16(t_o(t) + lane_off + (uint32_t)(c + hh), t16);
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x) t16[x] = 0.0f;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) chk = __fmaf_rn(t16[x], 0.0f, chk);
#pragma unroll
            for (int x = 0; x < 16; x += 2) pkd[(hh + x) / 2] = pack2<T>(t16[x] * inv, t16[x + 1] * inv);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t addr = stg + (uint32_t)(lane * 64 + ((x ^ ((lane >> 1) & 3)) * 16));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(pkd[4 * x]),
                         "r"(pkd[4 * x + 1]), "r"(pkd[4 * x + 2]), "r"(pkd[4 * x + 3])
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
            const int64_t to = __shfl_sync(0xffffffffu, ooff, rr);
            if (__shfl_sync(0xffffffffu, (int)in, rr)) *reinterpret_cast<uint4*>(o + to + c + qq * 8) = val;
          }
          __syncwarp();
        }
        if (in && lse != nullptr) lse[lse_at] = mod_lse(m_ref, l);
      }
      redo |= __any_sync(0xffffffffu, in && n > 0 && (chk != 0.0f || chk != chk || l != l));
      // the blocks that only the other tile has: in step with the issuing warp
      for (int b = n; b < nmax; ++b) {
        const int gg = g0 + b, rr = r0 + b;
        if (!tc_wait(bar(rnd(t, rr)), rpar(rr), f.max_polls, f.status)) {
          ok = false;
          atomicOr(f.status, DEV_TIMEOUT);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P + 2 * t + (gg & 1)));
      }
      advance(it);
    }
    if (redo) mod_fix_items<T, D, BIAS>(f, t, rt, q, k, v, o, lse);
  }
  if (!ok) atomicOr(f.status, DEV_TIMEOUT);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == S::ISSUE_WARP) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TCOLS) : "memory");
  }
}

}  // namespace smx
