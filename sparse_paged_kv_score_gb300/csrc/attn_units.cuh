// What the attention kernels over packed caches (4-bit and 8-bit pools, one blob of bytes for a page of one kv head) share:
// a warp's query fragments and running softmax, how the pages of all units are dealt to CTAs, brought to shared memory and
// merged, and how such a kernel is launched.  A format is a struct F with
//   CG, kByTokens   warps that share a page: each has some of its tokens, or eight of the query heads
//   W, TEAMS, kThreads, NS, L, kCols, kDesc, kWindow, kCtasPerSm   CTA shape, see CtaShape
//   kPage           bytes of a page-head
//   kCtaPages, kPartPages, kUnitPages, kEndPages   how pages are dealt, see below
//   Params          the kernel's parameters: a (AttnParams), pool, parts, part_pages
//   Held            what attend_units takes of them: a reference, or a copy (no call leaves the kernel, so that only the
//                   compiler's choice of registers differs)
//   Warp            a warp's arithmetic: reset(), load_q(), page() and store() as Softmax and the formats have them
//   score_factor(p, h), value_factor(p, h)   of kv head h: queries' scores to log2 units, values
#pragma once
#include <cuda_fp16.h>
#include <math_constants.h>

#include <cmath>
#include <initializer_list>

#include "common.cuh"

namespace spkv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with a zero accumulator going in.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float f16lo(uint32_t w) { return __half2float(__ushort_as_half(w & 0xFFFFu)); }
__device__ __forceinline__ float f16hi(uint32_t w) { return __half2float(__ushort_as_half(w >> 16)); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
// movmatrix_trans, without its ordering against everything volatile.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The running maximum moves only when a score passes it by kSlack (log2 units): weights stay below
// 2^(kShift + kSlack) = 2^15, inside f16, and a weight's lo part resolves 2^-(24 + kShift) of it.
constexpr float kShift = 7.f, kSlack = 8.f;

// A warp's state of a unit in shared memory: for each query head the reference (-inf: no token), the sum
// of weights and the weighted sum of values, its dims 16 r + 2 i (+ 1) at places 16 i + 2 r (+ 1) of a
// padded row, so that the stores meet no bank twice.
constexpr int kRow = kHeadDim + 4;
template <int COLS>
struct State {
  float o[COLS][kRow];
  float m[COLS];
  float l[COLS];
};

// Dims 32 c .. 32 c + 31 (c = lane % 4) of query row g (of G rows of 128 bf16 at q0; zeros behind), and the power of two that
// takes the row's largest magnitude into [2^13, 2^14) with its inverse; 1 for zero, infinity, NaN.
__device__ __forceinline__ float scaled_row(const uint16_t* q0, int g, int G, int c, uint32_t (&w)[16], float& inv) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = g < G ? *reinterpret_cast<const uint4*>(q0 + g * kHeadDim + 32 * c + 8 * j) : make_uint4(0, 0, 0, 0);
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = max(m, max((w[j] & 0x7FFFu), (w[j] >> 16) & 0x7FFFu));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int ex = static_cast<int>(m >> 7);
  const int field = ex == 0 || ex == 255 ? 127 : min(253, 267 - ex);
  inv = __uint_as_float(uint32_t(254 - field) << 23);
  return __uint_as_float(uint32_t(field) << 23);
}

// A warp's running softmax for up to eight query heads of one unit: query column lane / 4 in the query
// fragments, 2 (lane % 4) + {0, 1} in everything else.  PACK (at most four heads): columns 4..7 repeat
// the heads of columns 0..3; the weights' hi parts go into the first half and the lo parts into the
// second, so one MMA does both.
template <bool PACK>
struct Softmax {
  float ref[2];       // log2 weight reference: weights are 2^(x - ref)
  bool fresh;         // no token yet: ref is a stand-in
  float l[2];         // this lane's part of their sum
  float O[8][4];      // dims 16 r + 2 i, + 1 of m-tile i (r = lane / 4)
  uint32_t q[8][2];   // query fragments, f16
  float scale[2];     // scores to log2 units, per column

  __device__ __forceinline__ void reset() {
    fresh = true;
    ref[0] = ref[1] = 0.f;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[i][e] = 0.f;
  }

  // Query rows of one unit (G rows of 128 bf16 at q0), factor = gk / sqrt(128) log2 e.
  __device__ __forceinline__ void load_q(const uint16_t* q0, int G, float factor, int lane) {
    const int r = lane >> 2, c = lane & 3;
    uint32_t w[16];   // dims 32 c .. 32 c + 31
    float inv;
    const float f = scaled_row(q0, PACK ? (r & 3) : r, G, c, w, inv);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t x = w[2 * ks + j];
        q[ks][j] = pack_f16x2(bf16lo_to_f32(x) * f, bf16hi_to_f32(x) * f);
      }
    }
    // columns 2c, 2c + 1 are the rows of lanes 8c and 8c + 4
#pragma unroll
    for (int e = 0; e < 2; ++e) scale[e] = factor * __shfl_sync(0xffffffffu, inv, 4 * (2 * c + e));
  }
  // The state, to rows `col0` .. of a state in shared memory.
  template <int COLS>
  __device__ __forceinline__ void store(State<COLS>& to, int col0, int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      float s = l[cc];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      const int col = col0 + 2 * c + cc;
      if (r == 0 && (!PACK || c < 2)) {
        to.m[col] = fresh ? -CUDART_INF_F : ref[cc];
        to.l[col] = s;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float u = O[i][cc], v = O[i][cc + 2];
        if (PACK) {   // hi part (columns 0..3) and lo part (4..7) of the same weights
          u += __shfl_xor_sync(0xffffffffu, u, 2);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
        }
        if (!PACK || c < 2) *reinterpret_cast<float2*>(&to.o[col][16 * i + 2 * r]) = make_float2(u, v);
      }
    }
  }
};

// Physical page and valid tokens of entry i of unit (b, h)'s selection; 0 tokens for a bad entry.
__device__ __forceinline__ int page_of(const AttnParams& p, int u, int b, int i, int& phys) {
  const int lp = p.sel[int64_t(u) * p.sel_stride + i];
  uint32_t bad = 0;
  int valid = 0, ph = 0;
  if (lp < 0 || lp >= p.np_max) {
    bad = SPKV_DEVERR_PAGE_ID;
  } else {
    const int v = min(kPageTokens, p.seq_len[b] - kPageTokens * lp);
    if (p.slot) {
      const int sl = p.slot[int64_t(u) * p.sel_stride + i];
      ph = sl >= 0 && sl < p.n_slots ? b * p.n_slots + sl : -1;
      if (ph < 0) bad = SPKV_DEVERR_SLOT;
    } else {
      ph = page_lookup(p.page_table, p.np_max, p.pd, b, lp);
    }
    if (v <= 0) bad |= SPKV_DEVERR_PAGE_ID;
    else if (!bad && (ph < 0 || ph >= p.n_phys)) bad |= SPKV_DEVERR_PHYS;
    if (!bad) valid = v;
  }
  if (bad) {
    flag_error(p.err, bad);
    ph = 0;
  }
  phys = ph;
  return valid;
}

// CTA shape: four warps, of which CG share a page, up to COLS query heads, and a ring of NS page
// stages.  The barriers of the CTA's page j are number j % L of L, a multiple of the teams and of NS, so
// that all of a barrier's phases are waited for by the same warps: a wait tells phases by their parity.
template <int CG_, bool BY_TOKENS, int COLS, int NS_, int L_, int CTAS = 3>
struct CtaShape {
  static constexpr int CG = CG_;
  static constexpr bool kByTokens = BY_TOKENS;
  static constexpr int W = 4, TEAMS = W / CG, kThreads = W * 32;
  static constexpr int kStates = BY_TOKENS ? W : TEAMS;   // warps that share a page by heads share a state
  static constexpr int NS = NS_, L = L_;
  static constexpr int kCols = COLS;
  static constexpr int kDesc = kThreads;        // pages looked up at a time
  static constexpr int kWindow = 2 * kThreads;  // units among which they are looked up
  static constexpr int kCtasPerSm = CTAS;
  static_assert(L % NS == 0 && L % TEAMS == 0, "barriers");
};

template <class F>
struct SmemUnits {
  using C = F;
  uint8_t stage[C::NS][C::kPage];
  State<C::kCols> state[C::kStates];
  union {
    uint2 desc[C::kDesc];    // place in the pool; valid tokens, unit of the window << 8
    int scan[C::kThreads];   // until the first look-up: first page of each thread's units
  };
  uint64_t full[C::L];       // a page's copy has arrived
  int copied[C::NS];         // last page copied to a stage, -1: none
  int readers[C::NS];        // warps of a team that are through with it
  int first[C::kWindow + 1]; // first page of each unit of the window
  int sums[C::W];
  int last;
  float gv;                  // of the segment's unit: its head's value factor, its first query head
  int64_t row;
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Lane `ln`'s four places of a merged row (places 4 ln .. are dims d, d + 1, d + 16, d + 17) as output.
__device__ __forceinline__ void write_row(const AttnParams& p, int64_t row, int ln, float M, float L, float4 acc, float gv) {
  const float k = L == 0.f ? 0.f : gv / L;   // no valid page: zeros
  float* o = p.out + row * kHeadDim + 32 * (ln & 3) + 2 * (ln >> 2);
  *reinterpret_cast<float2*>(o) = make_float2(acc.x * k, acc.y * k);
  *reinterpret_cast<float2*>(o + 16) = make_float2(acc.z * k, acc.w * k);
  if (ln == 0) p.lse[row] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
}

// The pages of all units form one sequence of T pages, dealt evenly (with kEndPages places between units) to N
// CTAs, two or three to an SM so that one's look-ups and merges overlap the others' pages.  A CTA's segments are the
// units that it meets.  All threads look up its pages (128 at a time), each page-head arrives with one bulk
// copy, whoever is through with a stage copies its next page there, and at a segment's end the warps' states
// are merged in shared memory: into the output, or into the workspace for a unit that spans CTAs (a CTA has
// at most two such: its first and its last).  The CTA that arrives last at such a unit merges its parts in
// order, so the result does not depend on which one that is; every CTA arrives, so the counters are zero again
// after the call.  by_unit (units that fill the CTAs, of about one length): CTA c takes part c % parts of unit
// c / parts and meets no unit's end but its own.  Pages are dealt; or so or by unit as the pages turn out
// (EITHER); or by unit without counting other units' pages (BY_UNIT).  (With EITHER alone for the first two 256 units
// of 65 pages of a 4-bit cache take 0.5 us more.)
template <class F, bool EITHER, bool BY_UNIT>
__device__ __forceinline__ void attend_units(typename F::Held pf) {
  using C = F;
  constexpr int TEAMS = C::TEAMS, NS = C::NS, L = C::L;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SmemUnits<F>& S = *reinterpret_cast<SmemUnits<F>*>(smem_raw);
  const AttnParams& p = pf.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int team = warp / C::CG, piece = warp % C::CG, c8 = C::kByTokens ? 0 : 8 * piece;
  const int U = p.B * p.Hk, cta = blockIdx.x;
  if (tid < L) {
    mbar_init(&S.full[tid], 1);
    fence_mbar_init();
  }
  if (tid < NS) {
    S.copied[tid] = -1;
    S.readers[tid] = 0;
  }
  {
    // What the look-ups below will want, towards L2 while the kernel before this one ends (full lists
    // assumed; a prefetch reads nothing).
    const int64_t x = int64_t(U) * p.sel_stride * cta / gridDim.x, at = x + 32 * tid;
    const int u = static_cast<int>(x / p.sel_stride);
    if (cta == 0 || BY_UNIT)
      for (int i = 32 * tid; i < U; i += 32 * C::kThreads) prefetch_l2(p.n_sel + i);
    if (tid < 4 && at < int64_t(U) * p.sel_stride) {
      prefetch_l2(p.sel + at);
      if (p.slot) prefetch_l2(p.slot + at);
    }
    if (p.page_table && 32 * tid < p.np_max && u % p.Hk == 0) prefetch_l2(p.page_table + int64_t(u / p.Hk) * p.np_max + 32 * tid);
    if (tid < 2 * p.G)
      prefetch_l2(static_cast<const uint8_t*>(p.q) + (int64_t(u / p.Hk) * p.Hq + (u % p.Hk) * p.G) * (kHeadDim * 2) + tid * 128);
  }
  pdl_wait();
  pdl_trigger();

  auto count = [&](int u) { return u < U ? max(0, min(p.n_sel[u], p.sel_stride)) : 0; };
  auto row_of = [&](int u) { return int64_t(u / p.Hk) * p.Hq + (u % p.Hk) * p.G; };   // of a unit's first query head
  auto write_empty = [&](int u) {
    for (int i = tid; i < p.G * kHeadDim; i += C::kThreads) p.out[row_of(u) * kHeadDim + i] = 0.f;
    if (tid < p.G) p.lse[row_of(u) + tid] = -CUDART_INF_F;
  };
  // exclusive scan over the threads; `total` of all
  auto scan = [&](int own, int& total) {
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) S.sums[warp] = x;
    __syncthreads();
    total = 0;
    int before = 0;
#pragma unroll
    for (int w = 0; w < C::W; ++w) {
      before += w < warp ? S.sums[w] : 0;
      total += S.sums[w];
    }
    __syncthreads();
    return before + x - own;
  };
  // ---- this CTA's pages [x0, x1) of T, x1 as far as the window of units goes that it looks up; that window's first
  // unit and page.  Page x, of unit u, is place x + C::kEndPages u of those that are dealt.
  int x0, x1, base_u = 0, base_x = 0;
  bool last = true;           // x1 is the CTA's end
  bool by_unit = BY_UNIT;   // the CTA has a part of one unit
  int unit_parts = 1;
  int share = 1, extra = 0;   // places of a CTA, and how many CTAs take one more
  auto cta_begin = [&](int c) { return c * share + min(c, extra); };
  auto cta_of = [&](int x) {
    const int big = extra * (share + 1);
    return x < big ? x / (share + 1) : extra + (x - big) / share;
  };
  // first pages of the window's units
  auto look = [&]() {
    int total;
    const int a = count(base_u + 2 * tid), b = count(base_u + 2 * tid + 1);
    const int at = base_x + scan(a + b, total);
    S.first[2 * tid] = at;
    S.first[2 * tid + 1] = at + a;
    if (tid == 0) S.first[C::kWindow] = base_x + total;
    __syncthreads();
    return base_x + total;
  };
  // the first page at place v of the window or behind it
  auto page_at = [&](int v) {
    int m = 0;
#pragma unroll
    for (int o = C::kWindow / 2; o > 0; o >>= 1)
      if (S.first[m + o] + C::kEndPages * (base_u + m + o) <= v) m += o;
    return min(v - C::kEndPages * (base_u + m), S.first[m + 1]);
  };
  auto bound = [&]() {
    const int v = cta_begin(cta + 1);
    last = base_u + C::kWindow >= U || v < S.first[C::kWindow] + C::kEndPages * (base_u + C::kWindow);
    x1 = last ? page_at(v) : S.first[C::kWindow];
  };
  if (BY_UNIT) {
    base_u = cta / pf.parts;
    const int n = count(base_u), part = cta % pf.parts;
    unit_parts = min(pf.parts, (n + pf.part_pages - 1) / pf.part_pages);
    if (part == 0 && n == 0) write_empty(base_u);
    if (part >= unit_parts) return;
    x0 = n * part / unit_parts;   // (a CTA has at most 2 kUnitPages: no overflow)
    x1 = n * (part + 1) / unit_parts;
    if (tid == 0) S.first[0] = 0;
    for (int i = tid; i < C::kWindow; i += C::kThreads) S.first[i + 1] = n;
    __syncthreads();
  } else {
    int T;
    if (U <= C::kWindow) {
      T = look();
    } else {   // the sums of k consecutive units a thread, then the window that begins with a thread's
      const int k = (U + C::kThreads - 1) / C::kThreads;
      int own = 0;
      for (int u = tid * k; u < min(U, (tid + 1) * k); ++u) own += count(u);
      S.scan[tid] = scan(own, T);
      __syncthreads();
    }
    for (int u = cta; u < U; u += gridDim.x)
      if (count(u) == 0) write_empty(u);
    by_unit = EITHER && int64_t(T) * 8 >= int64_t(U) * p.sel_stride * 7;
    const int N = min(T, static_cast<int>(gridDim.x));
    if (cta >= (by_unit ? U * pf.parts : N)) return;
    const int V = T + C::kEndPages * U;
    share = V / N;
    extra = V - share * N;
    if (U > C::kWindow) {
      const int k = (U + C::kThreads - 1) / C::kThreads, v = cta_begin(cta);
      int t = 0;   // the last thread whose units begin at or before v
#pragma unroll
      for (int o = C::kThreads / 2; o > 0; o >>= 1)
        if (S.scan[t + o] + C::kEndPages * min((t + o) * k, U) <= v) t += o;
      base_u = t * k;
      base_x = S.scan[t];
      look();
    }
    if (by_unit) {
      const int f = S.first[cta / pf.parts], n = S.first[cta / pf.parts + 1] - f, part = cta % pf.parts;
      unit_parts = min(pf.parts, (n + pf.part_pages - 1) / pf.part_pages);
      if (part >= unit_parts) return;
      x0 = f + static_cast<int>(int64_t(n) * part / unit_parts);
      x1 = f + static_cast<int>(int64_t(n) * (part + 1) / unit_parts);
    } else {
      x0 = page_at(cta_begin(cta));
      bound();
    }
  }

  typename F::Warp w;
  int cur = -1;        // the unit that the warps' states are of
  bool ok = true;
  auto take = [&](int u) {   // the warps' states become those of unit u
    const int64_t row = row_of(u);
    if (tid == 0) {
      S.row = row;
      S.gv = F::value_factor(pf, u % p.Hk);
    }
    w.load_q(static_cast<const uint16_t*>(p.q) + (row + c8) * kHeadDim, p.G - c8, F::score_factor(pf, u % p.Hk), lane);
    w.reset();
    cur = u;
  };
  for (int x = x0; x < x1 || !last;) {
    // ---- as many pages as there are descriptors, and as the window has
    const int cnt = min(C::kDesc, x1 - x);          // none if the window's units are all empty
    int mine = 0;                                   // unit of page x + tid: the last that starts there or before
#pragma unroll
    for (int o = C::kWindow / 2; o > 0; o >>= 1)
      if (S.first[mine + o] <= x + tid) mine += o;
    const int j0 = x - x0;   // the CTA's page that is the first descriptor's
    auto copy = [&](int i, uint2 d) {   // descriptor i's page to its stage
      const int j = j0 + i, s = j % NS;
      const bool some = (d.y & 255) != 0;
      S.copied[s] = j;
      uint64_t* bar = &S.full[j % L];
      mbar_arrive_expect_tx(bar, some ? C::kPage : 0);
      if (some) bulk_load(S.stage[s], pf.pool + int64_t(d.x) * C::kPage, C::kPage, bar);
    };
    if (tid < cnt) {
      const int u = base_u + mine;
      int phys = 0;
      const uint32_t valid = page_of(p, u, u / p.Hk, x + tid - S.first[mine], phys);
      const uint2 d = make_uint2(static_cast<uint32_t>((u % p.Hk) * p.n_phys) + phys, valid | mine << 8);
      if (tid < NS && ok) copy(tid, d);
      S.desc[tid] = d;
    }
    if (cur < 0 && cnt > 0) {   // the first unit's queries come while the other threads look up
      int su = 0;
#pragma unroll
      for (int o = C::kWindow / 2; o > 0; o >>= 1)
        if (S.first[su + o] <= x) su += o;
      take(base_u + su);
    }
    __syncthreads();
    for (int kb = 0; kb < cnt;) {
      // ---- a segment: descriptors [kb, ke)
      const int su = S.desc[kb].y >> 8, u = base_u + su;
      const int f = S.first[su], e = S.first[su + 1], ke = min(cnt, e - x);
      if (u != cur) take(u);
      for (int i = kb + (team + TEAMS - (j0 + kb) % TEAMS) % TEAMS; i < ke && ok; i += TEAMS) {
        const int j = j0 + i, s = j % NS;
        ok = __all_sync(0xffffffffu, mbar_wait(&S.full[j % L], (j / L) & 1, p.wait_ns));
        if (!ok) break;
        w.page(smem_u32(S.stage[s]), S.desc[i].y & 255, lane, piece);
        __syncwarp();
        if (lane == 0 && i + NS < cnt) {
          bool free = true;
          if (C::CG > 1) {   // the last of the team
            __threadfence_block();
            free = atomicAdd(&S.readers[s], 1) % C::CG == C::CG - 1;
            __threadfence_block();
          }
          if (free) copy(i + NS, S.desc[i + NS]);
        }
        __syncwarp();
      }
      if (!ok && lane == 0) flag_error(p.err, SPKV_DEVERR_TIMEOUT);
      kb = ke;
      if (x + ke < min(e, x1)) break;   // it goes on with the next descriptors
      // ---- its end: the warps' states merged, a warp taking a query head at a time
      w.store(S.state[C::kByTokens ? warp : team], c8, lane);
      w.reset();   // nothing of it is kept over the merges
      const int gap = C::kEndPages * u;
      const bool whole = f >= x0 && e <= x1;   // a unit is in the window or out of it
      __syncthreads();
      const int64_t row = S.row;
      const float gv = S.gv;
      for (int g = warp; g < p.G; g += C::W) {
        float M = -CUDART_INF_F, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int t = 0; t < C::kStates; ++t) M = fmaxf(M, S.state[t].m[g]);
#pragma unroll
        for (int t = 0; t < C::kStates; ++t) {
          const float m = S.state[t].m[g], l = S.state[t].l[g];
          const float4 o = *reinterpret_cast<const float4*>(&S.state[t].o[g][4 * lane]);
          // no token: left out (a NaN sum is not)
          const float f = m == -CUDART_INF_F && l == 0.f ? 0.f : m == M ? 1.f : exp2f(m - M);
          sum += f * l;
          acc.x += f * o.x, acc.y += f * o.y, acc.z += f * o.z, acc.w += f * o.w;
        }
        if (whole) {
          write_row(p, row + g, lane, M, sum, acc, gv);
        } else {
          const int64_t at = (2 * cta + (!by_unit && f + gap > cta_begin(cta) ? 1 : 0)) * 16 + g;
          *reinterpret_cast<float4*>(p.ws_o + at * kHeadDim + 4 * lane) = acc;
          if (lane == 0) {
            p.ws_m[at] = M;
            p.ws_l[at] = sum;
          }
        }
      }
      __syncthreads();   // the states are free again; this CTA's part is written
      if (whole) continue;
      // ---- a unit of several CTAs: the last to arrive merges
      const int c0 = by_unit ? cta - cta % pf.parts : cta_of(f + gap);
      const int parts = by_unit ? unit_parts : cta_of(e - 1 + gap) - c0 + 1;
      const int late = !by_unit && f + gap > cta_begin(c0) ? 1 : 0;   // not the first unit of c0
      if (tid == 0) {
        int before;   // release: this CTA's part, which the barrier has ordered before; acquire: the others'
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.ws_parts + u) : "memory");
        S.last = before == parts - 1;
        if (S.last) p.ws_parts[u] = 0;
      }
      __syncthreads();
      if (S.last) {
        // A warp's heads together, kBatch parts at a time: all their rows are asked for before the first is
        // used.  Lane i has part i's reference and sum.
        constexpr int HG = (C::kCols + C::W - 1) / C::W, kBatch = HG == 4 ? 8 : 16;
        float M[HG], sum[HG];
        float4 acc[HG];
#pragma unroll
        for (int k = 0; k < HG; ++k) M[k] = -CUDART_INF_F, sum[k] = 0.f, acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto place = [&](int i, int k) {   // the unit is its CTA's first, but perhaps where it begins
          const int c = c0 + i;
          return int64_t(2 * c + (i == 0 ? late : 0)) * 16 + warp + C::W * k;
        };
        for (int i0 = 0; i0 < parts; i0 += kBatch) {
          float m[HG], l[HG];
          float4 o[HG][kBatch];
#pragma unroll
          for (int k = 0; k < HG; ++k) {
            const bool some = warp + C::W * k < p.G;
            m[k] = -CUDART_INF_F;
            l[k] = 0.f;
            if (some && lane < kBatch && i0 + lane < parts) {
              m[k] = __ldcg(p.ws_m + place(i0 + lane, k));
              l[k] = __ldcg(p.ws_l + place(i0 + lane, k));
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
              o[k][q] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (some && i0 + q < parts)
                o[k][q] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + place(i0 + q, k) * kHeadDim) + lane);
            }
          }
#pragma unroll
          for (int k = 0; k < HG; ++k) {
            float mb = fmaxf(M[k], m[k]);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, x));
            const float f0 = M[k] == mb ? 1.f : exp2f(M[k] - mb);
            const float f = m[k] == mb ? 1.f : exp2f(m[k] - mb);   // -inf: 0, or 1 times a zero (or NaN) state
            M[k] = mb;
            float s = f * l[k];
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            sum[k] = sum[k] * f0 + s;
            acc[k].x *= f0, acc[k].y *= f0, acc[k].z *= f0, acc[k].w *= f0;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
              const float fq = __shfl_sync(0xffffffffu, f, q);
              acc[k].x += fq * o[k][q].x, acc[k].y += fq * o[k][q].y;
              acc[k].z += fq * o[k][q].z, acc[k].w += fq * o[k][q].w;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < HG; ++k)
          if (warp + C::W * k < p.G) write_row(p, row + warp + C::W * k, lane, M[k], sum[k], acc[k], gv);
      }
    }
    if (__syncthreads_or(!ok)) ok = false;   // the descriptors and the window are free again
    x += cnt;
    if (x >= x1 && last) break;
    // the next window begins with the unit of the next page, or behind this one
    int next = C::kWindow;
    if (x < S.first[C::kWindow]) {
      next = 0;
#pragma unroll
      for (int o = C::kWindow / 2; o > 0; o >>= 1)
        if (S.first[next + o] <= x) next += o;
    }
    base_x = S.first[next];
    base_u += next;
    __syncthreads();
    if (!BY_UNIT) {   // one unit's window stays
      look();
      if (!by_unit) bound();
    }
  }
  // no copy is left in flight (with the full limit: copies end in microseconds)
  if (tid < NS && S.copied[tid] >= 0) mbar_wait(&S.full[S.copied[tid] % L], (S.copied[tid] / L) & 1);
}

// Launches one of a format's three kernels: pages dealt, either, by unit.
template <class F>
cudaError_t launch_units(void (*dealt)(typename F::Params), void (*either)(typename F::Params), void (*by_unit)(typename F::Params),
                         const spkv_cache* c, typename F::Params p, cudaStream_t st) {
  using C = F;
  const int64_t U = int64_t(p.a.B) * p.a.Hk, slots = int64_t(C::kCtasPerSm) * c->sm_count;
  const dim3 block(C::kThreads);
  const size_t smem = sizeof(SmemUnits<F>);
  // CTAs take parts of units (us, 4-bit cache; dealt / by unit): 2 units of 17 pages 10.3 / 6.8, 64 of 33 13.9 / 10.4, 128 of 17 14.5 /
  // 11.1, 256 of 5 13.4 / 8.3, 400 of 17 24.5 / 18.5.  Not where parts are long, as lists may then be of very different
  // lengths: 61 of 0 to 129 27 / 33; but there the kernel, which counts them, does where they are not: 64 of 129 26.0 / 25.7,
  // a step with 128 of 65 32.4 / 31.1.
  // A part's pages: the CTAs' time grows with them and the merge's with the parts, so with the root of the length
  // (129 pages in 16, 26, 33 parts 9.8, 10.2, 10.5; 500 in 16, 32, 63: 18.0, 15.3, 15.6).
  const int n = p.a.sel_stride;
  p.part_pages = max(C::kPartPages, static_cast<int>(0.6 * std::sqrt(static_cast<double>(n))));
  p.parts = static_cast<int>(min(int64_t(n + p.part_pages - 1) / p.part_pages, max(slots / U, int64_t(1))));
  const int64_t most = int64_t(C::kUnitPages) * p.parts * (U > C::kWindow ? 2 : 1);   // finding one's pages among more is slow
  if (U <= slots && n <= most)
    return launch_pdl(by_unit, dim3(static_cast<unsigned>(U * p.parts)), block, smem, st, p);
  // Four fifths of the CTAs; no more units than CTAs, which only a device with few SMs can have here.
  const bool fill = U <= C::kWindow && U <= slots && U * p.parts * 5 >= slots * 4;
  // Few long lists are not dealt to all CTAs (8, 16, 24 pages each: one list of 1000 24.0, 19.7, 20.1 us, one of 2000 39.5,
  // 26.4, 25.7, four of 900 27.7, 22.0, 20.1), many short ones are (256 of 17: 17.2 with 8, 22.4 with 24).
  const int least = max(C::kCtaPages, p.part_pages);
  const int64_t want = max((U * n + least - 1) / least, fill ? U * p.parts : 0);   // each part has its CTA
  const dim3 grid(static_cast<unsigned>(min(want, slots)));
  return launch_pdl(fill ? either : dealt, grid, block, smem, st, p);
}

template <class F>
cudaError_t allow_smem(std::initializer_list<void (*)(typename F::Params)> kernels) {
  static_assert(F::kCtasPerSm * (sizeof(SmemUnits<F>) + 1024) <= 233472, "shared memory");
  for (auto kernel : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(SmemUnits<F>)));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace spkv
