// Decode attention over selected pages of the 4-bit cache.
//
// For unit (b, h) with the group's queries q_g (bf16) and tokens t of its selected pages, whose keys
// and values are k_t = gk sk_t ck_t and v_t = gv sv_t cv_t (codes c, one scale s per 16 dims):
//   x_gt = q_g . k_t / sqrt(128),  out_g = sum_t softmax_t(x_gt) v_t,  lse_g = log sum_t exp(x_gt)
// in one pass with a running maximum and sum.
//
// The products run on mma.sync m16n8k16 in f16 with fp32 accumulators, keys (then value dims) as M
// and the query heads as N.  Nothing is lost on the way in: a code times its e4m3 scale has at most
// six significant bits, so f16 holds it exactly, and a query row is scaled by a power of two into
// f16's range (its bf16 has 8 bits); the weights are split into f16 hi + lo parts (22 bits).
#include <math_constants.h>

#include "q4.cuh"

namespace spkv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
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
// Both halves of a pair the low (high) one.
__device__ __forceinline__ uint32_t dup_lo(uint32_t w) { return __byte_perm(w, w, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t w) { return __byte_perm(w, w, 0x3232); }

// The running maximum moves only when a score passes it by kSlack (log2 units): weights stay below
// 2^(kShift + kSlack) = 2^15, inside f16, and a weight's lo part resolves 2^-(24 + kShift) of it.
constexpr float kShift = 7.f, kSlack = 8.f;

constexpr int kRow = kHeadDim + 4;   // floats of a state's row in shared memory

// State of one warp for one unit: query columns n = 8 nt + (lane / 4) in the query fragments, 8 nt +
// 2 (lane % 4) + {0, 1} in everything else.  PACK (at most four query heads): columns 4..7 repeat the
// heads of columns 0..3; the weights' hi parts go into the first half and the lo parts into the
// second, so one MMA does both.
template <int NT, bool PACK>
struct Warp4 {
  float ref[NT][2];        // log2 weight reference: weights are 2^(x - ref)
  bool fresh;              // no token yet: ref is a stand-in
  float l[NT][2];          // this lane's part of their sum
  float O[8][NT][4];       // dims 16 r + 2 i, + 1 of m-tile i (r = lane / 4)
  uint32_t q[8][NT][2];    // query fragments, f16
  float scale[NT][2];      // scores to log2 units, per column

  __device__ __forceinline__ void reset() {
    fresh = true;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[i][nt][e] = 0.f;
    }
  }

  // Query rows of one unit (G rows of 128 bf16 at q0), factor = gk / sqrt(128) log2 e.
  __device__ __forceinline__ void load_q(const uint16_t* q0, int G, float factor, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = PACK ? (r & 3) : 8 * nt + r;
      uint32_t w[16];   // dims 32 c .. 32 c + 31
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
      // power of two that takes the largest magnitude into [2^13, 2^14); 1 for zero, infinity, NaN
      const int ex = static_cast<int>(m >> 7);
      const int field = ex == 0 || ex == 255 ? 127 : min(253, 267 - ex);
      const float f = __uint_as_float(uint32_t(field) << 23), inv = __uint_as_float(uint32_t(254 - field) << 23);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t x = w[2 * ks + j];
          q[ks][nt][j] = pack_f16x2(bf16lo_to_f32(x) * f, bf16hi_to_f32(x) * f);
        }
      }
      // columns 2c, 2c + 1 of this n-tile are the rows of lanes 8c and 8c + 4
#pragma unroll
      for (int e = 0; e < 2; ++e) scale[nt][e] = factor * __shfl_sync(0xffffffffu, inv, 4 * (2 * c + e));
    }
  }

  // Tokens 32 half .. 32 half + 31 of the page-head at shared address `page`, of which `valid` (of all
  // 64) exist; nothing where none of these does.
  __device__ __forceinline__ void tokens(uint32_t page, int half, int valid, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const int left = valid - 32 * half;   // of these tokens
    if (left <= 0) return;
    const uint32_t mine = page + lane * 16, tiles = mine + half * 2048;
    const uint2 k2 = lds64(mine + kQ4KScale + half * 8);
    const uint32_t ksc[2] = {k2.x, k2.y};
    float y[2][NT][4];
    // ---- scores of the two 16-token tiles: rows r, r + 8 of a tile
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      const uint4 a4 = lds128(tiles + tg * 1024), b4 = lds128(tiles + tg * 1024 + 512);
      const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, bw[4] = {b4.x, b4.y, b4.z, b4.w};
      const uint32_t sa = e4m3_to_f16(ksc[tg]), sb = e4m3_to_f16(ksc[tg] >> 16);
      const uint32_t sas[2] = {dup_lo(sa), dup_hi(sa)}, sbs[2] = {dup_lo(sb), dup_hi(sb)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[tg][nt][e] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {   // 8 dims of either key: two k-steps
        uint32_t ka[4], kb[4];
        e2m1_to_f16(aw[w], ka);
        e2m1_to_f16(bw[w], kb);
#pragma unroll
        for (int j = 0; j < 4; ++j) ka[j] = hmul2(ka[j], sas[w >> 1]), kb[j] = hmul2(kb[j], sbs[w >> 1]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t a[4] = {ka[2 * s], kb[2 * s], ka[2 * s + 1], kb[2 * s + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(y[tg][nt], a, q[2 * w + s][nt][0], q[2 * w + s][nt][1]);
        }
      }
    }
    // ---- log2 of the weights; does any pass the slack?
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int tg = 0; tg < 2; ++tg) {
        fma_f32x2(y[tg][nt][0], y[tg][nt][1], y[tg][nt][0], y[tg][nt][1], scale[nt][0], scale[nt][1], -ref[nt][0], -ref[nt][1]);
        fma_f32x2(y[tg][nt][2], y[tg][nt][3], y[tg][nt][2], y[tg][nt][3], scale[nt][0], scale[nt][1], -ref[nt][0], -ref[nt][1]);
      }
      if (left < 32) {
#pragma unroll
        for (int tg = 0; tg < 2; ++tg)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * tg + r + 8 * (e >> 1) >= left) y[tg][nt][e] = -CUDART_INF_F;
      }
      float m = fmaxf(fmaxf(y[0][nt][0], y[0][nt][1]), fmaxf(y[0][nt][2], y[0][nt][3]));
      m = fmaxf(m, fmaxf(fmaxf(y[1][nt][0], y[1][nt][1]), fmaxf(y[1][nt][2], y[1][nt][3])));
      over |= m > kShift + kSlack;
    }
    if (fresh || __any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          float m = fmaxf(fmaxf(y[0][nt][cc], y[0][nt][cc + 2]), fmaxf(y[1][nt][cc], y[1][nt][cc + 2]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          // up only; from the start's reference to the first maximum whatever its sign
          const float d = fresh ? m - kShift : fmaxf(m - kShift, 0.f);
          const float f = fresh ? 0.f : exp2f(-d);
          ref[nt][cc] += d;
          l[nt][cc] *= f;
#pragma unroll
          for (int tg = 0; tg < 2; ++tg) y[tg][nt][cc] -= d, y[tg][nt][cc + 2] -= d;
#pragma unroll
          for (int i = 0; i < 8; ++i) O[i][nt][cc] *= f, O[i][nt][cc + 2] *= f;
        }
    }
    // ---- weights, their sum, and as B fragments (hi and lo parts)
    uint32_t ph[2][NT][2], pl[PACK ? 1 : 2][NT][2];
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = ex2(y[tg][nt][e]);
        add_f32x2(l[nt][0], l[nt][1], w[0], w[1]);
        add_f32x2(l[nt][0], l[nt][1], w[2], w[3]);
        const uint32_t h0 = pack_f16x2(w[0], w[1]), h1 = pack_f16x2(w[2], w[3]);
        const uint32_t l0 = pack_f16x2(w[0] - f16lo(h0), w[1] - f16hi(h0));
        const uint32_t l1 = pack_f16x2(w[2] - f16lo(h1), w[3] - f16hi(h1));
        if (PACK) {
          ph[tg][nt][0] = movmatrix_trans(c < 2 ? h0 : l0);
          ph[tg][nt][1] = movmatrix_trans(c < 2 ? h1 : l1);
        } else {
          ph[tg][nt][0] = movmatrix_trans(h0);
          ph[tg][nt][1] = movmatrix_trans(h1);
          pl[PACK ? 0 : tg][nt][0] = movmatrix_trans(l0);
          pl[PACK ? 0 : tg][nt][1] = movmatrix_trans(l1);
        }
      }
    }
    // ---- O^T += V^T P^T, half of the block's 16 dims at a time.  The products go into fresh
    // accumulators, added to O rounded to nearest: the tensor core cuts off what an addition shifts
    // out, an error that would grow with every page of a long list.
    const uint2 v2 = lds64(mine + kQ4VScale + half * 8);
    const uint32_t vsc[2] = {v2.x, v2.y};
    uint32_t sa[2], sb[2];
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      sa[tg] = e4m3_to_f16(vsc[tg]);
      sb[tg] = e4m3_to_f16(vsc[tg] >> 16);
      if (left < 32) {   // scales behind the last token may hold anything: weight 0 times them must be 0
        const int t = 16 * tg + 2 * c;
        sa[tg] = (t < left ? sa[tg] & 0xFFFFu : 0u) | (t + 1 < left ? sa[tg] & 0xFFFF0000u : 0u);
        sb[tg] = (t + 8 < left ? sb[tg] & 0xFFFFu : 0u) | (t + 9 < left ? sb[tg] & 0xFFFF0000u : 0u);
      }
    }
    uint4 va[2], vb[2];   // tokens 2c, 2c + 1 (va) and 8 + 2c, 9 + 2c (vb) of a tile, block r
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) va[tg] = lds128(tiles + kQ4V + tg * 1024), vb[tg] = lds128(tiles + kQ4V + tg * 1024 + 512);
#pragma unroll
    for (int w = 0; w < 2; ++w) {   // m-tiles 4w .. 4w + 3
      float acc[4][NT][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
#pragma unroll
      for (int tg = 0; tg < 2; ++tg) {
        const uint32_t a0 = w ? va[tg].y : va[tg].x, a1 = w ? va[tg].w : va[tg].z;
        const uint32_t b0 = w ? vb[tg].y : vb[tg].x, b1 = w ? vb[tg].w : vb[tg].z;
        // token pairs of one dim in a byte: even dims, odd dims
        uint32_t ea[4], oa[4], eb[4], ob[4];
        e2m1_to_f16((a0 & 0x0F0F0F0Fu) | ((a1 << 4) & 0xF0F0F0F0u), ea);
        e2m1_to_f16(((a0 >> 4) & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u), oa);
        e2m1_to_f16((b0 & 0x0F0F0F0Fu) | ((b1 << 4) & 0xF0F0F0F0u), eb);
        e2m1_to_f16(((b0 >> 4) & 0x0F0F0F0Fu) | (b1 & 0xF0F0F0F0u), ob);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a[4] = {hmul2(ea[i], sa[tg]), hmul2(oa[i], sa[tg]), hmul2(eb[i], sb[tg]), hmul2(ob[i], sb[tg])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(acc[i][nt], a, ph[tg][nt][0], ph[tg][nt][1]);
            if (!PACK) mma_f16_16816(acc[i][nt], a, pl[PACK ? 0 : tg][nt][0], pl[PACK ? 0 : tg][nt][1]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          add_f32x2(O[4 * w + i][nt][0], O[4 * w + i][nt][1], acc[i][nt][0], acc[i][nt][1]);
          add_f32x2(O[4 * w + i][nt][2], O[4 * w + i][nt][3], acc[i][nt][2], acc[i][nt][3]);
        }
    }
    fresh = false;
  }

  // The warp's state as (reference, sum, O) of every column, to shared memory.  Dim 16 r + 2 i (+ 1)
  // goes to place 16 i + 2 r (+ 1) of a row of kRow floats, so that the stores meet no bank twice.
  __device__ __forceinline__ void store(float* m, float* sum, float (*o)[kRow], int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float s = l[nt][cc];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int col = 8 * nt + 2 * c + cc;
        if (r == 0 && (!PACK || c < 2)) {
          m[col] = fresh ? -CUDART_INF_F : ref[nt][cc];
          sum[col] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float u = O[i][nt][cc], v = O[i][nt][cc + 2];
          if (PACK) {   // hi part (columns 0..3) and lo part (4..7) of the same weights
            u += __shfl_xor_sync(0xffffffffu, u, 2);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
          }
          if (!PACK || c < 2) *reinterpret_cast<float2*>(&o[col][16 * i + 2 * r]) = make_float2(u, v);
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

// CTA shape: W consumer warps in pairs (a pair takes a page, 32 tokens each), a producer warp, an
// epilogue warp; NS page stages, NB state buffers.  More stages than pairs keep copies in flight while
// pages are worked on: with a page to a warp, 14 pages held the 16 stages and loads and arithmetic
// took turns (70 us a call of 32 requests x 65 pages x 8 kv heads).
template <int NT, bool PACK>
struct Cfg {
  static constexpr int W = NT == 1 ? 14 : 6;
  static constexpr int NS = NT == 1 ? 14 : 15;
  static constexpr int NB = PACK ? 2 : 1;
  static constexpr int kCols = PACK ? 4 : 8 * NT;
  static constexpr int kThreads = (W + 2) * 32;
  // A stage's pages all go to one pair, so that nobody waits for a phase of its barriers before the
  // one before it has ended: a wait tells phases apart by their parity only.
  static_assert(NS % (W / 2) == 0 && NS <= 32, "stages");
};
constexpr int kMaxUnits = 4096;
constexpr int kDesc = 512;   // page descriptors: those ahead of the copies and those of pages still worked on

template <int NT, bool PACK>
struct SmemQ4 {
  using C = Cfg<NT, PACK>;
  uint8_t stage[C::NS][kQ4Page];
  float o[C::NB][C::W][C::kCols][kRow];
  float m[C::NB][C::W][8 * NT];
  float l[C::NB][C::W][8 * NT];
  uint2 desc[kDesc];         // page j at j % kDesc: its place in the pool; valid tokens, unit - u0 << 7, segment << 19
  uint64_t full[C::NS];      // producer -> consumer (the copy's bytes)
  uint64_t empty[C::NS];     // consumer pair -> producer
  uint64_t done[C::NB];      // consumers -> epilogue: every warp's state of a segment (count W)
  uint64_t free_[C::NB];     // epilogue -> consumers
  int scan[C::kThreads / 32];
  int last[2];
  int prefix[kMaxUnits + 1];
};

// What the merges need of a call.
struct Merge {
  float* out;
  float* lse;
  float* ws_m;
  float* ws_l;
  float* ws_o;
};
// Lane `ln` of 32's four places of a merged row (places 4 ln .. are dims d, d + 1, d + 16, d + 17) as output.
__device__ __forceinline__ void write_row(const Merge& g, int64_t row, int ln, float M, float L, float4 acc, float gv) {
  const float k = L == 0.f ? 0.f : gv / L;   // no valid page: zeros
  float* o = g.out + row * kHeadDim + 32 * (ln & 3) + 2 * (ln >> 2);
  *reinterpret_cast<float2*>(o) = make_float2(acc.x * k, acc.y * k);
  *reinterpret_cast<float2*>(o + 16) = make_float2(acc.z * k, acc.w * k);
  if (ln == 0) g.lse[row] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
}

// The pages of all units form one sequence of T pages, dealt evenly to N CTAs in order: a CTA's segments
// are the units that it meets there.  All threads look up the CTA's pages (512 at a time), the producer
// warp streams each page-head with one bulk copy into a ring of stages, lane s owning stage s (one lane
// issuing for all took 560 to 930 cycles a page); consumer pair i takes pages i, i + W / 2, .. and, at
// each change of segment, leaves its warps' states in shared memory and goes on; the epilogue warp merges
// them into the output, or into the workspace for a unit that spans CTAs (a CTA has at most two such:
// its first and its last).  The last segment is merged by all threads.  The CTA that arrives last at a
// spanning unit merges its parts in CTA order, so the result does not depend on which one that is.
// ALIGNED: CTA u takes unit u, no sequence.
template <int NT, bool PACK, bool ALIGNED>
__global__ void __launch_bounds__(Cfg<NT, PACK>::kThreads, 1) attn_q4_kernel(const __grid_constant__ AttnQ4Params p4) {
  using C = Cfg<NT, PACK>;
  constexpr int W = C::W, NS = C::NS, NB = C::NB;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SmemQ4<NT, PACK>& S = *reinterpret_cast<SmemQ4<NT, PACK>*>(smem_raw);
  const AttnParams& p = p4.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int U = p.B * p.Hk, cta = blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 2);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&S.done[i], W);
      mbar_init(&S.free_[i], 1);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();

  auto count = [&](int u) { return max(0, min(p.n_sel[u], p.sel_stride)); };
  auto row_of = [&](int u) { return int64_t(u / p.Hk) * p.Hq + (u % p.Hk) * p.G; };   // of a unit's first query head
  auto write_empty = [&](int u) {
    const int64_t row = row_of(u);
    for (int i = tid; i < p.G * kHeadDim; i += C::kThreads) p.out[row * kHeadDim + i] = 0.f;
    for (int i = tid; i < p.G; i += C::kThreads) p.lse[row + i] = -CUDART_INF_F;
  };
  int x0, x1, u0;               // this CTA's pages and the unit of the first
  int T = 0, N = 1;             // pages; CTAs that share them: no more than there are pages
  int share = 1, extra = 0;     // pages of a CTA, and how many CTAs take one more
  if (ALIGNED) {
    u0 = cta;
    x0 = 0;
    x1 = count(cta);
    if (tid == 0) {
      S.prefix[0] = 0;
      S.prefix[1] = x1;
    }
    __syncthreads();
    if (x1 == 0) {
      write_empty(cta);
      return;
    }
  } else {
    // each thread sums k consecutive units, then one scan of the threads' sums
    const int k = (U + C::kThreads - 1) / C::kThreads, c0 = min(U, tid * k), c1 = min(U, c0 + k);
    int own = 0;
    for (int u = c0; u < c1; ++u) {
      S.prefix[u] = own;
      own += count(u);
    }
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) S.scan[warp] = x;
    __syncthreads();
    constexpr int kW = C::kThreads / 32;
    const int ws = lane < kW ? S.scan[lane] : 0;
    const int at = x - own + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
    T = __reduce_add_sync(0xffffffffu, ws);
    for (int u = c0; u < c1; ++u) S.prefix[u] += at;
    if (tid == 0) S.prefix[U] = T;
    __syncthreads();
    for (int u = cta; u < U; u += gridDim.x)
      if (S.prefix[u + 1] == S.prefix[u]) write_empty(u);
    N = min(T, static_cast<int>(gridDim.x));
    if (cta >= N) return;
    share = T / N;
    extra = T - share * N;
    x0 = cta * share + min(cta, extra);
    x1 = x0 + share + (cta < extra ? 1 : 0);
  }
  const int base_u = ALIGNED ? cta : 0;   // unit of prefix[0]
  auto first_page = [&](int u) { return S.prefix[u - base_u]; };
  // the last unit that starts at or before page x: not an empty one
  auto unit_of = [&](int x) {
    if (ALIGNED) return cta;
    int lo = 0, hi = U;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (S.prefix[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const int n = x1 - x0;
  u0 = unit_of(x0);
  const int u_last = unit_of(x1 - 1);
  // segments before unit u
  auto seg_of = [&](int u) {
    int k = 0;
    for (int v = u0; v < u; ++v) k += first_page(v + 1) > first_page(v);
    return k;
  };
  const int n_seg = seg_of(u_last) + 1;
  // looks up the CTA's page j
  auto describe = [&](int j) {
    const int x = x0 + j, u = unit_of(x);
    int phys = 0;
    const int valid = page_of(p, u, u / p.Hk, x - first_page(u), phys);
    S.desc[j % kDesc] = make_uint2(static_cast<uint32_t>((u % p.Hk) * p.n_phys) + phys,
                                   valid | (u - u0) << 7 | seg_of(u) << 19);
  };
  // the first ring of descriptors: the copies and the consumers start with it
  if (tid < n) describe(tid);   // kThreads <= kDesc
  Warp4<NT, PACK> w;
  if (warp < W)   // the first unit's query rows, while the look-ups are on their way
    w.load_q(static_cast<const uint16_t*>(p.q) + row_of(u0) * kHeadDim, p.G, p.scale_log2 * p4.k_scale[u0 % p.Hk], lane);
  __syncthreads();
  const Merge mg{p.out, p.lse, p.ws_m, p.ws_l, p.ws_o};

  if (warp == W) {
    // ================================================================ producer warp
    int known = min(n, C::kThreads);             // descriptors [0, known) are written
    int j = lane < NS ? lane : INT32_MAX - NS;   // this lane's next page
    uint64_t idle = 0;
    for (;;) {
      const int slowest = __reduce_min_sync(0xffffffffu, j);
      if (slowest >= n) break;
      // 32 more pages may replace descriptors below slowest - NS only: a lane's last copied page, one
      // ring behind its next, may still be worked on
      if (known < n && known - slowest <= kDesc - 32 - NS) {
        if (known + lane < n) describe(known + lane);
        known = min(n, known + 32);
        __syncwarp();
      }
      const bool go = j < known && (j < NS || mbar_test_wait(&S.empty[lane], ((j / NS) - 1) & 1));
      if (go) {
        const uint2 d = S.desc[j % kDesc];
        const bool some = (d.y & 127u) != 0;
        mbar_arrive_expect_tx(&S.full[lane], some ? kQ4Page : 0);
        if (some) bulk_load(S.stage[lane], p4.pool + int64_t(d.x) * kQ4Page, kQ4Page, &S.full[lane]);
        j += NS;
      }
      if (__any_sync(0xffffffffu, go)) {
        idle = 0;
      } else {
        const uint64_t t = globaltimer_ns();
        if (idle == 0) idle = t;
        if (__any_sync(0xffffffffu, p.wait_ns == 0 || (t > idle && t - idle > p.wait_ns))) {
          if (lane == 0) flag_error(p.err, SPKV_DEVERR_TIMEOUT);
          break;
        }
      }
    }
    // no copy of this CTA is left in flight (with the full limit: copies end in microseconds)
    if (lane < NS && j >= NS) mbar_wait(&S.full[lane], ((j / NS) - 1) & 1);
  } else if (warp == W + 1) {
    // ================================================================ epilogue warp
    // merges the states of every segment but the last
    int u = u0;
    for (int seg = 0; seg < n_seg - 1; ++seg, ++u) {
      while (first_page(u + 1) == first_page(u)) ++u;
      const int buf = seg % NB;
      const float gv = p4.v_scale[u % p.Hk];
      if (!__all_sync(0xffffffffu, mbar_wait(&S.done[buf], (seg / NB) & 1, p.wait_ns))) {
        if (lane == 0) flag_error(p.err, SPKV_DEVERR_TIMEOUT);
        break;
      }
      const bool whole = first_page(u) >= x0;   // its end lies before the last segment
      const int64_t row = row_of(u);
      const int64_t slot = 2 * int64_t(cta);    // a first segment, if it is not whole
      for (int g = 0; g < p.G; ++g) {
        // lane w: warp w's reference and sum; a warp without a page is left out (a NaN sum is not)
        const float mw = lane < W ? S.m[buf][lane][g] : -CUDART_INF_F, lw = lane < W ? S.l[buf][lane][g] : 0.f;
        const bool in = mw != -CUDART_INF_F || lw != 0.f;
        const unsigned some = __ballot_sync(0xffffffffu, in);
        float M = mw;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float f = !in ? 0.f : mw == M ? 1.f : exp2f(mw - M);
        float L = f * lw;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const float fw = __shfl_sync(0xffffffffu, f, x);
          float4 o = *reinterpret_cast<const float4*>(&S.o[buf][x][g][4 * lane]);
          if (!(some >> x & 1)) o = make_float4(0.f, 0.f, 0.f, 0.f);
          acc.x += fw * o.x, acc.y += fw * o.y, acc.z += fw * o.z, acc.w += fw * o.w;
        }
        if (whole) {
          write_row(mg, row + g, lane, M, L, acc, gv);
        } else {
          *reinterpret_cast<float4*>(p.ws_o + (slot * 16 + g) * kHeadDim + 4 * lane) = acc;
          if (lane == 0) {
            p.ws_m[slot * 16 + g] = M;
            p.ws_l[slot * 16 + g] = L;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.free_[buf]);
    }
  } else {
    // ================================================================ consumer warps
    w.reset();
    int seg = 0;          // the segment that the state is of
    bool has = false;     // whether this warp had a page of it
    bool ok = true;
    // waits until the buffer of segment `seg` is free and puts the state there (none without a page)
    auto put = [&]() {
      const int buf = seg % NB, k = seg / NB;
      if (k > 0 && !__all_sync(0xffffffffu, mbar_wait(&S.free_[buf], (k - 1) & 1, p.wait_ns))) {
        if (lane == 0) flag_error(p.err, SPKV_DEVERR_TIMEOUT);
        ok = false;
        return;
      }
      if (has) {
        w.store(S.m[buf][warp], S.l[buf][warp], S.o[buf][warp], lane);
      } else if (lane < 8 * NT) {
        S.m[buf][warp][lane] = -CUDART_INF_F;
        S.l[buf][warp][lane] = 0.f;
      }
    };
    // moves on to segment `to`, leaving the states of those before it
    auto leave = [&](int to) {
      while (seg < to && ok) {
        put();
        if (!ok) return;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.done[seg % NB]);
        if (has) w.reset();
        has = false;
        ++seg;
      }
    };
    for (int j = warp >> 1; j < n && ok; j += W / 2) {
      const int s = j % NS;
      if (!__all_sync(0xffffffffu, mbar_wait(&S.full[s], (j / NS) & 1, p.wait_ns))) {
        if (lane == 0) flag_error(p.err, SPKV_DEVERR_TIMEOUT);
        ok = false;
        break;
      }
      const uint32_t d = S.desc[j % kDesc].y;
      leave(d >> 19);
      if (!ok) break;
      if (!has) {
        if (seg > 0) {
          const int u = u0 + (d >> 7 & 4095);
          w.load_q(static_cast<const uint16_t*>(p.q) + row_of(u) * kHeadDim, p.G, p.scale_log2 * p4.k_scale[u % p.Hk], lane);
        }
        has = true;
      }
      if (d & 127) w.tokens(smem_u32(S.stage[s]), warp & 1, d & 127, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.empty[s]);
    }
    leave(n_seg - 1);
    if (ok) put();   // the last segment's, for the merge below
  }

  // ---- the last segment, by all threads.  (Every CTA goes on to arrive at the units that it shares,
  // whatever its waits did, so that the counters are zero again after the call.)
  if (!ALIGNED && warp == W + 1) __threadfence();   // the epilogue warp's partial before the arrivals below
  __syncthreads();
  const bool whole = ALIGNED || (first_page(u_last) >= x0 && first_page(u_last + 1) <= x1);
  {
    const int buf = (n_seg - 1) % NB;
    const int64_t row = row_of(u_last), slot = 2 * int64_t(cta) + (n_seg > 1 ? 1 : 0);
    for (int x = tid; x < p.G * 32; x += C::kThreads) {
      const int g = x >> 5;   // a warp's lanes share it
      float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) M = fmaxf(M, S.m[buf][k][g]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float mk = S.m[buf][k][g], lk = S.l[buf][k][g];
        float4 o = *reinterpret_cast<const float4*>(&S.o[buf][k][g][4 * lane]);
        const bool in = mk != -CUDART_INF_F || lk != 0.f;
        const float f = !in ? 0.f : mk == M ? 1.f : exp2f(mk - M);
        if (!in) o = make_float4(0.f, 0.f, 0.f, 0.f);
        L += f * lk;
        acc.x += f * o.x, acc.y += f * o.y, acc.z += f * o.z, acc.w += f * o.w;
      }
      if (whole) {
        write_row(mg, row + g, lane, M, L, acc, p4.v_scale[u_last % p.Hk]);
      } else {
        *reinterpret_cast<float4*>(p.ws_o + (slot * 16 + g) * kHeadDim + 4 * lane) = acc;
        if (lane == 0) {
          p.ws_m[slot * 16 + g] = M;
          p.ws_l[slot * 16 + g] = L;
        }
      }
    }
  }
  if (ALIGNED) return;

  // ---- units that span CTAs: the last CTA to arrive merges
  auto cta_of = [&](int x) {
    const int big = extra * (share + 1);
    return x < big ? x / (share + 1) : extra + (x - big) / share;
  };
  auto parts = [&](int u, int& c0) {
    c0 = cta_of(first_page(u));
    return cta_of(first_page(u + 1) - 1) - c0 + 1;
  };
  if (!whole) __threadfence();
  __syncthreads();
  if (tid < 2) {
    const int u = tid == 0 ? u0 : u_last;
    int c0, k = 0;
    if (tid == 0 || u_last != u0) k = parts(u, c0);
    S.last[tid] = k > 1 && atomicAdd(&p.ws_parts[u], 1) == k - 1;
    if (S.last[tid]) p.ws_parts[u] = 0;
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    if (!S.last[k]) continue;
    __threadfence();
    const int u = k == 0 ? u0 : u_last;
    int c0;
    const int np = parts(u, c0);
    const int late = first_page(u) > c0 * share + min(c0, extra) ? 1 : 0;   // not the first segment of c0
    const int64_t row = row_of(u);
    const float gv = p4.v_scale[u % p.Hk];
    for (int x = tid; x < p.G * 32; x += C::kThreads) {
      const int g = x >> 5;
      float M = -CUDART_INF_F, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kBatch = 8;
      for (int i0 = 0; i0 < np; i0 += kBatch) {
        float m[kBatch], l[kBatch];
        float4 o[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          m[q] = -CUDART_INF_F;
          l[q] = 0.f;
          o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + q < np) {
            const int c = c0 + i0 + q;   // the unit is its CTA's first segment, but perhaps where it begins
            const int64_t at = (2 * int64_t(c) + (c == c0 ? late : 0)) * 16 + g;
            m[q] = __ldcg(p.ws_m + at);
            l[q] = __ldcg(p.ws_l + at);
            o[q] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + at * kHeadDim) + lane);
          }
        }
        float mb = M;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) mb = fmaxf(mb, m[q]);
        const float f = M == mb ? 1.f : exp2f(M - mb);
        L *= f;
        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
        M = mb;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const float fq = m[q] == M ? 1.f : exp2f(m[q] - M);   // -inf: 0, or 1 times a zero (or NaN) state
          L += fq * l[q];
          acc.x += fq * o[q].x, acc.y += fq * o[q].y, acc.z += fq * o[q].z, acc.w += fq * o[q].w;
        }
      }
      write_row(mg, row + g, lane, M, L, acc, gv);
    }
  }
}

template <int NT, bool PACK>
cudaError_t launch_one(const spkv_cache* c, const AttnQ4Params& p, cudaStream_t st) {
  using C = Cfg<NT, PACK>;
  const int64_t U = int64_t(p.a.B) * p.a.Hk;
  // A unit that a CTA's pairs take in three rounds is not worth splitting, while every unit can have an
  // SM; else the pages of all units are dealt evenly, four at least to a CTA.
  if (U <= c->sm_count && p.a.sel_stride <= 3 * (C::W / 2))
    return launch_pdl(attn_q4_kernel<NT, PACK, true>, dim3(static_cast<unsigned>(U)), dim3(C::kThreads),
                      sizeof(SmemQ4<NT, PACK>), st, p);
  const int64_t want = (U * p.a.sel_stride + 3) / 4;
  return launch_pdl(attn_q4_kernel<NT, PACK, false>, dim3(static_cast<unsigned>(min(want, int64_t(c->sm_count)))),
                    dim3(C::kThreads), sizeof(SmemQ4<NT, PACK>), st, p);
}

template <int NT, bool PACK>
cudaError_t set_attr() {
  static_assert(sizeof(SmemQ4<NT, PACK>) <= 232448, "shared memory");
  const int bytes = static_cast<int>(sizeof(SmemQ4<NT, PACK>));
  const cudaError_t e = cudaFuncSetAttribute(attn_q4_kernel<NT, PACK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(attn_q4_kernel<NT, PACK, false>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

cudaError_t attn_q4_init_attributes() {
  cudaError_t e;
  if ((e = set_attr<1, true>()) != cudaSuccess) return e;
  if ((e = set_attr<1, false>()) != cudaSuccess) return e;
  return set_attr<2, false>();
}

cudaError_t launch_attn_q4(const spkv_cache* c, const AttnParams& a, cudaStream_t st) {
  AttnQ4Params p{a, c->pool4, c->k_scale, c->v_scale};
  if (a.G <= 4) return launch_one<1, true>(c, p, st);
  if (a.G <= 8) return launch_one<1, false>(c, p, st);
  return launch_one<2, false>(c, p, st);
}

}  // namespace spkv
