// What the rotating appends share: where a list's rows belong in their requests' pages, and a half-warp's rotation of a row
// (lane l of 16 holds dims 4l .. 4l + 3 and 64 + 4l .. + 3, so both halves of every pair).
#pragma once
#include "common.cuh"

namespace spkv {
namespace {

constexpr int kMaxWindow = 16;
constexpr int kMaxRows = kMaxWindow + kSubblock - 1;

struct alignas(16) RowInfo {
  int b;        // request, -1: no request's row
  int at;       // position in the request's context
  int phys;     // physical page, -1: not appended, or not by this CTA
  int rot;      // positions within the table
  int first;    // the request's first new position
  int end;      // one past its last
};

// Where list row i = base + lane belongs, for a whole warp; `bad` gets the error bits.  The requests' bounds and
// lengths are read 32 at a time and passed between the lanes, so that few reads wait for one another (a search
// by halves had log2 B of them in front of the CTA's first barrier).
__device__ __forceinline__ RowInfo find_row(const AppendRopeParams& p, int base, int lane, int (&axis_pos)[4], uint32_t& bad) {
  RowInfo r{-1, 0, -1, 0, 0, 0};
  const int i = base + lane;
  int b = i, f = i, e = i + 1, L;
  if (p.row_first) {
    int lo = 0;   // at most the request of row `base`, the last that begins there or before; it, with B > 31
    for (int span = p.B > 31 ? p.B : 1; span > 1;) {
      const int step = (span + 31) / 32, x = lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, x < span && p.row_first[lo + min(x, span - 1)] <= base);
      const int k = m ? 31 - __clz(m) : 0;
      lo += k * step;
      span = min(step, span - k * step);
    }
    const int bound = p.row_first[min(lo + lane, p.B)], len = p.seq_len[min(lo + lane, p.B - 1)];
    int k = 0;    // of the 32 from lo on, the last that begins at row i or before
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (__shfl_sync(0xffffffffu, bound, k + o) <= i && lo + k + o < p.B) k += o;
    b = lo + k;
    f = __shfl_sync(0xffffffffu, bound, k);
    e = __shfl_sync(0xffffffffu, bound, min(k + 1, 31));
    L = __shfl_sync(0xffffffffu, len, k);
    if (k == 31) {   // it, or one of those behind
      int hi = p.B;
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.row_first[mid] <= i) b = mid;
        else hi = mid;
      }
      f = p.row_first[b];
      e = p.row_first[b + 1];
      L = p.seq_len[b];
    }
    if (i >= p.n_rows || f > i || i >= e) return r;
  } else {
    if (lane >= p.window || i >= p.n_rows) return r;   // a row behind the window is of no request in it
    L = p.seq_len[b];
  }
  const int64_t at = int64_t(L) - (int64_t(e) - i), first = int64_t(L) - (int64_t(e) - f);
  if (at < 0 || at / kPageTokens >= p.np_max || at > INT32_MAX - kPageTokens) {
    bad |= SPKV_DEVERR_PAGE_ID;
  } else {
    r.b = b;
    r.at = static_cast<int>(at);
    r.first = static_cast<int>(max(first, int64_t(0)));
    r.end = L;
    const int ph = p.page_table[int64_t(b) * p.np_max + at / kPageTokens];
    if (ph >= 0 && ph < p.n_phys) r.phys = ph;
    else bad |= SPKV_DEVERR_PHYS;
  }
  r.rot = 1;
  if (p.cos_sin) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a >= p.n_axes) break;
      const int64_t x = p.pos ? int64_t(p.pos[int64_t(i) * p.n_axes + a]) : at;
      axis_pos[a] = static_cast<int>(x);
      if (x < 0 || x >= p.n_pos) r.rot = 0;
    }
    if (!r.rot) bad |= SPKV_DEVERR_POS;
  }
  return r;
}

// Dims 4l .. 4l + 3 and 64 + 4l .. + 3 of a bf16 row.
__device__ __forceinline__ uint4 load_pairs(const uint16_t* row, int l) {
  const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * l), b = *reinterpret_cast<const uint2*>(row + 64 + 4 * l);
  return make_uint4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ float2 pair(uint32_t w) { return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w)); }

// Cosines and sines of pairs 4l .. 4l + 3.
struct CosSin {
  float2 c[2], s[2];
};
// x: a row's dims 4l .. + 3, 64 + 4l .. + 3, rotated (with `turn`) in fp32: products and sums rounded one by
// one (packed f32x2 products and sums were contracted: 1 value in 10^5 came out otherwise).
__device__ __forceinline__ void rotate(uint4 v, const CosSin& t, bool turn, float (&x)[8]) {
  const uint32_t a[2] = {v.x, v.y}, b[2] = {v.z, v.w};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float2 lo = pair(a[j]), hi = pair(b[j]);
    if (turn) {
      const float2 y = lo, z = hi, c = t.c[j], s = t.s[j];
      lo.x = __fsub_rn(__fmul_rn(y.x, c.x), __fmul_rn(z.x, s.x));
      lo.y = __fsub_rn(__fmul_rn(y.y, c.y), __fmul_rn(z.y, s.y));
      hi.x = __fadd_rn(__fmul_rn(z.x, c.x), __fmul_rn(y.x, s.x));
      hi.y = __fadd_rn(__fmul_rn(z.y, c.y), __fmul_rn(y.y, s.y));
    }
    x[2 * j] = lo.x, x[2 * j + 1] = lo.y;
    x[4 + 2 * j] = hi.x, x[5 + 2 * j] = hi.y;
  }
}
// x rounded to bf16, as load_pairs gives a row.
__device__ __forceinline__ uint4 round_pairs(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store_pairs(uint16_t* row, int l, uint4 v) {
  *reinterpret_cast<uint2*>(row + 4 * l) = make_uint2(v.x, v.y);
  *reinterpret_cast<uint2*>(row + 64 + 4 * l) = make_uint2(v.z, v.w);
}

// Cosines and sines of pairs 4l .. 4l + 3 at a row's positions.
__device__ __forceinline__ CosSin load_turn(const AppendRopeParams& p, const int (&at)[4], int l) {
  CosSin t;
  if (p.quads) {   // the four pairs have one axis
    const int axis = static_cast<int>(p.pair_axis[l >> 3] >> (8 * (l & 7))) & 3;
    const float* cs = p.cos_sin + int64_t(at[axis]) * kHeadDim + 4 * l;
    const float4 c = *reinterpret_cast<const float4*>(cs), s = *reinterpret_cast<const float4*>(cs + 64);
    t.c[0] = make_float2(c.x, c.y), t.c[1] = make_float2(c.z, c.w);
    t.s[0] = make_float2(s.x, s.y), t.s[1] = make_float2(s.z, s.w);
  } else {
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pr = 4 * l + j;
      const int axis = static_cast<int>(p.pair_axis[pr >> 5] >> (2 * (pr & 31))) & 3;
      const float* cs = p.cos_sin + int64_t(at[axis]) * kHeadDim + pr;
      c[j] = cs[0];
      s[j] = cs[64];
    }
    t.c[0] = make_float2(c[0], c[1]), t.c[1] = make_float2(c[2], c[3]);
    t.s[0] = make_float2(s[0], s[1]), t.s[1] = make_float2(s[2], s[3]);
  }
  return t;
}

constexpr int kHeads = 4;   // query heads of a half-warp whose rows are asked for together

// Query head g of kv head h's group in list row i.
__device__ __forceinline__ const uint16_t* q_row(const AppendRopeParams& p, int h, int i, int g) {
  return p.q + int64_t(i) * p.q_stride + (h * p.G + g) * kHeadDim;
}

// Rotates heads sub, sub + step, .. of the group in list row i into q_out; q points to the first of them, qv holds kHeads of them
// as they came, t gets the row's cosines and sines.  (With q formed here again 8192 rows to bf16 pages took 42.2 us for 41.6.)
__device__ __forceinline__ void turn_queries(const AppendRopeParams& p, int h, int i, const int (&at)[4], int sub, int step, int l,
                                             const uint16_t* q, uint4 (&qv)[kHeads], CosSin& t) {
  t = load_turn(p, at, l);
  uint16_t* to = p.q_out + (int64_t(i) * p.Hq + h * p.G + sub) * kHeadDim;
  const int next = kHeads * step * kHeadDim;
  for (int g = sub; g < p.G; g += kHeads * step, q += next, to += next) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (g + k * step >= p.G) break;
      if (g != sub) qv[k] = load_pairs(q + k * step * kHeadDim, l);
      float x[8];
      rotate(qv[k], t, true, x);
      store_pairs(to + k * step * kHeadDim, l, round_pairs(x));
    }
  }
}

}  // namespace
}  // namespace spkv
