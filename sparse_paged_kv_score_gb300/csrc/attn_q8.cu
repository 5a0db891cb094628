// Decode attention over selected pages of the 8-bit cache.
//
// For unit (b, h) with the group's queries q_g (bf16) and tokens t of its selected pages, whose keys and values are
// k_t = (ck_t + 1/2) sk, v_t = (cv_t + 1/2) sv (codes c, one scale s for 16 tokens):
//   x_gt = q_g . k_t / sqrt(128) = sk (q_g . ck_t + sum(q_g) / 2) / sqrt(128)
//   out_g = sum_t p_gt v_t / sum_t p_gt,  p_gt = exp(x_gt)
//   sum_t p_gt v_t = sum over sub-blocks of sv (sum_t p_gt cv_t + (sum_t p_gt) / 2)
// in one pass with a running maximum and sum.  So a scale costs one product for 16 tokens of a head's scores and one for
// their weighted values, in fp32, and the halves two sums.
//
// The products run on mma.sync m16n8k16 in f16 with fp32 accumulators, keys (then value dims) as M and the query heads
// as N: f16 holds a code exactly, a query row is scaled into f16 as the 4-bit attention's are (attn_units.cuh), the
// weights are split into f16 hi + lo parts (22 bits).  They are below 2^15 (attn_units.cuh) and meet sv in fp32, so sums over N tokens stay
// in range for values up to 2^113 / N.
#include "attn_units.cuh"
#include "q8.cuh"

namespace spkv {
namespace {

// The tokens of a page-head at shared address `at`, of whose 64 `valid` exist, that are piece's of CG: to w.tiles<N>(address,
// scales, number), a sub-block of 16 a tile.  A sub-block without tokens is not touched: its scale may be anything.
template <int CG, class W>
__device__ __forceinline__ void page_of_tiles(W& w, uint32_t at, int valid, int lane, int piece) {
  constexpr int N = 4 / CG;
  valid -= 16 * N * piece;
  if (valid <= 0) return;
  const uint4 k4 = lds128(at + kQ8KScale), v4 = lds128(at + kQ8VScale);
  float ks[4] = {__uint_as_float(k4.x), __uint_as_float(k4.y), __uint_as_float(k4.z), __uint_as_float(k4.w)};
  float vs[4] = {__uint_as_float(v4.x), __uint_as_float(v4.y), __uint_as_float(v4.z), __uint_as_float(v4.w)};
  if (CG == 2 && piece) ks[0] = ks[2], ks[1] = ks[3], vs[0] = vs[2], vs[1] = vs[3];
  if (CG == 4 && piece) ks[0] = piece == 1 ? ks[1] : piece == 2 ? ks[2] : ks[3], vs[0] = piece == 1 ? vs[1] : piece == 2 ? vs[2] : vs[3];
  const uint32_t mine = at + lane * 16 + piece * (N * 2048);
  if (N == 1 || valid > 16 * (N - 1)) return w.template tiles<N>(mine, ks, vs, valid, lane);
#pragma unroll
  for (int tg = 0; tg < N - 1; ++tg)
    if (valid > 16 * tg) w.template tiles<1>(mine + tg * 2048, ks + tg, vs + tg, valid - 16 * tg, lane);
}

// Up to eight query heads, tokens (then value dims) as M and the heads as N.
template <bool PACK, int CG>
struct Warp8 : Softmax<PACK> {
  using Base = Softmax<PACK>;
  using Base::fresh;
  using Base::l;
  using Base::O;
  using Base::q;
  using Base::ref;
  using Base::scale;
  float half_q[2];   // half of a query row's sum, per column
  float b[2];        // this lane's part of the sum of sv times weight

  __device__ __forceinline__ void reset() {
    Base::reset();
    b[0] = b[1] = 0.f;
  }

  __device__ __forceinline__ void load_q(const uint16_t* q0, int G, float factor, int lane) {
    Base::load_q(q0, G, factor, lane);
    float s = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) s += (f16lo(q[ks][0]) + f16hi(q[ks][0])) + (f16lo(q[ks][1]) + f16hi(q[ks][1]));
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    const int c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) half_q[e] = 0.5f * __shfl_sync(0xffffffffu, s, 4 * (2 * c + e));
  }

  // Products of a 16-token tile's key codes with the queries; `tile` is this lane's shared address.
  __device__ __forceinline__ void scores(uint32_t tile, float (&y)[4]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 a4 = lds128(tile + j * 512), b4 = lds128(tile + 1024 + j * 512);
      const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, bw[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a[4] = {q8_f16_lo(aw[w]), q8_f16_lo(bw[w]), q8_f16_hi(aw[w]), q8_f16_hi(bw[w])};
        if (j == 0 && w == 0) mma_f16_16816_first(y, a, q[0][0], q[0][1]);
        else mma_f16_16816(y, a, q[4 * j + w][0], q[4 * j + w][1]);
      }
    }
  }

  // Scores of N tiles to log2 weights, -inf behind the last of `valid` tokens; raises the references where a weight
  // passes the slack.
  template <int N>
  __device__ __forceinline__ void refer(float (&y)[N][4], const float* ks, int valid, int lane) {
    const int r = lane >> 2;
#pragma unroll
    for (int tg = 0; tg < N; ++tg) {
      const float f0 = scale[0] * ks[tg], f1 = scale[1] * ks[tg];
      const float c0 = fmaf(half_q[0], f0, -ref[0]), c1 = fmaf(half_q[1], f1, -ref[1]);
      fma_f32x2(y[tg][0], y[tg][1], y[tg][0], y[tg][1], f0, f1, c0, c1);
      fma_f32x2(y[tg][2], y[tg][3], y[tg][2], y[tg][3], f0, f1, c0, c1);
    }
    if (valid < 16 * N) {
#pragma unroll
      for (int tg = 0; tg < N; ++tg)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * tg + r + 8 * (e >> 1) >= valid) y[tg][e] = -CUDART_INF_F;
    }
    float top = -CUDART_INF_F;
#pragma unroll
    for (int tg = 0; tg < N; ++tg) top = fmaxf(top, fmaxf(fmaxf(y[tg][0], y[tg][1]), fmaxf(y[tg][2], y[tg][3])));
    if (fresh || __any_sync(0xffffffffu, top > kShift + kSlack)) {
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float m = fmaxf(y[0][cc], y[0][cc + 2]);
#pragma unroll
        for (int tg = 1; tg < N; ++tg) m = fmaxf(m, fmaxf(y[tg][cc], y[tg][cc + 2]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        // up only; from the start's reference to the first maximum whatever its sign
        const float d = fresh ? m - kShift : fmaxf(m - kShift, 0.f);
        const float f = fresh ? 0.f : exp2f(-d);
        ref[cc] += d;
        l[cc] *= f;
        b[cc] *= f;
#pragma unroll
        for (int tg = 0; tg < N; ++tg) y[tg][cc] -= d, y[tg][cc + 2] -= d;
#pragma unroll
        for (int i = 0; i < 8; ++i) O[i][cc] *= f, O[i][cc + 2] *= f;
      }
    }
    fresh = false;
  }

  // O^T += sv V^T P^T of a 16-token tile with the weights 2^y; `tile` is this lane's shared address of its keys.
  __device__ __forceinline__ void weigh(uint32_t tile, const float (&y)[4], float vs, int lane) {
    const int c = lane & 3;
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ex2(y[e]);
    float s0 = w[0], s1 = w[1];
    add_f32x2(s0, s1, w[2], w[3]);
    add_f32x2(l[0], l[1], s0, s1);
    fma_f32x2(b[0], b[1], s0, s1, vs, vs, b[0], b[1]);
    const uint32_t h0 = pack_f16x2(w[0], w[1]), h1 = pack_f16x2(w[2], w[3]);
    const uint32_t l0 = pack_f16x2(w[0] - f16lo(h0), w[1] - f16hi(h0));
    const uint32_t l1 = pack_f16x2(w[2] - f16lo(h1), w[3] - f16hi(h1));
    const uint32_t ph0 = transposed(PACK && c >= 2 ? l0 : h0), ph1 = transposed(PACK && c >= 2 ? l1 : h1);
    uint32_t pl0 = 0, pl1 = 0;
    if (!PACK) pl0 = transposed(l0), pl1 = transposed(l1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 a4 = lds128(tile + kQ8V + j * 512), b4 = lds128(tile + kQ8V + 1024 + j * 512);
      const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, bw[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a[4] = {q8_f16_lo(aw[i]), q8_f16_hi(aw[i]), q8_f16_lo(bw[i]), q8_f16_hi(bw[i])};
        float acc[4];
        mma_f16_16816_first(acc, a, ph0, ph1);
        if (!PACK) mma_f16_16816(acc, a, pl0, pl1);
        float(&o)[4] = O[4 * j + i];
        fma_f32x2(o[0], o[1], acc[0], acc[1], vs, vs, o[0], o[1]);
        fma_f32x2(o[2], o[3], acc[2], acc[3], vs, vs, o[2], o[3]);
      }
    }
  }

  // N tiles at this lane's shared address, with their scales, of which `valid` tokens exist (in all N tiles some).
  template <int N>
  __device__ __forceinline__ void tiles(uint32_t mine, const float* ks, const float* vs, int valid, int lane) {
    float y[N][4];
#pragma unroll
    for (int tg = 0; tg < N; ++tg) scores(mine + tg * 2048, y[tg]);
    refer<N>(y, ks, valid, lane);
#pragma unroll
    for (int tg = 0; tg < N; ++tg) weigh(mine + tg * 2048, y[tg], vs[tg], lane);
  }

  __device__ __forceinline__ void page(uint32_t at, int valid, int lane, int piece) { page_of_tiles<CG>(*this, at, valid, lane, piece); }

  template <int COLS>
  __device__ __forceinline__ void store(State<COLS>& to, int col0, int lane) {
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {   // the halves; PACK: into the hi parts' columns, to which the lo parts are added
      float s = b[cc];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      s = PACK && (lane & 2) ? 0.f : 0.5f * s;
#pragma unroll
      for (int i = 0; i < 8; ++i) O[i][cc] += s, O[i][cc + 2] += s;
    }
    Base::store(to, col0, lane);
  }
};

// Up to sixteen query heads as M, tokens (then value dims) as N: a code is unpacked once for all of them, and the weights
// come out of the scores' products as the next products take them.  Lane 4 r + c has the heads r and r + 8.
template <int CG>
struct Warp8Wide {
  float ref[2];       // as Softmax's, of the two heads
  bool fresh;
  float l[2], b[2];
  float scale[2], half_q[2];
  float O[16][4];     // dims 32 c + i and 32 c + 16 + i of head r, of head r + 8
  uint32_t q[8][4];   // query fragments, f16

  __device__ __forceinline__ void reset() {
    fresh = true;
#pragma unroll
    for (int e = 0; e < 2; ++e) ref[e] = l[e] = b[e] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[i][e] = 0.f;
  }

  __device__ __forceinline__ void load_q(const uint16_t* q0, int G, float factor, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t w[16];   // dims 32 c .. 32 c + 31
      float inv;
      const float f = scaled_row(q0, r + 8 * e, G, c, w, inv);
      float s = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t x = pack_f16x2(bf16lo_to_f32(w[2 * ks + j]) * f, bf16hi_to_f32(w[2 * ks + j]) * f);
          q[ks][2 * j + e] = x;
          s += f16lo(x) + f16hi(x);
        }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      half_q[e] = 0.5f * s;
      scale[e] = factor * inv;
    }
  }

  // Products of a tile's key codes with the queries: y[n] has the tokens 8 n + 2 c, + 1 of head r, then of head r + 8.
  __device__ __forceinline__ void scores(uint32_t tile, float (&y)[2][4]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 k4 = lds128(tile + n * 1024 + j * 512);
        const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (j == 0 && w == 0) mma_f16_16816_first(y[n], q[0], q8_f16_lo(kw[0]), q8_f16_hi(kw[0]));
          else mma_f16_16816(y[n], q[4 * j + w], q8_f16_lo(kw[w]), q8_f16_hi(kw[w]));
        }
      }
  }

  template <int N>
  __device__ __forceinline__ void refer(float (&y)[N][2][4], const float* ks, int valid, int lane) {
    const int c = lane & 3;
#pragma unroll
    for (int tg = 0; tg < N; ++tg) {
      const float f0 = scale[0] * ks[tg], f1 = scale[1] * ks[tg];
      const float c0 = fmaf(half_q[0], f0, -ref[0]), c1 = fmaf(half_q[1], f1, -ref[1]);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float(&z)[4] = y[tg][n];
        fma_f32x2(z[0], z[1], z[0], z[1], f0, f0, c0, c0);
        fma_f32x2(z[2], z[3], z[2], z[3], f1, f1, c1, c1);
      }
    }
    if (valid < 16 * N) {
#pragma unroll
      for (int tg = 0; tg < N; ++tg)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * tg + 8 * n + 2 * c + (e & 1) >= valid) y[tg][n][e] = -CUDART_INF_F;
    }
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
    for (int tg = 0; tg < N; ++tg)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e >> 1] = fmaxf(m[e >> 1], y[tg][n][e]);
    if (fresh || __any_sync(0xffffffffu, fmaxf(m[0], m[1]) > kShift + kSlack)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = m[h];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float d = fresh ? x - kShift : fmaxf(x - kShift, 0.f);
        const float f = fresh ? 0.f : exp2f(-d);
        ref[h] += d;
        l[h] *= f;
        b[h] *= f;
#pragma unroll
        for (int tg = 0; tg < N; ++tg)
#pragma unroll
          for (int n = 0; n < 2; ++n) y[tg][n][2 * h] -= d, y[tg][n][2 * h + 1] -= d;
#pragma unroll
        for (int i = 0; i < 16; ++i) O[i][2 * h] *= f, O[i][2 * h + 1] *= f;
      }
    }
    fresh = false;
  }

  // O += sv P V of a tile with the weights 2^y.
  __device__ __forceinline__ void weigh(uint32_t tile, const float (&y)[2][4], float vs) {
    uint32_t ph[4], pl[4];   // tokens 8 n + 2 c, + 1 of head r + 8 h at 2 n + h
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float w0 = ex2(y[n][2 * h]), w1 = ex2(y[n][2 * h + 1]);
        s[h] += w0 + w1;
        const uint32_t hi = pack_f16x2(w0, w1);
        ph[2 * n + h] = hi;
        pl[2 * n + h] = pack_f16x2(w0 - f16lo(hi), w1 - f16hi(hi));
      }
    add_f32x2(l[0], l[1], s[0], s[1]);
    fma_f32x2(b[0], b[1], s[0], s[1], vs, vs, b[0], b[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 a4 = lds128(tile + kQ8V + j * 512), b4 = lds128(tile + kQ8V + 1024 + j * 512);
      const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, bw[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v0 = i & 1 ? q8_f16_hi(aw[i >> 1]) : q8_f16_lo(aw[i >> 1]);
        const uint32_t v1 = i & 1 ? q8_f16_hi(bw[i >> 1]) : q8_f16_lo(bw[i >> 1]);
        float acc[4];
        mma_f16_16816_first(acc, ph, v0, v1);
        mma_f16_16816(acc, pl, v0, v1);
        float(&o)[4] = O[8 * j + i];
        fma_f32x2(o[0], o[1], acc[0], acc[1], vs, vs, o[0], o[1]);
        fma_f32x2(o[2], o[3], acc[2], acc[3], vs, vs, o[2], o[3]);
      }
    }
  }

  template <int N>
  __device__ __forceinline__ void tiles(uint32_t mine, const float* ks, const float* vs, int valid, int lane) {
    float y[N][2][4];
#pragma unroll
    for (int tg = 0; tg < N; ++tg) scores(mine + tg * 2048, y[tg]);
    refer<N>(y, ks, valid, lane);
#pragma unroll
    for (int tg = 0; tg < N; ++tg) weigh(mine + tg * 2048, y[tg], vs[tg]);
  }

  __device__ __forceinline__ void page(uint32_t at, int valid, int lane, int piece) { page_of_tiles<CG>(*this, at, valid, lane, piece); }

  template <int COLS>
  __device__ __forceinline__ void store(State<COLS>& to, int, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = l[h], x = b[h];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x *= 0.5f;
      if (c == 0) {
        to.m[r + 8 * h] = fresh ? -CUDART_INF_F : ref[h];
        to.l[r + 8 * h] = s;
      }
#pragma unroll
      for (int i = 0; i < 16; i += 2)   // dims 32 c + i, + 1 and 32 c + 16 + i, + 1
        *reinterpret_cast<float4*>(&to.o[r + 8 * h][8 * i + 4 * c]) =
            make_float4(O[i][2 * h] + x, O[i + 1][2 * h] + x, O[i][2 * h + 1] + x, O[i + 1][2 * h + 1] + x);
    }
  }
};

// HEADS: query heads at most, 4, 8 or 16.  Two warps share a page by tokens: a page is half as long in its stage, and few long
// lists end sooner (us, 1 / 2 / 4 warps a page: one request of 129 pages x 8 heads 12.6 / 11.9 / 12.9, 256 units of 65 pages 51.1 /
// 51.3 / 52.9).  Up to eight heads could be rows of the wide form too, but half of its first product would be zeros; sixteen
// as columns of two warps, each unpacking every page, took 71 us for 256 units of 65 pages, the wide form takes 60.
// Three CTAs an SM where registers and stages allow it; the wide form with three (168 registers, fewer stages) took 67 to 76.
template <int HEADS>
struct Shape8;
template <>
struct Shape8<4> : CtaShape<2, true, 4, 4, 4, 3> {
  using Warp = Warp8<true, CG>;
};
template <>
struct Shape8<8> : CtaShape<2, true, 8, 5, 10, 2> {
  using Warp = Warp8<false, CG>;
};
template <>
struct Shape8<16> : CtaShape<2, true, 16, 4, 4, 2> {
  using Warp = Warp8Wide<CG>;
};

template <int HEADS>
struct Units8 : Shape8<HEADS> {
  static constexpr int kPage = kQ8Page;
  // As the 4-bit attention's, with parts of two pages (2 units of 17 pages, parts of 2 / 3 / 4 / 6: 6.4 / 7.0 / 6.9 / 7.6 us); 8, 4, 2
  // places at a unit's end: 61 lists of up to 129 pages 26.0, 26.6, 27.9 us, the rest alike.
  static constexpr int kCtaPages = 8, kPartPages = 2, kUnitPages = 16, kEndPages = 8;
  using Params = AttnQ8Params;
  using Held = const AttnQ8Params&;   // (a copy: 64 units of 129 pages, 16 heads 37.0 us for 36.5; 4 and 8 heads within 0.2)
  static __device__ __forceinline__ float score_factor(const Params& p, int) { return p.a.scale_log2; }
  static __device__ __forceinline__ float value_factor(const Params&, int) { return 1.f; }
};

// Measured (GB300, from a replayed graph): 256 units of 65 pages, 4 heads 50.1 us = 275 MB at 5.5 TB/s (0.82 of the copy rate);
// 8 heads 49.1, 16 heads 60.2; 61 lists of up to 129 pages, 16 heads 26 us; 2 of 17 pages 6.4.  Times of 96 to 300 units lie on
// a line of 6.37 TB/s (0.95 of the copy rate) behind 8 us: lengths, lists, page table and first page read one after the
// other, and the CTAs' ends.  The 61 ragged lists (4138 pages, 9.8 us of bytes) take 19.4 us with 4 heads and 20.7 with 8, so 10 us and
// more of the 26 with 16 are not the heads'.  A page is 1000, 1030, 1300 instructions of its two warps together (4, 8, 16 heads) and a CTA's start,
// ends and merges 6400, 6600, 9100 beside its pages: a third of the ragged case's 8.2 million with 16 heads.  The
// rest of those is chains that two warps a scheduler (255 registers) do not hide: a third of the slots issue.
enum Mode { kDealt, kEither, kByUnit };

template <int HEADS, Mode MODE>
__global__ void __launch_bounds__(Units8<HEADS>::kThreads, Units8<HEADS>::kCtasPerSm)
    attn_q8_kernel(const __grid_constant__ AttnQ8Params p) {
  attend_units<Units8<HEADS>, MODE == kEither, MODE == kByUnit>(p);
}

template <int HEADS>
cudaError_t launch_one(const spkv_cache* c, const AttnQ8Params& p, cudaStream_t st) {
  return launch_units<Units8<HEADS>>(attn_q8_kernel<HEADS, kDealt>, attn_q8_kernel<HEADS, kEither>, attn_q8_kernel<HEADS, kByUnit>,
                                     c, p, st);
}

template <int HEADS>
cudaError_t set_attr() {
  return allow_smem<Units8<HEADS>>({attn_q8_kernel<HEADS, kDealt>, attn_q8_kernel<HEADS, kEither>, attn_q8_kernel<HEADS, kByUnit>});
}

}  // namespace

cudaError_t attn_q8_init_attributes() {
  cudaError_t e;
  if ((e = set_attr<4>()) != cudaSuccess) return e;
  if ((e = set_attr<8>()) != cudaSuccess) return e;
  return set_attr<16>();
}

cudaError_t launch_attn_q8(const spkv_cache* c, const AttnParams& a, cudaStream_t st) {
  const AttnQ8Params p{a, c->pool8, 1, 1};
  if (a.G <= 4) return launch_one<4>(c, p, st);
  if (a.G <= 8) return launch_one<8>(c, p, st);
  return launch_one<16>(c, p, st);
}

}  // namespace spkv
