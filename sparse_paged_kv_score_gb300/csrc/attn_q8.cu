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
// weights are split into f16 hi + lo parts (22 bits).
#include "attn_units.cuh"
#include "q8.cuh"

namespace spkv {
namespace {

template <bool PACK>
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

  // A page-head at shared address `at`, of whose 64 tokens `valid` exist.  A sub-block without tokens is not touched:
  // its scale may be anything.
  __device__ __forceinline__ void page(uint32_t at, int valid, int lane) {
    const uint4 k4 = lds128(at + kQ8KScale), v4 = lds128(at + kQ8VScale);
    const float ks[4] = {__uint_as_float(k4.x), __uint_as_float(k4.y), __uint_as_float(k4.z), __uint_as_float(k4.w)};
    const float vs[4] = {__uint_as_float(v4.x), __uint_as_float(v4.y), __uint_as_float(v4.z), __uint_as_float(v4.w)};
    const uint32_t mine = at + lane * 16;
    if (valid > 48) return tiles<4>(mine, ks, vs, valid, lane);
#pragma unroll
    for (int tg = 0; tg < 3; ++tg)
      if (valid > 16 * tg) tiles<1>(mine + tg * 2048, ks + tg, vs + tg, valid - 16 * tg, lane);
  }

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

template <int CG, bool PACK>
struct Units8 : CtaShape<CG, PACK, PACK ? 4 : 5, PACK ? 4 : 20, PACK ? 3 : 2> {
  static constexpr int kPage = kQ8Page;
  static constexpr int kCtaPages = 8, kPartPages = 4, kUnitPages = 16, kEndPages = 8;
  using Params = AttnQ8Params;
  using Warp = Warp8<PACK>;
  static __device__ __forceinline__ float score_factor(const Params& p, int) { return p.a.scale_log2; }
  static __device__ __forceinline__ float value_factor(const Params&, int) { return 1.f; }
};

enum Mode { kDealt, kEither, kByUnit };

template <int CG, bool PACK, Mode MODE>
__global__ void __launch_bounds__(Units8<CG, PACK>::kThreads, Units8<CG, PACK>::kCtasPerSm)
    attn_q8_kernel(const __grid_constant__ AttnQ8Params p) {
  attend_units<Units8<CG, PACK>, MODE == kEither, MODE == kByUnit>(p);
}

template <int CG, bool PACK>
cudaError_t launch_one(const spkv_cache* c, const AttnQ8Params& p, cudaStream_t st) {
  return launch_units<Units8<CG, PACK>>(attn_q8_kernel<CG, PACK, kDealt>, attn_q8_kernel<CG, PACK, kEither>,
                                        attn_q8_kernel<CG, PACK, kByUnit>, c, p, st);
}

template <int CG, bool PACK>
cudaError_t set_attr() {
  return allow_smem<Units8<CG, PACK>>({attn_q8_kernel<CG, PACK, kDealt>, attn_q8_kernel<CG, PACK, kEither>,
                                       attn_q8_kernel<CG, PACK, kByUnit>});
}

}  // namespace

cudaError_t attn_q8_init_attributes() {
  cudaError_t e;
  if ((e = set_attr<1, true>()) != cudaSuccess) return e;
  if ((e = set_attr<1, false>()) != cudaSuccess) return e;
  return set_attr<2, false>();
}

cudaError_t launch_attn_q8(const spkv_cache* c, const AttnParams& a, cudaStream_t st) {
  const AttnQ8Params p{a, c->pool8, 1, 1};
  if (a.G <= 4) return launch_one<1, true>(c, p, st);
  if (a.G <= 8) return launch_one<1, false>(c, p, st);
  return launch_one<2, false>(c, p, st);
}

}  // namespace spkv
