// Decode attention over selected pages of the 4-bit cache.
//
// For unit (b, h) with the group's queries q_g (bf16) and tokens t of its selected pages, whose keys
// and values are k_t = gk sk_t ck_t and v_t = gv sv_t cv_t (codes c, one scale s per 16 dims):
//   x_gt = q_g . k_t / sqrt(128),  out_g = sum_t softmax_t(x_gt) v_t,  lse_g = log sum_t exp(x_gt)
// in one pass with a running maximum and sum.
//
// The products run on mma.sync m16n8k16 in f16 with fp32 accumulators, keys (then value dims) as M
// and the query heads as N.  A code times its e4m3 scale has at most six significant bits, so f16 holds
// it exactly.  A query row is scaled by a power of two that takes its largest dim into [2^13, 2^14): dims
// within 30 powers of two of that one keep their 8 bits, smaller ones are off by at most f16's half step,
// 2^-38 of the largest (a row of bf16 subnormals becomes zeros: with g <= 2^64 its scores are below 2^-40).
// The weights are split into f16 hi + lo parts (22 bits).
#include "attn_units.cuh"
#include "q4.cuh"

namespace spkv {
namespace {

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Both halves of a pair the low (high) one.
__device__ __forceinline__ uint32_t dup_lo(uint32_t w) { return __byte_perm(w, w, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t w) { return __byte_perm(w, w, 0x3232); }
// A warp's arithmetic on 4-bit pages.
template <bool PACK>
struct Warp4 : Softmax<PACK> {
  using Softmax<PACK>::ref;
  using Softmax<PACK>::fresh;
  using Softmax<PACK>::l;
  using Softmax<PACK>::O;
  using Softmax<PACK>::q;
  using Softmax<PACK>::scale;

  // 32 tokens of a page-head: two 16-token tiles at this lane's shared address `tiles` (keys; values
  // follow at kQ4V), their key and value scales at `scales` (+ 512), of which `left` >= 1 tokens exist.
  struct Half {
    uint32_t tiles, scales;
    int left;
  };
  using Scores = float[2][4];   // rows r, r + 8 of a tile; columns 2c, 2c + 1

  // Products of the keys' codes and scales with the queries.
  __device__ __forceinline__ void scores(const Half& t, Scores& y) const {
    const uint2 k2 = lds64(t.scales);
    const uint32_t ksc[2] = {k2.x, k2.y};
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      const uint4 a4 = lds128(t.tiles + tg * 1024), b4 = lds128(t.tiles + tg * 1024 + 512);
      const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, bw[4] = {b4.x, b4.y, b4.z, b4.w};
      const uint32_t sa = e4m3_to_f16(ksc[tg]), sb = e4m3_to_f16(ksc[tg] >> 16);
      const uint32_t sas[2] = {dup_lo(sa), dup_hi(sa)}, sbs[2] = {dup_lo(sb), dup_hi(sb)};
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
          if (w == 0 && s == 0) mma_f16_16816_first(y[tg], a, q[0][0], q[0][1]);
          else mma_f16_16816(y[tg], a, q[2 * w + s][0], q[2 * w + s][1]);
        }
      }
    }
  }

  // Scores to log2 weights, -inf behind the last token; raises the references where a weight passes the
  // slack.  keep: masks of the value scales of the tokens that exist (what lies behind the last may be
  // anything, and weight 0 times it must be 0).
  __device__ __forceinline__ void refer(const Half& t, Scores& y, uint32_t (&keep)[2][2], int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      fma_f32x2(y[tg][0], y[tg][1], y[tg][0], y[tg][1], scale[0], scale[1], -ref[0], -ref[1]);
      fma_f32x2(y[tg][2], y[tg][3], y[tg][2], y[tg][3], scale[0], scale[1], -ref[0], -ref[1]);
    }
    keep[0][0] = keep[0][1] = keep[1][0] = keep[1][1] = 0xFFFFFFFFu;
    if (t.left < 32) {
#pragma unroll
      for (int tg = 0; tg < 2; ++tg) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * tg + r + 8 * (e >> 1) >= t.left) y[tg][e] = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int x = 16 * tg + 8 * k + 2 * c;
          keep[tg][k] = (x < t.left ? 0xFFFFu : 0u) | (x + 1 < t.left ? 0xFFFF0000u : 0u);
        }
      }
    }
    float top = fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3]));
    top = fmaxf(top, fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
    if (fresh || __any_sync(0xffffffffu, top > kShift + kSlack)) {
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float m = fmaxf(fmaxf(y[0][cc], y[0][cc + 2]), fmaxf(y[1][cc], y[1][cc + 2]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        // up only; from the start's reference to the first maximum whatever its sign
        const float d = fresh ? m - kShift : fmaxf(m - kShift, 0.f);
        const float f = fresh ? 0.f : exp2f(-d);
        ref[cc] += d;
        l[cc] *= f;
#pragma unroll
        for (int tg = 0; tg < 2; ++tg) y[tg][cc] -= d, y[tg][cc + 2] -= d;
#pragma unroll
        for (int i = 0; i < 8; ++i) O[i][cc] *= f, O[i][cc + 2] *= f;
      }
    }
    fresh = false;
  }

  // O^T += V^T P^T with the weights 2^y.
  __device__ __forceinline__ void weigh(const Half& t, const Scores& y, const uint32_t (&keep)[2][2], int lane) {
    const int c = lane & 3;
    // weights, their sum, and as B fragments (hi and lo parts)
    uint32_t ph[2][2], pl[PACK ? 1 : 2][2];
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = ex2(y[tg][e]);
      add_f32x2(l[0], l[1], w[0], w[1]);
      add_f32x2(l[0], l[1], w[2], w[3]);
      const uint32_t h0 = pack_f16x2(w[0], w[1]), h1 = pack_f16x2(w[2], w[3]);
      const uint32_t l0 = pack_f16x2(w[0] - f16lo(h0), w[1] - f16hi(h0));
      const uint32_t l1 = pack_f16x2(w[2] - f16lo(h1), w[3] - f16hi(h1));
      ph[tg][0] = transposed(PACK && c >= 2 ? l0 : h0);
      ph[tg][1] = transposed(PACK && c >= 2 ? l1 : h1);
      if (!PACK) {
        pl[PACK ? 0 : tg][0] = transposed(l0);
        pl[PACK ? 0 : tg][1] = transposed(l1);
      }
    }
    // Half of the block's 16 dims at a time.  The products go into fresh accumulators, added to O rounded
    // to nearest: the tensor core cuts off what an addition shifts out, an error that would grow with
    // every page of a long list.
    const uint2 v2 = lds64(t.scales + (kQ4VScale - kQ4KScale));
    const uint32_t vsc[2] = {v2.x, v2.y};
    uint32_t sa[2], sb[2];
    uint4 va[2], vb[2];   // tokens 2c, 2c + 1 (va) and 8 + 2c, 9 + 2c (vb) of a tile, block r
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      va[tg] = lds128(t.tiles + kQ4V + tg * 1024);
      vb[tg] = lds128(t.tiles + kQ4V + tg * 1024 + 512);
      sa[tg] = e4m3_to_f16(vsc[tg]) & keep[tg][0];
      sb[tg] = e4m3_to_f16(vsc[tg] >> 16) & keep[tg][1];
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {   // m-tiles 4w .. 4w + 3
      float acc[4][4];
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
          if (tg == 0) mma_f16_16816_first(acc[i], a, ph[tg][0], ph[tg][1]);
          else mma_f16_16816(acc[i], a, ph[tg][0], ph[tg][1]);
          if (!PACK) mma_f16_16816(acc[i], a, pl[PACK ? 0 : tg][0], pl[PACK ? 0 : tg][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        add_f32x2(O[4 * w + i][0], O[4 * w + i][1], acc[i][0], acc[i][1]);
        add_f32x2(O[4 * w + i][2], O[4 * w + i][3], acc[i][2], acc[i][3]);
      }
    }
  }

  // A page-head at shared address `at`, of whose 64 tokens `valid` exist.  The second half's scores do not
  // wait for the first's weights.
  __device__ __forceinline__ void page(uint32_t at, int valid, int lane, int) {
    if (valid <= 0) return;
    const uint32_t mine = at + lane * 16;
    const Half a{mine, mine + kQ4KScale, valid}, b{mine + 2048, mine + kQ4KScale + 8, valid - 32};
    Scores y, z;
    uint32_t keep[2][2];
    scores(a, y);
    refer(a, y, keep, lane);
    if (valid > 32) {
      scores(b, z);
      weigh(a, y, keep, lane);
      refer(b, z, keep, lane);
      weigh(b, z, keep, lane);
    } else {
      weigh(a, y, keep, lane);
    }
  }
};

template <int CG, bool PACK>
struct Units4 : CtaShape<CG, false, PACK ? 4 : 8 * CG, PACK ? 7 : 6, PACK ? 28 : 12> {
  static constexpr int kPage = kQ4Page;
  // Pages of a CTA where they are dealt, at least; of a part of a unit, at least; and of a part, at most, where the launch
  // alone lets CTAs take units.
  static constexpr int kCtaPages = 8, kPartPages = 4, kUnitPages = 16;
  // Places between two units' pages where the pages are dealt: what a unit's end (the warps waiting for one another,
  // merges, the next queries) costs the CTA that meets it.  Without them such CTAs end 2 to 5 us after the others.
  // 0 / 4 / 6 / 8 places: 64 units of 129 pages 28.0 / 26.9 / 26.3 / 26.0 us, 61 of up to 129 (16 heads) 28.4 / 26.0 /
  // 26.3 / 26.9, 256 of 65 37.2 / 37.5 / 37.3 / 37.2, a step with 128 of 65 38.3 / 40.3 / 38.8 / 37.9.
  static constexpr int kEndPages = 8;
  using Params = AttnQ4Params;
  // Through a reference the kernels by unit spill (16 bytes a thread for 5 to 8 heads).  Reference / copy (us): one unit of 17 pages,
  // 8 heads 8.35 / 7.85, 16 heads 11.4 / 10.3; 64 of 33, 8 heads 14.8 / 14.2; 64 of 129, 8 heads 26.3 / 26.2, 5 heads 25.7 /
  // 25.5; 256 of 65, 4 heads 36.6 / 36.6.
  using Held = const AttnQ4Params;
  using Warp = Warp4<PACK>;
  static __device__ __forceinline__ float score_factor(const Params& p, int h) { return p.a.scale_log2 * p.k_scale[h]; }
  static __device__ __forceinline__ float value_factor(const Params& p, int h) { return p.v_scale[h]; }
};

// Measured (GB300): 256 units of 65 pages, 4 heads 37 us = 153 MB at 4.1 TB/s (0.61 of the copy rate); 64 units of
// 129 pages, 5 heads 26 us; 61 of up to 129 pages, 16 heads 27 us; 2 of 17 pages 7 us.  Of the first 37: 6 us until
// the first pages are there (lengths, lists, page table and page read one after the other), 25 us at 6.3 TB/s, and
// 4 us from the first CTA's end to the last's, merges included.  The next two are bound by the latency of a page in
// one warp, 1340 to 1370 instructions (half unpack and scale codes) that three warps a scheduler (168 registers) do
// not hide: they issue in 41 % of the slots, 9 us of it, and the rest waits on fixed latencies, on barriers and for
// the same ends.
enum Mode { kDealt, kEither, kByUnit };

template <int CG, bool PACK, Mode MODE>
__global__ void __launch_bounds__(Units4<CG, PACK>::kThreads, Units4<CG, PACK>::kCtasPerSm)
    attn_q4_kernel(const __grid_constant__ AttnQ4Params p) {
  attend_units<Units4<CG, PACK>, MODE == kEither, MODE == kByUnit>(p);
}

template <int CG, bool PACK>
cudaError_t launch_one(const spkv_cache* c, const AttnQ4Params& p, cudaStream_t st) {
  return launch_units<Units4<CG, PACK>>(attn_q4_kernel<CG, PACK, kDealt>, attn_q4_kernel<CG, PACK, kEither>,
                                        attn_q4_kernel<CG, PACK, kByUnit>, c, p, st);
}

template <int CG, bool PACK>
cudaError_t set_attr() {
  return allow_smem<Units4<CG, PACK>>({attn_q4_kernel<CG, PACK, kDealt>, attn_q4_kernel<CG, PACK, kEither>,
                                       attn_q4_kernel<CG, PACK, kByUnit>});
}

}  // namespace

cudaError_t attn_q4_init_attributes() {
  cudaError_t e;
  if ((e = set_attr<1, true>()) != cudaSuccess) return e;
  if ((e = set_attr<1, false>()) != cudaSuccess) return e;
  return set_attr<2, false>();
}

cudaError_t launch_attn_q4(const spkv_cache* c, const AttnParams& a, cudaStream_t st) {
  const AttnQ4Params p{a, c->pool4, c->k_scale, c->v_scale, 1, 1};
  if (a.G <= 4) return launch_one<1, true>(c, p, st);
  if (a.G <= 8) return launch_one<1, false>(c, p, st);
  return launch_one<2, false>(c, p, st);
}

}  // namespace spkv
