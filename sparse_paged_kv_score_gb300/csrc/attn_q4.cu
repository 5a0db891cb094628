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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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
// Both halves of a pair the low (high) one.
__device__ __forceinline__ uint32_t dup_lo(uint32_t w) { return __byte_perm(w, w, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t w) { return __byte_perm(w, w, 0x3232); }

// The running maximum moves only when a score passes it by kSlack (log2 units): weights stay below
// 2^(kShift + kSlack) = 2^15, inside f16, and a weight's lo part resolves 2^-(24 + kShift) of it.
constexpr float kShift = 7.f, kSlack = 8.f;

// State of one warp for one unit: query columns n = 8 nt + (lane / 4) in the query fragments, 8 nt +
// 2 (lane % 4) + {0, 1} in everything else.  PACK (at most four query heads): columns 4..7 repeat the
// heads of columns 0..3; the weights' hi parts go into the first half and the lo parts into the
// second, so one MMA does both.
template <int NT, bool PACK>
struct Warp4 {
  float ref[NT][2];        // log2 weight reference: weights are 2^(x - ref)
  float l[NT][2];          // this lane's part of their sum
  float O[8][NT][4];       // dims 16 r + 2 i, + 1 of m-tile i (r = lane / 4)
  uint32_t q[8][NT][2];    // query fragments, f16
  float scale[NT][2];      // scores to log2 units, per column

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = -CUDART_INF_F;
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

  // One page-head (9216 bytes at `page`) with `valid` >= 1 tokens.
  __device__ __forceinline__ void page(const uint8_t* page, int valid, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const uint8_t* mine = page + lane * 16;
    const uint4 ks4 = *reinterpret_cast<const uint4*>(mine + kQ4KScale);
    const uint32_t ksc[4] = {ks4.x, ks4.y, ks4.z, ks4.w};
    float x[4][NT][4];
    // ---- scores of the four 16-token tiles: rows r, r + 8 of a tile
#pragma unroll
    for (int tg = 0; tg < 4; ++tg) {
      const uint4 a4 = *reinterpret_cast<const uint4*>(mine + tg * 1024);
      const uint4 b4 = *reinterpret_cast<const uint4*>(mine + tg * 1024 + 512);
      const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w}, bw[4] = {b4.x, b4.y, b4.z, b4.w};
      const uint32_t sa = e4m3_to_f16(ksc[tg]), sb = e4m3_to_f16(ksc[tg] >> 16);
      const uint32_t sas[2] = {dup_lo(sa), dup_hi(sa)}, sbs[2] = {dup_lo(sb), dup_hi(sb)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[tg][nt][e] = 0.f;
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
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(x[tg][nt], a, q[2 * w + s][nt][0], q[2 * w + s][nt][1]);
        }
      }
    }
    // ---- to log2 units; does any score pass the reference by the slack?
    bool over = false;
#pragma unroll
    for (int tg = 0; tg < 4; ++tg)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = x[tg][nt][e] * scale[nt][e & 1];
          x[tg][nt][e] = 16 * tg + r + 8 * (e >> 1) < valid ? v : -CUDART_INF_F;
          over |= x[tg][nt][e] > ref[nt][e & 1] + (kShift + kSlack);
        }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          float m = -CUDART_INF_F;
#pragma unroll
          for (int tg = 0; tg < 4; ++tg) m = fmaxf(m, fmaxf(x[tg][nt][cc], x[tg][nt][cc + 2]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          const float now = fmaxf(ref[nt][cc], m - kShift);
          const float f = ref[nt][cc] == now ? 1.f : exp2f(ref[nt][cc] - now);   // both -inf: nothing held yet
          ref[nt][cc] = now;
          l[nt][cc] *= f;
#pragma unroll
          for (int i = 0; i < 8; ++i) O[i][nt][cc] *= f, O[i][nt][cc + 2] *= f;
        }
    }
    // ---- weights, their sum, and as B fragments (hi and lo parts)
    const uint4 vs4 = *reinterpret_cast<const uint4*>(mine + kQ4VScale);
    const uint32_t vsc[4] = {vs4.x, vs4.y, vs4.z, vs4.w};
#pragma unroll
    for (int tg = 0; tg < 4; ++tg) {
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = exp2f(x[tg][nt][e] - ref[nt][e & 1]);
        l[nt][0] += w[0] + w[2];
        l[nt][1] += w[1] + w[3];
        const uint32_t h0 = pack_f16x2(w[0], w[1]), h1 = pack_f16x2(w[2], w[3]);
        const uint32_t l0 = pack_f16x2(w[0] - f16lo(h0), w[1] - f16hi(h0));
        const uint32_t l1 = pack_f16x2(w[2] - f16lo(h1), w[3] - f16hi(h1));
        if (PACK) {
          ph[nt][0] = movmatrix_trans(c < 2 ? h0 : l0);
          ph[nt][1] = movmatrix_trans(c < 2 ? h1 : l1);
        } else {
          ph[nt][0] = movmatrix_trans(h0);
          ph[nt][1] = movmatrix_trans(h1);
          pl[nt][0] = movmatrix_trans(l0);
          pl[nt][1] = movmatrix_trans(l1);
        }
      }
      // ---- O^T += V^T P^T: tokens 2c, 2c + 1 (a4) and 8 + 2c, 9 + 2c (b4) of the tile, block r
      const uint4 a4 = *reinterpret_cast<const uint4*>(mine + kQ4V + tg * 1024);
      const uint4 b4 = *reinterpret_cast<const uint4*>(mine + kQ4V + tg * 1024 + 512);
      uint32_t sa = e4m3_to_f16(vsc[tg]), sb = e4m3_to_f16(vsc[tg] >> 16);
      if (valid < 16 * tg + 16) {   // scales behind the last token may hold anything: weight 0 times them must be 0
        const int t = 16 * tg + 2 * c;
        sa = (t < valid ? sa & 0xFFFFu : 0u) | (t + 1 < valid ? sa & 0xFFFF0000u : 0u);
        sb = (t + 8 < valid ? sb & 0xFFFFu : 0u) | (t + 9 < valid ? sb & 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {   // 8 dims of the block: m-tiles 4w .. 4w + 3
        const uint32_t a0 = w ? a4.y : a4.x, a1 = w ? a4.w : a4.z, b0 = w ? b4.y : b4.x, b1 = w ? b4.w : b4.z;
        // token pairs of one dim in a byte: even dims, odd dims
        uint32_t ea[4], oa[4], eb[4], ob[4];
        e2m1_to_f16((a0 & 0x0F0F0F0Fu) | ((a1 << 4) & 0xF0F0F0F0u), ea);
        e2m1_to_f16(((a0 >> 4) & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u), oa);
        e2m1_to_f16((b0 & 0x0F0F0F0Fu) | ((b1 << 4) & 0xF0F0F0F0u), eb);
        e2m1_to_f16(((b0 >> 4) & 0x0F0F0F0Fu) | (b1 & 0xF0F0F0F0u), ob);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a[4] = {hmul2(ea[i], sa), hmul2(oa[i], sa), hmul2(eb[i], sb), hmul2(ob[i], sb)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(O[4 * w + i][nt], a, ph[nt][0], ph[nt][1]);
            if (!PACK) mma_f16_16816(O[4 * w + i][nt], a, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
  }

  // The warp's state as (reference, sum, O) of every column, to shared memory.
  __device__ __forceinline__ void store(float* m, float* sum, float (*o)[kHeadDim], int lane) {
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
          m[col] = ref[nt][cc];
          sum[col] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float u = O[i][nt][cc], v = O[i][nt][cc + 2];
          if (PACK) {   // hi part (columns 0..3) and lo part (4..7) of the same weights
            u += __shfl_xor_sync(0xffffffffu, u, 2);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
          }
          if (!PACK || c < 2) *reinterpret_cast<float2*>(&o[col][16 * r + 2 * i]) = make_float2(u, v);
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

constexpr int kWarps = 8;

template <int NT>
struct SmemQ4 {
  float m[kWarps][8 * NT];
  float l[kWarps][8 * NT];
  float o[kWarps][8 * NT][kHeadDim];
};

// One CTA per unit, its pages dealt to eight warps; their states are merged in shared memory.
template <int NT, bool PACK>
__global__ void __launch_bounds__(kWarps * 32) attn_q4_kernel(const __grid_constant__ AttnQ4Params p4) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SmemQ4<NT>& S = *reinterpret_cast<SmemQ4<NT>*>(smem_raw);
  const AttnParams& p = p4.a;
  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x, b = u / p.Hk, h = u % p.Hk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = max(0, min(p.n_sel[u], p.sel_stride));
  const int64_t row = int64_t(b) * p.Hq + h * p.G;
  Warp4<NT, PACK> w;
  w.reset();
  w.load_q(static_cast<const uint16_t*>(p.q) + row * kHeadDim, p.G, p.scale_log2 * p4.k_scale[h], lane);
  for (int i = warp; i < n; i += kWarps) {
    int phys = 0;
    const int valid = page_of(p, u, b, i, phys);
    if (valid > 0) w.page(p4.pool + (int64_t(h) * p.n_phys + phys) * kQ4Page, valid, lane);
  }
  w.store(S.m[warp], S.l[warp], S.o[warp], lane);
  __syncthreads();
  const float gv = p4.v_scale[h];
  for (int x = tid; x < p.G * kHeadDim; x += kWarps * 32) {
    const int g = x / kHeadDim, d = x % kHeadDim;
    float M = -CUDART_INF_F, L = 0.f, acc = 0.f;
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, S.m[k][g]);
    for (int k = 0; k < kWarps; ++k) {
      const float f = S.m[k][g] == -CUDART_INF_F ? (S.l[k][g] == 0.f ? 0.f : 1.f) : exp2f(S.m[k][g] - M);
      L += f * S.l[k][g];
      acc += f * S.o[k][g][d];
    }
    // L is 0 without a token; a NaN (from a NaN in the inputs) is passed on
    p.out[row * kHeadDim + x] = L == 0.f ? 0.f : acc / L * gv;
    if (d == 0) p.lse[row + g] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
  }
}

template <int NT, bool PACK>
cudaError_t launch_one(const AttnQ4Params& p, cudaStream_t st) {
  return launch_pdl(attn_q4_kernel<NT, PACK>, dim3(p.a.B * p.a.Hk), dim3(kWarps * 32), sizeof(SmemQ4<NT>), st, p);
}

template <int NT, bool PACK>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(attn_q4_kernel<NT, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(sizeof(SmemQ4<NT>)));
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
  if (a.G <= 4) return launch_one<1, true>(p, st);
  if (a.G <= 8) return launch_one<1, false>(p, st);
  return launch_one<2, false>(p, st);
}

}  // namespace spkv
