// Whole pages of the 4-bit cache: pooled-key sums at handle creation, and pages back as bf16.
#include "q4.cuh"
#include "summary.cuh"

namespace spkv {
namespace {

// One CTA per page-head, one thread per dim: sums of each sub-block's valid keys in token order,
// the codes times their scales first (exact in fp32) and the head's scale once at the end.
template <bool BF16>
__global__ void __launch_bounds__(kHeadDim)
    summary_build_q4_kernel(const uint8_t* __restrict__ pool, const float* __restrict__ k_scale,
                            const int32_t* __restrict__ page_cnt, void* __restrict__ ksum, int64_t n_phys) {
  pdl_wait();
  pdl_trigger();
  const int64_t ph = blockIdx.x;
  const int d = threadIdx.x;
  const int cnt = max(0, min(kPageTokens, page_cnt[ph % n_phys]));
  const uint8_t* page = pool + ph * kQ4Page;
  const float g = k_scale[ph / n_phys];
  for (int j = 0; j < kNSub; ++j) {
    float s = 0.f;
    for (int t = kSubblock * j; t < min(kSubblock * (j + 1), cnt); ++t) {
      const uint32_t n = page[q4_k_code(t) + d / 2] >> (4 * (d & 1));
      s += e2m1_to_f32(n) * e4m3_to_f32(page[q4_k_scale(t, d / kQ4Block)]);
    }
    const float v = __fmul_rn(s, g);
    const int64_t at = (ph * kNSub + j) * kHeadDim + d;
    if (BF16) reinterpret_cast<__nv_bfloat16*>(ksum)[at] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(ksum)[at] = v;
  }
}

// One CTA per (listed page, head).  A thread takes one block of 16 dims: 8 bytes of codes and a
// scale in, 32 bytes of bf16 out, consecutive threads consecutive blocks of a row.
__global__ void __launch_bounds__(256)
    unpack_q4_kernel(const uint8_t* __restrict__ pool, const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                     const int32_t* __restrict__ page_cnt, const int32_t* __restrict__ pages, int n_pages, int64_t n_phys,
                     uint4* __restrict__ k_out, uint4* __restrict__ v_out, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, h = blockIdx.y;
  const int p = pages[i];
  if (p < 0 || p >= n_phys) {
    if (threadIdx.x == 0 && h == 0) flag_error(err, SPKV_DEVERR_PHYS);
    return;
  }
  const int cnt = page_cnt ? max(0, min(kPageTokens, page_cnt[p])) : kPageTokens;
  const uint8_t* page = pool + (int64_t(h) * n_phys + p) * kQ4Page;
  const int64_t row0 = (int64_t(h) * n_pages + i) * kPageTokens;
  for (int x = threadIdx.x; x < 2 * cnt * 8; x += 256) {
    const bool val = x >= cnt * 8;
    const int t = (val ? x - cnt * 8 : x) >> 3, blk = x & 7;
    const uint2 w = *reinterpret_cast<const uint2*>(page + (val ? q4_v_code(t, blk) : q4_k_code(t) + blk * 8));
    const float s = e4m3_to_f32(page[val ? q4_v_scale(t, blk) : q4_k_scale(t, blk)]);
    const float g = val ? v_scale[h] : k_scale[h];
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = (j < 4 ? w.x : w.y) >> (8 * (j & 3));
      o[j] = pack_bf16x2(__fmul_rn(e2m1_to_f32(b) * s, g), __fmul_rn(e2m1_to_f32(b >> 4) * s, g));
    }
    uint4* dst = (val ? v_out : k_out) + (row0 + t) * (kHeadDim / 8) + blk * 2;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_summary_build_q4(const spkv_cache* c, cudaStream_t st) {
  const int64_t n_ph = int64_t(c->d.n_kv_heads) * c->d.n_phys_pages;
  return launch_pdl(c->d.ksum_bf16 ? summary_build_q4_kernel<true> : summary_build_q4_kernel<false>,
                    dim3(static_cast<unsigned>(n_ph)), dim3(kHeadDim), 0, st, c->pool4, c->k_scale,
                    static_cast<const int32_t*>(c->d.page_cnt), c->d.ksum, static_cast<int64_t>(c->d.n_phys_pages));
}

cudaError_t launch_unpack_q4(const spkv_cache* c, const int32_t* pages, int n_pages, void* k_out, void* v_out,
                             cudaStream_t st) {
  return launch_pdl(unpack_q4_kernel, dim3(n_pages, c->d.n_kv_heads), dim3(256), 0, st, c->pool4, c->k_scale, c->v_scale,
                    static_cast<const int32_t*>(c->d.page_cnt), pages, n_pages,
                    static_cast<int64_t>(c->d.n_phys_pages), static_cast<uint4*>(k_out), static_cast<uint4*>(v_out),
                    c->dev_err);
}

}  // namespace spkv
