// Whole pages of the 4-bit cache: pooled-key sums at handle creation, and pages back as bf16.
#include "q4.cuh"

namespace spkv {
namespace {

// One CTA per page-head, one thread per dim: sums of each sub-block's valid keys in token order,
// the codes times their scales first (exact in fp32) and the head's scale once at the end.  Bound by
// latency, one byte a load and one token after another: 65536 pages of 8 heads 4.4 ms = 3.5 GB (fp32 sums) at
// 0.8 TB/s, 8.5 times the floor.  It runs once, when a handle is made over a pool that holds rows.
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

// One CTA per (listed page, head).  A thread takes eight dims at a time, 4 bytes of codes in and 16 bytes of
// bf16 out, so that a warp's store is 512 contiguous bytes; four at once keep their loads in flight.  Code
// times scale is exact in f16; times g is rounded in fp32, then once to bf16.
// Bound by HBM: 2048 pages of 8 heads, 0.95 of their rows there, 98.5 us = 653 MB at 6.6 TB/s, 0.98 of the copy rate;
// 17 pages of 2 heads 2.5 us, a launch.
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
  const float gk = k_scale[h], gv = v_scale[h];
  constexpr int kBatch = 4, kOcts = kHeadDim / 8;   // eights of a row
  const int oct = threadIdx.x % kOcts, blk = oct / 2;
  for (int t0 = threadIdx.x / kOcts; t0 < 2 * kPageTokens; t0 += kBatch * (256 / kOcts)) {
    uint32_t code[kBatch], scale[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int x = t0 + k * (256 / kOcts), t = x % kPageTokens;
      const bool val = x >= kPageTokens;
      if (t < cnt) {
        code[k] = *reinterpret_cast<const uint32_t*>(page + (val ? q4_v_code(t, blk) : q4_k_code(t) + blk * 8) + (oct & 1) * 4);
        scale[k] = page[val ? q4_v_scale(t, blk) : q4_k_scale(t, blk)];
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int x = t0 + k * (256 / kOcts), t = x % kPageTokens;
      const bool val = x >= kPageTokens;
      if (t >= cnt) continue;
      const __half2 s = __half2half2(__ushort_as_half(static_cast<unsigned short>(e4m3_to_f16(scale[k]))));
      const float g = val ? gv : gk;
      uint32_t c[4], o[4];
      e2m1_to_f16(code[k], c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&c[j]), s));
        o[j] = pack_bf16x2(__fmul_rn(f.x, g), __fmul_rn(f.y, g));
      }
      __stcs((val ? v_out : k_out) + (row0 + t) * kOcts + oct, make_uint4(o[0], o[1], o[2], o[3]));
    }
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
