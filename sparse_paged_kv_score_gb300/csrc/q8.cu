// Whole pages of the 8-bit cache: pooled-key sums at handle creation, and pages back as bf16.
#include "q8.cuh"

namespace spkv {
namespace {

// A warp a page-head, four dims a lane: sums of each sub-block's valid codes, times its scale.  The sums of bytes are exact,
// so any order gives what the append gives.
// Runs when a cache is created: 16384 pages of 8 heads with fp32 sums, 1.34 GB, 372 us = 3.6 TB/s (0.54 of the copy rate).
template <bool BF16>
__global__ void __launch_bounds__(256)
    summary_build_q8_kernel(const uint8_t* __restrict__ pool, const int32_t* __restrict__ page_cnt, void* __restrict__ ksum,
                            int64_t n_ph, int64_t n_phys) {
  pdl_wait();
  pdl_trigger();
  const int64_t ph = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (ph >= n_ph) return;
  const int cnt = max(0, min(kPageTokens, page_cnt[ph % n_phys]));
  const uint8_t* page = pool + ph * kQ8Page;
#pragma unroll
  for (int j = 0; j < kNSub; ++j) {
    const int n = max(0, min(kSubblock, cnt - kSubblock * j));
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int t = 0; t < kSubblock; ++t) {
      if (t >= n) break;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(page + q8_k_code(kSubblock * j + t, 4 * lane));
      lo += w & 0x00FF00FFu;
      hi += (w >> 8) & 0x00FF00FFu;
    }
    const float s2 = n ? 0.5f * *reinterpret_cast<const float*>(page + kQ8KScale + 4 * j) : 0.f;
    const float4 a = make_float4(s2 * (2 * static_cast<int>(lo & 0xFFFFu) - 255 * n), s2 * (2 * static_cast<int>(hi & 0xFFFFu) - 255 * n),
                                 s2 * (2 * static_cast<int>(lo >> 16) - 255 * n), s2 * (2 * static_cast<int>(hi >> 16) - 255 * n));
    const int64_t at = (ph * kNSub + j) * kHeadDim + 4 * lane;
    if (BF16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(ksum) + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    else *reinterpret_cast<float4*>(static_cast<float*>(ksum) + at) = a;
  }
}

// Two codes (an f16 pair) times their scale, (c + 1/2) s = c s + s / 2, as bf16: exact.
__device__ __forceinline__ uint32_t open2(uint32_t f16, float s) {
  const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&f16));
  return pack_bf16x2(fmaf(c.x, s, 0.5f * s), fmaf(c.y, s, 0.5f * s));
}

// One CTA per (listed page, head).  Keys: a thread takes 8 dims of a token, 8 bytes in and 16 out, so that half a warp's
// store is a row.  Values: 8 dims of two tokens, 16 bytes in and 16 out for each.
// Bound by HBM: 2048 pages of 8 heads, 0.95 of their rows there (766 MB), 121 us from a replayed graph = 6.3 TB/s (0.94 of the copy
// rate); 17 pages of 2 heads 2.9 us, a launch and two reads one after the other.
__global__ void __launch_bounds__(256)
    unpack_q8_kernel(const uint8_t* __restrict__ pool, const int32_t* __restrict__ page_cnt, const int32_t* __restrict__ pages,
                     int n_pages, int64_t n_phys, uint4* __restrict__ k_out, uint4* __restrict__ v_out, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, h = blockIdx.y;
  const int p = pages[i];
  if (p < 0 || p >= n_phys) {
    if (threadIdx.x == 0 && h == 0) flag_error(err, SPKV_DEVERR_PHYS);
    return;
  }
  const int cnt = page_cnt ? max(0, min(kPageTokens, page_cnt[p])) : kPageTokens;
  const uint8_t* page = pool + (int64_t(h) * n_phys + p) * kQ8Page;
  const int64_t row0 = (int64_t(h) * n_pages + i) * kPageTokens;
  constexpr int kOcts = kHeadDim / 8;   // eights of a row
  const int oct = threadIdx.x % kOcts, r = threadIdx.x / kOcts;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = 16 * k + r;
    if (t >= cnt) break;
    const uint2 w = *reinterpret_cast<const uint2*>(page + q8_k_code(t, 8 * oct));
    const float s = *reinterpret_cast<const float*>(page + kQ8KScale + 4 * k);
    __stcs(k_out + (row0 + t) * kOcts + oct, make_uint4(open2(q8_f16_lo(w.x), s), open2(q8_f16_hi(w.x), s),
                                                        open2(q8_f16_lo(w.y), s), open2(q8_f16_hi(w.y), s)));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = 32 * k + 2 * r;
    if (t >= cnt) break;
    const uint4 w = *reinterpret_cast<const uint4*>(page + q8_v_code(t, 8 * oct));
    const float s = *reinterpret_cast<const float*>(page + kQ8VScale + 4 * (t / kSubblock));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (t + e >= cnt) break;
      const int sel = e ? 0x7531 : 0x6420;
      const uint32_t a = __byte_perm(w.x, w.y, sel), b = __byte_perm(w.z, w.w, sel);
      __stcs(v_out + (row0 + t + e) * kOcts + oct,
             make_uint4(open2(q8_f16_lo(a), s), open2(q8_f16_hi(a), s), open2(q8_f16_lo(b), s), open2(q8_f16_hi(b), s)));
    }
  }
}

}  // namespace

cudaError_t launch_summary_build_q8(const spkv_cache* c, cudaStream_t st) {
  const int64_t n_ph = int64_t(c->d.n_kv_heads) * c->d.n_phys_pages;
  return launch_pdl(c->d.ksum_bf16 ? summary_build_q8_kernel<true> : summary_build_q8_kernel<false>,
                    dim3(static_cast<unsigned>((n_ph + 7) / 8)), dim3(256), 0, st, c->pool8,
                    static_cast<const int32_t*>(c->d.page_cnt), c->d.ksum, n_ph, static_cast<int64_t>(c->d.n_phys_pages));
}

cudaError_t launch_unpack_q8(const spkv_cache* c, const int32_t* pages, int n_pages, void* k_out, void* v_out,
                             cudaStream_t st) {
  return launch_pdl(unpack_q8_kernel, dim3(n_pages, c->d.n_kv_heads), dim3(256), 0, st, c->pool8,
                    static_cast<const int32_t*>(c->d.page_cnt), pages, n_pages, static_cast<int64_t>(c->d.n_phys_pages),
                    static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), c->dev_err);
}

}  // namespace spkv
