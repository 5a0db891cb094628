// Appends new tokens with their rotary positions applied on the way, to a bf16 or a 4-bit cache:
// rotated queries out, rotated keys and values into their pages, the pooled-key sums of the
// sub-blocks they touch (summary.cuh's token order), page counts.
//
// Rotation of pair j (dims j, j + 64) by its position's cos and sin from the caller's table:
//   lo' = lo c - hi s,  hi' = hi c + lo s   (products and the sum rounded separately in fp32)
//
// One CTA takes `window` consecutive rows of one kv head: keys, values and the group's query heads
// are its tasks, one half-warp each (lane l of 16 holds dims 4l .. 4l + 3 and 64 + 4l .. + 3, so both
// halves of every pair).  A row's sub-block is summed by the CTA that holds its first new row; the
// at most 15 rows of it that lie in the next window are rotated again there, so no CTA waits for
// another's rows and one launch does.
#include "q4.cuh"
#include "summary.cuh"

namespace spkv {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kMaxWindow = 16;
constexpr int kMaxRows = kMaxWindow + kSubblock - 1;

struct RowInfo {
  int b;        // request, -1: no request's row
  int at;       // position in the request's context
  int first;    // the request's first new position
  int end;      // one past its last
  int phys;     // physical page, -1: not appended
  int rot;      // positions within the table
};

template <bool Q4>
__global__ void __launch_bounds__(kThreads)
    append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
  __shared__ RowInfo info[kMaxRows];
  __shared__ int axis_pos[kMaxRows][4];
  __shared__ __align__(16) float rows[kMaxRows][kHeadDim];   // the cache's values of the new keys (4-bit: without g)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, h = blockIdx.y, base = blockIdx.x * p.window;
  const int own = min(p.window, p.n_rows - base);

  if (tid < kMaxRows) {
    RowInfo r{-1, 0, 0, 0, -1, 0};
    const int i = base + tid;
    if (tid < p.window + kSubblock - 1 && i < p.n_rows) {
      int lo = 0, f = i, e = i + 1;
      if (p.row_first) {   // the last request whose first row is not after row i
        int hi = p.B;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (p.row_first[mid] <= i) lo = mid;
          else hi = mid;
        }
        f = p.row_first[lo];
        e = p.row_first[lo + 1];
      } else {
        lo = i;
      }
      if (f <= i && i < e) {
        const int64_t L = p.seq_len[lo];
        const int64_t at = L - (int64_t(e) - i), first = L - (int64_t(e) - f);
        uint32_t bad = 0;
        if (at < 0 || at / kPageTokens >= p.np_max || at > INT32_MAX - kPageTokens) {
          bad |= SPKV_DEVERR_PAGE_ID;
        } else {
          r.b = lo;
          r.at = static_cast<int>(at);
          r.first = static_cast<int>(max(first, int64_t(0)));
          r.end = static_cast<int>(L);
          const int ph = p.page_table[int64_t(lo) * p.np_max + at / kPageTokens];
          if (ph >= 0 && ph < p.n_phys) r.phys = ph;
          else bad |= SPKV_DEVERR_PHYS;
        }
        r.rot = 1;
        if (p.cos_sin) {
          for (int a = 0; a < p.n_axes; ++a) {
            const int64_t x = p.pos ? int64_t(p.pos[int64_t(i) * p.n_axes + a]) : at;
            axis_pos[tid][a] = static_cast<int>(x);
            if (x < 0 || x >= p.n_pos) r.rot = 0;
          }
          if (!r.rot) bad |= SPKV_DEVERR_POS;
        }
        if (tid < own && h == 0) flag_error(p.err, bad);
      }
    }
    info[tid] = r;
  }
  __syncthreads();
  // rows of the next window that belong to the sub-block of this window's last row
  int n_rows = own;
  if (own == p.window) {
    const RowInfo last = info[own - 1];
    if (last.b >= 0) {
      const int stop = min(last.end, (last.at / kSubblock + 1) * kSubblock);
      n_rows = min(own + stop - last.at - 1, kMaxRows);
    }
  }

  // ---- tasks: own rows' key, value and query heads, the other rows' key alone
  const int hw = tid >> 4, l = tid & 15;
  const int per_row = 2 + p.G;
  const int n_tasks = own * per_row + (n_rows - own);
  const float gk = Q4 ? p.k_scale[h] : 1.f, gv = Q4 ? p.v_scale[h] : 1.f;
  // both half-warps of a warp run the same number of rounds: the shuffles below name all lanes
  for (int t0 = 0; t0 < n_tasks; t0 += kHalfWarps) {
    const int task = t0 + hw;
    const bool live = task < n_tasks;
    const int row = !live ? 0 : task < own * per_row ? task / per_row : own + task - own * per_row;
    const int what = !live ? 1 : task < own * per_row ? task % per_row : 0;   // 0 key, 1 value, 2.. query head
    const RowInfo r = info[row];
    const int64_t i = base + row;
    const bool held = live && r.b >= 0 && r.phys >= 0 && r.rot;   // goes into the cache
    uint8_t* page = nullptr;
    int tok = 0;
    if (held) {
      page = p.pool + (int64_t(h) * p.n_phys + r.phys) * (Q4 ? kQ4Page : kPageTokens * kHeadDim * 2);
      tok = r.at % kPageTokens;
    }
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // key, query: dims 4l + (0..3), 64 + 4l + (0..3); value: 8l + (0..7)
    if (what == 1) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (held) w = *reinterpret_cast<const uint4*>(p.v_new + i * p.v_stride + h * kHeadDim + 8 * l);
      if (!Q4) {
        if (held)
          *reinterpret_cast<uint4*>(p.v_pool + (int64_t(h) * p.n_phys + r.phys) * (kPageTokens * kHeadDim * 2) +
                                    (tok * kHeadDim + 8 * l) * 2) = w;
      } else {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[2 * j] = bf16lo_to_f32(ws[j]);
          x[2 * j + 1] = bf16hi_to_f32(ws[j]);
        }
      }
    } else {
      const uint16_t* src = what == 0 ? p.k_new + i * p.k_stride + h * kHeadDim
                                      : p.q + i * p.q_stride + (int64_t(h) * p.G + what - 2) * kHeadDim;
      const bool read = live && r.rot && (what != 0 || held);
      if (read) {
        const uint2 a = *reinterpret_cast<const uint2*>(src + 4 * l), b = *reinterpret_cast<const uint2*>(src + 64 + 4 * l);
        float lo[4] = {bf16lo_to_f32(a.x), bf16hi_to_f32(a.x), bf16lo_to_f32(a.y), bf16hi_to_f32(a.y)};
        float hi[4] = {bf16lo_to_f32(b.x), bf16hi_to_f32(b.x), bf16lo_to_f32(b.y), bf16hi_to_f32(b.y)};
        if (p.cos_sin) {
          float c[4], s[4];
          if (p.n_axes == 1) {
            const float* cs = p.cos_sin + int64_t(axis_pos[row][0]) * kHeadDim + 4 * l;
            const float4 cv = *reinterpret_cast<const float4*>(cs), sv = *reinterpret_cast<const float4*>(cs + 64);
            c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
            s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int pair = 4 * l + j;
              const int axis = static_cast<int>(p.pair_axis[pair >> 5] >> (2 * (pair & 31))) & 3;
              const float* cs = p.cos_sin + int64_t(axis_pos[row][axis]) * kHeadDim + pair;
              c[j] = cs[0];
              s[j] = cs[64];
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = __fsub_rn(__fmul_rn(lo[j], c[j]), __fmul_rn(hi[j], s[j]));
            x[4 + j] = __fadd_rn(__fmul_rn(hi[j], c[j]), __fmul_rn(lo[j], s[j]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = lo[j], x[4 + j] = hi[j];
        }
      }
      if (what >= 2 || !Q4) {
        const uint2 a = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        const uint2 b = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        if (what >= 2) {
          if (live && r.rot) {
            uint16_t* dst = p.q_out + (i * p.Hq + int64_t(h) * p.G + what - 2) * kHeadDim;
            *reinterpret_cast<uint2*>(dst + 4 * l) = a;
            *reinterpret_cast<uint2*>(dst + 64 + 4 * l) = b;
          }
        } else if (held) {
          if (row < own) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(page) + tok * kHeadDim;
            *reinterpret_cast<uint2*>(dst + 4 * l) = a;
            *reinterpret_cast<uint2*>(dst + 64 + 4 * l) = b;
          }
          *reinterpret_cast<float4*>(&rows[row][4 * l]) =
              make_float4(bf16lo_to_f32(a.x), bf16hi_to_f32(a.x), bf16lo_to_f32(a.y), bf16hi_to_f32(a.y));
          *reinterpret_cast<float4*>(&rows[row][64 + 4 * l]) =
              make_float4(bf16lo_to_f32(b.x), bf16hi_to_f32(b.x), bf16lo_to_f32(b.y), bf16hi_to_f32(b.y));
        }
      }
    }
    if (Q4) {
      // a key's blocks: four lanes each (dims 16 (l / 4) .. and 64 + that); a value's: two lanes
      float y0[4] = {x[0], x[1], x[2], x[3]}, y1[4] = {x[4], x[5], x[6], x[7]};
      uint32_t m0 = abs_max_bits(y0), m1 = abs_max_bits(y1);
      const uint32_t mv = max(m0, m1);
      const uint32_t mv2 = max(mv, __shfl_xor_sync(0xffffffffu, mv, 1));
      m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
      m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
      m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 2));
      m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 2));
      if (held && what == 1) {
        const uint32_t sb = q4_scale_byte(mv2, gv);
        const float d = __fmul_rn(e4m3_to_f32(sb), gv);
        *reinterpret_cast<uint32_t*>(page + q4_v_code(tok, l >> 1) + (l & 1) * 4) = q4_codes(x, d);
        if (!(l & 1)) page[q4_v_scale(tok, l >> 1)] = static_cast<uint8_t>(sb);
      } else if (held && what == 0) {
        const uint32_t s0 = q4_scale_byte(m0, gk), s1 = q4_scale_byte(m1, gk);
        const float e0 = e4m3_to_f32(s0), e1 = e4m3_to_f32(s1);
        const uint32_t c0 = q4_codes(y0, __fmul_rn(e0, gk)), c1 = q4_codes(y1, __fmul_rn(e1, gk));
        if (row < own) {
          uint16_t* dst = reinterpret_cast<uint16_t*>(page + q4_k_code(tok));
          dst[l] = static_cast<uint16_t>(c0);
          dst[16 + l] = static_cast<uint16_t>(c1);
          if (!(l & 3)) {
            page[q4_k_scale(tok, l >> 2)] = static_cast<uint8_t>(s0);
            page[q4_k_scale(tok, 4 + (l >> 2))] = static_cast<uint8_t>(s1);
          }
        }
        *reinterpret_cast<float4*>(&rows[row][4 * l]) = make_float4(
            e2m1_to_f32(c0) * e0, e2m1_to_f32(c0 >> 4) * e0, e2m1_to_f32(c0 >> 8) * e0, e2m1_to_f32(c0 >> 12) * e0);
        *reinterpret_cast<float4*>(&rows[row][64 + 4 * l]) = make_float4(
            e2m1_to_f32(c1) * e1, e2m1_to_f32(c1 >> 4) * e1, e2m1_to_f32(c1 >> 8) * e1, e2m1_to_f32(c1 >> 12) * e1);
      }
    }
  }
  __syncthreads();

  // ---- sums of the sub-blocks whose first new row is one of this window's
  const int half = tid / kHeadDim, d = tid % kHeadDim;
  int seen = 0;
  for (int j = 0; j < own; ++j) {
    const RowInfo r = info[j];
    if (r.b < 0 || r.phys < 0 || !(r.at % kSubblock == 0 || r.at == r.first)) continue;
    if (seen++ % (kThreads / kHeadDim) != half) continue;
    const int64_t ph = int64_t(h) * p.n_phys + r.phys;
    const int s0 = r.at / kSubblock * kSubblock, s1 = min(r.end, s0 + kSubblock);   // new: [r.at, s1)
    const int cnt = max(0, min(kPageTokens, p.page_cnt[r.phys]));
    float sum = 0.f;
    for (int t = s0; t < s0 + kSubblock; ++t) {
      const int tok = t % kPageTokens;
      if (t >= r.at && t < s1) {
        if (info[j + t - r.at].rot) sum += rows[j + t - r.at][d];
      } else if (tok < cnt) {
        if (Q4) {
          const uint8_t* page = p.pool + ph * kQ4Page;
          sum += e2m1_to_f32(page[q4_k_code(tok) + d / 2] >> (4 * (d & 1))) * e4m3_to_f32(page[q4_k_scale(tok, d / kQ4Block)]);
        } else {
          const uint16_t w = reinterpret_cast<const uint16_t*>(p.pool)[(ph * kPageTokens + tok) * kHeadDim + d];
          sum += __uint_as_float(uint32_t(w) << 16);
        }
      }
    }
    if (Q4) sum = __fmul_rn(sum, gk);
    const int64_t at = (ph * kNSub + (s0 % kPageTokens) / kSubblock) * kHeadDim + d;
    if (p.ksum_bf16) reinterpret_cast<__nv_bfloat16*>(p.ksum)[at] = __float2bfloat16_rn(sum);
    else reinterpret_cast<float*>(p.ksum)[at] = sum;
  }
  if (h == 0 && tid < own) {
    const RowInfo r = info[tid];
    if (r.b >= 0 && r.phys >= 0 && r.rot) atomicMax(&p.page_cnt[r.phys], r.at % kPageTokens + 1);
  }
}

}  // namespace

cudaError_t launch_append_rope(const spkv_cache* c, AppendRopeParams& p, cudaStream_t st) {
  // rows per CTA: enough CTAs first, then fewer that share their row look-ups
  p.window = kMaxWindow;
  while (p.window > 1 && (int64_t(p.n_rows) + p.window - 1) / p.window * c->d.n_kv_heads < 4 * c->sm_count) p.window /= 4;
  const dim3 grid((p.n_rows + p.window - 1) / p.window, c->d.n_kv_heads);
  return launch_pdl(c->pool4 ? append_rope_kernel<true> : append_rope_kernel<false>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace spkv
