// Appends new tokens with their rotary positions applied on the way, to a bf16 or a 4-bit cache:
// rotated queries out, rotated keys and values into their pages, the pooled-key sums of the
// sub-blocks they touch (summary.cuh's token order), page counts.
//
// Rotation of pair j (dims j, j + 64) by its position's cos and sin from the caller's table:
//   lo' = lo c - hi s,  hi' = hi c + lo s   (products and the sum rounded separately in fp32)
//
// One CTA takes `window` consecutive rows of one kv head, a half-warp a row at a time (lane l of 16 holds dims
// 4l .. 4l + 3 and 64 + 4l .. + 3, so both halves of every pair); windows of fewer rows give a row's query heads
// to several.  The rows are asked for before their places are looked up.  A sub-block's keys and values, and its
// sums, are the CTA's that holds its first new row, with the at most 15 rows of it that lie behind the window,
// so no CTA waits for another's rows and one launch does.
//
// Measured (GB300): 8192 rows of 32 + 2 x 8 heads to bf16 pages 38.6 us = 206 MB at 5.3 TB/s (0.79 of the copy rate).
// Bound by latency and instructions: a CTA waits for the look-ups, for its rows, and at the barrier in front of the
// sums.
#include "append_rope.cuh"
#include "q4.cuh"

namespace spkv {
namespace {

// Scales (as e4m3 bytes) and codes of a lane's x[0 .. 3] and x[4 .. 7].  A block of 16 values is x[0 .. 3] (and
// another x[4 .. 7]) of four lanes, or with PAIRS all eight of two lanes.
template <bool PAIRS>
__device__ __forceinline__ void quantise(const float (&x)[8], float g, uint32_t (&scale)[2], uint32_t (&code)[2]) {
  const float y[2][4] = {{x[0], x[1], x[2], x[3]}, {x[4], x[5], x[6], x[7]}};
  uint32_t m[2] = {abs_max_bits(y[0]), abs_max_bits(y[1])};
  if (PAIRS) m[0] = max(m[0], m[1]);
#pragma unroll
  for (int j = 0; j < (PAIRS ? 1 : 2); ++j) {
    m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 1));
    if (!PAIRS) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 2));
    scale[j] = q4_scale_byte(m[j], g);
  }
  if (PAIRS) scale[1] = scale[0];
#pragma unroll
  for (int j = 0; j < 2; ++j) code[j] = q4_codes(y[j], __fmul_rn(e4m3_to_f32(scale[j]), g));
}

// Four CTAs of 256 threads an SM (64 registers) and four heads' rows asked for together: with two heads' rows the 8192 rows
// took 49.4 us for 43.6 then, with those and five CTAs 46.3.  Asking for a half-warp's second key and value early, or two
// kv heads a CTA, measured slower (45.0, 50.1).
template <bool Q4>
__global__ void __launch_bounds__(256, 4) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
  __shared__ RowInfo info[32];      // a warp looks up, the last is not of this window
  __shared__ int axis_pos[32][4];
  __shared__ __align__(16) float rows[kMaxRows][kHeadDim];   // the cache's values of the new keys (4-bit: without g)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hw = tid >> 4, l = lane & 15;
  const int n_warps = blockDim.x >> 5, n_hw = blockDim.x >> 4;
  const int h = blockIdx.y, base = blockIdx.x * p.window;
  const int own = min(p.window, p.n_rows - base);
  const float gk = Q4 ? p.k_scale[h] : 1.f;
  const bool turn = p.cos_sin != nullptr;
  // this half-warp's query heads: sub, sub + step, .. of row rq
  const int step = n_hw / p.window, rq = hw / step, sub = hw % step;

  // ---- the first rows are on their way while their places are looked up
  uint4 kx = make_uint4(0, 0, 0, 0), vx = kx, qv[kHeads];
  const uint16_t* const k_new = p.k_new + base * p.k_stride + h * kHeadDim;
  const uint16_t* const v_new = p.v_new + base * p.v_stride + h * kHeadDim + 8 * l;
  if (hw < own) {
    kx = load_pairs(k_new + hw * p.k_stride, l);
    vx = *reinterpret_cast<const uint4*>(v_new + hw * p.v_stride);
  }
  const uint16_t* const q = q_row(p, h, base + rq, sub);
  if (rq < own) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
      if (sub + k * step < p.G) qv[k] = load_pairs(q + k * step * kHeadDim, l);
  }
  if (warp == 0) {
    uint32_t bad = 0;
    RowInfo ri = find_row(p, base, lane, axis_pos[lane], bad);
    if (lane < own && h == 0) flag_error(p.err, bad);
    // its sub-block's first new row is one of the window's
    const int opens = lane - min(ri.at % kSubblock, ri.at - ri.first);
    if (opens < 0 || opens >= own) ri.b = ri.phys = -1;
    info[lane] = ri;
  }
  __syncthreads();

  // ---- query heads
  CosSin t{};
  if (rq < own && sub < p.G && info[rq].rot) turn_queries(p, h, base + rq, axis_pos[rq], sub, step, l, q, qv, t);
  // ---- keys and values of the window's sub-blocks
  for (int r = hw; r < n_hw * ((kMaxRows + n_hw - 1) / n_hw); r += n_hw) {
    const RowInfo ri = info[min(r, 31)];
    if (!__any_sync(0xffffffffu, r < kMaxRows && ri.b >= 0)) {
      if ((r & ~1) >= own) break;   // neither of the warp's two rows is this CTA's, nor is one behind them
      continue;
    }
    const bool held = r < kMaxRows && ri.phys >= 0 && ri.rot;
    if (held) {
      if (r != hw || r >= own) {
        kx = load_pairs(k_new + r * p.k_stride, l);
        vx = *reinterpret_cast<const uint4*>(v_new + r * p.v_stride);
      }
      if (turn) t = load_turn(p, axis_pos[r], l);
    }
    const int tok = ri.at % kPageTokens;
    const int64_t ph = int64_t(h) * p.n_phys + ri.phys;
    float x[8];
    rotate(kx, t, turn, x);
    if (!Q4) {
      if (held) {
        const uint4 y = round_pairs(x);
        store_pairs(reinterpret_cast<uint16_t*>(p.pool) + (ph * kPageTokens + tok) * kHeadDim, l, y);
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.v_pool) + (ph * kPageTokens + tok) * kHeadDim + 8 * l) = vx;
        *reinterpret_cast<float4*>(&rows[r][4 * l]) =
            make_float4(bf16lo_to_f32(y.x), bf16hi_to_f32(y.x), bf16lo_to_f32(y.y), bf16hi_to_f32(y.y));
        *reinterpret_cast<float4*>(&rows[r][64 + 4 * l]) =
            make_float4(bf16lo_to_f32(y.z), bf16hi_to_f32(y.z), bf16lo_to_f32(y.w), bf16hi_to_f32(y.w));
      }
      continue;
    }
    uint8_t* page = p.pool + ph * kQ4Page;
    uint32_t scale[2], code[2];
    quantise<false>(x, gk, scale, code);
    if (held) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(page + q4_k_code(tok));
      dst[l] = static_cast<uint16_t>(code[0]);
      dst[16 + l] = static_cast<uint16_t>(code[1]);
      if (!(l & 3)) {
        page[q4_k_scale(tok, l >> 2)] = static_cast<uint8_t>(scale[0]);
        page[q4_k_scale(tok, 4 + (l >> 2))] = static_cast<uint8_t>(scale[1]);
      }
      *reinterpret_cast<float4*>(&rows[r][4 * l]) = q4_values(code[0], e4m3_to_f32(scale[0]));
      *reinterpret_cast<float4*>(&rows[r][64 + 4 * l]) = q4_values(code[1], e4m3_to_f32(scale[1]));
    }
    const uint32_t w[4] = {vx.x, vx.y, vx.z, vx.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16lo_to_f32(w[j]);
      x[2 * j + 1] = bf16hi_to_f32(w[j]);
    }
    quantise<true>(x, p.v_scale[h], scale, code);
    if (held) {
      *reinterpret_cast<uint32_t*>(page + q4_v_code(tok, l >> 1) + (l & 1) * 4) = code[0] | code[1] << 16;
      if (!(l & 1)) page[q4_v_scale(tok, l >> 1)] = static_cast<uint8_t>(scale[0]);
    }
  }
  __syncthreads();

  // ---- sums of the sub-blocks whose first new row is one of this window's, a warp each (dims 4 lane .. + 3)
  unsigned turned, owners;   // rows that are in the cache; rows that are their sub-block's first new one
  {
    const RowInfo r = info[lane];
    const bool in = lane < kMaxRows && r.b >= 0 && r.phys >= 0;
    turned = __ballot_sync(0xffffffffu, in && r.rot);
    owners = __ballot_sync(0xffffffffu, in && lane < own && (r.at % kSubblock == 0 || r.at == r.first));
  }
  for (int n = 0; owners; owners &= owners - 1, ++n) {
    if (n % n_warps != warp) continue;
    const int j = __ffs(owners) - 1;
    const RowInfo r = info[j];
    const int64_t ph = int64_t(h) * p.n_phys + r.phys;
    const int s0 = r.at / kSubblock * kSubblock, s1 = min(r.end, s0 + kSubblock);   // new: [r.at, s1)
    const unsigned fresh = (1u << (s1 - s0)) - (1u << (r.at - s0)), got = (turned >> j) << (r.at - s0) & fresh;
    // The rows held before, all asked for before the first is added: those in front of the new ones, and what
    // page_cnt (which this call raises no further than its own rows) counts behind them.
    unsigned held = 0;
    uint2 raw[kSubblock];
    if (fresh != 0xFFFFu) {
      const int tok0 = s0 % kPageTokens, cnt = max(0, min(kPageTokens, p.page_cnt[r.phys]));
#pragma unroll
      for (int k = 0; k < kSubblock; ++k) {
        if (fresh >> k & 1) continue;
        if (Q4) {
          const uint8_t* page = p.pool + ph * kQ4Page;
          raw[k].x = *reinterpret_cast<const uint16_t*>(page + q4_k_code(tok0 + k) + 2 * lane);
          raw[k].y = page[q4_k_scale(tok0 + k, lane >> 2)];
        } else {
          raw[k] = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.pool) +
                                                   (ph * kPageTokens + tok0 + k) * kHeadDim + 4 * lane);
        }
      }
      held = ((1u << (r.at - s0)) - 1) | (0xFFFFu << (s1 - s0) & ((1u << max(0, min(kSubblock, cnt - tok0))) - 1));
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kSubblock; ++k) {
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);   // a row that is not there: + 0 changes no sum of this order
      if (got >> k & 1) {
        b = *reinterpret_cast<const float4*>(&rows[j + s0 + k - r.at][4 * lane]);
      } else if (held >> k & 1) {
        if (Q4) b = q4_values(raw[k].x, e4m3_to_f32(raw[k].y));
        else b = make_float4(bf16lo_to_f32(raw[k].x), bf16hi_to_f32(raw[k].x), bf16lo_to_f32(raw[k].y), bf16hi_to_f32(raw[k].y));
      }
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    if (Q4) a.x = __fmul_rn(a.x, gk), a.y = __fmul_rn(a.y, gk), a.z = __fmul_rn(a.z, gk), a.w = __fmul_rn(a.w, gk);
    const int64_t at = (ph * kNSub + (s0 % kPageTokens) / kSubblock) * kHeadDim + 4 * lane;
    if (p.ksum_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.ksum) + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.ksum) + at) = a;
  }
  if (h == 0 && tid < kMaxRows) {
    const RowInfo r = info[tid];
    if (r.b >= 0 && r.phys >= 0 && r.rot) atomicMax(&p.page_cnt[r.phys], r.at % kPageTokens + 1);
  }
}

}  // namespace

cudaError_t launch_append_rope(const spkv_cache* c, AppendRopeParams& p, cudaStream_t st) {
  // Rows per CTA: as many as leave a CTA for every SM.  In us with 1, 4, 16: 32 rows of a decode batch (8 kv heads) 3.8,
  // 3.9, 5.3; 200 of one 8.4, 4.8, 5.8; 300 of two prompts 7.2, 4.6, 4.2; 400 of three (1 kv head, 16 heads) 4.0, 5.0, 7.0.
  p.window = kMaxWindow;
  while (p.window > 1 && (int64_t(p.n_rows) + p.window - 1) / p.window * c->d.n_kv_heads < c->sm_count) p.window /= 4;
  const dim3 grid((p.n_rows + p.window - 1) / p.window, c->d.n_kv_heads);
  return launch_pdl(c->pool4 ? append_rope_kernel<true> : append_rope_kernel<false>, grid,
                    dim3(p.window == kMaxWindow ? 256 : 128), 0, st, p);
}

}  // namespace spkv
