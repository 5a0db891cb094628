// Appends new tokens with their rotary positions applied on the way to an 8-bit cache (q8.cuh): rotated queries out, rotated
// keys and values into their sub-blocks under one scale each, the pooled-key sums, page counts.  Rotation and the rows'
// places as append_rope.cu's.
//
// For each sub-block that gets rows, keys and values apart:
//   s' = max(s, scale of the new rows' largest magnitude)    (s: its scale, if it holds rows beside the new ones)
//   new rows:  c = floor(x / s'),   held rows:  c = floor(c s / s')
// and the keys' sums: s' (sum of c + n / 2) over its n rows, an integer times a power of two.
//
// One CTA takes `window` consecutive rows of one kv head as append_rope.cu's does; a sub-block is the CTA's that holds its
// first new row, with the at most 15 rows of it that lie behind the window.  A half-warp a row rotates it into shared
// memory and raises its sub-block's largest magnitudes; then a warp a sub-block (keys or values) makes the bytes of all its
// tokens, four dims a lane.
#include "append_rope.cuh"
#include "q8.cuh"

namespace spkv {
namespace {

// Largest magnitude's bits over the 8 values of each of 16 lanes (a half-warp's row).
__device__ __forceinline__ uint32_t row_max(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__global__ void __launch_bounds__(256, 4) append_q8_kernel(const __grid_constant__ AppendRopeParams p) {
  __shared__ RowInfo info[32];      // a warp looks up, the last is not of this window
  __shared__ int axis_pos[32][4];
  __shared__ uint32_t top[kMaxWindow][2];   // largest magnitudes of the sub-block that row j opens: keys, values
  __shared__ __align__(16) float keys[kMaxRows][kHeadDim];
  __shared__ __align__(16) uint32_t vals[kMaxRows][kHeadDim / 2];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hw = tid >> 4, l = lane & 15;
  const int n_warps = blockDim.x >> 5, n_hw = blockDim.x >> 4;
  const int h = blockIdx.y, base = blockIdx.x * p.window;
  const int own = min(p.window, p.n_rows - base);
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
  if (rq < own) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
      if (sub + k * step < p.G) qv[k] = load_pairs(q_row(p, h, base + rq, sub + k * step), l);
  }
  if (tid < 2 * kMaxWindow) top[tid >> 1][tid & 1] = 0;
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
  if (rq < own && sub < p.G && info[rq].rot) turn_queries(p, h, base + rq, axis_pos[rq], sub, step, l, qv, t);
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
    float x[8];
    rotate(kx, t, turn, x);
    const uint32_t mk = row_max(x);
    const uint32_t w[4] = {vx.x, vx.y, vx.z, vx.w};
    if (held) {
      *reinterpret_cast<float4*>(&keys[r][4 * l]) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(&keys[r][64 + 4 * l]) = make_float4(x[4], x[5], x[6], x[7]);
      *reinterpret_cast<uint4*>(&vals[r][4 * l]) = vx;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16lo_to_f32(w[j]);
      x[2 * j + 1] = bf16hi_to_f32(w[j]);
    }
    const uint32_t mv = row_max(x);
    if (held && l == 0) {
      const int j = r - min(ri.at % kSubblock, ri.at - ri.first);
      atomicMax(&top[j][0], mk);
      atomicMax(&top[j][1], mv);
    }
  }
  __syncthreads();

  // ---- sub-blocks whose first new row is one of this window's, a warp for the keys of one and a warp for its values
  unsigned turned, owners;   // rows that are appended; rows that are their sub-block's first new one
  {
    const RowInfo r = info[lane];
    const bool in = lane < kMaxRows && r.b >= 0 && r.phys >= 0;
    turned = __ballot_sync(0xffffffffu, in && r.rot);
    owners = __ballot_sync(0xffffffffu, in && lane < own && (r.at % kSubblock == 0 || r.at == r.first));
  }
  for (int n = 0; owners; owners &= owners - 1, n += 2) {
    const int side = (warp - n) & (n_warps - 1);   // 0: its keys are this warp's, 1: its values
    if (side > 1) continue;
    const int j = __ffs(owners) - 1;
    const RowInfo r = info[j];
    const int64_t ph = int64_t(h) * p.n_phys + r.phys;
    uint8_t* const page = p.pool + ph * kQ8Page;
    const int s0 = r.at / kSubblock * kSubblock, s1 = min(r.end, s0 + kSubblock);   // new: [r.at, s1)
    const int tok0 = s0 % kPageTokens, sb = tok0 / kSubblock;
    const unsigned fresh = (1u << (s1 - s0)) - (1u << (r.at - s0)), got = (turned >> j) << (r.at - s0) & fresh;
    // rows held before: those in front of the new ones, and what page_cnt (which this call raises no further than its own
    // rows) counts behind them
    unsigned held = 0;
    if (fresh != 0xFFFFu) {
      const int cnt = max(0, min(kPageTokens, p.page_cnt[r.phys]));
      held = ((1u << (r.at - s0)) - 1) | (0xFFFFu << (s1 - s0) & ((1u << max(0, min(kSubblock, cnt - tok0))) - 1));
    }
    uint32_t* const scale = reinterpret_cast<uint32_t*>(page + (side ? kQ8VScale : kQ8KScale)) + sb;
    const uint32_t was = held ? *scale & 0x7FFFFFFFu : 0u;
    const uint32_t is = max(was, q8_scale(top[j][side]));
    const int k = held ? q8_shift(was, is) : 0;
    const float inv = q8_inverse(is);
    const int row0 = j + s0 - r.at;   // row of the sub-block's token 0 in shared memory
    if (side == 0) {
      uint32_t old[kSubblock];
      if (held) {
#pragma unroll
        for (int i = 0; i < kSubblock; ++i)
          if (held >> i & 1) old[i] = *reinterpret_cast<const uint32_t*>(page + q8_k_code(tok0 + i, 4 * lane));
      }
      uint32_t lo = 0, hi = 0;   // sums of the bytes 0 and 2, 1 and 3
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) {
        uint32_t w;
        if (got >> i & 1) w = q8_bytes(*reinterpret_cast<const float4*>(&keys[row0 + i][4 * lane]), inv);
        else if (held >> i & 1) w = q8_shrink(old[i], k);
        else continue;
        lo += w & 0x00FF00FFu;
        hi += (w >> 8) & 0x00FF00FFu;
        if ((got >> i & 1) || k) *reinterpret_cast<uint32_t*>(page + q8_k_code(tok0 + i, 4 * lane)) = w;
      }
      // sum of (c + 1/2) s = (2 sum(u) - 255 n) s / 2
      const int n255 = 255 * __popc(got | held);
      const float s2 = 0.5f * __uint_as_float(is);
      const float4 a = make_float4(s2 * (2 * static_cast<int>(lo & 0xFFFFu) - n255), s2 * (2 * static_cast<int>(hi & 0xFFFFu) - n255),
                                   s2 * (2 * static_cast<int>(lo >> 16) - n255), s2 * (2 * static_cast<int>(hi >> 16) - n255));
      const int64_t at = (ph * kNSub + sb) * kHeadDim + 4 * lane;
      if (p.ksum_bf16)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.ksum) + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.ksum) + at) = a;
    } else {
      uint2 old[kSubblock / 2];
      const unsigned both = 0x5555u & got & (got >> 1);   // pairs of which both tokens are new
#pragma unroll
      for (int i = 0; i < kSubblock / 2; ++i)
        if (!(both >> (2 * i) & 1)) old[i] = *reinterpret_cast<const uint2*>(page + q8_v_code(tok0 + 2 * i, 4 * lane));
#pragma unroll
      for (int i = 0; i < kSubblock / 2; ++i) {
        uint32_t w[2];
        if (!(both >> (2 * i) & 1)) {
          w[0] = __byte_perm(old[i].x, old[i].y, 0x6420);
          w[1] = __byte_perm(old[i].x, old[i].y, 0x7531);
        }
        bool change = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int x = 2 * i + e;
          if (got >> x & 1) {
            const uint2 v = *reinterpret_cast<const uint2*>(&vals[row0 + x][2 * lane]);
            w[e] = q8_bytes(make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y)), inv);
            change = true;
          } else if ((held >> x & 1) && k) {
            w[e] = q8_shrink(w[e], k);
            change = true;
          }
        }
        if (change)
          *reinterpret_cast<uint2*>(page + q8_v_code(tok0 + 2 * i, 4 * lane)) =
              make_uint2(__byte_perm(w[0], w[1], 0x5140), __byte_perm(w[0], w[1], 0x7362));
      }
    }
    __syncwarp();
    if (lane == 0) *scale = is;
  }
  if (h == 0 && tid < kMaxRows) {
    const RowInfo r = info[tid];
    if (r.b >= 0 && r.phys >= 0 && r.rot) atomicMax(&p.page_cnt[r.phys], r.at % kPageTokens + 1);
  }
}

}  // namespace

cudaError_t launch_append_q8(const spkv_cache* c, AppendRopeParams& p, cudaStream_t st) {
  // Rows per CTA as in append_rope.cu: as many as leave a CTA for every SM.
  p.window = kMaxWindow;
  while (p.window > 1 && (int64_t(p.n_rows) + p.window - 1) / p.window * c->d.n_kv_heads < c->sm_count) p.window /= 4;
  const dim3 grid((p.n_rows + p.window - 1) / p.window, c->d.n_kv_heads);
  return launch_pdl(append_q8_kernel, grid, dim3(p.window == kMaxWindow ? 256 : 128), 0, st, p);
}

}  // namespace spkv
