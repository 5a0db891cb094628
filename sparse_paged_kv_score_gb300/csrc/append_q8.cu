// Appends new tokens with their rotary positions applied on the way to an 8-bit cache (q8.cuh): rotated queries out, rotated
// keys and values into their sub-blocks under one scale each, the pooled-key sums, page counts.  Rotation and the rows'
// places as append_rope.cu's.
//
// For each sub-block that gets rows, keys and values apart:
//   s' = max(s, scale of the new rows' largest magnitude)    (s: its scale, if it holds rows beside the new ones)
//   new rows:  c = floor(x / s'),   held rows:  c = floor(c s / s')
// and the keys' sums: s' (sum of c + n / 2) over its n rows, an integer times a power of two.
//
// A CTA takes `window` consecutive rows as append_rope.cu's does; a sub-block is the CTA's that holds its first new row, with
// the at most 15 rows of it that lie behind the window.  Few rows (a decode step): a CTA has one kv head, a half-warp rotates
// a row, its sub-block's largest magnitudes meet in shared memory, and a warp has the keys or the values of a sub-block.
// Many: a CTA has all kv heads, and a warp by itself the sixteen rows of a sub-block's keys, or values, of one head, from its
// loads to its stores, so that nothing waits for other warps; query heads have CTAs of their own.
//
// Measured (GB300, from a replayed graph): 32 rows of a decode batch, 32 + 2 x 8 heads 5.7 us, latency: lengths, page table,
// what the page holds, read one after the other between three barriers; 6000 rows of four prompts 31.7 us = 139 MB at 4.4 TB/s
// (0.66 of the copy rate; to bf16 pages 31), 20000 rows 96 us = 4.8 TB/s; the 6000 without queries 22.7, as one prompt from
// its first token 17.6 of 30.9.  With a CTA a window and head for many rows too (rows through shared memory, a barrier for
// the largest magnitudes and one for the bytes) 6000 and 20000 rows took 42 and 134 us: 600 instructions a warp for two
// rows, and every phase as long as its slowest warp.
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

// What a warp does for one sub-block: part 0 the keys and sums, 1 the values; of a sub-block that is all new 0 and 1 the keys
// of its first and second eight tokens, 2 and 3 the values, and each a quarter of the sums.
struct Task {
  int j;           // the sub-block's first new row, -1: no task
  int part;
  bool whole;
  int phys, tok0;  // its page, its first token there
  int row0;        // list row of its first token (in the window's numbers; before the first new row it is none)
  unsigned got;    // tokens that are appended
  unsigned fresh;  // that are the request's new ones
};
__device__ __forceinline__ Task block_of(const RowInfo& r, int j, unsigned turned) {
  Task t;
  const int s0 = r.at / kSubblock * kSubblock, a = r.at - s0, s1 = min(r.end - s0, kSubblock);   // new: [a, s1)
  t.j = j;
  t.part = -1;
  t.phys = r.phys;
  t.tok0 = s0 % kPageTokens;
  t.row0 = j - a;
  t.fresh = (1u << s1) - (1u << a);
  t.got = (turned >> j) << a & t.fresh;
  t.whole = t.got == 0xFFFFu;
  return t;
}

// Rotates heads [first, end) of the rows that begin in this CTA's window, a half-warp a row.
__device__ __forceinline__ void turn_rows(const AppendRopeParams& p, int first, int end) {
  __shared__ int at[32][4];
  __shared__ int turns[32];
  const int tid = threadIdx.x, lane = tid & 31, hw = tid >> 4, l = lane & 15, i = blockIdx.x * p.window + hw;
  uint4 v[kHeads];
  const uint16_t* q = p.q + int64_t(i) * p.q_stride + first * kHeadDim;
  const bool mine = hw < p.window && i < p.n_rows;
#pragma unroll
  for (int k = 0; k < kHeads; ++k)
    if (mine && first + k < end) v[k] = load_pairs(q + k * kHeadDim, l);
  if (tid < 32) {
    uint32_t bad = 0;   // (the CTAs of the keys report it)
    turns[lane] = find_row(p, blockIdx.x * p.window, lane, at[lane], bad).rot;
  }
  __syncthreads();
  if (!mine || !turns[hw]) return;
  const CosSin t = load_turn(p, at[hw], l);
  uint16_t* to = p.q_out + (int64_t(i) * p.Hq + first) * kHeadDim;
  for (int g = first; g < end; g += kHeads, to += kHeads * kHeadDim) {
    uint4 next[kHeads];
    q += kHeads * kHeadDim;
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
      if (g + kHeads + k < end) next[k] = load_pairs(q + k * kHeadDim, l);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (g + k >= end) break;
      float x[8];
      rotate(v[k], t, true, x);
      store_pairs(to + k * kHeadDim, l, round_pairs(x));
      v[k] = next[k];
    }
  }
}

// Sums of the values of dims 4 lane .. + 3 at element `at` of the sums, of n tokens whose bytes' sums are the halves of lo and hi:
// sum of (c + 1/2) s = (2 sum(u) - 255 n) s / 2.
__device__ __forceinline__ void put_sums(const AppendRopeParams& p, int64_t at, uint32_t lo, uint32_t hi, uint32_t scale, int n) {
  const float s2 = 0.5f * __uint_as_float(scale);
  const float4 a = make_float4(s2 * (2 * static_cast<int>(lo & 0xFFFFu) - 255 * n), s2 * (2 * static_cast<int>(hi & 0xFFFFu) - 255 * n),
                               s2 * (2 * static_cast<int>(lo >> 16) - 255 * n), s2 * (2 * static_cast<int>(hi >> 16) - 255 * n));
  if (p.ksum_bf16)
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.ksum) + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  else
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.ksum) + at) = a;
}

// A CTA's rows of one kv head, and what its sub-blocks need.  top, old_scale, held: of the sub-block that row j opens, keys
// and values: the new rows' largest magnitudes, its scale as it was (0 if it holds nothing else), and the tokens that it
// holds beside the new ones.
struct SmemHead {
  uint32_t keys[kMaxRows][kHeadDim];       // fp32, then a row's 32 words of codes
  uint32_t vals[kMaxRows][kHeadDim / 2];   // bf16, then 32 words of codes
  uint32_t top[kMaxWindow][2];
  uint32_t old_scale[kMaxWindow][2];
  uint32_t held[kMaxWindow];
};

// Few rows: a CTA has one kv head, and rotates its rows' queries of that head's group too.
__global__ void __launch_bounds__(128, 4) append_q8_rows_kernel(const __grid_constant__ AppendRopeParams p) {
  __shared__ __align__(16) SmemHead S;
  __shared__ RowInfo info[32];      // a warp looks up, the last is not of this window
  __shared__ int axis_pos[32][4];
  constexpr int n_warps = 4, n_hw = 8;
  constexpr int kSlots = (kMaxRows + n_hw - 1) / n_hw;   // rows of a half-warp: hw, hw + n_hw, ..
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hw = tid >> 4, l = lane & 15;
  const int h = blockIdx.y, base = blockIdx.x * p.window;
  const int own = min(p.window, p.n_rows - base);
  const bool turn = p.cos_sin != nullptr;
  // this half-warp's query heads: sub, sub + step, .. of row rq
  const int step = n_hw / p.window, rq = hw / step, sub = hw % step;

  // ---- the first rows are on their way while their places are looked up
  uint4 kx = make_uint4(0, 0, 0, 0), vx = kx, qv[kHeads];
  const uint16_t* const k_new = p.k_new + base * p.k_stride + h * kHeadDim;
  const uint16_t* const v_new = p.v_new + base * p.v_stride + h * kHeadDim + 8 * l;
  auto load = [&](int r) {
    kx = load_pairs(k_new + r * p.k_stride, l);
    vx = *reinterpret_cast<const uint4*>(v_new + r * p.v_stride);
  };
  if (hw < own) load(hw);
  const uint16_t* const q = q_row(p, h, base + rq, sub);
  if (rq < own) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
      if (sub + k * step < p.G) qv[k] = load_pairs(q + k * step * kHeadDim, l);
  }
  if (tid < 2 * kMaxWindow) S.top[tid >> 1][tid & 1] = 0;
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

  unsigned turned, opening;   // rows that are appended; rows that are their sub-block's first new one
  {
    const RowInfo r = info[lane];
    const bool in = lane < kMaxRows && r.b >= 0 && r.phys >= 0;
    turned = __ballot_sync(0xffffffffu, in && r.rot);
    opening = __ballot_sync(0xffffffffu, in && lane < own && (r.at % kSubblock == 0 || r.at == r.first));
  }
  // ---- this half-warp's rows: the sub-block that each belongs to (-1: not appended by this CTA), the first one's
  // rotation
  int opener[kSlots];
  CosSin t{};
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int r = hw + s * n_hw;
    opener[s] = -1;
    if (r >= kMaxRows || !(turned >> r & 1)) continue;
    opener[s] = r - min(info[r].at % kSubblock, info[r].at - info[r].first);
    if (s > 0) continue;
    if (r >= own) load(r);
    if (turn) t = load_turn(p, axis_pos[r], l);
  }
  // ---- thread 2 j + side: what the sub-block that row j opens holds beside the new rows, and its scale
  const bool asks = tid < 2 * kMaxWindow && opening >> (tid >> 1) & 1;
  uint32_t held = 0;          // the same for every head
  Task mine{};
  if (asks) {
    mine = block_of(info[tid >> 1], tid >> 1, turned);
    if (mine.fresh != 0xFFFFu) {
      // those in front of the new ones, and what page_cnt (which this call raises no further than its own rows) counts behind
      const int c = max(0, min(kPageTokens, p.page_cnt[mine.phys])) - mine.tok0, s1 = 32 - __clz(mine.fresh);
      held = (((mine.fresh & -mine.fresh) - 1) | (0xFFFFu << s1 & ((1u << max(0, min(kSubblock, c))) - 1))) & ~mine.got;
    }
  }

  auto page_at = [&](int phys) { return p.pool + (int64_t(h) * p.n_phys + phys) * kQ8Page; };
  const uint32_t was = held ? *(reinterpret_cast<const uint32_t*>(page_at(mine.phys) + (tid & 1 ? kQ8VScale : kQ8KScale)) + mine.tok0 / kSubblock) & 0x7FFFFFFFu : 0u;
  // ---- this warp's tasks; what the first one's sub-block holds is asked for
  unsigned owners = opening;
  int number = 0;            // of the next sub-block's first task
  auto next = [&]() {        // this warp's next task
    while (owners) {
      const int j = __ffs(owners) - 1;
      Task x = block_of(info[j], j, turned);
      owners &= owners - 1;
      x.part = (warp - number) & (n_warps - 1);
      const int n = x.whole ? 4 : 2;
      number += n;
      if (x.part < n) return x;
    }
    Task none{};
    none.j = -1;
    return none;
  };
  // the words of this lane's dims 4 lane .. + 3 of the tokens that are not new: keys one a token, values two a pair
  uint32_t old[kSubblock];
  auto ask = [&](const Task& x) {
    if (x.j < 0 || x.whole) return;
    const uint8_t* page = page_at(x.phys);
    if (x.part == 0) {
#pragma unroll
      for (int i = 0; i < kSubblock; ++i)
        if (!(x.got >> i & 1)) old[i] = *reinterpret_cast<const uint32_t*>(page + q8_k_code(x.tok0 + i, 4 * lane));
    } else {
#pragma unroll
      for (int i = 0; i < kSubblock; i += 2) {
        if ((x.got >> i & 3) == 3) continue;
        const uint2 y = *reinterpret_cast<const uint2*>(page + q8_v_code(x.tok0 + i, 4 * lane));
        old[i] = y.x, old[i + 1] = y.y;
      }
    }
  };
  Task task = next();
  ask(task);
  // ---- query heads
  if (rq < own && sub < p.G && info[rq].rot) {
    CosSin u;
    turn_queries(p, h, base + rq, axis_pos[rq], sub, step, l, q, qv, u);
  }
  // ---- rows rotated into shared memory, their sub-blocks' largest magnitudes
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (!__any_sync(0xffffffffu, opener[s] >= 0)) continue;
    const int r = hw + s * n_hw;
    if (s > 0 && opener[s] >= 0) {
      load(r);
      if (turn) t = load_turn(p, axis_pos[r], l);
    }
    float x[8];
    rotate(kx, t, turn, x);
    const uint32_t mk = row_max(x);
    // the largest bf16 magnitude, a NaN the largest
    const uint32_t w[4] = {vx.x, vx.y, vx.z, vx.w};
    uint32_t mv = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mv = max(mv, max((w[j] << 16) & 0x7FFF0000u, w[j] & 0x7FFF0000u));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    if (opener[s] < 0) continue;
    *reinterpret_cast<float4*>(&S.keys[r][4 * l]) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(&S.keys[r][64 + 4 * l]) = make_float4(x[4], x[5], x[6], x[7]);
    *reinterpret_cast<uint4*>(&S.vals[r][4 * l]) = vx;
    if (l == 0) {
      atomicMax(&S.top[opener[s]][0], mk);
      atomicMax(&S.top[opener[s]][1], mv);
    }
  }
  if (tid < 2 * kMaxWindow) {
    S.held[tid >> 1] = held;   // (the same from both threads)
    S.old_scale[tid >> 1][tid & 1] = held ? was : 0u;
  }
  __syncthreads();

  // ---- a row's values to bytes, in place
  auto scale_of = [&](int j, int side) { return max(S.old_scale[j][side], q8_scale(S.top[j][side])); };
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (!__any_sync(0xffffffffu, opener[s] >= 0)) continue;
    const int r = hw + s * n_hw;
    uint32_t code[4] = {};
    if (opener[s] >= 0) {
      const float ik = q8_inverse(scale_of(opener[s], 0)), iv = q8_inverse(scale_of(opener[s], 1));
      const uint4 v = *reinterpret_cast<const uint4*>(&S.vals[r][4 * l]);
      code[0] = ik == 0.f ? 0x80808080u : q8_bytes(*reinterpret_cast<const float4*>(&S.keys[r][4 * l]), ik);
      code[1] = ik == 0.f ? 0x80808080u : q8_bytes(*reinterpret_cast<const float4*>(&S.keys[r][64 + 4 * l]), ik);
      code[2] = iv == 0.f ? 0x80808080u : q8_bytes(make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y)), iv);
      code[3] = iv == 0.f ? 0x80808080u : q8_bytes(make_float4(bf16lo_to_f32(v.z), bf16hi_to_f32(v.z), bf16lo_to_f32(v.w), bf16hi_to_f32(v.w)), iv);
    }
    __syncwarp();   // both rows are read
    if (opener[s] >= 0) {
      S.keys[r][l] = code[0];
      S.keys[r][16 + l] = code[1];
      *reinterpret_cast<uint2*>(&S.vals[r][2 * l]) = make_uint2(code[2], code[3]);
    }
  }
  __syncthreads();

  // ---- the sub-blocks into the pool
  for (bool asked = true; task.j >= 0; task = next(), asked = false) {
    if (!asked) ask(task);
    uint8_t* const page = page_at(task.phys);
    const int sb = task.tok0 / kSubblock, row0 = task.row0;
    const int64_t sums = ((int64_t(h) * p.n_phys + task.phys) * kNSub + sb) * kHeadDim;
    uint32_t* const k_scale = reinterpret_cast<uint32_t*>(page + kQ8KScale) + sb;
    uint32_t* const v_scale = reinterpret_cast<uint32_t*>(page + kQ8VScale) + sb;
    if (task.whole) {
      const int half = 8 * (task.part & 1), r0 = row0 + half, t0 = task.tok0 + half;
      if (task.part < 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // piece: 16 dims of a token; in the pool's order
          const int x = lane + 32 * i, tk = x / 4 % 8, d = 32 * (x % 4) + 16 * (x / 32);
          *reinterpret_cast<uint4*>(page + q8_k_code(t0, 0) + 16 * x) = *reinterpret_cast<const uint4*>(&S.keys[r0 + tk][d / 4]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // 8 dims of two tokens
          const int x = lane + 32 * i, tk = 2 * (x % 4), d = 16 * (x / 4 % 8) + 8 * (x / 32);
          const uint2 a = *reinterpret_cast<const uint2*>(&S.vals[r0 + tk][d / 4]), b = *reinterpret_cast<const uint2*>(&S.vals[r0 + tk + 1][d / 4]);
          *reinterpret_cast<uint4*>(page + q8_v_code(t0, 0) + 16 * x) =
              make_uint4(__byte_perm(a.x, b.x, 0x5140), __byte_perm(a.x, b.x, 0x7362), __byte_perm(a.y, b.y, 0x5140), __byte_perm(a.y, b.y, 0x7362));
        }
      }
      // sums of dims 32 part .. + 31: four tokens a lane, eight lanes' words, then the four of them
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = S.keys[row0 + 4 * (lane >> 3) + i][8 * task.part + (lane & 7)];
        lo += w & 0x00FF00FFu;
        hi += (w >> 8) & 0x00FF00FFu;
      }
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        hi += __shfl_xor_sync(0xffffffffu, hi, o);
      }
      if (lane < 8) put_sums(p, sums + 32 * task.part + 4 * lane, lo, hi, scale_of(task.j, 0), kSubblock);
      if (lane == 0 && task.part == 0) *k_scale = scale_of(task.j, 0);
      if (lane == 0 && task.part == 2) *v_scale = scale_of(task.j, 1);
      continue;
    }
    const unsigned got = task.got, kept = S.held[task.j];
    const uint32_t is = scale_of(task.j, task.part);
    const int k = kept ? q8_shift(S.old_scale[task.j][task.part], is) : 0;
    if (task.part == 0) {
      uint32_t lo = 0, hi = 0;   // sums of the bytes 0 and 2, 1 and 3
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) {
        uint32_t w;
        if (got >> i & 1) w = S.keys[row0 + i][lane];
        else if (kept >> i & 1) w = q8_shrink(old[i], k);
        else continue;
        lo += w & 0x00FF00FFu;
        hi += (w >> 8) & 0x00FF00FFu;
        if ((got >> i & 1) || k) *reinterpret_cast<uint32_t*>(page + q8_k_code(task.tok0 + i, 4 * lane)) = w;
      }
      put_sums(p, sums + 4 * lane, lo, hi, is, __popc(got | kept));
      if (lane == 0) *k_scale = is;
    } else {
#pragma unroll
      for (int i = 0; i < kSubblock; i += 2) {
        uint32_t w[2];
        if ((got >> i & 3) != 3) {
          w[0] = __byte_perm(old[i], old[i + 1], 0x6420);
          w[1] = __byte_perm(old[i], old[i + 1], 0x7531);
        }
        bool change = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (got >> (i + e) & 1) w[e] = S.vals[row0 + i + e][lane], change = true;
          else if ((kept >> (i + e) & 1) && k) w[e] = q8_shrink(w[e], k), change = true;
        }
        if (change)
          *reinterpret_cast<uint2*>(page + q8_v_code(task.tok0 + i, 4 * lane)) =
              make_uint2(__byte_perm(w[0], w[1], 0x5140), __byte_perm(w[0], w[1], 0x7362));
      }
      if (lane == 0) *v_scale = is;
    }
  }
  if (h == 0 && tid < kMaxRows) {
    const RowInfo r = info[tid];
    if (r.b >= 0 && r.phys >= 0 && r.rot) atomicMax(&p.page_cnt[r.phys], r.at % kPageTokens + 1);
  }
}


// Many rows: the window's rows of all kv heads, a warp a task: the keys (or values) of one sub-block and head.
constexpr int kBlockWarps = 8;
constexpr int kCodeRow = kHeadDim / 4 + 4;   // words of a row's codes, padded: 16-byte pieces of neighbouring rows meet no bank twice
struct SmemBlocks {
  float turn[kMaxRows][kHeadDim];                   // cosines and sines of the rows
  uint32_t codes[kBlockWarps][kSubblock][kCodeRow]; // a warp's
  RowInfo info[32];
  int axis_pos[32][4];
};

// x / s rounded down, + 128, in the last 8 bits of the sum with 1.5 * 2^23 (see q8_bytes).
__device__ __forceinline__ uint32_t code_bits(float x, float inverse) { return __float_as_uint(__fmaf_rd(x, inverse, 12582912.f + 128.f)); }
constexpr uint32_t kCodeBase = 0x4B400000u;   // the bits of 1.5 * 2^23

// The words of dims 4 lane .. + 3 that a sub-block holds for tokens that are not new, as they lie: a token's keys, or two
// tokens' values.
__device__ __forceinline__ void ask_held(uint32_t (&w)[kSubblock], const uint8_t* page, const Task& task, int side, int lane) {
#pragma unroll
  for (int i = 0; i < kSubblock; i += 2) {
    if ((task.got >> i & 3) == 3) continue;
    if (side == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) w[i + e] = *reinterpret_cast<const uint32_t*>(page + q8_k_code(task.tok0 + i + e, 4 * lane));
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(page + q8_v_code(task.tok0 + i, 4 * lane));
      w[i] = v.x, w[i + 1] = v.y;
    }
  }
}
// Of a sub-block that is not all new: the codes of the new tokens lie in `codes`, what it holds is w; its bytes, scale and
// (keys) sums are written.
__device__ __forceinline__ void write_part(const AppendRopeParams& p, int64_t ph, const Task& task, int side, uint32_t held, uint32_t was, uint32_t is,
                                           const uint32_t (*codes)[kCodeRow], const uint32_t (&w)[kSubblock], int lane) {
  uint8_t* const page = p.pool + ph * kQ8Page;
  const int k = held ? q8_shift(was, is) : 0;
  uint32_t lo = 0, hi = 0;   // sums of the bytes 0 and 2, 1 and 3
#pragma unroll
  for (int i = 0; i < kSubblock; i += 2) {
    uint32_t x[2] = {w[i], w[i + 1]};
    if (side == 1 && (task.got >> i & 3) != 3) x[0] = __byte_perm(w[i], w[i + 1], 0x6420), x[1] = __byte_perm(w[i], w[i + 1], 0x7531);
    bool change[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool fresh = task.got >> (i + e) & 1, kept = held >> (i + e) & 1;
      if (fresh) x[e] = codes[i + e][lane];
      else if (kept) x[e] = q8_shrink(x[e], k);
      change[e] = fresh || (kept && k);
      if (fresh || kept) lo += x[e] & 0x00FF00FFu, hi += (x[e] >> 8) & 0x00FF00FFu;
      if (side == 0 && change[e]) *reinterpret_cast<uint32_t*>(page + q8_k_code(task.tok0 + i + e, 4 * lane)) = x[e];
    }
    if (side == 1 && (change[0] || change[1]))
      *reinterpret_cast<uint2*>(page + q8_v_code(task.tok0 + i, 4 * lane)) =
          make_uint2(__byte_perm(x[0], x[1], 0x5140), __byte_perm(x[0], x[1], 0x7362));
  }
  const int sb = task.tok0 / kSubblock;
  if (lane == 0) *(reinterpret_cast<uint32_t*>(page + (side ? kQ8VScale : kQ8KScale)) + sb) = is;
  if (side == 0) put_sums(p, (ph * kNSub + sb) * kHeadDim + 4 * lane, lo, hi, is, __popc(task.got | held));
}

__global__ void __launch_bounds__(32 * kBlockWarps, 2) append_q8_blocks_kernel(const __grid_constant__ AppendRopeParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SmemBlocks& S = *reinterpret_cast<SmemBlocks*>(smem_raw);
  pdl_wait();
  pdl_trigger();
  const int kv_ctas = (p.Hk + p.heads - 1) / p.heads;
  if (static_cast<int>(blockIdx.y) >= kv_ctas) {   // query heads
    const int slice = blockIdx.y - kv_ctas, slices = gridDim.y - kv_ctas;
    turn_rows(p, p.Hq * slice / slices, p.Hq * (slice + 1) / slices);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hw = tid >> 4, l = lane & 15;
  const int h0 = blockIdx.y * p.heads, heads = min(p.Hk - h0, p.heads), base = blockIdx.x * kMaxWindow;
  const int own = min(kMaxWindow, p.n_rows - base);
  const bool turn = p.cos_sin != nullptr;
  if (warp == 0) {
    uint32_t bad = 0;
    RowInfo ri = find_row(p, base, lane, S.axis_pos[lane], bad);
    if (lane < own && h0 == 0) flag_error(p.err, bad);
    // its sub-block's first new row is one of the window's
    const int opens = lane - min(ri.at % kSubblock, ri.at - ri.first);
    if (opens < 0 || opens >= own) ri.b = ri.phys = -1;
    S.info[lane] = ri;
  }
  __syncthreads();
  unsigned turned, opening;   // rows that are appended; rows that are their sub-block's first new one
  {
    const RowInfo r = S.info[lane];
    const bool in = lane < kMaxRows && r.b >= 0 && r.phys >= 0;
    turned = __ballot_sync(0xffffffffu, in && r.rot);
    opening = __ballot_sync(0xffffffffu, in && lane < own && (r.at % kSubblock == 0 || r.at == r.first));
  }
  if (turn) {
    for (int r = hw; r < kMaxRows; r += 2 * kBlockWarps) {
      if (!(turned >> r & 1)) continue;
      const CosSin t = load_turn(p, S.axis_pos[r], l);
      *reinterpret_cast<float4*>(&S.turn[r][4 * l]) = make_float4(t.c[0].x, t.c[0].y, t.c[1].x, t.c[1].y);
      *reinterpret_cast<float4*>(&S.turn[r][64 + 4 * l]) = make_float4(t.s[0].x, t.s[0].y, t.s[1].x, t.s[1].y);
    }
  }
  __syncthreads();
  uint32_t(*const codes)[kCodeRow] = S.codes[warp];
  const int per = 2 * heads;   // tasks of a sub-block: keys, values of its heads in turn
  for (int x = warp, before = 0; opening; x += kBlockWarps) {
    while (opening && x >= before + per) opening &= opening - 1, before += per;
    if (!opening) break;
    const int j = __ffs(opening) - 1, h = h0 + (x - before) / 2, side = (x - before) & 1;
    const Task task = block_of(S.info[j], j, turned);
    const int64_t ph = int64_t(h) * p.n_phys + task.phys;
    uint8_t* const page = p.pool + ph * kQ8Page;
    const int sb = task.tok0 / kSubblock;
    uint32_t held = 0, was = 0;
    if (!task.whole) {
      // rows held before: those in front of the new ones, and what page_cnt (which this call raises no further than its own
      // rows) counts behind
      const int c = max(0, min(kPageTokens, p.page_cnt[task.phys])) - task.tok0, s1 = 32 - __clz(task.fresh);
      was = *(reinterpret_cast<const uint32_t*>(page + (side ? kQ8VScale : kQ8KScale)) + sb) & 0x7FFFFFFFu;
      held = (((task.fresh & -task.fresh) - 1) | (0xFFFFu << s1 & ((1u << max(0, min(kSubblock, c))) - 1))) & ~task.got;
      if (!held) was = 0;
    }
    uint32_t old[kSubblock];
    if (!task.whole) ask_held(old, page, task, side, lane);
    if (side == 0) {
      // lane: dims 2 lane, 2 lane + 1 and 64 + those of every row, so that a pair is a lane's
      const uint16_t* from = p.k_new + (base + task.row0) * p.k_stride + h * kHeadDim + 2 * lane;
      uint32_t lo[kSubblock], hi[kSubblock];
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) {
        lo[i] = hi[i] = 0;
        if (!(task.got >> i & 1)) continue;
        lo[i] = *reinterpret_cast<const uint32_t*>(from + i * p.k_stride);
        hi[i] = *reinterpret_cast<const uint32_t*>(from + i * p.k_stride + 64);
      }
      float v[kSubblock][4];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) {
        const float2 y = pair(lo[i]), z = pair(hi[i]);
        v[i][0] = y.x, v[i][1] = y.y, v[i][2] = z.x, v[i][3] = z.y;
        if (turn && (task.got >> i & 1)) {   // products and sums rounded one by one, as rotate() does
          const float2 c = *reinterpret_cast<const float2*>(&S.turn[task.row0 + i][2 * lane]);
          const float2 s = *reinterpret_cast<const float2*>(&S.turn[task.row0 + i][64 + 2 * lane]);
          v[i][0] = __fsub_rn(__fmul_rn(y.x, c.x), __fmul_rn(z.x, s.x));
          v[i][1] = __fsub_rn(__fmul_rn(y.y, c.y), __fmul_rn(z.y, s.y));
          v[i][2] = __fadd_rn(__fmul_rn(z.x, c.x), __fmul_rn(y.x, s.x));
          v[i][3] = __fadd_rn(__fmul_rn(z.y, c.y), __fmul_rn(y.y, s.y));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const uint32_t is = max(was, q8_scale(top));
      const float inv = q8_inverse(is);
      uint32_t sum[4] = {};
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = code_bits(inv == 0.f ? 0.f : v[i][e], inv);
          sum[e] += u[e];
        }
        uint16_t* row = reinterpret_cast<uint16_t*>(codes[i]);
        row[lane] = static_cast<uint16_t>(__byte_perm(u[0], u[1], 0x0040));
        row[32 + lane] = static_cast<uint16_t>(__byte_perm(u[2], u[3], 0x0040));
      }
      __syncwarp();
      if (!task.whole) {
        write_part(p, ph, task, side, held, was, is, codes, old, lane);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // 16 dims of a token, in the pool's order
          const int piece = lane + 32 * i, t = 8 * (i >> 1) + (lane >> 2), d = 32 * (lane & 3) + 16 * (i & 1);
          *reinterpret_cast<uint4*>(page + q8_k_code(task.tok0, 0) + 16 * piece) = *reinterpret_cast<const uint4*>(&codes[t][d / 4]);
        }
        // sums of (c + 1/2) s = (2 sum(u) - 255 n) s / 2
        const float s2 = 0.5f * __uint_as_float(is);
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = s2 * (2 * static_cast<int>(sum[e] - kSubblock * kCodeBase) - 255 * kSubblock);
        const int64_t at = (ph * kNSub + sb) * kHeadDim + 2 * lane;
        if (p.ksum_bf16) {
          uint16_t* to = reinterpret_cast<uint16_t*>(p.ksum) + at;
          *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(a[0], a[1]);
          *reinterpret_cast<uint32_t*>(to + 64) = pack_bf16x2(a[2], a[3]);
        } else {
          float* to = reinterpret_cast<float*>(p.ksum) + at;
          *reinterpret_cast<float2*>(to) = make_float2(a[0], a[1]);
          *reinterpret_cast<float2*>(to + 64) = make_float2(a[2], a[3]);
        }
        if (lane == 0) *(reinterpret_cast<uint32_t*>(page + kQ8KScale) + sb) = is;
      }
    } else {
      // lane: dims 4 lane .. + 3 of every row
      const uint16_t* from = p.v_new + (base + task.row0) * p.v_stride + h * kHeadDim + 4 * lane;
      uint2 v[kSubblock];
      uint32_t top = 0;   // largest magnitudes of even and odd dims, bf16
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) {
        v[i] = make_uint2(0, 0);
        if (task.got >> i & 1) v[i] = *reinterpret_cast<const uint2*>(from + i * p.v_stride);
      }
#pragma unroll
      for (int i = 0; i < kSubblock; ++i) top = __vmaxu2(top, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
      top = __reduce_max_sync(0xffffffffu, max(top << 16, top & 0xFFFF0000u));
      const uint32_t is = max(was, q8_scale(top));
      const float inv = q8_inverse(is);
      uint32_t w[kSubblock];
#pragma unroll
      for (int i = 0; i < kSubblock; ++i)
        w[i] = inv == 0.f ? 0x80808080u : q8_bytes(make_float4(bf16lo_to_f32(v[i].x), bf16hi_to_f32(v[i].x), bf16lo_to_f32(v[i].y), bf16hi_to_f32(v[i].y)), inv);
      if (!task.whole) {
#pragma unroll
        for (int i = 0; i < kSubblock; ++i) codes[i][lane] = w[i];
        __syncwarp();
        write_part(p, ph, task, side, held, was, is, codes, old, lane);
      } else {
#pragma unroll
        for (int i = 0; i < kSubblock; i += 2)
          *reinterpret_cast<uint2*>(page + q8_v_code(task.tok0 + i, 4 * lane)) =
              make_uint2(__byte_perm(w[i], w[i + 1], 0x5140), __byte_perm(w[i], w[i + 1], 0x7362));
        if (lane == 0) *(reinterpret_cast<uint32_t*>(page + kQ8VScale) + sb) = is;
      }
    }
    __syncwarp();   // the warp's codes are free again
  }
  if (h0 == 0 && tid < kMaxRows) {
    const RowInfo r = S.info[tid];
    if (r.b >= 0 && r.phys >= 0 && r.rot) atomicMax(&p.page_cnt[r.phys], r.at % kPageTokens + 1);
  }
}

}  // namespace

cudaError_t append_q8_init_attributes() {
  return cudaFuncSetAttribute(append_q8_blocks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SmemBlocks));
}

cudaError_t launch_append_q8(const spkv_cache* c, AppendRopeParams& p, cudaStream_t st) {
  // Rows per CTA as in append_rope.cu: as many as leave a CTA for every SM.
  p.window = kMaxWindow;
  while (p.window > 1 && (int64_t(p.n_rows) + p.window - 1) / p.window * c->d.n_kv_heads < c->sm_count) p.window /= 4;
  const int x = (p.n_rows + p.window - 1) / p.window, Hk = c->d.n_kv_heads;
  if (p.window < kMaxWindow) return launch_pdl(append_q8_rows_kernel, dim3(x, Hk), dim3(128), 0, st, p);
  // kv heads of a CTA: all, or as few as leave a CTA for every place on the SMs
  p.heads = Hk;
  while (p.heads > 1 && int64_t(x) * ((Hk + p.heads - 1) / p.heads) < int64_t(2) * c->sm_count) --p.heads;
  // slices of 16 query heads: four batches of loads a half-warp
  return launch_pdl(append_q8_blocks_kernel, dim3(x, (Hk + p.heads - 1) / p.heads + (p.q ? (p.Hq + 15) / 16 : 0)),
                    dim3(32 * kBlockWarps), sizeof(SmemBlocks), st, p);
}

}  // namespace spkv
