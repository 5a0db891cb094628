// Beam search over a paged cache: the best continuations of a request's beams, and the beams' pages following them.
//
// beam_select.  For request b, beams w with logits x_wv and scores cum_w:
//   lse_w = log sum_v exp(x_wv),  score_wv = x_wv + (cum_w - lse_w),  the K best by score, then beam, then token.
// The logits are read once.  A warp takes 4 KiB of a row (32 lines of 128 bytes, counted from the row's first element
// wherever that lies in memory, so that rows with equal logits have equal sums): each line's maximum, the group's maximum
// m and sum of exp(x - m).  A second kernel, a CTA a request, has then only maxima to look through: it searches for a score
// that at least K of the groups' maxima reach, as then do the K best elements, for a score that K of those groups' lines
// reach, and reads the elements of the lines that reach it again.  Where more are alike than its lists hold, it takes exactly
// K groups, K of their lines and K elements, of equal ones the first each time (an element among the K best lies in a line
// whose maximum is among the K best of the lines', as each line ahead of it holds an element ahead of it, and likewise a line
// in its group; groups, lines and elements are numbered by beam and token).
// Sums are fp32 within 4 KiB, and over a row's groups, a 32nd of them to a lane: a beam's lse is off by up to 7.7e-6 at 128256 tokens (spkv.h
// has the bound; the largest error seen was 3e-7), and so is the order of different beams.  What is added to it has 48 bits, so that a large cum takes nothing
// from the order of a beam's own tokens and rows that are alike tie.
//
// beam_reorder.  Complete pages are shared, so a child takes its parent's table entries; of the part-filled page a parent's
// first child keeps the parent's own, and each other child gets the page of a beam without children, with the parent's rows
// copied into it.  There are as many such beams as such children.
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <new>

#include "common.cuh"

struct spkv_beam_plan {
  int device = 0;
  int max_rows = 0, max_vocab = 0, max_groups = 0;
  float* line_max = nullptr;     // [max_rows * max_groups][32]
  float2* group = nullptr;       // [max_rows * max_groups]: maximum, sum of exp(x - maximum)
};

namespace spkv {
namespace {

constexpr int kGroupBytes = 4096, kLineBytes = 128, kLines = kGroupBytes / kLineBytes;
constexpr int kMaxBeams = 64, kMaxBest = 128;
constexpr int kWarps = 16, kThreads = 32 * kWarps;   // of the second kernel
constexpr int kGroupThreads = 128, kCtasPerSm = 6, kStages = 2;   // of the first; groups of a warp in shared memory
constexpr int kMaxGroups = 32768;   // of a request: as many keys as shared memory holds

struct BeamParams {
  const uint8_t* logits;
  int64_t row_bytes;
  int W, V, K, groups;           // groups: 4 KiB pieces of a row
  int rows;
  const float* cum;
  int32_t* tokens;
  int32_t* parents;
  float* scores;
  float* line_max;
  float2* group;
  uint32_t* err;
};

template <typename T>
struct Traits;
template <>
struct Traits<float> {
  static constexpr uint32_t kNegInf = 0xFF800000u;   // in every element of a word
  static __device__ __forceinline__ float top(uint4 v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct Traits<__nv_bfloat16> {
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ float2 pair(uint32_t a) { return make_float2(bf16lo_to_f32(a), bf16hi_to_f32(a)); }
  static __device__ __forceinline__ float top(uint4 v) {
    const __nv_bfloat162 a = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&v.x), *reinterpret_cast<__nv_bfloat162*>(&v.y));
    const __nv_bfloat162 b = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&v.z), *reinterpret_cast<__nv_bfloat162*>(&v.w));
    const float2 f = __bfloat1622float2(__hmax2(a, b));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Traits<__half> {
  static constexpr uint32_t kNegInf = 0xFC00FC00u;
  static __device__ __forceinline__ float2 pair(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2*>(&a)); }
  static __device__ __forceinline__ float top(uint4 v) {
    const __half2 a = __hmax2(*reinterpret_cast<__half2*>(&v.x), *reinterpret_cast<__half2*>(&v.y));
    const __half2 b = __hmax2(*reinterpret_cast<__half2*>(&v.z), *reinterpret_cast<__half2*>(&v.w));
    const float2 f = __half22float2(__hmax2(a, b));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// s0 + s1 grow by 2^(x log2e - c) of each x: the product is exact within the fused addition, so a term is off by the
// rounding of its own exponent only.
__device__ __forceinline__ void add_exps(float& s0, float& s1, float x0, float x1, float c) {
  float t0, t1;
  fma_f32x2(t0, t1, x0, x1, kLog2e, kLog2e, -c, -c);
  add_f32x2(s0, s1, ex2(t0), ex2(t1));
}
template <typename T>
__device__ __forceinline__ void add_exps(float& s0, float& s1, uint4 v, float c) {
  if constexpr (sizeof(T) == 4) {
    add_exps(s0, s1, __uint_as_float(v.x), __uint_as_float(v.y), c);
    add_exps(s0, s1, __uint_as_float(v.z), __uint_as_float(v.w), c);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = Traits<T>::pair(w[j]);
      add_exps(s0, s1, x.x, x.y, c);
    }
  }
}
// exp(x - m) for any maximum m: NaN for NaN and for m = infinity, 0 for m = -infinity.
__device__ __forceinline__ float far_exp(float x, float m) {
  return x != x || m == CUDART_INF_F ? CUDART_NAN_F : m == -CUDART_INF_F ? 0.f : ex2((x - m) * kLog2e);
}
template <typename T>
__device__ __forceinline__ float far_exps(uint4 v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) {
      s += far_exp(__uint_as_float(w[j]), m);
    } else {
      const float2 x = Traits<T>::pair(w[j]);
      s += far_exp(x.x, m) + far_exp(x.y, m);
    }
  }
  return s;
}

// Numbers of about 48 bits: hi is the nearest fp32 number, lo the rest.  (This card's 64-bit units are few: a warp's
// addition keeps an SM's busy for 15 cycles, and the second kernel took twice as long with them.)
struct F2 {
  float hi, lo;
};
__device__ __forceinline__ F2 sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ F2 plus(F2 a, float b) {
  const F2 s = sum_of(a.hi, b);
  const float e = __fadd_rn(s.lo, a.lo), hi = __fadd_rn(s.hi, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, s.hi))};
}

// Quarters of scores (which stay in fp32's range) as integers of the same order; 0 for what is no candidate.
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float x, F2 off) {
  if (!(x > -CUDART_INF_F) || off.hi == -CUDART_INF_F) return 0;
  const F2 s = plus(off, 0.25f * x);
  return static_cast<Key>(float_order_key(s.hi)) << 32 | float_order_key(s.lo);
}
__device__ __forceinline__ float score_of(Key k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return 4.f * __uint_as_float(u >> 31 ? u & 0x7FFFFFFFu : ~u);
}
// A quarter of m + log s, s at least 1, to 2^-24: the log of s is that of a power of two and of a number in [1, 2).
__device__ __forceinline__ F2 quarter_lse(float m, float s) {
  constexpr float kHi = 0x1.62e4p-1f, kLo = 1.42860682e-6f;   // ln 2, the first with 15 bits
  const int bits = __float_as_int(s), e = (bits >> 23) - 127;
  const float f = __int_as_float((bits & 0x007FFFFF) | 0x3F800000);
  return plus(plus(sum_of(0.25f * m, e * (0.25f * kHi)), e * (0.25f * kLo)), 0.25f * logf(f));
}

// What a search may leave: groups, lines, elements.  `key` has room for the lines of as many groups at least.
constexpr int kListed = 256, kElements = 1024, kMinRoom = kListed * kLines;

struct SmemBeam {
  F2 off[kMaxBeams];         // a quarter of cum - lse; -infinity for a beam without candidates
  int groups[kListed], lines[kListed];
  Key best[kElements];       // the elements that are left
  int place[kElements];
  int list[kMaxBest], sorted[kMaxBest];
  Key lo[kWarps], hi[kWarps];
  int count[2][kWarps];
  int left[3];               // groups, lines, elements that reach the score
  int n;
  uint32_t key[kMinRoom];    // high halves of the keys of the items that are searched (more, for many groups)
};

// The sum of every thread's x; `turn` alternates between calls in a row.
__device__ __forceinline__ int block_sum(SmemBeam& S, int x, int& turn) {
  x = __reduce_add_sync(0xffffffffu, x);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) S.count[turn][threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < kWarps ? S.count[turn][threadIdx.x & 31] : 0);
}

// A half key that at least K of the n in S.key reach (0 is none), 1 if there are fewer, and at most `most` where they differ
// enough.  Each thread comes with the least, largest and number of keys of its own.  A search by halves.
__device__ __noinline__ uint32_t threshold(SmemBeam& S, int n, int K, int most, int& turn, uint32_t lo, uint32_t hi, int mine) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) S.lo[warp] = lo, S.hi[warp] = hi;
  int c = block_sum(S, mine, turn);     // keys that reach lo
  lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? static_cast<uint32_t>(S.lo[lane]) : lo);
  hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? static_cast<uint32_t>(S.hi[lane]) : hi);
  if (c < K) return 1;
  while (c > most && lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    int x = 0;
    for (int i = tid; i < n; i += kThreads) x += S.key[i] >= mid;
    x = block_sum(S, x, turn);
    if (x >= K) lo = mid, c = x;
    else hi = mid - 1;
  }
  return lo;
}

// The first min(K, candidates) of n items by key, then index: their indices, ascending, to S.sorted.  Returns how many.
// Searches by halves over keys, which are formed anew at each look, then for equal ones over indices.
template <typename F>
__device__ int select_best(SmemBeam& S, int n, int K, F make) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int turn = 0;
  auto count = [&](auto which) {
    int x = 0;
    for (int i = tid; i < n; i += kThreads) x += which(make(i), i);
    return block_sum(S, x, turn);
  };
  Key lo = ~0ull, hi = 0;
  for (int i = tid; i < n; i += kThreads) {
    const Key k = make(i);
    if (k) lo = min(lo, k), hi = max(hi, k);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (lane == 0) S.lo[warp] = lo, S.hi[warp] = hi;
  if (tid == 0) S.n = 0;
  int c = count([](Key k, int) { return k != 0; });
  for (int w = 0; w < kWarps; ++w) lo = min(lo, S.lo[w]), hi = max(hi, S.hi[w]);
  const int want = min(K, c);
  if (want == 0) return 0;
  while (c > want && lo < hi) {
    const Key mid = lo + (hi - lo + 1) / 2;
    const int x = count([&](Key k, int) { return k >= mid; });
    if (x >= want) lo = mid, c = x;
    else hi = mid - 1;
  }
  int until = n;    // of the items with the key lo, those with indices below this one
  if (c > want) {
    int a = 0, b = n;    // the smallest `until` that leaves enough lies in (a, b]
    while (b - a > 1) {
      const int mid = (a + b) / 2;
      if (count([&](Key k, int i) { return k > lo || (k == lo && i < mid); }) >= want) b = mid;
      else a = mid;
    }
    until = b;
  }
  for (int i = tid; i < n; i += kThreads) {
    const Key k = make(i);
    if (k > lo || (k == lo && i < until)) S.list[atomicAdd(&S.n, 1)] = i;
  }
  __syncthreads();
  if (tid < want) {
    const int i = S.list[tid];
    int at = 0;
    for (int j = 0; j < want; ++j) at += S.list[j] < i;
    S.sorted[at] = i;
  }
  __syncthreads();
  return want;
}

// An element, or a line's maximum, its beam, and an element's place.
struct Item {
  float x;
  int w, place;
};
constexpr int kLineBits = 20, kLineMask = (1 << kLineBits) - 1;
static_assert(kMaxGroups * kLines <= 1 << kLineBits && kMaxBeams <= 1 << (31 - kLineBits) && kLines == 32, "a line and its beam in an int");

// Where item i of a request's groups, of the lines of listed groups and of the elements of listed lines lies, and its key.
template <typename T>
struct Items {
  const BeamParams& p;
  const F2* off;
  int b;
  static constexpr int kEach = kLineBytes / sizeof(T);
  __device__ __forceinline__ int64_t first() const { return int64_t(b) * p.W * p.groups; }   // the request's first group
  __device__ __forceinline__ Key group(int g) const {
    return key_of(p.group[first() + g].x, off[g / p.groups]);
  }
  // Groups and lines are listed with their beam: line = beam << kLineBits | group * kLines + its line of the group.
  __device__ __forceinline__ int listed(int g) const { return (g / p.groups) << (kLineBits - 5) | g; }
  __device__ __forceinline__ Item line(int x) const { return {p.line_max[first() * kLines + (x & kLineMask)], x >> kLineBits, 0}; }
  // element e of line x; place: beam * V + token
  __device__ __forceinline__ Item element(int x, int e) const {
    const int w = x >> kLineBits, token = ((x & kLineMask) - w * p.groups * kLines) * kEach + e;
    if (token >= p.V) return {-CUDART_INF_F, w, w * p.V + token};
    return {Traits<T>::one(reinterpret_cast<const T*>(p.logits + (int64_t(b) * p.W + w) * p.row_bytes) + token), w, w * p.V + token};
  }
  __device__ __forceinline__ Key key(const Item& i) const { return key_of(i.x, off[i.w]); }
};

// The K best of n elements in S.best, S.place to the outputs, -1, -1, -infinity behind them: four lanes count what is ahead
// of an element.
__device__ __forceinline__ void write_best(SmemBeam& S, const BeamParams& p, int b, int n) {
  const int64_t o = int64_t(b) * p.K;
  for (int i = threadIdx.x >> 2; i - (threadIdx.x >> 2 & 7) < n; i += kThreads / 4) {   // by warps
    const Key k = i < n ? S.best[i] : ~0ull;
    const uint32_t half = static_cast<uint32_t>(k >> 32);
    int at = 0, same = 0;   // elements ahead by their half keys, with the same half (itself one of them)
    for (int j = threadIdx.x & 3; j < n; j += 4) {
      const uint32_t other = S.best[j] >> 32;
      at += other > half;
      same += other == half;
    }
    const int place = i < n ? S.place[i] : 0;
    if (__any_sync(0xffffffffu, i < n && same > (static_cast<int>(threadIdx.x & 3) == (i & 3))))
      for (int j = threadIdx.x & 3; j < n; j += 4) {
        const Key o = S.best[j];
        at += o >> 32 == half && (o > k || (o == k && S.place[j] < place));
      }
    at += __shfl_xor_sync(0xffffffffu, at, 1);
    at += __shfl_xor_sync(0xffffffffu, at, 2);
    if ((threadIdx.x & 3) || i >= n || at >= p.K) continue;
    const int w = place / p.V;
    p.tokens[o + at] = place - w * p.V;
    p.parents[o + at] = w;
    p.scores[o + at] = score_of(k);
  }
  for (int i = n + threadIdx.x; i < p.K; i += kThreads) {
    p.tokens[o + i] = p.parents[o + i] = -1;
    p.scores[o + i] = -CUDART_INF_F;
  }
}

constexpr int kVec = kGroupBytes / 512;   // 16-byte vectors of a lane

// A group's bytes in shared memory, from the 16-byte border at or before its first one on.
constexpr int kStage = kGroupBytes + 16;

// Asks for the group `from` of the row [begin, end), nothing outside the row.  By a warp.
template <typename T>
__device__ __forceinline__ void ask(uint8_t* stage, const uint8_t* from, const uint8_t* begin, const uint8_t* end, int lane) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
  const uint8_t* const at = from - off + lane * 16;
  const uint32_t to = smem_u32(stage) + lane * 16;
  if (from - off >= begin && from - off + kStage <= end) {
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * 512), "l"(at + k * 512) : "memory");
    if (lane == 0) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + kGroupBytes), "l"(at + kGroupBytes) : "memory");
    return;
  }
  auto copy = [&](int x) {   // 16 bytes from x on, zeros behind the row
    const int64_t left = end - (at + x);
    const int n = left >= 16 ? 16 : left > 0 ? static_cast<int>(left) : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + x), "l"(n ? at + x : begin - (reinterpret_cast<uintptr_t>(begin) & 15)), "r"(n) : "memory");
  };
  const bool head = at < begin;   // the row begins inside its first 16 bytes
#pragma unroll
  for (int k = 0; k < kVec; ++k)
    if (k > 0 || !head) copy(k * 512);
  if (lane == 0 && off) copy(kGroupBytes);
  if (head)
    for (const uint8_t* e = begin; e < at + 16 && e < end; e += sizeof(T)) *reinterpret_cast<T*>(stage + (e - at)) = *reinterpret_cast<const T*>(e);
}

// A group that has arrived: vector k of the lane holds the bytes from 512 k + 16 lane on, elements from `left` on as -infinity.
template <typename T>
__device__ __forceinline__ void take(uint4 (&v)[kVec], const uint8_t* stage, int off, int left, int lane) {
  const uint8_t* const at = stage + off + lane * 16;
  if (off == 0) {
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[k] = *reinterpret_cast<const uint4*>(at + k * 512);
  } else {
    const bool half = sizeof(T) == 2 && (off & 2);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(at - (half ? 2 : 0));
    const uint32_t pick = half ? 0x5432 : 0x3210;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const uint32_t a = w[k * 128], b = w[k * 128 + 1], c = w[k * 128 + 2], d = w[k * 128 + 3];
      const uint32_t e = half ? w[k * 128 + 4] : 0;
      v[k] = make_uint4(__byte_perm(a, b, pick), __byte_perm(b, c, pick), __byte_perm(c, d, pick), __byte_perm(d, e, pick));
    }
  }
  constexpr int kPer = 16 / sizeof(T);
  if (left < kGroupBytes / static_cast<int>(sizeof(T))) {
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const int n = left - k * (512 / static_cast<int>(sizeof(T))) - lane * kPer;   // elements of the vector that exist
      uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          if (j >= n) w[j] = Traits<T>::kNegInf;
        } else {
          if (2 * j + 1 >= n) w[j] = 2 * j >= n ? Traits<T>::kNegInf : (w[j] & 0xFFFFu) | (Traits<T>::kNegInf & 0xFFFF0000u);
        }
      }
      v[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// A group's maxima of lines, its own and its sum, from the lane's vectors.
template <typename T>
__device__ __forceinline__ void look_at_group(const BeamParams& p, const uint4 (&v)[kVec], int64_t i, int lane) {
  // vector k of eight lanes is line 4 k + lane / 8; each lane ends with that of k = lane % 8
  float m[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) m[k] = Traits<T>::top(v[k]);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const bool up = lane & o;
      const float give = up ? m[k] : m[k + o], keep = up ? m[k + o] : m[k];
      m[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  p.line_max[i * kLines + 4 * (lane & 7) + (lane >> 3)] = m[0];
  float top = m[0];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float s = 0.f;
  if (fabsf(top) < 0x1p24f) {   // c is off by 1 at most: so are the exponents, which the last factor puts right
    const float c = __fmul_rn(top, kLog2e);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < kVec; ++k) add_exps<T>(s0, s1, v[k], c);
    s = (s0 + s1) * ex2(-fmaf(top, kLog2e, -c));   // what c was rounded by
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k) s += far_exps<T>(v[k], top);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.group[i] = make_float2(top, s);
}

// A warp takes groups a grid of warps apart, with kStages - 1 of them on their way.
// Of bound: the logits' bytes, and beside them half of the issue slots (2 elements a packed conversion, maximum and exponential).
// 24 warps an SM with 8 KiB of ring each beat fewer with more (4 CTAs of 3 stages 27.6 us, 6 of 2 26.0 before the second
// kernel's last steps) and registers filled by plain loads (28.5).  32 requests x 8 beams x 128256 bf16, 65.7 MB, 9.8 us at the
// copy rate: both kernels 22.5 us from a replayed graph, fp16 22.5; fp32 32.9 (of 19.7).
template <typename T>
__global__ void __launch_bounds__(kGroupThreads, kCtasPerSm) beam_groups_kernel(const __grid_constant__ BeamParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* const mine = smem_raw + warp * kStages * kStage;
  const int step = gridDim.x * (kGroupThreads / 32), step_row = step / p.groups, step_g = step % p.groups;
  pdl_wait();
  pdl_trigger();
  struct Place {
    int row, g;
  };
  auto forward = [&](Place x) {
    x.row += step_row;
    x.g += step_g;
    if (x.g >= p.groups) x.g -= p.groups, ++x.row;
    return x;
  };
  auto cum_of = [&](Place x) { return x.row < p.rows ? p.cum[x.row] : 0.f; };
  const int first = blockIdx.x * (kGroupThreads / 32) + warp;
  Place next{first / p.groups, first % p.groups};   // to be asked for, with its beam's score (not waited for until then)
  float cum = cum_of(next);
  Place queue[kStages - 1];
  auto ask_next = [&](int s) {
    // a beam that has ended is not read, nor what would be written of it
    while (cum == -CUDART_INF_F) next = forward(next), cum = cum_of(next);
    const Place x = next;
    if (x.row < p.rows) {
      const uint8_t* const r0 = p.logits + x.row * p.row_bytes;
      ask<T>(mine + s * kStage, r0 + int64_t(x.g) * kGroupBytes, r0, r0 + int64_t(p.V) * sizeof(T), lane);
      next = forward(x);
      cum = cum_of(next);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return x;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) queue[s] = ask_next(s);
  for (int s = 0; queue[0].row < p.rows; s = s + 1 == kStages ? 0 : s + 1) {
    const Place x = queue[0];
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();   // every lane's copies are there, and every lane is through with the stage before
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) queue[k] = queue[k + 1];
    queue[kStages - 2] = ask_next(s == 0 ? kStages - 1 : s - 1);
    uint4 v[kVec];
    const uint8_t* const r0 = p.logits + x.row * p.row_bytes;
    take<T>(v, mine + s * kStage, static_cast<int>(reinterpret_cast<uintptr_t>(r0) & 15),   // (a group is a multiple of 16 bytes)
            p.V - x.g * (kGroupBytes / static_cast<int>(sizeof(T))), lane);
    look_at_group<T>(p, v, int64_t(x.row) * p.groups + x.g, lane);
  }
}

// A CTA a request: its K best from its groups' maxima and sums.
// Bound by latency: three searches, each reads what the one before has found.  4 beams x 32000 with the first kernel 6.5 us
// from a replayed graph, one row 6.0; 64-bit keys and scores in it took 12.1.  4 requests of 64 beams x 128256 fp32, K = 128, 54 us (19.7 for the bytes),
// by the instructions of one CTA a request: 59 with a division for each line and element and whole keys compared at the end.
template <typename T>
__global__ void __launch_bounds__(kThreads) beam_best_kernel(const __grid_constant__ BeamParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SmemBeam& S = *reinterpret_cast<SmemBeam*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  if (tid < 3) S.left[tid] = 0;
  pdl_wait();
  pdl_trigger();
  const Items<T> it{p, S.off, b};
  // ---- a warp a beam: its log of the sum of exponentials, its groups' keys
  uint32_t lo = ~0u, hi = 0;
  int mine = 0;
  auto keep = [&](int i, Key k) {
    const uint32_t half = static_cast<uint32_t>(k >> 32);
    S.key[i] = half;
    if (half) ++mine, lo = min(lo, half), hi = max(hi, half);
  };
  for (int w = warp; w < p.W; w += kWarps) {
    const float2* g = p.group + it.first() + int64_t(w) * p.groups;
    const float cum = p.cum[b * p.W + w];
    // the first groups of a lane are asked for at once, and with the score
    constexpr int kFew = 4;
    float2 x[kFew];
#pragma unroll
    for (int k = 0; k < kFew; ++k) x[k] = lane + 32 * k < p.groups ? g[lane + 32 * k] : make_float2(-CUDART_INF_F, 0.f);
    F2 off{-CUDART_INF_F, 0.f};
    if (cum != -CUDART_INF_F) {
      float m = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
      for (int i = lane + 32 * kFew; i < p.groups; i += 32) m = fmaxf(m, g[i].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float s = 0.f;
      auto add = [&](float2 y) { s += y.y == 0.f ? 0.f : y.y * expf(y.x - m); };   // (-infinity - m may be no number)
#pragma unroll
      for (int k = 0; k < kFew; ++k) add(x[k]);
      for (int i = lane + 32 * kFew; i < p.groups; i += 32) add(g[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const bool bad = !(cum < CUDART_INF_F) || !(s < CUDART_INF_F);   // NaN or +infinity among the logits or as score
      if (bad && lane == 0) flag_error(p.err, SPKV_DEVERR_BEAM);
      if (!bad && s > 0.f) {
        const F2 lse = quarter_lse(m, s);
        off = plus(sum_of(0.25f * cum, -lse.hi), -lse.lo);
      }
    }
#pragma unroll
    for (int k = 0; k < kFew; ++k)
      if (lane + 32 * k < p.groups) keep(w * p.groups + lane + 32 * k, key_of(x[k].x, off));
    for (int i = lane + 32 * kFew; i < p.groups; i += 32) keep(w * p.groups + i, key_of(g[i].x, off));
    if (lane == 0) S.off[w] = off;
  }
  const int n = p.W * p.groups, most = p.K + max(p.K / 2, 8);
  int turn = 0;
  // ---- the groups that reach a score that K groups reach (all, if there are fewer)
  uint32_t t = threshold(S, n, p.K, most, turn, lo, hi, mine);
  for (int i = tid; i < n; i += kThreads) {
    if (S.key[i] < t) continue;
    const int x = atomicAdd(&S.left[0], 1);
    if (x < kListed) S.groups[x] = it.listed(i);
  }
  __syncthreads();
  auto element_of = [&](int i) { return it.element(S.lines[i / it.kEach], i % it.kEach); };
  auto line_of = [&](int i) { return S.groups[i / kLines] * kLines + i % kLines; };
  bool fits = S.left[0] <= kListed;
  if (fits) {
    // ---- their lines that reach it; where those are many (groups that are much alike, or few), that reach a score that
    // K lines reach
    const int lines = S.left[0] * kLines;
    lo = ~0u, hi = 0, mine = 0;
    auto collect = [&](int i) {
      if (S.key[i] < t) return;
      const int at = atomicAdd(&S.left[1], 1);
      if (at < kListed) S.lines[at] = line_of(i);
    };
    for (int i = tid; i < lines; i += kThreads) {
      keep(i, it.key(it.line(line_of(i))));
      collect(i);
    }
    __syncthreads();
    if (S.left[1] > min(2 * most, kListed)) {
      t = threshold(S, lines, p.K, most, turn, lo, hi, mine);
      if (tid == 0) S.left[1] = 0;
      __syncthreads();
      for (int i = tid; i < lines; i += kThreads) collect(i);
      __syncthreads();
    }
    fits = S.left[1] <= kListed;
  }
  if (fits) {
    // ---- their elements that reach it
    for (int i = tid; i < S.left[1] * it.kEach; i += kThreads) {
      const Item x = element_of(i);
      const Key k = it.key(x);
      if (k >> 32 < t) continue;
      const int at = atomicAdd(&S.left[2], 1);
      if (at < kElements) S.best[at] = k, S.place[at] = x.place;
    }
    __syncthreads();
    if (S.left[2] <= kElements) return write_best(S, p, b, S.left[2]);
  }
  // ---- too many alike: exactly K groups, of their lines exactly K, of those lines' elements
  __syncthreads();
  const int ng = select_best(S, n, p.K, [&](int i) { return it.group(i); });
  if (tid < ng) S.groups[tid] = it.listed(S.sorted[tid]);
  __syncthreads();
  const int nl = select_best(S, ng * kLines, p.K, [&](int i) { return it.key(it.line(line_of(i))); });
  if (tid < nl) S.lines[tid] = line_of(S.sorted[tid]);
  __syncthreads();
  const int ne = select_best(S, nl * it.kEach, p.K, [&](int i) { return it.key(element_of(i)); });
  if (tid < ne) {
    const Item x = element_of(S.sorted[tid]);
    S.best[tid] = it.key(x);
    S.place[tid] = x.place;
  }
  __syncthreads();
  write_best(S, p, b, ne);
}

// ---------------------------------------------------------------------------------------------- reordering

struct ReorderParams {
  const int32_t* parents;
  int32_t* table;
  const int32_t* seq_len;
  int W, Hk, np_max;
  uint8_t* pool[2];              // of `planes` pools: page-heads of page_bytes
  int planes, page_bytes;
  int row_bytes;                 // of a token in them; 0: page-heads are copied whole
  uint8_t* ksum;
  int ksum_bytes;                // of a page-head
  int32_t* page_cnt;
  int64_t n_phys;
  int32_t* arrived;
  uint32_t* err;
};

constexpr int kStrip = 64;      // columns of a table that are permuted together
constexpr int kCopyThreads = 256, kCopyCtas = 4;
constexpr int kPieces = 5;      // 16-byte pieces of a page-head that a thread copies at most, of a plane
static_assert(kPieces * kCopyThreads * 16 >= 16416, "a page-head of any format");

struct SmemReorder {
  int parent[kMaxBeams];
  int first[kMaxBeams];     // a beam's first child, -1 if that is the beam itself, kMaxBeams if it has none
  int page[kMaxBeams];      // part-filled pages as they were, and their rows
  int rows[kMaxBeams];
  int page_of[kMaxBeams];   // the beam whose part-filled page becomes beam w's
  int copied[kMaxBeams];    // beams whose part-filled page is a copy
  unsigned keeps[2], used[2], copies[2];   // bits: children that keep a page, beams with children, children with copies
  int tile[kMaxBeams][kStrip];
};

// gridDim.x CTAs a request share its copies (a beam's part-filled page, one head) and its tables' strips; each finds out for
// itself what the request's beams do.  The last of them to have read the column of part-filled pages writes it.
// Bound by latency: four reads one after the other, lengths and parents, the column, the pages' rows, their bytes.  32 requests x
// 8 beams of about 4000 tokens, 8 heads, bf16, 88 pages copied, 10.9 us from a replayed graph (3.9 for the bytes); one of 4 beams
// 3.9; 8 beams of 262144 tokens 6.0, mostly tables.  A CTA a beam and head took 19.5, 4.9 and 9.3.
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ SmemReorder S;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y, x = blockIdx.x, W = p.W;
  int32_t* const table = p.table + int64_t(b) * W * p.np_max;
  const int L = p.seq_len[int64_t(b) * W], full = L / kPageTokens;
  const bool part = L % kPageTokens != 0;
  // ---- who goes on from whom
  int parent = -1;
  uint32_t bad = L < 0 || full + (part ? 1 : 0) > p.np_max ? SPKV_DEVERR_PAGE_ID : 0u;
  if (tid < W) {
    parent = p.parents[int64_t(b) * W + tid];
    if (parent < -1 || parent >= W || p.seq_len[int64_t(b) * W + tid] != L) bad |= SPKV_DEVERR_BEAM;
    S.parent[tid] = parent;
    S.first[tid] = kMaxBeams;
  }
  if (__syncthreads_or(bad != 0)) {
    if (x == 0) flag_error(p.err, bad);
    return;
  }
  if (part && tid < W) {   // (the pages' rows are not waited for before the copies need them)
    S.page[tid] = table[int64_t(tid) * p.np_max + full];
    if (parent >= 0) atomicMin(&S.first[parent], parent == tid ? -1 : tid);
  }
  __syncthreads();
  if (!part) {
  } else if (tid < kMaxBeams) {   // two warps
    const bool keep = tid < W && parent >= 0 && S.first[parent] == (parent == tid ? -1 : tid);
    const bool used = tid < W && S.first[tid] < kMaxBeams;
    const unsigned k = __ballot_sync(0xffffffffu, keep), u = __ballot_sync(0xffffffffu, used || tid >= W);
    const unsigned c = __ballot_sync(0xffffffffu, parent >= 0 && !keep);
    if (lane == 0) S.keeps[warp] = k, S.used[warp] = u, S.copies[warp] = c;
    if (tid < W) {
      const int ph = S.page[tid];
      S.rows[tid] = !p.page_cnt || ph < 0 || ph >= p.n_phys ? kPageTokens : p.page_cnt[ph];
    }
  }
  __syncthreads();
  int before = -1;
  if (part) {
    // every thread of this CTA has read the column
    if (tid == kCopyThreads - 1)
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived + b) : "memory");
    if (tid < W) {
      int from = parent;
      const bool keep = S.keeps[warp] >> lane & 1;
      if (!keep) {   // as many beams have no children as keep no page: the r-th for the r-th
        int r = __popc(~S.keeps[warp] & ((1u << lane) - 1)) + (warp ? __popc(~S.keeps[0]) : 0);
        unsigned f = ~S.used[0];
        int at = 0;
        if (r >= __popc(f)) r -= __popc(f), f = ~S.used[1], at = 32;
        while (r--) f &= f - 1;
        from = at + __ffs(f) - 1;
        if (parent >= 0) S.copied[__popc(S.copies[warp] & ((1u << lane) - 1)) + (warp ? __popc(S.copies[0]) : 0)] = tid;
      }
      S.page_of[tid] = from;
    }
  }
  __syncthreads();
  // ---- copies: a plane (keys, or values, or the one of a packed cache) of a head
  const int copies = part ? __popc(S.copies[0]) + __popc(S.copies[1]) : 0, each = p.Hk * p.planes;
  for (int i = x; i < copies * each; i += gridDim.x) {
    const int w = S.copied[i / each], h = i % each / p.planes, k = i % p.planes;
    const int src = S.page[S.parent[w]], dst = S.page[S.page_of[w]], rows = S.rows[S.parent[w]];
    if (src < 0 || src >= p.n_phys || dst < 0 || dst >= p.n_phys) {
      if (i % each == 0 && tid == 0) flag_error(p.err, SPKV_DEVERR_PHYS);
      continue;
    }
    const int bytes = p.row_bytes ? max(0, min(kPageTokens, rows)) * p.row_bytes : p.page_bytes;
    const int64_t from = int64_t(h) * p.n_phys + src, to = int64_t(h) * p.n_phys + dst;
    uint8_t* const pool = k ? p.pool[1] : p.pool[0];
    const bool sums = k == 0 && p.ksum && tid * 16 < p.ksum_bytes;
    uint4 v[kPieces], sum;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int at = (j * kCopyThreads + tid) * 16;
      if (at < bytes) v[j] = *reinterpret_cast<const uint4*>(pool + from * p.page_bytes + at);
    }
    if (sums) sum = *reinterpret_cast<const uint4*>(p.ksum + from * p.ksum_bytes + tid * 16);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int at = (j * kCopyThreads + tid) * 16;
      if (at < bytes) *reinterpret_cast<uint4*>(pool + to * p.page_bytes + at) = v[j];
    }
    if (sums) *reinterpret_cast<uint4*>(p.ksum + to * p.ksum_bytes + tid * 16) = sum;
    if (p.page_cnt && i % each == 0 && tid == 0) p.page_cnt[dst] = rows;
  }
  // ---- complete pages
  for (int c0 = x * kStrip; c0 < full; c0 += gridDim.x * kStrip) {
    const int n = min(kStrip, full - c0);
    for (int i = tid; i < W * kStrip; i += kCopyThreads)
      if (i % kStrip < n) S.tile[i / kStrip][i % kStrip] = table[int64_t(i / kStrip) * p.np_max + c0 + i % kStrip];
    __syncthreads();
    for (int i = tid; i < W * kStrip; i += kCopyThreads) {
      const int w = i / kStrip, from = S.parent[w];
      if (i % kStrip < n && from >= 0 && from != w) table[int64_t(w) * p.np_max + c0 + i % kStrip] = S.tile[from][i % kStrip];
    }
    __syncthreads();
  }
  // ---- the column of part-filled pages
  const bool last = before == static_cast<int>(gridDim.x) - 1;
  if (last) p.arrived[b] = 0;
  if (__syncthreads_or(last) && tid < W) table[int64_t(tid) * p.np_max + full] = S.page[S.page_of[tid]];
}

}  // namespace
}  // namespace spkv

using spkv::kCtasPerSm;
using spkv::kGroupBytes;
using spkv::kMaxBeams;
using spkv::kMaxBest;

namespace {

bool on_device(int device) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

size_t smem_of(int64_t keys) {
  return sizeof(spkv::SmemBeam) + sizeof(uint32_t) * (std::max(keys, int64_t(spkv::kMinRoom)) - spkv::kMinRoom);
}

template <typename T>
cudaError_t launch_select_beams(const spkv::BeamParams& p, int B, int sms, cudaStream_t st) {
  constexpr int each = spkv::kGroupThreads / 32;
  const int ctas = std::min((p.rows * p.groups + each - 1) / each, kCtasPerSm * sms);
  const cudaError_t e = spkv::launch_pdl(spkv::beam_groups_kernel<T>, dim3(ctas), dim3(spkv::kGroupThreads), each * spkv::kStages * spkv::kStage, st, p);
  if (e != cudaSuccess) return e;
  return spkv::launch_pdl(spkv::beam_best_kernel<T>, dim3(B), dim3(spkv::kThreads), smem_of(int64_t(p.W) * p.groups), st, p);
}

template <typename T>
cudaError_t allow_smem() {
  const cudaError_t e = cudaFuncSetAttribute(spkv::beam_groups_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             spkv::kGroupThreads / 32 * spkv::kStages * spkv::kStage);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(spkv::beam_best_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_of(spkv::kMaxGroups)));
}

}  // namespace

extern "C" {

int beam_plan_create(spkv_cache_t c, int max_rows, int max_vocab, spkv_beam_plan_t* out) {
  if (!out) return SPKV_EINVAL;
  *out = nullptr;
  if (!c || max_rows <= 0 || max_vocab <= 0 || !on_device(c->device)) return SPKV_EINVAL;
  if (max_rows > 65536 || max_vocab > (1 << 24)) return SPKV_EUNSUPPORTED;
  spkv_beam_plan* p = new (std::nothrow) spkv_beam_plan();
  if (!p) return SPKV_ENOMEM;
  p->device = c->device;
  p->max_rows = max_rows;
  p->max_vocab = max_vocab;
  p->max_groups = static_cast<int>((int64_t(max_vocab) * 4 + kGroupBytes - 1) / kGroupBytes);   // of fp32 rows
  const int64_t n = int64_t(max_rows) * p->max_groups;
  if (allow_smem<float>() != cudaSuccess || allow_smem<__nv_bfloat16>() != cudaSuccess || allow_smem<__half>() != cudaSuccess) {
    delete p;
    return SPKV_ECUDA;
  }
  if (cudaMalloc(&p->line_max, n * 32 * sizeof(float)) != cudaSuccess || cudaMalloc(&p->group, n * sizeof(float2)) != cudaSuccess) {
    cudaGetLastError();
    beam_plan_destroy(p);
    return SPKV_ENOMEM;
  }
  *out = p;
  return SPKV_OK;
}

int beam_plan_destroy(spkv_beam_plan_t p) {
  if (!p) return SPKV_EINVAL;
  cudaFree(p->line_max);
  cudaFree(p->group);
  delete p;
  return SPKV_OK;
}

int beam_select(spkv_cache_t c, spkv_beam_plan_t plan, const void* logits, int type, int64_t row_stride, int B, int W, int V,
                const float* cum, int K, int32_t* tokens, int32_t* parents, float* scores, void* stream) {
  if (!c || !plan || B < 0 || W <= 0 || V <= 0 || K <= 0) return SPKV_EINVAL;
  if (type != SPKV_F32 && type != SPKV_BF16 && type != SPKV_F16) return SPKV_EINVAL;
  if (W > kMaxBeams || K > kMaxBest) return SPKV_EUNSUPPORTED;
  const int es = type == SPKV_F32 ? 4 : 2;
  if (int64_t(B) * W > plan->max_rows || V > plan->max_vocab || row_stride < V) return SPKV_EINVAL;
  if (B == 0) return SPKV_OK;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % es != 0 || !cum || !tokens || !parents || !scores || plan->device != c->device ||
      !on_device(c->device))
    return SPKV_EINVAL;
  spkv::BeamParams p = {};
  p.logits = static_cast<const uint8_t*>(logits);
  p.row_bytes = row_stride * es;
  p.W = W;
  p.V = V;
  p.K = K;
  p.groups = static_cast<int>((int64_t(V) * es + kGroupBytes - 1) / kGroupBytes);
  p.rows = B * W;
  if (int64_t(W) * p.groups > spkv::kMaxGroups || int64_t(B) * W * p.groups > (int64_t(1) << 30)) return SPKV_EUNSUPPORTED;
  p.cum = cum;
  p.tokens = tokens;
  p.parents = parents;
  p.scores = scores;
  p.line_max = plan->line_max;
  p.group = plan->group;
  p.err = c->dev_err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == SPKV_F32    ? launch_select_beams<float>(p, B, c->sm_count, st)
                        : type == SPKV_BF16 ? launch_select_beams<__nv_bfloat16>(p, B, c->sm_count, st)
                                            : launch_select_beams<__half>(p, B, c->sm_count, st);
  return e == cudaSuccess ? SPKV_OK : SPKV_ECUDA;
}

int beam_reorder(spkv_cache_t c, const int32_t* parents, int B, int W, int32_t* page_table, int np_max, const int32_t* seq_len,
                 void* stream) {
  if (!c || B < 0 || W <= 0) return SPKV_EINVAL;
  if (W > kMaxBeams) return SPKV_EUNSUPPORTED;
  if (int64_t(B) * W * c->d.n_kv_heads > c->max_units) return SPKV_EINVAL;
  if (B == 0) return SPKV_OK;
  if (!parents || !page_table || np_max <= 0 || !seq_len || !on_device(c->device)) return SPKV_EINVAL;
  spkv::ReorderParams p = {};
  p.parents = parents;
  p.table = page_table;
  p.seq_len = seq_len;
  p.W = W;
  p.Hk = c->d.n_kv_heads;
  p.np_max = np_max;
  if (c->packed()) {
    p.pool[0] = c->pool4 ? c->pool4 : c->pool8;
    p.planes = 1;
    p.page_bytes = c->pool4 ? 9216 : 16416;
  } else {
    p.pool[0] = static_cast<uint8_t*>(c->d.k_pool);
    p.pool[1] = static_cast<uint8_t*>(c->d.v_pool);
    p.planes = 2;
    p.page_bytes = 16384;
    p.row_bytes = 256;
  }
  p.ksum = static_cast<uint8_t*>(c->d.ksum);
  p.ksum_bytes = 4 * 128 * (c->d.ksum_bf16 ? 2 : 4);
  p.page_cnt = c->d.page_cnt;
  p.n_phys = c->d.n_phys_pages;
  p.arrived = c->beam_cnt;
  p.err = c->dev_err;
  // CTAs of a request: as many as there are copies or strips, as many an SM in all as it has room for
  const int64_t work = std::max(int64_t(W - 1) * p.Hk * p.planes, int64_t(np_max + spkv::kStrip - 1) / spkv::kStrip);
  const int64_t x = std::max(int64_t(1), std::min(work, int64_t(spkv::kCopyCtas) * c->sm_count / B));
  return spkv::launch_pdl(spkv::beam_reorder_kernel, dim3(static_cast<unsigned>(x), B), dim3(spkv::kCopyThreads), 0,
                          static_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? SPKV_OK
             : SPKV_ECUDA;
}

}  // extern "C"
