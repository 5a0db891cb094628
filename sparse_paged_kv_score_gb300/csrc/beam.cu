// Beam search over a paged cache: the best continuations of a request's beams, and the beams' pages following them.
//
// beam_select.  For request b, beams w with logits x_wv and scores cum_w:
//   lse_w = log sum_v exp(x_wv),  score_wv = x_wv + (cum_w - lse_w),  the K best by score, then beam, then token.
// The logits are read once.  A warp takes 4 KiB of a row (32 lines of 128 bytes, counted from the row's first element
// wherever that lies in memory, so that rows with equal logits have equal sums): each line's maximum, the group's maximum
// m and sum of exp(x - m).  The last CTA of a request to arrive has
// then only maxima to look through: an element among the K best lies in a line whose maximum is among the K best of the
// lines' (each line ahead of it holds an element ahead of it), and likewise a line in its group.  So it finds the K best
// groups of all beams, of their lines the K best, and of those lines' elements, read again, the K best; of equal ones
// the first each time, which is the order asked for, as groups, lines and elements are numbered by beam and token.
// Sums are fp32 within 4 KiB, then 64 bits, as scores are: those of different beams may lie close together.
//
// beam_reorder.  Complete pages are shared, so a child takes its parent's table entries; of the part-filled page a parent's
// first child keeps the parent's own, and each other child gets the page of a beam without children, with the parent's rows
// copied into it.  There are as many such beams as such children.
#include <cuda_fp16.h>
#include <math_constants.h>

#include <new>

#include "common.cuh"

struct spkv_beam_plan {
  int device = 0;
  int max_rows = 0, max_vocab = 0, max_groups = 0;
  float* line_max = nullptr;     // [max_rows * max_groups][32]
  float2* group = nullptr;       // [max_rows * max_groups]: maximum, sum of exp(x - maximum)
  int32_t* arrived = nullptr;    // [max_rows], 0 between calls
};

namespace spkv {
namespace {

constexpr int kGroupBytes = 4096, kLineBytes = 128, kLines = kGroupBytes / kLineBytes;
constexpr int kMaxBeams = 64, kMaxBest = 128;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKept = 4096;   // keys that are kept in shared memory; more are formed anew at each look

struct BeamParams {
  const uint8_t* logits;
  int64_t row_bytes;
  int W, V, K, groups, ctas;     // groups: 4 KiB pieces of a row; ctas of a request
  const float* cum;
  int32_t* tokens;
  int32_t* parents;
  float* scores;
  float* line_max;
  float2* group;
  int32_t* arrived;
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
  static __device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
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

__device__ __forceinline__ float exp_of(float x, float m) {   // exp(x - m), x <= m
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - m) * 1.4426950408889634f));
  return y;
}
template <typename T>
__device__ __forceinline__ float exps_of(uint4 v, float m) {
  if constexpr (sizeof(T) == 4) {
    return (exp_of(__uint_as_float(v.x), m) + exp_of(__uint_as_float(v.y), m)) +
           (exp_of(__uint_as_float(v.z), m) + exp_of(__uint_as_float(v.w), m));
  } else {
    const float2 a = Traits<T>::pair(v.x), b = Traits<T>::pair(v.y), c = Traits<T>::pair(v.z), d = Traits<T>::pair(v.w);
    return ((exp_of(a.x, m) + exp_of(a.y, m)) + (exp_of(b.x, m) + exp_of(b.y, m))) +
           ((exp_of(c.x, m) + exp_of(c.y, m)) + (exp_of(d.x, m) + exp_of(d.y, m)));
  }
}

// Scores as integers of the same order; 0 for what is no candidate (-infinity, NaN).
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(double s) {
  const long long b = __double_as_longlong(s);
  if (!(s > -CUDART_INF)) return 0;
  return b < 0 ? ~static_cast<Key>(b) : static_cast<Key>(b) | 0x8000000000000000ull;
}
__device__ __forceinline__ double score_of(Key k) {
  return __longlong_as_double(static_cast<long long>(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

struct SmemBeam {
  Key key[kKept];
  double off[kMaxBeams];     // cum - lse; -infinity for a beam without candidates
  int list[kMaxBest], sorted[kMaxBest], from[kMaxBest];
  Key best[kMaxBest];
  Key lo[kWarps], hi[kWarps];
  int count[2][kWarps];
  int n;
  int last;
};

// The sum of every thread's x; `turn` alternates between calls in a row.
__device__ __forceinline__ int block_sum(SmemBeam& S, int x, int& turn) {
  x = __reduce_add_sync(0xffffffffu, x);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) S.count[turn][threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += S.count[turn][w];
  return s;
}

// The first min(K, candidates) of n items by key, then index: their indices, ascending, to S.sorted.  Returns how many.
// A search by halves over keys; where keys are equal at the end, one over indices.
template <typename F>
__device__ int select_best(SmemBeam& S, int n, int K, F make) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool kept = n <= kKept;
  Key lo = ~0ull, hi = 0;
  int mine = 0, turn = 0;
  for (int i = tid; i < n; i += kThreads) {
    const Key k = make(i);
    if (kept) S.key[i] = k;
    if (k) {
      ++mine;
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
  auto get = [&](int i) { return kept ? S.key[i] : make(i); };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (lane == 0) S.lo[warp] = lo, S.hi[warp] = hi;
  if (tid == 0) S.n = 0;
  const int some = block_sum(S, mine, turn);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) lo = min(lo, S.lo[w]), hi = max(hi, S.hi[w]);
  const int want = min(K, some);
  if (want == 0) {
    __syncthreads();
    return 0;
  }
  int until = n;    // of the items with the key lo, those with indices below this one
  int c = some;     // items with keys from lo on
  while (c > want && lo < hi) {
    const Key mid = lo + (hi - lo + 1) / 2;
    int x = 0;
    for (int i = tid; i < n; i += kThreads) x += get(i) >= mid;
    x = block_sum(S, x, turn);
    if (x >= want) lo = mid, c = x;
    else hi = mid - 1;
  }
  if (c > want) {   // more items with the key lo than there is room for
    int a = 0, b = n;    // the smallest `until` that leaves enough lies in (a, b]
    while (b - a > 1) {
      const int mid = (a + b) / 2;
      int x = 0;
      for (int i = tid; i < n; i += kThreads) {
        const Key k = get(i);
        x += k > lo || (k == lo && i < mid);
      }
      x = block_sum(S, x, turn);
      if (x >= want) b = mid;
      else a = mid;
    }
    until = b;
  }
  for (int i = tid; i < n; i += kThreads) {
    const Key k = get(i);
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

// A request's K best from its groups' maxima and sums.
template <typename T>
__device__ void finish(SmemBeam& S, const BeamParams& p, int b) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t g0 = int64_t(b) * p.W * p.groups;   // the request's first group
  for (int w = warp; w < p.W; w += kWarps) {
    const float2* g = p.group + g0 + int64_t(w) * p.groups;
    const float cum = p.cum[b * p.W + w];
    float m = -CUDART_INF_F;
    for (int i = lane; i < p.groups; i += 32) m = fmaxf(m, __ldcg(&g[i].x));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double s = 0;
    for (int i = lane; i < p.groups; i += 32) {
      const float2 x = __ldcg(&g[i]);
      if (x.y != 0.f) s += static_cast<double>(x.y) * expf(x.x - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      const bool bad = !(cum < CUDART_INF_F) || !(s < CUDART_INF);   // NaN or +infinity among the logits or as score
      flag_error(p.err, bad ? SPKV_DEVERR_BEAM : 0u);
      S.off[w] = bad || s == 0 || cum == -CUDART_INF_F ? -CUDART_INF : static_cast<double>(cum) - (m + log(s));
    }
  }
  __syncthreads();
  // groups of all beams
  const int ng = select_best(S, p.W * p.groups, p.K, [&](int i) {
    const double off = S.off[i / p.groups];
    return off == -CUDART_INF ? Key(0) : key_of(__ldcg(&p.group[g0 + i].x) + off);
  });
  if (tid < ng) S.from[tid] = S.sorted[tid];
  __syncthreads();
  // their lines
  const int nl = select_best(S, ng * kLines, p.K, [&](int i) {
    const int g = S.from[i / kLines];
    return key_of(__ldcg(&p.line_max[(g0 + g) * kLines + i % kLines]) + S.off[g / p.groups]);
  });
  int line = 0;   // thread t's: group * kLines + line of the t-th line
  if (tid < nl) line = S.from[S.sorted[tid] / kLines] * kLines + S.sorted[tid] % kLines;
  __syncthreads();
  if (tid < nl) S.from[tid] = line;
  __syncthreads();
  // their elements
  constexpr int kEach = kLineBytes / sizeof(T);
  auto look = [&](int i, int& w, int& token) {
    const int x = S.from[i / kEach], g = x / kLines;
    w = g / p.groups;
    token = ((g - w * p.groups) * kLines + x % kLines) * kEach + i % kEach;
    if (token >= p.V) return Key(0);
    return key_of(Traits<T>::one(reinterpret_cast<const T*>(p.logits + (int64_t(b) * p.W + w) * p.row_bytes) + token) + S.off[w]);
  };
  const int n = select_best(S, nl * kEach, p.K, [&](int i) {
    int w, token;
    return look(i, w, token);
  });
  int w = -1, token = -1;
  Key k = 0;
  if (tid < n) {
    k = look(S.sorted[tid], w, token);
    S.best[tid] = k;
  }
  __syncthreads();
  if (tid < p.K) {
    int at = tid;
    if (tid < n) {
      at = 0;
      for (int j = 0; j < n; ++j) at += S.best[j] > k || (S.best[j] == k && j < tid);
    }
    const int64_t o = int64_t(b) * p.K + at;
    p.tokens[o] = token;
    p.parents[o] = w;
    p.scores[o] = tid < n ? static_cast<float>(score_of(k)) : -CUDART_INF_F;
  }
}

constexpr int kVec = kGroupBytes / 512;   // 16-byte vectors of a lane

// The 16 bytes at `at` (16-byte aligned), elements outside [begin, end) as -infinity, which are not read.
template <typename T>
__device__ __forceinline__ uint4 load_inside(const uint8_t* at, const uint8_t* begin, const uint8_t* end) {
  if (at >= begin && at + 16 <= end) return *reinterpret_cast<const uint4*>(at);
  constexpr uint32_t none = Traits<T>::kNegInf;
  uint32_t word[4] = {none, none, none, none};
#pragma unroll
  for (int j = 0; j < 16 / static_cast<int>(sizeof(T)); ++j) {
    const uint8_t* e = at + j * sizeof(T);
    if (e < begin || e >= end) continue;
    if constexpr (sizeof(T) == 4) {
      word[j] = *reinterpret_cast<const uint32_t*>(e);
    } else {
      const uint32_t x = *reinterpret_cast<const uint16_t*>(e);
      word[j / 2] = j & 1 ? (word[j / 2] & 0xFFFFu) | x << 16 : (word[j / 2] & 0xFFFF0000u) | x;
    }
  }
  return make_uint4(word[0], word[1], word[2], word[3]);
}

// Vectors that begin Q words (and half a word) into the aligned ones v, in place: what lies behind a lane's own vector is
// the next lane's, for the last lane the first lane's of the next k (`last` for the last k).
template <int Q, bool HALF>
__device__ __forceinline__ void shift(uint4 (&v)[kVec], uint4 last, int lane) {
  constexpr int need = Q + (HALF ? 1 : 0);
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const uint4 mine = v[k], next = k + 1 < kVec ? v[k + 1 < kVec ? k + 1 : k] : last;
    const uint32_t give[4] = {lane ? mine.x : next.x, lane ? mine.y : next.y, lane ? mine.z : next.z, lane ? mine.w : next.w};
    uint32_t w[9] = {mine.x, mine.y, mine.z, mine.w, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < need; ++j) w[4 + j] = __shfl_sync(0xffffffffu, give[j], (lane + 1) & 31);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = HALF ? __byte_perm(w[Q + j], w[Q + j + 1], 0x5432) : w[Q + j];
    v[k] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// A group's 4 KiB at `from`, which may begin at any element, of the row [begin, end): vector k of the lane holds the bytes
// from 512 k + 16 lane on, -infinity behind the row.
template <typename T>
__device__ __forceinline__ void load_group(uint4 (&v)[kVec], const uint8_t* from, const uint8_t* begin, const uint8_t* end, int lane) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
  const uint8_t* const at = from - off + lane * 16;
  const uint8_t* const stop = from - off + kGroupBytes;   // the first vector behind the lanes', of which a part is the group's
  uint4 last = make_uint4(0, 0, 0, 0);
  if (from - off >= begin && stop + (off ? 16 : 0) <= end) {
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[k] = *reinterpret_cast<const uint4*>(at + k * 512);
    if (off && lane == 0) last = *reinterpret_cast<const uint4*>(stop);
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[k] = load_inside<T>(at + k * 512, begin, end);
    if (off && lane == 0) last = load_inside<T>(stop, begin, end);
  }
  // (a row that begins at the same place as its neighbours' lines goes one way for all its groups)
  if (off & 2) {
    if constexpr (sizeof(T) == 2) {
      switch (off >> 2) {
        case 0: return shift<0, true>(v, last, lane);
        case 1: return shift<1, true>(v, last, lane);
        case 2: return shift<2, true>(v, last, lane);
        default: return shift<3, true>(v, last, lane);
      }
    }
  }
  switch (off >> 2) {
    case 0: return;
    case 1: return shift<1, false>(v, last, lane);
    case 2: return shift<2, false>(v, last, lane);
    default: return shift<3, false>(v, last, lane);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const __grid_constant__ BeamParams p) {
  __shared__ SmemBeam S;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.ctas, i = (blockIdx.x % p.ctas) * kWarps + warp;   // group of the request
  if (i < p.W * p.groups) {
    const int w = i / p.groups, g = i - w * p.groups;
    const int64_t row = int64_t(b) * p.W + w, at_group = row * p.groups + g;
    const uint8_t* const r0 = p.logits + row * p.row_bytes;
    const uint8_t* const end = r0 + int64_t(p.V) * sizeof(T);
    const uint8_t* const from = r0 + int64_t(g) * kGroupBytes;
    float top = -CUDART_INF_F, sum = 0.f;
    if (p.cum[row] != -CUDART_INF_F) {   // a beam that ended is not read
      uint4 v[kVec];
      load_group<T>(v, from, r0, end, lane);
      // maxima of lines: vector k of eight lanes is line 4 k + lane / 8; each lane ends with that of k = lane % 8
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
      p.line_max[at_group * kLines + 4 * (lane & 7) + (lane >> 3)] = m[0];
      top = m[0];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float ref = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll
      for (int k = 0; k < kVec; ++k) sum += exps_of<T>(v[k], ref);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) p.group[at_group] = make_float2(top, sum);
  }
  __syncthreads();
  if (tid == 0) {
    int before;   // release: this CTA's groups, which the barrier has ordered before; acquire: the others'
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived + b) : "memory");
    S.last = before == p.ctas - 1;
    if (S.last) p.arrived[b] = 0;
  }
  __syncthreads();
  if (S.last) finish<T>(S, p, b);
}

// ---------------------------------------------------------------------------------------------- reordering

struct ReorderParams {
  const int32_t* parents;
  int32_t* table;
  const int32_t* seq_len;
  int W, Hk, np_max;
  uint8_t* pool[2];              // pages of 64 bytes_row bytes, or of page_bytes that are copied whole
  int64_t page_bytes;
  int row_bytes;                 // 0: whole pages
  uint8_t* ksum;
  int ksum_bytes;                // of a page-head
  int32_t* page_cnt;
  int64_t n_phys;
  int32_t* arrived;
  uint32_t* err;
};

constexpr int kStrip = 64;   // columns of a table that a CTA permutes

// What a request's beams do: where beam w's part-filled page comes from and whether it has to be copied there.
struct Family {
  int parent[kMaxBeams];
  int page_of[kMaxBeams];   // the beam whose part-filled page becomes beam w's
};

// Fills F from the parents of request b; false (and flags) where they cannot be followed.  Called by a whole CTA.
__device__ bool family(Family& F, const ReorderParams& p, int b, int& full, bool& part, bool report) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int L = p.seq_len[int64_t(b) * p.W];
  full = L / kPageTokens;
  part = L % kPageTokens != 0;
  bool ok = L >= 0;
  uint32_t bad = !ok || full + (part ? 1 : 0) > p.np_max ? SPKV_DEVERR_PAGE_ID : 0u;
  if (tid < p.W) {
    const int x = p.parents[int64_t(b) * p.W + tid];
    F.parent[tid] = x;
    if (x < -1 || x >= p.W || p.seq_len[int64_t(b) * p.W + tid] != L) bad |= SPKV_DEVERR_BEAM;
  }
  if (__syncthreads_or(bad != 0)) {
    if (report) flag_error(p.err, bad);
    return false;
  }
  if (tid < 32) {
    // beams with children, children that keep their parent's page: beams lane and lane + 32
    unsigned long long used = 0, keeps = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int w = lane + 32 * e, x = w < p.W ? F.parent[w] : -1;
      bool keep = x >= 0 && (x == w || F.parent[x] != x);
      if (x >= 0 && x != w)
        for (int j = 0; j < w; ++j) keep = keep && F.parent[j] != x;
      const unsigned long long bit = x >= 0 ? 1ull << x : 0ull;
      used |= static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bit))) |
              static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bit >> 32))) << 32;
      keeps |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, keep)) << (32 * e);
    }
    const unsigned long long all = p.W == 64 ? ~0ull : (1ull << p.W) - 1, free = all & ~used;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int w = lane + 32 * e;
      if (w >= p.W) continue;
      int from = F.parent[w];
      if (!(keeps >> w & 1)) {   // the r-th beam without children
        int r = __popcll(~keeps & ((1ull << w) - 1));
        unsigned long long f = free;
        while (r--) f &= f - 1;
        from = __ffsll(static_cast<long long>(f)) - 1;
      }
      F.page_of[w] = from;
    }
  }
  __syncthreads();
  return true;
}

// CTAs 0 .. W Hk - 1 of a request copy beam w's part-filled page of head h; the others permute kStrip columns each.
__global__ void __launch_bounds__(256) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ Family F;
  __shared__ int tile[kMaxBeams][kStrip];
  __shared__ int last;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, b = blockIdx.y, x = blockIdx.x, copies = p.W * p.Hk;
  int full;
  bool part;
  const bool ok = family(F, p, b, full, part, x == 0);
  int32_t* const table = p.table + int64_t(b) * p.W * p.np_max;
  if (x >= copies) {   // complete pages
    const int c0 = (x - copies) * kStrip, n = min(kStrip, full - c0);
    if (!ok || n <= 0) return;
    for (int i = tid; i < p.W * kStrip; i += blockDim.x)
      if (i % kStrip < n) tile[i / kStrip][i % kStrip] = table[int64_t(i / kStrip) * p.np_max + c0 + i % kStrip];
    __syncthreads();
    for (int i = tid; i < p.W * kStrip; i += blockDim.x) {
      const int w = i / kStrip, from = F.parent[w];
      if (i % kStrip < n && from >= 0 && from != w) table[int64_t(w) * p.np_max + c0 + i % kStrip] = tile[from][i % kStrip];
    }
    return;
  }
  if (!ok || !part) return;
  const int w = x / p.Hk, h = x % p.Hk, parent = F.parent[w], mine = F.page_of[w];
  if (parent >= 0 && mine != parent) {
    const int src = table[int64_t(parent) * p.np_max + full], dst = table[int64_t(mine) * p.np_max + full];
    if (src < 0 || src >= p.n_phys || dst < 0 || dst >= p.n_phys) {
      if (h == 0 && tid == 0) flag_error(p.err, SPKV_DEVERR_PHYS);
    } else {
      const int cnt = p.page_cnt ? p.page_cnt[src] : kPageTokens;
      const int64_t bytes = p.row_bytes ? int64_t(max(0, min(kPageTokens, cnt))) * p.row_bytes : p.page_bytes;
      const int64_t from = (int64_t(h) * p.n_phys + src) * p.page_bytes, to = (int64_t(h) * p.n_phys + dst) * p.page_bytes;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!p.pool[k]) continue;
        for (int64_t i = tid * 16; i < bytes; i += 256 * 16)
          *reinterpret_cast<uint4*>(p.pool[k] + to + i) = *reinterpret_cast<const uint4*>(p.pool[k] + from + i);
      }
      if (p.ksum)
        for (int i = tid * 16; i < p.ksum_bytes; i += 256 * 16)
          *reinterpret_cast<uint4*>(p.ksum + (int64_t(h) * p.n_phys + dst) * p.ksum_bytes + i) =
              *reinterpret_cast<const uint4*>(p.ksum + (int64_t(h) * p.n_phys + src) * p.ksum_bytes + i);
      if (p.page_cnt && h == 0 && tid == 0) p.page_cnt[dst] = cnt;
    }
  }
  // the last CTA that has read the column of part-filled pages writes it
  __syncthreads();
  if (tid == 0) {
    int before;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived + b) : "memory");
    last = before == copies - 1;
    if (last) p.arrived[b] = 0;
  }
  __syncthreads();
  if (!last) return;
  if (tid < p.W) tile[0][tid] = table[int64_t(F.page_of[tid]) * p.np_max + full];
  __syncthreads();
  if (tid < p.W) table[int64_t(tid) * p.np_max + full] = tile[0][tid];
}

}  // namespace
}  // namespace spkv

using spkv::kGroupBytes;
using spkv::kMaxBeams;
using spkv::kMaxBest;

namespace {

bool on_device(int device) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

template <typename T>
cudaError_t launch_select_beams(const spkv::BeamParams& p, int B, cudaStream_t st) {
  return spkv::launch_pdl(spkv::beam_select_kernel<T>, dim3(static_cast<unsigned>(B) * p.ctas), dim3(spkv::kThreads), 0, st, p);
}

}  // namespace

extern "C" {

int beam_plan_create(spkv_cache_t c, int max_rows, int max_vocab, void* stream, spkv_beam_plan_t* out) {
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
  const bool ok = cudaMalloc(&p->line_max, n * 32 * sizeof(float)) == cudaSuccess && cudaMalloc(&p->group, n * sizeof(float2)) == cudaSuccess &&
                  cudaMalloc(&p->arrived, max_rows * sizeof(int32_t)) == cudaSuccess &&
                  cudaMemsetAsync(p->arrived, 0, max_rows * sizeof(int32_t), static_cast<cudaStream_t>(stream)) == cudaSuccess;
  if (!ok) {
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
  cudaFree(p->arrived);
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
  p.ctas = (W * p.groups + spkv::kWarps - 1) / spkv::kWarps;
  p.cum = cum;
  p.tokens = tokens;
  p.parents = parents;
  p.scores = scores;
  p.line_max = plan->line_max;
  p.group = plan->group;
  p.arrived = plan->arrived;
  p.err = c->dev_err;
  if (int64_t(B) * p.ctas >= (int64_t(1) << 31)) return SPKV_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == SPKV_F32    ? launch_select_beams<float>(p, B, st)
                        : type == SPKV_BF16 ? launch_select_beams<__nv_bfloat16>(p, B, st)
                                            : launch_select_beams<__half>(p, B, st);
  return e == cudaSuccess ? SPKV_OK : SPKV_ECUDA;
}

int beam_reorder(spkv_cache_t c, const int32_t* parents, int B, int W, int32_t* page_table, int np_max, const int32_t* seq_len,
                 void* stream) {
  if (!c || B < 0 || W <= 0) return SPKV_EINVAL;
  if (W > kMaxBeams || c->d.n_kv_heads > 65535) return SPKV_EUNSUPPORTED;
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
    p.page_bytes = c->pool4 ? 9216 : 16416;
  } else {
    p.pool[0] = static_cast<uint8_t*>(c->d.k_pool);
    p.pool[1] = static_cast<uint8_t*>(c->d.v_pool);
    p.page_bytes = 16384;
    p.row_bytes = 256;
  }
  p.ksum = static_cast<uint8_t*>(c->d.ksum);
  p.ksum_bytes = 4 * 128 * (c->d.ksum_bf16 ? 2 : 4);
  p.page_cnt = c->d.page_cnt;
  p.n_phys = c->d.n_phys_pages;
  p.arrived = c->beam_cnt;
  p.err = c->dev_err;
  const int64_t strips = (np_max + spkv::kStrip - 1) / spkv::kStrip;
  return spkv::launch_pdl(spkv::beam_reorder_kernel, dim3(static_cast<unsigned>(W * p.Hk + strips), B), dim3(256), 0,
                          static_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? SPKV_OK
             : SPKV_ECUDA;
}

}  // extern "C"
