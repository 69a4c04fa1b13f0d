// logprob.cu -- log probabilities of given tokens with entropy and top
// alternatives, and their gradient.
//
// Each row of logits x scores one token t at temperature T.  With m = max x,
// y_j = (x_j - m) / T, e_j = exp(y_j) and S = sum e_j:
//   log p_j = y_j - ln S,   H = -sum p_j log p_j = ln S - (sum e_j y_j) / S.
// These are the log-probabilities that the truncated importance sampling
// weights compare ("Method steps", step 4).
//
// Forward: one pass over the row with the running maximum, S and sum e y of a
// thread's own elements; threads, warps and the CTAs of a cluster meet in a
// fixed tree, so the result has the same bits on every run.  Few rows are
// spread over clusters of up to 8 CTAs (partials meet through distributed
// shared memory: one launch, no workspace).
//
// Top alternatives cost no work in that pass.  A thread's running maximum is
// the largest of its elements, so the k-th largest thread maximum tau is a
// lower bound of the k-th largest element, and every element that is at least
// tau lies with a thread whose maximum is at least tau: about k threads (ties
// aside) of the CTA's 256, whose elements are read a second time.  Those at or
// above tau are few and are sorted by (value, lower index first), 32 to a warp (8192 x
// 1313: 39 us; with every warp's offered one by one to a list, 68); a row of many
// equal ones goes through sorted lists of one key per lane.
//
// Backward: dx_j = (g ([j = t] - p_j) - g_H p_j (log p_j + H)) / T from the
// saved (m, ln S) and H; elementwise, so dx may be x.
//
// Both are HBM-bound (one read; one read and one write): 4096 x 151936 bf16
// takes 185 us forward (6.7 TB/s; 1/32 of the rows there have no token and are
// not read) and 354 us backward (7.0 TB/s).  16 rows with 20 alternatives
// take 9.5 us, on clusters of 8.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8rl {
namespace {

constexpr int kLpThreads = 256;
constexpr int kGradThreads = 128;  // the gradient's
constexpr int kLpUnroll = 4;  // 16-byte pieces a thread loads before it uses the first
constexpr int kMaxTop = 32;   // one key per lane
constexpr int kHits = 256;    // elements at or above the bound that are sorted, 32 at a time
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kTinyExp2 = -200.0f;  // 2^-200 is 0 in fp32: exponents below it change nothing, and stay finite

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// fmaxf that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Masked logits.  An exponent of -inf would meet e = 0 in a product, so
// elements below kFloor are read as kFloor: beside a maximum within
// +-kFloor / 2 and with log2(e) / T within kMinScale and kMaxScale their e is 0
// all the same (their exponents are below -600), and every exponent is finite.
// Rows outside these limits take exponents one by one, clamped.  (-1e30 rounded to
// bf16, so that both types clamp alike.)
constexpr float kFloor = -0x1.94p+99f, kMinScale = 1e-27f, kMaxScale = 1e6f;
constexpr uint32_t kFloorBf16x2 = 0xF14AF14Au;
// log2(e) / T, finite for the smallest T too (0 times it is 0)
__host__ __device__ __forceinline__ float exp2_scale(float temperature) { return fminf(kLog2e / temperature, FLT_MAX); }
// the largest |m| for which exponents with scale c need no care (negative: none); from
// the host: tested beside c in the loop it costs the fp32 kernel with alternatives a
// sixth of its resident CTAs (4096 x 32000, top 20: 113 us; 107 so)
__host__ __device__ __forceinline__ float floor_limit(float c) { return c >= kMinScale && c <= kMaxScale ? -0.5f * kFloor : -1.0f; }

// A row's 16-byte pieces, counted from the 16-byte boundary at or below its
// first element: piece p holds elements [p * N - off, (p + 1) * N - off).
template <typename In>
struct Row {
  static constexpr int N = 16 / sizeof(In);
  const In* x;
  int32_t off, vocab, pieces;
  __device__ __forceinline__ Row(const In* row, int32_t v) : x(row), vocab(v) {
    off = (int32_t)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(In));
    pieces = (v + off + N - 1) / N;
  }
  __device__ __forceinline__ bool whole(int32_t p) const { return p * N >= off && (p + 1) * N - off <= vocab; }
  __device__ __forceinline__ uint4 load(int32_t p) const;
};

constexpr uint32_t kNegInfBf16x2 = 0xFF80FF80u, kNegInfF32 = 0xFF800000u;

// elements outside the row read as -inf
template <>
__device__ __forceinline__ uint4 Row<uint16_t>::load(int32_t p) const {
  if (whole(p)) return __ldg(reinterpret_cast<const uint4*>(x + (p * N - off)));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int32_t j = p * N - off + 2 * i + e;
      w[i] |= (j >= 0 && j < vocab ? (uint32_t)x[j] : 0xFF80u) << (16 * e);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 Row<float>::load(int32_t p) const {
  if (whole(p)) return __ldg(reinterpret_cast<const uint4*>(x + (p * N - off)));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t j = p * N - off + i;
    w[i] = j >= 0 && j < vocab ? __float_as_uint(x[j]) : kNegInfF32;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename In>
__device__ __forceinline__ uint4 absent() {
  const uint32_t w = sizeof(In) == 2 ? kNegInfBf16x2 : kNegInfF32;
  return make_uint4(w, w, w, w);
}

template <typename In>
__device__ __forceinline__ void values(uint4 u, float (&v)[Row<In>::N]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(In) == 2) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

// the values of a piece as fp32 pairs, none below kFloor
template <typename In>
__device__ __forceinline__ void floored_pairs(uint4 u, uint64_t (&v)[Row<In>::N / 2]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if (sizeof(In) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t f = max_nan_bf16x2(w[i], kFloorBf16x2);
      v[i % (Row<In>::N / 2)] = pair_of(bf16_lo(f), bf16_hi(f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = pair_of(max_nan(__uint_as_float(w[2 * i]), kFloor), max_nan(__uint_as_float(w[2 * i + 1]), kFloor));
  }
}

// the largest value of some pieces (NaN left out)
template <typename In, int U>
__device__ __forceinline__ float largest(const uint4 (&u)[U]) {
  if (sizeof(In) == 2) {
    uint32_t m = max_bf16x2(max_bf16x2(u[0].x, u[0].y), max_bf16x2(u[0].z, u[0].w));
#pragma unroll
    for (int i = 1; i < U; ++i) {
      m = max_bf16x2(m, max_bf16x2(u[i].x, u[i].y));
      m = max_bf16x2(m, max_bf16x2(u[i].z, u[i].w));
    }
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < U; ++i)
    m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(u[i].x), __uint_as_float(u[i].y)),
                       fmaxf(__uint_as_float(u[i].z), __uint_as_float(u[i].w))));
  return m;
}

// Running statistics in base 2: with t_j = (x_j - m) log2(e) / T,
// s = sum 2^t_j and w = sum 2^t_j t_j.  m = -inf: nothing seen.
struct Stat {
  float m, s, w;
};

// the same sums relative to a new maximum: t_j + d, d = (m - to) log2(e) / T
__device__ __forceinline__ void move_to(Stat& a, float to, float c) {
  if (a.m == -INFINITY) {
    a.m = to;  // s and w are 0, or NaN from a NaN element
    return;
  }
  const float d = max_nan((a.m - to) * c, kTinyExp2), f = ex2(d);
  a.w = f * fmaf(d, a.s, a.w);
  a.s *= f;
  a.m = to;
}

__device__ __forceinline__ Stat merge(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (a.m != m) move_to(a, m, c);
  if (b.m != m) move_to(b, m, c);
  a.s += b.s;
  a.w += b.w;
  return a;
}

// the sums of groups of L neighbouring lanes, in a tree that both lanes of a pair
// add up alike: the largest first, so that each lane moves once
template <int L>
__device__ __forceinline__ void merge_lanes(Stat& a, float c) {
  float m = a.m;
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (a.m != m) move_to(a, m, c);
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, d);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, d);
  }
}

// Keys that order like (value, lower index first): the value's bits as an
// ordered integer (-0 as 0, NaN below everything) above the complemented index.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return o == 0u ? __uint_as_float(0x7FC00000u) : __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, int32_t j) {
  return (uint64_t)ordered(v) << 32 | (uint32_t)~j;
}

// The warp's sorted list, lane i its i-th largest key (0: none), takes in
// every lane's `key` (0: none to offer).  Lanes >= top never count.
__device__ __forceinline__ void offer(uint64_t& list, uint64_t key, int top) {
  const int lane = threadIdx.x & 31;
  for (;;) {
    const uint64_t worst = __shfl_sync(0xffffffffu, list, top - 1);
    const uint32_t want = __ballot_sync(0xffffffffu, key > worst);
    if (!want) return;
    const int from = __ffs(want) - 1;
    const uint64_t k = __shfl_sync(0xffffffffu, key, from);
    const int at = __popc(__ballot_sync(0xffffffffu, list > k));
    const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
    if (lane == at) list = k;
    if (lane > at) list = up;
    if (lane == from) key = 0;
  }
}

// The 32 largest of two sorted lists, sorted: the larger of list[i] and
// other[31 - i] are those 32, and rise then fall, so five exchange steps order
// them (Batcher's bitonic merge).
__device__ __forceinline__ uint64_t merge_lists(uint64_t list, uint64_t other) {
  const int lane = threadIdx.x & 31;
  const uint64_t rev = __shfl_sync(0xffffffffu, other, 31 - lane);
  list = list > rev ? list : rev;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, list, d);
    list = ((lane & d) == 0) == (list > o) ? list : o;
  }
  return list;
}

// the warp's keys, largest first (Batcher's bitonic sort)
__device__ __forceinline__ uint64_t sort_keys(uint64_t key) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1) {
#pragma unroll
    for (int d = n >> 1; d > 0; d >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, key, d);
      const bool larger = ((lane & d) == 0) == ((lane & n) == 0);
      key = larger == (key > o) ? key : o;
    }
  }
  return key;
}

// Merge of the warps' lists: warp 0 returns the CTA's.  Every warp takes part.
template <int W>
__device__ __forceinline__ uint64_t merge_warps(uint64_t list, uint64_t (&lists)[W][kMaxTop]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int n = W / 2; n > 0; n >>= 1) {
    if (warp >= n && warp < 2 * n) lists[warp][lane] = list;
    __syncthreads();
    if (warp < n) list = merge_lists(list, lists[warp + n][lane]);
  }
  return list;
}

struct LpArgs {
  const void* x;
  const int32_t* tokens;
  float* lp;
  float* entropy;
  float2* stats;
  int32_t* top_ids;
  float* top_lp;
  int64_t ld;
  int32_t vocab, top;
  float temperature, limit;
  int64_t rows;
  uint32_t* err;  // debug builds' store checks
};

// grid (cluster, rows), clusters of gridDim.x CTAs: a CTA takes the pieces
// [rank, rank + 1) * ceil(pieces / cluster) of its row
template <typename In, bool TOP, int T>
__global__ void __launch_bounds__(T) logprob_kernel(const LpArgs a) {
  constexpr int N = Row<In>::N, U = kLpUnroll, W = T / 32;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int64_t r = blockIdx.y;
  const int rank = blockIdx.x, ranks = gridDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t t = a.tokens[r];
  if (t < 0 || t >= a.vocab) {  // no token: the whole cluster leaves
    if (rank == 0 && dcheck(r < a.rows, a.err)) {
      if (tid == 0) {
        a.lp[r] = 0.0f;
        a.entropy[r] = 0.0f;
        a.stats[r] = make_float2(0.0f, 0.0f);
      }
      if (TOP && tid < a.top) {
        a.top_ids[r * a.top + tid] = -1;
        a.top_lp[r * a.top + tid] = 0.0f;
      }
    }
    return;
  }
  const In* xr = static_cast<const In*>(a.x) + r * a.ld;
  const Row<In> row(xr, a.vocab);
  const int32_t share = (row.pieces + ranks - 1) / ranks;
  const int32_t p0 = rank * share, p1 = min(row.pieces, p0 + share);
  const float c = exp2_scale(a.temperature);
  float xt = 0.0f;  // needed at the end, requested now
  if (tid == 0 && rank == 0) {
    if (sizeof(In) == 2) xt = bf16_lo((uint32_t) reinterpret_cast<const uint16_t*>(xr)[t]);
    else xt = reinterpret_cast<const float*>(xr)[t];
  }

  Stat st{-INFINITY, 0.0f, 0.0f};
  uint64_t s2 = pair_of(0.0f, 0.0f), w2 = s2;  // s and w in two halves
  const uint64_t c2 = pair_of(c, c);
  auto fold = [&] {
    float lo, hi;
    ptx::f32x2_unpack(s2, lo, hi);
    st.s += lo + hi;
    ptx::f32x2_unpack(w2, lo, hi);
    st.w += lo + hi;
    s2 = w2 = pair_of(0.0f, 0.0f);
  };
  // (loading the next round ahead of this one's arithmetic costs the
  // registers of a third of the resident CTAs: 213 us for 195 at 4096 x 151936)
  for (int32_t p = p0 + tid; p < p1; p += U * T) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = p + i * T < p1 ? row.load(p + i * T) : absent<In>();
    const float big = largest<In>(u);
    if (big > st.m) {
      fold();
      move_to(st, big, c);
    }
    if (fabsf(st.m) <= a.limit) {
      const uint64_t nm2 = pair_of(-st.m, -st.m);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint64_t v[N / 2];
        floored_pairs<In>(u[i], v);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const uint64_t y = pair_mul(add2(v[e], nm2), c2);
          float y0, y1;
          ptx::f32x2_unpack(y, y0, y1);
          const uint64_t p2 = pair_of(ex2(y0), ex2(y1));
          s2 = add2(s2, p2);
          w2 = pair_fma(p2, y, w2);
        }
      }
    } else {
      const float m = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[N];
        values<In>(u[i], v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float y = max_nan((v[e] - m) * c, kTinyExp2), p2 = ex2(y);
          st.s += p2;
          st.w = fmaf(p2, y, st.w);
        }
      }
    }
  }
  fold();
  const float mine = st.m;  // the largest of this thread's elements

  __shared__ Stat warp_stat[W];
  __shared__ Stat cta_stat;
  __shared__ uint64_t lists[W][kMaxTop];
  __shared__ uint64_t cta_list[kMaxTop];
  __shared__ int16_t cand[T];
  __shared__ uint64_t hits[kHits];
  __shared__ int cands, n_hits;
  merge_lanes<32>(st, c);
  if (lane == 0) warp_stat[warp] = st;
  if (tid == 0) cands = n_hits = 0;
  __syncthreads();
  if (warp == 0) {
    st = warp_stat[lane % W];
    merge_lanes<W>(st, c);
    if (lane == 0) cta_stat = st;
  }

  uint64_t top_list = 0;
  if (TOP) {
    // tau: the top-th largest thread maximum (0 while fewer threads hold any)
    constexpr int kShift = 16;  // the upper half: all of a bf16 value, a lower bound of an fp32 one
    const uint32_t own = p0 + tid < p1 ? max(ordered(mine) >> kShift, 1u) : 0u;
    uint32_t lo = 0u;
    for (int b = p1 - p0 < a.top ? -1 : 31 - kShift; b >= 0; --b) {
      const uint32_t mid = lo | 1u << b;
      if (__syncthreads_count(own >= mid) >= a.top) lo = mid;
    }
    if (own >= lo && own > 0u) cand[atomicAdd(&cands, 1)] = (int16_t)tid;
    __syncthreads();
    // the candidates' pieces, spread over all threads
    const int32_t each = (p1 - p0 + T - 1) / T;
    const int32_t total = cands * each;
    auto piece_of = [&](int32_t f) { return f < total ? p0 + cand[f / each] + (f % each) * T : p1; };
    auto key_at = [&](int32_t p, int e, float v) -> uint64_t {
      const int32_t j = p * N - row.off + e;
      return p < p1 && j >= 0 && j < a.vocab && max(ordered(v) >> kShift, 1u) >= lo ? key_of(v, j) : 0;
    };
    for (int32_t f = tid; f < total; f += T) {
      const int32_t p = piece_of(f);
      const uint4 u[1] = {p < p1 ? row.load(p) : absent<In>()};
      if (max(ordered(largest<In>(u)) >> kShift, 1u) < lo) continue;
      float v[N];
      values<In>(u[0], v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint64_t key = key_at(p, e, v[e]);
        if (key == 0) continue;
        const int at = atomicAdd(&n_hits, 1);
        if (at < kHits) hits[at] = key;
      }
    }
    __syncthreads();
    if (n_hits <= kHits) {  // all but rows with many equal logits
      for (int h0 = warp * 32; h0 < n_hits; h0 += T) {
        const uint64_t more = sort_keys(h0 + lane < n_hits ? hits[h0 + lane] : 0);
        top_list = h0 < T ? more : merge_lists(top_list, more);
      }
      if (n_hits > 32) top_list = merge_warps(top_list, lists);
    } else {
      uint64_t list = 0;
      for (int32_t f0 = warp * 32; f0 < total; f0 += T) {
        const int32_t p = piece_of(f0 + lane);
        const uint4 u = p < p1 ? row.load(p) : absent<In>();
        float v[N];
        values<In>(u, v);
#pragma unroll
        for (int e = 0; e < N; ++e) offer(list, key_at(p, e, v[e]), a.top);
      }
      top_list = merge_warps(list, lists);
    }
    if (warp == 0) cta_list[lane] = top_list;
  }

  if (T == kLpThreads && ranks > 1) {
    ptx::cluster_sync();
    if (TOP && rank == 0) {  // warp i takes rank i's list
      uint64_t list = top_list;
      if (warp > 0) {
        const uint32_t l = ptx::mapa_shared(ptx::smem_u32(&cta_list[lane]), warp < ranks ? warp : 0);
        list = warp < ranks ? (uint64_t)ptx::ld_dsmem_u32(l + 4) << 32 | ptx::ld_dsmem_u32(l) : 0;
      }
      top_list = merge_warps(list, lists);
    }
  }
  if (rank == 0 && warp == 0) {
    __syncwarp();
    Stat all = cta_stat;
    if (T == kLpThreads && ranks > 1) {  // lane i reads rank i's sums; they are merged in rank order
      const uint32_t base = ptx::mapa_shared(ptx::smem_u32(&cta_stat), lane < ranks ? lane : 0);
      const Stat o{__uint_as_float(ptx::ld_dsmem_u32(base)), __uint_as_float(ptx::ld_dsmem_u32(base + 4)),
                   __uint_as_float(ptx::ld_dsmem_u32(base + 8))};
      for (int i = 1; i < ranks; ++i)
        all = merge(all, Stat{__shfl_sync(0xffffffffu, o.m, i), __shfl_sync(0xffffffffu, o.s, i), __shfl_sync(0xffffffffu, o.w, i)}, c);
    }
    const uint64_t list = top_list;
    // a row of -inf alone: every log-probability -inf, entropy 0
    const bool none = all.m == -INFINITY && all.s == 0.0f;
    const float ln_s = logf(all.s);
    auto log_prob = [&](float v) { return none ? -INFINITY : (v - all.m) / a.temperature - ln_s; };
    const bool in = dcheck(r < a.rows, a.err);
    if (lane == 0 && in) {
      a.lp[r] = log_prob(xt);
      a.entropy[r] = none ? 0.0f : ln_s - kLn2 * (all.w / all.s);
      a.stats[r] = make_float2(all.m, ln_s);
    }
    if (TOP && lane < a.top && in) {
      a.top_ids[r * a.top + lane] = (int32_t) ~(uint32_t)list;
      a.top_lp[r * a.top + lane] = log_prob(from_ordered((uint32_t)(list >> 32)));
    }
  }
  __syncwarp();
  if (T == kLpThreads && ranks > 1) ptx::cluster_sync();  // rank 0 has read the others' shared memory
}

// ------------------------------------------------------------------ backward

struct LpGradArgs {
  const void* x;
  void* dx;
  const int32_t* tokens;
  const float2* stats;
  const float* entropy;
  const float* g_lp;
  const float* g_ent;  // or null
  int64_t ldx, ldd;
  int32_t vocab;
  float temperature, limit;
  uint32_t* err;  // debug builds' store checks
};

// dx_j = p (a + b log2 p) with a = -(g + g_H H) / T and b = -g_H ln 2 / T;
// the token's own element has g / T on top
struct GradRow {
  float m, c, l2, a, b, top;
  int32_t t;
  bool zero;
};

// dx of element j with value v
__device__ __forceinline__ float grad_of(const GradRow& q, float v, int32_t j) {
  const float y = max_nan(fmaf(v - q.m, q.c, -q.l2), kTinyExp2);  // log2 p
  const float p = ex2(y), f = fmaf(q.b, y, q.a);
  const float d = p == 0.0f && fabsf(f) == INFINITY ? 0.0f : p * f;
  return j == q.t ? d + q.top : d;
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename In>
__device__ __forceinline__ void store1(In* p, float v);
template <>
__device__ __forceinline__ void store1<uint16_t>(uint16_t* p, float v) {
  *p = (uint16_t)bf16x2_rn(v, 0.0f);
}
template <>
__device__ __forceinline__ void store1<float>(float* p, float v) {
  *p = v;
}

// grid (slices, rows); dx may be x, so neither is read through the read-only path
template <typename In>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const LpGradArgs a) {
  constexpr int N = Row<In>::N, U = kLpUnroll;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int64_t r = blockIdx.y;
  const In* x = static_cast<const In*>(a.x) + r * a.ldx;
  In* dx = static_cast<In*>(a.dx) + r * a.ldd;
  GradRow q;
  q.t = a.tokens[r];
  const float2 st = a.stats[r];
  // no token, or a row of -inf alone (a NaN beside them left its mark in st.y)
  q.zero = q.t < 0 || q.t >= a.vocab || (st.x == -INFINITY && st.y == -INFINITY);
  q.m = st.x;
  q.c = exp2_scale(a.temperature);
  q.l2 = st.y * kLog2e;
  const float g = a.g_lp[r], gh = a.g_ent ? a.g_ent[r] : 0.0f, inv_t = 1.0f / a.temperature;
  auto over_t = [&](float v) { return inv_t <= FLT_MAX ? v * inv_t : v / a.temperature; };
  q.a = over_t(-(a.g_ent ? fmaf(gh, a.entropy[r], g) : g));
  q.b = over_t(-gh * kLn2);
  q.top = over_t(g);
  const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
  const int32_t stride = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
  if (!same) {  // rows that start at different places of a 16-byte piece: element by element
    for (int32_t j = first; j < a.vocab; j += stride) {
      float v;
      if (sizeof(In) == 2) v = bf16_lo((uint32_t) reinterpret_cast<const uint16_t*>(x)[j]);
      else v = reinterpret_cast<const float*>(x)[j];
      if (dcheck(j >= 0 && j < a.vocab, a.err)) store1<In>(dx + j, q.zero ? 0.0f : grad_of(q, v, j));
    }
    return;
  }
  const Row<In> row(x, a.vocab);
  // elements that are read as kFloor: p = 0 beside exponents y of up to `reach`, and
  // a + b y has to be finite for their product to be 0
  const float reach = fmaf(-1.5f * kFloor, q.c, fabsf(q.l2));
  const bool plain = !q.zero && fabsf(q.m) <= a.limit && fmaf(fabsf(q.b), reach, fabsf(q.a)) < 0.5f * FLT_MAX;
  const uint64_t nm2 = pair_of(-q.m, -q.m), c2 = pair_of(q.c, q.c), nl2 = pair_of(-q.l2, -q.l2), a2 = pair_of(q.a, q.a),
                 b2 = pair_of(q.b, q.b);
  for (int32_t p = first; p < row.pieces; p += U * stride) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int32_t pi = p + i * stride;
      if (pi < row.pieces && row.whole(pi) && !q.zero) u[i] = *reinterpret_cast<const uint4*>(x + (pi * N - row.off));
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int32_t pi = p + i * stride, j0 = pi * N - row.off;
      if (pi >= row.pieces) break;
      if (row.whole(pi)) {
        float d[N];
        if (plain) {
          uint64_t v[N / 2];
          floored_pairs<In>(u[i], v);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            const uint64_t y = pair_fma(add2(v[e], nm2), c2, nl2);
            float y0, y1;
            ptx::f32x2_unpack(y, y0, y1);
            ptx::f32x2_unpack(pair_mul(pair_of(ex2(y0), ex2(y1)), pair_fma(b2, y, a2)), d[2 * e], d[2 * e + 1]);
          }
          if ((uint32_t)(q.t - j0) < (uint32_t)N) {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (j0 + e == q.t) d[e] += q.top;
          }
        } else {
          float v[N];
          values<In>(u[i], v);
#pragma unroll
          for (int e = 0; e < N; ++e) d[e] = q.zero ? 0.0f : grad_of(q, v[e], j0 + e);
        }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = sizeof(In) == 2 ? bf16x2_rn(d[(2 * e) % N], d[(2 * e + 1) % N]) : __float_as_uint(d[e]);
        if (dcheck(j0 >= 0 && j0 + N <= a.vocab, a.err))
          __stcs(reinterpret_cast<uint4*>(dx + j0), make_uint4(w[0], w[1], w[2], w[3]));
      } else {
        for (int e = 0; e < N; ++e) {
          const int32_t j = j0 + e;
          if (j < 0 || j >= a.vocab) continue;
          float v;
          if (sizeof(In) == 2) v = bf16_lo((uint32_t) reinterpret_cast<const uint16_t*>(x)[j]);
          else v = reinterpret_cast<const float*>(x)[j];
          if (dcheck(j >= 0 && j < a.vocab, a.err)) store1<In>(dx + j, q.zero ? 0.0f : grad_of(q, v, j));
        }
      }
    }
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  return n;
}

// the word that debug builds' store checks report to (release builds have none)
bool check_word(uint32_t** err) {
#ifdef FP8RL_DEBUG
  *err = device_error_word();
  return *err != nullptr;
#else
  *err = nullptr;
  return true;
#endif
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxRows = 65535;             // grid y
constexpr int64_t kMaxVocab = (int64_t)1 << 30;  // 32-bit element and piece numbers

template <typename In, bool TOP, int T>
cudaError_t launch_logprob(const LpArgs& a, int64_t rows, cudaStream_t stream) {
  // Fewer rows than three and a half CTAs per SM are split over a cluster, down to one
  // load round (four pieces a thread) per CTA (338 x 151936: 27 us on clusters of two, 39
  // on one CTA; 200 x 50257: 8.8 on four, 10.1 on two, 11.6 on eight).
  const int64_t want = 7 * (int64_t)sm_count() / 2;
  const int64_t round = (int64_t)kLpThreads * kLpUnroll * Row<In>::N;
  int cluster = 1;
  while (T == kLpThreads && cluster < 8 && rows * cluster < want && (int64_t)a.vocab > cluster * round) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster, (unsigned)rows);
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<In, TOP, T>, a);
}

// Short rows are bound by a row's chain of waits, so they run in smaller CTAs, more of
// them at a time: 8192 x 1313 bf16 18 us with 64 threads, 34 with 256; 8192 x 14 506
// 55 with 128, 60 with 256 (at 50 257 256 are faster: 92 and 101).  Few rows
// gain from 256 threads as soon as they have work for them.
template <typename In, bool TOP>
cudaError_t launch_rows(const LpArgs& a, int64_t rows, cudaStream_t stream) {
  const int64_t pieces = ((int64_t)a.vocab + Row<In>::N - 1) / Row<In>::N;
  if (pieces <= 256) return launch_logprob<In, TOP, 64>(a, rows, stream);
  if (pieces <= 2048 && rows >= 2 * (int64_t)sm_count()) return launch_logprob<In, TOP, 128>(a, rows, stream);
  return launch_logprob<In, TOP, kLpThreads>(a, rows, stream);
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

extern "C" FP8RL_API fp8rl_status fp8rl_logprob(const void* d_logits, int32_t logits_fp32, int64_t rows, int64_t vocab,
                                                int64_t ld, float temperature, const int32_t* d_tokens, float* d_lp,
                                                float* d_entropy, float* d_stats, int64_t topk, int32_t* d_top_ids,
                                                float* d_top_lp, void* stream) {
  if (rows < 0 || vocab < 1 || ld < vocab || topk < 0 || !(temperature > 0.0f) || !(temperature <= FLT_MAX) ||
      (logits_fp32 != 0 && logits_fp32 != 1))
    return FP8RL_ERR_INVALID_ARG;
  if (rows == 0) return FP8RL_OK;
  if (!d_logits || !d_tokens || !d_lp || !d_entropy || !d_stats) return FP8RL_ERR_INVALID_ARG;
  if (topk > 0 && (!d_top_ids || !d_top_lp)) return FP8RL_ERR_INVALID_ARG;
  if (topk > kMaxTop || topk > vocab || vocab > kMaxVocab) return FP8RL_ERR_SHAPE;
  if (!aligned(d_logits, logits_fp32 ? 4 : 2) || !aligned(d_tokens, 4) || !aligned(d_lp, 4) || !aligned(d_entropy, 4) ||
      !aligned(d_stats, 8) || !aligned(d_top_ids, 4) || !aligned(d_top_lp, 4))
    return FP8RL_ERR_ALIGNMENT;
  uint32_t* err = nullptr;
  if (!check_word(&err)) return FP8RL_ERR_CUDA;
  const size_t size = logits_fp32 ? 4 : 2;
  for (int64_t r0 = 0; r0 < rows; r0 += kMaxRows) {
    const int64_t n = std::min(kMaxRows, rows - r0);
    LpArgs a{};
    a.x = static_cast<const char*>(d_logits) + r0 * ld * (int64_t)size;
    a.tokens = d_tokens + r0;
    a.lp = d_lp + r0;
    a.entropy = d_entropy + r0;
    a.stats = reinterpret_cast<float2*>(d_stats) + r0;
    a.top_ids = topk ? d_top_ids + r0 * topk : nullptr;
    a.top_lp = topk ? d_top_lp + r0 * topk : nullptr;
    a.ld = ld;
    a.vocab = (int32_t)vocab;
    a.top = (int32_t)topk;
    a.temperature = temperature;
    a.limit = floor_limit(exp2_scale(temperature));
    a.rows = n;
    a.err = err;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = logits_fp32 ? (topk ? launch_rows<float, true>(a, n, cs) : launch_rows<float, false>(a, n, cs))
                                      : (topk ? launch_rows<uint16_t, true>(a, n, cs) : launch_rows<uint16_t, false>(a, n, cs));
    if (e != cudaSuccess) {
      cudaGetLastError();
      return FP8RL_ERR_CUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}

extern "C" FP8RL_API fp8rl_status fp8rl_logprob_backward(const void* d_logits, int32_t logits_fp32, int64_t rows,
                                                         int64_t vocab, int64_t ld, float temperature,
                                                         const int32_t* d_tokens, const float* d_stats,
                                                         const float* d_entropy, const float* d_grad_lp,
                                                         const float* d_grad_entropy, void* d_dlogits, int64_t ldd,
                                                         void* stream) {
  if (rows < 0 || vocab < 1 || ld < vocab || ldd < vocab || !(temperature > 0.0f) || !(temperature <= FLT_MAX) ||
      (logits_fp32 != 0 && logits_fp32 != 1))
    return FP8RL_ERR_INVALID_ARG;
  if (rows == 0) return FP8RL_OK;
  if (!d_logits || !d_tokens || !d_stats || !d_grad_lp || !d_dlogits || (d_grad_entropy && !d_entropy))
    return FP8RL_ERR_INVALID_ARG;
  if (d_dlogits == d_logits && ldd != ld) return FP8RL_ERR_INVALID_ARG;
  if (vocab > kMaxVocab) return FP8RL_ERR_SHAPE;
  const uintptr_t size = logits_fp32 ? 4 : 2;
  if (!aligned(d_logits, size) || !aligned(d_dlogits, size) || !aligned(d_tokens, 4) || !aligned(d_stats, 8) ||
      !aligned(d_entropy, 4) || !aligned(d_grad_lp, 4) || !aligned(d_grad_entropy, 4))
    return FP8RL_ERR_ALIGNMENT;
  uint32_t* err = nullptr;
  if (!check_word(&err)) return FP8RL_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  for (int64_t r0 = 0; r0 < rows; r0 += kMaxRows) {
    const int64_t n = std::min(kMaxRows, rows - r0);
    LpGradArgs a{};
    a.x = static_cast<const char*>(d_logits) + r0 * ld * (int64_t)size;
    a.dx = static_cast<char*>(d_dlogits) + r0 * ldd * (int64_t)size;
    a.tokens = d_tokens + r0;
    a.stats = reinterpret_cast<const float2*>(d_stats) + r0;
    a.entropy = d_entropy ? d_entropy + r0 : nullptr;
    a.g_lp = d_grad_lp + r0;
    a.g_ent = d_grad_entropy ? d_grad_entropy + r0 : nullptr;
    a.ldx = ld;
    a.ldd = ldd;
    a.vocab = (int32_t)vocab;
    a.temperature = temperature;
    a.limit = floor_limit(exp2_scale(temperature));
    a.err = err;
    // Small CTAs, so that many rows are under way (8192 x 1000 fp32: 9.3 us with 64
    // threads, 11 with 128, 16 with 256; 8192 x 4000 43, 41 and 43).  A load round is
    // four pieces a thread.  CTAs of up to five rounds once that leaves many times
    // the resident CTAs (4096 x 151936 with 256 threads: 356 us, with one round
    // each 403, ten 363); one round each for small work.
    const int64_t pieces = (vocab * (int64_t)size + 15) / 16;
    const int threads = pieces <= 640 ? 64 : kGradThreads;
    const int64_t round = (int64_t)threads * kLpUnroll * (16 / (int64_t)size);
    const int64_t rounds = (vocab + round - 1) / round;
    const int64_t each = std::max<int64_t>(1, std::min<int64_t>(5, rounds * n / ((int64_t)sm_count() * 24)));
    const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(65535, (rounds + each - 1) / each)), (unsigned)n);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = cs;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    const cudaError_t e = logits_fp32 ? cudaLaunchKernelEx(&cfg, logprob_grad_kernel<float>, a)
                                      : cudaLaunchKernelEx(&cfg, logprob_grad_kernel<uint16_t>, a);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return FP8RL_ERR_CUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}
