// sample.cu -- tokens drawn from rows of logits with temperature, top-k, top-p
// and min-p, from given random numbers.
//
// A row x at temperature T has weights w_j = exp((x_j - m) / T), m = max x, and
// sum S.  Ordered by (x, lower index first), the kept tokens are a prefix: the first
// k; of these the shortest prefix with mass >= p times theirs; of these the ones with
// w_j >= min_p.  With W the kept mass, the token is the lowest kept j with
//   sum of kept w_i, i <= j,  >  u W.
//
// The answer is a whole number that a comparison of sums decides.  A sum that is off by
// e S gives another token for a share of about 2 e u's for each token heavier than
// that: with fp32 sums (e = 10^-7) a few per cent of the draws from a flat row of 150 000.
// Two kernels see to it.
//
// sample_kernel takes each row in one pass, as the log probabilities do: exponentials
// in fp32 against the running maximum, each thread's sum with a bound of its error.
// Where nothing is cut off, the token is found by descending from the sums of warps
// (each has a contiguous share of the row) to parts of one and to pieces, and
// stands if u W is further from both its borders than the sums can be wrong (what the shares before, behind and
// at it may be off by, each with its factor: 40 of 1024 rows stay open, with twice the whole
// sum's bound 128).  Where something
// is cut off, the thread maxima give a bound below which nothing is kept (the k-th
// largest; or so many of the largest that their masses alone reach p S), the few
// elements above it are collected, sorted, weighed exactly, cut and drawn from.  A row
// that cannot be decided so (a draw on a border, more elements than the list
// holds, temperatures or maxima out of range) is marked for
//
// sample_exact_kernel (sample_exact.cu), which follows at once and passes by all other rows.
//
// The order of all sums is fixed.
//
// Bound by HBM for many rows, by the chain of waits for few.  The exponentials' pass asks
// 10 instructions an element: 1024 x 151936 bf16 takes 70 us (4.4 TB/s), and the
// exact kernel 28 for the 40 or so draws of so many that fall among the lightest tokens; with
// top-50 and top-p 104 us.  Pieces come through a ring in shared memory, two
// rounds ahead of each lane (when both kernels took 127 us without, 120 so; 98 now).  16 rows: 11 us
// where nothing is cut off, 16 with top-50, 14 with min-p.
#include <algorithm>

#include "sample.cuh"

namespace fp8rl {
namespace sampling {
namespace {

// ------------------------------------------------------------------ one pass

constexpr int kStages = 2;    // of a lane's ring
constexpr int kCap = 1024;    // elements that a row's cut is made among
constexpr int kMassBins = 128;  // of the thread maxima, a quarter of a power of two each
constexpr float kStep = 0x1p-24f;  // an fp32 operation's largest relative error
constexpr float kSlope = 2.6f, kMoved = 2.4f;  // of the error's bound: kSlope kMoved > 6

// a warp's share of a row: sums against its maximum m
struct WarpStat {
  float m;
  Pair s;            // sum of w
  float wt;          // sum of w t (t <= 0: exponents in base 2), and what stands for moves of the maximum
  uint32_t masked;   // elements of -inf
  uint32_t pad[3];
};
static_assert(sizeof(WarpStat) == 32, "read as 8 words");

template <int T>
struct PassShared {
  WarpStat warp[T / 32];
  float bound;             // of this CTA's share: at least its part of the first k lies at or above
  // of the whole row, after the pass
  Pair total, left;
  float m, err, margin, tau;
  uint32_t finite;
  int owner, owner_warp;
  Pair part[T / 32];
};
// the lists of a cut, in the memory of the pass's ring
struct Lists {
  uint64_t list[kCap];  // this CTA's finds
  uint64_t key[kCap];   // rank 0: all of them, sorted
  Pair w[kCap];
};
template <int T>
struct CutShared {
  float2 table[256];
  float most[T];  // thread maxima
  uint32_t bins[kMassBins];
  Pair part[T / 32];
  double reach;
  int16_t cand[T];
  int hits, cands, last_bin, below[2], n_border, token;
};

// keys sorted, the largest first; n a power of two, the whole block
template <int T>
__device__ void sort_down(uint64_t* key, int n) {
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += T) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const uint64_t x = key[a], y = key[b];
        if ((x < y) == ((a & k) == 0)) {
          key[a] = y;
          key[b] = x;
        }
      }
    }
  }
  __syncthreads();
}

// The running sums of w[0 .. n): a thread takes kCap / T entries in a row and shows each to
// f(i, sum before, sum with); returns the whole sum
template <int T, typename F>
__device__ Pair sums_of(const Pair* w, int n, Pair* part, F f) {
  constexpr int E = kCap / T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = threadIdx.x * E;
  Pair own;
  for (int i = i0; i < min(n, i0 + E); ++i) own = own + w[i];
  const Pair incl = scan_lanes(own);
  Pair sum = shuffle_up(incl, 1);
  if (lane == 0) sum = Pair{};
  __syncthreads();
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  Pair all;
  for (int i = 0; i < T / 32; ++i) {
    if (i == warp) sum = all + sum;
    all = all + part[i];
  }
  for (int i = i0; i < min(n, i0 + E); ++i) {
    const Pair with = sum + w[i];
    f(i, sum, with);
    sum = with;
  }
  return all;
}

// the sum of the block's values up to and with this thread's, and of all
template <int T>
__device__ __forceinline__ Pair block_sums(Pair v, Pair* part, Pair& all) {
  constexpr int W = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Pair incl = scan_lanes(v);
  __syncthreads();  // the sums before have been read
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  Pair w = part[lane % W];
#pragma unroll
  for (int d = 1; d < W; d <<= 1) {
    const Pair o = shuffle_up(w, d);
    if (lane >= d) w = o + w;
  }
  all = shuffle(w, W - 1);
  const Pair ahead = shuffle(w, (warp + 31) & 31);
  return warp > 0 ? ahead + incl : incl;
}

// The draw from a list of at most one element a thread (rank 0's keys, in any order): `n_k` of them are the
// first k, `exact`: the list's masses are what top_p goes by (else the sum, known to err).
template <int T>
__device__ void draw_from_few(const SampleArgs& a, int64_t r, CutShared<T>& cs, Lists& lists, const Draw& draw, const Scale& s, int n, int n_k,
                              bool by_p, bool exact, Pair total, float err, float border, int finite) {
  const int tid = threadIdx.x;
  if (tid == 0 && (n & 1)) lists.key[n] = 0;
  __syncthreads();
  // by value: each counts the ones ahead of it
  const uint64_t mine = tid < n ? lists.key[tid] : 0;
  int place = 0;
  for (int i = 0; i < n; i += 2) {
    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&lists.key[i]);
    place += (two.x > mine) + (two.y > mine);
  }
  if (tid < n) lists.list[place] = mine;
  __syncthreads();
  const uint64_t key = tid < n ? lists.list[tid] : 0;
  const float x = from_ordered((uint32_t)(key >> 32));
  Pair w;
  if (tid < n) {
    w = weight(s, cs.table, x);
  }
  Pair all;
  const Pair upto = block_sums<T>(tid < n_k ? w : Pair{}, cs.part, all);
  int n_kept = n_k;
  if (by_p) {
    // how many sums lie below top_p's share (of the sum known to err: below its least and its largest)
    const Pair low = exact ? all : total + Pair{-err, 0.0f}, high = exact ? all : total + Pair{err, 0.0f}, p{draw.top_p, 0.0f};
    const int n_low = __syncthreads_count(tid < n_k && upto < p * low);
    const int n_high = exact ? n_low : __syncthreads_count(tid < n_k && upto < p * high);
    if (n_low != n_high || n_high >= n_k) {
      if (tid == 0) report(a, r, kUndecided, s.m, 0.0f, finite);
      return;
    }
    n_kept = n_low + 1;
  }
  n_kept = min(n_kept, __syncthreads_count(tid < n && x >= border));
  // in the row's order
  const bool kept = tid < n_kept;
  place = 0;
  for (int i = 0; i < n_kept; ++i) place += (uint32_t)lists.list[i] > (uint32_t)key;  // (low words: ~index)
  if (kept) {
    lists.w[place] = w;
    lists.key[place] = key;
  }
  __syncthreads();
  w = kept ? lists.w[tid] : Pair{};
  Pair mass;
  const Pair with = block_sums<T>(w, cs.part, mass);
  const Pair goal = pair_from(draw.u) * mass;
  // the last one with a mass whose predecessors' mass is at most u W
  if (kept && w.h > 0.0f && with - w <= goal) atomicMax(&cs.token, tid);
  __syncthreads();
  if (tid == 0) {
    const uint64_t won = lists.key[max(cs.token, 0)];
    const float y = (from_ordered((uint32_t)(won >> 32)) - s.m) / draw.temperature;
    report(a, r, (int32_t) ~(uint32_t)won, y - log_of(total), y - log_of(mass), n_kept);
  }
}

// The same from up to kCap elements
template <int T>
__device__ void draw_from_many(const SampleArgs& a, int64_t r, CutShared<T>& cs, Lists& lists, const Draw& draw, const Scale& s, int n, int n_k,
                               bool by_p, bool exact, Pair total, float err, float border, int finite) {
  const int tid = threadIdx.x;
  int n2 = 2;
  while (n2 < n) n2 *= 2;
  for (int i = n + tid; i < n2; i += T) lists.key[i] = 0;
  sort_down<T>(lists.key, n2);
  for (int i = tid; i < n; i += T) {
    const float x = from_ordered((uint32_t)(lists.key[i] >> 32));
    lists.w[i] = weight(s, cs.table, x);
    if (x >= border) atomicAdd(&cs.n_border, 1);
  }
  __syncthreads();
  int n_kept = n_k;
  if (by_p) {
    Pair low = total + Pair{-err, 0.0f}, high = total + Pair{err, 0.0f};
    if (exact) low = high = sums_of<T>(lists.w, n_k, cs.part, [](int, Pair, Pair) {});
    const Pair p{draw.top_p, 0.0f};
    low = p * low;
    high = p * high;
    sums_of<T>(lists.w, n_k, cs.part, [&](int, Pair, Pair with) {
      if (with < low) atomicAdd(&cs.below[0], 1);
      if (with < high) atomicAdd(&cs.below[1], 1);
    });
    __syncthreads();
    if (cs.below[0] != cs.below[1] || cs.below[1] >= n_k) {
      if (tid == 0) report(a, r, kUndecided, s.m, 0.0f, finite);
      return;
    }
    n_kept = cs.below[0] + 1;
  }
  n_kept = min(n_kept, cs.n_border);
  // the kept ones in the row's order (low words: ~index), with their place among the sorted
  n2 = 2;
  while (n2 < n_kept) n2 *= 2;
  for (int i = tid; i < n2; i += T) lists.list[i] = i < n_kept ? lists.key[i] << 32 | (uint32_t)i : 0;
  sort_down<T>(lists.list, n2);
  const Pair mass = sums_of<T>(lists.w, n_kept, cs.part, [](int, Pair, Pair) {});
  constexpr int E = kCap / T;
  Pair w[E];
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = tid * E + i < n_kept ? lists.w[(uint32_t)lists.list[tid * E + i]] : Pair{};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (tid * E + i < n_kept) lists.w[tid * E + i] = w[i];
  __syncthreads();
  const Pair goal = pair_from(draw.u) * mass;
  sums_of<T>(lists.w, n_kept, cs.part, [&](int i, Pair before, Pair) {
    if (lists.w[i].h > 0.0f && before <= goal) atomicMax(&cs.token, i);
  });
  __syncthreads();
  if (tid == 0) {
    const uint64_t key = lists.list[max(cs.token, 0)];
    const float y = (from_ordered((uint32_t)(lists.key[(uint32_t)key] >> 32)) - s.m) / draw.temperature;
    report(a, r, (int32_t) ~(uint32_t)(key >> 32), y - log_of(total), y - log_of(mass), n_kept);
  }
}

// grid (cluster, rows)
template <typename In, bool CUT, int T>
__global__ void __launch_bounds__(T) sample_kernel(const SampleArgs a) {
  constexpr int N = Row<In>::N, U = 4, W = T / 32;
  // each lane's own ring of pieces: the next rounds are under way while one is summed
  constexpr int kRing = kStages * U * T * (int)sizeof(uint4);
  __shared__ __align__(16) unsigned char ring_smem[CUT && kRing < (int)sizeof(Lists) ? sizeof(Lists) : kRing];
  __shared__ __align__(16) unsigned char smem[sizeof(PassShared<T>)];
  __shared__ __align__(16) unsigned char cut_smem[CUT ? sizeof(CutShared<T>) : 16];
  Lists& lists = *reinterpret_cast<Lists*>(ring_smem);
  auto& sh = *reinterpret_cast<PassShared<T>*>(smem);
  auto& cs = *reinterpret_cast<CutShared<T>*>(cut_smem);
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int64_t r = blockIdx.y;
  const int rank = blockIdx.x, ranks = gridDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Draw draw;
  if (!draw.load(a, r)) {  // the whole cluster leaves
    if (rank == 0 && tid == 0) report(a, r, -1, 0.0f, 0.0f, 0);
    return;
  }
  const float c = exp2_scale(draw.temperature), limit = floor_limit(c);
  const Row<In> row(static_cast<const In*>(a.x) + r * a.ld, a.vocab);
  const int32_t cta = (row.pieces + ranks - 1) / ranks, each = (cta + W - 1) / W;
  auto share = [&](int rk, int w, int32_t& p0, int32_t& p1) {  // the pieces of a warp
    const int32_t c0 = min(row.pieces, rk * cta), c1 = min(row.pieces, c0 + cta);
    p0 = min(c1, c0 + w * each);
    p1 = min(c1, p0 + each);
  };
  int32_t w0, w1;
  share(rank, warp, w0, w1);
  if (CUT) {
    for (int i = tid; i < 256; i += T) cs.table[i] = kExp2.v[i];
    for (int i = tid; i < kMassBins; i += T) cs.bins[i] = 0;
    if (tid == 0) {
      cs.hits = cs.cands = 0;
      cs.last_bin = INT_MAX;
      cs.below[0] = cs.below[1] = cs.n_border = 0;
      cs.token = -1;
      if (draw.min_p > 0.0f && rank == 0) cs.reach = draw.reach();
    }
  }

  // the pass: this thread's sums against its own maximum
  float m = -INFINITY, wt = 0.0f;
  Sum sum;
  uint64_t wt2 = 0;
  uint32_t masked = 0;
  const uint64_t c2 = both(c);
  const int32_t inner = w0 == 0 && row.off > 0 ? 0 : min(w1, (row.off + a.vocab) / N);  // (the first piece may lack elements too)
  constexpr uint32_t kStage = U * T * sizeof(uint4);
  static_assert(kStages == 2 && (kStage & (kStage - 1)) == 0, "one round behind the one that is summed, told apart by a bit");
  const uint32_t ring = ptx::smem_u32(ring_smem) + 16 * tid;
  const uint4* next = reinterpret_cast<const uint4*>(row.x + (w0 * N - row.off)) + lane;  // the piece that is requested next
  uint32_t stage = 0;
  auto request = [&](int32_t p0, uint32_t to) {  // a round of whole pieces
    if (p0 + 32 * U <= inner) {
#pragma unroll
      for (int i = 0; i < U; ++i) cp_async_16(ring + to + 16 * T * i, next + 32 * i);
    }
    next += 32 * U;
    ptx::cp_async_commit();
  };
  request(w0, 0);
  request(w0 + 32 * U, kStage);
  for (int32_t p0 = w0; p0 < w1; p0 += 32 * U, stage ^= kStage) {
    uint4 u[U];
    ptx::cp_async_wait<1>();
    if (p0 + 32 * U <= inner) {
#pragma unroll
      for (int i = 0; i < U; ++i) u[i] = ld_shared_16(ring + stage + 16 * T * i);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) u[i] = p0 + 32 * i + lane < w1 ? row.load(p0 + 32 * i + lane) : absent<In>();
    }
    const float big = largest<In>(u);
    request(p0 + 64 * U, stage);  // (all of the stage has been read for `big`)
    if (big > m) {
      // All sums so far times a power: the exponential's and the product's rounding, up to 6 kStep of them, which
      // kMoved stands for in wt.
      const float d = m == -INFINITY ? 0.0f : fmaxf((m - big) * c, kTinyExp2), f = m == -INFINITY ? 0.0f : ex2(d);
      float h0, h1, l0, l1;
      ptx::f32x2_unpack(sum.h, h0, h1);
      ptx::f32x2_unpack(sum.l, l0, l1);
      float t0, t1;
      ptx::f32x2_unpack(wt2, t0, t1);
      wt = f * fmaf(d - kMoved, h0 + h1, wt + t0 + t1);
      wt2 = 0;
      sum.h = pair_of(h0 * f, h1 * f);
      sum.l = pair_of(l0 * f, l1 * f);
      m = big;
    }
    if (fabsf(m) <= limit) {
      const uint64_t nm2 = both(-m);
      uint64_t s[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint64_t v[N / 2], p2[N / 2];
        floored_pairs<In>(u[i], v);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const uint64_t y = pair_mul(add2(v[e], nm2), c2);
          float y0, y1;
          ptx::f32x2_unpack(y, y0, y1);
          p2[e] = pair_of(ex2(y0), ex2(y1));
          wt2 = pair_fma(p2[e], y, wt2);
        }
        s[i] = add2(p2[0], p2[1]);
        if (N == 8) s[i] = add2(s[i], add2(p2[N / 2 - 2], p2[N / 2 - 1]));
      }
      sum.add(add2(add2(s[0], s[1]), add2(s[2], s[3])), 0);
    } else {
      // a maximum out of range (left to the exact kernel), or -inf alone; NaN marks the sum
      float bad = 0.0f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[N];
        values<In>(u[i], v);
#pragma unroll
        for (int e = 0; e < N; ++e) bad = isnan(v[e]) ? v[e] : bad;
      }
      sum.add(both(bad), 0);
    }
    // elements of -inf, where there are any
    if (holds_masked<In>(u)) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[N];
        values<In>(u[i], v);
        const int32_t j0 = (p0 + 32 * i + lane) * N - row.off;
        if (p0 + 32 * i + lane < w1) {
#pragma unroll
          for (int e = 0; e < N; ++e) masked += v[e] == -INFINITY && j0 + e >= 0 && j0 + e < a.vocab;
        }
      }
    }
  }
  ptx::cp_async_wait<0>();  // (the ring's memory has other uses)
  {
    float h0, h1, l0, l1;
    ptx::f32x2_unpack(sum.h, h0, h1);
    ptx::f32x2_unpack(sum.l, l0, l1);
    Pair s = Pair{h0, l0} + Pair{h1, l1};
    ptx::f32x2_unpack(wt2, h0, h1);
    wt += h0 + h1;
    const float own = m;
    if (CUT) cs.most[tid] = m;
    // the warp's, against the warp's maximum
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float d = own == -INFINITY ? 0.0f : fmaxf((own - m) * c, kTinyExp2), f = own == -INFINITY ? 0.0f : ex2(d);
    wt = f * fmaf(d - kMoved, s.h, wt);
    s = Pair{s.h * f, s.l * f};
    s = scan_lanes(s);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) wt += __shfl_xor_sync(0xffffffffu, wt, k);
    masked = __reduce_add_sync(0xffffffffu, masked);
    if (lane == 31) sh.warp[warp] = WarpStat{m, s, wt, masked, {}};
  }
  const bool by_rank = CUT && draw.k > 0 && draw.k <= kCap;
  if (CUT) {
    // Each CTA gives the first ceil(k / CTAs) of its threads' maxima; the least of these bounds is one of the
    // k-th largest element.  The upper half of the ordered number: a lower bound.  (More than a maximum a thread: no
    // bound, the row is the exact kernel's.)
    float bound = -INFINITY;
    if (by_rank) {
      const int want = (int)((draw.k + ranks - 1) / ranks);
      const uint32_t own = max(ordered(cs.most[tid]) >> 16, 1u);
      uint32_t lo = 0;
      if (want <= T) {
        for (int b = 15; b >= 0; --b) {
          const uint32_t mid = lo | 1u << b;
          if (__syncthreads_count(own >= mid) >= want) lo = mid;
        }
      }
      bound = lo >= 0x80u ? from_ordered(lo << 16) : -INFINITY;  // (below: -inf)
    }
    if (tid == 0) sh.bound = bound;
  }
  if (ranks > 1) cluster_sync();
  else __syncthreads();

  // the row's sums, in every CTA: lane i has the shares 2 i and 2 i + 1
  if (warp == 0) {
    WarpStat st[2];
    float tau = INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * lane + i;
      st[i] = WarpStat{-INFINITY, {}, 0.0f, 0, {}};
      if (e < ranks * W) {
        const uint32_t at = ptx::mapa_shared(ptx::smem_u32(&sh.warp[e % W]), e / W);
        const float4 x = ptx::ld_dsmem_f32x4(at);
        st[i] = WarpStat{x.x, {x.y, x.z}, x.w, ptx::ld_dsmem_u32(at + 16), {}};
      }
    }
    if (CUT && lane < ranks) tau = __uint_as_float(ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.bound), lane)));
    float top = fmaxf(st[0].m, st[1].m);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      tau = fminf(tau, __shfl_xor_sync(0xffffffffu, tau, d));
    }
    // What each sum may be off by: its exponentials (4 kStep each) and their sums four deep, and the n rounds' own
    // sum (n^2 2^-53 where all are equal: a step from 2^14 rounds on); and of each exponent x - m, log2(e) / T and
    // their product are rounded, 3.3 kStep ln 2 times the exponent (and a share for wt itself).
    const float rounds = (float)((each + 32 * U - 1) / (32 * U)), steps = fmaf(rounds * 0x1p-14f, rounds * 0x1p-14f, 9.0f);
    float off[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float d = st[i].m == -INFINITY ? 0.0f : fmaxf((st[i].m - top) * c, kTinyExp2), f = st[i].m == -INFINITY ? 0.0f : ex2(d);
      const float s = st[i].s.h;
      st[i].s = Pair{s * f, st[i].s.l * f};
      off[i] = kStep * fmaf(kSlope, fabsf(f * fmaf(d - kMoved, s, st[i].wt)), steps * st[i].s.h);
    }
    masked = __reduce_add_sync(0xffffffffu, st[0].masked + st[1].masked);
    const Pair incl = scan_lanes(st[0].s + st[1].s), total = shuffle(incl, 31);
    float off_upto = off[0] + off[1];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const float o = __shfl_up_sync(0xffffffffu, off_upto, k);
      if (lane >= k) off_upto += o;
    }
    const float err = __shfl_sync(0xffffffffu, off_upto, 31);
    Pair before = shuffle_up(incl, 1);
    if (lane == 0) before = Pair{};
    const Pair goal = pair_from(draw.u) * total, middle = before + st[0].s;
    int at = st[0].s.h > 0.0f && before <= goal ? 2 * lane : -1;
    Pair start = before;
    if (st[1].s.h > 0.0f && middle <= goal) {
      at = 2 * lane + 1;
      start = middle;
    }
    const uint32_t can = __ballot_sync(0xffffffffu, at >= 0);
    const int from = can ? 31 - __clz(can) : 0;
    // By how much u W, less the sum ahead of a token in that warp's share, may be off.  With e what each weight is
    // off by it is the sum of (1 - u) e over the shares before, of u e over those behind; the share itself is summed anew
    // as far as the token: (1 + u) e, and 24 steps for what follows in fp32 there (the pairs: 2^-40).
    const float u = (float)draw.u, own = at & 1 ? off[1] : off[0], ahead = off_upto - off[0] - off[1] + (at & 1 ? off[0] : 0.0f);
    float margin = fmaf(1.0f - u, ahead, u * fmaxf(err - ahead - own, 0.0f));
    margin += fmaf(1.0f + u, own, 24.0f * kStep * (at & 1 ? st[1].s.h : st[0].s.h));
    margin = __shfl_sync(0xffffffffu, fmaf(margin, 1.0f + 0x1p-10f, 0x1p-38f * total.h + 0x1p-20f * err), from);
    at = __shfl_sync(0xffffffffu, at, from);
    start = shuffle(start, from);
    if (lane == 0) {
      sh.total = total;
      sh.left = goal - start;
      sh.m = top;
      sh.err = err;
      sh.margin = margin;
      sh.tau = tau;
      sh.finite = (uint32_t)a.vocab - masked;
      sh.owner = at < 0 ? 0 : at / W;
      sh.owner_warp = at < 0 ? 0 : at % W;
    }
  }
  __syncthreads();
  if (ranks > 1) cluster_arrive();  // this CTA has read the others' sums
  const Pair total = sh.total;
  m = sh.m;
  const float err = sh.err;
  const uint32_t finite = sh.finite;
  const int64_t k = draw.k;
  const bool by_k = CUT && k > 0 && k < (int64_t)finite, by_p = CUT && draw.top_p < 1.0f && draw.top_p > 0.0f,
             by_q = CUT && draw.min_p > 0.0f;
  const bool cut = by_k || by_p || by_q;
  const bool odd = isnan(total.h) || !(fabsf(m) <= limit);  // NaN, infinities, -inf alone, out of range
  if (odd) {
    if (rank == 0 && tid == 0) {
      if (isnan(total.h) || m == INFINITY) report(a, r, -1, NAN, NAN, 0);
      else if (m == -INFINITY) report(a, r, -1, -INFINITY, -INFINITY, 0);
      else report(a, r, kUndecided, m, 0.0f, (int32_t)finite);
    }
  } else if (!cut) {
    if (rank == sh.owner) {
      int32_t a0, a1;
      share(rank, sh.owner_warp, a0, a1);
      const int32_t some = (a1 - a0 + W - 1) / W;
      const int32_t b0 = min(a1, a0 + warp * some), b1 = min(a1, b0 + some);
      const uint64_t nm2 = both(-m);
      auto exponentials = [&](uint4 u, float (&p)[N]) {
        uint64_t v[N / 2];
        floored_pairs<In>(u, v);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          float y0, y1;
          ptx::f32x2_unpack(pair_mul(add2(v[e], nm2), c2), y0, y1);
          p[2 * e] = ex2(y0);
          p[2 * e + 1] = ex2(y1);
        }
      };
      auto sum_of = [&](const float (&p)[N]) {
        const float s = (p[0] + p[1]) + (p[2] + p[3]);
        return N == 8 ? s + ((p[N - 4] + p[N - 3]) + (p[N - 2] + p[N - 1])) : s;
      };
      Pair mass;
      for (int32_t p0 = b0; p0 < b1; p0 += 32 * U) {
        uint4 u[U];
#pragma unroll
        for (int i = 0; i < U; ++i) u[i] = p0 + 32 * i + lane < b1 ? row.load(p0 + 32 * i + lane) : absent<In>();
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float p[N];
          exponentials(u[i], p);
          mass = mass + Pair{sum_of(p), 0.0f};
        }
      }
      mass = scan_lanes(mass);
      if (lane == 31) sh.part[warp] = mass;
      __syncthreads();
      Pair left = sh.left, start, run;
      int mine = 0;
      for (int i = 0; i < W; ++i) {
        const Pair v = sh.part[i];
        if (v.h > 0.0f && run <= left) {
          mine = i;
          start = run;
        }
        run = run + v;
      }
      left = left - start;
      if (mine == warp) {
        // pieces in the row's order, 32 at a time; rest: what is left of u W ahead of them
        Pair rest = left;
        float under = -1.0f, over = -1.0f, x = 0.0f;
        int32_t token = kUndecided;
        for (int32_t p0 = b0; p0 < b1 && rest.h >= 0.0f; p0 += 32) {
          const uint4 u = p0 + lane < b1 ? row.load(p0 + lane) : absent<In>();
          float p[N], v[N];
          exponentials(u, p);
          values<In>(u, v);
          const float own = sum_of(p);
          float incl = own;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const float o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
          }
          float before = incl - own;
          const uint32_t can = __ballot_sync(0xffffffffu, own > 0.0f && before <= rest.h);
          if (can) {
            int32_t j = 0;
            float lo = 0.0f, hi = 0.0f, xj = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
              if (p[e] > 0.0f && before <= rest.h) {
                j = (p0 + lane) * N - row.off + e;
                xj = v[e];
                lo = rest.h - before;
                hi = before + p[e] - rest.h;
              }
              before += p[e];
            }
            const int from = 31 - __clz(can);
            token = __shfl_sync(0xffffffffu, j, from);
            x = __shfl_sync(0xffffffffu, xj, from);
            under = __shfl_sync(0xffffffffu, lo, from);
            over = __shfl_sync(0xffffffffu, hi, from);
          }
          rest = rest - Pair{__shfl_sync(0xffffffffu, incl, 31), 0.0f};
        }
        if (lane == 0) {
          const float margin = sh.margin;
          if (under >= margin && over >= margin) {
            const float y = (x - m) / draw.temperature, lp = y - log_of(total);
            report(a, r, token, lp, lp, (int32_t)finite);
          } else {
            report(a, r, kUndecided, m, 0.0f, (int32_t)finite);
          }
        }
      }
    }
  } else if (CUT) {
    if (ranks > 1) cluster_wait();
    // what may be kept: at or above tau, the border, and the last bin of the thread maxima that reach top_p's mass
    const float tau = by_k ? sh.tau : -INFINITY;
    const float c4 = 4.0f * c;
    int last_bin = INT_MAX;
    if (by_p && !by_k) {
      for (int q = 0; q < ranks; ++q) {
        const float v = __uint_as_float(ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&cs.most[tid]), q)));
        const float t = (m - v) * c4;
        if (t < (float)kMassBins) atomicAdd(&cs.bins[(int)t], (uint32_t)(ex2(-0.25f * t) * 0x1.fff8p+19f));
      }
      __syncthreads();
      if (warp == 0) {
        uint32_t n[4], own = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n[i] = cs.bins[4 * lane + i];
          own += n[i];
        }
        uint32_t incl = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        uint32_t run = incl - own;
        const float want = draw.top_p * (total.h + 2.0f * err) * 0x1p+20f * (1.0f + 8.0f * kStep);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          uint32_t upto = run;
          for (int e = 0; e <= i; ++e) upto += n[e];
          if (__uint2float_rd(upto) >= want) atomicMin(&cs.last_bin, 4 * lane + i);
        }
      }
      __syncthreads();
      last_bin = cs.last_bin;
    }
    const bool flat = by_p && !by_k && last_bin == INT_MAX;  // not even all maxima reach it
    const float border = by_q ? border_of(m, ranks > 1 ? __hiloint2double((int)ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&cs.reach), 0) + 4),
                                                                           (int)ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&cs.reach), 0)))
                                                       : cs.reach)
                              : -INFINITY;
    const bool possible = a.vocab <= kCap || (!flat && (!by_k || (by_rank && tau > -INFINITY)));
    const float least = fmaxf(tau, by_p ? -INFINITY : border);  // (top_p's mass counts what min_p cuts off)
    auto may = [&](float v) {
      return v > -INFINITY && v >= least && (last_bin == INT_MAX || (m - v) * c4 < (float)(last_bin + 1));
    };
    if (possible) {
      // the elements of the threads whose maxima may be kept, spread over all threads
      if (may(cs.most[tid])) cs.cand[atomicAdd(&cs.cands, 1)] = (int16_t)tid;
      __syncthreads();
      const int32_t rounds = (each + 31) / 32, items = cs.cands * rounds;
      for (int32_t f = tid; f < items; f += T) {
        const int who = cs.cand[f / rounds];
        int32_t b0, b1;
        share(rank, who >> 5, b0, b1);
        const int32_t p = b0 + (who & 31) + 32 * (f % rounds);
        if (p >= b1) continue;
        float v[N];
        values<In>(row.load(p), v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (!may(v[e])) continue;
          const int at = atomicAdd(&cs.hits, 1);
          if (at < kCap) lists.list[at] = (uint64_t)ordered(v[e]) << 32 | (uint32_t) ~(p * N - row.off + e);
        }
      }
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    int n = 0;
    bool whole = possible;
    if (rank == 0) {
      // all finds, one CTA's behind the other's
      const uint32_t h = lane < ranks ? ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&cs.hits), lane)) : 0;
      uint32_t upto = min(h, (uint32_t)kCap + 1);
#pragma unroll
      for (int d = 1; d < kMaxCluster; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      n = (int)__shfl_sync(0xffffffffu, upto, ranks - 1);
      whole = whole && n <= kCap;
      if (whole) {
        for (int i0 = 0; i0 < n; i0 += T) {
          const int i = i0 + tid;
          int q = 0, start = 0;
          for (int e = 0; e < ranks; ++e) {
            const int end = (int)__shfl_sync(0xffffffffu, upto, e);
            if (i >= end) q = e + 1, start = end;
          }
          if (i < n) {
            const uint32_t at = ptx::mapa_shared(ptx::smem_u32(&lists.list[i - start]), q);
            lists.key[i] = (uint64_t)ptx::ld_dsmem_u32(at + 4) << 32 | ptx::ld_dsmem_u32(at);
          }
        }
      }
    }
    if (ranks > 1) cluster_sync();  // rank 0 has read the others' finds: they are done
    if (rank == 0) {
      if (!whole || n < 1) {
        if (tid == 0) report(a, r, kUndecided, m, 0.0f, (int32_t)finite);
      } else {
        const Scale s = scale_of(m, draw.temperature);
        const int n_k = by_k ? (int)min((int64_t)n, k) : n;
        const bool exact = by_k || n == (int)finite;
        if (n <= T) draw_from_few<T>(a, r, cs, lists, draw, s, n, n_k, by_p, exact, total, err, border, (int)finite);
        else draw_from_many<T>(a, r, cs, lists, draw, s, n, n_k, by_p, exact, total, err, border, (int)finite);
      }
    }
  }
  if (ranks > 1 && (odd || !cut)) cluster_wait();  // the others have read this CTA's sums
}

constexpr int64_t kMaxRows = 65535;             // grid y
constexpr int64_t kMaxVocab = (int64_t)1 << 30;  // 32-bit element and piece numbers

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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

template <typename In>
cudaError_t launch_sample(const SampleArgs& a, int64_t rows, cudaStream_t stream) {
  const bool cut = a.temperature || a.top_k || a.top_p || a.min_p || a.k > 0 || a.p < 1.0f || a.q > 0.0f || a.t == 0.0f;
  const int64_t pieces = ((int64_t)a.vocab + Row<In>::N - 1) / Row<In>::N;
  cudaError_t e;
  if (pieces <= 256) {
    e = cut ? launch_clusters(sample_kernel<In, true, 64>, a, 1, rows, 64, stream) : launch_clusters(sample_kernel<In, false, 64>, a, 1, rows, 64, stream);
  } else {
    // Few rows are split over a cluster, down to a load round per CTA, until there are five CTAs for two SMs
    // (256 rows with the top 50: 39 us on clusters of two, 45 on four, 60 on one CTA).
    const int64_t want = 5 * (int64_t)sm_count() / 2, round = 256 * 4;
    int cluster = 1;
    while (cluster < kMaxCluster && rows * cluster < want && pieces > cluster * round) cluster *= 2;
    e = cut ? launch_clusters(sample_kernel<In, true, 256>, a, cluster, rows, 256, stream)
            : launch_clusters(sample_kernel<In, false, 256>, a, cluster, rows, 256, stream);
  }
  if (e != cudaSuccess) return e;
  return launch_sample_exact(a, sizeof(In) == 4, cut, stream);
}

}  // namespace

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  return n;
}

}  // namespace sampling
}  // namespace fp8rl

using namespace fp8rl;
using namespace fp8rl::sampling;

extern "C" FP8RL_API fp8rl_status fp8rl_sample(const void* d_logits, int32_t logits_fp32, int64_t rows, int64_t vocab,
                                               int64_t ld, const double* d_uniform, float temperature, int64_t top_k,
                                               float top_p, float min_p, const float* d_temperature,
                                               const int32_t* d_top_k, const float* d_top_p, const float* d_min_p,
                                               int32_t* d_tokens, float* d_lp, float* d_lp_kept, int32_t* d_kept,
                                               void* stream) {
  if (rows < 0 || vocab < 1 || ld < vocab || (logits_fp32 != 0 && logits_fp32 != 1)) return FP8RL_ERR_INVALID_ARG;
  if ((!d_temperature && !(temperature >= 0.0f && temperature <= FLT_MAX)) || (!d_top_k && top_k < 0) ||
      (!d_top_p && !(top_p > 0.0f)) || (!d_min_p && !(min_p >= 0.0f && min_p <= 1.0f)))
    return FP8RL_ERR_INVALID_ARG;
  if (rows == 0) return FP8RL_OK;
  if (!d_logits || !d_uniform || !d_tokens) return FP8RL_ERR_INVALID_ARG;
  if (vocab > kMaxVocab) return FP8RL_ERR_SHAPE;
  if (!aligned(d_logits, logits_fp32 ? 4 : 2) || !aligned(d_uniform, 8) || !aligned(d_temperature, 4) || !aligned(d_top_k, 4) ||
      !aligned(d_top_p, 4) || !aligned(d_min_p, 4) || !aligned(d_tokens, 4) || !aligned(d_lp, 4) || !aligned(d_lp_kept, 4) ||
      !aligned(d_kept, 4))
    return FP8RL_ERR_ALIGNMENT;
  uint32_t* err = nullptr;
  if (!check_word(&err)) return FP8RL_ERR_CUDA;
  const size_t size = logits_fp32 ? 4 : 2;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  for (int64_t r0 = 0; r0 < rows; r0 += kMaxRows) {
    const int64_t n = std::min(kMaxRows, rows - r0);
    SampleArgs a{};
    a.x = static_cast<const char*>(d_logits) + r0 * ld * (int64_t)size;
    a.uniform = d_uniform + r0;
    a.temperature = d_temperature ? d_temperature + r0 : nullptr;
    a.top_k = d_top_k ? d_top_k + r0 : nullptr;
    a.top_p = d_top_p ? d_top_p + r0 : nullptr;
    a.min_p = d_min_p ? d_min_p + r0 : nullptr;
    a.tokens = d_tokens + r0;
    a.lp = d_lp ? d_lp + r0 : nullptr;
    a.lp_kept = d_lp_kept ? d_lp_kept + r0 : nullptr;
    a.kept = d_kept ? d_kept + r0 : nullptr;
    a.ld = ld;
    a.rows = n;
    a.k = top_k;
    a.t = temperature;
    a.p = top_p;
    a.q = min_p;
    a.vocab = (int32_t)vocab;
    a.err = err;
    const cudaError_t e = logits_fp32 ? launch_sample<float>(a, n, cs) : launch_sample<uint16_t>(a, n, cs);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return FP8RL_ERR_CUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}
