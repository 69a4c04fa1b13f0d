// sample_exact.cu -- the draws that sampling's pass leaves open: weights and sums to
// 2^-40, as a rule 2^-44.  (sample.cu says what is computed and why twice.)
//
// A cluster takes a row, a CTA a contiguous share of it, a warp a contiguous share of
// that and a lane a contiguous run of pieces, so that sums by place in the row fall
// out and the token is found by descending through them.  The cut of top-k and top-p: by
// counts of the values themselves (bf16), or by histograms of 1024 bins over the values
// (counts, or masses as fractions of the bin's heaviest, of up to 13 bits), refined until the bin
// with the cut holds one value or at most 256 elements, which are sorted.
//
// Bound by latency: a row takes one to four passes over its share (the first from L2, the
// others from L1), each followed by an exchange over the cluster of about 2 us.  A row of
// 151936 bf16 takes 14 us where nothing is cut off (one pass, whose weights are 4 us of
// fp32 arithmetic), 33 with top-p: counting the values 5, their sums and weights 4, the
// cut 4, the kept ones' mass by place 9.  Where nothing is cut off four CTAs share an SM
// (64 registers: 1024 x 151936 136 us for both kernels when that came, 199 with one of 512 threads; 98 now).
#include <algorithm>

#include "sample.cuh"

namespace fp8rl {
namespace sampling {
namespace {

constexpr int kBins = 1024;
constexpr int kBinades = 15;                     // of bf16 values that have bins of their own
constexpr int kValues = 2 * 128 * kBinades + 2;  // (+ the ones nearer to 0, + the ones below)
constexpr int kValueBins = 4096;
constexpr int kList = 256;  // elements that are sorted, at most one a thread
static_assert(kValues <= kValueBins, "every value has a bin");

// what threads, warps and CTAs add up: sums, a maximum, a minimum, counts
struct alignas(16) Part {
  Pair a, b;
  float most = -INFINITY, least = INFINITY;
  uint32_t n = 0, k = 0;
};
static_assert(sizeof(Part) == 32, "read as 8 words");

__device__ __forceinline__ Part merge(const Part& x, const Part& y) {
  Part r;
  r.a = x.a + y.a;
  r.b = x.b + y.b;
  r.most = max_nan(x.most, y.most);
  r.least = fminf(x.least, y.least);
  r.n = x.n + y.n;
  r.k = x.k + y.k;
  return r;
}

template <int L>
__device__ __forceinline__ Part merge_lanes(Part v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) {
    Part o;
    o.a = Pair{__shfl_xor_sync(0xffffffffu, v.a.h, d), __shfl_xor_sync(0xffffffffu, v.a.l, d)};
    o.b = Pair{__shfl_xor_sync(0xffffffffu, v.b.h, d), __shfl_xor_sync(0xffffffffu, v.b.l, d)};
    o.most = __shfl_xor_sync(0xffffffffu, v.most, d);
    o.least = __shfl_xor_sync(0xffffffffu, v.least, d);
    o.n = __shfl_xor_sync(0xffffffffu, v.n, d);
    o.k = __shfl_xor_sync(0xffffffffu, v.k, d);
    v = merge(v, o);
  }
  return v;
}

template <int T>
struct Shared {
  float2 table[256];
  uint32_t hist[kValueBins];
  uint64_t list[kList], sorted[kList];
  Pair mass[kList];
  Part warp[T / 32];       // the last gather's sums of this CTA's warps
  Part mine[2];            // of this CTA, read by the others (two take turns)
  Part all[kMaxCluster];   // of every CTA
  Pair part[T / 32];
  float border;            // min-p's
  int32_t n_list, bin, last;
  int32_t row, nearest[T / 32];
  uint32_t scan[T / 32];
  uint32_t ahead;          // elements, and mass, ahead of `bin`
  Pair ahead_mass;
};

// kept: at or above `border`, and above `x` or equal to it at an index up to j
struct Keep {
  float border = -INFINITY, x = -INFINITY;
  int32_t j = INT_MAX;
  __device__ __forceinline__ bool operator()(float v, int32_t i) const {
    return v > -INFINITY && v >= border && (v > x || (v == x && i <= j));
  }
};

// of the elements equal to x (and at or above the border), the first `need` in the row's order are kept too, each
// of weight w
struct Ties {
  float border = -INFINITY, x = 0.0f;
  uint32_t need = 0;
  Pair w;
  __device__ __forceinline__ bool operator()(float v) const { return need > 0 && v == x && v >= border; }
  // the mass of kept elements among which `n` are equal to x
  __device__ __forceinline__ Pair mass(Pair others, uint32_t n) const { return need > 0 ? others + w * pair_from(min(n, need)) : others; }
};

template <typename In, int T>
struct Team {
  static constexpr int N = Row<In>::N, kWarps = T / 32;
  static constexpr int kUnroll = T > 256 ? 3 : 2;  // pieces a lane loads before it uses the first
  static_assert(kList <= T && kBins % T == 0 && kValueBins % T == 0, "threads take list entries and bins by their number");
  Shared<T>& sh;
  const Row<In> row;
  uint32_t rank, ranks;
  int32_t w0, w1;  // this warp's pieces
  int lane, warp;
  int turn = 0;

  __device__ __forceinline__ Team(Shared<T>& s, const In* x, int32_t vocab, uint32_t r, uint32_t rs)
      : sh(s), row(x, vocab), rank(r), ranks(rs), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    share(rank, warp, w0, w1);
  }
  // the pieces of a warp
  __device__ __forceinline__ void share(uint32_t r, int w, int32_t& a, int32_t& b) const {
    const int32_t cta = (row.pieces + (int32_t)ranks - 1) / (int32_t)ranks, each = (cta + kWarps - 1) / kWarps;
    const int32_t c0 = min(row.pieces, (int32_t)r * cta), c1 = min(row.pieces, c0 + cta);
    a = min(c1, c0 + w * each);
    b = min(c1, a + each);
  }

  // f(values, index of the first) of the pieces [a, b), lane by lane, and then() after a few; elements of no piece
  // are -inf
  struct Nothing {
    __device__ __forceinline__ void operator()() const {}
  };
  template <typename F, typename G = Nothing>
  __device__ __forceinline__ void each(int32_t a, int32_t b, F f, G then = G{}) const {
    for (int32_t p0 = a; p0 < b; p0 += 32 * kUnroll) {
      uint4 u[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int32_t p = p0 + 32 * i + lane;
        u[i] = p < b ? row.load(p) : absent<In>();
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        float v[N];
        values<In>(u[i], v);
        f(v, (p0 + 32 * i + lane) * N - row.off);
      }
      then();
    }
  }

  // the sum over the cluster; the warps' and the CTAs' stay in sh.warp and sh.all
  __device__ Part gather(Part v) {
    v = merge_lanes<32>(v);
    __syncthreads();  // the sums before have been read
    if (lane == 0) sh.warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
      v = merge_lanes<kWarps>(sh.warp[lane % kWarps]);
      if (lane == 0) (ranks > 1 ? sh.mine[turn] : sh.all[0]) = v;
    }
    if (ranks > 1) {
      cluster_sync();
      if (threadIdx.x < ranks * 8) {
        const uint32_t r = threadIdx.x >> 3, w = threadIdx.x & 7;
        reinterpret_cast<uint32_t*>(&sh.all[r])[w] = ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.mine[turn]), r) + 4 * w);
      }
      turn ^= 1;
    }
    __syncthreads();
    Part t;
    if ((lane & (kMaxCluster - 1)) < (int)ranks) t = sh.all[lane & (kMaxCluster - 1)];
    return merge_lanes<kMaxCluster>(t);
  }

  // mass and number of the kept elements of the pieces [a, b), this lane's part
  __device__ Part mass(const Scale& s, const Keep& keep, int32_t a, int32_t b) const {
    LongSum sum;
    uint32_t n = 0;
    each(a, b, [&](float (&v)[N], int32_t j0) {
      bool any = false;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (keep(v[e], j0 + e)) {
          ++n;
          any = true;
        } else {
          v[e] = -INFINITY;
        }
      }
      if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        uint64_t h, l;
        weights(s, sh.table, v[e], v[e + 1], h, l);
        sum.add(h, l);
      }
    }, [&] { sum.fold(); });
    Part p;
    p.a = sum.value();
    p.n = n;
    return p;
  }

  // The share of `keep` (and of the ties, Ties) in this warp's pieces, a contiguous run of them for each lane;
  // ALL: of everything
  __device__ __forceinline__ int32_t run() const { return (w1 - w0 + 31) / 32; }
  template <bool ALL>
  __device__ Part mass_of_run(const Scale& s, const Keep& keep, const Ties& ties) const {
    LongSum sum;
    Part p;
    const int32_t a = w0 + lane * run();
    for (int32_t i0 = 0; i0 < run(); i0 += kUnroll) {
      uint4 u[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) u[i] = i0 + i < run() && a + i0 + i < w1 ? row.load(a + i0 + i) : absent<In>();
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int32_t j0 = (a + i0 + i) * N - row.off;
        float v[N];
        values<In>(u[i], v);
        if (!ALL) {
          bool any = false;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            if (keep(v[e], j0 + e)) {
              ++p.n;
              any = true;
            } else {
              p.k += ties(v[e]);
              v[e] = -INFINITY;
            }
          }
          if (!__any_sync(0xffffffffu, any)) continue;
        }
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          uint64_t h, l;
          weights(s, sh.table, v[e], v[e + 1], h, l);
          sum.add(h, l);
        }
      }
      sum.fold();
    }
    p.a = sum.value();
    return p;
  }

  // Top-k and top-p of bf16 rows by the values themselves: every value in 15 binades has a bin that
  // counts it, so a bin's mass is its count times one weight and a cut needs no second look.
  // False where a cut falls among the values nearer to 0 than that (or far below): nothing is changed then.
  __device__ bool by_value(const Scale& s, Keep& keep, Ties& ties, uint32_t k, float top_p, Pair& total) {
    constexpr int kEach = kValueBins / T, kTiny = 128 * kBinades, kRest = kValues - 1;
    // the binades below the largest magnitude that matters
    const float far = fmaxf(fabsf(s.m), 64.0f / s.hi - s.m);
    const int32_t lowest = max(0, (int32_t)(__float_as_uint(fminf(far, FLT_MAX)) >> 23) - (kBinades - 1)) << 7;  // its upper 16 bits
    auto place = [&](float x) {
      const uint32_t b = __float_as_uint(x) >> 16;
      const int32_t g = (int32_t)(b & 0x7FFFu) - lowest;  // magnitudes in steps of bf16
      if (g < 0 || (b & 0x7FFFu) == 0) return kTiny;      // (zeros of both signs together)
      if (b >> 15) return g < kTiny ? kTiny + 1 + g : kRest;
      return kTiny - 1 - g;  // (no value is above the largest binade)
    };
    auto value_at = [&](int b) {
      const uint32_t g = (uint32_t)(b < kTiny ? kTiny - 1 - b : b - kTiny - 1) + (uint32_t)lowest;
      return __uint_as_float((b < kTiny ? g : g | 0x8000u) << 16);
    };
    for (int i = threadIdx.x; i < kValueBins; i += T) sh.hist[i] = 0;
    __syncthreads();
    // counts, and the tiny ones' mass
    LongSum sum;
    each(w0, w1, [&](float (&v)[N], int32_t) {
      bool any = false;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (v[e] > -INFINITY) {
          const int b = place(v[e]);
          atomicAdd(&sh.hist[b], 1u);
          if (b == kTiny) any = true;
          else v[e] = -INFINITY;
        }
      }
      if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        uint64_t h, l;
        weights(s, sh.table, v[e], v[e + 1], h, l);
        sum.add(h, l);
      }
    }, [&] { sum.fold(); });
    Part tiny;
    tiny.a = sum.value();
    tiny = gather(tiny);  // (and the counts are there)
    // each CTA adds up its part of the bins, in the place that no other reads; then all read the sums
    const int part = kValueBins / (int)ranks;
    if (ranks > 1) {
      for (int i = threadIdx.x; i < part; i += T) {
        const uint32_t at = ptx::smem_u32(&sh.hist[rank * part + i]);
        uint32_t n = 0;
        for (uint32_t r = 0; r < ranks; ++r) n += ptx::ld_dsmem_u32(ptx::mapa_shared(at, r));
        sh.hist[rank * part + i] = n;
      }
      cluster_sync();
    }
    uint32_t count[kEach], n_own = 0;
    Pair mass[kEach], own;
    const uint32_t bins = ptx::mapa_shared(ptx::smem_u32(&sh.hist[kEach * threadIdx.x]), kEach * threadIdx.x / part);
#pragma unroll
    for (int i = 0; i < kEach; i += 4) {
      const float4 c = ptx::ld_dsmem_f32x4(bins + 4 * i);
      count[i] = __float_as_uint(c.x);
      count[i + 1] = __float_as_uint(c.y);
      count[i + 2] = __float_as_uint(c.z);
      count[i + 3] = __float_as_uint(c.w);
    }
#pragma unroll
    for (int i = 0; i < kEach; i += 2) {
      const int b = threadIdx.x * kEach + i;
      mass[i] = mass[i + 1] = Pair{};
      n_own += count[i] + count[i + 1];
      if (count[i] + count[i + 1] > 0) {
        uint64_t h, l;
        weights(s, sh.table, count[i] > 0 && b < kRest ? value_at(b) : -INFINITY,
                count[i + 1] > 0 && b + 1 < kRest ? value_at(b + 1) : -INFINITY, h, l);
        float h0, h1, l0, l1;
        ptx::f32x2_unpack(h, h0, h1);
        ptx::f32x2_unpack(l, l0, l1);
        mass[i] = b == kTiny ? tiny.a : normal(h0, l0) * pair_from(count[i]);
        mass[i + 1] = b + 1 == kTiny ? tiny.a : normal(h1, l1) * pair_from(count[i + 1]);
      }
      own = own + (mass[i] + mass[i + 1]);
    }
    // counts and masses ahead of this thread's bins
    uint32_t n_run = n_own;
    Pair run = scan_lanes(own);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, n_run, d);
      if (lane >= d) n_run += o;
    }
    if (lane == 31) {
      sh.part[warp] = run;
      sh.scan[warp] = n_run;
    }
    run = shuffle_up(run, 1);
    if (lane == 0) run = Pair{};
    n_run -= n_own;
    __syncthreads();
    const Pair upto = scan_lanes(lane < kWarps ? sh.part[lane] : Pair{});
    uint32_t n_upto = lane < kWarps ? sh.scan[lane] : 0;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, n_upto, d);
      if (lane >= d) n_upto += o;
    }
    const Pair all = shuffle(upto, kWarps - 1), ahead = shuffle(upto, (warp + 31) & 31);
    const uint32_t n_ahead = __shfl_sync(0xffffffffu, n_upto, (warp + 31) & 31);
    if (warp > 0) {
      run = ahead + run;
      n_run += n_ahead;
    }
    total = all;
    auto found = [&](auto reached) {  // the first bin at whose end `reached` holds; every thread hears of it
      if (threadIdx.x == 0) sh.bin = INT_MAX;
      __syncthreads();
      int mine = -1;
      uint32_t n = n_run, in = 0;
      Pair m = run;
      if (n_own > 0 && !reached(n_run, run) && reached(n_run + n_own, run + own)) {  // (one thread, roundings aside)
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          if (mine >= 0 || count[i] == 0) continue;
          in = count[i];
          if (reached(n + in, m + mass[i])) {
            mine = threadIdx.x * kEach + i;
          } else {
            n += in;
            m = m + mass[i];
          }
        }
        if (mine >= 0) atomicMin(&sh.bin, mine);
      }
      __syncthreads();
      const int b = sh.bin;
      if (b == mine) {
        sh.ahead = n;
        sh.ahead_mass = m;
        sh.last = (int)in;
      }
      __syncthreads();
      return b;
    };
    int bin = -1;
    uint32_t need = 0;  // elements of that bin that are kept
    Pair mass_k = all, w;
    if (k > 0) {
      bin = found([&](uint32_t n, Pair) { return n >= k; });
      if (bin == kTiny || bin >= kRest) return false;
      need = k - sh.ahead;
      w = weight(s, sh.table, value_at(bin));
      mass_k = sh.ahead_mass + w * pair_from(need);
    }
    if (top_p < 1.0f) {
      const Pair target = Pair{top_p, 0.0f} * mass_k;
      const int b = found([&](uint32_t, Pair m) { return target <= m; });
      if (b == kTiny || b == kRest) return false;
      if (b < kValues && (bin < 0 || b <= bin)) {  // (no bin: rounding; all of them, or the first k)
        w = weight(s, sh.table, value_at(b));
        need = first_reaching(target - sh.ahead_mass, w, b == bin ? need : (uint32_t)sh.last);
        bin = b;
      }
    }
    if (bin < 0) return true;
    keep.x = value_at(bin);
    keep.j = -1;
    ties.x = keep.x;
    ties.need = need;
    ties.w = w;
    return true;
  }

  // the smallest n in [1, most] with n w >= left: an fp32 quotient, corrected by its remainder
  static __device__ uint32_t first_reaching(Pair left, Pair w, uint32_t most) {
    if (!(w.h > 0.0f) || most <= 1) return 1;
    float n = fminf(fmaxf(floorf(left.h / w.h), 1.0f), (float)most);
    const Pair rest = left - w * pair_from((uint32_t)n);
    int32_t at = (int32_t)n + (int32_t)floorf(rest.h / w.h);
    at = max(1, min(at, (int32_t)most));
    while (at < (int32_t)most && w * pair_from((uint32_t)at) < left) ++at;
    while (at > 1 && left <= w * pair_from((uint32_t)(at - 1))) --at;
    return (uint32_t)at;
  }

  // The index of the need-th element (from 1) with value x among the kept, in the row's order
  __device__ int32_t nth_equal(float x, const Keep& keep, uint32_t need) {
    Part p;
    each(w0, w1, [&](float (&v)[N], int32_t j0) {
#pragma unroll
      for (int e = 0; e < N; ++e) p.n += v[e] == x && keep(v[e], j0 + e);
    });
    gather(p);
    uint32_t r = 0;
    while (r + 1 < ranks && need > sh.all[r].n) need -= sh.all[r++].n;
    Part found;
    if (r == rank) {
      int w = 0;
      while (w + 1 < kWarps && need > sh.warp[w].n) need -= sh.warp[w++].n;
      if (w == warp) {
        for (int32_t p0 = w0; p0 < w1; p0 += 32) {
          float v[N];
          values<In>(p0 + lane < w1 ? row.load(p0 + lane) : absent<In>(), v);
          const int32_t j0 = (p0 + lane) * N - row.off;
          uint32_t mine = 0;
#pragma unroll
          for (int e = 0; e < N; ++e) mine += v[e] == x && keep(v[e], j0 + e);
          uint32_t incl = mine;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
          }
          const uint32_t total = __shfl_sync(0xffffffffu, incl, 31);
          if (need <= total) {
            uint32_t left = need - (incl - mine);  // (past 2^31: not here)
            if (incl >= need && incl - mine < need) {
#pragma unroll
              for (int e = 0; e < N; ++e)
                if (v[e] == x && keep(v[e], j0 + e) && --left == 0) found.n = (uint32_t)(j0 + e) + 1;
            }
            break;
          }
          need -= total;
        }
      }
    }
    return (int32_t)gather(found).n - 1;
  }

  // Narrows `keep` to its first k elements (by count), or to the shortest prefix with mass >= target of `whole`.
  // Every CTA of the cluster comes to the same decisions, from the same sums.
  __device__ void select(const Scale& s, Keep& keep, bool by_count, uint32_t k, Pair target, Pair whole) {
    // bins over (hi - x) * pre * scale; a bin is `step` wide in t
    float hi = s.m, lo = -FLT_MAX, pre = 1.0f, scale = 16.0f * s.hi, step = 1.0f / 16.0f;
    Pair above;            // mass and number of what lies above the range
    uint32_t n_above = 0;
    // a bin adds up to `unit` an element: 13 bits, or as many as leave the sum of all of the row's below 2^32 (rows from
    // 2^19 on; a bin that wrapped misplaced the cut's first guess: 4.7 ms where 0.15 do)
    const float unit = (float)(8192u >> max(0, 32 - __clz(row.vocab) - 19));
    for (;;) {
      auto place = [&](float x, int32_t j, float& f) {  // the bin, or -1
        if (!(x <= hi && x >= lo && keep(x, j))) return -1;
        f = (hi - x) * pre * scale;
        return f < (float)(kBins - 1) ? (int)f : kBins - 1;
      };
      for (int i = threadIdx.x; i < kBins; i += T) sh.hist[i] = 0;
      if (threadIdx.x == 0) {
        sh.bin = INT_MAX;
        sh.last = 0;
      }
      __syncthreads();
      each(w0, w1, [&](float (&v)[N], int32_t j0) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float f;
          const int b = place(v[e], j0 + e, f);
          if (b < 0) continue;
          const uint32_t q = by_count ? 1u : (uint32_t)(ex2(fmaxf(((float)b - f) * step, -64.0f)) * unit);
          if (q) atomicAdd(&sh.hist[b], q);
        }
      });
      if (ranks > 1) cluster_sync();
      else __syncthreads();
      // the cluster's bins, some a thread
      constexpr int kEach = kBins / T;
      uint32_t c[kEach];
      float f[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        c[i] = 0;
        for (uint32_t r = 0; r < ranks; ++r) c[i] += ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.hist[kEach * threadIdx.x + i]), r));
        f[i] = (float)c[i];
      }
      // the first bin in which the running sum reaches what is asked for (counts exactly, masses nearly)
      const float t0 = (s.m - hi) * s.hi;
      uint32_t n_run = 0, n_own = 0;
      float f_run = 0.0f, f_own = 0.0f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        f[i] *= ex2(fmaxf(-t0 - (float)(kEach * threadIdx.x + i) * step, -120.0f));
        n_own += c[i];
        f_own += f[i];
      }
      n_run = n_own, f_run = f_own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, n_run, d);
        const float o = __shfl_up_sync(0xffffffffu, f_run, d);
        if (lane >= d) {
          n_run += n;
          f_run += o;
        }
      }
      if (lane == 31) {
        sh.warp[warp].n = n_run;
        sh.warp[warp].most = f_run;
      }
      __syncthreads();
      n_run -= n_own;
      f_run -= f_own;
      float f_all = 0.0f;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
          n_run += sh.warp[w].n;
          f_run += sh.warp[w].most;
        }
        f_all += sh.warp[w].most;
      }
      // (the masses are up to 1 / unit small: as shares of their own sum, head and tail are good to that)
      const float share = (target - above).h / whole.h * f_all;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (c[i] == 0) continue;
        const int b = kEach * threadIdx.x + i;
        atomicMax(&sh.last, b);
        n_run += c[i];
        f_run += f[i];
        if (by_count ? n_run >= k - n_above : f_run >= share) atomicMin(&sh.bin, b);
      }
      __syncthreads();
      int bin = min(sh.bin, sh.last);

      // what lies above the bin and in it
      Part t;
      for (int way = 0;;) {
        Part p;
        LongSum sa, sb;
        each(w0, w1, [&](float (&v)[N], int32_t j0) {
          bool any = false;
          bool in[N];
#pragma unroll
          for (int e = 0; e < N; ++e) {
            float g;
            const int b = place(v[e], j0 + e, g);
            in[e] = b == bin;
            if (in[e]) {
              p.most = fmaxf(p.most, v[e]);
              p.least = fminf(p.least, v[e]);
              ++p.k;
            } else if (b >= 0 && b < bin) {
              ++p.n;
            } else {
              v[e] = -INFINITY;
            }
            any |= v[e] > -INFINITY;
          }
          if (by_count || !__any_sync(0xffffffffu, any)) return;
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            uint64_t h, l;
            weights(s, sh.table, v[e], v[e + 1], h, l);
            float h0, h1, l0, l1;
            ptx::f32x2_unpack(h, h0, h1);
            ptx::f32x2_unpack(l, l0, l1);
            sb.add(pair_of(in[e] ? h0 : 0.0f, in[e + 1] ? h1 : 0.0f), pair_of(in[e] ? l0 : 0.0f, in[e + 1] ? l1 : 0.0f));
            sa.add(pair_of(in[e] ? 0.0f : h0, in[e + 1] ? 0.0f : h1), pair_of(in[e] ? 0.0f : l0, in[e + 1] ? 0.0f : l1));
          }
        }, [&] {
          sa.fold();
          sb.fold();
        });
        p.a = sa.value();
        p.b = sb.value();
        t = gather(p);
        if (by_count) break;
        // the histogram's masses are not exact: step to the neighbour until the cut lies inside
        const bool below = target <= above + t.a && t.n > 0;
        const bool past = above + t.a + t.b < target;
        if (below && way <= 0 && bin > 0) {
          way = -1;
          --bin;
        } else if ((past || t.k == 0) && way >= 0 && bin < kBins - 1) {
          way = 1;
          ++bin;
        } else {
          break;
        }
      }
      if (t.k == 0) return;  // nothing further down: all of `keep` stays
      above = above + t.a;
      n_above += t.n;
      if (t.k > (uint32_t)kList && t.most > t.least) {  // a closer look at the bin
        hi = t.most;
        lo = t.least;
        whole = t.b;
        const float width = hi - lo;
        pre = width < 0x1p-60f ? 0x1p+100f : 1.0f;
        scale = width > FLT_MAX ? 0x1p-119f : (float)(kBins - 1) / (width * pre);
        step = s.hi / (pre * scale);
        continue;
      }
      if (t.k > (uint32_t)kList) {  // many of one value
        uint32_t need = by_count ? k - n_above : 1;
        if (!by_count) {
          need = first_reaching(target - above, weight(s, sh.table, t.most), t.k);
        }
        need = max(1u, min(need, t.k));
        const int32_t j = need == t.k ? INT_MAX : nth_equal(t.most, keep, need);
        keep.j = t.most == keep.x ? min(keep.j, j) : j;
        keep.x = t.most;
        return;
      }
      // few: every CTA sorts them all
      if (threadIdx.x == 0) sh.n_list = 0;
      __syncthreads();
      each(w0, w1, [&](float (&v)[N], int32_t j0) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float g;
          if (place(v[e], j0 + e, g) != bin) continue;
          const int at = atomicAdd(&sh.n_list, 1);
          if (at < kList) sh.list[at] = (uint64_t)ordered(v[e]) << 32 | (uint32_t) ~(j0 + e);
        }
      });
      __syncthreads();
      Part count;
      if (threadIdx.x == 0) count.n = (uint32_t)min(sh.n_list, kList);
      const int32_t n = (int32_t)gather(count).n;
      uint64_t key = 0;
      if ((int32_t)threadIdx.x < n) {
        uint32_t r = 0, at = threadIdx.x;
        while (r + 1 < ranks && at >= sh.all[r].n) at -= sh.all[r++].n;
        const uint32_t from = ptx::mapa_shared(ptx::smem_u32(&sh.list[at]), r);
        key = (uint64_t)ptx::ld_dsmem_u32(from + 4) << 32 | ptx::ld_dsmem_u32(from);
        sh.sorted[threadIdx.x] = key;
      }
      if (ranks > 1) cluster_sync();
      else __syncthreads();
      int32_t at = 0;
      for (int32_t i = 0; i < n; ++i) at += sh.sorted[i] > key;
      __syncthreads();
      if ((int32_t)threadIdx.x < n) sh.list[at] = key;
      __syncthreads();
      int32_t cut = (int32_t)(k - n_above) - 1;
      if (!by_count) {
        if ((int32_t)threadIdx.x < n) {
          sh.mass[threadIdx.x] = weight(s, sh.table, from_ordered((uint32_t)(sh.list[threadIdx.x] >> 32)));
        } else if (threadIdx.x < kList) {
          sh.mass[threadIdx.x] = Pair{};
        }
        if (threadIdx.x == 0) sh.bin = n - 1;
        __syncthreads();
        if (warp == 0) {
          constexpr int kEntries = kList / 32;
          Pair sum;
          for (int i = 0; i < kEntries; ++i) sum = sum + sh.mass[lane * kEntries + i];
          Pair ahead = shuffle_up(scan_lanes(sum), 1);
          if (lane == 0) ahead = Pair{};
          Pair part = above + ahead;
          for (int i = 0; i < kEntries; ++i) {
            part = part + sh.mass[lane * kEntries + i];
            if (target <= part) {
              atomicMin(&sh.bin, lane * kEntries + i);
              break;
            }
          }
        }
        __syncthreads();
        cut = sh.bin;
      }
      cut = max(0, min(cut, n - 1));
      const uint64_t border = sh.list[cut];
      keep.x = from_ordered((uint32_t)(border >> 32));
      keep.j = (int32_t) ~(uint32_t)border;
      __syncthreads();
      return;
    }
  }
};


// ------------------------------------------------------------------ kernel

// The next row for this cluster: from `start` on, the first one still undecided that it gets hold of (a row is
// taken by writing kTaken over its mark), -1: none within the next `cover`.  All of the cluster call it; `cursor` is
// rank 0's place.  Rows are few and fall where they fall: with each cluster keeping to rows of its own, 128 of
// 1024 x 151936 (as many as the pass's wider margin left then; 40 or so now) took 50 us, five rows one behind the other
// somewhere.
constexpr int32_t kTaken = -3;
template <int T>
__device__ int64_t next_row(const SampleArgs& a, Shared<T>& sh, uint32_t rank, uint32_t ranks, int32_t start, int32_t cover, int32_t& cursor) {
  constexpr int kLook = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = (int32_t)a.rows;
  int32_t row = -1;
  if (rank == 0) {
    while (cursor < cover) {
      int32_t nearest = INT_MAX;
#pragma unroll
      for (int i = kLook - 1; i >= 0; --i) {
        const int32_t at = cursor + i * T + (int32_t)threadIdx.x;
        if (at >= cover) continue;
        const int32_t r = start + at < rows ? start + at : start + at - rows;
        if (__ldcg(a.tokens + r) == kUndecided) nearest = at;
      }
      nearest = __reduce_min_sync(0xffffffffu, nearest);
      __syncthreads();  // the look before has been read
      if (lane == 0) sh.nearest[warp] = nearest;
      __syncthreads();
      nearest = __reduce_min_sync(0xffffffffu, lane < T / 32 ? sh.nearest[lane] : INT_MAX);
      if (nearest == INT_MAX) {
        cursor += kLook * T;
        continue;
      }
      cursor = nearest + 1;
      const int32_t r = start + nearest < rows ? start + nearest : start + nearest - rows;
      if (threadIdx.x == 0) sh.row = dcheck(r >= 0 && r < rows, a.err) && atomicCAS(a.tokens + r, kUndecided, kTaken) == kUndecided ? r : -1;
      __syncthreads();
      row = sh.row;
      if (row >= 0) break;
    }
    if (row < 0) {
      __syncthreads();
      if (threadIdx.x == 0) sh.row = -1;
    }
  }
  if (ranks > 1) {
    cluster_sync();
    return (int32_t)ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.row), 0));
  }
  return row;
}

// grid (cluster, clusters): the rows that the pass has left.  CUT: something may be cut off
template <typename In, bool CUT, int T, int RESIDENT>
__global__ void __launch_bounds__(T, RESIDENT) sample_exact_kernel(const SampleArgs a) {
  __shared__ __align__(16) unsigned char smem[sizeof(Shared<T>)];
  Shared<T>& sh = *reinterpret_cast<Shared<T>*>(smem);
  constexpr int N = Row<In>::N;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const uint32_t rank = blockIdx.x, ranks = gridDim.x;
  bool first = true;
  const int32_t share = (int32_t)((a.rows + gridDim.y - 1) / gridDim.y), start = (int32_t)min(a.rows - 1, (int64_t)blockIdx.y * share);
  const int32_t cover = (int32_t)min(a.rows, max((int64_t)16 * share, (int64_t)8192));
  int32_t cursor = 0;
  const bool own = a.rows <= (int64_t)gridDim.y;  // a row to each cluster: nothing to agree on
  if (own && __ldcg(a.tokens + blockIdx.y) != kUndecided) return;
  for (;;) {
    const int64_t r = own ? (first ? (int64_t)blockIdx.y : -1) : next_row<T>(a, sh, rank, ranks, start, cover, cursor);
    if (r < 0) break;
    if (first) {
      for (int i = threadIdx.x; i < 256; i += T) sh.table[i] = kExp2.v[i];
      first = false;
    }
    Draw draw;
    draw.load(a, r);
    Team<In, T> team(sh, static_cast<const In*>(a.x) + r * a.ld, a.vocab, rank, ranks);
    // the maximum and the number of finite logits: the pass has left them, if it had where
    float m;
    uint32_t finite;
    Part p;
    if (a.lp && a.kept) {
      m = __ldcg(a.lp + r);
      finite = (uint32_t)__ldcg(a.kept + r);
    } else {
      team.each(team.w0, team.w1, [&](float (&v)[N], int32_t) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          p.most = fmaxf(p.most, v[e]);
          p.n += v[e] > -INFINITY;
        }
      });
      p = team.gather(p);
      m = p.most;
      finite = p.n;
    }
    const Scale s = scale_of(m, draw.temperature);
    Keep keep;
    Ties ties;
    Pair total;
    bool summed = false;
    if (threadIdx.x == 0) sh.border = CUT && draw.min_p > 0.0f ? border_of(m, draw.reach()) : -INFINITY;
    __syncthreads();  // (the table too)
    if (CUT) {
      // the cut, and the mass of all
      const bool by_k = draw.k > 0 && draw.k < (int64_t)finite, by_p = draw.top_p < 1.0f && draw.top_p > 0.0f;
      const float border = sh.border;
      if (by_k || by_p) {
        summed = sizeof(In) == 2 && team.by_value(s, keep, ties, by_k ? (uint32_t)draw.k : 0, by_p ? draw.top_p : 1.0f, total);
        if (!summed) {
          total = team.gather(team.mass(s, keep, team.w0, team.w1)).a;
          summed = true;
          if (by_k) team.select(s, keep, true, (uint32_t)draw.k, Pair{}, Pair{1.0f, 0.0f});
          if (by_p) {
            const Pair all = by_k ? team.gather(team.mass(s, keep, team.w0, team.w1)).a : total;
            team.select(s, keep, false, 0, Pair{draw.top_p, 0.0f} * all, all);
          }
        }
      }
      if (border > -INFINITY && !summed) {
        total = team.gather(team.mass(s, keep, team.w0, team.w1)).a;
        summed = true;
      }
      keep.border = ties.border = border;
    }
    const Part mine = team.template mass_of_run<!CUT>(s, keep, ties);  // of this lane's run
    p = team.gather(mine);
    const Pair mass = ties.mass(p.a, p.k);
    const int32_t kept = CUT ? (int32_t)(p.n + min(p.k, ties.need)) : (int32_t)finite;
    if (!summed) total = mass;

    // the last CTA, warp, lane and element with a mass of its own whose predecessors' mass is at most u W
    const Pair goal = pair_from(draw.u) * mass;
    Pair sum;  // of what lies ahead: the mass without ties, and the number of those
    uint32_t n = 0;
    auto descend = [&](const Part& v) {  // lane i has the i-th of the places to choose from
      const Pair incl = scan_lanes(v.a);
      Pair ahead = shuffle_up(incl, 1);
      if (team.lane == 0) ahead = Pair{};
      uint32_t n_incl = v.k;
      if (CUT) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, n_incl, d);
          if (team.lane >= d) n_incl += o;
        }
      }
      // (from `ahead`, not from the scan's next sum, which may round otherwise: an empty place adds nothing)
      const Pair before = ties.mass(sum + ahead, n + n_incl - v.k), after = ties.mass(sum + ahead + v.a, n + n_incl);
      const uint32_t can = __ballot_sync(0xffffffffu, before < after && before <= goal);
      const int at = can ? 31 - __clz(can) : 0;
      sum = sum + shuffle(ahead, at);
      n += __shfl_sync(0xffffffffu, n_incl - v.k, at);
      return at;
    };
    const int owner = descend(team.lane < (int)ranks ? sh.all[team.lane] : Part{});
    if (owner == (int)rank && descend(team.lane < T / 32 ? sh.warp[team.lane] : Part{}) == team.warp) {
      const int from = descend(mine);
      // that lane's elements, one a lane
      const int32_t first_j = (team.w0 + from * team.run()) * N - team.row.off, some = team.run() * N;
      int32_t token = -1;
      float x = 0.0f;
      for (int32_t e0 = 0; e0 < some; e0 += 32) {
        const int32_t j = first_j + e0 + team.lane;
        float v = -INFINITY;
        if (e0 + team.lane < some && j >= 0 && j < a.vocab) {
          if (sizeof(In) == 2) v = bf16_lo((uint32_t) reinterpret_cast<const uint16_t*>(team.row.x)[j]);
          else v = reinterpret_cast<const float*>(team.row.x)[j];
        }
        Part one;
        const bool in = keep(v, j);
        one.a = weight(s, sh.table, in ? v : -INFINITY);
        one.k = CUT && !in && ties(v);
        const Pair incl = scan_lanes(one.a);
        Pair ahead = shuffle_up(incl, 1);
        if (team.lane == 0) ahead = Pair{};
        const uint32_t tied = __ballot_sync(0xffffffffu, one.k != 0);
        const uint32_t t_ahead = __popc(tied & ((1u << team.lane) - 1));
        const Pair before = ties.mass(sum + ahead, n + t_ahead);
        const uint32_t can = __ballot_sync(0xffffffffu, before < ties.mass(sum + ahead + one.a, n + t_ahead + one.k) && before <= goal);
        if (can) {
          token = __shfl_sync(0xffffffffu, j, 31 - __clz(can));
          x = __shfl_sync(0xffffffffu, v, 31 - __clz(can));
        }
        sum = sum + shuffle(incl, 31);
        n += __popc(tied);
        if (goal < ties.mass(sum, n)) break;
      }
      if (team.lane == 0) {
        const float y = (x - m) / draw.temperature;
        report(a, r, token, y - log_of(total), y - log_of(mass), kept);
      }
    }
    if (ranks > 1) cluster_sync();  // the others have read this CTA's shared memory
    else __syncthreads();
  }
  if (ranks > 1 && !own) cluster_sync();  // the others have read that there is no row
}

template <typename In, bool CUT, int T, int RESIDENT>
cudaError_t launch_exact(const SampleArgs& a, cudaStream_t stream) {
  const int64_t pieces = ((int64_t)a.vocab + Row<In>::N - 1) / Row<In>::N;
  // Small clusters lose less time between a row's passes, large ones have a row done sooner: as many CTAs as
  // three resident waves take if all rows were left (a share of them is).
  const int sms = sm_count();
  int cluster = 1;
  while (cluster < kMaxCluster && pieces > (int64_t)cluster * T && (!CUT || a.rows * cluster < 3 * sms)) cluster *= 2;
  return launch_clusters(sample_exact_kernel<In, CUT, T, RESIDENT>, a, cluster,
                         std::min<int64_t>(a.rows, std::max(1, RESIDENT * sms / cluster)), T, stream);
}

}  // namespace

cudaError_t launch_sample_exact(const SampleArgs& a, bool fp32, bool cut, cudaStream_t stream) {
  if (cut) return fp32 ? launch_exact<float, true, 512, 1>(a, stream) : launch_exact<uint16_t, true, 512, 1>(a, stream);
  return fp32 ? launch_exact<float, false, 256, 4>(a, stream) : launch_exact<uint16_t, false, 256, 4>(a, stream);
}

}  // namespace sampling
}  // namespace fp8rl
