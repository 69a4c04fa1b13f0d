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
// stands if u W is further from both its borders than the sums can be wrong.  Where something
// is cut off, the thread maxima give a bound below which nothing is kept (the k-th
// largest; or so many of the largest that their masses alone reach p S), the few
// elements above it are collected, sorted, weighed exactly, cut and drawn from.  A row
// that cannot be decided so (a draw on a border, more elements than the list
// holds, temperatures or maxima out of range) is marked for
//
// sample_exact_kernel, which follows at once and passes by all other rows.  There
// weights and sums are carried to about 2^-43, as pairs of fp32 numbers: the exponent
// t = (m - x) log2(e) / T as a pair; 2^-t from a table of 2^-(i / 256) and a polynomial
// of the rest, whose first term is a pair too.  The cut of top-k and top-p is found by
// histograms of 1024 bins over the values (counts, or masses as 13-bit fractions of the
// bin's heaviest), refined until the bin with the cut holds one value or at most 256
// elements, which are sorted.
//
// The order of all sums is fixed.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace fp8rl {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;  // of the exact kernel
constexpr int kUnroll = 2;
constexpr int kBins = 1024;
constexpr int kBinades = 12;                           // of bf16 values that have bins of their own
constexpr int kValues = 2 * 128 * kBinades + 2;        // (+ the ones nearer to 0, + the ones below)
constexpr int kList = 256;  // elements that are sorted, at most one a thread
static_assert(kList <= kThreads && kBins % kThreads == 0, "threads take list entries and bins by their number");
constexpr int kMaxCluster = 8;
constexpr float kReach = 100.0f;  // weights below 2^-100 count as 0
constexpr int32_t kUndecided = -2;  // the token of a row that is left to the exact kernel

// ------------------------------------------------------------------ weights

// 2^-(i / 256) as pairs of fp32 numbers (the exponential's series; |y| < 0.7)
struct Exp2Table {
  float2 v[256];
};
constexpr Exp2Table make_table() {
  Exp2Table t{};
  for (int i = 0; i < 256; ++i) {
    const double y = -0.69314718055994530942 * i / 256;
    double sum = 1.0, term = 1.0;
    for (int n = 1; n < 30; ++n) {
      term *= y / n;
      sum += term;
    }
    const float hi = (float)sum;
    t.v[i].x = hi;
    t.v[i].y = (float)(sum - (double)hi);
  }
  return t;
}
__device__ const Exp2Table kExp2 = make_table();

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return pair_of(v, v); }

// A number as a pair of fp32 numbers, about 48 bits
struct Pair {
  float h = 0.0f, l = 0.0f;
};
__device__ __forceinline__ Pair normal(float h, float l) {  // |h| >= |l|
  const float s = h + l;
  return Pair{s, l - (s - h)};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float s = a.h + b.h, t = s - a.h;
  return normal(s, (a.h - (s - t)) + (b.h - t) + (a.l + b.l));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.h, -b.l}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);  // (not to be joined with the sum)
  return normal(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h));
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }
__device__ __forceinline__ bool operator<=(Pair a, Pair b) { return !(b < a); }
__device__ __forceinline__ Pair pair_from(double v) {
  const float h = (float)v;
  return Pair{h, (float)(v - (double)h)};
}
__device__ __forceinline__ Pair pair_from(uint32_t n) {  // n < 2^31
  const float h = (float)n;
  return Pair{h, (float)((int32_t)n - (int32_t)h)};
}
__device__ __forceinline__ Pair shuffle_up(Pair a, int d) {
  return Pair{__shfl_up_sync(0xffffffffu, a.h, d), __shfl_up_sync(0xffffffffu, a.l, d)};
}
__device__ __forceinline__ Pair shuffle(Pair a, int lane) {
  return Pair{__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}
// the sum over the lanes up to and with this one
__device__ __forceinline__ Pair scan_lanes(Pair a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Pair o = shuffle_up(a, d);
    if (lane >= d) a = o + a;
  }
  return a;
}
// ln of a sum of at least 1
__device__ __forceinline__ float log_of(Pair s) { return s.h < 2.0f ? log1pf((s.h - 1.0f) + s.l) : logf(s.h); }

// what a row's weights go by
struct Scale {
  float m;       // the maximum
  float hi, lo;  // log2(e) / T as a pair
  float cut;     // elements below have weight 0
};

__device__ __forceinline__ Scale scale_of(float m, float temperature) {
  constexpr float kLow = 1.92596299e-8f;  // log2(e) = kLog2e + kLow
  Scale s;
  s.m = m;
  s.hi = __fdiv_rn(kLog2e, temperature);
  s.lo = __fdiv_rn(fmaf(-s.hi, temperature, kLog2e) + kLow, temperature);
  s.cut = fmaxf(m - kReach * kLn2 * temperature, -FLT_MAX);
  return s;
}

// The weights of two elements, each hi + lo.  With d = m - x (exact as a pair) and t = d c
// (a pair), k = round(256 t) and the rest r: 2^-t = 2^-(k >> 8) 2^-((k & 255) / 256) e^g,
// g = -r ln 2, |g| < 0.0014.  e^g - 1 = g + g^2 (1/2 + g/6) with g a pair: the
// terms left out are below 2^-42.
__device__ __forceinline__ void weights(const Scale& s, const float2* table, float x0, float x1, uint64_t& h, uint64_t& l) {
  constexpr float kMagic = 49152.0f, kL2 = 0.693147182464599609375f, kL2Lo = -1.90465429995776804e-9f;
  const uint64_t m = both(s.m), x = pair_of(fmaxf(x0, s.cut), fmaxf(x1, s.cut));
  const uint64_t d = sub2(m, x), b = sub2(d, m);
  const uint64_t e = sub2(sub2(m, sub2(d, b)), add2(x, b));  // d + e = m - x
  const uint64_t nt = pair_mul(d, both(-s.hi));
  uint64_t tl = pair_fma(d, both(s.hi), nt);
  tl = pair_fma(d, both(s.lo), tl);
  tl = pair_fma(e, both(s.hi), tl);
  const uint64_t z = sub2(both(kMagic), nt);             // 256 t rounded, in its low bits
  const uint64_t nr = add2(nt, sub2(z, both(kMagic)));   // exact
  const uint64_t g = pair_mul(nr, both(kL2)), ng = pair_mul(nr, both(-kL2));
  uint64_t gl = pair_fma(nr, both(kL2), ng);
  gl = pair_fma(nr, both(kL2Lo), gl);
  gl = pair_fma(tl, both(-kL2), gl);
  const uint64_t q = pair_fma(pair_mul(g, g), pair_fma(g, both(1.0f / 6.0f), both(0.5f)), gl);
  float z0, z1;
  ptx::f32x2_unpack(z, z0, z1);
  const int32_t k0 = __float_as_int(z0) - 0x47400000, k1 = __float_as_int(z1) - 0x47400000;
  const float2 t0 = table[k0 & 255], t1 = table[k1 & 255];
  const uint64_t th = pair_of(t0.x, t1.x);
  const uint64_t p = pair_mul(th, g), np = pair_mul(th, ng);
  uint64_t lo = add2(pair_of(t0.y, t1.y), pair_fma(th, g, np));
  lo = pair_fma(th, q, lo);
  const uint64_t hi = add2(th, p);
  lo = add2(sub2(p, sub2(hi, th)), lo);
  const uint64_t by = pair_of(x0 >= s.cut ? __int_as_float((127 - (k0 >> 8)) << 23) : 0.0f,
                              x1 >= s.cut ? __int_as_float((127 - (k1 >> 8)) << 23) : 0.0f);
  h = pair_mul(hi, by);
  l = pair_mul(lo, by);
}

// a running sum of pairs, in two halves
struct Sum {
  uint64_t h = 0, l = 0;
  __device__ __forceinline__ void add(uint64_t vh, uint64_t vl) {
    const uint64_t s = add2(h, vh), b = sub2(s, h);
    const uint64_t e = add2(sub2(h, sub2(s, b)), sub2(vh, b));
    h = s;
    l = add2(l, add2(e, vl));
  }
  __device__ __forceinline__ Pair value() const {
    float a, b, c, d;
    ptx::f32x2_unpack(h, a, b);
    ptx::f32x2_unpack(l, c, d);
    return normal(a, c) + normal(b, d);
  }
};

// ------------------------------------------------------------------ the row's cluster

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

struct Shared {
  float2 table[256];
  uint32_t hist[(kValues + 3) / 4 * 4];
  uint64_t list[kList], sorted[kList];
  Pair mass[kList];
  Part warp[kWarps];       // the last gather's sums of this CTA's warps
  Part mine[2];            // of this CTA, read by the others (two take turns)
  Part all[kMaxCluster];   // of every CTA
  Pair part[kWarps];
  float border;            // min-p's
  int32_t n_list, bin, last;
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

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as 0
  return b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) { return __uint_as_float(o ^ ((int32_t)o < 0 ? 0x80000000u : 0xffffffffu)); }

template <typename In>
struct Team {
  static constexpr int N = Row<In>::N;
  Shared& sh;
  const Row<In> row;
  uint32_t rank, ranks;
  int32_t w0, w1;  // this warp's pieces
  int lane, warp;
  int turn = 0;

  __device__ __forceinline__ Team(Shared& s, const In* x, int32_t vocab, uint32_t r, uint32_t rs)
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

  // f(values, index of the first) of the pieces [a, b), lane by lane; elements of no piece are -inf
  template <typename F>
  __device__ __forceinline__ void each(int32_t a, int32_t b, F f) const {
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
      ptx::cluster_sync();
      if (threadIdx.x < ranks * 8) {
        const uint32_t r = threadIdx.x >> 3, w = threadIdx.x & 7;
        reinterpret_cast<uint32_t*>(&sh.all[r])[w] = ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.mine[turn]), r) + 4 * w);
      }
      turn ^= 1;
    }
    __syncthreads();
    Part t = sh.all[0];
    for (uint32_t r = 1; r < ranks; ++r) t = merge(t, sh.all[r]);
    return t;
  }

  // mass and number of the kept elements of the pieces [a, b), this lane's part
  __device__ Part mass(const Scale& s, const Keep& keep, int32_t a, int32_t b) const {
    Sum sum;
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
    });
    Part p;
    p.a = sum.value();
    p.n = n;
    return p;
  }

  // The same of this warp's pieces, a contiguous run of them for each lane
  __device__ __forceinline__ int32_t run() const { return (w1 - w0 + 31) / 32; }
  __device__ Part mass_of_run(const Scale& s, const Keep& keep) const {
    Sum sum;
    uint32_t n = 0;
    const int32_t a = w0 + lane * run();
    for (int32_t i = 0; i < run(); ++i) {
      const int32_t j0 = (a + i) * N - row.off;
      float v[N];
      values<In>(a + i < w1 ? row.load(a + i) : absent<In>(), v);
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
      if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        uint64_t h, l;
        weights(s, sh.table, v[e], v[e + 1], h, l);
        sum.add(h, l);
      }
    }
    Part p;
    p.a = sum.value();
    p.n = n;
    return p;
  }

  // Top-k and top-p of bf16 rows by the values themselves: every value in 12 binades has a bin that
  // counts it, so a bin's mass is its count times one weight and a cut needs no second look.
  // False where a cut falls among the values nearer to 0 than that (or far below): nothing is changed then.
  __device__ bool by_value(const Scale& s, Keep& keep, uint32_t k, float top_p, Pair& total) {
    constexpr int kEach = (kValues + kThreads - 1) / kThreads, kTiny = 128 * kBinades, kRest = kValues - 1;
    // the binades below the largest magnitude that matters
    const float far = fmaxf(fabsf(s.m), s.hi > 0.0f ? 64.0f / s.hi - s.m : 0.0f);
    const int32_t lowest = max(0, (int32_t)((__float_as_uint(fminf(far, FLT_MAX)) >> 23) - (kBinades - 1))) << 7;  // its upper 16 bits
    auto place = [&](float x) {
      const uint32_t b = __float_as_uint(x) >> 16;
      const int32_t g = (int32_t)(b & 0x7FFFu) - lowest;  // magnitudes in steps of bf16
      if (g < 0 || (b & 0x7FFFu) == 0) return kTiny;  // (zeros of both signs together)
      if (b >> 15) return g < kTiny ? kTiny + 1 + g : kRest;
      return kTiny - 1 - g;  // (no value is above the maximum's binade)
    };
    auto value_at = [&](int b) {
      const uint32_t g = (uint32_t)(b < kTiny ? kTiny - 1 - b : b - kTiny - 1) + (uint32_t)lowest;
      return __uint_as_float((b < kTiny ? g : g | 0x8000u) << 16);
    };
    for (int i = threadIdx.x; i < kValues; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    each(w0, w1, [&](float (&v)[N], int32_t) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (v[e] > -INFINITY) atomicAdd(&sh.hist[place(v[e])], 1u);
    });
    if (ranks > 1) ptx::cluster_sync();
    else __syncthreads();
    uint32_t count[kEach], n_own = 0;
    Pair mass[kEach], own;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int b = threadIdx.x * kEach + i;
      count[i] = 0;
      if (b < kValues)
        for (uint32_t r = 0; r < ranks; ++r) count[i] += ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.hist[b]), r));
      mass[i] = Pair{};
      if (count[i] > 0 && b != kTiny && b != kRest) {
        uint64_t h, l;
        weights(s, sh.table, value_at(b), -INFINITY, h, l);
        float h0, l0, none;
        ptx::f32x2_unpack(h, h0, none);
        ptx::f32x2_unpack(l, l0, none);
        mass[i] = normal(h0, l0) * pair_from(count[i]);
      }
      n_own += count[i];
    }
    // the tiny ones' mass, exactly
    Part tiny;
    each(w0, w1, [&](float (&v)[N], int32_t) {
      bool any = false;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (v[e] > -INFINITY && place(v[e]) == kTiny) any = true;
        else v[e] = -INFINITY;
      }
      if (!__any_sync(0xffffffffu, any)) return;
      Sum sum;
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        uint64_t h, l;
        weights(s, sh.table, v[e], v[e + 1], h, l);
        sum.add(h, l);
      }
      tiny.a = tiny.a + sum.value();
    });
    tiny = gather(tiny);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (threadIdx.x * kEach + i == kTiny) mass[i] = tiny.a;
      own = own + mass[i];
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
      sh.warp[warp].k = n_run;
    }
    run = shuffle_up(run, 1);
    if (lane == 0) run = Pair{};
    n_run -= n_own;
    __syncthreads();
    Pair all;
    uint32_t finite = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        run = all + run;
        n_run += finite;
      }
      all = all + sh.part[w];
      finite += sh.warp[w].k;
    }
    total = all;
    // (a bin, and how many of it are kept)
    int bin = -1;
    uint32_t need = 0, have = 0;
    auto found = [&](auto reached) {  // the first bin at whose end `reached` holds; every thread hears of it
      if (threadIdx.x == 0) sh.bin = INT_MAX;
      __syncthreads();
      uint32_t n = n_run;
      Pair m = run;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (count[i] == 0) continue;
        n += count[i];
        m = m + mass[i];
        if (reached(n, m)) {
          atomicMin(&sh.bin, (int)threadIdx.x * kEach + i);
          break;
        }
      }
      __syncthreads();
      const int b = sh.bin;
      if (b / kEach == (int)threadIdx.x) {
        n = n_run;
        m = run;
        for (int i = 0; i < b % kEach; ++i) {
          n += count[i];
          m = m + mass[i];
        }
        sh.ahead = n;
        sh.ahead_mass = m;
        sh.last = (int)count[b % kEach];
      }
      __syncthreads();
      return b;
    };
    Pair mass_k = all;
    if (k > 0) {
      bin = found([&](uint32_t n, Pair) { return n >= k; });
      if (bin == kTiny || bin == kRest) return false;
      need = k - sh.ahead;
      have = (uint32_t)sh.last;
      uint64_t h, l;
      weights(s, sh.table, value_at(bin), -INFINITY, h, l);
      float h0, l0, none;
      ptx::f32x2_unpack(h, h0, none);
      ptx::f32x2_unpack(l, l0, none);
      mass_k = sh.ahead_mass + normal(h0, l0) * pair_from(need);
    }
    if (top_p < 1.0f) {
      const Pair target = Pair{top_p, 0.0f} * mass_k;
      const int b = found([&](uint32_t, Pair m) { return target <= m; });
      if (b == kTiny || b == kRest) return false;
      if (b < kValues && (bin < 0 || b <= bin)) {  // (no bin: rounding; all of them, or the first k)
        const uint32_t most = b == bin ? need : (uint32_t)sh.last;
        uint64_t h, l;
        weights(s, sh.table, value_at(b), -INFINITY, h, l);
        float h0, l0, none;
        ptx::f32x2_unpack(h, h0, none);
        ptx::f32x2_unpack(l, l0, none);
        need = first_reaching(target - sh.ahead_mass, normal(h0, l0), most);
        bin = b;
        have = (uint32_t)sh.last;
      }
    }
    if (bin < 0) return true;
    keep.x = value_at(bin);
    keep.j = need >= have ? INT_MAX : nth_equal(keep.x, keep, need);
    return true;
  }

  // the smallest n in [1, most] with n w >= left
  static __device__ uint32_t first_reaching(Pair left, Pair w, uint32_t most) {
    const double a = (double)left.h + (double)left.l, b = (double)w.h + (double)w.l;
    const double n = b > 0.0 ? ceil(a / b) : 1.0;
    uint32_t need = (uint32_t)fmin(fmax(n, 1.0), (double)most);
    if (need > 1 && (double)(need - 1) * b >= a) --need;
    return need;
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
    for (;;) {
      auto place = [&](float x, int32_t j, float& f) {  // the bin, or -1
        if (!(x <= hi && x >= lo && keep(x, j))) return -1;
        f = (hi - x) * pre * scale;
        return f < (float)(kBins - 1) ? (int)f : kBins - 1;
      };
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
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
          const uint32_t q = by_count ? 1u : (uint32_t)(ex2(fmaxf(((float)b - f) * step, -64.0f)) * 8192.0f);
          if (q) atomicAdd(&sh.hist[b], q);
        }
      });
      if (ranks > 1) ptx::cluster_sync();
      else __syncthreads();
      // the cluster's bins, some a thread
      constexpr int kEach = kBins / kThreads;
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
      // (the masses are up to 2^-13 small: as shares of their own sum, head and tail are good to that)
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
        Sum sa, sb;
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
          uint64_t h, l;  // the first n with above + n w >= target
          weights(s, sh.table, t.most, -INFINITY, h, l);
          float h0, l0, none;
          ptx::f32x2_unpack(h, h0, none);
          ptx::f32x2_unpack(l, l0, none);
          need = first_reaching(target - above, normal(h0, l0), t.k);
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
      if (ranks > 1) ptx::cluster_sync();
      else __syncthreads();
      int32_t at = 0;
      for (int32_t i = 0; i < n; ++i) at += sh.sorted[i] > key;
      __syncthreads();
      if ((int32_t)threadIdx.x < n) sh.list[at] = key;
      __syncthreads();
      int32_t cut = (int32_t)(k - n_above) - 1;
      if (!by_count) {
        if ((int32_t)threadIdx.x < n) {
          uint64_t h, l;
          weights(s, sh.table, from_ordered((uint32_t)(sh.list[threadIdx.x] >> 32)), -INFINITY, h, l);
          float h0, l0, rest;
          ptx::f32x2_unpack(h, h0, rest);
          ptx::f32x2_unpack(l, l0, rest);
          sh.mass[threadIdx.x] = normal(h0, l0);
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

struct SampleArgs {
  const void* x;
  const float *temperature, *top_p, *min_p;  // of every row, or null
  const int32_t* top_k;
  const double* uniform;
  int32_t* tokens;
  float *lp, *lp_kept;
  int32_t* kept;
  int64_t ld, rows, k;
  float t, p, q;  // for all rows
  int32_t vocab;
  uint32_t* err;  // debug builds' store checks
};

__device__ __forceinline__ void report(const SampleArgs& a, int64_t r, int32_t token, float lp, float lp_kept, int32_t kept) {
  if (!dcheck(r < a.rows, a.err)) return;
  a.tokens[r] = token;
  if (a.lp) a.lp[r] = lp;
  if (a.lp_kept) a.lp_kept[r] = lp_kept;
  if (a.kept) a.kept[r] = kept;
}

// what one row is drawn with; false: no draw
struct Draw {
  double u;
  float temperature, top_p, min_p;
  int64_t k;
  __device__ __forceinline__ bool load(const SampleArgs& a, int64_t r) {
    u = a.uniform[r];
    temperature = a.temperature ? a.temperature[r] : a.t;
    top_p = a.top_p ? a.top_p[r] : a.p;
    min_p = a.min_p ? a.min_p[r] : a.q;
    k = a.top_k ? a.top_k[r] : a.k;
    if (!(u >= 0.0 && u < 1.0) || !(temperature >= 0.0f && temperature <= FLT_MAX) || isnan(top_p) || isnan(min_p)) return false;
    if (temperature == 0.0f) {
      temperature = 1.0f;
      k = 1;
    }
    if (top_p <= 0.0f) k = 1;
    temperature = fminf(fmaxf(temperature, 1e-30f), 1e30f);
    return true;
  }
  // T ln(min_p), and the smallest kept value
  __device__ __forceinline__ double reach() const { return (double)temperature * log((double)fminf(min_p, 1.0f)); }
};
__device__ __forceinline__ float border_of(float m, double reach) { return __double2float_ru((double)m + reach); }

// ------------------------------------------------------------------ one pass

constexpr int kCap = 1024;    // elements that a row's cut is made among
constexpr int kMassBins = 128;  // of the thread maxima, a quarter of a power of two each
constexpr float kStep = 0x1p-24f;  // an fp32 operation's largest relative error

// a warp's share of a row: sums against its maximum m
struct WarpStat {
  float m;
  Pair s;            // sum of w
  float err, wt;     // a bound of s's error so far; sum of w t (t <= 0: exponents in base 2)
  uint32_t masked;   // elements of -inf
  uint32_t pad[2];
};
static_assert(sizeof(WarpStat) == 32, "read as 8 words");

template <bool CUT, int T>
struct PassShared {
  WarpStat warp[T / 32];
  float bound;             // of this CTA's share: at least its part of the first k lies at or above
  // of the whole row, after the pass
  Pair total, left;
  float m, err, tau;
  uint32_t finite;
  int owner, owner_warp;
  Pair part[T / 32];
};
template <int T>
struct CutShared {
  float2 table[256];
  float most[T];           // thread maxima
  uint32_t bins[kMassBins];
  uint64_t list[kCap];     // this CTA's finds
  uint64_t key[kCap];      // rank 0: all of them, sorted
  Pair w[kCap];
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

// The draw from a list of at most one element a thread (rank 0's cs.key, in any order): `n_k` of them are the
// first k, `exact`: the list's masses are what top_p goes by (else the sum, known to err).
template <int T>
__device__ void draw_from_few(const SampleArgs& a, int64_t r, CutShared<T>& cs, const Draw& draw, const Scale& s, int n, int n_k,
                              bool by_p, bool exact, Pair total, float err, float border) {
  const int tid = threadIdx.x;
  if (tid == 0 && (n & 1)) cs.key[n] = 0;
  __syncthreads();
  // by value: each counts the ones ahead of it
  const uint64_t mine = tid < n ? cs.key[tid] : 0;
  int place = 0;
  for (int i = 0; i < n; i += 2) {
    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&cs.key[i]);
    place += (two.x > mine) + (two.y > mine);
  }
  if (tid < n) cs.list[place] = mine;
  __syncthreads();
  const uint64_t key = tid < n ? cs.list[tid] : 0;
  const float x = from_ordered((uint32_t)(key >> 32));
  Pair w;
  if (tid < n) {
    uint64_t h, l;
    weights(s, cs.table, x, -INFINITY, h, l);
    float h0, l0, none;
    ptx::f32x2_unpack(h, h0, none);
    ptx::f32x2_unpack(l, l0, none);
    w = normal(h0, l0);
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
      if (tid == 0) report(a, r, kUndecided, 0.0f, 0.0f, 0);
      return;
    }
    n_kept = n_low + 1;
  }
  n_kept = min(n_kept, __syncthreads_count(tid < n && x >= border));
  // in the row's order
  const bool kept = tid < n_kept;
  place = 0;
  for (int i = 0; i < n_kept; ++i) place += (uint32_t)cs.list[i] > (uint32_t)key;  // (low words: ~index)
  if (kept) {
    cs.w[place] = w;
    cs.key[place] = key;
  }
  __syncthreads();
  w = kept ? cs.w[tid] : Pair{};
  Pair mass;
  const Pair with = block_sums<T>(w, cs.part, mass);
  const Pair goal = pair_from(draw.u) * mass;
  // the last one with a mass whose predecessors' mass is at most u W
  if (kept && w.h > 0.0f && with - w <= goal) atomicMax(&cs.token, tid);
  __syncthreads();
  if (tid == 0) {
    const uint64_t won = cs.key[max(cs.token, 0)];
    const float y = (from_ordered((uint32_t)(won >> 32)) - s.m) / draw.temperature;
    report(a, r, (int32_t) ~(uint32_t)won, y - log_of(total), y - log_of(mass), n_kept);
  }
}

// grid (cluster, rows)
template <typename In, bool CUT, int T>
__global__ void __launch_bounds__(T) sample_kernel(const SampleArgs a) {
  constexpr int N = Row<In>::N, U = 4, W = T / 32;
  __shared__ __align__(16) unsigned char smem[sizeof(PassShared<CUT, T>)];
  __shared__ __align__(16) unsigned char cut_smem[CUT ? sizeof(CutShared<T>) : 16];
  auto& sh = *reinterpret_cast<PassShared<CUT, T>*>(smem);
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
  float m = -INFINITY, err = 0.0f, wt = 0.0f;
  Sum sum;
  uint64_t wt2 = 0;
  uint32_t masked = 0;
  const uint64_t c2 = both(c);
  for (int32_t p0 = w0; p0 < w1; p0 += 32 * U) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = p0 + 32 * i + lane < w1 ? row.load(p0 + 32 * i + lane) : absent<In>();
    const float big = largest<In>(u);
    if (big > m) {
      // (all sums so far times a power: one rounding of the exponential and of the product)
      const float d = m == -INFINITY ? 0.0f : fmaxf((m - big) * c, kTinyExp2), f = m == -INFINITY ? 0.0f : ex2(d);
      float h0, h1, l0, l1;
      ptx::f32x2_unpack(sum.h, h0, h1);
      ptx::f32x2_unpack(sum.l, l0, l1);
      float t0, t1;
      ptx::f32x2_unpack(wt2, t0, t1);
      wt = f * fmaf(d, h0 + h1, wt + t0 + t1);
      wt2 = 0;
      err = f * fmaf(6.0f * kStep, h0 + h1, err);
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
      if (m > -INFINITY) err = INFINITY;
    }
    // elements of -inf, where there are any
    bool any = false;
#pragma unroll
    for (int i = 0; i < U; ++i) any |= least_is_masked<In>(u[i]);
    if (any) {
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
    wt = f * fmaf(d, s.h, wt);
    err = f * fmaf(16.0f * kStep, s.h, err);  // this exponential, those of the sum and the additions
    s = Pair{s.h * f, s.l * f};
    s = scan_lanes(s);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      err += __shfl_xor_sync(0xffffffffu, err, k);
      wt += __shfl_xor_sync(0xffffffffu, wt, k);
    }
    masked = __reduce_add_sync(0xffffffffu, masked);
    if (lane == 31) sh.warp[warp] = WarpStat{m, s, err, wt, masked, {}};
  }
  const bool by_rank = CUT && draw.k > 0 && draw.k <= kCap;
  if (CUT) {
    // Each CTA gives the first ceil(k / CTAs) of its threads' maxima; the least of these bounds is one of the
    // k-th largest element.  The upper half of the ordered number: a lower bound.
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
  if (ranks > 1) ptx::cluster_sync();
  else __syncthreads();

  // the row's sums, in every CTA: lane i has the shares 2 i and 2 i + 1
  if (warp == 0) {
    WarpStat st[2];
    float tau = INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * lane + i;
      st[i] = WarpStat{-INFINITY, {}, 0.0f, 0.0f, 0, {}};
      if (e < ranks * W) {
        const uint32_t at = ptx::mapa_shared(ptx::smem_u32(&sh.warp[e % W]), e / W);
        const float4 x = ptx::ld_dsmem_f32x4(at), y = ptx::ld_dsmem_f32x4(at + 16);
        st[i] = WarpStat{x.x, {x.y, x.z}, x.w, y.x, __float_as_uint(y.y), {}};
      }
    }
    if (CUT && lane < ranks) tau = __uint_as_float(ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&sh.bound), lane)));
    float top = fmaxf(st[0].m, st[1].m);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      tau = fminf(tau, __shfl_xor_sync(0xffffffffu, tau, d));
    }
    err = wt = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float d = st[i].m == -INFINITY ? 0.0f : fmaxf((st[i].m - top) * c, kTinyExp2), f = st[i].m == -INFINITY ? 0.0f : ex2(d);
      wt += f * fmaf(d, st[i].s.h, st[i].wt);
      err += f * fmaf(6.0f * kStep, st[i].s.h, st[i].err);
      st[i].s = Pair{st[i].s.h * f, st[i].s.l * f};
    }
    masked = __reduce_add_sync(0xffffffffu, st[0].masked + st[1].masked);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      err += __shfl_xor_sync(0xffffffffu, err, k);
      wt += __shfl_xor_sync(0xffffffffu, wt, k);
    }
    const Pair incl = scan_lanes(st[0].s + st[1].s), total = shuffle(incl, 31);
    // exponents: x - m, log2(e) / T and their product are rounded
    err = fmaf(2.6f * kStep, fabsf(wt), err);
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
    at = __shfl_sync(0xffffffffu, at, from);
    start = shuffle(start, from);
    if (lane == 0) {
      sh.total = total;
      sh.left = goal - start;
      sh.m = top;
      sh.err = err;
      sh.tau = tau;
      sh.finite = (uint32_t)a.vocab - masked;
      sh.owner = at < 0 ? 0 : at / W;
      sh.owner_warp = at < 0 ? 0 : at % W;
    }
  }
  __syncthreads();
  const Pair total = sh.total;
  m = sh.m;
  err = sh.err;
  const uint32_t finite = sh.finite;
  const int64_t k = draw.k;
  const bool by_k = CUT && k > 0 && k < (int64_t)finite, by_p = CUT && draw.top_p < 1.0f && draw.top_p > 0.0f,
             by_q = CUT && draw.min_p > 0.0f;
  const bool odd = isnan(total.h) || !(fabsf(m) <= limit);  // NaN, infinities, -inf alone, out of range
  if (odd) {
    if (rank == 0 && tid == 0) {
      if (isnan(total.h) || m == INFINITY) report(a, r, -1, NAN, NAN, 0);
      else if (m == -INFINITY) report(a, r, -1, -INFINITY, -INFINITY, 0);
      else report(a, r, kUndecided, 0.0f, 0.0f, 0);
    }
  } else if (!by_k && !by_p && !by_q) {
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
          // both the sum ahead of the token and u W may be off by err, the last steps' by theirs
          const float margin = fmaf(2.0f, err, 24.0f * kStep * total.h);
          if (under >= margin && over >= margin) {
            const float y = (x - m) / draw.temperature, lp = y - log_of(total);
            report(a, r, token, lp, lp, (int32_t)finite);
          } else {
            report(a, r, kUndecided, 0.0f, 0.0f, 0);
          }
        }
      }
    }
  } else if (CUT) {
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
          if (at < kCap) cs.list[at] = (uint64_t)ordered(v[e]) << 32 | (uint32_t) ~(p * N - row.off + e);
        }
      }
    }
    if (ranks > 1) ptx::cluster_sync();
    else __syncthreads();
    if (rank == 0) {
      int n = 0;
      bool whole = possible;
      for (int q = 0; q < ranks; ++q) {
        const int h = (int)ptx::ld_dsmem_u32(ptx::mapa_shared(ptx::smem_u32(&cs.hits), q));
        if (n + h <= kCap && h <= kCap) {
          for (int i = tid; i < h; i += T) {
            const uint32_t at = ptx::mapa_shared(ptx::smem_u32(&cs.list[i]), q);
            cs.key[n + i] = (uint64_t)ptx::ld_dsmem_u32(at + 4) << 32 | ptx::ld_dsmem_u32(at);
          }
          n += h;
        } else {
          whole = false;
        }
      }
      if (!whole || n < 1) {
        if (tid == 0) report(a, r, kUndecided, 0.0f, 0.0f, 0);
      } else {
        const Scale s = scale_of(m, draw.temperature);
        if (n <= T) {
          draw_from_few<T>(a, r, cs, draw, s, n, by_k ? (int)min((int64_t)n, k) : n, by_p, by_k || n == (int)finite, total, err, border);
        } else {
        int n2 = 2;
        while (n2 < n) n2 *= 2;
        for (int i = n + tid; i < n2; i += T) cs.key[i] = 0;
        sort_down<T>(cs.key, n2);
        for (int i = tid; i < n; i += T) {
          uint64_t h, l;
          float h0, l0, none;
          const float x = from_ordered((uint32_t)(cs.key[i] >> 32));
          weights(s, cs.table, x, -INFINITY, h, l);
          ptx::f32x2_unpack(h, h0, none);
          ptx::f32x2_unpack(l, l0, none);
          cs.w[i] = normal(h0, l0);
          if (x >= border) atomicAdd(&cs.n_border, 1);
        }
        __syncthreads();
        const int n_k = by_k ? (int)min((int64_t)n, k) : n;
        int n_kept = n_k;
        bool sure = true;
        if (by_p) {
          // how many sums lie below top_p's share (of the sum known to err: below its least and its largest)
          Pair low = total + Pair{-err, 0.0f}, high = total + Pair{err, 0.0f};
          if (by_k || n == (int)finite) low = high = sums_of<T>(cs.w, n_k, cs.part, [](int, Pair, Pair) {});
          const Pair p{draw.top_p, 0.0f};
          low = p * low;
          high = p * high;
          sums_of<T>(cs.w, n_k, cs.part, [&](int, Pair, Pair with) {
            if (with < low) atomicAdd(&cs.below[0], 1);
            if (with < high) atomicAdd(&cs.below[1], 1);
          });
          __syncthreads();
          sure = cs.below[0] == cs.below[1] && cs.below[1] < n_k;
          n_kept = min(n_kept, cs.below[0] + 1);
        }
        n_kept = min(n_kept, cs.n_border);
        if (!sure) {
          if (tid == 0) report(a, r, kUndecided, 0.0f, 0.0f, 0);
        } else {
          // the kept ones in the row's order, with their place among the sorted
          n2 = 2;
          while (n2 < n_kept) n2 *= 2;
          for (int i = tid; i < n2; i += T) cs.list[i] = i < n_kept ? cs.key[i] << 32 | (uint32_t)i : 0;
          sort_down<T>(cs.list, n2);
          // (sorted keys low words are ~index: the largest first is the lowest index first)
          const Pair mass = sums_of<T>(cs.w, n_kept, cs.part, [](int, Pair, Pair) {});
          constexpr int E = kCap / T;
          Pair w[E];
#pragma unroll
          for (int i = 0; i < E; ++i) w[i] = tid * E + i < n_kept ? cs.w[(uint32_t)cs.list[tid * E + i]] : Pair{};
          __syncthreads();
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (tid * E + i < n_kept) cs.w[tid * E + i] = w[i];
          __syncthreads();
          const Pair goal = pair_from(draw.u) * mass;
          sums_of<T>(cs.w, n_kept, cs.part, [&](int i, Pair before, Pair) {
            if (cs.w[i].h > 0.0f && before <= goal) atomicMax(&cs.token, i);
          });
          __syncthreads();
          if (tid == 0) {
            const uint64_t key = cs.list[max(cs.token, 0)];
            const float x = from_ordered((uint32_t)(cs.key[(uint32_t)key] >> 32)), y = (x - m) / draw.temperature;
            report(a, r, (int32_t) ~(uint32_t)(key >> 32), y - log_of(total), y - log_of(mass), n_kept);
          }
        }
        }
      }
    }
  }
  if (ranks > 1) ptx::cluster_sync();  // the others have read this CTA's shared memory
}

// ------------------------------------------------------------------ exact

// grid (cluster, clusters): the rows that the pass has left
template <typename In>
__global__ void __launch_bounds__(kThreads) sample_exact_kernel(const SampleArgs a) {
  __shared__ __align__(16) unsigned char smem[sizeof(Shared)];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  constexpr int N = Row<In>::N;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const uint32_t rank = blockIdx.x, ranks = gridDim.x;
  bool first = true;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    if (__ldcg(a.tokens + r) != kUndecided) continue;
    if (first) {
      for (int i = threadIdx.x; i < 256; i += kThreads) sh.table[i] = kExp2.v[i];
      first = false;
    }
    Draw draw;
    draw.load(a, r);
    Team<In> team(sh, static_cast<const In*>(a.x) + r * a.ld, a.vocab, rank, ranks);
    Part p;
    team.each(team.w0, team.w1, [&](float (&v)[N], int32_t) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        p.most = fmaxf(p.most, v[e]);
        p.n += v[e] > -INFINITY;
      }
    });
    p = team.gather(p);
    const float m = p.most;
    const uint32_t finite = p.n;
    const Scale s = scale_of(m, draw.temperature);
    if (threadIdx.x == 0) sh.border = draw.min_p > 0.0f ? border_of(m, draw.reach()) : -INFINITY;
    __syncthreads();

    // the cut, and the mass of what is kept (and of all)
    Keep keep;
    const bool by_k = draw.k > 0 && draw.k < (int64_t)finite, by_p = draw.top_p < 1.0f && draw.top_p > 0.0f;
    Pair total;
    bool summed = false;
    if (by_k || by_p) {
      summed = sizeof(In) == 2 && team.by_value(s, keep, by_k ? (uint32_t)draw.k : 0, by_p ? draw.top_p : 1.0f, total);
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
    const float border = sh.border;
    if (border > -INFINITY && !summed) {
      total = team.gather(team.mass(s, keep, team.w0, team.w1)).a;
      summed = true;
    }
    keep.border = border;
    p = team.mass_of_run(s, keep);
    const Pair own = p.a;  // of this lane's run
    p = team.gather(p);
    const Pair mass = p.a;
    const int32_t kept = (int32_t)p.n;
    if (!summed) total = mass;

    // the last CTA, warp, lane and element with a mass of its own whose predecessors' mass is at most u W
    Pair left = pair_from(draw.u) * mass;
    auto descend = [&](int n, auto mass_of) {
      int at = 0;
      Pair sum, start;
      for (int i = 0; i < n; ++i) {
        const Pair v = mass_of(i);
        if (v.h > 0.0f && sum <= left) {
          at = i;
          start = sum;
        }
        sum = sum + v;
      }
      left = left - start;
      return at;
    };
    const int owner = descend((int)ranks, [&](int i) { return sh.all[i].a; });
    if (owner == (int)rank && descend(kWarps, [&](int i) { return sh.warp[i].a; }) == team.warp) {
      Pair before = shuffle_up(scan_lanes(own), 1);
      if (team.lane == 0) before = Pair{};
      const uint32_t lanes = __ballot_sync(0xffffffffu, own.h > 0.0f && before <= left);
      const int from = lanes ? 31 - __clz(lanes) : 0;
      left = left - shuffle(before, from);
      // that lane's elements, one a lane
      const int32_t first_j = (team.w0 + from * team.run()) * N - team.row.off, some = team.run() * N;
      int32_t token = -1;
      float x = 0.0f;
      Pair sum;
      for (int32_t e0 = 0; e0 < some && sum <= left; e0 += 32) {
        const int32_t j = first_j + e0 + team.lane;
        float v = -INFINITY;
        if (e0 + team.lane < some && j >= 0 && j < a.vocab) {
          if (sizeof(In) == 2) v = bf16_lo((uint32_t) reinterpret_cast<const uint16_t*>(team.row.x)[j]);
          else v = reinterpret_cast<const float*>(team.row.x)[j];
        }
        uint64_t h, l;
        weights(s, sh.table, keep(v, j) ? v : -INFINITY, -INFINITY, h, l);
        float h0, l0, none;
        ptx::f32x2_unpack(h, h0, none);
        ptx::f32x2_unpack(l, l0, none);
        const Pair w = normal(h0, l0), incl = scan_lanes(w);
        Pair ahead = shuffle_up(incl, 1);
        if (team.lane == 0) ahead = Pair{};
        const uint32_t can = __ballot_sync(0xffffffffu, w.h > 0.0f && sum + ahead <= left);
        if (can) {
          token = __shfl_sync(0xffffffffu, j, 31 - __clz(can));
          x = __shfl_sync(0xffffffffu, v, 31 - __clz(can));
        }
        sum = sum + shuffle(incl, 31);
      }
      if (team.lane == 0) {
        const float y = (x - m) / draw.temperature;
        report(a, r, token, y - log_of(total), y - log_of(mass), kept);
      }
    }
    if (ranks > 1) ptx::cluster_sync();  // the others have read this CTA's shared memory
    else __syncthreads();
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  return n;
}

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

constexpr int64_t kMaxRows = 65535;             // grid y
constexpr int64_t kMaxVocab = (int64_t)1 << 30;  // 32-bit element and piece numbers

template <typename K>
cudaError_t launch(K kernel, const SampleArgs& a, int cluster, int64_t rows, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster, (unsigned)rows);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename In>
cudaError_t launch_sample(const SampleArgs& a, int64_t rows, cudaStream_t stream) {
  const bool cut = a.temperature || a.top_k || a.top_p || a.min_p || a.k > 0 || a.p < 1.0f || a.q > 0.0f || a.t == 0.0f;
  const int64_t pieces = ((int64_t)a.vocab + Row<In>::N - 1) / Row<In>::N;
  cudaError_t e;
  if (pieces <= 256) {
    e = cut ? launch(sample_kernel<In, true, 64>, a, 1, rows, 64, stream) : launch(sample_kernel<In, false, 64>, a, 1, rows, 64, stream);
  } else {
    // few rows are split over a cluster, down to a load round per CTA
    const int64_t want = 7 * (int64_t)sm_count() / 2, round = (int64_t)kThreads * 4;
    int cluster = 1;
    while (cluster < kMaxCluster && rows * cluster < want && pieces > cluster * round) cluster *= 2;
    e = cut ? launch(sample_kernel<In, true, 256>, a, cluster, rows, 256, stream)
            : launch(sample_kernel<In, false, 256>, a, cluster, rows, 256, stream);
  }
  if (e != cudaSuccess) return e;
  int cluster = 1;
  while (cluster < kMaxCluster && pieces > (int64_t)cluster * kThreads * kUnroll) cluster *= 2;
  return launch(sample_exact_kernel<In>, a, cluster, std::min<int64_t>(rows, std::max(1, 2 * sm_count() / cluster)), kThreads, stream);
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

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
