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
// So weights and sums are carried to about 2^-43, as pairs of fp32 numbers: the
// exponent t = (m - x) log2(e) / T as a pair; 2^-t from a table of 2^-(i / 256) and
// a polynomial of the rest, whose first term is a pair too; lanes' sums as pairs,
// everything above them in fp64.  The order of all sums is fixed.
//
// A cluster takes a row, a CTA a contiguous share of it, a warp a contiguous share of
// that, so that sums by place in the row fall out: the token is found by descending
// from CTAs to warps to parts of a warp's share to pieces.  The cut of
// top-k and top-p is found by histograms of 1024 bins over the values (counts, or masses
// as 13-bit fractions of the bin's heaviest), refined until the bin with the cut holds
// one value or at most 256 elements, which are sorted.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace fp8rl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 2;
constexpr int kBins = 1024;
constexpr int kList = 256;  // elements that are sorted, one a thread
constexpr int kMaxCluster = 8;
constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;
constexpr float kReach = 100.0f;  // weights below 2^-100 count as 0

// ------------------------------------------------------------------ weights

// 2^-(i / 256) as pairs of fp32 numbers (the exponential's series; |y| < 0.7)
struct Exp2Table {
  float2 v[256];
};
constexpr Exp2Table make_table() {
  Exp2Table t{};
  for (int i = 0; i < 256; ++i) {
    const double y = -kLn2 * i / 256;
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

// what a row's weights go by
struct Scale {
  float m;       // the maximum
  float hi, lo;  // log2(e) / T as a pair
  float cut;     // elements below have weight 0
};

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
  __device__ __forceinline__ double value() const {
    float a, b, c, d;
    ptx::f32x2_unpack(h, a, b);
    ptx::f32x2_unpack(l, c, d);
    return ((double)a + (double)b) + ((double)c + (double)d);
  }
};

// ------------------------------------------------------------------ the row's cluster

// what threads, warps and CTAs add up: sums, a maximum, a minimum, counts
struct alignas(16) Part {
  double a = 0.0, b = 0.0;
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
    o.a = __shfl_xor_sync(0xffffffffu, v.a, d);
    o.b = __shfl_xor_sync(0xffffffffu, v.b, d);
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
  uint32_t hist[kBins];
  uint64_t list[kList], sorted[kList];
  double mass[kList];
  Part warp[kWarps];       // the last gather's sums of this CTA's warps
  Part mine[2];            // of this CTA, read by the others (two take turns)
  Part all[kMaxCluster];   // of every CTA
  double part[kWarps];
  uint64_t scan[kWarps];
  Scale scale;
  float border;            // min-p's
  int32_t n_list, bin, last;
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
  __device__ void select(const Scale& s, Keep& keep, bool by_count, uint32_t k, double target, double whole) {
    // bins over (hi - x) * pre * scale; a bin is `step` wide in t
    float hi = s.m, lo = -FLT_MAX, pre = 1.0f, scale = 16.0f * s.hi, step = 1.0f / 16.0f;
    double above = 0.0;    // mass and number of what lies above the range
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
      // the cluster's bins, four a thread
      uint32_t c[4] = {0, 0, 0, 0};
      float4 many = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (uint32_t r = 0; r < ranks; ++r) {
        const float4 v = ptx::ld_dsmem_f32x4(ptx::mapa_shared(ptx::smem_u32(&sh.hist[4 * threadIdx.x]), r));
        const uint32_t w[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] += w[i];
        many.x += (float)w[0], many.y += (float)w[1], many.z += (float)w[2], many.w += (float)w[3];
      }
      // the first bin in which the running sum reaches what is asked for (masses: nearly)
      const float t0 = (s.m - hi) * s.hi;
      float f[4] = {many.x, many.y, many.z, many.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] *= ex2(fmaxf(-t0 - (float)(4 * threadIdx.x + i) * step, -120.0f)) * (1.0f / 8192.0f);
      double own = by_count ? (double)c[0] + c[1] + c[2] + c[3] : (double)f[0] + f[1] + f[2] + f[3], run = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
      }
      if (lane == 31) sh.part[warp] = run;
      __syncthreads();
      run -= own;
      double sum = 0.0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) run += sh.part[w];
        sum += sh.part[w];
      }
      // (the masses are up to 2^-13 small: as shares of their own sum, head and tail are good to that)
      const double want = by_count ? (double)(k - n_above) : (target - above) / whole * sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c[i] == 0) continue;
        const int b = 4 * threadIdx.x + i;
        atomicMax(&sh.last, b);
        run += by_count ? (double)c[i] : (double)f[i];
        if (run >= want) atomicMin(&sh.bin, b);
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
        const bool below = above + t.a >= target && t.n > 0;
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
      above += t.a;
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
          const double w = t.b / t.k;
          double n = w > 0.0 ? ceil((target - above) / w) : 1.0;
          n = fmin(fmax(n, 1.0), (double)t.k);
          if (n > 1.0 && above + (n - 1.0) * w >= target) n -= 1.0;
          need = (uint32_t)n;
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
          sh.mass[threadIdx.x] = (double)h0 + (double)l0;
        } else {
          sh.mass[threadIdx.x] = 0.0;
        }
        if (threadIdx.x == 0) sh.bin = n - 1;
        __syncthreads();
        if (warp == 0) {
          constexpr int kEach = kList / 32;
          double sum = 0.0;
          for (int i = 0; i < kEach; ++i) sum += sh.mass[lane * kEach + i];
          double incl = sum;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
          }
          double part = above + (incl - sum);
          for (int i = 0; i < kEach; ++i) {
            part += sh.mass[lane * kEach + i];
            if (part >= target) {
              atomicMin(&sh.bin, lane * kEach + i);
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

// ln of a sum of at least 1
__device__ __forceinline__ float log_of(double s) { return s < 2.0 ? log1pf((float)(s - 1.0)) : logf((float)s); }

// grid (cluster, rows)
template <typename In>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  __shared__ __align__(16) unsigned char smem[sizeof(Shared)];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  constexpr int N = Row<In>::N;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int64_t r = blockIdx.y;
  const uint32_t rank = blockIdx.x, ranks = gridDim.x;
  const double u = a.uniform[r];
  float temperature = a.temperature ? a.temperature[r] : a.t;
  float top_p = a.top_p ? a.top_p[r] : a.p, min_p = a.min_p ? a.min_p[r] : a.q;
  int64_t k = a.top_k ? a.top_k[r] : a.k;
  // no draw for this row: the whole cluster leaves
  if (!(u >= 0.0 && u < 1.0) || !(temperature >= 0.0f && temperature <= FLT_MAX) || isnan(top_p) || isnan(min_p)) {
    if (rank == 0 && threadIdx.x == 0) report(a, r, -1, 0.0f, 0.0f, 0);
    return;
  }
  if (temperature == 0.0f) {
    temperature = 1.0f;
    k = 1;
  }
  if (top_p <= 0.0f) k = 1;
  temperature = fminf(fmaxf(temperature, 1e-30f), 1e30f);
  for (int i = threadIdx.x; i < 256; i += kThreads) sh.table[i] = kExp2.v[i];

  Team<In> team(sh, static_cast<const In*>(a.x) + r * a.ld, a.vocab, rank, ranks);
  Part p;
  team.each(team.w0, team.w1, [&](float (&v)[N], int32_t) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      p.most = max_nan(p.most, v[e]);
      p.n += v[e] > -INFINITY;
    }
  });
  p = team.gather(p);
  const float m = p.most;
  const uint32_t finite = p.n;
  if (!(m <= FLT_MAX && m >= -FLT_MAX)) {  // NaN or +inf; -inf alone
    const float lp = m == -INFINITY ? -INFINITY : NAN;
    if (rank == 0 && threadIdx.x == 0) report(a, r, -1, lp, lp, 0);
    if (ranks > 1) ptx::cluster_sync();  // the others have read this CTA's sums
    return;
  }
  if (threadIdx.x == 0) {
    const double c = kLog2e / (double)temperature;
    Scale s;
    s.m = m;
    s.hi = (float)c;
    s.lo = (float)(c - (double)s.hi);
    s.cut = fmaxf(__double2float_ru((double)m - (double)kReach * kLn2 * (double)temperature), -FLT_MAX);
    sh.scale = s;
    sh.border = min_p > 0.0f ? __double2float_ru((double)m + (double)temperature * log((double)fminf(min_p, 1.0f))) : -INFINITY;
  }
  __syncthreads();
  const Scale s = sh.scale;

  // all weights; then the cut, and the kept ones
  Keep keep;
  p = team.gather(team.mass(s, keep, team.w0, team.w1));
  const double total = p.a;
  const bool by_k = k > 0 && k < (int64_t)finite, by_p = top_p < 1.0f && top_p > 0.0f;
  if (by_k) team.select(s, keep, true, (uint32_t)k, 0.0, 0.0);
  if (by_p) {
    const double all = by_k ? team.gather(team.mass(s, keep, team.w0, team.w1)).a : total;
    team.select(s, keep, false, 0, (double)top_p * all, all);
  }
  keep.border = sh.border;
  if (by_k || by_p || keep.border > -INFINITY) p = team.gather(team.mass(s, keep, team.w0, team.w1));
  const double mass = p.a;
  const int32_t kept = (int32_t)p.n;

  // the last CTA, warp, part and piece with a mass of its own whose predecessors' mass is at most u W
  double left = u * mass;
  auto descend = [&](int n, auto mass_of) {
    int at = 0;
    double sum = 0.0, start = 0.0;
    for (int i = 0; i < n; ++i) {
      const double v = mass_of(i);
      if (v > 0.0 && sum <= left) {
        at = i;
        start = sum;
      }
      sum += v;
    }
    left -= start;
    return at;
  };
  const int owner = descend((int)ranks, [&](int i) { return sh.all[i].a; });
  if (owner == (int)rank) {
    const int w = descend(kWarps, [&](int i) { return sh.warp[i].a; });
    int32_t a0, a1;
    team.share(rank, w, a0, a1);
    const int32_t each = (a1 - a0 + kWarps - 1) / kWarps;
    const int32_t b0 = min(a1, a0 + team.warp * each), b1 = min(a1, b0 + each);
    const Part part = merge_lanes<32>(team.mass(s, keep, b0, b1));
    if (team.lane == 0) sh.part[team.warp] = part.a;
    __syncthreads();
    const int mine = descend(kWarps, [&](int i) { return sh.part[i]; });
    if (mine == team.warp) {
      int32_t token = -1;
      float x = 0.0f;
      double sum = 0.0;
      for (int32_t p0 = b0; p0 < b1 && sum <= left; p0 += 32) {
        float v[N];
        values<In>(p0 + team.lane < b1 ? team.row.load(p0 + team.lane) : absent<In>(), v);
        const int32_t j0 = (p0 + team.lane) * N - team.row.off;
        double w_of[N], own = 0.0;
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          uint64_t h, l;
          weights(s, sh.table, keep(v[e], j0 + e) ? v[e] : -INFINITY, keep(v[e + 1], j0 + e + 1) ? v[e + 1] : -INFINITY, h, l);
          float h0, h1, l0, l1;
          ptx::f32x2_unpack(h, h0, h1);
          ptx::f32x2_unpack(l, l0, l1);
          w_of[e] = (double)h0 + (double)l0;
          w_of[e + 1] = (double)h1 + (double)l1;
          own += w_of[e] + w_of[e + 1];
        }
        double incl = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const double o = __shfl_up_sync(0xffffffffu, incl, d);
          if (team.lane >= d) incl += o;
        }
        double before = sum + (incl - own);
        const uint32_t can = __ballot_sync(0xffffffffu, own > 0.0 && before <= left);
        int32_t j = -1;
        float xj = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (w_of[e] > 0.0 && before <= left) {
            j = j0 + e;
            xj = v[e];
          }
          before += w_of[e];
        }
        if (can) {
          const int from = 31 - __clz(can);
          token = __shfl_sync(0xffffffffu, j, from);
          x = __shfl_sync(0xffffffffu, xj, from);
        }
        sum += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (team.lane == 0) {
        const float y = (x - m) / temperature;
        report(a, r, token, y - log_of(total), y - log_of(mass), kept);
      }
    }
  }
  if (ranks > 1) ptx::cluster_sync();  // the others have read this CTA's shared memory
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

template <typename In>
cudaError_t launch_sample(const SampleArgs& a, int64_t rows, cudaStream_t stream) {
  // few rows are split over a cluster, down to a load round per CTA
  const int64_t want = 4 * (int64_t)sm_count(), round = (int64_t)kThreads * kUnroll * Row<In>::N;
  int cluster = 1;
  while (cluster < kMaxCluster && rows * cluster < want && (int64_t)a.vocab > cluster * round) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster, (unsigned)rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<In>, a);
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
