// sample.cuh -- what the two sampling kernels share: numbers as pairs of fp32
// numbers, exact weights, a row's parameters.
#pragma once

#include <cfloat>
#include <climits>

#include "common.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace fp8rl {
namespace sampling {

constexpr int kMaxCluster = 8;
constexpr float kReach = 100.0f;    // weights below 2^-100 count as 0
constexpr int32_t kUndecided = -2;  // the token of a row that is left to the exact kernel

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

// The weights of two elements, each hi + lo: a table-driven exponential (P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point arithmetic", ACM TOMS 15(2), 1989) in pairs
// of numbers (T. J. Dekker, "A floating-point technique for extending the available precision", 1971).  With d = m - x (exact as a pair) and t = d c
// (a pair), k = round(256 t) and the rest r: 2^-t = 2^-(k >> 8) 2^-((k & 255) / 256) e^g,
// g = -r ln 2, |g| < 0.0014.  e^g - 1 = g + g^2 (1/2 + g/6) with g a pair: g^4 / 24 is
// left out, below 2^-42.7.  The products of both numbers' low parts with g count: those of the table's (2^-25) and
// of t's (2^-24 t) are 2^-34 of a weight and more.  Off by 2^-41.6 at most for t up to 16, 2^-40 for the
// lightest, 2^-44 as a rule; rows of 151936 have their borders to 2^-46.
__device__ __forceinline__ void weights(const Scale& s, const float2* table, float x0, float x1, uint64_t& h, uint64_t& l) {
  constexpr float kMagic = 49152.0f, kL2 = 0.693147182464599609375f, kL2Lo = -1.90465429995776804e-9f;
  const uint64_t m = both(s.m), x = pair_of(fmaxf(x0, s.cut), fmaxf(x1, s.cut));
  const uint64_t d = sub2(m, x), b = sub2(d, m);
  const uint64_t e = sub2(sub2(m, sub2(d, b)), add2(x, b));  // d + e = m - x
  const uint64_t nt = pair_mul(d, both(-s.hi));  // (a product of its own: tl is what it lacks)
  uint64_t tl = pair_fma(d, both(s.hi), nt);
  tl = pair_fma(d, both(s.lo), tl);
  tl = pair_fma(e, both(s.hi), tl);
  const uint64_t z = sub2(both(kMagic), nt);             // 256 t rounded, in its low bits
  const uint64_t nr = add2(nt, sub2(z, both(kMagic)));   // exact
  const uint64_t g = pair_mul(nr, both(kL2)), ng = pair_mul(nr, both(-kL2));
  uint64_t gl = pair_fma(nr, both(kL2), ng);
  gl = pair_fma(nr, both(kL2Lo), gl);
  gl = pair_fma(tl, both(-kL2), gl);
  const uint64_t ga = add2(g, gl), q = pair_fma(pair_mul(ga, ga), pair_fma(ga, both(1.0f / 6.0f), both(0.5f)), gl);
  float z0, z1;
  ptx::f32x2_unpack(z, z0, z1);
  const int32_t k0 = __float_as_int(z0) - 0x47400000, k1 = __float_as_int(z1) - 0x47400000;
  const float2 t0 = table[k0 & 255], t1 = table[k1 & 255];
  // (The product of th and g is not named: a mul and an add of pairs may be made one fma, whose sum holds the
  // product's rounding that a remainder of its own would count a second time.)
  const uint64_t th = pair_of(t0.x, t1.x), tt = pair_of(t0.y, t1.y);
  const uint64_t hi = pair_fma(th, g, th);
  uint64_t lo = add2(pair_fma(th, g, sub2(th, hi)), pair_fma(tt, g, tt));
  lo = pair_fma(th, q, lo);
  const uint64_t by = pair_of(x0 >= s.cut ? __int_as_float((127 - (k0 >> 8)) << 23) : 0.0f,
                              x1 >= s.cut ? __int_as_float((127 - (k1 >> 8)) << 23) : 0.0f);
  h = pair_mul(hi, by);
  l = pair_mul(lo, by);
}

// that of one element
__device__ __forceinline__ Pair weight(const Scale& s, const float2* table, float x) {
  uint64_t h, l;
  weights(s, table, x, -INFINITY, h, l);
  float h0, l0, none;
  ptx::f32x2_unpack(h, h0, none);
  ptx::f32x2_unpack(l, l0, none);
  return normal(h0, l0);
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

// The same of many terms, in two steps.  Sum's low half is rounded at each addition, by 2^-25 of what n roundings of
// the upper one have left there: where the terms are equal these are of one sign, n^2 2^-53 of the sum in the end
// (2^-33 at the 1024 terms that a thread of 512 has of 2^20 elements: draws beside borders between two runs
// of equal logits then fell to the neighbour).  So a few terms' sum is folded into a pair that is kept
// normal, off by 2^-48 of it each time: 2^-43 in the end at 1024 terms, 2^-39 at 2^14.
struct LongSum {
  Sum part;
  uint64_t h = 0, l = 0;
  __device__ __forceinline__ void add(uint64_t vh, uint64_t vl) { part.add(vh, vl); }
  __device__ __forceinline__ void fold() {
    const uint64_t s = add2(h, part.h), b = sub2(s, h);
    const uint64_t e = add2(add2(sub2(h, sub2(s, b)), sub2(part.h, b)), add2(l, part.l));
    h = add2(s, e);
    l = sub2(e, sub2(h, s));
    part = Sum{};
  }
  __device__ __forceinline__ Pair value() const {  // of what has been folded
    Sum all;
    all.h = h;
    all.l = l;
    return all.value();
  }
};

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as 0
  return b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) { return __uint_as_float(o ^ ((int32_t)o < 0 ? 0x80000000u : 0xffffffffu)); }

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

// A cluster barrier in two halves: a CTA that only has to outlive the others' reads of its
// shared memory waits at its end
// (not .aligned: the lanes may come from code that some of them ran alone)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// 16-byte asynchronous global -> shared copy past L1
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// the rows that the pass has left (sample_exact.cu)
cudaError_t launch_sample_exact(const SampleArgs& a, bool fp32, bool cut, cudaStream_t stream);

int sm_count();  // of the current device

template <typename K>
cudaError_t launch_clusters(K kernel, const SampleArgs& a, int cluster, int64_t rows, int threads, cudaStream_t stream) {
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

}  // namespace sampling
}  // namespace fp8rl
