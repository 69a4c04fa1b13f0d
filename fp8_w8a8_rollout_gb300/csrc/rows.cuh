// rows.cuh -- rows of logits (bf16 or fp32, any alignment) as 16-byte pieces, and
// the small fp32 operations that the kernels over them share.
#pragma once

#include <cfloat>

#include "common.cuh"

namespace fp8rl {

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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

// whether some pieces hold an element of -inf (NaN left out)
template <typename In, int U>
__device__ __forceinline__ bool holds_masked(const uint4 (&u)[U]) {
  if (sizeof(In) == 2) {
    uint32_t m = min_bf16x2(min_bf16x2(u[0].x, u[0].y), min_bf16x2(u[0].z, u[0].w));
#pragma unroll
    for (int i = 1; i < U; ++i) {
      m = min_bf16x2(m, min_bf16x2(u[i].x, u[i].y));
      m = min_bf16x2(m, min_bf16x2(u[i].z, u[i].w));
    }
    return fminf(bf16_lo(m), bf16_hi(m)) == -INFINITY;
  }
  float m = INFINITY;
#pragma unroll
  for (int i = 0; i < U; ++i)
    m = fminf(m, fminf(fminf(__uint_as_float(u[i].x), __uint_as_float(u[i].y)),
                       fminf(__uint_as_float(u[i].z), __uint_as_float(u[i].w))));
  return m == -INFINITY;
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

}  // namespace fp8rl
