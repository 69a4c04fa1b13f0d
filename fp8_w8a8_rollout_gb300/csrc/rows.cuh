// rows.cuh -- rows of logits (bf16 or fp32, any alignment) as 16-byte pieces, and
// the small fp32 operations that the kernels over them share.
#pragma once

#include "common.cuh"

namespace fp8rl {

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

}  // namespace fp8rl
