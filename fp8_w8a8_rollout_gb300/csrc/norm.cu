// norm.cu -- RMS norm with the residual's addition and an E4M3 output.
//
// A decoder's residual branch ends in h = x + residual; the next W8A8 linear
// reads y = h * rsqrt(mean(h^2) + eps) * weight, quantised per 1x128 group
// ("Method steps", step 1: activations are quantised dynamically in every
// forward pass).  Fused, y never exists in bf16: h is the fp32 sum, y stays
// fp32 and is rounded once, to its E4M3 code ("Where Rounding Happens
// Matters": round once, at the end of the fused region); only the h that the
// next residual branch reads is rounded to bf16.
//
// HBM-bound: 7 bytes an element with a residual (x, residual, h, the code),
// 3 without; 8192 x 4096 takes 38.4 us back to back, 35 alone (6.1 and 6.7 TB/s;
// 128 threads with four pieces each 67, 512 with one 45).  A CTA takes one row and holds it in registers (8-column pieces,
// 16 consecutive lanes to a 128-column group), so each input is read once:
// all its loads, one CTA-wide sum of squares, then the group maxima by four
// shuffles.  Threads per row and pieces per thread follow k alone.
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8rl {
namespace {

constexpr int64_t kNormMaxK = 32768;  // a row's pieces held in registers: 1024 threads x 4 pieces x 8

constexpr int kNormThreadsPerSm = 1024;  // resident threads per SM: 64 registers each

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;     // or null
  const uint16_t* weight;
  uint16_t* h;             // or null (may be res or x: each element is read by the thread that writes it)
  uint8_t* q;
  void* scale;
  int64_t ldx, ldr, ldh, ldq, m;
  int32_t k;
  float eps;
  uint32_t* err;
};

// columns c .. c + 7 of a row; columns at or past k read as zero
__device__ __forceinline__ uint4 load8(const uint16_t* row, int32_t c, int32_t k) {
  return c < k ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void store8_bf16(uint16_t* row, int32_t c, int32_t k, const float (&v)[8], uint32_t* err) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
  if (c < k && dcheck(c + 8 <= k, err)) *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename S>
__device__ __forceinline__ void store_scale(const NormArgs& a, int32_t group, int64_t row, S s) {
  if (dcheck(group >= 0 && group * (int64_t)kBlock < a.k && row < a.m, a.err)) static_cast<S*>(a.scale)[group * a.m + row] = s;
}

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}

// the row's sum of squares from the threads': a fixed tree, the same bits on
// every run; part alternates between rows, so one barrier a row is enough
template <int T>
__device__ __forceinline__ float row_sum(float ss, float (&part)[T / 32]) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = part[0];
#pragma unroll
  for (int w = 1; w < T / 32; ++w) ss += part[w];
  return ss;
}

// k and every stride a multiple of 8 elements, every pointer 16-byte aligned
// (codes 8-byte): whole pieces only
template <int T, int NP, bool UE8M0>
__global__ void __launch_bounds__(T, kNormThreadsPerSm / T) rmsnorm_quant_kernel(const NormArgs a) {
  // rows of up to 8192 columns: the next row waits in registers
  constexpr bool kAhead = T * NP <= 1024;
  // as the activation quantiser: the next kernel may start, and this one
  // waits for the one before it ahead of its first read or write
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int tid = threadIdx.x;
  uint4 xv[NP], rv[NP];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int32_t c = (tid + j * T) * 8;
      xv[j] = load8(a.x + row * a.ldx, c, a.k);
      if (a.res) rv[j] = load8(a.res + row * a.ldr, c, a.k);
    }
  };
  if (kAhead) fetch(blockIdx.x);
  __shared__ float part[2][T / 32];  // alternating rows: one barrier a row
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, turn ^= 1) {
    if (!kAhead) fetch(row);
    float h[NP][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      unpack8(xv[j], h[j]);
      if (a.res) {
        float r[8];
        unpack8(rv[j], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] += r[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
    }
    if (kAhead && row + gridDim.x < a.m) fetch(row + gridDim.x);  // the next row's loads before this one's barrier
    if (a.h) {
      uint16_t* hr = a.h + row * a.ldh;
#pragma unroll
      for (int j = 0; j < NP; ++j) store8_bf16(hr, (tid + j * T) * 8, a.k, h[j], a.err);
    }
    ss = row_sum<T>(ss, part[turn]);
    const float rms = rsqrtf(ss / (float)a.k + a.eps);
    uint8_t* qr = a.q + row * a.ldq;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int32_t c = (tid + j * T) * 8;
      float w[8];
      unpack8(load8(a.weight, c, a.k), w);
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[j][e] = h[j][e] * rms * w[e];
        amax = fmaxf(amax, fabsf(h[j][e]));
      }
      // 16 consecutive lanes hold one 128-column group
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      if (c >= a.k) continue;
      uint32_t code[2];
      if (UE8M0) {
        const int e2 = scale_ue8m0_exponent(amax);
        const float f = exp2_neg(e2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          code[i] = e4m3x2(h[j][4 * i] * f, h[j][4 * i + 1] * f) | (e4m3x2(h[j][4 * i + 2] * f, h[j][4 * i + 3] * f) << 16);
        if ((tid & 15) == 0) store_scale(a, c / kBlock, row, (uint8_t)(e2 + 127));
      } else {
        const float s = scale_fp32(amax), r = __frcp_rn(s);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = s >= kFastDivMinScale ? div_by_scale(h[j][e], s, r) : __fdiv_rn(h[j][e], s);
#pragma unroll
        for (int i = 0; i < 2; ++i) code[i] = e4m3x2(y[4 * i], y[4 * i + 1]) | (e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16);
        if ((tid & 15) == 0) store_scale(a, c / kBlock, row, s);
      }
      if (dcheck(c + 8 <= a.k, a.err)) *reinterpret_cast<uint2*>(qr + c) = make_uint2(code[0], code[1]);
    }
  }
}

// Any k, strides and alignment, an element at a time: a warp takes whole groups,
// lane l their columns l, l + 32, l + 64 and l + 96, so that each access of the
// warp is contiguous (4392 x 6918: 79 us; pieces of eight columns a lane, each in
// eight accesses with a stride, 131).  Bound by the accesses' issue.
template <int T, int NP, bool UE8M0>
__global__ void __launch_bounds__(T, kNormThreadsPerSm / T) rmsnorm_quant_any_kernel(const NormArgs a) {
  constexpr int G = 2 * NP, W = T / 32;  // groups of a warp
  constexpr bool kAhead = T * NP <= 1024;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto column = [&](int j, int i) { return (warp + j * W) * (int)kBlock + 32 * i + lane; };
  auto load2 = [&](const uint16_t* row, int j, int i) {
    const int32_t c = column(j, i);
    return (c < a.k ? (uint32_t)row[c] : 0u) | (c + 32 < a.k ? (uint32_t)row[c + 32] << 16 : 0u);
  };
  uint32_t xv[G][2], rv[G][2];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xv[j][i] = load2(a.x + row * a.ldx, j, 2 * i);
        if (a.res) rv[j][i] = load2(a.res + row * a.ldr, j, 2 * i);
      }
  };
  if (kAhead) fetch(blockIdx.x);
  __shared__ float part[2][W];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, turn ^= 1) {
    if (!kAhead) fetch(row);
    float h[G][4];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[j][i] = i & 1 ? bf16_hi(xv[j][i >> 1]) : bf16_lo(xv[j][i >> 1]);
        if (a.res) h[j][i] += i & 1 ? bf16_hi(rv[j][i >> 1]) : bf16_lo(rv[j][i >> 1]);
        ss = fmaf(h[j][i], h[j][i], ss);
      }
    if (kAhead && row + gridDim.x < a.m) fetch(row + gridDim.x);
    if (a.h) {
      uint16_t* hr = a.h + row * a.ldh;
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t v = bf16x2_rn(h[j][2 * i], h[j][2 * i + 1]);
          const int32_t c = column(j, 2 * i);
          if (c < a.k && dcheck(c >= 0 && row < a.m, a.err)) hr[c] = (uint16_t)v;
          if (c + 32 < a.k && dcheck(c >= 0 && row < a.m, a.err)) hr[c + 32] = (uint16_t)(v >> 16);
        }
    }
    ss = row_sum<T>(ss, part[turn]);
    const float rms = rsqrtf(ss / (float)a.k + a.eps);
    uint8_t* qr = a.q + row * a.ldq;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int32_t group = warp + j * W;
      if (group * (int)kBlock >= a.k) continue;
      const uint32_t w[2] = {load2(a.weight, j, 0), load2(a.weight, j, 2)};
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[j][i] = h[j][i] * rms * (i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]));
        amax = fmaxf(amax, fabsf(h[j][i]));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      uint32_t code[2];
      if (UE8M0) {
        const int e2 = scale_ue8m0_exponent(amax);
        const float f = exp2_neg(e2);
#pragma unroll
        for (int i = 0; i < 2; ++i) code[i] = e4m3x2(h[j][2 * i] * f, h[j][2 * i + 1] * f);
        if (lane == 0) store_scale(a, group, row, (uint8_t)(e2 + 127));
      } else {
        const float s = scale_fp32(amax), r = __frcp_rn(s);
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = s >= kFastDivMinScale ? div_by_scale(h[j][i], s, r) : __fdiv_rn(h[j][i], s);
#pragma unroll
        for (int i = 0; i < 2; ++i) code[i] = e4m3x2(y[2 * i], y[2 * i + 1]);
        if (lane == 0) store_scale(a, group, row, s);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t c = column(j, 2 * i);
        if (c < a.k && dcheck(c >= 0 && row < a.m, a.err)) qr[c] = (uint8_t)code[i];
        if (c + 32 < a.k && dcheck(c >= 0 && row < a.m, a.err)) qr[c + 32] = (uint8_t)(code[i] >> 8);
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

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int T, int NP>
cudaError_t launch_norm(const NormArgs& a, bool vec, bool ue8m0, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(a.m, (int64_t)sm_count() * std::max(1, kNormThreadsPerSm / T)));
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  if (vec)
    return ue8m0 ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<T, NP, true>, a)
                 : cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<T, NP, false>, a);
  return ue8m0 ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_any_kernel<T, NP, true>, a)
               : cudaLaunchKernelEx(&cfg, rmsnorm_quant_any_kernel<T, NP, false>, a);
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

extern "C" FP8RL_API fp8rl_status fp8rl_rmsnorm_quant(const void* x_bf16, int64_t ldx, const void* residual_bf16,
                                                      int64_t ldr, const void* weight_bf16, float eps, int64_t m,
                                                      int64_t k, void* h_bf16, int64_t ldh, void* q_e4m3, int64_t ldq,
                                                      void* x_scale, fp8rl_scale_fmt fmt, void* stream) {
  if (fmt != FP8RL_SCALE_FP32 && fmt != FP8RL_SCALE_UE8M0) return FP8RL_ERR_INVALID_ARG;
  if (m < 0 || k < 0 || ldx < k || ldq < k || (residual_bf16 && ldr < k) || (h_bf16 && ldh < k) || !(eps >= 0.0f))
    return FP8RL_ERR_INVALID_ARG;
  if (m == 0 || k == 0) return FP8RL_OK;
  if (!x_bf16 || !weight_bf16 || !q_e4m3 || !x_scale) return FP8RL_ERR_INVALID_ARG;
  // in place, h's rows are those it replaces
  if (h_bf16 && ((h_bf16 == residual_bf16 && ldh != ldr) || (h_bf16 == x_bf16 && ldh != ldx))) return FP8RL_ERR_INVALID_ARG;
  if (k > kNormMaxK || m > INT32_MAX) return FP8RL_ERR_SHAPE;
  if (!aligned(x_bf16, 2) || !aligned(residual_bf16, 2) || !aligned(weight_bf16, 2) || !aligned(h_bf16, 2))
    return FP8RL_ERR_ALIGNMENT;
  if (fmt == FP8RL_SCALE_FP32 && !aligned(x_scale, 4)) return FP8RL_ERR_ALIGNMENT;
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.res = static_cast<const uint16_t*>(residual_bf16);
  a.weight = static_cast<const uint16_t*>(weight_bf16);
  a.h = static_cast<uint16_t*>(h_bf16);
  a.q = static_cast<uint8_t*>(q_e4m3);
  a.scale = x_scale;
  a.ldx = ldx, a.ldr = ldr, a.ldh = ldh, a.ldq = ldq, a.m = m;
  a.k = (int32_t)k;
  a.eps = eps;
#ifdef FP8RL_DEBUG  // only the store checks look at it
  a.err = device_error_word();
  if (!a.err) return FP8RL_ERR_CUDA;
#endif
  const bool vec = k % 8 == 0 && ldx % 8 == 0 && ldq % 8 == 0 && (!residual_bf16 || ldr % 8 == 0) &&
                   (!h_bf16 || ldh % 8 == 0) && aligned(x_bf16, 16) && aligned(residual_bf16, 16) &&
                   aligned(weight_bf16, 16) && aligned(h_bf16, 16) && aligned(q_e4m3, 8);
  const bool ue = fmt == FP8RL_SCALE_UE8M0;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (k <= 1024) e = launch_norm<128, 1>(a, vec, ue, cs);
  else if (k <= 2048) e = launch_norm<256, 1>(a, vec, ue, cs);
  else if (k <= 4096) e = launch_norm<256, 2>(a, vec, ue, cs);
  else if (k <= 8192) e = launch_norm<512, 2>(a, vec, ue, cs);
  else if (k <= 16384) e = launch_norm<1024, 2>(a, vec, ue, cs);
  else e = launch_norm<1024, 4>(a, vec, ue, cs);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FP8RL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}
