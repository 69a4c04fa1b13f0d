// rotary.cu -- rotary positions of queries and keys with one or several axes,
// their backward pass, and the form joined with the append to the E4M3 cache.
//
// Pair i of a head, (a, b), at position p on the pair's axis turns by the angle
// p f_i:  (a cos - b sin, a sin + b cos); the backward pass turns by -p f_i.
// The halves of the rotated part of a head are a and b (pair i: elements i and
// pairs + i), or they alternate (2 i and 2 i + 1).  Elements past the rotated part
// stay as they are.
//
// Angles of far positions lose their digits in fp32 (p f of 10^5 is known to
// 0.008), so a frequency is held as the 64-bit binary fraction F of a turn per
// position.  p F modulo 2^64 is the angle's fraction of a turn, exact for every
// 32-bit position but for F's rounding, 2^-65 of a turn a position (2^-34 at the
// last one); its upper 32 bits go to sincospi as fp32 half turns, 2^-26 of a turn.  The product is rotated in fp32 and rounded once:
// to bf16, or (keys of the append) to the E4M3 code of the IEEE quotient by the
// cache's scale.
//
// Bound by HBM: each element is read and written once.  A CTA takes a few tokens;
// their sines and cosines are computed once into shared memory, then a thread
// keeps those of 8 pairs of a token in registers and walks the heads with
// 16-byte pieces, two heads ahead (64 registers, four CTAs an SM; four heads ahead with
// three CTAs gave the same, with two 211 us for 198 below).  Heads of 128, 32 and 8:
// 65536 tokens 198 us (6.8 TB/s), 8192 29; with the append 65536 tokens 237 us (6.2 TB/s; the
// quotients' instructions), 4001 16.3, 16 tokens 3.0.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8rl {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotAhead = 2;  // heads a thread loads before it turns the first
constexpr int64_t kMaxHeadDim = 1024;

struct RotArgs {
  const uint16_t *q, *k, *v;
  uint16_t *qo, *ko;  // ko: null in an append that keeps codes alone
  int64_t ldq, ldk, ldv, ldqo, ldko, ldp;
  const int64_t* freqs;  // [2][pairs]: fractions of a turn, axes
  const int32_t* pos;    // [axes][ldp]
  int32_t tokens, hq, hkv, d, pairs, axes, tile;
  float sign;
  // append
  const int32_t* slots;
  uint8_t *kc, *vc;
  int64_t ldc, num_slots;
  const float* scales;
  uint32_t* err;  // debug builds' store checks
};

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// (plain loads: an output may be its input)
__device__ __forceinline__ uint4 ld_u4(const void* p) { return *static_cast<const uint4*>(p); }

// cos and sin of pair i at token t, the sine with the direction's sign
__device__ __forceinline__ float2 turn_of(const RotArgs& a, int32_t t, int32_t i) {
  const int64_t axis = a.freqs[a.pairs + i];
  const int64_t p = axis >= 0 && axis < a.axes ? a.pos[axis * a.ldp + t] : 0;
  const uint64_t turn = (uint64_t)p * (uint64_t)a.freqs[i];
  // half turns in [-1, 1)
  const float half = (float)(int32_t)(turn >> 32) * 0x1p-31f;
  float2 cs;
  sincospif(half, &cs.y, &cs.x);
  cs.y *= a.sign;
  return cs;
}

// the IEEE quotient x / s, r = RN(1 / s), of values whose codes do not saturate; 1024 stands for those of the
// others, infinities among them (s past 2^118 too, where 1024 s would be infinite).  A NaN stays one
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float most = fminf(1024.0f * s, FLT_MAX);
  const float q = s >= kFastDivMinScale ? div_by_scale(x, s, r) : __fdiv_rn(x, s);
  return fabsf(x) > most ? copysignf(1024.0f, x) : q;
}
__device__ __forceinline__ uint32_t codes4(const float* x, float s, float r) {
  return e4m3x2(quotient(x[0], s, r), quotient(x[1], s, r)) | e4m3x2(quotient(x[2], s, r), quotient(x[3], s, r)) << 16;
}

// A unit is 16 elements of a head: 8 pairs, or 16 elements behind the rotated part.
// Thread = (token of the tile, unit, share of the heads).
template <bool APPEND, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const RotArgs a) {
  extern __shared__ float4 smem4[];
  float* cs = reinterpret_cast<float*>(smem4);  // [tile][2][pairs]: cosines, sines
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int32_t t0 = blockIdx.x * a.tile, n = min(a.tile, a.tokens - t0);
  for (int32_t e = threadIdx.x; e < n * a.pairs; e += kRotThreads) {
    const int32_t i = e % a.pairs, tl = e / a.pairs;
    const float2 v = turn_of(a, t0 + tl, i);
    cs[tl * 2 * a.pairs + i] = v.x;
    cs[tl * 2 * a.pairs + a.pairs + i] = v.y;
  }
  __syncthreads();
  const int32_t units = a.d / 16, per_token = units * a.tile;
  const int32_t groups = kRotThreads / per_token;
  const int32_t u = threadIdx.x % units, g = threadIdx.x / units % groups, tl = threadIdx.x / units / groups;
  if (tl >= n) return;
  const int64_t t = t0 + tl;
  const bool turned = u < a.pairs / 8;
  // the unit's two 8-element pieces
  const int32_t c0 = !turned || INTERLEAVED ? 16 * u : 8 * u, c1 = !turned || INTERLEAVED ? c0 + 8 : a.pairs + 8 * u;
  float c[8], s[8];
  if (turned) {
    const float4* at = reinterpret_cast<const float4*>(cs + tl * 2 * a.pairs + 8 * u);
    const float4* st = reinterpret_cast<const float4*>(cs + tl * 2 * a.pairs + a.pairs + 8 * u);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = at[i], y = st[i];
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
  }
  int64_t slot = -1;
  float sk = 1.0f, sv = 1.0f, rk = 1.0f, rv = 1.0f;
  if (APPEND) {
    slot = a.slots[t];
    if (slot >= a.num_slots) slot = -1;
    sk = a.scales[0];
    sv = a.scales[1];
    rk = __frcp_rn(sk);
    rv = __frcp_rn(sv);
  }
  const int32_t keys = a.hq + a.hkv, heads = keys + (APPEND && slot >= 0 ? a.hkv : 0);
  for (int32_t h0 = g; h0 < heads; h0 += kRotAhead * groups) {
    uint4 x[kRotAhead][2];
#pragma unroll
    for (int j = 0; j < kRotAhead; ++j) {
      const int32_t h = h0 + j * groups;
      if (h >= heads) break;
      const uint16_t* row = h < a.hq ? a.q + t * a.ldq + h * a.d
                                     : h < keys ? a.k + t * a.ldk + (h - a.hq) * a.d : a.v + t * a.ldv + (h - keys) * a.d;
      x[j][0] = ld_u4(row + c0);
      x[j][1] = ld_u4(row + c1);
    }
#pragma unroll
    for (int j = 0; j < kRotAhead; ++j) {
      const int32_t h = h0 + j * groups;
      if (h >= heads) break;
      if (APPEND && h >= keys) {  // a value head: codes
        uint8_t* to = a.vc + slot * a.ldc + (h - keys) * a.d;
        if (dcheck(slot < a.num_slots && (h - keys + 1) * a.d <= a.ldc, a.err)) {
          *reinterpret_cast<uint2*>(to + c0) = quant8_div(x[j][0], sv, rv);
          *reinterpret_cast<uint2*>(to + c1) = quant8_div(x[j][1], sv, rv);
        }
        continue;
      }
      const uint32_t w[8] = {x[j][0].x, x[j][0].y, x[j][0].z, x[j][0].w, x[j][1].x, x[j][1].y, x[j][1].z, x[j][1].w};
      float y[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[2 * i] = bf16_lo(w[i]);
        y[2 * i + 1] = bf16_hi(w[i]);
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int p = INTERLEAVED ? 2 * i : i, r = INTERLEAVED ? 2 * i + 1 : i + 8;
          const float u0 = y[p], u1 = y[r];
          y[p] = fmaf(u0, c[i], -u1 * s[i]);
          y[r] = fmaf(u0, s[i], u1 * c[i]);
        }
      }
      const bool key = h >= a.hq;
      uint16_t* to = key ? a.ko : a.qo;
      if (!APPEND || !key || to) {
        to += key ? t * a.ldko + (h - a.hq) * a.d : t * a.ldqo + h * a.d;
        if (dcheck(t < a.tokens && h < keys, a.err)) {
          *reinterpret_cast<uint4*>(to + c0) = make_uint4(bf16x2_rn(y[0], y[1]), bf16x2_rn(y[2], y[3]), bf16x2_rn(y[4], y[5]), bf16x2_rn(y[6], y[7]));
          *reinterpret_cast<uint4*>(to + c1) = make_uint4(bf16x2_rn(y[8], y[9]), bf16x2_rn(y[10], y[11]), bf16x2_rn(y[12], y[13]), bf16x2_rn(y[14], y[15]));
        }
      }
      if (APPEND && key && slot >= 0) {
        uint8_t* code = a.kc + slot * a.ldc + (h - a.hq) * a.d;
        if (dcheck(slot < a.num_slots && (h - a.hq + 1) * a.d <= a.ldc, a.err)) {
          *reinterpret_cast<uint2*>(code + c0) = make_uint2(codes4(y, sk, rk), codes4(y + 4, sk, rk));
          *reinterpret_cast<uint2*>(code + c1) = make_uint2(codes4(y + 8, sk, rk), codes4(y + 12, sk, rk));
        }
      }
    }
  }
}

// Any size, stride and alignment: a token per CTA, a thread per pair or element
template <bool APPEND>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const RotArgs a, int32_t interleaved) {
  extern __shared__ float4 smem4[];
  float* cs = reinterpret_cast<float*>(smem4);
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int64_t t = blockIdx.x;
  for (int32_t i = threadIdx.x; i < a.pairs; i += kRotThreads) {
    const float2 v = turn_of(a, (int32_t)t, i);
    cs[i] = v.x;
    cs[a.pairs + i] = v.y;
  }
  __syncthreads();
  int64_t slot = -1;
  float sk = 1.0f, sv = 1.0f;
  if (APPEND) {
    slot = a.slots[t];
    if (slot >= a.num_slots) slot = -1;
    sk = a.scales[0];
    sv = a.scales[1];
  }
  const int32_t keys = a.hq + a.hkv, heads = keys + (APPEND && slot >= 0 ? a.hkv : 0);
  const int32_t items = a.d - a.pairs;  // of a head: pairs, then single elements
  for (int64_t e = threadIdx.x; e < (int64_t)heads * items; e += kRotThreads) {
    const int32_t h = (int32_t)(e / items), i = (int32_t)(e % items);
    const bool turned = i < a.pairs, value = h >= keys, key = h >= a.hq && !value;
    const int32_t c0 = !turned ? a.pairs + i : interleaved ? 2 * i : i, c1 = !turned ? c0 : interleaved ? c0 + 1 : a.pairs + i;
    const uint16_t* row = value ? a.v + t * a.ldv + (int64_t)(h - keys) * a.d
                                : key ? a.k + t * a.ldk + (int64_t)(h - a.hq) * a.d : a.q + t * a.ldq + (int64_t)h * a.d;
    const float u0 = bf16_lo((uint32_t)row[c0]), u1 = bf16_lo((uint32_t)row[c1]);
    float y0 = u0, y1 = u1;
    if (turned && !value) {
      y0 = fmaf(u0, cs[i], -u1 * cs[a.pairs + i]);
      y1 = fmaf(u0, cs[a.pairs + i], u1 * cs[i]);
    }
    uint16_t* to = key ? a.ko : a.qo;
    if (!value && to) {
      to += key ? t * a.ldko + (int64_t)(h - a.hq) * a.d : t * a.ldqo + (int64_t)h * a.d;
      if (dcheck(t < a.tokens && h < keys, a.err)) {
        to[c0] = (uint16_t)bf16x2_rn(y0, 0.0f);
        if (turned) to[c1] = (uint16_t)bf16x2_rn(y1, 0.0f);
      }
    }
    if (APPEND && (key || value) && slot >= 0) {
      const float sc = key ? sk : sv;
      uint8_t* code = (key ? a.kc : a.vc) + slot * a.ldc + (int64_t)(h - (key ? a.hq : keys)) * a.d;
      if (dcheck(slot < a.num_slots && (int64_t)(h - (key ? a.hq : keys) + 1) * a.d <= a.ldc, a.err)) {
        code[c0] = (uint8_t)e4m3x2(__fdiv_rn(y0, sc), 0.0f);
        if (turned) code[c1] = (uint8_t)e4m3x2(__fdiv_rn(y1, sc), 0.0f);
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

// what both entry points ask of their common arguments; FP8RL_OK with *none set: nothing to do
fp8rl_status check(const RotArgs& a, int64_t tokens, int64_t hq, int64_t hkv, int64_t d, int64_t pairs, int64_t axes,
                   int32_t interleaved, bool* none) {
  *none = false;
  if (tokens < 0 || hq < 0 || hkv < 0 || hq + hkv < 1 || d < 1 || pairs < 0 || 2 * pairs > d || axes < 1 || (a.ldp < tokens && a.ldp != 0) ||
      (interleaved != 0 && interleaved != 1))
    return FP8RL_ERR_INVALID_ARG;
  if (d > kMaxHeadDim || hq > 8192 || hkv > 8192 || tokens >= (int64_t)1 << 31 || axes > 64) return FP8RL_ERR_SHAPE;
  if (hq > 0 && (a.ldq < hq * d || a.ldqo < hq * d)) return FP8RL_ERR_INVALID_ARG;
  if (hkv > 0 && (a.ldk < hkv * d || (a.ko && a.ldko < hkv * d))) return FP8RL_ERR_INVALID_ARG;
  if (tokens == 0) {
    *none = true;
    return FP8RL_OK;
  }
  if ((hq > 0 && (!a.q || !a.qo)) || (hkv > 0 && !a.k) || !a.pos || (pairs > 0 && !a.freqs)) return FP8RL_ERR_INVALID_ARG;
  if ((a.q && a.q == a.qo && a.ldq != a.ldqo) || (a.ko && a.k == a.ko && a.ldk != a.ldko)) return FP8RL_ERR_INVALID_ARG;
  if (!aligned(a.q, 2) || !aligned(a.qo, 2) || !aligned(a.k, 2) || !aligned(a.ko, 2) || !aligned(a.pos, 4) || !aligned(a.freqs, 8))
    return FP8RL_ERR_ALIGNMENT;
  return FP8RL_OK;
}

template <bool APPEND>
fp8rl_status launch(RotArgs& a, int32_t interleaved, cudaStream_t stream) {
  if (!check_word(&a.err)) return FP8RL_ERR_CUDA;
  auto piece = [](const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; };
  const bool vec = a.d % 16 == 0 && a.pairs % 8 == 0 && a.d <= 16 * kRotThreads && piece(a.q, a.ldq) && piece(a.qo, a.ldqo) &&
                   piece(a.k, a.ldk) && piece(a.ko, a.ldko) &&
                   (!APPEND || (piece(a.v, a.ldv) && aligned(a.kc, 8) && aligned(a.vc, 8) && a.ldc % 8 == 0));
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRotThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cudaError_t e;
  if (vec) {
    // tokens a CTA takes: up to 8, fewer while that leaves SMs without one
    const int32_t units = a.d / 16;
    a.tile = 1;
    while (a.tile < 8 && 2 * a.tile * units <= kRotThreads && (int64_t)a.tokens > (int64_t)2 * a.tile * 4 * sm_count()) a.tile *= 2;
    cfg.gridDim = dim3((unsigned)(((int64_t)a.tokens + a.tile - 1) / a.tile));  // (2^31 - 1 tokens: the sum is past 32 bits)
    cfg.dynamicSmemBytes = (size_t)a.tile * 2 * a.pairs * sizeof(float);
    e = interleaved ? cudaLaunchKernelEx(&cfg, rotary_kernel<APPEND, true>, a) : cudaLaunchKernelEx(&cfg, rotary_kernel<APPEND, false>, a);
  } else {
    cfg.gridDim = dim3((unsigned)a.tokens);
    cfg.dynamicSmemBytes = (size_t)2 * a.pairs * sizeof(float);
    e = cudaLaunchKernelEx(&cfg, rotary_any_kernel<APPEND>, a, interleaved);
  }
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}

RotArgs common(const void* q, int64_t ldq, int64_t hq, const void* k, int64_t ldk, int64_t hkv, int64_t tokens, int64_t d,
               const int64_t* freqs, int64_t pairs, const int32_t* pos, int64_t ldp, int64_t axes, void* qo, int64_t ldqo,
               void* ko, int64_t ldko) {
  RotArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.qo = static_cast<uint16_t*>(qo);
  a.ko = static_cast<uint16_t*>(ko);
  a.ldq = ldq, a.ldk = ldk, a.ldqo = ldqo, a.ldko = ldko, a.ldp = ldp;
  a.freqs = freqs;
  a.pos = pos;
  a.tokens = (int32_t)tokens, a.hq = (int32_t)hq, a.hkv = (int32_t)hkv, a.d = (int32_t)d, a.pairs = (int32_t)pairs;
  a.axes = (int32_t)axes;
  a.sign = 1.0f;
  return a;
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

extern "C" FP8RL_API fp8rl_status fp8rl_rotary(const void* q_bf16, int64_t ldq, int64_t q_heads, const void* k_bf16,
                                               int64_t ldk, int64_t kv_heads, int64_t tokens, int64_t head_dim,
                                               const int64_t* d_freqs, int64_t pairs, const int32_t* d_positions,
                                               int64_t ldp, int64_t axes, int32_t interleaved, int32_t inverse,
                                               void* q_out, int64_t ldqo, void* k_out, int64_t ldko, void* stream) {
  RotArgs a = common(q_bf16, ldq, q_heads, k_bf16, ldk, kv_heads, tokens, head_dim, d_freqs, pairs, d_positions, ldp, axes,
                     q_out, ldqo, k_out, ldko);
  if (inverse != 0 && inverse != 1) return FP8RL_ERR_INVALID_ARG;
  if (kv_heads > 0 && ldko < kv_heads * head_dim) return FP8RL_ERR_INVALID_ARG;
  bool none;
  const fp8rl_status st = check(a, tokens, q_heads, kv_heads, head_dim, pairs, axes, interleaved, &none);
  if (st != FP8RL_OK || none) return st;
  if (kv_heads > 0 && !k_out) return FP8RL_ERR_INVALID_ARG;
  if (inverse) a.sign = -1.0f;
  return launch<false>(a, interleaved, static_cast<cudaStream_t>(stream));
}

extern "C" FP8RL_API fp8rl_status fp8rl_rotary_kv_append(
    const void* q_bf16, int64_t ldq, int64_t q_heads, const void* k_bf16, int64_t ldk, const void* v_bf16, int64_t ldv,
    int64_t kv_heads, int64_t tokens, int64_t head_dim, const int64_t* d_freqs, int64_t pairs, const int32_t* d_positions,
    int64_t ldp, int64_t axes, int32_t interleaved, void* q_out, int64_t ldqo, void* k_out, int64_t ldko,
    const int32_t* d_slot_mapping, void* k_cache, void* v_cache, int64_t ld_cache, int64_t num_slots, const float* d_scales,
    void* stream) {
  RotArgs a = common(q_bf16, ldq, q_heads, k_bf16, ldk, kv_heads, tokens, head_dim, d_freqs, pairs, d_positions, ldp, axes,
                     q_out, ldqo, k_out, ldko);
  bool none;
  if (kv_heads < 1 || num_slots < 0) return FP8RL_ERR_INVALID_ARG;
  const fp8rl_status st = check(a, tokens, q_heads, kv_heads, head_dim, pairs, axes, interleaved, &none);
  if (st != FP8RL_OK) return st;
  if (ldv < kv_heads * head_dim || ld_cache < kv_heads * head_dim) return FP8RL_ERR_INVALID_ARG;
  if (none) return FP8RL_OK;
  if (!v_bf16 || !d_slot_mapping || !k_cache || !v_cache || !d_scales) return FP8RL_ERR_INVALID_ARG;
  if (!aligned(v_bf16, 2) || !aligned(d_slot_mapping, 4) || !aligned(d_scales, 4)) return FP8RL_ERR_ALIGNMENT;
  a.v = static_cast<const uint16_t*>(v_bf16);
  a.ldv = ldv;
  a.slots = d_slot_mapping;
  a.kc = static_cast<uint8_t*>(k_cache);
  a.vc = static_cast<uint8_t*>(v_cache);
  a.ldc = ld_cache;
  a.num_slots = num_slots;
  a.scales = d_scales;
  return launch<true>(a, interleaved, static_cast<cudaStream_t>(stream));
}
