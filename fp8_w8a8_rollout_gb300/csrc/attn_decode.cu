// attn_decode.cu -- attention of one new token per sequence over the paged
// E4M3 KV cache that the append writes ("Method steps", step 3: the KV cache
// is stored in FP8 with one scale per tensor).
//
// For sequence b with n cached keys, KV head h and the query heads i that
// share it: s_ij = softmax_scale * sK * (q_i . k_j), p_ij = exp(s_ij - m_i),
// out_i = sV * sum_j p_ij v_j / sum_j p_ij, all heads of a group in one pass
// over the cache (each key and value byte is read once).
//
// The cache's codes feed the tensor cores exactly: an E4M3 value is an f16
// value, so codes are converted, not dequantised, and both scales are applied
// in fp32 to the scores and to the output.  q is bf16; each head's row is
// multiplied by a power of two that brings its largest magnitude to [1, 2)
// and rounded to f16, which holds every bf16 bit of values down to 2^-14 of
// that largest one (below it, absolute steps of 2^-24 of it).  p is rounded to
// f16 (11 bits); its reference lies 2^11 below the maximum that sets it, and up to
// 2^15 once that grows, so that nearly all of f16's range is left to small ones: 11
// bits down to 2^-25 of the largest, steps of 2^-35 of it further down.  (131 072
// keys 17 e-folds below a key that has no value: their output is 3e-4 off at
// most, where a reference at the maximum had it 44 % off in simulation; nothing
// slower, with 2^7 and 2^12 below neither.)  Scores, sums, maxima and the output
// accumulators are fp32.
//
// HBM-bound: 2 d bytes per key and KV head, a few operations per byte, so
// the products run on m16n8k16 tensor instructions with the roles swapped: the
// 16 rows are keys (scores) or output columns (values), the 8 columns are the
// query heads of the group, so a group of up to 8 heads costs one instruction.
// Groups of up to four sit on the even columns, so that a lane's second column
// needs no softmax (1024 caches of 100 to 300: 105 us instead of 111).
// KV heads of 64 run as pairs of neighbours, whose rows are 128 contiguous
// bytes: each product instruction serves one of the two, in columns of their
// own (256 caches of 2000 to 2100, 16 heads of 16: 192 us; a head at a time, in
// rows of 64 bytes, 357, 3.0 TB/s).  An odd number of KV heads of 64, or a group of more
// than 8, is taken a head at a time.
// Each warp streams its keys through a ring of its own in shared memory
// (16-byte asynchronous copies: no registers wait for them, no CTA-wide
// barrier).  A lane's 16 contiguous bytes of a key row are its operand words of
// four instructions (the order of the d columns is free as long as q uses the
// same); for values the bytes of two keys are interleaved by byte permutes.  Scores become the
// second product's operand by an 8x8 transpose in registers.
//
// GB300: 256 caches of up to 4096 keys (32 query, 8 KV heads of 128) 182 to 186 us
// by the device, 6.2 TB/s (0.91 to 0.93 of the measured copy rate); four of
// 100 000 to 131 071 (32 and 4 heads) 89 us, 5.6 TB/s; one of 1000 about 8 us, a
// chain of dependent loads.  Two stages of 32 keys and three CTAs per SM: with
// items of one head (205 us), 16-key steps with three to six stages took 217 to
// 268 us for the 256 caches, three or four 32-key stages with two CTAs per SM
// 217 and 252.
//
// Work split: the 128-key tiles of all sequences and KV heads form one list,
// shared out to the CTAs in equal contiguous ranges, whatever the lengths (an
// item of one sequence and KV head counts two tiles more, for its start:
// 209 us instead of 258 for the 256 caches, measured with items of one head).
// Where a call has many items, an item is two neighbouring heads (or pairs), each
// with two of the CTA's warps.  An item that spans CTAs leaves fp32 partials in the
// workspace; the CTA that arrives last merges them in CTA order, so the
// result has the same bits on every run.  Many partials are merged in two steps, by
// neighbours first (one cache of 100 000 with 8 heads on one KV head: 19 us, 55 in one step).
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8rl {
namespace {

constexpr int kAdWarps = 4;
constexpr int kAdThreads = kAdWarps * 32;
constexpr int kAdSubs = 2;                       // 16-key products of a step
constexpr int kAdStep = 16 * kAdSubs;            // keys a warp takes at a time
constexpr int kAdStages = 2;                     // steps in a warp's ring
constexpr int kAdItemCost = 2;                   // fixed cost of an item, in tiles
// Pieces of partials that a thread merges one behind the other.  In one step
// against two: 33 pieces 11 and 13 us, 56 90 and 91, 57 23 and 22, 99 25 and 18.
constexpr int kAdFlat = 56;
constexpr int kAdMaxBatch = 8192;                // prefix sums held in shared memory
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The reference of the exponentials (base 2): the maximum less kLead when it is set,
// raised again once a score lies kRescale above it, so p <= 2^15 (f16 ends at 65504).
constexpr float kLead = 11.0f, kRescale = 15.0f;

// How a call runs.  D: bytes of a key row that a step reads, one KV head's, or
// two neighbours' of 64 (P = 2); NT: 8-head column blocks; C: the columns in
// use of the two that a lane holds (1: on the even columns); W: neighbouring KV
// heads (or pairs) of an item, each with warps of its own.
template <int D_, int NT_, int C_, int P_, int W_>
struct Form {
  static constexpr int D = D_, NT = NT_, C = C_, P = P_, W = W_;
  static constexpr int kTile = kAdStep * kAdWarps / W;             // keys a CTA takes at a time
  static constexpr int kHead = D / P;                              // head size
  static constexpr bool kOwn = P == 2 && NT == 2;                  // a column block for each KV head of the pair
  static constexpr int kQ = P == 2 ? 1 : D / 64;                   // 64-column parts of a query head
  static constexpr int kO = kOwn ? D / 32 : D / 16;                // 16-row accumulators of a column block
  // resident CTAs per SM (registers): the work is shared out to exactly these
  static constexpr int kCtas = NT == 1 || kOwn ? (D == 64 ? 4 : 3) : 2;
  static constexpr int64_t kPart = (int64_t)8 * NT * (kHead + 2);  // floats of a KV head's (or pair's) partial: per head its accumulators, then m and l
};

struct AdArgs {
  const uint16_t* q;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* table;
  const int32_t* lens;
  const float* scales;
  uint16_t* out;
  float* lse;  // or null
  uint32_t* tickets;
  float* parts;
  int64_t ldq, num_slots, ldt, ldo;
  uint32_t ldc16;  // cache row stride in units of 16 bytes
  int32_t batch, hq, hkv, group, sub, page, page_shift, max_len;
  float softmax_scale;
  int64_t n_tickets, n_parts;  // the workspace's counters and floats
  uint32_t* err;               // debug builds' store checks
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two E4M3 codes (low 16 bits) -> two f16, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
// 16-byte asynchronous global -> shared copy past L1; bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp_async_16(uint32_t dst, const uint8_t* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A step of a warp in shared memory: kAdStep key rows of D bytes, then as many
// value rows.  The 16-byte chunks of a row are permuted so that eight lanes
// that read together (key reads: rows r, r + 1, four chunks each; value reads:
// rows r, r + 2, r + 4, r + 6, two chunks each) meet all 32 banks.
template <int D>
struct Ring {
  static constexpr uint32_t kV = kAdStep * D;               // value rows' offset in a stage
  static constexpr uint32_t kStage = 2 * kAdStep * D;
  static __device__ __forceinline__ uint32_t key(uint32_t row, uint32_t c) {
    return row * D + ((D == 128 ? c ^ ((row & 1u) << 2) : c) << 4);
  }
  static __device__ __forceinline__ uint32_t value(uint32_t row, uint32_t c) {
    if (D == 128) return kV + row * D + ((c ^ (row & 6u)) << 4);
    // two rows to a line of 128 bytes: r and r + 2
    const uint32_t line = (row >> 2) * 2 + (row & 1u), half = (row ^ (row >> 1)) & 1u;
    return kV + line * 128 + half * 64 + ((c ^ ((row >> 1) & 2u)) << 4);
  }
};

// request a step: off16 is this lane's key's cache row in units of 16 bytes
// (lane l: key l of the step), kMasked for a key that does not count
constexpr uint32_t kMasked = 0xFFFFFFFFu;
template <int D>
__device__ __forceinline__ void request(uint32_t stage, const uint8_t* kc, const uint8_t* vc, uint32_t off16) {
  constexpr int kLanesPerRow = D / 16, kRowsPerPass = 32 / kLanesPerRow;
  const int lane = threadIdx.x & 31, c = lane % kLanesPerRow, r0 = lane / kLanesPerRow;
#pragma unroll
  for (int i = 0; i < kAdStep / kRowsPerPass; ++i) {
    const int row = r0 + i * kRowsPerPass;
    const uint32_t o = __shfl_sync(0xffffffffu, off16, row);
    const uint32_t n = o == kMasked ? 0u : 16u;
    const uint64_t at = (uint64_t)(n ? o : 0u) * 16u + c * 16;
    cp_async_16(stage + Ring<D>::key(row, c), kc + at, n);
    cp_async_16(stage + Ring<D>::value(row, c), vc + at, n);
  }
}

// A segment's accumulators of the warps, merged at its end (over the rings)
template <class F>
struct AdMerge {
  float o[kAdWarps][8 * F::NT][F::kHead];
  float m[kAdWarps][8 * F::NT], l[kAdWarps][8 * F::NT];
};

template <class F>
__host__ __device__ constexpr uint32_t ad_smem() {
  constexpr uint32_t ring = kAdWarps * kAdStages * Ring<F::D>::kStage, merge = sizeof(AdMerge<F>);
  return ring > merge ? ring : merge;
}

__device__ __forceinline__ void add_scaled(float4& a, float f, float4 v) {
  a.x = fmaf(f, v.x, a.x);
  a.y = fmaf(f, v.y, a.y);
  a.z = fmaf(f, v.z, a.z);
  a.w = fmaf(f, v.w, a.w);
}

// outputs d .. d + 3 of a head from its sums; a head without keys gives zeros
__device__ __forceinline__ void finish(const AdArgs& a, int b, int h, int D, int d, float4 acc, float l, float m, float sv) {
  if (!dcheck(b < a.batch && h >= 0 && h < a.hq && d + 4 <= D, a.err)) return;
  const float f = l == 0.0f ? 0.0f : sv / l;
  *reinterpret_cast<uint2*>(a.out + b * a.ldo + (int64_t)h * D + d) = make_uint2(bf16x2_rn(acc.x * f, acc.y * f), bf16x2_rn(acc.z * f, acc.w * f));
  if (a.lse && d == 0) a.lse[(int64_t)b * a.hq + h] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
}

template <class F>
__global__ void __launch_bounds__(kAdThreads, F::kCtas) attn_decode_kernel(const AdArgs a) {
  constexpr int D = F::D, NT = F::NT, C = F::C, P = F::P, W = F::W, H = F::kHead, kTile = F::kTile;
  extern __shared__ __align__(128) uint8_t smem[];  // the warps' rings, or the merge; then batch + 1 running tile counts
  __shared__ int64_t warp_sum[kAdWarps];
  __shared__ int32_t last;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  AdMerge<F>& sm = *reinterpret_cast<AdMerge<F>*>(smem);
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + ad_smem<F>());
  const uint32_t ring = ptx::smem_u32(smem) + warp * kAdStages * Ring<D>::kStage;
  const int heads_sub = a.hkv / W * a.sub;  // items of a sequence: KV heads by W, times parts of the group

  // running counts of the sequences' tiles (each times heads_sub)
  {
    int64_t run = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kAdThreads) {
      const int b = b0 + tid;
      const int32_t n = b < a.batch ? min(max(a.lens[b], 0), a.max_len) : 0;
      int64_t x = n > 0 ? (int64_t)((n + kTile - 1) / kTile + kAdItemCost) * heads_sub : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      int64_t before = run;
      for (int w = 0; w < kAdWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        run += warp_sum[w];
      }
      if (b < a.batch) prefix[b + 1] = before + x;
      __syncthreads();
    }
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
  }
  const int64_t total = prefix[a.batch], cta = blockIdx.x;

  // sequences without keys: zeros, spread over the CTAs
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    for (int i = tid; i < a.hq * H; i += kAdThreads)
      if (dcheck(i < a.ldo, a.err)) a.out[b * a.ldo + i] = 0;
    if (a.lse)
      for (int i = tid; i < a.hq; i += kAdThreads) a.lse[(int64_t)b * a.hq + i] = -INFINITY;
  }

  // no CTA of the first `ctas` has an empty range, so a split item's CTAs are
  // consecutive and all of them arrive at its ticket
  // Between one and two units a CTA, two each: the largest share is the same, with
  // half the partials to merge (one cache of 8000: 11.4 us, 14.2 with all CTAs).
  const int64_t grid = gridDim.x, ctas = total <= grid ? total : total <= 2 * grid ? (total + 1) / 2 : grid;
  if (cta >= ctas) return;
  const int64_t w0 = cta * total / ctas, w1 = (cta + 1) * total / ctas;
  const float sk = a.scales[0], sv = a.scales[1];
  // the sequence of tile w0: the last b with prefix[b] <= w0
  int b = 0;
  {
    int hi = a.batch;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (prefix[mid] <= w0) b = mid;
      else hi = mid;
    }
  }
  int64_t w = w0;
  bool first_segment = true;
  while (w < w1) {
    while (prefix[b + 1] <= w) ++b;
    const int32_t n = min(a.lens[b], a.max_len);
    const int64_t tiles = (prefix[b + 1] - prefix[b]) / heads_sub - kAdItemCost;
    const int item = (int)((w - prefix[b]) / (tiles + kAdItemCost));  // kv head * sub + part of the group
    const int64_t item_w0 = prefix[b] + item * (tiles + kAdItemCost), item_w1 = item_w0 + tiles + kAdItemCost;
    const int64_t seg_w1 = min(w1, item_w1);
    // the first units of an item stand for its fixed cost, the others for its tiles
    const int64_t t0 = max(w - item_w0 - kAdItemCost, (int64_t)0), t1 = max(seg_w1 - item_w0 - kAdItemCost, (int64_t)0);
    w = seg_w1;
    if (t0 == t1) break;  // this CTA's range ends before the item's first tile
    const bool whole = t0 == 0 && t1 == tiles;
    const int kvh = item / a.sub * W + warp % W;  // KV head, or pair of them
    const int h0 = kvh * P * a.group + (item % a.sub) * 8 * NT;
    const int heads = min(8 * NT, P * a.group - (item % a.sub) * 8 * NT);
    // the head (from h0) of column `col` of block nt, -1 for none: a pair's first
    // KV head has the block's lower columns or block 0
    auto head_of = [&](int nt, int col) {
      if (C == 1 && (col & 1)) return -1;
      const int per = C == 1 ? 2 : 1;
      const int second = P == 1 ? 0 : F::kOwn ? nt : col >> 2;
      const int i = (P == 1 ? nt * 8 + col : F::kOwn ? col : col & 3) / per;
      const int lim = P == 1 ? heads : a.group;
      return i < lim ? second * a.group + i : -1;
    };
    const uint8_t* kc = a.kc + (int64_t)kvh * D;
    const uint8_t* vc = a.vc + (int64_t)kvh * D;
    const int32_t* table = a.table + (int64_t)b * a.ldt;

    // This warp's steps: keys [key, key + kAdStep), one tile apart.  The
    // first ones are requested before the queries are read.
    const int32_t k1 = (int32_t)min((int64_t)n, t1 * kTile);
    int32_t key = (int32_t)t0 * kTile + warp / W * kAdStep;
    // the cache row of key0 + lane
    auto row_of = [&](int32_t key0) -> uint32_t {
      const int32_t kk = key0 + lane;
      if (lane >= kAdStep || kk >= k1) return kMasked;
      const int32_t pg = a.page_shift >= 0 ? kk >> a.page_shift : kk / a.page;
      const int64_t blk = table[pg];
      const int64_t s = blk * a.page + (kk - pg * a.page);
      return blk >= 0 && s < a.num_slots ? (uint32_t)s * a.ldc16 : kMasked;
    };
    // `row` of the step at hand, `ahead` of the steps requested after it
    uint32_t row = row_of(key), ahead[kAdStages];
    if (key < k1) request<D>(ring, kc, vc, row);
    ptx::cp_async_commit();
#pragma unroll
    for (int i = 1; i < kAdStages; ++i) {
      ahead[i - 1] = row_of(key + i * kTile);
      if (i + 1 < kAdStages) {
        if (key + i * kTile < k1) request<D>(ring + i * Ring<D>::kStage, kc, vc, ahead[i - 1]);
        ptx::cp_async_commit();
      }
    }
    // the query heads as operand words (column = head): lane (g, t) holds
    // head g's columns d = 64 j + 16 t + [0, 16)
    uint32_t qf[NT][F::kQ][4][2];
    float qs[NT][C];  // score scale of this lane's result columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = head_of(nt, g);
      uint32_t raw[F::kQ][8];
      uint32_t big = 0;
#pragma unroll
      for (int j = 0; j < F::kQ; ++j) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + (int64_t)b * a.ldq + (int64_t)(h0 + max(h, 0)) * H + 64 * j + 16 * t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          raw[j][i] = h >= 0 ? src[i] : 0u;
          big = max(big, max(raw[j][i] & 0x7FFFu, (raw[j][i] >> 16) & 0x7FFFu));
        }
      }
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^-e of the largest magnitude's exponent (its row to [1, 2)); e kept
      // where 2^-e and 2^e are normal numbers
      const int e = min(max((int)(big >> 7) - 127, -126), 126);
      const float down = __int_as_float((127 - e) << 23), up = __int_as_float((127 + e) << 23);
#pragma unroll
      for (int j = 0; j < F::kQ; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          qf[nt][j][s][0] = f16x2_rn(bf16_lo(raw[j][2 * s]) * down, bf16_hi(raw[j][2 * s]) * down);
          qf[nt][j][s][1] = f16x2_rn(bf16_lo(raw[j][2 * s + 1]) * down, bf16_hi(raw[j][2 * s + 1]) * down);
        }
      const float f = up * (sk * a.softmax_scale * kLog2e);
#pragma unroll
      for (int c = 0; c < C; ++c) qs[nt][c] = __shfl_sync(0xffffffffu, f, 8 * t + 4 * c);  // lane of column 2t + c
    }

    float o[NT][F::kO][4];
    float m[NT][C], l[NT][C];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < F::kO; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) m[nt][c] = -INFINITY, l[nt][c] = 0.0f;
    }

    uint32_t stage = 0;
    for (; key < k1; key += kTile) {
      // request the last step that fits the ring, look up the rows of the one after it
      const uint32_t to = stage + kAdStages - 1 < kAdStages ? stage + kAdStages - 1 : stage - 1;
      ahead[kAdStages - 1] = row_of(key + kAdStages * kTile);
      if (key + (kAdStages - 1) * kTile < k1) request<D>(ring + to * Ring<D>::kStage, kc, vc, ahead[kAdStages - 2]);
      ptx::cp_async_commit();
      ptx::cp_async_wait<kAdStages - 1>();
      __syncwarp();
      const uint32_t at = ring + stage * Ring<D>::kStage;
      const uint32_t live = __ballot_sync(0xffffffffu, row != kMasked);  // bit i: key i counts

      float s[kAdSubs][NT][4];
#pragma unroll
      for (int u = 0; u < kAdSubs; ++u) {
        float second[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // scores of a pair's second KV head
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint4 x0 = lds128(at + Ring<D>::key(16 * u + g, 4 * j + t)), x1 = lds128(at + Ring<D>::key(16 * u + g + 8, 4 * j + t));
          const uint32_t r0[4] = {x0.x, x0.y, x0.z, x0.w}, r1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = e4m3x2_to_f16x2(r0[i]), a2 = e4m3x2_to_f16x2_hi(r0[i]);
            const uint32_t a1 = e4m3x2_to_f16x2(r1[i]), a3 = e4m3x2_to_f16x2_hi(r1[i]);
            if (P == 2) {
              mma_16816(j == 0 || F::kOwn ? s[u][F::kOwn ? j : 0] : second, a0, a1, a2, a3, qf[F::kOwn ? j : 0][0][i][0], qf[F::kOwn ? j : 0][0][i][1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(s[u][nt], a0, a1, a2, a3, qf[nt][j % F::kQ][i][0], qf[nt][j % F::kQ][i][1]);
            }
          }
        }
        if (P == 2 && !F::kOwn) {
#pragma unroll
          for (int c = 0; c < 4; ++c) s[u][0][c] = t < 2 ? s[u][0][c] : second[c];
        }
      }
      uint32_t pb[kAdSubs][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float big[C];
#pragma unroll
        for (int c = 0; c < C; ++c) big[c] = -INFINITY;
#pragma unroll
        for (int u = 0; u < kAdSubs; ++u) {
          const bool on0 = live >> (16 * u + g) & 1u, on1 = live >> (16 * u + g + 8) & 1u;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float &x0 = s[u][nt][c], &x1 = s[u][nt][c + 2];
            x0 *= qs[nt][c];
            x1 *= qs[nt][c];
            if (live != (kAdStep == 32 ? 0xFFFFFFFFu : 0xFFFFu)) {
              x0 = on0 ? x0 : -INFINITY;
              x1 = on1 ? x1 : -INFINITY;
            }
            big[c] = fmaxf(big[c], fmaxf(x0, x1));
          }
        }
        bool above = big[0] > m[nt][0] + kRescale;
        if (C == 2) above = above || big[C - 1] > m[nt][C - 1] + kRescale;
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) big[c] = fmaxf(big[c], __shfl_xor_sync(0xffffffffu, big[c], d));
            const float to_m = fmaxf(m[nt][c], big[c] - kLead);
            const float f = to_m == -INFINITY ? 1.0f : ex2(m[nt][c] - to_m);
            m[nt][c] = to_m;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < F::kO; ++i) {
              o[nt][i][c] *= f;
              o[nt][i][c + 2] *= f;
            }
          }
        }
        float ref[C];
#pragma unroll
        for (int c = 0; c < C; ++c) ref[c] = m[nt][c] == -INFINITY ? 0.0f : m[nt][c];
#pragma unroll
        for (int u = 0; u < kAdSubs; ++u) {
          float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < C; ++c) {
            p[c] = ex2(s[u][nt][c] - ref[c]);
            p[c + 2] = ex2(s[u][nt][c + 2] - ref[c]);
            l[nt][c] += p[c] + p[c + 2];
          }
          pb[u][nt][0] = transpose_8x8(f16x2_rn(p[0], p[1]));
          pb[u][nt][1] = transpose_8x8(f16x2_rn(p[2], p[3]));
        }
      }
#pragma unroll
      for (int u = 0; u < kAdSubs; ++u) {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t r = 16 * u + 2 * t + (i & 1) + 8 * (i >> 1);
          if (F::kOwn) {
            const uint2 x = lds64(at + Ring<D>::value(r, g >> 1) + 8 * (g & 1)), y = lds64(at + Ring<D>::value(r, 4 + (g >> 1)) + 8 * (g & 1));
            v[i][0] = x.x, v[i][1] = x.y, v[i][2 % (D / 32)] = y.x, v[i][3 % (D / 32)] = y.y;
          } else if (D == 128) {
            const uint4 x = lds128(at + Ring<D>::value(r, g));
            v[i][0] = x.x, v[i][1] = x.y, v[i][2 % (D / 32)] = x.z, v[i][3 % (D / 32)] = x.w;
          } else {
            const uint2 x = lds64(at + Ring<D>::value(r, g >> 1) + 8 * (g & 1));
            v[i][0] = x.x, v[i][1] = x.y;
          }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          // bytes of d and d + 1 of two keys, side by side per d
          const uint32_t x0 = __byte_perm(v[0][i], v[1][i], 0x5140), x1 = __byte_perm(v[0][i], v[1][i], 0x7362);
          const uint32_t y0 = __byte_perm(v[2][i], v[3][i], 0x5140), y1 = __byte_perm(v[2][i], v[3][i], 0x7362);
          const uint32_t a00 = e4m3x2_to_f16x2(x0), a01 = e4m3x2_to_f16x2_hi(x0), a02 = e4m3x2_to_f16x2(y0), a03 = e4m3x2_to_f16x2_hi(y0);
          const uint32_t a10 = e4m3x2_to_f16x2(x1), a11 = e4m3x2_to_f16x2_hi(x1), a12 = e4m3x2_to_f16x2(y1), a13 = e4m3x2_to_f16x2_hi(y1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (F::kOwn && nt != i / 2) continue;
            const int at_o = F::kOwn ? i % 2 : i;
            mma_16816(o[nt][2 * at_o], a00, a01, a02, a03, pb[u][nt][0], pb[u][nt][1]);
            mma_16816(o[nt][2 * at_o + 1], a10, a11, a12, a13, pb[u][nt][0], pb[u][nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage: the next iteration's request may overwrite it
      row = ahead[0];
#pragma unroll
      for (int i = 0; i + 1 < kAdStages; ++i) ahead[i] = ahead[i + 1];
      stage = stage + 1 < kAdStages ? stage + 1 : 0;
    }
    ptx::cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring

    // the warps' partials to shared memory; row d = 2 kO g + 2 i (+ 1) of the
    // lane's rows, of which a pair's second KV head has the upper half
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int h = head_of(nt, 2 * t + c);
        const bool upper = P == 2 && !F::kOwn && t >= 2;
        const int d = 2 * F::kO * g - (upper ? H : 0);
        if (h >= 0 && d >= 0 && d < H) {
#pragma unroll
          for (int i = 0; i < F::kO; ++i)
            *reinterpret_cast<float2*>(&sm.o[warp][h][d + 2 * i]) = make_float2(o[nt][i][c], o[nt][i][c + 2]);
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
        if (g == 0 && h >= 0) {
          sm.m[warp][h] = m[nt][c];
          sm.l[warp][h] = l[nt][c];
        }
      }
    }
    __syncthreads();
    float* part = a.parts + (2 * cta + (first_segment ? 0 : 1)) * W * F::kPart;
    const int h_item = h0 - warp % W * P * a.group, pieces = heads * (H / 4);
    for (int i = tid; i < W * pieces; i += kAdThreads) {
      const int wi = W == 2 && i >= pieces, h = (i - wi * pieces) / (H / 4), d = i % (H / 4) * 4;
      float mm = sm.m[wi][h];
#pragma unroll
      for (int x = W; x < kAdWarps; x += W) mm = fmaxf(mm, sm.m[wi + x][h]);
      const float ref = mm == -INFINITY ? 0.0f : mm;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float ll = 0.0f;
#pragma unroll
      for (int x = 0; x < kAdWarps; x += W) {
        const float f = ex2(sm.m[wi + x][h] - ref);
        add_scaled(acc, f, *reinterpret_cast<const float4*>(&sm.o[wi + x][h][d]));
        ll = fmaf(f, sm.l[wi + x][h], ll);
      }
      if (whole) {
        finish(a, b, h_item + wi * P * a.group + h, H, d, acc, ll, mm, sv);
      } else {
        float* to = part + wi * F::kPart;
        if (!dcheck(to >= a.parts && to + F::kPart <= a.parts + a.n_parts && h >= 0 && h < 8 * NT, a.err)) continue;
        *reinterpret_cast<float4*>(to + h * H + d) = acc;
        if (d == 0) {
          to[8 * NT * H + h] = mm;
          to[8 * NT * H + 8 * NT + h] = ll;
        }
      }
    }
    if (!whole) {
      // CTAs [c0, c1] hold tiles of this item: the CTA of unit x is
      // floor(((x + 1) * ctas - 1) / total)
      const int64_t c0 = ((item_w0 + kAdItemCost + 1) * ctas - 1) / total, c1 = (item_w1 * ctas - 1) / total;
      const int n_parts = (int)(c1 - c0) + 1;
      // A CTA's first segment went to its slot 0; the item's first CTA holds
      // the item as its first segment only if its range starts in the item.
      const bool second = c0 * total / ctas < item_w0;
      auto part_of = [&](int c) { return a.parts + (2 * (c0 + c) + (c == 0 && second ? 1 : 0)) * W * F::kPart; };
      // The last CTA to arrive at a counter merges: all parts at once, or, where a
      // thread would read more than kAdFlat pieces one behind the other, `by`
      // neighbours' into the first one's place, then those.
      const int by = n_parts * ((W * pieces + kAdThreads - 1) / kAdThreads) <= kAdFlat ? 1 : n_parts <= 64 ? 8 : 24;
      int from = 0, step = 1, count = n_parts;
      // the item's counter: a CTA is the first of at most one split item
      uint32_t* ticket = a.tickets + 3 * c0;
      if (by > 1) {
        from = (int)(cta - c0) / by * by;
        count = min(by, n_parts - from);
        ticket = a.tickets + 3 * (c0 + from) + (from ? 2 : 1);  // a CTA is past the first of at most one split item
      }
      for (;;) {
        __threadfence();
        __syncthreads();
        if (tid == 0 && !dcheck(ticket >= a.tickets && ticket < a.tickets + a.n_tickets, a.err)) last = 0;
        else if (tid == 0) {
          last = count == 1 || atomicAdd(ticket, 1u) == (uint32_t)(count - 1);
          if (last) *ticket = 0u;  // ready for the next call
        }
        __syncthreads();
        if (!last) break;
        __threadfence();
        const bool top = by == 1 || step > 1;
        if (top || count > 1) {
          // per head ("slot") of the item: the largest reference, each part's factor, the sum
          const int slots = W * heads;
          float* factor = reinterpret_cast<float*>(smem);  // [part][8 NT W], over the rings
          float* head_m = factor + count * 8 * NT * W;
          float* head_l = head_m + 8 * NT * W;
          auto stat_of = [&](int c, int slot) {
            const int wi = W == 2 && slot >= heads;
            return part_of(from + c * step) + wi * F::kPart + 8 * NT * H + slot - wi * heads;
          };
          constexpr int kSlots = 8 * NT * W / kAdWarps;  // of a warp: the first 32 parts' loaded at once
          float m0[kSlots], l0[kSlots];
#pragma unroll
          for (int x = 0; x < kSlots; ++x) {
            const int slot = warp + x * kAdWarps;
            const bool on = slot < slots && lane < count;
            const float* src = stat_of(on ? lane : 0, on ? slot : 0);
            m0[x] = on ? __ldcg(src) : -INFINITY;
            l0[x] = on ? __ldcg(src + 8 * NT) : 0.0f;
          }
#pragma unroll
          for (int x = 0; x < kSlots; ++x) {
            const int slot = warp + x * kAdWarps;
            if (slot >= slots) break;
            float mm = m0[x];
            for (int c = lane + 32; c < count; c += 32) mm = fmaxf(mm, __ldcg(stat_of(c, slot)));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
            const float ref = mm == -INFINITY ? 0.0f : mm;
            const float f0 = ex2(m0[x] - ref);
            if (lane < count) factor[lane * 8 * NT * W + slot] = f0;
            float ll = f0 * l0[x];
            for (int c = lane + 32; c < count; c += 32) {
              const float* src = stat_of(c, slot);
              const float f = ex2(__ldcg(src) - ref);
              factor[c * 8 * NT * W + slot] = f;
              ll = fmaf(f, __ldcg(src + 8 * NT), ll);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
            if (lane == 0) {
              head_m[slot] = mm;
              head_l[slot] = ll;
            }
          }
          __syncthreads();
          for (int i = tid; i < W * pieces; i += kAdThreads) {
            const int wi = W == 2 && i >= pieces, h = (i - wi * pieces) / (H / 4), d = i % (H / 4) * 4, slot = wi * heads + h;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int c = 0; c < count; ++c)
              add_scaled(acc, factor[c * 8 * NT * W + slot], __ldcg(reinterpret_cast<const float4*>(part_of(from + c * step) + wi * F::kPart + h * H + d)));
            if (top) {
              finish(a, b, h_item + wi * P * a.group + h, H, d, acc, head_l[slot], head_m[slot], sv);
            } else {
              float* to = part_of(from) + wi * F::kPart;
              if (!dcheck(to >= a.parts && to + F::kPart <= a.parts + a.n_parts && h >= 0 && h < 8 * NT, a.err)) continue;
              *reinterpret_cast<float4*>(to + h * H + d) = acc;
              if (d == 0) {
                to[8 * NT * H + h] = head_m[slot];
                to[8 * NT * H + 8 * NT + h] = head_l[slot];
              }
            }
          }
        }
        if (top) break;
        from = 0, step = by, count = (n_parts + by - 1) / by;
        ticket = a.tickets + 3 * c0;
      }
    }
    __syncthreads();  // sm is free for the next segment
    first_segment = false;
  }
}


int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  return n;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kAdMaxLen = (int64_t)1 << 30;  // 32-bit key numbers, two tiles of headroom

// fn(Form) of the form that a call's shape takes.  Heads of 64 run as pairs where
// their number is even: rows of 64 bytes, a KV head's alone, came at 3.0 TB/s
// where rows of 128 come at 5.5.
template <int W, class Fn>
auto with_shape(int64_t kv_heads, int64_t group, int64_t head_dim, Fn fn) {
  if (head_dim == 128) return group <= 4 ? fn(Form<128, 1, 1, 1, W>{}) : group <= 8 ? fn(Form<128, 1, 2, 1, W>{}) : fn(Form<128, 2, 2, 1, W>{});
  if (kv_heads % 2 == 0 && group <= 8)
    return group <= 2 ? fn(Form<128, 1, 1, 2, W>{}) : group <= 4 ? fn(Form<128, 1, 2, 2, W>{}) : fn(Form<128, 2, 2, 2, W>{});
  return group <= 8 ? fn(Form<64, 1, 2, 1, 1>{}) : fn(Form<64, 2, 2, 1, 1>{});
}

// Two neighbouring heads' rows of 128 bytes at a time come faster (256 caches to 4096:
// 185 us instead of 208; on a GPU with faster memory 182 instead of 189), but an item of
// two has more to merge where CTAs share it: taken from two items a CTA (with
// one, 256 caches of 2000 to 2100 and 4 KV heads, 96 instead of 94 us).  Items of four
// took 195 and 110 us for the two.
constexpr int64_t kAdTwoHeads = 2 * 3;  // items an SM (three CTAs)
template <class Fn>
auto with_form(int64_t batch, int64_t kv_heads, int64_t group, int64_t head_dim, Fn fn) {
  const int64_t rows = head_dim == 64 && group <= 8 && kv_heads % 2 == 0 ? kv_heads / 2 : kv_heads;
  return rows % 2 == 0 && batch * (rows / 2) >= kAdTwoHeads * sm_count() ? with_shape<2>(kv_heads, group, head_dim, fn)
                                                                             : with_shape<1>(kv_heads, group, head_dim, fn);
}

// The workspace starts with the items' counters: an area of one size for every
// shape, so that one workspace can serve several (partials never land on counters).
constexpr int kAdMaxCtas = 4;
int64_t ticket_count() { return (int64_t)sm_count() * kAdMaxCtas * 3; }
int64_t ticket_bytes() { return (ticket_count() * 4 + 255) / 256 * 256; }

template <class F>
cudaError_t launch_decode(AdArgs a, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  a.hkv /= F::P;
  a.sub = (F::P * a.group + 8 * F::NT - 1) / (8 * F::NT);
  static_assert(F::kCtas <= kAdMaxCtas);
  a.tickets = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + ticket_bytes());
  a.n_tickets = ticket_count();
  a.n_parts = ((int64_t)workspace_bytes - ticket_bytes()) / 4;
#ifdef FP8RL_DEBUG  // only the store checks look at it
  a.err = device_error_word();
  if (!a.err) return cudaErrorUnknown;
#endif
  const size_t smem = ad_smem<F>() + ((size_t)a.batch + 1) * 8;
  // the attribute lives in the context: set once per device and context, for the largest batch
  static std::atomic<uint64_t> ready[64];
  int dev = 0;
  const uint64_t ctx = current_context_id();
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ctx) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire) != ctx) {
    e = cudaFuncSetAttribute(attn_decode_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(ad_smem<F>() + (kAdMaxBatch + 1) * 8));
    if (e != cudaSuccess) return e;
    ready[dev].store(ctx, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() * F::kCtas));
  cfg.blockDim = dim3(kAdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<F>, a);
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

extern "C" FP8RL_API size_t fp8rl_attn_decode_workspace_size(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128)) return 0;
  return with_form(kAdMaxBatch, kv_heads, q_heads / kv_heads, head_dim, [](auto f) {  // the larger of a batch's forms
    using F = decltype(f);
    return (size_t)(ticket_bytes() + 2 * (int64_t)sm_count() * F::kCtas * F::W * F::kPart * 4);
  });
}

extern "C" FP8RL_API fp8rl_status fp8rl_attn_decode(const void* q_bf16, int64_t ldq, int64_t batch, int64_t q_heads,
                                                    int64_t kv_heads, int64_t head_dim, const void* k_cache,
                                                    const void* v_cache, int64_t ld_cache, int64_t num_slots,
                                                    const int32_t* d_block_table, int64_t ldt, int64_t max_blocks,
                                                    int64_t block_size, const int32_t* d_lens, const float* d_scales,
                                                    float softmax_scale, void* out_bf16, int64_t ldo, float* d_lse,
                                                    void* d_workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || num_slots < 0 || max_blocks < 0 || block_size < 1 ||
      ldt < max_blocks || q_heads % kv_heads != 0 || !(softmax_scale > 0.0f) || !(softmax_scale <= FLT_MAX))
    return FP8RL_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return FP8RL_ERR_SHAPE;
  if (q_heads > 65536 || ldq < q_heads * head_dim || ldo < q_heads * head_dim || ld_cache < kv_heads * head_dim)
    return FP8RL_ERR_INVALID_ARG;
  if (batch == 0) return FP8RL_OK;
  if (!q_bf16 || !d_lens || !out_bf16 || !d_scales || !d_workspace) return FP8RL_ERR_INVALID_ARG;
  if (max_blocks > 0 && (!d_block_table || !k_cache || !v_cache)) return FP8RL_ERR_INVALID_ARG;
  // cache rows are addressed by a 32-bit count of 16-byte units
  if (ld_cache > 0 && num_slots > ((int64_t)1 << 36) / ld_cache) return FP8RL_ERR_SHAPE;
  if (batch > kAdMaxBatch || block_size > kAdMaxLen || max_blocks > kAdMaxLen / block_size) return FP8RL_ERR_SHAPE;
  if (workspace_bytes < fp8rl_attn_decode_workspace_size(q_heads, kv_heads, head_dim)) return FP8RL_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 4) || ldq % 2 != 0 || !aligned(k_cache, 16) || !aligned(v_cache, 16) || ld_cache % 16 != 0 ||
      !aligned(out_bf16, 8) || ldo % 4 != 0 || !aligned(d_block_table, 4) || !aligned(d_lens, 4) || !aligned(d_scales, 4) ||
      !aligned(d_lse, 4) || !aligned(d_workspace, 16))
    return FP8RL_ERR_ALIGNMENT;
  AdArgs a{};
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.table = d_block_table;
  a.lens = d_lens;
  a.scales = d_scales;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.lse = d_lse;
  a.ldq = ldq, a.num_slots = num_slots, a.ldt = ldt, a.ldo = ldo;
  a.ldc16 = (uint32_t)(ld_cache / 16);
  a.batch = (int32_t)batch, a.hq = (int32_t)q_heads, a.hkv = (int32_t)kv_heads;
  a.group = (int32_t)(q_heads / kv_heads);
  a.page = (int32_t)block_size;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (block_size == (int64_t)1 << i) a.page_shift = i;
  a.max_len = (int32_t)(max_blocks * block_size);
  a.softmax_scale = softmax_scale;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = with_form(batch, kv_heads, a.group, head_dim, [&](auto f) { return launch_decode<decltype(f)>(a, d_workspace, workspace_bytes, cs); });
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FP8RL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}
