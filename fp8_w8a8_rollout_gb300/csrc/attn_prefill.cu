// attn_prefill.cu -- causal attention over whole prompts, packed, with grouped
// heads: the attention between the W8A8 linears of a prefill (queries, keys
// and values are column ranges of the qkv linear's bf16 output).
//
// For sequence position i and the keys j <= i of its sequence:
//   s_ij = softmax_scale (q_i . k_j),  out_i = sum_j exp(s_ij - m_i) v_j / l_i,
//   l_i = sum_j exp(s_ij - m_i),       lse_i = m_i + ln l_i.
//
// Compute-bound (4 d flop per query-key pair and head): both products run on
// tcgen05 with fp32 accumulators in TMEM.  GB300, 32 query and 8 KV heads of
// 128: 8192 tokens 324 us alone (1.70 PFLOP/s, 0.89 of the measured burst rate)
// and 352 back to back (the power limit); 24 packed prompts of up to 2048, 32
// and 4 heads, 192 to 199 us back to back (1.11 to 1.15 PFLOP/s; 180 by the
// device, one call alone).  With heads of 64, where the softmax weighs twice as
// much against the products, 274 and 148 us (1.00 and 0.74).  What is left: a tile's softmax
// (about 1.4 us) and its products (0.55 us) take turns, and the two tiles
// hide most of one another's, not all.  One CTA per SM walks work items; an
// item is two tiles of 128 query rows of one KV head.  A tile's rows are
// (position, head) pairs: the query heads that share a KV head lie side by
// side in memory, so a TMA box of `pack` heads x 128 / pack positions fills a
// tile and one pass over the keys serves all of them (and the diagonal
// wastes at most a key tile per 128 / pack positions).
//
// Roles: a TMA thread streams 128-key tiles of K and V through a ring of five
// 32 KB stages; an MMA thread issues S = Q K^T (shared memory x shared memory)
// and O += P V (P from TMEM, V as it lies in memory, d contiguous) for the two
// tiles in turn, so the tensor cores multiply for one tile while the other's
// softmax runs; two warpgroups do the softmax, a thread per row, with no
// exchange between threads: the row's 128 scores to registers, their maximum,
// exp2, the row sum, and P as bf16 back over the scores' columns.  The running
// maximum is allowed to lag by 8 (base 2): only when a row grows past that is
// its O read from TMEM, rescaled and written back, before P is handed over.
//
// P is rounded to bf16 because both operands of a tcgen05 f16-kind product
// have one type and V is bf16; l sums the unrounded fp32 values.  Statistics
// and accumulators are fp32, the output is rounded once.
//
// An output depends on its own positions alone: in the key tiles that an item
// does not see whole, a warp zeroes the value rows past the item's end and takes
// non-finite values out of the partly visible ones before they are multiplied
// (0 * NaN); the rows that see such a value get its term when they are stored, a
// handful of operations whatever the prompt's length.
//
// The plan (one per step, used by every layer) lists the items, longest key
// range first; CTAs take them in snake order, which evens the causal lengths
// out; a warp of its own reads it and hands the items to the others.  The
// kernel's size matters: at 73 KB of code, waits spelled out at every site, a
// fifth of the issue slots' stalls were instruction fetches (one call alone, 8192
// tokens 334 us, packed prompts 190; at 55 KB 324 and 174).  Every wait is bounded.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <mutex>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8rl {
namespace {

using namespace ptx;

constexpr int kApThreads = 512;     // warps 0-3: roles, 4-7 and 8-11: softmax of tile 0 and 1, 12-15: outputs
constexpr int kApTile = 128;        // query rows of a tile, keys of a key tile
constexpr int kApStages = 5;
// shares of the launch's 128 x 512 registers (setmaxnreg: their sum may not exceed it)
constexpr int kApRoleRegs = 88, kApSoftmaxRegs = 176, kApOutRegs = 72;
static_assert(128 * (kApRoleRegs + 2 * kApSoftmaxRegs + kApOutRegs) <= 128 * kApThreads, "register split");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;
constexpr uint32_t kApTimeoutNs = 2000000000u;  // of a 32-bit nanosecond counter

// a step of the longest item's waits stays well inside the limit (2^19 key tiles of about 1.5 us)
constexpr int64_t kApMaxTokens = (int64_t)1 << 26;

// the plan: a header, then one int4 per item {first token of the sequence,
// its length, first position of the item, 0}
struct PlanHeader {
  int32_t items, span, total, batch;  // span: positions of an item
};

struct ApArgs {
  const int4* plan;
  const uint16_t *q, *k, *v;  // for the terms of non-finite values (the tensor maps serve all others)
  int64_t ldq, ldk, ldv;
  uint16_t* out;
  float* lse;  // or null
  uint32_t* err;
  int64_t ldo;
  int32_t capacity, total, hq, hkv, group, pack;
  int32_t wide;  // output rows start on 32-byte boundaries
  float softmax_scale;
};

template <int D>
struct ApCfg {
  static constexpr int kHalves = D / 64;                      // 64-column (128-byte) parts of a row
  static constexpr uint32_t kHalfBytes = kApTile * 128;       // 16 KB
  static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  static constexpr uint32_t kRing = 2 * kTileBytes;           // byte offset of the key/value stages
  static constexpr uint32_t kBook = kRing + kApStages * kTileBytes;
  static constexpr uint32_t kItems = kBook + 384;             // the items at hand
  static constexpr uint32_t kRows = kBook + 512;              // row sums of the two tiles for the output warps
  static constexpr uint32_t kMarks = kRows + 2 * kApTile * 8; // per item at hand, which of its positions have values taken out
  static constexpr uint32_t kSmem = kMarks + 128 + 384;       // alignment
  static constexpr uint32_t kTmemS = 0, kTmemO = 256;         // S of tile x at 128 x, O at 256 + 128 x
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Instruction descriptor of tcgen05.mma kind::f16: D fp32 (bits 4-5 = 1), A
// and B bf16 (bits 7-9, 10-12 = 1), A K-major, B K-major or (bit 16) with its
// N index contiguous, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// Descriptor of a B tile whose N index is contiguous: rows (K index) of 128
// swizzled bytes = 64 N elements; the next 64 N elements `half` bytes further
// (leading byte offset), the next 8 rows 1024 bytes further (stride byte offset).
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t saddr, uint32_t half) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(half >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// D[tmem] (+)= A[smem] * B[smem], one M x N x 16 bf16 step
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// the same with A in TMEM (row r in lane r, two bf16 per 32-bit column)
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// tcgen05.wait::ld that the loaded registers pass through, so that nothing
// that uses them is moved ahead of it
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 16 columns of this thread's lane, waited for
__device__ __forceinline__ void tmem_ld_32x32b_x16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// A bounded wait in few instructions (there are some thirty in the kernel,
// which has to fit the instruction cache): suspended tries until the phase
// completes, another thread has given up, or the limit runs out; then raises
// *abort, which the teardown reports.
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = timer_lo();
  while (!mbar_try_wait_suspend(bar, parity, 20000u)) {
    if (*abort) return false;
    if (timer_lo() - t0 > kApTimeoutNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

struct alignas(16) Item {
  int32_t start, len, pos0;  // sequence's first token, its length, first position
  int32_t head0, kvh;        // first query head, KV head
  int32_t n0, n1;            // key tiles of the two query tiles; n0 = 0: no more items
  int32_t pad;
  __device__ __forceinline__ int32_t n(int x) const { return x ? n1 : n0; }
};
constexpr int kApItems = 4;           // items handed out ahead
constexpr int kApItemReaders = 15;    // TMA, MMA, mender, 8 softmax and 4 output warps

// work index w: item w / heads, head part w % heads
__device__ __forceinline__ Item item_of(const ApArgs& a, uint32_t w, int32_t parts) {
  const uint32_t per = (uint32_t)(a.hkv * parts), at = w / per;
  const int4 p = a.plan[1 + at];
  const int32_t hp = (int32_t)(w - at * per);
  Item it;
  it.start = p.x;
  it.len = p.y;
  it.pos0 = p.z;
  it.kvh = hp / parts;
  it.head0 = it.kvh * a.group + (hp % parts) * a.pack;
  it.pad = 0;
  const int32_t span = kApTile / a.pack;
  auto tiles = [&](int32_t first) { return first < it.len ? (min(it.len, first + span) + kApTile - 1) / kApTile : 0; };
  it.n0 = tiles(it.pos0);
  it.n1 = tiles(it.pos0 + span);
  return it;
}

constexpr int kApMarks = 8;  // words of an item: a bit for each of its (at most 256) positions

__device__ __forceinline__ bool any_marks(uint32_t p) {
  uint32_t a, b, c, d;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(p) : "memory");
  return (a | b | c | d) != 0;
}

__device__ __forceinline__ bool non_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7F80u) == 0x7F80u; }

// The terms p_j v_j of the values that were taken out of the product, onto the
// stored output row of position `pos`: of marked positions up to its own, from
// the row's final reference maximum (times the scale).  p_j's factor 1 / sum is
// left out: the terms are infinities and NaN.
template <int D>
__device__ __forceinline__ void add_taken_out(const ApArgs& a, const Item& it, const volatile uint32_t* marks, int32_t pos,
                                              int32_t head, float mc, uint16_t* dst) {
  const float c = a.softmax_scale * kLog2e;
  const int32_t rel = pos - it.pos0;
  const uint16_t* q = a.q + ((int64_t)it.start + pos) * a.ldq + (int64_t)head * D;
  asm volatile("" ::: "memory");  // the row's stores, of other types, come first
#pragma unroll 1
  for (int32_t w = 0; w <= rel >> 5; ++w) {
    uint32_t m = marks[w];
    if (w == rel >> 5) m &= (2u << (rel & 31)) - 1u;
#pragma unroll 1
    for (; m; m &= m - 1u) {
      const int64_t token = (int64_t)it.start + it.pos0 + 32 * w + __ffs(m) - 1;
      const uint16_t* k = a.k + token * a.ldk + (int64_t)it.kvh * D;
      const uint16_t* v = a.v + token * a.ldv + (int64_t)it.kvh * D;
      float s = 0.0f;
#pragma unroll 1
      for (int d = 0; d < D; d += 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(q + d), y = *reinterpret_cast<const uint32_t*>(k + d);
        s = fmaf(bf16_hi(x), bf16_hi(y), fmaf(bf16_lo(x), bf16_lo(y), s));
      }
      const float p = ex2(fmaf(s, c, -mc));
#pragma unroll 1
      for (int d = 0; d < D; ++d)
        if (non_finite(v[d])) dst[d] = (uint16_t)bf16x2_rn(fmaf(p, bf16_lo(v[d]), bf16_lo(dst[d])), 0.0f);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kApThreads, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const ApArgs a) {
  using C = ApCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(base_ptr + C::kBook);
  uint64_t* kv_empty = kv_full + kApStages;
  uint64_t* q_full = kv_empty + kApStages;  // one per tile
  uint64_t* q_empty = q_full + 2;           // a tile's scores of an item are done
  uint64_t* s_full = q_empty + 2;           // scores of a tile in TMEM
  uint64_t* p_half = s_full + 2;            // half of P of a tile in TMEM, O rescaled (128 threads)
  uint64_t* p_full = p_half + 2;            // the other half
  uint64_t* o_full = p_full + 2;            // O of a tile finished
  uint64_t* l_full = o_full + 2;            // its row sums in shared memory (128 threads)
  uint64_t* o_empty = l_full + 2;           // both read by the output warps (128 threads)
  uint64_t* mended = o_empty + 2;           // the mender is done with a stage (one per stage, in the ring's phases)
  uint64_t* drain = mended + kApStages;
  uint64_t* item_full = drain + 1;          // an item's slot is filled
  uint64_t* item_empty = item_full + kApItems;  // every reader has copied it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_empty + kApItems);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  uint32_t* marks = reinterpret_cast<uint32_t*>(base_ptr + C::kMarks);  // [item slot][kApMarks]
  volatile int* abortv = abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kApStages; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&mended[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), 2);  // the products', the mender's
    }
    mbar_init(smem_u32(drain), 1);
    for (int i = 0; i < kApItems; ++i) {
      mbar_init(smem_u32(&item_full[i]), 1);
      mbar_init(smem_u32(&item_empty[i]), kApItemReaders);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&q_full[x]), 1);
      mbar_init(smem_u32(&q_empty[x]), 1);
      mbar_init(smem_u32(&s_full[x]), 1);
      mbar_init(smem_u32(&p_half[x]), kApTile);
      mbar_init(smem_u32(&p_full[x]), kApTile);
      mbar_init(smem_u32(&o_full[x]), 1);
      mbar_init(smem_u32(&l_full[x]), kApTile);
      mbar_init(smem_u32(&o_empty[x]), kApTile);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything above touches this CTA alone; from here on the kernel before counts
  grid_dep_launch_dependents();
  grid_dep_wait();
  float2* row_sum = reinterpret_cast<float2*>(base_ptr + C::kRows);  // [tile][row]: reference maximum, sum

  const PlanHeader head = *reinterpret_cast<const PlanHeader*>(a.plan);
  const int32_t parts = a.group / a.pack;
  const bool fits = head.span == 2 * kApTile / a.pack && head.total == a.total && head.items >= 0 && head.items <= a.capacity;
  if (!fits && threadIdx.x == 0 && a.err) atomicOr(a.err, kErrDeviceCheck);
  const uint32_t work = fits ? (uint32_t)head.items * (uint32_t)(a.hkv * parts) : 0u;  // the host keeps it below 2^31
  const uint32_t grid = gridDim.x;
  // This CTA's items reach its warps through a ring of slots that a warp of
  // its own fills ahead (the plan's latency and the divisions off everyone's
  // path).  take() copies the i-th one; false past the end or after an abort.
  Item* slots = reinterpret_cast<Item*>(base_ptr + C::kItems);
  auto take = [&](uint32_t& i, Item& it, bool arrive) {
    const uint32_t slot = i % kApItems;
    if (!wait_for(smem_u32(&item_full[slot]), (i / kApItems) & 1, abortv)) return false;
    it = slots[slot];
    ++i;
    if (arrive) mbar_arrive(smem_u32(&item_empty[slot]));
    return it.n0 > 0;
  };
  // the same for a whole warp
  auto take_warp = [&](uint32_t& i, Item& it) {
    const bool got = take(i, it, false);
    const bool all = __all_sync(0xffffffffu, got);  // (every lane has its copy)
    if (lane == 0) mbar_arrive(smem_u32(&item_empty[(i - 1) % kApItems]));
    return all;
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kApRoleRegs));
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        uint32_t g = 0;
        uint32_t q_issued0 = 0, q_issued1 = 0;
        bool alive = true;
        auto load_kv = [&](const CUtensorMap* map, const Item& it, int32_t j) {
          const int s = g % kApStages;
          if (!wait_for(smem_u32(&kv_empty[s]), ((g / kApStages) & 1) ^ 1, abortv)) return false;
          const uint32_t bar = smem_u32(&kv_full[s]);
          mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(base + C::kRing + s * C::kTileBytes + h * C::kHalfBytes, map, 64 * h, it.kvh, it.start + j * kApTile, bar);
          ++g;
          return true;
        };
        auto load_q = [&](int x, const Item& it) {
          if (!wait_for(smem_u32(&q_empty[x]), ((x ? q_issued1 : q_issued0) & 1) ^ 1, abortv)) return false;
          const uint32_t bar = smem_u32(&q_full[x]);
          mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(base + x * C::kTileBytes + h * C::kHalfBytes, &map_q, 64 * h, it.head0,
                        it.start + it.pos0 + x * (kApTile / a.pack), bar);
          if (x) ++q_issued1;
          else ++q_issued0;
          return true;
        };
        Item it;
        for (uint32_t i = 0; alive && take(i, it, true);) {
          const int32_t n = max(it.n0, it.n1);
          // K of key tile 0, V of 0, K of 1, ...: the order of their use; the
          // queries around the first (the first tile's scores need no more)
#pragma unroll 1
          for (int32_t t = 0; t < 2 * n && alive; ++t) {
            if (t < 2 && it.n(t) > 0) alive = load_q(t, it);
            alive = alive && load_kv(t & 1 ? &map_v : &map_k, it, t >> 1);
          }
        }
        if (*abortv) {
          // let the copies still in flight land before shared memory is released
          for (uint32_t j = g > (uint32_t)kApStages ? g - kApStages : 0; j < g; ++j)
            mbar_wait_bounded(smem_u32(&kv_full[j % kApStages]), (j / kApStages) & 1, nullptr, nullptr, 10000000ull);
          if (q_issued0) mbar_wait_bounded(smem_u32(&q_full[0]), (q_issued0 - 1) & 1, nullptr, nullptr, 10000000ull);
          if (q_issued1) mbar_wait_bounded(smem_u32(&q_full[1]), (q_issued1 - 1) & 1, nullptr, nullptr, 10000000ull);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer: one elected thread
      if (elect_one()) {
        constexpr uint32_t kDescQk = idesc_bf16(kApTile, kApTile, false), kDescPv = idesc_bf16(kApTile, D, true);
        // descriptors differ in their address field alone (units of 16 bytes)
        const uint64_t q_desc = sw128_kmajor_desc(base), k_desc = sw128_kmajor_desc(base + C::kRing),
                       v_desc = sw128_nmajor_desc(base + C::kRing, C::kHalfBytes);
        uint32_t stage = 0, parity = 0;  // of the next tile in the ring
        auto advance = [&] {
          if (++stage == kApStages) stage = 0, parity ^= 1;
        };
        uint32_t q_phase = 0, p_phase = 0, o_phase = 3;  // bit x: the parity that tile x waits for next
        bool alive = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          return wait_for(smem_u32(bar), parity, abortv);
        };
        auto scores = [&](int x, uint32_t stage) {  // S_x = Q_x K^T
          const uint64_t qd = q_desc + x * (C::kTileBytes >> 4), kd = k_desc + stage * (C::kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k >> 2) * C::kHalfBytes + (k & 3) * 32) >> 4;
            mma_bf16_ss(tmem + C::kTmemS + 128 * x, qd + at, kd + at, kDescQk, k > 0);
          }
          mma_commit(smem_u32(&s_full[x]));
        };
        auto values = [&](int x, uint32_t stage, int half, bool first) {  // O_x (+)= P_x V, 64 keys
          const uint64_t vd = v_desc + stage * (C::kTileBytes >> 4);
#pragma unroll
          for (int i = 0; i < kApTile / 32; ++i) {
            const int k = half * (kApTile / 32) + i;
            mma_bf16_ts(tmem + C::kTmemO + 128 * x, tmem + C::kTmemS + 128 * x + 8 * k, vd + k * (2048 >> 4), kDescPv, !first || k > 0);
          }
        };
        // S_x of key tile j (of n) of an item from ring stage `stage`; the
        // last one frees Q_x
        auto item_scores = [&](int32_t n, int x, int32_t j, uint32_t stage) {
          if (j == 0) {
            if (!wait(&q_full[x], q_phase >> x & 1)) return false;
            q_phase ^= 1u << x;
            tc_fence_after();
          }
          scores(x, stage);
          if (j + 1 == n) mma_commit(smem_u32(&q_empty[x]));
          return true;
        };
        uint32_t i = 0;
        Item it, next;
        bool more = take(i, it, true);
        if (more) {
          alive = wait(&kv_full[0], 0);
          advance();
#pragma unroll 1
          for (int x = 0; x < 2; ++x) alive = alive && (it.n(x) == 0 || item_scores(it.n(x), x, 0, 0));
          mma_commit(smem_u32(&kv_empty[0]));
        }
        while (more && alive) {
          const int32_t n = max(it.n0, it.n1);
          more = take(i, next, true);
          for (int32_t j = 0; j < n && alive; ++j) {
            // (value tiles that the item does not see whole come by way of the mender)
            const uint32_t vs = stage;
            alive = wait(j >= it.pos0 / kApTile ? &mended[vs] : &kv_full[vs], parity);
            advance();
            // The scores to issue behind this step's products: of the next key
            // tile, or of the next item's first one, so that its softmax starts
            // while this item ends.
            const bool last = j + 1 == n, ahead = !last || more;
            const uint32_t kn = stage, kn_parity = parity;
            bool arrived = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (j < it.n(x)) {
                // the previous item's outputs have left O_x
                if (j == 0) {
                  alive = wait(&o_empty[x], o_phase >> x & 1);
                  o_phase ^= 1u << x;
                }
                alive = alive && wait(&p_half[x], p_phase >> x & 1);
                if (!alive) break;
                tc_fence_after();
                values(x, vs, 0, j == 0);
                alive = wait(&p_full[x], p_phase >> x & 1);
                p_phase ^= 1u << x;
                if (!alive) break;
                tc_fence_after();
                values(x, vs, 1, false);
                if (j + 1 == it.n(x)) mma_commit(smem_u32(&o_full[x]));
              }
              if (x == 1) mma_commit(smem_u32(&kv_empty[vs]));
              const int32_t to_n = last ? next.n(x) : it.n(x), tj = last ? 0 : j + 1;
              if (ahead && tj < to_n) {
                if (!arrived) alive = wait(&kv_full[kn], kn_parity);
                arrived = true;
                alive = alive && item_scores(to_n, x, tj, kn);
                if (!alive) break;
              }
            }
            if (!alive) break;
            if (ahead) {
              mma_commit(smem_u32(&kv_empty[kn]));
              advance();
            }
          }
          it = next;
        }
        // every product issued so far has finished with shared memory and TMEM
        mma_commit(smem_u32(drain));
        mbar_wait_bounded(smem_u32(drain), 0, nullptr, a.err, kApTimeoutNs);  // (whoever else gave up)
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ items: snake order over the plan
      if (lane == 0) {
        uint32_t i = 0;
        Item it;
        for (uint32_t r = 0;; ++r) {
          // round r is index r * grid plus this CTA's place in the round
          const uint32_t w = r * grid + ((r & 1) ? grid - 1 - blockIdx.x : blockIdx.x);
          const bool end = r * grid >= work;
          if (!end) {
            if (w >= work) continue;
            it = item_of(a, w, parts);
            if (it.n0 == 0) continue;
          } else {
            it.n0 = it.n1 = 0;
          }
          const uint32_t slot = i % kApItems;
          if (!wait_for(smem_u32(&item_empty[slot]), ((i / kApItems) & 1) ^ 1, abortv)) break;
          slots[slot] = it;
          mbar_arrive(smem_u32(&item_full[slot]));
          ++i;
          if (end) break;
        }
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------------ mender
      // A probability of 0 does not cancel a NaN or an infinity.  In the key
      // tiles that an item does not see whole, the value rows past its last
      // position (later ones, or another sequence's) are zeroed before they are
      // multiplied; in those from its first position on, which some of its rows see
      // and some do not, non-finite values are zeroed and their positions marked
      // for the output warps.  Every tile passes here and is held until it has: no
      // phase of the ring is missed, and none is signalled twice before the MMA
      // thread has seen it.  (An item's marks are written when its own tile is
      // mended, so never while the item four before it is still being stored: the
      // queries between them wait for its outputs.)
      uint32_t stage = 0, parity = 0;
      bool alive = true;
      Item it;
      for (uint32_t i = 0; alive && take_warp(i, it);) {
        const int32_t n = max(it.n0, it.n1);
        const int32_t end = min(it.len, it.pos0 + 2 * (kApTile / a.pack));
        for (int32_t t = 0; t < 2 * n; ++t) {
          alive = __all_sync(0xffffffffu, wait_for(smem_u32(&kv_full[stage]), parity, abortv));
          if (!alive) break;
          const int32_t k0 = (t >> 1) * kApTile;
          if ((t & 1) && k0 + kApTile > it.pos0) {
            uint8_t* tile = base_ptr + C::kRing + stage * C::kTileBytes;
            const int32_t r0 = max(it.pos0 - k0, 0), r1 = min(end - k0, kApTile);
            // the tile's own words: an item has 256 positions in two tiles, or fewer in one
            uint32_t* words = marks + ((i - 1) % kApItems) * kApMarks;
            if (lane < kApMarks / 2) words[(k0 > it.pos0 ? kApMarks / 2 : 0) + lane] = 0u;
            uint32_t worst = 0;  // packed magnitudes
            for (int32_t e = r0 * 8 + lane; e < kApTile * 8; e += 32)
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h) {
                uint4* p = reinterpret_cast<uint4*>(tile + h * C::kHalfBytes + e * 16);
                if (e < r1 * 8) worst = absmax_u4(worst, *p);
                else *p = make_uint4(0u, 0u, 0u, 0u);
              }
            if (__any_sync(0xffffffffu, max(worst & 0xFFFFu, worst >> 16) >= 0x7F80u)) {
              __syncwarp();
#pragma unroll 1
              for (int32_t e = r0 * 8 + lane; e < r1 * 8; e += 32)
#pragma unroll 1
                for (int h = 0; h < 4 * C::kHalves; ++h) {
                  uint32_t* p = reinterpret_cast<uint32_t*>(tile + (h >> 2) * C::kHalfBytes + e * 16) + (h & 3);
                  const uint32_t keep = (non_finite(*p) ? 0u : 0xFFFFu) | (non_finite(*p >> 16) ? 0u : 0xFFFF0000u);
                  if (keep == 0xFFFFFFFFu) continue;
                  *p &= keep;
                  const int32_t rel = k0 + (e >> 3) - it.pos0;
                  atomicOr(&words[rel >> 5], 1u << (rel & 31));
                }
            }
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&mended[stage]));
            mbar_arrive(smem_u32(&kv_empty[stage]));
          }
          if (++stage == kApStages) stage = 0, parity ^= 1;
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kApSoftmaxRegs));
    const int x = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + C::kTmemS + 128 * x, to = tmem + lanes + C::kTmemO + 128 * x;
    const float c = a.softmax_scale * kLog2e;
    const uint64_t c2 = f32x2(c, c);
    // While a row's scores are all -inf its p is 0: the reference is tested for that,
    // or starts finite.  The two differ in the code's layout alone: 8192 tokens of 32 / 8 heads
    // of 64 274 us tested, 282 started finite; heads of 128 327 and 322.
    constexpr bool kRefTested = D == 64;
    uint32_t s_seen = 0, o_seen = 0;
    bool alive = true;
    Item it;
    for (uint32_t i = 0; alive && take_warp(i, it);) {
      const int32_t n = it.n(x);
      if (n == 0) continue;
      const int32_t first = it.pos0 + x * (kApTile / a.pack), pos = first + row / a.pack;
      float mc = kRefTested ? -INFINITY : -FLT_MAX;  // reference maximum times c
      uint64_t l2[4];        // the row's sum, in eight strands
#pragma unroll
      for (int i = 0; i < 4; ++i) l2[i] = f32x2(0.0f, 0.0f);
      for (int32_t j = 0; j < n; ++j) {
        alive = wait_for(smem_u32(&s_full[x]), s_seen & 1, abortv);
        ++s_seen;
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
        tc_fence_after();
        // the row's scores, in quarters; the maximum of the first two while the
        // others arrive
        uint32_t s[4][32];
        const bool edge = j * kApTile + kApTile - 1 > first;  // a key tile that reaches past the tile's first position
        const int32_t lim = pos - j * kApTile;                // there, keys 0 .. lim of the tile count
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto mask = [&](int q) {
          if (edge) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * q + i > lim) s[q][i] = 0xFF800000u;
          }
        };
        auto largest = [&](int q) {
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], __uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1]));
        };
        // P of a quarter into TMEM, and its sum into l2
        auto exponentials = [&](int q) {
          const float ref = kRefTested && mc == -INFINITY ? 0.0f : mc;
          const uint64_t nm2 = f32x2(-ref, -ref);
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t y = fma_f32x2(f32x2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, nm2);
            float y0, y1;
            f32x2_unpack(y, y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            l2[i & 3] = add_f32x2(l2[i & 3], f32x2(y0, y1));
            p[i] = bf16x2_rn(y0, y1);
          }
          tmem_st_32x32b_x16(ts + 16 * q, p);
        };
        tmem_ld_32x32b_x32(ts, s[0]);
        tmem_ld_32x32b_x32(ts + 32, s[1]);
        tmem_wait_ld_regs(s[0]);
        tmem_wait_ld_regs(s[1]);
        tmem_ld_32x32b_x32(ts + 64, s[2]);
        tmem_ld_32x32b_x32(ts + 96, s[3]);
        mask(0);
        mask(1);
        largest(0);
        largest(1);
        tmem_wait_ld_regs(s[2]);
        tmem_wait_ld_regs(s[3]);
        mask(2);
        mask(3);
        largest(2);
        largest(3);
        const float big = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
        const bool grow = big > mc + kRescale;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(mc - big) : 1.0f;  // 0 for the first key tile
          if (grow) mc = big;
          const uint64_t f2 = f32x2(f, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) l2[i] = mul_f32x2(l2[i], f2);
          if (j > 0) {
            // O holds the products up to j - 1 (their completion came before s_full's)
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t o[16];
              tmem_ld_32x32b_x16_wait(to + 16 * i, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(to + 16 * i, o);
            }
          }
        }
        exponentials(0);
        exponentials(1);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&p_half[x]));
        exponentials(2);
        exponentials(3);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[x]));
      }
      if (!alive) break;
      // the row's sum for the output warps, once they have read the previous item's
      alive = __all_sync(0xffffffffu, wait_for(smem_u32(&o_empty[x]), (o_seen++ & 1) ^ 1, abortv));
      if (!alive) break;
      float la, lb;
      f32x2_unpack(add_f32x2(add_f32x2(l2[0], l2[1]), add_f32x2(l2[2], l2[3])), la, lb);
      row_sum[x * kApTile + row] = make_float2(mc, la + lb);
      mbar_arrive(smem_u32(&l_full[x]));
    }
  } else {
    // ------------------------------------------------------------ outputs: thread = row, the tiles in turn
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kApOutRegs));
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t phase = 0;  // bit x: the parity that tile x waits for next
    bool alive = true;
    Item it;
    for (uint32_t i = 0; alive && take_warp(i, it);) {
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        if (it.n(x) == 0) continue;
        alive = wait_for(smem_u32(&l_full[x]), phase >> x & 1, abortv) && wait_for(smem_u32(&o_full[x]), phase >> x & 1, abortv);
        phase ^= 1u << x;
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
        tc_fence_after();
        const float2 ml = row_sum[x * kApTile + row];
        const float inv = 1.0f / ml.y;
        const int32_t pos = it.pos0 + x * (kApTile / a.pack) + row / a.pack, head = it.head0 + row % a.pack;
        const int64_t token = (int64_t)it.start + pos;
        const bool store = pos < it.len && dcheck(token < a.total && head < a.hq, a.err);
        uint16_t* dst = a.out + token * a.ldo + (int64_t)head * D;
        // (the second words are those of an item's second 128 positions: the second tile's)
        const uint32_t* words = marks + ((i - 1) % kApItems) * kApMarks;
        const bool taken_out = any_marks(smem_u32(words)) || (x == 1 && a.pack == 1 && any_marks(smem_u32(words + kApMarks / 2)));
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tmem + lanes + C::kTmemO + 128 * x + 32 * e, o);
          tmem_wait_ld_regs(o);
          uint32_t v[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = bf16x2_rn(__uint_as_float(o[2 * q]) * inv, __uint_as_float(o[2 * q + 1]) * inv);
          if (e == D / 32 - 1) {  // O and the sums have been read: the next item may write them
            tc_fence_before();
            mbar_arrive(smem_u32(&o_empty[x]));
          }
          if (store) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 lo = make_uint4(v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3]);
              const uint4 hi = make_uint4(v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]);
              uint16_t* to = dst + 32 * e + 16 * q;
              if (a.wide) {
                st_global_v8(to, lo, hi);
              } else {
                *reinterpret_cast<uint4*>(to) = lo;
                *reinterpret_cast<uint4*>(to + 8) = hi;
              }
            }
          }
        }
        if (store && a.lse) a.lse[token * a.hq + head] = fmaf(ml.x, kLn2, logf(ml.y));
        if (taken_out) {
          if (store) add_taken_out<D>(a, it, words, pos, head, ml.x, dst);
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abortv) atomicOr(a.err, kErrTimeout);
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;
constexpr int kPlanLevels = 2048;

// One CTA: items of every sequence sorted by their number of key tiles, the
// most first (a counting sort over at most 2048 levels; the order among
// equals is free: it only says which CTA computes an item).
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const int32_t* __restrict__ cu, int32_t batch, int32_t total,
                                                                int32_t span, int32_t capacity, int4* __restrict__ plan) {
  __shared__ int32_t count[kPlanLevels];
  __shared__ int32_t warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t top = (total + kApTile - 1) / kApTile;
  int shift = 0;
  while ((top >> shift) >= kPlanLevels) ++shift;
  for (int i = tid; i < kPlanLevels; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  auto each = [&](auto&& f) {
    for (int32_t b = warp; b < batch; b += kPlanThreads / 32) {
      const int32_t start = min(max(cu[b], 0), total), end = min(max(cu[b + 1], start), total);
      for (int32_t p = lane * span; p < end - start; p += 32 * span) {
        const int32_t tiles = (min(end - start, p + span) + kApTile - 1) / kApTile;
        f(kPlanLevels - 1 - (tiles >> shift), start, end - start, p);
      }
    }
  };
  each([&](int level, int32_t, int32_t, int32_t) { atomicAdd(&count[level], 1); });
  __syncthreads();
  // exclusive scan, two levels a thread
  const int32_t c0 = count[2 * tid], c1 = count[2 * tid + 1];
  int32_t v = c0 + c1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int32_t s = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const int32_t before = (warp ? warp_sum[warp - 1] : 0) + v - c0 - c1;
  count[2 * tid] = before;
  count[2 * tid + 1] = before + c0;
  const int32_t items = warp_sum[31];
  __syncthreads();
  each([&](int level, int32_t start, int32_t len, int32_t p) {
    const int32_t at = atomicAdd(&count[level], 1);
    if (at < capacity) plan[1 + at] = make_int4(start, len, p, 0);
  });
  if (tid == 0) *reinterpret_cast<PlanHeader*>(plan) = PlanHeader{min(items, capacity), span, total, batch};
}

// ------------------------------------------------------------------ host

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// bf16 [tokens][heads][d], token stride ld elements: boxes of 64 columns x
// box_heads heads x box_tokens tokens, 128-byte swizzle, zeros past the end
bool make_map(CUtensorMap* map, const void* base, int64_t d, int64_t heads, int64_t tokens, int64_t ld, uint32_t box_heads,
              uint32_t box_tokens) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, box_heads, box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  return n;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool heads_ok(int64_t q_heads, int64_t kv_heads) { return q_heads >= 1 && kv_heads >= 1 && q_heads <= 65536 && q_heads % kv_heads == 0; }

// heads of a group in one tile: the largest power of two (at most 128) that divides it
int64_t pack_of(int64_t group) {
  int64_t p = 1;
  while (p < kApTile && group % (2 * p) == 0) p *= 2;
  return p;
}

int64_t plan_capacity(int64_t total, int64_t batch, int64_t pack) { return total / (2 * kApTile / pack) + batch; }

template <int D>
fp8rl_status launch_prefill(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const ApArgs& a,
                            cudaStream_t stream) {
  auto kernel = attn_prefill_kernel<D>;
  // the attribute lives in the context: set once per device and context
  static std::atomic<uint64_t> ready[64];
  int dev = 0;
  const uint64_t ctx = current_context_id();
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || !ctx) return FP8RL_ERR_CUDA;
  if (ready[dev].load(std::memory_order_acquire) != ctx) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ApCfg<D>::kSmem) != cudaSuccess) {
      cudaGetLastError();
      return FP8RL_ERR_CUDA;
    }
    ready[dev].store(ctx, std::memory_order_release);
  }
  const int64_t most = (int64_t)a.capacity * a.hkv * (a.group / a.pack);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(sm_count(), most)));
  cfg.blockDim = dim3(kApThreads);
  cfg.dynamicSmemBytes = ApCfg<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, a) != cudaSuccess) {
    cudaGetLastError();
    return FP8RL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

extern "C" FP8RL_API size_t fp8rl_attn_prefill_plan_size(int64_t total_tokens, int64_t batch, int64_t q_heads,
                                                         int64_t kv_heads) {
  if (total_tokens < 0 || total_tokens > kApMaxTokens || batch < 0 || batch > (1 << 20) || !heads_ok(q_heads, kv_heads)) return 0;
  return (size_t)(16 * (1 + plan_capacity(total_tokens, batch, pack_of(q_heads / kv_heads))));
}

extern "C" FP8RL_API fp8rl_status fp8rl_attn_prefill_plan(const int32_t* d_cu_seqlens, int64_t batch, int64_t total_tokens,
                                                          int64_t q_heads, int64_t kv_heads, void* d_plan,
                                                          size_t plan_bytes, void* stream) {
  if (batch < 0 || total_tokens < 0 || !heads_ok(q_heads, kv_heads)) return FP8RL_ERR_INVALID_ARG;
  if (total_tokens > kApMaxTokens || batch > (1 << 20)) return FP8RL_ERR_SHAPE;
  if (!d_plan || (batch > 0 && !d_cu_seqlens)) return FP8RL_ERR_INVALID_ARG;
  if (plan_bytes < fp8rl_attn_prefill_plan_size(total_tokens, batch, q_heads, kv_heads)) return FP8RL_ERR_INVALID_ARG;
  if (!aligned(d_plan, 16) || !aligned(d_cu_seqlens, 4)) return FP8RL_ERR_ALIGNMENT;
  const int64_t pack = pack_of(q_heads / kv_heads);
  attn_plan_kernel<<<1, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      d_cu_seqlens, (int32_t)batch, (int32_t)total_tokens, (int32_t)(2 * kApTile / pack),
      (int32_t)plan_capacity(total_tokens, batch, pack), static_cast<int4*>(d_plan));
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}

extern "C" FP8RL_API fp8rl_status fp8rl_attn_prefill(const void* q_bf16, int64_t ldq, const void* k_bf16, int64_t ldk,
                                                     const void* v_bf16, int64_t ldv, const void* d_plan,
                                                     size_t plan_bytes, int64_t batch, int64_t total_tokens,
                                                     int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                                     float softmax_scale, void* out_bf16, int64_t ldo, float* d_lse,
                                                     void* stream) {
  if (batch < 0 || total_tokens < 0 || !heads_ok(q_heads, kv_heads) || head_dim < 1 || !(softmax_scale > 0.0f) ||
      !(softmax_scale <= FLT_MAX))
    return FP8RL_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || total_tokens > kApMaxTokens || batch > (1 << 20)) return FP8RL_ERR_SHAPE;
  if (ldq < q_heads * head_dim || ldk < kv_heads * head_dim || ldv < kv_heads * head_dim || ldo < q_heads * head_dim)
    return FP8RL_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return FP8RL_OK;
  if (!q_bf16 || !k_bf16 || !v_bf16 || !d_plan || !out_bf16) return FP8RL_ERR_INVALID_ARG;
  if (plan_bytes < fp8rl_attn_prefill_plan_size(total_tokens, batch, q_heads, kv_heads)) return FP8RL_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(out_bf16, 16) || ldq % 8 != 0 ||
      ldk % 8 != 0 || ldv % 8 != 0 || ldo % 8 != 0 || !aligned(d_plan, 16) || !aligned(d_lse, 4))
    return FP8RL_ERR_ALIGNMENT;
  ApArgs a{};
  a.plan = static_cast<const int4*>(d_plan);
  a.q = static_cast<const uint16_t*>(q_bf16), a.k = static_cast<const uint16_t*>(k_bf16), a.v = static_cast<const uint16_t*>(v_bf16);
  a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.lse = d_lse;
  a.ldo = ldo;
  a.total = (int32_t)total_tokens;
  a.hq = (int32_t)q_heads, a.hkv = (int32_t)kv_heads;
  a.group = (int32_t)(q_heads / kv_heads);
  a.pack = (int32_t)pack_of(a.group);
  a.capacity = (int32_t)plan_capacity(total_tokens, batch, a.pack);
  a.wide = aligned(out_bf16, 32) && ldo % 16 == 0;
  a.softmax_scale = softmax_scale;
  // work is numbered in 32 bits (with a round of CTAs to spare)
  if ((int64_t)a.capacity * kv_heads * (a.group / a.pack) > INT32_MAX - 4096) return FP8RL_ERR_SHAPE;
  a.err = device_error_word();
  if (!a.err) return FP8RL_ERR_CUDA;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, q_bf16, head_dim, q_heads, total_tokens, ldq, (uint32_t)a.pack, (uint32_t)(kApTile / a.pack)) ||
      !make_map(&mk, k_bf16, head_dim, kv_heads, total_tokens, ldk, 1, kApTile) ||
      !make_map(&mv, v_bf16, head_dim, kv_heads, total_tokens, ldv, 1, kApTile))
    return FP8RL_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch_prefill<128>(mq, mk, mv, a, cs) : launch_prefill<64>(mq, mk, mv, a, cs);
}
