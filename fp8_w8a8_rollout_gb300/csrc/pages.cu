// pages.cu -- the pages of the E4M3 KV cache: room for new tokens, pages shared
// by several sequences, and used pages moved together.
//
// The book-keeping is three device arrays: the block table (the page of each
// piece of a sequence, as the cache attention reads it), the lengths, and for each
// page the number of table rows that hold it; 0 is free.  A row of length n holds
// ceil(n / block_size) pages, its first entries.  There is no list of free pages
// that could disagree with it: the lowest free pages are found by counting.
//
//   reserve  gives row r room for count[r] more tokens.  Pages are handed out in
//            the rows' order, the lowest free one first.  A last page that is
//            not full and that other rows hold too is copied for the row first.
//   fork     new row i holds what old row parent[i] held; parent -1: nothing.
//   compact  with n used pages, the k-th used page at or past n moves to the k-th
//            free one before n.
//
// Each is one planning kernel: a CTA, or a cluster of 8 once there is much to count,
// whose warps own runs of pages; ranks come from a scan over the warps and an
// exchange over the cluster, so the result does not depend on timing (reference counts
// are sums of integers).  Its latency bounds it (about 4 dependent loads): 256 rows and 64 000 pages
// 13.5 us (on one CTA 15.4), 512 rows on one CTA 12 (with a warp for every row's pages 24), a
// fork 4.  The pages' contents are copied by a second kernel, which starts while the plan
// runs and reads the list of copies that it left: a stream of 16-byte pieces over
// all layers' K and V, bound by HBM (64 rows in 72 caches compacted: 277 us, 6.6 TB/s).
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "ptx.cuh"

namespace fp8rl {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;
constexpr int kCopyThreads = 256;
constexpr int kCopyCtasPerSm = 24;
constexpr int kMaxCaches = 256;    // a launch's, by value
constexpr int64_t kMaxRows = 8192;
constexpr int kFewPages = 8;       // new pages of a row that one thread hands out
constexpr int kRun = 4;            // copies of one page that are written from one read
constexpr int kHeader = 16;        // ints of the workspace ahead of the lists

struct Copy {  // a page's first `rows` cache rows
  int32_t src, dst, rows, pad;
};

// the sum over the block's threads before this one (low and high word apart), and the total
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* sums, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // `sums` may still be read from the scan before
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint64_t w = sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint64_t ahead = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp > 0 ? ahead : 0) + x - v;
}
static_assert(kPlanThreads == 32 * 32, "block_scan takes 32 warps");

// The cluster's barrier, not .aligned: lanes come to it from code that some of them ran alone (one that stores, loops of
// different lengths), and an aligned barrier that a warp's lanes do not reach together is undefined
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// this CTA's place in the sum over the cluster's CTAs
__device__ __forceinline__ uint64_t cluster_scan(uint64_t mine, uint64_t* slot, uint32_t ranks, uint64_t& total) {
  if (ranks == 1) {
    total = mine;
    return 0;
  }
  if (threadIdx.x == 0) *slot = mine;
  cluster_sync();
  const uint32_t rank = ptx::cluster_ctarank();
  uint64_t before = 0;
  total = 0;
  for (uint32_t r = 0; r < ranks; ++r) {
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(slot), r);
    const uint64_t v = (uint64_t)ptx::ld_dsmem_u32(at + 4) << 32 | ptx::ld_dsmem_u32(at);
    if (r < rank) before += v;
    total += v;
  }
  return before;
}

__device__ __forceinline__ void sync_all(uint32_t ranks) {
  if (ranks == 1) __syncthreads();
  else cluster_sync();  // (its release and acquire cover global memory too)
}

// the sum over the block's warps before this one, and of all, from one value a warp
__device__ __forceinline__ uint64_t warps_scan(uint64_t v, uint64_t* sums, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // `sums` may still be read from the scan before
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  uint64_t w = sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint64_t ahead = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return warp > 0 ? ahead : 0;
}

// the pages of this warp among the cluster's: a run of whole 128s
__device__ __forceinline__ void own_run(int32_t pages, uint32_t ranks, uint32_t rank, int32_t& p0, int32_t& p1) {
  const int64_t warps = (int64_t)ranks * 32;
  const int64_t run = ((pages + warps - 1) / warps + 127) / 128 * 128;
  p0 = (int32_t)min((int64_t)pages, run * ((int64_t)rank * 32 + (threadIdx.x >> 5)));
  p1 = (int32_t)min((int64_t)pages, (int64_t)p0 + run);
}

// f(page, counts of it and the three behind it) of the warp's run [p0, p1), lane by lane; behind the run: `none`
template <typename F>
__device__ __forceinline__ void each_four(const int32_t* refs, int32_t p0, int32_t p1, bool vec, int32_t none, F f) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int32_t q = p0; q < p1; q += 128) {
    const int32_t p = q + 4 * lane;
    int4 c = make_int4(none, none, none, none);
    if (vec && p + 4 <= p1) {
      c = *reinterpret_cast<const int4*>(refs + p);
    } else {
      if (p < p1) c.x = refs[p];
      if (p + 1 < p1) c.y = refs[p + 1];
      if (p + 2 < p1) c.z = refs[p + 2];
      if (p + 3 < p1) c.w = refs[p + 3];
    }
    f(p, c);
  }
}

// the sum of the lanes before this one
__device__ __forceinline__ uint32_t lanes_before(uint32_t v, uint32_t& total) {
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
    if ((int)(threadIdx.x & 31) >= d) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  return x - v;
}

// ------------------------------------------------------------------ reserve

struct ReserveArgs {
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  const int32_t* cu;     // or null: row r's range of the slots is [r, r + 1) * each
  const int32_t* count;  // or null: the whole range
  int32_t* slots;
  int32_t* info;
  int32_t* header;       // workspace
  int4* row;             // [rows]: length before, tokens given, place in the list, place among the copies or -1
  int32_t* list;         // [list_cap]: the free pages that are handed out
  Copy* copies;          // [rows]
  int64_t ldt, total, each, list_cap;
  int32_t rows, cols, block, pages, vec;
  uint32_t* err;
};

struct RowNeed {
  int32_t len, count;  // length, tokens asked for
  int32_t last;        // the page that is copied first, or -1
  int32_t need;        // new pages
  bool fits;
};

__device__ __forceinline__ int32_t blocks_of(int32_t n, int32_t block) { return (int32_t)(((int64_t)n + block - 1) / block); }

__device__ __forceinline__ RowNeed need_of(const ReserveArgs& a, int32_t r) {
  RowNeed n;
  const int64_t most = (int64_t)a.cols * a.block;
  n.len = (int32_t)max((int64_t)0, min((int64_t)a.lens[r], most));
  n.count = (int32_t)a.each;
  if (a.cu) {
    const int64_t begin = max((int64_t)0, min((int64_t)a.cu[r], a.total));
    n.count = (int32_t)(max(begin, min((int64_t)a.cu[r + 1], a.total)) - begin);
  }
  if (a.count) n.count = max(0, min(n.count, a.count[r]));
  n.last = -1;
  n.need = 0;
  n.fits = (int64_t)n.len + n.count <= most;
  if (n.fits && n.count > 0) {
    const int32_t held = blocks_of(n.len, a.block);
    n.need = blocks_of(n.len + n.count, a.block) - held;
    if (n.len % a.block != 0) {
      const int32_t p = a.table[r * a.ldt + held - 1];
      if (p >= 0 && p < a.pages && a.refs[p] > 1) {
        n.last = p;
        ++n.need;
      }
    }
  }
  return n;
}

// the cache row of a position, or -1 where the table names no page
__device__ __forceinline__ int32_t slot_of(const ReserveArgs& a, int64_t r, int64_t pos) {
  const int32_t p = a.table[r * a.ldt + pos / a.block];
  return p >= 0 && p < a.pages ? p * a.block + (int32_t)(pos % a.block) : -1;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const ReserveArgs a) {
  __shared__ uint64_t sums[32];
  __shared__ uint64_t slot[2];
  __shared__ int32_t freed;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const uint32_t ranks = gridDim.x, rank = blockIdx.x;
  const int tid = threadIdx.x;
  if (tid == 0) freed = 0;

  // the free pages of this warp's run
  int32_t p0, p1;
  uint32_t mine = 0;
  own_run(a.pages, ranks, rank, p0, p1);
  each_four(a.refs, p0, p1, a.vec, 1, [&](int32_t, int4 c) { mine += (c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0); });
  mine = __reduce_add_sync(0xffffffffu, mine);
  uint64_t cta_free, n_free;
  const uint64_t before = warps_scan(mine, sums, cta_free);
  const uint64_t rank_before = cluster_scan(cta_free, &slot[0], ranks, n_free);
  const uint64_t avail = min(n_free, (uint64_t)a.list_cap);

  // what the rows need, in their order: every CTA the same
  uint64_t first = 0;              // pages asked for by the tiles before
  uint64_t copies = 0, taken = 0, refused = 0;
  bool many = false;               // a row that takes more pages than a thread should hand out
  for (int32_t r0 = 0; r0 < a.rows; r0 += kPlanThreads) {
    const int32_t r = r0 + tid;
    RowNeed n{};
    n.last = -1;
    n.fits = true;
    if (r < a.rows) n = need_of(a, r);
    uint64_t tile;
    const uint64_t at = first + block_scan((uint64_t)n.need, sums, tile);
    first += tile;
    const bool served = n.fits && (n.need == 0 || at + (uint64_t)n.need <= avail);
    many |= served && n.need > kFewPages;
    // copies (16 bits), rows refused (16 bits), pages given
    const uint64_t report = (served && n.last >= 0 ? 1u : 0u) | (uint64_t)!served << 16 | (served ? (uint64_t)n.need << 32 : 0);
    const uint64_t before_row = block_scan(report, sums, tile);
    if (r < a.rows && rank == 0 && dcheck((int64_t)at + n.need <= a.list_cap || !served, a.err)) {
      // (the third is the row's place in the list)
      a.row[r] = make_int4(n.len, served ? n.count : 0, (int32_t)min(at, (uint64_t)INT_MAX),
                           served && n.last >= 0 ? (int32_t)(copies + (before_row & 0xffffu)) : -1);
    }
    copies += tile & 0xffffu;
    refused += tile >> 16 & 0xffffu;
    taken += tile >> 32;
  }
  const uint64_t end = first;  // pages that the rows ask for

  // the lowest free pages, as many as may be handed out
  const uint64_t handed = min(end, avail);
  uint64_t rank_at = rank_before + before;
  if (mine > 0 && rank_at < handed) {
    each_four(a.refs, p0, p1, a.vec, 1, [&](int32_t p, int4 c) {
      if (rank_at >= handed) return;  // (all lanes alike)
      const int32_t v[4] = {c.x, c.y, c.z, c.w};
      uint32_t total;
      uint64_t at = rank_at + lanes_before((c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0), total);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (v[i] != 0) continue;
        if (at < handed && dcheck(at < (uint64_t)a.list_cap && p + i < a.pages, a.err)) a.list[at] = p + i;
        ++at;
      }
      rank_at += total;
    });
  }
  sync_all(ranks);  // nobody reads the counts, the rows' lengths and last pages from here on

  // the rows' pages: a thread per row, and a warp for each that takes many
  many = __syncthreads_or(many);
  auto hand_out = [&](int32_t r, int lane, int lanes) {
    const int4 info = a.row[r];
    const int32_t len = info.x, given = info.y, copy_at = info.w;
    if (given == 0) return;
    const int32_t held = blocks_of(len, a.block), after = blocks_of(len + given, a.block);
    if (many && (after - held + (copy_at >= 0) > kFewPages) != (lanes > 1)) return;
    int32_t* row = a.table + r * a.ldt;
    int32_t at = info.z;
    if (copy_at >= 0) {  // the shared last page's copy
      const int32_t fresh = a.list[at++];
      if (lane == 0) {
        const int32_t old = row[held - 1];
        if (dcheck(fresh >= 0 && fresh < a.pages && old >= 0 && old < a.pages && held <= a.cols && copy_at < a.rows, a.err)) {
          if (atomicSub(a.refs + old, 1) == 1) atomicAdd(&freed, 1);
          a.refs[fresh] = 1;
          row[held - 1] = fresh;
          a.copies[copy_at] = Copy{old, fresh, len % a.block, 0};
        }
      }
    }
    for (int32_t j = held + lane; j < after; j += lanes) {
      const int32_t p = a.list[at + j - held];
      if (dcheck(p >= 0 && p < a.pages && j < a.cols, a.err)) {
        a.refs[p] = 1;
        row[j] = p;
      }
    }
    if (lane == 0 && dcheck(after <= a.cols, a.err)) a.lens[r] = len + given;
  };
  for (int32_t r = (int32_t)rank * kPlanThreads + tid; r < a.rows; r += (int32_t)ranks * kPlanThreads) hand_out(r, 0, 1);
  if (many)
    for (int32_t r = (int32_t)rank * 32 + (tid >> 5); r < a.rows; r += (int32_t)ranks * 32) hand_out(r, tid & 31, 32);
  __syncthreads();
  uint64_t all_freed;
  cluster_scan((uint64_t)freed, &slot[1], ranks, all_freed);  // (with one CTA the barrier above is the one needed)
  if (rank == 0 && tid == 0 && dcheck(copies <= (uint64_t)a.rows && taken <= avail, a.err)) {
    a.header[0] = (int32_t)copies;
    if (a.info) {
      a.info[0] = (int32_t)(n_free - taken + all_freed);
      a.info[1] = (int32_t)refused;
    }
  }

  // the slots of the new tokens
  if (a.cu) {
    for (int64_t t = (int64_t)rank * kPlanThreads + tid; t < a.total; t += (int64_t)ranks * kPlanThreads) {
      int32_t lo = 0, hi = a.rows;  // the last row that begins at or before t
      while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      if (a.rows == 0 || t < a.cu[lo] || t >= a.cu[lo + 1]) continue;  // of no row
      const int4 info = a.row[lo];
      const int64_t i = t - max(0, a.cu[lo]), pos = info.x + i;  // (ranges are clamped to the entries)
      int32_t s = -1;
      if (i < info.y) s = slot_of(a, lo, pos);
      if (dcheck(i >= 0 && s < (int64_t)a.pages * a.block, a.err)) a.slots[t] = s;
    }
  } else {
    for (int64_t t = (int64_t)rank * kPlanThreads + tid; t < a.total; t += (int64_t)ranks * kPlanThreads) {
      const int64_t r = t / a.each, i = t % a.each;
      const int4 info = a.row[r];
      const int64_t pos = info.x + i;
      int32_t s = -1;
      if (i < info.y) s = slot_of(a, r, pos);
      if (dcheck(r < a.rows && s < (int64_t)a.pages * a.block, a.err)) a.slots[t] = s;
    }
  }
  if (ranks > 1) cluster_sync();  // the others have read this CTA's slot
}

// ------------------------------------------------------------------ fork

struct ForkArgs {
  const int32_t *in, *lens_in, *parent;
  int32_t *out, *lens_out, *refs;
  int64_t ld_in, ld_out;
  int32_t rows_in, rows_out, cols, block, pages, in_place;
  uint32_t* err;
};

// CTA r: gives back what old row r held, takes what new row r holds
__global__ void __launch_bounds__(128) fork_kernel(const ForkArgs a) {
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const int32_t r = blockIdx.x;
  const int64_t most = (int64_t)a.cols * a.block;
  auto length = [&](int32_t i) { return (int32_t)max((int64_t)0, min((int64_t)a.lens_in[i], most)); };
  int32_t p = r < a.rows_out ? a.parent[r] : -1;
  if (p < 0 || p >= a.rows_in) p = -1;
  // in place, a row's parent has to keep its own row: it is read while others are written
  if (a.in_place && p >= 0 && p != r && a.parent[p] != p) p = -1;
  const bool stays = p == r;
  const int32_t old_len = r < a.rows_in ? length(r) : 0, new_len = p >= 0 ? length(p) : 0;
  const int32_t old_held = stays ? 0 : blocks_of(old_len, a.block), held = blocks_of(new_len, a.block);
  __syncthreads();  // lens_out may be lens_in
  if (stays && a.in_place) return;
  for (int32_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
    if (j < old_held) {
      const int32_t page = a.in[r * a.ld_in + j];
      if (page >= 0 && page < a.pages) atomicSub(a.refs + page, 1);
    }
    if (r < a.rows_out) {
      int32_t page = -1;
      if (j < held) {
        page = a.in[p * a.ld_in + j];
        if (!stays && page >= 0 && page < a.pages) atomicAdd(a.refs + page, 1);
      }
      if (dcheck(j < a.ld_out && held <= a.cols, a.err)) a.out[r * a.ld_out + j] = page;
    }
  }
  if (threadIdx.x == 0 && r < a.rows_out && dcheck(held <= a.cols, a.err)) a.lens_out[r] = new_len;
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
  int32_t* refs;
  int32_t* used;
  int32_t* header;  // workspace: copies, used pages
  Copy* copies;     // [pages / 2 + 1]
  int32_t* to;      // [pages]: where a page at or past the used ones went
  int32_t pages, block, vec;
  uint32_t* err;
};

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
  __shared__ uint64_t sums[32];
  __shared__ uint64_t slot[2];
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  const uint32_t ranks = gridDim.x, rank = blockIdx.x;
  int32_t p0, p1;
  uint32_t mine = 0;
  own_run(a.pages, ranks, rank, p0, p1);
  each_four(a.refs, p0, p1, a.vec, 0, [&](int32_t, int4 c) { mine += (c.x > 0) + (c.y > 0) + (c.z > 0) + (c.w > 0); });
  mine = __reduce_add_sync(0xffffffffu, mine);
  uint64_t cta, all;
  warps_scan(mine, sums, cta);
  cluster_scan(cta, &slot[0], ranks, all);
  const int32_t n = (int32_t)all;
  // holes before n (low word) and used pages past it (high word): as many of one as of the other
  uint32_t holes = 0, movers = 0;
  each_four(a.refs, p0, p1, a.vec, 0, [&](int32_t p, int4 c) {
    const int32_t v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i < p1) {
        holes += p + i < n && v[i] <= 0;
        movers += p + i >= n && v[i] > 0;
      }
    }
  });
  holes = __reduce_add_sync(0xffffffffu, holes);
  movers = __reduce_add_sync(0xffffffffu, movers);
  uint64_t at = warps_scan((uint64_t)movers << 32 | holes, sums, cta);
  at += cluster_scan(cta, &slot[1], ranks, all);
  uint32_t hole = (uint32_t)at, mover = (uint32_t)(at >> 32);
  const int32_t moves = (int32_t)(all >> 32);
  each_four(a.refs, p0, p1, a.vec, 0, [&](int32_t p, int4 c) {
    const int32_t v[4] = {c.x, c.y, c.z, c.w};
    // (a run may lie on both sides of n)
    uint32_t here = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i < p1) here += p + i < n ? (v[i] <= 0 ? 1u : 0u) : (v[i] > 0 ? 0x10000u : 0u);
    }
    uint32_t total;
    const uint32_t ahead = lanes_before(here, total);
    uint32_t h = hole + (ahead & 0xffffu), m = mover + (ahead >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i >= p1) continue;
      if (p + i < n) {
        if (v[i] <= 0 && dcheck((int32_t)h <= a.pages / 2, a.err)) a.copies[h].dst = p + i;
        h += v[i] <= 0;
      } else if (v[i] > 0) {
        if (dcheck((int32_t)m <= a.pages / 2, a.err)) a.copies[m].src = p + i;
        ++m;
      } else if (dcheck(p >= 0 && p + i < a.pages, a.err)) {
        a.to[p + i] = p + i;  // (no row holds it, or the counts are wrong)
      }
    }
    hole += total & 0xffffu;
    mover += total >> 16;
  });
  if (rank == 0 && threadIdx.x == 0 && dcheck(moves <= a.pages / 2 && moves <= n && n <= a.pages, a.err)) {
    a.header[0] = moves;
    a.header[1] = n;
    if (a.used) a.used[0] = n;
  }
  sync_all(ranks);  // nobody counts from here on
  for (int32_t k = rank * kPlanThreads + threadIdx.x; k < moves; k += (int32_t)ranks * kPlanThreads) {
    Copy& c = a.copies[k];
    const int32_t src = c.src, dst = c.dst;
    if (dcheck(k <= a.pages / 2 && src >= n && src < a.pages && dst >= 0 && dst < n, a.err)) {
      c.rows = a.block;
      a.to[src] = dst;
      a.refs[dst] = a.refs[src];
      a.refs[src] = 0;
    }
  }
  if (ranks > 1) cluster_sync();  // the others have read this CTA's slots
}

// ------------------------------------------------------------------ contents

struct CopyArgs {
  void* caches[kMaxCaches];
  const int32_t* header;
  const Copy* copies;
  int64_t ld, width;  // bytes
  int32_t n_caches, block, pages;
  // the table of a compaction (null: none)
  int32_t* table;
  const int32_t* lens;
  const int32_t* to;
  int64_t ldt;
  int32_t rows, cols;
  uint32_t* err;
};

// a table's entries of pages that moved
__device__ __forceinline__ void follow(const CopyArgs& a) {
  const int32_t n = a.header[1];
  const int64_t entries = (int64_t)a.rows * a.cols, stride = (int64_t)gridDim.x * gridDim.y * kCopyThreads;
  for (int64_t e = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kCopyThreads + threadIdx.x; e < entries; e += stride) {
    const int64_t r = e / a.cols, j = e % a.cols;
    const int64_t len = max((int64_t)0, min((int64_t)a.lens[r], (int64_t)a.cols * a.block));
    if (j * a.block >= len) continue;  // (entries past a row's pages say nothing)
    int32_t* at = a.table + r * a.ldt + j;
    const int32_t p = *at;
    if (p >= n && p < a.pages && dcheck(j < a.ldt && a.to[p] >= 0 && a.to[p] <= p, a.err)) *at = a.to[p];
  }
}

// A CTA of a cache (x) takes every gridDim.y'th part of the copies.  Copies of one page
// follow one another in the list when its holders are neighbours (answers to one
// prompt): each piece is read once and written to up to kRun of them (512 answers to
// 32 prompts, 72 caches: 93 -> 68 us for fork and room together).  P: uint4, or single bytes
template <typename P>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int U = 4;
  ptx::grid_dep_launch_dependents();
  ptx::grid_dep_wait();
  if (a.table) follow(a);
  if (a.n_caches == 0) return;
  const int32_t copies = a.header[0];
  const int64_t per_row = a.width / (int64_t)sizeof(P), ld = a.ld / (int64_t)sizeof(P);
  P* base = static_cast<P*>(a.caches[blockIdx.x]);
  // (few copies: one a part; kRun once that leaves 8 CTAs an SM with work)
  const int32_t part = copies >= kRun * (int32_t)gridDim.y * 8 / kCopyCtasPerSm ? kRun : 1;
  for (int64_t first = (int64_t)blockIdx.y * part; first < copies; first += (int64_t)gridDim.y * part) {
    const int32_t end = (int32_t)min((int64_t)copies, first + part);
    for (int32_t at = (int32_t)first; at < end;) {
      const Copy c = a.copies[at];
      int32_t to[kRun], n = 1;
      to[0] = c.dst;
#pragma unroll
      for (int k = 1; k < kRun; ++k) {
        to[k] = c.dst;
        if (n == k && at + k < end) {
          const Copy d = a.copies[at + k];
          if (d.src == c.src && d.rows == c.rows) to[k] = d.dst, ++n;
        }
      }
      at += n;
      bool good = c.src >= 0 && c.src < a.pages && c.rows <= a.block;
#pragma unroll
      for (int k = 0; k < kRun; ++k) good = good && to[k] >= 0 && to[k] < a.pages;
      if (!dcheck(good, a.err)) continue;
      const P* src = base + (int64_t)c.src * a.block * ld;
      const uint32_t pieces = (uint32_t)(c.rows * per_row);  // (below 2^31, so that a thread's last numbers, past them, do not wrap)
      auto place = [&](uint32_t i) { return per_row == ld ? (int64_t)i : (i / per_row) * ld + i % per_row; };
      for (uint32_t i = threadIdx.x; i < pieces; i += U * kCopyThreads) {
        P v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + u * kCopyThreads < pieces) v[u] = src[place(i + u * kCopyThreads)];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          if (k >= n) break;
          P* dst = base + (int64_t)to[k] * a.block * ld;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (i + u * kCopyThreads < pieces) dst[place(i + u * kCopyThreads)] = v[u];
        }
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

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// a plan on one CTA while each of its threads has few pages (and tokens) to look at
int plan_ctas(int64_t pages, int64_t tokens) { return pages > 32 * kPlanThreads || tokens > 8 * kPlanThreads ? kPlanCluster : 1; }

template <typename K, typename A>
fp8rl_status launch_plan(K kernel, const A& a, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return FP8RL_ERR_CUDA;
  }
  return FP8RL_OK;
}

// the copies of all caches, in launches of up to kMaxCaches; the first follows the table
fp8rl_status launch_copies(CopyArgs& a, void* const* caches, int32_t n_caches, int64_t most, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  for (int32_t c0 = 0; c0 == 0 || c0 < n_caches; c0 += kMaxCaches) {
    a.n_caches = std::min(kMaxCaches, n_caches - c0);
    bool vec = a.ld % 16 == 0 && a.width % 16 == 0;
    for (int32_t i = 0; i < a.n_caches; ++i) {
      a.caches[i] = caches[c0 + i];
      vec = vec && aligned(caches[c0 + i], 16);
    }
    const int64_t x = std::max(1, a.n_caches), entries = a.table ? (int64_t)a.rows * a.cols : 0;
    const int64_t parts = std::max(a.n_caches > 0 ? most : 0, (entries + x * kCopyThreads - 1) / (x * kCopyThreads));
    const int64_t ctas = (int64_t)sm_count() * kCopyCtasPerSm;
    cfg.gridDim = dim3((unsigned)x, (unsigned)std::max<int64_t>(1, std::min(parts, ctas / x)));
    const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, copy_pages_kernel<uint4>, a) : cudaLaunchKernelEx(&cfg, copy_pages_kernel<uint8_t>, a);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return FP8RL_ERR_CUDA;
    }
    a.table = nullptr;
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}

// the sizes that the three calls share
fp8rl_status check_sizes(int64_t rows, int64_t max_blocks, int64_t ldt, int64_t block_size, int64_t pages) {
  if (rows < 0 || max_blocks < 0 || ldt < max_blocks || block_size < 1 || pages < 0) return FP8RL_ERR_INVALID_ARG;
  if (rows > kMaxRows || block_size > (1 << 30) || pages > (int64_t)INT_MAX / block_size || pages > (1 << 30) ||
      max_blocks > (int64_t)INT_MAX / block_size)
    return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

// (caches without a page may have no memory)
fp8rl_status check_caches(void* const* caches, int32_t n_caches, int64_t width, int64_t ld, int64_t block_size, int64_t pages) {
  if (n_caches < 0 || (n_caches > 0 && (!caches || width < 1 || ld < width))) return FP8RL_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n_caches; ++i)
    if (pages > 0 && !caches[i]) return FP8RL_ERR_INVALID_ARG;
  if (n_caches > 0 && width > (int64_t)INT_MAX / block_size) return FP8RL_ERR_SHAPE;
  return FP8RL_OK;
}

size_t reserve_list(int64_t rows, int64_t total_tokens, int64_t block_size) {
  return (size_t)(total_tokens / block_size + 2 * rows);  // a row's ends, and its copy
}

}  // namespace
}  // namespace fp8rl

using namespace fp8rl;

extern "C" FP8RL_API size_t fp8rl_kv_reserve_workspace_size(int64_t rows, int64_t total_tokens, int64_t block_size) {
  if (rows < 0 || rows > kMaxRows || total_tokens < 0 || total_tokens > INT_MAX || block_size < 1) return 0;
  return 4 * kHeader + (sizeof(int4) + sizeof(Copy)) * (size_t)rows + up16(4 * reserve_list(rows, total_tokens, block_size));
}

extern "C" FP8RL_API fp8rl_status fp8rl_kv_reserve(int32_t* d_block_table, int64_t ldt, int64_t rows, int64_t max_blocks,
                                                   int64_t block_size, int32_t* d_lens, int32_t* d_refs, int64_t pages,
                                                   const int32_t* d_cu_seqlens, const int32_t* d_count,
                                                   int64_t total_tokens, int32_t* d_slots, int32_t* d_info,
                                                   void* const* caches, int32_t n_caches, int64_t width, int64_t ld_cache,
                                                   void* d_workspace, size_t workspace_bytes, void* stream) {
  if (total_tokens < 0) return FP8RL_ERR_INVALID_ARG;
  fp8rl_status st = check_sizes(rows, max_blocks, ldt, block_size, pages);
  if (st != FP8RL_OK) return st;
  if ((st = check_caches(caches, n_caches, width, ld_cache, block_size, pages)) != FP8RL_OK) return st;
  if (total_tokens > INT_MAX) return FP8RL_ERR_SHAPE;
  if (!d_cu_seqlens && (rows > 0 ? total_tokens % rows != 0 : total_tokens != 0)) return FP8RL_ERR_INVALID_ARG;
  if (rows == 0) return FP8RL_OK;
  if ((max_blocks > 0 && !d_block_table) || !d_lens || (pages > 0 && !d_refs) || (total_tokens > 0 && !d_slots) || !d_workspace ||
      workspace_bytes < fp8rl_kv_reserve_workspace_size(rows, total_tokens, block_size))
    return FP8RL_ERR_INVALID_ARG;
  if (!aligned(d_block_table, 4) || !aligned(d_lens, 4) || !aligned(d_refs, 4) || !aligned(d_cu_seqlens, 4) ||
      !aligned(d_count, 4) || !aligned(d_slots, 4) || !aligned(d_info, 4) || !aligned(d_workspace, 16))
    return FP8RL_ERR_ALIGNMENT;
  ReserveArgs a{};
  if (!check_word(&a.err)) return FP8RL_ERR_CUDA;
  a.table = d_block_table;
  a.lens = d_lens;
  a.refs = d_refs;
  a.cu = d_cu_seqlens;
  a.count = d_count;
  a.slots = d_slots;
  a.info = d_info;
  a.header = static_cast<int32_t*>(d_workspace);
  a.row = reinterpret_cast<int4*>(a.header + kHeader);
  a.copies = reinterpret_cast<Copy*>(a.row + rows);
  a.list = reinterpret_cast<int32_t*>(a.copies + rows);
  a.ldt = ldt;
  a.total = total_tokens;
  a.each = total_tokens / rows;
  a.list_cap = (int64_t)reserve_list(rows, total_tokens, block_size);
  a.rows = (int32_t)rows, a.cols = (int32_t)max_blocks, a.block = (int32_t)block_size, a.pages = (int32_t)pages;
  a.vec = aligned(d_refs, 16);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if ((st = launch_plan(reserve_plan_kernel, a, plan_ctas(pages, total_tokens), cs)) != FP8RL_OK) return st;
  if (n_caches == 0 || total_tokens == 0) return FP8RL_OK;
  CopyArgs c{};
  c.header = a.header;
  c.copies = a.copies;
  c.ld = ld_cache, c.width = width;
  c.block = a.block, c.pages = a.pages;
  c.err = a.err;
  return launch_copies(c, caches, n_caches, rows, cs);
}

extern "C" FP8RL_API fp8rl_status fp8rl_kv_fork(const int32_t* d_block_table, int64_t ldt, int64_t rows,
                                                int64_t max_blocks, int64_t block_size, const int32_t* d_lens,
                                                const int32_t* d_parent, int64_t new_rows, int32_t* d_new_table,
                                                int64_t ld_new, int32_t* d_new_lens, int32_t* d_refs, int64_t pages,
                                                void* stream) {
  fp8rl_status st = check_sizes(rows, max_blocks, ldt, block_size, pages);
  if (st != FP8RL_OK) return st;
  if (new_rows < 0 || ld_new < max_blocks) return FP8RL_ERR_INVALID_ARG;
  if (new_rows > kMaxRows) return FP8RL_ERR_SHAPE;
  if (rows == 0 && new_rows == 0) return FP8RL_OK;
  if ((rows > 0 && ((max_blocks > 0 && !d_block_table) || !d_lens)) ||
      (new_rows > 0 && (!d_parent || (max_blocks > 0 && !d_new_table) || !d_new_lens)) || (pages > 0 && !d_refs))
    return FP8RL_ERR_INVALID_ARG;
  const bool in_place = new_rows > 0 && ((d_new_table && d_new_table == d_block_table) || d_new_lens == d_lens);
  if (in_place && (d_new_table != d_block_table || d_new_lens != d_lens || rows != new_rows || ldt != ld_new))
    return FP8RL_ERR_INVALID_ARG;
  if (!aligned(d_block_table, 4) || !aligned(d_lens, 4) || !aligned(d_parent, 4) || !aligned(d_new_table, 4) ||
      !aligned(d_new_lens, 4) || !aligned(d_refs, 4))
    return FP8RL_ERR_ALIGNMENT;
  ForkArgs a{};
  if (!check_word(&a.err)) return FP8RL_ERR_CUDA;
  a.in = d_block_table;
  a.lens_in = d_lens;
  a.parent = d_parent;
  a.out = d_new_table;
  a.lens_out = d_new_lens;
  a.refs = d_refs;
  a.ld_in = ldt, a.ld_out = ld_new;
  a.rows_in = (int32_t)rows, a.rows_out = (int32_t)new_rows, a.cols = (int32_t)max_blocks, a.block = (int32_t)block_size;
  a.pages = (int32_t)pages;
  a.in_place = in_place;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max(rows, new_rows));
  cfg.blockDim = dim3(128);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fork_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return FP8RL_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? FP8RL_OK : FP8RL_ERR_CUDA;
}

extern "C" FP8RL_API size_t fp8rl_kv_compact_workspace_size(int64_t pages) {
  if (pages < 0 || pages > (1 << 30)) return 0;
  return 4 * kHeader + sizeof(Copy) * (size_t)(pages / 2 + 1) + up16(4 * (size_t)pages);
}

extern "C" FP8RL_API fp8rl_status fp8rl_kv_compact(int32_t* d_block_table, int64_t ldt, int64_t rows, int64_t max_blocks,
                                                   int64_t block_size, const int32_t* d_lens, int32_t* d_refs, int64_t pages,
                                                   int32_t* d_used, void* const* caches, int32_t n_caches, int64_t width,
                                                   int64_t ld_cache, void* d_workspace, size_t workspace_bytes, void* stream) {
  fp8rl_status st = check_sizes(rows, max_blocks, ldt, block_size, pages);
  if (st != FP8RL_OK) return st;
  if ((st = check_caches(caches, n_caches, width, ld_cache, block_size, pages)) != FP8RL_OK) return st;
  if ((rows > 0 && ((max_blocks > 0 && !d_block_table) || !d_lens)) || (pages > 0 && !d_refs) || !d_used || !d_workspace ||
      workspace_bytes < fp8rl_kv_compact_workspace_size(pages))
    return FP8RL_ERR_INVALID_ARG;
  if (!aligned(d_block_table, 4) || !aligned(d_lens, 4) || !aligned(d_refs, 4) || !aligned(d_used, 4) || !aligned(d_workspace, 16))
    return FP8RL_ERR_ALIGNMENT;
  CompactArgs a{};
  if (!check_word(&a.err)) return FP8RL_ERR_CUDA;
  a.refs = d_refs;
  a.used = d_used;
  a.header = static_cast<int32_t*>(d_workspace);
  a.copies = reinterpret_cast<Copy*>(a.header + kHeader);
  a.to = reinterpret_cast<int32_t*>(a.copies + pages / 2 + 1);
  a.pages = (int32_t)pages;
  a.block = (int32_t)block_size;
  a.vec = aligned(d_refs, 16);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if ((st = launch_plan(compact_plan_kernel, a, plan_ctas(pages, 0), cs)) != FP8RL_OK) return st;
  CopyArgs c{};
  c.header = a.header;
  c.copies = a.copies;
  c.ld = ld_cache, c.width = width;
  c.block = a.block, c.pages = a.pages;
  c.table = rows > 0 && max_blocks > 0 ? d_block_table : nullptr;
  c.lens = d_lens;
  c.to = a.to;
  c.ldt = ldt;
  c.rows = (int32_t)rows, c.cols = (int32_t)max_blocks;
  c.err = a.err;
  if (n_caches == 0 && !c.table) return FP8RL_OK;
  return launch_copies(c, caches, n_caches, pages / 2, cs);
}
