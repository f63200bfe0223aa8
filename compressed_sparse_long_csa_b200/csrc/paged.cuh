// Internal arguments and the work schedule of the paged-cache attention kernels.
//
// A paged cache is a pool of pages [n_pages, page, d_k]; entry e of sequence b is row
// e % page of page table[b, e / page].
#pragma once
#include "common.cuh"

#include <atomic>

namespace csa {

// Raises a kernel's dynamic shared-memory limit, once per device (`done`: a bit per device,
// one word per kernel): the call takes longer on the host than all checks of a launch.
inline cudaError_t set_smem_once(const void* kernel, std::atomic<uint64_t>& done, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);             // the library takes devices 0 .. 63
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct PagedAttnArgs {
  const void* q;              // [B, H, dk]
  const void* pages;          // [n_pages, page, dk]
  int64_t n_pages;
  int page;
  unsigned page_mul;          // e / page = e * page_mul >> page_shift for 0 <= e < 2^31 (paged_divisor)
  int page_shift;
  const int32_t* table;       // [B, table_w] page of each run of `page` entries
  int table_w;
  const int32_t* n_entries;   // [B] (dense) or null
  const int32_t* idx;         // [B, k] (sparse) or null
  int k;
  const void* win;            // [B, W, dk]
  const int32_t* win_len;     // [B]
  int W;
  const float* sink;          // [H]
  int B, H, dk, dv;
  float sm_scale;
  void* out;                  // [B, H, dv]
  float* lse;                 // [B, H] or null
  float* part;                // partials of split sequences: paged_slots(units) blocks
  int units;                  // work units (CTAs per head group)
  int tile_log2;              // rows per tile of the schedule, as a power of two
  int min_tiles;              // least tiles of a unit
  int begin_cost;             // what beginning a sequence costs a unit, in tiles
  unsigned* err;
};

// Sets the multiplier: 2^(31 + s) / page rounded up, 2^s the power of two from page up.  It is off by
// less than 1, so e times it by less than 2^31 <= 2^(31 + s) / page: the quotient is exact.
inline void paged_divisor(PagedAttnArgs& a) {
  int s = 0;
  while ((1 << s) < a.page) ++s;
  a.page_mul = (unsigned)(((1ull << (31 + s)) + a.page - 1) / a.page);
  a.page_shift = 31 + s;
}
// The page that holds entry e (a division costs a dependent chain of some 30 instructions).
__device__ __forceinline__ int paged_page(const PagedAttnArgs& a, int e) {
  return (int)((unsigned long long)(unsigned)e * a.page_mul >> a.page_shift);
}

// Entries that the table has room for.
__host__ __device__ inline int64_t paged_capacity(const PagedAttnArgs& a) { return (int64_t)a.table_w * a.page; }

// ---- schedule ---------------------------------------------------------------------------------
// The rows of a sequence are cut into tiles of 2^tile_log2 rows: its entries (or index slots)
// first, then its window rows, so that no tile mixes the two.  The tiles of all sequences, in
// order, are dealt to the units in equal runs, so that every unit takes as long as the others
// however ragged the lengths are; the lengths are read on the device only.  Beginning a sequence
// costs a unit more than its tiles (queries, an empty pipeline, an epilogue): begin_cost places
// that hold no tile come before a sequence's first one (tensor cores: 2;
// CUDA cores, where a tile costs as much: 0).  A sequence whose tiles lie in one unit is
// finished there; one that is cut leaves a partial (o, m, l) in each unit it touches, and a merge
// kernel joins them.  A unit holds at most two partials: one of a sequence that began before it
// (slot 0) and one of a sequence that begins in it and goes on (slot 1).
__device__ __forceinline__ int paged_rows_a(const PagedAttnArgs& a, int b) {
  if (a.idx) return a.k;
  const int64_t n = a.n_entries[b], cap = paged_capacity(a);
  return (int)(n < 0 ? 0 : (n > cap ? cap : n));
}
__device__ __forceinline__ int paged_rows_w(const PagedAttnArgs& a, int b) {
  if (a.W == 0) return 0;
  const int n = a.win_len[b];
  return n < 0 ? 0 : (n > a.W ? a.W : n);
}
__device__ __forceinline__ int64_t paged_tiles(const PagedAttnArgs& a, int b) {
  const int na = paged_rows_a(a, b), nw = paged_rows_w(a, b), up = (1 << a.tile_log2) - 1;
  return (((int64_t)na + up) >> a.tile_log2) + ((nw + up) >> a.tile_log2);
}
// Places of a sequence: its tiles and what it costs to begin it.
__device__ __forceinline__ int64_t paged_places(const PagedAttnArgs& a, int b) {
  const int64_t tiles = paged_tiles(a, b);
  return tiles ? tiles + a.begin_cost : 0;
}

struct PagedPlan {
  int64_t total;     // places of all sequences
  int64_t per;       // places of a unit
  int64_t before;    // places of the sequences before sequence b
  int b;             // the sequence that holds the unit's first place (B when there is none)
};

// The plan of a unit.  All `threads` threads of the block call it; scratch: 66 int64 in shared
// memory.
__device__ __forceinline__ PagedPlan paged_plan(const PagedAttnArgs& a, int unit, int threads, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  const int chunk = (a.B + threads - 1) / threads;
  const int b0 = min(a.B, tid * chunk), b1 = min(a.B, b0 + chunk);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += paged_places(a, b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scratch[warp] = incl;
  if (tid == 0) { scratch[64] = 0; scratch[65] = a.B; }
  __syncthreads();
  int64_t at = incl - mine, total = 0;                // places before this thread's sequences, and all
  for (int w = 0; w < warps; ++w) {
    const int64_t v = scratch[w];
    if (w < warp) at += v;
    total += v;
  }
  int64_t per = (total + a.units - 1) / a.units;
  if (per < a.min_tiles) per = a.min_tiles;
  const int64_t first = (int64_t)unit * per;
  if (first >= at && first < at + mine) {             // one thread at most
    int b = b0;
    for (;; ++b) {
      const int64_t n = paged_places(a, b);
      if (first < at + n) break;
      at += n;
    }
    scratch[64] = at;
    scratch[65] = b;
  }
  __syncthreads();
  PagedPlan p;
  p.total = total;
  p.per = per;
  p.before = scratch[64];
  p.b = (int)scratch[65];
  return p;
}

// The segments of a unit: tiles [t0, t1) of sequence b.
struct PagedSeg {
  int next_b;
  int64_t next_p, left;                      // the next place of next_b; places left of the unit
  int b, na, nw;
  int64_t ta, t0, t1;                        // ta: tiles of the entries; the window's follow
  bool whole;                                // all tiles of the sequence
  __device__ __forceinline__ void start(const PagedPlan& p, int unit) {
    next_b = p.b;
    next_p = (int64_t)unit * p.per - p.before;
    left = p.total - (int64_t)unit * p.per;
    if (left > p.per) left = p.per;
    t0 = t1 = 0;
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs& a) {
    const int up = (1 << a.tile_log2) - 1;
    while (left > 0) {
      b = next_b++;
      na = paged_rows_a(a, b);
      nw = paged_rows_w(a, b);
      ta = ((int64_t)na + up) >> a.tile_log2;
      const int64_t tiles = ta + ((nw + up) >> a.tile_log2);
      const int64_t p0 = next_p, end = tiles ? tiles + a.begin_cost : 0;
      next_p = 0;
      if (p0 >= end) continue;
      const int64_t p1 = end < p0 + left ? end : p0 + left;
      left -= p1 - p0;
      t0 = p0 > a.begin_cost ? p0 - a.begin_cost : 0;
      t1 = p1 > a.begin_cost ? p1 - a.begin_cost : 0;
      if (t0 >= t1) continue;                // the unit holds the cost of the beginning only
      whole = t0 == 0 && t1 == tiles;
      return true;
    }
    return false;
  }
  // The slot of the segment's partial.
  __device__ __forceinline__ int slot(int unit) const { return 2 * unit + (t0 == 0 ? 1 : 0); }
};

// A partial of a cut sequence holds o (not normalised), m and l per head, for natural-log logits, in
// fp32: o as [dv / 4][H][4], then records [H][4] {m, l, -, -}.  Consecutive heads store contiguous
// 16-byte pieces.  (o in fp16 with a power of two per 128 dims halves the bytes, which cross the L2
// twice - 4 sequences of 8192 rows 31.8 us instead of 33.1, 32 ragged ones 96.0 instead of 98.9 - but
// rounds each piece's sums by up to 2^-11 before they are joined, and some percent of the bf16 outputs
// then come out a step away from the rounded sum.)
__host__ __device__ inline size_t paged_part_block(int H, int dv) { return (size_t)H * (dv + 4); }      // floats
__host__ __device__ inline size_t paged_part_val(int H, int h, int c) { return ((size_t)(c >> 2) * H + h) * 4 + (c & 3); }
__host__ __device__ inline size_t paged_part_rec(int H, int dv, int h) { return (size_t)dv * H + 4 * (size_t)h; }

// After the partials, one note per unit: {b, n} when sequence b begins in the unit and goes on
// in the n - 1 units after it, {-, 0} otherwise.
__host__ __device__ inline int2* paged_notes(const PagedAttnArgs& a) {
  return reinterpret_cast<int2*>(a.part + 2 * (size_t)a.units * paged_part_block(a.H, a.dv));
}
// Writes the unit's note (one thread).
__device__ __forceinline__ void paged_note(const PagedAttnArgs& a, const PagedPlan& p, int unit) {
  const int64_t end = (int64_t)(unit + 1) * p.per;    // first place of the next unit
  int2 note = make_int2(-1, 0);
  if (end < p.total) {
    int64_t at = p.before;
    for (int b = p.b;; ++b) {                         // the sequence that holds place `end`
      const int64_t n = paged_places(a, b);
      if (end < at + n) {
        const int64_t first = at + a.begin_cost;      // of its first tile
        if (first < end && first >= end - p.per) note = make_int2(b, (int)((at + n - 1) / p.per) - unit + 1);
        break;
      }
      at += n;
    }
  }
  paged_notes(a)[unit] = note;
}

// Row v of segment A (entries or index slots) of sequence b: its row in the pool, or -1
// (an unused slot, or a bad entry or page, which sets CSA_DEVERR_INDEX).
__device__ __forceinline__ int64_t paged_row(const PagedAttnArgs& a, int b, int v) {
  int e = v;
  if (a.idx) {
    e = a.idx[(size_t)b * a.k + v];
    if (e < 0) return -1;
    if ((int64_t)e >= paged_capacity(a)) { raise_err(a.err, CSA_DEVERR_INDEX); return -1; }
  }
  const int pg = paged_page(a, e), id = a.table[(size_t)b * a.table_w + pg];
  if (id < 0 || (int64_t)id >= a.n_pages) { raise_err(a.err, CSA_DEVERR_INDEX); return -1; }
  return (int64_t)id * a.page + (e - pg * a.page);
}

// The sink's share of the denominator, e^{sink - M} with M = max(sink, ...): exact where the sink is the
// maximum, so that an infinite one takes all of the probability; a NaN shows.
__device__ __forceinline__ float paged_sink(float sink, float M) {
  return sink == M ? (sink == -INFINITY ? 0.f : 1.f) : __expf(sink - M);
}

// Units of an attention launch over `ctas` CTAs per head group: no more than the tiles that
// the shapes allow, so that a short context launches few CTAs.
inline int paged_units(int ctas, int B, int64_t rows_max, int tile, int min_tiles) {
  const int64_t tiles = (int64_t)B * (rows_max / tile + 2);            // entries and window end in their own tiles
  const int64_t u = (tiles + min_tiles - 1) / min_tiles;
  return (int)(u < ctas ? (u < 1 ? 1 : u) : (ctas < 1 ? 1 : ctas));
}
// The launch knows entries and window apart: at most this many units of the above are of use.
inline int paged_units(const PagedAttnArgs& a, int units) {
  const int64_t rows = a.idx ? (int64_t)a.k : paged_capacity(a);
  const int up = (1 << a.tile_log2) - 1;
  const int64_t tiles = a.B * (((rows + up) >> a.tile_log2) + ((a.W + up) >> a.tile_log2));
  const int64_t u = (tiles + a.min_tiles - 1) / a.min_tiles;
  return (int)(u < units ? (u < 1 ? 1 : u) : units);
}
inline size_t paged_ws_bytes(int units, int H, int dv) {
  return 2 * (size_t)units * paged_part_block(H, dv) * sizeof(float) + (size_t)units * sizeof(int2);
}
// Rows that one sequence may have: the workspace size and the launch use the same number.
inline int64_t paged_rows_max(const PagedAttnArgs& a) { return (a.idx ? (int64_t)a.k : paged_capacity(a)) + a.W; }
int paged_units_cc(int B, int H, int64_t rows_max);
int paged_units_tc(int B, int H, int64_t rows_max);

// Joins the pieces of cut sequences (a.units as in the attention launch, whose notes name them).
cudaError_t launch_paged_merge(const PagedAttnArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_paged_attn_cc(PagedAttnArgs a, int dtype, cudaStream_t st);
// bf16, d_k = 576, d_v = 512 only.
cudaError_t launch_paged_attn_tc(PagedAttnArgs a, cudaStream_t st);

}  // namespace csa
