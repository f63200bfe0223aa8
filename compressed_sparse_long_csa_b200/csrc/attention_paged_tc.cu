// Attention of one new token per sequence over a paged latent cache on the 5th-generation
// tensor cores (tcgen05, sm_100a): bf16 rows of 576 = 512 + 64 dims, up to 128 heads.
//
// Mathematics as in attention_paged.cu (an online softmax over 64-row tiles).  A CTA takes
// 64 heads (the MMA M) and one unit of the schedule (paged.cuh): a run of tiles that may span
// several sequences ("segments").  Per tile:
//   1. five warps bring the 64 rows, in 128-byte swizzle atoms: runs of pages as TMA boxes of
//      gcd(page, 64) rows, others (selected entries, pages that share no factor of 8 with 64,
//      the last rows of a sequence) by tile::gather4; another warp looks the rows up a tile
//      ahead.  Dims 0-255 have a ring of two slots and dims 256-575 one of three.  Rows that are
//      not attended are never copied: P = 0 there, but 0 * NaN must not reach the sums;
//   2. one warp issues S = Q K^T (N = 64, 36 steps of K = 16) into TMEM.  The queries' dims 0-383
//      are the A operand from TMEM (they come through a ring slot and tcgen05.cp, once per
//      sequence), which leaves their 48 KB to the third slot;
//   3. eight softmax warps read S, agree on the running maximum and write P to shared memory
//      as two bf16 parts, P_hi = bf16(P) and P_lo = bf16(P - P_hi) (the second into the
//      tile's rotary atom, which only S reads): P is held to 2^-17, where bf16 alone would
//      add as much error as the rounding of the output;
//   4. O += P_hi V + P_lo V (N = 2 x 256, V read MN-major from the same tile), dims 0-255 first:
//      their slot is the next that a load waits for.
// The MMAs are the weight-stationary form at M = 64: O (64 x 512) takes 128 lanes x 256 columns
// and S 128 lanes x 32 columns, so lane l and lane l + 64 hold halves of the same head.
// At a segment's end O is normalised and stored, or left as a partial for the merge.
// Every wait on an mbarrier is bounded (CSA_DEVERR_TIMEOUT).  The named barriers between the lookup and
// the copying warps have no limit; all of these warps take every one of them: a copying warp that is to
// stop writes ld_stop before the barrier of a tile, all six read it behind that barrier and leave at
// the same tile, and what a warp does between two barriers waits on mbarriers only.
//
// Bound: at 64 heads HBM (two sequences of up to 131 072 rows: 71 us, 4.1 TB/s of 6.56 measured,
// start and merge included), at 128 heads the MMAs and the shared memory that they read (2432
// cycles of MMAs a tile; 32 ragged sequences of 200 296 rows in all: 98.5 us, 566 TFLOP/s, 1.9 us a
// tile, of which a tile's chain load 1.1 us, S 0.7, softmax 0.9, PV 0.8 is overlapped by two), for
// gathered rows the gathers (48 x 1152 rows: 51.4 us, 2.4 us a tile: 30 GB/s beside the MMAs' operands, 55
// alone), for one sequence latency (100 rows: 11.5 us).
// Two slots for all dims and all queries in shared memory: 10% more for the ragged ones, 5% for 64 heads.
// Why 64 heads a CTA: O of 128 heads (512 columns) would leave no TMEM for S.  Why two bf16
// parts of P: one part took 5% off 64 heads when that was tried, for the error above.
// Why few warps poll: all copying warps waiting on the slots' barriers cost the ragged batch
// 5% against one thread and a named barrier; each test of a barrier goes through the shared
// memory that the MMAs read.
#include "paged.cuh"
#include "tc.cuh"

#include <cudaTypedefs.h>

namespace csa {

namespace {

constexpr int PT_ROWS = 64;              // rows per tile (N of QK^T, K of PV)
constexpr int PT_HC = 64;                // heads per CTA (MMA M)
constexpr int PT_ATOMS = 9;              // 576 dims = 9 atoms of 64 dims (128 bytes)
constexpr int PT_LO = 4;                 // atoms of a tile's first half (dims 0-255)
constexpr int PT_SMW = 8;                // softmax warps: two warpgroups, one per half of a lane's columns
constexpr int PT_SW = 8;                 // the warp of the queries and S
constexpr int PT_PVW = 9;                // the warp of PV
constexpr int PT_LDW = 10;               // the warp that looks rows up
constexpr int PT_CPW = 11;               // first of five that copy them
constexpr int PT_CPT = 160, PT_LDT = 32 + PT_CPT;           // threads of the latter; of both
constexpr int PT_THREADS = PT_CPW * 32 + PT_CPT;
constexpr int PT_MIN_TILES = 2;         // (one sequence of two tiles: 11.6 us in one unit, 13.5 in two and a merge)
constexpr int PT_BEGIN_COST = 2;         // (32 ragged sequences: 100.8 us at 1, 98.5 at 2, 99.8 at 3)
constexpr float PT_RESCALE = 8.0f;       // base-2 units: O is rescaled once the maximum has grown 256-fold
constexpr int ATOM = PT_ROWS * 128;      // one 64-row x 128-byte swizzle atom
constexpr int PT_QT = 6;                 // atoms of the queries that live in TMEM
constexpr uint32_t TM_O = 0, TM_S = 256, TM_Q = 320, TM_COLS = 512;    // TMEM columns: O 256, S 2 x 32, queries 6 x 32
static_assert(PT_THREADS == 512, "16 warps: 128 registers a thread");

struct PtSmem {
  uint8_t q[PT_ATOMS - PT_QT][PT_HC * 128];  // 24 KB
  uint8_t lo[2][PT_LO][ATOM];                // 64 KB: dims 0-255 of two tiles
  uint8_t hi[3][PT_ATOMS - PT_LO][ATOM];     // 120 KB: dims 256-575 of three
  uint8_t p[PT_HC * 128];                    // P_hi: 64 heads x 64 rows bf16; between segments the row sums
  float smax[2][2][128];                     // per tile parity and warpgroup: the lanes' tile maxima
  alignas(16) int rowy[2][PT_ROWS];          // per tile mod 2: rows of the pool or the window, -1 = none
  uint32_t vmask[4][2];                      // per tile mod 4 (a tile's are written when the softmax is past those of
                                             // four tiles before): bit j of word j / 32 set when row j exists
  uint64_t lo_full[2], lo_empty[2], hi_full[3], hi_empty[3];
  uint64_t sfull[2], sfree[2];
  uint64_t pfull, pdone, qfull, qfree, ofree, drain[2];
  uint64_t headb[2], segb;                   // softmax warps: the four of the same heads; all eight
  uint32_t tmem_base;
  int abort_flag;
  int ld_stop;                               // 1 + the tile at which lookups and copies stop (0 = running)
};
static_assert(sizeof(PtSmem) <= 232448, "shared memory of one CTA (227 KB)");

struct PtMaps {
  CUtensorMap q;       // [B * H rows, 576], box 64 x 64
  CUtensorMap pages;   // [n_pages * page rows, 576], box 64 dims x box rows
  CUtensorMap win;     // [B * W rows, 576], box 64 x 64
  CUtensorMap rows, win_rows;   // pages and window again, box 64 dims x 1 row (tile::gather4)
};

__device__ __forceinline__ void named_bar(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 bytes by one store: a whole sector (`wide`: the address is a multiple of 32), or two of 16
__device__ __forceinline__ void st_global32(void* p, const uint32_t* w, bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  else
    for (int i = 0; i < 2; ++i) reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}
// 2^x by the MUFU.EX2 unit (relative error about 2^-22)
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// byte offset of 16-byte chunk c of row j in a 128-byte-swizzled atom
__device__ __forceinline__ uint32_t sw128_off(int j, int c) { return (j >> 3) * 1024 + (j & 7) * 128 + ((c ^ (j & 7)) << 4); }

// A place in a ring of slots and its phase.
struct RingPos {
  int at;
  uint32_t ph;
  __device__ __forceinline__ void step(int n) {
    if (++at == n) { at = 0; ph ^= 1; }
  }
};

template <bool SPARSE>
__global__ void __launch_bounds__(PT_THREADS, 1)
paged_attn_tc_kernel(const __grid_constant__ PtMaps maps, const __grid_constant__ PagedAttnArgs a, int halves, int box) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PtSmem& sm = *reinterpret_cast<PtSmem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / halves, hh = blockIdx.x - unit * halves;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 3; ++s) {
      tc::mbar_init(&sm.hi_full[s], 1);
      tc::mbar_init(&sm.hi_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.lo_full[s], 1);
      tc::mbar_init(&sm.lo_empty[s], 1);
      tc::mbar_init(&sm.sfull[s], 1);
      tc::mbar_init(&sm.sfree[s], PT_SMW);
      tc::mbar_init(&sm.drain[s], 1);
    }
    tc::mbar_init(&sm.pfull, PT_SMW);
    tc::mbar_init(&sm.pdone, 1);
    tc::mbar_init(&sm.qfull, 1);
    tc::mbar_init(&sm.qfree, 1);
    tc::mbar_init(&sm.ofree, PT_SMW);
    for (int s = 0; s < 2; ++s) tc::mbar_init(&sm.headb[s], 4);
    tc::mbar_init(&sm.segb, PT_SMW);
    sm.abort_flag = 0;
    sm.ld_stop = 0;
    tc::fence_mbar_init();
  }
  if (warp == PT_SW) { tc::tmem_alloc(&sm.tmem_base, TM_COLS); tc::tmem_relinquish(); }
  tc::griddep_wait();                               // the setup overlaps the preceding kernel's tail
  tc::fence_before_sync();
  const PagedPlan plan = paged_plan(a, unit, PT_THREADS, reinterpret_cast<int64_t*>(sm.q));
  tc::fence_after_sync();
  tc::fence_proxy_async_smem();
  __syncthreads();                                  // the plan's scratch is read; Q may land there
  const uint32_t tmem = sm.tmem_base;
  PagedSeg seg;                                     // every role walks the unit's segments by itself
  seg.start(plan, unit);

  if (warp >= PT_CPW) {
    // ------------------------------------------------------------------ copies (5 warps)
    // Ring slots, in order: per segment one for the queries' atoms that go to TMEM, then its tiles.
    const int w = warp - PT_CPW, ct = threadIdx.x - PT_CPW * 32;
    RingPos lo{0, 0}, hi{0, 0};                       // the next slot of each ring
    int n_lo = 0, n_hi = 0;                           // slots started (for the drain)
    auto half_free = [&](int x) { return x ? tc::mbar_wait(&sm.hi_empty[hi.at], hi.ph ^ 1) : tc::mbar_wait(&sm.lo_empty[lo.at], lo.ph ^ 1); };
    auto half_full = [&](int x) { return x ? &sm.hi_full[hi.at] : &sm.lo_full[lo.at]; };
    auto atom_of = [&](int at) { return at < PT_LO ? sm.lo[lo.at][at] : sm.hi[hi.at][at - PT_LO]; };
    int i = 0;
    bool go_on = true;
    while (go_on && seg.next(a)) {
      bool in_time = true;
      {
        // warps 0-3: an atom of dims 0-255 each; 4: the next two
        static_assert(PT_LO == 4 && PT_QT == 6 && PT_CPT == 160, "a warp's atoms");
        const int x = w >> 2;
        if (lane == 0) {
          in_time = half_free(x);
          if ((w & 3) == 0) tc::mbar_arrive_expect_tx(half_full(x), (x ? PT_QT - PT_LO : PT_LO) * ATOM);
          for (int at = w; in_time && at < w + 1 + x; ++at)
            tc::tma_load_2d(atom_of(at), &maps.q, half_full(x), 64 * at, seg.b * a.H + hh * PT_HC);
        }
        in_time = __shfl_sync(0xffffffffu, in_time, 0);
        ++n_lo;
        ++n_hi;
        lo.step(2);
        hi.step(3);
      }
      for (int64_t t = seg.t0; t < seg.t1; ++t, ++i) {
        const int st = i & 1;
        const bool in_a = t < seg.ta;
        if (*(volatile int*)&sm.abort_flag || !in_time) sm.ld_stop = i + 1;       // all leave together below
        named_bar(1, PT_LDT);                         // the tile's rows are there
        const int stop = *(volatile int*)&sm.ld_stop;
        if (stop != 0 && stop <= i + 1) { go_on = false; break; }
        const uint32_t v0 = sm.vmask[i & 3][0], v1 = sm.vmask[i & 3][1];
        const int rows = in_a ? box : PT_ROWS;        // rows per TMA box; box 0: pages that no box fits
        const bool boxes = (v0 & v1) == 0xffffffffu && (in_a ? !SPARSE && box > 0 : true);
        // Dims 256-575 (x = 1) first, whose slot has long been free; dims 0-255 as soon as the PV of two
        // tiles before is past them.
#pragma unroll 1
        for (int x = 1; x >= 0; --x) {
          const int at0 = x ? PT_LO : 0, at1 = x ? PT_ATOMS : PT_LO;
          // (one thread polls: five warps that do slow the MMAs' operands)
          if (ct == 0 && !half_free(x)) atomicExch(&sm.abort_flag, 1);
          named_bar(2, PT_CPT);
          in_time = !*(volatile int*)&sm.abort_flag;
          if ((v0 | v1) == 0u) {
            // no row at all: zeros
            for (int p = ct; p < (at1 - at0) * ATOM / 16 && in_time; p += PT_CPT)
              reinterpret_cast<uint4*>(atom_of(at0))[p] = make_uint4(0u, 0u, 0u, 0u);
            tc::fence_proxy_async_smem();
            named_bar(2, PT_CPT);
            if (ct == 0) tc::mbar_arrive(half_full(x));
          } else if (in_time) {
            if (ct == 0) tc::mbar_arrive_expect_tx(half_full(x), (at1 - at0) * ATOM);
            if (boxes) {
              // a run of rows, or of pages: atoms over the warps, a lane per box (one thread takes 0.1 us a copy)
              for (int at = at0 + w; at < at1; at += PT_CPT / 32)
                if (lane * rows < PT_ROWS)
                  tc::tma_load_2d(atom_of(at) + lane * rows * 128, in_a ? &maps.pages : &maps.win, half_full(x), 64 * at, sm.rowy[st][lane * rows]);
            } else {
              // scattered rows by tile::gather4, four rows of 128 bytes an instruction.  Alone, one warp
              // starts 16 GB/s of them, six 55 (cp.async by as many threads: 46, and it needs the issue
              // slots and shared-memory ports that the softmax uses).  An absent row is a second copy of one
              // that is there: its P is 0, and what it holds must not be less finite than the rest.
              const int there = sm.rowy[st][v0 ? __ffs(v0) - 1 : 31 + __ffs(v1)];
              const CUtensorMap* m = in_a ? &maps.rows : &maps.win_rows;
              for (int p = lane * (PT_CPT / 32) + w; p < (at1 - at0) * (PT_ROWS / 4); p += PT_CPT) {
                const int quad = p & (PT_ROWS / 4 - 1), at = at0 + p / (PT_ROWS / 4);
                int4 r = *reinterpret_cast<const int4*>(&sm.rowy[st][4 * quad]);
                r.x = r.x < 0 ? there : r.x;
                r.y = r.y < 0 ? there : r.y;
                r.z = r.z < 0 ? there : r.z;
                r.w = r.w < 0 ? there : r.w;
                tc::tma_gather4(atom_of(at) + quad * 512, m, half_full(x), 64 * at, r);
              }
            }
            __syncwarp();
          }
          if (x) ++n_hi; else ++n_lo;
        }
        lo.step(2);
        hi.step(3);
        if (!in_time) atomicExch(&sm.abort_flag, 1);
      }
    }
    // drain: no TMA write of this CTA may be in flight when the CTA exits
    if (ct == 0)
      for (int q = 0; q < 5; ++q) {
        const int uses = q < 2 ? (n_lo + 1 - q) / 2 : (n_hi + 4 - q) / 3;      // of a ring's slot
        if (uses > 0 && !tc::mbar_wait(q < 2 ? &sm.lo_full[q] : &sm.hi_full[q - 2], (uses - 1) & 1)) atomicExch(&sm.abort_flag, 1);
      }
    __syncwarp();
  } else if (warp >= PT_LDW) {
    // ------------------------------------------------------------------ row lookups
    // Lane j looks up rows j and j + 32 of the tiles ahead, a step of the chain entry -> page -> row per
    // tile, so that no load is waited for where it is issued; the rows of tile i + 1 while tile i is copied.
    struct Row {
      bool is, in_a;                                  // a tile of the unit; of the entries (else of the window)
      int b, e[2], at[2], id[2];                      // sequence; entry (or the window's row), -1 = none; its row in the page; page id
    };
    const int cap = (int)paged_capacity(a);
    int64_t t = 0;
    bool more = seg.next(a);
    if (more) t = seg.t0;
    auto entry_of = [&]() {                           // the next tile: the entries
      Row r{more, t < seg.ta, seg.b, {-1, -1}, {0, 0}, {0, 0}};
      if (!more) return r;
      const int v0 = (int)((r.in_a ? t : t - seg.ta) * PT_ROWS) + lane, n = r.in_a ? seg.na : seg.nw;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int v = v0 + 32 * u;
        if (v < n) r.e[u] = !r.in_a ? seg.b * a.W + v : SPARSE ? a.idx[(size_t)seg.b * a.k + v] : v;
      }
      if (++t == seg.t1) {
        more = seg.next(a);
        t = seg.t0;
      }
      return r;
    };
    auto page_of = [&](Row r) {                       // their pages
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        r.id[u] = -1;
        if (r.in_a && r.e[u] >= 0 && (!SPARSE || r.e[u] < cap)) {
          const int pg = paged_page(a, r.e[u]);
          r.at[u] = r.e[u] - pg * a.page;
          r.id[u] = a.table[(size_t)r.b * a.table_w + pg];
        }
      }
      return r;
    };
    // the rows of the pool or the window, -1 = none, and which there are
    auto publish = [&](int i, const Row& r) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        int y = r.e[u];
        if (r.in_a && y >= 0) {
          if ((unsigned)r.id[u] < (unsigned)a.n_pages) y = r.id[u] * a.page + r.at[u];       // (a pool has less than 2^31 rows)
          else { raise_err(a.err, CSA_DEVERR_INDEX); y = -1; }
        }
        sm.rowy[i & 1][lane + 32 * u] = y;            // (the copies of two tiles before are started)
        const uint32_t vb = __ballot_sync(0xffffffffu, y >= 0);
        if (lane == 0) sm.vmask[i & 3][u] = vb;
      }
    };
    Row now = page_of(entry_of()), next = now, after = now;
    if (now.is) publish(0, now);
    for (int i = 0; now.is; ++i) {
      named_bar(1, PT_LDT);
      const int stop = *(volatile int*)&sm.ld_stop;
      if (stop != 0 && stop <= i + 1) break;
      if (i == 0) {                                   // (the first tile's copies wait for no other's rows)
        next = entry_of();
        after = entry_of();
        next = page_of(next);
      }
      now = next;
      next = page_of(after);
      after = entry_of();
      if (now.is) publish(i + 1, now);
    }
  } else if (warp == PT_SW) {
    // ------------------------------------------------------------------ queries and S = Q K^T
    // The whole warp runs the loop (descriptors stay warp-uniform), one elected lane issues.  S
    // and PV have a warp each: every wait is then the one thing its warp waits for.  (One warp
    // that polled all barriers lost 800 to 2500 cycles per batch: under the MMAs' operand
    // traffic each test of a barrier takes hundreds.)
    constexpr uint32_t ID_S = tc::idesc(tc::FMT_BF16, tc::FMT_BF16, PT_HC, PT_ROWS);
    const uint64_t q_d = tc::desc_k_sw128(tc::smem_u32(sm.q[0]));
    const uint64_t lo_d = tc::desc_k_sw128(tc::smem_u32(sm.lo[0][0])), hi_d = tc::desc_k_sw128(tc::smem_u32(sm.hi[0][0]));
    RingPos lo{0, 0}, hi{0, 0};
    if (lane == 0) {
      tc::prefetch_tmap(&maps.q);
      tc::prefetch_tmap(&maps.pages);
      tc::prefetch_tmap(&maps.win);
      tc::prefetch_tmap(&maps.rows);
    }
    bool ok = true;
    int n = 0, i = 0;
    tc::ArmedLoads queries;
    for (; ok && seg.next(a); ++n) {
      // the segment before no longer reads Q once its last S is complete
      if (n > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(&sm.qfree, (n - 1) & 1))) { ok = false; break; }
      queries.arm();
      if (tc::elect_one()) {
        tc::mbar_arrive_expect_tx(&sm.qfull, (PT_ATOMS - PT_QT) * PT_HC * 128);
        for (int at = PT_QT; at < PT_ATOMS; ++at)
          tc::tma_load_2d(sm.q[at - PT_QT], &maps.q, &sm.qfull, 64 * at, seg.b * a.H + hh * PT_HC);
      }
      __syncwarp();
      for (int64_t t = seg.t0; t < seg.t1; ++i) {
        // The first turn issues nothing (live = 0): while the first tile loads, it brings the
        // instructions in; cold, the first S took 4 us, later ones 1.
        const uint32_t live = i > 0;
        const int x = i - 1, st = x & 1;
        const uint32_t d = tmem + TM_S + st * 32;
        if (live && t == seg.t0) {
          // the queries to TMEM (their slots are free again once that is done), and the rest of them
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.lo_full[lo.at], lo.ph));
          if (ok && tc::elect_one()) {
#pragma unroll 1
            for (int at = 0; at < PT_LO; ++at)
              tc::cp_atom_ws(tmem + TM_Q + 32 * at, lo_d + (uint64_t)((lo.at * PT_LO + at) * (ATOM >> 4)));
            tc::mma_commit(&sm.lo_empty[lo.at]);
          }
          __syncwarp();
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.hi_full[hi.at], hi.ph));
          if (ok && tc::elect_one()) {
#pragma unroll 1
            for (int at = PT_LO; at < PT_QT; ++at)
              tc::cp_atom_ws(tmem + TM_Q + 32 * at, hi_d + (uint64_t)((hi.at * (PT_ATOMS - PT_LO) + at - PT_LO) * (ATOM >> 4)));
            tc::mma_commit(&sm.hi_empty[hi.at]);
          }
          __syncwarp();
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.qfull, n & 1));
          if (!ok) break;
          lo.step(2);
          hi.step(3);
        }
        const uint64_t kl = lo_d + (uint64_t)(lo.at * PT_LO * (ATOM >> 4)), kh = hi_d + (uint64_t)(hi.at * (PT_ATOMS - PT_LO) * (ATOM >> 4));
        // (S of two tiles before has been read)
        const bool go = !live || (tc::mbar_wait(&sm.sfree[st], ((x >> 1) & 1) ^ 1) && tc::mbar_wait(&sm.hi_full[hi.at], hi.ph));
        ok = __all_sync(0xffffffffu, go && !*(volatile int*)&sm.abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int at = PT_LO; at < PT_QT; ++at)        // 4 steps of 16 dims an atom; atoms are 8 KB apart
          tc::mma_f16_ws_ts_x4<2>(d, tmem + TM_Q + 32 * at, kh + (uint64_t)((at - PT_LO) * (ATOM >> 4)), ID_S, at > PT_LO, live);
#pragma unroll
        for (int at = PT_QT; at < PT_ATOMS; ++at)
          tc::mma_f16_ws_x4<2>(d, q_d + (uint64_t)((at - PT_QT) * (ATOM >> 4)), kh + (uint64_t)((at - PT_LO) * (ATOM >> 4)), ID_S, 1, live);
        ok = __all_sync(0xffffffffu, !live || tc::mbar_wait(&sm.lo_full[lo.at], lo.ph));
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int at = 0; at < PT_LO; ++at)
          tc::mma_f16_ws_ts_x4<2>(d, tmem + TM_Q + 32 * at, kl + (uint64_t)(at * (ATOM >> 4)), ID_S, 1, live);
        if (live) {
          ++t;
          lo.step(2);
          hi.step(3);
          if (tc::elect_one()) {
            tc::mma_commit(&sm.sfull[st]);
            if (t == seg.t1) tc::mma_commit(&sm.qfree);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) atomicExch(&sm.abort_flag, 1);
    // no copy of the queries and no MMA is in flight when the CTA frees TMEM and exits
    if (queries.any()) tc::mbar_wait(&sm.qfull, queries.last());
    if (tc::elect_one()) tc::mma_commit(&sm.drain[0]);
    __syncwarp();
    if (!tc::mbar_wait(&sm.drain[0], 0) && lane == 0) atomicExch(&sm.abort_flag, 1);
  } else if (warp == PT_PVW) {
    // ------------------------------------------------------------------ O (+)= (P_hi + P_lo) V
    // Value dims 0-255 (atoms 0-3), then 256-511 (atoms 4-7), so that the slot of the first
    // is free early.  The two parts of P are two K ranges over the same V rows (a K step is 16
    // rows of 128 bytes).
    constexpr uint32_t ID_O = tc::idesc(tc::FMT_BF16, tc::FMT_BF16, PT_HC, 256, 0, 1);
    const uint64_t p_d = tc::desc_k_sw128(tc::smem_u32(sm.p));
    const uint64_t pl_d0 = tc::desc_k_sw128(tc::smem_u32(sm.hi[0][PT_ATOMS - PT_LO - 1]));
    const uint64_t lo_d = tc::desc_mn_sw128(tc::smem_u32(sm.lo[0][0]), ATOM, 1024), hi_d = tc::desc_mn_sw128(tc::smem_u32(sm.hi[0][0]), ATOM, 1024);
    RingPos lo{0, 0}, hi{0, 0};
    bool ok = true;
    int n = 0, i = 0;
    for (; ok && seg.next(a); ++n) {
      for (int64_t t = seg.t0; t < seg.t1; ++i) {
        const uint32_t live = i > 0;                  // the first turn issues nothing, as above
        const int x = i - 1;
        const bool first = t == seg.t0;               // overwrites O, which the epilogue before has read
        if (live && first) {                          // past the queries' slots
          lo.step(2);
          hi.step(3);
        }
        const uint64_t hi_at = (uint64_t)(hi.at * (PT_ATOMS - PT_LO) * (ATOM >> 4));
        const uint64_t vd = lo_d + (uint64_t)(lo.at * PT_LO * (ATOM >> 4)), vh = hi_d + hi_at, pl = pl_d0 + hi_at;
        const bool go = !live || ((!first || n == 0 || tc::mbar_wait(&sm.ofree, (n - 1) & 1)) && tc::mbar_wait(&sm.pfull, x & 1));
        ok = __all_sync(0xffffffffu, go && !*(volatile int*)&sm.abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        tc::mma_f16_ws_x4<128>(tmem + TM_O, p_d, vd, ID_O, !first, live);
        tc::mma_f16_ws_x4<128>(tmem + TM_O, pl, vd, ID_O, 1, live);
        if (live && tc::elect_one()) tc::mma_commit(&sm.lo_empty[lo.at]);
        __syncwarp();
        tc::mma_f16_ws_x4<128>(tmem + TM_O + 128, p_d, vh, ID_O, !first, live);
        tc::mma_f16_ws_x4<128>(tmem + TM_O + 128, pl, vh, ID_O, 1, live);
        if (live) {
          ++t;
          if (tc::elect_one()) {
            tc::mma_commit(&sm.hi_empty[hi.at]);
            tc::mma_commit(&sm.pdone);
          }
          lo.step(2);
          hi.step(3);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) atomicExch(&sm.abort_flag, 1);
    if (tc::elect_one()) tc::mma_commit(&sm.drain[1]);
    __syncwarp();
    if (!tc::mbar_wait(&sm.drain[1], 0) && lane == 0) atomicExch(&sm.abort_flag, 1);
  } else {
    // ------------------------------------------------------------------ softmax + epilogue, warps 0-7
    // Thread (wg, lane tl): head tl % 64; of S the tile rows 32 (tl / 64) + 16 wg .. + 15; of O
    // the dims 256 wg + 128 (tl / 64) .. + 127.
    const int wg = warp >> 2, quarter = warp & 3;
    const int tl = quarter * 32 + lane;
    const int hl = tl & 63, half = tl >> 6;
    const int h = hh * PT_HC + hl;
    const bool hv = h < a.H;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint64_t* const headb = &sm.headb[quarter & 1];
    // all softmax warps meet (a bounded wait, unlike a named barrier)
    uint32_t met = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.segb);
      return __all_sync(0xffffffffu, tc::mbar_wait(&sm.segb, met++ & 1));
    };
    // logits in the base-2 domain: P = 2^(s - m), m set to PT_RESCALE above the maximum, so that P <= 1
    // while O is not rescaled: sums of values come no nearer to the type's end than the formula's
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    const float scale2 = a.sm_scale * 1.4426950408889634f;
    const float scale = fmaxf(fabsf(scale2), 1.2e-38f);          // not 0: an absent row's -inf must stay one
    bool ok = true;
    int i = 0;                                        // tiles so far, over all segments
    RingPos lo{0, 0}, hi{0, 0};
    // sequences without a row (no unit has a tile of theirs): a lane looks at each, the warp clears
    for (int b0 = unit + warp * 32 * a.units; b0 < a.B; b0 += PT_SMW * 32 * a.units) {
      const int64_t bl = (int64_t)b0 + (int64_t)lane * a.units;
      const bool none = bl < a.B && paged_rows_a(a, (int)bl) == 0 && paged_rows_w(a, (int)bl) == 0;
      for (unsigned left = __ballot_sync(0xffffffffu, none); left; left &= left - 1) {
        const int b = b0 + (__ffs(left) - 1) * a.units, n = min(PT_HC, a.H - hh * PT_HC);
        uint4* o = reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + ((size_t)b * a.H + hh * PT_HC) * 512);
        for (int c = lane; c < n * 64; c += 32) o[c] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse)
          for (int c = hh * PT_HC + lane; c < hh * PT_HC + n; c += 32) a.lse[(size_t)b * a.H + c] = a.sink[c];
      }
    }
    __syncwarp();
    if (threadIdx.x == 0 && hh == 0) paged_note(a, plan, unit);
    while (ok && seg.next(a)) {
      const float sink = hv ? a.sink[h] : 0.f;
      float m_run = -INFINITY, l_run = 0.f;           // running maximum; this thread's row sum
      lo.step(2);                                     // past the queries' slots
      hi.step(3);
      for (int64_t t = seg.t0; t < seg.t1; ++t, ++i, lo.step(2), hi.step(3)) {
        const int st = i & 1;
        const uint32_t ph = (i >> 1) & 1;
        bool w = tc::mbar_wait(&sm.lo_full[lo.at], lo.ph);      // the mask of the tile's rows
        const uint32_t vm = sm.vmask[i & 3][half] >> (16 * wg);
        w = w && tc::mbar_wait(&sm.sfull[st], ph);
        w = __all_sync(0xffffffffu, w && !*(volatile int*)&sm.abort_flag);
        if (!w) { ok = false; break; }
        tc::fence_after_sync();
        float s[16];
        {
          uint32_t v[16];
          tc::tmem_ld16(tmem + lane_base + TM_S + st * 32 + 16 * wg, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = __uint_as_float(v[j]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.sfree[st]);
        if (scale2 < 0.f) {
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = -s[j];
        }
        if ((vm & 0xffffu) != 0xffffu) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (!((vm >> j) & 1u)) s[j] = -INFINITY;
        }
        float mq[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < 16; ++j) mq[j & 3] = fmaxf(mq[j & 3], s[j]);
        float mt = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * scale;
        // The tile's maximum over the head's four threads.  P is formed with the maximum so
        // far while theirs arrive, and once more where it has to rise.
        float* const mx = sm.smax[st][0];
        mx[wg * 128 + tl] = mt;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(headb);
        const bool p_free = i == 0 || tc::mbar_test(&sm.pdone, (i - 1) & 1);
        bool rescale = false;
        float alpha = 1.f, psum;
        uint32_t w8[8], l8[8];
        for (bool met_all = false;;) {
          const float m0 = m_run == -INFINITY ? 0.f : m_run;
          psum = 0.f;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float p0 = ex2_approx(fmaf(s[2 * u], scale, -m0)), p1 = ex2_approx(fmaf(s[2 * u + 1], scale, -m0));
            const __nv_bfloat162 hb = __floats2bfloat162_rn(p0, p1);
            const __nv_bfloat162 lb = __floats2bfloat162_rn(p0 - __low2float(hb), p1 - __high2float(hb));
            psum += p0 + p1;
            w8[u] = *reinterpret_cast<const uint32_t*>(&hb);
            l8[u] = *reinterpret_cast<const uint32_t*>(&lb);
          }
          if (met_all) break;
          if (!__all_sync(0xffffffffu, tc::mbar_wait(headb, i & 1))) { ok = false; break; }
          met_all = true;
          mt = fmaxf(fmaxf(mx[hl], mx[hl + 64]), fmaxf(mx[hl + 128], mx[hl + 192]));
          const bool raise = mt > m_run;
          if (!__any_sync(0xffffffffu, raise)) break;
          if (raise) {
            const float m_new = mt + PT_RESCALE;
            alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new);
            rescale = m_run != -INFINITY;
            m_run = m_new;
          }
        }
        if (!ok) break;
        const bool rescale_any = __any_sync(0xffffffffu, rescale);
        l_run = l_run * alpha + psum;
        // the PV before owns P and O until it completes
        if (!__all_sync(0xffffffffu, p_free || tc::mbar_wait(&sm.pdone, (i - 1) & 1))) { ok = false; break; }
        tc::fence_after_sync();
        if (rescale_any) {
#pragma unroll 1
          for (int c = 2 * wg; c < 2 * wg + 2; ++c) {
            uint32_t v[64];
            tc::tmem_ld64(tmem + lane_base + TM_O + c * 64, v);
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_st16(tmem + lane_base + TM_O + c * 64 + q * 16, v + q * 16);
          }
          tc::tmem_st_wait();
        }
        {
          // P_lo goes to the tile's rotary atom: S of this tile, its only reader, is complete
          const uint32_t pbase = tc::smem_u32(sm.p), lbase = tc::smem_u32(sm.hi[hi.at][PT_ATOMS - PT_LO - 1]);
          const int c0 = 4 * half + 2 * wg;           // 16-byte chunks (8 rows) of the head's P
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(pbase + sw128_off(hl, c0 + cc)), "r"(w8[4 * cc]),
                         "r"(w8[4 * cc + 1]), "r"(w8[4 * cc + 2]), "r"(w8[4 * cc + 3]) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(lbase + sw128_off(hl, c0 + cc)), "r"(l8[4 * cc]),
                         "r"(l8[4 * cc + 1]), "r"(l8[4 * cc + 2]), "r"(l8[4 * cc + 3]) : "memory");
          }
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.pfull);
      }
      // ---- the segment's end: wait for its last PV, then normalise or leave a partial
      if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.pdone, (i - 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      // the head's row sum: four threads' parts, through the idle P tile
      float* lx = reinterpret_cast<float*>(sm.p);     // [wg][128]
      lx[wg * 128 + tl] = l_run;
      if (!meet()) { ok = false; break; }
      const float l = (lx[hl] + lx[hl + 64]) + (lx[128 + hl] + lx[192 + hl]);
      if (!meet()) { ok = false; break; }             // P may be written again
      const float m = m_run * 0.6931471805599453f;
      float f = 1.f, M = 0.f, den = 0.f;
      float* blk = a.part + (size_t)seg.slot(unit) * paged_part_block(a.H, 512);
      if (seg.whole) {
        M = fmaxf(sink, m);
        const float e = m == -INFINITY ? 0.f : __expf(m - M);
        den = paged_sink(sink, M) + l * e;            // (logits that are all NaN have no maximum, but a sum)
        f = den == 0.f ? 0.f : e / den;
      }
      const int d0 = 256 * wg + 128 * half;
      if (!seg.whole && hv && wg == 0 && half == 0) *reinterpret_cast<float2*>(blk + paged_part_rec(a.H, 512, h)) = make_float2(m, l);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[64];
        __syncwarp();
        tc::tmem_ld64(tmem + lane_base + TM_O + 128 * wg + c * 64, v);
        if (c == 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.ofree);
        }
        if (!hv) continue;
        __nv_bfloat16* o = (__nv_bfloat16*)a.out + ((size_t)seg.b * a.H + h) * 512 + d0 + c * 64;
        if (seg.whole) {
          // each lane has a row of its own: whole sectors, or the store's lines cost as much again
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 bf = __floats2bfloat162_rn(__uint_as_float(v[q * 16 + 2 * j]) * f, __uint_as_float(v[q * 16 + 2 * j + 1]) * f);
              w[j] = *reinterpret_cast<const uint32_t*>(&bf);
            }
            st_global32(o + q * 16, w, wide);
          }
        } else {
          uint4* part = reinterpret_cast<uint4*>(blk + paged_part_val(a.H, h, d0 + c * 64));
#pragma unroll
          for (int q = 0; q < 16; ++q) part[(size_t)q * a.H] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
      __syncwarp();
      if (hv && wg == 0 && half == 0 && seg.whole && a.lse) a.lse[(size_t)seg.b * a.H + h] = den == 0.f ? -INFINITY : M + logf(den);
    }
    if (!ok) atomicExch(&sm.abort_flag, 1);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::griddep_launch_dependents();                  // the merge (which waits for this grid) may take the SM
  if (sm.abort_flag && threadIdx.x == 0) raise_err(a.err, CSA_DEVERR_TIMEOUT);
  if (warp == PT_SW) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, TM_COLS);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (PFN_cuTensorMapEncodeTiled_v12000)p;
  }();
  return fn;
}

// [rows, 576] bf16 rows (1152-byte pitch), box = 64 dims x box rows, 128-byte swizzle.
bool row_map(CUtensorMap* m, const void* base, uint64_t rows, int box) {
  auto enc = get_encode();
  if (!enc || rows == 0) return false;
  cuuint64_t dims[2] = {576, rows};
  cuuint64_t strides[1] = {576 * 2};
  cuuint32_t b[2] = {64, (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// One CTA per SM: with more than 64 heads two CTAs share a unit.
int paged_units_tc(int B, int H, int64_t rows_max) {
  return paged_units(num_sms() / (H > PT_HC ? 2 : 1), B, rows_max, PT_ROWS, PT_MIN_TILES);
}

cudaError_t launch_paged_attn_tc(PagedAttnArgs a, cudaStream_t st) {
  const int halves = a.H > PT_HC ? 2 : 1;
  a.tile_log2 = 6;
  static_assert(PT_ROWS == 1 << 6, "tile rows");
  a.min_tiles = PT_MIN_TILES;
  a.begin_cost = PT_BEGIN_COST;
  a.units = paged_units(a, paged_units_tc(a.B, a.H, paged_rows_max(a)));
  // the largest of 64, 32, 16, 8 rows that divides the pages: every box lies in one page
  int box = PT_ROWS;
  while (box >= 8 && a.page % box != 0) box >>= 1;
  if (box < 8) box = 0;
  PtMaps maps;
  if (!row_map(&maps.q, a.q, (uint64_t)a.B * a.H, PT_HC)) return cudaErrorUnknown;
  if (!row_map(&maps.pages, a.pages, (uint64_t)a.n_pages * a.page, box ? box : 8)) return cudaErrorUnknown;
  if (!row_map(&maps.rows, a.pages, (uint64_t)a.n_pages * a.page, 1)) return cudaErrorUnknown;
  if (a.W > 0) {
    if (!row_map(&maps.win, a.win, (uint64_t)a.B * a.W, PT_ROWS)) return cudaErrorUnknown;
    if (!row_map(&maps.win_rows, a.win, (uint64_t)a.B * a.W, 1)) return cudaErrorUnknown;
  } else {
    maps.win = maps.win_rows = maps.rows;            // no tile is ever a window tile
  }
  auto kern = a.idx ? paged_attn_tc_kernel<true> : paged_attn_tc_kernel<false>;
  static std::atomic<uint64_t> ready[2];               // bit per device: the kernel's shared-memory size is set
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), ready[a.idx ? 1 : 0], (int)sizeof(PtSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(halves * a.units);
  cfg.blockDim = dim3(PT_THREADS);
  cfg.dynamicSmemBytes = sizeof(PtSmem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddep_wait in the kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  e = cudaLaunchKernelEx(&cfg, kern, maps, a, halves, box);
  if (e != cudaSuccess) return e;
  return launch_paged_merge(a, CSA_BF16, st);
}

}  // namespace csa
