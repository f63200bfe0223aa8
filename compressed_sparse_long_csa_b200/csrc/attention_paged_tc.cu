// Attention of one new token per sequence over a paged latent cache on the 5th-generation
// tensor cores (tcgen05, sm_100a): bf16 rows of 576 = 512 + 64 dims, up to 128 heads.
//
// Mathematics as in attention_paged.cu (an online softmax over 64-row tiles).  A CTA takes
// 64 heads (the MMA M) and one unit of the schedule (paged.cuh): a run of tiles that may span
// several sequences ("segments").  Per tile:
//   1. a loader group brings the 64 rows into its stage of a two-stage ring, in 128-byte
//      swizzle atoms: runs of pages as TMA boxes of gcd(page, 64) rows, other rows (selected
//      entries, partial tiles, pages that share no factor of 8 with 64) as 16-byte cp.async
//      with the absent rows zeroed (P = 0 there, and 0 * NaN must not reach the sums);
//   2. the MMA warp issues S = Q K^T (N = 64, 36 steps of K = 16) into TMEM;
//   3. eight softmax warps read S, agree on the running maximum and write P to shared memory
//      as two bf16 parts, P_hi = bf16(P) and P_lo = bf16(P - P_hi) (the second into the
//      tile's rotary atom, which only S reads): P is held to 2^-17, where bf16 alone would
//      add as much error as the rounding of the output;
//   4. O += P_hi V + P_lo V (N = 2 x 256, V read MN-major from the same tile).
// The MMAs are the weight-stationary form at M = 64: O (64 x 512) takes 128 lanes x 256 columns
// and S 128 lanes x 32 columns, so lane l and lane l + 64 hold halves of the same head.
// At a segment's end O is normalised and stored, or left as a partial for the merge.
// Every wait is bounded (CSA_DEVERR_TIMEOUT).
#include "paged.cuh"
#include "tc.cuh"

#include <cudaTypedefs.h>

namespace csa {

namespace {

constexpr int PT_ROWS = 64;              // rows per tile (N of QK^T, K of PV)
constexpr int PT_HC = 64;                // heads per CTA (MMA M)
constexpr int PT_ATOMS = 9;              // 576 dims = 9 atoms of 64 dims (128 bytes)
constexpr int PT_CHUNKS = PT_ATOMS * 8;  // 16-byte chunks per row
constexpr int PT_GROUP = 96;             // threads per loader group; group g fills stage g
constexpr int PT_SMW = 8;                // softmax warps: two warpgroups, one per half of a lane's columns
constexpr int PT_MMAW = 8;               // the MMA warp
constexpr int PT_QW = 9;                 // the query warp
constexpr int PT_LDW = 10;               // first loader warp
constexpr int PT_THREADS = PT_LDW * 32 + 2 * PT_GROUP;
constexpr int PT_MIN_TILES = 2;
constexpr float PT_RESCALE = 8.0f;       // base-2 units: O is rescaled once the maximum grows 256-fold
constexpr int ATOM = PT_ROWS * 128;      // one 64-row x 128-byte swizzle atom
constexpr uint32_t TM_O = 0, TM_S = 256, TM_COLS = 512;    // TMEM columns: O 256, S 2 x 32
static_assert(PT_THREADS == 512, "16 warps: 128 registers a thread");

struct PtSmem {
  uint8_t q[PT_ATOMS][PT_HC * 128];          // 72 KB
  uint8_t kv[2][PT_ATOMS][ATOM];             // 144 KB
  uint8_t p[PT_HC * 128];                    // P_hi: 64 heads x 64 rows bf16; between segments the row sums
  float smax[2][2][128];                     // per tile parity and warpgroup: the lanes' tile maxima
  int rowy[2][PT_ROWS];                      // per stage: rows of the pool or the window, -1 = none
  uint32_t vmask[2][2];                      // per stage: bit j of word j / 32 set when row j is valid
  uint64_t full[2], empty[2], sfull[2], sfree[2];
  uint64_t pfull, pdone, qfull, qfree, ofree, drain;
  uint64_t pairb[4], segb;                   // softmax warps: the two of the same heads; all eight
  uint32_t tmem_base;
  int abort_flag;
  int ld_stop[2];                            // per loader group: 1 + the step at which it stops (0 = running)
};
static_assert(sizeof(PtSmem) <= 232448, "shared memory of one CTA (227 KB)");

struct PtMaps {
  CUtensorMap q;       // [B * H rows, 576], box 64 x 64
  CUtensorMap pages;   // [n_pages * page rows, 576], box 64 dims x box rows
  CUtensorMap win;     // [B * W rows, 576], box 64 x 64
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {   // bytes < 16: zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}
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
// 2^x by the MUFU.EX2 unit (relative error about 2^-22)
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// byte offset of 16-byte chunk c of row j in a 128-byte-swizzled atom
__device__ __forceinline__ uint32_t sw128_off(int j, int c) { return (j >> 3) * 1024 + (j & 7) * 128 + ((c ^ (j & 7)) << 4); }

// The segments of a unit: tiles [t0, t1) of sequence b.  Every role walks them by itself.
struct SegIter {
  int next_b;
  int64_t next_t, left;
  int b, na, nw;
  int64_t ta, t0, t1;                        // ta: tiles of the entries; the window's follow
  bool whole;
  __device__ __forceinline__ void start(const PagedPlan& p, int unit) {
    next_b = p.b;
    next_t = (int64_t)unit * p.per - p.before;
    left = p.total - (int64_t)unit * p.per;
    if (left > p.per) left = p.per;
    t0 = t1 = 0;
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs& a) {
    while (left > 0) {
      b = next_b++;
      na = paged_rows_a(a, b);
      nw = paged_rows_w(a, b);
      ta = ((int64_t)na + PT_ROWS - 1) / PT_ROWS;
      const int64_t tiles = ta + (nw + PT_ROWS - 1) / PT_ROWS;
      t0 = next_t;
      next_t = 0;
      if (t0 >= tiles) continue;
      t1 = tiles < t0 + left ? tiles : t0 + left;
      left -= t1 - t0;
      whole = t0 == 0 && t1 == tiles;
      return true;
    }
    return false;
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
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.full[s], PT_GROUP);
      tc::mbar_init(&sm.empty[s], 1);
      tc::mbar_init(&sm.sfull[s], 1);
      tc::mbar_init(&sm.sfree[s], PT_SMW);
      sm.ld_stop[s] = 0;
    }
    tc::mbar_init(&sm.pfull, PT_SMW);
    tc::mbar_init(&sm.pdone, 1);
    tc::mbar_init(&sm.qfull, 1);
    tc::mbar_init(&sm.qfree, 1);
    tc::mbar_init(&sm.ofree, PT_SMW);
    tc::mbar_init(&sm.drain, 1);
    for (int s = 0; s < 4; ++s) tc::mbar_init(&sm.pairb[s], 2);
    tc::mbar_init(&sm.segb, PT_SMW);
    sm.abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == PT_MMAW) { tc::tmem_alloc(&sm.tmem_base, TM_COLS); tc::tmem_relinquish(); }
  tc::griddep_wait();                               // the setup overlaps the preceding kernel's tail
  tc::fence_before_sync();
  const PagedPlan plan = paged_plan(a, unit, PT_THREADS, reinterpret_cast<int64_t*>(sm.q));
  tc::fence_after_sync();
  tc::fence_proxy_async_smem();
  __syncthreads();                                  // the plan's scratch is read; Q may land there
  const uint32_t tmem = sm.tmem_base;
  SegIter seg;
  seg.start(plan, unit);

  if (warp >= PT_LDW) {
    // ------------------------------------------------------------------ loader group g (96 threads)
    const int g = (warp - PT_LDW) / (PT_GROUP / 32);
    const int lg = threadIdx.x - PT_LDW * 32 - g * PT_GROUP;
    // The group's next tile, resolved into registers before its stage is free: every other
    // tile of the unit, counted over all segments.
    int64_t t = 0;
    bool more = seg.next(a), in_a = true;
    if (more) t = seg.t0;
    int y = -1;
    auto step = [&](int n) {                          // n tiles on
      while (more && n > 0) {
        if (t + n < seg.t1) { t += n; n = 0; }
        else {
          n -= (int)(seg.t1 - t);
          more = seg.next(a);
          if (more) t = seg.t0;
        }
      }
    };
    auto resolve = [&]() {
      in_a = t < seg.ta;
      y = -1;
      if (lg < PT_ROWS) {
        const int64_t v = (in_a ? t : t - seg.ta) * PT_ROWS + lg;
        if (in_a) {
          if (v < seg.na) y = (int)paged_row(a, seg.b, (int)v);
        } else if (v < seg.nw) {
          y = seg.b * a.W + (int)v;
        }
      }
    };
    step(g);
    if (more) resolve();
    int issued = 0;                                   // tiles this group started (for the drain)
    for (int i = 0; more; ++i) {
      const bool go = tc::mbar_wait(&sm.empty[g], (i & 1) ^ 1) && !*(volatile int*)&sm.abort_flag;
      if (!go) sm.ld_stop[g] = i + 1;                 // the group leaves together at this step's barrier
      if (lg < PT_ROWS) {
        sm.rowy[g][lg] = y;
        const uint32_t vb = __ballot_sync(0xffffffffu, y >= 0);
        if ((lg & 31) == 0) sm.vmask[g][lg >> 5] = vb;
      }
      const bool a_tile = in_a;
      named_bar(1 + g, PT_GROUP);
      const int stop = *(volatile int*)&sm.ld_stop[g];
      if (stop != 0 && stop <= i + 1) break;
      const bool all = (sm.vmask[g][0] & sm.vmask[g][1]) == 0xffffffffu;
      const int rows = a_tile ? box : PT_ROWS;        // rows per TMA box; box 0: pages that no box fits
      const bool tma = all && (a_tile ? !SPARSE && box > 0 : true);
      if (tma) {
        if (lg < PT_ROWS / rows) {
          if (lg == 0) tc::mbar_arrive_expect_tx(&sm.full[g], PT_ATOMS * ATOM);
          const CUtensorMap* m = a_tile ? &maps.pages : &maps.win;
          const int y0 = sm.rowy[g][lg * rows];
          for (int at = 0; at < PT_ATOMS; ++at) tc::tma_load_2d(sm.kv[g][at] + lg * rows * 128, m, &sm.full[g], 64 * at, y0);
        }
        if (lg != 0) tc::mbar_arrive(&sm.full[g]);
      } else {
        const uint8_t* base = reinterpret_cast<const uint8_t*>(a_tile ? a.pages : a.win);
        const uint32_t kv0 = tc::smem_u32(sm.kv[g][0]);
        int j = lg >= PT_CHUNKS ? 1 : 0, c = lg - j * PT_CHUNKS;
        for (int p = 0; p < PT_ROWS * PT_CHUNKS / PT_GROUP; ++p) {
          const int yr = sm.rowy[g][j];
          cp_async16(kv0 + (c >> 3) * ATOM + sw128_off(j, c & 7), base + (size_t)(yr < 0 ? 0 : yr) * (576 * 2) + c * 16,
                     yr < 0 ? 0 : 16);
          c += PT_GROUP - PT_CHUNKS;
          j += 1;
          if (c >= PT_CHUNKS) { c -= PT_CHUNKS; j += 1; }
        }
      }
      ++issued;
      // resolve the group's next tile while the copies are in flight
      step(2);
      if (more) resolve();
      if (!tma) {
        cp_async_wait_all();
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&sm.full[g]);
      }
    }
    cp_async_wait_all();
    // drain: no TMA write of this CTA may be in flight when the CTA exits
    if (lg == 0 && issued > 0) tc::mbar_wait(&sm.full[g], (issued - 1) & 1);
  } else if (warp == PT_QW) {
    // ------------------------------------------------------------------ queries of each segment
    if (lane == 0) {
      tc::prefetch_tmap(&maps.q);
      tc::prefetch_tmap(&maps.pages);
      tc::prefetch_tmap(&maps.win);
      int n = 0;
      for (; seg.next(a); ++n) {
        // the segment before no longer reads Q: its last S is complete
        if (n > 0 && !(tc::mbar_wait(&sm.qfree, (n - 1) & 1) && !*(volatile int*)&sm.abort_flag)) break;
        tc::mbar_arrive_expect_tx(&sm.qfull, PT_ATOMS * PT_HC * 128);
        for (int at = 0; at < PT_ATOMS; ++at)
          tc::tma_load_2d(sm.q[at], &maps.q, &sm.qfull, 64 * at, seg.b * a.H + hh * PT_HC);
      }
      if (n > 0) tc::mbar_wait(&sm.qfull, (n - 1) & 1);
    }
    __syncwarp();
  } else if (warp == PT_MMAW) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop (descriptors stay warp-uniform); lane 0 decides, one
    // elected lane (always the same) issues every MMA and commit.
    constexpr uint32_t ID_S = tc::idesc(tc::FMT_BF16, tc::FMT_BF16, PT_HC, PT_ROWS);
    constexpr uint32_t ID_O = tc::idesc(tc::FMT_BF16, tc::FMT_BF16, PT_HC, 256, 0, 1);
    const uint64_t q_d0 = tc::desc_k_sw128(tc::smem_u32(sm.q[0]));
    const uint64_t k_d0 = tc::desc_k_sw128(tc::smem_u32(sm.kv[0][0])), k_d1 = tc::desc_k_sw128(tc::smem_u32(sm.kv[1][0]));
    const uint64_t p_d0 = tc::desc_k_sw128(tc::smem_u32(sm.p));
    const uint64_t pl_d0 = tc::desc_k_sw128(tc::smem_u32(sm.kv[0][PT_ATOMS - 1])),
                   pl_d1 = tc::desc_k_sw128(tc::smem_u32(sm.kv[1][PT_ATOMS - 1]));
    const uint64_t v_d0 = tc::desc_mn_sw128(tc::smem_u32(sm.kv[0][0]), ATOM, 1024),
                   v_d1 = tc::desc_mn_sw128(tc::smem_u32(sm.kv[1][0]), ATOM, 1024);
    // Event-driven: S(ns) once its tile has landed and its buffer is free (and, at a
    // segment's first tile, its queries); PV(np) once P(np) is ready (and, at a first tile,
    // the epilogue before has read O).  s_* and p_*: the walks of the two over the segments.
    int ns = 0, np = 0;
    SegIter ps = seg;
    int s_seg = 0, p_seg = 0;
    int64_t s_left = 0, p_left = 0;
    bool s_first = true, p_first = true;
    bool s_more = seg.next(a), p_more = ps.next(a);
    if (s_more) { s_left = seg.t1 - seg.t0; p_left = s_left; }
    uint64_t t_idle = tc::now_ns();
    uint32_t spins = 0;
    bool ok = true;
    while (ok && p_more) {
      bool prog = false;
      if (s_more) {
        const int st = ns & 1;
        const uint32_t ph = (ns >> 1) & 1;
        bool ready = false;
        if (lane == 0)
          ready = tc::mbar_try_wait(&sm.full[st], ph) && tc::mbar_try_wait(&sm.sfree[st], ph ^ 1) &&
                  (!s_first || tc::mbar_try_wait(&sm.qfull, s_seg & 1));
        if (__shfl_sync(0xffffffffu, (int)ready, 0)) {
          tc::fence_after_sync();
          const uint32_t d = tmem + TM_S + st * 32;
          const uint64_t kd = st ? k_d1 : k_d0;
          if (tc::elect_one()) tc::mma_f16_ws<false>(d, q_d0, kd, ID_S);
#pragma unroll
          for (int i = 1; i < PT_ATOMS * 4; ++i) {
            const uint64_t off = (uint64_t)(((i >> 2) * ATOM + (i & 3) * 32) >> 4);
            if (tc::elect_one()) tc::mma_f16_ws<true>(d, q_d0 + off, kd + off, ID_S);
          }
          s_first = false;
          const bool last = --s_left == 0;
          if (tc::elect_one()) {
            tc::mma_commit(&sm.sfull[st]);
            if (last) tc::mma_commit(&sm.qfree);
          }
          __syncwarp();
          ++ns;
          if (last) {
            s_more = seg.next(a);
            s_left = seg.t1 - seg.t0;
            s_first = true;
            ++s_seg;
          }
          prog = true;
        }
      }
      if (np < ns) {
        bool ready = false;
        if (lane == 0)
          ready = tc::mbar_try_wait(&sm.pfull, np & 1) && (!p_first || p_seg == 0 || tc::mbar_try_wait(&sm.ofree, (p_seg - 1) & 1));
        if (__shfl_sync(0xffffffffu, (int)ready, 0)) {
          const int st = np & 1;
          tc::fence_after_sync();
          const uint64_t vd = st ? v_d1 : v_d0;
          const uint64_t pl = st ? pl_d1 : pl_d0;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint64_t vh = vd + (uint64_t)((4 * half * ATOM) >> 4);
            const uint32_t d = tmem + TM_O + 128 * half;
            if (tc::elect_one()) {
              if (p_first) tc::mma_f16_ws<false>(d, p_d0, vh, ID_O);
              else tc::mma_f16_ws<true>(d, p_d0, vh, ID_O);
            }
#pragma unroll
            for (int ks = 1; ks < PT_ROWS / 16; ++ks)
              if (tc::elect_one()) tc::mma_f16_ws<true>(d, p_d0 + (uint64_t)((ks * 32) >> 4), vh + (uint64_t)((ks * 16 * 128) >> 4), ID_O);
#pragma unroll
            for (int ks = 0; ks < PT_ROWS / 16; ++ks)
              if (tc::elect_one()) tc::mma_f16_ws<true>(d, pl + (uint64_t)((ks * 32) >> 4), vh + (uint64_t)((ks * 16 * 128) >> 4), ID_O);
          }
          if (tc::elect_one()) {
            tc::mma_commit(&sm.empty[st]);
            tc::mma_commit(&sm.pdone);
          }
          __syncwarp();
          p_first = false;
          ++np;
          if (--p_left == 0) {
            p_more = ps.next(a);
            p_left = ps.t1 - ps.t0;
            p_first = true;
            ++p_seg;
          }
          prog = true;
        }
      }
      if (prog) {
        spins = 0;
      } else if ((++spins & 63u) == 0u) {
        bool stop = false;
        if (lane == 0) {
          const uint64_t now = tc::now_ns();
          if (spins == 64u) t_idle = now;
          stop = *(volatile int*)&sm.abort_flag || now - t_idle > tc::WAIT_LIMIT_NS;
        }
        if (__shfl_sync(0xffffffffu, (int)stop, 0)) ok = false;
      }
    }
    if (!ok && lane == 0) atomicExch(&sm.abort_flag, 1);
    // every MMA the elected lane issued has completed before the CTA frees TMEM
    if (tc::elect_one()) tc::mma_commit(&sm.drain);
    __syncwarp();
    tc::mbar_wait(&sm.drain, 0);
  } else {
    // ------------------------------------------------------------------ softmax + epilogue, warps 0-7
    // Thread (wg, lane tl): head tl % 64; of S the tile rows 32 * (tl / 64) .. + 31, of which
    // it exponentiates 16 (warpgroup wg's half); of O the dims 256 wg + 128 (tl / 64) .. + 127.
    const int wg = warp >> 2, quarter = warp & 3;
    const int tl = quarter * 32 + lane;
    const int hl = tl & 63, half = tl >> 6;
    const int h = hh * PT_HC + hl;
    const bool hv = h < a.H;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint64_t* pairb = &sm.pairb[wg * 2 + (quarter & 1)];
    // all softmax warps meet (a bounded wait, unlike a named barrier)
    uint32_t met = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.segb);
      return __all_sync(0xffffffffu, tc::mbar_wait(&sm.segb, met++ & 1));
    };
    // logits in the base-2 domain: P = 2^(s - m)
    const float scale2 = a.sm_scale * 1.4426950408889634f;
    bool ok = true;
    int i = 0;                                        // tiles so far, over all segments
    // sequences without a row (no unit has a tile of theirs)
    for (int b = unit; b < a.B; b += a.units) {
      if (paged_rows_a(a, b) != 0 || paged_rows_w(a, b) != 0 || !hv) continue;
      uint4* o = reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + ((size_t)b * a.H + h) * 512 + 256 * wg + 128 * half);
      for (int c = 0; c < 16; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse && tl < 64 && wg == 0) a.lse[(size_t)b * a.H + h] = a.sink[h];
    }
    __syncwarp();
    while (ok && seg.next(a)) {
      const float sink = hv ? a.sink[h] : 0.f;
      float m_run = -INFINITY, l_run = 0.f;           // running maximum; this thread's row sum
      for (int64_t t = seg.t0; t < seg.t1; ++t, ++i) {
        const int st = i & 1;
        const uint32_t ph = (i >> 1) & 1;
        bool w = tc::mbar_wait(&sm.sfull[st], ph) && tc::mbar_wait(&sm.full[st], ph);
        w = __all_sync(0xffffffffu, w && !*(volatile int*)&sm.abort_flag);
        if (!w) { ok = false; break; }
        tc::fence_after_sync();
        float s[32];
        {
          uint32_t v[32];
          tc::tmem_ld16(tmem + lane_base + TM_S + st * 32, v);
          tc::tmem_ld16(tmem + lane_base + TM_S + st * 32 + 16, v + 16);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(v[j]) * scale2;
        }
        tc::fence_before_sync();
        if (lane == 0) tc::mbar_arrive(&sm.sfree[st]);
        const uint32_t vm = sm.vmask[st][half];
        if (vm != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((vm >> j) & 1u)) s[j] = -INFINITY;
        }
        float mq[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < 32; ++j) mq[j & 3] = fmaxf(mq[j & 3], s[j]);
        float mt = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        // the other half of the head's rows
        sm.smax[st][wg][tl] = mt;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(pairb);
        if (!__all_sync(0xffffffffu, tc::mbar_wait(pairb, i & 1))) { ok = false; break; }
        mt = fmaxf(mt, sm.smax[st][wg][tl ^ 64]);
        // the running maximum is raised lazily, by all four threads of a head alike
        bool rescale = false;
        float alpha = 1.f;
        if (mt > m_run + PT_RESCALE || (m_run == -INFINITY && mt != -INFINITY)) {
          const float m_new = fmaxf(mt, m_run);
          alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new);
          rescale = m_run != -INFINITY;
          m_run = m_new;
        }
        const bool rescale_any = __any_sync(0xffffffffu, rescale);
        uint32_t w8[8], l8[8];
        float psum = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float s0 = wg ? s[16 + 2 * u] : s[2 * u], s1 = wg ? s[17 + 2 * u] : s[2 * u + 1];
          const float p0 = m_run == -INFINITY ? 0.f : ex2_approx(s0 - m_run);
          const float p1 = m_run == -INFINITY ? 0.f : ex2_approx(s1 - m_run);
          const __nv_bfloat162 hb = __floats2bfloat162_rn(p0, p1);
          const float h0 = __low2float(hb), h1 = __high2float(hb);
          const __nv_bfloat162 lb = __floats2bfloat162_rn(p0 - h0, p1 - h1);
          psum += (h0 + __low2float(lb)) + (h1 + __high2float(lb));    // the normaliser sums what the MMA sees
          w8[u] = *reinterpret_cast<const uint32_t*>(&hb);
          l8[u] = *reinterpret_cast<const uint32_t*>(&lb);
        }
        l_run = l_run * alpha + psum;
        if (i > 0) {                                  // the PV before owns P and O until it completes
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.pdone, (i - 1) & 1))) { ok = false; break; }
          tc::fence_after_sync();
        }
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
          // P_lo goes to the stage's rotary atom: S of this tile, its only reader, is complete
          const uint32_t pbase = tc::smem_u32(sm.p), lbase = tc::smem_u32(sm.kv[st][PT_ATOMS - 1]);
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
      float* blk = a.part + (size_t)(2 * unit + (seg.t0 == 0 ? 1 : 0)) * paged_part_block(a.H, 512);
      if (seg.whole) {
        M = fmaxf(sink, m);
        float e = 0.f;
        if (M != -INFINITY) {
          e = m == -INFINITY ? 0.f : __expf(m - M);
          den = __expf(sink - M) + l * e;
        }
        f = den > 0.f ? e / den : 0.f;
      }
      const int d0 = 256 * wg + 128 * half;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[64];
        tc::tmem_ld64(tmem + lane_base + TM_O + 128 * wg + c * 64, v);
        if (c == 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.ofree);
        }
        if (!hv) {
        } else if (seg.whole) {
          __nv_bfloat16* o = (__nv_bfloat16*)a.out + ((size_t)seg.b * a.H + h) * 512 + d0 + c * 64;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float f8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f8[j] = __uint_as_float(v[q * 8 + j]) * f;
            Elem<__nv_bfloat16>::st_vec(o + q * 8, f8);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q)
            *reinterpret_cast<uint4*>(blk + paged_part_val(a.H, h, d0 + c * 64 + 4 * q)) =
                make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        __syncwarp();
      }
      if (hv && wg == 0 && half == 0) {
        if (seg.whole) {
          if (a.lse) a.lse[(size_t)seg.b * a.H + h] = den > 0.f ? M + logf(den) : -INFINITY;
        } else {
          *reinterpret_cast<float2*>(blk + paged_part_rec(a.H, 512, h)) = make_float2(m, l);
        }
      }
    }
    if (!ok) atomicExch(&sm.abort_flag, 1);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (sm.abort_flag && threadIdx.x == 0) raise_err(a.err, CSA_DEVERR_TIMEOUT);
  if (warp == PT_MMAW) {
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
  a.units = paged_units_tc(a.B, a.H, paged_rows_max(a));
  a.tile = PT_ROWS;
  a.min_tiles = PT_MIN_TILES;
  // the largest of 64, 32, 16, 8 rows that divides the pages: every box lies in one page
  int box = PT_ROWS;
  while (box >= 8 && a.page % box != 0) box >>= 1;
  if (box < 8) box = 0;
  PtMaps maps;
  if (!row_map(&maps.q, a.q, (uint64_t)a.B * a.H, PT_HC)) return cudaErrorUnknown;
  if (!row_map(&maps.pages, a.pages, (uint64_t)a.n_pages * a.page, box ? box : 8)) return cudaErrorUnknown;
  if (a.W > 0) {
    if (!row_map(&maps.win, a.win, (uint64_t)a.B * a.W, PT_ROWS)) return cudaErrorUnknown;
  } else {
    maps.win = maps.pages;                           // no tile is ever a window tile
  }
  auto kern = a.idx ? paged_attn_tc_kernel<true> : paged_attn_tc_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PtSmem));
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
