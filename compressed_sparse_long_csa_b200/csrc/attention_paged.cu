// Attention of one new token per sequence over a paged latent cache, CUDA-core path, and
// the merge of split sequences.
//
// For head h of sequence b, over its rows (all entries, or the selected ones, and the
// window rows):  l_r = s <q_h, row_r>,  out_h = sum_r e^{l_r - M} row_r[0:dv] / den,
// den = e^{sink_h - M} + sum_r e^{l_r - M}, M = max(sink_h, max_r l_r), lse_h = M + log den.
// The same attention as sparse_attn_decode / hca_attn_decode ("Техотчёт DeepSeek-V4
// (2026): миллион токенов контекста", section "Гибридное внимание: CSA и HCA", CSA step 3
// and the HCA paragraph; sink, window and latent of "Технический отчёт DeepSeek-V4 —
// часть 1/2"); the page table is the addition.
//
// This path takes every shape and both storage types in fp32 arithmetic.
#include "paged.cuh"

namespace csa {

namespace {

constexpr int PC_ROWS = 32;      // rows per tile: one lane per row in the logits
constexpr int PC_WARPS = 8;
constexpr int PC_HEADS = 8;      // heads per CTA
constexpr int PC_MIN_TILES = 1;  // (2: five sequences of up to 3001 rows of 64 dims 11.2 -> 13.6 us)
constexpr int PC_SMEM = 96 * 1024;     // two CTAs per SM

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool zero) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(zero ? 0 : 16) : "memory");
}

template <typename T> __device__ __forceinline__ void load4(const T* p, float* x);
template <> __device__ __forceinline__ void load4<float>(const float* p, float* x) { Elem<float>::ld_vec(p, x); }
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// grid (units, ceil(H / 8)); shared memory: `bufs` (1 or 2) tiles of 32 rows as stored, each row
// 16 bytes longer than it need be (lanes' loads spread over the banks), and the CTA's queries in fp32.  A tile is copied by 16-byte
// cp.async while the one before is worked on (two buffers); its rows are looked up a tile earlier.
// A warp takes HB heads and 32 / G rows of every tile (8 warps: G = 8 for up to 4 heads, 4 for 8),
// so that each value read from shared memory meets HB heads.
// Logits: G lanes share a row's dot products, which they exchange so that each ends with one row
// and head.  Values: lane i owns dims 4i .. 4i+3 (+128 j) of all HB heads; narrow rows leave lanes
// for other rows.  Each warp has its own maximum and sums; the G warps of a head meet where the
// unit leaves the sequence.
// Bound: latency for few rows (5.7 us for one tile: schedule 1.3, lookups and rows 2, its work 1,
// the warps' meeting and the store 1.4), issue slots and shared memory for many (48 x 4000 rows of 64
// dims in fp32: 4 heads 31 us, 16 heads 50; with a head per warp, 57 and 144).
template <typename T, int NO, int HB>
__global__ void __launch_bounds__(PC_WARPS * 32, 2)
paged_attn_cc_kernel(PagedAttnArgs a, int bufs, int log_g) {
  extern __shared__ uint4 smem16[];
  __shared__ int64_t scratch[66];
  __shared__ int rows_s[4][PC_ROWS];                  // rows of the tiles, by tile mod 4
  constexpr int VEC = Elem<T>::VEC;
  const int unit = blockIdx.x, hg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int dk = a.dk, dv = a.dv, pitch = dk + VEC, vecs = dk / VEC;
  T* const tiles_s = reinterpret_cast<T*>(smem16);
  float* const Qs = reinterpret_cast<float*>(tiles_s + (size_t)bufs * PC_ROWS * pitch);
  const int heads = min(a.H - hg * PC_HEADS, HB * (PC_WARPS >> log_g));
  const int hw = (warp >> log_g) * HB;                // the warp's first head, of the CTA's
  const bool live = hw < heads;
  const int log_r = 5 - log_g, r0 = (warp & ((1 << log_g) - 1)) << log_r;
  const int krow = r0 + (lane & ((1 << log_r) - 1)), kpart = lane >> log_r;
  // the lane whose logit is head u's of the warp's first row
  auto lane_of = [](int u) { return HB == 4 ? u << 3 : 0; };
  // lanes that copy a row, and (NO = 1) lanes that share a row's values; what is left of the warp takes other rows
  const int log_l = vecs <= 4 ? 2 : vecs <= 8 ? 3 : vecs <= 16 ? 4 : 5;
  const int log_v = NO > 1 || dv > 64 ? 5 : dv > 32 ? 4 : 3;
  const int vrow = lane >> log_v, vdim = 4 * (lane & ((1 << log_v) - 1));
  int voff[NO];                                       // (dims past the last: read, not stored)
#pragma unroll
  for (int i = 0; i < NO; ++i) voff[i] = vdim + 128 * i < dv ? vdim + 128 * i : 0;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // the merge waits for this grid itself
  const PagedPlan plan = paged_plan(a, unit, PC_WARPS * 32, scratch);
  // The last six warps clear the sequences without a row (no unit has a tile of theirs; a lane looks
  // at each) and write the unit's note, while the first two look up the rows of the first tiles.
  if (warp >= 2)
    for (int b0 = unit; b0 < a.B; b0 += 32 * a.units) {
      const int64_t bl = (int64_t)b0 + (int64_t)lane * a.units;
      for (unsigned none = __ballot_sync(0xffffffffu, bl < a.B && paged_tiles(a, (int)min(bl, (int64_t)a.B - 1)) == 0); none; none &= none - 1) {
        const int b = b0 + (__ffs(none) - 1) * a.units;
        for (int h = hg * PC_HEADS + warp - 2; h < min(a.H, (hg + 1) * PC_HEADS); h += PC_WARPS - 2) {
          for (int c = lane; c < dv; c += 32) Elem<T>::st((T*)a.out + ((size_t)b * a.H + h) * dv + c, 0.f);
          if (a.lse && lane == 0) a.lse[(size_t)b * a.H + h] = a.sink[h];
        }
      }
    }
  if (hg == 0 && threadIdx.x == (PC_WARPS - 1) * 32) paged_note(a, plan, unit);
  PagedSeg seg;
  seg.start(plan, unit);
  while (seg.next(a)) {
    const int b = seg.b, na = seg.na, nw = seg.nw;
    const int64_t ta = seg.ta, t1 = seg.t1;
    int64_t t = seg.t0;
    // one warp looks up a tile's rows: in the pool or the window, -1 = none
    auto resolve = [&](int64_t tile) {
      if (tile >= t1 || warp != ((int)(tile - seg.t0) & (PC_WARPS - 1))) return;
      const bool in_a = tile < ta;
      const int v = (int)((in_a ? tile : tile - ta) * PC_ROWS) + lane;
      rows_s[tile & 3][lane] = in_a ? (v < na ? (int)paged_row(a, b, v) : -1) : (v < nw ? b * a.W + v : -1);
    };
    auto copy = [&](int64_t tile, int buf) {
      if (tile >= t1) return;
      const T* base = tile < ta ? (const T*)a.pages : (const T*)a.win;
      T* dst = tiles_s + (size_t)buf * PC_ROWS * pitch;
      for (int r = warp * (32 >> log_l) + (lane >> log_l); r < PC_ROWS; r += PC_WARPS * (32 >> log_l)) {
        const int y = rows_s[tile & 3][r];
        const T* src = base + (size_t)(y < 0 ? 0 : y) * dk;
        for (int c = lane & ((1 << log_l) - 1); c < vecs; c += 1 << log_l)
          cp_async16_zfill(dst + r * pitch + c * VEC, src + c * VEC, y < 0);
      }
    };
    resolve(t);
    resolve(t + 1);
    __syncthreads();
    copy(t, 0);
    // the queries (heads past the last: zeros), while the first rows are on their way
    const T* qb = (const T*)a.q + ((size_t)b * a.H + hg * PC_HEADS) * dk;
    for (int c = threadIdx.x * VEC; c < HB * (PC_WARPS >> log_g) * dk; c += PC_WARPS * 32 * VEC) {
      float x[VEC];
#pragma unroll
      for (int u = 0; u < VEC; ++u) x[u] = 0.f;
      if (c < heads * dk) Elem<T>::ld_vec(qb + c, x);
#pragma unroll
      for (int u = 0; u < VEC; u += 4) *reinterpret_cast<float4*>(Qs + c + u) = make_float4(x[u], x[u + 1], x[u + 2], x[u + 3]);
    }
    float4 o[HB][NO];
#pragma unroll
    for (int u = 0; u < HB; ++u)
#pragma unroll
      for (int i = 0; i < NO; ++i) o[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m_run = -INFINITY, l_run = 0.f;             // of the lane's head; the sum of the lane's rows
    int buf = 0;
    for (; t < t1; ++t) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();                                // the tile is there, and the one before is read
      if (bufs == 2) copy(t + 1, buf ^ 1);
      resolve(t + 2);
      const T* Ks = tiles_s + (size_t)buf * PC_ROWS * pitch;
      if (live) {
        float s[HB][2];
#pragma unroll
        for (int u = 0; u < HB; ++u) s[u][0] = s[u][1] = 0.f;
        const T* kr = Ks + krow * pitch;
        const float* qh = Qs + hw * dk;
#pragma unroll 2
        for (int c = kpart * VEC; c < dk; c += VEC << log_g) {
          float x[VEC];
          Elem<T>::ld_vec(kr + c, x);
#pragma unroll
          for (int u = 0; u < HB; ++u)
#pragma unroll
            for (int v = 0; v < VEC; v += 4) {
              const float4 y = *reinterpret_cast<const float4*>(qh + u * dk + c + v);
              s[u][0] = fmaf(x[v], y.x, s[u][0]);
              s[u][1] = fmaf(x[v + 1], y.y, s[u][1]);
              s[u][0] = fmaf(x[v + 2], y.z, s[u][0]);
              s[u][1] = fmaf(x[v + 3], y.w, s[u][1]);
            }
        }
        float dot;
        if constexpr (HB == 4) {
          float d[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) d[u] = s[u][0] + s[u][1];
          const bool up = lane & 16, odd = lane & 8;  // these lanes go on with heads 2 and 3; with the odd one
          const float e0 = (up ? d[2] : d[0]) + __shfl_xor_sync(0xffffffffu, up ? d[0] : d[2], 16);
          const float e1 = (up ? d[3] : d[1]) + __shfl_xor_sync(0xffffffffu, up ? d[1] : d[3], 16);
          dot = (odd ? e1 : e0) + __shfl_xor_sync(0xffffffffu, odd ? e0 : e1, 8);
          if (log_r == 2) dot += __shfl_xor_sync(0xffffffffu, dot, 4);
        } else {
          dot = s[0][0] + s[0][1];
          for (int w = 1 << log_r; w < 32; w <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
        }
        const float logit = rows_s[t & 3][krow] >= 0 ? dot * a.sm_scale : -INFINITY;
        float m_new = fmaxf(m_run, logit);
        for (int w = 1; w < 1 << log_r; w <<= 1) m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, w));
        const float m0 = m_new == -INFINITY ? 0.f : m_new;   // no row so far: p = 0 (a NaN stays one)
        const float p = __expf(logit - m0);
        if (__any_sync(0xffffffffu, m_new > m_run)) {
          const float alpha = __expf(m_run - m0);
          l_run *= alpha;
          m_run = m_new;
#pragma unroll
          for (int u = 0; u < HB; ++u) {
            const float au = __shfl_sync(0xffffffffu, alpha, lane_of(u));
#pragma unroll
            for (int i = 0; i < NO; ++i) { o[u][i].x *= au; o[u][i].y *= au; o[u][i].z *= au; o[u][i].w *= au; }
          }
        }
        l_run += p;
#pragma unroll 2
        for (int k = vrow; k < 1 << log_r; k += 32 >> log_v) {            // whole warps
          float pr[HB];
#pragma unroll
          for (int u = 0; u < HB; ++u) pr[u] = __shfl_sync(0xffffffffu, p, lane_of(u) + k);
          const T* vr = Ks + (r0 + k) * pitch;
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            float x[4];
            load4<T>(vr + voff[i], x);
#pragma unroll
            for (int u = 0; u < HB; ++u) {
              o[u][i].x = fmaf(pr[u], x[0], o[u][i].x);
              o[u][i].y = fmaf(pr[u], x[1], o[u][i].y);
              o[u][i].z = fmaf(pr[u], x[2], o[u][i].z);
              o[u][i].w = fmaf(pr[u], x[3], o[u][i].w);
            }
          }
        }
      }
      if (bufs == 2) {
        buf ^= 1;
      } else {
        __syncthreads();
        copy(t + 1, 0);
      }
    }
    __syncthreads();                                  // all tiles are read
    // the G warps of a head meet in the tiles' memory: per warp and head {m, l, -, -, o}
    float* const left = reinterpret_cast<float*>(smem16);
    if (live) {
      float* const mine = left + (size_t)warp * HB * (dv + 4);
      for (int w = 1; w < 1 << log_r; w <<= 1) l_run += __shfl_xor_sync(0xffffffffu, l_run, w);
#pragma unroll
      for (int u = 0; u < HB; ++u) {
        if (NO == 1)                                  // the lanes of other rows
          for (int w = 1 << log_v; w < 32; w <<= 1) {
            o[u][0].x += __shfl_xor_sync(0xffffffffu, o[u][0].x, w);
            o[u][0].y += __shfl_xor_sync(0xffffffffu, o[u][0].y, w);
            o[u][0].z += __shfl_xor_sync(0xffffffffu, o[u][0].z, w);
            o[u][0].w += __shfl_xor_sync(0xffffffffu, o[u][0].w, w);
          }
        if (lane == lane_of(u)) *reinterpret_cast<float2*>(mine + u * (dv + 4)) = make_float2(m_run, l_run);
#pragma unroll
        for (int i = 0; i < NO; ++i)
          if (vdim + 128 * i < dv && vrow == 0) *reinterpret_cast<float4*>(mine + u * (dv + 4) + 4 + vdim + 128 * i) = o[u][i];
      }
    }
    __syncthreads();
    const int pieces = dv / 4;
    for (int i = threadIdx.x; i < heads * pieces; i += PC_WARPS * 32) {
      const int hh = i / pieces, c = 4 * (i - hh * pieces), h = hg * PC_HEADS + hh;
      const float* src = left + (size_t)(((hh / HB) << log_g) * HB + hh % HB) * (dv + 4);
      const size_t step = (size_t)HB * (dv + 4);
      float M = -INFINITY;
#pragma unroll 1
      for (int g = 0; g < 1 << log_g; ++g) M = fmaxf(M, src[g * step]);
      const float m0 = M == -INFINITY ? 0.f : M;
      float l = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int g = 0; g < 1 << log_g; ++g) {
        const float2 ml = *reinterpret_cast<const float2*>(src + g * step);
        const float4 x = *reinterpret_cast<const float4*>(src + g * step + 4 + c);
        const float w = __expf(ml.x - m0);
        l = fmaf(w, ml.y, l);
        y = make_float4(fmaf(w, x.x, y.x), fmaf(w, x.y, y.y), fmaf(w, x.z, y.z), fmaf(w, x.w, y.w));
      }
      if (seg.whole) {
        const float sk = a.sink[h], top = fmaxf(sk, M);
        const float f = M == -INFINITY ? 0.f : __expf(M - top), den = paged_sink(sk, top) + l * f;
        const float inv = den == 0.f ? 0.f : f / den;
        T* dst = (T*)a.out + ((size_t)b * a.H + h) * dv + c;
        Elem<T>::st(dst, y.x * inv);
        Elem<T>::st(dst + 1, y.y * inv);
        Elem<T>::st(dst + 2, y.z * inv);
        Elem<T>::st(dst + 3, y.w * inv);
        if (a.lse && c == 0) a.lse[(size_t)b * a.H + h] = den == 0.f ? -INFINITY : top + logf(den);
      } else {
        float* blk = a.part + (size_t)seg.slot(unit) * paged_part_block(a.H, dv);
        *reinterpret_cast<float4*>(blk + paged_part_val(a.H, h, c)) = y;
        if (c == 0) {
          *reinterpret_cast<float2*>(blk + paged_part_rec(a.H, dv, h)) = make_float2(M, l);
        }
      }
    }
    __syncthreads();                                  // the next segment's tiles may land
  }
}

// Joins the pieces of cut sequences: out = sum_p e^{m_p - M} o_p / (e^{sink - M} +
// sum_p e^{m_p - M} l_p).  The units noted which sequences they began and did not finish;
// every CTA gathers those notes and takes its share of the items (sequence, eight heads,
// slice of the dims), the slices as narrow as it takes to give every CTA an item.  Eight
// heads' 16-byte pieces of a partial are one 128-byte line.  Where a slice leaves threads
// over, they share its partials.  All sums run in a fixed order, so a result does not depend
// on the order in which the units ended.  Bound: latency (the notes, the records, the partials:
// three round trips and the launch, 4 to 6 us behind the attention) and the L2, 4 H (dv + 4)
// bytes per piece.  Sequences of few partials are a warp's work, so that many of them run at
// once (32 ragged sequences 102.7 us without, 98.5 with; sparse, 48 sequences 55.6 against 51.5).
constexpr int PM_THREADS = 256, PM_H = 8, PM_C = PM_THREADS / PM_H, PM_SLICES = 16;
constexpr int PM_EARLY = 5;      // partials on their way at once (9: two sequences of 131 072 rows, 64 heads 71.3 -> 71.9 us)
constexpr int PM_PER_SM = 2;     // (1: 32 ragged sequences 98.5 -> 103.2 us)
constexpr int PM_FEW = 8;        // partials that one warp joins by itself (4: 32 ragged sequences 98.9 -> 100.4 us)
constexpr int PM_ROUNDS = 2;     // notes of a thread: up to 512 units
// Shared memory per unit (under the 48 KB of a plain launch for the 296 units that fp32 may have)
constexpr size_t PM_UNIT_BYTES = PM_H * sizeof(float2) + sizeof(int4);
// acc += w times a 16-byte piece of a partial
__device__ __forceinline__ void merge_add(float4& acc, const float4& v, float w) {
  acc = make_float4(fmaf(w, v.x, acc.x), fmaf(w, v.y, acc.y), fmaf(w, v.z, acc.z), fmaf(w, v.w, acc.w));
}
__device__ __forceinline__ void merge_store(float* dst, const float4& v) { *reinterpret_cast<float4*>(dst) = v; }
__device__ __forceinline__ void merge_store(__nv_bfloat16* dst, const float4& v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <typename T>
__global__ void __launch_bounds__(PM_THREADS, PM_PER_SM)
paged_merge_kernel(PagedAttnArgs a) {
  // per unit: the list {unit, sequence, partials, -}; per partial and head: {m, l}, then {e^{m - M}, l}
  extern __shared__ int4 list[];
  float2* const wts = reinterpret_cast<float2*>(list + a.units);
  __shared__ float red[2][PM_THREADS / 32][PM_H];
  __shared__ float4 sums[PM_THREADS];
  __shared__ int counts[PM_ROUNDS * PM_THREADS / 32];
  const int dv = a.dv, H = a.H;
  const int hl = threadIdx.x & (PM_H - 1), j = threadIdx.x / PM_H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the list: sequences of few partials from the front, the others from the back; the same in every CTA
  int few[PM_ROUNDS], many[PM_ROUNDS];               // of the lanes below this one
  int2 note[PM_ROUNDS];
#pragma unroll
  for (int r = 0; r < PM_ROUNDS; ++r) {
    const int u = r * PM_THREADS + threadIdx.x;
    note[r] = u < a.units ? __ldcg(&paged_notes(a)[u]) : make_int2(-1, 0);
  }
#pragma unroll
  for (int r = 0; r < PM_ROUNDS; ++r) {
    const unsigned f = __ballot_sync(0xffffffffu, note[r].y > 0 && note[r].y <= PM_FEW), m = __ballot_sync(0xffffffffu, note[r].y > PM_FEW);
    few[r] = __popc(f & ((1u << lane) - 1u));
    many[r] = __popc(m & ((1u << lane) - 1u));
    if (lane == 0) counts[r * (PM_THREADS / 32) + warp] = __popc(f) | __popc(m) << 16;
  }
  __syncthreads();
  int all = 0;                                        // few in the low half, many in the high one
#pragma unroll
  for (int r = 0; r < PM_ROUNDS; ++r) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < PM_THREADS / 32; ++w) {
      if (w == warp) before = all;
      all += counts[r * (PM_THREADS / 32) + w];
    }
    if (note[r].y > 0)
      list[note[r].y <= PM_FEW ? (before & 0xffff) + few[r] : a.units - 1 - (before >> 16) - many[r]] =
          make_int4(r * PM_THREADS + threadIdx.x, note[r].x, note[r].y, 0);
  }
  __syncthreads();
  const int n_few = all & 0xffff, count = all >> 16;
  const int hb = (H + PM_H - 1) / PM_H, pieces = dv / 4;    // 16-byte pieces of a head's o
  int slices = 1;
  while (slices < PM_SLICES && 2 * count * hb * slices <= (int)gridDim.x && pieces / slices > 4) slices <<= 1;
  const int width = (pieces + slices - 1) / slices;   // 16-byte pieces of a slice
  const size_t block = paged_part_block(H, dv);
  {
    // Few partials: a warp takes eight heads and 8 pieces of the dims.  Lane (head, q): partials q and
    // q + 4 in the weights, pieces q and q + 4 in the sums; all loads are one round trip.
    const int q = lane >> 3, wide = (pieces + 7) / 8;
    for (int item = blockIdx.x * (PM_THREADS / 32) + warp; item < n_few * hb * wide; item += gridDim.x * (PM_THREADS / 32)) {
      const int cg = item % wide, blk8 = item / wide % hb;
      const int4 cut = list[item / (wide * hb)];
      const int b = cut.y, n = cut.z, h = blk8 * PM_H + hl;
      const bool hv = h < H;
      const int hc = hv ? h : H - 1;
      const float* part = a.part + (size_t)(2 * cut.x) * block;
      auto partial = [&](int p) { return part + (p ? 2 * p * block : block); };
      float4 x[2][4];                                 // four partials' pieces; the first four's are on their way
      auto load = [&](int p0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = cg * 8 + 4 * k + q;
            if (p0 + u < n && c < pieces) x[k][u] = __ldcg(reinterpret_cast<const float4*>(partial(p0 + u)) + (size_t)c * H + hc);
          }
        }
      };
      load(0);
      const size_t rec = paged_part_rec(H, dv, hc);
      const float sk = a.sink[hc];
      float m[2], l[2], w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int p = q + 4 * k;
        m[k] = -INFINITY;
        l[k] = 0.f;
        if (p < n) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(partial(p) + rec));
          m[k] = ml.x;
          l[k] = ml.y;
        }
      }
      float M = fmaxf(m[0], m[1]);
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
      M = fmaxf(fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16)), sk);
      float den = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float e = m[k] == -INFINITY ? 0.f : __expf(m[k] - M);
        den += e * l[k];
        w[k] = e;
      }
      den += __shfl_xor_sync(0xffffffffu, den, 8);
      den += __shfl_xor_sync(0xffffffffu, den, 16);
      den += paged_sink(sk, M);
      const float inv = den == 0.f ? 0.f : 1.f / den;
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
      for (int p0 = 0; p0 < n; p0 += 4) {
        if (p0) load(p0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (p0 + u < n) {
            const float wu = __shfl_sync(0xffffffffu, p0 ? w[1] : w[0], hl + 8 * u) * inv;
#pragma unroll
            for (int k = 0; k < 2; ++k) merge_add(acc[k], x[k][u], wu);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = cg * 8 + 4 * k + q;
        if (hv && c < pieces) merge_store((T*)a.out + ((size_t)b * H + h) * dv + 4 * c, acc[k]);
      }
      if (a.lse && cg == 0 && q == 0 && hv) a.lse[(size_t)b * H + h] = den == 0.f ? -INFINITY : M + logf(den);
    }
  }
  int gw = PM_C;                                      // threads along a slice; the other PM_C / gw share its partials
  while (gw > 4 && gw / 2 >= width) gw >>= 1;
  const int groups = PM_C / gw, g = j / gw, jc = j - g * gw;
  for (int item = blockIdx.x; item < count * hb * slices; item += gridDim.x) {
    const int sl = item % slices, blk8 = item / slices % hb;
    const int4 cut = list[a.units - 1 - item / (slices * hb)];
    const int b = cut.y, n = cut.z, h = blk8 * PM_H + hl;
    const bool hv = h < H;
    const int hc = hv ? h : H - 1;
    // partial 0 lies in slot 1 of the unit, partial p > 0 in slot 0 of unit + p
    const float* part = a.part + (size_t)(2 * cut.x) * block;
    auto partial = [&](int p) { return part + (p ? 2 * p * block : block); };
    auto load = [&](int p, int c) { return __ldcg(reinterpret_cast<const float4*>(partial(p)) + (size_t)c * H + hc); };
    const size_t rec = paged_part_rec(H, dv, hc);
    const float sk = a.sink[hc];
    const int cend = min(pieces, (sl + 1) * width);
    const int c0 = sl * width + jc;
    float M = sk;
    for (int p0 = j; p0 < n; p0 += 4 * PM_C) {        // four records' loads at a time
      float2 r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p0 + u * PM_C < n) r[u] = __ldcg(reinterpret_cast<const float2*>(partial(p0 + u * PM_C) + rec));
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p0 + u * PM_C < n) {
          wts[(p0 + u * PM_C) * PM_H + hl] = r[u];
          M = fmaxf(M, r[u].x);
        }
    }
#pragma unroll
    for (int o = PM_H; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane < PM_H) red[0][warp][lane] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < PM_THREADS / 32; ++w) M = fmaxf(M, red[0][w][hl]);
    float den = 0.f;
    for (int p = j; p < n; p += PM_C) {
      const float2 r = wts[p * PM_H + hl];            // this thread's own
      const float w = r.x == -INFINITY ? 0.f : __expf(r.x - M);
      den += w * r.y;
      wts[p * PM_H + hl].x = w;
    }
#pragma unroll
    for (int o = PM_H; o < 32; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < PM_H) red[1][warp][lane] = den;
    __syncthreads();
    den = paged_sink(sk, M);
#pragma unroll
    for (int w = 0; w < PM_THREADS / 32; ++w) den += red[1][w][hl];
    const float inv = den == 0.f ? 0.f : 1.f / den;
    for (int c = c0; c - jc < cend; c += gw) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < cend) {
#pragma unroll 1
        for (int p0 = g; p0 < n; p0 += PM_EARLY * groups) {
          float4 x[PM_EARLY];
#pragma unroll
          for (int u = 0; u < PM_EARLY; ++u)
            if (p0 + u * groups < n) x[u] = load(p0 + u * groups, c);
#pragma unroll
          for (int u = 0; u < PM_EARLY; ++u)
            if (p0 + u * groups < n) merge_add(acc, x[u], wts[(p0 + u * groups) * PM_H + hl].x);
        }
      }
      if (groups > 1) {                               // (the slice is one round of its threads)
        sums[threadIdx.x] = acc;
        __syncthreads();
        for (int o = 1; g == 0 && o < groups; ++o) merge_add(acc, sums[threadIdx.x + o * gw * PM_H], 1.f);
      }
      if (g == 0 && c < cend && hv)
        merge_store((T*)a.out + ((size_t)b * H + h) * dv + 4 * c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
    if (a.lse && j == 0 && sl == 0 && hv) a.lse[(size_t)b * H + h] = den == 0.f ? -INFINITY : M + logf(den);
    __syncthreads();                                  // the weights and sums are read
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedAttnArgs& a, int dtype, cudaStream_t st) {
  if (a.units > PM_ROUNDS * PM_THREADS) return cudaErrorInvalidConfiguration;
  if (a.units == 1) return cudaSuccess;                // nothing is ever cut
  const int64_t most = (int64_t)(a.units - 1) * ((a.H + PM_H - 1) / PM_H) * PM_SLICES;
  const int grid = PM_PER_SM * num_sms();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < grid ? most : grid));
  cfg.blockDim = dim3(PM_THREADS);
  cfg.dynamicSmemBytes = (size_t)a.units * PM_UNIT_BYTES;            // a sequence has at most `units` partials
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits for the pieces first of all
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return dtype == CSA_BF16 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<__nv_bfloat16>, a)
                           : cudaLaunchKernelEx(&cfg, paged_merge_kernel<float>, a);
}

// Two CTAs per SM over the head groups.
int paged_units_cc(int B, int H, int64_t rows_max) {
  const int groups = (H + PC_HEADS - 1) / PC_HEADS;
  return paged_units(2 * num_sms() / groups, B, rows_max, PC_ROWS, PC_MIN_TILES);
}

cudaError_t launch_paged_attn_cc(PagedAttnArgs a, int dtype, cudaStream_t st) {
  a.tile_log2 = 5;
  static_assert(PC_ROWS == 1 << 5, "tile rows");
  a.min_tiles = PC_MIN_TILES;
  a.begin_cost = 0;
  a.units = paged_units(a, paged_units_cc(a.B, a.H, paged_rows_max(a)));
  // Heads of a warp: 4 share each value read; 1 where that would leave warps' lanes to heads that are
  // not there (48 x 4000 rows of 64 dims in fp32: one head 28.5 us against 31.2 the other way, two
  // heads 28.8 against 31.1)
  const int hb = a.H <= 2 ? 1 : 4;
  int log_g = 3;                                      // warps of a head: the 8 over the CTA's heads
  while (log_g > 0 && (hb << (3 - log_g)) < (a.H < PC_HEADS ? a.H : PC_HEADS)) --log_g;
  auto go = [&](auto tag) {
    using T = decltype(tag);
    const size_t tile = (size_t)PC_ROWS * (a.dk + Elem<T>::VEC) * sizeof(T), qs = (size_t)PC_HEADS * a.dk * sizeof(float);
    // One buffer holds the warps' results in fp32 where the warps of all heads meet; in bf16 it takes
    // two, and two always fit.  (One for fp32 too: the sequences above 11.2 -> 11.5 us.)
    const int bufs = 2 * tile + qs <= PC_SMEM ? 2 : 1;
    const dim3 grid(a.units, (a.H + PC_HEADS - 1) / PC_HEADS);
    const int no = a.dv <= 128 ? 0 : a.dv <= 512 ? 1 : 2, at = hb == 1 ? no : 3 + no;
    void (*const kerns[])(PagedAttnArgs, int, int) = {paged_attn_cc_kernel<T, 1, 1>, paged_attn_cc_kernel<T, 4, 1>, paged_attn_cc_kernel<T, 5, 1>,
                                                      paged_attn_cc_kernel<T, 1, 4>, paged_attn_cc_kernel<T, 4, 4>, paged_attn_cc_kernel<T, 5, 4>};
    static std::atomic<uint64_t> ready[6];
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kerns[at]), ready[at], PC_SMEM);
    if (e != cudaSuccess) return e;
    note_launch();
    kerns[at]<<<grid, PC_WARPS * 32, bufs * tile + qs, st>>>(a, bufs, log_g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_paged_merge(a, dtype, st);
  };
  return dtype == CSA_BF16 ? go(__nv_bfloat16()) : go(float());
}

}  // namespace csa
