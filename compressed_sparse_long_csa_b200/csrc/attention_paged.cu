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

#include <cuda_fp16.h>

namespace csa {

namespace {

constexpr int PC_ROWS = 32;      // rows per tile: one lane per row in the logits
constexpr int PC_WARPS = 8;      // heads per CTA: one warp each
constexpr int PC_MAXD = 576;
constexpr int PC_MIN_TILES = 1;

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
// 16 bytes apart from the next, and the warps' queries in fp32.  Lane r of every warp knows row r
// of a tile; a tile is copied by 16-byte cp.async while the one before is worked on (two buffers)
// and its rows are looked up a tile earlier still.
// Logits: lane r of a head's warp forms the whole dot product of row r (no reduction across
// lanes); the pitch spreads the lanes' 16-byte loads over the banks.  Values: lane i owns dims
// 4i .. 4i+3 (+128 j).
// Bound: latency for few rows (about 5 us: lengths, table, rows, one tile's work, the store), the
// fp32 pipe and shared memory (two 16-byte loads for 4 or 8 products) for many.
template <typename T>
__global__ void __launch_bounds__(PC_WARPS * 32)
paged_attn_cc_kernel(PagedAttnArgs a, int bufs) {
  extern __shared__ uint4 smem16[];
  __shared__ int64_t scratch[66];
  constexpr int VEC = Elem<T>::VEC;
  const int unit = blockIdx.x, hg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
  const int dk = a.dk, dv = a.dv, pitch = dk + VEC, vecs = dk / VEC;
  T* const tiles_s = reinterpret_cast<T*>(smem16);
  float* const Qs = reinterpret_cast<float*>(tiles_s + (size_t)bufs * PC_ROWS * pitch) + (size_t)warp * dk;
  const int h = hg * PC_WARPS + warp;
  const bool hv = h < a.H;
  constexpr int NO = (PC_MAXD + 127) / 128;          // groups of 4 dims per lane

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // the merge waits for this grid itself
  const PagedPlan plan = paged_plan(a, unit, threads, scratch);
  // sequences without a row (no unit has a tile of theirs): a lane looks at each, the warp clears
  for (int b0 = unit; b0 < a.B; b0 += 32 * a.units) {
    const int64_t bl = (int64_t)b0 + (int64_t)lane * a.units;
    for (unsigned none = __ballot_sync(0xffffffffu, bl < a.B && paged_tiles(a, (int)min(bl, (int64_t)a.B - 1)) == 0); none; none &= none - 1) {
      const int b = b0 + (__ffs(none) - 1) * a.units;
      if (!hv) continue;
      for (int c = lane; c < dv; c += 32) Elem<T>::st((T*)a.out + ((size_t)b * a.H + h) * dv + c, 0.f);
      if (a.lse && lane == 0) a.lse[(size_t)b * a.H + h] = a.sink[h];
    }
  }
  if (hg == 0 && threadIdx.x == 0) paged_note(a, plan, unit);
  PagedSeg seg;
  seg.start(plan, unit);
  while (seg.next(a)) {
    const int b = seg.b, na = seg.na, nw = seg.nw;
    const int64_t ta = seg.ta, t1 = seg.t1;
    int64_t t = seg.t0;
    // the lane's row of a tile: in the pool or the window, -1 = none
    auto resolve = [&](int64_t tile) {
      if (tile >= t1) return -1;
      const bool in_a = tile < ta;
      const int64_t v = (in_a ? tile : tile - ta) * PC_ROWS + lane;
      if (in_a) return v < na ? (int)paged_row(a, b, (int)v) : -1;
      return v < nw ? (int)((int64_t)b * a.W + v) : -1;
    };
    auto copy = [&](int64_t tile, int row, int buf) {
      const T* base = tile < ta ? (const T*)a.pages : (const T*)a.win;
      T* dst = tiles_s + (size_t)buf * PC_ROWS * pitch;
      for (int i = threadIdx.x; i < PC_ROWS * vecs; i += threads) {       // whole warps
        const int r = i / vecs, c = (i - r * vecs) * VEC;
        const int y = __shfl_sync(0xffffffffu, row, r);
        cp_async16_zfill(dst + r * pitch + c, base + (size_t)(y < 0 ? 0 : y) * dk + c, y < 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int row = resolve(t), next = resolve(t + 1);
    copy(t, row, 0);
    if (hv)
      for (int c = lane * VEC; c < dk; c += 32 * VEC) {
        float x[VEC];
        Elem<T>::ld_vec((const T*)a.q + ((size_t)b * a.H + h) * dk + c, x);
#pragma unroll
        for (int u = 0; u < VEC; ++u) Qs[c + u] = x[u];
      }
    float4 o[NO];
#pragma unroll
    for (int i = 0; i < NO; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m_run = -INFINITY, l_run = 0.f;
    int buf = 0;
    for (; t < t1; ++t) {
      const bool ahead = bufs == 2 && t + 1 < t1;
      if (ahead) copy(t + 1, next, buf ^ 1);
      const int after = resolve(t + 2);                // its loads are in flight during the tile's work
      if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      const T* Ks = tiles_s + (size_t)buf * PC_ROWS * pitch;
      if (hv) {
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        const T* kr = Ks + lane * pitch;
#pragma unroll 4
        for (int c = 0; c < dk; c += VEC) {
          float x[VEC];
          Elem<T>::ld_vec(kr + c, x);
#pragma unroll
          for (int u = 0; u < VEC; u += 4) {
            const float4 y = *reinterpret_cast<const float4*>(Qs + c + u);
            s0 = fmaf(x[u], y.x, s0);
            s1 = fmaf(x[u + 1], y.y, s1);
            s2 = fmaf(x[u + 2], y.z, s2);
            s3 = fmaf(x[u + 3], y.w, s3);
          }
        }
        const float logit = row >= 0 ? ((s0 + s1) + (s2 + s3)) * a.sm_scale : -INFINITY;
        const float m_new = fmaxf(m_run, warp_max(logit));
        if (m_new != -INFINITY) {                      // else: no row of the piece so far
          const float alpha = __expf(m_run - m_new);
          const float p = __expf(logit - m_new);
          l_run = l_run * alpha + warp_sum(p);
          m_run = m_new;
#pragma unroll
          for (int i = 0; i < NO; ++i) { o[i].x *= alpha; o[i].y *= alpha; o[i].z *= alpha; o[i].w *= alpha; }
#pragma unroll 4
          for (int r = 0; r < PC_ROWS; ++r) {
            const float pr = __shfl_sync(0xffffffffu, p, r);
            const T* vr = Ks + r * pitch + 4 * lane;
#pragma unroll
            for (int i = 0; i < NO; ++i) {
              if (4 * lane + 128 * i < dv) {
                float x[4];
                load4<T>(vr + 128 * i, x);
                o[i].x = fmaf(pr, x[0], o[i].x);
                o[i].y = fmaf(pr, x[1], o[i].y);
                o[i].z = fmaf(pr, x[2], o[i].z);
                o[i].w = fmaf(pr, x[3], o[i].w);
              }
            }
          }
        }
      }
      __syncthreads();                                // the buffer is read
      row = next;
      next = after;
      if (bufs == 2) buf ^= 1;
      else if (t + 1 < t1) copy(t + 1, row, 0);
    }
    if (!hv) continue;
    if (seg.whole) {
      const float sk = a.sink[h], M = fmaxf(sk, m_run);
      float den = 0.f, f = 0.f;
      if (M != -INFINITY) {
        f = m_run == -INFINITY ? 0.f : __expf(m_run - M);
        den = __expf(sk - M) + l_run * f;
      }
      const float inv = den > 0.f ? f / den : 0.f;
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const int c = 4 * lane + 128 * i;
        if (c < dv) {
          T* dst = (T*)a.out + ((size_t)b * a.H + h) * dv + c;
          Elem<T>::st(dst, o[i].x * inv);
          Elem<T>::st(dst + 1, o[i].y * inv);
          Elem<T>::st(dst + 2, o[i].z * inv);
          Elem<T>::st(dst + 3, o[i].w * inv);
        }
      }
      if (a.lse && lane == 0) a.lse[(size_t)b * a.H + h] = den > 0.f ? M + logf(den) : -INFINITY;
    } else {
      float* blk = a.part + (size_t)seg.slot(unit) * paged_part_block(a.H, dv);
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const int c = 4 * lane + 128 * i;
        if (c < dv) *reinterpret_cast<float4*>(blk + paged_part_val(a.H, h, c)) = o[i];
      }
      if (lane == 0) {
        float4* rec = reinterpret_cast<float4*>(blk + paged_part_rec(a.H, dv, h));
        rec[0] = make_float4(m_run, l_run, 1.f, 1.f);
        rec[1] = make_float4(1.f, 1.f, 0.f, 0.f);
      }
    }
  }
}

// Joins the pieces of cut sequences: out = sum_p e^{m_p - M} o_p / (e^{sink - M} +
// sum_p e^{m_p - M} l_p).  The units noted which sequences they began and did not finish;
// every CTA gathers those notes and takes its share of the items (sequence, eight heads,
// slice of the dims), the slices as narrow as it takes to give every CTA an item.  Eight
// heads' 16-byte pieces of a partial are one 128-byte line.  Where a slice leaves threads
// over, they share its pieces.  All sums run in a fixed order, so a result does not depend
// on the order in which the units ended.  Bound: L2, H * (dv + 4) * 4 bytes per piece, and
// the latency of its few round trips.
constexpr int PM_THREADS = 256, PM_H = 8, PM_C = PM_THREADS / PM_H, PM_SLICES = 16, PM_EARLY = 5, PM_PER_SM = 2;
constexpr int PM_FEW = 8;        // partials that one warp joins by itself
// Shared memory per unit (under the 48 KB of a plain launch for the 296 units that fp32 may have)
constexpr size_t pm_unit_bytes(bool part16) { return PM_H * (sizeof(float4) + (part16 ? sizeof(float2) : 0)) + sizeof(int4); }
// acc += w times a 16-byte piece of a partial
template <bool PART16>
__device__ __forceinline__ void merge_add(float* acc, const uint4& v, float w) {
  const uint32_t u4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (PART16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u4[q]));
      acc[2 * q] = fmaf(w, f.x, acc[2 * q]);
      acc[2 * q + 1] = fmaf(w, f.y, acc[2 * q + 1]);
    } else {
      acc[q] = fmaf(w, __uint_as_float(u4[q]), acc[q]);
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void merge_store(T* dst, const float* v) {
  if constexpr (V == Elem<T>::VEC) {
    Elem<T>::st_vec(dst, v);
  } else {
#pragma unroll
    for (int u = 0; u < V; ++u) Elem<T>::st(dst + u, v[u]);
  }
}

template <typename T, bool PART16>
__global__ void __launch_bounds__(PM_THREADS, PM_PER_SM)
paged_merge_kernel(PagedAttnArgs a) {
  constexpr int V = PART16 ? 8 : 4;                  // dims of a 16-byte piece
  // per unit: the list {unit, sequence, partials, -}; per partial and head: {m, l, s0, s1}, then
  // e^{m - M} times the quarters' powers, and {s2, s3}
  extern __shared__ int4 list[];
  float4* const wts = reinterpret_cast<float4*>(list + a.units);
  float2* const s23 = reinterpret_cast<float2*>(wts + (size_t)a.units * PM_H);
  __shared__ float red[2][PM_THREADS / 32][PM_H];
  __shared__ float sums[V][PM_THREADS];
  __shared__ int counts[2];
  const int dv = a.dv, H = a.H;
  const int hl = threadIdx.x & (PM_H - 1), j = threadIdx.x / PM_H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the list: sequences of few partials from the front, the others from the back
  if (warp == 0) {
    const int2* notes = paged_notes(a);
    int few = 0, many = 0;
#pragma unroll 1
    for (int u0 = 0; u0 < a.units; u0 += 32) {
      const int2 note = u0 + lane < a.units ? __ldcg(&notes[u0 + lane]) : make_int2(-1, 0);
      const unsigned f = __ballot_sync(0xffffffffu, note.y > 0 && note.y <= PM_FEW), m = __ballot_sync(0xffffffffu, note.y > PM_FEW);
      const unsigned below = (1u << lane) - 1u;
      if (note.y > 0)
        list[note.y <= PM_FEW ? few + __popc(f & below) : a.units - 1 - many - __popc(m & below)] =
            make_int4(u0 + lane, note.x, note.y, 0);
      few += __popc(f);
      many += __popc(m);
    }
    if (lane == 0) { counts[0] = few; counts[1] = many; }
  }
  __syncthreads();
  const int count = counts[1];
  const int hb = (H + PM_H - 1) / PM_H, pieces = dv / V;
  int slices = 1;
  while (slices < PM_SLICES && 2 * count * hb * slices <= (int)gridDim.x && pieces / slices > 4) slices <<= 1;
  const int width = (pieces + slices - 1) / slices;   // 16-byte pieces of a slice
  const size_t block = paged_part_block(H, dv);
  {
    // Few partials: a warp takes eight heads and 8 pieces of the dims.  Lane (head, q): partials q and
    // q + 4 in the weights, pieces q and q + 4 in the sums; all loads are one round trip.
    const int q = lane >> 3, wide = (pieces + 7) / 8;
    for (int item = blockIdx.x * (PM_THREADS / 32) + warp; item < counts[0] * hb * wide; item += gridDim.x * (PM_THREADS / 32)) {
      const int cg = item % wide, blk8 = item / wide % hb;
      const int4 cut = list[item / (wide * hb)];
      const int b = cut.y, n = cut.z, h = blk8 * PM_H + hl;
      const bool hv = h < H;
      const int hc = hv ? h : H - 1;
      const float* part = a.part + (size_t)(2 * cut.x) * block;
      auto partial = [&](int p) { return part + (p ? 2 * p * block : block); };
      uint4 x[2][PM_FEW];
#pragma unroll
      for (int u = 0; u < PM_FEW; ++u) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = cg * 8 + 4 * k + q;
          if (u < n && c < pieces) x[k][u] = __ldcg(reinterpret_cast<const uint4*>(partial(u)) + (size_t)c * H + hc);
        }
      }
      const size_t rec = paged_part_rec(H, dv, hc);
      const float sk = a.sink[hc];
      float m[2], l[2], w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int p = q + 4 * k;
        m[k] = -INFINITY;
        l[k] = 0.f;
        w[k] = 1.f;
        if (p < n) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(partial(p) + rec));
          if (PART16) w[k] = __ldcg(partial(p) + rec + 2 + ((cg * 8) >> 4));      // 16 pieces a quarter
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
        w[k] *= e;
      }
      den += __shfl_xor_sync(0xffffffffu, den, 8);
      den += __shfl_xor_sync(0xffffffffu, den, 16);
      den += sk == -INFINITY ? 0.f : __expf(sk - M);
      const float inv = den > 0.f ? 1.f / den : 0.f;
      float acc[2][V];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int u = 0; u < V; ++u) acc[k][u] = 0.f;
#pragma unroll
      for (int u = 0; u < PM_FEW; ++u) {
        if (u < n) {
          const float wu = __shfl_sync(0xffffffffu, w[u >> 2], hl + 8 * (u & 3)) * inv;
#pragma unroll
          for (int k = 0; k < 2; ++k) merge_add<PART16>(acc[k], x[k][u], wu);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = cg * 8 + 4 * k + q;
        if (hv && c < pieces) merge_store<T, V>((T*)a.out + ((size_t)b * H + h) * dv + V * c, acc[k]);
      }
      if (a.lse && cg == 0 && q == 0 && hv) a.lse[(size_t)b * H + h] = den > 0.f ? M + logf(den) : -INFINITY;
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
    auto load = [&](int p, int c) { return __ldcg(reinterpret_cast<const uint4*>(partial(p)) + (size_t)c * H + hc); };
    const size_t rec = paged_part_rec(H, dv, hc);
    const float sk = a.sink[hc];
    float acc[V];
    const int cend = min(pieces, (sl + 1) * width);
    const int c0 = sl * width + jc;
    float M = sk;
    for (int p0 = j; p0 < n; p0 += 4 * PM_C) {        // four records' loads at a time
      float4 r0[4];
      float2 r1[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int p = p0 + u * PM_C;
        if (p < n) {
          const float4* r = reinterpret_cast<const float4*>(partial(p) + rec);
          r0[u] = __ldcg(r);
          if (PART16) r1[u] = __ldcg(reinterpret_cast<const float2*>(r + 1));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int p = p0 + u * PM_C;
        if (p < n) {
          wts[p * PM_H + hl] = r0[u];
          if (PART16) s23[p * PM_H + hl] = r1[u];
          M = fmaxf(M, r0[u].x);
        }
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
      const float4 r = wts[p * PM_H + hl];            // this thread's own
      const float w = r.x == -INFINITY ? 0.f : __expf(r.x - M);
      den += w * r.y;
      if (PART16) {
        const float2 s = s23[p * PM_H + hl];
        wts[p * PM_H + hl] = make_float4(w * r.z, w * r.w, w * s.x, w * s.y);
      } else {
        wts[p * PM_H + hl].x = w;
      }
    }
#pragma unroll
    for (int o = PM_H; o < 32; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < PM_H) red[1][warp][lane] = den;
    __syncthreads();
    den = sk == -INFINITY ? 0.f : __expf(sk - M);
#pragma unroll
    for (int w = 0; w < PM_THREADS / 32; ++w) den += red[1][w][hl];
    const float inv = den > 0.f ? 1.f / den : 0.f;
    for (int c = c0; c - jc < cend; c += gw) {
#pragma unroll
      for (int u = 0; u < V; ++u) acc[u] = 0.f;
      const float* wq = reinterpret_cast<const float*>(wts + hl) + (PART16 ? (c >> 4) & 3 : 0);
      if (c < cend) {
#pragma unroll 1
        for (int p0 = g; p0 < n; p0 += PM_EARLY * groups) {
          uint4 x[PM_EARLY];
#pragma unroll
          for (int u = 0; u < PM_EARLY; ++u)
            if (p0 + u * groups < n) x[u] = load(p0 + u * groups, c);
#pragma unroll
          for (int u = 0; u < PM_EARLY; ++u)
            if (p0 + u * groups < n) merge_add<PART16>(acc, x[u], wq[(p0 + u * groups) * PM_H * 4]);
        }
      }
      if (groups > 1) {                               // (the slice is one round of its threads)
#pragma unroll
        for (int u = 0; u < V; ++u) sums[u][threadIdx.x] = acc[u];
        __syncthreads();
        for (int o = 1; g == 0 && o < groups; ++o)
#pragma unroll
          for (int u = 0; u < V; ++u) acc[u] += sums[u][threadIdx.x + o * gw * PM_H];
      }
      if (g == 0 && c < cend && hv) {
#pragma unroll
        for (int u = 0; u < V; ++u) acc[u] *= inv;
        merge_store<T, V>((T*)a.out + ((size_t)b * H + h) * dv + V * c, acc);
      }
    }
    if (a.lse && j == 0 && sl == 0 && hv) a.lse[(size_t)b * H + h] = den > 0.f ? M + logf(den) : -INFINITY;
    __syncthreads();                                  // the weights and sums are read
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedAttnArgs& a, int dtype, bool part16, cudaStream_t st) {
  if (a.units == 1) return cudaSuccess;                // nothing is ever cut
  const int64_t most = (int64_t)(a.units - 1) * ((a.H + PM_H - 1) / PM_H) * PM_SLICES;
  const int grid = PM_PER_SM * num_sms();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < grid ? most : grid));
  cfg.blockDim = dim3(PM_THREADS);
  cfg.dynamicSmemBytes = (size_t)a.units * pm_unit_bytes(part16);            // a sequence has at most `units` partials
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits for the pieces first of all
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  if (part16) return cudaLaunchKernelEx(&cfg, paged_merge_kernel<__nv_bfloat16, true>, a);
  return dtype == CSA_BF16 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<__nv_bfloat16, false>, a)
                           : cudaLaunchKernelEx(&cfg, paged_merge_kernel<float, false>, a);
}

// Two CTAs per SM over the head groups.
int paged_units_cc(int B, int H, int64_t rows_max) {
  const int groups = (H + PC_WARPS - 1) / PC_WARPS;
  return paged_units(2 * num_sms() / groups, B, rows_max, PC_ROWS, PC_MIN_TILES);
}

cudaError_t launch_paged_attn_cc(PagedAttnArgs a, int dtype, cudaStream_t st) {
  a.tile_log2 = 5;
  static_assert(PC_ROWS == 1 << 5, "tile rows");
  a.min_tiles = PC_MIN_TILES;
  a.begin_cost = 0;
  a.units = paged_units(a, paged_units_cc(a.B, a.H, paged_rows_max(a)));
  const int warps = a.H < PC_WARPS ? a.H : PC_WARPS;
  auto go = [&](auto tag) {
    using T = decltype(tag);
    const size_t tile = (size_t)PC_ROWS * (a.dk + Elem<T>::VEC) * sizeof(T), qs = (size_t)warps * a.dk * sizeof(float);
    const int bufs = 2 * tile + qs <= 48 * 1024 ? 2 : 1;      // two only while several CTAs still share an SM
    const dim3 grid(a.units, (a.H + PC_WARPS - 1) / PC_WARPS);
    static std::atomic<uint64_t> ready;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(paged_attn_cc_kernel<T>), ready, 96 * 1024);
    if (e != cudaSuccess) return e;
    note_launch();
    paged_attn_cc_kernel<T><<<grid, warps * 32, bufs * tile + qs, st>>>(a, bufs);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_paged_merge(a, dtype, false, st);
  };
  return dtype == CSA_BF16 ? go(__nv_bfloat16()) : go(float());
}

}  // namespace csa
