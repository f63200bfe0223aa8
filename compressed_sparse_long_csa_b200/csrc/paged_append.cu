// Appending latent rows to a paged cache with the position rotation applied on the way, and
// the same rotation of the queries' rotary parts into the attention's query rows.
//
// "Технический отчёт DeepSeek-V4 — часть 1/2": the latent's last 64 of 576 dims carry the
// position (partial rotary embedding).  A pair (a, b) of the rotated dims at position p with
// frequency f becomes (a cos t - b sin t, a sin t + b cos t), t = p f.
//
// Bound: launch and load latency for single tokens; for chunks the loads that are in flight (a CTA
// loads, waits and stores): 4096 tokens of 128 heads 32.7 us, 4.3 TB/s of 6.56 measured, and 30.7 with
// query rows of the rotary part alone, so that where the rows are written is a small part of it.  A CTA
// takes one token and a share of its heads.
#include <type_traits>

#include "common.cuh"

namespace csa {

namespace {

constexpr int PA_MAX_HALF = 288;       // rotated pairs of a row (d_r <= 576)
constexpr int PA_THREADS = 128;
// Query pieces that a thread loads first of all, and the heads of a CTA: few of both while the
// grid does not fill the GPU (latency), many once it does (a token's entry, page and angles are
// then looked up once).  bf16, 128 heads: 160 tokens 3.8 us against 5.0 the other way, 400
// tokens 7.5 against 6.4.  Many is as measured for 128 heads of 64 rotated dims in bf16, neighbouring
// pairs: 8 pieces a thread (4096 tokens 32.7 us; 4: 35.4, 16: 38.4).  Pairs of halves have 4 such
// pieces and leave half of the slots unused (35.6 us), fp32 has 16 (55.9 us, halves 52.3).
constexpr int PA_FEW = 1, PA_MANY = 8;   // (few, two pieces of 32 heads: one token 2.8 us, not 2.4)
constexpr int PA_FEW_HEADS = 16;

struct AppendArgs {
  const void* rows; int64_t rows_ld;
  const int32_t *seq, *entry, *pos;
  const float* inv_freq; int dr;
  void* pages; int64_t n_pages; int page;
  const int32_t* table; int table_w;
  int B, d;
  const void* q_pe; int64_t qpe_ld_t, qpe_ld_h;
  void* q; int H, dq;
  int heads;                           // heads per CTA
  unsigned* err;
};

// cos and sin of pos * f.  The angle reaches 1e6 and more, where fp32 would lose its
// fraction of a turn: the product (exact to 2^-53) and its reduction to [-1/2, 1/2] turns
// are fp64.  The reduced angle is then rounded to fp32 (up to 2^-25 of half a turn) and the functions
// are fp32 ones: the narrow fp64 pipe would cost a single token more than its launch.  An fp32 row's
// error is 1.3 times that of cos and sin formed in 64 bits (3.9e-8 against 3.0e-8 relative to
// the rotated rows); a bf16 row's is its own rounding's.
__device__ __forceinline__ void turn(int pos, float f, float* c, float* s) {
  const double r = (double)pos * (double)f * 0.15915494309189533577;   // turns
  sincospif((float)(2.0 * (r - rint(r))), s, c);
}

// grid (T, ceil(H / heads)); the blockIdx.y = 0 CTA also writes the token's latent row.  Every
// thread's first pieces are on their way before the token's entry, page and angles are known:
// one latency instead of four in a row.
template <typename T, bool NEAR, int EARLY>
__global__ void __launch_bounds__(PA_THREADS)
latent_append_paged_kernel(AppendArgs a) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ float cs[PA_MAX_HALF], sn[PA_MAX_HALF];
  const int t = blockIdx.x, tid = threadIdx.x;
  const int half = a.dr / 2, base = a.d - a.dr;
  // rotated piece i of d_r values: near pairs, values VEC i ..; far pairs, VEC values of the first
  // half and the same of the second
  const int pieces = NEAR ? a.dr / VEC : half / VEC;
  struct Piece { uint4 lo, hi; };
  auto fetch = [&](const T* src, int i) {
    Piece p;
    p.lo = __ldcs(reinterpret_cast<const uint4*>(src + i * VEC));
    p.hi = NEAR ? p.lo : __ldcs(reinterpret_cast<const uint4*>(src + half + i * VEC));
    return p;
  };
  auto put = [&](T* dst, const float* v) {
    uint4 o;
    Elem<T>::st_vec(reinterpret_cast<T*>(&o), v);
    __stcs(reinterpret_cast<uint4*>(dst), o);
  };
  auto store = [&](T* dst, int i, const Piece& p) {
    float x[VEC], y[VEC];
    Elem<T>::ld_vec(reinterpret_cast<const T*>(&p.lo), x);
    if (NEAR) {
#pragma unroll
      for (int u = 0; u < VEC; u += 2) {
        const float c = cs[(i * VEC + u) >> 1], s = sn[(i * VEC + u) >> 1], v = x[u], w = x[u + 1];
        x[u] = v * c - w * s;
        x[u + 1] = v * s + w * c;
      }
    } else {
      Elem<T>::ld_vec(reinterpret_cast<const T*>(&p.hi), y);
#pragma unroll
      for (int u = 0; u < VEC; ++u) {
        const float c = cs[i * VEC + u], s = sn[i * VEC + u], v = x[u], w = y[u];
        x[u] = v * c - w * s;
        y[u] = v * s + w * c;
      }
      put(dst + half + i * VEC, y);
    }
    put(dst + i * VEC, x);
  };
  const int h0 = blockIdx.y * a.heads, n = a.q ? min(a.heads, a.H - h0) * pieces : 0;
  const T* q_src = (const T*)a.q_pe + (size_t)t * a.qpe_ld_t + (size_t)h0 * a.qpe_ld_h;
  T* q_dst = (T*)a.q + ((size_t)t * a.H + h0) * a.dq + (a.dq - a.dr);
  auto q_fetch = [&](int i) { return fetch(q_src + (size_t)(i / pieces) * a.qpe_ld_h, i % pieces); };
  Piece x[EARLY];
#pragma unroll
  for (int u = 0; u < EARLY; ++u)
    if (tid + u * PA_THREADS < n) x[u] = q_fetch(tid + u * PA_THREADS);
  const int plain = base / VEC, row_n = blockIdx.y == 0 ? plain + pieces : 0;
  const T* r_src = (const T*)a.rows + (size_t)t * a.rows_ld;
  Piece r;
  if (tid < row_n) {
    if (tid < plain) r.lo = *reinterpret_cast<const uint4*>(r_src + tid * VEC);
    else r = fetch(r_src + base, tid - plain);
  }

  const int e = a.entry[t], b = a.seq ? a.seq[t] : t;
  if (a.dr > 0) {
    const int p = a.pos ? a.pos[t] : e;
    for (int i = tid; i < half; i += PA_THREADS) turn(p, a.inv_freq[i], &cs[i], &sn[i]);
    __syncthreads();
  }
  if (e < 0) return;                                  // a padding row
  int64_t row = -1;
  if (b >= 0 && b < a.B && (int64_t)e < (int64_t)a.table_w * a.page) {
    const unsigned pg = (unsigned)e / (unsigned)a.page;
    const int id = a.table[(size_t)b * a.table_w + pg];
    if (id >= 0 && (int64_t)id < a.n_pages) row = (int64_t)id * a.page + (e - (int)pg * a.page);
  }
  if (row < 0) {
    if (tid == 0) raise_err(a.err, CSA_DEVERR_ENTRY);
    return;
  }
  T* r_dst = (T*)a.pages + (size_t)row * a.d;
  for (int i = tid; i < row_n; i += PA_THREADS) {
    if (i != tid) {
      if (i < plain) r.lo = *reinterpret_cast<const uint4*>(r_src + i * VEC);
      else r = fetch(r_src + base, i - plain);
    }
    if (i < plain) *reinterpret_cast<uint4*>(r_dst + i * VEC) = r.lo;
    else store(r_dst + base, i - plain, r);
  }
#pragma unroll
  for (int u = 0; u < EARLY; ++u) {
    const int i = tid + u * PA_THREADS;
    if (i < n) store(q_dst + (size_t)(i / pieces) * a.dq, i % pieces, x[u]);
  }
  for (int i = tid + EARLY * PA_THREADS; i < n; i += PA_THREADS) {
    const Piece p = q_fetch(i);
    store(q_dst + (size_t)(i / pieces) * a.dq, i % pieces, p);
  }
}

}  // namespace

cudaError_t launch_latent_append_paged(const void* rows, int64_t rows_ld, const int32_t* seq, const int32_t* entry,
                                       const int32_t* pos, const float* inv_freq, int dr, int near, void* pages,
                                       int64_t n_pages, int page, const int32_t* table, int table_w, int B, int T,
                                       int d, const void* q_pe, int64_t qpe_ld_t, int64_t qpe_ld_h, void* q, int H,
                                       int dq, int dtype, cudaStream_t st, unsigned* err) {
  AppendArgs a{rows, rows_ld, seq, entry, pos, inv_freq, dr, pages, n_pages, page, table, table_w, B, d,
               q_pe, qpe_ld_t, qpe_ld_h, q, H, dq, q ? H : 1, err};
  const bool few = q && (int64_t)T * ((H + PA_FEW_HEADS - 1) / PA_FEW_HEADS) <= 12 * num_sms();
  if (few && H > PA_FEW_HEADS) a.heads = PA_FEW_HEADS;
  const dim3 grid(T, q ? (H + a.heads - 1) / a.heads : 1);
  note_launch();
  auto go = [&](auto tag, auto early) {
    using E = decltype(tag);
    constexpr int N = decltype(early)::value;
    if (near) latent_append_paged_kernel<E, true, N><<<grid, PA_THREADS, 0, st>>>(a);
    else latent_append_paged_kernel<E, false, N><<<grid, PA_THREADS, 0, st>>>(a);
  };
  using Few = std::integral_constant<int, PA_FEW>;
  using Many = std::integral_constant<int, PA_MANY>;
  if (dtype == CSA_BF16) { if (few) go(__nv_bfloat16(), Few()); else go(__nv_bfloat16(), Many()); }
  else { if (few) go(float(), Few()); else go(float(), Many()); }
  return cudaGetLastError();
}

}  // namespace csa
