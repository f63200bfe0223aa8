// Appending latent rows to a paged cache with the position rotation applied on the way, and
// the same rotation of the queries' rotary parts into the attention's query rows.
//
// "Технический отчёт DeepSeek-V4 — часть 1/2": the latent's last 64 of 576 dims carry the
// position (partial rotary embedding).  A pair (a, b) of the rotated dims at position p with
// frequency f becomes (a cos t - b sin t, a sin t + b cos t), t = p f.
//
// Bound: HBM for chunks (each new row and rotary part read and written once), launch and
// load latency for single tokens.  A CTA takes one token and a share of its heads.
#include "common.cuh"

namespace csa {

namespace {

constexpr int PA_MAX_HALF = 288;       // rotated pairs of a row (d_r <= 576)
constexpr int PA_THREADS = 256;

struct AppendArgs {
  const void* rows; int64_t rows_ld;
  const int32_t *seq, *entry, *pos;
  const float* inv_freq; int dr, near;
  void* pages; int64_t n_pages; int page;
  const int32_t* table; int table_w;
  int B, T, d;
  const void* q_pe; int64_t qpe_ld_t, qpe_ld_h;
  void* q; int H, dq;
  int heads;                           // heads per CTA
  unsigned* err;
};

// cos and sin of pos * f.  The angle reaches 1e6 and more, where fp32 would lose its
// fraction of a turn: the product (exact to 2^-53) and its reduction to [-1/2, 1/2] turns
// are fp64, the functions of the reduced angle fp32.
__device__ __forceinline__ void turn(int pos, float f, float* c, float* s) {
  const double r = (double)pos * (double)f * 0.15915494309189533577;   // turns
  sincospif((float)(2.0 * (r - rint(r))), s, c);
}

// grid (T, ceil(H / heads)); the blockIdx.y = 0 CTA also writes the token's latent row.
template <typename T>
__global__ void __launch_bounds__(PA_THREADS)
latent_append_paged_kernel(AppendArgs a) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ float cs[PA_MAX_HALF], sn[PA_MAX_HALF];
  const int t = blockIdx.x;
  const int e = a.entry[t];
  if (e < 0) return;                                  // a padding row
  const int b = a.seq ? a.seq[t] : t;
  int64_t row = -1;
  if (b >= 0 && b < a.B && (int64_t)e < (int64_t)a.table_w * a.page) {
    const unsigned pg = (unsigned)e / (unsigned)a.page;
    const int id = a.table[(size_t)b * a.table_w + pg];
    if (id >= 0 && (int64_t)id < a.n_pages) row = (int64_t)id * a.page + (e - (int)pg * a.page);
  }
  if (row < 0) {
    if (threadIdx.x == 0) raise_err(a.err, CSA_DEVERR_ENTRY);
    return;
  }
  const int half = a.dr / 2, base = a.d - a.dr;
  if (a.dr > 0) {
    const int p = a.pos ? a.pos[t] : e;
    for (int i = threadIdx.x; i < half; i += PA_THREADS) turn(p, a.inv_freq[i], &cs[i], &sn[i]);
    __syncthreads();
  }
  // rotated piece i of a vector of dr dims: near pairs, VEC dims 8i ..; far pairs, VEC dims
  // of the first half and the same of the second
  const int pieces = a.near ? a.dr / VEC : half / VEC;
  auto rotate = [&](const T* src, T* dst, int i) {
    float x[VEC];
    Elem<T>::ld_vec(src + i * VEC, x);
    if (a.near) {
#pragma unroll
      for (int u = 0; u < VEC; u += 2) {
        const float c = cs[(i * VEC + u) >> 1], s = sn[(i * VEC + u) >> 1], p = x[u], q = x[u + 1];
        x[u] = p * c - q * s;
        x[u + 1] = p * s + q * c;
      }
    } else {
      float y[VEC];
      Elem<T>::ld_vec(src + half + i * VEC, y);
#pragma unroll
      for (int u = 0; u < VEC; ++u) {
        const float c = cs[i * VEC + u], s = sn[i * VEC + u], p = x[u], q = y[u];
        x[u] = p * c - q * s;
        y[u] = p * s + q * c;
      }
      Elem<T>::st_vec(dst + half + i * VEC, y);
    }
    Elem<T>::st_vec(dst + i * VEC, x);
  };
  if (blockIdx.y == 0) {
    const T* src = (const T*)a.rows + (size_t)t * a.rows_ld;
    T* dst = (T*)a.pages + (size_t)row * a.d;
    const int plain = base / VEC;
    for (int i = threadIdx.x; i < plain + pieces; i += PA_THREADS) {
      if (i < plain) *reinterpret_cast<uint4*>(dst + i * VEC) = *reinterpret_cast<const uint4*>(src + i * VEC);
      else rotate(src + base, dst + base, i - plain);
    }
  }
  if (a.q) {
    const int h0 = blockIdx.y * a.heads, n = min(a.heads, a.H - h0);
    for (int i = threadIdx.x; i < n * pieces; i += PA_THREADS) {
      const int h = h0 + i / pieces, c = i % pieces;
      rotate((const T*)a.q_pe + (size_t)t * a.qpe_ld_t + (size_t)h * a.qpe_ld_h,
             (T*)a.q + ((size_t)t * a.H + h) * a.dq + (a.dq - a.dr), c);
    }
  }
}

}  // namespace

cudaError_t launch_latent_append_paged(const void* rows, int64_t rows_ld, const int32_t* seq, const int32_t* entry,
                                       const int32_t* pos, const float* inv_freq, int dr, int near, void* pages,
                                       int64_t n_pages, int page, const int32_t* table, int table_w, int B, int T,
                                       int d, const void* q_pe, int64_t qpe_ld_t, int64_t qpe_ld_h, void* q, int H,
                                       int dq, int dtype, cudaStream_t st, unsigned* err) {
  AppendArgs a{rows, rows_ld, seq, entry, pos, inv_freq, dr, near, pages, n_pages, page, table, table_w, B, T, d,
               q_pe, qpe_ld_t, qpe_ld_h, q, H, dq, q ? H : 1, err};
  const dim3 grid(T, q ? (H + a.heads - 1) / a.heads : 1);
  note_launch();
  if (dtype == CSA_BF16) latent_append_paged_kernel<__nv_bfloat16><<<grid, PA_THREADS, 0, st>>>(a);
  else latent_append_paged_kernel<float><<<grid, PA_THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace csa
