// paged_append.cu - flint_attn_paged_append: new tokens' keys and values into
// the pages of a cache.
//
// Token t of sequence b (cu[b] <= t < cu[b+1]) has position p = lens[b] + t -
// cu[b]; k_hat = RoPE_p(RMSNorm(k)) and v go into slot p of the sequence, in
// the cache's type (Flint layers page, nemo_automodel.components.models.flint.
// layers, FlintAttention: per-head RMSNorm, then RoPE on selected layers).
//
// Bound by HBM: 512 bytes of K and V read per (token, KV head) and 512 (bf16)
// or 256 (e4m3) written, against ~100 operations. A block takes kTok tokens;
// it finds their slots and builds their cos/sin table once for all heads, then
// each half-warp moves one head's K and V row at a time with 16-byte accesses.
#include "paged.cuh"

namespace flint {

namespace {

constexpr int kTok = 4;
constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedAppendLaunch a) {
  __shared__ float cs[kTok][kHeadDim / 2], sn[kTok][kHeadDim / 2];
  __shared__ long long slot[kTok];     // element offset of the token's slot, -1: none
  __shared__ int pos_s[kTok];
  const int t0 = blockIdx.x * kTok;
  if (threadIdx.x < kTok) {
    const int t = t0 + threadIdx.x;
    long long off = -1;
    int pos = 0;
    if (t < a.T && t < __ldg(a.cu + a.N)) {          // tokens past the last sequence: none
      const int b = doc_of(a.cu, a.N, t);
      const int len = __ldg(a.lens + b);
      const long long p = (long long)len + t - __ldg(a.cu + b);
      if (len != -1) {                               // -1: a row that is not in use
        if (len >= 0 && p >= 0 && p < (long long)a.c.P * a.c.max_pages) {
          pos = (int)p;
          off = slot_offset(a.c, b, pos);
        }
        if (off < 0) atomicOr(a.status, kStatusDecodeRange);
      }
    }
    slot[threadIdx.x] = off;
    pos_s[threadIdx.x] = pos;
  }
  __syncthreads();
  if (a.rope) {
    for (int e = threadIdx.x; e < kTok * (kHeadDim / 2); e += kThreads) {
      const int i = e / (kHeadDim / 2), j = e % (kHeadDim / 2);
      rope_cos_sin(pos_s[i], j, a.rope_pow, &cs[i][j], &sn[i][j]);
    }
    __syncthreads();
  }
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4;
  float w[8];
  load8(a.wk + 8 * l, w);
  const int rows = kTok * a.c.Hk;
  const int iters = (rows + kThreads / 16 - 1) / (kThreads / 16);   // whole warps in every one
  for (int it = 0; it < iters; ++it) {
    const int rr = grp + it * (kThreads / 16);
    const int i = rr < rows ? rr / a.c.Hk : 0, g = rr % a.c.Hk;
    const bool live = rr < rows && slot[i] >= 0;
    float x[8] = {}, y[8] = {};
    if (live) {
      const long long t = t0 + i;
      load8(a.k + t * a.k_stride + g * kHeadDim + 8 * l, x);
      load8(a.v + t * a.v_stride + g * kHeadDim + 8 * l, y);
    }
    row_prologue(x, w, &cs[i][8 * (l & 7)], &sn[i][8 * (l & 7)], a.rope, a.eps);
    if (live) {
      const long long off = slot[i] + g * a.c.head_stride;
      store_row(a.c, a.c.k, off, x, a.c.k_scale ? __ldg(a.c.k_scale + g) : 1.f);
      store_row(a.c, a.c.v, off, y, a.c.v_scale ? __ldg(a.c.v_scale + g) : 1.f);
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t st) {
  ProfScope prof(kKPagedAppend, st);
  const unsigned grid = ((unsigned)a.T + kTok - 1) / kTok;
  paged_append_kernel<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace flint
