// paged_append.cu - flint_attn_paged_append: new tokens' keys and values into
// the pages of a cache.
//
// Token t of sequence b (cu[b] <= t < cu[b+1]) has position p = lens[b] + t -
// cu[b]; k_hat = RoPE_p(RMSNorm(k)) and v go into slot p of the sequence, in
// the cache's type (Flint layers page, nemo_automodel.components.models.flint.
// layers, FlintAttention: per-head RMSNorm, then RoPE on selected layers).
//
// Bound by HBM: 512 bytes of K and V read per (token, KV head) and 512 (bf16)
// or 256 (e4m3) written, against ~100 operations. A half-warp takes a token: it
// requests the rows of up to 8 heads, then finds the token's slot and its 64
// angles (four a lane, shared by all heads) while they come, and needs neither
// shared memory nor a barrier. Blocks are persistent, so a lane forms its four
// frequencies once.
//
// Measured (B200, 6.56 TB/s copy): 65536 prompt tokens of 4 KV heads 45 us (5.9
// TB/s), 131072 without RoPE 87 us (6.2 TB/s); 22539 tokens of 8 heads to e4m3 30 us
// (4.6 TB/s: half of the issue slots and 40% of HBM are used; 16 warps an SM overlap
// their loads and conversions too little). Requesting the next token's rows before the
// current one's are done was slower when tried (65536 tokens: 55 us for 48), and so
// were four tokens a half-warp at a time where there is one KV head (25.3, 26.1).
#include "paged.cuh"

namespace flint {

namespace {

constexpr int kThreads = 128;                // 8 tokens at a time

// Heads whose rows are in flight together (four loads of 8 bytes a lane each), and
// blocks per SM by the registers that takes (two heads: 64 registers, 24 bytes of a
// lane's state in memory in bf16, 8 in e4m3). Eight heads in two turns of 4 against one
// of 8 take 53.9 and 45.8 us (32768 tokens, bf16), 49.8 and 41.3 (to e4m3); four heads in
// a turn of 4 or half a turn of 8 45.0 and 46.7, 44.7 and 47.4 (65536 tokens); one head in
// a turn of its own or a quarter of one of 4 20.6 and 23.7, 22.8 and 24.8; two heads 26.9
// and 30.7, 30.2 and 30.9.
constexpr int blocks_per_sm(int heads) {
  return heads <= 2 ? 8 : heads == 4 ? 5 : 4;
}

// The sequence of token t: the last b with cu[b] <= t, so that none is empty.
__device__ __forceinline__ int seq_of(const int32_t* cu, int N, int t) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (load(cu + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool kE4m3, int kHeads>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(kHeads))
paged_append_kernel(const __grid_constant__ PagedAppendLaunch a) {
  const int l = threadIdx.x & 15;
  previous_done();
  const RowPart w = unpack_row(load_row(a.wk));
  double f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = rope_turns(4 * l + e, a.rope_pow);
  const int used = min(a.T, load(a.cu + a.N));      // tokens past the last sequence: none
  const long long step = (long long)gridDim.x * (kThreads / 16);
  const long long first = (long long)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  // Both half-warps of a warp take as many turns: the shuffles are the warp's.
  for (long long t0 = first - (threadIdx.x >> 4 & 1); t0 < used; t0 += step) {
    const long long t = t0 + (threadIdx.x >> 4 & 1);
    const bool live = t < used;
    const __nv_bfloat16* krow = a.k + (live ? t : t0) * a.k_stride;
    const __nv_bfloat16* vrow = a.v + (live ? t : t0) * a.v_stride;
    RowBits kb[kHeads], vb[kHeads];
    auto request = [&](int g0) {
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
        if (g0 + i < a.c.Hk) {
          kb[i] = load_row(krow + (g0 + i) * kHeadDim);
          vb[i] = load_row(vrow + (g0 + i) * kHeadDim);
        }
    };
    request(0);
    long long off = -1;                              // the token's slot, -1: none
    int pos = 0;
    if (live) {
      const int b = seq_of(a.cu, a.N, (int)t), len = load(a.lens + b);
      const long long p = len + t - load(a.cu + b);
      if (len >= 0 && p >= 0 && p < (long long)a.c.P * a.c.max_pages) {
        pos = (int)p;
        off = slot_offset(a.c, b, pos);
      }
      // -1 marks a sequence that is not in use
      if (off < 0 && len != -1 && l == 0) atomicOr(a.status, kStatusDecodeRange);
    }
    Angles angles{};
    if (a.rope) angles = row_angles(pos, f);
    for (int g0 = 0; g0 < a.c.Hk; g0 += kHeads) {
      if (g0) request(g0);
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int g = g0 + i;
        if (g >= a.c.Hk) break;
        RowPart x = unpack_row(kb[i]);
        row_prologue(x, w, angles, a.rope, a.eps);
        RowBits ko, vo = vb[i];
        if constexpr (kE4m3) {
          ko = pack_e4m3(x, inv_scale(a.c.k_scale, g));
          vo = pack_e4m3(unpack_row(vo), inv_scale(a.c.v_scale, g));
        } else {
          ko = pack_bf16(x);
        }
        if (off >= 0) {
          store_row<kE4m3>(a.c.k, off + g * a.c.head_stride, ko);
          store_row<kE4m3>(a.c.v, off + g * a.c.head_stride, vo);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& a, int num_sms, cudaStream_t st) {
  ProfScope prof(kKPagedAppend, st);
  const int per = kThreads / 16;
  const int blocks = (int)(((long long)a.T + per - 1) / per);
  // A grid of 1, 2 or 4 times the resident blocks, or of all (16 sequences, RoPE). More
  // blocks even out the SMs; every block forms its frequencies anew.
  //   bf16  262144 tokens of 1 head 76.7, 73.1, 71.0, 82.8 us; 131072 of 2 50.0, 48.5,
  //         48.3, 52.5; 65536 of 4 46.2, 45.7, 45.1, 46.6; 32768 of 8 49.5, 48.0, 45.6, 45.1
  //   e4m3  83.7, 79.0, 76.8, 88.5; 57.8, 54.1, 53.5, 57.8; 44.5, 44.0, 44.2, 47.1; 42.0,
  //         43.1, 42.7, 43.3
  // bf16 takes four times, e4m3 once: best with eight heads, as good with four, 8% slower
  // than four times with one or two.
  typedef void (*Kernel)(PagedAppendLaunch);
  static const Kernel kernels[2][4] = {
      {paged_append_kernel<false, 1>, paged_append_kernel<false, 2>,
       paged_append_kernel<false, 4>, paged_append_kernel<false, 8>},
      {paged_append_kernel<true, 1>, paged_append_kernel<true, 2>,
       paged_append_kernel<true, 4>, paged_append_kernel<true, 8>}};
  const int v = a.c.Hk == 1 ? 0 : a.c.Hk == 2 ? 1 : a.c.Hk <= 4 ? 2 : 3;
  const int most = blocks_per_sm(1 << v) * num_sms * (a.c.e4m3 ? 1 : 4);
  const int grid = blocks < most ? blocks : most;
  return launch_overlapped(kernels[a.c.e4m3][v], grid, kThreads, 0, st, a);
}

}  // namespace flint
