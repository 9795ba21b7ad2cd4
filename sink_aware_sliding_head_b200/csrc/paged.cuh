// paged.cuh - what the paged-cache kernels share: the cache's addressing and
// its checks, the prologue of one row (RMSNorm, then NeoX RoPE), and the
// rounding of a row to the type the cache stores.
//
// A pool holds num_pages pages of P slots; sequence b's token t lives in page
// block_table[b][t / P], slot t % P. The element of KV head g, channel d is at
//   page * page_stride + g * head_stride + slot * token_stride + d
// (strides in elements), so head-major [pages, Hk, P, D] and token-major
// [pages, P, Hk, D] pools, or K and V interleaved in one tensor, are one case.
#pragma once
#include <cmath>
#include <cuda.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace flint {

constexpr int kCacheBf16 = FLINT_CACHE_BF16, kCacheE4m3 = FLINT_CACHE_E4M3;

// A validated flint_paged_cache_t with its device pointers.
struct PagedCache {
  int num_pages, P, max_pages, Hk, e4m3;
  long long page_stride, head_stride, token_stride, table_stride;
  const int32_t* table;
  void *k, *v;
  const float *k_scale, *v_scale;   // [Hk], nullptr: 1
};

// Element offset of slot pos of KV head 0, or -1 if pos has no page or the
// table's entry is not a page of the pool.
__device__ __forceinline__ long long slot_offset(const PagedCache& c, int b, int pos) {
  const int col = pos / c.P;
  if (pos < 0 || col >= c.max_pages) return -1;
  const int page = __ldg(c.table + b * c.table_stride + col);
  if ((unsigned)page >= (unsigned)c.num_pages) return -1;
  return page * c.page_stride + (pos - col * c.P) * c.token_stride;
}

// RoPE's frequencies in turns a position, theta^(-2j/D) / 2 pi for j < 64, as
// powers: pow[i] = theta^(-2^i / 64), so six products in double give any of them.
struct RopePowers {
  double pow[6];
};
inline RopePowers rope_powers(double theta) {
  RopePowers r;
  for (int i = 0; i < 6; ++i) r.pow[i] = std::exp2(-(double)(1 << i) / 64 * std::log2(theta));
  return r;
}
// cos and sin of pos * theta^(-2j/D). The angle is formed and reduced in double:
// in float it would be off by 0.004 rad at position 131071. Taking it in turns
// makes the reduction exact and lets sinpi / cospi do without their own (with
// exp2 and sincosf here, a table of 64 angles took 5000 cycles).
__device__ __forceinline__ void rope_cos_sin(int pos, int j, const RopePowers& w, float* c,
                                             float* s) {
  double f = 0.15915494309189533577;         // 1 / 2 pi
#pragma unroll
  for (int i = 0; i < 6; ++i)
    if (j & (1 << i)) f *= w.pow[i];
  double turns = (double)pos * f;
  turns -= rint(turns);
  sincospif(2.f * (float)turns, s, c);
}

__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

// RMSNorm with weight w, then (rope) the rotation of channel j with j + 64. A
// half-warp owns the row, lane l of it channels 8l .. 8l+7, whose partners are
// in lane l ^ 8; cs, sn: the cosines and sines of the lane's channels (angles
// 8 (l & 7) ..). The whole warp calls it (full-mask shuffles). The append and
// the decode kernel use this one function, so both store the same bits for the
// same token.
__device__ __forceinline__ void row_prologue(float (&x)[8], const float (&w)[8], const float* cs,
                                             const float* sn, bool rope, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(ss * (1.0f / kHeadDim) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
  if (rope) {
    const float sign = (threadIdx.x & 8) ? 1.f : -1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float partner = __shfl_xor_sync(0xffffffffu, x[e], 8);
      x[e] = x[e] * cs[e] + partner * (sign * sn[e]);
    }
  }
}

// Eight values as the cache stores them: bf16 (16 bytes), or e4m3 of x / scale,
// saturated to +-448 (8 bytes). One rounding each, to nearest even.
__device__ __forceinline__ uint4 pack_bf16_row(const float (&x)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  return u;
}
__device__ __forceinline__ uint2 pack_e4m3_row(const float (&x)[8], float scale) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] / scale, x[2 * i + 1] / scale),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t bits) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)bits, __NV_E4M3)));
}
// Stores the lane's channels 8l .. 8l+7 of a row at element offset off (e4m3:
// the first 8 bytes of u).
__device__ __forceinline__ void store_bits(const PagedCache& c, void* pool, long long off,
                                           uint4 u) {
  const int l = threadIdx.x & 15;
  if (c.e4m3)
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + off + 8 * l) = make_uint2(u.x, u.y);
  else
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + off + 8 * l) = u;
}
__device__ __forceinline__ void store_row(const PagedCache& c, void* pool, long long off,
                                          const float (&x)[8], float scale) {
  if (c.e4m3) {
    const uint2 u = pack_e4m3_row(x, scale);
    store_bits(c, pool, off, make_uint4(u.x, u.y, 0, 0));
  } else {
    store_bits(c, pool, off, pack_bf16_row(x));
  }
}

// ------------------------------------------------------------------ launchers
struct PagedAppendLaunch {
  PagedCache c;
  int N, T, rope;
  long long k_stride, v_stride;   // elements between tokens
  RopePowers rope_pow;
  float eps;
  const __nv_bfloat16 *k, *v, *wk;
  const int32_t *cu, *lens;
  int* status;
};
cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t st);

struct PagedDecodeLaunch {
  PagedCache c;
  int B, H, G, W, rope, out_f32;
  long long q_stride, k_stride, v_stride;
  RopePowers rope_pow;
  float eps, scale;
  const __nv_bfloat16 *q, *k, *v, *wq, *wk;
  const float* sink;
  const int32_t* lens;
  void* out;
  float* lse;
  int* status;
};
// Bytes of workspace for B rows and Hk KV heads on a GPU of num_sms SMs.
size_t decode_paged_bytes(int B, int Hk, int num_sms);
cudaError_t launch_decode_paged(const PagedDecodeLaunch& a, int num_sms, cudaStream_t st);
// A pool as [page][head][half][slot][channels] with 128-byte rows (bf16: two
// halves of 64 channels, e4m3: one of 128) and 128-byte swizzle; a box is `box`
// slots of one head of one page, both halves. ok is cleared on failure.
CUtensorMap paged_tensor_map(const PagedCache& c, const void* pool, int box, bool* ok);

}  // namespace flint
