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
__device__ __forceinline__ double rope_turns(int j, const RopePowers& w) {
  double f = 0.15915494309189533577;         // 1 / 2 pi
#pragma unroll
  for (int i = 0; i < 6; ++i)
    if (j & (1 << i)) f *= w.pow[i];
  return f;
}
// cos and sin of pos turns of 2 pi f. The angle is formed and reduced in double:
// in float it would be off by 0.004 rad at position 131071. Taking it in turns
// makes the reduction exact and lets sinpi / cospi do without their own (with
// exp2 and sincosf here, a table of 64 angles took 5000 cycles).
__device__ __forceinline__ void rope_cos_sin(int pos, double f, float* c, float* s) {
  double turns = (double)pos * f;
  turns -= rint(turns);
  sincospif(2.f * (float)turns, s, c);
}

// A row of 128 channels belongs to a half-warp: lane l has channels 4l .. 4l+3 (x[0])
// and 64 + 4l .. (x[1]), which RoPE rotates with each other, so the rotation stays
// in the lane and takes four angles.
struct RowPart {
  float x[2][4];
};
// The lane's 8 bf16 of a row as they lie in memory; lo: channels 4l .., hi: 64 + 4l ..
struct RowBits {
  uint2 lo, hi;
};
__device__ __forceinline__ RowBits load_row(const __nv_bfloat16* row) {
  const int l = threadIdx.x & 15;
  return {*reinterpret_cast<const uint2*>(row + 4 * l),
          *reinterpret_cast<const uint2*>(row + kHeadDim / 2 + 4 * l)};
}
__device__ __forceinline__ RowPart unpack_row(RowBits b) {
  const uint32_t u[2][2] = {{b.lo.x, b.lo.y}, {b.hi.x, b.hi.y}};
  RowPart r;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r.x[h][2 * i] = __uint_as_float(u[h][i] << 16);
      r.x[h][2 * i + 1] = __uint_as_float(u[h][i] & 0xffff0000u);
    }
  return r;
}

// RMSNorm with weight w, then (rope) the rotation of channel j with j + 64 by the
// lane's angles 4l .. 4l+3. The whole warp calls it (full-mask shuffles). The
// append and the decode kernel use this one function, so both store the same
// bits for the same token.
__device__ __forceinline__ void row_prologue(RowPart& r, const RowPart& w, const float (&cs)[4],
                                             const float (&sn)[4], bool rope, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) ss += r.x[0][e] * r.x[0][e] + r.x[1][e] * r.x[1][e];
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = rsqrtf(ss * (1.0f / kHeadDim) + eps);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = r.x[0][e] * inv * w.x[0][e], b = r.x[1][e] * inv * w.x[1][e];
    r.x[0][e] = rope ? a * cs[e] - b * sn[e] : a;
    r.x[1][e] = rope ? b * cs[e] + a * sn[e] : b;
  }
}

// The lane's part of a row as the cache stores it: bf16 (4 + 4 values), or e4m3 of
// x * inv_scale, saturated to +-448 (lo.x and hi.x, 4 bytes each). One rounding
// to nearest even; the product with the reciprocal is within 2^-23 of the quotient
// (16 divisions a lane cost as much as the rest of the row).
__device__ __forceinline__ RowBits pack_bf16(const RowPart& r) {
  RowBits b;
  uint32_t u[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(r.x[h][2 * i], r.x[h][2 * i + 1]);
      u[h][i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  b.lo = make_uint2(u[0][0], u[0][1]);
  b.hi = make_uint2(u[1][0], u[1][1]);
  return b;
}
__device__ __forceinline__ RowBits pack_e4m3(const RowPart& r, float inv_scale) {
  uint32_t u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(
        make_float2(r.x[h][0] * inv_scale, r.x[h][1] * inv_scale), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(
        make_float2(r.x[h][2] * inv_scale, r.x[h][3] * inv_scale), __NV_SATFINITE, __NV_E4M3);
    u[h] = a | (b << 16);
  }
  return {make_uint2(u[0], 0), make_uint2(u[1], 0)};
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t bits) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)bits, __NV_E4M3)));
}
__device__ __forceinline__ RowPart unpack_e4m3(RowBits b, float scale) {
  RowPart r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r.x[0][e] = e4m3_to_f32((b.lo.x >> (8 * e)) & 0xff) * scale;
    r.x[1][e] = e4m3_to_f32((b.hi.x >> (8 * e)) & 0xff) * scale;
  }
  return r;
}
// Stores the lane's part of a row at element offset off.
template <bool kE4m3>
__device__ __forceinline__ void store_row(void* pool, long long off, RowBits b) {
  const int l = threadIdx.x & 15;
  if constexpr (kE4m3) {
    uint8_t* row = static_cast<uint8_t*>(pool) + off + 4 * l;
    *reinterpret_cast<uint32_t*>(row) = b.lo.x;
    *reinterpret_cast<uint32_t*>(row + kHeadDim / 2) = b.hi.x;
  } else {
    __nv_bfloat16* row = static_cast<__nv_bfloat16*>(pool) + off + 4 * l;
    *reinterpret_cast<uint2*>(row) = b.lo;
    *reinterpret_cast<uint2*>(row + kHeadDim / 2) = b.hi;
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
cudaError_t launch_paged_append(const PagedAppendLaunch& a, int num_sms, cudaStream_t st);

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
