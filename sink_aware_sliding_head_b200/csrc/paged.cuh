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
#include <cstdlib>
#include <cuda.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100_primitives.cuh"

namespace flint {

// Lengths, tables and scales may have been written by the kernel before this one, whose
// end these kernels may overlap (previous_done). So they are read by ordinary loads: the
// read-only path (__ldg) is for memory that nobody writes while the kernel lives, and its
// loads may be moved to before the wait.
template <typename T>
__device__ __forceinline__ T load(const T* p) { return *p; }

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
  const int page = load(c.table + b * c.table_stride + col);
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
  const double step = -std::log2(theta) / 64;
  for (int i = 0; i < 6; ++i) r.pow[i] = std::exp2(step * (1 << i));
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
  const float t = (float)turns;
  float s0, c0;
  sincospif(2.f * t, &s0, &c0);
  // what the float left out of the angle, to first order (up to 2^-25 of a turn)
  const float d = 6.2831853f * (float)(turns - (double)t);
  *s = fmaf(c0, d, s0);
  *c = fmaf(-s0, d, c0);
}

// A row of 128 channels belongs to a half-warp: lane l has channels 4l .. 4l+3 (x[0])
// and 64 + 4l .. (x[1]), which RoPE rotates with each other, so the rotation stays
// in the lane and takes four angles. Two channels to a register pair, so that the
// packed FP32 instructions do a row in half as many.
struct RowPart {
  uint64_t x[2][2];
  __device__ __forceinline__ void get(int h, float (&f)[4]) const {
    f2_split(x[h][0], f[0], f[1]);
    f2_split(x[h][1], f[2], f[3]);
  }
};
struct Angles {
  uint64_t c[2], s[2], minus_s[2];           // of channels 4l .. 4l+3
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
__device__ __forceinline__ uint64_t bf16x2_to_f2(uint32_t u) {
  return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ RowPart unpack_row(RowBits b) {
  return {{{bf16x2_to_f2(b.lo.x), bf16x2_to_f2(b.lo.y)},
           {bf16x2_to_f2(b.hi.x), bf16x2_to_f2(b.hi.y)}}};
}
// The row's four angles at pos; f: the lane's frequencies in turns.
__device__ __forceinline__ Angles row_angles(int pos, const double (&f)[4]) {
  float c[4], s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) rope_cos_sin(pos, f[e], &c[e], &s[e]);
  return {{f2(c[0], c[1]), f2(c[2], c[3])},
          {f2(s[0], s[1]), f2(s[2], s[3])},
          {f2(-s[0], -s[1]), f2(-s[2], -s[3])}};
}

// RMSNorm with weight w, then (rope) the rotation of channel j with j + 64 by the
// lane's angles. The whole warp calls it (full-mask shuffles). The append and the
// decode kernel use this one function, so both store the same bits for the same
// token.
__device__ __forceinline__ void row_prologue(RowPart& r, const RowPart& w, const Angles& t,
                                             bool rope, float eps) {
  const uint64_t q = ffma2(r.x[0][0], r.x[0][0], fmul2(r.x[0][1], r.x[0][1]));
  float s0, s1;
  f2_split(ffma2(r.x[1][0], r.x[1][0], ffma2(r.x[1][1], r.x[1][1], q)), s0, s1);
  float ss = s0 + s1;
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = rsqrtf(ss * (1.0f / kHeadDim) + eps);
  const uint64_t inv2 = f2(inv, inv);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t a = fmul2(fmul2(r.x[0][i], inv2), w.x[0][i]);
    const uint64_t b = fmul2(fmul2(r.x[1][i], inv2), w.x[1][i]);
    r.x[0][i] = rope ? ffma2(b, t.minus_s[i], fmul2(a, t.c[i])) : a;
    r.x[1][i] = rope ? ffma2(a, t.s[i], fmul2(b, t.c[i])) : b;
  }
}

// The lane's part of a row as the cache stores it: bf16 (4 + 4 values), or e4m3 of
// x * inv_scale, saturated to +-448 (lo.x and hi.x, 4 bytes each). One rounding
// to nearest even; the product with the reciprocal is within 2^-22 of the quotient
// (16 divisions a lane cost as much as the rest of the row).
__device__ __forceinline__ float inv_scale(const float* scale, int g) {
  float r = 1.f;
  if (scale) asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(load(scale + g)));
  return r;
}
__device__ __forceinline__ uint32_t f2_to_bf16x2(uint64_t v) {
  float a, b;
  f2_split(v, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ RowBits pack_bf16(const RowPart& r) {
  return {make_uint2(f2_to_bf16x2(r.x[0][0]), f2_to_bf16x2(r.x[0][1])),
          make_uint2(f2_to_bf16x2(r.x[1][0]), f2_to_bf16x2(r.x[1][1]))};
}
__device__ __forceinline__ uint32_t f2x2_to_e4m3(uint64_t u, uint64_t v) {
  float a, b, c, d;
  f2_split(u, a, b);
  f2_split(v, c, d);
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ RowBits pack_e4m3(const RowPart& r, float inv) {
  const uint64_t i2 = f2(inv, inv);
  return {make_uint2(f2x2_to_e4m3(fmul2(r.x[0][0], i2), fmul2(r.x[0][1], i2)), 0),
          make_uint2(f2x2_to_e4m3(fmul2(r.x[1][0], i2), fmul2(r.x[1][1], i2)), 0)};
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t bits) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)bits, __NV_E4M3)));
}
__device__ __forceinline__ RowPart unpack_e4m3(RowBits b, float scale) {
  RowPart r;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = (h ? b.hi.x : b.lo.x) >> (16 * i);
      r.x[h][i] = f2(e4m3_to_f32(u & 0xff) * scale, e4m3_to_f32((u >> 8) & 0xff) * scale);
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
// Both kernels are launched so that their blocks may be set up while the kernel
// before them on the stream drains; previous_done() waits for that kernel's end
// (and its writes) and precedes every access to global memory. Neither kernel lets the
// next one start before its own end. Back to back calls take 2 to 3 us less each (64
// sequences, window 4096: 93.4 -> 90.9 us, over e4m3 60.5 -> 57.4; 201 ragged rows 46.5
// -> 44.3; 65536 appended tokens 48.1 -> 45.9), replayed from a graph 0.3 to 0.7.
__device__ __forceinline__ void previous_done() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), int grid, int threads, int smem,
                              cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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
// slots of one head of one page, both halves. apart != 0 (e4m3): in place of the
// halves, this pool and the one `apart` bytes behind it. ok is cleared on failure.
CUtensorMap paged_tensor_map(const PagedCache& c, const void* pool, int box, long long apart,
                             bool* ok);

}  // namespace flint
