// decode_paged.cu - flint_attn_decode_paged: one new token per sequence over a
// paged KV cache.
//
// The definition is flint_attn_decode's (Flint layers page, nemo_automodel.
// components.models.flint.layers, FlintAttention.forward; the sink is one more
// softmax category with a zero value): the new key and value go into slot p =
// lens[b], and the new query sees slots max(0, p - W + 1) .. p plus the sink.
//
// One block per (KV head, sequence): each warp takes every eighth key, a lane
// four channels, in fp32; the warps' online softmaxes are joined at the end.
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace flint {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void load4(const PagedCache& c, const void* pool, long long off,
                                      float scale, float (&x)[4]) {
  if (c.e4m3) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pool) + off);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e4m3_to_f32((u >> (8 * e)) & 0xff) * scale;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(pool) + off);
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xffff0000u);
  }
}

__global__ void __launch_bounds__(kThreads) decode_paged_kernel(const PagedDecodeLaunch a) {
  __shared__ float cs[kHeadDim / 2], sn[kHeadDim / 2];
  __shared__ float qs[16][kHeadDim];
  __shared__ float part[kWarps][kHeadDim + 4];
  const int g = blockIdx.x, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int p = __ldg(a.lens + b);
  if (p == -1) return;
  if (p < 0 || p >= (long long)a.c.P * a.c.max_pages) {
    if (g == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusDecodeRange);
    return;
  }
  const int lo = a.W > 0 ? max(0, p - a.W + 1) : 0;
  const float ks = a.c.k_scale ? __ldg(a.c.k_scale + g) : 1.f;
  const float vs = a.c.v_scale ? __ldg(a.c.v_scale + g) : 1.f;
  if (a.rope && threadIdx.x < kHeadDim / 2)
    rope_cos_sin(p, threadIdx.x, a.log2_theta, &cs[threadIdx.x], &sn[threadIdx.x]);
  __syncthreads();
  {
    float x[8] = {}, w[8];
    load8(a.wq + 8 * l, w);
    if (grp < a.G) load8(a.q + b * a.q_stride + (g * a.G + grp) * kHeadDim + 8 * l, x);
    row_prologue(x, w, cs, sn, a.rope, a.eps);
    if (grp < a.G)
      for (int e = 0; e < 8; ++e) qs[grp][8 * l + e] = x[e] * a.scale * kLog2e;
  }
  if (warp == 0) {                                   // append (both halves the same row)
    const long long off = slot_offset(a.c, b, p);
    float x[8], y[8], w[8];
    load8(a.wk + 8 * l, w);
    load8(a.k + b * a.k_stride + g * kHeadDim + 8 * l, x);
    load8(a.v + b * a.v_stride + g * kHeadDim + 8 * l, y);
    row_prologue(x, w, cs, sn, a.rope, a.eps);
    if (off >= 0 && lane < 16) {
      store_row(a.c, a.c.k, off + g * a.c.head_stride, x, ks);
      store_row(a.c, a.c.v, off + g * a.c.head_stride, y, vs);
    }
  }
  __threadfence_block();
  __syncthreads();
  for (int r = 0; r < a.G; ++r) {
    float q[4];
    for (int e = 0; e < 4; ++e) q[e] = qs[r][4 * lane + e];
    float m = -INFINITY, sum = 0.f, o[4] = {};
    for (int j = lo + warp; j <= p; j += kWarps) {
      const long long off = slot_offset(a.c, b, j);
      if (off < 0) {                                 // no such page: the row becomes NaN
        if (lane == 0) atomicOr(a.status, kStatusDecodeRange);
        sum = NAN;
        continue;
      }
      float k[4], v[4];
      load4(a.c, a.c.k, off + g * a.c.head_stride + 4 * lane, ks, k);
      load4(a.c, a.c.v, off + g * a.c.head_stride + 4 * lane, vs, v);
      float z = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
      for (int d = 16; d >= 1; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
      const float mn = fmaxf(m, z), f = exp2f(m - mn), e = exp2f(z - mn);
      m = mn;
      sum = sum * f + e;
      for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * v[i];
    }
    for (int i = 0; i < 4; ++i) part[warp][4 * lane + i] = o[i];
    if (lane == 0) { part[warp][kHeadDim] = m; part[warp][kHeadDim + 1] = sum; }
    __syncthreads();
    if (warp == 0) {
      const float s2 = a.sink[g * a.G + r] * kLog2e;
      float M = s2;
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part[w][kHeadDim]);
      const float Mb = M == -INFINITY ? 0.f : M;
      float L = exp2f(s2 - Mb), O[4] = {};
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(part[w][kHeadDim] - Mb);
        L += part[w][kHeadDim + 1] * f;
        for (int i = 0; i < 4; ++i) O[i] += part[w][4 * lane + i] * f;
      }
      const long long row = (long long)b * a.H + g * a.G + r;
      const float inv = 1.f / L;
      if (a.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kHeadDim + 4 * lane) =
            make_float4(O[0] * inv, O[1] * inv, O[2] * inv, O[3] * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kHeadDim +
                                  4 * lane) =
            make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
      if (lane == 0) a.lse[row] = (M + log2f(L)) * kLn2;
    }
    __syncthreads();
  }
}

}  // namespace

size_t decode_paged_layout(int, int, int, void*) { return 256; }

cudaError_t launch_decode_paged(const PagedDecodeLaunch& a, cudaStream_t st) {
  ProfScope prof(kKDecodePaged, st);
  decode_paged_kernel<<<dim3(a.c.Hk, a.B), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace flint
