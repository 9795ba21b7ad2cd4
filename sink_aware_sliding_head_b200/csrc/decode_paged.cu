// decode_paged.cu - flint_attn_decode_paged: one new token per sequence over a
// paged KV cache.
//
// The definition is flint_attn_decode's (Flint layers page, nemo_automodel.
// components.models.flint.layers, FlintAttention.forward; the sink is one more
// softmax category with a zero value): the new key and value go into slot p =
// lens[b], and the new query sees slots max(0, p - W + 1) .. p plus the sink.
//
// Bound by HBM: a key costs 512 bytes of K and V (256 in e4m3) and feeds only
// the G query heads of its group, 2 G operations a byte.
//
//   * Work. The keys of all (sequence, KV head) pairs are laid end to end in
//     blocks of 64 positions and cut into one equal range per SM. A block of
//     threads walks its range as segments of one pair each; a segment that is a
//     whole pair writes its result, the others leave an unnormalised partial
//     (m, l, O) and the last of a pair's segments to finish joins them. The plan
//     is made on the device by every block (a scan over lens), so a captured
//     call follows its lengths and nothing but lens decides who sums what.
//   * Loads. One warp streams K and V of the range through a ring of shared
//     memory with TMA, across segment borders, so that the ring fills while the
//     other warps finish one segment and start the next. A tensor map in five
//     dimensions (64 channels, slot, channel half, head, page) takes any page,
//     head and token strides; a box is the largest power of two of slots that
//     divides the page, at most 64, so no box crosses a page.
//   * Math. Eight warps in two groups of four take the blocks in turn, 16 keys a
//     warp, on mma.sync m16n8k16 with FP32 accumulation. Eight query heads at a
//     time: S takes q as two 16-bit parts, hi in rows 0-7 and lo in rows 8-15 of
//     one A operand, so q keeps 16 bits of mantissa (22 over e4m3, whose
//     products run in fp16) and the LSE stays exact to ~1e-6. O^T += V^T P^T
//     has the heads as the MMA's N, and the P fragment that a lane holds is
//     already the B operand. P is rounded to 16 bits for that product only; the
//     row sums add the unrounded values. Over e4m3 the bytes become fp16 in
//     registers (exact), and the scales multiply S and O in FP32.
//   * The new token never goes through the cache: its score is formed from the
//     rounded row and enters when the warps of its segment are joined. Its row
//     is stored after the segment's last load has landed.
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace flint {

namespace {

constexpr int kBlk = 64;                     // positions per unit of work
constexpr int kMathWarps = 8;
constexpr int kMathThreads = 32 * kMathWarps;
constexpr int kThreads = kMathThreads + 32;  // + the loading warp
constexpr int kMergeRow = kHeadDim + 4;      // O, m, l (and two unused): rows stay 16-byte aligned
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;             // log2 units

// Shared memory: [ring | merge rows of the 8 warps (q rows before that) | Small].
// NG: query heads in groups of 8 (1: G <= 8, 2: G <= 16).
template <int NG, bool kF8>
struct Cfg {
  static constexpr int kRowBytes = kF8 ? kHeadDim : 2 * kHeadDim;
  static constexpr int kStageBytes = 2 * kBlk * kRowBytes;          // K, then V
  static constexpr int kMergeBytes = kMathWarps * 8 * NG * kMergeRow * 4;
  // Even: the two groups of warps take the blocks in turn, so each stage then
  // belongs to one group, which sees every phase of its barriers. With an odd
  // ring a group's parity wait could be two phases behind and pass too early.
  static constexpr int kStages = (NG == 1 ? 4 : 4) * (kF8 ? 2 : 1);
  static_assert(kStages % 2 == 0 && kStages <= 16, "see above");
  // P = 2^(s - m + bias): fp16 P starts at 2^-24, so its rows are lifted
  static constexpr float kBias = kF8 ? 6.f : 0.f;
};
struct Small {
  uint64_t full[16], empty[16];
  int bad[16];                               // the stage lacks a page
  float cs[kHeadDim / 2], sn[kHeadDim / 2];
  float knew[kHeadDim], vnew[kHeadDim];      // the new row as the cache stores it, times scale
  uint4 kbits[16], vbits[16];                // and its bits, a lane's channels each
  float snew[16];                            // its scores, log2 units
  long long scan[kThreads / 32], start_off;
  int start_b, no_page, abort_flag, last;
};
template <int NG, bool kF8>
constexpr int smem_bytes() {
  return Cfg<NG, kF8>::kStages * Cfg<NG, kF8>::kStageBytes + Cfg<NG, kF8>::kMergeBytes +
         (int)sizeof(Small) + 1024;
}

struct Args {
  PagedDecodeLaunch a;
  int box;                                   // slots per TMA box: 16, 32 or 64
  float scale_log2;
  int* counters;                             // [B * Hk], zero between calls
  float* part_ml;                            // [2 * blocks][16][2]
  float* part_o;                             // [2 * blocks][16][128]
};

// ------------------------------------------------------------------ the plan
struct Range {                               // what a row's new query reads of its cache
  int p, lo;                                 // cached positions lo .. p-1
  int first, n;                              // 64-position blocks; n = 0: nothing to do
};
__device__ __forceinline__ Range row_range(const PagedDecodeLaunch& a, int b) {
  Range r;
  r.p = __ldg(a.lens + b);
  r.lo = a.W > 0 ? max(0, r.p - a.W + 1) : 0;
  r.first = r.lo / kBlk;
  r.n = 0;
  if (r.p >= 0 && r.p < (long long)a.c.P * a.c.max_pages)
    r.n = r.p > r.lo ? (r.p - 1) / kBlk - r.first + 1 : 1;   // 1: only the new token
  return r;
}
// First unit of block i's range, and the block whose range holds unit u.
__device__ __forceinline__ long long range_begin(long long units, int i, int blocks) {
  return units * i / blocks;
}
__device__ __forceinline__ int range_of(long long units, long long u, int blocks) {
  return (int)(((u + 1) * blocks - 1) / units);
}

// The segments of one block's range, in order; the same for every thread.
struct Walk {
  int b;                                     // row
  long long off, left;                       // unit within the row's n * Hk; units left
  Range r;
  // the segment: KV head g, blocks blk .. blk + len - 1 of the pair's r.n
  int g, blk, len;
  __device__ bool next(const PagedDecodeLaunch& a, bool first) {
    if (!first) {
      off += len;
      left -= len;
      if (left == 0) return false;
      if (off == (long long)r.n * a.c.Hk) {
        off = 0;
        do r = row_range(a, ++b);            // ends: left > 0 units lie in later rows
        while (r.n == 0);
      }
    }
    g = (int)(off / r.n);
    blk = (int)(off - (long long)g * r.n);
    len = (int)min((long long)(r.n - blk), left);
    return true;
  }
};

// ------------------------------------------------------------------ small pieces
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int slot, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(slot), "r"(head), "r"(page)
      : "memory");
}
__device__ __forceinline__ void math_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kMathThreads) : "memory");
}
template <bool kF8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kF8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kTrans>
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// The four e4m3 bytes of a register as two fp16 pairs (exact): lo = bytes 0, 1.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(x));
}
// A 16-bit pair's hi part and the part left over.
template <bool kF8>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  if constexpr (kF8) {
    x0 = sat_f16(x0);
    x1 = sat_f16(x1);
    const __half2 h = __floats2half2_rn(x0, x1);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack_f16x2(x0 - __low2float(h), x1 - __high2float(h));
  } else {
    hi = pack_bf16x2(x0, x1);
    lo = pack_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
  }
}

// ------------------------------------------------------------------ the kernel
template <int NG, bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args A) {
  using C = Cfg<NG, kF8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  Small& sm = *reinterpret_cast<Small*>(smem + C::kStages * C::kStageBytes + C::kMergeBytes);
  const PagedDecodeLaunch& a = A.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), kMathWarps / 2);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  // ---- the plan: all units, and where this block's range begins
  long long units;
  int blocks;                                // that have a range: no range is empty
  Walk w;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const Range r = row_range(a, b);
      sum += r.n;
      if (r.n == 0 && r.p != -1 && blockIdx.x == 0) atomicOr(a.status, kStatusDecodeRange);
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    long long before = incl - sum, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sm.scan[i];
      total += sm.scan[i];
    }
    units = total * a.c.Hk;
    blocks = (int)min((long long)gridDim.x, units);
    const bool idle = (int)blockIdx.x >= blocks;
    const long long u0 = idle ? units : range_begin(units, blockIdx.x, blocks);
    w.left = idle ? 0 : range_begin(units, blockIdx.x + 1, blocks) - u0;
    long long at = u0 - before * a.c.Hk;
    if (at >= 0 && at < sum * a.c.Hk) {
      int b = b0;
      for (;; ++b) {                         // ends inside b0 .. b1-1: at < sum * Hk
        const long long n = (long long)row_range(a, b).n * a.c.Hk;
        if (at < n) break;
        at -= n;
      }
      sm.start_b = b;
      sm.start_off = at;
    }
    __syncthreads();
    if (w.left == 0) return;
    w.b = sm.start_b;
    w.off = sm.start_off;
    w.r = row_range(a, w.b);
  }
  const WaitCtx wc{&sm.abort_flag, a.status, kStatusTimeoutFwd};

  if (warp == kMathWarps) {
    // ---------------------------------------------------------------- loads
    const int nbox = kBlk / A.box;
    const uint32_t box_bytes = (uint32_t)A.box * C::kRowBytes;
    uint32_t n = 0;
    bool ok = true;
    for (bool more = w.next(a, true); more && ok; more = w.next(a, false)) {
      const int32_t* row = a.c.table + w.b * a.c.table_stride;
      // lane i < nbox holds the page of box i of the coming block
      auto page_of = [&](int blk) {
        const int pos = (w.r.first + blk) * kBlk + lane * A.box;
        const bool need = lane < nbox && pos + A.box > w.r.lo && pos < w.r.p;
        return need ? __ldg(row + pos / a.c.P) : -2;          // -2: no visible slot
      };
      int page = page_of(w.blk);
      for (int j = 0; j < w.len && ok; ++j, ++n) {
        const int cur = page;
        if (j + 1 < w.len) page = page_of(w.blk + j + 1);
        const int s = n % C::kStages;
        if (n >= C::kStages)
          ok = mbar_wait_warp(smem_u32(&sm.empty[s]), (n / C::kStages - 1) & 1, wc);
        if (!ok) break;
        const int pos = (w.r.first + w.blk + j) * kBlk + lane * A.box;
        const bool need = lane < nbox && pos + A.box > w.r.lo && pos < w.r.p;
        const bool good = need && (unsigned)cur < (unsigned)a.c.num_pages;
        const unsigned good_mask = __ballot_sync(0xffffffffu, good);
        const unsigned bad_mask = __ballot_sync(0xffffffffu, need && !good);
        const uint32_t full = smem_u32(&sm.full[s]);
        if (lane == 0) {
          sm.bad[s] = bad_mask != 0;
          if (bad_mask) atomicOr(a.status, kStatusDecodeRange);
          mbar_arrive_expect_tx(full, 2 * __popc(good_mask) * box_bytes);
        }
        __syncwarp();
        if (good) {
          const uint32_t dst = smem_u32(smem + s * C::kStageBytes) + lane * box_bytes;
          const int slot = pos % a.c.P;
          tma_load_5d(dst, &tm_k, full, slot, w.g, cur);
          tma_load_5d(dst + kBlk * C::kRowBytes, &tm_v, full, slot, w.g, cur);
        }
        __syncwarp();
      }
    }
    // Every copy has landed before the block can exit (immediate unless a wait
    // ran out: the math warps saw each one).
    volatile int no_abort = 0;
    const WaitCtx drain{&no_abort, a.status, kStatusTimeoutFwd};
    for (uint32_t i = n > C::kStages ? n - C::kStages : 0; i < n; ++i)
      mbar_wait_warp(smem_u32(&sm.full[i % C::kStages]), (i / C::kStages) & 1, drain);
    return;
  }

  // ------------------------------------------------------------------ math
  const int gid = lane >> 2, tig = lane & 3;
  const int half = threadIdx.x >> 4, l16 = threadIdx.x & 15;   // 16 half-warps
  const int group = warp >> 2;                                 // takes stages n % 2 == group
  const int key0 = 16 * (warp & 3);                            // of the block
  const uint32_t ring = smem_u32(smem);
  // the warp's 16 keys lie in one box (boxes have 16, 32 or 64 slots)
  const uint32_t key_base = (uint32_t)(key0 / A.box) * A.box * C::kRowBytes +
                            (uint32_t)(key0 % A.box) * 128;
  const uint32_t half_bytes = (uint32_t)A.box * 128;           // bf16: channels 64..127
  uint32_t n = 0;
  int last_b = -1;
  bool ok = true;

  for (bool more = w.next(a, true); more; more = w.next(a, false)) {
    const bool owner = w.blk + w.len == w.r.n;                 // this segment has the new token
    const int h0 = w.g * a.G;
    const float ks = kF8 && a.c.k_scale ? __ldg(a.c.k_scale + w.g) : 1.f;
    const float vs = kF8 && a.c.v_scale ? __ldg(a.c.v_scale + w.g) : 1.f;

    // ---- q rows (half-warps 0 .. G-1) and, in the last segment, the new row
    float x[8] = {}, wt[8] = {};
    uint4 uk{}, uv{}, uw{};
    const bool has_q = half < a.G;
    if (has_q) {
      load8(a.q + w.b * a.q_stride + (long long)(h0 + half) * kHeadDim + 8 * l16, x);
      load8(a.wq + 8 * l16, wt);
    }
    long long dst = 0;                                         // the new row's slot, -1: no page
    if (owner && warp == kMathWarps - 1) {                     // both half-warps the same row
      dst = slot_offset(a.c, w.b, w.r.p);
      uk = *reinterpret_cast<const uint4*>(a.k + w.b * a.k_stride + w.g * kHeadDim + 8 * l16);
      uv = *reinterpret_cast<const uint4*>(a.v + w.b * a.v_stride + w.g * kHeadDim + 8 * l16);
      uw = *reinterpret_cast<const uint4*>(a.wk + 8 * l16);
    }
    if (a.rope && w.b != last_b && threadIdx.x < kHeadDim / 2)
      rope_cos_sin(w.r.p, threadIdx.x, a.log2_theta, &sm.cs[threadIdx.x], &sm.sn[threadIdx.x]);
    last_b = w.b;
    math_sync();                                               // table; merge area free
    row_prologue(x, wt, sm.cs, sm.sn, a.rope, a.eps);
    float (*qs)[kHeadDim] = reinterpret_cast<float (*)[kHeadDim]>(merge);
    if (half < 8 * NG) {                                       // zero past G
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= A.scale_log2;
      *reinterpret_cast<float4*>(&qs[half][8 * l16]) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(&qs[half][8 * l16 + 4]) = make_float4(x[4], x[5], x[6], x[7]);
    }
    if (owner && warp == kMathWarps - 1) {
      float xk[8], xv[8], wk[8];
      unpack8(uk, xk);
      unpack8(uv, xv);
      unpack8(uw, wk);
      row_prologue(xk, wk, sm.cs, sm.sn, a.rope, a.eps);
      if (lane == 0) sm.no_page = dst < 0;
      if (lane < 16) {
        float rk[8], rv[8];
        if constexpr (kF8) {
          const uint2 bk = pack_e4m3_row(xk, ks), bv = pack_e4m3_row(xv, vs);
          sm.kbits[lane] = make_uint4(bk.x, bk.y, 0, 0);
          sm.vbits[lane] = make_uint4(bv.x, bv.y, 0, 0);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            rk[e] = e4m3_to_f32(((e < 4 ? bk.x : bk.y) >> (8 * (e & 3))) & 0xff) * ks;
            rv[e] = e4m3_to_f32(((e < 4 ? bv.x : bv.y) >> (8 * (e & 3))) & 0xff) * vs;
          }
        } else {
          sm.kbits[lane] = pack_bf16_row(xk);
          sm.vbits[lane] = uv;
          unpack8(sm.kbits[lane], rk);
          unpack8(uv, rv);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sm.knew[8 * l16 + e] = rk[e];
          sm.vnew[8 * l16 + e] = rv[e];
        }
      }
    }
    math_sync();

    // ---- A operand of S: rows 0-7 the hi parts, rows 8-15 the lo parts of 8 heads.
    // Over e4m3 a lane's four bytes of a 16-channel chunk are channels 4 tig ..,
    // so the chunk's channels are taken in that order by q as well.
    uint32_t qa[NG][8][4];
#pragma unroll
    for (int t = 0; t < NG; ++t)
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const float* q = qs[8 * t + gid] + 16 * kk;
        const float2 u = *reinterpret_cast<const float2*>(q + (kF8 ? 4 * tig : 2 * tig));
        const float2 v = *reinterpret_cast<const float2*>(q + (kF8 ? 4 * tig + 2 : 2 * tig + 8));
        split_pair<kF8>(u.x, u.y, qa[t][kk][0], qa[t][kk][1]);
        split_pair<kF8>(v.x, v.y, qa[t][kk][2], qa[t][kk][3]);
      }
    if (owner) {                                               // the new token's scores
      for (int h = warp; h < a.G; h += kMathWarps) {
        const float4 q = *reinterpret_cast<const float4*>(&qs[h][4 * lane]);
        const float4 k = *reinterpret_cast<const float4*>(&sm.knew[4 * lane]);
        float z = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) sm.snew[h] = z;
      }
    }
    math_sync();                                               // qs is free for the merge

    // ---- the segment's keys
    // o: O^T, 8 m-tiles of 16 channels x 8 heads; m (log2 units, less kBias) and
    // l of head gid (a lane's keys only until the end).
    float o[NG][8][4], m[NG], l[NG];
#pragma unroll
    for (int t = 0; t < NG; ++t) {
      m[t] = -INFINITY;
      l[t] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }
    for (int j = 0; j < w.len; ++j, ++n) {
      if ((n & 1) != (uint32_t)group) continue;
      const int s = n % C::kStages;
      if (ok) ok = mbar_wait_warp(smem_u32(&sm.full[s]), (n / C::kStages) & 1, wc);
      const int pos0 = (w.r.first + w.blk + j) * kBlk + key0;  // the warp's first key
      if (sm.bad[s]) {
#pragma unroll
        for (int t = 0; t < NG; ++t) l[t] = NAN;
      }
      if (pos0 < w.r.p && pos0 + 16 > w.r.lo) {
        const bool edge = pos0 < w.r.lo || pos0 + 16 > w.r.p;
        const uint32_t kst = ring + s * C::kStageBytes + key_base;
        const uint32_t vst = kst + kBlk * C::kRowBytes;
        // S of keys pos0 + 8 nt + 2 tig, + 1 for head gid: hi + lo parts
        float sc[NG][2][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float acc[NG][2][4];                               // even and odd steps apart
#pragma unroll
          for (int t = 0; t < NG; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              acc[t][h][0] = acc[t][h][1] = acc[t][h][2] = acc[t][h][3] = 0.f;
          const int key = nt * 8 + (lane & 7);
          if constexpr (kF8) {
#pragma unroll
            for (int kq = 0; kq < 2; ++kq) {                 // 64 channels
              uint32_t r[4];
              ldsm_x4<false>(kst + key * 128 + (((4 * kq + (lane >> 3)) ^ (lane & 7)) << 4), r);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                e4m3x4_to_f16(r[i], b0, b1);
#pragma unroll
                for (int t = 0; t < NG; ++t) mma16816<kF8>(acc[t][i & 1], qa[t][4 * kq + i], b0, b1);
              }
            }
          } else {
#pragma unroll
            for (int kp = 0; kp < 4; ++kp) {                 // 32 channels
              uint32_t r[4];
              ldsm_x4<false>(kst + (kp >> 1) * half_bytes + key * 128 +
                                 (((4 * (kp & 1) + (lane >> 3)) ^ (lane & 7)) << 4), r);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < NG; ++t)
                  mma16816<kF8>(acc[t][h], qa[t][2 * kp + h], r[2 * h], r[2 * h + 1]);
            }
          }
#pragma unroll
          for (int t = 0; t < NG; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sc[t][nt][e] = (acc[t][0][e] + acc[t][1][e]) + (acc[t][0][2 + e] + acc[t][1][2 + e]);
              if constexpr (kF8) sc[t][nt][e] *= ks;
            }
        }
        uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;         // V of keys outside the window: 0
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = pos0 + nt * 8 + 2 * tig + e;
              if (pos < w.r.lo || pos >= w.r.p) {
#pragma unroll
                for (int t = 0; t < NG; ++t) sc[t][nt][e] = -INFINITY;
                (nt ? vm1 : vm0) &= e ? 0x0000ffffu : 0xffff0000u;
              }
            }
        }
        uint32_t pb[NG][2];
#pragma unroll
        for (int t = 0; t < NG; ++t) {
          float mx = fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][1][0], sc[t][1][1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // lazy: the running max moves only when it grows by more than 2^8
          float alpha = 1.f;
          if (mx > m[t] + (C::kBias + kRescale)) {
            alpha = ex2_approx(m[t] - (mx - C::kBias));        // 0 from -inf
            m[t] = mx - C::kBias;
            l[t] *= alpha;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            // this lane's O^T columns are heads 2 tig and 2 tig + 1
            const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * tig);
            const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * tig + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[t][i][0] *= a0; o[t][i][1] *= a1; o[t][i][2] *= a0; o[t][i][3] *= a1;
            }
          }
          const float mb = m[t] == -INFINITY ? 0.f : m[t];
          const float p0 = ex2_approx(sc[t][0][0] - mb), p1 = ex2_approx(sc[t][0][1] - mb);
          const float p2 = ex2_approx(sc[t][1][0] - mb), p3 = ex2_approx(sc[t][1][1] - mb);
          l[t] += (p0 + p1) + (p2 + p3);
          pb[t][0] = kF8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          pb[t][1] = kF8 ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3);
        }
        if constexpr (kF8) {
          // ldmatrix on byte pairs: a lane gets channels 2 gid, 2 gid + 1 of keys
          // 2 tig, 2 tig + 1; rows gid and gid + 8 of the m-tile are those channels
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t r[4], av[2][4];
            const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
            ldsm_x4<true>(vst + key * 128 + (((2 * i + (lane >> 4)) ^ (lane & 7)) << 4), r);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              e4m3x4_to_f16(__byte_perm(r[2 * c], 0, 0x3120), av[c][0], av[c][1]);
              e4m3x4_to_f16(__byte_perm(r[2 * c + 1], 0, 0x3120), av[c][2], av[c][3]);
              if (edge) { av[c][0] &= vm0; av[c][1] &= vm0; av[c][2] &= vm1; av[c][3] &= vm1; }
#pragma unroll
              for (int t = 0; t < NG; ++t) mma16816<kF8>(o[t][2 * i + c], av[c], pb[t][0], pb[t][1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t av[4];
            const int key = (lane & 7) + ((lane >> 4) & 1) * 8;
            ldsm_x4<true>(vst + (i >> 2) * half_bytes + key * 128 +
                              (((2 * (i & 3) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4), av);
            if (edge) { av[0] &= vm0; av[1] &= vm0; av[2] &= vm1; av[3] &= vm1; }
#pragma unroll
            for (int t = 0; t < NG; ++t) mma16816<kF8>(o[t][i], av, pb[t][0], pb[t][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[s]));
    }

    // ---- join the warps
    {
      float* rows = merge + warp * 8 * NG * kMergeRow;
#pragma unroll
      for (int t = 0; t < NG; ++t) {
        l[t] += __shfl_xor_sync(0xffffffffu, l[t], 1);
        l[t] += __shfl_xor_sync(0xffffffffu, l[t], 2);
        if (tig == 0) {
          float* r = rows + (8 * t + gid) * kMergeRow;
          r[kHeadDim] = m[t];
          r[kHeadDim + 1] = l[t];
        }
        float* r0 = rows + (8 * t + 2 * tig) * kMergeRow;
        float* r1 = r0 + kMergeRow;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d0 = kF8 ? 16 * i + 2 * gid : 16 * i + gid, d1 = kF8 ? d0 + 1 : d0 + 8;
          r0[d0] = o[t][i][0];
          r1[d0] = o[t][i][1];
          r0[d1] = o[t][i][2];
          r1[d1] = o[t][i][3];
        }
      }
    }
    math_sync();                                               // all of the segment's loads seen
    const bool whole = w.len == w.r.n;
    const int slot = 2 * blockIdx.x + (w.blk == 0 ? 1 : 0);    // of a partial
    const bool no_page = owner && sm.no_page;
    for (int e = threadIdx.x; e < a.G * (kHeadDim / 4); e += kMathThreads) {
      const int r = e / (kHeadDim / 4), d = 4 * (e % (kHeadDim / 4));
      float M = owner ? sm.snew[r] : -INFINITY;
#pragma unroll
      for (int i = 0; i < kMathWarps; ++i)
        M = fmaxf(M, merge[(i * 8 * NG + r) * kMergeRow + kHeadDim]);
      const float s2 = whole ? __ldg(a.sink + h0 + r) * kLog2e : -INFINITY;
      M = fmaxf(M, s2);
      const float Mb = M == -INFINITY ? 0.f : M;
      float L = ex2_approx(s2 - Mb);
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kMathWarps; ++i) {
        const float* row = merge + (i * 8 * NG + r) * kMergeRow;
        const float f = ex2_approx(row[kHeadDim] - Mb);
        const float4 v = *reinterpret_cast<const float4*>(row + d);
        L += row[kHeadDim + 1] * f;
        O.x += v.x * f; O.y += v.y * f; O.z += v.z * f; O.w += v.w * f;
      }
      O.x *= vs; O.y *= vs; O.z *= vs; O.w *= vs;
      if (owner) {
        const float f = ex2_approx(sm.snew[r] - Mb);
        const float4 v = *reinterpret_cast<const float4*>(&sm.vnew[d]);
        L += no_page ? NAN : f;
        O.x += v.x * f; O.y += v.y * f; O.z += v.z * f; O.w += v.w * f;
      }
      if (whole) {
        const long long row = (long long)w.b * a.H + h0 + r;
        const float inv = 1.f / L;
        if (a.out_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kHeadDim + d) =
              make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kHeadDim + d) =
              make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
        if (d == 0) a.lse[row] = (M + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(A.part_o + ((long long)slot * 16 + r) * kHeadDim + d) = O;
        if (d == 0)
          *reinterpret_cast<float2*>(A.part_ml + ((long long)slot * 16 + r) * 2) =
              make_float2(M, L);
      }
    }
    if (owner && warp == kMathWarps - 1 && lane < 16 && !no_page) {
      const long long off = dst + w.g * a.c.head_stride;
      store_bits(a.c, a.c.k, off, sm.kbits[lane]);
      store_bits(a.c, a.c.v, off, sm.vbits[lane]);
    }
    if (no_page && threadIdx.x == 0) atomicOr(a.status, kStatusDecodeRange);
    if (whole) continue;

    // ---- the last of the pair's segments joins them and adds the sink
    const long long pair0 = range_begin(units, blockIdx.x, blocks);   // this range's first unit
    const long long u_seg = pair0 + (range_begin(units, blockIdx.x + 1, blocks) - pair0) - w.left;
    const long long u_pair = u_seg - w.blk;
    const int c0 = range_of(units, u_pair, blocks), c1 = range_of(units, u_pair + w.r.n - 1, blocks);
    __threadfence();
    math_sync();
    if (threadIdx.x == 0) {
      int* counter = A.counters + (long long)w.b * a.c.Hk + w.g;
      const int done = atomicAdd(counter, 1) == c1 - c0;
      if (done) *counter = 0;                                  // ready for the next call
      sm.last = done;
    }
    math_sync();
    if (!sm.last) continue;
    __threadfence();
    for (int e = threadIdx.x; e < a.G * (kHeadDim / 4); e += kMathThreads) {
      const int r = e / (kHeadDim / 4), d = 4 * (e % (kHeadDim / 4));
      const float s2 = __ldg(a.sink + h0 + r) * kLog2e;
      float M = s2;
#pragma unroll 8
      for (int c = c0; c <= c1; ++c)
        M = fmaxf(M, __ldcg(A.part_ml + ((2LL * c + (c == c0)) * 16 + r) * 2));
      const float Mb = M == -INFINITY ? 0.f : M;
      float L = ex2_approx(s2 - Mb);
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int c = c0; c <= c1; ++c) {
        const long long at = (2LL * c + (c == c0)) * 16 + r;
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(A.part_ml) + at);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(A.part_o + at * kHeadDim + d));
        const float f = ex2_approx(ml.x - Mb);
        L += ml.y * f;
        O.x += v.x * f; O.y += v.y * f; O.z += v.z * f; O.w += v.w * f;
      }
      const long long row = (long long)w.b * a.H + h0 + r;
      const float inv = 1.f / L;
      if (a.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kHeadDim + d) =
            make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kHeadDim + d) =
            make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
      if (d == 0) a.lse[row] = (M + log2f(L)) * kLn2;
    }
  }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

template <int NG, bool kF8>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Args& A, int grid,
                   cudaStream_t st) {
  static PerDeviceOnce once;
  constexpr int bytes = smem_bytes<NG, kF8>();
  static_assert(bytes <= 227 * 1024, "exceeds the shared memory of one block");
  cudaError_t e = smem_limit_once(once, decode_paged_kernel<NG, kF8>, bytes);
  if (e != cudaSuccess) return e;
  ProfScope prof(kKDecodePaged, st);
  decode_paged_kernel<NG, kF8><<<grid, kThreads, bytes, st>>>(tk, tv, A);
  return cudaGetLastError();
}

}  // namespace

// Workspace: [status int[64] | part_ml | part_o | counters]. Only the last
// region's size depends on the call, so that calls of any sizes leave the
// counters of all others at zero.
size_t decode_paged_bytes(int B, int Hk, int num_sms) {
  return 256 + round256((size_t)2 * num_sms * 16 * (2 + kHeadDim) * 4) +
         round256((size_t)B * Hk * 4);
}

cudaError_t launch_decode_paged(const PagedDecodeLaunch& a, int num_sms, cudaStream_t st) {
  Args A;
  A.a = a;
  A.box = a.c.P % 64 == 0 ? 64 : a.c.P % 32 == 0 ? 32 : 16;
  A.scale_log2 = a.scale * kLog2e;
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.status);
  const size_t rows = (size_t)2 * num_sms * 16;
  A.part_ml = reinterpret_cast<float*>(ws + 256);
  A.part_o = A.part_ml + rows * 2;
  A.counters = reinterpret_cast<int*>(ws + 256 + round256(rows * (2 + kHeadDim) * 4));
  bool ok = true;
  const CUtensorMap tk = paged_tensor_map(a.c, a.c.k, A.box, &ok);
  const CUtensorMap tv = paged_tensor_map(a.c, a.c.v, A.box, &ok);
  if (!ok) return cudaErrorInvalidValue;
  if (a.c.e4m3)
    return a.G <= 8 ? launch<1, true>(tk, tv, A, num_sms, st)
                    : launch<2, true>(tk, tv, A, num_sms, st);
  return a.G <= 8 ? launch<1, false>(tk, tv, A, num_sms, st)
                  : launch<2, false>(tk, tv, A, num_sms, st);
}

}  // namespace flint
