// decode_paged.cu - flint_attn_decode_paged: one new token per sequence over a
// paged KV cache.
//
// The definition is flint_attn_decode's (Flint layers page, nemo_automodel.
// components.models.flint.layers, FlintAttention.forward; the sink is one more
// softmax category with a zero value): the new key and value go into slot p =
// lens[b], and the new query sees slots max(0, p - W + 1) .. p plus the sink.
//
// Bound by HBM: a key costs 512 bytes of K and V (256 in e4m3) and feeds only
// the G query heads of its group with 512 G operations: G a byte (2 G in e4m3).
//
//   * Work. The keys of all (sequence, KV head) pairs are laid end to end in
//     blocks of 64 positions, each pair behind a few units of nothing that stand
//     for its fixed cost, and cut into one equal range per SM. A block of
//     threads walks its range as segments of one pair each; a segment that is a
//     whole pair writes its result, the others leave an unnormalised partial
//     (m, l, O) and the last of a pair's segments to finish joins them. The plan
//     is made on the device by every block (a scan over lens), so a captured
//     call follows its lengths and nothing but lens decides who sums what.
//   * Loads. Two warps stream K and V of the range, a block each in turn, through
//     a ring of shared memory with TMA, across segment borders, so that the ring
//     fills while the math warps finish one segment and start the next. A tensor
//     map in five dimensions (64 channels, slot, channel half, head, page) takes
//     any page, head and token strides; a box is the largest power of two of slots
//     that divides the page, at most 64, so no box crosses a page. Issuing a copy
//     costs a warp 130 cycles or more, so e4m3, whose rows need no halves, takes
//     that dimension for K and V and copies both at once (64 sequences, window
//     4096, 16-slot pages: 60.3 us with a copy each, 56.1 with one for both).
//   * Rows. With the rings of 148 SMs full, 24 MB are in flight (19 MB with 9 to 16
//     heads) and any load waits 3 to 4 us behind them. Two more warps
//     therefore fetch, normalise and rotate the q rows and the new row of the coming
//     segments, up to four ahead, and lay q out as the products take it.
//   * Math. Eight warps take the blocks in turn, 32 keys and eight query heads a
//     warp (up to 8 heads: four pairs of warps, a block each; 9 to 16: two groups
//     of four), on mma.sync m16n8k16 with FP32 accumulation: at G or 2 G operations
//     a byte the tensor pipe is a fifth busy over bf16 and a quarter over e4m3, and
//     the heads are too few rows for a tcgen05 tile. S takes q as two 16-bit parts,
//     hi in rows 0-7 and lo in rows 8-15 of one A operand. O^T += V^T P^T has the
//     heads as the MMA's N, and the P fragment that a lane holds is already the B
//     operand; P is a hi and a lo part as well. The row sums add the unrounded
//     values. Over e4m3 the bytes become fp16 in registers (exact), q and P are fp16,
//     and the scales multiply S and O in FP32.
//   * Precision. Two parts are 16 bits of q and P over bf16 and 22 over e4m3 (a power
//     of two lifts q there). A score is off by at most 2^-17 scale sum |q_i K_i| over
//     bf16 and 2^-22 over e4m3, beside FP32's own. Against 64 bits, with a float32
//     output (64 sequences, window 4096): the output by 3.9e-6 of its size over bf16
//     and 2.8e-7 over e4m3, the LSE by 6e-7 and 4e-7 (root mean squares; at most 2e-6
//     and 1e-6). With one part of P it was 2.0e-4 over e4m3 (and the kernel 2% faster),
//     and the error of a bf16 output rose by 1.4 over bf16. A third part of q and of P
//     over bf16 would be 1.9e-6 at 94.3 us for 89.6 and, with nine heads to a KV head,
//     56 us for 43: not taken, a bf16 output rounds by 1.7e-3.
//   * The new token never goes through the cache: its score is formed from the
//     rounded row and enters when the warps of its segment are joined. Its row
//     is stored after the segment's last load has landed.
//
// Measured (B200, 6.56 TB/s copy): 64 sequences of 4096 visible keys, 32 query and
// 4 KV heads, 89 us in bf16 (6.0 TB/s), 56 us in e4m3 (4.8 TB/s); four sequences
// near 131072 keys 142 us (6.6 TB/s; 154 on a slower card); one row of 230 keys 6.2 to
// 6.5 us. The fixed part is ~5 us: the plan, the first rows and pages (each a trip to
// HBM), and the join.
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace flint {

namespace {

constexpr int kBlk = 64;                     // positions per unit of work
constexpr int kKeys = 32;                    // of a block, per warp
constexpr int kMathWarps = 8;
constexpr int kLoadWarps = 2;                // block n is loaded by warp n % 2
constexpr int kRowWarps = 2;                 // four half-warps, a row each in turn
constexpr int kMathThreads = 32 * kMathWarps;
constexpr int kThreads = kMathThreads + 32 * (kLoadWarps + kRowWarps);
constexpr int kMergeRow = kHeadDim + 4;      // O, m, l (and two unused): rows stay 16-byte aligned
constexpr int kSegs = 4;                     // segments described ahead
constexpr int kLensKept = 512;               // rows whose lens a block keeps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;             // log2 units

// What the math warps need of a segment, made by the row warps.
template <int NG>
struct __align__(16) Seg {
  // A operand of S, 8 heads and 16 channels each: rows 0-7 the hi parts, rows
  // 8-15 the lo parts of the heads' q_hat, as the lanes hold it; times scale * log2(e)
  // over bf16, times q_lift over e4m3 (where ks brings S to log2 units)
  uint4 frag[NG * 8 * 32];
  float vnew[kHeadDim];                      // the new value as the cache stores it, times scale
  RowBits kbits[16], vbits[16];              // the new row as the cache stores it, by lane
  float snew[16];                            // the new token's scores, log2 units
  float sink[16], ks, vs;
  long long dst;                             // the new token's slot (KV head 0), -1: no page
  int b, g;
  int blk, len, n;                           // blocks blk .. blk + len - 1 of the pair's n
  int p, lo, first;                          // of the row, as in Range
  int c0, c1;                                // the ranges that share the pair
  int final;                                 // the range's last segment
};
constexpr int kMaxBars = 20;
struct Small {
  uint64_t full[kMaxBars], empty[kMaxBars], seg_full[kSegs], seg_empty[kSegs];
  int bad[kMaxBars];                         // the block lacks a page
  long long scan[kThreads / 32], start_off;
  int start_b, abort_flag, last[2];
  int lens[kLensKept];
};
// Shared memory: [ring | merge rows of the 8 warps | segments | Small].
// NG: query heads in groups of 8 (1: G <= 8, 2: G <= 16).
template <int NG, bool kF8>
struct Cfg {
  static constexpr int kRowBytes = kF8 ? kHeadDim : 2 * kHeadDim;
  static constexpr int kStageBytes = 2 * kBlk * kRowBytes;          // boxes of K and V rows
  // A pair's fixed cost in units. 201 rows of up to 2513 keys, nine heads to a KV
  // head, cost 0, 4, 8, 12: 49.3, 43.0, 44.9, 46.2 us in bf16, 51.0, 43.2, 45.3, 46.7
  // in e4m3; 250 rows of up to 900, eight heads: 73.4, 51.1, 53.2, 55.3 in bf16, 75.8,
  // 45.7, 45.4, 46.6 in e4m3 (whose blocks have half the bytes; 4 would do there, too).
  static constexpr int kCost = kF8 ? 8 : 4;
  static constexpr int kGroupWarps = 2 * NG, kGroups = kMathWarps / kGroupWarps;
  // Block u goes to stage u % kStages, to group u % kGroups, and has the barriers
  // u % kBars: a multiple of the stages, the groups and the loading warps, so each
  // barrier belongs to one group and one loading warp, which see every phase of
  // it. Were the barriers the stages', a parity wait of a group that does not
  // divide them could be two phases behind and pass early.
  static constexpr int kStages = (NG == 1 ? 5 : 4) * (kF8 ? 2 : 1);
  static constexpr int kBars = NG == 1 ? 20 : 8;
  static_assert(kBars % kStages == 0 && kBars % kGroups == 0 && kBars % kLoadWarps == 0 &&
                kBars <= kMaxBars, "see above");
  static constexpr int kMergeBytes = kMathWarps * 8 * kMergeRow * 4;
  static constexpr int kOffMerge = kStages * kStageBytes;
  static constexpr int kOffSegs = kOffMerge + kMergeBytes;
  static constexpr int kOffSmall = kOffSegs + kSegs * (int)sizeof(Seg<NG>);
  static constexpr int kSmemBytes = kOffSmall + (int)sizeof(Small) + 1024;   // + alignment
  // P = 2^(s - m + bias): fp16 P starts at 2^-24, so its rows are lifted
  static constexpr float kBias = kF8 ? 6.f : 0.f;
};

struct Args {
  PagedDecodeLaunch a;
  int box;                                   // slots per TMA box: 16, 32 or 64
  int joint, v_first;                        // one copy for K and V; V's rows lie before K's
  uint32_t page_mul, page_shift;             // pos / P = umulhi(pos, page_mul) >> page_shift
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
__device__ __forceinline__ Range row_range(const PagedDecodeLaunch& a, int p) {
  Range r;
  r.p = p;
  r.lo = a.W > 0 ? max(0, p - a.W + 1) : 0;
  r.first = r.lo / kBlk;
  r.n = 0;
  if (p >= 0 && p < (long long)a.c.P * a.c.max_pages)
    r.n = p > r.lo ? (p - 1) / kBlk - r.first + 1 : 1;   // 1: only the new token
  return r;
}
// (Quotients of numbers below 2^32 take the short division.)
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// The segments of one block's range, in order. A pair of n blocks is cost + n
// units; a segment is the blocks among a range's units of one pair.
struct Walk {
  int cost;
  int b, b0;                                 // row; the first whose lens is kept
  long long off, left;                       // unit within the row's (cost + n) * Hk; units left
  Range r;
  int g, blk, len;                           // the segment: KV head, blocks of the pair's r.n
  int units;                                 // of the pair in this range
  // false: nothing but a pair's fixed cost is left
  __device__ bool cut() {
    g = (int)quotient(off, cost + r.n);
    const int at = (int)(off - (long long)g * (cost + r.n));
    units = (int)min((long long)(cost + r.n - at), left);
    blk = max(0, at - cost);
    len = max(0, at + units - cost) - blk;
    return len > 0;
  }
  __device__ bool next(const PagedDecodeLaunch& a, const int* lens) {
    off += units;
    left -= units;
    if (left <= 0) return false;
    if (off == (long long)(cost + r.n) * a.c.Hk) {
      off = 0;
      do {                                   // ends: left > 0 units lie in later rows
        ++b;
        r = row_range(a, b - b0 < kLensKept ? lens[b - b0] : load(a.lens + b));
      } while (r.n == 0);
    }
    return cut();
  }
};

// ------------------------------------------------------------------ small pieces
__device__ __forceinline__ int page_col(const Args& A, int pos) {
  return (int)(__umulhi((uint32_t)pos, A.page_mul) >> A.page_shift);
}
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
__device__ __forceinline__ bool math_sync_and(bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"((int)x), "n"(kMathThreads) : "memory");
  return r != 0;
}
template <bool kF8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint4 a, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kF8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void add4(float (&x)[4], const float (&y)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    f2_split(fadd2(f2(x[e], x[e + 1]), f2(y[e], y[e + 1])), x[e], x[e + 1]);
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
// A 16-bit pair's hi part and the part left over (fp16: |x| below 65504).
template <bool kF8>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  if constexpr (kF8) {
    const __half2 h = __floats2half2_rn(x0, x1);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack_f16x2(x0 - __low2float(h), x1 - __high2float(h));
  } else {
    hi = pack_bf16x2(x0, x1);
    lo = pack_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
  }
}

// Over e4m3 q enters S in fp16, whose steps stop shrinking at 2^-24: it is lifted by
// the power of two 2^(11 - k), max|w_q| in 2^k .. 2^(k+1). |q_hat| <= sqrt(128) max|w_q|
// then lies below 2^15.6 (fp16 ends at 65504), and its two parts are off by 2^-22 of a
// channel or 2^-36 max|w_q|, whatever the weights, the cache's scales and softmax_scale
// (unlifted, weights of 2^-10 against key scales of 2^10 times the usual put the LSE off
// by 3e-5, and 2^-20 by 3e-2). Every lane of the half-warp gets it.
__device__ __forceinline__ float q_lift(const RowPart& w) {
  float m = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[4];
    w.get(h, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(x[e]));
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int exponent = 127 + 11 - ((__float_as_int(m) >> 23) - 127);
  return __int_as_float(min(max(exponent, 2), 252) << 23);   // its inverse is normal, too
}
__device__ __forceinline__ float inverse_of_power(float p) {
  return __int_as_float((254 << 23) - __float_as_int(p));
}

// Channels d .. d+3 of an output row from the joined sums, and its LSE once.
__device__ __forceinline__ void write_out(const PagedDecodeLaunch& a, long long row, int d,
                                          float4 O, float M, float L) {
  const float inv = 1.f / L;
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kHeadDim + d) =
        make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kHeadDim + d) =
        make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
  if (d == 0) a.lse[row] = (M + log2f(L)) * kLn2;
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
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  Seg<NG>* segs = reinterpret_cast<Seg<NG>*>(smem + C::kOffSegs);
  Small& sm = *reinterpret_cast<Small*>(smem + C::kOffSmall);
  const PagedDecodeLaunch& a = A.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == kMathThreads) {
    for (int s = 0; s < C::kBars; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), C::kGroupWarps);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(smem_u32(&sm.seg_full[s]), kRowWarps);
      mbar_init(smem_u32(&sm.seg_empty[s]), kMathWarps);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  previous_done();

  // ---- the plan: all units, and where this block's range begins
  Walk w;
  long long share, u0;                       // units a range; this one's first
  if (a.B == 1) {
    // One row's pairs are all alike: each gets ranges of its own, as many as
    // there are SMs for, but not below a block for each group of math warps
    // (those take as long as one: 230 keys take 8.7 us in four ranges a pair and
    // a join, 6.5 in one); the cost fills up a pair's first range.
    w.b = w.b0 = 0;
    w.r = row_range(a, load(a.lens));
    __syncthreads();
    const int n = w.r.n, most = (int)gridDim.x / a.c.Hk;
    if (n == 0) {
      if (w.r.p != -1 && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(a.status, kStatusDecodeRange);
      return;
    }
    if (most > 0) {
      const int ranges = min(most, (n + C::kGroups - 1) / C::kGroups);
      const int blocks = (n + ranges - 1) / ranges;
      share = blocks;
      w.cost = (n + blocks - 1) / blocks * blocks - n;
    } else {                                 // more KV heads than SMs: several pairs a range
      w.cost = C::kCost;
      share = (long long)(w.cost + n) * ((a.c.Hk + gridDim.x - 1) / gridDim.x);
    }
    const long long units = (long long)(w.cost + n) * a.c.Hk;
    u0 = share * blockIdx.x;
    w.off = u0;
    w.left = units - u0 < share ? units - u0 : share;
    if (w.left <= 0) return;
  } else {
    w.cost = C::kCost;
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int p = load(a.lens + b);
      const Range r = row_range(a, p);
      if (a.B <= kLensKept) sm.lens[b] = p;
      sum += r.n ? w.cost + r.n : 0;
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
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sm.scan[i];
      total += sm.scan[i];
    }
    const long long units = total * a.c.Hk;
    share = max(quotient(units + gridDim.x - 1, gridDim.x), (long long)(w.cost + C::kGroups));
    u0 = share * blockIdx.x;
    w.left = units - u0 < share ? units - u0 : share;
    if (w.left <= 0) return;
    long long at = u0 - before * a.c.Hk;
    if (at >= 0 && at < sum * a.c.Hk) {
      int b = b0;
      for (;; ++b) {                         // ends inside b0 .. b1-1: at < sum * Hk
        const int n = row_range(a, a.B <= kLensKept ? sm.lens[b] : load(a.lens + b)).n;
        const long long units_b = n ? (long long)(w.cost + n) * a.c.Hk : 0;
        if (at < units_b) break;
        at -= units_b;
      }
      sm.start_b = b;
      sm.start_off = at;
    }
    __syncthreads();
    if (a.B > kLensKept) {                   // the rows from the range's first
      for (int i = threadIdx.x; i < min(kLensKept, a.B - sm.start_b); i += kThreads)
        sm.lens[i] = load(a.lens + sm.start_b + i);
      __syncthreads();
    }
    w.b = sm.start_b;
    w.b0 = a.B > kLensKept ? w.b : 0;
    w.off = sm.start_off;
    w.r = row_range(a, sm.lens[w.b - w.b0]);
  }
  const long long u_end = u0 + w.left;
  if (!w.cut()) return;                      // not a block in this range
  const WaitCtx wc{&sm.abort_flag, a.status, kStatusTimeoutFwd};

  if (warp >= kMathWarps + kRowWarps) {
    // ---------------------------------------------------------------- loads
    const int nbox = kBlk / A.box;                             // 1, 2 or 4 boxes a block
    const uint32_t box_bytes = (uint32_t)A.box * C::kRowBytes;  // of K; a box has K's and V's rows
    const uint32_t lw = warp - kMathWarps - kRowWarps;         // takes blocks n % kLoadWarps == lw
    uint32_t n = 0, issued = 0;                                // issued: its last block + 1
    bool ok = true;
    // The table is read 32 boxes at a time and ahead: lane i holds the page and
    // slot of box at + i of a segment (-2: nothing visible; -1: a bad page).
    struct Box { int page, slot; };
    auto fetch = [&](const Walk& v, int at) {
      const int i = at + lane, pos = (v.r.first + v.blk) * kBlk + i * A.box;
      const bool need = i < v.len * nbox && pos + A.box > v.r.lo && pos < v.r.p;
      const int col = page_col(A, pos);
      const int32_t* row = a.c.table + v.b * a.c.table_stride;
      return Box{need ? max(load(row + col), -1) : -2, pos - col * a.c.P};
    };
    Box next = fetch(w, 0);
    while (true) {
      Walk nx = w;
      Box cur = next, ahead{};
      bool more = false, looked = false;
      auto look_ahead = [&] {                                  // after the first block's copies
        ahead = fetch(w, 32);
        more = nx.next(a, sm.lens);
        if (more) next = fetch(nx, 0);
        looked = true;
      };
      int batch = 0;
      for (int j = (int)((lw - n) & (kLoadWarps - 1)); j < w.len; j += kLoadWarps) {
        const int i = j * nbox;                                // the block's first box
        if (i / 32 != batch) {                                 // a turn has at most 8 boxes
          cur = ahead;
          ahead = fetch(w, 32 * (++batch + 1));
        }
        const uint32_t u = n + j;
        const int s = u % C::kStages, bar = u % C::kBars;
        if (u >= C::kStages) {                                 // the stage's last block is done
          const uint32_t d = u - C::kStages;
          ok = mbar_wait_warp(smem_u32(&sm.empty[d % C::kBars]), (d / C::kBars) & 1, wc);
        }
        if (!ok) break;
        issued = u + 1;
        const int page = __shfl_sync(0xffffffffu, cur.page, (i + lane) & 31);
        const int slot = __shfl_sync(0xffffffffu, cur.slot, (i + lane) & 31);
        const bool need = lane < nbox && page != -2;
        const bool good = need && (unsigned)page < (unsigned)a.c.num_pages;
        const unsigned good_mask = __ballot_sync(0xffffffffu, good);
        const unsigned bad_mask = __ballot_sync(0xffffffffu, need && !good);
        const uint32_t full = smem_u32(&sm.full[bar]);
        if (lane == 0) {
          sm.bad[bar] = bad_mask != 0;
          if (bad_mask) atomicOr(a.status, kStatusDecodeRange);
          mbar_arrive_expect_tx(full, 2 * __popc(good_mask) * box_bytes);
        }
        __syncwarp();
        if (good) {
          const uint32_t dst = smem_u32(smem + s * C::kStageBytes) + 2 * lane * box_bytes;
          tma_load_5d(dst, &tm_k, full, slot, w.g, page);      // joint: V's rows with it
          if (!A.joint) tma_load_5d(dst + box_bytes, &tm_v, full, slot, w.g, page);
        }
        __syncwarp();
        if (!looked) look_ahead();
      }
      if (!looked) look_ahead();
      n += w.len;
      if (!ok || !more) break;
      w = nx;
    }
    // Every copy has landed before the block can exit (immediate unless a wait
    // ran out: the math warps saw each one).
    volatile int no_abort = 0;
    const WaitCtx drain{&no_abort, a.status, kStatusTimeoutFwd};
    for (uint32_t u = issued > C::kStages ? issued - C::kStages : 0; u < issued; ++u)
      if (u % kLoadWarps == lw)
        mbar_wait_warp(smem_u32(&sm.full[u % C::kBars]), (u / C::kBars) & 1, drain);
    return;
  }

  if (warp >= kMathWarps) {
    // ---------------------------------------------------------------- rows
    const int hw = (threadIdx.x - kMathThreads) >> 4, l16 = lane & 15;   // half-warp, its lane
    constexpr int kHw = 2 * kRowWarps, kRows = 8 * NG / kHw;   // rows of a half-warp: hw + kHw i
    const bool lead = warp == kMathWarps;
    const RowPart wq = unpack_row(load_row(a.wq)), wk = unpack_row(load_row(a.wk));
    const float lift = kF8 ? q_lift(wq) : A.scale_log2;        // what q is multiplied by
    Angles angles{};
    double f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = rope_turns(4 * l16 + e, a.rope_pow);
    // What a segment takes from memory, requested one segment ahead.
    struct Raw { RowBits q[kRows], k, v; int page, slot; float sink, ks, vs; };
    auto look = [&](const Walk& v) {
      Raw h;
      const __nv_bfloat16* q = a.q + v.b * a.q_stride + (long long)v.g * a.G * kHeadDim;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = hw + kHw * i;
        h.q[i] = r < a.G ? load_row(q + r * kHeadDim) : RowBits{};
      }
      h.k = load_row(a.k + v.b * a.k_stride + v.g * kHeadDim);
      h.v = load_row(a.v + v.b * a.v_stride + v.g * kHeadDim);
      const int col = page_col(A, v.r.p);
      h.page = load(a.c.table + v.b * a.c.table_stride + col);
      h.slot = v.r.p - col * a.c.P;
      h.sink = lane < a.G ? load(a.sink + v.g * a.G + lane) : 0.f;
      h.ks = kF8 && a.c.k_scale ? load(a.c.k_scale + v.g) : 1.f;
      h.vs = kF8 && a.c.v_scale ? load(a.c.v_scale + v.g) : 1.f;
      return h;
    };
    Raw h = look(w);
    int last_b = -1;
    for (uint32_t k = 0;; ++k) {
      Walk nx = w;
      const bool more = nx.next(a, sm.lens);
      const Raw cur = h;
      if (more) h = look(nx);
      if (a.rope && w.b != last_b) angles = row_angles(w.r.p, f);
      last_b = w.b;
      Seg<NG>& sg = segs[k % kSegs];
      if (k >= kSegs &&
          !mbar_wait_warp(smem_u32(&sm.seg_empty[k % kSegs]), (k / kSegs - 1) & 1, wc))
        break;
      const bool owner = w.blk + w.len == w.r.n;
      // what brings a product of the lifted q and a stored key to log2 units
      const float s_scale = kF8 ? cur.ks * (inverse_of_power(lift) * A.scale_log2) : 1.f;
      RowPart kn{};                                            // as the cache stores it
      if (owner) {                                             // every half-warp the same row
        kn = unpack_row(cur.k);
        RowPart vn = unpack_row(cur.v);
        row_prologue(kn, wk, angles, a.rope, a.eps);
        RowBits kb, vb = cur.v;
        if constexpr (kF8) {
          kb = pack_e4m3(kn, inv_scale(a.c.k_scale, w.g));
          vb = pack_e4m3(vn, inv_scale(a.c.v_scale, w.g));
          kn = unpack_e4m3(kb, 1.f);                           // its scale goes into s_scale
          vn = unpack_e4m3(vb, cur.vs);
        } else {
          kb = pack_bf16(kn);
          kn = unpack_row(kb);
        }
        if (hw == 0) {
          sg.kbits[l16] = kb;
          sg.vbits[l16] = vb;
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2)
            *reinterpret_cast<ulonglong2*>(&sg.vnew[64 * h2 + 4 * l16]) =
                make_ulonglong2(vn.x[h2][0], vn.x[h2][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = hw + kHw * i;
        RowPart x = unpack_row(cur.q[i]);
        row_prologue(x, wq, angles, a.rope, a.eps);
        float z = 0.f, xs[2][4];
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          float kh[4];
          x.get(h2, xs[h2]);
          kn.get(h2, kh);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            xs[h2][e] = r < a.G ? xs[h2][e] * lift : 0.f;      // zero past G
            z += xs[h2][e] * kh[e];
          }
        }
        if (owner) {                                           // the new token's score
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
          if (l16 == 0) sg.snew[r] = z * s_scale;
        }
        // The lane's channels 4 l16 .. are a quarter of chunk l16 / 4 (and of chunk
        // l16 / 4 + 4). bf16: the lanes of head r (4 r + tig) hold channels 2 tig,
        // + 1 (x, y) and 2 tig + 8, + 9 (z, w) of a chunk. Over e4m3 a lane's four
        // bytes are channels 4 tig .., so q takes them in that order as well.
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t hi0, lo0, hi1, lo1;
          split_pair<kF8>(xs[h2][0], xs[h2][1], hi0, lo0);
          split_pair<kF8>(xs[h2][2], xs[h2][3], hi1, lo1);
          uint4* fr = sg.frag + ((r >> 3) * 8 + 4 * h2 + (l16 >> 2)) * 32 + 4 * (r & 7);
          if constexpr (kF8) {
            fr[l16 & 3] = make_uint4(hi0, lo0, hi1, lo1);
          } else {
            const int tig0 = 2 * (l16 & 1), zw = (l16 >> 1) & 1;
            reinterpret_cast<uint2*>(fr + tig0)[zw] = make_uint2(hi0, lo0);
            reinterpret_cast<uint2*>(fr + tig0 + 1)[zw] = make_uint2(hi1, lo1);
          }
        }
      }
      if (lead && lane < 16) sg.sink[lane] = cur.sink;
      if (lead && lane == 0) {
        sg.ks = s_scale;
        sg.vs = cur.vs;
        sg.dst = (unsigned)cur.page < (unsigned)a.c.num_pages
                     ? cur.page * a.c.page_stride + cur.slot * a.c.token_stride : -1;
        sg.b = w.b;
        sg.g = w.g;
        sg.blk = w.blk;
        sg.len = w.len;
        sg.n = w.r.n;
        sg.p = w.r.p;
        sg.lo = w.r.lo;
        sg.first = w.r.first;
        sg.final = !more;
        if (w.len < w.r.n) {
          // the pair's first and last block are units of these ranges
          const long long end = u_end - w.left + w.units;
          const long long last = end - 1 + (w.r.n - w.blk - w.len);
          sg.c0 = (int)quotient(last - (w.r.n - 1), share);
          sg.c1 = (int)quotient(last, share);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_full[k % kSegs]));
      if (!more) break;
      w = nx;
    }
    return;
  }

  // ------------------------------------------------------------------ math
  const int gid = lane >> 2, tig = lane & 3;
  const int group = warp / C::kGroupWarps;                     // takes blocks n % kGroups == group
  const int key0 = kKeys * (warp & 1);                         // of the block
  const int t8 = NG == 1 ? 0 : 8 * ((warp >> 1) & 1);          // the warp's first query head
  const uint32_t ring = smem_u32(smem);
  // 16 of the warp's keys lie in one box (boxes have 16, 32 or 64 slots)
  const uint32_t box_bytes = (uint32_t)A.box * C::kRowBytes;
  const uint32_t k_at = A.v_first ? box_bytes : 0, v_at = box_bytes - k_at;
  uint32_t chunk_at[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    chunk_at[c] = (uint32_t)((key0 + 16 * c) / A.box) * 2 * box_bytes +
                  (uint32_t)((key0 + 16 * c) % A.box) * 128;
  const uint32_t half_bytes = (uint32_t)A.box * 128;           // bf16: channels 64..127
  uint32_t n = 0;
  bool ok = true;
  // Partials, with their pair's ranges c0 .. c1: of a pair that began in an
  // earlier range (first), and of one that goes on in a later range (last).
  struct Part { int b, g, c0, c1; } first_part{-1, 0, 0, 0}, last_part{-1, 0, 0, 0};

  for (uint32_t k = 0;; ++k) {
    const Seg<NG>& sg = segs[k % kSegs];
    ok = mbar_wait_warp(smem_u32(&sm.seg_full[k % kSegs]), (k / kSegs) & 1, wc) && ok;
    // A segment is entered by all warps or none: len stays 0 where its wait ran out.
    const int len = ok ? sg.len : 0, p = sg.p, lo = sg.lo;
    const bool owner = sg.blk + sg.len == sg.n;                // this segment has the new token
    const float ks = sg.ks;
    uint4 qf[8];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) qf[kk] = sg.frag[(t8 + kk) * 32 + lane];

    // ---- the segment's keys
    // o: O^T, 8 m-tiles of 16 channels x 8 heads; m (log2 units, less kBias) and
    // l of head gid (a lane's keys only until the end).
    float o[8][4], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const int base = (sg.first + sg.blk) * kBlk + key0;
    for (int j = (int)((group - n) & (C::kGroups - 1)); j < len; j += C::kGroups) {
      const uint32_t u = n + j;
      const int s = u % C::kStages, bar = u % C::kBars;
      if (ok) ok = mbar_wait_warp(smem_u32(&sm.full[bar]), (u / C::kBars) & 1, wc);
      const int pos0 = base + j * kBlk;                        // the warp's first key
      if (sm.bad[bar]) l = NAN;
      if (pos0 < p && pos0 + kKeys > lo) {
        const bool edge = pos0 < lo || pos0 + kKeys > p;
        const uint32_t st = ring + s * C::kStageBytes + k_at;
        // S of keys pos0 + 8 nt + 2 tig, + 1 for head gid: hi + lo parts
        float sc[4][2];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float acc[2][4] = {};                              // even and odd steps apart
          const uint32_t kst = st + chunk_at[nt >> 1] + ((nt & 1) * 8 + (lane & 7)) * 128;
          if constexpr (kF8) {
#pragma unroll
            for (int kq = 0; kq < 2; ++kq) {                 // 64 channels
              uint32_t r[4];
              ldsm_x4<false>(kst + (((4 * kq + (lane >> 3)) ^ (lane & 7)) << 4), r);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                e4m3x4_to_f16(r[i], b0, b1);
                mma16816<kF8>(acc[i & 1], qf[4 * kq + i], b0, b1);
              }
            }
          } else {
#pragma unroll
            for (int kp = 0; kp < 4; ++kp) {                 // 32 channels
              uint32_t r[4];
              ldsm_x4<false>(kst + (kp >> 1) * half_bytes +
                                 (((4 * (kp & 1) + (lane >> 3)) ^ (lane & 7)) << 4), r);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                mma16816<kF8>(acc[h], qf[2 * kp + h], r[2 * h], r[2 * h + 1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sc[nt][e] = (acc[0][e] + acc[1][e]) + (acc[0][2 + e] + acc[1][2 + e]);
            if constexpr (kF8) sc[nt][e] *= ks;
          }
        }
        uint32_t vm[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (edge) {                                            // V of keys out of view: 0
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = pos0 + nt * 8 + 2 * tig + e;
              if (pos < lo || pos >= p) {
                sc[nt][e] = -INFINITY;
                vm[nt] &= e ? 0x0000ffffu : 0xffff0000u;
              }
            }
        }
        uint32_t pb[4], pl[4];                                 // P's hi and lo parts
        {
          float mx = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
          mx = fmaxf(mx, fmaxf(fmaxf(sc[2][0], sc[2][1]), fmaxf(sc[3][0], sc[3][1])));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // lazy: the running max moves only when it grows by more than 2^8
          float alpha = 1.f;
          if (mx > m + (C::kBias + kRescale)) {
            alpha = ex2_approx(m - (mx - C::kBias));        // 0 from -inf
            m = mx - C::kBias;
            l *= alpha;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            // this lane's O^T columns are heads 2 tig and 2 tig + 1
            const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * tig);
            const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * tig + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][0] *= a0; o[i][1] *= a1; o[i][2] *= a0; o[i][3] *= a1;
            }
          }
          const float mb = m == -INFINITY ? 0.f : m;
          float sum[4];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const float p0 = ex2_approx(sc[nt][0] - mb), p1 = ex2_approx(sc[nt][1] - mb);
            sum[nt] = p0 + p1;
            split_pair<kF8>(p0, p1, pb[nt], pl[nt]);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        const uint32_t vst = ring + s * C::kStageBytes + v_at;
        // The products of the block's 32 keys are summed on their own, then added to O: an
        // MMA cuts its sum off, toward zero, and a running O would be cut at every step. A
        // whole pair of 131072 keys in one range, values around one: O 8.2e-5 too small that
        // way, now within 2e-7; 64 rows of 4096 keys 89.1 us for 88.7, over e4m3 56.8 for
        // 54.5, 201 ragged rows with nine heads 43.3 for 41.1.
        if constexpr (kF8) {
          // ldmatrix on byte pairs: a lane gets channels 2 gid, 2 gid + 1 of keys
          // 2 tig, 2 tig + 1; rows gid and gid + 8 of the m-tile are those channels
          const uint32_t row = vst + ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float t[2][4] = {};
#pragma unroll
            for (int c = 0; c < 2; ++c) {                      // 16 keys
              uint32_t r[4];
              ldsm_x4<true>(row + chunk_at[c] + (((2 * i + (lane >> 4)) ^ (lane & 7)) << 4), r);
              uint4 av[2];
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                e4m3x4_to_f16(__byte_perm(r[2 * d], 0, 0x3120), av[d].x, av[d].y);
                e4m3x4_to_f16(__byte_perm(r[2 * d + 1], 0, 0x3120), av[d].z, av[d].w);
                if (edge) {
                  av[d].x &= vm[2 * c]; av[d].y &= vm[2 * c];
                  av[d].z &= vm[2 * c + 1]; av[d].w &= vm[2 * c + 1];
                }
                mma16816<kF8>(t[d], av[d], pb[2 * c], pb[2 * c + 1]);
              }
#pragma unroll
              for (int d = 0; d < 2; ++d)
                mma16816<kF8>(t[d], av[d], pl[2 * c], pl[2 * c + 1]);
            }
#pragma unroll
            for (int d = 0; d < 2; ++d) add4(o[2 * i + d], t[d]);
          }
        } else {
          const uint32_t row = vst + ((lane & 7) + ((lane >> 4) & 1) * 8) * 128;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float t[4] = {};
#pragma unroll
            for (int c = 0; c < 2; ++c) {                      // 16 keys
              uint32_t r[4];
              ldsm_x4<true>(row + chunk_at[c] + (i >> 2) * half_bytes +
                                (((2 * (i & 3) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4), r);
              uint4 av = make_uint4(r[0], r[1], r[2], r[3]);
              if (edge) {
                av.x &= vm[2 * c]; av.y &= vm[2 * c];
                av.z &= vm[2 * c + 1]; av.w &= vm[2 * c + 1];
              }
              mma16816<kF8>(t, av, pb[2 * c], pb[2 * c + 1]);
              mma16816<kF8>(t, av, pl[2 * c], pl[2 * c + 1]);
            }
            add4(o[i], t);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[bar]));
    }
    n += len;

    // ---- join the warps
    if (!math_sync_and(ok)) break;                             // the merge rows are free
    {
      float* rows = merge + warp * 8 * kMergeRow;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (tig == 0) {
        rows[gid * kMergeRow + kHeadDim] = m;
        rows[gid * kMergeRow + kHeadDim + 1] = l;
      }
      float* r0 = rows + 2 * tig * kMergeRow;
      float* r1 = r0 + kMergeRow;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d0 = kF8 ? 16 * i + 2 * gid : 16 * i + gid, d1 = kF8 ? d0 + 1 : d0 + 8;
        r0[d0] = o[i][0];
        r1[d0] = o[i][1];
        r0[d1] = o[i][2];
        r1[d1] = o[i][3];
      }
    }
    math_sync();                                               // all of the segment's loads seen
    const bool whole = len == sg.n;
    const int slot = 2 * blockIdx.x + (sg.blk == 0 ? 1 : 0);   // of a partial
    const bool no_page = owner && sg.dst < 0;
    for (int e = threadIdx.x; e < a.G * (kHeadDim / 4); e += kMathThreads) {
      const int r = e / (kHeadDim / 4), d = 4 * (e % (kHeadDim / 4));
      // the warps that have head r, as row r % 8 of theirs
      auto part = [&](int i) {
        const int wp = NG == 1 ? i : 4 * (i >> 1) + 2 * (r >> 3) + (i & 1);
        return merge + (wp * 8 + (r & 7)) * kMergeRow;
      };
      float M = owner ? sg.snew[r] : -INFINITY;
#pragma unroll
      for (int i = 0; i < kMathWarps / NG; ++i) M = fmaxf(M, part(i)[kHeadDim]);
      const float s2 = whole ? sg.sink[r] * kLog2e : -INFINITY;
      M = fmaxf(M, s2);
      const float Mb = M == -INFINITY ? 0.f : M;
      float L = ex2_approx(s2 - Mb);
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kMathWarps / NG; ++i) {
        const float* row = part(i);
        const float f = ex2_approx(row[kHeadDim] - Mb);
        const float4 v = *reinterpret_cast<const float4*>(row + d);
        L += row[kHeadDim + 1] * f;
        O.x += v.x * f; O.y += v.y * f; O.z += v.z * f; O.w += v.w * f;
      }
      if constexpr (kF8) {
        const float vs = sg.vs;
        O.x *= vs; O.y *= vs; O.z *= vs; O.w *= vs;
      }
      if (owner) {
        const float f = ex2_approx(sg.snew[r] - Mb);
        const float4 v = *reinterpret_cast<const float4*>(&sg.vnew[d]);
        L += no_page ? NAN : f;
        O.x += v.x * f; O.y += v.y * f; O.z += v.z * f; O.w += v.w * f;
      }
      if (whole) {
        write_out(a, (long long)sg.b * a.H + sg.g * a.G + r, d, O, M, L);
      } else {
        *reinterpret_cast<float4*>(A.part_o + ((long long)slot * 16 + r) * kHeadDim + d) = O;
        if (d == 0)
          *reinterpret_cast<float2*>(A.part_ml + ((long long)slot * 16 + r) * 2) =
              make_float2(M, L);
      }
    }
    if (owner && warp == kMathWarps - 1 && lane < 16 && !no_page) {
      const long long off = sg.dst + sg.g * a.c.head_stride;
      store_row<kF8>(a.c.k, off, sg.kbits[lane]);
      store_row<kF8>(a.c.v, off, sg.vbits[lane]);
    }
    if (no_page && threadIdx.x == 0) atomicOr(a.status, kStatusDecodeRange);
    if (!whole) {                                              // to be joined at the end
      const Part q{sg.b, sg.g, sg.c0, sg.c1};
      if (sg.blk == 0) last_part = q;
      else first_part = q;
    }
    const bool final = sg.final;
    __syncwarp();
    if (final) break;
    if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[k % kSegs]));
  }

  // ---- the last of a pair's segments to finish joins them and adds the sink.
  // Both of a block's partials (its range's first and last segment) are counted
  // here, after all of its loads, so that no join holds up the stream.
  if (first_part.b < 0 && last_part.b < 0) return;
  math_sync();                                                 // the partials are written
  if (threadIdx.x % (kMathThreads / 2) == 0) {                 // one thread for each partial
    const int i = threadIdx.x / (kMathThreads / 2);
    const Part q = i ? last_part : first_part;
    int last = 0;
    if (q.b >= 0) {
      int* counter = A.counters + (long long)q.b * a.c.Hk + q.g;
      int arrived;                                             // releases this block's partial,
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"   // acquires the others'
                   : "=r"(arrived) : "l"(counter) : "memory");
      if (arrived == q.c1 - q.c0) {
        *counter = 0;                                          // ready for the next call
        last = 1;
      }
    }
    sm.last[i] = last;
  }
  math_sync();
  // All warps join the one partial, or half of them each when both are due. A
  // warp takes a head: lane i weighs partial c + i, then all lanes add up O.
  const bool both = sm.last[0] && sm.last[1];
  if (!sm.last[0] && !sm.last[1]) return;
  const int part_warps = both ? kMathWarps / 2 : kMathWarps;
  const Part q = (both ? warp >= part_warps : sm.last[1]) ? last_part : first_part;
  for (int r = warp % part_warps; r < a.G; r += part_warps) {
    float M = load(a.sink + q.g * a.G + r) * kLog2e, L = 1.f;   // the sink first, then in order
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = q.c0; c <= q.c1; c += 32) {
      const int n = min(32, q.c1 - c + 1);
      auto at = [&](int i) { return (2LL * (c + i) + (c + i == q.c0)) * 16 + r; };
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = __ldcg(reinterpret_cast<const float2*>(A.part_ml) + at(lane));
      constexpr int kAtOnce = 16;                              // rows of O in flight
      float4 v[kAtOnce];
      auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (i0 + i < n)
            v[i] = __ldcg(reinterpret_cast<const float4*>(A.part_o + at(i0 + i) * kHeadDim) + lane);
      };
      fetch(0);
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(mx, M);
      const float mb = mx == -INFINITY ? 0.f : mx;
      const float f = ex2_approx(M - mb), t = ex2_approx(ml.x - mb);
      M = mx;
      float l = ml.y * t;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      L = L * f + l;
      O.x *= f; O.y *= f; O.z *= f; O.w *= f;
      for (int i0 = 0; i0 < n; i0 += kAtOnce) {
        if (i0) fetch(i0);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const float ti = __shfl_sync(0xffffffffu, t, (i0 + i) & 31);
          if (i0 + i < n) {
            O.x += v[i].x * ti; O.y += v[i].y * ti; O.z += v[i].z * ti; O.w += v[i].w * ti;
          }
        }
      }
    }
    write_out(a, (long long)q.b * a.H + q.g * a.G + r, 4 * lane, O, M, L);
  }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

template <int NG, bool kF8>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Args& A, int grid,
                   cudaStream_t st) {
  static PerDeviceOnce once;
  constexpr int bytes = Cfg<NG, kF8>::kSmemBytes;
  static_assert(bytes <= 227 * 1024, "exceeds the shared memory of one block");
  cudaError_t e = smem_limit_once(once, decode_paged_kernel<NG, kF8>, bytes);
  if (e != cudaSuccess) return e;
  ProfScope prof(kKDecodePaged, st);
  return launch_overlapped(decode_paged_kernel<NG, kF8>, grid, kThreads, bytes, st, tk, tv, A);
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
  // ceil(2^(31 + s) / P) with 2^s >= P gives exact quotients of numbers below 2^31
  uint32_t s = 0;
  while ((1u << s) < (uint32_t)a.c.P) ++s;
  A.page_mul = (uint32_t)(((1ull << (31 + s)) + a.c.P - 1) / a.c.P);
  A.page_shift = s - 1;
  A.scale_log2 = a.scale * kLog2e;
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.status);
  const size_t rows = (size_t)2 * num_sms * 16;
  A.part_ml = reinterpret_cast<float*>(ws + 256);
  A.part_o = A.part_ml + rows * 2;
  A.counters = reinterpret_cast<int*>(ws + 256 + round256(rows * (2 + kHeadDim) * 4));
  // The distance of the pools is a stride of the joint map (40 bits, not 0).
  const long long apart = static_cast<char*>(a.c.v) - static_cast<char*>(a.c.k);
  A.joint = a.c.e4m3 && apart != 0 && std::llabs(apart) < (1LL << 40);
  A.v_first = A.joint && apart < 0;
  bool ok = true;
  const CUtensorMap tk = paged_tensor_map(a.c, A.v_first ? a.c.v : a.c.k, A.box,
                                          A.joint ? std::llabs(apart) : 0, &ok);
  const CUtensorMap tv = A.joint ? tk : paged_tensor_map(a.c, a.c.v, A.box, 0, &ok);
  if (!ok) return cudaErrorInvalidValue;
  if (a.c.e4m3)
    return a.G <= 8 ? launch<1, true>(tk, tv, A, num_sms, st)
                    : launch<2, true>(tk, tv, A, num_sms, st);
  return a.G <= 8 ? launch<1, false>(tk, tv, A, num_sms, st)
                  : launch<2, false>(tk, tv, A, num_sms, st);
}

}  // namespace flint
