// Block-scaled FP8 (E4M3) matrix product of any size:
//   C[m,n] = sum_b sa[m,b] sb[n',b] sum_{k in block b} A[m,k] B[n,k]
// over blocks b of 128 along k, A with one fp32 scale per (row, block), B with one per
// (row, block) or per 128 rows and block (n' = n or n / 128).  A block's partial sum of code
// products is formed by the matrix cores and promoted as acc += partial * (sa * sb) in fp32.
// The codes of a row's last block past K are taken as zeros, whatever the pad holds.
//
// How a block's sum is formed goes by C's type (kWide):
//   bf16 C: the FP8 matrix instruction (16x16x128 f8f6f4, neutral E8M0 scales: the fp32 scales
//     are not powers of two), 5 PFLOP/s.  It aligns the 8 products of adjacent k to their
//     largest and keeps 13 bits below that one's leading bit (found by products of powers of
//     two: 2^16 + 2^3 is exact, 2^16 + 2^2 is not; across groups of 8 the sum has fp32's 24
//     bits).  On normally distributed codes that is 1.5e-5 of the result, a hundredth of
//     bf16's own rounding.
//   fp32 C (weight gradients): the codes are widened to bf16 in registers, exactly, and
//     multiplied by the bf16 instruction (32x32x16, 2.5 PFLOP/s), whose sums have 24 bits.
//     The FP8 instruction's 13 bits would be most of an fp32 result's error.
//
// k_fp8_tile: BM x BN outputs a workgroup of WM x WN waves, one block of k a step.  Codes and
// scales go from memory straight to a ring of LDS stages (buffer loads with the LDS
// destination bit; rows of 128 bytes, 16-byte chunks xor-swizzled by the row), rows past M or
// N arrive as zeros by the descriptor's range check.  B is the matrix instruction's first
// operand, so a lane's results lie in one row of C and take one activation scale.  Split over
// k (few tiles): fp32 partial sums to the workspace, k_fp8_join adds them in order.
//   bf16 C, 4096 x 4096 x 7168: 107-111 us, 2200 TFLOP/s, the matrix cores busy 49% of the cycles;
//   products with their promotions alone reach 3200 on random codes, by the card's power.
//   fp32 C, 2048 x 7168 x 4099, both operands scaled by the row: 152 us, 790 TFLOP/s, bound by the
//   vector unit (widening, two scales) and by 448 tiles on 256 CUs.
//   128 x 4096 x 7168: 14.5 + 4 us, 14 dependent steps and the join of four parts.
//   1 x 7168 x 2048 (k_fp8_rows): 5.5 us, launch and one round of loads.
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace moe {
namespace {

constexpr int GBK = 128;

typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

// byte of (row, 16-byte chunk c) in a stage
__device__ __forceinline__ int at128(int r, int c) { return r * GBK + ((c ^ (r >> 1)) & 7) * 16; }

__device__ __forceinline__ u32x4 lds16(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((uintptr_t)addr);
}
__device__ __forceinline__ bf16x8 widen8(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// The matrix instruction of each form and its lane layout.  A sub-tile has kT x kT outputs, kR
// of them a lane: of row `row` of A and columns col(i) of B.  A lane reads kC chunks of 16 codes
// of its row, chunk(i), of both operands (the same k meet in a product, whatever their order).
// kD sub-tiles are in flight (see the loop).
template <bool kWide>
struct Op;
template <>
struct Op<false> {
  static constexpr int kT = 16, kR = 4, kC = 2, kD = 4;
  typedef f32x4 Acc;
  struct Frag {
    i32x8 v;
  };
  static __device__ __forceinline__ int row(int lane) { return lane & 15; }
  static __device__ __forceinline__ int col(int lane, int i) { return 4 * (lane >> 4) + i; }
  static __device__ __forceinline__ int chunk(int lane, int i) { return (lane >> 4) + 4 * i; }
  static __device__ __forceinline__ Frag from(const u32x4 (&c)[kC]) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = (int)c[i >> 2][i & 3];
    return f;
  }
  static __device__ __forceinline__ Acc mul(const Frag& b, const Frag& a) {
    const Acc z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, z, 0, 0, 0, 127, 0, 127);
  }
};
template <>
struct Op<true> {
  static constexpr int kT = 32, kR = 16, kC = 4, kD = 2;
  typedef f32x16 Acc;
  struct Frag {
    bf16x8 v[8];
  };
  static __device__ __forceinline__ int row(int lane) { return lane & 31; }
  static __device__ __forceinline__ int col(int lane, int i) {
    return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
  }
  static __device__ __forceinline__ int chunk(int lane, int i) {
    return 4 * (i >> 1) + 2 * (lane >> 5) + (i & 1);
  }
  static __device__ __forceinline__ Frag from(const u32x4 (&c)[kC]) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f.v[i] = widen8((int)c[i >> 1][2 * (i & 1)], (int)c[i >> 1][2 * (i & 1) + 1]);
    return f;
  }
  static __device__ __forceinline__ Acc mul(const Frag& b, const Frag& a) {
    Acc t;
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[i], a.v[i], t, 0, 0, 0);
    return t;
  }
};

typedef const __attribute__((address_space(4))) float* ConstPtr;

struct GemmArgs {
  const uint8_t *a, *b;
  const float *sa, *sb;
  void* c;       // C, or the partial sums [splits, M, ldc] fp32
  int64_t lda, ldb, ldc, M, N, K;
  int mt, nt;    // tiles along M and N
  int splits, steps;  // k is cut into `splits` parts of `steps` blocks
  int c_f32, accumulate;
};

// 16 bytes of a row of C from v (8 bf16 or 4 fp32 values), n of its columns valid
__device__ __forceinline__ void store16(char* p, uint4 v, int n, bool f32, bool vec,
                                        bool accumulate) {
  if (f32) {
    float* q = reinterpret_cast<float*>(p);
    const float w[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                        __uint_as_float(v.w)};
    if (vec && n >= 4) {
      float4 o = make_float4(w[0], w[1], w[2], w[3]);
      if (accumulate) {
        const float4 c = *reinterpret_cast<const float4*>(q);
        o = make_float4(c.x + o.x, c.y + o.y, c.z + o.z, c.w + o.w);
      }
      *reinterpret_cast<float4*>(q) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) q[i] = accumulate ? q[i] + w[i] : w[i];
    }
  } else if (vec && n >= 8) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

template <int BM, int BN, int WM, int WN, int NST, bool kWide, bool kRowB>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_fp8_tile(GemmArgs g) {
  using O = Op<kWide>;
  constexpr int W = WM * WN, kT = O::kT, SM = BM / WM / kT, SN = BN / WN / kT;
  constexpr int kStage = (BM + BN) * GBK;
  // A's scales.  !kRowB: in chunks of kSc steps, 16 bytes of a row of scales at a time (a
  // step's alone, each lane's 4 bytes lie in a line of their own: 129 us at 4096 x 4096 x 7168
  // against 122), kG loads of 16 rows a chunk; a chunk's loads go out with the stages of the
  // chunk before it, from the stage on whose issue finds its buffer read for the last time, kL
  // a wave and stage.  kRowB: a step's with its stage, A's rows and then B's, because B's are
  // wanted four rows at a time, which a chunk's layout does not give (163 us at 2048 x 7168 x
  // 4099 against 192).
  constexpr int kSc = 4, kG = BM / 16;
  constexpr int kSlots = (kSc - (NST - 1)) * W, kL = kRowB ? 1 : (kG + kSlots - 1) / kSlots;
  constexpr int NA = BM / 8 / W, NB = BN / 8 / W, kPer = NA + NB + kL;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0, "whole load instructions");
  static_assert(W * 32 * (BN / WN) * 4 <= NST * kStage, "output staging fits the ring");
  __shared__ __attribute__((aligned(1024))) char smem[NST * kStage];
  // !kRowB: [2][BM * kSc], the scale of (row r, step k of the chunk) at r * kSc +
  // (k ^ (r / 16)) % kSc; kRowB: [NST][BM + BN]
  constexpr int kScBuf = kRowB ? BM + BN : BM * kSc;
  __shared__ __attribute__((aligned(16))) float s_sc[kRowB ? NST : 2][kScBuf];
  // tiles in bands of 8 row tiles, column-major inside a band, one contiguous range per XCD
  const int total = g.mt * g.nt * g.splits;
  const int per = (total + kXcds - 1) / kXcds;
  const int work = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
  if (blockIdx.x / kXcds >= per || work >= total) return;
  const int part = work / (g.mt * g.nt), tile = work % (g.mt * g.nt);
  constexpr int kBand = 8;
  const int band = tile / (kBand * g.nt), within = tile % (kBand * g.nt);
  const int rb = min(kBand, g.mt - band * kBand);
  const int64_t m0 = (int64_t)(band * kBand + within % rb) * BM, n0 = (int64_t)(within / rb) * BN;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv / WN, wn = wv % WN, fr = O::row(lane);
  const int nk = (int)((g.K + GBK - 1) / GBK);
  const int k0 = part * g.steps, k1 = min(k0 + g.steps, nk);
  const int m_rows = (int)min((int64_t)BM, g.M - m0), n_rows = (int)min((int64_t)BN, g.N - n0);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const uint32_t lds_sc = __builtin_amdgcn_readfirstlane(lds_offset(&s_sc[0][0]));
  // a tile's last row ends with its codes: there may be no memory behind it
  const int64_t k16 = (g.K + 15) / 16 * 16;
  const i32x4 ar = buffer_rsrc(g.a + m0 * g.lda, (uint32_t)((m_rows - 1) * g.lda + k16));
  const i32x4 br = buffer_rsrc(g.b + n0 * g.ldb, (uint32_t)((n_rows - 1) * g.ldb + k16));
  // instruction i of wave wv fills rows 8 (i W + wv) .. +7 of the stage (A's, then B's)
  const int lrow = 8 * wv + (lane >> 3);
  const int lchunk = (lane & 7) ^ ((4 * (wv & 1) + (lane >> 4)) & 7);
  uint32_t ao[NA], bo[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) ao[i] = (uint32_t)((8 * W * i + lrow) * g.lda) + 16 * lchunk;
#pragma unroll
  for (int i = 0; i < NB; ++i) bo[i] = (uint32_t)((8 * W * i + lrow) * g.ldb) + 16 * lchunk;
  const i32x4 sar = buffer_rsrc(g.sa + m0 * nk, (uint32_t)(m_rows * (int64_t)nk * 4));
  const i32x4 sbr = buffer_rsrc(g.sb + (kRowB ? n0 * nk : 0),
                                kRowB ? (uint32_t)(n_rows * (int64_t)nk * 4) : 0u);
  // !kRowB: scales of rows 16 q .. +15 of A for chunk c
  auto chunk = [&](int c, int q) {
    const int k = k0 + kSc * c + ((lane ^ q) & 3);
    load4_to_lds(sar, lds_sc + ((c & 1) * kScBuf + 64 * q) * 4,
                 (uint32_t)((16 * q + (lane >> 2)) * nk + k) * 4);
  };
  // load instruction i (of kPer) of a wave for step kt's stage
  auto load = [&](int kt, int st, int i) {
    const uint32_t dst = lds0 + st * kStage + 8 * wv * GBK, ko = (uint32_t)kt * GBK;
    if (i < NA) {
      load16_to_lds(ar, dst + i * 8 * W * GBK, ao[i] + ko);
    } else if (i < NA + NB) {
      load16_to_lds(br, dst + (BM + (i - NA) * 8 * W) * GBK, bo[i < NA + NB ? i - NA : 0] + ko);
    } else if (kRowB) {  // 64 rows' scales a wave; waves past the last repeat a group
      const int q = wv % ((BM + BN) / 64);
      const int row = 64 * (q < BM / 64 ? q : q - BM / 64) + lane;
      load4_to_lds(q < BM / 64 ? sar : sbr, lds_sc + (st * kScBuf + 64 * q) * 4,
                   (uint32_t)(row * nk + kt) * 4);
    } else {
      const int c = (kt - k0) / kSc, at = (kt - k0) % kSc - (NST - 1);
      const int q = (at * W + wv) * kL + i - NA - NB;
      // nothing of the next chunk to load: one of its own again (every wave's count of loads in
      // flight stays the same)
      const bool ahead = at >= 0 && q < kG;
      chunk(ahead ? c + 1 : c, ahead ? q : wv % kG);
    }
  };
  auto stage = [&](int kt, int st) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) load(kt, st, i);
  };
  // !kRowB: the scales of the wave's 128-row block (the last one where the wave is past N)
  // read through the constant address space: as scalar loads they stay out of the count of
  // vector loads in flight (as vector loads, each step waited for its own: 2 us a step)
  const ConstPtr sbp =
      (ConstPtr)(uintptr_t)(g.sb + min((n0 + wn * (BN / WN)) / 128, (g.N - 1) / 128) * nk);

  // this lane's chunks of its row, the same in every sub-tile (the swizzle repeats every 16
  // rows)
  uint32_t off[O::kC];
#pragma unroll
  for (int i = 0; i < O::kC; ++i) off[i] = (uint32_t)at128(fr, O::chunk(lane, i));
  auto codes = [&](uint32_t base, u32x4 (&c)[O::kC]) {
#pragma unroll
    for (int i = 0; i < O::kC; ++i) c[i] = lds16(off[i] + base);
  };

  typename O::Acc acc[SM][SN];
#pragma unroll
  for (int m = 0; m < SM; ++m)
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int i = 0; i < O::kR; ++i) acc[m][n][i] = 0.0f;

  if (!kRowB)
    for (int q = wv; q < kG; q += W) chunk(0, q);
#pragma unroll
  for (int j = 0; j < NST - 1; ++j) stage(k0 + j, j);
  constexpr int kIssue = SM * SN / 2 > 0 ? SM * SN / 2 : 1;
  int st = 0;
  float sw_next = kRowB ? 1.0f : sbp[k0];
  for (int kt = k0; kt < k1; ++kt) {
    const float sw = sw_next;
    wait_vm<(NST - 2) * kPer>();
    __syncthreads();
    // the loads of step kt + NST - 1 go out between the products below, over the first
    // kIssue sub-tiles: all at once they hold the waves up for 800 cycles of 4600, the time
    // that a CU takes to fetch 64 KiB (past the last step they fetch what nothing reads)
    const int kt_ld = kt + NST - 1, st_ld = st == 0 ? NST - 1 : st - 1;
    if (kt == nk - 1 && (g.K & (GBK - 1))) {  // the last block's codes past K
      const int left = (int)(g.K & (GBK - 1));
      for (int q = tid; q < (BM + BN) * 8; q += 64 * W) {
        const int n = left - 16 * (q & 7);
        if (n >= 16) continue;
        uint4* p = reinterpret_cast<uint4*>(smem + st * kStage + at128(q >> 3, q & 7));
        uint32_t w[4] = {0, 0, 0, 0};
        if (n > 0) {
          const uint4 v = *p;
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = n >= 4 * i + 4 ? u[i] : n > 4 * i ? u[i] & ((1u << (8 * (n - 4 * i))) - 1u) : 0u;
        }
        *p = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncthreads();
    }
    if (!kRowB) sw_next = sbp[min(kt + 1, nk - 1)];
    // The sub-tiles in a software pipeline: while the matrix cores form sub-tile j's partial
    // sum, the vector unit promotes that of sub-tile j - kD + 1 and the codes of the next column
    // group come from LDS.  (Left to the compiler, each promotion waited for its own products
    // and each product for its LDS reads.)
    const uint32_t a_at = lds0 + st * kStage + wm * (BM / WM) * GBK;
    const uint32_t b_at = lds0 + st * kStage + (BM + wn * (BN / WN)) * GBK;
    const int kr = kt - k0;
    const float* sc = s_sc[kRowB ? st : (kr / kSc) & 1];
    typename O::Frag fa[SM], fb;
    u32x4 next[O::kC];
    float sa[SM];
    codes(b_at, next);
#pragma unroll
    for (int m = 0; m < SM; ++m) {
      u32x4 c[O::kC];
      codes(a_at + kT * m * GBK, c);
      fa[m] = O::from(c);
    }
#pragma unroll
    for (int m = 0; m < SM; ++m) {
      const int r = wm * (BM / WM) + kT * m + fr;
      sa[m] = kRowB ? sc[r] : sc[r * kSc + ((kr ^ (r >> 4)) & 3)] * sw;
    }
    typename O::Acc t[O::kD];
    auto promote = [&](int j) {
      const int m = j % SM, n = j / SM;
#pragma unroll
      for (int q = 0; q < O::kR / 4; ++q) {
        float4 sb = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        if (kRowB)
          sb = *reinterpret_cast<const float4*>(
              sc + BM + wn * (BN / WN) + kT * n + O::col(lane, 4 * q));
        const float s[4] = {sb.x, sb.y, sb.z, sb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[m][n][4 * q + i] = __builtin_fmaf(t[j % O::kD][4 * q + i],
                                                kRowB ? sa[m] * s[i] : sa[m], acc[m][n][4 * q + i]);
      }
    };
#pragma unroll
    for (int j = 0; j < SM * SN; ++j) {
      const int m = j % SM, n = j / SM;
      if (m == 0) {
        fb = O::from(next);
        if (n + 1 < SN) codes(b_at + kT * (n + 1) * GBK, next);
      }
      t[j % O::kD] = O::mul(fb, fa[m]);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * kIssue / kPer == j) load(kt_ld, st_ld, i);
      if (j >= O::kD - 1) promote(j - (O::kD - 1));
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = SM * SN - (O::kD - 1); j < SM * SN; ++j) promote(j);
    if (++st == NST) st = 0;
  }
  wait_vm<0>();
  __syncthreads();  // every wave is done with the ring, which now stages the output

  // a wave's kT x (BN/WN) outputs of sub-tile row m in LDS (16-byte chunks swizzled by the
  // row), stored back 16 bytes a lane along the rows
  auto store = [&](auto is_f32) {
    constexpr bool f32 = decltype(is_f32)::value;
    constexpr int es = f32 ? 4 : 2, kCols = BN / WN, row_bytes = kCols * es;
    constexpr int chunks = row_bytes / 16, mask = (chunks < 16 ? chunks : 16) - 1;
    char* stg = smem + wv * kT * kCols * 4;
    char* out = static_cast<char*>(g.c) + (g.splits > 1 ? (int64_t)part * g.M * g.ldc * 4 : 0);
    const bool vec = g.ldc * es % 16 == 0;
    const bool add = g.accumulate && g.splits == 1;
#pragma unroll
    for (int m = 0; m < SM; ++m) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int n = 0; n < SN; ++n)
#pragma unroll
        for (int q = 0; q < O::kR / 4; ++q) {
          const auto& a = acc[m][n];
          const int col = kT * n + O::col(lane, 4 * q);  // 4 adjacent columns
          char* p = stg + fr * row_bytes + (((col * es / 16) ^ (fr & mask)) << 4);
          if (f32)
            *reinterpret_cast<float4*>(p) =
                make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
          else
            *reinterpret_cast<uint2*>(p + (col & 4) * 2) =
                pack4_bf16(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int64_t row0 = m0 + wm * (BM / WM) + kT * m;
#pragma unroll
      for (int e0 = 0; e0 < kT * chunks; e0 += 64) {
        const int r = (e0 + lane) / chunks, ch = (e0 + lane) % chunks;
        const int64_t n = n0 + wn * kCols + ch * (16 / es);
        const uint4 v =
            *reinterpret_cast<const uint4*>(stg + r * row_bytes + ((ch ^ (r & mask)) << 4));
        if (row0 + r < g.M && n < g.N)
          store16(out + ((row0 + r) * g.ldc + n) * es, v, (int)min((int64_t)8, g.N - n), f32, vec,
                  add);
      }
    }
  };
  if (kWide || g.splits > 1) store(std::true_type());
  else store(std::false_type());
}

// Few rows: a workgroup takes 16 columns and every row of A, its 8 waves every 8th block of k
// each, with the codes of kU blocks on their way from memory straight into registers, and they
// add their sums in LDS, in order.  B is read once in all, A once a workgroup (from the L2): the
// form is bound by B's bytes, or by latency, until A's rows weigh more.  B is the first
// operand of the 16 x 16 products: a lane holds row l%16 of A and columns 4 (l/16) .. +3 of B,
// and chunks l/16 and l/16 + 4 of a row's block of codes.
template <bool kWide>
__device__ __forceinline__ f32x4 mul16(const u32x4 (&b)[2], const u32x4 (&a)[2]) {
  f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (kWide) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          widen8((int)b[i >> 1][2 * (i & 1)], (int)b[i >> 1][2 * (i & 1) + 1]),
          widen8((int)a[i >> 1][2 * (i & 1)], (int)a[i >> 1][2 * (i & 1) + 1]), t, 0, 0, 0);
  } else {
    i32x8 x, y;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = (int)b[i >> 2][i & 3];
      y[i] = (int)a[i >> 2][i & 3];
    }
    t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, t, 0, 0, 0, 127, 0, 127);
  }
  return t;
}

// 16 codes at k of a row of K, zeros past K
__device__ __forceinline__ u32x4 codes_at(const uint8_t* __restrict__ row, int64_t k, int64_t K) {
  u32x4 v = {0, 0, 0, 0};
  if (k >= K) return v;
  v = *reinterpret_cast<const u32x4*>(row + k);
  const int n = (int)min((int64_t)16, K - k);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n < 4 * i + 4) v[i] = n > 4 * i ? v[i] & ((1u << (8 * (n - 4 * i))) - 1u) : 0u;
  return v;
}

template <int MG, int kU, bool kWide, bool kRowB>
__global__ __launch_bounds__(512) void k_fp8_rows(GemmArgs g) {
  constexpr int kW = 8, kM = 16 * MG;
  __shared__ float s_sum[kW][kM][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int nk = (int)((g.K + GBK - 1) / GBK), whole = (int)(g.K / GBK);
  // rows past M or N repeat the last one (their results are not stored)
  const uint8_t* ap[MG];
  const float *sap[MG], *sbp[4];
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    const int64_t row = min((int64_t)16 * m + r, g.M - 1);
    ap[m] = g.a + row * g.lda + 16 * q;
    sap[m] = g.sa + row * nk;
  }
  const uint8_t* bp = g.b + min(n0 + r, g.N - 1) * g.ldb + 16 * q;
#pragma unroll
  for (int i = 0; i < 4; ++i) sbp[i] = g.sb + min(n0 + 4 * q + i, g.N - 1) * (kRowB ? nk : 0);
  const ConstPtr sbu = (ConstPtr)(uintptr_t)(g.sb + n0 / 128 * nk);  // !kRowB
  struct Block {
    u32x4 a[MG][2], b[2];
    float sa[MG], sb[4];
  };
  auto scales = [&](Block& v, int blk) {
#pragma unroll
    for (int m = 0; m < MG; ++m) v.sa[m] = sap[m][blk];
#pragma unroll
    for (int i = 0; i < 4; ++i) v.sb[i] = kRowB ? sbp[i][blk] : i ? v.sb[0] : sbu[blk];
  };
  auto load = [&](Block& v, int blk) {  // a whole block
    const int64_t k = (int64_t)blk * GBK;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v.b[h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(bp + k + 64 * h));
#pragma unroll
      for (int m = 0; m < MG; ++m) v.a[m][h] = *reinterpret_cast<const u32x4*>(ap[m] + k + 64 * h);
    }
    scales(v, blk);
  };
  f32x4 acc[MG];
#pragma unroll
  for (int m = 0; m < MG; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const Block& v) {
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      const f32x4 t = mul16<kWide>(v.b, v.a[m]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[m][i] = __builtin_fmaf(t[i], v.sa[m] * v.sb[i], acc[m][i]);
    }
  };
  Block v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (wv + kW * u < whole) load(v[u], wv + kW * u);
  for (int b = wv; b < whole; b += kW * kU)
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int blk = b + kW * u;
      if (blk >= whole) break;
      add(v[u]);
      if (blk + kW * kU < whole) load(v[u], blk + kW * kU);
    }
  if (whole < nk && whole % kW == wv) {  // the last, partial block
    const int64_t k = (int64_t)whole * GBK, left = g.K - k - 16 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[0].b[h] = codes_at(bp + k, 64 * h, left);
#pragma unroll
      for (int m = 0; m < MG; ++m) v[0].a[m][h] = codes_at(ap[m] + k, 64 * h, left);
    }
    scales(v[0], whole);
    add(v[0]);
  }
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[wv][16 * m + r][4 * q + i] = acc[m][i];
  __syncthreads();
  for (int e = tid; e < kM * 16; e += 512) {
    const int m = e >> 4, n = e & 15;
    if (m >= g.M || n0 + n >= g.N) continue;
    float s = s_sum[0][m][n];
#pragma unroll
    for (int w = 1; w < kW; ++w) s += s_sum[w][m][n];
    const int64_t at = m * g.ldc + n0 + n;
    if (g.c_f32) {
      float* p = static_cast<float*>(g.c) + at;
      *p = g.accumulate ? *p + s : s;
    } else {
      static_cast<uint16_t*>(g.c)[at] = f32_to_bf16_bits(s);
    }
  }
}

// C = the parts' sum, in order
__global__ __launch_bounds__(256) void k_fp8_join(const float* __restrict__ part, int splits,
                                                  int64_t M, int64_t N, int64_t ldp,
                                                  void* __restrict__ c, int64_t ldc, int c_f32,
                                                  int accumulate) {
  const int64_t per = ldp / 4, total = M * per, stride = (int64_t)gridDim.x * 256;
  const bool vec = ldc * (c_f32 ? 4 : 2) % 16 == 0;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += stride) {
    const int64_t r = e / per, n = (e - r * per) * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p = 0; p < splits; ++p) {
      const float4 v = *reinterpret_cast<const float4*>(part + (p * M + r) * ldp + n);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const int left = (int)min((int64_t)4, N - n);
    if (c_f32) {
      store16(static_cast<char*>(c) + (r * ldc + n) * 4,
              make_uint4(__float_as_uint(s.x), __float_as_uint(s.y), __float_as_uint(s.z),
                         __float_as_uint(s.w)),
              left, true, vec, accumulate);
    } else {
      const uint2 w = pack4_bf16(s.x, s.y, s.z, s.w);
      uint16_t* p = static_cast<uint16_t*>(c) + r * ldc + n;
      if (vec && left == 4) {
        *reinterpret_cast<uint2*>(p) = w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) p[i] = (uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
      }
    }
  }
}

struct Plan {
  int bm, bn, splits, steps;
};

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

// The form, the tile and the split over k, from the sizes and the form of the products.
//   k_fp8_rows (us against the tile's): 16 x 4096 x 7168 11.8 (13.9), 32 x 1024 x 1024 7.1 (9.7),
//     32 x 4096 x 7168 16.2 (14.3)
//   256 x 256 (fp32 C: 256 x 128) once that leaves 192 CUs a tile: 2048 x 6400 x 4096 58 us
//     against 81 in tiles of 128 x 128
//   else the cheaper of 128 x 64 and 128 x 128, whole or split, by what was measured of each: a
//     step of a round of 256 workgroups, and for a split 3 us of k_fp8_join and its partial sums'
//     way out and in at 4 TB/s.  bf16 C: 1000 x 2048 x 2048 11.4 us as 128 x 64 (128 x 128: 14.2,
//     and 22.7 split in two); 640 x 2048 x 7168 24.8 as 128 x 128 in three parts (128 x 64
//     whole: 30.3); 128 x 4096 x 7168 16.6 as 128 x 64 in four (128 x 128 in eight: 18.3)
Plan plan(int64_t M, int64_t N, int64_t K, bool wide) {
  const int64_t nk = (K + GBK - 1) / GBK;
  Plan p;
  if (M <= 16 || (M <= 32 && K <= 2048)) {  // k_fp8_rows
    p.bm = M <= 16 ? 16 : 32;
    p.bn = 16;
    p.splits = 1;
    p.steps = (int)nk;
    return p;
  }
  p.splits = 1;
  p.steps = (int)nk;
  if (M > 128 && N > 128 && ((M + 255) / 256) * ((N + 255) / 256) >= 192) {
    p.bm = p.bn = 256;
    return p;
  }
  p.bm = 128;
  double best = 1e30;
  for (int bn = 64; bn <= 128; bn += 64) {
    const double step_us = bn == 64 ? (wide ? 0.73 : 0.55) : (wide ? 1.2 : 0.69);
    const int64_t tiles = ((M + 127) / 128) * ((N + bn - 1) / bn);
    for (int64_t s = 1; s == 1 || (s * tiles <= 256 && s <= nk / 8); ++s) {
      const int64_t steps = (nk + s - 1) / s, parts = (nk + steps - 1) / steps;
      double us = (double)((tiles * parts + 255) / 256 * steps) * step_us;
      if (parts > 1) us += 3.0 + 2e-6 * (double)(parts * M * N);
      if (us >= best) continue;
      best = us;
      p.bn = bn;
      p.splits = (int)parts;
      p.steps = (int)steps;
    }
  }
  return p;
}

template <int BM, int BN, int WM, int WN, int NST, bool kWide>
void launch_tile(GemmArgs g, bool row_b, hipStream_t st) {
  g.mt = (int)((g.M + BM - 1) / BM);
  g.nt = (int)((g.N + BN - 1) / BN);
  const int per = (g.mt * g.nt * g.splits + kXcds - 1) / kXcds;
  if (row_b)
    hipLaunchKernelGGL((k_fp8_tile<BM, BN, WM, WN, NST, kWide, true>), dim3(per * kXcds),
                       dim3(64 * WM * WN), 0, st, g);
  else
    hipLaunchKernelGGL((k_fp8_tile<BM, BN, WM, WN, NST, kWide, false>), dim3(per * kXcds),
                       dim3(64 * WM * WN), 0, st, g);
}

template <int MG, int kU, bool kWide>
void launch_rows(const GemmArgs& g, bool row_b, hipStream_t st) {
  const dim3 grid((unsigned)((g.N + 15) / 16));
  if (row_b) hipLaunchKernelGGL((k_fp8_rows<MG, kU, kWide, true>), grid, dim3(512), 0, st, g);
  else hipLaunchKernelGGL((k_fp8_rows<MG, kU, kWide, false>), grid, dim3(512), 0, st, g);
}
template <bool kWide>
void launch_rows(const Plan& p, const GemmArgs& g, bool row_b, hipStream_t st) {
  if (p.bm == 16) launch_rows<1, 4, kWide>(g, row_b, st);
  else launch_rows<2, 4, kWide>(g, row_b, st);
}

}  // namespace

size_t gemm_fp8_ws_bytes(int64_t M, int64_t N, int64_t K) {
  int splits = 1;  // the larger of the two forms
  for (int wide = 0; wide < 2; ++wide) splits = std::max(splits, plan(M, N, K, wide).splits);
  return splits > 1 ? (size_t)splits * (size_t)M * (size_t)up4(N) * 4 : 0;
}

hipError_t launch_gemm_fp8(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                           const float* sa, const uint8_t* b, int64_t ldb, const float* sb,
                           int b_rows, void* c, int64_t ldc, int c_f32, int accumulate, void* ws,
                           hipStream_t st) {
  const Plan p = plan(M, N, K, c_f32);
  GemmArgs g{a, b, sa, sb, c, lda, ldb, ldc, M, N, K, 0, 0, p.splits, p.steps, c_f32, accumulate};
  if (p.splits > 1) {
    g.c = ws;
    g.ldc = up4(N);
  }
  const bool row_b = b_rows == 1;
  if (p.bn == 16) {
    if (c_f32) launch_rows<true>(p, g, row_b, st);
    else launch_rows<false>(p, g, row_b, st);
  } else if (p.bn == 64) {
    if (c_f32) launch_tile<128, 64, 4, 2, 3, true>(g, row_b, st);
    else launch_tile<128, 64, 4, 2, 3, false>(g, row_b, st);
  } else if (p.bn == 128 && (M + 127) / 128 * ((N + 127) / 128) * p.splits <= 256) {
    // one workgroup a CU: three stages (1408 x 2048 x 7168: 39 us, with two 52); more of them:
    // two stages, with which a CU holds two workgroups (2048 x 4096 x 4096: 45 us, with three 56)
    if (c_f32) launch_tile<128, 128, 4, 2, 3, true>(g, row_b, st);
    else launch_tile<128, 128, 4, 2, 3, false>(g, row_b, st);
  } else if (p.bn == 128) {
    if (c_f32) launch_tile<128, 128, 4, 2, 2, true>(g, row_b, st);
    else launch_tile<128, 128, 4, 2, 2, false>(g, row_b, st);
  } else {
    if (c_f32) launch_tile<256, 128, 4, 2, 3, true>(g, row_b, st);
    else launch_tile<256, 256, 4, 2, 2, false>(g, row_b, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t blocks = (M * (up4(N) / 4) + 255) / 256;
  hipLaunchKernelGGL(k_fp8_join, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                     st, static_cast<const float*>(ws), p.splits, M, N, up4(N), c, ldc, c_f32,
                     accumulate);
  return hipGetLastError();
}

}  // namespace moe
