// Block-scaled FP8 (E4M3) matrix product of any size:
//   C[m,n] = sum_b sa[m,b] sb[n',b] sum_{k in block b} A[m,k] B[n,k]
// over blocks b of 128 along k, A with one fp32 scale per (row, block), B with one per
// (row, block) or per 128 rows and block (n' = n or n / 128).  A block's partial sum of code
// products is formed by the matrix cores and promoted as acc += partial * (sa * sb) in fp32.
// The codes of a row's last block past K are taken as zeros, whatever the pad holds.
//
// How a block's sum is formed goes by C's type (kWide):
//   bf16 C: the FP8 matrix instruction (32x32x64 f8f6f4, neutral E8M0 scales: the fp32 scales
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
#include "common.h"

namespace moe {
namespace {

constexpr int GBK = 128;

typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

// byte of (row, 16-byte chunk c) in a stage
__device__ __forceinline__ int at128(int r, int c) { return r * GBK + ((c ^ (r >> 1)) & 7) * 16; }

// 32 codes as the operand of one FP8 product, or widened for four bf16 products (the same k of
// both operands meet, whatever their order within the 64)
__device__ __forceinline__ i32x8 codes32(const char* p0, const char* p1) {
  const uint4 u0 = *reinterpret_cast<const uint4*>(p0);
  const uint4 u1 = *reinterpret_cast<const uint4*>(p1);
  i32x8 f;
  f[0] = u0.x; f[1] = u0.y; f[2] = u0.z; f[3] = u0.w;
  f[4] = u1.x; f[5] = u1.y; f[6] = u1.z; f[7] = u1.w;
  return f;
}
__device__ __forceinline__ bf16x8 widen8(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <bool kWide>
struct Frag;
template <>
struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void load(const char* p0, const char* p1) { v = codes32(p0, p1); }
  static __device__ __forceinline__ f32x16 mul(const Frag& b, const Frag& a, f32x16 t) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.v, a.v, t, 0, 0, 0, 127, 0, 127);
  }
};
template <>
struct Frag<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void load(const char* p0, const char* p1) {
    const i32x8 c = codes32(p0, p1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = widen8(c[2 * i], c[2 * i + 1]);
  }
  static __device__ __forceinline__ f32x16 mul(const Frag& b, const Frag& a, f32x16 t) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.v[i], a.v[i], t, 0, 0, 0);
    return t;
  }
};

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
  constexpr int W = WM * WN, SM = BM / WM / 32, SN = BN / WN / 32;
  constexpr int kStage = (BM + BN) * GBK;
  constexpr int NA = BM / 8 / W, NB = BN / 8 / W, kPer = NA + NB + 1;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0, "whole load instructions");
  static_assert(W * 32 * (BN / WN) * 4 <= NST * kStage, "output staging fits the ring");
  __shared__ __attribute__((aligned(1024))) char smem[NST * kStage];
  __shared__ __attribute__((aligned(16))) float s_sc[NST][BM + BN];
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
  const int wm = wv / WN, wn = wv % WN, fr = lane & 31, kq = lane >> 5;
  const int nk = (int)((g.K + GBK - 1) / GBK);
  const int k0 = part * g.steps, k1 = min(k0 + g.steps, nk);
  const int m_rows = (int)min((int64_t)BM, g.M - m0), n_rows = (int)min((int64_t)BN, g.N - n0);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const uint32_t lds_sc = __builtin_amdgcn_readfirstlane(lds_offset(&s_sc[0][0]));
  const i32x4 ar = buffer_rsrc(g.a + m0 * g.lda, (uint32_t)(m_rows * g.lda));
  const i32x4 br = buffer_rsrc(g.b + n0 * g.ldb, (uint32_t)(n_rows * g.ldb));
  // instruction i of wave wv fills rows 8 (i W + wv) .. +7 of the stage (A's, then B's)
  const int lrow = 8 * wv + (lane >> 3);
  const int lchunk = (lane & 7) ^ ((4 * (wv & 1) + (lane >> 4)) & 7);
  uint32_t ao[NA], bo[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) ao[i] = (uint32_t)((8 * W * i + lrow) * g.lda) + 16 * lchunk;
#pragma unroll
  for (int i = 0; i < NB; ++i) bo[i] = (uint32_t)((8 * W * i + lrow) * g.ldb) + 16 * lchunk;
  // one scale load a wave: 64 rows of A's, then (kRowB) of B's; waves past those repeat one
  constexpr int kScGroups = (BM + (kRowB ? BN : 0)) / 64;
  const int sg = wv % kScGroups;
  const bool sg_a = sg < BM / 64;
  const int s_row = 64 * sg + lane - (sg_a ? 0 : BM);
  const float* s_base = sg_a ? g.sa + m0 * nk : g.sb + n0 * nk;
  const i32x4 sr = buffer_rsrc(s_base, (uint32_t)((sg_a ? m_rows : n_rows) * (int64_t)nk * 4));
  const uint32_t so = (uint32_t)(s_row * nk) * 4;
  const uint32_t s_lds = lds_sc + 64 * sg * 4;
  auto stage = [&](int kt, int st) {
    const uint32_t dst = lds0 + st * kStage + 8 * wv * GBK, ko = (uint32_t)kt * GBK;
#pragma unroll
    for (int i = 0; i < NA; ++i) load16_to_lds(ar, dst + i * 8 * W * GBK, ao[i] + ko);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      load16_to_lds(br, dst + (BM + i * 8 * W) * GBK, bo[i] + ko);
    load4_to_lds(sr, s_lds + st * (BM + BN) * 4, so + (uint32_t)kt * 4);
  };
  // !kRowB: the scales of the wave's 128-row block (the last one where the wave is past N)
  const float* sbp = g.sb + min((n0 + wn * (BN / WN)) / 128, (g.N - 1) / 128) * nk;

  f32x16 acc[SM][SN];
#pragma unroll
  for (int m = 0; m < SM; ++m)
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;

#pragma unroll
  for (int j = 0; j < NST - 1; ++j)
    if (k0 + j < k1) stage(k0 + j, j);
  int st = 0;
  for (int kt = k0; kt < k1; ++kt) {
    float sw = 1.0f;
    if (!kRowB) sw = sbp[kt];
    if (k1 - kt >= NST - 1) wait_vm<(NST - 2) * kPer>();
    else wait_vm<0>();
    __syncthreads();
    if (kt + NST - 1 < k1) stage(kt + NST - 1, st == 0 ? NST - 1 : st - 1);
    char* as = smem + st * kStage;
    char* bs = as + BM * GBK;
    if (kt == nk - 1 && (g.K & (GBK - 1))) {  // the last block's codes past K
      const int left = (int)(g.K & (GBK - 1));
      for (int q = tid; q < (BM + BN) * 8; q += 64 * W) {
        const int n = left - 16 * (q & 7);
        if (n >= 16) continue;
        uint4* p = reinterpret_cast<uint4*>(as + at128(q >> 3, q & 7));
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
    Frag<kWide> fa[SM][2];
    float sa[SM];
#pragma unroll
    for (int m = 0; m < SM; ++m) {
      const int r = wm * (BM / WM) + 32 * m + fr;
      fa[m][0].load(as + at128(r, 2 * kq), as + at128(r, 2 * kq + 1));
      fa[m][1].load(as + at128(r, 4 + 2 * kq), as + at128(r, 5 + 2 * kq));
      sa[m] = s_sc[st][r] * sw;
    }
#pragma unroll
    for (int n = 0; n < SN; ++n) {
      const int r = wn * (BN / WN) + 32 * n + fr;
      Frag<kWide> fb[2];
      fb[0].load(bs + at128(r, 2 * kq), bs + at128(r, 2 * kq + 1));
      fb[1].load(bs + at128(r, 4 + 2 * kq), bs + at128(r, 5 + 2 * kq));
      float sb[16];
      if (kRowB) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(
              &s_sc[st][BM + wn * (BN / WN) + 32 * n + 8 * q + 4 * kq]);
          sb[4 * q] = v.x; sb[4 * q + 1] = v.y; sb[4 * q + 2] = v.z; sb[4 * q + 3] = v.w;
        }
      }
#pragma unroll
      for (int m = 0; m < SM; ++m) {
        f32x16 t;
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = 0.0f;
        t = Frag<kWide>::mul(fb[0], fa[m][0], t);
        t = Frag<kWide>::mul(fb[1], fa[m][1], t);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[m][n][i] = __builtin_fmaf(t[i], kRowB ? sa[m] * sb[i] : sa[m], acc[m][n][i]);
      }
    }
    if (++st == NST) st = 0;
  }
  wait_vm<0>();
  __syncthreads();  // every wave is done with the ring, which now stages the output

  // a wave's 32 x (BN/WN) outputs of sub-tile m in LDS (16-byte chunks swizzled by the row),
  // stored back 16 bytes a lane along the rows
  const bool f32 = g.c_f32 || g.splits > 1;
  const int es = f32 ? 4 : 2;
  constexpr int kCols = BN / WN;
  const int row_bytes = kCols * es, chunks = row_bytes / 16, mask = min(chunks, 16) - 1;
  char* stg = smem + wv * 32 * kCols * 4;
  char* out = static_cast<char*>(g.c) + (g.splits > 1 ? (int64_t)part * g.M * g.ldc * 4 : 0);
  const bool vec = g.ldc * es % 16 == 0;
  const bool add = g.accumulate && g.splits == 1;
#pragma unroll
  for (int m = 0; m < SM; ++m) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& a = acc[m][n];
        const int col = 32 * n + 8 * q + 4 * kq;
        if (f32) {
          const int ch = col / 4;
          *reinterpret_cast<float4*>(stg + fr * row_bytes + ((ch ^ (fr & mask)) << 4)) =
              make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
        } else {
          const int ch = col / 8;
          *reinterpret_cast<uint2*>(stg + fr * row_bytes + ((ch ^ (fr & mask)) << 4) + 8 * kq) =
              pack4_bf16(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int64_t row0 = m0 + wm * (BM / WM) + 32 * m;
    for (int e = lane; e < 32 * chunks; e += 64) {
      const int r = e / chunks, ch = e % chunks;
      const int64_t n = n0 + wn * kCols + ch * (16 / es);
      const uint4 v = *reinterpret_cast<const uint4*>(stg + r * row_bytes + ((ch ^ (r & mask)) << 4));
      if (row0 + r < g.M && n < g.N)
        store16(out + ((row0 + r) * g.ldc + n) * es, v, (int)min((int64_t)8, g.N - n), f32, vec,
                add);
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

// The tile and the split over k, from the sizes alone (the workspace's size depends on it).
Plan plan(int64_t M, int64_t N, int64_t K) {
  const int64_t nk = (K + GBK - 1) / GBK;
  Plan p;
  if (M <= 64) { p.bm = 64; p.bn = 128; }
  else if (((M + 255) / 256) * ((N + 255) / 256) >= 192) { p.bm = 256; p.bn = 256; }
  else { p.bm = 128; p.bn = 128; }
  const int64_t tiles = ((M + p.bm - 1) / p.bm) * ((N + p.bn - 1) / p.bn);
  int64_t s = tiles >= 192 ? 1 : 256 / tiles;
  s = s < nk / 4 ? s : nk / 4;  // at least 4 blocks a part
  if (s < 1) s = 1;
  p.steps = (int)((nk + s - 1) / s);
  p.splits = (int)((nk + p.steps - 1) / p.steps);
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

}  // namespace

size_t gemm_fp8_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const Plan p = plan(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)up4(N) * 4 : 0;
}

hipError_t launch_gemm_fp8(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                           const float* sa, const uint8_t* b, int64_t ldb, const float* sb,
                           int b_rows, void* c, int64_t ldc, int c_f32, int accumulate, void* ws,
                           hipStream_t st) {
  const Plan p = plan(M, N, K);
  GemmArgs g{a, b, sa, sb, c, lda, ldb, ldc, M, N, K, 0, 0, p.splits, p.steps, c_f32, accumulate};
  if (p.splits > 1) {
    g.c = ws;
    g.ldc = up4(N);
  }
  const bool row_b = b_rows == 1;
  if (p.bm == 64) {
    if (c_f32) launch_tile<64, 128, 1, 4, 3, true>(g, row_b, st);
    else launch_tile<64, 128, 1, 4, 3, false>(g, row_b, st);
  } else if (p.bm == 128) {
    if (c_f32) launch_tile<128, 128, 2, 2, 2, true>(g, row_b, st);
    else launch_tile<128, 128, 2, 2, 2, false>(g, row_b, st);
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
