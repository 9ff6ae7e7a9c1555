// MXFP4 matrix product of any size: C[m,n] = sum_k A[m,k] B[n,k] over E2M1 codes with one E8M0
// scale per (row, 32 of k) on either side.  The matrix instructions take codes and scales as they
// are and add in fp32 (products of two codes are multiples of 1/4 up to 36, so the sum of a block's
// is exact; what is rounded is the sum over blocks).
//
// k_mx_gemm: BM x BN outputs a workgroup of WM x WN waves, 256 of k a step.  Codes go from memory
// straight to a ring of LDS stages (buffer loads with the LDS destination bit; rows of 128 bytes,
// 16-byte chunks xor-swizzled by the row), rows past M or N arrive as zeros by the descriptor's
// range check, chunks past K by an offset outside it.  Scales come 16 bytes of a row at a time,
// two steps' worth, into a ring of their own.  Within a step's 256 of k, part s (of 128) and
// instruction u of it take the blocks 4 s + 2 h + u in lane half h, the same on both sides, so
// that a lane's two scales of a part are adjacent bytes.  B is the instruction's first operand: a
// lane's results lie in one row of C.  Split over k (few tiles): fp32 partial sums to the
// workspace, k_mx_join adds them in order.
//   4096 x 4096 x 7168, bf16 out, 256 x 256 tiles: 65 to 73 us by card, 3.3 to 3.7 PFLOP/s.  A round of
//   128 of k takes 0.97 us; its 4.3 GFLOP take 0.66 at the rate of a loop of the matrix instruction
//   alone on random codes (6.5 PFLOP/s: the card's power holds that loop's clock at 1.7 GHz; on zeros it
//   runs 9.7 at 2.4).  What is between them is LDS reads, loads and the barrier.  12 to 14 us do not
//   grow with K: the first loads, and 7 to 8 for the 34 MB of C that all 256 workgroups store at once,
//   with one workgroup a CU and nothing to run beside them.  2048 x 7168 x 4099, fp32 out: 49 us, 12 of
//   them the 59 MB of C.
//   128 x 4096 x 7168, 64 x 64 tiles: 11.7 us, of 28 dependent steps at 0.33 and the first loads.
// Read and stored once: C goes past the caches, operands through them (they are read again by the
// other tiles of their band).
// k_mx_gemm_rows: few rows of A; see there.
#include <algorithm>
#include <type_traits>

#include "mxfp4.h"

namespace moe {
namespace {

constexpr int kStep = 256;       // of k, of k_mx_gemm_rows
constexpr int kRow = kStep / 2;  // bytes of a row in a step
constexpr uint32_t kOut = 0x7ffffff0u;  // an offset past every descriptor's range

__device__ __forceinline__ u32x4 lds16(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((uintptr_t)addr);
}

struct GemmArgs {
  const uint8_t *a, *b, *sa, *sb;
  void* c;  // C, or the partial sums [splits, M, ldc] fp32
  int64_t lda, ldb, ldsa, ldsb, ldc, M, N, K;
  int mt, nt;         // tiles along M and N
  int splits, steps;  // k is cut into `splits` parts of `steps` stages
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
      const u32x4 w4 = {__float_as_uint(o.x), __float_as_uint(o.y), __float_as_uint(o.z),
                        __float_as_uint(o.w)};
      __builtin_nontemporal_store(w4, reinterpret_cast<u32x4*>(q));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) q[i] = accumulate ? q[i] + w[i] : w[i];
    }
  } else if (vec && n >= 8) {
    const u32x4 w4 = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w4, reinterpret_cast<u32x4*>(p));
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// kParts: 128 of k a part, a stage holds one or two of them (rows of 64 or 128 bytes, 16-byte chunks
// xor-swizzled by the row so that 8 rows read at one chunk lie in different banks)
template <int kParts>
__device__ __forceinline__ int chunk_at(int r, int c) {
  if (kParts == 2) return r * 128 + ((c ^ (r >> 1)) & 7) * 16;
  return r * 64 + ((c ^ (r >> 2)) & 3) * 16;
}

template <int BM, int BN, int WM, int WN, int kParts, int NST>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_mx_gemm(GemmArgs g) {
  constexpr int W = WM * WN, SM = BM / WM / 32, SN = BN / WN / 32;
  constexpr int kChunks = 4 * kParts, kRowB = 16 * kChunks, kStage = (BM + BN) * kRowB;
  constexpr int kRpi = 1024 / kRowB;  // rows of a load instruction
  constexpr int kPerSc = 4 / kParts;  // stages of 16 bytes of scales
  constexpr int kScBuf = (BM + BN) * 16;
  constexpr int NA = BM / kRpi / W, NB = BN / kRpi / W;      // code loads of a wave and stage
  constexpr int kG = (BM + BN) / 64, NS = (kG + W - 1) / W;  // scale loads: 64 rows each
  constexpr int kPer = NA + NB, kJ = 2 * kParts;             // kJ products a sub-tile and stage
  static_assert(BM % (kRpi * W) == 0 && BN % (kRpi * W) == 0 && BM % 64 == 0 && BN % 64 == 0,
                "whole load instructions");
  static_assert(NST >= 4, "one stage in use, one complete, two on their way");
  static_assert(W * 32 * (BN / WN) * 4 <= NST * kStage, "output staging fits the ring");
  __shared__ __attribute__((aligned(1024))) char smem[NST * kStage];
  // scales of 512 of k, 16 bytes a row: stage kt + 3's arrive while stage kt's are read
  constexpr int kScBufs = kParts == 2 ? 3 : 2;
  __shared__ __attribute__((aligned(16))) char s_sc[kScBufs * kScBuf];
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
  const int wm = wv / WN, wn = wv % WN, fr = lane & 31, h = lane >> 5;
  const int nb = (int)((g.K + kMxBlock - 1) / kMxBlock);  // blocks of k
  const int nk = (nb + kChunks - 1) / kChunks;
  const int k0 = part * g.steps, k1 = min(k0 + g.steps, nk);
  const int m_rows = (int)min((int64_t)BM, g.M - m0), n_rows = (int)min((int64_t)BN, g.N - n0);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const uint32_t lds_sc = __builtin_amdgcn_readfirstlane(lds_offset(s_sc));
  // a tile's last row of codes ends with its blocks: there may be no memory behind it
  const i32x4 ar = buffer_rsrc(g.a + m0 * g.lda, (uint32_t)((m_rows - 1) * g.lda + 16 * nb));
  const i32x4 br = buffer_rsrc(g.b + n0 * g.ldb, (uint32_t)((n_rows - 1) * g.ldb + 16 * nb));
  const i32x4 sar = buffer_rsrc(g.sa + m0 * g.ldsa, (uint32_t)(m_rows * g.ldsa));
  const i32x4 sbr = buffer_rsrc(g.sb + n0 * g.ldsb, (uint32_t)(n_rows * g.ldsb));
  // instruction i of wave wv fills rows kRpi (i W + wv) .. of the stage (A's, then B's)
  const int lrow = kRpi * wv + lane / kChunks;
  const int lchunk = kParts == 2 ? (lane & 7) ^ ((4 * (wv & 1) + (lane >> 4)) & 7)
                                 : (lane & 3) ^ (lane >> 4);
  const uint32_t ao = (uint32_t)(lrow * g.lda) + 16 * lchunk;
  const uint32_t bo = (uint32_t)(lrow * g.ldb) + 16 * lchunk;
  const uint32_t a_next = (uint32_t)(kRpi * W * g.lda), b_next = (uint32_t)(kRpi * W * g.ldb);
  uint32_t so[NS];  // scale load i: rows 64 q .. +63 of A, then of B, q = i W + wv
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int q = i * W + wv;
    so[i] = (uint32_t)(q < BM / 64 ? (64 * q + lane) * g.ldsa : (64 * q - BM + lane) * g.ldsb);
  }
  // load instruction i (of kPer) of a wave for stage kt; past the last stage it fetches what nothing
  // reads
  auto load = [&](int kt, int st, int i) {
    const uint32_t dst = lds0 + st * kStage + wv * 1024, ko = (uint32_t)kt * kRowB;
    const bool in = kChunks * kt + lchunk < nb;
    if (i < NA)
      load16_to_lds(ar, dst + i * W * 1024, in ? ao + (i * a_next + ko) : kOut);
    else
      load16_to_lds(br, dst + BM * kRowB + (i - NA) * W * 1024,
                    in ? bo + ((i - NA) * b_next + ko) : kOut);
  };
  // the scales of stage kt and of those that share its 16 bytes, with the first of them
  auto load_scales = [&](int kt) {
    if (kt % kPerSc != 0) return;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int q = i * W + wv;
      if (q < kG)
        load16_to_lds(q < BM / 64 ? sar : sbr,
                      lds_sc + kt / kPerSc % kScBufs * kScBuf + 1024 * q,
                      so[i] + 16 * (uint32_t)(kt / kPerSc));
    }
  };

  f32x16 acc[SM][SN];
#pragma unroll
  for (int m = 0; m < SM; ++m)
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;

  // Blocks past K have zero codes (their loads are out of range), and their scales become 2^-127: the
  // pad may hold the NaN.  Once the last 512 of k's have come, before any is read.
  auto clear_scales = [&](int kt) {
    if (nb % 16 == 0 || kt / kPerSc != (nk - 1) / kPerSc) return;
    char* sc = s_sc + kt / kPerSc % kScBufs * kScBuf;
    for (int r = tid; r < BM + BN; r += 64 * W)
      for (int b = nb % 16; b < 16; ++b) sc[16 * r + b] = 0;
    __syncthreads();
  };
  // The last block's codes past K are cleared in A, once the last stage has come.
  auto clear_codes = [&](int kt, int st) {
    const int n = (int)(g.K & (kMxBlock - 1));
    if (n == 0 || kt != nk - 1) return;
    for (int r = tid; r < BM; r += 64 * W) {
      uint32_t* p = reinterpret_cast<uint32_t*>(smem + st * kStage +
                                                chunk_at<kParts>(r, nb - 1 - kChunks * kt));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n < 8 * i + 8) p[i] = n > 8 * i ? p[i] & ((1u << (4 * (n - 8 * i))) - 1u) : 0u;
    }
    __syncthreads();
  };
  // Operands of the product at hand and of the next kAhead: one where a wave has many sub-tiles, whose
  // products cover the LDS's latency, else as many as reach into the next stage.
  constexpr int kAhead = SM * SN >= 8 || kParts == 1 ? 1 : 3, kBufs = kAhead + 1;
  u32x4 fa[kBufs][SM], fb[kBufs][SN];
  u32x4 qa[SM], qb[SN];        // scales of 512 of k, 4 bytes a part
  uint32_t sa[SM], sb[SN];     // of the part at hand: the lane's two
  // operand i (A's, then B's) of product j = 2 s + u of stage st
  auto frag = [&](int st, int j, int buf, int i) {
    const uint32_t at = lds0 + st * kStage + chunk_at<kParts>(fr, 4 * (j >> 1) + 2 * h + (j & 1));
    if (i < SM) fa[buf][i < SM ? i : 0] = lds16(at + (wm * (BM / WM) + 32 * i) * kRowB);
    else fb[buf][i < SM ? 0 : i - SM] = lds16(at + (BM + wn * (BN / WN) + 32 * (i - SM)) * kRowB);
  };
  auto scale = [&](int kt, int i) {  // operand i's scales of the 512 of k with stage kt
    const uint32_t at = lds_sc + kt / kPerSc % kScBufs * kScBuf + 16 * fr;
    if (i < SM) qa[i < SM ? i : 0] = lds16(at + 16 * (wm * (BM / WM) + 32 * i));
    else qb[i < SM ? 0 : i - SM] = lds16(at + 16 * (BM + wn * (BN / WN) + 32 * (i - SM)));
  };
  constexpr int kOps = SM + SN, kMul = SM * SN;

#pragma unroll
  for (int j = 0; j < NST - 1; ++j) {
    load_scales(k0 + j);
#pragma unroll
    for (int i = 0; i < kPer; ++i) load(k0 + j, j, i);
  }
  wait_vm<(NST - 2) * kPer>();
  __syncthreads();
  clear_scales(k0);
  clear_codes(k0, 0);
  int st = 0;
#pragma unroll
  for (int i = 0; i < kOps; ++i) scale(k0, i);
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
#pragma unroll
    for (int i = 0; i < kOps; ++i) frag(0, j, j, i);
  // k1 - k0 stages, 512 of k a turn of the outer loop (k0 a multiple).  A stage's first
  // operands are in registers when its turn comes, and the stage after it is complete in LDS behind
  // its barrier, so that the matrix cores do not run dry at the barriers.
  for (int kc = k0; kc < k1; kc += kPerSc) {
#pragma unroll
    for (int t = 0; t < kPerSc; ++t) {
      const int kt = kc + t;
      if (kt >= k1) break;
      wait_vm<(NST - 3) * kPer>();
      // nothing but loads fills the ring, and this wave's reads of what is filled next are behind
      // its products: the barrier alone, without waiting for the reads ahead
      asm volatile("s_barrier" ::: "memory");
      const int st1 = st + 1 == NST ? 0 : st + 1, st_ld = st == 0 ? NST - 1 : st - 1;
      if (t == kPerSc - 1) clear_scales(kt + 1);
      clear_codes(kt + 1, st1);
      load_scales(kt + NST - 1);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int part = t * kParts + (j >> 1);  // of the 512 of k
        const int buf = (t * kJ + j) % kBufs, next = (buf + kAhead) % kBufs;
        if ((j & 1) == 0) {
#pragma unroll
          for (int i = 0; i < SM; ++i) sa[i] = qa[i][part] >> (16 * h);
#pragma unroll
          for (int i = 0; i < SN; ++i) sb[i] = qb[i][part] >> (16 * h);
        }
#pragma unroll
        for (int p = 0; p < kMul; ++p) {
          const int m = p % SM, n = p / SM;
          acc[m][n] = (j & 1) ? mx_mfma32<1, 1>(fb[buf][n], fa[buf][m], acc[m][n], sb[n], sa[m])
                              : mx_mfma32<0, 0>(fb[buf][n], fa[buf][m], acc[m][n], sb[n], sa[m]);
          // what follows each product, in this order (left to the compiler, all of a stage's products
          // sank below its last LDS read): reads for the next product, a load for the ring
          asm volatile("" : "+a"(acc[m][n]) : : "memory");
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < kOps; ++i)
            if (i * kMul / kOps == p) {
              if (j + kAhead < kJ) frag(st, j + kAhead, next, i);
              else frag(st1, j + kAhead - kJ, next, i);
              // the next 512 of k's scales, once this one's last are taken
              if ((j & 1) == 0 && part == 3) scale(kt + 1, i);
            }
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (i * kJ * kMul / kPer == j * kMul + p) load(kt + NST - 1, st_ld, i);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      st = st1;
    }
  }
  wait_vm<0>();
  __syncthreads();  // every wave is done with the ring, which now stages the output

  // a wave's 32 x (BN/WN) outputs of sub-tile row m in LDS (16-byte chunks swizzled by the row),
  // stored back 16 bytes a lane along the rows
  auto store = [&](auto is_f32) {
    constexpr bool f32 = decltype(is_f32)::value;
    constexpr int es = f32 ? 4 : 2, kCols = BN / WN, row_bytes = kCols * es;
    constexpr int chunks = row_bytes / 16, mask = (chunks < 16 ? chunks : 16) - 1;
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
          const auto& a = acc[m][n];
          const int col = 32 * n + 8 * q + 4 * h;  // 4 adjacent columns
          char* p = stg + fr * row_bytes + (((col * es / 16) ^ (fr & mask)) << 4);
          if (f32)
            *reinterpret_cast<float4*>(p) =
                make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
          else
            *reinterpret_cast<uint2*>(p + (col & 4) * 2) =
                pack4_bf16(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int64_t row0 = m0 + wm * (BM / WM) + 32 * m;
#pragma unroll
      for (int e0 = 0; e0 < 32 * chunks; e0 += 64) {
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
  if (g.c_f32 || g.splits > 1) store(std::true_type());
  else store(std::false_type());
}

// Few tiles: a workgroup of 8 waves takes 16 MG rows x 16 NG columns, its waves every 8th step of
// 256 of k each, with the codes of kU steps on their way from memory straight into registers, and
// they add their sums in LDS, in order.  Nothing waits for another wave before the end.  The 16 x 16 x
// 128 instruction: B the first operand, lane l holds block l / 16 of its row, l % 16, and the
// result's rows 4 (l / 16) .. +3 of B for row l % 16 of A.
// 1 x 7168 x 2048: 4.3 us for 7.8 MB, a launch, one step a wave and the join in LDS (1.6 us at a
// copy's rate).
struct Half {  // a row's 128 of k: the lane's block and its scale
  u32x4 q;
  uint32_t s;
};
__device__ __forceinline__ f32x4 mul16(const Half& b, const Half& a, const f32x4& c) {
  const i32x8 x = {(int)b.q[0], (int)b.q[1], (int)b.q[2], (int)b.q[3], 0, 0, 0, 0};
  const i32x8 y = {(int)a.q[0], (int)a.q[1], (int)a.q[2], (int)a.q[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)b.s, 0, (int)a.s);
}

template <int MG, int NG, int kU>
__global__ __launch_bounds__(512, 1) void k_mx_gemm_rows(GemmArgs g) {
  constexpr int kW = 8, kM = 16 * MG, kN = 16 * NG;
  __shared__ float s_sum[kW][kM][kN + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)(blockIdx.x / g.mt) * kN, m0 = (int64_t)(blockIdx.x % g.mt) * kM;
  const int nb = (int)((g.K + kMxBlock - 1) / kMxBlock), nk = (nb + 7) / 8;
  const int whole = (int)(g.K / kStep);
  // rows past M or N repeat the last one (their results are not stored)
  uint32_t ao[MG], sao[MG], bo[NG], sbo[NG];  // from the tile's first row on
#pragma unroll
  for (int m = 0; m < MG; ++m) {
    const uint32_t row = (uint32_t)min((int64_t)16 * m + r, g.M - 1 - m0);
    ao[m] = row * (uint32_t)g.lda + 16 * q;
    sao[m] = row * (uint32_t)g.ldsa;
  }
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const uint32_t row = (uint32_t)min((int64_t)16 * n + r, g.N - 1 - n0);
    bo[n] = row * (uint32_t)g.ldb + 16 * q;
    sbo[n] = row * (uint32_t)g.ldsb;
  }
  const uint8_t *ap = g.a + m0 * g.lda, *sap = g.sa + m0 * g.ldsa;
  const uint8_t *bp = g.b + n0 * g.ldb, *sbp = g.sb + n0 * g.ldsb;
  struct Step {
    Half a[MG][2], b[NG][2];
  };
  auto scale = [&](const uint8_t* p, Half (&v)[2]) {
    const uint2 s = *reinterpret_cast<const uint2*>(p);
    v[0].s = s.x >> (8 * q);
    v[1].s = s.y >> (8 * q);
  };
  auto load = [&](Step& v, int st) {  // a whole step
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const uint8_t* p = bp + st * kRow + bo[n];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v.b[n][h].q = MG == 1 && NG == 1  // B is read once in all
                          ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 64 * h))
                          : *reinterpret_cast<const u32x4*>(p + 64 * h);
      scale(sbp + 8 * st + sbo[n], v.b[n]);
    }
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      const uint8_t* p = ap + st * kRow + ao[m];
#pragma unroll
      for (int h = 0; h < 2; ++h) v.a[m][h].q = *reinterpret_cast<const u32x4*>(p + 64 * h);
      scale(sap + 8 * st + sao[m], v.a[m]);
    }
  };
  f32x4 acc[MG][NG];
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int n = 0; n < NG; ++n) acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const Step& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MG; ++m)
#pragma unroll
        for (int n = 0; n < NG; ++n) acc[m][n] = mul16(v.b[n][h], v.a[m][h], acc[m][n]);
  };
  Step v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (wv + kW * u < whole) load(v[u], wv + kW * u);
  for (int b = wv; b < whole; b += kW * kU)
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int st = b + kW * u;
      if (st >= whole) break;
      add(v[u]);
      if (st + kW * kU < whole) load(v[u], st + kW * kU);
    }
  if (whole < nk && whole % kW == wv) {  // the last, partial step
    const u32x4 zero = {0, 0, 0, 0};
    // this lane's block of half h: zeros past K, and in A the codes past K cleared
    auto partial = [&](const uint8_t* p, const uint8_t* sp, int h, bool clear, Half& v) {
      const int b = 8 * whole + 4 * h + q;
      const bool in = b < nb;
      v.q = in ? *reinterpret_cast<const u32x4*>(p + whole * kRow + 64 * h) : zero;
      v.s = in ? sp[b] : 0;
      const int n = clear ? (int)min((int64_t)kMxBlock, g.K - (int64_t)kMxBlock * b) : kMxBlock;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n < 8 * i + 8) v.q[i] = n > 8 * i ? v.q[i] & ((1u << (4 * (n - 8 * i))) - 1u) : 0u;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < NG; ++n) partial(bp + bo[n], sbp + sbo[n], h, false, v[0].b[n][h]);
#pragma unroll
      for (int m = 0; m < MG; ++m) partial(ap + ao[m], sap + sao[m], h, true, v[0].a[m][h]);
    }
    add(v[0]);
  }
#pragma unroll
  for (int m = 0; m < MG; ++m)
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_sum[wv][16 * m + r][16 * n + 4 * q + i] = acc[m][n][i];
  __syncthreads();
  for (int e = tid; e < kM * kN; e += 512) {
    const int m = e / kN, n = e % kN;
    if (m0 + m >= g.M || n0 + n >= g.N) continue;
    float s = s_sum[0][m][n];
#pragma unroll
    for (int w = 1; w < kW; ++w) s += s_sum[w][m][n];
    const int64_t at = (m0 + m) * g.ldc + n0 + n;
    if (g.c_f32) {
      float* p = static_cast<float*>(g.c) + at;
      *p = g.accumulate ? *p + s : s;
    } else {
      static_cast<uint16_t*>(g.c)[at] = f32_to_bf16_bits(s);
    }
  }
}

// C = the parts' sum, in order
__global__ __launch_bounds__(256) void k_mx_join(const float* __restrict__ part, int splits,
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

// The form, the tile and the split over k, from the sizes.
//   Few rows, or few outputs: k_mx_gemm_rows in 16 or 32 rows x 16 columns, or in 32 x 32 where that
//     is one round of workgroups and no long sum (256 x 1024 x 7168 10.7 us, as tiles of 64 x 64 13.1;
//     300 x 300 x 300 4.3, 5.5; 33 x 7168 x 2048, two rounds, 9.0, 6.0; 40 x 40 x 16384 23.4, 20.8).
//   Else the tile, whole or split, that is cheapest by what was measured of each: a step of a round
//     of 256 workgroups, and for a split 3 us of k_mx_join and its partial sums' way out and in at 4
//     TB/s.  128 x 4096 x 7168: 64 x 64 12.0 us, 128 x 64 14.5, that in four parts 14.9; 512 x 4096 x
//     4096: 128 x 64 12.0, 64 x 64 16.4, 128 x 128 13.0; 2048 x 4096 x 4096: 128 x 256 26, 128 x 128 29,
//     256 x 256 33; 4096 x 4096 x 7168: 256 x 256 66, 128 x 256 80, 128 x 128 84.
Plan plan(int64_t M, int64_t N, int64_t K) {
  const int64_t nk = (K + kStep - 1) / kStep;
  Plan p;
  p.splits = 1;
  p.steps = (int)nk;
  if (M <= 32) {
    p.bm = M <= 16 ? 16 : 32;
    p.bn = 16;
    return p;
  }
  const auto tiles = [&](int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); };
  if (tiles(32, 32) <= 256 && nk <= 32) {
    p.bm = p.bn = 32;
    return p;
  }
  static constexpr struct {
    int bm, bn;
    double step_us;
  } kForms[] = {{64, 64, 0.33}, {128, 64, 0.50}, {128, 128, 0.74}, {128, 256, 1.38}, {256, 256, 1.94}};
  double best = 1e30;
  for (const auto& f : kForms)
    for (int64_t s = 1; s == 1 || (s * tiles(f.bm, f.bn) <= 256 && s <= nk / 4); ++s) {
      // a part begins at a multiple of 512 of k
      const int64_t steps = s == 1 ? nk : ((nk + s - 1) / s + 1) / 2 * 2;
      const int64_t parts = (nk + steps - 1) / steps;
      double us = (double)((tiles(f.bm, f.bn) * parts + 255) / 256 * steps) * f.step_us;
      if (parts > 1) us += 3.0 + 2e-6 * (double)(parts * M * N);
      if (us >= best) continue;
      best = us;
      p.bm = f.bm;
      p.bn = f.bn;
      p.splits = (int)parts;
      p.steps = (int)steps;
    }
  return p;
}

template <int MG, int NG, int kU>
void launch_rows(GemmArgs g, hipStream_t st) {
  g.mt = (int)((g.M + 16 * MG - 1) / (16 * MG));
  const int64_t nt = (g.N + 16 * NG - 1) / (16 * NG);
  hipLaunchKernelGGL((k_mx_gemm_rows<MG, NG, kU>), dim3((unsigned)(g.mt * nt)), dim3(512), 0, st, g);
}

template <int BM, int BN, int WM, int WN, int kParts, int NST>
void launch_tile(GemmArgs g, hipStream_t st) {
  g.steps *= 2 / kParts;
  g.mt = (int)((g.M + BM - 1) / BM);
  g.nt = (int)((g.N + BN - 1) / BN);
  const int per = (g.mt * g.nt * g.splits + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((k_mx_gemm<BM, BN, WM, WN, kParts, NST>), dim3(per * kXcds), dim3(64 * WM * WN), 0, st,
                     g);
}

}  // namespace

size_t gemm_mxfp4_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const int splits = plan(M, N, K).splits;
  return splits > 1 ? (size_t)splits * (size_t)M * (size_t)up4(N) * 4 : 0;
}

hipError_t launch_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                             const uint8_t* sa, int64_t ldsa, const uint8_t* b, int64_t ldb,
                             const uint8_t* sb, int64_t ldsb, void* c, int64_t ldc, int c_f32,
                             int accumulate, void* ws, hipStream_t st) {
  const Plan p = plan(M, N, K);
  GemmArgs g{a, b, sa, sb, c, lda, ldb, ldsa, ldsb, ldc, M, N, K, 0, 0, p.splits, p.steps, c_f32,
             accumulate};
  if (p.splits > 1) {
    g.c = ws;
    g.ldc = up4(N);
  }
  if (p.bn == 16) {
    if (p.bm == 16) launch_rows<1, 1, 4>(g, st);
    else launch_rows<2, 1, 4>(g, st);
  } else if (p.bn == 32) {
    launch_rows<2, 2, 4>(g, st);
  } else if (p.bn == 64) {
    if (p.bm == 64) launch_tile<64, 64, 2, 2, 2, 6>(g, st);
    else launch_tile<128, 64, 2, 2, 2, 4>(g, st);
  } else if (p.bn == 128) {
    launch_tile<128, 128, 4, 2, 2, 4>(g, st);
  } else {
    if (p.bm == 128) launch_tile<128, 256, 2, 4, 1, 4>(g, st);
    else launch_tile<256, 256, 4, 2, 1, 4>(g, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t blocks = (M * (up4(N) / 4) + 255) / 256;
  hipLaunchKernelGGL(k_mx_join, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                     st, static_cast<const float*>(ws), p.splits, M, N, up4(N), c, ldc, c_f32,
                     accumulate);
  return hipGetLastError();
}

}  // namespace moe
