// Router backward for a dense gradient of the logits, dz [T, E] (the balance loss gives every
// expert's logit one, not the chosen ones alone):
//   dx[t] = sum_e dz[t,e] W_r[e]      dW_r[e] = sum_t dz[t,e] x[t]
// in fp32 on the 16-bit matrix instructions (2.5 PFLOP/s against 0.16 for fp32 operands): each
// fp32 operand is split once into 16-bit parts whose sum it is, and the products of the parts
// are added in fp32, in a fixed order.
//   dx:  two fp16 parts of dz and of W_r.  A row of dz and a column of W_r are first scaled by
//     a power of two that brings their largest value to [2^14, 2^15): hi = fp16(v), lo =
//     fp16(v - hi) then hold 22 bits of every value within 2^-17 of the largest, and an error
//     under 2^-40 of the largest of smaller ones.  hi hi + lo hi + hi lo leaves out 2^-22 of a
//     product; three products.
//   dW:  bf16 x is taken as it is, dz in three bf16 parts (24 bits, any exponent): three
//     products.  fp32 x in three parts as well, and the six products above 2^-24.
//   k_rd_split: the parts of dz (both kinds) and of W_r, transposed, with their exponents.
//   k_rd_products, 4 waves a workgroup:
//     dx: 128 (or 64) tokens x 128 columns; both operands have k innermost, so a step is 32 of
//       k, both parts (128-byte rows, as in the FP8 product).
//     dW: 128 (or 64) experts x 128 columns, 32 tokens a step (16 for fp32 x); both operands have
//       k outermost and are read with ds_read_b64_tr_b16 (gemm_bwd.hip).  fp32 x is split on
//       its way to LDS (a pass of its own before the products moved 16 bytes an element more:
//       T=8192 H=4096 E=64 143 us).  Split over the tokens; k_rd_join adds the parts in order.
// T=4096 H=7168 E=256, bf16 x: products 91 us (90 GFLOP of parts, 1000 TFLOP/s, the matrix cores
// busy 46% of the time, beside 117 MB of fp32 dx), split 7 us, join 5 us.  T=3137 H=384 E=48, fp32
// x: 18 us, of three launches.
#include <algorithm>

#include "common.h"

namespace moe {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;

constexpr int DBN = 128;       // columns of a tile
constexpr int kRdWaves = 4;    // of a workgroup, 2 x 2
constexpr int kRdLds = 65536;  // a ring of two stages

struct RdArgs {
  const uint16_t *zh, *zp, *wh;
  const void* x;
  const int32_t *ze, *we;
  float *dx, *dw;  // dw: dW or its partial sums [parts, E, H]
  int64_t T, part_rows;
  int H, E, Ep, mt, nt, dw_tiles, dw_blocks;
};

__device__ __forceinline__ uint16_t f16_bits(_Float16 v) {
  return __builtin_bit_cast(uint16_t, v);
}
// exponent that brings |v| < 2^127 to [2^14, 2^15); 0 for 0
__device__ __forceinline__ int lift(float amax) {
  return amax > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(amax) : 0;
}
// Where the fp16 parts of a row's element e stand: 32 hi values, then their 32 lo values, so that
// 128 bytes of a row hold both parts of 32 of k.
__device__ __forceinline__ int pair_at(int e) { return (e >> 5) * 64 + (e & 31); }
// the three bf16 parts of v: each the rounding of what is left
__device__ __forceinline__ void parts3(float v, uint16_t* p) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = f32_to_bf16_bits(v);
    v -= bf16_bits_to_f32(p[i]);
  }
}

// Blocks 0 .. zb-1: 4 rows of dz each, one a wave, a lane's experts 4 adjacent ones of each 256.
// The rest: 32 columns of W_r each, 8 threads a column, kW experts a thread.
template <int kW>
__global__ __launch_bounds__(256) void k_rd_split(
    const float* __restrict__ dz, const float* __restrict__ w, int64_t T, int H, int E, int Ep,
    int64_t zb, uint16_t* __restrict__ zh, uint16_t* __restrict__ zp, int32_t* __restrict__ ze,
    uint16_t* __restrict__ wh, int32_t* __restrict__ we) {
  const int tid = threadIdx.x;
  if (blockIdx.x < zb) {
    const int lane = tid & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (tid >> 6);
    if (t >= T) return;
    constexpr int kG = kW / 32;  // groups of 256 experts
    float v[kG][4], m = 0.0f;
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int e = 256 * j + 4 * lane;
      if ((E & 3) == 0) {
        float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (e < E) r = *reinterpret_cast<const float4*>(dz + t * E + e);
        v[j][0] = r.x; v[j][1] = r.y; v[j][2] = r.z; v[j][3] = r.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = e + i < E ? dz[t * E + e + i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[j][i]));
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
    const int ex = lift(m);
    if (lane == 0) ze[t] = ex;
    const int64_t plane = T * Ep;
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int e = 256 * j + 4 * lane;
      if (e >= Ep) break;
      uint32_t hi[2], lo[2], b[3][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = __builtin_ldexpf(v[j][i], ex);
        const _Float16 h = (_Float16)s;
        const uint32_t hb = f16_bits(h), lb = f16_bits((_Float16)(s - (float)h));
        uint16_t p[3];
        parts3(v[j][i], p);
        const int k = i >> 1, sh = 16 * (i & 1);
        hi[k] = i & 1 ? hi[k] | hb << sh : hb;
        lo[k] = i & 1 ? lo[k] | lb << sh : lb;
#pragma unroll
        for (int n = 0; n < 3; ++n) b[n][k] = i & 1 ? b[n][k] | (uint32_t)p[n] << sh : p[n];
      }
      const int64_t at = t * Ep + e;
      uint16_t* q = zh + t * 2 * Ep + pair_at(e);
      *reinterpret_cast<uint2*>(q) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(q + 32) = make_uint2(lo[0], lo[1]);
#pragma unroll
      for (int n = 0; n < 3; ++n)
        *reinterpret_cast<uint2*>(zp + n * plane + at) = make_uint2(b[n][0], b[n][1]);
    }
    return;
  }
  __shared__ float s_m[8][32];
  __shared__ uint32_t s_t[32][65];  // hi | lo << 16 of 32 columns x 64 experts
  const int c = tid & 31, g = tid >> 5;
  const int h0 = (int)(blockIdx.x - zb) * 32;
  float v[kW], m = 0.0f;
#pragma unroll
  for (int i = 0; i < kW; ++i) v[i] = 8 * i + g < E ? w[(int64_t)(8 * i + g) * H + h0 + c] : 0.0f;
#pragma unroll
  for (int i = 0; i < kW; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
  s_m[g][c] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, s_m[i][c]);
  const int ex = lift(m);
  if (g == 0) we[h0 + c] = ex;
#pragma unroll
  for (int e0 = 0; e0 < 8 * kW; e0 += 64) {
    if (e0 >= Ep) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = __builtin_ldexpf(v[e0 / 8 + i], ex);
      const _Float16 hi = (_Float16)s;
      s_t[c][8 * i + g] = f16_bits(hi) | (uint32_t)f16_bits((_Float16)(s - (float)hi)) << 16;
    }
    __syncthreads();
    // column c2's 64 experts: 8 lanes x 8 of them, both parts
    const int c2 = tid >> 3, l = tid & 7;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = s_t[c2][8 * l + 2 * i], b = s_t[c2][8 * l + 2 * i + 1];
      hi[i] = (a & 0xFFFFu) | b << 16;
      lo[i] = a >> 16 | (b & 0xFFFF0000u);
    }
    uint16_t* q = wh + (int64_t)(h0 + c2) * 2 * Ep + pair_at(e0 + 8 * l);
    *reinterpret_cast<uint4*>(q) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(q + 32) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// tile `work` of mt x nt in bands of 8 row tiles, column-major inside a band
__device__ __forceinline__ void band_tile(int tile, int mt, int nt, int* m, int* n) {
  constexpr int kBand = 8;
  const int band = tile / (kBand * nt), within = tile % (kBand * nt);
  const int rb = min(kBand, mt - band * kBand);
  *m = band * kBand + within % rb;
  *n = within / rb;
}

// 16-byte chunk c of a 128-byte row r
__device__ __forceinline__ int at128(int r, int c) { return r * 128 + ((c ^ (r >> 1)) & 7) * 16; }

// dx: 32 of k a step, hi hi + lo hi + hi lo of (dz, W_r).  The W_r part is the first operand, so
// a lane's results lie in one row.
template <int BM>
__device__ __forceinline__ void rd_dx(char* smem, int block, const uint16_t* __restrict__ zh,
                                      const int32_t* __restrict__ ze,
                                      const uint16_t* __restrict__ wh,
                                      const int32_t* __restrict__ we, float* __restrict__ dx,
                                      int64_t T, int H, int Ep, int mt, int nt) {
  constexpr int W = kRdWaves, WM = 2, WN = 2, SM = BM / WM / 32, SN = DBN / WN / 32;
  constexpr int kStage = (BM + DBN) * 128, NA = BM / 8 / W, NB = DBN / 8 / W;
  static_assert(2 * kStage <= kRdLds, "the ring fits");
  static_assert(W * 32 * (DBN / WN) * 4 <= 2 * kStage, "output staging fits the ring");
  const int total = mt * nt, per = (total + kXcds - 1) / kXcds;
  const int work = (block % kXcds) * per + block / kXcds;
  if (block / kXcds >= per || work >= total) return;
  int mi, ni;
  band_tile(work, mt, nt, &mi, &ni);
  const int64_t m0 = (int64_t)mi * BM;
  const int n0 = ni * DBN;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / WN, wn = wv % WN, fr = lane & 31, kq = lane >> 5;
  const int m_rows = (int)min((int64_t)BM, T - m0);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const uint32_t row_b = 4 * Ep;  // bytes of a row of either operand
  const int lrow = 8 * wv + (lane >> 3);
  const uint32_t lchunk = 16 * ((lane & 7) ^ ((4 * (wv & 1) + (lane >> 4)) & 7));
  const int nk = Ep / 32;
  // rows past T arrive as zeros
  const i32x4 ar = buffer_rsrc(zh + m0 * 2 * Ep, m_rows * row_b);
  const i32x4 br = buffer_rsrc(wh + (int64_t)n0 * 2 * Ep, DBN * row_b);
  auto stage = [&](int kt, int st) {
    const uint32_t dst = lds0 + st * kStage + 8 * wv * 128, ko = (uint32_t)kt * 128;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      load16_to_lds(ar, dst + i * 8 * W * 128, (8 * W * i + lrow) * row_b + lchunk + ko);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      load16_to_lds(br, dst + (BM + i * 8 * W) * 128, (8 * W * i + lrow) * row_b + lchunk + ko);
  };
  f32x16 acc[SM][SN];
#pragma unroll
  for (int m = 0; m < SM; ++m)
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
  stage(0, 0);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vm<0>();
    __syncthreads();
    if (kt + 1 < nk) stage(kt + 1, (kt + 1) & 1);
    const char* as = smem + (kt & 1) * kStage;
    const char* bs = as + BM * 128;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f16x8 a[2][SM], b[2][SN];  // hi, lo
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int m = 0; m < SM; ++m)
          a[p][m] = *reinterpret_cast<const f16x8*>(
              as + at128(wm * (BM / WM) + 32 * m + fr, 4 * p + 2 * s + kq));
#pragma unroll
        for (int n = 0; n < SN; ++n)
          b[p][n] = *reinterpret_cast<const f16x8*>(
              bs + at128(wn * (DBN / WN) + 32 * n + fr, 4 * p + 2 * s + kq));
      }
      // the small products first
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int m = 0; m < SM; ++m)
#pragma unroll
          for (int n = 0; n < SN; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[p >> 1][n], a[p & 1][m],
                                                               acc[m][n], 0, 0, 0);
    }
  }
  __syncthreads();  // every wave is done with the ring, which now stages the output
  constexpr int kCols = DBN / WN, kChunks = kCols / 4, kMask = kChunks < 16 ? kChunks - 1 : 15;
  char* stg = smem + wv * 32 * kCols * 4;
  const int h0 = n0 + wn * kCols;
#pragma unroll
  for (int m = 0; m < SM; ++m) {
    const int64_t row0 = m0 + wm * (BM / WM) + 32 * m;
    const int er = row0 + fr < T ? ze[row0 + fr] : 0;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 32 * n + 8 * q + 4 * kq;
        const int4 ec = *reinterpret_cast<const int4*>(we + h0 + col);
        const f32x16& a = acc[m][n];
        *reinterpret_cast<float4*>(stg + fr * kCols * 4 + (((col / 4) ^ (fr & kMask)) << 4)) =
            make_float4(__builtin_ldexpf(a[4 * q], -er - ec.x),
                        __builtin_ldexpf(a[4 * q + 1], -er - ec.y),
                        __builtin_ldexpf(a[4 * q + 2], -er - ec.z),
                        __builtin_ldexpf(a[4 * q + 3], -er - ec.w));
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int e = lane; e < 32 * kChunks; e += 64) {
      const int r = e / kChunks, ch = e % kChunks;
      const u32x4 v =
          *reinterpret_cast<const u32x4*>(stg + r * kCols * 4 + ((ch ^ (r & kMask)) << 4));
      if (row0 + r < T)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dx + (row0 + r) * H + h0 + 4 * ch));
    }
  }
}

// k-outer stages: rows (tokens) of 256 bytes, 16-byte chunk c of row r at slot c ^ 4 (r & 3).
// A fragment read's lane offset for columns 32 p .. +31 (see gemm_bwd.hip, whose rows have 512
// bytes): 8 consecutive k of a column per lane by two transposing reads.
constexpr int kORow = 256;
__device__ __forceinline__ uint32_t ko_off(int lane, int p) {
  const int g = lane >> 4, j = lane & 15, i = j >> 2;
  const int row = 8 * (g >> 1) + i;
  const int c = 4 * p + 2 * (g & 1) + ((j & 3) >> 1);
  return (uint32_t)(row * kORow + ((c ^ (4 * i)) << 4) + (j & 1) * 8);
}
__device__ __forceinline__ bf16x8 ko_frag(uint32_t addr) {
  typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
  const v4i16 both[2] = {
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)addr),
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(addr + 4 * kORow))};
  bf16x8 f;
  __builtin_memcpy(&f, both, 16);
  return f;
}

// dW partial sums over the tokens of a part: BM experts x 128 columns a workgroup.  XP parts of
// x: 1 (bf16 x itself) or 3 (fp32 x, 8 elements a thread and step, loaded a step before they
// are split into the stage).
template <int BM, int XP>
__device__ __forceinline__ void rd_dw(char* smem, int tile, int part,
                                      const uint16_t* __restrict__ zp,
                                      const void* __restrict__ x, float* __restrict__ out,
                                      int64_t T, int H, int E, int Ep, int64_t part_rows, int nt) {
  constexpr int W = kRdWaves, WM = 2, WN = 2, SM = BM / WM / 32, SN = DBN / WN / 32;
  constexpr int kWStep = XP == 1 ? 32 : 16;  // tokens of a step
  constexpr int kZ = kWStep * kORow;         // a plane of a stage (BM = 64: half used)
  constexpr int kStage = (3 + XP) * kZ;
  constexpr int kI = kWStep / 4 / W;         // load instructions of a plane and wave
  static_assert(2 * kStage <= kRdLds, "the ring fits");
  const int mi = tile / nt, n0 = (tile % nt) * DBN;
  const int64_t t0 = (int64_t)part * part_rows, t1 = min(t0 + part_rows, T);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / WN, wn = wv % WN;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  // instruction i of wave wv fills rows 4 (i W + wv) .. +3; columns past the tile's BM
  // experts (BM = 64) are not loaded
  const int lr = lane >> 4, lc = (lane & 15) ^ (4 * lr);
  auto stage = [&](int64_t t, int st) {
    const int rows = (int)min((int64_t)kWStep, t1 - t);  // later ones arrive as zeros
    const uint32_t dst = lds0 + st * kStage + 4 * wv * kORow;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const i32x4 r = buffer_rsrc(zp + (p * T + t) * Ep, (uint32_t)(rows * Ep * 2));
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const uint32_t o = (uint32_t)((4 * (i * W + wv) + lr) * Ep + mi * BM + 8 * lc) * 2;
        load16_to_lds(r, dst + p * kZ + i * 4 * W * kORow, 8 * lc < BM ? o : 0x7ffffff0u);
      }
    }
    if constexpr (XP == 1) {
      const i32x4 r =
          buffer_rsrc(static_cast<const uint16_t*>(x) + t * H, (uint32_t)(rows * H * 2));
#pragma unroll
      for (int i = 0; i < kI; ++i)
        load16_to_lds(r, dst + 3 * kZ + i * 4 * W * kORow,
                      (uint32_t)((4 * (i * W + wv) + lr) * H + n0 + 8 * lc) * 2);
    }
  };
  // XP == 3: elements 8 (tid % 16) .. +7 of the step's token tid / 16
  const int xr = threadIdx.x >> 4, xc = threadIdx.x & 15;
  float4 xv[2];
  auto load_x = [&](int64_t t) {
    xv[0] = xv[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t + xr < t1) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) +
                                                        (t + xr) * H + n0 + 8 * xc);
      xv[0] = p[0];
      xv[1] = p[1];
    }
  };
  auto split_x = [&](int st) {
    static_assert(XP == 1 || kWStep * 16 == 64 * kRdWaves, "a row's chunk a thread");
    float v[8] = {xv[0].x, xv[0].y, xv[0].z, xv[0].w, xv[1].x, xv[1].y, xv[1].z, xv[1].w};
    char* to = smem + st * kStage + 3 * kZ + xr * kORow + ((xc ^ (4 * (xr & 3))) << 4);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t w[4];  // the hardware's conversion: round to nearest even, as f32_to_bf16_bits
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, bf16x2));
      *reinterpret_cast<uint4*>(to + p * kZ) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] -= __uint_as_float(w[i] << 16);
        v[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  };
  f32x16 acc[SM][SN];
#pragma unroll
  for (int m = 0; m < SM; ++m)
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
  uint32_t oa[SM], ob[SN];
#pragma unroll
  for (int m = 0; m < SM; ++m) oa[m] = ko_off(lane, wm * SM + m);
#pragma unroll
  for (int n = 0; n < SN; ++n) ob[n] = ko_off(lane, wn * SN + n);
  stage(t0, 0);
  if constexpr (XP == 3) {
    load_x(t0);
    split_x(0);
    load_x(t0 + kWStep);
  }
  int st = 0;
  for (int64_t t = t0; t < t1; t += kWStep, st ^= 1) {
    wait_vm<0>();
    __syncthreads();
    if (t + kWStep < t1) {
      stage(t + kWStep, st ^ 1);
      if constexpr (XP == 3) {
        split_x(st ^ 1);
        load_x(t + 2 * kWStep);
      }
    }
    const uint32_t zs = lds0 + st * kStage, xs = zs + 3 * kZ;
#pragma unroll
    for (int s = 0; s < kWStep / 16; ++s) {
      bf16x8 a[3][SM], b[XP][SN];
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int m = 0; m < SM; ++m) a[p][m] = ko_frag(zs + p * kZ + s * 16 * kORow + oa[m]);
#pragma unroll
      for (int p = 0; p < XP; ++p)
#pragma unroll
        for (int n = 0; n < SN; ++n) b[p][n] = ko_frag(xs + p * kZ + s * 16 * kORow + ob[n]);
      // the smallest products first
#pragma unroll
      for (int sum = 2; sum >= 0; --sum)
#pragma unroll
        for (int p = 0; p <= sum; ++p) {
          const int q = sum - p;  // part p of dz, part q of x
          if (q >= XP) continue;
#pragma unroll
          for (int m = 0; m < SM; ++m)
#pragma unroll
            for (int n = 0; n < SN; ++n)
              acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[p][m], b[q][n], acc[m][n], 0, 0, 0);
        }
    }
  }
  // element i of a lane: expert 8 (i/4) + 4 (lane/32) + i%4, column lane%32: 32 lanes store one
  // 128-byte line
#pragma unroll
  for (int m = 0; m < SM; ++m)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = mi * BM + wm * (BM / WM) + 32 * m + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
      if (e >= E) continue;
      float* p = out + ((int64_t)part * E + e) * H + n0 + wn * (DBN / WN) + (lane & 31);
#pragma unroll
      for (int n = 0; n < SN; ++n) p[32 * n] = acc[m][n][i];
    }
}

// Both products in one launch, two workgroups a CU: the first dw_blocks workgroups take dW's
// tiles and parts, the others dx's tiles, whose stores (most of the bytes) then overlap with
// products of either.
template <int BMX, int BMW, int XP>
__global__ __launch_bounds__(64 * kRdWaves, 1) void k_rd_products(RdArgs g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRdLds];
  if ((int)blockIdx.x < g.dw_blocks)
    rd_dw<BMW, XP>(smem, blockIdx.x % g.dw_tiles, blockIdx.x / g.dw_tiles, g.zp, g.x, g.dw, g.T,
                   g.H, g.E, g.Ep, g.part_rows, g.nt);
  else
    rd_dx<BMX>(smem, blockIdx.x - g.dw_blocks, g.zh, g.ze, g.wh, g.we, g.dx, g.T, g.H, g.Ep, g.mt,
               g.nt);
}

__global__ __launch_bounds__(256) void k_rd_join(const float* __restrict__ part, int parts,
                                                 int64_t n, float* __restrict__ dw) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4 s = *reinterpret_cast<const float4*>(part + i);
  int p = 1;
  for (; p + 8 <= parts; p += 8) {  // 8 loads on their way (24 parts: 6.6 us one after another)
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const float4*>(part + (p + u) * n + i);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      s.x += v[u].x; s.y += v[u].y; s.z += v[u].z; s.w += v[u].w;
    }
  }
  for (; p < parts; ++p) {
    const float4 v = *reinterpret_cast<const float4*>(part + p * n + i);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  *reinterpret_cast<float4*>(dw + i) = s;
}

struct RdPlan {
  int Ep, bm;         // experts padded to whole tiles, experts of a k_rd_dw tile
  int parts;          // of the tokens
  int64_t part_rows;
  size_t zh, zp, ze, wh, we, part, bytes;  // byte offsets in the workspace
};

RdPlan rd_plan(const Dims& d) {
  RdPlan p;
  p.bm = d.E <= 64 ? 64 : 128;
  p.Ep = (d.E + p.bm - 1) / p.bm * p.bm;
  // bf16 x and 128 experts a tile: about one workgroup a CU (T=8192 H=1024 E=256 54 us, two 59;
  // T=4096 H=7168 half a one 127 us, one 110); 64 experts, or fp32 x, twice the products: two
  // (T=16384 H=2048 E=64 70 us, one 76; fp32 T=8192 H=4096 E=64 82 us, one 91).  Parts of at
  // least 128 tokens (T=1000 H=1024 E=64, fp32 16 us, of 256 19), where the tiles are many of 512
  // (T=512 H=7168 E=256 24 us, of 256 30), and at most 32 parts (T=16384 H=512 E=100, fp32: 60 us,
  // 64 parts 61, 128 parts 82).
  const bool f32 = d.act == MOE_F32;
  const int64_t tiles = (int64_t)(p.Ep / p.bm) * (d.H / DBN);
  const int64_t steps = (d.T + 31) / 32;
  int64_t s = (f32 || p.bm == 64 ? 512 : 256) / tiles;
  s = std::min(s, std::min<int64_t>(steps / (tiles >= 64 ? 16 : 4), 32));
  if (s < 1) s = 1;
  p.part_rows = (steps + s - 1) / s * 32;
  p.parts = (int)((d.T + p.part_rows - 1) / p.part_rows);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  const size_t TE = (size_t)d.T * p.Ep, HE = (size_t)d.H * p.Ep;
  p.zh = take(TE * 4);
  p.zp = take(TE * 6);
  p.ze = take((size_t)d.T * 4);
  p.wh = take(HE * 4);
  p.we = take((size_t)d.H * 4);
  p.part = take(p.parts > 1 ? (size_t)p.parts * d.E * d.H * 4 : 0);
  p.bytes = at;
  return p;
}

template <int BMX, int BMW, int XP>
void launch_products(RdArgs& g, int parts, hipStream_t st) {
  g.mt = (int)((g.T + BMX - 1) / BMX);
  g.dw_tiles = g.Ep / BMW * g.nt;
  g.dw_blocks = g.dw_tiles * parts;
  const int dx_blocks = (g.mt * g.nt + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((k_rd_products<BMX, BMW, XP>), dim3(g.dw_blocks + dx_blocks),
                     dim3(64 * kRdWaves), 0, st, g);
}
template <int BMX>
void launch_products(RdArgs& g, const RdPlan& p, bool f32, hipStream_t st) {
  if (p.bm == 64) {
    if (f32) launch_products<BMX, 64, 3>(g, p.parts, st);
    else launch_products<BMX, 64, 1>(g, p.parts, st);
  } else {
    if (f32) launch_products<BMX, 128, 3>(g, p.parts, st);
    else launch_products<BMX, 128, 1>(g, p.parts, st);
  }
}

}  // namespace

size_t router_dense_ws_bytes(const Dims& d) { return rd_plan(d).bytes; }

hipError_t launch_router_dense_bwd(const Dims& d, const void* x, const float* w, const float* dz,
                                   float* dx, float* dw, void* ws, hipStream_t st) {
  const RdPlan p = rd_plan(d);
  char* b = static_cast<char*>(ws);
  uint16_t* zh = reinterpret_cast<uint16_t*>(b + p.zh);
  uint16_t* zp = reinterpret_cast<uint16_t*>(b + p.zp);
  int32_t* ze = reinterpret_cast<int32_t*>(b + p.ze);
  uint16_t* wh = reinterpret_cast<uint16_t*>(b + p.wh);
  int32_t* we = reinterpret_cast<int32_t*>(b + p.we);
  const int64_t zb = (d.T + 3) / 4;
  auto split = d.E <= 256 ? k_rd_split<32> : k_rd_split<64>;
  hipLaunchKernelGGL(split, dim3((unsigned)(zb + d.H / 32)), dim3(256), 0, st, dz, w, d.T,
                     d.H, d.E, p.Ep, zb, zh, zp, ze, wh, we);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool f32 = d.act == MOE_F32;
  float* out = p.parts > 1 ? reinterpret_cast<float*>(b + p.part) : dw;
  RdArgs g{zh, zp, wh, x, ze, we, dx, out, d.T, p.part_rows, d.H, d.E, p.Ep, 0, d.H / DBN, 0, 0};
  // 128 tokens a tile of dx once that gives every CU one (T=4096 H=7168 E=256: 110 us, with 64
  // tokens 120; T=128: 14.8 us with 64, 16.8 with 128)
  if ((d.T + 127) / 128 * g.nt >= 256) launch_products<128>(g, p, f32, st);
  else launch_products<64>(g, p, f32, st);
  if ((e = hipGetLastError()) != hipSuccess || p.parts == 1) return e;
  const int64_t n = (int64_t)d.E * d.H;
  hipLaunchKernelGGL(k_rd_join, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, out,
                     p.parts, n, dw);
  return hipGetLastError();
}

}  // namespace moe
