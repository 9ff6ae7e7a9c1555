// Router backward for a dense gradient of the logits, dz [T, E] (the balance loss gives every
// expert's logit one, not the chosen ones alone):
//   dx[t] = sum_e dz[t,e] W_r[e]      dW_r[e] = sum_t dz[t,e] x[t]
// in fp32 on the bf16 matrix instructions (2.5 PFLOP/s against 0.16 for fp32 operands): each fp32
// operand is split once into three bf16 parts whose sum it is, and the products of the parts
// are added in fp32, in a fixed order, the small ones first.
//   Parts of 8 bits each, every one the rounding of what is left: 24 bits of the value, under 2^-27
//   of it dropped, at any exponent (bf16 has fp32's range), so that a term's error is counted
//   against the term, whatever stands beside it in the row.  (Two fp16 parts under a row's and a
//   column's common exponent took three products in place of six, but kept only 2^-39 of the
//   row's largest value times the column's: nothing of a large dz times a small W_r where the row
//   and the column span 2^30.)
//   Products: those of parts p and q with p + q <= 2, down to 2^-18 of the term; what is left out
//   is below 2^-26.  Six for fp32 times fp32; three for bf16 x, which is one part by itself.
//   k_rd_split: the parts of dz and of W_r, transposed, in the order that both products read:
//     blocks of 32 rows (tokens, or columns of W_r) x 16 experts, a part 1 KB: the first 8 experts
//     of each row, then the other 8.  A lane's operand of a 32 x 32 x 16 product is 16 bytes at 16
//     times its number, in memory and in LDS.
//   k_rd_products, 4 waves a workgroup:
//     dx: 128 (or 64) tokens x 128 columns, 16 experts a step, whole blocks to LDS.
//     dW: 128 (or 64) experts x 128 columns, 32 tokens a step (16 for fp32 x); both operands have
//       k outermost and are read with ds_read_b64_tr_b16 (gemm_bwd.hip).  fp32 x is split on
//       its way to LDS (a pass of its own before the products moved 16 bytes an element more:
//       T=8192 H=4096 E=64 143 us).  Split over the tokens; k_rd_join adds the parts in order.
// T=4096 H=7168 E=256, bf16 x: 139 us; products 120-127 us (135 GFLOP of parts, 1100 TFLOP/s, the
// matrix cores busy 50% of the time, beside 117 MB of fp32 dx; three stages of dx in flight took
// as long as two), split 6 us, join 5 us.  T=3137 H=384 E=48, fp32 x: 17.5 us, of three launches.
#include <algorithm>

#include "common.h"

namespace moe {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

constexpr int DBN = 128;       // columns of a tile
constexpr int kRdWaves = 4;    // of a workgroup, 2 x 2
constexpr int kRdLds = 65536;  // a ring of two stages

struct RdArgs {
  const uint16_t *zp, *wp;  // parts of dz and of W_r
  const void* x;
  float *dx, *dw;  // dw: dW or its partial sums [parts, E, H]
  int64_t T, part_rows;
  int H, E, Ep, mt, nt, dw_tiles, dw_blocks;
};

// the bf16 roundings of two numbers, as the hardware makes them (to nearest even, NaN kept)
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// A number past bf16's largest is not rounded to infinity: its first part is that largest one.
__device__ __forceinline__ float first_part(float v) {
  constexpr float kMost = 0x1.fep127f;
  const float h = __uint_as_float(bf16_pair(v, 0.0f) << 16);
  return __builtin_fabsf(h) > kMost && __builtin_fabsf(v) <= 0x1.fffffep127f
             ? __builtin_copysignf(kMost, v) : h;
}

// A thread takes 8 experts of a row of either operand (a token's of dz, a column's of W_r); 32
// threads take 32 rows, so that a wave writes 1 KB of each part.
__global__ __launch_bounds__(256) void k_rd_split(const float* __restrict__ dz,
                                                  const float* __restrict__ w, int64_t T, int H,
                                                  int E, int Ep, uint32_t zb,
                                                  uint16_t* __restrict__ zp,
                                                  uint16_t* __restrict__ wp) {
  const bool is_w = blockIdx.x >= zb;
  const uint32_t at = (is_w ? blockIdx.x - zb : blockIdx.x) * 256 + threadIdx.x;
  const uint32_t chunk = (at >> 5) % (uint32_t)(Ep / 8), rb = (at >> 5) / (uint32_t)(Ep / 8);
  const int r = at & 31, e = 8 * (int)chunk;
  const int64_t row = (int64_t)rb * 32 + r;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (is_w) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < E) v[i] = w[(int64_t)(e + i) * H + row];
  } else if (row < T) {  // rows past T are zeros
    const float* p = dz + row * E + e;
    if ((E & 3) == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (e + 4 * h < E) {
          const float4 q = *reinterpret_cast<const float4*>(p + 4 * h);
          v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
        }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < E) v[i] = p[i];
    }
  }
  uint16_t* to = (is_w ? wp : zp) +
                 ((int64_t)rb * (Ep / 16) + (chunk >> 1)) * 1536 + (chunk & 1) * 256 + r * 8;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p == 0) {
        const float a = first_part(v[2 * i]), b = first_part(v[2 * i + 1]);
        o[i] = bf16_pair(a, b);
      } else {
        o[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
      }
      v[2 * i] -= __uint_as_float(o[i] << 16);
      v[2 * i + 1] -= __uint_as_float(o[i] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint4*>(to + 512 * p) = make_uint4(o[0], o[1], o[2], o[3]);
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

// dx: 16 experts a step, a stage the tile's blocks of both operands.  The W_r part is the first
// operand, so a lane's results lie in one row.
template <int BM>
__device__ __forceinline__ void rd_dx(char* smem, int block, const uint16_t* __restrict__ zp,
                                      const uint16_t* __restrict__ wp, float* __restrict__ dx,
                                      int64_t T, int H, int Ep, int mt, int nt) {
  constexpr int W = kRdWaves, WM = 2, WN = 2, SM = BM / WM / 32, SN = DBN / WN / 32;
  constexpr int kBA = BM / 32, kBB = DBN / 32;  // blocks of either operand
  constexpr int kStage = (kBA + kBB) * 3072;
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
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const int nk = Ep / 16;
  const uint32_t blk = (uint32_t)nk * 3072;  // bytes of a block of rows
  // blocks past T arrive as zeros
  const int a_blocks = (int)min((int64_t)kBA, (T + 31) / 32 - m0 / 32);
  const i32x4 ar = buffer_rsrc(zp + m0 / 32 * nk * 1536, a_blocks * blk);
  const i32x4 br = buffer_rsrc(wp + (int64_t)(n0 / 32) * nk * 1536, kBB * blk);
  auto stage = [&](int kt, int st) {
    const uint32_t dst = lds0 + st * kStage;
#pragma unroll
    for (int j = 0; j < ((kBA + kBB) * 3 + W - 1) / W; ++j) {
      const int i = j * W + wv;  // 1 KB: part i % 3 of block i / 3
      if (i >= (kBA + kBB) * 3) break;
      const int b = i / 3, p = i - 3 * b;
      const bool is_a = b < kBA;
      load16_to_lds(is_a ? ar : br, dst + i * 1024,
                    (is_a ? b : b - kBA) * blk + (uint32_t)(kt * 3 + p) * 1024 + 16 * lane);
    }
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
    const char* as = smem + (kt & 1) * kStage + 16 * lane;
    bf16x8 a[3][SM], b[3][SN];
#pragma unroll
    for (int p = 2; p >= 0; --p) {
#pragma unroll
      for (int m = 0; m < SM; ++m)
        a[p][m] = *reinterpret_cast<const bf16x8*>(as + ((wm * SM + m) * 3 + p) * 1024);
#pragma unroll
      for (int n = 0; n < SN; ++n)
        b[p][n] = *reinterpret_cast<const bf16x8*>(as + ((kBA + wn * SN + n) * 3 + p) * 1024);
    }
    // the smallest products first
#pragma unroll
    for (int sum = 2; sum >= 0; --sum)
#pragma unroll
      for (int p = 0; p <= sum; ++p)
#pragma unroll
        for (int m = 0; m < SM; ++m)
#pragma unroll
          for (int n = 0; n < SN; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[sum - p][n], a[p][m],
                                                                acc[m][n], 0, 0, 0);
  }
  __syncthreads();  // every wave is done with the ring, which now stages the output
  constexpr int kCols = DBN / WN, kChunks = kCols / 4, kMask = kChunks < 16 ? kChunks - 1 : 15;
  char* stg = smem + wv * 32 * kCols * 4;
  const int h0 = n0 + wn * kCols;
#pragma unroll
  for (int m = 0; m < SM; ++m) {
    const int64_t row0 = m0 + wm * (BM / WM) + 32 * m;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int n = 0; n < SN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 32 * n + 8 * q + 4 * kq;
        const f32x16& a = acc[m][n];
        *reinterpret_cast<float4*>(stg + fr * kCols * 4 + (((col / 4) ^ (fr & kMask)) << 4)) =
            make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
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
    const int rows = (int)min((int64_t)kWStep, t1 - t);  // later ones: zeros, of either operand
    const uint32_t dst = lds0 + st * kStage + 4 * wv * kORow;
    // the step's tokens lie in one block of 32 (parts of the tokens are whole blocks)
    const i32x4 zr = buffer_rsrc(zp + (t >> 5) * (Ep / 16) * 1536, (uint32_t)(Ep / 16) * 3072);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const uint32_t r = (uint32_t)(t & 31) + 4 * (i * W + wv) + lr;
        const uint32_t o = ((uint32_t)(mi * (BM / 16) + (lc >> 1)) * 3 + p) * 1024 +
                           (lc & 1) * 512 + r * 16;
        load16_to_lds(zr, dst + p * kZ + i * 4 * W * kORow, 8 * lc < BM ? o : 0x7ffffff0u);
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
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
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
    rd_dx<BMX>(smem, blockIdx.x - g.dw_blocks, g.zp, g.wp, g.dx, g.T, g.H, g.Ep, g.mt, g.nt);
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
  size_t zp, wp, part, bytes;  // byte offsets in the workspace
};

RdPlan rd_plan(const Dims& d) {
  RdPlan p;
  p.bm = d.E <= 64 ? 64 : 128;
  p.Ep = (d.E + p.bm - 1) / p.bm * p.bm;
  // bf16 x and 128 experts a tile: about one workgroup a CU (T=8192 H=1024 E=256 58 us, two 58, half
  // a one 57; T=4096 H=7168 one 137, half a one 160); 64 experts, or fp32 x, twice the products:
  // two (T=16384 H=7168 E=8 169 us, one 198; fp32 T=8192 H=4096 E=64 78, one 86; but bf16
  // T=16384 H=2048 E=64 69, one 63).  Parts of at least 128 tokens (T=1000 H=1024 E=64, fp32 16
  // us, of 256 19), where the tiles are many of 512 (T=512 H=7168 E=256 28 us, of 256 34), and at
  // most 48 parts (T=16384 H=512 E=100, fp32: 44 us, 32 parts 46, 128 parts 50; T=8192 H=384 E=48,
  // fp32: 20.3, 32 parts 22.7, 128 parts 21).
  const bool f32 = d.act == MOE_F32;
  const int64_t tiles = (int64_t)(p.Ep / p.bm) * (d.H / DBN);
  const int64_t steps = (d.T + 31) / 32;
  int64_t s = (f32 || p.bm == 64 ? 512 : 256) / tiles;
  s = std::min(s, std::min<int64_t>(steps / (tiles >= 64 ? 16 : 4), 48));
  if (s < 1) s = 1;
  p.part_rows = (steps + s - 1) / s * 32;
  p.parts = (int)((d.T + p.part_rows - 1) / p.part_rows);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  p.zp = take((size_t)((d.T + 31) / 32 * 32) * p.Ep * 6);
  p.wp = take((size_t)d.H * p.Ep * 6);
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
  uint16_t* zp = reinterpret_cast<uint16_t*>(b + p.zp);
  uint16_t* wp = reinterpret_cast<uint16_t*>(b + p.wp);
  // Ep is a multiple of 64: a workgroup's 256 threads take 32 rows x 64 experts
  const uint32_t per = p.Ep / 64, zb = (uint32_t)((d.T + 31) / 32) * per;
  hipLaunchKernelGGL(k_rd_split, dim3(zb + d.H / 32 * per), dim3(256), 0, st, dz, w, d.T, d.H,
                     d.E, p.Ep, zb, zp, wp);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool f32 = d.act == MOE_F32;
  float* out = p.parts > 1 ? reinterpret_cast<float*>(b + p.part) : dw;
  RdArgs g{zp, wp, x, dx, out, d.T, p.part_rows, d.H, d.E, p.Ep, 0, d.H / DBN, 0, 0};
  // 128 tokens a tile of dx once that gives every CU one (T=4096 H=7168 E=256: 139 us, with 64
  // tokens 156; T=128: 16.4 us with 64, 19.2 with 128)
  if ((d.T + 127) / 128 * g.nt >= 256) launch_products<128>(g, p, f32, st);
  else launch_products<64>(g, p, f32, st);
  if ((e = hipGetLastError()) != hipSuccess || p.parts == 1) return e;
  const int64_t n = (int64_t)d.E * d.H;
  hipLaunchKernelGGL(k_rd_join, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, out,
                     p.parts, n, dw);
  return hipGetLastError();
}

}  // namespace moe
