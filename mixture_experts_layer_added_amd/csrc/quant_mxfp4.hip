// MXFP4 quantisation of matrices of any size, along the rows, along the columns (written
// transposed), or both from one read of the matrix, and the values of quantised matrices again.
// A code is off by at most half a step: a quarter of the value where that is at least its scale
// (1/2, 1, 2 are the steps of 0 .. 2, 2 .. 4, 4 .. 6), a quarter of the scale below.
// Each element is read once and each code written once.
//   k_mx_rows: 4 lanes take a block of 32 columns, 8 elements a lane.  128 x 7168 bf16: 3.0 us, a
//     launch and one round of loads (its 2.3 MB would take 0.5).  4099 x 7168: 17 us, 4.3 TB/s of 74
//     MB; with random bytes 24, 4.3 TB/s.
//   k_mx_tile: a workgroup takes 128 x 64 elements through LDS and writes both orders.  4099 x 7168
//     bf16 with random bytes: 43 us, 2.8 TB/s of its 119 MB (24 us at a copy's rate).  The waits
//     between its passes bind it (memory, LDS, LDS, memory) with 6 workgroups to a CU by their LDS;
//     the vector unit is busy for under half of the time.  Stochastic rounding an element at a time,
//     8 operations where the conversion takes 4, took 45, tiles of 64 x 64 50.  To the nearest 32; the
//     transposed form alone 22, with random bytes 32.
//   Rows that do not begin at multiples of 16 bytes are read element by element (random bytes whose row
//     does not begin at a multiple of 8 one by one): rows of 7169 elements, 40 us for the rows, 50 for
//     the transposed form, 58 for both, with random bytes 44, 62 and 73.
//   k_mx_values: 8 values a lane.  7168 x 4099 to bf16, rows at odd 2-byte starts: 20.5 us for 74 MB;
//     4099 x 7168, rows at 16 bytes: 14.8, 5.0 TB/s.
#include <algorithm>

#include "mxfp4.h"

namespace moe {
namespace {

constexpr int kTileR = 128, kTileC = 64;  // of k_mx_tile

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// 8 elements from p, zeros from the n-th on
template <bool kVec>
__device__ __forceinline__ void read8(const uint16_t* __restrict__ p, int n, float* v) {
  if (kVec && n >= 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_bits_to_f32(p[i]) : 0.0f;
  }
}
template <bool kVec>
__device__ __forceinline__ void read8(const float* __restrict__ p, int n, float* v) {
  if (kVec && n >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}
// 8 random bytes, the first n of them there, as mx_code_random takes them
template <typename T>
__device__ __forceinline__ uint2 read8r(const uint8_t* __restrict__ p, int n) {
  constexpr uint32_t kFlip = sizeof(T) == 2 ? 0xffffffffu : 0u;
  uint32_t w[2] = {0, 0};
  if (n >= 8 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  }
  return make_uint2(w[0] ^ kFlip, w[1] ^ kFlip);
}

__device__ __forceinline__ uint32_t max8(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

// the larger of the magnitudes of two pairs, a pair's each by itself, as bits
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b & 0x7fff7fffu);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}

// the bytes that sel takes of r[0], r[1] and of r[2], r[3]
__device__ __forceinline__ uint32_t bytes_of(const uint32_t* r, uint32_t sel) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(r[3], r[2], sel),
                               __builtin_amdgcn_perm(r[1], r[0], sel), 0x05040100u);
}

// 8 codes of one block, whose scale code is sc
template <typename T, bool kRandom>
__device__ __forceinline__ uint32_t codes8(const float* v, uint32_t sc, uint2 r) {
  if (sc == 255) return 0;
  if (!kRandom) return mx_pack8(v, mx_scale(sc));
  if (sizeof(T) == 2) return mx_pack8_random(v, sc, r);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w |= mx_code_random(v[i], sc, ((i < 4 ? r.x : r.y) >> (8 * (i & 3))) & 255u) << (4 * i);
  return w;
}

template <typename T, bool kVec, bool kRandom>
__global__ __launch_bounds__(256) void k_mx_rows(const T* __restrict__ x, int64_t rows,
                                                 int64_t cols, int64_t ldx,
                                                 const uint8_t* __restrict__ rnd,
                                                 uint8_t* __restrict__ q, int64_t ldq,
                                                 uint8_t* __restrict__ scale, int64_t lds,
                                                 int64_t kb) {
  const int l = threadIdx.x & 3;
  const int64_t total = rows * kb, stride = (int64_t)gridDim.x * 64;
  for (int64_t g = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 2); g < total; g += stride) {
    const int64_t r = (uint64_t)total >> 32 ? g / kb : (int64_t)((uint32_t)g / (uint32_t)kb);
    const int64_t b = g - r * kb, c = b * kMxBlock + 8 * l;
    const int n = (int)max((int64_t)0, min((int64_t)8, cols - c));
    float v[8];
    read8<kVec>(x + r * ldx + c, n, v);
    uint2 rb = make_uint2(0, 0);
    if (kRandom) rb = read8r<T>(rnd + r * cols + c, n);
    uint32_t m = max8(v);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const uint32_t sc = mx_scale_code<kRandom>(m);
    *reinterpret_cast<uint32_t*>(q + r * ldq + 16 * b + 4 * l) = codes8<T, kRandom>(v, sc, rb);
    if (l == 0) scale[r * lds + b] = (uint8_t)sc;
  }
}

template <typename T>
struct Pair;
template <>
struct Pair<uint16_t> {
  typedef uint32_t type;
  static __device__ __forceinline__ float lo(uint32_t p) { return __uint_as_float(p << 16); }
  static __device__ __forceinline__ float hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }
};
template <>
struct Pair<float> {
  typedef float2 type;
  static __device__ __forceinline__ float lo(const float2& p) { return p.x; }
  static __device__ __forceinline__ float hi(const float2& p) { return p.y; }
};
__device__ __forceinline__ void keep8(uint16_t* p, const float* v) {  // exact: v came as bf16
  uint4 o;
  uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __float_as_uint(v[2 * i]) >> 16 | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void keep8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// 128 x 64 elements a workgroup.  Rows: 8 lanes a row, 8 elements a lane, which also go to LDS as
// they are.  Columns: half h of wave w takes rows 32 w + 16 h .. +15, a lane two adjacent columns; the
// halves share a block's maximum.  Row r lies at r ^ (r / 16 & 1), so that the halves' rows lie in
// different banks.
template <typename T, bool kVec, bool kRandom>
__global__ __launch_bounds__(256) void k_mx_tile(const T* __restrict__ x, int64_t rows,
                                                 int64_t cols, int64_t ldx,
                                                 const uint8_t* __restrict__ rnd,
                                                 uint8_t* __restrict__ q, int64_t ldq,
                                                 uint8_t* __restrict__ scale, int64_t lds,
                                                 uint8_t* __restrict__ qt, int64_t ldqt,
                                                 uint8_t* __restrict__ scale_t, int64_t ldst,
                                                 int64_t nb) {
  typedef Pair<T> P;
  __shared__ __attribute__((aligned(16))) T tile[kTileR * kTileC];
  __shared__ __attribute__((aligned(16))) uint8_t s_r[kRandom ? kTileR * kTileC : 16];
  __shared__ __attribute__((aligned(4))) uint8_t s_sc[kTileC][4];  // scales of the columns' blocks
  const int tid = threadIdx.x, l = tid & 7;
  const int64_t rb = blockIdx.x / nb, cb = blockIdx.x - rb * nb;
  const int64_t r0 = rb * kTileR, c0 = cb * kTileC;
  const int n = (int)max((int64_t)0, min((int64_t)8, cols - c0 - 8 * l));
  float v[4][8];
  uint2 rr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 32 * i + (tid >> 3);
    const int nr = r < rows ? n : 0;
    read8<kVec>(x + r * ldx + c0 + 8 * l, nr, v[i]);
    rr[i] = make_uint2(0, 0);
    if (kRandom) rr[i] = read8r<T>(rnd + r * cols + c0 + 8 * l, nr);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = 32 * i + (tid >> 3), to = at ^ (at >> 4 & 1);
    const int64_t r = r0 + at;
    keep8(tile + to * kTileC + 8 * l, v[i]);
    if (kRandom) *reinterpret_cast<uint2*>(s_r + to * kTileC + 8 * l) = rr[i];
    if (!q) continue;
    uint32_t m = max8(v[i]);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const int64_t c = c0 + 8 * (l & ~3);  // the block's first column
    if (r < rows && c < cols) {
      const uint32_t sc = mx_scale_code<kRandom>(m);
      *reinterpret_cast<uint32_t*>(q + r * ldq + (c0 + 8 * l) / 2) =
          codes8<T, kRandom>(v[i], sc, rr[i]);
      // both blocks' scales in one store (lds is a multiple of 16, the first block even)
      const uint32_t next = (uint32_t)__shfl_down((int)sc, 4);
      uint8_t* to_scale = scale + r * lds + c / kMxBlock;
      if (l == 0 && c + kMxBlock < cols)
        *reinterpret_cast<uint16_t*>(to_scale) = (uint16_t)(sc | next << 8);
      else if (l == 0)
        *to_scale = (uint8_t)sc;
    }
  }
  __syncthreads();
  const int lane = tid & 63, wv = tid >> 6, p = lane & 31, h = lane >> 5;
  typename P::type u[16];
  uint32_t m0 = 0, m1 = 0, both = 0;
  auto row_of = [&](int k) {
    const int r = 32 * wv + 16 * h + k;
    return r ^ (r >> 4 & 1);
  };
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    u[k] = *reinterpret_cast<const typename P::type*>(tile + row_of(k) * kTileC + 2 * p);
    if constexpr (sizeof(T) == 2) {
      both = pair_max(both, u[k]);
    } else {
      m0 = max(m0, abs_bits(P::lo(u[k])));
      m1 = max(m1, abs_bits(P::hi(u[k])));
    }
  }
  if constexpr (sizeof(T) == 2) {
    m0 = both << 16;
    m1 = both & 0xffff0000u;
  }
  m0 = max(m0, (uint32_t)__shfl_xor((int)m0, 32));
  m1 = max(m1, (uint32_t)__shfl_xor((int)m1, 32));
  const uint32_t sc[2] = {mx_scale_code<kRandom>(m0), mx_scale_code<kRandom>(m1)};
  uint32_t w[2][2];
  if (kRandom) {
    const uint32_t s0 = min(sc[0], 254u), s1 = min(sc[1], 254u);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t r[8];  // bytes of the two columns
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = 8 * j + i;
        r[i] = *reinterpret_cast<const uint16_t*>(s_r + row_of(k) * kTileC + 2 * p);
        a[i] = P::lo(u[k]);
        b[i] = P::hi(u[k]);
      }
      uint2 ra, rb;
      ra = make_uint2(bytes_of(r, 0x0c0c0400u), bytes_of(r + 4, 0x0c0c0400u));
      rb = make_uint2(bytes_of(r, 0x0c0c0501u), bytes_of(r + 4, 0x0c0c0501u));
      w[0][j] = codes8<T, true>(a, s0, ra);
      w[1][j] = codes8<T, true>(b, s1, rb);
    }
  } else {
    const float s0 = mx_scale(sc[0]), s1 = mx_scale(sc[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = P::lo(u[8 * j + i]);
        b[i] = P::hi(u[8 * j + i]);
      }
      w[0][j] = mx_pack8(a, s0);
      w[1][j] = mx_pack8(b, s1);
    }
  }
  __syncthreads();
  // every wave has its part of the tile in registers: the tile's memory now takes the codes, 64
  // bytes a column (16-byte chunks swizzled by the column's pair), so that 4 lanes write 64 bytes
  char* codes = reinterpret_cast<char*>(tile);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int cc = 2 * p + j;
    const bool nan = sc[j] == 255;
    *reinterpret_cast<uint2*>(codes + cc * 64 + ((wv ^ (p & 3)) << 4) + 8 * h) =
        make_uint2(nan ? 0 : w[j][0], nan ? 0 : w[j][1]);
    if (h == j) s_sc[cc][wv] = (uint8_t)sc[j];
  }
  __syncthreads();
  const int ch = tid & 3, cc = tid >> 2;
  if (r0 + kMxBlock * ch >= rows || c0 + cc >= cols) return;
  // four blocks' scales in one store
  uint8_t* to_scale = scale_t + (c0 + cc) * ldst + r0 / kMxBlock;
  if (r0 + 3 * kMxBlock >= rows) to_scale[ch] = s_sc[cc][ch];
  else if (ch == 0) *reinterpret_cast<uint32_t*>(to_scale) = *reinterpret_cast<uint32_t*>(s_sc[cc]);
  *reinterpret_cast<uint4*>(qt + (c0 + cc) * ldqt + r0 / 2 + 16 * ch) =
      *reinterpret_cast<const uint4*>(codes + cc * 64 + ((ch ^ ((cc >> 1) & 3)) << 4));
}

// values of 8 codes: exact in bf16 too (two significant bits, at least 2^-128), NaN for scale 255
__device__ __forceinline__ void put8(uint16_t* __restrict__ p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __float_as_uint(v[2 * i]) >> 16 | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* __restrict__ p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put1(uint16_t* __restrict__ p, float v) {
  *p = (uint16_t)(__float_as_uint(v) >> 16);
}
__device__ __forceinline__ void put1(float* __restrict__ p, float v) { *p = v; }

// A lane takes 8 outputs that begin at a multiple of 16 bytes in memory.  kShift: wherever the row
// begins, so that up to 7 of the first ones lie before it; a lane's codes are then 8 of the 16 around
// them, and may lie in two blocks.
template <typename T, bool kShift>
__global__ __launch_bounds__(256) void k_mx_values(int64_t rows, int64_t cols,
                                                   const uint8_t* __restrict__ q, int64_t ldq,
                                                   const uint8_t* __restrict__ scale, int64_t lds,
                                                   T* __restrict__ out, int64_t ldo) {
  constexpr int kEl = kShift ? 16 / sizeof(T) : 1;  // elements in 16 bytes
  const int64_t per = (cols + 7 + kEl - 1) / 8, total = rows * per;
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < total; g += stride) {
    const int64_t r = (uint64_t)total >> 32 ? g / per : (int64_t)((uint32_t)g / (uint32_t)per);
    T* row = out + r * ldo;
    const int before = kShift ? (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) % kEl) : 0;
    const int64_t c = (g - r * per) * 8 - before;  // the first of the 8, from -(kEl - 1) on
    if (c >= cols) continue;
    const int64_t last = (cols + kMxBlock - 1) / kMxBlock * 4 - 1;  // dword of codes
    const int64_t d = c >> 3;  // rounds down: -1 for what lies before the row
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(q + r * ldq);
    const uint32_t lo = qr[max(d, (int64_t)0)], hi = before ? qr[min(d + 1, last)] : 0u;
    const uint32_t w = before ? (uint32_t)(((uint64_t)hi << 32 | lo) >> (4 * (int)(c & 7))) : lo;
    const int64_t c0 = max(c, (int64_t)0), c1 = min(c + 7, cols - 1);
    const uint8_t* sr = scale + r * lds;
    const uint32_t sc0 = sr[c0 / kMxBlock], sc1 = before ? sr[c1 / kMxBlock] : sc0;
    const float s0 = sc0 == 255 ? __uint_as_float(0x7fc00000u) : mx_scale(sc0);
    const float s1 = sc1 == 255 ? __uint_as_float(0x7fc00000u) : mx_scale(sc1);
    const int turn = before ? kMxBlock - (int)(c & (kMxBlock - 1)) : 8;  // codes of the first block
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3)};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (i & 1 ? p[i >> 1].y : p[i >> 1].x) * (i < turn ? s0 : s1);
    if (c >= 0 && c + 8 <= cols) {
      put8(row + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= 0 && c + i < cols) put1(row + c + i, v[i]);
    }
  }
}

template <typename T, bool kRandom>
hipError_t quantize(const T* x, int64_t rows, int64_t cols, int64_t ldx, const uint8_t* rnd,
                    uint8_t* q, int64_t ldq, uint8_t* scale, int64_t lds, uint8_t* qt,
                    int64_t ldqt, uint8_t* scale_t, int64_t ldst, hipStream_t st) {
  // 16-byte loads need every row to start at a multiple of 16 bytes
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx * sizeof(T) % 16 == 0;
  if (qt) {
    const int64_t nb = (cols + kTileC - 1) / kTileC, nr = (rows + kTileR - 1) / kTileR;
    auto k = vec ? k_mx_tile<T, true, kRandom> : k_mx_tile<T, false, kRandom>;
    hipLaunchKernelGGL(k, dim3((unsigned)(nb * nr)), dim3(256), 0, st, x, rows, cols, ldx, rnd, q,
                       ldq, scale, lds, qt, ldqt, scale_t, ldst, nb);
  } else {
    const int64_t kb = (cols + kMxBlock - 1) / kMxBlock;
    const int64_t blocks = std::min<int64_t>((rows * kb + 63) / 64, 1 << 20);
    auto k = vec ? k_mx_rows<T, true, kRandom> : k_mx_rows<T, false, kRandom>;
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(256), 0, st, x, rows, cols, ldx, rnd, q,
                       ldq, scale, lds, kb);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                                 const uint8_t* rnd, uint8_t* q, int64_t ldq, uint8_t* scale,
                                 int64_t lds, uint8_t* qt, int64_t ldqt, uint8_t* scale_t,
                                 int64_t ldst, hipStream_t st) {
#define MX_QUANT(T, R)                                                                        \
  return quantize<T, R>(static_cast<const T*>(x), rows, cols, ldx, rnd, q, ldq, scale, lds, qt, \
                        ldqt, scale_t, ldst, st)
  if (dtype == MOE_BF16) {
    if (rnd) MX_QUANT(uint16_t, true);
    MX_QUANT(uint16_t, false);
  }
  if (rnd) MX_QUANT(float, true);
  MX_QUANT(float, false);
#undef MX_QUANT
}

hipError_t launch_dequantize_mxfp4(int64_t rows, int64_t cols, const uint8_t* q, int64_t ldq,
                                   const uint8_t* scale, int64_t lds, void* out, int64_t ldo,
                                   int dtype, hipStream_t st) {
  const int64_t n = rows * ((cols + 14) / 8);
  const dim3 g((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20));
  const int es = dtype == MOE_BF16 ? 2 : 4;
  const bool shift = (reinterpret_cast<uintptr_t>(out) & 15) != 0 || ldo * es % 16 != 0;
#define MX_VALUES(T, S)                                                                          \
  hipLaunchKernelGGL((k_mx_values<T, S>), g, dim3(256), 0, st, rows, cols, q, ldq, scale, lds, \
                     static_cast<T*>(out), ldo)
  if (dtype == MOE_BF16) {
    if (shift) MX_VALUES(uint16_t, true);
    else MX_VALUES(uint16_t, false);
  } else {
    if (shift) MX_VALUES(float, true);
    else MX_VALUES(float, false);
  }
#undef MX_VALUES
  return hipGetLastError();
}

}  // namespace moe
