// E4M3 quantisation of matrices of any size with one fp32 scale per 128 elements, along the
// rows, along the columns (written transposed), or both from one read of the matrix; and the
// 8-bit activation checkpoints of the expert backward, which are the row form.
//   scale = amax/448 over the block (1 where that is 0), code = RNE-saturating E4M3 of
//   x/scale (IEEE division)
// A NaN has a NaN code and no part in amax; an infinity makes the scale infinite, its own code
// NaN and the others 0, so that the whole block comes back as NaN.
// A code's relative rounding error is at most 2^-4 for values above 2^-6 scale; smaller ones
// round to multiples of 2^-9 scale.
// Each element is read once and each code written once.
//   k_quant_rows: 16 lanes take a block of 128 columns, 8 elements a lane (36,864 x 4096 bf16:
//     91 us, 5.0 TB/s; four blocks a turn with their loads ahead of their codes took as long).
//   k_quant_tile: a workgroup takes 128 x 128 elements through LDS and writes both orders
//     (4099 x 7168 bf16, both: 36 us, 3.3 TB/s; two quantisations an element weigh as much as the
//     bytes).
//     fp32: 51 us.
//   k_ckpt_restore: 8 columns of h a lane from the gate and the up codes (36,864 x 4096 to bf16 au
//     and h: 105 us, 5.8 TB/s).
#include <algorithm>

#include "common.h"

namespace moe {
namespace {

constexpr int kQB = 128;  // elements under one scale

__device__ __forceinline__ float block_scale(float amax) {
  const float s = amax / 448.0f;
  return s > 0.0f ? s : 1.0f;  // 0 as well where amax is so small that the quotient is 0
}

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

__device__ __forceinline__ float amax8(const float* v) {  // fmax passes a NaN by
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
  return m;
}

// A rounded quotient v/d from r, the rounded 1/d: q = v r is within an ulp or so of it, and the
// remainder v - q d, exact in one fused operation, corrects it to the nearest.  r comes in the
// same way from an estimate within an ulp, except where d's mantissa is all ones.  (P.
// Markstein's theorems on division and reciprocals with a fused multiply-add, IBM J. Res. Dev.
// 34, 1990.)  3 operations in place of the 10 of a division, for the codes and for the scale.
// Blocks near the ends of the exponent range, where r or a remainder would not be a normal
// number, of zeros, of NaN alone, with an infinity, or with the mantissa named, are divided
// plainly; there the quotient may pass 448, and is clamped by comparisons, which leave a NaN.
struct Scale {
  float s, r;
  bool plain;
  static __device__ __forceinline__ float quotient(float v, float d, float r) {
    const float q = v * r;
    return __builtin_fmaf(__builtin_fmaf(-q, d, v), r, q);
  }
  __device__ __forceinline__ explicit Scale(float amax) {
    constexpr float k1By448 = 1.0f / 448.0f;
    s = quotient(amax, 448.0f, k1By448);
    const float e = __builtin_amdgcn_rcpf(s);
    r = __builtin_fmaf(__builtin_fmaf(-s, e, 1.0f), e, e);
    plain = !(amax > 0x1p-90f && amax < 0x1p100f) || (__float_as_uint(s) & 0x7fffffu) == 0x7fffffu;
    if (plain) s = block_scale(amax);
  }
  __device__ __forceinline__ float of(float v) const { return quotient(v, s, r); }
  __device__ __forceinline__ float plain_of(float v) const {
    const float q = v / s;
    return q > 448.0f ? 448.0f : q < -448.0f ? -448.0f : q;
  }
  // N groups of 4 codes
  template <int N, typename F>
  __device__ __forceinline__ void codes(F v, uint32_t* w) const {
    if (plain) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(plain_of(v(4 * i)), plain_of(v(4 * i + 1)),
                                                       0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(plain_of(v(4 * i + 2)),
                                                         plain_of(v(4 * i + 3)), lo, true);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = quick(v(4 * i), v(4 * i + 1), v(4 * i + 2), v(4 * i + 3));
  }
  __device__ __forceinline__ uint32_t quick(float a, float b, float c, float d) const {
    // no saturation needed: |v| <= amax and s >= amax/448 (1 - 2^-24), so |v/s| < 448.0001, whose
    // code is 448's (the conversion overflows from 464 on)
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(of(a), of(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(of(c), of(d), w, true);
  }
};

// the codes of v/s to q, whose first n bytes are the row's
__device__ __forceinline__ void write8(uint8_t* __restrict__ q, int n, const float* v,
                                       const Scale& s) {
  uint32_t w[2];
  s.codes<2>([&](int i) { return v[i]; }, w);
  if (n >= 8) {
    *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

template <typename T, bool kVec>
__global__ __launch_bounds__(256) void k_quant_rows(const T* __restrict__ x, int64_t rows,
                                                    int64_t cols, int64_t ldx,
                                                    uint8_t* __restrict__ q, int64_t ldq,
                                                    float* __restrict__ scale, int64_t kb) {
  const int l = threadIdx.x & 15;
  const int64_t total = rows * kb, stride = (int64_t)gridDim.x * 16;
  for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < total; g += stride) {
    const int64_t r = (uint64_t)total >> 32 ? g / kb : (int64_t)((uint32_t)g / (uint32_t)kb);
    const int64_t b = g - r * kb, c = b * kQB + 8 * l;
    const int n = (int)max((int64_t)0, min((int64_t)8, cols - c));
    float v[8];
    read8<kVec>(x + r * ldx + c, n, v);
    float m = amax8(v);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
    const Scale s(m);
    write8(q + r * ldq + c, n, v, s);
    if (l == 0) scale[r * kb + b] = s.s;
  }
}

// 128 x 128 elements a workgroup.  Rows: 16 lanes a row, 8 elements a lane, which also go to
// LDS as they are.  Columns: lane l of wave w takes columns 2 l and 2 l + 1 of rows 32 w .. +31
// (a wave reads whole rows, without bank conflicts), and the waves' maxima meet in LDS.
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

template <typename T, bool kVec>
__global__ __launch_bounds__(256) void k_quant_tile(const T* __restrict__ x, int64_t rows,
                                                    int64_t cols, int64_t ldx,
                                                    uint8_t* __restrict__ q, int64_t ldq,
                                                    float* __restrict__ scale, int64_t kb,
                                                    uint8_t* __restrict__ qt, int64_t ldqt,
                                                    float* __restrict__ scale_t, int64_t kbt) {
  typedef Pair<T> P;
  __shared__ __attribute__((aligned(16))) T tile[kQB * kQB];
  __shared__ float s_m[4][kQB];
  const int tid = threadIdx.x, l = tid & 15;
  const int64_t rb = blockIdx.x / kb, cb = blockIdx.x - rb * kb;
  const int64_t r0 = rb * kQB, c0 = cb * kQB;
  const int n = (int)max((int64_t)0, min((int64_t)8, cols - c0 - 8 * l));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = r0 + 64 * h + 16 * i + (tid >> 4);
      read8<kVec>(x + r * ldx + c0 + 8 * l, r < rows ? n : 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = 64 * h + 16 * i + (tid >> 4);
      const int64_t r = r0 + rr;
      keep8(tile + rr * kQB + 8 * l, v[i]);
      if (!q) continue;
      float m = amax8(v[i]);
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
      if (r < rows) {
        const Scale s(m);
        write8(q + r * ldq + c0 + 8 * l, n, v[i], s);
        if (l == 0) scale[r * kb + cb] = s.s;
      }
    }
  }
  __syncthreads();
  const int lane = tid & 63, wv = tid >> 6;
  typename P::type v[32];
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    v[k] = *reinterpret_cast<const typename P::type*>(tile + (32 * wv + k) * kQB + 2 * lane);
    m0 = __builtin_fmaxf(m0, __builtin_fabsf(P::lo(v[k])));
    m1 = __builtin_fmaxf(m1, __builtin_fabsf(P::hi(v[k])));
  }
  *reinterpret_cast<float2*>(&s_m[wv][2 * lane]) = make_float2(m0, m1);
  __syncthreads();
  // every wave has its part of the tile in registers: the tile's memory now takes the codes, 128
  // bytes a column (16-byte chunks swizzled by the column's pair), so that 8 lanes write a line
  char* codes = reinterpret_cast<char*>(tile);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int cc = 2 * lane + h;
    const int64_t c = c0 + cc;
    const Scale s(__builtin_fmaxf(__builtin_fmaxf(s_m[0][cc], s_m[1][cc]),
                                  __builtin_fmaxf(s_m[2][cc], s_m[3][cc])));
    uint32_t w[8];
    s.codes<8>([&](int i) { return h ? P::hi(v[i]) : P::lo(v[i]); }, w);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(codes + cc * kQB + (((2 * wv + i) ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    if (wv == 0 && c < cols) scale_t[c * kbt + rb] = s.s;
  }
  __syncthreads();
  const int ch = tid & 7;
  const int nr = (int)max((int64_t)0, min((int64_t)16, rows - r0 - 16 * ch));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int cc = 32 * i + (tid >> 3);
    if (c0 + cc >= cols) continue;
    const uint4 u =
        *reinterpret_cast<const uint4*>(codes + cc * kQB + ((ch ^ ((cc >> 1) & 7)) << 4));
    uint8_t* p = qt + (c0 + cc) * ldqt + r0 + 16 * ch;
    if (nr == 16) {
      *reinterpret_cast<uint4*>(p) = u;
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k < nr) p[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
    }
  }
}

// value of each of 4 codes times its scale, rounded to T (the width that the backward reads)
__device__ __forceinline__ void from_codes(uint32_t w, float s, float* v, const uint16_t*) {
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * s;
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * s;
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * s;
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * s;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = bf16_bits_to_f32(f32_to_bf16_bits(v[i]));
}
__device__ __forceinline__ void from_codes(uint32_t w, float s, float* v, const float*) {
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * s;
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * s;
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * s;
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * s;
}
__device__ __forceinline__ void put8(uint16_t* __restrict__ p, const float* v) {
  const uint2 a = pack4_bf16(v[0], v[1], v[2], v[3]), b = pack4_bf16(v[4], v[5], v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void put8(float* __restrict__ p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T>
__global__ __launch_bounds__(256) void k_ckpt_restore(const uint8_t* __restrict__ q,
                                                      const float* __restrict__ scale, int64_t R,
                                                      int I, T* __restrict__ au,
                                                      T* __restrict__ h) {
  const int per = I / 8, kb = 2 * I / kQB;
  const int64_t n = R * per, stride = (int64_t)gridDim.x * 256;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < n; g += stride) {
    const int64_t r = g / per;
    const int c = (int)(g - r * per) * 8;
    const uint8_t* p = q + r * 2 * I + c;
    const uint2 aq = *reinterpret_cast<const uint2*>(p);
    const uint2 uq = *reinterpret_cast<const uint2*>(p + I);
    const float as = scale[r * kb + c / kQB], us = scale[r * kb + (I + c) / kQB];
    float a[8], u[8];
    from_codes(aq.x, as, a, au);
    from_codes(aq.y, as, a + 4, au);
    from_codes(uq.x, us, u, au);
    from_codes(uq.y, us, u + 4, au);
    if (au) {
      put8(au + r * 2 * I + c, a);
      put8(au + r * 2 * I + I + c, u);
    }
    if (h) {
      float hv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[i] = a[i] / (1.0f + __expf(-a[i])) * u[i];
      put8(h + r * I + c, hv);
    }
  }
}

template <typename T>
hipError_t quantize(const T* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q, int64_t ldq,
                    float* scale, uint8_t* qt, int64_t ldqt, float* scale_t, hipStream_t st) {
  const int64_t kb = (cols + kQB - 1) / kQB, kbt = (rows + kQB - 1) / kQB;
  // 16-byte loads need every row to start at a multiple of 16 bytes
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx * sizeof(T) % 16 == 0;
  if (qt) {
    auto k = vec ? k_quant_tile<T, true> : k_quant_tile<T, false>;
    hipLaunchKernelGGL(k, dim3((unsigned)(kb * kbt)), dim3(256), 0, st, x, rows, cols, ldx, q,
                       ldq, scale, kb, qt, ldqt, scale_t, kbt);
  } else {
    const int64_t blocks = std::min<int64_t>((rows * kb + 15) / 16, 1 << 20);
    auto k = vec ? k_quant_rows<T, true> : k_quant_rows<T, false>;
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(256), 0, st, x, rows, cols, ldx, q, ldq,
                       scale, kb);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                               uint8_t* q, int64_t ldq, float* scale, uint8_t* qt, int64_t ldqt,
                               float* scale_t, hipStream_t st) {
  if (dtype == MOE_BF16)
    return quantize(static_cast<const uint16_t*>(x), rows, cols, ldx, q, ldq, scale, qt, ldqt,
                    scale_t, st);
  return quantize(static_cast<const float*>(x), rows, cols, ldx, q, ldq, scale, qt, ldqt, scale_t,
                  st);
}

hipError_t launch_ckpt_restore(const Dims& d, const uint8_t* q, const float* scale, void* au,
                               void* h, hipStream_t st) {
  const int64_t blocks = (d.R() * (d.I / 8) + 255) / 256;
  const dim3 g((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (d.act == MOE_BF16)
    hipLaunchKernelGGL(k_ckpt_restore<uint16_t>, g, dim3(256), 0, st, q, scale, d.R(), d.I,
                       static_cast<uint16_t*>(au), static_cast<uint16_t*>(h));
  else
    hipLaunchKernelGGL(k_ckpt_restore<float>, g, dim3(256), 0, st, q, scale, d.R(), d.I,
                       static_cast<float*>(au), static_cast<float*>(h));
  return hipGetLastError();
}

}  // namespace moe
