// Router backward for a dense gradient of the logits, dz [T, E] (the balance loss gives every
// expert's logit one, not the chosen ones alone):
//   dx[t] = sum_e dz[t,e] W_r[e]      dW_r[e] = sum_t dz[t,e] x[t]
// both in fp32, summed in a fixed order.
#include "common.h"

namespace moe {
namespace {

__device__ __forceinline__ float val(const float* p) { return *p; }
__device__ __forceinline__ float val(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// C[m,n] = sum_k A(m,k) B(k,n), 64 x 64 a workgroup, 4 x 4 a thread, 16 of k a step; A(m,k) at
// m * am + k * ak, B(k,n) at k * ldb + n
template <typename TB>
__global__ __launch_bounds__(256) void k_rd_tile(const float* __restrict__ A, int64_t am,
                                                 int64_t ak, const TB* __restrict__ B,
                                                 int64_t ldb, float* __restrict__ C, int64_t M,
                                                 int64_t N, int64_t K, int64_t mt) {
  __shared__ float as[16][65], bs[16][65];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t m0 = (blockIdx.x % mt) * 64, n0 = (blockIdx.x / mt) * 64;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + 256 * i;
      const int kr = ak == 1 ? e & 15 : e >> 6, mr = ak == 1 ? e >> 4 : e & 63;
      as[kr][mr] = m0 + mr < M && k0 + kr < K ? A[(m0 + mr) * am + (k0 + kr) * ak] : 0.0f;
      const int kc = e >> 6, nc = e & 63;
      bs[kc][nc] = n0 + nc < N && k0 + kc < K ? val(B + (k0 + kc) * ldb + n0 + nc) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_fmaf(as[k][ty + 16 * i], bs[k][tx + 16 * j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < M && n < N) C[m * N + n] = acc[i][j];
    }
}

}  // namespace

size_t router_dense_ws_bytes(const Dims& d) { return 256; }

hipError_t launch_router_dense_bwd(const Dims& d, const void* x, const float* w, const float* dz,
                                   float* dx, float* dw, void* ws, hipStream_t st) {
  const int64_t nt = (d.H + 63) / 64;
  const int64_t mx = (d.T + 63) / 64, mw = (d.E + 63) / 64;
  hipLaunchKernelGGL(k_rd_tile<float>, dim3((unsigned)(mx * nt)), dim3(256), 0, st, dz,
                     (int64_t)d.E, (int64_t)1, w, (int64_t)d.H, dx, d.T, (int64_t)d.H,
                     (int64_t)d.E, mx);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (d.act == MOE_BF16)
    hipLaunchKernelGGL(k_rd_tile<uint16_t>, dim3((unsigned)(mw * nt)), dim3(256), 0, st, dz,
                       (int64_t)1, (int64_t)d.E, static_cast<const uint16_t*>(x), (int64_t)d.H,
                       dw, (int64_t)d.E, (int64_t)d.H, d.T, mw);
  else
    hipLaunchKernelGGL(k_rd_tile<float>, dim3((unsigned)(mw * nt)), dim3(256), 0, st, dz,
                       (int64_t)1, (int64_t)d.E, static_cast<const float*>(x), (int64_t)d.H, dw,
                       (int64_t)d.E, (int64_t)d.H, d.T, mw);
  return hipGetLastError();
}

}  // namespace moe
