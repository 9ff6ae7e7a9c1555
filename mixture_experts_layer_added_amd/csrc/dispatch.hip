// A share of the experts (first .. first + count - 1, one GPU's): the (token, choice) pairs that
// chose one of them sorted by expert, the tokens' rows sent there with or without their weights,
// the experts' rows back, and the gradients of both ways.
//
// Sorting: a pair p = t K + k of local expert e gets row offsets[e] + (pairs of e before p), -1
// where its expert is not here.  Ranks come from one 64-bit mask per (wave, expert), a lane's bit a
// pair, so any index may occur any number of times and no order of atomics shows.
//   k_sort_small: up to 1024 pairs, one workgroup, one launch.
//   k_sort_count (1024 pairs a workgroup), k_sort_scan (a workgroup an expert; up to 64 workgroups of
//     pairs sum the counts themselves), k_sort_place.
//   512 pairs 3.3 us, 18,822 pairs 8 in two launches: latency, of the barriers of ranking and
//   scanning in the one, of the second launch in the other.
// Moving: everything goes by token, one read or write of a token's own row and one of each of its
// rows among the experts':
//   k_spread: rows[r] = w t;  with the rows' partner given also dw = <t, partner[r]>
//   k_gather: t = sum w rows[r];  with the token's partner given also dw = <partner, rows[r]>
// Sums and dots in fp32, in the order of the choices; a row is rounded once.
// Memory bounds them: T = 4096, K = 8, H = 7168 in bf16, k_gather 86 us (6.1 TB/s of 529 MB, mostly
// reads), k_spread with dots 208 us (4.8 TB/s of 1 GB; a copy reaches 5.0).  T = 3137, K = 6, H = 2000
// in fp32, half of the pairs here: 22 us, with dots 28.5.
#include <algorithm>

#include "launch_added.h"

namespace moe {
namespace {

constexpr int kPairs = 1024;    // of a sorting workgroup
constexpr int kFewBlocks = 64;  // workgroups whose counts each of them can sum up by itself
constexpr int kMostK = 16, kMostE = 512;

__device__ __forceinline__ int local_expert(const int32_t* __restrict__ idx, int64_t p, int64_t n,
                                            int first, int count) {
  if (p >= n) return -1;
  const int64_t e = (int64_t)idx[p] - first;
  return e >= 0 && e < count ? (int)e : -1;
}

// Ranks of the workgroup's pairs (-1: not here) and, in s_count, its pairs of each expert.
__device__ __forceinline__ int rank_pairs(int e, int count, unsigned long long* mask,
                                          int* s_count) {
  const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63;
  for (int i = tid; i < 16 * count; i += kPairs) mask[i] = 0ull;
  __syncthreads();
  if (e >= 0) atomicOr(&mask[wv * count + e], 1ull << lane);
  __syncthreads();
  int r = -1;
  if (e >= 0) {
    r = __popcll(mask[wv * count + e] & ((1ull << lane) - 1ull));
    for (int w = 0; w < wv; ++w) r += __popcll(mask[w * count + e]);
  }
  for (int i = tid; i < count; i += kPairs) {
    int c = 0;
    for (int w = 0; w < 16; ++w) c += __popcll(mask[w * count + i]);
    s_count[i] = c;
  }
  __syncthreads();
  return r;
}

// s[i] becomes the sum of s[0 .. i] for i < kMostE (entries past count: 0)
__device__ __forceinline__ void scan_experts(int* s) {
  const int i = threadIdx.x;
  for (int d = 1; d < kMostE; d <<= 1) {
    const int v = i >= d && i < kMostE ? s[i - d] : 0;
    __syncthreads();
    if (i < kMostE) s[i] += v;
    __syncthreads();
  }
}

__global__ __launch_bounds__(kPairs) void k_sort_small(const int32_t* __restrict__ idx, int64_t n,
                                                       int K, int first, int count,
                                                       int32_t* __restrict__ offsets,
                                                       int32_t* __restrict__ token,
                                                       int32_t* __restrict__ row) {
  __shared__ unsigned long long mask[16 * kMostE];
  __shared__ int s[kMostE];
  const int tid = threadIdx.x;
  if (tid < kMostE) s[tid] = 0;
  const int e = local_expert(idx, tid, n, first, count);
  const int r = rank_pairs(e, count, mask, s);
  scan_experts(s);
  if (tid < count) offsets[tid + 1] = s[tid];
  if (tid == 0) offsets[0] = 0;
  if (tid < n) {
    const int at = e < 0 ? -1 : (e ? s[e - 1] : 0) + r;
    row[tid] = at;
    if (e >= 0) token[at] = tid / K;
  }
}

__global__ __launch_bounds__(kPairs) void k_sort_count(const int32_t* __restrict__ idx, int64_t n,
                                                       int first, int count, int64_t nb,
                                                       int32_t* __restrict__ blocks,
                                                       int32_t* __restrict__ row) {
  __shared__ unsigned long long mask[16 * kMostE];
  __shared__ int s[kMostE];
  const int64_t p = (int64_t)blockIdx.x * kPairs + threadIdx.x;
  const int r = rank_pairs(local_expert(idx, p, n, first, count), count, mask, s);
  if (p < n) row[p] = r;  // the rank in the workgroup, made a row by k_sort_place
  // by expert where k_sort_scan sums them, else by workgroup
  for (int i = threadIdx.x; i < count; i += kPairs)
    blocks[nb > kFewBlocks ? i * nb + blockIdx.x : (int64_t)blockIdx.x * count + i] = s[i];
}

// an expert's counts [nb] become the sums of those before, its total goes to totals
__global__ __launch_bounds__(256) void k_sort_scan(int32_t* __restrict__ blocks, int64_t nb,
                                                   int32_t* __restrict__ totals) {
  __shared__ int s[4];
  int32_t* p = blocks + blockIdx.x * nb;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int run = 0;
  for (int64_t b0 = 0; b0 < nb; b0 += 256) {
    const int v = b0 + tid < nb ? p[b0 + tid] : 0;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 63) s[wv] = incl;
    __syncthreads();
    int before = run;
    for (int w = 0; w < wv; ++w) before += s[w];
    if (b0 + tid < nb) p[b0 + tid] = before + incl - v;
    run += s[0] + s[1] + s[2] + s[3];
    __syncthreads();
  }
  if (tid == 0) totals[blockIdx.x] = run;
}

__global__ __launch_bounds__(kPairs) void k_sort_place(const int32_t* __restrict__ idx, int64_t n,
                                                       int K, int first, int count, int64_t nb,
                                                       const int32_t* __restrict__ blocks,
                                                       const int32_t* __restrict__ totals,
                                                       int32_t* __restrict__ offsets,
                                                       int32_t* __restrict__ token,
                                                       int32_t* __restrict__ row) {
  __shared__ int s[kMostE], s_before[kMostE];
  const int tid = threadIdx.x;
  if (nb > kFewBlocks) {
    if (tid < kMostE) s[tid] = tid < count ? totals[tid] : 0;
  } else if (tid < kMostE) {  // a thread an expert: its total, and what lies before this workgroup
    int sum = 0, before = 0;
    if (tid < count) {
#pragma unroll 8
      for (int b = 0; b < (int)nb; ++b) {
        const int v = blocks[b * count + tid];
        sum += v;
        if (b < (int)blockIdx.x) before += v;
      }
    }
    s[tid] = sum;
    s_before[tid] = before;
  }
  __syncthreads();
  scan_experts(s);
  if (blockIdx.x == 0) {
    if (tid < count) offsets[tid + 1] = s[tid];
    if (tid == 0) offsets[0] = 0;
  }
  const int64_t p = (int64_t)blockIdx.x * kPairs + tid;
  const int e = local_expert(idx, p, n, first, count);
  if (e < 0) return;
  const int before = nb > kFewBlocks ? blocks[e * nb + blockIdx.x] : s_before[e];
  const int at = (e ? s[e - 1] : 0) + before + row[p];
  row[p] = at;
  token[at] = (int)(p / K);
}

__global__ void k_no_pairs(int32_t* __restrict__ offsets, int count) {
  for (int i = threadIdx.x; i <= count; i += blockDim.x) offsets[i] = 0;
}

// ---- moving rows ----
// 16 bytes of a row as they lie in memory, n elements of them there (zeros behind)
template <bool kVec>
__device__ __forceinline__ u32x4 get(const uint16_t* __restrict__ p, int n) {
  u32x4 u = {0, 0, 0, 0};
  if (kVec && n >= 8) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) u[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return u;
}
template <bool kVec>
__device__ __forceinline__ u32x4 get(const float* __restrict__ p, int n) {
  u32x4 u = {0, 0, 0, 0};
  if (kVec && n >= 4) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) u[i] = __float_as_uint(p[i]);
  return u;
}
__device__ __forceinline__ float value(const u32x4& u, int i, const uint16_t*) {
  return __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
}
__device__ __forceinline__ float value(const u32x4& u, int i, const float*) {
  return __uint_as_float(u[i]);
}
// bf16 bits of a number to nearest even; NaN stays one
__device__ __forceinline__ uint32_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  return f != f ? (u >> 16 | 0x40u) : (uint32_t)f32_to_bf16_bits(f);
}
template <bool kVec>
__device__ __forceinline__ void put(uint16_t* __restrict__ p, int n, const float* v) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_bf16(v[2 * i]) | to_bf16(v[2 * i + 1]) << 16;
  if (kVec && n >= 8) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
template <bool kVec>
__device__ __forceinline__ void put(float* __restrict__ p, int n, const float* v) {
  if (kVec && n >= 4) {
    const u32x4 u = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}

struct MoveArgs {
  int64_t T, H;
  int K;
  const int32_t* row;  // [T, K]
  const float* w;      // [T, K] or nullptr (1)
  float* dw;           // [T, K] or nullptr
  const void *tok, *rows, *partner;
  void* out;
  int64_t ld_tok, ld_rows, ld_partner, ld_out;
};

constexpr int kMove = 128;  // threads: 16 bytes each, 1024 bf16 elements a turn

// dots of the workgroup's threads, one a choice, to dw of a token (0 where there is no row)
template <int kK>
__device__ __forceinline__ void write_dots(const float* dot, const int* rows, int K, float* dw) {
  __shared__ float red[2][kK];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    if (k < K) {
      float v = dot[k];
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
      if (lane == 0) red[wv][k] = rows[k] < 0 ? 0.0f : v;
    }
  }
  __syncthreads();
  if (tid < K) dw[tid] = red[0][tid] + red[1][tid];
  __syncthreads();
}

// kSpread: out = rows, tok the tokens' rows, partner (kDot) the experts' rows of the dots.
// Else (gather): out = the tokens' rows, rows the experts', partner (kDot) the tokens' of the dots.
// With dots a workgroup takes a token, else a token's slice of kMove chunks of 16 bytes, the slices of
// a token next to each other, so that its rows' pieces are read together.  All rows' loads of a turn
// are on their way before the first is used.  kK >= K choices.
template <typename T, int kK, bool kVec, bool kSpread, bool kDot>
__global__ __launch_bounds__(kMove) void k_move(MoveArgs g) {
  constexpr int N = 16 / sizeof(T);
  const T* type = nullptr;
  const int64_t slices = kDot ? 1 : (g.H + kMove * N - 1) / (kMove * N);
  const int64_t work = g.T * slices;
  for (int64_t b = blockIdx.x; b < work; b += gridDim.x) {
    const int64_t t = b / slices;
    int row[kK];
    float w[kK], dot[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      row[k] = k < g.K ? g.row[t * g.K + k] : -1;
      w[k] = k < g.K && g.w ? g.w[t * g.K + k] : 1.0f;
      dot[k] = 0.0f;
    }
    const int64_t c0 = kDot ? 0 : (b - t * slices) * kMove * N;
    const int64_t c1 = kDot ? g.H : min(g.H, c0 + kMove * N);
    for (int64_t c = c0 + threadIdx.x * N; c < c1; c += kMove * N) {
      const int n = (int)min((int64_t)N, g.H - c);
      u32x4 u[kK], x = {0, 0, 0, 0};
      if constexpr (kSpread) x = get<kVec>(static_cast<const T*>(g.tok) + t * g.ld_tok + c, n);
      else if constexpr (kDot)
        x = get<kVec>(static_cast<const T*>(g.partner) + t * g.ld_partner + c, n);
      if constexpr (kDot || !kSpread) {
        const T* p = static_cast<const T*>(kSpread ? g.partner : g.rows) + c;
        const int64_t ld = kSpread ? g.ld_partner : g.ld_rows;
#pragma unroll
        for (int k = 0; k < kK; ++k)
          if (row[k] >= 0) u[k] = get<kVec>(p + row[k] * ld, n);
      }
      float s[N];
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = 0.0f;
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        if (row[k] < 0) continue;
        if constexpr (kDot) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            dot[k] = __builtin_fmaf(value(x, i, type), value(u[k], i, type), dot[k]);
        }
        if constexpr (kSpread) {
          float o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = w[k] * value(x, i, type);
          put<kVec>(static_cast<T*>(g.out) + row[k] * g.ld_out + c, n, o);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) s[i] = __builtin_fmaf(w[k], value(u[k], i, type), s[i]);
        }
      }
      if constexpr (!kSpread) put<kVec>(static_cast<T*>(g.out) + t * g.ld_out + c, n, s);
    }
    if constexpr (kDot) write_dots<kK>(dot, row, g.K, g.dw + t * g.K);
  }
}

bool whole16(const void* p, int64_t ld, size_t es) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * es % 16 == 0);
}

template <typename T, int kK, bool kSpread>
hipError_t move(const MoveArgs& g, hipStream_t st) {
  const bool vec = whole16(g.tok, g.ld_tok, sizeof(T)) && whole16(g.rows, g.ld_rows, sizeof(T)) &&
                   whole16(g.partner, g.ld_partner, sizeof(T)) &&
                   whole16(g.out, g.ld_out, sizeof(T));
  const int64_t per = kMove * (16 / sizeof(T));
  const int64_t work = g.T * (g.dw ? 1 : (g.H + per - 1) / per);
  const dim3 grid((unsigned)std::min<int64_t>(work, 1 << 20));
  auto k = g.dw ? (vec ? k_move<T, kK, true, kSpread, true> : k_move<T, kK, false, kSpread, true>)
                : (vec ? k_move<T, kK, true, kSpread, false> : k_move<T, kK, false, kSpread, false>);
  hipLaunchKernelGGL(k, grid, dim3(kMove), 0, st, g);
  return hipGetLastError();
}
template <typename T, bool kSpread>
hipError_t move(const MoveArgs& g, hipStream_t st) {
  return g.K <= 8 ? move<T, 8, kSpread>(g, st) : move<T, kMostK, kSpread>(g, st);
}

}  // namespace

size_t sort_ws_bytes(int64_t n, int count) {
  return n <= kPairs ? 0 : sizeof(int32_t) * (size_t)count * ((n + kPairs - 1) / kPairs + 1);
}

hipError_t launch_sort_by_expert(int64_t n, int K, const int32_t* idx, int first, int count,
                                 int32_t* offsets, int32_t* token, int32_t* row, void* ws,
                                 hipStream_t st) {
  if (n == 0) {
    hipLaunchKernelGGL(k_no_pairs, dim3(1), dim3(256), 0, st, offsets, count);
    return hipGetLastError();
  }
  if (n <= kPairs) {
    hipLaunchKernelGGL(k_sort_small, dim3(1), dim3(kPairs), 0, st, idx, n, K, first, count, offsets,
                       token, row);
    return hipGetLastError();
  }
  const int64_t nb = (n + kPairs - 1) / kPairs;
  int32_t* blocks = static_cast<int32_t*>(ws);
  int32_t* totals = blocks + count * nb;
  hipLaunchKernelGGL(k_sort_count, dim3((unsigned)nb), dim3(kPairs), 0, st, idx, n, first, count,
                     nb, blocks, row);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (nb > kFewBlocks) {
    hipLaunchKernelGGL(k_sort_scan, dim3(count), dim3(256), 0, st, blocks, nb, totals);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_sort_place, dim3((unsigned)nb), dim3(kPairs), 0, st, idx, n, K, first, count,
                     nb, blocks, totals, offsets, token, row);
  return hipGetLastError();
}

hipError_t launch_spread(int dtype, int64_t T, int K, int64_t H, const void* tok, int64_t ld_tok,
                         const int32_t* row, const float* w, const void* partner,
                         int64_t ld_partner, void* out, int64_t ld_out, float* dw,
                         hipStream_t st) {
  const MoveArgs g{T, H, K, row, w, dw, tok, nullptr, partner, out, ld_tok, 0, ld_partner, ld_out};
  return dtype == MOE_BF16 ? move<uint16_t, true>(g, st) : move<float, true>(g, st);
}

hipError_t launch_gather(int dtype, int64_t T, int K, int64_t H, const void* rows, int64_t ld_rows,
                         const int32_t* row, const float* w, const void* partner,
                         int64_t ld_partner, void* out, int64_t ld_out, float* dw,
                         hipStream_t st) {
  const MoveArgs g{T, H, K, row, w, dw, nullptr, rows, partner, out, 0, ld_rows, ld_partner, ld_out};
  return dtype == MOE_BF16 ? move<uint16_t, false>(g, st) : move<float, false>(g, st);
}

}  // namespace moe
