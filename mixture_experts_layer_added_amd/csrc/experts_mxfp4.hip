// MXFP4 expert FFN as grouped products over packed weights: per group of rows (one expert's),
//   h = mx(silu(x W1^T) * (x W3^T)),  y = h W2^T,
// activations and weights E2M1 codes with one E8M0 scale per 32, fp32 sums, h rounded to MXFP4 in
// the first product's epilogue (one scale per 32 of its columns), y to bf16.
//
// Packed weights.  A group's matrix (rows x Kd codes) is cut into blocks of 64 rows and steps of
// 128 of k; a (group, block, step) is 4352 contiguous bytes: four fragments 2 n + u of 1 KiB, one
// load instruction each, whose lane l = 32 h + c holds 32 codes of row r(n, c) from
// 128 kt + 64 h + 32 u on, the matrix instruction's operand as it is; then 64 dwords of scales, byte
// 2 n + u of lane l's being the scale of those codes.  Rows: gate/up: half n of block b holds 16
// columns of h, 32 b + 16 n + 8 (q/2) + c % 8 of the gate (q = c / 8 even) or the up matrix (odd),
// so that a lane's results of a sub-tile are the gate and the up values of the same columns, and a
// block's 32 columns share one scale of h; down: 64 b + 32 n + c.
//
// Kernel.  A workgroup of 4 waves takes up to 128 rows of one group x 4 blocks, a wave one block
// and every row: weights go from memory to the operand registers, three steps ahead, and are used
// for all rows; activations (gathered through sorted_token, or in order) go by direct-to-LDS
// loads into a three-slot ring, 256 of k (a 128-byte line a row) a slot, their scales 16 bytes a
// row, 512 of k, at a time.  Two workgroups share a CU.
#include "mxfp4.h"
#include "schedule.h"

namespace moe {
namespace {

using sched::build_costs;
using sched::build_schedule;
using sched::decode_tile;
using sched::kMaxGroups;
using sched::Tile;
using sched::xcd_boundary;

constexpr int kRows = 128;               // rows of a tile
constexpr int kUnit = 4352;              // bytes of a (block, step) of packed weights
constexpr int kSlot = kRows * 128;       // activations of 256 of k
constexpr int kRing = 3 * kSlot;
constexpr int kScSlot = kRows * 16;      // their scales, of 512 of k
constexpr int kDeep = 3;                 // weight steps on their way
constexpr uint32_t kOut = 0x7ffffff0u;   // an offset past every descriptor's range

__device__ __forceinline__ float silu(float a) { return a / (1.0f + __expf(-a)); }

__device__ __forceinline__ int at128(int r, int c) { return r * 128 + ((c ^ (r >> 1)) & 7) * 16; }
__device__ __forceinline__ u32x4 lds16(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((uintptr_t)addr);
}
__device__ __forceinline__ uint32_t lds2(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>((uintptr_t)addr);
}

// row of the natural matrix for row c of half n of block b
__device__ __forceinline__ int weight_row(int b, int n, int c, int I, int swiglu) {
  if (!swiglu) return 64 * b + 32 * n + c;
  const int q = c >> 3;
  return (q & 1 ? I : 0) + 32 * b + 16 * n + 8 * (q >> 1) + (c & 7);
}

// pack: a thread per 16 bytes of the output (272 a unit: 256 of codes, 16 of scales)
__global__ __launch_bounds__(256) void k_mx_pack(const uint8_t* __restrict__ w,
                                                 const uint8_t* __restrict__ scale,
                                                 uint8_t* __restrict__ p, int64_t chunks, int nblk,
                                                 int nk, int rows, int I, int swiglu) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < chunks; e += stride) {
    const int64_t unit = e / 272;
    const int at = (int)(e - unit * 272);
    const int kt = (int)(unit % nk);
    const int64_t gb = unit / nk;
    const int b = (int)(gb % nblk);
    const int64_t row0 = gb / nblk * rows;
    uint4 o;
    if (at < 256) {
      const int n = at >> 7, u = (at >> 6) & 1, h = (at >> 5) & 1, c = at & 31;
      const int64_t r = row0 + weight_row(b, n, c, I, swiglu);
      o = *reinterpret_cast<const uint4*>(w + r * nk * 64 + 64 * kt + 32 * h + 16 * u);
    } else {
      uint32_t* d = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int l = 4 * (at - 256) + i, h = l >> 5, c = l & 31;
        d[i] = 0;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int64_t r = row0 + weight_row(b, n, c, I, swiglu);
          const uint16_t s =
              *reinterpret_cast<const uint16_t*>(scale + r * nk * 4 + 4 * kt + 2 * h);
          d[i] |= (uint32_t)s << (16 * n);
        }
      }
    }
    *reinterpret_cast<uint4*>(p + 16 * e) = o;
  }
}

struct GroupArgs {
  const uint8_t *a, *sa;  // activations and scales: x through `gather`, or h in its own order
  int64_t lda, ldsa;
  int64_t a_rows;         // of x (gather)
  const int32_t *gather, *offsets;
  const uint8_t* w;       // packed
  uint8_t *hq, *hs;       // up: h's codes and scales, rows of ldh and ldhs bytes
  int64_t ldh, ldhs;
  uint16_t* y;            // down: [rows, n_out]
  int NG, Kd, nblk, n_out;
};

// one tile of MS sub-tiles of 32 rows
template <bool kSwiglu, int MS>
__device__ __forceinline__ void mx_group_tile(const GroupArgs& g, int group, int n_idx,
                                              int64_t row0, int m_rows, char* smem, uint32_t lds0,
                                              uint32_t lds_sc) {
  const int lane = threadIdx.x & 63, fr = lane & 31, h = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = g.Kd / 128, ns = (nk + 1) / 2;
  const int b = 4 * n_idx + wv;
  const bool on = b < g.nblk;  // a wave without a block streams the tile's first one
  const uint8_t* wp =
      g.w + ((int64_t)group * g.nblk + (on ? b : 4 * n_idx)) * nk * kUnit + lane * 16;
  const int32_t* gather = g.gather;
  const i32x4 ar = gather ? buffer_rsrc(g.a, (uint32_t)(g.a_rows * g.lda))
                          : buffer_rsrc(g.a + row0 * g.lda, (uint32_t)(m_rows * g.lda));
  const i32x4 sr = gather ? buffer_rsrc(g.sa, (uint32_t)(g.a_rows * g.ldsa))
                          : buffer_rsrc(g.sa + row0 * g.ldsa, (uint32_t)(m_rows * g.ldsa));
  // activations: instruction i of wave wv fills rows 32 i + 8 wv .. +7 of a slot
  const int lchunk = (lane & 7) ^ ((4 * (wv & 1) + (lane >> 4)) & 7);
  uint32_t ao[MS];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const int r = 32 * i + 8 * wv + (lane >> 3);
    ao[i] = r < m_rows ? (uint32_t)((gather ? gather[row0 + r] : r) * g.lda) + 16 * lchunk : kOut;
  }
  // scales: rows 64 (wv & 1) + lane
  const int srow = 64 * (wv & 1) + lane;
  const uint32_t so =
      srow < m_rows ? (uint32_t)((gather ? gather[row0 + srow] : srow) * g.ldsa) : kOut;
  constexpr int kA = MS + 1;  // loads of a wave and slot
  auto aload = [&](int s) {   // 256 of k
    const int sc = min(s, ns - 1);
#pragma unroll
    for (int i = 0; i < MS; ++i)
      load16_to_lds(ar, lds0 + (s % 3) * kSlot + (32 * i + 8 * wv) * 128,
                    ao[i] + (uint32_t)sc * 128);
    // two slots' scales with the even one; the odd one fills an area that nothing reads, so that
    // every slot brings as many loads
    const bool now = (s & 1) == 0;
    load16_to_lds(sr, lds_sc + (now ? ((s >> 1) & 1) * kScSlot + 1024 * (wv & 1) : 2 * kScSlot),
                  so + 16 * (uint32_t)(sc >> 1));
  };
  u32x4 wb[kDeep + 1][4];
  uint32_t ws[kDeep + 1];
  auto wload = [&](int kk, int buf) {
    const uint8_t* p = wp + (int64_t)min(kk, nk - 1) * kUnit;
#pragma unroll
    for (int i = 0; i < 4; ++i) wb[buf][i] = *reinterpret_cast<const u32x4*>(p + i * 1024);
    ws[buf] = *reinterpret_cast<const uint32_t*>(p + 4096 - lane * 12);
  };
  f32x16 acc[MS][2];
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.0f;

  // the order A(0) W(0) A(1) W(1) W(2), then at each slot's start A(s + 2) and before each step
  // W(kk + 3): when slot s begins, A(s) and W(2 s) are the oldest, with A(s + 1) and two steps'
  // weights behind them
  __syncthreads();  // the previous tile's LDS use is over before the ring is refilled
  aload(0);
  wload(0, 0);
  aload(1);
  wload(1, 1);
  wload(2, 2);
  for (int kt = 0; kt < nk; kt += kDeep + 1) {
#pragma unroll
    for (int j = 0; j <= kDeep; ++j) {
      const int kk = kt + j;
      if (kk >= nk) break;
      const int s = kk >> 1;
      if ((j & 1) == 0) {
        wait_vm<kA + 10>();
        __syncthreads();
        aload(s + 2);
      }
      wload(kk + kDeep, (j + kDeep) % (kDeep + 1));
      __builtin_amdgcn_sched_barrier(0);
      if (!on) continue;
      const uint32_t a_at = lds0 + (s % 3) * kSlot;
      const uint32_t s_at =
          lds_sc + ((s >> 1) & 1) * kScSlot + 8 * (s & 1) + 4 * (j & 1) + 16 * fr + 2 * h;
      uint32_t sa[MS];
#pragma unroll
      for (int m = 0; m < MS; ++m) sa[m] = lds2(s_at + 512 * m);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t off = (uint32_t)at128(fr, 4 * (j & 1) + 2 * h + u);
#pragma unroll
        for (int m = 0; m < MS; ++m) {
          const u32x4 a = lds16(a_at + 32 * m * 128 + off);
          if (u == 0) {
            acc[m][0] = mx_mfma32<0, 0>(wb[j][0], a, acc[m][0], ws[j], sa[m]);
            acc[m][1] = mx_mfma32<2, 0>(wb[j][2], a, acc[m][1], ws[j], sa[m]);
          } else {
            acc[m][0] = mx_mfma32<1, 1>(wb[j][1], a, acc[m][0], ws[j], sa[m]);
            acc[m][1] = mx_mfma32<3, 1>(wb[j][3], a, acc[m][1], ws[j], sa[m]);
          }
        }
      }
    }
  }
  wait_vm<0>();
  __syncthreads();  // every wave is done with the ring, which now stages the outputs
  if (!on) return;
  if constexpr (kSwiglu) {
    // a lane holds 16 of its row's 32 columns, 16 n + 8 j + 4 h + i, its partner in the other half
    // of the wave the others; it then writes the 8 bytes of half n = h
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      float v[2][8];
      uint32_t top = 0;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = silu(acc[m][n][8 * j + i]) * acc[m][n][8 * j + 4 + i];
            v[n][4 * j + i] = x;
            top = max(top, __float_as_uint(x) & 0x7fffffffu);
          }
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      const uint32_t sc = mx_scale_code<false>(top);
      uint32_t w[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) w[n] = sc == 255 ? 0 : mx_pack8(v[n], mx_scale(sc));
      // w[n]: columns j = 0 in the low, j = 1 in the high half; exchange half 1 - h
      const uint32_t got = (uint32_t)__shfl_xor((int)(h ? w[0] : w[1]), 32);
      const uint32_t mine = h ? w[1] : w[0];
      const uint32_t lo = h ? got : mine, hi = h ? mine : got;  // of lane half 0 and 1
      const int r = 32 * m + fr;
      if (r < m_rows) {
        *reinterpret_cast<uint2*>(g.hq + (row0 + r) * g.ldh + 16 * b + 8 * h) =
            make_uint2((lo & 0xffffu) | hi << 16, lo >> 16 | (hi & 0xffff0000u));
        if (h == 0) g.hs[(row0 + r) * g.ldhs + b] = (uint8_t)sc;
      }
    }
  } else {
    // 32 rows x 64 bf16 columns, a 128-byte line a row, staged in LDS
    char* stg = smem + wv * 4096;
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2*>(stg + fr * 128 + (((4 * n + q) ^ (fr & 7)) << 4) + h * 8) =
              pack4_bf16(acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2],
                         acc[m][n][4 * q + 3]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 3), ch = lane & 7;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + r * 128 + ((ch ^ (r & 7)) << 4));
        if (32 * m + r < m_rows)
          __builtin_nontemporal_store(
              v, reinterpret_cast<u32x4*>(g.y + (row0 + 32 * m + r) * g.n_out + 64 * b + 8 * ch));
      }
    }
  }
}

template <bool kSwiglu>
__global__ __launch_bounds__(256, 2) void k_mx_group(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRing];
  __shared__ __attribute__((aligned(16))) char s_sc[2 * kScSlot + 1024];
  __shared__ int mt_start[kMaxGroups + 1];
  // the cost prefix is only needed before the first tile's loads overwrite the ring
  long long* s_cost = reinterpret_cast<long long*>(smem);
  static_assert(sizeof(long long) * (kMaxGroups + 1) <= kRing, "cost prefix fits the ring");
  build_schedule(g.offsets, g.NG, kRows, mt_start);
  const int nt = (g.nblk + 3) / 4;
  build_costs(g.offsets, mt_start, g.NG, kRows, nt, s_cost);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const uint32_t lds_sc = __builtin_amdgcn_readfirstlane(lds_offset(s_sc));
  const int per_xcd = gridDim.x / kXcds;
  const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
  const int begin = xcd_boundary(xcd, g.offsets, mt_start, s_cost, g.NG, kRows, nt);
  const int end = xcd_boundary(xcd + 1, g.offsets, mt_start, s_cost, g.NG, kRows, nt);
  for (int tile = begin + slot; tile < end; tile += per_xcd) {
    const Tile tl = decode_tile(tile, mt_start, g.NG, nt);
    const int group = __builtin_amdgcn_readfirstlane(tl.g);
    const int n_idx = __builtin_amdgcn_readfirstlane(tl.n_idx);
    const int m0 = __builtin_amdgcn_readfirstlane(tl.m_idx) * kRows;
    const int first = g.offsets[group];
    const int m_rows = min(kRows, g.offsets[group + 1] - first - m0);
    const int64_t row0 = (int64_t)first + m0;
    switch ((m_rows + 31) >> 5) {
      case 1: mx_group_tile<kSwiglu, 1>(g, group, n_idx, row0, m_rows, smem, lds0, lds_sc); break;
      case 2: mx_group_tile<kSwiglu, 2>(g, group, n_idx, row0, m_rows, smem, lds0, lds_sc); break;
      case 3: mx_group_tile<kSwiglu, 3>(g, group, n_idx, row0, m_rows, smem, lds0, lds_sc); break;
      case 4: mx_group_tile<kSwiglu, 4>(g, group, n_idx, row0, m_rows, smem, lds0, lds_sc); break;
      default: break;
    }
  }
}

int group_grid() { return std::max(device_cu_count() * 2 / kXcds, 1) * kXcds; }

}  // namespace

hipError_t launch_pack_mxfp4(const uint8_t* w, const uint8_t* scale, uint8_t* packed, int64_t batch,
                             int rows, int cols, bool swiglu, hipStream_t st) {
  const int nblk = rows / 64, nk = cols / 128;
  const int64_t chunks = batch * nblk * nk * (kUnit / 16);
  hipLaunchKernelGGL(k_mx_pack, dim3(8192), dim3(256), 0, st, w, scale, packed, chunks, nblk, nk,
                     rows, rows / 2, swiglu ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_ffn_up_mxfp4(const Dims& d, const uint8_t* xq, const uint8_t* xs, int64_t ldxs,
                               const int32_t* gather, const int32_t* offsets, const uint8_t* w,
                               uint8_t* hq, uint8_t* hs, int64_t ldhs, hipStream_t st) {
  GroupArgs g{xq, xs, d.H / 2, ldxs, d.T, gather, offsets, w, hq, hs, d.I / 2, ldhs, nullptr,
              d.E + d.S, d.H, 2 * d.I / 64, d.I};
  hipLaunchKernelGGL(k_mx_group<true>, dim3(group_grid()), dim3(256), 0, st, g);
  return hipGetLastError();
}

hipError_t launch_ffn_down_mxfp4(const Dims& d, const uint8_t* hq, const uint8_t* hs, int64_t ldhs,
                                 const int32_t* offsets, const uint8_t* w, void* y,
                                 hipStream_t st) {
  GroupArgs g{hq, hs, d.I / 2, ldhs, 0, nullptr, offsets, w, nullptr, nullptr, 0, 0,
              static_cast<uint16_t*>(y), d.E + d.S, d.I, d.H / 64, d.H};
  hipLaunchKernelGGL(k_mx_group<false>, dim3(group_grid()), dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace moe
