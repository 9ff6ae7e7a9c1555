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
// and every row: weights go from memory to the operand registers, three steps ahead (seven where up
// to 64 rows leave the registers for it), and are used for all rows; activations (gathered through
// sorted_token, or in order) go by direct-to-LDS loads into a ring of four slots, 256 of k (a
// 128-byte line a row) a slot, their scales 16 bytes a row, 512 of k, at a time.  Two workgroups
// share a CU.
// 32 + 1 experts of H = 7168, I = 2048, both products and the quantiser, 8 choices a token:
//   16 tokens: 126 to 139 us by card, 5.5 to 6.1 TB/s of 771 MB.  The weights' way from memory bounds it.
//   512 tokens (a tile or two of up to 128 rows a group): 212 to 223 us, up 131 to 138, down 72.  Tiles of
//   128 rows x 256 columns do not fill whole rounds of the chip, and a group with two row tiles reads
//   its weights from the L2 the second time.
//   4096 tokens: 940 to 1015 us by card, 3.2 to 3.4 PFLOP/s, up 556 to 642.  The matrix cores are busy 50%
//   (up) and 39% (down) of the cycles, at 1.55 and 1.63 GHz (2.4 unloaded): half is the clock that the
//   card's power leaves, half are waits; up also fetches 1970 MB, weights and rows read again for row
//   tiles and columns, and a tenth of the cycles are LDS conflicts.
// 256 + 1 experts, the groups found over five rounds of 64: 128 tokens, 230 groups with rows, 915 us, 5.9
// TB/s of weights as with 32 + 1.
#include <algorithm>

#include "mxfp4.h"

namespace moe {
namespace {

constexpr int kRows = 128;               // rows of a tile
constexpr int kUnit = 4352;              // bytes of a (block, step) of packed weights
constexpr int kSlot = kRows * 128;       // activations of 256 of k
constexpr int kRing = 4 * kSlot;
constexpr int kScSlot = kRows * 16;      // their scales, of 512 of k
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

// One tile of MS sub-tiles of 32 rows, D weight steps on their way.  kOnce: no other tile reads these
// weights, and they pass the L2 by (16 tokens over 32 + 1 experts: 134 us, through the L2 145; weights
// that several row tiles share lose by it, 4096 tokens 1126 us, 963).
template <bool kSwiglu, int MS, int D, bool kOnce>
__device__ __forceinline__ void mx_group_tile(const GroupArgs& g, int group, int n_idx,
                                              int64_t row0, int m_rows, char* smem, uint32_t lds0,
                                              uint32_t lds_sc) {
  const int lane = threadIdx.x & 63, fr = lane & 31, h = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = g.Kd / 128, ns = (nk + 1) / 2;
  const int b = 4 * n_idx + wv;
  const bool on = b < g.nblk;  // a wave without a block streams the tile's first one
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.w) + ((int64_t)group * g.nblk + (on ? b : 4 * n_idx)) * nk * kUnit, 0,
      nk * kUnit, 0x00020000);
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
  auto aload = [&](int s) {  // 256 of k, and two slots' scales with the even one
    if ((s & 1) == 0)
      load16_to_lds(sr, lds_sc + ((s >> 1) % 3) * kScSlot + 1024 * (wv & 1),
                    so + 16 * (uint32_t)(min(s, ns - 1) >> 1));
    const bool in = 8 * s + lchunk < 4 * nk;  // past K: zeros
#pragma unroll
    for (int i = 0; i < MS; ++i)
      load16_to_lds(ar, lds0 + (s & 3) * kSlot + (32 * i + 8 * wv) * 128,
                    in ? ao[i] + (uint32_t)s * 128 : kOut);
  };
  u32x4 wb[D + 1][4];
  uint32_t ws[D + 1];
  auto wload = [&](int kk, int buf) {
    const int at = min(kk, nk - 1) * kUnit;
    constexpr int kNt = kOnce ? 2 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      wb[buf][i] = __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16 + i * 1024, at, kNt);
    ws[buf] = __builtin_amdgcn_raw_buffer_load_b32(wr, lane * 4, at + 4096, kNt);
  };
  f32x16 acc[MS][2];
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.0f;
  // operand i = MS u + m of step kk: sub-tile m's codes at instruction u; and its scales
  constexpr int kF = 2 * MS, kAhead = 3, kN = kAhead + 1;
  static_assert((D + 1) * kF % kN == 0, "a turn of the loop ends with the register it began with");
  u32x4 af[kN];
  uint32_t sa[2][MS];
  uint32_t fo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) fo[i] = (uint32_t)at128(fr, 4 * (i >> 1) + 2 * h + (i & 1));
  auto frag = [&](int kk, int odd, int i, int buf) {  // odd: kk's parity, known to the compiler
    kk += i / kF;
    odd ^= i / kF & 1;
    const int u = i % kF / MS, m = i % MS;
    af[buf] = lds16(lds0 + ((kk >> 1) & 3) * kSlot + fo[2 * odd + u] + 4096 * m);
  };
  auto scale = [&](int kk, int m, int buf) {
    kk = min(kk, nk - 1);
    sa[buf][m] = lds2(lds_sc + ((kk >> 2) % 3) * kScSlot + 4 * (kk & 3) + 16 * fr + 2 * h +
                      512 * m);
  };

  // The order of loads: A(0) A(1) A(2) W(0) .. W(D-1), then at each slot's start A(s + 3) and
  // before each step W(kk + D).  A slot is complete in LDS one slot ahead of its turn, so that the
  // next step's first operands can be read before this one's products are done.  The loop's count
  // holds for the slots that it asks for itself, A(3) and on: the first three are waited for here.
  __syncthreads();  // the ring is refilled only when the LDS is free
  aload(0);
  aload(1);
  aload(2);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < D; ++j) {
    wload(j, j);
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_vm<5 * D>();  // A(0), A(1), A(2)
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int m = 0; m < MS; ++m) scale(0, m, 0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) frag(0, 0, i, i % kN);
  for (int kt = 0; kt < nk; kt += D + 1) {
    // steps past nk - 1 (at most D) multiply by zeros: with conditions in the loop the waits for the
    // weights would have to suit every way through it
#pragma unroll
    for (int j = 0; j <= D; ++j) {
      const int kk = kt + j;
      if ((j & 1) == 0) {
        // A(kk/2 + 1) is complete: behind it are four steps' weights and A(kk/2 + 2) (kk >= 4)
        wait_vm<MS + 20>();
        asm volatile("s_barrier" ::: "memory");
        aload((kk >> 1) + 3);
      }
      wload(kk + D, (j + D) % (D + 1));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kF; ++i) {
        const int u = i / MS, m = i % MS, buf = (j * kF + i) % kN;
        const uint32_t sm = sa[j & 1][m];
        if (u == 0) {
          acc[m][0] = mx_mfma32<0, 0>(wb[j][0], af[buf], acc[m][0], ws[j], sm);
          acc[m][1] = mx_mfma32<2, 0>(wb[j][2], af[buf], acc[m][1], ws[j], sm);
        } else {
          acc[m][0] = mx_mfma32<1, 1>(wb[j][1], af[buf], acc[m][0], ws[j], sm);
          acc[m][1] = mx_mfma32<3, 1>(wb[j][3], af[buf], acc[m][1], ws[j], sm);
        }
        // the products stay here, with the reads for later ones between them
        asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]) : : "memory");
        __builtin_amdgcn_sched_barrier(0);
        frag(kk, j & 1, i + kAhead, (j * kF + i + kAhead) % kN);
        if (u == 1) scale(kk + 1, m, (j + 1) & 1);
        __builtin_amdgcn_sched_barrier(0);
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

// The tile of a workgroup.  Tiles are ordered (group, column of blocks, row tile), so that those
// that share weights or activations are neighbours (with columns and row tiles exchanged 4096 tokens
// took 1045 us in place of 973), and each XCD takes one contiguous range of an eighth of the cost; a
// tile's cost is kTileCost and one for each 32 rows.
// Every wave finds its tile by itself, 64 groups at a time, a lane each: no barrier, and one load's
// latency where there are no more groups than that.
struct Pick {
  int group, n_idx, m0, m_rows;
  bool once;  // the group's only row tile
  int64_t row0;
};
constexpr int kTileCost = 12;
struct Chunk64 {  // of a lane's group: row tiles, cost, and the sums over all groups before it
  int mt, c, mt0, c0, first, m;
};
__device__ __forceinline__ Chunk64 group_chunk(const int32_t* __restrict__ offsets, int NG, int g0,
                                               int mt_run, int c_run) {
  const int lane = threadIdx.x & 63, g = g0 + lane;
  Chunk64 k;
  k.first = offsets[min(g, NG)];
  k.m = offsets[min(g + 1, NG)] - k.first;
  k.mt = (k.m + kRows - 1) / kRows;
  k.c = kTileCost * k.mt + (k.m + 31) / 32;
  int a = k.mt, b = k.c;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int x = __shfl_up(a, d), y = __shfl_up(b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  k.mt0 = mt_run + a - k.mt;
  k.c0 = c_run + b - k.c;
  return k;
}
__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// f(chunk, its first group) over the groups; one chunk is kept where it is all of them
template <typename F>
__device__ __forceinline__ void each_chunk(const int32_t* __restrict__ offsets, int NG,
                                           const Chunk64& all, F f) {
  if (NG <= kWave) {
    f(all, 0);
    return;
  }
  int mt_run = 0, c_run = 0;
  for (int g0 = 0; g0 < NG; g0 += kWave) {
    const Chunk64 k = group_chunk(offsets, NG, g0, mt_run, c_run);
    f(k, g0);
    mt_run = lane_of(k.mt0 + k.mt, 63);
    c_run = lane_of(k.c0 + k.c, 63);
  }
}

__device__ __forceinline__ bool pick_tile(const int32_t* __restrict__ offsets, int NG, int nt,
                                          int xcd, int slot, Pick& p) {
  const Chunk64 all = group_chunk(offsets, NG, 0, 0, 0);
  int tiles = 0, cost = 0;
  each_chunk(offsets, NG, all, [&](const Chunk64& k, int) {
    tiles = lane_of(k.mt0 + k.mt, 63);
    cost = lane_of(k.c0 + k.c, 63);
  });
  int begin = 0, end = tiles * nt;
  each_chunk(offsets, NG, all, [&](const Chunk64& k, int g0) {
    // first tile of XCD x: in the last group that begins at or before x eighths of the cost
    auto bound = [&](int x, int& at) {
      const int64_t t = (int64_t)cost * nt * x / kXcds;
      const bool in = g0 + (int)(threadIdx.x & 63) < NG && (int64_t)k.c0 * nt <= t;
      const uint64_t mask = __ballot(in);
      if (!mask) return;
      const int l = 63 - __clzll(mask), c = lane_of(k.c, l), mt = lane_of(k.mt, l);
      const int64_t past = t - (int64_t)lane_of(k.c0, l) * nt;
      const int n = nt * mt;  // tiles of this group
      at = lane_of(k.mt0, l) * nt + (c ? (int)min((double)n, (double)past * mt / (double)c) : 0);
    };
    if (xcd > 0) bound(xcd, begin);
    if (xcd < kXcds - 1) bound(xcd + 1, end);
  });
  const int tile = begin + slot;
  if (tile >= end) return false;
  each_chunk(offsets, NG, all, [&](const Chunk64& k, int g0) {
    const uint64_t mask = __ballot(k.mt > 0 && k.mt0 * nt <= tile);
    if (!mask) return;
    const int l = 63 - __clzll(mask), mt = lane_of(k.mt, l);
    const int local = tile - lane_of(k.mt0, l) * nt;
    p.group = g0 + l;
    p.n_idx = local / mt;
    p.m0 = local % mt * kRows;
    p.m_rows = min(kRows, lane_of(k.m, l) - p.m0);
    p.once = mt == 1;
    p.row0 = (int64_t)lane_of(k.first, l) + p.m0;
  });
  return true;
}

template <bool kSwiglu>
__global__ __launch_bounds__(256, 2) void k_mx_group(GroupArgs g) {
  __shared__ __attribute__((aligned(1024))) char smem[kRing];
  __shared__ __attribute__((aligned(16))) char s_sc[3 * kScSlot];
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(smem));
  const uint32_t lds_sc = __builtin_amdgcn_readfirstlane(lds_offset(s_sc));
  // One tile a workgroup: the hardware hands them out as others end, so that tiles of all costs fill
  // the chip (a grid of resident ones with a fixed share of the tiles each left it idle for a sixth
  // of the time).  There are more workgroups than tiles; those past their XCD's range leave.
  Pick p;
  if (!pick_tile(g.offsets, g.NG, (g.nblk + 3) / 4, blockIdx.x % kXcds, blockIdx.x / kXcds, p))
    return;
  const int group = __builtin_amdgcn_readfirstlane(p.group);
  const int n_idx = __builtin_amdgcn_readfirstlane(p.n_idx);
  const int m_rows = __builtin_amdgcn_readfirstlane(p.m_rows);
  const int64_t row0 = p.row0;
  const bool once = __builtin_amdgcn_readfirstlane(p.once);
#define MX_TILE(MS, D)                                                                           \
  case MS:                                                                                       \
    if (once)                                                                                    \
      mx_group_tile<kSwiglu, MS, D, true>(g, group, n_idx, row0, m_rows, smem, lds0, lds_sc);    \
    else                                                                                         \
      mx_group_tile<kSwiglu, MS, D, false>(g, group, n_idx, row0, m_rows, smem, lds0, lds_sc);   \
    break
  switch ((m_rows + 31) >> 5) {
    MX_TILE(1, 7);
    MX_TILE(2, 7);
    MX_TILE(3, 3);
    MX_TILE(4, 3);
    default: break;
  }
#undef MX_TILE
}

// Workgroups that suffice for R rows in NG groups: nt tiles for each of at most mt row tiles, and in
// an XCD's range, an eighth of the cost, no more than if all of them had the least cost.
int64_t group_grid(int64_t R, int NG, int nblk) {
  const int64_t nt = (nblk + 3) / 4, some = std::min<int64_t>(NG, R), mt = some + R / kRows;
  const int64_t cost = nt * (kTileCost * mt + R / 32 + some);
  return std::min(nt * mt, cost / kXcds / (kTileCost + 1) + 2) * kXcds;
}

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
  hipLaunchKernelGGL(k_mx_group<true>, dim3((unsigned)group_grid(d.R(), g.NG, g.nblk)), dim3(256), 0, st, g);
  return hipGetLastError();
}

hipError_t launch_ffn_down_mxfp4(const Dims& d, const uint8_t* hq, const uint8_t* hs, int64_t ldhs,
                                 const int32_t* offsets, const uint8_t* w, void* y,
                                 hipStream_t st) {
  GroupArgs g{hq, hs, d.I / 2, ldhs, 0, nullptr, offsets, w, nullptr, nullptr, 0, 0,
              static_cast<uint16_t*>(y), d.E + d.S, d.I, d.H / 64, d.H};
  hipLaunchKernelGGL(k_mx_group<false>, dim3((unsigned)group_grid(d.R(), g.NG, g.nblk)), dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace moe
