// Sequence-wise balance loss on the router's affinities, with its counts and gradient.
// With s = sigmoid(clamp(z, +-80)), S_t = sum_e s[t,e], a sequence q of L tokens and n[q,e]
// its choices of expert e:
//   f[q,e] = E/(K L) n[q,e]            (1 for every expert when the loads are uniform)
//   P[q,e] = 1/L sum_t s[t,e]/S_t
//   loss[q] = sum_e f[q,e] P[q,e]
// The counts are piecewise constant, so the gradient runs through P alone: with
// c[q,e] = dloss[q] f[q,e]/L and m_t = sum_e c[q,e] s[t,e]/S_t,
//   dz[t,e] = (c[q,e] - m_t)/S_t s(1-s), 0 where |z| > 80 (the clamp is flat there).
// It is formed as k (n' - m') (s/S)(1-s), with c = k n, n' the count from the uniform share on and
// m' the mean of n': near the lower clamp s and S are about 1e-35, where c s would not be a normal
// number and c/S would be infinite, while n' s is normal and s/S at most 1.
// The backward joins the gradient of the chosen gates to it (the formula of the router's
// backward), so a training step reads the logits once for both.
//
// Forward, two launches (one for a small batch) and no atomics on floats (the sums' order is
// fixed):
//   k_balance_part: one workgroup per chunk of C tokens.  A chunk may hold pieces of several
//     sequences; chunk c's piece of sequence q is slot c + q of the workspace (pieces in
//     order raise c or q by at least one, so slots do not collide).  Lanes own 4 adjacent
//     experts each and LP lanes a token, so a wave takes 64/LP tokens at a time; the
//     shares add up in registers, the choices in an LDS histogram.
//   k_balance_seq: one workgroup per sequence sums its slots and forms P and the loss.
// k_balance_short is both for a small batch.
// Both passes are bound by the logits' bytes: 262,144 tokens x 256 experts in 38 sequences, forward
// 56 + 6 us (4.8 TB/s), backward with the gates' part 110 us (4.9 TB/s); a batch of 128 tokens by
// the latency of its dependent loads, 6 us a kernel.
#include "common.h"

namespace moe {
namespace {

constexpr int kBalMaxE = 512;
constexpr int kBalMaxK = 16;

// exp(-z) to about an ulp: z log2(e) as a rounded product and its remainder, the latter
// applied to first order (|z| <= 80, so the result is a normal number).
__device__ __forceinline__ float exp_neg(float z) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float a = -z;
  const float hi = a * kLog2e;
  const float lo = __builtin_fmaf(a, kLog2eLo, __builtin_fmaf(a, kLog2e, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return __builtin_fmaf(e * lo, kLn2, e);
}

__device__ __forceinline__ float clamp80(float z) {
  return __builtin_amdgcn_fmed3f(z, -80.0f, 80.0f);
}

// first q in [0, n] with off[q + 1] > t (n: none)
__device__ __forceinline__ int seq_after(const int32_t* __restrict__ off, int n, int64_t t) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// 4 adjacent values of a row of E, `fill` past its end
template <bool kVec>
__device__ __forceinline__ float4 load_row4(const float* __restrict__ row, int e, int E,
                                            float fill) {
  float4 v = make_float4(fill, fill, fill, fill);
  if (kVec) {
    if (e < E) v = *reinterpret_cast<const float4*>(row + e);
  } else {
    if (e < E) v.x = row[e];
    if (e + 1 < E) v.y = row[e + 1];
    if (e + 2 < E) v.z = row[e + 2];
    if (e + 3 < E) v.w = row[e + 3];
  }
  return v;
}

// A NaN among four logits.  The clamp (a median of three) makes a NaN -80, which would hide a
// diverged router behind a finite loss: such a token's sum of affinities is made NaN instead.
// (A clamp that keeps a NaN, by the two instructions of IEEE 754-2019's maximum and minimum, cost
// 180 us at 262,144 x 256 with its gradient, against 170.)
__device__ __forceinline__ bool any_nan(const float4& v) {
  return __builtin_isunordered(v.x, v.y) | __builtin_isunordered(v.z, v.w);
}

// element i of the four at expert e lies past the row.  By its place, not by the fill: a caller's
// own -inf is a logit as any other, clamped to -80.
template <bool kVec>
__device__ __forceinline__ bool past(int e, int i, int E) {
  return kVec ? e >= E : e + i >= E;
}

template <int LP>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// LP lanes a token, SL groups of 4 experts a lane (expert 4 LP j + 4 l + i): 16 lanes up to 256
// experts, so that 4 tokens share each step of a sum across lanes (with 64 lanes a token the
// backward spent more on those than on its bytes: 146 us at 262,144 tokens and 256 experts)
// kFull: E = 4 LP SL, no lane's expert is past E
template <int LP, int SL, bool kVec, bool kFull>
__global__ __launch_bounds__(256) void k_balance_part(
    const float* __restrict__ z, const int32_t* __restrict__ idx, const int32_t* __restrict__ off,
    int n_seq, int64_t T, int E, int E4, int K, int C, float* __restrict__ part_p,
    int32_t* __restrict__ part_n) {
  constexpr int TPW = 64 / LP, kWaves = 4, kStep = TPW * kWaves;
  constexpr int U = SL < 4 ? 4 : 2;  // rows in flight per lane group
  __shared__ int hist[kBalMaxE];
  __shared__ float4 s_p[kWaves][LP * SL];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int seg = lane / LP, l = lane % LP;
  const int c = blockIdx.x;
  const int64_t t0 = (int64_t)c * C, t1 = min(t0 + C, T);
  for (int e = tid; e < E; e += 256) hist[e] = 0;
  int64_t at = t0;
  for (;;) {
    const int q = seq_after(off, n_seq, at);
    if (q >= n_seq) break;
    const int64_t lo = max((int64_t)off[q], at), hi = min((int64_t)off[q + 1], t1);
    if (lo >= hi) break;  // the next sequence starts behind this chunk
    __syncthreads();      // the histogram is clear, the last piece's sums are read
    for (int64_t i = lo * K + tid; i < hi * K; i += 256) {
      const int e = idx[i];
      if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
    }
    float acc[SL][4];
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    for (int64_t t = lo + wv * TPW + seg; t < hi + (int64_t)wv * TPW + seg; t += U * kStep) {
      // every lane of the wave runs the same number of rounds; rows past hi read as -inf
      float4 v[U][SL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tt = t + u * kStep;
#pragma unroll
        for (int j = 0; j < SL; ++j)
          v[u][j] = load_row4<kVec>(z + tt * E, 4 * (LP * j + l), tt < hi ? E : 0, -INFINITY);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float s[SL][4], sum = 0.0f;
        bool lost = false;
#pragma unroll
        for (int j = 0; j < SL; ++j) {
          lost |= any_nan(v[u][j]);
          const float w[4] = {v[u][j].x, v[u][j].y, v[u][j].z, v[u][j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[j][i] = __builtin_amdgcn_rcpf(1.0f + exp_neg(clamp80(w[i])));
            if (!kFull && past<kVec>(4 * (LP * j + l), i, E)) s[j][i] = 0.0f;
            sum += s[j][i];
          }
        }
        sum = seg_sum<LP>(lost ? NAN : sum);
        const float inv = t + u * kStep < hi ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
        for (int j = 0; j < SL; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(s[j][i], inv, acc[j][i]);
      }
    }
    // the wave's token groups, then the waves
#pragma unroll
    for (int o = LP; o < 64; o <<= 1)
#pragma unroll
      for (int j = 0; j < SL; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += __shfl_xor(acc[j][i], o);
    if (seg == 0)
#pragma unroll
      for (int j = 0; j < SL; ++j)
        s_p[wv][LP * j + l] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    __syncthreads();
    const int64_t slot = (int64_t)c + q;
    for (int i = tid; i < E4 / 4; i += 256) {
      const float4 a = s_p[0][i], b = s_p[1][i], d = s_p[2][i], g = s_p[3][i];
      reinterpret_cast<float4*>(part_p + slot * E4)[i] =
          make_float4((a.x + b.x) + (d.x + g.x), (a.y + b.y) + (d.y + g.y),
                      (a.z + b.z) + (d.z + g.z), (a.w + b.w) + (d.w + g.w));
    }
    for (int e = tid; e < E4; e += 256) {
      part_n[slot * E4 + e] = e < E ? hist[e] : 0;
      if (e < E) hist[e] = 0;
    }
    at = hi;
    if (at >= t1) break;
  }
}

// One workgroup per sequence: the sums of its slots.  Thread (r, i) of G4 = 2^g >= E/4
// columns adds rows r, r + blockDim/G4, ... of expert group i.
__global__ __launch_bounds__(1024) void k_balance_seq(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_n,
    const int32_t* __restrict__ off, int64_t T, int E, int E4, int K, int C, int log_g4,
    int32_t* __restrict__ counts, float* __restrict__ prob, float* __restrict__ loss) {
  __shared__ float4 s_p[1024];
  __shared__ int4 s_n[1024];
  __shared__ float s_l[16];
  const int q = blockIdx.x, tid = threadIdx.x;
  const int i = tid & ((1 << log_g4) - 1), r = tid >> log_g4, nr = blockDim.x >> log_g4;
  const int64_t lo = max(0, off[q]), hi = min((int64_t)off[q + 1], T), L = hi - lo;
  float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  int4 n = make_int4(0, 0, 0, 0);
  if (L > 0 && 4 * i < E4) {
    const int64_t c0 = lo / C, c1 = (hi - 1) / C;
    auto add = [&](const float4& a, const int4& b) {
      p.x += a.x; p.y += a.y; p.z += a.z; p.w += a.w;
      n.x += b.x; n.y += b.y; n.z += b.z; n.w += b.w;
    };
    int64_t c = c0 + r;
    for (; c + 3 * nr <= c1; c += 4 * nr) {
      float4 a[4];
      int4 b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t at = (c + u * nr + q) * E4 + 4 * i;
        a[u] = *reinterpret_cast<const float4*>(part_p + at);
        b[u] = *reinterpret_cast<const int4*>(part_n + at);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) add(a[u], b[u]);
    }
    for (; c <= c1; c += nr) {
      const int64_t at = (c + q) * E4 + 4 * i;
      add(*reinterpret_cast<const float4*>(part_p + at),
          *reinterpret_cast<const int4*>(part_n + at));
    }
  }
  s_p[tid] = p;
  s_n[tid] = n;
  for (int h = nr >> 1; h >= 1; h >>= 1) {
    __syncthreads();
    if (r < h) {
      const float4 a = s_p[tid + (h << log_g4)];
      const int4 b = s_n[tid + (h << log_g4)];
      p.x += a.x; p.y += a.y; p.z += a.z; p.w += a.w;
      n.x += b.x; n.y += b.y; n.z += b.z; n.w += b.w;
      s_p[tid] = p;
      s_n[tid] = n;
    }
  }
  float mine = 0.0f;
  if (r == 0 && 4 * i < E4) {
    const float len = L > 0 ? (float)L : 1.0f;
    const float per = (float)E / ((float)K * len);
    const float pv[4] = {p.x / len, p.y / len, p.z / len, p.w / len};
    const int nv[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = 4 * i + k;
      if (e < E) {
        counts[(int64_t)q * E + e] = nv[k];
        prob[(int64_t)q * E + e] = pv[k];
        mine = __builtin_fmaf((float)nv[k] * per, pv[k], mine);
      }
    }
  }
  mine = seg_sum<64>(mine);
  if ((tid & 63) == 0) s_l[tid >> 6] = mine;
  __syncthreads();
  if (tid == 0) {
    float v = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) v += s_l[w];
    loss[q] = v;
  }
}

// A small batch (T <= kShort): one workgroup per sequence does all of it, in one launch.  Loss and
// gradient of 128 x 256: 13.5 us, in two launches 16.8; of 512 x 256 in four sequences 14.6, of 513
// in two launches 17.4.  The rule goes by T alone, so it also holds where a batch is one
// sequence, and there from about 300 tokens on the two launches would be the faster ones: 300
// tokens 16.8 us, 512 22.7, 513 in two launches 16.5.
constexpr int kShort = 512;
template <int LP, int SL, bool kVec, bool kFull>
__global__ __launch_bounds__(1024) void k_balance_short(
    const float* __restrict__ z, const int32_t* __restrict__ idx, const int32_t* __restrict__ off,
    int64_t T, int E, int K, int32_t* __restrict__ counts, float* __restrict__ prob,
    float* __restrict__ loss) {
  constexpr int TPW = 64 / LP, kWaves = 16;
  __shared__ int hist[4 * LP * SL];
  __shared__ float s_p[kWaves][4 * LP * SL];
  __shared__ float s_l[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int seg = lane / LP, l = lane % LP, q = blockIdx.x;
  const int64_t lo = max(0, off[q]), hi = min((int64_t)off[q + 1], T), L = hi - lo;
  for (int e = tid; e < 4 * LP * SL; e += 1024) hist[e] = 0;
  __syncthreads();
  for (int64_t i = lo * K + tid; i < hi * K; i += 1024) {
    const int e = idx[i];
    if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
  }
  float acc[SL][4] = {};
  for (int64_t t0 = lo + wv * TPW; t0 < hi; t0 += kWaves * TPW) {
    const int64_t t = t0 + seg;
    float s[SL][4], sum = 0.0f;
    bool lost = false;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      const float4 v = load_row4<kVec>(z + t * E, 4 * (LP * j + l), t < hi ? E : 0, -INFINITY);
      lost |= any_nan(v);
      const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j][i] = __builtin_amdgcn_rcpf(1.0f + exp_neg(clamp80(w[i])));
        if (!kFull && past<kVec>(4 * (LP * j + l), i, E)) s[j][i] = 0.0f;
        sum += s[j][i];
      }
    }
    sum = seg_sum<LP>(lost ? NAN : sum);
    const float inv = t < hi ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(s[j][i], inv, acc[j][i]);
  }
#pragma unroll
  for (int o = LP; o < 64; o <<= 1)
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] += __shfl_xor(acc[j][i], o);
  if (seg == 0)
#pragma unroll
    for (int j = 0; j < SL; ++j)
      *reinterpret_cast<float4*>(&s_p[wv][4 * (LP * j + l)]) =
          make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  const float len = L > 0 ? (float)L : 1.0f;
  const float per = (float)E / ((float)K * len);
  float mine = 0.0f;
  for (int e = tid; e < E; e += 1024) {
    float p = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) p += s_p[w][e];
    p /= len;
    counts[(int64_t)q * E + e] = hist[e];
    prob[(int64_t)q * E + e] = p;
    mine = __builtin_fmaf((float)hist[e] * per, p, mine);
  }
  mine = seg_sum<64>(mine);
  if (lane == 0) s_l[wv] = mine;
  __syncthreads();
  if (tid == 0) {
    float v = 0.0f;
    for (int w = 0; w < kWaves; ++w) v += s_l[w];
    loss[q] = v;
  }
}

// LP lanes a token as in the forward; a group takes TW consecutive tokens and looks its
// sequence up once.  gates: dgate != nullptr.
template <int LP, int SL, bool kVec, bool kFull>
__global__ __launch_bounds__(256) void k_balance_bwd(
    const float* __restrict__ z, const int32_t* __restrict__ off, int n_seq,
    const int32_t* __restrict__ counts, const float* __restrict__ dloss,
    const int32_t* __restrict__ idx, const float* __restrict__ gate,
    const float* __restrict__ dgate, int64_t T, int E, int K, int TW, float* __restrict__ dz) {
  constexpr int TPW = 64 / LP, NK = (kBalMaxK + LP - 1) / LP;
  __shared__ float s_d[4][64 * 4 * SL];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int seg = lane / LP, l = lane % LP;
  float* sd = &s_d[wv][seg * LP * 4 * SL];
  const int64_t first = (((int64_t)blockIdx.x * 4 + wv) * TPW + seg) * TW;
  int q = first < T ? seq_after(off, n_seq, first) : n_seq;
  int64_t q_lo = 0, q_hi = -1;  // the sequence whose coefficients are held
  float cf[SL][4], scale = 0.0f;  // the counts, and what they are to be scaled by
#pragma unroll
  for (int j = 0; j < SL; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) cf[j][i] = 0.0f;
  // the logits and choices of token first + w, loaded a turn ahead
  float4 row[SL];
  int ek[NK];
  float gk[NK], dk[NK];
  auto choices = [&](int64_t t, int n, int* e, float* g, float* dg) {
    const int k = n * LP + l;
    const bool on = t < T && k < K;
    *e = on ? idx[t * K + k] : -1;
    *g = on ? gate[t * K + k] : 0.0f;
    *dg = on ? dgate[t * K + k] : 0.0f;
  };
#pragma unroll
  for (int j = 0; j < SL; ++j)
    row[j] = load_row4<kVec>(z + first * E, 4 * (LP * j + l), first < T ? E : 0, -INFINITY);
  if (dgate)
#pragma unroll
    for (int n = 0; n < NK; ++n) choices(first, n, &ek[n], &gk[n], &dk[n]);
  for (int w = 0; w < TW; ++w) {
    const int64_t t = first + w;
    const bool live = t < T;
    float4 next[SL];
#pragma unroll
    for (int j = 0; j < SL; ++j)
      next[j] = load_row4<kVec>(z + (t + 1) * E, 4 * (LP * j + l),
                                w + 1 < TW && t + 1 < T ? E : 0, -INFINITY);
    int ek1[NK];
    float gk1[NK], dk1[NK];
    if (dgate)
#pragma unroll
      for (int n = 0; n < NK; ++n) choices(w + 1 < TW ? t + 1 : T, n, &ek1[n], &gk1[n], &dk1[n]);
    if (live && t >= q_hi && q < n_seq) {
      if (q_hi >= 0) q = seq_after(off, n_seq, t);
      if (q < n_seq) {
        q_lo = off[q];
        q_hi = off[q + 1];
        const float len = (float)(q_hi - q_lo);
        scale = dloss[q] * ((float)E / ((float)K * len)) / len;
        // the counts from the uniform share on, in whole numbers: a constant in c drops out of
        // c - m, and near balance, where the counts are nearly equal, it would cancel badly
        const int uniform = (int)((q_hi - q_lo) * K / E);
#pragma unroll
        for (int j = 0; j < SL; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * (LP * j + l) + i;
            cf[j][i] = e < E ? (float)(counts[(int64_t)q * E + e] - uniform) : 0.0f;
          }
      }
    }
    const bool in = live && q < n_seq && t >= q_lo;
    float s[SL][4], o[SL][4], sum = 0.0f, dot = 0.0f;  // o = 1 - s, without cancellation
    bool lost = false;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      lost |= any_nan(row[j]);
      const float x[4] = {row[j].x, row[j].y, row[j].z, row[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = clamp80(x[i]), em = exp_neg(c);
        const float a = __builtin_amdgcn_rcpf(1.0f + em);
        s[j][i] = !kFull && past<kVec>(4 * (LP * j + l), i, E) ? 0.0f : a;
        o[j][i] = c == x[i] ? em * a : 0.0f;  // 0 where the clamp is flat
        sum += s[j][i];
        dot = __builtin_fmaf(cf[j][i], s[j][i], dot);
      }
    }
    sum = seg_sum<LP>(lost ? NAN : sum);
    dot = seg_sum<LP>(dot);
    const float inv = in ? __builtin_amdgcn_rcpf(sum) : 0.0f;
    const float mean = dot * inv, k = in ? scale : 0.0f;
    float d[SL][4];
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[j][i] = (cf[j][i] - mean) * k * (s[j][i] * inv * o[j][i]);
    if (dgate) {
      // the chosen gates' part: their logits come from, and their gradients are added to, the
      // token's row in the group's LDS (LDS operations of a wave run in order)
      auto put = [&](int j, float a, float b, float c, float e) {
        *reinterpret_cast<float4*>(sd + 4 * (LP * j + l)) = make_float4(a, b, c, e);
      };
#pragma unroll
      for (int j = 0; j < SL; ++j) put(j, row[j].x, row[j].y, row[j].z, row[j].w);
      __builtin_amdgcn_wave_barrier();
      float sl[NK], tot = 0.0f, gd = 0.0f;
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        sl[n] = 0.0f;
        if (ek[n] >= 0 && ek[n] < E) {
          const float x = sd[ek[n]], c = clamp80(x), em = exp_neg(c);
          const float a = x != x ? x : __builtin_amdgcn_rcpf(1.0f + em);
          sl[n] = c == x ? a * (em * a) : 0.0f;
          gd = __builtin_fmaf(gk[n], dk[n], gd);
          tot += a;
        }
      }
      tot = seg_sum<LP>(tot);
      gd = seg_sum<LP>(gd);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < SL; ++j) put(j, d[j][0], d[j][1], d[j][2], d[j][3]);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int n = 0; n < NK; ++n)
        if (ek[n] >= 0 && ek[n] < E) atomicAdd(sd + ek[n], (dk[n] - gd) * (sl[n] / tot));
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < SL; ++j) {
        const float4 g = *reinterpret_cast<const float4*>(sd + 4 * (LP * j + l));
        d[j][0] = g.x; d[j][1] = g.y; d[j][2] = g.z; d[j][3] = g.w;
      }
      __builtin_amdgcn_wave_barrier();
    }
    if (live) {
#pragma unroll
      for (int j = 0; j < SL; ++j) {
        const int e = 4 * (LP * j + l);
        float* p = dz + t * E + e;
        if (kVec) {
          const f32x4 v = {d[j][0], d[j][1], d[j][2], d[j][3]};
          if (e < E) __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(p));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < E) p[i] = d[j][i];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < SL; ++j) row[j] = next[j];
    if (dgate)
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        ek[n] = ek1[n];
        gk[n] = gk1[n];
        dk[n] = dk1[n];
      }
  }
}

// Tokens per chunk, at least 16: about 256 chunks (one a CU) of a small batch, which leaves
// k_balance_seq few slots, and from chunks of 64 tokens on about 1024 of a large one.  Loss and
// gradient at E=256: 16,384 tokens 28.4 us (1024 chunks 36.7), 262,144 tokens 171 us (256
// chunks 194).
int chunk_tokens(int64_t T) {
  int64_t c = 16;
  while (c * (c < 64 ? 256 : 1024) < T) c *= 2;
  return (int)c;
}

}  // namespace

size_t balance_ws_bytes(const Dims& d, int n_seq) {
  const int C = chunk_tokens(d.T);
  const size_t slots = (size_t)((d.T + C - 1) / C) + (size_t)n_seq;
  return slots * (size_t)((d.E + 3) / 4 * 4) * 8;
}

#define BAL_SHAPES(CALL)                                 \
  if (d.E % 4 == 0) {                                    \
    if (d.E <= 16) CALL(4, 1, true, false);              \
    else if (d.E <= 32) CALL(8, 1, true, false);         \
    else if (d.E == 64) CALL(16, 1, true, true);         \
    else if (d.E <= 64) CALL(16, 1, true, false);        \
    else if (d.E == 128) CALL(16, 2, true, true);        \
    else if (d.E <= 128) CALL(16, 2, true, false);       \
    else if (d.E == 256) CALL(16, 4, true, true);        \
    else if (d.E <= 256) CALL(16, 4, true, false);       \
    else if (d.E == 512) CALL(32, 4, true, true);        \
    else CALL(32, 4, true, false);                       \
  } else {                                               \
    if (d.E <= 64) CALL(16, 1, false, false);            \
    else if (d.E <= 256) CALL(16, 4, false, false);      \
    else CALL(32, 4, false, false);                      \
  }

hipError_t launch_balance_loss(const Dims& d, const float* z, const int32_t* idx,
                               const int32_t* off, int n_seq, int32_t* counts, float* prob,
                               float* loss, void* ws, hipStream_t st) {
  const int C = chunk_tokens(d.T), E4 = (d.E + 3) / 4 * 4;
  const int64_t nch = (d.T + C - 1) / C;
  float* pp = static_cast<float*>(ws);
  int32_t* pn = reinterpret_cast<int32_t*>(pp + (nch + n_seq) * E4);
  if (d.T <= kShort) {
#define BAL_SHORT(LP, SL, V, F)                                                                  \
  hipLaunchKernelGGL((k_balance_short<LP, SL, V, F>), dim3((unsigned)n_seq), dim3(1024), 0, st, z, \
                     idx, off, d.T, d.E, d.K, counts, prob, loss)
    BAL_SHAPES(BAL_SHORT)
#undef BAL_SHORT
    return hipGetLastError();
  }
#define BAL_PART(LP, SL, V, F)                                                                 \
  hipLaunchKernelGGL((k_balance_part<LP, SL, V, F>), dim3((unsigned)nch), dim3(256), 0, st, z, \
                     idx, off, n_seq, d.T, d.E, E4, d.K, C, pp, pn)
  BAL_SHAPES(BAL_PART)
#undef BAL_PART
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int log_g4 = 0;
  while ((4 << log_g4) < d.E) ++log_g4;
  // (16,384 x 256 in 4 sequences 36 us, with 256 threads 46; 262,144 x 64 in 2000 78 us, with
  // 1024 threads 92)
  const int threads = nch > 16 * (int64_t)n_seq ? 1024 : 256;
  hipLaunchKernelGGL(k_balance_seq, dim3((unsigned)n_seq), dim3(threads), 0, st, pp, pn, off, d.T,
                     d.E, E4, d.K, C, log_g4, counts, prob, loss);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const Dims& d, const float* z, const int32_t* off, int n_seq,
                              const int32_t* counts, const float* dloss, const int32_t* idx,
                              const float* gate, const float* dgate, float* dz, hipStream_t st) {
  // Consecutive tokens of a lane group, once that leaves every CU its waves: fewer look-ups, and
  // the next row's load a turn ahead; rows of at most one line stay with 2, so that a wave's
  // loads lie together.  Loss and gradient with 8 / 2 / 1: 262,144 x 256 171 / 185 / 206 us, 32,768
  // x 256 43 / 37 / 39, 8,192 x 256 36 / 23 / 23, 1,000,000 x 16 121 / 93 / 95.
  const int TW = d.T < 32768 ? 1 : d.T < 65536 || d.E <= 32 ? 2 : 8;
#define BAL_BWD(LP, SL, V, F)                                                                 \
  hipLaunchKernelGGL((k_balance_bwd<LP, SL, V, F>),                                            \
                     dim3((unsigned)((d.T + 256 / LP * TW - 1) / (256 / LP * TW))), dim3(256), \
                     0, st, z, off, n_seq, counts, dloss, idx, gate, dgate, d.T, d.E, d.K, TW, dz)
  BAL_SHAPES(BAL_BWD)
#undef BAL_BWD
  return hipGetLastError();
}
#undef BAL_SHAPES

}  // namespace moe
