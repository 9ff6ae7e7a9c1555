// C ABI of libmoe: argument validation, workspace layout and launches.
// Every call validates first and enqueues nothing when it returns an error.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "launch_added.h"

namespace moe {

namespace {
thread_local char g_err[512] = "";

moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status fail(moe_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

moe_status hip_fail(hipError_t e, const char* what) {
  return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int kMaxDevices = 64;
std::once_flag g_dev_once[kMaxDevices];
int g_dev_cus[kMaxDevices];
bool g_dev_ok[kMaxDevices];

// Device checks are cached per device: gfx950 and its CU count.
moe_status check_device(int* cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MOE_ERR_UNSUPPORTED, "device %d out of range", dev);
  std::call_once(g_dev_once[dev], [dev] {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) == hipSuccess) {
      g_dev_ok[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
      g_dev_cus[dev] = prop.multiProcessorCount;
    }
  });
  if (!g_dev_ok[dev]) return fail(MOE_ERR_UNSUPPORTED, "device %d is not gfx950 (MI355X)", dev);
  if (cus) *cus = g_dev_cus[dev];
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// share: for calls that take the experts as they come, without routing to them; a token of a share
// of the experts may have more choices than the share has experts
moe_status validate(const moe_problem* p, Dims* d, bool share = false) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "problem is NULL");
  if (p->T < 1) return fail(MOE_ERR_INVALID_ARG, "T=%lld must be >= 1", (long long)p->T);
  if (p->K < 1 || p->K > 16) return fail(MOE_ERR_INVALID_ARG, "K=%d must be in [1,16]", p->K);
  if (p->T * (int64_t)(p->K + 1) >= (int64_t)1 << 31)
    return fail(MOE_ERR_INVALID_ARG, "T*(K+1) must be < 2^31");
  if (p->H < 128 || p->H > 65536 || p->H % 128)
    return fail(MOE_ERR_INVALID_ARG, "H=%d must be a multiple of 128 in [128,65536]", p->H);
  if (p->I < 128 || p->I > 32768 || p->I % 128)
    return fail(MOE_ERR_INVALID_ARG, "I=%d must be a multiple of 128 in [128,32768]", p->I);
  if ((int64_t)p->H * p->I > ((int64_t)1 << 28))
    return fail(MOE_ERR_INVALID_ARG, "H*I=%lld must be <= 2^28 (32-bit buffer offsets)",
                (long long)p->H * p->I);
  if (p->E < 1 || p->E > 512) return fail(MOE_ERR_INVALID_ARG, "E=%d must be in [1,512]", p->E);
  if (p->G < 1 || p->G > 64 || p->E % p->G)
    return fail(MOE_ERR_INVALID_ARG, "G=%d must divide E=%d and be in [1,64]", p->G, p->E);
  const int gs = p->E / p->G;
  if (p->M < 1 || p->M > p->G) return fail(MOE_ERR_INVALID_ARG, "M=%d must be in [1,G]", p->M);
  if (p->J < 1 || p->J > gs || p->J > 8)
    return fail(MOE_ERR_INVALID_ARG, "J=%d must be in [1,min(E/G,8)]", p->J);
  if (!share && p->K > p->M * gs)
    return fail(MOE_ERR_INVALID_ARG, "K=%d exceeds M*E/G=%d", p->K, p->M * gs);
  if (p->S != 0 && p->S != 1) return fail(MOE_ERR_INVALID_ARG, "S=%d must be 0 or 1", p->S);
  const bool ok_dtypes = (p->act_dtype == MOE_F32 && p->expert_dtype == MOE_F32) ||
                         (p->act_dtype == MOE_BF16 &&
                          (p->expert_dtype == MOE_BF16 || p->expert_dtype == MOE_FP8_E4M3 ||
                           p->expert_dtype == MOE_MXFP4));
  if (!ok_dtypes)
    return fail(MOE_ERR_INVALID_ARG, "dtypes act=%d expert=%d not supported", p->act_dtype,
                p->expert_dtype);
  d->T = p->T; d->H = p->H; d->E = p->E; d->G = p->G; d->M = p->M; d->K = p->K;
  d->J = p->J; d->I = p->I; d->S = p->S; d->act = p->act_dtype; d->expert = p->expert_dtype;
  return MOE_OK;
}

// the calls that have kernels of their own for this type (moe_..._mxfp4)
moe_status refuse_mxfp4(const Dims& d, const char* call) {
  if (d.expert == MOE_MXFP4)
    return fail(MOE_ERR_UNSUPPORTED, "%s is not built for MXFP4 experts", call);
  return MOE_OK;
}

size_t route_ws_bytes(const Dims& d) { return sizeof(float) * (size_t)d.T * d.E; }

#define REQUIRE_PTR(ptr)                                                   \
  do {                                                                     \
    if (!(ptr)) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #ptr);      \
    if (!aligned16(ptr)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #ptr); \
  } while (0)

}  // namespace

int device_cu_count() {
  int cus = 0;
  if (check_device(&cus) != MOE_OK || cus <= 0) return 256;
  return cus;
}

}  // namespace moe

using namespace moe;

extern "C" {

const char* moe_status_str(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported";
    case MOE_ERR_WORKSPACE: return "workspace too small";
    case MOE_ERR_HIP: return "HIP error";
  }
  return "unknown status";
}

const char* moe_last_error(void) { return g_err; }

size_t moe_workspace_bytes(const moe_problem* p, int32_t which_call) {
  Dims d;
  if (validate(p, &d) != MOE_OK) return 0;
  switch (which_call) {
    case MOE_CALL_ROUTE: return route_ws_bytes(d);
    case MOE_CALL_PERMUTE: return permute_ws_bytes(d);
    case MOE_CALL_EXPERT_FFN:
      if (d.expert == MOE_MXFP4) {
        fail(MOE_ERR_UNSUPPORTED, "moe_expert_ffn is not built for MXFP4 experts");
        return 0;
      }
      return ffn_ws_bytes(d);
    case MOE_CALL_ROUTER_BACKWARD_DENSE: return router_dense_ws_bytes(d);
  }
  fail(MOE_ERR_INVALID_ARG, "unknown call id %d", which_call);
  return 0;
}

moe_status moe_route(const moe_problem* p, const void* x, const float* w_router,
                     const float* bias, int32_t* topk_idx, float* topk_gate,
                     int32_t* expert_counts, float* logits_out, void* ws, size_t ws_bytes,
                     void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_router);
  if (!bias || !topk_idx || !topk_gate || !expert_counts)
    return fail(MOE_ERR_INVALID_ARG, "bias, topk_idx, topk_gate and expert_counts are required");
  float* z = logits_out;
  if (!z) {
    if (!ws || ws_bytes < route_ws_bytes(d))
      return fail(MOE_ERR_WORKSPACE, "route needs %zu workspace bytes, got %zu",
                  route_ws_bytes(d), ws ? ws_bytes : (size_t)0);
    z = static_cast<float*>(ws);
  }
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_route(d, x, w_router, bias, topk_idx, topk_gate, expert_counts, z,
                              static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_route launch");
}

moe_status moe_permute(const moe_problem* p, const void* x, const int32_t* topk_idx,
                       int32_t* offsets, int32_t* sorted_token, int32_t* inv_perm,
                       void* x_sorted, float* x_sorted_scale, void* ws, size_t ws_bytes,
                       void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if (!topk_idx || !offsets || !sorted_token || !inv_perm)
    return fail(MOE_ERR_INVALID_ARG, "topk_idx, offsets, sorted_token and inv_perm are required");
  if (x_sorted) {  // NULL: index maps only
    if (d.expert == MOE_MXFP4)
      return fail(MOE_ERR_UNSUPPORTED, "MXFP4 experts gather their rows: x_sorted must be NULL");
    REQUIRE_PTR(x);
    REQUIRE_PTR(x_sorted);
    if (d.expert == MOE_FP8_E4M3 && !x_sorted_scale)
      return fail(MOE_ERR_INVALID_ARG, "x_sorted_scale is required for the FP8 path");
  }
  if (!ws || ws_bytes < permute_ws_bytes(d))
    return fail(MOE_ERR_WORKSPACE, "permute needs %zu workspace bytes, got %zu",
                permute_ws_bytes(d), ws ? ws_bytes : (size_t)0);
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_permute(d, x, topk_idx, offsets, sorted_token, inv_perm, x_sorted,
                                x_sorted_scale, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_permute launch");
}

moe_status moe_count_invalid_ids(const moe_problem* p, const int32_t* topk_idx,
                                 int32_t* n_invalid, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  REQUIRE_PTR(topk_idx);
  REQUIRE_PTR(n_invalid);
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_count_invalid(d, topk_idx, n_invalid, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_count_invalid_ids launch");
}

moe_status moe_permute_noalloc(const moe_problem* p, const void* x, const int32_t* topk_idx,
                               int32_t* offsets, int32_t* sorted_token, int32_t* inv_perm,
                               void* x_sorted, float* x_sorted_scale, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if (!topk_idx || !offsets || !sorted_token || !inv_perm)
    return fail(MOE_ERR_INVALID_ARG, "topk_idx, offsets, sorted_token and inv_perm are required");
  if (x_sorted) {  // NULL: index maps only
    if (d.expert == MOE_MXFP4)
      return fail(MOE_ERR_UNSUPPORTED, "MXFP4 experts gather their rows: x_sorted must be NULL");
    REQUIRE_PTR(x);
    REQUIRE_PTR(x_sorted);
    if (d.expert == MOE_FP8_E4M3 && !x_sorted_scale)
      return fail(MOE_ERR_INVALID_ARG, "x_sorted_scale is required for the FP8 path");
  }
  if (permute_ws_bytes(d) > permute_scratch_capacity())
    return fail(MOE_ERR_WORKSPACE,
                "moe_permute_noalloc: this problem needs %zu scratch bytes, the library holds "
                "%zu (T*K + 2*ceil(T/256)*E must be at most %zu); use moe_permute",
                permute_ws_bytes(d), permute_scratch_capacity(),
                (permute_scratch_capacity() - 256) / sizeof(int32_t));
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  void* ws = nullptr;
  hipError_t e = permute_scratch(&ws);
  if (e != hipSuccess) return hip_fail(e, "moe_permute_noalloc: device address of the scratch");
  e = launch_permute(d, x, topk_idx, offsets, sorted_token, inv_perm, x_sorted, x_sorted_scale,
                     ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_permute_noalloc launch");
}

moe_status moe_expert_ffn_up(const moe_problem* p, const void* x_sorted,
                             const float* x_sorted_scale, const int32_t* offsets,
                             const void* w13, const float* w13_scale, void* h, float* h_scale,
                             void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = refuse_mxfp4(d, "moe_expert_ffn_up")) != MOE_OK) return s;
  REQUIRE_PTR(x_sorted);
  REQUIRE_PTR(w13);
  REQUIRE_PTR(h);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if (d.expert == MOE_FP8_E4M3 && (!x_sorted_scale || !w13_scale || !h_scale))
    return fail(MOE_ERR_INVALID_ARG, "the FP8 path needs x_sorted_scale, w13_scale, h_scale");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_ffn_up(d, x_sorted, x_sorted_scale, offsets, nullptr, w13, w13_scale, h,
                               h_scale, static_cast<hipStream_t>(stream));
  if (e == hipErrorNotSupported)
    return fail(MOE_ERR_UNSUPPORTED, "no expert FFN kernel for expert dtype %d", d.expert);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_up launch");
}

moe_status moe_expert_ffn_up_gather(const moe_problem* p, const void* x, const float* x_scale,
                                    const int32_t* sorted_token, const int32_t* offsets,
                                    const void* w13, const float* w13_scale, void* h,
                                    float* h_scale, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = refuse_mxfp4(d, "moe_expert_ffn_up_gather")) != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w13);
  REQUIRE_PTR(h);
  if (!offsets || !sorted_token)
    return fail(MOE_ERR_INVALID_ARG, "offsets and sorted_token are required");
  if (d.expert == MOE_FP8_E4M3 && (!x_scale || !w13_scale || !h_scale))
    return fail(MOE_ERR_INVALID_ARG, "the FP8 path needs x_scale, w13_scale, h_scale");
  const int es = d.expert == MOE_FP8_E4M3 ? 1 : (d.expert == MOE_F32 ? 4 : 2);
  if (d.T * (int64_t)d.H * es >= ((int64_t)1 << 31) - 16)
    return fail(MOE_ERR_INVALID_ARG, "T*H*%d must be < 2^31 - 16 (32-bit row offsets)", es);
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_ffn_up(d, x, x_scale, offsets, sorted_token, w13, w13_scale, h, h_scale,
                               static_cast<hipStream_t>(stream));
  if (e == hipErrorNotSupported)
    return fail(MOE_ERR_UNSUPPORTED, "no expert FFN kernel for expert dtype %d", d.expert);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_up_gather launch");
}

moe_status moe_quantize_act_fp8(const moe_problem* p, const void* x, void* x_q, float* x_scale,
                                void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if (d.expert != MOE_FP8_E4M3 || d.act != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "moe_quantize_act_fp8 needs act BF16 and expert FP8_E4M3");
  REQUIRE_PTR(x);
  REQUIRE_PTR(x_q);
  if (!x_scale) return fail(MOE_ERR_INVALID_ARG, "x_scale is NULL");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_quantize_act(d, static_cast<const uint16_t*>(x), static_cast<uint8_t*>(x_q),
                                     x_scale, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_quantize_act_fp8 launch");
}

moe_status moe_expert_ffn_down(const moe_problem* p, const void* h, const float* h_scale,
                               const int32_t* offsets, const void* w2, const float* w2_scale,
                               void* y_sorted, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = refuse_mxfp4(d, "moe_expert_ffn_down")) != MOE_OK) return s;
  REQUIRE_PTR(h);
  REQUIRE_PTR(w2);
  REQUIRE_PTR(y_sorted);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if (d.expert == MOE_FP8_E4M3 && (!h_scale || !w2_scale))
    return fail(MOE_ERR_INVALID_ARG, "the FP8 path needs h_scale and w2_scale");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_ffn_down(d, h, h_scale, offsets, w2, w2_scale, y_sorted,
                                 static_cast<hipStream_t>(stream));
  if (e == hipErrorNotSupported)
    return fail(MOE_ERR_UNSUPPORTED, "no expert FFN kernel for expert dtype %d", d.expert);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_down launch");
}

moe_status moe_expert_ffn(const moe_problem* p, const void* x_sorted,
                          const float* x_sorted_scale, const int32_t* offsets,
                          const void* w13, const float* w13_scale, const void* w2,
                          const float* w2_scale, void* y_sorted, void* ws, size_t ws_bytes,
                          void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = refuse_mxfp4(d, "moe_expert_ffn")) != MOE_OK) return s;
  REQUIRE_PTR(x_sorted);
  REQUIRE_PTR(w13);
  REQUIRE_PTR(w2);
  REQUIRE_PTR(y_sorted);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if (d.expert == MOE_FP8_E4M3 && (!x_sorted_scale || !w13_scale || !w2_scale))
    return fail(MOE_ERR_INVALID_ARG, "the FP8 path needs x_sorted_scale, w13_scale, w2_scale");
  if (!ws || ws_bytes < ffn_ws_bytes(d) || !aligned16(ws))
    return fail(MOE_ERR_WORKSPACE, "expert_ffn needs %zu aligned workspace bytes, got %zu",
                ffn_ws_bytes(d), ws ? ws_bytes : (size_t)0);
  float* h_scale = d.expert == MOE_FP8_E4M3 ? ffn_ws_h_scale(d, ws) : nullptr;
  s = moe_expert_ffn_up(p, x_sorted, x_sorted_scale, offsets, w13, w13_scale, ws, h_scale, stream);
  if (s != MOE_OK) return s;
  return moe_expert_ffn_down(p, ws, h_scale, offsets, w2, w2_scale, y_sorted, stream);
}

moe_status moe_combine(const moe_problem* p, const void* y_sorted, const int32_t* inv_perm,
                       const float* topk_gate, void* y, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  REQUIRE_PTR(y_sorted);
  REQUIRE_PTR(y);
  if (!inv_perm || !topk_gate)
    return fail(MOE_ERR_INVALID_ARG, "inv_perm and topk_gate are required");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_combine(d, y_sorted, inv_perm, topk_gate, y,
                                static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_combine launch");
}

moe_status moe_bias_update(const moe_problem* p, const int32_t* expert_counts, float gamma,
                           float* bias, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if (!expert_counts || !bias)
    return fail(MOE_ERR_INVALID_ARG, "expert_counts and bias are required");
  if (!(gamma >= 0.0f) || gamma > 1e30f)
    return fail(MOE_ERR_INVALID_ARG, "gamma must be finite and >= 0");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_bias_update(d, expert_counts, gamma, bias,
                                    static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_bias_update launch");
}

moe_status moe_seq_load_stats(const moe_problem* p, const int32_t* topk_idx,
                              const int32_t* seq_offsets, int32_t n_seq, int32_t* seq_counts,
                              int32_t* seq_stats, float* seq_ratio, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if (!topk_idx || !seq_offsets || !seq_counts || !seq_stats || !seq_ratio)
    return fail(MOE_ERR_INVALID_ARG,
                "topk_idx, seq_offsets, seq_counts, seq_stats and seq_ratio are required");
  if (n_seq < 1 || n_seq > (1 << 24) || (int64_t)n_seq * d.E >= ((int64_t)1 << 31))
    return fail(MOE_ERR_INVALID_ARG, "n_seq=%d must be in [1, 2^24] with n_seq*E < 2^31", n_seq);
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_seq_load_stats(d, topk_idx, seq_offsets, n_seq, seq_counts, seq_stats,
                                       seq_ratio, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_seq_load_stats launch");
}

static moe_status require_no_fp8(const Dims& d, const char* call) {
  if (d.expert == MOE_FP8_E4M3 || d.expert == MOE_MXFP4)
    return fail(MOE_ERR_UNSUPPORTED, "%s: the backward is built for the bf16 and fp32 paths", call);
  return MOE_OK;
}

moe_status moe_combine_backward(const moe_problem* p, const void* dy, const void* y_sorted,
                                const int32_t* inv_perm, const float* topk_gate, void* dy_sorted,
                                float* dgate, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_combine_backward")) != MOE_OK) return s;
  REQUIRE_PTR(dy);
  REQUIRE_PTR(y_sorted);
  REQUIRE_PTR(dy_sorted);
  if (!inv_perm || !topk_gate || !dgate)
    return fail(MOE_ERR_INVALID_ARG, "inv_perm, topk_gate and dgate are required");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_combine_bwd(d, dy, y_sorted, inv_perm, topk_gate, dy_sorted, dgate,
                                    static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_combine_backward launch");
}

moe_status moe_router_backward(const moe_problem* p, const void* x, const float* w_router,
                               const float* logits, const int32_t* topk_idx,
                               const float* topk_gate, const float* dgate,
                               const int32_t* offsets, const int32_t* sorted_token, float* dz,
                               float* dx_router, float* dw_router, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_router_backward")) != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_router);
  REQUIRE_PTR(dx_router);
  REQUIRE_PTR(dw_router);
  if (!logits || !topk_idx || !topk_gate || !dgate || !offsets || !sorted_token || !dz)
    return fail(MOE_ERR_INVALID_ARG,
                "logits, topk_idx, topk_gate, dgate, offsets, sorted_token and dz are required");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_router_bwd(d, x, w_router, logits, topk_idx, topk_gate, dgate, offsets,
                                   sorted_token, dz, dx_router, dw_router,
                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_router_backward launch");
}

moe_status moe_unpermute_sum(const moe_problem* p, const void* dx_sorted,
                             const int32_t* inv_perm, const float* dx_router, void* dx,
                             void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_unpermute_sum")) != MOE_OK) return s;
  REQUIRE_PTR(dx_sorted);
  REQUIRE_PTR(dx);
  if (dx_router && !aligned16(dx_router))
    return fail(MOE_ERR_INVALID_ARG, "dx_router is not 16-byte aligned");
  if (!inv_perm) return fail(MOE_ERR_INVALID_ARG, "inv_perm is NULL");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_unpermute_sum(d, dx_sorted, inv_perm, dx_router, dx,
                                      static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_unpermute_sum launch");
}

moe_status moe_expert_ffn_up_save(const moe_problem* p, const void* x,
                                  const int32_t* sorted_token, const int32_t* offsets,
                                  const void* w13, void* h, void* au, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_expert_ffn_up_save")) != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w13);
  REQUIRE_PTR(h);
  REQUIRE_PTR(au);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  const int es = d.expert == MOE_F32 ? 4 : 2;
  if (sorted_token && d.T * (int64_t)d.H * es >= ((int64_t)1 << 31) - 16)
    return fail(MOE_ERR_INVALID_ARG, "T*H*%d must be < 2^31 - 16 (32-bit row offsets)", es);
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_ffn_up(d, x, nullptr, offsets, sorted_token, w13, nullptr, h, nullptr,
                               static_cast<hipStream_t>(stream), au);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_up_save launch");
}

static moe_status check_bwd_rows(const Dims& d) {
  const int es = d.expert == MOE_F32 ? 4 : 2;
  const int64_t widest = d.H > 2 * d.I ? d.H : 2 * d.I;
  if (d.R() * widest * es >= ((int64_t)1 << 31) - 16)
    return fail(MOE_ERR_INVALID_ARG,
                "R*max(H,2I)*%d must be < 2^31 - 16 (32-bit row offsets in the backward)", es);
  return MOE_OK;
}

moe_status moe_expert_ffn_backward_input(const moe_problem* p, const int32_t* offsets,
                                         const void* w13, const void* w2, const void* au,
                                         const void* dy_sorted, void* dau, void* dx_sorted,
                                         void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_expert_ffn_backward_input")) != MOE_OK) return s;
  REQUIRE_PTR(w13);
  REQUIRE_PTR(w2);
  REQUIRE_PTR(au);
  REQUIRE_PTR(dy_sorted);
  REQUIRE_PTR(dau);
  REQUIRE_PTR(dx_sorted);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if ((s = check_bwd_rows(d)) != MOE_OK) return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_ffn_bwd_input(d, offsets, w13, w2, au, dy_sorted, dau, dx_sorted,
                                      static_cast<hipStream_t>(stream));
  if (e == hipErrorNotSupported)
    return fail(MOE_ERR_UNSUPPORTED, "no backward kernel for expert dtype %d", d.expert);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_backward_input launch");
}

moe_status moe_expert_ffn_backward_weight(const moe_problem* p, const void* x,
                                          const int32_t* sorted_token, const int32_t* offsets,
                                          const void* h, const void* dy_sorted, const void* dau,
                                          float* dw13, float* dw2, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_expert_ffn_backward_weight")) != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(h);
  REQUIRE_PTR(dy_sorted);
  REQUIRE_PTR(dau);
  REQUIRE_PTR(dw13);
  REQUIRE_PTR(dw2);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if ((s = check_bwd_rows(d)) != MOE_OK) return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  hipError_t e = launch_ffn_bwd_weight(d, x, sorted_token, offsets, h, dy_sorted, dau, dw13, dw2,
                                       static_cast<hipStream_t>(stream));
  if (e == hipErrorNotSupported)
    return fail(MOE_ERR_UNSUPPORTED, "no backward kernel for expert dtype %d", d.expert);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_backward_weight launch");
}

static moe_status require_packed(const Dims& d, const char* call) {
  if (!packed_supported(d))
    return fail(MOE_ERR_UNSUPPORTED,
                "%s: packed weights are built for act dtype BF16 with expert dtype BF16 or FP8",
                call);
  return MOE_OK;
}

moe_status moe_pack_expert_weights(const moe_problem* p, const void* w13, const void* w2,
                                   void* w13_packed, void* w2_packed, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_packed(d, "moe_pack_expert_weights")) != MOE_OK) return s;
  if (!w13 && !w2) return fail(MOE_ERR_INVALID_ARG, "w13 and w2 are both NULL");
  if ((w13 && !w13_packed) || (w2 && !w2_packed))
    return fail(MOE_ERR_INVALID_ARG, "a packed output is NULL for a given input");
  if ((w13 && w13 == w13_packed) || (w2 && w2 == w2_packed))
    return fail(MOE_ERR_INVALID_ARG, "packing cannot run in place");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = d.expert == MOE_FP8_E4M3
                     ? launch_pack_weights_fp8(d, w13, w2, w13_packed, w2_packed, st)
                     : launch_pack_weights(d, w13, w2, w13_packed, w2_packed, st);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_pack_expert_weights launch");
}

static moe_status require_bf16_pair(const Dims& d, const char* call) {
  if (d.act != MOE_BF16 || d.expert != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "%s: built for act and expert dtype BF16", call);
  return MOE_OK;
}

moe_status moe_pack_expert_weights_transposed(const moe_problem* p, const void* w13,
                                              const void* w2, void* w13t_packed,
                                              void* w2t_packed, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_bf16_pair(d, "moe_pack_expert_weights_transposed")) != MOE_OK) return s;
  if (!w13 && !w2) return fail(MOE_ERR_INVALID_ARG, "w13 and w2 are both NULL");
  if ((w13 && !w13t_packed) || (w2 && !w2t_packed))
    return fail(MOE_ERR_INVALID_ARG, "a packed output is NULL for a given input");
  if ((w13 && w13 == w13t_packed) || (w2 && w2 == w2t_packed))
    return fail(MOE_ERR_INVALID_ARG, "packing cannot run in place");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e =
      launch_pack_weights_t(d, w13, w2, w13t_packed, w2t_packed, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_pack_expert_weights_transposed launch");
}

moe_status moe_expert_ffn_backward_input_packed(const moe_problem* p, const int32_t* offsets,
                                                const void* w13t_packed,
                                                const void* w2t_packed, const void* au,
                                                const void* dy_sorted, void* dau,
                                                void* dx_sorted, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_bf16_pair(d, "moe_expert_ffn_backward_input_packed")) != MOE_OK) return s;
  REQUIRE_PTR(w13t_packed);
  REQUIRE_PTR(w2t_packed);
  REQUIRE_PTR(au);
  REQUIRE_PTR(dy_sorted);
  REQUIRE_PTR(dau);
  REQUIRE_PTR(dx_sorted);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if ((s = check_bwd_rows(d)) != MOE_OK) return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_ffn_bwd_input_packed(d, offsets, w13t_packed, w2t_packed, au,
                                                   dy_sorted, dau, dx_sorted,
                                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_backward_input_packed launch");
}

moe_status moe_expert_ffn_up_packed(const moe_problem* p, const void* x, const float* x_scale,
                                    const int32_t* sorted_token, const int32_t* offsets,
                                    const void* w13, const void* w13_packed,
                                    const float* w13_scale, void* h, float* h_scale, void* au,
                                    void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_packed(d, "moe_expert_ffn_up_packed")) != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w13);
  REQUIRE_PTR(w13_packed);
  REQUIRE_PTR(h);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  const bool fp8 = d.expert == MOE_FP8_E4M3;
  if (fp8 && (!x_scale || !w13_scale || !h_scale))
    return fail(MOE_ERR_INVALID_ARG, "the FP8 path needs x_scale, w13_scale, h_scale");
  if (fp8 && au)
    return fail(MOE_ERR_INVALID_ARG, "au (the pre-activations) is kept by the bf16 path only");
  const int es = fp8 ? 1 : 2;
  if (sorted_token && d.T * (int64_t)d.H * es >= ((int64_t)1 << 31) - 16)
    return fail(MOE_ERR_INVALID_ARG, "T*H*%d must be < 2^31 - 16 (32-bit row offsets)", es);
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = fp8 ? launch_ffn_up_packed_fp8(d, x, x_scale, offsets, sorted_token, w13,
                                                w13_packed, w13_scale, h, h_scale, st)
                     : launch_ffn_up_packed(d, x, offsets, sorted_token, w13, w13_packed, h, au,
                                            st);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_up_packed launch");
}

moe_status moe_expert_ffn_down_packed(const moe_problem* p, const void* h, const float* h_scale,
                                      const int32_t* offsets, const void* w2_packed,
                                      const float* w2_scale, void* y_sorted, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_packed(d, "moe_expert_ffn_down_packed")) != MOE_OK) return s;
  REQUIRE_PTR(h);
  REQUIRE_PTR(w2_packed);
  REQUIRE_PTR(y_sorted);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  const bool fp8 = d.expert == MOE_FP8_E4M3;
  if (fp8 && (!h_scale || !w2_scale))
    return fail(MOE_ERR_INVALID_ARG, "the FP8 path needs h_scale and w2_scale");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = fp8 ? launch_ffn_down_packed_fp8(d, h, h_scale, offsets, w2_packed, w2_scale,
                                                  y_sorted, st)
                     : launch_ffn_down_packed(d, h, offsets, w2_packed, y_sorted, st);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_down_packed launch");
}

moe_status moe_quantize_weights_fp8(const void* w_bf16, void* w_fp8, float* scale,
                                    int64_t batch, int32_t rows, int32_t cols, void* stream) {
  if (batch < 1 || rows < 128 || cols < 128 || rows % 128 || cols % 128)
    return fail(MOE_ERR_INVALID_ARG, "batch >= 1 and rows, cols multiples of 128 are required");
  if (batch * (rows / 128) * (int64_t)(cols / 128) >= ((int64_t)1 << 31))
    return fail(MOE_ERR_INVALID_ARG, "too many 128x128 blocks");
  REQUIRE_PTR(w_bf16);
  REQUIRE_PTR(w_fp8);
  if (!scale) return fail(MOE_ERR_INVALID_ARG, "scale is NULL");
  moe_status s = check_device(nullptr);
  if (s != MOE_OK) return s;
  hipError_t e = launch_quantize_weights(static_cast<const uint16_t*>(w_bf16),
                                         static_cast<uint8_t*>(w_fp8), scale, batch, rows, cols,
                                         static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_quantize_weights_fp8 launch");
}

static moe_status check_sequences(int32_t n_seq) {
  // one workgroup of 1024 threads a sequence; a launch holds fewer than 2^32 threads
  if (n_seq < 1 || n_seq >= (1 << 22))
    return fail(MOE_ERR_INVALID_ARG, "n_seq=%d must be in [1, 2^22)", n_seq);
  return MOE_OK;
}

static moe_status check_ws(const char* call, const void* ws, size_t got, size_t need) {
  if (need && (!ws || got < need || !aligned16(ws)))
    return fail(MOE_ERR_WORKSPACE, "%s needs %zu workspace bytes, 16-byte aligned, got %zu", call,
                need, ws ? got : (size_t)0);
  return MOE_OK;
}

size_t moe_balance_loss_workspace_bytes(const moe_problem* p, int32_t n_seq) {
  Dims d;
  if (validate(p, &d) != MOE_OK || check_sequences(n_seq) != MOE_OK) return 0;
  return balance_ws_bytes(d, n_seq);
}

moe_status moe_balance_loss(const moe_problem* p, const float* logits, const int32_t* topk_idx,
                            const int32_t* seq_offsets, int32_t n_seq, int32_t* seq_counts,
                            float* seq_prob, float* seq_loss, void* ws, size_t ws_bytes,
                            void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = check_sequences(n_seq)) != MOE_OK) return s;
  REQUIRE_PTR(logits);
  REQUIRE_PTR(topk_idx);
  REQUIRE_PTR(seq_counts);
  REQUIRE_PTR(seq_prob);
  if (!seq_offsets || !seq_loss)
    return fail(MOE_ERR_INVALID_ARG, "seq_offsets and seq_loss are required");
  if ((s = check_ws("moe_balance_loss", ws, ws_bytes, balance_ws_bytes(d, n_seq))) != MOE_OK)
    return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_balance_loss(d, logits, topk_idx, seq_offsets, n_seq, seq_counts,
                                           seq_prob, seq_loss, ws,
                                           static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_balance_loss launch");
}

moe_status moe_balance_loss_backward(const moe_problem* p, const float* logits,
                                     const int32_t* seq_offsets, int32_t n_seq,
                                     const int32_t* seq_counts, const float* dseq_loss,
                                     const int32_t* topk_idx, const float* topk_gate,
                                     const float* dgate, float* dlogits, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = check_sequences(n_seq)) != MOE_OK) return s;
  REQUIRE_PTR(logits);
  REQUIRE_PTR(seq_counts);
  REQUIRE_PTR(dlogits);
  if (!seq_offsets || !dseq_loss)
    return fail(MOE_ERR_INVALID_ARG, "seq_offsets and dseq_loss are required");
  if (dgate && (!topk_idx || !topk_gate))
    return fail(MOE_ERR_INVALID_ARG, "dgate needs topk_idx and topk_gate");
  if (dlogits == logits)
    return fail(MOE_ERR_INVALID_ARG, "dlogits cannot be written over logits");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_balance_bwd(d, logits, seq_offsets, n_seq, seq_counts, dseq_loss,
                                          topk_idx, topk_gate, dgate, dlogits,
                                          static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_balance_loss_backward launch");
}

moe_status moe_router_backward_dense(const moe_problem* p, const void* x, const float* w_router,
                                     const float* dlogits, float* dx_router, float* dw_router,
                                     void* ws, size_t ws_bytes, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_router);
  REQUIRE_PTR(dlogits);
  REQUIRE_PTR(dx_router);
  REQUIRE_PTR(dw_router);
  // a launch holds fewer than 2^32 threads
  if (d.T > (1 << 25) || d.T * d.H > ((int64_t)1 << 36))
    return fail(MOE_ERR_INVALID_ARG, "T=%lld must be <= 2^25 with T*H <= 2^36", (long long)d.T);
  if ((s = check_ws("moe_router_backward_dense", ws, ws_bytes, router_dense_ws_bytes(d))) != MOE_OK)
    return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_router_dense_bwd(d, x, w_router, dlogits, dx_router, dw_router, ws,
                                               static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_router_backward_dense launch");
}

moe_status moe_checkpoint_save(const moe_problem* p, const void* au, void* au_q, float* au_scale,
                               void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_checkpoint_save")) != MOE_OK) return s;
  REQUIRE_PTR(au);
  REQUIRE_PTR(au_q);
  if (!au_scale) return fail(MOE_ERR_INVALID_ARG, "au_scale is NULL");
  if (au == au_q) return fail(MOE_ERR_INVALID_ARG, "the codes cannot be written over au");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e =
      launch_quantize_fp8(au, d.act, d.R(), 2 * (int64_t)d.I, 2 * (int64_t)d.I,
                          static_cast<uint8_t*>(au_q), 2 * (int64_t)d.I, au_scale, nullptr, 0,
                          nullptr, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_checkpoint_save launch");
}

moe_status moe_checkpoint_restore(const moe_problem* p, const void* au_q, const float* au_scale,
                                  void* au, void* h, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_no_fp8(d, "moe_checkpoint_restore")) != MOE_OK) return s;
  REQUIRE_PTR(au_q);
  if (!au_scale) return fail(MOE_ERR_INVALID_ARG, "au_scale is NULL");
  if (!au && !h) return fail(MOE_ERR_INVALID_ARG, "au and h are both NULL");
  if (!aligned16(au) || !aligned16(h))
    return fail(MOE_ERR_INVALID_ARG, "au or h is not 16-byte aligned");
  if (au == au_q || h == au_q || (au && au == h))
    return fail(MOE_ERR_INVALID_ARG, "au, h and au_q must be buffers of their own");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_ckpt_restore(d, static_cast<const uint8_t*>(au_q), au_scale, au, h,
                                           static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_checkpoint_restore launch");
}

moe_status moe_expert_ffn_backward_input_checkpoint(const moe_problem* p, const int32_t* offsets,
                                                    const void* w13t_packed,
                                                    const void* w2t_packed, const void* au_q,
                                                    const float* au_scale,
                                                    const void* dy_sorted, void* dau, void* h,
                                                    void* dx_sorted, void* stream) {
  Dims d;
  moe_status s = validate(p, &d);
  if (s != MOE_OK) return s;
  if ((s = require_bf16_pair(d, "moe_expert_ffn_backward_input_checkpoint")) != MOE_OK) return s;
  REQUIRE_PTR(w13t_packed);
  REQUIRE_PTR(w2t_packed);
  REQUIRE_PTR(au_q);
  REQUIRE_PTR(dy_sorted);
  REQUIRE_PTR(dau);
  REQUIRE_PTR(h);
  REQUIRE_PTR(dx_sorted);
  if (!offsets || !au_scale)
    return fail(MOE_ERR_INVALID_ARG, "offsets and au_scale are required");
  if ((s = check_bwd_rows(d)) != MOE_OK) return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_ffn_bwd_input_packed(
      d, offsets, w13t_packed, w2t_packed, nullptr, dy_sorted, dau, dx_sorted,
      static_cast<hipStream_t>(stream), static_cast<const uint8_t*>(au_q), au_scale, h);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_backward_input_checkpoint launch");
}

moe_status moe_quantize_fp8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                            void* q, int64_t ldq, float* scale, void* qt, int64_t ldqt,
                            float* scale_t, void* stream) {
  if (dtype != MOE_BF16 && dtype != MOE_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d must be MOE_BF16 or MOE_F32", dtype);
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (rows < 1 || cols < 1 || rows > kMost || cols > kMost)
    return fail(MOE_ERR_INVALID_ARG, "rows and cols must be in [1, 2^40]");
  // the transpose takes a workgroup of 256 threads a block, and a launch holds fewer than 2^32
  if (((rows + 127) / 128) * (double)((cols + 127) / 128) >= (qt ? 16777216.0 : 2147483648.0))
    return fail(MOE_ERR_INVALID_ARG, "too many 128x128 blocks");
  if (ldx < cols) return fail(MOE_ERR_INVALID_ARG, "ldx=%lld < cols", (long long)ldx);
  if (!x || (reinterpret_cast<uintptr_t>(x) & (dtype == MOE_F32 ? 3 : 1)))
    return fail(MOE_ERR_INVALID_ARG, "x is NULL or not aligned to its element");
  if (!q && !qt) return fail(MOE_ERR_INVALID_ARG, "q and qt are both NULL");
  if (q && (!aligned16(q) || !scale || ldq < cols || ldq % 16))
    return fail(MOE_ERR_INVALID_ARG,
                "q needs 16-byte alignment, scale and ldq >= cols, a multiple of 16");
  if (qt && (!aligned16(qt) || !scale_t || ldqt < rows || ldqt % 16))
    return fail(MOE_ERR_INVALID_ARG,
                "qt needs 16-byte alignment, scale_t and ldqt >= rows, a multiple of 16");
  if (x == q || x == qt || (q && q == qt))
    return fail(MOE_ERR_INVALID_ARG, "x, q and qt must be buffers of their own");
  moe_status s = check_device(nullptr);
  if (s != MOE_OK) return s;
  const hipError_t e = launch_quantize_fp8(x, dtype, rows, cols, ldx, static_cast<uint8_t*>(q),
                                           ldq, scale, static_cast<uint8_t*>(qt), ldqt, scale_t,
                                           static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_quantize_fp8 launch");
}

static moe_status check_gemm_fp8(int64_t M, int64_t N, int64_t K) {
  // workgroups of 512 threads take 16 columns (few rows) or tiles of 128 x 64 to 256 x 256, and
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kMost = (int64_t)1 << 26;
  if (M < 1 || N < 1 || K < 1 || M > kMost || N > kMost || K > ((int64_t)1 << 22))
    return fail(MOE_ERR_INVALID_ARG, "M, N must be in [1, 2^26] and K in [1, 2^22]");
  if (M * N > ((int64_t)1 << 37)) return fail(MOE_ERR_INVALID_ARG, "M*N must be <= 2^37");
  return MOE_OK;
}

size_t moe_gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (check_gemm_fp8(M, N, K) != MOE_OK) return 0;
  return gemm_fp8_ws_bytes(M, N, K);
}

moe_status moe_gemm_fp8(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda,
                        const float* a_scale, const void* b, int64_t ldb, const float* b_scale,
                        int32_t b_rows, void* c, int64_t ldc, int32_t c_dtype, int32_t accumulate,
                        void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_gemm_fp8(M, N, K);
  if (s != MOE_OK) return s;
  REQUIRE_PTR(a);
  REQUIRE_PTR(b);
  REQUIRE_PTR(c);
  if (!a_scale || !b_scale)
    return fail(MOE_ERR_INVALID_ARG, "a_scale and b_scale are required");
  constexpr int64_t kMostLd = (int64_t)1 << 22;
  if (lda < K || ldb < K || lda % 16 || ldb % 16 || lda > kMostLd || ldb > kMostLd)
    return fail(MOE_ERR_INVALID_ARG,
                "lda and ldb must be multiples of 16, at least K and at most 2^22");
  if (ldc < N) return fail(MOE_ERR_INVALID_ARG, "ldc=%lld < N", (long long)ldc);
  if (b_rows != 1 && b_rows != 128)
    return fail(MOE_ERR_INVALID_ARG, "b_rows=%d must be 1 or 128", b_rows);
  if (c_dtype != MOE_BF16 && c_dtype != MOE_F32)
    return fail(MOE_ERR_INVALID_ARG, "c_dtype=%d must be MOE_BF16 or MOE_F32", c_dtype);
  if (accumulate != 0 && (accumulate != 1 || c_dtype != MOE_F32))
    return fail(MOE_ERR_INVALID_ARG, "accumulate must be 0, or 1 with c_dtype MOE_F32");
  if (c == a || c == b) return fail(MOE_ERR_INVALID_ARG, "c cannot be written over a or b");
  if ((s = check_ws("moe_gemm_fp8", ws, ws_bytes, gemm_fp8_ws_bytes(M, N, K))) != MOE_OK) return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_gemm_fp8(
      M, N, K, static_cast<const uint8_t*>(a), lda, a_scale, static_cast<const uint8_t*>(b), ldb,
      b_scale, b_rows, c, ldc, c_dtype == MOE_F32, accumulate, ws,
      static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_gemm_fp8 launch");
}

// ---- MXFP4 ----
static moe_status require_mxfp4(const Dims& d, const char* call) {
  if (d.expert != MOE_MXFP4)
    return fail(MOE_ERR_INVALID_ARG, "%s needs act BF16 and expert MXFP4", call);
  return MOE_OK;
}

// a workgroup of 256 threads a tile of 128 rows x 256 columns, somewhat more of them than tiles,
// and a launch holds fewer than 2^32 threads
static moe_status check_mx_tiles(const Dims& d) {
  const int64_t wide = d.H > 2 * d.I ? d.H : 2 * d.I;
  if ((d.E + d.S + d.R() / 128) * ((wide + 255) / 256) >= ((int64_t)1 << 23))
    return fail(MOE_ERR_INVALID_ARG, "(E+S+R/128)*max(2I,H)/256 must be < 2^23");
  return MOE_OK;
}

// codes and scales of a quantised matrix [rows, cols]: `name` in messages
static moe_status check_mx(const char* name, const void* q, int64_t ldq, const void* scale,
                           int64_t lds, int64_t cols) {
  const int64_t kb = (cols + 31) / 32;
  if (!aligned16(q) || ldq % 16 || ldq < 16 * kb)
    return fail(MOE_ERR_INVALID_ARG,
                "%s needs 16-byte alignment and a row stride of at least 16*ceil(%lld/32) bytes, a "
                "multiple of 16", name, (long long)cols);
  if (!scale || !aligned16(scale) || lds % 16 || lds < kb)
    return fail(MOE_ERR_INVALID_ARG,
                "%s's scales need 16-byte alignment and a row stride of at least ceil(%lld/32) "
                "bytes, a multiple of 16", name, (long long)cols);
  return MOE_OK;
}

moe_status moe_quantize_mxfp4(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                              void* q, int64_t ldq, void* scale, int64_t lds, void* qt,
                              int64_t ldqt, void* scale_t, int64_t ldst, const void* random,
                              void* stream) {
  if (dtype != MOE_BF16 && dtype != MOE_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d must be MOE_BF16 or MOE_F32", dtype);
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (rows < 1 || cols < 1 || rows > kMost || cols > kMost)
    return fail(MOE_ERR_INVALID_ARG, "rows and cols must be in [1, 2^40]");
  // the transpose takes two workgroups of 256 threads a block, and a launch holds fewer than 2^32
  if (((rows + 127) / 128) * (double)((cols + 127) / 128) >= (qt ? 8388608.0 : 2147483648.0))
    return fail(MOE_ERR_INVALID_ARG, "too many 128x128 blocks");
  if (ldx < cols) return fail(MOE_ERR_INVALID_ARG, "ldx=%lld < cols", (long long)ldx);
  if (!x || (reinterpret_cast<uintptr_t>(x) & (dtype == MOE_F32 ? 3 : 1)))
    return fail(MOE_ERR_INVALID_ARG, "x is NULL or not aligned to its element");
  if (!q && !qt) return fail(MOE_ERR_INVALID_ARG, "q and qt are both NULL");
  moe_status s;
  if (q && (s = check_mx("q", q, ldq, scale, lds, cols)) != MOE_OK) return s;
  if (qt && (s = check_mx("qt", qt, ldqt, scale_t, ldst, rows)) != MOE_OK) return s;
  const void* outs[4] = {q, q ? scale : nullptr, qt, qt ? scale_t : nullptr};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    bool twice = outs[i] == x || outs[i] == random;
    for (int j = 0; j < i; ++j) twice = twice || outs[i] == outs[j];
    if (twice)
      return fail(MOE_ERR_INVALID_ARG, "codes and scales need buffers of their own");
  }
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_quantize_mxfp4(
      x, dtype, rows, cols, ldx, static_cast<const uint8_t*>(random), static_cast<uint8_t*>(q), ldq,
      static_cast<uint8_t*>(scale), lds, static_cast<uint8_t*>(qt), ldqt,
      static_cast<uint8_t*>(scale_t), ldst, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_quantize_mxfp4 launch");
}

moe_status moe_dequantize_mxfp4(int64_t rows, int64_t cols, const void* q, int64_t ldq,
                                const void* scale, int64_t lds, void* out, int64_t ldo,
                                int32_t dtype, void* stream) {
  if (dtype != MOE_BF16 && dtype != MOE_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d must be MOE_BF16 or MOE_F32", dtype);
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (rows < 1 || cols < 1 || rows > kMost || cols > kMost ||
      rows * (double)cols >= 1.15e18)
    return fail(MOE_ERR_INVALID_ARG, "rows and cols must be in [1, 2^40], rows*cols < 2^60");
  if (!q) return fail(MOE_ERR_INVALID_ARG, "q is NULL");
  moe_status s = check_mx("q", q, ldq, scale, lds, cols);
  if (s != MOE_OK) return s;
  if (ldo < cols) return fail(MOE_ERR_INVALID_ARG, "ldo=%lld < cols", (long long)ldo);
  if (!out || (reinterpret_cast<uintptr_t>(out) & (dtype == MOE_F32 ? 3 : 1)))
    return fail(MOE_ERR_INVALID_ARG, "out is NULL or not aligned to its element");
  if (out == q || out == scale)
    return fail(MOE_ERR_INVALID_ARG, "out needs a buffer of its own");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_dequantize_mxfp4(
      rows, cols, static_cast<const uint8_t*>(q), ldq, static_cast<const uint8_t*>(scale), lds, out,
      ldo, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dequantize_mxfp4 launch");
}

size_t moe_gemm_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (check_gemm_fp8(M, N, K) != MOE_OK) return 0;
  return gemm_mxfp4_ws_bytes(M, N, K);
}

moe_status moe_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda,
                          const void* a_scale, int64_t ldsa, const void* b, int64_t ldb,
                          const void* b_scale, int64_t ldsb, void* c, int64_t ldc, int32_t c_dtype,
                          int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_gemm_fp8(M, N, K);  // the same limits
  if (s != MOE_OK) return s;
  REQUIRE_PTR(a);
  REQUIRE_PTR(b);
  REQUIRE_PTR(c);
  if ((s = check_mx("a", a, lda, a_scale, ldsa, K)) != MOE_OK) return s;
  if ((s = check_mx("b", b, ldb, b_scale, ldsb, K)) != MOE_OK) return s;
  constexpr int64_t kMostLd = (int64_t)1 << 22;
  if (lda > kMostLd || ldb > kMostLd || ldsa > kMostLd || ldsb > kMostLd)
    return fail(MOE_ERR_INVALID_ARG, "row strides must be at most 2^22 bytes");
  if (ldc < N) return fail(MOE_ERR_INVALID_ARG, "ldc=%lld < N", (long long)ldc);
  if (c_dtype != MOE_BF16 && c_dtype != MOE_F32)
    return fail(MOE_ERR_INVALID_ARG, "c_dtype=%d must be MOE_BF16 or MOE_F32", c_dtype);
  if (accumulate != 0 && (accumulate != 1 || c_dtype != MOE_F32))
    return fail(MOE_ERR_INVALID_ARG, "accumulate must be 0, or 1 with c_dtype MOE_F32");
  if (c == a || c == b || c == a_scale || c == b_scale)
    return fail(MOE_ERR_INVALID_ARG, "c cannot be written over an operand");
  if ((s = check_ws("moe_gemm_mxfp4", ws, ws_bytes, gemm_mxfp4_ws_bytes(M, N, K))) != MOE_OK)
    return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_gemm_mxfp4(
      M, N, K, static_cast<const uint8_t*>(a), lda, static_cast<const uint8_t*>(a_scale), ldsa,
      static_cast<const uint8_t*>(b), ldb, static_cast<const uint8_t*>(b_scale), ldsb, c, ldc,
      c_dtype == MOE_F32, accumulate, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_gemm_mxfp4 launch");
}

size_t moe_mxfp4_packed_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 1 || batch > 65536 || rows < 64 || rows % 64 || rows > 65536 || cols < 128 ||
      cols % 128 || cols > 65536) {
    fail(MOE_ERR_INVALID_ARG,
         "batch must be in [1, 65536], rows a multiple of 64 and cols of 128, at most 65536");
    return 0;
  }
  return (size_t)batch * rows * cols / 32 * 17;
}

moe_status moe_pack_expert_weights_mxfp4(const moe_problem* p, const void* w13,
                                         const void* w13_scale, const void* w2,
                                         const void* w2_scale, void* w13_packed, void* w2_packed,
                                         void* stream) {
  Dims d;
  moe_status s = validate(p, &d, true);
  if (s != MOE_OK) return s;
  if ((s = require_mxfp4(d, "moe_pack_expert_weights_mxfp4")) != MOE_OK) return s;
  if (!w13_packed && !w2_packed)
    return fail(MOE_ERR_INVALID_ARG, "w13_packed and w2_packed are both NULL");
  const void* in[4] = {w13, w13_scale, w2, w2_scale};
  const char* name[4] = {"w13", "w13_scale", "w2", "w2_scale"};
  for (int i = 0; i < 4; ++i) {
    if (!(i < 2 ? w13_packed : w2_packed)) continue;
    if (!in[i]) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name[i]);
    if (!aligned16(in[i])) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name[i]);
    if (in[i] == w13_packed || in[i] == w2_packed)
      return fail(MOE_ERR_INVALID_ARG, "packed weights need buffers of their own");
  }
  if (!aligned16(w13_packed) || !aligned16(w2_packed))
    return fail(MOE_ERR_INVALID_ARG, "w13_packed or w2_packed is not 16-byte aligned");
  if (w13_packed == w2_packed)
    return fail(MOE_ERR_INVALID_ARG, "packed weights need buffers of their own");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (w13_packed)
    e = launch_pack_mxfp4(static_cast<const uint8_t*>(w13), static_cast<const uint8_t*>(w13_scale),
                          static_cast<uint8_t*>(w13_packed), d.E + d.S, 2 * d.I, d.H, true, st);
  if (e == hipSuccess && w2_packed)
    e = launch_pack_mxfp4(static_cast<const uint8_t*>(w2), static_cast<const uint8_t*>(w2_scale),
                          static_cast<uint8_t*>(w2_packed), d.E + d.S, d.H, d.I, false, st);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_pack_expert_weights_mxfp4 launch");
}

moe_status moe_expert_ffn_up_mxfp4(const moe_problem* p, const void* x_q, const void* x_scale,
                                   int64_t ldxs, const int32_t* sorted_token,
                                   const int32_t* offsets, const void* w13_packed, void* h_q,
                                   void* h_scale, int64_t ldhs, void* stream) {
  Dims d;
  moe_status s = validate(p, &d, true);
  if (s != MOE_OK) return s;
  if ((s = require_mxfp4(d, "moe_expert_ffn_up_mxfp4")) != MOE_OK) return s;
  if ((s = check_mx_tiles(d)) != MOE_OK) return s;
  REQUIRE_PTR(x_q);
  REQUIRE_PTR(w13_packed);
  REQUIRE_PTR(h_q);
  if ((s = check_mx("x_q", x_q, d.H / 2, x_scale, ldxs, d.H)) != MOE_OK) return s;
  if ((s = check_mx("h_q", h_q, d.I / 2, h_scale, ldhs, d.I)) != MOE_OK) return s;
  if (!sorted_token || !offsets)
    return fail(MOE_ERR_INVALID_ARG, "sorted_token and offsets are required");
  if (d.T * (d.H / 2) >= ((int64_t)1 << 31) - 16 || d.T * ldxs >= ((int64_t)1 << 31) - 16 ||
      ldhs > ((int64_t)1 << 22))
    return fail(MOE_ERR_INVALID_ARG,
                "T*H/2 and T*ldxs must be < 2^31 - 16 (32-bit row offsets), ldhs at most 2^22");
  if (h_q == x_q || h_q == h_scale || h_scale == x_scale || h_q == x_scale || h_scale == x_q)
    return fail(MOE_ERR_INVALID_ARG, "h_q and h_scale need buffers of their own");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_ffn_up_mxfp4(
      d, static_cast<const uint8_t*>(x_q), static_cast<const uint8_t*>(x_scale), ldxs, sorted_token,
      offsets, static_cast<const uint8_t*>(w13_packed), static_cast<uint8_t*>(h_q),
      static_cast<uint8_t*>(h_scale), ldhs, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_up_mxfp4 launch");
}

moe_status moe_expert_ffn_down_mxfp4(const moe_problem* p, const void* h_q, const void* h_scale,
                                     int64_t ldhs, const int32_t* offsets, const void* w2_packed,
                                     void* y_sorted, void* stream) {
  Dims d;
  moe_status s = validate(p, &d, true);
  if (s != MOE_OK) return s;
  if ((s = require_mxfp4(d, "moe_expert_ffn_down_mxfp4")) != MOE_OK) return s;
  if ((s = check_mx_tiles(d)) != MOE_OK) return s;
  REQUIRE_PTR(h_q);
  REQUIRE_PTR(w2_packed);
  REQUIRE_PTR(y_sorted);
  if ((s = check_mx("h_q", h_q, d.I / 2, h_scale, ldhs, d.I)) != MOE_OK) return s;
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if (ldhs > ((int64_t)1 << 22)) return fail(MOE_ERR_INVALID_ARG, "ldhs must be at most 2^22");
  if (y_sorted == h_q || y_sorted == h_scale)
    return fail(MOE_ERR_INVALID_ARG, "y_sorted needs a buffer of its own");
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_ffn_down_mxfp4(
      d, static_cast<const uint8_t*>(h_q), static_cast<const uint8_t*>(h_scale), ldhs, offsets,
      static_cast<const uint8_t*>(w2_packed), y_sorted, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_expert_ffn_down_mxfp4 launch");
}

// ---- a share of the experts ----
static moe_status check_pairs(int64_t T, int32_t K) {
  if (K < 1 || K > 16) return fail(MOE_ERR_INVALID_ARG, "K=%d must be in [1,16]", K);
  if (T < 0 || T > ((int64_t)1 << 31) / K - 1024)
    return fail(MOE_ERR_INVALID_ARG, "T=%lld must be >= 0 with T*K < 2^31 - 1024*K", (long long)T);
  return MOE_OK;
}

size_t moe_sort_by_expert_workspace_bytes(int64_t T, int32_t K, int32_t count) {
  if (check_pairs(T, K) != MOE_OK) return 0;
  if (count < 1 || count > 512) {
    fail(MOE_ERR_INVALID_ARG, "count=%d must be in [1,512]", count);
    return 0;
  }
  return sort_ws_bytes(T * K, count) + 16;
}

moe_status moe_sort_by_expert(int64_t T, int32_t K, const int32_t* topk_idx, int32_t first,
                              int32_t count, int32_t* offsets, int32_t* sorted_token,
                              int32_t* pair_row, void* ws, size_t ws_bytes, void* stream) {
  const size_t need = moe_sort_by_expert_workspace_bytes(T, K, count);
  if (!need) return MOE_ERR_INVALID_ARG;
  if (first < 0) return fail(MOE_ERR_INVALID_ARG, "first=%d must be >= 0", first);
  if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
  if (T && (!topk_idx || !sorted_token || !pair_row))
    return fail(MOE_ERR_INVALID_ARG, "topk_idx, sorted_token and pair_row are required");
  if (T && (topk_idx == pair_row || topk_idx == sorted_token || sorted_token == pair_row))
    return fail(MOE_ERR_INVALID_ARG, "topk_idx, sorted_token and pair_row need buffers of their own");
  moe_status s = MOE_OK;
  if (T && (s = check_ws("moe_sort_by_expert", ws, ws_bytes, need)) != MOE_OK) return s;
  if ((s = check_device(nullptr)) != MOE_OK) return s;
  const hipError_t e = launch_sort_by_expert(T * K, K, topk_idx, first, count, offsets,
                                             sorted_token, pair_row, ws,
                                             static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_sort_by_expert launch");
}

// a matrix of `dtype` rows; `there` false: not used
static moe_status check_rows(const char* name, bool there, const void* x, int64_t ld, int64_t H,
                             int32_t dtype) {
  if (!there) return MOE_OK;
  if (!x) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(x) & (dtype == MOE_F32 ? 3 : 1))
    return fail(MOE_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  if (ld < H || ld > ((int64_t)1 << 31))
    return fail(MOE_ERR_INVALID_ARG, "the row stride of %s must be at least H and at most 2^31",
                name);
  return MOE_OK;
}

static moe_status check_move(int32_t dtype, int64_t T, int32_t K, int64_t H, const void* row) {
  if (dtype != MOE_BF16 && dtype != MOE_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d must be MOE_BF16 or MOE_F32", dtype);
  moe_status s = check_pairs(T, K);
  if (s != MOE_OK) return s;
  if (H < 1 || H > ((int64_t)1 << 20))
    return fail(MOE_ERR_INVALID_ARG, "H=%lld must be in [1, 2^20]", (long long)H);
  if (T && !row) return fail(MOE_ERR_INVALID_ARG, "pair_row is NULL");
  return MOE_OK;
}

moe_status moe_dispatch(int32_t dtype, int64_t T, int32_t K, int64_t H, const void* x, int64_t ldx,
                        const int32_t* pair_row, const float* weights, void* x_sorted, int64_t ldxs,
                        void* stream) {
  moe_status s = check_move(dtype, T, K, H, pair_row);
  if (s != MOE_OK) return s;
  if ((s = check_rows("x", T > 0, x, ldx, H, dtype)) != MOE_OK) return s;
  if ((s = check_rows("x_sorted", T > 0, x_sorted, ldxs, H, dtype)) != MOE_OK) return s;
  if (T && x == x_sorted)
    return fail(MOE_ERR_INVALID_ARG, "x_sorted needs a buffer of its own");
  if ((s = check_device(nullptr)) != MOE_OK || T == 0) return s;
  const hipError_t e = launch_spread(dtype, T, K, H, x, ldx, pair_row, weights, nullptr, 0,
                                     x_sorted, ldxs, nullptr, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dispatch launch");
}

moe_status moe_dispatch_backward(int32_t dtype, int64_t T, int32_t K, int64_t H,
                                 const void* dx_sorted, int64_t lddxs, const int32_t* pair_row,
                                 const float* weights, const void* x, int64_t ldx, void* dx,
                                 int64_t lddx, float* dweights, void* stream) {
  moe_status s = check_move(dtype, T, K, H, pair_row);
  if (s != MOE_OK) return s;
  if (dweights && !weights)
    return fail(MOE_ERR_INVALID_ARG, "dweights without weights");
  if ((s = check_rows("dx_sorted", T > 0, dx_sorted, lddxs, H, dtype)) != MOE_OK) return s;
  if ((s = check_rows("x", T > 0 && dweights, x, ldx, H, dtype)) != MOE_OK) return s;
  if ((s = check_rows("dx", T > 0, dx, lddx, H, dtype)) != MOE_OK) return s;
  if (T && (dx == dx_sorted || (dweights && dx == x)))
    return fail(MOE_ERR_INVALID_ARG, "dx needs a buffer of its own");
  if ((s = check_device(nullptr)) != MOE_OK || T == 0) return s;
  const hipError_t e =
      launch_gather(dtype, T, K, H, dx_sorted, lddxs, pair_row, weights, dweights ? x : nullptr,
                    dweights ? ldx : 0, dx, lddx, dweights, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_dispatch_backward launch");
}

moe_status moe_collect(int32_t dtype, int64_t T, int32_t K, int64_t H, const void* y_sorted,
                       int64_t ldys, const int32_t* pair_row, const float* weights, void* y,
                       int64_t ldy, void* stream) {
  moe_status s = check_move(dtype, T, K, H, pair_row);
  if (s != MOE_OK) return s;
  if ((s = check_rows("y_sorted", T > 0, y_sorted, ldys, H, dtype)) != MOE_OK) return s;
  if ((s = check_rows("y", T > 0, y, ldy, H, dtype)) != MOE_OK) return s;
  if (T && y == y_sorted) return fail(MOE_ERR_INVALID_ARG, "y needs a buffer of its own");
  if ((s = check_device(nullptr)) != MOE_OK || T == 0) return s;
  const hipError_t e = launch_gather(dtype, T, K, H, y_sorted, ldys, pair_row, weights, nullptr, 0,
                                     y, ldy, nullptr, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_collect launch");
}

moe_status moe_collect_backward(int32_t dtype, int64_t T, int32_t K, int64_t H, const void* dy,
                                int64_t lddy, const int32_t* pair_row, const float* weights,
                                const void* y_sorted, int64_t ldys, void* dy_sorted, int64_t lddys,
                                float* dweights, void* stream) {
  moe_status s = check_move(dtype, T, K, H, pair_row);
  if (s != MOE_OK) return s;
  if (dweights && !weights)
    return fail(MOE_ERR_INVALID_ARG, "dweights without weights");
  if ((s = check_rows("dy", T > 0, dy, lddy, H, dtype)) != MOE_OK) return s;
  if ((s = check_rows("y_sorted", T > 0 && dweights, y_sorted, ldys, H, dtype)) != MOE_OK)
    return s;
  if ((s = check_rows("dy_sorted", T > 0, dy_sorted, lddys, H, dtype)) != MOE_OK) return s;
  if (T && (dy_sorted == dy || (dweights && dy_sorted == y_sorted)))
    return fail(MOE_ERR_INVALID_ARG, "dy_sorted needs a buffer of its own");
  if ((s = check_device(nullptr)) != MOE_OK || T == 0) return s;
  const hipError_t e = launch_spread(dtype, T, K, H, dy, lddy, pair_row, weights,
                                     dweights ? y_sorted : nullptr, dweights ? ldys : 0, dy_sorted,
                                     lddys, dweights, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_collect_backward launch");
}

}  // extern "C"
