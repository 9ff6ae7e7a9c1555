// Launchers of the MXFP4 operators and of a share of the experts (definitions in the files
// named below; argument checks in api.hip).
#pragma once
#include "common.h"

namespace moe {

// MXFP4 (quant_mxfp4.hip, gemm_mxfp4.hip, experts_mxfp4.hip)
hipError_t launch_quantize_mxfp4(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                                 const uint8_t* rnd, uint8_t* q, int64_t ldq, uint8_t* scale,
                                 int64_t lds, uint8_t* qt, int64_t ldqt, uint8_t* scale_t,
                                 int64_t ldst, hipStream_t st);
hipError_t launch_dequantize_mxfp4(int64_t rows, int64_t cols, const uint8_t* q, int64_t ldq,
                                   const uint8_t* scale, int64_t lds, void* out, int64_t ldo,
                                   int dtype, hipStream_t st);
size_t gemm_mxfp4_ws_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                             const uint8_t* sa, int64_t ldsa, const uint8_t* b, int64_t ldb,
                             const uint8_t* sb, int64_t ldsb, void* c, int64_t ldc, int c_f32,
                             int accumulate, void* ws, hipStream_t st);
// swiglu: the gate/up layout (rows = 2 I), else the down layout
hipError_t launch_pack_mxfp4(const uint8_t* w, const uint8_t* scale, uint8_t* packed, int64_t batch,
                             int rows, int cols, bool swiglu, hipStream_t st);
hipError_t launch_ffn_up_mxfp4(const Dims& d, const uint8_t* xq, const uint8_t* xs, int64_t ldxs,
                               const int32_t* gather, const int32_t* offsets, const uint8_t* w,
                               uint8_t* hq, uint8_t* hs, int64_t ldhs, hipStream_t st);
hipError_t launch_ffn_down_mxfp4(const Dims& d, const uint8_t* hq, const uint8_t* hs, int64_t ldhs,
                                 const int32_t* offsets, const uint8_t* w, void* y,
                                 hipStream_t st);

// a share of the experts: sorting n = T*K pairs, and rows to the experts and back (dispatch.hip);
// w == nullptr: weights 1; dw == nullptr: no dots (then partner is not read)
size_t sort_ws_bytes(int64_t n, int count);
hipError_t launch_sort_by_expert(int64_t n, int K, const int32_t* idx, int first, int count,
                                 int32_t* offsets, int32_t* token, int32_t* row, void* ws,
                                 hipStream_t st);
hipError_t launch_spread(int dtype, int64_t T, int K, int64_t H, const void* tok, int64_t ld_tok,
                         const int32_t* row, const float* w, const void* partner,
                         int64_t ld_partner, void* out, int64_t ld_out, float* dw, hipStream_t st);
hipError_t launch_gather(int dtype, int64_t T, int K, int64_t H, const void* rows, int64_t ld_rows,
                         const int32_t* row, const float* w, const void* partner,
                         int64_t ld_partner, void* out, int64_t ld_out, float* dw, hipStream_t st);

}  // namespace moe
