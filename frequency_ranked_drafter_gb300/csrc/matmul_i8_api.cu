// vt_matmul_i8: argument checks and the choice of kernel.
#include "matmul_i8.cuh"
#include "ranges.cuh"

extern "C" size_t vt_matmul_i8_workspace_size(void) { return 256; }

namespace vt {
namespace {

// budget: the tensor-core kernel with waits that give up after so many clocks (0:
// any kernel, its own limit).
vt_status product(const int8_t* X, const float* x_scale, int32_t M, const int8_t* W,
                  const float* w_scale, int32_t N, int32_t d, const float* bias, void* out,
                  int32_t out_dtype, int64_t ldo, void* ws, size_t ws_bytes, int64_t budget,
                  void* stream) {
  if (out_dtype != VT_FP32 && out_dtype != VT_BF16)
    return fail(VT_ERR_INVALID_ARG, "vt_matmul_i8: outputs are fp32 or bf16");
  if (M < 0 || N < 0 || M > 65535 || d < 16 || d > 16384 || d % 16 != 0)
    return fail(VT_ERR_INVALID_ARG,
                "vt_matmul_i8: need 0 <= M <= 65535, N >= 0, 16 <= d <= 16384, d % 16 == 0");
  if (N > 1 << 30) return fail(VT_ERR_UNSUPPORTED, "vt_matmul_i8: N > 2^30");
  if (M == 0 || N == 0) return VT_OK;
  if (!X || !x_scale || !W || !w_scale || !out)
    return fail(VT_ERR_INVALID_ARG, "vt_matmul_i8: null pointer");
  if (M > 1 && ldo < N) return fail(VT_ERR_INVALID_ARG, "vt_matmul_i8: ldo < N");
  const int size = out_dtype == VT_FP32 ? 4 : 2;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(bias, 4) || !aligned(out, size))
    return fail(VT_ERR_INVALID_ARG, "vt_matmul_i8: misaligned pointer (X, W 16 bytes)");
  if (outputs_overlap({rows_range(out, M, ldo, N, size)},
                      {{X, (int64_t)M * d}, {W, (int64_t)N * d}, {x_scale, 4ll * M},
                       {w_scale, 4ll * N}, {bias, 4ll * N}}))
    return fail(VT_ERR_INVALID_ARG, "vt_matmul_i8: out overlaps an input");
  if (!ws || ws_bytes < vt_matmul_i8_workspace_size() || !aligned(ws, 256))
    return fail(VT_ERR_WORKSPACE, "vt_matmul_i8: workspace missing, too small or misaligned");
  DeviceInfo di;
  if (!current_device(&di)) return VT_ERR_CUDA;
  const I8Args a = {X,   x_scale, W, w_scale, bias, out, M == 1 ? (int64_t)N : ldo,
                    M,   N,       d, out_dtype == VT_BF16};
  const bool gemv = M <= 4, mma = !gemv && matmul_i8_mma_fits(M, N, d, di);
  if (budget && (gemv || mma))
    return fail(VT_ERR_UNSUPPORTED,
                "vt_selftest_matmul_i8: these sizes take a kernel without waits");
  // One to four rows of X: dp4a (M = 4: 22.8 us against 32.4 of mma.sync and
  // 35.9 of tcgen05 at N = 32768, d = 4096).
  if (gemv) return matmul_i8_gemv(a, di, (cudaStream_t)stream);
  if (mma) return matmul_i8_mma(a, di, (cudaStream_t)stream);
  return matmul_i8_tc(a, reinterpret_cast<unsigned*>(static_cast<char*>(ws) + 128), budget, di,
                      (cudaStream_t)stream);
}

}  // namespace
}  // namespace vt

extern "C" vt_status vt_matmul_i8(const int8_t* X, const float* x_scale, int32_t M,
                                  const int8_t* W, const float* w_scale, int32_t N, int32_t d,
                                  const float* bias, void* out, int32_t out_dtype, int64_t ldo,
                                  void* ws, size_t ws_bytes, void* stream) {
  return vt::product(X, x_scale, M, W, w_scale, N, d, bias, out, out_dtype, ldo, ws, ws_bytes, 0,
                     stream);
}

extern "C" vt_status vt_selftest_matmul_i8(const int8_t* X, const float* x_scale, int32_t M,
                                           const int8_t* W, const float* w_scale, int32_t N,
                                           int32_t d, const float* bias, void* out,
                                           int32_t out_dtype, int64_t ldo, void* ws,
                                           size_t ws_bytes, int64_t budget_cycles, void* stream) {
  if (budget_cycles < 1 || budget_cycles > (int64_t(1) << 31))
    return vt::fail(VT_ERR_INVALID_ARG,
                    "vt_selftest_matmul_i8: budget must be 1 .. 2^31 cycles");
  return vt::product(X, x_scale, M, W, w_scale, N, d, bias, out, out_dtype, ldo, ws, ws_bytes,
                     budget_cycles, stream);
}
