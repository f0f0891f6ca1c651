// Arguments of the int8 product, and what its kernels share.
#pragma once

#include <cuda_bf16.h>

#include "vt_checks.cuh"
#include "vt_common.cuh"

namespace vt {

struct I8Args {
  const int8_t* X;   // [M][d]
  const float* xs;   // [M]
  const int8_t* W;   // [N][d]
  const float* ws;   // [N]
  const float* bias; // [N] or null
  void* out;         // [M][ldo], fp32 or bf16
  int64_t ldo;
  int M, N, d;
  int out_bf16;
};

// One output, at i = m * ldo + n: the exact integer sum, rounded to fp32 once, then one rounding
// each for the scales' product, the product with it and the bias; bf16 outputs
// round once more.
__device__ __forceinline__ void i8_store(const I8Args& a, int64_t i, int acc, float xs, float ws,
                                         float b) {
  float y = __fmul_rn(__int2float_rn(acc), __fmul_rn(xs, ws));
  if (a.bias) y = __fadd_rn(y, b);
  if (!VT_CHECKED(i >= 0 && i < (a.M - 1) * a.ldo + a.N && i % a.ldo < a.N)) return;
  if (a.out_bf16)
    static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(y);
  else
    static_cast<float*>(a.out)[i] = y;
}

// Four bytes of W as the fp16 numbers (w + 128) * 2^-24, in the order 0, 2, 1, 3.
__device__ __forceinline__ void w_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = (w & 0x00ff00ffu) ^ 0x00800080u;
  hi = ((w >> 8) & 0x00ff00ffu) ^ 0x00800080u;
}
// Four bytes of X as fp16 in the same order: x + 128 in the low mantissa bits
// of 1024 (0x6400), then 1152 is taken away.
__device__ __forceinline__ void x_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = v ^ 0x80808080u;
  const uint32_t a = __byte_perm(x, 0x64646464u, 0x4240);
  const uint32_t b = __byte_perm(x, 0x64646464u, 0x4341);
  asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

vt_status matmul_i8_gemv(const I8Args& a, const DeviceInfo& di, cudaStream_t s);
// Whether the warp-level kernel is to be taken: up to 16 rows of X that fit
// shared memory as fp16, and few enough rows of W.
bool matmul_i8_mma_fits(int M, int N, int d, const DeviceInfo& di);
vt_status matmul_i8_mma(const I8Args& a, const DeviceInfo& di, cudaStream_t s);
// budget: clocks after which a wait gives up (0: its own limit, about a second).
vt_status matmul_i8_tc(const I8Args& a, unsigned* err, long long budget, const DeviceInfo& di,
                       cudaStream_t s);

}  // namespace vt
