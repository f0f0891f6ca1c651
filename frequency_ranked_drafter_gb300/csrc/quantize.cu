// vt_quantize_rows — rows of an lm_head (gathered through trimmed_to_full)
// or hidden states as 8-bit integers with one scale a row.
//
//   s    = max(max_j |x_j| * (1/127), 2^-126)      (fp32, 1/127 rounded too)
//   q_j  = the integer nearest to x_j / s, ties to even, in [-127, 127]
//
// The quotient is not rounded before it is rounded to an integer: r = rint(
// x * (1 / s)) is off by at most one and only next to a half, and
// e = x - r * s, one fused multiply-add, is exact there (both terms are
// multiples of half the last place of s and |e| < s), so comparing |e| with
// s / 2 settles the integer.  (s / 2 has to be an fp32 number for that: a row whose
// scale is below 2^-125 is multiplied by 2^24 first.)  Every build and every order
// of work gives the same bytes.
//
// Bound by HBM: R * d * (size + 1) bytes, each value read once.  A row is
// held in registers between the maximum and the rounding (16 chunks of 16
// bytes a lane), by as few warps as hold it (1, 2 or 8), or by eight where
// there are too few rows to fill the SMs with warps.  The rounding was what
// bounded it at first: with the exact test behind one branch for a chunk and
// the maximum taken on packed bits, 32768 gathered rows of 4096 bf16 went from
// 98.7 to 66.2 us (6.1 TB/s of reads and writes, 0.90 of the measured copy; rows in
// order 64.2, fp16 62.8, fp32 100.9 us, two warps a row).
#include <cuda_fp16.h>

#include "ranges.cuh"
#include "vt_checks.cuh"
#include "vt_common.cuh"

namespace vt {
namespace {

constexpr int kQThreads = 256;
constexpr int kQChunks = 16;  // 16-byte chunks of a row a lane holds

struct QuantArgs {
  const char* X;
  int64_t V, ldx;  // rows of X, row stride in elements
  int d, R;
  const int32_t* ids;
  int8_t* Q;
  float* scale;
  unsigned long long* n_invalid;
};

// The values of one 16-byte chunk as fp32 (exact).
template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[DT == VT_FP32 ? 4 : 8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == VT_FP32) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (DT == VT_BF16) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// A chunk of tiny values, times 2^24 (exact in either type).
template <int DT>
__device__ __forceinline__ uint4 times_2_24(const uint4& v) {
  auto up = [](uint32_t w) {
    if constexpr (DT == VT_FP32) return __float_as_uint(__uint_as_float(w) * 0x1p24f);
    return (__float_as_uint(bf16hi(w) * 0x1p24f) & 0xffff0000u) |
           __float_as_uint(bf16lo(w) * 0x1p24f) >> 16;
  };
  return make_uint4(up(v.x), up(v.y), up(v.z), up(v.w));
}

// Nearest integers to x / s in the low bytes (two's complement); inv = 1 / s,
// half = s / 2.  Only where some remainder reaches half a step (rarely) is any
// integer looked at again.
template <int N>
__device__ __forceinline__ void to_int8(const float (&x)[N], float s, float inv, float half,
                                        uint32_t (&q)[N]) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = fmaf(x[i], inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(-(t - kMagic), s, x[i])));
    q[i] = __float_as_uint(t);
  }
  if (far >= half) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = fmaf(-(__uint_as_float(q[i]) - kMagic), s, x[i]);
      if (fabsf(e) > half || (fabsf(e) == half && (q[i] & 1))) q[i] += e > 0.f ? 1u : ~0u;
    }
  }
}

// The larger of `m` and the chunk's largest |x|, as the bits of the type (an
// order that puts infinities and NaN on top); 16-bit types two at a time.
template <int DT>
__device__ __forceinline__ uint32_t max_bits(const uint4& v, uint32_t m) {
  if constexpr (DT == VT_FP32) {
    m = max(max(m, v.x & 0x7fffffffu), v.y & 0x7fffffffu);
    return max(max(m, v.z & 0x7fffffffu), v.w & 0x7fffffffu);
  } else {
    m = __vmaxu2(__vmaxu2(m, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
    return __vmaxu2(__vmaxu2(m, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
  }
}
// ... as the bits of the fp32 value.
template <int DT>
__device__ __forceinline__ uint32_t max_fp32(uint32_t m) {
  if constexpr (DT == VT_FP32) return m;
  m = max(m & 0xffffu, m >> 16);
  if constexpr (DT == VT_BF16) return m << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// kRowWarps warps a row; kQChunks chunks a lane cover the row.
template <int DT, int kRowWarps>
__global__ void __launch_bounds__(kQThreads, 2) quantize_rows_kernel(QuantArgs a) {
  constexpr int kVals = DT == VT_FP32 ? 4 : 8;
  constexpr int kSize = DT == VT_FP32 ? 4 : 2;
  constexpr int kWarps = kQThreads / 32;
  constexpr int kStep = 32 * kRowWarps;
  __shared__ uint32_t wmax[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / kRowWarps, part = warp % kRowWarps;
  constexpr int rows_per_cta = kWarps / kRowWarps;
  // the warps of a row meet at a barrier of their own
  auto meet = [&]() {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kRowWarps) : "memory");
  };
  const int nchunks = a.d / kVals;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x * rows_per_cta + group; row < a.R;
       row += gridDim.x * rows_per_cta) {
    const int64_t src = a.ids ? (int64_t)__ldg(a.ids + row) : row;
    int8_t* out = a.Q + row * a.d;
    const bool known = src >= 0 && src < a.V;
    const uint4* x4 = reinterpret_cast<const uint4*>(a.X + (known ? src : 0) * a.ldx * kSize);
    uint4 v[kQChunks];
    uint32_t mx = 0;  // largest |x| as bits: an order that puts inf and NaN on top
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) {
      const int c = lane + 32 * part + kStep * j;
      v[j] = known && c < nchunks ? ld_stream_u4(x4 + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) mx = max_bits<DT>(v[j], mx);
    mx = __reduce_max_sync(~0u, max_fp32<DT>(mx));
    if constexpr (kRowWarps > 1) {
      meet();  // the previous row's maxima have been read
      if (lane == 0) wmax[warp] = mx;
      meet();
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) mx = max(mx, wmax[group * kRowWarps + w]);
    }
    // a row with an infinity or a NaN: integers 0 and scale NaN, so that a
    // product with it is NaN
    const bool finite = mx < 0x7f800000u;
    const float s = fmaxf((finite ? __uint_as_float(mx) : 0.f) * (1.f / 127.f), 0x1p-126f);
    float step = s;
    if (DT != VT_FP16 && s < 0x1p-125f) {
      step = s * 0x1p24f;
#pragma unroll
      for (int j = 0; j < kQChunks; ++j) v[j] = times_2_24<DT>(v[j]);
    }
    const float inv = __fdiv_rn(1.f, step), half = 0.5f * step;
#pragma unroll
    for (int j = 0; j < kQChunks; ++j) {
      const int c = lane + 32 * part + kStep * j;
      if (c >= nchunks) break;
      float x[kVals];
      unpack<DT>(v[j], x);
      uint32_t q[kVals];
      to_int8<kVals>(x, step, inv, half, q);
      if (!finite) {
#pragma unroll
        for (int i = 0; i < kVals; ++i) q[i] = 0u;
      }
      if (VT_CHECKED((c + 1) * kVals <= a.d)) {
        if constexpr (kVals == 8)
          reinterpret_cast<uint2*>(out)[c] =
              make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
        else
          reinterpret_cast<uint32_t*>(out)[c] = pack4(q[0], q[1], q[2], q[3]);
      }
    }
    if (lane == 0 && part == 0) {
      a.scale[row] = !known ? 0.f : finite ? s : __int_as_float(0x7fffffff);
      if (!known && a.n_invalid) atomicAdd(a.n_invalid, 1ull);
    }
  }
}

template <int DT>
vt_status launch(const QuantArgs& a, const DeviceInfo& di, cudaStream_t s) {
  constexpr int kVals = DT == VT_FP32 ? 4 : 8;
  // Eight warps a row while all rows, or nearly, run at once that way (bf16,
  // d = 4096: 1 row 1.55 us against 2.50 with one warp, 450 rows 3.08 and 4.14,
  // 900 rows 5.14 and 4.81; d = 1024: 300 rows 2.01 and 2.16, 450 rows 2.74 and
  // 2.34); else as few as hold a row (32768 rows of 4096: 66 us with one, 179
  // with eight).
  constexpr int kHold = 32 * kQChunks * kVals;  // values a warp holds
  const bool few = a.R <= (a.d < kHold ? 2 : 3) * di.num_sms;
  const int row_warps = few || a.d > 2 * kHold ? 8 : a.d > kHold ? 2 : 1;
  const int per_cta = kQThreads / 32 / row_warps;
  const int grid = (int)std::min<int64_t>(((int64_t)a.R + per_cta - 1) / per_cta,
                                          (int64_t)di.num_sms * 8);
  auto kernel = row_warps == 1   ? quantize_rows_kernel<DT, 1>
                : row_warps == 2 ? quantize_rows_kernel<DT, 2>
                                 : quantize_rows_kernel<DT, 8>;
  const cudaError_t e = launch_dependent(kernel, dim3(grid), dim3(kQThreads), 0, s, a);
  if (e != cudaSuccess)
    return fail(VT_ERR_CUDA, std::string("quantize_rows_kernel: ") + cudaGetErrorString(e));
  return launch_status("quantize_rows_kernel");
}

}  // namespace
}  // namespace vt

extern "C" vt_status vt_quantize_rows(const void* X, int32_t dtype, int64_t V, int32_t d,
                                      int64_t ldx, const int32_t* ids, int32_t R, int8_t* Q,
                                      float* scale, uint64_t* n_invalid, void* stream) {
  using namespace vt;
  if (dtype != VT_BF16 && dtype != VT_FP16 && dtype != VT_FP32)
    return fail(VT_ERR_INVALID_ARG, "vt_quantize_rows: unknown dtype");
  const int size = dtype == VT_FP32 ? 4 : 2;
  if (R < 0 || V < 0 || d < 16 || d > 16384 || d % 16 != 0)
    return fail(VT_ERR_INVALID_ARG,
                "vt_quantize_rows: need R >= 0, V >= 0, 16 <= d <= 16384, d % 16 == 0");
  if (!ids && R != 0 && V != R)
    return fail(VT_ERR_INVALID_ARG, "vt_quantize_rows: without ids, R must be V");
  if (R == 0) return VT_OK;
  if (!Q || !scale || (!X && V > 0))
    return fail(VT_ERR_INVALID_ARG, "vt_quantize_rows: null pointer");
  if ((V > 1 && ldx < d) || ldx * size % 16 != 0)
    return fail(VT_ERR_INVALID_ARG,
                "vt_quantize_rows: row stride below d or not a multiple of 16 bytes");
  if (!aligned(X, 16) || !aligned(Q, 16) || !aligned(scale, 4) || !aligned(ids, 4) ||
      !aligned(n_invalid, 8))
    return fail(VT_ERR_INVALID_ARG,
                "vt_quantize_rows: X, Q not 16B, scale, ids not 4B or n_invalid not 8B aligned");
  if (outputs_overlap({{Q, (int64_t)R * d}, {scale, 4ll * R}, {n_invalid, 8}},
                      {rows_range(X, V, ldx, d, size), {ids, 4ll * R}}))
    return fail(VT_ERR_INVALID_ARG, "vt_quantize_rows: an output overlaps X, ids or another");
  DeviceInfo di;
  if (!current_device(&di)) return VT_ERR_CUDA;
  const QuantArgs a = {static_cast<const char*>(X), V, ldx, d, R, ids, Q, scale,
                       reinterpret_cast<unsigned long long*>(n_invalid)};
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == VT_BF16   ? launch<VT_BF16>(a, di, s)
         : dtype == VT_FP16 ? launch<VT_FP16>(a, di, s)
                            : launch<VT_FP32>(a, di, s);
}
