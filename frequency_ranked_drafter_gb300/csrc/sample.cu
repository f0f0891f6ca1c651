// vt_sample_logits — temperature, top-k, top-p and min-p over rows of logits,
// the draw from what is left with the caller's uniform, and (optionally) the
// filtered distribution that the acceptance test of verification reads.
//
//   z_i = (x_i - max x) / T,  w_i = exp(z_i); in descending order of x (equal
//   logits by lower index) keep the first top_k; of those the shortest prefix
//   whose mass reaches top_p of theirs; of those the ones with w_i >= min_p.
//   p_i = w_i / S, S = sum of kept w;  draw: the first index i, in the order
//   of the logits, with (sum of kept w_j, j <= i) > u * S.
//
// What is kept is always a prefix of the sorted order, so it is described by
// a logit and a count: every logit above `thr`, and the first `ties` (by
// index) of those equal to it.  The row is never sorted.
//
// One cluster of up to 16 CTAs per row.  The row is read once, into the
// CTAs' shared memory as fp32, a contiguous slice each and a contiguous
// segment of that for each warp; everything after works on chip:
//   * the filters: a histogram of counts over linear bins of max - x names
//     the bin that holds the border (of the k-th logit, or of the mass, whose
//     sums over bins are bounded from counts and the bins' edges);
//   * where at most 256 logits reach that bin they are gathered into the
//     first CTA, which ranks them by counting and settles everything;
//   * otherwise histograms over ever narrower ranges of the logits' ordered
//     bit patterns find the border's value; the masses that decide are exact.
//     For top-p each warp first packs the logits that may be kept (few of a
//     language model's, placed by a sample of the row) into a short list in
//     the order of the row, and all further passes go over those;
//   * the draw: segment sums, a scan over warps and CTAs, and one warp walks
//     its segment.
// Weights are fixed point, 2^42 for the largest (`Weight`), summed as
// integers, so sums are exact, independent of the order and of how the row is
// split; a weight is within 2^-28 of its value (fp32 exponentials would be
// 2^-22 off, enough to draw another token about once in a thousand rows of a
// flat vocabulary).
//
// What bounds it: one row, the chain of barriers over the cluster and of passes
// between them (32768 fp32 logits, top-k and top-p: 7.6 us; 128256 bf16 logits:
// top-k 8.6 us, top-p 21 us); many rows, the instructions of the weights, some
// 25 a logit and pass, and the search for top-p's border (60 rows of 128256 bf16
// logits: no filter 27 us, its distribution too 41, top-k 20, top-p 59; reading
// and writing alone would take 2.3 and 6.8 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "cluster.cuh"
#include "ranges.cuh"
#include "vt_checks.cuh"
#include "vt_common.cuh"

namespace vt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBins = 1024;
constexpr int kPer = kBins / kThreads;  // bins a thread scans
constexpr int kList = 256;        // logits the first CTA ranks (one a thread)
constexpr int kMaxN = 1 << 19;    // 2^19 weights of 2^42 stay below 2^62
constexpr uint32_t kKeyNegInf = 0x007fffffu;
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int n, seg;  // seg: elements of a warp's segment, a multiple of 128
  int cap;     // packed ones that a warp's list holds, a multiple of 128
  const float* u;
  const int32_t* t2f;
  float T, top_p, min_p;
  int top_k;
  const float *T_row, *top_p_row, *min_p_row;
  const int32_t* top_k_row;
  int32_t* ids;
  float* probs;
  float* dist;
  int64_t ld_dist;
};

// Orders floats as unsigned integers (no -0 among them: loads add +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
// Logits that come from 16-bit types differ in their high key bits only: keys
// are shortened by `drop` bits (zeros in positive logits, ones in negative).
__device__ __forceinline__ uint32_t short_key(float x, int drop) { return key_of(x) >> drop; }
__device__ __forceinline__ float of_short(uint32_t k, int drop) {
  const uint32_t f = k << drop;
  return of_key(f & 0x80000000u ? f : f | ((1u << drop) - 1u));
}

// 2^(j/32), the fp32 nearest to it and the rest.
__device__ const float2 kTable[32] = {
    {1.0f, 0.000000000e+00f}, {1.0218971967697144f, -4.811559768e-08f},
    {1.0442737340927124f, 4.833470144e-08f}, {1.0671404600143433f, -5.933751964e-08f},
    {1.0905077457427979f, -1.307754019e-08f}, {1.114386796951294f, -5.435540141e-08f},
    {1.1387885808944702f, 5.386222144e-08f}, {1.1637248992919922f, -4.051441467e-08f},
    {1.1892070770263672f, 3.797635388e-08f}, {1.215247392654419f, -3.267395007e-08f},
    {1.2418577671051025f, 4.496838151e-08f}, {1.2690509557724f, 1.419333320e-09f},
    {1.2968395948410034f, -4.018999375e-08f}, {1.3252366781234741f, -3.496373283e-08f},
    {1.3542555570602417f, -1.012334897e-08f}, {1.3839099407196045f, -5.875577254e-08f},
    {1.4142135381698608f, 2.420323421e-08f}, {1.4451807737350464f, 3.324200023e-08f},
    {1.4768261909484863f, -4.500898702e-08f}, {1.5091644525527954f, -2.495937267e-08f},
    {1.5422108173370361f, 8.070904691e-09f}, {1.5759809017181396f, -5.661025316e-08f},
    {1.610490322113037f, 9.836217199e-09f}, {1.6457555294036865f, -5.124972168e-08f},
    {1.6817928552627563f, -2.475532726e-08f}, {1.7186193466186523f, -4.849617443e-08f},
    {1.7562521696090698f, -9.235770341e-09f}, {1.7947090864181519f, -1.141504467e-08f},
    {1.8340080976486206f, -1.123927814e-08f}, {1.8741676807403564f, -4.663005654e-08f},
    {1.9152065515518188f, 9.845328446e-09f}, {1.9571441411972046f, -1.702180432e-08f}};

// Two floats in one register pair, one instruction for both: weights are what
// the passes over a row spend their instructions on (60 rows of 128256, own
// settings and distributions: 67.6 us with single ones, 62.6).
struct F2 {
  unsigned long long v;
  F2() = default;
  __device__ __forceinline__ F2(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

// Weights exp((x - max) / T).  y = 32 * log2(e) * (x - max) / T is split into
// an integer, whose low five bits choose 2^(j/32) from a table and whose rest
// is the exponent, and a remainder r, |r| <= 1, from which 2^(r/32) - 1 is a
// polynomial of degree 4 (Taylor; its error is below 2^-34).  r is taken with
// two fused steps from two-part constants, so its error is that of one fp32
// rounding near 1, 2^-25 of a 32nd of an octave.  A weight is the sum of two
// floats, (a + b) * s with s the power of two.
struct Weight {
  float shift, c_hi, c_lo, b_hi, b_lo, bm;
  float cut, cut_real;  // logits at or below: fixed-point weight 0, weight 0
  float top;            // the maximum
  bool top_only;        // T = 0, or the maximum is +inf: weight 1 there alone

  // Constants for a row; every step is exact or carried in two floats.
  __device__ __forceinline__ void init(float max, float T) {
    top = max;
    top_only = T == 0.f || max == INFINITY;
    T = fmaxf(T, 1e-30f);
    constexpr float kC = 46.16624130844683f;           // 32 log2(e), and
    constexpr float kCrest = (float)(46.166241308446828 - (double)46.16624130844683f);
    c_hi = __fdiv_rn(kC, T);
    c_lo = __fdiv_rn(fmaf(-c_hi, T, kC) + kCrest, T);
    const float p = max * c_hi;
    // far from 0 in units of the table, distances to the maximum are exact in
    // fp32 wherever there is a weight, and products with the logits are not
    const bool far = !(fabsf(p) <= 1048576.f) && !top_only;
    shift = far ? max : 0.f;
    const float rest = far ? 0.f : fmaf(max, c_hi, -p) + max * c_lo;
    const float b = far ? 0.f : -p;
    // b_hi has few enough digits that b_hi - k is exact for every integer k
    // down to fp32's smallest exponent
    const float m = 1.5f * __int_as_float(
        (int)((__float_as_uint(fabsf(b) + 8192.f) & 0x7f800000u) + (1u << 23)));
    b_hi = (b + m) - m;
    b_lo = (b - b_hi) - rest;
    bm = kMagic + b_hi;
    // 2^-43, 2^-126; never the maximum itself, however small T is
    const float below = nextafterf(max, -INFINITY);
    cut = fminf(max - T * 29.8f, below);
    cut_real = fminf(max - T * 87.3f, below);
  }

  static constexpr float a1 = 0.021660849392498290f, a2 = 2.3459619820e-4f,
                         a3 = 1.6938509724e-6f, a4 = 9.1725627e-9f;  // (ln 2 / 32)^i / i!

  // For a logit above cut_real; th, tl: table entry of the lane's n & 31.
  __device__ __forceinline__ float scaled(float x, int& n) const {
    const float xs = x - shift;
    const float nf = fmaf(xs, c_hi, bm);
    const float kf = nf - kMagic;
    float r = fmaf(xs, c_hi, b_hi - kf);
    r += fmaf(xs, c_lo, b_lo);
    n = __float_as_int(nf);
    return r * fmaf(r, fmaf(r, fmaf(r, a4, a3), a2), a1);
  }
  // 2^(n >> 5) for the integer in n's low bits
  static __device__ __forceinline__ float power(int n) {
    return __int_as_float((int)(((uint32_t)n << 18) & 0xff800000u) + 0x3f800000);
  }
  // Fixed point in two parts: hi * 2^22 + lo = weight * 2^42.
  static constexpr uint32_t kHi0 = 0x41400000u;  // 12, whose last place is 2^-20
  static constexpr uint32_t kLo0 = 0x36400000u;  // 1.5 * 2^-19, last place 2^-42
  static __device__ __forceinline__ void split(float a, float b, float s, uint32_t& hi,
                                               uint32_t& lo) {
    const float as = a * s;
    const float t1 = fmaf(b, s, as) + 12.f;
    const float rest = fmaf(b, s, as - (t1 - 12.f));
    hi = __float_as_uint(t1);
    lo = __float_as_uint(rest + __uint_as_float(kLo0));
  }
  // One logit alone (any lane), from the table in memory.
  __device__ __forceinline__ long long fixed(float x, const float2* table) const {
    if (top_only) return x == top ? 1ll << 42 : 0ll;
    if (!(x > cut)) return 0;
    int n;
    const float q = scaled(x, n);
    const float2 t = table[n & 31];
    uint32_t hi, lo;
    split(t.x, fmaf(t.x, q, t.y), power(n), hi, lo);
    return ((long long)(hi - kHi0) << 22) + (int)(lo - kLo0);
  }
  // The weight as fp32, with all its digits however small it is.
  __device__ __forceinline__ float real(float x, const float2* table) const {
    if (top_only) return x == top ? 1.f : 0.f;
    if (!(x > cut_real)) return 0.f;
    int n;
    const float q = scaled(x, n);
    const float2 t = table[n & 31];
    return (t.x + fmaf(t.x, q, t.y)) * power(n);
  }
};

// Sums of weights over a lane's logits, as raw bits of the two parts.
struct Sum {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ long long value(int count) const {
    return ((long long)(uint32_t)(hi - (uint32_t)count * Weight::kHi0) << 22) +
           (int)(lo - (uint32_t)count * Weight::kLo0);
  }
};

struct Shared {
  uint32_t hist[kBins];    // this CTA's counts
  uint32_t total[kBins];   // the cluster's
  long long sums[2][3][kMaxCluster];  // per-CTA sums of a round
  __align__(16) uint32_t warp_max[kMaxCluster * kWarps];  // keys, of the whole cluster
  float cta_sum[kMaxCluster];
  uint32_t cta_cnt[kMaxCluster];
  long long fin_sum[kMaxCluster];
  uint32_t fin_ties[kMaxCluster];
  long long warp_a[kWarps], warp_b[kWarps], warp_c[kWarps];
  uint32_t warp_u[kWarps];
  float warp_f[kWarps], warp_g[kWarps];
  float2 table[32];
  double min_off;  // T ln(min_p)
  int sel_bin[2];
  long long sel_before[2];
  uint32_t sel_cnt, edge[2], kth;
  unsigned found;                    // logits this CTA has put in its list
  uint32_t list_cnt[kMaxCluster];    // and every other one

  // A CTA's own list lies in its histogram, the first CTA's joined list where
  // the cluster's counts were: nobody counts while there are lists.
  __device__ __forceinline__ uint64_t* own_list() {  // key, then lower index first
    return reinterpret_cast<uint64_t*>(hist);
  }
  __device__ __forceinline__ uint64_t* list_key() { return reinterpret_cast<uint64_t*>(total); }
  __device__ __forceinline__ long long* list_w() {
    return reinterpret_cast<long long*>(total + 2 * kList);
  }
};
static_assert(4 * kList <= kBins && kList <= kThreads, "the lists fit the histograms");
static_assert(kMaxCluster * kWarps <= kThreads, "one thread a warp's maximum");

struct Row {  // what every CTA of the row agrees on
  float max, thr;  // kept: logits above thr, and the first `ties` equal to it
  uint32_t ties;
  float summed;    // logits above it are in this warp's `above` already
  long long above;
};

// floor (or ceil) of z * f, f in [0, 1], exactly.
__device__ __forceinline__ long long mul_frac(long long z, float f, bool up) {
  if (f >= 1.f) return z;
  if (!(f > 0.f)) return 0;
  const uint32_t b = __float_as_uint(f);
  const int ex = ::max((int)(b >> 23), 1);
  const uint64_t m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
  const int s = 150 - ex;  // f = m * 2^-s, s >= 24
  const uint64_t lo = (uint64_t)z * m, hi = __umul64hi((uint64_t)z, m);
  if (s >= 88) return up ? 1 : 0;  // z * m < 2^87
  uint64_t r, rest;
  if (s >= 64) {
    r = s == 64 ? hi : hi >> (s - 64);
    rest = lo | (s == 64 ? 0 : hi << (128 - s));
  } else {
    r = (hi << (64 - s)) | (lo >> s);
    rest = lo << (64 - s);
  }
  return (long long)(r + (up && rest ? 1u : 0u));
}

// ceil(a / b) for 0 < a <= b * 2^19.
__device__ __forceinline__ long long ceil_div(long long a, long long b) {
  long long q = (long long)__fdividef(__ll2float_rn(a), __ll2float_rn(b));  // within 1
  while (q > 0 && (q - 1) * b >= a) --q;
  while (q * b < a) ++q;
  return q;
}

// Inclusive scan of one value a thread over the CTA; `tmp` holds kWarps.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();  // tmp is free
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  T before = 0;
#pragma unroll
  for (int w = 0; w < kWarps - 1; ++w) before += w < warp ? tmp[w] : (T)0;
  return v + before;
}

// Sum over the CTA, in every thread.
__device__ __forceinline__ long long block_sum64(long long v, long long* tmp) {
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  long long t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += tmp[w];
  return t;
}

// Bin of a logit on the linear scale; kBins (not counted) from there on.
__device__ __forceinline__ uint32_t lin_bin(float x, float max, float scale) {
  return (uint32_t)(int)fminf((max - x) * scale, (float)kBins);
}

// Four logits from shared memory, where they lie in their own type.
template <int DT>
__device__ __forceinline__ float4 unpack4(const void* p, int i) {
  if constexpr (DT == VT_FP32) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    if constexpr (DT == VT_BF16) {
      return make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y));
    } else {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
      return make_float4(a.x, a.y, b.x, b.y);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int i, float x) {  // x is of the type
  if constexpr (DT == VT_FP32)
    static_cast<float*>(p)[i] = x;
  else if constexpr (DT == VT_BF16)
    static_cast<uint16_t*>(p)[i] = (uint16_t)(__float_as_uint(x) >> 16);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(x);
}
template <int DT>
__device__ __forceinline__ float load1(const void* p, int i) {
  if constexpr (DT == VT_FP32) return static_cast<const float*>(p)[i];
  if constexpr (DT == VT_BF16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return __half2float(static_cast<const __half*>(p)[i]);
}

template <int DT>
struct Ctx {
  static constexpr int drop = DT == VT_BF16 ? 16 : DT == VT_FP16 ? 13 : 0;
  Shared& s;
  const Weight& w;
  const void* xs;   // this warp's segment, or the logits packed from it
  float2 entry;     // this lane's table entry
  int seg;          // its length
  uint32_t rank, C;
  const uint16_t* pos = nullptr;  // places in the segment of packed logits
  int round = 0;  // histogram rounds so far

  template <typename F>
  __device__ __forceinline__ void each4(F f) const {
#pragma unroll 1
    for (int i = 4 * (threadIdx.x & 31); i < seg; i += 128)
      f(i, unpack4<DT>(xs, i));
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each4([&](int, const float4& x) {
      f(x.x);
      f(x.y);
      f(x.z);
      f(x.w);
    });
  }
  // Parts of the weight of each lane's logit (0 where !keep); the whole warp.
  __device__ __forceinline__ void add(float x, bool keep, uint32_t& hi, uint32_t& lo) const {
    int n;
    const float q = w.scaled(keep ? x : w.top, n);
    const float th = __shfl_sync(~0u, entry.x, n), tl = __shfl_sync(~0u, entry.y, n);
    Weight::split(th, fmaf(th, q, tl), keep ? Weight::power(n) : 0.f, hi, lo);
  }
  // For two logits of each lane: their table entries, the remainders'
  // exponentials minus one and the integers' floats (Weight::scaled, two
  // logits an instruction).  The whole warp.
  __device__ __forceinline__ void scaled2(float x0, float x1, F2& th, F2& tl, F2& q, int& n0,
                                          int& n1) const {
    const F2 xs = add2(F2(x0, x1), F2(-w.shift));
    const F2 nf = fma2(xs, F2(w.c_hi), F2(w.bm));
    const F2 k = fma2(nf, F2(-1.f), F2(kMagic));  // minus the integer
    F2 r = fma2(xs, F2(w.c_hi), add2(F2(w.b_hi), k));
    r = add2(r, fma2(xs, F2(w.c_lo), F2(w.b_lo)));
    q = mul2(r, fma2(r, fma2(r, fma2(r, F2(Weight::a4), F2(Weight::a3)), F2(Weight::a2)),
                     F2(Weight::a1)));
    float f0, f1;
    nf.get(f0, f1);
    n0 = __float_as_int(f0);
    n1 = __float_as_int(f1);
    th = F2(__shfl_sync(~0u, entry.x, n0), __shfl_sync(~0u, entry.x, n1));
    tl = F2(__shfl_sync(~0u, entry.y, n0), __shfl_sync(~0u, entry.y, n1));
  }
  // Adds the weights of four logits of each lane to `t` (0 where !keep), the
  // same numbers as `add` gives.
  __device__ __forceinline__ void add4(const float (&x)[4], const bool (&keep)[4], Sum& t) const {
    const F2 neg(-1.f), twelve(12.f);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      F2 th, tl, q;
      int n0, n1;
      scaled2(keep[e] ? x[e] : w.top, keep[e + 1] ? x[e + 1] : w.top, th, tl, q, n0, n1);
      const F2 s(keep[e] ? Weight::power(n0) : 0.f, keep[e + 1] ? Weight::power(n1) : 0.f);
      const F2 b = fma2(th, q, tl), as = mul2(th, s);
      const F2 t1 = add2(fma2(b, s, as), twelve);
      const F2 lo = add2(fma2(b, s, add2(as, fma2(t1, neg, twelve))),
                         F2(__uint_as_float(Weight::kLo0)));
      float h0, h1, l0, l1;
      t1.get(h0, h1);
      lo.get(l0, l1);
      t.hi += __float_as_uint(h0) + __float_as_uint(h1);
      t.lo += __float_as_uint(l0) + __float_as_uint(l1);
    }
  }
  // p = weight * inv of four logits of each lane (0 where !keep); the whole warp.
  __device__ __forceinline__ void real4(const float (&x)[4], const bool (&keep)[4], float inv,
                                        float (&p)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      if (w.top_only) {
        p[e] = keep[e] ? w.real(x[e], s.table) * inv : 0.f;
        p[e + 1] = keep[e + 1] ? w.real(x[e + 1], s.table) * inv : 0.f;
        continue;
      }
      const bool in0 = keep[e] && x[e] > w.cut_real, in1 = keep[e + 1] && x[e + 1] > w.cut_real;
      F2 th, tl, q;
      int n0, n1;
      scaled2(in0 ? x[e] : w.top, in1 ? x[e + 1] : w.top, th, tl, q, n0, n1);
      const F2 f = add2(th, fma2(th, q, tl));
      const F2 v = mul2(mul2(f, F2(Weight::power(n0), Weight::power(n1))), F2(inv));
      float v0, v1;
      v.get(v0, v1);
      p[e] = in0 ? v0 : 0.f;
      p[e + 1] = in1 ? v1 : 0.f;
    }
  }
  __device__ __forceinline__ int per_lane() const { return seg >> 5; }
  // Place in the warp's segment of the i-th logit passed over.
  __device__ __forceinline__ int place(int i) const { return pos ? (int)pos[i] : i; }

  // Adds a, b and c over the cluster.
  __device__ __forceinline__ void sum_over(long long& a, long long& b, long long& c) {
    const int p = round & 1;
    put_sums(a, b, c, p);
    cl::sync();
    get_sums(a, b, c, p);
    ++round;
  }
  __device__ __forceinline__ void put_sums(long long a, long long b, long long c, int p) {
    const int warp = threadIdx.x >> 5;
    a = warp_sum64(a);
    b = warp_sum64(b);
    c = warp_sum64(c);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      s.warp_a[warp] = a;
      s.warp_b[warp] = b;
      s.warp_c[warp] = c;
    }
    __syncthreads();
    if (threadIdx.x < 3 * C) {
      const uint32_t to = threadIdx.x / 3, which = threadIdx.x % 3;
      const long long* v = which == 0 ? s.warp_a : which == 1 ? s.warp_b : s.warp_c;
      long long t = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) t += v[i];
      cl::st_u64(cl::map(&s.sums[p][which][rank], to), (uint64_t)t);
    }
  }
  __device__ __forceinline__ void get_sums(long long& a, long long& b, long long& c, int p) {
    a = b = c = 0;
    for (uint32_t r = 0; r < C; ++r) {
      a += s.sums[p][0][r];
      b += s.sums[p][1][r];
      c += s.sums[p][2][r];
    }
  }

  // The cluster's counts come together in two steps, because a CTA reads other
  // CTAs' shared memory at some 13 bytes a clock: CTA r adds up the r-th part
  // of everyone's bins, then hands the sums to everyone.
  __device__ __forceinline__ int part() const {  // groups of four bins a CTA adds up
    return (kBins / 4 + (int)C - 1) / (int)C;
  }
  __device__ __forceinline__ uint32_t* begin_round() {
    __syncthreads();  // the last round's counts have been used
    reinterpret_cast<uint4*>(s.hist)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    if ((int)threadIdx.x < part() && (int)rank * part() + (int)threadIdx.x < kBins / 4)
      reinterpret_cast<uint4*>(s.total)[rank * part() + threadIdx.x] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    return s.hist;
  }
  // Ends a round: thread t gets the cluster's counts of bins kPer * t, ..; with
  // kSums, the threads' a, b, c are added over the cluster too.
  template <bool kSums>
  __device__ __forceinline__ uint4 end_round(long long& a, long long& b, long long& c) {
    const int p = round & 1;
    if (kSums) put_sums(a, b, c, p);
    cl::sync();
    const int n = part();  // n * C items, one or two a thread
    for (int i = threadIdx.x; i < n * (int)C; i += kThreads) {
      const int g = (int)rank * n + i % n;  // group of four bins, from CTA i / n
      if (g < kBins / 4) {
        const uint4 v = cl::ld_u32x4(cl::map(&s.hist[4 * g], i / n));
        if (v.x) atomicAdd(&s.total[4 * g], v.x);
        if (v.y) atomicAdd(&s.total[4 * g + 1], v.y);
        if (v.z) atomicAdd(&s.total[4 * g + 2], v.z);
        if (v.w) atomicAdd(&s.total[4 * g + 3], v.w);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * (int)C; i += kThreads) {
      const int g = (int)rank * n + i % n;  // to CTA i / n
      if (g < kBins / 4 && i / n != (int)rank)
        cl::st_u32x4(cl::map(&s.total[4 * g], i / n),
                     *reinterpret_cast<const uint4*>(&s.total[4 * g]));
    }
    cl::sync();
    if (kSums) get_sums(a, b, c, p);
    ++round;
    return *reinterpret_cast<const uint4*>(&s.total[kPer * threadIdx.x]);
  }
  __device__ __forceinline__ uint4 end_round() {
    long long z;
    return end_round<false>(z, z, z);
  }
};

// Smallest short key in [-inf, max] whose linear bin is at most `bin` (bins
// never grow with the key, so a search by 32 finds it); one warp.
__device__ uint32_t first_key(uint32_t bin, float max, float scale, int drop) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = kKeyNegInf >> drop, hi = short_key(max, drop);
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 32 + 1;
    const uint32_t c = (uint32_t)::min((uint64_t)lo + (uint64_t)lane * step, (uint64_t)hi);
    const uint32_t ok = __ballot_sync(~0u, lin_bin(of_short(c, drop), max, scale) <= bin);
    if (!ok) {
      lo = __shfl_sync(~0u, c, 31) + 1;
      continue;
    }
    const int f = __ffs(ok) - 1;
    hi = __shfl_sync(~0u, c, f);
    lo = f > 0 ? __shfl_sync(~0u, c, f - 1) + 1 : hi;
  }
  return hi;
}

// Bits to drop from keys of a range so that it fits the bins.
__device__ __forceinline__ int range_shift(uint32_t width) {
  return ::max(0, 32 - __clz((int)width) - 10);
}

// The bin of the need-th of the counted logits, into s.sel_*: its number (-1:
// fewer are counted), how many come before it and how many it holds.
__device__ __forceinline__ void select_bin(Shared& s, const uint4& cnt, uint32_t need) {
  const uint32_t c[kPer] = {cnt.x, cnt.y, cnt.z, cnt.w};
  const uint32_t inc = block_scan<uint32_t>(cnt.x + cnt.y + cnt.z + cnt.w, s.warp_u);
  uint32_t run = inc - (cnt.x + cnt.y + cnt.z + cnt.w);
  if (threadIdx.x == kThreads - 1 && inc < need) {
    s.sel_bin[0] = -1;
    s.sel_before[0] = inc;
    s.sel_cnt = 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (run < need && run + c[i] >= need) {
      s.sel_bin[0] = kPer * threadIdx.x + i;
      s.sel_before[0] = run;
      s.sel_cnt = c[i];
    }
    run += c[i];
  }
  __syncthreads();
}

// The key that stands n-th (from 0) among the cluster's warps' maxima.
__device__ __forceinline__ uint32_t nth_max(Shared& s, int W, int n) {
  if ((int)threadIdx.x < W) {
    const uint32_t k = s.warp_max[threadIdx.x];
    int at = 0;
#pragma unroll 4
    for (int i = 0; i < W; i += 4) {  // W is a multiple of kWarps
      const uint4 o = *reinterpret_cast<const uint4*>(&s.warp_max[i]);
      at += o.x > k || (o.x == k && i < (int)threadIdx.x);
      at += o.y > k || (o.y == k && i + 1 < (int)threadIdx.x);
      at += o.z > k || (o.z == k && i + 2 < (int)threadIdx.x);
      at += o.w > k || (o.w == k && i + 3 < (int)threadIdx.x);
    }
    if (at == n) s.kth = k;
  }
  __syncthreads();
  return s.kth;
}

// Keeps the logits above the value of short key `k` and `ties` equal to it.
__device__ __forceinline__ void set_border(Row& row, uint32_t k, uint32_t ties, int drop) {
  const bool all = k < (kKeyNegInf >> drop);
  if (k == 0x7fffffffu >> drop) --k;  // -0, which no logit is: just below +0
  row.thr = all ? -INFINITY : of_short(k, drop);
  row.ties = all ? 0u : ties;
}

// The prefix of the k largest logits, from the linear histogram's selection
// (s.sel_*, for need = k) on.
template <int DT>
__device__ void find_count(Ctx<DT>& c, Row& row, uint32_t k, float scale) {
  Shared& s = c.s;
  constexpr int drop = Ctx<DT>::drop;
  const int bin = s.sel_bin[0];
  uint32_t need = k - (uint32_t)s.sel_before[0], in_bin = s.sel_cnt;
  if (threadIdx.x < 64) {
    const int v = threadIdx.x >> 5;
    uint32_t e;
    if (v == 0)
      e = bin < 0 ? kKeyNegInf >> drop : first_key(bin, row.max, scale, drop);
    else
      e = bin == 0 ? short_key(row.max, drop)
                   : first_key((bin < 0 ? kBins : bin) - 1, row.max, scale, drop) - 1;
    if ((threadIdx.x & 31) == 0) s.edge[v] = e;
  }
  __syncthreads();
  uint32_t lo = s.edge[0], hi = s.edge[1];
  __syncthreads();
  if (bin >= 0 && in_bin == need) {  // the whole bin is kept
    set_border(row, lo - 1, 0, drop);
    return;
  }
  while (true) {  // the range shrinks by 2^10 a round
    const int sh = range_shift(hi - lo);
    uint32_t* h = c.begin_round();
    c.each([&](float x) {
      const uint32_t at = hi - short_key(x, drop);
      if (at <= hi - lo) atomicAdd(&h[at >> sh], 1u);
    });
    select_bin(s, c.end_round(), need);
    const uint32_t b = (uint32_t)s.sel_bin[0];
    need -= (uint32_t)s.sel_before[0];
    in_bin = s.sel_cnt;
    __syncthreads();
    if (b >= (uint32_t)kBins) return;  // cannot be: the range holds the k-th logit
    const uint32_t top = hi - (b << sh);
    if (sh == 0) {
      set_border(row, top, need, drop);
      return;
    }
    const uint32_t width = (1u << sh) - 1;
    lo = top - lo > width ? top - width : lo;
    hi = top;
    if (in_bin == need) {
      set_border(row, lo - 1, 0, drop);
      return;
    }
  }
}

// Bins that hold the border of the mass, from counts over linear bins (step: z
// from one to the next, in octaves): the first whose upper bound reaches the
// target, and the first whose lower bound does (kBins: none).  Also how many
// logits lie in bins up to the second.
__device__ __forceinline__ void bound_mass(Shared& s, const uint4& cnt, float target, float step,
                                           int& b0, int& b1, uint32_t& upto) {
  const uint32_t c[kPer] = {cnt.x, cnt.y, cnt.z, cnt.w};
  const float ratio = exp2f(-step);
  float e = exp2f(-step * (float)(kPer * threadIdx.x));
  float up[kPer], dn[kPer], su = 0.f, sd = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    up[i] = su += (float)c[i] * e;
    e *= ratio;
    dn[i] = sd += (float)c[i] * e;
  }
  const float iu = block_scan<float>(su, s.warp_f), id = block_scan<float>(sd, s.warp_g);
  const uint32_t ic = block_scan<uint32_t>(c[0] + c[1] + c[2] + c[3], s.warp_u);
  if (threadIdx.x == 0) s.sel_bin[0] = s.sel_bin[1] = kBins;
  __syncthreads();
  // A thousandth covers the rounding of the fp32 sums and of the bins' edges.
  // A thread's first bin that reaches the target, or none: the same numbers say
  // both (id - sd + sd may round to less than id).
  b0 = b1 = kBins;
#pragma unroll
  for (int i = kPer - 1; i >= 0; --i) {
    if ((i == kPer - 1 ? iu : iu - su + up[i]) >= target * 0.999f)
      b0 = kPer * (int)threadIdx.x + i;
    if ((i == kPer - 1 ? id : id - sd + dn[i]) >= target * 1.001f)
      b1 = kPer * (int)threadIdx.x + i;
  }
  if (b0 < kBins) atomicMin(&s.sel_bin[0], b0);
  if (b1 < kBins) atomicMin(&s.sel_bin[1], b1);
  __syncthreads();
  b0 = s.sel_bin[0];
  b1 = s.sel_bin[1];
  if ((int)threadIdx.x == b1 / kPer) {
    uint32_t t = ic;
#pragma unroll
    for (int i = kPer - 1; i > 0; --i)
      if (i > b1 % kPer) t -= c[i];
    s.sel_cnt = t;
  }
  __syncthreads();
  upto = b1 < kBins ? s.sel_cnt : 0xffffffffu;
}

// Narrows the prefix to the shortest one with at least the mass `need`; the
// border's logit has a short key in [lo, hi], if the bounds that gave them are
// right (if not, the range becomes everything).
template <int DT>
__device__ void find_mass(Ctx<DT>& c, Row& row, long long need, uint32_t lo, uint32_t hi) {
  Shared& s = c.s;
  const Weight& w = c.w;
  const int t = threadIdx.x;
  constexpr int drop = Ctx<DT>::drop;
  const uint32_t all = ::max(short_key(row.thr, drop), kKeyNegInf >> drop);
  const uint32_t low = row.ties ? all : all + 1;  // smallest key of the prefix
  lo = ::max(lo, low);
  hi = ::max(hi, lo);
  if (hi == 0x7fffffffu >> drop) lo = ::min(lo, --hi);  // -0, which no logit is
  long long above = 0;
  uint32_t from = short_key(row.max, drop);  // keys above it are in `above`
  // Starts again with the whole prefix as the range, once.
  bool again = true;
  auto everything = [&]() {
    if (!again) return false;  // cannot be: the border lies in the whole prefix
    again = false;
    lo = low;
    hi = from = short_key(row.max, drop);
    above = row.above = 0;
    return true;
  };
  // The largest logit whose key is not above k (-0 is no logit's).
  auto largest_to = [&](uint32_t k) {
    return of_short(k == 0x7fffffffu >> drop ? k - 1 : k, drop);
  };
  // The warp's mass of keys above `a`, up to `b`, into its sums; and those in
  // the range into the bins.
  auto pass = [&](uint32_t a, uint32_t b, uint32_t* h, int sh) {
    long long sum = 0;
    c.each4([&](int, const float4& x4) {
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
      bool in[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t key = short_key(x[e], drop), at = hi - key;
        if (h && at <= hi - lo) atomicAdd(&h[at >> sh], 1u);
        in[e] = key > a && key <= b && x[e] > w.cut;
      }
      if (__any_sync(~0u, in[0] || in[1] || in[2] || in[3])) {
        Sum t4;
        c.add4(x, in, t4);
        sum += t4.value(4);
      }
    });
    return sum;
  };
  while (true) {
    const int sh = range_shift(hi - lo);
    uint32_t* h = c.begin_round();
    long long a = pass(hi, from, h, sh), z0 = 0, z1 = 0;
    row.above += warp_sum64(a);
    row.summed = largest_to(hi);
    const uint4 cnt4 = c.template end_round<true>(a, z0, z1);
    const uint32_t cnt[kPer] = {cnt4.x, cnt4.y, cnt4.z, cnt4.w};
    above += a;
    if (above >= need) {  // the range lies below the border
      if (!everything()) return;
      continue;
    }
    from = hi;
    const uint32_t k0 = hi - ((uint32_t)(kPer * t) << sh);
    if (sh == 0) {
      // a bin is one logit: exact masses
      long long m[kPer], wv[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        wv[i] = cnt[i] ? w.fixed(of_short(k0 - i, drop), s.table) : 0;
        sum += m[i] = wv[i] * cnt[i];
      }
      if (t == 0) s.sel_before[0] = 0;
      long long run = above + block_scan<long long>(sum, s.warp_a) - sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (run < need && run + m[i] >= need) {
          s.edge[0] = k0 - i;
          s.sel_before[0] = ceil_div(need - run, wv[i]);
        }
        run += m[i];
      }
      __syncthreads();
      const uint32_t key = s.edge[0];
      const uint32_t ties = (uint32_t)s.sel_before[0];
      __syncthreads();
      if (ties == 0) {  // the range lies above the border
        if (!everything()) return;
        continue;
      }
      set_border(row, key, ties, drop);
      return;
    }
    // bounds of the bins' masses from the weights at their edges
    const uint32_t width = (1u << sh) - 1;
    long long up[kPer], dn[kPer], su = 0, sd = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (cnt[i]) {
        const uint32_t k = k0 - ((uint32_t)i << sh);
        const long long wu = w.fixed(of_short(k, drop), s.table);
        const long long wd = w.fixed(of_short(k - lo > width ? k - width : lo, drop), s.table);
        su += (wu + (wu >> 20) + 1) * cnt[i];
        sd += ::max(wd - (wd >> 20) - 1, 0ll) * cnt[i];
      }
      up[i] = su;
      dn[i] = sd;
    }
    const long long iu = above + block_scan<long long>(su, s.warp_a) - su;
    const long long id = above + block_scan<long long>(sd, s.warp_b) - sd;
    if (t == 0) {
      s.sel_bin[0] = INT_MAX;
      s.sel_bin[1] = INT_MAX;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (iu + up[i] >= need) atomicMin(&s.sel_bin[0], kPer * t + i);
      if (id + dn[i] >= need) atomicMin(&s.sel_bin[1], kPer * t + i);
    }
    __syncthreads();
    const uint32_t b0 = (uint32_t)s.sel_bin[0], b1 = (uint32_t)s.sel_bin[1];
    __syncthreads();
    if (b0 == INT_MAX && !(lo == low)) {  // the range lies above the border
      if (!everything()) return;
      continue;
    }
    const uint32_t last = (hi - lo) >> sh;  // the range's last bin
    const uint32_t f0 = ::min(b0, last), f1 = ::min(b1, last);
    if ((uint64_t)(f1 - f0 + 1) << sh > (uint64_t)(hi - lo) / 2) {
      // the bounds are too wide (T far below the bins' width): halve the range
      const uint32_t half = hi - ((hi - lo) / 2 + 1);  // lo <= half < hi
      c.begin_round();
      long long part = pass(half, hi, nullptr, 0), z2 = 0, z3 = 0;
      const long long mine = warp_sum64(part);
      c.template end_round<true>(part, z2, z3);
      if (above + part >= need) {
        lo = half + 1;
      } else {
        above += part;
        row.above += mine;
        row.summed = largest_to(half);
        hi = from = half;
      }
      continue;
    }
    const uint32_t nhi = hi - (f0 << sh);
    const uint32_t e = hi - (f1 << sh);
    lo = e - lo > width ? e - width : lo;
    hi = nhi;
  }
}

// Four logits from global memory into the form they have in shared memory
// (fp32, or 16-bit pairs), with -0 as +0; `vec`: four may be read at once.
template <int DT>
struct Four {
  uint32_t w[DT == VT_FP32 ? 4 : 2];

  __device__ __forceinline__ void load(const void* p, int g, int n, bool vec) {
    if constexpr (DT == VT_FP32) {
      const float* x = static_cast<const float*>(p);
      if (vec && g + 3 < n) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(x + g));
        w[0] = __float_as_uint(v.x);
        w[1] = __float_as_uint(v.y);
        w[2] = __float_as_uint(v.z);
        w[3] = __float_as_uint(v.w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = g + e < n ? __float_as_uint(__ldcg(x + g + e)) : 0xff800000u;
      }
    } else {
      constexpr uint32_t kNegInf = DT == VT_BF16 ? 0xff80u : 0xfc00u;
      const unsigned short* x = static_cast<const unsigned short*>(p);
      if (vec && g + 3 < n) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2*>(x + g));
        w[0] = v.x;
        w[1] = v.y;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t a = g + 2 * e < n ? __ldcg(x + g + 2 * e) : kNegInf;
          const uint32_t b = g + 2 * e + 1 < n ? __ldcg(x + g + 2 * e + 1) : kNegInf;
          w[e] = a | b << 16;
        }
      }
    }
  }
  __device__ __forceinline__ void store(void* slice, int i) {
    if constexpr (DT == VT_FP32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) + 0.f);
      *reinterpret_cast<uint4*>(static_cast<float*>(slice) + i) =
          make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) w[e] &= ~__vcmpeq2(w[e], 0x80008000u);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(slice) + i) = make_uint2(w[0], w[1]);
    }
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a) {
  constexpr int kSize = DT == VT_FP32 ? 4 : 2;
  extern __shared__ __align__(16) unsigned char slice[];
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl::rank();
  uint32_t C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const int m = blockIdx.x / C;
  const int seg0 = ((int)rank * kWarps + warp) * a.seg;  // first element of the segment
  unsigned char* xs = slice + (size_t)warp * a.seg * kSize;

  cl::arrive();  // waited for before another CTA's shared memory is touched
  if (tid < 32) s.table[tid] = kTable[tid];
  if (tid == 0) s.found = 0;
  const float2 entry = kTable[lane];
  grid_launch_dependents();
  grid_dependency_wait();
  const float T = a.T_row ? __ldg(a.T_row + m) : a.T;
  const float top_p = a.top_p_row ? __ldg(a.top_p_row + m) : a.top_p;
  const float min_p = a.min_p_row ? __ldg(a.min_p_row + m) : a.min_p;
  const int top_k = a.top_k_row ? __ldg(a.top_k_row + m) : a.top_k;
  const float u = a.u ? __ldg(a.u + m) : 0.f;
  const bool needs_k = top_k > 0 && top_k < a.n, needs_p = top_p < 1.f;

  // ---- the row into shared memory and its maximum
  const char* row_p = static_cast<const char*>(a.logits) + (int64_t)m * a.ld * kSize;
  const bool vec = (reinterpret_cast<uintptr_t>(row_p) & (4 * kSize - 1)) == 0;
  constexpr int kBatch = 4;
  for (int i0 = 4 * lane; i0 < a.seg; i0 += 128 * kBatch) {
    Four<DT> v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (i0 + 128 * b < a.seg) v[b].load(row_p, seg0 + i0 + 128 * b, a.n, vec);
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (i0 + 128 * b < a.seg) v[b].store(xs, i0 + 128 * b);
  }
  if (tid == 32 && min_p > 0.f) s.min_off = (double)T * log((double)fminf(min_p, 1.f));
  __syncwarp();
  Weight w;
  Ctx<DT> c{s, w, xs, entry, a.seg, rank, C};
  float mx = -INFINITY, sum = 0.f;
  uint32_t cnt = 0;
  bool nan = false;
  c.each([&](float x) {
    nan |= x != x;
    mx = fmaxf(mx, x);
  });
  // The k-th largest of the warps' maxima has at least k logits at or above
  // it, and not many more; where there are not k warps, the mean of the finite
  // logits places the bins of the search for the k-th logit.
  const bool by_max = top_k <= (int)C * kWarps;
  if (needs_k && !by_max)
    c.each([&](float x) {
      if (fabsf(x) < 1e30f) {
        sum += x;
        ++cnt;
      }
    });
  float least = 0.f;
  if (needs_p && !needs_k) {
    // The 10th largest of 128 of the warp's logits, from all over its segment,
    // to 16 bits of its key: an estimate of where 8 % lie above.
    uint32_t key[4], t = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      key[e] = key_of(load1<DT>(xs, ((a.seg >> 7) * e >> 2 << 7) + 4 * lane + e)) >> 16;
    for (int b = 15; b >= 0; --b) {
      const uint32_t v = t | 1u << b;
      int n = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) n += __popc(__ballot_sync(~0u, key[e] >= v));
      if (n >= 10) t = v;
    }
    least = fmaxf(of_key(t << 16), -1e30f);
  }
  {
    // NaN travels as the largest key
    const uint32_t k = __reduce_max_sync(~0u, nan ? 0xffffffffu : key_of(mx));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    cnt = __reduce_add_sync(~0u, cnt);
    if (lane == 0) {
      s.warp_u[warp] = k;
      s.warp_f[warp] = sum;
      s.warp_a[warp] = cnt;
      s.warp_g[warp] = least;
    }
    __syncthreads();
    cl::wait();
    if (tid < (int)C * kWarps)
      cl::st_u32(cl::map(&s.warp_max[rank * kWarps + tid % kWarps], tid / kWarps),
                 s.warp_u[tid % kWarps]);
    if (needs_k && !by_max && tid < (int)C) {
      uint32_t bc = 0;
      float bs = 0.f;
      for (int i = 0; i < kWarps; ++i) {
        bs += s.warp_f[i];
        bc += (uint32_t)s.warp_a[i];
      }
      cl::st_u32(cl::map(&s.cta_sum[rank], tid), __float_as_uint(bs));
      cl::st_u32(cl::map(&s.cta_cnt[rank], tid), bc);
    } else if (tid < (int)C) {
      float t = 0.f;  // of the warps with a whole segment
      uint32_t k = 0;
      for (int i = 0; i < kWarps; ++i)
        if (((int)rank * kWarps + i + 1) * a.seg <= a.n) {
          t += s.warp_g[i];
          ++k;
        }
      cl::st_u32(cl::map(&s.cta_sum[rank], tid), __float_as_uint(t));
      cl::st_u32(cl::map(&s.cta_cnt[rank], tid), k);
    }
    cl::sync();
  }
  Row row;
  uint32_t kmax = 0, kth = 0;
  float place = 0.f;  // few of the top k lie below
  for (int i = lane; i < (int)C * kWarps; i += 32) kmax = ::max(kmax, s.warp_max[i]);
  kmax = __reduce_max_sync(~0u, kmax);
  if (needs_k && by_max) {
    kth = nth_max(s, (int)C * kWarps, top_k - 1);
    place = of_key(kth);
  } else if (needs_k) {
    uint32_t k = 0;
    for (uint32_t r = 0; r < C; ++r) {
      place += s.cta_sum[r];
      k += s.cta_cnt[r];
    }
    place = k ? place / (float)k : 0.f;
  }
  float least_mean = -INFINITY;
  if (needs_p && !needs_k) {
    uint32_t k = 0;
    float t = 0.f;
    for (uint32_t r = 0; r < C; ++r) {
      t += s.cta_sum[r];
      k += s.cta_cnt[r];
    }
    if (k) least_mean = t / (float)k;
  }
  row.max = of_key(kmax);
  row.thr = -INFINITY;
  row.ties = 0;
  row.summed = INFINITY;
  row.above = 0;
  const bool bad = kmax == 0xffffffffu || !(T >= 0.f && T < INFINITY) || !(top_p == top_p) ||
                   !(min_p == min_p) || top_k < 0 || !(u >= 0.f && u <= 1.f);
  if (bad || kmax <= kKeyNegInf) {
    // a NaN among the logits or settings: id -1, NaN; nothing left: -1, 0
    const float v = bad ? __int_as_float(0x7fffffff) : 0.f;
    if (rank == 0 && tid == 0 && a.ids) {
      a.ids[m] = -1;
      a.probs[m] = v;
    }
    if (a.dist)
      for (int i = lane; i < a.seg; i += 32)
        if (seg0 + i < a.n) a.dist[(int64_t)m * a.ld_dist + seg0 + i] = v;
    return;  // no CTA touches another's shared memory after the last barrier
  }
  w.init(row.max, T);
  // the smallest logit that min-p keeps
  const float min_x =
      min_p > 0.f ? __double2float_ru((double)row.max + s.min_off) + 0.f : -INFINITY;
  float* dist = a.dist ? a.dist + (int64_t)m * a.ld_dist : nullptr;
  const bool dvec = (reinterpret_cast<uintptr_t>(dist) & 15) == 0;

  // Zeros for this warp's segment of the distribution.
  auto clear_dist = [&]() {
    if (!dist) return;
    for (int i = 4 * lane; i < a.seg; i += 128) {
      const int g = seg0 + i;
      if (dvec && g + 3 < a.n) {
        *reinterpret_cast<float4*>(dist + g) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + e < a.n) dist[g + e] = 0.f;
      }
    }
  };

  // ---- the prefix that is kept
  if (w.top_only) {
    row.thr = row.max;
    row.ties = 1;  // T = 0: the first maximum.  +inf: settled by the count below
  } else if (needs_k || needs_p) {
    float scale = 1.f;
    auto set_scale = [&](float range) {
      scale = (float)(kBins - 1) / range;
      if (!(scale > 0.f && scale < 1e37f)) scale = 1.f;
    };
    // Counts the prefix's logits into the linear bins.
    auto count_bins = [&]() {
      uint32_t* h = c.begin_round();
      if (row.ties && rank == 0 && tid == 0) {
        const uint32_t b = lin_bin(row.thr, row.max, scale);
        if (b < kBins) atomicAdd(&h[b], row.ties);
      }
      c.each([&](float x) {
        const uint32_t b = lin_bin(x, row.max, scale);
        if (b < kBins && x > row.thr) atomicAdd(&h[b], 1u);
      });
    };
    // Puts the logits that pass into the CTAs' lists; how many there are in all.
    auto gather = [&](auto pass) {
      uint64_t* own = s.own_list();
      c.each4([&](int i, const float4& x4) {
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (pass(x[e])) {
            const unsigned k = atomicAdd(&s.found, 1u);
            if (k < kList)
              own[k] = (uint64_t)key_of(x[e]) << 32 | (uint32_t)~(seg0 + c.place(i + e));
          }
      });
      __syncthreads();
      if (tid < (int)C) cl::st_u32(cl::map(&s.list_cnt[rank], tid), s.found);
      cl::sync();
      uint32_t n = 0;
      for (uint32_t r = 0; r < C; ++r) n += s.list_cnt[r];
      return n;
    };
    uint32_t L = 0;       // logits in the lists; 0: the search goes on
    long long mass = 0;   // of the whole row, where top-p alone needs it
    if (needs_k) {
      uint32_t n = 0xffffffffu;
      // gathered at the k-th largest of the warps' maxima, without a histogram
      // first (1 x 128256, top-k 50: 8.8 us, 12.0 with one; 60 rows: 21.3, 29.1)
      if (by_max && kth > kKeyNegInf) {
        clear_dist();
        n = gather([&](float x) { return x >= place; });
      }
      if (n > kList) {
        set_scale(row.max - place);
        count_bins();
        select_bin(s, c.end_round(), (uint32_t)top_k);
        const int b = s.sel_bin[0];
        const uint32_t in = (uint32_t)s.sel_before[0] + s.sel_cnt;
        // few enough to be ranked in one place (1 x 32768, top-k and top-p:
        // 9.9 us; with the searches over keys 25.7)
        if (b >= 0 && in <= kList) {
          if (tid == 0) s.found = 0;
          __syncthreads();
          clear_dist();
          n = gather([&](float x) { return lin_bin(x, row.max, scale) <= (uint32_t)b; });
        } else {
          find_count(c, row, (uint32_t)top_k, scale);
          __syncthreads();
        }
      }
      if (n <= kList) L = n;
    }
    if (needs_p && L == 0) {
      // The prefix's exact mass, and counts over bins that reach down to the
      // prefix's end, or to where all n logits together weigh e^-5 of what
      // top_p leaves out at the least.  A language model's nucleus is a few
      // per cent of its vocabulary: the logits above `least`, about 8 % of
      // them, are packed on the way, and if their mass holds the border,
      // nothing else is looked at again (128256 logits, top-p 0.9: 1 row 20.2
      // us, 24.6 without; 60 rows 59, 71).
      float range = T * (__logf((float)a.n / fmaxf(1.f - top_p, 1e-7f)) + 5.f);
      const float have = row.max - row.thr;
      if (have < range) range = have;
      const float near = needs_k ? range : fminf(range, row.max - least_mean);
      const float keep = fmaxf(row.thr, w.cut);
      const bool pack = near < range && near > 0.f;
      const float least = row.max - near;
      Sum all;
      int n = 0;  // packed logits; past the list's end: too many
      const uint32_t lanes_before = (1u << lane) - 1u;
      unsigned char* list = slice + (size_t)kWarps * a.seg * kSize + (size_t)warp * a.cap * kSize;
      uint16_t* pos = reinterpret_cast<uint16_t*>(slice + (size_t)kWarps * (a.seg + a.cap) * kSize) +
                      warp * a.cap;
      c.each4([&](int i, const float4& x4) {
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
        const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(~0u, top > keep)) {
          const bool in[4] = {x[0] > keep, x[1] > keep, x[2] > keep, x[3] > keep};
          c.add4(x, in, all);
        } else {
          all.hi += 4u * Weight::kHi0;
          all.lo += 4u * Weight::kLo0;
        }
        if (pack && __any_sync(~0u, top >= least)) {
          int at = n, sum = 0;  // place of this lane's first
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t in = __ballot_sync(~0u, x[e] >= least);
            at += __popc(in & lanes_before);
            sum += __popc(in);
          }
          if (n + sum <= a.cap) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (x[e] >= least) {
                store1<DT>(list, at, x[e]);
                pos[at++] = (uint16_t)(i + e);
              }
          }
          n += sum;
        }
      });
      mass = all.value(c.per_lane());
      long long packed = 0, full = !pack || n > a.cap;  // their mass; lists that are short
      if (!full) {
        for (int i = n + lane; i < (n + 127) / 128 * 128; i += 32) store1<DT>(list, i, -INFINITY);
        __syncwarp();
        for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
          const float x = i < n ? load1<DT>(list, i) : -INFINITY;
          uint32_t p, l;
          c.add(x, x > keep, p, l);
          packed += ((long long)(p - Weight::kHi0) << 22) + (int)(l - Weight::kLo0);
        }
      }
      c.sum_over(mass, packed, full);
      if (row.ties) mass += w.fixed(row.thr, s.table) * (long long)row.ties;
      const long long need = ::min(::max(mul_frac(mass, top_p, true), 1ll), mass);
      const float target = __ll2float_rn(need) * 0x1p-42f;
      if (full == 0 && packed >= need) {  // the border lies among the packed logits
        c.xs = list;
        c.pos = pos;
        c.seg = (n + 127) / 128 * 128;
        range = near;
      }
      set_scale(range);
      const float step = 1.44269504f / (T * scale);
      int b0, b1;
      uint32_t upto;
      count_bins();
      bound_mass(s, c.end_round(), target, step, b0, b1, upto);
      // (1 x 32768, top-p 0.5: 13.2 us, 21.0 with the search over keys)
      if (!needs_k && upto <= kList) {
        if (tid == 0) s.found = 0;
        __syncthreads();
        clear_dist();
        L = gather([&](float x) { return lin_bin(x, row.max, scale) <= (uint32_t)b1; });
      } else {
        if (tid < 64) {
          const int v = tid >> 5;
          const uint32_t e = v == 0 ? (b1 == kBins ? 0u : first_key(b1, row.max, scale, c.drop))
                             : b0 > 0 ? first_key(b0 - 1, row.max, scale, c.drop) - 1
                                      : short_key(row.max, c.drop);
          if (lane == 0) s.edge[v] = e;
        }
        __syncthreads();
        const uint32_t end = c.pos ? short_key(least, c.drop) : 0u;  // nothing below it
        const uint32_t lo = ::max(s.edge[0], end), hi = s.edge[1];
        __syncthreads();
        find_mass(c, row, need, lo, hi);
      }
    }
    if (L > 0) {
      // ---- few logits can be kept: the first CTA takes the lists over (no
      // other leaves before it has) and settles everything
      uint64_t key = 0;
      if (rank == 0 && tid < (int)L) {
        uint32_t r = 0, at = tid;
        while (at >= s.list_cnt[r]) at -= s.list_cnt[r++];
        key = cl::ld_u64(cl::map(s.own_list() + at, r));
      }
      cl::sync();
      if (rank != 0) return;
      uint64_t* keys = s.list_key();
      long long* ws = s.list_w();
      if (tid < (int)L) keys[tid] = key;
      const float x = of_key((uint32_t)(key >> 32));
      const int idx = (int)~(uint32_t)key;
      const long long wi = tid < (int)L ? w.fixed(x, s.table) : 0;
      if (tid < (int)L) ws[tid] = wi;
      __syncthreads();
      int nth = 0;          // in the sorted order
      long long over = 0;   // mass before it
      if (warp * 32 < (int)L)
        for (int j = 0; j < (int)L; ++j) {
          const bool before = keys[j] > key;
          nth += before;
          over += before ? ws[j] : 0;
        }
      bool keep = tid < (int)L;
      if (needs_k) {
        keep = keep && nth < top_k;
        if (needs_p) mass = block_sum64(keep ? wi : 0, s.warp_b);
      }
      if (needs_p) {
        const long long need = ::min(::max(mul_frac(mass, top_p, true), 1ll), mass);
        keep = keep && over < need;
      }
      keep = keep && x >= min_x;
      const long long kept = keep ? wi : 0;
      const long long total = block_sum64(kept, s.warp_c);
      if (tid < (int)L) ws[tid] = kept;
      __syncthreads();
      const float inv = 0x1p42f / __ll2float_rn(total);
      const float p = keep ? w.real(x, s.table) * inv : 0.f;
      if (a.ids) {
        long long run = 0;  // kept mass at lower indexes
        if (warp * 32 < (int)L)
          for (int j = 0; j < (int)L; ++j) run += (int)~(uint32_t)keys[j] < idx ? ws[j] : 0;
        const long long target = ::min(mul_frac(total, u, false), total - 1);
        if (keep && run <= target && target < run + wi && VT_CHECKED(idx >= 0 && idx < a.n)) {
          a.ids[m] = a.t2f ? __ldg(a.t2f + idx) : idx;
          a.probs[m] = p;
        }
      }
      if (dist && keep && VT_CHECKED(idx >= 0 && idx < a.n)) dist[idx] = p;
      return;
    }
  }
  if (!w.top_only && min_x > -INFINITY) {
    // as a border: the largest value below it is dropped
    const float below = nextafterf(min_x, -INFINITY);
    if (below >= row.thr) {
      row.thr = below;
      row.ties = 0;
    }
  }

  // ---- sums of the kept weights over segments, CTAs and the row
  // (the search for the border has summed some of them; min-p may since have
  // dropped logits from among those)
  const float keep_x = fmaxf(row.thr, w.cut);
  long long ws = 0;
  uint32_t ties = 0;
  if (!w.top_only) {
    const bool some = row.thr <= row.summed && row.summed < INFINITY;
    const float below_x = some ? row.summed : INFINITY;
    Sum t;
    c.each4([&](int, const float4& x) {
      const float v[4] = {x.x, x.y, x.z, x.w};
      bool in[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        in[e] = v[e] > keep_x && v[e] <= below_x;
        if (row.ties) ties += v[e] == row.thr;
      }
      if (__any_sync(~0u, in[0] || in[1] || in[2] || in[3])) {
        c.add4(v, in, t);
      } else {
        t.hi += 4u * Weight::kHi0;
        t.lo += 4u * Weight::kLo0;
      }
    });
    ws = warp_sum64(t.value(c.per_lane())) + (some ? row.above : 0);
  }
  if (w.top_only) c.each([&](float x) { ties += x == row.thr; });
  ties = __reduce_add_sync(~0u, ties);
  __syncthreads();
  if (lane == 0) {
    s.warp_a[warp] = ws;
    s.warp_u[warp] = ties;
  }
  __syncthreads();
  if (tid < (int)C) {
    long long t = 0;
    uint32_t e = 0;
    for (int i = 0; i < kWarps; ++i) {
      t += s.warp_a[i];
      e += s.warp_u[i];
    }
    cl::st_u64(cl::map(&s.fin_sum[rank], tid), (uint64_t)t);
    cl::st_u32(cl::map(&s.fin_ties[rank], tid), e);
  }
  cl::sync();
  // no CTA touches another's shared memory from here on
  if (w.top_only && T > 0.f) {
    // +inf logits share the mass equally; the filters count them
    uint32_t e = 0;
    for (uint32_t r = 0; r < C; ++r) e += s.fin_ties[r];
    if (top_k > 0) e = ::min(e, (uint32_t)top_k);
    if (needs_p) e = ::max((uint32_t)mul_frac(e, top_p, true), 1u);
    row.ties = e;
  }
  const long long wt = row.ties ? w.fixed(row.thr, s.table) : 0;
  long long total = 0, before = 0;
  uint32_t left = row.ties;  // ties not yet given out
  uint32_t my_left = 0;
  for (uint32_t r = 0; r < C; ++r) {
    if (r == rank) {
      before = total;
      my_left = left;
    }
    const uint32_t e = ::min(left, s.fin_ties[r]);
    total += s.fin_sum[r] + wt * e;
    left -= e;
  }
  for (int i = 0; i < warp; ++i) {
    const uint32_t e = ::min(my_left, s.warp_u[i]);
    before += s.warp_a[i] + wt * e;
    my_left -= e;
  }
  const long long mine = ws + wt * ::min(my_left, ties);

  // Which of a lane's four logits are kept, given the ties still to give out
  // before these 128; the whole warp.  Returns the ties among the 128.
  auto kept4 = [&](const float (&x)[4], uint32_t budget, bool (&keep)[4]) -> uint32_t {
    uint32_t tie = 0, tb = 0, all = 0;
    if (row.ties) {
#pragma unroll
      for (int e = 0; e < 4; ++e) tie += x[e] == row.thr;
      if (__any_sync(~0u, tie)) {
        tb = tie;  // ties in the lanes before, then in this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(~0u, tb, o);
          if (lane >= o) tb += y;
        }
        all = __shfl_sync(~0u, tb, 31);
        tb -= tie;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      keep[e] = x[e] > row.thr;
      if (row.ties && x[e] == row.thr) keep[e] = tb++ < budget;
    }
    return all;
  };

  // ---- the draw: the segment that holds it walks through its elements
  const float inv = 0x1p42f / __ll2float_rn(total);
  const long long target = ::min(mul_frac(total, u, false), total - 1);
  if (a.ids && before <= target && target < before + mine) {
    long long run = before;
    uint32_t budget = my_left;
    for (int i = 4 * lane; i < c.seg; i += 128) {
      const float4 x4 = unpack4<DT>(c.xs, i);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
      bool keep[4];
      const uint32_t block_ties = kept4(x, budget, keep);
      long long v[4], sumv = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) sumv += v[e] = keep[e] ? w.fixed(x[e], s.table) : 0;
      const long long inc = warp_scan64(sumv, lane);
      const uint32_t hit = __ballot_sync(~0u, run + inc > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          long long at = run + inc - sumv;
          int e = 0;
          while (e < 3 && at + v[e] <= target) at += v[e++];
          const int g = seg0 + c.place(i + e);
          if (VT_CHECKED(g < a.n)) {
            const float xe = e == 0 ? x[0] : e == 1 ? x[1] : e == 2 ? x[2] : x[3];
            a.ids[m] = a.t2f ? __ldg(a.t2f + g) : g;
            a.probs[m] = w.real(xe, s.table) * inv;
          }
        }
        break;
      }
      run += __shfl_sync(~0u, inc, 31);
      budget -= ::min(budget, block_ties);
    }
  }

  // ---- the filtered distribution
  if (dist && c.pos) {
    clear_dist();
    __syncwarp();
    uint32_t budget = my_left;
    for (int i = 4 * lane; i < c.seg; i += 128) {
      const float4 x4 = unpack4<DT>(c.xs, i);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
      bool keep[4];
      const uint32_t block_ties = kept4(x, budget, keep);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (keep[e]) {
          const int g = seg0 + c.place(i + e);
          if (VT_CHECKED(g < a.n)) dist[g] = w.real(x[e], s.table) * inv;
        }
      budget -= ::min(budget, block_ties);
    }
  } else if (dist) {
    uint32_t budget = my_left;
    for (int i = 4 * lane; i < a.seg; i += 128) {
      const float4 x4 = unpack4<DT>(xs, i);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
      float p[4] = {0.f, 0.f, 0.f, 0.f};
      if (__any_sync(~0u, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= row.thr)) {
        bool keep[4];
        const uint32_t block_ties = kept4(x, budget, keep);
        c.real4(x, keep, inv, p);
        budget -= ::min(budget, block_ties);
      }
      const int g = seg0 + i;
      if (dvec && g + 3 < a.n) {
        *reinterpret_cast<float4*>(dist + g) = make_float4(p[0], p[1], p[2], p[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + e < a.n) dist[g + e] = p[e];
      }
    }
  }
}

// Packed logits: a quarter of a segment (three times what is expected, since
// frequent tokens tend to lie together).
int list_cap(int seg) { return (seg / 4 + 127) / 128 * 128; }
// Shared memory of a CTA: segments, lists, and places.
size_t slice_bytes(int seg, int size) {
  return (size_t)kWarps * ((size_t)(seg + list_cap(seg)) * size + list_cap(seg) * 2);
}
int segment(int n, int C) { return ((n + C * kWarps - 1) / (C * kWarps) + 127) / 128 * 128; }

// CTAs per row (0: none fits): the least time of waves * (the chain of
// barriers, and the logits an SM's resident CTAs work through), with the
// number of clusters that run at a time as the device gives it (1 x 32768: 12.4,
// 7.8, 7.5 us with 4, 8, 16; 60 x 128256, top-p: 61, 59, 63, 67, 73 us with 7,
// 9, 10, 12, 14; it takes 16 and 9).  Asked once per shape.
template <int DT>
int choose_cluster(int M, int n, const DeviceInfo& di) {
  constexpr int kSize = DT == VT_FP32 ? 4 : 2;
  static std::mutex mu;
  static std::map<std::tuple<int, int, int>, int> chosen;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(di.device, n, M);
  const auto it = chosen.find(key);
  if (it != chosen.end()) return it->second;
  int C = 0;
  float best = 0.f;
  for (int c = 1; c <= kMaxCluster && (c == 1 || n >= c * 1024); ++c) {
    const int seg = segment(n, c);
    const size_t smem = slice_bytes(seg, kSize);
    if (smem + sizeof(Shared) + 64 > (size_t)di.max_smem_optin) continue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, sample_kernel<DT>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      continue;
    }
    if (active < 1) continue;
    const float waves = (float)((M + active - 1) / active);
    const float per_sm = fmaxf(1.f, (float)std::min(M, active) * c / di.num_sms);
    const float t = waves * (6.f + (float)(seg * kWarps) * per_sm * 2.6e-4f);
    if (C == 0 || t < best) {
      best = t;
      C = c;
    }
  }
  try {
    if (chosen.size() > 4096) chosen.clear();
    chosen.emplace(key, C);
  } catch (...) {  // no memory: asked again next time
  }
  return C;
}

template <int DT>
vt_status launch(SampleArgs a, int M, const DeviceInfo& di, cudaStream_t s) {
  constexpr int kSize = DT == VT_FP32 ? 4 : 2;
  auto kernel = sample_kernel<DT>;
  if (!allow_max_smem(kernel, di)) return VT_ERR_CUDA;
  static std::atomic<uint64_t> wide{0};  // devices whose kernel may have 16 CTAs a cluster
  const uint64_t bit = 1ull << (di.device & 63);
  if (!(wide.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
      return fail(VT_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
    wide.fetch_or(bit);
  }
  const int C = choose_cluster<DT>(M, a.n, di);
  if (C == 0) return fail(VT_ERR_UNSUPPORTED, "vt_sample_logits: no cluster fits this device");
  a.seg = segment(a.n, C);
  a.cap = list_cap(a.seg);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(M * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = slice_bytes(a.seg, kSize);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess)
    return fail(VT_ERR_CUDA, std::string("sample_kernel: ") + cudaGetErrorString(e));
  return launch_status("sample_kernel");
}

}  // namespace
}  // namespace vt

extern "C" vt_status vt_sample_logits(const void* logits, int32_t dtype, int32_t M, int32_t n,
                                      int64_t ld, const vt_sample_options* opts, const float* u,
                                      const int32_t* t2f, int32_t* out_ids, float* out_probs,
                                      float* out_dist, int64_t ld_dist, void* stream) {
  using namespace vt;
  if (dtype != VT_BF16 && dtype != VT_FP16 && dtype != VT_FP32)
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: unknown dtype");
  if (M < 0 || n < 1) return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: need M >= 0, n >= 1");
  if (n > kMaxN) return fail(VT_ERR_UNSUPPORTED, "vt_sample_logits: n > 2^19");
  if (M > 65535) return fail(VT_ERR_UNSUPPORTED, "vt_sample_logits: M > 65535");
  vt_sample_options o = {1.f, 0, 1.f, 0.f, nullptr, nullptr, nullptr, nullptr};
  if (opts) o = *opts;
  if (!o.temperature_rows && !(o.temperature >= 0.f && o.temperature < INFINITY))
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: temperature must be finite and >= 0");
  if (!o.top_k_rows && o.top_k < 0)
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: top_k must be >= 0");
  if (!o.top_p_rows && !(o.top_p == o.top_p))
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: top_p is NaN");
  if (!o.min_p_rows && !(o.min_p == o.min_p))
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: min_p is NaN");
  if (M == 0) return VT_OK;
  const int size = dtype == VT_FP32 ? 4 : 2;
  if (!logits) return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: null logits");
  if ((u || out_ids || out_probs) && !(u && out_ids && out_probs))
    return fail(VT_ERR_INVALID_ARG,
                "vt_sample_logits: u, out_ids and out_probs come together or not at all");
  if (!u && !out_dist) return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: nothing to compute");
  if (M > 1 && (ld < n || (out_dist && ld_dist < n)))
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: row stride below n");
  if (!aligned(logits, size) || !aligned(u, 4) || !aligned(t2f, 4) || !aligned(out_ids, 4) ||
      !aligned(out_probs, 4) || !aligned(out_dist, 4) || !aligned(o.temperature_rows, 4) ||
      !aligned(o.top_k_rows, 4) || !aligned(o.top_p_rows, 4) || !aligned(o.min_p_rows, 4))
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: misaligned pointer");
  if (outputs_overlap({rows_range(out_dist, M, ld_dist, n, 4), {out_ids, 4ll * M},
                       {out_probs, 4ll * M}},
                      {rows_range(logits, M, ld, n, size), {u, 4ll * M}, {t2f, 4ll * n},
                       {o.temperature_rows, 4ll * M}, {o.top_k_rows, 4ll * M},
                       {o.top_p_rows, 4ll * M}, {o.min_p_rows, 4ll * M}}))
    return fail(VT_ERR_INVALID_ARG, "vt_sample_logits: an output overlaps an input or another");
  DeviceInfo di;
  if (!current_device(&di)) return VT_ERR_CUDA;
  SampleArgs a;
  a.logits = logits;
  a.ld = ld;
  a.n = n;
  a.seg = a.cap = 0;
  a.u = u;
  a.t2f = t2f;
  a.T = o.temperature;
  a.top_p = o.top_p;
  a.min_p = o.min_p;
  a.top_k = o.top_k;
  a.T_row = o.temperature_rows;
  a.top_p_row = o.top_p_rows;
  a.min_p_row = o.min_p_rows;
  a.top_k_row = o.top_k_rows;
  a.ids = out_ids;
  a.probs = out_probs;
  a.dist = out_dist;
  a.ld_dist = ld_dist;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == VT_BF16   ? launch<VT_BF16>(a, M, di, s)
         : dtype == VT_FP16 ? launch<VT_FP16>(a, M, di, s)
                            : launch<VT_FP32>(a, M, di, s);
}
