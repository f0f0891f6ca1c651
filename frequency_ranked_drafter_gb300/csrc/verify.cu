// vt_verify_draft — the acceptance test of speculative decoding over a chain
// of drafted tokens.
//
// "FR-Spec: ...", Method > Key design: the target verifies with rejection
// sampling, which keeps the output exactly the target's distribution.  For
// position j of a sequence, with the target's p_j, the drafter's q_j and a
// uniform u_j, the drafted token x_j is accepted while u_j * q_j(x_j) <
// p_j(x_j); at the first rejection the next token is drawn from
// max(p_j - q_j, 0), and after the last accepted draft from p_j, both by
// inverse CDF in the order of the ids with the sequence's last uniform.  q may
// cover only the kept ids of a trimmed drafter (f2t maps ids to its columns;
// a dropped id has q = 0).
//
// One cluster of up to 16 CTAs per sequence; no workspace.  Every CTA settles
// the chain for itself (K loads, three dependent round trips), then the CTAs
// stream the one row pair that is needed, a contiguous segment a warp.  Masses
// are fixed point (2^44 for probability 1), taken apart by fp32 additions and
// summed as integers, so sums are exact and do not depend on the split.  The
// product u * q is compared in fp64, where it is exact.  The warp whose segment
// holds the draw reads it again (it lies in L2) and walks through it.
// Bound by reading the two rows (8 V bytes a sequence) where there are many
// sequences (B = 256, V = 128256: 56 us, 4.7 TB/s; B = 64: 18 us, 3.7 TB/s); few
// are bound by the chain of dependent round trips, some 5 us (B = 1: 7 us).
#include <algorithm>
#include <atomic>
#include <climits>

#include "cluster.cuh"
#include "ranges.cuh"
#include "verify_plan.cuh"
#include "vt_checks.cuh"
#include "vt_common.cuh"

namespace vt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = kVerifyMaxCluster;
constexpr int kMaxV = 1 << 19;  // 2^19 probabilities of at most 2^44 stay below 2^63
constexpr int kBatch = 4;       // 16-byte loads of each row a lane has in flight

struct VerifyArgs {
  const int32_t* draft;  // [B][K]
  const int32_t* n_draft;
  int K, V, Vq, seg;  // seg: a warp's ids, a multiple of 128
  const float* p;
  int64_t p_seq, p_pos;  // strides of p between sequences and positions
  const float* q;
  int64_t q_seq, q_pos;
  const int32_t* f2t;
  const float* u;  // [B][K + 1]
  int32_t* accepted;
  int32_t* out;  // [B][K + 1]
};

// A probability in fixed point: hi * 2^22 + lo = p * 2^44 (raw float bits, of
// which differences are taken).  NaN and negative values count as 0, values
// above 1 as 1.
__device__ __forceinline__ void split(float p, int& hi, int& lo) {
  p = fminf(fmaxf(p, 0.f), 1.f);
  const float t = p + 3.f;  // last place 2^-22
  hi = __float_as_int(t);
  lo = __float_as_int((p - (t - 3.f)) + 0x1.8p-21f);  // last place 2^-44
}
// max(p - q, 0), in two parts.
__device__ __forceinline__ void residual(float p, float q, int& hi, int& lo) {
  int ph, pl, qh, ql;
  split(p, ph, pl);
  split(q, qh, ql);
  hi = ph - qh;
  lo = pl - ql;
  // the parts' sum has the sign of the difference
  if (!((hi > 0) || (hi == 0 && lo > 0))) hi = lo = 0;
}
__device__ __forceinline__ long long join(int hi, int lo) { return ((long long)hi << 22) + lo; }

struct Rows {
  const float* p;
  const float* q;  // null: nothing is taken away
  const int32_t* f2t;
  int V, Vq;
  bool vec;  // four ids at a time

  __device__ __forceinline__ float q_at(int i) const {
    if (!f2t) return __ldg(q + i);
    const int col = __ldg(f2t + i);
    return col >= 0 && col < Vq ? __ldg(q + col) : 0.f;
  }
  // The four ids from i on (0 past the end).
  __device__ __forceinline__ void load(int i, float (&a)[4], float (&b)[4]) const {
    if (vec && i + 3 < V) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
      if (!q) {
        b[0] = b[1] = b[2] = b[3] = 0.f;
      } else if (!f2t) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(q + i));
        b[0] = w.x; b[1] = w.y; b[2] = w.z; b[3] = w.w;
      } else {
        const int4 c = __ldg(reinterpret_cast<const int4*>(f2t + i));
        b[0] = c.x >= 0 && c.x < Vq ? __ldg(q + c.x) : 0.f;
        b[1] = c.y >= 0 && c.y < Vq ? __ldg(q + c.y) : 0.f;
        b[2] = c.z >= 0 && c.z < Vq ? __ldg(q + c.z) : 0.f;
        b[3] = c.w >= 0 && c.w < Vq ? __ldg(q + c.w) : 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = i + e < V ? __ldg(p + i + e) : 0.f;
        b[e] = i + e < V && q ? q_at(i + e) : 0.f;
      }
    }
  }
};

// Mass of a warp's ids [i0, end).
__device__ __forceinline__ long long segment_mass(const Rows& r, int i0, int end) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int i = i0 + 4 * lane; i < end; i += 128 * kBatch) {
    float a[kBatch][4], b[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + 128 * k < end) r.load(i + 128 * k, a[k], b[k]);
    int sh = 0, sl = 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + 128 * k < end)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int hi, lo;
          residual(a[k][e], b[k][e], hi, lo);
          sh += hi;
          sl += lo;
        }
    sum += join(sh, sl);
  }
  return warp_sum64(sum);
}

__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
  __shared__ long long warp_sum[kWarps];
  __shared__ long long cta_sum[2][kMaxCluster];
  __shared__ int s_acc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl::rank();
  uint32_t C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const int b = blockIdx.x / C;
  cl::arrive();  // waited for before another CTA's shared memory is touched
  grid_launch_dependents();
  grid_dependency_wait();

  // ---- the chain: the first position that is rejected, or the draft's length
  const float* p_seq = a.p + (int64_t)b * a.p_seq;
  const float* q_seq = a.q + (int64_t)b * a.q_seq;
  const float* u = a.u + (int64_t)b * (a.K + 1);
  const int len = a.n_draft ? ::min(::max(__ldg(a.n_draft + b), 0), a.K) : a.K;
  const float un = __ldg(u + a.K);
  if (warp == 0) {
    int acc = len;
    for (int j0 = 0; j0 < len; j0 += 32) {
      const int j = j0 + lane;
      bool ok = true;
      if (j < len) {
        const int x = __ldg(a.draft + (int64_t)b * a.K + j);
        const float uj = __ldg(u + j);
        ok = x >= 0 && x < a.V;  // another id is rejected
        if (ok) {
          const float px = __ldg(p_seq + (int64_t)j * a.p_pos + x);
          const int col = a.f2t ? __ldg(a.f2t + x) : x;
          const float qx =
              col >= 0 && col < a.Vq ? __ldg(q_seq + (int64_t)j * a.q_pos + col) : 0.f;
          ok = (double)uj * (double)qx < (double)px;
        }
      }
      const uint32_t no = __ballot_sync(~0u, !ok);
      if (no) {
        acc = j0 + __ffs(no) - 1;
        break;
      }
    }
    if (lane == 0) s_acc = acc;
  }
  __syncthreads();
  const int acc = s_acc;
  Rows rows;
  rows.p = p_seq + (int64_t)acc * a.p_pos;
  rows.q = acc < len && a.Vq > 0 ? q_seq + (int64_t)acc * a.q_pos : nullptr;
  rows.f2t = a.f2t;
  rows.V = a.V;
  rows.Vq = a.Vq;
  const uintptr_t other = a.f2t ? reinterpret_cast<uintptr_t>(a.f2t)
                                : reinterpret_cast<uintptr_t>(rows.q);
  rows.vec = ((reinterpret_cast<uintptr_t>(rows.p) | other) & 15) == 0;

  int32_t* out = a.out + (int64_t)b * (a.K + 1);
  if (rank == 0) {
    if (tid == 0) a.accepted[b] = acc;
    for (int j = tid; j <= a.K; j += kThreads)
      if (j != acc) out[j] = j < acc ? __ldg(a.draft + (int64_t)b * a.K + j) : -1;
  }

  // ---- masses of max(p - q, 0); once more of p where that is nothing at all
  const int seg0 = ((int)rank * kWarps + warp) * a.seg;
  const int end = ::min(seg0 + a.seg, a.V);
  cl::wait();
  long long mine = 0, total = 0;
  int turn = 0;
  for (; turn < 2; ++turn) {
    mine = segment_mass(rows, seg0, end);
    if (lane == 0) warp_sum[warp] = mine;
    __syncthreads();
    if (tid < (int)C) {
      long long t = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += warp_sum[w];
      cl::st_u64(cl::map(&cta_sum[turn][rank], tid), (uint64_t)t);
    }
    cl::sync();
    for (uint32_t r = 0; r < C; ++r) total += cta_sum[turn][r];
    if (total > 0 || !rows.q) break;
    rows.q = nullptr;  // p nowhere above q: draw from p
  }
  // no CTA touches another's shared memory from here on
  if (total <= 0 || !(un >= 0.f && un <= 1.f)) {  // nothing to draw from, or no uniform
    if (rank == 0 && tid == 0) out[acc] = -1;
    return;
  }
  const long long target = ::min((long long)((double)un * (double)total), total - 1);
  long long run = 0;
  for (uint32_t r = 0; r < rank; ++r) run += cta_sum[turn][r];
  for (int w = 0; w < warp; ++w) run += warp_sum[w];
  if (run > target || run + mine <= target) return;

  // ---- this warp's segment holds the token
  for (int i0 = seg0; i0 < end; i0 += 128 * kBatch) {
    float x[kBatch][4], y[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + 128 * k < end) rows.load(i0 + 128 * k + 4 * lane, x[k], y[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + 128 * k >= end) break;
      long long v[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int hi, lo;
        residual(x[k][e], y[k][e], hi, lo);
        sum += v[e] = join(hi, lo);
      }
      const long long inc = warp_scan64(sum, lane);
      const uint32_t hit = __ballot_sync(~0u, run + inc > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          long long at = run + inc - sum;
          int e = 0;
#pragma unroll
          for (int n = 0; n < 3; ++n)
            if (e == n && at + v[n] <= target) {
              at += v[n];
              e = n + 1;
            }
          const int id = i0 + 128 * k + 4 * lane + e;
          if (VT_CHECKED(id < a.V)) out[acc] = id;
        }
        return;
      }
      run += __shfl_sync(~0u, inc, 31);
    }
  }
}

// The largest cluster (a power of two) that the device can hold, asked once: where
// SMs are shared out or missing, 16 free ones may not lie together.
vt_status largest_cluster(const DeviceInfo& di, int* largest) {
  static std::atomic<int> known[64];
  std::atomic<int>& k = known[di.device & 63];
  *largest = k.load();
  if (*largest > 0) return VT_OK;
  cudaError_t e =
      cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess)
    return fail(VT_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
  for (*largest = kMaxCluster; *largest > 1; *largest /= 2) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = *largest;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)*largest);
    cfg.blockDim = dim3(kThreads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int active = 0;
    e = cudaOccupancyMaxActiveClusters(&active, verify_kernel, &cfg);
    if (e == cudaSuccess && active > 0) break;
    if (e != cudaSuccess) (void)cudaGetLastError();
  }
  k.store(*largest);
  return VT_OK;
}

}  // namespace
}  // namespace vt

extern "C" vt_status vt_verify_draft(const int32_t* draft_ids, const int32_t* n_draft, int32_t B,
                                     int32_t K, int32_t V, const float* p, int64_t p_seq,
                                     int64_t p_pos, const float* q, int64_t q_seq, int64_t q_pos,
                                     int32_t Vq, const int32_t* f2t, const float* u,
                                     int32_t* n_accepted, int32_t* out_ids, void* stream) {
  using namespace vt;
  if (B < 0 || K < 0 || V < 1 || Vq < 0)
    return fail(VT_ERR_INVALID_ARG, "vt_verify_draft: need B >= 0, K >= 0, V >= 1, Vq >= 0");
  if (V > kMaxV || B > 65535 || K > 65535)
    return fail(VT_ERR_UNSUPPORTED, "vt_verify_draft: V > 2^19, or B or K > 65535");
  if (!f2t && K > 0 && Vq != V)
    return fail(VT_ERR_INVALID_ARG, "vt_verify_draft: without f2t, q must have V columns");
  if (B == 0) return VT_OK;
  if (!p || !u || !n_accepted || !out_ids || (K > 0 && (!draft_ids || (!q && Vq > 0))))
    return fail(VT_ERR_INVALID_ARG, "vt_verify_draft: null pointer");
  if (p_seq < 0 || p_pos < 0 || q_seq < 0 || q_pos < 0 || (K > 0 && p_pos < V) ||
      (K > 1 && q_pos < Vq))
    return fail(VT_ERR_INVALID_ARG, "vt_verify_draft: a row stride is below the row's length");
  if (!aligned(p, 4) || !aligned(q, 4) || !aligned(u, 4) || !aligned(f2t, 4) ||
      !aligned(draft_ids, 4) || !aligned(n_draft, 4) || !aligned(n_accepted, 4) ||
      !aligned(out_ids, 4))
    return fail(VT_ERR_INVALID_ARG, "vt_verify_draft: misaligned pointer");
  const int64_t BK = (int64_t)B * K;
  if (outputs_overlap({{n_accepted, 4ll * B}, {out_ids, 4 * (BK + B)}},
                      {{draft_ids, 4 * BK}, {n_draft, 4ll * B}, {u, 4 * (BK + B)},
                       {f2t, 4ll * V}, rows_range(p, B, p_seq, K * p_pos + V, 4),
                       rows_range(K > 0 ? q : nullptr, B, q_seq, (K - 1) * q_pos + Vq, 4)}))
    return fail(VT_ERR_INVALID_ARG, "vt_verify_draft: an output overlaps an input or the other");
  DeviceInfo di;
  if (!current_device(&di)) return VT_ERR_CUDA;
  int largest;
  const vt_status st = largest_cluster(di, &largest);
  if (st != VT_OK) return st;
  const int C = verify_ctas(B, V, di.num_sms, largest);
  VerifyArgs a;
  a.draft = draft_ids;
  a.n_draft = n_draft;
  a.K = K;
  a.V = V;
  a.Vq = Vq;
  a.seg = (V + C * kWarps - 1) / (C * kWarps);
  a.seg = (a.seg + 127) / 128 * 128;
  a.p = p;
  a.p_seq = p_seq;
  a.p_pos = p_pos;
  a.q = q;
  a.q_seq = q_seq;
  a.q_pos = q_pos;
  a.f2t = f2t;
  a.u = u;
  a.accepted = n_accepted;
  a.out = out_ids;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel, a);
  if (e != cudaSuccess)
    return fail(VT_ERR_CUDA, std::string("verify_kernel: ") + cudaGetErrorString(e));
  return launch_status("verify_kernel");
}
