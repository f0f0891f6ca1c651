// vt_matmul_i8, many rows of X: tensor cores (tcgen05).
//
//   y[m][n] = float(sum_k X[m][k] * W[n][k]) * (xs[m] * ws[n]) + bias[n]
//
// sm_103a's tensor cores have no 8-bit integer kind at a useful rate, but
// 8-bit integers are fp16 numbers, and sums of their products are exact in the
// fp32 accumulator up to 2^24.  A byte of W becomes fp16 without arithmetic:
// w + 128, an unsigned byte u, as the bits of an fp16 is the subnormal u * 2^-24
// (one LOP3 for two values).  X's bytes become fp16 by a byte permute and a
// subtraction.  So the MMA sums u * x * 2^-24; after 512 terms (512 * 255 * 128
// < 2^24) the accumulator is read out, converted and added to 32-bit integers
// in registers, and 128 * sum_k x is taken away at the end.  The sums are exact
// for every input, as dp4a's are.
//
// W's rows are the MMA's M side (128 lanes), the rows of X its N side.  Per
// CTA, persistent over tiles of up to 256 rows of W:
//   warp 0      streams stages of 128 k (the rows' bytes, X's bytes) by TMA;
//   warps 8-23  turn W's bytes into fp16 in tensor memory, the MMA's A operand
//               (a thread is a row), so the doubled bytes never pass through
//               shared memory; two sets of eight warps take turns at stages,
//               because a stage's chain of wait, load, convert, store and
//               signal is longer than its share of the stream;
//   warps 4-7   turn X's bytes into fp16 in shared memory, the B operand (with
//               one MMA a tile, warps 8-15 suffice for W and 16-19 help here);
//   warp 1      issues the MMAs;
//   warps 24-31 read finished accumulators and keep the integer sums (64 a
//               thread: registers are moved to them from the other warps).
// Tiles of W are cut so that every SM gets the same number of rows (a multiple
// of 8, not of 128): up to about 100 rows of X the product is bound by
// reading W once, which needs all SMs, while unused lanes of the MMA cost
// nothing.  Two 128-row MMAs share each converted block of X while the
// accumulators allow (up to 64 rows of X); more rows of X than 128 are taken
// in blocks, the tile of W being read again from L2.  Few rows of W are cut into
// tiles of 128 all the same, and the CTAs of a cluster share a tile's k: each
// sends its sums to the CTA that has their rows of X, which adds them up.
//
// What bounds it (N = 32768, d = 4096: M = 16 29.5 us, 4.6 TB/s; M = 60 37.3 us,
// 3.8 TB/s, 0.56 of the measured copy): the chain of a stage, whose bytes are
// converted, multiplied and its place freed in some 3000 clocks with three
// stages under way.  With 128 rows of X and more (N = 128256, d = 2048: M = 128
// 94 us, 720 TFLOP/s; M = 256 185 us) the same chain, longer by X's bytes, which
// pass through shared memory four times (in, out, back as fp16, to the MMA).  Measured and not used: 64 k a
// stage (M = 60: 50 us), tensor loads ahead of the ring into L2 (34 to 37 us
// where streaming alone took 29), stores of 16 columns to tensor memory and W
// loaded before its place is free (no change), a ring of its own for X (M = 60
// 36.6 us, but M = 256 188 to 250).
//
// Waits on mbarriers are bounded; one that gives up records VT_ERR_TIMEOUT in
// the error word and ends the CTA's other roles too; the loads and MMAs that the
// CTA has issued are waited for before it frees its TMEM and leaves.
#include <cudaTypedefs.h>

#include <mutex>

#include "cluster.cuh"
#include "matmul_i8.cuh"
#include "tc_ptx.cuh"

namespace vt {
namespace {

constexpr int kThreads = 1024;
constexpr int kConvB0 = 4;   // four warps convert X,
constexpr int kConvA0 = 8;   // sixteen W; with one MMA a tile eight W, four
constexpr int kConvB1 = 16;  // more X, and four have nothing to do
constexpr int kEpi0 = 24, kEpiWarps = 8;
// Registers a thread: 6 * 128 * 48 + 2 * 128 * 112 = 1024 * 64.
constexpr int kRegsEpi = 112, kRegsOther = 48;
constexpr int kStageK = 128;     // bytes of a row per stage, one swizzle row
constexpr int kChunkStages = 4;  // 512 k: the accumulator stays exact
constexpr int kMaxStages = 8;
constexpr int kMaxConv = 8;
constexpr int kBlockM = 128;     // rows of X per block at most
constexpr int kMaxRows = 1024;   // rows of X per launch
constexpr int kMaxBlocks = kMaxRows / kBlockM;
constexpr long long kWaitBudget = 2000000000LL;  // clocks

// What the epilogue needs of a row of X: -128 times the sum of its bytes, and
// its scale.
struct __align__(8) RowInfo {
  int shift;
  float scale;
};

struct I8TcArgs {
  I8Args g;
  int rt;       // rows of W per tile, a multiple of 8
  int subs;     // 128-row MMAs per tile (1 or 2)
  int nt;       // rows of X per block, a multiple of 16
  int ntc;      // TMEM columns of one accumulator, a multiple of 32
  int acol;     // first TMEM column of the A operand
  int mblocks;
  int ntiles, nk;
  int splits, per;  // CTAs that share a tile's k, and the stages of each
  int stages, conv, accs;  // raw stages, converted buffers, accumulators
  unsigned* err;
  long long budget;  // kShort: clocks after which a wait gives up
};

__device__ __forceinline__ void tmem_st_32x32_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor: fp32 accumulator, fp16 A and B, both K-major.
__device__ __forceinline__ uint32_t idesc_f16(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
}

// True in one lane of a full warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// mbarrier.try_wait with a hint of how long the thread may sleep in it (ns):
// polls cost issue slots that the converting warps need.
__device__ __forceinline__ bool try_wait_hint(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// mbarrier.test_wait, which never sleeps.
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait that also gives up once another role has.  Warps whose lanes
// go on together vote on its result.  With kShort it gives up after `budget`
// clocks and never sleeps.
template <bool kShort>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         long long budget) {
  auto done = [&]() { return kShort ? test_wait(bar, parity) : try_wait_hint(bar, parity); };
  if (done()) return true;
  const long long t0 = clock64();
  while (!done()) {
    if (*abort) return false;
    if (clock64() - t0 > (kShort ? budget : kWaitBudget)) return false;
  }
  return true;
}
__device__ __forceinline__ void give_up(unsigned* err, volatile int* abort) {
  *abort = 1;
  atomicExch(err, (unsigned)VT_ERR_TIMEOUT);
}

// A ring position: index and the parity of its phase.
struct Ring {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      ph ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(int n) {  // two on, n >= 2
    i += 2;
    if (i >= n) {
      i -= n;
      ph ^= 1u;
    }
  }
};

// kSplit, for few rows of W: a cluster's CTAs share a tile's k (one CTA may be
// all of it), and blocks of X have CTAs of their own (blockIdx.y; mblocks is 1).
// kShort, for the self-test: waits of a.budget clocks (as a run-time limit in every
// launch it cost 3 to 5 %: 256 x 128256 x 2048 190 to 199 us).
template <bool kSplit, bool kShort>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_i8_tc_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmX, I8TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t raw_full[kMaxStages], raw_empty[kMaxStages];
  __shared__ __align__(8) uint64_t cv_full[kMaxConv], cv_empty[kMaxConv];
  __shared__ __align__(8) uint64_t d_full[2], d_empty[2], drain, rows_full[kMaxBlocks];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag;
  __shared__ int loads;  // stages whose loads have been issued

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's tiles, and its stages of each
  const int splits = kSplit ? a.splits : 1, rank = (int)blockIdx.x % splits;
  const int tile0 = (int)blockIdx.x / splits, tiles = (int)gridDim.x / splits;
  const int m_base = kSplit ? (int)blockIdx.y * a.nt : 0;
  const int kb0 = kSplit ? rank * a.per : 0, nk = kSplit ? min(a.per, a.nk - kb0) : a.nk;
  const int a_bytes = a.rt * kStageK, x_bytes = a.nt * kStageK;
  const int stage_bytes = a_bytes + x_bytes;
  uint8_t* bbuf = smem + a.stages * stage_bytes;  // converted X: 2 atoms of 64 k each
  const int b_bytes = a.nt * kStageK * 2;
  RowInfo* rows = reinterpret_cast<RowInfo*>(bbuf + a.conv * b_bytes);  // [mblocks][nt]
  // with splits: the sums of this CTA's part of the rows of X, from each CTA
  const int mine = a.nt / splits;
  int* parts = reinterpret_cast<int*>(rows + a.mblocks * a.nt);  // [splits][mine][rt]

  // warps of a set (every second stage) that convert X, and all of a set
  const int xw = a.subs == 2 ? 2 : 4;
  const uint32_t set_warps = (uint32_t)(4 * a.subs + xw);

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      tc::mbar_init(&raw_full[s], 1);
      tc::mbar_init(&raw_empty[s], set_warps);
    }
    for (int b = 0; b < a.conv; ++b) {
      tc::mbar_init(&cv_full[b], set_warps);
      tc::mbar_init(&cv_empty[b], 1);
    }
    for (int b = 0; b < a.accs; ++b) {
      tc::mbar_init(&d_full[b], 1);
      tc::mbar_init(&d_empty[b], kEpiWarps);
    }
    tc::mbar_init(&drain, 1);
    for (int b = 0; b < a.mblocks; ++b) tc::mbar_init(&rows_full[b], 2 * xw);
    abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&tmW);
    tc::prefetch_tensormap(&tmX);
  }
  for (int m = threadIdx.x; m < a.mblocks * a.nt; m += kThreads) rows[m].shift = 0;
  auto await = [&](uint64_t* bar, uint32_t parity) {
    return wait_bar<kShort>(bar, parity, &abort_flag, a.budget);
  };
  auto load_stage = [&](int s, int tile, int mb, int kb) {
    uint8_t* st = smem + s * stage_bytes;
    tc::mbar_arrive_expect_tx(&raw_full[s], (uint32_t)stage_bytes);
    tc::tma_load_2d(st, &tmW, &raw_full[s], (kb0 + kb) * kStageK, tile * a.rt);
    tc::tma_load_2d(st + a_bytes, &tmX, &raw_full[s], (kb0 + kb) * kStageK, m_base + mb * a.nt);
  };
  const int filled = min(a.stages, nk);
  if (warp == 1) tc::tmem_alloc(&tmem_base, 512);
  // Everything read here may have been written by the kernel ahead (weights
  // too), so nothing is loaded before it has ended; then the producer fills
  // the stages while the others set up.
  if (threadIdx.x == 0) {
    grid_launch_dependents();
    grid_dependency_wait();
    for (int kb = 0; kb < filled; ++kb) load_stage(kb, tile0, 0, kb);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_base;
  if (splits > 1) cl::arrive();  // waited for before another CTA's memory is written
  grid_dependency_wait();

  // (the register counts are set inside each role's branch: the compiler
  // takes the smaller one where branches meet)
  if (warp < kConvB0) {
    give_registers();
    if (warp == 0) {
      if (lane == 0) {  // ------------------------------------ TMA producer
        Ring r;
        int issued = 0;
        bool ok = true;
        for (int tile = tile0; ok && tile < a.ntiles; tile += tiles)
          for (int mb = 0; ok && mb < a.mblocks; ++mb)
            for (int kb = 0; kb < nk; ++kb) {
              if (issued >= filled) {
                if (!await(&raw_empty[r.i], r.ph ^ 1u)) {
                  ok = false;
                  break;
                }
                load_stage(r.i, tile, mb, kb);
              }
              ++issued;
              r.next(a.stages);
            }
        if (!ok) give_up(a.err, &abort_flag);
        loads = issued;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------- MMA issuer
      // The whole warp walks the loop, so that operands stay in uniform
      // registers, and one elected lane issues.
      const uint32_t idesc = idesc_f16(a.nt);
      const uint64_t b0 = tc::sdesc_k_sw128(tc::smem_u32(bbuf));
      Ring c, d;
      bool ok = true;
      for (int tile = tile0; ok && tile < a.ntiles; tile += tiles)
        for (int mb = 0; ok && mb < a.mblocks; ++mb)
          for (int kb = 0; kb < nk; ++kb) {
            const bool first = kb % kChunkStages == 0;
            const bool last = kb % kChunkStages == kChunkStages - 1 || kb == nk - 1;
            if (!__all_sync(~0u, (!first || await(&d_empty[d.i], d.ph ^ 1u)) &&
                                     await(&cv_full[c.i], c.ph))) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint32_t at = tmem + (uint32_t)(a.acol + c.i * a.subs * (kStageK / 2));
            const uint32_t dt = tmem + (uint32_t)(d.i * a.subs * a.ntc);
            const uint64_t bd = b0 + (uint64_t)((uint32_t)(c.i * b_bytes) >> 4);
            const uint64_t bd1 = bd + (uint64_t)((uint32_t)x_bytes >> 4);
            if (elect_one()) {
              const uint32_t more = first ? 0u : 1u;
  #pragma unroll
              for (int j = 0; j < kStageK / 16; ++j)
                mma_f16_ta(dt, at + 8u * j, (j < 4 ? bd : bd1) + 2 * (j & 3), idesc,
                           j > 0 ? 1u : more);
              if (a.subs == 2) {
  #pragma unroll
                for (int j = 0; j < kStageK / 16; ++j)
                  mma_f16_ta(dt + a.ntc, at + kStageK / 2 + 8u * j,
                             (j < 4 ? bd : bd1) + 2 * (j & 3), idesc, j > 0 ? 1u : more);
              }
              tc::mma_commit(&cv_empty[c.i]);
              if (last) tc::mma_commit(&d_full[d.i]);
            }
            __syncwarp();
            c.next(a.conv);
            if (last) d.next(a.accs);
          }
      if (!ok && lane == 0) give_up(a.err, &abort_flag);
      __syncwarp();
    }
  } else if (warp >= kConvA0 && warp < kConvA0 + 8 * a.subs) {
    give_registers();
    // ------------------------------------------- W: bytes to fp16 in TMEM
    // set u takes every second stage, four warps (a quadrant of lanes each)
    // for each 128-row MMA
    const int q = warp & 3, sub = ((warp - kConvA0) >> 2) % a.subs;
    const int u = (warp - kConvA0) / (4 * a.subs);
    const bool any = sub * 128 + 32 * q < a.rt;
    const int row = min(sub * 128 + 32 * q + lane, a.rt - 1);  // of the tile
    const int x = row & 7;
    const int total = (a.ntiles - tile0 + tiles - 1) / tiles * a.mblocks * nk;
    Ring r, c;
    if (u) {
      r.next(a.stages);
      c.next(a.conv);
    }
    bool ok = true;
    for (int i = u; i < total; i += 2) {
      // The converted place first.  The sets take turns at a stage's place when
      // the places are odd in number, and a parity cannot tell phase k - 2 from
      // phase k: with the place of stage i - conv free again, every stage up to
      // that one (of this place too) has landed, so the bytes' phase is the one
      // waited for.  In the other order a stage could be read before it lay there.
      if (!__all_sync(~0u, await(&cv_empty[c.i], c.ph ^ 1u) &&
                               await(&raw_full[r.i], r.ph))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      if (any) {
        const uint4* src =
            reinterpret_cast<const uint4*>(smem + r.i * stage_bytes + row * kStageK);
        const uint32_t dst = tmem + ((uint32_t)(32 * q) << 16) +
                             (uint32_t)(a.acol + (c.i * a.subs + sub) * (kStageK / 2));
        uint4 v[4];
        auto load = [&](int ch) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = src[(ch + e) ^ x];
        };
        auto put = [&](uint32_t col) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h[8];
            w_to_f16(v[e].x, h[0], h[1]);
            w_to_f16(v[e].y, h[2], h[3]);
            w_to_f16(v[e].z, h[4], h[5]);
            w_to_f16(v[e].w, h[6], h[7]);
            tmem_st_32x32_x8(dst + col + 8 * e, h);
          }
        };
        load(0);
        put(0);
        load(4);
        put(32);
        tmem_st_wait();
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&cv_full[c.i]);
        tc::mbar_arrive(&raw_empty[r.i]);
      }
      c.skip(a.conv);  // the other set's stage
      r.skip(a.stages);
    }
    if (!ok && lane == 0) give_up(a.err, &abort_flag);
  } else if (warp < kConvA0 || (a.subs == 1 && warp >= kConvB1 && warp < kConvB1 + 4)) {
    give_registers();
    // --------------------------------- X: bytes to fp16 in shared memory
    // and the rows' sums of bytes, on the CTA's first tile.  Two sets of xw
    // warps take turns at stages; a warp takes 8 / xw chunks of 16 k
    const int bw = warp < kConvA0 ? warp - kConvB0 : warp - kConvB1 + 4;
    const int u = bw & 1, ch0 = (bw >> 1) * (8 / xw);
    Ring r, c;
    if (u) {
      r.next(a.stages);
      c.next(a.conv);
    }
    bool ok = true;
    int kb = u;  // this set's next stage, counted from the block's first
    for (int tile = tile0; ok && tile < a.ntiles; tile += tiles)
      for (int mb = 0; ok && mb < a.mblocks; ++mb) {
        const bool first = tile == tile0;
        int sum[kBlockM / 32] = {};
        for (; kb < nk; kb += 2) {
          if (!__all_sync(~0u, await(&cv_empty[c.i], c.ph ^ 1u) &&
                                   await(&raw_full[r.i], r.ph))) {  // (as W's warps do)
            ok = false;
            break;
          }
          const uint4* src = reinterpret_cast<const uint4*>(smem + r.i * stage_bytes + a_bytes);
          const uint32_t dst = tc::smem_u32(bbuf + c.i * b_bytes);
#pragma unroll
          for (int e = 0; e < kBlockM / 32; ++e) {
            if (32 * e >= a.nt) break;
            const int row = lane + 32 * e;
            const uint32_t x = row & 7;
            if (row < a.nt)
              for (int ch = ch0; ch < ch0 + 8 / xw; ch += 2) {
                uint4 v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  v[h] = src[row * (kStageK / 16) + ((ch + h) ^ x)];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t f[8];
                  x_to_f16(v[h].x, f[0], f[1]);
                  x_to_f16(v[h].y, f[2], f[3]);
                  x_to_f16(v[h].z, f[4], f[5]);
                  x_to_f16(v[h].w, f[6], f[7]);
                  const int o = ch + h;  // its two chunks of the fp16 atom
                  const uint32_t d0 = dst + (o >> 2) * x_bytes + row * 128;
                  sts128(d0 + (((2 * (o & 3)) ^ x) << 4), f[0], f[1], f[2], f[3]);
                  sts128(d0 + (((2 * (o & 3) + 1) ^ x) << 4), f[4], f[5], f[6], f[7]);
                  if (first) {
                    sum[e] = __dp4a((int)v[h].x, 0x01010101, sum[e]);
                    sum[e] = __dp4a((int)v[h].y, 0x01010101, sum[e]);
                    sum[e] = __dp4a((int)v[h].z, 0x01010101, sum[e]);
                    sum[e] = __dp4a((int)v[h].w, 0x01010101, sum[e]);
                  }
                }
              }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(&cv_full[c.i]);
            tc::mbar_arrive(&raw_empty[r.i]);
          }
          c.skip(a.conv);  // the other set's stage
          r.skip(a.stages);
        }
        kb -= nk;
        if (first && ok) {
#pragma unroll
          for (int e = 0; e < kBlockM / 32; ++e) {
            const int row = lane + 32 * e, m = mb * a.nt + row;
            if (row < a.nt) {
              atomicAdd(&rows[m].shift, -128 * sum[e]);
              if (bw == 0)
                rows[m].scale = m_base + m < a.g.M ? __ldg(a.g.xs + m_base + m) : 0.f;
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&rows_full[mb]);
        }
      }
    if (!ok && lane == 0) give_up(a.err, &abort_flag);
  } else if (warp < kEpi0) {
    give_registers();  // warps without work
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // ------------------------------------------------------- epilogue
    const int q = warp & 3, part = (warp - kEpi0) >> 2;
    const int sub = a.subs == 2 ? part : 0;
    const int col0 = a.subs == 2 ? 0 : 64 * part;  // this warp's columns: 64
    const int trow = sub * 128 + 32 * q + lane;
    const bool any = col0 < a.nt && sub * 128 + 32 * q < a.rt;
    Ring d;
    bool ok = true;
    for (int tile = tile0; ok && tile < a.ntiles; tile += tiles)
      for (int mb = 0; ok && mb < a.mblocks; ++mb) {
        const int m0 = mb * a.nt + col0;
        int acc[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0;
        for (int kb = 0; kb < nk; kb += kChunkStages) {
          if (!__all_sync(~0u, await(&d_full[d.i], d.ph))) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          if (any) {
            const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) +
                               (uint32_t)((d.i * a.subs + sub) * a.ntc + col0);
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
              if (col0 + 16 * h < a.nt) {
                // two loads in flight
                float v0[16], v1[16];
                const bool two = col0 + 16 * h + 16 < a.nt;
                tc::tmem_ld_32x32_x16(t + 16u * h, v0);
                if (two) tc::tmem_ld_32x32_x16(t + 16u * h + 16u, v1);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[16 * h + j] += __float2int_rn(v0[j] * 0x1p24f);
                if (two) {
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    acc[16 * h + 16 + j] += __float2int_rn(v1[j] * 0x1p24f);
                }
              }
            }
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&d_empty[d.i]);
          d.next(a.accs);
        }
        if (ok && !__all_sync(~0u, await(&rows_full[mb], 0u))) ok = false;
        if (splits > 1) {
          // every CTA's sums to the CTA that has their rows of X, which adds
          // them up (each warp of the cluster passes the barrier, whatever
          // became of it)
          cl::wait();
          if (ok && any && trow < a.rt) {
            int to = col0 / mine, at = col0 % mine;
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              if (col0 + j < a.nt) {
                cl::st_u32(cl::map(parts + (rank * mine + at) * a.rt + trow, to),
                           (uint32_t)(acc[j] + rows[col0 + j].shift));
                if (++at == mine) {
                  at = 0;
                  ++to;
                }
              }
            }
          }
          cl::sync();
          // (a thread has a row of W, or two, and every second of this CTA's
          // rows of X)
          for (int row = 32 * q + lane; ok && row < a.rt; row += 128) {
            const int n = tile * a.rt + row;
            if (n >= a.g.N) break;
            const float ws = __ldg(a.g.ws + n);
            const float b = a.g.bias ? __ldg(a.g.bias + n) : 0.f;
            const int last = min(mine, a.g.M - m_base - rank * mine);
#pragma unroll 4
            for (int i = part; i < last; i += 2) {
              int sum = 0;
              for (int c = 0; c < splits; ++c) sum += parts[(c * mine + i) * a.rt + row];
              const int m = rank * mine + i;
              i8_store(a.g, (m_base + m) * a.g.ldo + n, sum, rows[m].scale, ws, b);
            }
          }
          continue;
        }
        if (!ok || !any) continue;
        const int n = tile * a.rt + trow;
        const int cols = min(min(64, a.nt - col0), a.g.M - m_base - m0);
        if (trow < a.rt && n < a.g.N) {
          const float ws = __ldg(a.g.ws + n);
          const float b = a.g.bias ? __ldg(a.g.bias + n) : 0.f;
          const RowInfo* info = rows + m0;
          const int64_t at = (int64_t)(m_base + m0) * a.g.ldo + n;
          // eight columns at a time, so that their latencies overlap (a row's
          // info exists up to nt, a multiple of 16)
#pragma unroll
          for (int g = 0; g < 64; g += 8) {
            if (g < cols) {
              RowInfo t[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) t[j] = info[g + j];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (g + j < cols)
                  i8_store(a.g, at + (g + j) * a.g.ldo, acc[g + j] + t[j].shift, t[j].scale, ws, b);
            }
          }
        }
      }
    if (!ok && lane == 0) give_up(a.err, &abort_flag);
  }

  if (splits > 1 && warp < kEpi0) {
    cl::wait();
    cl::sync();
  }
  __syncthreads();
  if (abort_flag) {
    // Some role gave up, whichever it was: loads and MMAs that nobody has waited
    // for may still be under way.  The last load of each stage, and all MMAs: a
    // commit covers the work of the thread that makes it, and elect.sync names
    // the same lane every time.
    if (threadIdx.x == 0)
      for (int i = loads - min(loads, a.stages); i < loads; ++i)
        tc::mbar_wait(&raw_full[i % a.stages], (uint32_t)(i / a.stages) & 1u, kWaitBudget);
    if (warp == 1) {
      if (elect_one()) {
        tc::mma_commit(&drain);
        tc::mbar_wait(&drain, 0u, kWaitBudget);
      }
      __syncwarp();
    }
  }
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// rows x d bytes, box of 128 bytes x box_rows, 128-byte swizzle, zero fill.
bool byte_map(CUtensorMap* map, const void* base, int rows, int d, int box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d};
  const cuuint32_t box[2] = {(cuuint32_t)kStageK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Clusters of `c` CTAs of the kernel that the device holds at a time; asked once.
static int resident_clusters(int c, const DeviceInfo& di) {
  static std::mutex mu;
  static int known[64][4] = {};
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[di.device & 63][c / 4 + 1];
  if (n == 0) {
    cudaFuncAttributes fa;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(kThreads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int active = 0;
    if (cudaFuncGetAttributes(&fa, matmul_i8_tc_kernel<true, false>) != cudaSuccess) return 0;
    cfg.dynamicSmemBytes = di.max_smem_optin - fa.sharedSizeBytes;
    if (cudaOccupancyMaxActiveClusters(&active, matmul_i8_tc_kernel<true, false>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    n = active > 0 ? active : -1;
  }
  return n;
}

static vt_status launch_tc(const I8Args& g, unsigned* err, long long budget, const DeviceInfo& di,
                           cudaStream_t s) {
  if (!allow_max_smem(matmul_i8_tc_kernel<false, false>, di) ||
      !allow_max_smem(matmul_i8_tc_kernel<true, false>, di) ||
      (budget && (!allow_max_smem(matmul_i8_tc_kernel<false, true>, di) ||
                  !allow_max_smem(matmul_i8_tc_kernel<true, true>, di))))
    return VT_ERR_CUDA;
  I8TcArgs a;
  a.g = g;
  a.err = err;
  a.budget = budget;
  a.mblocks = (g.M + kBlockM - 1) / kBlockM;
  a.nt = ((g.M + a.mblocks - 1) / a.mblocks + 15) / 16 * 16;
  a.ntc = (a.nt + 31) / 32 * 32;
  a.nk = (g.d + kStageK - 1) / kStageK;
  // Where tiles of 128 rows do not fill the SMs, the CTAs of a cluster share a
  // tile's k, since a stage takes its time however few rows it has (M = 60,
  // d = 4096: N = 1000 22.5 us alone, 11.6 split in 8; N = 4096 22.4, 15.1 in 4;
  // N = 8192 23.2, 20.6 in 2).  The sums' meeting costs 2 to 3 us, which short
  // rows do not give back (d = 1024: N = 4096 10.6 alone, 11.3 in 4, 13.5 in 2).
  const int blocks = a.mblocks, sms = di.num_sms;
  const int tiles = (g.N + 127) / 128;
  a.splits = 1;
  a.per = a.nk;
  int ways = sms;  // tiles at a time
  bool few = false;
  for (int c = 8; c > 1 && !few; c /= 2) {
    const int w = a.nk >= (c > 2 ? 12 : 24) ? resident_clusters(c, di) / blocks : 0;
    const int per = (a.nk + c - 1) / c;
    if (tiles <= w && (c - 1) * per < a.nk) {
      few = true;
      a.splits = c;
      a.per = per;
      ways = w;
    }
  }
  if (!few && blocks > 1) {
    // Blocks of X on CTAs of their own, by how often a CTA goes through k: side
    // by side, and in turn with each tile of W read once (d = 4096: M = 256,
    // N = 4096 31.7 and 55.2 us; M = 1024, N = 9000 126 and 209; at twice as
    // often in turn and more it is never slower).
    const int64_t beside = ((int64_t)tiles * blocks + sms - 1) / sms;
    const int64_t turns = (tiles + sms - 1) / sms * (int64_t)blocks;
    few = 2 * beside <= turns;
    if (few) ways = std::max(sms / blocks, tiles);
  }
  if (few) a.mblocks = 1;
  // Rows per tile: as many as the waves need, the same for every SM; two MMAs a
  // tile where the accumulators allow (N = 32768, d = 4096: M = 60 37.3 us, 41.3
  // with one; M = 16 29.5 and 36.9).
  const int cap = a.nt <= 64 ? 256 : 128;
  const int waves = (int)(((int64_t)g.N + (int64_t)cap * ways - 1) / ((int64_t)cap * ways));
  const int want = (int)(((int64_t)g.N + (int64_t)waves * ways - 1) / ((int64_t)waves * ways));
  a.rt = std::min(cap, (want + 7) / 8 * 8);
  a.subs = a.rt > 128 ? 2 : 1;
  a.ntiles = (g.N + a.rt - 1) / a.rt;
  // Two accumulators of the tile, so that one is read while the next is
  // summed, and as many A operands as the other columns hold, up to three.
  // Two 128-row accumulators of 64 columns leave room for two operands only:
  // then a third operand hides the reading better than a second accumulator
  // (M = 60, N = 32768, d = 4096: 36.8 us against 38.4).
  a.accs = a.subs == 2 && a.nt > 32 ? 1 : 2;
  a.acol = a.accs * a.subs * a.ntc;
  a.conv = std::min(3, (512 - a.acol) / (a.subs * (kStageK / 2)));
  const int stage_bytes = (a.rt + a.nt) * kStageK;
  // converted X and what the epilogue needs of its rows, after the stages
  const int b_bytes = a.conv * a.nt * kStageK * 2 + a.mblocks * a.nt * (int)sizeof(RowInfo) +
                      (a.splits > 1 ? a.nt * a.rt * 4 : 0);
  a.stages = std::min(kMaxStages, (di.max_smem_optin - 2048 - b_bytes) / stage_bytes);
  // (the converting warps' waits rely on a.conv <= a.stages, or two stages)
  if (a.stages < 2) return fail(VT_ERR_UNSUPPORTED, "vt_matmul_i8: stages do not fit");
  CUtensorMap tmW, tmX;
  if (!byte_map(&tmW, g.W, g.N, g.d, a.rt) || !byte_map(&tmX, g.X, g.M, g.d, a.nt))
    return fail(VT_ERR_CUDA, "vt_matmul_i8: cuTensorMapEncodeTiled failed");
  auto kernel = budget ? (few ? matmul_i8_tc_kernel<true, true> : matmul_i8_tc_kernel<false, true>)
                       : few ? matmul_i8_tc_kernel<true, false>
                             : matmul_i8_tc_kernel<false, false>;
  const int grid = std::min(a.ntiles, ways) * a.splits;
  const size_t smem = (size_t)a.stages * stage_bytes + b_bytes + 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, few ? blocks : 1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, a);
  if (e != cudaSuccess)
    return fail(VT_ERR_CUDA, std::string("matmul_i8_tc_kernel: ") + cudaGetErrorString(e));
  return launch_status("matmul_i8_tc_kernel");
}

vt_status matmul_i8_tc(const I8Args& g, unsigned* err, long long budget, const DeviceInfo& di,
                       cudaStream_t s) {
  for (int m = 0; m < g.M; m += kMaxRows) {
    I8Args p = g;
    p.M = std::min(kMaxRows, g.M - m);
    p.X = g.X + (int64_t)m * g.d;
    p.xs = g.xs + m;
    p.out = static_cast<char*>(g.out) + (int64_t)m * g.ldo * (g.out_bf16 ? 2 : 4);
    const vt_status st = launch_tc(p, err, budget, di, s);
    if (st != VT_OK) return st;
  }
  return VT_OK;
}

}  // namespace vt
