// zo_head.cu -- log probabilities of given tokens and entropy straight from hidden states and
// the head matrix (zo_head_logprobs): for x[r][j] = hidden[r] . W[j],
//
//   lse_r = log sum_j exp(x_rj),  logprob_r = x_{r,t} - lse_r,  H_r = lse_r - sum_j p_rj x_rj,
//
// without the [rows][vocab] logits in memory.  The product runs on the tensor cores as in
// zo_gemm.cu (TMA ring, tcgen05.mma, fp32 accumulators in tensor memory); instead of storing the
// accumulator, the epilogue threads, one row each, keep m (largest logit times log2 e),
// s = sum 2^(x log2 e - m) and u = sum 2^(x log2 e - m) (x log2 e - m) over all columns that
// they see, and write one triple per row at the end.  A second kernel joins a row's triples in a
// fixed order.
//
// Up to 128 rows, one CTA of every SM takes them all and a contiguous range of W's rows in units
// of 32 (so that ranges differ by one unit, not by one tile), 256 at a time; the last tile of a
// range may be narrower (the MMA's N and the number of loaded boxes follow).  More rows run on CTA
// pairs (cta_group::2): 256 rows, each CTA holding 128 of them and half of W's tile, which takes two
// thirds of the shared-memory traffic; ranges in units of 64.
#include <algorithm>
#include <cmath>

#include "zo_internal.cuh"
#include "zo_tc.cuh"

namespace zo {
namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994530942;
// 2^t for t below -kLowest (that of a ruled out token's -inf, or of no column) is 0, and so is 2^t t.
constexpr float kLowest = 1e30f;
constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kBox = 32;  // rows of W in one TMA box
constexpr int kEpiWarps = 16;  // 4 for each quarter of a tile's columns: the exponentials need warps to wait for
constexpr int kThreads = 32 * (4 + kEpiWarps);  // loads, MMAs, two idle ones; epilogue
// Registers of a thread: 4 warps x kFew + 16 x kMany = 20 x 96 of the launch.
constexpr int kFew = 32, kMany = 112;
// The tensor cores truncate each addition to an fp32 accumulator: over a width of 2048 the entropy
// came out off by 1.1e-6 and over 4096 by 2.1e-6, where rounded sums give 1e-7 to 9e-7.  So an
// accumulator takes a part of the width, and the epilogue adds accumulators up, rounded: 1024 leave
// 6e-7 at a width of 2048 and 1.7e-6 at 4096 and cost 1% of the time, 512 leave 3e-7 and 8e-7 and cost 3.5%.
__host__ __device__ constexpr int chunk_steps(int width) { return width <= 2048 ? 16 : 8; }  // of 64

template <bool PAIR>
struct HeadCfg {
  static constexpr int kStages = PAIR ? 6 : 4;
  static constexpr int kUnit = PAIR ? 2 * kBox : kBox;  // unit of a range of W's rows
  static constexpr int kRows = PAIR ? 2 * kBM : kBM;    // rows of a CTA or pair
  static constexpr uint32_t kABytes = kBM * kBK * 2;
  static constexpr uint32_t kBBytes = (PAIR ? kBN / 2 : kBN) * kBK * 2;
  static constexpr uint32_t kBoxBytes = kBox * kBK * 2;
  static constexpr uint32_t kBarOffset = kStages * (kABytes + kBBytes);
  static constexpr uint32_t kStatsOffset = kBarOffset + 256;  // RowStats [quarter][128]
  static constexpr uint32_t kBytes = kStatsOffset + (kEpiWarps / 4) * kBM * 24 + 1024;
  static_assert((2 * kStages + 5) * 8 + 8 <= 256, "barrier area");
};

struct HeadArgs {
  int rows, vocab, width;
  int splits;             // ranges of W's rows
  int units;              // of W's rows
  int a_rows;             // rows of a box of `hidden` (a multiple of 8; those behind are not loaded)
  const int32_t *targets; // may be null
  float4 *part;           // [rows][splits] (m, s, u, what s lost to rounding)
  float *target_logit;    // [rows]
  uint32_t *err;
};

// Rows of W of range i: [first, last), whole units except at the end of the vocabulary.
__device__ __forceinline__ int range_first(int i, int units, int splits, int unit) {
  return (int)((int64_t)units * i / splits) * unit;
}

// Statistics of one row over the columns that a thread sees.  m is a whole number, so that a
// larger one rescales by an exact power of two; 32 columns are summed in fp32, in four chains,
// their sums in fp64: one conversion and addition in 32, where fp32 sums over a vocabulary's
// thousands of columns lose three digits more than the products do.
struct RowStats {
  float m = -INFINITY;
  double s = 0.0, u = 0.0;

  // Nothing seen.
  __device__ __forceinline__ bool empty() const { return m == -INFINITY && s == 0.0 && u == 0.0; }
  // These sums relative to `top` (a whole number, m at least), added to (s, u) there.
  __device__ __forceinline__ void add_to(float top, double &ts, double &tu) const {
    if (empty()) return;
    const float d = m == top ? 0.f : m - top;  // (both may be -inf)
    const double e = (double)tc::ex2(d);
    ts += e * s;
    tu += e * (u + (double)d * s);
  }

  __device__ __forceinline__ void take(const float *v) {  // 32 columns
    float x4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < 32; i += 8) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x4[c] = i + 4 < 32 ? tc::max3f(x4[c], v[i + c], v[i + 4 + c]) : fmaxf(x4[c], v[i + c]);
    }
    const float top = ceilf(tc::max3f(x4[0], x4[1], fmaxf(x4[2], x4[3])) * kLog2E);
    if (top > m) {
      if (m != -INFINITY) {
        const float d = m - top;
        const double e = (double)tc::ex2(d);
        u = e * (u + (double)d * s);
        s *= e;
      }
      m = top;
    }
    const float ref = m == -INFINITY ? 0.f : m;  // nothing but -inf so far: 2^-inf = 0
    float s4[4] = {}, u4[4] = {};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float t0, t1;
      tc::fma2_bc(v[i], v[i + 1], kLog2E, -ref, t0, t1);
      t0 = tc::max_nan(t0, -kLowest);
      t1 = tc::max_nan(t1, -kLowest);
      const float p0 = tc::ex2(t0), p1 = tc::ex2(t1);
      const int h = i & 2;
      tc::add2(s4[h], s4[h + 1], p0, p1);
      tc::fma2(u4[h], u4[h + 1], p0, p1, t0, t1);
    }
    s += (double)((s4[0] + s4[1]) + (s4[2] + s4[3]));
    u += (double)((u4[0] + u4[1]) + (u4[2] + u4[3]));
  }
};

static_assert(sizeof(RowStats) == 24, "HeadCfg::kBytes");

// The triple of one row over a CTA's columns, from those of its quarters (kBM apart).
__device__ __forceinline__ void write_part(const HeadArgs &a, const RowStats *quarter, int row, int split) {
  RowStats r;
#pragma unroll
  for (int k = 0; k < kEpiWarps / 4; ++k) r.m = fmaxf(r.m, quarter[k * kBM].m);
#pragma unroll
  for (int k = 0; k < kEpiWarps / 4; ++k) quarter[k * kBM].add_to(r.m, r.s, r.u);
  a.part[(int64_t)row * a.splits + split] = make_float4(r.m, (float)r.s, (float)r.u, (float)(r.s - (double)(float)r.s));
}

// What an epilogue thread does with one accumulator: its row's 64 columns from taddr on, added to x.
__device__ __forceinline__ void add_columns(float (&x)[64], uint32_t taddr, bool first) {
#pragma unroll
  for (int c = 0; c < 64; c += 16) {
    float v[16];
    tc::tmem_ld16(taddr + (uint32_t)c, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[c + i] = first ? v[i] : x[c + i] + v[i];
  }
}

// One row's logits of W's rows n0 .. n0 + 63, of which `cols` exist, into its statistics.
__device__ __forceinline__ void take_columns(RowStats &st, float (&x)[64], int n0, int cols, int target,
                                             float *target_logit) {
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    if (c < cols) {
      const int hit = target - (n0 + c);
      if (__any_sync(0xFFFFFFFFu, hit >= 0 && hit < 32)) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v = i == hit ? x[c + i] : v;
        if (hit >= 0 && hit < min(32, cols - c)) *target_logit = v;
      }
      if (c + 32 > cols) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[c + i] = c + i < cols ? x[c + i] : -INFINITY;
      }
      st.take(x + c);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
head_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, HeadArgs a) {
  using S = HeadCfg<false>;
  constexpr int kStages = S::kStages, kUnit = S::kUnit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem, *sB = smem + kStages * S::kABytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBarOffset);
  uint64_t *empty = full + kStages;
  uint64_t *acc_full = empty + kStages;  // [2]
  uint64_t *acc_empty = acc_full + 2;    // [2]
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  RowStats *stats = reinterpret_cast<RowStats *>(smem + S::kStatsOffset);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int m0 = blockIdx.x * kBM, split = blockIdx.y;
  const int n_first = range_first(split, a.units, a.splits, kUnit);
  const int n_last = min(range_first(split + 1, a.units, a.splits, kUnit), a.vocab);
  const int tiles = (n_last - n_first + kBN - 1) / kBN;
  const int nk = (a.width + kBK - 1) / kBK, chunk = chunk_steps(a.width);
  // loaded rows of a tile: whole units (rows past the vocabulary read as zero and are masked)
  auto tile_units = [&](int t) { return min(kBN / kUnit, (n_last - n_first - t * kBN + kUnit - 1) / kUnit); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], kEpiWarps);
    }
    tc::mbar_init(mma_done, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_holder, 2 * kBN);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  tc::pdl_wait();

  uint32_t issued = 0;
  if (warp < 4) {
    tc::regs_dec<kFew>();
    if (warp == 0 && lane == 0) {
      tc::tma_prefetch_desc(&tmA);
      tc::tma_prefetch_desc(&tmB);
      for (int t = 0; t < tiles && !*abort_flag; ++t) {
        const int boxes = tile_units(t);
        for (int kb = 0; kb < nk; ++kb) {
          const uint32_t s = issued % kStages, ph = (issued / kStages) & 1u;
          if (*abort_flag || !tc::mbar_wait(&empty[s], ph ^ 1u)) {
            atomicOr(a.err, ZO_FLAG_TIMEOUT);
            *abort_flag = 1;
            break;
          }
          tc::mbar_arrive_expect_tx(&full[s], (uint32_t)a.a_rows * kBK * 2 + (uint32_t)boxes * S::kBoxBytes);
          tc::tma_load_2d(sA + s * S::kABytes, &tmA, &full[s], kb * kBK, m0);
          for (int b = 0; b < boxes; ++b)
            tc::tma_load_2d(sB + s * S::kBBytes + b * S::kBoxBytes, &tmB, &full[s], kb * kBK,
                            n_first + t * kBN + b * kUnit);
          ++issued;
        }
      }
      tc::pdl_launch_dependents();  // (the joining kernel, which waits for this one's end at its start)
    } else if (warp == 1) {  // MMAs: the warp in step, one lane issues
      const uint32_t a0 = tc::desc_k128_lo(__shfl_sync(0xFFFFFFFFu, tc::smem_addr(sA), 0));
      const uint32_t b0 = tc::desc_k128_lo(__shfl_sync(0xFFFFFFFFu, tc::smem_addr(sB), 0));
      const uint32_t tm0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      tc::RingPos<kStages> pos;
      uint32_t accs = 0;
      bool ok = true;
      for (int t = 0; ok && t < tiles; ++t) {
        const uint32_t idesc = tc::idesc_bf16_f32(kBM, tile_units(t) * kUnit);
        for (int k0 = 0; ok && k0 < nk; k0 += chunk, ++accs) {
          const uint32_t b = accs & 1u, d = tm0 + b * (uint32_t)kBN;
          ok = tc::warp_wait_fast(&acc_empty[b], ((accs >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          tc::tc_fence_after();
          const int kb_end = min(nk, k0 + chunk);
          for (int kb = k0; kb < kb_end; ++kb) {
            ok = tc::warp_wait_fast(&full[pos.slot], pos.phase, abort_flag);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t al = a0 + (uint32_t)pos.slot * (S::kABytes >> 4), bl = b0 + (uint32_t)pos.slot * (S::kBBytes >> 4);
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)
                tc::mma_bf16_lo(d, al + 2u * k, bl + 2u * k, idesc, kb > k0 || k > 0 ? 1u : 0u);
              tc::mma_commit(&empty[pos.slot]);
              if (kb + 1 == kb_end) tc::mma_commit(&acc_full[b]);
            }
            __syncwarp();
            pos.next();
          }
        }
      }
      if (!ok && lane == 0) {
        atomicOr(a.err, ZO_FLAG_TIMEOUT);
        *abort_flag = 1;
      }
      __syncwarp();
      if (tc::elect_one()) tc::mma_commit(mma_done);  // arrives once every MMA above has retired
    }
  } else {
    tc::regs_inc<kMany>();
    const int q = warp & 3, quarter = (warp - 4) / 4;  // TMEM lane quadrant; quarter of the columns
    const int row = m0 + 32 * q + lane;
    const int target = a.targets && row < a.rows ? a.targets[row] : -1;
    const bool any = m0 + 32 * q < a.rows;  // a warp without a row only passes the accumulators on
    RowStats st;
    bool ok = true;
    uint32_t accs = 0;
    for (int t = 0; ok && t < tiles; ++t) {
      // this warp's columns of the tile
      const int n0 = n_first + t * kBN + quarter * (kBN / 4), cols = min(kBN / 4, n_last - n0);
      float x[64];
      for (int k0 = 0; k0 < nk; k0 += chunk, ++accs) {
        const uint32_t b = accs & 1u;
        if (!tc::warp_wait_fast(&acc_full[b], (accs >> 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (any && cols > 0)
          add_columns(x, tmem + b * kBN + (uint32_t)(quarter * (kBN / 4)) + ((uint32_t)(q * 32) << 16), k0 == 0);
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[b]);
      }
      if (ok && any && cols > 0) take_columns(st, x, n0, cols, target, a.target_logit + row);
    }
    if (!ok && lane == 0) {
      atomicOr(a.err, ZO_FLAG_TIMEOUT);
      *abort_flag = 1;
    }
    stats[quarter * kBM + 32 * q + lane] = st;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (threadIdx.x < kBM && m0 + (int)threadIdx.x < a.rows) write_part(a, stats + threadIdx.x, m0 + threadIdx.x, split);
  if (warp == 0 && lane == 0 && *abort_flag) {
    // let this CTA's TMA loads still in flight land before it exits (bounded)
    for (uint32_t s = 0; s < (uint32_t)kStages; ++s) {
      if (issued <= s) continue;
      const uint32_t last = s + ((issued - 1 - s) / kStages) * kStages;
      if (!tc::mbar_wait(&full[s], (last / kStages) & 1u)) atomicOr(a.err, ZO_FLAG_TIMEOUT);
    }
  }
  if (warp == 1) {
    if (lane == 0 && !tc::mbar_wait(mma_done, 0)) atomicOr(a.err, ZO_FLAG_TIMEOUT);
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 2 * kBN);
  }
}

// The CTA-pair form (tmW: a whole tile's rows of W in one box.  Four boxes of 32 rows a stage, which the
// last tile of a range still takes, held the tensor pipe at 63%: 4096 x 151936 x 2048 took 1950 us, with
// whole boxes 1648): the roles of head_kernel, with the leader (CTA 0) issuing the MMAs of both and
// each CTA's epilogue warps reading the 128 rows of its own tensor memory.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
head_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmW, HeadArgs a) {
  using S = HeadCfg<true>;
  constexpr int kStages = S::kStages, kUnit = S::kUnit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem, *sB = smem + kStages * S::kABytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBarOffset);  // used in the leader
  uint64_t *empty = full + kStages;
  uint64_t *acc_full = empty + kStages;  // [2]
  uint64_t *acc_empty = acc_full + 2;    // [2] used in the leader: both CTAs' epilogue warps
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  RowStats *stats = reinterpret_cast<RowStats *>(smem + S::kStatsOffset);

  const uint32_t rank = tc::cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int m0 = (int)blockIdx.x * kBM, split = blockIdx.y;  // blockIdx.x / 2 is the pair's row tile
  const int n_first = range_first(split, a.units, a.splits, kUnit);
  const int n_last = min(range_first(split + 1, a.units, a.splits, kUnit), a.vocab);
  const int tiles = (n_last - n_first + kBN - 1) / kBN;
  const int nk = (a.width + kBK - 1) / kBK, chunk = chunk_steps(a.width);
  auto tile_units = [&](int t) { return min(kBN / kUnit, (n_last - n_first - t * kBN + kUnit - 1) / kUnit); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    tc::mbar_init(mma_done, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc_pair(tmem_holder, 2 * kBN);
  tc::tc_fence_before();
  tc::cluster_sync();  // both CTAs' barriers initialised and tensor memory allocated
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  tc::pdl_wait();
  const uint32_t full_leader = tc::map_to_rank(full, 0);
  const uint32_t acc_empty_leader = tc::map_to_rank(acc_empty, 0);
  const uint32_t abort_peer = tc::map_to_rank(const_cast<int *>(abort_flag), rank ^ 1u);
  auto raise_abort = [&]() {
    atomicOr(a.err, ZO_FLAG_TIMEOUT);
    *abort_flag = 1;
    tc::st_remote_u32(abort_peer, 1u);
  };

  uint32_t issued = 0;
  if (warp < 4) {
    tc::regs_dec<kFew>();
    if (warp == 0 && lane == 0) {
      tc::tma_prefetch_desc(&tmA);
      tc::tma_prefetch_desc(&tmB);
      tc::tma_prefetch_desc(&tmW);
      for (int t = 0; t < tiles && !*abort_flag; ++t) {
        const int boxes = tile_units(t);  // of each CTA: the tile's W rows split in the middle
        const int b_row = n_first + t * kBN + (int)rank * boxes * kBox;
        for (int kb = 0; kb < nk; ++kb) {
          const uint32_t s = issued % kStages, ph = (issued / kStages) & 1u;
          if (*abort_flag || !tc::mbar_wait(&empty[s], ph ^ 1u)) {
            raise_abort();
            break;
          }
          if (leader) tc::mbar_arrive_expect_tx(&full[s], 2 * (S::kABytes + (uint32_t)boxes * S::kBoxBytes));
          tc::tma_load_2d_pair(sA + s * S::kABytes, &tmA, full_leader + 8u * s, kb * kBK, m0);
          if (boxes == kBN / 2 / kBox)
            tc::tma_load_2d_pair(sB + s * S::kBBytes, &tmW, full_leader + 8u * s, kb * kBK, b_row);
          else for (int b = 0; b < boxes; ++b)
            tc::tma_load_2d_pair(sB + s * S::kBBytes + b * S::kBoxBytes, &tmB, full_leader + 8u * s, kb * kBK,
                                 b_row + b * kBox);
          ++issued;
        }
      }
      tc::pdl_launch_dependents();  // (the joining kernel, which waits for this one's end at its start)
    } else if (warp == 1 && leader) {  // MMAs: the warp in step, one lane issues
      const uint32_t a0 = tc::desc_k128_lo(__shfl_sync(0xFFFFFFFFu, tc::smem_addr(sA), 0));
      const uint32_t b0 = tc::desc_k128_lo(__shfl_sync(0xFFFFFFFFu, tc::smem_addr(sB), 0));
      const uint32_t tm0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      tc::RingPos<kStages> pos;
      uint32_t accs = 0;
      bool ok = true;
      for (int t = 0; ok && t < tiles; ++t) {
        const uint32_t idesc = tc::idesc_bf16_f32(2 * kBM, tile_units(t) * kUnit);
        for (int k0 = 0; ok && k0 < nk; k0 += chunk, ++accs) {
          const uint32_t b = accs & 1u, d = tm0 + b * (uint32_t)kBN;
          ok = tc::warp_wait_fast(&acc_empty[b], ((accs >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          tc::tc_fence_after();
          const int kb_end = min(nk, k0 + chunk);
          for (int kb = k0; kb < kb_end; ++kb) {
            ok = tc::warp_wait_fast(&full[pos.slot], pos.phase, abort_flag);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t al = a0 + (uint32_t)pos.slot * (S::kABytes >> 4), bl = b0 + (uint32_t)pos.slot * (S::kBBytes >> 4);
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)
                tc::mma_bf16_pair_lo(d, al + 2u * k, bl + 2u * k, idesc, kb > k0 || k > 0 ? 1u : 0u);
              tc::mma_commit_pair(&empty[pos.slot]);
              if (kb + 1 == kb_end) tc::mma_commit_pair(&acc_full[b]);
            }
            __syncwarp();
            pos.next();
          }
        }
      }
      if (!ok && lane == 0) raise_abort();
      __syncwarp();
      if (tc::elect_one()) tc::mma_commit_pair(mma_done);  // arrives (in both CTAs) once every MMA above has retired
    }
  } else {
    tc::regs_inc<kMany>();
    const int q = warp & 3, quarter = (warp - 4) / 4;
    const int row = m0 + 32 * q + lane;
    const int target = a.targets && row < a.rows ? a.targets[row] : -1;
    const bool any = m0 + 32 * q < a.rows;
    RowStats st;
    bool ok = true;
    uint32_t accs = 0;
    for (int t = 0; ok && t < tiles; ++t) {
      // this warp's columns of the tile
      const int n0 = n_first + t * kBN + quarter * (kBN / 4), cols = min(kBN / 4, n_last - n0);
      float x[64];
      for (int k0 = 0; k0 < nk; k0 += chunk, ++accs) {
        const uint32_t b = accs & 1u;
        if (!tc::warp_wait_fast(&acc_full[b], (accs >> 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (any && cols > 0)
          add_columns(x, tmem + b * kBN + (uint32_t)(quarter * (kBN / 4)) + ((uint32_t)(q * 32) << 16), k0 == 0);
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) tc::mbar_arrive(&acc_empty[b]);
          else tc::mbar_arrive_remote(acc_empty_leader + 8u * b);
        }
      }
      if (ok && any && cols > 0) take_columns(st, x, n0, cols, target, a.target_logit + row);
    }
    if (!ok && lane == 0) raise_abort();
    stats[quarter * kBM + 32 * q + lane] = st;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (threadIdx.x < kBM && m0 + (int)threadIdx.x < a.rows) write_part(a, stats + threadIdx.x, m0 + threadIdx.x, split);
  if (warp == 0 && lane == 0 && *abort_flag) {
    if (leader) {
      // let the pair's loads still in flight land before either CTA exits (bounded)
      for (uint32_t s = 0; s < (uint32_t)kStages; ++s) {
        if (issued <= s) continue;
        const uint32_t last = s + ((issued - 1 - s) / kStages) * kStages;
        if (!tc::mbar_wait(&full[s], (last / kStages) & 1u)) atomicOr(a.err, ZO_FLAG_TIMEOUT);
      }
    } else {
      __nanosleep(1000000);  // the peer cannot observe its loads' completion: give them time
    }
  }
  __syncwarp();
  if (warp == 1) {
    if (lane == 0 && !tc::mbar_wait(mma_done, 0)) atomicOr(a.err, ZO_FLAG_TIMEOUT);
    __syncwarp();
    tc::tc_fence_after();
  }
  tc::cluster_sync();  // no remote arrival or MMA touches either CTA after this point
  if (warp == 1) tc::tmem_dealloc_pair(tmem, 2 * kBN);
}

// One warp per row: its triples joined lane by lane, then across the lanes, in fp64.
__global__ void __launch_bounds__(256)
head_join_kernel(HeadArgs a, float *logprob, float *entropy) {
  constexpr int N = (kSmCount + 31) / 32;  // triples of a lane (148 at most in all)
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  tc::pdl_wait();
  if (row >= a.rows) return;
  const float4 *part = a.part + (int64_t)row * a.splits;
  const int32_t target = logprob ? a.targets[row] : -1;
  const float target_logit = a.target_logit[row];  // not written without a target in range
  float4 t[N];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    t[k] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (lane + 32 * k < a.splits) t[k] = part[lane + 32 * k];
  }
#pragma unroll
  for (int k = 0; k < N; ++k) m = fmaxf(m, t[k].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  double s = 0.0, u = 0.0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    RowStats r;
    r.m = t[k].x;
    r.s = (double)t[k].y + (double)t[k].w;
    r.u = (double)t[k].z;
    r.add_to(m, s, u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
  }
  if (lane != 0) return;
  const double log2s = log2(s);
  if (entropy) entropy[row] = (float)(kLn2 * (log2s - u / s));
  if (logprob) {
    float v = __uint_as_float(0x7FC00000u);
    if (target == -1) v = 0.f;
    else if (target >= 0 && target < a.vocab)
      v = (float)(kLn2 * ((double)target_logit * (double)kLog2E - (double)m - log2s));
    logprob[row] = v;
  }
}

// Pairs from the 129th row on: one CTA a tile reads twice the bytes of W for the rows of two.
bool head_pairs(int64_t rows) { return rows > kBM; }

struct HeadShape {
  int64_t unit, row_tiles, slots, units;
  int64_t most;  // ranges: one for every CTA or pair of the machine for one row tile, at most 32 for more
};
HeadShape head_shape(int64_t rows, int64_t vocab) {
  const bool pairs = head_pairs(rows);
  const int64_t tile = pairs ? HeadCfg<true>::kRows : HeadCfg<false>::kRows;
  HeadShape h;
  h.unit = pairs ? HeadCfg<true>::kUnit : HeadCfg<false>::kUnit;
  h.slots = pairs ? kSmCount / 2 : kSmCount;
  h.row_tiles = (rows + tile - 1) / tile;
  h.units = (vocab + h.unit - 1) / h.unit;
  h.most = h.row_tiles * 32 < h.slots ? h.slots / h.row_tiles : 32;
  if (h.most > h.units) h.most = h.units;
  return h;
}

// The number of ranges whose estimated time is least: waves of CTAs (or pairs), each a fixed cost
// (start, first loads, last epilogue: about 4 us) and its units' products (9 TFLOP/s an
// SM) or exponentials (16 a clock).
int head_splits(const HeadShape &h, int64_t width) {
  const double flops = 2.0 * kBM * (double)h.unit * (double)((width + kBK - 1) / kBK * kBK);
  const double unit_us = std::fmax(flops / 9.0e6, kBM * (double)h.unit / 16.0 / 1.8e3);
  int64_t best = 1;
  double least = 1e300;
  for (int64_t s = 1; s <= h.most; ++s) {
    const int64_t waves = (h.row_tiles * s + h.slots - 1) / h.slots;
    const double us = (double)waves * (4.0 + unit_us * (double)((h.units + s - 1) / s));
    if (us < least * 0.995) {
      least = us;
      best = s;
    }
  }
  return (int)best;
}

bool head_sizes_ok(int64_t rows, int64_t vocab) {
  return rows >= 1 && rows < INT32_MAX - 256 && vocab >= 1 && vocab < INT32_MAX - 512;
}

int64_t head_bytes_of(int64_t rows, int64_t vocab) {
  return rows * (head_shape(rows, vocab).most * (int64_t)sizeof(float4)) + ((rows * 4 + 15) / 16) * 16;
}

// Enough for these rows and for fewer, some of which take more ranges: those of one CTA, and those of
// the last row of one, two, .. row tiles, up to where the number of ranges no longer falls.
int64_t head_bytes(int64_t rows, int64_t vocab) {
  int64_t most = std::max(head_bytes_of(rows, vocab), head_bytes_of(std::min<int64_t>(rows, kBM), vocab));
  for (int64_t tiles = 1; tiles * 32 < kSmCount / 2; ++tiles)
    most = std::max(most, head_bytes_of(std::min<int64_t>(rows, tiles * HeadCfg<true>::kRows), vocab));
  return most;
}

}  // namespace
}  // namespace zo

using namespace zo;

extern "C" {

zo_status zo_head_logprobs_workspace(int64_t rows, int64_t vocab, int64_t *bytes) {
  if (!bytes || !head_sizes_ok(rows, vocab)) return ZO_ERR_INVALID;
  *bytes = head_bytes(rows, vocab);
  return ZO_OK;
}

zo_status zo_head_logprobs(zo_ctx *ctx, const void *hidden, const void *W, int64_t rows, int64_t vocab,
                           int64_t width, int64_t ldh, int64_t ldw, const int32_t *targets,
                           float *logprob, float *entropy, void *workspace, int64_t workspace_bytes) {
  if (!ctx) return ZO_ERR_INVALID;
  ctx->err.clear();
  if (!hidden || !W || !workspace || (logprob && !targets) || (!logprob && !entropy))
    return fail(ctx, ZO_ERR_INVALID, "null head_logprobs argument");
  if (!head_sizes_ok(rows, vocab) || width < 1 || width >= INT32_MAX - 64 || width % 8 || ldh < width ||
      ldw < width || ldh > INT32_MAX || ldw > INT32_MAX || ldh % 8 || ldw % 8)
    return fail(ctx, ZO_ERR_INVALID, "head_logprobs: need rows, vocab, width >= 1 (below 2^31), width, ldh "
                "and ldw multiples of 8, ldh and ldw >= width");
  if ((reinterpret_cast<uintptr_t>(hidden) | reinterpret_cast<uintptr_t>(W) |
       reinterpret_cast<uintptr_t>(workspace)) & 15u)
    return fail(ctx, ZO_ERR_INVALID, "head_logprobs: hidden, W and the workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(targets) | reinterpret_cast<uintptr_t>(logprob) |
       reinterpret_cast<uintptr_t>(entropy)) % 4)
    return fail(ctx, ZO_ERR_INVALID, "head_logprobs: pointers not aligned to their elements");
  if (workspace_bytes < head_bytes(rows, vocab))
    return fail(ctx, ZO_ERR_INVALID, "head_logprobs: workspace of %lld bytes, %lld needed",
                (long long)workspace_bytes, (long long)head_bytes(rows, vocab));
  const DeviceScope device(ctx);
  if (device.status != cudaSuccess)
    return fail(ctx, ZO_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(device.status));
  const bool pairs = head_pairs(rows);
  const HeadShape shape = head_shape(rows, vocab);
  HeadArgs a;
  a.rows = (int)rows;
  a.vocab = (int)vocab;
  a.width = (int)width;
  a.splits = head_splits(shape, width);
  a.units = (int)shape.units;
  a.a_rows = rows < kBM ? (int)(rows + 7) / 8 * 8 : kBM;
  a.targets = targets;
  a.part = static_cast<float4 *>(workspace);
  a.target_logit = reinterpret_cast<float *>(a.part + rows * a.splits);
  a.err = &ctx->dstate->flags;
  CUtensorMap ta, tb, tw;
  if (!tile_map_bf16(&ta, hidden, rows, width, ldh, a.a_rows) || !tile_map_bf16(&tb, W, vocab, width, ldw, kBox) ||
      (pairs && !tile_map_bf16(&tw, W, vocab, width, ldw, kBN / 2)))
    return fail(ctx, ZO_ERR_CUDA, "head_logprobs: cuTensorMapEncodeTiled failed");
  const void *kernel = pairs ? reinterpret_cast<const void *>(head_pair_kernel) : reinterpret_cast<const void *>(head_kernel);
  const int smem = (int)(pairs ? HeadCfg<true>::kBytes : HeadCfg<false>::kBytes);
  cudaError_t e = ensure_smem_limit(kernel, smem);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "head_kernel attribute: %s", cudaGetErrorString(e));
  const int64_t m = (rows + kBM - 1) / kBM;
  const dim3 grid((unsigned)(pairs ? (m + 1) / 2 * 2 : m), (unsigned)a.splits);
  e = pairs ? launch_early(head_pair_kernel, grid, kThreads, smem, ctx->stream, ta, tb, tw, a)
            : launch_early(head_kernel, grid, kThreads, smem, ctx->stream, ta, tb, a);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "head_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  e = launch_early(head_join_kernel, dim3((unsigned)((rows + 7) / 8)), 256, 0, ctx->stream, a, logprob, entropy);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "head_join_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
}

}  // extern "C"
