// zo_attn_packed.cu -- causal grouped-query attention within packed sequences of different
// lengths (zo_attention_packed), on the tensor cores; forward only:
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   over the rows j of i's own sequence.
//
// One CTA (6 warps) per (128-query tile of one sequence, head), two CTAs per SM.  The grid holds
// as many blocks as tiles are possible (ceil(total / 128) + n_seqs); a block finds its sequence
// and tile by counting tiles over cu_seqlens, which is read on the device only.  Key tiles of 64
// keys flow through the pipeline of zo_attn_tc.cu: one warp issues TMA loads, one the MMAs
// (S = Q K^T into tensor memory, O += P V with P read from tensor memory), four compute the
// softmax, one query row per thread.  What packing adds:
//   - tiles start at any row, so the last key tile of a sequence also holds rows of the next one
//     (or padding): their scores are masked, their value rows cleared in shared memory before
//     they are multiplied;
//   - within the diagonal tile a later token's value row is multiplied by probability 0, which is
//     not 0 for an infinity or NaN: a row whose output is not finite is looked at again
//     (repair_rows) and recomputed from its own keys alone where a later row is to blame.
#include <cmath>

#include "zo_internal.cuh"
#include "zo_tc.cuh"

namespace zo {
namespace {

using tc::add2;
using tc::ex2;
using tc::fma2_bc;
using tc::max3f;
using tc::ring_parity;
using tc::warp_wait;

constexpr int kTBM = 128, kTThreads = 192;
constexpr uint32_t kQBox = 128 * 128;  // bytes of one 128-row x 64-column bf16 box

template <int HD> struct PackedCfg {
  static constexpr int kBN = 64;
  static constexpr int kKS = HD == 128 ? 2 : 4;  // K stages
  static constexpr int kVS = HD == 128 ? 2 : 4;  // V stages
  static constexpr int kCtas = 2;
  static constexpr int kTmemCols = 256;
  static constexpr uint32_t kKBox = kBN * 128;  // bytes of one kBN-row x 64-column bf16 box
};

template <int HD>
struct PackedSmem {
  static constexpr int kKS = PackedCfg<HD>::kKS, kVS = PackedCfg<HD>::kVS;
  static constexpr uint32_t kQTile = (HD / 64) * kQBox;
  static constexpr uint32_t kKTile = (HD / 64) * PackedCfg<HD>::kKBox;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kQTile;        // [kKS]
  static constexpr uint32_t kV = kK + kKS * kKTile;  // [kVS]
  static constexpr uint32_t kBar = kV + kVS * kKTile;
  static constexpr int kNumBars = 1 + 2 * kKS + 2 * kVS + 2 + 2 + 2 + 1;
  static constexpr uint32_t kBytes = kBar + 256 + 1024;  // barriers + alignment slack
  static_assert(kNumBars * 8 + 8 <= 256, "barrier area");
};

struct PackedArgs {
  const uint16_t *q, *k, *v;
  uint16_t *out;
  const int32_t *cu;
  int n_seqs, total, H, Hk;
  int64_t ldq, ldk, ldv, ldo;
  float scale_log2;
  uint32_t *err;
};

struct Tile {
  int row0, len;  // the sequence's first row and length (0: no such tile)
  int qt;         // query tile within the sequence
};

// The sequence and query tile of tile number `slot`, counting ceil(len / 128) tiles for every
// sequence in order.  All threads of the block call; each warp counts by itself, 32 sequences at a
// time.  Pairs of offsets that decrease or leave [0, total] count no tile; `check` goes on to the
// last one and raises ZO_FLAG_OFFSETS for them.
__device__ __forceinline__ Tile find_tile(const PackedArgs &a, int slot, bool check) {
  const int lane = threadIdx.x & 31;
  Tile t{0, 0, 0};
  int base = 0;
  for (int i0 = 0; i0 < a.n_seqs; i0 += 32) {
    const int i = i0 + lane;
    int s = 0, e = 0;
    if (i < a.n_seqs) {
      s = __ldg(a.cu + i);
      e = __ldg(a.cu + i + 1);
      if (s < 0 || e < s || e > a.total) {
        if (check && threadIdx.x < 32) atomicOr(a.err, ZO_FLAG_OFFSETS);
        s = e = 0;
      }
    }
    const int n = (e - s + kTBM - 1) / kTBM;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, base + incl > slot);
    if (past && t.len == 0) {
      const int l = __ffs(past) - 1;
      t.row0 = __shfl_sync(0xFFFFFFFFu, s, l);
      t.len = __shfl_sync(0xFFFFFFFFu, e, l) - t.row0;
      t.qt = slot - (base + __shfl_sync(0xFFFFFFFFu, incl - n, l));
      if (!check) break;
    }
    base += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return t;
}

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }

// Rows first + (bits of `rows`) of the tile came out infinite or NaN.  That is right if a value
// row that they attend to says so; it is wrong where only a later row of the tile's last keys
// (up to key_end) does.  One warp: a row with a non-finite later value row, and with a non-finite
// output that no own key's value explains, is computed again from keys 0 .. r alone, in fp32.
template <int HD>
__device__ __noinline__ void repair_rows(const PackedArgs &a, const Tile &tile, int first, uint32_t rows,
                                         int h, int kvh, int key_end) {
  constexpr int C = HD / 32;  // output columns of a lane: C lane .. C lane + C - 1
  const int lane = threadIdx.x & 31;
  const uint16_t *K = a.k + (int64_t)tile.row0 * a.ldk + kvh * HD;
  const uint16_t *V = a.v + (int64_t)tile.row0 * a.ldv + kvh * HD + C * lane;
  for (; rows; rows &= rows - 1) {
    const int r = first + __ffs(rows) - 1;
    bool later = false;
    for (int j = r + 1; j < min(key_end, tile.len); ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) later |= !finite_bf16(V[(int64_t)j * a.ldv + c]);
    if (!__any_sync(0xFFFFFFFFu, later)) continue;
    uint16_t *orow = a.out + (int64_t)(tile.row0 + r) * a.ldo + h * HD + C * lane;
    uint32_t open = 0;  // this lane's non-finite outputs not explained yet
#pragma unroll
    for (int c = 0; c < C; ++c) open |= finite_bf16(orow[c]) ? 0u : 1u << c;
    for (int j = 0; j <= r && __any_sync(0xFFFFFFFFu, open); ++j)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (!finite_bf16(V[(int64_t)j * a.ldv + c])) open &= ~(1u << c);
    if (!__any_sync(0xFFFFFFFFu, open)) continue;
    const uint16_t *q = a.q + (int64_t)(tile.row0 + r) * a.ldq + h * HD;
    float m = -INFINITY, l = 0.f, acc[C] = {};
    for (int j0 = 0; j0 <= r; j0 += 32) {
      const int j = j0 + lane;
      float s = -INFINITY;
      if (j <= r) {
        s = 0.f;
        for (int e = 0; e < HD; ++e)
          s = fmaf(bf16_bits_to_f32(q[e]), bf16_bits_to_f32(K[(int64_t)j * a.ldk + e]), s);
        s *= a.scale_log2;
      }
      float mx = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      mx = fmaxf(mx, m);
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float f = ex2(m - ref), p = j <= r ? ex2(s - ref) : 0.f;
      float sum = p;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      l = l * f + sum;
      m = mx;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] *= f;
      for (int t = 0; t < 32 && j0 + t <= r; ++t) {
        const float pt = __shfl_sync(0xFFFFFFFFu, p, t);
#pragma unroll
        for (int c = 0; c < C; ++c)
          acc[c] = fmaf(pt, bf16_bits_to_f32(V[(int64_t)(j0 + t) * a.ldv + c]), acc[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) orow[c] = f32_to_bf16_bits(acc[c] / l);
  }
}

template <int HD>
__global__ void __launch_bounds__(kTThreads, PackedCfg<HD>::kCtas)
attn_packed_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv,
                   PackedArgs a) {
  using SM = PackedSmem<HD>;
  constexpr int KS = SM::kKS, VS = SM::kVS;
  constexpr uint32_t kCols = PackedCfg<HD>::kTmemCols;
  constexpr int kTBN = PackedCfg<HD>::kBN;
  constexpr uint32_t kKBox = PackedCfg<HD>::kKBox;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + SM::kBar);
  uint64_t *q_full = bars;
  uint64_t *k_full = q_full + 1, *k_empty = k_full + KS;
  uint64_t *v_full = k_empty + KS, *v_empty = v_full + VS;
  uint64_t *s_full = v_empty + VS;  // [2] scores of tile j in buffer j % 2
  uint64_t *p_full = s_full + 2;    // [2] probabilities of tile j written (4 softmax warps)
  uint64_t *pv_done = p_full + 2;   // [2] O += P_j V_j completed
  uint64_t *mma_done = pv_done + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, kvh = h / (a.H / a.Hk);
  const Tile tile = find_tile(a, blockIdx.x, blockIdx.x == 0 && h == 0);
  if (tile.len == 0) return;  // more blocks than tiles (uniform over the block)
  const int row0 = tile.row0, S = tile.len;
  const int q_first = tile.qt * kTBM;
  const int last_q = min(q_first + kTBM, S) - 1;
  const int n_kt = last_q / kTBN + 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < SM::kNumBars; ++i) tc::mbar_init(&bars[i], 1);
    tc::mbar_init(&p_full[0], 4);  // one arrival per softmax warp
    tc::mbar_init(&p_full[1], 4);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_holder, kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tO = tmem + 2 * kTBN;  // S/P buffers at columns 0 and kTBN

  if (warp == 0) {
    if (lane == 0) {  // TMA producer: Q once, then K_j ahead of V_{j-1}
      tc::tma_prefetch_desc(&tmq);
      tc::tma_prefetch_desc(&tmk);
      tc::tma_prefetch_desc(&tmv);
      tc::mbar_arrive_expect_tx(q_full, SM::kQTile);
#pragma unroll
      for (int c = 0; c < HD / 64; ++c)
        tc::tma_load_2d(sm + SM::kQ + c * kQBox, &tmq, q_full, h * HD + 64 * c, row0 + q_first);
      int k_issued = 0, v_issued = 0;
      auto load_k = [&](int j) -> bool {
        if (*abort_flag || !tc::mbar_wait(&k_empty[j % KS], ring_parity(j, KS) ^ 1u)) return false;
        tc::mbar_arrive_expect_tx(&k_full[j % KS], SM::kKTile);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
          tc::tma_load_2d(sm + SM::kK + (j % KS) * SM::kKTile + c * kKBox, &tmk, &k_full[j % KS],
                          kvh * HD + 64 * c, row0 + j * kTBN);
        k_issued = j + 1;
        return true;
      };
      auto load_v = [&](int j) -> bool {
        if (*abort_flag || !tc::mbar_wait(&v_empty[j % VS], ring_parity(j, VS) ^ 1u)) return false;
        tc::mbar_arrive_expect_tx(&v_full[j % VS], SM::kKTile);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
          tc::tma_load_2d(sm + SM::kV + (j % VS) * SM::kKTile + c * kKBox, &tmv, &v_full[j % VS],
                          kvh * HD + 64 * c, row0 + j * kTBN);
        v_issued = j + 1;
        return true;
      };
      bool ok = true;
      for (int j = 0; ok && j <= n_kt; ++j) {
        if (j < n_kt) ok = load_k(j);
        if (ok && j >= 1) ok = load_v(j - 1);
      }
      if (!ok) {
        atomicOr(a.err, ZO_FLAG_TIMEOUT);
        *abort_flag = 1;
        // let this CTA's loads land before it exits (bounded)
        tc::mbar_wait(q_full, 0);
        for (int i = k_issued - KS > 0 ? k_issued - KS : 0; i < k_issued; ++i)
          tc::mbar_wait(&k_full[i % KS], ring_parity(i, KS));
        for (int i = v_issued - VS > 0 ? v_issued - VS : 0; i < v_issued; ++i)
          tc::mbar_wait(&v_full[i % VS], ring_parity(i, VS));
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {  // MMA issuer
      constexpr uint32_t idS = tc::idesc_bf16_f32(kTBM, kTBN);
      constexpr uint32_t idO = tc::idesc_bf16_f32(kTBM, HD) | (1u << 16);  // B (V) MN-major
      const uint32_t qa = tc::smem_addr(sm + SM::kQ);
      // S_j = Q K_j^T into score buffer j % 2
      auto issue_s = [&](int j) -> bool {
        if (*abort_flag || !tc::mbar_wait(&k_full[j % KS], ring_parity(j, KS))) return false;
        tc::tc_fence_after();
        const uint32_t ka = tc::smem_addr(sm + SM::kK + (j % KS) * SM::kKTile);
        const uint32_t tS = tmem + (uint32_t)((j & 1) * kTBN);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t kk = (uint32_t)(k & 3) * 32u;
          tc::mma_bf16(tS, tc::smem_desc_k128(qa + (uint32_t)(k >> 2) * kQBox + kk),
                       tc::smem_desc_k128(ka + (uint32_t)(k >> 2) * kKBox + kk), idS, k > 0 ? 1u : 0u);
        }
        tc::mma_commit(&s_full[j & 1]);
        tc::mma_commit(&k_empty[j % KS]);
        return true;
      };
      bool ok = tc::mbar_wait(q_full, 0) && issue_s(0) && (n_kt < 2 || issue_s(1));
      for (int j = 0; ok && j < n_kt; ++j) {
        // O += P_j V_j once the softmax has written P_j (in place of S_j) and V_j has landed
        ok = tc::mbar_wait(&p_full[j & 1], ring_parity(j, 2)) &&
             tc::mbar_wait(&v_full[j % VS], ring_parity(j, VS));
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t va = tc::smem_addr(sm + SM::kV + (j % VS) * SM::kKTile);
        const uint32_t tP = tmem + (uint32_t)((j & 1) * kTBN);
#pragma unroll
        for (int k = 0; k < kTBN / 16; ++k) {
          if (j * kTBN + 16 * k >= S) break;  // keys behind the sequence: not multiplied
          const uint32_t boff = (uint32_t)k * 16u * 128u;  // 16 keys of 128-byte V rows
          tc::mma_bf16_tmem_a(tO, tP + 8u * k, tc::smem_desc_mn128(va + boff, kKBox), idO,
                              (j > 0 || k > 0) ? 1u : 0u);
        }
        tc::mma_commit(&pv_done[j & 1]);
        tc::mma_commit(&v_empty[j % VS]);
        if (j + 2 < n_kt) {
          // S_{j+2} reuses buffer j % 2: wait until P_j V_j has read it
          ok = tc::mbar_wait(&pv_done[j & 1], ring_parity(j, 2)) && issue_s(j + 2);
        }
      }
      if (!ok) {
        atomicOr(a.err, ZO_FLAG_TIMEOUT);
        *abort_flag = 1;
      }
      tc::mma_commit(mma_done);  // arrives once every MMA issued above has retired
    }
  } else {  // softmax warps: TMEM lane quadrant qd holds the tile's query rows 32 qd .. +31
    const int qd = warp & 3;
    const int tr = 32 * qd + lane;  // row within the tile
    const int r = q_first + tr;     // query position in the sequence
    const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kt; ++j) {
      const uint32_t tS = tmem + (uint32_t)((j & 1) * kTBN) + lane_off;
      if (!warp_wait(&s_full[j & 1], ring_parity(j, 2), abort_flag)) { ok = false; break; }
      tc::tc_fence_after();
      float s[kTBN];
#pragma unroll
      for (int c = 0; c < kTBN / 32; ++c) tc::tmem_ld32(tS + 32u * c, s + 32 * c);
      const int key0 = j * kTBN;
      // the causal / sequence-end mask touches only the tiles that reach the diagonal or the
      // end (uniform across the CTA: a real branch, not per-element selects)
      if (key0 + kTBN - 1 > q_first || key0 + kTBN > S) {
#pragma unroll
        for (int c = 0; c < kTBN; ++c)
          if (key0 + c > r || key0 + c >= S) s[c] = -INFINITY;
      }
      // the maximum of the raw scores (the scale is positive), then 2^(s * scale - m) with the
      // scaling folded into the exponent's fused multiply-add
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // 4 independent chains
#pragma unroll
      for (int c = 0; c < kTBN; c += 2) mx4[(c >> 1) & 3] = max3f(mx4[(c >> 1) & 3], s[c], s[c + 1]);
      const float mx = max3f(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3])) * a.scale_log2;
      const float m_new = fmaxf(m_used, mx);
      // Lazy rescaling: keep the running maximum unless it grows by more than 2^8 (then
      // O and l are rescaled, once the previous tile's P V has completed).
      const bool need = j > 0 && m_new > m_used + 8.f;
      const float m_old = m_used;
      if (j == 0 || need) m_used = m_new;
      const float msc = m_used == -INFINITY ? 0.f : m_used;
      uint32_t pk[kTBN / 2];
      float ls4[4] = {0.f, 0.f, 0.f, 0.f};  // two packed pairs of partial sums
#pragma unroll
      for (int c = 0; c < kTBN; c += 2) {
        float x0, x1;
        fma2_bc(s[c], s[c + 1], a.scale_log2, -msc, x0, x1);
        const float p0 = ex2(x0), p1 = ex2(x1);
        if ((c >> 1) & 1) add2(ls4[2], ls4[3], p0, p1);
        else add2(ls4[0], ls4[1], p0, p1);
        pk[c / 2] = pack_bf16x2(p0, p1);
      }
      const float lsum = (ls4[0] + ls4[1]) + (ls4[2] + ls4[3]);
      if (__any_sync(0xFFFFFFFFu, need)) {
        // O holds P_{j-1} V_{j-1} only once that MMA has completed
        if (!warp_wait(&pv_done[(j - 1) & 1], ring_parity(j - 1, 2), abort_flag)) { ok = false; break; }
        tc::tc_fence_after();
        const float f = need ? ex2(m_old - m_new) : 1.f;
        l *= f;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          float o[32];
          tc::tmem_ld32(tO + lane_off + 32u * c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f;
          tc::tmem_st32(tO + lane_off + 32u * c, o);
        }
      }
      // P_j overwrites the first kTBN / 2 columns of S_j (already read into registers)
      tc::tmem_st32u(tS, pk);
      l += lsum;
      if (key0 + kTBN > S) {
        // The rows behind the sequence (another one's, or padding) must not reach P V even with
        // probability 0: 0 * NaN is NaN.  Thread t clears row t of the value tile.
        if (!warp_wait(&v_full[j % VS], ring_parity(j, VS), abort_flag)) { ok = false; break; }
        if (tr < kTBN && key0 + tr >= S) {
          uint8_t *vrow = sm + SM::kV + (j % VS) * SM::kKTile + tr * 128;
#pragma unroll
          for (int c = 0; c < HD / 64; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4 *>(vrow + c * kKBox + 16 * i) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&p_full[j & 1]);
    }
    if (ok && !warp_wait(&pv_done[(n_kt - 1) & 1], ring_parity(n_kt - 1, 2), abort_flag)) ok = false;
    if (ok) {
      tc::tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      uint16_t *orow = a.out + (int64_t)(row0 + r) * a.ldo + h * HD;
      float worst = 0.f;  // NaN if any output of the row is not finite
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float o[32];
        tc::tmem_ld32(tO + lane_off + 32u * c, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i] *= inv;
          worst = fmaf(o[i], 0.f, worst);
        }
        if (r < S) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 w = make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]),
                                       pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                                       pack_bf16x2(o[8 * q + 4], o[8 * q + 5]),
                                       pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
            *reinterpret_cast<uint4 *>(orow + 32 * c + 8 * q) = w;
          }
        }
      }
      const uint32_t suspects = __ballot_sync(0xFFFFFFFFu, r < S && worst != worst);
      __syncwarp();
      if (suspects) repair_rows<HD>(a, tile, q_first + 32 * qd, suspects, h, kvh, n_kt * kTBN);
    } else if (lane == 0) {
      atomicOr(a.err, ZO_FLAG_TIMEOUT);
      *abort_flag = 1;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0 && !tc::mbar_wait(mma_done, 0)) atomicOr(a.err, ZO_FLAG_TIMEOUT);
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kCols);
  }
}

template <int HD>
zo_status launch(zo_ctx *ctx, const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                 const PackedArgs &a) {
  using SM = PackedSmem<HD>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(attn_packed_kernel<HD>), (int)SM::kBytes);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "attn_packed_kernel attribute: %s", cudaGetErrorString(e));
  const dim3 grid((unsigned)((int64_t)(a.total + kTBM - 1) / kTBM + a.n_seqs), a.H);
  attn_packed_kernel<HD><<<grid, kTThreads, SM::kBytes, ctx->stream>>>(tmq, tmk, tmv, a);
  return check_launch(ctx, "attn_packed_kernel");
}

}  // namespace
}  // namespace zo

using namespace zo;

extern "C" zo_status zo_attention_packed(zo_ctx *ctx, const void *q, const void *k, const void *v, void *out,
                                         const int32_t *cu_seqlens, int32_t n_seqs, int64_t total_tokens,
                                         int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldo,
                                         int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale) {
  if (!ctx) return ZO_ERR_INVALID;
  ctx->err.clear();
  if (!q || !k || !v || !out || !cu_seqlens) return fail(ctx, ZO_ERR_INVALID, "null attention argument");
  if (head_dim != 64 && head_dim != 128)
    return fail(ctx, ZO_ERR_UNSUPPORTED, "attention_packed: head_dim must be 64 or 128");
  if (n_heads < 1 || n_heads > 65535 || n_kv_heads < 1 || n_heads % n_kv_heads)
    return fail(ctx, ZO_ERR_INVALID, "attention_packed: n_kv_heads must divide n_heads (1 .. 65535)");
  if (n_seqs < 1 || total_tokens < 1 || total_tokens > INT32_MAX - 256 || n_seqs > INT32_MAX / 2)
    return fail(ctx, ZO_ERR_INVALID, "attention_packed: need n_seqs >= 1 and total_tokens in [1, 2^31 - 257]");
  const int64_t wq = (int64_t)n_heads * head_dim, wk = (int64_t)n_kv_heads * head_dim;
  if (ldq < wq || ldo < wq || ldk < wk || ldv < wk || (ldq | ldk | ldv | ldo) % 8 || (ldq | ldk | ldv) >= ((int64_t)1 << 38))
    return fail(ctx, ZO_ERR_INVALID, "attention_packed: row strides must cover the heads and be multiples of 8");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out)) & 15u || reinterpret_cast<uintptr_t>(cu_seqlens) % 4)
    return fail(ctx, ZO_ERR_INVALID, "attention_packed: buffers must be 16-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return fail(ctx, ZO_ERR_INVALID, "attention_packed: scale must be finite and > 0");
  const DeviceScope device(ctx);
  if (device.status != cudaSuccess)
    return fail(ctx, ZO_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(device.status));
  CUtensorMap tmq, tmk, tmv;
  constexpr int kBN = PackedCfg<128>::kBN;  // the same for both head dims
  if (!tile_map_bf16(&tmq, q, total_tokens, wq, ldq, kTBM) ||
      !tile_map_bf16(&tmk, k, total_tokens, wk, ldk, kBN) ||
      !tile_map_bf16(&tmv, v, total_tokens, wk, ldv, kBN))
    return fail(ctx, ZO_ERR_CUDA, "attention_packed: cuTensorMapEncodeTiled failed");
  const PackedArgs a{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                     static_cast<const uint16_t *>(v), static_cast<uint16_t *>(out), cu_seqlens, n_seqs,
                     (int)total_tokens, n_heads, n_kv_heads, ldq, ldk, ldv, ldo,
                     scale * 1.4426950408889634f, &ctx->dstate->flags};
  return head_dim == 64 ? launch<64>(ctx, tmq, tmk, tmv, a) : launch<128>(ctx, tmq, tmk, tmv, a);
}
