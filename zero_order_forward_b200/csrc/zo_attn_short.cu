// zo_attn_short.cu -- the sequences of at most kShortSeq tokens of zo_attention_packed: one block of two
// warps per sequence and head, all of its keys and values in shared memory, the whole softmax of a
// row at once:
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j.
//
// A warp takes 16 query rows.  Scores, probabilities and outputs stay in registers (mma.sync m16n8k16:
// the scores' accumulator is, packed, the probabilities' operand), keys only up to the rows' own
// sixteen.
//
// Bound: latency.  So short a sequence is a few products of 16 x 16 x 16; through the pipeline of
// zo_attn_packed.cu, made for long ones, each takes that kernel's whole chain of hand-overs (loads,
// scores, softmax, products, output: about 3 us), and one chain runs on an SM at a time.  Here an SM
// holds a dozen blocks, and a chain has two block barriers.  The warp-level products are slow on this
// part (about 37 clocks each on an SM quarter, an eighteenth of the tensor pipe's rate), and blocks of more
// warps, for longer sequences, start late: with 16 query and 8 key/value heads of 128, blocks for up to 128
// tokens took 60 us for 64 sequences of 128 where the pipeline takes 25, 37 us for 64 of 64 where it takes
// 20, and 21 us for 64 of 16, which blocks for 32 finish in 8.3.
#include "zo_attn_packed.cuh"

namespace zo {
namespace {

constexpr int kWarps = kShortSeq / 16, kThreads = 32 * kWarps;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool some) {  // zeros if not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int HD>
__global__ void __launch_bounds__(kThreads)
attn_short_kernel(const __grid_constant__ PackedArgs a) {
  constexpr int kChunks = HD / 8;            // pieces of 16 bytes of a row
  constexpr int kGroups = kShortSeq / 16;    // of 16 keys or rows
  extern __shared__ __align__(128) uint8_t smem[];
  tc::pdl_wait();
  const int h = blockIdx.x, i = (int)(blockIdx.z * gridDim.y + blockIdx.y);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Seq seq = load_seq(a, i);
  if (seq.bad && h == 0 && threadIdx.x == 0) atomicOr(a.err, ZO_FLAG_OFFSETS);
  if (seq.len == 0 || seq.len > kShortSeq) return;
  const int kvh = h / a.shared;
  const uint32_t sK = tc::smem_addr(smem), sV = sK + kShortSeq * HD * 2;
  // piece c of row r at c ^ (r % 8): eight rows' same piece in eight different banks' groups
  auto at = [&](int r, int c) { return (uint32_t)(r * HD * 2 + ((c ^ (r & 7)) << 4)); };
  {
    // whole groups of 16 rows; those behind the sequence are zeros (0 * NaN of another one would be NaN)
    const uint16_t *K = a.k + (int64_t)seq.row0 * a.ldk + kvh * HD, *V = a.v + (int64_t)seq.row0 * a.ldv + kvh * HD;
    const int pieces = (seq.len + 15) / 16 * 16 * kChunks;
    for (int p = threadIdx.x; p < pieces; p += kThreads) {
      const int r = p / kChunks, c = p % kChunks;
      const bool in = r < seq.len;
      copy16(sK + at(r, c), K + (in ? r : 0) * a.ldk + 8 * c, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int p = threadIdx.x; p < pieces; p += kThreads) {
      const int r = p / kChunks, c = p % kChunks;
      const bool in = r < seq.len;
      copy16(sV + at(r, c), V + (in ? r : 0) * a.ldv + 8 * c, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const int tile = warp;  // rows 16 tile .. + 15
  const bool any = 16 * tile < seq.len;
  const int r = 16 * tile + lane / 4;              // this lane's first row; the other is 8 behind
  float s[kGroups][2][4];
  uint32_t q[HD / 16][4];
  if (any) {
    const uint16_t *Q = a.q + (int64_t)(seq.row0 + r) * a.ldq + h * HD + 2 * (lane % 4);
#pragma unroll
    for (int k = 0; k < HD / 16; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q[k][e] = r + 8 * (e & 1) < seq.len
                      ? __ldg(reinterpret_cast<const uint32_t *>(Q + 8 * (e & 1) * a.ldq + 16 * k + 8 * (e >> 1)))
                      : 0u;
  }
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncthreads();
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  if (any) {
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][n][e] = 0.f;
    // groups innermost: their products do not wait for one another
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        if (j > tile) break;
        uint32_t b[4];
        ldmatrix4(b, sK + at(16 * j + lane / 16 * 8 + lane % 8, 2 * k + lane / 8 % 2));
        mma(s[j][0], q[k], b[0], b[1]);
        mma(s[j][1], q[k], b[2], b[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      if (j > tile) break;
      // keys behind the row: only the last group has any
      if (j == tile) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * j + 8 * n + 2 * (lane % 4) + (e & 1) > r + 8 * (e >> 1)) s[j][n][e] = -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        m[x] = fmaxf(m[x], fmaxf(tc::max3f(s[j][0][2 * x], s[j][0][2 * x + 1], s[j][1][2 * x]), s[j][1][2 * x + 1]));
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      m[x] = fmaxf(m[x], __shfl_xor_sync(0xFFFFFFFFu, m[x], 1));
      m[x] = fmaxf(m[x], __shfl_xor_sync(0xFFFFFFFFu, m[x], 2));
      m[x] = m[x] == -INFINITY ? 0.f : m[x] * a.scale_log2;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  if (!any) return;
  float o[HD / 8][4] = {};
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    if (j > tile) break;
    // probabilities 2^(s scale - m), rounded to bf16 for the product; the sum takes them unrounded
    uint32_t p[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float x0, x1;
        tc::fma2_bc(s[j][n][2 * x], s[j][n][2 * x + 1], a.scale_log2, -m[x], x0, x1);
        const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);
        l[x] += p0 + p1;
        p[2 * n + x] = pack_bf16x2(p0, p1);
      }
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      uint32_t b[4];
      ldmatrix4_trans(b, sV + at(16 * j + lane / 8 % 2 * 8 + lane % 8, 2 * d + lane / 16));
      mma(o[2 * d], p, b[0], b[1]);
      mma(o[2 * d + 1], p, b[2], b[3]);
    }
  }
  float inv[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 1);
    l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 2);
    inv[x] = 1.f / l[x];  // (l = 0: every score of the row is -inf, and 0 infinity = NaN)
  }
  uint16_t *out = a.out + (int64_t)(seq.row0 + r) * a.ldo + h * HD + 8 * (lane % 4);
  uint32_t worst[2] = {0, 0};  // bf16 pairs, not 0 (NaN) if any output of the row is not finite
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int d = 0; d < HD / 8; d += 4) {
      // four eights of columns lie across the quad; transposed, each lane has one
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = pack_bf16x2(o[d + k][2 * x] * inv[x], o[d + k][2 * x + 1] * inv[x]);
        worst[x] = tc::zero_or_nan2(v[k], worst[x]);
      }
      quad_transpose(v);
      if (r + 8 * x < seq.len)
        *reinterpret_cast<uint4 *>(out + 8 * x * a.ldo + 8 * d) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  const uint32_t bad[2] = {__ballot_sync(0xFFFFFFFFu, r < seq.len && worst[0] != 0),
                           __ballot_sync(0xFFFFFFFFu, r + 8 < seq.len && worst[1] != 0)};
  __syncwarp();
  if (bad[0] | bad[1]) {
    uint32_t rows = 0;
    for (int k = 0; k < 16; ++k) rows |= (bad[k / 8] >> (k % 8 * 4) & 15u ? 1u : 0u) << k;
    repair_rows<HD, 1>(a, seq.row0, seq.len, 16 * tile, rows, h, kvh, 16 * tile + 16);
  }
}

template <int HD>
zo_status launch(zo_ctx *ctx, const PackedArgs &a) {
  constexpr int kBytes = 2 * kShortSeq * HD * 2;
  const auto kernel = attn_short_kernel<HD>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kernel), kBytes);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "attn_short_kernel attribute: %s", cudaGetErrorString(e));
  const unsigned y = a.n_seqs < 65535 ? (unsigned)a.n_seqs : 65535u;
  const dim3 grid((unsigned)a.H, y, ((unsigned)a.n_seqs + y - 1) / y);
  e = launch_early(kernel, grid, kThreads, kBytes, ctx->stream, a);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "attn_short_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
}

}  // namespace

zo_status launch_attn_short(zo_ctx *ctx, const PackedArgs &a, int head_dim) {
  return head_dim == 64 ? launch<64>(ctx, a) : launch<128>(ctx, a);
}

}  // namespace zo
