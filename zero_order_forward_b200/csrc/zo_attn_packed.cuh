// zo_attn_packed.cuh -- what the kernels of zo_attention_packed share: arguments, sequences, outputs of
// 64 bytes a row, and rows that a later token's value must not reach.
#pragma once

#include "zo_internal.cuh"
#include "zo_tc.cuh"

namespace zo {

struct PackedArgs {
  const uint16_t *q, *k, *v;
  uint16_t *out;
  const int32_t *cu;
  int n_seqs, total, H, Hk;
  int64_t ldq, ldk, ldv, ldo;
  float scale_log2;
  int mode, shared;  // query heads of a key/value head
  int handled;       // sequences of at most this length are another kernel's
  uint32_t *err;
};

// A sequence's first row and length; no rows if its offsets decrease or leave [0, total].
struct Seq {
  int row0, len;
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const PackedArgs &a, int i) {
  if (i >= a.n_seqs) return {0, 0, false};
  const int s = __ldg(a.cu + i), e = __ldg(a.cu + i + 1);
  const bool bad = s < 0 || e < s || e > a.total;
  return {s, bad ? 0 : e - s, bad};
}

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }

// Rows first + (bits of `rows`) of the tile came out infinite or NaN somewhere.  That is right if a
// value row that they attend to says so, but in the tile's last keys (up to key_end) a later row's
// infinity or NaN reaches them as well, as 0 * infinity = NaN.  So a column with such an output and a
// non-finite later value is computed again from the row's own keys, in fp32, whatever they hold; the
// row's other columns stay.  One warp: key by key from the row's own backwards, 32 at a time, until
// each such column is NaN for good.
template <int HD>
__device__ __noinline__ void repair_rows(const PackedArgs &a, int row0, int len, int first, uint32_t rows,
                                         int h, int kvh, int key_end) {
  constexpr int C = HD / 32;  // output columns of a lane: C lane .. C lane + C - 1
  const int lane = threadIdx.x & 31;
  const uint16_t *K = a.k + (int64_t)row0 * a.ldk + kvh * HD;
  const uint16_t *V = a.v + (int64_t)row0 * a.ldv + kvh * HD + C * lane;
  for (; rows; rows &= rows - 1) {
    const int r = first + __ffs(rows) - 1;
    uint16_t *orow = a.out + (int64_t)(row0 + r) * a.ldo + h * HD + C * lane;
    uint32_t bad = 0, later = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) bad |= finite_bf16(orow[c]) ? 0u : 1u << c;
    if (!__any_sync(0xFFFFFFFFu, bad)) continue;
#pragma unroll 4
    for (int j = r + 1; j < min(key_end, len); ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) later |= finite_bf16(V[(int64_t)j * a.ldv + c]) ? 0u : 1u << c;
    const uint32_t open = bad & later;  // this lane's columns to compute again
    if (!__any_sync(0xFFFFFFFFu, open)) continue;
    const uint16_t *q = a.q + (int64_t)(row0 + r) * a.ldq + h * HD;
    float m = -INFINITY, l = 0.f, acc[C] = {};
    for (int j0 = r; j0 >= 0; j0 -= 32) {  // keys j0, j0 - 1, ..
      const int j = j0 - lane;
      float s = -INFINITY;
      if (j >= 0) {
        s = 0.f;
#pragma unroll 4
        for (int e = 0; e < HD; e += 8) {
          const uint4 x = *reinterpret_cast<const uint4 *>(q + e);
          const uint4 y = *reinterpret_cast<const uint4 *>(K + (int64_t)j * a.ldk + e);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            s = fmaf(__uint_as_float(u[t] << 16), __uint_as_float(w[t] << 16), s);
            s = fmaf(__uint_as_float(u[t] & 0xFFFF0000u), __uint_as_float(w[t] & 0xFFFF0000u), s);
          }
        }
        s *= a.scale_log2;
      }
      float mx = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      mx = fmaxf(mx, m);
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float f = tc::ex2(m - ref), p = j >= 0 ? tc::ex2(s - ref) : 0.f;
      float sum = p;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      l = l * f + sum;
      m = mx;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] *= f;
#pragma unroll 8
      for (int t = 0; t < min(32, j0 + 1); ++t) {
        const float pt = __shfl_sync(0xFFFFFFFFu, p, t);
#pragma unroll
        for (int c = 0; c < C; ++c)
          acc[c] = fmaf(pt, bf16_bits_to_f32(V[(int64_t)(j0 - t) * a.ldv + c]), acc[c]);
      }
      bool more = false;  // (a NaN stays one)
#pragma unroll
      for (int c = 0; c < C; ++c) more |= (open >> c & 1u) && acc[c] == acc[c];
      if (!__any_sync(0xFFFFFFFFu, more)) break;
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (open >> c & 1u) orow[c] = f32_to_bf16_bits(acc[c] / l);
  }
}

// The words a[0 .. 3] of a quad's lanes transposed: a[k] becomes lane k's word of this lane's number.
__device__ __forceinline__ void quad_transpose(uint32_t (&a)[4]) {
  const int c = threadIdx.x & 3;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const uint32_t v = __shfl_xor_sync(0xFFFFFFFFu, c & 1 ? a[k] : a[k + 1], 1);
    if (c & 1) a[k] = v;
    else a[k + 1] = v;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t v = __shfl_xor_sync(0xFFFFFFFFu, c & 2 ? a[k] : a[k + 2], 2);
    if (c & 2) a[k] = v;
    else a[k + 2] = v;
  }
}

// Attention of the sequences of at most kShortSeq tokens (zo_attn_short.cu), on ctx's stream.
constexpr int kShortSeq = 32;
zo_status launch_attn_short(zo_ctx *ctx, const PackedArgs &a, int head_dim);

}  // namespace zo
