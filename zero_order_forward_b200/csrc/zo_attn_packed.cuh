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

// Rows first + (bits of `rows`) of the tile again, where their outputs are infinite or NaN.  That is right if
// a value row that they attend to says so, but in the tile's last keys (up to key_end) a later row's
// infinity or NaN reaches them as well, as 0 * infinity = NaN.  So a column with such an output and a
// non-finite later value is computed again from the row's own keys, in fp32, whatever they hold; the
// row's other columns stay.  One warp, R rows at a time (what 32 keys' loads wait for is then shared), from
// the last key backwards, 32 at a time, until each such column is NaN for good: a lane takes a key for the
// scores and C columns for the outputs.
template <int HD, int R>
__device__ __noinline__ void repair_rows(const PackedArgs &a, int row0, int len, int first, uint32_t rows,
                                         int h, int kvh, int key_end) {
  constexpr int C = HD / 32;  // output columns of a lane: C lane .. C lane + C - 1
  const int lane = threadIdx.x & 31;
  const uint16_t *Q = a.q + (int64_t)row0 * a.ldq + h * HD;
  const uint16_t *K = a.k + (int64_t)row0 * a.ldk + kvh * HD;
  const uint16_t *V = a.v + (int64_t)row0 * a.ldv + kvh * HD + C * lane;
  uint16_t *O = a.out + (int64_t)row0 * a.ldo + h * HD + C * lane;
  while (rows) {
    // the next R rows that have such columns
    int row[R], last = -1;  // -1: none
    uint32_t open = 0;      // this lane's columns of row i: bits C i ..
#pragma unroll
    for (int i = 0; i < R; ++i) {
      row[i] = -1;
      for (; rows && row[i] < 0; rows &= rows - 1) {
        const int r = first + __ffs(rows) - 1;
        uint32_t bad = 0, later = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) bad |= finite_bf16(O[r * a.ldo + c]) ? 0u : 1u << c;
        if (!__any_sync(0xFFFFFFFFu, bad)) continue;
#pragma unroll 4
        for (int j = r + 1; j < min(key_end, len); ++j)
#pragma unroll
          for (int c = 0; c < C; ++c) later |= finite_bf16(V[j * a.ldv + c]) ? 0u : 1u << c;
        if (!__any_sync(0xFFFFFFFFu, bad & later)) continue;
        row[i] = last = r;
        open |= (bad & later) << (C * i);
      }
    }
    if (last < 0) return;
    float m[R], l[R], acc[R][C];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = last; j0 >= 0; j0 -= 32) {  // keys j0, j0 - 1, ..
      const int j = j0 - lane;
      float s[R] = {};
#pragma unroll 4
      for (int e = 0; e < HD; e += 8) {
        const uint4 y = *reinterpret_cast<const uint4 *>(K + max(j, 0) * a.ldk + e);
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint4 x = *reinterpret_cast<const uint4 *>(Q + max(row[i], 0) * a.ldq + e);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            s[i] = fmaf(__uint_as_float(u[t] << 16), __uint_as_float(w[t] << 16), s[i]);
            s[i] = fmaf(__uint_as_float(u[t] & 0xFFFF0000u), __uint_as_float(w[t] & 0xFFFF0000u), s[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool in = j >= 0 && j <= row[i];
        s[i] = in ? s[i] * a.scale_log2 : -INFINITY;
        float mx = s[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        mx = fmaxf(mx, m[i]);
        const float ref = mx == -INFINITY ? 0.f : mx, f = tc::ex2(m[i] - ref);
        s[i] = in ? tc::ex2(s[i] - ref) : 0.f;
        m[i] = mx;
        float sum = s[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        l[i] = l[i] * f + sum;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[i][c] *= f;
      }
#pragma unroll 4
      for (int t = 0; t < min(32, j0 + 1); ++t) {
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = bf16_bits_to_f32(V[(j0 - t) * a.ldv + c]);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float p = __shfl_sync(0xFFFFFFFFu, s[i], t);
          if (j0 - t <= row[i])
#pragma unroll
            for (int c = 0; c < C; ++c) acc[i][c] = fmaf(p, v[c], acc[i][c]);
        }
      }
      bool more = false;  // (a NaN stays one)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c) more |= (open >> (C * i + c) & 1u) && acc[i][c] == acc[i][c];
      if (!__any_sync(0xFFFFFFFFu, more)) break;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (open >> (C * i + c) & 1u) O[row[i] * a.ldo + c] = f32_to_bf16_bits(acc[i][c] / l[i]);
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
