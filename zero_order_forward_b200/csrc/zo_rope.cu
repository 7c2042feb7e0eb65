// zo_rope.cu -- rotary positions as an operator of its own (zo_rope):
//
//   t_i = positions[row] f_i,  (a, b) -> magnitude (a cos t_i - b sin t_i, b cos t_i + a sin t_i)
//
// for the rot_dim / 2 feature pairs of every head, in the half layout (i with i + rot_dim/2) or
// the interleaved one (2 i with 2 i + 1).  The frequencies, scaled for long contexts or not, are
// computed in fp64 on the host and travel as a kernel parameter.
//
// A block takes R rows.  Its threads first compute the rows' cosines and sines, once per (row,
// pair) and not per head, into shared memory: position x (f_i / 2 pi) in fp64, the fraction of a
// turn kept (exact enough at any int32 position: the product carries 53 bits, at most 31 of them
// before the point), then sincospi in fp32.  Then every group of threads that covers one head
// takes heads of the R rows in turn: 16 bytes of each half (half layout) or 16 bytes
// (interleaved) per thread.
// Bound: HBM, two passes over the rotated heads.
#include <cmath>
#include <cstring>

#include "zo_internal.cuh"

namespace zo {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = ZO_ROPE_MAX_HEAD_DIM / 2;
constexpr int kMaxRows = 16;  // rows of a block: kMaxRows x kMaxPairs float2 of shared memory

struct RopeArgs {
  const void *x;
  void *out;
  const int32_t *positions;
  int64_t rows, ldx, ldo;
  int heads, head_dim, pairs;
  int units;       // threads that cover one head
  int rot_units;   // of them, those that rotate (the others copy features behind rot_dim)
  int rows_block;  // R
  int heads_block; // heads of a block (blockIdx.y takes the next ones)
  float magnitude;
  double turns[kMaxPairs];  // f_i / (2 pi): turns per position
};

template <typename T> struct Elem;
template <> struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(uint16_t v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return f32_to_bf16_bits(v); }
};

template <typename T, int VEC> struct Pack;
template <> struct Pack<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void open(const Raw &r, float f[4]) {
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  }
  static __device__ __forceinline__ Raw close(const float f[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <> struct Pack<uint16_t, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void open(const Raw &r, float f[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f[2 * t] = __uint_as_float(w[t] << 16);
      f[2 * t + 1] = __uint_as_float(w[t] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ Raw close(const float f[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <typename T> struct Pack<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ void open(const T &r, float f[1]) { f[0] = Elem<T>::get(r); }
  static __device__ __forceinline__ T close(const float f[1]) { return Elem<T>::put(f[0]); }
};

// VEC: elements of one access (16 bytes' worth, or 1 where a pointer, a stride or a dimension is
// not a multiple of 16 bytes).  A rotating unit of the half layout covers VEC pairs with one
// access in each half; of the interleaved layout VEC / 2 pairs (VEC = 1: one pair, two accesses).
template <typename T, bool IL, int VEC>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs[kMaxRows * kMaxPairs];
  using P = Pack<T, VEC>;
  using Raw = typename P::Raw;
  const int64_t row0 = (int64_t)blockIdx.x * a.rows_block;
  const int rows = (int)min((int64_t)a.rows_block, a.rows - row0);
  for (int i = threadIdx.x; i < rows * a.pairs; i += kRopeThreads) {
    const int r = i / a.pairs, f = i - r * a.pairs;
    const int64_t row = row0 + r;
    const double t = (a.positions ? (double)a.positions[row] : (double)row) * a.turns[f];
    float s, c;
    sincospif(2.f * (float)(t - rint(t)), &s, &c);
    cs[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();
  const int group = threadIdx.x / a.units, unit = threadIdx.x - group * a.units;
  const int groups = kRopeThreads / a.units;
  if (group >= groups) return;
  const int head0 = blockIdx.y * a.heads_block;
  const int heads = min(a.heads_block, a.heads - head0);
  const T *x = static_cast<const T *>(a.x);
  T *out = static_cast<T *>(a.out);
  const int half = a.pairs;  // distance of a pair's features in the half layout
  for (int p = group; p < rows * heads; p += groups) {
    const int r = p / heads, h = head0 + p - r * heads;
    const T *xi = x + (row0 + r) * a.ldx + (int64_t)h * a.head_dim;
    T *oi = out + (row0 + r) * a.ldo + (int64_t)h * a.head_dim;
    const float2 *c = cs + r * a.pairs;
    if (unit >= a.rot_units) {
      const int f = 2 * a.pairs + (unit - a.rot_units) * VEC;
      *reinterpret_cast<Raw *>(oi + f) = *reinterpret_cast<const Raw *>(xi + f);
    } else if (IL && VEC > 1) {
      const int f = unit * VEC;
      float u[VEC];
      P::open(*reinterpret_cast<const Raw *>(xi + f), u);
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const float2 w = c[(f + i) / 2];
        const float va = u[i], vb = u[i + 1];
        u[i] = va * w.x - vb * w.y;
        u[i + 1] = vb * w.x + va * w.y;
      }
      *reinterpret_cast<Raw *>(oi + f) = P::close(u);
    } else {
      const int fa = IL ? 2 * unit : unit * VEC, fb = IL ? fa + 1 : fa + half;
      float u[VEC], v[VEC];
      P::open(*reinterpret_cast<const Raw *>(xi + fa), u);
      P::open(*reinterpret_cast<const Raw *>(xi + fb), v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float2 w = c[unit * VEC + i];
        const float va = u[i], vb = v[i];
        u[i] = va * w.x - vb * w.y;
        v[i] = vb * w.x + va * w.y;
      }
      *reinterpret_cast<Raw *>(oi + fa) = P::close(u);
      *reinterpret_cast<Raw *>(oi + fb) = P::close(v);
    }
  }
}

template <typename T>
cudaError_t launch(RopeArgs &a, bool interleaved, bool in_place, cudaStream_t st) {
  constexpr int kVec = Elem<T>::kVec;
  const uint64_t bytes = (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                          (uint64_t)a.ldx * sizeof(T) | (uint64_t)a.ldo * sizeof(T) |
                          (uint64_t)a.head_dim * sizeof(T));
  const int rest = a.head_dim - 2 * a.pairs;
  const bool wide = bytes % 16 == 0 && rest % kVec == 0 &&
                    (interleaved ? 2 * a.pairs : a.pairs) % kVec == 0;
  const int vec = wide ? kVec : 1;
  a.rot_units = interleaved && wide ? 2 * a.pairs / vec : a.pairs / vec;
  a.units = a.rot_units + (in_place ? 0 : rest / vec);
  const int groups = kRopeThreads / a.units;
  // A block's threads take about four heads each; its rows share the grid's other dimension when
  // one row has more than that.
  int64_t r = 4 * (int64_t)groups / a.heads;
  r = r < 1 ? 1 : r > kMaxRows ? kMaxRows : r;
  const int64_t spread = (a.rows + 2 * kSmCount - 1) / (2 * kSmCount);  // fill the SMs first
  if (r > spread) r = spread;
  a.rows_block = (int)r;
  a.heads_block = a.heads;
  if (r == 1 && a.heads > 4 * groups) a.heads_block = 4 * groups;
  const unsigned gy = (unsigned)((a.heads + a.heads_block - 1) / a.heads_block);
  const dim3 grid((unsigned)((a.rows + r - 1) / r), gy);
  if (interleaved) {
    if (wide) rope_kernel<T, true, kVec><<<grid, kRopeThreads, 0, st>>>(a);
    else rope_kernel<T, true, 1><<<grid, kRopeThreads, 0, st>>>(a);
  } else {
    if (wide) rope_kernel<T, false, kVec><<<grid, kRopeThreads, 0, st>>>(a);
    else rope_kernel<T, false, 1><<<grid, kRopeThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

// Why `c` is not a rotary configuration, or null.
const char *rope_cfg_error(const zo_rope_cfg &c) {
  if (!(c.theta > 0.f) || !std::isfinite(c.theta)) return "rope: theta must be finite and > 0";
  if (c.rot_dim < 2 || c.rot_dim > ZO_ROPE_MAX_HEAD_DIM || c.rot_dim % 2)
    return "rope: rot_dim must be even, in [2, 256]";
  if (c.interleaved != 0 && c.interleaved != 1) return "rope: interleaved must be 0 or 1";
  if (!std::isfinite(c.magnitude)) return "rope: magnitude must be finite";
  if (c.scaling == ZO_ROPE_PLAIN) return nullptr;
  if (c.scaling != ZO_ROPE_LINEAR && c.scaling != ZO_ROPE_BANDS) return "rope: unknown scaling";
  if (!(c.factor > 0.f) || !std::isfinite(c.factor)) return "rope: factor must be finite and > 0";
  if (c.scaling == ZO_ROPE_LINEAR) return nullptr;
  if (!(c.orig_len > 0.f) || !std::isfinite(c.orig_len)) return "rope: orig_len must be finite and > 0";
  if (!(c.band_low < c.band_high) || !std::isfinite(c.band_low) || !std::isfinite(c.band_high))
    return "rope: need band_low < band_high, both finite";
  return nullptr;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

// Frequency i of a valid configuration, radians per position.
double rope_frequency(const zo_rope_cfg &c, int i) {
  const double f = std::pow((double)c.theta, -2.0 * i / c.rot_dim);
  if (c.scaling == ZO_ROPE_LINEAR) return f / (double)c.factor;
  if (c.scaling == ZO_ROPE_BANDS) {
    const double turns = (double)c.orig_len * f / kTwoPi;
    double g = (turns - (double)c.band_low) / ((double)c.band_high - (double)c.band_low);
    g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
    return g * f + (1.0 - g) * f / (double)c.factor;
  }
  return f;
}

}  // namespace
}  // namespace zo

using namespace zo;

extern "C" {

zo_status zo_rope_frequencies(const zo_rope_cfg *cfg, double *radians) {
  if (!cfg || !radians || rope_cfg_error(*cfg)) return ZO_ERR_INVALID;
  for (int i = 0; i < cfg->rot_dim / 2; ++i) radians[i] = rope_frequency(*cfg, i);
  return ZO_OK;
}

zo_status zo_rope(zo_ctx *ctx, const void *x, void *out, int dtype, const int32_t *positions,
                  const zo_rope_cfg *cfg, int64_t rows, int64_t ldx, int64_t ldo, int32_t n_heads,
                  int32_t head_dim) {
  if (!ctx) return ZO_ERR_INVALID;
  ctx->err.clear();
  if (!x || !out || !cfg) return fail(ctx, ZO_ERR_INVALID, "null rope argument");
  if (const char *why = rope_cfg_error(*cfg)) return fail(ctx, ZO_ERR_INVALID, "%s", why);
  if (dtype != ZO_F32 && dtype != ZO_BF16) return fail(ctx, ZO_ERR_INVALID, "rope: dtype must be fp32 or bf16");
  if (head_dim < cfg->rot_dim || head_dim > ZO_ROPE_MAX_HEAD_DIM)
    return fail(ctx, ZO_ERR_INVALID, "rope: head_dim outside [rot_dim, %d]", ZO_ROPE_MAX_HEAD_DIM);
  if (rows < 1 || rows > INT32_MAX || n_heads < 1 || n_heads > 65535 || ldx < (int64_t)n_heads * head_dim ||
      ldo < (int64_t)n_heads * head_dim)
    return fail(ctx, ZO_ERR_INVALID, "rope: need 1 <= rows < 2^31, 1 <= n_heads <= 65535, row strides >= n_heads head_dim");
  const uintptr_t es = dtype == ZO_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) % es ||
      reinterpret_cast<uintptr_t>(positions) % 4)
    return fail(ctx, ZO_ERR_INVALID, "rope: pointers not aligned to their elements");
  if (x == out && ldx != ldo) return fail(ctx, ZO_ERR_INVALID, "rope: in place needs ldo == ldx");
  const DeviceScope device(ctx);
  if (device.status != cudaSuccess)
    return fail(ctx, ZO_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(device.status));
  RopeArgs a;
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.rows = rows;
  a.ldx = ldx;
  a.ldo = ldo;
  a.heads = n_heads;
  a.head_dim = head_dim;
  a.pairs = cfg->rot_dim / 2;
  a.magnitude = cfg->magnitude;
  for (int i = 0; i < kMaxPairs; ++i) a.turns[i] = i < a.pairs ? rope_frequency(*cfg, i) / kTwoPi : 0.0;
  const cudaError_t e = dtype == ZO_F32 ? launch<float>(a, cfg->interleaved != 0, x == out, ctx->stream)
                                        : launch<uint16_t>(a, cfg->interleaved != 0, x == out, ctx->stream);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "rope_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
}

}  // extern "C"
