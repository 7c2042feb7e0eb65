// zo_rope.cu -- rotary positions as an operator of its own (zo_rope):
//
//   t_i = positions[row] f_i,  (a, b) -> magnitude (a cos t_i - b sin t_i, b cos t_i + a sin t_i)
//
// for the rot_dim / 2 feature pairs of every head, in the half layout (i with i + rot_dim/2) or
// the interleaved one (2 i with 2 i + 1).  The frequencies, scaled for long contexts or not, are
// computed in fp64 on the host and travel as a kernel parameter.
//
// A group of threads covers one head, 16 bytes of each half (half layout) or 16 bytes (interleaved) a
// thread, and takes HEADS (4 or 8) heads of one row: their loads are under way before the thread computes
// the cosines and sines of its own pairs, once for those heads: position x (f_i / 2 pi) in fp64, the
// fraction of a turn kept (exact enough at any int32 position: the product carries 53 bits, at most
// 31 of them before the point), then sincospi in fp32.  Computing them again for every HEADS heads
// costs less than a block that computes them once, waits and shares them: 8192 rows of 24 heads of
// 128 took 22.3 us that way.
// Bound: HBM, two passes over the rotated heads.
#include <cmath>
#include <cstring>

#include "zo_internal.cuh"
#include "zo_tc.cuh"

namespace zo {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = ZO_ROPE_MAX_HEAD_DIM / 2;

struct RopeArgs {
  const void *x;
  void *out;
  const int32_t *positions;
  int64_t rows, ldx, ldo;
  int heads, head_dim, pairs;
  int units;      // threads that cover one head
  int rot_units;  // of them, those that rotate (the others copy features behind rot_dim)
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
template <typename T, bool IL, int VEC, int HEADS>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeArgs a) {
  using P = Pack<T, VEC>;
  using Raw = typename P::Raw;
  constexpr bool kOne = IL && VEC > 1;           // a pair's features lie in one access
  constexpr int kPairs = kOne ? VEC / 2 : VEC;  // of a unit
  tc::pdl_wait();
  const int group = threadIdx.x / a.units, unit = threadIdx.x - group * a.units;
  const int groups = kRopeThreads / a.units;
  const int64_t row = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * groups + group;
  if (group >= groups || row >= a.rows) return;
  const int head0 = blockIdx.x * HEADS, heads = min(HEADS, a.heads - head0);
  const bool turns = unit < a.rot_units;  // the other units copy features behind rot_dim
  // the unit's first access, and its second in the rotating part
  const int fa = !turns ? 2 * a.pairs + (unit - a.rot_units) * VEC : IL && VEC == 1 ? 2 * unit : unit * VEC;
  const int fb = IL ? fa + 1 : fa + a.pairs;
  const T *xi = static_cast<const T *>(a.x) + row * a.ldx + (int64_t)head0 * a.head_dim;
  T *oi = static_cast<T *>(a.out) + row * a.ldo + (int64_t)head0 * a.head_dim;
  const double pos = a.positions ? (double)a.positions[row] : (double)row;
  Raw first[HEADS], second[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h < heads) {
      first[h] = *reinterpret_cast<const Raw *>(xi + h * a.head_dim + fa);
      if (!kOne && turns) second[h] = *reinterpret_cast<const Raw *>(xi + h * a.head_dim + fb);
    }
  }
  if (!turns) {
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h < heads) *reinterpret_cast<Raw *>(oi + h * a.head_dim + fa) = first[h];
    return;
  }
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const double t = pos * a.turns[unit * kPairs + i];
    sincospif(2.f * (float)(t - rint(t)), &s[i], &c[i]);
    c[i] *= a.magnitude;
    s[i] *= a.magnitude;
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h < heads) {
      float u[VEC], v[VEC];
      P::open(first[h], u);
      if (kOne) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float va = u[2 * i], vb = u[2 * i + 1 < VEC ? 2 * i + 1 : 0];
          u[2 * i] = va * c[i] - vb * s[i];
          u[2 * i + 1 < VEC ? 2 * i + 1 : 0] = vb * c[i] + va * s[i];
        }
      } else {
        P::open(second[h], v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float va = u[i], vb = v[i];
          u[i] = va * c[i] - vb * s[i];
          v[i] = vb * c[i] + va * s[i];
        }
        *reinterpret_cast<Raw *>(oi + h * a.head_dim + fb) = P::close(v);
      }
      *reinterpret_cast<Raw *>(oi + h * a.head_dim + fa) = P::close(u);
    }
  }
}

template <typename T, bool IL, int VEC, int HEADS>
cudaError_t run(const RopeArgs &a, cudaStream_t st) {
  const int64_t groups = kRopeThreads / a.units, blocks = (a.rows + groups - 1) / groups;
  const int64_t y = blocks < 65535 ? blocks : 65535;  // row blocks over y and z
  const dim3 grid((unsigned)((a.heads + HEADS - 1) / HEADS), (unsigned)y, (unsigned)((blocks + y - 1) / y));
  return launch_early(rope_kernel<T, IL, VEC, HEADS>, grid, kRopeThreads, 0, st, a);
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
  // Heads of a group: 4 keep most loads in flight, 8 share the angles among more.  4 / 8, us: 8192 rows of
  // 24 heads of 128 17.3 / 17.7, 30000 of 2 of 256 19.1 / 22.6, but 29710 of 6 of 128 fp32 38 / 28.5, and
  // element by element 8192 of 24 of 128 50 / 41.
  const bool more = a.heads > 4 && (a.heads <= 8 || !wide);
  if (interleaved) {
    if (wide) return more ? run<T, true, kVec, 8>(a, st) : run<T, true, kVec, 4>(a, st);
    return more ? run<T, true, 1, 8>(a, st) : run<T, true, 1, 4>(a, st);
  }
  if (wide) return more ? run<T, false, kVec, 8>(a, st) : run<T, false, kVec, 4>(a, st);
  return more ? run<T, false, 1, 8>(a, st) : run<T, false, 1, 4>(a, st);
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

// The rot_dim / 2 frequencies of a valid configuration, radians per position: theta^(-2 i / rot_dim) as
// the product of one of 16 steps of eight i and one of eight steps of one (three roundings of
// 2^-53; the powers are most of what this call costs).
void rope_frequencies(const zo_rope_cfg &c, double *f) {
  double step[8];
  for (int i = 0; i < 8; ++i) step[i] = std::pow((double)c.theta, -2.0 * i / c.rot_dim);
  double block = 1.0;
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    if (i % 8 == 0) block = std::pow((double)c.theta, -2.0 * i / c.rot_dim);
    f[i] = block * step[i % 8];
    if (c.scaling == ZO_ROPE_LINEAR) f[i] /= (double)c.factor;
    if (c.scaling == ZO_ROPE_BANDS) {
      const double turns = (double)c.orig_len * f[i] / kTwoPi;
      double g = (turns - (double)c.band_low) / ((double)c.band_high - (double)c.band_low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f[i] = g * f[i] + (1.0 - g) * f[i] / (double)c.factor;
    }
  }
}

}  // namespace
}  // namespace zo

using namespace zo;

extern "C" {

zo_status zo_rope_frequencies(const zo_rope_cfg *cfg, double *radians) {
  if (!cfg || !radians || rope_cfg_error(*cfg)) return ZO_ERR_INVALID;
  rope_frequencies(*cfg, radians);
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
  rope_frequencies(*cfg, a.turns);
  for (int i = 0; i < a.pairs; ++i) a.turns[i] *= 1.0 / kTwoPi;
  const cudaError_t e = dtype == ZO_F32 ? launch<float>(a, cfg->interleaved != 0, x == out, ctx->stream)
                                        : launch<uint16_t>(a, cfg->interleaved != 0, x == out, ctx->stream);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "rope_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
}

}  // extern "C"
