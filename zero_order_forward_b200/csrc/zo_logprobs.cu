// zo_logprobs.cu -- log probabilities of given tokens, entropy and the largest alternatives from
// rows of logits (zo_logprobs), in one pass over the logits:
//
//   p_j = exp(x_j - lse),  lse = log sum_j exp(x_j),  logprob = x_t - lse,  H = lse - sum_j p_j x_j.
//
// One block per row.  Every thread keeps, over the 16-byte vectors that it reads, a reference m
// (the largest logit so far times log2 e), s = sum 2^(x log2 e - m) and
// u = sum 2^(x log2 e - m) (x log2 e - m); a larger maximum rescales both.  The block joins the
// threads' triples in a fixed order, so that H = ln 2 (log2 s - u / s) and
// logprob = ln 2 (x_t log2 e - m - log2 s); the logarithms are fp64, once per row.
//
// Alternatives: a thread also keeps which of its vectors holds its largest logit first.  The
// top-th largest of the threads' (value, vector) keys is a bound that at least `top` logits of
// the row reach, and only threads whose own key reaches it can hold such logits: their vectors
// are read again (from L2) and what reaches the bound is sorted.  Keys are unique, so equal
// logits come in the order of their index.
#include <cmath>

#include "zo_internal.cuh"
#include "zo_tc.cuh"

namespace zo {
namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994530942;
// Logits below -kLowest count as that in the fast sums: 2^(x log2 e - m) is 0 all the same, and
// 0 (x log2 e - m) stays 0 (not 0 * inf).  The rounding of m cancels, but 2^ of it must stay in
// range: a row whose largest logit is kHuge or more in magnitude takes the exact form
// (row_stats_huge), and a thread whose own largest is -kHuge or less adds nothing.
constexpr float kLowest = 1e30f, kHuge = 1e8f;
constexpr int kCandidates = 1024;  // logits that may reach the bound before the slow selection

struct LogprobArgs {
  const void *logits;
  int64_t ld;
  int vocab, top;
  const int32_t *targets;
  float *logprob, *entropy;
  int32_t *top_ids;
  float *top_logprobs;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Order of fp32 values as unsigned integers: NaN above +inf, -0 and +0 equal.
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
// Larger value first, then smaller index; 0 is below every key, ~0 above.
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) {
  return ((uint64_t)order << 32) | (0xFFFFFFFEu - index);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xFFFFFFFEu - (uint32_t)key; }

template <typename T> struct Row;
template <> struct Row<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float one(const float *p) { return __ldg(p); }
  static __device__ __forceinline__ void vec(const float *p, float f[4]) {
    const float4 r = __ldg(reinterpret_cast<const float4 *>(p));
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  }
};
template <> struct Row<uint16_t> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float one(const uint16_t *p) { return bf16_bits_to_f32(__ldg(p)); }
  static __device__ __forceinline__ void vec(const uint16_t *p, float f[8]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f[2 * t] = __uint_as_float(w[t] << 16);
      f[2 * t + 1] = __uint_as_float(w[t] & 0xFFFF0000u);
    }
  }
};

struct Stats {
  float m, s, u;  // see above; m = -inf: nothing yet (s = u = 0)
};

// Joins two triples (order matters only in the last bits).
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b) {
  const float m = max_nan(a.m, b.m);
  if (m == -INFINITY) return a;
  const float da = a.m - m, db = b.m - m;  // one of them 0; -inf where a side is empty
  const float fa = tc::ex2(da), fb = tc::ex2(db);
  Stats r;
  r.m = m;
  r.s = a.s * fa + b.s * fb;
  r.u = (fa > 0.f ? fa * (a.u + da * a.s) : 0.f) + (fb > 0.f ? fb * (b.u + db * b.s) : 0.f);
  return r;
}

// Descending bitonic sort of one key per lane.
__device__ __forceinline__ uint64_t warp_sort(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, k, stride);
      const bool larger = ((lane & stride) == 0) == ((lane & size) == 0);
      k = (k > o) == larger ? k : o;
    }
  }
  return k;
}
// The 32 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t warp_merge(uint64_t a, uint64_t b) {
  const int lane = threadIdx.x & 31;
  const uint64_t r = __shfl_sync(0xFFFFFFFFu, b, 31 - lane);
  uint64_t k = a > r ? a : r;
#pragma unroll
  for (int stride = 16; stride > 0; stride >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, k, stride);
    k = (k > o) == ((lane & stride) == 0) ? k : o;
  }
  return k;
}

// The 32 largest of all warps' sorted lists, in lanes of warp 0 (descending).  All threads call.
template <int WARPS>
__device__ __forceinline__ uint64_t block_merge(uint64_t k, uint64_t (*list)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int n = WARPS; n > 1; n >>= 1) {
    if (warp >= n / 2 && warp < n) list[warp][lane] = k;
    __syncthreads();
    if (warp < n / 2) k = warp_merge(k, list[warp + n / 2][lane]);
    __syncthreads();
  }
  return k;
}

// One row of `vocab` logits as vectors of kVec elements at 16-byte addresses: vector j covers
// elements j kVec - skew .. + kVec - 1; the first and the last may be cut off by the row.
template <typename T>
struct RowView {
  const T *p;
  int vocab, skew, vectors;
  __device__ RowView(const T *row, int n) : p(row), vocab(n) {
    skew = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    vectors = (n + skew + Row<T>::kVec - 1) / Row<T>::kVec;
  }
  __device__ __forceinline__ int first(int j) const { return j * Row<T>::kVec - skew; }
  __device__ __forceinline__ bool whole(int j) const {
    return first(j) >= 0 && first(j) + Row<T>::kVec <= vocab;
  }
  // Elements of vector j; those outside the row read as -inf.
  __device__ __forceinline__ void read(int j, float f[Row<T>::kVec]) const {
    const int e = first(j);
    if (whole(j)) {
      Row<T>::vec(p + e, f);
    } else {
#pragma unroll
      for (int i = 0; i < Row<T>::kVec; ++i)
        f[i] = e + i >= 0 && e + i < vocab ? Row<T>::one(p + e + i) : -INFINITY;
    }
  }
};

// The sums of a row whose largest logit `top` is kHuge or more in magnitude and finite: differences first,
// so that nothing overflows (rare; every thread over its own vectors, then joined as usual).
template <typename T, int THREADS>
__device__ __noinline__ Stats row_stats_huge(const RowView<T> &row, float top) {
  constexpr int V = Row<T>::kVec;
  Stats st{0.f, 0.f, 0.f};
  for (int j = threadIdx.x; j < row.vectors; j += THREADS) {
    float f[V];
    row.read(j, f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float t = (f[i] - top) * kLog2E, p = tc::ex2(t);
      if (p > 0.f) {
        st.s += p;
        st.u = fmaf(p, t, st.u);
      }
    }
  }
  return st;
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS)
logprobs_kernel(const LogprobArgs a) {
  constexpr int V = Row<T>::kVec, WARPS = THREADS / 32, U = 4;
  __shared__ Stats warp_stats[WARPS];
  __shared__ uint64_t list[WARPS][32];
  __shared__ uint64_t cand[kCandidates];
  __shared__ uint64_t s_bound;
  __shared__ int hot[THREADS];
  __shared__ int n_hot, n_cand;
  __shared__ float s_top;
  __shared__ double s_lse2;  // log2 of the sum of 2^(x log2 e)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t r = blockIdx.x;
  const RowView<T> row(static_cast<const T *>(a.logits) + r * a.ld, a.vocab);
  if (tid == 0) n_hot = n_cand = 0;

  // ---- one pass: statistics, and the thread's largest logit with its vector
  float top = -INFINITY;  // largest logit of this thread (NaN once it has seen one)
  int top_vec = -1;
  Stats st{-INFINITY, 0.f, 0.f};
  auto take = [&](const float (&f)[U][V], const int (&jv)[U], int n) {
#pragma unroll
    for (int g = 0; g < U; ++g) {
      if (g < n) {
        float vm = f[g][0];
#pragma unroll
        for (int i = 1; i < V; ++i) vm = max_nan(vm, f[g][i]);
        if (top_vec < 0 || (!(vm <= top) && top == top)) {
          top = vm;
          top_vec = jv[g];
        }
      }
    }
    if (!(top > -kHuge)) return;
    const float ref = top * kLog2E;
    if (ref > st.m) {
      if (st.m != -INFINITY) {
        const float d = st.m - ref, e = tc::ex2(d);
        st.u = e * (st.u + d * st.s);
        st.s *= e;
      }
      st.m = ref;
    }
#pragma unroll
    for (int g = 0; g < U; ++g) {
      if (g < n) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float t = fmaf(max_nan(f[g][i], -kLowest), kLog2E, -st.m), p = tc::ex2(t);
          st.s += p;
          st.u = fmaf(p, t, st.u);
        }
      }
    }
  };
  int j = tid;
  for (; j + (U - 1) * THREADS < row.vectors; j += U * THREADS) {
    float f[U][V];
    int jv[U];
#pragma unroll
    for (int g = 0; g < U; ++g) {
      jv[g] = j + g * THREADS;
      row.read(jv[g], f[g]);
    }
    take(f, jv, U);
  }
  for (; j < row.vectors; j += THREADS) {
    float f[U][V];
    const int jv[U] = {j, 0, 0, 0};
    row.read(j, f[0]);
    take(f, jv, 1);
  }

  // ---- the row's statistics
  float rmax = top_vec < 0 ? -INFINITY : top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rmax = max_nan(rmax, __shfl_xor_sync(0xFFFFFFFFu, rmax, o));
  if (lane == 0) warp_stats[warp].m = rmax;
  __syncthreads();
  if (tid == 0) {
    float m = warp_stats[0].m;
    for (int w = 1; w < WARPS; ++w) m = max_nan(m, warp_stats[w].m);
    s_top = m;
  }
  __syncthreads();
  const float row_top = s_top;
  const bool huge = fabsf(row_top) >= kHuge && fabsf(row_top) < INFINITY;
  if (huge) st = row_stats_huge<T, THREADS>(row, row_top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stats b;
    b.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
    b.s = __shfl_xor_sync(0xFFFFFFFFu, st.s, o);
    b.u = __shfl_xor_sync(0xFFFFFFFFu, st.u, o);
    st = lane & o ? join(b, st) : join(st, b);
  }
  if (lane == 0) warp_stats[warp] = st;
  __syncthreads();
  if (tid == 0) {
    Stats t = warp_stats[0];
    for (int w = 1; w < WARPS; ++w) t = join(t, warp_stats[w]);
    // the distribution's logarithm, relative to the row's largest logit where that is huge
    const bool none = !(row_top > -INFINITY) || row_top == INFINITY;
    const double nan = __longlong_as_double(0x7FF8000000000000ll);
    const double lse2 = none ? nan : (double)t.m + log2((double)t.s);
    s_lse2 = lse2;
    if (a.entropy) a.entropy[r] = none ? (float)nan : (float)(kLn2 * (log2((double)t.s) - (double)t.u / (double)t.s));
    if (a.logprob) {
      const int32_t g = a.targets[r];
      float v = (float)nan;
      if (g == -1) v = 0.f;
      else if (g >= 0 && g < a.vocab) {
        const float x = Row<T>::one(row.p + g);
        v = huge ? (float)((double)x - (double)row_top - kLn2 * lse2)
                 : (float)(kLn2 * ((double)x * (double)kLog2E - lse2));
      }
      a.logprob[r] = v;
    }
  }
  if (a.top == 0) return;

  // ---- alternatives: the bound, the logits that reach it, the largest of them in order
  uint64_t k = top_vec < 0 ? 0 : key_of(order_of(top), (uint32_t)top_vec);
  const uint64_t mine = k;
  k = block_merge<WARPS>(warp_sort(k), list);
  if (warp == 0 && lane == a.top - 1) s_bound = k;
  __syncthreads();
  const uint64_t bound = s_bound;  // 0: fewer threads than that have any logit
  if (mine != 0 && mine >= bound) hot[atomicAdd(&n_hot, 1)] = tid;
  __syncthreads();
  for (int i = warp; i < n_hot; i += WARPS) {
    for (int jj = hot[i] + lane * THREADS; jj < row.vectors; jj += 32 * THREADS) {
      float f[V];
      row.read(jj, f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const uint32_t o = order_of(f[e]);
        const int index = row.first(jj) + e;
        if (key_of(o, (uint32_t)jj) >= bound && index >= 0 && index < a.vocab) {
          const int at = atomicAdd(&n_cand, 1);
          if (at < kCandidates) cand[at] = key_of(o, (uint32_t)index);
        }
      }
    }
  }
  __syncthreads();
  if (n_cand <= kCandidates) {
    k = 0;
    for (int i = warp * 32; i < n_cand; i += THREADS) {
      const uint64_t c = warp_sort(i + lane < n_cand ? cand[i + lane] : 0);
      k = warp_merge(k, c);
    }
    k = block_merge<WARPS>(k, list);
  } else {
    // more than that reach the bound: take the largest key below the last one, `top` times
    uint64_t last = ~0ull, got = 0;
    for (int n = 0; n < a.top; ++n) {
      uint64_t best = 0;
      for (int jj = tid; jj < row.vectors; jj += THREADS) {
        float f[V];
        row.read(jj, f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int index = row.first(jj) + e;
          const uint64_t c = key_of(order_of(f[e]), (uint32_t)index);
          if (index >= 0 && index < a.vocab && c < last && c > best) best = c;
        }
      }
      best = block_merge<WARPS>(warp_sort(best), list);
      if (tid == 0) s_bound = best;
      __syncthreads();
      last = s_bound;
      __syncthreads();
      if (warp == 0 && lane == n) got = last;
    }
    k = got;
  }
  if (warp == 0 && lane < a.top) {
    const float x = value_of((uint32_t)(k >> 32));
    if (a.top_ids) a.top_ids[r * a.top + lane] = (int32_t)index_of(k);
    if (a.top_logprobs)
      a.top_logprobs[r * a.top + lane] =
          huge ? (float)((double)x - (double)row_top - kLn2 * s_lse2)
               : (float)(kLn2 * ((double)x * (double)kLog2E - s_lse2));
  }
}

template <typename T>
cudaError_t launch(const LogprobArgs &a, int64_t rows, cudaStream_t st) {
  if (a.vocab >= 8192) logprobs_kernel<T, 512><<<(unsigned)rows, 512, 0, st>>>(a);
  else logprobs_kernel<T, 128><<<(unsigned)rows, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace zo

using namespace zo;

extern "C" zo_status zo_logprobs(zo_ctx *ctx, const void *logits, int dtype, int64_t rows, int64_t vocab,
                                 int64_t ld, const int32_t *targets, float *logprob, float *entropy,
                                 int32_t top, int32_t *top_ids, float *top_logprobs) {
  if (!ctx) return ZO_ERR_INVALID;
  ctx->err.clear();
  if (!logits || (logprob && !targets)) return fail(ctx, ZO_ERR_INVALID, "null logprobs argument");
  if (dtype != ZO_F32 && dtype != ZO_BF16)
    return fail(ctx, ZO_ERR_INVALID, "logprobs: dtype must be fp32 or bf16");
  if (rows < 1 || rows > INT32_MAX || vocab < 1 || ld < vocab || ld > INT32_MAX)
    return fail(ctx, ZO_ERR_INVALID, "logprobs: need 1 <= rows < 2^31, 1 <= vocab <= ld < 2^31");
  if (top < 0 || top > ZO_MAX_TOP || top > vocab)
    return fail(ctx, ZO_ERR_INVALID, "logprobs: top outside [0, min(%d, vocab)]", ZO_MAX_TOP);
  if (!logprob && !entropy && (top == 0 || (!top_ids && !top_logprobs)))
    return fail(ctx, ZO_ERR_INVALID, "logprobs: no output");
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == ZO_F32 ? 4 : 2) ||
      (reinterpret_cast<uintptr_t>(targets) | reinterpret_cast<uintptr_t>(logprob) |
       reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(top_ids) |
       reinterpret_cast<uintptr_t>(top_logprobs)) % 4)
    return fail(ctx, ZO_ERR_INVALID, "logprobs: pointers not aligned to their elements");
  const DeviceScope device(ctx);
  if (device.status != cudaSuccess)
    return fail(ctx, ZO_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(device.status));
  const LogprobArgs a{logits, ld, (int)vocab, top_ids || top_logprobs ? top : 0, targets, logprob, entropy,
                      top_ids, top_logprobs};
  const cudaError_t e = dtype == ZO_F32 ? launch<float>(a, rows, ctx->stream)
                                        : launch<uint16_t>(a, rows, ctx->stream);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "logprobs_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
}
