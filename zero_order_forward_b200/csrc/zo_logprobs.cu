// zo_logprobs.cu -- log probabilities of given tokens, entropy and the largest alternatives from
// rows of logits (zo_logprobs), in one pass over the logits:
//
//   p_j = exp(x_j - lse),  lse = log sum_j exp(x_j),  logprob = x_t - lse,  H = lse - sum_j p_j x_j.
//
// A row is one block's, or, where rows are few, a cluster's of up to 8 blocks.  Every thread keeps,
// over the 16-byte vectors that it reads, m (its largest logit so far), s = sum 2^t and
// u = sum 2^t t with t = (x - m) log2 e; a larger maximum rescales both.  The triples are joined
// in a fixed order, so that H = ln 2 (log2 s - u / s) and logprob = (x_t - m) - ln 2 log2 s.  s is fp32
// over 4 vectors, u over a sixteenth of a thread's (or 4), and beyond, as the logarithm, fp64: with all of a
// thread's u in fp32 the entropy of 2^28 nearly equal logits was off by 3.1e-5, now by 4e-7, and 2048 rows
// of 151936 take 125.4 us instead of 124.2 (with u in fp64 from 4 vectors on 125.6; without alternatives, 4096
// rows, 221, 224 and 231).  The difference x - m is taken before the scaling, so that rows of huge logits
// lose and overflow nothing.
//
// Alternatives: a thread also keeps which of its vectors holds its largest logit first.  The
// top-th largest of the block's (value, vector) keys is a bound that at least `top` of its logits
// reach, and only threads whose own key reaches it can hold such logits: their vectors are read
// again (from L2) and what reaches the bound is sorted.  Keys are unique, so equal logits come
// in the order of their index.
#include <cmath>

#include "zo_internal.cuh"
#include "zo_tc.cuh"

namespace zo {
namespace {

constexpr float kLog2E = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994530942;
// t below -kLowest (a masked logit's is -inf) counts as that: 2^t is 0 all the same, and 0 t stays 0.
constexpr float kLowest = 1e30f;
constexpr int kMaxSplits = 8;  // blocks of a row (a portable cluster)
constexpr int kManyHot = 64;   // threads that reach the bound before it is made exact
constexpr int kGroups = 16;    // groups of consecutive vectors of a thread

// Rows of a block: a warp's rows need no barrier of the block, and blocks of one warp start too slowly.
__host__ __device__ constexpr int rows_of_block(int threads) { return threads == 32 ? 4 : 1; }

struct LogprobArgs {
  const void *logits;
  int64_t ld, rows;
  int vocab, top, splits;
  const int32_t *targets;
  float *logprob, *entropy;
  int32_t *top_ids;
  float *top_logprobs;
};

using tc::max_nan;

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
  static constexpr uint32_t kNone = 0xFF800000u;  // -inf, in every element of a 32-bit word
  static __device__ __forceinline__ float one(const float *p) { return __ldg(p); }
  static __device__ __forceinline__ void set(uint4 &r, int i, const float *p) {
    (&r.x)[i] = __float_as_uint(__ldg(p));
  }
  static __device__ __forceinline__ void open(const uint4 &r, float f[4]) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  // The largest element, NaN if there is one.
  static __device__ __forceinline__ float largest(const uint4 &r) {
    return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)),
                   max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
};
template <> struct Row<uint16_t> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  static __device__ __forceinline__ float one(const uint16_t *p) { return bf16_bits_to_f32(__ldg(p)); }
  static __device__ __forceinline__ void set(uint4 &r, int i, const uint16_t *p) {
    uint32_t &w = (&r.x)[i / 2];
    w = i & 1 ? (w & 0xFFFFu) | ((uint32_t)__ldg(p) << 16) : (w & 0xFFFF0000u) | __ldg(p);
  }
  static __device__ __forceinline__ void open(const uint4 &r, float f[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f[2 * t] = __uint_as_float(w[t] << 16);
      f[2 * t + 1] = __uint_as_float(w[t] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float largest(const uint4 &r) {
    const uint32_t m = max2(max2(r.x, r.y), max2(r.z, r.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
};

// Sums in fp64: where one token has nearly all the probability, s is 1 and a little, and the little is
// the entropy; fp32 joins left it off by 2e-6.
struct Stats {
  float m;      // see above; m = -inf: nothing yet (s = u = 0)
  double s, u;
};

// The lanes' triples joined, in every lane: the sums relative to the largest m, then added in a
// tree of fixed order.  top: the largest of the lanes', NaN if one is.
__device__ __forceinline__ void warp_join(Stats &t, float &top) {
  float m = t.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  const float d = fmaxf((t.m - m) * kLog2E, -kLowest), f = tc::ex2(d);  // (-inf) - (-inf): -kLowest
  t.u = f > 0.f ? (double)f * (t.u + (double)d * t.s) : 0.0;
  t.s *= (double)f;
  t.m = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, o);
    t.u += __shfl_xor_sync(0xFFFFFFFFu, t.u, o);
  }
}

// (d0, d1) = ((a0, a1) + b) * c, each operation rounded.
__device__ __forceinline__ void add_scale2(float a0, float a1, float b, float c, float &d0, float &d1) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmul.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b), "f"(c));
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

// Barrier over a row's threads, and the count of those whose `p` holds.
template <int THREADS>
__device__ __forceinline__ void row_sync() {
  if (THREADS == 32) __syncwarp();
  else __syncthreads();
}
template <int THREADS>
__device__ __forceinline__ int row_count(bool p) {
  return THREADS == 32 ? __popc(__ballot_sync(0xFFFFFFFFu, p)) : __syncthreads_count(p);
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
  __device__ __forceinline__ uint4 read_whole(int j) const {
    return __ldg(reinterpret_cast<const uint4 *>(p + first(j)));
  }
  // Vector j; elements outside the row read as -inf.
  __device__ __forceinline__ uint4 read(int j) const {
    const int e = first(j);
    if (e >= 0 && e + Row<T>::kVec <= vocab) return read_whole(j);
    uint4 r = make_uint4(Row<T>::kNone, Row<T>::kNone, Row<T>::kNone, Row<T>::kNone);
#pragma unroll
    for (int i = 0; i < Row<T>::kVec; ++i)
      if (e + i >= 0 && e + i < vocab) Row<T>::set(r, i, p + e + i);
    return r;
  }
};

// What one thread has seen.
template <typename T>
struct Scan {
  static constexpr int V = Row<T>::kVec;
  float top = -INFINITY;  // its largest logit (NaN once it has seen one)
  int top_vec;            // the first vector that holds it
  float m = -INFINITY, u = 0.f;  // u: since the last flush
  double s = 0.0, u_sum = 0.0;

  __device__ __forceinline__ void flush() {
    u_sum += (double)u;
    u = 0.f;
  }

  template <int U>
  __device__ __forceinline__ float take(const uint4 (&r)[U], int j, int step) {  // returns the largest
    float all = -INFINITY;
#pragma unroll
    for (int g = 0; g < U; ++g) {
      const float v = Row<T>::largest(r[g]);
      all = max_nan(all, v);
      if (v > top || (v != v && top == top)) {
        top = v;
        top_vec = j + g * step;
      }
    }
    if (!(top > -INFINITY)) return all;
    if (top > m) {
      if (m != -INFINITY) {
        const float d = fmaxf((m - top) * kLog2E, -kLowest), e = tc::ex2(d);
        u_sum = (double)e * (u_sum + (double)d * s);
        u *= e;
        s *= (double)e;
      }
      m = top;
    }
    float s4[4] = {}, u4[4] = {};  // of these U vectors, in four chains
#pragma unroll
    for (int g = 0; g < U; ++g) {
      float f[V];
      Row<T>::open(r[g], f);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        float t0, t1;
        add_scale2(f[i], f[i + 1], -m, kLog2E, t0, t1);
        t0 = fmaxf(t0, -kLowest);
        t1 = fmaxf(t1, -kLowest);
        const float p0 = tc::ex2(t0), p1 = tc::ex2(t1);
        constexpr int kPairs = 2;
        const int h = (i / 2) % kPairs * 2;
        tc::add2(s4[h], s4[h + 1], p0, p1);
        tc::fma2(u4[h], u4[h + 1], p0, p1, t0, t1);
      }
    }
    s += (double)((s4[0] + s4[1]) + (s4[2] + s4[3]));
    u += (u4[0] + u4[1]) + (u4[2] + u4[3]);
    return all;
  }
};

// Shared memory of a block; `row_*` are of use in a row's first block.
template <int THREADS>
struct Shared {
  static constexpr int WARPS = THREADS / 32;
  // logits that may reach the bound before the slow selection: 8 of every thread at most
  static constexpr int kCandidates = THREADS < 128 ? 8 * THREADS : 1024;
  Stats warp_stats[WARPS];
  float warp_top[WARPS];
  uint64_t list[WARPS][32];
  uint64_t cand[kCandidates];
  uint64_t bound;
  uint16_t group_top[kGroups][THREADS];  // order prefix of a group's largest logit
  uint16_t hot[kManyHot * kGroups];      // threads, or thread + THREADS * group
  int n_hot, n_cand;
  Stats row_stats[kMaxSplits];
  float row_top[kMaxSplits];
  uint64_t row_list[kMaxSplits][32];
};

template <typename V>
__device__ __forceinline__ void put_first(V *p, const V &v) {  // p's counterpart in the cluster's block 0
  static_assert(sizeof(V) % 4 == 0, "words");
  const uint32_t at = tc::map_to_rank(p, 0);
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i) tc::st_remote_u32(at + 4 * i, w[i]);
}

// THREADS threads a block, `splits` blocks (a cluster, if more than one) a row.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS * rows_of_block(THREADS), 1024 / (THREADS * rows_of_block(THREADS)))
logprobs_kernel(const LogprobArgs a) {
  constexpr int V = Row<T>::kVec, WARPS = THREADS / 32, U = 4;
  constexpr int kMany = THREADS == 32 ? 26 : kManyHot;  // (nearly all lanes of a warp)
  using Sh = Shared<THREADS>;
  __shared__ Sh shared[rows_of_block(THREADS)];
  Sh &sh = shared[threadIdx.y];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = a.splits > 1 ? (int)(blockIdx.x % (unsigned)a.splits) : 0;
  const int64_t r = rows_of_block(THREADS) * (int64_t)(a.splits > 1 ? blockIdx.x / (unsigned)a.splits : blockIdx.x) +
                    threadIdx.y;
  if (rows_of_block(THREADS) > 1 && r >= a.rows) return;
  const RowView<T> row(static_cast<const T *>(a.logits) + r * a.ld, a.vocab);
  const int j_first = (int)((int64_t)row.vectors * part / a.splits);
  const int j_end = (int)((int64_t)row.vectors * (part + 1) / a.splits);
  if (tid == 0) sh.n_hot = sh.n_cand = 0;
  if (THREADS == 32) __syncwarp();  // (the votes of a warp's selection do not order memory, barriers do)
  if (a.splits > 1) tc::cluster_arrive();  // block 0 has to run before its memory is written
  tc::pdl_wait();
  // the given token's logit, wanted at the end
  int32_t target = -1;
  float target_logit = 0.f;
  if (tid == 0 && part == 0 && a.logprob) {
    target = a.targets[r];
    if (target >= 0 && target < a.vocab) target_logit = Row<T>::one(row.p + target);
  }

  // ---- one pass: statistics, and the thread's largest logit with its vector.  The next U vectors
  // are on their way while U are worked on.  Only the first and the last vector of a row may be
  // cut off by it.
  Scan<T> scan;
  int j = j_first + tid;
  scan.top_vec = j < j_end ? j : -1;
  const bool cut = j_end == row.vectors && row.first(row.vectors - 1) + V > a.vocab;
  const int j_whole = cut ? j_end - 1 : j_end;
  const int group_rounds = ((j_end - j_first - 1) / (U * THREADS) + kGroups) / kGroups;  // rounds of U a group
  int round = 0, group = 0;
  float group_top = -INFINITY;
  uint4 next[U];
  if (j + (U - 1) * THREADS < j_whole) {
    next[0] = row.read(j);
#pragma unroll
    for (int g = 1; g < U; ++g) next[g] = row.read_whole(j + g * THREADS);
  }
  for (; j + (U - 1) * THREADS < j_whole; j += U * THREADS) {
    uint4 cur[U];
#pragma unroll
    for (int g = 0; g < U; ++g) cur[g] = next[g];
    if (j + (2 * U - 1) * THREADS < j_whole) {
#pragma unroll
      for (int g = 0; g < U; ++g) next[g] = row.read_whole(j + (U + g) * THREADS);
    }
    group_top = max_nan(group_top, scan.template take<U>(cur, j, THREADS));
    if (++round == group_rounds) {
      scan.flush();
      sh.group_top[group++][tid] = (uint16_t)(order_of(group_top) >> 16);
      group_top = -INFINITY;
      round = 0;
    }
  }
  if (j < j_end) {  // at most U left: their loads together, too
    uint4 last[U];
#pragma unroll
    for (int g = 0; g < U; ++g)
      if (j + g * THREADS < j_end) last[g] = row.read(j + g * THREADS);
#pragma unroll
    for (int g = 0; g < U; ++g) {
      if (j + g * THREADS < j_end) {
        const uint4 one[1] = {last[g]};
        group_top = max_nan(group_top, scan.template take<1>(one, j + g * THREADS, THREADS));
      }
    }
    ++round;
  }
  if (round) sh.group_top[group++][tid] = (uint16_t)(order_of(group_top) >> 16);

  // ---- the statistics of the block's part
  float top = scan.top;
  scan.flush();
  Stats st{scan.m, scan.s, scan.u_sum};
  warp_join(st, top);
  if (lane == 0) {
    sh.warp_stats[warp] = st;
    sh.warp_top[warp] = top;
  }

  // ---- alternatives of the block's part: the bound, then the logits that reach it
  uint64_t k = 0;
  if (a.top != 0) {
    const uint64_t mine = scan.top_vec < 0 ? 0 : key_of(order_of(scan.top), (uint32_t)scan.top_vec);
    // the largest 16-bit prefix of an order that the keys of `top` threads reach, if that many have one
    uint32_t prefix = 0;
    int reach = THREADS;
#pragma unroll 1
    for (uint32_t bit = 0x8000u; bit != 0; bit >>= 1) {
      const int n = row_count<THREADS>((uint32_t)(mine >> 48) >= (prefix | bit));
      if (n >= a.top) {
        prefix |= bit;
        reach = n;
      }
    }
    // The prefix alone is the bound, unless many threads or too many logits reach it: then the exact key.
    bool exact = reach > kMany;
#pragma unroll 1
    while (true) {
      uint64_t bound = (uint64_t)prefix << 48;
      if (exact) {
        k = block_merge<WARPS>(warp_sort(mine), sh.list);
        if (warp == 0 && lane == a.top - 1) sh.bound = k;
        row_sync<THREADS>();
        bound = sh.bound;  // 0: fewer threads than that have any logit
      }
      // vector jj again: its logits that reach the bound
      auto gather = [&](int jj) {
        float f[V];
        Row<T>::open(row.read(jj), f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const uint32_t o = order_of(f[e]);
          const int index = row.first(jj) + e;
          if (key_of(o, (uint32_t)jj) >= bound && index >= 0 && index < a.vocab) {
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < Sh::kCandidates) sh.cand[at] = key_of(o, (uint32_t)index);
          }
        }
      };
      if (exact) {
        if (mine != 0 && mine >= bound) sh.hot[atomicAdd(&sh.n_hot, 1)] = (uint16_t)tid;
        row_sync<THREADS>();
        for (int i = warp; i < sh.n_hot; i += WARPS)
          for (int jj = j_first + sh.hot[i] + lane * THREADS; jj < j_end; jj += 32 * THREADS) gather(jj);
      } else {
        if (mine != 0 && mine >= bound)
          for (int g = 0; g < group; ++g)
            if (sh.group_top[g][tid] >= prefix) sh.hot[atomicAdd(&sh.n_hot, 1)] = (uint16_t)(tid + THREADS * g);
        row_sync<THREADS>();
        const int per = U * group_rounds;  // vectors of a group
        for (int i = tid; i < sh.n_hot * per; i += THREADS) {
          const int h = sh.hot[i / per];
          const int jj = j_first + h % THREADS + (h / THREADS * per + i % per) * THREADS;
          if (jj < j_end) gather(jj);
        }
      }
      row_sync<THREADS>();
      if (exact || sh.n_cand <= Sh::kCandidates) break;
      row_sync<THREADS>();
      if (tid == 0) sh.n_hot = sh.n_cand = 0;
      row_sync<THREADS>();
      exact = true;
    }
    const int n_list = sh.n_cand;
    if (n_list > 32) {
      if (n_list <= Sh::kCandidates) {
        k = 0;
        for (int i = warp * 32; i < n_list; i += THREADS) {
          const uint64_t c = warp_sort(i + lane < n_list ? sh.cand[i + lane] : 0);
          k = warp_merge(k, c);
        }
        k = block_merge<WARPS>(k, sh.list);
      } else {
        // more than that reach the bound: take the largest key below the last one, `top` times
        uint64_t last = ~0ull, got = 0;
        for (int n = 0; n < a.top; ++n) {
          uint64_t best = 0;
          for (int jj = j_first + tid; jj < j_end; jj += THREADS) {
            float f[V];
            Row<T>::open(row.read(jj), f);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const int index = row.first(jj) + e;
              const uint64_t c = key_of(order_of(f[e]), (uint32_t)index);
              if (index >= 0 && index < a.vocab && c < last && c > best) best = c;
            }
          }
          best = block_merge<WARPS>(warp_sort(best), sh.list);
          if (tid == 0) sh.bound = best;
          row_sync<THREADS>();
          last = sh.bound;
          row_sync<THREADS>();
          if (warp == 0 && lane == n) got = last;
        }
        k = got;
      }
    } else if (warp == 0) {
      k = lane < n_list ? sh.cand[lane] : 0;
    }
  } else {
    row_sync<THREADS>();  // warp_stats
  }

  // ---- the row: its parts' statistics and alternatives meet in block 0
  if (warp == 0) {
    if (WARPS > 1) {
      st = lane < WARPS ? sh.warp_stats[lane] : Stats{-INFINITY, 0.0, 0.0};
      top = lane < WARPS ? sh.warp_top[lane] : -INFINITY;
      warp_join(st, top);
    }
  }
  if (a.splits > 1) {
    __syncwarp();
    tc::cluster_wait();
    if (warp == 0) {
      if (lane == 0) {
        put_first(&sh.row_stats[part], st);
        put_first(&sh.row_top[part], top);
      }
      if (a.top != 0) put_first(&sh.row_list[part][lane], k);
    }
    __syncwarp();
    tc::cluster_sync();
    if (part != 0) return;
    if (a.top != 0) {
      if (WARPS >= kMaxSplits) {
        k = warp_sort(warp < a.splits ? sh.row_list[warp][lane] : 0);
        k = block_merge<WARPS>(k, sh.list);
      } else if (warp == 0) {
        k = 0;
        for (int i = 0; i < a.splits; ++i) k = warp_merge(k, warp_sort(sh.row_list[i][lane]));
      }
    }
    if (warp != 0) return;
    st = lane < a.splits ? sh.row_stats[lane] : Stats{-INFINITY, 0.0, 0.0};
    top = lane < a.splits ? sh.row_top[lane] : -INFINITY;
    warp_join(st, top);
  } else {
    if (warp != 0) return;
    if (a.top != 0 && sh.n_cand <= 32) k = warp_sort(k);
  }
  top = __shfl_sync(0xFFFFFFFFu, top, 0);
  const bool none = !(top > -INFINITY) || top == INFINITY;
  const double nan = __longlong_as_double(0x7FF8000000000000ll);
  const double log2s = none ? nan : log2(__shfl_sync(0xFFFFFFFFu, st.s, 0));
  const double big = (double)__shfl_sync(0xFFFFFFFFu, st.m, 0);
  if (lane == 0) {
    if (a.entropy) a.entropy[r] = (float)(kLn2 * (log2s - st.u / st.s));
    if (a.logprob) {
      float v = (float)nan;
      if (target == -1) v = 0.f;
      else if (target >= 0 && target < a.vocab) v = (float)((double)target_logit - big - kLn2 * log2s);
      a.logprob[r] = v;
    }
  }
  if (lane < a.top) {
    const float x = value_of((uint32_t)(k >> 32));
    if (a.top_ids) a.top_ids[r * a.top + lane] = (int32_t)index_of(k);
    if (a.top_logprobs) a.top_logprobs[r * a.top + lane] = (float)((double)x - big - kLn2 * log2s);
  }
}

template <typename T, int THREADS>
cudaError_t launch_one(const LogprobArgs &a, int64_t rows, cudaStream_t st) {
  constexpr int kRows = rows_of_block(THREADS);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.splits > 1 ? rows * a.splits : (rows + kRows - 1) / kRows));
  cfg.blockDim = dim3(THREADS, kRows);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];  // may start before its predecessor's end (pdl_wait); clusters
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return taken(cudaLaunchKernelEx(&cfg, logprobs_kernel<T, THREADS>, a));
}

template <typename T>
cudaError_t launch(LogprobArgs &a, int64_t rows, cudaStream_t st) {
  const int vectors = (a.vocab + Row<T>::kVec - 1) / Row<T>::kVec;
  a.splits = 1;
  // several blocks a row while that leaves SMs to fill and every thread has a vector
  while (a.splits < kMaxSplits && rows * a.splits <= kSmCount && vectors >= 2 * a.splits * 256) a.splits *= 2;
  // As few threads a row as still fill the SMs with loads (148 x 32 warps fit): a row's joins and
  // selection cost about the same on a warp as on 8, which also wait for one another, but a warp's bound
  // lets more candidates of a long row through.  bf16, 5 alternatives, on 32 / 128 / 256 threads:
  // 12000 x 4000 42 / 78 / 129 us, 1000 x 4000 12 / 8.2 / 12, 30 x 20000 9.9 / 9.5 / 7.1; fp32, 20
  // alternatives, 509 x 49999: 128 threads 38, 256 25.
  if (rows >= 4000 && vectors < 2048) return launch_one<T, 32>(a, rows, st);
  if (rows >= 6 * kSmCount || vectors < 1024) return launch_one<T, 128>(a, rows, st);
  return launch_one<T, 256>(a, rows, st);
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
  if (rows < 1 || rows > INT32_MAX || vocab < 1 || vocab > INT32_MAX - 16 || ld < vocab || ld > INT32_MAX)
    return fail(ctx, ZO_ERR_INVALID, "logprobs: need 1 <= rows < 2^31, 1 <= vocab < 2^31 - 16, vocab <= ld < 2^31");
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
  LogprobArgs a{logits, ld, rows, (int)vocab, top_ids || top_logprobs ? top : 0, 1, targets, logprob, entropy,
                top_ids, top_logprobs};
  const cudaError_t e = dtype == ZO_F32 ? launch<float>(a, rows, ctx->stream)
                                        : launch<uint16_t>(a, rows, ctx->stream);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "logprobs_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
}
