// zo_attn_packed.cu -- causal grouped-query attention within packed sequences of different
// lengths (zo_attention_packed), on the tensor cores; forward only:
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   over the rows j of i's own sequence.
//
// One CTA of 12 warps per SM takes items, one after another: two streams of 128 query rows each that
// share key and value tiles of 128 keys,
//   kHeads  two query heads of one key/value head (an even number of them share it),
//   kPair64 two heads of dim 64 with their own key/value heads, which lie side by side in the rows,
//   kRows   256 rows of one head otherwise.
// A warp issues the TMA loads, one the MMAs (S = Q K^T into tensor memory, O += P V with P read from
// tensor memory, where it replaces S), and four per stream compute the softmax, one query row per
// thread: while one stream's exponentials run, the tensor cores work on the other's products.  Two
// streams of 128 x 128 scores take all 512 columns of tensor memory (hd 128).
//
// Items are numbered by falling length (the number of key tiles), heads fastest; CTA c takes item
// c of every round of gridDim.x, in turn from the front and from the back, so that the CTAs' sums
// differ little.  cu_seqlens is read on the device only: one warp counts the sequences that have a
// query tile of the length in turn and hands the items on.
//
// What packing adds:
//   - tiles start at any row, so the last key tile of a sequence also holds rows of the next one
//     (or padding): their scores are masked, groups of 16 keys behind the sequence are not
//     multiplied, and value rows behind it in its last group are cleared in shared memory;
//   - within the diagonal tile a later token's value row is multiplied by probability 0, which is
//     not 0 for an infinity or NaN: a row whose output is not finite is looked at again at the CTA's
//     end (repair_rows), and its columns that a later value reached are computed from its own keys alone.
#include <cmath>

#include "zo_attn_packed.cuh"

namespace zo {
namespace {

using tc::add2;
using tc::ex2;
using tc::fma2_bc;
using tc::max3f;
using tc::ring_parity;

constexpr int kM = 128;                // query rows of a stream, keys of a tile (2^7: Schedule)
constexpr int kWarps = 12;             // loads, MMAs, items, an idle one; 2 x 4 softmax
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kBox = kM * 128;    // bytes of one 128-row x 64-column bf16 box
constexpr int kItems = 2;              // items on hand

// Sequences of at most kShortSeq tokens go to a kernel of their own where the mean length (the buffer's
// over their number; lengths are known on the device only) lets there be many of them.  16 query and 8
// key/value heads of 128: 64 sequences of 16 tokens take 8.3 us instead of 16.4, 64 of 32 10.1 instead of
// 16.5, 2000 of one 84 instead of 341; where it finds none, 64 of 64 take 22.0 instead of 20.0 and 64 of
// 128 28.5 instead of 25.4.
constexpr int kShortMean = 256;

// From this many sequences on, up to 32 long ones among them are held in the lanes of the warp that
// deals out the items, which is then spared a search for each.
constexpr int kManySeqs = 1024;

enum Mode { kHeads, kPair64, kRows };

template <int HD, bool SPLIT>  // SPLIT: the streams have key/value heads of their own (kPair64)
struct PackedSmem {
  static constexpr uint32_t kQTile = (HD / 64) * kBox;                     // of one stream
  static constexpr uint32_t kStage = (SPLIT ? 2 : HD / 64) * kBox;         // one key or value tile
  static constexpr int kStages = HD == 128 ? 5 : SPLIT ? 6 : 10;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kKV = 2 * kQTile;
  static constexpr uint32_t kBar = kKV + kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 2 + 8 + 2 * kItems + 1;
  static constexpr uint32_t kItem = kBar + 8 * ((kNumBars + 2) / 2 * 2);   // Item [kItems]
  static constexpr uint32_t kBytes = kItem + kItems * 48 + 1024;           // + alignment slack
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// What the two streams of an item do.
struct alignas(16) Item {
  int row0, len;  // the sequence's first row and length (0: no more items)
  int kvh;        // key/value head (of stream 0)
  int most;       // key tiles of the longer stream (0: nothing to do)
  int q[2];       // first query row
  int head[2];    // query head
  int keys[2];    // keys of the stream's tile (0: no such stream)
  int tiles[2];   // key tiles
  // The last tile's value rows behind the sequence share a group of 16 with its own.
  __device__ __forceinline__ bool ragged() const { return most * kM >= len && len % 16 != 0; }
};

// Item of tile `qt` (of 128 rows, or 256: kRows) of a sequence and its heads' number `h`.
__device__ __forceinline__ Item make_item(const PackedArgs &a, int row0, int len, int qt, int h) {
  const bool rows = a.mode == kRows;
  Item it;
  it.row0 = row0;
  it.len = len;
  it.most = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    it.q[i] = rows ? 2 * kM * qt + kM * i : kM * qt;
    it.head[i] = rows ? h : 2 * h + i;
    it.keys[i] = it.q[i] < len ? min(it.q[i] + kM, len) : 0;
    it.tiles[i] = (it.keys[i] + kM - 1) / kM;
    it.most = max(it.most, it.tiles[i]);
  }
  it.kvh = it.head[0] / a.shared;
  return it;
}

// Tiles of 2^shift rows of a sequence that are this kernel's.
__device__ __forceinline__ int tiles_of(const PackedArgs &a, int shift, const Seq &s) {
  return s.len <= a.handled ? 0 : (int)(((uint32_t)s.len + (1u << shift) - 1u) >> shift);
}

// The number of the lane-th of the `count` (at most 32) sequences of more than `level` tiles.
__device__ __forceinline__ int hold(const PackedArgs &a, int shift, int level, int count) {
  const int lane = threadIdx.x & 31;
  int held = 0;
#pragma unroll 1
  for (int i0 = 0, got = 0; got < count && i0 < a.n_seqs; i0 += 32) {
    uint32_t in = __ballot_sync(0xFFFFFFFFu, tiles_of(a, shift, load_seq(a, i0 + lane)) > level);
#pragma unroll 1
    for (; in; in &= in - 1, ++got)
      if (lane == got) held = i0 + __ffs(in) - 1;
  }
  return held;
}

// The items of one CTA in their order (one warp).
//
// The offsets are scanned once for every distinct number of tiles that occurs (as many sequences have
// more than t tiles for all t between two such numbers); where the offsets are many, up to 32 sequences
// that are that long are held in the lanes.  One sequence of 16384 tokens among 131072 empty ones took
// 137 ms with a scan for every number of tiles, 2.7 so.
struct Schedule {
  const PackedArgs &a;
  int shift, group;        // log2 of a tile's rows; items of one tile (heads, or pairs of them)
  int lane;
  Seq first;               // this lane's of the first 32 sequences
  int level, count;        // sequences with more than `level` tiles: `count`,
  int below;               // the same ones as with more than `below`
  int held;                // the lane-th of them, if there are few()
  int64_t base, total;     // items of the longer levels; of all
  int longest;             // tiles of the longest sequence
  int from, before;        // sequences [0, from) have `before` of the level's
  __device__ __forceinline__ Schedule(const PackedArgs &args) : a(args) {
    lane = threadIdx.x & 31;
    shift = a.mode == kRows ? 8 : 7;
    from = before = 0;
    group = a.mode == kRows ? a.H : a.H / 2;
    first = load_seq(a, lane);
    int tiles = tiles_of(first), most = tiles;  // (fewer than 2^25 in all)
    bool bad = first.bad;
    // (unrolled, four steps' loads are on their way together: 2000 sequences of one token 84.5 us, not 93)
#pragma unroll 4
    for (int i0 = 32; i0 < a.n_seqs; i0 += 32) {
      const Seq s = load_seq(a, i0 + lane);
      const int t = tiles_of(s);
      most = max(most, t);
      tiles += t;
      bad |= s.bad;
    }
    if (blockIdx.x == 0 && bad) atomicOr(a.err, ZO_FLAG_OFFSETS);
    total = (int64_t)__reduce_add_sync(0xFFFFFFFFu, tiles) * group;
    longest = __reduce_max_sync(0xFFFFFFFFu, most);
    level = longest - 1;
    base = 0;
    count = below = 0;
    held = 0;
    if (level >= 0) count_level();
  }
  __device__ __forceinline__ int tiles_of(const Seq &s) const { return zo::tiles_of(a, shift, s); }
  __device__ __forceinline__ bool few() const { return a.n_seqs > kManySeqs && count <= 32; }
  // One scan for the new `level` (two where the sequences are held).
  __device__ __forceinline__ void count_level() {
    int n = 0, low = 0;
#pragma unroll 1  // (this code is on the way to the first item: unrolled too, 64 sequences of 128 cost 1.7 us more)
    for (int i0 = 0; i0 < a.n_seqs; i0 += 32) {
      const int t = tiles_of(i0 == 0 ? first : load_seq(a, i0 + lane));
      n += t > level ? 1 : 0;
      low = max(low, t > level ? 0 : t);
    }
    count = __reduce_add_sync(0xFFFFFFFFu, n);
    below = __reduce_max_sync(0xFFFFFFFFu, low);
    if (few()) held = hold(a, shift, level, count);
  }
  // Slot of this CTA's round `n`: to and fro; the last round, which has items for some CTAs only, for
  // those with the least so far.
  __device__ __forceinline__ int64_t slot(int n) const {
    const bool back = (n & 1) || (n > 0 && (int64_t)(n + 1) * gridDim.x >= total);
    return (int64_t)n * gridDim.x + (back ? (int64_t)gridDim.x - 1 - blockIdx.x : (int64_t)blockIdx.x);
  }
  // Item `slot`; slots must not decrease from call to call.  After kPatience steps (of 32 sequences)
  // of scans it returns an item of no tiles and goes on when called again, so that the warps that wait
  // for items never do so for more than five scans: 2^19 steps of 0.26 us each at 2^24 sequences, 0.7 s
  // in all, a third of their limit.
  __device__ __forceinline__ Item at(int64_t slot) {
    constexpr int kPatience = 1 << 15;
    Item it{};
    int steps = 0;
    while (level >= 0 && slot >= base + (int64_t)count * group) {
      base += (int64_t)count * group;
      --level;
      from = before = 0;
      if (level >= 0 && level < below) {
        count_level();
        if ((steps += (a.n_seqs + 31) / 32) > kPatience) {
          it.len = 1;
          it.row0 = -1;
          return it;
        }
      }
    }
    if (level < 0) return it;
    const int index = (int)(slot - base);
    const int nth = index / group;
    if (few()) {
      const Seq s = load_seq(a, __shfl_sync(0xFFFFFFFFu, held, nth));
      return make_item(a, s.row0, s.len, level, index - nth * group);
    }
    for (; from < a.n_seqs; from += 32) {
      const Seq s = from == 0 ? first : load_seq(a, from + lane);
      const uint32_t in = __ballot_sync(0xFFFFFFFFu, tiles_of(s) > level);
      if (nth < before + __popc(in)) {
        const uint32_t lower = in & ((1u << lane) - 1u);
        const int i = __ffs(__ballot_sync(0xFFFFFFFFu, (in >> lane & 1u) && before + __popc(lower) == nth)) - 1;
        it = make_item(a, __shfl_sync(0xFFFFFFFFu, s.row0, i), __shfl_sync(0xFFFFFFFFu, s.len, i), level,
                       index - nth * group);
        break;
      }
      before += __popc(in);
    }
    return it;
  }
};

// The rows of one softmax warp's items (its stream's, 32 from 32 qd on of each tile) again, where their
// outputs are not finite.  For the end of a CTA: inside the pipeline other warps' bounded waits would have to
// last as long (32 rows behind 65536 keys: 97 ms at head dim 64, 150 at 128; eight rows at a time 58 and
// 109, but with registers that cost the pipeline 2 to 6%).
template <int HD>
__device__ __noinline__ void repair_items(const PackedArgs &a, int i, int qd) {
  Schedule sched(a);
  for (int round = 0;;) {
    const Item w = sched.at(sched.slot(round));
    round += w.row0 >= 0;
    if (w.len == 0) break;
    const int first = (i ? w.q[1] : w.q[0]) + 32 * qd, tiles = i ? w.tiles[1] : w.tiles[0];
    const int head = i ? w.head[1] : w.head[0], rows = min(32, w.len - first);
    if (tiles != 0 && rows > 0)
      repair_rows<HD, 4>(a, w.row0, w.len, first, 0xFFFFFFFFu >> (32 - rows), head, head / a.shared, tiles * kM);
  }
}

// One row's step over the first 32 NC keys of a tile: its scores from tensor memory at tS, maximum,
// probabilities back to the first 16 NC columns there, sum.  MASK: keys behind `last` do not count
// (their scores may be anything).
template <int HD, int NC, bool MASK>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, float scale_log2, bool first, int last,
                                             float &m_used, float &l) {
  float s[32 * NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) tc::tmem_ld32_async(tS + 32u * c, s + 32 * c);
  tc::tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < NC; ++c) tc::tmem_ld_seal(s + 32 * c);
  if (MASK) {
    // (of a tile on the diagonal, a warp's rows have one group of 32 keys that is neither in nor out)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (__any_sync(0xFFFFFFFFu, last < 32 * c + 31)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (32 * c + e > last) s[32 * c + e] = -INFINITY;
      }
    }
  }
  // the maximum of the raw scores (the scale is positive), then 2^(s * scale - m) with the
  // scaling folded into the exponent's fused multiply-add
  float mx8[8] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 32 * NC; e += 2) mx8[(e >> 1) & 7] = max3f(mx8[(e >> 1) & 7], s[e], s[e + 1]);
  const float mx = max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * scale_log2;
  const float m_new = fmaxf(m_used, mx);
  // Lazy rescaling: keep the running maximum unless it grows by more than 2^8 (then O and l
  // are rescaled; P_{j-1} V_{j-1} has completed, as S_j was issued after it).
  const bool need = !first && m_new > m_used + 8.f;
  if (__any_sync(0xFFFFFFFFu, need)) {
    const float f = need ? ex2(m_used - m_new) : 1.f;
    l *= f;
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
      float o[16];
      tc::tmem_ld16(tO + 16u * c, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= f;
      tc::tmem_st16(tO + 16u * c, o);
    }
  }
  if (first || need) m_used = m_new;
  const float msc = m_used == -INFINITY ? 0.f : m_used;
  float ls4[4] = {0.f, 0.f, 0.f, 0.f};  // two packed pairs of partial sums
  // P_j overwrites columns of S_j (already read into registers)
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float x0, x1;
      fma2_bc(s[32 * c + e], s[32 * c + e + 1], scale_log2, -msc, x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      if ((e >> 1) & 1) add2(ls4[2], ls4[3], p0, p1);
      else add2(ls4[0], ls4[1], p0, p1);
      pk[e / 2] = pack_bf16x2(p0, p1);
    }
    tc::tmem_st16u_async(tS + 16u * c, pk);
  }
  l += (ls4[0] + ls4[1]) + (ls4[2] + ls4[3]);
  tc::tmem_st_wait();
}

template <int HD, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
attn_packed_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const __grid_constant__ PackedArgs a) {
  using SM = PackedSmem<HD, SPLIT>;
  constexpr int NS = SM::kStages;
  constexpr uint32_t kCols = 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + SM::kBar);  // [NS] ring of tiles K_0 V_0 K_1 V_1 ...
  uint64_t *empty = full + NS;                                   // [NS]
  uint64_t *q_full = empty + NS, *q_empty = q_full + 1;
  uint64_t *s_full = q_empty + 1;   // [2] a stream's scores
  uint64_t *p_full = s_full + 2;    // [2] its probabilities (4 warps)
  uint64_t *pv_done = p_full + 2;   // [2] its O += P V
  uint64_t *o_free = pv_done + 2;   // [2] its output has been read (4 warps)
  uint64_t *item_full = o_free + 2, *item_empty = item_full + kItems;  // [kItems]
  uint64_t *mma_done = item_empty + kItems;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  Item *items = reinterpret_cast<Item *>(sm + SM::kItem);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SM::kNumBars; ++i) tc::mbar_init(&full[i], 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&p_full[i], 4);
      tc::mbar_init(&o_free[i], 4);
    }
    for (int i = 0; i < kItems; ++i) tc::mbar_init(&item_empty[i], 2 + 8);  // loads, MMAs, softmax
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_holder, kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;  // scores of stream i at column 128 i, output at 256 + HD i
  tc::pdl_wait();  // the kernels ahead in the stream have ended

  auto give_up = [&]() {
    atomicOr(a.err, ZO_FLAG_TIMEOUT);
    *abort_flag = 1;
  };
  auto wait = [&](uint64_t *bar, uint32_t parity) { return !*abort_flag && tc::mbar_wait(bar, parity); };
  // Item n of this CTA, for one thread; one arrival on item_empty when it has been copied.
  auto next_item = [&](int n, Item &it) {
    if (!wait(&item_full[n % kItems], ring_parity(n, kItems))) return false;
    it = items[n % kItems];
    tc::mbar_arrive(&item_empty[n % kItems]);
    return true;
  };

  // Registers of a thread from here on: 4 warps x kFew + 8 x kMany = 12 x 168 of the launch.  With 88 and
  // 208 the softmax of head dim 64 reloads a spilled word in its loop: 44.8 us for the case of 43.2.
  constexpr int kFew = 72, kMany = 216;
  if (warp < 4) {
    tc::regs_dec<kFew>();
    if (warp == 0) {
      int issued = 0;  // tiles of the ring
      if (lane == 0) {
        tc::tma_prefetch_desc(&tmq);
        tc::tma_prefetch_desc(&tmk);
        tc::tma_prefetch_desc(&tmv);
        auto load = [&](const CUtensorMap &map, int kvh, int row) -> bool {
          const int st = issued % NS;
          if (!wait(&empty[st], ring_parity(issued, NS) ^ 1u)) return false;
          tc::mbar_arrive_expect_tx(&full[st], SM::kStage);
#pragma unroll
          for (int c = 0; c < (int)(SM::kStage / kBox); ++c)
            tc::tma_load_2d(sm + SM::kKV + st * SM::kStage + c * kBox, &map, &full[st], kvh * HD + 64 * c, row);
          ++issued;
          return true;
        };
        bool ok = true;
        int n_q = 0;
        for (int n = 0; ok; ++n) {
          Item w;
          ok = next_item(n, w);
          if (!ok || w.len == 0) break;
          if (w.most == 0) continue;
          ok = wait(q_empty, ((uint32_t)n_q & 1u) ^ 1u);
          if (!ok) break;
          ++n_q;
          tc::mbar_arrive_expect_tx(q_full, (w.tiles[1] ? 2 : 1) * SM::kQTile);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (w.tiles[i])
              for (int c = 0; c < HD / 64; ++c)
                tc::tma_load_2d(sm + SM::kQ + i * SM::kQTile + c * kBox, &tmq, q_full, w.head[i] * HD + 64 * c,
                                w.row0 + w.q[i]);
          for (int j = 0; ok && j < w.most; ++j)
            ok = load(tmk, w.kvh, w.row0 + j * kM) && load(tmv, w.kvh, w.row0 + j * kM);
        }
        if (!ok) {
          give_up();
          // let this CTA's loads land before it exits (bounded)
          if (n_q > 0) tc::mbar_wait(q_full, (uint32_t)(n_q - 1) & 1u);
          for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) tc::mbar_wait(&full[i % NS], ring_parity(i, NS));
        }
      }
    } else if (warp == 1) {  // MMAs: the warp in step, one lane issues
      const uint32_t sm0 = __shfl_sync(0xFFFFFFFFu, tc::smem_addr(sm), 0);
      const uint32_t tm0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      bool ok = true;
      uint32_t done[2] = {0, 0}, outs[2] = {0, 0};  // tiles and items of each stream so far
      tc::RingPos<NS> key[2], val;                  // of the next key tile for each stream; of the value tile
      val.next();
      uint32_t n_q = 0;
      for (int n = 0; ok; ++n) {
        if (!tc::warp_wait_fast(&item_full[n % kItems], ring_parity(n, kItems), abort_flag)) { ok = false; break; }
        Item w = items[n % kItems];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&item_empty[n % kItems]);
        // alike in all lanes, which the compiler is to know
        w.len = __shfl_sync(0xFFFFFFFFu, w.len, 0);
        w.most = __shfl_sync(0xFFFFFFFFu, w.most, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w.keys[i] = __shfl_sync(0xFFFFFFFFu, w.keys[i], 0);
          w.tiles[i] = __shfl_sync(0xFFFFFFFFu, w.tiles[i], 0);
        }
        if (w.len == 0) break;
        if (w.most == 0) continue;
        // K_j is there (it is for the second stream if the first has used it)
        auto wait_k = [&](int i, int j) -> bool {
          return (i == 1 && j < w.tiles[0]) || tc::warp_wait_fast(&full[key[i].slot], key[i].phase, abort_flag);
        };
        // S_j of stream i; the stream that uses K_j (and Q) last releases it
        auto issue_s = [&](int i, int j) {
          const int st = key[i].slot;
          tc::tc_fence_after();
          key[i].next();
          key[i].next();
          const int keys = min(kM, w.keys[i] - j * kM);
          const uint32_t id = tc::idesc_bf16_f32(kM, (keys + 15) / 16 * 16);
          const uint32_t qa = tc::desc_k128_lo(sm0 + SM::kQ + i * SM::kQTile);
          const uint32_t ka = tc::desc_k128_lo(sm0 + SM::kKV + st * SM::kStage + (SPLIT ? (uint32_t)i * kBox : 0u));
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
              const uint32_t off = ((uint32_t)(k >> 2) * kBox + (uint32_t)(k & 3) * 32u) >> 4;
              tc::mma_bf16_lo(tm0 + (uint32_t)(kM * i), qa + off, ka + off, id, k > 0 ? 1u : 0u);
            }
            tc::mma_commit(&s_full[i]);
            if (i == (w.tiles[1] > j ? 1 : 0)) {
              tc::mma_commit(&empty[st]);
              if (j == w.most - 1) tc::mma_commit(q_empty);
            }
          }
          __syncwarp();
        };
        ok = tc::warp_wait_fast(q_full, n_q++ & 1u, abort_flag) && wait_k(0, 0);
        if (ok) {
          issue_s(0, 0);
          if (w.tiles[1]) issue_s(1, 0);
        }
        for (int j = 0; ok && j < w.most; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || j >= w.tiles[i]) continue;
            // O += P_j V_j once the softmax has written P_j (in place of S_j) and V_j has landed
            const int st = val.slot;
            // (tiles that the other stream has seen land need no second look)
            if (i == 0 || j >= w.tiles[0]) ok = tc::warp_wait_fast(&full[st], val.phase, abort_flag);
            ok = ok && tc::warp_wait_fast(&p_full[i], done[i] & 1u, abort_flag);
            if (ok && j == 0) ok = tc::warp_wait_fast(&o_free[i], (outs[i] & 1u) ^ 1u, abort_flag);
            if (!ok) break;
            tc::tc_fence_after();
            constexpr uint32_t idO = tc::idesc_bf16_f32(kM, HD) | (1u << 16);  // B (V) MN-major
            const uint32_t va =
                tc::desc_mn128_lo(sm0 + SM::kKV + st * SM::kStage + (SPLIT ? (uint32_t)i * kBox : 0u), kBox);
            const uint32_t tO = tm0 + 2u * kM + (uint32_t)(HD * i), tP = tm0 + (uint32_t)(kM * i);
            const int steps = (min(kM, w.keys[i] - j * kM) + 15) / 16;  // keys behind are not multiplied
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < kM / 16; ++k)
                if (k < steps)
                  tc::mma_bf16_tmem_a_lo(tO, tP + 8u * k, va + (uint32_t)k * (2048u >> 4), idO,
                                         (j > 0 || k > 0) ? 1u : 0u);
              tc::mma_commit(&pv_done[i]);
              if (i == (w.tiles[1] > j ? 1 : 0)) tc::mma_commit(&empty[st]);
            }
            __syncwarp();
            // S_{j+1} replaces P_j, which the product must have read
            if (j + 1 < w.tiles[i]) ok = wait_k(i, j + 1);
            ok = ok && tc::warp_wait_fast(&pv_done[i], done[i] & 1u, abort_flag);
            ++done[i];
            if (ok && j + 1 < w.tiles[i]) issue_s(i, j + 1);
          }
          val.next();
          val.next();
        }
        // a stream that took fewer tiles goes on behind the item's last
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          outs[i] += w.tiles[i] != 0;
          for (int j = w.tiles[i]; j < w.most; ++j) {
            key[i].next();
            key[i].next();
          }
        }
      }
      if (!ok && lane == 0) give_up();
      __syncwarp();
      if (tc::elect_one()) tc::mma_commit(mma_done);  // arrives once every MMA issued above has retired
    } else if (warp == 2) {  // items
      Schedule sched(a);
      for (int n = 0, round = 0;; ++n) {
        const Item it = sched.at(sched.slot(round));
        round += it.row0 >= 0;  // (an item of no tiles that only passes time keeps the slot)
        // an item takes its tiles' time: one wait for every 2^18 of them (about 0.4 s)
        int waits = 1 + (sched.longest >> 18);
        bool ok = false;
        while (!ok && waits-- > 0 && !*abort_flag)
          ok = tc::warp_wait_fast(&item_empty[n % kItems], ring_parity(n, kItems) ^ 1u, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          if (lane == 0) give_up();
          break;
        }
        if (lane == 0) {
          items[n % kItems] = it;
          tc::mbar_arrive(&item_full[n % kItems]);  // (release: the item is visible)
        }
        if (it.len == 0) break;
      }
    }
  } else {  // softmax: TMEM lane quadrant qd holds the stream's query rows 32 qd .. +31
    tc::regs_inc<kMany>();
    const int i = (warp - 4) / 4, qd = warp & 3;
    const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
    const uint32_t tS = tmem + (uint32_t)(kM * i) + lane_off, tO = tmem + 2u * kM + (uint32_t)(HD * i) + lane_off;
    uint32_t done = 0;  // tiles of the stream so far
    int base = 0;       // key tiles of the items before
    bool ok = true, suspect = false;  // this lane's outputs so far hold an infinity or NaN
    for (int n = 0; ok; ++n) {
      if (!tc::warp_wait_fast(&item_full[n % kItems], ring_parity(n, kItems), abort_flag)) {
        ok = false;
        break;
      }
      const Item w = items[n % kItems];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&item_empty[n % kItems]);
      if (w.len == 0) break;
      const int q0 = i ? w.q[1] : w.q[0], tiles = i ? w.tiles[1] : w.tiles[0], head = i ? w.head[1] : w.head[0];
      const int key_end = i ? w.keys[1] : w.keys[0];
      const int at = 2 * (base + w.most - 1) + 1;  // the last value tile's place in the ring
      base += w.most;
      if (tiles == 0) continue;
      const int r = q0 + 32 * qd + lane;                     // query position in the sequence
      const bool any = q0 + 32 * qd < w.len;                 // this warp has a row
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < tiles; ++j, ++done) {
        if (!tc::warp_wait_fast(&s_full[i], done & 1u, abort_flag)) { ok = false; break; }
        tc::tc_fence_after();
        const int key0 = j * kM;
        const int last = min(r, w.len - 1) - key0;                // the row's last key in the tile
        // the causal / sequence-end mask touches only the tiles that reach the diagonal or the end
        if (!any) {
          // rows behind the sequence: whatever P holds, their outputs are not read
        } else if (key0 + kM - 1 <= min(q0 + 32 * qd, w.len - 1))
          softmax_tile<HD, 4, false>(tS, tO, a.scale_log2, j == 0, last, m_used, l);
        else if (key_end - key0 > 64)  // the keys that P V reads (uniform over the stream)
          softmax_tile<HD, 4, true>(tS, tO, a.scale_log2, j == 0, last, m_used, l);
        else if (key_end - key0 > 32)
          softmax_tile<HD, 2, true>(tS, tO, a.scale_log2, j == 0, last, m_used, l);
        else
          softmax_tile<HD, 1, true>(tS, tO, a.scale_log2, j == 0, last, m_used, l);
        if (j == w.most - 1 && w.ragged() && i == (w.tiles[0] == w.most ? 0 : 1)) {
          // The value rows behind the sequence (another one's, or padding) in its last group of 16
          // keys must not reach P V even with probability 0: 0 * NaN is NaN.  The stream whose
          // product comes first clears them.
          if (!tc::warp_wait_fast(&full[at % NS], ring_parity(at, NS), abort_flag)) { ok = false; break; }
          const int first = w.len - key0, n = (16 - first % 16) * 8;  // n pieces of 16 bytes a box
          uint8_t *tile = sm + SM::kKV + (at % NS) * SM::kStage + first * 128;
          if (32 * qd + lane < n) {
#pragma unroll
            for (int c = 0; c < (int)(SM::kStage / kBox); ++c)
              *reinterpret_cast<uint4 *>(tile + c * kBox + 16 * (32 * qd + lane)) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[i]);
      }
      if (!ok) break;
      if (!tc::warp_wait_fast(&pv_done[i], (done - 1u) & 1u, abort_flag)) { ok = false; break; }
      tc::tc_fence_after();
      const float inv = 1.f / l;  // (l = 0: every score of the row is -inf, and 0 infinity = NaN)
      const int r_quad = r - lane % 4;
      uint16_t *orow = a.out + (int64_t)(w.row0 + r_quad) * a.ldo + (int64_t)head * HD + 8 * (lane % 4);
      uint32_t worst = 0;  // two bf16, NaN if any output of the row is not finite
#pragma unroll 1
      for (int c = 0; any && c < HD; c += 32) {
        float o[32];
        tc::tmem_ld32(tO + (uint32_t)c, o);
        // the quad's 4 rows x 4 pieces of 16 bytes transposed: a store takes 64 bytes of 8 rows, not 16
        // bytes of 32 rows
        uint32_t v[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[e][k] = pack_bf16x2(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
            worst = tc::zero_or_nan2(v[e][k], worst);
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) quad_transpose(v[e]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r_quad + k < w.len)
            *reinterpret_cast<uint4 *>(orow + k * a.ldo + c) = make_uint4(v[0][k], v[1][k], v[2][k], v[3][k]);
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&o_free[i]);
      suspect |= r < w.len && worst != 0;
    }
    if (!ok && lane == 0) give_up();
    if (__any_sync(0xFFFFFFFFu, suspect) && ok) repair_items<HD>(a, i, qd);
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

template <int HD, bool SPLIT>
zo_status launch(zo_ctx *ctx, const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                 const PackedArgs &a) {
  using SM = PackedSmem<HD, SPLIT>;
  const auto kernel = attn_packed_kernel<HD, SPLIT>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void *>(kernel), (int)SM::kBytes);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "attn_packed_kernel attribute: %s", cudaGetErrorString(e));
  // at most this many items
  const int64_t per = a.mode == kRows ? 2 * kM : kM, group = a.mode == kRows ? a.H : a.H / 2;
  const int64_t items = (((int64_t)a.total + per - 1) / per + a.n_seqs) * group;
  e = launch_early(kernel, dim3((unsigned)(items < kSmCount ? items : kSmCount)), kThreads, (int)SM::kBytes, ctx->stream,
                   tmq, tmk, tmv, a);
  if (e != cudaSuccess) return fail(ctx, ZO_ERR_CUDA, "attn_packed_kernel: %s", cudaGetErrorString(e));
  ctx->launches += 1;
  return ZO_OK;
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
  if (n_seqs < 1 || n_seqs > 1 << 24 || total_tokens < 1 || total_tokens > INT32_MAX - 256)
    return fail(ctx, ZO_ERR_INVALID, "attention_packed: need n_seqs in [1, 2^24] and total_tokens in [1, 2^31 - 257]");
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
  const int shared = n_heads / n_kv_heads;
  const Mode mode = shared % 2 == 0 ? kHeads : head_dim == 64 && shared == 1 && n_heads % 2 == 0 ? kPair64 : kRows;
  PackedArgs a{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
               static_cast<const uint16_t *>(v), static_cast<uint16_t *>(out), cu_seqlens, n_seqs,
               (int)total_tokens, n_heads, n_kv_heads, ldq, ldk, ldv, ldo,
               scale * 1.4426950408889634f, (int)mode, shared, 0, &ctx->dstate->flags};
  if (total_tokens / n_seqs <= kShortMean) {
    const zo_status st = launch_attn_short(ctx, a, head_dim);
    if (st != ZO_OK || total_tokens <= kShortSeq) return st;
    a.handled = kShortSeq;
  }
  CUtensorMap tmq, tmk, tmv;
  if (!tile_map_bf16(&tmq, q, total_tokens, wq, ldq, kM) || !tile_map_bf16(&tmk, k, total_tokens, wk, ldk, kM) ||
      !tile_map_bf16(&tmv, v, total_tokens, wk, ldv, kM))
    return fail(ctx, ZO_ERR_CUDA, "attention_packed: cuTensorMapEncodeTiled failed");
  if (head_dim == 128) return launch<128, false>(ctx, tmq, tmk, tmv, a);
  return mode == kPair64 ? launch<64, true>(ctx, tmq, tmk, tmv, a) : launch<64, false>(ctx, tmq, tmk, tmv, a);
}
