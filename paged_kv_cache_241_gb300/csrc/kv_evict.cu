// kv_evict.cu -- shorten sequences of the paged cache to their heaviest keys.
//
// For each (sequence, kv head) whose context is longer than `budget`, the last
// `recent` tokens stay, and of the others the `budget - recent` with the
// largest accumulated attention weight.  Decode reads a sequence's keys in any
// order (their positions are already in the keys), so a kept token that sits
// inside the first budget - recent places stays where it is and only the kept
// ones behind them move, each into a place that an evicted token leaves: the
// rows moved are those evicted there, not the whole budget.  The recent tokens
// keep their order at the end, so that "the last `recent`" means the same at
// the next eviction.
//
// Two launches: one CTA per (sequence, kv head) selects and writes `kept` (the
// old position of what is to sit at each place), then CTAs per (sequence, kv
// head, K or V, run of places) move the rows that `kept` says.
//
// The moves are bound by HBM, in rows of 128 or 256 bytes, the selection by its
// barriers and by shared memory's atomics (a pass over a unit's keys is short).
// Measured: 64 sequences of 1025 to 1280 tokens down to 1024 (8 kv heads, D = 128:
// 131 MB) 39 us, the selection 12 and the moves 26 (5 TB/s); 16 prompts of 2000 to
// 16384 tokens down to 2048 (149 MB) 48 us, 20 and 28 (5.2 TB/s).
#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kBins = 256;              // selection by digits of 8 bits
constexpr int kCopies = 8;              // of a bin, side by side: lanes with equal digits collide less
constexpr int kRankWords = 4;           // bitmap words per entry of the rank table
constexpr int kMaxContext = 1 << 20;    // the bitmap of kept positions is in shared memory
constexpr int kKeyCache = 40 << 10;     // candidates whose keys stay in shared memory, at most
constexpr int kKeepEquals = 1 << 18;    // tables up to here also keep a bitmap of the equal keys (the
                                        // selections of 256 threads always: kLongContext)
constexpr int kSelectBytes = 216 << 10; // shared memory of the selection, beside its counters
constexpr int kLongContext = 4096;      // from here on a selecting CTA has 1024 threads, not 256
static_assert(kLongContext <= kKeepEquals, "");
constexpr int kMoveThreads = 256;
constexpr int kMoveList = 1024;         // moves that a CTA can list
constexpr int kMoveCtas = 2048;         // of the second launch, about
constexpr int kMinPlaces = 128;         // places per CTA of the second launch at least
constexpr int kMoveDepth = 8;           // 16-byte vectors that a thread has in flight

struct EvictParams {
  uint16_t *k_cache;
  uint16_t *v_cache;
  float *key_weights;
  const int32_t *block_tables;
  const int32_t *context_lens;
  int32_t *kept;
  int32_t *new_lens;
  int32_t *status;
  int64_t num_blocks;
  int num_seqs;
  int num_kv_heads;
  int row_vecs;  // 16-byte vectors per row of one kv head
  int block_shift;
  int max_blocks_per_seq;
  int budget;
  int recent;
  int places;  // per CTA of the second launch
  int aligned;  // key_weights to 16 bytes
};

// Weights as integers of the same order: NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Slot of position i of the sequence whose table row is bt.
__device__ __forceinline__ int64_t slot_at(const int32_t *bt, int i, int shift) {
  return ((int64_t)bt[i >> shift] << shift) + (i & ((1 << shift) - 1));
}

// Index of a slot's sum for kv head j: key_weights is [num_blocks, Hkv, block_size].
__device__ __forceinline__ int64_t weight_at(const int32_t *bt, int i, int shift, int Hkv, int j) {
  return (((int64_t)bt[i >> shift] * Hkv + j) << shift) + (i & ((1 << shift) - 1));
}

// The digit bin of the `need`-th largest among the counted keys; `need` becomes
// the rank inside that bin, `all` says whether it is the bin's last.  All threads
// call it and get the same answer.
__device__ int pick_bin(const int *hist, int *warp_sums, int *found, int &need,
                        bool &all) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int count = 0, incl = 0;
  if (warp < kBins / 32) {  // thread t has the t-th bin from the top
    const int4 *bin = reinterpret_cast<const int4 *>(hist + (kBins - 1 - tid) * kCopies);
    const int4 a = bin[0], b = bin[1];
    count = (a.x + a.y) + (a.z + a.w) + (b.x + b.y) + (b.z + b.w);
    incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
  }
  __syncthreads();
  if (warp < kBins / 32) {
    const int before =
        incl - count + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
    if (before < need && need <= before + count) {
      found[0] = kBins - 1 - tid;
      found[1] = need - before;
      found[2] = count;
    }
  }
  __syncthreads();
  need = found[1];
  all = need == found[2];
  return found[0];
}

// Position of the n-th (from 0) set bit of a word that has more than n.
__device__ __forceinline__ int nth_bit(uint32_t word, int n) {
  int base = 0;
#pragma unroll
  for (int width = 16; width > 0; width >>= 1) {
    const int c = __popc(word & ((1u << width) - 1));
    if (n >= c) {
      n -= c;
      word >>= width;
      base += width;
    } else {
      word &= (1u << width) - 1;
    }
  }
  return base;
}

// Shared memory of the selection: keys, bitmaps, rank table.  The table's length
// sizes the bitmaps; past kKeepEquals positions (32 KB a bitmap) the second one
// is counted again instead, and the keys take what is left (14 K of them at 2^20).
struct SelectSmem {
  int keys, words, equals, ranks;  // entries
  __host__ __device__ SelectSmem(int room) {
    words = (room + 31) / 32 + kRankWords;
    equals = room <= kKeepEquals ? words : 0;
    ranks = words / kRankWords + 2;
    const int left = (kSelectBytes / 4 - words - equals - ranks) & ~3;
    keys = left < kKeyCache ? left : kKeyCache;
    if (room < keys) keys = room;
  }
  __host__ __device__ int bytes() const { return (keys + words + equals + ranks) * 4; }
};

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, kSelThreads == 256 ? 6 : 1)
    evict_select_kernel(const EvictParams p) {
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ __align__(16) int hist[kBins * kCopies];
  __shared__ int warp_sums[2][32];
  __shared__ int found[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / p.num_kv_heads;
  const int j = blockIdx.x - s * p.num_kv_heads;
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  int32_t *kept = p.kept + (int64_t)blockIdx.x * p.budget;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the kernel before the call)
  const int L = p.context_lens[s];
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  const int shift = p.block_shift;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const SelectSmem lay((int)room);
  uint32_t *keys = dyn;
  uint32_t *bits = dyn + lay.keys;  // bit i: position i is kept
  uint32_t *equals = bits + lay.words;                      // its key equals the last kept one
  int *ranks = reinterpret_cast<int *>(equals + lay.equals);  // kept positions before each 128

  // Candidates [0, N), of which H are kept; their keys are read as the blocks are checked.
  const int N = L - p.recent;
  const int H = p.budget - p.recent;
  const bool cuts = L > p.budget && L <= room;  // (H < N then)
  bool bad = L < 0 || L > room;
  if (bad && j == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  const int cached = cuts && H > 0 ? min(N, lay.keys) : 0;
  if (!bad) {
    int wrong = 0;
    const int nb = (int)(((int64_t)L + (1 << shift) - 1) >> shift);
    for (int b = tid; b < nb; b += kSelThreads) wrong |= bt[b] < 0 || bt[b] >= p.num_blocks;
    // Four neighbours at a time: they share a block, which has room behind N too.
#pragma unroll 4
    for (int i = tid * 4; i < cached; i += kSelThreads * 4) {
      const int blk = bt[i >> shift];
      if (blk < 0 || blk >= p.num_blocks) continue;
      const float *from = p.key_weights + weight_at(bt, i, shift, p.num_kv_heads, j);
      float4 w;
      if (p.aligned) w = *reinterpret_cast<const float4 *>(from);
      else w = make_float4(from[0], from[1], from[2], from[3]);
      *reinterpret_cast<uint4 *>(keys + i) =
          make_uint4(order_key(w.x), order_key(w.y), order_key(w.z), order_key(w.w));
    }
    bad = __syncthreads_or(wrong) != 0;
    if (bad && j == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
  }
  if (j == 0 && tid == 0) p.new_lens[s] = cuts && !bad ? p.budget : L;
  if (bad || !cuts) {  // nothing moves
    for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = (!bad && i < L) ? i : -1;
    return;
  }
  for (int i = tid; i < p.recent; i += kSelThreads) kept[H + i] = N + i;
  if (H == 0) return;
  auto key_at = [&](int i) {
    return i < cached ? keys[i]
                      : order_key(p.key_weights[weight_at(bt, i, shift, p.num_kv_heads, j)]);
  };

  // The H-th largest key T, digit by digit; `need` of the keys equal to T are
  // kept.  (A thread reads back the keys that it stored.)
  uint32_t T = 0;
  int need = H;
#pragma unroll 1
  for (int lo = 24; lo >= 0; lo -= 8) {
    for (int b = tid; b < kBins * kCopies / 4; b += kSelThreads)
      reinterpret_cast<int4 *>(hist)[b] = make_int4(0, 0, 0, 0);
    __syncthreads();
    int *mine = hist + (lane & (kCopies - 1));
    auto count = [&](uint32_t u) {
      if (lo == 24 || (u >> (lo + 8)) == (T >> (lo + 8)))  // (the digits known so far)
        atomicAdd(mine + ((u >> lo) & (kBins - 1)) * kCopies, 1);
    };
#pragma unroll 2
    for (int i = tid * 4; i < cached; i += kSelThreads * 4) {
      const uint4 u = *reinterpret_cast<const uint4 *>(keys + i);
      count(u.x);
      if (i + 1 < N) count(u.y);
      if (i + 2 < N) count(u.z);
      if (i + 3 < N) count(u.w);
    }
    for (int i = cached + tid; i < N; i += kSelThreads) count(key_at(i));
    __syncthreads();
    bool all;
    T |= (uint32_t)pick_bin(hist, warp_sums[0], found, need, all) << lo;
    // All keys with these digits are kept: the digits behind do not matter (of
    // keys that differ the third pass is mostly the last, of few the second).
    // (Not all keys are kept, so a smaller one exists and T is not 0.)
    if (all) {
      T -= 1;
      need = 0;
      break;
    }
  }

  // Kept: keys above T, and the first `need` of those equal to it.  Each warp
  // takes a run of whole entries of the rank table, in order.
  const int words = (N + 31) >> 5;
  const int entries = (words + kRankWords - 1) / kRankWords;
  const int per_warp = ((entries + kSelWarps - 1) / kSelWarps) * kRankWords;
  const int w0 = min(warp * per_warp, entries * kRankWords);
  const int w1 = min(w0 + per_warp, entries * kRankWords);
  int above = 0, equal = 0;
  for (int w = w0; w < w1; ++w) {
    const int i = w * 32 + lane;
    const uint32_t u = i < N ? key_at(i) : 0u;
    const uint32_t more = __ballot_sync(0xffffffffu, i < N && u > T);
    const uint32_t same = __ballot_sync(0xffffffffu, i < N && u == T);
    if (lane == 0) {
      bits[w] = more;
      if (kSelThreads == 256 || lay.equals > 0) equals[w] = same;
    }
    above += __popc(more);
    equal += __popc(same);
  }
  if (lane == 0) {
    warp_sums[0][warp] = above;
    warp_sums[1][warp] = equal;
  }
  __syncthreads();
  // Above T, and equal to it, before this warp's positions.
  int run = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[0][lane] : 0);
  int rank = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[1][lane] : 0);
  run += min(rank, need);
  for (int base = w0; base < w1; base += 32) {  // a word per lane
    const int w = base + lane;
    uint32_t same = 0;
    if (kSelThreads == 256 || lay.equals > 0) {
      same = w < w1 ? equals[w] : 0u;
    } else {
      for (int x = base; x < min(base + 32, w1); ++x) {
        const int i = x * 32 + lane;
        const uint32_t all = __ballot_sync(0xffffffffu, i < N && key_at(i) == T);
        if (w == x) same = all;
      }
    }
    uint32_t word = w < w1 ? bits[w] : 0u;
    int before = __popc(same);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    const int all_same = __shfl_sync(0xffffffffu, before, 31);
    const int left = need - (rank + before - __popc(same));  // of this word's, so many are kept
    if (left >= __popc(same)) word |= same;
    else if (left > 0) word |= same & ((1u << nth_bit(same, left)) - 1);
    int kept_to = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, kept_to, o);
      if (lane >= o) kept_to += y;
    }
    if (w < w1) {
      bits[w] = word;
      if (w % kRankWords == 0) ranks[w / kRankWords] = run + kept_to - __popc(word);
    }
    rank += all_same;
    run += __shfl_sync(0xffffffffu, kept_to, 31);
  }
  __syncthreads();
  auto kept_before = [&](int i) {  // kept positions in [0, i)
    const int w = i >> 5;
    int c = ranks[w / kRankWords];
    for (int x = w & ~(kRankWords - 1); x < w; ++x) c += __popc(bits[x]);
    return c + __popc(bits[w] & ((1u << (i & 31)) - 1));
  };
  for (int i = tid; i < H; i += kSelThreads)
    if ((bits[i >> 5] >> (i & 31)) & 1) kept[i] = i;
  // The r-th free place below H takes the r-th kept position behind: each is
  // looked up by its number, among the free ones or the kept ones before it.
  const int inside = kept_before(H);
  for (int r = tid; r < H - inside; r += kSelThreads) {
    auto find = [&](int want, int free) {  // (free: 1 to count the positions that are not kept)
      auto before = [&](int e) { return free ? e * kRankWords * 32 - ranks[e] : ranks[e]; };
      int lo = 0, hi = entries - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before(mid) <= want) lo = mid;
        else hi = mid - 1;
      }
      int left = want - before(lo);
      int w = lo * kRankWords;
      const uint32_t flip = free ? 0xFFFFFFFFu : 0u;
      for (int c = __popc(bits[w] ^ flip); left >= c; c = __popc(bits[w] ^ flip)) {
        left -= c;
        ++w;
      }
      return w * 32 + nth_bit(bits[w] ^ flip, left);
    };
    kept[find(r, 1)] = find(inside + r, 0);
  }
}

// Rows move from kept[i] to i, for the places of this CTA.  Places in [0, H) take
// rows from positions at or behind H, and the recent rows move down to
// [H, budget).  A CTA lists its moves and does them in batches, each of which
// reads all of its rows before it writes any.  Rows that some move overwrites
// are read by the CTA that does, and in time: CTA 0 of a unit moves the recent
// rows in ascending order (a row's new place is never behind its old one) and,
// listed before them, every row that they overwrite.  (In series, 128 rows a batch: one
// sequence of 3000 tokens down to 2048 takes 15 us with 32 recent ones, 20 with 256,
// 34 with 1024.)  Rows at or behind
// `budget` that move below H are written by none: the CTAs of a unit share them
// by place.
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictParams p) {
  __shared__ int2 moves[kMoveList];  // (from, to)
  __shared__ int count;
  const int unit = blockIdx.x >> 1;
  const int s = unit / p.num_kv_heads;
  const int j = unit - s * p.num_kv_heads;
  const int L = p.context_lens[s];
  // (The launch must not end before the first one has: what follows on the stream
  // reads that one's outputs.  One CTA waits for it whatever there is to move.)
  if (L <= p.budget && (blockIdx.x | blockIdx.y) != 0) return;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) count = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (L <= p.budget) return;
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  const int32_t *kept = p.kept + (int64_t)unit * p.budget;
  if (kept[p.budget - 1] < 0) return;  // (a sequence that was refused)
  const int H = p.budget - p.recent;
  const bool sums = (blockIdx.x & 1) == 0;  // the K units move the weights too
  uint4 *cache = reinterpret_cast<uint4 *>(sums ? p.k_cache : p.v_cache);
  const int shift = p.block_shift, Hkv = p.num_kv_heads;
  const int V = p.row_vecs, vshift = V == 16 ? 4 : 3;
  auto at = [&](int i, int v) { return ((slot_at(bt, i, shift) * Hkv + j) << vshift) + v; };
  __syncthreads();

  auto do_moves = [&](int n) {  // the first n listed
    const int total = n << vshift;
    for (int base = 0; base < total; base += kMoveThreads * kMoveDepth) {
      uint4 a[kMoveDepth];
      float w[kMoveDepth];
#pragma unroll
      for (int u = 0; u < kMoveDepth; ++u) {
        const int x = base + u * kMoveThreads + tid;
        if (x >= total) break;
        const int from = moves[x >> vshift].x, v = x & (V - 1);
        a[u] = cache[at(from, v)];
        if (sums && v == 0) w[u] = p.key_weights[weight_at(bt, from, shift, Hkv, j)];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveDepth; ++u) {
        const int x = base + u * kMoveThreads + tid;
        if (x >= total) break;
        const int to = moves[x >> vshift].y, v = x & (V - 1);
        cache[at(to, v)] = a[u];
        if (sums && v == 0) p.key_weights[weight_at(bt, to, shift, Hkv, j)] = w[u];
      }
    }
  };
  // Lists the moves to places [begin, end): CTA 0 those of rows that recent ones
  // overwrite, and in a CTA's own run of places the others.
  auto list_places = [&](int begin, int end, bool own, bool overwritten) {
    int srcs[kMoveList / kMoveThreads];  // (all asked for at once; no run is longer than the list)
#pragma unroll
    for (int u = 0; u < kMoveList / kMoveThreads; ++u) {
      const int i = begin + u * kMoveThreads + tid;
      srcs[u] = i < end ? kept[i] : i;
    }
#pragma unroll
    for (int u = 0; u < kMoveList / kMoveThreads; ++u) {
      if (begin + u * kMoveThreads >= end) break;
      const int i = begin + u * kMoveThreads + tid, src = srcs[u];
      const bool take = src != i && (src < p.budget ? overwritten : own);
      const uint32_t all = __ballot_sync(0xffffffffu, take);
      int first = 0;
      if (lane == 0 && all) first = atomicAdd(&count, __popc(all));
      first = __shfl_sync(0xffffffffu, first, 0) + __popc(all & ((1u << lane) - 1));
      if (take) moves[first] = make_int2(src, i);
    }
    __syncthreads();
  };
  const bool lead = blockIdx.y == 0;
  const int first = min(H, (int)blockIdx.y * p.places), end = min(H, first + p.places);
  list_places(first, end, true, lead);
  // (without recent rows nothing is overwritten: no mover is below the budget)
  for (int begin = end; lead && p.recent > 0 && begin < H; begin += kMoveList / 2) {
    const int listed = count;
    __syncthreads();  // (all have read it: the next places add to it)
    if (listed > kMoveList / 2) {
      do_moves(listed);
      __syncthreads();
      if (tid == 0) count = 0;
      __syncthreads();
    }
    list_places(begin, min(H, begin + kMoveList / 2), false, true);
  }
  int n = count;
  int done = 0;  // recent rows listed so far
  while (lead && done < p.recent) {
    const int more = min(p.recent - done, kMoveList - n);
    for (int x = tid; x < more; x += kMoveThreads)
      moves[n + x] = make_int2(L - p.recent + done + x, H + done + x);
    n += more;
    done += more;
    __syncthreads();
    if (done == p.recent) break;
    do_moves(n);
    __syncthreads();
    n = 0;
  }
  do_moves(n);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_kv_evict(uint16_t *k_cache, uint16_t *v_cache, float *key_weights,
                                   const int32_t *block_tables, const int32_t *context_lens,
                                   int num_seqs, int num_kv_heads, int head_dim, int block_size,
                                   int max_blocks_per_seq, int64_t num_blocks, int budget,
                                   int recent, int32_t *kept, int32_t *new_lens,
                                   int32_t *dev_status, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || budget <= 0 || recent < 0 || recent > budget)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (block_size != 64 && block_size != 128 && block_size != 256 && block_size != 512)
    return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > kMaxContext || budget > kMaxContext)
    return PKV_ERR_UNSUPPORTED;
  const int64_t units = (int64_t)num_seqs * num_kv_heads;
  if (units > 0x3FFFFFFFLL) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !key_weights || !block_tables || !context_lens || !kept || !new_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(key_weights) & 3u) != 0)
    return PKV_ERR_INVALID_ARG;
  // Buffers that share memory: K and V rows are moved by CTAs of their own, and every
  // kv head reads the old lengths.
  // (in double: any number of blocks, and distances below 2^53 exactly)
  auto overlap = [](const void *a, const void *b, double bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return (double)(x < y ? y - x : x - y) < bytes;
  };
  if (overlap(k_cache, v_cache, (double)num_blocks * block_size * num_kv_heads * head_dim * 2) ||
      overlap(context_lens, new_lens, num_seqs * 4.0))
    return PKV_ERR_INVALID_ARG;

  EvictParams prm;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.key_weights = key_weights;
  prm.block_tables = block_tables;
  prm.context_lens = context_lens;
  prm.kept = kept;
  prm.new_lens = new_lens;
  prm.status = dev_status;
  prm.num_blocks = num_blocks;
  prm.num_seqs = num_seqs;
  prm.num_kv_heads = num_kv_heads;
  prm.row_vecs = head_dim / 8;
  prm.block_shift = 31 - __builtin_clz((unsigned)block_size);
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.budget = budget;
  prm.recent = recent;
  prm.places = 0;
  prm.aligned = aligned16(key_weights) ? 1 : 0;
  const int room = max_blocks_per_seq * block_size;
  const int smem = SelectSmem(room).bytes();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Short contexts: small CTAs, several per SM, hide one another's barriers; long
  // ones: more threads for a sequence's keys.  Measured, both sides: 512 units of
  // 1025 to 1280 tokens 42.4 us with 256 threads and 58.2 with 1024; 128 units of
  // 2000 to 16384 tokens 66.0 and 51.2.  The host knows the table's width, not the
  // contexts, so a wide table of short ones takes the wide form: those 512 units 30 us
  // in a table of 1280 tokens, 31 in one of 4096, 44 in one of 8192, 46 in one of 2^20.
  const bool is_long = room > kLongContext;
  if (!kernel_smem_setup(is_long ? (const void *)evict_select_kernel<1024>
                                 : (const void *)evict_select_kernel<256>,
                         is_long ? 1024 : 256, smem, nullptr))
    return PKV_ERR_CUDA;
  // Both programmatic dependents, the first one of the kernel before the call (16
  // prompts 50.5 -> 48.0 us from call to call, the copy of their sums included).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3(is_long ? 1024 : 256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t err =
      cudaLaunchKernelEx(&cfg, is_long ? evict_select_kernel<1024> : evict_select_kernel<256>, prm);
  // Enough CTAs to fill the GPU: a unit's places in several parts when there are
  // few units.
  const int64_t heavy = budget - recent;
  const int64_t wanted = (kMoveCtas + 2 * units - 1) / (2 * units);
  int64_t places = (heavy + wanted - 1) / wanted;
  if (places < kMinPlaces) places = kMinPlaces;
  if (places > kMoveList) places = kMoveList;
  prm.places = (int)places;
  cfg.gridDim = dim3((unsigned)(2 * units),
                     (unsigned)(heavy > 0 ? (heavy + places - 1) / places : 1));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  if (err == cudaSuccess) err = cudaLaunchKernelEx(&cfg, evict_move_kernel, prm);
  return launch_status();  // (either launch's error, which it clears)
}
