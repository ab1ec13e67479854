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
// old position of what is to sit at each place), then one per (sequence, kv
// head, K or V) moves the rows that `kept` says.
#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;             // selection by digits of 11, 11 and 10 bits
constexpr int kSuper = 1024;            // positions per entry of the rank table
constexpr int kMaxContext = 1 << 20;    // the bitmap of kept positions is in shared memory
constexpr int kMoveThreads = 256;

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

// The digit bin of the `need`-th largest among the counted keys; *need becomes
// the rank inside that bin.  All threads call it and get the same answer.
__device__ int pick_bin(const int *hist, int *warp_sums, int *found, int &need) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int per = kBins / kSelThreads;
  // Thread t owns bins in descending order: bins kBins - 1 - (t * per + x).
  int local = 0;
#pragma unroll
  for (int x = 0; x < per; ++x) local += hist[kBins - 1 - (tid * per + x)];
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = incl - local;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
#pragma unroll
  for (int x = 0; x < per; ++x) {
    const int c = hist[kBins - 1 - (tid * per + x)];
    if (before < need && need <= before + c) {
      found[0] = kBins - 1 - (tid * per + x);
      found[1] = need - before;
    }
    before += c;
  }
  __syncthreads();
  need = found[1];
  return found[0];
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t bits[];  // bit i: position i is kept; then the rank table
  __shared__ int hist[kBins];
  __shared__ int warp_sums[kSelWarps];
  __shared__ int found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / p.num_kv_heads;
  const int j = blockIdx.x - s * p.num_kv_heads;
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  int32_t *kept = p.kept + (int64_t)blockIdx.x * p.budget;
  const int L = p.context_lens[s];
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  const int shift = p.block_shift;

  bool bad = false;
  if (L < 0 || L > room) {
    bad = true;
    if (j == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  } else {
    const int nb = (int)(((int64_t)L + (1 << shift) - 1) >> shift);
    int wrong = 0;
    for (int b = tid; b < nb; b += kSelThreads) wrong |= bt[b] < 0 || bt[b] >= p.num_blocks;
    bad = __syncthreads_or(wrong) != 0;
    if (bad && j == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
  }
  if (j == 0 && tid == 0) p.new_lens[s] = (bad || L <= p.budget) ? L : p.budget;
  if (bad || L <= p.budget) {  // nothing moves
    for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = (!bad && i < L) ? i : -1;
    return;
  }

  const int N = L - p.recent;            // candidates: positions [0, N)
  const int H = p.budget - p.recent;     // of which H are kept (H < N)
  for (int i = tid; i < p.recent; i += kSelThreads) kept[H + i] = N + i;
  if (H == 0) return;

  auto key_at = [&](int i) { return order_key(p.key_weights[weight_at(bt, i, shift, p.num_kv_heads, j)]); };

  // The H-th largest key T, digit by digit; `need` of the keys equal to T are kept.
  uint32_t T = 0;
  int need = H;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int lo = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
    for (int i = tid; i < N; i += kSelThreads) {
      const uint32_t u = key_at(i);
      const bool in = pass == 0 || (u >> (lo + (pass == 1 ? 11 : 10))) == (T >> (lo + (pass == 1 ? 11 : 10)));
      if (in) atomicAdd(&hist[(u >> lo) & mask], 1);
    }
    __syncthreads();
    T |= (uint32_t)pick_bin(hist, warp_sums, found, need) << lo;
  }

  // Kept: keys above T, and the first `need` of those equal to it.  Each warp
  // takes a run of whole words of the bitmap, in order.
  const int words = (N + 31) >> 5;
  const int per_warp = (words + kSelWarps - 1) / kSelWarps;
  const int w0 = min(warp * per_warp, words), w1 = min(w0 + per_warp, words);
  int equal = 0;
  for (int w = w0; w < w1; ++w) {
    const int i = w * 32 + lane;
    const uint32_t u = i < N ? key_at(i) : 0u;
    equal += __popc(__ballot_sync(0xffffffffu, i < N && u == T));
  }
  if (lane == 0) warp_sums[warp] = equal;
  __syncthreads();
  int rank = 0;
  for (int w = 0; w < warp; ++w) rank += warp_sums[w];
  __syncthreads();
  for (int w = w0; w < w1; ++w) {
    const int i = w * 32 + lane;
    const uint32_t u = i < N ? key_at(i) : 0u;
    const bool eq = i < N && u == T;
    const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
    const bool keep = (i < N && u > T) || (eq && rank + __popc(eqs & ((1u << lane) - 1)) < need);
    const uint32_t word = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) bits[w] = word;
    rank += __popc(eqs);
  }
  __syncthreads();

  // Kept positions before each group of kSuper: the rank table.
  int *table = reinterpret_cast<int *>(bits + words);
  const int supers = (N + kSuper - 1) / kSuper;
  for (int x = warp; x < supers; x += kSelWarps) {
    const int w = x * (kSuper / 32) + lane;
    int c = w < words ? __popc(bits[w]) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (lane == 0) table[x + 1] = c;
  }
  __syncthreads();
  if (tid == 0) {
    table[0] = 0;
    for (int x = 0; x < supers; ++x) table[x + 1] += table[x];
  }
  __syncthreads();
  auto kept_before = [&](int i) {  // kept positions in [0, i)
    int c = table[i / kSuper];
    const int w = i >> 5;
    for (int x = (i / kSuper) * (kSuper / 32); x < w; ++x) c += __popc(bits[x]);
    if (i & 31) c += __popc(bits[w] & ((1u << (i & 31)) - 1));
    return c;
  };
  const int inside = kept_before(H);  // kept tokens that need not move
  for (int w = tid; w < words; w += kSelThreads) {
    uint32_t word = bits[w];
    if (word == 0) continue;
    int r = w * 32 + 31 >= H ? kept_before(w * 32) : 0;
    while (word != 0) {
      const int i = w * 32 + __ffs(word) - 1;
      word &= word - 1;
      if (i < H) {
        kept[i] = i;
        ++r;
        continue;
      }
      // The (r - inside)-th place in [0, H) that is not kept.
      const int hole_rank = r - inside;
      ++r;
      int lo = 0, hi = (H - 1) / kSuper;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (mid * kSuper - table[mid] <= hole_rank) lo = mid;
        else hi = mid - 1;
      }
      int left = hole_rank - (lo * kSuper - table[lo]);
      int x = lo * (kSuper / 32);
      for (;; ++x) {
        const int holes = 32 - __popc(bits[x]);
        if (left < holes) break;
        left -= holes;
      }
      uint32_t free_bits = ~bits[x];
      for (; left > 0; --left) free_bits &= free_bits - 1;
      kept[x * 32 + __ffs(free_bits) - 1] = i;
    }
  }
}

// Rows move from kept[i] to i.  Places in [0, H) only take from positions at or
// behind H, so their copies are independent; after them the recent rows move
// down in order, each step reading its rows before any of them is written (a
// place is written only after the row that was there has been read: a row's
// new place is never behind its old one).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  const int unit = blockIdx.x >> 1;
  const int s = unit / p.num_kv_heads;
  const int j = unit - s * p.num_kv_heads;
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  const int32_t *kept = p.kept + (int64_t)unit * p.budget;
  const int H = p.budget - p.recent;
  const int L = p.context_lens[s];
  if (L <= p.budget || kept[p.budget - 1] < 0) return;  // (-1 in the last place: a bad sequence)
  uint4 *cache = reinterpret_cast<uint4 *>((blockIdx.x & 1) ? p.v_cache : p.k_cache);
  const bool sums = (blockIdx.x & 1) == 0;  // the K unit moves the weights too
  const int shift = p.block_shift;
  const int V = p.row_vecs;
  auto row = [&](int i) { return cache + (slot_at(bt, i, shift) * p.num_kv_heads + j) * V; };

  for (int x = threadIdx.x; x < H * V; x += kMoveThreads) {
    const int i = x / V, v = x - i * V;
    const int src = kept[i];
    if (src != i) {
      row(i)[v] = row(src)[v];
      if (sums && v == 0)
        p.key_weights[weight_at(bt, i, shift, p.num_kv_heads, j)] =
            p.key_weights[weight_at(bt, src, shift, p.num_kv_heads, j)];
    }
  }
  __syncthreads();
  const int total = p.recent * V;
  for (int base = 0; base < total; base += kMoveThreads) {
    const int x = base + threadIdx.x;
    const int i = x / V, v = x - i * V;
    uint4 a = make_uint4(0, 0, 0, 0);
    float w = 0.f;
    if (x < total) {
      a = row(L - p.recent + i)[v];
      if (sums && v == 0) w = p.key_weights[weight_at(bt, L - p.recent + i, shift, p.num_kv_heads, j)];
    }
    __syncthreads();
    if (x < total) {
      row(H + i)[v] = a;
      if (sums && v == 0) p.key_weights[weight_at(bt, H + i, shift, p.num_kv_heads, j)] = w;
    }
  }
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
  if (new_lens == context_lens) return PKV_ERR_INVALID_ARG;  // every kv head reads the old length

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
  const int room = max_blocks_per_seq * block_size;
  const int smem = (room / 32 + room / kSuper + 4) * 4;
  int ctas = 0;
  if (!kernel_smem_setup((const void *)evict_select_kernel, kSelThreads, smem, &ctas))
    return PKV_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  evict_select_kernel<<<(unsigned)units, kSelThreads, smem, st>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  evict_move_kernel<<<(unsigned)(2 * units), kMoveThreads, 0, st>>>(prm);
  return launch_status();
}
