// prefill_weights.cu -- the attention weight that a prompt chunk's last queries
// give to each key (tcgen05).
//
// For sequence s with n new queries, c cached tokens and R = min(window, n),
// the sum of key p (kv head j) receives
//   a[p] = sum over queries i in [n - R, n) with c + i >= p, and over the query
//          heads h of j's group, of softmax_p(scale <q[i,h], K[p,j]>):
// added for keys cached before the chunk, set for the chunk's own: the first pass
// clears the sums of those, and the second one, which runs when all of the first
// has ended, adds to every key's.  (A sequence's own key may be another one's
// cached key, where both hold a block and are in the same call: cleared before
// anything is added, its sum has the weights of both whichever comes first.)
//
// A weight needs its row's softmax denominator, which needs the whole row, so
// the product Q K^T is computed twice rather than kept (a pair's logit is 4
// bytes; computing it again is 2 D operations on operands that are in L2):
//  1. Rows: S = Q K^T with the rows in the lanes of tensor memory (M = 128 rows:
//     128 / G queries of the G heads that share the keys; N = 128 keys).  A
//     thread owns a row and keeps its running maximum and sum over the row's key
//     tiles.
//  2. Keys: S^T = K Q^T with the keys in the lanes, so that summing a key's
//     weights over the rows is a sum inside one thread.
// A step is one 128 x 128 product of a key tile and a row tile that sees any of
// it.  All steps of the call, in the order (sequence, kv head, row tile, key
// tile) or, second pass, (sequence, kv head, key tile, row tile), are cut into
// one run of equal length per CTA, whatever the lengths of the sequences.  A row
// tile (key tile) whose steps fall to several CTAs is joined by the last of them
// to finish (a counter; nothing waits), from the parts in their order, so the
// result does not depend on which one that is.
// Both passes are the same persistent kernel: warp 0 loads tiles (TMA, 128-byte
// swizzle, through the block table), warps 1 and 2 issue tcgen05.mma in turn (one
// fills the queue while the other waits for its operands) into four 128-column
// buffers of tensor memory, warp 3 clears the sums of the chunks' keys (first pass)
// or fetches the rows' denominators (second pass), warps 4-19 exponentiate and sum,
// a group of four for each buffer.  Loads, products and exponentials of different
// steps overlap.
//
// A row's denominator is kept as one fp32, its -log2 (the maximum included), rounded
// by 2^-24 of itself: each weight of the row is off by 2^-24 ln 2 times that number,
// 1e-6 where it is 24 (1000 keys of logits near 10).  Maximum and sum apart would be
// exact to the sum, and cost a second read of shared memory for every exponential of
// the second pass, where the one there is takes 6 of 80 us.
//
// Measured (first and second pass alone, us; the call):
//   window of 32, 16 prompts to 4096 tokens, 16 heads on 8, D = 128:  26 + 23, 35
//   12 chunks of 100 to 512 on up to 7800 cached, window 64, 32 heads on 8,
//   D = 64:                                                           41 + 51, 80
//   8 whole prompts of 300 to 2048, 16 heads on 8, D = 128:           49 + 54, 90
// A window's first pass is the reading of K (73 MB) and the two prologues.  In the
// others no single stage is the bound: a step takes 0.40 to 0.50 us, its 16384
// exponentials alone 0.26 (62 a nanosecond and SM), with scaling and sum 0.33; its
// product 0.17 (D = 64) or 0.33; and copies without exponentials, tensor-memory loads
// and three quarters of each product were only 9 to 17 % faster.  What is left is the
// hand-over between steps: a group has one S buffer, and from its last load of it
// until the next product has arrived it has the last 32 columns' exponentials to do.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;       // rows and keys per tile
constexpr int kGroups = 4;       // of four warps: exponentials and sums
constexpr int kIssuers = 2;
constexpr int kThreads = 128 + kGroups * 128;
constexpr int kBufs = kGroups;   // S buffers of 128 columns: all of tensor memory
constexpr int kKeep = 2;         // row tiles that stay in their slots for a whole head
constexpr int kStatSlots = 8;    // row tiles' denominators (second pass)
constexpr int kStatAhead = 4;    // of them on their way at a time
constexpr int kMaxTokens = 1 << 20;  // of a sequence (a head's steps are counted in 32 bits)
constexpr int kMaxCtas = 512;    // places for cut tiles in the workspace (CTAs of a grid at most)
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int PASS>
struct Layout {
  static constexpr int kTileBytes = kTile * D * 2;
  // Row tiles stream in the second pass (8 whole prompts: 58 us with 2 and 4 slots,
  // 55 with 3 and 3 or 4 and 2; a window of 32, where keys stream there too, 21, 21
  // and 23), keys in the first.
  static constexpr int kQSlots = PASS == 1 ? 2 : 3;
  static constexpr int kKSlots = (D == 128 ? 6 : 8) - kQSlots;
  static constexpr int q = 0;
  static constexpr int k = q + kQSlots * kTileBytes;
  static constexpr int bars = k + kKSlots * kTileBytes;
  // q_full/q_empty[Q], st_empty[T], k_full/k_empty[K], s_full/s_empty[B],
  // x_empty[quarter][2], drain
  static constexpr int kNumBars =
      2 * kQSlots + kStatSlots + 2 * kKSlots + 2 * kBufs + 8 + 1;
  static constexpr int stat = (bars + kNumBars * 8 + 15) & ~15;  // [T][128] -log2 denominators
  static constexpr int ex = stat + kStatSlots * kTile * 4;       // [2][groups][128] (maximum, sum)
  static constexpr int misc = ex + 2 * kGroups * kTile * 8;  // tensor memory address, abort, run, scan
  static constexpr int total = misc + 512;
  // One CTA per SM (it takes all of tensor memory): more than half of an SM's
  // shared memory, so that a second one never waits for tensor memory.
  static_assert(total + 1024 <= 232448 && total > 114 * 1024, "shared memory");
};

struct PromptParams {
  float *key_weights;
  const int32_t *block_tables;
  const int32_t *cu_q;
  const int32_t *cu_k;
  float *neg_lse;           // [stat rows, Hq]: -log2 of a row's softmax denominator
  float2 *parts;            // [CTA][2][128]: parts of tiles cut between CTAs
  unsigned int *tickets;    // [2][kMaxCtas][4]: parts of a cut tile that are done, by its first CTA and lane quarter
  int32_t *status;
  int64_t num_blocks;
  int64_t total_q;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int group;         // Hq / Hkv: 1 << group_shift
  int group_shift;
  int block_shift;
  int max_blocks_per_seq;
  int max_seqlen_q;
  int window;
  int rows;          // min(window, max_seqlen_q): counted queries per sequence at most
  int by_query;      // a row's statistics are filed under its query (else sequence and rank)
  int loading[2];    // CTAs of each pass that load their tiles: all, but in a test
  float qscale;
};

// One sequence of the call: its last R queries count, from position base on.
struct Seq {
  int q_first;  // the first counted query's row of q
  int R, c, len_k, base;
  int nrt, nkt;  // row tiles, key tiles
};

// False when the sequence has no queries or its lengths do not fit (then
// flagged, if told to).
__device__ __forceinline__ bool seq_at(const PromptParams &p, int s, Seq &q, bool tell) {
  const int q_begin = p.cu_q[s];
  const int n = p.cu_q[s + 1] - q_begin;
  q.len_k = p.cu_k[s + 1] - p.cu_k[s];
  q.c = q.len_k - n;
  if (n == 0) return false;
  if (n < 0 || n > p.max_seqlen_q || q.c < 0 || q_begin < 0 ||
      q.len_k > ((int64_t)p.max_blocks_per_seq << p.block_shift) ||
      (int64_t)q_begin + n > p.total_q) {
    if (tell) flag_status(p.status, PKV_DEV_BAD_SEQLEN);
    return false;
  }
  q.R = min(n, p.window);
  q.q_first = q_begin + n - q.R;
  q.base = q.len_k - q.R;
  q.nrt = (q.R + (kTile >> p.group_shift) - 1) >> (7 - p.group_shift);
  q.nkt = (q.len_k + kTile - 1) >> 7;
  return true;
}

// (128 / G is a power of two: divisions by it, and by a tile, are shifts)
__device__ __forceinline__ int tq_shift(const PromptParams &p) { return 7 - p.group_shift; }
static_assert(kTile == 128 && kThreads / 32 <= 32, "shifts by 7; a lane per warp");

// Key tiles that row tile rt sees: up to its last query's position.
__device__ __forceinline__ int tiles_seen(const PromptParams &p, const Seq &q, int rt) {
  return ((q.base + min((rt + 1) << tq_shift(p), q.R) - 1) >> 7) + 1;
}
// The first row tile that sees any of key tile kt.
__device__ __forceinline__ int first_rt(const PromptParams &p, const Seq &q, int kt) {
  return max(kt * kTile - q.base, 0) >> tq_shift(p);  // (queries before that one see none of it)
}
// Steps of one head's first m row tiles (at most 2^30: kMaxTokens).  Row tile
// rt + G starts 128 positions later than rt, so it sees one tile more: whole
// turns of G row tiles sum in closed form.
__device__ __forceinline__ int steps_of_rows(const PromptParams &p, const Seq &q, int m) {
  const int turns = m >> p.group_shift, rest = m & (p.group - 1);
  int sum = p.group * (turns * (turns - 1) / 2) + turns * rest;
  for (int r = 0; r < p.group; ++r)
    sum += (((q.base + ((r + 1) << tq_shift(p)) - 1) >> 7) + 1) * (turns + (r < rest ? 1 : 0));
  return sum;
}
// Steps of one head's first k key tiles: row tiles from first_rt on, which grows
// by G with every key tile once it is past zero.  With k = nkt: all steps.
__device__ __forceinline__ int steps_of_keys(const PromptParams &p, const Seq &q, int k) {
  const int e = (q.base + (1 << tq_shift(p)) - 1) >> tq_shift(p);  // first_rt(kt) = max(0, G kt - e)
  const int k1 = min((e + p.group - 1) >> p.group_shift, k);
  const int n = k - k1;
  return k * q.nrt - (p.group * (k1 * n + n * (n - 1) / 2) - e * n);
}

// The order of the call's work: heads, in them tiles (first pass: row tiles,
// whose steps are key tiles; second pass: the other way round), in them steps.
// A run's length counts a tile's beginning and end too, and a head's, as so many
// steps ahead of it: with one row tile per head and a key tile or two, they are
// most of the work.  Measured: window of 32 queries, 16 prompts of 64 to 4096
// tokens, 47.7 us without and 40.4 us with them; 8 whole prompts 110.7 and 99.5,
// and 93.3 with a second pass's tile (joined between the groups, filed and added)
// counted as two steps.
template <int PASS>
struct Order {
  // Second pass: so few row tiles that they stay in their slots for the whole
  // head, else each step loads its own.
  static __device__ __forceinline__ bool keeps(const Seq &q) { return PASS == 2 && q.nrt <= kKeep; }
  static __device__ __forceinline__ int tiles(const Seq &q) { return PASS == 1 ? q.nrt : q.nkt; }
  static __device__ __forceinline__ int per_tile(const Seq &q) { return keeps(q) ? 0 : PASS; }
  static __device__ __forceinline__ int per_head(const Seq &q) { return keeps(q) ? 2 : 0; }
  // Where tile m of a head starts.
  static __device__ __forceinline__ int start(const PromptParams &p, const Seq &q, int m) {
    return (PASS == 1 ? steps_of_rows(p, q, m) : steps_of_keys(p, q, m)) + m * per_tile(q) +
           per_head(q);
  }
  static __device__ __forceinline__ int length(const PromptParams &p, const Seq &q) {  // of a head
    return steps_of_keys(p, q, q.nkt) + tiles(q) * per_tile(q) + per_head(q);
  }
};

// A CTA's run: from step `in` of tile `tile` of head j of sequence s on, up to
// step `end_in` of end_tile of end_j of end_s, which is the next run's first.
struct Run {
  int64_t begin, end, length;  // in the order; of every CTA's run
  int s, j, tile, in;
  int end_s, end_j, end_tile, end_in;
  Seq q;                       // sequence s
};

// A role's walk over its CTA's run, head by head: of head (s, j) the tiles
// [t0, t1], of which the first may have lost its first steps to the CTA before
// and the last its last ones to the next.
template <int PASS>
struct Walk {
  const PromptParams &p;
  const Run *run;
  Seq q;
  int s, j, t0, t1;
  int in, out;
  bool some;

  __device__ __forceinline__ Walk(const PromptParams &prm, const Run *r) : p(prm), run(r) {
    some = r->begin < r->end;
    q = r->q;
    s = r->s;
    j = r->j;
    t0 = r->tile;
    in = r->in;
    set_end();
  }
  __device__ __forceinline__ bool last() const { return s == run->end_s && j == run->end_j; }
  __device__ __forceinline__ void set_end() {
    t1 = Order<PASS>::tiles(q) - 1;
    out = 0x7FFFFFFF;
    if (last()) {
      const bool part = run->end_in > 0;
      t1 = run->end_tile - (part ? 0 : 1);
      if (part) out = run->end_in;
      some = some && t0 <= t1;
    }
  }
  __device__ __forceinline__ bool more() const { return some; }
  __device__ __forceinline__ void next() {
    if (last()) {
      some = false;
      return;
    }
    t0 = in = 0;
    if (++j == p.num_kv_heads) {
      j = 0;
      do {
        if (++s == run->end_s && run->end_j + run->end_tile + run->end_in == 0) {
          some = false;  // (also the end of the batch)
          return;
        }
      } while (!seq_at(p, s, q, false));
    }
    set_end();
  }
  __device__ __forceinline__ bool keeps() const { return Order<PASS>::keeps(q); }
  // Steps [b0, b1) of tile t, of which [x0, x1) are here.
  __device__ __forceinline__ void steps(int t, int &b0, int &b1, int &x0, int &x1) const {
    b0 = PASS == 1 ? 0 : first_rt(p, q, t);
    b1 = PASS == 1 ? tiles_seen(p, q, t) : q.nrt;
    x0 = b0 + (t == t0 ? in : 0);
    x1 = t == t1 ? min(b1 - b0, out) + b0 : b1;
  }
  // The statistics' row of row `row` of row tile rt.
  __device__ __forceinline__ int64_t stat_at(int rt, int row) const {
    const int r = (rt << tq_shift(p)) + (row >> p.group_shift);
    const int64_t at = p.by_query ? (int64_t)q.q_first + r : (int64_t)s * p.rows + r;
    return at * p.num_q_heads + (j << p.group_shift) + (row & (p.group - 1));
  }
  // Last key that row `row` of row tile rt sees; -1: no such row.
  __device__ __forceinline__ int sees(int rt, int row) const {
    const int r = (rt << tq_shift(p)) + (row >> p.group_shift);
    return r < q.R ? q.base + r : -1;
  }
  // The sum of a key in block blk.
  __device__ __forceinline__ float *sum_of(int blk, int key) const {
    return p.key_weights + ((((int64_t)blk * p.num_kv_heads + j) << p.block_shift) +
                            (key & ((1 << p.block_shift) - 1)));
  }
  __device__ __forceinline__ int tile_rows(int rt) const {
    return min(1 << tq_shift(p), q.R - (rt << tq_shift(p))) << p.group_shift;
  }
};

// Wait on a barrier of the pass.  What the second pass's roles wait for can depend
// on denominators, hence on the first pass, which may have long to go when a CTA
// that shares the GPU with its tail begins (runs are equal by steps, not by time: up
// to a fifth of the pass).  So the limit counts from the first pass's end on.
template <int PASS>
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  if (PASS == 2) asm volatile("griddepcontrol.wait;" ::: "memory");
  return mbar_wait_slow(bar, parity, abort);
}
template <int PASS>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const bool ok = wait_bar<PASS>(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// Arrive n times at once.
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
               : "memory");
}

// Load 32 consecutive fp32 columns of this thread's lane of tensor memory with
// their maximum (NaN ignored), and wait for them.
__device__ __forceinline__ void tmem_load32_max(uint32_t taddr, float (&v)[32], float &vmax) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(vmax)
      : "r"(taddr)
      : "memory");
}

// Copy 4 bytes to shared memory, asynchronously.
__device__ __forceinline__ void cp_async4(float *dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A count in shared memory that one warp raises and others wait for.
__device__ __forceinline__ void count_set(int *count, int n) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(count)), "r"(n) : "memory");
}
__device__ __forceinline__ int count_get(const int *count) {
  int n;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(n) : "r"(smem_u32(count)) : "memory");
  return n;
}
// Raise it by one and return what it was.
__device__ __forceinline__ int count_add(int *count) {
  int n;
  asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
               : "=r"(n)
               : "r"(smem_u32(count))
               : "memory");
  return n;
}
// Whole warp, second pass: wait until the count has passed n, as long as a barrier's
// wait may last.
__device__ __forceinline__ bool count_wait(const int *count, int n, volatile int *abort) {
  bool ok = true;
  if (count_get(count) - n <= 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1; ok && count_get(count) - n <= 0; ++i) {
      if ((i & 15u) == 0) {
        if (*abort) ok = false;
        else if (global_timer_ns() - t0 > g_wait_limit_ns) {
          *abort = 1;
          ok = false;
        }
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Position in a ring of n slots whose barriers alternate phases.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;  // of the slot's "full"; its "empty" is waited for with phase ^ 1
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};
// The position x places on (x <= n).
__device__ __forceinline__ Ring ring_at(Ring r, int x, int n) {
  r.slot += x;
  if (r.slot >= n) {
    r.slot -= n;
    r.phase ^= 1;
  }
  return r;
}

// Warp: the tile of a head that place `at` of it belongs to, and the step of
// that tile; 32 candidates at a time.
template <int PASS>
__device__ __forceinline__ int find_tile(const PromptParams &p, const Seq &q, int at, int &in) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = Order<PASS>::tiles(q);  // in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int x = lo + lane * step;
    // (the head's own places go to its first tile)
    const bool starts = x == lo || (x < hi && Order<PASS>::start(p, q, x) <= at);
    const int n = __popc(__ballot_sync(0xffffffffu, starts));
    hi = min(hi, lo + n * step);
    lo += (n - 1) * step;
  }
  in = max(at - Order<PASS>::start(p, q, lo) - Order<PASS>::per_tile(q), 0);
  return lo;
}

// All threads: the CTA's run.
template <int PASS>
__device__ void find_run(const PromptParams &p, Run *run, int64_t *scratch, bool tell) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs;
  const int per = (S + kThreads - 1) / kThreads;  // (one, for batches up to kThreads)
  const int s0 = min(tid * per, S), s1 = min(s0 + per, S);
  int64_t local = 0;
  int each = 0;
  Seq q;
  Seq *qs = reinterpret_cast<Seq *>(scratch + kThreads / 32);  // that of the next run's first place
  for (int s = s0; s < s1; ++s) {
    each = 0;
    if (seq_at(p, s, q, tell)) {
      each = Order<PASS>::length(p, q);
      local += (int64_t)each * p.num_kv_heads;
    }
  }
  int64_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  // The warps that have sequences go on (for most batches one; all of them, each
  // adding up the warps' sums one by one, took 2000 of the prologue's 5700 cycles).
  if (warp * 32 * per < S) {
    const int64_t own = lane < kThreads / 32 ? scratch[lane] : 0;
    int64_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
    const int64_t before = incl - local + __shfl_sync(0xffffffffu, upto - own, warp);
    const int64_t most = total + gridDim.x - 1;
    const int64_t length = most <= 0xFFFFFFFFll ? (int64_t)((uint32_t)most / gridDim.x)
                                                : most / gridDim.x;
    const int64_t begin = min(length * blockIdx.x, total), end = min(begin + length, total);
    if (tid == 0) {
      run->begin = begin;
      run->end = end;
      run->length = length;
      if (end == total) {  // the end of the batch
        run->end_s = S;
        run->end_j = run->end_tile = run->end_in = 0;
      }
    }
    // The sequence and head of the run's first place, then of the next run's.
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t at = x == 0 ? begin : end;
      if (at >= total || at < before || at >= before + local) continue;
      int64_t b = before;
      int s = s0;
      if (per > 1) {
        for (; s < s1; ++s) {
          if (!seq_at(p, s, q, false)) continue;
          each = Order<PASS>::length(p, q);
          if (at < b + (int64_t)each * p.num_kv_heads) break;
          b += (int64_t)each * p.num_kv_heads;
        }
      }
      const int64_t offset = at - b;
      const int j = offset <= 0xFFFFFFFFll ? (int)((uint32_t)offset / (uint32_t)each)
                                           : (int)(offset / each);
      const int in = (int)(offset - (int64_t)j * each);  // (place in the head, until the tile is found)
      if (x == 0) {
        run->s = s;
        run->j = j;
        run->in = in;
        run->q = q;
      } else {
        run->end_s = s;
        run->end_j = j;
        run->end_in = in;
        *qs = q;
      }
    }
  }
  __syncthreads();
  if (warp == 0 ? run->begin < run->end : warp == 1 && run->end_s < S) {
    int in;
    const int tile =
        find_tile<PASS>(p, warp == 0 ? run->q : *qs, warp == 0 ? run->in : run->end_in, in);
    __syncwarp();
    if (lane == 0) {
      if (warp == 0) {
        run->tile = tile;
        run->in = in;
      } else {
        run->end_tile = tile;
        run->end_in = in;
      }
    }
  }
}

// All threads of a first-pass CTA whose waits ran out: the row tiles of its run may
// hold no denominators, or an earlier call's.  They are set to weigh nothing, so that
// the second pass leaves their rows out.  (Another CTA may have finished a tile that
// they share, or be about to: such a row counts or does not.  A call of its own: the
// kernel has no registers to spare.)
__device__ __noinline__ void leave_out(const PromptParams &p, const Run *run) {
  const int row = threadIdx.x;
  if (row >= kTile) return;
  for (Walk<1> w(p, run); w.more(); w.next())
    for (int t = w.t0; t <= w.t1; ++t)
      if (w.sees(t, row) >= 0) p.neg_lse[w.stat_at(t, row)] = -INFINITY;
}

template <int D, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ PromptParams p) {
  using L = Layout<D, PASS>;
  constexpr int XR = D / 64;  // 128-byte regions across D
  constexpr int kKSlots = L::kKSlots, kQSlots = L::kQSlots;
  static_assert((kStatSlots & (kStatSlots - 1)) == 0 && kBufs == 4 && kIssuers == 2,
                "by the low bits of a count");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem + L::q, *sK = smem + L::k;
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *q_empty = q_full + kQSlots;
  uint64_t *st_empty = q_empty + kQSlots;
  uint64_t *k_full = st_empty + kStatSlots;
  uint64_t *k_empty = k_full + kKSlots;
  uint64_t *s_full = k_empty + kKSlots;
  uint64_t *s_empty = s_full + kBufs;
  uint64_t *x_empty = s_empty + kBufs;
  uint64_t *drain = x_empty + 8;
  float *stat = reinterpret_cast<float *>(smem + L::stat);
  float2 *ex = reinterpret_cast<float2 *>(smem + L::ex);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  int *stats_in = reinterpret_cast<int *>(smem + L::misc + 8);  // row tiles whose denominators are in
  int *parts_in = reinterpret_cast<int *>(smem + L::misc + 16);  // groups that are through with a tile, [quarter][2]
  Run *run = reinterpret_cast<Run *>(smem + L::misc + 48);
  int64_t *scratch = reinterpret_cast<int64_t *>(smem + L::misc + 160);
  static_assert(sizeof(Run) <= 112 && 160 + kThreads / 32 * 8 + sizeof(Seq) <= 512, "");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], kIssuers);
    }
    for (int i = 0; i < kStatSlots; ++i) mbar_init(&st_empty[i], kGroups * 4);
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], PASS == 1 ? 1 : kIssuers);  // (a step's own, or all of a tile's)
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&x_empty[i], 1);
      parts_in[i] = 0;
    }
    mbar_init(drain, kIssuers);
    *abort_flag = 0;
    *stats_in = 0;
    fence_barrier_init();
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
  }
  __syncwarp();
  // (the first pass may start under the tail of the kernel before the call; the
  // second one starts when all of the first pass is past this point)
  if (PASS == 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  find_run<PASS>(p, run, scratch, PASS == 1 && blockIdx.x == 0);
  // Tensor memory after that wait only: the kernel before the call may still have
  // to take its own, and would wait for this CTA's as this CTA for its end.  (The
  // second pass's CTAs wait for first-pass ones, which have theirs and end.)
  if (warp == 1) {
    tmem_alloc(tmem_slot, kBufs * kTile);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  if (PASS == 1) {
    // This pass is alone on the stream until it lets the second one start: it
    // clears that one's counters (and the second pass clears this one's).
    if (threadIdx.x < 4) p.tickets[(kMaxCtas + blockIdx.x) * 4 + threadIdx.x] = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }

  // Every role walks the same run.  First pass: a Q tile per tile, a K tile per
  // step.  Second pass: a K tile per tile, a Q tile per step or, where all row
  // tiles of a sequence fit the slots, one load of each per (sequence, head).
  // A wait on a barrier tells only two phases apart, so whoever waits for a slot
  // must see every use of it: S buffer g belongs to group g and to issuer g & 1;
  // both issuers wait for, and release, every Q tile, and every K tile of the
  // second pass; the denominators, which a group may skip many of, are counted.
  if (warp == 0) {
    // ---- loads ----
    if (lane == 0) {
      Ring rk, rq;
      int k_loads = 0, q_loads = 0;
      bool ok = (int)blockIdx.x < p.loading[PASS - 1];
      const uint32_t in_block = (1u << p.block_shift) - 1;
      const bool two = in_block < kTile - 1;  // blocks of 64: two per tile
      for (Walk<PASS> w(p, run); ok && w.more(); w.next()) {
        const int32_t *bt = p.block_tables + (int64_t)w.s * p.max_blocks_per_seq;
        // A tile's block ids: one, or of blocks of 64 two, the second of which
        // may lie past the keys (it is then the first again, unused).  The next
        // tile's are asked for as a tile is loaded.
        int near = -1, blk0 = 0, blk1 = 0;  // of tile `near`
        auto ask_blocks = [&](int kt) {
          near = kt;
          const int at1 = kt * kTile + 64;
          blk0 = bt[(kt * kTile) >> p.block_shift];
          blk1 = two && at1 < w.q.len_k ? bt[at1 >> p.block_shift] : blk0;
        };
        auto load_k = [&](int kt) -> bool {
          if (near != kt) ask_blocks(kt);
          if (blk0 < 0 || blk0 >= p.num_blocks || blk1 < 0 || blk1 >= p.num_blocks) {
            flag_status(p.status, PKV_DEV_BAD_BLOCK);
            if (blk0 < 0 || blk0 >= p.num_blocks) blk0 = 0;
            if (blk1 < 0 || blk1 >= p.num_blocks) blk1 = 0;
          }
          if (!wait_bar<PASS>(&k_empty[rk.slot], rk.phase ^ 1, abort_flag)) return false;
          uint8_t *kd = sK + rk.slot * L::kTileBytes;
          mbar_arrive_expect_tx(&k_full[rk.slot], L::kTileBytes);
#pragma unroll
          for (int x = 0; x < XR; ++x) {
            uint8_t *region = kd + x * kTile * 128;
            tma_load_4d(region, &tm_k, &k_full[rk.slot], x * 64, w.j, (kt * kTile) & in_block, blk0);
            if (two) tma_load_4d(region + 64 * 128, &tm_k, &k_full[rk.slot], x * 64, w.j, 0, blk1);
          }
          if (kt + 1 < w.q.nkt) ask_blocks(kt + 1);
          ++k_loads;
          rk.next(kKSlots);
          return true;
        };
        auto load_q = [&](int rt) -> bool {
          const int slot = rq.slot;
          if (!wait_bar<PASS>(&q_empty[slot], rq.phase ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(&q_full[slot], L::kTileBytes);
#pragma unroll
          for (int x = 0; x < XR; ++x)
            tma_load_3d(sQ + slot * L::kTileBytes + x * kTile * 128, &tm_q, &q_full[slot], x * 64,
                        w.j << p.group_shift, w.q.q_first + (rt << tq_shift(p)));
          ++q_loads;
          rq.next(kQSlots);
          return true;
        };
        const bool keeps = w.keeps();
        for (int t = w.t0; ok && t <= w.t1; ++t) {
          int b0, b1, x0, x1;
          w.steps(t, b0, b1, x0, x1);
          if (PASS == 1) {
            ok = load_q(t);
            for (int x = x0; ok && x < x1; ++x) ok = load_k(x);
          } else {
            ok = load_k(t);
            if (keeps) {
              for (int x = 0; ok && t == w.t0 && x < w.q.nrt; ++x) ok = load_q(x);
            } else {
              for (int x = x0; ok && x < x1; ++x) ok = load_q(x);
            }
          }
        }
      }
      // Do not leave while copies into this CTA's shared memory are in flight.
      for (int i = max(0, k_loads - kKSlots); i < k_loads; ++i)
        if (!mbar_wait_bounded(&k_full[i % kKSlots], (i / kKSlots) & 1, nullptr))
          flag_status(p.status, PKV_DEV_TIMEOUT);
      for (int i = max(0, q_loads - kQSlots); i < q_loads; ++i)
        if (!mbar_wait_bounded(&q_full[i % kQSlots], (i / kQSlots) & 1, nullptr))
          flag_status(p.status, PKV_DEV_TIMEOUT);
    }
  } else if (warp <= kIssuers) {
    // ---- products: the two warps take the steps in turn ----
    if (lane == 0) {
      const int me = warp - 1;
      Ring rk, rq;
      const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = umma_desc_sw128(smem_u32(sK), 16, 1024);
      bool ok = true;
      int k = 0;  // steps taken in turn
      uint32_t uses = 0;  // bit g: parity of the uses of buffer g
      // The product of a Q slot and a K slot into buffer g.
      auto product = [&](int qslot, int kslot, int g, uint32_t idesc) -> bool {
        if (!wait_bar<PASS>(&s_empty[g], ((uses >> g) & 1) ^ 1, abort_flag)) return false;
        uses ^= 1u << g;
        tc_fence_after_sync();
        const uint64_t a = dq + (uint64_t)((qslot * L::kTileBytes) >> 4);
        const uint64_t b = dk + (uint64_t)((kslot * L::kTileBytes) >> 4);
        const uint32_t d = tmem + g * kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk / 4) * kTile * 128 + (kk & 3) * 32) >> 4);
          umma_bf16(d, PASS == 1 ? a + off : b + off, PASS == 1 ? b + off : a + off, idesc,
                    kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[g]);
        return true;
      };
      for (Walk<PASS> w(p, run); ok && w.more(); w.next()) {
        const bool keeps = w.keeps();
        if (keeps) {
          for (int x = 0; ok && x < w.q.nrt; ++x) {
            const Ring at = ring_at(rq, x, kQSlots);
            ok = wait_bar<PASS>(&q_full[at.slot], at.phase, abort_flag);
          }
        }
        for (int t = w.t0; ok && t <= w.t1; ++t) {
          int b0, b1, x0, x1;
          w.steps(t, b0, b1, x0, x1);
          if (PASS == 1) {
            ok = wait_bar<PASS>(&q_full[rq.slot], rq.phase, abort_flag);
            for (int x = x0; ok && x < x1; ++x, ++k) {
              if ((k & 1) == me) {
                ok = wait_bar<PASS>(&k_full[rk.slot], rk.phase, abort_flag) &&
                     product(rq.slot, rk.slot, k & 3,
                             umma_idesc_bf16(kTile, kTile, false, false));
                if (ok) umma_commit(&k_empty[rk.slot]);
              }
              rk.next(kKSlots);
            }
            if (ok) umma_commit(&q_empty[rq.slot]);
            rq.next(kQSlots);
            continue;
          }
          ok = wait_bar<PASS>(&k_full[rk.slot], rk.phase, abort_flag);
          for (int x = x0; ok && x < x1; ++x) {
            // (no more columns than the row tile has rows, to 16)
            const uint32_t idesc = umma_idesc_bf16(kTile, (w.tile_rows(x) + 15) & ~15, false, false);
            if (keeps) {
              if ((t & 1) == me) ok = product(ring_at(rq, x, kQSlots).slot, rk.slot, t & 3, idesc);
              continue;
            }
            ok = wait_bar<PASS>(&q_full[rq.slot], rq.phase, abort_flag);
            if ((k & 1) != me) {
              if (ok) mbar_arrive(&q_empty[rq.slot]);
            } else if (ok) {
              ok = product(rq.slot, rk.slot, k & 3, idesc);
              if (ok) umma_commit(&q_empty[rq.slot]);
            }
            rq.next(kQSlots);
            ++k;
          }
          if (ok) umma_commit(&k_empty[rk.slot]);
          rk.next(kKSlots);
        }
        if (keeps) {
          for (int x = 0; ok && x < w.q.nrt; ++x)
            umma_commit(&q_empty[ring_at(rq, x, kQSlots).slot]);
          rq = ring_at(rq, w.q.nrt, kQSlots);
        }
      }
      // Wait for the products of both before tensor memory is freed.
      umma_commit(drain);
      if (!wait_bar<PASS>(drain, 0, nullptr)) flag_status(p.status, PKV_DEV_TIMEOUT);
    }
  } else if (warp == 3) {
    if (PASS == 1) {
      // ---- first pass: the sums of the chunks' own keys start at zero ----
      // (The last row tile of a head sees all of its keys, so each key tile is a
      // step of it once.)
      for (Walk<PASS> w(p, run); w.more(); w.next()) {
        if (w.t1 != w.q.nrt - 1) continue;
        int b0, b1, x0, x1;
        w.steps(w.t1, b0, b1, x0, x1);
        for (int x = max(x0, w.q.c >> 7); x < x1; ++x) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = x * kTile + i * 32 + lane;
            if (key < w.q.c || key >= w.q.len_k) continue;
            const int blk =
                p.block_tables[(int64_t)w.s * p.max_blocks_per_seq + (key >> p.block_shift)];
            if (blk >= 0 && blk < p.num_blocks) *w.sum_of(blk, key) = 0.f;
          }
        }
      }
    } else {
      // ---- second pass: the rows' denominators ----
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (lane < 4) p.tickets[blockIdx.x * 4 + lane] = 0;
      int q_loads = 0;
      bool ok = true;
      const int apart = 32 >> p.group_shift;  // queries from a lane's row to its next
      // All but the last `ahead` row tiles asked for are in.
      auto tell = [&](auto ahead) {
        asm volatile("cp.async.wait_group %0;" ::"n"(decltype(ahead)::value) : "memory");
        __syncwarp();
        if (lane == 0) count_set(stats_in, q_loads - (int)decltype(ahead)::value);
      };
      for (Walk<PASS> w(p, run); ok && w.more(); w.next()) {
        // (asynchronous copies, kStatAhead row tiles in flight: one row tile every
        // 500 cycles instead of 1200, a step's products taking about 900)
        const float *mine = p.neg_lse + w.stat_at(0, lane);  // this lane's of row tile 0
        auto fill = [&](int rt) -> bool {
          const int slot = q_loads & (kStatSlots - 1);
          if (!warp_wait<PASS>(&st_empty[slot], ((q_loads / kStatSlots) & 1) ^ 1, abort_flag)) return false;
          float *to = stat + slot * kTile + lane;
          const float *from = mine + (int64_t)(rt << tq_shift(p)) * p.num_q_heads;
          const int left = w.q.R - (rt << tq_shift(p)) - (lane >> p.group_shift);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i * apart < left) cp_async4(to + i * 32, from + (int64_t)i * apart * p.num_q_heads);
            else to[i * 32] = -INFINITY;
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          ++q_loads;
          tell(std::integral_constant<int, kStatAhead - 1>());
          return true;
        };
        if (w.keeps()) {
          for (int x = 0; ok && x < w.q.nrt; ++x) ok = fill(x);
          continue;
        }
        for (int t = w.t0; ok && t <= w.t1; ++t) {
          int b0, b1, x0, x1;
          w.steps(t, b0, b1, x0, x1);
          for (int x = x0; ok && x < x1; ++x) ok = fill(x);
        }
      }
      tell(std::integral_constant<int, 0>());
    }
  } else {
    // ---- exponentials and sums: a group of four warps for each S buffer ----
    // They take the steps in turn or, where a tile has few (second pass, row
    // tiles that stay in their slots), the tiles.
    const int quarter = warp & 3;
    const int side = (warp - 4) >> 2;     // the group
    const int row = quarter * 32 + lane;  // the thread's lane of tensor memory
    const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + side * kTile;
    const float qs = p.qscale;
    const float2 qs2 = make_float2(qs, qs);
    bool ok = true;
    int q_loads = 0, swaps = 0, k = 0;  // (k: steps taken in turn)
    uint32_t phase_s = 0;  // of this group's buffer
    auto wait_product = [&]() -> bool {
      if (!warp_wait<PASS>(&s_full[side], phase_s, abort_flag)) return false;
      phase_s ^= 1;
      tc_fence_after_sync();
      return true;
    };
    auto release_product = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[side]);
    };
    auto join = [&](float2 a, float2 b) -> float2 {
      if (PASS == 2) return make_float2(0.f, a.y + b.y);
      const float mn = fmaxf(a.x, b.x);
      const float ref = mn == -INFINITY ? 0.f : mn;
      return make_float2(mn, a.y * fast_exp2(a.x - ref) + b.y * fast_exp2(b.x - ref));
    };
    for (Walk<PASS> w(p, run); ok && w.more(); w.next()) {
      const bool keeps = w.keeps();
      if (keeps) ok = count_wait(stats_in, q_loads + w.q.nrt - 1, abort_flag);
      // (keeps: a group's tiles are those of its number, modulo the groups)
      for (int t = keeps ? w.t0 + ((side - w.t0) & 3) : w.t0; ok && t <= w.t1; t += keeps ? kGroups : 1) {
        int b0, b1, x0, x1;
        w.steps(t, b0, b1, x0, x1);
        // (maximum, sum) of the row, or (-, sum) of the key, over this thread's steps.
        float2 mine = make_float2(PASS == 1 ? -INFINITY : 0.f, 0.f);
        int blk = -1;
        if (PASS == 1) {
          const int last = w.sees(t, row);
          const int most = __reduce_max_sync(0xffffffffu, last);
          const int least = __reduce_min_sync(0xffffffffu, last);
          for (int x = x0 + ((side - k) & 3); x < x1; x += kGroups) {
            ok = wait_product();
            if (!ok) break;
            if (qs > 0.f && x * kTile + kTile - 1 <= least) {  // every key, by every row of the warp
#pragma unroll 4
              for (int c = 0; c < kTile / 32; ++c) {
                float v[32];
                float top;
                tmem_load32_max(ta + c * 32, v, top);
                if (c + 1 == kTile / 32) release_product();
                float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
                const float mn = fmaxf(mine.x, top * qs);
                const float ref = mn == -INFINITY ? 0.f : mn;
                const float2 nref = make_float2(-ref, -ref);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float2 z0 = __ffma2_rn(make_float2(v[i], v[i + 1]), qs2, nref);
                  const float2 z1 = __ffma2_rn(make_float2(v[i + 2], v[i + 3]), qs2, nref);
                  sum0 = __fadd2_rn(sum0, make_float2(fast_exp2(z0.x), fast_exp2(z0.y)));
                  sum1 = __fadd2_rn(sum1, make_float2(fast_exp2(z1.x), fast_exp2(z1.y)));
                }
                sum0 = __fadd2_rn(sum0, sum1);
                mine.y = fmaf(mine.y, fast_exp2(mine.x - ref), sum0.x + sum0.y);
                mine.x = mn;
              }
              continue;
            }
            // Runs of 32 keys, up to the last that any of the warp's rows sees.
            const int runs = min((most - x * kTile + 32) >> 5, kTile / 32);
            if (runs <= 0) release_product();
#pragma unroll 1
            for (int c = 0; c < runs; ++c) {
              const int shown = last - (x * kTile + c * 32);  // of these keys, the last that the row sees
              float v[32];
              float top;
              tmem_load32_max(ta + c * 32, v, top);
              if (c + 1 == runs) release_product();  // (the product is read: the next one may come)
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              float mn, ref;
              // Keys past the row's position are hidden; a scale that is not
              // positive puts the largest logit elsewhere.
              top = -INFINITY;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                v[i] = i <= shown ? v[i] * qs : -INFINITY;
                top = fmaxf(top, v[i]);
              }
              mn = fmaxf(mine.x, top);
              ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                sum[(i >> 1) & 1] = __fadd2_rn(
                    sum[(i >> 1) & 1], make_float2(fast_exp2(v[i] - ref), fast_exp2(v[i + 1] - ref)));
              mine.y = mine.y * fast_exp2(mine.x - ref) +
                       ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
              mine.x = mn;
            }
          }
          k += x1 - x0;
        } else {
          const int key = t * kTile + row;
          if (key < w.q.len_k)
            blk = p.block_tables[(int64_t)w.s * p.max_blocks_per_seq + (key >> p.block_shift)];
          const int skip = keeps ? 0 : (side - k) & 3, by = keeps ? 1 : kGroups;
          float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
          for (int x = x0 + skip; x < x1; x += by) {
            const int load = q_loads + (keeps ? x : x - x0);
            ok = (keeps || count_wait(stats_in, load, abort_flag)) && wait_product();
            if (!ok) break;
            const int rows = w.tile_rows(x);
            // Columns of this key's weights: from its first row that sees it on.
            const int first = (key - w.q.base - (x << tq_shift(p))) * p.group;
            // Every row of the tile sees every key of the tile.
            const bool open = t * kTile + kTile - 1 <= w.q.base + (x << tq_shift(p));
            const float4 *ns =
                reinterpret_cast<const float4 *>(stat + (load & (kStatSlots - 1)) * kTile);
            // No row or key is hidden: all four runs unrolled, where the exponentials
            // are the bound (D = 64, the chunks: 86.3 us without and 83.4 with it;
            // D = 128, where the products take as long, window 39.7 and 41.0, whole
            // prompts 93.3 and 94.2).
            auto open_run = [&](int c0) {
              float v[32];
              tmem_load32(ta + c0, v);
              if (c0 + 32 >= rows) release_product();  // (the product is read: the next one may come)
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 n = ns[(c0 + i) / 4];
                const float2 z0 = __ffma2_rn(make_float2(v[i], v[i + 1]), qs2, make_float2(n.x, n.y));
                const float2 z1 =
                    __ffma2_rn(make_float2(v[i + 2], v[i + 3]), qs2, make_float2(n.z, n.w));
                acc0 = __fadd2_rn(acc0, make_float2(fast_exp2(z0.x), fast_exp2(z0.y)));
                acc1 = __fadd2_rn(acc1, make_float2(fast_exp2(z1.x), fast_exp2(z1.y)));
              }
            };
            auto any_run = [&](int c0) {
              float v[32];
              tmem_load32(ta + c0, v);
              if (c0 + 32 >= rows) release_product();
              const int lo = max(first - c0, 0), n_in = max(min(rows - c0, 32) - lo, 0);
              if (!__any_sync(0xffffffffu, n_in > 0)) return;
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 n = ns[(c0 + i) / 4];
                const float e0 = fast_exp2(fmaf(v[i], qs, n.x)), e1 = fast_exp2(fmaf(v[i + 1], qs, n.y));
                const float e2 = fast_exp2(fmaf(v[i + 2], qs, n.z)), e3 = fast_exp2(fmaf(v[i + 3], qs, n.w));
                acc0.x += (unsigned)(i - lo) < (unsigned)n_in ? e0 : 0.f;
                acc0.y += (unsigned)(i + 1 - lo) < (unsigned)n_in ? e1 : 0.f;
                acc1.x += (unsigned)(i + 2 - lo) < (unsigned)n_in ? e2 : 0.f;
                acc1.y += (unsigned)(i + 3 - lo) < (unsigned)n_in ? e3 : 0.f;
              }
            };
            if (D == 64 && open && rows == kTile) {
#pragma unroll
              for (int c0 = 0; c0 < kTile; c0 += 32) open_run(c0);
            } else if (D == 64) {
#pragma unroll 1
              for (int c0 = 0; c0 < rows; c0 += 32) any_run(c0);
            } else {
#pragma unroll 1
              for (int c0 = 0; c0 < rows; c0 += 32) {
                if (open && c0 + 32 <= rows) open_run(c0);
                else any_run(c0);
              }
            }
            // (this group alone used the step's denominators: it releases them for all)
            if (!keeps) {
              __syncwarp();
              if (lane == 0) mbar_arrive_n(&st_empty[load & (kStatSlots - 1)], kGroups);
            }
          }
          mine.y = (acc0.x + acc0.y) + (acc1.x + acc1.y);
          if (!keeps) {
            k += x1 - x0;
            q_loads += x1 - x0;
          }
        }
        if (!ok) break;

        // The tile ends here.  Steps taken in turn: the last of the groups to
        // arrive, warp by warp, joins the parts of all, in order; none waits for
        // the others (8 whole prompts 94.8 -> 93.2 us).
        if (!keeps) {
          const int buf = swaps & 1, bar = quarter * 2 + buf;
          ok = warp_wait<PASS>(&x_empty[bar], ((swaps >> 1) & 1) ^ 1, abort_flag);
          if (!ok) break;
          ++swaps;
          float2 *part = ex + buf * kGroups * kTile + row;
          part[side * kTile] = mine;
          __syncwarp();
          int in = 0;
          if (lane == 0) in = count_add(&parts_in[bar]);
          in = __shfl_sync(0xffffffffu, in, 0);
          __syncwarp();
          if (in != kGroups - 1) continue;
          mine = part[0];
#pragma unroll
          for (int x = 1; x < kGroups; ++x) mine = join(mine, part[x * kTile]);
          __syncwarp();
          if (lane == 0) {
            parts_in[bar] = 0;
            mbar_arrive(&x_empty[bar]);
          }
        }
        if (x0 != b0 || x1 != b1) {
          // A part of a tile that several CTAs share: filed by CTA, place 0 if
          // the tile began before it, place 1 if it begins here.  The warp that
          // is the last to file its 32 rows joins all of them, in order.
          const int64_t at = x1 != b1 ? run->end - (x1 - x0) : run->begin;  // the place of step x0
          const int c0 = (int)((at - (x0 - b0)) / run->length);
          const int c1 = (int)((at + (b1 - x0) - 1) / run->length);
          __stcg(p.parts + ((int64_t)blockIdx.x * 2 + (x0 != b0 ? 0 : 1)) * kTile + row, mine);
          __threadfence();
          __syncwarp();
          unsigned int done = 0;
          if (lane == 0) {
            done = atomicAdd(&p.tickets[((PASS - 1) * kMaxCtas + c0) * 4 + quarter], 1u);
            __threadfence();
          }
          done = __shfl_sync(0xffffffffu, done, 0);
          if (done != (unsigned int)(c1 - c0)) continue;
          mine = __ldcg(p.parts + ((int64_t)c0 * 2 + 1) * kTile + row);
          for (int c = c0 + 1; c <= c1; ++c)
            mine = join(mine, __ldcg(p.parts + (int64_t)c * 2 * kTile + row));
        }
        if (PASS == 1) {
          if (w.sees(t, row) >= 0) p.neg_lse[w.stat_at(t, row)] = -(mine.x + log2f(mine.y));
        } else if (blk >= 0 && blk < p.num_blocks) {
          atomicAdd(w.sum_of(blk, t * kTile + row), mine.y);
        }
      }
      if (keeps) {  // every group releases the head's denominators
        __syncwarp();
        for (int x = 0; ok && lane == 0 && x < w.q.nrt; ++x) mbar_arrive(&st_empty[(q_loads + x) & (kStatSlots - 1)]);
        q_loads += w.q.nrt;
      }
    }
  }

  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) flag_status(p.status, PKV_DEV_TIMEOUT);
    if (PASS == 1) leave_out(p, run);
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kBufs * kTile);
  }
}

// The workspace: counters, parts of cut tiles, the rows' denominators.
struct Plan {
  int64_t rows, stat_rows;
  bool by_query;
  size_t parts, neg_lse, total;
  Plan(int64_t num_seqs, int64_t total_q, int64_t max_seqlen_q, int64_t window, int64_t Hq) {
    rows = window < max_seqlen_q ? window : max_seqlen_q;
    // Rows are filed under (sequence, rank) or, where that is more, under their query.
    by_query = rows > total_q / num_seqs;
    stat_rows = by_query ? total_q : num_seqs * rows;
    parts = 2 * kMaxCtas * 4 * sizeof(unsigned int);
    neg_lse = parts + (size_t)kMaxCtas * 2 * kTile * sizeof(float2);
    total = neg_lse + (size_t)(stat_rows * Hq) * sizeof(float);
  }
};

// Test-only fault injection, set by pkv_test_prompt_fault: PromptParams::loading of
// the calls that follow.
std::atomic<int> g_loading[2] = {{kMaxCtas}, {kMaxCtas}};

template <int D>
pkv_status launch(const CUtensorMap &tq, const CUtensorMap &tk, const PromptParams &prm,
                  int64_t most_steps, cudaStream_t stream) {
  constexpr int smem = Layout<D, 1>::total + 1024;
  const int sms = device_sm_count();
  if (sms <= 0 ||
      !kernel_smem_setup((const void *)prompt_weights_kernel<D, 1>, kThreads, smem, nullptr) ||
      !kernel_smem_setup((const void *)prompt_weights_kernel<D, 2>, kThreads, smem, nullptr))
    return PKV_ERR_CUDA;
  int64_t grid = sms < kMaxCtas ? sms : kMaxCtas;
  if (grid > most_steps) grid = most_steps;
  // Both programmatic dependents, the first one of the kernel before the call (a
  // window of 32: 37.2 -> 35.0 us from call to call).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prompt_weights_kernel<D, 1>, tq, tk, prm) == cudaSuccess)
    cudaLaunchKernelEx(&cfg, prompt_weights_kernel<D, 2>, tq, tk, prm);
  return launch_status();  // (either launch's error, which it clears)
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_prefill_weights_workspace_size(int num_seqs, int64_t total_q,
                                                     int max_seqlen_q, int window,
                                                     int num_q_heads, int num_kv_heads,
                                                     int max_blocks_per_seq, int block_size) {
  using namespace pkv;
  if (num_seqs <= 0 || total_q <= 0 || max_seqlen_q <= 0 || window <= 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || max_blocks_per_seq <= 0 || block_size <= 0)
    return 0;
  // (bounded so that no product below can wrap)
  const int64_t group = num_q_heads / num_kv_heads;
  if (group < 1 || num_q_heads > (1 << 16) || total_q > 0x7FFFFFFFLL ||
      (int64_t)max_blocks_per_seq * block_size > 0x7FFFFFFFLL)
    return 0;
  return Plan(num_seqs, total_q, max_seqlen_q, window, num_q_heads).total;
}

extern "C" pkv_status pkv_paged_prefill_weights(
    float *key_weights, const uint16_t *q, const uint16_t *k_cache, const int32_t *block_tables,
    const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs, int64_t total_q,
    int max_seqlen_q, int window, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    int max_blocks_per_seq, int64_t num_blocks, float scale, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || window <= 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / num_kv_heads;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (G != 1 && G != 2 && G != 4 && G != 8) return PKV_ERR_UNSUPPORTED;
  if (block_size != 64 && block_size != 128 && block_size != 256 && block_size != 512)
    return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > kMaxTokens) return PKV_ERR_UNSUPPORTED;
  // NaN or infinite, itself or in the exponentials' base 2 (a logit of zero would be NaN)
  if (!isfinite(scale * kLog2e)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return PKV_OK;
  if (total_q > 0x7FFFFFFFLL) return PKV_ERR_UNSUPPORTED;
  if (!key_weights || !q || !k_cache || !block_tables || !cu_seqlens_q || !cu_seqlens_k)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || (reinterpret_cast<uintptr_t>(key_weights) & 3u) != 0)
    return PKV_ERR_INVALID_ARG;
  const size_t need = pkv_prefill_weights_workspace_size(num_seqs, total_q, max_seqlen_q, window,
                                                         num_q_heads, num_kv_heads,
                                                         max_blocks_per_seq, block_size);
  if (need == 0) return PKV_ERR_INVALID_ARG;  // a workspace that size cannot be addressed
  if (workspace == nullptr || workspace_bytes < need ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_WORKSPACE;
  const Plan plan(num_seqs, total_q, max_seqlen_q, window, num_q_heads);
  PromptParams prm;
  prm.key_weights = key_weights;
  prm.block_tables = block_tables;
  prm.cu_q = cu_seqlens_q;
  prm.cu_k = cu_seqlens_k;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  prm.tickets = reinterpret_cast<unsigned int *>(ws);
  prm.parts = reinterpret_cast<float2 *>(ws + plan.parts);
  prm.neg_lse = reinterpret_cast<float *>(ws + plan.neg_lse);
  prm.status = dev_status;
  prm.num_blocks = num_blocks;
  prm.total_q = total_q;
  prm.num_seqs = num_seqs;
  prm.num_q_heads = num_q_heads;
  prm.num_kv_heads = num_kv_heads;
  prm.group = G;
  prm.group_shift = 31 - __builtin_clz((unsigned)G);
  prm.block_shift = 31 - __builtin_clz((unsigned)block_size);
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.max_seqlen_q = max_seqlen_q;
  prm.window = window;
  prm.rows = (int)plan.rows;
  prm.by_query = plan.by_query ? 1 : 0;
  prm.loading[0] = g_loading[0];
  prm.loading[1] = g_loading[1];
  prm.qscale = scale * kLog2e;

  // q as {D, Hq, T}: a box is 64 dims x the G heads of a kv head x 128 / G
  // queries, in shared memory 128 rows with the heads of a query side by side.
  const uint64_t qdims[3] = {(uint64_t)head_dim, (uint64_t)num_q_heads, (uint64_t)total_q};
  const uint64_t qstr[2] = {(uint64_t)head_dim * 2, (uint64_t)num_q_heads * head_dim * 2};
  const uint32_t qbox[3] = {64u, (uint32_t)G, (uint32_t)(kTile / G)};
  // cache as {D, Hkv, block_size, NB}: a box is 64 dims x 1 head x 128 tokens (64
  // of blocks that have no more) x 1 block.
  const uint64_t kdims[4] = {(uint64_t)head_dim, (uint64_t)num_kv_heads, (uint64_t)block_size,
                             (uint64_t)num_blocks};
  const uint64_t kstr[3] = {(uint64_t)head_dim * 2, (uint64_t)num_kv_heads * head_dim * 2,
                            (uint64_t)block_size * num_kv_heads * head_dim * 2};
  const uint32_t kbox[4] = {64u, 1u, (uint32_t)(block_size < kTile ? 64 : kTile), 1u};
  CUtensorMap tq, tk;
  if (!encode_bf16_map(&tq, q, 3, qdims, qstr, qbox, true) ||
      !encode_bf16_map(&tk, k_cache, 4, kdims, kstr, kbox, true))
    return PKV_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Steps that the batch can have at most, a row tile or more each (a small one
  // needs fewer CTAs).
  const int64_t row_tiles = ((int64_t)plan.rows * G + kTile - 1) / kTile;
  const int64_t key_tiles = ((int64_t)max_blocks_per_seq * block_size + kTile - 1) / kTile;
  const double most = (double)num_seqs * num_kv_heads * row_tiles * key_tiles;
  const int64_t most_steps = most < kMaxCtas ? (int64_t)most : kMaxCtas;
  return head_dim == 128 ? launch<128>(tq, tk, prm, most_steps, st)
                         : launch<64>(tq, tk, prm, most_steps, st);
}

// ---------------------------------------------------------------------------
// Test-only fault injection for the bounded waits of the prompt kernel.
// ---------------------------------------------------------------------------

extern "C" pkv_status pkv_test_prompt_fault(int64_t wait_limit_ns, int pass, int loading_ctas) {
  if (wait_limit_ns <= 0 || (pass != 1 && pass != 2) || loading_ctas < -1)
    return PKV_ERR_INVALID_ARG;
  const unsigned long long limit = (unsigned long long)wait_limit_ns;
  if (cudaMemcpyToSymbol(pkv::g_wait_limit_ns, &limit, sizeof(limit)) != cudaSuccess)
    return PKV_ERR_CUDA;
  for (int x = 0; x < 2; ++x)
    pkv::g_loading[x] = pass == x + 1 && loading_ctas >= 0 ? loading_ctas : pkv::kMaxCtas;
  return PKV_OK;
}
