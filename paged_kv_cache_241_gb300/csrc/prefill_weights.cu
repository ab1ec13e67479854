// prefill_weights.cu -- the attention weight that a prompt chunk's last queries
// give to each key (tcgen05).
//
// For sequence s with n new queries, c cached tokens and R = min(window, n),
// the sum of key p (kv head j) receives
//   a[p] = sum over queries i in [n - R, n) with c + i >= p, and over the query
//          heads h of j's group, of softmax_p(scale <q[i,h], K[p,j]>):
// added for keys cached before the chunk, set for the chunk's own.
//
// A weight needs its row's softmax denominator, which needs the whole row, so
// the product Q K^T is computed twice rather than kept (a pair's logit is 4
// bytes; computing it again is 2 D operations on operands that are in L2):
//  1. Rows: S = Q K^T with the rows in the lanes of tensor memory (M = 128 rows:
//     128 / G queries of the G heads that share the keys; N = 128 keys).  A
//     thread owns a row and keeps its running maximum and sum over the row's key
//     tiles (two groups of four warps take the tiles in turn).
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
// swizzle, through the block table), warp 1 issues tcgen05.mma into four
// 128-column buffers of tensor memory, warps 2 and 3 fetch the rows'
// denominators (second pass), warps 4-11 exponentiate and sum.  Loads, products
// and exponentials of different steps overlap.
#include <math.h>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;       // rows and keys per tile
constexpr int kThreads = 384;
constexpr int kEpilogue = 256;   // threads of warps 4-11
constexpr int kBufs = 4;         // S buffers of 128 columns: all of tensor memory
constexpr int kQSlots = 2;       // row tiles, with their denominators (a kept pair is slot0, slot1)
constexpr int kMaxCtas = 512;    // places for cut tiles in the workspace (CTAs of a grid at most)
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Layout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kKSlots = D == 128 ? 4 : 6;
  static constexpr int q = 0;
  static constexpr int k = q + kQSlots * kTileBytes;
  static constexpr int bars = k + kKSlots * kTileBytes;
  // q_full/q_empty[Q], k_full/k_empty[K], s_full/s_empty[B], st_full/st_empty[Q], drain
  static constexpr int kNumBars = 4 * kQSlots + 2 * kKSlots + 2 * kBufs + 1;
  static constexpr int stat = (bars + kNumBars * 8 + 15) & ~15;  // [Q][128] -log2 denominators
  static constexpr int qpos = stat + kQSlots * kTile * 4;        // [Q][128] last visible key, -1: no row
  static constexpr int red = qpos + kQSlots * kTile * 4;         // [2][2][128] exchange between halves
  static constexpr int misc = red + 4 * kTile * 4;  // tensor memory address, abort, last, start, scan
  static constexpr int total = misc + 256;
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
  unsigned int *tickets;    // [2][kMaxCtas]: parts of a cut tile that are done, by its first CTA
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
  const int tq = kTile >> p.group_shift;
  q.nrt = (q.R + tq - 1) / tq;
  q.nkt = (q.len_k + kTile - 1) / kTile;
  return true;
}

// (128 / G is a power of two: divisions by it, and by a tile, are shifts)
__device__ __forceinline__ int tq_shift(const PromptParams &p) { return 7 - p.group_shift; }
static_assert(kTile == 128, "shifts by 7");

// Key tiles that row tile rt sees: up to its last query's position.
__device__ __forceinline__ int tiles_seen(const PromptParams &p, const Seq &q, int rt) {
  return ((q.base + min((rt + 1) << tq_shift(p), q.R) - 1) >> 7) + 1;
}
// The first row tile that sees any of key tile kt.
__device__ __forceinline__ int first_rt(const PromptParams &p, const Seq &q, int kt) {
  return max(kt * kTile - q.base, 0) >> tq_shift(p);  // (queries before that one see none of it)
}
// Steps of the first m row tiles.  Row tile rt + G starts 128 positions later
// than rt, so it sees one tile more: whole turns of G row tiles sum in closed form.
__device__ __forceinline__ int64_t steps_of_rows(const PromptParams &p, const Seq &q, int m) {
  int64_t extra = 0;
  if (m == q.nrt) {  // (the last row tile can be short)
    extra = q.nkt;
    --m;
  }
  const int G = p.group;
  const int64_t turns = m >> p.group_shift;
  const int rest = m & (G - 1);
  int64_t sum = (int64_t)G * (turns * (turns - 1) / 2) + turns * rest;
  for (int r = 0; r < G; ++r) {
    const int64_t seen = (q.base + (r + 1) * (kTile >> p.group_shift) - 1) / kTile + 1;
    sum += seen * (turns + (r < rest ? 1 : 0));
  }
  return sum + extra;
}
// Steps of the first k key tiles (second pass): row tiles from first_rt on, which
// grows by G with every key tile once it is past zero.
__device__ __forceinline__ int64_t steps_of_keys(const PromptParams &p, const Seq &q, int k) {
  const int tq = kTile >> p.group_shift;
  const int64_t e = (q.base + tq - 1) / tq;                 // first_rt(kt) = max(0, G kt - e)
  const int64_t k1 = min((e + p.group - 1) >> p.group_shift, (int64_t)k);
  const int64_t n = k - k1;
  const int64_t skipped = p.group * (k1 * n + n * (n - 1) / 2) - e * n;
  return (int64_t)k * q.nrt - skipped;
}
__device__ __forceinline__ int64_t steps_of(const PromptParams &p, const Seq &q) {
  return steps_of_rows(p, q, q.nrt);
}

// Where a CTA's run of steps starts (found once, by all threads).
struct Start {
  int64_t begin, end;  // steps of the call
  int64_t run;         // steps per CTA
  int64_t offset;      // of `begin` within its sequence
  int s;
};

// A role's walk over its CTA's steps.
template <int PASS>
struct Walk {
  const PromptParams &p;
  int64_t pos, end, run;
  Seq q;
  int s, j, rt, kt, tq;
  int tile_left;   // steps of the tile from this one on, here or not
  bool last_tile;  // of the (sequence, head)
  int loaded;     // second pass, few row tiles: those in their slots for this (sequence, head)
  bool cut_left;  // the current tile's first steps are another CTA's

  __device__ Walk(const PromptParams &prm, const Start &st) : p(prm) {
    pos = st.begin;
    end = st.end;
    run = st.run;
    s = st.s;
    j = rt = kt = loaded = tile_left = 0;
    last_tile = false;
    cut_left = false;
    tq = kTile >> p.group_shift;
    if (pos >= end) return;
    seq_at(p, s, q, false);
    const int64_t each = steps_of(p, q);
    j = (int)(st.offset / each);
    const int64_t at = st.offset - j * each;
    int lo = 0, hi = (PASS == 1 ? q.nrt : q.nkt) - 1;  // the last tile that starts at or before `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((PASS == 1 ? steps_of_rows(p, q, mid) : steps_of_keys(p, q, mid)) <= at) lo = mid;
      else hi = mid - 1;
    }
    const int in = (int)(at - (PASS == 1 ? steps_of_rows(p, q, lo) : steps_of_keys(p, q, lo)));
    cut_left = in > 0;
    if (PASS == 1) {
      rt = lo;
      kt = in;
    } else {
      kt = lo;
      rt = first_rt(p, q, kt) + in;
    }
    enter_tile();
    if (PASS == 1) tile_left -= in;
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ void enter_tile() {
    if (PASS == 1) {
      tile_left = tiles_seen(p, q, rt);
      last_tile = rt + 1 == q.nrt;
    } else {
      tile_left = q.nrt - rt;
      last_tile = kt + 1 == q.nkt;
    }
  }
  // The tile (row tile, or key tile) ends with this step.
  __device__ __forceinline__ bool tile_done() const { return tile_left == 1; }
  // This step is the last of the tile here.
  __device__ __forceinline__ bool last_here() const { return tile_left == 1 || pos + 1 == end; }
  // (sequence, head) ends with this step, here.
  __device__ __forceinline__ bool head_done() const {
    return (last_tile && tile_left == 1) || pos + 1 == end;
  }
  // The first and the last CTA of the current tile.
  __device__ __forceinline__ void ctas(int &first, int &last) const {
    const int done = PASS == 1 ? kt : rt - first_rt(p, q, kt);  // steps of the tile before this one
    first = (int)((pos - done) / run);
    last = (int)((pos + tile_left - 1) / run);
  }
  // Second pass: so few row tiles that they stay in their slots for the whole
  // (sequence, head), else each step loads its own.
  __device__ __forceinline__ bool keeps() const { return PASS == 2 && q.nrt <= kQSlots; }
  __device__ __forceinline__ void next() {
    ++pos;
    if (--tile_left > 0) {
      if (PASS == 1) ++kt;
      else ++rt;
      return;
    }
    if (!more()) return;
    cut_left = false;
    if (!last_tile) {
      if (PASS == 1) {
        ++rt;
        kt = 0;
      } else {
        ++kt;
        rt = first_rt(p, q, kt);
      }
    } else {
      loaded = rt = kt = 0;
      if (++j == p.num_kv_heads) {
        j = 0;
        do ++s; while (!seq_at(p, s, q, false));
      }
    }
    enter_tile();
  }
  // The statistics' row of the tile's row-th product row.
  __device__ __forceinline__ int64_t stat_at(int row) const {
    const int r = rt * tq + (row >> p.group_shift);
    const int64_t at = p.by_query ? (int64_t)q.q_first + r : (int64_t)s * p.rows + r;
    return at * p.num_q_heads + (j << p.group_shift) + (row & (p.group - 1));
  }
  // Last key that product row `row` of row tile rt sees; -1: no such row.
  __device__ __forceinline__ int sees(int row) const {
    const int r = rt * tq + (row >> p.group_shift);
    return r < q.R ? q.base + r : -1;
  }
  __device__ __forceinline__ int tile_rows() const { return min(tq, q.R - rt * tq) << p.group_shift; }
};

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const bool ok = mbar_wait_bounded(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// Barrier of the epilogue warps; true when any thread brought pred, so that all
// of them leave together when a wait has run out.
__device__ __forceinline__ bool epilogue_sync_any(bool pred) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %2, 0;\n\t"
      "bar.red.or.pred q, 1, %1, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(kEpilogue), "r"(pred ? 1 : 0)
      : "memory");
  return r != 0;
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

// All threads: the total number of steps, and where this CTA's run starts.
__device__ void find_start(const PromptParams &p, Start *out, int64_t *warp_sums, bool tell) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs;
  const int per = (S + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, S), s1 = min(s0 + per, S);
  int64_t local = 0;
  for (int s = s0; s < s1; ++s) {
    Seq q;
    if (seq_at(p, s, q, tell)) local += steps_of(p, q) * p.num_kv_heads;
  }
  int64_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - local, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  const int64_t run = max((total + gridDim.x - 1) / gridDim.x, (int64_t)1);
  const int64_t begin = min(run * blockIdx.x, total), end = min(begin + run, total);
  if (tid == 0) {
    out->begin = begin;
    out->end = end;
    out->run = run;
  }
  if (begin < end && before <= begin && begin < before + local) {
    for (int s = s0; s < s1; ++s) {
      Seq q;
      if (!seq_at(p, s, q, false)) continue;
      const int64_t n = steps_of(p, q) * p.num_kv_heads;
      if (begin < before + n) {
        out->s = s;
        out->offset = begin - before;
        break;
      }
      before += n;
    }
  }
  __syncthreads();
}

template <int D, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k, const PromptParams p) {
  using L = Layout<D>;
  constexpr int XR = D / 64;  // 128-byte regions across D
  constexpr int kKSlots = L::kKSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem + L::q, *sK = smem + L::k;
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *q_empty = q_full + kQSlots;
  uint64_t *st_full = q_empty + kQSlots;
  uint64_t *st_empty = st_full + kQSlots;
  uint64_t *k_full = st_empty + kQSlots;
  uint64_t *k_empty = k_full + kKSlots;
  uint64_t *s_full = k_empty + kKSlots;
  uint64_t *s_empty = s_full + kBufs;
  uint64_t *drain = s_empty + kBufs;
  float *stat = reinterpret_cast<float *>(smem + L::stat);
  int *qpos = reinterpret_cast<int *>(smem + L::qpos);
  float *red = reinterpret_cast<float *>(smem + L::red);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  volatile int *last_flag = reinterpret_cast<volatile int *>(smem + L::misc + 8);
  Start *start = reinterpret_cast<Start *>(smem + L::misc + 16);
  int64_t *warp_sums = reinterpret_cast<int64_t *>(smem + L::misc + 64);
  static_assert(sizeof(Start) <= 48 && 64 + kThreads / 32 * 8 <= 256, "");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&st_full[i], 64);
      mbar_init(&st_empty[i], kEpilogue / 32);
    }
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kBufs * kTile);
    tmem_relinquish();
  }
  find_start(p, start, warp_sums, PASS == 1 && blockIdx.x == 0);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  if (PASS == 1) {
    // This pass is alone on the stream until it lets the second one start: it
    // clears that one's counters (and the second pass clears this one's).
    if (threadIdx.x == 0) p.tickets[kMaxCtas + blockIdx.x] = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }

  // Every role walks the same steps.  A K tile stays while the key tile does; a
  // Q tile for its row tile (first pass), for one step, or, where all row tiles
  // of a sequence fit the slots, for the whole (sequence, head).
  if (warp == 0) {
    // ---- loads ----
    if (lane == 0) {
      Ring rq, rk;
      int q_loads = 0, k_loads = 0;
      bool ok = true;
      int kt_in = -1;
      for (Walk<PASS> w(p, *start); w.more(); w.next()) {
        const bool load_q = PASS == 1 ? kt_in < 0 : !(w.keeps() && (w.loaded >> w.rt & 1));
        if (PASS == 1 || kt_in < 0) {
          ok = mbar_wait_bounded(&k_empty[rk.slot], rk.phase ^ 1, abort_flag);
          if (!ok) break;
          uint8_t *kd = sK + rk.slot * L::kTileBytes;
          mbar_arrive_expect_tx(&k_full[rk.slot], L::kTileBytes);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // (a tile's second half may lie past the keys: it reads the first half's block, unused)
            int at = w.kt * kTile + half * 64;
            if (at >= w.q.len_k) at = w.kt * kTile;
            int blk = p.block_tables[(int64_t)w.s * p.max_blocks_per_seq + (at >> p.block_shift)];
            if (blk < 0 || blk >= p.num_blocks) {
              flag_status(p.status, PKV_DEV_BAD_BLOCK);
              blk = 0;
            }
#pragma unroll
            for (int x = 0; x < XR; ++x)
              tma_load_4d(kd + x * kTile * 128 + half * 64 * 128, &tm_k, &k_full[rk.slot], x * 64,
                          w.j, at & ((1 << p.block_shift) - 1), blk);
          }
          ++k_loads;
          rk.next(kKSlots);
        }
        if (load_q) {
          ok = mbar_wait_bounded(&q_empty[rq.slot], rq.phase ^ 1, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&q_full[rq.slot], L::kTileBytes);
#pragma unroll
          for (int x = 0; x < XR; ++x)
            tma_load_3d(sQ + rq.slot * L::kTileBytes + x * kTile * 128, &tm_q, &q_full[rq.slot],
                        x * 64, w.j << p.group_shift, w.q.q_first + w.rt * w.tq);
          ++q_loads;
          rq.next(kQSlots);
          if (w.keeps()) w.loaded |= 1 << w.rt;
        }
        kt_in = w.last_here() ? -1 : w.kt;  // (>= 0: the tile goes on)
      }
      // Do not leave while copies into this CTA's shared memory are in flight.
      for (int i = max(0, k_loads - kKSlots); i < k_loads; ++i)
        if (!mbar_wait_bounded(&k_full[i % kKSlots], (i / kKSlots) & 1, nullptr))
          flag_status(p.status, PKV_DEV_TIMEOUT);
      for (int i = max(0, q_loads - kQSlots); i < q_loads; ++i)
        if (!mbar_wait_bounded(&q_full[i % kQSlots], (i / kQSlots) & 1, nullptr))
          flag_status(p.status, PKV_DEV_TIMEOUT);
    }
  } else if (warp == 1) {
    // ---- products ----
    if (lane == 0) {
      Ring rq, rk, rs;
      const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = umma_desc_sw128(smem_u32(sK), 16, 1024);
      bool ok = true, fresh = true;
      int qslot = 0, kslot = 0, slot0 = 0, slot1 = 0;
      for (Walk<PASS> w(p, *start); w.more(); w.next()) {
        const bool keeps = w.keeps();
        const bool load_q = PASS == 1 ? fresh : !(keeps && (w.loaded >> w.rt & 1));
        if (PASS == 1 || fresh) {
          ok = mbar_wait_bounded(&k_full[rk.slot], rk.phase, abort_flag);
          kslot = rk.slot;
          rk.next(kKSlots);
        }
        if (ok && load_q) {
          ok = mbar_wait_bounded(&q_full[rq.slot], rq.phase, abort_flag);
          qslot = rq.slot;
          rq.next(kQSlots);
          if (keeps) {
            w.loaded |= 1 << w.rt;
            if (w.rt == 0) slot0 = qslot;
            else slot1 = qslot;
          }
        } else if (keeps) {
          qslot = w.rt == 0 ? slot0 : slot1;
        }
        if (ok) ok = mbar_wait_bounded(&s_empty[rs.slot], rs.phase ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t a = dq + (uint64_t)((qslot * L::kTileBytes) >> 4);
        const uint64_t b = dk + (uint64_t)((kslot * L::kTileBytes) >> 4);
        // (second pass: no more columns than the row tile has rows, to 16)
        const uint32_t idesc = PASS == 1
                                   ? umma_idesc_bf16(kTile, kTile, false, false)
                                   : umma_idesc_bf16(kTile, (w.tile_rows() + 15) & ~15, false, false);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk / 4) * kTile * 128 + (kk & 3) * 32) >> 4);
          umma_bf16(tmem + rs.slot * kTile, PASS == 1 ? a + off : b + off,
                    PASS == 1 ? b + off : a + off, idesc, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[rs.slot]);
        rs.next(kBufs);
        fresh = w.last_here();
        if (PASS == 1 || fresh) umma_commit(&k_empty[kslot]);
        if (PASS == 1 ? fresh : !keeps) umma_commit(&q_empty[qslot]);
        if (keeps && w.head_done()) {
          if (w.loaded & 1) umma_commit(&q_empty[slot0]);
          if (w.loaded & 2) umma_commit(&q_empty[slot1]);
        }
      }
      // Wait for the products before tensor memory is freed.
      umma_commit(drain);
      if (!mbar_wait_bounded(drain, 0, nullptr)) flag_status(p.status, PKV_DEV_TIMEOUT);
    }
  } else if (warp < 4) {
    // ---- second pass: the rows' denominators, beside their Q tiles ----
    if (PASS == 2) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (threadIdx.x == 64) p.tickets[blockIdx.x] = 0;
      Ring r;
      for (Walk<PASS> w(p, *start); w.more(); w.next()) {
        const bool keeps = w.keeps();
        if (keeps && (w.loaded >> w.rt & 1)) continue;
        if (!warp_wait(&st_empty[r.slot], r.phase ^ 1, abort_flag)) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = (warp - 2) * 64 + x * 32 + lane;
          const int last = w.sees(row);
          stat[r.slot * kTile + row] = last >= 0 ? __ldcg(p.neg_lse + w.stat_at(row)) : 0.f;
          qpos[r.slot * kTile + row] = last;
        }
        mbar_arrive(&st_full[r.slot]);
        r.next(kQSlots);
        if (keeps) w.loaded |= 1 << w.rt;
      }
    }
  } else {
    // ---- exponentials and sums: two groups of four warps take the steps in turn ----
    const int quarter = warp & 3;
    const int side = (warp - 4) >> 2;     // the group
    const int row = quarter * 32 + lane;  // the thread's lane of tensor memory
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float qs = p.qscale;
    const float2 qs2 = make_float2(qs, qs);
    Ring rs, rst;
    bool ok = true;
    int parity = 0;  // of the exchange buffers
    int turn = 0;    // the group whose step it is
    float m = -INFINITY, l = 0.f;        // first pass: the row's maximum and sum, of this group's steps
    float2 acc = make_float2(0.f, 0.f);  // second pass: the key's sum, of this group's steps
    int sslot = 0, slot0 = 0, slot1 = 0;
    for (Walk<PASS> w(p, *start); w.more(); w.next()) {
      const bool mine_now = turn == side;
      turn ^= 1;
      const bool keeps = w.keeps();
      if (PASS == 2) {
        if (!(keeps && (w.loaded >> w.rt & 1))) {
          ok = warp_wait(&st_full[rst.slot], rst.phase, abort_flag);
          sslot = rst.slot;
          rst.next(kQSlots);
          if (keeps) {
            w.loaded |= 1 << w.rt;
            if (w.rt == 0) slot0 = sslot;
            else slot1 = sslot;
          }
        } else {
          sslot = w.rt == 0 ? slot0 : slot1;
        }
      }
      if (ok && mine_now) ok = warp_wait(&s_full[rs.slot], rs.phase, abort_flag);
      if (ok && mine_now) {
        tc_fence_after_sync();
        const uint32_t ta = tmem + lane_base + rs.slot * kTile;
        if (PASS == 1) {
          const int last = w.sees(row);
          if (__any_sync(0xffffffffu, last >= 0)) {
#pragma unroll 1
            for (int c0 = 0; c0 < kTile; c0 += 64) {
              float v[64];
              float top;
              tmem_load64_max(ta + c0, v, top);
              const int key0 = w.kt * kTile + c0;
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              float mn, ref;
              // Keys past the row's position are hidden; a negative scale makes
              // the smallest product the largest logit.
              if (qs < 0.f || !__all_sync(0xffffffffu, key0 + 63 <= last)) {
                top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                  v[i] = key0 + i <= last ? v[i] * qs : -INFINITY;
                  top = fmaxf(top, v[i]);
                }
                mn = fmaxf(m, top);
                ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                  sum[(i >> 1) & 1] = __fadd2_rn(
                      sum[(i >> 1) & 1], make_float2(fast_exp2(v[i] - ref), fast_exp2(v[i + 1] - ref)));
              } else {
                mn = fmaxf(m, top * qs);
                ref = mn == -INFINITY ? 0.f : mn;
                const float2 nref = make_float2(-ref, -ref);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                  const float2 z = __ffma2_rn(make_float2(v[i], v[i + 1]), qs2, nref);
                  sum[(i >> 1) & 1] =
                      __fadd2_rn(sum[(i >> 1) & 1], make_float2(fast_exp2(z.x), fast_exp2(z.y)));
                }
              }
              l = l * fast_exp2(m - ref) + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
              m = mn;
            }
          }
        } else {
          const int key = w.kt * kTile + row;
          const int rows = w.tile_rows();
          // Every row of the tile sees every key of the tile.
          const bool open = w.kt * kTile + kTile - 1 <= w.q.base + w.rt * w.tq;
#pragma unroll 1
          for (int c0 = 0; c0 < rows; c0 += 32) {
            float v[32];
            tmem_load32(ta + c0, v);
            const float4 *ns = reinterpret_cast<const float4 *>(stat + sslot * kTile + c0);
            if (open && c0 + 32 <= rows) {
              float2 more = make_float2(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 n = ns[i / 4];
                const float2 z0 = __ffma2_rn(make_float2(v[i], v[i + 1]), qs2, make_float2(n.x, n.y));
                const float2 z1 = __ffma2_rn(make_float2(v[i + 2], v[i + 3]), qs2, make_float2(n.z, n.w));
                acc = __fadd2_rn(acc, make_float2(fast_exp2(z0.x), fast_exp2(z0.y)));
                more = __fadd2_rn(more, make_float2(fast_exp2(z1.x), fast_exp2(z1.y)));
              }
              acc = __fadd2_rn(acc, more);
            } else {
              const int4 *qp = reinterpret_cast<const int4 *>(qpos + sslot * kTile + c0);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 n = ns[i / 4];
                const int4 last = qp[i / 4];
                acc.x += key <= last.x ? fast_exp2(fmaf(v[i], qs, n.x)) : 0.f;
                acc.y += key <= last.y ? fast_exp2(fmaf(v[i + 1], qs, n.y)) : 0.f;
                acc.x += key <= last.z ? fast_exp2(fmaf(v[i + 2], qs, n.z)) : 0.f;
                acc.y += key <= last.w ? fast_exp2(fmaf(v[i + 3], qs, n.w)) : 0.f;
              }
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[rs.slot]);
      }
      rs.next(kBufs);
      // (both groups release a row tile's denominators, each after its last use)
      if (PASS == 2 && ok) {
        __syncwarp();
        if (lane == 0) {
          if (!keeps) {
            mbar_arrive(&st_empty[sslot]);
          } else if (w.head_done()) {
            if (w.loaded & 1) mbar_arrive(&st_empty[slot0]);
            if (w.loaded & 2) mbar_arrive(&st_empty[slot1]);
          }
        }
      }
      if (ok && !w.last_here()) continue;

      // The tile ends here (or a wait ran out: then all eight warps meet and
      // leave).  The groups' sums are joined by the first group's threads.
      float *ex = red + parity * 2 * kTile;
      parity ^= 1;
      if (side == 1) {
        ex[row] = PASS == 1 ? m : acc.x + acc.y;
        if (PASS == 1) ex[kTile + row] = l;
      }
      if (epilogue_sync_any(!ok)) break;
      float2 mine = make_float2(0.f, 0.f);  // (maximum, sum), or (-, sum)
      auto join = [&](float2 x) {
        if (PASS == 1) {
          const float mn = fmaxf(mine.x, x.x);
          const float ref = mn == -INFINITY ? 0.f : mn;
          mine.y = mine.y * fast_exp2(mine.x - ref) + x.y * fast_exp2(x.x - ref);
          mine.x = mn;
        } else {
          mine.y += x.y;
        }
      };
      if (side == 0) {
        mine = PASS == 1 ? make_float2(m, l) : make_float2(0.f, acc.x + acc.y);
        join(PASS == 1 ? make_float2(ex[row], ex[kTile + row]) : make_float2(0.f, ex[row]));
      }
      m = -INFINITY;
      l = 0.f;
      acc = make_float2(0.f, 0.f);
      bool finish = true;
      if (w.cut_left || !w.tile_done()) {
        // A part of a tile that several CTAs share: filed by CTA, place 0 if
        // the tile began before it, place 1 if it begins here.
        int c0, c1;
        w.ctas(c0, c1);
        if (side == 0) {
          __stcg(p.parts + ((int64_t)blockIdx.x * 2 + (w.cut_left ? 0 : 1)) * kTile + row, mine);
          __threadfence();
        }
        if (epilogue_sync_any(false)) break;
        if (threadIdx.x == 128) {
          const unsigned int done = atomicAdd(&p.tickets[(PASS - 1) * kMaxCtas + c0], 1u);
          *last_flag = done == (unsigned int)(c1 - c0) ? 1 : 0;
          __threadfence();
        }
        if (epilogue_sync_any(false)) break;
        finish = *last_flag != 0;
        if (finish && side == 0) {
          mine = __ldcg(p.parts + ((int64_t)c0 * 2 + 1) * kTile + row);
          for (int c = c0 + 1; c <= c1; ++c) join(__ldcg(p.parts + (int64_t)c * 2 * kTile + row));
        }
      }
      if (!finish || side != 0) continue;
      if (PASS == 1) {
        if (w.sees(row) >= 0) p.neg_lse[w.stat_at(row)] = -(mine.x + log2f(mine.y));
      } else {
        const int key = w.kt * kTile + row;
        if (key < w.q.len_k) {
          const int blk = p.block_tables[(int64_t)w.s * p.max_blocks_per_seq + (key >> p.block_shift)];
          if (blk >= 0 && blk < p.num_blocks) {
            float *to = p.key_weights + ((((int64_t)blk * p.num_kv_heads + w.j) << p.block_shift) +
                                         (key & ((1 << p.block_shift) - 1)));
            if (key >= w.q.c) *to = mine.y;
            else atomicAdd(to, mine.y);
          }
        }
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(p.status, PKV_DEV_TIMEOUT);
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
    parts = 2 * kMaxCtas * sizeof(unsigned int);
    neg_lse = parts + (size_t)kMaxCtas * 2 * kTile * sizeof(float2);
    total = neg_lse + (size_t)(stat_rows * Hq) * sizeof(float);
  }
};

template <int D>
pkv_status launch(const CUtensorMap &tq, const CUtensorMap &tk, const PromptParams &prm,
                  int64_t most_steps, cudaStream_t stream) {
  const int smem = Layout<D>::total + 1024;
  const int sms = device_sm_count();
  int ctas = 0;
  if (sms <= 0 ||
      !kernel_smem_setup((const void *)prompt_weights_kernel<D, 1>, kThreads, smem, &ctas) ||
      !kernel_smem_setup((const void *)prompt_weights_kernel<D, 2>, kThreads, smem, &ctas))
    return PKV_ERR_CUDA;
  int64_t grid = sms < kMaxCtas ? sms : kMaxCtas;
  if (grid > most_steps) grid = most_steps;
  prompt_weights_kernel<D, 1><<<(unsigned)grid, kThreads, smem, stream>>>(tq, tk, prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
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
  if (cudaLaunchKernelEx(&cfg, prompt_weights_kernel<D, 2>, tq, tk, prm) != cudaSuccess)
    return PKV_ERR_CUDA;
  return launch_status();
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
  if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;  // NaN or infinite
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
  prm.qscale = scale * kLog2e;

  // q as {D, Hq, T}: a box is 64 dims x the G heads of a kv head x 128 / G
  // queries, in shared memory 128 rows with the heads of a query side by side.
  const uint64_t qdims[3] = {(uint64_t)head_dim, (uint64_t)num_q_heads, (uint64_t)total_q};
  const uint64_t qstr[2] = {(uint64_t)head_dim * 2, (uint64_t)num_q_heads * head_dim * 2};
  const uint32_t qbox[3] = {64u, (uint32_t)G, (uint32_t)(kTile / G)};
  // cache as {D, Hkv, block_size, NB}: a box is 64 dims x 1 head x 64 tokens x 1 block.
  const uint64_t kdims[4] = {(uint64_t)head_dim, (uint64_t)num_kv_heads, (uint64_t)block_size,
                             (uint64_t)num_blocks};
  const uint64_t kstr[3] = {(uint64_t)head_dim * 2, (uint64_t)num_kv_heads * head_dim * 2,
                            (uint64_t)block_size * num_kv_heads * head_dim * 2};
  const uint32_t kbox[4] = {64u, 1u, 64u, 1u};
  CUtensorMap tq, tk;
  if (!encode_bf16_map(&tq, q, 3, qdims, qstr, qbox, true) ||
      !encode_bf16_map(&tk, k_cache, 4, kdims, kstr, kbox, true))
    return PKV_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Steps that the batch can have at most (a small one needs fewer CTAs).
  const int64_t row_tiles = ((int64_t)plan.rows * G + kTile - 1) / kTile;
  const int64_t key_tiles = ((int64_t)max_blocks_per_seq * block_size + kTile - 1) / kTile;
  const double most = (double)num_seqs * num_kv_heads * row_tiles * key_tiles;
  const int64_t most_steps = most < kMaxCtas ? (int64_t)most : kMaxCtas;
  return head_dim == 128 ? launch<128>(tq, tk, prm, most_steps, st)
                         : launch<64>(tq, tk, prm, most_steps, st);
}
