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
//     thread owns a row (for half of a tile's keys) and keeps its running maximum
//     and sum over the unit's key tiles.  Long rows are split over several units.
//  2. Keys: S^T = K Q^T with the keys in the lanes, so that summing a key's
//     weights over the rows is a sum inside one thread.  One unit holds all row
//     tiles of its keys: no sum is shared between CTAs and no order varies.
// Both are the same persistent kernel: warp 0 loads tiles (TMA, 128-byte
// swizzle, through the block table), warp 1 issues tcgen05.mma into four
// 128-column buffers of tensor memory, warps 2 and 3 prepare the rows'
// denominators (second pass), warps 4-11 exponentiate and sum.  Loads, products
// and exponentials of different tiles overlap, across units too.
#include <math.h>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;       // rows and keys per tile
constexpr int kThreads = 384;
constexpr int kEpilogue = 256;   // threads of warps 4-11
constexpr int kBufs = 4;         // S buffers of 128 columns: all of tensor memory
constexpr int kQSlots = 2;
constexpr int kStatSlots = 3;    // row statistics (second pass)
constexpr int kMaxSplitTiles = 8;
constexpr int kUnitsWanted = 304;  // two units per SM, where the work allows
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Layout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kKSlots = D == 128 ? 4 : 6;
  static constexpr int q = 0;
  static constexpr int k = q + kQSlots * kTileBytes;
  static constexpr int bars = k + kKSlots * kTileBytes;
  // q_full/q_empty[Q], k_full/k_empty[K], s_full/s_empty[B], st_full/st_empty[T], drain
  static constexpr int kNumBars = 2 * kQSlots + 2 * kKSlots + 2 * kBufs + 2 * kStatSlots + 1;
  static constexpr int stat = (bars + kNumBars * 8 + 15) & ~15;  // [T][128] -log2 denominators
  static constexpr int qpos = stat + kStatSlots * kTile * 4;     // [T][128] last visible key, -1: no row
  static constexpr int red = qpos + kStatSlots * kTile * 4;      // [2][2][128] exchange between halves
  static constexpr int misc = red + 4 * kTile * 4;               // tensor memory address, abort flag
  static constexpr int total = misc + 16;
  // One CTA per SM (it takes all of tensor memory): more than half of an SM's
  // shared memory, so that a second one never waits for tensor memory.
  static_assert(total + 1024 <= 232448 && total > 114 * 1024, "shared memory");
};

struct PromptParams {
  float *key_weights;
  const int32_t *block_tables;
  const int32_t *cu_q;
  const int32_t *cu_k;
  float2 *part;  // [splits, stat rows, Hq]: (maximum in log2 units, sum) of a row over a split
  int32_t *status;
  int64_t num_blocks;
  int64_t total_q;
  int64_t stat_rows;
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
  int row_tiles;     // row tiles of a sequence, at most
  int splits;        // splits of a row's keys, at most
  int split_tiles;   // key tiles per split (first pass)
  int groups;        // groups of key tiles of a sequence, at most (second pass)
  int group_tiles;   // key tiles per group
  int64_t units;
  float qscale;
};

// One sequence of the call; false when it has no queries or its lengths do not
// fit (then flagged, if told to).
struct Seq {
  int q_begin, n, c, len_k, R;
};
__device__ __forceinline__ bool seq_at(const PromptParams &p, int s, Seq &q, bool tell) {
  q.q_begin = p.cu_q[s];
  q.n = p.cu_q[s + 1] - q.q_begin;
  q.len_k = p.cu_k[s + 1] - p.cu_k[s];
  q.c = q.len_k - q.n;
  q.R = min(q.n, p.window);
  if (q.n == 0) return false;
  if (q.n < 0 || q.n > p.max_seqlen_q || q.c < 0 || q.q_begin < 0 ||
      q.len_k > ((int64_t)p.max_blocks_per_seq << p.block_shift) ||
      (int64_t)q.q_begin + q.n > p.total_q) {
    if (tell) flag_status(p.status, PKV_DEV_BAD_SEQLEN);
    return false;
  }
  return true;
}

// A unit of work: row tiles [rt0, rt1) against key tiles [kt0, kt1) of kv head
// j of a sequence; of those, a key tile kt takes part with row tiles from
// first_rt(kt) on (the ones that see any of it).
struct Unit {
  Seq q;
  int s, j, rt0, rt1, kt0, kt1, tq;
  // Queries of a row tile, counted from the first that counts; the last one's position.
  __device__ __forceinline__ int last_pos(int rt) const {
    return q.c + q.n - q.R + min((rt + 1) * tq, q.R) - 1;
  }
  __device__ __forceinline__ int first_pos(int rt) const { return q.c + q.n - q.R + rt * tq; }
  __device__ __forceinline__ int first_rt(int kt) const {
    const int over = kt * kTile - (q.c + q.n - q.R);  // queries before this one see none of it
    return over <= 0 ? rt0 : max(rt0, over / tq);
  }
};

// Unit number -> unit; heads innermost, so that concurrent CTAs read the same tokens' rows.
template <int PASS>
__device__ __forceinline__ bool unit_at(const PromptParams &p, int64_t idx, Unit &u) {
  u.j = (int)(idx % p.num_kv_heads);
  idx /= p.num_kv_heads;
  u.tq = kTile >> p.group_shift;
  if (PASS == 1) {
    const int rt = (int)(idx % p.row_tiles);
    idx /= p.row_tiles;
    const int split = (int)(idx % p.splits);
    u.s = (int)(idx / p.splits);
    if (!seq_at(p, u.s, u.q, u.j == 0 && rt == 0 && split == 0)) return false;
    if (rt * u.tq >= u.q.R) return false;
    u.rt0 = rt;
    u.rt1 = rt + 1;
    u.kt0 = split * p.split_tiles;
    u.kt1 = min(u.kt0 + p.split_tiles, u.last_pos(rt) / kTile + 1);
  } else {
    const int g = (int)(idx % p.groups);
    u.s = (int)(idx / p.groups);
    if (!seq_at(p, u.s, u.q, false)) return false;
    u.rt0 = 0;
    u.rt1 = (u.q.R + u.tq - 1) / u.tq;
    u.kt0 = g * p.group_tiles;
    u.kt1 = min(u.kt0 + p.group_tiles, (u.q.len_k + kTile - 1) / kTile);
  }
  return u.kt0 < u.kt1;
}

// The statistics' row of the r-th counted query.
__device__ __forceinline__ int64_t stat_row(const PromptParams &p, const Unit &u, int r) {
  return p.by_query ? (int64_t)u.q.q_begin + u.q.n - u.q.R + r : (int64_t)u.s * p.rows + r;
}

// Product columns of a row tile in the second pass: its rows, to a multiple of 16.
__device__ __forceinline__ int tile_rows(const PromptParams &p, const Unit &u, int rt) {
  return min(u.tq, u.q.R - rt * u.tq) << p.group_shift;
}

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
  uint64_t *k_full = q_empty + kQSlots;
  uint64_t *k_empty = k_full + kKSlots;
  uint64_t *s_full = k_empty + kKSlots;
  uint64_t *s_empty = s_full + kBufs;
  uint64_t *st_full = s_empty + kBufs;
  uint64_t *st_empty = st_full + kStatSlots;
  uint64_t *drain = st_empty + kStatSlots;
  float *stat = reinterpret_cast<float *>(smem + L::stat);
  int *qpos = reinterpret_cast<int *>(smem + L::qpos);
  float *red = reinterpret_cast<float *>(smem + L::red);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kEpilogue / 32);
    }
    for (int i = 0; i < kStatSlots; ++i) {
      mbar_init(&st_full[i], 64);
      mbar_init(&st_empty[i], kEpilogue / 32);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kBufs * kTile);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // The second pass may be scheduled as SMs become free; it waits for this
  // grid's end where it reads the statistics.
  if (PASS == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Every role walks the same units, and in them the same steps: key tile by
  // key tile, its row tiles.  Q stays while the row tile does, K while the key
  // tile does.
  if (warp == 0) {
    // ---- loads ----
    if (lane == 0) {
      tma_prefetch_map(&tm_q);
      tma_prefetch_map(&tm_k);
      Ring rq, rk;
      int q_loads = 0, k_loads = 0;
      bool ok = true;
      Unit u;
      for (int64_t idx = blockIdx.x; idx < p.units && ok; idx += gridDim.x) {
        if (!unit_at<PASS>(p, idx, u)) continue;
        const int64_t bt = (int64_t)u.s * p.max_blocks_per_seq;
        int held = -1;  // row tile in the current Q slot
        for (int kt = u.kt0; kt < u.kt1 && ok; ++kt) {
          ok = mbar_wait_bounded(&k_empty[rk.slot], rk.phase ^ 1, abort_flag);
          if (!ok) break;
          uint8_t *kd = sK + rk.slot * L::kTileBytes;
          mbar_arrive_expect_tx(&k_full[rk.slot], L::kTileBytes);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // (a tile's second half may lie past the keys: it reads the first half's block, unused)
            int pos = kt * kTile + half * 64;
            if (pos >= u.q.len_k) pos = kt * kTile;
            int blk = p.block_tables[bt + (pos >> p.block_shift)];
            if (blk < 0 || blk >= p.num_blocks) {
              flag_status(p.status, PKV_DEV_BAD_BLOCK);
              blk = 0;
            }
#pragma unroll
            for (int x = 0; x < XR; ++x)
              tma_load_4d(kd + x * kTile * 128 + half * 64 * 128, &tm_k, &k_full[rk.slot], x * 64,
                          u.j, pos & ((1 << p.block_shift) - 1), blk);
          }
          ++k_loads;
          rk.next(kKSlots);
          for (int rt = PASS == 1 ? u.rt0 : u.first_rt(kt); rt < u.rt1 && ok; ++rt) {
            if (rt == held) continue;
            held = rt;
            ok = mbar_wait_bounded(&q_empty[rq.slot], rq.phase ^ 1, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(&q_full[rq.slot], L::kTileBytes);
#pragma unroll
            for (int x = 0; x < XR; ++x)
              tma_load_3d(sQ + rq.slot * L::kTileBytes + x * kTile * 128, &tm_q, &q_full[rq.slot],
                          x * 64, u.j << p.group_shift,
                          u.q.q_begin + u.q.n - u.q.R + rt * u.tq);
            ++q_loads;
            rq.next(kQSlots);
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
  } else if (warp == 1) {
    // ---- products ----
    if (lane == 0) {
      Ring rq, rk, rs;
      const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = umma_desc_sw128(smem_u32(sK), 16, 1024);
      bool ok = true;
      Unit u;
      for (int64_t idx = blockIdx.x; idx < p.units && ok; idx += gridDim.x) {
        if (!unit_at<PASS>(p, idx, u)) continue;
        int held = -1;
        for (int kt = u.kt0; kt < u.kt1 && ok; ++kt) {
          ok = mbar_wait_bounded(&k_full[rk.slot], rk.phase, abort_flag);
          const int rt0 = PASS == 1 ? u.rt0 : u.first_rt(kt);
          for (int rt = rt0; rt < u.rt1 && ok; ++rt) {
            if (rt != held) {
              ok = mbar_wait_bounded(&q_full[rq.slot], rq.phase, abort_flag);
              held = rt;
            }
            if (ok) ok = mbar_wait_bounded(&s_empty[rs.slot], rs.phase ^ 1, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t a = dq + (uint64_t)((rq.slot * L::kTileBytes) >> 4);
            const uint64_t b = dk + (uint64_t)((rk.slot * L::kTileBytes) >> 4);
            const uint32_t idesc =
                PASS == 1 ? umma_idesc_bf16(kTile, kTile, false, false)
                          : umma_idesc_bf16(kTile, (tile_rows(p, u, rt) + 15) & ~15, false, false);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk / 4) * kTile * 128 + (kk & 3) * 32) >> 4);
              umma_bf16(tmem + rs.slot * kTile, PASS == 1 ? a + off : b + off,
                        PASS == 1 ? b + off : a + off, idesc, kk > 0 ? 1u : 0u);
            }
            umma_commit(&s_full[rs.slot]);
            rs.next(kBufs);
            // Q is done with when the next step of the unit has another row
            // tile, or there is none.
            const bool next_same = kt + 1 < u.kt1 && rt + 1 == u.rt1 &&
                                   (PASS == 1 ? u.rt0 : u.first_rt(kt + 1)) == rt;
            if (!next_same) {
              umma_commit(&q_empty[rq.slot]);
              rq.next(kQSlots);
              held = -1;
            }
          }
          if (ok) umma_commit(&k_empty[rk.slot]);
          rk.next(kKSlots);
        }
      }
      // Wait for the products before tensor memory is freed.
      umma_commit(drain);
      if (!mbar_wait_bounded(drain, 0, nullptr)) flag_status(p.status, PKV_DEV_TIMEOUT);
    }
  } else if (warp < 4) {
    // ---- second pass: the rows' denominators, one slot per Q load ----
    if (PASS == 2) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      Ring rt_ring;
      bool ok = true;
      Unit u;
      for (int64_t idx = blockIdx.x; idx < p.units && ok; idx += gridDim.x) {
        if (!unit_at<PASS>(p, idx, u)) continue;
        int held = -1;
        for (int kt = u.kt0; kt < u.kt1 && ok; ++kt) {
          for (int rt = u.first_rt(kt); rt < u.rt1; ++rt) {
            if (rt == held) continue;
            held = rt;
            ok = warp_wait(&st_empty[rt_ring.slot], rt_ring.phase ^ 1, abort_flag);
            if (!ok) break;
            const int splits = u.last_pos(rt) / (kTile * p.split_tiles) + 1;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int row = (warp - 2) * 64 + x * 32 + lane;
              const int r = rt * u.tq + (row >> p.group_shift);
              float neg = 0.f;
              int pos = -1;
              if (r < u.q.R) {
                pos = u.q.c + u.q.n - u.q.R + r;
                const float2 *part = p.part + stat_row(p, u, r) * p.num_q_heads +
                                     (u.j << p.group_shift) + (row & (p.group - 1));
                float m = -INFINITY, l = 0.f;
                for (int i = 0; i < splits; ++i) {
                  const float2 ml = __ldcg(part + (int64_t)i * p.stat_rows * p.num_q_heads);
                  const float mn = fmaxf(m, ml.x);
                  const float ref = mn == -INFINITY ? 0.f : mn;
                  l = l * exp2f(m - ref) + ml.y * exp2f(ml.x - ref);
                  m = mn;
                }
                neg = -(m + log2f(l));
              }
              stat[rt_ring.slot * kTile + row] = neg;
              qpos[rt_ring.slot * kTile + row] = pos;
            }
            mbar_arrive(&st_full[rt_ring.slot]);
            rt_ring.next(kStatSlots);
          }
        }
      }
    }
  } else {
    // ---- exponentials and sums: two warps per lane quarter, which share the columns ----
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float qs = p.qscale;
    Ring rs, rst;
    bool ok = true;
    int parity = 0;  // of the exchange buffers
    Unit u;
    for (int64_t idx = blockIdx.x; idx < p.units && ok; idx += gridDim.x) {
      if (!unit_at<PASS>(p, idx, u)) continue;
      if (PASS == 1) {
        const int r = u.rt0 * u.tq + (row >> p.group_shift);
        const int pos = r < u.q.R ? u.q.c + u.q.n - u.q.R + r : -1;  // last visible key
        const bool any = __any_sync(0xffffffffu, pos >= 0);
        float m = -INFINITY, l = 0.f;
        for (int kt = u.kt0; kt < u.kt1; ++kt) {
          ok = warp_wait(&s_full[rs.slot], rs.phase, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
          if (any) {
            float v[64];
            float top;
            tmem_load64_max(tmem + lane_base + rs.slot * kTile + half * 64, v, top);
            const int key0 = kt * kTile + half * 64;
            // Keys past the row's position are hidden; a negative scale makes
            // the smallest product the largest logit.
            if (qs < 0.f || !__all_sync(0xffffffffu, key0 + 63 <= pos)) {
              top = -INFINITY;
#pragma unroll
              for (int i = 0; i < 64; ++i) {
                v[i] = key0 + i <= pos ? v[i] * qs : -INFINITY;
                top = fmaxf(top, v[i]);
              }
              const float mn = fmaxf(m, top);
              const float ref = mn == -INFINITY ? 0.f : mn;
              float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < 64; ++i) sum[i & 3] += fast_exp2(v[i] - ref);
              l = l * fast_exp2(m - ref) + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
              m = mn;
            } else {
              const float mn = fmaxf(m, top * qs);
              const float ref = mn == -INFINITY ? 0.f : mn;
              float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < 64; ++i) sum[i & 3] += fast_exp2(fmaf(v[i], qs, -ref));
              l = l * fast_exp2(m - ref) + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
              m = mn;
            }
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[rs.slot]);
          rs.next(kBufs);
        }
        // The two halves of a row's keys, joined by the first half's thread.
        float *ex = red + parity * 2 * kTile;
        if (half == 1) {
          ex[row] = m;
          ex[kTile + row] = l;
        }
        if (epilogue_sync_any(!ok)) break;
        if (half == 0 && pos >= 0) {
          const float m2 = ex[row], l2 = ex[kTile + row];
          const float mn = fmaxf(m, m2);
          const float ref = mn == -INFINITY ? 0.f : mn;
          l = l * fast_exp2(m - ref) + l2 * fast_exp2(m2 - ref);
          p.part[((int64_t)(u.kt0 / p.split_tiles) * p.stat_rows + stat_row(p, u, r)) *
                     p.num_q_heads +
                 (u.j << p.group_shift) + (row & (p.group - 1))] = make_float2(mn, l);
        }
        parity ^= 1;
      } else {
        int held = -1;
        for (int kt = u.kt0; kt < u.kt1 && ok; ++kt) {
          const int key = kt * kTile + row;
          float2 acc = make_float2(0.f, 0.f);
          for (int rt = u.first_rt(kt); rt < u.rt1; ++rt) {
            if (rt != held) {
              ok = warp_wait(&st_full[rst.slot], rst.phase, abort_flag);
              held = rt;
            }
            if (ok) ok = warp_wait(&s_full[rs.slot], rs.phase, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
            const int rows = tile_rows(p, u, rt);
            const bool open = kt * kTile + kTile - 1 <= u.first_pos(rt);  // every row sees the tile
            for (int c0 = half * 32; c0 < rows; c0 += 64) {
              float v[32];
              tmem_load32(tmem + lane_base + rs.slot * kTile + c0, v);
              const float4 *ns = reinterpret_cast<const float4 *>(stat + rst.slot * kTile + c0);
              if (open && c0 + 32 <= rows) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float4 n = ns[i / 4];
                  acc.x += fast_exp2(fmaf(v[i], qs, n.x));
                  acc.y += fast_exp2(fmaf(v[i + 1], qs, n.y));
                  acc.x += fast_exp2(fmaf(v[i + 2], qs, n.z));
                  acc.y += fast_exp2(fmaf(v[i + 3], qs, n.w));
                }
              } else {
                const int4 *qp = reinterpret_cast<const int4 *>(qpos + rst.slot * kTile + c0);
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
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[rs.slot]);
            rs.next(kBufs);
            const bool next_same = kt + 1 < u.kt1 && rt + 1 == u.rt1 && u.first_rt(kt + 1) == rt;
            if (!next_same) {
              if (lane == 0) mbar_arrive(&st_empty[rst.slot]);
              rst.next(kStatSlots);
              held = -1;
            }
          }
          float *ex = red + parity * kTile;
          if (half == 1) ex[row] = acc.x + acc.y;
          ok = !epilogue_sync_any(!ok);
          if (half == 0 && ok && key < u.q.len_k) {
            const float a = (acc.x + acc.y) + ex[row];
            const int blk = p.block_tables[(int64_t)u.s * p.max_blocks_per_seq + (key >> p.block_shift)];
            if (blk >= 0 && blk < p.num_blocks) {
              float *w = p.key_weights + ((((int64_t)blk * p.num_kv_heads + u.j) << p.block_shift) +
                                          (key & ((1 << p.block_shift) - 1)));
              if (key >= u.q.c) *w = a;
              else atomicAdd(w, a);
            }
          }
          parity ^= 1;
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

// How a call is cut into units (host), from its arguments alone.
struct Plan {
  int64_t rows, row_tiles, key_tiles, stat_rows, splits, split_tiles, groups, group_tiles;
  bool by_query, fits;
  Plan(int64_t num_seqs, int64_t total_q, int64_t max_seqlen_q, int64_t window, int64_t group,
       int64_t num_kv_heads, int64_t max_tokens) {
    rows = window < max_seqlen_q ? window : max_seqlen_q;
    const int64_t tq = kTile / group;
    row_tiles = (rows + tq - 1) / tq;
    key_tiles = (max_tokens + kTile - 1) / kTile;
    by_query = num_seqs * rows > total_q;
    stat_rows = by_query ? total_q : num_seqs * rows;
    // First pass: a row's keys in splits of up to 8 tiles (1024 keys), fewer
    // while there are not two units for every SM.
    split_tiles = kMaxSplitTiles;
    const double heads = (double)num_seqs * num_kv_heads;  // (a product of arguments may pass 64 bits)
    while (split_tiles > 1 &&
           heads * row_tiles * ((key_tiles + split_tiles - 1) / split_tiles) < kUnitsWanted)
      split_tiles /= 2;
    splits = (key_tiles + split_tiles - 1) / split_tiles;
    // Second pass: key tiles in groups of about 8 steps.
    group_tiles = kMaxSplitTiles / row_tiles;
    if (group_tiles < 1) group_tiles = 1;
    while (group_tiles > 1 && heads * ((key_tiles + group_tiles - 1) / group_tiles) < kUnitsWanted)
      group_tiles /= 2;
    groups = (key_tiles + group_tiles - 1) / group_tiles;
    fits = heads * row_tiles * splits < 4e18 && heads * groups < 4e18;
  }
};

template <int D>
pkv_status launch(const CUtensorMap &tq, const CUtensorMap &tk, PromptParams prm, const Plan &plan,
                  cudaStream_t stream) {
  const int smem = Layout<D>::total + 1024;
  const int sms = device_sm_count();
  int ctas = 0;
  if (sms <= 0 ||
      !kernel_smem_setup((const void *)prompt_weights_kernel<D, 1>, kThreads, smem, &ctas) ||
      !kernel_smem_setup((const void *)prompt_weights_kernel<D, 2>, kThreads, smem, &ctas))
    return PKV_ERR_CUDA;
  prm.units = (int64_t)prm.num_seqs * plan.splits * plan.row_tiles * prm.num_kv_heads;
  int64_t grid = prm.units < sms ? prm.units : sms;
  prompt_weights_kernel<D, 1><<<(unsigned)grid, kThreads, smem, stream>>>(tq, tk, prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  prm.units = (int64_t)prm.num_seqs * plan.groups * prm.num_kv_heads;
  grid = prm.units < sms ? prm.units : sms;
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
  if (group < 1 || group > kTile || num_q_heads > (1 << 16) || total_q > 0x7FFFFFFFLL ||
      (int64_t)max_blocks_per_seq * block_size > 0x7FFFFFFFLL)
    return 0;
  const Plan plan(num_seqs, total_q, max_seqlen_q, window, group, num_kv_heads,
                  (int64_t)max_blocks_per_seq * block_size);
  if (plan.splits * num_q_heads > (INT64_MAX / 16) / plan.stat_rows) return 0;
  return 256 + (size_t)(plan.splits * num_q_heads * plan.stat_rows) * sizeof(float2);
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
  const Plan plan(num_seqs, total_q, max_seqlen_q, window, G, num_kv_heads,
                  (int64_t)max_blocks_per_seq * block_size);
  if (!plan.fits) return PKV_ERR_UNSUPPORTED;  // more units than 64 bits number
  PromptParams prm;
  prm.key_weights = key_weights;
  prm.block_tables = block_tables;
  prm.cu_q = cu_seqlens_q;
  prm.cu_k = cu_seqlens_k;
  prm.part = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + 256);
  prm.status = dev_status;
  prm.num_blocks = num_blocks;
  prm.total_q = total_q;
  prm.stat_rows = plan.stat_rows;
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
  prm.row_tiles = (int)plan.row_tiles;
  prm.splits = (int)plan.splits;
  prm.split_tiles = (int)plan.split_tiles;
  prm.groups = (int)plan.groups;
  prm.group_tiles = (int)plan.group_tiles;
  prm.units = 0;
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
  return head_dim == 128 ? launch<128>(tq, tk, prm, plan, st) : launch<64>(tq, tk, prm, plan, st);
}
