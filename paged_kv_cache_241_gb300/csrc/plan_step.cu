// plan_step.cu -- a step's blocks, slots and positions from the sequences' lengths.
//
// What the host block manager does for one sequence at a time (a new block when the
// length reaches a multiple of the block size plus one: CSDN essay "from nanoVLLM to
// vLLM", Mountain 1), done for a batch on the device, so that a captured step can go
// on without the host.  With L[s] tokens held, n[s] new ones, BS tokens to a block:
//   have = ceil(L / BS), need = ceil((L + n) / BS) - have  (n > 0),
//   give = have - borrowed  (n = -1: the sequence ends)
// and the exclusive prefix sums of need, give and n over the sequences say where in
// the stack of free blocks a sequence's blocks go to or come from, and which rows of
// the step are its own.
//
// A small step is one CTA's.  For a larger one a launch over the whole GPU writes the rows,
// and a cluster of eight the tables, the stack and the lengths; every CTA scans the lengths
// by itself (12 bytes a sequence).  A block that is given back and taken again in the same
// step is looked up in the table that it comes from, not on the stack, so nothing that is
// read is written in the same step but lengths and counters (in place): those last, once
// everybody has read.  So the second launch scans beside the first, and waits for it only
// before it writes the lengths.
//
// Bound by latency: a step of 64 sequences reads and writes 2 KB, and takes one load of
// the lengths, one of blocks from the stack or a table, and the barriers between them: 4.1
// us in a graph of calls (two sequences 2.9, 500 prompts with 2 MB of rows and tables 6.9).
#include "cta_scan.cuh"
#include "host_common.h"
#include "pkv_common.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kPlanMaxSeqs = 16384;
constexpr int kPlanCluster = 8;     // portable cluster size
// Up to so many rows and sequences one CTA of as many threads as sequences does the step, a
// thread four rows at most (decode: 256 rows 5.2 us, in two launches 5.6; eight prompts with
// 1000 rows 4.7 and 5.0, with 1500 5.8 and 5.0; 500 sequences by one CTA of 512 threads 6.2,
// in two launches 5.8).  A single launch of the cluster alone did 1000 rows in 8.3 us and
// 16 thousand in 8.5 (two launches: 6.8 and 5.3).
constexpr int kPlanSmallRows = 1024;
constexpr int kPlanSmallSeqs = 256;
// Threads of a CTA of a larger step: two CTAs of 512 have an SM's registers, so that the
// launches overlap (1000 rows 6.8 us, 7.9 with 1024 threads), but many sequences are scanned
// faster by 1024 (4000 of them: 15.3 and 13.8).
constexpr int kPlanThreads = 512, kPlanManyThreads = 1024, kPlanManySeqs = 2048;

enum { kAll, kRows, kState };  // what a launch does: all of it, or in two launches a part each

struct PlanParams {
  const int32_t *new_lens;
  const int32_t *context_lens;
  const int32_t *borrowed;   // may be null
  int32_t *block_tables;
  int32_t *free_blocks;
  const int32_t *num_free;
  int32_t *new_context_lens;
  int32_t *new_num_free;
  int32_t *slots;
  int32_t *positions;
  int32_t *cu_q;
  int32_t *cu_k;
  int32_t *status;
  int64_t num_rows;
  int64_t num_blocks;
  int capacity;      // of free_blocks
  int num_seqs;
  int max_blocks_per_seq;
  int block_shift;
  int rows_16b;      // slots and positions are 16-byte aligned
};

__device__ __forceinline__ int saturated(int64_t x) {
  return x > 0x7FFFFFFF ? 0x7FFFFFFF : (int)x;
}

// A value of the lengths, tables or stack.  The launch beside the rows' reads them without a
// wait of its own (they are in memory: every CTA of the rows' launch has waited for what wrote
// them): past the SM's L1, which may hold them as they were before.
template <int kPart>
__device__ __forceinline__ int load(const int32_t *x) {
  return kPart == kState ? __ldcg(x) : *x;
}

// A sequence's lengths, checked.
struct PlanSeq {
  int L;       // tokens held (0 if the length given does not fit the table)
  int n;       // rows of the step (0: none)
  int have, need, give, borrowed;
  bool ends, out;  // out: its lengths do not fit, it takes no part but for its rows
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanParams &p, int L, int n, int borrowed, bool tell) {
  PlanSeq q;
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  int bad = 0;
  q.out = L < 0 || L > room;
  q.L = q.out ? 0 : L;
  q.n = n > 0 ? n : 0;
  q.ends = n == -1 && !q.out;
  if (n < -1) bad |= PKV_DEV_BAD_SEQLEN;
  if (q.L + (int64_t)q.n > room) q.out = true;
  if (q.out) bad |= PKV_DEV_BAD_CONTEXT;
  const int bs1 = (1 << p.block_shift) - 1;
  q.have = (int)(((int64_t)q.L + bs1) >> p.block_shift);
  if (borrowed < 0 || borrowed > q.have) {
    bad |= PKV_DEV_BAD_CONTEXT;
    borrowed = borrowed < 0 ? 0 : q.have;
  }
  q.borrowed = borrowed;
  q.give = q.ends ? q.have - borrowed : 0;
  q.need = q.out || q.n == 0 ? 0 : (int)(((int64_t)q.L + q.n + bs1) >> p.block_shift) - q.have;
  if (tell && bad) flag_status(p.status, bad);
  return q;
}

// `each(lane, i)` for the items i < count of every lane, spread over the warp's lanes.
template <typename F>
__device__ __forceinline__ void for_items(int count, F each) {
  const int lane = threadIdx.x & 31;
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  for (int i0 = 0; i0 < total; i0 += 32) {
    const int i = i0 + lane;
    int owner = 0;  // lanes whose items all come before i
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const int last = __shfl_sync(0xffffffffu, incl, owner + o - 1);
      if (last <= i) owner += o;
    }
    const int before = __shfl_sync(0xffffffffu, incl - count, owner & 31);
    each(owner & 31, i - before, i < total);
  }
}

// Slots and positions of the rows t0 .. t0 + kEach - 1.  first_row [S + 1]: the rows of
// sequence s begin there; held[s]: tokens before them, or -1 - those when it gets no
// slots; block_of(s, tokens before, block of the table): where its id is.
template <int kEach, typename F>
__device__ __forceinline__ void write_rows(const PlanParams &p, const int *first_row, const int *held,
                                           int64_t t0, F block_of) {
  const int shift = p.block_shift, S = p.num_seqs, rows = first_row[S];
  int pos[kEach], blk[kEach];
  bool real[kEach];
  int s = -1;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t t = t0 + i;
    pos[i] = 0;
    blk[i] = -1;
    real[i] = false;
    if (t >= rows || t >= p.num_rows) continue;
    if (s < 0) s = seq_of(first_row, S, (int)t);
    else while (first_row[s + 1] <= t) ++s;
    const int h = held[s], L = h < 0 ? -1 - h : h;
    pos[i] = (int)((uint32_t)L + (uint32_t)(t - first_row[s]));
    real[i] = h >= 0;
    if (h >= 0) blk[i] = block_of(s, L, pos[i] >> shift);
  }
  int slot[kEach];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool in = blk[i] >= 0 && blk[i] < p.num_blocks;
    bad = bad || (real[i] && !in);
    slot[i] = in ? (blk[i] << shift) + (pos[i] & ((1 << shift) - 1)) : -1;
  }
  if (bad) flag_status(p.status, PKV_DEV_BAD_BLOCK);
  if (kEach == 4 && p.rows_16b && t0 + kEach <= p.num_rows) {
    *reinterpret_cast<int4 *>(p.slots + t0) = make_int4(slot[0], slot[1 % kEach], slot[2 % kEach], slot[3 % kEach]);
    *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1 % kEach], pos[2 % kEach], pos[3 % kEach]);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (t0 + i < p.num_rows) {
        p.slots[t0 + i] = slot[i];
        p.positions[t0 + i] = pos[i];
      }
    }
  }
}

template <int kPart>
__global__ void __launch_bounds__(kPlanManyThreads) plan_step_kernel(const PlanParams p) {
  extern __shared__ int plan_smem[];
  __shared__ int64_t sums3[32][3];
  __shared__ int64_t sums1[32][1];
  const int S = p.num_seqs, shift = p.block_shift, bs1 = (1 << shift) - 1;
  int *first_row = plan_smem;           // [S + 1]
  int *held = first_row + S + 1;        // [S]: L, or -1 - L when the sequence gets no slots;
                                        // when it ends the first block that it gives
  int *base = held + S;                 // [S]: blocks needed before it; -1 - blocks given
                                        // before it when it ends
  uint16_t *ending = reinterpret_cast<uint16_t *>(base + S);  // [those that end]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int rank = (int)blockIdx.x, ctas = (int)gridDim.x;  // (the rows' grid, else one cluster)
  const bool tells = kPart != kRows && rank == 0;

  // (The launch behind the rows' began after all of that one's CTAs had waited for what came
  // before them both.)
  if (kPart != kState) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  const int free_given = load<kPart>(p.num_free);
  const int per = (S + blockDim.x - 1) / (int)blockDim.x;
  const int s0 = min(tid * per, S), s1 = min(s0 + per, S);
  // Blocks given (2^38 at most) and, above them, sequences that end; need; rows.
  constexpr int kEnds = 44;
  constexpr int64_t kGive = ((int64_t)1 << kEnds) - 1;
  int64_t at[3] = {0, 0, 0}, total[3];
  PlanSeq mine = {};                    // (the thread's last: its only one, mostly)
  auto lengths_of = [&](int s, bool tell) {
    const int L = load<kPart>(p.context_lens + s), n = load<kPart>(p.new_lens + s);
    return plan_seq(p, L, n, p.borrowed != nullptr ? load<kPart>(p.borrowed + s) : 0, tell);
  };
  for (int s = s0; s < s1; ++s) {
    if (kPart == kState && per > 1) {  // (the thread's second look, too: 1000 rows 7.1 -> 6.9 us)
      held[s] = load<kPart>(p.context_lens + s);
      first_row[s] = load<kPart>(p.new_lens + s);
      base[s] = p.borrowed != nullptr ? load<kPart>(p.borrowed + s) : 0;
      mine = plan_seq(p, held[s], first_row[s], base[s], tells);
    } else {
      mine = lengths_of(s, tells);
    }
    at[0] += mine.give + ((int64_t)mine.ends << kEnds);
    at[1] += mine.need;
    at[2] += mine.n;
  }
  const int free0 = min(max(free_given, 0), p.capacity);
  if (free0 != free_given && tells && tid == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
  scan_cta<3>(at, total, sums3);
  const int64_t given = total[0] & kGive;
  const int ends = (int)(total[0] >> kEnds);
  const int left = (int)min((int64_t)free0 + given, (int64_t)p.capacity);
  if (free0 + given > p.capacity && tells && tid == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
  int64_t keys[1] = {0}, all_keys[1], taken = 0;
  {
    int64_t give = at[0], need = at[1], row = at[2];
    for (int s = s0; s < s1; ++s) {
      const PlanSeq q = per == 1          ? mine
                        : kPart == kState ? plan_seq(p, held[s], first_row[s], base[s], false)
                                          : lengths_of(s, false);
      const bool no_blocks = q.need > 0 && need + q.need > left;
      const bool no_rows = q.n > 0 && row + q.n > p.num_rows;
      if (tells && (no_blocks || no_rows))
        flag_status(p.status, (no_blocks ? PKV_DEV_NO_BLOCKS : 0) | (no_rows ? PKV_DEV_BAD_SEQLEN : 0));
      const bool refused = no_blocks || no_rows || q.out;
      first_row[s] = saturated(row);
      held[s] = q.ends ? q.borrowed : refused ? -1 - q.L : q.L;
      base[s] = q.ends ? -1 - saturated(min(give & kGive, (int64_t)p.capacity)) : saturated(need);
      if (q.ends) ending[give >> kEnds] = (uint16_t)s;
      if (!refused && q.need > 0) taken = need + q.need;
      if (!refused && !q.ends) keys[0] += q.L + q.n;
      give += q.give + ((int64_t)q.ends << kEnds);
      need += q.need;
      row += q.n;
    }
  }
  if (tid == 0) first_row[S] = saturated(total[2]);
  if (kPart == kRows) {
    __syncthreads();
  } else {
    // Blocks taken: those up to the last sequence that takes any.
    int64_t most = taken;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const int64_t y = __shfl_xor_sync(0xffffffffu, most, o);
      most = y > most ? y : most;
    }
    if (lane == 0) sums3[warp][0] = most;
    scan_cta<1>(keys, all_keys, sums1);  // (its barriers also publish the arrays)
  }
  // (nobody reads lengths or counters any more)
  if (ctas > 1 && kPart != kRows) asm volatile("barrier.cluster.arrive.release;" ::: "memory");

  // The e-th of the sequences that end gives its blocks from held[s] on as numbers
  // given_before(e), ... of those that come back.
  auto given_before = [&](int e) { return -1 - base[ending[e]]; };
  // Block number b of the blocks needed, from the top of the stack.
  auto block_at = [&](int64_t b) -> int {
    const int64_t i = (int64_t)left - 1 - b;
    if (i < free0) return i >= 0 ? load<kPart>(p.free_blocks + i) : -1;
    const int k = (int)(i - free0);
    int lo = 0, hi = ends;  // the last one with given_before <= k
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (given_before(mid) <= k) lo = mid;
      else hi = mid;
    }
    const int s = ending[lo];
    return load<kPart>(p.block_tables + (int64_t)s * p.max_blocks_per_seq + held[s] + k - given_before(lo));
  };
  // Rows: one a thread where that is enough of them.
  const int64_t threads = (int64_t)ctas * blockDim.x, me = (int64_t)rank * blockDim.x + tid;
  if (kPart != kState) {
    auto block_of = [&](int s, int L, int b) {
      const int have = (L + bs1) >> shift;
      return b < have ? load<kPart>(p.block_tables + (int64_t)s * p.max_blocks_per_seq + b)
                      : block_at((int64_t)base[s] + b - have);
    };
    if (p.num_rows <= threads) {
      if (me < p.num_rows) write_rows<1>(p, first_row, held, me, block_of);
    } else {
      for (int64_t t0 = me * 4; t0 < p.num_rows; t0 += threads * 4)
        write_rows<4>(p, first_row, held, t0, block_of);
    }
  }
  if (kPart == kRows) return;
  // Few rows: the stack and the tables are for other warps than the rows (each waits for a
  // load of its own).
  const int W = ctas * warps, w = warp * ctas + rank;
  const int row_warps = ctas == 1 && kPart == kAll && 64 * p.num_rows <= 32 * threads ? (int)(p.num_rows + 31) >> 5 : 0;
  // Sequences that end give their blocks back, the first one's first.
  // (few of them to a warp: its lanes are for their blocks)
  {
    const int chunk = min((ends + W - 1) / W, 32);
    for (int c = (w + W - row_warps) % W * chunk; c < ends; c += W * chunk) {
      const int e = c + lane;
      int count = 0, to = 0;
      int64_t from = 0;
      if (lane < chunk && e < ends) {
        const int s = ending[e];
        to = given_before(e);
        count = (e + 1 < ends ? given_before(e + 1) : (int)min(given, (int64_t)p.capacity)) - to;
        from = (int64_t)s * p.max_blocks_per_seq + held[s];
      }
      for_items(count, [&](int owner, int i, bool live) {
        const int64_t at = __shfl_sync(0xffffffffu, from, owner) + i;
        const int64_t place = (int64_t)free0 + __shfl_sync(0xffffffffu, to, owner) + i;
        if (live && place < p.capacity) p.free_blocks[place] = load<kPart>(p.block_tables + at);
      });
    }
  }
  // Tables.
  if (total[1] > 0) {
    const int first = row_warps > 0 ? W / 2 : 0, some = W - first;
    const int chunk = min((S + some - 1) / some, 32);
    for (int c = (w - first) * chunk; w >= first && c < S; c += some * chunk) {
      const int s = c + lane;
      int count = 0, have = 0, from = 0;
      if (lane < chunk && s < S && held[s] >= 0 && base[s] >= 0) {
        const int L = held[s], n = first_row[s + 1] - first_row[s];
        have = (L + bs1) >> shift;
        count = n == 0 ? 0 : (int)(((int64_t)L + n + bs1) >> shift) - have;
        from = base[s];
      }
      for_items(count, [&](int owner, int i, bool live) {
        const int at = __shfl_sync(0xffffffffu, have, owner) + i;
        const int64_t b = (int64_t)__shfl_sync(0xffffffffu, from, owner) + i;
        if (live) p.block_tables[(int64_t)(c + owner) * p.max_blocks_per_seq + at] = block_at(b);
      });
    }
  }
  // Lengths and sums, once every CTA has read those from before.
  if (kPart == kState) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (rank == ctas - 1) {
    int64_t key = keys[0];
    for (int s = s0; s < s1; ++s) {
      const int h = held[s], n = first_row[s + 1] - first_row[s];
      const int after = base[s] < 0 ? 0 : h < 0 ? -1 : h + n;
      p.cu_q[s] = first_row[s];
      p.cu_k[s] = saturated(key);
      if (after > 0) key += after;
      if (after >= 0) p.new_context_lens[s] = after;
      else p.new_context_lens[s] = load<kPart>(p.context_lens + s);  // as it was
    }
    if (tid == 0) {
      int64_t got = 0;
      for (int i = 0; i < warps; ++i) got = sums3[i][0] > got ? sums3[i][0] : got;
      *p.new_num_free = left - (int)got;
      p.cu_q[S] = first_row[S];
      p.cu_k[S] = saturated(all_keys[0]);
      if (all_keys[0] > 0x7FFFFFFF || total[2] > 0x7FFFFFFF)
        flag_status(p.status, PKV_DEV_BAD_SEQLEN);
    }
  }
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_plan_step(const int32_t *new_lens, const int32_t *context_lens,
                                    const int32_t *borrowed_blocks, int32_t *block_tables,
                                    int32_t *free_blocks, const int32_t *num_free,
                                    int32_t *new_context_lens, int32_t *new_num_free,
                                    int32_t *slot_mapping, int32_t *positions,
                                    int32_t *cu_seqlens_q, int32_t *cu_seqlens_k, int num_seqs,
                                    int64_t num_rows, int max_blocks_per_seq, int block_size,
                                    int64_t num_blocks, int64_t free_capacity,
                                    int32_t *dev_status, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_rows < 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
      num_blocks <= 0 || free_capacity < 0)
    return PKV_ERR_INVALID_ARG;
  if (block_size != 64 && block_size != 128 && block_size != 256 && block_size != 512)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs > kPlanMaxSeqs || num_rows > 0x7FFFFFFELL || free_capacity > 0x7FFFFFFFLL ||
      num_blocks > 0x7FFFFFFFLL / block_size ||
      (int64_t)max_blocks_per_seq * block_size > (1 << 30))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 && num_rows > 0) return PKV_ERR_INVALID_ARG;
  if (!num_free || !new_num_free || !cu_seqlens_q || !cu_seqlens_k) return PKV_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!new_lens || !context_lens || !block_tables || !new_context_lens))
    return PKV_ERR_INVALID_ARG;
  if (num_rows > 0 && (!slot_mapping || !positions)) return PKV_ERR_INVALID_ARG;
  if (free_capacity > 0 && !free_blocks) return PKV_ERR_INVALID_ARG;
  // (the same lengths in and out, or others: nothing between)
  const uintptr_t in = reinterpret_cast<uintptr_t>(context_lens);
  const uintptr_t after = reinterpret_cast<uintptr_t>(new_context_lens);
  if (in != after && (in < after ? after - in : in - after) < (uintptr_t)num_seqs * 4)
    return PKV_ERR_INVALID_ARG;

  PlanParams prm;
  prm.new_lens = new_lens;
  prm.context_lens = context_lens;
  prm.borrowed = borrowed_blocks;
  prm.block_tables = block_tables;
  prm.free_blocks = free_blocks;
  prm.num_free = num_free;
  prm.new_context_lens = new_context_lens;
  prm.new_num_free = new_num_free;
  prm.slots = slot_mapping;
  prm.positions = positions;
  prm.cu_q = cu_seqlens_q;
  prm.cu_k = cu_seqlens_k;
  prm.status = dev_status;
  prm.num_rows = num_rows;
  prm.num_blocks = num_blocks;
  prm.capacity = (int)free_capacity;
  prm.num_seqs = num_seqs;
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.block_shift = 31 - __builtin_clz((unsigned)block_size);

  prm.rows_16b = aligned16(slot_mapping) && aligned16(positions) ? 1 : 0;

  const bool small = num_rows <= kPlanSmallRows && num_seqs <= kPlanSmallSeqs;
  const int threads = small ? kPlanSmallSeqs : num_seqs <= kPlanManySeqs ? kPlanThreads : kPlanManyThreads;
  const int smem = (3 * num_seqs + 1) * 4 + (num_seqs * 2 + 3) / 4 * 4;
  static_assert((3 * kPlanMaxSeqs + 1) * 4 + kPlanMaxSeqs * 2 + 1024 <= 232448, "shared memory");
  const bool rows_apart = !small && num_rows > 0;
  const auto kernel = rows_apart ? plan_step_kernel<kState> : plan_step_kernel<kAll>;
  if (!kernel_smem_setup((const void *)kernel, threads, smem, nullptr) ||
      (rows_apart && !kernel_smem_setup((const void *)plan_step_kernel<kRows>, threads, smem, nullptr)))
    return PKV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = small ? 1 : kPlanCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cudaError_t err = cudaSuccess;
  if (rows_apart) {
    const int sms = device_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    // A row a thread on up to half of the SMs, else four (115 thousand rows 7.0 us with one
    // and 6.0 with four, which leave SMs to the launch behind; 1000 6.8 and 7.0).
    int64_t ctas = (num_rows + threads - 1) / threads;
    if (ctas > sms / 2) ctas = (num_rows + 4 * threads - 1) / (4 * threads);
    cfg.gridDim = dim3((unsigned)(ctas < sms ? ctas : sms));
    cfg.blockDim = dim3(threads);
    cfg.numAttrs = 1;  // (no cluster)
    err = cudaLaunchKernelEx(&cfg, plan_step_kernel<kRows>, prm);
  }
  if (err == cudaSuccess) {
    cfg.gridDim = dim3(small ? 1 : kPlanCluster);
    cfg.blockDim = dim3(threads);
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, kernel, prm);
  }
  return launch_status();
}
