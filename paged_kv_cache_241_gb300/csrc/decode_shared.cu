// decode_shared.cu -- decode attention for a batch whose sequences share prefixes.
//
// The block manager lets sequences with the same beginning hold the same blocks (CSDN
// essay "from nanoVLLM to vLLM", Mountain 1; nano-vllm hub page, "core tech 4").  Plain
// decode reads those blocks once for every sequence.  Here a group of neighbouring
// sequences with the same first blocks reads them once: for a kv head, the query rows
// of all (sequence, head of its group) are one matrix Q [m G, D], and over the prefix's
// keys, which every row sees whole,
//   M = max_p z,  l = sum_p exp(z_p - M),  o = sum_p exp(z_p - M) V_p,  z = scale Q K^T
// is a product on the tensor cores.  What a sequence has behind the prefix is split-K
// decode.  All parts (M, l, o) of a row are then joined:
//   out = sum_i exp(M_i - M) o_i / sum_i exp(M_i - M) l_i.
//
// Three launches, each a programmatic dependent of the one before:
//  1. plan: one CTA.  A group's prefix ends where its shortest sequence does; prefix
//     sums of the work of groups (steps of 64 keys) and of sequences (tiles of 4 KiB
//     of K) go to the workspace, and how many CTAs work on prefixes.
//  2. attention: one CTA per SM.  Some of them take the prefixes, units of (group, kv
//     head, 256 rows) by steps, cut into runs of equal cost, a CTA for each (tcgen05,
//     TMA); the others the tails, all sequences' own tokens, cut into runs of equal
//     length, a warp for each run and kv head (m16n8k16, cp.async; bound by HBM).
//  3. join.
// A small batch shares nothing and has two: in place of the plan every CTA of the second
// sums up the lengths.  One of few and short contexts has a single launch, of a CTA for each
// sequence and kv head.
//
// What bounds it: long prefixes HBM and the tensor cores (of 128 rows, D = 128, 0.74 us per
// 64 keys of a CTA, 6.7 TB/s over the GPU; of 256 rows 1.29 us, its products with S about
// 600 of 2470 cycles, those with V 460, for each row tile: one of 128 x 64 takes nearly as
// long as one of 128 x 128, but with S of 128 keys at a time, which leaves one S buffer to a
// chain, a step took 1.43); tails HBM; and all of it a fixed part of 15 to 18 us: the plan 3
// us, from the beginning of a CTA to its first product 4.5, from a run's last product to its
// stores 2.5, the join 2.5, what is between the launches 3.  In a graph of calls, floors by
// bytes in brackets: 64 sequences behind 2048 tokens 31.1 us [21.8], 50 in 6 groups 26.3
// [9.7], 16 on a document of 32,000 37.3 [20.9], 128 behind 8192 48.9 [25.5], 2 short 3.8
// (in tables of two blocks; of 8192 tokens 6.5).
#include <math.h>

#include <atomic>

#include "cta_scan.cuh"
#include "host_common.h"
#include "pkv_common.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kSharedMaxSeqs = 8192;
constexpr int kMaxTokens = 1 << 20;      // of a sequence
constexpr int kPlanThreads = 1024;
constexpr int kWarpsMost = 8;            // warps per CTA of the tails (one CTA per SM)
constexpr int kStages = 3;               // ring of tiles per warp
constexpr int kMaxCtas = 160;            // CTAs of the attention's grid at most (places for
constexpr int kMaxWarps = kMaxCtas * kWarpsMost;  // parts; a GB300 has 152 SMs)
constexpr int kThreads = 384;            // of the attention's CTAs
// A batch of at most so many sequences whose tables have room for no more K and V than
// kSmallBytes is small: reading it whole takes 2 us or so, and a prefix's pipeline alone 6
// (two sequences behind 256 tokens: 6.3 us in two launches, 9.4 planned but not shared, 12.6
// shared).
constexpr int64_t kSmallBytes = 16 << 20;
constexpr int kSmallSeqs = kThreads;
// One whose tables have room for at most so many tokens a sequence (half as many with eight
// heads to a kv head), and of so many sequences and kv heads per SM, is done in a single
// launch (us so and otherwise; 2 x 2 heads of 64 dims, 2 sequences behind 256 tokens 3.2 and
// 6.3, 1024 5.3 and 6.6, 2048 8.3 and 7.7; 2 x 8 of 128, 8 behind 1024 8.1 and 13.7, 32 behind
// 1024 15.5 and 16.2, 100 behind 256 21.2 and 16.7; 8 x 8 of 128, 2 behind 512 7.6 and 8.7,
// behind 1024 11.3 and 10.5).
constexpr int kShortTokens = 1024;
constexpr int kShortCtas = 2;
constexpr int kNearGroups = 32;          // groups whose plans fit a CTA's shared memory
constexpr int kMaxDynamicSmem = 232448;  // opt-in shared memory per CTA on sm_103 (227 KiB)
constexpr int BM = 128;                  // rows of a product
constexpr int BN = 64;                   // keys of a step
constexpr int kPairRows = 2 * BM;        // rows of a unit: two products share its keys
constexpr int kUnitSlots = 4;
constexpr int kJoinWarps = 4;            // per CTA
constexpr float kLog2e = 1.4426950408889634f;

// The prefix of a group, in the workspace.
struct GroupPlan {
  int64_t cost0;  // cost of the groups before it
  int start;      // its first sequence
  int lead;       // the sequence whose row of the block tables is read
  int members;
  int tiles;      // steps of 64 keys (0: nothing is shared)
  int pad[2];
};
// The cost of a step, in cost_ns: of a unit with two row tiles 5 (its products), of one
// with a single row tile 3 (its loads).  A unit's beginning costs kUnitCost ahead of its
// steps (a run that goes through the end of one into the next drains its pipeline there);
// a kv head's units follow one another.
constexpr int kUnitCost = 15;
constexpr int kPairCost = 5, kSingleCost = 3;
__device__ __forceinline__ int step_cost(int rows) { return rows > BM ? kPairCost : kSingleCost; }
__device__ __forceinline__ int64_t full_unit_cost(const GroupPlan &g) {  // of 256 rows
  return kUnitCost + kPairCost * (int64_t)g.tiles;
}
__device__ __forceinline__ int64_t head_cost(const GroupPlan &g, int group_size) {
  const int rows = g.members * group_size, last = rows % kPairRows;
  return rows / kPairRows * full_unit_cost(g) +
         (last == 0 || g.tiles == 0 ? 0 : kUnitCost + (int64_t)step_cost(last) * g.tiles);
}

// A sequence's tail, in the workspace.
struct SeqPlan {
  int tile0;  // tiles of the tails before it
  int begin;  // its first token
  int len;    // tokens of the sequence (0: no output)
  int pad;
};

// What the join needs of a sequence, in the workspace.
struct JoinPlan {
  int row0;      // the sequence's number and its tail's first run (tail_ml, tail_o)
  int tails;     // parts of its tail
  int place;     // of the sequence in its group
  int members;   // GroupPlan of its group
  int tiles;     // (0, too, where the sequence has no tokens)
  int pad;
  int64_t cost0;
  int64_t run_cost;  // Totals
  int64_t pad2;
};
static_assert(sizeof(JoinPlan) == 48, "three loads");

struct Totals {
  int64_t cost;      // of all prefixes
  int64_t run_cost;  // of a run of them
  int tiles;         // of all tails
  int run_tiles;     // of a run of them
  int prefix_ctas;   // CTAs that take the prefixes; the others take the tails
  int pad;
};

struct SharedParams {
  uint16_t *out;
  const uint16_t *q;
  const uint16_t *k_cache;
  const uint16_t *v_cache;
  const int32_t *block_tables;
  const int32_t *context_lens;
  const int32_t *group_starts;
  const int32_t *shared_blocks;
  Totals *totals;
  GroupPlan *groups;   // [num_groups]
  SeqPlan *seqs;       // [num_seqs]
  JoinPlan *joins;     // [num_seqs]
  float *tail_ml;      // [num_seqs + runs, Hkv, G, 2]   (max in log2 units, sum)
  float *tail_o;       // [num_seqs + runs, Hkv, G, D]
  float *first_ml;     // [num_seqs, Hq, 2]: a unit's first part
  float *first_o;      // [num_seqs, Hq, D]
  float *run_ml;       // [CTAs, 256, 2]: the part with which a run begins inside a unit
  float *run_o;        // [CTAs, 256, D]
  int32_t *status;
  int64_t num_blocks;
  int num_seqs;
  int num_groups;
  int num_kv_heads;
  int group_size;      // G
  int block_shift;
  int max_blocks_per_seq;
  int ctas;            // of the attention's grid
  int tail_warps;      // warps of a CTA that takes tails
  int loading;         // CTAs that load their prefixes: all, but in a test
  int share_always;    // whatever it saves (test)
  int small;           // no plan was launched
  int groups_at;       // where the groups' plans are in a CTA's shared memory
  int head_dim;
  float qscale;        // scale * log2(e)
};

// Tokens of K in a tile of a tail: 4 KiB.
__host__ __device__ constexpr int tail_rows(int D) { return 2048 / D; }
__device__ __forceinline__ int tail_tiles(int tokens, int D) {
  return D == 64 ? (tokens + 31) >> 5 : (tokens + 15) >> 4;
}
static_assert(tail_rows(64) == 32 && tail_rows(128) == 16, "shifts");

// (Divisions of 64 bits take four times as long.)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Tiles per run of the tails; run r's part of sequence s is filed under s + r (a part
// begins where a sequence or a run does, so no two have the same number).  Cost per run of
// the prefixes (at least that of the dearest step, so that every run between a unit's first
// and last has a step of it).
__device__ __forceinline__ void cut_runs(const SharedParams &p, Totals &t) {
  const int runs = max((p.ctas - t.prefix_ctas) * p.tail_warps / p.num_kv_heads, 1);
  t.run_tiles = max((t.tiles + runs - 1) / runs, 1);
  const int n = max(t.prefix_ctas, 1);
  t.run_cost = max(quotient(t.cost + n - 1, n), (int64_t)kPairCost);
}
__device__ __forceinline__ JoinPlan join_plan(const Totals &t, int s, int tile0, int tiles, int place,
                                              const GroupPlan &g, bool live) {
  JoinPlan x;
  const int r0 = tile0 / t.run_tiles;
  x.row0 = s + r0;
  x.tails = tiles > 0 ? (tile0 + tiles - 1) / t.run_tiles - r0 + 1 : 0;
  x.place = place;
  x.members = g.members;
  x.tiles = live ? g.tiles : 0;
  x.cost0 = g.cost0;
  x.run_cost = t.run_cost;
  x.pad = 0;
  x.pad2 = 0;
  return x;
}

// ----------------------------------------------------------------------- 1. plan

// How many of the CTAs take the prefixes: what lets both kinds end together.  Times in
// nanoseconds, as measured: of a unit of cost, and the beginning and end of a run; of a
// tile of a tail (K and V of tail_rows tokens, a kv head) for all of a CTA's warps, and
// of their beginning; and what sharing costs beside.
constexpr int kPrefixNs = 6000, kTailNs = 2500, kSharingNs = 2800;
__device__ __forceinline__ float cost_ns(const SharedParams &p) {
  return p.head_dim == 64 ? 220.f : 255.f;
}
// (A tile of 64 dims is two slices of 16 tokens, and eight heads take two products with V.)
__device__ __forceinline__ float tile_ns(const SharedParams &p) {
  return p.head_dim == 64 ? (p.group_size == 8 ? 165.f : 150.f) : p.group_size == 8 ? 140.f : 115.f;
}

__device__ __forceinline__ int split_ctas(const SharedParams &p, float cost, float tiles) {
  const float a = cost * cost_ns(p), b = tiles * p.num_kv_heads * tile_ns(p);
  if (a == 0.f) return 0;
  if (b == 0.f) return p.ctas;
  // a / n + kPrefixNs = b / (ctas - n) + kTailNs, solved for n: the whole number beside
  // it that ends sooner (one CTA of a kind at least).
  const float N = p.ctas, d = kPrefixNs - kTailNs, e = d * N - a - b;
  const float root = sqrtf(e * e + 4.f * d * a * N);
  const float n = e >= 0.f ? (e + root) / (2.f * d) : 2.f * a * N / (root - e);  // (no cancellation)
  auto time = [&](float n) {
    return fmaxf(__fdividef(a, n) + kPrefixNs, __fdividef(b, N - n) + kTailNs);
  };
  const float low = fminf(fmaxf(floorf(n), 1.f), N - 1.f), high = fminf(low + 1.f, N - 1.f);
  return (int)(time(high) < time(low) ? high : low);
}
static_assert(kPrefixNs > kTailNs, "the equation's quadratic term");

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedParams p) {
  extern __shared__ int plan_smem[];
  __shared__ int64_t sums[32][2];
  const int S = p.num_seqs, N = p.num_groups, tid = threadIdx.x;
  int *starts = plan_smem;       // [N + 1]
  int *eff = starts + N + 1;     // [N]: blocks that the group shares
  int *lead = eff + N;           // [N]: its first sequence with tokens
  int *count = lead + N;         // [N]: its sequences with tokens
  int64_t *cost0 = reinterpret_cast<int64_t *>(plan_smem + ((4 * N + 2) & ~1));  // [N]
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  auto tokens = [&](int L) { return L <= 0 ? 0 : (int)min((int64_t)L, room); };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int first_L = tid < S ? p.context_lens[tid] : 0;  // (asked for ahead)
  bool ok = true;
  for (int g = tid; g <= N; g += blockDim.x) {
    const int x = p.group_starts[g];
    starts[g] = x;
    ok = ok && (g > 0 || x == 0) && (g < N || x == S);
    if (g < N) {
      const int b = p.shared_blocks[g];
      if (b < 0 || b > p.max_blocks_per_seq) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
      eff[g] = min(max(b, 0), p.max_blocks_per_seq);
      lead[g] = 0x7FFFFFFF;
      count[g] = 0;
    }
  }
  __syncthreads();
  for (int g = tid; g < N; g += blockDim.x) ok = ok && starts[g] <= starts[g + 1];
  ok = __syncthreads_and(ok) != 0;
  // (no groups then: every sequence by itself)
  if (!ok && tid == 0) flag_status(p.status, PKV_DEV_BAD_SEQLEN);
  if (ok) {
    for (int s0 = tid & ~31; s0 < S; s0 += blockDim.x) {
      const int s = s0 + (tid & 31);
      const int L = s < S ? tokens(s == tid ? first_L : p.context_lens[s]) : 0;
      const int g = s < S ? seq_of(starts, N, s) : -1;
      // (a warp's sequences are neighbours: mostly one group)
      const unsigned peers = __match_any_sync(0xffffffffu, L > 0 ? g : -1);
      if (L > 0) {
        const int least = __reduce_min_sync(peers, L >> p.block_shift);
        if ((tid & 31) == __ffs(peers) - 1) {
          atomicMin(&eff[g], least);
          atomicMin(&lead[g], s);
          atomicAdd(&count[g], __popc(peers));
        }
      }
    }
  }
  __syncthreads();
  const int per_g = N <= (int)blockDim.x ? 1 : (N + blockDim.x - 1) / (int)blockDim.x;
  const int g0 = min(tid * per_g, N), g1 = min(g0 + per_g, N);
  auto plan = [&](int g) {
    GroupPlan x;
    const int blocks = ok && count[g] >= 2 ? eff[g] : 0;
    x.start = starts[g];
    x.members = blocks > 0 ? starts[g + 1] - starts[g] : 0;
    x.lead = blocks > 0 ? lead[g] : 0;
    x.tiles = blocks << (p.block_shift - 6);
    x.pad[0] = x.pad[1] = 0;
    x.cost0 = 0;
    return x;
  };
  static_assert(BN == 64, "a shift by 6");
  auto cost_of = [&](const GroupPlan &x) {
    return head_cost(x, p.group_size) * p.num_kv_heads;
  };
  const int per = S <= (int)blockDim.x ? 1 : (S + blockDim.x - 1) / (int)blockDim.x;
  const int s0 = min(tid * per, S), s1 = min(s0 + per, S);
  auto first = [&](int s, int L, int &g) {
    g = ok ? seq_of(starts, N, s) : 0;
    return L > 0 && ok && count[g] >= 2 ? eff[g] << p.block_shift : 0;
  };
  // Cost of the prefixes; tiles of the tails, and without sharing (2^29 at most: both in
  // one 64-bit sum).
  int64_t at[2] = {0, 0}, sum[2];
  int64_t my_cost = 0;  // (of the thread's last group, and sequence: mostly its only ones)
  int my_g = 0, my_b = 0, my_L = 0;
  for (int g = g0; g < g1; ++g) at[0] += my_cost = cost_of(plan(g));
  for (int s = s0; s < s1; ++s) {
    const int L0 = per == 1 ? first_L : p.context_lens[s];
    my_L = tokens(L0);
    my_b = first(s, my_L, my_g);
    at[1] += (int64_t)tail_tiles(my_L - my_b, p.head_dim) << 32 | tail_tiles(my_L, p.head_dim);
    if (my_L != L0 || my_L == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  }
  scan_cta<2>(at, sum, sums);
  int64_t cost = sum[0];
  int tile = (int)(at[1] >> 32), tiles = (int)(sum[1] >> 32);
  // Little work: reading every context whole takes less than a run of a prefix at its
  // best, and so nothing is shared (of 8 x 2 heads: 8 sequences behind 1024 tokens 13.0 us
  // so and 15.1 shared, behind 2048 14.9 and 16.8, 16 behind 2048 19.2 and 16.8).
  if (!p.share_always &&
      (float)(int)sum[1] * p.num_kv_heads * tile_ns(p) + (float)kTailNs * p.ctas <=
          (float)cost * cost_ns(p) + (float)(kPrefixNs + kSharingNs) * p.ctas) {
    ok = false;
    at[0] = cost = 0;
    tile = (int)at[1];
    tiles = (int)sum[1];
    my_cost = my_b = my_g = 0;
  }
  Totals t;
  t.cost = cost;
  t.tiles = tiles;
  t.prefix_ctas = split_ctas(p, (float)cost, (float)tiles);
  t.pad = 0;
  cut_runs(p, t);
  if (tid == 0) *p.totals = t;
  for (int g = g0; g < g1; ++g) {
    GroupPlan x = plan(g);
    x.cost0 = cost0[g] = at[0];
    p.groups[g] = x;
    at[0] += per_g == 1 ? my_cost : cost_of(x);
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    if (per > 1) {
      my_L = tokens(p.context_lens[s]);
      my_b = first(s, my_L, my_g);
    }
    *reinterpret_cast<int4 *>(p.seqs + s) = make_int4(tile, my_b, my_L, 0);
    const int mine = tail_tiles(my_L - my_b, p.head_dim);
    GroupPlan x = plan(my_g);
    x.cost0 = cost0[my_g];
    p.joins[s] = join_plan(t, s, tile, mine, s - x.start, x, my_L > 0);
    tile += mine;
  }
}

// ---------------------------------------------------------------------- 2. tails

// Shared memory of one warp: a ring of tiles (tail_rows tokens of K, then of V), and
// as many places for the query rows of the sequences in flight.
template <int D, int G>
struct WarpSmem {
  static constexpr int kRows = tail_rows(D);
  static constexpr int kHalf = kRows * D * 2;     // 4 KiB of K or V
  static constexpr int kQ = G * D * 2;
  static constexpr int bytes = kStages * (2 * kHalf + kQ);
};

// A warp streams the K and V of its run, for its kv head, through its own ring, up to
// two tiles ahead and across sequences; nothing in the loop waits for another warp, and
// the warps of the other kv heads of the same tokens run beside it.  Per 16 tokens:
// S = K q^T (tokens x dims x heads) and O^T += V^T P (dims x tokens x heads).  P is an
// operand in bf16: it goes in as the sum of two, the weight cut and what that leaves, so
// that it is off by 2^-16 of itself and not by 2^-8 (paged_decode_attn keeps it in
// fp32).  With at most four heads columns 4 to 7 repeat the heads of 0 to 3 and take the
// second parts; eight heads need a second product.
//
// smem_raw: the warps' rings, then [S + 1] first tiles, [S] first tokens and [S] lengths
// of the sequences' tails, which are there already.  kOne: there is one sequence, `seq`, of
// which a CTA's warps share the tiles for kv head `kvh`, and their parts go to `parts` in
// shared memory, [warps, G] rows of D values of O, then of (max, sum).
template <int D, int G, bool kOne>
__device__ __forceinline__ void tails(const SharedParams &p, const Totals &sum, uint8_t *smem_raw,
                                      int seq, int kvh, float *parts) {
  using W = WarpSmem<D, G>;
  constexpr int kRows = W::kRows;
  constexpr int kCols = D / 8;              // 16-byte columns per row
  constexpr int kRowsPer = 32 / kCols;      // rows per warp-wide copy
  constexpr int kSlices = kRows / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = p.tail_warps;
  uint8_t *mine = smem_raw + warp * W::bytes;
  const int S = kOne ? 1 : p.num_seqs, Hkv = p.num_kv_heads, shift = p.block_shift;
  const int32_t *tables = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
  int *tile0 = reinterpret_cast<int *>(smem_raw + warps * W::bytes);  // [S + 1]
  int *begin = tile0 + S + 1;                                         // [S]
  int *len = begin + S;                                               // [S]
  const uint32_t tiles = smem_u32(mine);
  const uint32_t qslots = tiles + kStages * 2 * W::kHalf;

  if (warp >= warps) return;
  const int total = tile0[S];
  const int per_run = kOne ? max((total + warps - 1) / warps, 1) : sum.run_tiles;
  const int runs = (total + per_run - 1) / per_run;
  const int64_t jobs = kOne ? runs : (int64_t)runs * Hkv;  // (run, head), heads innermost
  const uint64_t policy = l2_policy_evict_first();
  const int col = lane % kCols, row0 = lane / kCols;
  for (int64_t job = kOne ? warp : (int64_t)(blockIdx.x - sum.prefix_ctas) * warps + warp; job < jobs;
       job += kOne ? jobs : (int64_t)(p.ctas - sum.prefix_ctas) * warps) {
    const int r = kOne ? warp : (int)(job / Hkv), j = kOne ? kvh : (int)(job - (int64_t)r * Hkv);
    const int t_begin = r * per_run, t_end = min(t_begin + per_run, total);

    // The loading side: tile in_t of the batch, at token in_tok of sequence in_s (in_L
    // tokens), in block blk; blk_next is the block after it, of this sequence or the next.
    int in_t = t_begin, in_s = seq_of(tile0, S, t_begin);
    int in_tok = begin[in_s] + (t_begin - tile0[in_s]) * kRows;
    int in_L = len[in_s];
    int in_slot = 0, in_q = 0;
    bool in_first = true;  // the sequence's first tile of this run
    auto block_of = [&](int s, int tok) {
      int blk = tables[(int64_t)s * p.max_blocks_per_seq + (tok >> shift)];
      if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
        blk = 0;
      }
      return blk;
    };
    auto next_seq = [&](int s) {  // the next sequence with a tail
      do ++s; while (s < S && tile0[s + 1] == tile0[s]);
      return s;
    };
    auto block_after = [&]() {
      const int tok = ((in_tok >> shift) + 1) << shift;
      if (tok < in_L) return block_of(in_s, tok);
      const int s = next_seq(in_s);
      return s < S ? block_of(s, begin[s]) : 0;
    };
    int blk = block_of(in_s, in_tok), blk_next = block_after();
    auto issue = [&]() {
      if (in_t < t_end) {
        if (in_first) {
          const uint16_t *q = p.q + ((int64_t)(seq + in_s) * Hkv + j) * G * D;
          for (int x = lane; x < G * kCols; x += 32)
            copy16(qslots + in_q * W::kQ + tile_at<D>(x / kCols, x % kCols), q + x * 8, true, policy);
          in_q = in_q + 1 == kStages ? 0 : in_q + 1;
          in_first = false;
        }
        const int64_t slot = ((int64_t)blk << shift) + (in_tok & ((1 << shift) - 1));
        const int64_t at = ((slot + row0) * Hkv + j) * D + col * 8;
        const int64_t step = (int64_t)kRowsPer * Hkv * D;
        const uint32_t dst = tiles + in_slot * 2 * W::kHalf;
#pragma unroll
        for (int i = 0; i < kRows / kRowsPer; ++i) {
          const int t = in_tok + row0 + i * kRowsPer;
          const uint32_t to = dst + tile_at<D>(row0 + i * kRowsPer, col);
          copy16(to, p.k_cache + at + i * step, t < in_L, policy);
          copy16(to + W::kHalf, p.v_cache + at + i * step, t < in_L, policy);
        }
        ++in_t;
        in_slot = in_slot + 1 == kStages ? 0 : in_slot + 1;
        if (in_t < t_end) {
          in_tok += kRows;
          const bool ends = in_tok >= in_L;
          if (ends || (in_tok & ((1 << shift) - 1)) == 0) {
            if (ends) {
              in_s = next_seq(in_s);
              in_tok = begin[in_s];
              in_L = len[in_s];
              in_first = true;
            }
            blk = blk_next;
            blk_next = block_after();
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    // The consuming side: sequence after sequence of the run.
    const int h0 = 2 * (lane & 3);  // this lane's heads: columns h0, h0 + 1 of the group
    const bool owner = h0 < G;      // (of the 8 columns only G are heads of their own)
    int slot = 0, qslot = 0;
    for (int s = seq_of(tile0, S, t_begin), tile = t_begin; tile < t_end; s = next_seq(s)) {
      const int L = len[s];
      const int first = begin[s] + (tile - tile0[s]) * kRows;       // tokens [first, last) are here
      const int last = min(L, first + (t_end - tile) * kRows);
      uint32_t qf[D / 16][2];
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float o[D / 16][4];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      for (int tok = first; tok < last; tok += kRows, ++tile) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();  // every lane's copies are in, and the slot filled next is read out
        issue();
        if (tok == first) {
          // q as the second operand: lane (head, dim pair) per 8 dims.  With fewer than
          // eight heads, rows 4 to 7 are 0 to 3 again, those past G the last one.
          const uint32_t qa = qslots + qslot * W::kQ;
          const int row = G == 8 ? lane & 7 : min(lane & 3, G - 1);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t f[4];
            ldmatrix4(f, qa + tile_at<D>(row, i * 4 + (lane >> 3)));
            qf[2 * i][0] = f[0];
            qf[2 * i][1] = f[1];
            qf[2 * i + 1][0] = f[2];
            qf[2 * i + 1][1] = f[3];
          }
          qslot = qslot + 1 == kStages ? 0 : qslot + 1;
        }
        const uint32_t ka = tiles + slot * 2 * W::kHalf, va = ka + W::kHalf;
#pragma unroll
        for (int sl = 0; sl < kSlices; ++sl) {
          // S: rows are tokens (lane / 4 and + 8), columns the lane's two heads.
          float s_even[4] = {0.f, 0.f, 0.f, 0.f}, s_odd[4] = {0.f, 0.f, 0.f, 0.f};
          const int kr = sl * 16 + (lane & 15);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
            ldmatrix4(a, ka + tile_at<D>(kr, 2 * i + (lane >> 4)));
            if (i & 1) mma16816(s_odd, a, qf[i][0], qf[i][1]);
            else mma16816(s_even, a, qf[i][0], qf[i][1]);
          }
          const int i0 = sl * 16 + (lane >> 2), i1 = i0 + 8;  // rows of the tile
          float z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = (s_even[i] + s_odd[i]) * p.qscale;
          if (tok + i0 >= L) z[0] = z[1] = -INFINITY;
          if (tok + i1 >= L) z[2] = z[3] = -INFINITY;
          float n0 = fmaxf(z[0], z[2]), n1 = fmaxf(z[1], z[3]);
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, k));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, k));
          }
          n0 = fmaxf(n0, m0);
          n1 = fmaxf(n1, m1);
          // (a maximum of -inf: every weight so far is zero, whatever the reference)
          const float r0 = n0 == -INFINITY ? 0.f : n0, r1 = n1 == -INFINITY ? 0.f : n1;
          const float a0 = fast_exp2(m0 - r0), a1 = fast_exp2(m1 - r1);
          m0 = n0;
          m1 = n1;
          const float p0 = fast_exp2(z[0] - r0), p1 = fast_exp2(z[1] - r1);
          const float p2 = fast_exp2(z[2] - r0), p3 = fast_exp2(z[3] - r1);
          l0 = fmaf(l0, a0, p0 + p2);
          l1 = fmaf(l1, a1, p1 + p3);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][0] *= a0;
            o[i][1] *= a1;
            o[i][2] *= a0;
            o[i][3] *= a1;
          }
          // P as the second operand of the next product, in two parts (see above);
          // the sums keep the fp32 weights.
          uint32_t first0 = cut_bf16x2(p0, p1), first1 = cut_bf16x2(p2, p3);
          const uint32_t rest0 = rest_bf16x2(p0, p1, first0);
          const uint32_t rest1 = rest_bf16x2(p2, p3, first1);
          if (G < 8 && (lane & 2)) {
            first0 = rest0;
            first1 = rest1;
          }
          const uint32_t b0 = transpose8x8(first0), b1 = transpose8x8(first1);
          uint32_t c0 = 0, c1 = 0;
          if (G == 8) {
            c0 = transpose8x8(rest0);
            c1 = transpose8x8(rest1);
          }
          // V^T: two 8-token halves by two 8-dim columns, transposed on the way.
          const int vr = sl * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
            ldmatrix4_trans(a, va + tile_at<D>(vr, 2 * i + ((lane >> 3) & 1)));
            mma16816(o[i], a, b0, b1);
            if (G == 8) mma16816(o[i], a, c0, c1);
          }
        }
        slot = slot + 1 == kStages ? 0 : slot + 1;
      }
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, k);
        l1 += __shfl_xor_sync(0xffffffffu, l1, k);
      }
      if (G < 8) {  // the two halves of O
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[i][x] += __shfl_xor_sync(0xffffffffu, o[i][x], 2);
      }
      if (owner) {
        const int64_t part = kOne ? warp * G + h0 : ((int64_t)(s + r) * Hkv + j) * G + h0;
        float *po = (kOne ? parts : p.tail_o) + part * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int d = i * 16 + (lane >> 2);
          po[d] = o[i][0];
          po[d + 8] = o[i][2];
          if (G > 1) {
            po[D + d] = o[i][1];
            po[D + d + 8] = o[i][3];
          }
        }
        if (lane < 4) {
          float2 *ml = reinterpret_cast<float2 *>(kOne ? parts + warps * G * D : p.tail_ml) + part;
          ml[0] = make_float2(m0, l0);
          if (G > 1) ml[1] = make_float2(m1, l1);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
}

// ------------------------------------------------------------------- 3. prefixes

// A piece of a unit: steps [tile, tile + n) of rows [256 pair, 256 pair + rows) of the
// group that begins at sequence start, for kv head kvh.
struct Piece {
  int start, lead, kvh, pair, rows, tile, n;
  int first;  // it begins where the unit does: its parts are filed by row, else by run
  int once;   // no other unit reads its keys
};

template <int D>
struct PrefixLayout {
  static constexpr int kQBytes = BM * D * 2;
  static constexpr int kKVBytes = BN * D * 2;
  static constexpr int kSlots0 = (kMaxDynamicSmem - 6144 - 2 * kQBytes) / kKVBytes;
  static constexpr int kSlots = kSlots0 < 16 ? kSlots0 : 16;
  static constexpr int kKStages = (kSlots * 2 + 2) / 5;  // (a V slot is held longer)
  static constexpr int kVStages = kSlots - kKStages;
  static constexpr int q = 0;
  static constexpr int k = q + 2 * kQBytes;
  static constexpr int v = k + kKStages * kKVBytes;
  static constexpr int bars = v + kVStages * kKVBytes;
  // q_full, q_empty, k_full[SK], v_full[SV], k_empty[SK], v_empty[SV], s_full[2][2],
  // p_full[2][2], p_free[2][2], o_free[2], unit_full[U], unit_empty[U], ex_full, drain
  static constexpr int kNumBars = 2 + 2 * kKStages + 2 * kVStages + 14 + 2 * kUnitSlots + 2;
  static constexpr int misc = bars + kNumBars * 8;  // tensor memory address, abort flag
  static constexpr int ring = misc + 8;
  static constexpr int ex = ring + (int)sizeof(Piece) * kUnitSlots;  // [2][2][128] (max, sum)
  static constexpr int total = ex + 4 * BM * 8;
  // One CTA per SM (it takes all of tensor memory): more than half of an SM's shared
  // memory, so that a second one never waits for tensor memory.
  static_assert(total + 1024 <= kMaxDynamicSmem && total > 114 * 1024, "shared memory");
};

// There are two chains of S, softmax and P.V.  A piece of more than 128 rows has a row
// tile for each, and both see every step; of one row tile they take the steps in turn
// and add up at its end, so that the softmax of two steps is in flight either way.
// Tensor memory columns (lane = row): O of the two chains at 0 and D, then two S
// buffers of 64 columns for each.  A buffer holds S (fp32), then over it P as two bf16
// terms, 32 columns each: the weight cut to bf16, and what that leaves.
template <int D>
struct PrefixCols {
  static constexpr uint32_t kS = 2 * D;
};

// One thread of the warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// A value that all of the warp has, as one of the warp.
__device__ __forceinline__ int warp_same(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const bool ok = mbar_wait_bounded(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void store32(float *ptr, const float (&v)[32], int i) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(ptr), "f"(v[i]),
               "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]),
               "f"(v[i + 6]), "f"(v[i + 7])
               : "memory");
}

// Steps [0, n) of a piece that chain h takes.
__device__ __forceinline__ int chain_steps(const Piece &u, int h) {
  return u.rows > BM ? u.n : (u.n + 1 - h) >> 1;
}

template <int D>
__device__ __forceinline__ void prefixes(const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                         const SharedParams &p, const Totals &sum,
                                         const GroupPlan *groups, uint8_t *smem_raw) {
  using L = PrefixLayout<D>;
  constexpr int XR = D / 64;  // 128-byte swizzle regions across D
  constexpr int kKStages = L::kKStages, kVStages = L::kVStages;
  constexpr uint32_t kSCol = PrefixCols<D>::kS;
  constexpr int kKWarp = 0, kSWarp = 1, kVWarp = 2, kPVWarp = 3;

  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem + L::q, *sK = smem + L::k, *sV = smem + L::v;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint64_t *q_full = bars;
  uint64_t *q_empty = bars + 1;             // the piece's S products no longer read Q
  uint64_t *k_full = bars + 2;
  uint64_t *v_full = k_full + kKStages;
  uint64_t *k_empty = v_full + kVStages;
  uint64_t *v_empty = k_empty + kKStages;
  uint64_t *s_full = v_empty + kVStages;    // [row tile][buffer]: S is in
  uint64_t *p_full = s_full + 4;            // P is written over it
  uint64_t *p_free = p_full + 4;            // that P.V is done (O updated, buffer free)
  uint64_t *o_free = p_free + 4;            // [row tile]: O has been read
  uint64_t *unit_full = o_free + 2;
  uint64_t *unit_empty = unit_full + kUnitSlots;
  uint64_t *ex_full = unit_empty + kUnitSlots;  // every softmax warp's (max, sum) of a piece
  uint64_t *drain = ex_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::misc + 4);
  Piece *ring = reinterpret_cast<Piece *>(smem + L::ring);  // start < 0 ends

  float2 *ex = reinterpret_cast<float2 *>(smem + L::ex);

  const int warp = warp_same(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int64_t len = sum.run_cost;
  const int64_t x0 = (int64_t)blockIdx.x * len;
  if (x0 >= sum.cost) return;
  const int64_t x1 = x0 + len < sum.cost ? x0 + len : sum.cost;

  if (threadIdx.x < L::kNumBars) {  // a thread each
    uint64_t *bar = bars + threadIdx.x;
    int count = 1;
    if (bar >= p_full && bar < p_free) count = 128;
    if (bar >= o_free && bar < unit_full) count = 8;  // every softmax warp, or a chain's own four twice
    if (bar >= unit_empty && bar < ex_full) count = 1 + 2 + 8;  // V loader, issuers, softmax warps
    if (bar == ex_full) count = 8;
    if (bar == drain) count = 2;
    mbar_init(bar, count);
    fence_barrier_init();
  }
  if (threadIdx.x == kThreads - 1) {
    *abort_flag = 0;
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
  }
  __syncthreads();
  // (the loaders go ahead; the others wait for tensor memory)
  uint32_t tmem = 0;
  if (warp != kKWarp && warp != kVWarp) {
    if (warp == kSWarp) {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
    tc_fence_before_sync();
    named_bar_sync(1, kThreads - 64);
    tc_fence_after_sync();
    tmem = warp_same(*tmem_slot);
  }

  auto next_piece = [&](int &iu, Piece &u) -> bool {
    const int slot = iu % kUnitSlots;
    if (!warp_wait(&unit_full[slot], (iu / kUnitSlots) & 1, abort_flag)) return false;
    u = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&unit_empty[slot]);
    ++iu;
    return u.start >= 0;
  };

  if (warp == kKWarp) {
    // Warp 0 walks the run (handing its pieces to the other roles) and loads Q and K.
    const bool loads = (int)blockIdx.x < p.loading;
    const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
    int iu = 0, g = 0, q_loads = 0;
    bool ok = true;
    int64_t x = x0;
    int grp = 0;
    GroupPlan gp = {};
    int64_t per_head = 1;
    int64_t gp_end = -1;  // cost up to the end of the group in gp
    for (;;) {
      Piece u;
      // The run has the steps that begin in [x0, x1).
      bool have = false;
      while (x < x1) {
        if (x >= gp_end) {
          // The group at x: the last one that begins there or before.
          int lo = grp, hi = p.num_groups;
          while (hi - lo > 1) {
            const int stride = (hi - lo + 31) / 32;
            const int at = lo + lane * stride;
            const bool before = at < hi && groups[at].cost0 <= x;
            const int k = __popc(__ballot_sync(0xffffffffu, before));
            const int from = lo + (k - 1) * stride;
            hi = min(hi, from + stride);
            lo = from;
          }
          grp = lo;
          const int4 a = reinterpret_cast<const int4 *>(groups + grp)[0];
          const int4 b = reinterpret_cast<const int4 *>(groups + grp)[1];
          gp.cost0 = (int64_t)(uint32_t)a.x | ((int64_t)a.y << 32);
          gp.start = a.z;
          gp.lead = a.w;
          gp.members = b.x;
          gp.tiles = b.y;
          per_head = head_cost(gp, p.group_size);
          gp_end = gp.cost0 + per_head * p.num_kv_heads;
        }
        u.kvh = (int)quotient(x - gp.cost0, per_head);
        const int64_t head0 = gp.cost0 + u.kvh * per_head;
        u.pair = (int)quotient(x - head0, full_unit_cost(gp));
        const int64_t step0 = head0 + u.pair * full_unit_cost(gp) + kUnitCost;
        u.rows = min(kPairRows, gp.members * p.group_size - u.pair * kPairRows);
        const int each = step_cost(u.rows);
        u.tile = x <= step0 ? 0 : (int)quotient(x - step0 + each - 1, each);
        const int end = x1 <= step0 ? 0 : (int)min((int64_t)gp.tiles, quotient(x1 - step0 + each - 1, each));
        u.n = end - u.tile;
        u.start = gp.start;
        u.lead = gp.lead;
        u.first = u.tile == 0;
        u.once = gp.members * p.group_size <= kPairRows;
        x = step0 + (int64_t)end * each;
        if (u.n > 0) {
          have = true;
          break;
        }
      }
      if (!have) u.start = -1;
      const int slot = iu % kUnitSlots;
      if (iu >= kUnitSlots)
        ok = warp_wait(&unit_empty[slot], ((iu / kUnitSlots) - 1) & 1, abort_flag);
      if (!ok) break;
      if (lane == 0) {
        ring[slot] = u;
        mbar_arrive(&unit_full[slot]);  // (release: orders the stores above)
      }
      ++iu;
      if (!have || !loads) break;
      if (lane == 0) {
        const int32_t *row = p.block_tables + (int64_t)u.lead * p.max_blocks_per_seq;
        int blk = row[u.tile * BN >> p.block_shift];  // (asked for ahead of Q)
        // Q of this piece once the last one's S products are done with it.
        if (iu >= 2) ok = mbar_wait_bounded(q_empty, (iu - 2) & 1, abort_flag);
        if (ok) {
          ++q_loads;
          const int each = u.rows > BM ? 2 : 1;
          mbar_arrive_expect_tx(q_full, each * L::kQBytes);
          for (int h = 0; h < each; ++h)
            for (int xr = 0; xr < XR; ++xr)
              tma_load_3d(sQ + h * L::kQBytes + xr * BM * 128, &tm_q, q_full, xr * 64,
                          u.kvh * p.group_size,
                          u.start + (u.pair * kPairRows + h * BM) / p.group_size);
        }
        for (int i = 0; i < u.n && ok; ++i, ++g) {
          const int st = g % kKStages;
          if (g >= kKStages && !mbar_wait_bounded(&k_empty[st], ((g / kKStages) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const int key0 = (u.tile + i) * BN;
          const int off = key0 & ((1 << p.block_shift) - 1);
          if (i > 0 && off == 0) blk = row[key0 >> p.block_shift];
          int from = blk;
          if (from < 0 || (int64_t)from >= p.num_blocks) {
            flag_status(p.status, PKV_DEV_BAD_BLOCK);
            from = 0;
          }
          mbar_arrive_expect_tx(&k_full[st], L::kKVBytes);
          for (int xr = 0; xr < XR; ++xr)
            tma_load_4d_hint(sK + st * L::kKVBytes + xr * BN * 128, &tm_k, &k_full[st], xr * 64,
                             u.kvh, off, from, u.once ? once : again);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      g = __shfl_sync(0xffffffffu, g, 0);
      if (!ok) break;
    }
    if (lane == 0) {
      // Do not leave while copies into this CTA's shared memory are in flight.
      if (q_loads > 0 && !mbar_wait_bounded(q_full, (q_loads - 1) & 1, nullptr))
        flag_status(p.status, PKV_DEV_TIMEOUT);
      for (int i = max(0, g - kKStages); i < g; ++i)
        if (!mbar_wait_bounded(&k_full[i % kKStages], (i / kKStages) & 1, nullptr))
          flag_status(p.status, PKV_DEV_TIMEOUT);
    }
  } else if (warp == kVWarp) {
    // Warp 2 copies V with cp.async, a second load path beside the SM's TMA unit, in the
    // swizzle that TMA would write.  Copies of up to kAhead steps are in flight; a step's
    // are made visible to the tensor cores' proxy and published when they are in.
    constexpr int kAhead = kVStages - 2;
    constexpr int kChunks = D / 8;          // 16-byte chunks of a row
    constexpr int kRowsPer = 32 / kChunks;  // rows per warp-wide copy
    const int col = lane % kChunks, row0 = lane / kChunks;
    const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
    int iu = 0, g = 0, published = 0;
    bool ok = true;
    Piece u;
    auto publish = [&]() {  // the oldest step that is not, whose copies are in
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[published % kVStages]);
      ++published;
    };
    while (ok && next_piece(iu, u)) {
      const int32_t *row = p.block_tables + (int64_t)u.lead * p.max_blocks_per_seq;
      int blk = row[u.tile * BN >> p.block_shift];
      for (int i = 0; i < u.n; ++i, ++g) {
        const int st = g % kVStages;
        if (g >= kVStages) ok = warp_wait(&v_empty[st], ((g / kVStages) - 1) & 1, abort_flag);
        if (!ok) break;
        const int key0 = (u.tile + i) * BN;
        const int off = key0 & ((1 << p.block_shift) - 1);
        if (i > 0 && off == 0) blk = row[key0 >> p.block_shift];
        const int64_t from = blk < 0 || (int64_t)blk >= p.num_blocks ? 0 : blk;  // (flagged by warp 0)
        const uint16_t *src =
            p.v_cache + ((((from << p.block_shift) + off + row0) * p.num_kv_heads + u.kvh) * D + col * 8);
        const int64_t step = (int64_t)kRowsPer * p.num_kv_heads * D;
        const uint32_t dst = smem_u32(sV) + st * L::kKVBytes + (col >> 3) * BN * 128;
#pragma unroll 8
        for (int r = 0; r < BN / kRowsPer; ++r) {
          const int at = row0 + r * kRowsPer;
          copy16(dst + at * 128 + (((col & 7) ^ (at & 7)) << 4), src + r * step, true, u.once ? once : again);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (g - published >= kAhead) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
          publish();
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (ok)
        while (published < g) publish();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp == kSWarp || warp == kPVWarp) {
    // Issuers: warp 1 S = Q K^T, warp 3 O += P V.  gh[h]: steps of chain h so far, uh[h]:
    // pieces of which it had any.  All of the warp goes through the steps and an elected
    // thread issues, so that addresses and descriptors are the warp's (with one thread's a
    // product took 100 cycles to issue, more than to compute).
    int iu = 0, g = 0;
    int gh[2] = {0, 0}, uh[2] = {0, 0};
    bool ok = true;
    Piece u;
    if (warp == kSWarp) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(BM, BN, false, false);
      const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = umma_desc_sw128(smem_u32(sK), 16, 1024);
      while (ok && next_piece(iu, u)) {
        const bool both = warp_same(u.rows) > BM;
        const int n = warp_same(u.n);
        ok = warp_wait(q_full, (iu - 1) & 1, abort_flag);
        for (int i = 0; i < n && ok; ++i, ++g) {
          const int st = g % kKStages;
          ok = warp_wait(&k_full[st], (g / kKStages) & 1, abort_flag);
          const uint64_t dk_st = dk + (uint64_t)((st * L::kKVBytes) >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!ok) break;
            if (!both && h != (i & 1)) continue;
            const int gt = gh[h] + (both ? i : i >> 1), b = gt & 1;
            if (gt >= 2) ok = warp_wait(&p_free[2 * h + b], ((gt - 2) >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem + kSCol + (2 * h + b) * BN;
            const uint64_t dq_h = dq + (uint64_t)((both ? h * L::kQBytes : 0) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk & 3) * 32;
                umma_bf16(d, dq_h + (uint64_t)(((kk / 4) * BM * 128 + off) >> 4),
                          dk_st + (uint64_t)(((kk / 4) * BN * 128 + off) >> 4), idesc_s,
                          kk > 0 ? 1u : 0u);
              }
              umma_commit(&s_full[2 * h + b]);
            }
            __syncwarp();
          }
          if (ok && elect_one()) umma_commit(&k_empty[st]);
          __syncwarp();
        }
        if (ok && elect_one()) umma_commit(q_empty);
        __syncwarp();
        gh[0] += both ? n : (n + 1) >> 1;
        gh[1] += both ? n : n >> 1;
      }
    } else {
      constexpr uint32_t idesc_o = umma_idesc_bf16(BM, D, false, true);
      const uint64_t dv = umma_desc_sw128(smem_u32(sV), BN * 128, 1024);
      while (ok && next_piece(iu, u)) {
        const bool both = warp_same(u.rows) > BM;
        const int n = warp_same(u.n);
        for (int i = 0; i < n && ok; ++i, ++g) {
          const int st = g % kVStages;
          ok = warp_wait(&v_full[st], (g / kVStages) & 1, abort_flag);
          const uint64_t dv_st = dv + (uint64_t)((st * L::kKVBytes) >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!ok) break;
            if (!both && h != (i & 1)) continue;
            const int ih = both ? i : i >> 1;  // the chain's own number of the step
            const int gt = gh[h] + ih, b = gt & 1;
            ok = warp_wait(&p_full[2 * h + b], (gt >> 1) & 1, abort_flag);
            if (ok && ih == 0 && uh[h] >= 1) ok = warp_wait(&o_free[h], (uh[h] - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t pa = tmem + kSCol + (2 * h + b) * BN;
            const uint32_t onto = ih > 0 ? 1u : 0u;
            // Both terms of P: columns 0-31 and 32-63 of the buffer.
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BN / 8; ++kk)
                umma_bf16_tmem_a(tmem + h * D, pa + kk * 8,
                                 dv_st + (uint64_t)(((kk % (BN / 16)) * 16 * 128) >> 4), idesc_o,
                                 kk > 0 ? 1u : onto);
              umma_commit(&p_free[2 * h + b]);
            }
            __syncwarp();
          }
          if (ok && elect_one()) umma_commit(&v_empty[st]);
          __syncwarp();
        }
        for (int h = 0; h < 2; ++h) {
          const int m = both ? n : (n + 1 - h) >> 1;
          gh[h] += m;
          uh[h] += m > 0 ? 1 : 0;
        }
      }
    }
    // Wait for the products of both issuers before tensor memory is freed.
    if (elect_one()) umma_commit(drain);
    if (lane == 0 && !mbar_wait_bounded(drain, 0, nullptr)) flag_status(p.status, PKV_DEV_TIMEOUT);
  } else {
    // Softmax: four warps per chain, a thread per row (chain 0: warps 4, 5, 10, 11).
    const int h = (((warp - 4) >> 1) ^ ((warp - 4) >> 2)) & 1;
    const int quarter = warp & 3;   // tensor memory lanes this warp may access
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float qs = p.qscale;
    const int Hq = p.num_kv_heads * p.group_size;
    int iu = 0, turn = 0;
    int gh[2] = {0, 0};  // steps of the chains before this piece
    bool ok = true;
    Piece u;
    while (ok && next_piece(iu, u)) {
      const bool both = u.rows > BM;
      const int n = chain_steps(u, h);
      // A warp whose rows all lie behind the piece's skips the arithmetic.
      const int row0 = both ? h * BM : 0;
      const bool live = row0 + quarter * 32 < u.rows;
      // Running max in log2 units, raised (and O rescaled) only when a step's exceeds it
      // by more than 8: P stays <= 2^8, and l and O share the reference.
      float m_ref = -INFINITY, l_run = 0.f;
      for (int i = 0; i < n && ok; ++i) {
        const int gt = gh[h] + i, b = gt & 1;
        const uint32_t sp = tmem + lane_base + kSCol + (2 * h + b) * BN;
        ok = warp_wait(&s_full[2 * h + b], (gt >> 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        float alpha = 1.f, rs = 0.f;
        if (live) {
          float sv[BN], mt;
          if (qs > 0.f) {
            tmem_load64_max(sp, sv, mt);
          } else {
            tmem_load64(sp, sv);
            mt = sv[0];
#pragma unroll
            for (int c = 1; c < BN; ++c) mt = fminf(mt, sv[c]);
          }
          mt *= qs;
          if (i == 0 || mt > m_ref + 8.f) {
            const float m_new = fmaxf(m_ref, mt);
            alpha = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m_new);
            m_ref = m_new;
          }
          // (a maximum of -inf: every weight so far is zero, whatever the reference)
          const float ref = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 q2 = make_float2(qs, qs), nm2 = make_float2(-ref, -ref);
          const float2 up2 = make_float2(kAboveCut, kAboveCut);
          float2 r01 = make_float2(0.f, 0.f), r23 = make_float2(0.f, 0.f);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float hi[16], lo[16];
#pragma unroll
            for (int c = hf * 32; c < hf * 32 + 32; c += 4) {
              const float2 x01 = __ffma2_rn(make_float2(sv[c], sv[c + 1]), q2, nm2);
              const float2 x23 = __ffma2_rn(make_float2(sv[c + 2], sv[c + 3]), q2, nm2);
              const float2 p01 = make_float2(fast_exp2(x01.x), fast_exp2(x01.y));
              const float2 p23 = make_float2(fast_exp2(x23.x), fast_exp2(x23.y));
              r01 = __fadd2_rn(r01, p01);
              r23 = __fadd2_rn(r23, p23);
              const uint32_t h01 = cut_bf16x2(p01.x, p01.y), h23 = cut_bf16x2(p23.x, p23.y);
              const int w = (c - hf * 32) / 2;
              hi[w] = __uint_as_float(h01);
              hi[w + 1] = __uint_as_float(h23);
              // (rest_bf16x2, two at a time)
              const float2 d01 = __ffma2_rn(p01, up2, make_float2(-bf16lo(h01), -bf16hi(h01)));
              const float2 d23 = __ffma2_rn(p23, up2, make_float2(-bf16lo(h23), -bf16hi(h23)));
              lo[w] = __uint_as_float(pack_bf16x2(d01.x, d01.y));
              lo[w + 1] = __uint_as_float(pack_bf16x2(d23.x, d23.y));
            }
            tmem_store16_async(sp + hf * 16, hi);
            tmem_store16_async(sp + 32 + hf * 16, lo);
          }
          tmem_wait_st();
          rs = (r01.x + r01.y) + (r23.x + r23.y);
        }
        if (live && i > 0 && __any_sync(0xffffffffu, alpha < 1.f)) {
          // O is rescaled once the chain's last P.V has landed in it (the next waits for
          // this step's P).
          ok = warp_wait(&p_free[2 * h + ((gt - 1) & 1)], ((gt - 1) >> 1) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            float ov[32];
            const uint32_t oa = tmem + lane_base + h * D + cc * 32;
            tmem_load32(oa, ov);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] *= alpha;
            tmem_store32(oa, ov);
          }
        }
        l_run = l_run * alpha + rs;
        tc_fence_before_sync();
        mbar_arrive(&p_full[2 * h + b]);
      }
      if (!ok) break;

      // The piece's (max, sum, O) as a part, once its last P.V are in O.  Their barriers
      // cannot run ahead: a chain's next P.V waits until O has been read (o_free).
      gh[0] += chain_steps(u, 0);
      gh[1] += chain_steps(u, 1);
      const int other = both ? 0 : chain_steps(u, 1 - h);
      float a_mine = 1.f, a_other = 0.f;
      if (n > 0) {
        const int gl = gh[h] - 1;
        ok = warp_wait(&p_free[2 * h + (gl & 1)], (gl >> 1) & 1, abort_flag);
        if (!ok) break;
      }
      if (!both) {
        // Chains that took the steps in turn: the joint maximum, and a half of the dims for
        // each to add up and write.
        // (two places in turn: a warp may be at the next piece's end when another reads)
        float2 *mine = ex + ((turn & 1) * 2 + h) * BM, *its = ex + ((turn & 1) * 2 + 1 - h) * BM;
        mine[row] = make_float2(m_ref, l_run);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ex_full);
        ok = warp_wait(ex_full, turn & 1, abort_flag);
        if (!ok) break;
        ++turn;
        const float2 x = its[row];
        const float M = fmaxf(m_ref, x.x), ref = M == -INFINITY ? 0.f : M;
        a_mine = fast_exp2(m_ref - ref);
        a_other = fast_exp2(x.x - ref);
        l_run = l_run * a_mine + x.y * a_other;
        m_ref = M;
      }
      // (the other chain's last P.V is in, too: its warps have waited for it)
      tc_fence_after_sync();
      const int r = row0 + row;
      if (live) {
        const int idx = u.pair * kPairRows + r;  // of the group's rows
        const int64_t at = u.first ? (int64_t)(u.start + idx / p.group_size) * Hq +
                                         u.kvh * p.group_size + idx % p.group_size
                                   : (int64_t)blockIdx.x * kPairRows + r;
        // (eight dims of a row at a time: the same with eight dims of all rows together,
        // whose stores fill whole lines, ended a piece 0.5 us sooner and the join 1.5 later;
        // rows turned through shared memory into whole lines took 1 us more)
        float *o = (u.first ? p.first_o : p.run_o) + at * D;
        const int c0 = both ? 0 : h * (D / 2), c1 = both ? D : c0 + D / 2;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          float ov[32], v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0.f;
          if (n > 0) tmem_load32(tmem + lane_base + h * D + c, ov);
          if (!both) {
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] *= a_mine;
            if (other > 0) {
              tmem_load32(tmem + lane_base + (1 - h) * D + c, v);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = fmaf(v[e], a_other, ov[e]);
            }
          }
          if (r < u.rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(o + c + e, ov, e);
          }
        }
        if (r < u.rows && (both || h == 0))
          reinterpret_cast<float2 *>(u.first ? p.first_ml : p.run_ml)[at] = make_float2(m_ref, l_run);
      }
      // O has been read: of its own chain, or of both that had steps.
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (both || n > 0) mbar_arrive(&o_free[h]);
        if (both) mbar_arrive(&o_free[h]);
        if (!both && other > 0) mbar_arrive(&o_free[1 - h]);
      }
    }
    tc_fence_before_sync();
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(p.status, PKV_DEV_TIMEOUT);
  if (warp == kSWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// The launch of both.
template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1)
    shared_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const SharedParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  // (before any of tensor memory is taken, too)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const GroupPlan *groups = p.groups;
  if (p.num_groups <= kNearGroups) {  // (asked for beside the totals; read behind a barrier)
    GroupPlan *near = reinterpret_cast<GroupPlan *>(smem_raw + p.groups_at);
    if (threadIdx.x < 2 * p.num_groups)
      reinterpret_cast<int4 *>(near)[threadIdx.x] =
          __ldcg(reinterpret_cast<const int4 *>(p.groups) + threadIdx.x);
    groups = near;
  }
  Totals sum;
  sum.cost = __ldcg(&p.totals->cost);
  sum.run_cost = __ldcg(&p.totals->run_cost);
  sum.tiles = __ldcg(&p.totals->tiles);
  sum.run_tiles = __ldcg(&p.totals->run_tiles);
  sum.prefix_ctas = __ldcg(&p.totals->prefix_ctas);
  if ((int)blockIdx.x < sum.prefix_ctas) {
    prefixes<D>(tm_q, tm_k, p, sum, groups, smem_raw);
    return;
  }
  int *tile0 = reinterpret_cast<int *>(smem_raw + p.tail_warps * WarpSmem<D, G>::bytes);
  int *begin = tile0 + p.num_seqs + 1, *len = begin + p.num_seqs;
  for (int s = threadIdx.x; s < p.num_seqs; s += blockDim.x) {
    const int4 x = __ldcg(reinterpret_cast<const int4 *>(p.seqs + s));
    tile0[s] = x.x;
    begin[s] = x.y;
    len[s] = x.z;
  }
  if (threadIdx.x == 0) tile0[p.num_seqs] = sum.tiles;
  __syncthreads();
  tails<D, G, false>(p, sum, smem_raw, 0, 0, nullptr);
}

// What the groups say is looked at, but not used, where nothing is shared.
__device__ __forceinline__ void check_groups(const SharedParams &p) {
  for (int g = threadIdx.x; g <= p.num_groups; g += blockDim.x) {
    const int x = p.group_starts[g];
    if (g < p.num_groups ? (g == 0 && x != 0) || p.group_starts[g + 1] < x : x != p.num_seqs)
      flag_status(p.status, PKV_DEV_BAD_SEQLEN);
    if (g < p.num_groups && (p.shared_blocks[g] < 0 || p.shared_blocks[g] > p.max_blocks_per_seq))
      flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  }
}

// The launch of a small batch: every context is a tail, of which each CTA knows by itself
// where it begins.
template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) shared_small_kernel(const SharedParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int64_t sums[32][1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int S = p.num_seqs, s = threadIdx.x;  // (kSmallSeqs: a thread each)
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  int *tile0 = reinterpret_cast<int *>(smem_raw + p.tail_warps * WarpSmem<D, G>::bytes);
  int *begin = tile0 + S + 1, *len = begin + S;
  const int given = s < S ? p.context_lens[s] : 1;
  const int L = given <= 0 ? 0 : (int)min((int64_t)given, room);
  if (blockIdx.x == 0) {
    if (s < S && (L != given || L == 0)) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    check_groups(p);
  }
  int64_t at[1] = {s < S ? tail_tiles(L, D) : 0}, all[1];
  scan_cta<1>(at, all, sums);
  Totals sum;
  sum.cost = 0;
  sum.tiles = (int)all[0];
  sum.prefix_ctas = 0;
  cut_runs(p, sum);
  if (s < S) {
    tile0[s] = (int)at[0];
    begin[s] = 0;
    len[s] = L;
    if (blockIdx.x == 0)
      p.joins[s] = join_plan(sum, s, (int)at[0], tail_tiles(L, D), 0, GroupPlan{}, true);
  }
  if (s == 0) tile0[S] = (int)all[0];
  __syncthreads();
  tails<D, G, false>(p, sum, smem_raw, 0, 0, nullptr);
}

// The launch of a batch whose contexts are short, all of it: a CTA for each sequence and kv
// head, whose warps share the tiles; their parts are joined in shared memory.
template <int D, int G>
__global__ void __launch_bounds__(kWarpsMost * 32, 1) shared_short_kernel(const SharedParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warps = p.tail_warps, seq = blockIdx.x / p.num_kv_heads, kvh = blockIdx.x - seq * p.num_kv_heads;
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  const int given = p.context_lens[seq];
  const int L = given <= 0 ? 0 : (int)min((int64_t)given, room);
  if (kvh == 0 && threadIdx.x == 0 && (L != given || L == 0)) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  if (blockIdx.x == 0) check_groups(p);
  if (L == 0) return;  // (left as it was)
  uint8_t *behind = smem_raw + warps * WarpSmem<D, G>::bytes;
  int *one = reinterpret_cast<int *>(behind);  // (see tails)
  float *parts = reinterpret_cast<float *>(behind + 16);
  if (threadIdx.x == 0) {
    one[0] = one[2] = 0;
    one[1] = tail_tiles(L, D);
    one[3] = L;
  }
  __syncthreads();
  tails<D, G, true>(p, Totals{}, smem_raw, seq, kvh, parts);
  __syncthreads();
  const float2 *ml = reinterpret_cast<const float2 *>(parts + warps * G * D);
  const int tiles = tail_tiles(L, D), per_run = (tiles + warps - 1) / warps;
  const int n = (tiles + per_run - 1) / per_run;
  for (int i = threadIdx.x * 2; i < G * D; i += blockDim.x * 2) {
    const int row = i / D, d = i % D;
    float M = -INFINITY;
    for (int w = 0; w < n; ++w) M = fmaxf(M, ml[w * G + row].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float l = 0.f, a = 0.f, b = 0.f;
    for (int w = 0; w < n; ++w) {
      const float2 x = ml[w * G + row];
      const float2 o = *reinterpret_cast<const float2 *>(parts + (w * G + row) * D + d);
      const float weight = fast_exp2(x.x - ref);
      l = fmaf(x.y, weight, l);
      a = fmaf(o.x, weight, a);
      b = fmaf(o.y, weight, b);
    }
    const float inv = 1.f / l;
    *reinterpret_cast<uint32_t *>(p.out + (((int64_t)seq * p.num_kv_heads + kvh) * G + row) * D + d) =
        pack_bf16x2(a * inv, b * inv);
  }
}

// ----------------------------------------------------------------------- 4. join

// A row (sequence, query head) is joined by kShare of a CTA's four warps, which take its
// parts in turn, a lane four (D = 64: two) of the D values.
template <int D, int kShare>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_kernel(const SharedParams p) {
  constexpr int kEach = D / 32, kRows = kJoinWarps / kShare;
  constexpr int kAhead = 8;  // parts asked for at a time
  __shared__ float acc_s[kJoinWarps][D];
  __shared__ float2 ml_s[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % kShare;
  const int Hkv = p.num_kv_heads, G = p.group_size, Hq = Hkv * G;
  const int64_t rows = (int64_t)p.num_seqs * Hq;
  const int64_t row = (int64_t)blockIdx.x * kRows + warp / kShare;
  const int s = (int)(min(row, rows - 1) / Hq), head = (int)(min(row, rows - 1) - (int64_t)s * Hq);
  const int j = head / G, g = head - j * G;
  // (Planned by a launch of its own, the plan is there: the launch before began after it,
  // and this one after that.)
  if (p.small) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 *plan = reinterpret_cast<const int4 *>(p.joins + s);
  const int4 a = __ldcg(plan), b = __ldcg(plan + 1), c = __ldcg(plan + 2);
  // The parts of the tail: of runs r0, r0 + 1, ...
  const int n_tail = a.y;
  const int64_t tail_row = ((int64_t)a.x * Hkv + j) * G + g;
  // Those of the prefix: of the unit that has the row, its first step's and of the runs
  // behind that one.
  int n_pre = 0;
  int64_t run_row = 0;
  if (b.x > 0) {
    GroupPlan gp = {};
    gp.members = a.w;
    gp.tiles = b.x;
    gp.cost0 = (int64_t)(uint32_t)b.z | ((int64_t)b.w << 32);
    const int64_t len = (int64_t)(uint32_t)c.x | ((int64_t)c.y << 32);
    const int idx = a.z * G + g, pair = idx / kPairRows;
    const int64_t step0 = gp.cost0 + j * head_cost(gp, G) + pair * full_unit_cost(gp) + kUnitCost;
    const int each = step_cost(gp.members * G - pair * kPairRows);
    const int64_t c0 = quotient(step0, len);
    run_row = c0 * kPairRows + idx % kPairRows;
    n_pre = (int)(quotient(step0 + (int64_t)(gp.tiles - 1) * each, len) - c0 + 1);
  }
  const int n = row < rows ? n_tail + n_pre : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // A warp's parts: 32 of their maxima at a time, a lane each.
  float m = -INFINITY, l = 0.f;
  float acc[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
  for (int base = share; base < n; base += 32 * kShare) {
    int i = base + lane * kShare;
    const int count = min(32, (n - base + kShare - 1) / kShare);
    float2 x = make_float2(-INFINITY, 0.f);
    const float *o = p.tail_o;
    if (i < n) {  // part i: its row of its kind's arrays
      const float *ml = p.tail_ml;
      int64_t at = tail_row + (int64_t)i * Hkv * G;
      i -= n_tail;
      if (i >= 0) {
        ml = i == 0 ? p.first_ml : p.run_ml;
        o = i == 0 ? p.first_o : p.run_o;
        at = i == 0 ? row : run_row + (int64_t)i * kPairRows;
      }
      x = __ldcg(reinterpret_cast<const float2 *>(ml) + at);
      o += at * D;
    }
    float mn = x.x;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, k));
    mn = fmaxf(mn, m);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float old = fast_exp2(m - ref), w = fast_exp2(x.x - ref);
    float lw = x.y * w;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, k);
    l = l * old + lw;
    m = mn;
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc[e] *= old;
    for (int k0 = 0; k0 < count; k0 += kAhead) {
      float y[kAhead][kEach];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float *from = reinterpret_cast<const float *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), (k0 + u) & 31));
#pragma unroll
        for (int e = 0; e < kEach; ++e) y[u][e] = 0.f;
        if (k0 + u < count) {
          if constexpr (kEach == 4)
            *reinterpret_cast<float4 *>(y[u]) = __ldcg(reinterpret_cast<const float4 *>(from) + lane);
          else
            *reinterpret_cast<float2 *>(y[u]) = __ldcg(reinterpret_cast<const float2 *>(from) + lane);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + u) & 31);
        if (k0 + u < count) {
#pragma unroll
          for (int e = 0; e < kEach; ++e) acc[e] = fmaf(wk, y[u][e], acc[e]);
        }
      }
    }
  }
  // The sums of a row's warps.
  float M = m;
  if constexpr (kShare > 1) {
    if (lane == 0) ml_s[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc_s[warp][lane * kEach + e] = acc[e];
    __syncthreads();
    if (share != 0) return;
#pragma unroll
    for (int w = 1; w < kShare; ++w) M = fmaxf(M, ml_s[warp + w].x);
    const float ref = M == -INFINITY ? 0.f : M;
    const float a0 = fast_exp2(m - ref);
    l *= a0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc[e] *= a0;
#pragma unroll
    for (int w = 1; w < kShare; ++w) {
      const float2 y = ml_s[warp + w];
      const float a = fast_exp2(y.x - ref);
      l = fmaf(y.y, a, l);
#pragma unroll
      for (int e = 0; e < kEach; ++e) acc[e] = fmaf(acc_s[warp + w][lane * kEach + e], a, acc[e]);
    }
  }
  if (n == 0) return;  // (no such row, or an empty context: left as it was)
  const float inv = 1.f / l;
  uint16_t *out = p.out + row * D + lane * kEach;
  if constexpr (kEach == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                 pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

// ------------------------------------------------------------------------- host

// Test-only, set by pkv_test_shared_fault: SharedParams::loading and share_always of the
// process's calls.
std::atomic<int> g_loading{kMaxCtas};
std::atomic<int> g_share_always{0};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
  size_t totals, groups, seqs, joins, tail_ml, tail_o, first_ml, first_o, run_ml, run_o, total;
  Workspace(int64_t S, int64_t N, int64_t Hq, int64_t Hkv, int64_t D) {
    const int64_t parts = S * Hq + (kMaxWarps + Hkv) * (Hq / Hkv);  // (num_seqs + runs) of each head
    totals = 0;
    groups = 256;
    seqs = groups + align256((size_t)N * sizeof(GroupPlan));
    joins = seqs + align256((size_t)S * sizeof(SeqPlan));
    tail_ml = joins + align256((size_t)S * sizeof(JoinPlan));
    tail_o = tail_ml + align256((size_t)parts * 8);
    first_ml = tail_o + align256((size_t)(parts * D) * 4);
    first_o = first_ml + align256((size_t)(S * Hq) * 8);
    run_ml = first_o + align256((size_t)(S * Hq * D) * 4);
    run_o = run_ml + align256((size_t)kMaxCtas * kPairRows * 8);
    total = run_o + align256((size_t)(kMaxCtas * kPairRows * D) * 4);
  }
};

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, unsigned threads, int smem,
                             cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// q as {D, Hq, S}: a box is 64 dims x the G heads of a kv head x 128 / G sequences.
// k_cache as {D, Hkv, block_size, NB}: a box is 64 dims x 1 head x 64 tokens x 1 block.
bool encode_maps(const SharedParams &p, CUtensorMap *tq, CUtensorMap *tk) {
  const uint64_t D = p.head_dim, Hkv = p.num_kv_heads, Hq = Hkv * p.group_size;
  const uint64_t block = (uint64_t)1 << p.block_shift;
  const uint64_t qdims[3] = {D, Hq, (uint64_t)p.num_seqs}, qstr[2] = {D * 2, Hq * D * 2};
  const uint32_t qbox[3] = {64u, (uint32_t)p.group_size, (uint32_t)(BM / p.group_size)};
  const uint64_t kdims[4] = {D, Hkv, block, (uint64_t)p.num_blocks};
  const uint64_t kstr[3] = {D * 2, Hkv * D * 2, block * Hkv * D * 2};
  const uint32_t kbox[4] = {64u, 1u, (uint32_t)BN, 1u};
  return encode_bf16_map(tq, p.q, 3, qdims, qstr, qbox, true) &&
         encode_bf16_map(tk, p.k_cache, 4, kdims, kstr, kbox, true);
}

template <int D, int G>
pkv_status launch(SharedParams prm, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  const int S = prm.num_seqs;
  const int64_t room = (int64_t)prm.max_blocks_per_seq << prm.block_shift;
  const bool small = S <= kSmallSeqs && S * room * prm.num_kv_heads * (4 * D) <= kSmallBytes &&
                     !prm.share_always;
  if (room <= (G == 8 ? kShortTokens / 2 : kShortTokens) &&
      (int64_t)S * prm.num_kv_heads <= kShortCtas * sms && !prm.share_always) {
    constexpr int each = WarpSmem<D, G>::bytes + G * (D * 4 + 8);  // of a warp, with its part
    constexpr int fit = (kMaxDynamicSmem - 16) / each;
    prm.tail_warps = fit < kWarpsMost ? fit : kWarpsMost;
    prm.ctas = S * prm.num_kv_heads;
    const int smem = prm.tail_warps * each + 16;
    if (!kernel_smem_setup((const void *)shared_short_kernel<D, G>, prm.tail_warps * 32, smem, nullptr))
      return PKV_ERR_CUDA;
    launch_dependent<SharedParams>(shared_short_kernel<D, G>, (unsigned)prm.ctas, prm.tail_warps * 32, smem,
                                   stream, prm);
    return launch_status();
  }
  const int groups_smem = kNearGroups * (int)sizeof(GroupPlan) + 16;
  const int seq_smem = (3 * S + 1) * 4;
  int warps = (kMaxDynamicSmem - 2048 - seq_smem - groups_smem) / WarpSmem<D, G>::bytes;
  if (warps > kWarpsMost) warps = kWarpsMost;
  static_assert((kMaxDynamicSmem - 4096 - (3 * kSharedMaxSeqs + 1) * 4) / WarpSmem<D, G>::bytes >= 1, "");
  static_assert(kNearGroups * sizeof(GroupPlan) + 16 <= 2048, "");
  static_assert(PrefixLayout<D>::total + 1024 + 16 + kNearGroups * sizeof(GroupPlan) <= kMaxDynamicSmem, "");
  int smem = warps * WarpSmem<D, G>::bytes + seq_smem;
  if (!small && smem < PrefixLayout<D>::total + 1024) smem = PrefixLayout<D>::total + 1024;
  prm.small = small;
  prm.groups_at = (smem + 15) & ~15;
  if (!small) smem += groups_smem;
  const int plan_smem = ((4 * prm.num_groups + 2) & ~1) * 4 + prm.num_groups * 8;
  if (small ? !kernel_smem_setup((const void *)shared_small_kernel<D, G>, kThreads, smem, nullptr)
            : !kernel_smem_setup((const void *)shared_plan_kernel, kPlanThreads, plan_smem, nullptr) ||
                  !kernel_smem_setup((const void *)shared_attn_kernel<D, G>, kThreads, smem, nullptr))
    return PKV_ERR_CUDA;
  CUtensorMap tq, tk;
  if (!small && !encode_maps(prm, &tq, &tk)) return PKV_ERR_CUDA;
  // A CTA per SM, and no more than the longest possible batch has work for: a warp per
  // tile and kv head, a CTA per step of the prefixes.  (Two at least: one of a kind.)
  const int rows = tail_rows(D);
  const int64_t tiles = (int64_t)S * ((room + rows - 1) / rows) * prm.num_kv_heads;
  const int64_t pairs = (int64_t)S * G / kPairRows + (S + 1) / 2;  // of a kv head, at most
  const int64_t steps = pairs * prm.num_kv_heads * (room / BN);
  int64_t ctas = (tiles + warps - 1) / warps + steps;
  if (ctas > sms) ctas = sms;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  if (ctas < 2) ctas = 2;
  prm.ctas = (int)ctas;
  prm.tail_warps = warps;
  cudaError_t err;
  if (small) {
    err = launch_dependent<SharedParams>(shared_small_kernel<D, G>, (unsigned)ctas, kThreads, smem,
                                         stream, prm);
  } else {
    // (few sequences: fewer threads to wait for; 100 of them 22.4 -> 21.3 us, 1000 72.9 -> 77.3)
    err = launch_dependent<SharedParams>(shared_plan_kernel, 1, S <= 256 ? 256 : kPlanThreads,
                                         plan_smem, stream, prm);
    if (err == cudaSuccess)
      err = launch_dependent<CUtensorMap, CUtensorMap, SharedParams>(
          shared_attn_kernel<D, G>, (unsigned)ctas, kThreads, smem, stream, tq, tk, prm);
  }
  if (err == cudaSuccess) {
    // As many warps to a row as leave the join's CTAs one turn on the GPU (eight to an SM):
    // 1024 rows of about 20 parts took 6.7 us with one and 4.4 with two, 4096 of 6 the
    // other way round (two turns) 4.0 and 7.5.
    const int64_t rows = (int64_t)S * prm.num_kv_heads * G, room = 8 * (int64_t)sms;
    const int share = rows <= room ? 4 : rows <= 2 * room ? 2 : 1;
    const unsigned grid = (unsigned)((rows + kJoinWarps / share - 1) / (kJoinWarps / share));
    err = launch_dependent<SharedParams>(share == 4   ? shared_join_kernel<D, 4>
                                         : share == 2 ? shared_join_kernel<D, 2>
                                                      : shared_join_kernel<D, 1>,
                                         grid, kJoinWarps * 32, 0, stream, prm);
  }
  return launch_status();  // (any launch's error, which it clears)
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads,
                                                   int num_kv_heads, int head_dim) {
  using namespace pkv;
  if (num_seqs <= 0 || num_groups <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return 0;
  // (more sequences than any call takes: their bytes need not fit 64 bits)
  if (num_seqs > kSharedMaxSeqs || num_q_heads > (1 << 16) || head_dim > (1 << 16) ||
      num_q_heads < num_kv_heads)
    return 0;
  return Workspace(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim).total;
}

extern "C" pkv_status pkv_paged_decode_shared_attn(
    uint16_t *out, const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
    const int32_t *block_tables, const int32_t *context_lens, const int32_t *group_starts,
    const int32_t *shared_blocks, int num_seqs, int num_groups, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
    float scale, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_groups < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / num_kv_heads;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (G != 1 && G != 2 && G != 4 && G != 8) return PKV_ERR_UNSUPPORTED;
  if (block_size != 64 && block_size != 128 && block_size != 256 && block_size != 512)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs > kSharedMaxSeqs || num_kv_heads > 4096 ||
      (int64_t)max_blocks_per_seq * block_size > kMaxTokens)
    return PKV_ERR_UNSUPPORTED;
  // NaN or infinite, itself or in the exponentials' base 2 (a logit of zero would be NaN)
  if (!isfinite(scale * kLog2e)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (num_groups == 0 || num_groups > num_seqs) return PKV_ERR_INVALID_ARG;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !group_starts ||
      !shared_blocks)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  const size_t need = pkv_decode_shared_workspace_size(num_seqs, num_groups, num_q_heads,
                                                       num_kv_heads, head_dim);
  if (workspace == nullptr || workspace_bytes < need ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_WORKSPACE;

  const Workspace lay(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  SharedParams prm;
  prm.out = out;
  prm.q = q;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.context_lens = context_lens;
  prm.group_starts = group_starts;
  prm.shared_blocks = shared_blocks;
  prm.totals = reinterpret_cast<Totals *>(ws + lay.totals);
  prm.groups = reinterpret_cast<GroupPlan *>(ws + lay.groups);
  prm.seqs = reinterpret_cast<SeqPlan *>(ws + lay.seqs);
  prm.joins = reinterpret_cast<JoinPlan *>(ws + lay.joins);
  prm.tail_ml = reinterpret_cast<float *>(ws + lay.tail_ml);
  prm.tail_o = reinterpret_cast<float *>(ws + lay.tail_o);
  prm.first_ml = reinterpret_cast<float *>(ws + lay.first_ml);
  prm.first_o = reinterpret_cast<float *>(ws + lay.first_o);
  prm.run_ml = reinterpret_cast<float *>(ws + lay.run_ml);
  prm.run_o = reinterpret_cast<float *>(ws + lay.run_o);
  prm.status = dev_status;
  prm.num_blocks = num_blocks;
  prm.num_seqs = num_seqs;
  prm.num_groups = num_groups;
  prm.num_kv_heads = num_kv_heads;
  prm.group_size = G;
  prm.block_shift = 31 - __builtin_clz((unsigned)block_size);
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.ctas = 0;
  prm.tail_warps = 0;
  prm.small = 0;
  prm.groups_at = 0;
  prm.head_dim = head_dim;
  prm.loading = g_loading.load(std::memory_order_relaxed);
  prm.share_always = g_share_always.load(std::memory_order_relaxed);
  prm.qscale = scale * kLog2e;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define PKV_CASE(DD, GG) \
  if (head_dim == DD && G == GG) return launch<DD, GG>(prm, st);
  PKV_CASE(64, 1)
  PKV_CASE(64, 2)
  PKV_CASE(64, 4)
  PKV_CASE(64, 8)
  PKV_CASE(128, 1)
  PKV_CASE(128, 2)
  PKV_CASE(128, 4)
  PKV_CASE(128, 8)
#undef PKV_CASE
  return PKV_ERR_UNSUPPORTED;
}

extern "C" pkv_status pkv_test_shared_fault(int64_t wait_limit_ns, int loading_ctas, int share_always) {
  if (wait_limit_ns <= 0 || loading_ctas < -1) return PKV_ERR_INVALID_ARG;
  const unsigned long long limit = (unsigned long long)wait_limit_ns;
  if (cudaMemcpyToSymbol(pkv::g_wait_limit_ns, &limit, sizeof(limit)) != cudaSuccess)
    return PKV_ERR_CUDA;
  pkv::g_loading = loading_ctas >= 0 ? loading_ctas : pkv::kMaxCtas;
  pkv::g_share_always = share_always != 0;
  return PKV_OK;
}
