// decode_weights.cu -- paged decode attention that also collects key weights.
//
// One new token per sequence attends over its paged context, and the weight
// that each key receives, summed over the query heads of its kv head, is added
// to the key's running sum (the newest key's starts anew: its slot held another
// token's).  The weights need the softmax's denominator, which is known only
// when the whole context has been read, so the logits (4 G bytes a key and kv
// head, beside the 4 D bytes of its K and V) go through the workspace:
//
//  1. Split-K attention.  All tokens of the batch, sequence after sequence in
//     tiles, are cut into runs of equal length whatever the sequences' lengths;
//     a warp takes one run for one kv head.  Of every sequence in its run it
//     writes the logits (log2 units), and a part: their maximum and sum, and the
//     unnormalised output.  The run with a sequence's newest key clears its sum.
//  2. Join, a programmatic dependent launch: every CTA joins the maxima and sums
//     of a sequence's parts, then adds the weights of its own tokens to the sums
//     and writes its share of the output.
//
// Bound by HBM.  Measured: 64 sequences of 128 to 2048 tokens with their store
// (16 heads on 8, D = 128: 283 MB) 56 us, of which the first launch alone 50 to 55 at
// 5.2 to 5.6 TB/s (about 80 % of a copy); 64 skewed ones to 8192 tokens (594 MB) 110 us,
// 98 at 6.0 TB/s; two of 24 K to 33 K tokens (64 heads on 8: 236 MB) 52 us, 45 at 5.2
// TB/s.  What is above the reading is the second launch (11, 16 and 13 us alone, its
// caches cold): it starts when the last maximum is known.
#include <math.h>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kWarpsMost = 8;        // warps per CTA (one CTA per SM)
constexpr int kStages = 3;           // ring of tiles per warp
constexpr int kMaxSeqs = 16384;
constexpr int kMaxWarps = 4096;      // warps of a grid at most (places for parts)
constexpr int kShortTiles = 64;      // a sequence of so many tiles may have a run for each
constexpr int kMaxDynamicSmem = 232448;  // opt-in shared memory per CTA on sm_103 (227 KiB)
// Threads of the second launch's CTAs: fewer tokens each where a token has eight
// logits (registers; two long sequences 55.3 -> 54.1 us), more where it has few
// (a CTA's fixed work counts more; 64 skewed sequences 114 -> 109 us).
__host__ __device__ constexpr int join_threads(int G) { return G == 8 ? 256 : 128; }
constexpr int kJoinTokens = 1024;    // tokens that a CTA of the second launch takes at a time, at most
// CTAs of the second launch, about: the table may be far longer than the contexts,
// and past this many a CTA takes several parts of its sequence rather than the
// launch having one for every part that the table has room for.
constexpr int kJoinCtas = 16384;
constexpr int kJoinFill = 2;         // CTAs per SM that make smaller parts unnecessary
constexpr float kLog2e = 1.4426950408889634f;

struct WeightsParams {
  uint16_t *out;
  float *key_weights;
  const uint16_t *q;
  const uint16_t *k_cache;
  const uint16_t *v_cache;
  const int32_t *block_tables;
  const int32_t *context_lens;
  // Fused store (null unless the call also stores this step's tokens): row s
  // of new_k / new_v is the newest token of sequence s, to go to new_slots[s].
  const uint16_t *new_k;
  const uint16_t *new_v;
  const int32_t *new_slots;
  uint16_t *k_cache_w;
  uint16_t *v_cache_w;
  int32_t *tile_prefix;   // [num_seqs + 1]: first tile of each sequence
  float *part_ml;         // [num_seqs + runs, Hkv, G, 2]   (max in log2 units, sum)
  float *part_o;          // [num_seqs + runs, Hkv, D, G]
  float *logits;          // [tiles, Hkv, tile, G]
  int32_t *status;
  int64_t num_blocks;
  int64_t max_tiles;
  int num_seqs;
  int num_kv_heads;
  int block_shift;
  int runs;   // runs of the batch's tiles at most
  int join_tokens;  // tokens that a CTA of the second launch takes at a time
  int max_blocks_per_seq;
  float qscale;  // scale * log2(e)
};

// Visible tokens of a sequence: context_lens, at most what its table holds.
__device__ __forceinline__ int visible(const WeightsParams &p, int s) {
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  const int L = p.context_lens[s];
  return L <= 0 ? 0 : (int)min((int64_t)L, room);
}

// First tile of every sequence into prefix[0 .. S] (shared memory), by all
// threads; returns the number of tiles.  (Summed in 64 bits: lengths that the
// workspace has no room for may be any; the prefix holds for those that fit.)
template <int kRows>
__device__ int64_t scan_tiles(const WeightsParams &p, int *prefix, int64_t *warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs;
  const int per = (S + blockDim.x - 1) / blockDim.x;
  const int begin = min(tid * per, S), end = min(begin + per, S);
  int64_t local = 0;
  for (int s = begin; s < end; ++s) local += (visible(p, s) + kRows - 1) / kRows;
  int64_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int64_t run = incl - local, total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) run += warp_sums[w];
    total += warp_sums[w];
  }
  for (int s = begin; s < end; ++s) {
    prefix[s] = (int)run;
    run += (visible(p, s) + kRows - 1) / kRows;
  }
  if (tid == 0) prefix[S] = (int)total;
  __syncthreads();
  return total;
}

// The sequence that tile t belongs to (the last s with prefix[s] <= t).
__device__ __forceinline__ int seq_of(const int *prefix, int S, int t) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Tiles per run.  Run r has tiles [r * n, (r + 1) * n) of the batch; its part of
// sequence s is filed under s + r: every part begins where a sequence or a run
// does, so no two have the same number.  A run of one tile is the shortest way
// through the first launch, but the join reads a part for each: 2 sequences under
// 300 tokens 13.0 us with runs of four tiles and 10.9 with one; 4 sequences of 1000
// to 2000 tokens, two kv heads, 16.4 with two and 19.5 with one.
__device__ __forceinline__ int run_tiles(const WeightsParams &p, int tiles) {
  const int least = tiles > (int64_t)kShortTiles * p.num_seqs ? 2 : 1;
  return max((tiles + p.runs - 1) / p.runs, least);
}

// 16-byte asynchronous copy; zeros instead when !take.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool take, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(take ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// d (16 x 8, fp32) += a (16 x 16, bf16) * b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared memory of one warp: a ring of tiles (kRows tokens of K, then of V),
// and as many places for the query rows of the sequences in flight.
template <int D, int G>
struct WarpSmem {
  static constexpr int kRows = 2048 / D;          // 16 tokens of 128 dims, 32 of 64
  static constexpr int kHalf = kRows * D * 2;     // 4 KiB of K or V
  static constexpr int kQ = G * D * 2;
  static constexpr int bytes = kStages * (2 * kHalf + kQ);
};

// Byte offset of 16-byte column c of row r in a tile of rows of D values: the
// columns of eight consecutive rows are spread over the banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// First launch.  A warp is by itself: it streams the K and V of its run, for its
// kv head, through its own ring with cp.async, up to two tiles ahead and across
// sequences, so nothing in the loop waits for another warp; the warps of the
// other kv heads of the same tokens run beside it (whole rows of the cache are
// read at about the same time).  Per 16 tokens the products are m16n8k16: S = K q^T
// (tokens x dims x heads; the G heads of the group are the columns, of 8) and
// O^T += V^T P (dims x tokens x heads), in which a lane's two heads are the
// same in S, in P and in O, so maximum and rescaling need no exchange of O.
// Decode moves D * 4 bytes for 4 G D operations, far below what these products
// run at: the loop is there to keep loads in flight (128 KB per SM).
//
// P is an operand in bf16: it goes in as the sum of two, its rounding and what
// that leaves, so that a weight is off by 2^-18 of itself and not by 2^-9 (the
// attention of paged_decode_attn keeps it in fp32; the outputs of the two then
// differ by their own rounding alone).  A group of at most four heads has columns
// to spare: columns 4 to 7 repeat the heads of 0 to 3 and take the second parts,
// and the two halves of O are added at the end.  Eight heads need a second product.
template <int D, int G>
__global__ void __launch_bounds__(kWarpsMost * 32, 1) decode_weights_kernel(const WeightsParams p) {
  using W = WarpSmem<D, G>;
  constexpr int kRows = W::kRows;
  constexpr int kCols = D / 8;              // 16-byte columns per row
  constexpr int kRowsPer = 32 / kCols;      // rows per warp-wide copy
  constexpr int kSlices = kRows / 16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int64_t warp_sums[kWarpsMost];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  uint8_t *mine = smem_raw + warp * W::bytes;
  int *prefix = reinterpret_cast<int *>(smem_raw + warps * W::bytes);  // [S + 1]
  const uint32_t tiles = smem_u32(mine);
  const uint32_t qslots = tiles + kStages * 2 * W::kHalf;
  const int S = p.num_seqs, Hkv = p.num_kv_heads, shift = p.block_shift;

  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the kernel before the call)
  const int64_t all = scan_tiles<kRows>(p, prefix, warp_sums);
  const bool over = all > p.max_tiles;
  const int total = (int)all;
  if (blockIdx.x == 0) {
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
      const int L = p.context_lens[s];
      if (L <= 0 || L != visible(p, s)) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    }
    if (over && threadIdx.x == 0) flag_status(p.status, PKV_DEV_WORKSPACE);
    for (int s = threadIdx.x; s <= S; s += blockDim.x) p.tile_prefix[s] = over ? 0 : prefix[s];
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (over) return;

  const int per_run = run_tiles(p, total);
  const int runs = (total + per_run - 1) / per_run;
  const int64_t jobs = (int64_t)runs * Hkv;  // (run, head), heads innermost
  const uint64_t policy = l2_policy_evict_first();
  const int col = lane % kCols, row0 = lane / kCols;
  for (int64_t job = (int64_t)blockIdx.x * warps + warp; job < jobs;
       job += (int64_t)gridDim.x * warps) {
    const int r = (int)(job / Hkv), j = (int)(job - (int64_t)r * Hkv);
    const int t_begin = r * per_run, t_end = min(t_begin + per_run, total);

    // The loading side, ahead of the consuming side by up to two tiles: tile in_t
    // of the batch, at token in_tok of sequence in_s (in_L tokens), in block
    // blk; blk_next is the block after it, of this sequence or the next one.
    int in_t = t_begin, in_s = seq_of(prefix, S, t_begin);
    int in_tok = (t_begin - prefix[in_s]) * kRows;
    int in_L = visible(p, in_s);
    int in_slot = 0, in_q = 0;
    bool in_first = true;  // the sequence's first tile of this run
    auto block_of = [&](int s, int tok) {
      int blk = p.block_tables[(int64_t)s * p.max_blocks_per_seq + (tok >> shift)];
      if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
        blk = 0;
      }
      return blk;
    };
    auto next_seq = [&](int s) {  // the next sequence with tokens
      do ++s; while (s < S && prefix[s + 1] == prefix[s]);
      return s;
    };
    auto block_after = [&]() {
      const int tok = ((in_tok >> shift) + 1) << shift;
      if (tok < in_L) return block_of(in_s, tok);
      const int s = next_seq(in_s);
      return s < S ? block_of(s, 0) : 0;
    };
    int blk = block_of(in_s, in_tok), blk_next = block_after();
    auto issue = [&]() {
      if (in_t < t_end) {
        if (in_first) {
          const uint16_t *q = p.q + ((int64_t)in_s * Hkv + j) * G * D;
          for (int x = lane; x < G * kCols; x += 32)
            copy16(qslots + in_q * W::kQ + tile_at<D>(x / kCols, x % kCols), q + x * 8, true, policy);
          in_q = in_q + 1 == kStages ? 0 : in_q + 1;
          in_first = false;
        }
        const int64_t slot = ((int64_t)blk << shift) + (in_tok & ((1 << shift) - 1));
        const int64_t at = ((slot + row0) * Hkv + j) * D + col * 8;
        const int64_t step = (int64_t)kRowsPer * Hkv * D;
        const int64_t fresh = ((int64_t)in_s * Hkv + j) * D + col * 8;
        // (the newest token comes from the inputs when the call stores it)
        const int newest = p.new_k != nullptr && in_L == p.context_lens[in_s] ? in_L - 1 : -1;
        const uint32_t dst = tiles + in_slot * 2 * W::kHalf;
#pragma unroll
        for (int i = 0; i < kRows / kRowsPer; ++i) {
          const int t = in_tok + row0 + i * kRowsPer;
          const uint32_t to = dst + tile_at<D>(row0 + i * kRowsPer, col);
          const bool is_new = t == newest;
          copy16(to, is_new ? p.new_k + fresh : p.k_cache + at + i * step, t < in_L, policy);
          copy16(to + W::kHalf, is_new ? p.new_v + fresh : p.v_cache + at + i * step, t < in_L, policy);
        }
        ++in_t;
        in_slot = in_slot + 1 == kStages ? 0 : in_slot + 1;
        if (in_t < t_end) {
          in_tok += kRows;
          const bool ends = in_tok >= in_L;
          if (ends || (in_tok & ((1 << shift) - 1)) == 0) {
            if (ends) {
              in_s = next_seq(in_s);
              in_tok = 0;
              in_L = visible(p, in_s);
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
    for (int s = seq_of(prefix, S, t_begin), tile = t_begin; tile < t_end; s = next_seq(s)) {
      const int L = visible(p, s);
      const int first = (tile - prefix[s]) * kRows;                  // tokens [first, last) are here
      const int last = min(L, first + (t_end - tile) * kRows);
      uint32_t qf[D / 16][2];
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float o[D / 16][4];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      for (int tok = first; tok < last; tok += kRows, ++tile) {
        float *lg = p.logits + ((int64_t)tile * Hkv + j) * kRows * G;
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
          const bool in0 = tok + i0 < L, in1 = tok + i1 < L;
          float z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = (s_even[i] + s_odd[i]) * p.qscale;
          if (owner) {
            if (G == 1) {
              if (in0) lg[i0] = z[0];
              if (in1) lg[i1] = z[2];
            } else {
              if (in0) *reinterpret_cast<float2 *>(lg + i0 * G + h0) = make_float2(z[0], z[1]);
              if (in1) *reinterpret_cast<float2 *>(lg + i1 * G + h0) = make_float2(z[2], z[3]);
            }
          }
          if (!in0) z[0] = z[1] = -INFINITY;
          if (!in1) z[2] = z[3] = -INFINITY;
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
          uint32_t first0 = pack_bf16x2(p0, p1), first1 = pack_bf16x2(p2, p3);
          const uint32_t rest0 = pack_bf16x2(p0 - bf16lo(first0), p1 - bf16hi(first0));
          const uint32_t rest1 = pack_bf16x2(p2 - bf16lo(first1), p3 - bf16hi(first1));
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
      const int64_t part = (int64_t)(s + r) * Hkv + j;
      if (owner) {
        float *po = p.part_o + part * G * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int d = i * 16 + (lane >> 2);
          if (G == 1) {
            po[d] = o[i][0];
            po[d + 8] = o[i][2];
          } else {
            *reinterpret_cast<float2 *>(po + d * G + h0) = make_float2(o[i][0], o[i][1]);
            *reinterpret_cast<float2 *>(po + (d + 8) * G + h0) = make_float2(o[i][2], o[i][3]);
          }
        }
        if (lane < 4) {
          float *ml = p.part_ml + (part * G + h0) * 2;
          ml[0] = m0;
          ml[1] = l0;
          if (G > 1) {
            ml[2] = m1;
            ml[3] = l1;
          }
        }
      }
      if (last != L || L != p.context_lens[s]) continue;
      // The run with the newest token: its sum starts at zero.  (Here, and not by
      // a store beside the second launch's additions: the slot may be in a block
      // that another sequence of the call holds, too, as one of its older keys.)
      if (lane == 0) {
        const int blk = p.block_tables[(int64_t)s * p.max_blocks_per_seq + ((L - 1) >> shift)];
        if (blk >= 0 && blk < p.num_blocks)
          p.key_weights[(((int64_t)blk * Hkv + j) << shift) + ((L - 1) & ((1 << shift) - 1))] = 0.f;
      }
      // And it is stored (no run of the call reads its slot).
      if (p.new_k != nullptr) {
        const int64_t to = p.new_slots[s];
        if (to >= 0 && to < p.num_blocks << shift) {
          if (lane < kCols) {
            const int64_t from = ((int64_t)s * Hkv + j) * kCols + lane;
            const int64_t at = (to * Hkv + j) * kCols + lane;
            reinterpret_cast<uint4 *>(p.k_cache_w)[at] = reinterpret_cast<const uint4 *>(p.new_k)[from];
            reinterpret_cast<uint4 *>(p.v_cache_w)[at] = reinterpret_cast<const uint4 *>(p.new_v)[from];
          }
        } else if (to != -1 && lane == 0) {
          flag_status(p.status, PKV_DEV_BAD_SLOT);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
}

// Second launch: one CTA per (sequence, kv head, kJoinTokens tokens), or several
// such parts of a sequence.  It joins the maxima and sums of all of its sequence's
// runs, then adds the weights of its own tokens and writes its share of the output.
template <int D, int G>
__global__ void __launch_bounds__(join_threads(G)) decode_weights_join_kernel(const WeightsParams p) {
  constexpr int kJoinThreads = join_threads(G);
  __shared__ float4 acc_s[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  constexpr int kRows = WarpSmem<D, G>::kRows;
  const int Hkv = p.num_kv_heads, shift = p.block_shift;
  const int s = blockIdx.x / Hkv, j = blockIdx.x - s * Hkv;
  const int L = visible(p, s);  // an input of the call: the first launch does not write it
  const int begin = blockIdx.y * p.join_tokens;
  // (The launch must not end before the first one has, or a next call on the
  // stream could share the workspace with it: one CTA always waits.)
  if (begin >= L && (blockIdx.x | blockIdx.y) != 0) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (begin >= L) return;
  const int tiles = p.tile_prefix[p.num_seqs];
  const int tile0 = p.tile_prefix[s];
  if (tiles == 0) return;  // the call was refused for want of workspace
  const int per_run = run_tiles(p, tiles);
  const int r0 = tile0 / per_run;                                        // the sequence's runs
  const int n = (tile0 + (L + kRows - 1) / kRows - 1) / per_run - r0 + 1;
  const int64_t part0 = (int64_t)(s + r0) * Hkv + j;
  const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + part0 * G;
  const int64_t ml_step = (int64_t)Hkv * G;
  // A thread's tokens: their logits and blocks, asked for before the statistics.
  const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
  constexpr int kEach = kJoinTokens / kJoinThreads;
  float z[kEach][G];
  int blk[kEach];
  auto ask = [&](int begin) {
    const int end = min(L, begin + p.join_tokens);
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int i = begin + tid + x * kJoinThreads;
      blk[x] = -1;
      if (i >= end) continue;
      blk[x] = bt[i >> shift];
      const float *lg = p.logits + (((int64_t)(tile0 + i / kRows) * Hkv + j) * kRows + i % kRows) * G;
      if constexpr (G >= 4) {
#pragma unroll
        for (int g = 0; g < G; g += 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4 *>(lg + g));
          z[x][g] = y.x;
          z[x][g + 1] = y.y;
          z[x][g + 2] = y.z;
          z[x][g + 3] = y.w;
        }
      } else if constexpr (G == 2) {
        const float2 y = __ldcg(reinterpret_cast<const float2 *>(lg));
        z[x][0] = y.x;
        z[x][1] = y.y;
      } else {
        z[x][0] = __ldcg(lg);
      }
    }
  };
  ask(begin);
  // Lane (part, head) of every warp: running maximum and sum over its parts;
  // then over the parts of all lanes.  (No barrier: a CTA's warps do this alike.)
  float M[G], inv[G];
  {
    const int g = lane % G;
    float m = -INFINITY, l = 0.f;
    constexpr int kStep = 32 / G, kBatch = 8;  // (a batch's loads are asked for at once)
    for (int first = lane / G; first < n; first += kStep * kBatch) {
      float2 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int r = first + u * kStep;
        x[u] = r < n ? __ldcg(ml + r * ml_step + g) : make_float2(-INFINITY, 0.f);
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, x[u].x);
      const float ref = mn == -INFINITY ? 0.f : mn;
      l *= fast_exp2(m - ref);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) l = fmaf(x[u].y, fast_exp2(x[u].x - ref), l);
      m = mn;
    }
#pragma unroll
    for (int k = G; k < 32; k <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, k);
      const float l2 = __shfl_xor_sync(0xffffffffu, l, k);
      const float mn = fmaxf(m, m2);
      const float ref = mn == -INFINITY ? 0.f : mn;
      l = l * fast_exp2(m - ref) + l2 * fast_exp2(m2 - ref);
      m = mn;
    }
    l = 1.f / l;
#pragma unroll
    for (int x = 0; x < G; ++x) {
      M[x] = __shfl_sync(0xffffffffu, m, x);
      inv[x] = __shfl_sync(0xffffffffu, l, x);
    }
  }
  // Their weights, and those of the CTA's further parts.
  auto add = [&](int begin) {
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int i = begin + tid + x * kJoinThreads;
      if (blk[x] < 0 || blk[x] >= p.num_blocks) continue;  // (also: past the end)
      float a = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) a = fmaf(fast_exp2(z[x][g] - M[g]), inv[g], a);
      atomicAdd(p.key_weights + ((((int64_t)blk[x] * Hkv + j) << shift) + (i & ((1 << shift) - 1))), a);
    }
  };
  add(begin);
  const int stride = gridDim.y * p.join_tokens;
  for (int more = begin + stride; more < L; more += stride) {
    ask(more);
    add(more);
  }
  // Output: the sequence's CTAs share the D * G values, four at a time; the
  // threads of a CTA share the parts.
  constexpr int kQuads = D * G / 4;
  const int parts = min((L + p.join_tokens - 1) / p.join_tokens, (int)gridDim.y);
  const int per = (kQuads + parts - 1) / parts;
  const int q0 = min((int)blockIdx.y * per, kQuads), q1 = min(q0 + per, kQuads);
  const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + part0 * kQuads;
  for (int qb = q0; qb < q1; qb += kJoinThreads) {
    const int width = min(q1 - qb, kJoinThreads);
    const int lanes = kJoinThreads / width;  // threads per quad
    const int q = qb + tid % width, mine = tid / width;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int e = q * 4;  // value e is dim e / G of head e % G
    // The value of head (e + x) % G, x < 4.
    auto of_head = [&](const float (&of)[G], int x) {
      if constexpr (G == 8) return (e & 4) ? of[4 + x] : of[x];
      else return of[x % G];
    };
    if (mine < lanes) {
#pragma unroll 4
      for (int r = mine; r < n; r += lanes) {
        const float4 y = __ldcg(po + (int64_t)r * Hkv * kQuads + q);
        const float *mr = reinterpret_cast<const float *>(ml + r * ml_step);
        acc.x = fmaf(fast_exp2(__ldcg(mr + 2 * (e % G)) - of_head(M, 0)), y.x, acc.x);
        acc.y = fmaf(fast_exp2(__ldcg(mr + 2 * ((e + 1) % G)) - of_head(M, 1)), y.y, acc.y);
        acc.z = fmaf(fast_exp2(__ldcg(mr + 2 * ((e + 2) % G)) - of_head(M, 2)), y.z, acc.z);
        acc.w = fmaf(fast_exp2(__ldcg(mr + 2 * ((e + 3) % G)) - of_head(M, 3)), y.w, acc.w);
      }
    }
    __syncthreads();
    acc_s[tid] = acc;
    __syncthreads();
    if (tid < width) {
      for (int k = 1; k < lanes; ++k) {
        const float4 y = acc_s[k * width + tid];
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
      }
      const float v[4] = {acc.x, acc.y, acc.z, acc.w};
      uint16_t *out = p.out + ((int64_t)s * Hkv + j) * G * D;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int g = (e + k) % G, d = (e + k) / G;
        out[g * D + d] = (uint16_t)pack_bf16x2(v[k] * of_head(inv, k), 0.f);
      }
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
  size_t prefix, ml, o, logits, total;
  // Tokens: all that max_total_blocks blocks hold, in whole tiles.
  Workspace(int64_t S, int64_t Hq, int64_t Hkv, int64_t D, int64_t tokens) {
    const int64_t parts = (S + 1) * Hkv + kMaxWarps;  // of a head: num_seqs + runs
    const int64_t G = Hq / Hkv;
    prefix = 256;
    ml = prefix + align256((size_t)(S + 1) * 4);
    o = ml + align256((size_t)(parts * G) * 8);
    logits = o + align256((size_t)(parts * G * D) * 4);
    total = logits + align256((size_t)(tokens * Hq) * 4);
  }
};

template <int D, int G>
pkv_status launch(WeightsParams prm, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  const int prefix = (prm.num_seqs + 1) * 4;
  int warps = (kMaxDynamicSmem - 1024 - prefix) / WarpSmem<D, G>::bytes;
  if (warps > kWarpsMost) warps = kWarpsMost;
  static_assert((kMaxDynamicSmem - 1024 - (kMaxSeqs + 1) * 4) / WarpSmem<D, G>::bytes >= 1, "");
  const int smem = warps * WarpSmem<D, G>::bytes + prefix;
  if (!kernel_smem_setup((const void *)decode_weights_kernel<D, G>, warps * 32, smem, nullptr))
    return PKV_ERR_CUDA;
  const int64_t room = (int64_t)prm.max_blocks_per_seq << prm.block_shift;
  const int kRows = WarpSmem<D, G>::kRows;
  // As many runs as give every warp of the GPU one of a kv head, and no more
  // than the longest possible batch has tiles.
  int64_t all = (int64_t)sms * warps;
  if (all > kMaxWarps) all = kMaxWarps;
  int64_t runs = all / prm.num_kv_heads;
  int64_t tiles = (int64_t)prm.num_seqs * ((room + kRows - 1) / kRows);
  if (tiles > prm.max_tiles) tiles = prm.max_tiles;
  if (runs > tiles) runs = tiles;
  if (runs < 1) runs = 1;
  prm.runs = (int)runs;
  int64_t grid = (runs * prm.num_kv_heads + warps - 1) / warps;
  if (grid > sms) grid = sms;
  // Few sequences: parts down to a token per thread, so that the join has CTAs for
  // the GPU too (one sequence of 1000 tokens, eight kv heads: 18.5 us with 1024
  // tokens per CTA, 14.4 with 128; with four query heads each of 16 sequences of
  // 100 to 900 tokens 21.9 and 18.5).
  const int64_t units = (int64_t)prm.num_seqs * prm.num_kv_heads;
  prm.join_tokens = kJoinTokens;
  while (prm.join_tokens > join_threads(G) && units * room < (int64_t)prm.join_tokens * kJoinFill * sms)
    prm.join_tokens /= 2;
  // Both launches are programmatic dependents of what precedes them, the first one
  // of the kernel before the call: 2.0 to 2.6 us less from call to call (64 sequences
  // with their store 58.5 -> 56.0).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t err = cudaLaunchKernelEx(&cfg, decode_weights_kernel<D, G>, prm);
  int64_t parts = (room + prm.join_tokens - 1) / prm.join_tokens;
  if (parts * units > kJoinCtas) parts = units < kJoinCtas ? kJoinCtas / units : 1;
  cfg.gridDim = dim3((unsigned)units, (unsigned)parts);
  cfg.blockDim = dim3(join_threads(G));
  cfg.dynamicSmemBytes = 0;
  if (err == cudaSuccess) err = cudaLaunchKernelEx(&cfg, decode_weights_join_kernel<D, G>, prm);
  return launch_status();  // (either launch's error, which it clears)
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_weights_workspace_size(int num_seqs, int num_q_heads,
                                                    int num_kv_heads, int head_dim,
                                                    int block_size, int64_t max_total_blocks) {
  using namespace pkv;
  if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || max_total_blocks < 0)
    return 0;
  if (num_q_heads > (1 << 16) || head_dim > (1 << 16) || num_kv_heads > (1 << 16) ||
      block_size > (1 << 16))
    return 0;
  // (bounded so that no product below can wrap)
  if (num_q_heads < num_kv_heads) return 0;
  if ((double)num_seqs * num_q_heads * head_dim > 1e17) return 0;
  const int64_t per_token = (int64_t)num_q_heads * 4;
  if (max_total_blocks > (INT64_MAX / 4) / (per_token * block_size)) return 0;
  return Workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, max_total_blocks * block_size)
      .total;
}

extern "C" pkv_status pkv_paged_decode_weights_attn(
    uint16_t *out, float *key_weights, const uint16_t *q, const uint16_t *new_k,
    const uint16_t *new_v, const int32_t *slot_mapping, uint16_t *k_cache, uint16_t *v_cache,
    const int32_t *block_tables, const int32_t *context_lens, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
    int64_t max_total_blocks, float scale, void *workspace, size_t workspace_bytes,
    int32_t *dev_status, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || max_total_blocks < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / num_kv_heads;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (G != 1 && G != 2 && G != 4 && G != 8) return PKV_ERR_UNSUPPORTED;
  if (block_size != 64 && block_size != 128 && block_size != 256 && block_size != 512)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs > kMaxSeqs) return PKV_ERR_UNSUPPORTED;
  // (the second launch's grid: sequences and heads by parts of kJoinTokens)
  if ((int64_t)num_seqs * num_kv_heads > 0x7FFFFFFFLL ||
      (int64_t)max_blocks_per_seq * block_size > (int64_t)65535 * kJoinTokens)
    return PKV_ERR_UNSUPPORTED;
  // NaN or infinite, itself or in the exponentials' base 2 (a logit of zero would be NaN)
  if (!isfinite(scale * kLog2e)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !key_weights || !q || !k_cache || !v_cache || !block_tables || !context_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(key_weights) & 3u) != 0)
    return PKV_ERR_INVALID_ARG;
  const int stores = (new_k != nullptr) + (new_v != nullptr) + (slot_mapping != nullptr);
  if (stores != 0 && stores != 3) return PKV_ERR_INVALID_ARG;
  if (stores == 3 && (!aligned16(new_k) || !aligned16(new_v))) return PKV_ERR_INVALID_ARG;
  const size_t need = pkv_decode_weights_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                        head_dim, block_size, max_total_blocks);
  if (need == 0) return PKV_ERR_INVALID_ARG;  // a workspace that size cannot be addressed
  if (workspace == nullptr || workspace_bytes < need ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_WORKSPACE;

  WeightsParams prm;
  // (32-bit tile numbers: a bound of more tiles is refused)
  const int rows = 2048 / head_dim;
  prm.max_tiles = max_total_blocks * block_size / rows;
  if (prm.max_tiles > 0x7FFFFFFFLL) return PKV_ERR_UNSUPPORTED;
  const Workspace lay(num_seqs, num_q_heads, num_kv_heads, head_dim, max_total_blocks * block_size);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  prm.out = out;
  prm.key_weights = key_weights;
  prm.q = q;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.context_lens = context_lens;
  prm.new_k = new_k;
  prm.new_v = new_v;
  prm.new_slots = slot_mapping;
  prm.k_cache_w = k_cache;
  prm.v_cache_w = v_cache;
  prm.tile_prefix = reinterpret_cast<int32_t *>(ws + lay.prefix);
  prm.part_ml = reinterpret_cast<float *>(ws + lay.ml);
  prm.part_o = reinterpret_cast<float *>(ws + lay.o);
  prm.logits = reinterpret_cast<float *>(ws + lay.logits);
  prm.status = dev_status;
  prm.num_blocks = num_blocks;
  prm.num_seqs = num_seqs;
  prm.num_kv_heads = num_kv_heads;
  prm.block_shift = 31 - __builtin_clz((unsigned)block_size);
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.qscale = scale * kLog2e;
  prm.runs = 0;
  prm.join_tokens = 0;
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
