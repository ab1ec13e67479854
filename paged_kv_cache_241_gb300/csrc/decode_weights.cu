// decode_weights.cu -- paged decode attention that also collects key weights.
//
// One new token per sequence attends over its paged context, and the weight
// that each key receives, summed over the query heads of its kv head, is added
// to the key's running sum (the newest key's sum is set: its slot held another
// token's).  The weights need the softmax's denominator, which is known only
// when the whole context has been read, so the logits (4 G bytes a key and kv
// head, beside the 4 D bytes of its K and V) go through the workspace:
//
//  1. Split-K attention.  An item is (chunk of a sequence's tokens, kv head).
//     It writes its logits (log2 units), its maximum and sum, and its
//     unnormalised output.
//  2. Join, a programmatic dependent launch over the same items: every CTA
//     joins the maxima and sums of its sequence's chunks, writes its share of
//     the output, and adds its chunk's weights to the sums.
#include <math.h>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSeqs = 16384;
constexpr int kMaxChunk = 512;
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
  int32_t *chunk_prefix;  // [num_seqs + 1]: first chunk of each sequence
  float *part_ml;         // [chunks, Hkv, G, 2]   (max in log2 units, sum)
  float *part_o;          // [chunks, Hkv, G, D]
  float *logits;          // [chunks, Hkv, chunk, G]
  int32_t *status;
  int64_t num_blocks;
  int64_t max_chunks;
  int num_seqs;
  int num_kv_heads;
  int block_shift;
  int chunk;  // tokens per item: 64 << n
  int max_blocks_per_seq;
  float qscale;  // scale * log2(e)
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Visible tokens of a sequence: context_lens, at most what its table holds.
__device__ __forceinline__ int visible(const WeightsParams &p, int s) {
  const int64_t room = (int64_t)p.max_blocks_per_seq << p.block_shift;
  const int L = p.context_lens[s];
  return L <= 0 ? 0 : (int)min((int64_t)L, room);
}

// First chunk of every sequence into prefix[0 .. S] (shared memory), by all
// threads; returns the number of chunks.
__device__ int scan_chunks(const WeightsParams &p, int *prefix, int *warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs;
  const int per = (S + kThreads - 1) / kThreads;
  const int begin = min(tid * per, S), end = min(begin + per, S);
  int local = 0;
  for (int s = begin; s < end; ++s) local += (visible(p, s) + p.chunk - 1) / p.chunk;
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int run = incl - local, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) run += warp_sums[w];
    total += warp_sums[w];
  }
  for (int s = begin; s < end; ++s) {
    prefix[s] = run;
    run += (visible(p, s) + p.chunk - 1) / p.chunk;
  }
  if (tid == 0) prefix[S] = total;
  __syncthreads();
  return total;
}

// The sequence that chunk c belongs to (the last s with prefix[s] <= c).
__device__ __forceinline__ int seq_of(const int *prefix, int S, int c) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads) decode_weights_kernel(const WeightsParams p) {
  extern __shared__ int prefix[];  // [S + 1]
  __shared__ float qs[G][D];
  __shared__ float lg[kMaxChunk][G];
  __shared__ int64_t slots[kMaxChunk];
  __shared__ float stat[2][G];
  __shared__ int warp_sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs, Hkv = p.num_kv_heads, C = p.chunk;
  const int total = scan_chunks(p, prefix, warp_sums);
  if (blockIdx.x == 0) {
    for (int s = tid; s < S; s += kThreads) {
      const int L = p.context_lens[s];
      if (L <= 0 || L != visible(p, s)) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    }
    const bool over = total > p.max_chunks;
    if (over && tid == 0) flag_status(p.status, PKV_DEV_WORKSPACE);
    for (int s = tid; s <= S; s += kThreads) p.chunk_prefix[s] = over ? 0 : prefix[s];
  }
  if (total > p.max_chunks) return;
  for (int64_t item = blockIdx.x; item < (int64_t)total * Hkv; item += gridDim.x) {
    const int c = (int)(item / Hkv), j = (int)(item - (int64_t)c * Hkv);
    const int s = seq_of(prefix, S, c);
    const int first = (c - prefix[s]) * C;
    const int L = visible(p, s);
    const int valid = min(C, L - first);
    const int newest = p.new_k != nullptr && L == p.context_lens[s] ? L - 1 - first : -1;
    const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    __syncthreads();
    for (int e = tid; e < G * D; e += kThreads)
      qs[e / D][e % D] = bf16lo(p.q[((int64_t)s * Hkv + j) * G * D + e]) * p.qscale;
    for (int t = tid; t < valid; t += kThreads) {
      const int i = first + t;
      int blk = bt[i >> p.block_shift];
      if (blk < 0 || blk >= p.num_blocks) {
        flag_status(p.status, PKV_DEV_BAD_BLOCK);
        blk = 0;
      }
      slots[t] = ((int64_t)blk << p.block_shift) + (i & ((1 << p.block_shift) - 1));
    }
    __syncthreads();
    for (int t = tid; t < valid; t += kThreads) {
      const uint16_t *k = t == newest ? p.new_k + ((int64_t)s * Hkv + j) * D
                                      : p.k_cache + (slots[t] * Hkv + j) * D;
      float acc[G];
      for (int g = 0; g < G; ++g) acc[g] = 0.f;
      for (int d = 0; d < D; ++d)
        for (int g = 0; g < G; ++g) acc[g] = fmaf(bf16lo(k[d]), qs[g][d], acc[g]);
      for (int g = 0; g < G; ++g) {
        lg[t][g] = acc[g];
        p.logits[(item * C + t) * G + g] = acc[g];
      }
    }
    __syncthreads();
    for (int g = warp; g < G; g += kWarps) {
      float m = -INFINITY;
      for (int t = lane; t < valid; t += 32) m = fmaxf(m, lg[t][g]);
      m = warp_max(m);
      float l = 0.f;
      for (int t = lane; t < valid; t += 32) {
        const float e = exp2f(lg[t][g] - m);
        lg[t][g] = e;
        l += e;
      }
      l = warp_sum(l);
      if (lane == 0) {
        stat[0][g] = m;
        stat[1][g] = l;
      }
    }
    __syncthreads();
    for (int e = tid; e < G * D; e += kThreads) {
      const int g = e / D, d = e - g * D;
      float acc = 0.f;
      for (int t = 0; t < valid; ++t) {
        const uint16_t *v = t == newest ? p.new_v + ((int64_t)s * Hkv + j) * D
                                        : p.v_cache + (slots[t] * Hkv + j) * D;
        acc = fmaf(lg[t][g], bf16lo(v[d]), acc);
      }
      p.part_o[item * G * D + e] = acc;
    }
    if (tid < G) {
      p.part_ml[(item * G + tid) * 2] = stat[0][tid];
      p.part_ml[(item * G + tid) * 2 + 1] = stat[1][tid];
    }
    if (newest >= 0 && newest < valid) {
      const int64_t slot = p.new_slots[s];
      if (slot >= 0 && slot < p.num_blocks << p.block_shift) {
        for (int d = tid; d < D; d += kThreads) {
          p.k_cache_w[(slot * Hkv + j) * D + d] = p.new_k[((int64_t)s * Hkv + j) * D + d];
          p.v_cache_w[(slot * Hkv + j) * D + d] = p.new_v[((int64_t)s * Hkv + j) * D + d];
        }
      } else if (slot != -1 && tid == 0) {
        flag_status(p.status, PKV_DEV_BAD_SLOT);
      }
    }
  }
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads) decode_weights_join_kernel(const WeightsParams p) {
  __shared__ float stat[2][G];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs, Hkv = p.num_kv_heads, C = p.chunk;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = p.chunk_prefix[S];
  for (int64_t item = blockIdx.x; item < (int64_t)total * Hkv; item += gridDim.x) {
    const int c = (int)(item / Hkv), j = (int)(item - (int64_t)c * Hkv);
    const int s = seq_of(p.chunk_prefix, S, c);
    const int c0 = p.chunk_prefix[s], n = p.chunk_prefix[s + 1] - c0;
    const int first = (c - c0) * C;
    const int L = visible(p, s);
    const int valid = min(C, L - first);
    const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    __syncthreads();
    for (int g = warp; g < G; g += kWarps) {
      float m = -INFINITY, l = 0.f;
      for (int r = lane; r < n; r += 32)
        m = fmaxf(m, p.part_ml[(((int64_t)(c0 + r) * Hkv + j) * G + g) * 2]);
      m = warp_max(m);
      for (int r = lane; r < n; r += 32) {
        const float *ml = p.part_ml + (((int64_t)(c0 + r) * Hkv + j) * G + g) * 2;
        l += exp2f(ml[0] - m) * ml[1];
      }
      l = warp_sum(l);
      if (lane == 0) {
        stat[0][g] = m;
        stat[1][g] = 1.f / l;
      }
    }
    __syncthreads();
    if (c == c0) {
      for (int e = tid; e < G * D; e += kThreads) {
        const int g = e / D;
        float acc = 0.f;
        for (int r = 0; r < n; ++r) {
          const int64_t it = (int64_t)(c0 + r) * Hkv + j;
          acc = fmaf(exp2f(p.part_ml[(it * G + g) * 2] - stat[0][g]), p.part_o[it * G * D + e], acc);
        }
        p.out[((int64_t)s * Hkv + j) * G * D + e] = (uint16_t)pack_bf16x2(acc * stat[1][g], 0.f);
      }
    }
    for (int t = tid; t < valid; t += kThreads) {
      const int i = first + t;
      const int blk = bt[i >> p.block_shift];
      if (blk < 0 || blk >= p.num_blocks) continue;
      float a = 0.f;
      for (int g = 0; g < G; ++g)
        a = fmaf(exp2f(p.logits[(item * C + t) * G + g] - stat[0][g]), stat[1][g], a);
      float *w = p.key_weights + ((((int64_t)blk * Hkv + j) << p.block_shift) +
                                  (i & ((1 << p.block_shift) - 1)));
      if (i == p.context_lens[s] - 1) *w = a;
      else atomicAdd(w, a);
    }
  }
}

// Tokens per item: the largest chunk that still leaves some 2000 items, for
// which a batch's context lengths count as long as its block bound allows.
int chunk_for(int64_t max_total_blocks, int block_size, int num_kv_heads) {
  int c = kMaxChunk;
  while (c > 64 && max_total_blocks * block_size / c * num_kv_heads < 2048) c >>= 1;
  return c;
}

// Chunks that sequences of at most max_total_blocks blocks in all can have.
int64_t chunks_for(int64_t max_total_blocks, int block_size, int chunk) {
  return chunk >= block_size ? max_total_blocks : max_total_blocks * (block_size / chunk);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
  size_t prefix, ml, o, logits, total;
  Workspace(int64_t S, int64_t Hq, int64_t D, int64_t chunks, int64_t chunk) {
    prefix = 256;
    ml = prefix + align256((size_t)(S + 1) * 4);
    o = ml + align256((size_t)(chunks * Hq) * 8);
    logits = o + align256((size_t)(chunks * Hq * D) * 4);
    total = logits + align256((size_t)(chunks * Hq * chunk) * 4);
  }
};

template <int D, int G>
pkv_status launch(const WeightsParams &prm, cudaStream_t stream) {
  const int smem = (prm.num_seqs + 1) * 4;
  int ctas = 0;
  if (!kernel_smem_setup((const void *)decode_weights_kernel<D, G>, kThreads, smem, &ctas))
    return PKV_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  int64_t items = (int64_t)prm.num_seqs * (((int64_t)prm.max_blocks_per_seq << prm.block_shift) + prm.chunk - 1) / prm.chunk;
  if (items > prm.max_chunks) items = prm.max_chunks;
  items *= prm.num_kv_heads;
  if (items < 1) items = 1;
  int64_t grid = (int64_t)sms * ctas;
  if (grid > items) grid = items;
  decode_weights_kernel<D, G><<<(unsigned)grid, kThreads, smem, stream>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  decode_weights_join_kernel<D, G><<<(unsigned)grid, kThreads, 0, stream>>>(prm);
  return launch_status();
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
  if (max_total_blocks > (int64_t)1 << 40) return 0;
  const int64_t per_block = (int64_t)num_q_heads * (head_dim + 2 + block_size) * 4 * ((block_size + 63) / 64 + 8);
  if (max_total_blocks > (INT64_MAX / 2) / per_block) return 0;
  const int c = chunk_for(max_total_blocks, block_size, num_kv_heads);
  return Workspace(num_seqs, num_q_heads, head_dim, chunks_for(max_total_blocks, block_size, c), c)
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
  if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;  // NaN or infinite
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
  prm.chunk = chunk_for(max_total_blocks, block_size, num_kv_heads);
  prm.max_chunks = chunks_for(max_total_blocks, block_size, prm.chunk);
  const Workspace lay(num_seqs, num_q_heads, head_dim, prm.max_chunks, prm.chunk);
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
  prm.chunk_prefix = reinterpret_cast<int32_t *>(ws + lay.prefix);
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
