// prefill_weights.cu -- the attention weight that a prompt chunk's last queries
// give to each key.
//
// For sequence s with n new queries, c cached tokens and R = min(window, n),
// the sum of key p (kv head j) receives
//   a[p] = sum over queries i in [n - R, n) with c + i >= p, and over the query
//          heads h of j's group, of softmax_p(scale <q[i,h], K[p,j]>):
// added for keys cached before the chunk, set for the chunk's own.
// Two launches: the softmax denominators of every (query, head), then the
// weights summed over the queries, key by key.
#include <math.h>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct PromptParams {
  float *key_weights;
  const uint16_t *q;
  const uint16_t *k_cache;
  const int32_t *block_tables;
  const int32_t *cu_q;
  const int32_t *cu_k;
  float *lse;  // [num_seqs, rows, Hq]: log2 of the softmax denominator
  int32_t *status;
  int64_t num_blocks;
  int64_t total_q;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;
  int block_shift;
  int max_blocks_per_seq;
  int max_seqlen_q;
  int window;
  int rows;  // min(window, max_seqlen_q)
  float qscale;
};

// One sequence of the call; false (with a flag) when its lengths do not fit.
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

__device__ __forceinline__ const uint16_t *key_row(const PromptParams &p, int s, int j, int i) {
  int blk = p.block_tables[(int64_t)s * p.max_blocks_per_seq + (i >> p.block_shift)];
  if (blk < 0 || blk >= p.num_blocks) {
    flag_status(p.status, PKV_DEV_BAD_BLOCK);
    blk = 0;
  }
  const int64_t slot = ((int64_t)blk << p.block_shift) + (i & ((1 << p.block_shift) - 1));
  return p.k_cache + (slot * p.num_kv_heads + j) * p.head_dim;
}

__global__ void __launch_bounds__(kThreads) prompt_lse_kernel(const PromptParams p) {
  __shared__ float qs[128];
  __shared__ float red[2][kThreads];
  const int tid = threadIdx.x;
  const int h = blockIdx.x % p.num_q_heads;
  const int r = (blockIdx.x / p.num_q_heads) % p.rows;
  const int s = blockIdx.x / p.num_q_heads / p.rows;
  Seq q;
  if (!seq_at(p, s, q, tid == 0 && h == 0 && r == 0) || r >= q.R) return;
  const int i = q.n - q.R + r;
  const int j = h / (p.num_q_heads / p.num_kv_heads);
  for (int d = tid; d < p.head_dim; d += kThreads)
    qs[d] = bf16lo(p.q[((int64_t)(q.q_begin + i) * p.num_q_heads + h) * p.head_dim + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f;
  for (int x = tid; x <= q.c + i; x += kThreads) {
    const uint16_t *k = key_row(p, s, j, x);
    float z = 0.f;
    for (int d = 0; d < p.head_dim; ++d) z = fmaf(qs[d], bf16lo(k[d]), z);
    z *= p.qscale;
    const float mn = fmaxf(m, z);
    if (mn != -INFINITY) {
      l = l * exp2f(m - mn) + exp2f(z - mn);
      m = mn;
    }
  }
  red[0][tid] = m;
  red[1][tid] = l;
  __syncthreads();
  if (tid == 0) {
    float M = -INFINITY, Lsum = 0.f;
    for (int t = 0; t < kThreads; ++t) M = fmaxf(M, red[0][t]);
    for (int t = 0; t < kThreads; ++t)
      if (red[1][t] != 0.f) Lsum += red[1][t] * exp2f(red[0][t] - M);
    p.lse[((int64_t)s * p.rows + r) * p.num_q_heads + h] = M + log2f(Lsum);
  }
}

__global__ void __launch_bounds__(kThreads) prompt_weights_kernel(const PromptParams p) {
  __shared__ float qs[128];
  const int tid = threadIdx.x;
  const int j = blockIdx.x % p.num_kv_heads;
  const int tiles = (int)((((int64_t)p.max_blocks_per_seq << p.block_shift) + kThreads - 1) / kThreads);
  const int x = (blockIdx.x / p.num_kv_heads) % tiles * kThreads + tid;
  const int s = blockIdx.x / p.num_kv_heads / tiles;
  const int G = p.num_q_heads / p.num_kv_heads;
  Seq q;
  if (!seq_at(p, s, q, false) || x - tid >= q.len_k) return;
  const uint16_t *k = x < q.len_k ? key_row(p, s, j, x) : nullptr;
  float a = 0.f;
  for (int r = 0; r < q.R; ++r) {
    const int i = q.n - q.R + r;
    for (int g = 0; g < G; ++g) {
      const int h = j * G + g;
      __syncthreads();
      for (int d = tid; d < p.head_dim; d += kThreads)
        qs[d] = bf16lo(p.q[((int64_t)(q.q_begin + i) * p.num_q_heads + h) * p.head_dim + d]);
      __syncthreads();
      if (k != nullptr && x <= q.c + i) {
        float z = 0.f;
        for (int d = 0; d < p.head_dim; ++d) z = fmaf(qs[d], bf16lo(k[d]), z);
        a += exp2f(z * p.qscale - p.lse[((int64_t)s * p.rows + r) * p.num_q_heads + h]);
      }
    }
  }
  if (k == nullptr) return;
  const int blk = p.block_tables[(int64_t)s * p.max_blocks_per_seq + (x >> p.block_shift)];
  if (blk < 0 || blk >= p.num_blocks) return;
  float *w = p.key_weights + ((((int64_t)blk * p.num_kv_heads + j) << p.block_shift) +
                              (x & ((1 << p.block_shift) - 1)));
  if (x >= q.c) *w = a;
  else atomicAdd(w, a);
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_prefill_weights_workspace_size(int num_seqs, int64_t total_q,
                                                     int max_seqlen_q, int window,
                                                     int num_q_heads, int num_kv_heads,
                                                     int max_blocks_per_seq, int block_size) {
  if (num_seqs <= 0 || total_q <= 0 || max_seqlen_q <= 0 || window <= 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || max_blocks_per_seq <= 0 || block_size <= 0)
    return 0;
  const int64_t rows = window < max_seqlen_q ? window : max_seqlen_q;
  if (num_seqs * rows > (INT64_MAX / 8) / num_q_heads) return 0;
  return 256 + (size_t)num_seqs * rows * num_q_heads * 4;
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
  PromptParams prm;
  prm.key_weights = key_weights;
  prm.q = q;
  prm.k_cache = k_cache;
  prm.block_tables = block_tables;
  prm.cu_q = cu_seqlens_q;
  prm.cu_k = cu_seqlens_k;
  prm.lse = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + 256);
  prm.status = dev_status;
  prm.num_blocks = num_blocks;
  prm.total_q = total_q;
  prm.num_seqs = num_seqs;
  prm.num_q_heads = num_q_heads;
  prm.num_kv_heads = num_kv_heads;
  prm.head_dim = head_dim;
  prm.block_shift = 31 - __builtin_clz((unsigned)block_size);
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.max_seqlen_q = max_seqlen_q;
  prm.window = window;
  prm.rows = window < max_seqlen_q ? window : max_seqlen_q;
  prm.qscale = scale * kLog2e;
  const int64_t tiles = ((int64_t)max_blocks_per_seq * block_size + kThreads - 1) / kThreads;
  const int64_t a = (int64_t)num_seqs * prm.rows * num_q_heads, b = (int64_t)num_seqs * tiles * num_kv_heads;
  if (a > 0x7FFFFFFFLL || b > 0x7FFFFFFFLL) return PKV_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prompt_lse_kernel<<<(unsigned)a, kThreads, 0, st>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  prompt_weights_kernel<<<(unsigned)b, kThreads, 0, st>>>(prm);
  return launch_status();
}
