// norm_rope.cu -- from the projections of a step to what attention reads: the norm of
// each head's query and key, the rotation by position, and the store of K and V.
//
// For a head x of D values with weight w (or no norm: y = x):
//   y = x / sqrt(mean(x^2) + eps) * w
// and for each pair (a, b) of the first R dims, pair i being dims (i, i + R/2) or, in
// the interleaved layout, (2i, 2i + 1), with angle = position * inv_freq[i]:
//   a' = amplitude (a cos - b sin),  b' = amplitude (b cos + a sin)
// fp32 throughout, rounded once to bf16.  V is copied bit for bit.  (The pages' engine
// writes K/V through the slot mapping by a kernel of its own behind the layer's other
// operations: nano-vllm hub page, "core tech 2"; here it is the same pass.)
//
// Angles: a frequency comes as the 64-bit fixed-point fraction of a turn per position,
// so position * turns modulo 2^64 is the fraction of a turn of the whole angle, exact
// in integers however far the position; its upper 32 bits go to sincospi.  The product
// position * inv_freq in fp32 would be off by 2^-24 of itself, 0.06 radians at 2^20.
//
// Bound by HBM: every value is read once and written once.
#include <math.h>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeTokens = 8;  // tokens of a CTA, where there are many

struct RopeParams {
  uint16_t *q_out;
  uint16_t *k_out;      // may be null
  const uint16_t *q;
  const uint16_t *k;
  const uint16_t *v;    // null when there is no store
  uint16_t *k_cache;    // null when there is no store
  uint16_t *v_cache;
  const int32_t *slots;
  const int32_t *positions;
  const uint64_t *turns;
  const uint16_t *q_weight;   // null: no norm
  const uint16_t *k_weight;
  int32_t *status;
  int64_t num_tokens;
  int64_t q_stride, k_stride, v_stride;  // values between tokens
  int64_t num_slots;
  int num_q_heads;
  int num_kv_heads;
  int rotary;           // R
  int tokens_per_cta;
  float eps;
  float amplitude;
};

__device__ __forceinline__ uint4 load16(const uint16_t *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  x[0] = bf16lo(w.x);
  x[1] = bf16hi(w.x);
  x[2] = bf16lo(w.y);
  x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z);
  x[5] = bf16hi(w.z);
  x[6] = bf16lo(w.w);
  x[7] = bf16hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// A head is D / 16 lanes, each with two runs of eight dims: with the halves paired,
// dims 8j and R/2 + 8j on (lane j < R/16), so that a lane has both of a pair; behind
// the rotated part, and interleaved, 16 neighbouring dims.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;         // lanes of a head
  constexpr int kHeads = 32 / kLanes;    // heads a warp takes at a time
  extern __shared__ float rope_smem[];   // [tokens][cos: R/2, sin: R/2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int R = p.rotary, half = R >> 1;
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
  const int heads = Hq + Hkv + (p.k_cache != nullptr ? Hkv : 0);
  const int per_token = (heads + kHeads - 1) / kHeads;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int tokens = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - t0);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // cos and sin of the CTA's tokens, once for all of their heads.
  for (int i = tid; i < tokens * half; i += blockDim.x) {
    const int t = i / half, a = i - t * half;
    const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + t] * p.turns[a];
    // (signed: the nearest whole turn is left out, which keeps small angles' bits)
    const float x = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // in half turns, [-1, 1)
    float sn, cs;
    sincospif(x, &sn, &cs);
    rope_smem[t * R + a] = cs * p.amplitude;
    rope_smem[t * R + half + a] = sn * p.amplitude;
  }
  __syncthreads();

  const int j = lane % kLanes, sub = lane / kLanes;
  const bool rotates = 16 * j < R;
  const int da = kInterleaved ? 16 * j : rotates ? 8 * j : 16 * j;
  const int db = kInterleaved ? da + 8 : rotates ? half + 8 * j : da + 8;
  for (int item = warp; item < tokens * per_token; item += warps) {
    const int ti = item / per_token;
    const int64_t t = t0 + ti;
    const int h = (item - ti * per_token) * kHeads + sub;
    const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv;
    const int hk = is_k ? h - Hq : h - Hq - Hkv;  // head of k or v
    int64_t slot = -1;
    bool live = h < heads;
    if (live && !is_q && p.k_cache != nullptr) {
      slot = p.slots[t];
      if (slot < -1 || slot >= p.num_slots) {
        if (hk == 0 && is_k && j == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);
        slot = -1;
      }
      if (!is_k && slot < 0) live = false;
    }
    const uint16_t *src = is_q   ? p.q + t * p.q_stride + (int64_t)h * D
                          : is_k ? p.k + t * p.k_stride + (int64_t)hk * D
                                 : p.v + t * p.v_stride + (int64_t)hk * D;
    uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
    if (live) {
      wa = load16(src + da);
      wb = load16(src + db);
    }
    float a[8], b[8];
    unpack8(wa, a);
    unpack8(wb, b);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
    for (int k = 1; k < kLanes; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (is_q || is_k) {
      if (p.q_weight != nullptr) {
        const float inv = rsqrtf(sum * (1.f / D) + p.eps);
        const uint16_t *weight = is_q ? p.q_weight : p.k_weight;
        float ua[8], ub[8];
        unpack8(*reinterpret_cast<const uint4 *>(weight + da), ua);
        unpack8(*reinterpret_cast<const uint4 *>(weight + db), ub);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = a[i] * inv * ua[i];
          b[i] = b[i] * inv * ub[i];
        }
      }
      if (rotates) {
        const float *cs = rope_smem + ti * R + 8 * j, *sn = cs + half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // The lane's i-th pair.
          float &x = kInterleaved ? (i < 4 ? a[2 * i & 7] : b[2 * i & 7]) : a[i];
          float &y = kInterleaved ? (i < 4 ? a[(2 * i + 1) & 7] : b[(2 * i + 1) & 7]) : b[i];
          const float x0 = x, y0 = y;
          x = x0 * cs[i] - y0 * sn[i];
          y = y0 * cs[i] + x0 * sn[i];
        }
      }
      // Without norm and rotation a value stays as it is, to the bit.
      if (p.q_weight != nullptr || rotates) {
        wa = pack8(a);
        wb = pack8(b);
      }
    }
    if (!live) continue;
    auto put = [&](uint16_t *dst) {
      *reinterpret_cast<uint4 *>(dst + da) = wa;
      *reinterpret_cast<uint4 *>(dst + db) = wb;
    };
    if (is_q) {
      put(p.q_out + (t * Hq + h) * D);
    } else {
      if (is_k && p.k_out != nullptr) put(p.k_out + (t * Hkv + hk) * D);
      if (slot >= 0) put((is_k ? p.k_cache : p.v_cache) + (slot * Hkv + hk) * D);
    }
  }
}

template <int D, bool kInterleaved>
pkv_status launch_rope(RopeParams prm, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  // Few tokens: one per CTA, so that the step is on as many SMs as it can be.
  prm.tokens_per_cta = prm.num_tokens <= 8 * (int64_t)sms ? 1 : kRopeTokens;
  const int64_t grid = (prm.num_tokens + prm.tokens_per_cta - 1) / prm.tokens_per_cta;
  if (grid > 0x7FFFFFFFLL) return PKV_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kRopeWarps * 32);
  cfg.dynamicSmemBytes = (size_t)prm.tokens_per_cta * prm.rotary * sizeof(float);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, kInterleaved>, prm);
  return launch_status();
}

// [a, a + n) and [b, b + m) values of 16 bits have any in common.
bool overlap16(const uint16_t *a, int64_t n, const uint16_t *b, int64_t m) {
  if (a == nullptr || b == nullptr || n <= 0 || m <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? (uint64_t)(y - x) / 2 < (uint64_t)n : (uint64_t)(x - y) / 2 < (uint64_t)m;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_rope_turns(const double *inv_freq, int num_pairs, uint64_t *turns) {
  if (num_pairs < 0) return PKV_ERR_INVALID_ARG;
  if (num_pairs > 0 && (!inv_freq || !turns)) return PKV_ERR_INVALID_ARG;
  for (int i = 0; i < num_pairs; ++i)
    if (!(fabs(inv_freq[i]) <= 1e6)) return PKV_ERR_INVALID_ARG;  // (NaN too)
  for (int i = 0; i < num_pairs; ++i) {
    const double turn = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    double part = turn - floor(turn);                          // [0, 1]
    if (part >= 1.0) part = 0.0;
    // 2^64 times it, the upper and the lower half by themselves (each exact)
    const double hi = floor(part * 0x1p32);
    const double lo = floor((part * 0x1p32 - hi) * 0x1p32 + 0.5);
    turns[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
  }
  return PKV_OK;
}

extern "C" pkv_status pkv_norm_rope_store(
    uint16_t *q_out, uint16_t *k_out, const uint16_t *q, const uint16_t *k, const uint16_t *v,
    uint16_t *k_cache, uint16_t *v_cache, const int32_t *slot_mapping, const int32_t *positions,
    const uint64_t *turns, const uint16_t *q_weight, const uint16_t *k_weight,
    int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int64_t q_token_stride,
    int64_t k_token_stride, int64_t v_token_stride, int rotary_dim, int interleaved, float eps,
    float amplitude, int64_t num_blocks, int block_size, int32_t *dev_status, void *stream) {
  using namespace pkv;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      rotary_dim < 0 || rotary_dim > head_dim)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads > (1 << 16) || num_kv_heads > (1 << 16)) return PKV_ERR_UNSUPPORTED;
  if (!isfinite(eps) || eps < 0.f || !isfinite(amplitude)) return PKV_ERR_INVALID_ARG;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return PKV_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  if (q_token_stride == 0) q_token_stride = q_row;
  if (k_token_stride == 0) k_token_stride = kv_row;
  if (v_token_stride == 0) v_token_stride = kv_row;
  if (q_token_stride < q_row || k_token_stride < kv_row || v_token_stride < kv_row ||
      q_token_stride % 8 != 0 || k_token_stride % 8 != 0 || v_token_stride % 8 != 0)
    return PKV_ERR_INVALID_ARG;
  const int stores = (k_cache != nullptr) + (v_cache != nullptr) + (slot_mapping != nullptr);
  if (stores != 0 && (num_blocks <= 0 || block_size <= 0 || num_blocks > INT64_MAX / block_size))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (stores != 0 && stores != 3) return PKV_ERR_INVALID_ARG;
  if (stores == 0 && k_out == nullptr) return PKV_ERR_INVALID_ARG;
  if (!q_out || !q || !k || (stores == 3 && !v) || (rotary_dim > 0 && (!turns || !positions)))
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(k_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q_weight) || !aligned16(k_weight))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens > (INT64_MAX / 4) / q_token_stride || num_tokens > (INT64_MAX / 4) / k_token_stride ||
      num_tokens > (INT64_MAX / 4) / v_token_stride)
    return PKV_ERR_INVALID_ARG;
  // Outputs may take the place of their own inputs, row by row, and of nothing else.
  const int64_t q_all = (num_tokens - 1) * q_token_stride + q_row;
  const int64_t k_all = (num_tokens - 1) * k_token_stride + kv_row;
  const int64_t v_all = stores == 3 ? (num_tokens - 1) * v_token_stride + kv_row : 0;
  const bool q_place = q_out == q && q_token_stride == q_row;
  const bool k_place = k_out == k && k_token_stride == kv_row;
  if ((!q_place && overlap16(q_out, num_tokens * q_row, q, q_all)) ||
      overlap16(q_out, num_tokens * q_row, k, k_all) ||
      overlap16(q_out, num_tokens * q_row, v, v_all) ||
      overlap16(q_out, num_tokens * q_row, k_out, num_tokens * kv_row) ||
      overlap16(k_out, num_tokens * kv_row, q, q_all) ||
      (!k_place && overlap16(k_out, num_tokens * kv_row, k, k_all)) ||
      overlap16(k_out, num_tokens * kv_row, v, v_all))
    return PKV_ERR_INVALID_ARG;

  RopeParams prm;
  prm.q_out = q_out;
  prm.k_out = k_out;
  prm.q = q;
  prm.k = k;
  prm.v = stores == 3 ? v : nullptr;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.slots = slot_mapping;
  prm.positions = positions;
  prm.turns = turns;
  prm.q_weight = q_weight;
  prm.k_weight = k_weight;
  prm.status = dev_status;
  prm.num_tokens = num_tokens;
  prm.q_stride = q_token_stride;
  prm.k_stride = k_token_stride;
  prm.v_stride = v_token_stride;
  prm.num_slots = stores == 3 ? num_blocks * (int64_t)block_size : 0;
  prm.num_q_heads = num_q_heads;
  prm.num_kv_heads = num_kv_heads;
  prm.rotary = rotary_dim;
  prm.tokens_per_cta = 0;
  prm.eps = eps;
  prm.amplitude = amplitude;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128)
    return interleaved ? launch_rope<128, true>(prm, st) : launch_rope<128, false>(prm, st);
  return interleaved ? launch_rope<64, true>(prm, st) : launch_rope<64, false>(prm, st);
}
