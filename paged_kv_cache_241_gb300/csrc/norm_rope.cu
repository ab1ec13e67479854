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
// Bound by HBM where there are many tokens, as every value is read once and written once:
// 16 prompts of 16 + 8 + 8 heads (537 MB) 89 us, 89 % of a copy's rate, 11 far chunks of
// 32 + 8 + 8 (258 MB) 44.3 us, 86 %.  By latency where there are few (up to 64 tokens 2.8
// us in a graph of calls: one load, the angles, one store).
#include <math.h>

#include <atomic>

#include "host_common.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeTokens = 8;  // tokens of a CTA, where there are many, too wide to stream
constexpr int kRopeAhead = 2;   // tokens that a warp has asked for at a time
// Stream: tokens that a warp has in shared memory, and warps of a CTA (one per SM).  16
// prompts of 16 + 8 + 8 heads (537 MB): 89.5 us with 2 and 12 (88 % of a copy), 95.0 with
// 3 and 8, 98.4 with 4 and 6, 90.7 with 2 and 10; from registers, without the copies
// through shared memory, 100.8.
constexpr int kRopePlaces = 2;
constexpr int kRopeStreamWarps = 12;
constexpr int kRopeSmem = 220 * 1024;
// Tokens per SM from which on they are streamed, in halves, and from which on whole (us,
// of 16 + 8 + 8 heads: one token to a CTA, eight, streamed in halves, streamed whole):
//   150 tokens 2.8 6.7 4.0 6.1, 600 5.3 7.4 4.2 6.1, 1800 12.0 9.9 7.9 8.1,
//   3500 25.7 13.6 14.9 15.6, 6000 41.8 23.2 23.1 24.5, 12000 80.6 42.8 41.0 38.6
// (From about 2000 to 5000 tokens eight to a CTA are up to a tenth faster.  Other layouts,
// us by these rules and floors of bytes at a copy's rate: of 4 + 2 + 2 heads of 64 dims 600
// tokens 3.3 and 0.2, 3500 5.1 and 1.1, 12000 14.2 and 3.6; of 32 + 8 + 8 of 128 600 5.7 and
// 2.2, 3500 19.8 and 12.7, 12000 55.3 and 43.4.)
constexpr int kRopeStreamTokens = 3;
constexpr int kRopeWholeTokens = 64;

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
  int warp_bytes;       // shared memory of a warp (stream)
  int first_heads;      // query heads of the first half of a token (stream; 0: no halves)
  int loading;          // CTAs that load their tokens (stream): all, but in a test
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
// the rotated part, and interleaved, 16 neighbouring dims.  A warp keeps its block of
// heads (and with it their weights, in registers) over the CTA's tokens.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;         // lanes of a head
  constexpr int kHeads = 32 / kLanes;    // heads of a warp's block
  extern __shared__ float rope_smem[];   // [tokens][cos: R/2, sin: R/2], [tokens] slots
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int R = p.rotary, half = R >> 1;
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
  const bool store = p.k_cache != nullptr;
  const int heads = Hq + Hkv + (store ? Hkv : 0);
  const int blocks = (heads + kHeads - 1) / kHeads;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int tokens = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - t0);
  int64_t *slots = reinterpret_cast<int64_t *>(rope_smem + p.tokens_per_cta * R);

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
  for (int t = tid; t < tokens; t += blockDim.x) {
    int64_t slot = store ? p.slots[t0 + t] : -1;
    if (slot < -1 || slot >= p.num_slots) {
      if (store) flag_status(p.status, PKV_DEV_BAD_SLOT);
      slot = -1;
    }
    slots[t] = slot;
  }
  __syncthreads();

  const int j = lane % kLanes, sub = lane / kLanes;
  const bool rotates = 16 * j < R;
  const int da = kInterleaved ? 16 * j : rotates ? 8 * j : 16 * j;
  const int db = kInterleaved ? da + 8 : rotates ? half + 8 * j : da + 8;
  const bool norm = p.q_weight != nullptr;
  // More warps than blocks: those of one block share the tokens.
  const int share = max(warps / blocks, 1), first = warp / blocks;
  if (first >= share && blocks < warps) return;
  for (int block = blocks < warps ? warp % blocks : warp; block < blocks; block += min(blocks, warps)) {
    const int h = block * kHeads + sub;
    const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv, live = h < heads;
    const int hk = is_k ? h - Hq : h - Hq - Hkv;  // head of k or v
    const int64_t stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
    const uint16_t *src = (is_q ? p.q + h * D : (is_k ? p.k : p.v) + hk * D) + t0 * stride;
    uint16_t *cache = (is_k ? p.k_cache : p.v_cache) + hk * D;
    float ua[8], ub[8];
    if (norm && live && (is_q || is_k)) {
      const uint16_t *weight = is_q ? p.q_weight : p.k_weight;
      unpack8(*reinterpret_cast<const uint4 *>(weight + da), ua);
      unpack8(*reinterpret_cast<const uint4 *>(weight + db), ub);
    }
    for (int ti0 = first; ti0 < tokens; ti0 += share * kRopeAhead) {
      uint4 in[kRopeAhead][2];
#pragma unroll
      for (int x = 0; x < kRopeAhead; ++x) {
        const int ti = ti0 + x * share;
        in[x][0] = in[x][1] = make_uint4(0, 0, 0, 0);
        if (ti < tokens && live) {
          in[x][0] = load16(src + ti * stride + da);
          in[x][1] = load16(src + ti * stride + db);
        }
      }
#pragma unroll
      for (int x = 0; x < kRopeAhead; ++x) {
        const int ti = ti0 + x * share;
        if (ti >= tokens) break;
        uint4 wa = in[x][0], wb = in[x][1];
        float a[8], b[8];
        unpack8(wa, a);
        unpack8(wb, b);
        if (norm) {  // (all lanes: a block may have heads of two kinds)
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
          for (int k = 1; k < kLanes; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
          const float inv = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = a[i] * inv * ua[i];
            b[i] = b[i] * inv * ub[i];
          }
        }
        if (is_q || is_k) {
          if (rotates) {
            const float *cs = rope_smem + ti * R + 8 * j, *sn = cs + half;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // The lane's i-th pair.
              float &y0 = kInterleaved ? (i < 4 ? a[2 * i & 7] : b[2 * i & 7]) : a[i];
              float &y1 = kInterleaved ? (i < 4 ? a[(2 * i + 1) & 7] : b[(2 * i + 1) & 7]) : b[i];
              const float x0 = y0, x1 = y1;
              y0 = x0 * cs[i] - x1 * sn[i];
              y1 = x1 * cs[i] + x0 * sn[i];
            }
          }
          // Without norm and rotation a value stays as it is, to the bit.
          if (norm || rotates) {
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
          put(p.q_out + ((t0 + ti) * Hq + h) * D);
        } else {
          if (is_k && p.k_out != nullptr) put(p.k_out + ((t0 + ti) * Hkv + hk) * D);
          const int64_t slot = slots[ti];
          if (slot >= 0) put(cache + slot * Hkv * D);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ many tokens

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {  // all but the last N groups are read out
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// A warp takes tokens by itself, every (number of warps)-th, or halves of them where
// tokens are wide: the first half is a token's first query heads, the second the others
// with its keys and values, about as much.  An item's rows come as bulk copies into one of
// the warp's places in shared memory, q and k are normed and turned there, and all leave as
// bulk copies, v without ever being in a register.  The next item's copies in and the last
// one's out are under way meanwhile; no warp waits for another.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeStreamWarps * 32, 1) norm_rope_stream_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;
  constexpr int kHeads = 32 / kLanes;
  extern __shared__ __align__(128) uint8_t stream_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.rotary, half = R >> 1;
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
  const bool store = p.k_cache != nullptr, norm = p.q_weight != nullptr;
  const int halves = p.first_heads > 0 ? 1 : 0;
  const int Q0 = p.first_heads;  // query heads of the first half
  const uint32_t q0_bytes = Q0 * D * 2, q1_bytes = (Hq - Q0) * D * 2, kv_bytes = Hkv * D * 2;
  const uint32_t half1_bytes = q1_bytes + kv_bytes * (store ? 2 : 1);
  const uint32_t row_bytes = q0_bytes > half1_bytes ? q0_bytes : half1_bytes;  // of a place
  const int64_t items = p.num_tokens << halves;
  uint8_t *rows = stream_smem + (size_t)warp * p.warp_bytes;   // [kRopePlaces][row_bytes]
  float *angles = reinterpret_cast<float *>(rows + kRopePlaces * row_bytes);  // [cos: R/2, sin: R/2]
  uint64_t *full = reinterpret_cast<uint64_t *>(angles + R);
  if (lane == 0) {
    for (int i = 0; i < kRopePlaces; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t first = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const uint64_t policy = l2_policy_evict_first();
  const bool loads = (int)blockIdx.x < p.loading;
  auto load = [&](int64_t item, int place) {  // (lane 0)
    if (!loads) return;
    const int64_t t = item >> halves;
    uint8_t *to = rows + place * row_bytes;
    if (halves && (item & 1) == 0) {
      mbar_arrive_expect_tx(&full[place], q0_bytes);
      bulk_load(to, p.q + t * p.q_stride, q0_bytes, &full[place], policy);
      return;
    }
    mbar_arrive_expect_tx(&full[place], half1_bytes);
    if (q1_bytes > 0) bulk_load(to, p.q + t * p.q_stride + Q0 * D, q1_bytes, &full[place], policy);
    bulk_load(to + q1_bytes, p.k + t * p.k_stride, kv_bytes, &full[place], policy);
    if (store) bulk_load(to + q1_bytes + kv_bytes, p.v + t * p.v_stride, kv_bytes, &full[place], policy);
  };
  if (lane == 0)
    for (int i = 0; i < kRopePlaces - 1; ++i)
      if (first + i * step < items) load(first + i * step, i);

  const int j = lane % kLanes, sub = lane / kLanes;
  const bool rotates = 16 * j < R;
  const int da = kInterleaved ? 16 * j : rotates ? 8 * j : 16 * j;
  const int db = kInterleaved ? da + 8 : rotates ? half + 8 * j : da + 8;
  float wq[16], wk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) wq[i] = wk[i] = 1.f;
  if (norm) {
    auto weights = [&](const uint16_t *from, float (&w)[16]) {
      float a[8], b[8];
      unpack8(*reinterpret_cast<const uint4 *>(from + da), a);
      unpack8(*reinterpret_cast<const uint4 *>(from + db), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = a[i];
        w[8 + i] = b[i];
      }
    };
    weights(p.q_weight, wq);
    weights(p.k_weight, wk);
  }
  int position = 0, slot_next = -1;
  if (first < items) {
    if (R > 0) position = p.positions[first >> halves];
    if (store) slot_next = p.slots[first >> halves];
  }
  int place = 0, phase = 0;
  bool ok = true;
  for (int64_t item = first; item < items; item += step) {
    const int64_t t = item >> halves;
    const bool second = !halves || (item & 1);  // (with the keys and values)
    int64_t slot = slot_next;
    if (slot < -1 || slot >= p.num_slots) {
      if (store && second && lane == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);
      slot = -1;
    }
    for (int a = lane; a < half; a += 32) {
      const uint64_t turn = (uint64_t)(int64_t)position * p.turns[a];
      const float x = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // (see norm_rope_kernel)
      float sn, cs;
      sincospif(x, &sn, &cs);
      angles[a] = cs * p.amplitude;
      angles[half + a] = sn * p.amplitude;
    }
    if (item + step < items) {  // (the next one's, asked for ahead)
      if (R > 0) position = p.positions[(item + step) >> halves];
      if (store) slot_next = p.slots[(item + step) >> halves];
    }
    __syncwarp();
    float cs[8], sn[8];
    if (rotates) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = angles[8 * j + i];
        sn[i] = angles[half + 8 * j + i];
      }
    }
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[place], phase, nullptr));
    if (!ok) break;
    uint8_t *at = rows + place * row_bytes;
    auto turn_heads = [&](uint8_t *base, int heads, const float (&w)[16]) {
#pragma unroll 2
      for (int h0 = 0; h0 < heads; h0 += kHeads) {
        const int h = h0 + sub;
        const bool live = h < heads;
        uint8_t *row = base + (live ? h : heads - 1) * (D * 2);
        uint4 *pa = reinterpret_cast<uint4 *>(row + da * 2), *pb = reinterpret_cast<uint4 *>(row + db * 2);
        float a[8], b[8];
        unpack8(*pa, a);
        unpack8(*pb, b);
        if (norm) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
          for (int k = 1; k < kLanes; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
          const float inv = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = a[i] * inv * w[i];
            b[i] = b[i] * inv * w[8 + i];
          }
        }
        if (rotates) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float &y0 = kInterleaved ? (i < 4 ? a[2 * i & 7] : b[2 * i & 7]) : a[i];
            float &y1 = kInterleaved ? (i < 4 ? a[(2 * i + 1) & 7] : b[(2 * i + 1) & 7]) : b[i];
            const float x0 = y0, x1 = y1;
            y0 = x0 * cs[i] - x1 * sn[i];
            y1 = x1 * cs[i] + x0 * sn[i];
          }
        }
        // (what neither norm nor rotation touches stays as it is, to the bit)
        if (live && (norm || rotates)) {
          *pa = pack8(a);
          *pb = pack8(b);
        }
      }
    };
    turn_heads(at, second ? Hq - Q0 : Q0, wq);
    if (second) turn_heads(at + q1_bytes, Hkv, wk);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (!second) {
        bulk_store(p.q_out + t * Hq * D, at, q0_bytes);
      } else {
        if (q1_bytes > 0) bulk_store(p.q_out + (t * Hq + Q0) * D, at, q1_bytes);
        if (p.k_out != nullptr) bulk_store(p.k_out + t * Hkv * D, at + q1_bytes, kv_bytes);
        if (slot >= 0) {
          bulk_store(p.k_cache + slot * Hkv * D, at + q1_bytes, kv_bytes);
          bulk_store(p.v_cache + slot * Hkv * D, at + q1_bytes + kv_bytes, kv_bytes);
        }
      }
      bulk_commit();
      // The place of the item before is read out: the next copies in go there.
      const int64_t next = item + (kRopePlaces - 1) * step;
      if (next < items) {
        bulk_wait_read<1>();
        load(next, place == 0 ? kRopePlaces - 1 : place - 1);
      }
    }
    if (++place == kRopePlaces) {
      place = 0;
      phase ^= 1;
    }
  }
  if (lane == 0) {
    if (!ok) {  // (a wait ran out: the copies still under way end before the CTA does)
      flag_status(p.status, PKV_DEV_TIMEOUT);
      for (int i = 0; i < kRopePlaces; ++i) mbar_wait_bounded(&full[i], i < place ? phase ^ 1 : phase, nullptr);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

pkv_status launch_dependent(void (*kernel)(RopeParams), unsigned grid, int threads, int smem,
                            cudaStream_t stream, const RopeParams &prm) {
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
  cudaLaunchKernelEx(&cfg, kernel, prm);
  return launch_status();
}

template <int D, bool kInterleaved>
pkv_status launch_rope(RopeParams prm, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  // More than a few tokens: streamed; in halves, in whole blocks of heads, where there are
  // not very many, or where whole ones leave no room for all warps of a CTA (11 chunks of
  // 32 + 8 + 8 heads, 12 KB a token: 47.0 us whole, 44.3 in halves; 16 prompts of 16 + 8 +
  // 8: 88.9 and 100).
  const int kv_heads = prm.num_kv_heads * (prm.k_cache != nullptr ? 2 : 1);
  const int64_t heads = (int64_t)prm.num_q_heads + kv_heads;
  auto warp_room = [&](int64_t heads) {
    return (kRopePlaces * heads * D * 2 + prm.rotary * 4 + kRopePlaces * 8 + 127) & ~(int64_t)127;
  };
  int64_t warp_bytes = warp_room(heads);
  if (prm.num_tokens <= kRopeWholeTokens * (int64_t)sms || warp_bytes * kRopeStreamWarps > kRopeSmem) {
    const int block = 16 * 32 / D;
    const int64_t half = heads / 2 / block * block;
    prm.first_heads = (int)(half < prm.num_q_heads ? half : prm.num_q_heads);
    const int64_t rest = heads - prm.first_heads;
    warp_bytes = warp_room(rest > prm.first_heads ? rest : prm.first_heads);
  }
  int warps = warp_bytes <= kRopeSmem ? (int)(kRopeSmem / warp_bytes) : 0;
  if (warps > kRopeStreamWarps) warps = kRopeStreamWarps;
  if (prm.num_tokens > kRopeStreamTokens * (int64_t)sms && warps >= 4) {
    const int smem = (int)(warps * warp_bytes);
    int per_sm = 1;
    prm.warp_bytes = (int)warp_bytes;
    if (!kernel_smem_setup((const void *)norm_rope_stream_kernel<D, kInterleaved>, warps * 32, smem, &per_sm))
      return PKV_ERR_CUDA;
    int64_t grid = (int64_t)sms * per_sm;
    const int64_t items = prm.num_tokens << (prm.first_heads > 0 ? 1 : 0);
    if (grid > (items + warps - 1) / warps) grid = (items + warps - 1) / warps;
    return launch_dependent(norm_rope_stream_kernel<D, kInterleaved>, (unsigned)grid, warps * 32, smem, stream, prm);
  }
  // Few tokens: one per CTA, so that the step is on as many SMs as it can be.
  prm.tokens_per_cta = prm.num_tokens <= kRopeStreamTokens * (int64_t)sms ? 1 : kRopeTokens;
  const int64_t grid = (prm.num_tokens + prm.tokens_per_cta - 1) / prm.tokens_per_cta;
  if (grid > 0x7FFFFFFFLL) return PKV_ERR_UNSUPPORTED;
  return launch_dependent(norm_rope_kernel<D, kInterleaved>, (unsigned)grid, kRopeWarps * 32,
                          (int)(prm.tokens_per_cta * (prm.rotary * sizeof(float) + sizeof(int64_t))), stream, prm);
}

// Test-only, set by pkv_test_rope_fault: RopeParams::loading of the process's calls.
constexpr int kRopeAllLoad = 0x7FFFFFFF;
std::atomic<int> g_loading{kRopeAllLoad};

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
  prm.warp_bytes = 0;
  prm.first_heads = 0;
  prm.loading = g_loading.load(std::memory_order_relaxed);
  prm.eps = eps;
  prm.amplitude = amplitude;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128)
    return interleaved ? launch_rope<128, true>(prm, st) : launch_rope<128, false>(prm, st);
  return interleaved ? launch_rope<64, true>(prm, st) : launch_rope<64, false>(prm, st);
}

extern "C" pkv_status pkv_test_rope_fault(int64_t wait_limit_ns, int loading_ctas) {
  if (wait_limit_ns <= 0 || loading_ctas < -1) return PKV_ERR_INVALID_ARG;
  const unsigned long long limit = (unsigned long long)wait_limit_ns;
  if (cudaMemcpyToSymbol(pkv::g_wait_limit_ns, &limit, sizeof(limit)) != cudaSuccess)
    return PKV_ERR_CUDA;
  pkv::g_loading = loading_ctas >= 0 ? loading_ctas : pkv::kRopeAllLoad;
  return PKV_OK;
}
