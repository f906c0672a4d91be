// Rotary positions on q and k, fused with the slot-mapped cache write (rotary_and_cache).
//
// Mathematics: pair i of a token's head turns by theta = position * inv_freq[i], so
// (x, y) -> (x cos - y sin, y cos + x sin). All heads of a token share its R / 2 angles: one
// CTA takes one token, forms the angles once into shared memory and every thread turns
// 32 bytes at a time. The angle is position * inv_freq / (2 pi) in float64, reduced to a
// turn in [-1/2, 1/2]: a float32 product would be off by 0.03 rad at position 10^6. It is
// R / 2 double multiplications per token, nothing beside the memory traffic.
//
// Bound: HBM. Per token it reads q, k, v once and writes q_out and the two cache rows once;
// the unfused sequence would write k and read it again. Loads are issued before the angles
// are formed. A step's few tokens are bound by latency instead (4 us).
#pragma once

#include "common.cuh"

namespace pa {
namespace rot {

struct RotaryArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  const int32_t* positions;
  const int64_t* slot_mapping;
  const float* inv_freq;
  const float* k_scales;
  const float* v_scales;
  const int32_t* k_zeros;
  const int32_t* v_zeros;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim;
  int sec_end[4];  // first frequency behind each axis
  int adjacent, block_size, num_blocks;
};

// Eight elements as they lie in memory, kept packed until they are used.
template <pa_dtype IN>
struct Raw8;
template <>
struct Raw8<PA_BF16> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { x[2 * j] = bf16_lo(w[j]); x[2 * j + 1] = bf16_hi(w[j]); }
  }
};
template <>
struct Raw8<PA_F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// Eight values to memory in type T (quantised with scale s and zero point z), one rounding.
template <pa_dtype T>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8], float s, int z) {
  if constexpr (T == PA_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else if constexpr (T == PA_BF16) {
    uint4 w;
    w.x = pack_bf16x2(x[0], x[1]); w.y = pack_bf16x2(x[2], x[3]);
    w.z = pack_bf16x2(x[4], x[5]); w.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
  } else if constexpr (T == PA_INT8) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = fminf(fmaxf(__fdiv_rn(x[j], s), -1024.f), 1024.f);
      const int c = min(127, max(-128, __float2int_rn(y) + z));
      w[j >> 2] |= ((uint32_t)c & 0xffu) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + i) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      w[j] = (uint32_t)pack_e4m3x2(__fdiv_rn(x[4 * j], s), __fdiv_rn(x[4 * j + 1], s)) |
             (uint32_t)pack_e4m3x2(__fdiv_rn(x[4 * j + 2], s), __fdiv_rn(x[4 * j + 3], s)) << 16;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + i) = make_uint2(w[0], w[1]);
  }
}

// Small CTAs, sixteen to an SM (eight for float32 rows, twice the registers): a token goes
// through slot, loads, angles, a barrier and stores one after the other, and only other tokens
// fill those waits. 16384 tokens of 32 + 2 x 8 heads into a bf16 cache take 64 us with 64
// threads x 3 units x 16 CTAs (6.2 TB/s, 95 % of the measured copy), 68 with 128 x 3 x 8, 81 with
// 128 x 2 and no bound on registers, 105 with 256 x 2, 130 with one thread for every unit.
constexpr int kThreads = 64;
constexpr int kBatch = 3;  // 32-byte units a thread has in flight

// A unit is 16 channels of one head: the two 8-channel chunks that turn together (half-split
// pairs: 8u.. and R / 2 + 8u..), or two neighbouring chunks.
template <pa_dtype IN, pa_dtype CACHE>
__global__ void __launch_bounds__(kThreads, IN == PA_F32 ? 8 : 16)
rotary_kernel(const RotaryArgs a) {
  __shared__ float s_cos[128], s_sin[128];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0) return;  // padding token
  if (slot >= (int64_t)a.num_blocks * a.block_size) {
    if (tid == 0) flag_error(PA_DEVERR_SLOT);
    return;
  }
  const int64_t blk = slot / a.block_size;
  const int off = (int)(slot - blk * a.block_size);
  const int D = a.head_dim, half = a.rotary_dim / 2;
  const int lg = 31 - __clz(D / 16), turning = a.rotary_dim / 16;   // 2^lg units to a head
  const int qk = (a.num_q_heads + a.num_kv_heads) << lg;
  const int units = qk + (a.num_kv_heads << lg);

  // unit i: head h of all (q, then k, then v), channels c0 .. and c1 .. of it
  struct Unit {
    int h, c0, c1;
    bool turn;
  };
  auto unit = [&](int i) {
    Unit u;
    u.h = i >> lg;
    const int r = i - (u.h << lg);
    u.turn = i < qk && r < turning;
    if (u.turn && !a.adjacent) {
      u.c0 = 8 * r;
      u.c1 = half + 8 * r;
    } else {
      u.c0 = 16 * r;
      u.c1 = 16 * r + 8;
    }
    return u;
  };
  auto source = [&](int h, const void*& p, int64_t& at) {
    if (h < a.num_q_heads) {
      p = a.q;
      at = t * a.q_stride + (int64_t)h * D;
    } else if (h < a.num_q_heads + a.num_kv_heads) {
      p = a.k;
      at = t * a.k_stride + (int64_t)(h - a.num_q_heads) * D;
    } else {
      p = a.v;
      at = t * a.v_stride + (int64_t)(h - a.num_q_heads - a.num_kv_heads) * D;
    }
  };
  bool angles = false;
  for (int base = tid; base < units || !angles; base += kBatch * kThreads) {
    Raw8<IN> x0[kBatch], x1[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = base + j * kThreads;
      if (i < units) {
        const Unit u = unit(i);
        const void* p;
        int64_t at;
        source(u.h, p, at);
        x0[j].load(p, at + u.c0);
        x1[j].load(p, at + u.c1);
      }
    }
    if (!angles) {
      angles = true;
      for (int f = tid; f < half; f += kThreads) {
        int axis = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) axis += f >= a.sec_end[k];
        const double turns = (double)a.positions[(int64_t)axis * a.num_tokens + t] *
                             (double)a.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
        sincospif(2.f * (float)(turns - rint(turns)), &s_sin[f], &s_cos[f]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = base + j * kThreads;
      if (i >= units) continue;
      const Unit u = unit(i);
      float x[8], y[8];
      x0[j].get(x);
      x1[j].get(y);
      if (u.turn) {
        if (!a.adjacent) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float c = s_cos[u.c0 + e], s = s_sin[u.c0 + e], xe = x[e];
            x[e] = xe * c - y[e] * s;
            y[e] = y[e] * c + xe * s;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int f = u.c0 / 2 + e / 2;
            const float c0 = s_cos[f], n0 = s_sin[f], c1 = s_cos[f + 4], n1 = s_sin[f + 4];
            const float xe = x[e], ye = y[e];
            x[e] = xe * c0 - x[e + 1] * n0;
            x[e + 1] = x[e + 1] * c0 + xe * n0;
            y[e] = ye * c1 - y[e + 1] * n1;
            y[e + 1] = y[e + 1] * c1 + ye * n1;
          }
        }
      }
      if (u.h < a.num_q_heads) {
        const int64_t o = t * a.q_out_stride + (int64_t)u.h * D;
        store8<IN>(a.q_out, o + u.c0, x, 1.f, 0);
        store8<IN>(a.q_out, o + u.c1, y, 1.f, 0);
        continue;
      }
      const bool is_v = u.h >= a.num_q_heads + a.num_kv_heads;
      const int h = u.h - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
      const int64_t bh = blk * a.num_kv_heads + h;
      float s = 1.f;
      int z = 0;
      if constexpr (CACHE == PA_FP8_E4M3 || CACHE == PA_INT8) s = (is_v ? a.v_scales : a.k_scales)[bh];
      if constexpr (CACHE == PA_INT8) {
        z = (is_v ? a.v_zeros : a.k_zeros)[bh];
        if (!zero_in_range(z)) {  // the row is not written
          flag_error(PA_DEVERR_ZERO);
          continue;
        }
      }
      void* cache = is_v ? a.v_cache : a.k_cache;
      const int64_t o = (bh * a.block_size + off) * D;
      store8<CACHE>(cache, o + u.c0, x, s, z);
      store8<CACHE>(cache, o + u.c1, y, s, z);
    }
  }
}

}  // namespace rot
}  // namespace pa
