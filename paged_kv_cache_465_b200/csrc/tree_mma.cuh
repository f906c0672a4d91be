// Attention of drafted tokens over the paged cache on the tensor cores, with warp-level
// products (mma.sync m16n8k16).
//
// Mathematics: for a tile of R rows, a row being a (drafted token, query head of the kv head's
// group) pair, S = Q K^T over 64 keys at a time, a running maximum m and sum l per row (log2
// domain), O = sum 2^(S - m) V; a row sees every key before the drafts and, of the drafts, those
// in its mask. Parts of one context join as
//   M = max m_p,  out = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p.
//
// Work split: one CTA of four warps per (part of the context, row tile, kv head, sequence). 32 rows
// split over two pairs of warps (16 rows each), a pair taking half of a tile's keys, and the pairs
// join at the end; 64 rows are 16 to a warp. 16 rows keep a warp within 168 registers with Q in
// them, and three CTAs on an SM, which hides each other's waits: 256 sequences of 1024 fp8 tokens
// take 173 us (212 with two CTAs of 32 rows to a warp) and 8 x 65536 bf16 tokens 352 (398). 128 rows do take 32 to a warp, a fragment of K or V then feeding two products
// (1560 us for 8 x 131072 tokens with 128 rows; two 64-row tiles, the second reading K and V from
// L2, 1741).
// Keys pass through a ring of shared-memory stages that asynchronous copies fill; zero for what is
// not there, so that no product reads undefined memory. There are no flags or barriers in memory
// and no waits but the CTA's own.
//
// Bound: HBM for a bf16 cache and up to 32 rows of long contexts (8 x 65536 tokens: 352 us, 93 % of
// the measured copy rate). Beyond, and for codes, the latency of the chain fragment - product -
// softmax - product in the few warps that registers leave: with 128 rows the tensor pipe is busy
// 49 % of the time and the issue slots 32 % (HBM 42 % at 8 x 131072 tokens, 1560 us); for fp8 with 32
// rows tensor 40 %, alu 46 %, issue 52 % (each code becomes f16 in every warp whose rows need it; HBM
// 52 % at 8 x 65536 tokens, 314 us). Ragged batches are bound by the longest part (library.cu).
//
// Types: a bf16 cache is multiplied as it is, with P rounded to bf16. Codes of one byte become
// f16 in registers: E4M3 values and code - zero are exact. Q rows are brought to [2^14, 2^15) by
// a power of two each (2^126 at most: short of that for rows below 2^-112), and bf16's eight bits
// survive that down to 2^-28 of the row's largest element. P carries V scale / v_ref * 2^7, v_ref
// a power of two, for each row no smaller than any |V scale| of the keys that it has seen: at most
// 2^15, and f16 holds it to 11 bits down to 2^-21 of the largest. Scales of keys that a row does
// not see, infinite ones too, do not reach it.
#pragma once

#include "decode_tc.cuh"
#include "tree_simt.cuh"

namespace pa {
namespace tree {

constexpr int kMmaThreads = 128;
constexpr int kKeys = 64;             // keys of a tile
constexpr int kMmaDim = 128;
constexpr int kPartMax = 5120;        // tokens whose block ids and scales are held at a time
constexpr int kCombRow = kMmaDim + 4; // floats of a row where the warps join

template <pa_dtype KV, int MT, int WR>
struct MmaLayout {
  static constexpr bool kQuant = KV != PA_BF16;
  static constexpr int kRowsT = 16 * MT * WR, kWK = 4 / WR;
  static constexpr int kTileBytes = kKeys * kMmaDim * (kQuant ? 1 : 2);   // K or V of a tile
  static constexpr int kStages = kQuant ? (MT == 1 ? 3 : 4) : 2;
  static constexpr int kCtas = MT == 1 ? 3 : 2;                           // on an SM
  static constexpr bool kHold = MT == 1;                                  // Q stays in registers
  // Q that goes to registers waits in the last stage, which is filled after that
  static constexpr int kOffQ = (kHold ? kStages - 1 : kStages) * 2 * kTileBytes;
  static constexpr int kQBytes = kHold ? 2 * kTileBytes : kRowsT * 256;
  static_assert(!kHold || kRowsT * 256 <= 2 * kTileBytes, "Q fits a stage");
  static constexpr int kCombBytes = kWK * kRowsT * kCombRow * 4;          // over stages and Q
  static constexpr int kOffIds = kOffQ + kQBytes > kCombBytes ? kOffQ + kQBytes : kCombBytes;
  static constexpr int kIds = kPartMax / 8;
  static constexpr int kOffMl = kOffIds + kIds * 4 * (KV == PA_BF16 ? 1 : KV == PA_INT8 ? 5 : 3);
  static constexpr int kOffDown = kOffMl + 2 * 128 * 4;
  static constexpr int kOffOdd = kOffDown + kRowsT * 4;
  static constexpr int kSmem = kOffOdd + 16 * 4;
};

// A row's view of a key tile, bit e: the row sees key t0 + e. Keys before `base` are seen, keys
// at or behind ctx are not.
__device__ __forceinline__ uint64_t tile_view(const TreeArgs& a, int64_t row, int t0, int base,
                                              int ctx) {
  const int below = min(max(base - t0, 0), kKeys);   // keys of the committed context
  uint64_t v = below >= 64 ? ~0ull : ((1ull << below) - 1ull);
  if (below < kKeys) {
    // draft bits from index t0 + below - base on, placed at bit `below`
    const uint32_t* m = a.tree_mask + row * a.mask_words;
    const int j0 = t0 + below - base;
    uint64_t bits = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int w = (j0 >> 5) + k;
      const uint64_t x = w < a.mask_words ? m[w] : 0u;
      const int sh = 32 * k - (j0 & 31);
      bits |= sh >= 64 ? 0ull : (sh >= 0 ? x << sh : x >> -sh);
    }
    v |= bits << below;
    const int live = ctx - t0;
    if (live < kKeys) v &= (1ull << live) - 1ull;
  }
  return v;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool go) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(go ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <int BS, pa_dtype KV, int MT, int WR>
__global__ void __launch_bounds__(kMmaThreads, MmaLayout<KV, MT, WR>::kCtas)
tree_mma_kernel(const TreeArgs a, int rts) {
  using L = MmaLayout<KV, MT, WR>;
  constexpr bool QUANT = L::kQuant;
  constexpr int R = L::kRowsT, WK = L::kWK, KW = kKeys / WK;   // a warp's keys of a tile
  constexpr int C = KW < 32 ? KW : 32, NT = C / 8;             // keys of a step, in eights
  constexpr bool HOLD = L::kHold;                              // Q stays in registers
  constexpr int CPR = QUANT ? 8 : 16;                          // 16-byte chunks of a key
  extern __shared__ __align__(1024) uint8_t smem[];
  int* s_id = reinterpret_cast<int*>(smem + L::kOffIds);
  float* s_ks = reinterpret_cast<float*>(s_id + L::kIds);
  float* s_vs = s_ks + L::kIds;
  int* s_kz = reinterpret_cast<int*>(s_vs + L::kIds);
  int* s_vz = s_kz + L::kIds;
  float* s_m = reinterpret_cast<float*>(smem + L::kOffMl);     // [WK][R]
  float* s_l = s_m + 128;
  float* s_down = reinterpret_cast<float*>(smem + L::kOffDown);
  uint32_t* s_odd = reinterpret_cast<uint32_t*>(smem + L::kOffOdd);   // [8] drafts, then two flags
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp % WR, wk = warp / WR, qr = lane >> 2, t = lane & 3;
  const int Hkv = a.num_kv_heads, G = a.group, TM = R / G;
  // row tiles of the same keys are neighbours: the second finds them in L2
  const int part = blockIdx.x / rts, rt = blockIdx.x % rts, kvh = blockIdx.y, s = blockIdx.z;

  int q0, n, ctx;
  if (!seq_range(a, s, q0, n, ctx)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) flag_error(PA_DEVERR_QUERY);
    return;
  }
  if (rt * TM >= n || (int64_t)part * a.part_tokens >= ctx) return;
  const int begin = part * a.part_tokens, end = min((int64_t)ctx, (int64_t)begin + a.part_tokens);
  // the stretch at hand: all of a part but for very long ones
  int t0 = begin, t1 = min(end, begin + kPartMax), ntiles = (t1 - t0 + kKeys - 1) / kKeys;
  const int base = ctx - n, rows = min(TM, n - rt * TM);
  const int row0 = q0 + rt * TM;

  if (tid < 10) s_odd[tid] = 0;
  __syncthreads();
  // ---- Q on its way; the part's blocks ----
  // 16 lanes to a row of 128 channels; a row of no token is zero
  constexpr int kQIts = R / (kMmaThreads / 16);
  const int ch = lane & 15;
  uint4 qx[kQIts];
#pragma unroll
  for (int i = 0; i < kQIts; ++i) {
    const int r = (tid >> 4) + i * (kMmaThreads / 16);
    qx[i] = make_uint4(0, 0, 0, 0);
    if (r < rows * G)
      qx[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                ((int64_t)(row0 + r / G) * a.num_q_heads + kvh * G + r % G) * kMmaDim + ch * 8);
  }
  auto load_ids = [&]() {
    const int32_t* bt = a.block_tables + (int64_t)s * a.max_blocks_per_seq + t0 / BS;
    const int nb = (t1 - t0 + BS - 1) / BS;
    // up to the last tile's end; what is not there or cannot be read has id -1 and zeros
    for (int i = tid; i < ntiles * (kKeys / BS); i += kMmaThreads) {
      int p = i < nb ? bt[i] : -1;
      if (i < nb && (p < 0 || p >= a.num_blocks)) {
        flag_error(PA_DEVERR_BLOCK_ID);
        p = -1;
      }
      if constexpr (QUANT) {
        const int64_t bh = (int64_t)max(p, 0) * Hkv + kvh;
        if constexpr (KV == PA_INT8) {
          const int kz = p >= 0 ? a.k_zeros[bh] : 0, vz = p >= 0 ? a.v_zeros[bh] : 0;
          if (!zero_in_range(kz) || !zero_in_range(vz)) {
            flag_error(PA_DEVERR_ZERO);
            p = -1;
          }
          s_kz[i] = p >= 0 ? kz : 0;
          s_vz[i] = p >= 0 ? vz : 0;
        }
        s_ks[i] = p >= 0 ? a.k_scales[bh] : 0.f;
        s_vs[i] = p >= 0 ? a.v_scales[bh] : 0.f;
      }
      s_id[i] = p;
      if (i < nb && p < 0) s_odd[9] = 1;
    }
  };
  load_ids();
  __syncthreads();
  bool any_bad = s_odd[9] != 0;

  // ---- keys: K and V of tile j into stage j % kStages ----
  const uint32_t s0 = tc::smem_u32(smem);
  const int64_t bstride = (int64_t)Hkv * BS * (CPR * 16);
  // a thread's copies are of one chunk, kKeyStep keys apart
  const int c0 = tid % CPR, key00 = tid / CPR;
  constexpr int kKeyStep = kMmaThreads / CPR;
  const int64_t head_off = (int64_t)kvh * BS * (CPR * 16) + c0 * 16;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.k_cache) + head_off;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.v_cache) + head_off;
  auto issue = [&](int j) {
    if (j < ntiles) {
      const uint32_t dk = s0 + (j % L::kStages) * 2 * L::kTileBytes, dv = dk + L::kTileBytes;
      const int live = t1 - t0 - j * kKeys;
      const int* ids = s_id + j * (kKeys / BS);
#pragma unroll
      for (int i = 0; i < kKeys / kKeyStep; ++i) {
        const int key = key00 + i * kKeyStep;
        // a block's rows behind the context are zero too
        const int p = key < live ? ids[key / BS] : -1;
        const int64_t off = (int64_t)max(p, 0) * bstride + (key % BS) * (CPR * 16);
        const int ck = QUANT ? c0 ^ (4 * (key & 1)) : c0 ^ (key & 7), cv = c0 ^ (key & 7);
        copy16(dk + key * CPR * 16 + ck * 16, kbase + off, p >= 0);
        copy16(dv + key * CPR * 16 + cv * 16, vbase + off, p >= 0);
      }
    }
    copies_commit();
  };
#pragma unroll 1
  for (int j = 0; j < L::kStages - 1; ++j) issue(j);

  const uint32_t sQ = tc::smem_u32(smem + L::kOffQ);
#pragma unroll
  for (int i = 0; i < kQIts; ++i) {
    const int r = (tid >> 4) + i * (kMmaThreads / 16);
    uint4 x = qx[i];
    if constexpr (QUANT) {
      uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int eb = (int)((__float_as_uint(amax) >> 23) & 0xff);
      // -113 for the largest bf16; both 2^e and 2^-e stay normal, so rows of subnormals stop at 126
      const int e = amax == 0.f || eb == 0xff ? 0 : min(126, 14 - (eb - 127));
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = pack_f16x2(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
      x = make_uint4(w[0], w[1], w[2], w[3]);
      if (ch == 0) s_down[r] = __uint_as_float((uint32_t)(127 - e) << 23);
    }
    // chunks XORed so that the fragments below are read without conflicts
    *reinterpret_cast<uint4*>(smem + L::kOffQ + r * 256 + ((ch ^ (r & (QUANT ? 1 : 7))) << 4)) = x;
  }
  __syncthreads();

  // A fragments of product step kk (16 channels). Codes: the steps take the channels in the order
  // in which a lane finds them in a K row: step 4 h + j, lane t: 64 h + 16 t + 4 j .. + 3.
  uint32_t qh[HOLD ? MT : 1][HOLD ? 8 : 1][4];
  auto q_bf16 = [&](int mt, int kk, uint32_t (&x)[4]) {
    const int r = wr * 16 * MT + mt * 16 + (lane & 15), c = kk * 2 + (lane >> 4);
    tc::ldsm_x4(sQ + r * 256 + ((c ^ (r & 7)) << 4), x);
  };
  auto q_f16 = [&](int mt, int h, int b, uint32_t (&x0)[4], uint32_t (&x1)[4]) {  // steps 4h + 2b, + 1
    const int r = wr * 16 * MT + mt * 16 + qr, c = h * 8 + 2 * t + b;   // r + 8 has r's parity
    const uint4 u = lds128(sQ + r * 256 + ((c ^ (r & 1)) << 4));
    const uint4 v = lds128(sQ + (r + 8) * 256 + ((c ^ (r & 1)) << 4));
    x0[0] = u.x; x0[1] = v.x; x0[2] = u.y; x0[3] = v.y;
    x1[0] = u.z; x1[1] = v.z; x1[2] = u.w; x1[3] = v.w;
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      if constexpr (QUANT) {
#pragma unroll
        for (int k = 0; k < 4; ++k) q_f16(mt, k >> 1, k & 1, qh[mt][2 * k], qh[mt][2 * k + 1]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) q_bf16(mt, k, qh[mt][k]);
      }
  }

  float o[MT][16][4], m[MT * 2], l[MT * 2], sl2[MT * 2];
#pragma unroll
  for (int i = 0; i < MT * 2; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    sl2[i] = a.scale_log2 * (QUANT ? s_down[wr * 16 * MT + i * 8 + qr] : 1.f);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[mt][i][k] = 0.f;
  // codes: the power of two that a row's V scales are relative to. Rows differ only from the first
  // key on that some of them do not see: in unmasked tiles, which come before, all are alike.
  float vref[MT * 2];
#pragma unroll
  for (int i = 0; i < MT * 2; ++i) vref[i] = 0.f;

  while (true) {
#pragma unroll 1
    for (int j = 0; j < ntiles; ++j) {
      copies_wait<L::kStages - 2>();
      __syncthreads();   // tile j is there, and every warp is done with tile j - 1
      issue(j + L::kStages - 1);
      const uint32_t sK = s0 + (j % L::kStages) * 2 * L::kTileBytes, sV = sK + L::kTileBytes;
      const int key0 = t0 + j * kKeys;
      const bool masked = key0 + kKeys > base || any_bad;
      uint64_t view[MT * 2];
      if (masked) {
        if constexpr (KV != PA_INT8) {
          // A NaN or infinity in a draft's V row would reach rows that do not see it, as 0 times
          // itself: it is taken out here and given back at the end to rows that do see it.
          if (key0 + kKeys > base) {
            const uint32_t vt = sV - s0;
            for (int x = tid; x < kKeys * CPR; x += kMmaThreads) {
              const int key = x / CPR, at = key0 + key;
              if (at < base || at >= ctx) continue;
              uint32_t* w = reinterpret_cast<uint32_t*>(smem + vt + key * CPR * 16 + (x % CPR) * 16);
              bool odd = false;
#pragma unroll 1
              for (int i = 0; i < 4; ++i) {
                uint32_t keep = ~0u;
                if constexpr (QUANT) {
#pragma unroll
                  for (int b = 0; b < 4; ++b)
                    if (((w[i] >> (8 * b)) & 0x7fu) == 0x7fu) keep &= ~(0xffu << (8 * b));
                } else {
                  if ((w[i] & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
                  if ((w[i] & 0x7f800000u) == 0x7f800000u) keep &= 0x0000ffffu;
                }
                if (keep != ~0u) {
                  w[i] &= keep;
                  odd = true;
                }
              }
              if (odd) {
                atomicOr(&s_odd[(at - base) >> 5], 1u << ((at - base) & 31));
                s_odd[8] = 1;
              }
            }
            __syncthreads();
          }
        }
        uint64_t gone = 0;
        if (any_bad) {
#pragma unroll
          for (int b = 0; b < kKeys / BS; ++b)
            if (key0 + b * BS < t1 && s_id[j * (kKeys / BS) + b] < 0) gone |= ((1ull << BS) - 1ull) << (b * BS);
        }
#pragma unroll
        for (int i = 0; i < MT * 2; ++i) {
          const int tok = min((wr * 16 * MT + i * 8 + qr) / G, rows - 1);
          view[i] = tile_view(a, row0 + tok, key0, base, ctx) & ~gone;
        }
      }
#pragma unroll 1
      for (int cc = 0; cc < KW / C; ++cc) {
        const int k0 = wk * KW + cc * C;     // first of the step's keys in the tile
        if (key0 + k0 >= t1) break;          // none of them exists (a warp's view: uniform)
        // ---- S ----
        float sv[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sv[mt][nt][k] = 0.f;
        if constexpr (!QUANT) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t qa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (HOLD) {
#pragma unroll
                for (int k = 0; k < 4; ++k) qa[mt][k] = qh[mt][kk][k];
              } else {
                q_bf16(mt, kk, qa[mt]);
              }
            }
#pragma unroll
            for (int np = 0; np < NT / 2; ++np) {
              uint32_t b[4];
              const int key = k0 + np * 16 + (lane & 7) + ((lane >> 4) << 3);
              const int c = kk * 2 + ((lane >> 3) & 1);
              tc::ldsm_x4(sK + key * 256 + ((c ^ (key & 7)) << 4), b);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                tc::mma16816<false>(sv[mt][2 * np], qa[mt], b[0], b[1]);
                tc::mma16816<false>(sv[mt][2 * np + 1], qa[mt], b[2], b[3]);
              }
            }
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 kc[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int key = k0 + nt * 8 + qr;
              kc[nt] = lds128(sK + key * 128 + (((t + 4 * h) ^ (4 * (key & 1))) << 4));
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint32_t qa[MT][2][4];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                if constexpr (HOLD) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    qa[mt][0][k] = qh[mt][4 * h + 2 * b][k];
                    qa[mt][1][k] = qh[mt][4 * h + 2 * b + 1][k];
                  }
                } else {
                  q_f16(mt, h, b, qa[mt][0], qa[mt][1]);
                }
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t zc = 0;
                if constexpr (KV == PA_INT8) {
                  const float z = 1152.f + (float)s_kz[(j * kKeys + k0 + nt * 8) / BS];
                  zc = pack_f16x2(z, z);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t w = b ? (e ? kc[nt].w : kc[nt].z) : (e ? kc[nt].y : kc[nt].x);
                  uint32_t b0, b1;
                  if constexpr (KV == PA_INT8) {
                    const uint32_t u = w ^ 0x80808080u;
                    b0 = tc::i8x2_to_f16x2(u, 0x4140, zc);
                    b1 = tc::i8x2_to_f16x2(u, 0x4342, zc);
                  } else {
                    b0 = e4m3x2_to_f16x2((uint16_t)(w & 0xffffu));
                    b1 = e4m3x2_to_f16x2((uint16_t)(w >> 16));
                  }
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) tc::mma16816<true>(sv[mt][nt], qa[mt][e], b0, b1);
                }
              }
            }
          }
        }
        // ---- softmax ----
        float ks[NT], vs[NT], rv[MT * 2];
        if constexpr (QUANT) {
          float vmax = 0.f, seen[MT * 2];   // the largest |V scale|, of all keys and of a row's
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int b = (j * kKeys + k0 + nt * 8) / BS;
            ks[nt] = s_ks[b];
            vs[nt] = s_vs[b];
            vmax = fmaxf(vmax, fabsf(vs[nt]));
          }
          bool up = vmax > vref[0];   // unmasked: of all rows
#pragma unroll
          for (int i = 0; i < MT * 2; ++i) seen[i] = vmax;
          if (masked) {
            up = false;
#pragma unroll
            for (int i = 0; i < MT * 2; ++i) {
              const uint32_t v = (uint32_t)(view[i] >> k0);
              seen[i] = 0.f;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                if ((v >> (8 * nt)) & 0xffu) seen[i] = fmaxf(seen[i], fabsf(vs[nt]));
              up = up || seen[i] > vref[i];
            }
          }
          if (__any_sync(0xffffffffu, up)) {
            // The next power of two, within a range in which 2^7 over it is one too; what was
            // summed against a lower one is scaled down.
#pragma unroll
            for (int i = 0; i < MT * 2; ++i) {
              if (!(seen[i] > vref[i])) continue;
              const int e = max(8, min(253, (int)((__float_as_uint(seen[i]) >> 23) & 0xff) + 1));
              const float now = fmaxf(vref[i], __uint_as_float((uint32_t)e << 23));
              const float down = vref[i] / now;
              vref[i] = now;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                o[i >> 1][k][2 * (i & 1)] *= down;
                o[i >> 1][k][2 * (i & 1) + 1] *= down;
              }
            }
          }
          // 2^7 / v_ref by its exponent; 0: every V scale so far is
#pragma unroll
          for (int i = 0; i < MT * 2; ++i)
            rv[i] = vref[i] > 0.f ? __uint_as_float((261u << 23) - __float_as_uint(vref[i])) : 0.f;
        }
        uint32_t pf[MT][NT / 2][4];
        // P against the standing reference, without looking for the maximum: right when no lane's
        // sum passes 2^8 (a score that outgrew the reference, or is no number, makes one)
        auto weights = [&](int i, float f0, bool scaled) {
          const float ref = m[i] == -INFINITY && scaled ? 0.f : -m[i];
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float f = scaled ? 1.f : QUANT ? f0 * ks[nt] : f0;
            float p0 = fast_exp2(fmaf(sv[i >> 1][nt][2 * (i & 1)], f, ref));
            float p1 = fast_exp2(fmaf(sv[i >> 1][nt][2 * (i & 1) + 1], f, ref));
            sum += p0 + p1;
            if constexpr (QUANT) {   // P carries its block's V scale; a key that is not seen, none
              const float w = vs[nt] * rv[scaled ? i : 0];   // rows are alike in unmasked tiles
              p0 = scaled && p0 == 0.f ? 0.f : p0 * w;
              p1 = scaled && p1 == 0.f ? 0.f : p1 * w;
            }
            pf[i >> 1][nt >> 1][2 * (nt & 1) + (i & 1)] = QUANT ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
          return sum;
        };
        bool fast = false;
        if (!masked) {
          float sum[MT * 2];
          bool good = true;
#pragma unroll
          for (int i = 0; i < MT * 2; ++i) {
            sum[i] = weights(i, sl2[i], false);
            good = good && sum[i] <= 256.f;
          }
          fast = __all_sync(0xffffffffu, good);
          if (fast) {
#pragma unroll
            for (int i = 0; i < MT * 2; ++i) l[i] += sum[i];
          }
        }
        if (!fast) {
          float alpha[MT * 2];
          bool grown = false;
#pragma unroll
          for (int i = 0; i < MT * 2; ++i) {
            const uint32_t v = masked ? (uint32_t)(view[i] >> (k0 + 2 * t)) : ~0u;
            float mx = m[i];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float f = QUANT ? sl2[i] * ks[nt] : sl2[i];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& x = sv[i >> 1][nt][2 * (i & 1) + e];
                x *= f;
                if (masked && !((v >> (nt * 8 + e)) & 1u)) x = -INFINITY;
                mx = fmaxf(mx, x);
              }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            alpha[i] = 1.f;
            if (mx > m[i] + 8.f) {   // lazy: P stays at or below 2^8 otherwise
              alpha[i] = fast_exp2(m[i] - mx);
              m[i] = mx;
              grown = true;
            }
          }
          if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[mt][i][k] *= alpha[mt * 2 + (k >> 1)];
          }
#pragma unroll
          for (int i = 0; i < MT * 2; ++i) l[i] = l[i] * alpha[i] + weights(i, 1.f, true);
        }
        // ---- O += P V ----
#pragma unroll
        for (int kp = 0; kp < NT / 2; ++kp) {
          const int key = k0 + kp * 16 + (lane & 15);
          uint32_t z0 = 0, z1 = 0;
          if constexpr (KV == PA_INT8) {
            const int b = (j * kKeys + k0 + kp * 16) / BS;
            const float f0 = 1152.f + (float)s_vz[b];
            const float f1 = 1152.f + (float)s_vz[BS == 8 ? b + 1 : b];
            z0 = pack_f16x2(f0, f0);
            z1 = pack_f16x2(f1, f1);
          }
          if constexpr (!QUANT) {
#pragma unroll
            for (int cb = 0; cb < 8; ++cb) {   // 16 channels
              uint32_t b[4];
              tc::ldsm_x4_t(sV + key * 256 + (((cb * 2 + (lane >> 4)) ^ (key & 7)) << 4), b);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                tc::mma16816<false>(o[mt][2 * cb], pf[mt][kp], b[0], b[1]);
                tc::mma16816<false>(o[mt][2 * cb + 1], pf[mt][kp], b[2], b[3]);
              }
            }
          } else {
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {   // 32 channels
              uint32_t w[4];   // (keys 0-7, 8-15) x (channels 0-15, 16-31); lane: two keys, two channels
              tc::ldsm_x4_t(sV + key * 128 + (((cb * 2 + (lane >> 4)) ^ (key & 7)) << 4), w);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t ev[2], od[2];   // the even and the odd channel of both keys
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t u = __byte_perm(w[2 * x + y], 0, 0x3120);
                  if constexpr (KV == PA_INT8) {
                    const uint32_t ub = u ^ 0x80808080u;
                    ev[y] = tc::i8x2_to_f16x2(ub, 0x4140, y ? z1 : z0);
                    od[y] = tc::i8x2_to_f16x2(ub, 0x4342, y ? z1 : z0);
                  } else {
                    ev[y] = e4m3x2_to_f16x2((uint16_t)(u & 0xffffu));
                    od[y] = e4m3x2_to_f16x2((uint16_t)(u >> 16));
                  }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  tc::mma16816<true>(o[mt][4 * cb + 2 * x], pf[mt][kp], ev[0], ev[1]);
                  tc::mma16816<true>(o[mt][4 * cb + 2 * x + 1], pf[mt][kp], od[0], od[1]);
                }
              }
            }
          }
        }
      }
    }
    copies_wait<0>();
    __syncthreads();   // stages and Q are free: the next stretch's keys, or the warps join there
    if (t1 == end) break;
    t0 = t1;
    t1 = min(end, t0 + kPartMax);
    ntiles = (t1 - t0 + kKeys - 1) / kKeys;
    load_ids();
    __syncthreads();
    any_bad = s_odd[9] != 0;
#pragma unroll 1
    for (int j = 0; j < L::kStages - 1; ++j) issue(j);
  }

  float* comb = reinterpret_cast<float*>(smem);   // [WK][R][kCombRow]
#pragma unroll
  for (int i = 0; i < MT * 2; ++i) {
    float x = l[i];
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    const int r = wr * 16 * MT + i * 8 + qr;
    if (t == 0) {
      s_m[wk * R + r] = m[i];
      s_l[wk * R + r] = x;
    }
    float* d = comb + (wk * R + r) * kCombRow;
    const int k = 2 * (i & 1);
    const float unit = QUANT ? vref[i] * (1.f / 128.f) : 1.f;
#pragma unroll
    for (int cb = 0; cb < 8; ++cb) {
      float(&e)[4] = o[i >> 1][2 * cb];
      float(&f)[4] = o[i >> 1][2 * cb + 1];
      if constexpr (QUANT) {
        *reinterpret_cast<float4*>(d + cb * 16 + 4 * t) =
            make_float4(e[k] * unit, f[k] * unit, e[k + 1] * unit, f[k + 1] * unit);
      } else {
        *reinterpret_cast<float2*>(d + cb * 16 + 2 * t) = make_float2(e[k], e[k + 1]);
        *reinterpret_cast<float2*>(d + cb * 16 + 8 + 2 * t) = make_float2(f[k], f[k + 1]);
      }
    }
  }
  __syncthreads();
  const bool whole = ctx <= a.part_tokens, odd = KV != PA_INT8 && s_odd[8] != 0;
  for (int x = tid; x < rows * G * 32; x += kMmaThreads) {
    const int r = x >> 5, c = (x & 31) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WK; ++w) M = fmaxf(M, s_m[w * R + r]);
    const float ref = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float f = fast_exp2(s_m[w * R + r] - ref);
      const float4 v = *reinterpret_cast<const float4*>(comb + (w * R + r) * kCombRow + c);
      sum = fmaf(f, s_l[w * R + r], sum);
      y.x = fmaf(f, v.x, y.x); y.y = fmaf(f, v.y, y.y); y.z = fmaf(f, v.z, y.z); y.w = fmaf(f, v.w, y.w);
    }
    const int64_t trow = row0 + r / G, row = trow * a.num_q_heads + kvh * G + r % G;
    if (odd) {   // rare
      float* e = &y.x;
#pragma unroll 1
      for (int d = 0; d < n; ++d) {
        const int key = base + d;
        if (key < begin || key >= end || !((s_odd[d >> 5] >> (d & 31)) & 1u) ||
            !((a.tree_mask[trow * a.mask_words + (d >> 5)] >> (d & 31)) & 1u))
          continue;
        const int64_t blk = a.block_tables[(int64_t)s * a.max_blocks_per_seq + key / BS];
        const int64_t at = ((blk * Hkv + kvh) * BS + key % BS) * kMmaDim + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (!QUANT) {
            const float v = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.v_cache)[at + k] << 16);
            if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) e[k] += v;
          } else if ((static_cast<const uint8_t*>(a.v_cache)[at + k] & 0x7f) == 0x7f) {
            e[k] = __uint_as_float(0x7fc00000u);
          }
        }
      }
    }
    if (whole) {
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kMmaDim + c) =
          make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
      if (c == 0 && a.lse_out != nullptr)
        a.lse_out[row] = sum != 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
    } else {
      const int64_t pr = row * a.parts + part;
      *reinterpret_cast<float4*>(a.part_acc + pr * kMmaDim + c) = y;
      if (c == 0) { a.part_m[pr] = M; a.part_l[pr] = sum; }
    }
  }
}

template <int BS, pa_dtype KV, int MT, int WR>
inline cudaError_t launch_mma_wr(const TreeArgs& a, cudaStream_t st) {
  using L = MmaLayout<KV, MT, WR>;
  static_assert(L::kCtas * (L::kSmem + 1024) <= 228 * 1024, "CTAs on an SM");
  static tc::DeviceCache slots;
  int per_sm = 0;
  cudaError_t e = tc::resident_per_sm(tree_mma_kernel<BS, KV, MT, WR>, kMmaThreads, L::kSmem, slots, &per_sm);
  if (e != cudaSuccess) return e;
  const int tm = L::kRowsT / a.group, rts = (a.max_query_len + tm - 1) / tm;
  e = launch_pdl(tree_mma_kernel<BS, KV, MT, WR>, dim3(a.parts * rts, a.num_kv_heads, a.num_seqs),
                 dim3(kMmaThreads), L::kSmem, st, a, rts);
  if (e != cudaSuccess || a.parts == 1) return e;
  return launch_reduce<kMmaDim>(a, st);
}

// Rows of a tile: as many as the longest draft fills, 32, 64 or 128.
inline int mma_rows(int max_query_len, int group) {
  const int most = max_query_len * group;
  return most <= 32 ? 32 : most <= 64 ? 64 : 128;
}

template <int BS, pa_dtype KV>
inline cudaError_t launch_mma_bs(const TreeArgs& a, cudaStream_t st) {
  switch (mma_rows(a.max_query_len, a.group)) {
    case 32: return launch_mma_wr<BS, KV, 1, 2>(a, st);
    case 64: return launch_mma_wr<BS, KV, 1, 4>(a, st);
    default: return launch_mma_wr<BS, KV, 2, 4>(a, st);
  }
}

template <pa_dtype KV>
inline cudaError_t launch_mma(const TreeArgs& a, cudaStream_t st) {
  if (a.block_size == 8) return launch_mma_bs<8, KV>(a, st);
  if (a.block_size == 32) return launch_mma_bs<32, KV>(a, st);
  return launch_mma_bs<16, KV>(a, st);
}

}  // namespace tree
}  // namespace pa
