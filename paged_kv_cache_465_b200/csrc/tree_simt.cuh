// Attention of drafted tokens over the paged cache on the CUDA cores (fp32 FMA): every
// supported type, head dimension and group; the path of the shapes that the tensor-core
// kernel (tree_mma.cuh) does not take, and the reference-precision one.
//
// One CTA of 4 warps per (token row, kv head, part of the context), the row's G query heads
// together. Warps step through 16-key sub-tiles as the decode kernel does, with two
// differences: keys behind the committed context are read only where the row's mask has
// their bit, and a part's result goes to a workspace indexed by token row. Every row reads
// its whole context again (L2 serves the rows of one sequence), so the kernel is bound by
// arithmetic and L2, not by HBM.
#pragma once

#include "decode_simt.cuh"

namespace pa {
namespace tree {

struct TreeArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;  // [S][max_blocks_per_seq]
  const int32_t* context_lens;  // [S], rows of the step included
  const int32_t* query_start;   // [S + 1]
  const uint32_t* tree_mask;    // [T][mask_words]
  void* out;                    // [T][Hq][d]
  float* lse_out;               // [T][Hq] or null
  const float* k_scales;
  const float* v_scales;
  const int32_t* k_zeros;
  const int32_t* v_zeros;
  float scale_log2;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, group;
  int max_blocks_per_seq, num_blocks, block_size, mask_words;
  int max_context_len, max_query_len;
  pa_dtype q_dtype, out_dtype;
  // parts of the context
  float* part_m;                // [T][Hq][parts]
  float* part_l;
  float* part_acc;              // [T][Hq][parts][d]
  int part_tokens, parts;
  int reduce_heads;             // of a warp of the joining kernel
  int direct;                   // rows of one part are written by the kernel that computes them
};

// Rows of sequence s: q0 .. q0 + n - 1, the last n of ctx positions. False when the ranges
// do not fit together.
__device__ __forceinline__ bool seq_range(const TreeArgs& a, int s, int& q0, int& n, int& ctx) {
  q0 = a.query_start[s];
  const int q1 = a.query_start[s + 1];
  ctx = a.context_lens[s];
  n = q1 - q0;
  return q0 >= 0 && q1 >= q0 && q1 <= a.num_tokens && n <= ctx && ctx <= a.max_context_len &&
         n <= a.max_query_len;
}

// The last sequence that begins at or before row t, by a 32-way search of the whole warp.
__device__ __forceinline__ int seq_of_row(const int32_t* query_start, int num_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int p = lo + lane * step;
    const unsigned v =
        __ballot_sync(0xffffffffu, lane == 0 || (p < hi && query_start[p] <= t));
    lo += (31 - __clz(v)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

template <pa_dtype KV, int D, int GP>
__global__ void __launch_bounds__(kSimtWarps * 32) tree_simt_kernel(const TreeArgs a) {
  constexpr int ES = KvTraits<KV>::bytes;
  constexpr int HALF = D / 2, EPC = 16 / ES, CH = HALF / EPC, NV = D / 32, QROW = D + 4;
  __shared__ __align__(16) float sq[GP * QROW];
  __shared__ __align__(16) float sp[kSimtWarps][kSub][GP];
  __shared__ float sm[kSimtWarps][GP], sl[kSimtWarps][GP];
  __shared__ __align__(16) float sacc[kSimtWarps][GP][D];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, kvh = blockIdx.y, part = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.group;
  const int s = seq_of_row(a.query_start, a.num_seqs, t);
  int q0, n, ctx;
  const bool ok = seq_range(a, s, q0, n, ctx);
  if (!ok || t < q0 || t >= q0 + n) {  // a row of no sequence is left alone
    if (!ok && threadIdx.x == 0) flag_error(PA_DEVERR_QUERY);
    return;
  }
  const int base = ctx - n;
  const int t0 = part * a.part_tokens;
  if (t0 >= ctx && part > 0) return;
  const int t1 = min(ctx, t0 + a.part_tokens);
  const uint32_t* mask = a.tree_mask + (int64_t)t * a.mask_words;

  for (int i = threadIdx.x; i < GP * D; i += blockDim.x) {
    const int g = i / D, d = i % D;
    float x = 0.f;
    if (g < G) x = load_q(a.q, a.q_dtype, ((int64_t)t * a.num_q_heads + kvh * G + g) * D + d) *
                   a.scale_log2;
    sq[g * QROW + d + (d >= HALF ? 4 : 0)] = x;
  }
  __syncthreads();

  float m[GP], lsum[GP], acc[GP][NV];
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    m[g] = -INFINITY;
    lsum[g] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[g][j] = 0.f;
  }
  const int tok = lane & 15, half = lane >> 4, BS = a.block_size;
  const int32_t* bt = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.k_cache);
  const uint8_t* vbase = static_cast<const uint8_t*>(a.v_cache);

  for (int c = t0 / kSub + warp; c < (t1 + kSub - 1) / kSub; c += kSimtWarps) {
    const int key = c * kSub + tok;
    bool see = key < t1;
    if (see && key >= base) {
      const int j = key - base;
      see = j < 32 * a.mask_words && ((mask[j >> 5] >> (j & 31)) & 1u);
    }
    int64_t row = -1;  // byte offset of the key's K / V row; -1: not read
    float ks = 1.f, vs = 1.f, kz = 0.f, vz = 0.f;
    if (see) {
      const int phys = bt[key / BS];
      if (phys < 0 || phys >= a.num_blocks) {
        if (half == 0) flag_error(PA_DEVERR_BLOCK_ID);
        see = false;
      } else {
        const int64_t bh = (int64_t)phys * a.num_kv_heads + kvh;
        row = (bh * BS + key % BS) * D * ES;
        if constexpr (KV == PA_FP8_E4M3 || KV == PA_INT8) {
          ks = a.k_scales[bh];
          vs = a.v_scales[bh];
        }
        if constexpr (KV == PA_INT8) {
          const int kzi = a.k_zeros[bh], vzi = a.v_zeros[bh];
          if (!zero_in_range(kzi) || !zero_in_range(vzi)) {
            if (half == 0) flag_error(PA_DEVERR_ZERO);
            see = false;
            row = -1;
          }
          kz = (float)kzi;
          vz = (float)vzi;
        }
      }
    }
    if (!__any_sync(0xffffffffu, see)) continue;
    float sc[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) sc[g] = 0.f;
    if (see) {
      const uint4* krow = reinterpret_cast<const uint4*>(kbase + row + half * HALF * ES);
#pragma unroll
      for (int cc = 0; cc < CH; ++cc) {
        float kx[EPC];
        unpack16<KV>(__ldg(krow + cc), kx);
        if constexpr (KV == PA_INT8) {
#pragma unroll
          for (int e = 0; e < EPC; ++e) kx[e] -= kz;
        }
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          const float* qr = sq + g * QROW + half * (HALF + 4) + cc * EPC;
#pragma unroll
          for (int e = 0; e < EPC; ++e) sc[g] = fmaf(qr[e], kx[e], sc[g]);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      float z = sc[g] + __shfl_xor_sync(0xffffffffu, sc[g], 16);
      z = see ? z * ks : -INFINITY;
      float bm = z;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
      const float mn = fmaxf(m[g], bm);
      // nothing but -inf so far (scores can underflow to it): the weights are 0, not NaN
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = fast_exp2(m[g] - ref);
      m[g] = mn;
      const float p = see ? fast_exp2(z - ref) : 0.f;
      lsum[g] = lsum[g] * alpha + (half == 0 ? p : 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[g][j] *= alpha;
      if (half == 0) sp[warp][tok][g] = see ? p * vs : 0.f;
    }
    __syncwarp();
    // rows of V that this row does not see are not read: they may hold anything
#pragma unroll 4
    for (int tt = 0; tt < kSub; ++tt) {
      const int64_t r = __shfl_sync(0xffffffffu, row, tt);
      if (r < 0) continue;
      float vx[NV];
      load_vslice<KV, D>(vbase + r, lane, vx);
      if constexpr (KV == PA_INT8) {
        const float z = __shfl_sync(0xffffffffu, vz, tt);
#pragma unroll
        for (int j = 0; j < NV; ++j) vx[j] -= z;
      }
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float pg = sp[warp][tt][g];
#pragma unroll
        for (int j = 0; j < NV; ++j) acc[g][j] = fmaf(pg, vx[j], acc[g][j]);
      }
    }
    __syncwarp();
  }

#pragma unroll
  for (int g = 0; g < GP; ++g) {
    float l = lsum[g];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) { sm[warp][g] = m[g]; sl[warp][g] = l; }
#pragma unroll
    for (int j = 0; j < NV; ++j) sacc[warp][g][lane * NV + j] = acc[g][j];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += blockDim.x) {
    const int g = i / D, d = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) M = fmaxf(M, sm[w][g]);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, A = 0.f;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) {
      const float f = fast_exp2(sm[w][g] - ref);
      L = fmaf(f, sl[w][g], L);
      A = fmaf(f, sacc[w][g][d], A);
    }
    const int64_t row = (int64_t)t * a.num_q_heads + kvh * G + g;
    if (a.parts == 1) {
      store_out(a.out, a.out_dtype, row * D + d, L != 0.f ? A / L : 0.f);
      if (d == 0 && a.lse_out != nullptr)
        a.lse_out[row] = L != 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
    } else {
      const int64_t pr = row * a.parts + part;
      a.part_acc[pr * D + d] = A;
      if (d == 0) { a.part_m[pr] = M; a.part_l[pr] = L; }
    }
  }
}

// Joins the parts, in order: one warp per (token row, a.reduce_heads query heads). Bound by latency:
// rows of one part leave as soon as their sequence is known.

template <int D>
__global__ void __launch_bounds__(128) tree_reduce_kernel(const TreeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, groups = (a.num_q_heads + a.reduce_heads - 1) / a.reduce_heads;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)a.num_tokens * groups) return;
  const int t = (int)(w / groups), h0 = (int)(w % groups) * a.reduce_heads;
  const int s = seq_of_row(a.query_start, a.num_seqs, t);
  int q0, n, ctx;
  if (!seq_range(a, s, q0, n, ctx) || t < q0 || t >= q0 + n) return;
  const int np = (ctx + a.part_tokens - 1) / a.part_tokens;
  if (a.direct && np == 1) return;
#pragma unroll 1
  for (int h = h0; h < min(a.num_q_heads, h0 + a.reduce_heads); ++h) {
    const int64_t row = (int64_t)t * a.num_q_heads + h;
    const float* pm = a.part_m + row * a.parts;
    const float* pl = a.part_l + row * a.parts;
    float M = -INFINITY;
    for (int p = lane; p < np; p += 32) M = fmaxf(M, pm[p]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float acc[D / 32], L = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] = 0.f;
#pragma unroll 4
    for (int p = 0; p < np; ++p) {
      const float f = fast_exp2(pm[p] - ref);
      L = fmaf(f, pl[p], L);
      const float* src = a.part_acc + (row * a.parts + p) * D;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) acc[j] = fmaf(f, src[lane + 32 * j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      store_out(a.out, a.out_dtype, row * D + lane + 32 * j, L != 0.f ? acc[j] / L : 0.f);
    if (lane == 0 && a.lse_out != nullptr)
      a.lse_out[row] = L != 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
  }
}

template <int D>
inline cudaError_t launch_reduce(TreeArgs a, cudaStream_t st) {
  // Four heads to a warp where there are rows enough to fill the SMs several times over (256
  // sequences, most of one part: 16400 CTAs of one head to a warp took 19 us).
  a.reduce_heads = (int64_t)a.num_tokens * a.num_q_heads >= 32768 ? 4 : 1;
  const int64_t warps = (int64_t)a.num_tokens * ((a.num_q_heads + a.reduce_heads - 1) / a.reduce_heads);
  return launch_pdl(tree_reduce_kernel<D>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, a);
}

}  // namespace tree
}  // namespace pa
