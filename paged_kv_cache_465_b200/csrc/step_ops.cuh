// The bookkeeping of a drafted step on the GPU: block tables, slot map, positions and
// ancestor masks from request lengths (paged_build_step), blocks back to the free queue
// (paged_release_blocks), the accepted path of a draft tree (tree_verify) and its K/V moved
// behind the context (compact_accepted).
//
// All of them move a few hundred KB at most, so launch and dependent reads bound them, not
// bandwidth. The first two need sums over all sequences: every CTA forms them itself (a
// sequence is three ints, and L2 serves them), which costs less than a second launch and
// leaves no scratch that two calls could share.
#pragma once

#include "common.cuh"

namespace pa {
namespace step {

constexpr int kMaxTree = 256;      // rows of one draft tree
constexpr int kMaxWords = kMaxTree / 32;

struct BuildArgs {
  const int32_t* context_lens;
  const int32_t* new_lens;
  const int32_t* blocks_held;
  const int32_t* parents;
  int32_t* block_tables;
  const int32_t* free_blocks;
  const int32_t* queue_state;
  int32_t* total_lens;
  int32_t* query_start;
  int32_t* blocks_held_out;
  int32_t* queue_state_out;
  int64_t* slot_mapping;
  int32_t* positions;
  uint32_t* tree_mask;
  int32_t* status;
  int num_seqs, max_blocks_per_seq, block_size, num_blocks, free_capacity, max_tokens, mask_words;
};

// Exclusive sums of x and y over the CTA's threads in order, their totals, and the OR of
// `bits`, in 64 bits: 65535 sequences of up to 2^31 tokens cannot wrap. W warps; the
// scratch arrays hold one entry per warp.
template <int W>
__device__ __forceinline__ void scan2(int64_t& x, int64_t& y, unsigned& bits, int64_t& xt,
                                      int64_t& yt, int64_t (&sx)[W], int64_t (&sy)[W],
                                      unsigned (&sb)[W]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, ix, o), b = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) { ix += a; iy += b; }
  }
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (lane == 31) { sx[warp] = ix; sy[warp] = iy; }
  if (lane == 0) sb[warp] = bits;
  __syncthreads();
  // every warp sums the warps' totals itself (W <= 32): one barrier
  int64_t wx = lane < W ? sx[lane] : 0, wy = lane < W ? sy[lane] : 0;
  bits = __reduce_or_sync(0xffffffffu, lane < W ? sb[lane] : 0u);
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, wx, o), b = __shfl_up_sync(0xffffffffu, wy, o);
    if (lane >= o) { wx += a; wy += b; }
  }
  xt = __shfl_sync(0xffffffffu, wx, W - 1);
  yt = __shfl_sync(0xffffffffu, wy, W - 1);
  const int64_t px = __shfl_sync(0xffffffffu, wx, (warp + 31) & 31);
  const int64_t py = __shfl_sync(0xffffffffu, wy, (warp + 31) & 31);
  x = ix - x + (warp > 0 ? px : 0);
  y = iy - y + (warp > 0 ? py : 0);
}

__device__ __forceinline__ int ceil_div64(int64_t a, int b) { return (int)((a + b - 1) / b); }

// New blocks of a sequence of c cached and n new tokens that holds h blocks; the PA_DEVERR
// bits of what is wrong with it.
__device__ __forceinline__ unsigned seq_need(const BuildArgs& a, int c, int n, int h, int& need) {
  need = 0;
  const int64_t cap = (int64_t)a.max_blocks_per_seq * a.block_size;
  if (c < 0 || n < 0 || h < 0 || h > a.max_blocks_per_seq || (int64_t)c + n > cap ||
      h < ceil_div64(c, a.block_size))
    return PA_DEVERR_CONTEXT;
  if (a.tree_mask != nullptr && n > 32 * a.mask_words) return PA_DEVERR_TREE;
  need = max(0, ceil_div64((int64_t)c + n, a.block_size) - h);
  return 0;
}

// A step's lengths do not exceed an int together (max_tokens is one), but a long prompt or
// many sequences may: the sums are 64-bit. One CTA per 1024 token rows, one thread per row;
// each CTA scans all sequences (thread t takes a run of consecutive ones), marks in shared
// memory where the sequences that reach into its rows begin, and a max-scan over the marks
// tells every row its sequence. Row, table and ring entries are then independent. Only CTA
// 0 writes what there is one of per sequence.
constexpr int kBuildThreads = 1024;

__global__ void __launch_bounds__(kBuildThreads) build_step_kernel(const BuildArgs a) {
  constexpr int W = kBuildThreads / 32;
  __shared__ int64_t sx[W], sy[W];
  __shared__ unsigned sb[W];
  __shared__ int mark_seq[kBuildThreads], mark_qs[kBuildThreads], mark_last[W];
  __shared__ int64_t mark_off[kBuildThreads];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.num_seqs + kBuildThreads - 1) / kBuildThreads;
  const int s0 = min(a.num_seqs, tid * per), s1 = min(a.num_seqs, s0 + per);
  const int head = a.queue_state[0], count = a.queue_state[1];
  int64_t n_sum = 0, b_sum = 0;
  unsigned bits = 0;
  for (int s = s0; s < s1; ++s) {
    int need;
    const int n = a.new_lens[s];
    bits |= seq_need(a, a.context_lens[s], n, a.blocks_held[s], need);
    n_sum += n;
    b_sum += need;
  }
  int64_t n_total, b_total;
  scan2<W>(n_sum, b_sum, bits, n_total, b_total, sx, sy, sb);
  if (bits == 0) {  // the sums mean something
    if (n_total > a.max_tokens) bits |= PA_DEVERR_QUERY;
    if (head < 0 || head >= a.free_capacity || count < 0 || count > a.free_capacity)
      bits |= PA_DEVERR_QUEUE;
    else if (b_total > count)
      bits |= PA_DEVERR_BLOCKS;
  }
  const bool ok = bits == 0;

  if (blockIdx.x == 0) {
    int64_t qs = n_sum;
    for (int s = s0; s < s1; ++s) {
      const int c = a.context_lens[s], n = a.new_lens[s], h = a.blocks_held[s];
      int need = 0;
      if (ok) seq_need(a, c, n, h, need);
      a.query_start[s] = ok ? (int)qs : 0;
      a.total_lens[s] = ok ? c + n : c;
      a.blocks_held_out[s] = h + need;
      qs += n;
    }
    if (tid == 0) {
      a.query_start[a.num_seqs] = ok ? (int)n_total : 0;
      a.queue_state_out[0] = ok ? (int)((head + b_total) % a.free_capacity) : head;
      a.queue_state_out[1] = ok ? (int)(count - b_total) : count;
      if (a.status != nullptr) a.status[0] = (int)bits;
      if (!ok) flag_error(bits);
    }
  }

  // ---- which sequence each of the CTA's rows belongs to ----
  const int64_t t0 = (int64_t)blockIdx.x * kBuildThreads;
  mark_seq[tid] = -1;
  __syncthreads();
  if (ok) {
    int64_t qs = n_sum, off = b_sum;
    for (int s = s0; s < s1 && qs < t0 + kBuildThreads; ++s) {
      const int n = a.new_lens[s];
      int need;
      seq_need(a, a.context_lens[s], n, a.blocks_held[s], need);
      if (n > 0 && qs + n > t0) {
        const int m = qs > t0 ? (int)(qs - t0) : 0;
        mark_seq[m] = s;
        mark_qs[m] = (int)qs;
        mark_off[m] = off;
      }
      qs += n;
      off += need;
    }
  }
  __syncthreads();
  int m = mark_seq[tid] >= 0 ? tid : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m = max(m, v);
  }
  if (lane == 31) mark_last[warp] = m;
  __syncthreads();
  // the last mark of the warps before this one
  const int before = __reduce_max_sync(0xffffffffu, lane < warp ? mark_last[lane] : -1);
  m = max(m, before);

  const int64_t t = t0 + tid;
  if (t >= a.max_tokens) return;
  int64_t slot = -1;
  int pos_out = 0;
  uint32_t bitsm[kMaxWords];
#pragma unroll
  for (int w = 0; w < kMaxWords; ++w) bitsm[w] = 0;
  if (m >= 0 && t < n_total) {
    const int s = mark_seq[m], q0 = mark_qs[m];
    const int i = (int)(t - q0), c = a.context_lens[s], held = a.blocks_held[s];
    const int pos = c + i, blk = pos / a.block_size, off = pos - blk * a.block_size;
    int32_t* row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
    int id;
    if (blk < held) {
      id = row[blk];
    } else {
      const int64_t at = head + mark_off[m] + (blk - held);  // below twice the ring's size
      id = a.free_blocks[at < a.free_capacity ? at : at - a.free_capacity];
      // held blocks cover the context, so a fresh block's first token is one of this step's
      if (off == 0) row[blk] = id;
    }
    if (id < 0 || id >= a.num_blocks) flag_error(PA_DEVERR_BLOCK_ID);
    else slot = (int64_t)id * a.block_size + off;
    if (a.parents == nullptr) {
      pos_out = pos;
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w)
        bitsm[w] = i >= 32 * w + 31 ? 0xffffffffu : (i < 32 * w ? 0u : (2u << (i - 32 * w)) - 1u);
    } else if (a.positions != nullptr || a.tree_mask != nullptr) {
      int cur = i, depth = 0;
      while (true) {  // ends: every step goes to a smaller index
#pragma unroll
        for (int w = 0; w < kMaxWords; ++w)
          if ((cur >> 5) == w) bitsm[w] |= 1u << (cur & 31);
        const int p = a.parents[q0 + cur];
        if (p < 0 || p >= cur) {
          if (p != -1) flag_error(PA_DEVERR_TREE);
          break;
        }
        cur = p;
        ++depth;
      }
      pos_out = c + depth;
    }
  }
  a.slot_mapping[t] = slot;
  if (a.positions != nullptr) a.positions[t] = pos_out;
  if (a.tree_mask != nullptr) {
#pragma unroll
    for (int w = 0; w < kMaxWords; ++w)
      if (w < a.mask_words) a.tree_mask[t * a.mask_words + w] = bitsm[w];
  }
}

struct ReleaseArgs {
  const int32_t* keep_lens;
  const int32_t* blocks_held;
  const int32_t* block_tables;
  int32_t* free_blocks;
  const int32_t* queue_state;
  int32_t* blocks_held_out;
  int32_t* queue_state_out;
  int32_t* status;
  int num_seqs, max_blocks_per_seq, block_size, free_capacity, seqs_per_cta;
};

// One CTA per `seqs_per_cta` sequences, one warp per sequence at a time; every CTA scans all
// sequences (as above) and keeps the queue offsets of its own.
constexpr int kReleaseThreads = 512, kReleaseSeqs = 512;

__global__ void __launch_bounds__(kReleaseThreads) release_blocks_kernel(const ReleaseArgs a) {
  constexpr int W = kReleaseThreads / 32;
  __shared__ int64_t sx[W], sy[W];
  __shared__ unsigned sb[W];
  __shared__ int64_t s_off[kReleaseSeqs];
  __shared__ int s_kept[kReleaseSeqs], s_held[kReleaseSeqs];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.num_seqs + kReleaseThreads - 1) / kReleaseThreads;
  const int s0 = min(a.num_seqs, tid * per), s1 = min(a.num_seqs, s0 + per);
  const int head = a.queue_state[0], count = a.queue_state[1];
  int64_t back = 0, none = 0;
  unsigned bits = 0;
  auto kept_of = [&](int s, int h) { return min(h, ceil_div64(a.keep_lens[s], a.block_size)); };
  for (int s = s0; s < s1; ++s) {
    const int h = a.blocks_held[s];
    if (a.keep_lens[s] < 0 || h < 0 || h > a.max_blocks_per_seq) bits |= PA_DEVERR_CONTEXT;
    else back += h - kept_of(s, h);
  }
  int64_t total, unused;
  scan2<W>(back, none, bits, total, unused, sx, sy, sb);
  if (bits == 0 && (head < 0 || head >= a.free_capacity || count < 0 ||
                    count + total > a.free_capacity))
    bits |= PA_DEVERR_QUEUE;
  const bool ok = bits == 0;
  const int f0 = blockIdx.x * a.seqs_per_cta, f1 = min(a.num_seqs, f0 + a.seqs_per_cta);
  for (int s = s0; s < s1; ++s) {
    const int h = a.blocks_held[s], kept = ok ? kept_of(s, h) : h;
    if (s >= f0 && s < f1) {
      a.blocks_held_out[s] = kept;
      s_off[s - f0] = back;
      s_kept[s - f0] = kept;
      s_held[s - f0] = h;
    }
    back += h - kept;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.queue_state_out[0] = head;
    a.queue_state_out[1] = ok ? (int)(count + total) : count;
    if (a.status != nullptr) a.status[0] = (int)bits;
    if (!ok) flag_error(bits);
  }
  __syncthreads();
  if (!ok) return;
  for (int k = warp; k < f1 - f0; k += W) {
    const int kept = s_kept[k], n = s_held[k] - kept;
    const int32_t* row = a.block_tables + (int64_t)(f0 + k) * a.max_blocks_per_seq + kept;
    const int64_t at = head + (int64_t)count + s_off[k];  // + n: at most twice the ring's size
#pragma unroll 4
    for (int j = lane; j < n; j += 32)
      a.free_blocks[at + j < a.free_capacity ? at + j : at + j - a.free_capacity] = row[j];
  }
}

struct VerifyArgs {
  const int32_t* parents;
  const int64_t* draft;
  const int64_t* target;
  const int32_t* query_start;
  const int32_t* context_lens;
  int32_t* accepted;
  int32_t* num_accepted;
  int64_t* next_tokens;
  int32_t* kept_lens;
  int num_seqs, num_tokens, max_accept;
};

// One warp per sequence: lane l holds rows l, l + 32, .. (parent and drafted token, read
// once, together); a step of the walk is one read of the model's choice and one vote per 32
// rows. A tree of up to 64 rows takes two register pairs.
__global__ void __launch_bounds__(128) tree_verify_kernel(const VerifyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (s >= a.num_seqs) return;
  const int q0 = a.query_start[s], q1 = a.query_start[s + 1], ctx = a.context_lens[s];
  int n = q1 - q0;
  const bool range = q0 >= 0 && q1 >= q0 && q1 <= a.num_tokens && ctx >= n;
  if (!range || n > kMaxTree) {
    if (lane == 0) flag_error(range ? PA_DEVERR_TREE : PA_DEVERR_QUERY);
    n = 0;
  }
  int par[kMaxWords];
  int64_t tok[kMaxWords];
#pragma unroll
  for (int w = 0; w < kMaxWords; ++w) {
    const int i = 32 * w + lane;
    par[w] = i < n ? a.parents[q0 + i] : -2;
    tok[w] = i < n ? a.draft[q0 + i] : 0;
  }
  int32_t* out = a.accepted + (int64_t)s * a.max_accept;
  int cur = 0, len = 0, mine = -1;  // lane l keeps path entry l of the current 32
  int64_t want = -1;
  while (len < a.max_accept && len < n) {
    if (lane == (len & 31)) mine = cur;
    ++len;
    if ((len & 31) == 0) {
      out[len - 32 + lane] = mine;
      mine = -1;
    }
    want = a.target[q0 + cur];
    int next = -1;
#pragma unroll
    for (int w = kMaxWords - 1; w >= 0; --w) {
      if (32 * w >= n) continue;
      // a child has a larger index than its parent, so the walk ends
      const unsigned v = __ballot_sync(
          0xffffffffu, par[w] == cur && tok[w] == want && 32 * w + lane > cur);
      if (v) next = 32 * w + __ffs(v) - 1;
    }
    if (next < 0) break;
    cur = next;
  }
  for (int i = (len & ~31) + lane; i < a.max_accept; i += 32)
    out[i] = i < ((len & ~31) + 32) ? mine : -1;
  if (lane == 0) {
    a.num_accepted[s] = len;
    a.next_tokens[s] = want;
    a.kept_lens[s] = n > 0 ? ctx - n + len : ctx;
  }
}

struct CompactArgs {
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* accepted;
  const int32_t* num_accepted;
  const float* k_scales;
  const float* v_scales;
  const int32_t* k_zeros;
  const int32_t* v_zeros;
  int num_seqs, max_accept, max_blocks_per_seq, num_kv_heads, row_bytes, block_size, num_blocks;
};

// 16 one-byte codes from one block's scale (and zero point) to another's, in float32: the
// value code * scale is rounded once, then divided and rounded as the cache write does.
template <pa_dtype KV>
__device__ __forceinline__ uint4 requantise(uint4 w, float s0, float s1, int z0, int z1) {
  uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (KV == PA_INT8) {
      uint32_t o = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __fmul_rn((float)((int)(int8_t)(r[k] >> (8 * e)) - z0), s0);
        const float y = fminf(fmaxf(__fdiv_rn(x, s1), -1024.f), 1024.f);
        const int c = min(127, max(-128, __float2int_rn(y) + z1));
        o |= ((uint32_t)c & 0xffu) << (8 * e);
      }
      r[k] = o;
    } else {
      uint32_t o = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 f = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(r[k] >> (16 * e))));
        o |= (uint32_t)pack_e4m3x2(__fdiv_rn(__fmul_rn(f.x, s0), s1),
                                   __fdiv_rn(__fmul_rn(f.y, s0), s1)) << (16 * e);
      }
      r[k] = o;
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// One CTA per sequence; a thread owns a 16-byte column of one (K or V, kv head) and moves
// the path's rows in order, eight read before the first of them is written. The path
// ascends (accepted[i] >= i), so a row is read before or with the batch that overwrites it,
// and columns do not depend on one another. Rows that stay in place are not touched.
template <pa_dtype KV>
__global__ void __launch_bounds__(256) compact_accepted_kernel(const CompactArgs a) {
  constexpr bool QUANT = KV == PA_FP8_E4M3 || KV == PA_INT8;
  __shared__ int s_src[kMaxTree], s_dst[kMaxTree], s_src_off[kMaxTree], s_dst_off[kMaxTree];
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, tid = threadIdx.x;
  const int n = a.query_start[s + 1] - a.query_start[s], ctx = a.context_lens[s];
  const int len = a.num_accepted[s];
  if (len <= 0) return;
  const int64_t cap = (int64_t)a.max_blocks_per_seq * a.block_size;
  const int32_t* path = a.accepted + (int64_t)s * a.max_accept;
  const int32_t* row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
  int bad = 0;  // 1: the path, 2: a length, 4: a block id
  int moves = 0;
  if (n < 0 || ctx < n || ctx > cap) bad = 2;
  else if (len > a.max_accept || len > n) bad = 1;
  if (!bad && tid < len) {
    const int p = path[tid];
    if (p < 0 || p >= n || (tid > 0 && p <= path[tid - 1])) {
      bad = 1;
    } else {
      moves = p != tid;
      const int f = ctx - n + p, t = ctx - n + tid;
      s_src[tid] = row[f / a.block_size];
      s_src_off[tid] = f % a.block_size;
      s_dst[tid] = row[t / a.block_size];
      s_dst_off[tid] = t % a.block_size;
      if (moves && ((unsigned)s_src[tid] >= (unsigned)a.num_blocks ||
                    (unsigned)s_dst[tid] >= (unsigned)a.num_blocks)) {
        flag_error(PA_DEVERR_BLOCK_ID);
        s_src[tid] = -1;  // this row is skipped
      }
      if (!moves) s_src[tid] = -1;
    }
  }
  // one bad entry stops the whole sequence
  if (__syncthreads_or(bad)) {
    if (bad) flag_error(bad == 2 ? PA_DEVERR_CONTEXT : PA_DEVERR_TREE);
    return;
  }
  if (!__syncthreads_or(moves)) return;
  const int chunks = a.row_bytes / 16;
  const int cols = a.num_kv_heads * chunks;
  for (int i = tid; i < 2 * cols; i += blockDim.x) {
    const bool is_v = i >= cols;
    const int h = (i - (is_v ? cols : 0)) / chunks, c = (i - (is_v ? cols : 0)) % chunks;
    uint8_t* cache = (is_v ? a.v_cache : a.k_cache) + c * 16;
    const float* sc = is_v ? a.v_scales : a.k_scales;
    const int32_t* zp = is_v ? a.v_zeros : a.k_zeros;
    auto at = [&](int blk, int off) {
      return reinterpret_cast<uint4*>(
          cache + (((int64_t)blk * a.num_kv_heads + h) * a.block_size + off) * a.row_bytes);
    };
    for (int b = 0; b < len; b += 8) {
      uint4 x[8];
      bool go[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        go[j] = b + j < len && s_src[b + j] >= 0;
        if (go[j]) x[j] = *at(s_src[b + j], s_src_off[b + j]);
      }
      if constexpr (QUANT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!go[j] || s_src[b + j] == s_dst[b + j]) continue;
          const int64_t f = (int64_t)s_src[b + j] * a.num_kv_heads + h;
          const int64_t t = (int64_t)s_dst[b + j] * a.num_kv_heads + h;
          int z0 = 0, z1 = 0;
          if constexpr (KV == PA_INT8) {
            z0 = zp[f];
            z1 = zp[t];
            if (!zero_in_range(z0) || !zero_in_range(z1)) {  // the row is not written
              flag_error(PA_DEVERR_ZERO);
              go[j] = false;
              continue;
            }
          }
          const float s0 = sc[f], s1 = sc[t];
          if (s0 != s1 || z0 != z1) x[j] = requantise<KV>(x[j], s0, s1, z0, z1);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (go[j]) *at(s_dst[b + j], s_dst_off[b + j]) = x[j];
    }
  }
}

}  // namespace step
}  // namespace pa
