// Attention of drafted tokens over the paged cache on the fifth-generation tensor cores.
//
// Mathematics: for a tile of 128 rows, a row being a (drafted token, query head of the kv
// head's group) pair, S = Q K^T over 64 keys at a time, a running maximum m and sum l per row
// (log2 domain), O = sum 2^(S - m) V; a row sees every key before the drafts and, of the
// drafts, those in its mask. Parts of one context join as
//   M = max m_p,  out = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p.
//
// Bound: HBM while a sequence drafts at most one row tile (a key's K and V cross HBM once for
// all its rows), tensor and exponential units beyond.
//
// Work split: the batch is laid out as one line of key tiles (row tile by row tile, sequence
// by sequence, kv head by kv head) and cut into equal runs, one per CTA, two CTAs per SM, all
// resident. Every CTA streams its run without a pause from one (sequence, kv head) to the
// next, so neither ragged lengths nor few long contexts leave an SM idle, and at most two
// pieces of a run (its ends) are partial: those go to a workspace whose size does not depend
// on the contexts, and a second, small launch joins them. Each CTA finds its run by summing
// the sequences' tiles itself; there is no plan kernel and no counter to reset. Cuts fall by
// lengths only, so results do not depend on where blocks sit.
//
//   warp 5       TMA: Q of the run's current row tile; K and V tiles through their rings, one
//                (block, 64-channel half) box per lane; block ids and scales read a window of
//                32 blocks ahead;
//   warp 4       tcgen05.mma, one lane: S(g + 1) = Q K^T into one of two buffers in tensor
//                memory while S(g) is in softmax, then O += P(g) V, P read from tensor memory;
//   warps 0-3    softmax, one thread per row (= tensor-memory lane): mask, running maximum
//                with lazy rescaling, P as 16-bit pairs over S; O / l or the partial at the end;
//   warps 6-9    fp8 / int8 caches: turn the codes that TMA staged into the f16 tiles the
//                products read (exact values; scales go to the scores and to P), and Q into f16.
// Two CTAs per SM hide each other's starts, ends and waits.
//
// Types: a bf16 cache is multiplied as it is, with P rounded to bf16. Codes of one byte become
// f16 (one instruction per two E4M3 codes; bf16 takes five and made the converters the limit):
// E4M3 values and code - zero are exact in f16. Q rows are brought to [2^14, 2^15) by a power
// of two each, which bf16's eight bits survive down to 2^-28 of the row's largest element. P
// carries V scale / v_ref * 2^7, v_ref a power of two no smaller than any V scale so far: at
// most 2^15, and f16 holds it to 11 bits down to 2^-21 of the largest (bf16 would hold 8).
//
// Every wait is bounded; a CTA that gives up flags PA_DEVERR_TIMEOUT, lets its copies and
// products finish and releases its tensor memory.
#pragma once

#include "prefill_tc.cuh"
#include "tree_simt.cuh"

namespace pa {
namespace tree {

using pf::sdesc;
using pf::tc_fence_after;
using pf::tc_fence_before;
using pf::tmem_ld32;
using pf::tmem_st32;
using pf::tmem_wait_ld;
using pf::tmem_wait_st;
using pf::umma_commit;
using tc::mbar_arrive;
using tc::mbar_arrive_tx;
using tc::mbar_init;
using tc::smem_u32;

// Bounded wait for the phase with the given parity: false after 2^22 polls (a poll that waits
// is itself suspended by the hardware for a while). Kept this short because the kernel has
// dozens of waits and its speed hangs on its code fitting the instruction cache.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  bool done = tc::mbar_try_wait(bar, parity);
#pragma unroll 1
  for (int i = 0; !done && i < (1 << 22); ++i) done = tc::mbar_try_wait(bar, parity);
  return done;
}

constexpr int kRows = 128;                 // rows of a tile
constexpr int kKeys = 64;                  // keys of a tile
constexpr int kDim = 128;
constexpr int kStreams = 296;              // runs the batch is cut into: two CTAs per SM of 148
// What a piece costs beside its key tiles (Q, first scores, last products, output), in key
// tiles: short contexts would otherwise pile up in few runs.
#ifndef PA_TREE_PIECE_COST
#define PA_TREE_PIECE_COST 4
#endif
constexpr int kPieceCost = PA_TREE_PIECE_COST;
constexpr int kMmaWarp = 4, kTmaWarp = 5, kConvWarp = 6;
constexpr int kConvWarps = 2;              // converter warps for K, and as many for V
constexpr int kQBytes = 2 * kRows * 128;   // Q: one tile of 128 rows, or smaller ones
constexpr int kCodeSt = 3;                 // staged codes: a ring of tiles, K and V in turn
constexpr int kKVSlab = kKeys * 128;       // 64 channels x 64 keys
constexpr int kKVBytes = 2 * kKVSlab;
constexpr int kCodeBytes = kKeys * 128;    // one-byte codes of 64 keys
constexpr int kMaxTileBlocks = kKeys / 8;  // blocks of a key tile, at most
constexpr int kInfo = 8;                   // ring of per-tile facts for softmax and converters
constexpr uint32_t kCols = 256;            // tensor memory: S at 0 and 64 (P over it), O at 128
constexpr uint32_t kOCol = 128;

// A key tile as the producer describes it to the other warps (one slot of a ring): only the
// producer walks the batch.
enum : int { kFirst = 1, kLast = 2, kEnd = 4, kWhole = 8 };
struct TileInfo {
  int flags;        // first / last tile of its piece; the run is over; the piece is a whole pair
  uint32_t bad;     // bit b: block b of the tile cannot be read
  int key0;         // position of the tile's first key
  // of the piece, and only in its first tile's slot:
  int base, ctx;    // context without and with the step's rows
  int row0, rows;   // first token row of the row tile, its tokens
  int s, kvh;
  int slot;         // workspace slot of a partial piece
  float ks[kMaxTileBlocks], vs[kMaxTileBlocks];
  int kz[kMaxTileBlocks], vz[kMaxTileBlocks];
};

// A piece of a run: key tiles [t0, t1) of row tile rt, sequence s, kv head kvh.
struct Piece {
  int rt, s, kvh, t0, t1, tiles;
  int q0, n, ctx;
};

// Up to 32 consecutive blocks of a piece on their way to the producer (a ring of windows in
// shared memory that asynchronous copies fill): block ids, then their scales.
struct Window {
  int id[32];       // -1: cannot be read, or none
  float ks[32], vs[32];
  int kz[32], vz[32];
  Piece pc;
  int tile0, ntiles, first, any;   // its key tiles; first of its piece; exists
};
constexpr int kWindows = 4;

template <bool QUANT>
struct Layout {
  static constexpr int kThreads = QUANT ? 192 + 64 * kConvWarps : 192;
  // 16-bit tiles of K and of V: two each, but for codes and 128 rows, whose Q takes the place
  // of the second K tile (k_st below)
  static constexpr int kVSt = 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = QUANT ? kQBytes / 2 : kQBytes;
  static constexpr int kOffV = kOffK + 2 * kKVBytes;
  static constexpr int kOffC = kOffV + kVSt * kKVBytes;
  static constexpr int kOffInfo = kOffC + (QUANT ? kCodeSt * kCodeBytes : 0);
  static constexpr int kOffWin = kOffInfo + kInfo * (int)sizeof(TileInfo);
  static constexpr int kOffMisc = kOffWin + kWindows * (int)sizeof(Window);
  static constexpr int kOffDown = kOffMisc + 384;          // float [4][kRows]: what undoes Q's factors
  static constexpr int kOffBar = kOffDown + (QUANT ? 4 * kRows * 4 : 0);
  // barriers
  static constexpr int kBarQF = 0, kBarQE = 2;   // [2] each
  static constexpr int kBarKF = 4, kBarKE = kBarKF + 2;
  static constexpr int kBarVF = kBarKE + 2, kBarVE = kBarVF + kVSt;
  static constexpr int kBarSF = kBarVE + kVSt;   // [2] S in tensor memory
  static constexpr int kBarP = kBarSF + 2;       // [2] P in tensor memory
  static constexpr int kBarO = kBarP + 2;        // [2] P V done
  static constexpr int kBarInfo = kBarO + 2;     // [kInfo]
  static constexpr int kBarCF = kBarInfo + kInfo, kBarCE = kBarCF + (QUANT ? kCodeSt : 0);
  static constexpr int kBarQR = kBarCE + (QUANT ? kCodeSt : 0);  // [4] Q converted
  static constexpr int kBarSm = kBarQR + (QUANT ? 4 : 0);  // the four softmax warps, once a piece
  static constexpr int kBarFin = kBarSm + 1;
  static constexpr int kNumBars = kBarFin + 1;
  static constexpr int kSmem = kOffBar + 8 * kNumBars + 1024;  // + alignment slack
};
static_assert(Layout<true>::kSmem <= 113 * 1024 && Layout<false>::kSmem <= 113 * 1024,
              "two CTAs per SM");
static_assert((kInfo * sizeof(TileInfo) + kWindows * sizeof(Window)) % 8 == 0,
              "barriers are 8-byte aligned");

// S = Q K^T: A and B K-major, N = 64 keys. O += P V: A from tensor memory, B MN-major, N = 128.
// Both operands bf16 (1 << 7, 1 << 10), or both f16.
constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);
constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(kDim >> 3) << 17) |
                              ((uint32_t)(kRows >> 4) << 24);

// Workspace: what CTA b's run is, then the partial pieces.
struct RunInfo {
  int64_t per;       // length of a run
  int64_t begin;     // where the (row tile, sequence, kv head) that the run begins in begins
  int rt, s, kvh, tiles;  // that one, and its key tiles; tiles = 0: the run is empty
};
struct Workspace {
  RunInfo* runs;     // [kStreams]
  float* m;          // [kStreams][2][kRows]: piece 0 begins the run, piece 1 ends it
  float* l;
  float* acc;        // [kStreams][2][kDim / 4][kRows][4]
};
constexpr size_t kRunBytes = (size_t)kStreams * sizeof(RunInfo);
constexpr size_t kPieceRows = (size_t)kStreams * 2 * kRows;
constexpr size_t kWorkspaceBytes =
    (kRunBytes + 255) / 256 * 256 + kPieceRows * (2 + kDim) * sizeof(float);
inline Workspace workspace_at(void* p) {
  Workspace w;
  char* c = static_cast<char*>(p);
  w.runs = reinterpret_cast<RunInfo*>(c);
  w.m = reinterpret_cast<float*>(c + (kRunBytes + 255) / 256 * 256);
  w.l = w.m + kPieceRows;
  w.acc = w.l + kPieceRows;
  return w;
}

// True in one lane of a converged warp, always the same one. Unlike `lane == 0` it tells the
// compiler that one thread runs what follows, whose operands then stay in uniform registers.
__device__ __forceinline__ bool one_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// A four-byte asynchronous copy into shared memory, or four zero bytes.
__device__ __forceinline__ void copy4(void* dst, const void* src, bool go) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(go ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ int tiles_of(int ctx) { return (ctx + kKeys - 1) / kKeys; }
__device__ __forceinline__ int row_tiles_of(int n, int G) {
  return (int)(((int64_t)n * G + kRows - 1) / kRows);
}

// The pieces of a run in order, the same for every warp that walks it: 32 sequences' ranges
// are held one per lane. All members but those are warp-uniform; every lane takes part.
struct Walk {
  int64_t left;                // of the run
  int rt, s, kvh, tiles, base;
  int at;                      // place in the current (row tile, sequence, kv head): its first
                               // kPieceCost places hold no tile
  int l_q0, l_n, l_ctx;  // this lane's sequence base + lane (n = 0: none, or nothing to do)

  __device__ __forceinline__ void load(const TreeArgs& a) {
    const int k = base + (threadIdx.x & 31);
    l_n = 0;
    if (k < a.num_seqs && !seq_range(a, k, l_q0, l_n, l_ctx)) l_n = 0;
  }
  __device__ __forceinline__ void start(const TreeArgs& a, int64_t count, int rt_, int s_, int kvh_,
                                        int at_) {
    left = count;
    rt = rt_;
    s = s_;
    kvh = kvh_;
    at = at_;
    base = s & ~31;
    if (left > 0) {
      load(a);
      tiles = tiles_of(__shfl_sync(0xffffffffu, l_ctx, s & 31));
    }
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, Piece& p) {
    while (left > 0) {
      if (at == tiles + kPieceCost) {
        at = 0;
        if (++kvh == a.num_kv_heads) {
          kvh = 0;
          int from = (s & 31) + 1;
          while (true) {
            const unsigned v = __ballot_sync(
                0xffffffffu, (int)(threadIdx.x & 31) >= from &&
                                 (int64_t)l_n * a.group > (int64_t)rt * kRows);
            if (v) {
              s = base + __ffs(v) - 1;
              break;
            }
            from = 0;
            base += 32;
            if (base >= a.num_seqs) {
              base = 0;
              if ((int64_t)++rt * kRows >= (int64_t)a.max_query_len * a.group) {
                left = 0;  // cannot happen while `left` counts what exists
                return false;
              }
            }
            load(a);
          }
          tiles = tiles_of(__shfl_sync(0xffffffffu, l_ctx, s & 31));
        }
      }
      const int take = (int)min(left, (int64_t)(tiles + kPieceCost - at));
      p.t0 = max(0, at - kPieceCost);
      p.t1 = max(0, at + take - kPieceCost);
      left -= take;
      at += take;
      if (p.t1 > p.t0) {
        p.rt = rt;
        p.s = s;
        p.kvh = kvh;
        p.tiles = tiles;
        p.q0 = __shfl_sync(0xffffffffu, l_q0, s & 31);
        p.n = __shfl_sync(0xffffffffu, l_n, s & 31);
        p.ctx = __shfl_sync(0xffffffffu, l_ctx, s & 31);
        return true;
      }
    }
    return false;
  }
};

// Exclusive sum of x over the CTA's threads in order, and the total.
template <int W>
__device__ __forceinline__ int64_t scan1(int64_t x, int64_t& total, int64_t* sw) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t i = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, i, o);
    if (lane >= o) i += v;
  }
  if (lane == 31) sw[warp] = i;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += sw[w];
    total += sw[w];
  }
  __syncthreads();
  return before + i - x;
}

// One mask word pair of a row's view of a key tile: bit e of the result: the row sees key
// t0 + e. Keys before `base` are seen, keys at or behind ctx are not.
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

// The softmax of one tile for one row: S (64 columns of this lane in tensor memory at `sbuf`) to
// P (16-bit pairs over its first 32 columns; rvs: the factor of the V scales). Two passes of 32 columns each over S, which keeps
// half the registers and code of one pass that holds all 64. `view`: keys the row sees (read
// only when MASKED). Returns the factor that O and l have to be multiplied with.
template <int BS, bool QUANT, bool MASKED>
__device__ __forceinline__ float softmax_tile(uint32_t sbuf, const TileInfo& ti, float sl2,
                                              float rvs, uint64_t view, float& m_used, float& l) {
  float m_new = m_used;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t sv[32];
    tmem_ld32(sbuf + c * 32, sv);
    tmem_wait_ld(sv);
    const uint32_t v = MASKED ? (uint32_t)(view >> (32 * c)) : 0u;
    float mx[4] = {m_new, m_new, m_new, m_new};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float f = QUANT ? sl2 * ti.ks[c * (32 / BS) + e / BS] : sl2;
      float z = __uint_as_float(sv[e]) * f;
      if (MASKED && !((v >> e) & 1u)) z = -INFINITY;
      mx[e & 3] = fmaxf(mx[e & 3], z);
    }
    m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  }
  float alpha = 1.f;
  if (m_new > m_used + 8.f) {  // lazy: P stays at or below 2^8 otherwise
    alpha = fast_exp2(m_used - m_new);
    m_used = m_new;
  }
  const float ref = m_used == -INFINITY ? 0.f : -m_used;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t sv[32], pk[16];
    tmem_ld32(sbuf + c * 32, sv);
    tmem_wait_ld(sv);
    const uint32_t v = MASKED ? (uint32_t)(view >> (32 * c)) : 0u;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float f = QUANT ? sl2 * ti.ks[c * (32 / BS) + e / BS] : sl2;
      float p0 = fast_exp2(fmaf(__uint_as_float(sv[e]), f, ref));
      float p1 = fast_exp2(fmaf(__uint_as_float(sv[e + 1]), f, ref));
      if (MASKED) {
        p0 = ((v >> e) & 1u) ? p0 : 0.f;
        p1 = ((v >> (e + 1)) & 1u) ? p1 : 0.f;
      }
      sum[e & 3] += p0;
      sum[(e + 1) & 3] += p1;
      if constexpr (QUANT) {  // P carries its block's V scale; a key that is not seen, none
        const float vs = ti.vs[c * (32 / BS) + e / BS] * rvs;
        p0 = MASKED && p0 == 0.f ? 0.f : p0 * vs;
        p1 = MASKED && p1 == 0.f ? 0.f : p1 * vs;
      }
      pk[e >> 1] = QUANT ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
    }
    pf::tmem_st16(sbuf + c * 16, pk);  // over columns that both passes have read
  }
  l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
  tmem_wait_st();
  return alpha;
}

// The same for a tile that every row sees whole, against the reference as it stands, in one
// pass without the maximum. True when that was right: the weights' sum is below 2^8, so none of
// them is above it. Otherwise (a score outgrew the reference, or is no number) nothing was
// written and the two passes above have to be taken. Most tiles end here, with half the
// instructions: the softmax of few rows is one warp's, and sets the pace.
template <int BS, bool QUANT>
__device__ __forceinline__ bool softmax_tile_fast(uint32_t sbuf, const TileInfo& ti, float sl2,
                                                  float rvs, float m_used, float& l) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t pk[32];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t sv[32];
    tmem_ld32(sbuf + c * 32, sv);
    tmem_wait_ld(sv);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float f = QUANT ? sl2 * ti.ks[c * (32 / BS) + e / BS] : sl2;
      float p0 = fast_exp2(fmaf(__uint_as_float(sv[e]), f, -m_used));
      float p1 = fast_exp2(fmaf(__uint_as_float(sv[e + 1]), f, -m_used));
      sum[e & 3] += p0;
      sum[(e + 1) & 3] += p1;
      if constexpr (QUANT) {
        const float vs = ti.vs[c * (32 / BS) + e / BS] * rvs;
        p0 *= vs;
        p1 *= vs;
      }
      pk[c * 16 + (e >> 1)] = QUANT ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
    }
  }
  const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  // one vote: a warp takes one path, its loads and stores are collective
  if (!__all_sync(0xffffffffu, s <= 256.f)) return false;
  tmem_st32(sbuf, pk);
  l += s;
  tmem_wait_st();
  return true;
}

template <int BS, pa_dtype KV>
__global__ void __launch_bounds__(Layout<KV != PA_BF16>::kThreads, 2)
tree_tc_kernel(const TreeArgs a, const Workspace ws, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr bool QUANT = KV != PA_BF16;
  using L = Layout<QUANT>;
  constexpr int kThreads = L::kThreads, W = kThreads / 32;
  constexpr int NB = kKeys / BS;           // blocks of a key tile
  constexpr int WT = 32 / NB;              // tiles of a window of 32 blocks
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform, and known to be
  const int G = a.group, TM = kRows / G, Hkv = a.num_kv_heads;
  // A step of few rows per sequence keeps two pieces' Q (the product still reads 128 rows:
  // what lies behind Q gives rows that nobody uses), or a second K tile.
  const int q_rows = a.q_rows;
  const int q_bufs = q_rows == (QUANT ? kRows / 4 : kRows / 2) ? 2 : 1;
  const int k_st = QUANT && q_rows == kRows ? 1 : 2;
  auto k_of = [&](int g) { return k_st == 2 ? g & 1 : 0; };         // tile g's K: its stage,
  auto k_use = [&](int g) { return k_st == 2 ? g >> 1 : g; };       // and which use of it
  const uint32_t sQ = smem_u32(smem + L::kOffQ);
  const uint32_t sK = smem_u32(smem + (k_st == 1 ? kQBytes : L::kOffK));
  const uint32_t sV = smem_u32(smem + L::kOffV);
  const uint32_t bar0 = smem_u32(smem + L::kOffBar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + L::kOffInfo);
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + L::kOffMisc);          // [16]
  int* s_start = reinterpret_cast<int*>(s_scan + 16);                       // rt, s, kvh, place
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_start + 4);
  // drafts of the current piece whose V row holds a NaN or infinity, by draft index (a ring
  // of four lists: the converters may be two pieces ahead of the softmax)
  uint32_t* s_odd = reinterpret_cast<uint32_t*>(tmem_slot + 2);              // [4][8]
  volatile int* any_odd = reinterpret_cast<volatile int*>(s_odd + 32);       // [4]

  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      uint32_t count = 1;
      if (i == L::kBarP || i == L::kBarP + 1 || i == L::kBarSm) count = kRows;
      if (QUANT && ((i >= L::kBarKF && i < L::kBarKF + 2) ||
                    (i >= L::kBarVF && i < L::kBarVF + L::kVSt) ||
                    (i >= L::kBarCE && i < L::kBarCE + kCodeSt) ||
                    (i >= L::kBarQR && i < L::kBarQR + 4)))
        count = 32 * kConvWarps;
      mbar_init(bar(i), count);
    }
    for (int i = 0; i < 32; ++i) s_odd[i] = 0;
    for (int i = 0; i < 4; ++i) any_odd[i] = 0;
    s_start[0] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    pf::tmem_alloc(smem_u32(tmem_slot), kCols);
    pf::tmem_relinquish();
  }
  pdl_wait();
  // the joining launch may take its place on idle SMs now; it waits for this grid's end
  pdl_trigger();
  // ---- the batch's key tiles, and where this CTA's run begins ----
  const int rts = row_tiles_of(a.max_query_len, G);
  const int seqs_per = (a.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min(a.num_seqs, tid * seqs_per), s1 = min(a.num_seqs, s0 + seqs_per);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    int q0, n, ctx;
    if (seq_range(a, s, q0, n, ctx)) mine += (int64_t)row_tiles_of(n, G) * (tiles_of(ctx) + kPieceCost);
    else if (blockIdx.x == 0) flag_error(PA_DEVERR_QUERY);
  }
  int64_t total;
  const int64_t before = scan1<W>(mine, total, s_scan);
  const int64_t seq_total = total;
  total *= Hkv;
  const int64_t per = (total + kStreams - 1) / kStreams;
  const int64_t w0 = per * blockIdx.x, count = min(per, total - w0);
  if (count <= 0) {
    if (tid == 0) ws.runs[blockIdx.x].tiles = 0;
    if (warp == 0) pf::tmem_dealloc(*tmem_slot, kCols);   // its own warp's allocation
    return;
  }
  int64_t done = 0;
#pragma unroll 1
  for (int rt = 0; rt < rts; ++rt) {
    int64_t sum = mine, all = seq_total, at = before;   // all there is with one row tile
    if (rts > 1) {
      sum = 0;
      for (int s = s0; s < s1; ++s) {
        int q0, n, ctx;
        if (seq_range(a, s, q0, n, ctx) && row_tiles_of(n, G) > rt) sum += tiles_of(ctx) + kPieceCost;
      }
      at = scan1<W>(sum, all, s_scan);
    }
    if (w0 < done + all * Hkv) {
      at = done + at * Hkv;
      if (w0 >= at && w0 < at + sum * Hkv) {  // one thread's sequences hold it
        for (int s = s0; s < s1; ++s) {
          int q0, n, ctx;
          if (!seq_range(a, s, q0, n, ctx) || row_tiles_of(n, G) <= rt) continue;
          const int nt = tiles_of(ctx) + kPieceCost;
          if (w0 < at + (int64_t)nt * Hkv) {
            const int h = (int)((w0 - at) / nt);
            s_start[0] = rt;
            s_start[1] = s;
            s_start[2] = h;
            s_start[3] = (int)(w0 - at - (int64_t)h * nt);
            ws.runs[blockIdx.x] = RunInfo{per, at + (int64_t)h * nt, rt, s, h, tiles_of(ctx)};
            break;
          }
          at += (int64_t)nt * Hkv;
        }
      }
      break;
    }
    done += all * Hkv;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // waits are made warp-uniform
  auto wait_all = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity)) != 0;
  };
  auto wait_info = [&](int g) { return wait_all(bar(L::kBarInfo + g % kInfo), (g / kInfo) & 1); };
  bool ok = true;

  if (warp == kTmaWarp) {
    // ------------------------------ producer ------------------------------
    // Windows pass through three stages, so that nothing is waited for as soon as it is asked
    // for: window w is in use, the scales of w + 1 and the block ids of w + 2 are on their way.
    Window* win = reinterpret_cast<Window*>(smem + L::kOffWin);
    Walk walk;
    walk.start(a, s_start[0] >= 0 ? count : 0, s_start[0], s_start[1], s_start[2], s_start[3]);
    Piece pc;
    pc.t1 = 0;
    int wt = 0;          // next tile of the piece that the newest window belongs to
    bool more = true, run_first = true;
    const uint64_t keep = tc::evict_first_policy();
    int g = 0, pieces = 0;
    auto fetch_ids = [&](int i) {
      Window& w = win[i % kWindows];
      const bool first = wt == pc.t1;
      if (more && first) {
        more = walk.next(a, pc);
        wt = pc.t0;
      }
      const int n = min(WT, pc.t1 - wt), blk = wt * NB + lane;
      if (lane == 0) {
        w.pc = pc;
        w.tile0 = wt;
        w.ntiles = n;
        w.first = first;
        w.any = more;
      }
      const bool want = more && lane < n * NB && blk * BS < pc.ctx;
      if (more && first) {
        // the rows' masks into L1: the softmax reads them when the piece begins
        const int toks = min(TM, pc.n - pc.rt * TM);
        const uint32_t* m = a.tree_mask + (int64_t)(pc.q0 + pc.rt * TM) * a.mask_words;
        for (int i = lane * 32; i < toks * a.mask_words; i += 1024)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(m + i) : "memory");
      }
      copy4(&w.id[lane], a.block_tables + (want ? (int64_t)pc.s * a.max_blocks_per_seq + blk : 0), want);
      wt += n;
    };
    auto fetch_scales = [&](int i) {
      Window& w = win[i % kWindows];
      int p = w.id[lane];
      const bool want = w.any && lane < w.ntiles * NB && (w.tile0 * NB + lane) * BS < w.pc.ctx;
      if (want && (p < 0 || p >= a.num_blocks)) flag_error(PA_DEVERR_BLOCK_ID);
      if (!want || p < 0 || p >= a.num_blocks) p = -1;
      w.id[lane] = p;
      if constexpr (QUANT) {  // zero scales for what is not there: P's reference ignores it
        const int64_t bh = p >= 0 ? (int64_t)p * Hkv + w.pc.kvh : 0;
        copy4(&w.ks[lane], a.k_scales + bh, p >= 0);
        copy4(&w.vs[lane], a.v_scales + bh, p >= 0);
        if constexpr (KV == PA_INT8) {
          copy4(&w.kz[lane], a.k_zeros + bh, p >= 0);
          copy4(&w.vz[lane], a.v_zeros + bh, p >= 0);
        }
      }
    };
    fetch_ids(0);
    copies_done();
    __syncwarp();
    fetch_scales(0);
    fetch_ids(1);
#pragma unroll 1
    for (int i = 0;; ++i) {
      copies_done();
      __syncwarp();
      Window& w = win[i % kWindows];
      if (!w.any) break;
      if (KV == PA_INT8 && w.id[lane] >= 0 &&
          (!zero_in_range(w.kz[lane]) || !zero_in_range(w.vz[lane]))) {
        flag_error(PA_DEVERR_ZERO);
        w.id[lane] = -1;
        w.vs[lane] = 0.f;
      }
      fetch_scales(i + 1);
      fetch_ids(i + 2);
      __syncwarp();
      const int kvh = w.pc.kvh, ctx = w.pc.ctx, tile0 = w.tile0, ntiles = w.ntiles;
      if (w.first) {
        // the last S product of the piece that used this buffer has read it
        const int qb = q_bufs == 2 ? pieces & 1 : 0, use = q_bufs == 2 ? pieces >> 1 : pieces;
        if (use > 0) ok = wait_all(bar(L::kBarQE + qb), (use - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          const int slab = q_rows * 128;
          mbar_arrive_tx(bar(L::kBarQF + qb), 2 * slab);
#pragma unroll 1
          for (int h = 0; h < 2; ++h)
            pf::tma_load_4d(sQ + (2 * qb + h) * slab, &qmap, 0, h, kvh * G,
                            w.pc.q0 + w.pc.rt * TM, bar(L::kBarQF + qb), keep);
        }
        __syncwarp();
        ++pieces;
      }
      // Lane l copies block l of the window whenever its tile's turn comes. What the whole
      // window shares is worked out here: a tile's own code is kept to a few instructions.
      const int p = w.id[lane], mine = lane / NB, row = (p * Hkv + kvh) * BS;
      const uint32_t good = __ballot_sync(0xffffffffu, p >= 0);
      const uint32_t gone = __ballot_sync(0xffffffffu, p < 0 && lane < ntiles * NB &&
                                                           (tile0 * NB + lane) * BS < ctx);
      const uint32_t off = (uint32_t)(lane & (NB - 1)) * BS * 128;
      float ks = 0.f, vs = 0.f;
      int kz = 0, vz = 0;
      if constexpr (QUANT) {
        ks = w.ks[lane];
        vs = w.vs[lane];
        if constexpr (KV == PA_INT8) {
          kz = w.kz[lane];
          vz = w.vz[lane];
        }
      }
      const int last_tile = w.pc.t1 - 1 - tile0;
      const int whole = w.pc.t0 == 0 && w.pc.t1 == w.pc.tiles ? kWhole : 0;
#pragma unroll 1
      for (int k = 0; k < ntiles; ++k, ++g) {
        const uint32_t bytes = (uint32_t)__popc((good >> (k * NB)) & ((1u << NB) - 1u)) * BS * 128u;
        const bool my_turn = mine == k && p >= 0;
        TileInfo& ti = info[g % kInfo];
        // K or V of this tile into its ring's stage, free once its last reader is done
        auto copy = [&](const CUtensorMap* map, int full, int empty, int st, int use, uint32_t dst) {
          if (use > 0) ok = wait_all(bar(empty + st), (use - 1) & 1);
          if (!ok) return;
          if (lane == 0) mbar_arrive_tx(bar(full + st), QUANT ? bytes : 2 * bytes);
          __syncwarp();
          if (my_turn) {
            if constexpr (QUANT) {
              tc::tma_load_2d(dst + off, map, 0, row, bar(full + st), keep);
            } else {
              pf::tma_load_3d(dst + off, map, 0, 0, row, bar(full + st));
              pf::tma_load_3d(dst + kKVSlab + off, map, 0, 1, row, bar(full + st));
            }
          }
        };
        const uint32_t sC = smem_u32(smem + L::kOffC);
        int c = 2 * g;   // codes: K and V of a tile follow one another through one ring
        if constexpr (QUANT) {
          copy(&kmap, L::kBarCF, L::kBarCE, c % kCodeSt, c / kCodeSt, sC + (c % kCodeSt) * kCodeBytes);
        } else {
          copy(&kmap, L::kBarKF, L::kBarKE, k_of(g), k_use(g), sK + k_of(g) * kKVBytes);
        }
        if (!ok) break;
        // The description's slot is free. bf16: K(g - 2) was read by S(g - 2), issued behind
        // P V (g - 4). Codes: those of V(g - 2) at least are converted, into a tile that
        // P V (g - 4) had read. So softmax and converters are past tile g - 4 > g - kInfo.
        if (QUANT && mine == k) {
          ti.ks[lane & (NB - 1)] = ks;
          ti.vs[lane & (NB - 1)] = vs;
          if constexpr (KV == PA_INT8) {
            ti.kz[lane & (NB - 1)] = kz;
            ti.vz[lane & (NB - 1)] = vz;
          }
        }
        if (lane == 0) {
          const bool first = k == 0 && w.first;
          ti.flags = (first ? kFirst : 0) | (k == last_tile ? kLast : 0) | whole;
          ti.bad = (gone >> (k * NB)) & ((1u << NB) - 1u);
          ti.key0 = (tile0 + k) * kKeys;
          if (first) {
            ti.base = ctx - w.pc.n;
            ti.ctx = ctx;
            ti.row0 = w.pc.q0 + w.pc.rt * TM;
            ti.rows = min(TM, w.pc.n - w.pc.rt * TM);
            ti.s = w.pc.s;
            ti.kvh = kvh;
            ti.slot = blockIdx.x * 2 + (run_first ? 0 : 1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarInfo + g % kInfo));
        ++c;
        if constexpr (QUANT) {
          copy(&vmap, L::kBarCF, L::kBarCE, c % kCodeSt, c / kCodeSt, sC + (c % kCodeSt) * kCodeBytes);
        } else {
          copy(&vmap, L::kBarVF, L::kBarVE, g % L::kVSt, g / L::kVSt, sV + (g % L::kVSt) * kKVBytes);
        }
        if (!ok) break;
      }
      if (!ok) break;
      if (w.tile0 + w.ntiles == w.pc.t1) run_first = false;
      __syncwarp();
    }
    copies_done();
    if (lane == 0) {
      if (ok) {  // the slot is free as above
        info[g % kInfo].flags = kEnd;
        mbar_arrive(bar(L::kBarInfo + g % kInfo));
      } else {
        // copies in flight complete (each barrier's last phase) before shared memory is released
        for (int i = max(0, pieces - q_bufs); i < pieces; ++i)
          mbar_wait(bar(L::kBarQF + i % q_bufs), (i / q_bufs) & 1);
        if (QUANT) {
          for (int c = max(0, 2 * g + 1 - kCodeSt); c <= 2 * g + 1; ++c)
            mbar_wait(bar(L::kBarCF + c % kCodeSt), (c / kCodeSt) & 1);
        } else {
          for (int j = max(0, g - 2); j <= g; ++j) {
            mbar_wait(bar(L::kBarKF + k_of(j)), k_use(j) & 1);
            mbar_wait(bar(L::kBarVF + j % L::kVSt), (j / L::kVSt) & 1);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------ MMA issuer ------------------------------
    int g = 0, pieces = 0, q_buf = 0;   // tiles whose S is issued; pieces whose Q is in use
    uint32_t q_lo = 0;                  // low half of Q's descriptor
    uint32_t fresh = 0;                 // bit b: P V from S buffer b begins a piece
    // Descriptors differ in their low half alone, the address in 16-byte units (which never
    // carries into the fields above): one addition each.
    const uint64_t kmajor = sdesc(0, 16, 1024), vmajor = sdesc(0, kKVSlab, 1024);
    const uint32_t q_slab = (uint32_t)q_rows * 8;
    // S of the run's next tile; false when there is none (or a wait gave up)
    auto next_s = [&]() {
      ok = wait_info(g);
      if (!ok) return false;
      const int flags = __shfl_sync(0xffffffffu, info[g % kInfo].flags, 0);
      if (flags & kEnd) return false;
      if (flags & kFirst) {
        q_buf = q_bufs == 2 ? pieces & 1 : 0;
        ok = QUANT ? wait_all(bar(L::kBarQR + (pieces & 3)), (pieces >> 2) & 1)
                   : wait_all(bar(L::kBarQF + q_buf), (q_bufs == 2 ? pieces >> 1 : pieces) & 1);
        if (!ok) return false;
        q_lo = (sQ >> 4) + q_buf * q_rows * 16;
        ++pieces;
      }
      ok = wait_all(bar(L::kBarKF + k_of(g)), k_use(g) & 1);
      if (!ok) return false;
      tc_fence_after();
      const uint32_t b = 1u << (g & 1);
      fresh = (flags & kFirst) ? fresh | b : fresh & ~b;
      if (one_lane()) {
        const uint64_t kd = kmajor + ((sK + k_of(g) * kKVBytes) >> 4);
        const uint64_t qd0 = kmajor + q_lo, qd1 = qd0 + q_slab;
#pragma unroll
        for (int kk = 0; kk < kDim / 16; ++kk)
          pf::umma_bf16(tmem + (g & 1) * kKeys, (kk < 4 ? qd0 : qd1) + (kk & 3) * 2,
                        kd + (kk >> 2) * (kKVSlab / 16) + (kk & 3) * 2,
                        kIdescS | (QUANT ? 0 : kBf16), kk > 0);
        umma_commit(bar(L::kBarSF + (g & 1)));
        umma_commit(bar(L::kBarKE + k_of(g)));
        if (flags & kLast) umma_commit(bar(L::kBarQE + q_buf));
      }
      __syncwarp();
      ++g;
      return true;
    };
    bool more = next_s();
#pragma unroll 1
    for (int j = 0; ok && j < g; ++j) {
      // S of tile j + 1 first: it runs while tile j is in softmax. (P V first whenever its
      // operands were there lost a fifth, the softmax then waits for S; polling for whichever
      // came first lost 5 %.)
      if (more) more = next_s();
      if (!ok) break;
      ok = wait_all(bar(L::kBarP + (j & 1)), (j >> 1) & 1) &&
           wait_all(bar(L::kBarVF + j % L::kVSt), (j / L::kVSt) & 1);
      if (!ok) break;
      tc_fence_after();
      if (one_lane()) {
        const uint64_t vd = vmajor + ((sV + (j % L::kVSt) * kKVBytes) >> 4);
        const bool acc = !((fresh >> (j & 1)) & 1u);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          pf::umma_bf16_ts(tmem + kOCol, tmem + (j & 1) * kKeys + kk * 8,
                           vd + kk * 128, kIdescPV | (QUANT ? 0 : kBf16),
                           acc || kk > 0);
        umma_commit(bar(L::kBarO + (j & 1)));
        umma_commit(bar(L::kBarVE + j % L::kVSt));
      }
      __syncwarp();
    }
    if (one_lane()) {
      // every product of the CTA completes before tensor memory is released
      umma_commit(bar(L::kBarFin));
      mbar_wait(bar(L::kBarFin), 0);
    }
    __syncwarp();
  } else if (QUANT && warp >= kConvWarp) {
    // ------------------------------ converters ------------------------------
    // The first kConvWarps warps turn K tiles (and Q), the others V tiles, sharing a tile's rows.
    // A lane takes 16 codes at a time: value = the E4M3 code's value or code - zero, exact in
    // f16, stored where TMA would put a 16-bit type (128-byte rows of 64 channels, 16-byte
    // chunks XORed with row % 8). V rows that cannot be read or lie behind the context become
    // zero, and so do NaN codes of drafts: P is zero for rows that do not see them, but 0 * NaN
    // is not (rows that see one get it back at the end).
    const int kv = (warp - kConvWarp) / kConvWarps, sub = (warp - kConvWarp) % kConvWarps;
    constexpr int kIts = kKeys / 4 / kConvWarps;   // 4 keys an iteration
    // rows 4 (sub + kConvWarps i) + lane / 8: their low three bits do not change with i
    static_assert(kConvWarps == 2, "a warp's keys repeat modulo 8");
    const int q8 = lane & 7, key0 = sub * 4 + (lane >> 3), c0 = 2 * (q8 & 3);
    const uint32_t at0 = (q8 >> 2) * kKVSlab + key0 * 128 + ((c0 ^ (key0 & 7)) << 4);
    const uint32_t at1 = (q8 >> 2) * kKVSlab + key0 * 128 + (((c0 + 1) ^ (key0 & 7)) << 4);
    int pieces = 0, ctx = 0, base = 0;
#pragma unroll 1
    for (int g = 0;; ++g) {
      const int st = kv ? g % L::kVSt : k_of(g), use = kv ? g / L::kVSt : k_use(g);
      const int c = 2 * g + kv, cst = c % kCodeSt;
      ok = wait_info(g);
      if (!ok) break;
      const TileInfo& ti = info[g % kInfo];
      const int flags = ti.flags;
      if (flags & kEnd) break;
      if (flags & kFirst) {
        ctx = ti.ctx;
        base = ti.base;
        if (!kv) {
          // Q of the piece: 16 lanes to a row of 128 channels, in place
          const int qb = q_bufs == 2 ? pieces & 1 : 0;
          ok = wait_all(bar(L::kBarQF + qb), (q_bufs == 2 ? pieces >> 1 : pieces) & 1);
          if (!ok) break;
          float* down = reinterpret_cast<float*>(smem + L::kOffDown) + (pieces & 3) * kRows;
          const int rows = ti.rows * G;
#pragma unroll 1
          for (int r = sub * 2 + (lane >> 4); r < ((rows + 3) & ~3); r += 2 * kConvWarps) {
            const int ch = lane & 15;
            const uint32_t at = sQ + (2 * qb + (ch >> 3)) * q_rows * 128 + r * 128 +
                                (((ch & 7) ^ (r & 7)) << 4);
            uint32_t x[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int eb = (int)((__float_as_uint(amax) >> 23) & 0xff);
            // 2^e puts the row's largest element into [2^14, 2^15)
            const int e = eb == 0 || eb == 0xff ? 0 : max(-100, min(100, 14 - (eb - 127)));
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = pack_f16x2(bf16_lo(x[i]) * up, bf16_hi(x[i]) * up);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
            if (ch == 0) down[r] = __uint_as_float((uint32_t)(127 - e) << 23);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(bar(L::kBarQR + (pieces & 3)));
        }
        ++pieces;
      }
      ok = wait_all(bar(L::kBarCF + cst), (c / kCodeSt) & 1);
      if (ok && use > 0) ok = wait_all(bar((kv ? L::kBarVE : L::kBarKE) + st), (use - 1) & 1);
      if (!ok) break;
      const uint8_t* src = smem + L::kOffC + cst * kCodeBytes + key0 * 128 + q8 * 16;
      const uint32_t dst = (kv ? sV : sK) + st * kKVBytes;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint4 raw[kIts / 2];   // loads first: the stores below are ordered among themselves
#pragma unroll
        for (int i = 0; i < kIts / 2; ++i)
          raw[i] = *reinterpret_cast<const uint4*>(src + (h * (kIts / 2) + i) * kConvWarps * 512);
#pragma unroll
        for (int i = 0; i < kIts / 2; ++i) {
          const int step = (h * (kIts / 2) + i) * kConvWarps;
          const uint32_t wd[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          uint32_t o[8];
          if constexpr (KV == PA_INT8) {
            const int b = (key0 + step * 4) / BS;
            const float z = 1152.f + (float)(kv ? ti.vz[b] : ti.kz[b]);
            const uint32_t zc = pack_f16x2(z, z);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t u = wd[k] ^ 0x80808080u;
              o[2 * k] = tc::i8x2_to_f16x2(u, 0x4140, zc);
              o[2 * k + 1] = tc::i8x2_to_f16x2(u, 0x4342, zc);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = e4m3x2_to_f16x2((uint16_t)(wd[k] & 0xffffu));
              o[2 * k + 1] = e4m3x2_to_f16x2((uint16_t)(wd[k] >> 16));
            }
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       ::"r"(dst + at0 + step * 512), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       ::"r"(dst + at1 + step * 512), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                       : "memory");
        }
      }
      const int live = ctx - ti.key0, draft0 = base - ti.key0;
      const uint32_t bad = ti.bad;
      if (kv && (live < kKeys || bad != 0 || (KV == PA_FP8_E4M3 && draft0 < kKeys))) {
        const int par = (pieces - 1) & 3;
#pragma unroll 1
        for (int i = 0; i < kIts; ++i) {
          const int step = i * kConvWarps, key = key0 + step * 4;
          const bool gone = key >= live || ((bad >> (key / BS)) & 1u);
          if (gone) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                           ::"r"(dst + (k ? at1 : at0) + step * 512), "r"(0) : "memory");
          } else if (KV == PA_FP8_E4M3 && key >= draft0) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + step * 512);
            const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
            uint32_t nan = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) nan |= (wd[k] & 0x7f7f7f7fu) + 0x01010101u;
            if (!(nan & 0x80808080u)) continue;
#pragma unroll 1
            for (int e = 0; e < 16; ++e)
              if ((src[step * 512 + e] & 0x7f) == 0x7f)
                asm volatile("st.shared.b16 [%0], %1;"
                             ::"r"(dst + (e < 8 ? at0 : at1) + step * 512 + (e & 7) * 2),
                               "h"((uint16_t)0) : "memory");
            const int j = key - draft0;
            atomicOr(&s_odd[par * 8 + (j >> 5)], 1u << (j & 31));
            any_odd[par] = 1;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(bar(L::kBarCE + cst));
      mbar_arrive(bar((kv ? L::kBarVF : L::kBarKF) + st));
    }
  } else if (warp < 4) {
    // ------------------------------ softmax ------------------------------
    const int r = tid;                                 // row of the tile = tensor-memory lane
    const int tok = r / G, head = r - tok * G;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    float sl2 = a.scale_log2;
    int par = 3, pieces = 0;
    uint32_t syncs = 0;
    float m_used = -INFINITY, l = 0.f;
    int base = 0, ctx = 0, rows = 0, kvh = 0, seq = 0, slot = 0;   // of the piece
    int64_t row = 0;    // this thread's token row
    bool live_warp = false;
    float vref = 1.f;   // fp8 / int8: the power of two that P's V scales are relative to
    // the four warps meet, within a bound (one of them may have given up)
    auto meet = [&]() {
      mbar_arrive(bar(L::kBarSm));
      return wait_all(bar(L::kBarSm), syncs++ & 1);
    };
#pragma unroll 1
    for (int g = 0;; ++g) {
      ok = wait_info(g);
      if (!ok) break;
      const TileInfo& ti = info[g % kInfo];
      const int flags = ti.flags;
      if (flags & kEnd) break;
      if (flags & kFirst) {
        m_used = -INFINITY;
        l = 0.f;
        par = (par + 1) & 3;
        base = ti.base;
        ctx = ti.ctx;
        rows = ti.rows;
        kvh = ti.kvh;
        seq = ti.s;
        slot = ti.slot;
        row = ti.row0 + min(tok, rows - 1);
        live_warp = warp * 32 < rows * G;
        if constexpr (QUANT) {
          vref = 0.f;
          ok = wait_all(bar(L::kBarQR + (pieces & 3)), (pieces >> 2) & 1);
          if (!ok) break;
          sl2 = a.scale_log2 * reinterpret_cast<const float*>(smem + L::kOffDown)[(pieces & 3) * kRows + r];
          ++pieces;
        }
      }
      float beta = 1.f;
      if constexpr (QUANT) {
        float vmax = ti.vs[0];
#pragma unroll
        for (int b = 1; b < NB; ++b) vmax = fmaxf(vmax, ti.vs[b]);
        if (!(vmax <= vref)) {
          // the next power of two, within a range whose reciprocal is one too
          const int e = max(27, min(227, (int)((__float_as_uint(vmax) >> 23) & 0xff) + 1));
          const float up = __uint_as_float((uint32_t)e << 23);
          beta = vref > 0.f ? fminf(vref / up, 1.f) : 1.f;
          vref = fmaxf(vref, up);
        }
      }
      const uint32_t bad = ti.bad;
      const int key0 = ti.key0, live = ctx - key0, draft0 = base - key0;
      const bool masked = draft0 < kKeys || bad != 0;
      uint64_t view = ~0ull;
      if (masked && live_warp) {
        view = tile_view(a, row, key0, base, ctx);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if ((bad >> b) & 1u) view &= ~(((1ull << BS) - 1ull) << (b * BS));
      }
      ok = wait_all(bar(L::kBarSF + (g & 1)), (g >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (live_warp) {
        const uint32_t sbuf = lanes + (g & 1) * kKeys;
        const float rvs = vref > 0.f ? 128.f / vref : 0.f;   // 0: every V scale so far is
        const bool fast = !masked && !(flags & kFirst) && beta == 1.f &&
                          softmax_tile_fast<BS, QUANT>(sbuf, ti, sl2, rvs, m_used, l);
        const float alpha = fast ? 1.f :
            beta * (masked ? softmax_tile<BS, QUANT, true>(sbuf, ti, sl2, rvs, view, m_used, l)
                           : softmax_tile<BS, QUANT, false>(sbuf, ti, sl2, rvs, view, m_used, l));
        if (!fast && !(flags & kFirst) && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O holds the tiles before this one once their last product is done
          ok = wait_all(bar(L::kBarO + ((g - 1) & 1)), ((g - 1) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(lanes + kOCol + c * 32, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(lanes + kOCol + c * 32, o);
          }
          tmem_wait_st();
        }
      }
      if constexpr (!QUANT) {
        // V rows that cannot be read or lie behind the context may hold anything: zero them.
        // A NaN or infinity in a draft's V row is taken out too (see the converters).
        if (masked || live < kKeys) {
          ok = wait_all(bar(L::kBarVF + g % L::kVSt), (g / L::kVSt) & 1);
          if (!ok) break;
          const int key = r & (kKeys - 1);
          const uint32_t vrow = sV + (g % L::kVSt) * kKVBytes + (r >> 6) * kKVSlab + key * 128;
          const bool gone = key >= live || ((bad >> (key / BS)) & 1u);
          if (gone || key >= draft0) {
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const uint32_t addr = vrow + ((k + r) & 7) * 16;
              uint32_t x[4] = {0, 0, 0, 0};
              bool odd = false;
              if (!gone) {
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr) : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const bool lo = (x[i] & 0x7f80u) == 0x7f80u, hi = (x[i] & 0x7f800000u) == 0x7f800000u;
                  odd |= lo || hi;
                  x[i] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                }
              }
              if (gone || odd)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                             ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
              if (odd) {
                const int j = key - draft0;
                atomicOr(&s_odd[par * 8 + (j >> 5)], 1u << (j & 31));
                any_odd[par] = 1;
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      tc_fence_before();
      mbar_arrive(bar(L::kBarP + (g & 1)));
      if (!(flags & kLast)) continue;

      // ---- the piece is done: O / l, or the partial ----
      const bool has_drafts = key0 + kKeys > base;
      const bool live_row = tok < rows, whole = (flags & kWhole) != 0;
      ok = wait_all(bar(L::kBarO + (g & 1)), (g >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      // rows that see a draft with a NaN or infinity in V get it back: the four warps have
      // all written the list before one reads it, and read it before it is emptied
      bool odd = false;
      if (KV != PA_INT8 && has_drafts) {
        ok = meet();
        if (!ok) break;
        odd = any_odd[par] != 0;
      }
      const int64_t orow = row * a.num_q_heads + kvh * G + head;
      uint16_t* op = static_cast<uint16_t*>(a.out) + orow * kDim;
      float4* ap = reinterpret_cast<float4*>(ws.acc) + (int64_t)slot * (kDim / 4) * kRows + r;
      const float unit = QUANT ? vref * (1.f / 128.f) : 1.f;
      const float inv = l != 0.f ? unit / l : 0.f;
      if (live_warp) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(lanes + kOCol + c * 32, o);
          tmem_wait_ld(o);
          if (live_row && whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 w;
              w.x = pack_bf16x2(__uint_as_float(o[8 * k + 0]) * inv, __uint_as_float(o[8 * k + 1]) * inv);
              w.y = pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv);
              w.z = pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv);
              w.w = pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv);
              *reinterpret_cast<uint4*>(op + c * 32 + 8 * k) = w;
            }
          } else if (live_row) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              ap[(c * 8 + k) * kRows] =
                  make_float4(__uint_as_float(o[4 * k]) * unit, __uint_as_float(o[4 * k + 1]) * unit,
                              __uint_as_float(o[4 * k + 2]) * unit, __uint_as_float(o[4 * k + 3]) * unit);
          }
          __syncwarp();
        }
        if (live_row) {
          if (whole) {
            if (a.lse_out != nullptr)
              a.lse_out[orow] = l != 0.f ? (m_used + __log2f(l)) * kLn2 : -INFINITY;
          } else {
            ws.m[slot * kRows + r] = m_used;
            ws.l[slot * kRows + r] = l;
          }
        }
      }
      if (odd) {  // rare: what this thread wrote is mended in place
        if (live_row) {
#pragma unroll 1
          for (int j = 0; j < ctx - base; ++j) {
            if (!((s_odd[par * 8 + (j >> 5)] >> (j & 31)) & 1u)) continue;
            if (!((a.tree_mask[row * a.mask_words + (j >> 5)] >> (j & 31)) & 1u)) continue;
            const int key = base + j;
            const int64_t blk = a.block_tables[(int64_t)seq * a.max_blocks_per_seq + key / BS];
            const int64_t at = ((blk * Hkv + kvh) * BS + key % BS) * kDim;
#pragma unroll 1
            for (int d = 0; d < kDim; ++d) {
              float v;
              if constexpr (!QUANT) {
                v = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.v_cache)[at + d] << 16);
                if ((__float_as_uint(v) & 0x7f800000u) != 0x7f800000u) continue;
              } else {
                if ((static_cast<const uint8_t*>(a.v_cache)[at + d] & 0x7f) != 0x7f) continue;
                v = __uint_as_float(0x7fc00000u);
              }
              if (whole) {
                const float x = __uint_as_float((uint32_t)op[d] << 16) + v;
                op[d] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xffff);
              } else {
                reinterpret_cast<float*>(ap + (d >> 2) * kRows)[d & 3] += v;
              }
            }
          }
        }
        ok = meet();
        if (!ok) break;
        if (tid < 8) s_odd[par * 8 + tid] = 0;
        if (tid == 0) any_odd[par] = 0;
        ok = meet();
        if (!ok) break;
      }
      tc_fence_before();  // O is read before the next P is handed over
    }
  }
  if (!ok && lane == 0) flag_error(PA_DEVERR_TIMEOUT);

  // ------------------------------ teardown ------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    pf::tmem_dealloc(tmem, kCols);
  }
}

// Joins the pieces of every (row tile, sequence, kv head) that a cut falls into: grid (cuts,
// 4 x 32 rows). The cut where it is first cut does the work; thread (warp w, lane) takes row
// lane of the group and channels 8 w .. 8 w + 7, pieces in order, eight pieces' reads in
// flight (a context of 20000 tokens in a small batch has two dozen). Bound by latency: two
// dependent reads and a round trip per eight pieces.
constexpr int kReduceThreads = 512;

__global__ void __launch_bounds__(kReduceThreads) tree_tc_reduce_kernel(const TreeArgs a,
                                                                        const Workspace ws) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x + 1;
  const RunInfo run = ws.runs[b];
  const int64_t tile0 = run.begin + kPieceCost;               // where its first tile is
  if (run.tiles == 0 || run.per * b <= tile0) return;         // no run, or no tile cut off
  const int first = (int)(tile0 / run.per);
  if (first != b - 1) return;
  const int last = (int)((tile0 + run.tiles - 1) / run.per);
  const int G = a.group, TM = kRows / G;
  const int q0 = a.query_start[run.s], n = a.query_start[run.s + 1] - q0;
  const int rows = min(TM, n - run.rt * TM) * G;
  const int r = 32 * blockIdx.y + (threadIdx.x & 31), w = threadIdx.x >> 5;
  if (r >= rows) return;
  // a pair that begins inside run `first` is its last piece, one that begins it its first
  const int64_t slot0 = (int64_t)first * 2 + (run.begin > run.per * first ? 1 : 0);
  auto slot_of = [&](int k) { return k == first ? slot0 : (int64_t)k * 2; };
  float M = -INFINITY;
#pragma unroll 8
  for (int k = first; k <= last; ++k) M = fmaxf(M, ws.m[slot_of(k) * kRows + r]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 8
  for (int k = first; k <= last; ++k) {
    const int64_t slot = slot_of(k);
    const float4* src = reinterpret_cast<const float4*>(ws.acc) + (slot * (kDim / 4) + 2 * w) * kRows + r;
    const float4 u = src[0], v = src[kRows];
    const float f = fast_exp2(ws.m[slot * kRows + r] - ref);
    L = fmaf(f, ws.l[slot * kRows + r], L);
    x.x = fmaf(f, u.x, x.x); x.y = fmaf(f, u.y, x.y); x.z = fmaf(f, u.z, x.z); x.w = fmaf(f, u.w, x.w);
    y.x = fmaf(f, v.x, y.x); y.y = fmaf(f, v.y, y.y); y.z = fmaf(f, v.z, y.z); y.w = fmaf(f, v.w, y.w);
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  const int64_t row = (int64_t)(q0 + run.rt * TM + r / G) * a.num_q_heads + run.kvh * G + r % G;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * kDim + 8 * w) =
      make_uint4(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv),
                 pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
  if (w == 0 && a.lse_out != nullptr)
    a.lse_out[row] = L != 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

// q [T][Hq][128] as (64 channels, half, head, token); a box is the Q tile's rows of one half.
inline bool make_q_map(CUtensorMap* m, const TreeArgs& a) {
  auto enc = tc::encoder();
  if (enc == nullptr) return false;
  const int rows = a.q_rows;
  cuuint64_t dims[4] = {64, 2, (cuuint64_t)a.num_q_heads, (cuuint64_t)a.num_tokens};
  cuuint64_t strides[3] = {128, 256, (cuuint64_t)a.num_q_heads * 256};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)a.group, (cuuint32_t)(rows / a.group)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int BS, pa_dtype KV>
inline cudaError_t launch_bs(TreeArgs a, const Workspace& ws, cudaStream_t st) {
  using L = Layout<KV != PA_BF16>;
  const int most = a.max_query_len * a.group;   // rows of a sequence and kv head
  a.q_rows = most > kRows / 2 ? kRows : KV != PA_BF16 && most <= kRows / 4 ? kRows / 4 : kRows / 2;
  CUtensorMap qm, km, vm;
  const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * BS;
  const bool maps = KV == PA_BF16 ? pf::make_kv_map(&km, a.k_cache, rows, BS) &&
                                        pf::make_kv_map(&vm, a.v_cache, rows, BS)
                                  : pf::make_kv8_map(&km, a.k_cache, rows, BS) &&
                                        pf::make_kv8_map(&vm, a.v_cache, rows, BS);
  if (!maps || !make_q_map(&qm, a))
    return cudaErrorInvalidValue;
  static tc::DeviceCache slots;
  int per_sm = 0;
  cudaError_t e = tc::resident_per_sm(tree_tc_kernel<BS, KV>, L::kThreads, L::kSmem, slots, &per_sm);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_tc_kernel<BS, KV>, dim3(kStreams), dim3(L::kThreads), L::kSmem, st, a, ws,
                 qm, km, vm);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_tc_reduce_kernel, dim3(kStreams - 1, kRows / 32),
                    dim3(kReduceThreads), 0, st, a, ws);
}

inline cudaError_t launch_tc(const TreeArgs& a, pa_dtype kv, const Workspace& ws, cudaStream_t st) {
  auto by_bs = [&](auto kvc) -> cudaError_t {
    constexpr pa_dtype KV = decltype(kvc)::value;
    if (a.block_size == 8) return launch_bs<8, KV>(a, ws, st);
    if (a.block_size == 32) return launch_bs<32, KV>(a, ws, st);
    return launch_bs<16, KV>(a, ws, st);
  };
  if (kv == PA_FP8_E4M3) return by_bs(std::integral_constant<pa_dtype, PA_FP8_E4M3>{});
  if (kv == PA_INT8) return by_bs(std::integral_constant<pa_dtype, PA_INT8>{});
  return by_bs(std::integral_constant<pa_dtype, PA_BF16>{});
}

}  // namespace tree
}  // namespace pa
