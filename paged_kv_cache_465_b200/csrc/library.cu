// The library's one CUDA translation unit (so that every kernel shares one device error word
// and one kernel-family setting): decode, prefill and cache entry points (pagedattn.cu), and
// those of a drafted step. Declarations and contracts: include/pagedattn.h.
#include <algorithm>
#include <initializer_list>

#include "pagedattn.cu"

#include "rotary.cuh"
#include "step_ops.cuh"
#include "tree_mma.cuh"
#include "tree_simt.cuh"

namespace pa {
namespace {

// Memory of one buffer of a call; `out`: the call writes it.
struct Span {
  const void* p;
  int64_t bytes;
  bool out;
};

// Whether no output shares memory with another buffer (absent ones have no pointer).
bool apart(std::initializer_list<Span> all) {
  for (const Span& a : all) {
    if (!a.out || a.p == nullptr || a.bytes == 0) continue;
    const char* a0 = static_cast<const char*>(a.p);
    for (const Span& b : all) {
      const char* b0 = static_cast<const char*>(b.p);
      if (&a != &b && b0 != nullptr && b.bytes > 0 && a0 < b0 + b.bytes && b0 < a0 + a.bytes) return false;
    }
  }
  return true;
}

// Parts of the context on the CUDA-core path: enough CTAs for about eight per SM, at most
// one part per 512 tokens (below that the joining costs more than the split gives).
int tree_simt_parts(const pa_decode_desc* d, int num_tokens, int max_context_len) {
  const int64_t rows = std::max<int64_t>(1, (int64_t)num_tokens * d->num_kv_heads);
  const int64_t most = (max_context_len + 511) / 512;
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, (1184 + rows - 1) / rows));
}

// What the tensor-core kernel takes: bf16 q / out, a bf16, fp8 or int8 cache, head_dim 128, a group
// that divides its row tiles, blocks of 8, 16 or 32 tokens.
bool tree_mma(const pa_decode_desc* d) { return prefill_tc_supported(d); }

// Tokens of a part on the tensor cores. Few (row tile, sequence, kv head)s: as many parts as make
// just under 1776 CTAs when every context is as long as allowed, four rounds of the 444 places that
// tiles of 32 and 64 rows have, six of 296 with 128 rows (8 x 65536 bf16 tokens: 27 parts 352 us;
// 28, which begin a fifth round of a few CTAs, 380; 61 parts 415, 17 parts 397). Many: parts of 2048
// tokens, so that the longest contexts do not make the last round alone (256 of 16 .. 8192 fp8
// tokens: 215 us; 4096-token parts 227, 1024 229, whole contexts 251). Contexts of one length pay
// for that cut: 256 of 2056 fp8 tokens, cut into 2048 and 8, take 364 us and 297 whole (256 of 1032,
// left whole, 173, and 228 in halves). Parts under 128 tokens cost more to join than they give. The
// parts' results stay within 192 MB (a thousandth of the GPU's memory): longer parts otherwise.
// The rule knows what is allowed, not the lengths, which are on the device: with 131072 allowed,
// 32 requests of at most 4112 bf16 tokens take 113 us instead of 45, 256 of at most 8200 fp8 tokens
// 265 instead of 215, 13 of at most 20064 int8 tokens 413 instead of 113.
int tree_mma_part(const pa_decode_desc* d, int num_tokens, int max_query_len,
                  int max_context_len) {
  const int group = d->num_q_heads / d->num_kv_heads, R = tree::mma_rows(max_query_len, group);
  const int tm = R / group;
  const int64_t pairs = (int64_t)((max_query_len + tm - 1) / tm) * d->num_seqs * d->num_kv_heads;
  constexpr int64_t kCtas = 6 * 296;
  const int64_t fit = std::max<int64_t>(
      1, (192ll << 20) / ((int64_t)num_tokens * d->num_q_heads * (2 + d->head_dim) * 4));
  const int64_t want = pairs >= kCtas ? 1 : kCtas / pairs;
  int64_t p = pairs >= kCtas
                  ? 2048 : std::max<int64_t>(128, ((int64_t)max_context_len + want - 1) / want);
  p = std::max<int64_t>(p, ((int64_t)max_context_len + fit - 1) / fit);
  return (int)std::min<int64_t>((p + 63) / 64 * 64, 1 << 30);
}

int parts_of(int max_context_len, int part) {
  return (int)(((int64_t)max_context_len + part - 1) / part);
}

size_t tree_bytes(const pa_decode_desc* d, int num_tokens, int max_query_len, int max_context_len) {
  // either kernel family, so that pa_set_decode_impl does not change it
  int parts = tree_simt_parts(d, num_tokens, max_context_len);
  if (tree_mma(d))
    parts = std::max(parts, parts_of(max_context_len, tree_mma_part(d, num_tokens, max_query_len,
                                                                    max_context_len)));
  return parts == 1 ? 0 : (size_t)num_tokens * d->num_q_heads * parts * (2 + d->head_dim) * 4;
}

template <pa_dtype KV, int D, int GP>
cudaError_t launch_tree_simt(const tree::TreeArgs& a, cudaStream_t st) {
  if constexpr (GP * D <= 2048) {
    const dim3 grid(a.num_tokens, a.num_kv_heads, a.parts);
    cudaError_t e = launch_pdl(tree::tree_simt_kernel<KV, D, GP>, grid, dim3(kSimtWarps * 32), 0, st, a);
    if (e != cudaSuccess || a.parts == 1) return e;
    return tree::launch_reduce<D>(a, st);
  } else {
    return cudaErrorInvalidValue;
  }
}

template <pa_dtype KV, int D>
cudaError_t launch_tree_simt_g(const tree::TreeArgs& a, cudaStream_t st) {
  switch (pad_group(a.group)) {
    case 1: return launch_tree_simt<KV, D, 1>(a, st);
    case 2: return launch_tree_simt<KV, D, 2>(a, st);
    case 4: return launch_tree_simt<KV, D, 4>(a, st);
    case 8: return launch_tree_simt<KV, D, 8>(a, st);
    default: return launch_tree_simt<KV, D, 16>(a, st);
  }
}

template <pa_dtype KV>
cudaError_t launch_tree_simt_d(const tree::TreeArgs& a, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_tree_simt_g<KV, 64>(a, st);
    case 128: return launch_tree_simt_g<KV, 128>(a, st);
    default: return launch_tree_simt_g<KV, 256>(a, st);
  }
}

bool tree_desc_ok(const pa_decode_desc* d, int num_tokens, int max_query_len, int max_context_len) {
  return desc_ok(d) && (d->partition_size == 0 || d->partition_size == PA_PARTITION_AUTO) &&
         num_tokens >= 0 && max_query_len >= 0 && max_query_len <= step::kMaxTree &&
         max_context_len >= max_query_len;
}

// desc_supported reads the partition of a decode call; a tree call has none
bool tree_supported(const pa_decode_desc* d) {
  pa_decode_desc one = *d;
  one.partition_size = 0;
  return desc_supported(&one);
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status paged_build_step(const int32_t* context_lens, const int32_t* new_lens,
                           const int32_t* blocks_held, const int32_t* parents,
                           int32_t* block_tables, const int32_t* free_blocks,
                           const int32_t* queue_state, int num_seqs, int max_blocks_per_seq,
                           int block_size, int num_blocks, int free_capacity, int max_tokens,
                           int mask_words, int32_t* total_lens, int32_t* query_start,
                           int32_t* blocks_held_out, int32_t* queue_state_out,
                           int64_t* slot_mapping, int32_t* positions, uint32_t* tree_mask,
                           int32_t* status, void* stream) {
  if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || block_size <= 0 ||
      num_blocks <= 0 || free_capacity <= 0 || max_tokens < 0 ||
      (int64_t)max_blocks_per_seq * block_size > INT32_MAX)
    return PA_ERR_INVALID;
  if (tree_mask && (mask_words < 1 || mask_words > step::kMaxWords)) return PA_ERR_INVALID;
  if (num_seqs == 0) {
    if (!context_lens && new_lens) return PA_OK;  // no batch at all
  } else if (!context_lens || !new_lens || !blocks_held || !block_tables || !total_lens ||
             !blocks_held_out) {
    return PA_ERR_INVALID;
  }
  // an idle step's outputs are written like any other's
  if (!free_blocks || !queue_state || !query_start || !queue_state_out ||
      (max_tokens > 0 && !slot_mapping))
    return PA_ERR_INVALID;
  // every CTA reads the inputs while the first writes the outputs
  const int64_t S4 = 4 * (int64_t)num_seqs, T4 = 4 * (int64_t)max_tokens;
  if (!apart({{context_lens, S4, false}, {new_lens, S4, false}, {blocks_held, S4, false},
              {parents, T4, false}, {block_tables, S4 * max_blocks_per_seq, true},
              {free_blocks, 4 * (int64_t)free_capacity, false}, {queue_state, 8, false},
              {total_lens, S4, true}, {query_start, S4 + 4, true}, {blocks_held_out, S4, true},
              {queue_state_out, 8, true}, {slot_mapping, 2 * T4, true}, {positions, T4, true},
              {tree_mask, T4 * mask_words, true}, {status, 4, true}}))
    return PA_ERR_INVALID;
  const step::BuildArgs a{context_lens, new_lens, blocks_held, parents, block_tables, free_blocks,
                          queue_state, total_lens, query_start, blocks_held_out, queue_state_out,
                          slot_mapping, positions, tree_mask, status, num_seqs,
                          max_blocks_per_seq, block_size, num_blocks, free_capacity, max_tokens,
                          mask_words};
  const unsigned grid = (unsigned)std::max<int64_t>(
      1, ((int64_t)max_tokens + step::kBuildThreads - 1) / step::kBuildThreads);
  const cudaError_t e = launch_pdl(step::build_step_kernel, dim3(grid), dim3(step::kBuildThreads), 0,
                                   as_stream(stream), a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status paged_release_blocks(const int32_t* keep_lens, const int32_t* blocks_held,
                               const int32_t* block_tables, int32_t* free_blocks,
                               const int32_t* queue_state, int num_seqs,
                               int max_blocks_per_seq, int block_size, int free_capacity,
                               int32_t* blocks_held_out, int32_t* queue_state_out,
                               int32_t* status, void* stream) {
  if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || block_size <= 0 ||
      free_capacity <= 0)
    return PA_ERR_INVALID;
  if (num_seqs == 0) {
    if (!keep_lens && blocks_held) return PA_OK;  // no batch at all
  } else if (!keep_lens || !blocks_held || !block_tables || !blocks_held_out) {
    return PA_ERR_INVALID;
  }
  if (!free_blocks || !queue_state || !queue_state_out) return PA_ERR_INVALID;
  const int64_t S4 = 4 * (int64_t)num_seqs;
  if (!apart({{keep_lens, S4, false}, {blocks_held, S4, false},
              {block_tables, S4 * max_blocks_per_seq, false},
              {free_blocks, 4 * (int64_t)free_capacity, true}, {queue_state, 8, false},
              {blocks_held_out, S4, true}, {queue_state_out, 8, true}, {status, 4, true}}))
    return PA_ERR_INVALID;
  // 64 sequences per CTA, more when that would be over one CTA per SM (148 of them)
  const int per = std::max(64, (num_seqs + 147) / 148);
  const step::ReleaseArgs a{keep_lens, blocks_held, block_tables, free_blocks, queue_state,
                            blocks_held_out, queue_state_out, status, num_seqs,
                            max_blocks_per_seq, block_size, free_capacity, per};
  const cudaError_t e = launch_pdl(step::release_blocks_kernel,
                                   dim3(std::max(1, (num_seqs + per - 1) / per)),
                                   dim3(step::kReleaseThreads), 0, as_stream(stream), a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status rotary_and_cache(const void* q, const void* k, const void* v, void* q_out,
                           void* k_cache, void* v_cache, const int32_t* positions,
                           const int64_t* slot_mapping, const float* inv_freq,
                           const pa_rotary_desc* desc, const float* k_scales,
                           const float* v_scales, const int32_t* k_zeros,
                           const int32_t* v_zeros, void* stream) {
  if (desc == nullptr) return PA_ERR_INVALID;
  const pa_rotary_desc& d = *desc;
  if (d.num_tokens < 0 || d.num_q_heads <= 0 || d.num_kv_heads <= 0 || d.block_size <= 0 ||
      d.num_blocks <= 0 || d.num_axes < 1 || d.num_axes > 4 || d.rotary_dim <= 0 ||
      d.rotary_dim % 16 != 0 || d.rotary_dim > d.head_dim)
    return PA_ERR_INVALID;
  int sum = 0;
  for (int i = 0; i < d.num_axes; ++i) {
    if (d.sections[i] < 0 || d.sections[i] > d.rotary_dim / 2) return PA_ERR_INVALID;
    sum += d.sections[i];
  }
  if (sum != d.rotary_dim / 2) return PA_ERR_INVALID;
  if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (d.in_dtype != PA_F32 && d.in_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (d.cache_dtype != PA_F32 && d.cache_dtype != PA_BF16 && d.cache_dtype != PA_FP8_E4M3 &&
      d.cache_dtype != PA_INT8)
    return PA_ERR_UNSUPPORTED;
  if (d.cache_dtype == PA_F32 && d.in_dtype != PA_F32) return PA_ERR_UNSUPPORTED;
  if (d.num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !q_out || !k_cache || !v_cache || !positions || !slot_mapping || !inv_freq)
    return PA_ERR_INVALID;
  const int64_t qrow = (int64_t)d.num_q_heads * d.head_dim, krow = (int64_t)d.num_kv_heads * d.head_dim;
  if (d.q_stride < qrow || d.q_out_stride < qrow || d.k_stride < krow || d.v_stride < krow)
    return PA_ERR_INVALID;
  const int64_t align = d.in_dtype == PA_F32 ? 4 : 8;  // 16-byte accesses
  if (d.q_stride % align || d.k_stride % align || d.v_stride % align || d.q_out_stride % align)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
      !aligned16(v_cache))
    return PA_ERR_INVALID;
  // q_out is q or lies apart from it
  const int64_t es = dtype_bytes(d.in_dtype), more = d.num_tokens - 1;
  if (q_out == q ? d.q_out_stride != d.q_stride
                 : !apart({{q, (more * d.q_stride + qrow) * es, false},
                           {q_out, (more * d.q_out_stride + qrow) * es, true}}))
    return PA_ERR_INVALID;
  const bool quant = d.cache_dtype == PA_FP8_E4M3 || d.cache_dtype == PA_INT8;
  if (quant && (!k_scales || !v_scales)) return PA_ERR_INVALID;
  if (d.cache_dtype == PA_INT8 && (!k_zeros || !v_zeros)) return PA_ERR_INVALID;
  rot::RotaryArgs a{q, k, v, q_out, k_cache, v_cache, positions, slot_mapping, inv_freq,
                    k_scales, v_scales, k_zeros, v_zeros, d.q_stride, d.k_stride, d.v_stride,
                    d.q_out_stride, d.num_tokens, d.num_q_heads, d.num_kv_heads, d.head_dim,
                    d.rotary_dim, {0, 0, 0, 0}, d.adjacent_pairs != 0, d.block_size, d.num_blocks};
  for (int i = 0, end = 0; i < 4; ++i) {
    if (i < d.num_axes) end += d.sections[i];
    a.sec_end[i] = i < d.num_axes ? end : d.rotary_dim / 2;
  }
  const cudaStream_t st = as_stream(stream);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(d.num_tokens), dim3(rot::kThreads), 0, st, a);
  };
  cudaError_t e;
  if (d.in_dtype == PA_F32) {
    switch (d.cache_dtype) {
      case PA_F32: e = go(rot::rotary_kernel<PA_F32, PA_F32>); break;
      case PA_BF16: e = go(rot::rotary_kernel<PA_F32, PA_BF16>); break;
      case PA_INT8: e = go(rot::rotary_kernel<PA_F32, PA_INT8>); break;
      default: e = go(rot::rotary_kernel<PA_F32, PA_FP8_E4M3>); break;
    }
  } else {
    switch (d.cache_dtype) {
      case PA_BF16: e = go(rot::rotary_kernel<PA_BF16, PA_BF16>); break;
      case PA_INT8: e = go(rot::rotary_kernel<PA_BF16, PA_INT8>); break;
      default: e = go(rot::rotary_kernel<PA_BF16, PA_FP8_E4M3>); break;
    }
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t paged_attn_tree_workspace_size(const pa_decode_desc* desc, int num_tokens,
                                      int max_query_len, int max_context_len) {
  if (!tree_desc_ok(desc, num_tokens, max_query_len, max_context_len) || !tree_supported(desc) ||
      desc->num_seqs == 0 || num_tokens == 0 || max_query_len == 0)
    return 0;
  return tree_bytes(desc, num_tokens, max_query_len, max_context_len);
}

pa_status paged_attn_tree(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens,
                          const int32_t* query_start, const uint32_t* tree_mask,
                          int mask_words, int num_tokens, int max_query_len, float scale,
                          void* out, const pa_decode_desc* desc, int max_context_len,
                          const float* k_scales, const float* v_scales, const int32_t* k_zeros,
                          const int32_t* v_zeros, float* lse_out, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!tree_desc_ok(desc, num_tokens, max_query_len, max_context_len) || !std::isfinite(scale) ||
      mask_words < 1 || mask_words > step::kMaxWords || max_query_len > 32 * mask_words)
    return PA_ERR_INVALID;
  if (!tree_supported(desc)) return PA_ERR_UNSUPPORTED;
  if (desc->num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !tree_mask ||
      !out)
    return PA_ERR_INVALID;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q) || !aligned16(out))
    return PA_ERR_INVALID;
  if ((int64_t)desc->max_blocks_per_seq * desc->block_size < (int64_t)max_context_len)
    return PA_ERR_INVALID;
  const bool quant = desc->kv_dtype == PA_FP8_E4M3 || desc->kv_dtype == PA_INT8;
  if (quant && (!k_scales || !v_scales)) return PA_ERR_INVALID;
  if (desc->kv_dtype == PA_INT8 && (!k_zeros || !v_zeros)) return PA_ERR_INVALID;
  const size_t need = paged_attn_tree_workspace_size(desc, num_tokens, max_query_len, max_context_len);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;

  tree::TreeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.block_tables = block_tables; a.context_lens = context_lens; a.query_start = query_start;
  a.tree_mask = tree_mask; a.out = out; a.lse_out = lse_out;
  a.k_scales = k_scales; a.v_scales = v_scales; a.k_zeros = k_zeros; a.v_zeros = v_zeros;
  a.scale_log2 = scale * kLog2e;
  a.num_seqs = desc->num_seqs; a.num_tokens = num_tokens;
  a.num_q_heads = desc->num_q_heads; a.num_kv_heads = desc->num_kv_heads;
  a.group = desc->num_q_heads / desc->num_kv_heads;
  a.max_blocks_per_seq = desc->max_blocks_per_seq; a.num_blocks = desc->num_blocks;
  a.block_size = desc->block_size; a.mask_words = mask_words;
  a.max_context_len = max_context_len; a.max_query_len = max_query_len;
  a.q_dtype = desc->q_dtype; a.out_dtype = desc->out_dtype;
  const cudaStream_t st = as_stream(stream);
  cudaError_t e;
  const bool mma = tree_mma(desc) && g_decode_impl.load(std::memory_order_relaxed) != 1;
  if (mma) {
    a.part_tokens = tree_mma_part(desc, num_tokens, max_query_len, max_context_len);
    a.parts = parts_of(max_context_len, a.part_tokens);
  } else {
    a.parts = tree_simt_parts(desc, num_tokens, max_context_len);
    a.part_tokens = (int)round_up((size_t)(max_context_len + a.parts - 1) / a.parts, kSub);
  }
  a.direct = mma;
  const size_t rows = (size_t)num_tokens * desc->num_q_heads * a.parts;
  a.part_acc = static_cast<float*>(workspace);
  a.part_m = a.part_acc + rows * desc->head_dim;
  a.part_l = a.part_m + rows;
  if (mma) {
    e = desc->kv_dtype == PA_BF16 ? tree::launch_mma<PA_BF16>(a, st)
        : desc->kv_dtype == PA_INT8 ? tree::launch_mma<PA_INT8>(a, st)
                                    : tree::launch_mma<PA_FP8_E4M3>(a, st);
  } else switch (desc->kv_dtype) {
    case PA_F32: e = launch_tree_simt_d<PA_F32>(a, desc->head_dim, st); break;
    case PA_BF16: e = launch_tree_simt_d<PA_BF16>(a, desc->head_dim, st); break;
    case PA_INT8: e = launch_tree_simt_d<PA_INT8>(a, desc->head_dim, st); break;
    default: e = launch_tree_simt_d<PA_FP8_E4M3>(a, desc->head_dim, st); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status tree_verify(const int32_t* parents, const int64_t* draft_tokens,
                      const int64_t* target_tokens, const int32_t* query_start,
                      const int32_t* context_lens, int num_seqs, int num_tokens,
                      int max_accept, int32_t* accepted, int32_t* num_accepted,
                      int64_t* next_tokens, int32_t* kept_lens, void* stream) {
  if (num_seqs < 0 || num_seqs > 65535 || num_tokens < 0 || max_accept < 1) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if ((num_tokens > 0 && (!parents || !draft_tokens || !target_tokens)) || !query_start ||
      !context_lens || !accepted || !num_accepted || !next_tokens || !kept_lens)
    return PA_ERR_INVALID;
  const int64_t S4 = 4 * (int64_t)num_seqs, T4 = 4 * (int64_t)num_tokens;
  if (!apart({{parents, T4, false}, {draft_tokens, 2 * T4, false}, {target_tokens, 2 * T4, false},
              {query_start, S4 + 4, false}, {context_lens, S4, false},
              {accepted, S4 * max_accept, true}, {num_accepted, S4, true},
              {next_tokens, 2 * S4, true}, {kept_lens, S4, true}}))
    return PA_ERR_INVALID;
  const step::VerifyArgs a{parents, draft_tokens, target_tokens, query_start, context_lens,
                           accepted, num_accepted, next_tokens, kept_lens, num_seqs, num_tokens,
                           max_accept};
  const cudaError_t e = launch_pdl(step::tree_verify_kernel, dim3((num_seqs + 3) / 4), dim3(128), 0,
                                   as_stream(stream), a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status compact_accepted(void* k_cache, void* v_cache, const int32_t* block_tables,
                           const int32_t* context_lens, const int32_t* query_start,
                           const int32_t* accepted, const int32_t* num_accepted, int num_seqs,
                           int max_accept, int max_blocks_per_seq, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks, pa_dtype cache_dtype,
                           const float* k_scales, const float* v_scales,
                           const int32_t* k_zeros, const int32_t* v_zeros, void* stream) {
  if (num_seqs < 0 || num_seqs > 65535 || max_accept < 1 || max_accept > step::kMaxTree ||
      max_blocks_per_seq <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks <= 0)
    return PA_ERR_INVALID;
  if (cache_dtype != PA_F32 && cache_dtype != PA_BF16 && cache_dtype != PA_FP8_E4M3 &&
      cache_dtype != PA_INT8)
    return PA_ERR_UNSUPPORTED;
  const int64_t row_bytes = (int64_t)head_dim * dtype_bytes(cache_dtype);
  if (row_bytes % 16 != 0 || row_bytes > 65536) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !query_start || !accepted ||
      !num_accepted || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID;
  const bool quant = cache_dtype == PA_FP8_E4M3 || cache_dtype == PA_INT8;
  if (quant && (!k_scales || !v_scales)) return PA_ERR_INVALID;
  if (cache_dtype == PA_INT8 && (!k_zeros || !v_zeros)) return PA_ERR_INVALID;
  const step::CompactArgs a{static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
                            block_tables, context_lens, query_start, accepted, num_accepted,
                            k_scales, v_scales, k_zeros, v_zeros, num_seqs, max_accept,
                            max_blocks_per_seq, num_kv_heads, (int)row_bytes, block_size,
                            num_blocks};
  const cudaStream_t st = as_stream(stream);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(num_seqs), dim3(256), 0, st, a);
  };
  cudaError_t e;
  switch (cache_dtype) {
    case PA_FP8_E4M3: e = go(step::compact_accepted_kernel<PA_FP8_E4M3>); break;
    case PA_INT8: e = go(step::compact_accepted_kernel<PA_INT8>); break;
    default: e = go(step::compact_accepted_kernel<PA_BF16>); break;  // rows move as bytes
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
