// fd_prefix_api.cu -- the C ABI of attention over shared prompts (include/fd.h): argument
// checks, the prompt pass's split count, workspace layout, and the three launches of a call:
// partials over the shared prompts (fd_prefix.cuh), partials over each row's own cache (the
// kernels of fd_decode_partial), and the merge of both sets.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "fd.h"
#include "fd_internal.h"
#include "fd_prefix.cuh"

namespace {

constexpr int32_t kMaxSplits = 4096;
constexpr size_t kAlign = 256;
constexpr int kRowTile = 256;           // query rows a CTA of the prompt pass serves at most
constexpr int64_t kMinSplitTokens = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

fd_status bad(const char* message) { return fd::record_error(FD_ERR_INVALID_ARG, message); }
fd_status unsupported(const char* message) { return fd::record_error(FD_ERR_UNSUPPORTED, message); }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int esize(int32_t dtype) { return dtype == FD_F8E4M3 ? 1 : dtype == FD_BF16 ? 2 : 4; }

bool sizes_ok(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv, int64_t d, int64_t P, int64_t Lp,
              int32_t prefix_splits) {
  return B > 0 && Q > 0 && Hq > 0 && Hkv > 0 && d > 0 && P > 0 && Lp > 0 && prefix_splits >= 0 &&
         prefix_splits <= kMaxSplits && Hq % Hkv == 0 && B * Q * Hq <= INT32_MAX;
}

// Workspace: what fd_decode_partial needs for the rows' own splits (its header of device
// flags first), then the prompts' LSE_i [B, Q, Hq, S] and O_i [B, Q, Hq, S, d].
struct Layout {
  size_t own, lse_off, o_off, total;
};
Layout layout(int32_t B, int32_t Q, int32_t Hq, int32_t Hkv, int32_t d, int32_t Sp, int32_t S) {
  Layout w;
  const size_t rows = (size_t)B * Q * Hq;
  w.own = fd_workspace_size(B, Q * Hq, Hkv, d, S);
  w.lse_off = align_up(w.own);
  w.o_off = align_up(w.lse_off + rows * Sp * sizeof(float));
  w.total = align_up(w.o_off + rows * Sp * d * sizeof(float));
  return w;
}

// Splits of the rows' own keys: the count of a plain decode call, except where its kernel
// leaves SMs without work because it expects long rows.
//  - Small pages (16 and 32 tokens) run head-group tiles, four kv heads a CTA: two CTAs per SM
//    of at least 128 tokens (32 rows of up to 1024 tokens, 16-token pages: 49 -> 22 us).
//  - More than 16 query rows per kv head plan for one CTA per SM: two of at least 64 tokens.
// small_pages: of the table, or true to ask for the larger count of the two (workspace sizes).
int32_t own_splits(int32_t B, int32_t Q, int32_t Hq, int32_t Hkv, int32_t d, int64_t L_cap, int32_t num_splits,
                   bool small_pages) {
  const int32_t s = fd_resolve_num_splits_q(B, Q, Hq, Hkv, d, L_cap, num_splits);
  const bool wide = Q * (Hq / Hkv) > fd::kMaxNarrowRows;
  if (num_splits > 0 || !(wide || (small_pages && d == 128 && Hkv % fd::kHeadGroup == 0))) return s;
  const int64_t ctas = (int64_t)B * (wide ? Hkv : Hkv / fd::kHeadGroup), sms = fd::sm_count();
  const int64_t want = wide ? std::min(2 * sms / ctas, (L_cap + 63) / 64)
                            : std::min(2 * sms / ctas, (L_cap + 127) / 128);
  return (int32_t)std::max<int64_t>(s, std::min<int64_t>(want, kMaxSplits));
}

// Splits of the prompts: those of (row tile, kv head) pairs of groups of equal size fill one
// wave of CTAs.
int32_t prompt_splits(int32_t B, int32_t Q, int32_t Hq, int32_t Hkv, int32_t P, int64_t L_cap,
                      int32_t prefix_splits, int row_tile, int ctas_per_sm, int64_t min_tokens) {
  if (!sizes_ok(B, Q, Hq, Hkv, 1, P, L_cap, prefix_splits)) return 1;
  if (prefix_splits > 0) return prefix_splits;
  const int64_t per = ((int64_t)(B + P - 1) / P) * Q * (Hq / Hkv);
  const int64_t units = (int64_t)Hkv * std::min<int64_t>(P, B) * ((per + row_tile - 1) / row_tile);
  const int64_t s = std::min<int64_t>((int64_t)ctas_per_sm * fd::sm_count() / units,
                                      (L_cap + min_tokens - 1) / min_tokens);
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>(s, kMaxSplits));
}
// Of the CUDA-core pass: 64-row tiles, two CTAs per SM, no split below two of its 64-token
// tiles (its tiles are slow, so a split of 256 tokens is a long chain: 33 rows on 2049 tokens,
// f32, 43 -> 35 us).
int32_t simt_splits(int32_t B, int32_t Q, int32_t Hq, int32_t Hkv, int32_t P, int64_t L_cap, int32_t prefix_splits) {
  return prompt_splits(B, Q, Hq, Hkv, P, L_cap, prefix_splits, 64, 2, 128);
}

// Fewer splits of the tensor-core pass where SMs left to the pass over the rows' own keys,
// which runs at the same time, shorten the whole: the prompts get SMs in proportion to their
// work.  Work is in SM microseconds, from sizes alone (own rows taken as half full):
//   prompts  units x tiles x 0.85 us a 128-token tile (1.2 with two row tiles, 1.6 with pages of
//            up to 16 tokens, 0.2 more for FP8), times 1.7, the weight that fitted best
//   own      SMs x (3 us, 6 with more than 16 query rows per kv head, + bytes / 5.8 TB/s)
// Since the rows may be shorter than their capacity, the prompt pass may get at most 7 us or 12 %
// longer than on all SMs; and it never gives up SMs that the own pass has no CTAs for.
// Measured (one wave of splits -> this count): 32 rows on 8192 tokens, own 1024, 16-token pages
// 36.7 -> 27.9 us (19 -> 8 splits), contiguous 34.7 -> 29.7 (6), 48 rows on 3 prompts 31.5 ->
// 28.3 (6 -> 3), FP8 48 rows on 10000 tokens 36.9 -> 31.5 (19 -> 9 or 10), 64 rows on 4096 tokens
// 31.1 -> 25.0 (16 -> 6).
int32_t side_by_side_splits(const fd::PrefixParams& p, int32_t wave, int d, bool fp8, double own_bytes,
                            int64_t own_ctas) {
  const double sms = fd::sm_count();
  if (sms <= 0) return wave;
  const int64_t per = ((int64_t)(p.B + p.P - 1) / p.P) * p.Q * p.G;
  const double units = (double)p.Hkv * std::min(p.P, p.B) * ((per + kRowTile - 1) / kRowTile);
  const int64_t tiles = (p.L_cap + 127) / 128;
  double tile_us = per > 128 ? 1.2 : 0.85;
  if (p.page_size > 0 && p.page_size <= 16) tile_us = 1.6;
  if (fp8) tile_us += 0.2;
  if (d == 64) tile_us *= 0.6;
  const double prompts = units * tiles * tile_us * 1.7;
  const double own = sms * ((p.Q * p.G > fd::kMaxNarrowRows ? 6.0 : 3.0) + own_bytes / 2 / 5.8e6);
  const double share = std::max(sms * prompts / (prompts + own), sms - (double)((own_ctas + 1) / 2));
  int32_t s = (int32_t)std::max<int64_t>(1, std::min<int64_t>(wave, (int64_t)(share / units + 0.5)));
  auto us = [&](int32_t n) { return (double)((tiles + n - 1) / n) * tile_us; };
  while (s < wave && us(s) > us(wave) + std::max(7.0, 0.12 * us(wave))) ++s;
  return s;
}

struct PromptPass {
  const fd::PrefixParams* p;
  const CUtensorMap *tk, *tv;       // tk nullptr: CUDA cores
  int32_t dtype;
  int d;
  cudaStream_t stream;
};
fd_status launch_prompt_pass(void* arg) {
  const PromptPass& a = *static_cast<const PromptPass*>(arg);
  const cudaError_t e =
      a.tk ? fd::launch_prefix_tc(*a.p, a.dtype == FD_F8E4M3, a.d, *a.tk, *a.tv, a.stream)
           : fd::launch_prefix_simt(*a.p, a.dtype, a.d, a.stream);
  return e == cudaSuccess ? FD_OK : fd::record_error(FD_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int32_t fd_resolve_prefix_splits(int32_t B, int32_t Q, int32_t Hq, int32_t Hkv, int32_t P,
                                 int64_t L_cap, int32_t prefix_splits) {
  return prompt_splits(B, Q, Hq, Hkv, P, L_cap, prefix_splits, kRowTile, 1, kMinSplitTokens);
}

size_t fd_shared_prefix_workspace_size(int32_t B, int32_t Q, int32_t Hq, int32_t Hkv, int32_t d,
                                       int32_t P, int64_t L_prefix_cap, int64_t L_cap,
                                       int32_t prefix_splits, int32_t num_splits) {
  if (!sizes_ok(B, Q, Hq, Hkv, d, P, L_prefix_cap, prefix_splits) || L_cap <= 0 || num_splits < 0 ||
      num_splits > kMaxSplits)
    return 0;
  // The larger of the two passes' counts: the sizes do not say which will run.
  return layout(B, Q, Hq, Hkv, d,
                std::max(fd_resolve_prefix_splits(B, Q, Hq, Hkv, P, L_prefix_cap, prefix_splits),
                         simt_splits(B, Q, Hq, Hkv, P, L_prefix_cap, prefix_splits)),
                own_splits(B, Q, Hq, Hkv, d, L_cap, num_splits, true))
      .total;
}

}  // extern "C"

// A call; stall > 0: fd_selftest_stalled_shared_prefix.
static fd_status run_shared_prefix(const fd_tensor* q, const fd_tensor* k_prefix,
                                   const fd_tensor* v_prefix, const int32_t* prefix_lens,
                                   const int32_t* group_start, const fd_tensor* prefix_table,
                                   const fd_tensor* k_cache, const fd_tensor* v_cache,
                                   const float* k_scale, const float* v_scale,
                                   const int32_t* seq_lens, const fd_tensor* block_table,
                                   int32_t page_size, int32_t prefix_splits, int32_t num_splits,
                                   fd_tensor* out, float* lse_out, void* workspace,
                                   size_t workspace_bytes, void* stream, const fd_options* options,
                                   int32_t stall) {
  if (!q || !k_prefix || !v_prefix || !k_cache || !v_cache || !out)
    return bad("q, k_prefix, v_prefix, k_cache, v_cache and out are required");
  if (!q->data || !k_prefix->data || !v_prefix->data || !k_cache->data || !v_cache->data || !out->data)
    return bad("a tensor has a NULL data pointer");
  if (!prefix_lens || !seq_lens) return bad("prefix_lens and seq_lens are required");
  if (!workspace) return bad("workspace is NULL");
  if ((q->ndim != 3 && q->ndim != 4) || k_prefix->ndim != 4 || v_prefix->ndim != 4 ||
      k_cache->ndim != 4 || v_cache->ndim != 4 || out->ndim != q->ndim)
    return bad("ranks must be q 3 or 4, k/v 4, out as q");
  if (prefix_splits < 0 || prefix_splits > kMaxSplits || num_splits < 0 || num_splits > kMaxSplits)
    return bad("prefix_splits and num_splits must be in [0, 4096]");
  const bool multi = q->ndim == 4;
  const int hd = multi ? 2 : 1;
  const int64_t B = q->shape[0], Q = multi ? q->shape[1] : 1, Hq = q->shape[hd], d = q->shape[hd + 1];
  const int64_t Hkv = k_cache->shape[1];
  if (B <= 0 || Q <= 0 || Hq <= 0 || d <= 0 || Hkv <= 0) return bad("empty shape");
  for (int i = 0; i < q->ndim; ++i)
    if (out->shape[i] != q->shape[i]) return bad("out must have q's shape");
  for (int i = 0; i < 4; ++i) {
    if (k_prefix->shape[i] != v_prefix->shape[i]) return bad("k_prefix and v_prefix shapes differ");
    if (k_prefix->shape[i] <= 0) return bad("empty prefix shape");
  }
  if (k_prefix->shape[1] != Hkv || k_prefix->shape[3] != d)
    return bad("the prefix's heads or head dim differ from the cache's or q's");
  if (Hq % Hkv != 0) return bad("Hq is not a multiple of Hkv");
  // ---- types (those of the rows' own cache are checked with its partial pass)
  const int32_t kd = k_cache->dtype;
  if (k_prefix->dtype != kd || v_prefix->dtype != kd) return bad("the prefix must have the cache's dtype");
  const bool fp8 = kd == FD_F8E4M3;
  if ((k_scale || v_scale) && !fp8) return bad("k_scale / v_scale belong to an FP8 E4M3 cache only");
  if (q->dtype != (fp8 ? FD_BF16 : kd) || (kd != FD_BF16 && kd != FD_F32 && !fp8))
    return bad("q must have the caches' dtype (bf16 or f32), or be bf16 with FP8 caches");
  if (out->dtype != FD_F32 && !(out->dtype == FD_BF16 && q->dtype == FD_BF16))
    return unsupported("out must be f32, or bf16 with bf16 inputs");
  if (d != 64 && d != 128) return unsupported("head dim not in {64, 128}");
  if (fp8 && d != 128) return unsupported("the FP8 KV cache needs head dim 128");
  // ---- strides and alignment
  const int es = esize(kd);
  if (q->stride[q->ndim - 1] != 1 || k_prefix->stride[3] != 1 || v_prefix->stride[3] != 1 ||
      out->stride[out->ndim - 1] != 1)
    return bad("the last dimension of q, k, v and out must be contiguous");
  if (!aligned16(q->data) || !aligned16(k_prefix->data) || !aligned16(v_prefix->data) || !aligned16(out->data))
    return bad("q, k_prefix, v_prefix and out must be 16-byte aligned");
  for (int i = 0; i + 1 < q->ndim; ++i) {
    if ((q->stride[i] * esize(q->dtype)) % 16) return bad("q strides must be multiples of 16 bytes");
    if ((out->stride[i] * esize(out->dtype)) % 16) return bad("out strides must be multiples of 16 bytes");
    if (out->stride[i] <= 0 && out->shape[i] > 1) return bad("out strides must be positive");
  }
  for (int i = 0; i < 3; ++i)
    if (k_prefix->stride[i] <= 0 || v_prefix->stride[i] <= 0 || (k_prefix->stride[i] * es) % 16 ||
        (v_prefix->stride[i] * es) % 16)
      return bad("prefix strides must be positive multiples of 16 bytes");
  if (k_prefix->stride[2] < d || v_prefix->stride[2] < d) return bad("prefix token rows overlap");
  // ---- prompts: contiguous or paged
  int64_t P = k_prefix->shape[0], Lp = k_prefix->shape[2];
  int log2_page = 0;
  if (prefix_table) {
    if (!prefix_table->data) return bad("prefix_table has a NULL data pointer");
    if (prefix_table->ndim != 2 || prefix_table->dtype != FD_I32 || prefix_table->shape[0] <= 0 ||
        prefix_table->shape[1] <= 0 || prefix_table->stride[1] != 1)
      return bad("prefix_table must be int32 [P, max_pages] with contiguous rows");
    if (page_size < 8 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
      return bad("page_size must be a power of two in [8, 65536]");
    if (k_prefix->shape[2] != page_size) return bad("paged prefixes must be [num_pages, Hkv, page_size, d]");
    while ((1 << log2_page) < page_size) ++log2_page;
    P = prefix_table->shape[0];
    Lp = prefix_table->shape[1] * page_size;
  }
  if (!prefix_table && !block_table && page_size != 0) return bad("page_size must be 0 without a table");
  if (Lp >= (int64_t{1} << 31)) return bad("prefix capacity must be below 2^31");
  if (!group_start && P != 1) return bad("group_start is required for more than one prefix");
  if (P > 65535 || B > 65535 || Hkv > 65535) return unsupported("grid too large");
  if (lse_out && ((uintptr_t)lse_out & 3)) return bad("lse_out must be 4-byte aligned");
  if (((uintptr_t)prefix_lens & 3) || ((uintptr_t)group_start & 3)) return bad("prefix_lens and group_start must be 4-byte aligned");
  int path;
  if (!fd::call_path(options, &path))
    return bad("fd_options holds an unknown path, merge mode or schedule");
  // ---- splits and workspace
  const int64_t G = Hq / Hkv;
  if (Q * G > fd::kMaxRows) return unsupported("more than 64 query rows per kv head (Q x Hq / Hkv)");
  if (G > 64 || (G & (G - 1)) != 0) return unsupported("group size not in {1, 2, 4, 8, 16, 32, 64}");
  if ((block_table ? block_table->shape[0] : k_cache->shape[0]) != B)
    return bad("k_cache or block_table has another batch size than q");
  const int64_t L_cap = block_table ? block_table->shape[1] * page_size : k_cache->shape[2];
  // ---- the prompt pass: tensor cores for bf16 and FP8, CUDA cores for f32 or when asked for
  // (with FP8 that is refused with the rows' own keys below)
  const bool tc = kd != FD_F32 && path != FD_PATH_SIMT;
  const int32_t Sp = (tc ? fd_resolve_prefix_splits : simt_splits)((int32_t)B, (int32_t)Q, (int32_t)Hq, (int32_t)Hkv,
                                                                   (int32_t)P, Lp, prefix_splits);
  const int32_t S = own_splits((int32_t)B, (int32_t)Q, (int32_t)Hq, (int32_t)Hkv, (int32_t)d, L_cap, num_splits,
                               block_table && (page_size == 16 || page_size == 32));
  if (((uintptr_t)workspace & (kAlign - 1)) != 0) return bad("workspace must be 256-byte aligned");
  const Layout wl = layout((int32_t)B, (int32_t)Q, (int32_t)Hq, (int32_t)Hkv, (int32_t)d, Sp, S);
  if (workspace_bytes < wl.total)
    return fd::record_error(FD_ERR_WORKSPACE_TOO_SMALL, "workspace is smaller than fd_shared_prefix_workspace_size");
  if (fd::prefix_row_tiles(B, Q * G, group_start != nullptr, P, 16) > 65535) return unsupported("grid too large");

  fd::PrefixParams p;
  memset(&p, 0, sizeof p);
  p.B = (int32_t)B, p.Q = (int32_t)Q, p.Hq = (int32_t)Hq, p.Hkv = (int32_t)Hkv, p.G = (int32_t)G, p.P = (int32_t)P;
  while ((1 << p.log2_g) < p.G) ++p.log2_g;
  p.per_row_inv = Q * G > 1 ? (uint32_t)(((uint64_t{1} << 32) + Q * G - 1) / (Q * G)) : 0;
  p.q = q->data;
  p.q_sb = q->stride[0], p.q_sj = multi ? q->stride[1] : 0, p.q_sh = q->stride[hd];
  p.k = k_prefix->data, p.v = v_prefix->data;
  p.k_sb = k_prefix->stride[0], p.k_sh = k_prefix->stride[1], p.k_st = k_prefix->stride[2];
  p.v_sb = v_prefix->stride[0], p.v_sh = v_prefix->stride[1], p.v_st = v_prefix->stride[2];
  p.prefix_lens = prefix_lens;
  p.group_start = group_start;
  p.table = prefix_table ? static_cast<const int32_t*>(prefix_table->data) : nullptr;
  p.table_sb = prefix_table ? prefix_table->stride[0] : 0;
  p.num_pages = prefix_table ? k_prefix->shape[0] : 0;
  p.L_cap = Lp;
  p.page_size = prefix_table ? page_size : 0;
  p.log2_page = log2_page;
  p.S = Sp;
  if (tc && prefix_splits == 0)
    p.S = side_by_side_splits(p, Sp, (int)d, fp8, 2.0 * B * L_cap * Hkv * d * es, B * Hkv * S);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.lse_part = reinterpret_cast<float*>(ws + wl.lse_off);
  p.o_part = reinterpret_cast<float*>(ws + wl.o_off);
  p.flags = reinterpret_cast<uint32_t*>(ws);
  p.scale_log2 = (float)(1.4426950408889634 / __builtin_sqrt((double)d));
  p.selftest_stall = stall;
  p.k_scale = fp8 ? k_scale : nullptr;
  p.v_scale = fp8 ? v_scale : nullptr;

  CUtensorMap tk, tv;
  if (tc) {
    uint32_t tokens, lines;
    fd::prefix_tc_box(p.page_size, &tokens, &lines);
    fd_status st = fd::kv_map(k_prefix, tokens, lines, &tk);
    if (st == FD_OK) st = fd::kv_map(v_prefix, tokens, lines, &tv);
    if (st != FD_OK) return st;
  }

  // The rows' own keys: once their arguments are accepted too, the prompt pass is launched (on
  // error nothing is), and their pass right behind it, to run on the SMs that it leaves free --
  // it is bound by the tensor cores with many rows, theirs by memory.
  PromptPass prompt = {&p, tc ? &tk : nullptr, &tv, kd, (int)d, (cudaStream_t)stream};
  const fd_status st = fd::run_partial_behind(q, k_cache, v_cache, k_scale, v_scale, seq_lens, block_table,
                                              block_table ? page_size : 0, S, workspace, wl.own, stream,
                                              options, &launch_prompt_pass, &prompt);
  if (st != FD_OK) return st;
  const cudaStream_t s = (cudaStream_t)stream;

  fd::MergeParams mp;
  memset(&mp, 0, sizeof mp);
  mp.rows = (int32_t)(B * Q * Hq);
  mp.Q = (int32_t)Q, mp.Hq = (int32_t)Hq, mp.d = (int32_t)d;
  mp.S[0] = p.S, mp.S[1] = S;
  mp.lse[0] = p.lse_part, mp.o[0] = p.o_part;
  float *lse_own = nullptr, *o_own = nullptr;
  fd_workspace_partials(workspace, (int32_t)B, (int32_t)(Q * Hq), (int32_t)d, S, &lse_own, &o_own);
  mp.lse[1] = lse_own, mp.o[1] = o_own;
  mp.out = out->data;
  mp.out_sb = out->stride[0], mp.out_sj = multi ? out->stride[1] : 0, mp.out_sh = out->stride[hd];
  mp.out_bf16 = out->dtype == FD_BF16 ? 1 : 0;
  mp.lse_out = lse_out;
  const cudaError_t e = fd::launch_prefix_merge(mp, s);
  if (e != cudaSuccess) return fd::record_error(FD_ERR_CUDA, cudaGetErrorString(e));
  return FD_OK;
}

extern "C" {

fd_status fd_decode_shared_prefix(const fd_tensor* q, const fd_tensor* k_prefix,
                                  const fd_tensor* v_prefix, const int32_t* prefix_lens,
                                  const int32_t* group_start, const fd_tensor* prefix_table,
                                  const fd_tensor* k_cache, const fd_tensor* v_cache,
                                  const float* k_scale, const float* v_scale,
                                  const int32_t* seq_lens, const fd_tensor* block_table,
                                  int32_t page_size, int32_t prefix_splits, int32_t num_splits,
                                  fd_tensor* out, float* lse_out, void* workspace,
                                  size_t workspace_bytes, void* stream,
                                  const fd_options* options) {
  return run_shared_prefix(q, k_prefix, v_prefix, prefix_lens, group_start, prefix_table, k_cache,
                           v_cache, k_scale, v_scale, seq_lens, block_table, page_size,
                           prefix_splits, num_splits, out, lse_out, workspace, workspace_bytes,
                           stream, options, 0);
}

fd_status fd_selftest_stalled_shared_prefix(
    const fd_tensor* q, const fd_tensor* k_prefix, const fd_tensor* v_prefix,
    const int32_t* prefix_lens, const int32_t* group_start, const fd_tensor* prefix_table,
    const fd_tensor* k_cache, const fd_tensor* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* seq_lens, const fd_tensor* block_table, int32_t page_size, int32_t prefix_splits,
    int32_t num_splits, fd_tensor* out, float* lse_out, void* workspace, size_t workspace_bytes,
    void* stream, const fd_options* options, int32_t stall_copy) {
  if (stall_copy < 0) return bad("stall_copy must be >= 0");
  return run_shared_prefix(q, k_prefix, v_prefix, prefix_lens, group_start, prefix_table, k_cache,
                           v_cache, k_scale, v_scale, seq_lens, block_table, page_size,
                           prefix_splits, num_splits, out, lse_out, workspace, workspace_bytes,
                           stream, options, stall_copy + 1);
}

}  // extern "C"
