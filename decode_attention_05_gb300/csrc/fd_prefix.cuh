// fd_prefix.cuh -- attention of a batch whose rows share prompts: what its kernels have in
// common (fd_decode_shared_prefix; the host side is fd_prefix_api.cu).
//
// Rows group_start[p] .. group_start[p + 1] - 1 of the batch share prompt p (prefix_lens[p]
// tokens).  The softmax over a row's keys -- the prompt's, then its own -- is cut at that
// border as the split-KV merge cuts a sequence ("AI Infra: math and infra optimisation in
// large models", section 2.6, Flash-Decoding Split-K): a partial (O_i, LSE_i) of every piece,
// merged with weights exp(LSE_i - max).  For the prompt's pieces the queries of all rows of
// the group are one tall matrix (n rows x Q query tokens x G heads for each kv head), so its
// K and V are read once for the group and not once a row.  Every key of the prompt precedes
// every query: no causal mask there.
//
// Work is cut into row tiles of BM query rows of one group (x kv heads x splits of the
// prompt).  Splits are even shares of each prompt's own length, in whole BN-token tiles.
#pragma once

#include "fd_device.cuh"

namespace fd {

struct PrefixParams {
  int32_t B, Q, Hq, Hkv, G, P;
  int32_t log2_g;                   // G is a power of two
  uint32_t per_row_inv;             // ceil(2^32 / (Q G)), 0 for Q G = 1: see prefix_row
  const void* q;                    // [B, Q, Hq, d]
  int64_t q_sb, q_sj, q_sh;
  const void *k, *v;                // [P, Hkv, L_cap, d] or pages [num_pages, Hkv, page, d]
  int64_t k_sb, k_sh, k_st, v_sb, v_sh, v_st;
  const int32_t* prefix_lens;       // [P]
  const int32_t* group_start;       // [P + 1], or nullptr: one group of all rows (P = 1)
  const int32_t* table;             // [P, pages] or nullptr
  int64_t table_sb, num_pages, L_cap;
  int32_t page_size, log2_page;
  int32_t S;                        // splits of a prompt
  float* lse_part;                  // [B, Q, Hq, S], -inf: no key in the split
  float* o_part;                    // [B, Q, Hq, S, d]
  uint32_t* flags;
  float scale_log2;                 // log2(e) / sqrt(d)
  int32_t selftest_stall;           // n > 0: CTA (0, 0, 0)'s producer stops before its copy n - 1
  const float *k_scale, *v_scale;   // FP8: per kv head, or nullptr = 1
};

// One CTA's work: BM query rows (from row0 of the group's) against one split of a prompt.
struct PrefixTile {
  int32_t group;        // P: the rows behind the last group, which have no prompt
  int32_t b0;           // first batch row of the group
  int32_t row0, rows;   // first query row of the tile in the group, and its rows (<= BM)
  int64_t L;            // the prompt's length (clamped)
  int64_t lo, hi;       // the split's tokens
};

// Batch rows [b0, b1) of group g; out-of-range or unordered offsets are clamped and flagged.
__device__ __forceinline__ void group_rows(const PrefixParams& p, int g, int& b0, int& b1) {
  if (p.group_start == nullptr) {
    b0 = g == 0 ? 0 : p.B;
    b1 = p.B;
    return;
  }
  const int s0 = g == 0 ? 0 : p.group_start[g];
  const int s1 = g < p.P ? p.group_start[g + 1] : p.B;
  b0 = min(max(s0, 0), p.B);
  b1 = min(max(s1, b0), p.B);
  if (b0 != s0 || b1 != s1 || (g == 0 && p.group_start[0] != 0)) atomicOr(p.flags, FD_DEVFLAG_OFFSETS);
}

// The tile that index z names: the groups' tiles in order, and behind them those of the
// rows that no group holds.  Called by one whole warp (32 groups at a time); false: there
// is no such tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const PrefixParams& p, int z, PrefixTile& t) {
  const int lane = threadIdx.x & 31;
  const int per_row = p.Q * p.G;
  if (p.group_start == nullptr) {             // one group: no search
    t.group = 0;
    t.b0 = 0;
    t.row0 = z * BM;
    t.rows = min(BM, p.B * per_row - t.row0);
    return t.rows > 0;
  }
  int before = 0;
  for (int g0 = 0; g0 <= p.P; g0 += 32) {
    const int g = g0 + lane;
    int b0 = 0, b1 = 0;
    if (g <= p.P) group_rows(p, g, b0, b1);
    const int tiles = (int)(((int64_t)(b1 - b0) * per_row + BM - 1) / BM);
    int upto = tiles;                         // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > z);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      const int first = __shfl_sync(0xffffffffu, before + upto - tiles, src);
      const int rows = __shfl_sync(0xffffffffu, (b1 - b0) * per_row, src);
      t.group = g0 + src;
      t.b0 = __shfl_sync(0xffffffffu, b0, src);
      t.row0 = (z - first) * BM;
      t.rows = min(BM, rows - t.row0);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// The tile's prompt length and split `s` of it: whole BN-token tiles, evenly shared.
template <int BN>
__device__ __forceinline__ void split_of(const PrefixParams& p, int s, PrefixTile& t) {
  int64_t L = t.group < p.P ? p.prefix_lens[t.group] : 0;
  if (L < 0 || L > p.L_cap) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.flags, FD_DEVFLAG_SEQ_LEN);
    L = L < 0 ? 0 : p.L_cap;
  }
  t.L = L;
  const int64_t tiles = (L + BN - 1) / BN;
  t.lo = tiles * s / p.S * BN;
  t.hi = min(tiles * (s + 1) / p.S * BN, L);
}

// Query row r of a tile: its batch row b, query token j and head g G + h.  A row's place x in
// its group is divided by Q G as floor(x inv / 2^32), inv = ceil(2^32 / (Q G)): exact as long as
// x (Q G - 1) < 2^32, and x < 65536 * 64, Q G <= 64.
__device__ __forceinline__ void prefix_row(const PrefixParams& p, const PrefixTile& t, int r, int& b, int& j, int& h) {
  const int x = t.row0 + r;
  const int i = p.per_row_inv ? (int)__umulhi((unsigned)x, p.per_row_inv) : x;
  const int y = x - i * p.Q * p.G;
  b = t.b0 + i;
  j = y >> p.log2_g;
  h = y & (p.G - 1);
}
// Its flat index over [B, Q, Hq], and where its query starts.
__device__ __forceinline__ int64_t prefix_flat_row(const PrefixParams& p, const PrefixTile& t, int g, int r) {
  int b, j, h;
  prefix_row(p, t, r, b, j, h);
  return ((int64_t)b * p.Q + j) * p.Hq + (int64_t)g * p.G + h;
}
__device__ __forceinline__ int64_t prefix_q_offset(const PrefixParams& p, const PrefixTile& t, int g, int r) {
  int b, j, h;
  prefix_row(p, t, r, b, j, h);
  return (int64_t)b * p.q_sb + (int64_t)j * p.q_sj + ((int64_t)g * p.G + h) * p.q_sh;
}

// The merge of a row's partials: those of its prompt (set 0) and of its own keys (set 1).
struct MergeParams {
  int32_t rows, Q, Hq, d;
  int32_t S[2];
  const float* lse[2];              // [rows, S]
  const float* o[2];                // [rows, S, d]
  void* out;
  int64_t out_sb, out_sj, out_sh;
  int32_t out_bf16;
  float* lse_out;                   // [rows] or nullptr
};

// Tiles of BM query rows that a call can have at most: with group_start each non-empty group,
// and the rows behind the last (one group may have some too), may end in a tile of its own.
inline int64_t prefix_row_tiles(int64_t B, int64_t per_row, bool grouped, int64_t P, int64_t BM) {
  if (!grouped) return (B * per_row + BM - 1) / BM;
  const int64_t parts = P + 1 < B ? P + 1 : B;
  return B * per_row / BM + parts;
}

cudaError_t launch_prefix_simt(const PrefixParams& p, int32_t dtype, int d, cudaStream_t stream);
// The tensor-core pass: bf16 or FP8 caches; boxes of the tensor maps tk, tv as prefix_tc_box says.
void prefix_tc_box(int page_size, uint32_t* tokens, uint32_t* lines);
cudaError_t launch_prefix_tc(const PrefixParams& p, bool fp8, int d, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t stream);
cudaError_t launch_prefix_merge(const MergeParams& p, cudaStream_t stream);

// Launch with programmatic dependent launch, as the partial kernels are.
template <class Kernel, class... Args>
cudaError_t launch_pdl(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fd
