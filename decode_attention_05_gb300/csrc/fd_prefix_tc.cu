// fd_prefix_tc.cu -- attention of many query rows over a shared prompt on the 5th-generation
// tensor cores (fd_prefix.cuh says what the pass computes): bf16 q; bf16 caches with d 64 or
// 128, or FP8 E4M3 caches with d = 128.
//
// A CTA serves one kv head, one split of one prompt and up to 256 query rows of its group, as
// two streams of 128 rows, one softmax warpgroup each:
//   S_w[128 rows, 128 tokens] = Q_w . K_tile^T     tcgen05.mma, both operands in shared memory
//   thread r of the warpgroup reads row r of S from tensor memory, keeps the running maximum m
//   and sum l of the softmax, and writes P = bf16(2^(S - m)) over S's own columns
//   O_w[128, d] += P . V_tile                      tcgen05.mma, P in tensor memory
// ("AI Infra: math and infra optimisation in large models", section 2.6, the FlashAttention
// block update.)  With more than 128 rows the streams are two row tiles that share every K and
// V tile.  With at most 128 rows both streams have the same rows and take alternate tiles, as
// two independent partial softmaxes that are merged at the end: one stream's products run
// while the other's softmax does, whatever the number of rows.
//
// Each stream has a warp that issues its products: P V of a tile, then at once Q K^T of the
// next (in order behind the read of P, whose columns it overwrites).  So the tensor cores work
// on one stream while the other's warps do their softmax.  The softmax uses the maximum m of
// the tiles before, and O is rescaled (and the tile's weights formed again) only when the
// tile's maximum exceeds m by more than 8 (base 2): weights then reach at most 2^8, and l and
// O use the same m, so the result is the same -- and the exponentials need not wait for the
// maximum.
//
// Bound: with 256 rows a CTA does 2 x 4 x 128 x 128 x d flops on a tile of 512 d bytes of K
// and V: the tensor cores (2048 cycles a tile at d = 128) and the SM's share of HBM bandwidth
// (about 24 bytes a cycle: 2700 cycles) are near balance; several row tiles read a prompt's
// tiles from L2.
//
// Warps: 0-3 and 4-7 the softmax of stream 0 and 1, 8 the TMA producer, 9 and 10 the issuers,
// 12-19 the widening (FP8).  Tensor memory: S_0, S_1 (128 columns each, P over their first halves), O_0, O_1 (d each).  Shared
// memory: Q (2 x 128 rows), then a ring of K and V tiles (32 KB at d = 128, 5 of them), each
// [64-dim slab][token][128 B], 128-byte swizzle.  A page of fewer than 128 tokens is loaded
// slab by slab, so that a tile has the same layout whatever the page size.
//
// FP8 caches: TMA fills a ring of code tiles (16 KB), and two more warpgroups widen them, one
// the K and one the V tiles, to f16 (exactly: E4M3 fits f16) into the operand ring, so the
// products are those of f16 q, K, P and V.  (8-bit products would need q and P in 8 bits.)  A
// weight in f16 is off by 2^-11 of itself or, below 2^-14, by 2^-25: over n keys the output by
// at most n 2^-25 max |v|, far below its own rounding.  A kv head's scale of K multiplies the
// scores, its scale of V the output.
//
// Measured (GB300; 8 kv heads, d = 128): 64 rows of 64 heads on 131072 tokens, bf16: 172 us of
// this kernel, 1.6 PFLOP/s on 144 SMs; 512 rows a kv head on 16384 tokens 34 us, 10 us of them
// the start and the 19 MB of partials; 128 rows of 32 heads on 32768 tokens, FP8: 62 us, bound
// by shared memory (operands, codes in, tiles widened out).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fd_prefix.cuh"
#include "fd_tcgen05.cuh"

namespace fd {
namespace {

constexpr int kRows = 128, kTok = 128;
constexpr uint32_t kCols = 512, kOCol = 256;
constexpr int kMaxStages = 9;
constexpr int kPad = 4;              // floats behind each row of the results' scratch

template <int D_, bool FP8_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool FP8 = FP8_;
  static constexpr int THREADS = FP8 ? 640 : 384;
  static constexpr uint32_t TYPE = FP8 ? 0u : 1u;               // operands f16 or bf16
  // Weights (16-bit pairs) formed between stores: fewer where five warpgroups share the registers.
  static constexpr int CH = FP8 ? 16 : 32;
  static constexpr int SLABS = D / 64;
  static constexpr uint32_t SLAB_BYTES = kTok * 128;            // 64 dims of 128 tokens
  static constexpr uint32_t TILE_BYTES = SLABS * SLAB_BYTES;
  static constexpr int STAGES = FP8 ? 4 : D == 128 ? 5 : 8;
  static constexpr uint32_t RING_OFF = 2 * TILE_BYTES;          // behind Q
  // The ring of a CTA with one row tile (bf16) also has the second one's place of Q.
  static __device__ __forceinline__ uint32_t ring_off(bool two_rows) {
    return FP8 || two_rows ? RING_OFF : RING_OFF - TILE_BYTES;
  }
  static __device__ __forceinline__ int stages(bool two_rows) { return FP8 || two_rows ? STAGES : STAGES + 1; }
  // FP8: tiles of codes.  Two, and two more in the second row tile's place of Q where there
  // is none (with few rows the pass is bound by how much it has in flight).
  static constexpr uint32_t RAW_BYTES = kTok * 128;
  static constexpr uint32_t RAW_OFF = RING_OFF + STAGES * TILE_BYTES;
  static constexpr uint32_t CTL_OFF = RAW_OFF + (FP8 ? 2 * RAW_BYTES : 0);
  static __device__ __forceinline__ uint32_t raw_offset(int st) {
    return st < 2 ? RAW_OFF + st * RAW_BYTES : TILE_BYTES + (st - 2) * RAW_BYTES;
  }
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];   // ring: a K or V tile has landed / been read
  uint64_t raw_full[4], raw_empty[4];             // FP8: a tile of codes has landed / been widened
  uint64_t s_full[2];                             // S of the stream's next tile is complete
  uint64_t p_half[2][2];                          // the first / second 64 tokens of P are in place
  uint64_t o_full[2];                             // the stream's last product is complete
  uint64_t turn[2];                               // the other stream's products have been issued
  uint64_t mma_done;                              // all products of the CTA are complete
  uint32_t bad[8];                                // tile n mod 8: bit j = its page j is invalid
  int32_t abort, found;
  uint32_t tmem;
  PrefixTile tile;
};

template <class SH>
constexpr size_t smem_bytes() {
  return SH::CTL_OFF + sizeof(Ctl);
}
static_assert(smem_bytes<Shape<128, false>>() <= 227 * 1024 && smem_bytes<Shape<64, false>>() <= 227 * 1024 &&
                  smem_bytes<Shape<128, true>>() <= 227 * 1024,
              "one CTA per SM");
static_assert(2 * kRows * (128 + kPad) * 4 <= 5 * Shape<128, false>::TILE_BYTES &&
                  2 * kRows * (64 + kPad) * 4 <= 8 * Shape<64, false>::TILE_BYTES &&
                  2 * kRows * (128 + kPad) * 4 <= Shape<128, true>::CTL_OFF - Shape<128, true>::RING_OFF,
              "the results' scratch lies in the drained ring");

__device__ __forceinline__ bool aborted(Ctl* c) {
  return *reinterpret_cast<volatile int32_t*>(&c->abort) != 0;
}
__device__ __forceinline__ void set_abort(const PrefixParams& p, Ctl* c) {
  *reinterpret_cast<volatile int32_t*>(&c->abort) = 1;
  atomicOr(p.flags, kDevFlagTimeout);
}
// A bounded wait that also gives up once another role has.  The clock is read only after some
// tries: a wait in a running pipeline ends within a few.
__device__ __forceinline__ bool wait_or_abort(Ctl* c, uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_probe(bar, parity, 200u)) {
    if (aborted(c) || global_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}
// The same for a warp whose lanes have to agree.
__device__ __forceinline__ bool warp_wait(Ctl* c, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_abort(c, bar, parity));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two f32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------- TMA producer (one warp)
// Ring entry 2 n is the K tile n of the split, 2 n + 1 its V tile.  bf16 tiles go to the
// operand ring, codes to the raw one.
template <class SH>
__device__ void produce(const PrefixParams& p, const PrefixTile& t, int g, int n_tiles, int raw_stages,
                        bool two_rows, const CUtensorMap* tk, const CUtensorMap* tv, uint32_t base, Ctl* ctl,
                        int lane) {
  const uint64_t pol = policy_evict_first();
  const bool paged = p.table != nullptr;
  const int ps = p.page_size;
  const int boxes = paged && ps < kTok ? kTok / ps : 1;      // pages of a tile
  const int64_t used = paged ? (t.L + ps - 1) >> p.log2_page : 0;
  const int stages = SH::FP8 ? raw_stages : SH::stages(two_rows);
  uint64_t* fulls = SH::FP8 ? ctl->raw_full : ctl->full;
  uint64_t* empties = SH::FP8 ? ctl->raw_empty : ctl->empty;
  auto drain = [&](int n) {         // let the copies in flight land before the CTA ends
    for (int i = max(0, n - stages); i < n; ++i) mbar_wait(smem_addr(&fulls[i % stages]), (i / stages) & 1);
  };
  int issued = 0, st = 0, round = 0;          // entry, its stage, and how often the ring wrapped
  bool ok = true;
  for (int n = 0; n < n_tiles && ok; ++n) {
    const int64_t t0 = t.lo + (int64_t)n * kTok;
    int32_t id = t.group;
    int slot = (int)t0;
    if (paged) {                    // lane j: page j of the tile
      const int64_t pi = (t0 >> p.log2_page) + lane;
      id = -2;
      if (lane < boxes && pi < used) id = p.table[(int64_t)t.group * p.table_sb + pi];
      const bool wrong = lane < boxes && pi < used && (id < 0 || id >= p.num_pages);
      const uint32_t bad = __ballot_sync(0xffffffffu, wrong);
      if (bad != 0 && lane == 0) atomicOr(p.flags, FD_DEVFLAG_PAGE);
      if (lane == 0) ctl->bad[n & 7] = bad;
      if (wrong || id == -2) id = 0;          // something to copy: its tokens are masked
      slot = boxes > 1 ? 0 : (int)(t0 & (ps - 1));
    } else if (lane == 0) {
      ctl->bad[n & 7] = 0u;
    }
    __syncwarp();
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t full = smem_addr(&fulls[st]);
      if (p.selftest_stall > 0 && issued == p.selftest_stall - 1 && blockIdx.x == 0 && blockIdx.y == 0 &&
          blockIdx.z == 0)
        return drain(issued);       // as if the next copies never arrived: the others' waits run out
      if (round > 0) ok = warp_wait(ctl, smem_addr(&empties[st]), (round - 1) & 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(full, SH::FP8 ? SH::RAW_BYTES : SH::TILE_BYTES);
      __syncwarp();
      const uint32_t dst = base + (SH::FP8 ? SH::raw_offset(st) : SH::ring_off(two_rows) + st * SH::TILE_BYTES);
      const CUtensorMap* map = kv ? tv : tk;
      if (boxes == 1) {
        if (lane == 0) tma_load_5d(dst, map, full, 0, slot, 0, g, id, pol);
      } else if (lane < boxes) {
#pragma unroll
        for (int x = 0; x < (SH::FP8 ? 1 : SH::SLABS); ++x)
          tma_load_5d(dst + x * SH::SLAB_BYTES + lane * ps * 128, map, full, 0, 0, x, g, id, pol);
      }
      ++issued;
      if (++st == stages) st = 0, ++round;
    }
  }
  if (!ok) {
    if (lane == 0) set_abort(p, ctl);
    drain(issued);
  }
}

// ---------------------------------------------------------------- widening (FP8, two warpgroups)
// Warpgroup kv widens the K (0) or V (1) tiles, thread r token row r of each: 16 codes of one
// 16-byte group become two groups of f16.  A quarter warp's eight rows hit eight different bank groups in both layouts.  Rows
// of tokens without weight become zeros.
template <class SH>
__device__ void widen(const PrefixParams& p, const PrefixTile& t, int n_tiles, int raw_stages, uint8_t* base,
                      Ctl* ctl, int kv, int r) {
  const int lane = r & 31;
  const bool pages = p.table != nullptr && p.page_size < kTok;
  bool ok = true;
  int rs = kv, round = 0;
  for (int n = 0; n < n_tiles; ++n) {
    const int e = 2 * n + kv, st = e % SH::STAGES;
    ok = warp_wait(ctl, smem_addr(&ctl->raw_full[rs]), round & 1);
    if (ok && e >= SH::STAGES) ok = warp_wait(ctl, smem_addr(&ctl->empty[st]), ((e / SH::STAGES) - 1) & 1);
    if (!ok) break;
    const int64_t tok = t.lo + (int64_t)n * kTok + r;
    const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[n & 7]);
    const bool live = tok < t.hi && !((bad >> (pages ? r >> p.log2_page : 0)) & 1u);
    const uint8_t* src = base + SH::raw_offset(rs) + r * 128;
    uint8_t* dst = base + SH::RING_OFF + st * SH::TILE_BYTES + r * 128;
#pragma unroll 4
    for (int c = 0; c < 8; ++c) {
      const uint4 x = live ? *reinterpret_cast<const uint4*>(src + ((c ^ (r & 7)) << 4)) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
            : "r"(w[i]));
      }
      uint8_t* slab = dst + (c >> 2) * SH::SLAB_BYTES;
      const int c0 = (2 * c) & 7;
      *reinterpret_cast<uint4*>(slab + ((c0 ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(slab + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_addr(&ctl->raw_empty[rs]));
      mbar_arrive(smem_addr(&ctl->full[st]));
    }
    rs += 2;
    if (rs >= raw_stages) rs -= raw_stages, ++round;
  }
  if (!ok && lane == 0) set_abort(p, ctl);
}

// ---------------------------------------------------------------- product issuer (a warp a stream)
// The whole warp walks the schedule, so that operand descriptors and addresses stay in uniform
// registers; one elected lane issues the instructions.  (With the schedule inside a branch of
// one lane every product took about 100 cycles to issue, more than it takes to run.)
__device__ __forceinline__ bool elected() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
template <class SH>
__device__ __forceinline__ void issue(const PrefixParams& p, int w, int n_tiles_, bool two_rows_, uint32_t base,
                                      Ctl* ctl) {
  constexpr int D = SH::D;
  constexpr uint32_t id_s = instr_desc(kRows, kTok, 0, SH::TYPE), id_o = instr_desc(kRows, D, 1, SH::TYPE);
  const int n_tiles = __shfl_sync(0xffffffffu, n_tiles_, 0);
  const int two_rows = __shfl_sync(0xffffffffu, two_rows_ ? 1 : 0, 0);
  const int step = two_rows ? 1 : 2;          // a stream's next tile
  const uint64_t q = smem_desc(base + (two_rows ? w * SH::TILE_BYTES : 0u), 0, 1024);
  const uint32_t ring = base + SH::ring_off(two_rows != 0);
  const int stages = SH::stages(two_rows != 0);
  const uint64_t k0 = smem_desc(ring, 0, 1024), v0 = smem_desc(ring, SH::SLAB_BYTES, 1024);
  constexpr uint32_t kTile16 = SH::TILE_BYTES >> 4, kSlab16 = SH::SLAB_BYTES >> 4;   // descriptor units
  // Ring position (stage, parity of its use) of the next K and V tile of this stream.
  const int jump = 2 * step;
  int ks = 0, kp = 0, vs = 0, vp = 0;
  auto advance = [&](int& st, int& par, int by) {
    st += by;
    if (st >= stages) st -= stages, par ^= 1;
  };
  if (!two_rows && w == 1) advance(ks, kp, 2);
  vs = ks, vp = kp;
  advance(vs, vp, 1);
  // What follows is issued by the elected lane.  A ring entry is free once both issuers have
  // committed to it: with one row tile its only user does so twice.
  auto release = [&](int st) {
    tc_commit(smem_addr(&ctl->empty[st]));
    if (!two_rows) tc_commit(smem_addr(&ctl->empty[st]));
  };
  auto scores = [&]() {
    const uint64_t k = k0 + (uint32_t)ks * kTile16;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t off = (i >> 2) * kSlab16 + (i & 3) * 2u;
      tc_mma_ss(w * kTok, q + off, k + off, id_s, i > 0);
    }
  };
  bool ok = true;
  const int first = two_rows ? 0 : w;
  if (first < n_tiles) {
    ok = warp_wait(ctl, smem_addr(&ctl->full[ks]), kp);
    if (ok && elected()) {
      scores();
      tc_commit(smem_addr(&ctl->s_full[w]));
      release(ks);
    }
    __syncwarp();
    advance(ks, kp, jump);
  }
  int i = 0;
  for (int n = first; n < n_tiles && ok; n += step, ++i) {
    const bool more = n + step < n_tiles;
    // Everything but the second half of P before this stream's turn: even a wait that is over
    // takes over a hundred cycles, in which the tensor cores would run dry.  The streams take
    // turns so that they stay out of step, one's products under the other's softmax.
    ok = warp_wait(ctl, smem_addr(&ctl->full[vs]), vp) &&
         (!more || warp_wait(ctl, smem_addr(&ctl->full[ks]), kp)) &&
         ((w == 0 && i == 0) || warp_wait(ctl, smem_addr(&ctl->turn[w]), (w ? i : i - 1) & 1)) &&
         warp_wait(ctl, smem_addr(&ctl->p_half[w][0]), i & 1);
    if (!ok) break;
    const uint64_t v = v0 + (uint32_t)vs * kTile16;
    auto outputs = [&](int half) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        tc_mma_ts(kOCol + w * D, w * kTok + (half * 4 + x) * 8, v + (half * 4 + x) * (2048u >> 4), id_o,
                  (i > 0 || half + x > 0) ? 1u : 0u);
    };
    tc_fence_after();
    if (elected()) outputs(0);
    __syncwarp();
    ok = warp_wait(ctl, smem_addr(&ctl->p_half[w][1]), i & 1);
    if (!ok) break;
    tc_fence_after();
    if (elected()) {
      outputs(1);
      if (more) scores();
      mbar_arrive(smem_addr(&ctl->turn[w ^ 1]));
      tc_commit(smem_addr(more ? &ctl->s_full[w] : &ctl->o_full[w]));   // S is complete behind P V
      if (more) release(ks);
      release(vs);
    }
    __syncwarp();
    if (more) advance(ks, kp, jump);
    advance(vs, vp, jump);
  }
  if (!ok && elected()) set_abort(p, ctl);
  __syncwarp();
  if (elected()) tc_commit(smem_addr(&ctl->mma_done));   // never leave with products in flight
  __syncwarp();
  if (!mbar_wait(smem_addr(&ctl->mma_done), 0)) atomicOr(p.flags, kDevFlagTimeout);
}

// ---------------------------------------------------------------- softmax (a warpgroup a stream)
// The weights 2^(s sl2 - base) of 2 CH scores as pairs of 16-bit operands, added to `sum`.
template <class SH>
__device__ __forceinline__ void weights(const float* s, uint64_t scale2, uint64_t off2, uint32_t* pk, uint64_t* sum) {
#pragma unroll
  for (int j = 0; j < SH::CH; ++j) {
    float a, b;
    unpair(fma2(pair(s[2 * j], s[2 * j + 1]), scale2, off2), a, b);
    a = ex2(a);
    b = ex2(b);
    sum[j & 1] = add2(sum[j & 1], pair(a, b));
    pk[j] = SH::FP8 ? pack_f16(a, b) : pack_bf16(a, b);
  }
}

// Stream w, lane row r.  False if a wait gave up.
template <class SH>
__device__ __forceinline__ bool softmax(const PrefixParams& p, const PrefixTile& t, int n_tiles, bool two_rows,
                                        int w, int r, float sl2, uint8_t* data, Ctl* ctl, float& m, float& l) {
  constexpr int D = SH::D;
  const int lane = r & 31;
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t sc = lanes + w * kTok, oc = lanes + kOCol + w * D;
  const int step = two_rows ? 1 : 2;
  const uint64_t scale2 = pair(sl2, sl2);
  m = kNegInf;
  l = 0.f;
  int left = (int)(t.hi - t.lo) - (two_rows ? 0 : w) * kTok;  // tokens from this tile on
  for (int n = two_rows ? 0 : w, i = 0; n < n_tiles; n += step, ++i, left -= step * kTok) {
    if (!warp_wait(ctl, smem_addr(&ctl->s_full[w]), i & 1)) return false;
    tc_fence_after();
    float s[kTok];
    tc_ld32x2(sc, sc + 32, s);
    tc_ld32x2(sc + 64, sc + 96, s + 64);
    const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[n & 7]);
    if (left < kTok || bad != 0u) { // past the prompt's end, or on an invalid page: no weight
      const int log2_page = p.page_size > 0 && p.page_size < kTok ? p.log2_page : 7;
#pragma unroll
      for (int j = 0; j < kTok; ++j) s[j] = j >= left ? kNegInf : s[j];
      if (bad != 0u) {
#pragma unroll
        for (int j = 0; j < kTok; ++j) s[j] = (bad >> (j >> log2_page)) & 1u ? kNegInf : s[j];
      }
      if constexpr (!SH::FP8) {     // (widen() has cleared them)
        // Their V rows may hold anything, and 0 * NaN would reach O: clear them.
        const int e = 2 * n + 1, stages = SH::stages(two_rows);
        if (!warp_wait(ctl, smem_addr(&ctl->full[e % stages]), (e / stages) & 1)) return false;
        if (r >= left || ((bad >> (r >> log2_page)) & 1u)) {
          uint8_t* v = data + SH::ring_off(two_rows) + (size_t)(e % stages) * SH::TILE_BYTES + r * 128;
#pragma unroll
          for (int c = 0; c < SH::SLABS * 8; ++c)
            *reinterpret_cast<uint4*>(v + (c >> 3) * SH::SLAB_BYTES + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
    }
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int j = 4; j < kTok; j += 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mx[k] = j + 4 + k < kTok ? max3(mx[k], s[j + k], s[j + 4 + k]) : fmaxf(mx[k], s[j + k]);
    }
    const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
    // A row without a key so far takes this tile's maximum (there is nothing to rescale).
    float base = m == kNegInf ? (mt == kNegInf ? 0.f : mt) : m;
    uint32_t pk[SH::CH];
    uint64_t sum[2] = {0ull, 0ull};
    weights<SH>(s, scale2, pair(-base, -base), pk, sum);
    const bool grows = m != kNegInf && mt > m + 8.f;
    if (m == kNegInf) m = mt;
    if (__any_sync(0xffffffffu, grows)) {
      // S of this tile is complete, so the product before it is too: O is stable.
      const float c = grows ? ex2(m - mt) : 1.f;
      l *= c;
      if (grows) base = m = mt;
#pragma unroll 1
      for (int q = 0; q < D / 16; ++q) {      // few columns at a time: S waits in registers
        float o[16];
        tc_ld16(oc + q * 16, o);
        uint32_t x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(o[j] * c);
        tc_st16(oc + q * 16, x);
      }
      sum[0] = sum[1] = 0ull;
      weights<SH>(s, scale2, pair(-base, -base), pk, sum);
    }
#pragma unroll
    for (int c = 0; c < kTok / 2 / SH::CH; ++c) {
      if (c > 0) weights<SH>(s + c * 2 * SH::CH, scale2, pair(-base, -base), pk, sum);
      if constexpr (SH::CH == 32) tc_st32w(sc + c * SH::CH, pk);
      else tc_st16(sc + c * SH::CH, pk);
      if ((c + 1) * SH::CH % 32 != 0) continue;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl->p_half[w][(c + 1) * SH::CH / 32 - 1]));
    }
    float a, b;
    unpair(add2(sum[0], sum[1]), a, b);
    l += a + b;
  }
  const bool any = two_rows || w < n_tiles;
  if (any && !warp_wait(ctl, smem_addr(&ctl->o_full[w]), 0)) return false;
  tc_fence_after();
  return true;
}

// ---------------------------------------------------------------- results
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? kNegInf : (m + __log2f(l)) * 0.6931471805599453f;   // NaN stays NaN
}

// A warp's 32 rows of COLS f32 (lane = row, `at` its row of o_part or -1) to memory by way of
// shared memory: written from the lanes' registers directly, every store would touch 32 lines
// (128 KB a CTA took 7000 cycles).  Rows are padded by 16 bytes against bank conflicts.
template <int D, int COLS>
__device__ __forceinline__ void store_rows(float* o_part, int64_t at, int col, float* scratch, int lane) {
  constexpr int LD = COLS + kPad, PER = COLS / 4;     // lanes that hold one row
  __syncwarp();
#pragma unroll 8
  for (int i = 0; i < 32; i += 32 / PER) {
    const int r = i + lane / PER, c = lane % PER * 4;
    const int64_t to = __shfl_sync(0xffffffffu, at, r);
    const float4 x = *reinterpret_cast<const float4*>(scratch + r * LD + c);
    if (to >= 0) *reinterpret_cast<float4*>(o_part + to * D + col + c) = x;
  }
}

// Two row tiles: a thread's row is row r of stream w.
template <int D>
__device__ void write_rows(const PrefixParams& p, const PrefixTile& t, int g, int split, int w, int r, float m,
                           float l, float vscale, float* ring) {
  const uint32_t oc = ((uint32_t)(r & ~31) << 16) + kOCol + w * D;
  const bool mine = w * kRows + r < t.rows;
  const int64_t at = mine ? prefix_flat_row(p, t, g, w * kRows + r) * p.S + split : 0;
  float* scratch = ring + (size_t)(w * kRows + (r & ~31)) * (D + kPad);
  const float f = vscale / l;
#pragma unroll 1                    // (code that runs once is fetched while it runs: keep it short)
  for (int q = 0; q < D / 32; ++q) {
    float o[32];
    tc_ld32(oc + q * 32, o);
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      *reinterpret_cast<float4*>(scratch + (r & 31) * (D + kPad) + q * 32 + j) =
          make_float4(o[j] * f, o[j + 1] * f, o[j + 2] * f, o[j + 3] * f);
  }
  if (mine) p.lse_part[at] = lse_of(m, l);
  store_rows<D, D>(p.o_part, mine && l != 0.f ? at : -1, 0, scratch, r & 31);
}

// Two streams of the same rows: merge them (M = max m, c = 2^(m - M), O = sum c O / sum c l).
// Both streams' O of a row lie in its TMEM lane: either thread of the row forms half the dims.
template <int D>
__device__ void merge_rows(const PrefixParams& p, const PrefixTile& t, int g, int split, int n_tiles, int half,
                           int r, const float (&m)[2], const float (&l)[2], float vscale, float* ring) {
  constexpr int N = D / 2;
  const uint32_t oc = ((uint32_t)(r & ~31) << 16) + kOCol + half * N;
  const float M = fmaxf(m[0], m[1]);
  float c[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) c[w] = l[w] == 0.f ? 0.f : M == kNegInf ? 1.f : ex2(m[w] - M);
  const float L = l[0] * c[0] + l[1] * c[1], f = vscale / L;
  const bool mine = r < t.rows;
  const int64_t at = mine ? prefix_flat_row(p, t, g, r) * p.S + split : 0;
  float* scratch = ring + (size_t)(half * kRows + (r & ~31)) * (N + kPad);
#pragma unroll 1
  for (int q = 0; q < N / 32; ++q) {
    float o[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = 0.f;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
      if (w >= n_tiles) continue;             // a split of one tile has no second stream
      const float cw = w ? c[1] : c[0];
      float x[32];
      tc_ld32(oc + w * D + q * 32, x);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = cw != 0.f ? fmaf(x[j], cw * f, o[j]) : o[j];
    }
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      *reinterpret_cast<float4*>(scratch + (r & 31) * (N + kPad) + q * 32 + j) =
          make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
  }
  if (mine && half == 0) p.lse_part[at] = lse_of(M, L);
  store_rows<D, N>(p.o_part, mine && L != 0.f ? at : -1, half * N, scratch, r & 31);
}

template <class SH>
__global__ void __launch_bounds__(SH::THREADS, 1)
    fd_prefix_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ PrefixParams p) {
  constexpr int D = SH::D;
  extern __shared__ __align__(1024) uint8_t base[];   // whole swizzle atoms
  Ctl* ctl = reinterpret_cast<Ctl*>(base + SH::CTL_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, g = blockIdx.y;
  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), SH::FP8 ? 4 : 1);   // FP8: the widening warps arrive
      mbar_init(smem_addr(&ctl->empty[s]), 2);
    }
    for (int s = 0; SH::FP8 && s < 4; ++s) {
      mbar_init(smem_addr(&ctl->raw_full[s]), 1);
      mbar_init(smem_addr(&ctl->raw_empty[s]), 4);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&ctl->s_full[w]), 1);
      mbar_init(smem_addr(&ctl->p_half[w][0]), 4);
      mbar_init(smem_addr(&ctl->p_half[w][1]), 4);
      mbar_init(smem_addr(&ctl->o_full[w]), 1);
      mbar_init(smem_addr(&ctl->turn[w]), 1);
    }
    mbar_init(smem_addr(&ctl->mma_done), 2);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tc_alloc(smem_addr(&ctl->tmem), kCols);
    tc_relinquish();
  }
  pdl_wait();
  pdl_trigger();                    // the pass over the rows' own keys runs next to this one
  if (warp == 8) {
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
    PrefixTile t;
    const bool ok = find_tile<2 * kRows>(p, (int)blockIdx.z, t);
    if (ok) split_of<kTok>(p, split, t);
    if (lane == 0) {
      ctl->tile = t;
      ctl->found = ok ? 1 : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool found = ctl->found != 0;
  const PrefixTile t = ctl->tile;
  const int n_tiles = found && t.lo < t.hi ? (int)((t.hi - t.lo + kTok - 1) / kTok) : 0;
  const bool two_rows = t.rows > kRows;
  const int raw_stages = two_rows ? 2 : 4;

  if (n_tiles > 0) {
    // Registers of the warpgroups (softmax twice, producer and issuers, widening twice): 2 x 216
    // + 72 is what three were launched with (168 each), 2 x 168 + 48 + 2 x 48 five (96).
    if (warp >= 12) {
      if constexpr (SH::FP8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        widen<SH>(p, t, n_tiles, raw_stages, base, ctl, (warp - 12) >> 2, tid & 127);
      }
    } else if (warp >= 8) {
      if constexpr (SH::FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp == 8) {
        produce<SH>(p, t, g, n_tiles, raw_stages, two_rows, &tk, &tv, smem_addr(base), ctl, lane);
      } else if (warp < 11) {
        named_bar_sync(2, 320);               // Q is in place
        issue<SH>(p, warp - 9, n_tiles, two_rows, smem_addr(base), ctl);
      }
    } else {
      if constexpr (SH::FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      const int w = warp >> 2, r = tid & 127;
      // A scale of K multiplies the scores (its sign q, since the running maximum is taken
      // before the factor; a factor of 0 becomes one that only keeps -inf what it is).
      const float ks = p.k_scale != nullptr ? p.k_scale[g] : 1.f;
      const float sl2 = SH::FP8 ? fmaxf(p.scale_log2 * fabsf(ks), 1e-37f) : p.scale_log2;
      // Q to shared memory, [64-dim slab][row][128 B] with 16-byte groups XORed by the row.  A
      // warp has 32 rows (16, of a single row tile): each lane finds where one of them starts,
      // then LPR lanes read a whole row, eight loads of a thread in flight.
      {
        constexpr int LPR = D / 8, AT_ONCE = 8;
        const int rows = two_rows ? 32 : 16, row0 = warp * rows, c = lane % LPR;
        const int64_t mine = prefix_q_offset(p, t, g, min(row0 + lane, t.rows - 1));
        const uint4* q = static_cast<const uint4*>(p.q) + c;
        const float f = ks < 0.f ? -1.f : 1.f;
        uint8_t* dst = base + (row0 / kRows) * SH::TILE_BYTES + (c >> 3) * SH::SLAB_BYTES;
#pragma unroll 1
        for (int r0 = lane / LPR; r0 < rows; r0 += AT_ONCE * (32 / LPR)) {
          uint4 x[AT_ONCE];
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) x[k] = q[__shfl_sync(0xffffffffu, mine, r0 + k * (32 / LPR)) >> 3];
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) {
            const int i = r0 + k * (32 / LPR), row = row0 + i;
            if (row >= t.rows) x[k] = make_uint4(0, 0, 0, 0);
            if constexpr (SH::FP8) {          // q as f16
              uint32_t* y = &x[k].x;
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = pack_f16(bf16lo_to_f32(y[e]) * f, bf16hi_to_f32(y[e]) * f);
            }
            if (i < rows) *reinterpret_cast<uint4*>(dst + (row % kRows) * 128 + (((c & 7) ^ (row & 7)) << 4)) = x[k];
          }
        }
      }
      fence_proxy_async_smem();
      named_bar_sync(2, 320);
      float m, l;
      if (!softmax<SH>(p, t, n_tiles, two_rows, w, r, sl2, base, ctl, m, l) && lane == 0) set_abort(p, ctl);
      named_bar_sync(1, 256);                 // both streams are done, or one gave up
      float2* stats = reinterpret_cast<float2*>(base);        // Q is not needed any more
      stats[w * kRows + r] = make_float2(m, l);
      named_bar_sync(1, 256);
      // Read again rather than kept through the loop, whose registers are all in use.
      const PrefixTile done = ctl->tile;
      const float vs = p.v_scale != nullptr ? p.v_scale[g] : 1.f;
      float* scratch = reinterpret_cast<float*>(base + SH::RING_OFF);
      if (aborted(ctl)) {
        const int row = done.rows > kRows ? w * kRows + r : r;
        if (row < done.rows && (done.rows > kRows || w == 0))
          p.lse_part[prefix_flat_row(p, done, g, row) * p.S + split] = kNegInf;
      } else if (done.rows > kRows) {
        write_rows<D>(p, done, g, split, w, r, m, l, vs, scratch);
      } else {
        const float2 a = stats[r], b = stats[kRows + r];
        const float ms[2] = {a.x, b.x}, ls[2] = {a.y, b.y};
        merge_rows<D>(p, done, g, split, n_tiles, w, r, ms, ls, vs, scratch);
      }
    }
  } else if (found) {               // nothing of the prompt in this split
    if (tid < t.rows) p.lse_part[prefix_flat_row(p, t, g, tid) * p.S + split] = kNegInf;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tc_dealloc(ctl->tmem, kCols);
  }
}

template <class SH>
cudaError_t launch(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  auto kernel = fd_prefix_tc_kernel<SH>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.apply(kernel, (int)smem_bytes<SH>());
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.S, (unsigned)p.Hkv,
                  (unsigned)prefix_row_tiles(p.B, (int64_t)p.Q * p.G, p.group_start != nullptr, p.P, 2 * kRows));
  return launch_pdl(kernel, grid, SH::THREADS, smem_bytes<SH>(), stream, tk, tv, p);
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixParams& p, bool fp8, int d, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t stream) {
  if (fp8) return launch<Shape<128, true>>(p, tk, tv, stream);
  return d == 128 ? launch<Shape<128, false>>(p, tk, tv, stream) : launch<Shape<64, false>>(p, tk, tv, stream);
}

// Tokens and 128-byte lines of this kernel's TMA boxes.
void prefix_tc_box(int page_size, uint32_t* tokens, uint32_t* lines) {
  const bool small = page_size > 0 && page_size < kTok;
  *tokens = small ? (uint32_t)page_size : (uint32_t)kTok;
  *lines = small ? 1u : 0u;
}

}  // namespace fd
