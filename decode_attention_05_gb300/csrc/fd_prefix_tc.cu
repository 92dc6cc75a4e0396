// fd_prefix_tc.cu -- attention of many query rows over a shared prompt on the 5th-generation
// tensor cores (fd_prefix.cuh says what the pass computes): bf16 q; bf16 caches with d 64 or
// 128, or FP8 E4M3 caches with d = 128.
//
// A CTA serves one kv head, one split of one prompt and up to 256 query rows of its group, as
// two streams of 128 rows, one per softmax warpgroup:
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
// One thread issues all products: P V of a stream's tile, then at once Q K^T of its next tile
// (in order behind the read of P, whose columns it overwrites), then the other stream's.  So
// the tensor cores work on one stream while the other's warps do their softmax.  O is rescaled
// only when a tile's maximum exceeds m by more than 8 (base 2): weights then reach at most 2^8,
// and l and O use the same m, so the result is the same.
//
// Bound: with 256 rows a CTA does 2 x 4 x 128 x 128 x d flops on a tile of 512 d bytes of K
// and V: the tensor cores (2048 cycles a tile at d = 128) and the SM's share of HBM bandwidth
// (about 24 bytes a cycle: 2700 cycles) are near balance; several row tiles read a prompt's
// tiles from L2.
//
// Warps: 0-3 and 4-7 the softmax of stream 0 and 1, 8 the TMA producer, 9 the issuer.  Tensor
// memory: S_0, S_1 (128 columns each, P over their first halves), O_0, O_1 (d each).  Shared
// memory: Q (2 x 128 rows), then a ring of K and V tiles (32 KB at d = 128, 5 of them), each
// [64-dim slab][token][128 B], 128-byte swizzle.  A page of fewer than 128 tokens is loaded
// slab by slab, so that a tile has the same layout whatever the page size.
//
// FP8 caches: TMA fills a ring of code tiles (16 KB), and a fourth warpgroup widens them to
// f16 (exactly: E4M3 fits f16) into the operand ring, so the products are those of f16 q, K, P
// and V.  (8-bit products would need q and P in 8 bits.)  A kv head's scale of K multiplies
// the scores, its scale of V the output.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fd_prefix.cuh"
#include "fd_tcgen05.cuh"

namespace fd {
namespace {

constexpr int kRows = 128, kTok = 128;
constexpr uint32_t kCols = 512, kOCol = 256;
constexpr int kMaxStages = 8;

template <int D_, bool FP8_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool FP8 = FP8_;
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr uint32_t TYPE = FP8 ? 0u : 1u;               // operands f16 or bf16
  static constexpr int SLABS = D / 64;
  static constexpr uint32_t SLAB_BYTES = kTok * 128;            // 64 dims of 128 tokens
  static constexpr uint32_t TILE_BYTES = SLABS * SLAB_BYTES;
  static constexpr int STAGES = FP8 ? 4 : D == 128 ? 5 : 8;
  static constexpr uint32_t RING_OFF = 2 * TILE_BYTES;          // behind Q
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
  uint64_t mma_done;                              // all products of the CTA are complete
  uint32_t bad[8];                                // tile n mod 8: bit j = its page j is invalid
  int32_t abort, found;
  uint32_t tmem;
  PrefixTile tile;
};

template <class SH>
constexpr size_t smem_bytes() {
  return 1024 + SH::CTL_OFF + sizeof(Ctl);
}
static_assert(smem_bytes<Shape<128, false>>() <= 227 * 1024 && smem_bytes<Shape<64, false>>() <= 227 * 1024 &&
                  smem_bytes<Shape<128, true>>() <= 227 * 1024,
              "one CTA per SM");

__device__ __forceinline__ bool aborted(Ctl* c) {
  return *reinterpret_cast<volatile int32_t*>(&c->abort) != 0;
}
__device__ __forceinline__ void set_abort(const PrefixParams& p, Ctl* c) {
  *reinterpret_cast<volatile int32_t*>(&c->abort) = 1;
  atomicOr(p.flags, kDevFlagTimeout);
}
// A bounded wait that also gives up once another role has.
__device__ __forceinline__ bool wait_or_abort(Ctl* c, uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_probe(bar, parity, 200u)) {
    if (aborted(c) || global_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}
// The same for a warp whose lanes have to agree.
__device__ __forceinline__ bool warp_wait(Ctl* c, uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_or_abort(c, bar, parity));
}

// 128 columns of this thread's lane.
__device__ __forceinline__ void ld128(uint32_t taddr, float* v) {
  tc_ld32x2(taddr, taddr + 32, v);
  tc_ld32x2(taddr + 64, taddr + 96, v + 64);
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
__device__ __forceinline__ void store8(float* a, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// ---------------------------------------------------------------- TMA producer (one warp)
// Ring entry 2 n is the K tile n of the split, 2 n + 1 its V tile.  bf16 tiles go to the
// operand ring, codes to the raw one.
template <class SH>
__device__ void produce(const PrefixParams& p, const PrefixTile& t, int g, int n_tiles, int raw_stages,
                        const CUtensorMap* tk, const CUtensorMap* tv, uint32_t base, Ctl* ctl, int lane) {
  const uint64_t pol = policy_evict_first();
  const bool paged = p.table != nullptr;
  const int ps = p.page_size;
  const int boxes = paged && ps < kTok ? kTok / ps : 1;      // pages of a tile
  const int64_t used = paged ? (t.L + ps - 1) >> p.log2_page : 0;
  const int stages = SH::FP8 ? raw_stages : SH::STAGES;
  uint64_t* fulls = SH::FP8 ? ctl->raw_full : ctl->full;
  uint64_t* empties = SH::FP8 ? ctl->raw_empty : ctl->empty;
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
      if (round > 0) ok = warp_wait(ctl, smem_addr(&empties[st]), (round - 1) & 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(full, SH::FP8 ? SH::RAW_BYTES : SH::TILE_BYTES);
      __syncwarp();
      const uint32_t dst = base + (SH::FP8 ? SH::raw_offset(st) : SH::RING_OFF + st * SH::TILE_BYTES);
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
  if (!ok) {                        // let the copies in flight land before the CTA ends
    if (lane == 0) set_abort(p, ctl);
    for (int i = max(0, issued - stages); i < issued; ++i)
      mbar_wait(smem_addr(&fulls[i % stages]), (i / stages) & 1);
  }
}

// ---------------------------------------------------------------- widening (FP8, a warpgroup)
// Thread r widens token row r of every tile: 16 codes of one 16-byte group become two groups
// of f16.  A quarter warp's eight rows hit eight different bank groups in both layouts.  Rows
// of tokens without weight become zeros.
template <class SH>
__device__ void widen(const PrefixParams& p, const PrefixTile& t, int n_tiles, int raw_stages, uint8_t* base,
                      Ctl* ctl, int r) {
  const int lane = r & 31;
  const bool pages = p.table != nullptr && p.page_size < kTok;
  bool ok = true;
  int rs = 0, round = 0;
  for (int e = 0; e < 2 * n_tiles; ++e) {
    const int n = e >> 1, st = e % SH::STAGES;
    ok = warp_wait(ctl, smem_addr(&ctl->raw_full[rs]), round & 1);
    if (ok && e >= SH::STAGES) ok = warp_wait(ctl, smem_addr(&ctl->empty[st]), ((e / SH::STAGES) - 1) & 1);
    if (!ok) break;
    const int64_t tok = t.lo + (int64_t)n * kTok + r;
    const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[n & 7]);
    const bool live = tok < t.hi && !((bad >> (pages ? r >> p.log2_page : 0)) & 1u);
    const uint8_t* src = base + SH::raw_offset(rs) + r * 128;
    uint8_t* dst = base + SH::RING_OFF + st * SH::TILE_BYTES + r * 128;
#pragma unroll
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
    if (++rs == raw_stages) rs = 0, ++round;
  }
  if (!ok && lane == 0) set_abort(p, ctl);
}

// ---------------------------------------------------------------- product issuer (one thread)
template <class SH>
__device__ void issue(const PrefixParams& p, int n_tiles, bool two_rows, uint32_t qbase,
                      uint32_t ring, Ctl* ctl, uint32_t tmem) {
  constexpr int D = SH::D;
  constexpr uint32_t id_s = instr_desc(kRows, kTok, 0, SH::TYPE), id_o = instr_desc(kRows, D, 1, SH::TYPE);
  const int step = two_rows ? 1 : 2;          // a stream's next tile
  auto tile_at = [&](int e) { return ring + (uint32_t)(e % SH::STAGES) * SH::TILE_BYTES; };
  auto landed = [&](int e) {
    return wait_or_abort(ctl, smem_addr(&ctl->full[e % SH::STAGES]), (e / SH::STAGES) & 1);
  };
  auto release = [&](int e) { tc_commit(smem_addr(&ctl->empty[e % SH::STAGES])); };
  auto scores = [&](int w, int n) {
    const uint32_t q = qbase + (two_rows ? w * SH::TILE_BYTES : 0u), k = tile_at(2 * n);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t off = (ks >> 2) * SH::SLAB_BYTES + (ks & 3) * 32u;
      tc_mma_ss(tmem + w * kTok, smem_desc(q + off, 0, 1024), smem_desc(k + off, 0, 1024), id_s, ks > 0);
    }
    tc_commit(smem_addr(&ctl->s_full[w]));
  };
  bool ok = true;
  for (int w = 0; w < 2 && ok; ++w) {         // the streams' first scores
    const int n = two_rows ? 0 : w;
    if (n >= n_tiles) break;
    ok = landed(2 * n);
    if (!ok) break;
    scores(w, n);
    if (!two_rows || w == 1) release(2 * n);
  }
  for (int n = 0; n < n_tiles && ok; ++n) {
    ok = landed(2 * n + 1);
    const int next = n + step, i = two_rows ? n : n >> 1;
    for (int w = two_rows ? 0 : n & 1; w < 2 && ok; ++w) {
      const uint32_t v = tile_at(2 * n + 1);
#pragma unroll
      for (int ks = 0; ks < kTok / 16; ++ks) {
        if (ks % 4 == 0) {
          ok = wait_or_abort(ctl, smem_addr(&ctl->p_half[w][ks / 4]), i & 1);
          if (!ok) break;
          tc_fence_after();
        }
        tc_mma_ts(tmem + kOCol + w * D, tmem + w * kTok + ks * 8,
                  smem_desc(v + ks * 2048u, SH::SLAB_BYTES, 1024), id_o, (i > 0 || ks > 0) ? 1u : 0u);
      }
      if (!ok) break;
      const bool last_use = !two_rows || w == 1;
      if (last_use) release(2 * n + 1);
      if (next < n_tiles) {
        if (!two_rows || w == 0) ok = landed(2 * next);
        if (!ok) break;
        scores(w, next);
        if (last_use) release(2 * next);
      } else {
        tc_commit(smem_addr(&ctl->o_full[w]));
      }
      if (!two_rows) break;
    }
  }
  if (!ok) set_abort(p, ctl);
  tc_commit(smem_addr(&ctl->mma_done));       // never leave with products in flight
  if (!mbar_wait(smem_addr(&ctl->mma_done), 0)) atomicOr(p.flags, kDevFlagTimeout);
}

// ---------------------------------------------------------------- softmax (a warpgroup)
// Stream w, lane row r.  False if a wait gave up.
template <class SH>
__device__ bool softmax(const PrefixParams& p, const PrefixTile& t, int n_tiles, bool two_rows,
                        int w, int r, float sl2, uint8_t* ring, Ctl* ctl, uint32_t tmem, float& m,
                        float& l) {
  constexpr int D = SH::D;
  const int lane = r & 31;
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t sc = tmem + lanes + w * kTok, oc = tmem + lanes + kOCol + w * D;
  const int log2_page = p.log2_page;
  const bool pages = p.table != nullptr && p.page_size < kTok;
  const int step = two_rows ? 1 : 2;
  m = kNegInf;
  l = 0.f;
  for (int n = two_rows ? 0 : w, i = 0; n < n_tiles; n += step, ++i) {
    if (!warp_wait(ctl, smem_addr(&ctl->s_full[w]), i & 1)) return false;
    tc_fence_after();
    float s[kTok];
    ld128(sc, s);
    const int64_t t0 = t.lo + (int64_t)n * kTok;
    const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[n & 7]);
    const bool clean = t0 + kTok <= t.hi && bad == 0u;
    if (!clean) {                   // past the prompt's end, or on an invalid page: no weight
      const int live = (int)min((int64_t)kTok, t.hi - t0);
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const bool out = j >= live || ((bad >> (pages ? j >> log2_page : 0)) & 1u);
        s[j] = out ? kNegInf : s[j];
      }
      if constexpr (!SH::FP8) {     // (widen() has cleared them)
        // Their V rows may hold anything, and 0 * NaN would reach O: clear them.
        const int e = 2 * n + 1;
        if (!warp_wait(ctl, smem_addr(&ctl->full[e % SH::STAGES]), (e / SH::STAGES) & 1)) return false;
        if (r >= live || ((bad >> (pages ? r >> log2_page : 0)) & 1u)) {
          uint8_t* v = ring + (size_t)(e % SH::STAGES) * SH::TILE_BYTES + r * 128;
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
    const float mn = fmaxf(m, mt);
    const bool resc = i > 0 && m != kNegInf && mn > m + 8.f;
    const float mu = (m == kNegInf || resc) ? mn : m;
    if (__any_sync(0xffffffffu, resc)) {
      // S of this tile is complete, so the product before it is too: O is stable.
      const float c = resc ? ex2(m - mn) : 1.f;
      l *= c;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        tc_ld32(oc + q * 32, o);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] *= c;
        tc_st32(oc + q * 32, o);
      }
    }
    m = mu;
    const float base = mu == kNegInf ? 0.f : mu;
    const uint64_t scale2 = pair(sl2, sl2), off2 = pair(-base, -base);
    uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t pk[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int k = half * 64 + 2 * j;
        float a, b;
        unpair(fma2(pair(s[k], s[k + 1]), scale2, off2), a, b);
        a = ex2(a);
        b = ex2(b);
        sum[j & 3] = add2(sum[j & 3], pair(a, b));
        pk[j] = SH::FP8 ? pack_f16(a, b) : pack_bf16(a, b);
      }
      tc_st32w(sc + half * 32, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl->p_half[w][half]));
    }
    float a, b;
    unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
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

// Two row tiles: a thread writes its row.
template <int D>
__device__ void write_rows(const PrefixParams& p, const PrefixTile& t, int g, int split, int w,
                           int r, float m, float l, float vscale, uint32_t tmem) {
  const uint32_t oc = tmem + ((uint32_t)(r & ~31) << 16) + kOCol + w * D;
  const bool mine = w * kRows + r < t.rows;
  const int64_t at = mine ? prefix_flat_row(p, t, g, w * kRows + r) * p.S + split : 0;
  const float f = vscale / l;
#pragma unroll
  for (int q = 0; q < D / 32; ++q) {
    float o[32];
    __syncwarp();
    tc_ld32(oc + q * 32, o);
    if (mine && l != 0.f) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] *= f;
#pragma unroll
      for (int j = 0; j < 32; j += 8) store8(p.o_part + at * D + q * 32 + j, o + j);
    }
  }
  if (mine) p.lse_part[at] = lse_of(m, l);
}

// Two streams of the same rows: merge them (M = max m, c = 2^(m - M), O = sum c O / sum c l).
// Warpgroup w forms dims w d/2 .. of every row: each hands the other half of its own O over
// in the drained ring, rows padded to 16-byte groups that fall into different banks.
template <int D>
__device__ void merge_rows(const PrefixParams& p, const PrefixTile& t, int g, int split, int n_tiles,
                           int w, int r, float m, float l, float vscale, uint8_t* ring, Ctl* ctl,
                           uint32_t tmem) {
  constexpr int HALF = D / 2, LD = HALF + 4;
  const uint32_t oc = tmem + ((uint32_t)(r & ~31) << 16) + kOCol + w * D;
  float2* stats = reinterpret_cast<float2*>(ring + 2 * kRows * LD * sizeof(float));
  stats[w * kRows + r] = make_float2(m, l);
  named_bar_sync(1, 256);
  const float m0 = stats[r].x, m1 = stats[kRows + r].x, M = fmaxf(m0, m1);
  const float l0 = stats[r].y, l1 = stats[kRows + r].y;
  const float c0 = l0 == 0.f ? 0.f : M == kNegInf ? 1.f : ex2(m0 - M);
  const float c1 = l1 == 0.f ? 0.f : M == kNegInf ? 1.f : ex2(m1 - M);
  const float L = l0 * c0 + l1 * c1;
  const float c = w ? c1 : c0;
  const bool has = w < n_tiles;               // a split of one tile has no second stream
  float* theirs = reinterpret_cast<float*>(ring) + (size_t)((w ^ 1) * kRows + r) * LD;
  const float* given = reinterpret_cast<const float*>(ring) + (size_t)(w * kRows + r) * LD;
#pragma unroll
  for (int q = 0; q < HALF / 32; ++q) {
    float o[32];
    if (has) tc_ld32(oc + (w ^ 1) * HALF + q * 32, o);
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = has && c != 0.f ? o[j] * c : 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      *reinterpret_cast<float4*>(theirs + q * 32 + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
  }
  named_bar_sync(1, 256);
  const bool mine = r < t.rows;
  const int64_t at = mine ? prefix_flat_row(p, t, g, r) * p.S + split : 0;
  const float f = vscale / L;
#pragma unroll
  for (int q = 0; q < HALF / 32; ++q) {
    float o[32];
    __syncwarp();
    if (has) tc_ld32(oc + w * HALF + q * 32, o);
    if (mine && L != 0.f) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 x = *reinterpret_cast<const float4*>(given + q * 32 + j);
        o[j] = ((has && c != 0.f ? o[j] * c : 0.f) + x.x) * f;
        o[j + 1] = ((has && c != 0.f ? o[j + 1] * c : 0.f) + x.y) * f;
        o[j + 2] = ((has && c != 0.f ? o[j + 2] * c : 0.f) + x.z) * f;
        o[j + 3] = ((has && c != 0.f ? o[j + 3] * c : 0.f) + x.w) * f;
      }
#pragma unroll
      for (int j = 0; j < 32; j += 8) store8(p.o_part + at * D + w * HALF + q * 32 + j, o + j);
    }
  }
  if (mine && w == 0) p.lse_part[at] = lse_of(M, L);
}

template <class SH>
__global__ void __launch_bounds__(SH::THREADS, 1)
    fd_prefix_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ PrefixParams p) {
  constexpr int D = SH::D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = base + SH::RING_OFF;
  Ctl* ctl = reinterpret_cast<Ctl*>(base + SH::CTL_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, g = blockIdx.y;
  if (tid == 0) {
    for (int s = 0; s < SH::STAGES; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), SH::FP8 ? 4 : 1);   // FP8: the widening warps arrive
      mbar_init(smem_addr(&ctl->empty[s]), 1);
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
    }
    mbar_init(smem_addr(&ctl->mma_done), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tc_alloc(smem_addr(&ctl->tmem), kCols);
    tc_relinquish();
  }
  pdl_wait();
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
  const uint32_t tmem = ctl->tmem;
  const bool found = ctl->found != 0;
  const PrefixTile t = ctl->tile;
  const int n_tiles = found && t.lo < t.hi ? (int)((t.hi - t.lo + kTok - 1) / kTok) : 0;
  const bool two_rows = t.rows > kRows;
  const int raw_stages = two_rows ? 2 : 4;

  if (n_tiles > 0) {
    // Registers of the warpgroups (softmax, softmax, producer and issuer, widening): 216 +
    // 216 + 72 is what three were launched with (168 each), 184 + 184 + 56 + 88 four (128).
    if (warp >= 12) {
      if constexpr (SH::FP8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        widen<SH>(p, t, n_tiles, raw_stages, base, ctl, tid & 127);
      }
    } else if (warp >= 8) {
      if constexpr (SH::FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp == 8) {
        produce<SH>(p, t, g, n_tiles, raw_stages, &tk, &tv, smem_addr(base), ctl, lane);
      } else if (warp == 9) {
        named_bar_sync(2, 288);               // Q is in place
        if (lane == 0) issue<SH>(p, n_tiles, two_rows, smem_addr(base), smem_addr(ring), ctl, tmem);
        __syncwarp();
      }
    } else {
      if constexpr (SH::FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
      else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      const int w = warp >> 2, r = tid & 127;
      // A scale of K multiplies the scores (its sign q, since the running maximum is taken
      // before the factor; a factor of 0 becomes one that only keeps -inf what it is).
      const float ks = p.k_scale != nullptr ? p.k_scale[g] : 1.f;
      const float vs = p.v_scale != nullptr ? p.v_scale[g] : 1.f;
      const float sl2 = SH::FP8 ? fmaxf(p.scale_log2 * fabsf(ks), 1e-37f) : p.scale_log2;
      // Q to shared memory, [64-dim slab][row][128 B] with 16-byte groups XORed by the row.
      // Two row tiles: a thread its row; one: the two threads of a row half of it each.
      {
        const int row = two_rows ? w * kRows + r : r;
        const bool live = row < t.rows;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                          (live ? prefix_q_offset(p, t, g, row) : 0));
        uint8_t* dst = base + (two_rows ? w * SH::TILE_BYTES : 0u) + r * 128;
        const int c0 = two_rows ? 0 : w * (D / 16), c1 = two_rows ? D / 8 : c0 + D / 16;
#pragma unroll 4
        for (int c = c0; c < c1; ++c) {
          uint4 x = live ? src[c] : make_uint4(0, 0, 0, 0);
          if constexpr (SH::FP8) {            // q as f16
            uint32_t* y = &x.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float f = ks < 0.f ? -1.f : 1.f;
              y[i] = pack_f16(bf16lo_to_f32(y[i]) * f, bf16hi_to_f32(y[i]) * f);
            }
          }
          *reinterpret_cast<uint4*>(dst + (c >> 3) * SH::SLAB_BYTES + (((c & 7) ^ (r & 7)) << 4)) = x;
        }
      }
      fence_proxy_async_smem();
      named_bar_sync(2, 288);
      float m, l;
      if (!softmax<SH>(p, t, n_tiles, two_rows, w, r, sl2, ring, ctl, tmem, m, l) && lane == 0)
        set_abort(p, ctl);
      named_bar_sync(1, 256);                 // both streams are done, or one gave up
      if (aborted(ctl)) {
        const int row = two_rows ? w * kRows + r : r;
        if (row < t.rows && (two_rows || w == 0))
          p.lse_part[prefix_flat_row(p, t, g, row) * p.S + split] = kNegInf;
      } else if (two_rows) {
        write_rows<D>(p, t, g, split, w, r, m, l, vs, tmem);
      } else {
        merge_rows<D>(p, t, g, split, n_tiles, w, r, m, l, vs, ring, ctl, tmem);
      }
    }
  } else if (found) {               // nothing of the prompt in this split
    if (tid < t.rows) p.lse_part[prefix_flat_row(p, t, g, tid) * p.S + split] = kNegInf;
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == 9) {
    tc_fence_after();
    tc_dealloc(tmem, kCols);
  }
}

template <class SH>
cudaError_t launch(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  auto kernel = fd_prefix_tc_kernel<SH>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.apply(kernel, (int)smem_bytes<SH>());
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.S, (unsigned)p.Hkv,
                  (unsigned)prefix_row_tiles(p.B, (int64_t)p.Q * p.G, p.group_start ? p.P : 1, 2 * kRows));
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
