// fd_append.cu -- writing the KV cache: the keys and values of new tokens go to their
// cache slots, keys and queries rotated by their positions on the way (fd_append_kv).
//
// A rotation of position p turns each pair (x_a, x_b) of a head's first `rot` dims by the
// angle theta_i(p):  (x_a c - x_b s,  x_b c + x_a s),  c = cos theta_i(p), s = sin theta_i(p),
// with c and s read from the caller's table ("AI Infra: math and infra optimisation in large
// models", appendix: a precomputed [max_pos, rotary_dim] cos/sin table instead of SFU
// trigonometry) and pairs (i, i + rot/2) or (2i, 2i + 1).  Computed in f32 and rounded once
// to the destination's type; an FP8 code is the E4M3 rounding of x / scale, saturating.
//
// Bound: memory.  A token costs its q, k and v read once, q_out and the two cache slots
// written once, and its table row; the arithmetic is 3 flops per element.  8191 tokens of 64
// + 8 + 8 heads (d = 128, bf16): 54.7 us, 6.2 TB/s of reads and writes; 32768 tokens into an
// FP8 cache: 214 us, 6.0 TB/s.  A decode step of 16 rows takes 2.3 us in a graph, the launch.
//
// Layout: a thread owns 16 elements of one head row, as two groups of 8 that hold whole
// pairs (for half-split pairs the groups lie rot/2 apart), so a rotation needs no exchange
// between threads and q may be rotated in place.  d / 16 threads cover a row, a warp 4
// (d = 128) or 8 (d = 64) rows of one token; all its loads of q, k and v are issued before
// the token's place in the cache is known (row search, length, block table: a chain of
// dependent loads), and the token's cos / sin stay in registers over a warp's rows.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <cstring>

#include "fd_device.cuh"

namespace fd {
namespace {

struct AppendParams {
  const void *q, *k, *v;          // q may be nullptr
  void* q_out;
  uint8_t *k_cache, *v_cache;
  // element strides: of a token's batch row and of a token inside it (4-D inputs), of a head
  int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh, qo_sb, qo_st, qo_sh;
  int64_t kc_sb, kc_sh, kc_st, vc_sb, vc_sh, vc_st;   // caches: page (or row), head, token
  int32_t T, Q, B;                // tokens in all; tokens per row where cu_tokens is null
  int32_t Hq, Hkv;
  int32_t rot;                    // rotated dims (0: none), a multiple of 16
  int32_t interleaved;
  const int32_t* cu_tokens;       // [B + 1] or nullptr
  const int32_t* seq_lens;        // [B], lengths after the append
  const int32_t* pos_offset;      // [B] or nullptr
  const float* cos_sin;           // [max_pos, rot]: cos of the rot/2 pairs, then sin
  int64_t cs_stride, max_pos;
  const int32_t* block_table;     // or nullptr
  int64_t bt_sb;
  int32_t page_size, log2_page;
  int64_t num_pages, L_cap;
  const float *k_scale, *v_scale; // FP8: per kv head, nullptr = 1
  uint32_t* flags;                // or nullptr
};

__device__ __forceinline__ void flag(const AppendParams& p, uint32_t f) {
  if (p.flags != nullptr) atomicOr(p.flags, f);
}

// Eight consecutive elements as they lie in memory (half the registers of f32 for bf16, which
// is what decides how many loads an SM has in flight), and widened to f32.
template <class T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* a) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(a) + i);
  }
  __device__ __forceinline__ void widen(float* x) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
          x[2 * j] = bf16lo_to_f32(w[j]);
          x[2 * j + 1] = bf16hi_to_f32(w[j]);
        } else {
          x[4 * i + j] = __uint_as_float(w[j]);
        }
      }
    }
  }
};
__device__ __forceinline__ void load8(const float* a, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 r = reinterpret_cast<const float4*>(a)[i];
    x[4 * i] = r.x, x[4 * i + 1] = r.y, x[4 * i + 2] = r.z, x[4 * i + 3] = r.w;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* a, const float* x, float) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(a) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* a, const float* x, float) {
  reinterpret_cast<float4*>(a)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(a)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// E4M3 codes of x / scale: a true division, so that a code is the rounding of the quotient
// (a reciprocal's own rounding would move values that sit near a border between codes).
// A quotient past 448 takes the largest code; NaN stays NaN.
__device__ __forceinline__ void store8(__nv_fp8_e4m3* a, const float* x, float scale) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)), __NV_SATFINITE,
        __NV_E4M3);
    w[i >> 1] |= (uint32_t)c << (16 * (i & 1));
  }
  *reinterpret_cast<uint2*>(a) = make_uint2(w[0], w[1]);
}

// The batch row of token t: the number of rows that end at or before it (cu_tokens is
// non-decreasing), by a search that cuts the range 32-fold a step, one probe per lane.
__device__ __forceinline__ int row_of_token(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B;                          // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + (lane + 1) * step;    // rows lo .. at - 1 end at or before t?
    const bool past = at <= lo + n && cu[at] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, past));
    lo += k * step;
    n = min(step - 1, n - k * step);
  }
  return lo;
}

constexpr int kAppendThreads = 128;

// TI: q, k, v and q_out; TC: the caches.  A warp takes ITER x 32 / (D / 16) head rows
// of one token; rows are numbered q heads first, then k, then v.
template <class TI, class TC, int D, int ITER>
__global__ void __launch_bounds__(kAppendThreads, ITER == 1 ? 9 : sizeof(TI) == 2 ? 6 : 4) fd_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int TPR = D / 16;                 // threads per head row
  constexpr int RPW = 32 / TPR;               // rows of a warp at once
  pdl_trigger();
  pdl_wait();                                 // q, k, v and the cache's earlier readers are done
  const int lane = threadIdx.x & 31, unit = lane % TPR;
  const int n_rows = (p.q != nullptr ? p.Hq : 0) + 2 * p.Hkv;
  const int groups = (n_rows + ITER * RPW - 1) / (ITER * RPW);
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int64_t t64 = w / groups;
  if (t64 >= p.T) return;                     // whole warps only
  const int t = (int)t64;
  const int r0 = (int)(w - t64 * groups) * ITER * RPW + lane / TPR;
  const int kbase = p.q != nullptr ? p.Hq : 0, vbase = kbase + p.Hkv;

  // Where the unit's two groups of eight start inside a row.
  const bool turned = unit * 16 < p.rot;
  const bool split = turned && !p.interleaved;
  const int e0 = split ? unit * 8 : unit * 16;
  const int e1 = split ? e0 + p.rot / 2 : e0 + 8;

  // The inputs, before anything is known of the token's place.
  const int tb = p.cu_tokens == nullptr ? t / p.Q : 0;         // batch row of a 4-D input
  const int tj = p.cu_tokens == nullptr ? t - tb * p.Q : t;
  Raw8<TI> x0[ITER], x1[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int r = r0 + i * RPW;
    if (r >= n_rows) continue;
    const TI* src;
    if (r < kbase) {
      src = static_cast<const TI*>(p.q) + tb * p.q_sb + tj * p.q_st + (int64_t)r * p.q_sh;
    } else if (r < vbase) {
      src = static_cast<const TI*>(p.k) + tb * p.k_sb + tj * p.k_st + (int64_t)(r - kbase) * p.k_sh;
    } else {
      src = static_cast<const TI*>(p.v) + tb * p.v_sb + tj * p.v_st + (int64_t)(r - vbase) * p.v_sh;
    }
    // v rows are stored as they are: their groups need not follow the pairs, but a common
    // layout keeps the warp in step.
    x0[i].load(src + e0);
    x1[i].load(src + e1);
  }

  // The token's row, position and slot.
  int b = tb;
  int64_t begin = (int64_t)tb * p.Q, end = begin + p.Q;
  if (p.cu_tokens != nullptr) {
    b = row_of_token(p.cu_tokens, p.B, t, lane);
    if (b >= p.B) return;                     // behind the last row's tokens
    begin = p.cu_tokens[b];
    end = p.cu_tokens[b + 1];
    if (begin < 0 || t < begin || t >= end) { // offsets out of order, or not starting at 0
      if (lane == 0) flag(p, FD_DEVFLAG_OFFSETS);
      return;
    }
  }
  const int64_t L = p.seq_lens[b];
  if (L < 0 || L > p.L_cap) {
    if (lane == 0) flag(p, FD_DEVFLAG_SEQ_LEN);
    return;
  }
  const int64_t pos = L - end + t;
  if (pos < 0) return;                        // a row shorter than its new tokens: padding
  int64_t rp = pos;
  if (p.rot > 0) {
    if (p.pos_offset != nullptr) rp += p.pos_offset[b];
    if (rp < 0 || rp >= p.max_pos) {
      if (lane == 0) flag(p, FD_DEVFLAG_POSITION);
      return;
    }
  }
  int64_t place = b, slot = pos;
  if (p.block_table != nullptr) {
    place = p.block_table[(int64_t)b * p.bt_sb + (pos >> p.log2_page)];
    slot = pos & (p.page_size - 1);
    if (place < 0 || place >= p.num_pages) {
      if (lane == 0) flag(p, FD_DEVFLAG_PAGE);
      return;
    }
  }
  float c[8], s[8];
  if (turned) {
    const float* cs = p.cos_sin + rp * p.cs_stride + unit * 8;
    load8(cs, c);
    load8(cs + p.rot / 2, s);
  }

#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int r = r0 + i * RPW;
    if (r >= n_rows) continue;
    float a[8], h[8];
    x0[i].widen(a);
    x1[i].widen(h);
    if (turned && r < vbase) {
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u0 = a[2 * j], u1 = a[2 * j + 1];
          a[2 * j] = u0 * c[j] - u1 * s[j];
          a[2 * j + 1] = u1 * c[j] + u0 * s[j];
          const float v0 = h[2 * j], v1 = h[2 * j + 1];
          h[2 * j] = v0 * c[4 + j] - v1 * s[4 + j];
          h[2 * j + 1] = v1 * c[4 + j] + v0 * s[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u0 = a[j], u1 = h[j];
          a[j] = u0 * c[j] - u1 * s[j];
          h[j] = u1 * c[j] + u0 * s[j];
        }
      }
    }
    if (r < kbase) {
      TI* dst = static_cast<TI*>(p.q_out) + tb * p.qo_sb + tj * p.qo_st + (int64_t)r * p.qo_sh;
      store8(dst + e0, a, 1.f);
      store8(dst + e1, h, 1.f);
    } else {
      const bool key = r < vbase;
      const int g = r - (key ? kbase : vbase);
      const float* scales = key ? p.k_scale : p.v_scale;
      const float scale = scales != nullptr ? scales[g] : 1.f;
      TC* dst = reinterpret_cast<TC*>(key ? p.k_cache : p.v_cache) +
                (key ? place * p.kc_sb + g * p.kc_sh + slot * p.kc_st
                     : place * p.vc_sb + g * p.vc_sh + slot * p.vc_st);
      store8(dst + e0, a, scale);
      store8(dst + e1, h, scale);
    }
  }
}

template <class TI, class TC, int D>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16), WARPS = kAppendThreads / 32;
  const int n_rows = (p.q != nullptr ? p.Hq : 0) + 2 * p.Hkv;
  // One row group per warp while the warps fit the GPU at once (a decode step: latency; 256
  // rows of 32 + 8 + 8 heads 3.8 us).  Beyond, four: a warp then has four times the loads in
  // flight and looks its token up once for all of them.
  const int64_t warps1 = (int64_t)p.T * ((n_rows + RPW - 1) / RPW);
  const bool many = warps1 > (int64_t)sm_count() * 64;
  const int64_t warps = many ? (int64_t)p.T * ((n_rows + 4 * RPW - 1) / (4 * RPW)) : warps1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + WARPS - 1) / WARPS));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, fd_append_kernel<TI, TC, D, 4>, p)
              : cudaLaunchKernelEx(&cfg, fd_append_kernel<TI, TC, D, 1>, p);
}

template <class T>
cudaError_t launch_d(int d, const AppendParams& p, cudaStream_t stream) {
  return d == 128 ? launch<T, T, 128>(p, stream) : launch<T, T, 64>(p, stream);
}

fd_status bad(const char* message) { return record_error(FD_ERR_INVALID_ARG, message); }
fd_status unsupported(const char* message) { return record_error(FD_ERR_UNSUPPORTED, message); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int esize(int32_t dtype) { return dtype == FD_F8E4M3 ? 1 : dtype == FD_BF16 ? 2 : 4; }

// Rows of 16-byte groups: a contiguous last dimension, a 16-byte aligned base and other
// strides that are non-negative multiples of 16 bytes.
bool vectors(const fd_tensor* t) {
  if (t->stride[t->ndim - 1] != 1 || !aligned16(t->data)) return false;
  for (int i = 0; i + 1 < t->ndim; ++i)
    if (t->stride[i] < 0 || (t->stride[i] * esize(t->dtype)) % 16 != 0) return false;
  return true;
}

}  // namespace
}  // namespace fd

extern "C" fd_status fd_append_kv(const fd_tensor* q, const fd_tensor* k, const fd_tensor* v,
                                  const int32_t* cu_tokens, const int32_t* seq_lens,
                                  const fd_tensor* cos_sin, int32_t rope_style,
                                  const int32_t* pos_offset, fd_tensor* q_out,
                                  fd_tensor* k_cache, fd_tensor* v_cache, const float* k_scale,
                                  const float* v_scale, const fd_tensor* block_table,
                                  int32_t page_size, void* workspace, void* stream) {
  using namespace fd;
  if (!k || !v || !k_cache || !v_cache) return bad("k, v, k_cache and v_cache are required");
  if (!seq_lens) return bad("seq_lens is NULL");
  if ((q == nullptr) != (q_out == nullptr)) return bad("q and q_out go together");
  if (!k->data || !v->data || !k_cache->data || !v_cache->data || (q && (!q->data || !q_out->data)))
    return bad("a tensor has a NULL data pointer");
  if ((k->ndim != 3 && k->ndim != 4) || v->ndim != k->ndim || k_cache->ndim != 4 ||
      v_cache->ndim != 4 || (q && (q->ndim != k->ndim || q_out->ndim != k->ndim)))
    return bad("ranks must be k 3 or 4, v, q and q_out as k, caches 4");
  const bool multi = k->ndim == 4;
  if (multi && cu_tokens) return bad("cu_tokens belongs to 3-D q, k and v");
  const int hd = multi ? 2 : 1;               // index of the head dimension
  const int64_t Hkv = k->shape[hd], d = k->shape[hd + 1];
  const int64_t T = multi ? k->shape[0] * k->shape[1] : k->shape[0];
  for (int i = 0; i < k->ndim; ++i) {
    if (k->shape[i] <= 0) return bad("empty shape");
    if (v->shape[i] != k->shape[i]) return bad("k and v shapes differ");
    if (q && q->shape[i] != k->shape[i] && i != hd) return bad("q and k shapes differ outside the heads");
    if (q && q_out->shape[i] != q->shape[i]) return bad("q_out must have q's shape");
  }
  if (q && q->shape[hd] <= 0) return bad("empty shape");
  for (int i = 0; i < 4; ++i) {
    if (k_cache->shape[i] <= 0) return bad("empty cache shape");
    if (k_cache->shape[i] != v_cache->shape[i]) return bad("k_cache and v_cache shapes differ");
  }
  if (k_cache->shape[1] != Hkv || k_cache->shape[3] != d)
    return bad("the caches' heads or head dim differ from k's");
  // ---- types
  if (k->dtype != FD_BF16 && k->dtype != FD_F32) return unsupported("k and v must be bf16 or f32");
  if (v->dtype != k->dtype || (q && (q->dtype != k->dtype || q_out->dtype != k->dtype)))
    return bad("q, k, v and q_out must share one dtype");
  if (v_cache->dtype != k_cache->dtype) return bad("k_cache and v_cache must share one dtype");
  const bool fp8 = k_cache->dtype == FD_F8E4M3;
  if (fp8 ? k->dtype != FD_BF16 : k_cache->dtype != k->dtype)
    return unsupported("caches must have k's dtype, or FP8 E4M3 with bf16 k and v");
  if (d != 64 && d != 128) return unsupported("head dim not in {64, 128}");
  if (fp8 && d != 128) return unsupported("the FP8 KV cache needs head dim 128");
  if (!fp8 && (k_scale || v_scale)) return bad("k_scale / v_scale belong to an FP8 E4M3 cache only");
  if (((uintptr_t)k_scale & 3) || ((uintptr_t)v_scale & 3)) return bad("scales must be 4-byte aligned");
  // ---- strides and alignment
  if (!vectors(k) || !vectors(v) || (q && (!vectors(q) || !vectors(q_out))))
    return bad("q, k, v and q_out need contiguous 16-byte aligned rows and strides of whole 16 bytes");
  if (!vectors(k_cache) || !vectors(v_cache)) return bad("cache strides must be whole 16 bytes, rows contiguous and aligned");
  for (int i = 0; i < 3; ++i)
    if (k_cache->stride[i] <= 0 || v_cache->stride[i] <= 0) return bad("cache strides must be positive");
  for (int i = 0; q && i < hd + 1; ++i)
    if (q_out->stride[i] <= 0 && q_out->shape[i] > 1) return bad("q_out strides must be positive");
  if (k_cache->stride[2] < d || v_cache->stride[2] < d) return bad("cache token rows overlap");
  // ---- batch rows and capacity
  const bool paged = block_table != nullptr;
  int64_t B = 0, L_cap = 0;
  int log2_page = 0;
  if (paged) {
    if (!block_table->data) return bad("block_table has a NULL data pointer");
    if (block_table->ndim != 2 || block_table->dtype != FD_I32 || block_table->shape[0] <= 0 ||
        block_table->shape[1] <= 0 || block_table->stride[1] != 1)
      return bad("block_table must be int32 [B, max_pages] with contiguous rows");
    if (page_size < 8 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
      return bad("page_size must be a power of two in [8, 65536]");
    if (k_cache->shape[2] != page_size) return bad("paged caches must be [num_pages, Hkv, page_size, d]");
    B = block_table->shape[0];
    L_cap = block_table->shape[1] * page_size;
    while ((1 << log2_page) < page_size) ++log2_page;
  } else {
    if (page_size != 0) return bad("page_size must be 0 without a block table");
    B = k_cache->shape[0];
    L_cap = k_cache->shape[2];
  }
  if (L_cap >= (int64_t{1} << 31)) return bad("cache capacity must be below 2^31");
  if (T >= (int64_t{1} << 31) || B >= (int64_t{1} << 31)) return unsupported("2^31 tokens or rows or more");
  if (!cu_tokens && (multi ? k->shape[0] : T) != B)
    return bad("without cu_tokens k needs one leading entry per batch row");
  // ---- rotation
  int64_t rot = 0;
  if (cos_sin) {
    if (!cos_sin->data || cos_sin->ndim != 2 || cos_sin->dtype != FD_F32 || cos_sin->stride[1] != 1 ||
        cos_sin->shape[0] <= 0 || !aligned16(cos_sin->data) || cos_sin->stride[0] % 4 != 0 ||
        cos_sin->stride[0] < 0)
      return bad("cos_sin must be f32 [max_pos, rot] with contiguous, 16-byte aligned rows");
    rot = cos_sin->shape[1];
    if (rot <= 0 || rot > d) return bad("cos_sin must have 1 to d columns");
    if (rot % 16 != 0) return unsupported("the rotated dims must be a multiple of 16");
    if (rope_style != FD_ROPE_HALF && rope_style != FD_ROPE_INTERLEAVED) return bad("unknown rope_style");
  } else if (pos_offset) {
    return bad("pos_offset belongs to a rotation (cos_sin)");
  }
  if (workspace && ((uintptr_t)workspace & 255)) return bad("workspace must be 256-byte aligned");
  const int64_t Hq = q ? q->shape[hd] : 0;
  if (Hq + 2 * Hkv > (1 << 20) || T * ((Hq + 2 * Hkv + 3) / 4) > (int64_t{1} << 32))
    return unsupported("grid too large");

  AppendParams p;
  memset(&p, 0, sizeof p);
  p.q = q ? q->data : nullptr;
  p.k = k->data;
  p.v = v->data;
  p.q_out = q ? q_out->data : nullptr;
  p.k_cache = static_cast<uint8_t*>(k_cache->data);
  p.v_cache = static_cast<uint8_t*>(v_cache->data);
  const int td = multi ? 1 : 0;               // index of the token dimension
  p.k_sb = multi ? k->stride[0] : 0, p.k_st = k->stride[td], p.k_sh = k->stride[hd];
  p.v_sb = multi ? v->stride[0] : 0, p.v_st = v->stride[td], p.v_sh = v->stride[hd];
  if (q) {
    p.q_sb = multi ? q->stride[0] : 0, p.q_st = q->stride[td], p.q_sh = q->stride[hd];
    p.qo_sb = multi ? q_out->stride[0] : 0, p.qo_st = q_out->stride[td], p.qo_sh = q_out->stride[hd];
  }
  if (!multi && !cu_tokens) {                 // one token per row: the row is the batch index
    p.k_sb = p.k_st, p.v_sb = p.v_st, p.q_sb = p.q_st, p.qo_sb = p.qo_st;
  }
  p.kc_sb = k_cache->stride[0], p.kc_sh = k_cache->stride[1], p.kc_st = k_cache->stride[2];
  p.vc_sb = v_cache->stride[0], p.vc_sh = v_cache->stride[1], p.vc_st = v_cache->stride[2];
  p.T = (int32_t)T;
  p.Q = multi ? (int32_t)k->shape[1] : 1;
  p.B = (int32_t)B;
  p.Hq = (int32_t)Hq;
  p.Hkv = (int32_t)Hkv;
  p.rot = (int32_t)rot;
  p.interleaved = rope_style == FD_ROPE_INTERLEAVED ? 1 : 0;
  p.cu_tokens = cu_tokens;
  p.seq_lens = seq_lens;
  p.pos_offset = pos_offset;
  p.cos_sin = cos_sin ? static_cast<const float*>(cos_sin->data) : nullptr;
  p.cs_stride = cos_sin ? cos_sin->stride[0] : 0;
  p.max_pos = cos_sin ? cos_sin->shape[0] : 0;
  p.block_table = paged ? static_cast<const int32_t*>(block_table->data) : nullptr;
  p.bt_sb = paged ? block_table->stride[0] : 0;
  p.page_size = page_size;
  p.log2_page = log2_page;
  p.num_pages = paged ? k_cache->shape[0] : 0;
  p.L_cap = L_cap;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.flags = static_cast<uint32_t*>(workspace);
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = fp8                    ? launch<__nv_bfloat16, __nv_fp8_e4m3, 128>(p, s)
                        : k->dtype == FD_BF16 ? launch_d<__nv_bfloat16>((int)d, p, s)
                                              : launch_d<float>((int)d, p, s);
  if (e != cudaSuccess) return record_error(FD_ERR_CUDA, cudaGetErrorString(e));
  return FD_OK;
}
