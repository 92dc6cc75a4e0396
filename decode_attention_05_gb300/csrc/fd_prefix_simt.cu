// fd_prefix_simt.cu -- attention of many query rows over a shared prompt, on CUDA cores
// (fd_prefix.cuh says what the pass computes): f32 inputs, and bf16 as a cross-check.
//
// A CTA holds 64 query rows (16 for groups of at most that many) of one group and kv head and walks its split of the prompt in
// tiles of 64 tokens: S = Q K^T, the running maximum and sum of the softmax ("AI Infra: math
// and infra optimisation in large models", section 2.6), O = O 2^(m_old - m_new) + P V.  All
// in f32.  256 threads: thread (ty, tx) of a 16 x 16 grid has the scores of rows 4 ty .. + 3 (row ty)
// and tokens tx + 16 j (j < 4), and the outputs of the same rows and D / 16 dims, so a row's 16
// threads lie in one half warp and reduce with shuffles.
//
// Bound: the FMA pipes.  Every 16-byte read of shared memory feeds 8 FMAs of the scores (10 of
// the outputs at D = 128), rows are padded by 16 bytes so that neither the tokens' rows nor P's
// columns collide in banks, and the next tile's rows are in registers while the current one is
// worked on.  K and V take turns in one buffer, which leaves room for two CTAs per SM.
#include <cuda_bf16.h>

#include "fd_prefix.cuh"

namespace fd {
namespace {

constexpr int kBN = 64, kThreads = 256;

template <int D, int BM>
struct Smem {
  static constexpr int LD = D + 4, LP = BM + 4;   // padded leading dimensions of q, k, v and p
  float q[BM * LD];
  float kv[kBN * LD];               // the tile's K, then its V
  float p[kBN * LP];
  float mask[kBN];                  // 0, or -inf for a token without weight
  PrefixTile tile;
  int found;
};

__device__ __forceinline__ float4 load4(const float* a) { return *reinterpret_cast<const float4*>(a); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* a) {
  const uint2 r = *reinterpret_cast<const uint2*>(a);
  return make_float4(bf16lo_to_f32(r.x), bf16hi_to_f32(r.x), bf16lo_to_f32(r.y), bf16hi_to_f32(r.y));
}

template <class T, int D, int BM>
__global__ void __launch_bounds__(kThreads, 2) fd_prefix_simt_kernel(const __grid_constant__ PrefixParams p) {
  using SM = Smem<D, BM>;
  constexpr int LD = SM::LD, kPs = SM::LP, DV = D / 16;
  constexpr int R = BM / 16;                   // query rows of a thread: 4 or 1
  constexpr int RPT = kThreads / (D / 4);      // tile rows that the threads load at once
  constexpr int NR = kBN / RPT;                // ... and how often
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  pdl_wait();
  pdl_trigger();                    // the pass over the rows' own keys runs next to this one
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int split = blockIdx.x, g = blockIdx.y;
  if (tid < 32) {
    PrefixTile t;
    const bool ok = find_tile<BM>(p, (int)blockIdx.z, t);
    if (ok) split_of<kBN>(p, split, t);
    if (tid == 0) {
      sm.tile = t;
      sm.found = ok ? 1 : 0;
    }
  }
  __syncthreads();
  if (!sm.found) return;
  const PrefixTile t = sm.tile;
  if (t.lo >= t.hi) {               // nothing of the prompt in this split
    if (tid < t.rows) p.lse_part[prefix_flat_row(p, t, g, tid) * p.S + split] = kNegInf;
    return;
  }
  const int lr = tid / (D / 4), lc = tid % (D / 4) * 4;   // this thread's row and dims of a load
  for (int r = lr; r < BM; r += RPT) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < t.rows) x = load4(static_cast<const T*>(p.q) + prefix_q_offset(p, t, g, r) + lc);
    const float f = p.scale_log2;
    *reinterpret_cast<float4*>(sm.q + r * LD + lc) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  }

  // Where the rows of a tile that this thread loads lie: page (or prompt) and slot, -1: none.
  bool bad_page = false;
  int64_t place[NR];
  int32_t slot[NR];
  auto locate = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int64_t tok = t0 + lr + i * RPT;
      place[i] = t.group;
      slot[i] = tok < t.hi ? (int32_t)tok : -1;
      if (slot[i] >= 0 && p.table != nullptr) {
        place[i] = p.table[(int64_t)t.group * p.table_sb + (tok >> p.log2_page)];
        slot[i] = (int32_t)(tok & (p.page_size - 1));
        if (place[i] < 0 || place[i] >= p.num_pages) {
          slot[i] = -1;
          bad_page = true;
        }
      }
    }
  };
  float4 next[NR];
  auto fetch = [&](const void* base, int64_t sb, int64_t sh, int64_t st) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
      next[i] = slot[i] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : load4(static_cast<const T*>(base) + place[i] * sb + g * sh + slot[i] * st + lc);
  };
  auto store = [&] {
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<float4*>(sm.kv + (lr + i * RPT) * LD + lc) = next[i];
  };

  float m[R], l[R], acc[R][DV];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[i][e] = 0.f;
  }
  locate(t.lo);
  fetch(p.k, p.k_sb, p.k_sh, p.k_st);
  for (int64_t t0 = t.lo; t0 < t.hi; t0 += kBN) {
    store();                        // K of this tile
    if (lc == 0) {
#pragma unroll
      for (int i = 0; i < NR; ++i) sm.mask[lr + i * RPT] = slot[i] < 0 ? kNegInf : 0.f;
    }
    __syncthreads();
    fetch(p.v, p.v_sb, p.v_sh, p.v_st);
    float s[R][4] = {};
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
      float4 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sm.kv + (tx + 16 * j) * LD + k);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float4 a = *reinterpret_cast<const float4*>(sm.q + (ty * R + i) * LD + k);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(a.x, b[j].x, fmaf(a.y, b[j].y, fmaf(a.z, b[j].z, fmaf(a.w, b[j].w, s[i][j]))));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool out = sm.mask[tx + 16 * j] != 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) s[i][j] = out ? kNegInf : s[i][j];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mt = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m[i], mt);
      const float c = mn == kNegInf ? 1.f : ex2(m[i] - mn);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = s[i][j] == kNegInf ? 0.f : ex2(s[i][j] - mn);
      l[i] = l[i] * c + ((s[i][0] + s[i][1]) + (s[i][2] + s[i][3]));
#pragma unroll
      for (int e = 0; e < DV; ++e) acc[i][e] *= c;
      m[i] = mn;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float* dst = sm.p + (tx + 16 * j) * kPs + ty * R;
      if constexpr (R == 4) *reinterpret_cast<float4*>(dst) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
      else *dst = s[0][j];
    }
    __syncthreads();                // K has been read by all
    store();                        // V
    __syncthreads();
    if (t0 + kBN < t.hi) {
      locate(t0 + kBN);
      fetch(p.k, p.k_sb, p.k_sh, p.k_st);
    }
#pragma unroll 4
    for (int k = 0; k < kBN; ++k) {
      float a[R];
      if constexpr (R == 4) {
        const float4 x = *reinterpret_cast<const float4*>(sm.p + k * kPs + ty * 4);
        a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
      } else {
        a[0] = sm.p[k * kPs + ty];
      }
#pragma unroll
      for (int e = 0; e < DV; e += 4) {
        const float4 b = *reinterpret_cast<const float4*>(sm.kv + k * LD + tx * 4 + (e / 4) * 64);
        const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int f = 0; f < 4; ++f) {
#pragma unroll
          for (int i = 0; i < R; ++i) acc[i][e + f] = fmaf(a[i], bb[f], acc[i][e + f]);
        }
      }
    }
    __syncthreads();                // V and P have been read by all
  }
  if (bad_page) atomicOr(p.flags, FD_DEVFLAG_PAGE);
#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    const int r = ty * R + i;
    if (r >= t.rows) continue;
    const int64_t at = prefix_flat_row(p, t, g, r) * p.S + split;
    if (tx == 0) p.lse_part[at] = l[i] == 0.f ? kNegInf : (m[i] + __log2f(l[i])) * 0.6931471805599453f;
    const float f = 1.f / l[i];
#pragma unroll
    for (int e = 0; e < DV; e += 4)
      *reinterpret_cast<float4*>(p.o_part + at * D + tx * 4 + (e / 4) * 64) =
          make_float4(acc[i][e] * f, acc[i][e + 1] * f, acc[i][e + 2] * f, acc[i][e + 3] * f);
  }
}

template <class T, int D, int BM>
cudaError_t launch(const PrefixParams& p, cudaStream_t stream) {
  auto kernel = fd_prefix_simt_kernel<T, D, BM>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.apply(kernel, (int)sizeof(Smem<D, BM>));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.S, (unsigned)p.Hkv,
                  (unsigned)prefix_row_tiles(p.B, (int64_t)p.Q * p.G, p.group_start != nullptr, p.P, BM));
  return launch_pdl(kernel, grid, kThreads, sizeof(Smem<D, BM>), stream, p);
}

// 16-row tiles where groups of equal size would not have more: such a call is bound by its
// reads of K and V, and 64-row tiles would do four times the arithmetic on padding.
template <class T, int D>
cudaError_t launch_rows(const PrefixParams& p, cudaStream_t stream) {
  const int64_t rows = ((int64_t)p.B + p.P - 1) / p.P * p.Q * p.G;
  return rows <= 16 ? launch<T, D, 16>(p, stream) : launch<T, D, 64>(p, stream);
}

}  // namespace

// dtype: that of q and the caches, f32 or bf16.
cudaError_t launch_prefix_simt(const PrefixParams& p, int32_t dtype, int d, cudaStream_t stream) {
  if (dtype == FD_F32) return d == 128 ? launch_rows<float, 128>(p, stream) : launch_rows<float, 64>(p, stream);
  return d == 128 ? launch_rows<__nv_bfloat16, 128>(p, stream) : launch_rows<__nv_bfloat16, 64>(p, stream);
}

}  // namespace fd
