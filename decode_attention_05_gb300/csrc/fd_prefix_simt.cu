// fd_prefix_simt.cu -- attention of many query rows over a shared prompt, on CUDA cores
// (fd_prefix.cuh says what the pass computes).
//
// A CTA holds 64 query rows of one group and kv head and walks its split of the prompt in
// tiles of 32 tokens: S = Q K^T, the running maximum and sum of the softmax ("AI Infra: math
// and infra optimisation in large models", section 2.6), O = O 2^(m_old - m_new) + P V.  All
// in f32.  256 threads: thread (ty, tx) of a 16 x 16 grid has the scores of rows 4 ty .. + 3
// and tokens 2 tx, 2 tx + 1, and the outputs of the same rows and D / 16 dims, so a row's 16
// threads lie in one half warp and reduce with shuffles.
#include <cuda_bf16.h>

#include "fd_prefix.cuh"

namespace fd {
namespace {

constexpr int kBM = 64, kBN = 32, kThreads = 256;
constexpr int kQs = kBM + 4, kKs = kBN + 4, kPs = kBM + 4;   // padded leading dimensions

template <int D>
constexpr size_t smem_bytes() {
  return (size_t)(D * kQs + D * kKs + kBN * D + kBN * kPs) * sizeof(float);
}

__device__ __forceinline__ void load4(const float* a, float* x) {
  const float4 r = *reinterpret_cast<const float4*>(a);
  x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* a, float* x) {
  const uint2 r = *reinterpret_cast<const uint2*>(a);
  x[0] = bf16lo_to_f32(r.x), x[1] = bf16hi_to_f32(r.x);
  x[2] = bf16lo_to_f32(r.y), x[3] = bf16hi_to_f32(r.y);
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) fd_prefix_simt_kernel(const __grid_constant__ PrefixParams p) {
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;                 // [D][kQs], rows of the tile along the last index
  float* ks = qs + D * kQs;         // [D][kKs]
  float* vs = ks + D * kKs;         // [kBN][D]
  float* ps = vs + kBN * D;         // [kBN][kPs]
  __shared__ PrefixTile tile;
  __shared__ int found;
  pdl_wait();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int split = blockIdx.x, g = blockIdx.y;
  if (tid < 32) {
    PrefixTile t;
    const bool ok = find_tile<kBM>(p, (int)blockIdx.z, t);
    if (ok) split_of<kBN>(p, split, t);
    if (tid == 0) {
      tile = t;
      found = ok ? 1 : 0;
    }
  }
  __syncthreads();
  if (!found) return;
  const PrefixTile t = tile;
  if (t.lo >= t.hi) {               // nothing of the prompt in this split
    if (tid < t.rows) p.lse_part[prefix_flat_row(p, t, g, tid) * p.S + split] = kNegInf;
    return;
  }
  for (int i = tid; i < kBM * (D / 4); i += kThreads) {
    const int r = i % kBM, c = i / kBM;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < t.rows) load4(static_cast<const T*>(p.q) + prefix_q_offset(p, t, g, r) + c * 4, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) qs[(c * 4 + e) * kQs + r] = x[e] * p.scale_log2;
  }

  constexpr int DV = D / 16;
  float m[4], l[4], acc[4][DV];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[i][e] = 0.f;
  }
  bool bad_page = false;
  for (int64_t t0 = t.lo; t0 < t.hi; t0 += kBN) {
    __syncthreads();                // the previous tile has been read
    for (int i = tid; i < kBN * (D / 4); i += kThreads) {
      const int r = i % kBN, c = i / kBN;
      const int64_t tok = t0 + r;
      float kx[4] = {0.f, 0.f, 0.f, 0.f}, vx[4] = {0.f, 0.f, 0.f, 0.f};
      bool live = tok < t.hi;
      int64_t place = t.group, slot = tok;
      if (live && p.table != nullptr) {
        place = p.table[(int64_t)t.group * p.table_sb + (tok >> p.log2_page)];
        slot = tok & (p.page_size - 1);
        if (place < 0 || place >= p.num_pages) {
          live = false;
          bad_page = true;
        }
      }
      if (live) {
        load4(static_cast<const T*>(p.k) + place * p.k_sb + g * p.k_sh + slot * p.k_st + c * 4, kx);
        load4(static_cast<const T*>(p.v) + place * p.v_sb + g * p.v_sh + slot * p.v_st + c * 4, vx);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) ks[(c * 4 + e) * kKs + r] = kx[e];
      *reinterpret_cast<float4*>(vs + r * D + c * 4) = make_float4(vx[0], vx[1], vx[2], vx[3]);
      if (c == 0) ps[r * kPs] = live ? 0.f : kNegInf;   // which tokens count, until P is written
    }
    __syncthreads();
    float s[4][2] = {};
#pragma unroll 8
    for (int k = 0; k < D; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(qs + k * kQs + ty * 4);
      const float2 b = *reinterpret_cast<const float2*>(ks + k * kKs + tx * 2);
      s[0][0] = fmaf(a.x, b.x, s[0][0]), s[0][1] = fmaf(a.x, b.y, s[0][1]);
      s[1][0] = fmaf(a.y, b.x, s[1][0]), s[1][1] = fmaf(a.y, b.y, s[1][1]);
      s[2][0] = fmaf(a.z, b.x, s[2][0]), s[2][1] = fmaf(a.z, b.y, s[2][1]);
      s[3][0] = fmaf(a.w, b.x, s[3][0]), s[3][1] = fmaf(a.w, b.y, s[3][1]);
    }
    const bool out0 = ps[(tx * 2) * kPs] == kNegInf, out1 = ps[(tx * 2 + 1) * kPs] == kNegInf;
    float pr[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i][0] = out0 ? kNegInf : s[i][0];
      s[i][1] = out1 ? kNegInf : s[i][1];
      float mt = fmaxf(s[i][0], s[i][1]);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m[i], mt);
      const float c = mn == kNegInf ? 1.f : ex2(m[i] - mn);
      pr[i][0] = s[i][0] == kNegInf ? 0.f : ex2(s[i][0] - mn);
      pr[i][1] = s[i][1] == kNegInf ? 0.f : ex2(s[i][1] - mn);
      l[i] = l[i] * c + pr[i][0] + pr[i][1];
#pragma unroll
      for (int e = 0; e < DV; ++e) acc[i][e] *= c;
      m[i] = mn;
    }
    __syncthreads();                // the marks have been read
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float4*>(ps + (tx * 2 + j) * kPs + ty * 4) =
          make_float4(pr[0][j], pr[1][j], pr[2][j], pr[3][j]);
    __syncwarp();                   // a row's P is written and read by its own half warp
#pragma unroll 4
    for (int k = 0; k < kBN; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(ps + k * kPs + ty * 4);
#pragma unroll
      for (int e = 0; e < DV; e += 4) {
        const float4 b = *reinterpret_cast<const float4*>(vs + k * D + tx * 4 + (e / 4) * 64);
        const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          acc[0][e + f] = fmaf(a.x, bb[f], acc[0][e + f]);
          acc[1][e + f] = fmaf(a.y, bb[f], acc[1][e + f]);
          acc[2][e + f] = fmaf(a.z, bb[f], acc[2][e + f]);
          acc[3][e + f] = fmaf(a.w, bb[f], acc[3][e + f]);
        }
      }
    }
  }
  if (bad_page) atomicOr(p.flags, FD_DEVFLAG_PAGE);
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    const int r = ty * 4 + i;
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

template <class T, int D>
cudaError_t launch(const PrefixParams& p, cudaStream_t stream) {
  auto kernel = fd_prefix_simt_kernel<T, D>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.apply(kernel, (int)smem_bytes<D>());
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.S, (unsigned)p.Hkv,
                  (unsigned)prefix_row_tiles(p.B, (int64_t)p.Q * p.G, p.group_start ? p.P : 1, kBM));
  return launch_pdl(kernel, grid, kThreads, smem_bytes<D>(), stream, p);
}

}  // namespace

// dtype: that of q and the caches, f32 or bf16.
cudaError_t launch_prefix_simt(const PrefixParams& p, int32_t dtype, int d, cudaStream_t stream) {
  if (dtype == FD_F32) return d == 128 ? launch<float, 128>(p, stream) : launch<float, 64>(p, stream);
  return d == 128 ? launch<__nv_bfloat16, 128>(p, stream)
                  : launch<__nv_bfloat16, 64>(p, stream);
}

}  // namespace fd
