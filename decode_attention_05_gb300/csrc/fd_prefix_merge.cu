// fd_prefix_merge.cu -- the merge of a row's partials over its prompt and over its own keys
// (fd_prefix.cuh): one softmax over both sets' LSEs,
//   M = max LSE_i,  w_i = exp(LSE_i - M),  out = sum_i w_i O_i / sum_i w_i,
//   lse_out = M + log(sum_i w_i)
// ("FlashDecoding interview notes" (gtnt.cn/news/53829), section three).  A partial with
// LSE_i = -inf has no key: weight 0, and its O_i (never written) is not used.  A row without
// any key gets out = 0 and lse_out = -inf.
#include <cuda_bf16.h>

#include "fd_prefix.cuh"

namespace fd {
namespace {

constexpr int kWarps = 4, kBatch = 4;

// W warps fold the partials of one row (W = 4: one row a CTA; 1: four rows a CTA); a lane
// holds D / 32 dims.
template <int D, int W>
__global__ void __launch_bounds__(kWarps * 32) fd_prefix_merge_kernel(const __grid_constant__ MergeParams p) {
  constexpr int VEC = D / 32;
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  __shared__ float wm[kWarps], ww[kWarps];
  __shared__ __align__(16) float accs[kWarps][D];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = W == 1 ? (int)blockIdx.x * kWarps + warp : (int)blockIdx.x;
  if (row >= p.rows) return;
  float M = kNegInf, sum = 0.f, acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int set = 0; set < 2; ++set) {
    // Pointers that step from batch to batch, so that a partial costs no address arithmetic:
    // with thousands of rows the instructions, not the bytes, set this kernel's time.
    int left = p.S[set] - (W == 1 ? 0 : warp);
    const int64_t first = (int64_t)row * p.S[set] + (W == 1 ? 0 : warp);
    const float* lse = p.lse[set] + first;
    const float* o = p.o[set] + first * D + lane * VEC;
#pragma unroll 1
    for (; left > 0; left -= W * kBatch, lse += W * kBatch, o += W * kBatch * D) {
      float ls[kBatch], v[kBatch][VEC];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const bool in = W * u < left;
        ls[u] = in ? lse[W * u] * kLog2e : kNegInf;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[u][e] = 0.f;
        if (in) {
          if constexpr (VEC == 4) {
            const float4 x = *reinterpret_cast<const float4*>(o + W * u * D);
            v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(o + W * u * D);
            v[u][0] = x.x, v[u][1] = x.y;
          }
        }
      }
      float mn = M;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, ls[u]);
      const float c = M == kNegInf ? 0.f : ex2(M - mn);
      sum *= c;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] *= c;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const bool live = ls[u] != kNegInf;    // a NaN counts: it is the row's result
        const float w = live ? ex2(ls[u] - mn) : 0.f;
        sum += w;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(w, live ? v[u][e] : 0.f, acc[e]);
      }
      M = mn;
    }
  }
  if constexpr (W > 1) {                       // the warps' states, by the same rule
#pragma unroll
    for (int e = 0; e < VEC; ++e) accs[warp][lane * VEC + e] = acc[e];
    if (lane == 0) {
      wm[warp] = M;
      ww[warp] = sum;
    }
    __syncthreads();
    if (warp != 0) return;
    float c[kWarps];
    M = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      c[w] = wm[w] == kNegInf ? (ww[w] == 0.f ? 0.f : 1.f) : ex2(wm[w] - M);
      sum = fmaf(ww[w], c[w], sum);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) acc[e] = fmaf(accs[w][lane * VEC + e], c[w], acc[e]);
    }
  }
  const bool none = sum == 0.f;                // no key at all
  const float inv = none ? 0.f : 1.f / sum;
  const int bj = row / p.Hq, b = bj / p.Q;
  const int64_t at = b * p.out_sb + (bj - b * p.Q) * p.out_sj + (row - bj * p.Hq) * p.out_sh + lane * VEC;
  if (p.out_bf16) {
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) o[e / 2] = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  } else {
    float2* o = reinterpret_cast<float2*>(static_cast<float*>(p.out) + at);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) o[e / 2] = make_float2(acc[e] * inv, acc[e + 1] * inv);
  }
  if (lane == 0 && p.lse_out != nullptr) p.lse_out[row] = none ? kNegInf : (M + __log2f(sum)) * kLn2;
}

template <int D>
cudaError_t launch(const MergeParams& p, cudaStream_t stream) {
  // A warp per row once that gives every SM a few rows to overlap; before that four warps
  // share a row, whose loads then run side by side.
  if (p.rows >= 8 * (int64_t)sm_count())
    return launch_pdl(fd_prefix_merge_kernel<D, 1>, dim3((unsigned)((p.rows + kWarps - 1) / kWarps)),
                      kWarps * 32, 0, stream, p);
  return launch_pdl(fd_prefix_merge_kernel<D, kWarps>, dim3((unsigned)p.rows), kWarps * 32, 0, stream, p);
}

}  // namespace

cudaError_t launch_prefix_merge(const MergeParams& p, cudaStream_t stream) {
  return p.d == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace fd
