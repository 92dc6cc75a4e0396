// fd_device.cuh -- device helpers: mbarriers, TMA tile loads, bounded waits, and the
// address of an element in a 128-byte-swizzled shared-memory tile.
//
// All waits are bounded by wall-clock time (%globaltimer): a wait that has not
// completed after kWaitLimitNs gives up, the caller raises a device error flag and
// leaves its loop, so a logic error can never hang the GPU.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd_internal.h"

namespace fd {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the phase with the given parity to complete; false after limit_ns.
__device__ __forceinline__ bool mbar_wait_for(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_ns() - t0 > limit_ns) return false;
  }
  return true;
}

// The kernels' wait: false after kWaitLimitNs.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  return mbar_wait_for(bar, parity, kWaitLimitNs);
}

// One tiled TMA load of a 5-D box into shared memory, completing on `bar`.
// Coordinate c0 (innermost) is always 0 here, so the 16-byte rule on it holds.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3, int c4,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(c4), "l"(policy)
      : "memory");
}

// L2 prefetch of one 5-D box of a tensor map (no shared memory, no barrier; a hint).
__device__ __forceinline__ void tma_prefetch_5d(const CUtensorMap* map, int c0, int c1, int c2,
                                                int c3, int c4) {
  asm volatile(
      "cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %3, %4, %5}];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// L2 policy for data read exactly once per step (the KV cache): evict first.
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Named barrier among `nthreads` threads (ids 1..15; 0 is __syncthreads).
__device__ __forceinline__ void named_bar_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// Programmatic dependent launch: let the next kernel in the stream start launching /
// wait until the previous kernel's memory is visible.
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The start of a partial kernel: wait for the previous kernel's memory -- or, with
// Params::late_wait, only make sure that nothing read from here on comes from an L1 line
// older than this point (what this pass reads was written before that kernel started).
__device__ __forceinline__ void pdl_start(const Params& p) {
  if (p.late_wait) __threadfence();
  else pdl_wait();
}
// Its end, called by every CTA's producer (or by a CTA without work): one CTA holds the grid
// open until the previous kernel is complete.
__device__ __forceinline__ void pdl_end(const Params& p) {
  if (p.late_wait && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    pdl_trigger();
    pdl_wait();
  }
}

// Base-2 exponential on the SFU (MUFU.EX2).  ex2(-inf) = +0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Widen bf16 to f32 exactly: a bf16 is the upper 16 bits of an f32.
__device__ __forceinline__ float bf16lo_to_f32(uint32_t packed) {
  return __uint_as_float(packed << 16);
}
__device__ __forceinline__ float bf16hi_to_f32(uint32_t packed) {
  return __uint_as_float(packed & 0xffff0000u);
}

// Byte offset, inside a tile written by a SWIZZLE_128B TMA box, of the 16-byte chunk
// `chunk` (0..7) of 128-byte line `line` (line index from a 1024-byte aligned base):
// the hardware stores chunk c of line X at position c XOR (X mod 8).
__device__ __forceinline__ uint32_t swz128(uint32_t line, uint32_t chunk) {
  return line * 128u + ((chunk ^ (line & 7u)) << 4);
}

// Byte offset, inside a K or V tile, of 16-byte chunk `c16` (0 .. row bytes / 16 - 1) of
// token row `r`.  The tile is a sequence of TMA boxes of R = 2^lb rows each (the whole
// tile, or one page); a box holds its rows line-slice by line-slice, [line][row][128 B],
// so row r sits in box r >> lb, and its line l is 128-byte line
// ((r >> lb) * LINES + l) * R + (r mod R) of the tile.  R is a multiple of 8, so the
// swizzle phase of that line is r mod 8: 8 consecutive rows of one 16-byte column hit 8
// different bank groups (conflict-free ldmatrix).
template <int LINES>
__device__ __forceinline__ uint32_t tile_chunk(uint32_t r, uint32_t c16, uint32_t lb) {
  const uint32_t X = ((((r >> lb) * LINES) + (c16 >> 3)) << lb) | (r & ((1u << lb) - 1u));
  return swz128(X, c16 & 7u);
}

}  // namespace fd
