// Cross-attention to an encoder's states: the problem as the kernels see it,
// and the launchers of its implementations.
#pragma once

#include "vdn_internal.h"

namespace vdn {

struct XDims {
  int B, Tq, L, H, Hkv, G, d;  // G = H / Hkv query heads share a key head
  float scale;
  long long ks, vs;            // elements between tokens of k and of v
  const int* kv_len;           // [B] valid encoder states, or null: L everywhere
};

struct XArgs {
  const void *q, *k, *v;
  const void *y;       // forward: written; backward: the forward's output
  float* lse;          // [B, Tq, H]; forward: written unless null; backward: read
  const void* dy;
  void *dq, *dk, *dv;
  uint32_t* status;    // status words of the bounded waits; a call's first kernel clears them
  void* scratch;       // backward: behind the status words
  long long wait_limit;  // of the tensor-core kernels' bounded waits, in clock cycles; 0: the default
};

__device__ __forceinline__ int kv_valid(const XDims& d, int b) {
  if (d.kv_len == nullptr) return d.L;
  const int n = __ldg(d.kv_len + b);
  return n < 0 ? 0 : n > d.L ? d.L : n;
}

// The items of a persistent kernel's CTA: every gridDim.x-th of a mixed-radix
// count (d0 fastest).  Stepping adds the stride's digits, without divisions.
struct ItemGrid {
  int items, r0, r1, r2;   // all items, radices of the first three digits
  int s0, s1, s2, s3;      // digits of the grid's size
};
inline ItemGrid item_grid(int items, int r0, int r1, int r2, int grid) {
  return {items, r0, r1, r2, grid % r0, grid / r0 % r1, grid / r0 / r1 % r2, grid / r0 / r1 / r2};
}
struct ItemPos {
  int item, d0, d1, d2, d3;
  __device__ __forceinline__ void start(const ItemGrid& g) {
    item = blockIdx.x;
    int r = item;
    d0 = r % g.r0; r /= g.r0;
    d1 = r % g.r1; r /= g.r1;
    d2 = r % g.r2; d3 = r / g.r2;
  }
  __device__ __forceinline__ bool on(const ItemGrid& g) const { return item < g.items; }
  __device__ __forceinline__ void next(const ItemGrid& g) {
    item += gridDim.x;
    d0 += g.s0;
    d1 += g.s1;
    d2 += g.s2;
    d3 += g.s3;
    if (d0 >= g.r0) { d0 -= g.r0; ++d1; }
    if (d1 >= g.r1) { d1 -= g.r1; ++d2; }
    if (d2 >= g.r2) { d2 -= g.r2; ++d3; }
  }
};

// Clears the two status words: a call's first kernel does it as it starts, long before a bounded wait can run out.
__device__ __forceinline__ void clear_status(uint32_t* status) {
  if (blockIdx.x == 0 && threadIdx.x < 2) status[threadIdx.x] = 0;
}

// SIMT, float32 arithmetic: float32 at d = 32, 64 or 128, bf16 at d = 32 (vdn_xattn.cu)
cudaError_t launch_xattn_simt(const XDims& d, const XArgs& a, bool bf16, cudaStream_t s);
// needs the scratch of xattn_simt_bwd_scratch: <dO, o> per query row, and partial sums
size_t xattn_simt_bwd_scratch(const XDims& d);
cudaError_t launch_xattn_simt_bwd(const XDims& d, const XArgs& a, bool bf16, cudaStream_t s);

// bf16, d = 64 or 128, up to 16 query rows for a key head (vdn_xattn_few.cu); no scratch
bool xattn_few_supported(const XDims& d);
cudaError_t launch_xattn_few(const XDims& d, const XArgs& a, cudaStream_t s);

// bf16 on the tensor cores, d = 64 or 128 (vdn_xattn_tc.cu); scratch: partial results
bool xattn_tc_supported(const XDims& d);
size_t xattn_tc_scratch(const XDims& d);
cudaError_t launch_xattn_tc(const XDims& d, const XArgs& a, cudaStream_t s);
// its backward (vdn_xattn_bwd_tc.cu); scratch: <dO, o> per query row and partial sums
size_t xattn_tc_bwd_scratch(const XDims& d);
cudaError_t launch_xattn_tc_bwd(const XDims& d, const XArgs& a, cudaStream_t s);

}  // namespace vdn
