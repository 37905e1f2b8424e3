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
  uint32_t* status;    // status words of the bounded waits
  void* scratch;       // backward: behind the status words
};

__device__ __forceinline__ int kv_valid(const XDims& d, int b) {
  if (d.kv_len == nullptr) return d.L;
  const int n = __ldg(d.kv_len + b);
  return n < 0 ? 0 : n > d.L ? d.L : n;
}

// SIMT, float32 arithmetic: any type, d = 32, 64 or 128 (vdn_xattn.cu)
cudaError_t launch_xattn_simt(const XDims& d, const XArgs& a, bool bf16, cudaStream_t s);
// needs the scratch of xattn_simt_bwd_scratch: <dO, o> per query row
size_t xattn_simt_bwd_scratch(const XDims& d);
cudaError_t launch_xattn_simt_bwd(const XDims& d, const XArgs& a, bool bf16, cudaStream_t s);

// bf16 on the tensor cores, d = 64 or 128 (vdn_xattn_tc.cu); scratch: partial results
bool xattn_tc_supported(const XDims& d);
size_t xattn_tc_scratch(const XDims& d);
cudaError_t launch_xattn_tc(const XDims& d, const XArgs& a, cudaStream_t s);
// its backward (vdn_xattn_bwd_tc.cu); scratch: <dO, o> per query row and partial sums
size_t xattn_tc_bwd_scratch(const XDims& d);
cudaError_t launch_xattn_tc_bwd(const XDims& d, const XArgs& a, cudaStream_t s);

}  // namespace vdn
