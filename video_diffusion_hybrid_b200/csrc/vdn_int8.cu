// The 8-bit integer linear layer: quantisation of the rows, and the product
// for few rows.  (For many rows the product runs on the tensor cores,
// vdn_gemm_tc.cu.)
//
//   s[m] = amax_k |x[m, k]| / 127,  q[m, k] = round(x[m, k] / s[m])  (half to even)
//   out[m, n] = (sum_k q[m, k] w[n, k]) s[m] w_scale[n] + bias[n]
// A row whose amax is below 2^-119 counts as zero (s = 1, codes 0: 1 / s stays
// finite); a row that holds an infinity or a NaN has s = NaN and codes 0, so
// its outputs are NaN.
#include <cuda_bf16.h>

#include "vdn_internal.h"

namespace vdn {
namespace {

// 8 consecutive elements, 16-byte aligned
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// |x| as its bit pattern orders like |x|, with infinities and NaNs on top
__device__ __forceinline__ uint32_t abs_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

struct Scale {
  float s, inv;  // inv = 0: the row's codes are 0
};
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
  Scale r;
  if (amax_bits >= 0x7F800000u) {
    r.s = __uint_as_float(0x7FC00000u);
    r.inv = 0.f;
  } else if (amax_bits < ((127u - 119u) << 23)) {
    r.s = 1.f;
    r.inv = 0.f;
  } else {
    r.s = __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
    r.inv = 1.0f / r.s;
  }
  return r;
}

// round(x / s), half to even, exactly: x * inv is off by less than one code,
// and the remainder x - q s, one fused operation without a rounding error at
// this size, decides about the neighbour.
__device__ __forceinline__ int code(float x, const Scale& c) {
  if (c.inv == 0.f) return 0;
  float q = rintf(x * c.inv);
  const float r = fmaf(-q, c.s, x), h = 0.5f * c.s;
  const bool odd = ((int)q & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.f;
  else if (r < -h || (r == -h && odd)) q -= 1.f;
  return (int)q;
}
// The same for 8 elements: x inv + 1.5 * 2^23 in one fused operation is the
// nearest integer, with its two's complement in the low byte.  inv is off by a
// relative 2^-24, a quotient by less than 10^-5: only a quotient that near to
// a tie (one in 50,000) takes the exact way.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Scale& c) {
  constexpr float kMagic = 12582912.f;
  if (c.inv == 0.f) return make_uint2(0u, 0u);
  uint32_t t[8];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = fmaf(v[i], c.inv, kMagic);
    t[i] = __float_as_uint(u);
    far = fmaxf(far, fabsf(fmaf(v[i], c.inv, kMagic - u)));
  }
  if (far > 0.49999f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (uint32_t)code(v[i], c);
  }
  uint2 r;
  r.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
  return r;
}

// 8 elements as they are stored, and the largest |x| among them as bits
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };
template <typename T> __device__ __forceinline__ Raw8<T> raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void expand8(const Raw8<float>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void expand8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// TPR threads a row, up to VPT vectors of 8 elements each kept in registers, as
// stored, between the maximum and the codes (one read of x); longer rows are
// read twice.  Bound by HBM: 2 (4) bytes read and one written for an element.
template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(256) k_quantize_rows(const T* __restrict__ x, int rows, int cols, uint2* __restrict__ q,
                                                       float* __restrict__ scale, uint32_t* status) {
  if (status != nullptr && blockIdx.x == 0 && threadIdx.x < 2) status[threadIdx.x] = 0;
  const int t = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const bool on = row < rows;
  const int nv = cols / 8;
  const T* p = x + row * cols;
  Raw8<T> raw[VPT];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (on && t + i * TPR < nv) raw[i] = raw8(p + 8 * (t + i * TPR));
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (on && t + i * TPR < nv) {
      float v[8];
      expand8(raw[i], v);
      m = max(m, abs_bits(v));
    }
  for (int i = t + VPT * TPR; on && i < nv; i += TPR) {
    float u[8];
    load8(p + 8 * i, u);
    m = max(m, abs_bits(u));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (TPR > 32) {
    __shared__ uint32_t red[8];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    const int first = threadIdx.x / TPR * (TPR / 32);
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) m = max(m, red[first + i]);
  }
  if (!on) return;
  const Scale c = scale_of(m);
  if (t == 0) scale[row] = c.s;
  uint2* o = q + row * nv;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * TPR < nv) {
      float v[8];
      expand8(raw[i], v);
      o[t + i * TPR] = codes8(v, c);
    }
  for (int i = t + VPT * TPR; i < nv; i += TPR) {
    float u[8];
    load8(p + 8 * i, u);
    o[i] = codes8(u, c);
  }
}

template <typename T>
cudaError_t quantize(const T* x, int rows, int cols, uint2* q, float* scale, uint32_t* st, cudaStream_t s) {
  // a warp a row keeps up to 1024 columns in registers, a block a row 8192
  if (cols <= 1024) k_quantize_rows<T, 32, 4><<<(unsigned)((rows + 7LL) / 8), 256, 0, s>>>(x, rows, cols, q, scale, st);
  else k_quantize_rows<T, 256, 4><<<rows, 256, 0, s>>>(x, rows, cols, q, scale, st);
  return cudaGetLastError();
}

// ------------------------------------------------------------- few rows --
// Up to kFewRows rows: the product is bound by the read of the weight, once.
// Every block forms the codes of all rows in shared memory by itself (x is
// small and stays in L2), which saves a launch; a warp has NC output channels
// and walks K in steps of 512 bytes, four byte products per instruction.  Its
// first AHEAD steps of the weight are under way while the codes are formed.
// (The two sides meet there, us a call from bf16 rows, this kernel / the quantiser and the tensor cores: 6,144 x 4,096
// 9.8 / 24.3 at one row, 18.2 / 25.1 at 4, 24.3 / 25.0 at 8; 1,280 x 784 3.1 / 7.5, 5.2 / 7.6, 8.2 / 7.7.)
constexpr int kFewRows = 8;
constexpr int NC = 2;           // channels per warp
constexpr int AHEAD = 8;        // steps
constexpr int kFewThreads = 256;
constexpr size_t kFewSmem = 200 * 1024;

// a read-only load that stays where it is written, ahead of the work that hides it
__device__ __forceinline__ uint4 load_pinned(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <typename T, typename To, int MR>
__global__ void __launch_bounds__(kFewThreads) k_int8_few(int M, int K, int N, const void* __restrict__ xp,
                                                          const float* __restrict__ x_scale, const uint4* __restrict__ w,
                                                          const float* __restrict__ w_scale, const float* __restrict__ bias,
                                                          To* __restrict__ out, uint32_t* status) {
  if (status != nullptr && blockIdx.x == 0 && threadIdx.x < 2) status[threadIdx.x] = 0;  // nothing here waits
  extern __shared__ __align__(16) unsigned char sm[];
  __shared__ uint32_t red[kFewThreads / 32];
  __shared__ float sx[MR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nv = K / 16;
  const int n0 = (blockIdx.x * (kFewThreads / 32) + warp) * NC;
  const uint4* wr = w + (size_t)n0 * nv;  // N is a multiple of NC
  uint4 first[AHEAD][NC];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      first[i][j] = make_uint4(0, 0, 0, 0);
      if (n0 < N && lane + 32 * i < nv) first[i][j] = load_pinned(wr + (size_t)j * nv + lane + 32 * i);
    }
  // rows' codes and scales: one row by the whole block, several by a warp each (M <= 8 = the warps)
  if (x_scale != nullptr) {
    for (int i = threadIdx.x; i < M * nv; i += kFewThreads) reinterpret_cast<uint4*>(sm)[i] = __ldg(static_cast<const uint4*>(xp) + i);
    if (threadIdx.x < M) sx[threadIdx.x] = __ldg(x_scale + threadIdx.x);
  } else if (MR == 1 || warp < M) {
    const int m = MR == 1 ? 0 : warp, t0 = MR == 1 ? threadIdx.x : lane;
    constexpr int TS = MR == 1 ? kFewThreads : 32;
    const T* src = static_cast<const T*>(xp) + (size_t)m * K;
    uint32_t mx = 0;
#pragma unroll 4
    for (int i = t0; i < K / 8; i += TS) {
      float v[8];
      load8(src + 8 * i, v);
      mx = max(mx, abs_bits(v));
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (MR == 1) {
      if (lane == 0) red[warp] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kFewThreads / 32; ++i) mx = max(mx, red[i]);
    }
    const Scale c = scale_of(mx);
    if (t0 == 0) sx[m] = c.s;
    uint2* dst = reinterpret_cast<uint2*>(sm + (size_t)m * K);
#pragma unroll 4
    for (int i = t0; i < K / 8; i += TS) {
      float v[8];
      load8(src + 8 * i, v);
      dst[i] = codes8(v, c);
    }
  }
  __syncthreads();
  if (n0 >= N) return;
  int acc[MR][NC];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[m][j] = 0;
  auto step = [&](const uint4 (&u)[NC], int i) {
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      if (m >= M) continue;
      const uint4 a = reinterpret_cast<const uint4*>(sm + (size_t)m * K)[i];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        acc[m][j] = __dp4a((int)a.x, (int)u[j].x, acc[m][j]);
        acc[m][j] = __dp4a((int)a.y, (int)u[j].y, acc[m][j]);
        acc[m][j] = __dp4a((int)a.z, (int)u[j].z, acc[m][j]);
        acc[m][j] = __dp4a((int)a.w, (int)u[j].w, acc[m][j]);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (lane + 32 * i < nv) step(first[i], lane + 32 * i);
#pragma unroll 4
  for (int i = lane + 32 * AHEAD; i < nv; i += 32) {
    uint4 u[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) u[j] = __ldg(wr + (size_t)j * nv + i);
    step(u, i);
  }
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int s = __reduce_add_sync(0xffffffffu, acc[m][j]);
      if (lane == 0) {
        const float r = scaled_sum(s, sx[m], __ldg(w_scale + n0 + j), bias ? __ldg(bias + n0 + j) : 0.f);
        if constexpr (sizeof(To) == 2) out[(size_t)m * N + n0 + j] = __float2bfloat16_rn(r);
        else out[(size_t)m * N + n0 + j] = r;
      }
    }
  }
}

template <typename T, typename To, int MR>
cudaError_t few(const vdn_int8_cfg& c, const vdn_int8_args& a, cudaStream_t s) {
  auto kern = k_int8_few<T, To, MR>;
  const size_t smem = (size_t)c.M * c.K;
  const cudaError_t e = allow_smem<k_int8_few<T, To, MR>>(kFewSmem);
  if (e != cudaSuccess) return e;
  const int per = kFewThreads / 32 * NC;
  kern<<<(c.N + per - 1) / per, kFewThreads, smem, s>>>(c.M, c.K, c.N, a.x, c.x_dtype == VDN_I8 ? a.x_scale : nullptr,
                                                        static_cast<const uint4*>(a.w), a.w_scale, a.bias,
                                                        static_cast<To*>(a.out), a.status);
  return cudaGetLastError();
}
template <typename T, typename To>
cudaError_t few_rows(const vdn_int8_cfg& c, const vdn_int8_args& a, cudaStream_t s) {
  if (c.M == 1) return few<T, To, 1>(c, a, s);
  if (c.M <= 4) return few<T, To, 4>(c, a, s);
  return few<T, To, kFewRows>(c, a, s);
}
template <typename T>
cudaError_t few_out(const vdn_int8_cfg& c, const vdn_int8_args& a, cudaStream_t s) {
  return c.out_dtype == VDN_BF16 ? few_rows<T, __nv_bfloat16>(c, a, s) : few_rows<T, float>(c, a, s);
}

}  // namespace

cudaError_t launch_quantize_int8(const void* x, int dtype, int rows, int cols, void* q, float* scale, uint32_t* status,
                                 cudaStream_t s) {
  uint2* o = static_cast<uint2*>(q);
  return dtype == VDN_BF16 ? quantize(static_cast<const __nv_bfloat16*>(x), rows, cols, o, scale, status, s)
                           : quantize(static_cast<const float*>(x), rows, cols, o, scale, status, s);
}

bool int8_few_supported(int M, int K, int N) { return M <= kFewRows && (size_t)M * K <= kFewSmem && N % NC == 0; }

cudaError_t launch_int8_few(const vdn_int8_cfg& c, const vdn_int8_args& a, cudaStream_t s) {
  return c.x_dtype == VDN_F32 ? few_out<float>(c, a, s) : few_out<__nv_bfloat16>(c, a, s);
}

}  // namespace vdn
