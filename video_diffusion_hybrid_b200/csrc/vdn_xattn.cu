// Cross-attention to an encoder's states of another length, SIMT kernels in
// float32 arithmetic: the exact mode (float32 tensors), and head sizes that
// the tensor-core kernels do not take.
//
// For query row (b, t, h) over the first n = kv_len[b] states of batch b and
// key head h / G:
//   P = softmax(s q K^T), o = P V, lse = ln sum_j exp(s q k_j)
// and with dO the gradient of o, Delta = <dO, o>:
//   dS = P (dO V^T - Delta),  dq = s dS K,  dk = s sum_h dS^T q,  dv = sum_h P^T dO
// the sums over the G query heads of the key head.  n = 0: o = 0, lse = -inf,
// no gradient.  States past n are never read: they may hold anything.
//
// A block of 256 threads has 64 rows against tiles of 64 columns; a thread has
// a 4 x 4 piece of the score tile and 4 x D/16 of the product behind it, fed
// by 16-byte shared-memory reads of transposed operands.  Bound by the fp32
// pipe and those reads; one launch (the backward: three, or four) without atomics.
#include <cuda_bf16.h>

#include "vdn_xattn.h"

namespace vdn {
namespace {

constexpr int BT = 64;       // rows and columns of a tile
constexpr int PT = BT + 4;   // padded row of a transposed or score tile (floats)
constexpr int kThr = 256;

__device__ __forceinline__ float ld(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float* p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float4 ld4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

// Rows [0, n) of src (row stride in elements) to dst[c][r] (transposed, TR) or
// dst[r][c] (row of D + 4 floats); rows past n as zeros.  Four columns a thread;
// transposed, neighbours take neighbouring rows (no bank is hit twice, and L1
// has the rest of a row's sectors for the next turn).
template <typename T, int D, bool TR>
__device__ __forceinline__ void load_tile(float* dst, const T* src, long long stride, int n) {
#pragma unroll 4
  for (int i = threadIdx.x; i < BT * D / 4; i += kThr) {
    const int r = TR ? i % BT : i / (D / 4), c = 4 * (TR ? i / BT : i % (D / 4));
    const float4 v = r < n ? ld4(src + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (TR) {
      dst[c * PT + r] = v.x;
      dst[(c + 1) * PT + r] = v.y;
      dst[(c + 2) * PT + r] = v.z;
      dst[(c + 3) * PT + r] = v.w;
    } else {
      *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = v;
    }
  }
}

// acc[i][j] += sum_c a[c][4 ty + i] b[c][CT tx + j], both transposed tiles: CT columns a thread, 16 CT in all
template <int D, int CT>
__device__ __forceinline__ void dot_cols(float (&acc)[4][4], const float* a, const float* b, int ty, int tx) {
#pragma unroll 4
  for (int c = 0; c < D; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(a + c * PT + 4 * ty);
    float ys[4];
    if constexpr (CT == 4) {
      const float4 y = *reinterpret_cast<const float4*>(b + c * PT + 4 * tx);
      ys[0] = y.x; ys[1] = y.y; ys[2] = y.z; ys[3] = y.w;
    } else if constexpr (CT == 2) {
      const float2 y = *reinterpret_cast<const float2*>(b + c * PT + 2 * tx);
      ys[0] = y.x; ys[1] = y.y;
    } else {
      ys[0] = b[c * PT + tx];
    }
    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
  }
}
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float* a, const float* b, int ty, int tx) {
  dot_cols<D, 4>(acc, a, b, ty, tx);
}

// o[i][2 m + e] += sum_j p[j][4 ty + i] v[j][2 (tx + 16 m) + e]: p [column][row] (PT), v [column][D + 4]
template <int D>
__device__ __forceinline__ void acc_tile(float (&o)[4][D / 16], const float* p, const float* v, int ty, int tx, int n = BT) {
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const float4 x = *reinterpret_cast<const float4*>(p + j * PT + 4 * ty);
    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
      const float2 y = *reinterpret_cast<const float2*>(v + j * (D + 4) + 2 * (tx + 16 * m));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i][2 * m] = fmaf(xs[i], y.x, o[i][2 * m]);
        o[i][2 * m + 1] = fmaf(xs[i], y.y, o[i][2 * m + 1]);
      }
    }
  }
}

template <typename T, int D>
__device__ __forceinline__ void store_rows(T* dst, long long stride, int n, const float (&o)[4][D / 16], const float (&f)[4],
                                           int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= n) continue;
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
      st(dst + r * stride + 2 * (tx + 16 * m), o[i][2 * m] * f[i]);
      st(dst + r * stride + 2 * (tx + 16 * m) + 1, o[i][2 * m + 1] * f[i]);
    }
  }
}

// sum / max over the 16 threads of a row group (a half warp)
__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// block -> (b, h, first row) with `per` tiles of rows for each of the `heads` heads
__device__ __forceinline__ void where(long long item, long long per, int heads, int& b, int& h, int& r0) {
  r0 = (int)(item % per) * BT;
  const long long bh = item / per;
  b = (int)(bh / heads);
  h = (int)(bh % heads);
}

template <int D> constexpr size_t fwd_smem() { return sizeof(float) * (2 * D * PT + BT * (D + 4) + BT * PT); }
template <int D> constexpr size_t bwd_smem() { return sizeof(float) * (4 * D * PT + 2 * BT * (D + 4) + BT * PT); }

// Scores of 64 rows against nk <= 16 CT states, their weights to p[state][row]; running maximum and sum, output rescaled
template <int D, int CT>
__device__ __forceinline__ void attend(const float* q, const float* k, float* p, float scale, int nk, int ty, int tx, float (&m)[4],
                                       float (&l)[4], float (&o)[4][D / 16]) {
  float s[4][4] = {};
  dot_cols<D, CT>(s, q, k, ty, tx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float mx = m[i];
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      s[i][j] = CT * tx + j < nk ? s[i][j] * scale : -INFINITY;
      mx = fmaxf(mx, s[i][j]);
    }
    mx = half_max(mx);
    // a row whose scores are all -inf so far keeps its reference at zero: no inf - inf
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float f = expf(m[i] - ref);
    m[i] = mx;
    l[i] *= f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[i][j] *= f;
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      s[i][j] = expf(s[i][j] - ref);
      l[i] += s[i][j];
    }
  }
#pragma unroll
  for (int j = 0; j < CT; ++j)
    *reinterpret_cast<float4*>(p + (CT * tx + j) * PT + 4 * ty) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThr) k_xattn(const XDims d, const XArgs a) {
  clear_status(a.status);
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sK = sQ + D * PT, *sV = sK + D * PT, *sP = sV + BT * (D + 4);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int b, h, q0;
  where(blockIdx.x, (d.Tq + BT - 1) / BT, d.H, b, h, q0);
  const int nq = min(BT, d.Tq - q0), n = kv_valid(d, b), hk = h / d.G;
  const long long qrow = ((long long)b * d.Tq + q0) * d.H + h;
  const T* k = static_cast<const T*>(a.k) + (long long)b * d.L * d.ks + (long long)hk * D;
  const T* v = static_cast<const T*>(a.v) + (long long)b * d.L * d.vs + (long long)hk * D;
  load_tile<T, D, true>(sQ, static_cast<const T*>(a.q) + qrow * D, (long long)d.H * D, nq);
  float m[4], l[4], o[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
  }
  for (int k0 = 0; k0 < n; k0 += BT) {
    const int nk = min(BT, n - k0);
    __syncthreads();
    load_tile<T, D, true>(sK, k + k0 * d.ks, d.ks, nk);
    load_tile<T, D, false>(sV, v + k0 * d.vs, d.vs, nk);
    __syncthreads();
    // a tile's columns: four a thread, or two or one where no more states are left
    if (nk > 32) attend<D, 4>(sQ, sK, sP, d.scale, nk, ty, tx, m, l, o);
    else if (nk > 16) attend<D, 2>(sQ, sK, sP, d.scale, nk, ty, tx, m, l, o);
    else attend<D, 1>(sQ, sK, sP, d.scale, nk, ty, tx, m, l, o);
    __syncthreads();
    acc_tile<D>(o, sP, sV, ty, tx, nk);
  }
  float inv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = half_sum(l[i]);
    inv[i] = n > 0 ? 1.0f / t : 0.f;
    if (a.lse != nullptr && tx == 0 && 4 * ty + i < nq)
      a.lse[qrow + (long long)(4 * ty + i) * d.H] = n > 0 ? m[i] + logf(t) : -INFINITY;
  }
  store_rows<T, D>(static_cast<T*>(const_cast<void*>(a.y)) + qrow * D, (long long)d.H * D, nq, o, inv, ty, tx);
}

// Delta = <dO, o> of every query row: a warp a row
template <typename T>
__global__ void __launch_bounds__(256) k_xattn_delta(const T* __restrict__ y, const T* __restrict__ dy, float* __restrict__ delta,
                                                     long long rows, int D, uint32_t* status) {
  clear_status(status);
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  float s = 0.f;
  for (int c = threadIdx.x & 31; c < D; c += 32) s = fmaf(ld(y + row * D + c), ld(dy + row * D + c), s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) delta[row] = s;
}

// dq of 64 query rows of one head
template <typename T, int D>
__global__ void __launch_bounds__(kThr) k_xattn_dq(const XDims d, const XArgs a, const float* delta) {
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sDO = sQ + D * PT, *sK = sDO + D * PT, *sV = sK + D * PT, *sKr = sV + D * PT, *sS = sKr + BT * (D + 4);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int b, h, q0;
  where(blockIdx.x, (d.Tq + BT - 1) / BT, d.H, b, h, q0);
  const int nq = min(BT, d.Tq - q0), n = kv_valid(d, b), hk = h / d.G;
  const long long qrow = ((long long)b * d.Tq + q0) * d.H + h;
  const T* k = static_cast<const T*>(a.k) + (long long)b * d.L * d.ks + (long long)hk * D;
  const T* v = static_cast<const T*>(a.v) + (long long)b * d.L * d.vs + (long long)hk * D;
  load_tile<T, D, true>(sQ, static_cast<const T*>(a.q) + qrow * D, (long long)d.H * D, nq);
  load_tile<T, D, true>(sDO, static_cast<const T*>(a.dy) + qrow * D, (long long)d.H * D, nq);
  float lse[4], del[4], o[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool on = 4 * ty + i < nq && n > 0;
    lse[i] = on ? a.lse[qrow + (long long)(4 * ty + i) * d.H] : INFINITY;
    del[i] = on ? delta[qrow + (long long)(4 * ty + i) * d.H] : 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
  }
  for (int k0 = 0; k0 < n; k0 += BT) {
    const int nk = min(BT, n - k0);
    __syncthreads();
    load_tile<T, D, true>(sK, k + k0 * d.ks, d.ks, nk);
    load_tile<T, D, true>(sV, v + k0 * d.vs, d.vs, nk);
    load_tile<T, D, false>(sKr, k + k0 * d.ks, d.ks, nk);
    __syncthreads();
    float s[4][4] = {}, t[4][4] = {};
    dot_tile<D>(s, sQ, sK, ty, tx);
    dot_tile<D>(t, sDO, sV, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = 4 * tx + j < nk ? expf(fmaf(s[i][j], d.scale, -lse[i])) : 0.f;
        sS[(4 * tx + j) * PT + 4 * ty + i] = p * (t[i][j] - del[i]);
      }
    __syncthreads();
    acc_tile<D>(o, sS, sKr, ty, tx);
  }
  const float f[4] = {d.scale, d.scale, d.scale, d.scale};
  store_rows<T, D>(static_cast<T*>(a.dq) + qrow * D, (long long)d.H * D, nq, o, f, ty, tx);
}

// Splits of the dk / dv sums over the group's query tiles, so that there is about a CTA for every SM (they take one
// each): partial sums [ns][B L Hkv][D] in fp32, joined in order.
struct KvSplit {
  int ns, per;       // splits, query tiles of each (over the G heads of a group, tile fastest)
  float *dk, *dv;    // partial sums, null with one split
};

// dk and dv of 64 states of one key head, over its G query heads and all query rows (or a split's share of them)
template <typename T, int D>
__global__ void __launch_bounds__(kThr) k_xattn_dkv(const XDims d, const XArgs a, const float* delta, const KvSplit sp) {
  extern __shared__ __align__(16) float sm[];
  float *sK = sm, *sV = sK + D * PT, *sQ = sV + D * PT, *sDO = sQ + D * PT, *sQr = sDO + D * PT, *sDOr = sQr + BT * (D + 4),
        *sP = sDOr + BT * (D + 4);  // P, then dS: one buffer (D = 128 has no room for two)
  __shared__ float sL[BT], sD[BT];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int b, hk, k0;
  where(blockIdx.x / sp.ns, (d.L + BT - 1) / BT, d.Hkv, b, hk, k0);
  const int split = blockIdx.x % sp.ns, nqt = (d.Tq + BT - 1) / BT, u0 = split * sp.per, u1 = min(u0 + sp.per, d.G * nqt);
  const int rows = min(BT, d.L - k0), nk = max(0, min(rows, kv_valid(d, b) - k0));
  const T* k = static_cast<const T*>(a.k) + ((long long)b * d.L + k0) * d.ks + (long long)hk * D;
  const T* v = static_cast<const T*>(a.v) + ((long long)b * d.L + k0) * d.vs + (long long)hk * D;
  load_tile<T, D, true>(sK, k, d.ks, nk);
  load_tile<T, D, true>(sV, v, d.vs, nk);
  float ok[4][D / 16], ov[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < D / 16; ++j) ok[i][j] = ov[i][j] = 0.f;
  if (nk > 0)
    for (int u = u0; u < u1; ++u) {
      const int g = u / nqt, q0 = u % nqt * BT, nq = min(BT, d.Tq - q0);
      const long long qrow = ((long long)b * d.Tq + q0) * d.H + hk * d.G + g;
      const T *q = static_cast<const T*>(a.q) + qrow * D, *dy = static_cast<const T*>(a.dy) + qrow * D;
      __syncthreads();
      load_tile<T, D, true>(sQ, q, (long long)d.H * D, nq);
      load_tile<T, D, true>(sDO, dy, (long long)d.H * D, nq);
      load_tile<T, D, false>(sQr, q, (long long)d.H * D, nq);
      load_tile<T, D, false>(sDOr, dy, (long long)d.H * D, nq);
      if (threadIdx.x < BT) {
        const bool on = threadIdx.x < nq;
        sL[threadIdx.x] = on ? a.lse[qrow + (long long)threadIdx.x * d.H] : INFINITY;
        sD[threadIdx.x] = on ? delta[qrow + (long long)threadIdx.x * d.H] : 0.f;
      }
      __syncthreads();
      float s[4][4] = {}, t[4][4] = {};
      dot_tile<D>(s, sK, sQ, ty, tx);
      dot_tile<D>(t, sV, sDO, ty, tx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 4 * tx + j;
          const float p = 4 * ty + i < nk ? expf(fmaf(s[i][j], d.scale, -sL[c])) : 0.f;
          sP[c * PT + 4 * ty + i] = p;
          t[i][j] = p * (t[i][j] - sD[c]);
        }
      __syncthreads();
      acc_tile<D>(ov, sP, sDOr, ty, tx);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sP[(4 * tx + j) * PT + 4 * ty + i] = t[i][j];
      __syncthreads();
      acc_tile<D>(ok, sP, sQr, ty, tx);
    }
  // selected, not left to the weights of zero: 0 times a NaN or an infinity of dO is no zero
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * ty + i >= nk) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) ok[i][j] = ov[i][j] = 0.f;
    }
  const float fk[4] = {d.scale, d.scale, d.scale, d.scale}, fv[4] = {1.f, 1.f, 1.f, 1.f};
  const long long krow = ((long long)b * d.L + k0) * d.Hkv + hk;
  if (sp.dk != nullptr) {
    const long long at = (split * (long long)d.B * d.L * d.Hkv + krow) * D;
    store_rows<float, D>(sp.dk + at, (long long)d.Hkv * D, rows, ok, fk, ty, tx);
    store_rows<float, D>(sp.dv + at, (long long)d.Hkv * D, rows, ov, fv, ty, tx);
    return;
  }
  store_rows<T, D>(static_cast<T*>(a.dk) + krow * D, (long long)d.Hkv * D, rows, ok, fk, ty, tx);
  store_rows<T, D>(static_cast<T*>(a.dv) + krow * D, (long long)d.Hkv * D, rows, ov, fv, ty, tx);
}

// the splits' sums in order, an element of dk and one of dv a thread
template <typename T>
__global__ void __launch_bounds__(256) k_xattn_join(const KvSplit sp, T* dk, T* dv, long long n) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float k = 0.f, v = 0.f;
  for (int s = 0; s < sp.ns; ++s) {
    k += sp.dk[s * n + i];
    v += sp.dv[s * n + i];
  }
  st(dk + i, k);
  st(dv + i, v);
}

KvSplit kv_split(const XDims& d) {
  const long long items = (long long)d.B * d.Hkv * ((d.L + BT - 1) / BT), all = (long long)d.G * ((d.Tq + BT - 1) / BT);
  long long ns = items < 148 ? 148 / items : 1;
  if (ns > all) ns = all;
  KvSplit s{};
  s.per = (int)((all + ns - 1) / ns);
  s.ns = (int)((all + s.per - 1) / s.per);
  return s;
}
size_t delta_bytes(const XDims& d) { return ((size_t)d.B * d.Tq * d.H * sizeof(float) + 255) / 256 * 256; }

template <typename T, int D>
cudaError_t fwd(const XDims& d, const XArgs& a, cudaStream_t s) {
  const long long items = (long long)d.B * d.H * ((d.Tq + BT - 1) / BT);
  const cudaError_t e = allow_smem<k_xattn<T, D>>(fwd_smem<D>());
  if (e != cudaSuccess) return e;
  k_xattn<T, D><<<(unsigned)items, kThr, fwd_smem<D>(), s>>>(d, a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const XDims& d, const XArgs& a, cudaStream_t s) {
  const long long rows = (long long)d.B * d.Tq * d.H;
  float* delta = static_cast<float*>(a.scratch);
  k_xattn_delta<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(static_cast<const T*>(a.y), static_cast<const T*>(a.dy), delta, rows, D, a.status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = allow_smem<k_xattn_dq<T, D>>(bwd_smem<D>())) != cudaSuccess || (e = allow_smem<k_xattn_dkv<T, D>>(bwd_smem<D>())) != cudaSuccess)
    return e;
  const long long qi = (long long)d.B * d.H * ((d.Tq + BT - 1) / BT), ki = (long long)d.B * d.Hkv * ((d.L + BT - 1) / BT);
  k_xattn_dq<T, D><<<(unsigned)qi, kThr, bwd_smem<D>(), s>>>(d, a, delta);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  KvSplit sp = kv_split(d);
  const long long n = (long long)d.B * d.L * d.Hkv * D;
  if (sp.ns > 1) {
    sp.dk = reinterpret_cast<float*>(static_cast<char*>(a.scratch) + delta_bytes(d));
    sp.dv = sp.dk + sp.ns * n;
  }
  k_xattn_dkv<T, D><<<(unsigned)(ki * sp.ns), kThr, bwd_smem<D>(), s>>>(d, a, delta, sp);
  if ((e = cudaGetLastError()) != cudaSuccess || sp.ns == 1) return e;
  k_xattn_join<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(sp, static_cast<T*>(a.dk), static_cast<T*>(a.dv), n);
  return cudaGetLastError();
}

}  // namespace

size_t xattn_simt_bwd_scratch(const XDims& d) {
  const KvSplit s = kv_split(d);
  return delta_bytes(d) + (s.ns > 1 ? 2 * (size_t)s.ns * d.B * d.L * d.Hkv * d.d * sizeof(float) : 0);
}

cudaError_t launch_xattn_simt(const XDims& d, const XArgs& a, bool bf16, cudaStream_t s) {
  switch (d.d) {
    case 32: return bf16 ? fwd<__nv_bfloat16, 32>(d, a, s) : fwd<float, 32>(d, a, s);
    case 64: return bf16 ? cudaErrorInvalidValue : fwd<float, 64>(d, a, s);
    case 128: return bf16 ? cudaErrorInvalidValue : fwd<float, 128>(d, a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_xattn_simt_bwd(const XDims& d, const XArgs& a, bool bf16, cudaStream_t s) {
  switch (d.d) {
    case 32: return bf16 ? bwd<__nv_bfloat16, 32>(d, a, s) : bwd<float, 32>(d, a, s);
    case 64: return bf16 ? cudaErrorInvalidValue : bwd<float, 64>(d, a, s);
    case 128: return bf16 ? cudaErrorInvalidValue : bwd<float, 128>(d, a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace vdn
