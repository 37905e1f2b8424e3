// Cross-attention for few query rows (a token of a stream, a short draft): all
// rows that share a key head, up to 8, against its states.  bf16 in and out,
// fp32 arithmetic.
//
// Bound by the read of k and v, once.  The states of a key head are split over
// a cluster of up to 8 CTAs, over their warps, and over the D / 8 lanes that
// hold a state's row with 8 columns each; every group of lanes keeps a running
// maximum, sum and output of its own (no exchange inside the loop but the sums
// of a score), with the next states' k and v on their way into shared memory
// (cp.async; a lane copies what it reads itself, so there are no barriers).
// At the end the warps' results are joined across the cluster through
// distributed shared memory: one launch, no scratch.
// A row of a tensor-core tile would be one of 128: the tile kernel took 39 us
// where this one takes 20 (8 requests of 1,408 to 4,096 states, 8 key heads of
// 3 queries, d = 128, nothing in L2), most of it the fetch of its longer code.
#include <cuda_bf16.h>

#include "vdn_xattn.h"

namespace vdn {
namespace {

constexpr int NS = 3;             // stages of a warp's ring
constexpr int U = 4;              // states of a group of lanes in a stage
constexpr int kStage = 2 * U * 32;  // uint4 of a warp's stage: k and v
constexpr int kMaxCluster = 8;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

struct XfDev {
  int B, Tq, L, H, G, rows;  // rows = Tq G of a key head
  int ns;                    // CTAs of a cluster
  float scale;
  long long ks, vs;
  const int* kv_len;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* y;
  float* lse;
  uint32_t* status;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void expand(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
// the float at this shared address in CTA `rank` of the cluster
__device__ __forceinline__ float remote(const float* p, int rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int D, int R>
__global__ void __launch_bounds__(R > 4 ? 256 : 512) k_xattn_few(const XfDev x) {
  constexpr int LPK = D / 8, KPW = 32 / LPK, STEP = U * KPW;  // lanes a state, states a warp has at once, and in a stage
  extern __shared__ uint4 ring[];
  clear_status(x.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int li = lane % LPK, grp = lane / LPK;
  const int rank = blockIdx.x % x.ns, bh = blockIdx.x / x.ns, Hkv = x.H / x.G, b = bh / Hkv, hk = bh % Hkv;
  int n = x.L;
  if (x.kv_len != nullptr) n = max(0, min(__ldg(x.kv_len + b), x.L));
  // this CTA's states, in whole stages
  const int all = (n + STEP - 1) / STEP, per = (all + x.ns - 1) / x.ns, lo = min(rank * per, all), hi = min(lo + per, all);
  const __nv_bfloat16* kp = x.k + (long long)b * x.L * x.ks + hk * D + 8 * li;
  const __nv_bfloat16* vp = x.v + (long long)b * x.L * x.vs + hk * D + 8 * li;
  uint4* mine = ring + warp * NS * kStage + lane;
  auto fetch = [&](int stage, int it) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long key = (long long)it * STEP + u * KPW + grp;
      const bool on = it < hi && key < n;
      copy16(mine + stage * kStage + u * 32, on ? kp + key * x.ks : kp, on);
      copy16(mine + stage * kStage + (U + u) * 32, on ? vp + key * x.vs : vp, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int it = lo + warp;
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) fetch(s, it + s * nw);
  // the rows, times scale and log2 e
  float2 q[R][4], o[R][4];
  float m[R], l[R];
  const float c = x.scale * kLog2e;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (r < x.rows)
      raw = __ldg(reinterpret_cast<const uint4*>(x.q + (((long long)b * x.Tq + r / x.G) * x.H + hk * x.G + r % x.G) * D + 8 * li));
    expand(raw, q[r]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[r][i].x *= c;
      q[r][i].y *= c;
      o[r][i] = make_float2(0.f, 0.f);
    }
  }
  int st = 0;
#pragma unroll 1
  for (; it < hi; it += nw) {
    fetch(st == 0 ? NS - 1 : st - 1, it + (NS - 1) * nw);
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
    const uint4* at = mine + st * kStage;
    st = st + 1 == NS ? 0 : st + 1;
    float s[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 k[4];
      expand(at[u * 32], k);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) a = fma2(k[i], q[r][i], a);
        s[u][r] = a.x + a.y;
      }
    }
#pragma unroll
    for (int w = LPK / 2; w > 0; w >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) s[u][r] += __shfl_xor_sync(0xffffffffu, s[u][r], w);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((long long)it * STEP + u * KPW + grp >= n) {
#pragma unroll
        for (int r = 0; r < R; ++r) s[u][r] = -INFINITY;
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mx = m[r];
#pragma unroll
      for (int u = 0; u < U; ++u) mx = fmaxf(mx, s[u][r]);
      // no score above -inf so far: the reference stays at zero, weights of 0 and not of inf - inf
      const float ref = mx == -INFINITY ? 0.f : mx, f = ex2(m[r] - ref);
      m[r] = mx;
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[r][i].x *= f;
        o[r][i].y *= f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u][r] = ex2(s[u][r] - ref);
        l[r] += s[u][r];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 v[4];
      expand(at[(U + u) * 32], v);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[r][i] = fma2(make_float2(s[u][r], s[u][r]), v[i], o[r][i]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // the groups of a warp
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int w = LPK; w < 32; w <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[r], w), mx = fmaxf(m[r], mo), ref = mx == -INFINITY ? 0.f : mx;
      const float f = ex2(m[r] - ref);
      m[r] = mx;
      l[r] *= f;
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[r][i].x *= f;
        o[r][i].y *= f;
        o[r][i].x += __shfl_xor_sync(0xffffffffu, o[r][i].x, w);
        o[r][i].y += __shfl_xor_sync(0xffffffffu, o[r][i].y, w);
      }
    }
  }
  // the warps' results in shared memory: [warp][R][D + 2] = o, m, l; then the CTA's, [R][D + 2] behind them
  __syncthreads();
  constexpr int RW = D + 2;
  float* res = reinterpret_cast<float*>(ring);
  float* cta = res + nw * R * RW;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float* p = res + (warp * R + r) * RW;
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(p + 8 * li + 2 * i) = o[r][i];
      if (li == 0) {
        p[D] = m[r];
        p[D + 1] = l[r];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * D; i += blockDim.x) {
    const int r = i / D, col = i % D;
    float mx = -INFINITY;
    for (int w = 0; w < nw; ++w) mx = fmaxf(mx, res[(w * R + r) * RW + D]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, out = 0.f;
    for (int w = 0; w < nw; ++w) {
      const float* p = res + (w * R + r) * RW;
      const float f = ex2(p[D] - ref);
      sum = fmaf(f, p[D + 1], sum);
      out = fmaf(f, p[col], out);
    }
    cta[r * RW + col] = out;
    if (col == 0) {
      cta[r * RW + D] = mx;
      cta[r * RW + D + 1] = sum;
    }
  }
  cluster_sync();
  // the cluster's: the elements dealt to its CTAs, every CTA's part of one loaded before the first is used
  for (int i = rank * blockDim.x + threadIdx.x; i < x.rows * D; i += x.ns * blockDim.x) {
    const int r = i / D, col = i % D;
    float pm[kMaxCluster], pl[kMaxCluster], po[kMaxCluster], mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      const int from = k < x.ns ? k : 0;
      pm[k] = remote(cta + r * RW + D, from);
      pl[k] = remote(cta + r * RW + D + 1, from);
      po[k] = remote(cta + r * RW + col, from);
    }
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < x.ns) mx = fmaxf(mx, pm[k]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, out = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < x.ns) {
        const float f = ex2(pm[k] - ref);
        sum = fmaf(f, pl[k], sum);
        out = fmaf(f, po[k], out);
      }
    const long long row = ((long long)b * x.Tq + r / x.G) * x.H + hk * x.G + r % x.G;
    x.y[row * D + col] = __float2bfloat16_rn(n > 0 ? out / sum : 0.f);
    if (col == 0 && x.lse != nullptr) x.lse[row] = (n > 0 ? ref + __log2f(sum) : -INFINITY) * kLn2;
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <int D, int R>
cudaError_t launch(const XfDev& x, int warps, unsigned grid, cudaStream_t s) {
  const size_t smem = (size_t)warps * NS * kStage * sizeof(uint4);
  static_assert(NS * kStage * sizeof(uint4) >= 2 * R * (D + 2) * sizeof(float), "the ring holds the warps' results and the CTA's");
  auto kern = k_xattn_few<D, R>;
  // the most a block takes: 16 warps
  const cudaError_t e = allow_smem<k_xattn_few<D, R>>((size_t)16 * NS * kStage * sizeof(uint4));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(32 * warps);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)x.ns, 1, 1};
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, x);
}

template <int D>
cudaError_t pick(const XfDev& x, int warps, unsigned grid, cudaStream_t s) {
  if (x.rows == 1) return launch<D, 1>(x, warps, grid, s);
  if (x.rows == 2) return launch<D, 2>(x, warps, grid, s);
  if (x.rows == 3) return launch<D, 3>(x, warps, grid, s);
  if (x.rows == 4) return launch<D, 4>(x, warps, grid, s);
  return launch<D, 8>(x, warps, grid, s);
}

}  // namespace

bool xattn_few_supported(const XDims& d) {
  return (d.d == 64 || d.d == 128) && (long long)d.Tq * d.G <= 8 && (long long)d.B * d.Hkv <= (1LL << 31) / kMaxCluster - 1;
}

cudaError_t launch_xattn_few(const XDims& d, const XArgs& a, cudaStream_t s) {
  XfDev x{};
  x.B = d.B; x.Tq = d.Tq; x.L = d.L; x.H = d.H; x.G = d.G; x.rows = d.Tq * d.G;
  x.scale = d.scale;
  x.ks = d.ks; x.vs = d.vs;
  x.kv_len = d.kv_len;
  x.q = static_cast<const __nv_bfloat16*>(a.q);
  x.k = static_cast<const __nv_bfloat16*>(a.k);
  x.v = static_cast<const __nv_bfloat16*>(a.v);
  x.y = static_cast<__nv_bfloat16*>(const_cast<void*>(a.y));
  x.lse = a.lse;
  x.status = a.status;
  // CTAs of 4 warps while they fill the SMs (up to 4 on each); fewer key heads get more warps each.  A CTA has four
  // stages of states a warp at least where there are several.
  const long long base = (long long)d.B * d.Hkv;
  const int stages = (d.L + U * 32 / (d.d / 8) - 1) / (U * 32 / (d.d / 8));
  x.ns = 1;
  while (x.ns < kMaxCluster && base * x.ns < 4 * 148 && stages >= 2 * x.ns * 16) x.ns *= 2;
  const int warps = base * x.ns <= 148 && x.rows <= 4 ? 16 : base * x.ns <= 296 ? 8 : 4;
  const unsigned grid = (unsigned)(base * x.ns);
  return d.d == 128 ? pick<128>(x, warps, grid, s) : pick<64>(x, warps, grid, s);
}

}  // namespace vdn
