// Cross-attention for few query rows (a token of a stream, a short draft): all
// rows that share a key head, up to 16, against its states.  bf16 in and out,
// fp32 scores, softmax and accumulation.
//
// Bound by the read of k and v, once.  The states of a key head are split over
// a cluster of up to 8 CTAs and over their warps.  A warp takes 16 states at a
// time from a ring of its own in shared memory (cp.async, so that the next
// ones are on their way; no block barrier), forms the 16 x 16 scores and adds
// P V with warp-level matrix products (16 rows are the smallest tile those
// have, and all that there are; with the 128 rows of a tcgen05 tile this took
// 39 us where this takes 28), and keeps a running maximum, sum and output.
// At the end the warps' results are joined across the cluster through
// distributed shared memory: one launch, no scratch.
// (Dot products on the FMA pipe, a row of k in 16 lanes, took 31 us: the sums
// over lanes alone are 48 shuffles for 8 states and 3 rows.)
#include <cuda_bf16.h>

#include "tc_common.cuh"
#include "vdn_xattn.h"

namespace vdn {
namespace {
using tc::ex2;
using tc::pack_bf16;

constexpr int NS = 3;      // stages of a warp's ring
constexpr int KT = 16;     // states of a stage
constexpr int ROWS = 16;   // query rows of a key head
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
// four 8 x 8 blocks of 16-bit values, lane l giving the address of row l % 8 of block l / 8
__device__ __forceinline__ void blocks4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void blocks4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c (16 x 8) += a (16 x 16) b (16 x 8), bf16 with fp32 sums
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int D> constexpr int stage_chunks() { return 2 * KT * D / 8; }  // 16-byte chunks: k, then v
template <int D> constexpr int most_warps() { return D == 128 ? 8 : 16; }
template <int D> constexpr size_t warp_smem() { return (size_t)NS * stage_chunks<D>() * 16; }

template <int D>
__global__ void __launch_bounds__(32 * most_warps<D>()) k_xattn_few(const XfDev x) {
  constexpr int CPR = D / 8, KPI = 32 / CPR;  // chunks of a row, rows a warp copies at once
  extern __shared__ uint4 ring[];
  clear_status(x.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int g = lane >> 2, t2 = 2 * (lane & 3);  // of a 16 x 8 result: rows g and g + 8, columns t2 and t2 + 1
  const int rank = blockIdx.x % x.ns, bh = blockIdx.x / x.ns, Hkv = x.H / x.G, b = bh / Hkv, hk = bh % Hkv;
  int n = x.L;
  if (x.kv_len != nullptr) n = max(0, min(__ldg(x.kv_len + b), x.L));
  // this CTA's states, in whole stages
  const int all = (n + KT - 1) / KT, per = (all + x.ns - 1) / x.ns, lo = min(rank * per, all), hi = min(lo + per, all);
  uint4* mine = ring + warp * NS * stage_chunks<D>();
  const int ck = lane % CPR, rk = lane / CPR;  // the chunk and the first row that this lane copies
  const __nv_bfloat16* kp = x.k + ((long long)b * x.L + rk) * x.ks + hk * D + 8 * ck;
  const __nv_bfloat16* vp = x.v + ((long long)b * x.L + rk) * x.vs + hk * D + 8 * ck;
  // chunk c of row r lies at c ^ (r % 8): the eight rows of a block in eight different groups of banks
  auto fetch = [&](int stage, int it) {
    uint4* sk = mine + stage * stage_chunks<D>();
#pragma unroll
    for (int i = 0; i < KT / KPI; ++i) {
      const int r = rk + i * KPI;
      const long long key = (long long)it * KT + i * KPI;
      const bool on = it < hi && it * KT + r < n;
      uint4* dst = sk + r * CPR + (ck ^ (r & 7));
      copy16(dst, on ? kp + key * x.ks : x.k, on);
      copy16(dst + KT * CPR, on ? vp + key * x.vs : x.v, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int it = lo + warp;
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) fetch(s, it + s * nw);
  // the query rows as left operands: rows g and g + 8, columns t2 and t2 + 8 of every 16
  uint32_t qa[D / 16][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(x.q + (((long long)b * x.Tq + r / x.G) * x.H + hk * x.G + r % x.G) * D + t2);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      qa[i][h] = r < x.rows ? __ldg(p + 8 * i) : 0u;
      qa[i][h + 2] = r < x.rows ? __ldg(p + 8 * i + 4) : 0u;
    }
  }
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const float c = x.scale * kLog2e;
  int st = 0;
#pragma unroll 1
  for (; it < hi; it += nw) {
    __syncwarp();  // the stage filled next was read by every lane
    fetch(st == 0 ? NS - 1 : st - 1, it + (NS - 1) * nw);
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
    __syncwarp();
    const uint4* sk = mine + st * stage_chunks<D>();
    const uint4* sv = sk + KT * CPR;
    st = st + 1 == NS ? 0 : st + 1;
    // scores of states 0..7 and 8..15, two chains each
    float s[2][2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][0][e] = s[j][1][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 8 * j + (lane & 7);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t kb[4];
        blocks4(kb, smem_addr(sk + r * CPR + ((4 * i + (lane >> 3)) ^ (r & 7))));
        mma16(s[j][0], qa[2 * i], kb[0], kb[1]);
        mma16(s[j][1], qa[2 * i + 1], kb[2], kb[3]);
      }
    }
    uint32_t pa[4];
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float z[4], mx = m[h];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = it * KT + 8 * (e >> 1) + t2 + (e & 1);
        z[e] = (s[e >> 1][0][2 * h + (e & 1)] + s[e >> 1][1][2 * h + (e & 1)]) * c;
        if (key >= n) z[e] = -INFINITY;
        mx = fmaxf(mx, z[e]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // no score above -inf so far: the reference stays at zero, weights of 0 and not of inf - inf
      const float ref = mx == -INFINITY ? 0.f : mx;
      f[h] = ex2(m[h] - ref);
      m[h] = mx;
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = ex2(z[e] - ref);
      l[h] = fmaf(l[h], f[h], (z[0] + z[1]) + (z[2] + z[3]));
      pa[h] = pack_bf16(z[0], z[1]);      // the product's operand type; l adds the unrounded weights
      pa[h + 2] = pack_bf16(z[2], z[3]);
    }
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= f[0];
        o[i][1] *= f[0];
        o[i][2] *= f[1];
        o[i][3] *= f[1];
      }
    }
    const int r = lane & 15;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t vb[4];
      blocks4_t(vb, smem_addr(sv + r * CPR + ((2 * i + (lane >> 4)) ^ (r & 7))));
      mma16(o[2 * i], pa, vb[0], vb[1]);
      mma16(o[2 * i + 1], pa, vb[2], vb[3]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // the warps' results in shared memory: [warp][rows][D + 2] = o, m, l; then the CTA's, [rows][D + 2] behind them
  __syncthreads();
  constexpr int RW = D + 2;
  float* res = reinterpret_cast<float*>(ring);
  float* cta = res + nw * x.rows * RW;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (g + 8 * h < x.rows) {
      float* p = res + (warp * x.rows + g + 8 * h) * RW;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(p + 8 * i + t2) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
      if (t2 == 0) {
        p[D] = m[h];
        p[D + 1] = l[h];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < x.rows * D; i += blockDim.x) {
    const int r = i / D, col = i % D;
    float mx = -INFINITY;
    for (int w = 0; w < nw; ++w) mx = fmaxf(mx, res[(w * x.rows + r) * RW + D]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, out = 0.f;
    for (int w = 0; w < nw; ++w) {
      const float* p = res + (w * x.rows + r) * RW;
      const float e = ex2(p[D] - ref);
      sum = fmaf(e, p[D + 1], sum);
      out = fmaf(e, p[col], out);
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
        const float e = ex2(pm[k] - ref);
        sum = fmaf(e, pl[k], sum);
        out = fmaf(e, po[k], out);
      }
    const long long row = ((long long)b * x.Tq + r / x.G) * x.H + hk * x.G + r % x.G;
    x.y[row * D + col] = __float2bfloat16_rn(n > 0 ? out / sum : 0.f);
    if (col == 0 && x.lse != nullptr) x.lse[row] = (n > 0 ? ref + __log2f(sum) : -INFINITY) * kLn2;
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <int D>
cudaError_t launch(XfDev x, cudaStream_t s) {
  // A ring of 24 KB (d = 128) a warp: two CTAs of 4 warps on an SM, or one of 8.  The states are split over as many CTAs
  // as still run at once, while a warp has two stages or more.
  constexpr int W = most_warps<D>() / 2;
  const long long base = (long long)x.B * (x.H / x.G);
  const int stages = (x.L + KT - 1) / KT;
  x.ns = 1;
  while (x.ns < kMaxCluster && base * 2 * x.ns <= 2 * 148 && stages >= 2 * x.ns * 2 * W) x.ns *= 2;
  const int warps = base * x.ns <= 148 ? 2 * W : W;
  static_assert(warp_smem<D>() >= 2 * ROWS * (D + 2) * sizeof(float), "the ring holds the warps' results and the CTA's");
  const cudaError_t e = allow_smem<k_xattn_few<D>>(most_warps<D>() * warp_smem<D>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(base * x.ns));
  lc.blockDim = dim3(32 * warps);
  lc.dynamicSmemBytes = warps * warp_smem<D>();
  lc.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)x.ns, 1, 1};
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, k_xattn_few<D>, x);
}

}  // namespace

bool xattn_few_supported(const XDims& d) {
  return (d.d == 64 || d.d == 128) && (long long)d.Tq * d.G <= ROWS && (long long)d.B * d.Hkv <= (1LL << 31) / kMaxCluster - 1;
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
  return d.d == 128 ? launch<128>(x, s) : launch<64>(x, s);
}

}  // namespace vdn
