// Cross-attention for few query rows (a token of a stream, a short draft): all
// rows that share a key head, up to 16, against its states.  bf16 in and out,
// fp32 scores, softmax and accumulation.
//
// Bound by the read of k and v, once.  The states of a key head are split over
// a cluster of up to 8 CTAs and over their warps.  A warp takes 16 states at a
// time from a ring of its own in shared memory (cp.async, so that the next
// ones are on their way; no block barrier), forms the scores of 8 or 16 rows and
// adds P V with warp-level matrix products, and keeps a running reference, sum
// and output.  Both products have the states or columns as their 16 rows and
// the query rows as their 8 columns (S^T = K q^T, O^T = V^T P^T), which is the
// finest step in query rows there is: with the query rows as the 16 rows of
// the result it took 28 us where this takes 20.5 (one token of 8 requests over
// 1,408 to 4,096 states, 24 / 8 heads, d = 128), and the tcgen05 kernel with its
// tiles of 128 rows 45.8 a call.
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
constexpr float kSlack = 8.f;
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
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {  // off: 16 bytes of zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
// four 8 x 8 blocks of 16-bit values, lane l giving the address of row l % 8 of block l / 8
__device__ __forceinline__ void blocks4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// the same transposed, blocks 1 and 2 swapped
__device__ __forceinline__ void blocks4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[2]), "=r"(r[1]), "=r"(r[3]) : "r"(addr) : "memory");
}
// the transpose of an 8 x 8 block spread over the warp as a result is
__device__ __forceinline__ uint32_t turned(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
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

// NB: blocks of 8 query rows
template <int D, int NB>
__global__ void __launch_bounds__(32 * most_warps<D>()) k_xattn_few(const XfDev x) {
  constexpr int CPR = D / 8, KPI = 32 / CPR;  // chunks of a row, rows a warp copies at once
  constexpr int TURN = 8 / KPI;               // copies until the rows' places repeat
  constexpr uint32_t ROW = CPR * 16, HALF = KT * ROW, STAGE = 2 * HALF;
  extern __shared__ uint4 ring[];
  clear_status(x.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int g = lane >> 2, t2 = 2 * (lane & 3);  // of a 16 x 8 result: rows g and g + 8, columns t2 and t2 + 1
  const int rank = blockIdx.x % x.ns, bh = blockIdx.x / x.ns, Hkv = x.H / x.G, b = bh / Hkv, hk = bh % Hkv;
  int n = x.L;
  if (x.kv_len != nullptr) n = max(0, min(__ldg(x.kv_len + b), x.L));
  // this CTA's states, in whole stages
  const int all = (n + KT - 1) / KT, per = (all + x.ns - 1) / x.ns, lo = min(rank * per, all), hi = min(lo + per, all);
  const uint32_t mine = smem_addr(ring) + warp * NS * STAGE;
  const int ck = lane % CPR, rk = lane / CPR;  // the chunk and the first row that this lane copies
  int it = lo + warp, next = it;               // the stage worked on, and the one to copy
  const long long first = (long long)b * x.L + (long long)it * KT + rk, kstep = KPI * x.ks * 2, vstep = KPI * x.vs * 2;
  const char* kp = reinterpret_cast<const char*>(x.k + first * x.ks + hk * D + 8 * ck);
  const char* vp = reinterpret_cast<const char*>(x.v + first * x.vs + hk * D + 8 * ck);
  // chunk c of row r lies at c ^ (r % 8): the eight rows of a block in eight different groups of banks
  uint32_t to[TURN], from[4];
#pragma unroll
  for (int i = 0; i < TURN; ++i) to[i] = (rk + i * KPI) * ROW + (ck ^ ((rk + i * KPI) & 7)) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) from[i] = (lane & 15) * ROW + ((2 * i + (lane >> 4)) ^ (lane & 7)) * 16;
  auto fetch = [&](uint32_t base) {
    const char *ka = kp, *va = vp;
    if (next < hi && next * KT + KT <= n) {
#pragma unroll
      for (int i = 0; i < KT / KPI; ++i, ka += kstep, va += vstep) {
        const uint32_t dst = base + to[i % TURN] + i / TURN * 8 * ROW;
        copy16(dst, ka);
        copy16(dst + HALF, va);
      }
    } else if (next < hi) {  // the last stage: rows past the length are zeros
#pragma unroll
      for (int i = 0; i < KT / KPI; ++i, ka += kstep, va += vstep) {
        const uint32_t dst = base + to[i % TURN] + i / TURN * 8 * ROW;
        const bool on = next * KT + rk + i * KPI < n;
        copy16(dst, on ? ka : reinterpret_cast<const char*>(x.k), on);
        copy16(dst + HALF, on ? va : reinterpret_cast<const char*>(x.v), on);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += nw;
    kp += nw * (KT / KPI) * kstep;
    vp += nw * (KT / KPI) * vstep;
  };
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) fetch(mine + s * STAGE);
  // the query rows as right operands: row g of a block, columns t2 and t2 + 8 of every 16
  uint32_t qb[NB][D / 16][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = g + 8 * nb;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(x.q + (((long long)b * x.Tq + r / x.G) * x.H + hk * x.G + r % x.G) * D + t2);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      qb[nb][i][0] = r < x.rows ? __ldg(p + 8 * i) : 0u;
      qb[nb][i][1] = r < x.rows ? __ldg(p + 8 * i + 4) : 0u;
    }
  }
  // of rows t2 and t2 + 1 of a block: the output's columns, the reference (log2 units) and this lane's part of the sum
  float o[NB][D / 16][4], m[NB][2], l[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
  }
  const float c = x.scale * kLog2e;
  uint32_t sk = mine, fill = mine + (NS - 1) * STAGE;
#pragma unroll 1
  for (; it < hi; it += nw) {
    __syncwarp();  // the stage filled next was read by every lane
    fetch(fill);
    fill = fill == mine + (NS - 1) * STAGE ? mine : fill + STAGE;
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
    __syncwarp();
    // scores of 16 states, two chains
    float s[NB][2][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nb][0][e] = s[nb][1][e] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      blocks4(a, sk + from[i % 4] + i / 4 * 128);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16(s[nb][i & 1], a, qb[nb][i][0], qb[nb][i][1]);
    }
    bool above = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[nb][0][e] = (s[nb][0][e] + s[nb][1][e]) * c;
        if (it * KT + KT > n && it * KT + g + 8 * (e >> 1) >= n) s[nb][0][e] = -INFINITY;
        above |= s[nb][0][e] > m[nb][e & 1] + kSlack;
      }
    // The reference moves only once a score exceeds it by 2^8: weights up to 2^8 lose nothing, and the maximum over the
    // lanes and the rescaling of the output stay out of most stages.
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[nb][0][e], s[nb][0][e + 2]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          mx = fmaxf(mx, m[nb][e]);
          f[e] = mx == -INFINITY ? 1.f : ex2(m[nb][e] - mx);
          m[nb][e] = mx;
          l[nb][e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[nb][i][0] *= f[0];
          o[nb][i][1] *= f[1];
          o[nb][i][2] *= f[0];
          o[nb][i][3] *= f[1];
        }
      }
    }
    uint32_t pb[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // no score above -inf so far: weights of 0 and not of inf - inf
        const float ref = m[nb][e & 1] == -INFINITY ? 0.f : m[nb][e & 1];
        z[e] = ex2(s[nb][0][e] - ref);
      }
      l[nb][0] += z[0] + z[2];
      l[nb][1] += z[1] + z[3];
      pb[nb][0] = turned(pack_bf16(z[0], z[1]));  // the product's operand type; l adds the unrounded weights
      pb[nb][1] = turned(pack_bf16(z[2], z[3]));
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      blocks4_t(a, sk + HALF + from[i % 4] + i / 4 * 128);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16(o[nb][i], a, pb[nb][0], pb[nb][1]);
    }
    sk = sk == mine + (NS - 1) * STAGE ? mine : sk + STAGE;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // the warps' results in shared memory: [warp][rows][D + 2] = o, m, l; then the CTA's, [rows][D + 2] behind them
  __syncthreads();
  constexpr int RW = D + 2;
  float* res = reinterpret_cast<float*>(ring);
  float* cta = res + nw * x.rows * RW;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], d);
      const int r = 8 * nb + t2 + e;
      if (r < x.rows) {
        float* p = res + (warp * x.rows + r) * RW;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          p[16 * i + g] = o[nb][i][e];
          p[16 * i + 8 + g] = o[nb][i][e + 2];
        }
        if (g == 0) {
          p[D] = m[nb][e];
          p[D + 1] = l[nb][e];
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

template <int D, int NB>
cudaError_t launch(XfDev x, cudaStream_t s) {
  // A ring of 24 KB (d = 128) a warp: two CTAs of 4 warps on an SM, or one of 8.  The states are split over as many CTAs
  // as still run at once, while a warp has two stages or more.  CTAs of 8 warps only up to 96 of them: a cluster of 8 needs
  // 8 free SMs of one GPC then, and 16 clusters do not all fit at once (2 requests over 4,096 states: 16.0 us, with 4
  // warps 12.1); 12 still do (11.0 us, with 4 warps 11.6), and one request takes 9.7 us (10.4).
  constexpr int W = most_warps<D>() / 2;
  const long long base = (long long)x.B * (x.H / x.G);
  const int stages = (x.L + KT - 1) / KT;
  x.ns = 1;
  while (x.ns < kMaxCluster && base * 2 * x.ns <= 2 * 148 && stages >= 2 * x.ns * 2 * W) x.ns *= 2;
  const int warps = base * x.ns <= 96 ? 2 * W : W;
  static_assert(warp_smem<D>() >= 2 * ROWS * (D + 2) * sizeof(float), "the ring holds the warps' results and the CTA's");
  const cudaError_t e = allow_smem<k_xattn_few<D, NB>>(most_warps<D>() * warp_smem<D>());
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
  return cudaLaunchKernelEx(&lc, k_xattn_few<D, NB>, x);
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
  if (x.rows > 8) return d.d == 128 ? launch<128, 2>(x, s) : launch<64, 2>(x, s);
  return d.d == 128 ? launch<128, 1>(x, s) : launch<64, 1>(x, s);
}

}  // namespace vdn
