// Backward of the cross-attention on the tensor cores (tcgen05): bf16 operands,
// fp32 scores, statistics and accumulation.
//
//   P = exp(s q k^T - lse),  Delta = <dO, o>,  dS = P (dO v^T - Delta)
//   dq = s dS K,   dk = s sum_g dS^T q,   dv = sum_g P^T dO     (g: the query heads of a key head)
//
// Two kernels, so that every gradient is summed by one CTA (or by a few whose
// partial sums are joined in a fixed order) and no atomics are needed:
//
//   k_xattn_dq_tc : 128 query rows of a head over its key tiles; three products
//                   a tile (S = Q K^T, dP = dO V^T, dQ += dS K).
//   k_xattn_dkv_tc: 128 states of a key head over the query tiles of its group;
//                   four products a tile (S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q).
//
// Seven products a pair of tiles, against five with one kernel that adds dq
// into memory atomically.  Both are persistent: a CTA on every SM walks its
// items and nothing separates one item from the next; an item's output is
// written inside the next one's first tile, behind its exponentials.
//
// The order on the tensor pipe is set so that it runs while the softmax warps
// work.  dq: the scores are two tiles ahead (two S buffers); after dS(j) the
// pipe has dP(j+1), dQ(j) and S(j+2), while the warps form P(j+1), which needs
// no dP.  dkv: at d = 128 TMEM is full (S, dP, dV, dK), P goes over S and dS
// over dP: after P(j) the pipe has dV(j) and S(j+1), after dS(j) it has dK(j)
// and dP(j+1), which run under the exponentials of P(j+1).  At d = 64 there is
// room for two score tiles, and the scores are two query tiles ahead.
//
// Roles (640 threads): warp 0 TMA producer, warp 1 TMEM allocator and MMA
// issuer, warp 2 the rows' statistics, warps 4..19 softmax: four warps for each
// TMEM lane quadrant (lane = row), each with a quarter of the columns.
//
// Nothing past kv_len is used: dq masks P and dS and zeroes those rows of K in
// shared memory; in dkv they are rows of their own that are stored as zeros.
// Query rows past Tq come as zeros from the tensor map, with a weight of zero.
// Every wait is bounded (see the forward).
#include "tc_common.cuh"
#include "vdn_xattn.h"

namespace vdn {
namespace {
using namespace tc;

constexpr int BR = 128;
constexpr int kThr = 640;
constexpr int kSoftWarps = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSms = 148;

struct XbDev {
  int B, Tq, L, H, Hkv, G;
  int nqt;                  // query tiles
  int ns, per;              // dq: splits of the key tiles; dkv: splits of G nqt query tiles, `per` each
  // dq: splits, heads, query tiles, batch elements; dkv: key tiles, key heads, splits, batch elements.  CTAs that run
  // at the same time so share the tokens: their heads' rows lie side by side in memory
  ItemGrid grid;
  float scale;
  const int* kv_len;
  const float* lse;
  const __nv_bfloat16 *y, *dy;
  float* delta;             // [B, Tq, H]
  __nv_bfloat16 *dq, *dk, *dv;
  float *part, *part2;      // partial sums: dq [ns][B Tq H][D], or dk and dv [ns][B L Hkv][D]; null: none
  uint32_t* status;
  long long wait_limit;     // of the bounded waits, in clock cycles; 0: the default
};

__device__ __forceinline__ int valid_states(const XbDev& x, int b) {
  return x.kv_len == nullptr ? x.L : max(0, min(__ldg(x.kv_len + b), x.L));
}
// the same with b alike in the whole warp, the answer in a uniform register
__device__ __forceinline__ int valid_states_warp(const XbDev& x, int b) {
  return x.kv_len == nullptr ? x.L : __reduce_max_sync(0xffffffffu, valid_states(x, b));
}

// packed bf16 pairs of a 128-column tile: columns [32 h, 32 h + 32) as 16 packed columns from 32 h on
__host__ __device__ constexpr uint32_t pk_k(int k) { return 8u * (k & 1) + 32u * (k >> 1); }

static __device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
static __device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

static __device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// 16 floats as bf16: 32 bytes, a whole sector where the pointer allows it
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* v, float f) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = pack_bf16(v[2 * i] * f, v[2 * i + 1] * f);
  store32(p, u, (reinterpret_cast<uintptr_t>(p) & 31) == 0);
}

// 16 columns of an accumulator row (times f) to a bf16 row or a partial sum
__device__ __forceinline__ void emit16(__nv_bfloat16* o, float* part, long long at, const float (&v)[16], float f) {
  if (part != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4*>(part + at + i) = make_float4(v[i] * f, v[i + 1] * f, v[i + 2] * f, v[i + 3] * f);
  } else {
    store16(o + at, v, f);
  }
}

// D(128 x 128) = A(128 x D) B(128 x D)^T, both K-major in 64-column blocks; by a converged warp, `el` its elected lane
template <int D>
__device__ __forceinline__ void gemm_t(uint32_t dst, uint64_t a, uint64_t b, uint32_t el) {
  constexpr uint32_t ID = idesc_bf16(BR, BR, false);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = (k >> 2) * (BR * 128) + (k & 3) * 32;
    mma_bf16_w(dst, dadd(a, off), dadd(b, off), ID, k > 0 ? 1u : 0u, el);
  }
}
// D(128 x D) (+)= A(TMEM, 128 x 128 packed) B(128 x D, MN-major)
template <int D>
__device__ __forceinline__ void gemm_ts(uint32_t dst, uint32_t a, uint64_t b, bool first, uint32_t el) {
  constexpr uint32_t ID = idesc_bf16(BR, D, true);
#pragma unroll
  for (int k = 0; k < BR / 16; ++k) mma_bf16_ts_w(dst, a + pk_k(k), dadd(b, k * 16 * 128), ID, (first && k == 0) ? 0u : 1u, el);
}

// -------------------------------------------------------------------- dq --
struct QItem {
  int b, h, q0, sp;   // q0: first token of the tile within its batch element
  int k0, nk, nt;     // first state (over all batch elements), valid states, key tiles
};
__device__ __forceinline__ QItem decode_q(const XbDev& x, const ItemPos& p) {
  QItem t;
  t.sp = p.d0;
  t.h = p.d1;
  t.q0 = p.d2 * BR;
  t.b = p.d3;
  const int n = valid_states_warp(x, t.b), all = (n + BR - 1) / BR;
  int lo = 0, hi = all;
  if (x.ns > 1) {
    const int per = (all + x.ns - 1) / x.ns;
    lo = min(t.sp * per, all);
    hi = min(lo + per, all);
  }
  t.nt = hi - lo;
  t.k0 = t.b * x.L + lo * BR;
  t.nk = min(n, hi * BR) - lo * BR;
  return t;
}
// a CTA's key tiles in order, `n` counting them over its items and `i` the items that have any (whole warps)
struct QWalk {
  ItemPos pos;
  int j, n, i;
  bool on;
  QItem it;
  __device__ __forceinline__ void settle(const XbDev& x) {
    for (; pos.on(x.grid); pos.next(x.grid)) {
      it = decode_q(x, pos);
      if (it.nt > 0) return;
    }
    on = false;
  }
  __device__ __forceinline__ void start(const XbDev& x) {
    pos.start(x.grid);
    j = n = i = 0;
    on = true;
    settle(x);
  }
  __device__ __forceinline__ void next(const XbDev& x) {
    ++n;
    if (++j < it.nt) return;
    j = 0;
    ++i;
    pos.next(x.grid);
    settle(x);
  }
  __device__ __forceinline__ bool last() const { return j + 1 == it.nt; }
};

template <int D>
__global__ void __launch_bounds__(kThr, 1)
k_xattn_dq_tc(const XbDev x, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmdo,
              const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  constexpr int NB = D / 64, KST = 3, VST = 2;
  constexpr uint32_t TILE = BR * D * 2;
  constexpr uint32_t COL_S = 0, COL_P = 256, COL_Q = 384;  // S buffers at 0 and 128
  enum { B_QFULL = 0, B_QEMPTY, B_OFULL, B_OEMPTY, B_KFULL, B_KEMPTY = B_KFULL + KST, B_KFIX = B_KEMPTY + KST,
         B_VFULL = B_KFIX + KST, B_VEMPTY = B_VFULL + VST, B_SFULL = B_VEMPTY + VST, B_PFULL = B_SFULL + 2, B_DS, B_ACC,
         B_STFULL, B_STEMPTY, B_DRAIN, NBARS };
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sQ = sm;
  unsigned char* sO = sQ + TILE;
  unsigned char* sK = sO + TILE;
  unsigned char* sV = sK + KST * TILE;
  float2* stat = reinterpret_cast<float2*>(sV + VST * TILE);  // [BR] (-lse in log2 units, -Delta) of the item's rows
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + BR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{abort_flag, x.status, (unsigned)VDN_TAG_XATTN_BWD, x.wait_limit};
  auto bar = [&](int i) { return smem_u32(bars + i); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i) mbar_init(bar(i), i == B_DS || i == B_STEMPTY ? kSoftWarps : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---- producer: Q and dO of an item (dO once its first V is under way), the K and V rings
    // Loads issued, each counted at its own place and before the next wait: after a give-up the counts are what there is to
    // drain (a Q counted only behind the wait for K's stage could still be on its way into a CTA that has ended).
    QWalk w;
    int nq = 0, no = 0, nk = 0, nv = 0;
    for (w.start(x); w.on; w.next(x)) {
      const int sk = w.n % KST, sv = w.n % VST;
      if (w.j == 0) {
        if (w.i > 0 && !mbar_wait_warp(bar(B_QEMPTY), (w.i - 1) & 1, ctl)) break;
        if (lane == 0) {
          mbar_expect_tx(bar(B_QFULL), TILE);
          for (int c = 0; c < NB; ++c) tma_load_4d(smem_u32(sQ + c * BR * 128), &tmq, bar(B_QFULL), c * 64, w.it.h, w.it.q0, w.it.b);
        }
        nq = w.i + 1;
      }
      if (w.n >= KST && !mbar_wait_warp(bar(B_KEMPTY + sk), (w.n / KST - 1) & 1, ctl)) break;
      if (lane == 0) {
        mbar_expect_tx(bar(B_KFULL + sk), TILE);
        for (int c = 0; c < NB; ++c)
          tma_load_3d(smem_u32(sK + sk * TILE + c * BR * 128), &tmk, bar(B_KFULL + sk), c * 64, w.it.h / x.G, w.it.k0 + w.j * BR);
      }
      nk = w.n + 1;
      if (w.j == 0) {
        if (w.i > 0 && !mbar_wait_warp(bar(B_OEMPTY), (w.i - 1) & 1, ctl)) break;
        if (lane == 0) {
          mbar_expect_tx(bar(B_OFULL), TILE);
          for (int c = 0; c < NB; ++c) tma_load_4d(smem_u32(sO + c * BR * 128), &tmdo, bar(B_OFULL), c * 64, w.it.h, w.it.q0, w.it.b);
        }
        no = w.i + 1;
      }
      if (w.n >= VST && !mbar_wait_warp(bar(B_VEMPTY + sv), (w.n / VST - 1) & 1, ctl)) break;
      if (lane == 0) {
        mbar_expect_tx(bar(B_VFULL + sv), TILE);
        for (int c = 0; c < NB; ++c)
          tma_load_3d(smem_u32(sV + sv * TILE + c * BR * 128), &tmv, bar(B_VFULL + sv), c * 64, w.it.h / x.G, w.it.k0 + w.j * BR);
      }
      nv = w.n + 1;
      const int valid = w.it.nk - w.j * BR;
      if (valid < BR) {  // rows of K past the last state: zeros
        if (!mbar_wait_warp(bar(B_KFULL + sk), (w.n / KST) & 1, ctl)) break;
        for (int c = 0; c < NB; ++c) {
          uint4* base = reinterpret_cast<uint4*>(sK + sk * TILE + c * BR * 128);
          for (int i = valid * 8 + lane; i < BR * 8; i += 32) base[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(bar(B_KFIX + sk));
      }
    }
    if (lane == 0) {
      // what was issued has landed
      if (nq > 0) mbar_drain(bar(B_QFULL), (nq - 1) & 1);
      if (no > 0) mbar_drain(bar(B_OFULL), (no - 1) & 1);
      for (int n = max(nk - KST, 0); n < nk; ++n) mbar_drain(bar(B_KFULL + n % KST), (n / KST) & 1);
      for (int n = max(nv - VST, 0); n < nv; ++n) mbar_drain(bar(B_VFULL + n % VST), (n / VST) & 1);
    }
  } else if (warp == 1) {
    // ---- MMA issuer (the whole warp, converged; one elected lane issues)
    const uint32_t el = elect_one();
    const uint64_t qd = sdesc(smem_u32(sQ), 16, 1024), od = sdesc(smem_u32(sO), 16, 1024);
    const uint64_t kd = sdesc(smem_u32(sK), 16, 1024), vd = sdesc(smem_u32(sV), 16, 1024);
    const uint64_t kmn = sdesc(smem_u32(sK), BR * 128, 1024);  // K as the MN-major B of dQ += dS K
    QWalk ws, wp, w;  // scores, dP, dQ
    ws.start(x);
    wp.start(x);
    w.start(x);
    uint32_t fixes = 0;  // a bit for each K stage: parity of its next hand-over by the producer's zeroing
    auto scores = [&]() -> bool {
      const int sk = ws.n % KST;
      if (ws.j == 0 && !mbar_wait_warp(bar(B_QFULL), ws.i & 1, ctl)) return false;
      if (!mbar_wait_warp(bar(B_KFULL + sk), (ws.n / KST) & 1, ctl)) return false;
      if (ws.it.nk - ws.j * BR < BR) {
        if (!mbar_wait_warp(bar(B_KFIX + sk), (fixes >> sk) & 1, ctl)) return false;
        fixes ^= 1u << sk;
      }
      tc_fence_after();
      gemm_t<D>(tmem + COL_S + 128 * (ws.n & 1), qd, dadd(kd, sk * TILE), el);
      mma_commit_w(bar(B_SFULL + (ws.n & 1)), el);
      if (ws.last()) mma_commit_w(bar(B_QEMPTY), el);
      ws.next(x);
      return true;
    };
    auto dprod = [&]() -> bool {
      const int sv = wp.n % VST;
      if (wp.j == 0 && !mbar_wait_warp(bar(B_OFULL), wp.i & 1, ctl)) return false;
      if (!mbar_wait_warp(bar(B_VFULL + sv), (wp.n / VST) & 1, ctl)) return false;
      tc_fence_after();
      gemm_t<D>(tmem + COL_P, od, dadd(vd, sv * TILE), el);
      mma_commit_w(bar(B_PFULL), el);
      mma_commit_w(bar(B_VEMPTY + sv), el);
      if (wp.last()) mma_commit_w(bar(B_OEMPTY), el);
      wp.next(x);
      return true;
    };
    bool ok = !ws.on || (scores() && dprod() && (!ws.on || scores()));
    for (; ok && w.on; w.next(x)) {
      ok = mbar_wait_warp(bar(B_DS), w.n & 1, ctl);
      if (!ok) break;
      tc_fence_after();
      if (wp.on && !(ok = dprod())) break;
      gemm_ts<D>(tmem + COL_Q, tmem + COL_S + 128 * (w.n & 1), dadd(kmn, (w.n % KST) * TILE), w.j == 0, el);
      mma_commit_w(bar(B_KEMPTY + w.n % KST), el);
      if (w.last()) mma_commit_w(bar(B_ACC), el);
      if (ws.on) ok = scores();  // over the buffer whose dS the product above reads first
    }
    mma_commit_w(bar(B_DRAIN), el);
    mbar_drain(bar(B_DRAIN), 0);
  } else if (warp == 2) {
    // ---- the rows' statistics, an item ahead
    QWalk w;
    for (w.start(x); w.on; w.next(x)) {
      if (w.j > 0) continue;
      const long long row0 = ((long long)w.it.b * x.Tq + w.it.q0) * x.H + w.it.h;
      float2 v[BR / 32];
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) {
        const int r = lane + 32 * i;
        const bool on = w.it.q0 + r < x.Tq;
        v[i].x = on ? __ldg(x.lse + row0 + (long long)r * x.H) * -kLog2e : -INFINITY;  // 2^(s c - inf) = 0: no weight
        v[i].y = on ? -__ldg(x.delta + row0 + (long long)r * x.H) : 0.f;
      }
      if (w.i > 0 && !mbar_wait_warp(bar(B_STEMPTY), (w.i - 1) & 1, ctl)) break;
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) stat[lane + 32 * i] = v[i];
      mbar_arrive_warp(bar(B_STFULL));
    }
  } else if (warp >= 4) {
    // ---- softmax: lane = query row, each of a quadrant's four warps a quarter of the columns
    const int quad = warp & 3, part = (warp - 4) >> 2, row = quad * 32 + lane;
    const uint32_t la = tmem + ((uint32_t)(quad * 32) << 16);
    const float2 c2 = make_float2(x.scale * kLog2e, x.scale * kLog2e);
    bool ok = true, pend = false;
    int n = 0, ni = 0;      // key tiles, items with any
    long long prow = 0;     // the pending output's row
    bool pvalid = false;
    auto emit = [&]() -> bool {  // the pending item's dq, this quarter's columns
      if (!mbar_wait_warp(bar(B_ACC), (ni - 1) & 1, ctl)) return false;
      tc_fence_after();
#pragma unroll
      for (int q = part * (D / 64); q < (part + 1) * (D / 64); ++q) {
        float v[16];
        tmem_ld16(la + COL_Q + 16 * q, v);
        tmem_wait_ld();
        if (pvalid) emit16(x.dq, x.part, prow * D + 16 * q, v, x.scale);
      }
      tc_fence_before();
      return true;
    };
    const long long rows = (long long)x.B * x.Tq * x.H;
    ItemPos pos;
    for (pos.start(x.grid); ok && pos.on(x.grid); pos.next(x.grid)) {
      const QItem it = decode_q(x, pos);
      const bool valid = it.q0 + row < x.Tq;
      const long long orow = ((long long)it.b * x.Tq + it.q0 + row) * x.H + it.h + (x.part != nullptr ? it.sp * rows : 0);
      if (it.nt == 0) {  // no states: dq is zero (a split without states leaves nothing)
        if (valid && x.part == nullptr) {
          float z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.f;
          for (int q = part * (D / 64); q < (part + 1) * (D / 64); ++q) emit16(x.dq, nullptr, orow * D + 16 * q, z, 1.f);
        }
        continue;
      }
      if (!mbar_wait_warp(bar(B_STFULL), ni & 1, ctl)) { ok = false; break; }
      const float2 st = stat[row];
      mbar_arrive_warp(bar(B_STEMPTY));
      const float2 nl2 = make_float2(st.x, st.x), nd2 = make_float2(st.y, st.y);
      for (int j = 0; j < it.nt; ++j, ++n) {
        const uint32_t sb = la + COL_S + 128 * (n & 1) + 32 * part;
        const int kv = it.nk - j * BR - 32 * part;  // valid columns of this quarter
        if (!mbar_wait_warp(bar(B_SFULL + (n & 1)), (n >> 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        float p[32];
        tmem_ld32(sb, p);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 e = fma2(make_float2(p[i], p[i + 1]), c2, nl2);
          p[i] = ex2(e.x);
          p[i + 1] = ex2(e.y);
        }
        if (pend) {
          if (!emit()) { ok = false; break; }
          pend = false;
        }
        if (!mbar_wait_warp(bar(B_PFULL), n & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        float v[32];
        tmem_ld32(la + COL_P + 32 * part, v);
        tmem_wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 d = mul2(make_float2(p[2 * i], p[2 * i + 1]), add2(make_float2(v[2 * i], v[2 * i + 1]), nd2));
          if (kv < 32) {  // selected, not multiplied: what V holds past the last state may be NaN
            d.x = 2 * i < kv ? d.x : 0.f;
            d.y = 2 * i + 1 < kv ? d.y : 0.f;
          }
          pk[i] = pack_bf16(d.x, d.y);
        }
        tmem_st16(sb, pk);  // over this quarter's own scores
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(bar(B_DS));
      }
      if (!ok) break;
      pend = true;
      pvalid = valid;
      prow = orow;
      ++ni;
    }
    if (ok && pend) emit();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, 512);
}

// ------------------------------------------------------------------- dkv --
struct KItem {
  int b, hk, k0, sp;   // k0: first state of the tile within its batch element
  int lo, nt;          // first and number of its query tiles, counted over the group's heads
};
__device__ __forceinline__ KItem decode_k(const XbDev& x, const ItemPos& p) {
  KItem t;
  t.k0 = p.d0 * BR;
  t.hk = p.d1;
  t.sp = p.d2;
  t.b = p.d3;
  const int all = x.G * x.nqt;
  t.lo = min(t.sp * x.per, all);
  t.nt = t.k0 < valid_states_warp(x, t.b) ? min(x.per, all - t.lo) : 0;
  return t;
}
// a CTA's query tiles in order; g and q: head of the group and query tile (whole warps)
struct KWalk {
  ItemPos pos;
  int j, n, i, g, q;
  bool on;
  KItem it;
  __device__ __forceinline__ void settle(const XbDev& x) {
    for (; pos.on(x.grid); pos.next(x.grid)) {
      it = decode_k(x, pos);
      if (it.nt > 0) {
        g = it.lo / x.nqt;
        q = it.lo % x.nqt;
        return;
      }
    }
    on = false;
  }
  __device__ __forceinline__ void start(const XbDev& x) {
    pos.start(x.grid);
    j = n = i = 0;
    on = true;
    settle(x);
  }
  __device__ __forceinline__ void next(const XbDev& x) {
    ++n;
    if (++q == x.nqt) {
      q = 0;
      ++g;
    }
    if (++j < it.nt) return;
    j = 0;
    ++i;
    pos.next(x.grid);
    settle(x);
  }
  __device__ __forceinline__ bool last() const { return j + 1 == it.nt; }
  __device__ __forceinline__ int head(const XbDev& x) const { return it.hk * x.G + g; }
  __device__ __forceinline__ int tok() const { return q * BR; }
};

constexpr int kQst = 3, kOst = 2;
template <int D> constexpr size_t dkv_smem() {
  return (size_t)(2 + kQst + kOst) * BR * D * 2 + 2 * BR * sizeof(float2) + 32 * 8 + 16;
}

template <int D>
__global__ void __launch_bounds__(kThr, 1)
k_xattn_dkv_tc(const XbDev x, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmdo,
               const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  constexpr int NB = D / 64, QST = kQst, OST = kOst;
  constexpr uint32_t TILE = BR * D * 2;
  constexpr bool TWO = D == 64;  // two S buffers, at 0 and 128
  constexpr uint32_t COL_S = 0, COL_P = TWO ? 256 : 128, COL_V = COL_P + 128, COL_K = COL_V + D;
  enum { B_KFULL = 0, B_KEMPTY, B_VFULL, B_VEMPTY, B_QFULL, B_QEMPTY = B_QFULL + QST, B_OFULL = B_QEMPTY + QST,
         B_OEMPTY = B_OFULL + OST, B_STFULL = B_OEMPTY + OST, B_STEMPTY = B_STFULL + 2, B_SFULL = B_STEMPTY + 2, B_P = B_SFULL + 2,
         B_PFULL = B_P + 2, B_DS, B_ACC, B_DRAIN, NBARS };
  // The barriers of S and P go by buffer: with two, a softmax warp may be a query tile ahead of another at P (it is
  // held there by dP, which waits for every warp's dS).
  auto sbuf = [](int n) { return TWO ? n & 1 : 0; };
  auto phase = [](int n) { return (uint32_t)(TWO ? n >> 1 : n) & 1u; };
  // the ring leaves no room for a manual alignment: the swizzled tiles need a base on 1024 bytes, which the check below asserts
  extern __shared__ __align__(1024) unsigned char sm[];
  unsigned char* sK = sm;
  unsigned char* sV = sK + TILE;
  unsigned char* sQ = sV + TILE;
  unsigned char* sO = sQ + QST * TILE;
  float* stat = reinterpret_cast<float*>(sO + OST * TILE);  // [2][2][BR] -lse (log2 units) and -Delta of a tile's query rows
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat + 4 * BR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  if ((smem_u32(sm) & 1023u) != 0) {  // uniform
    if (threadIdx.x == 0) {
      atomicOr(x.status, 1u);
      atomicExch(x.status + 1, (unsigned)VDN_TAG_XATTN_BWD);
    }
    return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{abort_flag, x.status, (unsigned)VDN_TAG_XATTN_BWD, x.wait_limit};
  auto bar = [&](int i) { return smem_u32(bars + i); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i)
      mbar_init(bar(i), i == B_P || i == B_P + 1 || i == B_DS || i == B_STEMPTY || i == B_STEMPTY + 1 ? kSoftWarps : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---- producer: K and V of an item, the Q and dO rings
    KWalk w;
    int nk = 0, nq = 0, nv = 0, no = 0;  // loads issued, counted as in dq's producer
    for (w.start(x); w.on; w.next(x)) {
      const int sq = w.n % QST, so = w.n % OST, h = w.head(x), t0 = w.tok();
      if (w.j == 0) {
        if (w.i > 0 && !mbar_wait_warp(bar(B_KEMPTY), (w.i - 1) & 1, ctl)) break;
        if (lane == 0) {
          mbar_expect_tx(bar(B_KFULL), TILE);
          for (int c = 0; c < NB; ++c)
            tma_load_3d(smem_u32(sK + c * BR * 128), &tmk, bar(B_KFULL), c * 64, w.it.hk, w.it.b * x.L + w.it.k0);
        }
        nk = w.i + 1;
      }
      if (w.n >= QST && !mbar_wait_warp(bar(B_QEMPTY + sq), (w.n / QST - 1) & 1, ctl)) break;
      if (lane == 0) {
        mbar_expect_tx(bar(B_QFULL + sq), TILE);
        for (int c = 0; c < NB; ++c)
          tma_load_4d(smem_u32(sQ + sq * TILE + c * BR * 128), &tmq, bar(B_QFULL + sq), c * 64, h, t0, w.it.b);
      }
      nq = w.n + 1;
      if (w.j == 0) {
        if (w.i > 0 && !mbar_wait_warp(bar(B_VEMPTY), (w.i - 1) & 1, ctl)) break;
        if (lane == 0) {
          mbar_expect_tx(bar(B_VFULL), TILE);
          for (int c = 0; c < NB; ++c)
            tma_load_3d(smem_u32(sV + c * BR * 128), &tmv, bar(B_VFULL), c * 64, w.it.hk, w.it.b * x.L + w.it.k0);
        }
        nv = w.i + 1;
      }
      if (w.n >= OST && !mbar_wait_warp(bar(B_OEMPTY + so), (w.n / OST - 1) & 1, ctl)) break;
      if (lane == 0) {
        mbar_expect_tx(bar(B_OFULL + so), TILE);
        for (int c = 0; c < NB; ++c)
          tma_load_4d(smem_u32(sO + so * TILE + c * BR * 128), &tmdo, bar(B_OFULL + so), c * 64, h, t0, w.it.b);
      }
      no = w.n + 1;
    }
    if (lane == 0) {
      if (nk > 0) mbar_drain(bar(B_KFULL), (nk - 1) & 1);
      if (nv > 0) mbar_drain(bar(B_VFULL), (nv - 1) & 1);
      for (int n = max(nq - QST, 0); n < nq; ++n) mbar_drain(bar(B_QFULL + n % QST), (n / QST) & 1);
      for (int n = max(no - OST, 0); n < no; ++n) mbar_drain(bar(B_OFULL + n % OST), (n / OST) & 1);
    }
  } else if (warp == 1) {
    // ---- MMA issuer
    const uint32_t el = elect_one();
    const uint64_t kd = sdesc(smem_u32(sK), 16, 1024), vd = sdesc(smem_u32(sV), 16, 1024);
    const uint64_t qd = sdesc(smem_u32(sQ), 16, 1024), od = sdesc(smem_u32(sO), 16, 1024);
    const uint64_t qmn = sdesc(smem_u32(sQ), BR * 128, 1024), omn = sdesc(smem_u32(sO), BR * 128, 1024);
    KWalk ws, wp, w;
    ws.start(x);
    wp.start(x);
    w.start(x);
    auto scores = [&]() -> bool {  // S^T = K Q^T
      const int sq = ws.n % QST;
      if (ws.j == 0 && !mbar_wait_warp(bar(B_KFULL), ws.i & 1, ctl)) return false;
      if (!mbar_wait_warp(bar(B_QFULL + sq), (ws.n / QST) & 1, ctl)) return false;
      tc_fence_after();
      gemm_t<D>(tmem + COL_S + 128 * sbuf(ws.n), kd, dadd(qd, sq * TILE), el);
      mma_commit_w(bar(B_SFULL + sbuf(ws.n)), el);
      if (ws.last()) mma_commit_w(bar(B_KEMPTY), el);
      ws.next(x);
      return true;
    };
    auto dprod = [&]() -> bool {  // dP^T = V dO^T
      const int so = wp.n % OST;
      if (wp.j == 0 && !mbar_wait_warp(bar(B_VFULL), wp.i & 1, ctl)) return false;
      if (!mbar_wait_warp(bar(B_OFULL + so), (wp.n / OST) & 1, ctl)) return false;
      tc_fence_after();
      gemm_t<D>(tmem + COL_P, vd, dadd(od, so * TILE), el);
      mma_commit_w(bar(B_PFULL), el);
      if (wp.last()) mma_commit_w(bar(B_VEMPTY), el);
      wp.next(x);
      return true;
    };
    bool ok = !ws.on || (scores() && dprod() && (!TWO || !ws.on || scores()));
    for (; ok && w.on; w.next(x)) {
      ok = mbar_wait_warp(bar(B_P + sbuf(w.n)), phase(w.n), ctl);
      if (!ok) break;
      tc_fence_after();
      gemm_ts<D>(tmem + COL_V, tmem + COL_S + 128 * sbuf(w.n), dadd(omn, (w.n % OST) * TILE), w.j == 0, el);  // dV += P^T dO
      mma_commit_w(bar(B_OEMPTY + w.n % OST), el);
      if (ws.on && !(ok = scores())) break;  // over P^T, which the product above reads first
      ok = mbar_wait_warp(bar(B_DS), w.n & 1, ctl);
      if (!ok) break;
      tc_fence_after();
      gemm_ts<D>(tmem + COL_K, tmem + COL_P, dadd(qmn, (w.n % QST) * TILE), w.j == 0, el);  // dK += dS^T Q
      mma_commit_w(bar(B_QEMPTY + w.n % QST), el);
      if (w.last()) mma_commit_w(bar(B_ACC), el);
      if (wp.on) ok = dprod();
    }
    mma_commit_w(bar(B_DRAIN), el);
    mbar_drain(bar(B_DRAIN), 0);
  } else if (warp == 2) {
    // ---- the query rows' statistics, two tiles ahead
    KWalk w;
    for (w.start(x); w.on; w.next(x)) {
      const int s = w.n & 1, t0 = w.tok();
      const long long row0 = ((long long)w.it.b * x.Tq + t0) * x.H + w.head(x);
      float2 v[BR / 32];
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) {
        const int r = lane + 32 * i;
        const bool on = t0 + r < x.Tq;
        v[i].x = on ? __ldg(x.lse + row0 + (long long)r * x.H) * -kLog2e : -INFINITY;  // 2^(s c - inf) = 0: no weight
        v[i].y = on ? -__ldg(x.delta + row0 + (long long)r * x.H) : 0.f;
      }
      if (w.n >= 2 && !__all_sync(0xffffffffu, mbar_wait(bar(B_STEMPTY + s), (w.n / 2 - 1) & 1, ctl))) break;
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) {
        stat[2 * s * BR + lane + 32 * i] = v[i].x;
        stat[(2 * s + 1) * BR + lane + 32 * i] = v[i].y;
      }
      mbar_arrive_warp(bar(B_STFULL + s));
    }
  } else if (warp >= 4) {
    // ---- softmax: lane = state, each of a quadrant's four warps a quarter of the columns (query rows)
    const int quad = warp & 3, part = (warp - 4) >> 2, row = quad * 32 + lane;
    const uint32_t la = tmem + ((uint32_t)(quad * 32) << 16);
    const float2 c2 = make_float2(x.scale * kLog2e, x.scale * kLog2e);
    bool ok = true, pend = false, pin = false, plive = false;
    int n = 0, ni = 0;
    long long prow = 0;  // the pending output's row; pin: inside L; plive: inside kv_len
    auto emit = [&]() -> bool {
      if (!mbar_wait_warp(bar(B_ACC), (ni - 1) & 1, ctl)) return false;
      tc_fence_after();
#pragma unroll
      for (int q = part * (D / 64); q < (part + 1) * (D / 64); ++q) {
        float v[16], u[16];
        tmem_ld16(la + COL_V + 16 * q, v);
        tmem_ld16(la + COL_K + 16 * q, u);
        tmem_wait_ld();
        if (!plive) {  // selected: a row past the last state may hold NaN
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = u[i] = 0.f;
        }
        if (pin) {
          emit16(x.dv, x.part2, prow * D + 16 * q, v, 1.f);
          emit16(x.dk, x.part, prow * D + 16 * q, u, x.scale);
        }
      }
      tc_fence_before();
      return true;
    };
    const long long rows = (long long)x.B * x.L * x.Hkv;
    ItemPos pos;
    for (pos.start(x.grid); ok && pos.on(x.grid); pos.next(x.grid)) {
      const KItem it = decode_k(x, pos);
      const bool in = it.k0 + row < x.L, live = it.k0 + row < valid_states_warp(x, it.b);
      const long long orow = ((long long)it.b * x.L + it.k0 + row) * x.Hkv + it.hk + (x.part != nullptr ? it.sp * rows : 0);
      if (it.nt == 0) {  // past the last state: zeros (which the join writes where there are partial sums)
        if (in && x.part == nullptr) {
          float z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.f;
          for (int q = part * (D / 64); q < (part + 1) * (D / 64); ++q) {
            emit16(x.dv, nullptr, orow * D + 16 * q, z, 1.f);
            emit16(x.dk, nullptr, orow * D + 16 * q, z, 1.f);
          }
        }
        continue;
      }
      for (int j = 0; j < it.nt; ++j, ++n) {
        const float4* nl = reinterpret_cast<const float4*>(stat + 2 * (n & 1) * BR + 32 * part);
        const float4* nd = nl + BR / 4;
        const uint32_t sb = la + COL_S + 128 * sbuf(n) + 32 * part;
        if (!mbar_wait_warp(bar(B_STFULL + (n & 1)), (n >> 1) & 1, ctl) ||
            !mbar_wait_warp(bar(B_SFULL + sbuf(n)), phase(n), ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float p[32];
        uint32_t pk[16];
        tmem_ld32(sb, p);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 l = nl[i / 4];
          const float2 e = fma2(make_float2(p[i], p[i + 1]), c2, make_float2(l.x, l.y));
          const float2 f = fma2(make_float2(p[i + 2], p[i + 3]), c2, make_float2(l.z, l.w));
          p[i] = ex2(e.x);
          p[i + 1] = ex2(e.y);
          p[i + 2] = ex2(f.x);
          p[i + 3] = ex2(f.y);
          pk[i / 2] = pack_bf16(p[i], p[i + 1]);
          pk[i / 2 + 1] = pack_bf16(p[i + 2], p[i + 3]);
        }
        if (pend) {
          if (!emit()) { ok = false; break; }
          pend = false;
        }
        tmem_st16(sb, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(bar(B_P + sbuf(n)));
        if (!mbar_wait_warp(bar(B_PFULL), n & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        float v[32];
        tmem_ld32(la + COL_P + 32 * part, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 d = nd[i / 4];
          const float2 e = mul2(make_float2(p[i], p[i + 1]), add2(make_float2(v[i], v[i + 1]), make_float2(d.x, d.y)));
          const float2 f = mul2(make_float2(p[i + 2], p[i + 3]), add2(make_float2(v[i + 2], v[i + 3]), make_float2(d.z, d.w)));
          pk[i / 2] = pack_bf16(e.x, e.y);
          pk[i / 2 + 1] = pack_bf16(f.x, f.y);
        }
        tmem_st16(la + COL_P + 32 * part, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(bar(B_DS));
        mbar_arrive_warp(bar(B_STEMPTY + (n & 1)));
      }
      if (!ok) break;
      pend = true;
      pin = in;
      plive = live;
      prow = orow;
      ++ni;
    }
    if (ok && pend) emit();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, 512);
}

// ----------------------------------------------------------------- Delta --
// <dO, o> of every query row: 16 bytes a lane, D / 8 lanes a row, coalesced over rows that follow one another.
// (Formed by two warps of the dq kernel instead, it held that kernel back: 1,171 against 1,040 us with both kernels at
// 90,720 x 24 rows.)
template <int D>
__global__ void __launch_bounds__(256) k_xattn_delta_bf16(const XbDev x, long long rows) {
  constexpr int LR = D / 8, U = 4;  // U rows a thread, loads first
  clear_status(x.status);
  const long long base = (long long)blockIdx.x * (256 / LR) * U + threadIdx.x / LR;
  const int li = threadIdx.x % LR;
  uint4 a[U], g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = min(base + u * (256 / LR), rows - 1);
    a[u] = __ldg(reinterpret_cast<const uint4*>(x.y + row * D) + li);
    g[u] = __ldg(reinterpret_cast<const uint4*>(x.dy + row * D) + li);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t av[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, gv[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(av[i] << 16), __uint_as_float(gv[i] << 16), s);
      s = fmaf(__uint_as_float(av[i] & 0xFFFF0000u), __uint_as_float(gv[i] & 0xFFFF0000u), s);
    }
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const long long row = base + u * (256 / LR);
    if (li == 0 && row < rows) x.delta[row] = s;
  }
}

// --------------------------------------------------------- joining splits --
// Sums of the partial results in the order of the splits, four columns a thread.
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ void join4(const float* part, long long i4, long long n4, int parts, __nv_bfloat16* o) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < parts; ++p) s = add4(s, __ldg(reinterpret_cast<const float4*>(part) + p * n4 + i4));
  reinterpret_cast<uint2*>(o)[i4] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}
__global__ void __launch_bounds__(256) k_xattn_join_dq(const XbDev x, int D) {
  const long long n4 = (long long)x.B * x.Tq * x.H * D / 4, i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const int b = (int)(i / (n4 / x.B)), all = (valid_states(x, b) + BR - 1) / BR, per = (all + x.ns - 1) / x.ns;
  join4(x.part, i, n4, all == 0 ? 0 : (all + per - 1) / per, x.dq);
}
__global__ void __launch_bounds__(256) k_xattn_join_dkv(const XbDev x, int D) {
  const long long n4 = (long long)x.B * x.L * x.Hkv * D / 4, i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const long long tok = i / ((long long)x.Hkv * D / 4);
  const int parts = (int)(tok % x.L) < valid_states(x, (int)(tok / x.L)) ? x.ns : 0;
  join4(x.part, i, n4, parts, x.dk);
  join4(x.part2, i, n4, parts, x.dv);
}

// ------------------------------------------------------------------- host --
// Splits of `steps` tiles a base item: the number that ends first on kSms CTAs,
// an item costing `head` steps beside its own, and partial sums two more in all.
int choose_split(long long base, int steps, double head, int most) {
  int best = 1;
  double cost = 0;
  for (int ns = 1; ns <= steps && ns <= most; ++ns) {
    if (ns > 1 && base * ns > 4 * kSms) break;
    const int per = (steps + ns - 1) / ns;
    const double t = (double)((base * ns + kSms - 1) / kSms) * (per + head) + (ns > 1 ? 2.0 : 0.0);
    if (ns == 1 || t < cost) {
      cost = t;
      best = ns;
    }
  }
  return best;
}

struct BwdCut {
  int nqt, nkt, qs, ks, kper;
  size_t delta, dq, dk, bytes;  // offsets of Delta's end: partial dq, partial dk, partial dv
};
BwdCut bwd_cut(const XDims& d) {
  BwdCut c;
  c.nqt = (d.Tq + BR - 1) / BR;
  c.nkt = (d.L + BR - 1) / BR;
  c.qs = choose_split((long long)d.B * d.H * c.nqt, c.nkt, 1.0, 64);
  const int steps = d.G * c.nqt;
  c.ks = choose_split((long long)d.B * d.Hkv * c.nkt, steps, 3.0, 64);
  c.kper = (steps + c.ks - 1) / c.ks;
  c.ks = (steps + c.kper - 1) / c.kper;  // no empty split
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t rows = (size_t)d.B * d.Tq * d.H, krows = (size_t)d.B * d.L * d.Hkv;
  c.delta = 0;
  c.dq = up(rows * sizeof(float));
  const size_t dqb = c.qs > 1 ? up((size_t)c.qs * rows * d.d * sizeof(float)) : 0;
  const size_t kb = c.ks > 1 ? up((size_t)c.ks * krows * d.d * sizeof(float)) : 0;
  c.dk = c.dq + dqb;
  c.bytes = c.dk + 2 * kb;
  return c;
}

// 4-D map over [B][tokens][H][D] bf16: 64 dims x 1 head x 128 tokens of one batch element, zeros past its last token
bool make_batch_map(CUtensorMap* m, const void* base, int B, int T, int H, int D) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)T * H * D * 2};
  cuuint32_t box[4] = {64, 1, BR, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const XDims& d, const XArgs& a, cudaStream_t s) {
  const BwdCut c = bwd_cut(d);
  CUtensorMap mq, mo, mk, mv;
  if (!make_batch_map(&mq, a.q, d.B, d.Tq, d.H, D) || !make_batch_map(&mo, a.dy, d.B, d.Tq, d.H, D) ||
      !make_token_map_strided(&mk, a.k, (long long)d.B * d.L, d.Hkv, D, d.ks, 1, BR) ||
      !make_token_map_strided(&mv, a.v, (long long)d.B * d.L, d.Hkv, D, d.vs, 1, BR))
    return cudaErrorInvalidValue;
  char* ws = static_cast<char*>(a.scratch);
  XbDev x{};
  x.B = d.B; x.Tq = d.Tq; x.L = d.L; x.H = d.H; x.Hkv = d.Hkv; x.G = d.G;
  x.nqt = c.nqt;
  x.scale = d.scale;
  x.kv_len = d.kv_len;
  x.lse = a.lse;
  x.y = static_cast<const __nv_bfloat16*>(a.y);
  x.dy = static_cast<const __nv_bfloat16*>(a.dy);
  x.delta = reinterpret_cast<float*>(ws + c.delta);
  x.dq = static_cast<__nv_bfloat16*>(a.dq);
  x.dk = static_cast<__nv_bfloat16*>(a.dk);
  x.dv = static_cast<__nv_bfloat16*>(a.dv);
  x.status = a.status;
  x.wait_limit = a.wait_limit;
  const long long qi = (long long)d.B * d.H * c.nqt * c.qs, ki = (long long)d.B * d.Hkv * c.nkt * c.ks;
  if (qi > 0x7FFFFFFFLL || ki > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const size_t smq = 1024 + (size_t)7 * BR * D * 2 + BR * sizeof(float2) + 32 * 8 + 16, smk = dkv_smem<D>();
  cudaError_t e = allow_smem<k_xattn_dq_tc<D>>(smq);
  if (e != cudaSuccess) return e;
  if ((e = allow_smem<k_xattn_dkv_tc<D>>(smk)) != cudaSuccess) return e;
  const long long rows = (long long)d.B * d.Tq * d.H, per = 256 / (D / 8) * 4;
  k_xattn_delta_bf16<D><<<(unsigned)((rows + per - 1) / per), 256, 0, s>>>(x, rows);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  XbDev xq = x;
  xq.ns = c.qs;
  const int qgrid = (int)(qi < kSms ? qi : kSms), kgrid = (int)(ki < kSms ? ki : kSms);
  xq.grid = item_grid((int)qi, c.qs, d.H, c.nqt, qgrid);
  xq.part = c.qs > 1 ? reinterpret_cast<float*>(ws + c.dq) : nullptr;
  k_xattn_dq_tc<D><<<qgrid, kThr, smq, s>>>(xq, mq, mo, mk, mv);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  XbDev xk = x;
  xk.ns = c.ks;
  xk.per = c.kper;
  xk.grid = item_grid((int)ki, c.nkt, d.Hkv, c.ks, kgrid);
  if (c.ks > 1) {
    xk.part = reinterpret_cast<float*>(ws + c.dk);
    xk.part2 = reinterpret_cast<float*>(ws + c.dk + (c.bytes - c.dk) / 2);
  }
  k_xattn_dkv_tc<D><<<kgrid, kThr, smk, s>>>(xk, mq, mo, mk, mv);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (c.qs > 1) {
    k_xattn_join_dq<<<(unsigned)(((long long)d.B * d.Tq * d.H * D / 4 + 255) / 256), 256, 0, s>>>(xq, D);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (c.ks > 1) {
    k_xattn_join_dkv<<<(unsigned)(((long long)d.B * d.L * d.Hkv * D / 4 + 255) / 256), 256, 0, s>>>(xk, D);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

size_t xattn_tc_bwd_scratch(const XDims& d) { return bwd_cut(d).bytes; }

cudaError_t launch_xattn_tc_bwd(const XDims& d, const XArgs& a, cudaStream_t s) {
  return d.d == 128 ? launch<128>(d, a, s) : launch<64>(d, a, s);
}

}  // namespace vdn
