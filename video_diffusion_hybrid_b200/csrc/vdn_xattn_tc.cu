// Cross-attention to an encoder's states on the tensor cores (tcgen05): bf16 q,
// k, v, fp32 scores, softmax and accumulation.
//
//   o = softmax(s q K^T) V over the first kv_len[b] states, lse = ln sum_j exp(s q k_j)
//
// The work is cut into items: two tiles of up to 128 query rows of one batch
// element and head, against a run of key tiles of 128 states.  A persistent
// CTA on every SM walks its items, and all roles run on from one item to the
// next without a barrier between them: while the softmax warps write one
// item's output, the next item's scores are computed and its tiles loaded.
// (One CTA for each item, with its own prologue and epilogue, left the tensor
// cores idle for half of the time at four key tiles an item.)
//
//  - Heads that share a key head can share a tile: a row is (token, head of the
//    group), token-major, one TMA box; it is done where it gives fewer items.
//  - Few items: the key tiles of an item are split over several CTAs, partial
//    outputs and log-sum-exps go to the workspace in fp32 and a second kernel
//    joins them in a fixed order.
//
// Roles (384 threads): warp 0 K producer (TMA, three stages), warp 1 TMEM
// allocator and MMA issuer, warp 2 V producer (two stages; it zeroes the rows
// past the last valid state, whose weight is zero but whose content may be
// NaN), warp 3 Q producer, warps 4..7 and 8..11 the softmax of tile 0 and 1
// (thread = TMEM lane = row).  On the tensor pipe, for every key tile,
//   O_0 += P_0 V, S_0 = Q_0 K_next^T, O_1 += P_1 V, S_1 = Q_1 K_next^T
// so that one tile's softmax runs while the other's products do.
//
// The softmax takes a key tile in two halves of 64 states and keeps a row's
// reference m while no weight exceeds 2^8 (checked by the half's sum), so O is
// rescaled only when the maximum grew by more than 8 in exp2 units.  P is
// rounded to bf16 for the product (the operand's type: a relative 2^-8 at most
// of each weight); the row sum adds the unrounded values in fp32.
//
// TMEM (512 columns): O_0 [0,128), O_1 [128,256), S_0 [256,384), S_1 [384,512);
// P_t over the first 64 columns of S_t.  One thread issues every product, in
// order, so P_t(j) is read before S_t(j+1) overwrites it; the first product of
// an item into O_t waits for P_t, which the softmax warps hand over only
// after they read the previous item's O_t.
//
// Every wait is bounded: on expiry the CTA records the timeout, stops issuing,
// drains its copies and products and frees its TMEM.
#include "tc_common.cuh"
#include "vdn_xattn.h"

namespace vdn {
namespace {
using namespace tc;

constexpr int BM = 128;  // rows of a query tile
constexpr int BN = 128;  // states of a key tile
constexpr int kThr = 384;
constexpr int KST = 3, VST = 2;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

__host__ __device__ constexpr uint32_t col_o(int t) { return 128u * t; }
__host__ __device__ constexpr uint32_t col_s(int t) { return 256u + 128u * t; }

struct XtDev {
  int B, Tq, L, H, G;
  int P, TT;           // heads and tokens of a tile (P TT <= 128 rows)
  int ns;              // splits of the states
  ItemGrid grid;       // splits, head groups, tile pairs over the tokens, batch elements: CTAs that run at the
                       // same time share the tokens, and their heads' rows lie side by side in memory
  float scale;
  const int* kv_len;
  __nv_bfloat16* y;
  float* lse;          // or null
  float *po, *pl;      // partial outputs [parts][B Tq H][D] and log-sum-exps (log2 units), or null
  long long rows;      // B Tq H
  uint32_t* status;
  long long wait_limit;  // of the bounded waits, in clock cycles; 0: the default
};

struct Item {
  int b, hg, q0;       // q0: first query token (over all batch elements)
  int left;            // query tokens of the batch element from q0 on
  int k0, nk, nt;      // first state (over all batch elements), valid states, key tiles
  int sp;
};

// the same for every lane (and known to be: the reduction's result is a uniform register)
__device__ __forceinline__ int valid_states(const XtDev& x, int b) {
  if (x.kv_len == nullptr) return x.L;
  return __reduce_max_sync(0xffffffffu, max(0, min(__ldg(x.kv_len + b), x.L)));
}

// call with the whole warp
__device__ __forceinline__ Item decode(const XtDev& x, const ItemPos& p) {
  Item t;
  t.sp = p.d0;
  t.hg = p.d1;
  t.b = p.d3;
  const int first = p.d2 * 2 * x.TT;
  t.q0 = t.b * x.Tq + first;
  t.left = x.Tq - first;
  const int n = valid_states(x, t.b), all = (n + BN - 1) / BN;
  int lo = 0, hi = all;
  if (x.ns > 1) {
    const int per = (all + x.ns - 1) / x.ns;
    lo = min(t.sp * per, all);
    hi = min(lo + per, all);
  }
  t.nt = hi - lo;
  t.k0 = t.b * x.L + lo * BN;
  t.nk = min(n, hi * BN) - lo * BN;
  return t;
}
// tile t has rows in this item
__device__ __forceinline__ bool has_rows(const XtDev& x, const Item& it, int t) { return t == 0 || it.left > x.TT; }

// A CTA's key tiles in order; `n` counts them over all items (its ring position).
struct Walk {
  ItemPos pos;
  int j, n;
  bool on;
  Item it;
  __device__ __forceinline__ void settle(const XtDev& x) {  // the first item from here on that has key tiles
    for (; pos.on(x.grid); pos.next(x.grid)) {
      it = decode(x, pos);
      if (it.nt > 0) return;
    }
    on = false;
  }
  __device__ __forceinline__ void start(const XtDev& x) {
    pos.start(x.grid);
    j = n = 0;
    on = true;
    settle(x);
  }
  __device__ __forceinline__ void next(const XtDev& x) {
    ++n;
    if (++j < it.nt) return;
    j = 0;
    pos.next(x.grid);
    settle(x);
  }
};

template <int D>
__global__ void __launch_bounds__(kThr, 1)
k_xattn_tc(const XtDev x, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
           const __grid_constant__ CUtensorMap tmv) {
  constexpr int NB = D / 64;  // 64-wide column blocks of a row
  constexpr uint32_t QTILE = BM * D * 2, KVBYTES = BN * D * 2;
  enum { B_QFULL = 0, B_QEMPTY = 2, B_KFULL = 4, B_KEMPTY = B_KFULL + KST, B_VFULL = B_KEMPTY + KST, B_VEMPTY = B_VFULL + VST,
         B_VFIX = B_VEMPTY + VST, B_SFULL = B_VFIX + VST, B_PFULL = B_SFULL + 2, B_PFULL2 = B_PFULL + 2, B_OHALF = B_PFULL2 + 2,
         B_ODONE = B_OHALF + 2, B_DRAIN = B_ODONE + 2, NBARS };
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sQ = sm;
  unsigned char* sK = sQ + 2 * QTILE;
  unsigned char* sV = sK + KST * KVBYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + VST * KVBYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{abort_flag, x.status, (unsigned)VDN_TAG_XATTN, x.wait_limit};
  auto bar = [&](int i) { return smem_u32(bars + i); };

  clear_status(x.status);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i) mbar_init(bar(i), i >= B_PFULL && i < B_OHALF ? 4 : 1);  // P: an arrival per softmax warp
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // rows past a tile's own are never loaded: zeros, so that nothing a warp does depends on what they hold
  for (int i = threadIdx.x; i < 2 * NB * (BM - x.P * x.TT) * 8; i += kThr) {
    const int blk = i / ((BM - x.P * x.TT) * 8), at = i % ((BM - x.P * x.TT) * 8);
    reinterpret_cast<uint4*>(sQ + blk * BM * 128 + x.P * x.TT * 128)[at] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ K producer
    Walk w;
    int issued = 0;
    for (w.start(x); w.on; w.next(x)) {
      const int s = w.n % KST;
      if (w.n >= KST && !mbar_wait_warp(bar(B_KEMPTY + s), (w.n / KST - 1) & 1, ctl)) break;
      if (lane == 0) {
        mbar_expect_tx(bar(B_KFULL + s), KVBYTES);
        for (int c = 0; c < NB; ++c)
          tma_load_3d(smem_u32(sK + s * KVBYTES + c * BN * 128), &tmk, bar(B_KFULL + s), c * 64, w.it.hg * x.P / x.G,
                      w.it.k0 + w.j * BN);
      }
      issued = w.n + 1;
    }
    if (lane == 0)
      for (int n = max(issued - KST, 0); n < issued; ++n) mbar_drain(bar(B_KFULL + n % KST), (n / KST) & 1);
  } else if (warp == 2) {
    // ------------------------------------------------------------ V producer
    Walk w;
    int issued = 0;
    for (w.start(x); w.on; w.next(x)) {
      const int s = w.n % VST;
      if (w.n >= VST && !mbar_wait_warp(bar(B_VEMPTY + s), (w.n / VST - 1) & 1, ctl)) break;
      if (lane == 0) {
        mbar_expect_tx(bar(B_VFULL + s), KVBYTES);
        for (int c = 0; c < NB; ++c)
          tma_load_3d(smem_u32(sV + s * KVBYTES + c * BN * 128), &tmv, bar(B_VFULL + s), c * 64, w.it.hg * x.P / x.G,
                      w.it.k0 + w.j * BN);
      }
      issued = w.n + 1;
      const int valid = w.it.nk - w.j * BN;
      if (valid < BN) {  // rows past the last state: zeros
        if (!mbar_wait_warp(bar(B_VFULL + s), (w.n / VST) & 1, ctl)) break;
        for (int c = 0; c < NB; ++c) {
          uint4* base = reinterpret_cast<uint4*>(sV + s * KVBYTES + c * BN * 128);
          for (int i = valid * 8 + lane; i < BN * 8; i += 32) base[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(bar(B_VFIX + s));
      }
    }
    if (lane == 0)
      for (int n = max(issued - VST, 0); n < issued; ++n) mbar_drain(bar(B_VFULL + n % VST), (n / VST) & 1);
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q producer
    const uint32_t bytes = (uint32_t)(x.P * x.TT) * 128u * NB;
    int cnt[2] = {0, 0};  // loads into each tile
    bool ok = true;
    ItemPos pos;
    for (pos.start(x.grid); ok && pos.on(x.grid); pos.next(x.grid)) {
      const Item it = decode(x, pos);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || it.nt == 0 || !has_rows(x, it, t)) continue;
        if (cnt[t] > 0 && !mbar_wait_warp(bar(B_QEMPTY + t), (cnt[t] - 1) & 1, ctl)) { ok = false; continue; }
        if (lane == 0) {
          mbar_expect_tx(bar(B_QFULL + t), bytes);
          for (int c = 0; c < NB; ++c)
            tma_load_3d(smem_u32(sQ + t * QTILE + c * BM * 128), &tmq, bar(B_QFULL + t), c * 64, it.hg * x.P,
                        it.q0 + t * x.TT);
        }
        ++cnt[t];
      }
    }
    if (lane == 0)
      for (int t = 0; t < 2; ++t)
        if (cnt[t] > 0) mbar_drain(bar(B_QFULL + t), (cnt[t] - 1) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp, converged; one elected lane issues)
    constexpr uint32_t ID_S = idesc_bf16(BM, BN, false);
    constexpr uint32_t ID_O = idesc_bf16(BM, D, true);
    const uint32_t el = elect_one();
    const uint64_t qd0 = sdesc(smem_u32(sQ), 16, 1024), kd0 = sdesc(smem_u32(sK), 16, 1024);
    const uint64_t vd0 = sdesc(smem_u32(sV), BN * 128, 1024);
    uint32_t qpar = 0, ppar = 0, fixes = 0;  // parities: of tile t's next Q, its next P, the next zeroed V of a stage
    Walk w, nx;  // the key tile at hand, the one after it
    // S_t = Q_t K^T of the key tile n
    auto scores = [&](int t, const Walk& n) -> bool {
      const int s = n.n % KST;
      if (n.j == 0) {
        if (!mbar_wait_warp(bar(B_QFULL + t), (qpar >> t) & 1, ctl)) return false;
        qpar ^= 1u << t;
      }
      if (t == 0 && !mbar_wait_warp(bar(B_KFULL + s), (n.n / KST) & 1, ctl)) return false;
      tc_fence_after();
      const uint64_t qd = dadd(qd0, t * QTILE), kd = dadd(kd0, s * KVBYTES);
      const uint32_t dst = tmem + col_s(t);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_bf16_w(dst, dadd(qd, (k >> 2) * (BM * 128) + (k & 3) * 32), dadd(kd, (k >> 2) * (BN * 128) + (k & 3) * 32), ID_S,
                   k > 0 ? 1u : 0u, el);
      mma_commit_w(bar(B_SFULL + t), el);
      if (t == 1 || !has_rows(x, n.it, 1)) mma_commit_w(bar(B_KEMPTY + s), el);  // read by both tiles
      if (n.j + 1 == n.it.nt) mma_commit_w(bar(B_QEMPTY + t), el);               // the item's last scores
      return true;
    };
    w.start(x);
    nx = w;
    bool ok = true, begun = false;  // the first turn only forms the scores of the first key tile
#pragma unroll 1
    while (ok && (w.on || !begun)) {
      const int sv = w.n % VST;
      const bool part = w.it.nk - w.j * BN < BN;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (begun && has_rows(x, w.it, t)) {
          if (t == 0)  // V of this key tile
            ok = mbar_wait_warp(bar(B_VFULL + sv), (w.n / VST) & 1, ctl) &&
                 (!part || mbar_wait_warp(bar(B_VFIX + sv), (fixes >> sv) & 1, ctl));
          if (!ok) break;  // not lost to the waits below: no product on a V that is not there, or not zeroed
          // O_t += P_t V in two halves of 64 states, the first one while the softmax forms the second
          const uint64_t vd = dadd(vd0, sv * KVBYTES);
          const uint32_t dst = tmem + col_o(t), pa = tmem + col_s(t);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = mbar_wait_warp(bar(B_PFULL + 2 * h + t), (ppar >> t) & 1, ctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16_ts_w(dst, pa + 32 * h + 8 * k, dadd(vd, (64 * h + 16 * k) * 128), ID_O, (w.j == 0 && h == 0 && k == 0) ? 0u : 1u, el);
            mma_commit_w(bar(B_OHALF + 2 * h + t), el);
          }
          if (!ok) break;
          if (t == 1 || !has_rows(x, w.it, 1)) mma_commit_w(bar(B_VEMPTY + sv), el);
          ppar ^= 1u << t;
        }
        // the next key tile's scores, over the P that the products above read first
        if (nx.on && has_rows(x, nx.it, t)) {
          ok = scores(t, nx);
          if (!ok) break;
        }
      }
      if (begun && part) fixes ^= 1u << sv;
      w = nx;
      if (nx.on) nx.next(x);
      begun = true;
    }
    mma_commit_w(bar(B_DRAIN), el);
    mbar_drain(bar(B_DRAIN), 0);
  } else {
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lane_addr + col_s(t), ocol = lane_addr + col_o(t);
    const float c = x.scale * kLog2e;       // log2 units
    const float thresh = fminf(kRescaleLog2 / c, 1e30f);  // raw scores; finite, so that a first maximum is always taken
    const int rtok = row / x.P, rhead = row % x.P;
    const bool whole = (reinterpret_cast<uintptr_t>(x.y) & 31) == 0;
    int n = 0;  // key tiles of this tile so far
    bool ok = true;
    ItemPos pos;
    for (pos.start(x.grid); ok && pos.on(x.grid); pos.next(x.grid)) {
      const Item it = decode(x, pos);
      if (!has_rows(x, it, t)) continue;
      float m_used = -INFINITY, l_sum = 0.f;
      bool any = false;
      for (int j = 0; ok && j < it.nt; ++j, ++n) {
        // every TMEM access is warp-collective: control flow stays warp-uniform
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_SFULL + t), n & 1, ctl))) { ok = false; break; }
        tc_fence_after();
        const int kvalid = it.nk - j * BN;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t sh = scol + 64 * h;  // scores of states [64 h, 64 h + 64) of the tile
          const int kvh = kvalid - 64 * h;    // valid ones (may be <= 0)
          bool done = false;
          // A full half after the item's first: one pass with the reference kept, where the sum of P is at most 2^8
          if ((any || h == 1) && kvh >= 64) {
            const float2 c2 = make_float2(c, c), nmc2 = make_float2(-m_used * c, -m_used * c);
            float2 ps[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) ps[u] = make_float2(0.f, 0.f);
            float pk[32];
            auto chunk = [&](const float (&v)[32], int o) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = fma2(make_float2(v[2 * i], v[2 * i + 1]), c2, nmc2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                ps[i & 3] = add2(ps[i & 3], p);
                pk[o + i] = __uint_as_float(pack_bf16(p.x, p.y));
              }
            };
            float va[32], vb[32];
            tmem_ld32(sh, va);
            tmem_wait_ld();
            tmem_ld32(sh + 32, vb);
            chunk(va, 0);
            tmem_wait_ld();
            chunk(vb, 16);
            const float2 pt = add2(add2(ps[0], ps[1]), add2(ps[2], ps[3]));
            const float psum = pt.x + pt.y;
            if (!__any_sync(0xffffffffu, !(psum <= 256.0f))) {
              tmem_st32(scol + 32 * h, pk);
              l_sum += psum;
              done = true;
            }
          }
          if (!done) {
            // its maximum, O rescaled where a row's reference moves, then P
            float v0[32], v1[32];
            tmem_ld32(sh, v0);
            tmem_ld32(sh + 32, v1);
            tmem_wait_ld();
            float pm[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) pm[u] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v0[i] = i < kvh ? v0[i] : -INFINITY;
              v1[i] = 32 + i < kvh ? v1[i] : -INFINITY;
              pm[i & 7] = fmaxf(pm[i & 7], fmaxf(v0[i], v1[i]));
            }
            const float mx = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])),
                                   fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7])));
            const bool need = mx > m_used + thresh;
            float f = 1.0f;
            if (need) {
              f = m_used == -INFINITY ? 0.f : ex2((m_used - mx) * c);
              l_sum *= f;
              m_used = mx;
            }
            // O holds the item's products so far: those of its last key tile (h = 0) or this one's first half
            if ((any || h == 1) && __any_sync(0xffffffffu, need)) {
              const bool st = h == 0 ? mbar_wait(bar(B_ODONE + t), (n - 1) & 1, ctl) : mbar_wait(bar(B_OHALF + t), n & 1, ctl);
              if (!__all_sync(0xffffffffu, st)) { ok = false; break; }
              tc_fence_after();
              float v[32];
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                tmem_ld32(ocol + q * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= f;
                tmem_st32(ocol + q * 32, v);
              }
              tmem_wait_st();
            }
            // a row with no finite score so far takes the reference 0: weights of 0, not of inf - inf
            const float mc = m_used == -INFINITY ? 0.f : m_used * c;
            const float2 c2 = make_float2(c, c), nmc2 = make_float2(-mc, -mc);
            float2 ps[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) ps[u] = make_float2(0.f, 0.f);
            float pk[32];
            auto chunk = [&](const float (&v)[32], int o) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = fma2(make_float2(v[2 * i], v[2 * i + 1]), c2, nmc2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                ps[i & 3] = add2(ps[i & 3], p);
                pk[o + i] = __uint_as_float(pack_bf16(p.x, p.y));
              }
            };
            chunk(v0, 0);
            chunk(v1, 16);
            tmem_st32(scol + 32 * h, pk);
            const float2 pt = add2(add2(ps[0], ps[1]), add2(ps[2], ps[3]));
            l_sum += pt.x + pt.y;
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive_warp(bar(h == 0 ? B_PFULL + t : B_PFULL2 + t));
        }
        any = true;
      }
      if (!ok) break;
      // ---- epilogue: O / l
      if (any && !__all_sync(0xffffffffu, mbar_wait(bar(B_ODONE + t), (n - 1) & 1, ctl))) { ok = false; break; }
      tc_fence_after();
      const int tok = it.q0 + t * x.TT + rtok;
      const bool valid = rtok < x.TT && rtok < it.left - t * x.TT;
      const long long gr = (long long)tok * x.H + it.hg * x.P + rhead;
      const float inv = any ? 1.0f / l_sum : 0.f;
      const float lse2 = any ? m_used * c + __log2f(l_sum) : -INFINITY;
      if (x.po == nullptr) {
        if (valid && x.lse != nullptr) x.lse[gr] = lse2 * kLn2;
        __nv_bfloat16* y = x.y + gr * D;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float v[32];
          if (any) {
            tmem_ld32(ocol + q * 32, v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          uint32_t u[2][8];
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i >> 3][i & 7] = pack_bf16(v[2 * i] * inv, v[2 * i + 1] * inv);
          if (valid) {
            store32(y + q * 32, u[0], whole);
            store32(y + q * 32 + 16, u[1], whole);
          }
        }
      } else {
        const long long pr = it.sp * x.rows + gr;
        if (valid) x.pl[pr] = lse2;
        if (any) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            float v[32];
            tmem_ld32(ocol + q * 32, v);
            tmem_wait_ld();
            if (valid) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(x.po + pr * D + q * 32 + i) =
                    make_float4(v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv);
            }
          }
        }
      }
      tc_fence_before();  // the reads of O before the next item's first P is handed over
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, kTmemCols);
}

// The partial results of a row joined: o = sum_i 2^(lse_i - lse) o_i, a warp a row.
template <int D>
__global__ void __launch_bounds__(256) k_xattn_join(const XtDev x, int parts) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= x.rows) return;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 32) m = fmaxf(m, x.pl[i * x.rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f, acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
  for (int i = 0; i < parts; ++i) {
    const float l = x.pl[i * x.rows + row];
    if (l == -INFINITY) continue;  // no states, and no output written
    const float w = ex2(l - ref);
    s += w;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(w, x.po[(i * x.rows + row) * D + (D / 32) * lane + e], acc[e]);
  }
  const int b = (int)(row / ((long long)x.Tq * x.H));  // one row a warp
  const bool none = valid_states(x, b) == 0;
  const float inv = none ? 0.f : 1.0f / s;
  uint32_t u[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) u[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  __nv_bfloat16* y = x.y + row * D + (D / 32) * lane;
  if constexpr (D == 128) *reinterpret_cast<uint2*>(y) = make_uint2(u[0], u[1]);
  else *reinterpret_cast<uint32_t*>(y) = u[0];
  if (lane == 0 && x.lse != nullptr) x.lse[row] = (none ? -INFINITY : ref + __log2f(s)) * kLn2;
}

// How a problem is cut.  A key tile costs one unit, an item about 1.5 more (its
// start and its output), a split's partial results and their join about two.
constexpr int kSms = 148;
constexpr int kMaxSplit = 64;
struct Cut {
  int P, TT, HG, pairs, ns, parts;
  long long items;
};
Cut cut(const XDims& d) {
  Cut best{};
  double cost = 0;
  for (int pack = 0; pack < 2; ++pack) {
    if (pack && (d.G == 1 || d.G > BM)) continue;
    Cut c;
    c.P = pack ? d.G : 1;
    c.TT = BM / c.P;
    c.HG = d.H / c.P;
    const int nt = (d.L + BN - 1) / BN;
    c.pairs = (int)(((long long)d.Tq + 2 * c.TT - 1) / (2 * c.TT));
    const long long base = (long long)d.B * c.HG * c.pairs;
    for (int ns = 1; ns <= kMaxSplit && ns <= nt; ++ns) {
      if (ns > 1 && base * ns > 2 * kSms) break;
      const int per = (nt + ns - 1) / ns;
      const double t = (double)((base * ns + kSms - 1) / kSms) * (per + 1.5) + (ns > 1 ? 2.0 : 0.0);
      if (best.items == 0 || t < cost) {
        cost = t;
        best = c;
        best.ns = ns;
        best.items = base * ns;
        best.parts = ns > 1 ? ns : 0;
      }
    }
  }
  return best;
}

template <int D>
cudaError_t launch(const XDims& d, const XArgs& a, cudaStream_t s) {
  const Cut c = cut(d);
  if (c.items > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  CUtensorMap mq, mk, mv;
  if (!make_token_map_strided(&mq, a.q, (long long)d.B * d.Tq, d.H, D, (long long)d.H * D, c.P, c.TT) ||
      !make_token_map_strided(&mk, a.k, (long long)d.B * d.L, d.Hkv, D, d.ks, 1, BN) ||
      !make_token_map_strided(&mv, a.v, (long long)d.B * d.L, d.Hkv, D, d.vs, 1, BN))
    return cudaErrorInvalidValue;
  XtDev x{};
  x.B = d.B; x.Tq = d.Tq; x.L = d.L; x.H = d.H; x.G = d.G;
  const unsigned grid = (unsigned)(c.items < kSms ? c.items : kSms);
  x.P = c.P; x.TT = c.TT; x.ns = c.ns;
  x.grid = item_grid((int)c.items, c.ns, c.HG, c.pairs, (int)grid);
  x.scale = d.scale;
  x.kv_len = d.kv_len;
  x.y = static_cast<__nv_bfloat16*>(const_cast<void*>(a.y));
  x.lse = a.lse;
  x.rows = (long long)d.B * d.Tq * d.H;
  if (c.parts) {
    x.po = static_cast<float*>(a.scratch);
    x.pl = x.po + (long long)c.parts * x.rows * D;
  }
  x.status = a.status;
  x.wait_limit = a.wait_limit;
  const size_t smem = 1024 + (size_t)2 * BM * D * 2 + (size_t)(KST + VST) * BN * D * 2 + 40 * 8 + 16;
  cudaError_t e = allow_smem<k_xattn_tc<D>>(smem);
  if (e != cudaSuccess) return e;
  k_xattn_tc<D><<<grid, kThr, smem, s>>>(x, mq, mk, mv);
  if ((e = cudaGetLastError()) != cudaSuccess || !c.parts) return e;
  k_xattn_join<D><<<(unsigned)((x.rows + 7) / 8), 256, 0, s>>>(x, c.parts);
  return cudaGetLastError();
}

}  // namespace

bool xattn_tc_supported(const XDims& d) { return d.d == 64 || d.d == 128; }

size_t xattn_tc_scratch(const XDims& d) {
  const Cut c = cut(d);
  return (size_t)c.parts * d.B * d.Tq * d.H * (d.d + 1) * sizeof(float);
}

cudaError_t launch_xattn_tc(const XDims& d, const XArgs& a, cudaStream_t s) {
  return d.d == 128 ? launch<128>(d, a, s) : launch<64>(d, a, s);
}

}  // namespace vdn
