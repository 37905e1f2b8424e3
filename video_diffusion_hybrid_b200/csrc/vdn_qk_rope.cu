// RMSNorm of every query and key head and the rotation by position, in one
// pass over q and k (they enter the attention core and the cross-attention
// this way), and the backward of both.
//
//   z = x rstd w,  rstd = 1 / sqrt(mean x^2 + eps)        (per head, over d)
//   (a, b) -> (a cos - b sin, a sin + b cos)               on the pairs of the first `rot` columns
// cos and sin come from a table row of the token's position on the pair's
// axis.  Backward, with g the gradient of the output:
//   dz = the rotation by the negative angle of g,  dw = sum over tokens of dz x rstd
//   dx = rstd (dz w - xh mean(dz w xh)),  xh = x rstd
//
// Bound by HBM: 9 (16 backward) flops an element against 4 bytes or more.  A
// row (one head of one token) is held by LPR lanes with 8 columns each, so
// every access is a 16-byte vector and the row's sums are shuffles.  A thread
// has the same columns of HU heads of a token: the token's positions and its
// angles are read and addressed once for all of them (with one head a thread
// the instructions around the data, 25 an element, kept the kernel at 55 % of
// the memory's rate).  Its heads stay the same over all the tokens that the
// block walks, so the norm's weights, and in the backward their gradient, stay
// in registers.  The tokens to come are copied into shared memory ahead
// (cp.async; a row is copied and read by lanes of one warp, so no block barrier),
// and the next token's angles into registers: with loads at their use the
// threads waited for memory, and for the angles, between tokens.
// The weights' gradient: a block adds its threads' sums in shared memory and
// writes them (fp32), a second kernel adds the blocks', both in a fixed order,
// so results do not depend on timing.
#include <climits>

#include <cuda_bf16.h>

#include "vdn_internal.h"

namespace vdn {
namespace {

constexpr int kThreads = 256;

struct QkDev {
  const void *q, *k;
  long long qs, ks;  // elements between tokens
  const float *wq, *wk, *table;
  const int* pos;
  void *qo, *ko;          // forward: outputs; backward: dq, dk (dense)
  const void *gq, *gk;    // backward: gradients of the outputs (dense)
  float* part;            // backward: partial weight gradients [gx][Hq + Hk][d], or [gx nch][2][d] for shared weights; or null
  long long tokens;
  int Hq, Ht, d, rot, axes, rows;  // rows: table rows (unsigned: 2^31 where there is no table)
  int sec0, sec01;                 // first pair of axis 1 and of axis 2
  int per_head, vec;               // vec: no lane's pairs straddle two axes
  int zero_skipped;                // forward: skipped tokens' rows are written as zeros
  int hc, tpi, nch, gx;            // head slots of a block, tokens per block step, head chunks (of HU hc heads), blocks per chunk
  int threads;                     // of a block: its row slots' lanes
  float eps;
};

// 8 consecutive elements as stored: one 16-byte vector (bf16) or two (fp32)
template <typename T> struct Raw { uint4 v[sizeof(T) / 2]; };

// The ring of a block: NV vectors of every thread for each of NS tokens.  A row's
// 16-byte chunks lie in order; lane li copies chunks li, LPR + li (whole sectors
// in every instruction) and reads the ones of its 8 columns.
template <int NV, int NS, int LPR>
struct Ring {
  uint4* base;
  int st;  // stage of the token at hand
  __device__ __forceinline__ Ring(uint4* smem) : base(smem), st(0) {}
  // vectors v .. v + V - 1 of the row of this thread's slot
  template <int V>
  __device__ __forceinline__ uint4* row(int stage, int v) const {
    return base + (stage * NV + v) * kThreads + threadIdx.x / LPR * (LPR * V);
  }
  // the row at p (d elements, null: zeros) into vectors v.. of the stage `ahead` tokens on
  template <typename T>
  __device__ __forceinline__ void copy(int ahead, int v, const T* p, const void* any, int d) const {
    constexpr int V = sizeof(T) / 2;
    const int s = st + ahead >= NS ? st + ahead - NS : st + ahead, li = threadIdx.x % LPR;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * LPR + li;
      const bool on = p != nullptr && c * (16 / (int)sizeof(T)) < d;
      const void* src = on ? static_cast<const void*>(reinterpret_cast<const uint4*>(p) + c) : any;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(row<V>(s, v) + c)),
                   "l"(src), "r"(on ? 16 : 0)
                   : "memory");
    }
  }
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // the token at hand has landed, for the whole warp
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
    __syncwarp();
  }
  template <typename T>
  __device__ __forceinline__ Raw<T> read(int v) const {
    constexpr int V = sizeof(T) / 2;
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = row<V>(st, v)[threadIdx.x % LPR * V + i];
    return r;
  }
  __device__ __forceinline__ void next() {
    __syncwarp();  // read by every lane, before any copies over it
    st = st + 1 == NS ? 0 : st + 1;
  }
};
__device__ __forceinline__ void expand(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void expand(const Raw<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x);
    x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z);
    x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = u;
}

// x where the mask's bits are set, else zeros (whatever x is)
__device__ __forceinline__ void store8_masked(float* p, const float (&x)[8], uint32_t m) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(__float_as_uint(x[i]) & m);
  store8(p, y);
}
__device__ __forceinline__ void store8_masked(__nv_bfloat16* p, const float (&x)[8], uint32_t m) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h) & m;
  }
  *reinterpret_cast<uint4*>(p) = u;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's view of the rotation: which pairs it has and where its partner is.
template <int LPR, bool SPLIT>
struct Turn {
  int pair0, partner;  // first pair of this lane, lane holding the other half (SPLIT)
  bool on, second;     // this lane's columns are rotated; it holds the second half (SPLIT)
  static constexpr int NP = SPLIT ? 8 : 4;
  float cs[NP], sn[NP];

  __device__ __forceinline__ Turn(const QkDev& a, int li, int lane) {
    const int c = 8 * li, half = a.rot >> 1;
    on = c < a.rot;
    second = SPLIT && on && c >= half;
    pair0 = SPLIT ? (second ? c - half : c) : (c >> 1);
    partner = !SPLIT || !on ? lane : (second ? lane - half / 8 : lane + half / 8);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
  }
  __device__ __forceinline__ void take(const Turn& o) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      cs[i] = o.cs[i];
      sn[i] = o.sn[i];
    }
  }
  // the angles of one token (its positions are inside the table)
  __device__ __forceinline__ void angles(const QkDev& a, const int (&p)[3]) {
    if (!on) return;
    const int half = a.rot >> 1;
    if (a.vec) {
      const int r = pair0 >= a.sec01 ? p[2] : pair0 >= a.sec0 ? p[1] : p[0];
      const float4* t = reinterpret_cast<const float4*>(a.table + ((long long)r * half + pair0) * 2);
#pragma unroll
      for (int i = 0; i < NP / 2; ++i) {
        const float4 f = __ldg(t + i);
        cs[2 * i] = f.x; sn[2 * i] = f.y;
        cs[2 * i + 1] = f.z; sn[2 * i + 1] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int j = pair0 + i;
        const int r = j >= a.sec01 ? p[2] : j >= a.sec0 ? p[1] : p[0];
        const float2 f = __ldg(reinterpret_cast<const float2*>(a.table) + (long long)r * half + j);
        cs[i] = f.x;
        sn[i] = f.y;
      }
    }
  }
  // x rotated by dir * angle; all lanes of the warp take part
  __device__ __forceinline__ void apply(float (&x)[8], float dir) const {
    if (SPLIT) {
      const float s = second ? dir : -dir;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, x[i], partner);
        x[i] = fmaf(o, s * sn[SPLIT ? i : 0], x[i] * cs[SPLIT ? i : 0]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], v = x[2 * i + 1], s = dir * sn[i];
        x[2 * i] = fmaf(-v, s, u * cs[i]);
        x[2 * i + 1] = fmaf(u, s, v * cs[i]);
      }
    }
  }
};

// The token's positions; false when one lies outside the table (the token is skipped).
__device__ __forceinline__ bool positions(const QkDev& a, long long t, int (&p)[3]) {
  p[0] = p[1] = p[2] = 0;
  if (a.pos == nullptr) {
    p[0] = (int)t;
    return a.rot == 0 || t < a.rows;
  }
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < a.axes) {
      p[i] = __ldg(a.pos + t * a.axes + i);
      ok = ok && (unsigned)p[i] < (unsigned)a.rows;
    }
  return ok;
}

// Where this thread's row slot lies: lane within the row, token of the step, its heads.
template <int LPR, int HU>
struct Slot {
  int li, ti, head0;  // head i of the thread: head0 + i hc
  bool row, active;  // the slot has a token; the lane has columns
  __device__ __forceinline__ Slot(const QkDev& a) {
    const int lane = threadIdx.x & 31, slot = threadIdx.x / LPR;
    li = lane % LPR;
    ti = slot / a.hc;
    head0 = (int)(blockIdx.x % a.nch) * a.hc * HU + slot % a.hc;
    row = ti < a.tpi;
    active = row && 8 * li < a.d;
  }
};

// One head of a thread: its columns' offset within a dense token, and the norm's weights there.
struct Head {
  int row, off;  // of the head; of the lane's columns
  bool on, isq;
  float w[8];
  __device__ __forceinline__ void init(const QkDev& a, int head, int li, bool active) {
    on = active && head < a.Ht;
    isq = head < a.Hq;
    row = head < a.Ht ? (isq ? head : head - a.Hq) * a.d : -1;
    off = (isq ? head : head - a.Hq) * a.d + 8 * li;
    const float* p = isq ? a.wq : a.wk;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = on && p != nullptr ? __ldg(p + (a.per_head ? off : 8 * li) + i) : 1.f;
  }
  // the columns in a pair of tensors, the token tq (tk) elements from their start
  template <typename P>
  __device__ __forceinline__ P* at(P* q, P* k, long long tq, long long tk) const {
    return (isq ? q + tq : k + tk) + off;
  }
  // the head's row there
  template <typename P>
  __device__ __forceinline__ P* row_at(P* q, P* k, long long tq, long long tk) const {
    return (isq ? q + tq : k + tk) + row;
  }
};

template <typename T, int HU> constexpr int fwd_stages() { return HU > 1 ? 4 : sizeof(T) == 2 ? 8 : 4; }
template <typename T, int HU> constexpr size_t fwd_smem() {
  return (size_t)fwd_stages<T, HU>() * HU * (sizeof(T) / 2) * kThreads * 16;
}
template <typename T, typename G, int HU> constexpr int bwd_vectors() { return HU * (int)(sizeof(T) + sizeof(G)) / 2; }
template <typename T, typename G, int HU> constexpr int bwd_stages() { return bwd_vectors<T, G, HU>() >= 8 ? 3 : 4; }
template <typename T, typename G, int HU> constexpr size_t bwd_smem() {
  return (size_t)bwd_stages<T, G, HU>() * bwd_vectors<T, G, HU>() * kThreads * 16;
}

template <typename T, int LPR, bool SPLIT, int HU>
__global__ void __launch_bounds__(kThreads, 3) k_qk_fwd(const QkDev a) {
  constexpr int NS = fwd_stages<T, HU>(), V = sizeof(T) / 2;
  extern __shared__ uint4 qk_smem[];
  Ring<HU * V, NS, LPR> ring(qk_smem);
  const Slot<LPR, HU> s(a);
  Head hd[HU];
#pragma unroll
  for (int i = 0; i < HU; ++i) hd[i].init(a, s.head0 + i * a.hc, s.li, s.active);
  Turn<LPR, SPLIT> turn(a, s.li, threadIdx.x & 31);
  const long long step = (long long)a.gx * a.tpi, dq = (long long)a.Hq * a.d, dk = (long long)(a.Ht - a.Hq) * a.d;
  const float inv_d = 1.0f / (float)a.d;
  auto fetch = [&](int ahead, long long t) {
    const bool on = s.row && t < a.tokens;
    const long long tq = t * a.qs, tk = t * a.ks;
#pragma unroll
    for (int i = 0; i < HU; ++i)
      ring.copy(ahead, i * V,
                on && hd[i].row >= 0 ? hd[i].row_at(static_cast<const T*>(a.q), static_cast<const T*>(a.k), tq, tk) : nullptr, a.q, a.d);
    ring.commit();
  };
  const long long first = (long long)(blockIdx.x / a.nch) * a.tpi;
#pragma unroll
  for (int k = 0; k < NS - 1; ++k) fetch(k, first + k * step + s.ti);
  // the token at hand's turn; the next one's, under way; the positions of the one after that
  Turn<LPR, SPLIT> after = turn;
  int p[3], pn[3];
  const long long t0 = first + s.ti;
  bool on = s.active && t0 < a.tokens && positions(a, t0, p);
  bool onn = s.active && t0 + step < a.tokens && positions(a, t0 + step, pn);
  if (on) turn.angles(a, p);
  for (long long base = first; base < a.tokens; base += step) {
    const long long t = base + s.ti;
    if (onn) after.angles(a, pn);
    const bool ona = s.active && t + 2 * step < a.tokens && positions(a, t + 2 * step, pn);
    fetch(NS - 1, t + (NS - 1) * step);
    ring.wait();
    const long long oq = t * dq, ok = t * dk;
    // A skipped token's rows, where they are to be zeros: its values masked behind the rounding.  90,720 tokens of 48 heads
    // take 455 us, without it 442; predicated stores of zeros and a branch around them took 467 and 462 to 471 where this
    // took 463, walks of their own behind or before the loop 486 and 502 to 542; a kernel of its own was as fast but 3 us
    // more for a single token.
    const bool st = on || (a.zero_skipped && s.active && t < a.tokens);
    const uint32_t mask = on ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < HU; ++i) {
      float x[8], ss = 0.f;
      expand(ring.template read<T>(i * V), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      const float rstd = rsqrtf(fmaf(row_sum<LPR>(ss), inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= rstd * hd[i].w[e];
      turn.apply(x, 1.f);
      if (st && hd[i].on) store8_masked(hd[i].at(static_cast<T*>(a.qo), static_cast<T*>(a.ko), oq, ok), x, mask);
    }
    ring.next();
    turn.take(after);
    on = onn;
    onn = ona;
  }
}

template <typename T, typename G, int LPR, bool SPLIT, int HU>
__global__ void __launch_bounds__(kThreads, 2) k_qk_bwd(const QkDev a) {
  constexpr int NS = bwd_stages<T, G, HU>(), V = sizeof(T) / 2, VG = sizeof(G) / 2, NV = V + VG;
  extern __shared__ uint4 qk_smem[];
  Ring<HU * NV, NS, LPR> ring(qk_smem);
  const Slot<LPR, HU> s(a);
  Head hd[HU];
  float acc[HU][8];
#pragma unroll
  for (int i = 0; i < HU; ++i) {
    hd[i].init(a, s.head0 + i * a.hc, s.li, s.active);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  }
  Turn<LPR, SPLIT> turn(a, s.li, threadIdx.x & 31);
  const long long step = (long long)a.gx * a.tpi, dq = (long long)a.Hq * a.d, dk = (long long)(a.Ht - a.Hq) * a.d;
  const float inv_d = 1.0f / (float)a.d;
  auto fetch = [&](int ahead, long long t) {
    const bool on = s.row && t < a.tokens;
    const long long tq = t * a.qs, tk = t * a.ks, oq = t * dq, ok = t * dk;
#pragma unroll
    for (int i = 0; i < HU; ++i) {
      const bool ld = on && hd[i].row >= 0;
      ring.copy(ahead, i * NV, ld ? hd[i].row_at(static_cast<const T*>(a.q), static_cast<const T*>(a.k), tq, tk) : nullptr, a.q, a.d);
      ring.copy(ahead, i * NV + V, ld ? hd[i].row_at(static_cast<const G*>(a.gq), static_cast<const G*>(a.gk), oq, ok) : nullptr, a.q,
                a.d);
    }
    ring.commit();
  };
  const long long first = (long long)(blockIdx.x / a.nch) * a.tpi;
#pragma unroll
  for (int k = 0; k < NS - 1; ++k) fetch(k, first + k * step + s.ti);
  for (long long base = first; base < a.tokens; base += step) {
    const long long t = base + s.ti;
    int p[3];
    const bool in = s.active && t < a.tokens, on = in && positions(a, t, p);
    if (on) turn.angles(a, p);
    fetch(NS - 1, t + (NS - 1) * step);
    ring.wait();
    const long long oq = t * dq, ok = t * dk;
#pragma unroll
    for (int i = 0; i < HU; ++i) {
      float x[8], g[8], ss = 0.f, dot = 0.f;
      expand(ring.template read<T>(i * NV), x);
      expand(ring.template read<G>(i * NV + V), g);
      if (!on) {
        // a skipped token's output does not depend on its input: its gradient is zero, whatever the two arrays hold there
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = g[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      turn.apply(g, -1.f);
      const float rstd = rsqrtf(fmaf(row_sum<LPR>(ss), inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= rstd;
        acc[i][e] = fmaf(g[e], x[e], acc[i][e]);
        g[e] *= hd[i].w[e];
        dot = fmaf(g[e], x[e], dot);
      }
      dot = row_sum<LPR>(dot) * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = rstd * fmaf(-x[e], dot, g[e]);
      if (in && hd[i].on) store8(hd[i].at(static_cast<T*>(a.qo), static_cast<T*>(a.ko), oq, ok), g);
    }
    ring.next();
  }
  if (a.part == nullptr) return;
  // the block's sums: columns c of the LPR lanes' 8 LPR, slot after slot, in the ring's memory
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  static_assert(bwd_smem<T, G, HU>() >= (size_t)HU * kThreads * 8 * sizeof(float), "the ring holds the sums");
  float* buf = reinterpret_cast<float*>(qk_smem);
  constexpr int W = 8 * LPR, PLANE = kThreads * 8;
  const int blk = blockIdx.x / a.nch, chunk = blockIdx.x % a.nch;
#pragma unroll
  for (int i = 0; i < HU; ++i) store8(buf + i * PLANE + threadIdx.x * 8, acc[i]);
  __syncthreads();
  if (a.per_head) {
    for (int j = threadIdx.x; j < HU * a.hc * W; j += blockDim.x) {
      const int c = j % W, h = j / W, hs = h % a.hc, head = chunk * a.hc * HU + h;  // h = hs + i hc
      float v = 0.f;
      for (int t = 0; t < a.tpi; ++t) v += buf[h / a.hc * PLANE + (t * a.hc + hs) * W + c];
      if (head < a.Ht && c < a.d) a.part[((long long)blk * a.Ht + head) * a.d + c] = v;
    }
  } else {
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
      float sum[2] = {0.f, 0.f};  // queries, keys
      for (int i = 0; i < HU; ++i)
        for (int sl = 0; sl < a.hc * a.tpi; ++sl) {
          const int head = chunk * a.hc * HU + sl % a.hc + i * a.hc;
          if (head < a.Hq) sum[0] += buf[i * PLANE + sl * W + c];
          else if (head < a.Ht) sum[1] += buf[i * PLANE + sl * W + c];
        }
#pragma unroll
      for (int k = 0; k < 2; ++k) a.part[(((long long)blk * a.nch + chunk) * 2 + k) * a.d + c] = sum[k];
    }
  }
}

// dw[j] = sum of the blocks' partials, rows of `sets` [d].  A block has 32
// columns and 32 row lanes; one block column for each set (a head, or 0 =
// queries and 1 = keys).
__global__ void __launch_bounds__(1024) k_qk_dw(const float* __restrict__ part, float* __restrict__ dwq,
                                                float* __restrict__ dwk, int rows, int sets, int nq, int d) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), rl = threadIdx.x >> 5, set = blockIdx.y;
  float* dst = set < nq ? dwq : dwk;
  if (dst == nullptr) return;  // uniform over the block
  float s = 0.f;
  if (c < d)
    for (int i = rl; i < rows; i += 32) s += part[((long long)i * sets + set) * d + c];
  red[rl][threadIdx.x & 31] = s;
  __syncthreads();
  if (rl == 0 && c < d) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x & 31];
    dst[(long long)(set < nq ? set : set - nq) * d + c] = v;
  }
}

// Most blocks of one head chunk (the size of the backward's workspace does not depend on the device).
int qk_max_blocks(int nch) { return nch < 640 ? 640 / nch : 1; }

int lanes_per_row(int d) {
  int l = 1;
  while (8 * l < d) l *= 2;
  return l < 2 ? 2 : l;
}

// Heads of a thread: several where a block's row slots still hold all the heads
// of a token or nearly so (at most an eighth of the threads' heads unused).
int heads_per_thread(const vdn_qk_cfg& c, bool f32) {
  const int lpr = lanes_per_row(c.d), slots = kThreads / lpr, ht = c.Hq + c.Hk, hu = f32 ? 2 : 3;
  if (lpr < 8) return 1;
  const int nch = (ht + slots * hu - 1) / (slots * hu), hc = (ht + nch * hu - 1) / (nch * hu);
  const int used = slots / hc * hc;  // row slots with a token
  return 8 * (long long)ht * used >= 7LL * nch * hc * hu * slots ? hu : 1;
}

// Row slots of a block: chunks of heads of equal size, and as many tokens per
// step as fit beside one chunk.
void qk_slots(const vdn_qk_cfg& c, int hu, int* hc, int* tpi, int* nch) {
  const int slots = kThreads / lanes_per_row(c.d), ht = c.Hq + c.Hk;
  *nch = (ht + slots * hu - 1) / (slots * hu);
  *hc = (ht + *nch * hu - 1) / (*nch * hu);
  *tpi = slots / *hc;
}

// The block's row slots over heads and tokens, and the grid: `resident` blocks
// on every SM, or fewer when there are fewer tokens.
bool plan(const vdn_qk_cfg& c, QkDev& a, int hu, int resident) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  qk_slots(c, hu, &a.hc, &a.tpi, &a.nch);
  a.threads = (a.hc * a.tpi * lanes_per_row(c.d) + 31) / 32 * 32;
  const long long steps = ((long long)c.tokens + a.tpi - 1) / a.tpi;
  long long gx = (long long)resident * (kThreads / a.threads) * sms / a.nch;
  if (gx > qk_max_blocks(a.nch)) gx = qk_max_blocks(a.nch);
  if (gx < 1) gx = 1;
  a.gx = (int)(steps < gx ? steps : gx);
  return true;
}

QkDev device_args(const vdn_qk_cfg& c, const vdn_qk_args& in) {
  QkDev a{};
  a.q = in.q; a.k = in.k;
  a.qs = c.q_stride ? c.q_stride : (long long)c.Hq * c.d;
  a.ks = c.k_stride ? c.k_stride : (long long)c.Hk * c.d;
  a.wq = in.wq; a.wk = in.wk; a.table = in.table; a.pos = in.pos;
  a.qo = in.q_out; a.ko = in.k_out;
  a.tokens = c.tokens;
  a.Hq = c.Hq; a.Ht = c.Hq + c.Hk; a.d = c.d; a.rot = c.rot; a.axes = c.axes;
  a.rows = c.rot == 0 && c.table_rows == 0 ? INT_MIN : c.table_rows;  // compared as unsigned: every position from 0 on
  a.sec0 = c.axes > 1 ? c.sections[0] : 1 << 30;
  a.sec01 = c.axes > 2 ? c.sections[0] + c.sections[1] : 1 << 30;
  const int grain = c.pairing == VDN_PAIR_SPLIT ? 8 : 4;
  a.vec = (c.axes < 2 || a.sec0 % grain == 0) && (c.axes < 3 || a.sec01 % grain == 0);
  a.per_head = c.per_head;
  a.zero_skipped = c.zero_skipped;
  a.eps = c.eps > 0.f ? c.eps : 1e-6f;
  return a;
}

template <auto Kernel>
cudaError_t go(const QkDev& a, size_t smem, unsigned grid, cudaStream_t s) {
  const cudaError_t e = allow_smem<Kernel>(smem);
  if (e != cudaSuccess) return e;
  Kernel<<<grid, a.threads, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int LPR, int HU>
cudaError_t go_fwd(const QkDev& a, bool split, unsigned grid, cudaStream_t s) {
  return split ? go<k_qk_fwd<T, LPR, true, HU>>(a, fwd_smem<T, HU>(), grid, s)
               : go<k_qk_fwd<T, LPR, false, HU>>(a, fwd_smem<T, HU>(), grid, s);
}
template <typename T, typename G, int LPR, int HU>
cudaError_t go_bwd(const QkDev& a, bool split, unsigned grid, cudaStream_t s) {
  return split ? go<k_qk_bwd<T, G, LPR, true, HU>>(a, bwd_smem<T, G, HU>(), grid, s)
               : go<k_qk_bwd<T, G, LPR, false, HU>>(a, bwd_smem<T, G, HU>(), grid, s);
}
template <typename T, int LPR>
cudaError_t run_fwd(const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  constexpr int HU = LPR < 8 ? 1 : sizeof(T) == 2 ? 3 : 2;
  return hu > 1 ? go_fwd<T, LPR, HU>(a, split, grid, s) : go_fwd<T, LPR, 1>(a, split, grid, s);
}
template <typename T, typename G, int LPR>
cudaError_t run_bwd(const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  constexpr int HU = LPR < 8 ? 1 : sizeof(T) == 2 ? 3 : 2;
  return hu > 1 ? go_bwd<T, G, LPR, HU>(a, split, grid, s) : go_bwd<T, G, LPR, 1>(a, split, grid, s);
}
template <typename T>
cudaError_t fwd_lanes(int lpr, const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  switch (lpr) {
    case 2: return run_fwd<T, 2>(a, split, hu, grid, s);
    case 4: return run_fwd<T, 4>(a, split, hu, grid, s);
    case 8: return run_fwd<T, 8>(a, split, hu, grid, s);
    case 16: return run_fwd<T, 16>(a, split, hu, grid, s);
    default: return run_fwd<T, 32>(a, split, hu, grid, s);
  }
}
template <typename T, typename G>
cudaError_t bwd_lanes(int lpr, const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  switch (lpr) {
    case 2: return run_bwd<T, G, 2>(a, split, hu, grid, s);
    case 4: return run_bwd<T, G, 4>(a, split, hu, grid, s);
    case 8: return run_bwd<T, G, 8>(a, split, hu, grid, s);
    case 16: return run_bwd<T, G, 16>(a, split, hu, grid, s);
    default: return run_bwd<T, G, 32>(a, split, hu, grid, s);
  }
}

}  // namespace

size_t qk_bwd_workspace(const vdn_qk_cfg& c) {
  int hc, tpi, nch;
  qk_slots(c, heads_per_thread(c, c.dtype == VDN_F32), &hc, &tpi, &nch);
  return (size_t)qk_max_blocks(nch) * (c.per_head ? c.Hq + c.Hk : 2 * nch) * c.d * sizeof(float);
}

cudaError_t launch_qk_fwd(const vdn_qk_cfg& c, const vdn_qk_args& in, cudaStream_t s) {
  QkDev a = device_args(c, in);
  const int hu = heads_per_thread(c, c.dtype == VDN_F32);
  if (!plan(c, a, hu, 3)) return cudaErrorInvalidDevice;
  const unsigned grid = (unsigned)a.gx * a.nch;
  const bool split = c.pairing == VDN_PAIR_SPLIT;
  return c.dtype == VDN_BF16 ? fwd_lanes<__nv_bfloat16>(lanes_per_row(c.d), a, split, hu, grid, s)
                             : fwd_lanes<float>(lanes_per_row(c.d), a, split, hu, grid, s);
}

cudaError_t launch_qk_bwd(const vdn_qk_cfg& c, const vdn_qk_args& in, const vdn_qk_grads& g, cudaStream_t s) {
  QkDev a = device_args(c, in);
  const int hu = heads_per_thread(c, c.dtype == VDN_F32);
  if (!plan(c, a, hu, 2)) return cudaErrorInvalidDevice;
  a.qo = g.dq; a.ko = g.dk; a.gq = g.dq_out; a.gk = g.dk_out;
  const bool want = g.dwq != nullptr || g.dwk != nullptr;
  a.part = want ? static_cast<float*>(g.workspace) : nullptr;
  const unsigned grid = (unsigned)a.gx * a.nch;
  const bool split = c.pairing == VDN_PAIR_SPLIT;
  const int lpr = lanes_per_row(c.d);
  const cudaError_t e = c.dtype == VDN_F32        ? bwd_lanes<float, float>(lpr, a, split, hu, grid, s)
                        : c.grad_dtype == VDN_F32 ? bwd_lanes<__nv_bfloat16, float>(lpr, a, split, hu, grid, s)
                                                  : bwd_lanes<__nv_bfloat16, __nv_bfloat16>(lpr, a, split, hu, grid, s);
  if (e != cudaSuccess || !want) return e;
  const int sets = c.per_head ? a.Ht : 2;
  k_qk_dw<<<dim3((c.d + 31) / 32, sets), 1024, 0, s>>>(a.part, g.dwq, c.Hk > 0 ? g.dwk : nullptr, c.per_head ? a.gx : a.gx * a.nch,
                                                       sets, c.per_head ? c.Hq : 1, c.d);
  return cudaGetLastError();
}

}  // namespace vdn
