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
// in registers.  With few heads a thread has U tokens in flight instead.
// The weights' gradient: a block adds its threads' sums in shared memory and
// writes them (fp32), a second kernel adds the blocks', both in a fixed order,
// so results do not depend on timing.
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
  int Hq, Ht, d, rot, axes, rows;  // rows: table rows
  int sec0, sec01;                 // first pair of axis 1 and of axis 2
  int per_head, vec;               // vec: no lane's pairs straddle two axes
  int hc, tpi, nch, gx;            // head slots of a block, tokens per block step, head chunks (of HU hc heads), blocks per chunk
  float eps;
};

// 8 consecutive elements as stored: one 16-byte vector (bf16) or two (fp32)
template <typename T> struct Raw { uint4 v[sizeof(T) / 2]; };

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T> __device__ __forceinline__ Raw<T> zero_raw() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}
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
  float cs[SPLIT ? 8 : 4], sn[SPLIT ? 8 : 4];

  __device__ __forceinline__ Turn(const QkDev& a, int li, int lane) {
    const int c = 8 * li, half = a.rot >> 1;
    on = c < a.rot;
    second = SPLIT && on && c >= half;
    pair0 = SPLIT ? (second ? c - half : c) : (c >> 1);
    partner = !SPLIT || !on ? lane : (second ? lane - half / 8 : lane + half / 8);
#pragma unroll
    for (int i = 0; i < (SPLIT ? 8 : 4); ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
  }
  // the angles of one token (its positions are inside the table)
  __device__ __forceinline__ void angles(const QkDev& a, const int (&p)[3]) {
    if (!on) return;
    const int half = a.rot >> 1;
    constexpr int NP = SPLIT ? 8 : 4;
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
  bool active;
  __device__ __forceinline__ Slot(const QkDev& a) {
    const int lane = threadIdx.x & 31, slot = threadIdx.x / LPR;
    li = lane % LPR;
    ti = slot / a.hc;
    head0 = (int)(blockIdx.x % a.nch) * a.hc * HU + slot % a.hc;
    active = ti < a.tpi && 8 * li < a.d;
  }
};

// One head of a thread: where its columns lie in the inputs and outputs, and the norm's weights there.
template <typename T>
struct Head {
  const T* x;
  T* o;
  long long off, xs, os;  // offset within a token of a dense [tokens, H, d] tensor, token strides of input and output
  float w[8];
  bool on, isq;
  __device__ __forceinline__ void init(const QkDev& a, int head, int li, bool active) {
    on = active && head < a.Ht;
    isq = head < a.Hq;
    const int h = isq ? head : head - a.Hq;
    off = (long long)h * a.d + 8 * li;
    xs = isq ? a.qs : a.ks;
    os = (long long)(isq ? a.Hq : a.Ht - a.Hq) * a.d;
    x = static_cast<const T*>(isq ? a.q : a.k) + off;
    o = static_cast<T*>(isq ? a.qo : a.ko) + off;
    const float* p = isq ? a.wq : a.wk;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = on && p != nullptr ? __ldg(p + (a.per_head ? off : 8 * li) + i) : 1.f;
  }
};

template <typename T, int LPR, bool SPLIT, int HU, int U>
__global__ void __launch_bounds__(kThreads, 3) k_qk_fwd(const QkDev a) {
  const Slot<LPR, HU> s(a);
  Head<T> hd[HU];
#pragma unroll
  for (int i = 0; i < HU; ++i) hd[i].init(a, s.head0 + i * a.hc, s.li, s.active);
  Turn<LPR, SPLIT> turn(a, s.li, threadIdx.x & 31);
  const long long step = (long long)a.gx * a.tpi;
  const float inv_d = 1.0f / (float)a.d;
  for (long long base = (long long)(blockIdx.x / a.nch) * a.tpi; base < a.tokens; base += U * step) {
    Raw<T> raw[U][HU];
    int p[U][3];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = base + u * step + s.ti;
      on[u] = s.active && t < a.tokens;
#pragma unroll
      for (int i = 0; i < HU; ++i) raw[u][i] = on[u] && hd[i].on ? load_raw(hd[i].x + t * hd[i].xs) : zero_raw<T>();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) on[u] = on[u] && positions(a, base + u * step + s.ti, p[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = base + u * step + s.ti;
      if (on[u]) turn.angles(a, p[u]);
#pragma unroll
      for (int i = 0; i < HU; ++i) {
        float x[8], ss = 0.f;
        expand(raw[u][i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        const float rstd = rsqrtf(fmaf(row_sum<LPR>(ss), inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= rstd * hd[i].w[e];
        turn.apply(x, 1.f);
        if (on[u] && hd[i].on) store8(hd[i].o + t * hd[i].os, x);
      }
    }
  }
}

template <typename T, typename G, int LPR, bool SPLIT, int HU, int U>
__global__ void __launch_bounds__(kThreads, 2) k_qk_bwd(const QkDev a) {
  const Slot<LPR, HU> s(a);
  Head<T> hd[HU];
  float acc[HU][8];
#pragma unroll
  for (int i = 0; i < HU; ++i) {
    hd[i].init(a, s.head0 + i * a.hc, s.li, s.active);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  }
  Turn<LPR, SPLIT> turn(a, s.li, threadIdx.x & 31);
  const long long step = (long long)a.gx * a.tpi;
  const float inv_d = 1.0f / (float)a.d;
  for (long long base = (long long)(blockIdx.x / a.nch) * a.tpi; base < a.tokens; base += U * step) {
    Raw<T> rx[U][HU];
    Raw<G> rg[U][HU];
    int p[U][3];
    bool on[U], in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = base + u * step + s.ti;
      in[u] = s.active && t < a.tokens;
#pragma unroll
      for (int i = 0; i < HU; ++i) {
        const bool ld = in[u] && hd[i].on;
        rx[u][i] = ld ? load_raw(hd[i].x + t * hd[i].xs) : zero_raw<T>();
        rg[u][i] = ld ? load_raw(static_cast<const G*>(hd[i].isq ? a.gq : a.gk) + hd[i].off + t * hd[i].os) : zero_raw<G>();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) on[u] = in[u] && positions(a, base + u * step + s.ti, p[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = base + u * step + s.ti;
      if (on[u]) turn.angles(a, p[u]);
#pragma unroll
      for (int i = 0; i < HU; ++i) {
        float x[8], g[8], ss = 0.f, dot = 0.f;
        expand(rx[u][i], x);
        expand(rg[u][i], g);
        if (!on[u]) {
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
        if (in[u] && hd[i].on) store8(hd[i].o + t * hd[i].os, g);
      }
    }
  }
  if (a.part == nullptr) return;
  // the block's sums: columns c of the LPR lanes' 8 LPR, slot after slot
  __shared__ float buf[kThreads * 8];
  constexpr int W = 8 * LPR, SLOTS = kThreads / LPR;
  const int blk = blockIdx.x / a.nch, chunk = blockIdx.x % a.nch;
  float sum[2] = {0.f, 0.f};  // shared weights: queries, keys
#pragma unroll
  for (int i = 0; i < HU; ++i) {
    __syncthreads();
    store8(buf + threadIdx.x * 8, acc[i]);
    __syncthreads();
    if (a.per_head) {
      for (int j = threadIdx.x; j < a.hc * W; j += kThreads) {
        const int hs = j / W, c = j % W, head = chunk * a.hc * HU + hs + i * a.hc;
        float v = 0.f;
        for (int t = 0; t < a.tpi; ++t) v += buf[(t * a.hc + hs) * W + c];
        if (head < a.Ht && c < a.d) a.part[((long long)blk * a.Ht + head) * a.d + c] = v;
      }
    } else if (threadIdx.x < W) {
      for (int sl = 0; sl < SLOTS && sl < a.hc * a.tpi; ++sl) {
        const int head = chunk * a.hc * HU + sl % a.hc + i * a.hc;
        if (head < a.Ht) sum[head < a.Hq ? 0 : 1] += buf[sl * W + threadIdx.x];
      }
    }
  }
  if (!a.per_head && threadIdx.x < W && threadIdx.x < a.d) {
#pragma unroll
    for (int k = 0; k < 2; ++k) a.part[(((long long)blk * a.nch + chunk) * 2 + k) * a.d + threadIdx.x] = sum[k];
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
  const long long steps = (c.tokens + a.tpi - 1) / a.tpi;
  long long gx = (long long)resident * sms / a.nch;
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
  a.Hq = c.Hq; a.Ht = c.Hq + c.Hk; a.d = c.d; a.rot = c.rot; a.axes = c.axes; a.rows = c.table_rows;
  a.sec0 = c.axes > 1 ? c.sections[0] : 1 << 30;
  a.sec01 = c.axes > 2 ? c.sections[0] + c.sections[1] : 1 << 30;
  const int grain = c.pairing == VDN_PAIR_SPLIT ? 8 : 4;
  a.vec = (c.axes < 2 || a.sec0 % grain == 0) && (c.axes < 3 || a.sec01 % grain == 0);
  a.per_head = c.per_head;
  a.eps = c.eps > 0.f ? c.eps : 1e-6f;
  return a;
}

template <typename T, int LPR>
void run_fwd(const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  constexpr int HU = LPR < 8 ? 1 : sizeof(T) == 2 ? 3 : 2, U = sizeof(T) == 2 ? 4 : 2;
  if (hu > 1) {
    if (split) k_qk_fwd<T, LPR, true, HU, 1><<<grid, kThreads, 0, s>>>(a);
    else k_qk_fwd<T, LPR, false, HU, 1><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (split) k_qk_fwd<T, LPR, true, 1, U><<<grid, kThreads, 0, s>>>(a);
    else k_qk_fwd<T, LPR, false, 1, U><<<grid, kThreads, 0, s>>>(a);
  }
}
template <typename T, typename G, int LPR>
void run_bwd(const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  constexpr int HU = LPR < 8 ? 1 : sizeof(T) == 2 ? 3 : 2, U = sizeof(T) == 2 ? 3 : 2;
  if (hu > 1) {
    if (split) k_qk_bwd<T, G, LPR, true, HU, 1><<<grid, kThreads, 0, s>>>(a);
    else k_qk_bwd<T, G, LPR, false, HU, 1><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (split) k_qk_bwd<T, G, LPR, true, 1, U><<<grid, kThreads, 0, s>>>(a);
    else k_qk_bwd<T, G, LPR, false, 1, U><<<grid, kThreads, 0, s>>>(a);
  }
}
template <typename T>
void fwd_lanes(int lpr, const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
  switch (lpr) {
    case 2: return run_fwd<T, 2>(a, split, hu, grid, s);
    case 4: return run_fwd<T, 4>(a, split, hu, grid, s);
    case 8: return run_fwd<T, 8>(a, split, hu, grid, s);
    case 16: return run_fwd<T, 16>(a, split, hu, grid, s);
    default: return run_fwd<T, 32>(a, split, hu, grid, s);
  }
}
template <typename T, typename G>
void bwd_lanes(int lpr, const QkDev& a, bool split, int hu, unsigned grid, cudaStream_t s) {
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
  if (c.dtype == VDN_BF16) fwd_lanes<__nv_bfloat16>(lanes_per_row(c.d), a, split, hu, grid, s);
  else fwd_lanes<float>(lanes_per_row(c.d), a, split, hu, grid, s);
  return cudaGetLastError();
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
  if (c.dtype == VDN_F32) bwd_lanes<float, float>(lpr, a, split, hu, grid, s);
  else if (c.grad_dtype == VDN_F32) bwd_lanes<__nv_bfloat16, float>(lpr, a, split, hu, grid, s);
  else bwd_lanes<__nv_bfloat16, __nv_bfloat16>(lpr, a, split, hu, grid, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !want) return e;
  const int sets = c.per_head ? a.Ht : 2;
  k_qk_dw<<<dim3((c.d + 31) / 32, sets), 1024, 0, s>>>(a.part, g.dwq, c.Hk > 0 ? g.dwk : nullptr, c.per_head ? a.gx : a.gx * a.nch,
                                                       sets, c.per_head ? c.Hq : 1, c.d);
  return cudaGetLastError();
}

}  // namespace vdn
