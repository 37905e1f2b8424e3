// C ABI entry points of the layer's operators around the core: norm and
// rotation of queries and keys, cross-attention with lengths, the 8-bit
// integer linear layer.  Argument validation and dispatch; the kernels are in
// vdn_qk_rope.cu, vdn_xattn*.cu, vdn_int8.cu and vdn_gemm_tc.cu.
#include <atomic>
#include <cstdint>

#include "vdn_xattn.h"

namespace vdn {
namespace {

constexpr size_t kAlign = 256;
constexpr long long kMax31 = 1LL << 31;
constexpr unsigned long long kMostWaitCycles = 2000000000ULL;  // the default limit of a bounded wait
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool ok_ptr(const void* p, size_t a) { return p != nullptr && aligned(p, a); }
bool float_type(int t) { return t == VDN_F32 || t == VDN_BF16; }
size_t size_of(int t) { return t == VDN_BF16 ? 2 : 4; }

// a token stride: 0 (dense), or at least the dense row and a multiple of 16 bytes
bool stride_ok(long long s, long long row, int dtype) {
  return s == 0 || (s >= row && s < (1LL << 40) && (s * (long long)size_of(dtype)) % 16 == 0);
}

// ------------------------------------------------------- norm and rotation
vdn_status check_qk(const vdn_qk_cfg* c) {
  if (!c) return VDN_ERR_INVALID_ARG;
  if (c->tokens < 1 || c->Hq < 1 || c->Hk < 0 || c->d < 8 || c->d > 256 || c->d % 8) return VDN_ERR_INVALID_ARG;
  if (c->rot < 0 || c->rot > c->d || c->rot % 16) return VDN_ERR_INVALID_ARG;
  if (c->pairing != VDN_PAIR_INTERLEAVED && c->pairing != VDN_PAIR_SPLIT) return VDN_ERR_INVALID_ARG;
  if (c->axes < 1 || c->axes > 3 || c->table_rows < (c->rot > 0 ? 1 : 0)) return VDN_ERR_INVALID_ARG;
  long long pairs = 0;
  for (int i = 0; i < c->axes; ++i) {
    if (c->sections[i] < 0) return VDN_ERR_INVALID_ARG;
    pairs += c->sections[i];
  }
  if (pairs != c->rot / 2) return VDN_ERR_INVALID_ARG;
  if ((c->per_head != 0 && c->per_head != 1) || (c->zero_skipped != 0 && c->zero_skipped != 1)) return VDN_ERR_INVALID_ARG;
  if (!float_type(c->dtype) || !float_type(c->grad_dtype)) return VDN_ERR_INVALID_ARG;
  if (!(c->eps == c->eps)) return VDN_ERR_INVALID_ARG;
  if (!stride_ok(c->q_stride, (long long)c->Hq * c->d, c->dtype) ||
      !stride_ok(c->k_stride, (long long)c->Hk * c->d, c->dtype))
    return VDN_ERR_INVALID_ARG;
  if ((long long)c->Hq + c->Hk > 65535) return VDN_ERR_UNSUPPORTED;
  return VDN_OK;
}

vdn_status check_qk_args(const vdn_qk_cfg* c, const vdn_qk_args* a) {
  if (!a || !ok_ptr(a->q, 16) || !aligned(a->wq, 4) || !aligned(a->wk, 4) || !aligned(a->pos, 4)) return VDN_ERR_INVALID_ARG;
  if (c->Hk > 0 && !ok_ptr(a->k, 16)) return VDN_ERR_INVALID_ARG;
  if (c->rot > 0 ? !ok_ptr(a->table, 16) : a->table != nullptr) return VDN_ERR_INVALID_ARG;
  if (!a->pos && (c->axes != 1 || (c->rot > 0 && c->table_rows < c->tokens))) return VDN_ERR_INVALID_ARG;
  return VDN_OK;
}

// ---------------------------------------------------------- cross-attention
vdn_status check_x(const vdn_xattn_cfg* c) {
  if (!c) return VDN_ERR_INVALID_ARG;
  if (c->B < 1 || c->Tq < 1 || c->L < 1 || c->H < 1 || c->Hkv < 1 || c->d < 1 || c->H % c->Hkv) return VDN_ERR_INVALID_ARG;
  if (!float_type(c->dtype) || !(c->scale == c->scale)) return VDN_ERR_INVALID_ARG;
  const long long row = (long long)c->Hkv * c->d;
  if (!stride_ok(c->k_stride, row, c->dtype) || !stride_ok(c->v_stride, row, c->dtype)) return VDN_ERR_INVALID_ARG;
  if (c->d != 32 && c->d != 64 && c->d != 128) return VDN_ERR_UNSUPPORTED;
  // token coordinates of the tensor maps, with a tile of overhang, and blocks of a launch
  if ((long long)c->B * c->Tq >= kMax31 - 512 || (long long)c->B * c->L >= kMax31 - 512) return VDN_ERR_UNSUPPORTED;
  const double items = (double)c->B * c->H * (c->Tq / 64 + 1), kitems = (double)c->B * c->Hkv * (c->L / 64 + 1);
  if (items >= 2147483647.0 || kitems >= 2147483647.0 || (double)c->B * c->Tq * c->H >= 8.0 * 2147483647.0)
    return VDN_ERR_UNSUPPORTED;
  return VDN_OK;
}

XDims xdims(const vdn_xattn_cfg* c, const vdn_xattn_args* a) {
  XDims d;
  d.B = c->B; d.Tq = c->Tq; d.L = c->L; d.H = c->H; d.Hkv = c->Hkv; d.G = c->H / c->Hkv; d.d = c->d;
  d.scale = c->scale > 0.f ? c->scale : 1.0f / sqrtf((float)c->d);
  d.ks = c->k_stride ? c->k_stride : (long long)c->Hkv * c->d;
  d.vs = c->v_stride ? c->v_stride : (long long)c->Hkv * c->d;
  d.kv_len = a ? a->kv_len : nullptr;
  return d;
}

vdn_status check_x_args(const vdn_xattn_cfg* c, const vdn_xattn_args* a, size_t need) {
  if (!a || !ok_ptr(a->q, 16) || !ok_ptr(a->k, 16) || !ok_ptr(a->v, 16) || !ok_ptr(a->y, 16)) return VDN_ERR_INVALID_ARG;
  if (!aligned(a->kv_len, 4) || !aligned(a->lse, 4)) return VDN_ERR_INVALID_ARG;
  if (!a->workspace || !aligned(a->workspace, kAlign) || a->workspace_bytes < need) return VDN_ERR_WORKSPACE;
  return VDN_OK;
}

// set by vdn_debug_set_layer_wait_limit, read at every launch
std::atomic<long long> g_wait_limit{0};

XArgs xargs(const vdn_xattn_args* a, const vdn_xattn_grads* g) {
  XArgs x{};
  x.q = a->q; x.k = a->k; x.v = a->v; x.y = a->y; x.lse = a->lse;
  if (g) {
    x.dy = g->dy; x.dq = g->dq; x.dk = g->dk; x.dv = g->dv;
  }
  x.status = static_cast<uint32_t*>(a->workspace);
  x.scratch = static_cast<char*>(a->workspace) + kAlign;
  x.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  return x;
}

bool few_rows(const vdn_xattn_cfg* c) { return c->dtype == VDN_BF16 && xattn_few_supported(xdims(c, nullptr)); }
bool on_tensor_cores(const vdn_xattn_cfg* c) { return c->dtype == VDN_BF16 && xattn_tc_supported(xdims(c, nullptr)); }

// --------------------------------------------------------------- 8-bit layer
vdn_status check_int8(const vdn_int8_cfg* c) {
  if (!c) return VDN_ERR_INVALID_ARG;
  if (c->M < 1 || c->K < 16 || c->N < 16 || c->K % 16 || c->N % 16 || c->K > 131056) return VDN_ERR_INVALID_ARG;
  if (!float_type(c->out_dtype) || !(float_type(c->x_dtype) || c->x_dtype == VDN_I8)) return VDN_ERR_INVALID_ARG;
  return VDN_OK;
}

size_t int8_scratch(const vdn_int8_cfg& c) {
  if (c.x_dtype == VDN_I8 || int8_few_supported(c.M, c.K, c.N)) return 0;
  return up((size_t)c.M * c.K) + up((size_t)c.M * sizeof(float));
}

// a call's two status words, on the host
vdn_status read_status(const void* words, vdn_stream_t stream, unsigned* where) {
  if (!words) return VDN_ERR_INVALID_ARG;
  uint32_t host[2] = {0, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(host, words, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess) return VDN_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return VDN_ERR_CUDA;
  if (where) *where = host[1];
  return host[0] ? VDN_ERR_TIMEOUT : VDN_OK;
}

}  // namespace
}  // namespace vdn

using namespace vdn;

extern "C" {

vdn_status vdn_qk_norm_rope(const vdn_qk_cfg* cfg, const vdn_qk_args* args, vdn_stream_t stream) {
  vdn_status st = check_qk(cfg);
  if (st != VDN_OK) return st;
  if ((st = check_qk_args(cfg, args)) != VDN_OK) return st;
  if (!ok_ptr(args->q_out, 16) || (cfg->Hk > 0 && !ok_ptr(args->k_out, 16))) return VDN_ERR_INVALID_ARG;
  return launch_qk_fwd(*cfg, *args, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

size_t vdn_qk_norm_rope_bwd_workspace_size(const vdn_qk_cfg* cfg) {
  return check_qk(cfg) == VDN_OK ? qk_bwd_workspace(*cfg) : 0;
}

vdn_status vdn_qk_norm_rope_bwd(const vdn_qk_cfg* cfg, const vdn_qk_args* args, const vdn_qk_grads* g,
                                vdn_stream_t stream) {
  vdn_status st = check_qk(cfg);
  if (st != VDN_OK) return st;
  if (cfg->dtype == VDN_F32 && cfg->grad_dtype != VDN_F32) return VDN_ERR_INVALID_ARG;
  if ((st = check_qk_args(cfg, args)) != VDN_OK) return st;
  if (!g || !ok_ptr(g->dq_out, 16) || !ok_ptr(g->dq, 16) || !aligned(g->dwq, 4) || !aligned(g->dwk, 4))
    return VDN_ERR_INVALID_ARG;
  if (cfg->Hk > 0 && (!ok_ptr(g->dk_out, 16) || !ok_ptr(g->dk, 16))) return VDN_ERR_INVALID_ARG;
  if ((g->dwq || g->dwk) && (!g->workspace || !aligned(g->workspace, kAlign) || g->workspace_bytes < qk_bwd_workspace(*cfg)))
    return VDN_ERR_WORKSPACE;
  return launch_qk_bwd(*cfg, *args, *g, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

size_t vdn_cross_attn_workspace_size(const vdn_xattn_cfg* cfg) {
  if (check_x(cfg) != VDN_OK) return 0;
  return kAlign + (!few_rows(cfg) && on_tensor_cores(cfg) ? up(xattn_tc_scratch(xdims(cfg, nullptr))) : 0);
}

size_t vdn_cross_attn_bwd_workspace_size(const vdn_xattn_cfg* cfg) {
  if (check_x(cfg) != VDN_OK) return 0;
  const XDims d = xdims(cfg, nullptr);
  return kAlign + up(on_tensor_cores(cfg) ? xattn_tc_bwd_scratch(d) : xattn_simt_bwd_scratch(d));
}

int vdn_cross_attn_impl(const vdn_xattn_cfg* cfg, int backward) {
  if (check_x(cfg) != VDN_OK) return -1;
  return !backward && few_rows(cfg) ? 2 : on_tensor_cores(cfg) ? 1 : 0;
}

vdn_status vdn_cross_attn(const vdn_xattn_cfg* cfg, const vdn_xattn_args* args, vdn_stream_t stream) {
  vdn_status st = check_x(cfg);
  if (st != VDN_OK) return st;
  if ((st = check_x_args(cfg, args, vdn_cross_attn_workspace_size(cfg))) != VDN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const XDims d = xdims(cfg, args);
  const XArgs a = xargs(args, nullptr);
  if (few_rows(cfg)) return launch_xattn_few(d, a, s) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
  if (on_tensor_cores(cfg)) return launch_xattn_tc(d, a, s) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
  return launch_xattn_simt(d, a, cfg->dtype == VDN_BF16, s) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

vdn_status vdn_cross_attn_bwd(const vdn_xattn_cfg* cfg, const vdn_xattn_args* args, const vdn_xattn_grads* g,
                              vdn_stream_t stream) {
  vdn_status st = check_x(cfg);
  if (st != VDN_OK) return st;
  if ((st = check_x_args(cfg, args, vdn_cross_attn_bwd_workspace_size(cfg))) != VDN_OK) return st;
  if (!args->lse || !g || !ok_ptr(g->dy, 16) || !ok_ptr(g->dq, 16) || !ok_ptr(g->dk, 16) || !ok_ptr(g->dv, 16))
    return VDN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const XDims d = xdims(cfg, args);
  const XArgs a = xargs(args, g);
  if (on_tensor_cores(cfg)) return launch_xattn_tc_bwd(d, a, s) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
  return launch_xattn_simt_bwd(d, a, cfg->dtype == VDN_BF16, s) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

vdn_status vdn_cross_attn_device_status(const void* workspace, vdn_stream_t stream, unsigned* where) {
  return read_status(workspace, stream, where);
}

vdn_status vdn_debug_set_layer_wait_limit(unsigned long long cycles) {
  if (cycles > kMostWaitCycles) return VDN_ERR_INVALID_ARG;
  g_wait_limit.store((long long)cycles, std::memory_order_relaxed);
  return VDN_OK;
}

vdn_status vdn_quantize_int8(const void* x, int x_dtype, int rows, int cols, void* q, float* scale, vdn_stream_t stream) {
  if (!ok_ptr(x, 16) || !ok_ptr(q, 16) || !ok_ptr(scale, 4) || !float_type(x_dtype)) return VDN_ERR_INVALID_ARG;
  if (rows < 1 || cols < 16 || cols % 16) return VDN_ERR_INVALID_ARG;
  return launch_quantize_int8(x, x_dtype, rows, cols, q, scale, nullptr, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? VDN_OK : VDN_ERR_CUDA;
}

size_t vdn_linear_int8_workspace_size(const vdn_int8_cfg* cfg) { return check_int8(cfg) == VDN_OK ? int8_scratch(*cfg) : 0; }

int vdn_linear_int8_impl(const vdn_int8_cfg* cfg) {
  if (check_int8(cfg) != VDN_OK) return -1;
  return int8_few_supported(cfg->M, cfg->K, cfg->N) ? 0 : s8_tile(cfg->M, cfg->N);
}

vdn_status vdn_linear_int8(const vdn_int8_cfg* cfg, const vdn_int8_args* args, vdn_stream_t stream) {
  vdn_status st = check_int8(cfg);
  if (st != VDN_OK) return st;
  if (!args || !ok_ptr(args->x, 16) || !ok_ptr(args->w, 16) || !ok_ptr(args->w_scale, 16) || !ok_ptr(args->out, 16) ||
      !aligned(args->bias, 16) || !aligned(args->status, 4))
    return VDN_ERR_INVALID_ARG;
  if (cfg->x_dtype == VDN_I8 ? !ok_ptr(args->x_scale, 4) : args->x_scale != nullptr) return VDN_ERR_INVALID_ARG;
  const size_t need = int8_scratch(*cfg);
  if (need && (!args->workspace || !aligned(args->workspace, kAlign) || args->workspace_bytes < need)) return VDN_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (int8_few_supported(cfg->M, cfg->K, cfg->N))
    return launch_int8_few(*cfg, *args, s) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
  uint32_t* status = args->status ? args->status : status_of_proj();
  if (!status) return VDN_ERR_CUDA;
  const void* codes = args->x;
  const float* scale = args->x_scale;
  if (cfg->x_dtype != VDN_I8) {
    char* ws = static_cast<char*>(args->workspace);
    float* sc = reinterpret_cast<float*>(ws + up((size_t)cfg->M * cfg->K));
    if (launch_quantize_int8(args->x, cfg->x_dtype, cfg->M, cfg->K, ws, sc, status, s) != cudaSuccess) return VDN_ERR_CUDA;
    codes = ws;
    scale = sc;
  }
  return gemm_s8(cfg->M, cfg->K, cfg->N, cfg->out_dtype, codes, scale, args->w, args->w_scale, args->bias, args->out,
                 status, cfg->x_dtype == VDN_I8, g_wait_limit.load(std::memory_order_relaxed), s);
}

vdn_status vdn_linear_int8_device_status(const unsigned* status, vdn_stream_t stream, unsigned* where) {
  return read_status(status, stream, where);
}

}  // extern "C"
