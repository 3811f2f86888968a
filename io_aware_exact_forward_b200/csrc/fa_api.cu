// fa_api.cu -- the C ABI of libfa (declared in include/fa.h): argument
// checks, TMA descriptor set-up and kernel launches.  Every kernel of the
// library is compiled in this one translation unit.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "fa_status.h"
#include "fa_ptx.cuh"
#include "fa_fwd.cuh"
#include "fa_bwd.cuh"
#include "fa_bwd_dq.cuh"
#include "fa_decode.cuh"
#include "fa_rope.cuh"
#include "fa_kv4.cuh"

namespace fa {

// Limit for every bounded wait inside the kernels.  Far above any legitimate
// wait (the longest kernels run for tens of milliseconds).
static constexpr unsigned long long kWaitLimitNs = 4000000000ull;

// ---------------------------------------------------------------------------
// Driver entry point for TMA descriptors (resolved through the runtime, so
// the library links no driver stub and loads on machines without a GPU).
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// 4-D bf16 tensor [n3][n2][n1][n0] (n0 contiguous) with box {64, 1, box_rows, 1}
// along (n0, n1, n2, n3) and the 128-byte swizzle, or no swizzle when
// `swizzle` is false (then box_inner elements along n0).
// elt = 2: bf16 elements; elt = 1: 8-bit (E4M3) elements.
static int make_tmap_4d(CUtensorMap* m, const void* base, uint64_t n0, uint64_t n1, uint64_t n2,
                        uint64_t n3, uint32_t box_inner, uint32_t box_rows, bool swizzle, int elt = 2) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return FA_ERR_CUDA;
  const cuuint64_t dims[4] = {n0, n1, n2, n3};
  const cuuint64_t strides[3] = {n0 * elt, n0 * n1 * elt, n0 * n1 * n2 * elt};
  const cuuint32_t box[4] = {box_inner, 1, box_rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, elt == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                  const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// 4-D fp32 tensor [n3][n2][n1][n0] with box {32, 1, 128, 1} and the 128-byte
// swizzle (the dQ accumulator, written by bulk tensor reduce-add).
static int make_tmap_f32_4d(CUtensorMap* m, const void* base, uint64_t n0, uint64_t n1, uint64_t n2,
                            uint64_t n3) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return FA_ERR_CUDA;
  const cuuint64_t dims[4] = {n0, n1, n2, n3};
  const cuuint64_t strides[3] = {n0 * 4, n0 * n1 * 4, n0 * n1 * n2 * 4};
  const cuuint32_t box[4] = {32, 1, 128, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Per-device set-up: architecture check and shared-memory opt-in, once.
// ---------------------------------------------------------------------------
static constexpr int kMaxDevices = 64;

template <typename Fn>
static int set_smem(Fn* kernel, int bytes) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// The forward kernels move registers between warpgroups with setmaxnreg;
// the split adds up only if the block is launched with exactly the per-thread
// count it was planned for (an increase beyond the launch's pool would wait
// forever), so a build that came out differently is refused, not launched.
template <int D, bool F8, bool DROP, bool SINK = false>
static int fwd_setup_one() {
  using C = FwdCfg<D, F8, DROP>;
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(fa_fwd_kernel<D, F8, DROP, SINK>)) != cudaSuccess)
    return FA_ERR_CUDA;
  if (a.numRegs != C::REG_LAUNCH) return FA_ERR_UNSUPPORTED;
  return set_smem(fa_fwd_kernel<D, F8, DROP, SINK>, C::SMEM_BYTES);
}

template <int D, int G>
static int decode_setup_one() {
  int st = set_smem(fa_decode_split_kernel<D, G>, DecCfg<D, G>::SMEM_BYTES);
  if (!st) st = set_smem(fa_decode_split_kernel<D, G, true>, DecCfg<D, G>::SMEM_BYTES);
  if (!st) st = set_smem(fa_kv4_split_kernel<D, G>, Kv4Cfg<D, G>::SMEM_BYTES);
  return st;
}

static int decode_setup() {
  int st = FA_OK;
  if (!st) st = decode_setup_one<64, 1>();
  if (!st) st = decode_setup_one<64, 2>();
  if (!st) st = decode_setup_one<64, 4>();
  if (!st) st = decode_setup_one<64, 8>();
  if (!st) st = decode_setup_one<128, 1>();
  if (!st) st = decode_setup_one<128, 2>();
  if (!st) st = decode_setup_one<128, 4>();
  if (!st) st = decode_setup_one<128, 8>();
  return st;
}

static int device_setup_impl() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  if (major != 10 || minor != 0) return FA_ERR_UNSUPPORTED;
  int st = FA_OK;
  if (!st) st = fwd_setup_one<64, false, false>();
  if (!st) st = fwd_setup_one<128, false, false>();
  if (!st) st = fwd_setup_one<128, true, false>();
  if (!st) st = fwd_setup_one<64, false, true>();
  if (!st) st = fwd_setup_one<128, false, true>();
  if (!st) st = fwd_setup_one<64, false, false, true>();
  if (!st) st = fwd_setup_one<128, false, false, true>();
  if (!st) st = bwd_setup();
  if (!st) st = bwd_dq_setup();
  if (!st) st = decode_setup();
  return st;
}

static int device_setup() {
  static int state[kMaxDevices];  // 0 = not done, else status + 1
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(mu);
  if (state[dev] == 0) state[dev] = device_setup_impl() + 1;
  return state[dev] - 1;
}

// Persistent decode grid: CTAs per SM.
static constexpr int kDecodeCtasPerSm = 2;

// Number of SMs of the current device (persistent grids use one CTA per SM).
static int sm_count(int* n) {
  static int cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  if (cache[dev] == 0) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return FA_ERR_CUDA;
    cache[dev] = v;
  }
  *n = cache[dev];
  return FA_OK;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int launch_status() {
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Launches a kernel that calls pdl_wait() behind one that calls pdl_launch().
template <typename P>
static int launch_after(void (*kernel)(P), unsigned blocks, unsigned threads, cudaStream_t s, const P& p) {
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Checks shared by the prefill entry points.
static int check_prefill(int B, int Hq, int Hkv, int Tq, int Tk, int d, float scale, int causal) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Tq < 0 || Tk < 0) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // Tensor-map extents are 32-bit and row/item indices are int; (batch, KV
  // head) pairs index the backward's second grid dimension (at most 65535).
  if ((int64_t)Tq > (1 << 30) || (int64_t)Tk > (1 << 30) || (int64_t)B * Hq > 65535 ||
      (int64_t)B * Hq * ((Tq + 255) / 256) > (1ll << 30))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Sinks are a few first tokens; the limit bounds the backward's partial sums.
static constexpr int kMaxSinks = 1024;

}  // namespace fa

using namespace fa;

extern "C" {

const char* fa_status_string(int s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_ALIGNMENT: return "FA_ERR_ALIGNMENT";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
    default: return "FA_ERR_UNKNOWN";
  }
}

int fa_version(void) { return 100; }

}  // extern "C"

// Dropout keep threshold t = round(256 (1 - p)) clamped to [1, 256]; 256
// means no dropout.  Returns 0 for a rate outside [0, 1).
static uint32_t keep_threshold(float p_drop) {
  if (!(p_drop >= 0.f && p_drop < 1.f)) return 0;
  long t = lrintf(256.f * (1.f - p_drop));
  return (uint32_t)(t < 1 ? 1 : (t > 256 ? 256 : t));
}

// window > 0: sliding window of that many keys (the caller passes causal = 1).
// f8: q, k, v are E4M3; `qk_factor` multiplies the scores' scale and
// `o_scale` the output (the dequantising factors).  drop_t in 1..255: dropout
// on P with keep threshold drop_t (o_scale is then 256 / drop_t), Philox key
// (seed_lo, seed_hi) and counter word `drop_offset`.
static int forward_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                        int Hkv, int Tq, int Tk, int d, float scale, int causal, int window, void* stream,
                        bool f8 = false, float qk_factor = 1.f, float o_scale = 1.f, uint32_t drop_t = 256,
                        uint32_t seed_lo = 0, uint32_t seed_hi = 0, uint32_t drop_offset = 0, int sinks = 0) {
  const bool drop = drop_t < 256;
  int st = check_prefill(B, Hq, Hkv, Tq, Tk, d, scale, causal);
  if (st) return st;
  if (window < 0 || window > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (sinks < 0 || sinks > kMaxSinks) return FA_ERR_INVALID_ARG;
  if (f8 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Tq == 0) return FA_OK;
  if (!q || !o || !lse || (Tk > 0 && (!k || !v))) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || (Tk > 0 && (!aligned16(k) || !aligned16(v))))
    return FA_ERR_ALIGNMENT;
  st = device_setup();
  if (st) return st;
  FwdParams p;
  memset(&p, 0, sizeof(p));
  const int elt = f8 ? 1 : 2, box_inner = 128 / elt;  // one 128-byte swizzle row per box
  st = make_tmap_4d(&p.tm_q, q, d, Hq, Tq, B, box_inner, 128, true, elt);
  if (!st && Tk > 0) st = make_tmap_4d(&p.tm_k, k, d, Hkv, Tk, B, box_inner, 128, true, elt);
  if (!st && Tk > 0) st = make_tmap_4d(&p.tm_v, v, d, Hkv, Tk, B, box_inner, 128, true, elt);
  if (st) return st;
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Tq = Tq; p.Tk = Tk;
  p.causal = causal;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * qk_factor * 1.4426950408889634f;
  p.o_scale = o_scale;
  p.drop_t = drop_t;
  p.seed_lo = seed_lo;
  p.seed_hi = seed_hi;
  p.drop_offset = drop_offset;
  p.n_mblocks = (Tq + 255) / 256;
  p.n_items = B * Hq * p.n_mblocks;
  p.wait_limit_ns = kWaitLimitNs;
  // Uniform (non-causal or sliding-window) items: persistent, one CTA per
  // SM.  Causal items differ in cost: one CTA per item, heaviest first,
  // balanced by the block scheduler.
  int nsm = 0;
  if ((st = sm_count(&nsm))) return st;
  // Sliding-window items are about equally long: persistent as well.
  dim3 grid(causal && window == 0 ? p.n_items : std::min(p.n_items, nsm));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (f8)
    fa_fwd_kernel<128, true><<<grid, FwdCfg<128, true>::THREADS, FwdCfg<128, true>::SMEM_BYTES, s>>>(p);
  else if (drop && d == 64)
    fa_fwd_kernel<64, false, true><<<grid, FwdCfg<64, false, true>::THREADS, FwdCfg<64, false, true>::SMEM_BYTES, s>>>(p);
  else if (drop)
    fa_fwd_kernel<128, false, true><<<grid, FwdCfg<128, false, true>::THREADS, FwdCfg<128, false, true>::SMEM_BYTES, s>>>(p);
  else if (sinks > 0 && d == 64)
    fa_fwd_kernel<64, false, false, true><<<grid, FwdCfg<64>::THREADS, FwdCfg<64>::SMEM_BYTES, s>>>(p);
  else if (sinks > 0)
    fa_fwd_kernel<128, false, false, true><<<grid, FwdCfg<128>::THREADS, FwdCfg<128>::SMEM_BYTES, s>>>(p);
  else if (d == 64)
    fa_fwd_kernel<64><<<grid, FwdCfg<64>::THREADS, FwdCfg<64>::SMEM_BYTES, s>>>(p);
  else
    fa_fwd_kernel<128><<<grid, FwdCfg<128>::THREADS, FwdCfg<128>::SMEM_BYTES, s>>>(p);
  return launch_status();
}

extern "C" {

int fa_forward(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
               int Hkv, int Tq, int Tk, int d, float scale, int causal, void* stream) {
  return forward_impl(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0, stream);
}

int fa_forward_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                      int Hkv, int Tq, int Tk, int d, float scale, int window, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return forward_impl(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, d, scale, 1, window, stream);
}

int fa_forward_sinks(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                     int Tq, int Tk, int d, float scale, int window, int sinks, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  // unseen scores are masked with -inf, and the maximum taken, before the scaling
  if (sinks > 0 && !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  return forward_impl(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, d, scale, 1, window, stream, false, 1.f, 1.f, 256, 0, 0, 0,
                      sinks);
}

int fa_forward_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                       int Hkv, int Tq, int Tk, int d, float scale, int causal, float p_drop,
                       unsigned long long seed, unsigned int offset, void* stream) {
  const uint32_t t = keep_threshold(p_drop);
  if (!t) return FA_ERR_INVALID_ARG;
  return forward_impl(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0, stream, false, 1.f,
                      256.f / (float)t, (uint32_t)t, (uint32_t)(seed & 0xFFFFFFFFull), (uint32_t)(seed >> 32),
                      offset);
}

int fa_forward_fp8(const void* q, const void* k, const void* v, float q_descale, float k_descale,
                   float v_descale, void* o, float* lse, int B, int Hq, int Hkv, int Tq, int Tk, int d,
                   float scale, int causal, void* stream) {
  for (float f : {q_descale, k_descale, v_descale})
    if (!(f > 0.f) || !isfinite(f)) return FA_ERR_INVALID_ARG;
  if (!isfinite(scale * q_descale * k_descale)) return FA_ERR_INVALID_ARG;
  return forward_impl(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0, stream, true,
                      q_descale * k_descale, v_descale);
}

static size_t round256(size_t x) { return (x + 255) / 256 * 256; }

static int tq_pad(int Tq) { return (Tq + 127) / 128 * 128; }

size_t fa_backward_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int d) {
  (void)Hkv; (void)Tk;
  if (B < 0 || Hq < 1 || Tq < 0 || (d != 64 && d != 128)) return 0;
  return round256((size_t)B * Tq * Hq * d * 4) + 2 * round256((size_t)B * Hq * tq_pad(Tq) * 4);
}

// Workspace pieces of the backward pass.
struct BwdWs {
  float* dq_acc;
  float* Dv;
  float* lse2;
};
static BwdWs bwd_ws(void* ws, int B, int Hq, int Tq, int d) {
  BwdWs w;
  w.dq_acc = reinterpret_cast<float*>(ws);
  w.Dv = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256((size_t)B * Tq * Hq * d * 4));
  w.lse2 = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(w.Dv) + round256((size_t)B * Hq * tq_pad(Tq) * 4));
  return w;
}

static int check_ws(void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk, int d) {
  const size_t need = fa_backward_workspace_bytes(B, Hq, Hkv, Tq, Tk, d);
  if (!ws || ws_bytes < need || !aligned16(ws)) return FA_ERR_WORKSPACE;
  return FA_OK;
}

static int check_ptrs(std::initializer_list<const void*> ptrs) {
  for (const void* ptr : ptrs) {
    if (!ptr) return FA_ERR_INVALID_ARG;
    if (!aligned16(ptr)) return FA_ERR_ALIGNMENT;
  }
  return FA_OK;
}

// How the backward cuts up the key tiles that hold sinks (see BwdParams): a
// piece is about as many query tiles as a windowed key tile sees, so that no
// item outlasts the others by far; at most 32 pieces, and no more than keep the
// partial sums within twice the fp32 dQ accumulator's bytes (with pieces of four
// query tiles they are half of its bytes per sink tile, divided by the query heads
// per KV head: several sink tiles have that many more items without being cut so fine).
struct SinkPlan {
  int tiles, pieces;
  size_t part_bytes;
};
static SinkPlan sink_plan(int B, int Hq, int Hkv, int Tq, int Tk, int d, int window, int sinks) {
  SinkPlan s;
  s.tiles = (std::min(sinks, Tk) + 127) / 128;
  const int n_qt = (Tq + 127) / 128;
  const int per = std::max(4, (int)(((long long)window + 127) / 128) + 1);
  const size_t piece_bytes = (size_t)B * Hkv * s.tiles * 2 * 128 * d * 4, acc_bytes = (size_t)B * Tq * Hq * d * 4;
  const int most = piece_bytes > 0 ? (int)std::min<size_t>(32, 2 * acc_bytes / piece_bytes) : 1;
  s.pieces = std::max(1, std::min(most, (n_qt + per - 1) / per));
  s.part_bytes = s.pieces > 1 ? round256(piece_bytes * s.pieces) : 0;
  return s;
}

size_t fa_backward_sinks_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int d, int window, int sinks) {
  const size_t base = fa_backward_workspace_bytes(B, Hq, Hkv, Tq, Tk, d);
  if (base == 0 || Hkv < 1 || Tk < 0 || window < 1 || sinks < 0 || sinks > kMaxSinks) return base;
  return base + sink_plan(B, Hq, Hkv, Tq, Tk, d, window, sinks).part_bytes;
}

// zero_acc = false leaves the fp32 dQ accumulator alone (a backward whose dQ
// pass writes dq directly does not read it).
static int preprocess_impl(const void* o, const float* lse, const void* dO, void* ws, size_t ws_bytes, int B,
                           int Hq, int Hkv, int Tq, int Tk, int d, void* stream, bool zero_acc,
                           float p_log2 = 0.f) {
  int st = check_prefill(B, Hq, Hkv, Tq, Tk, d, 1.f, 0);
  if (st) return st;
  if (B == 0 || Tq == 0) return FA_OK;
  if ((st = check_ptrs({o, lse, dO}))) return st;
  if ((st = check_ws(ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d))) return st;
  if ((st = device_setup())) return st;
  const BwdWs w = bwd_ws(ws, B, Hq, Tq, d);
  const int Tp = tq_pad(Tq);
  const long long threads = std::max((long long)B * Tq * Hq * (d / 8), (long long)B * Hq * (Tp - Tq));
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const __nv_bfloat16* o16 = reinterpret_cast<const __nv_bfloat16*>(o);
  const __nv_bfloat16* do16 = reinterpret_cast<const __nv_bfloat16*>(dO);
  float* acc = zero_acc ? w.dq_acc : nullptr;
  if (d == 64)
    fa_bwd_preprocess_kernel<64><<<blocks, 256, 0, s>>>(o16, do16, lse, w.Dv, w.lse2, acc, B, Hq, Tq, Tp, p_log2);
  else
    fa_bwd_preprocess_kernel<128><<<blocks, 256, 0, s>>>(o16, do16, lse, w.Dv, w.lse2, acc, B, Hq, Tq, Tp, p_log2);
  return launch_status();
}

int fa_backward_preprocess(const void* o, const float* lse, const void* dO, void* ws, size_t ws_bytes,
                           int B, int Hq, int Hkv, int Tq, int Tk, int d, void* stream) {
  return preprocess_impl(o, lse, dO, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, stream, true);
}

}  // extern "C"

// drop_t in 1..255: dropout on P with that keep threshold and Philox key
// (seed_lo, seed_hi), counter word drop_offset (the forward's mask).
// det: dQ from the separate, deterministic pass (fa_bwd_dq.cuh) after the
// dK/dV kernel built without dQ, into the fp32 accumulator or, when dq_out
// is given, as bf16 straight into dq_out (no dropout).
static int dkdv_impl(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, void* ws,
                     size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk, int d, float scale, int causal,
                     int window, void* stream, uint32_t drop_t = 256, uint32_t seed_lo = 0, uint32_t seed_hi = 0,
                     uint32_t drop_offset = 0, bool det = false, void* dq_out = nullptr, int sinks = 0) {
  const bool drop = drop_t < 256;
  int st = check_prefill(B, Hq, Hkv, Tq, Tk, d, scale, causal);
  if (st) return st;
  if (window < 0 || window > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (B == 0 || Tk == 0) return FA_OK;
  if ((st = check_ptrs({k, v, dk, dv}))) return st;
  if (Tq > 0 && (st = check_ptrs({q, dO}))) return st;
  if ((st = check_ws(ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d))) return st;
  if ((st = device_setup())) return st;
  const BwdWs w = bwd_ws(ws, B, Hq, Tq, d);
  BwdParams p;
  memset(&p, 0, sizeof(p));
  if (Tq > 0) {
    st = make_tmap_4d(&p.tm_q, q, d, Hq, Tq, B, 64, 128, true);
    if (!st) st = make_tmap_4d(&p.tm_do, dO, d, Hq, Tq, B, 64, 128, true);
  }
  if (!st) st = make_tmap_4d(&p.tm_k, k, d, Hkv, Tk, B, 64, 128, true);
  if (!st) st = make_tmap_4d(&p.tm_v, v, d, Hkv, Tk, B, 64, 128, true);
  if (!st && Tq > 0) st = make_tmap_f32_4d(&p.tm_dq, w.dq_acc, d, Hq, Tq, B);
  if (st) return st;
  p.lse2 = w.lse2;
  p.Dv = w.Dv;
  p.dq_acc = w.dq_acc;
  p.dk = reinterpret_cast<__nv_bfloat16*>(dk);
  p.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Tq = Tq; p.Tk = Tk; p.causal = causal;
  p.window = window;
  p.Tq_pad = tq_pad(Tq);
  p.dv_scale = sinks > 0 ? exp2f(-SINK_P_LOG2) : 1.f;
  p.scale = scale * p.dv_scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.n_kv_tiles = (Tk + 127) / 128;
  p.n_items = p.n_kv_tiles * B * Hkv;
  if (sinks > 0) {
    const SinkPlan sp = sink_plan(B, Hq, Hkv, Tq, Tk, d, window, sinks);
    if (ws_bytes < fa_backward_sinks_workspace_bytes(B, Hq, Hkv, Tq, Tk, d, window, sinks)) return FA_ERR_WORKSPACE;
    const long long items = (long long)B * Hkv * (p.n_kv_tiles + (long long)sp.tiles * (sp.pieces - 1));
    if (items > 0x7FFFFFFFll) return FA_ERR_INVALID_ARG;
    p.n_items = (int)items;
    p.sinks = sinks;
    p.n_sink_tiles = sp.tiles;
    p.pieces = sp.pieces;
    p.sink_part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) +
                                           fa_backward_workspace_bytes(B, Hq, Hkv, Tq, Tk, d));
  }
  p.drop_t = drop_t;
  p.seed_lo = seed_lo;
  p.seed_hi = seed_hi;
  p.drop_offset = drop_offset;
  p.drop_scale = 256.f / (float)drop_t;
  p.wait_limit_ns = kWaitLimitNs;
  // Non-causal d = 64: one persistent CTA per SM, whose next item's K/V
  // load overlaps the current item (two K/V buffers); items are all the
  // same length there.  Causal: one CTA per item, since items differ in
  // length and the hardware scheduler balances them.
  int nsm = 0;
  if ((st = sm_count(&nsm))) return st;
  // With sinks the items are alike by construction (the sink tiles' pieces are
  // as long as a windowed item) and, in a short window, only a few tiles long.
  const bool persistent = d == 64 && (!causal || sinks > 0);
  dim3 grid(persistent ? std::min(p.n_items, nsm) : p.n_items);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (drop && (window > 0 || det)) return FA_ERR_UNSUPPORTED;
  if (drop) {
    if (d == 64)
      fa_bwd_dkdv_kernel<64, false, true><<<grid, BwdCfg<64, true>::THREADS, BwdCfg<64, true>::SMEM_BYTES, s>>>(p);
    else
      fa_bwd_dkdv_kernel<128, false, true><<<grid, BwdCfg<128, true>::THREADS, BwdCfg<128, true>::SMEM_BYTES, s>>>(p);
    return launch_status();
  }
  // dK and dV of cut-up sink tiles, once their pieces are done
  auto sum_sinks = [&]() -> int {
    if (sinks == 0 || p.pieces == 1) return FA_OK;
    const dim3 g((unsigned)(B * Hkv * p.n_sink_tiles * (d / 8)), 2);
    if (d == 64)
      fa_bwd_sink_sum_kernel<64><<<g, 256, 0, s>>>(p.sink_part, p.dk, p.dv, Hkv, Tk, p.n_sink_tiles, p.pieces);
    else
      fa_bwd_sink_sum_kernel<128><<<g, 256, 0, s>>>(p.sink_part, p.dk, p.dv, Hkv, Tk, p.n_sink_tiles, p.pieces);
    return launch_status();
  };
  if (!det) {
    if (sinks > 0) {
      if (d == 64)
        fa_bwd_dkdv_kernel<64, 2><<<grid, BwdCfg<64>::THREADS, BwdCfg<64>::SMEM_BYTES, s>>>(p);
      else
        fa_bwd_dkdv_kernel<128, 2><<<grid, BwdCfg<128>::THREADS, BwdCfg<128>::SMEM_BYTES, s>>>(p);
      if ((st = launch_status())) return st;
      return sum_sinks();
    }
    if (d == 64 && window > 0)
      fa_bwd_dkdv_kernel<64, true><<<grid, BwdCfg<64>::THREADS, BwdCfg<64>::SMEM_BYTES, s>>>(p);
    else if (d == 64)
      fa_bwd_dkdv_kernel<64, false><<<grid, BwdCfg<64>::THREADS, BwdCfg<64>::SMEM_BYTES, s>>>(p);
    else if (window > 0)
      fa_bwd_dkdv_kernel<128, true><<<grid, BwdCfg<128>::THREADS, BwdCfg<128>::SMEM_BYTES, s>>>(p);
    else
      fa_bwd_dkdv_kernel<128, false><<<grid, BwdCfg<128>::THREADS, BwdCfg<128>::SMEM_BYTES, s>>>(p);
    return launch_status();
  }
  // deterministic: dK/dV without dQ, then the dQ pass
  using C64 = BwdCfg<64, false, false>;
  using C128 = BwdCfg<128, false, false>;
  if (sinks > 0 && d == 64)
    fa_bwd_dkdv_kernel<64, 2, false, false><<<grid, C64::THREADS, C64::SMEM_BYTES, s>>>(p);
  else if (sinks > 0)
    fa_bwd_dkdv_kernel<128, 2, false, false><<<grid, C128::THREADS, C128::SMEM_BYTES, s>>>(p);
  else if (d == 64 && window > 0)
    fa_bwd_dkdv_kernel<64, true, false, false><<<grid, C64::THREADS, C64::SMEM_BYTES, s>>>(p);
  else if (d == 64)
    fa_bwd_dkdv_kernel<64, false, false, false><<<grid, C64::THREADS, C64::SMEM_BYTES, s>>>(p);
  else if (window > 0)
    fa_bwd_dkdv_kernel<128, true, false, false><<<grid, C128::THREADS, C128::SMEM_BYTES, s>>>(p);
  else
    fa_bwd_dkdv_kernel<128, false, false, false><<<grid, C128::THREADS, C128::SMEM_BYTES, s>>>(p);
  if ((st = launch_status())) return st;
  if ((st = sum_sinks())) return st;
  if (Tq == 0) return FA_OK;
  DqParams qp;
  memset(&qp, 0, sizeof(qp));
  qp.tm_q = p.tm_q;
  qp.tm_do = p.tm_do;
  qp.tm_k = p.tm_k;
  qp.tm_v = p.tm_v;
  qp.lse2 = w.lse2;
  qp.Dv = w.Dv;
  qp.dq_acc = w.dq_acc;
  qp.dq = reinterpret_cast<__nv_bfloat16*>(dq_out);
  qp.B = B; qp.Hq = Hq; qp.Hkv = Hkv; qp.Tq = Tq; qp.Tk = Tk; qp.causal = causal;
  qp.window = window;
  qp.sinks = sinks;
  qp.Tq_pad = p.Tq_pad;
  qp.scale = p.scale;
  qp.scale_log2 = p.scale_log2;
  qp.n_qt = (Tq + 127) / 128;
  const long long n_items = (long long)B * Hq * qp.n_qt;
  if (n_items > 0x7FFFFFFFll) return FA_ERR_INVALID_ARG;
  qp.n_items = (int)n_items;
  qp.wait_limit_ns = kWaitLimitNs;
  const unsigned nblk = (unsigned)qp.n_items;
  if (sinks > 0 && d == 64)
    fa_bwd_dq_kernel<64, 2><<<nblk, DqCfg<64>::THREADS, DqCfg<64>::SMEM_BYTES, s>>>(qp);
  else if (sinks > 0)
    fa_bwd_dq_kernel<128, 2><<<nblk, DqCfg<128>::THREADS, DqCfg<128>::SMEM_BYTES, s>>>(qp);
  else if (d == 64 && window > 0)
    fa_bwd_dq_kernel<64, true><<<nblk, DqCfg<64>::THREADS, DqCfg<64>::SMEM_BYTES, s>>>(qp);
  else if (d == 64)
    fa_bwd_dq_kernel<64, false><<<nblk, DqCfg<64>::THREADS, DqCfg<64>::SMEM_BYTES, s>>>(qp);
  else if (window > 0)
    fa_bwd_dq_kernel<128, true><<<nblk, DqCfg<128>::THREADS, DqCfg<128>::SMEM_BYTES, s>>>(qp);
  else
    fa_bwd_dq_kernel<128, false><<<nblk, DqCfg<128>::THREADS, DqCfg<128>::SMEM_BYTES, s>>>(qp);
  return launch_status();
}

extern "C" {

int fa_backward_dkdv(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv,
                     void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk, int d,
                     float scale, int causal, void* stream) {
  return dkdv_impl(q, k, v, dO, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0, stream);
}

int fa_backward_dkdv_window(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv,
                            void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk, int d,
                            float scale, int window, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return dkdv_impl(q, k, v, dO, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, 1, window, stream);
}

int fa_backward_dkdv_dropout(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv,
                             void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk, int d,
                             float scale, int causal, float p_drop, unsigned long long seed, unsigned int offset,
                             void* stream) {
  const uint32_t t = keep_threshold(p_drop);
  if (!t) return FA_ERR_INVALID_ARG;
  return dkdv_impl(q, k, v, dO, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0, stream, t,
                   (uint32_t)(seed & 0xFFFFFFFFull), (uint32_t)(seed >> 32), offset);
}

int fa_backward_dq_finalize(void* dq, void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk,
                            int d, void* stream) {
  int st = check_prefill(B, Hq, Hkv, Tq, Tk, d, 1.f, 0);
  if (st) return st;
  if (B == 0 || Tq == 0) return FA_OK;
  if ((st = check_ptrs({dq}))) return st;
  if ((st = check_ws(ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d))) return st;
  if ((st = device_setup())) return st;
  const BwdWs w = bwd_ws(ws, B, Hq, Tq, d);
  const long long n8 = (long long)B * Tq * Hq * d / 8;
  fa_bwd_dq_convert_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      w.dq_acc, reinterpret_cast<__nv_bfloat16*>(dq), n8);
  return launch_status();
}

}  // extern "C"

static int backward_impl(const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int B, int Hq,
                         int Hkv, int Tq, int Tk, int d, float scale, int causal, int window, void* stream,
                         uint32_t drop_t = 256, uint32_t seed_lo = 0, uint32_t seed_hi = 0,
                         uint32_t drop_offset = 0, bool det = false, int sinks = 0) {
  int st = check_prefill(B, Hq, Hkv, Tq, Tk, d, scale, causal);
  if (st) return st;
  if (window < 0 || window > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (sinks < 0 || sinks > kMaxSinks) return FA_ERR_INVALID_ARG;
  if (B == 0 || (Tq == 0 && Tk == 0)) return FA_OK;
  if (Tq > 0 && (st = check_ptrs({q, o, lse, dO, dq}))) return st;
  if (Tk > 0 && (st = check_ptrs({k, v, dk, dv}))) return st;
  if ((st = check_ws(ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d))) return st;
  if (sinks > 0 && ws_bytes < fa_backward_sinks_workspace_bytes(B, Hq, Hkv, Tq, Tk, d, window, sinks))
    return FA_ERR_WORKSPACE;
  // deterministic: the dQ pass writes dq itself (when there are keys; with
  // none, dq is the zeroed accumulator converted)
  const bool direct = det && Tq > 0 && Tk > 0;
  if ((st = preprocess_impl(o, lse, dO, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, stream, !direct,
                            sinks > 0 ? (float)SINK_P_LOG2 : 0.f)))
    return st;
  if ((st = dkdv_impl(q, k, v, dO, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, causal, window, stream,
                      drop_t, seed_lo, seed_hi, drop_offset, det, direct ? dq : nullptr, sinks)))
    return st;
  if (direct) return FA_OK;
  return fa_backward_dq_finalize(dq, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, stream);
}

extern "C" {

int fa_backward(const void* q, const void* k, const void* v, const void* o, const float* lse,
                const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int B,
                int Hq, int Hkv, int Tq, int Tk, int d, float scale, int causal, void* stream) {
  return backward_impl(q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0,
                       stream);
}

int fa_backward_dropout(const void* q, const void* k, const void* v, const void* o, const float* lse,
                        const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int B, int Hq,
                        int Hkv, int Tq, int Tk, int d, float scale, int causal, float p_drop,
                        unsigned long long seed, unsigned int offset, void* stream) {
  const uint32_t t = keep_threshold(p_drop);
  if (!t) return FA_ERR_INVALID_ARG;
  return backward_impl(q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, causal, 0,
                       stream, t, (uint32_t)(seed & 0xFFFFFFFFull), (uint32_t)(seed >> 32), offset);
}

int fa_backward_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                       const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int B,
                       int Hq, int Hkv, int Tq, int Tk, int d, float scale, int window, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return backward_impl(q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, 1, window,
                       stream);
}

int fa_backward_deterministic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                              const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int B,
                              int Hq, int Hkv, int Tq, int Tk, int d, float scale, int causal, int window,
                              void* stream) {
  if (window < 0 || (window > 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  return backward_impl(q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, causal, window,
                       stream, 256, 0, 0, 0, true);
}

int fa_backward_sinks(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                      void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tq, int Tk,
                      int d, float scale, int window, int sinks, int deterministic, void* stream) {
  if (window < 1 || (deterministic != 0 && deterministic != 1)) return FA_ERR_INVALID_ARG;
  return backward_impl(q, k, v, o, lse, dO, dq, dk, dv, ws, ws_bytes, B, Hq, Hkv, Tq, Tk, d, scale, 1, window, stream,
                       256, 0, 0, 0, deterministic != 0, sinks);
}

static size_t decode_nchunk(int Tk_max, int chunk) { return ((size_t)Tk_max + chunk - 1) / chunk; }

static size_t decode_ws_bytes(int B, int Hq, size_t n, int d) {
  return round256((size_t)B * Hq * n * d * 4) + round256((size_t)B * Hq * n * 4);
}

size_t fa_decode_workspace_bytes(int B, int Hq, int Tk_max, int d, int chunk) {
  if (B < 0 || Hq < 1 || Tk_max < 0 || chunk < 1 || (d != 64 && d != 128)) return 0;
  return decode_ws_bytes(B, Hq, decode_nchunk(Tk_max, chunk), d);
}

// Chunks of a sequence that can be visible: those that hold sinks and those
// that a window can touch.
static size_t decode_visible_chunks(int Tk_max, int chunk, int window, int sinks) {
  return std::min(decode_nchunk(Tk_max, chunk),
                  ((size_t)sinks + chunk - 1) / chunk + ((size_t)window + chunk - 2) / chunk + 1);
}

size_t fa_decode_sinks_workspace_bytes(int B, int Hq, int Tk_max, int d, int chunk, int window, int sinks) {
  if (B < 0 || Hq < 1 || Tk_max < 0 || chunk < 1 || (d != 64 && d != 128) || window < 1 || sinks < 0 ||
      sinks > kMaxSinks)
    return 0;
  return decode_ws_bytes(B, Hq, sinks > 0 ? decode_visible_chunks(Tk_max, chunk, window, sinks)
                                          : decode_nchunk(Tk_max, chunk), d);
}

}  // extern "C"

// `o` receives bf16 O, or, when `o32` is non-null instead, fp32 O.
static int decode_impl(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k, void* o,
                       float* o32, float* lse, void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tk_max,
                       int d, float scale, int chunk, int window, void* stream, int sinks = 0) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Tk_max < 0 || Hq % Hkv != 0 || !isfinite(scale))
    return FA_ERR_INVALID_ARG;
  if (window < 0 || window > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (sinks < 0 || sinks > kMaxSinks) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return FA_ERR_UNSUPPORTED;
  if (chunk < 64 || chunk % 64 != 0 || chunk * G > 4096) return FA_ERR_INVALID_ARG;
  // one warp per (sequence, head) row in the merge kernels: 32 * B * Hq
  // threads must stay below 2^31
  if ((int64_t)Tk_max > (1 << 30) || (int64_t)B * Hq > (1 << 26)) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!q || !seqlens_k || (!o == !o32) || !lse || (Tk_max > 0 && (!k_cache || !v_cache)))
    return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o ? o : o32) || !aligned16(lse) || (reinterpret_cast<uintptr_t>(seqlens_k) & 3u) ||
      (Tk_max > 0 && (!aligned16(k_cache) || !aligned16(v_cache))))
    return FA_ERR_ALIGNMENT;
  // with sinks, only the chunks that can be visible are items
  const size_t n = sinks > 0 ? decode_visible_chunks(Tk_max, chunk, window, sinks) : decode_nchunk(Tk_max, chunk);
  const size_t need = decode_ws_bytes(B, Hq, n, d);
  if (!ws || ws_bytes < need || !aligned16(ws)) return FA_ERR_WORKSPACE;
  int st = device_setup();
  if (st) return st;
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  if (Tk_max > 0) {
    st = make_tmap_4d(&p.tm_k, k_cache, d, Hkv, Tk_max, B, 64, 64, true);
    if (!st) st = make_tmap_4d(&p.tm_v, v_cache, d, Hkv, Tk_max, B, 64, 64, true);
    if (st) return st;
  }
  if ((size_t)B * Hkv * n > (size_t)(1 << 30)) return FA_ERR_INVALID_ARG;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.seqlens = seqlens_k;
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_lse = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256((size_t)B * Hq * n * d * 4));
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.o32 = o32;
  p.lse = lse;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Tk_max = Tk_max; p.chunk = chunk; p.nchunk = (int)n;
  p.n_items = (int)((size_t)B * Hkv * n);
  p.window = window;
  p.sinks = sinks;
  p.sink_chunks = (sinks + chunk - 1) / chunk;
  p.inv_chunk = chunk_inverse(chunk);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = kWaitLimitNs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (Tk_max > 0) {
    int nsm = 0;
    if ((st = sm_count(&nsm))) return st;
    // persistent: two CTAs per SM walk the (sequence, KV head, chunk) items
    dim3 grid((unsigned)std::min<long long>(p.n_items, (long long)kDecodeCtasPerSm * nsm));
#define FA_DEC_LAUNCH(DD, GG)                                                                             \
    (sinks > 0 ? fa_decode_split_kernel<DD, GG, true><<<grid, DecCfg<DD, GG>::THREADS, DecCfg<DD, GG>::SMEM_BYTES, s>>>(p) \
               : fa_decode_split_kernel<DD, GG><<<grid, DecCfg<DD, GG>::THREADS, DecCfg<DD, GG>::SMEM_BYTES, s>>>(p))
    if (d == 64) {
      if (G == 1) FA_DEC_LAUNCH(64, 1); else if (G == 2) FA_DEC_LAUNCH(64, 2);
      else if (G == 4) FA_DEC_LAUNCH(64, 4); else FA_DEC_LAUNCH(64, 8);
    } else {
      if (G == 1) FA_DEC_LAUNCH(128, 1); else if (G == 2) FA_DEC_LAUNCH(128, 2);
      else if (G == 4) FA_DEC_LAUNCH(128, 4); else FA_DEC_LAUNCH(128, 8);
    }
#undef FA_DEC_LAUNCH
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }
  const int warps = B * Hq;
  const int blocks = (warps * 32 + 255) / 256;
  if (sinks > 0) {
    return launch_after(d == 64 ? fa_decode_combine_kernel<64, true> : fa_decode_combine_kernel<128, true>, blocks, 256,
                        s, p);
  }
  if (Tk_max > 0) {
    if (d == 64)
      fa_decode_combine_kernel<64><<<blocks, 256, 0, s>>>(p);
    else
      fa_decode_combine_kernel<128><<<blocks, 256, 0, s>>>(p);
  }
  if (d == 64)
    fa_decode_empty_kernel<64><<<blocks, 256, 0, s>>>(p);
  else
    fa_decode_empty_kernel<128><<<blocks, 256, 0, s>>>(p);
  return launch_status();
}

extern "C" {

int fa_decode_splitkv(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k,
                      void* o, float* lse, void* ws, size_t ws_bytes, int B, int Hq, int Hkv,
                      int Tk_max, int d, float scale, int chunk, void* stream) {
  return decode_impl(q, k_cache, v_cache, seqlens_k, o, nullptr, lse, ws, ws_bytes, B, Hq, Hkv, Tk_max, d, scale,
                     chunk, 0, stream);
}

int fa_decode_splitkv_partial(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k,
                              float* o, float* lse, void* ws, size_t ws_bytes, int B, int Hq, int Hkv,
                              int Tk_max, int d, float scale, int chunk, void* stream) {
  return decode_impl(q, k_cache, v_cache, seqlens_k, nullptr, o, lse, ws, ws_bytes, B, Hq, Hkv, Tk_max, d, scale,
                     chunk, 0, stream);
}

int fa_decode_merge(const float* o_parts, size_t o_stride, const float* lse_parts, size_t lse_stride, void* o,
                    float* lse, int R, int B, int Hq, int d, void* stream) {
  if (R < 1 || R > (1 << 20) || B < 0 || Hq < 1 || (int64_t)B * Hq > (1 << 26)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const size_t rows = (size_t)B * Hq;
  if (rows == 0) return FA_OK;
  if (!o_parts || !lse_parts || !o || !lse) return FA_ERR_INVALID_ARG;
  if (R > 1 && (o_stride < rows * d || lse_stride < rows)) return FA_ERR_INVALID_ARG;
  if (!aligned16(o_parts) || !aligned16(o) || (o_stride & 3u) ||
      (reinterpret_cast<uintptr_t>(lse_parts) & 3u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FA_ERR_ALIGNMENT;
  int st = device_setup();
  if (st) return st;
  MergeParams p;
  p.o_parts = o_parts;
  p.lse_parts = lse_parts;
  p.o_stride = o_stride;
  p.lse_stride = lse_stride;
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.R = R;
  p.rows = (int)rows;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned blocks = (unsigned)((rows * 32 + 255) / 256);
  if (d == 64)
    fa_decode_merge_kernel<64><<<blocks, 256, 0, s>>>(p);
  else
    fa_decode_merge_kernel<128><<<blocks, 256, 0, s>>>(p);
  return launch_status();
}

int fa_decode_splitkv_window(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k,
                             void* o, float* lse, void* ws, size_t ws_bytes, int B, int Hq, int Hkv,
                             int Tk_max, int d, float scale, int chunk, int window, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return decode_impl(q, k_cache, v_cache, seqlens_k, o, nullptr, lse, ws, ws_bytes, B, Hq, Hkv, Tk_max, d, scale,
                     chunk, window, stream);
}

int fa_decode_splitkv_sinks(const void* q, const void* k_cache, const void* v_cache, const int* seqlens_k, void* o,
                            float* lse, void* ws, size_t ws_bytes, int B, int Hq, int Hkv, int Tk_max, int d,
                            float scale, int chunk, int window, int sinks, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return decode_impl(q, k_cache, v_cache, seqlens_k, o, nullptr, lse, ws, ws_bytes, B, Hq, Hkv, Tk_max, d, scale,
                     chunk, window, stream, sinks);
}

int fa_check(void* stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_fa_status, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_fa_status, &zero, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return v;
}

}  // extern "C"

namespace fa {
// One block, one thread waits on a barrier that nothing completes.
__global__ void selftest_wait_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(smem_u32(&bar), 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    WaitCtl w{&abort_flag, limit_ns};
    mbar_wait(smem_u32(&bar), 0, w);
  }
  __syncthreads();
}
}  // namespace fa

namespace fa {
__global__ void selftest_exp2_poly_kernel(const float* x, float* y, int n) {
  const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= n) return;
  const float2 in = make_float2(x[i], i + 1 < n ? x[i + 1] : 0.f);
  const float2 out = exp2_poly2(in);
  y[i] = out.x;
  if (i + 1 < n) y[i + 1] = out.y;
}
}  // namespace fa

extern "C" int fa_selftest_exp2_poly(const float* x, float* y, int n, void* stream) {
  if (n < 0 || (n > 0 && (!x || !y))) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  int st = device_setup();
  if (st) return st;
  const int pairs = (n + 1) / 2;
  selftest_exp2_poly_kernel<<<(pairs + 255) / 256, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, y, n);
  return launch_status();
}

extern "C" int fa_selftest_chunk_of(int key, int chunk) {
  if (key < 0 || chunk < 64 || chunk > 4096 || chunk % 64 != 0) return -1;
  return (int)div_chunk((unsigned)key, chunk_inverse(chunk));
}

extern "C" int fa_selftest_bounded_wait(int limit_us, void* stream) {
  if (limit_us < 1 || limit_us > 1000000) return FA_ERR_INVALID_ARG;
  int st = device_setup();
  if (st) return st;
  selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      (unsigned long long)limit_us * 1000ull);
  return launch_status();
}

// ---------------------------------------------------------------------------
// Split-KV decode without caller-provided workspace.
//
// For callers that cannot allocate device memory at the call site --
// plug-in interfaces that hand over only the input and output tensors and
// no allocator, or latency-critical loops where cudaMalloc's implicit
// device synchronisation is not acceptable.  The chunk partials live in one
// file-scope device array that every GPU loading this library keeps until
// the process exits.
// ---------------------------------------------------------------------------
namespace fa {

static constexpr size_t kDecodeScratchBytes = 32u << 20;  // 32 MiB
static __device__ __align__(256) unsigned char g_decode_scratch[kDecodeScratchBytes];

// Device address of g_decode_scratch for the current device, looked up once
// per device (host code may not use the symbol itself as an address).
static int decode_scratch_ptr(void** out) {
  static void* cache[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  if (!cache[dev]) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_decode_scratch) != cudaSuccess || !ptr) return FA_ERR_CUDA;
    cache[dev] = ptr;
  }
  *out = cache[dev];
  return FA_OK;
}

}  // namespace fa

extern "C" int fa_decode_splitkv_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                         const int* seqlens_k, void* o, float* lse, int B, int Hq, int Hkv,
                                         int Tk_max, int d, float scale, int chunk, void* stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Tk_max < 0 || chunk < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // The partials of this call must fit in the built-in scratch array.
  if (fa_decode_workspace_bytes(B, Hq, Tk_max, d, chunk) > kDecodeScratchBytes) return FA_ERR_WORKSPACE;
  // No rows: the workspace entry point checks the remaining arguments the
  // same way and returns before it touches the (empty) workspace.
  if (B == 0)
    return fa_decode_splitkv(q, k_cache, v_cache, seqlens_k, o, lse, nullptr, 0, B, Hq, Hkv, Tk_max, d, scale, chunk,
                             stream);
  void* scratch = nullptr;
  const int st = decode_scratch_ptr(&scratch);
  if (st) return st;
  // Every partial the combine step reads is written first by the split step
  // of the same call, so nothing in the scratch needs clearing.
  return fa_decode_splitkv(q, k_cache, v_cache, seqlens_k, o, lse, scratch, kDecodeScratchBytes, B, Hq, Hkv,
                           Tk_max, d, scale, chunk, stream);
}

// ---------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------
namespace fa {

// The layout [B][T][H][d] with these strides: every element its own place.
static bool rope_dense_enough(const int64_t* st, int B, int T, int H, int d) {
  struct Dim { int64_t stride, size; } dim[3] = {{st[0], B}, {st[1], T}, {st[2], H}};
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t extent = d;
  for (const Dim& m : dim) {
    if (m.size < 2) continue;
    if (m.stride < extent) return false;
    extent = m.stride * (m.size - 1) + extent;
  }
  return true;
}

// Whether x (Hx heads) may share memory with y (Hy heads): no, if it can be
// shown that their ranges are apart, or that they are different slices of the
// same repeating slots (heads of the same packed rows or batches).
static bool rope_collide(const void* x, const int64_t* sx, int Hx, const void* y, const int64_t* sy, int Hy, int B,
                         int T, int d) {
  const int64_t n[2] = {B, T};
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  const bool y_first = y0 < x0;
  const int64_t diff = (int64_t)(y_first ? x0 - y0 : y0 - x0) / 2;
  // Slots are counted over the axes in `outer` (bit 0: sequences, bit 1: tokens),
  // which both must step through alike; the others belong to the slice.
  for (int outer = 0; outer < 4; ++outer) {
    int64_t ex = sx[2] * (Hx - 1) + d, ey = sy[2] * (Hy - 1) + d;  // a slice's extent
    int64_t step[2] = {0, 0}, count[2] = {1, 1};
    int axes = 0;
    bool alike = true;
    for (int a = 0; a < 2; ++a) {
      if (n[a] == 1) continue;
      if (outer >> a & 1) {
        alike = alike && sx[a] == sy[a];
        step[axes] = sx[a];
        count[axes++] = n[a];
      } else {
        ex += sx[a] * (n[a] - 1);
        ey += sy[a] * (n[a] - 1);
      }
    }
    if (!alike) continue;
    const int64_t front = y_first ? ey : ex, back = y_first ? ex : ey;  // in memory's order
    if (axes == 0) {
      if (diff >= front) return false;
      continue;
    }
    const int in = axes == 2 && step[1] < step[0] ? 1 : 0;  // the inner of the stepping axes
    const int64_t slot = step[in];
    if (slot < 1) continue;  // broadcast: nothing to count by
    const bool even = axes == 1 || step[1 - in] % slot == 0;          // slots repeat throughout
    const bool nested = axes == 1 || step[1 - in] >= slot * count[in];  // slots never overlap
    const int64_t off = even ? diff % slot : diff;
    if ((even || nested) && off >= front && off + back <= slot) return false;
  }
  return true;
}

// Checks one tensor and its output (strides st[0..2] and st[3..5]).
static int rope_tensor(RopeTensor* r, const void* x, void* y, const int64_t* st, const int64_t* so, int B, int T,
                       int H, int d) {
  if (!x || !y) return FA_ERR_INVALID_ARG;
  const int64_t n[3] = {B, T, H};
  bool same = x == y;  // in place: the same memory, the same strides
  for (int i = 0; i < 3; ++i) {
    // 2^60 elements per axis, so that offsets cannot leave 64 bits
    const int64_t most = (1ll << 60) / n[i];
    if (st[i] < 0 || so[i] < 0 || st[i] > most || so[i] > most) return FA_ERR_INVALID_ARG;
    same = same && (n[i] == 1 || st[i] == so[i]);
  }
  if (!rope_dense_enough(so, B, T, H, d)) return FA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y)) return FA_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if ((st[i] & 7) || (so[i] & 7)) return FA_ERR_ALIGNMENT;
  if (!same && rope_collide(x, st, H, y, so, H, B, T, d)) return FA_ERR_INVALID_ARG;
  r->x = reinterpret_cast<const __nv_bfloat16*>(x);
  r->y = reinterpret_cast<__nv_bfloat16*>(y);
  r->xb = st[0]; r->xt = st[1]; r->xh = st[2];
  r->yb = so[0]; r->yt = so[1]; r->yh = so[2];
  return FA_OK;
}

static int rope_impl(const void* q, void* q_out, const void* k, void* k_out, const int64_t* strides,
                     const int* positions, const double* freqs, int rotary_dim, int interleaved, float amplitude,
                     float sign, int B, int T, int Hq, int Hkv, int d, void* stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || Hq + (int64_t)Hkv < 1 || Hq > 65535 || Hkv > 65535)
    return FA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > d || rotary_dim % 16 != 0 || !isfinite(amplitude)) return FA_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return FA_OK;
  if (!strides || !freqs) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(freqs) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return FA_ERR_ALIGNMENT;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  int st = FA_OK;
  if (Hq > 0) st = rope_tensor(&p.q, q, q_out, strides, strides + 3, B, T, Hq, d);
  if (!st && Hkv > 0) st = rope_tensor(&p.k, k, k_out, strides + 6, strides + 9, B, T, Hkv, d);
  if (st) return st;
  // one tensor's output may not touch the other tensor
  if (Hq > 0 && Hkv > 0 &&
      (rope_collide(q_out, strides + 3, Hq, k_out, strides + 9, Hkv, B, T, d) ||
       rope_collide(q_out, strides + 3, Hq, k, strides + 6, Hkv, B, T, d) ||
       rope_collide(k_out, strides + 9, Hkv, q, strides, Hq, B, T, d)))
    return FA_ERR_INVALID_ARG;
  p.positions = positions;
  p.freqs = freqs;
  p.n_tokens = (long long)B * T;
  p.T = T;
  p.Hq = Hq;
  p.heads = Hq + Hkv;
  p.rot = rotary_dim;
  p.amplitude = amplitude;
  p.sign = sign;
  if ((st = device_setup())) return st;
  const int tpb = p.n_tokens >= 4096 ? 4 : 1;
  const long long blocks = (p.n_tokens + tpb - 1) / tpb;
  if (blocks > 0x7FFFFFFFll) return FA_ERR_INVALID_ARG;
  const size_t smem = (size_t)tpb * (rotary_dim / 2) * sizeof(float2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64 && interleaved)
    fa_rope_kernel<64, true><<<(unsigned)blocks, 256, smem, s>>>(p, tpb);
  else if (d == 64)
    fa_rope_kernel<64, false><<<(unsigned)blocks, 256, smem, s>>>(p, tpb);
  else if (interleaved)
    fa_rope_kernel<128, true><<<(unsigned)blocks, 256, smem, s>>>(p, tpb);
  else
    fa_rope_kernel<128, false><<<(unsigned)blocks, 256, smem, s>>>(p, tpb);
  return launch_status();
}

}  // namespace fa

extern "C" int fa_rope(const void* q, void* q_out, const void* k, void* k_out, const int64_t* strides,
                       const int* positions, const double* freqs, int rotary_dim, int interleaved, float amplitude,
                       int B, int T, int Hq, int Hkv, int d, void* stream) {
  return rope_impl(q, q_out, k, k_out, strides, positions, freqs, rotary_dim, interleaved, amplitude, 1.f, B, T, Hq,
                   Hkv, d, stream);
}

extern "C" int fa_rope_backward(const void* dq, void* dq_out, const void* dk, void* dk_out, const int64_t* strides,
                                const int* positions, const double* freqs, int rotary_dim, int interleaved,
                                float amplitude, int B, int T, int Hq, int Hkv, int d, void* stream) {
  return rope_impl(dq, dq_out, dk, dk_out, strides, positions, freqs, rotary_dim, interleaved, amplitude, -1.f, B, T,
                   Hq, Hkv, d, stream);
}

// ---------------------------------------------------------------------------
// The 4-bit cache
// ---------------------------------------------------------------------------
namespace fa {

static int kv4_check_cache(const void* k_codes, const void* k_params, const void* v_codes, const void* v_params) {
  for (const void* ptr : {k_codes, k_params, v_codes, v_params}) {
    if (!ptr) return FA_ERR_INVALID_ARG;
    if (!aligned16(ptr)) return FA_ERR_ALIGNMENT;
  }
  return FA_OK;
}

static bool overlap(const void* x, size_t nx, const void* y, size_t ny) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b ? b - a < nx : a - b < ny;
}

// Whether any two of a cache's four buffers share memory: K's and V's blocks run
// in any order.
static bool kv4_cache_overlaps(const void* k_codes, const void* k_params, const void* v_codes, const void* v_params,
                               int B, int Hkv, int Tk_max, int d) {
  const size_t rows = (size_t)B * Hkv * Tk_max;
  const void* ptr[4] = {k_codes, k_params, v_codes, v_params};
  const size_t bytes[4] = {rows * (d / 2), rows * (d / 8), rows * (d / 2), rows * (d / 8)};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(ptr[i], bytes[i], ptr[j], bytes[j])) return true;
  return false;
}

static int kv4_check_sizes(int B, int Hkv, int Tk_max, int d) {
  if (B < 0 || Hkv < 1 || Tk_max < 0 || Tk_max % 64 != 0 || Tk_max > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

static int kv4_rows_blocks(Kv4RowsParams* p, int B, int T, int Hkv, int Tk_max, int d, unsigned* blocks) {
  p->T = T;
  p->H = Hkv;
  p->Tk_max = Tk_max;
  if (Hkv > (1 << 24) || T > (1 << 30)) return FA_ERR_INVALID_ARG;
  int nsm = 0;
  if (const int st = sm_count(&nsm)) return st;
  // Eight steps along the tokens where that still leaves four blocks a
  // multiprocessor, fewer where it does not.
  p->heads = Hkv >= 2 ? 2 : 1;
  p->parts = (Hkv + p->heads - 1) / p->heads;
  p->tokens = 256 / (p->heads * (d / 8));
  p->steps = 1;
  while (p->steps < 8 && (long long)B * (T / (p->tokens * p->steps * 2)) * p->parts >= 4 * nsm) p->steps *= 2;
  const long long per_seq = (((long long)T + p->tokens * p->steps - 1) / (p->tokens * p->steps)) * p->parts;
  const long long n = per_seq * B;
  if (n > 0x7FFFFFFFll) return FA_ERR_INVALID_ARG;
  p->blocks_per_seq = (unsigned)per_seq;
  *blocks = (unsigned)n;
  return FA_OK;
}

}  // namespace fa

extern "C" int fa_kv4_append(const void* k, const void* v, const int64_t* strides, void* k_codes, void* k_params,
                             void* v_codes, void* v_params, const int* start, const int* count, int B, int T, int Hkv,
                             int Tk_max, int d, void* stream) {
  int st = kv4_check_sizes(B, Hkv, Tk_max, d);
  if (st) return st;
  if (T < 0) return FA_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || Tk_max == 0) return FA_OK;
  if (!k || !v || !strides || !start) return FA_ERR_INVALID_ARG;
  if ((st = kv4_check_cache(k_codes, k_params, v_codes, v_params))) return st;
  for (int i = 0; i < 6; ++i)
    if (strides[i] < 0 || strides[i] > (1ll << 40)) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(start) & 3u) ||
      (reinterpret_cast<uintptr_t>(count) & 3u))
    return FA_ERR_ALIGNMENT;
  for (int i = 0; i < 6; ++i)
    if (strides[i] & 7) return FA_ERR_ALIGNMENT;
  if (kv4_cache_overlaps(k_codes, k_params, v_codes, v_params, B, Hkv, Tk_max, d)) return FA_ERR_INVALID_ARG;
  Kv4RowsParams p;
  memset(&p, 0, sizeof(p));
  unsigned blocks = 0;
  if ((st = kv4_rows_blocks(&p, B, T, Hkv, Tk_max, d, &blocks))) return st;
  p.x[0] = reinterpret_cast<const __nv_bfloat16*>(k);
  p.x[1] = reinterpret_cast<const __nv_bfloat16*>(v);
  for (int w = 0; w < 2; ++w) {
    p.xb[w] = strides[3 * w];
    p.xt[w] = strides[3 * w + 1];
    p.xh[w] = strides[3 * w + 2];
  }
  p.codes[0] = reinterpret_cast<uint8_t*>(k_codes);
  p.codes[1] = reinterpret_cast<uint8_t*>(v_codes);
  p.params[0] = reinterpret_cast<__nv_bfloat16*>(k_params);
  p.params[1] = reinterpret_cast<__nv_bfloat16*>(v_params);
  p.start = start;
  p.count = count;
  if ((st = device_setup())) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64)
    fa_kv4_append_kernel<64><<<dim3(blocks, 2), 256, 0, s>>>(p);
  else
    fa_kv4_append_kernel<128><<<dim3(blocks, 2), 256, 0, s>>>(p);
  return launch_status();
}

extern "C" int fa_kv4_read(void* k, void* v, const void* k_codes, const void* k_params, const void* v_codes,
                           const void* v_params, const int* start, const int* count, int B, int T, int Hkv,
                           int Tk_max, int d, void* stream) {
  int st = kv4_check_sizes(B, Hkv, Tk_max, d);
  if (st) return st;
  if (T < 0) return FA_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return FA_OK;
  if (!k || !v || !start) return FA_ERR_INVALID_ARG;
  if (Tk_max > 0 && (st = kv4_check_cache(k_codes, k_params, v_codes, v_params))) return st;
  if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(start) & 3u) ||
      (reinterpret_cast<uintptr_t>(count) & 3u))
    return FA_ERR_ALIGNMENT;
  const size_t out_bytes = (size_t)B * T * Hkv * d * 2;
  if (overlap(k, out_bytes, v, out_bytes)) return FA_ERR_INVALID_ARG;
  Kv4RowsParams p;
  memset(&p, 0, sizeof(p));
  unsigned blocks = 0;
  if ((st = kv4_rows_blocks(&p, B, T, Hkv, Tk_max, d, &blocks))) return st;
  p.y[0] = reinterpret_cast<__nv_bfloat16*>(k);
  p.y[1] = reinterpret_cast<__nv_bfloat16*>(v);
  p.codes[0] = reinterpret_cast<uint8_t*>(const_cast<void*>(k_codes));
  p.codes[1] = reinterpret_cast<uint8_t*>(const_cast<void*>(v_codes));
  p.params[0] = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(k_params));
  p.params[1] = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(v_params));
  p.start = start;
  p.count = count;
  if ((st = device_setup())) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64)
    fa_kv4_read_kernel<64><<<dim3(blocks, 2), 256, 0, s>>>(p);
  else
    fa_kv4_read_kernel<128><<<dim3(blocks, 2), 256, 0, s>>>(p);
  return launch_status();
}

namespace fa {

// Workspace pieces: prefix, then (maximum, sum), then O of every slot.
struct Kv4Ws {
  size_t ml, o, bytes;
};
static Kv4Ws kv4_ws(int B, int Hq, int Hkv, int d) {
  const size_t nb = std::min(B, kKv4MaxSeqs);
  const size_t rows = (nb * Hkv + kKv4MaxGrid) * (Hq / Hkv);
  Kv4Ws w;
  w.ml = round256((nb + 1) * 4);
  w.o = w.ml + round256(rows * 8);
  w.bytes = w.o + round256(rows * d * 4);
  return w;
}

template <int D, int G>
static int kv4_launch(const Kv4DecodeParams& p, cudaStream_t s) {
  fa_kv4_split_kernel<D, G><<<p.n_cta, Kv4Cfg<D, G>::THREADS, Kv4Cfg<D, G>::SMEM_BYTES, s>>>(p);
  return launch_status();
}

}  // namespace fa

extern "C" size_t fa_kv4_decode_workspace_bytes(int B, int Hq, int Hkv, int Tk_max, int d) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Tk_max < 0 || (d != 64 && d != 128)) return 0;
  return kv4_ws(B, Hq, Hkv, d).bytes;
}

extern "C" int fa_kv4_decode(const void* q, const void* k_codes, const void* k_params, const void* v_codes,
                             const void* v_params, const int* seqlens_k, void* o, float* lse, void* ws,
                             size_t ws_bytes, int B, int Hq, int Hkv, int Tk_max, int d, float scale, int window,
                             int sinks, void* stream) {
  int st = kv4_check_sizes(B, Hkv, Tk_max, d);
  if (st) return st;
  if (Hq < 1 || Hq % Hkv != 0 || !isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (window < 0 || window > (1 << 30) || sinks < 0 || sinks > kMaxSinks || (sinks > 0 && window == 0))
    return FA_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return FA_ERR_UNSUPPORTED;
  // tiles of the list and (sequence, KV head) pairs are counted in 31 bits
  if ((int64_t)B * Hq > (1 << 26) || (int64_t)B * Hkv * (Tk_max / 64) > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!q || !seqlens_k || !o || !lse) return FA_ERR_INVALID_ARG;
  if (Tk_max > 0 && (st = kv4_check_cache(k_codes, k_params, v_codes, v_params))) return st;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || (reinterpret_cast<uintptr_t>(seqlens_k) & 3u))
    return FA_ERR_ALIGNMENT;
  const Kv4Ws w = kv4_ws(B, Hq, Hkv, d);
  if (!ws || ws_bytes < w.bytes || !aligned16(ws)) return FA_ERR_WORKSPACE;
  if ((st = device_setup())) return st;
  int nsm = 0;
  if ((st = sm_count(&nsm))) return st;
  Kv4DecodeParams p;
  memset(&p, 0, sizeof(p));
  p.k_codes = reinterpret_cast<const uint8_t*>(k_codes);
  p.v_codes = reinterpret_cast<const uint8_t*>(v_codes);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  p.ws_prefix = reinterpret_cast<int*>(base);
  p.ws_ml = reinterpret_cast<float*>(base + w.ml);
  p.ws_o = reinterpret_cast<float*>(base + w.o);
  p.k_params = reinterpret_cast<const __nv_bfloat16*>(k_params);
  p.v_params = reinterpret_cast<const __nv_bfloat16*>(v_params);
  p.Hq = Hq; p.Hkv = Hkv; p.Tk_max = Tk_max;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int b0 = 0; b0 < B; b0 += kKv4MaxSeqs) {
    p.B = std::min(B - b0, kKv4MaxSeqs);
    p.pair0 = b0 * Hkv;
    p.q = reinterpret_cast<const __nv_bfloat16*>(q) + (size_t)b0 * Hq * d;
    p.seqlens = seqlens_k + b0;
    p.o = reinterpret_cast<__nv_bfloat16*>(o) + (size_t)b0 * Hq * d;
    p.lse = lse + (size_t)b0 * Hq;
    // no more blocks than the longest possible list has tiles
    const long long tiles = (long long)p.B * Hkv * (Tk_max / 64);
#define FA_KV4_LAUNCH(DD, GG)                                                                                   \
    (p.n_cta = (int)std::min({(long long)nsm * Kv4Cfg<DD, GG>::CTAS, (long long)kKv4MaxGrid, std::max(tiles, 1ll)}), \
     st = kv4_launch<DD, GG>(p, s))
    if (d == 64) {
      if (G == 1) FA_KV4_LAUNCH(64, 1); else if (G == 2) FA_KV4_LAUNCH(64, 2);
      else if (G == 4) FA_KV4_LAUNCH(64, 4); else FA_KV4_LAUNCH(64, 8);
    } else {
      if (G == 1) FA_KV4_LAUNCH(128, 1); else if (G == 2) FA_KV4_LAUNCH(128, 2);
      else if (G == 4) FA_KV4_LAUNCH(128, 4); else FA_KV4_LAUNCH(128, 8);
    }
#undef FA_KV4_LAUNCH
    if (st) return st;
    const unsigned blocks = (unsigned)(((size_t)p.B * Hq * 32 + 127) / 128);
    if ((st = launch_after(d == 64 ? fa_kv4_combine_kernel<64> : fa_kv4_combine_kernel<128>, blocks, 128, s, p)))
      return st;
  }
  return FA_OK;
}
