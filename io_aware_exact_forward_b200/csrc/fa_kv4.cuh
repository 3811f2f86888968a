// fa_kv4.cuh -- a KV cache held in 4 bits: appending, reading back, and
// split-KV decode over it.
//
// Format.  A row of d values is cut into groups of 32.  With lo and hi the
// group's least and largest value,
//   s = bf16((hi - lo) / 15),  z = bf16(lo + 8 s),
//   c = clamp(round((x - z) / s), -8, 7) + 8   (ties to even; 8 where s = 0),
// and the value held is z + s (c - 8).  Codes: d / 2 bytes a row, dim 2i in
// the low nibble of byte i.  Params: the row's steps s, then its centres z, as
// bf16.  Rows of one (sequence, KV head) are contiguous: codes
// [B][Hkv][Tk_max][d/2], params [B][Hkv][Tk_max][2 d/32].  A key and its value
// take 160 bytes at d = 128, against 512 in bf16.  The centre, not the least
// value, is kept, so that the codes' part of a value is as small as it can be
// and rounding a probability times a step costs what rounding the probability
// alone does.  (hi - lo) is formed as 0.5 hi - 0.5 lo over 7.5, which cannot
// overflow.  A group that holds a NaN or an infinity reads back non-finite.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

static constexpr int kKv4Group = 32;

struct Kv4RowsParams {
  const __nv_bfloat16* x[2];  // append: K, V rows [B][T][H][d], last dim contiguous
  long long xb[2], xt[2], xh[2];
  __nv_bfloat16* y[2];        // read: [B][T][H][d], dense
  uint8_t* codes[2];
  __nv_bfloat16* params[2];
  const int* start;           // [B]: cache position of row t = 0
  const int* count;           // [B] rows of sequence b, or null: all T
  long long units;            // B * T * H * (d / 8)
  int T, H, Tk_max;
};

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight elements (16 bytes) of one row per thread; the four threads of a
// group exchange its least and largest value by shuffles.  blockIdx.y = 0: K,
// 1: V.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_append_kernel(const __grid_constant__ Kv4RowsParams p) {
  constexpr int CH = D / 8, NG = D / kKv4Group;
  const int which = blockIdx.y;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const bool in = i < p.units;
  const long long j = in ? i : 0;
  const int ch = (int)(j % CH);
  const long long row = j / CH;
  const int h = (int)(row % p.H);
  const long long bt = row / p.H;
  const int t = (int)(bt % p.T);
  const int b = (int)(bt / p.T);
  const long long pos = (long long)p.start[b] + t;
  const bool keep = in && t < (p.count ? p.count[b] : p.T) && pos >= 0 && pos < p.Tk_max;
  const uint4 raw =
      *reinterpret_cast<const uint4*>(p.x[which] + b * p.xb[which] + t * p.xt[which] + h * p.xh[which] + ch * 8);
  const uint32_t* rw = reinterpret_cast<const uint32_t*>(&raw);
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&rw[e]));
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = min_nan(lo, x[e]);
    hi = max_nan(hi, x[e]);
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(0.5f * hi, 0.5f * lo), 7.5f));
  const float s = __bfloat162float(sb);
  const __nv_bfloat16 zb = __float2bfloat16_rn(fmaf(8.f, s, lo));  // 8 s alone may overflow
  const float z = __bfloat162float(zb);
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float c = rintf(__fdiv_rn(__fsub_rn(x[e], z), s));
    c = fminf(fmaxf(c, -8.f), 7.f);
    const int code = s > 0.f ? (int)c + 8 : 8;
    word |= (uint32_t)(code & 15) << (4 * e);
  }
  if (keep) {
    const size_t r = ((size_t)b * p.H + h) * p.Tk_max + (size_t)pos;
    *reinterpret_cast<uint32_t*>(p.codes[which] + r * (D / 2) + ch * 4) = word;
    if ((ch & 3) == 0) {
      __nv_bfloat16* pr = p.params[which] + r * (2 * NG) + (ch >> 2);
      pr[0] = sb;
      pr[NG] = zb;
    }
  }
}

// The values of cache rows, rounded to bf16.  Rows past a sequence's count or
// outside the cache are written as zeros.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const __grid_constant__ Kv4RowsParams p) {
  constexpr int CH = D / 8, NG = D / kKv4Group;
  const int which = blockIdx.y;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.units) return;
  const int ch = (int)(i % CH);
  const long long row = i / CH;
  const int h = (int)(row % p.H);
  const long long bt = row / p.H;
  const int t = (int)(bt % p.T);
  const int b = (int)(bt / p.T);
  const long long pos = (long long)p.start[b] + t;
  uint4 out = make_uint4(0u, 0u, 0u, 0u);
  if (t < (p.count ? p.count[b] : p.T) && pos >= 0 && pos < p.Tk_max) {
    const size_t r = ((size_t)b * p.H + h) * p.Tk_max + (size_t)pos;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(p.codes[which] + r * (D / 2) + ch * 4);
    const __nv_bfloat16* pr = p.params[which] + r * (2 * NG) + (ch >> 2);
    const float s = __bfloat162float(pr[0]), z = __bfloat162float(pr[NG]);
    uint32_t* w = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c0 = (float)((int)((word >> (8 * e)) & 15u) - 8);
      const float c1 = (float)((int)((word >> (8 * e + 4)) & 15u) - 8);
      // s (c - 8) is exact in 32 bits (8 by 4 bits), so one rounding each
      w[e] = pack_bf16x2(fmaf(s, c0, z), fmaf(s, c1, z));
    }
  }
  *reinterpret_cast<uint4*>(p.y[which] + row * D + ch * 8) = out;
}

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
struct Kv4DecodeParams {
  const __nv_bfloat16* q;  // [B][Hq][d]
  const uint8_t* k_codes;  // [B][Hkv][Tk_max][d/2]
  const uint8_t* v_codes;
  const __nv_bfloat16* k_params;  // [B][Hkv][Tk_max][2 d/32]
  const __nv_bfloat16* v_params;
  const int* seqlens;      // [B]
  float* ws_o;             // [B * Hkv][nsplit][G][d], O scaled by its own maximum
  float* ws_ml;            // [B * Hkv][nsplit][G][2], maximum (log2 units) and sum
  __nv_bfloat16* o;        // [B][Hq][d]
  float* lse;              // [B][Hq]
  int B, Hq, Hkv, Tk_max, nsplit, chunk;
  int window, sinks;       // window > 0: only the last `window` keys and the first `sinks`
  float scale_log2;
};

__device__ __forceinline__ int kv4_len(const Kv4DecodeParams& p, int b) { return min(max(p.seqlens[b], 0), p.Tk_max); }

// One block per (chunk, sequence and KV head): four warps take the chunk's
// keys in turn, each lane d / 32 dims of all G query heads.
template <int D, int G>
__global__ void __launch_bounds__(128) fa_kv4_split_kernel(const __grid_constant__ Kv4DecodeParams p) {
  constexpr int E = D / 32, NG = D / kKv4Group;
  __shared__ float so[4][G][D];
  __shared__ float sml[4][G][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.Hkv, hkv = bh % p.Hkv;
  const int len = kv4_len(p, b);
  const int lo = p.window > 0 ? max(0, len - p.window) : 0;
  const int k0 = blockIdx.x * p.chunk, k1 = min(k0 + p.chunk, len);
  float q[G][E], o[G][E], m[G], l[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[g][e] = __bfloat162float(p.q[((size_t)b * p.Hq + hkv * G + g) * D + lane * E + e]);
      o[g][e] = 0.f;
    }
  }
  for (int key = k0 + warp; key < k1; key += 4) {
    if (key < lo && key >= p.sinks) continue;
    const size_t r = (size_t)bh * p.Tk_max + key;
    float kv[2][E];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* c = (w ? p.v_codes : p.k_codes) + r * (D / 2) + lane * (E / 2);
      const __nv_bfloat16* pr = (w ? p.v_params : p.k_params) + r * 2 * NG + lane * E / kKv4Group;
      const float s = __bfloat162float(pr[0]), z = __bfloat162float(pr[NG]);
#pragma unroll
      for (int e = 0; e < E; ++e) kv[w][e] = fmaf(s, (float)((c[e >> 1] >> (4 * (e & 1))) & 15) - 8.f, z);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) d = fmaf(q[g][e], kv[0][e], d);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      d *= p.scale_log2;
      const float mn = fmaxf(m[g], d);
      const float ref = mn == -INFINITY ? 0.f : mn;  // a NaN score stays one
      const float a = ex2_approx(m[g] - ref);
      const float w = ex2_approx(d - ref);
      m[g] = mn;
      l[g] = fmaf(l[g], a, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = fmaf(w, kv[1][e], o[g][e] * a);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][g][lane * E + e] = o[g][e];
    if (lane == 0) {
      sml[warp][g][0] = m[g];
      sml[warp][g][1] = l[g];
    }
  }
  __syncthreads();
  const size_t slot = (size_t)bh * p.nsplit + blockIdx.x;
  for (int i = threadIdx.x; i < G * D; i += 128) {
    const int g = i / D, e = i % D;
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sml[w][g][0]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = sml[w][g][0] == -INFINITY ? 0.f : ex2_approx(sml[w][g][0] - M);
      L = fmaf(f, sml[w][g][1], L);
      O = fmaf(f, so[w][g][e], O);
    }
    p.ws_o[(slot * G + g) * D + e] = O;
    if (e == 0) {
      p.ws_ml[(slot * G + g) * 2] = M;
      p.ws_ml[(slot * G + g) * 2 + 1] = L;
    }
  }
}

// One warp per (sequence, query head): the chunks' results joined.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_combine_kernel(const __grid_constant__ Kv4DecodeParams p) {
  constexpr int E = D / 32;
  const int row = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (row >= p.B * p.Hq) return;
  const int G = p.Hq / p.Hkv;
  const int b = row / p.Hq, h = row % p.Hq;
  const size_t s0 = ((size_t)b * p.Hkv + h / G) * p.nsplit;
  float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int c = 0; c < p.nsplit; ++c) M = fmaxf(M, p.ws_ml[((s0 + c) * G + h % G) * 2]);
  for (int c = 0; c < p.nsplit; ++c) {
    const size_t at = (s0 + c) * G + h % G;
    const float m = p.ws_ml[at * 2];
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - M);
    L = fmaf(f, p.ws_ml[at * 2 + 1], L);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(f, p.ws_o[at * D + lane * E + e], o[e]);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __nv_bfloat16* dst = p.o + (size_t)row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (lane == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace fa
