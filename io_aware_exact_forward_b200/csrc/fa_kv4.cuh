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

#include "fa_decode.cuh"
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
  int T, H, Tk_max;
  // a block: `heads` heads (one of `parts` such groups) of `tokens` tokens side by
  // side, `steps` times along the tokens
  unsigned blocks_per_seq;
  int heads, tokens, parts, steps;
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

// The constants of the conversions are in registers that the compiler cannot see
// through: as literals, the mask and the OR are two instructions (an instruction
// takes one literal), not one.
struct Kv4PairsBf16 {
  uint32_t m128, m136;  // pairs of 128 and 136
  __device__ __forceinline__ Kv4PairsBf16() {
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(m128));
    asm volatile("mov.b32 %0, 0x43084308;" : "=r"(m136));
  }
  // Nibble k of both halves as the bf16 pair u - 8: ORed into 128, less 136.
  __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w, int k) const {
    uint32_t u;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(u) : "r"(w >> (4 * k)), "r"(m128));
    return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&m136));
  }
};
struct Kv4PairsF16 {
  uint32_t h1024, h1032, h16, h72;  // pairs of 1024, -1032, 1 / 16, -72
  __device__ __forceinline__ Kv4PairsF16() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(h1024));
    asm volatile("mov.b32 %0, 0xE408E408;" : "=r"(h1032));
    asm volatile("mov.b32 %0, 0x2C002C00;" : "=r"(h16));
    asm volatile("mov.b32 %0, 0xD480D480;" : "=r"(h72));
  }
  // Nibbles 0 and 1 of both halves as the fp16 pairs u - 8 (of the word shifted
  // by 8: nibbles 2 and 3), from 1024 + u and 1024 + 16 u.
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t& n0, uint32_t& n1) const {
    uint32_t a, b;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(a) : "r"(w), "r"(h1024));
    asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(b) : "r"(w), "r"(h1024));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(n0) : "r"(a), "r"(h1032));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(n1) : "r"(b), "r"(h16), "r"(h72));
  }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Both kernels below take units of eight elements of one row.  A thread keeps its
// head and its place in the row and walks along the tokens, so that indexes are
// divided out once; a block has two heads of 8 tokens (d = 128; 16 at 64) side by
// side, so that it meets 512 contiguous bytes on either side at a time.  The bytes
// (2 an element on one side and 0.625 on the other) would take 27 us each way for
// 32k tokens of 8 heads of 128: read takes 31.  Append takes 54, by issue and the
// half-rate integer pipe: 165 instructions per warp and unit, 47% of them on that
// pipe, keep it 73% busy and the issue slots 77%.  One index per unit
// divided out in 64 bits and a division per element took 110 and 56 us, in 32 bits
// without the divisions 64 and 45.
struct Kv4Place {
  int b, h, ch, t;  // sequence, head, unit of the row, first token
  bool in;
  template <int CH>
  static __device__ __forceinline__ Kv4Place of(const Kv4RowsParams& p) {
    Kv4Place w;
    w.b = (int)(blockIdx.x / p.blocks_per_seq);
    const unsigned r = blockIdx.x - (unsigned)w.b * p.blocks_per_seq;
    const unsigned tb = r / (unsigned)p.parts, part = r - tb * (unsigned)p.parts;
    const unsigned row = threadIdx.x / CH;
    const unsigned tl = p.heads == 2 ? row >> 1 : row;
    w.ch = (int)(threadIdx.x % CH);
    w.h = (int)(part * p.heads + (row - tl * p.heads));
    w.in = w.h < p.H;
    if (!w.in) w.h = 0;
    w.t = (int)(tb * (unsigned)(p.tokens * p.steps) + tl);
    return w;
  }
};

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// round(t / s) + 8 of eight values, clamped to 0..15, as nibbles.  The quotient is
// t inv + t inv_lo with inv + inv_lo = 1 / s to 45 bits: rounded once to fp32 it is
// the division's own result (a quotient by an 8-bit s stays 2^-32 or more away from
// where the rounding turns), ties of the code included, of which bf16 inputs have
// many (a third of a percent of N(0,1) values).  Added to 1.5 2^23 + 8, the code is
// the sum's low bits.
__device__ __forceinline__ uint32_t kv4_codes(const float2 (&t)[4], float s) {
  constexpr float M = 12582912.f;  // 1.5 2^23
  uint32_t word = 0u;
  if (s >= 0x1p-100f && s <= 0x1p100f) {
    const float inv = rcp_approx(s), inv_lo = fmaf(-s, inv, 1.f) * inv;
    const float2 i2 = make_float2(inv, inv), l2 = make_float2(inv_lo, inv_lo), m2 = make_float2(M + 8.f, M + 8.f);
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      const float2 y = __fadd2_rn(__ffma2_rn(t[e], i2, __fmul2_rn(t[e], l2)), m2);
      word = word * 16u + __float_as_uint(fminf(fmaxf(y.y, M), M + 15.f));
      word = word * 16u + __float_as_uint(fminf(fmaxf(y.x, M), M + 15.f));
    }
    return word - 0x4B400000u * 0x11111111u;  // M's own bits, eight times over
  }
  if (!(s > 0.f)) return 0x88888888u;
#pragma unroll
  for (int e = 7; e >= 0; --e) {
    const float c = fminf(fmaxf(rintf(__fdiv_rn(e & 1 ? t[e >> 1].y : t[e >> 1].x, s)), -8.f), 7.f);
    word = word * 16u + (uint32_t)((int)c + 8);
  }
  return word;
}

// x / 7.5, rounded once: x times 1 / 7.5 in two parts, as above.
__device__ __forceinline__ float div_7_5(float x) {
  constexpr float inv = 1.f / 7.5f, inv_lo = (float)(1.0 / 7.5 - (double)inv);
  if (x >= 0x1p-90f && x <= 0x1p127f) return fmaf(x, inv, __fmul_rn(x, inv_lo));
  return __fdiv_rn(x, 7.5f);
}

// The four threads of a group exchange its least and largest value by shuffles.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_append_kernel(const __grid_constant__ Kv4RowsParams p) {
  constexpr int CH = D / 8, NG = D / kKv4Group;
  const int which = blockIdx.y;
  const Kv4Place w = Kv4Place::of<CH>(p);
  const int start = p.start[w.b], count = p.count ? min(p.count[w.b], p.T) : p.T;
  const __nv_bfloat16* x = p.x[which] + w.b * p.xb[which] + w.h * p.xh[which] + w.ch * 8;
  const size_t row0 = ((size_t)w.b * p.H + w.h) * p.Tk_max;
  uint8_t* codes = p.codes[which] + row0 * (D / 2) + w.ch * 4;
  __nv_bfloat16* params = p.params[which] + row0 * (2 * NG);
  const long long xt = p.xt[which];
  constexpr int U = 4;  // loads in flight
  for (int n0 = 0; n0 < p.steps; n0 += U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // every thread takes part in the shuffles; one past the end reads row 0
      const int t = w.t + (n0 + u) * p.tokens;
      raw[u] = *reinterpret_cast<const uint4*>(x + (w.in && n0 + u < p.steps && t < p.T ? t : 0) * xt);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (n0 + u >= p.steps) break;
      const int t = w.t + (n0 + u) * p.tokens;
      const uint32_t rw[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      auto pair = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
      auto bits = [](__nv_bfloat162 w) { return *reinterpret_cast<const uint32_t*>(&w); };
      uint32_t lo2 = bits(__hmin2_nan(__hmin2_nan(pair(rw[0]), pair(rw[1])), __hmin2_nan(pair(rw[2]), pair(rw[3]))));
      uint32_t hi2 = bits(__hmax2_nan(__hmax2_nan(pair(rw[0]), pair(rw[1])), __hmax2_nan(pair(rw[2]), pair(rw[3]))));
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        lo2 = bits(__hmin2_nan(pair(lo2), pair(__shfl_xor_sync(0xffffffffu, lo2, off))));
        hi2 = bits(__hmax2_nan(pair(hi2), pair(__shfl_xor_sync(0xffffffffu, hi2, off))));
      }
      const float lo = min_nan(bf16_lo(lo2), bf16_hi(lo2)), hi = max_nan(bf16_lo(hi2), bf16_hi(hi2));
      const __nv_bfloat16 sb = __float2bfloat16_rn(div_7_5(__fsub_rn(0.5f * hi, 0.5f * lo)));
      const float s = __bfloat162float(sb);
      const __nv_bfloat16 zb = __float2bfloat16_rn(fmaf(8.f, s, lo));  // 8 s alone may overflow
      const float z = __bfloat162float(zb);
      float2 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(make_float2(bf16_lo(rw[e]), bf16_hi(rw[e])), make_float2(-z, -z));
      const uint32_t word = kv4_codes(v, s);
      // the row's steps and centres at its first thread, for one store
      const __nv_bfloat162 sz = __halves2bfloat162(sb, zb);
      const uint32_t w0 = bits(sz);
      const uint32_t w1 = __shfl_down_sync(0xffffffffu, w0, 4, CH);
      uint32_t w2 = 0u, w3 = 0u;
      if constexpr (NG == 4) {
        w2 = __shfl_down_sync(0xffffffffu, w0, 8, CH);
        w3 = __shfl_down_sync(0xffffffffu, w0, 12, CH);
      }
      const long long pos = (long long)start + t;
      if (w.in && t < count && pos >= 0 && pos < p.Tk_max) {
        *reinterpret_cast<uint32_t*>(codes + (size_t)pos * (D / 2)) = word;
        if (w.ch == 0) {
          const uint32_t s01 = __byte_perm(w0, w1, 0x5410), z01 = __byte_perm(w0, w1, 0x7632);
          __nv_bfloat16* pr = params + (size_t)pos * (2 * NG);
          if constexpr (NG == 4)
            *reinterpret_cast<uint4*>(pr) = make_uint4(s01, __byte_perm(w2, w3, 0x5410), z01,
                                                       __byte_perm(w2, w3, 0x7632));
          else
            *reinterpret_cast<uint2*>(pr) = make_uint2(s01, z01);
        }
      }
    }
  }
}

// The values of cache rows, rounded to bf16.  Rows past a sequence's count or
// outside the cache are written as zeros.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const __grid_constant__ Kv4RowsParams p) {
  constexpr int CH = D / 8, NG = D / kKv4Group;
  const int which = blockIdx.y;
  const Kv4Place w = Kv4Place::of<CH>(p);
  if (!w.in) return;
  const Kv4PairsBf16 bf;
  const int start = p.start[w.b], count = p.count ? min(p.count[w.b], p.T) : p.T;
  const size_t row0 = ((size_t)w.b * p.H + w.h) * p.Tk_max;
  const uint8_t* codes = p.codes[which] + row0 * (D / 2) + w.ch * 4;
  const __nv_bfloat16* params = p.params[which] + row0 * (2 * NG) + (w.ch >> 2);
  __nv_bfloat16* y = p.y[which] + ((size_t)w.b * p.T * p.H + w.h) * D + w.ch * 8;
  constexpr int U = 4;  // loads in flight
  for (int n = 0; n < p.steps; n += U) {
    uint32_t word[U];
    __nv_bfloat16 s[U], z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = w.t + (n + u) * p.tokens;
      const long long pos = (long long)start + t;
      word[u] = 0x88888888u;  // zeros
      s[u] = z[u] = __float2bfloat16_rn(0.f);
      if (n + u < p.steps && t < count && pos >= 0 && pos < p.Tk_max) {
        word[u] = *reinterpret_cast<const uint32_t*>(codes + (size_t)pos * (D / 2));
        const __nv_bfloat16* pr = params + (size_t)pos * (2 * NG);
        s[u] = pr[0];
        z[u] = pr[NG];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = w.t + (n + u) * p.tokens;
      // pairs (k, k + 4) of the row: s (u - 8) + z in one fused, once rounded step
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 x =
            __hfma2(__halves2bfloat162(s[u], s[u]), bf.pair(word[u], k), __halves2bfloat162(z[u], z[u]));
        q[k] = *reinterpret_cast<const uint32_t*>(&x);
      }
      if (n + u < p.steps && t < p.T)
        *reinterpret_cast<uint4*>(y + (size_t)t * p.H * D) =
            make_uint4(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                       __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
    }
  }
}

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
// With u = code as an integer 0..15 and s, z of key j and group c,
//   S_j = scale sum_c ( s_jc sum_{i in c} q_i (u_ij - 8) + z_jc sum_{i in c} q_i ),
//   O_i = sum_j ( p_j s_jc (u_ij - 8) + p_j z_jc ) / l       (i in group c),
// so the steps never touch the d codes of a row: they scale 32-bit sums of four
// group products of a score, and the probabilities on the way into P V.
//
// On the tensor cores (mma.sync m16n8k16: a decode has too few rows for a
// tcgen05 tile) the codes are the fp16 numbers u - 8, without a conversion: a
// nibble masked and ORed into 1024, where it stands (1024 + u, or 1024 + 16 u), is
// brought to u - 8 by one exact fp16 addition or fused multiply-add, so that a
// 32-bit word of eight codes takes one shift.  (bf16 holds one nibble of every
// four, hence three shifts; the shifts and masks go through the half-rate integer
// pipe, the busiest of this kernel.)
// Q enters as fp16 after scaling its row by a power of two to a largest value in
// [2^14, 2^15): a bf16 value is then exact down to 2^-31 of the row's largest, and
// smaller ones are within 2^-39 of it.  The centres' parts are two small bf16
// products of their own: z against sum q (in three bf16 parts, 24 bits), and p
// against z.
//
// p s is formed in 32 bits and rounded to fp16 once (2^-11 of itself); l sums the
// unrounded p.  fp16's range: V's steps, and nothing else, carry a power of two
// that brings the largest so far to 2^19 .. 2^20 against a p of 2^-16 and less (the
// reference of the exponentials is 16 above the maximum, so that sums of p times
// large centres have room).  It is lowered when a step eight times as large comes,
// and the sums of the codes' part with it; m, l and the centres' part, and so the
// log-sum-exp, do not depend on it.  Each group of the dims has its own, so that an
// infinity or a very large value in one leaves the others as they are.  A p s that is 2^18
// below the largest possible loses bits and one 2^28 below it is dropped: that is p
// itself, or a key whose step is that much smaller than others of its group that
// the same warp has met.  A slice's steps are scaled where they lie in shared
// memory, a key by each lane (four instructions a slice; as factors on the
// probabilities they would be sixteen).
//
// Operand layouts.  A 16-byte chunk of a row's codes is one group.  For K,
// ldmatrix gives lane (g, t) of a warp the word of key g's dims 8t .. 8t + 7 of
// the group: nibble k of its halves is the pair of dims (8t + k, 8t + 4 + k),
// and Q is permuted to match.  For V, ldmatrix.trans gives keys 2t and 2t + 1
// (the halves) at dims 4g .. 4g + 3: nibble k is the pair of keys that P^T's
// operand wants, so V^T enters as the row operand, 16 dims by 16 keys, and P^T
// as the column operand: both come out of the score's accumulator in place.
//
// Work.  A persistent grid; every sequence's visible 128-key tiles, in the order
// of (sequence, KV head), are one long list that the blocks share out evenly
// whatever the lengths are.  A block's stretch of one (sequence, KV head) ends
// in a partial result (slot: block + pair, both grow along the list), and a
// second kernel joins them.  64 sequences of 1k to 32k keys (8 KV heads of 128,
// 1.39 GB) take 288 us, 4.81 TB/s; the bytes alone would take 214.  What holds it
// back then is latency: about 337 instructions per warp and 16 keys are issued at
// 0.59 a cycle, no pipe is busy half of the time (ALU 48%, tensor 38%, FMA 37%), and
// the largest stall is the fixed wait for the instruction before, which three warps
// a scheduler do not cover.
// Each warp of a block takes 32 keys of every tile through a ring of its own, which
// all its lanes fill with 16-byte asynchronous copies: no warp waits for another
// before a stretch ends, none is spent on loading, and a slice costs ten copies (as
// four bulk copies issued by one lane it cost the warp about twice the
// instructions, and 313 us where the copies take 297).
static constexpr int kKv4MaxSeqs = 1024;  // sequences per launch
static constexpr int kKv4MaxGrid = 1024;

static constexpr int kKv4RefAbove = 16;  // exponentials' reference above the maximum, in log2 units

// The powers of two on V's steps, of two groups in a bf16 pair: 2^126 at first
// and at most, 2^-105 at least (any finite step is below 2^20 then).
static constexpr uint32_t kKv4FactorMax = 0x7E807E80u;
static constexpr uint32_t kKv4ScaledMax = 0x4B004B00u;  // 2^23: a step that is larger when scaled lowers its factor
// The factor (its bf16 exponent) that brings a step, a bf16, to 2^19 .. 2^20.
__device__ __forceinline__ int kv4_factor_exp(uint32_t step) {
  return 277 - min(max((int)((step >> 7) & 0xFFu) + 4, 24), 255);
}

struct Kv4DecodeParams {
  const __nv_bfloat16* q;  // [B][Hq][d]
  const uint8_t* k_codes;  // [B][Hkv][Tk_max][d/2]
  const uint8_t* v_codes;
  const __nv_bfloat16* k_params;  // [B][Hkv][Tk_max][2 d/32]
  const __nv_bfloat16* v_params;
  const int* seqlens;      // [B]
  int* ws_prefix;          // [B + 1] visible tiles before sequence b
  float* ws_ml;            // [slot][G][2], maximum (log2 units) and sum
  float* ws_o;             // [slot][G][d], unnormalised
  __nv_bfloat16* o;        // [B][Hq][d]
  float* lse;              // [B][Hq]
  int B, Hq, Hkv, Tk_max;
  int pair0;               // (sequence, KV head) pairs before this launch's in the cache
  int n_cta;
  int window, sinks;       // window > 0: only the last `window` keys and the first `sinks`
  float scale_log2;
};

// Visible tiles of a sequence: 0 .. n_sink - 1, then lo_tile ..; `count` in all.
struct Kv4Seq {
  int len, lo, n_sink, lo_tile, count;
  __device__ __forceinline__ Kv4Seq(const Kv4DecodeParams& p, int seqlen) {
    len = min(max(seqlen, 0), p.Tk_max);
    lo = p.window > 0 ? max(0, len - p.window) : 0;
    const int end = (len + 127) >> 7;
    n_sink = min(end, (p.sinks + 127) >> 7);
    lo_tile = max(n_sink, lo >> 7);
    count = n_sink + max(0, end - lo_tile);
  }
  __device__ __forceinline__ int tile(int j) const { return j < n_sink ? j : lo_tile + j - n_sink; }
};

template <int D, int G>
struct Kv4Cfg {
  static constexpr int SLICE = 32;                    // keys of a warp's stage
  static constexpr int NWARP = 4;
  static constexpr int TILE = NWARP * SLICE;
  static constexpr int THREADS = NWARP * 32;
  static constexpr int CB = D / 2, NG = D / kKv4Group, PB = 4 * NG;  // bytes of a row's codes, groups, bytes of params
  static constexpr int OFF_K = 0, OFF_V = SLICE * CB, OFF_KP = 2 * SLICE * CB, OFF_VP = OFF_KP + SLICE * PB;
  static constexpr int STAGE_BYTES = OFF_VP + SLICE * PB;
  static constexpr int NSTAGE = (D == 128) ? 2 : 4;              // per warp
  static constexpr int OFF_MRG = NWARP * NSTAGE * STAGE_BYTES;   // [NWARP][G][D / 2] fp32: half the dims at a time
  static constexpr int OFF_ML = OFF_MRG + NWARP * G * D * 2;     // m, l: [NWARP][8] each
  static constexpr int OFF_PRE = OFF_ML + 2 * NWARP * 8 * 4;     // prefix [kKv4MaxSeqs + 1]
  static constexpr int OFF_SCAN = OFF_PRE + (kKv4MaxSeqs + 4) * 4;
  static constexpr int SMEM_BYTES = OFF_SCAN + 64 + 1024;        // + alignment slack
  // Blocks per SM: 12 warps of 168 registers at d = 128 (285 us on 64 sequences of
  // 1k to 32k keys where 16 of 128 took 297), 16 of 128 at d = 64 (178 where 12 took
  // 186); 288 and 177 with V's steps scaled in shared memory.
  static constexpr int CTAS = D == 128 ? 3 : 4;
  static constexpr float RESCALE_THRESHOLD = 8.0f;
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 233472, "shared memory of an SM");
};

// Byte offset of 16-byte chunk c of row r of a code tile: the chunk is moved so
// that the 8 rows of an ldmatrix fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t kv4_swz(int r, int c) {
  if constexpr (D == 128) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
}
// D = A B with k = 8.
__device__ __forceinline__ void mma_1688_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
// D = A B (C = 0) and D += A B in fp16.
__device__ __forceinline__ void mma_f16_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t x, uint32_t y) {  // a number, of a number and a NaN
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Whether either of a bf16 pair is above its limit (NaN is not).
__device__ __forceinline__ bool bf16x2_any_gt(uint32_t x, uint32_t lim) {
  uint32_t r;
  asm("{\n\t.reg .pred p, q;\n\tsetp.gt.bf16x2 p|q, %1, %2;\n\tor.pred p, p, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x), "r"(lim));
  return r != 0;
}

// Asynchronous copy of N bytes, global to shared, past L1 where N is 16.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The steps of one row's params, as words of two.
template <int NG>
__device__ __forceinline__ void kv4_steps(uint32_t addr, uint32_t (&w)[NG / 2]) {
  if constexpr (NG == 4) {
    const uint2 v = lds64(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = lds32(addr);
  }
}

// One stretch of the tile list within one (sequence, KV head), as one warp
// walks it: its slice of the stretch's j-th tile starts at key(j).
struct Kv4Stretch {
  int n, pair;             // tiles; (sequence, KV head) within this launch
  int len, lo;             // the sequence's keys, and the first in its window
  int n_sink, key_a, key_b;
  __device__ __forceinline__ Kv4Stretch(const Kv4DecodeParams& p, const int* pre, int at, int left, int tile,
                                        int slice_off) {
    // the sequence whose tiles hold `at`: the last b with pre[b] * Hkv <= at
    int b = 0, hi = p.B - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (pre[mid] * p.Hkv <= at) b = mid; else hi = mid - 1;
    }
    const int count = pre[b + 1] - pre[b];
    const int off = at - pre[b] * p.Hkv;
    const int hkv = off / count, first = off - hkv * count;
    const Kv4Seq sq(p, p.seqlens[b]);
    n = min(count - first, left);
    pair = b * p.Hkv + hkv;
    len = sq.len;
    lo = sq.lo;
    n_sink = sq.n_sink - first;
    key_a = first * tile + slice_off;
    key_b = (sq.lo_tile - sq.n_sink + first) * tile + slice_off;
  }
};

template <int D, int G>
__global__ void __launch_bounds__(Kv4Cfg<D, G>::THREADS, Kv4Cfg<D, G>::CTAS)
fa_kv4_split_kernel(const __grid_constant__ Kv4DecodeParams p) {
  using C = Kv4Cfg<D, G>;
  constexpr int NG = C::NG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* mrg = reinterpret_cast<float*>(smem + C::OFF_MRG);
  float* m_s = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* l_s = m_s + C::NWARP * 8;
  int* pre = reinterpret_cast<int*>(smem + C::OFF_PRE);
  int* scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t ring_off = warp * C::NSTAGE * C::STAGE_BYTES;  // this warp's ring
  pdl_launch();  // fa_kv4_combine_kernel; its blocks need no shared memory and wait at their start
  // ---- prefix sum of the sequences' visible tiles, the same in every block
  {
    constexpr int PER = kKv4MaxSeqs / C::THREADS + 1;  // up to and with the total at index B
    const int i0 = threadIdx.x * PER;
    int cnt[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      cnt[i] = i0 + i < p.B ? Kv4Seq(p, p.seqlens[i0 + i]).count : 0;
      sum += cnt[i];
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += scan[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (i0 + i <= p.B) {
        pre[i0 + i] = base;
        if (blockIdx.x == 0) p.ws_prefix[i0 + i] = base;
      }
      base += cnt[i];
    }
  }
  __syncthreads();
  const int total = pre[p.B] * p.Hkv;  // at most 2^30, checked on the host
  const int n_cta = min(p.n_cta, total);
  if ((int)blockIdx.x >= n_cta) return;
  int at = (int)((long long)total * blockIdx.x / n_cta);
  int left = (int)((long long)total * (blockIdx.x + 1) / n_cta) - at;

  const int g = lane >> 2, t4 = lane & 3;
  const Kv4PairsF16 codes16;
  // Lane offsets into a stage; rows 8 or 16 further on have the same swizzle,
  // and the second pair of V's chunks is the first with chunk bit 1 flipped.
  const uint32_t off_k = C::OFF_K + (D == 128 ? kv4_swz<D>(lane & 7, lane >> 3)
                                              : kv4_swz<D>(((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1));
  const uint32_t off_v = C::OFF_V + kv4_swz<D>(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4);
  const uint32_t off_kz = C::OFF_KP + g * C::PB + 2 * NG + (NG == 4 ? 4 * (t4 & 1) : 0);
  const uint32_t off_ks = C::OFF_KP + 2 * t4 * C::PB;
  const uint32_t off_vz = C::OFF_VP + (((lane >> 4) << 3) + (lane & 7)) * C::PB;

  auto key_of = [&](const Kv4Stretch& sg, int j) { return (j < sg.n_sink ? sg.key_a : sg.key_b) + j * C::TILE; };
  auto needed = [&](const Kv4Stretch& sg, int ks) {
    return ks < sg.len && (ks + C::SLICE > sg.lo || ks < p.sinks);
  };
  // The warp copies its slice of tile j itself, 16 bytes a lane (8 for params at
  // d = 64), as one asynchronous group; a slice that is not needed, or past the
  // stretch, is an empty group, so that groups count tiles.
  constexpr int ROWS = 512 / C::CB;  // rows of a warp-wide copy of codes
  const uint32_t dst_c = sbase + ring_off + kv4_swz<D>(lane * 16 / C::CB, lane % (C::CB / 16));
  const uint32_t dst_p = sbase + ring_off + C::OFF_KP + lane * C::PB;
  auto load = [&](const Kv4Stretch& sg, int j) {
    const int ks = key_of(sg, j);
    if (j < sg.n && needed(sg, ks)) {
      const uint32_t so = (j % C::NSTAGE) * C::STAGE_BYTES;
      // slices of 32 rows are counted in 32 bits (checked on the host)
      const uint32_t slice = (uint32_t)(p.pair0 + sg.pair) * (uint32_t)(p.Tk_max / C::SLICE) + (uint32_t)(ks / C::SLICE);
      const uint8_t* kc = p.k_codes + (size_t)slice * (C::SLICE * C::CB) + lane * 16;
      const uint8_t* vc = p.v_codes + (size_t)slice * (C::SLICE * C::CB) + lane * 16;
#pragma unroll
      for (int i = 0; i < C::SLICE / ROWS; ++i) {
        cp_async<16>(dst_c + so + C::OFF_K + 512 * i, kc + 512 * i);
        cp_async<16>(dst_c + so + C::OFF_V + 512 * i, vc + 512 * i);
      }
      cp_async<C::PB>(dst_p + so, reinterpret_cast<const uint8_t*>(p.k_params) + (size_t)slice * (C::SLICE * C::PB) + lane * C::PB);
      cp_async<C::PB>(dst_p + so + (C::OFF_VP - C::OFF_KP),
                      reinterpret_cast<const uint8_t*>(p.v_params) + (size_t)slice * (C::SLICE * C::PB) + lane * C::PB);
    }
    cp_async_commit();
  };

  Kv4Stretch sg(p, pre, at, left, C::TILE, warp * C::SLICE);
#pragma unroll
  for (int j = 0; j < C::NSTAGE; ++j) load(sg, j);

  while (true) {
    at += sg.n;
    left -= sg.n;
    // Q as the row operand: row g, dims of group c in the order the codes have
    // (an operand's four registers are neighbours: rows 8..15, which no query
    // has, hold the next group's Q rather than zeros, so that every operand is
    // four registers that stay)
    uint32_t qa[NG][4];
    float qscale;            // what the row's products are multiplied by
    uint32_t za0, za1 = 0u;  // sum q: parts 0 and 1 in row g, part 2 in row g + 8
    {
      const __nv_bfloat16* qrow = p.q + ((size_t)sg.pair * G + (g < G ? g : 0)) * D;
      uint4 v[NG];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < NG; ++c) {
        v[c] = *reinterpret_cast<const uint4*>(qrow + 32 * c + 8 * t4);
        if (g >= G) v[c] = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = max_nan(amax, max_nan(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
      }
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^-e brings the row's largest value into [2^14, 2^15) (less below 2^-98);
      // a row with a NaN, an infinity or anything from 2^118 on, whose scores
      // would leave fp32, gives NaN
      const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -112);
      const bool fine = amax < 0x1p118f;
      const float down = fine ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
      qscale = fine ? __uint_as_float((uint32_t)(127 + e) << 23) * p.scale_log2 : NAN;
      float qs[NG];
#pragma unroll
      for (int c = 0; c < NG; ++c) {
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
        float q8 = 0.f;
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = make_float2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
          q8 += x[i].x + x[i].y;
        }
        qa[c][0] = pack_f16x2(x[0].x, x[2].x);  // dims 8t, 8t + 4
        qa[c][1] = pack_f16x2(x[0].y, x[2].y);
        qa[c][2] = pack_f16x2(x[1].x, x[3].x);
        qa[c][3] = pack_f16x2(x[1].y, x[3].y);
        q8 += __shfl_xor_sync(0xffffffffu, q8, 1);
        q8 += __shfl_xor_sync(0xffffffffu, q8, 2);
        qs[c] = q8;
      }
      // sum q of every group in three bf16 parts: columns (part, group) of the
      // row operand that meets the centres
      uint32_t part[3][NG / 2];
#pragma unroll
      for (int c = 0; c < NG; c += 2) {
        float x = qs[c], y = qs[c + 1];
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const uint32_t w = pack_bf16x2(x, y);
          part[n][c / 2] = w;
          x -= bf16_lo(w);
          y -= bf16_hi(w);
        }
      }
      if constexpr (NG == 4) {
        za0 = t4 == 0 ? part[0][0] : t4 == 1 ? part[0][1] : t4 == 2 ? part[1][0] : part[1][1];
        za1 = t4 == 0 ? part[2][0] : t4 == 1 ? part[2][1] : 0u;
      } else {
        za0 = t4 == 0 ? part[0][0] : t4 == 1 ? part[1][0] : t4 == 2 ? part[2][0] : 0u;
      }
    }

    float m_run = -INFINITY, l_part = 0.f;   // row g
    uint32_t fac[NG / 2];                    // what V's steps are scaled by, a pair of groups each
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) fac[w] = kKv4FactorMax;
    float oacc[NG][2][4];                    // dims 32c + 4g + 2kk (+1), queries 2t, 2t + 1
    float zacc[4] = {0.f, 0.f, 0.f, 0.f};    // sum of p z, by group
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[c][k][e] = 0.f;

    for (int j = 0; j < sg.n; ++j) {
      const int s = j % C::NSTAGE;
      const int ks = key_of(sg, j);
      if (!needed(sg, ks)) {
        load(sg, j + C::NSTAGE);
        continue;
      }
      cp_async_wait<C::NSTAGE - 1>();  // all groups but those of the tiles after this one
      __syncwarp();
      const bool whole = ks + C::SLICE <= sg.len && (ks >= sg.lo || ks + C::SLICE <= p.sinks);
      auto visible = [&](int key) { return key < sg.len && (key >= sg.lo || key < p.sinks); };
      if (!whole) {
        // A masked key's p is 0, but 0 times what an unwritten row's params
        // may hold (NaN, infinity) is not: zero them.
        if (!visible(ks + lane)) {
          uint32_t* row =
              reinterpret_cast<uint32_t*>(smem + ring_off + s * C::STAGE_BYTES + C::OFF_VP + lane * C::PB);
#pragma unroll
          for (int i = 0; i < C::PB / 4; ++i) row[i] = 0u;
        }
        __syncwarp();
      }
      const uint32_t st = sbase + ring_off + s * C::STAGE_BYTES;

      // ---- scores of row g against keys ks + 16 u + 8 nb + 2t (+1)
      float2 sc[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t kc[2][NG];
        if constexpr (D == 128) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
            ldsm_x4(st + off_k + (16 * u + 8 * nb) * C::CB, kc[nb][0], kc[nb][1], kc[nb][2], kc[nb][3]);
        } else {
          ldsm_x4(st + off_k + 16 * u * C::CB, kc[0][0], kc[0][1], kc[1][0], kc[1][1]);
        }
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          const uint32_t zw = lds32(st + off_kz + (16 * u + 8 * nb) * C::PB);
          uint32_t s0[NG / 2], s1[NG / 2];
          kv4_steps<NG>(st + off_ks + (16 * u + 8 * nb) * C::PB, s0);
          kv4_steps<NG>(st + off_ks + (16 * u + 8 * nb + 1) * C::PB, s1);
          float sz[4];
          mma_1688_z(sz, za0, za1, zw);
          float2 tot = NG == 4 ? __fadd2_rn(make_float2(sz[0], sz[1]), make_float2(sz[2], sz[3]))
                               : make_float2(sz[0], sz[1]);
#pragma unroll
          for (int c = 0; c < NG; c += 2) {
            // group c in the accumulator's rows 0..7, group c + 1 in the other's 8..15
            float x[4], y[4];
            const uint32_t w0 = kc[nb][c], w1 = kc[nb][c + 1];
            uint32_t b0, b1;
            codes16.pairs(w0, b0, b1);
            mma_f16_z(x, qa[c][0], qa[c + 1][0], qa[c][1], qa[c + 1][1], b0, b1);
            codes16.pairs(w1, b0, b1);
            mma_f16_z(y, qa[c][0], qa[c + 1][0], qa[c][1], qa[c + 1][1], b0, b1);
            codes16.pairs(w0 >> 8, b0, b1);
            mma_f16(x, qa[c][2], qa[c + 1][2], qa[c][3], qa[c + 1][3], b0, b1);
            codes16.pairs(w1 >> 8, b0, b1);
            mma_f16(y, qa[c][2], qa[c + 1][2], qa[c][3], qa[c + 1][3], b0, b1);
            tot = __ffma2_rn(make_float2(bf16_lo(s0[c / 2]), bf16_lo(s1[c / 2])), make_float2(x[0], x[1]), tot);
            tot = __ffma2_rn(make_float2(bf16_hi(s0[c / 2]), bf16_hi(s1[c / 2])), make_float2(y[2], y[3]), tot);
          }
          sc[u][nb] = __fmul2_rn(tot, make_float2(qscale, qscale));
        }
      }
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = ks + 8 * e + 2 * t4;
          if (!visible(key)) sc[e >> 1][e & 1].x = -INFINITY;
          if (!visible(key + 1)) sc[e >> 1][e & 1].y = -INFINITY;
        }
      }

      // ---- online softmax with a lazily moved reference, as elsewhere
      float mx = fmaxf(fmax3(sc[0][0].x, sc[0][0].y, sc[0][1].x), fmax3(sc[0][1].y, sc[1][0].x, sc[1][0].y));
      mx = fmax3(mx, sc[1][1].x, sc[1][1].y);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const bool move = mx > m_run + (C::RESCALE_THRESHOLD - kKv4RefAbove) || (m_run == -INFINITY && mx != -INFINITY);
      uint32_t ps[NG / 2];  // V's steps of key `lane`, scaled
      // the same address from what is in registers anyway: 288 us against 291 at d =
      // 128 (64 sequences of 1k to 32k keys); the other way round, 183 against 177, at 64
      const uint32_t at_sw = D == 128 ? dst_p + s * C::STAGE_BYTES + (C::OFF_VP - C::OFF_KP)
                                      : st + C::OFF_VP + lane * C::PB;
      kv4_steps<NG>(at_sw, ps);
      bool wide = false;
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) {
        ps[w] = bf16x2_mul(ps[w], fac[w]);
        wide |= bf16x2_any_gt(ps[w], kKv4ScaledMax);
      }
      if (__any_sync(0xffffffffu, move || wide)) {
        const float m_new = move ? mx + kKv4RefAbove : m_run;
        const float alpha = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new);
        m_run = m_new;
        l_part *= alpha;
        const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t4);      // row 2t
        const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * t4 + 4);  // row 2t + 1
        kv4_steps<NG>(at_sw, ps);
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) {
          uint32_t big = ps[w];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) big = bf16x2_max(big, __shfl_xor_sync(0xffffffffu, big, off));
          int now[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int old = (int)(fac[w] >> (h ? 23 : 7)) & 0xFF;
            now[h] = min(old, kv4_factor_exp(h ? big >> 16 : big & 0xFFFFu));
            const float f = __uint_as_float((uint32_t)max(127 + now[h] - old, 0) << 23);
            const float f0 = a0 * f, f1 = a1 * f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) oacc[2 * w + h][k][e] *= (e & 1) ? f1 : f0;
          }
          fac[w] = (uint32_t)now[0] << 7 | (uint32_t)now[1] << 23;
          ps[w] = bf16x2_mul(ps[w], fac[w]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) zacc[e] *= (e & 1) ? a1 : a0;
      }
      if constexpr (NG == 4)
        sts64(at_sw, ps[0], ps[1]);
      else
        sts32(at_sw, ps[0]);
      const float ref = m_run == -INFINITY ? 0.f : m_run;
      float2 pv[2][2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = sc[e >> 1][e & 1];
        pv[e >> 1][e & 1] = make_float2(ex2_approx(x.x - ref), ex2_approx(x.y - ref));
      }
      const float2 lsum = __fadd2_rn(__fadd2_rn(pv[0][0], pv[0][1]), __fadd2_rn(pv[1][0], pv[1][1]));
      l_part += lsum.x + lsum.y;

      // ---- O^T += V^T P^T
      __syncwarp();  // the scaled steps
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t vs = st + off_ks + (C::OFF_VP - C::OFF_KP) + 16 * u * C::PB;
        uint32_t sv[4][NG / 2];
#pragma unroll
        for (int e = 0; e < 4; ++e) kv4_steps<NG>(vs + (8 * (e >> 1) + (e & 1)) * C::PB, sv[e]);
        {
          uint32_t z0, z1, z2, z3;
          if constexpr (NG == 4) {
            // row g: the steps (0..3, not wanted) and the centres (4..7) of keys
            // 2t, 2t + 1; rows 8..15 the same again
            ldsm_x4_t(st + off_vz + 16 * u * C::PB, z0, z1, z2, z3);
          } else {
            const uint32_t a = vs + 4;  // the centres' words of keys 2t, 2t + 1 (+ 8)
            const uint32_t sel = g == 0 ? 0x5410u : 0x7632u;
            z0 = __byte_perm(lds32(a), lds32(a + C::PB), sel);
            z2 = __byte_perm(lds32(a + 8 * C::PB), lds32(a + 9 * C::PB), sel);
            z1 = z0;
            z3 = z2;
          }
          mma_16816(zacc, z0, z1, z2, z3, pack_bf16x2(pv[u][0].x, pv[u][0].y), pack_bf16x2(pv[u][1].x, pv[u][1].y));
        }
#pragma unroll
        for (int c2 = 0; c2 < NG; c2 += 2) {
          uint32_t vc[2][2];  // [group of the two][keys 0..7, 8..15]
          ldsm_x4_t(((st + off_v) ^ (16 * c2)) + 16 * u * C::CB, vc[0][0], vc[0][1], vc[1][0], vc[1][1]);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int c = c2 + cc;
            const float2 f0 = cc ? make_float2(bf16_hi(sv[0][c2 / 2]), bf16_hi(sv[1][c2 / 2]))
                                 : make_float2(bf16_lo(sv[0][c2 / 2]), bf16_lo(sv[1][c2 / 2]));
            const float2 f1 = cc ? make_float2(bf16_hi(sv[2][c2 / 2]), bf16_hi(sv[3][c2 / 2]))
                                 : make_float2(bf16_lo(sv[2][c2 / 2]), bf16_lo(sv[3][c2 / 2]));
            const float2 p0 = __fmul2_rn(pv[u][0], f0), p1 = __fmul2_rn(pv[u][1], f1);
            const uint32_t b0 = pack_f16x2(p0.x, p0.y), b1 = pack_f16x2(p1.x, p1.y);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t v0, v1, v2, v3;
              codes16.pairs(vc[cc][0] >> (8 * k), v0, v1);
              codes16.pairs(vc[cc][1] >> (8 * k), v2, v3);
              mma_f16(oacc[c][k], v0, v1, v2, v3, b0, b1);
            }
          }
        }
      }
      __syncwarp();  // the stage has been read
      load(sg, j + C::NSTAGE);
    }

    // the next stretch's first loads fly while this one's results are joined
    const size_t slot = (size_t)blockIdx.x + sg.pair;
    if (left > 0) {
      sg = Kv4Stretch(p, pre, at, left, C::TILE, warp * C::SLICE);
#pragma unroll
      for (int j = 0; j < C::NSTAGE; ++j) load(sg, j);
    }
    const bool more = left > 0;

    // ---- the four warps' results, joined
    float l_row = l_part + __shfl_xor_sync(0xffffffffu, l_part, 1);
    l_row += __shfl_xor_sync(0xffffffffu, l_row, 2);
    if (t4 == 0) {
      m_s[warp * 8 + g] = m_run;
      l_s[warp * 8 + g] = l_row;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // half of the dims at a time
#pragma unroll
      for (int c = h * (NG / 2); c < (h + 1) * (NG / 2); ++c) {
        const int zrow = NG == 4 ? 4 + c : c;
        const float add0 = __shfl_sync(0xffffffffu, zacc[0], 4 * zrow + t4);
        const float add1 = __shfl_sync(0xffffffffu, zacc[1], 4 * zrow + t4);
        const int at_d = 32 * c - h * (D / 2) + 4 * g;
        const float un = __uint_as_float((254u - ((fac[c / 2] >> (c & 1 ? 23 : 7)) & 0xFFu)) << 23);  // 1 / factor
        if (2 * t4 < G)
          *reinterpret_cast<float4*>(&mrg[(warp * G + 2 * t4) * (D / 2) + at_d]) =
              make_float4(fmaf(oacc[c][0][0], un, add0), fmaf(oacc[c][0][2], un, add0),
                          fmaf(oacc[c][1][0], un, add0), fmaf(oacc[c][1][2], un, add0));
        if (2 * t4 + 1 < G)
          *reinterpret_cast<float4*>(&mrg[(warp * G + 2 * t4 + 1) * (D / 2) + at_d]) =
              make_float4(fmaf(oacc[c][0][1], un, add1), fmaf(oacc[c][0][3], un, add1),
                          fmaf(oacc[c][1][1], un, add1), fmaf(oacc[c][1][3], un, add1));
      }
      __syncthreads();
      for (int idx = threadIdx.x; idx < G * (D / 2); idx += C::THREADS) {
        const int gg = idx / (D / 2), dd = idx % (D / 2);
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < C::NWARP; ++w) M = fmaxf(M, m_s[w * 8 + gg]);
#pragma unroll
        for (int w = 0; w < C::NWARP; ++w) {
          const float f = m_s[w * 8 + gg] == -INFINITY ? 0.f : ex2_approx(m_s[w * 8 + gg] - M);
          L = fmaf(f, l_s[w * 8 + gg], L);
          O = fmaf(f, mrg[(w * G + gg) * (D / 2) + dd], O);
        }
        p.ws_o[(slot * G + gg) * D + h * (D / 2) + dd] = O;
        if (h == 0 && dd == 0) *reinterpret_cast<float2*>(&p.ws_ml[(slot * G + gg) * 2]) = make_float2(M, L);
      }
      __syncthreads();
    }
    if (!more) break;
  }
  cp_async_wait<0>();
}

// One warp per (sequence, query head): the partial results of its stretch of
// the list, joined; eight of them in flight at a time.
template <int D>
__global__ void __launch_bounds__(128) fa_kv4_combine_kernel(const __grid_constant__ Kv4DecodeParams p) {
  constexpr int E = D / 32, U = 8;
  const int row = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (row >= p.B * p.Hq) return;
  pdl_wait();
  const int G = p.Hq / p.Hkv;
  const int b = row / p.Hq, hkv = row % p.Hq / G, gq = row % G;
  const int before = p.ws_prefix[b], count = p.ws_prefix[b + 1] - before;
  const int total = p.ws_prefix[p.B] * p.Hkv;
  const int n_cta = min(p.n_cta, total);
  float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (count > 0) {
    const long long first = (long long)before * p.Hkv + (long long)hkv * count;
    // block i of tile t: the last with total * i / n <= t
    const int c0 = (int)(((first + 1) * n_cta - 1) / total), c1 = (int)(((first + count) * n_cta - 1) / total);
    const size_t at0 = ((size_t)b * p.Hkv + hkv + c0) * G + gq;  // partial i at at0 + i * G
    const int n = c1 - c0 + 1;
    float m_own = -INFINITY, l_own = 0.f;  // partial `lane`
    if (lane < n) {
      const float2 ml = *reinterpret_cast<const float2*>(&p.ws_ml[(at0 + (size_t)lane * G) * 2]);
      m_own = ml.x;
      l_own = ml.y;
    }
    M = m_own;
    for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, p.ws_ml[(at0 + (size_t)i * G) * 2]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int i0 = 0; i0 < n; i0 += U) {
      float f[U], v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + u, n - 1);
        const float* src = p.ws_o + (at0 + (size_t)i * G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = *reinterpret_cast<const float2*>(src + e);
          v[u][e] = x.x;
          v[u][e + 1] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        float m = -INFINITY, l = 0.f;
        if (i0 + U <= 32) {
          m = __shfl_sync(0xffffffffu, m_own, i & 31);
          l = __shfl_sync(0xffffffffu, l_own, i & 31);
        } else if (i < n) {
          const float2 ml = *reinterpret_cast<const float2*>(&p.ws_ml[(at0 + (size_t)i * G) * 2]);
          m = ml.x;
          l = ml.y;
        }
        f[u] = i >= n || m == -INFINITY ? 0.f : ex2_approx(m - M);
        if (i < n) L = fmaf(f[u], l, L);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < n) {
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(f[u], v[u][e], o[e]);
        }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __nv_bfloat16* dst = p.o + (size_t)row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (lane == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace fa
