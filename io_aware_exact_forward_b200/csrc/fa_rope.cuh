// fa_rope.cuh -- rotary positions on q and k ahead of the attention kernels,
// and their transpose for the gradients.
//
// Pair i of a head's first R dims is turned by the angle theta = pos * f_i and
// scaled by a:
//   (x, y) -> a (x cos theta - y sin theta, x sin theta + y cos theta),
// with the pair at dims (2i, 2i + 1) or (i, i + R / 2); dims R .. d - 1 are
// copied.  The transpose (the gradient) turns by -theta.
//
// Angles.  pos * f_i reaches 10^5 to 10^6 radians, of which 32 bits leave
// nothing below 10^-2, so the turn count pos * f_i / 2 pi is formed in 64
// bits, its whole part dropped there, and only the remaining fraction of a
// turn goes to sincospif.  The angles of a token are shared by all its heads:
// a block forms them once, in shared memory.
//
// Bound by HBM: 4 bytes per element and a few operations.  32k tokens of 40 heads
// of 128 out of a packed projection take 117 us, 5.7 TB/s; 64k tokens of 32 heads
// of 64, half of each turned, 82 us, 6.5 TB/s.  A single step's 64 tokens take 5
// us alone, 3 in a row of such calls in a graph: the latency of a launch, the angles
// and one round trip to memory.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

struct RopeTensor {
  const __nv_bfloat16* x;  // [B][T][H][d], last dim contiguous, other strides in elements
  __nv_bfloat16* y;
  long long xb, xt, xh, yb, yt, yh;
};

struct RopeParams {
  RopeTensor q, k;
  const int* positions;   // [B][T], or null: position t
  const double* freqs;    // [R / 2], radians per position
  long long n_tokens;     // B * T
  int T, Hq, heads;       // heads = Hq + Hkv
  int rot;                // R, a multiple of 16
  float amplitude, sign;  // sign = -1: the transpose
};

// One unit is 16 elements of one head: 8 pairs (two 16-byte accesses each
// way), or 16 copied dims.
template <int D, bool INTER>
__global__ void __launch_bounds__(256) fa_rope_kernel(const __grid_constant__ RopeParams p, int tokens_per_block) {
  extern __shared__ float2 rope_cs[];  // [tokens_per_block][R / 2]
  const int half = p.rot >> 1;
  const long long tok0 = (long long)blockIdx.x * tokens_per_block;
  const int n_tok = (int)min((long long)tokens_per_block, p.n_tokens - tok0);
  for (int i = threadIdx.x; i < n_tok * half; i += blockDim.x) {
    const int tl = i / half, f = i - tl * half;
    const long long tok = tok0 + tl;
    const int pos = p.positions ? p.positions[tok] : (int)(tok % p.T);
    const double turns = (double)pos * (p.freqs[f] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    rope_cs[i] = make_float2(c * p.amplitude, s * p.amplitude * p.sign);
  }
  __syncthreads();

  constexpr int UNITS = D / 16;
  const int per_tok = p.heads * UNITS;
  for (int i = threadIdx.x; i < n_tok * per_tok; i += blockDim.x) {
    const int tl = i / per_tok, r = i - tl * per_tok;
    int h = r / UNITS;
    const int u = r % UNITS;
    const long long tok = tok0 + tl;
    const long long b = tok / p.T, t = tok - b * p.T;
    const bool is_k = h >= p.Hq;
    const RopeTensor& a = is_k ? p.k : p.q;
    if (is_k) h -= p.Hq;
    const __nv_bfloat16* x = a.x + b * a.xb + t * a.xt + h * a.xh;
    __nv_bfloat16* y = a.y + b * a.yb + t * a.yt + h * a.yh;
    const bool turn = u * 16 < p.rot;
    const int o0 = (turn && !INTER) ? u * 8 : u * 16;
    const int o1 = (turn && !INTER) ? half + u * 8 : u * 16 + 8;
    uint4 v0 = *reinterpret_cast<const uint4*>(x + o0);
    uint4 v1 = *reinterpret_cast<const uint4*>(x + o1);
    if (turn) {
      uint32_t* w0 = reinterpret_cast<uint32_t*>(&v0);
      uint32_t* w1 = reinterpret_cast<uint32_t*>(&v1);
      const float2* cs = rope_cs + tl * half + u * 8;
      if constexpr (INTER) {
        // word j of the 16 elements is pair j
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t& w = j < 4 ? w0[j] : w1[j - 4];
          const float2 e = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
          const float2 c = cs[j];
          w = pack_bf16x2(e.x * c.x - e.y * c.y, e.x * c.y + e.y * c.x);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w0[j]));
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w1[j]));
          const float2 c0 = cs[2 * j], c1 = cs[2 * j + 1];
          w0[j] = pack_bf16x2(e.x * c0.x - f.x * c0.y, e.y * c1.x - f.y * c1.y);
          w1[j] = pack_bf16x2(e.x * c0.y + f.x * c0.x, e.y * c1.y + f.y * c1.x);
        }
      }
    }
    *reinterpret_cast<uint4*>(y + o0) = v0;
    *reinterpret_cast<uint4*>(y + o1) = v1;
  }
}

}  // namespace fa
