// q / k / v of a layer's fused projection: split, root-mean-square norm of every
// query and key head, position rotation, in one pass.
//
// For a head x of 128 channels with weight w, y = x w / sqrt(mean(x^2) + eps), then
// the first `rotary` channels are turned in pairs (a, c) by the angle
// pos * inv_freq: (a cos - c sin, c cos + a sin). Pairs are (i, i + rotary / 2), or
// neighbours (2 i, 2 i + 1) with `interleaved`. Everything between the bf16 input
// and the bf16 output is fp32, with one rounding at the end.
//
// Angles: a float32 angle of position 10^5 is off by 4e-3, so the frequency is
// kept as a 64-bit fraction of a turn and multiplied by the position in integer
// arithmetic: the product modulo 2^64 IS the angle modulo one turn, exact to
// pos * 2^-65 turns, with no range reduction left to do.
//
// Bound: HBM (each element read and written once).
#include "oscar_internal.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kTokensPerCta = 4;

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// CTA: `tpc` tokens; half-warp per head, 8 channels per lane. The launch uses no
// early trigger: what follows may read q, k and v as soon as it starts.
__global__ void __launch_bounds__(kThreads) oscar_qkv_norm_rope_kernel(RopeParams p, int tpc) {
  __shared__ float2 cs[kTokensPerCta][kMaxPairs];
  const int tid = threadIdx.x, sub = tid & 15, hw = tid >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * tpc;
  const int nt = (int)min((int64_t)tpc, p.tokens - t0);
  const int half = p.rotary / 2, heads = p.num_q_heads + 2 * p.num_kv_heads;
  pdl_wait();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int t = i / half, c = i - t * half;
    const unsigned long long turn = (unsigned long long)(long long)p.pos[t0 + t] * p.turns[c];
    float s, co;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &co);   // 2^-31: half turns
    cs[t][c] = make_float2(co, s);
  }
  __syncthreads();
  float w[2][8];
  if (p.q_weight) {
    unpack8(*reinterpret_cast<const uint4*>(p.q_weight + 8 * sub), w[0]);
    unpack8(*reinterpret_cast<const uint4*>(p.k_weight + 8 * sub), w[1]);
  }
  // half-split pairs: channels below `half` pair with lane + half / 8, the others back
  const int c0 = 8 * sub;
  const bool turned = c0 < p.rotary, low = c0 < half;
  const int partner = p.interleaved || !turned ? sub : (low ? sub + half / 8 : sub - half / 8);
  const int lane_partner = (tid & 16) | partner;
  for (int i = hw; i < nt * heads; i += kThreads / 16) {
    const int t = i / heads, hd = i - t * heads;
    const int64_t tok = t0 + t;
    const uint4 in = *reinterpret_cast<const uint4*>(p.qkv + tok * p.row_stride + (int64_t)hd * kHeadDim + c0);
    if (hd >= p.num_q_heads + p.num_kv_heads) {
      const int64_t at = tok * p.num_kv_heads + (hd - p.num_q_heads - p.num_kv_heads);
      *reinterpret_cast<uint4*>(p.v + at * kHeadDim + c0) = in;
      continue;
    }
    const bool isk = hd >= p.num_q_heads;
    const uint32_t mask = 0xffffu << (tid & 16);   // this half-warp
    float x[8];
    unpack8(in, x);
    if (p.q_weight) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float r = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (isk ? w[1][e] : w[0][e]);
    }
    float y[8];
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = turned ? cs[t][4 * sub + e] : make_float2(1.f, 0.f);
        y[2 * e] = x[2 * e] * a.x - x[2 * e + 1] * a.y;
        y[2 * e + 1] = x[2 * e + 1] * a.x + x[2 * e] * a.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl_sync(mask, x[e], lane_partner);
        const float2 a = turned ? cs[t][(low ? c0 : c0 - half) + e] : make_float2(1.f, 0.f);
        y[e] = turned ? fmaf(x[e], a.x, low ? -other * a.y : other * a.y) : x[e];
      }
    }
    const uint4 out = pack8(y);
    if (isk)
      *reinterpret_cast<uint4*>(p.k + (tok * p.num_kv_heads + (hd - p.num_q_heads)) * kHeadDim + c0) = out;
    else
      *reinterpret_cast<uint4*>(p.q + (tok * p.num_q_heads + hd) * kHeadDim + c0) = out;
  }
}

}  // namespace

cudaError_t launch_qkv_norm_rope(const RopeParams& p, cudaStream_t s) {
  const int tpc = p.tokens >= 4096 ? kTokensPerCta : 1;
  const int64_t ctas = (p.tokens + tpc - 1) / tpc;
  const cudaError_t e = launch_pdl(oscar_qkv_norm_rope_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, s, p, tpc);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
