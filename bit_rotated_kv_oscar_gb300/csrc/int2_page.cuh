// Reading INT2 page blocks as tensor-core operands: code extraction and the
// masking of tokens outside a range, shared by the attention kernels.
//
// A 2-bit code c in the low mantissa bits of an fp16 lane is the subnormal
// c * 2^-24, an exact tensor-core operand; slot i of a code word sits at bits 2i
// of each half and reads as c * slot_factor(i) * 2^-24 after one AND (slots 5..7
// after a 10-bit shift). The block layout is the one in include/oscar.h.
#pragma once

#include "oscar_internal.cuh"

namespace oscar {

// factor of a code read from slot i
__host__ __device__ constexpr float slot_factor(int i) {
  return i <= 4 ? (float)(1 << (2 * i)) : (float)(1 << (2 * (i - 5)));
}

// w: a code word, wh = w >> 10 (computed once per word, shared by slots 5..7)
template <int I>
__device__ __forceinline__ uint32_t slot_bits(uint32_t w, uint32_t wh) {
  if constexpr (I <= 4) {
    return w & (0x00030003u << (2 * I));
  } else {
    return wh & (0x00030003u << (2 * (I - 5)));
  }
}
__device__ __forceinline__ uint4 shr10(uint4 w) { return make_uint4(w.x >> 10, w.y >> 10, w.z >> 10, w.w >> 10); }

// bits t of the tokens t in [0, 16) of a page at position pos that lie in [lo, hi)
__device__ __forceinline__ uint32_t page_token_bits(bool ok, int pos, int lo, int hi) {
  const int a = max(lo - pos, 0), e = min(hi - pos, kPage);
  return (ok && e > a) ? (((1u << (e - a)) - 1u) << a) : 0u;
}

// zero the value scales and zeros of the tokens of two staged pages whose bit in
// `valid` is clear (bit t: page A token t, bit 16 + t: page B token t); lane:
// page lane / 16, 16-byte chunk c = 4 g + bb of the value metadata, whose 32-bit
// word w holds tokens 8 (w % 2) + 2 bb and + 1 (scales for w < 2, zeros after)
template <int NG>
__device__ __forceinline__ void zero_masked_value_meta(uint8_t* sbA, uint8_t* sbB, uint32_t valid, int lane) {
  const int c = lane & 15;
  if (c >= 4 * NG) return;  // NG groups: 4 NG chunks
  const uint32_t vpage = (lane >> 4) ? (valid >> 16) : (valid & 0xffffu);
  uint4* chunk = reinterpret_cast<uint4*>(((lane >> 4) ? sbB : sbA) + vscale_off(NG, 0, 0) + 16 * c);
  uint32_t keep[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int tw = 8 * (w & 1) + 2 * (c & 3);
    keep[w] = (((vpage >> tw) & 1u) ? 0x0000ffffu : 0u) | (((vpage >> (tw + 1)) & 1u) ? 0xffff0000u : 0u);
  }
  uint4 x = *chunk;
  x.x &= keep[0];
  x.y &= keep[1];
  x.z &= keep[2];
  x.w &= keep[3];
  *chunk = x;
}

}  // namespace oscar
