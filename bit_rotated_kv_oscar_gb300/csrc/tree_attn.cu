// Attention of a tree of drafted tokens over the OSCAR INT2 cache.
//
// A speculative-decoding step verifies T drafted tokens of a request at once.
// They form a tree: node 0 is the last token sampled (its key and value are not
// cached yet), every other node hangs on an earlier one. Node i attends over all
// L cached positions and over its own ancestors and itself:
//   o_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(q_i k_t * softmax_scale),
//   t over the cache and over {j : j = i or j an ancestor of i}.
// The cached part is the mixed-precision read path of the decode attention
// ("OSCAR: Offline Spectral Covariance-Aware Rotation ..." (gist.science, it),
// Riepilogo Tecnico 2.2 B; "Juntos, AI Open-Sources OSCAR ..." (7minutos.es), "El
// sistema de servicio"): BF16 sink and ring in the raw basis, INT2 history in the
// rotated basis against q R_K, the value sums un-rotated once by R_V^T. The tree
// itself is this library's addition: the pages describe one token per step.
//
// The T g query rows of one KV head (g query heads share it) are columns of one
// problem over the same keys, so a page is read once for a tile of them:
//   1. oscar_tree_rotate_kernel  q~ = q R_K * scale * log2(e) of a tile of rows as
//      mma operand fragments (fp16, one power-of-two scale per tile).
//   2. oscar_tree_attn_kernel    grid (row tiles x (window chunks + splits), Hkv, B):
//      the INT2 CTAs stream a slice of the pages, the others attend over 128 tokens
//      of sink, ring and tree; one partial row (sum, maximum, denominator) each.
//   3. oscar_tree_merge_kernel   log-sum-exp merge, R_V^T, normalisation, bf16.
#include "int2_page.cuh"
#include "tree_attn.cuh"
#include "warp_mma.cuh"

namespace oscar {
namespace {

using namespace wm;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;                      // pages in flight per warp
constexpr int kRow = kHeadDim + 8;              // 16-bit elements per staged row (272 bytes: no bank conflicts)
constexpr int kPartRow = kHeadDim + 8;          // floats per row of a warp's partial in shared memory
constexpr float kLazyLog2 = 8.f;                // the running maximum moves only past this (see decode_attn.cu)

// query record of a tile of 32 rows: [2 row blocks][8 slots][32 lanes] uint4 of
// q~ fragments, [2][32] uint2 of group-sum fragments, the score unit
constexpr int kRecFrag = 2 * 8 * 32 * 4;
constexpr int kRecSums = kRecFrag;
constexpr int kRecUnit = kRecSums + 2 * 32 * 2;

// --------------------------------------------------------------------------
// 1. query rotation: q (bf16, exact) times R_K = hi + lo (bf16 images), fp32
//    sums, so q~ carries about 17 bits before its one rounding to fp16
// --------------------------------------------------------------------------
constexpr int kRotThreads = 128;
constexpr int kImage = kHeadDim * kHeadDim * 2;   // bytes of one bf16 image
constexpr int kRotSmem = 2 * kImage + 32 * kRow * 2;

// WIDE: the record is the wide kernel's image (tree_attn.cuh)
template <bool WIDE>
__global__ void __launch_bounds__(kRotThreads) oscar_tree_rotate_kernel(TreeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int g = p.gqa;
  const uint32_t simg = (uint32_t)__cvta_generic_to_shared(smem);
  __nv_bfloat16* qrows = reinterpret_cast<__nv_bfloat16*>(smem + 2 * kImage);   // [32][kRow]
  const uint32_t sq = simg + 2 * kImage;
  __shared__ float wmax[4];
  __shared__ float gsum[32][4];
  // constant data before the wait
  const uint8_t* img = p.images + (size_t)h * 4 * kImage;                       // R_K hi, R_K lo
  for (int i = tid; i < 2 * kImage / 16; i += kRotThreads) cp_async16(simg + 16 * i, img + 16 * i);
  cp_commit();
  pdl_wait();   // draft lengths; the record is read by an earlier call's attention
  pdl_trigger();
  const int len = min(max(p.draft_len ? p.draft_len[b] : p.nodes, 0), p.nodes);
  const int ncol = len * g, col0 = 32 * tile;
  if (col0 >= ncol) {
    cp_wait<0>();
    return;
  }
  for (int i = tid; i < 32 * 16; i += kRotThreads) {
    const int r = i >> 4, u = i & 15, col = col0 + r, node = col / g, m = col - node * g;
    const bool in = col < ncol;
    const size_t off = in ? (((size_t)b * p.nodes + node) * p.num_q_heads + h * g + m) * kHeadDim + 8 * u : 0;
    cp_async16(sq + (r * kRow + 8 * u) * 2, p.q + off, in ? 16u : 0u);
  }
  cp_commit();
  cp_wait<0>();
  __syncthreads();
  float acc[2][4][4] = {};
  // warp w: channels 32 w .. 32 w + 31 (4 column tiles), both row blocks
  for (int kk = 0; kk < 8; ++kk) {
    uint4 a[2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
      a[mt] = ldsm_x4(sq + ((16 * mt + (lane & 15)) * kRow + 16 * kk + 8 * (lane >> 4)) * 2);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int n = 32 * warp + 8 * nt + gid;
      const uint8_t* base = smem + (kk >> 2) * 16384 + n * 128 + 4 * tig;
      const int c0 = (((kk & 3) * 2) ^ (n & 7)) * 16, c1 = (((kk & 3) * 2 + 1) ^ (n & 7)) * 16;
#pragma unroll
      for (int part = 1; part >= 0; --part) {   // the small terms first
        const uint32_t b0 = *reinterpret_cast<const uint32_t*>(base + part * kImage + c0);
        const uint32_t b1 = *reinterpret_cast<const uint32_t*>(base + part * kImage + c1);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) mma16816_bf16(acc[mt][nt], a[mt], b0, b1);
      }
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[mt][nt][i] *= p.scale_log2;
        amax = fmaxf(amax, fabsf(acc[mt][nt][i]));
      }
  amax = warp_maxf(amax);
  if (lane == 0) wmax[warp] = amax;
  __syncthreads();   // also: every warp is done with the staged q rows
  amax = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
  // operand scale 2^k keeps the largest entry in [2^13, 2^14); one scale per tile
  // is enough: an entry 2^-19 of the largest still rounds at full fp16 precision,
  // smaller ones lose at most 2^-31 of the largest in absolute terms
  int e = 0;
  if (amax > 0.f && amax < INFINITY) frexpf(amax, &e);
  const int k = amax > 0.f ? min(14 - e, 100) : 0;
  const float s2k = ldexpf(1.f, k), gscale = ldexpf(1.f, k - 24);
  __half* hs = reinterpret_cast<__half*>(qrows);   // [32][kRow]
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float x0 = acc[mt][nt][2 * half], x1 = acc[mt][nt][2 * half + 1];
        sum += x0 + x1;
        const int c = 32 * warp + 8 * nt + 2 * tig;
        const float f = s2k / slot_factor(c >> 4);   // a power of two: exact
        *reinterpret_cast<uint32_t*>(hs + (16 * mt + 8 * half + gid) * kRow + c) = f2_to_h2_bits(x0 * f, x1 * f);
      }
      sum = quad_sum(sum);
      if (tig == 0) gsum[16 * mt + 8 * half + gid][warp] = sum * (WIDE ? s2k * 0x1p-9f : gscale);   // 2^-9: far below fp16's end
    }
  __syncthreads();
  if constexpr (WIDE) {
    uint8_t* img = reinterpret_cast<uint8_t*>(p.qrec) +
                   (((size_t)b * p.num_kv_heads + h) * p.images128 + (tile >> 2)) * kWideRecBytes;
    const int r0 = 32 * (tile & 3);
    for (int i = tid; i < 32 * 16; i += kRotThreads) {
      const int r = i >> 4, u = i & 15;
      *reinterpret_cast<uint4*>(img + sw128_off(r0 + r, u)) = *reinterpret_cast<const uint4*>(hs + r * kRow + 8 * u);
    }
    if (tid < 32) {   // hi and lo parts of the group sums, then zeros
      const int ng = p.ngroups;
      uint32_t w[8] = {};
      for (int gq = 0; gq < ng; ++gq) {
        const float v = ng == kGroups ? gsum[tid][gq] : gsum[tid][2 * gq] + gsum[tid][2 * gq + 1];
        const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
        w[gq >> 1] |= (uint32_t)__half_as_ushort(hi) << (16 * (gq & 1));
        w[(ng + gq) >> 1] |= (uint32_t)__half_as_ushort(lo) << (16 * (gq & 1));
      }
      uint8_t* x = img + kWideImage;
      *reinterpret_cast<uint4*>(x + extra_off(r0 + tid, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(x + extra_off(r0 + tid, 1)) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (tid == 0) reinterpret_cast<float*>(img + kWideUnits)[tile & 3] = ldexpf(1.f, -k);
    return;
  }
  uint32_t* rec = p.qrec + (((size_t)b * p.num_kv_heads + h) * p.row_tiles + tile) * kTreeRecWords;
  for (int i = tid; i < 2 * 8 * 32; i += kRotThreads) {
    const int l = i & 31, kb = (i >> 5) & 7, mt = i >> 8;
    const __half* src = hs + (16 * mt + (l >> 2)) * kRow + 16 * kb + 2 * (l & 3);
    uint4 f;
    f.x = *reinterpret_cast<const uint32_t*>(src);
    f.y = *reinterpret_cast<const uint32_t*>(src + 8 * kRow);
    f.z = *reinterpret_cast<const uint32_t*>(src + 8);
    f.w = *reinterpret_cast<const uint32_t*>(src + 8 * kRow + 8);
    reinterpret_cast<uint4*>(rec)[i] = f;
  }
  // zero-point operand (k = 8): columns 0 .. NG-1 the fp16 hi parts of the group
  // sums of q~, NG .. 2 NG - 1 the lo parts
  if (tid < 64) {
    const int l = tid & 31, mt = tid >> 5, t = l & 3, ng = p.ngroups;
    uint32_t w[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float* s = gsum[16 * mt + 8 * half + (l >> 2)];
      uint32_t x = 0u;
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const int kx = 2 * t + e2;
        if (kx < 2 * ng) {
          const int gq = kx % ng;
          const float v = ng == kGroups ? s[gq] : s[2 * gq] + s[2 * gq + 1];
          const __half hi = __float2half_rn(v);
          const __half part = kx < ng ? hi : __float2half_rn(v - __half2float(hi));
          x |= (uint32_t)__half_as_ushort(part) << (16 * e2);
        }
      }
      w[half] = x;
    }
    *reinterpret_cast<uint2*>(rec + kRecSums + 2 * tid) = make_uint2(w[0], w[1]);
  }
  if (tid == 0) rec[kRecUnit] = __float_as_uint(ldexpf(1.f, 24 - k));
}

// --------------------------------------------------------------------------
// 2. attention over a slice of the keys for MT x 16 query rows
// --------------------------------------------------------------------------
// The query rows are the row operand, tokens the columns of the score product and
// the reduction of the value product, so the probabilities of the score
// accumulators are the value product's row operand as they stand. A page's K words
// (token 8 th + gid, channels 16 i + 8 x + 2 tig, + 1 in slot i) are the column
// fragments b_x of token tile th; its V words (tokens 8 tt + 2 tig, + 1, channel
// 16 i + 8 x + gid) the fragments b_tt of channel tile (i, x).
template <int MT>
struct State {
  float o[MT][8][2][4];   // value sums: channels 16 i + 8 x + 2 tig, + 1 of rows gid (0, 1) and gid + 8 (2, 3)
  float oz[MT][4];        // columns 0 .. NG-1: value zero-point sums of the groups, column 4: the denominator
  float m[MT][2];         // running (lazy) maxima of rows gid, gid + 8, in score units
};

// scores of one page in score units: u[mt][th] tokens 8 th + 2 tig, + 1 of rows gid, gid + 8
template <int NG, int MT>
__device__ __forceinline__ void page_scores(const uint8_t* sb, const uint4* qs, const uint2 (&zs)[MT], int lane,
                                            float (&u)[MT][2][4]) {
  const int gid = lane >> 2, tig = lane & 3;
  const uint4 kw = *reinterpret_cast<const uint4*>(sb + lane * 16);
  const uint4 kh = shr10(kw);
  {
    const int zo = kzero_off(NG, gid, NG == kGroups ? 2 * (tig & 1) : 0);
    constexpr int step = kzero_off(NG, 8, 0) - kzero_off(NG, 0, 0);
    const bool on = NG == kGroups || tig < 2;
    const uint32_t z0 = on ? *reinterpret_cast<const uint32_t*>(sb + zo) : 0u;
    const uint32_t z1 = on ? *reinterpret_cast<const uint32_t*>(sb + zo + step) : 0u;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      mma1688_z(u[mt][0], zs[mt], z0);
      mma1688_z(u[mt][1], zs[mt], z1);
    }
  }
  const uint8_t* s0 = sb + kscale_off(NG, 2 * tig, 0);   // tokens 2 tig (+ 8): next, tokens 2 tig + 1 (+ 8)
#pragma unroll
  for (int gq = 0; gq < NG; ++gq) {
    float c[MT][2][4];
#define OSCAR_QK(I, FIRST)                                                             \
  {                                                                                    \
    const uint32_t x0 = slot_bits<I>(kw.x, kh.x), x1 = slot_bits<I>(kw.y, kh.y);       \
    const uint32_t y0 = slot_bits<I>(kw.z, kh.z), y1 = slot_bits<I>(kw.w, kh.w);       \
    _Pragma("unroll") for (int mt = 0; mt < MT; ++mt) {                                \
      const uint4 a = qs[(mt * 8 + (I)) * 32 + lane];                                  \
      if (FIRST) {                                                                     \
        mma16816_z(c[mt][0], a, x0, x1);                                               \
        mma16816_z(c[mt][1], a, y0, y1);                                               \
      } else {                                                                         \
        mma16816(c[mt][0], a, x0, x1);                                                 \
        mma16816(c[mt][1], a, y0, y1);                                                 \
      }                                                                                \
    }                                                                                  \
  }
    if constexpr (NG == kGroups) {
      if (gq == 0) { OSCAR_QK(0, true) OSCAR_QK(1, false) }
      if (gq == 1) { OSCAR_QK(2, true) OSCAR_QK(3, false) }
      if (gq == 2) { OSCAR_QK(4, true) OSCAR_QK(5, false) }
      if (gq == 3) { OSCAR_QK(6, true) OSCAR_QK(7, false) }
    } else {
      if (gq == 0) { OSCAR_QK(0, true) OSCAR_QK(1, false) OSCAR_QK(2, false) OSCAR_QK(3, false) }
      if (gq == 1) { OSCAR_QK(4, true) OSCAR_QK(5, false) OSCAR_QK(6, false) OSCAR_QK(7, false) }
    }
#undef OSCAR_QK
    const float2 se = h2_bits_to_f2(*reinterpret_cast<const uint32_t*>(s0 + 4 * gq));            // 2 tig, 2 tig + 8
    const float2 so = h2_bits_to_f2(*reinterpret_cast<const uint32_t*>(s0 + 4 * NG + 4 * gq));   // 2 tig + 1, + 9
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      u[mt][0][0] = fmaf(se.x, c[mt][0][0], u[mt][0][0]);
      u[mt][0][1] = fmaf(so.x, c[mt][0][1], u[mt][0][1]);
      u[mt][0][2] = fmaf(se.x, c[mt][0][2], u[mt][0][2]);
      u[mt][0][3] = fmaf(so.x, c[mt][0][3], u[mt][0][3]);
      u[mt][1][0] = fmaf(se.y, c[mt][1][0], u[mt][1][0]);
      u[mt][1][1] = fmaf(so.y, c[mt][1][1], u[mt][1][1]);
      u[mt][1][2] = fmaf(se.y, c[mt][1][2], u[mt][1][2]);
      u[mt][1][3] = fmaf(so.y, c[mt][1][3], u[mt][1][3]);
    }
  }
}

// running maxima and rescaling for NP pages' scores; us: score units per log2 unit
template <int MT, int NP>
__device__ __forceinline__ void update_max(State<MT>& st, const float (&u)[NP][MT][2][4], float us, float tau) {
  float mx[MT][2];
  bool over = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x = -INFINITY;
#pragma unroll
      for (int n = 0; n < NP; ++n)
        x = fmaxf(x, fmaxf(fmaxf(u[n][mt][0][2 * r], u[n][mt][0][2 * r + 1]),
                           fmaxf(u[n][mt][1][2 * r], u[n][mt][1][2 * r + 1])));
      mx[mt][r] = x;
      over |= x > st.m[mt][r] + tau;
    }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float x = quad_max(mx[mt][r]);
        const bool bump = x > st.m[mt][r] + tau;
        const float a = bump ? ex2((st.m[mt][r] - x) * us) : 1.f;
        st.m[mt][r] = bump ? x : st.m[mt][r];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int xh = 0; xh < 2; ++xh) {
            st.o[mt][i][xh][2 * r] *= a;
            st.o[mt][i][xh][2 * r + 1] *= a;
          }
        st.oz[mt][2 * r] *= a;
        st.oz[mt][2 * r + 1] *= a;
      }
  }
}

// o += P V of one page; P: fp16 probabilities (times pscale) as row fragments
template <int NG, int MT>
__device__ __forceinline__ void page_values(const uint8_t* sb, int lane, const uint4 (&P)[MT], State<MT>& st) {
  const int gid = lane >> 2, tig = lane & 3;
  const uint4 vw = *reinterpret_cast<const uint4*>(sb + 512 + lane * 16);
  const uint4 vh = shr10(vw);
  constexpr int vbase = vscale_off(NG, 0, 0);
#pragma unroll
  for (int gq = 0; gq < NG; ++gq) {
    // scales of tokens (2 tig, 2 tig + 1) and (2 tig + 8, 2 tig + 9)
    const uint2 mv = *reinterpret_cast<const uint2*>(sb + vbase + 16 * (4 * gq + tig));
    uint4 a[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      a[mt] = make_uint4(hmul2_bits(P[mt].x, mv.x), hmul2_bits(P[mt].y, mv.x), hmul2_bits(P[mt].z, mv.y),
                         hmul2_bits(P[mt].w, mv.y));
#define OSCAR_PV(I)                                                                    \
  {                                                                                    \
    const uint32_t x0 = slot_bits<I>(vw.x, vh.x), x1 = slot_bits<I>(vw.z, vh.z);       \
    const uint32_t y0 = slot_bits<I>(vw.y, vh.y), y1 = slot_bits<I>(vw.w, vh.w);       \
    _Pragma("unroll") for (int mt = 0; mt < MT; ++mt) {                                \
      mma16816(st.o[mt][I][0], a[mt], x0, x1);                                         \
      mma16816(st.o[mt][I][1], a[mt], y0, y1);                                         \
    }                                                                                  \
  }
    if constexpr (NG == kGroups) {
      if (gq == 0) { OSCAR_PV(0) OSCAR_PV(1) }
      if (gq == 1) { OSCAR_PV(2) OSCAR_PV(3) }
      if (gq == 2) { OSCAR_PV(4) OSCAR_PV(5) }
      if (gq == 3) { OSCAR_PV(6) OSCAR_PV(7) }
    } else {
      if (gq == 0) { OSCAR_PV(0) OSCAR_PV(1) OSCAR_PV(2) OSCAR_PV(3) }
      if (gq == 1) { OSCAR_PV(4) OSCAR_PV(5) OSCAR_PV(6) OSCAR_PV(7) }
    }
#undef OSCAR_PV
  }
  // columns 0 .. NG-1: the value zeros of the groups; column 4: ones, so that the
  // denominator sums the same rounded probabilities as the numerator
  constexpr uint32_t kOnes = 0x3c003c00u;
  uint2 mz = make_uint2(gid == 4 ? kOnes : 0u, gid == 4 ? kOnes : 0u);
  if (gid < NG) mz = *reinterpret_cast<const uint2*>(sb + vbase + 16 * (4 * gid + tig) + 8);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) mma16816(st.oz[mt], P[mt], mz.x, mz.y);
}

// INT2 positions [lo, hi) of KV head h: slice `split` of `nsplits` of their pages
template <int NG, int MT>
__device__ void int2_part(const TreeParams& p, int b, int h, int tile, int split, int nsplits, int lo, int hi,
                          uint8_t* smem, uint4* qs, State<MT>& st, float& unit, float& inv_ps) {
  constexpr int NP = 1;   // pages per softmax step
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int first = lo / kPage;
  const int npages = hi > lo ? (hi - 1) / kPage - first + 1 : 0;
  const int chunk = (npages + nsplits - 1) / nsplits;
  const int pbeg = first + split * chunk, pend = min(pbeg + chunk, first + npages);
  // warp w takes pages pbeg + w + 8 j
  const int nmine = pend - pbeg - warp > 0 ? (pend - pbeg - warp + kWarps - 1) / kWarps : 0;

  // row tiles of 16 rows read half of a 32-row record
  const uint32_t* rec = p.qrec + (((size_t)b * p.num_kv_heads + h) * p.row_tiles + tile * MT / 2) * kTreeRecWords;
  const int mt0 = MT == 1 ? tile & 1 : 0;
  for (int i = tid; i < MT * 8 * 32; i += kThreads) qs[i] = reinterpret_cast<const uint4*>(rec)[mt0 * 256 + i];
  uint2 zs[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) zs[mt] = *reinterpret_cast<const uint2*>(rec + kRecSums + 2 * ((mt0 + mt) * 32 + lane));
  unit = __uint_as_float(rec[kRecUnit]);
  const float tau = kLazyLog2 / unit;
  const float pscale = p.pv_scale[h], lg_ps = log2f(pscale);
  inv_ps = 1.f / pscale;

  uint8_t* sbuf = smem + warp * kStages * kBlockBytes;
  const uint32_t sring = (uint32_t)__cvta_generic_to_shared(sbuf) + lane * 16;
  constexpr int kBB = block_bytes(NG);
  const uint8_t* pool_h = p.pool + (size_t)h * kBB + lane * 16;
  const size_t stride = (size_t)p.num_kv_heads * kBB;
  const int32_t* row = p.page_table + (size_t)b * p.pt_stride;
  // page ids of pages 32 n .. 32 n + 31 of this warp, one per lane, and the next 32
  bool bad = false;
  auto load_ids = [&](int j0) {
    const int j = j0 + lane, at = pbeg + warp + kWarps * j;
    int id = -1;
    if (j < nmine) {
      id = at < p.pt_stride ? row[at] : -1;
      if (id < 0 || id >= p.num_pages) {
        bad = true;
        id = -1;
      }
    }
    return id;
  };
  int ids = load_ids(0), ids_next = load_ids(32);
  uint32_t okbits = 0u;   // bit j % 32: page j of those in flight has a valid id
  auto issue = [&](int j) {
    if (j && (j & 31) == 0) {
      ids = ids_next;
      ids_next = load_ids(j + 32);
    }
    const int id = j < nmine ? __shfl_sync(0xffffffffu, ids, j & 31) : -1;
    const uint32_t nb = id >= 0 ? 16u : 0u;
    okbits = (okbits & ~(1u << (j & 31))) | ((uint32_t)(id >= 0) << (j & 31));
    const uint8_t* src = pool_h + (size_t)max(id, 0) * stride;
    const uint32_t dst = sring + (j & (kStages - 1)) * kBlockBytes;
    cp_async16(dst, src, nb);
    cp_async16(dst + 512, src + 512, nb);
    if (NG == kGroups || lane < 16) cp_async16(dst + 1024, src + 1024, nb);
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) issue(s);
  __syncthreads();   // q~ fragments visible to every warp

  for (int j = 0; j < nmine; j += NP) {
    cp_wait<kStages - NP>();
    __syncwarp();
    float u[NP][MT][2][4];
    uint8_t* sb[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      sb[n] = sbuf + ((j + n) & (kStages - 1)) * kBlockBytes;
      page_scores<NG, MT>(sb[n], qs, zs, lane, u[n]);
    }
    // tokens outside [lo, hi), on a page this warp does not have or whose id is
    // outside the pool: scores -inf, value scales and zeros 0 in shared memory
    uint32_t valid = 0u;
#pragma unroll
    for (int n = 0; n < NP; ++n)
      valid |= page_token_bits((okbits >> ((j + n) & 31)) & 1u, (pbeg + warp + kWarps * (j + n)) * kPage, lo, hi) << (16 * n);
    if (valid != (NP == 2 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!((valid >> (16 * n + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1))) & 1u)) u[n][mt][i >> 2][i & 3] = -INFINITY;
      zero_masked_value_meta<NG>(sb[0], sb[NP - 1], NP == 2 ? valid : valid | (valid << 16), lane);
      __syncwarp();
    }
    update_max<MT, NP>(st, u, unit, tau);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      uint4 P[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // every row sees the same tokens: a maximum of -inf means none so far
        const float n0 = st.m[mt][0] == -INFINITY ? 0.f : fmaf(-st.m[mt][0], unit, lg_ps);
        const float n1 = st.m[mt][1] == -INFINITY ? 0.f : fmaf(-st.m[mt][1], unit, lg_ps);
        float e[2][4];
#pragma unroll
        for (int th = 0; th < 2; ++th)
#pragma unroll
          for (int i = 0; i < 4; ++i) e[th][i] = ex2(fmaf(u[n][mt][th][i], unit, i < 2 ? n0 : n1));
        // rounded to fp16 for the tensor cores: half a step is 2^-12 of a
        // probability, and the denominator sums the rounded ones
        P[mt] = make_uint4(f2_to_h2_bits(e[0][0], e[0][1]), f2_to_h2_bits(e[0][2], e[0][3]),
                           f2_to_h2_bits(e[1][0], e[1][1]), f2_to_h2_bits(e[1][2], e[1][3]));
      }
      page_values<NG, MT>(sb[n], lane, P, st);
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NP; ++n) issue(j + n + kStages);
  }
  cp_wait<0>();
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err_flags, OSCAR_FLAG_BAD_PAGE_ID);
}

constexpr int kBfChunk = kTreeWindowChunk;   // tokens per BF16 CTA: one 16-token tile for each warp
constexpr int kBfSmem(int mt) { return (2 * kBfChunk + 16 * mt) * kRow * 2; }

// BF16 tokens [128 chunk, + 128) of the sink, the ring and the tree's own nodes, raw basis
template <int MT>
__device__ void bf16_part(const TreeParams& p, int b, int h, int tile, int chunk, const oscar_seq_state& seq, int len,
                          uint8_t* smem, State<MT>& st) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int g = p.gqa, S = p.sink, W = p.recent;
  __shared__ unsigned long long anc[kTreeNodes];
  __shared__ int jump[kTreeNodes];
  const int L = seq.seq_len, ns = min(S, L), rb = max(seq.int2_end, S), nr = L > rb ? L - rb : 0;
  const int t0 = chunk * kBfChunk, total = ns + nr + len;
  const int n = min(kBfChunk, total - t0);
  const uint32_t sk = (uint32_t)__cvta_generic_to_shared(smem), sv = sk + kBfChunk * kRow * 2, sq = sv + kBfChunk * kRow * 2;
  const size_t slots = (size_t)(S + W);
  const __nv_bfloat16* wk = p.window + ((size_t)seq.window_row * p.num_kv_heads + h) * 2 * slots * kHeadDim;
  const __nv_bfloat16* wv = wk + slots * kHeadDim;
  const int nfill = (n + 15) / 16 * 16;   // rows up to a whole tile are zero-filled
  for (int i = tid; i < nfill * 16; i += kThreads) {
    const int r = i >> 4, u = i & 15, t = t0 + r;
    const bool in = r < n;
    const __nv_bfloat16 *ks = wk, *vs = wv;
    if (in) {
      if (t < ns + nr) {
        const size_t slot = t < ns ? t : S + (rb + t - ns) % W;
        ks = wk + slot * kHeadDim + 8 * u;
        vs = wv + slot * kHeadDim + 8 * u;
      } else {
        const size_t off = (((size_t)b * p.nodes + (t - ns - nr)) * p.num_kv_heads + h) * kHeadDim + 8 * u;
        ks = p.k + off;
        vs = p.v + off;
      }
    }
    cp_async16(sk + (r * kRow + 8 * u) * 2, ks, in ? 16u : 0u);
    cp_async16(sv + (r * kRow + 8 * u) * 2, vs, in ? 16u : 0u);
  }
  const int ncol = len * g, col0 = tile * 16 * MT;
  for (int i = tid; i < 16 * MT * 16; i += kThreads) {
    const int r = i >> 4, u = i & 15, col = col0 + r, node = col / g, m = col - node * g;
    const bool in = col < ncol;
    const size_t off = in ? (((size_t)b * p.nodes + node) * p.num_q_heads + h * g + m) * kHeadDim + 8 * u : 0;
    cp_async16(sq + (r * kRow + 8 * u) * 2, p.q + off, in ? 16u : 0u);
  }
  cp_commit();
  if (warp == 0) ancestor_masks(p.parent + (size_t)b * p.nodes, len, anc, jump, lane);
  cp_wait<0>();
  __syncthreads();
  if (16 * warp >= n) return;   // no barrier below in this function
  float u[1][MT][2][4] = {};
  const uint32_t krow = sk + ((16 * warp + (lane & 7) + 8 * (lane >> 4)) * kRow + 8 * ((lane >> 3) & 1)) * 2;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint4 kf = ldsm_x4(krow + 32 * kk);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4 a = ldsm_x4(sq + ((16 * mt + (lane & 15)) * kRow + 16 * kk + 8 * (lane >> 4)) * 2);
      mma16816_bf16(u[0][mt][0], a, kf.x, kf.y);
      mma16816_bf16(u[0][mt][1], a, kf.z, kf.w);
    }
  }
  const int tree0 = ns + nr - t0;   // row of node 0 in this chunk
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int node = min((col0 + 16 * mt + 8 * r + gid) / g, kTreeNodes - 1);
      const unsigned long long sees = anc[node];
#pragma unroll
      for (int th = 0; th < 2; ++th)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 16 * warp + 8 * th + 2 * tig + e, d = t - tree0;
          const bool on = t < n && (d < 0 || ((sees >> d) & 1ull));
          float& x = u[0][mt][th][2 * r + e];
          x = on ? x * p.scale_log2 : -INFINITY;
        }
    }
  update_max<MT, 1>(st, u, 1.f, 0.f);
  // probabilities and values on the bf16 tensor cores, the probabilities split
  // into two bf16 parts (16 bits), so that any bf16 value is exact
  uint4 hi[MT], lo[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    uint32_t hw[4], lw[4];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int th = 0; th < 2; ++th)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float nb = st.m[mt][r] == -INFINITY ? 0.f : -st.m[mt][r];
        const float e0 = ex2(u[0][mt][th][2 * r] + nb), e1 = ex2(u[0][mt][th][2 * r + 1] + nb);
        const uint32_t x = f2_to_bf2_bits(e0, e1);
        const float2 xf = bf2_bits_to_f2(x);
        const uint32_t y = f2_to_bf2_bits(e0 - xf.x, e1 - xf.y);
        const float2 yf = bf2_bits_to_f2(y);
        hw[2 * th + r] = x;
        lw[2 * th + r] = y;
        sum[r] += (xf.x + yf.x) + (xf.y + yf.y);
      }
    hi[mt] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    lo[mt] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    const float l0 = quad_sum(sum[0]), l1 = quad_sum(sum[1]);
    st.oz[mt][0] = tig == 2 ? l0 : 0.f;   // column 4 is the denominator, no zero points
    st.oz[mt][2] = tig == 2 ? l1 : 0.f;
  }
  const uint32_t vrow = sv + ((16 * warp + (lane & 15)) * kRow + 8 * (lane >> 4)) * 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 vf = ldsm_x4_t(vrow + 32 * i);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      mma16816_bf16(st.o[mt][i][0], lo[mt], vf.x, vf.y);
      mma16816_bf16(st.o[mt][i][1], lo[mt], vf.z, vf.w);
      mma16816_bf16(st.o[mt][i][0], hi[mt], vf.x, vf.y);
      mma16816_bf16(st.o[mt][i][1], hi[mt], vf.z, vf.w);
    }
  }
}

constexpr int tree_smem(int mt) {
  const int merge = (kWarps * 16 * mt * kPartRow + kWarps * 16 * mt * 3 + 16 * mt * 2) * 4;
  const int int2 = kWarps * kStages * kBlockBytes + mt * 8 * 32 * 16;
  const int bf = kBfSmem(mt);
  return merge > int2 ? (merge > bf ? merge : bf) : (int2 > bf ? int2 : bf);
}

template <int NG, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 2 : 1) oscar_tree_attn_kernel(TreeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int ntiles = p.col_tiles, tile = blockIdx.x % ntiles, slot = blockIdx.x / ntiles;
  const int h = blockIdx.y, b = blockIdx.z;
  constexpr int NC = 16 * MT;
  pdl_wait();
  pdl_trigger();
  const oscar_seq_state seq = p.state[b];
  const int len = p.draft_len ? p.draft_len[b] : p.nodes;
  const int ncol = len * p.gqa, col0 = tile * NC;
  // a bad state or length: the merge writes the request's zeros and reads no partial
  if (!state_ok(seq, p.sink, p.recent, p.max_batch) || len < 0 || len > p.nodes || col0 >= ncol) return;
  State<MT> st;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    st.m[mt][0] = st.m[mt][1] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) st.oz[mt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) st.o[mt][i][j >> 2][j & 3] = 0.f;
  }
  const int nslots = p.win_slots + p.splits;
  const int rows = p.nodes * p.gqa;
  float* part = p.part + (((size_t)b * p.num_kv_heads + h) * nslots + slot) * rows * (size_t)kPartFloats;
  float unit = 1.f, inv_ps = 1.f;
  const bool int2 = slot >= p.win_slots;
  const int lo = p.sink, hi = min(seq.int2_end, seq.seq_len);
  bool empty;
  if (int2) {
    const int npages = hi > lo ? (hi - 1) / kPage - lo / kPage + 1 : 0;
    empty = (slot - p.win_slots) * ((npages + p.splits - 1) / p.splits) >= npages;
  } else {
    const int rb = max(seq.int2_end, p.sink);
    empty = slot * kBfChunk >= min(p.sink, seq.seq_len) + max(seq.seq_len - rb, 0) + len;
  }
  if (empty) {   // no keys: the merge skips the slot
    for (int i = tid; i < min(NC, ncol - col0); i += kThreads) {
      part[(size_t)(col0 + i) * kPartFloats + kHeadDim] = -INFINITY;
      part[(size_t)(col0 + i) * kPartFloats + kHeadDim + 1] = 0.f;
    }
    return;
  }
  if (int2)
    int2_part<NG, MT>(p, b, h, tile, slot - p.win_slots, p.splits, lo, hi, smem,
                      reinterpret_cast<uint4*>(smem + kWarps * kStages * kBlockBytes), st, unit, inv_ps);
  else
    bf16_part<MT>(p, b, h, tile, slot, seq, len, smem, st);

  // ---- the 8 warps' partials -> shared memory, then the CTA's merge -----------
  __syncthreads();   // staging buffers are reused
  float* wpart = reinterpret_cast<float*>(smem);            // [8 warps][NC][kPartRow]
  float* wml = wpart + kWarps * NC * kPartRow;              // [8 warps][NC][2]
  float* wts = wml + kWarps * NC * 2;                       // [NC][8]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // zero-point sums of channel block i's group: lane tig = group / 2, element group % 2
      const int gq = i / (8 / NG), src = (lane & ~3) | (gq >> 1);
      const float z0 = __shfl_sync(0xffffffffu, st.oz[mt][gq & 1], src) * inv_ps;
      const float z1 = __shfl_sync(0xffffffffu, st.oz[mt][2 + (gq & 1)], src) * inv_ps;
      const float sc = int2 ? 16777216.f / slot_factor(i) * inv_ps : 1.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float* dst = wpart + (warp * NC + 16 * mt + gid) * kPartRow + 16 * i + 8 * x + 2 * tig;
        const float* a = st.o[mt][i][x];
        *reinterpret_cast<float2*>(dst) = make_float2(fmaf(a[0], sc, z0), fmaf(a[1], sc, z0));
        *reinterpret_cast<float2*>(dst + 8 * kPartRow) = make_float2(fmaf(a[2], sc, z1), fmaf(a[3], sc, z1));
      }
    }
    if (tig == 2) {
      float* d0 = wml + (warp * NC + 16 * mt + gid) * 2;
      d0[0] = st.m[mt][0] * unit;
      d0[1] = st.oz[mt][0] * inv_ps;
      d0[16] = st.m[mt][1] * unit;
      d0[17] = st.oz[mt][2] * inv_ps;
    }
  }
  __syncthreads();
  if (tid < NC * kWarps) {   // thread (row n, warp w): the 8 warps of a row are consecutive lanes
    const int n = tid >> 3, w = tid & 7;
    const float mw = wml[(w * NC + n) * 2];
    float M = mw;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float sw = mw == -INFINITY ? 0.f : exp2f(mw - M);
    float l = sw * wml[(w * NC + n) * 2 + 1];
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    wts[n * kWarps + w] = sw;
    if (w == 0 && col0 + n < ncol) {
      float* dst = part + (size_t)(col0 + n) * kPartFloats + kHeadDim;
      dst[0] = M;
      dst[1] = l;
    }
  }
  __syncthreads();
  for (int i = tid; i < min(NC, ncol - col0) * 32; i += kThreads) {
    const int n = i >> 5, c = 4 * (i & 31);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = wts[n * kWarps + w];
      const float4 x = *reinterpret_cast<const float4*>(wpart + (w * NC + n) * kPartRow + c);
      o.x = fmaf(a, x.x, o.x);
      o.y = fmaf(a, x.y, o.y);
      o.z = fmaf(a, x.z, o.z);
      o.w = fmaf(a, x.w, o.w);
    }
    *reinterpret_cast<float4*>(part + (size_t)(col0 + n) * kPartFloats + c) = o;
  }
}

// --------------------------------------------------------------------------
// 3. merge: CTA x handles 16 query rows of (request z, KV head y)
// --------------------------------------------------------------------------
constexpr int kMergeThreads = 128;
constexpr int kMergeRows = 16;

__global__ void __launch_bounds__(kMergeThreads) oscar_tree_merge_kernel(TreeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, row0 = blockIdx.x * kMergeRows, g = p.gqa;
  const int nslots = p.win_slots + p.splits, rows = p.nodes * g;
  float* wts = reinterpret_cast<float*>(smem);            // [nslots][16]
  __shared__ __align__(16) __half ox[kMergeRows][kRow];   // INT2 sums over the denominator (R_V basis)
  __shared__ __align__(16) float ow[kMergeRows][kHeadDim + 4];   // window and tree sums over it
  // un-rotation operand, constant: warp w produces channels 32 w .. 32 w + 31,
  // out[n] = sum_k x[k] R_V[n][k]
  uint2 bf[4][8];
  if (!p.fold_rv) {
    const __half* rv = p.rv16 + (size_t)h * kHeadDim * kHeadDim;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const __half* src = rv + (32 * warp + 8 * nt + gid) * kHeadDim + 16 * kk + 2 * tig;
        bf[nt][kk] = make_uint2(*reinterpret_cast<const uint32_t*>(src), *reinterpret_cast<const uint32_t*>(src + 8));
      }
  }
  pdl_wait();
  pdl_trigger();
  const oscar_seq_state seq = p.state[b];
  const int len = p.draft_len ? p.draft_len[b] : p.nodes;
  bool ok = len >= 0 && len <= p.nodes;
  if (ok)
    for (int i = tid; i < len; i += kMergeThreads) {
      const int q = p.parent[(size_t)b * p.nodes + i];
      ok = ok && (i == 0 ? q == -1 : q >= 0 && q < i);
    }
  const bool tree_ok = __syncthreads_and(ok);
  const bool seq_ok = state_ok(seq, p.sink, p.recent, p.max_batch);
  if (!tree_ok || !seq_ok) {
    if (tid == 0 && blockIdx.x == 0 && h == 0)
      atomicOr(p.err_flags, (tree_ok ? 0u : OSCAR_FLAG_BAD_TREE) | (seq_ok ? 0u : OSCAR_FLAG_BAD_STATE));
    for (int i = tid; i < min(kMergeRows, rows - row0) * kHeadDim; i += kMergeThreads) {
      const int r = row0 + i / kHeadDim, node = r / g;
      p.o[(((size_t)b * p.nodes + node) * p.num_q_heads + h * g + (r - node * g)) * kHeadDim + i % kHeadDim] =
          __float2bfloat16(0.f);
    }
    return;
  }
  const int nrows = min(kMergeRows, len * g - row0);
  if (nrows <= 0) return;   // rows of nodes the request does not use: left as they are
  const float* part = p.part + (((size_t)b * p.num_kv_heads + h) * nslots * rows + row0) * kPartFloats;
  const size_t slot_stride = (size_t)rows * kPartFloats;
  // thread (row r, eighth j): slot weights over the denominator
  const int r = tid >> 3, j = tid & 7;
  float inv = 0.f;
  {
    float M = -INFINITY;
    if (r < nrows)
      for (int s = j; s < nslots; s += 8) M = fmaxf(M, part[s * slot_stride + r * kPartFloats + kHeadDim]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.f;
    for (int s = j; s < nslots; s += 8) {
      const float2 ml = r < nrows ? *reinterpret_cast<const float2*>(part + s * slot_stride + r * kPartFloats + kHeadDim)
                                  : make_float2(-INFINITY, 0.f);
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      wts[s * kMergeRows + r] = w;
      l = fmaf(w, ml.y, l);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    inv = 1.f / l;   // a row always sees itself: l >= 1 up to rounding
  }
  __syncwarp();
  float a2[16] = {}, aw[16] = {};
  for (int s = 0; s < nslots; ++s) {
    const float w = wts[s * kMergeRows + r];
    if (w != 0.f) {   // a slot without keys left its sums unwritten
      const float* src = part + s * slot_stride + r * kPartFloats + 4 * j;
      const bool win = s < p.win_slots;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = *reinterpret_cast<const float4*>(src + 32 * c);
        float* a = win ? aw + 4 * c : a2 + 4 * c;
        a[0] = fmaf(w, x.x, a[0]);
        a[1] = fmaf(w, x.y, a[1]);
        a[2] = fmaf(w, x.z, a[2]);
        a[3] = fmaf(w, x.w, a[3]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    *reinterpret_cast<float4*>(&ow[r][32 * c + 4 * j]) =
        make_float4(aw[4 * c] * inv, aw[4 * c + 1] * inv, aw[4 * c + 2] * inv, aw[4 * c + 3] * inv);
    // the un-rotation runs on fp16 operands (2^-12 of a value each); with the
    // rotation folded into the model the sums are the result and stay fp32
    if (p.fold_rv) {
      float* d = &ow[r][32 * c + 4 * j];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = fmaf(a2[4 * c + e], inv, d[e]);
    } else {
      *reinterpret_cast<uint2*>(&ox[r][32 * c + 4 * j]) =
          make_uint2(f2_to_h2_bits(a2[4 * c] * inv, a2[4 * c + 1] * inv),
                     f2_to_h2_bits(a2[4 * c + 2] * inv, a2[4 * c + 3] * inv));
    }
  }
  __syncthreads();
  float acc[4][4] = {};
  if (!p.fold_rv) {
    const uint32_t sx = (uint32_t)__cvta_generic_to_shared(&ox[0][0]);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint4 a = ldsm_x4(sx + ((lane & 15) * kRow + 16 * kk + 8 * (lane >> 4)) * 2);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) mma16816(acc[nt], a, bf[nt][kk].x, bf[nt][kk].y);
    }
  }
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int rr = gid + 8 * half, c = 32 * warp + 8 * nt + 2 * tig;
      if (rr < nrows) {
        const int row = row0 + rr, node = row / g;
        const size_t at = (((size_t)b * p.nodes + node) * p.num_q_heads + h * g + (row - node * g)) * kHeadDim + c;
        *reinterpret_cast<uint32_t*>(p.o + at) =
            f2_to_bf2_bits(acc[nt][2 * half] + ow[rr][c], acc[nt][2 * half + 1] + ow[rr][c + 1]);
      }
    }
}

template <int NG>
cudaError_t set_attrs() {
  cudaError_t e = cudaFuncSetAttribute(oscar_tree_attn_kernel<NG, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, tree_smem(1));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(oscar_tree_attn_kernel<NG, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, tree_smem(2));
  return e;
}

}  // namespace

cudaError_t launch_tree_attn(const TreeParams& p, cudaStream_t s) {
  static PerDeviceOnce attrs;
  const cudaError_t ea = once_for_current_device(attrs, [] {
    cudaError_t e = set_attrs<kGroups>();
    if (e == cudaSuccess) e = set_attrs<2>();
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(oscar_tree_rotate_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRotSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(oscar_tree_rotate_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRotSmem);
    return e;
  });
  if (ea != cudaSuccess) return ea;
  static_assert(kRecUnit < kTreeRecWords, "query record");
  const int nslots = p.win_slots + p.splits, rows = p.nodes * p.gqa;
  const bool wide = p.tile_rows == 2 * kWideRows;
  cudaError_t e = launch_pdl(wide ? oscar_tree_rotate_kernel<true> : oscar_tree_rotate_kernel<false>, dim3(p.row_tiles, p.num_kv_heads, p.batch), dim3(kRotThreads),
                             kRotSmem, s, p);
  const dim3 grid(p.col_tiles * nslots, p.num_kv_heads, p.batch);
  const bool one = p.tile_rows == 16;
  if (e == cudaSuccess && wide) e = launch_tree_wide(p, s);
  if (e == cudaSuccess && !wide)
    e = p.ngroups == kGroups
            ? launch_pdl(one ? oscar_tree_attn_kernel<kGroups, 1> : oscar_tree_attn_kernel<kGroups, 2>, grid,
                         dim3(kThreads), tree_smem(one ? 1 : 2), s, p)
            : launch_pdl(one ? oscar_tree_attn_kernel<2, 1> : oscar_tree_attn_kernel<2, 2>, grid, dim3(kThreads),
                         tree_smem(one ? 1 : 2), s, p);
  if (e == cudaSuccess)
    e = launch_pdl(oscar_tree_merge_kernel, dim3((rows + kMergeRows - 1) / kMergeRows, p.num_kv_heads, p.batch),
                   dim3(kMergeThreads), nslots * kMergeRows * 4, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
