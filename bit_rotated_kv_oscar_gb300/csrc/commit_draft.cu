// Commit of accepted drafted tokens: the rows of a draft's k and v that the
// verification accepted are appended to the OSCAR cache.
//
// The result is oscar_quant_append of the gathered rows, byte for byte: with L, E
// the state before, n accepted rows and E' = max(E, sink, L + n - recent), positions
// below the sink limit and those from E' on go to the BF16 sink / ring, positions
// [E, E') are rotated, clipped, group-quantised and packed ("Juntos, AI Open-Sources
// OSCAR ..." (7minutos.es), "El sistema de servicio"). How many rows a request
// accepted is known to the device only, so the counts and row indices are read
// there and every request may append a different number.
//
// CTA (x, h, kind) takes the keys or the values of KV head h of requests x, x + gridDim.x,
// ..., sixteen at a time: one warp reads and checks one request's state, count and path. The
// rotation (64 KiB) is staged in shared memory once, two CTAs per SM, and the rows that
// all of these requests quantise are rotated sixteen at a time, eight rows by two channels to
// a thread; the next sixteen are on their way meanwhile. The sums keep the append kernel's
// order (two chains of 64 terms per channel, then their sum), which the byte equality needs
// and which leaves the tensor cores out.
//
// Bound: latency for one request (7.5 us with the launch; state, rows, rotation and stores
// follow one another). 64 requests, 552 rows, 8 heads: 29 us, of which 6 remain without rows
// to quantise; the rest is two or three rounds of sixteen rows for a CTA, about 5 us of
// rotation (shared-memory reads) and 4 us of fetch, quantisation and stores each.
#include <type_traits>

#include "oscar_internal.cuh"
#include "token_quant.cuh"
#include "warp_mma.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 512;
constexpr int kReqs = kThreads / 32;        // requests read at once
constexpr int kRows = 16;                   // rows rotated at once
static_assert(kRows == kThreads / 32, "a warp stores a row");
constexpr int kMat = kHeadDim * kHeadDim;
struct CommitSmem {
  float rot[kMat];                          // R_K[h] or R_V[h]
  float x[kRows][kHeadDim];                 // rows being quantised
  float red[kRows][2][kHeadDim];            // their rotations, two half sums per channel
  __nv_bfloat16 raw[2][kRows][kHeadDim];    // the same rows as they lie in the cache or the draft, and the next
  uint8_t codes[kRows][2][kHeadDim];        // one kind's is used (store_token_block's layout)
  __half meta[kRows][2][kGroups][2];
  int path[kReqs][kTreeNodes];
  int n[kReqs], L[kReqs], E[kReqs], row[kReqs];   // accepted rows, state and window row; n = 0: nothing to do
  int first[kReqs + 1];                     // rows to quantise before each request
  int page[2][kRows], slot[2][kRows];       // page ids of the rows in raw, and their places in them
};

__global__ void __launch_bounds__(kThreads, 2) oscar_commit_draft_kernel(CommitParams p) {
  extern __shared__ __align__(16) uint8_t dsm[];
  CommitSmem& sm = *reinterpret_cast<CommitSmem*>(dsm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, kind = blockIdx.z;
  const int S = p.sink, W = p.recent, Hkv = p.num_kv_heads, ng = p.ngroups;
  // constant data before the wait
  const float* rot = (kind ? p.R_V : p.R_K) + (size_t)h * kMat;
  const bool fold = kind && p.fold_rv;   // the values arrive in the R_V basis
  const uint32_t srot = (uint32_t)__cvta_generic_to_shared(&sm.rot[0]);
  if (!fold)
    for (int i = tid; i < kMat / 4; i += kThreads) wm::cp_async16(srot + 16 * i, rot + 4 * i);
  wm::cp_commit();
  pdl_wait();
  pdl_trigger();
  const float clip = (kind ? p.clip_V : p.clip_K)[h];
  const size_t slots = (size_t)(S + W);
  const __nv_bfloat16* input = kind ? p.v : p.k;
  auto window_of = [&](int q) { return p.window + (((size_t)sm.row[q] * Hkv + h) * 2 + kind) * slots * kHeadDim; };
  for (int b0 = blockIdx.x; b0 < p.batch; b0 += kReqs * gridDim.x) {
    auto request = [&](int q) { return b0 + q * (int)gridDim.x; };
    __syncthreads();   // the previous requests' shared data is consumed
    oscar_seq_state out{};   // this warp's request afterwards
    uint32_t bad = 0u;
    {
      const int b = request(warp);
      int n = 0, m = 0;
      if (b < p.batch) {
        const oscar_seq_state st = p.state[b];
        const int c = p.count[b];
        bool good = c >= 0 && c <= p.nodes;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = lane + 32 * e;
          if (i < p.nodes) {
            const int r = p.path[(size_t)b * p.nodes + i];
            sm.path[warp][i] = r;
            if (i < c) good = good && r >= 0 && r < p.nodes;
          }
        }
        const bool path_ok = __all_sync(0xffffffffu, good), seq_ok = state_ok(st, S, W, p.max_batch);
        if (path_ok && seq_ok) n = c;
        const int64_t nl = (int64_t)st.seq_len + n, ne = nl - W;
        const int e0 = st.int2_end, e1 = max(e0, S);   // state_ok: int2_end >= sink
        const int e2 = (int)(ne > e1 ? ne : e1);
        m = n > 0 ? e2 - e0 : 0;
        if (lane == 0) {
          sm.L[warp] = st.seq_len;
          sm.E[warp] = e0;
          sm.row[warp] = st.window_row;
        }
        out = st;
        out.seq_len = (int32_t)nl;
        out.int2_end = e2;
        bad = (path_ok ? 0u : OSCAR_FLAG_BAD_TREE) | (seq_ok ? 0u : OSCAR_FLAG_BAD_STATE);
      }
      if (lane == 0) {
        sm.n[warp] = n;
        sm.first[warp + 1] = m;
      }
    }
    __syncthreads();
    if (warp == 0) {
      int m = lane < kReqs ? sm.first[lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < kReqs; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m += up;
      }
      if (lane < kReqs) sm.first[lane + 1] = m;
      if (lane == 0) sm.first[0] = 0;
    }
    __syncthreads();
    const int M = sm.first[kReqs];
    auto fetch = [&](int r0, int buf) {   // rows r0 .. of the M: a half-warp a row, 16-byte pieces
      if (tid < kRows * 16) {
        const int r = tid >> 4, c = 8 * (tid & 15), at = r0 + r;
        const uint32_t before = __ballot_sync(0xffffffffu, at >= sm.first[(lane & 15) + 1]);
        const int q = __popc((before >> (lane & 16)) & 0xffffu);   // its request
        if (at < M) {
          const int pos = sm.E[q] + (at - sm.first[q]), L = sm.L[q];
          const __nv_bfloat16* src =
              pos < L ? window_of(q) + (size_t)(S + pos % W) * kHeadDim + c
                      : input + (((size_t)request(q) * p.nodes + sm.path[q][pos - L]) * Hkv + h) * kHeadDim + c;
          wm::cp_async16((uint32_t)__cvta_generic_to_shared(&sm.raw[buf][r][c]), src);
          if ((tid & 15) == 0) {
            const int pidx = pos / kPage;
            sm.slot[buf][r] = pos % kPage;
            if (pidx < p.pt_stride)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"((uint32_t)__cvta_generic_to_shared(&sm.page[buf][r])),
                           "l"(p.page_table + (size_t)request(q) * p.pt_stride + pidx));
            else
              sm.page[buf][r] = -1;
          }
        }
      }
      wm::cp_commit();
    };
    if (M > 0) fetch(0, 0);
    for (int r0 = 0, buf = 0; r0 < M; r0 += kRows, buf ^= 1) {
      const int rows = min(kRows, M - r0);
      if (r0 + kRows < M) {
        fetch(r0 + kRows, buf ^ 1);
        wm::cp_wait<1>();
      } else {
        wm::cp_wait<0>();
      }
      __syncthreads();
      for (int i = tid; i < rows * 32; i += kThreads) {
        const uint2 w = reinterpret_cast<const uint2*>(&sm.raw[buf][0][0])[i];
        reinterpret_cast<float4*>(&sm.x[0][0])[i] =
            make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xffff0000u));
      }
      __syncthreads();
      {
        // thread (rows 8 g .., half, channels c, c + 1): 64 terms of x R in order, for each.
        // Half of the threads: what counts is shared-memory reads per product, and 16 sums
        // a thread halve those of x (64 requests, 552 rows: 32 us against 36)
        const int g = tid >> 7, half = (tid >> 6) & 1, c = 2 * (tid & 63), k0 = 64 * half, n = rows - 8 * g;
        if (fold) {
          if (g < 2)
            for (int r = 8 * g; r < min(rows, 8 * g + 8); ++r)
              *reinterpret_cast<float2*>(&sm.red[r][half][c]) =
                  half ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2*>(&sm.x[r][c]);
        } else if (g < 2 && n > 0) {
          const float* R = sm.rot + k0 * kHeadDim + c;
          auto rotate = [&](auto count) {
            constexpr int N = decltype(count)::value;
            float2 acc[N] = {};
#pragma unroll 2
            for (int i = 0; i < 64; i += 4) {
              float2 v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float2*>(R + (i + e) * kHeadDim);
#pragma unroll
              for (int r = 0; r < N; ++r) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.x[8 * g + r][k0 + i]);
                const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  acc[r].x = fmaf(xs[e], v[e].x, acc[r].x);
                  acc[r].y = fmaf(xs[e], v[e].y, acc[r].y);
                }
              }
            }
#pragma unroll
            for (int r = 0; r < N; ++r)   // rows past the last are not used
              *reinterpret_cast<float2*>(&sm.red[8 * g + r][half][c]) = acc[r];
          };
          if (n > 4) rotate(std::integral_constant<int, 8>());
          else if (n > 1) rotate(std::integral_constant<int, 4>());
          else rotate(std::integral_constant<int, 1>());
        }
      }
      __syncthreads();
      // warp item (row, 64 channels): clip, group extremes, scale, zero, codes
      for (int it = warp; it < rows * 2; it += kThreads / 32) {
        const int r = it >> 1, c = 64 * (it & 1) + lane;
        float x[2], mn[2], mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = sm.red[r][0][c + 32 * e] + sm.red[r][1][c + 32 * e];
          x[e] = fminf(fmaxf(v, -clip), clip);
          mn[e] = mx[e] = x[e];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
          }
        if (ng != kGroups) {
          mn[0] = mn[1] = fminf(mn[0], mn[1]);
          mx[0] = mx[1] = fmaxf(mx[0], mx[1]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          __half s16, z16;
          group_scale_zero(mn[e], mx[e], s16, z16);
          sm.codes[r][kind][c + 32 * e] = (uint8_t)group_code(x[e], __half2float(s16), __half2float(z16));
          const int ch = c + 32 * e, gsz = kHeadDim / ng;
          if ((ch & (gsz - 1)) == 0) {
            sm.meta[r][kind][ch / gsz][0] = s16;
            sm.meta[r][kind][ch / gsz][1] = z16;
          }
        }
      }
      __syncthreads();
      if (warp < rows) {   // a warp per row
        // the roles of this kind: K codes 0 .. 7, metadata 64 .. 67; V codes 32 .. 47, metadata 68 .. 71
        const int r = warp, ncodes = kind ? 16 : 8, role = lane < ncodes ? 32 * kind + lane : 64 + 4 * kind + lane - ncodes;
        if (lane < ncodes + 4) {
          const int id = sm.page[buf][r];
          if (id >= 0 && id < p.num_pages)
            store_token_block(p.pool + ((size_t)id * Hkv + h) * block_bytes(ng), sm.slot[buf][r], role, ng, sm.codes[r], sm.meta[r]);
          else if (lane == 0)
            atomicOr(p.err_flags, OSCAR_FLAG_BAD_PAGE_ID);
        }
      }
      __syncthreads();   // the next fetch overwrites the page ids read here
    }
    __syncthreads();
    // every ring entry that leaves has been read: the new rows take their places. A
    // half-warp per row (16 pieces of 16 bytes), four rows' loads before their stores
    const int nreq = min(kReqs, (p.batch - b0 + (int)gridDim.x - 1) / (int)gridDim.x), nrows = nreq * p.nodes;
    for (int i0 = tid >> 4; i0 < nrows; i0 += 4 * (kThreads / 16)) {
      uint4 x[4];
      __nv_bfloat16* dst[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * (kThreads / 16), q = i / p.nodes, j = i - q * p.nodes, c = 8 * (tid & 15);
        dst[u] = nullptr;
        if (i >= nrows || j >= sm.n[q]) continue;
        const int pos = sm.L[q] + j, e2 = sm.E[q] + (sm.first[q + 1] - sm.first[q]);
        if (pos >= S && pos < e2) continue;
        dst[u] = window_of(q) + (size_t)(pos < S ? pos : S + pos % W) * kHeadDim + c;
        x[u] = *reinterpret_cast<const uint4*>(
            input + (((size_t)request(q) * p.nodes + sm.path[q][j]) * Hkv + h) * kHeadDim + c);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = x[u];
    }
    // the last of a request's 2 Hkv CTAs to have read its state publishes the new one: each
    // reads it before taking its ticket. The counters belong to window rows and wrap to 0, so
    // calls on other requests may run at the same time
    if (lane == 0 && request(warp) < p.batch) {
      if (bad) {
        if (h == 0 && kind == 0) atomicOr(p.err_flags, bad);
      } else {
        asm volatile("fence.acq_rel.gpu;\n" ::: "memory");
        if (atomicInc(p.tickets + out.window_row, 2u * Hkv - 1u) == 2u * Hkv - 1u) {
          asm volatile("fence.acq_rel.gpu;\n" ::: "memory");
          p.state[request(warp)] = out;
        }
      }
    }
  }
  wm::cp_wait<0>();
}

}  // namespace

cudaError_t launch_commit_draft(const CommitParams& p, int num_sms, cudaStream_t s) {
  static PerDeviceOnce attrs;
  const cudaError_t ea = once_for_current_device(attrs, [] {
    return cudaFuncSetAttribute(oscar_commit_draft_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(CommitSmem));
  });
  if (ea != cudaSuccess) return ea;
  int nx = num_sms / p.num_kv_heads;   // two CTAs per SM, keys and values
  nx = nx < 1 ? 1 : (nx > p.batch ? p.batch : nx);
  const cudaError_t e = launch_pdl(oscar_commit_draft_kernel, dim3((unsigned)nx, (unsigned)p.num_kv_heads, 2), dim3(kThreads),
                                   sizeof(CommitSmem), s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
