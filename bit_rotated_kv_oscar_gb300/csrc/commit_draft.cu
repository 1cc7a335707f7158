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
// CTA (x, h) takes KV head h of requests x, x + gridDim.x, ...: the head's two
// rotations (128 KiB) are staged in shared memory once, and the rows to quantise
// are rotated eight at a time, so that one shared-memory read of a rotation entry
// feeds eight FMAs. The sums keep the append kernel's order (two chains of 64 terms
// per channel, then their sum), which the byte equality needs.
#include "oscar_internal.cuh"
#include "token_quant.cuh"
#include "warp_mma.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 8;                    // rows rotated at once
constexpr int kMat = kHeadDim * kHeadDim;
struct CommitSmem {
  float rot[2][kMat];                       // R_K[h], R_V[h]
  float x[kRows][2][kHeadDim];              // rows being quantised, K and V
  float red[kRows][2][2][kHeadDim];         // their rotations, two half sums per channel
  uint8_t codes[kRows][2][kHeadDim];
  __half meta[kRows][2][kGroups][2];
  int path[kTreeNodes];
};

__global__ void __launch_bounds__(kThreads, 1) oscar_commit_draft_kernel(CommitParams p) {
  extern __shared__ __align__(16) uint8_t dsm[];
  CommitSmem& sm = *reinterpret_cast<CommitSmem*>(dsm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
  const int S = p.sink, W = p.recent, Hkv = p.num_kv_heads, ng = p.ngroups;
  // constant data before the wait
  const float* rk = p.R_K + (size_t)h * kMat;
  const float* rv = p.R_V + (size_t)h * kMat;
  const uint32_t srot = (uint32_t)__cvta_generic_to_shared(&sm.rot[0][0]);
  for (int i = tid; i < kMat / 4; i += kThreads) {
    wm::cp_async16(srot + 16 * i, rk + 4 * i);
    if (!p.fold_rv) wm::cp_async16(srot + kMat * 4 + 16 * i, rv + 4 * i);
  }
  wm::cp_commit();
  pdl_wait();
  pdl_trigger();
  bool staged = false;
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    __syncthreads();   // the previous request's shared data is consumed
    const oscar_seq_state st = p.state[b];
    const int n = p.count[b];
    bool good = n >= 0 && n <= p.nodes;
    if (good && tid < n) {
      const int r = p.path[(size_t)b * p.nodes + tid];
      sm.path[tid] = r;
      good = r >= 0 && r < p.nodes;
    }
    const bool path_ok = __syncthreads_and(good);
    const bool seq_ok = state_ok(st, S, W, p.max_batch);
    if (tid == 0) {
      // the last of the request's Hkv CTAs to have read its state publishes the
      // new one: each reads it before taking its ticket
      asm volatile("fence.acq_rel.gpu;\n" ::: "memory");
      if (atomicAdd(p.tickets + b, 1u) == (unsigned)Hkv - 1u) {
        asm volatile("fence.acq_rel.gpu;\n" ::: "memory");
        if (path_ok && seq_ok) {
          const int64_t nl = (int64_t)st.seq_len + n, ne = nl - W;
          oscar_seq_state out = st;
          out.seq_len = (int32_t)nl;
          out.int2_end = (int32_t)(ne > max(st.int2_end, S) ? ne : max(st.int2_end, S));
          p.state[b] = out;
        } else {
          atomicOr(p.err_flags, (path_ok ? 0u : OSCAR_FLAG_BAD_TREE) | (seq_ok ? 0u : OSCAR_FLAG_BAD_STATE));
        }
        p.tickets[b] = 0u;
      }
    }
    if (!path_ok || !seq_ok || n == 0) continue;
    const int64_t L = st.seq_len, E = st.int2_end;
    int64_t E2 = L + n - W;
    if (E2 < E) E2 = E;
    if (E2 < S) E2 = S;
    const size_t slots = (size_t)(S + W);
    __nv_bfloat16* win = p.window + ((size_t)st.window_row * Hkv + h) * 2 * slots * kHeadDim;   // K rows, then V rows
    const int m = (int)(E2 - E);   // rows to quantise: positions E .. E2 - 1, at most n
    if (m > 0 && !staged) {
      wm::cp_wait<0>();
      staged = true;   // visible to the other threads after the barrier below
    }
    for (int i0 = 0; i0 < m; i0 += kRows) {
      const int rows = min(kRows, m - i0);
      // 8 rows x 2 kinds x 128 channels, 4 channels per thread
      for (int i = tid; i < rows * 64; i += kThreads) {
        const int r = i >> 6, kind = (i >> 5) & 1, c = 4 * (i & 31);
        const int64_t pos = E + i0 + r;
        const __nv_bfloat16* src;
        if (pos < L)
          src = win + (kind * slots + S + pos % W) * kHeadDim + c;
        else
          src = (kind ? p.v : p.k) + (((size_t)b * p.nodes + sm.path[pos - L]) * Hkv + h) * kHeadDim + c;
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        *reinterpret_cast<float4*>(&sm.x[r][kind][c]) =
            make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xffff0000u));
      }
      __syncthreads();
      {
        // thread (kind, half, channel c): 64 terms of x R in order, for every row
        const int kind = tid >> 8, half = (tid >> 7) & 1, c = tid & 127, k0 = 64 * half;
        if (kind == 1 && p.fold_rv) {
          for (int r = 0; r < rows; ++r) sm.red[r][1][half][c] = half ? 0.f : sm.x[r][1][c];
        } else {
          float acc[kRows] = {};
          const float* R = sm.rot[kind] + k0 * kHeadDim + c;
#pragma unroll 4
          for (int i = 0; i < 64; i += 4) {
            const float r0 = R[i * kHeadDim], r1 = R[(i + 1) * kHeadDim], r2 = R[(i + 2) * kHeadDim],
                        r3 = R[(i + 3) * kHeadDim];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
              if (r < rows) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.x[r][kind][k0 + i]);
                acc[r] = fmaf(x.x, r0, acc[r]);
                acc[r] = fmaf(x.y, r1, acc[r]);
                acc[r] = fmaf(x.z, r2, acc[r]);
                acc[r] = fmaf(x.w, r3, acc[r]);
              }
            }
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (r < rows) sm.red[r][kind][half][c] = acc[r];
        }
      }
      __syncthreads();
      // warp item (row, kind, 64 channels): clip, group extremes, scale, zero, codes
      for (int it = warp; it < rows * 4; it += kThreads / 32) {
        const int r = it >> 2, kind = (it >> 1) & 1, c = 64 * (it & 1) + lane;
        const float clip = (kind ? p.clip_V : p.clip_K)[h];
        float x[2], mn[2], mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = sm.red[r][kind][0][c + 32 * e] + sm.red[r][kind][1][c + 32 * e];
          x[e] = fminf(fmaxf(v, -clip), clip);
          mn[e] = mx[e] = x[e];
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
          }
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
      for (int r = tid >> 7; r < rows; r += kThreads / 128) {
        const int role = tid & 127;
        if (role < 72) {
          const int64_t pos = E + i0 + r, pidx = pos / kPage;
          const int id = pidx < p.pt_stride ? p.page_table[(size_t)b * p.pt_stride + pidx] : -1;
          if (id >= 0 && id < p.num_pages)
            store_token_block(p.pool + ((size_t)id * Hkv + h) * block_bytes(ng), (int)(pos % kPage), role, ng, sm.codes[r],
                              sm.meta[r]);
          else if (role == 0)
            atomicOr(p.err_flags, OSCAR_FLAG_BAD_PAGE_ID);
        }
      }
      __syncthreads();
    }
    // every ring entry that leaves has been read: the new rows take their places
    for (int i = tid; i < n * 32; i += kThreads) {
      const int j = i >> 5, kind = (i >> 4) & 1, c = 8 * (i & 15);
      const int64_t pos = L + j;
      if (pos < S || pos >= E2) {
        const size_t slot = pos < S ? pos : S + pos % W;
        *reinterpret_cast<uint4*>(win + (kind * slots + slot) * kHeadDim + c) = *reinterpret_cast<const uint4*>(
            (kind ? p.v : p.k) + (((size_t)b * p.nodes + sm.path[j]) * Hkv + h) * kHeadDim + c);
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
  int nx = num_sms / p.num_kv_heads;   // one CTA per SM
  nx = nx < 1 ? 1 : (nx > p.batch ? p.batch : nx);
  const cudaError_t e = launch_pdl(oscar_commit_draft_kernel, dim3((unsigned)nx, (unsigned)p.num_kv_heads), dim3(kThreads),
                                   sizeof(CommitSmem), s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace oscar
