// Dense attentions: all entries of paged FP4 sequences, and the sliding
// window with its first tokens.  One softmax per (query, head) over every
// visible key, K = V shared by the heads.
//
// First form: a block per (query, 8 heads), one warp per head; the block's
// keys are dequantised to fp32 tiles of 32 in shared memory, lane = key for
// the logits and lane = channel for the values, with the running maximum and
// sum of the softmax in registers.
#include "common.cuh"
#include "kernels.h"

namespace csa2 {

namespace {

constexpr int kWarps = 8;
constexpr int kKeys = 32;

// Row of the pool's planes that holds entry e of pool sequence s, or -1.
__device__ __forceinline__ int pool_slot(const DenseAttnArgs &a, int s, int e) {
  const int pg = a.pool.table[(size_t)s * a.pool.max_pages + e / a.pool.page];
  if (pg < 0 || pg >= a.pool.n_pages) {
    flag(a.status, CSA2_DEV_INDEX_RANGE);
    return -1;
  }
  return pg * a.pool.page + e % a.pool.page;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_dense_simple_kernel(const DenseAttnArgs a) {
  extern __shared__ float sm[];
  float *kt = sm;                       // [32][D + 1]
  float *qs = sm + kKeys * (D + 1);     // [8][D]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, b = row / a.T_q, h = blockIdx.y * kWarps + warp;
  pdl_launch_dependents();
  pdl_wait();
  const int t = a.q_pos[row];
  for (int c = lane; c < D; c += 32)
    qs[warp * D + c] = h < a.H ? bf16_to_f32(a.q[((size_t)row * a.H + h) * D + c]) * a.scale : 0.f;
  float o[D / 32];
#pragma unroll
  for (int u = 0; u < D / 32; ++u) o[u] = 0.f;
  float m = -INFINITY, l = 0.f;

  int n_ent = 0, s = -1;
  if (a.pool.codes && t >= 0) {
    s = a.seq[b];
    if (s < 0 || s >= a.pool.n_seq) {
      flag(a.status, CSA2_DEV_BAD_SEQUENCE);
    } else {
      n_ent = a.pool.n_entries[s];
      const int vis = (t + 1) / a.pool.m, room = a.pool.max_pages * a.pool.page;
      n_ent = n_ent < vis ? n_ent : vis;
      n_ent = n_ent < room ? n_ent : room;
    }
  }
  const int s0 = a.pool.codes ? a.seq[0] : -1;
  int wlo = t - a.window + 1;
  if (wlo < 0) wlo = 0;
  const int n_win = a.swa_rows && a.window > 0 && t >= 0 ? t - wlo + 1 : 0;
  const int n_snk = a.sink_rows && t >= 0 ? (a.n_sink < wlo ? a.n_sink : wlo) : 0;
  const int total = n_ent + n_snk + n_win;

  for (int k0 = 0; k0 < total; k0 += kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * (D / 16); i += kWarps * 32) {   // 16 channels of a key per item
      const int r = i / (D / 16), g = i % (D / 16), k = k0 + r;
      float v[16];
      bool have = false;
      if (k < n_ent) {
        const int sq = k < a.n_shared && s0 >= 0 && s0 < a.pool.n_seq ? s0 : s;
        const int at = pool_slot(a, sq, k);
        if (at >= 0) {
          have = true;
          const float sc = e4m3_to_f32(a.pool.scales[(size_t)at * (D / 16) + g]);
          const uint2 w = *reinterpret_cast<const uint2 *>(a.pool.codes + (size_t)at * (D / 2) + 8 * g);
#pragma unroll
          for (int u = 0; u < 16; ++u) v[u] = e2m1_to_f32(((u < 8 ? w.x : w.y) >> (4 * (u & 7))) & 15u) * sc;
        }
      } else if (k < total) {
        have = true;
        const bool snk = k < n_ent + n_snk;
        const uint8_t *p = snk ? a.sink_rows + ((size_t)b * a.sink_cap + (k - n_ent)) * D
                               : a.swa_rows + ((size_t)b * a.W_cap + (wlo + k - n_ent - n_snk) % a.W_cap) * D;
        const float sc = snk ? a.s_sink : a.s_swa;
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = e4m3_to_f32(p[16 * g + u]) * sc;
      }
      float *dst = kt + r * (D + 1);
#pragma unroll
      for (int u = 0; u < 16; ++u) dst[16 * g + u] = have ? v[u] : (u == 0 && g == 0 ? NAN : 0.f);
    }
    __syncthreads();
    float x = 0.f;
    const float *kr = kt + lane * (D + 1);
#pragma unroll 8
    for (int c = 0; c < D; ++c) x = fmaf(qs[warp * D + c], kr[c], x);
    const bool ok = k0 + lane < total && kr[0] == kr[0];
    x = ok ? x : -INFINITY;
    float mx = x;
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float al = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = ok ? expf(x - mn) : 0.f;
    float ps = p;
    for (int w = 16; w > 0; w >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, w);
    l = l * al + ps;
    m = mn;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) o[u] *= al;
    for (int k = 0; k < kKeys; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      if (pk == 0.f) continue;
#pragma unroll
      for (int u = 0; u < D / 32; ++u) o[u] = fmaf(pk, kt[k * (D + 1) + lane + 32 * u], o[u]);
    }
  }
  if (h < a.H) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const __nv_bfloat16 v = __float2bfloat16_rn(o[u] * inv);
      a.out[((size_t)row * a.H + h) * D + lane + 32 * u] = *reinterpret_cast<const uint16_t *>(&v);
    }
  }
}

template <int D>
cudaError_t launch_simple(const DenseAttnArgs &a, cudaStream_t s) {
  const size_t smem = (size_t)(kKeys * (D + 1) + kWarps * D) * 4;
  cudaError_t e = cudaFuncSetAttribute(attn_dense_simple_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_dense_simple_kernel<D>, dim3(a.B * a.T_q, (a.H + kWarps - 1) / kWarps), dim3(kWarps * 32), smem,
                    s, dim3(1, 1, 1), a);
}

cudaError_t launch_simple_d(const DenseAttnArgs &a, cudaStream_t s) {
  switch (a.D) {
    case 128: return launch_simple<128>(a, s);
    case 256: return launch_simple<256>(a, s);
    default: return launch_simple<512>(a, s);
  }
}

}  // namespace

size_t prefix_attn_workspace_bytes(int, int, int, int, int) { return 0; }
size_t window_attn_workspace_bytes(int, int, int, int, int, int, int) { return 0; }
cudaError_t launch_prefix_attn(const DenseAttnArgs &a, int, cudaStream_t s) { return launch_simple_d(a, s); }
cudaError_t launch_window_attn(const DenseAttnArgs &a, int, cudaStream_t s) { return launch_simple_d(a, s); }

}  // namespace csa2
