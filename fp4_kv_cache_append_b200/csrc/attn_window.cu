// Sliding-window attention with sinks, resident form: windows whose rows, for
// all the queries of 128 flattened (query, head) rows, fit shared memory.
// DeepSeek-V4.1-Flash (jaehun.me review), "새로운 접근법" and its flowchart:
// layers 1-2 use sliding-window attention only.
//   out = sum_k softmax_k(scale q . x_k) x_k over the window's tokens and the
//   first tokens before it, K = V shared by the heads.
//
// A block walks over consecutive row tiles of a sequence and keeps the window's
// rows as a bf16 ring in shared memory (E4M3 is exact in bf16; slot = token mod
// ring size: the order of keys does not matter, a row's visible slots are a bit
// mask), so each window row is fetched and converted once per block, not once
// per query, and Q goes from memory to the tensor core by TMA as it is.  All
// keys of a tile are in one S = Q K^T (M 128, N = ring), so the softmax needs no
// running maximum and O no rescaling.  P is split into two bf16 terms (their sum
// is within 2^-17 of P): O = P V takes twice the products, which the tensor
// cores have to spare, instead of a conversion of Q, which the other warps have
// not.  O is formed 64 channels at a time in a three-deep ring of
// tensor-memory columns and stored as it is formed.  What is left is the traffic
// of q and the output, 4 bytes per (row, channel): 132 FLOP per byte at a window
// of 128 and D 512.
// 8,192 tokens of 64 heads, D 512, window 128 and 4 sinks: 223 to 244 us alone =
// 4.4 to 4.8 TB/s (164 us of traffic at the copy rate), tensor core 48% busy; 270
// to 288 us in a long loop, where the power limit holds the SMs near 1.35 GHz.
// With P in one term the loop takes 248 us, at 2^-9 instead of 2^-17 of P.
// Warp roles, all persistent, handing work over through mbarriers:
//   warps 0-3, 4-7    softmax, one row per thread, each group half of the keys
//                (they exchange the row maxima); P replaces S in tensor memory
//   warps 8-11, 12-15  O / l -> bf16 -> output, every other 64-channel block each,
//                through a per-warp staging tile so that whole sectors are stored
//   warps 16, 18 tcgen05.mma issuers of S and of O (one lane each)
//   warp 17      TMA loads of Q, 64 channels at a time
//   warp 19      scheduler: passes (below) through a ring of three descriptors, and
//                the new window rows into the ring (a whole window, when the ring
//                starts anew, by the softmax and output warps too)
// The three stages of a pass (S, softmax, O) each take about as long as q and the
// output take from and to memory; two S buffers keep two passes in flight.
// A pass is a row tile with the range of tokens it needs; a tile whose queries'
// windows do not fit one range (positions far apart) takes several passes, each
// storing the rows it covers.  Sinks and window rows enter unscaled; with y =
// log2 of a weight times its key's scale, P = 2^(y - max y) and the sum of the
// weights is sum(P of sinks) / s_sink + sum(P of window) / s_window.
// Every wait is bounded: one that gives up flags the device status and stops
// every role; issued MMAs and copies are drained and TMEM freed before the block
// exits.
#include "attn_dense.cuh"
#include "kernels_paged.h"

namespace csa2 {

namespace {

constexpr int kEpiWarp0 = 8, kMmaWarp = 16, kQWarp = 17, kPvWarp = 18, kSchedWarp = 19;
constexpr int kThreads = 20 * 32;
constexpr int kColdWarps = 17;               // warps that bring a whole window's rows
// Registers per thread of the warpgroups (2 x softmax, 2 x output, MMA); their
// sum is at most the launch's 5 x 96.
constexpr int kRegsSoftmax = 104, kRegsEpi = 88, kRegsMma = 96;
constexpr int kPasses = 3;                   // descriptors
constexpr int kOBufs = 3;                    // ring of 64-channel O blocks
constexpr int kLive = 8;                     // passes that can be unfinished at once (bounded by the rings above)
constexpr uint32_t kTmemCols = 512;

// Most keys that a ring holds (144 KB at D 512); 64-channel chunks of Q in flight.
__host__ __device__ constexpr int ring_keys(int D) { return D == 512 ? 144 : 160; }
__host__ __device__ constexpr int q_slots(int D) { return D == 512 ? 3 : 4; }

struct Pass {
  int more;                // 0: no further pass
  int row0, nrows, b;
  int q0, nq;
  int end;                 // the covered queries see tokens below this one
  int from;                // queries before this token were covered by an earlier pass of the tile
  int first;               // first pass of the tile (it also covers padded queries)
  int load_lo;             // window rows [load_lo, end) enter the ring
  int load_sinks;          // a new sequence: its sinks enter too
  int wait_for;            // passes that must be complete before the rows enter
  int cold;                // > 0: the ring starts anew (the how-manieth time), all warps bring rows
  int pos[kMaxQ];
};

template <int D>
struct WinSmem {
  static constexpr int QSL = q_slots(D);
  alignas(1024) uint8_t kr[(D / 64) * ring_keys(D) * 128];     // ring: chunks of [R keys x 128 B]
  alignas(1024) uint8_t q[QSL][kRows * 128];        // Q chunks
  alignas(16) uint8_t stage[8][32 * 64];            // per output warp: 32 rows x 32 channels bf16
  float top[2][2][kRows];                           // row maxima of the two halves of the keys, by pass parity
  float lsum[4][2][kRows];                          // sums of the halves, negative: row not covered
  uint64_t q_full[QSL], q_empty[QSL], k_full[4], k_cold, s_full[2], top_full[2], p_full[2], pv_done[2];
  uint64_t o_full[kOBufs], o_empty[kOBufs], pass_full[kPasses], pass_empty[kPasses], fin;
  uint32_t tmem_base;
  int abort;
  int passes_done;                                  // complete O products
  Pass pass[kPasses];
};

// TMEM columns: S of two passes (each later its P), then the O ring
constexpr uint32_t kSCols = 160, kColS = 0, kColO = 2 * kSCols;
static_assert(kColO + kOBufs * 64 <= kTmemCols, "tensor memory");


// E4M3 bytes with the NaN codes (0x7F, 0xFF) made zero: rows between two
// queries' windows may never have been written.
__device__ __forceinline__ uint32_t no_nan(uint32_t w) {
  const uint32_t m = (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
  return w & ~(m * 0xFFu);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_window_kernel(const DenseAttnArgs a, const int rt_own, const int R,
                                                                  const __grid_constant__ CUtensorMap q_map) {
  constexpr int QSL = q_slots(D), NCH = D / 64;
  const uint32_t id_s = mma_idesc(kRows, R, 1u, 1u);   // N = R keys, a multiple of 16
  constexpr uint32_t kIdO = mma_idesc(kRows, 64, 1u, 1u) | (1u << 16);   // B (V) MN-major
  extern __shared__ uint8_t smem_raw[];
  WinSmem<D> &S = *reinterpret_cast<WinSmem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int *abort = &S.abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_sink = a.n_sink, rw = R - n_sink > 0 ? R - n_sink : 1;   // ring: slots [0, n_sink) sinks, then token mod rw
  if (tid == 0) {
    for (int i = 0; i < QSL; ++i) { mbar_init(&S.q_full[i], 1); mbar_init(&S.q_empty[i], 1); }
    for (int i = 0; i < 4; ++i) mbar_init(&S.k_full[i], 1);
    mbar_init(&S.k_cold, kColdWarps);
    for (int i = 0; i < 2; ++i) { mbar_init(&S.s_full[i], 1); mbar_init(&S.top_full[i], 8); mbar_init(&S.p_full[i], 8); mbar_init(&S.pv_done[i], 1); }
    for (int i = 0; i < kOBufs; ++i) { mbar_init(&S.o_full[i], 1); mbar_init(&S.o_empty[i], 4); }
    // readers of a descriptor: softmax and output warps, S, O, Q
    for (int i = 0; i < kPasses; ++i) { mbar_init(&S.pass_full[i], 1); mbar_init(&S.pass_empty[i], 8 + 8 + 3); }
    mbar_init(&S.fin, 2);
    S.abort = 0;
    S.passes_done = 0;
    fence_barrier_init();
    prefetch_tmap(&q_map);
  }
  // slots that no row has entered hold zeros
  for (int i = tid; i < NCH * R * 8; i += kThreads) reinterpret_cast<uint4 *>(S.kr)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (warp == kMmaWarp) {
    tmem_alloc(&S.tmem_base, kTmemCols);
    tmem_relinquish();
    pdl_launch_dependents();   // behind the allocation: a dependent on this SM that allocated first would wait for this grid
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  pdl_wait();

  // this pass's descriptor; every role takes all passes in order
  uint32_t pi = 0;
  auto next_pass = [&]() -> bool {
    const bool w_ok = __all_sync(0xffffffffu, wait_or_abort(&S.pass_full[pi % kPasses], (pi / kPasses) & 1u, abort)) != 0;
    __syncwarp();   // (as in all_wait)
    return w_ok && S.pass[pi % kPasses].more != 0;
  };
  auto free_pass = [&]() {   // the descriptor is not needed any more (one arrival per warp)
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.pass_empty[pi % kPasses]);
  };
  // The rows that enter the ring for a pass: this warp's share (w of nw).
  auto bring_rows = [&](const Pass &ps, int w, int nw, uint64_t *bar) {
    constexpr int LPK = D / 16, RPI = 32 / LPK;       // lanes per window row (16 bytes each), rows per warp access
    constexpr int BATCH = 8;                          // accesses in flight
    const int kl = lane % LPK, kr = lane / LPK, b = ps.b;
    auto put_row = [&](int slot, uint4 v) {           // 16 channels of a key into the ring
      uint32_t h[8];
      e4m3x4_to_f16x2(no_nan(v.x), h);
      e4m3x4_to_f16x2(no_nan(v.y), h + 2);
      e4m3x4_to_f16x2(no_nan(v.z), h + 4);
      e4m3x4_to_f16x2(no_nan(v.w), h + 6);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        const __nv_bfloat162 v2 = __floats2bfloat162_rn(f.x, f.y);
        h[j] = *reinterpret_cast<const uint32_t *>(&v2);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint4 *>(S.kr + sw_off(slot, 2 * kl + j, R)) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
    };
    if (ps.load_sinks) {
#pragma unroll 1
      for (int s = w * RPI + kr; s < n_sink; s += nw * RPI)
        put_row(s, __ldg(reinterpret_cast<const uint4 *>(a.sink_rows + ((size_t)b * a.sink_cap + s) * D) + kl));
    }
    // token t: row t mod W_cap of the sequence, slot t mod rw of the ring, both advanced without dividing again
    int t = ps.load_lo + w * RPI + kr;
    const int step = nw * RPI;
    if (t < ps.end) {
      int src = t % a.W_cap, slot = t % rw;
      const int src_step = step % a.W_cap, slot_step = step % rw;
      const uint4 *base = reinterpret_cast<const uint4 *>(a.swa_rows + (size_t)b * a.W_cap * D) + kl;
#pragma unroll 1
      while (t < ps.end) {
        uint4 v[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          v[u] = t + u * step < ps.end ? __ldg(base + (size_t)src * (D / 16)) : make_uint4(0, 0, 0, 0);
          src += src_step;
          if (src >= a.W_cap) src -= a.W_cap;
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          if (t < ps.end) put_row(n_sink + slot, v[u]);
          t += step;
          slot += slot_step;
          if (slot >= rw) slot -= rw;
        }
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // Until `n` passes are complete (their O products: nothing reads their keys any more).
  auto wait_done = [&](int n) -> bool {
    const volatile int *done = &S.passes_done;
    for (uint32_t i = 0; n > 0 && *done < n; ++i) {   // (all lanes: see all_wait)
      if (i >= kWaitLimit || *abort) {
        *abort = 1;
        return false;
      }
      __nanosleep(64);
    }
    return true;
  };
  // A converged warp's wait, polled by all its lanes: one that lane 0 polls for
  // the others leaves it behind at times, and the tcgen05 instructions that
  // follow have to be met by all lanes at once.
  auto all_wait = [&](uint64_t *bar, uint32_t parity) {
    const bool w_ok = __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort)) != 0;
    __syncwarp();
    return w_ok;
  };

  if (warp < kEpiWarp0) {
    // ================================================ softmax: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int q = warp & 3, part = warp >> 2, row = 32 * q + lane;
    const uint32_t lrow = tmem + ((uint32_t)(32 * q) << 16);
    // y = log2(weight x key scale) = S x l + o, with the sign of the softmax
    // scale taken into S and the factor never 0, so that a hidden key's -inf stays
    // (nor so small that o, at most 280 / factor, leaves fp32)
    const float s_win = a.window > 0 ? a.s_swa : a.s_sink, s_snk = n_sink > 0 ? a.s_sink : s_win;
    const float lw = fmaxf(fabsf(a.scale) * s_win * kLog2e, 1e-36f), ls = fabsf(a.scale) * s_snk * kLog2e;
    const float rs_w = 1.f / s_win, rs_s = 1.f / s_snk;
    const float s2w = ls / lw, o2w = (log2f(s_snk) - log2f(s_win)) / lw;   // a sink's S as a window row's of the same y
    bool ok = true;
    while (ok && next_pass()) {
      const Pass &ps = S.pass[pi % kPasses];
      if (ps.cold) {
        ok = wait_done(ps.wait_for);
        if (!ok) break;
        bring_rows(ps, warp, kColdWarps, &S.k_cold);
      }
      const int frow = ps.row0 + row;
      const bool live = row < ps.nrows;
      const int t = live ? ps.pos[frow / a.H - ps.q0] : -1;
      // covered by this pass: its window ends in [from, end), so no earlier pass covered it
      const bool mine = live && (t < 0 ? ps.first != 0 : (t >= ps.from && t < ps.end));
      // the slots this row sees, one bit per key
      int wlo = a.window > 0 ? t - a.window + 1 : t + 1;
      if (wlo < 0) wlo = 0;
      const int NW = (R + 31) / 32;
      const int len = mine && t >= 0 && a.window > 0 ? t - wlo + 1 : 0;
      const int s0 = n_sink + wlo % rw, e0 = s0 + len;              // [s0, e0), wrapping from R to n_sink
      const int e1 = e0 < R ? e0 : R, w1 = e0 > R ? n_sink + e0 - R : n_sink;
      const int ns = mine && t >= 0 ? (n_sink < wlo ? n_sink : wlo) : 0;
      auto span = [&](int w, int lo, int hi) -> uint32_t {          // bits [lo, hi) of word w
        lo -= 32 * w; hi -= 32 * w;
        lo = lo < 0 ? 0 : lo; hi = hi > 32 ? 32 : hi;
        return hi > lo ? (0xFFFFFFFFu >> (32 - (hi - lo))) << lo : 0u;
      };
      auto seen_word = [&](int w) -> uint32_t { return span(w, s0, e1) | span(w, n_sink, w1) | span(w, 0, ns); };
      const uint32_t buf = pi & 1u, scol = lrow + kColS + buf * kSCols;
      ok = all_wait(&S.s_full[buf], (pi >> 1) & 1u);
      if (!ok) break;
      tc_fence_after();
      // words of 32 keys, [w0, w0 + nw) by this warp; S is read twice (the
      // code of a word is a loop's body: straight-line code for all of them is
      // fetched from L2 every pass).  What a last word of 16 reads behind the
      // ring's keys has no bit set.
      const int HALF = (NW + 1) / 2;
      const int w0 = part * HALF, w_end = part ? NW : HALF;
      auto hide = [&](uint32_t seen, uint32_t *x) {
        if (!__all_sync(0xffffffffu, seen == 0xFFFFFFFFu)) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((seen >> j) & 1u)) x[j] = 0xFF800000u;
        }
      };
      auto logits = [&](int w, uint32_t *x) {   // a row's S of word w, to be multiplied by lw; hidden: -inf
        tmem_ld_x32(scol + 32 * w, x);
        const uint32_t seen = seen_word(w), sinks = span(w, 0, n_sink);
        tmem_wait_ld();
        if (a.scale < 0.f) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] ^= 0x80000000u;
        }
        if (sinks) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if ((sinks >> j) & 1u) x[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), s2w, o2w));
        }
        hide(seen, x);
        return sinks;
      };
      float top = -INFINITY;
#pragma unroll 1
      for (int w = w0; w < w_end; ++w) {
        uint32_t x[32];
        logits(w, x);
        float m4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m4[j] = __uint_as_float(x[j]);
#pragma unroll
        for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(x[j]));
        top = fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
      }
      S.top[buf][part][row] = top;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.top_full[buf]);
      ok = all_wait(&S.top_full[buf], (pi >> 1) & 1u);
      if (!ok) break;
      top = fmaxf(top, S.top[buf][part ^ 1][row]);
      // P = 2^(y - max y) = hi + lo, in place (columns [0, 16) and [16, 32) of
      // the word's 32), and the sums of the two sorts of keys
      const float mu = top == -INFINITY ? 0.f : top * lw;
      float sum_s = 0.f;
      uint64_t sum2 = 0;
      const uint64_t l2 = f32x2(lw, lw), m2 = f32x2(-mu, -mu);
#pragma unroll 1
      for (int w = w0; w < w_end; ++w) {
        uint32_t x[32], pr[32];
        const uint32_t sinks = logits(w, x);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 y = unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), l2, m2));
          const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
          x[j] = __float_as_uint(p0);
          x[j + 1] = __float_as_uint(p1);
          const __nv_bfloat162 hv = __floats2bfloat162_rn(p0, p1);
          const uint32_t hi = *reinterpret_cast<const uint32_t *>(&hv);
          const __nv_bfloat162 lv = __floats2bfloat162_rn(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u));
          pr[j / 2] = hi;
          pr[16 + j / 2] = *reinterpret_cast<const uint32_t *>(&lv);
        }
        tmem_st_x32(scol + 32 * w, pr);
        if (sinks) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const bool k = (sinks >> j) & 1u;
            sum_s += k ? __uint_as_float(x[j]) : 0.f;
            x[j] = k ? 0u : x[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2) sum2 = add_f32x2(sum2, f32x2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
      }
      const float2 st2 = unpack_f32x2(sum2);
      S.lsum[pi & 3u][part][row] = mine ? sum_s * rs_s + (st2.x + st2.y) * rs_w : -1.f;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[buf]);
      free_pass();
      ++pi;
    }
  } else if (warp < kMmaWarp) {
    // ================================================ output
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const int q = warp & 3;
    const uint32_t lrow = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t part = (warp - kEpiWarp0) >> 2;
    uint8_t *stage = S.stage[warp - kEpiWarp0];
    uint32_t oi = 0;
    bool ok = true;
    while (ok && next_pass()) {
      const int row0 = S.pass[pi % kPasses].row0 + 32 * q;
      if (S.pass[pi % kPasses].cold) {
        ok = wait_done(S.pass[pi % kPasses].wait_for);
        if (!ok) break;
        bring_rows(S.pass[pi % kPasses], warp, kColdWarps, &S.k_cold);
      }
      free_pass();
      ++pi;   // (passes done when this one is)
      float inv = -1.f;
      uint32_t covered = 0;
      oi += part;
#pragma unroll 1
      for (int c = (int)part; c < NCH; c += 2) {
        const uint32_t ob = oi % kOBufs;
        ok = all_wait(&S.o_full[ob], (oi / kOBufs) & 1u);
        if (!ok) break;
        oi += 2;
        tc_fence_after();
        if (c == (int)part) {   // the O product follows the softmax: its sums are there
          const float l0 = S.lsum[(pi - 1) & 3u][0][32 * q + lane], l = l0 + S.lsum[(pi - 1) & 3u][1][32 * q + lane];
          inv = l0 < 0.f ? -1.f : (l > 0.f ? 1.f / l : 0.f);
          covered = __ballot_sync(0xffffffffu, inv >= 0.f);
        }
        uint32_t o[64];
        tmem_ld_x32(lrow + kColO + ob * 64, o);
        tmem_ld_x32(lrow + kColO + ob * 64 + 32, o + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.o_empty[ob]);
          if (c == NCH - 1 && q == 0) *reinterpret_cast<volatile int *>(&S.passes_done) = (int)pi;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // 32 channels: rows through the stage, whole sectors out
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            uint32_t pk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int i = 32 * h + 8 * p + 2 * j;
              const __nv_bfloat162 bv = __floats2bfloat162_rn(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
              pk[j] = *reinterpret_cast<const uint32_t *>(&bv);
            }
            *reinterpret_cast<uint4 *>(stage + lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + lane / 4, p = lane % 4;
            const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((p ^ ((r >> 1) & 3)) << 4));
            if ((covered >> r) & 1u) reinterpret_cast<uint4 *>(a.out + (size_t)(row0 + r) * D + c * 64 + h * 32)[p] = v;
          }
          __syncwarp();
        }
      }
      oi -= part;   // (the pass's blocks are counted by both)
    }
  } else {
    // ================================================ scheduler and window rows, MMA issuers, Q
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kSchedWarp) {
      const int units = a.B * rt_own, rows = a.T_q * a.H;
      const int u_end = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);
      int u = (int)((long long)units * blockIdx.x / gridDim.x);
      int cold = 0;                                    // times that the ring started anew
      int res_b = -1, res_lo = 0, res_hi = 0;          // ring: tokens [res_lo, res_hi) of sequence res_b
      int old[kLive];                                  // first token of the last passes (newest first)
#pragma unroll
      for (int i = 0; i < kLive; ++i) old[i] = INT_MAX;
      bool ok = true;
      while (ok) {
        const bool more = u < u_end;
        const int b = u / rt_own, rt = u % rt_own;
        const int row0 = b * rows + rt * kRows, nrows = rows - rt * kRows < kRows ? rows - rt * kRows : kRows;
        int from = 0, first = 1;                       // passes of this tile
        do {
          Pass &ps = S.pass[pi % kPasses];
          ok = all_wait(&S.pass_empty[pi % kPasses], ((pi / kPasses) & 1u) ^ 1u);
          if (!ok) break;
          if (!more) {
            if (lane == 0) ps.more = 0;
          } else {
            const int q0 = row0 / a.H, nq = (row0 + nrows - 1) / a.H - q0 + 1;
            int lo = INT_MAX;
            for (int i = lane; i < nq; i += 32) {
              int t = __ldg(a.q_pos + q0 + i);
              if (t > kMaxPos) {
                flag(a.status, CSA2_DEV_BAD_POSITION);
                t = -1;
              }
              ps.pos[i] = t;
              if (t >= from && t >= 0) {
                int l = a.window > 0 ? t - a.window + 1 : t + 1;
                l = l < 0 ? 0 : l;
                lo = l < lo ? l : lo;
              }
            }
            __syncwarp();
            lo = __reduce_min_sync(0xffffffffu, lo);
            // the queries whose windows lie in [lo, lo + rw) (no window: any)
            int end = 0, next = INT_MAX;
            if (lo != INT_MAX) {
              const int lim = a.window > 0 ? lo + rw : INT_MAX;
              for (int i = lane; i < nq; i += 32) {
                const int t = ps.pos[i];
                if (t >= from && t >= 0) {
                  if (t < lim) end = t + 1 > end ? t + 1 : end;
                  else next = t < next ? t : next;
                }
              }
              end = __reduce_max_sync(0xffffffffu, end);
              next = __reduce_min_sync(0xffffffffu, next);
            } else {
              lo = 0;
            }
            // rows that enter: behind what the ring holds, or all of them (padded queries alone: none)
            const bool none = end == 0;
            const bool same = none || (b == res_b && lo >= res_lo && lo <= res_hi);
            int load_lo = same ? (res_hi < end ? res_hi : end) : lo;
            if (a.window <= 0 || none) load_lo = end;
            int wait_for = 0;
            if (!same) {
              wait_for = (int)pi;
              ++cold;
            } else if (end > load_lo) {
              // slots of tokens below end - rw are overwritten: every unfinished pass that needs one of them
#pragma unroll
              for (int i = kLive - 1; i >= 0; --i)
                if (old[i] < end - rw) wait_for = (int)pi - i;
            }
            if (lane == 0) {
              ps.more = 1; ps.row0 = row0; ps.nrows = nrows; ps.b = b; ps.q0 = q0; ps.nq = nq;
              ps.end = end; ps.from = from; ps.first = first;
              ps.load_lo = load_lo; ps.load_sinks = !none && b != res_b; ps.wait_for = wait_for;
              ps.cold = same ? 0 : cold;
            }
#pragma unroll
            for (int i = kLive - 1; i > 0; --i) old[i] = old[i - 1];
            old[0] = end > lo ? lo : INT_MAX;
            if (!same) { res_lo = lo; res_hi = lo; }
            if (!none) {
              res_b = b;
              res_hi = end > res_hi ? end : res_hi;
              if (res_lo < res_hi - rw) res_lo = res_hi - rw;
            }
            from = next == INT_MAX ? INT_MAX : end;
            first = 0;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.pass_full[pi % kPasses]);
          if (more) {
            const Pass &pr = S.pass[pi % kPasses];
            ok = wait_done(pr.wait_for);
            if (!ok) break;
            if (pr.cold) {
              bring_rows(pr, kColdWarps - 1, kColdWarps, &S.k_cold);
              if (lane == 0) mbar_arrive(&S.k_full[pi & 3u]);   // (k_full's phases stay in step with the passes)
            } else {
              bring_rows(pr, 0, 1, &S.k_full[pi & 3u]);
            }
          }
          ++pi;
        } while (more && from != INT_MAX);
        if (!more) break;
        ++u;
      }
    } else if (warp == kMmaWarp) {
      // one lane runs the whole loop, its waits included (a converged warp that
      // elects a lane per group of MMAs issues them at half the rate)
      if (elect_one()) {
        uint32_t qi = 0;
        bool ok = true;
        while (ok) {
          ok = wait_or_abort(&S.pass_full[pi % kPasses], (pi / kPasses) & 1u, abort);
          if (!ok || !S.pass[pi % kPasses].more) break;
          const int cold = S.pass[pi % kPasses].cold;
          mbar_arrive(&S.pass_empty[pi % kPasses]);
          const uint32_t buf = pi & 1u, scol = tmem + kColS + buf * kSCols;
          ok = wait_or_abort(&S.k_full[pi & 3u], (pi >> 2) & 1u, abort);
          if (ok && cold) ok = wait_or_abort(&S.k_cold, (cold - 1) & 1, abort);
          if (ok && pi >= 2) ok = wait_or_abort(&S.pv_done[buf], ((pi >> 1) & 1u) ^ 1u, abort);   // the buffer's last P has been used
          if (!ok) break;
#pragma unroll 1
          for (int c = 0; c < NCH; ++c) {
            const uint32_t slot = qi % QSL;
            ok = wait_or_abort(&S.q_full[slot], (qi / QSL) & 1u, abort);
            if (!ok) break;
            ++qi;
            tc_fence_after();
            const uint64_t da = smem_desc_kmajor(smem_u32(S.q[slot]), 128);
            const uint64_t db = smem_desc_kmajor(smem_u32(S.kr) + c * (R * 128), 128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16(scol, da + ((kk * 32) >> 4), db + ((kk * 32) >> 4), id_s, (c > 0 || kk > 0) ? 1u : 0u);
            tc_commit(&S.q_empty[slot]);
          }
          if (!ok) break;
          tc_commit(&S.s_full[buf]);
          ++pi;
        }
      }
      __syncwarp();
    } else if (warp == kQWarp) {
      if (elect_one()) {
        uint32_t qi = 0;
        bool ok = true;
        while (ok) {
          ok = wait_or_abort(&S.pass_full[pi % kPasses], (pi / kPasses) & 1u, abort);
          if (!ok || !S.pass[pi % kPasses].more) break;
          const int row0 = S.pass[pi % kPasses].row0;
          mbar_arrive(&S.pass_empty[pi % kPasses]);
#pragma unroll 1
          for (int c = 0; c < NCH; ++c) {   // (rows behind the tile's last one are some other rows or zeros: never used)
            const uint32_t slot = qi % QSL;
            ok = wait_or_abort(&S.q_empty[slot], ((qi / QSL) & 1u) ^ 1u, abort);
            if (!ok) break;
            ++qi;
            mbar_arrive_expect_tx(&S.q_full[slot], kRows * 128);
            tma_load_2d(S.q[slot], &q_map, c * 64, row0, &S.q_full[slot]);
          }
          ++pi;
        }
        if (!ok)   // copies in flight land before the block may end
          for (uint32_t i = 1; i <= (uint32_t)QSL && i <= qi; ++i)
            mbar_wait_bounded(&S.q_full[(qi - i) % QSL], ((qi - i) / QSL) & 1u, kWaitLimit);
      }
      __syncwarp();
    } else if (warp == kPvWarp) {
      if (elect_one()) {
        uint32_t oi = 0;
        bool ok = true;
        while (ok) {
          ok = wait_or_abort(&S.pass_full[pi % kPasses], (pi / kPasses) & 1u, abort);
          if (!ok || !S.pass[pi % kPasses].more) break;
          mbar_arrive(&S.pass_empty[pi % kPasses]);
          const uint32_t buf = pi & 1u, pcol = tmem + kColS + buf * kSCols;
          ok = wait_or_abort(&S.p_full[buf], (pi >> 1) & 1u, abort);
          if (!ok) break;
#pragma unroll 1
          for (int c = 0; c < NCH; ++c) {
            const uint32_t ob = oi % kOBufs;
            ok = wait_or_abort(&S.o_empty[ob], ((oi / kOBufs) & 1u) ^ 1u, abort);
            if (!ok) break;
            ++oi;
            tc_fence_after();
            const uint64_t dv = smem_desc_mnmajor_sw128(smem_u32(S.kr) + c * (R * 128), R * 128, 1024);
#pragma unroll 1
            for (int w = 0; 32 * w < R; ++w)   // a word's two steps of 16 keys, hi and lo of each
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (32 * w + 16 * (k / 2) < R)
                  tc_mma_f16_ta(tmem + kColO + ob * 64, pcol + 32 * w + 8 * (k / 2) + 16 * (k % 2),
                                dv + (uint64_t)((w * 4096 + (k / 2) * 2048) >> 4), kIdO, (w > 0 || k > 0) ? 1u : 0u);
            tc_commit(&S.o_full[ob]);
          }
          if (!ok) break;
          tc_commit(&S.pv_done[buf]);
          ++pi;
        }
      }
      __syncwarp();
    }
  }
  // ---- every role is through, or a wait gave up
  const bool dead = __syncthreads_or(*abort != 0) != 0;
  if (dead) {
    if (tid == 0) flag(a.status, CSA2_DEV_TIMEOUT);
    if (warp == kMmaWarp || warp == kPvWarp) {   // every MMA issued so far is done before its memory goes
      if (elect_one()) {
        tc_commit(&S.fin);
        mbar_wait_bounded(&S.fin, 0, kWaitLimit);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Queries that 128 rows can touch.
static int tile_queries(const DenseAttnArgs &a) {
  const int nq = (kRows - 1 + a.H - 1) / a.H + 1;
  return a.T_q < nq ? a.T_q : nq;
}

template <int D>
static cudaError_t launch_t(const CUtensorMap &q_map, const DenseAttnArgs &a, int sms, cudaStream_t s) {
  const size_t smem = sizeof(WinSmem<D>) + 1024;
  static_assert(sizeof(WinSmem<D>) + 1024 <= 232448, "shared memory");
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem_once(attn_window_kernel<D>, smem, &allowed);
  if (e != cudaSuccess) return e;
  const int rt_own = (a.T_q * a.H + kRows - 1) / kRows;
  const long long units = (long long)a.B * rt_own;
  const int grid = units < sms ? (int)units : sms;
  // the keys of a tile, and room for the rows of the next two while a tile's are in use
  const int most = tile_queries(a), need = a.n_sink + (a.window > 0 ? a.window + most - 1 : 0);
  int R = (need + 2 * most + 15) / 16 * 16;
  if (R > ring_keys(D)) R = ring_keys(D);
  return launch_pdl(attn_window_kernel<D>, dim3(grid), dim3(kThreads), smem, s, dim3(1, 1, 1), a, rt_own, R, q_map);
}

// The resident form takes the launches whose windows fit, but for those where a
// sequence is one row tile: no key is met twice there, and the other form, which
// has two blocks for a tile of D 512 and starts sooner, is ahead, unless its
// second block makes a second wave or all keys are one tile of its own.  us,
// resident | other, one token of H heads, window 128 and 4 sinks: B 16 H 64 D 512
// 16.1 | 14.9, B 74 16.6 | 16.5, B 148 19.0 | 29.7, B 512 66.9 | 99.4; H 16 D 256
// B 64 13.9 | 12.0, B 600 54.9 | 47.0 (window of 16: 35.6 | 42.4); H 64 D 128
// B 148 13.2 | 11.0, B 1,000 66.4 | 55.4.  Chunks of tokens: 8 x 8, H 64 D 512
// 16.6 | 17.7; 64 x 4 18.8 | 33.1; 1 x 8,192 228 | 796.  (Where it does not hold:
// few heads of D 128, 1 x 8,192, H 8 39.9 | 36.4 and 1 x 1,024 14.2 | 10.7.)
bool window_takes_ring(const DenseAttnArgs &a, int sms) {
  const int keys = a.n_sink + (a.window > 0 ? a.window + tile_queries(a) - 1 : 0);
  if (keys > ring_keys(a.D)) return false;
  const bool one_tile = a.T_q * a.H <= kRows, one_wave = a.D < 512 || 2 * a.B <= sms;
  return !(one_tile && one_wave && keys > 64);
}

cudaError_t launch_window_ring(const CUtensorMap &q_map, const DenseAttnArgs &a, int sms, cudaStream_t s) {
  switch (a.D) {
    case 128: return launch_t<128>(q_map, a, sms, s);
    case 256: return launch_t<256>(q_map, a, sms, s);
    default: return launch_t<512>(q_map, a, sms, s);
  }
}

}  // namespace csa2
