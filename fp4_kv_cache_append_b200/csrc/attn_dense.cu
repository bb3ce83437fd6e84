// Dense attentions: all entries of paged FP4 sequences (a prefix that the
// batch shares computed once), and the sliding window with its first tokens.
// One softmax per (query, head) over every visible key, K = V shared by the
// heads:  out = sum_k softmax_k(scale q . x_k) x_k.
//
// Because all heads (and, over a shared prefix, all sequences) meet the same
// keys, 128 flattened (query, head) rows form the M of the matrix products
// whatever their number of heads: S = Q K^T (M 128, N 64 keys, K 16 x D / 16)
// and O += P V (M 128, N up to 256 channels).  For D = 512 the O of 128 rows
// fills the tensor memory, so two blocks take 256 channels each and both form
// S.
//
// One persistent block per SM; keys in tiles of 64.  Warp roles, handing work
// over through mbarriers:
//   warp 13     loads: Q of the unit; then, by tensor copies, the raw bytes of a
//               step (256 channels of a tile's FP4 codes and scales, page by page,
//               or 128 of its FP8 rows) into one of three stages
//   warps 0-7   dequantise, exactly, to fp16 into a ring of chunk groups
//               (64-channel chunks, K-major, 128B swizzle); two teams of four
//               warps take the groups in turn.  The chunks that only S needs
//               come first and are freed first
//   warps 8-11  softmax, one row per thread: no exchange between threads.  The
//               reference, 2^9 below the maximum, moves only when a weight
//               passes 2^15.9 against it; O is then rescaled in tensor memory.  P
//               goes back to tensor memory (fp16) as the A operand of the second
//               product
//   warps 12, 14  tcgen05.mma issuers of S and of O, one lane each: S of tile
//               i + 1 runs during tile i's softmax, O of tile i as soon as its P
//               is there
//   warp 15     writes the next segment (see below) while this one runs
// Q lands as bf16 (its first chunks in the ring's last groups, the rest in place)
// and is converted by the softmax and the dequantising warps to fp16, each row
// times a power of two that the logits' factor takes back: 2^6 where the row's
// largest element lies in [2^-8, 2^9), else the one that brings it to [2^14,
// 2^15), so that rounding moves an element by 2^-23 of the row's largest at most.
// That one is found in the same pass; rows that need another power are converted
// a second time.  (A single token's 15.2 us at D 512 without any of it, 15.7 so,
// 16.1 with the largest found in a pass of its own.)  Up to four chunks
// of Q (256 channels) go to tensor memory as the A operand, the rest stays in
// shared memory: a K step of 16 with Q in tensor memory takes 33 cycles, with Q
// in shared memory 49 (128 rows of A and 64 of B are read), and the room it
// leaves holds the stages and a fourth ring group (with three, the fetch of a
// tile waits for the O product of the tile two before it).  S has two buffers;
// P replaces its tile's S.
// Rows are given by unit (128 rows x a list of keys); a unit's key list is
// split over blocks wherever the even division of all tiles over the SMs cuts
// it, each part leaving (O, max, sum) in the workspace for a merge kernel.
// Window rows enter unscaled: their scale multiplies the logits, and O is
// converted once where the key list changes from one scale to another.
// Each role runs its own loop over the block's segments and meets the others
// at named barriers, so that the registers can be divided between the roles.
// Every wait is bounded: one that gives up flags the device status and stops
// every role; issued MMAs and copies are drained and TMEM freed before the block
// exits.
//
// What bounds it (D 512, H 64, 32 sequences of one token, 65,536 shared entries
// and 512 to 1,024 own ones: 320 to 335 us alone, 363 to 375 us in a long loop,
// where the power limit holds the SMs near 1.6 GHz; 755 TFLOP/s of the 4 D FLOP
// per row and key): shared memory.  A tile of 64 keys and a channel half moves 260 KB through
// it (S with Q in shared memory 96, in tensor memory 32, O 32, the fp16 keys
// written 64, the raw bytes in and out 36; the bank counters say the same): 2,030
// cycles at the 128 bytes a cycle that the S product reaches, of 2,350 measured;
// the tensor core is busy for 1,830 of them.  For D 128 and 256 all of Q is in
// tensor memory and the softmax's own chain (about 1,650 cycles a tile: 64
// exponentials on a scheduler's pipe take 512) is the longest: the same case at D
// 256 takes 129 us (1,080 TFLOP/s), with 32 heads of D 128 71 us.
// Loads with a copy instruction per 16 bytes (cp.async) took 2,560 cycles of the
// loading warp per tile, more than the tile itself: 424 us against 384 us then.
// A softmax split over two threads per row halves its arithmetic but has them
// exchange maxima through shared memory in every tile: 440 us against 384 us
// then, and at D 256, where no S operand of Q is read beside it, 193 us against
// 138 us then.
#include "attn_dense.cuh"
#include "kernels_paged.h"

namespace csa2 {

namespace {

constexpr int kDqWarps = 8;
constexpr int kDq = kDqWarps * 32, kTeam = kDqWarps / 2;   // dequantise threads; warps of a team
constexpr int kSmWarp0 = 8;                  // softmax warps 8..11
constexpr int kMmaWarp = 12;
constexpr int kTile = 64;                    // keys per tile
constexpr int kThreads = 16 * 32;            // four warpgroups: registers are split between them
// Named barriers: a segment's start and end (all threads); Q in place (arrivals of
// the softmax and dequantising warps, awaited by the issuer of S); the largest
// elements of Q's rows (of the softmax and dequantising warps).
constexpr int kSegBar = 1, kQBar = 2, kQTopBar = 3;
constexpr int kSchedWarp = 15;               // writes the next segment
// Registers per thread of the warpgroups: 2 x fetch, softmax, MMA (a tile's
// logits stay in registers; what is spilled goes to L2, since shared memory takes
// all of the L1's room: at D 128 and in the paged D 512 kernel one word a thread,
// written once and read in four or five places).  Their sum is at most the
// launch's 4 x 128.
constexpr int kRegsFetch = 88, kRegsSoftmax = 208, kRegsMma = 128;
constexpr int kLoadWarp = 13;                // loader
constexpr int kPvWarp = 14;                  // MMA issuer of O (kMmaWarp: of S)
constexpr int kStages = 3;                   // raw steps in flight or in use
// A stage: 64 rows of 128 bytes (codes, 64 bytes for D 128, or FP8 values),
// then 64 rows of scales (16 bytes, 8 for D 128).
constexpr int kRawRow = 128, kRawSc = kTile * kRawRow, kRawBytes = kRawSc + kTile * 16;
// A unit's start and end in tiles (see Schedule::ov), fitted at D 512: the case
// above takes 427 us with 2, 363 with 5, 343 with 8, 345 with 10 and 349 with 16.
// (At D 128 and 256, where a tile takes less, it was not fitted.)
constexpr int kUnitCost = 8;
// P = 2^(x - reference), where the reference is set kBias below the largest x so
// far once P would pass 2^(kBias + kLazy) = 61,147 (fp16 ends at 65,504).  The
// row's largest weight is then at least 2^9, weights down to 2^-23 of it keep
// fp16's 11 bits and none above 2^-34 of it becomes 0, while the
// denominator sums all of them in fp32: n keys lose at most n 2^-34 of the row's
// weight.  (Without the bias n 2^-25: one key 17 nats above a million equal ones
// took 3% from the output.)  A lower limit moves the reference more often: a
// window of 333 at D 256 takes 30.6 us with limits of 15 and 6.9, 30.8 with 7
// and a bias of 8, 31.2 with 5.9 and 10.
constexpr float kBias = 9.0f, kLazy = 6.9f;
// TMEM columns: O, S of two tiles (each later its P), Q's first chunks
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 384, kTmemCols = 512;

template <int D>
struct Cfg {
  static constexpr int DO = D < 256 ? D : 256;           // output channels of a block
  static constexpr int CS = D / DO;                      // blocks that share a unit's channels
  static constexpr int NCH = D / 64;                     // 64-channel chunks of a key
  static constexpr int GC = DO / 64;                     // chunks of a ring group
  static constexpr int NG = D == 128 ? 8 : 4;             // ring groups
  static constexpr int QT = NCH < 4 ? NCH : 4;           // chunks of Q in tensor memory, the first in S's order
  static constexpr int QS = NCH - QT;                    // ... in shared memory
  static constexpr int CB = DO / 2, SB = DO / 16;        // bytes of codes and of scales of a key in a step
};

// What a block does next: a part of a unit's key list.
struct Segment {
  int half;                // channel half
  int b;                   // batch row of the window rows (0 over the shared prefix)
  int row0;                // first flattened row
  int nrows;
  int n_sink, n_fp4, n_win;   // tiles of each sort, in this order
  int key0;                // first entry of the first FP4 tile
  int key_lo, key_end;     // entries below and from here on count as zeros
  int seq;                 // pool sequence whose table is read (-1: none)
  size_t ml_at, o_at;      // partial result's (max, sum) and O in the workspace (bytes)
  int o_rows;              // rows of its planes
  int q0, nq;              // queries of the rows
  int win_lo, win_hi;      // window tokens, where they are one stretch; else win_hi = -1
  int pos[kMaxQ];          // their token positions
};

template <int D>
struct DenseSmem {
  alignas(1024) uint8_t q[(Cfg<D>::QS > 0 ? Cfg<D>::QS : 1) * kRows * 128];       // chunks of [128 rows x 128 B]
  alignas(1024) uint8_t kv[Cfg<D>::NG][Cfg<D>::GC * kTile * 128];                // groups of chunks [64 keys x 128 B]
  alignas(1024) uint8_t raw[kStages][kRawBytes];
  uint64_t raw_full[kStages], raw_empty[kStages];
  uint64_t full[Cfg<D>::NG];
  uint64_t empty[Cfg<D>::NG];
  uint64_t q_moved;                                                              // ... and its first chunks are in tensor memory
  uint64_t q_full;                                                               // a segment's Q has landed
  uint64_t s_full[2], p_full[2], pv_done[2], fin;                                // of a tile's buffer
  uint32_t tmem_base;
  int abort;
  uint32_t qtop[3][kRows];                                                       // largest magnitudes (row_pow) of Q's first chunks and of the rest's halves
  int more[2];
  Segment seg[2];                                                                // this one and the next
};

// Place of 16-byte piece pc of row r (of ROW bytes) in a raw stage: the
// pattern in which a tensor copy with the swizzle of that width writes it.
// Eight lanes that read a piece of eight neighbouring rows meet eight columns.
template <int ROW>
__device__ __forceinline__ uint32_t raw_off(int r, int pc) {
  static_assert(ROW == 128 || ROW == 64, "row");
  return (uint32_t)(r * ROW + ((ROW == 128 ? pc ^ (r & 7) : pc ^ ((r >> 1) & 3)) << 4));
}

// *p where `live`, else `other`.  Nothing depends on the value until its first
// use: a select on it (as a conditional expression would be) waits for the load.
__device__ __forceinline__ int load_if(const int32_t *p, bool live, int other) {
  int v;
  asm volatile("{\n.reg .pred q;\nsetp.ne.s32 q, %2, 0;\nmov.b32 %0, %3;\n@q ld.global.nc.b32 %0, [%1];\n}"
               : "=&r"(v)
               : "l"(p), "r"((int)live), "r"(other));
  return v;
}

// Asynchronous copies to shared memory; `live` false writes zeros instead.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void named_bar_arrive(int id, int n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// Arrive on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// Power of two that a row of Q is multiplied by, as fp32's exponent field; `top2`:
// the largest magnitudes of its even and odd channels as bits of bf16.
constexpr uint32_t kQPow = 127 + 6;
__device__ __forceinline__ uint32_t row_pow(uint32_t top2) {
  const uint32_t top = top2 >> 16 > (top2 & 0xFFFFu) ? top2 >> 16 : top2 & 0xFFFFu, e = top >> 7;
  if (top == 0 || (e >= 127 - 8 && e < 127 + 9)) return kQPow;
  return e < 15u ? 253u : 268u - e;   // (2^126 at most)
}
__device__ __forceinline__ uint32_t top_of(uint32_t top2, uint4 v) {
  top2 = __vimax3_u16x2(top2, v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
  return __vimax3_u16x2(top2, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
}

// The next stretch of at most 64 window tokens at or behind `cur` that the
// unit's queries see, every token of it seen by one of them (what lies between
// their windows is never read).  Called by converged warps; false: none.
__device__ __forceinline__ bool next_window(const Segment &sg, int window, int cur, int lane, int *start, int *end) {
  int lo = INT_MAX;
#pragma unroll 1
  for (int i = lane; i < sg.nq; i += 32) {
    const int t = sg.pos[i];
    if (t >= 0 && t >= cur) {
      int l = t - window + 1;
      l = l < cur ? cur : l;
      l = l < 0 ? 0 : l;
      lo = l < lo ? l : lo;
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lo == INT_MAX) return false;
  int e = lo;
#pragma unroll 1
  while (e < lo + kTile) {
    int m = e;
#pragma unroll 1
    for (int i = lane; i < sg.nq; i += 32) {
      const int t = sg.pos[i];
      if (t >= e && t - window + 1 <= e) m = t + 1 > m ? t + 1 : m;
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (m == e) break;
    e = m;
  }
  *start = lo;
  *end = e < lo + kTile ? e : lo + kTile;
  return true;
}

// The same, by arithmetic alone where the windows make one stretch.
__device__ __forceinline__ bool next_stretch(const Segment &sg, int win_lo, int win_hi, int window, int cur, int lane,
                                             int *start, int *end) {
  if (win_hi < 0) return next_window(sg, window, cur, lane, start, end);
  const int s = cur > win_lo ? cur : win_lo;
  if (s >= win_hi) return false;
  *start = s;
  *end = win_hi - s < kTile ? win_hi : s + kTile;
  return true;
}

// Division of non-negative numbers that nearly always fit 32 bits.
__device__ __forceinline__ long long div64(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// ------------------------------------------------------------------ schedule of the prefix attention

struct Schedule {
  int box;                 // entries of a copy: divides the page and the tile
  int own0;                // first entry of the sequences' own tiles: n_shared rounded down to a box
  int rt_sh, nt_sh;        // row tiles over all rows; key tiles of the prefix
  int rt_own;              // row tiles of a sequence
  int wt;                  // tiles that a window counts for
  int ov;                  // tiles' worth of time that starting and ending a unit takes
  int units;               // units of a channel half
  int cs;
  int grid;
};

inline Schedule make_schedule(const DenseAttnArgs &a, int cs, int grid) {
  Schedule s;
  s.box = prefix_attn_box(a.pool.page);
  s.own0 = a.n_shared - a.n_shared % s.box;
  const long long rows = (long long)a.B * a.T_q * a.H;
  s.rt_sh = (int)((rows + kRows - 1) / kRows);
  s.nt_sh = (a.n_shared + kTile - 1) / kTile;
  s.rt_own = (a.T_q * a.H + kRows - 1) / kRows;
  s.wt = a.window > 0 ? (a.window + kTile - 1) / kTile : 0;
  s.ov = kUnitCost;
  s.units = s.rt_sh + a.B * s.rt_own;
  s.cs = cs;
  s.grid = grid;
  return s;
}

// The linear order of all tiles of a channel half: the prefix's row tiles, then
// the sequences' own row tiles; a unit's length is ov + FP4 tiles + wt.
__host__ __device__ __forceinline__ long long shared_length(const Schedule &s) {
  return s.nt_sh > 0 ? (long long)s.ov + s.nt_sh : 0;
}
__device__ __forceinline__ long long own_length(const Schedule &s, int own) {
  return own + s.wt > 0 ? (long long)s.ov + own + s.wt : 0;
}

// Pool sequence of batch row b (-1 when out of range) and its entries.
__device__ __forceinline__ int seq_entries(const DenseAttnArgs &a, int b, int *n) {
  const int s = a.seq[b];
  *n = 0;
  if (s < 0 || s >= a.pool.n_seq) return -1;
  const long long room = (long long)a.pool.max_pages * a.pool.page;
  const int v = a.pool.n_entries[s];
  *n = v < 0 ? 0 : (v > room ? (int)room : v);
  return s;
}
__device__ __forceinline__ int tiles_of(const DenseAttnArgs &a, const Schedule &s, int n) {
  return n > a.n_shared ? (n - s.own0 + kTile - 1) / kTile : 0;
}
__device__ __forceinline__ int own_tiles(const DenseAttnArgs &a, const Schedule &s, int b) {
  int n;
  seq_entries(a, b, &n);
  return tiles_of(a, s, n);
}

// Workspace: per unit {first slot, slots}; per slot of a unit of the prefix (0)
// or of a sequence's own keys (1) [rows] (max, sum) and [DO / 4][rows] float4 of
// O, rows = 128 or, where a sequence has fewer, its number.
struct DenseWs {
  size_t off_ml[2], off_o[2], bytes;
  int rows[2];
};
__host__ __device__ __forceinline__ DenseWs dense_ws(int rt_sh, long long own_units, int seq_rows, int cs, int grid, int DO) {
  DenseWs w;
  w.bytes = ((size_t)cs * (rt_sh + own_units) * 8 + 255) & ~size_t(255);
  for (int k = 0; k < 2; ++k) {
    w.rows[k] = k == 0 || seq_rows > kRows ? kRows : seq_rows;
    const size_t slots = (size_t)(cs * (k == 0 ? rt_sh : own_units) + grid);
    w.off_ml[k] = w.bytes;
    w.off_o[k] = w.off_ml[k] + ((slots * w.rows[k] * 8 + 255) & ~size_t(255));
    w.bytes = w.off_o[k] + ((slots * w.rows[k] * DO * 4 + 255) & ~size_t(255));
  }
  return w;
}
__device__ __forceinline__ DenseWs dense_ws(const DenseAttnArgs &a, const Schedule &sc, int DO) {
  return dense_ws(sc.rt_sh, (long long)a.B * sc.rt_own, a.T_q * a.H, sc.cs, sc.grid, DO);
}

// Where the search for the sequence at a linear position was last: the first
// sequence of a group of 32 and its position within a half's own part.
struct Cursor {
  int half, b0;
  long long at;
};

// The scheduler's warp: the segment at linear position *x (before x_end); advances
// *x.  `lead`: the batch row through whose table the prefix is read.
template <int DO>
__device__ __forceinline__ bool next_prefix_segment(const DenseAttnArgs &a, const Schedule &sc, int lead, long long th,
                                    long long chunk, long long *x, long long x_end, int lane, Cursor &cur, Segment &sg) {
#pragma unroll 1
  while (*x < x_end) {
    const int half = *x >= th ? 1 : 0;   // at most two channel halves
    const long long base = (long long)half * th;
    long long y = *x - base;
    const long long one = shared_length(sc), sh = sc.rt_sh * one;
    int unit, nt, wt, b = 0, rt;
    long long tile, unit_at;
    if (y < sh) {
      rt = (int)div64(y, one);
      unit = rt; tile = y - rt * one - sc.ov; nt = sc.nt_sh; wt = 0;
      unit_at = base + rt * one;
    } else {
      y -= sh;
      if (cur.half != half) cur = Cursor{half, 0, 0};   // (positions only grow)
      long long at = cur.at;   // linear position of sequence b0 within the own part
      int b0 = cur.b0, own = 0;
#pragma unroll 1
      for (;;) {
        const int bb = b0 + lane;
        own = bb < a.B ? own_tiles(a, sc, bb) : 0;
        const long long c = bb < a.B ? sc.rt_own * own_length(sc, own) : 0;
        long long inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, at + inc > y);
        if (hit) {
          cur.b0 = b0;
          cur.at = at;
          const int l = __ffs(hit) - 1;
          b = b0 + l;
          at += __shfl_sync(0xffffffffu, inc - c, l);
          own = __shfl_sync(0xffffffffu, own, l);
          break;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
        b0 += 32;
        if (b0 >= a.B) return false;   // not reached: th is the sum of these
      }
      nt = own; wt = sc.wt;
      const long long len = own_length(sc, own);
      rt = (int)div64(y - at, len);
      tile = y - at - rt * len - sc.ov;
      unit = sc.rt_sh + b * sc.rt_own + rt;
      unit_at = base + sh + at + rt * len;
    }
    if (tile < 0) {    // in the unit's overhead: its first tile is the next position
      *x -= tile;
      continue;
    }
    if (tile > nt) {   // behind the start of the window's tiles: the window went with its first one
      *x = unit_at + sc.ov + nt + wt;
      continue;
    }
    long long n = nt - tile;
    if (n > x_end - *x) n = x_end - *x;
    const bool win = wt > 0 && *x + (nt - tile) < x_end;
    const long long done = win ? unit_at + sc.ov + nt + wt : *x + n;
    if (lane == 0) {
      const bool shared = unit < sc.rt_sh;
      sg.half = half;
      sg.b = b;
      if (shared) {
        const int rows = a.B * a.T_q * a.H;
        sg.row0 = rt * kRows;
        sg.nrows = rows - sg.row0 < kRows ? rows - sg.row0 : kRows;
      } else {
        const int rows = a.T_q * a.H;
        sg.row0 = b * rows + rt * kRows;
        sg.nrows = rows - rt * kRows < kRows ? rows - rt * kRows : kRows;
      }
      int ents = 0;
      sg.seq = seq_entries(a, shared ? lead : b, &ents);
      sg.n_sink = 0;
      sg.n_fp4 = (int)n;
      sg.n_win = win ? 1 : 0;   // counted below
      sg.key0 = (shared ? 0 : sc.own0) + (int)tile * kTile;
      sg.key_lo = shared ? 0 : a.n_shared;
      sg.key_end = shared && ents > a.n_shared ? a.n_shared : ents;
      const int u = half * sc.units + unit;
      const int g0 = (int)div64(unit_at + sc.ov, chunk);
      // (a unit's parts lie in consecutive blocks, and the next unit starts in
      // the last one's block or behind it: no two parts meet in a slot)
      const int u_sort = shared ? half * sc.rt_sh + unit : half * (sc.units - sc.rt_sh) + unit - sc.rt_sh;
      const DenseWs w = dense_ws(a, sc, DO);
      const size_t slot = (size_t)((int)blockIdx.x + u_sort);
      sg.o_rows = shared ? w.rows[0] : w.rows[1];
      sg.ml_at = (shared ? w.off_ml[0] : w.off_ml[1]) + slot * sg.o_rows * 8;
      sg.o_at = (shared ? w.off_o[0] : w.off_o[1]) + slot * sg.o_rows * DO * 4;
      if (g0 == (int)blockIdx.x) {
        const long long last = unit_at + sc.ov + (wt > 0 ? nt : nt - 1);
        reinterpret_cast<int2 *>(a.ws)[u] = make_int2(g0 + u_sort, (int)div64(last, chunk) - g0 + 1);
      }
    }
    *x = done;
    return true;
  }
  return false;
}

// Pages of the boxes of a segment's FP4 tiles, tile by tile: lane = box.
struct BoxPages {
  const int32_t *row;      // the sequence's page list
  int e, end;              // first entry of the lane's box in the next tile; the segment's last
  int idx, off;            // its page's place in the list, its place in the page (advanced without dividing again)
  int page, adv_p, adv_o;
  bool mine;
  __device__ __forceinline__ BoxPages(const Segment &sg, const Schedule &sc, const PagePoolArgs &pool, int lane) {
    page = pool.page > 0 ? pool.page : 1;
    row = sg.seq >= 0 ? pool.table + (size_t)sg.seq * pool.max_pages : nullptr;
    mine = lane * sc.box < kTile;
    e = sg.key0 + lane * sc.box;
    end = sg.key_end;
    idx = e / page;
    off = e % page;
    adv_p = kTile / page;
    adv_o = kTile % page;
  }
  // The page of this lane's box (as the list has it; -1 without a list), `none`
  // where the box holds nothing, `more` says that there is a tile; steps on.
  __device__ __forceinline__ int next(bool more, int none) {
    const bool in = more && mine && e < end;
    const int v = load_if(row + idx, in && row != nullptr, in ? -1 : none);
    e += kTile;
    idx += adv_p;
    off += adv_o;
    if (off >= page) { off -= page; ++idx; }
    return v;
  }
};

}  // namespace

// MODE 0: prefix attention (paged entries and an optional window), partial
// results; MODE 1: window with sinks, straight to the output.
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) attn_dense_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                 const __grid_constant__ CUtensorMap codes_map,
                                                                 const __grid_constant__ CUtensorMap scales_map,
                                                                 const __grid_constant__ CUtensorMap swa_map,
                                                                 const __grid_constant__ CUtensorMap sink_map,
                                                                 const DenseAttnArgs a, const Schedule sc) {
  using F = Cfg<D>;
  constexpr int DO = F::DO, CS = F::CS, NCH = F::NCH, GC = F::GC, NG = F::NG, QT = F::QT, QS = F::QS;
  constexpr uint32_t kIdS = mma_idesc(kRows, kTile, 0u, 0u);
  constexpr uint32_t kIdO = mma_idesc(kRows, DO, 0u, 0u) | (1u << 16);   // B (V) MN-major
  extern __shared__ uint8_t smem_raw[];
  DenseSmem<D> &S = *reinterpret_cast<DenseSmem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~uintptr_t(1023));
  volatile int *abort = &S.abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int g = 0; g < NG; ++g) {
      mbar_init(&S.full[g], kTeam);
      mbar_init(&S.empty[g], 1);
    }
    for (int u = 0; u < kStages; ++u) {
      mbar_init(&S.raw_full[u], 32);
      mbar_init(&S.raw_empty[u], kTeam);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&S.s_full[u], 1);
      mbar_init(&S.p_full[u], 4);
      mbar_init(&S.pv_done[u], 1);
    }
    mbar_init(&S.q_full, 1);
    mbar_init(&S.q_moved, 4);
    mbar_init(&S.fin, 2);
    S.abort = 0;
    fence_barrier_init();
  }
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

  bool dead = false;
  // A segment's start: the scheduler warp has written it (or that there is
  // none).  Its end: true when a wait of any role gave up.
  uint32_t seg_i = 0;
  auto begin_segment = [&]() -> bool {
    named_bar(kSegBar, kThreads);
    return S.more[seg_i & 1u] != 0;
  };
  constexpr int kQBarThreads = kDq + 4 * 32 + 32;
  // Where chunk k of Q's first ones lands: in the ring's last two groups from
  // here on, so that the first ones can be filled meanwhile.
  auto q_staging = [&](uint32_t g0, int k) -> uint8_t * {
    return S.kv[(g0 + NG - 2 + (uint32_t)(k / (GC / 2))) % NG] + (k % (GC / 2)) * (kRows * 128);
  };
  auto end_segment = [&]() -> bool {
    ++seg_i;
    return named_bar_or(kSegBar, kThreads, *abort != 0);
  };
  // Chunk of Q (64 channels) that S takes k-th: the other half's channels
  // first.
  auto q_chunk = [&](int k, int half) -> int { return CS > 1 ? (k + (half == 0 ? GC : 0)) % NCH : k; };
  // bf16 -> fp16 times the row's power of two, with the sign of the softmax scale
  // (so that the logits' own factor is not negative).
  auto q_factor = [&](uint32_t field) -> float { return __uint_as_float((field << 23) | (a.scale < 0.f ? 0x80000000u : 0u)); };
  auto to_f16x2 = [&](uint32_t w, float pow) -> uint32_t {
    const __half2 hv = __floats2half2_rn(bf16_to_f32(w & 0xFFFFu) * pow, bf16_to_f32(w >> 16) * pow);
    return *reinterpret_cast<const uint32_t *>(&hv);
  };
  auto to_f16x4 = [&](uint4 v, float pow) -> uint4 {   // (8 elements)
    return make_uint4(to_f16x2(v.x, pow), to_f16x2(v.y, pow), to_f16x2(v.z, pow), to_f16x2(v.w, pow));
  };
  // A converged warp's wait, polled by all its lanes: one that lane 0 polls for
  // the others leaves it behind at times, and the tcgen05 instructions that
  // follow have to be met by all lanes at once.
  auto all_wait = [&](uint64_t *bar, uint32_t parity) {
    const bool w_ok = __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort)) != 0;
    __syncwarp();
    return w_ok;
  };
  uint32_t gcount = 0, tcount = 0;   // ring groups and tiles so far (each role advances them alike)
  uint32_t scount = 0;               // raw steps so far (load and dequantise)

  if (warp < kDqWarps) {
    // ================================================ fetch + dequantise
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFetch));
    while (begin_segment()) {
      const Segment &sg = S.seg[seg_i & 1u];
      // (what the tile loop needs in registers: beside the S product a load from
      // shared memory takes 320 cycles instead of 43)
      const int n_sink = sg.n_sink, n_fp4 = sg.n_fp4, n_tiles = n_sink + n_fp4 + sg.n_win;
      const int key0 = sg.key0, key_lo = sg.key_lo, key_end = sg.key_end;
      const int win_lo = sg.win_lo, win_hi = sg.win_hi;
      // ---- Q's chunks of shared memory: bf16 -> fp16 in place.  Without any (D
      // 128 and 256) the first groups are filled while Q is on its way: 31.3 us
      // against 33.1 us (3 x 517 tokens of 20 heads, D 256, window 333)
      constexpr bool kEarly = QS == 0;
      bool ok = true;
      if constexpr (QS > 0) {
        // (thread = a row's share of the chunks)
        static_assert(kDq == 2 * kRows && QS % 2 == 0, "a row's chunks in two shares");
        constexpr int SH = QS / 2;
        const int row = tid % kRows, part = tid / kRows;
        auto piece = [&](int k, int i) {
          return reinterpret_cast<uint4 *>(S.q + (part * SH + k) * (kRows * 128) + row * 128 + ((i ^ (row & 7)) << 4));
        };
        const bool landed = all_wait(&S.q_full, seg_i & 1u);
        uint32_t top2 = 0;
        if (landed) {
          const float pow = q_factor(kQPow);
#pragma unroll 1
          for (int k = 0; k < SH; ++k) {
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
              uint4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = *piece(k, h + i);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                top2 = top_of(top2, v[i]);
                *piece(k, h + i) = to_f16x4(v[i], pow);
              }
            }
          }
        }
        S.qtop[1 + part][row] = top2;
        named_bar(kQTopBar, kDq + 4 * 32);
        const uint32_t qf = row_pow(__vimax3_u16x2(S.qtop[0][row], S.qtop[1][row], S.qtop[2][row]));
        if (landed && qf != kQPow) {   // once more, from memory (rows behind the last are zeros: not here)
          const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (size_t)(sg.row0 + row) * D);
#pragma unroll 1
          for (int k = 0; k < SH; ++k)
#pragma unroll 1
            for (int i = 0; i < 8; ++i)
              *piece(k, i) = to_f16x4(__ldg(src + q_chunk(QT + part * SH + k, sg.half) * 8 + i), q_factor(qf));
        }
        fence_proxy_async();
      }
      named_bar_arrive(kQBar, kQBarThreads);
      if (!kEarly) ok = all_wait(&S.q_moved, seg_i & 1u);
      const uint32_t g_first = gcount;
      // ---- team t takes the groups whose running number is t modulo 2: the
      // two halves of a tile's channels (D 512), or every other tile.  Lane =
      // (row, 16-byte piece) so that the eight lanes of a load's or a store's
      // phase meet eight different 16-byte columns of the swizzled rows
      const uint32_t team = warp / kTeam;
      const int p4 = lane >> 3;                                // piece 0..3 (then 4..7)
      const int r0 = (warp % kTeam) * 16 + (lane & 7);         // keys r0 and r0 + 8
      auto hand_over = [&](uint64_t *bar) {   // generic stores -> visible to the tensor core
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      // A step's bytes.  The stage's step before may be the other team's: that
      // it has been consumed comes first, since the copies land in any order
      // and a wait for this step's phase, met in the phase before the last,
      // would pass at once.  The one before that, 2 x kStages back, has been
      // consumed, or the first wait would pass a phase early too: a warp that
      // asks for step n has seen its team's last one, s, and s was issued once
      // step s - kStages had been consumed, so n - s <= kStages is needed.  The
      // other team's steps in between are one group's: FP8_S at most.
      auto raw_wait = [&](uint32_t step) -> bool {
        const uint32_t st = step % kStages, ph = (step / kStages) & 1u;
        return all_wait(&S.raw_empty[st], ph ^ 1u) && all_wait(&S.raw_full[st], ph);
      };
      constexpr int FP8_S = GC / 2;                        // steps of a group of FP8 rows
      static_assert(FP8_S + 1 <= kStages, "a team's next step is at most kStages behind its last");
#pragma unroll 1
      for (int it = 0; it < n_tiles && ok; ++it) {
        const bool fp4 = it >= n_sink && it < n_sink + n_fp4;
        const uint32_t g_mine = CS > 1 ? team : 0u;
        const bool mine = CS > 1 || (gcount & 1u) == team;
        uint32_t step = scount + g_mine * (fp4 ? 1u : (uint32_t)FP8_S);
        const uint32_t gi = gcount + g_mine;
        gcount += CS;
        scount += fp4 ? CS : CS * FP8_S;
        if (!mine) continue;
        const uint32_t slot = gi % NG, ph = (gi / NG) & 1u;
        uint8_t *kv = S.kv[slot];
        // the groups that Q's first chunks landed in
        if (kEarly && gi - g_first >= NG - 2 && gi - g_first < NG) {
          ok = all_wait(&S.q_moved, seg_i & 1u);
          if (!ok) break;
        }
        if (fp4) {
          const uint32_t st = step % kStages;
          ok = raw_wait(step);
          if (!ok) break;
          constexpr int NU = GC / 2;                       // pieces of 32 channels per key
          uint4 rv[NU][2];
          uint32_t sb[NU][2];
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              rv[u][y] = *reinterpret_cast<const uint4 *>(S.raw[st] + raw_off<F::CB>(r0 + 8 * y, p4 + 4 * u));
              sb[u][y] = *reinterpret_cast<const uint16_t *>(S.raw[st] + kRawSc + (r0 + 8 * y) * F::SB + (p4 + 4 * u) * 2);
            }
          // this warp's part of the stage is in registers.  (The fence: an arrival
          // overtakes loads that wait for shared memory beside the S product, and
          // a tensor copy would then write what they have yet to read.)
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.raw_empty[st]);
          const int k0 = key0 + (it - n_sink) * kTile;
          if (k0 < key_lo || k0 + kTile > key_end) {   // what the copies brought of other entries: zeros
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int k = k0 + r0 + 8 * y;
              if (k >= key_lo && k < key_end) continue;
#pragma unroll
              for (int u = 0; u < NU; ++u) {
                rv[u][y] = make_uint4(0, 0, 0, 0);
                sb[u][y] = 0;
              }
            }
          }
          ok = all_wait(&S.empty[slot], ph ^ 1u);
          if (!ok) break;
#pragma unroll
          for (int u = 0; u < NU; ++u) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t s0 = e4m3x2_to_f16x2(__byte_perm(sb[u][y], 0, 0x0000));
              const uint32_t s1 = e4m3x2_to_f16x2(__byte_perm(sb[u][y], 0, 0x1111));
              const uint32_t w[4] = {rv[u][y].x, rv[u][y].y, rv[u][y].z, rv[u][y].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t h[4];
                e2m1x8_to_f16x2(w[j], h);
                const __half2 sk = *reinterpret_cast<const __half2 *>(j < 2 ? &s0 : &s1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&h[e]), sk);
                  h[e] = *reinterpret_cast<const uint32_t *>(&v);
                }
                *reinterpret_cast<uint4 *>(kv + sw_off(r0 + 8 * y, 4 * (p4 + 4 * u) + j, kTile)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
              }
            }
          }
        } else {
          // rows of the tile that are keys; what the copies brought behind them: zeros
          int keys = kTile;
          if (it < n_sink) keys = key_end - it * kTile;
          else if (win_hi >= 0) keys = win_hi - win_lo - (it - n_sink - n_fp4) * kTile;
#pragma unroll 1
          for (int sub = 0; sub < FP8_S; ++sub, ++step) {  // two chunks a step
            const uint32_t st = step % kStages;
            ok = raw_wait(step);
            if (!ok) break;
            uint4 rv[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                rv[u][y] = *reinterpret_cast<const uint4 *>(S.raw[st] + raw_off<kRawRow>(r0 + 8 * y, p4 + 4 * u));
            fence_proxy_async();   // (as above)
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.raw_empty[st]);
            if (keys < kTile) {
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (r0 + 8 * y >= keys) rv[0][y] = rv[1][y] = make_uint4(0, 0, 0, 0);
            }
            if (sub == 0) ok = all_wait(&S.empty[slot], ph ^ 1u);
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < 2; ++u) {                  // 16 channels of chunk 2 sub + u
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t h[8];
                e4m3x4_to_f16x2(rv[u][y].x, h);
                e4m3x4_to_f16x2(rv[u][y].y, h + 2);
                e4m3x4_to_f16x2(rv[u][y].z, h + 4);
                e4m3x4_to_f16x2(rv[u][y].w, h + 6);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  *reinterpret_cast<uint4 *>(kv + sw_off(r0 + 8 * y, 16 * sub + 8 * u + 2 * p4 + j, kTile)) =
                      make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
              }
            }
          }
          if (!ok) break;
        }
        hand_over(&S.full[slot]);
      }
      dead = end_segment();
      if (dead) break;
    }
  } else if (warp < kSmWarp0 + 4) {
    // ================================================ softmax: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    while (begin_segment()) {
      const Segment &sg = S.seg[seg_i & 1u];
      const int n_sink = sg.n_sink, n_fp4 = sg.n_fp4, n_tiles = n_sink + n_fp4 + sg.n_win;
      const int half = sg.half;
      const int key0 = sg.key0, key_lo = sg.key_lo, key_end = sg.key_end;
      const int win_lo = sg.win_lo, win_hi = sg.win_hi;
      const int q = warp & 3, row = 32 * q + lane;
      const uint32_t lrow = tmem + ((uint32_t)(32 * q) << 16);
      const int frow = sg.row0 + row;
      const bool live = row < sg.nrows;
      // ---- Q's first chunks, which landed in the ring: this thread's row into its tensor-memory lane.  A rolled loop: at
      // a kernel's start the instructions come from far
      bool ok = all_wait(&S.q_full, seg_i & 1u);
      uint32_t top2 = 0;
      auto move_q = [&](float pow) {
#pragma unroll 1
        for (int k = 0; k < QT; ++k) {
          const uint8_t *qs = q_staging(tcount * CS, k) + row * 128;
          uint32_t h[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(qs + ((i ^ (row & 7)) << 4));
            top2 = top_of(top2, v);
            h[4 * i] = to_f16x2(v.x, pow); h[4 * i + 1] = to_f16x2(v.y, pow);
            h[4 * i + 2] = to_f16x2(v.z, pow); h[4 * i + 3] = to_f16x2(v.w, pow);
          }
          tmem_st_x32(lrow + kColQ + 32 * k, h);
        }
      };
      float qpow = q_factor(kQPow), unpow = __uint_as_float((254u - kQPow) << 23);
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {   // twice where a row of the warp needs another power
        if (ok) move_q(qpow);
        if (turn > 0) break;
        if constexpr (QS > 0) {
          S.qtop[0][row] = top2;
          named_bar(kQTopBar, kDq + 4 * 32);
          top2 = __vimax3_u16x2(top2, S.qtop[1][row], S.qtop[2][row]);
        }
        const uint32_t qf = row_pow(top2);
        const bool same = __all_sync(0xffffffffu, qf == kQPow) != 0;
        __syncwarp();
        if (same) break;
        qpow = q_factor(qf);
        unpow = __uint_as_float((254u - qf) << 23);
        tmem_wait_st();
      }
      const float lscale = fabsf(a.scale) * kLog2e * unpow;   // of a logit in base 2, but for the key's scale
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_moved);
      __syncwarp();
      named_bar_arrive(kQBar, kQBarThreads);
      const int t = live ? sg.pos[frow / a.H - sg.q0] : -1;
      int vis = 0;                                 // entries this row sees
      if (MODE == 0 && t >= 0) {
        int n;
        const int b = frow / (a.T_q * a.H);
        if (seq_entries(a, b, &n) < 0) flag(a.status, CSA2_DEV_BAD_SEQUENCE);
        const int v = (t + 1) / a.pool.m;
        vis = n < v ? n : v;
        if (vis > key_end) vis = key_end;
      }
      int wlo = t - a.window + 1;
      if (wlo < 0) wlo = 0;
      const int snk = MODE == 1 && t >= 0 ? (a.window > 0 ? wlo : t + 1) : 0;   // sinks below this token
      // Pages of the next FP4 tile (lane = box of the tile), looked up a tile
      // ahead and judged when the tile comes: a slot without a page gave zeros,
      // its keys are hidden.
      BoxPages pages(sg, sc, a.pool, lane);
      float m_ref = -INFINITY, l = 0.f, vsc = 1.f;
      int page_ahead = MODE == 0 ? pages.next(n_fp4 > 0, 0) : 0;
      int wcur = 0;
#pragma unroll 1
      for (int it = 0; it < n_tiles && ok; ++it) {
        const uint32_t tc = tcount + it;
        // the keys of this tile that this row sees: [ja, jb)
        int ja = 0, jb;
        float ksc = 1.f;
        uint32_t badp = 0;
        if (it < n_sink) {
          jb = (snk < key_end ? snk : key_end) - it * kTile;
          ksc = a.s_sink;
        } else if (it < n_sink + n_fp4) {
          const int k0 = key0 + (it - n_sink) * kTile;
          ja = key_lo - k0;
          jb = vis - k0;
          badp = __ballot_sync(0xffffffffu, (uint32_t)page_ahead >= (uint32_t)a.pool.n_pages);
          page_ahead = pages.next(it + 1 < n_sink + n_fp4, 0);
        } else {
          int s = 0, e = 0;
          next_stretch(sg, win_lo, win_hi, a.window, wcur, lane, &s, &e);
          wcur = e;
          ja = wlo - s;
          jb = (t < e ? t + 1 : e) - s;
          if (t < 0) jb = 0;
          ksc = a.s_swa;
        }
        const bool whole = __all_sync(0xffffffffu, ja <= 0 && jb >= kTile) && badp == 0;
        const uint32_t buf = tc & 1u, ph = (tc >> 1) & 1u;
        const uint32_t scol = lrow + kColS + buf * kTile;
        ok = all_wait(&S.s_full[buf], ph);
        if (!ok) break;
        tc_fence_after();
        // logits in base 2: lsc x S; never 0, so that a hidden key's -inf stays
        const float lsc = fmaxf(lscale * ksc, 1e-30f);
        uint32_t sv[kTile];
        tmem_ld_x32(scol, sv);
        tmem_ld_x32(scol + 32, sv + 32);
        tmem_wait_ld();
        if (!whole) {
          // bit j: key j is seen
          const int lo = ja < 0 ? 0 : ja, hi = jb > kTile ? kTile : jb;
          uint64_t seen = hi > lo ? (~0ull >> (kTile - (hi - lo))) << lo : 0ull;
          if (badp) {   // rare
            if (lane == 0) flag(a.status, CSA2_DEV_INDEX_RANGE);
#pragma unroll 1
            for (int j = 0; j < kTile; ++j)
              if ((badp >> (j / sc.box)) & 1u) seen &= ~(1ull << j);
          }
          const uint32_t s_lo = (uint32_t)seen, s_hi = (uint32_t)(seen >> 32);
#pragma unroll
          for (int j = 0; j < kTile; ++j)
            if (!(((j < 32 ? s_lo : s_hi) >> (j & 31)) & 1u)) sv[j] = 0xFF800000u;
        }
        float mx4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) mx4[u] = __uint_as_float(sv[u]);
#pragma unroll
        for (int j = 4; j < kTile; j += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mx4[u] = j + 4 + u < kTile ? fmaxf(mx4[u], fmaxf(__uint_as_float(sv[j + u]), __uint_as_float(sv[j + 4 + u])))
                                       : fmaxf(mx4[u], __uint_as_float(sv[j + u]));
        // The largest exponent against the reference, by the operation that forms the
        // exponents, so that the rounding of a large logit does not take P out of
        // fp16's range.  The reference may be rounded, up: it is what all are relative
        // to, and the largest weight is 2^9 less a step of the logits' fp32 at least
        // (2^-7 up to 2^28, where a step is 16).  Without a reference yet the exponent
        // is +inf, or NaN if nothing is seen.
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        float al = 1.f;
        if (fmaf(mx, lsc, -m_ref) > kBias + kLazy) {
          const float m_new = __fmaf_ru(mx, lsc, -kBias);
          al = ex2_approx(m_ref - m_new);
          m_ref = m_new;
          l *= al;
        }
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        uint32_t pr[kTile / 2];
        {
          const uint64_t l2 = f32x2(lsc, lsc), m2 = f32x2(-mu, -mu);
          uint64_t ls0 = 0, ls1 = 0;
#pragma unroll
          for (int j = 0; j < kTile / 2; ++j) {
            const float2 y = unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), l2, m2));
            const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
            if (j & 1) ls1 = add_f32x2(ls1, f32x2(p0, p1));
            else ls0 = add_f32x2(ls0, f32x2(p0, p1));
            const __half2 hv = __floats2half2_rn(p0, p1);
            pr[j] = *reinterpret_cast<const uint32_t *>(&hv);
          }
          const float2 t2 = unpack_f32x2(add_f32x2(ls0, ls1));
          l += t2.x + t2.y;
        }
        tmem_st_x32(scol, pr);   // this tile's S is in registers
        // O moves with the reference maximum, and from one key scale to the next
        const float conv = it > 0 && ksc != vsc ? vsc / ksc : 1.f;
        const float f = al * conv;
        if (it > 0 && __any_sync(0xffffffffu, f != 1.f)) {
          const uint32_t pt = tc - 1;                      // O of the tile before is complete
          ok = all_wait(&S.pv_done[pt & 1u], (pt >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DO; c += 32) {
            uint32_t o[32];
            tmem_ld_x32(lrow + kColO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st_x32(lrow + kColO + c, o);
          }
        }
        vsc = ksc;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[buf]);
      }
      // ================================================ the segment's result
      if (ok && n_tiles > 0) {
        const uint32_t pt = tcount + n_tiles - 1;
        ok = all_wait(&S.pv_done[pt & 1u], (pt >> 1) & 1u);
        tc_fence_after();
      }
      if (MODE == 1 && ok) {
        // through the ring (no group is in use any more), so that the lanes of
        // a store lie along a row: a store per lane and row would touch 32 lines
        const float inv = l > 0.f ? vsc / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < DO; c += 64) {
          uint32_t o[64];
          if (n_tiles > 0) {
            tmem_ld_x32(lrow + kColO + c, o);
            tmem_ld_x32(lrow + kColO + c + 32, o + 32);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) o[j] = 0;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t pk[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const __nv_bfloat162 bv = __floats2bfloat162_rn(__uint_as_float(o[8 * j + 2 * u]) * inv,
                                                              __uint_as_float(o[8 * j + 2 * u + 1]) * inv);
              pk[u] = *reinterpret_cast<const uint32_t *>(&bv);
            }
            *reinterpret_cast<uint4 *>(S.kv[0] + sw_off(row, c / 8 + j, kRows)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        __syncwarp();   // a warp stores the rows that it has written
        uint16_t *op = a.out + (size_t)sg.row0 * D + half * DO;
        const int nrows = sg.nrows;
#pragma unroll 8
        for (int i = lane; i < 32 * (DO / 8); i += 32) {
          const int r = 32 * q + i / (DO / 8), pc = i % (DO / 8);
          const uint4 v = *reinterpret_cast<const uint4 *>(S.kv[0] + sw_off(r, pc, kRows));
          if (r < nrows) *reinterpret_cast<uint4 *>(op + (size_t)r * D + 8 * pc) = v;
        }
        fence_proxy_async();   // the next segment's Q lands here
      } else if (MODE == 0 && ok) {
        float2 *ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.ws) + sg.ml_at);
        float4 *po = reinterpret_cast<float4 *>(static_cast<uint8_t *>(a.ws) + sg.o_at);
        const int R = sg.o_rows;
        if (live) ml[row] = make_float2(m_ref, l);
#pragma unroll 1
        for (int c = 0; c < DO; c += 64) {
          uint32_t o[64];
          if (n_tiles > 0) {
            tmem_ld_x32(lrow + kColO + c, o);
            tmem_ld_x32(lrow + kColO + c + 32, o + 32);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) o[j] = 0;
          }
          if (live) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              po[(size_t)(c / 4 + j) * R + row] =
                  make_float4(__uint_as_float(o[4 * j]) * vsc, __uint_as_float(o[4 * j + 1]) * vsc,
                              __uint_as_float(o[4 * j + 2]) * vsc, __uint_as_float(o[4 * j + 3]) * vsc);
          }
        }
      }
      tc_fence_before();
      tcount += n_tiles;
      dead = end_segment();
      if (dead) break;
      tc_fence_after();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == kSchedWarp) {
      // ================================================ scheduler: this block's share of the
      // work is [x, x_end) of the tiles' linear order (prefix), every grid-th unit (window)
      long long th = 0, chunk = 1, x, x_end;
      Cursor cur{-1, 0, 0};
      int lead = 0;
      if (MODE == 0) {
        // the prefix is read through the first sequence that holds most of it, of
        // those with a query (a padded row may name any sequence)
        long long sum = 0;
        int most = -1, first = 0;
        for (int b = lane; b < a.B; b += 32) {
          int n;
          seq_entries(a, b, &n);
          sum += own_length(sc, tiles_of(a, sc, n));
          n = n < a.n_shared ? n : a.n_shared;
          if (n > most) {
            int j = 0;
#pragma unroll 1
            while (j < a.T_q && a.q_pos[(size_t)b * a.T_q + j] < 0) ++j;
            if (j < a.T_q) {
              most = n;
              first = b;
            }
          }
        }
        const int top = __reduce_max_sync(0xffffffffu, most);
        lead = __reduce_min_sync(0xffffffffu, most == top ? first : INT_MAX);
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        th = sc.rt_sh * shared_length(sc) + sc.rt_own * sum;
        chunk = div64(th * CS + sc.grid - 1, sc.grid);
        x = chunk * blockIdx.x;
        x_end = x + chunk < th * CS ? x + chunk : th * CS;
      } else {
        x = blockIdx.x;
        x_end = (long long)a.B * sc.rt_own * CS;
      }
      auto write_segment = [&](uint32_t i) -> bool {
        Segment &sg = S.seg[i & 1u];
        bool more;
        if (MODE == 0) {
          more = next_prefix_segment<DO>(a, sc, lead, th, chunk, &x, x_end, lane, cur, sg);
        } else {
          more = x < x_end;
          if (more && lane == 0) {
            const int half = (int)x % CS, u = (int)x / CS;
            const int b = u / sc.rt_own, rt = u % sc.rt_own, rows = a.T_q * a.H;
            sg.half = half; sg.b = b;
            sg.row0 = b * rows + rt * kRows;
            sg.nrows = rows - rt * kRows < kRows ? rows - rt * kRows : kRows;
            sg.n_fp4 = 0; sg.key0 = 0; sg.key_lo = 0; sg.key_end = 0; sg.seq = -1;
            sg.n_sink = 0;
            sg.n_win = 1;
          }
          x += sc.grid;
        }
        __syncwarp();
        if (more) {
          const int q0 = sg.row0 / a.H, nq = (sg.row0 + sg.nrows - 1) / a.H - q0 + 1;
          int top = -1;   // sinks end where the latest query's window starts
          int wlo = INT_MAX, whi = -1;
          bool one = true;   // positions never fall and never skip a token: the windows are one stretch
          for (int i = lane; i < nq; i += 32) {
            int t = a.q_pos[q0 + i];
            if (t > kMaxPos) {   // sums with a tile or a window stay in 32 bits
              flag(a.status, CSA2_DEV_BAD_POSITION);
              t = -1;
            }
            sg.pos[i] = t;
            if (t >= 0) {
              int lo = a.window > 0 ? t - a.window + 1 : t + 1;
              lo = lo < 0 ? 0 : lo;
              top = lo > top ? lo : top;
              wlo = lo < wlo ? lo : wlo;
              whi = t + 1 > whi ? t + 1 : whi;
            }
            if (i > 0) {
              const int before = a.q_pos[q0 + i - 1];
              if (before < 0 || t < before || t - before > a.window) one = false;
            }
            if (t < 0) one = false;
          }
          wlo = __reduce_min_sync(0xffffffffu, wlo);
          whi = __reduce_max_sync(0xffffffffu, whi);
          one = __all_sync(0xffffffffu, one) && a.window > 0;
          top = __reduce_max_sync(0xffffffffu, top);
          if (lane == 0) {
            sg.q0 = q0;
            sg.nq = nq;
            sg.win_lo = wlo;
            sg.win_hi = one ? whi : -1;
            if (MODE == 1) {
              const int n = top < a.n_sink ? top : a.n_sink;
              sg.key_end = n > 0 ? n : 0;
              sg.n_sink = n > 0 ? (n + kTile - 1) / kTile : 0;
            }
          }
          __syncwarp();
          if (sg.n_win) {
            int n = 0, cur = 0, s, e;
            if (one)
              n = (whi - wlo + kTile - 1) / kTile;
            else if (a.window > 0)
              while (next_window(sg, a.window, cur, lane, &s, &e)) { ++n; cur = e; }
            __syncwarp();
            if (lane == 0) sg.n_win = n;
          }
        }
        if (lane == 0) S.more[i & 1u] = more;
        return more;
      };
      write_segment(0);
      while (begin_segment()) {
        write_segment(seg_i + 1);
        dead = end_segment();
        if (dead) break;
      }
    } else {
    // ================================================ MMA issuer, loaders
    while (begin_segment()) {
      const Segment &sg = S.seg[seg_i & 1u];
      const int n_sink = sg.n_sink, n_fp4 = sg.n_fp4, n_tiles = n_sink + n_fp4 + sg.n_win;
      const int half = sg.half;
      if (warp == kMmaWarp) {
        named_bar(kQBar, kQBarThreads);
        // One elected lane runs the whole loop, its waits included: measured, a
        // converged warp that elects a lane per group of MMAs issues the S
        // product at 59 cycles per MMA even with nothing else on the SM (130 in
        // this kernel), one lane at the tensor core's own 38.
        if (elect_one()) {
          tc_fence_after();
          const uint64_t dq0 = smem_desc_kmajor(smem_u32(S.q), 128);
          bool ok = true;
#pragma unroll 1
          for (int it = 0; it < n_tiles && ok; ++it) {
            // the buffer's last P has been used; both barriers are asked before
            // either answer is needed (a wait behind issued MMAs costs about
            // 150 cycles, ready or not)
            const uint32_t tc = tcount + it, buf = tc & 1u, pp = ((tc >> 1) & 1u) ^ 1u;
            const uint32_t scol = tmem + kColS + buf * kTile;
            uint32_t slot = gcount % NG, ph = (gcount / NG) & 1u;
            const bool r0 = tc < 2 || mbar_test_wait(&S.pv_done[buf], pp);
            const bool r1 = mbar_test_wait(&S.full[slot], ph);
            if (!r0) ok = wait_or_abort(&S.pv_done[buf], pp, abort);
            if (ok && !r1) ok = wait_or_abort(&S.full[slot], ph, abort);
            if (!ok) break;
#pragma unroll
            for (int g = 0; g < CS; ++g) {   // groups of chunks in S's order, straight-line code
              if (g > 0) {
                slot = gcount % NG;
                ph = (gcount / NG) & 1u;
                ok = wait_or_abort(&S.full[slot], ph, abort);
                if (!ok) break;
              }
              ++gcount;
              tc_fence_after();
              const uint64_t db = smem_desc_kmajor(smem_u32(S.kv[slot]), 128);
#pragma unroll
              for (int c = 0; c < GC; ++c) {
                const int k = g * GC + c;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t bd = db + (uint64_t)((c * (kTile * 128) + kk * 32) >> 4);
                  if (k < QT)
                    tc_mma_f16_ta(scol, tmem + kColQ + 32 * k + 8 * kk, bd, kIdS, (k > 0 || kk > 0) ? 1u : 0u);
                  else
                    tc_mma_f16(scol, dq0 + (uint64_t)(((k - QT) * (kRows * 128) + kk * 32) >> 4), bd, kIdS, 1u);
                }
              }
              if (CS > 1 && g == 0) tc_commit(&S.empty[slot]);   // the other half's channels: only S needs them
            }
            if (!ok) break;
            tc_commit(&S.s_full[buf]);
          }
        }
        __syncwarp();
      } else if (warp == kPvWarp) {
        if (elect_one()) {
#pragma unroll 1
          for (int it = 0; it < n_tiles; ++it) {
            const uint32_t slot = (gcount + CS - 1) % NG;   // the tile's group of this block's channels
            gcount += CS;
            const uint32_t tc = tcount + it, buf = tc & 1u;
            if (!wait_or_abort(&S.p_full[buf], (tc >> 1) & 1u, abort)) break;
            tc_fence_after();
            const uint64_t dv = smem_desc_mnmajor_sw128(smem_u32(S.kv[slot]), kTile * 128, 1024);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma_f16_ta(tmem + kColO, tmem + kColS + buf * kTile + ks * 8, dv + ((2 * ks * 1024) >> 4), kIdO,
                            (it > 0 || ks > 0) ? 1u : 0u);
            tc_commit(&S.empty[slot]);
            tc_commit(&S.pv_done[buf]);
          }
        }
        __syncwarp();
      } else if (warp == kLoadWarp) {
        // ---- Q by tensor copies, in S's order of the chunks: the first into the
        // ring, the rest into their own place (rows that are not the unit's
        // are not seen by anything that leaves the block)
        if (lane == 0) {
          fence_proxy_async();
          mbar_arrive_expect_tx(&S.q_full, NCH * kRows * 128);
#pragma unroll 1
          for (int k = 0; k < NCH; ++k)
            tma_load_2d(k < QT ? q_staging(tcount * CS, k) : S.q + (k - QT) * (kRows * 128), &q_map, q_chunk(k, half) * 64,
                        sg.row0, &S.q_full);
        }
        __syncwarp();
        // ---- the raw steps.  FP4: the page's boxes by tensor copies, lane =
        // box (codes, then scales; rows behind the pool are filled with zeros:
        // that is where boxes without a page point).  FP8: rows by
        // asynchronous copies, whose lanes lie along the rows
        BoxPages pages(sg, sc, a.pool, lane);
        int off = pages.off, page_ahead = MODE == 0 ? pages.next(n_fp4 > 0, -1) : 0;
        const int nowhere = a.pool.n_pages * a.pool.page;
        int wcur = 0;
        bool ok = true;
        auto acquire = [&](uint32_t st) {
          return __all_sync(0xffffffffu, wait_or_abort(&S.raw_empty[st], ((scount / kStages) & 1u) ^ 1u, abort)) != 0;
        };
        auto share_rows = [&](int y, int mine, int *rows) {   // rows[8 y + i]: row of key 32 y + 4 i + lane / 8
#pragma unroll
          for (int i = 0; i < 8; ++i) rows[y * 8 + i] = __shfl_sync(0xffffffffu, mine, i * 4 + lane / 8);
        };
        if (MODE == 0) fence_proxy_async();   // stages that the last segment's window wrote
#pragma unroll 1
        for (int it = 0; it < n_tiles && ok; ++it) {
          if (MODE == 0 && it < n_fp4) {
            int er = (uint32_t)page_ahead < (uint32_t)a.pool.n_pages ? page_ahead * a.pool.page + off : nowhere;
            off = pages.off;
            page_ahead = pages.next(it + 1 < n_fp4, -1);
#pragma unroll 1
            for (int g = 0; g < CS; ++g) {
              const uint32_t st = scount % kStages;
              ok = acquire(st);
              if (!ok) break;
              const int c0 = q_chunk(g * GC, half);
              if (lane == 0) {
                mbar_arrive_expect_tx(&S.raw_full[st], kTile * (F::CB + F::SB));
                mbar_arrive_n(&S.raw_full[st], 31);
              }
              __syncwarp();
              if (lane * sc.box < kTile) {
                uint8_t *raw = S.raw[st];
                tma_load_2d(raw + lane * sc.box * F::CB, &codes_map, c0 * 32, er, &S.raw_full[st]);
                if (D == 128)   // two keys' scales make a row of the map
                  tma_load_2d(raw + kRawSc + lane * sc.box * F::SB, &scales_map, 0, er >> 1, &S.raw_full[st]);
                else
                  tma_load_2d(raw + kRawSc + lane * sc.box * F::SB, &scales_map, c0 * 4, er, &S.raw_full[st]);
              }
              ++scount;
            }
          } else {
            // rows that follow one another in their plane: a tensor copy of 64
            // (what lies behind the last key is taken as zeros later)
            int at = -1;                           // first row
            const uint8_t *base;                   // the rows' sequence
            int row[2] = {-1, -1};
            if (it < n_sink) {
              base = a.sink_rows + (size_t)sg.b * a.sink_cap * D;
              at = sg.b * a.sink_cap + it * kTile;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int key = it * kTile + 32 * y + lane;
                if (key < sg.key_end) row[y] = key;
              }
            } else {
              base = a.swa_rows + (size_t)sg.b * a.W_cap * D;
              int s = 0, e = 0;
              next_stretch(sg, sg.win_lo, sg.win_hi, a.window, wcur, lane, &s, &e);
              wcur = e;
              const int s_row = s % a.W_cap;
              if (sg.win_hi >= 0 && s_row + (e - s) <= a.W_cap) {
                at = sg.b * a.W_cap + s_row;
              } else {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int tok = s + 32 * y + lane;
                  if (tok < e) row[y] = tok % a.W_cap;
                }
              }
            }
            if (at >= 0) {
              const CUtensorMap *map = it < n_sink ? &sink_map : &swa_map;
#pragma unroll 1
              for (int k = 0; k < NCH; k += 2) {   // two chunks a step, in S's order
                const uint32_t st = scount % kStages;
                ok = acquire(st);
                if (!ok) break;
                if (lane == 0) {
                  fence_proxy_async();             // a stage that the other form wrote last
                  mbar_arrive_expect_tx(&S.raw_full[st], kTile * kRawRow);
                  mbar_arrive_n(&S.raw_full[st], 31);
                  tma_load_2d(S.raw[st], map, q_chunk(k, half) * 64, at, &S.raw_full[st]);
                }
                __syncwarp();
                ++scount;
              }
              continue;
            }
            int rows[16];
            share_rows(0, row[0], rows);
            share_rows(1, row[1], rows);
#pragma unroll 1
            for (int k = 0; k < NCH; k += 2) {   // two chunks a step, in S's order
              const uint32_t st = scount % kStages;
              ok = acquire(st);
              if (!ok) break;
              const uint32_t dst = smem_u32(S.raw[st]);
              const uint8_t *src = base + q_chunk(k, half) * 64 + (lane & 7) * 16;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                cp_async16(dst + raw_off<kRawRow>(4 * i + lane / 8, lane & 7), src + (size_t)(rows[i] < 0 ? 0 : rows[i]) * D,
                           rows[i] >= 0);
              cp_async_arrive(&S.raw_full[st]);
              ++scount;
            }
          }
        }
        // none in flight when the segment (or, after a wait that gave up, the block) ends
        cp_async_wait_all();
        mbar_wait_bounded(&S.q_full, seg_i & 1u, kWaitLimit);
        for (uint32_t u = scount < kStages ? 0 : scount - kStages; u < scount; ++u)
          mbar_wait_bounded(&S.raw_full[u % kStages], (u / kStages) & 1u, kWaitLimit);
        __syncwarp();
      }
      tcount += n_tiles;
      dead = end_segment();
      if (dead) break;
    }
    }
  }
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

// Joins the parts of every row: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// Block: a row tile of 128 flattened rows x 8 channels; thread = (row, share of
// the parts).  One pass with a running maximum, kMergeBatch parts in flight per
// thread; the parts' planes are [channel / 4][row], so every load is coalesced.
constexpr int kMergeShares = 4, kMergeCh = 8, kMergeBatch = 2;
template <int D>
__global__ void __launch_bounds__(kRows * kMergeShares, 2) attn_dense_merge_kernel(const DenseAttnArgs a, const Schedule sc) {
  using F = Cfg<D>;
  constexpr int DO = F::DO;
  __shared__ float2 red[kMergeShares][kRows];   // (maximum, sum) of a share
  __shared__ float4 racc[kMergeShares - 1][kMergeCh / 4][kRows];
  const int row = threadIdx.x % kRows, share = threadIdx.x / kRows;
  pdl_launch_dependents();
  pdl_wait();
  const long long rows = (long long)a.B * a.T_q * a.H;
  const long long frow = (long long)blockIdx.x * kRows + row;
  const bool live = frow < rows;
  const int ch0 = blockIdx.y * kMergeCh, half = ch0 / DO, c0 = ch0 % DO;
  const int b = live ? (int)(frow / ((long long)a.T_q * a.H)) : 0;
  const int orow = live ? (int)(frow - (long long)b * a.T_q * a.H) : 0;
  const DenseWs w = dense_ws(a, sc, DO);
  const uint8_t *ws = static_cast<const uint8_t *>(a.ws);
  const int2 *desc = reinterpret_cast<const int2 *>(ws) + (size_t)half * sc.units;
  int2 sh = make_int2(0, 0), ow = make_int2(0, 0);   // (first slot, slots) of the prefix and of the row's own keys
  if (live && sc.nt_sh > 0) sh = __ldcg(desc + blockIdx.x);
  if (live && own_tiles(a, sc, b) + sc.wt > 0) ow = __ldcg(desc + sc.rt_sh + b * sc.rt_own + orow / kRows);
  const int parts = sh.y + ow.y;
  // this row and channel range in the first part of either sort
  const int R1 = w.rows[1], r1 = orow % kRows;
  const float2 *ml0 = reinterpret_cast<const float2 *>(ws + w.off_ml[0]) + (size_t)sh.x * kRows + row;
  const float2 *ml1 = reinterpret_cast<const float2 *>(ws + w.off_ml[1]) + (size_t)ow.x * R1 + r1;
  const float4 *po0 = reinterpret_cast<const float4 *>(ws + w.off_o[0]) + ((size_t)sh.x * (DO / 4) + c0 / 4) * kRows + row;
  const float4 *po1 = reinterpret_cast<const float4 *>(ws + w.off_o[1]) + ((size_t)ow.x * (DO / 4) + c0 / 4) * R1 + r1;
  float M = -INFINITY, L = 0.f;
  float4 acc[kMergeCh / 4];
#pragma unroll
  for (int j = 0; j < kMergeCh / 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = share; s0 < parts; s0 += kMergeShares * kMergeBatch) {
    float2 v[kMergeBatch];
    float4 o[kMergeBatch][kMergeCh / 4];
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int s = s0 + u * kMergeShares;
      v[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < kMergeCh / 4; ++j) o[u][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < parts) {
        const int k = s < sh.y ? s : s - sh.y, R = s < sh.y ? kRows : R1;
        const float4 *p = (s < sh.y ? po0 : po1) + (size_t)k * ((DO / 4) * R);
        v[u] = __ldcg((s < sh.y ? ml0 : ml1) + (size_t)k * R);
#pragma unroll
        for (int j = 0; j < kMergeCh / 4; ++j) o[u][j] = __ldcg(p + (size_t)j * R);
      }
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) Mn = fmaxf(Mn, v[u].x);
    const float Mu = Mn == -INFINITY ? 0.f : Mn;
    const float f0 = exp2f(M - Mu);
    M = Mn;
    L *= f0;
#pragma unroll
    for (int j = 0; j < kMergeCh / 4; ++j) { acc[j].x *= f0; acc[j].y *= f0; acc[j].z *= f0; acc[j].w *= f0; }
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float f = exp2f(v[u].x - Mu);
      L = fmaf(f, v[u].y, L);
#pragma unroll
      for (int j = 0; j < kMergeCh / 4; ++j) {
        acc[j].x = fmaf(f, o[u][j].x, acc[j].x);
        acc[j].y = fmaf(f, o[u][j].y, acc[j].y);
        acc[j].z = fmaf(f, o[u][j].z, acc[j].z);
        acc[j].w = fmaf(f, o[u][j].w, acc[j].w);
      }
    }
  }
  red[share][row] = make_float2(M, L);
  if (share > 0) {
#pragma unroll
    for (int j = 0; j < kMergeCh / 4; ++j) racc[share - 1][j][row] = acc[j];
  }
  __syncthreads();
  if (share > 0 || !live) return;
#pragma unroll
  for (int u = 1; u < kMergeShares; ++u) M = fmaxf(M, red[u][row].x);
  float f[kMergeShares];
  L = 0.f;
#pragma unroll
  for (int u = 0; u < kMergeShares; ++u) {
    f[u] = exp2f(red[u][row].x - (M == -INFINITY ? 0.f : M));
    L = fmaf(f[u], red[u][row].y, L);
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  uint32_t pk[kMergeCh / 2];
#pragma unroll
  for (int j = 0; j < kMergeCh / 4; ++j) {
    acc[j].x *= f[0]; acc[j].y *= f[0]; acc[j].z *= f[0]; acc[j].w *= f[0];
#pragma unroll
    for (int u = 1; u < kMergeShares; ++u) {
      const float4 v = racc[u - 1][j][row];
      acc[j].x = fmaf(f[u], v.x, acc[j].x);
      acc[j].y = fmaf(f[u], v.y, acc[j].y);
      acc[j].z = fmaf(f[u], v.z, acc[j].z);
      acc[j].w = fmaf(f[u], v.w, acc[j].w);
    }
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[j].x * inv, acc[j].y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[j].z * inv, acc[j].w * inv);
    pk[2 * j] = *reinterpret_cast<const uint32_t *>(&x);
    pk[2 * j + 1] = *reinterpret_cast<const uint32_t *>(&y);
  }
  *reinterpret_cast<uint4 *>(a.out + frow * D + ch0) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

namespace {

template <int D, int MODE>
cudaError_t launch_dense(const DenseMaps &m, const DenseAttnArgs &a, const Schedule &sc, cudaStream_t s) {
  const size_t smem = sizeof(DenseSmem<D>) + 1024;
  static_assert(sizeof(DenseSmem<D>) + 1024 <= 232448, "shared memory");
  static_assert(Cfg<D>::QT * kRows == 2 * Cfg<D>::GC * kTile && Cfg<D>::NG > 2, "Q's staging in the ring");
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem_once(attn_dense_kernel<D, MODE>, smem, &allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_dense_kernel<D, MODE>, dim3(sc.grid), dim3(kThreads), smem, s, dim3(1, 1, 1), m.q, m.codes,
                    m.scales, m.swa, m.sinks, a, sc);
}

template <int D>
cudaError_t launch_prefix_t(const DenseMaps &m, const DenseAttnArgs &a, int sms, cudaStream_t s) {
  const Schedule sc = make_schedule(a, Cfg<D>::CS, sms);
  cudaError_t e = launch_dense<D, 0>(m, a, sc, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_dense_merge_kernel<D>, dim3(sc.rt_sh, D / kMergeCh), dim3(kRows * kMergeShares), 0, s, dim3(1, 1, 1), a, sc);
}

template <int D>
cudaError_t launch_window_t(const DenseMaps &m, const DenseAttnArgs &a, int sms, cudaStream_t s) {
  Schedule sc = make_schedule(a, Cfg<D>::CS, sms);
  const long long units = (long long)a.B * sc.rt_own * Cfg<D>::CS;
  if (units < sc.grid) sc.grid = (int)units;
  return launch_dense<D, 1>(m, a, sc, s);
}

}  // namespace

size_t prefix_attn_workspace_bytes(int B, int T_q, int H, int D, int sms) {
  const long long rows = (long long)B * T_q * H;
  const long long own_units = (long long)B * ((T_q * H + kRows - 1) / kRows);
  return dense_ws((int)((rows + kRows - 1) / kRows), own_units, T_q * H, D > 256 ? D / 256 : 1, sms, D < 256 ? D : 256).bytes;
}
cudaError_t launch_prefix_attn(const DenseMaps &m, const DenseAttnArgs &a, int sms, cudaStream_t s) {
  switch (a.D) {
    case 128: return launch_prefix_t<128>(m, a, sms, s);
    case 256: return launch_prefix_t<256>(m, a, sms, s);
    default: return launch_prefix_t<512>(m, a, sms, s);
  }
}
size_t window_attn_workspace_bytes(int, int, int, int, int, int, int) { return 0; }
cudaError_t launch_window_attn(const DenseMaps &m, const DenseAttnArgs &a, int sms, cudaStream_t s) {
  switch (a.D) {
    case 128: return launch_window_t<128>(m, a, sms, s);
    case 256: return launch_window_t<256>(m, a, sms, s);
    default: return launch_window_t<512>(m, a, sms, s);
  }
}

}  // namespace csa2
