// Pages of the FP4 cache: append (cut, copy-on-write, allocate), fork / free,
// compact.  Bookkeeping is on the device, so a serving step never waits for
// the host: pages carry reference counts, tables hold page ids, and the free
// pages are those of count 0, taken lowest index first (so the result of
// every call is a function of the pool's state, whatever the timing).
//
// All three are byte moves: 2 x (bytes moved) over HBM, or the launch and the
// bookkeeping chain when little moves.  Each is a one-block (or one block per
// sequence) plan and a wide copy, chained by programmatic dependent launch, but
// for short fork lists (one launch).
// Measured: compacting 8,192 pages of 128 entries, D 512, half of them live (2,048
// move, 151 MB): plan 6 us, move 26 us = 5.8 TB/s, 88% of a plain copy.  Appends,
// a call in a replayed graph, first into pages that the sequences hold alone, then
// with the pool as it was before (fresh pages, shared last pages copied): 49,152
// entries (28 MB) 9.5 and 8.8 us, one entry for each of 32 sequences 6.7 and 8.4
// us.  Back to back from the host 10 to 11 us, which it takes for a call and its
// two launches.
#include "common.cuh"
#include "kernels_paged.h"

namespace csa2 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyEntries = 64;      // entries a copy block moves per turn

struct AppendPlan {   // one per listed sequence
  int seq;            // pool sequence; < 0: skipped
  int at, cnt;
  int cow_src;        // page whose first at % page entries are copied, or -1
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Exclusive prefix sum over the block of one int per thread; *total gets the
// sum.  `sm` holds kPlanWarps + 1 ints; callers sync before reusing it.
__device__ __forceinline__ int block_exclusive(int v, int *sm, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = sm[lane];
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sm[lane] = s - w;
    if (lane == 31) sm[kPlanWarps] = s;
  }
  __syncthreads();
  *total = sm[kPlanWarps];
  return sm[warp] + x - v;
}

// refs[4 i .. 4 i + 3], -1 behind the last page.
__device__ __forceinline__ int4 load_refs(const int32_t *refs, int n_pages, int i) {
  const int p = 4 * i;
  if (p + 4 <= n_pages) return *reinterpret_cast<const int4 *>(refs + p);
  return make_int4(p < n_pages ? refs[p] : -1, p + 1 < n_pages ? refs[p + 1] : -1, p + 2 < n_pages ? refs[p + 2] : -1, -1);
}

}  // namespace

// ------------------------------------------------------------------ append

// Workspace: plans [n], needs [n], bit words [n][words] (slots that get a
// fresh page), free pages [n_pages].
struct PageAppendWs {
  size_t off_need, off_bits, off_free, bytes;
  int words;
};
static PageAppendWs page_append_ws(int n, int max_pages, int n_pages) {
  auto up = [](size_t x) { return (x + 15) & ~size_t(15); };
  PageAppendWs w;
  w.words = (max_pages + 31) / 32;
  w.off_need = up((size_t)n * sizeof(AppendPlan));
  w.off_bits = w.off_need + up((size_t)n * 4);
  w.off_free = w.off_bits + up((size_t)n * w.words * 4);
  w.bytes = w.off_free + up((size_t)n_pages * 4);
  return w;
}
static size_t page_fork_ws(int n, int max_pages) {   // rows [n][max_pages], lengths [n] (-2: skipped)
  return (((size_t)n * max_pages * 4 + 15) & ~size_t(15)) + (((size_t)n * 4 + 15) & ~size_t(15));
}
static size_t page_compact_ws(int n_pages) {         // {moves}, from [n_pages], to [n_pages]
  return 16 + 2 * (((size_t)n_pages * 4 + 15) & ~size_t(15));
}
size_t pages_workspace_bytes(int n, int max_pages, int n_pages) {
  size_t b = page_append_ws(n, max_pages, n_pages).bytes;
  if (page_fork_ws(n, max_pages) > b) b = page_fork_ws(n, max_pages);
  if (page_compact_ws(n_pages) > b) b = page_compact_ws(n_pages);
  return b;
}

// One block.  Per listed sequence (a warp each): which table slots need a
// fresh page.  Decisions are taken on the reference counts as they stand when
// the call starts, kept as bit words, and applied once every sequence's
// decision is made.
__global__ void __launch_bounds__(kPlanThreads) page_append_plan_kernel(const PageAppendArgs a, AppendPlan *plans,
                                                                        int *need, uint32_t *bits, int words,
                                                                        int *free_list) {
  __shared__ int sm[kPlanWarps + 1];
  const PagePoolArgs &P = a.pool;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  // ---- per sequence: checks, and the slots that need a fresh page
  for (int i = warp; i < a.n; i += kPlanWarps) {
    const int s = a.seq[i];
    AppendPlan p{-1, 0, 0, -1};
    int nd = 0;
    bool bad = s < -1 || s >= P.n_seq;
    if (s >= 0 && !bad) {
      bool dup = false;
      for (int j = lane; j < i; j += 32) dup |= a.seq[j] == s;
      bad = __any_sync(0xffffffffu, dup);
    }
    if (s >= 0 && !bad) {
      const int old = P.n_entries[s];
      const int at = a.at ? a.at[i] : old;
      const int first = a.first ? a.first[i] : 0;
      int n_src = a.src_n[i];
      n_src = n_src < a.src_cap ? n_src : a.src_cap;
      const int cnt = n_src > first ? n_src - first : 0;
      const long long room = (long long)P.max_pages * P.page;
      if (first < 0 || at < 0 || at > old || old > room) {
        bad = true;
      } else if ((long long)at + cnt > room) {
        if (lane == 0) flag(P.status, CSA2_DEV_NO_PAGE);
      } else {
        const int keep = ceil_div(at, P.page), held = ceil_div(old, P.page), want = ceil_div(at + cnt, P.page);
        const int32_t *row = P.table + (size_t)s * P.max_pages;
        const bool part = at % P.page != 0 && cnt > 0;
        const int lo = keep > 0 ? keep - 1 : 0, hi = held < want ? held : want;
        bool broken = false;
        int cow = -1;
        for (int j0 = lo & ~31; j0 < hi; j0 += 32) {
          const int j = j0 + lane;
          bool fresh = false;
          int pg = -1;
          if (j >= lo && j < hi) {
            pg = row[j];
            if (pg < 0 || pg >= P.n_pages) broken = true;
            else if (P.refs[pg] > 1) fresh = j >= keep || part;
          }
          const uint32_t w = __ballot_sync(0xffffffffu, fresh);
          const uint32_t c = __ballot_sync(0xffffffffu, fresh && j < keep);
          if (c) cow = __shfl_sync(0xffffffffu, pg, __ffs(c) - 1);
          if (lane == 0) bits[(size_t)i * words + (j0 >> 5)] = w;
          nd += __popc(w);
        }
        if (__any_sync(0xffffffffu, broken)) {   // a table slot without a page: leave the sequence alone
          if (lane == 0) flag(P.status, CSA2_DEV_INDEX_RANGE);
          nd = 0;
        } else {
          const int from = held > keep ? held : keep;
          nd += want > from ? want - from : 0;
          p = AppendPlan{s, at, cnt, cow};
        }
      }
    }
    if (lane == 0) {
      if (bad) flag(P.status, CSA2_DEV_BAD_SEQUENCE);
      plans[i] = p;
      need[i] = nd;
    }
  }
  __syncthreads();
  // ---- the pages each sequence's share of the free list starts at
  int carry = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int total;
    const int v = i < a.n ? need[i] : 0;
    const int ex = block_exclusive(v, sm, &total);
    if (i < a.n) need[i] = carry + ex;   // from here on: the exclusive sum
    carry += total;
    __syncthreads();
  }
  const int wanted = carry;
  // ---- the lowest `wanted` free pages
  int found = 0;
  for (int q0 = 0; 4 * q0 < P.n_pages && found < wanted; q0 += kPlanThreads) {
    const int4 r = load_refs(P.refs, P.n_pages, q0 + tid);
    const int mine = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int total;
    int k = found + block_exclusive(mine, sm, &total);
    const int p0 = 4 * (q0 + tid);
    if (r.x == 0) free_list[k++] = p0;
    if (r.y == 0) free_list[k++] = p0 + 1;
    if (r.z == 0) free_list[k++] = p0 + 2;
    if (r.w == 0) free_list[k++] = p0 + 3;
    found += total;
    __syncthreads();
  }
  __syncthreads();
  // ---- apply: tables, counts, lengths
  for (int i = warp; i < a.n; i += kPlanWarps) {
    AppendPlan p = plans[i];
    if (p.seq < 0) continue;
    const int base = need[i];
    const int end = i + 1 < a.n ? need[i + 1] : wanted;
    if (end > base && end > found) {   // too few free pages: the sequence stays as it was
      if (lane == 0) {
        flag(P.status, CSA2_DEV_NO_PAGE);
        plans[i].seq = -1;
      }
      continue;
    }
    const int old = P.n_entries[p.seq];
    const int keep = ceil_div(p.at, P.page), held = ceil_div(old, P.page), want = ceil_div(p.at + p.cnt, P.page);
    int32_t *row = P.table + (size_t)p.seq * P.max_pages;
    const int lo = keep > 0 ? keep - 1 : 0, hi = held < want ? held : want;
    const int last = held > want ? held : want;
    int used = base;
    for (int j0 = lo & ~31; j0 < last; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t w = j0 < hi ? bits[(size_t)i * words + (j0 >> 5)] : 0u;
      const bool in = j >= lo && j < last;
      const bool fresh = in && j < want && (j >= held || ((w >> lane) & 1u));
      const bool drop = in && j < held && (fresh || j >= want);
      const uint32_t m = __ballot_sync(0xffffffffu, fresh);
      if (drop) {
        const int pg = row[j];
        if (pg >= 0 && pg < P.n_pages) atomicSub(P.refs + pg, 1);
      }
      if (fresh) {
        const int pg = free_list[used + __popc(m & ((1u << lane) - 1u))];
        row[j] = pg;
        atomicAdd(P.refs + pg, 1);
      } else if (in && j >= want) {
        row[j] = -1;
      }
      used += __popc(m);
    }
    __syncwarp();
    if (lane == 0) P.n_entries[p.seq] = p.at + p.cnt;
  }
}

// Copies of the planned entries: those kept of a shared page first, then the
// new ones.  grid (x, n): x blocks take turns of kCopyEntries entries of a
// sequence; the entries' places are looked up once per entry.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) page_append_copy_kernel(const PageAppendArgs a, const AppendPlan *plans) {
  __shared__ int from_row[kCopyEntries], to_row[kCopyEntries];
  const PagePoolArgs &P = a.pool;
  const int tid = threadIdx.x, i = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  const AppendPlan p = plans[i];
  if (p.seq < 0) return;
  const int kept = p.cow_src >= 0 ? p.at % P.page : 0;
  const int total = kept + p.cnt;
  const int32_t *row = P.table + (size_t)p.seq * P.max_pages;
  const int first = a.first ? a.first[i] : 0;
  constexpr int NC = D / 32, NS = D / 128;   // 16-byte pieces of an entry's codes, 8-byte pieces of its scales
  for (int e0 = blockIdx.x * kCopyEntries; e0 < total; e0 += gridDim.x * kCopyEntries) {
    if (tid < kCopyEntries && e0 + tid < total) {
      const int e = e0 + tid;
      const int dst = e < kept ? p.at - kept + e : p.at + (e - kept);   // entry of the pool sequence
      to_row[tid] = row[dst / P.page] * P.page + dst % P.page;
      from_row[tid] = e < kept ? -1 - (p.cow_src * P.page + e) : first + (e - kept);
    }
    __syncthreads();
    const int n = total - e0 < kCopyEntries ? total - e0 : kCopyEntries;
    auto pool_row = [](int f) { return -1 - f; };
    uint4 v[kCopyEntries * NC / kCopyThreads];
#pragma unroll
    for (int u = 0; u < kCopyEntries * NC / kCopyThreads; ++u) {
      const int k = tid + u * kCopyThreads, e = k / NC, c = k % NC;
      if (e < n) {
        const int f = from_row[e];
        const uint8_t *src = f < 0 ? P.codes + (size_t)pool_row(f) * (D / 2)
                                   : a.src_codes + ((size_t)i * a.src_cap + f) * (D / 2);
        v[u] = reinterpret_cast<const uint4 *>(src)[c];
      }
    }
    uint2 w[(kCopyEntries * NS + kCopyThreads - 1) / kCopyThreads];
#pragma unroll
    for (int u = 0; u < (kCopyEntries * NS + kCopyThreads - 1) / kCopyThreads; ++u) {
      const int k = tid + u * kCopyThreads, e = k / NS, c = k % NS;
      if (e < n) {
        const int f = from_row[e];
        const uint8_t *src = f < 0 ? P.scales + (size_t)pool_row(f) * (D / 16)
                                   : a.src_scales + ((size_t)i * a.src_cap + f) * (D / 16);
        w[u] = reinterpret_cast<const uint2 *>(src)[c];
      }
    }
#pragma unroll
    for (int u = 0; u < kCopyEntries * NC / kCopyThreads; ++u) {
      const int k = tid + u * kCopyThreads, e = k / NC, c = k % NC;
      if (e < n) reinterpret_cast<uint4 *>(P.codes + (size_t)to_row[e] * (D / 2))[c] = v[u];
    }
#pragma unroll
    for (int u = 0; u < (kCopyEntries * NS + kCopyThreads - 1) / kCopyThreads; ++u) {
      const int k = tid + u * kCopyThreads, e = k / NS, c = k % NS;
      if (e < n) reinterpret_cast<uint2 *>(P.scales + (size_t)to_row[e] * (D / 16))[c] = w[u];
    }
    __syncthreads();
  }
}

cudaError_t launch_page_append(const PageAppendArgs &a, void *ws, int sms, cudaStream_t s) {
  const PageAppendWs w = page_append_ws(a.n, a.pool.max_pages, a.pool.n_pages);
  uint8_t *b = static_cast<uint8_t *>(ws);
  AppendPlan *plans = reinterpret_cast<AppendPlan *>(b);
  cudaError_t e = launch_pdl(page_append_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, dim3(1, 1, 1), a, plans,
                             reinterpret_cast<int *>(b + w.off_need), reinterpret_cast<uint32_t *>(b + w.off_bits),
                             w.words, reinterpret_cast<int *>(b + w.off_free));
  if (e != cudaSuccess) return e;
  // enough blocks for every SM, none beyond the turns the longest sequence can take
  const int turns = (a.src_cap + a.pool.page + kCopyEntries - 1) / kCopyEntries;
  int gx = (8 * sms + a.n - 1) / a.n;
  if (gx > turns) gx = turns;
  const dim3 grid(gx, a.n), block(kCopyThreads), one(1, 1, 1);
  switch (a.pool.D) {
    case 128: return launch_pdl(page_append_copy_kernel<128>, grid, block, 0, s, one, a, plans);
    case 256: return launch_pdl(page_append_copy_kernel<256>, grid, block, 0, s, one, a, plans);
    default: return launch_pdl(page_append_copy_kernel<512>, grid, block, 0, s, one, a, plans);
  }
}

// ------------------------------------------------------------------ fork / free

// Every child's new row is taken (and its pages' counts raised) before any row
// is overwritten, so that a sequence can be a parent and a child in one call.

// Whether pair j sets child c: a pair whose parent is out of range does not use
// up its child.
__device__ __forceinline__ bool pair_sets(const PageForkArgs &a, int j, int c) {
  if (a.child[j] != c) return false;
  const int p = a.parent[j];
  return p >= -1 && p < a.pool.n_seq;
}

// Short lists: one cluster, pair i in block i % 8, with a cluster barrier between
// the two halves and the taken rows in registers.  One launch instead of two:
// 6.9 us a call instead of 9.8 (8 sequences of 40 pages, back to back: what the
// host takes for it; 3.9 us in a replayed graph).
constexpr int kForkBlocks = 8, kForkSlots = 8;   // blocks of the cluster; slots per thread
__global__ void __launch_bounds__(kPlanThreads) page_fork_kernel(const PageForkArgs a) {
  const PagePoolArgs &P = a.pool;
  __shared__ int parent[kPlanWarps], child[kPlanWarps], len[kPlanWarps];   // of the block's pairs; len -2: skipped
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int i = rank + kForkBlocks * warp;
  if (i < a.n) {
    const int p = a.parent[i], c = a.child[i];
    bool bad = p < -1 || p >= P.n_seq || c < 0 || c >= P.n_seq;
    for (int j = lane; j < i; j += 32) bad |= pair_sets(a, j, c);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (bad) flag(P.status, CSA2_DEV_BAD_SEQUENCE);
      parent[warp] = p;
      child[warp] = c;
      len[warp] = bad ? -2 : (p < 0 ? 0 : P.n_entries[p]);
    }
  }
  __syncthreads();
  const int slots = a.n > rank ? (a.n - rank + kForkBlocks - 1) / kForkBlocks * P.max_pages : 0;
  int pg[kForkSlots];
#pragma unroll
  for (int u = 0; u < kForkSlots; ++u) {
    const int x = tid + u * kPlanThreads, r = x / P.max_pages;
    pg[u] = -1;
    if (x < slots && len[r] >= -1 && parent[r] >= 0) pg[u] = P.table[(size_t)parent[r] * P.max_pages + x % P.max_pages];
    if (pg[u] >= P.n_pages) pg[u] = -1;
  }
#pragma unroll
  for (int u = 0; u < kForkSlots; ++u)
    if (pg[u] >= 0) atomicAdd(P.refs + pg[u], 1);
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
  for (int u = 0; u < kForkSlots; ++u) {
    const int x = tid + u * kPlanThreads, r = x / P.max_pages;
    if (x >= slots || len[r] < -1) continue;
    int32_t *slot = P.table + (size_t)child[r] * P.max_pages + x % P.max_pages;
    const int old = *slot;
    if (old >= 0 && old < P.n_pages) atomicSub(P.refs + old, 1);
    *slot = pg[u];
  }
  if (lane == 0 && i < a.n && len[warp] >= -1) P.n_entries[child[warp]] = len[warp];
}

// Long lists: one block per pair, twice.
__global__ void __launch_bounds__(kCopyThreads) page_fork_take_kernel(const PageForkArgs a, int32_t *rows, int32_t *lens) {
  const PagePoolArgs &P = a.pool;
  const int tid = threadIdx.x, i = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int p = a.parent[i], c = a.child[i];
  bool dup = false;
  for (int j = tid; j < i; j += kCopyThreads) dup |= pair_sets(a, j, c);
  const bool bad = __syncthreads_or(dup) || p < -1 || p >= P.n_seq || c < 0 || c >= P.n_seq;
  if (tid == 0) {
    if (bad) flag(P.status, CSA2_DEV_BAD_SEQUENCE);
    lens[i] = bad ? -2 : (p < 0 ? 0 : P.n_entries[p]);
  }
  if (bad) return;
  int32_t *out = rows + (size_t)i * P.max_pages;
  for (int j = tid; j < P.max_pages; j += kCopyThreads) {
    int pg = p < 0 ? -1 : P.table[(size_t)p * P.max_pages + j];
    if (pg >= P.n_pages) pg = -1;
    if (pg >= 0) atomicAdd(P.refs + pg, 1);
    out[j] = pg;
  }
}

__global__ void __launch_bounds__(kCopyThreads) page_fork_put_kernel(const PageForkArgs a, const int32_t *rows,
                                                                     const int32_t *lens) {
  const PagePoolArgs &P = a.pool;
  const int tid = threadIdx.x, i = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int len = lens[i];
  if (len < -1) return;
  const int c = a.child[i];
  int32_t *row = P.table + (size_t)c * P.max_pages;
  for (int j = tid; j < P.max_pages; j += kCopyThreads) {
    const int old = row[j];
    if (old >= 0 && old < P.n_pages) atomicSub(P.refs + old, 1);
    row[j] = rows[(size_t)i * P.max_pages + j];
  }
  if (tid == 0) P.n_entries[c] = len;
}

cudaError_t launch_page_fork(const PageForkArgs &a, void *ws, cudaStream_t s) {
  const int pairs = (a.n + kForkBlocks - 1) / kForkBlocks;   // of a block, at most
  if (pairs <= kPlanWarps && (long long)pairs * a.pool.max_pages <= kForkSlots * kPlanThreads)
    return launch_pdl(page_fork_kernel, dim3(kForkBlocks), dim3(kPlanThreads), 0, s, dim3(kForkBlocks, 1, 1), a);
  int32_t *rows = static_cast<int32_t *>(ws);
  int32_t *lens = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) +
                                              (((size_t)a.n * a.pool.max_pages * 4 + 15) & ~size_t(15)));
  cudaError_t e = launch_pdl(page_fork_take_kernel, dim3(a.n), dim3(kCopyThreads), 0, s, dim3(1, 1, 1), a, rows, lens);
  if (e != cudaSuccess) return e;
  return launch_pdl(page_fork_put_kernel, dim3(a.n), dim3(kCopyThreads), 0, s, dim3(1, 1, 1), a,
                    (const int32_t *)rows, (const int32_t *)lens);
}

// ------------------------------------------------------------------ compact

// One block: L = live pages; the k-th live page at or above L moves to the
// k-th hole below L (as many of the one as of the other, and no page is both
// a source and a target, so the moves need no order).
__global__ void __launch_bounds__(kPlanThreads) page_compact_plan_kernel(const PagePoolArgs P, int32_t *n_live,
                                                                         int32_t *head, int32_t *from, int32_t *to) {
  __shared__ int sm[kPlanWarps + 1];
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int quads = (P.n_pages + 3) / 4;
  int mine = 0;
  for (int q = tid; q < quads; q += kPlanThreads) {
    const int4 r = load_refs(P.refs, P.n_pages, q);
    mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  int L;
  block_exclusive(mine, sm, &L);
  __syncthreads();
  // one pass: holes below L and live pages above it are counted in the two
  // halves of one integer (at most n_pages / 1024 of each per thread and pass)
  int holes = 0, lives = 0;
  for (int q0 = 0; q0 < quads; q0 += kPlanThreads) {
    const int4 r = q0 + tid < quads ? load_refs(P.refs, P.n_pages, q0 + tid) : make_int4(-1, -1, -1, -1);
    const int p0 = 4 * (q0 + tid);
    const int v[4] = {r.x, r.y, r.z, r.w};
    int h = 0, l = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      h += v[u] == 0 && p0 + u < L;
      l += v[u] > 0 && p0 + u >= L;
    }
    int total;
    const int ex = block_exclusive(h | (l << 16), sm, &total);
    int kh = holes + (ex & 0xFFFF), kl = lives + (ex >> 16);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (v[u] == 0 && p0 + u < L) to[kh++] = p0 + u;
      if (v[u] > 0 && p0 + u >= L) from[kl++] = p0 + u;
    }
    holes += total & 0xFFFF;
    lives += total >> 16;
    __syncthreads();
  }
  if (tid == 0) {
    // as many of the one as of the other, unless a count is negative (such a
    // page is neither): only what has both ends moves
    if (lives != holes) flag(P.status, CSA2_DEV_INDEX_RANGE);
    head[0] = lives < holes ? lives : holes;
    head[1] = L;
    if (n_live) *n_live = L;
  }
}

// Data in pieces of 8 KB (so that few moves still fill the GPU), then the
// tables: a slot whose page moved finds it by bisection.
__global__ void __launch_bounds__(kCopyThreads) page_compact_move_kernel(const PagePoolArgs P, const int32_t *head,
                                                                         const int32_t *from, const int32_t *to) {
  constexpr int kPiece = 512;   // 16-byte units
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int moves = head[0], L = head[1];
  if (moves == 0) return;
  const int cu = P.page * P.D / 32, su = P.page * P.D / 256;   // 16-byte units of a page's codes and scales
  const int cp = (cu + kPiece - 1) / kPiece, sp = (su + kPiece - 1) / kPiece;
  const long long items = (long long)moves * (cp + sp);
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int k = (int)(it / (cp + sp)), pc = (int)(it % (cp + sp));
    const int f = from[k], t = to[k];
    const bool sc = pc >= cp;
    const int n = sc ? su : cu, u0 = (sc ? pc - cp : pc) * kPiece;
    const uint4 *src = reinterpret_cast<const uint4 *>(sc ? P.scales : P.codes) + (size_t)f * n;
    uint4 *dst = reinterpret_cast<uint4 *>(sc ? P.scales : P.codes) + (size_t)t * n;
    uint4 v[kPiece / kCopyThreads];
#pragma unroll
    for (int u = 0; u < kPiece / kCopyThreads; ++u) {
      const int x = u0 + tid + u * kCopyThreads;
      if (x < n) v[u] = src[x];
    }
#pragma unroll
    for (int u = 0; u < kPiece / kCopyThreads; ++u) {
      const int x = u0 + tid + u * kCopyThreads;
      if (x < n) dst[x] = v[u];
    }
    if (pc == 0 && tid == 0) {
      P.refs[t] = P.refs[f];
      P.refs[f] = 0;
    }
  }
  const long long slots = (long long)P.n_seq * P.max_pages;
  for (long long x = (long long)blockIdx.x * kCopyThreads + tid; x < slots; x += (long long)gridDim.x * kCopyThreads) {
    const int pg = P.table[x];
    if (pg < L || pg >= P.n_pages) continue;
    int lo = 0, hi = moves - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (from[mid] < pg) lo = mid + 1;
      else hi = mid;
    }
    if (from[lo] == pg) P.table[x] = to[lo];
    else flag(P.status, CSA2_DEV_INDEX_RANGE);   // a slot that holds a page without references (or one that could not move)
  }
}

cudaError_t launch_page_compact(const PagePoolArgs &p, int32_t *n_live, void *ws, int sms, cudaStream_t s) {
  int32_t *head = static_cast<int32_t *>(ws);
  int32_t *from = head + 4;
  int32_t *to = from + (((size_t)p.n_pages * 4 + 15) & ~size_t(15)) / 4;
  cudaError_t e = launch_pdl(page_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, dim3(1, 1, 1), p, n_live,
                             head, from, to);
  if (e != cudaSuccess) return e;
  return launch_pdl(page_compact_move_kernel, dim3(8 * sms), dim3(kCopyThreads), 0, s, dim3(1, 1, 1), p,
                    (const int32_t *)head, (const int32_t *)from, (const int32_t *)to);
}

}  // namespace csa2
