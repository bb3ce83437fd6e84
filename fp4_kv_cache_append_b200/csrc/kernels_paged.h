// Launches of the paged cache (pages.cu) and of the dense attentions
// (attn_dense.cu, attn_window.cu).
#pragma once
#include "kernels.h"

namespace csa2 {

// Paged FP4 cache (see csa2_page_pool).
struct PagePoolArgs {
  uint8_t *codes, *scales;
  int32_t *refs, *table, *n_entries;
  int n_pages, page, n_seq, max_pages, D, m;
  unsigned int *status;
};
struct PageAppendArgs {
  PagePoolArgs pool;
  const uint8_t *src_codes, *src_scales;   // [n][src_cap][..]
  const int32_t *src_n, *first, *seq, *at; // [n]; first / at may be nullptr
  int n, src_cap;
};
struct PageForkArgs {
  PagePoolArgs pool;
  const int32_t *parent, *child;           // [n]
  int n;
};
constexpr int kPageListMax = 4096;         // listed sequences of one call
size_t pages_workspace_bytes(int n, int max_pages, int n_pages);
cudaError_t launch_page_append(const PageAppendArgs &a, void *ws, int sms, cudaStream_t s);
cudaError_t launch_page_fork(const PageForkArgs &a, void *ws, cudaStream_t s);
cudaError_t launch_page_compact(const PagePoolArgs &p, int32_t *n_live, void *ws, int sms, cudaStream_t s);

// Dense attentions: every entry of paged sequences (a shared prefix once for
// all) and / or the rows of a window ring and its first tokens.
struct DenseAttnArgs {
  PagePoolArgs pool;        // codes == nullptr: no entries
  const int32_t *seq;       // [B] pool sequence of each batch row
  int n_shared;
  const uint8_t *swa_rows;  // [B][W_cap][D] or nullptr
  float s_swa;
  int W_cap, window;
  const uint8_t *sink_rows; // [B][sink_cap][D] or nullptr: token s in row s
  float s_sink;
  int n_sink, sink_cap;
  const uint16_t *q;        // [B][T_q][H][D]
  const int32_t *q_pos;     // [B][T_q]
  int B, T_q, H, D;
  float scale;
  uint16_t *out;            // [B][T_q][H][D]
  void *ws;
  unsigned int *status;
};
size_t prefix_attn_workspace_bytes(int B, int T_q, int H, int D, int sms);
// Entries that a copy of the pool's planes takes: the largest of 16, 32 and 64
// that divides the page.
inline int prefix_attn_box(int page) { return page % 64 == 0 ? 64 : (page % 32 == 0 ? 32 : 16); }
struct DenseMaps {
  CUtensorMap q;            // rows of D bf16, boxes of 128 rows x 64 channels in the 128B swizzle
  // the pool's planes, rows = entries (two entries for the scales of D 128);
  // boxes of prefix_attn_box entries x 256 channels at most, the codes in the
  // swizzle of the box's width
  CUtensorMap codes, scales;
  CUtensorMap swa, sinks;   // rows of D bytes, boxes of 64 rows x 128 channels in the 128B swizzle
};
cudaError_t launch_prefix_attn(const DenseMaps &m, const DenseAttnArgs &a, int sms, cudaStream_t s);
size_t window_attn_workspace_bytes(int B, int T_q, int H, int D, int window, int n_sink, int sms);
cudaError_t launch_window_attn(const DenseMaps &m, const DenseAttnArgs &a, int sms, cudaStream_t s);
// The resident form (attn_window.cu), for the launches it takes.
bool window_takes_ring(const DenseAttnArgs &a, int sms);
cudaError_t launch_window_ring(const CUtensorMap &q_map, const DenseAttnArgs &a, int sms, cudaStream_t s);

}  // namespace csa2
