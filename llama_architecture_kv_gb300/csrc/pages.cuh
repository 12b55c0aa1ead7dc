// Page tables whose rows fork, shrink, grow and are freed, and copies of pages (declarations).
#pragma once
#include "qcache.cuh"

namespace llm {

// Row r holds length[r] positions in pages table[r][0 .. ceil(length / kPage) - 1] of a pool of `pages`.
struct PageBook {
  int32_t* table;   // [rows][per_row]
  int32_t* length;  // [rows]
  int32_t rows, per_row, pages;
};

// ints of workspace that an update or a compaction of such a book needs
uint64_t pages_workspace(int rows, int pages);
cudaError_t launch_pages_update(const PageBook& from, const PageBook& to, const int32_t* parent, const int32_t* length,
                                int32_t* moves, int32_t* counts, int32_t* ws, int32_t* status, cudaStream_t s);
cudaError_t launch_pages_compact(const PageBook& from, const PageBook& to, int32_t* moves, int32_t* counts, int32_t* ws,
                                 int32_t* status, cudaStream_t s);

// Copies of pages in the caches of up to kCopyLayers layers: `bytes` per position of a key/value head in
// k and v [rows][kv][cap], and scales [rows][kv][cap / kQBlock] where there are some.
constexpr int kCopyLayers = 96;  // (their addresses are kernel arguments: 3 KB of the 4 that every driver takes)
struct CopyArgs {
  uint8_t *k[kCopyLayers], *v[kCopyLayers];
  float *ks[kCopyLayers], *vs[kCopyLayers];  // null: no scales
  int32_t layers, rows, kv, cap, bytes;
  const int32_t* moves;   // [m][2] from, to; negative: none
  int32_t m;
  const int32_t* counts;  // how many of them there are, or null: m
  int32_t* status;
};
cudaError_t launch_copy_pages(const CopyArgs& a, cudaStream_t s);

}  // namespace llm
