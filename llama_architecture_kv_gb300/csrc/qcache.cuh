// 8-bit key/value caches: e4m3 codes with one power-of-two scale per block of kQBlock positions
// and key/value head (declarations and the device helpers its kernels share).
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace llm {

constexpr int kQBlock = 16;  // positions that share a scale; a page holds kPage / kQBlock blocks

// The cache of one layer: codes [rows][kv][cap][hd], scales [rows][kv][cap / kQBlock]; cap is a
// multiple of kQBlock.  The value of a code is its e4m3 value times its block's scale.
struct QCacheView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int32_t rows, kv, cap, hd;
};

// The rows of a call.  Without a step: row b holds `first[b]` (a first position, or a length) and
// `count[b]` tokens (S where count is null), its positions found through table [B][stride] or, with
// no table, in cache row b; everything read from device memory is checked against these bounds and
// an error is recorded in *status (where given).  With a step: row b is row entry0 + b * entry_step of a
// decode step, or that entry of a prefill pass, of a handle (common.cuh), which the host has validated.
struct QRows {
  const int32_t* first;
  const int32_t* count;
  const int32_t* table;
  int32_t stride;
  int32_t B, S;
  int32_t limit;         // positions a row can hold
  const StepState* step;
  int32_t* status;
  int32_t entry0, entry_step;  // with a step (0 and 1 but for a verification pass, which takes one token
                               // of every row at a time)
};
LLM_D int q_entry(const QRows& r, int b) { return r.entry0 + b * r.entry_step; }

// device error codes (same values as llm.h)
constexpr int32_t kErrPosRange = 4;
constexpr int32_t kErrArg = 7;

LLM_D void q_report(int32_t* status, int32_t code) {
  if (status) atomicCAS(status, 0, code);
}

// tokens of row b (0 with an error recorded when the count is outside 0..S)
LLM_D int q_count(const QRows& r, int b) {
  if (!r.count) return r.S;
  const int n = r.count[b];
  if (n >= 0 && n <= r.S) return n;
  q_report(r.status, kErrArg);
  return 0;
}

// the cache row and position of position pos inside pool page `page`; false outside the pool
LLM_HD bool q_page_slot(int rows, int cap, int page, int pos, int& row, int& pp) {
  const int per_row = cap / kPage;
  if (page < 0 || page >= rows * per_row) return false;
  row = page / per_row;
  pp = (page - row * per_row) * kPage + (pos & (kPage - 1));
  return true;
}

// the cache row and position that hold position pos of row b; false (with an error recorded) for
// a page outside the pool
LLM_D bool q_place(const QRows& r, const QCacheView& c, int b, int pos, int& row, int& pp) {
  if (!r.table) {
    row = b;
    pp = pos;
    return true;
  }
  if (q_page_slot(c.rows, c.cap, r.table[(size_t)b * r.stride + pos / kPage], pos, row, pp)) return true;
  q_report(r.status, kErrArg);
  return false;
}

// ---- e4m3 ---------------------------------------------------------------------------------
// two f32 to e4m3 codes (lo in the low byte), to nearest even; callers keep |x| <= 448
LLM_D uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// the values of the two codes in the low half of x (exact in f16)
LLM_D float2 e4m3_pair(uint32_t x) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
LLM_D float4 e4m3_quad(uint32_t x) {
  const float2 a = e4m3_pair(x), b = e4m3_pair(x >> 16);
  return make_float4(a.x, a.y, b.x, b.y);
}

// two f32 rounded to bf16 (x0 in the low half)
LLM_D uint32_t bf16x2(float x0, float x1) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x1), "f"(x0));
  return r;
}

// the least power of two s >= 2^-126 with amax / s <= 448 = 1.75 * 2^8 (amax finite, >= 0)
LLM_D float q_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 8;                 // amax = 1.m * 2^(e + 8 - 127)
  if ((u & 0x7fffffu) > 0x600000u) ++e;       // 1.m > 1.75
  return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}
// 1 / s for a power of two s in 2^-126 .. 2^120
LLM_D float q_recip(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// blocks that S tokens can touch
LLM_HD int q_span(int S) { return (S - 1) / kQBlock + ((S - 1) % kQBlock ? 2 : 1); }

// ---- launches -----------------------------------------------------------------------------
bool qcache_head_supported(int hd);
// (B * q_span(S) * kv * 2, the warps of a write or read, below 2^31: the callers check)
// keys and values of a call's tokens into the cache: rows of `stride` elements, bf16 (st 1) or f32
cudaError_t launch_qcache_write(const QCacheView& c, const QRows& r, const void* k, const void* v, int st,
                                int64_t stride, cudaStream_t s);
// the same for the rows of a handle's step, or the entries of a prefill pass: staged [B][kv][hd]
cudaError_t launch_qcache_write_step(const QCacheView& c, const QRows& r, const void* k, const void* v, int st,
                                     cudaStream_t s, bool pdl);
// Verification passes: entry b * T + i of the step is token i of row b.  keep: the codes and scales of the
// blocks that the rows' first tokens go into (where their positions before hold something) to the kept_*
// arrays; settle: after accepted[b] of the T - 1 drafts were kept, the block that ends with the last of the kept
// tokens as if no other had been written, from what was kept and the tokens' staged values, and the blocks behind it
// empty.
struct QVerify {
  QCacheView c;                // layer 0; the others follow
  int32_t layers, T;
  QRows r;                     // with a step; entry_step = T
  uint8_t *kept_k, *kept_v;    // [layers][rows][kv][kQBlock][hd]
  float *kept_ks, *kept_vs;    // [layers][rows][kv]
  const void *stage_k, *stage_v;  // [layers][stage_rows][kv][hd], bf16 (st 1) or f32
  int64_t stage_rows;
  const int32_t* accepted;
};
cudaError_t launch_qcache_keep(const QVerify& v, cudaStream_t s);
cudaError_t launch_qcache_settle(const QVerify& v, int st, cudaStream_t s);
// the scales of block blk of cache row `row` to 0 in `layers` caches that follow one another, c the first
cudaError_t launch_qcache_clear(const QCacheView& c, int layers, int row, int blk, cudaStream_t s);
cudaError_t launch_qcache_read(const QCacheView& c, const QRows& r, void* k, void* v, int st, int64_t stride,
                               cudaStream_t s);

// attention of the rows' tokens (a row's `first` is its length): q and out are rows of H * hd
// elements (H = kv * g) at the given strides, f32 (qt 0) or bf16 (qt 1)
struct QAttnArgs {
  QCacheView c;
  QRows r;
  const void* q;
  void* out;
  int64_t q_stride, out_stride;
  int32_t g;
  float scale;
  unsigned char* ws;      // workspace (qattn_workspace bytes): tickets zero between calls, then partials
  const int32_t* tiles;   // a prefill pass's tiles (attention.cuh), of at most qattn_tile_tokens(g) tokens, or null
  int32_t krow0;          // row of the cache's position 0 of (row 0, kv head 0) in the tensor maps (step calls)
  // a decode step's keys and values [B][kv][hd] of type new_t (0 f32, 1 bf16), which the attention itself
  // quantises into the cache (tensor cores only); null where they are there already
  const void *new_k, *new_v;
  int32_t new_t;
  // set by launch_qattn: parts of a token's positions (CUDA cores), or tokens per tile and tiles per row
  int32_t splits, tpt, nct;
};
constexpr int kQattnTickets = 4096;  // bytes of tickets (one 32-bit word per CTA) before the partials
// whether the tiles of a call can be counted in 31 bits
bool qattn_fits(const QCacheView& c, int g, int qt, int B, int S, int limit, int num_sms);
uint64_t qattn_workspace(const QCacheView& c, int g, int B, int S, int num_sms);
// the same for the steps and passes of at most NT rows of a handle (f32 queries)
uint64_t qattn_step_workspace(const QCacheView& c, int g, int NT, int num_sms);
// kmap, vmap: tensor maps of qattn_make_map over the whole caches; null: made for this call
cudaError_t launch_qattn(const QAttnArgs& a, int qt, int num_sms, cudaStream_t s, bool pdl,
                         const CUtensorMap* kmap = nullptr, const CUtensorMap* vmap = nullptr);
bool qattn_uses_tc(int hd);
bool qattn_make_map(CUtensorMap* map, const void* codes, int hd, uint64_t rows);
// tokens of one sequence that share a tile of the tensor-core kernel (f32 queries)
int qattn_tile_tokens(int g);

}  // namespace llm
