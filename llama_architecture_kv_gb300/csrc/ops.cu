// Entry points of the operators that need no handle (include/llm.h): 8-bit key/value caches, page tables
// that fork, the verification of drafted tokens and the sampler with settings per row.  Each checks its arguments on the host, then launches on the
// caller's stream; what only device memory knows (positions, counts, pages) the kernels check.
#include <math.h>
#include <stdio.h>

#include "attention.cuh"
#include "llm.h"
#include "pages.cuh"
#include "qcache.cuh"
#include "sampler.cuh"
#include "verify.cuh"

using namespace llm;

namespace llm {
llm_status fail_thread(llm_status s, const char* why);  // llm.cu
}

namespace {

#define REFUSE(cond, status, why) \
  if (cond) return fail_thread(status, why)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

llm_status check_cache(const llm_qcache* c) {
  REFUSE(!c->k || !c->v || !c->k_scale || !c->v_scale, LLM_ERR_ARG, "NULL cache memory");
  REFUSE(c->rows < 1 || c->kv_heads < 1, LLM_ERR_CONFIG, "a cache has at least one row and one key/value head");
  REFUSE(!qcache_head_supported(c->head), LLM_ERR_CONFIG, "head size must be 16, 32, 64, 128 or 256");
  REFUSE(c->max_seq < kQBlock || c->max_seq % kQBlock, LLM_ERR_CONFIG, "max_seq must be a positive multiple of 16");
  REFUSE((int64_t)c->rows * c->kv_heads >= ((int64_t)1 << 31) / c->max_seq, LLM_ERR_CONFIG,
         "rows x kv heads x positions must be below 2^31");
  REFUSE(!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale), LLM_ERR_ARG,
         "codes must be aligned to 16 bytes, scales to 4");
  return LLM_OK;
}

// the rows of a call: B rows of at most S tokens, `first` positions or lengths, optional counts and pages
llm_status check_rows(const llm_qcache* c, int32_t B, int32_t S, const int32_t* first, const int32_t* count,
                      const int32_t* table, int32_t pages_per_row, int32_t* status, QCacheView* view, QRows* rows) {
  REFUSE(!first, LLM_ERR_ARG, "NULL positions or lengths");
  REFUSE(B < 1 || (!table && B > c->rows), LLM_ERR_BATCH, "batch must be at least 1, and at most the cache's rows without a page table");
  REFUSE(S < 1, LLM_ERR_ARG, "tokens per row must be at least 1");
  REFUSE((int64_t)B * S >= (int64_t)1 << 31, LLM_ERR_ARG, "rows x tokens must be below 2^31");
  if (table) {
    REFUSE(c->max_seq % kPage, LLM_ERR_CONFIG, "pages need max_seq to be a multiple of 64");
    REFUSE(pages_per_row < 1 || (int64_t)pages_per_row * kPage * c->kv_heads > 0x7fffffff - 1024, LLM_ERR_ARG,
           "pages per row must be at least 1, and their positions x kv heads below 2^31 - 1024");
  }
  REFUSE(!aligned4(first) || !aligned4(count) || !aligned4(table) || !aligned4(status), LLM_ERR_ARG, "int32 arrays must be aligned");
  *view = QCacheView{(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale, c->v_scale, c->rows, c->kv_heads, c->max_seq, c->head};
  *rows = QRows{first, count, table, pages_per_row, B, S, table ? pages_per_row * kPage : c->max_seq, nullptr, status};
  return LLM_OK;
}

// writes and reads take a warp per block, head and side
llm_status check_warps(const QCacheView& c, const QRows& r) {
  REFUSE((int64_t)r.B * q_span(r.S) >= ((int64_t)1 << 30) / c.kv, LLM_ERR_ARG,
         "too large for one call: rows x blocks of 16 tokens x kv heads must stay below 2^30");
  return LLM_OK;
}

// rows of `width` elements, `stride` elements apart, of a 16-byte aligned buffer
llm_status check_buffer(const void* p, int32_t dtype, int64_t stride, int64_t width) {
  REFUSE(!p, LLM_ERR_ARG, "NULL buffer");
  REFUSE(dtype != LLM_DTYPE_F32 && dtype != LLM_DTYPE_BF16, LLM_ERR_ARG, "dtype must be LLM_DTYPE_F32 or LLM_DTYPE_BF16");
  REFUSE(stride < width, LLM_ERR_ARG, "rows overlap: the stride is below the row's width");
  REFUSE(!aligned16(p) || (stride * (dtype == LLM_DTYPE_BF16 ? 2 : 4)) % 16, LLM_ERR_ARG,
         "buffers and their strides must be multiples of 16 bytes");
  return LLM_OK;
}

llm_status launched(cudaError_t e) {
  if (e == cudaSuccess) return LLM_OK;
  cudaGetLastError();
  return fail_thread(LLM_ERR_CUDA, cudaGetErrorString(e));
}

llm_status device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return launched(e);
}

#define TRY(x)                   \
  do {                           \
    llm_status s_ = (x);         \
    if (s_ != LLM_OK) return s_; \
  } while (0)

}  // namespace

extern "C" {

llm_status llm_qcache_write(const llm_qcache* cache, const void* k_dev, const void* v_dev, int32_t dtype, int64_t stride,
                            int32_t B, int32_t S, const int32_t* pos_dev, const int32_t* count_dev,
                            const int32_t* table_dev, int32_t pages_per_row, int32_t* status_dev, void* cuda_stream) {
  REFUSE(!cache, LLM_ERR_ARG, "NULL cache");
  QCacheView c;
  QRows r;
  TRY(check_cache(cache));
  TRY(check_rows(cache, B, S, pos_dev, count_dev, table_dev, pages_per_row, status_dev, &c, &r));
  TRY(check_warps(c, r));
  TRY(check_buffer(k_dev, dtype, stride, (int64_t)c.kv * c.hd));
  TRY(check_buffer(v_dev, dtype, stride, (int64_t)c.kv * c.hd));
  return launched(launch_qcache_write(c, r, k_dev, v_dev, dtype, stride, (cudaStream_t)cuda_stream));
}

llm_status llm_qcache_read(const llm_qcache* cache, int32_t B, int32_t S, const int32_t* pos_dev,
                           const int32_t* count_dev, const int32_t* table_dev, int32_t pages_per_row, void* k_dev,
                           void* v_dev, int32_t dtype, int64_t stride, int32_t* status_dev, void* cuda_stream) {
  REFUSE(!cache, LLM_ERR_ARG, "NULL cache");
  QCacheView c;
  QRows r;
  TRY(check_cache(cache));
  TRY(check_rows(cache, B, S, pos_dev, count_dev, table_dev, pages_per_row, status_dev, &c, &r));
  TRY(check_warps(c, r));
  TRY(check_buffer(k_dev, dtype, stride, (int64_t)c.kv * c.hd));
  TRY(check_buffer(v_dev, dtype, stride, (int64_t)c.kv * c.hd));
  return launched(launch_qcache_read(c, r, k_dev, v_dev, dtype, stride, (cudaStream_t)cuda_stream));
}

llm_status llm_qcache_workspace(const llm_qcache* cache, int32_t group, int32_t B, int32_t S, uint64_t* bytes) {
  REFUSE(!cache || !bytes, LLM_ERR_ARG, "NULL argument");
  TRY(check_cache(cache));
  REFUSE(!attn_supported(cache->head, group), LLM_ERR_CONFIG, "group must be 1..16 with group x head size at most 1024");
  REFUSE(B < 1, LLM_ERR_BATCH, "batch must be at least 1");
  REFUSE(S < 1 || (int64_t)B * S >= (int64_t)1 << 31, LLM_ERR_ARG, "tokens per row out of range");
  int sms = 0;
  TRY(device_sms(&sms));
  const QCacheView c = {nullptr, nullptr, nullptr, nullptr, cache->rows, cache->kv_heads, cache->max_seq, cache->head};
  *bytes = qattn_workspace(c, group, B, S, sms);
  return LLM_OK;
}

llm_status llm_qcache_attend(const llm_qcache* cache, const void* q_dev, int32_t dtype, int64_t q_stride, int32_t group,
                             int32_t B, int32_t S, const int32_t* length_dev, const int32_t* count_dev,
                             const int32_t* table_dev, int32_t pages_per_row, float scale, void* out_dev,
                             int64_t out_stride, void* workspace_dev, uint64_t workspace_bytes, int32_t* status_dev,
                             void* cuda_stream) {
  REFUSE(!cache, LLM_ERR_ARG, "NULL cache");
  QAttnArgs a = {};
  TRY(check_cache(cache));
  TRY(check_rows(cache, B, S, length_dev, count_dev, table_dev, pages_per_row, status_dev, &a.c, &a.r));
  REFUSE(!attn_supported(cache->head, group), LLM_ERR_CONFIG, "group must be 1..16 with group x head size at most 1024");
  const int64_t width = (int64_t)a.c.kv * group * a.c.hd;
  TRY(check_buffer(q_dev, dtype, q_stride, width));
  TRY(check_buffer(out_dev, dtype, out_stride, width));
  REFUSE(!isfinite(scale), LLM_ERR_ARG, "scale must be finite");
  int sms = 0;
  TRY(device_sms(&sms));
  REFUSE(!qattn_fits(a.c, group, dtype, B, S, a.r.limit, sms), LLM_ERR_ARG,
         "too large for one call: rows x tokens x kv heads x 128-position tiles must stay below 2^31");
  const uint64_t need = qattn_workspace(a.c, group, B, S, sms);
  if (need > 0) {
    REFUSE(!workspace_dev || workspace_bytes < need, LLM_ERR_ARG, "workspace smaller than llm_qcache_workspace says");
    REFUSE(!aligned16(workspace_dev), LLM_ERR_ARG, "the workspace must be aligned to 16 bytes");
  }
  a.q = q_dev; a.out = out_dev; a.q_stride = q_stride; a.out_stride = out_stride; a.g = group; a.scale = scale;
  a.ws = (unsigned char*)workspace_dev;
  return launched(launch_qattn(a, dtype, sms, (cudaStream_t)cuda_stream, false));
}

llm_status llm_qcache_shared_workspace(const llm_qcache* cache, int32_t group, int32_t B, int32_t S, int32_t groups, uint64_t* bytes) {
  REFUSE(!cache || !bytes, LLM_ERR_ARG, "NULL argument");
  TRY(check_cache(cache));
  REFUSE(!attn_supported(cache->head, group), LLM_ERR_CONFIG, "group must be 1..16 with group x head size at most 1024");
  REFUSE(B < 1, LLM_ERR_BATCH, "batch must be at least 1");
  REFUSE(S < 1 || (int64_t)B * S >= (int64_t)1 << 31, LLM_ERR_ARG, "tokens per row out of range");
  REFUSE(groups < 1 || groups > B, LLM_ERR_ARG, "groups must be 1..B");
  int sms = 0;
  TRY(device_sms(&sms));
  const QCacheView c = {nullptr, nullptr, nullptr, nullptr, cache->rows, cache->kv_heads, cache->max_seq, cache->head};
  *bytes = qattn_shared_workspace(c, group, B, S, groups, sms);
  return LLM_OK;
}

llm_status llm_qcache_attend_shared(const llm_qcache* cache, const void* q_dev, int32_t dtype, int64_t q_stride, int32_t group,
                                    int32_t B, int32_t S, const int32_t* length_dev, const int32_t* count_dev,
                                    const int32_t* table_dev, int32_t pages_per_row, const int32_t* groups_dev,
                                    const int32_t* shared_dev, int32_t groups, float scale, void* out_dev, int64_t out_stride,
                                    void* workspace_dev, uint64_t workspace_bytes, int32_t* status_dev, void* cuda_stream) {
  REFUSE(!cache, LLM_ERR_ARG, "NULL cache");
  QAttnArgs a = {};
  TRY(check_cache(cache));
  TRY(check_rows(cache, B, S, length_dev, count_dev, table_dev, pages_per_row, status_dev, &a.c, &a.r));
  REFUSE(!attn_supported(cache->head, group), LLM_ERR_CONFIG, "group must be 1..16 with group x head size at most 1024");
  const int64_t width = (int64_t)a.c.kv * group * a.c.hd;
  TRY(check_buffer(q_dev, dtype, q_stride, width));
  TRY(check_buffer(out_dev, dtype, out_stride, width));
  REFUSE(!isfinite(scale), LLM_ERR_ARG, "scale must be finite");
  REFUSE(groups < 1 || groups > B, LLM_ERR_ARG, "groups must be 1..B");
  REFUSE(!groups_dev || !shared_dev || !aligned4(groups_dev) || !aligned4(shared_dev), LLM_ERR_ARG,
         "the groups' bounds and shared positions must be given, as aligned int32 arrays");
  int sms = 0;
  TRY(device_sms(&sms));
  a.g = group; a.ngroups = groups;
  REFUSE(qattn_shared_way(a, dtype, sms) == kSharedTooLarge, LLM_ERR_ARG,
         "too large for one call: rows x tokens x kv heads x 128-position tiles must stay below 2^31");
  const uint64_t need = qattn_shared_workspace(a.c, group, B, S, groups, sms);
  if (need > 0) {
    REFUSE(!workspace_dev || workspace_bytes < need, LLM_ERR_ARG, "workspace smaller than llm_qcache_shared_workspace says");
    REFUSE(!aligned16(workspace_dev), LLM_ERR_ARG, "the workspace must be aligned to 16 bytes");
  }
  a.q = q_dev; a.out = out_dev; a.q_stride = q_stride; a.out_stride = out_stride; a.scale = scale;
  a.ws = (unsigned char*)workspace_dev;
  a.groups = groups_dev; a.shared = shared_dev;
  return launched(launch_qattn_shared(a, dtype, sms, (cudaStream_t)cuda_stream));
}

llm_status llm_qcache_copy_pages(const llm_qcache* caches, int32_t n, const int32_t* moves_dev, int32_t m,
                                 const int32_t* counts_dev, int32_t* status_dev, void* cuda_stream) {
  REFUSE(!caches || n < 1, LLM_ERR_ARG, "at least one cache is needed");
  REFUSE(!moves_dev || m < 1, LLM_ERR_ARG, "at least one move is needed");
  REFUSE(!aligned4(moves_dev) || !aligned4(counts_dev) || !aligned4(status_dev), LLM_ERR_ARG, "int32 arrays must be aligned");
  for (int32_t i = 0; i < n; ++i) {
    TRY(check_cache(caches + i));
    REFUSE(caches[i].rows != caches[0].rows || caches[i].kv_heads != caches[0].kv_heads ||
               caches[i].max_seq != caches[0].max_seq || caches[i].head != caches[0].head,
           LLM_ERR_CONFIG, "the caches of a call must have one shape");
  }
  REFUSE(caches->max_seq % kPage, LLM_ERR_CONFIG, "pages need max_seq to be a multiple of 64");
  REFUSE((int64_t)m * caches->kv_heads >= ((int64_t)1 << 32) / kCopyLayers, LLM_ERR_ARG,
         "too large for one call: moves x kv heads must stay below 2^32 / 96");
  CopyArgs a = {};
  a.rows = caches->rows; a.kv = caches->kv_heads; a.cap = caches->max_seq; a.bytes = caches->head;
  a.moves = moves_dev; a.m = m; a.counts = counts_dev; a.status = status_dev;
  for (int32_t i = 0; i < n; i += kCopyLayers) {
    a.layers = n - i < kCopyLayers ? n - i : kCopyLayers;
    for (int32_t l = 0; l < a.layers; ++l) {
      a.k[l] = (uint8_t*)caches[i + l].k;
      a.v[l] = (uint8_t*)caches[i + l].v;
      a.ks[l] = caches[i + l].k_scale;
      a.vs[l] = caches[i + l].v_scale;
    }
    TRY(launched(launch_copy_pages(a, (cudaStream_t)cuda_stream)));
  }
  return LLM_OK;
}

static llm_status check_pages(const llm_pages* p) {
  REFUSE(!p->table || !p->length || !aligned4(p->table) || !aligned4(p->length), LLM_ERR_ARG,
         "a page table and lengths are needed, aligned to 4 bytes");
  REFUSE(p->rows < 1 || p->pages_per_row < 1 || p->pages < 1, LLM_ERR_CONFIG, "rows, pages per row and pages must be at least 1");
  REFUSE(p->pages > 1 << 28 || p->pages_per_row > 1 << 24 || (int64_t)p->rows * (p->pages_per_row + 1) > 0x7fffffff, LLM_ERR_CONFIG,
         "too large: pages at most 2^28, pages per row 2^24, rows x (pages per row + 1) below 2^31");
  return LLM_OK;
}

static bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)m * 4 && y < x + (uintptr_t)n * 4;
}

// the two books of an update or a compaction, and where its copies and counts go
static llm_status check_books(const llm_pages* from, const llm_pages* to, const int32_t* moves, const int32_t* counts,
                              const void* ws, uint64_t ws_bytes, const int32_t* status, PageBook* x, PageBook* y) {
  REFUSE(!from || !to, LLM_ERR_ARG, "NULL pages");
  TRY(check_pages(from));
  TRY(check_pages(to));
  REFUSE(from->rows != to->rows || from->pages_per_row != to->pages_per_row || from->pages != to->pages, LLM_ERR_CONFIG,
         "both tables must have one shape, over one pool");
  const int64_t R = from->rows, n = R * from->pages_per_row;
  REFUSE(overlap(from->table, n, to->table, n) || overlap(from->length, R, to->length, R) ||
             overlap(from->table, n, to->length, R) || overlap(from->length, R, to->table, n),
         LLM_ERR_ARG, "the new table and lengths must not overlap the old ones");
  REFUSE(!moves || !counts || !aligned4(moves) || !aligned4(counts) || !aligned4(status), LLM_ERR_ARG,
         "moves and counts are needed, as aligned int32 arrays");
  REFUSE(!ws || !aligned4(ws) || ws_bytes < pages_workspace(from->rows, from->pages) * 4, LLM_ERR_ARG,
         "workspace smaller than llm_pages_workspace says");
  *x = PageBook{from->table, from->length, from->rows, from->pages_per_row, from->pages};
  *y = PageBook{to->table, to->length, to->rows, to->pages_per_row, to->pages};
  return LLM_OK;
}

llm_status llm_pages_workspace(const llm_pages* pages, uint64_t* bytes) {
  REFUSE(!pages || !bytes, LLM_ERR_ARG, "NULL argument");
  TRY(check_pages(pages));
  *bytes = pages_workspace(pages->rows, pages->pages) * 4;
  return LLM_OK;
}

llm_status llm_pages_update(const llm_pages* from, const llm_pages* to, const int32_t* parent_dev, const int32_t* length_dev,
                            int32_t* moves_dev, int32_t* counts_dev, void* workspace_dev, uint64_t workspace_bytes,
                            int32_t* status_dev, void* cuda_stream) {
  PageBook x, y;
  TRY(check_books(from, to, moves_dev, counts_dev, workspace_dev, workspace_bytes, status_dev, &x, &y));
  REFUSE(!aligned4(parent_dev) || !aligned4(length_dev), LLM_ERR_ARG, "int32 arrays must be aligned");
  return launched(launch_pages_update(x, y, parent_dev, length_dev, moves_dev, counts_dev, (int32_t*)workspace_dev, status_dev,
                                      (cudaStream_t)cuda_stream));
}

llm_status llm_pages_compact(const llm_pages* from, const llm_pages* to, int32_t* moves_dev, int32_t* counts_dev,
                             void* workspace_dev, uint64_t workspace_bytes, int32_t* status_dev, void* cuda_stream) {
  PageBook x, y;
  TRY(check_books(from, to, moves_dev, counts_dev, workspace_dev, workspace_bytes, status_dev, &x, &y));
  return launched(launch_pages_compact(x, y, moves_dev, counts_dev, (int32_t*)workspace_dev, status_dev, (cudaStream_t)cuda_stream));
}

llm_status llm_sample_rows(const float* logits_dev, int64_t stride, int32_t B, int32_t V, const float* temp_dev,
                           const int32_t* k_dev, const float* p_dev, const float* min_p_dev, const float* u_dev,
                           int32_t* ids_dev, int32_t* status_dev, void* cuda_stream) {
  REFUSE(!logits_dev || !u_dev || !ids_dev, LLM_ERR_ARG, "NULL argument");
  REFUSE(B < 1 || B > 1 << 24, LLM_ERR_BATCH, "batch out of range");
  REFUSE(V < 1 || V > kSampleRowsMost, LLM_ERR_ARG, "the vocabulary must be in 1..524280");
  REFUSE(stride < V, LLM_ERR_ARG, "rows overlap: the stride is below the vocabulary");
  REFUSE(!aligned4(logits_dev) || !aligned4(temp_dev) || !aligned4(k_dev) || !aligned4(p_dev) || !aligned4(min_p_dev) ||
             !aligned4(u_dev) || !aligned4(ids_dev) || !aligned4(status_dev),
         LLM_ERR_ARG, "arrays must be aligned to 4 bytes");
  const SampleRowsArgs a = {logits_dev, stride, B, V, temp_dev, k_dev, p_dev, min_p_dev, u_dev, ids_dev, status_dev};
  return launched(launch_sample_rows(a, (cudaStream_t)cuda_stream));
}

llm_status llm_verify(const float* p_dev, const float* q_dev, const int32_t* drafts_dev, const int32_t* count_dev,
                      int32_t B, int32_t S, int32_t V, const float* u_dev, int32_t* ids_dev, int32_t* accepted_dev,
                      void* cuda_stream) {
  REFUSE(!p_dev || !drafts_dev || !u_dev || !ids_dev || !accepted_dev, LLM_ERR_ARG, "NULL argument");
  REFUSE(B < 1 || B > 1 << 24, LLM_ERR_BATCH, "batch out of range");
  REFUSE(S < 1 || S > 65535 || V < 1 || V > 1 << 30, LLM_ERR_ARG,
         "drafts per row must be in 1..65535 and the vocabulary in 1..2^30");
  REFUSE(!aligned4(p_dev) || !aligned4(q_dev) || !aligned4(drafts_dev) || !aligned4(count_dev) || !aligned4(u_dev) ||
             !aligned4(ids_dev) || !aligned4(accepted_dev),
         LLM_ERR_ARG, "arrays must be aligned to 4 bytes");
  const VerifyArgs a = {p_dev, q_dev, drafts_dev, count_dev, u_dev, B, S, V, ids_dev, accepted_dev};
  return launched(launch_verify(a, (cudaStream_t)cuda_stream));
}

}  // extern "C"
