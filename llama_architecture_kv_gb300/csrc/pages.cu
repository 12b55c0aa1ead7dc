// Page tables: rows that fork, shrink, grow and are freed; pages in use moved to the front of the pool;
// and the copies of pages that both ask for.
//
// Update.  New row r takes keep = min(length[parent], new length) positions of its parent (none without
// one) and so its first ceil(keep / 64) pages; the rest of its ceil(new / 64) pages are new.  All rows
// change at once, so a row can be dropped and be a parent in one call.  A page that a row holds whole
// can be shared by any number of rows: none writes it again.  The last page of a row whose keep ends
// inside it is open: the row writes there next.  An open page stays with one row -- the lowest that has
// it open, if no row holds it whole -- and every other row that has it open gets a copy.  Pages are
// taken from those that no new row claims, lowest first, in the order of the rows, and a row's copy
// before its new pages.  Sources of copies are claimed and destinations are not, so copies can run in
// any order.
//
// Compaction.  With U pages in use, the n of them with numbers of U and above move to the n unused
// ones below U, both in ascending order: the fewest copies that leave pages 0 .. U - 1 in use.
//
// Both are integer bookkeeping over rows x pages and the pool, a few kilobytes: bound by latency, that
// is by how many times all threads have to meet.  One cluster does it (one CTA where the tables are
// small), whose CTAs meet in its barrier: claims are marked with stores and minima, whose order does not
// matter, then counted page by page (each CTA a contiguous stretch of the pool), and the tables
// written.  Everything is checked before anything is written; a call that cannot be done hands the
// rows on unchanged.
#include <algorithm>

#include "pages.cuh"

namespace llm {

namespace {

constexpr int32_t kErrOom = 3;
constexpr int kPgThreads = 1024;
constexpr int kPgCluster = 8;
constexpr int kPgSmall = 16384;  // table entries and pages up to which one CTA does it
constexpr int kPgChunk = 128;    // entries of a row that a warp takes at a time

// words of the workspace before its arrays: the first error, and counts of the CTAs' stretches
constexpr int kPgErr = 0, kPgCount = 16, kPgCount2 = kPgCount + kPgCluster, kPgHead = 64;

struct PgCluster {
  int rank, size;
};
LLM_D PgCluster pg_cluster() {
  PgCluster c;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(c.rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(c.size));
  return c;
}
// all threads meet; what they wrote to global memory is there for the others
LLM_D void pg_sync(const PgCluster& c) {
  if (c.size == 1) {
    __syncthreads();
    return;
  }
  __threadfence();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// exclusive sum over the CTA's threads in their order, and the total
LLM_D int pg_scan(int v, int& total) {
  __shared__ int s_warp[kPgThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  const int w = s_warp[lane];
  int y = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  total = __shfl_sync(0xffffffffu, y, 31);
  const int before = __shfl_sync(0xffffffffu, y - w, warp);
  __syncthreads();
  return before + x - v;
}

// sum of a cluster's counts, and of those before this CTA
LLM_D int pg_sum(const int32_t* counts, const PgCluster& c, int& before) {
  int all = 0;
  before = 0;
  for (int i = 0; i < c.size; ++i) {
    const int n = __ldcg(counts + i);
    if (i < c.rank) before += n;
    all += n;
  }
  return all;
}

LLM_HD int pg_pages(int positions) { return (positions + kPage - 1) / kPage; }

struct PgRow {
  int parent, keep, kept, total;  // positions and pages of the parent that stay, and pages in all
  bool open;                      // the last page that stays is written next
};
// row r of an update; err: what is wrong with it (then the row is empty)
LLM_D PgRow pg_row(const PageBook& from, const int32_t* parent, const int32_t* length, int r, int32_t& err) {
  PgRow x = {parent ? parent[r] : r, 0, 0, 0, false};
  if (x.parent < -1 || x.parent >= from.rows) {
    err = kErrArg;
    x.parent = -1;
  }
  if (x.parent < 0) return x;
  const int most = from.per_row * kPage, old = from.length[x.parent], now = length ? length[r] : old;
  if (old < 0 || old > most || now < 0 || now > most) {
    err = kErrPosRange;
    x.parent = -1;
    return x;
  }
  x.keep = min(old, now);
  x.kept = pg_pages(x.keep);
  x.total = pg_pages(now);
  x.open = x.keep % kPage != 0;
  return x;
}

// the tables as they were, and nothing to copy
LLM_D void pg_hand_on(const PageBook& from, const PageBook& to, int32_t* moves, int m, int32_t* counts, int t, int nt) {
  const int64_t n = (int64_t)from.rows * from.per_row;
  for (int64_t i = t; i < n; i += nt) to.table[i] = from.table[i];
  for (int i = t; i < from.rows; i += nt) to.length[i] = from.length[i];
  for (int i = t; i < 2 * m; i += nt) moves[i] = -1;
  if (t == 0) {
    counts[0] = 0;
    counts[1] = -1;
  }
}

// workspace: head, [pages] held whole by a row, [pages] lowest row that has it open, [pages] the free
// pages in order, [rows] first free page of a row, [rows] copies of the rows before
__global__ void __launch_bounds__(kPgThreads)
    pages_update_kernel(const PageBook from, const PageBook to, const int32_t* parent, const int32_t* length, int32_t* moves,
                        int32_t* counts, int32_t* ws, int32_t* status) {
  grid_dep_launch();
  const PgCluster c = pg_cluster();
  const int t = c.rank * kPgThreads + threadIdx.x, nt = c.size * kPgThreads;
  const int lane = threadIdx.x & 31, warp = t >> 5, nw = nt >> 5;
  const int R = from.rows, P = from.pages;
  int32_t* err = ws + kPgErr;
  int32_t* whole = ws + kPgHead;
  int32_t* lowest = whole + P;
  int32_t* free_ = lowest + P;
  int32_t* first = free_ + P;
  int32_t* copies = first + R;
  for (int i = t; i < P; i += nt) {
    __stcg(whole + i, 0);
    __stcg(lowest + i, R);
  }
  if (t == 0) __stcg(err, 0);
  pg_sync(c);
  // claims
  const int chunks = (from.per_row + kPgChunk - 1) / kPgChunk;
  const int64_t units = (int64_t)R * chunks;
  for (int64_t u = warp; u < units; u += nw) {
    const int r = (int)(u / chunks), j0 = (int)(u - (int64_t)r * chunks) * kPgChunk;
    int32_t bad = 0;
    const PgRow x = pg_row(from, parent, length, r, bad);
#pragma unroll
    for (int y = 0; y < kPgChunk; y += 32) {
      const int j = j0 + y + lane;
      if (j >= x.kept) continue;
      const int page = from.table[(int64_t)x.parent * from.per_row + j];
      if (page < 0 || page >= P) bad = kErrArg;
      else if (x.open && j == x.kept - 1) atomicMin(lowest + page, r);
      else __stcg(whole + page, 1);
    }
    if (bad) atomicCAS(err, 0, bad);
  }
  pg_sync(c);
  const int32_t bad = __ldcg(err);
  if (bad) {
    if (t == 0) q_report(status, bad);
    pg_hand_on(from, to, moves, R, counts, t, nt);
    return;  // (alike in every thread of the cluster)
  }
  // this CTA's stretch of the pool: its free pages, counted
  const int per = (P + nt - 1) / nt;   // pages of a thread, neighbours
  const int p0 = min(P, t * per), p1 = min(P, p0 + per);
  auto is_free = [&](int p) { return __ldcg(whole + p) == 0 && __ldcg(lowest + p) == R; };
  auto copied = [&](int r, const PgRow& x) {
    if (!x.open) return false;
    const int page = from.table[(int64_t)x.parent * from.per_row + x.kept - 1];
    return __ldcg(whole + page) != 0 || __ldcg(lowest + page) != r;
  };
  int mine = 0, total;
  for (int p = p0; p < p1; ++p) mine += is_free(p);
  const int before = pg_scan(mine, total);
  if (threadIdx.x == 0) __stcg(ws + kPgCount + c.rank, total);
  // the last CTA: what every row needs, summed over the rows
  if (c.rank == c.size - 1) {
    int need_sum = 0, copy_sum = 0;
    for (int r0 = 0; r0 < R; r0 += kPgThreads) {
      const int r = r0 + threadIdx.x;
      int need = 0, copy = 0;
      if (r < R) {
        int32_t none = 0;
        const PgRow x = pg_row(from, parent, length, r, none);
        copy = copied(r, x);
        need = copy + x.total - x.kept;
      }
      int sum, n;
      const int at = pg_scan(need, sum), ct = pg_scan(copy, n);
      if (r < R) {
        // (sums stay below 2^31: rows x pages per row do)
        __stcg(first + r, need_sum + at);
        __stcg(copies + r, copy_sum + ct);
      }
      need_sum += sum;
      copy_sum += n;
    }
    if (threadIdx.x == 0) {
      __stcg(ws + kPgCount2, need_sum);
      __stcg(ws + kPgCount2 + 1, copy_sum);
    }
  }
  pg_sync(c);
  int lead;
  const int nfree = pg_sum(ws + kPgCount, c, lead);
  const int need = __ldcg(ws + kPgCount2), ncopy = __ldcg(ws + kPgCount2 + 1);
  if (need > nfree) {
    if (t == 0) q_report(status, kErrOom);
    pg_hand_on(from, to, moves, R, counts, t, nt);
    return;
  }
  int at = lead + before;
  for (int p = p0; p < p1 && at < need; ++p)
    if (is_free(p)) __stcg(free_ + at++, p);
  pg_sync(c);
  // the new rows
  for (int64_t u = warp; u < units; u += nw) {
    const int r = (int)(u / chunks), j0 = (int)(u - (int64_t)r * chunks) * kPgChunk;
    int32_t none = 0;
    const PgRow x = pg_row(from, parent, length, r, none);
    const bool copy = copied(r, x);
    const int f = __ldcg(first + r);
#pragma unroll
    for (int y = 0; y < kPgChunk; y += 32) {
      const int j = j0 + y + lane;
      if (j >= from.per_row) continue;
      int page = -1;
      if (copy && j == x.kept - 1) page = __ldcg(free_ + f);
      else if (j < x.kept) page = from.table[(int64_t)x.parent * from.per_row + j];
      else if (j < x.total) page = __ldcg(free_ + f + copy + j - x.kept);
      to.table[(int64_t)r * from.per_row + j] = page;
    }
    if (j0 == 0 && lane == 0) {
      to.length[r] = x.parent < 0 ? 0 : length ? length[r] : x.keep;
      if (copy) {
        const int n = __ldcg(copies + r);
        moves[2 * n] = from.table[(int64_t)x.parent * from.per_row + x.kept - 1];
        moves[2 * n + 1] = __ldcg(free_ + f);
      }
      if (r >= ncopy) moves[2 * r] = moves[2 * r + 1] = -1;
    }
  }
  if (t == 0) {
    counts[0] = ncopy;
    counts[1] = P - nfree + need;
  }
}

// workspace: head, [pages] a page's new number; the copy that moves it, as -2 - its number; or -1: not in use
__global__ void __launch_bounds__(kPgThreads)
    pages_compact_kernel(const PageBook from, const PageBook to, int32_t* moves, int m, int32_t* counts, int32_t* ws,
                         int32_t* status) {
  grid_dep_launch();
  const PgCluster c = pg_cluster();
  const int t = c.rank * kPgThreads + threadIdx.x, nt = c.size * kPgThreads;
  const int lane = threadIdx.x & 31, warp = t >> 5, nw = nt >> 5;
  const int R = from.rows, P = from.pages;
  int32_t* err = ws + kPgErr;
  int32_t* now = ws + kPgHead;
  for (int i = t; i < P; i += nt) __stcg(now + i, -1);
  if (t == 0) __stcg(err, 0);
  pg_sync(c);
  const int chunks = (from.per_row + kPgChunk - 1) / kPgChunk;
  const int64_t units = (int64_t)R * chunks;
  for (int64_t u = warp; u < units; u += nw) {
    const int r = (int)(u / chunks), j0 = (int)(u - (int64_t)r * chunks) * kPgChunk;
    const int len = from.length[r];
    int32_t bad = len < 0 || len > from.per_row * kPage ? kErrPosRange : 0;
    const int held = bad ? 0 : pg_pages(len);
#pragma unroll
    for (int y = 0; y < kPgChunk; y += 32) {
      const int j = j0 + y + lane;
      if (j >= held) continue;
      const int page = from.table[(int64_t)r * from.per_row + j];
      if (page < 0 || page >= P) bad = kErrArg;
      else __stcg(now + page, page);
    }
    if (bad) atomicCAS(err, 0, bad);
  }
  pg_sync(c);
  const int32_t bad = __ldcg(err);
  if (bad) {
    if (t == 0) q_report(status, bad);
    pg_hand_on(from, to, moves, m, counts, t, nt);
    return;
  }
  const int per = (P + nt - 1) / nt;
  const int p0 = min(P, t * per), p1 = min(P, p0 + per);
  int mine = 0, total, lead;
  for (int p = p0; p < p1; ++p) mine += __ldcg(now + p) >= 0;
  pg_scan(mine, total);
  if (threadIdx.x == 0) __stcg(ws + kPgCount + c.rank, total);
  pg_sync(c);
  const int used = pg_sum(ws + kPgCount, c, lead);
  // ranks of this thread's pages among those that leave, and among the places that they go to
  int out = 0, in = 0, nout, nin;
  for (int p = p0; p < p1; ++p) {
    const bool u = __ldcg(now + p) >= 0;
    out += u && p >= used;
    in += !u && p < used;
  }
  int out_at = pg_scan(out, nout), in_at = pg_scan(in, nin);
  if (threadIdx.x == 0) {
    __stcg(ws + kPgCount2 + c.rank, nout);
    __stcg(ws + kPgCount2 + kPgCluster + c.rank, nin);
  }
  pg_sync(c);
  const int n = pg_sum(ws + kPgCount2, c, lead);
  out_at += lead;
  pg_sum(ws + kPgCount2 + kPgCluster, c, lead);
  in_at += lead;
  for (int p = p0; p < p1; ++p) {
    const bool u = __ldcg(now + p) >= 0;
    if (u && p >= used) {
      __stcg(moves + 2 * out_at, p);
      __stcg(now + p, -2 - out_at++);
    } else if (!u && p < used) {
      __stcg(moves + 2 * in_at++ + 1, p);
    }
  }
  for (int i = 2 * n + t; i < 2 * m; i += nt) moves[i] = -1;
  pg_sync(c);
  for (int64_t u = warp; u < units; u += nw) {
    const int r = (int)(u / chunks), j0 = (int)(u - (int64_t)r * chunks) * kPgChunk;
    const int len = from.length[r], held = pg_pages(len);
#pragma unroll
    for (int y = 0; y < kPgChunk; y += 32) {
      const int j = j0 + y + lane;
      if (j >= from.per_row) continue;
      int page = -1;
      if (j < held) {
        page = __ldcg(now + from.table[(int64_t)r * from.per_row + j]);
        if (page < 0) page = __ldcg(moves + 2 * (-2 - page) + 1);
      }
      to.table[(int64_t)r * from.per_row + j] = page;
    }
    if (j0 == 0 && lane == 0) to.length[r] = len;
  }
  if (t == 0) {
    counts[0] = n;
    counts[1] = used;
  }
}

// A page's codes of one layer, head and side are one run of 64 positions; a warp copies it with as many
// 16-byte loads in flight as a lane has registers for, and its four scales.  Bound by HBM.
constexpr int kCopyThreads = 128;
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int per = a.layers * a.kv * 2;           // warps of a move
  const int64_t w = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  const int i = (int)(w / per);
  if (i >= a.m || (a.counts && i >= *a.counts)) return;
  const int x = (int)(w - (int64_t)i * per), side = x & 1, l = (x >> 1) / a.kv, h = (x >> 1) - l * a.kv;
  const int from = a.moves[2 * i], to = a.moves[2 * i + 1];
  if (from < 0 && to < 0) return;
  int row0, pos0, row1, pos1;
  if (!q_page_slot(a.rows, a.cap, from, 0, row0, pos0) || !q_page_slot(a.rows, a.cap, to, 0, row1, pos1)) {
    if (lane == 0) q_report(a.status, kErrArg);
    return;
  }
  const size_t at0 = ((size_t)row0 * a.kv + h) * a.cap + pos0, at1 = ((size_t)row1 * a.kv + h) * a.cap + pos1;
  uint8_t* base = side ? a.v[l] : a.k[l];
  float* scales = side ? a.vs[l] : a.ks[l];
  const uint4* src = reinterpret_cast<const uint4*>(base + at0 * a.bytes);
  uint4* dst = reinterpret_cast<uint4*>(base + at1 * a.bytes);
  constexpr int U = 8;
  const int n = kPage * a.bytes / 16;
  if (scales && lane < kPage / kQBlock) scales[at1 / kQBlock + lane] = scales[at0 / kQBlock + lane];
  for (int q = lane; q < n; q += 32 * U) {
    uint4 v[U];
#pragma unroll
    for (int y = 0; y < U; ++y)
      if (q + 32 * y < n) v[y] = __ldcs(src + q + 32 * y);
#pragma unroll
    for (int y = 0; y < U; ++y)
      if (q + 32 * y < n) __stcs(dst + q + 32 * y, v[y]);
  }
}

template <class... P, class... A>
cudaError_t launch_cluster(void (*fn)(P...), int64_t work, cudaStream_t s, A... args) {
  const unsigned size = work <= kPgSmall ? 1u : (unsigned)kPgCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kPgThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

uint64_t pages_workspace(int rows, int pages) { return kPgHead + 3 * (uint64_t)pages + 2 * (uint64_t)rows; }

cudaError_t launch_pages_update(const PageBook& from, const PageBook& to, const int32_t* parent, const int32_t* length,
                                int32_t* moves, int32_t* counts, int32_t* ws, int32_t* status, cudaStream_t s) {
  const int64_t work = std::max<int64_t>((int64_t)from.rows * from.per_row, from.pages);
  return launch_cluster(pages_update_kernel, work, s, from, to, parent, length, moves, counts, ws, status);
}

cudaError_t launch_pages_compact(const PageBook& from, const PageBook& to, int32_t* moves, int32_t* counts, int32_t* ws,
                                 int32_t* status, cudaStream_t s) {
  const int64_t work = std::max<int64_t>((int64_t)from.rows * from.per_row, from.pages);
  return launch_cluster(pages_compact_kernel, work, s, from, to, moves, std::max(1, from.pages / 2), counts, ws, status);
}

cudaError_t launch_copy_pages(const CopyArgs& a, cudaStream_t s) {
  const int64_t warps = (int64_t)a.m * a.layers * a.kv * 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32)));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  // (behind an update of the table it is on the SMs when that is done: one row forked into four 10.9 to 10.4 us)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel, a);
}

}  // namespace llm
