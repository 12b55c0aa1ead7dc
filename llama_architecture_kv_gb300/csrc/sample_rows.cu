// One token per row from its logits, with temperature, top-k, top-p and min-p of its own.
//
// With top the row's largest logit, a candidate's distance from it is
//   d = floor(2^27 min((top - v) (1 / temp), 30))       (the products f32, rounded one by one)
// and its weight w = round(2^31 exp(-d / 2^27)), the exp of sampler.cuh.  Candidates are ordered by d, ties
// by id.  Top-k keeps the first k; top-p, of those, the ones whose weights before them sum to less than
// p times the sum of all k (always the first); min-p the ones with w >= 2^31 min_p.  Each keeps a head of
// the order.  The draw u picks the first whose running sum is above u times the sum of what is kept.
//
// Weights are whole numbers and their sums exact in 64 bits, in any order.  So nothing is sorted: a
// place in the order (the k-th candidate, or the one where the weights reach a sum) is found by a
// histogram of d, and only the candidates of the bin that holds it are put in order.
//
// One row, a cluster of 8 CTAs, each a contiguous stretch of ids: the largest logit; a histogram of d in
// 2048 bins over the range that it has (counts and weights, in shared memory, joined bin by bin through
// distributed shared memory so that every CTA has the whole row's); then for each place the bin's
// candidates, which every CTA gets and orders for itself.  A bin of more candidates than fit (equal logits,
// or logits far narrower than the range) is split by the next 11 bits of d until they do or d is the
// same for all, where the order is that of the ids.  Candidates that weigh nothing are in no bin.
#include <math.h>

#include "sampler.cuh"

namespace llm {

namespace {

constexpr int32_t kErrArg = 7;
constexpr int kSrThreads = 512;
constexpr int kSrWarps = kSrThreads / 32;
constexpr int kSrCluster = 8;
constexpr int kSrBins = 2048;
constexpr int kSrBits = 11;
constexpr int kSrMost = 1024;                 // candidates of a bin that are put in order
constexpr uint32_t kSrFar = 30u << 27;        // the largest distance
constexpr uint32_t kSrNothing = 2977044472u;  // exp(-d / 2^27) < 2^-32 from here on: the weight is 0
constexpr uint32_t kSrNone = 0xffffffffu;     // no candidate: it weighs nothing

LLM_D uint32_t sr_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
LLM_D void sr_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
LLM_D uint32_t sr_map(const void* p, uint32_t rank) {
  uint32_t local = (uint32_t)__cvta_generic_to_shared(p), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  return remote;
}
LLM_D void sr_put(uint64_t* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(sr_map(p, rank)), "l"(v) : "memory");
}
LLM_D void sr_put32(uint32_t* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sr_map(p, rank)), "r"(v) : "memory");
}
LLM_D uint32_t sr_get32(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(sr_map(p, rank)) : "memory");
  return v;
}
LLM_D uint32_t sr_add(uint32_t* p, uint32_t rank, uint32_t n) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(sr_map(p, rank)), "r"(n) : "memory");
  return old;
}

// floor(part * total / 2^24), part at most 2^24
LLM_D uint64_t sr_share(uint64_t total, uint32_t part) { return part * (total >> 24) + (part * (total & 0xffffffu) >> 24); }
// floor(2^24 x) for x in 0 .. 1
LLM_D uint32_t sr_part(float x) { return (uint32_t)(x * 16777216.0f); }

LLM_D uint32_t sr_weight(uint32_t d) { return __float2uint_rn(exp_s(-(float)d * 0x1p-27f) * 2147483648.0f); }

struct SrShared {
  uint32_t hist[3][kSrBins];        // this CTA's counts, and sums of the low and high 16 bits of the weights
  uint64_t weight[2][kSrBins];      // the row's: sums of weights of the bins before; of a bin's split
  uint32_t count[2][kSrBins];       // counts of the bins before
  uint64_t list[3][kSrMost];        // candidates of the bins of the three places: d, id
  uint32_t listed[3];
  uint64_t top[kSrCluster];         // the CTAs' largest logits, as key and -id
  uint32_t low[kSrCluster];         // and the keys of their smallest
  uint64_t above[kSrCluster];       // sums of weights that min-p keeps
  uint32_t same[kSrCluster];        // candidates at one distance
  uint64_t sum[kSrWarps];
  uint32_t num[kSrWarps];
  uint64_t all_weight[2];
  uint32_t all_count[2];
  uint32_t pick;
};

// an order-preserving key; 0 for NaN
LLM_D uint32_t sr_key(float v) {
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return v != v ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
LLM_D float sr_unkey(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// exclusive sums over the CTA's threads in their order
LLM_D void sr_scan(SrShared& s, uint32_t n, uint64_t w, uint32_t& n0, uint64_t& w0, uint32_t& nall, uint64_t& wall) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = n;
  uint64_t y = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x, o);
    const uint64_t b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.num[warp] = x;
    s.sum[warp] = y;
  }
  __syncthreads();
  n0 = x - n;
  w0 = y - w;
  nall = 0u;
  wall = 0ull;
  for (int i = 0; i < kSrWarps; ++i) {
    if (i < warp) {
      n0 += s.num[i];
      w0 += s.sum[i];
    }
    nall += s.num[i];
    wall += s.sum[i];
  }
}

struct SrRow {
  const float* v;     // this CTA's stretch
  int n, id0;         // its length and first id
  float top, scale;   // the largest logit; 1 / temp
  uint32_t rank;
  LLM_D uint32_t dist(float x) const {
    // (NaN, and what is infinitely far: nothing; all of +inf at the top are at it)
    if (!(x > -INFINITY)) return kSrNone;
    const float a = x == top ? 0.0f : __fmul_rn(__fsub_rn(top, x), scale);
    const uint32_t d = a < 30.0f ? (uint32_t)(a * 134217728.0f) : kSrFar;
    return d >= kSrNothing ? kSrNone : d;
  }
};

// counts and weights of the candidates with d >> (shift + bits) == bin, by the `bits` bits below; the sums of the
// bins before each, for the whole row, in every CTA, in s.weight[to] and s.count[to]
LLM_D void sr_histogram(SrShared& s, const SrRow& r, int shift, int bits, uint32_t bin, int to) {
  for (int i = threadIdx.x; i < 3 * kSrBins; i += kSrThreads) s.hist[0][i] = 0u;
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < r.n; i += kSrThreads) {
    const uint32_t d = r.dist(r.v[i]);
    if (d == kSrNone || (uint32_t)((uint64_t)d >> (shift + bits)) != bin) continue;
    const uint32_t w = sr_weight(d), b = d >> shift & ((1u << bits) - 1u);
    atomicAdd(&s.hist[0][b], 1u);
    atomicAdd(&s.hist[1][b], w & 0xffffu);
    atomicAdd(&s.hist[2][b], w >> 16);
  }
  sr_sync();
  constexpr int per = kSrBins / kSrCluster;
  if (threadIdx.x < per) {
    const int b = r.rank * per + threadIdx.x;
    uint32_t n = 0u;
    uint64_t w = 0ull;
    for (uint32_t c = 0; c < kSrCluster; ++c) {
      n += sr_get32(&s.hist[0][b], c);
      w += sr_get32(&s.hist[1][b], c) + ((uint64_t)sr_get32(&s.hist[2][b], c) << 16);
    }
    for (uint32_t c = 0; c < kSrCluster; ++c) {
      sr_put32(&s.count[to][b], c, n);
      sr_put(&s.weight[to][b], c, w);
    }
  }
  sr_sync();
  // bins before: thread = 4 bins
  constexpr int T = kSrBins / kSrThreads;
  uint32_t n[T], sn = 0u, n0, nall;
  uint64_t w[T], sw = 0ull, w0, wall;
#pragma unroll
  for (int y = 0; y < T; ++y) {
    n[y] = s.count[to][threadIdx.x * T + y];
    w[y] = s.weight[to][threadIdx.x * T + y];
    sn += n[y];
    sw += w[y];
  }
  sr_scan(s, sn, sw, n0, w0, nall, wall);
#pragma unroll
  for (int y = 0; y < T; ++y) {
    s.count[to][threadIdx.x * T + y] = n0;
    s.weight[to][threadIdx.x * T + y] = w0;
    n0 += n[y];
    w0 += w[y];
  }
  if (threadIdx.x == 0) {
    s.all_count[to] = nall;
    s.all_weight[to] = wall;
  }
  __syncthreads();
}

struct SrPlace {
  uint64_t upto;  // weights up to the candidate, its own among them
  int32_t id;
};

// The candidate at place t of the order: by count (weights false), or the one whose weight holds the t-th unit of
// the sum; t is below the whole row's.  Every CTA gets it; all walk through the same calls.
LLM_D SrPlace sr_find(SrShared& s, const SrRow& r, int shift, uint64_t t, bool weights, int place) {
  uint64_t n0 = 0ull, w0 = 0ull;  // candidates and weights before the bin in hand
  uint32_t bin = 0u;              // its bits of d
  int of = 0, bits = kSrBits;     // bits of the histogram in hand
  uint32_t in_bin;
  while (true) {
    // the last bin whose sum before is at most t
    int lo = 0, hi = kSrBins - 1;
    const uint64_t goal = t - (weights ? w0 : n0);
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((weights ? s.weight[of][mid] : (uint64_t)s.count[of][mid]) <= goal) lo = mid;
      else hi = mid - 1;
    }
    in_bin = (lo + 1 < kSrBins ? s.count[of][lo + 1] : s.all_count[of]) - s.count[of][lo];
    n0 += s.count[of][lo];
    w0 += s.weight[of][lo];
    bin = bin << bits | (uint32_t)lo;
    if (in_bin <= kSrMost || shift == 0) break;
    __syncthreads();  // (read by all before it is overwritten)
    bits = min(shift, kSrBits);
    shift -= bits;
    of = 1;
    sr_histogram(s, r, shift, bits, bin, 1);
  }
  if (in_bin > kSrMost) {
    // all at one distance: by id, stretch by stretch
    uint32_t mine = 0u;
    for (int i = threadIdx.x; i < r.n; i += kSrThreads) mine += r.dist(r.v[i]) == bin;
    uint32_t x, n;
    uint64_t y, z;
    sr_scan(s, mine, 0ull, x, y, n, z);
    if (threadIdx.x < kSrCluster) sr_put32(&s.same[r.rank], threadIdx.x, n);
    if (threadIdx.x == 0) s.pick = kSrNone;
    sr_sync();
    const uint64_t w = sr_weight(bin);
    uint64_t at = weights ? (t - w0) / w : t - n0;
    const uint64_t upto = w0 + (at + 1) * w;
    uint32_t before = 0u;
    for (uint32_t c = 0; c < r.rank; ++c) before += s.same[c];
    if (at >= before && at < before + n) {
      // the (at - before)-th of this stretch: threads take neighbouring ids
      const int per = (r.n + kSrThreads - 1) / kSrThreads, i0 = min(r.n, (int)threadIdx.x * per), i1 = min(r.n, i0 + per);
      mine = 0u;
      for (int i = i0; i < i1; ++i) mine += r.dist(r.v[i]) == bin;
      sr_scan(s, mine, 0ull, x, y, n, z);
      uint32_t left = (uint32_t)(at - before);
      if (left >= x && left < x + mine)
        for (int i = i0; i < i1; ++i)
          if (r.dist(r.v[i]) == bin && left-- == x)
            for (uint32_t c = 0; c < kSrCluster; ++c) sr_put32(&s.pick, c, (uint32_t)(r.id0 + i));
    }
    sr_sync();
    return SrPlace{upto, (int32_t)s.pick};
  }
  // the bin's candidates to every CTA
  uint64_t* list = s.list[place];
  const uint32_t lo = bin << shift, width = 1u << shift;
  for (int i = threadIdx.x; i < r.n; i += kSrThreads) {
    const uint32_t d = r.dist(r.v[i]);
    if (d == kSrNone || d - lo >= width) continue;
    const uint64_t e = (uint64_t)d << 32 | (uint32_t)(r.id0 + i);
    for (uint32_t c = 0; c < kSrCluster; ++c) {
      const uint32_t at = sr_add(&s.listed[place], c, 1u);
      if (at < kSrMost) sr_put(&list[at], c, e);
    }
  }
  sr_sync();
  const int n = (int)min(s.listed[place], (uint32_t)kSrMost);
  int n2 = 1;
  while (n2 < n) n2 <<= 1;
  for (int i = n + threadIdx.x; i < n2; i += kSrThreads) list[i] = ~0ull;
  __syncthreads();
  for (int size = 2; size <= n2; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      for (int i = threadIdx.x; i < n2; i += kSrThreads) {
        const int j = i ^ step;
        if (j > i) {
          const uint64_t a = list[i], b = list[j];
          if ((a > b) == ((i & size) == 0)) {
            list[i] = b;
            list[j] = a;
          }
        }
      }
      __syncthreads();
    }
  // running sums: thread = neighbours
  constexpr int T = kSrMost / kSrThreads;
  uint64_t w[T], sw = 0ull, at, wall;
  uint32_t nat, nall;
#pragma unroll
  for (int y = 0; y < T; ++y) {
    const int i = threadIdx.x * T + y;
    w[y] = i < n ? sr_weight((uint32_t)(list[i] >> 32)) : 0ull;
    sw += w[y];
  }
  sr_scan(s, 0u, sw, nat, at, nall, wall);
#pragma unroll
  for (int y = 0; y < T; ++y) {
    const int i = threadIdx.x * T + y;
    const uint64_t goal = t - (weights ? w0 : n0);
    if (i < n && (weights ? at <= goal && goal < at + w[y] : (uint64_t)i == goal)) {
      s.pick = (uint32_t)list[i];
      s.all_weight[1] = at + w[y];
    }
    at += w[y];
  }
  __syncthreads();
  const SrPlace got = {w0 + s.all_weight[1], (int32_t)s.pick};
  __syncthreads();
  return got;
}

// cluster = row
__global__ void __launch_bounds__(kSrThreads) sample_rows_kernel(const SampleRowsArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  SrShared& s = *reinterpret_cast<SrShared*>(raw);
  const int b = blockIdx.x / kSrCluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  SrRow r;
  r.rank = sr_rank();
  const int per = (a.V + kSrCluster - 1) / kSrCluster;
  r.id0 = min(a.V, (int)r.rank * per);
  r.n = min(a.V, r.id0 + per) - r.id0;
  r.v = a.logits + (int64_t)b * a.stride + r.id0;
  const float temp = a.temp ? a.temp[b] : 1.0f, p = a.p ? a.p[b] : 1.0f, min_p = a.min_p ? a.min_p[b] : 0.0f;
  const int k = a.k ? a.k[b] : a.V;
  const float u = a.u ? a.u[b] : 0.0f;
  const bool greedy = temp == 0.0f;
  const bool fine = temp >= 0.0f && temp < INFINITY && (greedy || (k >= 1 && p > 0.0f && p <= 1.0f && min_p >= 0.0f && min_p <= 1.0f &&
                                                                    u >= 0.0f && u < 1.0f));
  if (!fine) {  // (alike in the whole cluster)
    if (r.rank == 0 && tid == 0) {
      if (a.status) atomicCAS(a.status, 0, kErrArg);
      a.ids[b] = -1;
    }
    return;
  }
  if (tid < 3) s.listed[tid] = 0u;
  // ---- the largest logit and its first id; the smallest that is not -inf ----
  uint64_t top = 0ull;
  uint32_t low = 0xffffffffu;
#pragma unroll 8
  for (int i = tid; i < r.n; i += kSrThreads) {
    const uint32_t key = sr_key(r.v[i]);
    const uint64_t e = (uint64_t)key << 32 | (uint32_t)~(r.id0 + i);
    top = e > top ? e : top;
    if (key > 0x007fffffu) low = min(low, key);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t x = __shfl_xor_sync(0xffffffffu, top, o);
    top = x > top ? x : top;
  }
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) {
    s.sum[warp] = top;
    s.num[warp] = low;
  }
  // (the first barrier of the cluster: every CTA has started and set its list's length before another writes to it)
  sr_sync();
  if (tid < kSrCluster) {
    uint64_t x = 0ull;
    uint32_t y = 0xffffffffu;
    for (int i = 0; i < kSrWarps; ++i) {
      x = s.sum[i] > x ? s.sum[i] : x;
      y = min(y, s.num[i]);
    }
    sr_put(&s.top[r.rank], tid, x);
    sr_put32(&s.low[r.rank], tid, y);
  }
  sr_sync();
  for (int i = 0; i < kSrCluster; ++i) {
    top = s.top[i] > top ? s.top[i] : top;
    low = min(low, s.low[i]);
  }
  const uint32_t key = (uint32_t)(top >> 32);
  const bool none = key <= 0x007fffffu;  // every logit is -inf or NaN
  if (none || greedy) {
    if (r.rank == 0 && tid == 0) a.ids[b] = none ? 0 : (int32_t)~(uint32_t)top;
    return;
  }
  r.top = sr_unkey(key);
  r.scale = fminf(__fdiv_rn(1.0f, temp), 3.402823466e38f);
  // ---- the histogram over the range that the distances have ----
  const float span = __fmul_rn(__fsub_rn(r.top, sr_unkey(low)), r.scale);
  const uint32_t most = span < 22.2f ? (uint32_t)(span * 134217728.0f) : 0xb1a00000u;
  const int shift = max(0, 32 - __clz((int)most) - kSrBits);
  sr_histogram(s, r, shift, kSrBits, 0u, 0);
  const uint64_t all = s.all_weight[0];
  const uint32_t count = s.all_count[0];
  // ---- what is kept ----
  uint64_t kept = all;
  if ((uint32_t)k < count) kept = sr_find(s, r, shift, (uint64_t)(k - 1), false, 0).upto;
  const uint32_t part = sr_part(p);
  if (part < 1u << 24) {
    const uint64_t limit = sr_share(kept, part);
    kept = sr_find(s, r, shift, limit ? limit - 1 : 0ull, true, 1).upto;
  }
  const uint32_t least = (uint32_t)(min_p * 2147483648.0f);
  if (least > 0u) {
    uint64_t x = 0ull, y, z;
    uint32_t n, m;
    for (int i = tid; i < r.n; i += kSrThreads) {
      const uint32_t d = r.dist(r.v[i]);
      if (d == kSrNone) continue;
      const uint32_t w = sr_weight(d);
      if (w >= least) x += w;
    }
    sr_scan(s, 0u, x, n, y, m, z);
    if (tid < kSrCluster) sr_put(&s.above[r.rank], tid, z);
    sr_sync();
    x = 0ull;
    for (int i = 0; i < kSrCluster; ++i) x += s.above[i];
    kept = min(kept, x);
  }
  const int32_t id = sr_find(s, r, shift, sr_share(kept, sr_part(u)), true, 2).id;
  if (r.rank == 0 && tid == 0) a.ids[b] = id;
}

}  // namespace

cudaError_t launch_sample_rows(const SampleRowsArgs& a, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(sample_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SrShared));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * kSrCluster);
  cfg.blockDim = dim3(kSrThreads);
  cfg.dynamicSmemBytes = sizeof(SrShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSrCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_rows_kernel, a);
}

}  // namespace llm
