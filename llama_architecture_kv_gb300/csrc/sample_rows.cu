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
// One row, a cluster of up to 8 CTAs, each a contiguous stretch of ids that stays in shared memory, read once:
// the largest logit; a histogram of d in 2048 bins over the range that it has (counts and weights, joined bin by
// bin through distributed shared memory so that every CTA has the whole row's).  A place's bin bounds the sum
// that is kept, and so the bins that the next place can be in, seldom more than one or two: the candidates of all
// places' bins go to the first CTA in one pass, which orders them and finds the places.  Where they are
// too many (equal logits, or logits far narrower than the range), the places are found one after the other, a
// bin split by the next 11 bits of d until its candidates fit or d is the same for all, where the order is that
// of the ids.  Candidates that weigh nothing are in no bin.
//
// For k up to 1024 the histogram is of counts alone, one addition a candidate and no weight, and all candidates up to the
// k-th one's bin are gathered.
//
// What bounds it: for one row barriers of the cluster and the block, some thirty one after the other (15 us at 49152;
// 29 with the places one after the other and every pass from global memory); for many rows a candidate's weight (some
// 40 instructions; 48% of issue slots busy) and the histogram, whose three additions each serve the 32 banks' longest
// queue (32 rows of 128256: 32 us, 86 before; 256 of 50257: 75, 249 before).
#include <math.h>

#include "sampler.cuh"

namespace llm {

namespace {

constexpr int32_t kErrArg = 7;
constexpr int kSrCluster = 8;                 // CTAs of a row, at most
constexpr int kSrBins = 2048;
constexpr int kSrBits = 11;
constexpr int kSrMost = 1024;                 // candidates of a bin that are put in order
constexpr int kSrList = 2 * kSrMost;          // and of the bins of all places
constexpr uint32_t kSrNear = 1u << 12;        // what a distance found by logf may be off, and the weights' rounding
constexpr uint32_t kSrNothing = 2977044472u;  // exp(-d / 2^27) < 2^-32 from here on: the weight is 0
constexpr uint32_t kSrNone = 0xffffffffu;     // no candidate: it weighs nothing

LLM_D uint32_t sr_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
LLM_D uint32_t sr_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
LLM_D void sr_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
LLM_D void sr_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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
LLM_D uint2 sr_get64(const uint32_t* p, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(sr_map(p, rank)) : "memory");
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

// 2^31 exp(-d / 2^27), d below kSrNothing: the operations of exp_s for arguments of -23 to 0, its last factor and 2^31
// as one power of two (all three products exact but for the first, of p)
LLM_D uint32_t sr_weight(uint32_t d) {
  const float x = __fmul_rn((float)d, -0x1p-27f);
  const float t = __fadd_rn(__fmul_rn(x, 1.44269504088896340736f), 12582912.0f);  // rint + 1.5 2^23
  const float nf = __fsub_rn(t, 12582912.0f);
  float r = __fmaf_rn(-nf, 0.693145751953125f, x);
  r = __fmaf_rn(-nf, (float)(0.69314718055994530942 - 0.693145751953125), r);
  float p = (float)(1.0 / 40320.0);
  p = __fmaf_rn(p, r, (float)(1.0 / 5040.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 720.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 120.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 24.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 6.0));
  p = __fmaf_rn(p, r, 0.5f);
  p = __fmaf_rn(p, r, 1.0f);
  p = __fmaf_rn(p, r, 1.0f);
  return __float2uint_rn(__fmul_rn(p, __uint_as_float((__float_as_uint(t) - 0x4b400000u + 31u + 127u) << 23)));
}

struct alignas(16) SrShared {
  union {
    uint32_t hist[3][kSrBins];      // this CTA's counts, and sums of the low and high 16 bits of the weights
    uint64_t places[kSrList];       // candidates of the places' bins (the first CTA's: the row's): d, id
    uint64_t list[2][kSrMost];      // candidates of one place's bin
    struct {
      uint64_t weight[kSrBins];     // as below, of a bin's split
      uint32_t count[kSrBins];
    } split;
  };
  uint64_t weight[kSrBins];         // the row's: sums of weights of the bins before
  uint32_t count[kSrBins];          // counts of the bins before
  uint32_t listed[4];
  uint32_t top[kSrCluster];         // the keys of the CTAs' largest logits
  uint32_t low[kSrCluster];         // and of their smallest
  uint64_t above[kSrCluster];       // sums of weights that min-p keeps
  uint32_t same[kSrCluster];        // candidates at one distance
  uint64_t sum[32];                 // by warp
  uint32_t num[32];
  uint32_t low_of[32];
  uint64_t all_weight[2];
  uint32_t all_count[2];
  uint64_t upto[3];
  uint32_t bin[5];
  uint32_t pick;
};

// an order-preserving key; 0 for NaN
LLM_D uint32_t sr_key(float v) {
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return v != v ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
LLM_D float sr_unkey(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// exclusive sums over the CTA's threads in their order
template <int NT>
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
  // each warp for itself: the warps' sums
  uint32_t wn = lane < NT / 32 ? s.num[lane] : 0u;
  uint64_t ww = lane < NT / 32 ? s.sum[lane] : 0ull;
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, wn, o);
    const uint64_t b = __shfl_up_sync(0xffffffffu, ww, o);
    if (lane >= o) {
      wn += a;
      ww += b;
    }
  }
  nall = __shfl_sync(0xffffffffu, wn, NT / 32 - 1);
  wall = __shfl_sync(0xffffffffu, ww, NT / 32 - 1);
  const uint32_t before_n = __shfl_sync(0xffffffffu, wn, max(warp - 1, 0));
  const uint64_t before_w = __shfl_sync(0xffffffffu, ww, max(warp - 1, 0));
  n0 = x - n + (warp > 0 ? before_n : 0u);
  w0 = y - w + (warp > 0 ? before_w : 0ull);
}

struct SrRow {
  const float* v;     // this CTA's stretch
  int n, id0;         // its length and first id
  float top, scale;   // the largest logit; 1 / temp
  uint32_t rank, size; // of the CTA and of the cluster
  // the stretch in fours from a 16-byte boundary before it on, what is outside as NaN; in shared memory, logits and
  // then distances, where it has room, else null
  uint4* kept;
  int pad, quads;     // floats from the boundary to the stretch; fours
  LLM_D uint4 logits(int j) const {
    if (kept) return kept[j];
    const int i = 4 * j - pad;
    auto at = [&](int i) { return __float_as_uint(i >= 0 && i < n ? v[i] : NAN); };
    return make_uint4(at(i), at(i + 1), at(i + 2), at(i + 3));
  }
  LLM_D uint4 far(uint4 x) const {
    return make_uint4(dist(__uint_as_float(x.x)), dist(__uint_as_float(x.y)), dist(__uint_as_float(x.z)), dist(__uint_as_float(x.w)));
  }
  LLM_D uint4 d(int j) const { return kept ? kept[j] : far(logits(j)); }
  LLM_D int id(int j) const { return id0 + 4 * j - pad; }
  LLM_D uint32_t dist(float x) const {
    // (all of +inf at the top are at it; NaN, and what weighs nothing: none.  kSrNothing's f32 is the least at or above it)
    const float f = __fmul_rn(__fmul_rn(x == top ? 0.0f : __fsub_rn(top, x), scale), 134217728.0f);
    return f < (float)kSrNothing ? (uint32_t)f : kSrNone;
  }
};

// Counts and weights of the candidates with d >> (shift + bits) == bin, by the `bits` bits below; the sums of the
// bins before each, for the whole row, in every CTA.  FIRST: of all candidates; `fresh`: r.kept holds logits yet, and
// distances from then on.  WEIGHTS false: counts alone
template <int NT, bool FIRST, bool WEIGHTS>
LLM_D void sr_histogram(SrShared& s, const SrRow& r, int shift, int bits, uint32_t bin, bool fresh) {
  constexpr int T = kSrBins / NT, R = (T + 1) / 2;
  uint64_t* weight = FIRST ? s.weight : s.split.weight;
  uint32_t* count = FIRST ? s.count : s.split.count;
  if (!fresh) {
    sr_sync();  // (the cluster's reads of what this overwrites)
    for (int i = threadIdx.x; i < 3 * kSrBins; i += NT) s.hist[0][i] = 0u;
    __syncthreads();
  }
  auto put = [&](uint32_t d) {
    const bool in = FIRST ? d != kSrNone : d != kSrNone && (uint32_t)((uint64_t)d >> (shift + bits)) == bin;
    const uint32_t w = WEIGHTS ? sr_weight(d) : 0u, b = FIRST ? d >> shift : d >> shift & ((1u << bits) - 1u);
    if (in) {
      atomicAdd(&s.hist[0][b], 1u);
      if (WEIGHTS) {
        atomicAdd(&s.hist[1][b], w & 0xffffu);
        atomicAdd(&s.hist[2][b], w >> 16);
      }
    }
  };
#pragma unroll 2
  for (int j = threadIdx.x; j < r.quads; j += NT) {
    uint4 d;
    if (FIRST && fresh) {
      d = r.far(r.logits(j));
      if (r.kept) r.kept[j] = d;
    } else {
      d = r.d(j);
    }
    put(d.x);
    put(d.y);
    put(d.z);
    put(d.w);
  }
  sr_sync();
  // CTA = a share of the bins, two to a thread: their sums, to all
  const int per = kSrBins / r.size, b0 = r.rank * per + 2 * threadIdx.x;
  const bool mine = 2 * (int)threadIdx.x < per;
  uint32_t jn[R][2];
  uint64_t jw[R][2];
#pragma unroll
  for (int y = 0; y < R; ++y) {
    jn[y][0] = jn[y][1] = 0u;
    jw[y][0] = jw[y][1] = 0ull;
    const int b = b0 + 2 * y * NT;
    if (mine && 2 * y * NT < per) {
      uint2 n[kSrCluster], lo[kSrCluster], hi[kSrCluster];
#pragma unroll
      for (uint32_t c = 0; c < kSrCluster; ++c) {
        n[c] = lo[c] = hi[c] = make_uint2(0u, 0u);
        if (c < r.size) {
          n[c] = sr_get64(&s.hist[0][b], c);
          if (WEIGHTS) {
            lo[c] = sr_get64(&s.hist[1][b], c);
            hi[c] = sr_get64(&s.hist[2][b], c);
          }
        }
      }
#pragma unroll
      for (uint32_t c = 0; c < kSrCluster; ++c) {
        jn[y][0] += n[c].x;
        jn[y][1] += n[c].y;
        jw[y][0] += lo[c].x + ((uint64_t)hi[c].x << 16);
        jw[y][1] += lo[c].y + ((uint64_t)hi[c].y << 16);
      }
    }
  }
  if (!FIRST) sr_sync();  // (the histograms are read before the sums take their place)
#pragma unroll
  for (int y = 0; y < R; ++y) {
    const int b = b0 + 2 * y * NT;
    if (mine && 2 * y * NT < per) {
#pragma unroll
      for (uint32_t c = 0; c < kSrCluster; ++c)
        if (c < r.size) {
          sr_put(reinterpret_cast<uint64_t*>(&count[b]), c, (uint64_t)jn[y][1] << 32 | jn[y][0]);
          if (WEIGHTS) {
            sr_put(&weight[b], c, jw[y][0]);
            sr_put(&weight[b + 1], c, jw[y][1]);
          }
        }
    }
  }
  sr_sync();
  // bins before: thread = T bins
  uint32_t n[T], sn = 0u, n0, nall;
  uint64_t w[T], sw = 0ull, w0, wall;
#pragma unroll
  for (int y = 0; y < T; ++y) {
    n[y] = count[threadIdx.x * T + y];
    w[y] = WEIGHTS ? weight[threadIdx.x * T + y] : 0ull;
    sn += n[y];
    sw += w[y];
  }
  sr_scan<NT>(s, sn, sw, n0, w0, nall, wall);
#pragma unroll
  for (int y = 0; y < T; ++y) {
    count[threadIdx.x * T + y] = n0;
    if (WEIGHTS) weight[threadIdx.x * T + y] = w0;
    n0 += n[y];
    w0 += w[y];
  }
  if (threadIdx.x == 0) {
    s.all_count[FIRST ? 0 : 1] = nall;
    s.all_weight[FIRST ? 0 : 1] = wall;
  }
  __syncthreads();
}

// a[0 .. n) in ascending order, n at most kSrList; what is behind them up to a power of two is overwritten
template <int NT>
LLM_D void sr_sort(uint64_t* a, int n) {
  int n2 = 32;
  while (n2 < n) n2 <<= 1;
  for (int i = n + threadIdx.x; i < n2; i += NT) a[i] = ~0ull;
  __syncthreads();
  // steps of less than a warp's width by shuffles, i the same in all of them
  auto near = [&](int size, int step) {
    for (int i = threadIdx.x; i < n2; i += NT) {
      uint64_t x = a[i];
      for (int z = size; z <= 32 || z == size; z <<= 1) {
        const bool up = (i & z) == 0;
        for (int o = z == size ? step : z >> 1; o > 0; o >>= 1) {
          const uint64_t y = __shfl_xor_sync(0xffffffffu, x, o);
          if ((y < x) == (((i & o) == 0) == up)) x = y;
        }
        if (z > 32) break;
      }
      a[i] = x;
    }
    __syncthreads();
  };
  near(2, 1);
  for (int size = 64; size <= n2; size <<= 1) {
    for (int step = size >> 1; step > 16; step >>= 1) {
      for (int i = threadIdx.x; i < n2 / 2; i += NT) {
        const int lo = (i & ~(step - 1)) << 1 | (i & (step - 1)), hi = lo | step;
        const uint64_t x = a[lo], y = a[hi];
        if ((x > y) == ((lo & size) == 0)) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      __syncthreads();
    }
    near(size, 16);
  }
}

struct SrPlace {
  uint64_t upto;  // weights up to the candidate, its own among them
  int32_t id;
};

// The candidate at place t of the order: by count (weights false), or the one whose weight holds the t-th unit of
// the sum; t is below the whole row's.  Every CTA gets it; all walk through the same calls.
template <int NT>
LLM_D SrPlace sr_find(SrShared& s, const SrRow& r, int shift, uint64_t t, bool weights, int place) {
  uint64_t n0 = 0ull, w0 = 0ull;  // candidates and weights before the bin in hand
  uint32_t bin = 0u;              // its bits of d
  int bits = kSrBits;             // bits of the histogram in hand
  bool split = false;
  uint32_t in_bin;
  while (true) {
    // the last bin whose sum before is at most t
    const uint64_t* weight = split ? s.split.weight : s.weight;
    const uint32_t* count = split ? s.split.count : s.count;
    int lo = 0, hi = kSrBins - 1;
    const uint64_t goal = t - (weights ? w0 : n0);
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((weights ? weight[mid] : (uint64_t)count[mid]) <= goal) lo = mid;
      else hi = mid - 1;
    }
    in_bin = (lo + 1 < kSrBins ? count[lo + 1] : s.all_count[split]) - count[lo];
    n0 += count[lo];
    w0 += weight[lo];
    bin = bin << bits | (uint32_t)lo;
    if (in_bin <= kSrMost || shift == 0) break;
    bits = min(shift, kSrBits);
    shift -= bits;
    split = true;
    sr_histogram<NT, false, true>(s, r, shift, bits, bin, false);
  }
  if (split) sr_sync();  // (the split's sums are read by all before the list takes their place)
  if (in_bin > kSrMost) {
    // all at one distance: by id, stretch by stretch
    uint32_t mine = 0u;
    for (int j = threadIdx.x; j < r.quads; j += NT) {
      const uint4 d = r.d(j);
      mine += (d.x == bin) + (d.y == bin) + (d.z == bin) + (d.w == bin);
    }
    uint32_t x, n;
    uint64_t y, z;
    sr_scan<NT>(s, mine, 0ull, x, y, n, z);
    if (threadIdx.x < r.size) sr_put32(&s.same[r.rank], threadIdx.x, n);
    if (threadIdx.x == 0) s.pick = kSrNone;
    sr_sync();
    const uint64_t w = sr_weight(bin);
    uint64_t at = weights ? (t - w0) / w : t - n0;
    const uint64_t upto = w0 + (at + 1) * w;
    uint32_t before = 0u;
    for (uint32_t c = 0; c < r.rank; ++c) before += s.same[c];
    if (at >= before && at < before + n) {
      // the (at - before)-th of this stretch: threads take neighbouring ids
      const int per = (r.quads + NT - 1) / NT, j0 = min(r.quads, (int)threadIdx.x * per), j1 = min(r.quads, j0 + per);
      mine = 0u;
      for (int j = j0; j < j1; ++j) {
        const uint4 d = r.d(j);
        mine += (d.x == bin) + (d.y == bin) + (d.z == bin) + (d.w == bin);
      }
      sr_scan<NT>(s, mine, 0ull, x, y, n, z);
      uint32_t left = (uint32_t)(at - before);
      if (left >= x && left < x + mine)
        for (int j = j0; j < j1; ++j) {
          const uint4 d = r.d(j);
          const uint32_t e[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (e[y] == bin && left-- == x)
              for (uint32_t c = 0; c < r.size; ++c) sr_put32(&s.pick, c, (uint32_t)(r.id(j) + y));
        }
    }
    sr_sync();
    return SrPlace{upto, (int32_t)s.pick};
  }
  // the bin's candidates to every CTA
  uint64_t* list = s.list[place & 1];
  const uint32_t lo = bin << shift, width = 1u << shift;
  for (int j = threadIdx.x; j < r.quads; j += NT) {
    const uint4 d4 = r.d(j);
    const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (d[y] == kSrNone || d[y] - lo >= width) continue;
      const uint64_t e = (uint64_t)d[y] << 32 | (uint32_t)(r.id(j) + y);
      for (uint32_t c = 0; c < r.size; ++c) {
        const uint32_t at = sr_add(&s.listed[place], c, 1u);
        if (at < kSrMost) sr_put(&list[at], c, e);
      }
    }
  }
  sr_sync();
  const int n = (int)min(s.listed[place], (uint32_t)kSrMost);
  sr_sort<NT>(list, n);
  // running sums: thread = neighbours
  constexpr int T = kSrMost / NT;
  uint64_t w[T], sw = 0ull, at, wall;
  uint32_t nat, nall;
#pragma unroll
  for (int y = 0; y < T; ++y) {
    const int i = threadIdx.x * T + y;
    w[y] = i < n ? sr_weight((uint32_t)(list[i] >> 32)) : 0ull;
    sw += w[y];
  }
  sr_scan<NT>(s, 0u, sw, nat, at, nall, wall);
#pragma unroll
  for (int y = 0; y < T; ++y) {
    const int i = threadIdx.x * T + y;
    const uint64_t goal = t - (weights ? w0 : n0);
    if (i < n && (weights ? at <= goal && goal < at + w[y] : (uint64_t)i == goal)) {
      s.pick = (uint32_t)list[i];
      s.upto[0] = at + w[y];
    }
    at += w[y];
  }
  __syncthreads();
  const SrPlace got = {w0 + s.upto[0], (int32_t)s.pick};
  __syncthreads();
  return got;
}

// Bins lo .. lo + len - 1
struct SrBinRange {
  uint32_t lo, len;
};

// The places one after the other, each with a gathering of its own: any number of candidates at any distances
template <int NT>
LLM_D int32_t sr_one_by_one(SrShared& s, const SrRow& r, int shift, uint32_t k, uint32_t part, uint32_t least, uint32_t u) {
  uint64_t kept = s.all_weight[0];
  int place = 0;
  if (k < s.all_count[0]) kept = sr_find<NT>(s, r, shift, (uint64_t)(k - 1), false, place++).upto;
  if (part < 1u << 24) {
    const uint64_t limit = sr_share(kept, part);
    kept = sr_find<NT>(s, r, shift, limit ? limit - 1 : 0ull, true, place++).upto;
  }
  if (least > 0u) {
    uint64_t x = 0ull, y, z;
    uint32_t n, m;
    for (int j = threadIdx.x; j < r.quads; j += NT) {
      const uint4 d = r.d(j);
      auto add = [&](uint32_t d) {
        const uint32_t w = d == kSrNone ? 0u : sr_weight(d);
        if (w >= least) x += w;
      };
      add(d.x);
      add(d.y);
      add(d.z);
      add(d.w);
    }
    sr_scan<NT>(s, 0u, x, n, y, m, z);
    if (threadIdx.x < r.size) sr_put(&s.above[r.rank], threadIdx.x, z);
    sr_sync();
    x = 0ull;
    for (uint32_t i = 0; i < r.size; ++i) x += s.above[i];
    kept = min(kept, x);
  }
  return sr_find<NT>(s, r, shift, sr_share(kept, u), true, place).id;
}

// The places together.  The histogram bounds the sum that each place keeps, so the bins that the next can be in: one
// gathering of the candidates of all these bins, and the rest is the first CTA's alone.  HEAD, for a small k: all up to
// the k-th candidate's bin, of which only the counts are known.  False if they are too many.
template <int NT, bool HEAD>
LLM_D bool sr_together(SrShared& s, const SrRow& r, int shift, uint32_t k, uint32_t part, uint32_t least, uint32_t u, int32_t& id) {
  constexpr int T = kSrBins / NT;
  const int tid = threadIdx.x;
  const uint64_t all = HEAD ? (uint64_t)0 : s.all_weight[0];
  const uint32_t count = s.all_count[0];
  auto weight_at = [&](uint32_t b) { return HEAD ? (uint64_t)0 : b < kSrBins ? s.weight[b] : all; };
  auto count_at = [&](uint32_t b) { return b < kSrBins ? s.count[b] : count; };
  uint64_t w[T + 1];
#pragma unroll
  for (int y = 0; y <= T; ++y) w[y] = weight_at(tid * T + y);
  auto mark = [&](uint64_t goal, int slot) {
#pragma unroll
    for (int y = 0; y < T; ++y)
      if (w[y] <= goal && goal < w[y + 1]) s.bin[slot] = tid * T + y;
  };
  SrBinRange in[4] = {{0u, 0u}, {0u, 0u}, {0u, 0u}, {0u, 0u}};
  uint64_t lo = all, hi = all;  // bounds of the sum that is kept
  uint32_t least_lo = 0u, least_hi = 0u;
  if (k < count) {
#pragma unroll
    for (int y = 0; y < T; ++y)
      if (count_at(tid * T + y) <= k - 1 && k - 1 < count_at(tid * T + y + 1)) s.bin[0] = tid * T + y;
    __syncthreads();
    const uint32_t b = s.bin[0];
    in[0] = HEAD ? SrBinRange{0u, b + 1u} : SrBinRange{b, 1u};
    lo = weight_at(b);
    hi = weight_at(b + 1);
  } else if (HEAD) {
    in[0] = SrBinRange{0u, (uint32_t)kSrBins};
  }
  auto before = [](uint64_t limit) { return limit ? limit - 1 : 0ull; };
  if (!HEAD && part < 1u << 24) {
    mark(before(sr_share(lo, part)), 1);
    mark(before(sr_share(hi, part)), 2);
    __syncthreads();
    in[1] = SrBinRange{s.bin[1], s.bin[2] - s.bin[1] + 1};
    lo = weight_at(s.bin[1]);
    hi = weight_at(s.bin[2] + 1);
  }
  if (least > 0u) {
    // weights round to `least` or more up to about this distance
    const uint32_t d = (uint32_t)fmaxf(-logf(((float)least - 0.5f) * 0x1p-31f) * 134217728.0f, 0.0f);
    least_lo = min((d > kSrNear ? d - kSrNear : 0u) >> shift, (uint32_t)kSrBins - 1);
    least_hi = min((d + kSrNear) >> shift, (uint32_t)kSrBins - 1);
    if (HEAD) {
      // (all of the bins in which a weight can be on either side of `least`, or none)
      if (least_lo < in[0].len) in[0].len = max(in[0].len, least_hi + 1);
      least_lo = 0u;
      least_hi = kSrBins - 1;
    } else {
      in[2] = SrBinRange{least_lo, least_hi - least_lo + 1};
      lo = min(lo, weight_at(least_lo));
      hi = min(hi, weight_at(least_hi + 1));
    }
  }
  if (!HEAD) {
    mark(sr_share(lo, u), 3);
    mark(sr_share(hi, u), 4);
    __syncthreads();
    in[3] = SrBinRange{s.bin[3], s.bin[4] - s.bin[3] + 1};
  }
  // in order, those that touch as one
  auto swap = [&](int a, int b) {
    if (in[a].lo > in[b].lo) {
      const SrBinRange x = in[a];
      in[a] = in[b];
      in[b] = x;
    }
  };
  swap(0, 1); swap(2, 3); swap(0, 2); swap(1, 3); swap(1, 2);
  uint32_t n = 0u;
#pragma unroll
  for (int j = 1; j < 4; ++j)
    if (in[j - 1].len == 0u || in[j].lo <= in[j - 1].lo + in[j - 1].len) {
      const uint32_t end = max(in[j - 1].lo + in[j - 1].len, in[j].lo + in[j].len);
      if (in[j - 1].len > 0u) in[j] = SrBinRange{in[j - 1].lo, end - in[j - 1].lo};
      in[j - 1].len = 0u;
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) n += count_at(in[j].lo + in[j].len) - count_at(in[j].lo);
  if (n > kSrList) return false;
  // ---- the candidates: to a list of the CTA's own, and that to the first CTA's ----
  auto take = [&](uint32_t d, int id) {
    const uint32_t b = d >> shift;
    if ((b - in[0].lo < in[0].len || b - in[1].lo < in[1].len || b - in[2].lo < in[2].len || b - in[3].lo < in[3].len) && d != kSrNone)
      s.places[atomicAdd(&s.listed[3], 1u)] = (uint64_t)d << 32 | (uint32_t)id;
  };
#pragma unroll 2
  for (int j = tid; j < r.quads; j += NT) {
    const uint4 d = r.d(j);
    const int id = r.id(j);
    take(d.x, id);
    take(d.y, id + 1);
    take(d.z, id + 2);
    take(d.w, id + 3);
  }
  if (r.size > 1) {
    __syncthreads();
    if (r.rank != 0) {
      const uint32_t mine = s.listed[3];
      if (tid == 0) s.pick = sr_add(&s.listed[3], 0, mine);
      __syncthreads();
      const uint32_t base = s.pick;
      for (uint32_t i = tid; i < mine; i += NT) sr_put(&s.places[base + i], 0, s.places[i]);
    }
    sr_sync();
    if (r.rank != 0) return true;
  } else {
    __syncthreads();
  }
  uint64_t* list = s.places;
  sr_sort<NT>(list, (int)n);
  // ---- running sums, and with the bins that were left out ----
  constexpr int E = kSrList / NT;
  uint64_t at[E], wt[E], own = 0ull, wall;
  uint32_t rank[E], x, y;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t i = tid * E + e;
    wt[e] = i < n ? sr_weight((uint32_t)(list[i] >> 32)) : 0ull;
    own += wt[e];
  }
  // (by range: what was left out since the one before)
  uint64_t skip_w[4], end_w = 0ull, run;
  uint32_t skip_n[4], end_n = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    skip_w[j] = 0ull;
    skip_n[j] = 0u;
    if (in[j].len > 0u) {
      skip_w[j] = weight_at(in[j].lo) - end_w;
      skip_n[j] = count_at(in[j].lo) - end_n;
      end_w = weight_at(in[j].lo + in[j].len);
      end_n = count_at(in[j].lo + in[j].len);
    }
  }
  sr_scan<NT>(s, 0u, own, x, run, y, wall);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t i = tid * E + e, b = i < n ? (uint32_t)(list[i] >> 32) >> shift : 0u;
    at[e] = run;
    rank[e] = i;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (b >= in[j].lo) {
        at[e] += skip_w[j];
        rank[e] += skip_n[j];
      }
    run += wt[e];
  }
  uint64_t kept = HEAD ? wall : all;
  if (k < count) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (wt[e] > 0ull && rank[e] == k - 1) s.upto[0] = at[e] + wt[e];
    __syncthreads();
    kept = s.upto[0];
  }
  auto place = [&](uint64_t goal, int slot) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (at[e] <= goal && goal < at[e] + wt[e]) {
        s.upto[slot] = at[e] + wt[e];
        s.pick = (uint32_t)list[tid * E + e];
      }
    __syncthreads();
  };
  if (part < 1u << 24) {
    place(before(sr_share(kept, part)), 1);
    kept = s.upto[1];
  }
  if (least > 0u) {
    uint64_t above = 0ull, z;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t b = wt[e] > 0ull ? (uint32_t)(list[tid * E + e] >> 32) >> shift : 0u;
      if (b >= least_lo && b <= least_hi && wt[e] >= least) above += wt[e];
    }
    sr_scan<NT>(s, 0u, above, x, z, y, wall);
    kept = min(kept, weight_at(least_lo) + wall);
  }
  __syncthreads();
  place(sr_share(kept, u), 2);
  id = (int32_t)s.pick;
  return true;
}

// cluster = row; the CTA's stretch stays in shared memory if `keep`
template <int NT>
__global__ void __launch_bounds__(NT) sample_rows_kernel(const SampleRowsArgs a, int keep) {
  extern __shared__ __align__(16) unsigned char raw[];
  SrShared& s = *reinterpret_cast<SrShared*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  SrRow r;
  r.rank = sr_rank();
  r.size = sr_size();
  const int b = blockIdx.x / r.size;
  const int per = (a.V + r.size - 1) / r.size;
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
  if (tid < 4) s.listed[tid] = 0u;
  sr_arrive();
  // ---- the largest logit, and the smallest that is not -inf ----
  r.pad = (int)(reinterpret_cast<uintptr_t>(r.v) >> 2 & 3u);
  r.quads = r.n > 0 ? (r.pad + r.n + 3) >> 2 : 0;
  r.kept = nullptr;
  uint4* kept = reinterpret_cast<uint4*>(raw + sizeof(SrShared));
  float most_v = -INFINITY, least_v = INFINITY;
  const float4* v4 = reinterpret_cast<const float4*>(r.v - r.pad);  // (read where all four are the stretch's)
#pragma unroll 8
  for (int j = tid; j < r.quads; j += NT) {
    uint4 x;
    if (4 * j >= r.pad && 4 * j + 4 <= r.pad + r.n) x = *reinterpret_cast<const uint4*>(v4 + j);
    else x = r.logits(j);
    if (keep) kept[j] = x;
    auto see = [&](uint32_t bits) {  // (maxima and minima leave NaN out)
      const float v = __uint_as_float(bits);
      most_v = fmaxf(most_v, v);
      least_v = fminf(least_v, v == -INFINITY ? INFINITY : v);
    };
    see(x.x);
    see(x.y);
    see(x.z);
    see(x.w);
  }
  if (keep) r.kept = kept;
  // (as keys, which are whole numbers; an empty stretch: those of -inf and +inf)
  const uint32_t top = __reduce_max_sync(0xffffffffu, sr_key(most_v)), low = __reduce_min_sync(0xffffffffu, sr_key(least_v));
  if (lane == 0) {
    s.num[warp] = top;
    s.low_of[warp] = low;
  }
  for (int i = tid; i < 3 * kSrBins / 4; i += NT) reinterpret_cast<uint4*>(s.hist[0])[i] = make_uint4(0u, 0u, 0u, 0u);
  // (every CTA has started and set its lists' lengths before another writes to it)
  __syncthreads();
  sr_wait();
  if (warp == 0) {
    const uint32_t x = __reduce_max_sync(0xffffffffu, lane < NT / 32 ? s.num[lane] : 0u);
    const uint32_t y = __reduce_min_sync(0xffffffffu, lane < NT / 32 ? s.low_of[lane] : 0xffffffffu);
    if (lane < r.size) {
      sr_put32(&s.top[r.rank], lane, x);
      sr_put32(&s.low[r.rank], lane, y);
    }
  }
  sr_sync();
  uint32_t key = 0u, low_key = 0xffffffffu;
  for (uint32_t i = 0; i < r.size; ++i) {
    key = max(key, s.top[i]);
    low_key = min(low_key, s.low[i]);
  }
  if (key <= 0x007fffffu) {  // every logit is -inf or NaN
    if (r.rank == 0 && tid == 0) a.ids[b] = 0;
    return;
  }
  r.top = sr_unkey(key);
  if (greedy) {
    // the first that is as large
    int first = 0x7fffffff;
    for (int j = tid; j < r.quads; j += NT) {
      const uint4 x = r.logits(j);
      const int id = r.id(j);
      const float v[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (v[y] == r.top) first = min(first, id + y);
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) s.num[warp] = (uint32_t)first;
    __syncthreads();
    if (warp == 0) {
      first = (int)__reduce_min_sync(0xffffffffu, lane < NT / 32 ? s.num[lane] : 0x7fffffffu);
      if (lane == 0) sr_put32(&s.same[r.rank], 0, (uint32_t)first);
    }
    sr_sync();
    if (r.rank == 0 && tid == 0) {
      for (uint32_t i = 0; i < r.size; ++i) first = min(first, (int)s.same[i]);
      a.ids[b] = first;
    }
    return;
  }
  r.scale = fminf(__fdiv_rn(1.0f, temp), 3.402823466e38f);
  // ---- the histogram over the range that the distances have ----
  const float span = __fmul_rn(__fsub_rn(r.top, sr_unkey(low_key)), r.scale);
  const uint32_t most = span < 22.2f ? (uint32_t)(span * 134217728.0f) : 0xb1a00000u;
  const int shift = max(0, 32 - __clz((int)most) - kSrBits);
  const uint32_t part = sr_part(p), least = (uint32_t)(min_p * 2147483648.0f);
  int32_t id = 0;
  const bool small = k <= kSrMost;  // (one addition a candidate, and no weight, in place of three)
  if (small) {
    sr_histogram<NT, true, false>(s, r, shift, kSrBits, 0u, true);
    if (sr_together<NT, true>(s, r, shift, (uint32_t)k, part, least, sr_part(u), id)) {
      if (r.rank == 0 && tid == 0) a.ids[b] = id;
      return;
    }
  }
  sr_histogram<NT, true, true>(s, r, shift, kSrBits, 0u, !small);
  // ---- what is kept, and the draw from it ----
  if (!sr_together<NT, false>(s, r, shift, (uint32_t)k, part, least, sr_part(u), id))
    id = sr_one_by_one<NT>(s, r, shift, (uint32_t)k, part, least, sr_part(u));
  if (r.rank == 0 && tid == 0) a.ids[b] = id;
}

template <int NT>
cudaError_t sr_launch(const SampleRowsArgs& a, int size, cudaStream_t s) {
  const size_t stretch = ((size_t)((a.V + size - 1) / size) + 6) / 4 * 16;
  const bool keep = sizeof(SrShared) + stretch <= 227u * 1024u;
  const size_t bytes = sizeof(SrShared) + (keep ? stretch : 0);
  cudaError_t e = cudaFuncSetAttribute(sample_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * size);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_rows_kernel<NT>, a, (int)keep);
}

}  // namespace

cudaError_t launch_sample_rows(const SampleRowsArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs of a row: as many as have an SM each, so that few rows take little time and many few barriers and joins
  // (8 / 4 / 2: 1 row of 49152 15 / 17 / 21 us, 32 of 128256 42 / 32 / 48, 256 of 50257 183 / 109 / 75);
  // more where a stretch has no room in shared memory, or a bin's sum none in 32 bits
  int size = (int64_t)a.B * 8 <= sms ? 8 : (int64_t)a.B * 4 <= sms ? 4 : 2;
  while (size < kSrCluster && sizeof(SrShared) + (size_t)a.V / size * 4 > 226u * 1024u) size *= 2;
  // (512 threads: 15 us for that row, 1024 16)
  return (a.V + size - 1) / size <= 8192 ? sr_launch<512>(a, size, s) : sr_launch<1024>(a, size, s);
}

}  // namespace llm
