// Attention over an 8-bit cache on the 5th-generation tensor cores, head sizes 64 and 128: the
// kernel template (its instantiations, a translation unit each: qattn_tc<head size>_<type>.cu).
//
// The codes go from HBM to shared memory by TMA, the keys' from there into e4m3 MMAs as they are.  The
// f32 (bf16) queries that meet them enter as NP e4m3 pieces, x = 2^e (x_0 + x_1 / 32 + x_2 / 32^2 + ...)
// with |x| / 2^e <= 256, each piece the rounding of what the ones before left over (at most half a step, 8
// of 256, so 32 times it is in range again).  A piece takes four bits: four pieces leave 2^-16 of an element
// at worst, or 2^-33 of the largest where it is tiny (f32); two hold a bf16 query's eight bits.  The pieces
// are columns of their own, so every accumulator sums like with like in f32 and the powers of 32 are applied
// once, in registers.  The values are widened to bf16 (exact) in shared memory, in the place of the tile's
// keys and values: their softmax weights, as bf16 pieces, have the exponents of f32, so that a weight keeps its
// digits however small it is beside the largest.  (As e4m3 pieces, codes as they lie, tiles took 5 to 15% less
// time -- 32 rows of up to 2100: 30 us, 131072 positions with 8 tokens: 81 -- but weights below 2^-20 (f32:
// 2^-27) of the largest were lost, and where the heavy positions' values are small those are the result.)
//
// A tile is 128 positions of one row and key/value head against up to C = 16 NC / NP columns, the
// (token, query head) pairs of up to C / g tokens that share the codes:
//   S [128 positions][16 NC]  = K [128][HD] Q^T      A = keys, K-major as stored; B = query pieces
//   softmax                     thread = position: pieces summed, block scales applied, weights split
//   O [HD][NW]               += V^T [HD][128] P^T     A = widened values, M-major; B = weight pieces
// With the positions on the M side a tile costs HD / 32 + 8 MMAs however few columns there are, and a thread
// writes its position's pieces with 16-byte stores, one per 8 pieces (B's N-major layout).
//
// Running maxima are lazy: a column's reference makes the first tile's largest weight 1 and moves only when
// a weight exceeds 2^32 (then that one becomes 1), so the accumulators in tensor memory are hardly ever
// rescaled.  The values' block scales ride on the weights, relative to the largest scale seen (also lazy).
//
// One CTA: a producer warp (a ring of tiles by TMA, their block scales by 4-byte asynchronous copies), a
// warp that issues the MMAs, and 16 softmax warps per SM: two groups of four take the tiles of a segment
// in turn, each with its own accumulators, so that one group's softmax overlaps the other's loads and
// products; up to 8 columns two CTAs share an SM, beyond that a tile's columns are halved between two
// groups.  What runs once per segment is kept
// in short loops: cold straight-line code runs at the pace of instruction fetch (unrolled over 32
// columns, the end of a segment took 25 us).  The (row, token tile, kv head, tile) sequence is cut into
// one equal run per CTA; the parts of a unit cut across CTAs meet in global memory once a CTA's run is
// done, where the last CTA to arrive (a ticket, nobody waits) adds them in CTA order.  So rows of any
// lengths fill the SMs evenly and the result does not depend on timing.
//
// Bound by HBM where a tile's columns are few and rows long, by the latency of a tile's chain (scores, widening,
// weights, products) from about 16 columns on (32 columns: 49% of issue slots busy, shared memory below half, the
// tensor pipe at 14%), and by latencies where a CTA has only a few tiles (a segment costs about 4 us besides its
// tiles: first loads, the groups'
// sums, the join).  Widening by integer steps instead of conversions, rolled or before the scores are there,
// measured the same.  GB300, f32 queries, heads of 128, groups of 4, 8 key/value heads: 8 rows of 32768
// positions 92 us (538 MB: 5.8 TB/s, 86% of the copy rate); one row of 131072 56 us (4.8 TB/s); 32 rows of up
// to 2100 34 us (108 MB: 3.2 TB/s); one row of 2048 10.1 us; five tokens in each of 32 rows of 2048 69 us (20
// columns).  bf16 queries, 8 tokens at 131072 positions (32 columns): 94 us (269 MB: 2.9 TB/s).
#pragma once
#include "attention.cuh"
#include "qcache.cuh"
#include "tc.cuh"

namespace llm {

constexpr int kQaTile = 128;                       // positions per tile
constexpr uint64_t kQaWaitCycles = 1000000000ull;  // about 0.5 s
constexpr float kQaMost = 32.0f;                   // log2 of the largest weight that moves no reference
// Tiles that a group's products are summed over in their accumulator before they are added to the group's sums: a
// product's additions are not rounded to nearest but cut off (8 per tile, each by up to 2^-23 of the sum), so
// that with all of a run's tiles in one accumulator digits of one sign are lost.  f32, 8 rows of 32768 positions:
// 3.9e-6 of the result, with 4 tiles 0.9e-6, with one 0.8e-6 at 1 to 6% more time (f32 sums in one order:
// 1.4e-6).  bf16: 256 cuts are still 2^-16, well below the output's rounding (32 columns: 94 us, with 4 tiles 96).
template <int QT> constexpr int kQaRun = QT ? 32 : 4;
constexpr int kQaNear = 4;                         // most tiles by which a cut moves to a unit's end
constexpr float kQaNone = -3.0e38f;                // a reference before any score
constexpr size_t kQaSmem = 232448;                 // shared memory a CTA can have

template <int HD, int NP, int NC>
struct QaShape {
  static constexpr int N = 16 * NC;                // score columns
  static constexpr int C = N / NP;                 // (token, head) columns
  static constexpr int CPC = 16 / NP;              // of them per 16 score columns
  // Up to 8 columns two CTAs per SM (16 rows of 5 tokens of 32 heads of 64: 30 us against 43 us with one; 32 rows
  // of one token of groups of 4: 34 against 40; one row of 131072: 56 against 64), more in one CTA whose groups
  // halve them (16 rows of 16 columns at 2048 positions: 33 us against 42 us as two CTAs of whole columns)
  static constexpr int CTAS = C <= 8 ? 2 : 1;
  static constexpr int HV = C <= 8 ? 1 : 2;        // groups that share a tile's columns
  static constexpr int CT = C / HV;                // columns of a thread
  static constexpr int NCH = NC / HV;              // 16-column chunks of scores of a thread
  // A weight's bf16 pieces: three for f32 queries (2^-26 of the weight; with two, 2^-17, outputs are twice as far
  // off as f32 sums leave them), two for bf16 (with one the outputs' error is 2.4e-3 of them instead of the
  // 1.7e-3 that their own rounding makes).  A thread's pieces y of its columns c lie at y * CTP + c, 8 in 16 bytes.
  static constexpr int WP = NP == 4 ? 3 : 2;
  static constexpr int CTP = CT <= 4 ? 4 : (CT + 7) / 8 * 8;
  static constexpr int NCW = (WP * CTP + 7) / 8;   // 16-byte chunks of pieces of a thread
  static constexpr int HW = 8 * NCW;               // accumulator columns of a thread
  static constexpr int NW = (HV * HW + 15) / 16 * 16;  // of the product over the values (an MMA takes multiples of 16;
                                                       // what is more is never read)
  static constexpr int KB = kQaTile * HD;          // bytes of a tile of keys (or values)
  static constexpr int STAGE = 2 * KB;
  static constexpr int QB = N * HD;                // query pieces of a segment
  static constexpr int PB = 2 * kQaTile * NW;      // weight pieces of one parity's groups
  static constexpr int COLS = 2 * (N + NW + C);
  static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;  // columns
  static constexpr int NS = 256 * HV;              // softmax threads
  static constexpr int NT = NS + 64;               // all threads
  static constexpr size_t MISC = 4096;
  static constexpr size_t BUDGET = kQaSmem / CTAS - (CTAS > 1 ? 1024 : 0);
  static constexpr int FIT = (int)((BUDGET - QB - 2 * PB - MISC - 1024) / STAGE);
  static constexpr int ST = FIT < 8 ? FIT : 8;     // ring stages
  static constexpr size_t SMEM = 1024 + (size_t)ST * STAGE + QB + 2 * PB + MISC;
  static constexpr uint32_t SWZ = HD == 128 ? 2 : 4;  // 128- or 64-byte swizzle
  static_assert(ST >= 2, "ring");
  static_assert(CT % 4 == 0 && COLS <= 512, "columns");
  // (the weights' buffers hold a segment's sums at its end)
  static_assert(2 * PB >= C * HD * 4 && 2 * PB >= (NS > C * HD / 4 ? NS * 16 : 0), "sums");
};

// one tile of tokens: ntok tokens whose queries are rows qrow .. of q; token i sees start <= t < end0 + i
struct QaUnit {
  int b;          // the row (or pass entry) whose places hold the positions
  int ntok;
  int64_t qrow;
  int start, end0, last;  // last: positions the last token sees end here
  int tile0, nt;  // its position tiles
};

LLM_D QaUnit qa_unit(const QAttnArgs& a, int t) {
  QaUnit u;
  if (a.r.step) {
    if (a.tiles) {
      const int32_t* e = a.tiles + 4 + 4 * (size_t)t;
      u.b = e[0];
      u.ntok = e[1];
      u.start = e[3];
    } else {
      u.b = q_entry(a.r, t);
      u.ntok = 1;
      u.start = row_start(a.r.step, u.b);
    }
    u.qrow = u.b;
    u.end0 = row_pos(a.r.step, u.b) + 1;
  } else {
    u.b = a.nct == 1 ? t : (int)((uint32_t)t / (uint32_t)a.nct);
    const int n = q_count(a.r, u.b), i0 = (t - u.b * a.nct) * a.tpt;
    int len = a.r.first[u.b];
    if (len < 0 || len > a.r.limit) {
      q_report(a.r.status, kErrPosRange);
      len = 0;
    }
    u.ntok = max(0, min(a.tpt, n - i0));
    u.qrow = (int64_t)u.b * a.r.S + i0;
    u.start = 0;
    u.end0 = len - n + i0 + 1;
  }
  u.last = u.end0 + u.ntok - 1;
  u.tile0 = u.start / kQaTile;
  u.nt = u.ntok > 0 && u.last > u.start ? (u.last + kQaTile - 1) / kQaTile - u.tile0 : 0;
  return u;
}

LLM_D bool qa_place(const QAttnArgs& a, int b, int pos, int& row, int& pp) {
  if (!a.r.step) return q_place(a.r, a.c, b, pos, row, pp);
  cache_slot(a.r.step, a.c.cap, b, pos, row, pp);
  return true;
}

// The new key and value of row b and kv head j of a decode step into the cache, by one warp: lanes 0..15 the
// key, 16..31 the value, as quantise_run (qcache.cu) does for one token.  The block lies in the row's last
// tile, which one CTA loads, so nothing else of this call reads it.  A kernel of its own for it is one more
// launch per layer (8B shape, a step of one row: 2.87 ms against 2.82 ms; of 32 rows: 4.79 against 4.74).
template <int HD>
LLM_D void qa_store_new(const QAttnArgs& a, int b, int j) {
  constexpr int E = HD / 16;
  const int lane = threadIdx.x & 31, side = lane >> 4, sub = lane & 15;
  const void* src = side ? a.new_v : a.new_k;
  const int64_t at = ((int64_t)b * a.c.kv + j) * HD + sub * E;
  float x[E];
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    if (a.new_t) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(src) + at + e);
      x[e] = bf16_lo(u.x); x[e + 1] = bf16_hi(u.x); x[e + 2] = bf16_lo(u.y); x[e + 3] = bf16_hi(u.y);
    } else {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + at + e);
      x[e] = f.x; x[e + 1] = f.y; x[e + 2] = f.z; x[e + 3] = f.w;
    }
  }
  int row, pp;
  cache_slot(a.r.step, a.c.cap, b, row_pos(a.r.step, b), row, pp);
  const int t0 = pp % kQBlock;
  const size_t head = (size_t)row * a.c.kv + j;
  uint8_t* codes = (side ? a.c.v : a.c.k) + (head * a.c.cap + (pp - t0)) * HD;
  float* scale = (side ? a.c.vs : a.c.ks) + head * (a.c.cap / kQBlock) + pp / kQBlock;
  const float s_old = t0 > 0 ? *scale : 0.f;
  uint32_t top = 0u;
#pragma unroll
  for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool fine = top < 0x7f800000u && s_old == s_old;
  const float s = fine ? fmaxf(q_scale(__uint_as_float(top)), s_old) : __uint_as_float(0x7fc00000u);
  if (fine && s > s_old && t0 > 0) {
    const float f = s_old * q_recip(s);
    uint32_t* c4 = reinterpret_cast<uint32_t*>(codes);
#pragma unroll 1
    for (int q = sub; q < t0 * (HD / 4); q += 16) {
      const float4 v = e4m3_quad(c4[q]);
      c4[q] = e4m3x2(v.x * f, v.y * f) | e4m3x2(v.z * f, v.w * f) << 16;
    }
  }
  const float r = fine ? q_recip(s) : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 4)
    *reinterpret_cast<uint32_t*>(codes + t0 * HD + sub * E + e) =
        fine ? e4m3x2(x[e] * r, x[e + 1] * r) | e4m3x2(x[e + 2] * r, x[e + 3] * r) << 16 : 0u;
  __syncwarp();  // every lane has read the old scale
  if (sub == 0) *scale = s;
  fence_proxy_async_global();  // (the tile's bulk copies read these codes)
  __syncwarp();
}

// a 4-byte asynchronous copy to shared memory, and this thread's arrival on an mbarrier once its copies
// are done
LLM_D void qa_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
LLM_D void qa_copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// f32 maxima by the integer reduction: an order-preserving map of the bits (NaN left out as -inf)
LLM_D float qa_warp_max(float v) {
  const uint32_t u = __float_as_uint(v == v ? v : -INFINITY);
  const uint32_t m = __reduce_max_sync(0xffffffffu, u & 0x80000000u ? ~u : u | 0x80000000u);
  return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
}

LLM_D float qa_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// T tiles cut into G runs, the first T % G of them one longer; a cut within `near` tiles of a unit's
// start or end moves there: a segment costs about as much as four tiles besides its tiles, and a cut unit
// its join, which whole units save at the price of runs that are uneven by as much (16 rows of 5 tokens,
// 32 heads of 64, about 900 positions: 35 us without, 30 us with; 32 rows of up to 2100 positions, 8 heads of
// 128: 33 without, 34 with).
struct QaCut {
  int q, r, near;
  LLM_D void make(int T, int G) {
    q = (int)((uint32_t)T / (uint32_t)G);
    r = T - q * G;
    near = min(kQaNear, q * 3 / 8);
  }
  LLM_D int begin(int c) const { return c * q + min(c, r); }
  // the run that holds tile i, before cuts move
  LLM_D int owner(int i) const {
    const int head = r * (q + 1);
    const bool in = i < head;
    return (in ? 0 : r) + (int)((uint32_t)(in ? i : i - head) / (uint32_t)(in ? q + 1 : q));
  }
  // a cut at x inside the unit of nt tiles from u0
  LLM_D int moved(int x, int u0, int nt) const {
    const int d0 = x - u0, d1 = nt - d0;
    return d0 <= d1 ? (d0 <= near ? u0 : x) : d1 <= near ? u0 + nt : x;
  }
  // the first and last run of a unit that is cut: its cuts lie more than `near` from both ends
  LLM_D int first(int u0) const { return owner(u0 + near); }
  LLM_D int last(int u0, int nt) const { return owner(u0 + nt - 1 - near); }
};

// four elements of the output
template <int QT>
LLM_D void qa_put4(void* out, int64_t at, float4 o) {
  if constexpr (QT)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = o;
}

// sixteen e4m3 codes to bf16 (exact)
LLM_D void qa_widen16(const uint4& u, uint4& lo, uint4& hi) {
  const float4 a = e4m3_quad(u.x), b = e4m3_quad(u.y), c = e4m3_quad(u.z), d = e4m3_quad(u.w);
  lo = make_uint4(bf16x2(a.x, a.y), bf16x2(a.z, a.w), bf16x2(b.x, b.y), bf16x2(b.z, b.w));
  hi = make_uint4(bf16x2(c.x, c.y), bf16x2(c.z, c.w), bf16x2(d.x, d.y), bf16x2(d.z, d.w));
}

// The values of a tile in bf16, in the place of its keys and values (`stage`), whose scores are done: the row of
// a position has HD bytes in either half of the stage; the first HD / 2 dimensions go where its key was, the
// others where its codes were, swizzled as the codes were.  HV lanes of one warp share a row (r; sub: the lane's
// place), so that no other warp touches what this one reads or writes, and a step overwrites only codes that
// have been read.  Rows that no column sees (live false: dead data, any code, NaN's among them) become zeros.
template <int HD, int HV>
LLM_D void qa_widen_row(unsigned char* stage, int r, int sub, bool live) {
  constexpr int HB = HD / 32;  // 16-byte chunks of codes of half a row
  const int swz = HD == 128 ? r & 7 : r >> 1 & 3;
  unsigned char* codes = stage + kQaTile * HD + r * HD;
#pragma unroll 4
  for (int i = 0; i < 2 * HB; i += HV) {
    const int from = i + sub, to = 2 * (from % HB);
    uint4 x = *reinterpret_cast<const uint4*>(codes + (from ^ swz) * 16), lo, hi;
    if (!live) x = make_uint4(0u, 0u, 0u, 0u);
    if (HV > 1) __syncwarp();
    qa_widen16(x, lo, hi);
    unsigned char* dst = i < HB ? stage + r * HD : codes;
    *reinterpret_cast<uint4*>(dst + (to ^ swz) * 16) = lo;
    *reinterpret_cast<uint4*>(dst + ((to + 1) ^ swz) * 16) = hi;
  }
}

// the walk of one CTA's run over (token tile, kv head, position tiles)
struct QaWalk {
  QaUnit u;
  int t, j, k0, k1;
  int st, end, off;  // off: place of (t, head 0) in the sequence
  LLM_D void begin(const QAttnArgs& a, int t_, int off_, int c0, int c1) {
    t = t_; off = off_; st = c0; end = c1;
    if (st >= end) return;
    u = qa_unit(a, t);
    if (st - off == a.c.kv * u.nt) {  // (a cut moved to the end of its token tile)
      off = st;
      do u = qa_unit(a, ++t);
      while (u.nt == 0);
    }
    j = (int)((uint32_t)(st - off) / (uint32_t)u.nt);
    k0 = st - off - j * u.nt;
    cut();
  }
  LLM_D void cut() { k1 = min(u.nt, k0 + (end - st)); }
  LLM_D bool there() const { return st < end; }
  LLM_D int unit0() const { return off + j * u.nt; }
  LLM_D void next(const QAttnArgs& a) {
    st += k1 - k0;
    if (st >= end) return;  // (a unit that goes on belongs to the next CTA)
    k0 = 0;
    if (++j == a.c.kv) {
      j = 0;
      off += a.c.kv * u.nt;
      do u = qa_unit(a, ++t);
      while (u.nt == 0);
    }
    cut();
  }
};

template <int HD, int NP, int NC, int QT>
__global__ void __launch_bounds__(QaShape<HD, NP, NC>::NT, QaShape<HD, NP, NC>::CTAS)
    qattn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const QAttnArgs a) {
  using X = QaShape<HD, NP, NC>;
  constexpr int N = X::N, C = X::C, CPC = X::CPC, ST = X::ST, CT = X::CT, NCH = X::NCH, HV = X::HV, NS = X::NS;
  constexpr int NW = X::NW, WP = X::WP, CTP = X::CTP, NCW = X::NCW;
  extern __shared__ unsigned char qraw[];
  const uint32_t s_raw = smem_u32(qraw);
  unsigned char* base = qraw + (((s_raw + 1023u) & ~1023u) - s_raw);
  const uint32_t s_ring = smem_u32(base);
  unsigned char* qbuf = base + (size_t)ST * X::STAGE;
  unsigned char* pbuf = qbuf + X::QB;                        // [2][PB]
  float* qsc = reinterpret_cast<float*>(pbuf + 2 * X::PB);   // [C] query scale, in units of log2
  int* cend = reinterpret_cast<int*>(qsc + C);               // [C] end of the positions a column sees
  float* gref = reinterpret_cast<float*>(cend + C);          // [2][C] references, by parity of the tile
  float* wmax = gref + 2 * C;                                // [2][4][C] warps' maxima; at the end, their sums
  float* ffac = wmax + 8 * C;                                // [2][C] at the end: factors of the two parities
  float* ssc = ffac + 2 * C;                                 // [ST][16] a tile's block scales: keys (-1: not seen), values
  float* wvs = ssc + 16 * ST;                                // [4][4] warps' largest value scales
  float* gvs = wvs + 16;                                     // [4] the groups' value scales
  int64_t* coff = reinterpret_cast<int64_t*>(gvs + 4);       // [C] a column's place in the unit's output
  const uint32_t bars = (smem_u32(coff + C) + 7u) & ~7u;
  const uint32_t b_full = bars, b_empty = b_full + 8 * ST, b_s = b_empty + 8 * ST, b_p = b_s + 16, b_pv = b_p + 16,
                 b_q = b_pv + 16;
  static_assert((size_t)C * 4 * 16 + 80 + 80 * ST + 8 * C + 112 <= X::MISC, "shared memory");
  __shared__ uint32_t s_tmem;
  __shared__ int s_t, s_off, s_total, s_begin, s_end;
  // the units that this CTA holds a part of (the first and the last of its run)
  struct Pending {
    int64_t qrow;
    int j, used, first, np, last;
  };
  __shared__ Pending s_pend[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 32) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(b_full + 8u * i, 17);
      mbar_init(b_empty + 8u * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8u * i, 1);
      mbar_init(b_p + 8u * i, 128 * HV);
      mbar_init(b_pv + 8u * i, 1);
    }
    mbar_init(b_q, 1);
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), X::TMEM);
    tmem_relinquish();
  }

  // (a step's state and tiles were written before its kernels: only queries and cache wait for the
  // previous kernel, below)
  // this CTA's run: the token tiles' position tiles are counted lane by lane (contiguous stretches),
  // and the lane whose stretch holds the run's start finds its token tile
  const int nq = a.r.step ? (a.tiles ? a.tiles[1] : a.r.B) : a.r.B * a.nct;
  if (warp == 0) {
    // (unsigned: sums of numbers below 2^31)
    const uint32_t nu = (uint32_t)nq, pu = (nu + 31u) / 32u, tu = min(nu, lane * pu);
    const int per = (int)pu, t0 = (int)tu, t1 = (int)min(nu, tu + pu);
    int sum = 0;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) sum += qa_unit(a, t).nt;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31) * a.c.kv;
    // (never more runs than tiles, so that every CTA of a unit's range holds a part of it)
    const int ge = min((int)gridDim.x, total);
    if (lane == 0) s_total = s_begin = s_end = total;
    __syncwarp();
    if (cta < ge) {
      QaCut cut;
      cut.make(total, ge);
      const int lo = (incl - sum) * a.c.kv, hi = incl * a.c.kv;  // this lane's stretch
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {  // the run's start, then its end
        const int x = cut.begin(cta + side);
        if (sum == 0 || x < lo || x >= hi) continue;
        int off = lo, t = t0, nt = sum;  // (one token tile per lane: it is the one)
#pragma unroll 1
        for (; per > 1; ++t) {
          nt = qa_unit(a, t).nt;
          if (x < off + nt * a.c.kv) break;
          off += nt * a.c.kv;
        }
        const int to = cut.moved(x, x - (int)((uint32_t)(x - off) % (uint32_t)nt), nt);
        if (side) {
          s_end = to;
        } else {
          s_t = t;
          s_off = off;
          s_begin = to;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (only now: a later kernel's CTA on this SM could take the tensor memory first, and wait for this kernel
  // while this kernel waits for the tensor memory)
  grid_dep_launch();
  const uint32_t tmem = s_tmem;
  QaWalk w;
  w.begin(a, s_t, s_off, s_begin, s_end);
  grid_dep_wait();
  bool ok = true;  // a wait that gave up: no further waits, but every loop and barrier is still walked
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, kQaWaitCycles)) {
      ok = false;
      q_report(a.r.status, kErrDeviceTimeout);
    }
  };

  if (warp == 0) {
    // ---- producer: lane 0 the tiles, lanes 0..15 their block scales (keys, then values) ----
    if (lane == 0) {
      tma_prefetch_map(&kmap);
      tma_prefetch_map(&vmap);
    }
    uint32_t it = 0u, slot = 0u, par = 1u;
    const int blk = lane & 7;
    for (; w.there() && ok; w.next(a)) {
      const float* sc = lane < 8 ? a.c.ks : a.c.vs;
#pragma unroll 1
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        if constexpr (QT == 0) {  // (a handle's queries are f32)
          if (a.new_k && k == w.u.nt - 1) qa_store_new<HD>(a, w.u.b, w.j);
        }
        // the place of this lane's block, and with it of its half of the tile (pages hold 64 positions)
        const int p0 = (w.u.tile0 + k) * kQaTile, pos = p0 + kQBlock * blk;
        int row = 0, pp = 0;
        const bool seen = pos < w.u.last && qa_place(a, w.u.b, pos, row, pp);
        const int y = a.krow0 + (row * a.c.kv + w.j) * a.c.cap + pp;
        const int y0 = __shfl_sync(0xffffffffu, y, 0), y1 = __shfl_sync(0xffffffffu, y, 4);
        const uint32_t have = __ballot_sync(0xffffffffu, seen);
        wait(b_empty + 8u * slot, par);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t bar = b_full + 8u * slot;
        if (lane == 0) {
          const uint32_t dst = s_ring + slot * X::STAGE;
          mbar_expect_tx(bar, ((have & 1u) + (have >> 4 & 1u)) * 2 * 64 * HD);
          if (have & 1u) {
            tma_load_2d(dst, &kmap, bar, 0, y0);
            tma_load_2d(dst + X::KB, &vmap, bar, 0, y0);
          }
          if (have & 16u) {
            tma_load_2d(dst + 64 * HD, &kmap, bar, 0, y1);
            tma_load_2d(dst + X::KB + 64 * HD, &vmap, bar, 0, y1);
          }
        }
        if (lane < 16) {
          float* dst = ssc + slot * 16 + lane;
          if (seen) {
            qa_copy4(smem_u32(dst), sc + ((size_t)row * a.c.kv + w.j) * (a.c.cap / kQBlock) + pp / kQBlock);
            qa_copy_arrive(bar);
          } else {
            *dst = lane < 8 ? -1.f : 0.f;
            mbar_arrive(bar);
          }
        }
        if (++slot == ST) slot = 0u, par ^= 1u;
      }
    }
    // no copy may still be writing shared memory when the CTA exits
    ok = true;
#pragma unroll 1
    for (uint32_t i = it > ST ? it - ST : 0u; i < it; ++i) wait(b_full + 8u * (i % ST), (i / ST) & 1u);
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0) {
      const uint32_t id_s = idesc_e4m3_f32(kQaTile, N), id_o = idesc_bf16_f32(HD, NW, 1);
      const uint32_t q_addr = smem_u32(qbuf), p_addr = smem_u32(pbuf);
      uint32_t cnt[2] = {0u, 0u};   // tiles whose weights each parity's groups have written
      uint32_t qpar = 0u;
      uint32_t ss = 0u, spar = 0u;  // ring slot and phase of the next tile to score
      uint32_t vs = 0u;             // ring slot of the next tile to weigh
      auto scores = [&](int t) {
        wait(b_full + 8u * ss, spar);
        if (ok) {
          tc_fence_after();
          const uint32_t k_addr = s_ring + ss * X::STAGE;
#pragma unroll
          for (int ks = 0; ks < HD / 32; ++ks)
            tc_mma_e4m3(tmem + (t & 1) * N, smem_desc(k_addr + ks * 32, 16, 8 * HD, X::SWZ),
                        smem_desc(q_addr + ks * 32, 16, 8 * HD, X::SWZ), id_s, ks > 0);
          tc_commit(b_s + 8u * (t & 1));
        }
        if (++ss == ST) ss = 0u, spar ^= 1u;
      };
      for (; w.there(); w.next(a)) {
        const int n = w.k1 - w.k0;
        wait(b_q, qpar);
        qpar ^= 1u;
        tc_fence_after();
        scores(0);
        if (n > 1) scores(1);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
          const int gp = t & 1;
          wait(b_p + 8u * gp, cnt[gp]++ & 1u);
          if (ok) {
            tc_fence_after();
            const uint32_t v_addr = s_ring + vs * X::STAGE;
#pragma unroll
            for (int kk = 0; kk < kQaTile / 16; ++kk)
              tc_mma_bf16(tmem + 2 * N + gp * NW, smem_desc(v_addr + kk * 16 * HD, X::KB, 8 * HD, X::SWZ),
                          smem_desc(p_addr + gp * X::PB + kk * 256, 128, 2048, 0), id_o, (t >> 1) % kQaRun<QT> != 0 || kk > 0);
            tc_commit(b_pv + 8u * gp);
            tc_commit(b_empty + 8u * vs);
          }
          if (++vs == ST) vs = 0u;
          if (t + 2 < n) scores(t + 2);
        }
      }
    }
  } else {
    // ---- softmax groups: group = (half of the columns, parity of the tiles) ----
    const int sw = warp - 2, gp = (sw >> 2) & 1, half = sw >> 3, gw = sw & 3, group = sw >> 2;
    const int quad = warp & 3;              // the tensor-memory lanes this warp reads
    const int stid = tid - 64, gtid = stid & 127;
    const int c0 = half * CT;               // this thread's columns
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + gp * N + c0 * NP + lanes, t_o = tmem + 2 * N + gp * NW + half * X::HW + lanes,
                   t_r = tmem + 2 * (N + NW) + gp * C + c0 + lanes;
    unsigned char* pmine = pbuf + gp * X::PB + half * NCW * 2048 + (quad * 32 + lane) * 16;
    const int H = a.c.kv * a.g;
    auto all_sync = [&]() { named_sync(5, NS); };
    auto group_sync = [&]() { named_sync(1 + group, 128); };
    // four columns of the products: the accumulator's pieces, and what was added up before
    auto sum4 = [&](int c, bool more, float (&v)[4]) {
      float d[WP][4], r[4];
#pragma unroll
      for (int y = 0; y < WP; ++y) tc_ld4(t_o + y * CTP + c, d[y]);
      if (more) tc_ld4(t_r + c, r);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = d[WP - 1][i];
#pragma unroll
        for (int y = WP - 2; y >= 0; --y) v[i] += d[y][i];
        if (more) v[i] += r[i];
      }
    };
    // tokens that see nothing and share a tile with none that does: zeros
#pragma unroll 1
    for (uint32_t t = cta; t < (uint32_t)nq; t += gridDim.x) {
      const QaUnit u = qa_unit(a, (int)t);
      if (u.nt == 0 && u.ntok > 0)
#pragma unroll 1
        for (int64_t i = stid; i < (int64_t)u.ntok * H * HD; i += NS) {
          const int64_t at = (u.qrow + i / (H * HD)) * a.out_stride + i % (H * HD);
          if constexpr (QT) static_cast<uint16_t*>(a.out)[at] = 0;
          else static_cast<float*>(a.out)[at] = 0.f;
        }
    }
    uint32_t cs = 0u, cpv = 0u;             // score tiles read, value products waited for
    uint32_t sb = 0u, spar = 0u;            // ring slot and phase of the segment's first tile
    int pending = 0;
    for (; w.there(); w.next(a)) {
      const int n = w.k1 - w.k0, used = w.u.ntok * a.g;
      // ---- query pieces: warp = column ----
#pragma unroll 1
      for (int c = sw; c < C; c += NS / 32) {
        constexpr int E = HD / 32;  // elements per lane
        const int tok = c / a.g;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
        if (c < used) {
          const int64_t at = (w.u.qrow + tok) * a.q_stride + (int64_t)(w.j * a.g + c - tok * a.g) * HD + lane * E;
          if constexpr (QT == 0) {
            const float* p = static_cast<const float*>(a.q) + at;
            if constexpr (E == 4) {
              const float4 v = *reinterpret_cast<const float4*>(p);
              x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            } else {
              const float2 v = *reinterpret_cast<const float2*>(p);
              x[0] = v.x; x[1] = v.y;
            }
          } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const uint32_t v = p[e / 2];
              x[e] = bf16_lo(v);
              x[e + 1] = bf16_hi(v);
            }
          }
        }
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        const bool fine = top < 0x7f800000u;
        const float s = q_scale(fine ? __uint_as_float(top) * 1.75f : 0.f), r = q_recip(s);  // |x| r <= 256
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fine ? x[e] * r : 0.f;
#pragma unroll
        for (int y = 0; y < NP; ++y) {
          const int row = c * NP + y;
          uint32_t code = 0u;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const uint32_t p = e4m3x2(x[e], x[e + 1]);
            const float2 v = e4m3_pair(p);
            x[e] = (x[e] - v.x) * 32.f;
            x[e + 1] = (x[e + 1] - v.y) * 32.f;
            code |= p << (8 * e);
          }
          if constexpr (HD == 128)
            *reinterpret_cast<uint32_t*>(qbuf + row * 128 + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4) = code;
          else
            *reinterpret_cast<uint16_t*>(qbuf + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + (lane & 7) * 2) = (uint16_t)code;
        }
        if (lane == 0) {
          // a query that is not finite makes its scores NaN
          qsc[c] = c < used ? (fine ? s * (a.scale * 1.4426950408889634f) : __uint_as_float(0x7fc00000u)) : 0.f;
          cend[c] = c < used ? w.u.end0 + tok : 0;
        }
      }
      fence_proxy_async_smem();
      all_sync();  // (also: the segment before is written, its shared memory is free)
      if (stid == 0) mbar_arrive(b_q);
      float* ref = gref + gp * C + c0;      // references of the group's columns, alike for all its threads
      if (gtid < CT) ref[gtid] = c0 + gtid < used ? kQaNone : INFINITY;  // (no token: weights 2^-inf)
      group_sync();
      const float* qsg = qsc + c0;
      const int* ceg = cend + c0;
      uint32_t slot = sb + gp, fpar = spar;  // ring slot and phase of this group's next tile
      if (slot >= ST) slot -= ST, fpar ^= 1u;
      float l[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) l[c] = 0.f;
      float vref = 0.f, vinv = 0.f;         // the largest value scale seen, and its reciprocal
      bool pend = false;                    // a product over the values not waited for yet
#pragma unroll 1
      for (int t = gp; t < n; t += 2) {
        const int p0 = (w.u.tile0 + w.k0 + t) * kQaTile, pos = p0 + quad * 32 + lane;
        wait(b_full + 8u * slot, fpar);
        const float ks = ssc[slot * 16 + quad * 2 + (lane >> 4)], vs = ssc[slot * 16 + 8 + quad * 2 + (lane >> 4)];
        const bool good = !(ks < 0.f) && pos < w.u.last && pos >= w.u.start;
        const bool whole = __all_sync(0xffffffffu, good) && p0 + kQaTile <= w.u.end0;
        const int mypos = good ? pos : 0x7fffffff;
        const int wr = quad * 32 + (HV == 1 ? lane : half * 16 + (lane & 15));
        const bool wlive = HV == 1 ? good : __ballot_sync(0xffffffffu, good) >> (wr & 31) & 1u;
        wait(b_s + 8u * gp, cs++ & 1u);
        __syncwarp();
        tc_fence_after();
        float s[CT], above = -INFINITY;  // scores, and the most by which one is above its reference
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          float d[16];
          tc_ld16(t_s + ch * 16, d);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < CPC; i += 4) {
            const float4 qv = *reinterpret_cast<const float4*>(qsg + ch * CPC + i);
            const float4 rv = *reinterpret_cast<const float4*>(ref + ch * CPC + i);
            const float q4[4] = {qv.x, qv.y, qv.z, qv.w}, r4[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float v = d[(i + y) * NP + NP - 1];
#pragma unroll
              for (int x = NP - 2; x >= 0; --x) v = fmaf(v, 0.03125f, d[(i + y) * NP + x]);
              v *= ks * q4[y];
              s[ch * CPC + i + y] = v;
              above = fmaxf(above, v - r4[y]);
            }
          }
        }
        float vr = good ? vs * vinv : 0.f;
        if (!whole) {
          // columns see positions below their cend
          above = -INFINITY;
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            if (mypos >= ceg[c]) s[c] = -INFINITY;
            above = fmaxf(above, s[c] - ref[c]);
          }
        }
        const bool low = !(above > kQaMost) && !(good && vs > vref);
        if (!named_sync_and(1 + group, 128, low)) {
          // references move (rare): the group's maxima, then each column's new reference and what the
          // sums relative to the old one are worth under it
          float* wm = wmax + gp * 4 * C + c0;
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const float m = qa_warp_max(s[c]);
            if (lane == 0) wm[gw * C + c] = m;
          }
          const float mv = qa_warp_max(good ? vs : 0.f);
          if (lane == 0) wvs[group * 4 + gw] = mv;
          group_sync();
          if (gtid < CT) {
            const float old = ref[gtid];
            const float top = fmaxf(old, fmaxf(fmaxf(wm[gtid], wm[C + gtid]), fmaxf(wm[2 * C + gtid], wm[3 * C + gtid])));
            ref[gtid] = top;
            wm[gtid] = top == old ? 1.f : qa_exp2(old - top);
          }
          const float* wv = wvs + group * 4;
          const float v1 = fmaxf(fmaxf(wv[0], wv[1]), fmaxf(wv[2], wv[3]));
          float vcorr = 1.f;
          if (v1 > vref) {
            vcorr = vref * q_recip(v1);
            vref = v1;
            vinv = q_recip(v1);
            vr = good ? vs * vinv : 0.f;
          }
          group_sync();
#pragma unroll
          for (int c = 0; c < CT; ++c) l[c] *= wm[c];
          if (t > gp) {
            // the accumulators, once the product before is in them
            if (pend) {
              wait(b_pv + 8u * gp, cpv++ & 1u);
              pend = false;
            }
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < (t >= 2 * kQaRun<QT> ? WP + 1 : WP) * (CT / 4); ++k) {  // (and the sums, once there are some)
              const int y = k / (CT / 4), c = k % (CT / 4) * 4;
              const uint32_t at = y < WP ? t_o + y * CTP + c : t_r + c;
              float d[4];
              tc_ld4(at, d);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] *= wm[c + i] * vcorr;
              tc_st4(at, d);
            }
            tc_wait_st();
          }
        }
        if (__any_sync(0xffffffffu, vr != vr)) {
          // a block of values that are NaN: so are the weights of the columns that see it, and no others
          if (vr != vr) {
            vr = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c)
              if (s[c] > -INFINITY) s[c] = __uint_as_float(0x7fc00000u);
          }
        }
        qa_widen_row<HD, HV>(base + slot * X::STAGE, wr, lane >> 4 & (HV - 1), wlive);
        if (pend) wait(b_pv + 8u * gp, cpv++ & 1u);  // the weights' buffer is free again
        if (t >= 2 * kQaRun<QT> && (t >> 1) % kQaRun<QT> == 0) {
          // the accumulator starts anew with this tile: what it holds goes to the sums
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < CT; c += 4) {
            float v[4];
            sum4(c, t >= 4 * kQaRun<QT>, v);
            tc_st4(t_r + c, v);
          }
          tc_wait_st();
        }
#pragma unroll
        for (int c8 = 0; c8 < CT; c8 += 8) {
          uint32_t o[WP][4];  // the pieces of 8 columns, in pairs
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c8 + 2 * i;
            if (c >= CT) {
#pragma unroll
              for (int y = 0; y < WP; ++y) o[y][i] = 0u;
              continue;
            }
            const float2 rv = *reinterpret_cast<const float2*>(ref + c);
            // a weight (0 where the column does not see the position), its sum, and with the value's
            // scale on it
            float x0 = qa_exp2(s[c] - rv.x), x1 = qa_exp2(s[c + 1] - rv.y);
            l[c] += x0;
            l[c + 1] += x1;
            x0 *= vr;
            x1 *= vr;
#pragma unroll
            for (int y = 0; y < WP; ++y) {  // each piece the rounding of what the ones before left over
              o[y][i] = bf16x2(x0, x1);
              x0 -= bf16_lo(o[y][i]);
              x1 -= bf16_hi(o[y][i]);
            }
          }
          if constexpr (CT == 4) {
            static_assert(CT != 4 || WP == 3, "pieces of four columns");
            *reinterpret_cast<uint4*>(pmine) = make_uint4(o[0][0], o[0][1], o[1][0], o[1][1]);
            *reinterpret_cast<uint4*>(pmine + 2048) = make_uint4(o[WP - 1][0], o[WP - 1][1], 0u, 0u);
          } else {
#pragma unroll
            for (int y = 0; y < WP; ++y)
              *reinterpret_cast<uint4*>(pmine + (y * (CTP / 8) + c8 / 8) * 2048) = make_uint4(o[y][0], o[y][1], o[y][2], o[y][3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(b_p + 8u * gp);
        pend = true;
        slot += 2;
        if (slot >= ST) slot -= ST, fpar ^= 1u;
      }
      if (pend) wait(b_pv + 8u * gp, cpv++ & 1u);
      __syncwarp();
      tc_fence_after();
      spar ^= ((sb + n) / ST) & 1u;
      sb = (sb + n) % ST;

      // ---- the segment's end: the parities' sums meet, parity 0 writes ----
      {
        // the lanes' sums of every column at once: each exchange halves the columns a lane holds
        constexpr int CP = CT <= 4 ? 4 : CT <= 8 ? 8 : 16;  // (a power of two)
        float x[CP];
#pragma unroll
        for (int c = 0; c < CP; ++c) x[c] = c < CT ? l[c < CT ? c : 0] : 0.f;
        int col = 0;
#pragma unroll
        for (int o = 16, m = CP; o > 0; o >>= 1) {
          if (m > 1) {
            m >>= 1;
            const bool up = lane & o;
            col += up ? m : 0;
#pragma unroll
            for (int c = 0; c < m; ++c) {
              const float give = up ? x[c] : x[c + m], keep = up ? x[c + m] : x[c];
              x[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
          }
        }
        if (col < CT) wmax[(gp * 4 + gw) * C + c0 + col] = x[0];  // (lanes of one column write the same sum)
        if (gtid == 0) gvs[group] = vref;
      }
      all_sync();  // (every product is done: the weights' buffers are free)
      const bool both = n > 1, alone = w.k0 == 0 && w.k1 == w.u.nt;  // alone: this CTA holds the whole unit
      // parts of units cut across CTAs: [CTA][the unit's first part?]{[C][HD] sums, [C] (reference, weight)}
      float* parts = reinterpret_cast<float*>(a.ws + kQattnTickets);
      float* mine = parts + ((size_t)cta * 2 + (w.k0 == 0 ? 1 : 0)) * C * (HD + 2);
      if (stid < used) {
        // column stid: the parities' common reference and what each one's sums are worth under it
        const int c = stid, hv = c / CT;
        const float* x = wmax + c;
        const float r0 = gref[c], r1 = both ? gref[C + c] : kQaNone, M = fmaxf(r0, r1);
        const float f0 = qa_exp2(r0 - M), f1 = both ? qa_exp2(r1 - M) : 0.f;
        float L = (x[0] + x[C] + x[2 * C] + x[3 * C]) * f0;
        if (both) L = fmaf(x[4 * C] + x[5 * C] + x[6 * C] + x[7 * C], f1, L);
        const float r = alone ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
        ffac[c] = f0 * gvs[2 * hv] * r;
        ffac[C + c] = f1 * (both ? gvs[2 * hv + 1] : 0.f) * r;
        const int tok = c / a.g;
        coff[c] = tok * a.out_stride + (c - tok * a.g) * HD;
        if (!alone) *reinterpret_cast<float2*>(mine + C * HD + 2 * c) = make_float2(M, L);
      }
      all_sync();
      const int d_row = HD == 128 ? quad * 32 + lane : quad * 16 + (lane & 15);  // the dimension of this lane
      const bool d_on = HD == 128 || lane < 16;
      float* other = reinterpret_cast<float*>(pbuf);  // [C][HD]: parity 1's sums
      const int64_t obase = w.u.qrow * a.out_stride + (int64_t)w.j * a.g * HD;
#pragma unroll 1
      for (int pass = 1; pass >= 0; --pass) {
        if (gp == pass && (both || pass == 0)) {
#pragma unroll 1
          for (int c4 = 0; c4 < CT && c0 + c4 < used; c4 += 4) {
            float v4[4];
            sum4(c4, n > 2 * kQaRun<QT> + gp, v4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = c0 + c4 + i;
              float v = v4[i];
              v *= ffac[pass * C + c];
              if (d_on && c < used) {
                if (pass == 0 && both) v += other[c * HD + d_row];
                if (pass == 0 && alone) {
                  const int64_t at = obase + coff[c] + d_row;
                  if constexpr (QT) static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v);
                  else static_cast<float*>(a.out)[at] = v;
                } else {
                  (pass ? other : mine)[c * HD + d_row] = v;
                }
              }
            }
          }
        }
        if (pass == 1 && both) all_sync();
      }
      if (!alone) {
        if (stid == 0) {
          QaCut cut;
          cut.make(s_total, min((int)gridDim.x, s_total));
          const int first = cut.first(w.unit0());
          s_pend[pending] = Pending{w.u.qrow, w.j, used, first, cut.last(w.unit0(), w.u.nt) - first + 1, 0};
        }
        ++pending;
      }
    }
    // ---- units of several CTAs: the last of them to get here adds the parts in CTA order ----
    if (pending > 0) {
      __threadfence();
      all_sync();
      if (stid < pending) {
        Pending& u = s_pend[stid];
        u.last = atomicInc(reinterpret_cast<uint32_t*>(a.ws) + u.first, (uint32_t)(u.np - 1)) == (uint32_t)(u.np - 1);
      }
      all_sync();
      __threadfence();
    }
#pragma unroll 1
    for (int pi = 0; pi < pending; ++pi) {
      const Pending u = s_pend[pi];
      if (!u.last) continue;
      all_sync();  // (the unit before is written)
      const int np = u.np, first = u.first, used = u.used;
      const float* parts = reinterpret_cast<const float*>(a.ws + kQattnTickets);
      auto part = [&](int i) { return parts + ((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * C * (HD + 2); };
      auto stat = [&](int i, int c) { return __ldcg(reinterpret_cast<const float2*>(part(i) + C * HD + 2 * c)); };
      // (the ring is idle: factors [used][np], then the slices' sums; short loops, see above)
      float* fac = reinterpret_cast<float*>(base);
#pragma unroll 1
      for (int c = sw; c < used; c += NS / 32) {  // warp = column, lanes = parts
        float M = kQaNone, L = 0.f;
#pragma unroll 1
        for (int i = lane; i < np; i += 32) M = fmaxf(M, stat(i, c).x);
        M = qa_warp_max(M);
#pragma unroll 1
        for (int i = lane; i < np; i += 32) {
          const float2 x = stat(i, c);
          const float f = qa_exp2(x.x - M);
          fac[c * np + i] = f;
          L = fmaf(x.y, f, L);
        }
        L = warp_sum(L);
        const int tok = c / a.g;
        if (lane == 0) {
          wmax[c] = L;
          coff[c] = tok * a.out_stride + (c - tok * a.g) * HD;
        }
      }
      all_sync();
      // thread = four dimensions of a column, and every SL-th part where there are fewer of these than threads
      constexpr int X4 = C * HD / 4, SL = NS > X4 ? NS / X4 : 1, U = 8;
      static_assert((size_t)C * kQattnTickets <= (size_t)ST * X::STAGE, "factors of as many parts as there can be CTAs");
      const int64_t obase = u.qrow * a.out_stride + (int64_t)u.j * a.g * HD;
      float4* sums = reinterpret_cast<float4*>(pbuf);  // [SL][X4]
#pragma unroll 1
      for (int x = stid % X4; x < used * (HD / 4); x += NS) {
        const int c = x / (HD / 4), sl = stid / X4 % SL;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i = sl; i < np; i += SL * U) {
          float4 v[U];
#pragma unroll
          for (int y = 0; y < U; ++y) v[y] = __ldcg(reinterpret_cast<const float4*>(part(min(i + y * SL, np - 1))) + x);
#pragma unroll
          for (int y = 0; y < U; ++y) {
            const float f = i + y * SL < np ? fac[c * np + i + y * SL] : 0.f;
            o.x = fmaf(f, v[y].x, o.x);
            o.y = fmaf(f, v[y].y, o.y);
            o.z = fmaf(f, v[y].z, o.z);
            o.w = fmaf(f, v[y].w, o.w);
          }
        }
        const float r = wmax[c] == 0.f ? 0.f : 1.f / wmax[c];
        o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
        if constexpr (SL > 1) {
          sums[sl * X4 + x] = o;  // (one turn of this loop: X4 < NS)
        } else {
          qa_put4<QT>(a.out, obase + coff[c] + x % (HD / 4) * 4, o);
        }
      }
      if constexpr (SL > 1) {
        all_sync();
        if (stid < used * (HD / 4)) {
          float4 o = sums[stid];
#pragma unroll
          for (int i = 1; i < SL; ++i) {
            const float4 v = sums[i * X4 + stid];
            o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
          }
          qa_put4<QT>(a.out, obase + coff[stid / (HD / 4)] + stid % (HD / 4) * 4, o);
        }
      }
    }
  }
  // ---- everyone leaves together; the products are done, the tensor memory goes back ----
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, X::TMEM);
}

// one instantiation per translation unit (they take half a minute each to compile)
template <int HD, int NP, int NC, int QT>
cudaError_t launch_qattn_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const QAttnArgs& a, int grid,
                            cudaStream_t s, bool pdl) {
  constexpr size_t smem = QaShape<HD, NP, NC>::SMEM;
  auto fn = qattn_tc_kernel<HD, NP, NC, QT>;
  // (the limit belongs to the device's context: set on every call, a fraction of a microsecond)
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(QaShape<HD, NP, NC>::NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, kmap, vmap, a);
}

#define LLM_QATTN_TC(NAME) \
  cudaError_t NAME(const CUtensorMap& kmap, const CUtensorMap& vmap, const QAttnArgs& a, int nc, int grid, \
                   cudaStream_t s, bool pdl)
LLM_QATTN_TC(qattn_tc64_f32);
LLM_QATTN_TC(qattn_tc64_f32_wide);
LLM_QATTN_TC(qattn_tc64_bf16);
LLM_QATTN_TC(qattn_tc128_f32);
LLM_QATTN_TC(qattn_tc128_f32_wide);
LLM_QATTN_TC(qattn_tc128_bf16);

}  // namespace llm
