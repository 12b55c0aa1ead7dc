// Attention over positions that many columns share, in an 8-bit cache, on the 5th-generation tensor cores (head sizes
// 64 and 128): the kernel template (an instantiation each in qshare<head size>_<type>.cu).
//
// The (token, query head) pairs of a group's rows that read a key/value head at the same places are columns of one
// product, up to 128 of them.  Queries are on the M side, positions on the N side, so that a thread has a column's scores
// to itself:
//   S [128 columns][TN positions] = Q K^T     A = query pieces (shared memory), B = keys' codes as they lie
//   softmax                                   thread = column: weights against a reference, their sum
//   O [128][HD]                  += P V       A = weight pieces (tensor memory), B = widened values
// The reference is a power of two that follows the column's largest score lazily: it moves when a weight would
// exceed 2^24, which after a run's first tile is rare, and what was added up so far is then rescaled in tensor memory
// (exactly).  So weights go from 2^24 down to 2^-126 of it with all their digits, no maximum is waited for, and a tile's
// products go on top of those before.  The blocks' value scales ride on the weights, relative to a power of two that moves in the
// same way.  O is read after RUN of a group's tiles (kQaRun says what longer runs lose) into sums in local memory.
//
// Pieces.  A query is scaled by a power of two so that its largest element is between 128 and 256, and enters as e4m3 pieces, each
// the rounding of what the ones before left over (made once for the call, qshare.cu).  A piece takes four bits and the sign of what
// is left a fifth, so two leave 2^-9 of an element's binade, or 2^-10, half the least step of e4m3.  bf16: two, summed in one accumulator,
// which are an element's eight bits down to 2^-9 of the largest and leave 2^-17 of the largest of smaller ones.  f32: four, the last two
// 2^10 times larger in an accumulator of their own, which leave 2^-19 of an element or 2^-20, 2^-27 of the largest.  (The kernel for few
// columns has an accumulator a piece, each 2^5 times larger than the one before: 2^-32 of the largest.)  The softmax weights are
// bf16 pieces, two (bf16 queries: 2^-17 of a weight, half of 2^-9 being the output's own rounding) or three (f32: 2^-26), over values
// widened to bf16, exactly; bf16 has f32's exponents, so that a weight keeps its digits however small it is.
//
// One CTA per SM, 16 warps: warp 0 loads the tiles and queries by TMA; warps 1 and 3 issue the products; warp 2 walks the CTA's share of
// the work (segments: runs of tiles of one unit) ahead of the others and tells them each segment; four warps widen values; two
// groups of four softmax warps take the tiles in turn, each with scores, sums and references of its own in tensor memory, so that one
// group's products run while the other weighs.  The units' tiles are shared out in equal runs; a unit's sums over a CTA's
// run go to global memory, a part for each group, and another kernel joins each column's parts in CTA order, so the result does
// not depend on timing.
//
// What bounds it (131072 positions, 64 rows of 32 heads of 128 behind them, bf16: 230 us of a call's 269, for 85 of which the tensor pipe
// is busy): a tile of 128 x 128 takes about 4100 clocks, its softmax 4800 in either group, of which the 32-score steps
// take 1000 each (293 instructions for 32 scores; the schedulers issue 47% of the time), then 1400 for its product and 750 for
// its next scores.  f32 queries: 3400 clocks a tile of 64 positions.  Slower: the value product's columns in halves, more registers for
// the softmax warps (setmaxnreg), tiles of 64 with two score buffers a group (289 us).  The product's positions in halves, the
// first under way while the second is weighed: 266 us, for two more barriers a group.
#pragma once
#include <type_traits>

#include "qattn_tc.cuh"

namespace llm {

constexpr int kShRows = 128;         // columns of a unit: the M side
constexpr int kShSegs = 8;           // segments told ahead
constexpr int kShWarps = 16;         // loads, scores, walk, values' products; two softmax groups of four; four that widen
constexpr int kShThreads = 32 * kShWarps;
constexpr int kShWiden = 128;        // threads that widen
// A wait's limit, about 4 s: all warps but that of the loads wait for data from when the CTA starts, and with that for the rest of the
// kernel before, which may be a long one.  (A wait for that kernel alone in each warp took 3 to 9 us of the 269 above more.)
constexpr uint64_t kShWaitCycles = 8 * kQaWaitCycles;
constexpr float kShMost = 24.0f;     // log2 of the largest weight that moves no reference

template <int HD, int QT>
struct ShShape {
  static constexpr int NP = QT ? 2 : 4;              // query pieces
  static constexpr int WP = QT ? 2 : 3;              // weight pieces
  static constexpr int TN = QT ? 128 : 64;           // positions per tile
  static constexpr int NB = TN / kQBlock;            // their blocks
  static constexpr int KB = TN * HD;                 // bytes of a tile's keys (or values)
  static constexpr int QB = NP * kShRows * HD;       // query pieces
  static constexpr int VB = 2 * TN * HD;             // widened values of a tile
  static constexpr int KS = HD == 64 || !QT ? 6 : 4, VS = HD == 64 || !QT ? 6 : 3;  // ring stages
  static constexpr int RUN = (QT ? 4096 : 512) / TN;            // a group's tiles whose products are summed in tensor memory
  static constexpr size_t MISC = 14336;
  static constexpr size_t SMEM = 1024 + (size_t)(KS + VS) * KB + QB + 2 * VB + MISC;
  static constexpr uint32_t SWZ = HD == 128 ? 2 : 4;
  // Tensor memory: a group's scores, in 128 columns (f32: coarse and fine pieces apart) that its weights reuse; behind both
  // groups' their O
  static constexpr uint32_t BUF = 128, O = 2 * BUF;
  static_assert(SMEM <= kQaSmem && O + 2 * HD <= 512, "memory");
  static_assert((KS + VS) * KB >= kShUnits * 4, "the walk's counts");
};

// what the walk tells the others of a segment
struct ShSeg {
  int n;             // tiles; 0: no more
  int p0;            // position of the first
  int start, stop;   // positions that count
  int place;         // the row whose places hold them
  int gt, used;      // first token, columns
  int j;             // key/value head
  int part;          // as sh_put takes it: 0: the unit's first run, 2: a run that goes on
  int cta0, ctas;    // CTAs that hold the unit: the first, and how many come after it
};

template <int HD, int QT>
__global__ void __launch_bounds__(kShThreads, 1)
    qshare_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap,
                  const QAttnArgs a) {
  using X = ShShape<HD, QT>;
  constexpr int NP = X::NP, WP = X::WP, TN = X::TN, NB = X::NB, KS = X::KS, VS = X::VS;
  extern __shared__ unsigned char qraw[];
  const uint32_t s_raw = smem_u32(qraw);
  unsigned char* base = qraw + (((s_raw + 1023u) & ~1023u) - s_raw);
  unsigned char* qbuf = base;                                // [NP][128][HD]
  unsigned char* wide = qbuf + X::QB;                        // [2][VB]
  unsigned char* kring = wide + 2 * X::VB;                   // [KS][KB]
  unsigned char* vring = kring + (size_t)KS * X::KB;         // [VS][KB]
  float* ssc = reinterpret_cast<float*>(vring + (size_t)VS * X::KB);  // [VS][16] block scales: keys (-1: unseen), values
  float* qsc = ssc + 16 * VS;                                // [kShSegs][128] a column's scale, in units of log2
  int* lim = reinterpret_cast<int*>(qsc + kShSegs * kShRows);  // [kShSegs][128] positions that it sees end here
  float* wsc = reinterpret_cast<float*>(lim + kShSegs * kShRows);  // [8][16] a softmax warp's block scales
  ShSeg* segs = reinterpret_cast<ShSeg*>(wsc + 128);         // [kShSegs]
  const uint32_t bars = (smem_u32(segs + kShSegs) + 7u) & ~7u;
  const uint32_t b_kf = bars, b_ke = b_kf + 8 * KS, b_vf = b_ke + 8 * KS, b_ve = b_vf + 8 * VS, b_wf = b_ve + 8 * VS,
                 b_we = b_wf + 16, b_sf = b_we + 16, b_pf = b_sf + 16, b_of = b_pf + 16, b_oe = b_of + 16, b_qe = b_oe + 16,
                 b_qf = b_qe + 8, b_gf = b_qf + 8 * kShSegs, b_ge = b_gf + 8 * kShSegs,
                 b_end = b_ge + 8 * kShSegs, b_end2 = b_end + 8;
  static_assert(64 * VS + 8 * 128 * kShSegs + 512 + sizeof(ShSeg) * kShSegs + 16 * (KS + VS) + 144 + 24 * kShSegs + 8 <= X::MISC,
                "shared memory");
  __shared__ uint32_t s_tmem;
  __shared__ int s_warp[kShWarps], s_total, s_slot, s_at;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 32) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(b_kf + 8u * i, 1);
      mbar_init(b_ke + 8u * i, 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(b_vf + 8u * i, 1 + 2 * NB);
      mbar_init(b_ve + 8u * i, 8);          // the warps that widen, and those of the group that reads the scales
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_wf + 8u * i, kShWiden);
      mbar_init(b_we + 8u * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_sf + 8u * i, 1);
      mbar_init(b_pf + 8u * i, 128);
      mbar_init(b_of + 8u * i, 1);
      mbar_init(b_oe + 8u * i, 128);
    }
    mbar_init(b_end, 1);
    mbar_init(b_end2, 1);
    mbar_init(b_qe, 1);
    for (int i = 0; i < kShSegs; ++i) {
      mbar_init(b_qf + 8u * i, 33);          // the loads, and the lanes that copy the scales
      mbar_init(b_gf + 8u * i, 32);
      mbar_init(b_ge + 8u * i, 3 + 12);
    }
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  // ---- the units' tiles, counted by all threads; the unit that this CTA's run starts in ----
  const bool sharing = sh_fine(a);
  const int slots = a.r.B * a.sh.cpr;  // (prefix units alone: the rows' own positions are the other kernel's)
  int* before = reinterpret_cast<int*>(kring);  // [slots] (the rings are idle yet)
  int G = gridDim.x;
  {
    const int per = (slots + kShThreads - 1) / kShThreads, s0 = min(slots, tid * per), s1 = min(slots, s0 + per);
    int sum = 0;
    for (int s = s0; s < s1; ++s) {
      before[s] = sum;
      sum += sh_unit<TN, false>(a, s, sharing).nt;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int lead = incl - sum, all = 0;
    for (int w = 0; w < kShWarps; ++w) {
      if (w < warp) lead += s_warp[w];
      all += s_warp[w];
    }
    for (int s = s0; s < s1; ++s) before[s] += lead;
    if (tid == 0) s_total = all * a.c.kv;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (only now: a later kernel's CTA on this SM could take the tensor memory first)
  grid_dep_launch();
  const uint32_t tmem = s_tmem;
  const int total = s_total;
  G = min(G, total);
  ShCut cut;
  cut.make(total, max(G, 1));
  const int run0 = cta < G ? cut.begin(cta) : 0, run1 = cta < G ? cut.begin(cta + 1) : 0;
  if (tid == 0 && run0 < run1) {
    // the last unit that starts at run0 or before
    const int goal = run0 / a.c.kv;
    int lo = 0, hi = slots - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= goal) lo = mid;
      else hi = mid - 1;
    }
    s_slot = lo;
    s_at = before[lo] * a.c.kv;
  }
  fence_proxy_async_smem();  // the counts, written and read here, come before the copies that fill the rings
  __syncthreads();

  bool ok = true;  // a wait that gave up: no further waits, but every loop is still walked to its end
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, kShWaitCycles)) {
      ok = false;
      q_report(a.r.status, kErrDeviceTimeout);
    }
  };
  // the tiles of the next segment, alike in the warp; 0: none
  uint32_t gslot = 0u, gpar = 0u;
  auto next_seg = [&]() {
    wait(b_gf + 8u * gslot, gpar);
    ok = __all_sync(0xffffffffu, ok);
    return ok ? segs[gslot].n : 0;
  };
  auto seg_done = [&]() {  // this warp has read what it needs of the segment
    __syncwarp();
    if (lane == 0) mbar_arrive(b_ge + 8u * gslot);
    if (++gslot == kShSegs) gslot = 0u, gpar ^= 1u;
  };

  if (warp == 2) {
    // ---- the walk: what each segment is, and where its columns' positions end ----
    uint32_t gs = 0u, gp = 1u;
    int s = s_slot, at = s_at, run = run0;
    QaUnit u = {};
    int e[kShRows / 32], last = 0;  // this lane's columns
    auto ends = [&]() {
      const int used = u.ntok * a.g;
      last = 0;
#pragma unroll
      for (int i = 0; i < kShRows / 32; ++i) {
        const int c = lane + 32 * i;
        e[i] = 0;
        if (c < used) {
          const int gt = (int)u.qrow + c / a.g, b = gt / a.r.S;
          e[i] = min(sh_end(a, b, gt - b * a.r.S), u.last);
        }
        last = max(last, e[i]);
      }
      last = __reduce_max_sync(0xffffffffu, last);
    };
    if (run < run1) {
      u = sh_unit<TN, false>(a, s, sharing);
      ends();
    }
    while (run < run1 && ok) {
      if (u.nt == 0 || run >= at + u.nt * a.c.kv) {  // (the run holds a tile, so a unit with it comes)
        at += u.nt * a.c.kv;
        s = sh_next(a, s, sharing);
        if (s >= slots) break;  // (only if lengths or groups change while the call runs)
        u = sh_unit<TN, false>(a, s, sharing);
        if (u.nt > 0) ends();
        continue;
      }
      const int j = (run - at) / u.nt, k0 = run - at - j * u.nt, n = min(u.nt - k0, run1 - run);
      wait(b_ge + 8u * gs, gp);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kShRows / 32; ++i) lim[gs * kShRows + lane + 32 * i] = e[i];
      if (lane == 0) {
        const int first = at + j * u.nt, c0 = cut.owner(first);
        segs[gs] = ShSeg{n, (u.tile0 + k0) * TN, u.start, last, u.b, (int)u.qrow, u.ntok * a.g, j, k0 > 0 ? 2 : 0, c0, cut.owner(first + u.nt - 1) - c0};
      }
      __syncwarp();
      mbar_arrive(b_gf + 8u * gs);
      if (++gs == kShSegs) gs = 0u, gp ^= 1u;
      run += n;
    }
    // the end
    wait(b_ge + 8u * gs, gp);
    if (lane == 0) segs[gs].n = 0;
    __syncwarp();
    mbar_arrive(b_gf + 8u * gs);
  } else if (warp == 0) {
    // ---- the loads ----
    grid_dep_wait();  // (the queries' pieces are the work of a kernel before)
    fence_proxy_async_global();
    if (lane == 0) {
      tma_prefetch_map(&kmap);
      tma_prefetch_map(&vmap);
      tma_prefetch_map(&qmap);
    }
    uint32_t ks = 0u, kpar = 1u, vs = 0u, vpar = 1u, nk = 0u, qpar = 1u;
    const float* sc = lane < NB ? a.c.ks : a.c.vs;
    const int blk = lane & (NB - 1);
    // places of 32 pages, one per lane: of row `held` from page `page0` on (of a unit's heads all the same)
    int held = -1, held_start = 0, held_stop = 0, page0 = 0, prow = -1, ppos = 0;
    while (const int n = next_seg()) {
      const int p0 = segs[gslot].p0, start = segs[gslot].start, stop = segs[gslot].stop, place = segs[gslot].place, j = segs[gslot].j;
      {
        // the queries, once the products of the segment before have read theirs (the rows behind the unit's columns are
        // others' or what was there: finite, and of no use)
        const int col = (j * a.r.B * a.r.S + segs[gslot].gt) * a.g, used = segs[gslot].used, cols = a.r.B * a.r.S * a.c.kv * a.g;
        wait(b_qe, qpar);
        qpar ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t bar = b_qf + 8u * gslot;
        if (lane == 0) {
          const int boxes = used > 64 ? 2 : 1;
          mbar_expect_tx(bar, NP * boxes * 64 * HD);
          for (int p = 0; p < NP; ++p)
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(smem_u32(qbuf) + (p * kShRows + 64 * i) * HD, &qmap, bar, 0, p * cols + col + 64 * i);
        }
        for (int c = lane; c < used; c += 32) qa_copy4(smem_u32(qsc + gslot * kShRows + c), a.sh.qs + col + c);
        qa_copy_arrive(bar);
      }
      seg_done();
#pragma unroll 1
      for (int k = 0; k < n; ++k, ++nk) {
        const int t0 = p0 + k * TN, pg = t0 / kPage;
        if (place != held || start != held_start || stop != held_stop || pg < page0 || pg + (TN - 1) / kPage >= page0 + 32) {
          held = place;
          held_start = start;
          held_stop = stop;
          page0 = pg;
          prow = -1;
          const int pos = (pg + lane) * kPage;
          if (pos < stop && pos + kPage > start && !q_place(a.r, a.c, place, pos, prow, ppos)) prow = -1;
        }
        const int r0 = __shfl_sync(0xffffffffu, prow, pg - page0), q0 = __shfl_sync(0xffffffffu, ppos, pg - page0);
        int r1 = -1, q1 = 0;
        if constexpr (TN > kPage) {
          r1 = __shfl_sync(0xffffffffu, prow, pg + 1 - page0);
          q1 = __shfl_sync(0xffffffffu, ppos, pg + 1 - page0);
        }
        const int pos = t0 + kQBlock * blk, row = blk < 4 ? r0 : r1, pp = (blk < 4 ? q0 : q1) + (blk & 3) * kQBlock;
        const bool seen = lane < 2 * NB && pos < stop && pos + kQBlock > start && row >= 0;
        // (a half tile is loaded if one of its blocks is seen)
        const uint32_t have = __ballot_sync(0xffffffffu, seen);
        const bool h0 = have & 15u, h1 = NB == 8 && (have & 0xf0u);
        wait(b_ke + 8u * ks, kpar);
        wait(b_ve + 8u * vs, vpar);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t kb = b_kf + 8u * ks, vb = b_vf + 8u * vs, bytes = ((uint32_t)h0 + (uint32_t)h1) * 64 * HD;
          const uint32_t kd = smem_u32(kring) + ks * X::KB, vd = smem_u32(vring) + vs * X::KB;
          const int y0 = (r0 * a.c.kv + j) * a.c.cap + q0, y1 = (r1 * a.c.kv + j) * a.c.cap + q1;
          mbar_expect_tx(kb, bytes);
          mbar_expect_tx(vb, bytes);
          if (h0) {
            tma_load_2d(kd, &kmap, kb, 0, y0);
            tma_load_2d(vd, &vmap, vb, 0, y0);
          }
          if (h1) {
            tma_load_2d(kd + 64 * HD, &kmap, kb, 0, y1);
            tma_load_2d(vd + 64 * HD, &vmap, vb, 0, y1);
          }
        }
        if (lane < 2 * NB) {
          float* dst = ssc + vs * 16 + lane;
          if (seen) {
            qa_copy4(smem_u32(dst), sc + ((size_t)row * a.c.kv + j) * (a.c.cap / kQBlock) + pp / kQBlock);
            qa_copy_arrive(b_vf + 8u * vs);
          } else {
            *dst = lane < NB ? -1.f : 0.f;
            mbar_arrive(b_vf + 8u * vs);
          }
        }
        if (++ks == KS) ks = 0u, kpar ^= 1u;
        if (++vs == VS) vs = 0u, vpar ^= 1u;
      }
      if (!ok) break;
    }
    // no copy may still be writing shared memory when the CTA exits (the queries' have been waited for with their use)
    ok = true;
#pragma unroll 1
    for (uint32_t i = nk > KS ? nk - KS : 0u; i < nk; ++i) wait(b_kf + 8u * (i % KS), (i / KS) & 1u);
#pragma unroll 1
    for (uint32_t i = nk > VS ? nk - VS : 0u; i < nk; ++i) wait(b_vf + 8u * (i % VS), (i / VS) & 1u);
  } else if (warp == 1) {
    // ---- the products of queries and keys: a group's next as soon as its columns are free ----
    const uint32_t id_s = idesc_e4m3_f32(kShRows, TN);
    const uint32_t q_addr = smem_u32(qbuf), k_ring = smem_u32(kring);
    uint32_t ks = 0u, kpar = 0u, it = 0u;
    const uint32_t one = lane == 0;  // (the lane that issues: the addresses stay uniform over the warp)
    while (const int n = __reduce_max_sync(0xffffffffu, next_seg())) {
      wait(b_qf + 8u * gslot, gpar);
      seg_done();
#pragma unroll 1
      for (int k = 0; k < n; ++k, ++it) {
        const uint32_t gp = it & 1u;
        if (it >= 2u) wait(b_of + 8u * gp, (it >> 1 & 1u) ^ 1u);  // (the product has read the weights there)
        wait(b_kf + 8u * ks, kpar);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t k_addr = k_ring + ks * X::KB;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int i = 0; i < HD / 32; ++i)
            tc_mma_e4m3_if(tmem + gp * X::BUF + (p >= 2 ? 64u : 0u), smem_desc(q_addr + p * kShRows * HD + i * 32, 16, 8 * HD, X::SWZ),
                           smem_desc(k_addr + i * 32, 16, 8 * HD, X::SWZ), id_s, (p & 1) != 0 || i > 0, one);
        tc_commit_if(b_sf + 8u * gp, one);
        tc_commit_if(b_ke + 8u * ks, one);
        if (k + 1 == n) tc_commit_if(b_qe, one);
        __syncwarp();
        if (++ks == KS) ks = 0u, kpar ^= 1u;
      }
      if (!ok) break;
    }
    if (!ok) {  // (no product may be at work when the CTA exits)
      tc_commit_if(b_end, one);
      mbar_wait(b_end, 0u, kShWaitCycles);
    }
  } else if (warp == 3) {
    // ---- the products of weights and values, from a warp of its own: in one, each kind's issue waits for the other's (131072
    // positions 274 us against 269, 32768 with f32 queries 108 against 100) ----
    const uint32_t id_o = idesc_bf16_f32(kShRows, HD) | 1u << 16, w_addr = smem_u32(wide);
    uint32_t it = 0u, opar[2] = {1u, 1u};
    const uint32_t one = lane == 0;
    while (const int n = __reduce_max_sync(0xffffffffu, next_seg())) {
      seg_done();
#pragma unroll 1
      for (int k = 0; k < n; ++k, ++it) {
        const uint32_t gp = it & 1u, ph = it >> 1 & 1u;  // the tile's group, and the phase of its barriers
        wait(b_wf + 8u * gp, ph);
        wait(b_pf + 8u * gp, ph);
        const bool start = (k >> 1) % X::RUN == 0;  // of a run of the group's tiles
        if (start) {  // (the sums of the run before have been read)
          wait(b_oe + 8u * gp, opar[gp]);
          opar[gp] ^= 1u;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t v_addr = w_addr + gp * X::VB;
#pragma unroll
        for (int kk = 0; kk < TN / 16; ++kk) {
          const uint64_t vd = smem_desc(v_addr + kk * 16 * HD, X::KB, 8 * HD, X::SWZ);
#pragma unroll
          for (int y = 0; y < WP; ++y)
            tc_mma_bf16_ts(tmem + X::O + gp * HD, tmem + gp * X::BUF + kk * 16 + (y < 2 ? y * 8 : 64), vd, id_o,
                           !start || kk > 0 || y > 0, one);
        }
        tc_commit_if(b_of + 8u * gp, one);
        tc_commit_if(b_we + 8u * gp, one);
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok) {
      tc_commit_if(b_end2, one);
      mbar_wait(b_end2, 0u, kShWaitCycles);
    }
  } else if (warp < 12) {
    // ---- softmax: thread = column; the groups take the tiles in turn, each with scores, sums and references of its own ----
    const uint32_t group = (warp - 4) >> 2;
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + group * X::BUF + lanes, t_o = tmem + X::O + group * HD + lanes;
    float* sc = wsc + (warp - 4) * 16;
    float sums[HD];                          // of the runs before (local memory: rarely touched)
    float ref = kQaNone, l = 0.f;            // reference of the column's weights, and their sum
    float vref = 0.f;                        // a power of two that the values' scales are relative to
    uint32_t it = 0u, vs = 0u, vpar = 0u;
    // what waits to be read from tensor memory until the next tile's weights are on their way: a segment's end
    bool pend = false, earlier = false;      // earlier: the segment has sums of runs before
    uint32_t pslot = 0u;
    float pm = 0.f, pl = 0.f, pback = 0.f;
    // where this column's sums of a segment go (its statistics are put down)
    auto place = [&](const ShSeg& o, float m, float sum) {
      return sh_put(a, o.part, group, ((int64_t)o.j * a.r.B * a.r.S + o.gt) * a.g + row, row, m, sum, cta, o.cta0, o.ctas);
    };
    // the products of the group's tiles up to tile t: to the sums, or with the segment's end to global memory
    auto flush = [&](uint32_t t, bool ends) {
      wait(b_of + 8u * group, t >> 1 & 1u);
      __syncwarp();
      const uint32_t slot = ends ? pslot : gslot;
      const int used = segs[slot].used;
      if (quad * 32 < used) {
        const bool write = row < used && ok;
        float* dst = ends && write ? place(segs[slot], pm, pl) : nullptr;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          float v[16];
          tc_ld16(t_o + c, v);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (earlier) v[i] += sums[c + i];
            if (!ends) sums[c + i] = v[i];
          }
          if (dst)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(dst + c + i) = make_float4(v[i] * pback, v[i + 1] * pback, v[i + 2] * pback, v[i + 3] * pback);
        }
        tc_fence_before();
      }
      mbar_arrive(b_oe + 8u * group);
      earlier = !ends;
      if (ends) {
        pend = false;
        __syncwarp();
        if (lane == 0) mbar_arrive(b_ge + 8u * pslot);  // (the segment is read no more)
      }
    };
    while (const int n = next_seg()) {
      wait(b_qf + 8u * gslot, gpar);
      const int start = segs[gslot].start, used = segs[gslot].used;
      int p0 = segs[gslot].p0;
      const float cs = qsc[gslot * kShRows + row];
      const int end = lim[gslot * kShRows + row];
      const bool idle = quad * 32 >= used;
      const int all_end = __reduce_min_sync(0xffffffffu, row < used ? end : 0x7fffffff);
      int own = 0;  // of the segment's tiles, this group's so far
#pragma unroll 1
      for (int k = 0; k < n; ++k, ++it, p0 += TN) {
        if ((it & 1u) == group) {
          // (scores first: once they are there the tile before this one in the ring's stage has been used up, so the
          // stage's barrier, which this group looks at in some of its phases only, can be no phase behind)
          wait(b_sf + 8u * group, it >> 1 & 1u);
          wait(b_vf + 8u * vs, vpar);
          __syncwarp();
          const float x0 = lane < 2 * NB ? ssc[vs * 16 + lane] : 0.f;
          const uint32_t dead = __ballot_sync(0xffffffffu, lane < NB && x0 < 0.f);
          const float vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, lane >= NB && x0 == x0 ? __float_as_uint(x0) : 0u));
          if (lane < 2 * NB) sc[lane] = x0;
          __syncwarp();
          if (lane == 0) mbar_arrive(b_ve + 8u * vs);
          if (own == 0) {  // (what the segment before had goes with its sums)
            if (pend) {
              pm = ref;
              pl = l;
              pback = vref;
            }
            ref = kQaNone;
            l = 0.f;
            vref = 0.f;
          }
          if (!idle) {
            const bool whole = dead == 0u && p0 >= start && p0 + TN <= all_end;
            // the positions of block c that this column sees, as bits
            auto sees = [&](int c) {
              const int lo = min(max(start - p0 - 16 * c, 0), 16), hi = min(max(end - p0 - 16 * c, 0), 16);
              const uint32_t bits = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
              return dead >> c & 1u ? 0u : bits;
            };
            tc_fence_after();
            // Four steps of 32 accumulator columns: 32 positions (bf16), or 16 with what the finer pieces add (f32)
            constexpr int SB = NB / 4;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              uint32_t v[32];
              if constexpr (QT) {
                tc_ld32(t_s + 32 * h, v);
              } else {
                tc_ld16_raw(t_s + 16 * h, v);
                tc_ld16_raw(t_s + 64 + 16 * h, v + 16);
              }
              float f1[SB], w1[SB];
              uint32_t see[SB];
#pragma unroll
              for (int b = 0; b < SB; ++b) {
                see[b] = whole ? 0xffffu : sees(h * SB + b);
                f1[b] = sc[h * SB + b] * cs;
                w1[b] = sc[NB + h * SB + b];
              }
              tc_wait_ld();
              if constexpr (!QT) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(fmaf(__uint_as_float(v[16 + i]), 0x1p-10f, __uint_as_float(v[i])));
              }
              float m = kQaNone;
#pragma unroll
              for (int b = 0; b < SB; ++b) {
                if (!whole) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) v[16 * b + i] = see[b] >> i & 1u ? v[16 * b + i] : 0xff800000u;
                }
                float t[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  t[i] = fmaxf(fmaxf(__uint_as_float(v[16 * b + i]), __uint_as_float(v[16 * b + 4 + i])),
                               fmaxf(__uint_as_float(v[16 * b + 8 + i]), __uint_as_float(v[16 * b + 12 + i])));
                if (see[b]) m = fmaxf(m, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * f1[b]);
              }
              // (a lane without a column has the scores of whatever queries were there: they move no reference of the others,
              // whose roundings would depend on what ran before)
              if (row >= used) m = kQaNone;
              // (references move when a weight exceeds 2^24, or a value's scale 2^16 times, what they are relative to: rarely
              // but with a segment's first tile)
              if (__any_sync(0xffffffffu, m > ref + kShMost) || vtop > vref * 65536.f) {
                const float to = fmaxf(ref, ceilf(m)), corr = qa_exp2(ref - to);
                const float vto = vtop > vref ? __uint_as_float(min(max(__float_as_uint(vtop) >> 23, 1u), 253u) << 23) : vref;
                const float f = vto == vref ? corr : corr * (vref * q_recip(vto));
                ref = to;
                l *= corr;
                vref = vto;
                // the weights of the steps before, once they are there
                if (h > 0) tc_wait_st();
#pragma unroll 1
                for (int c = 0; c < h * SB * WP; ++c) {
                  const uint32_t at = t_s + 16 * (c / WP) + (c % WP < 2 ? 8 * (c % WP) : 64);
                  uint32_t o[8];
#pragma unroll
                  for (int i = 0; i < 8; i += 4) {
                    float d[4];
                    tc_ld4(at + i, d);
                    tc_wait_ld();
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                      const uint32_t u = __float_as_uint(d[z]);
                      o[i + z] = bf16x2(bf16_lo(u) * f, bf16_hi(u) * f);
                    }
                  }
                  tc_st8(at, o);
                }
                if (own > 0) {
                  // what has been added up so far, once the product before is in it
                  wait(b_of + 8u * group, (it - 2u) >> 1 & 1u);
                  __syncwarp();
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < HD; c += 8) {
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                      float d[4];
                      tc_ld4(t_o + c + i, d);
                      tc_wait_ld();
#pragma unroll
                      for (int z = 0; z < 4; ++z) o[i + z] = __float_as_uint(d[z] * f);
                    }
                    tc_st8(t_o + c, o);
                    if (earlier)
#pragma unroll
                      for (int i = 0; i < 8; ++i) sums[c + i] *= f;
                  }
                }
                tc_wait_st();
              }
              const float vinv = vref > 0.f ? q_recip(vref) : 0.f;
              const uint64_t minus = pack2(-ref, -ref), less = pack2(-1.f, -1.f);
#pragma unroll
              for (int b = 0; b < SB; ++b) {
                const int c = h * SB + b;
                // (a block that the column does not see: neither its scale nor its values' counts)
                const float fb = see[b] ? f1[b] : 1.f, wb = see[b] ? w1[b] * vinv : 0.f;
                const uint64_t f = pack2(fb, fb), w = pack2(wb, wb);
                // (stage by stage over the eight pairs, whose chains are long)
                uint64_t p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  p[i] = fma2(pack2(__uint_as_float(v[16 * b + 2 * i]), __uint_as_float(v[16 * b + 2 * i + 1])), f, minus);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float y0, y1;
                  unpack2(p[i], y0, y1);
                  if (!whole) {  // (a scale of 0 would make a hidden score NaN)
                    y0 = v[16 * b + 2 * i] == 0xff800000u ? -INFINITY : y0;
                    y1 = v[16 * b + 2 * i + 1] == 0xff800000u ? -INFINITY : y1;
                  }
                  p[i] = pack2(qa_exp2(y0), qa_exp2(y1));
                }
                const uint64_t s0 = add2(add2(p[0], p[1]), add2(p[2], p[3])), s1 = add2(add2(p[4], p[5]), add2(p[6], p[7]));
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = mul2(p[i], w);
#pragma unroll
                for (int y = 0; y < WP; ++y) {  // each piece the rounding of what the ones before left over
                  uint32_t o[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    float y0, y1;
                    unpack2(p[i], y0, y1);
                    o[i] = bf16x2(y0, y1);
                  }
                  if (y + 1 < WP)
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = fma2(pack2(bf16_lo(o[i]), bf16_hi(o[i])), less, p[i]);
                  tc_st8(t_s + 16 * c + (y < 2 ? 8 * y : 64), o);
                }
                float y0, y1;
                unpack2(add2(s0, s1), y0, y1);
                l += y0 + y1;
              }
            }
            tc_wait_st();
            tc_fence_before();
          }
          mbar_arrive(b_pf + 8u * group);
          // the run before, so that this one's products can start
          if (pend) flush(it - 2u, true);
          else if (own > 0 && own % X::RUN == 0) flush(it - 2u, false);
          ++own;
        }
        if (++vs == VS) vs = 0u, vpar ^= 1u;
      }
      if (own > 0) {
        pend = true;
        pslot = gslot;
      } else {
        // no tile of the segment was this group's
        if (row < used) place(segs[gslot], kQaNone, 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_ge + 8u * gslot);
      }
      if (++gslot == kShSegs) gslot = 0u, gpar ^= 1u;
    }
    if (pend && ok) {
      pm = ref;
      pl = l;
      pback = vref;
      flush(((it - 1u) & 1u) == group ? it - 1u : it - 2u, true);  // (the group's last tile)
    }
  } else {
    // ---- values widened ----
    const int wid = tid - 384;
    uint32_t vs = 0u, vpar = 0u, it = 0u;
    while (const int n = next_seg()) {
      const int start = segs[gslot].start, stop = segs[gslot].stop;
      int p0 = segs[gslot].p0;
      seg_done();
#pragma unroll 1
      for (int k = 0; k < n; ++k, ++it, p0 += TN) {
        wait(b_vf + 8u * vs, vpar);
        wait(b_we + 8u * (it & 1u), (it >> 1 & 1u) ^ 1u);
        __syncwarp();
        {
          constexpr int HB = HD / 32, CH = HD / 16, SH = kShWiden / TN, PER = CH / SH;
          const int r = wid % TN, i0 = wid / TN * PER, swz = HD == 128 ? r & 7 : r >> 1 & 3;
          const bool live = p0 + r >= start && p0 + r < stop && !(ssc[vs * 16 + r / kQBlock] < 0.f);
          const unsigned char* src = vring + vs * X::KB + r * HD;
          unsigned char* dst = wide + (it & 1u) * X::VB + r * HD;
#pragma unroll 4
          for (int i = 0; i < PER; ++i) {
            const int from = i0 + i, to = 2 * (from % HB);
            uint4 v = *reinterpret_cast<const uint4*>(src + ((from ^ swz) << 4)), lo, hi;
            if (!live) v = make_uint4(0u, 0u, 0u, 0u);
            qa_widen16(v, lo, hi);
            unsigned char* d = dst + (from < HB ? 0 : X::KB);
            *reinterpret_cast<uint4*>(d + ((to ^ swz) << 4)) = lo;
            *reinterpret_cast<uint4*>(d + (((to + 1) ^ swz) << 4)) = hi;
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(b_wf + 8u * (it & 1u));
        __syncwarp();
        if (lane == 0) mbar_arrive(b_ve + 8u * vs);
        if (++vs == VS) vs = 0u, vpar ^= 1u;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// one instantiation per translation unit
template <int HD, int QT>
cudaError_t launch_qshare(const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap, const QAttnArgs& a, int grid, cudaStream_t s, bool pdl) {
  constexpr size_t smem = ShShape<HD, QT>::SMEM;
  auto fn = qshare_kernel<HD, QT>;
  // (the limit belongs to the device's context: set on every call, a fraction of a microsecond)
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kShThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, kmap, vmap, qmap, a);
}

#define LLM_QSHARE(NAME) \
  cudaError_t NAME(const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap, const QAttnArgs& a, int grid, cudaStream_t s, bool pdl)
LLM_QSHARE(qshare64_f32);
LLM_QSHARE(qshare64_bf16);
LLM_QSHARE(qshare128_f32);
LLM_QSHARE(qshare128_bf16);

}  // namespace llm
