// Attention of rows that share positions, read once for all that share them: which kernel takes which part of a call, and the join
// of what they sum.  (Calls that gain nothing from it are attended row by row, qattn.cu.)
//
// Both kernels sum over a share of the units' position tiles per CTA and leave their sums in the workspace.  Units of
// few columns -- a row's own positions, or a prefix that few rows share -- run on the kernel of the ordinary attention
// (qattn_tc.cuh, positions on the M side: a tile of up to 32 columns costs little more than its loads), a prefix that
// many columns share on that of qshare.cuh (columns on the M side, 128 of them a tile).  The last kernel joins each
// column's parts, its prefix's and its own, in CTA order, so the result does not depend on timing.
#include <algorithm>

#include "qshare.cuh"

namespace llm {

namespace {

constexpr int kMergeThreads = 256;

// One, two or four warps to a column (`split`): its parts' statistics a lane each in every one of them, then the parts' sums,
// eight loads in flight, by turns (heads of 64: two parts at a time, half a warp each).  Bound by the reads of the sums, which
// lie in L2 (32 rows of 32 heads behind 8192 positions: 1024 columns of some 40 parts, 21 MB).
template <int HD, int QT>
__global__ void __launch_bounds__(kMergeThreads) qshare_merge_kernel(const QAttnArgs a, const ShSide prefix, const ShSide own, int split) {
  __shared__ float4 half[kMergeThreads];
  const int BS = a.r.B * a.r.S, cols = BS * a.c.kv * a.g, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool sharing = sh_fine(a);
  const int at_warp = blockIdx.x * (kMergeThreads / 32) + warp, col = at_warp / split, mine_of = at_warp - col * split;
  const int jt = col / a.g, h = col - jt * a.g, j = jt / BS, gt = jt - j * BS, b = gt / a.r.S, i = gt - b * a.r.S;
  const bool live = col < cols && i < q_count(a.r, b);
  int lead, last;
  const int sh = live && sharing ? sh_group(a, b, lead, last) : 0, end = live ? sh_end(a, b, i) : 0;
  // (a column that sees something of a side is in a unit that has tiles there)
  const bool there[2] = {sh > 0 && end > 0, end > sh};
  grid_dep_wait();
  // parts, by side and group: the unit's first run, then those of the CTAs that go on with it
  float4 st[4] = {};
  int before[5] = {0, 0, 0, 0, 0};
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const ShSide& x = y / 2 ? own : prefix;
    int n = 0;
    if (there[y / 2] && y % 2 < x.groups) {
      st[y] = __ldcg(x.stats + (int64_t)y * cols + col);
      const int c0 = __float_as_int(st[y].z), runs = __float_as_int(st[y].w) >> 8;
      // (where a wait gave up, there is nothing to go by)
      n = c0 < 0 || runs < 0 || runs >= x.ctas - c0 ? 1 : runs + 1;
    }
    before[y + 1] = before[y] + n;
  }
  const int np = before[4];
  // a part's statistics, and where its sums are
  auto part = [&](int p, const float*& at) {
    const int y = (p >= before[1]) + (p >= before[2]) + (p >= before[3]);
    const ShSide& x = y / 2 ? own : prefix;
    const float4 s = y == 0 ? st[0] : y == 1 ? st[1] : y == 2 ? st[2] : st[3];
    const int c = p - (y == 0 ? 0 : y == 1 ? before[1] : y == 2 ? before[2] : before[3]);
    if (c == 0) {
      at = x.parts + ((int64_t)y * cols + col) * HD;
      return make_float2(s.x, s.y);
    }
    const int64_t place = (int64_t)((__float_as_int(s.z) + c) * x.groups + y % 2) * x.pitch + min(__float_as_int(s.w) & 255, x.pitch - 1);
    at = x.more + place * HD;
    return __ldcg(x.mstats + place);
  };
  float M = kQaNone;
  const float* at = nullptr;
  float2 mine = make_float2(kQaNone, 0.f);
  for (int p0 = 0; p0 < np; p0 += 32) {
    if (p0 + lane < np) mine = part(p0 + lane, at);
    M = fmaxf(M, mine.x);
  }
  M = warp_max(M);
  constexpr int W = HD / 4, SIDE = 32 / W;  // lanes of a part, parts at a time
  const int k4 = lane % W, sub = lane / W;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < np; p0 += 32) {
    if (np > 32) mine = p0 + lane < np ? part(p0 + lane, at) : make_float2(kQaNone, 0.f);
    // (a part without weight has no sums)
    const float f = mine.y == 0.f ? 0.f : qa_exp2(mine.x - M);
    L = fmaf(f, mine.y, L);
    const int n = min(32, np - p0);
    constexpr int U = 8;
    for (int q0 = 0; q0 < n; q0 += U * SIDE) {
      if ((p0 + q0) / (U * SIDE) % split != mine_of) continue;
      float4 v[U];
      float fp[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * SIDE + sub, from = min(q, 31);
        const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), from));
        fp[u] = __shfl_sync(0xffffffffu, f, from);
        if (q >= n) fp[u] = 0.f;
        v[u] = fp[u] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(reinterpret_cast<const float4*>(src) + k4);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        o.x = fmaf(fp[u], v[u].x, o.x);
        o.y = fmaf(fp[u], v[u].y, o.y);
        o.z = fmaf(fp[u], v[u].z, o.z);
        o.w = fmaf(fp[u], v[u].w, o.w);
      }
    }
  }
  L = warp_sum(L);
  if constexpr (SIDE == 2) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
  }
  if (split > 1) {  // (a column's warps, in their order)
    half[threadIdx.x] = o;
    __syncthreads();
    if (!live || mine_of > 0) return;
    for (int w = 1; w < split; ++w) {
      const float4 x = half[threadIdx.x + 32 * w];
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
  }
  if (!live) return;
  const float r = L == 0.f ? 0.f : 1.f / L;
  if (sub == 0)
    qa_put4<QT>(a.out, (int64_t)gt * a.out_stride + (int64_t)(j * a.g + h) * HD + 4 * k4, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
}

// Queries in e4m3 pieces (qshare.cuh), warp = column; of tokens that are not there: zeros.  As a kernel of its own
// (3 us) they are made once; four warps of each CTA of the attention took 13 us for 128 columns.
template <int HD, int QT>
__global__ void __launch_bounds__(kMergeThreads) qshare_pieces_kernel(const QAttnArgs a) {
  constexpr int NP = QT ? 2 : 4, E = HD / 32;
  grid_dep_launch();
  const int BS = a.r.B * a.r.S, cols = BS * a.c.kv * a.g, lane = threadIdx.x & 31;
  const int col = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (col >= cols) return;
  const int jt = col / a.g, h = col - jt * a.g, j = jt / BS, gt = jt - j * BS, b = gt / a.r.S;
  float v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = 0.f;
  if (gt - b * a.r.S < q_count(a.r, b)) {
    const int64_t at = (int64_t)gt * a.q_stride + (int64_t)(j * a.g + h) * HD + lane * E;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      if constexpr (QT) {
        const uint32_t f = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at + i);
        v[i] = bf16_lo(f);
        v[i + 1] = bf16_hi(f);
      } else {
        const float2 f = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + i);
        v[i] = f.x;
        v[i + 1] = f.y;
      }
    }
  }
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  const bool fine = top < 0x7f800000u;
  const float s = q_scale(fine ? __uint_as_float(top) * 1.75f : 0.f), r = a.scale < 0.f ? -q_recip(s) : q_recip(s);  // |x| r <= 256
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = fine ? v[i] * r : 0.f;
#pragma unroll
  for (int y = 0; y < NP; ++y) {
    uint32_t code = 0u;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint32_t p = e4m3x2(v[i], v[i + 1]);
      const float2 f = e4m3_pair(p);
      v[i] = (v[i] - f.x) * (y == 1 ? 1024.f : 1.f);
      v[i + 1] = (v[i + 1] - f.y) * (y == 1 ? 1024.f : 1.f);
      code |= p << (8 * i);
    }
    uint8_t* dst = a.sh.qp + ((int64_t)y * cols + col) * HD + lane * E;
    if constexpr (E == 4) *reinterpret_cast<uint32_t*>(dst) = code;
    else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)code;
  }
  // (a query that is not finite makes its scores NaN)
  if (lane == 0) a.sh.qs[col] = fine ? s * (fabsf(a.scale) * 1.4426950408889634f) : __uint_as_float(0x7fc00000u);
}

// Which kernel takes the prefixes: that of many columns where a group has more than this on average.  Its tile costs the
// same for any number of columns, twice as much with f32 queries as with bf16; the other's grows with every 32 (8 kv heads
// of 128, 4 groups behind 16000 positions, microseconds with the kernel for many and the one for few: bf16 24 columns 88 and 71, 32 92
// and 98, 40 98 and 108, 64 102 and 153; f32 32 columns 190 and 104, 64 201 and 161, 128 (2 groups) 153 and 147)
constexpr int kShFew[2] = {100, 40};  // f32, bf16
struct ShPlan {
  bool many;
  int nc, cols;        // the other kernel's accumulator columns in 16s, and columns of a unit
  int64_t columns;     // of the call
};
ShPlan plan_of(const QCacheView& c, int g, int qt, int64_t B, int64_t S, int64_t ngroups) {
  ShPlan p;
  const int64_t group = (B * S * g + ngroups - 1) / ngroups;
  p.many = group > kShFew[qt];
  const int np = qt ? 2 : 4, most = qt ? 4 : 8;
  const int64_t want = std::min<int64_t>(32, std::max(S * g, p.many ? 0 : group));
  p.nc = 1;
  while (p.nc < most && p.nc * 16 / np < want) p.nc *= 2;
  p.cols = p.nc * 16 / np;
  p.columns = B * S * c.kv * g;
  return p;
}
ShSide side_of(int64_t B, int64_t S, int g, int cols, int sides, int groups) {
  ShSide x = {};
  x.tpt = (int)std::min<int64_t>(cols / g, S);
  x.cpr = (int)((S + x.tpt - 1) / x.tpt);
  x.rpt = x.cpr == 1 ? (int)std::min<int64_t>(B, cols / g / S) : 1;
  x.sides = sides;
  x.pitch = cols;
  x.groups = groups;
  return x;
}
// CTAs of the two kernels at most
int few_ctas(int cols, int num_sms) { return num_sms * (cols <= 8 ? 2 : 1); }

}  // namespace

bool qshare_fits(const QCacheView& c, int g, int qt, int B, int S, int ngroups, int limit) {
  const ShPlan p = plan_of(c, g, qt, B, S, ngroups);
  const ShSide x = side_of(B, S, g, p.cols, 3, 1);
  const int64_t units = 2 * (int64_t)B * x.cpr;
  return units <= kShUnits && p.columns < (1ll << 31) / c.hd && units * c.kv * ((int64_t)limit / 64 + 2) < 1ll << 31;
}

uint64_t qshare_workspace(const QCacheView& c, int g, int B, int S, int num_sms) {
  const uint64_t columns = (uint64_t)B * S * c.kv * g;
  return kQattnTickets + 4 * columns * (c.hd * 4 + 16) + columns * (4 * c.hd + 16) + (uint64_t)num_sms * (2 * kShRows + 2 * 32) * (c.hd * 4 + 8);
}

namespace {
cudaError_t launch(void* fn, int64_t grid, void** args, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}
}  // namespace

// The kernels of a call follow one another programmatically: each but the first may start before the one before
// is done, waits for it before it reads what that wrote, and is done only after it.  (Side by side, each on SMs of its own in
// proportion to its work, they took 45 us in place of 54 behind 8192 positions, but 302 in place of 274 behind 131072: CTAs of one
// next to SMs that run the other are up to 15% slower, and the slowest decides.)
cudaError_t launch_qshare_all(const QAttnArgs& a0, int qt, int num_sms, cudaStream_t s) {
  QAttnArgs a = a0;
  const int64_t B = a.r.B, S = a.r.S;
  const int hd = a.c.hd, np = qt ? 2 : 4;
  const ShPlan p = plan_of(a.c, a.g, qt, B, S, a.ngroups);
  ShSide few = side_of(B, S, a.g, p.cols, p.many ? 2 : 3, 1), many = side_of(B, S, a.g, kShRows, 1, 2);
  few.ctas = few_ctas(p.cols, num_sms);
  many.ctas = num_sms;
  unsigned char* w = a.ws + kQattnTickets;  // (the ordinary attention's tickets stay as they are)
  auto take = [&](uint64_t n) {
    unsigned char* at = w;
    w += n;
    return at;
  };
  const uint64_t columns = (uint64_t)p.columns;
  few.parts = many.parts = reinterpret_cast<float*>(take(4 * columns * hd * 4));
  few.stats = many.stats = reinterpret_cast<float4*>(take(4 * columns * 16));
  many.qp = take(columns * 4 * hd);
  many.qs = reinterpret_cast<float*>(take(columns * 16));
  for (ShSide* x : {&few, &many}) {
    const uint64_t n = (uint64_t)x->ctas * x->groups * x->pitch;
    x->more = reinterpret_cast<float*>(take(n * hd * 4));
    x->mstats = reinterpret_cast<float2*>(take(n * 8));
  }
  CUtensorMap kmap, vmap, qmap;
  const uint64_t rows = (uint64_t)a.c.rows * a.c.kv * a.c.cap;
  if (!qattn_make_map(&kmap, a.c.k, hd, rows) || !qattn_make_map(&vmap, a.c.v, hd, rows)) return cudaErrorInvalidValue;
  auto grid = [&](int64_t warps) { return (warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32); };
  cudaError_t e = cudaSuccess;
  if (p.many) {
    if (!qattn_make_map(&qmap, many.qp, hd, np * columns)) return cudaErrorInvalidValue;
    a.sh = many;
    void* args[] = {&a};
    auto fn = hd == 64 ? (qt ? qshare_pieces_kernel<64, 1> : qshare_pieces_kernel<64, 0>)
                       : (qt ? qshare_pieces_kernel<128, 1> : qshare_pieces_kernel<128, 0>);
    e = launch((void*)fn, grid(p.columns), args, s, false);
    if (e != cudaSuccess) return e;
  }
  a.sh = few;
  auto fn = hd == 64 ? (qt ? qattn_sh64_bf16 : qattn_sh64_f32) : (qt ? qattn_sh128_bf16 : qattn_sh128_f32);
  e = fn(kmap, vmap, a, p.nc, few.ctas, s, p.many);
  if (e != cudaSuccess) return e;
  if (p.many) {
    a.sh = many;
    auto fm = hd == 64 ? (qt ? qshare64_bf16 : qshare64_f32) : (qt ? qshare128_bf16 : qshare128_f32);
    e = fm(kmap, vmap, qmap, a, many.ctas, s, true);
    if (e != cudaSuccess) return e;
  }
  // warps of a column: as many as the SMs hold at once, two CTAs each (1 / 2 / 4: 1024 columns behind 8192 positions 54 / 52 / 57
  // us a call, 64 behind 65536 45 / 43 / 42, 1536 behind 2047 72 / 75 / 78)
  int split = 1;
  while (split < 4 && p.columns * split * 2 <= (int64_t)num_sms * (2 * kMergeThreads / 32)) split *= 2;
  void* args[] = {&a, p.many ? &many : &few, &few, &split};
  auto fj = hd == 64 ? (qt ? qshare_merge_kernel<64, 1> : qshare_merge_kernel<64, 0>)
                     : (qt ? qshare_merge_kernel<128, 1> : qshare_merge_kernel<128, 0>);
  return launch((void*)fj, grid(p.columns * split), args, s, true);
}

}  // namespace llm
