// Attention of rows that share positions: which kernel takes which part of a call, and the join of what they sum.
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

constexpr int kMergeThreads = 128;

// Thread = (column, four dimensions).  Bound by the reads of the sums, which lie in L2.
template <int QT>
__global__ void __launch_bounds__(kMergeThreads) qshare_merge_kernel(const QAttnArgs a, const ShSide prefix, const ShSide own) {
  const int q4 = a.c.hd / 4, BS = a.r.B * a.r.S, cols = BS * a.c.kv * a.g;
  const bool sharing = sh_fine(a);
  const int64_t t = (int64_t)blockIdx.x * kMergeThreads + threadIdx.x;
  const int col = (int)(t / q4), k4 = (int)(t - (int64_t)col * q4);
  if (col >= cols) return;
  const int jt = col / a.g, h = col - jt * a.g, j = jt / BS, gt = jt - j * BS, b = gt / a.r.S, i = gt - b * a.r.S;
  if (i >= q_count(a.r, b)) return;
  int lead, last;
  const int sh = sharing ? sh_group(a, b, lead, last) : 0, end = sh_end(a, b, i);
  // (a column that sees something of a side is in a unit that has tiles there)
  const bool there[2] = {sh > 0 && end > 0, end > sh};
  grid_dep_wait();
  // the parts: by side and group, each the unit's first run and those of the CTAs that go on with it
  float4 st[4] = {};
  int first[4] = {}, runs[4] = {}, at[4] = {};
  float M = kQaNone, L = 0.f;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const ShSide& x = y / 2 ? own : prefix;
    if (!there[y / 2] || y % 2 >= x.groups) continue;
    st[y] = __ldcg(x.stats + (int64_t)y * cols + col);
    M = fmaxf(M, st[y].x);
    first[y] = __float_as_int(st[y].z) + 1;
    runs[y] = __float_as_int(st[y].w) >> 8;
    at[y] = min(__float_as_int(st[y].w) & 255, x.pitch - 1);
    // (where a wait gave up, there is nothing to go by)
    if (first[y] < 1 || runs[y] < 0 || runs[y] > x.ctas - first[y]) runs[y] = 0;
#pragma unroll 4
    for (int c = 0; c < runs[y]; ++c) M = fmaxf(M, __ldcg(x.mstats + ((first[y] + c) * x.groups + y % 2) * x.pitch + at[y]).x);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // (a part without weight has no sums)
  auto plus = [&](float m, float l, const float* v) {
    if (l == 0.f) return;
    const float f = qa_exp2(m - M);
    const float4 s = __ldcg(reinterpret_cast<const float4*>(v) + k4);
    L = fmaf(f, l, L);
    o.x = fmaf(f, s.x, o.x); o.y = fmaf(f, s.y, o.y); o.z = fmaf(f, s.z, o.z); o.w = fmaf(f, s.w, o.w);
  };
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const ShSide& x = y / 2 ? own : prefix;
    if (!there[y / 2] || y % 2 >= x.groups) continue;
    plus(st[y].x, st[y].y, x.parts + ((int64_t)y * cols + col) * a.c.hd);
#pragma unroll 4
    for (int c = 0; c < runs[y]; ++c) {
      const int64_t part = (int64_t)((first[y] + c) * x.groups + y % 2) * x.pitch + at[y];
      const float2 s = __ldcg(x.mstats + part);
      plus(s.x, s.y, x.more + part * a.c.hd);
    }
  }
  const float r = L == 0.f ? 0.f : 1.f / L;
  qa_put4<QT>(a.out, (int64_t)gt * a.out_stride + (int64_t)(j * a.g + h) * a.c.hd + 4 * k4, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
}

// Which kernel takes the prefixes: that of many columns where a group has more than kShFew on average
constexpr int kShFew = 40;
struct ShPlan {
  bool many;
  int nc, cols;        // the other kernel's accumulator columns in 16s, and columns of a unit
  int64_t columns;     // of the call
};
ShPlan plan_of(const QCacheView& c, int g, int qt, int64_t B, int64_t S, int64_t ngroups) {
  ShPlan p;
  const int64_t group = (B * S * g + ngroups - 1) / ngroups;
  p.many = group > kShFew;
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
  return units <= kShSlots && p.columns < (1ll << 31) / c.hd && units * c.kv * ((int64_t)limit / 64 + 2) < 1ll << 31;
}

uint64_t qshare_workspace(const QCacheView& c, int g, int B, int S, int num_sms) {
  const uint64_t columns = (uint64_t)B * S * c.kv * g;
  return 4 * columns * (c.hd * 4 + 16) + (uint64_t)num_sms * (2 * kShRows + 2 * 32) * (c.hd * 4 + 8);
}

cudaError_t launch_qshare_all(const QAttnArgs& a0, int qt, int num_sms, cudaStream_t s) {
  QAttnArgs a = a0;
  const int64_t B = a.r.B, S = a.r.S;
  const ShPlan p = plan_of(a.c, a.g, qt, B, S, a.ngroups);
  ShSide few = side_of(B, S, a.g, p.cols, p.many ? 2 : 3, 1), many = side_of(B, S, a.g, kShRows, 1, 2);
  few.ctas = few_ctas(p.cols, num_sms);
  many.ctas = num_sms;
  unsigned char* w = a.ws;
  auto take = [&](uint64_t n) {
    unsigned char* at = w;
    w += n;
    return at;
  };
  few.parts = many.parts = reinterpret_cast<float*>(take(4 * (uint64_t)p.columns * a.c.hd * 4));
  few.stats = many.stats = reinterpret_cast<float4*>(take(4 * (uint64_t)p.columns * 16));
  for (ShSide* x : {&few, &many}) {
    const uint64_t n = (uint64_t)x->ctas * x->groups * x->pitch;
    x->more = reinterpret_cast<float*>(take(n * a.c.hd * 4));
    x->mstats = reinterpret_cast<float2*>(take(n * 8));
  }
  CUtensorMap kmap, vmap;
  const uint64_t rows = (uint64_t)a.c.rows * a.c.kv * a.c.cap;
  if (!qattn_make_map(&kmap, a.c.k, a.c.hd, rows) || !qattn_make_map(&vmap, a.c.v, a.c.hd, rows)) return cudaErrorInvalidValue;
  a.sh = few;
  auto fn = a.c.hd == 64 ? (qt ? qattn_sh64_bf16 : qattn_sh64_f32) : (qt ? qattn_sh128_bf16 : qattn_sh128_f32);
  cudaError_t e = fn(kmap, vmap, a, p.nc, few.ctas, s, false);
  if (e != cudaSuccess) return e;
  if (p.many) {
    a.sh = many;
    auto fm = a.c.hd == 64 ? (qt ? qshare64_bf16 : qshare64_f32) : (qt ? qshare128_bf16 : qshare128_f32);
    e = fm(kmap, vmap, a, many.ctas, s, true);
    if (e != cudaSuccess) return e;
  }
  const int64_t threads = p.columns * (a.c.hd / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((threads + kMergeThreads - 1) / kMergeThreads));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qt ? qshare_merge_kernel<1> : qshare_merge_kernel<0>, a, p.many ? many : few, few);
}

}  // namespace llm
