// Writing into and reading from an 8-bit key/value cache.
//
// A block is kQBlock consecutive positions of one cache row and key/value head.  Its scale s is a
// power of two, so dividing by it, multiplying by it and moving a code from one scale to another
// are exact in f32 but for the rounding to e4m3 itself (to nearest even, off by at most 2^-4 of the
// value while |x| / s >= 2^-6, by at most 2^-10 s below).  A float format keeps its relative error
// over 14 binades below the largest value of the block, so the scale only has to place the largest
// value near 448 and a power of two loses at most a factor of two of the range.
//
// Writing tokens p0 .. p0 + n - 1 of a row, per block that they touch:
//   need = the least power of two >= 2^-126 with max |x| / need <= 448 over the new values;
//   s    = need if the call writes the block's first position, else max(s_old, need), and the
//          codes of the block's positions before p0 are rounded again from s_old to s;
//   code = e4m3(x / s).
// Values that are not finite make need NaN (their codes are 0): the block then reads as NaN until
// its first position is written anew, and no code is ever NaN, so a product over codes stays finite
// for every token that does not see the block.  Codes of positions after the new tokens are not
// touched.
//
// Bounds: both directions are HBM-bound for long inputs and launch-latency-bound for one token per
// row.  One warp owns a (block, head, keys or values): its 16 tokens' rows are all loaded at once
// (16 independent 16-byte loads a lane at hd 128, f32), reduced in registers and stored as codes, so
// each value is read once and the maximum costs no second pass.  Reading mirrors it, every store of a
// warp one contiguous run.  GB300, copy rate 6.79 TB/s: 32 rows of one token (8 heads of 128) written in
// 2.6 us; 16 rows of up to 2048 bf16 tokens (174 MB in and out) in 30.3 us, 85% of the copy rate, with the
// values packed as read (widened to f32 in registers: 46 us, half the warps in flight); 32 such rows read
// back (315 MB) in 48.8 us, 95% (rounding to bf16 in integer steps instead of one conversion per pair:
// 77 us).
#include <algorithm>
#include <type_traits>

#include "qcache.cuh"

namespace llm {

namespace {

constexpr int kQThreads = 128;

// 16 bytes of a row of type ST (0 f32, 1 bf16): E elements
template <int ST> constexpr int kE = ST ? 8 : 4;
template <int ST>
LLM_D uint4 load16(const void* p, int64_t i) {
  return ST ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i)
            : *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
}
// the largest |element| of 16 bytes, as the bits of an f32 (ordered; not finite: >= 0x7f800000)
template <int ST>
LLM_D uint32_t top16(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t t = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t = max(t, w[i] & (ST ? 0x7fff0000u : 0x7fffffffu));
    if constexpr (ST) t = max(t, w[i] << 16 & 0x7fff0000u);
  }
  return t;
}

// One warp: n tokens (1 <= t0 + n <= kQBlock) at positions t0 .. t0 + n - 1 of a block, whose codes
// start at `codes` and whose scale is *scale; token i's values are the HD elements at src + i * stride.
// The values stay packed as they were read (bf16: half the registers, twice the warps in flight).
template <int HD, int ST>
LLM_D void quantise_run(uint8_t* codes, float* scale, int t0, int n, const void* src, int64_t base, int64_t stride) {
  constexpr int E = kE<ST>;
  constexpr int QR = HD / E;                  // 16-byte pieces per token
  constexpr int NQ = (kQBlock * QR + 31) / 32;  // pieces per lane
  const int lane = threadIdx.x & 31;
  const int nq = n * QR;
  const float s_old = t0 > 0 ? *scale : 0.0f;
  uint4 x[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int q = lane + 32 * i;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (q < nq) x[i] = load16<ST>(src, base + (int64_t)(q / QR) * stride + (q % QR) * E);
  }
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < NQ; ++i) top = max(top, top16<ST>(x[i]));
  top = __reduce_max_sync(0xffffffffu, top);
  const bool fine = top < 0x7f800000u && s_old == s_old;
  float s = fine ? q_scale(__uint_as_float(top)) : __uint_as_float(0x7fc00000u);
  if (fine && t0 > 0) s = fmaxf(s, s_old);
  if (fine && s > s_old && t0 > 0) {
    // the tokens before, from s_old to s: their values times s_old / s < 1 (both powers of two)
    const float f = s_old * q_recip(s);
    uint32_t* c4 = reinterpret_cast<uint32_t*>(codes);
    for (int q = lane; q < t0 * (HD / 4); q += 32) {
      const float4 v = e4m3_quad(c4[q]);
      c4[q] = e4m3x2(v.x * f, v.y * f) | e4m3x2(v.z * f, v.w * f) << 16;
    }
  }
  const float r = fine ? q_recip(s) : 0.0f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(codes + t0 * HD);
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int q = lane + 32 * i;
    if (q < nq) {
      if constexpr (ST) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t c[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) c[y] = fine ? e4m3x2(bf16_lo(w[y]) * r, bf16_hi(w[y]) * r) : 0u;
        reinterpret_cast<uint2*>(dst)[q] = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
      } else {
        const float4 f = make_float4(__uint_as_float(x[i].x), __uint_as_float(x[i].y), __uint_as_float(x[i].z),
                                     __uint_as_float(x[i].w));
        dst[q] = fine ? e4m3x2(f.x * r, f.y * r) | e4m3x2(f.z * r, f.w * r) << 16 : 0u;
      }
    }
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *scale = s;
}

// warp w of the grid: (row, touched block, kv head, keys or values), the last the fastest
template <int HD, int ST>
__global__ void __launch_bounds__(kQThreads)
    qcache_write_kernel(const QCacheView c, const QRows r, const void* k, const void* v, int64_t stride, int span) {
  const uint32_t w = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);  // (below 2^31: the host refuses more)
  const int side = (int)(w & 1);
  const uint32_t bj = (w >> 1) / (uint32_t)c.kv;
  const int h = (int)((w >> 1) - bj * (uint32_t)c.kv), b = (int)(bj / (uint32_t)span), j = (int)bj - b * span;
  if (b >= r.B) return;
  const int p0 = r.first[b], n = q_count(r, b);
  if (n == 0) return;
  if (p0 < 0 || p0 > r.limit - n) {
    q_report(r.status, kErrPosRange);
    return;
  }
  const int blk = p0 / kQBlock + j;           // the block in the row
  const int lo = max(p0, blk * kQBlock), hi = min(p0 + n, (blk + 1) * kQBlock);
  if (lo >= hi) return;
  int row, pp;
  if (!q_place(r, c, b, blk * kQBlock, row, pp)) return;
  const size_t head = (size_t)row * c.kv + h;
  uint8_t* codes = (side ? c.v : c.k) + (head * c.cap + pp) * HD;
  float* scale = (side ? c.vs : c.ks) + head * (c.cap / kQBlock) + pp / kQBlock;
  quantise_run<HD, ST>(codes, scale, lo - blk * kQBlock, hi - lo, side ? v : k,
                       ((int64_t)b * r.S + (lo - p0)) * stride + (int64_t)h * HD, stride);
}

// Rows of a handle's step (heads of 64 and 128: only a prefill pass's entries; their decode steps store
// within the attention): warp (entry, kv head, keys or values); staged values [entries][kv][HD].  A
// prefill pass (all of its entries at once: entry_step 1) lists the entries of a cache row in position order, so the entries of one block
// follow one another: the first of them (the leader) writes all, run by run of consecutive
// positions, and the others' warps leave.
template <int HD, int ST>
__global__ void __launch_bounds__(kQThreads)
    qcache_write_step_kernel(const QCacheView c, const QRows r, const void* k, const void* v) {
  grid_dep_launch();
  const uint32_t w = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
  const int side = (int)(w & 1);
  const int b = (int)((w >> 1) / (uint32_t)c.kv), h = (int)((w >> 1) - (uint32_t)b * (uint32_t)c.kv);
  if (b >= r.B) return;
  const int e = q_entry(r, b);
  auto slot = [&](int i, int& row, int& pp) { cache_slot(r.step, c.cap, i, row_pos(r.step, i), row, pp); };
  int row, pp;
  slot(e, row, pp);
  int n = 1;
  if (r.step->rowmap && r.entry_step == 1) {
    int pr, pq;
    if (e > 0) {
      slot(e - 1, pr, pq);
      if (pr == row && pq / kQBlock == pp / kQBlock) return;
    }
    n = 0;
    while (n < kQBlock && e + n < r.B) {
      slot(e + n, pr, pq);
      if (pr != row || pq / kQBlock != pp / kQBlock) break;
      ++n;
    }
  }
  const size_t head = (size_t)row * c.kv + h;
  const int blk = pp / kQBlock;
  uint8_t* codes = (side ? c.v : c.k) + (head * c.cap + (size_t)blk * kQBlock) * HD;
  float* scale = (side ? c.vs : c.ks) + head * (c.cap / kQBlock) + blk;
  const int64_t stride = (int64_t)c.kv * HD;
  grid_dep_wait();  // (the step's state was written before its kernels; the staged values were not)
  for (int i = 0; i < n;) {
    int r0, q0, len = 1;
    slot(e + i, r0, q0);
    while (i + len < n) {
      int r1, q1;
      slot(e + i + len, r1, q1);
      if (q1 != q0 + len) break;
      ++len;
    }
    quantise_run<HD, ST>(codes, scale, q0 - blk * kQBlock, len, side ? v : k, (int64_t)(e + i) * stride + (int64_t)h * HD,
                         stride);
    __syncwarp();
    i += len;
  }
}

// CTA (layer and kv head, row)
__global__ void __launch_bounds__(kQThreads) qcache_keep_kernel(const QVerify v) {
  const int l = blockIdx.x / v.c.kv, h = blockIdx.x - l * v.c.kv, b = blockIdx.y;
  const int e = q_entry(v.r, b), hd = v.c.hd;
  int row, pp;
  cache_slot(v.r.step, v.c.cap, e, row_pos(v.r.step, e), row, pp);
  const int t0 = pp % kQBlock;
  if (t0 == 0) return;
  const size_t head = ((size_t)l * v.c.rows + row) * v.c.kv + h, kept = ((size_t)l * v.c.rows + b) * v.c.kv + h;
  const size_t from = (head * v.c.cap + (pp - t0)) * hd, to = kept * kQBlock * hd;
  for (int i = threadIdx.x; i < t0 * hd / 16; i += kQThreads) {
    reinterpret_cast<uint4*>(v.kept_k + to)[i] = reinterpret_cast<const uint4*>(v.c.k + from)[i];
    reinterpret_cast<uint4*>(v.kept_v + to)[i] = reinterpret_cast<const uint4*>(v.c.v + from)[i];
  }
  if (threadIdx.x == 0) {
    const size_t sc = head * (v.c.cap / kQBlock) + pp / kQBlock;
    v.kept_ks[kept] = v.c.ks[sc];
    v.kept_vs[kept] = v.c.vs[sc];
  }
}

// warp (layer, row, kv head, keys or values)
template <int HD, int ST>
__global__ void __launch_bounds__(kQThreads) qcache_settle_kernel(const QVerify v) {
  const int64_t w = (int64_t)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
  const int side = (int)(w & 1), lane = threadIdx.x & 31;
  const int64_t u = w >> 1;
  const int h = (int)(u % v.c.kv), b = (int)(u / v.c.kv % v.r.B), l = (int)(u / v.c.kv / v.r.B);
  if (l >= v.layers) return;
  const int e = q_entry(v.r, b), kept_drafts = v.accepted[b];
  if (kept_drafts >= v.T - 1) return;         // nothing else was written
  const int p0 = row_pos(v.r.step, e), last = p0 + kept_drafts;
  const int t1 = last % kQBlock + 1;          // tokens of the block up to the last that was kept
  int row, pp;
  cache_slot(v.r.step, v.c.cap, e, last, row, pp);
  const size_t head = ((size_t)l * v.c.rows + row) * v.c.kv + h;
  uint8_t* codes = (side ? v.c.v : v.c.k) + (head * v.c.cap + (pp + 1 - t1)) * HD;
  float* scale = (side ? v.c.vs : v.c.ks) + head * (v.c.cap / kQBlock) + pp / kQBlock;
  // the blocks behind hold nothing
  for (int i = 1 + lane; i <= (p0 + v.T - 1) / kQBlock - last / kQBlock; i += 32) scale[i] = 0.f;
  if (t1 == kQBlock) return;
  const int t0 = max(0, p0 - (last + 1 - t1));  // tokens of the block before this call's
  if (t0 > 0) {
    const size_t kept = ((size_t)l * v.c.rows + b) * v.c.kv + h;
    const uint4* from = reinterpret_cast<const uint4*>((side ? v.kept_v : v.kept_k) + kept * kQBlock * HD);
    for (int i = lane; i < t0 * HD / 16; i += 32) reinterpret_cast<uint4*>(codes)[i] = from[i];
    if (lane == 0) *scale = (side ? v.kept_vs : v.kept_ks)[kept];
    __syncwarp();
  }
  const int64_t stride = (int64_t)v.c.kv * HD;
  const int64_t base = ((int64_t)l * v.stage_rows + e + (last + 1 - t1 + t0 - p0)) * stride + (int64_t)h * HD;
  for (int t = t0; t < t1; ++t) {
    quantise_run<HD, ST>(codes, scale, t, 1, side ? v.stage_v : v.stage_k, base + (t - t0) * stride, stride);
    __syncwarp();
  }
}

// warp (row, touched block, kv head, keys or values): E codes a lane and store of 16 bytes, so that
// every store of the warp is one contiguous run
template <int HD, int ST>
__global__ void __launch_bounds__(kQThreads)
    qcache_read_kernel(const QCacheView c, const QRows r, void* k, void* v, int64_t stride, int span) {
  constexpr int E = kE<ST>, QR = HD / E, NQ = (kQBlock * QR + 31) / 32;
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);  // (below 2^31: the host refuses more)
  const int side = (int)(w & 1);
  const uint32_t bj = (w >> 1) / (uint32_t)c.kv;
  const int h = (int)((w >> 1) - bj * (uint32_t)c.kv), b = (int)(bj / (uint32_t)span), j = (int)bj - b * span;
  if (b >= r.B) return;
  const int p0 = r.first[b], n = q_count(r, b);
  if (n == 0) return;
  if (p0 < 0 || p0 > r.limit - n) {
    q_report(r.status, kErrPosRange);
    return;
  }
  const int blk = p0 / kQBlock + j;
  const int lo = max(p0, blk * kQBlock), hi = min(p0 + n, (blk + 1) * kQBlock);
  if (lo >= hi) return;
  int row, pp;
  if (!q_place(r, c, b, blk * kQBlock, row, pp)) return;
  const size_t head = (size_t)row * c.kv + h;
  const uint8_t* codes = (side ? c.v : c.k) + (head * c.cap + pp + lo - blk * kQBlock) * HD;
  const float s = (side ? c.vs : c.ks)[head * (c.cap / kQBlock) + pp / kQBlock];
  const int64_t base = ((int64_t)b * r.S + (lo - p0)) * stride + (int64_t)h * HD;
  const int nq = (hi - lo) * QR;
  uint2 x[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int q = lane + 32 * i;
    x[i] = make_uint2(0u, 0u);
    if (q < nq) {
      if constexpr (ST) x[i] = reinterpret_cast<const uint2*>(codes)[q];
      else x[i].x = reinterpret_cast<const uint32_t*>(codes)[q];
    }
  }
  void* dst = side ? v : k;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int q = lane + 32 * i;
    if (q >= nq) break;
    const int64_t o = base + (int64_t)(q / QR) * stride + (q % QR) * E;
    float4 f = e4m3_quad(x[i].x);
    f.x *= s; f.y *= s; f.z *= s; f.w *= s;
    if constexpr (ST == 0) {
      *reinterpret_cast<float4*>(static_cast<float*>(dst) + o) = f;
    } else {
      float4 g = e4m3_quad(x[i].y);
      g.x *= s; g.y *= s; g.z *= s; g.w *= s;
      // (codes hold four significant bits: rounding to bf16 changes only values below 2^-126)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + o) =
          make_uint4(bf16x2(f.x, f.y), bf16x2(f.z, f.w), bf16x2(g.x, g.y), bf16x2(g.z, g.w));
    }
  }
}

// a thread per (layer, kv head): the scales of one block of a cache row to 0, so that nothing of what the
// block held counts for a write that starts behind its first position
__global__ void __launch_bounds__(kQThreads)
    qcache_clear_kernel(float* ks, float* vs, int n, int rows, int kv, int blocks, int row, int blk) {
  const int i = blockIdx.x * kQThreads + threadIdx.x;
  if (i >= n) return;
  const int l = i / kv, j = i - l * kv;
  const size_t at = (((size_t)l * rows + row) * kv + j) * blocks + blk;
  ks[at] = 0.f;
  vs[at] = 0.f;
}

// calls f with the head size and the element type as compile-time numbers
template <class F>
cudaError_t with_shape(int hd, int st, F f) {
#define LLM_CASE(HD) \
  case HD: return st ? f(std::integral_constant<int, HD>{}, std::integral_constant<int, 1>{}) \
                     : f(std::integral_constant<int, HD>{}, std::integral_constant<int, 0>{});
  switch (hd) {
    LLM_CASE(16)
    LLM_CASE(32)
    LLM_CASE(64)
    LLM_CASE(128)
    LLM_CASE(256)
    default: return cudaErrorInvalidValue;
  }
#undef LLM_CASE
}

}  // namespace

bool qcache_head_supported(int hd) { return hd == 16 || hd == 32 || hd == 64 || hd == 128 || hd == 256; }

cudaError_t launch_qcache_write(const QCacheView& c, const QRows& r, const void* k, const void* v, int st,
                                int64_t stride, cudaStream_t s) {
  const int span = q_span(r.S);
  const int64_t grid = ((int64_t)r.B * span * c.kv * 2 + kQThreads / 32 - 1) / (kQThreads / 32);
  return with_shape(c.hd, st, [&](auto hd, auto t) {
    qcache_write_kernel<hd.value, t.value><<<(unsigned)grid, kQThreads, 0, s>>>(c, r, k, v, stride, span);
    return cudaGetLastError();
  });
}

cudaError_t launch_qcache_clear(const QCacheView& c, int layers, int row, int blk, cudaStream_t s) {
  const int n = layers * c.kv;
  qcache_clear_kernel<<<(n + kQThreads - 1) / kQThreads, kQThreads, 0, s>>>(c.ks, c.vs, n, c.rows, c.kv,
                                                                            c.cap / kQBlock, row, blk);
  return cudaGetLastError();
}

cudaError_t launch_qcache_keep(const QVerify& v, cudaStream_t s) {
  qcache_keep_kernel<<<dim3((unsigned)(v.layers * v.c.kv), (unsigned)v.r.B), kQThreads, 0, s>>>(v);
  return cudaGetLastError();
}

cudaError_t launch_qcache_settle(const QVerify& v, int st, cudaStream_t s) {
  const int64_t grid = ((int64_t)v.layers * v.r.B * v.c.kv * 2 + kQThreads / 32 - 1) / (kQThreads / 32);
  return with_shape(v.c.hd, st, [&](auto hd, auto t) {
    qcache_settle_kernel<hd.value, t.value><<<(unsigned)grid, kQThreads, 0, s>>>(v);
    return cudaGetLastError();
  });
}

cudaError_t launch_qcache_write_step(const QCacheView& c, const QRows& r, const void* k, const void* v, int st,
                                     cudaStream_t s, bool pdl) {
  const int64_t grid = ((int64_t)r.B * c.kv * 2 + kQThreads / 32 - 1) / (kQThreads / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kQThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return with_shape(c.hd, st, [&](auto hd, auto t) {
    return cudaLaunchKernelEx(&cfg, qcache_write_step_kernel<hd.value, t.value>, c, r, k, v);
  });
}

cudaError_t launch_qcache_read(const QCacheView& c, const QRows& r, void* k, void* v, int st, int64_t stride,
                               cudaStream_t s) {
  const int span = q_span(r.S);
  const int64_t grid = ((int64_t)r.B * span * c.kv * 2 + kQThreads / 32 - 1) / (kQThreads / 32);
  return with_shape(c.hd, st, [&](auto hd, auto t) {
    qcache_read_kernel<hd.value, t.value><<<(unsigned)grid, kQThreads, 0, s>>>(c, r, k, v, stride, span);
    return cudaGetLastError();
  });
}

}  // namespace llm
