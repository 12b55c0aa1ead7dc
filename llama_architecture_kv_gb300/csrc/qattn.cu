// Grouped-query attention over an 8-bit cache (qcache.cuh).
//
// Token i of row b (its query heads h = j*g + n read key/value head j) attends to the positions
// start <= t < end of its row, end = length - count + i + 1:
//   o_h = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q_h . k_t - max),  k_t, v_t = code * block scale.
// A token that no position is visible to gets zeros.
//
// Head sizes 64 and 128 run on the tensor cores (qattn_tc.cuh: 32 rows of up to 2100 positions, 8 heads
// of 128, groups of 4, in 34 us, against 170 us with the kernel here).  qattn_simple_kernel takes the
// others (16, 32, 256; on the tensor cores they would take other tiles: a 32-byte swizzle and value products of
// 64 rows for 32, two boxes a row and two value products for 256): a CTA of four warps takes one token, one key/value head and one contiguous part of the positions.  Each warp takes 32 positions at a
// time: lane = position for the scores of the group's heads (the codes widened to f32, the scale applied
// to the dot product once), a warp-wide running maximum and sum per head, then lane = dimensions for the
// values.  Statistics, weights and sums are f32.  The parts of a token meet in qattn_merge_kernel in their
// order, so the result does not depend on timing.  Bound by its arithmetic (each code is widened and
// multiplied on the CUDA cores): GB300, 8 rows of 4096 positions, 37 us with 8 heads of 32 and groups of 4,
// 93 us with 4 heads of 256 and groups of 2.
#include <algorithm>
#include <type_traits>

#include "attention.cuh"
#include "gemm.cuh"
#include "qattn_tc.cuh"
#include "qcache.cuh"

namespace llm {

namespace {

constexpr int kSimpleThreads = 128;
constexpr int kSimpleSplits = 32;  // most parts of one token's positions

template <int QT>
LLM_D float load_q(const void* q, int64_t i) {
  return QT ? bf16_to_f32(static_cast<const uint16_t*>(q)[i]) : static_cast<const float*>(q)[i];
}
template <int QT>
LLM_D void store_o(void* o, int64_t i, float v) {
  if constexpr (QT) static_cast<uint16_t*>(o)[i] = f32_to_bf16(v);
  else static_cast<float*>(o)[i] = v;
}

// positions [start, end) of token t of a call (t = b * S + i; of a step: of its row b, the entry whose place the
// token's positions and rows of q and out have); false: the token is not there
LLM_D bool token_range(const QRows& r, int t, int& b, int& start, int& end) {
  start = 0;
  if (r.step) {
    b = q_entry(r, t);
    start = row_start(r.step, b);
    end = row_pos(r.step, b) + 1;
    return true;
  }
  b = t / r.S;
  const int i = t - b * r.S, n = q_count(r, b);
  if (i >= n) return false;
  int len = r.first[b];
  if (len < 0 || len > r.limit) {
    q_report(r.status, kErrPosRange);
    len = 0;
  }
  end = max(0, len - n + i + 1);
  return true;
}

LLM_D bool token_place(const QRows& r, const QCacheView& c, int b, int pos, int& row, int& pp) {
  if (!r.step) return q_place(r, c, b, pos, row, pp);
  cache_slot(r.step, c.cap, b, pos, row, pp);
  return true;
}

// HD: head size; GM: bound of the group size; QT: 0 f32, 1 bf16 queries and outputs
template <int HD, int GM, int QT>
__global__ void __launch_bounds__(kSimpleThreads) qattn_simple_kernel(const QAttnArgs a) {
  constexpr int NW = kSimpleThreads / 32;
  constexpr int DPL = HD >= 32 ? HD / 32 : 1;  // dimensions per lane of the values
  grid_dep_wait();
  grid_dep_launch();
  const int split = blockIdx.x, j = blockIdx.y;
  const int g = a.g, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ __align__(16) float qs[GM * HD];
  __shared__ __align__(16) float wb[NW][32 * GM];
  __shared__ float part[NW][GM * (HD + 2)];
  for (int64_t t64 = blockIdx.z; t64 < (int64_t)a.r.B * a.r.S; t64 += gridDim.z) {
    const int t = (int)t64;
    int b, start, end;
    if (!token_range(a.r, t, b, start, end)) continue;
    const int64_t qrow = a.r.step ? b : t64;
    // this part's positions: a whole number of 32-position chunks, aligned so that none crosses a page
    const int base = start & ~31;
    const int nch = end > start ? (end - base + 31) / 32 : 0;
    const int c0 = (int)((int64_t)nch * split / a.splits), c1 = (int)((int64_t)nch * (split + 1) / a.splits);
    __syncthreads();  // the previous token's shared memory is free
    for (int i = tid; i < g * HD; i += kSimpleThreads)
      qs[i] = load_q<QT>(a.q, qrow * a.q_stride + (int64_t)j * g * HD + i);
    __syncthreads();
    float m[GM], l[GM], o[GM][DPL];
#pragma unroll
    for (int h = 0; h < GM; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < DPL; ++e) o[h][e] = 0.f;
    }
    for (int ch = c0 + warp; ch < c1; ch += NW) {
      const int pb = base + ch * 32;
      int row, pp;
      if (!token_place(a.r, a.c, b, pb, row, pp)) continue;
      const size_t head = (size_t)row * a.c.kv + j;
      const uint8_t* kp = a.c.k + (head * a.c.cap + pp) * HD;
      const uint8_t* vp = a.c.v + (head * a.c.cap + pp) * HD;
      const int lo = max(0, start - pb), hi = min(32, end - pb);
      const bool seen = lane >= lo && lane < hi;
      float acc[GM];
#pragma unroll
      for (int h = 0; h < GM; ++h) acc[h] = 0.f;
      float ks = 0.f, vs = 0.f;
      if (seen) {
        const size_t sc = head * (a.c.cap / kQBlock) + (pp + lane) / kQBlock;
        ks = a.c.ks[sc] * a.scale;
        vs = a.c.vs[sc];
#pragma unroll
        for (int e = 0; e < HD / 16; ++e) {
          const uint4 u = *reinterpret_cast<const uint4*>(kp + (size_t)lane * HD + e * 16);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 k4 = e4m3_quad(w[i]);
#pragma unroll
            for (int h = 0; h < GM; ++h)
              if (h < g) {
                const float4 q4 = *reinterpret_cast<const float4*>(qs + h * HD + e * 16 + 4 * i);
                acc[h] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, acc[h]))));
              }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < GM; ++h)
        if (h < g) {
          const float s = seen ? acc[h] * ks : -INFINITY;
          const float mn = fmaxf(m[h], warp_max(s));
          const float corr = m[h] == -INFINITY ? 0.f : expf(m[h] - mn);
          const float w = seen ? expf(s - mn) : 0.f;
          m[h] = mn;
          l[h] = fmaf(l[h], corr, w);
#pragma unroll
          for (int e = 0; e < DPL; ++e) o[h][e] *= corr;
          wb[warp][lane * GM + h] = seen ? w * vs : 0.f;  // the value's scale rides on its weight
        }
      __syncwarp();
      if (lane * DPL < HD) {
        for (int p = lo; p < hi; ++p) {
          float v[DPL];
          const uint8_t* src = vp + (size_t)p * HD + lane * DPL;
          if constexpr (DPL == 1) {
            v[0] = e4m3_pair(*src).x;
          } else if constexpr (DPL == 2) {
            const float2 f = e4m3_pair(*reinterpret_cast<const uint16_t*>(src));
            v[0] = f.x;
            v[1] = f.y;
          } else {
#pragma unroll
            for (int e = 0; e < DPL; e += 4) {
              const float4 f = e4m3_quad(*reinterpret_cast<const uint32_t*>(src + e));
              v[e] = f.x; v[e + 1] = f.y; v[e + 2] = f.z; v[e + 3] = f.w;
            }
          }
#pragma unroll
          for (int h = 0; h < GM; ++h)
            if (h < g)
#pragma unroll
              for (int e = 0; e < DPL; ++e) o[h][e] = fmaf(wb[warp][p * GM + h], v[e], o[h][e]);
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int h = 0; h < GM; ++h)
      if (h < g) {
        const float ls = warp_sum(l[h]);
        if (lane * DPL < HD)
#pragma unroll
          for (int e = 0; e < DPL; ++e) part[warp][h * (HD + 2) + lane * DPL + e] = o[h][e];
        if (lane == 0) {
          part[warp][h * (HD + 2) + HD] = m[h];
          part[warp][h * (HD + 2) + HD + 1] = ls;
        }
      }
    __syncthreads();
    for (int i = tid; i < g * HD; i += kSimpleThreads) {
      const int h = i / HD, e = i - h * HD;
      float M = -INFINITY, O = 0.f, L = 0.f;
      for (int w = 0; w < NW; ++w) M = fmaxf(M, part[w][h * (HD + 2) + HD]);
      for (int w = 0; w < NW; ++w) {
        const float mw = part[w][h * (HD + 2) + HD], lw = part[w][h * (HD + 2) + HD + 1];
        // (a part whose every score is NaN has no maximum, and a NaN sum that has to stay)
        const float f = mw == -INFINITY ? (lw == 0.f ? 0.f : 1.f) : expf(mw - M);
        O = fmaf(f, part[w][h * (HD + 2) + e], O);
        L = fmaf(f, lw, L);
      }
      const int head = j * g + h;
      if (a.splits == 1) {
        store_o<QT>(a.out, qrow * a.out_stride + (int64_t)head * HD + e, L == 0.f ? 0.f : O / L);
      } else {
        float* dst = reinterpret_cast<float*>(a.ws + kQattnTickets) + ((t64 * a.c.kv * g + head) * a.splits + split) * (HD + 2);
        dst[e] = O;
        if (e == 0) {
          dst[HD] = M;
          dst[HD + 1] = L;
        }
      }
    }
  }
}

// the parts of one (token, head) in their order; CTA (head, token), one thread per dimension
template <int QT>
__global__ void qattn_merge_kernel(const QAttnArgs a) {
  const int HD = a.c.hd, H = a.c.kv * a.g, head = blockIdx.x, e = threadIdx.x;
  for (int64_t t = blockIdx.y; t < (int64_t)a.r.B * a.r.S; t += gridDim.y) {
    int b, start, end;
    if (!token_range(a.r, (int)t, b, start, end)) continue;
    const float* src = reinterpret_cast<const float*>(a.ws + kQattnTickets) + (t * H + head) * a.splits * (HD + 2);
    float M = -INFINITY, O = 0.f, L = 0.f;
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, src[s * (HD + 2) + HD]);
    for (int s = 0; s < a.splits; ++s) {
      const float ms = src[s * (HD + 2) + HD], ls = src[s * (HD + 2) + HD + 1];
      const float f = ms == -INFINITY ? (ls == 0.f ? 0.f : 1.f) : expf(ms - M);
      O = fmaf(f, src[s * (HD + 2) + e], O);
      L = fmaf(f, ls, L);
    }
    store_o<QT>(a.out, (a.r.step ? b : t) * a.out_stride + (int64_t)head * HD + e, L == 0.f ? 0.f : O / L);
  }
}

// parts per token: about two CTAs per SM, none of fewer than 128 positions
int simple_splits(const QCacheView& c, int64_t tokens, int limit, int num_sms) {
  const int64_t units = tokens * c.kv;
  const int64_t want = (2 * num_sms + units - 1) / units;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, kSimpleSplits, limit / 128}));
}

template <int HD, int QT>
cudaError_t launch_simple(const QAttnArgs& a0, int num_sms, cudaStream_t s, bool pdl) {
  QAttnArgs a = a0;
  const int64_t tokens = (int64_t)a.r.B * a.r.S;
  a.splits = simple_splits(a.c, tokens, std::min(a.r.limit, a.c.rows * a.c.cap), num_sms);
  void (*fn)(const QAttnArgs) = nullptr;
  if (a.g <= 4) fn = qattn_simple_kernel<HD, 4, QT>;
  else if constexpr (HD <= 128) {
    if (a.g <= 8) fn = qattn_simple_kernel<HD, 8, QT>;
    else if constexpr (HD <= 64) fn = qattn_simple_kernel<HD, 16, QT>;
  }
  if (!fn) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.splits, a.c.kv, (unsigned)std::min<int64_t>(tokens, 65535));
  cfg.blockDim = dim3(kSimpleThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a);
  if (e != cudaSuccess || a.splits == 1) return e;
  qattn_merge_kernel<QT><<<dim3(a.c.kv * a.g, (unsigned)std::min<int64_t>(tokens, 65535)), HD, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

namespace {

// the tensor-core kernel's tiles: 16 nc accumulator columns of np pieces, the smallest that holds all
// of a row's (token, head) columns, else the largest: a tile's cost grows with its columns (five tokens of
// a group of four in each of 32 rows of 2048 positions: 69 us with 24 columns, 74 us with 32), and every
// further tile reads the codes again
int64_t q_tiles_of(int limit) { return ((int64_t)limit + kQaTile - 1) / kQaTile; }
struct TcPlanQ {
  int nc, cols, tokens, grid;
};
TcPlanQ plan_tc_q(const QCacheView& c, int g, int qt, int64_t rows, int64_t S, int limit, int num_sms) {
  const int np = qt ? 2 : 4, most = qt ? 4 : 8;
  TcPlanQ p;
  p.nc = 1;
  // (f32: 1, 2, 4, 6 or 8; bf16: 1, 2 or 4)
  while (p.nc < most && p.nc * 16 / np < S * g) p.nc = p.nc < 4 ? p.nc * 2 : p.nc + 2;
  p.cols = p.nc * 16 / np;
  p.tokens = p.cols / g;
  const int64_t units = rows * ((S + p.tokens - 1) / p.tokens) * c.kv;
  const int64_t tiles = units * q_tiles_of(limit);
  const int64_t ctas = std::min(num_sms * (p.cols <= 8 ? 2 : 1), kQattnTickets / 4);
  p.grid = (int)std::max<int64_t>(1, std::min(tiles, ctas));
  return p;
}

}  // namespace

bool qattn_uses_tc(int hd) { return hd == 64 || hd == 128; }
int qattn_tile_tokens(int g) { return 32 / g; }

bool qattn_make_map(CUtensorMap* map, const void* codes, int hd, uint64_t rows) {
  return make_map_2d(map, codes, 1, (uint64_t)hd, rows, (uint32_t)hd, 64,
                     hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

bool qattn_fits(const QCacheView& c, int g, int qt, int B, int S, int limit, int num_sms) {
  if (!qattn_uses_tc(c.hd)) return true;
  const TcPlanQ p = plan_tc_q(c, g, qt, B, S, limit, num_sms);
  return (double)B * (((int64_t)S + p.tokens - 1) / p.tokens) * c.kv * q_tiles_of(limit) < 2147483648.0;
}

uint64_t qattn_workspace(const QCacheView& c, int g, int B, int S, int num_sms) {
  const int64_t tokens = (int64_t)B * S;
  const int limit = c.rows * c.cap;
  if (qattn_uses_tc(c.hd)) {
    uint64_t most = 0;
    for (int qt = 0; qt < 2; ++qt) {
      const TcPlanQ p = plan_tc_q(c, g, qt, B, S, limit, num_sms);
      most = std::max(most, (uint64_t)p.grid * 2 * p.cols * (c.hd + 2) * 4);
    }
    return kQattnTickets + most;
  }
  const int splits = simple_splits(c, tokens, limit, num_sms);
  return splits == 1 ? 0 : kQattnTickets + (uint64_t)tokens * c.kv * g * splits * (c.hd + 2) * 4;
}

uint64_t qattn_step_workspace(const QCacheView& c, int g, int NT, int num_sms) {
  uint64_t most = 0;
  for (int b = 1; b <= NT; ++b) most = std::max(most, qattn_workspace(c, g, b, 1, num_sms));
  if (qattn_uses_tc(c.hd)) most = std::max(most, qattn_workspace(c, g, NT, qattn_tile_tokens(g), num_sms));
  return most;
}

cudaError_t launch_qattn(const QAttnArgs& a0, int qt, int num_sms, cudaStream_t s, bool pdl, const CUtensorMap* kmap,
                         const CUtensorMap* vmap) {
  QAttnArgs a = a0;
  if (qattn_uses_tc(a.c.hd)) {
    CUtensorMap maps[2];
    if (!kmap) {
      const uint64_t rows = (uint64_t)a.c.rows * a.c.kv * a.c.cap;
      if (!qattn_make_map(&maps[0], a.c.k, a.c.hd, rows) || !qattn_make_map(&maps[1], a.c.v, a.c.hd, rows))
        return cudaErrorInvalidValue;
      kmap = &maps[0];
      vmap = &maps[1];
    }
    const int S = a.tiles ? qattn_tile_tokens(a.g) : a.r.S;  // (a tile is a row of its own)
    // (a page table can name a page more than once: rows longer than the pool get no more CTAs)
    const TcPlanQ p = plan_tc_q(a.c, a.g, qt, a.r.B, S, std::min(a.r.limit, a.c.rows * a.c.cap), num_sms);
    a.tpt = p.tokens;
    a.nct = a.r.step ? 1 : (int)(((int64_t)a.r.S + p.tokens - 1) / p.tokens);
    const bool wide = p.nc > 4;
    auto fn = a.c.hd == 64 ? (qt ? qattn_tc64_bf16 : wide ? qattn_tc64_f32_wide : qattn_tc64_f32)
                           : (qt ? qattn_tc128_bf16 : wide ? qattn_tc128_f32_wide : qattn_tc128_f32);
    return fn(*kmap, *vmap, a, p.nc, p.grid, s, pdl);
  }
  switch (a.c.hd) {
    case 16: return qt ? launch_simple<16, 1>(a, num_sms, s, pdl) : launch_simple<16, 0>(a, num_sms, s, pdl);
    case 32: return qt ? launch_simple<32, 1>(a, num_sms, s, pdl) : launch_simple<32, 0>(a, num_sms, s, pdl);
    case 256: return qt ? launch_simple<256, 1>(a, num_sms, s, pdl) : launch_simple<256, 0>(a, num_sms, s, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace llm
