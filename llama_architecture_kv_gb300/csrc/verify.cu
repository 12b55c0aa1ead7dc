// Verification of drafted tokens against the target model's probabilities (speculative sampling).
//
// Row b brings n drafts x_0 .. x_{n-1}, the target's probabilities p_0 .. p_n after each of them,
// the draft model's q_0 .. q_{n-1} (or none: a deterministic draft, q_i(x_i) = 1) and draws u.
//   draft i is kept while u_i q_i(x_i) < p_i(x_i);
//   after r kept drafts one more token is drawn with u_S from the weights
//     w = max(p_r - q_r, 0)  (r < n; without q: p_r with x_r left out),  w = p_n  (r = n),
// so the tokens are distributed as if the target had drawn them one by one.
//
// The products u q are exact in f64 and the weights are whole multiples of 2^-61 (p - q is one f32
// subtraction; an f32 of at least 2^-38 is such a multiple), so every sum is an exact 64-bit integer
// whatever its order: the drawn token is that of a sequential walk over the row, on any split.
//
// Bound: the two rows of V floats that the last token is drawn from (everything else is a few
// scalars), and for a few rows the chain of dependent loads: drafts, their probabilities, the rows.  A
// cluster of 8 CTAs shares a row, since one SM's loads would need about 10 us for 1 MB: each warp sums
// one contiguous stretch with coalesced loads, the stretches' sums meet through distributed shared
// memory behind one cluster barrier, and the warp whose stretch holds the draw reads it again from L2 in
// two rounds (in rounds of 32 ids it took 11 us).  Loads of one id per lane do for rows of any alignment
// (16-byte loads of aligned rows measured the same), and short loops: unrolled 16 times the sum was
// slower, waiting for its own instructions.  GB300: 5.9 us for one row of 49152 ids, 15.1 us for 32 rows
// of 128256 with q (33 MB: 2.2 TB/s; the chain and the launch are 6 us of it).
#include "verify.cuh"

namespace llm {

namespace {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerCluster = 8;

LLM_D uint32_t ver_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
LLM_D void ver_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
LLM_D uint64_t ver_remote(const uint64_t* p, uint32_t rank) {
  uint32_t local = (uint32_t)__cvta_generic_to_shared(p), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
  return v;
}

// a weight in units of 2^-61 (NaN and negative values weigh nothing)
LLM_D uint64_t ver_units(float w) {
  // w 2^61 = its 24-bit significand shifted: w = s 2^(e - 150)
  const uint32_t u = __float_as_uint(w > 0.0f ? fminf(w, 1.0f) : 0.0f);
  const int up = (int)(u >> 23) - (150 - 61);
  const uint64_t s = (u & 0x7fffffu) | 0x800000u;
  return up >= 0 ? s << up : up > -24 ? s >> -up : 0ull;  // (f32 subnormals are far below 2^-61)
}

struct VerRow {
  const float* p;   // [V]
  const float* q;   // [V] or null
  int skip;         // id left out, or -1
};
LLM_D uint64_t ver_weight(const VerRow& r, int v) {
  float w = r.p[v];
  if (r.q) w = __fsub_rn(w, r.q[v]);
  return v == r.skip ? 0ull : ver_units(w);
}

// a store to the same variable of another CTA of the cluster
LLM_D void ver_put(uint64_t* p, uint32_t rank, uint64_t v) {
  uint32_t local = (uint32_t)__cvta_generic_to_shared(p), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}
// a running sum over the lanes
LLM_D uint64_t ver_scan(uint64_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// cluster = row
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyArgs a) {
  __shared__ int s_r;
  __shared__ uint64_t s_warp[kVerWarps];   // sums of this CTA's stretches
  __shared__ uint64_t s_all[2][kVerCluster];  // the CTAs' sums, by attempt
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ver_rank();
  const int b = blockIdx.x / kVerCluster;
  const int S = a.S, V = a.V;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before the first store to another CTA)
  if (tid == 0) s_r = S;
  __syncthreads();
  int n = a.count ? a.count[b] : S;
  n = n < 0 ? 0 : n > S ? S : n;
  if (tid == 0) atomicMin(&s_r, n);
  for (int i = tid; i < S; i += kVerThreads) {
    const int x = a.drafts[(size_t)b * S + i];
    const float u = a.u[(size_t)b * (S + 1) + i];
    bool kept = false;
    if (x >= 0 && x < V) {
      const float p = a.p[((size_t)b * (S + 1) + i) * V + x];
      const float q = a.q ? a.q[((size_t)b * S + i) * V + x] : 1.0f;
      kept = (double)u * (double)q < (double)p;
    }
    if (!kept) atomicMin(&s_r, i);
  }
  __syncthreads();
  const int r = s_r;
  VerRow row = {a.p + ((size_t)b * (S + 1) + r) * V, nullptr, -1};
  if (r < n) {
    if (a.q) row.q = a.q + ((size_t)b * S + r) * V;
    else row.skip = a.drafts[(size_t)b * S + r];
  }
  // stretches of ids, warp by warp over the cluster
  const int per = (V + kVerCluster * kVerWarps - 1) / (kVerCluster * kVerWarps);
  const int64_t i0_ = (int64_t)((int)rank * kVerWarps + warp) * per;
  const int i0 = (int)min((int64_t)V, i0_), i1 = (int)min((int64_t)V, i0_ + per);
  int32_t* ids = a.ids + (size_t)b * (S + 1);
  // no weight at all (not a row of probabilities): id 0; the draw's owner writes over it after the
  // cluster barrier
  if (rank == 0 && tid == 0) ids[r] = 0;
  uint64_t total = 0, before = 0;
  for (int attempt = 0; attempt < 2; ++attempt) {
    uint64_t sum = 0;
#pragma unroll 4
    for (int v = i0 + lane; v < i1; v += 32) sum += ver_weight(row, v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (attempt == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA has started
    if (warp == 0) {
      uint64_t t = lane < kVerWarps ? s_warp[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane < kVerCluster) ver_put(&s_all[attempt][rank], (uint32_t)lane, t);
    }
    ver_cluster_sync();  // every sum is here; nothing is stored to another CTA after the last of these
    total = before = 0;
    for (int c = 0; c < kVerCluster; ++c) {
      if (c == (int)rank) before = total;
      total += s_all[attempt][c];
    }
    if (total > 0 || (!row.q && row.skip < 0)) break;
    // nothing left over (p <= q everywhere): the target's own probabilities
    row.q = nullptr;
    row.skip = -1;
  }
  // floor(u * 2^24) * total / 2^24, below total
  const float u = a.u[(size_t)b * (S + 1) + S];
  const uint64_t d = u > 0.0f ? (uint64_t)(min(u, 0.99999994f) * 16777216.0f) : 0ull;
  const uint64_t goal = d * (total >> 24) + ((d * (total & 0xffffffull)) >> 24);
  if (rank == 0) {
    for (int i = tid; i <= S; i += kVerThreads)
      if (i != r) ids[i] = i < r ? a.drafts[(size_t)b * S + i] : -1;
    if (tid == 0) a.accepted[b] = r;
  }
  for (int x = 0; x < warp; ++x) before += s_warp[x];
  if (goal < before || goal - before >= s_warp[warp]) return;
  // this warp's stretch holds the draw: lanes sum equal pieces of it, then the piece that holds the draw is
  // walked 32 ids at a time
  const int piece = (i1 - i0 + 31) / 32, l0 = min(i1, i0 + lane * piece), l1 = min(i1, l0 + piece);
  uint64_t part = 0;
#pragma unroll 8
  for (int v = l0; v < l1; ++v) part += ver_weight(row, v);
  const uint64_t upto = ver_scan(part);
  const int who = __ffs(__ballot_sync(0xffffffffu, before + upto > goal)) - 1;  // (one does: goal is in this stretch)
  before += __shfl_sync(0xffffffffu, upto - part, who);
  const int v0 = __shfl_sync(0xffffffffu, l0, who), v1 = __shfl_sync(0xffffffffu, l1, who);
  for (int v = v0; v < v1; v += 32) {
    const uint64_t incl = ver_scan(v + lane < v1 ? ver_weight(row, v + lane) : 0ull);
    const uint32_t above = __ballot_sync(0xffffffffu, before + incl > goal);
    if (above) {
      if (lane == 0) ids[r] = v + __ffs(above) - 1;
      return;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Logits to probabilities, a cluster of 8 CTAs per row: each CTA's slice is read once (the exponentials
// are taken in place and scaled when the row's sum is known), the maxima and sums meet through
// distributed shared memory in CTA order.  Two passes over a slice of V / 8 floats, which stays in L2.
__global__ void __launch_bounds__(kVerThreads) probs_kernel(float* x, int V, float temp) {
  __shared__ float s_v[kVerWarps];
  __shared__ int s_i[kVerWarps];
  __shared__ uint64_t s_cta, s_all[kVerCluster];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ver_rank();
  float* row = x + (size_t)(blockIdx.x / kVerCluster) * V;
  const int per = (V + kVerCluster - 1) / kVerCluster;
  const int i0 = min(V, (int)rank * per), i1 = min(V, i0 + per);
  // every CTA's value through the cluster: bits of a float, and an index
  auto share = [&](float v, int i) {
    if (tid == 0) s_cta = (uint64_t)__float_as_uint(v) << 32 | (uint32_t)i;
    ver_cluster_sync();
    if (tid < kVerCluster) s_all[tid] = ver_remote(&s_cta, (uint32_t)tid);
    ver_cluster_sync();  // (also: nobody leaves or writes its value again before all have read it)
  };
  float top = -INFINITY;
  int at = 0x7fffffff;
  for (int i = i0 + tid; i < i1; i += kVerThreads) {
    const float v = row[i];
    if (v > top) {
      top = v;
      at = i;
    }
  }
  auto better = [&](float v, int i) {
    if (v > top || (v == top && i < at)) {
      top = v;
      at = i;
    }
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, top, o);
    better(v, __shfl_xor_sync(0xffffffffu, at, o));
  }
  if (lane == 0) {
    s_v[warp] = top;
    s_i[warp] = at;
  }
  __syncthreads();
  for (int w = 0; w < kVerWarps; ++w) better(s_v[w], s_i[w]);
  share(top, at);
  for (int c = 0; c < kVerCluster; ++c) better(__uint_as_float((uint32_t)(s_all[c] >> 32)), (int)(uint32_t)s_all[c]);
  if (temp == 0.0f) {
    if (at == 0x7fffffff) at = 0;  // (no logit above -inf)
    for (int i = i0 + tid; i < i1; i += kVerThreads) row[i] = i == at ? 1.0f : 0.0f;
    return;
  }
  float sum = 0.0f;
  for (int i = i0 + tid; i < i1; i += kVerThreads) {
    const float e = expf((row[i] - top) / temp);
    row[i] = e;
    sum += e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_v[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < kVerWarps; ++w) sum += s_v[w];
  share(sum, 0);
  sum = 0.0f;
  for (int c = 0; c < kVerCluster; ++c) sum += __uint_as_float((uint32_t)(s_all[c] >> 32));
  for (int i = i0 + tid; i < i1; i += kVerThreads) row[i] /= sum;
}

template <class... P, class... A>
cudaError_t launch_cluster(void (*fn)(P...), int rows, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * kVerCluster);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kVerCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

cudaError_t launch_probs(float* x, int rows, int V, float temp, cudaStream_t s) {
  return launch_cluster(probs_kernel, rows, s, x, V, temp);
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  return launch_cluster(verify_kernel, a.B, s, a);
}

}  // namespace llm
