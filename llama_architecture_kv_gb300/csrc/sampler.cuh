// Greedy and temperature / top-k / top-p sampling (declarations).
#pragma once
#include "common.cuh"

namespace llm {

struct SampleArgs {
  const float* logits;   // [B][logits_stride]
  int32_t logits_stride;
  int32_t V;
  int32_t V_pad;         // row pitch of the scratch arrays
  uint32_t* keys;        // scratch [B][2][V_pad]
  int32_t* idx;          // scratch [B][2][V_pad]
  float* pre;            // scratch [B][V_pad]: weights, then their running sums
  uint32_t* hist;        // scratch [B][digits][sample_slices(V)]: digit counts, then offsets, per CTA slice
  size_t hist_per_row;   // uint32 entries of hist per row: 256 digits (8-bit) need 256 * slices
  const float* u;        // [B] uniform draws
  int32_t* ids;          // [B] drawn ids
  const StepState* step; // temp, k, p
};

// exp(x) as a fixed sequence of IEEE operations (sampler.cu)
LLM_D float exp_s(float x) {
  if (x != x) return x;
  if (x > 88.5f) return INFINITY;
  if (x < -104.0f) return 0.0f;
  const float LOG2E = 1.44269504088896340736f;
  const float LN2_HI = 0.693145751953125f;  // ln 2 to 16 significant bits: n * LN2_HI is exact
  const float LN2_LO = (float)(0.69314718055994530942 - 0.693145751953125);
  const float nf = rintf(__fmul_rn(x, LOG2E));
  const int n = (int)nf;
  float r = __fmaf_rn(-nf, LN2_HI, x);
  r = __fmaf_rn(-nf, LN2_LO, r);
  float p = (float)(1.0 / 40320.0);
  p = __fmaf_rn(p, r, (float)(1.0 / 5040.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 720.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 120.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 24.0));
  p = __fmaf_rn(p, r, (float)(1.0 / 6.0));
  p = __fmaf_rn(p, r, 0.5f);
  p = __fmaf_rn(p, r, 1.0f);
  p = __fmaf_rn(p, r, 1.0f);
  if (n >= -126) return __fmul_rn(p, __uint_as_float((uint32_t)(n + 127) << 23));
  return __fmul_rn(__fmul_rn(p, __uint_as_float((uint32_t)(n + 64 + 127) << 23)),
                   __uint_as_float((uint32_t)(-64 + 127) << 23));
}

constexpr int kSortMaxSlicesPerRow = 64;
constexpr size_t kSampleHistPerRow = 256 * kSortMaxSlicesPerRow;  // uint32 entries a row needs at most (8-bit digits)

int sample_slices(int V);
// greedy: one argmax kernel; select (top-k with k <= sample_select_max()): one radix-select
// kernel per row; otherwise the sort chain and the draw (temp, k, p from *step)
cudaError_t launch_sample(const SampleArgs& a, int B, bool greedy, cudaStream_t s, bool pdl, bool select = false);
int sample_select_max();
// One token per row, every row with its own settings (sample_rows.cu); null arrays: 1 (temp), V (k), 1 (p), 0 (min_p)
struct SampleRowsArgs {
  const float* logits;  // [B] rows of V, `stride` apart
  int64_t stride;
  int32_t B, V;
  const float* temp;
  const int32_t* k;
  const float *p, *min_p, *u;
  int32_t* ids;
  int32_t* status;
};
constexpr int kSampleRowsMost = 8 * 65535;  // ids of a row
cudaError_t launch_sample_rows(const SampleRowsArgs& a, cudaStream_t s);
// loads the allocation-free sampler's fixed array on the current device and records its address
cudaError_t noalloc_prepare();

}  // namespace llm
