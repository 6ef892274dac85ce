// Interface between the linear attention entry points (srnl_lattn.cu) and the passes, on the tensor
// cores (srnl_lattn_tc.cu) and for a few tokens (srnl_lattn_short.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace srnl {

// A decayed pass over rows a, b, c of every token (see srnl_lattn.cu).
struct LaPass {
  const __nv_bfloat16 *a, *b, *c;
  __nv_bfloat16* out;
  int64_t lda, ldb, ldc, ldo;   // elements between tokens
  const float* z0;              // [B][heads][D][D] or nullptr
  float* zn;                    // final state or nullptr
  int z0_t;                     // z0 is the transpose of Z
  int reverse;                  // tokens from the last to the first; z0 enters undecayed, zn leaves decayed once more
};

struct LaArgs {
  LaPass pass[3];
  int passes, B, T, heads, d, segs, seg_len;   // segments of seg_len tokens per sequence
  const float* log2g;                       // [heads]
  const int* lengths;                       // [B] or nullptr
  int longest_first;                        // CTAs take the longest sequences first
  float* seg_state;                         // [pass][B][heads][segs][D][D]: what each segment adds, then its start
  int* err;
};

// CTAs that a sequence's heads take (two heads of up to 64 channels share one).
int la_groups(int heads, int d);
// Segments per sequence for that many sequences x groups: one when they fill the GPU by themselves.
int la_tc_segments(int T, int seqs, int sms);
cudaError_t launch_la_tc(LaArgs& a, int sms, cudaStream_t s);
cudaError_t prepare_la_tc(int d);
// The same passes over at most kShortTokens tokens (srnl_lattn_short.cu).
constexpr int kShortTokens = 16;
cudaError_t launch_la_short(const LaArgs& a, cudaStream_t s);

}  // namespace srnl
