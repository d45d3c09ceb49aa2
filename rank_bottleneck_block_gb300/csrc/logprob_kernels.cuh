// Log probabilities of given tokens, entropy and most probable tokens of each row of logits, and their gradient
// (lr_logprob_fwd / lr_logprob_bwd).  Of any part of a row, with c = scale log2(e) and x its logits,
//     m = max x,  s = sum 2^d,  w = sum 2^d d,  d_j = c (x_j - m);
// two parts join by scaling both to the larger m (with e = c (m - m'): s' = 2^e s, w' = 2^e (w + s e)), and of the row
//     lse = scale m + ln 2 log2 s,  logp = scale (x_target - m) - ln 2 log2 s,  entropy = ln 2 (log2 s - w / s):
// differences to the maximum throughout, so neither logp nor the entropy loses digits to the size of the logits, and
// logits of the type's lowest value do not leave the range.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace lr {

constexpr int kLogprobMaxTop = 32;
constexpr int kLogprobMaxV = 1 << 19;
constexpr int kLogprobMaxSplits = 64;
constexpr int kLogprobSeg = 256;

// How a forward cuts its rows.
struct LogprobPlan {
  int nseg;    // segments of kLogprobSeg logits per row, whose maxima are kept (top > 0)
  int splits;  // blocks per row, of
  int chunk;   // this many logits each, a multiple of 1024
};
LogprobPlan logprob_plan(int T, int V, int es, int sms);

struct LogprobFwd {
  const void* logits;
  long long ld;
  const int* target;
  float *logp, *entropy, *lse;
  int* top_ids;
  float* top_logp;
  float4* part;  // [T, splits]: m, s, w (splits > 1 or top > 0)
  float* segmax;  // [T, nseg] (top > 0)
  int T, V, top;
  float scale;
};
template <typename ST>
cudaError_t launch_logprob_fwd(const LogprobFwd& a, const LogprobPlan& plan, cudaStream_t st);
// Whether the forward takes a second launch, which joins the parts of each row and finds its largest logits ...
inline bool logprob_joins(const LogprobPlan& plan, int top) { return plan.splits > 1 || top > 0; }
template <typename ST>
cudaError_t launch_logprob_join(const LogprobFwd& a, const LogprobPlan& plan, cudaStream_t st);

struct LogprobBwd {
  const void* logits;
  long long ld;
  const int* target;
  const float *lse, *entropy, *dlogp, *dentropy;  // entropy, dentropy may be null together
  void* out;
  long long ldo;
  int T, V;
  float scale;
};
template <typename ST>
cudaError_t launch_logprob_bwd(const LogprobBwd& a, int sms, cudaStream_t st);

}  // namespace lr
