// The norm over a list of gradient tensors and their scaling (lr_grad_norm / lr_grad_clip):
//     norm = sqrt(sum_i sum_j g_ij^2),  scale = min(1, max_norm / (norm + 1e-6)),  out_i = scale g_i.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace lr {

constexpr int kGradTable = 1024;  // most tensors of one launch
constexpr int kGradChunk = 8192;  // elements a block takes at a time (32 a thread)
constexpr int kGradParts = 4096;  // most blocks of one launch, each writing one partial sum
constexpr int kGradFew = 512;     // partial sums that the scaling blocks add up themselves

// The tensors of one launch, passed by value with it (no host-to-device copy, so a call can be captured).
// Tensor i is cut into chunks first[i] .. first[i + 1] - 1; a block takes `each` consecutive ones.
template <int N>
struct GradTable {
  const void* src[N];
  void* dst[N];
  long long numel[N];
  int first[N + 1];
  int n, each;
};

// What becomes of the sums: norm -> stat[0], scale -> stat[1] unless it has only been asked for the norm.
struct GradStat {
  const double* part;  // nparts partial sums, or nparts = 0: stat already holds the results
  int nparts;
  float max_norm;
  float* stat;
  bool norm_only;
};

// part[0 .. blocks - 1]: sums of squares in fp64, one for every `each` chunks.
inline int grad_blocks(int chunks, int each) { return (chunks + each - 1) / each; }
template <typename ST, int N>
cudaError_t launch_grad_sumsq(const GradTable<N>& tab, double* part, cudaStream_t st);
// norm and scale from any number of partial sums, by one block.
cudaError_t launch_grad_stat(const GradStat& gs, cudaStream_t st);
// The tensors scaled; with gs.nparts > 0 every block first adds the partial sums up, and the first writes stat.
template <typename ST, int N>
cudaError_t launch_grad_scale(const GradTable<N>& tab, const GradStat& gs, bool in_place, cudaStream_t st);

}  // namespace lr
