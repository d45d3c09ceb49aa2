// The norm over a list of gradient tensors and their scaling (lr_grad_norm / lr_grad_clip):
//     norm = sqrt(sum_i sum_j g_ij^2),  scale = min(1, max_norm / (norm + 1e-6)),  out_i = scale g_i.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace lr {

constexpr int kGradTable = 1024;  // tensors of one launch
constexpr int kGradChunk = 8192;  // elements one block takes at a time
constexpr int kGradParts = 1216;  // most blocks of one launch, each writing one partial sum

// The tensors of one launch, passed by value with it (no host-to-device copy, so a call can be captured).
// Tensor i is cut into chunks first[i] .. first[i + 1] - 1.
template <int N>
struct GradTable {
  const void* src[N];
  void* dst[N];
  long long numel[N];
  int first[N + 1];
  int n;
};

// part[0 .. blocks - 1]: sums of squares in fp64.  blocks = grad_blocks(chunks).
int grad_blocks(int chunks);
template <typename ST, int N>
cudaError_t launch_grad_sumsq(const GradTable<N>& tab, double* part, cudaStream_t st);
// norm and scale from the nparts partials: stat[0] = norm if write_stat > 0, stat[1] = scale if write_stat > 1;
// then the tensors of `tab` scaled (none if tab.n == 0).
template <typename ST, int N>
cudaError_t launch_grad_scale(const GradTable<N>& tab, const double* part, int nparts, float max_norm, float* stat,
                              int write_stat, cudaStream_t st);

}  // namespace lr
