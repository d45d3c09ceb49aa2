// The norm over a list of gradient tensors and their scaling (lr_grad_norm / lr_grad_clip):
//     norm = sqrt(sum_i sum_j g_ij^2),  scale = min(1, max_norm / (norm + 1e-6)),  out_i = scale g_i.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace lr {

constexpr int kGradTable = 1024;        // most tensors of one launch
constexpr int kGradOwners = 256;        // entries that say where to look for a chunk's tensor
constexpr int kGradChunkBytes = 32768;  // what 256 threads take at a time (8 16-byte words each)
constexpr int kGradParts = 3040;        // most blocks of one launch that sums, each writing one partial sum
constexpr int kGradFew = 512;           // partial sums that the scaling blocks add up themselves
constexpr int kGradKeepBytes = 64 << 20;  // the last of a launch's reads, which a scaling right behind it finds in L2
constexpr int kGradSmall = 32;          // chunks that one cluster sums and scales in one launch

// The tensors of one launch, passed by value with it (no host-to-device copy, so a call can be captured).
// Tensor i is cut into chunks first[i] .. first[i + 1] - 1; a block that sums takes `each` consecutive ones, and
// chunks before `keep` are read so that they leave L2 first.
// A chunk's tensor is found from owner[chunk >> shift], the tensor of the first chunk with that prefix.
template <int N>
struct GradTable {
  const void* src[N];
  void* dst[N];
  long long numel[N];
  int first[N + 1];
  unsigned short owner[kGradOwners];
  int n, each, keep, shift;
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
// Sums and scaling of at most kGradSmall chunks (tab.dst null: the norm only).
template <typename ST>
cudaError_t launch_grad_small(const GradTable<16>& tab, const GradStat& gs, cudaStream_t st);
// The tensors scaled; with gs.nparts > 0 every block first adds the partial sums up, and the first writes stat.
template <typename ST, int N>
cudaError_t launch_grad_scale(const GradTable<N>& tab, const GradStat& gs, bool in_place, cudaStream_t st);

}  // namespace lr
