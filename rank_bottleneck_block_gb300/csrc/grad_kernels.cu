#include "grad_kernels.cuh"

namespace lr {

int grad_blocks(int chunks) { return chunks < kGradParts ? chunks : kGradParts; }

// The tensor that owns `chunk`: the last i with first[i] <= chunk (tensors without elements own none).
template <int N>
__device__ __forceinline__ int owner_of(const GradTable<N>& tab, int chunk) {
  int lo = 0, hi = tab.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Sum over the block, valid in every thread; fixed order.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[256];
  red[threadIdx.x] = v;
  __syncthreads();
  for (int s = 128; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  return red[0];
}

template <typename ST, int N>
__global__ void grad_sumsq_kernel(const __grid_constant__ GradTable<N> tab, double* part) {
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int ch = blockIdx.x; ch < tab.first[tab.n]; ch += gridDim.x) {
    const int i = owner_of(tab, ch);
    const ST* g = static_cast<const ST*>(tab.src[i]);
    const long long e0 = static_cast<long long>(ch - tab.first[i]) * kGradChunk;
    const long long e1 = min(e0 + kGradChunk, tab.numel[i]);
    for (long long e = e0 + threadIdx.x; e < e1; e += 256) {
      const double v = static_cast<double>(static_cast<float>(g[e]));
      sum += v * v;
    }
  }
  const double s = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <typename ST, int N>
__global__ void grad_scale_kernel(const __grid_constant__ GradTable<N> tab, const double* part, int nparts,
                                  float max_norm, float* stat, int write_stat) {
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int i = threadIdx.x; i < nparts; i += 256) sum += part[i];
  const float norm = static_cast<float>(sqrt(block_sum(sum)));
  const float c = max_norm / (norm + 1e-6f);
  const float scale = c > 1.f ? 1.f : c;  // a NaN norm stays visible
  if (write_stat && blockIdx.x == 0 && threadIdx.x == 0) {
    stat[0] = norm;
    if (write_stat > 1) stat[1] = scale;
  }
  for (int ch = blockIdx.x; ch < tab.first[tab.n]; ch += gridDim.x) {
    const int i = owner_of(tab, ch);
    const ST* g = static_cast<const ST*>(tab.src[i]);
    ST* o = static_cast<ST*>(tab.dst[i]);
    const long long e0 = static_cast<long long>(ch - tab.first[i]) * kGradChunk;
    const long long e1 = min(e0 + kGradChunk, tab.numel[i]);
    for (long long e = e0 + threadIdx.x; e < e1; e += 256)
      o[e] = static_cast<ST>(scale * static_cast<float>(g[e]));
  }
}

template <typename ST, int N>
cudaError_t launch_grad_sumsq(const GradTable<N>& tab, double* part, cudaStream_t st) {
  return launch_pdl(grad_sumsq_kernel<ST, N>, dim3(grad_blocks(tab.first[tab.n])), dim3(256), 0, st, tab, part);
}

template <typename ST, int N>
cudaError_t launch_grad_scale(const GradTable<N>& tab, const double* part, int nparts, float max_norm, float* stat,
                              int write_stat, cudaStream_t st) {
  const int chunks = tab.first[tab.n];
  return launch_pdl(grad_scale_kernel<ST, N>, dim3(chunks > 0 ? grad_blocks(chunks) : 1), dim3(256), 0, st, tab, part,
                    nparts, max_norm, stat, write_stat);
}

#define LR_GRAD_INST(ST, N)                                                                           \
  template cudaError_t launch_grad_sumsq<ST, N>(const GradTable<N>&, double*, cudaStream_t);       \
  template cudaError_t launch_grad_scale<ST, N>(const GradTable<N>&, const double*, int, float, float*, int, \
                                               cudaStream_t);
LR_GRAD_INST(float, kGradTable)
LR_GRAD_INST(bf16, kGradTable)
#undef LR_GRAD_INST

}  // namespace lr
