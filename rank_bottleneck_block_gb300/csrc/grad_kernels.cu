// Both passes are bound by memory: a thread has 32 elements in flight (16-byte loads), a block takes a run of
// consecutive chunks of the tensors' concatenation, and there are some times as many blocks as run at once.  The
// scaling pass goes through the chunks backwards, so that it finds in L2 what the sum read last.
#include "grad_kernels.cuh"

#include <cfloat>

namespace lr {

constexpr int kThreads = 256;
constexpr int kEach = kGradChunk / kThreads;  // elements of a thread

// Where a block is in the tensors: the tensor that owns a chunk is the last i with first[i] <= chunk (tensors without
// elements own none).
template <int N>
struct Place {
  int i;
  __device__ __forceinline__ Place(const GradTable<N>& tab, int chunk) {
    int lo = 0, hi = tab.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tab.first[mid] <= chunk) lo = mid;
      else hi = mid;
    }
    i = lo;
  }
  __device__ __forceinline__ void forward(const GradTable<N>& tab, int chunk) {
    while (tab.first[i + 1] <= chunk) ++i;
  }
  __device__ __forceinline__ void backward(const GradTable<N>& tab, int chunk) {
    while (tab.first[i] > chunk) --i;
  }
};

// A thread's part of a chunk of n elements at g: whole 16-byte words, kThreads apart (zeros past the end), and at most
// one of the elements behind the last whole word.
template <typename ST>
struct Part {
  static constexpr int kPer = 16 / sizeof(ST), kWords = kEach / kPer;
  uint4 w[kWords];
  int words, tail;  // tail: the element, or -1

  __device__ __forceinline__ void load(const ST* g, int n) {
    words = n / kPer;
    tail = words * kPer + threadIdx.x < n ? words * kPer + static_cast<int>(threadIdx.x) : -1;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int v = threadIdx.x + k * kThreads;
      w[k] = v < words ? reinterpret_cast<const uint4*>(g)[v] : make_uint4(0, 0, 0, 0);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(ST) == 4) {
          f(__uint_as_float(u[i]));
        } else {
          f(__uint_as_float(u[i] << 16));
          f(__uint_as_float(u[i] & 0xffff0000u));
        }
      }
    }
  }
  __device__ __forceinline__ void store_scaled(ST* o, const ST* g, float scale) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int v = threadIdx.x + k * kThreads;
      if (v >= words) break;
      const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(ST) == 4) {
          r[i] = __float_as_uint(scale * __uint_as_float(u[i]));
        } else {
          const __nv_bfloat162 h =
              __floats2bfloat162_rn(scale * __uint_as_float(u[i] << 16), scale * __uint_as_float(u[i] & 0xffff0000u));
          r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      reinterpret_cast<uint4*>(o)[v] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    if (tail >= 0) o[tail] = static_cast<ST>(scale * static_cast<float>(g[tail]));
  }
};

// Sum over the block in a fixed order, valid in every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[32];
  const int warps = blockDim.x / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < warps; ++i) v += red[i];
  return v;
}

// A thread's 32 squares are summed in fp32, and from there on in fp64.  Where that sum leaves the safe range (squares
// beyond 2^128, or so small that the sum has lost digits), the same 32 are summed again in fp64.
template <typename ST, int N>
__global__ void __launch_bounds__(kThreads) grad_sumsq_kernel(const __grid_constant__ GradTable<N> tab, double* part) {
  pdl_wait();
  pdl_trigger();
  const int c0 = blockIdx.x * tab.each, c1 = min(c0 + tab.each, tab.first[tab.n]);
  Place<N> at(tab, c0);
  double sum = 0.0;
  for (int ch = c0; ch < c1; ++ch) {
    at.forward(tab, ch);
    const long long e = static_cast<long long>(ch - tab.first[at.i]) * kGradChunk;
    const ST* g = static_cast<const ST*>(tab.src[at.i]) + e;
    Part<ST> p;
    p.load(g, static_cast<int>(min(static_cast<long long>(kGradChunk), tab.numel[at.i] - e)));
    float a = 0.f, b = 0.f;
    int k = 0;
    p.each([&](float v) {
      float& s = k++ & 1 ? b : a;
      s = fmaf(v, v, s);
    });
    const float s = a + b;
    if (s >= 0x1p-80f && s <= FLT_MAX) {
      sum += static_cast<double>(s);
    } else {
      float any = 0.f;
      p.each([&](float v) { any = v == 0.f ? any : 1.f; });
      if (any != 0.f) p.each([&](float v) { sum += static_cast<double>(v) * static_cast<double>(v); });
    }
    if (p.tail >= 0) {
      const double v = static_cast<double>(static_cast<float>(g[p.tail]));
      sum += v * v;
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The scale, and with `write` the results for the caller.
__device__ __forceinline__ float scale_of(const GradStat& gs, bool write) {
  if (gs.nparts == 0) return gs.stat[1];
  double sum = 0.0;
#pragma unroll 2
  for (int i = threadIdx.x; i < gs.nparts; i += blockDim.x) sum += gs.part[i];
  const float norm = static_cast<float>(sqrt(block_sum(sum)));
  const float c = gs.max_norm / (norm + 1e-6f);
  const float scale = c > 1.f ? 1.f : c;  // a NaN norm stays visible
  if (write && threadIdx.x == 0) {
    gs.stat[0] = norm;
    if (!gs.norm_only) gs.stat[1] = scale;
  }
  return scale;
}

__global__ void __launch_bounds__(1024) grad_stat_kernel(const __grid_constant__ GradStat gs) {
  pdl_wait();
  pdl_trigger();
  scale_of(gs, true);
}

template <typename ST, int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ GradTable<N> tab,
                                                              const __grid_constant__ GradStat gs, bool in_place) {
  pdl_wait();
  pdl_trigger();
  const int all = tab.first[tab.n], c1 = all - blockIdx.x * tab.each, c0 = max(0, c1 - tab.each);
  Place<N> at(tab, c1 - 1);
  float scale = 1.f;
  bool known = false;
  if (in_place) {
    scale = scale_of(gs, blockIdx.x == 0);
    known = true;
    if (scale == 1.f) return;  // nothing changes
  }
  for (int ch = c1 - 1; ch >= c0; --ch) {
    at.backward(tab, ch);
    const long long e = static_cast<long long>(ch - tab.first[at.i]) * kGradChunk;
    const ST* g = static_cast<const ST*>(tab.src[at.i]) + e;
    Part<ST> p;
    p.load(g, static_cast<int>(min(static_cast<long long>(kGradChunk), tab.numel[at.i] - e)));
    if (!known) {  // with the first loads in flight
      scale = scale_of(gs, blockIdx.x == 0);
      known = true;
    }
    p.store_scaled(static_cast<ST*>(tab.dst[at.i]) + e, g, scale);
  }
}

template <typename ST, int N>
cudaError_t launch_grad_sumsq(const GradTable<N>& tab, double* part, cudaStream_t st) {
  return launch_pdl(grad_sumsq_kernel<ST, N>, dim3(grad_blocks(tab.first[tab.n], tab.each)), dim3(kThreads), 0, st, tab,
                    part);
}

cudaError_t launch_grad_stat(const GradStat& gs, cudaStream_t st) {
  return launch_pdl(grad_stat_kernel, dim3(1), dim3(1024), 0, st, gs);
}

template <typename ST, int N>
cudaError_t launch_grad_scale(const GradTable<N>& tab, const GradStat& gs, bool in_place, cudaStream_t st) {
  return launch_pdl(grad_scale_kernel<ST, N>, dim3(grad_blocks(tab.first[tab.n], tab.each)), dim3(kThreads), 0, st, tab,
                    gs, in_place);
}

#define LR_GRAD_INST(ST, N)                                                                  \
  template cudaError_t launch_grad_sumsq<ST, N>(const GradTable<N>&, double*, cudaStream_t); \
  template cudaError_t launch_grad_scale<ST, N>(const GradTable<N>&, const GradStat&, bool, cudaStream_t);
LR_GRAD_INST(float, 16)
LR_GRAD_INST(bf16, 16)
LR_GRAD_INST(float, 256)
LR_GRAD_INST(bf16, 256)
LR_GRAD_INST(float, kGradTable)
LR_GRAD_INST(bf16, kGradTable)
#undef LR_GRAD_INST

}  // namespace lr
