// Both passes are bound by memory: a thread has 128 bytes in flight (16-byte loads), a block takes consecutive chunks of
// the tensors' concatenation, and there are several times as many blocks as run at once, since SMs do not get the same
// share of the bandwidth.  A launch that scales goes through its chunks backwards, so that one that takes the whole list
// finds in L2 what the sum read last: all but the last 64 MB of a launch's reads and all of the outputs are marked to
// leave L2 first.  Lists of more than kGradTable tensors are scaled launch by launch in the order of their sums,
// which loses that unless L2 holds the whole list.
// Measured, fp32, clipped into other tensors, three sets of buffers in turn (in brackets the same ones each time, of
// which L2 still holds some): 283 million elements (168 tensors) 484 us (478), of which the sum 154 us; 80 million (16
// tensors) 141 us (135); what both passes move at the copy rate is 509 and 144 us less the part found in L2, and reading
// and writing once would be 339 and 96 us.  20 million bf16 elements in 613 tensors of uneven sizes 24 us; 181,000 fp32
// elements in one launch 5 us.
#include "grad_kernels.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>

namespace lr {

constexpr int kThreads = 256;
template <typename ST>
constexpr int kChunk = kGradChunkBytes / static_cast<int>(sizeof(ST));

// The tensor that owns a chunk, from a tensor at or before it: the last i with first[i] <= chunk (tensors without
// elements own none).
template <int N>
__device__ __forceinline__ int owner_from(const GradTable<N>& tab, int i, int chunk) {
  while (tab.first[i + 1] <= chunk) ++i;
  return i;
}
template <int N>
__device__ __forceinline__ int owner_of(const GradTable<N>& tab, int chunk) {
  return owner_from(tab, tab.owner[chunk >> tab.shift], chunk);
}

// A chunk's elements.
template <typename ST>
struct Chunk {
  long long e;  // of tensor i, from element e
  int n;
  template <int N>
  __device__ __forceinline__ Chunk(const GradTable<N>& tab, int i, int chunk) {
    e = static_cast<long long>(chunk - tab.first[i]) * kChunk<ST>;
    n = static_cast<int>(min(static_cast<long long>(kChunk<ST>), tab.numel[i] - e));
  }
};

// One of kThreads threads' part of a chunk of n elements at g: whole 16-byte words, kThreads apart (zeros past the end),
// and at most one of the elements behind the last whole word.
template <typename ST>
struct Part {
  static constexpr int kPer = 16 / sizeof(ST), kWords = kGradChunkBytes / 16 / kThreads;
  uint4 w[kWords];
  int words, tail;  // tail: the element, or -1

  // evict_first: nothing will read these lines again before they would have left L2 anyway.
  __device__ __forceinline__ void load(const ST* g, int n, bool evict_first = false) {
    const int me = threadIdx.x % kThreads;
    words = n / kPer;
    tail = words * kPer + me < n ? words * kPer + me : -1;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int v = me + k * kThreads;
      const uint4* from = reinterpret_cast<const uint4*>(g) + v;
      w[k] = v >= words ? make_uint4(0, 0, 0, 0) : evict_first ? __ldcs(from) : *from;
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
      const int v = threadIdx.x % kThreads + k * kThreads;
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
      __stcs(reinterpret_cast<uint4*>(o) + v, make_uint4(r[0], r[1], r[2], r[3]));
    }
    if (tail >= 0) o[tail] = static_cast<ST>(scale * static_cast<float>(g[tail]));
  }
  // Adds the squares to the warp's sum: lane 0's, but for what the slow path and the tail leave in other lanes
  // (`spread`).  The warp's words are summed in fp32 (16 or 32 in a row, then pairwise), and from there on in fp64; where
  // that sum is no number, beyond fp32 or so small that squares have lost digits, the same squares are summed in fp64
  // (2048 squares and sums below 2^-126 are off by 2^-139 together: a 2^-29th of 2^-110).
  __device__ __forceinline__ void add_squares(const ST* g, double& sum, bool& spread) const {
    float a = 0.f, b = 0.f;
    int k = 0;
    each([&](float v) {
      float& s = k++ & 1 ? b : a;
      s = fmaf(v, v, s);
    });
    float s = a + b;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (s >= 0x1p-110f && s <= FLT_MAX) {  // the same in every lane
      if (threadIdx.x % 32 == 0) sum += static_cast<double>(s);
    } else {
      uint32_t any = 0;
#pragma unroll
      for (int k = 0; k < kWords; ++k) any |= w[k].x | w[k].y | w[k].z | w[k].w;
      if (any & (sizeof(ST) == 4 ? 0x7fffffffu : 0x7fff7fffu)) {
#pragma unroll 1
        for (int v = threadIdx.x % kThreads * kPer; v < words * kPer; v += kThreads * kPer)
#pragma unroll 1
          for (int i = 0; i < kPer; ++i) {
            const double x = static_cast<double>(static_cast<float>(g[v + i]));
            sum += x * x;
          }
      }
      spread = true;
    }
    if (tail >= 0) {
      const double v = static_cast<double>(static_cast<float>(g[tail]));
      sum += v * v;
      spread = true;
    }
  }
};

// A warp's sum in all of its lanes.
__device__ __forceinline__ double warp_sum(double v, bool spread) {
  if (__any_sync(0xffffffffu, spread)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  return __shfl_sync(0xffffffffu, v, 0);
}

template <typename ST, int N>
__global__ void __launch_bounds__(kThreads, 4) grad_sumsq_kernel(const __grid_constant__ GradTable<N> tab, double* part) {
  pdl_wait();
  pdl_trigger();
  const int c0 = blockIdx.x * tab.each, c1 = min(c0 + tab.each, tab.first[tab.n]);
  int i = owner_of(tab, c0);
  double sum = 0.0;
  bool spread = false;
  for (int ch = c0; ch < c1; ++ch) {
    i = owner_from(tab, i, ch);
    const Chunk<ST> c(tab, i, ch);
    const ST* g = static_cast<const ST*>(tab.src[i]) + c.e;
    Part<ST> p;
    p.load(g, c.n, ch < tab.keep);
    p.add_squares(g, sum, spread);
  }
  __shared__ double red[kThreads / 32];
  sum = warp_sum(sum, spread);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += red[w];
    part[blockIdx.x] = sum;
  }
}

// norm and scale of a sum of squares, by one thread, which writes them with `write`.
__device__ __forceinline__ float scale_from(double sum, const GradStat& gs, bool write) {
  const float norm = static_cast<float>(sqrt(sum));
  const float c = gs.max_norm / (norm + 1e-6f);
  const float scale = c > 1.f ? 1.f : c;  // a NaN norm stays visible
  if (write) {
    gs.stat[0] = norm;
    if (!gs.norm_only) gs.stat[1] = scale;
  }
  return scale;
}

// The scale in every thread of the block.  fp64 arithmetic is scarce (a warp's addition takes 16 cycles of the SM's one
// fp64 pipe), so one warp does what is left of it after the threads' own sums, and one thread the root.
__device__ __forceinline__ float scale_of(const GradStat& gs, bool write) {
  if (gs.nparts == 0) return gs.stat[1];
  __shared__ double red[kThreads];
  __shared__ float scale;
  double sum = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < gs.nparts; i += kThreads) sum += gs.part[i];
  red[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    for (int i = 32; i < kThreads && i < gs.nparts; i += 32) sum += red[threadIdx.x + i];
    sum = warp_sum(sum, true);
    if (threadIdx.x == 0) scale = scale_from(sum, gs, write);
  }
  __syncthreads();
  return scale;
}

__global__ void __launch_bounds__(kThreads) grad_stat_kernel(const __grid_constant__ GradStat gs) {
  pdl_wait();
  pdl_trigger();
  scale_of(gs, true);
}

template <typename ST, int N>
__global__ void __launch_bounds__(kThreads, 4) grad_scale_kernel(const __grid_constant__ GradTable<N> tab,
                                                              const __grid_constant__ GradStat gs, int each, bool in_place) {
  pdl_wait();
  pdl_trigger();
  float scale = 1.f;
  if (in_place) {
    scale = scale_of(gs, blockIdx.x == 0);
    if (scale == 1.f) return;  // nothing changes
  }
  const int c1 = tab.first[tab.n] - blockIdx.x * each, c0 = max(0, c1 - each);
  int i = owner_of(tab, c0);
  bool known = in_place;
  for (int ch = c0; ch < c1; ++ch) {
    i = owner_from(tab, i, ch);
    const Chunk<ST> c(tab, i, ch);
    const ST* g = static_cast<const ST*>(tab.src[i]) + c.e;
    Part<ST> p;
    p.load(g, c.n);
    if (!known) scale = scale_of(gs, blockIdx.x == 0);  // with the first loads in flight
    known = true;
    p.store_scaled(static_cast<ST*>(tab.dst[i]) + c.e, g, scale);
  }
}

// Few chunks: one cluster holds them in registers, a chunk for 256 of a block's threads, and exchanges the blocks' sums.
constexpr int kSmallThreads = 512;
template <typename ST>
__global__ void __launch_bounds__(kSmallThreads) grad_small_kernel(const __grid_constant__ GradTable<16> tab,
                                                                   const __grid_constant__ GradStat gs) {
  namespace cg = cooperative_groups;
  pdl_wait();
  pdl_trigger();
  const cg::cluster_group cluster = cg::this_cluster();
  const int ch = blockIdx.x * (kSmallThreads / kThreads) + threadIdx.x / kThreads;
  const bool mine = ch < tab.first[tab.n];
  const int i = mine ? owner_of(tab, ch) : 0;
  const ST* g = nullptr;
  long long e = 0;
  Part<ST> p;
  double sum = 0.0;
  bool spread = false;
  if (mine) {
    const Chunk<ST> c(tab, i, ch);
    e = c.e;
    g = static_cast<const ST*>(tab.src[i]) + e;
    p.load(g, c.n);
    p.add_squares(g, sum, spread);
  }
  __shared__ double red[32];
  __shared__ double total;
  sum = warp_sum(sum, spread);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    sum = warp_sum(threadIdx.x < kSmallThreads / 32 ? red[threadIdx.x] : 0.0, true);
    if (threadIdx.x == 0) total = sum;
  }
  cluster.sync();
  __shared__ float scale_shared;
  if (threadIdx.x < 32) {  // a lane for each block's sum
    sum = warp_sum(threadIdx.x < cluster.num_blocks() ? *cluster.map_shared_rank(&total, threadIdx.x) : 0.0, true);
    if (threadIdx.x == 0) scale_shared = scale_from(sum, gs, blockIdx.x == 0);
  }
  __syncthreads();
  const float scale = scale_shared;
  auto token = cluster.barrier_arrive();  // the sums stay until every block has read them
  if (mine && !gs.norm_only) p.store_scaled(static_cast<ST*>(tab.dst[i]) + e, g, scale);
  cluster.barrier_wait(std::move(token));
}

template <typename ST, int N>
cudaError_t launch_grad_sumsq(const GradTable<N>& tab, double* part, cudaStream_t st) {
  return launch_pdl(grad_sumsq_kernel<ST, N>, dim3(grad_blocks(tab.first[tab.n], tab.each)), dim3(kThreads), 0, st, tab,
                    part);
}

cudaError_t launch_grad_stat(const GradStat& gs, cudaStream_t st) {
  return launch_pdl(grad_stat_kernel, dim3(1), dim3(kThreads), 0, st, gs);
}

template <typename ST, int N>
cudaError_t launch_grad_scale(const GradTable<N>& tab, const GradStat& gs, bool in_place, cudaStream_t st) {
  // Chunks of a block.  In place the launch often finds a scale of 1, and then only starts and ends its blocks: of 283
  // million fp32 elements, two chunks to a block take 169 us with the sum (484 where they are scaled), four 162 (487),
  // the same buffers each time.
  constexpr int kInPlaceEach = 4;
  const int chunks = tab.first[tab.n], each = in_place ? std::min(kInPlaceEach, std::max(2, chunks / 2432)) : 2;
  return launch_pdl(grad_scale_kernel<ST, N>, dim3(grad_blocks(chunks, each)), dim3(kThreads), 0, st, tab, gs, each,
                    in_place);
}

template <typename ST>
cudaError_t launch_grad_small(const GradTable<16>& tab, const GradStat& gs, cudaStream_t st) {
  constexpr int per = kSmallThreads / kThreads;
  static_assert(kGradSmall <= 16 * per, "a cluster has at most 16 blocks");
  const int blocks = tab.first[tab.n] > per ? (tab.first[tab.n] + per - 1) / per : 1;
  if (blocks > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(grad_small_kernel<ST>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grad_small_kernel<ST>, tab, gs);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template cudaError_t launch_grad_small<float>(const GradTable<16>&, const GradStat&, cudaStream_t);
template cudaError_t launch_grad_small<bf16>(const GradTable<16>&, const GradStat&, cudaStream_t);

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
