// The list of blocks of the packed-attention kernels (packed_device.cuh), made by one thread block: it checks the
// offsets (any that is out of order leaves an empty list and an error bit), counts each sequence's blocks, and sorts
// the blocks into 1024 bins of work.  Blocks of one bin may come in any order; no result depends on it.
//
// It takes 3 to 4 us for the sequences of a usual batch, most of it its barriers, and about 20 us for 16384 blocks.
#include "packed_device.cuh"

#include <algorithm>

namespace lr {
namespace packed {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 1024;

// Sum over the thread block of the values of the threads before this one; total: of all.
__device__ __forceinline__ int scan(int v, int* warps, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  int w = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  __syncthreads();
  return before + s - v;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PackedArgs a, int tokens, int work, Plan plan, unsigned* err) {
  __shared__ int warps[32], bins[kBins], s_bad, s_longest;
  const int tid = threadIdx.x;
  pdl_wait();
  if (tid == 0) s_bad = s_longest = 0;
  bins[tid] = 0;
  __syncthreads();
  // Blocks before each sequence.
  int count = 0, longest = 0;
  bool bad = false;
  for (int base = 0; base < a.nseq; base += kThreads) {
    const int i = base + tid;
    int n = 0;
    if (i < a.nseq) {
      const int b = a.offs[i], e = a.offs[i + 1];
      if (b < 0 || e < b || e > a.T) {
        bad = true;
      } else {
        n = (e - b + tokens - 1) / tokens;
        longest = max(longest, e - b);
      }
    }
    int total;
    const int before = scan(n, warps, total);
    if (i < a.nseq) plan.starts[i] = count + before;
    count += total;
    if (__syncthreads_or(bad)) break;  // the counts may not fit
  }
  if (bad) s_bad = 1;
  if (longest) atomicMax(&s_longest, longest);
  __syncthreads();
  if (s_bad) count = 0;
  if (tid == 0) {
    *plan.next = 0;
    *plan.nblocks = count;
    if (s_bad) atomicOr(err, DEV_ERR_OFFSETS);
  }
  if (count == 0) return;
  // The block at place p of a sequence of n tokens has work for its last token's keys, or for the queries after it.
  int shift = 0;
  while (s_longest >> shift >= kBins) ++shift;
  auto bin = [&](int place, int n) {
    const int w = work > 0 ? min(place + tokens, n) : n - place;
    return kBins - 1 - (w >> shift);
  };
  auto block = [&](int t) {
    int lo = 0, hi = a.nseq;  // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (plan.starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int b = a.offs[lo];
    return make_int4(b, a.offs[lo + 1] - b, (t - plan.starts[lo]) * tokens, 0);
  };
  for (int t = tid; t < count; t += kThreads) {
    const int4 v = block(t);
    atomicAdd(&bins[bin(v.z, v.y)], 1);
  }
  __syncthreads();
  int total;
  const int first = scan(bins[tid], warps, total);
  bins[tid] = first;
  __syncthreads();
  for (int t = tid; t < count; t += kThreads) {
    const int4 v = block(t);
    plan.blocks[atomicAdd(&bins[bin(v.z, v.y)], 1)] = v;
  }
}

}  // namespace

size_t plan_layout(int T, int nseq, int tokens, void* base, Plan* plan) {
  char* p = static_cast<char*>(base);
  size_t at = 256;
  const size_t blocks = at;
  at += sizeof(int4) * plan_capacity(T, nseq, tokens);
  const size_t starts = at;
  at += (sizeof(int) * (static_cast<size_t>(nseq) + 1) + 255) / 256 * 256;
  if (plan) {
    plan->next = reinterpret_cast<unsigned*>(p);
    plan->nblocks = reinterpret_cast<int*>(p) + 1;
    plan->blocks = reinterpret_cast<int4*>(p + blocks);
    plan->starts = reinterpret_cast<int*>(p + starts);
  }
  return (at + 255) / 256 * 256;
}

cudaError_t launch_plan(const PackedArgs& a, int tokens, int work, const Plan& plan, unsigned* err, cudaStream_t st) {
  return launch_pdl(plan_kernel, dim3(1), dim3(kThreads), 0, st, a, tokens, work, plan, err);
}

}  // namespace packed
}  // namespace lr
