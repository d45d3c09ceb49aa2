// The first launch of the packed-attention calls.  One thread block for each list of blocks (packed_device.cuh): it checks the
// offsets (any that is out of order leaves an empty list and an error bit), counts each sequence's blocks, and sorts
// the blocks into 1024 bins of work.  Blocks of one bin may come in any order; no result depends on it.
//
// In the backward the other blocks take D = dout.o of every row and head: 8 or 16 lanes a head, 16 bytes of both tensors a
// lane, two heads in flight (rows of no sequence too: nothing reads theirs).  In 32 registers two blocks fit an SM, so that
// one loads while the other sums: 268 MB in 41 us (6.5 TB/s); four heads in flight and one block took 52.
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

__device__ __forceinline__ void make_list(const PackedArgs& a, int tokens, int work, const Plan& plan, unsigned* err) {
  __shared__ int warps[32], bins[kBins], s_bad, s_longest;
  const int tid = threadIdx.x;
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

struct Jobs {
  PlanJob job[2];
};

constexpr int kDots = 2;

// D of kDots consecutive (row, head) for each group of `lanes` lanes.
__device__ __forceinline__ void row_dots(const PackedArgs& a, float* D, int block, int lanes) {
  const int shift = lanes == 16 ? 4 : 3, group = threadIdx.x >> shift, lane = threadIdx.x & (lanes - 1), c = 8 * lane;
  const unsigned first = (static_cast<unsigned>(block) * (kThreads >> shift) + group) * kDots, all = 1u * a.T * a.Hq;
  unsigned t = first / a.Hq, h = first - t * a.Hq;
  uint4 x[kDots], y[kDots];
#pragma unroll
  for (int u = 0; u < kDots; ++u) {
    x[u] = y[u] = make_uint4(0, 0, 0, 0);
    if (first + u < all && c < a.dh) {
      const int col = static_cast<int>(h) * a.dh + c;
      x[u] = *reinterpret_cast<const uint4*>(a.o.p + t * a.o.ld + col);
      y[u] = *reinterpret_cast<const uint4*>(a.dout.p + t * a.dout.ld + col);
    }
    if (++h == static_cast<unsigned>(a.Hq)) {
      h = 0;
      ++t;
    }
  }
#pragma unroll
  for (int u = 0; u < kDots; ++u) {
    float v[8], w[8], s = 0.f;
    load8(reinterpret_cast<const bf16*>(&x[u]), v);
    load8(reinterpret_cast<const bf16*>(&y[u]), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[e], w[e], s);
    for (int o = lanes >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && first + u < all) D[first + u] = s;
  }
}

__global__ void __launch_bounds__(kThreads, 2) prepare_kernel(PackedArgs a, Jobs jobs, int njobs, float* D, int lanes,
                                                           unsigned* err) {
  pdl_wait();
  pdl_trigger();
  const int b = static_cast<int>(blockIdx.x);
  if (b < njobs) {
    const PlanJob j = b == 0 ? jobs.job[0] : jobs.job[1];
    make_list(a, j.tokens, j.work, j.plan, err);
  } else {
    row_dots(a, D, b - njobs, lanes);
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

cudaError_t launch_prepare(const PackedArgs& a, const PlanJob* jobs, int njobs, float* D, unsigned* err,
                           cudaStream_t st) {
  Jobs j{};
  for (int i = 0; i < njobs; ++i) j.job[i] = jobs[i];
  const int lanes = a.dh > 64 ? 16 : 8;
  const long long each = kThreads / lanes * kDots, dots = D ? (1LL * a.T * a.Hq + each - 1) / each : 0;
  return launch_as(false, prepare_kernel, dim3(static_cast<unsigned>(njobs + dots)), dim3(kThreads), 0, st, a, j, njobs, D,
                   lanes, err);
}

}  // namespace packed
}  // namespace lr
