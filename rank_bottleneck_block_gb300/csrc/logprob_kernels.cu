// Kernels of lr_logprob_fwd / lr_logprob_bwd (the mathematics is in the header).
//
// Both are bound by memory: the forward reads each logit once, the backward reads it and writes its gradient.  A block
// takes one row's chunk; a warp reads 256 consecutive logits at a time, each lane 8 of them (16 bytes of bf16, 32 of
// fp32), four such groups in flight.  Rows may begin anywhere (an odd V leaves no row but the first on a 16-byte
// boundary): groups are cut at aligned addresses, and the first and last of a row are read element by element.
// A long row of few is cut over blocks, whose parts the join adds up in a fixed order.
//
// The largest logits: the maximum of each segment of 256 or 1024 logits is kept beside the sums (a warp reduction and
// 4 bytes for 256 logits).  By (value descending, index ascending) the K largest logits lie in the K segments whose
// maxima are the largest by the same order; so the join ranks the segments and reads K of them again.  Ranking a list
// takes its threads' own maxima first: the K-th of these bounds what can be among the K largest, and only what reaches
// it is compared with each other (K times a thread's share at most, whatever the values).
#include "logprob_kernels.cuh"

#include <algorithm>

namespace lr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 8;            // logits of a lane's load
constexpr int kWarpRun = 32 * kGroup;  // of a warp's
constexpr int kUnroll = 4;           // groups in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Differences to the maximum are cut off here (2^-200 is 0 in fp32), so that a logit of -inf gives 0 and not 0 * inf.
constexpr float kFloor = -200.f;
constexpr float kMax = 3.4028234663852886e38f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger, or NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

template <typename ST>
__device__ __forceinline__ ST from_float(float v);
template <>
__device__ __forceinline__ bf16 from_float<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }

// Elements between the 16-byte boundary before a row and the row.
template <typename ST>
__device__ __forceinline__ int lead(const ST* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(ST));
}

// Logits i .. i + 7 of a row of V (i may be negative: i + lead is a multiple of 8); -inf outside it.
template <typename ST>
__device__ __forceinline__ void load_edge(const ST* row, int i, int V, float* v) {
#pragma unroll
  for (int e = 0; e < kGroup; ++e) v[e] = i + e >= 0 && i + e < V ? to_float(row[i + e]) : neg_inf();
}

template <typename ST>
__device__ __forceinline__ void load_group(const ST* row, int i, int V, float* v) {
  if (i >= 0 && i + kGroup <= V)
    load8(row + i, v);
  else
    load_edge(row, i, V, v);
}

// m, s, w of a part of a row.
struct Part {
  float m, s, w;
};

__device__ __forceinline__ Part join(Part a, Part b, float c) {
  const float m = max_nan(a.m, b.m);
  if (!(m > neg_inf())) return Part{m, 0.f, 0.f};  // nothing but -inf, or a NaN
  auto at = [&](Part p) {  // p, scaled to m
    if (p.m == neg_inf()) return Part{m, 0.f, 0.f};
    const float d = fmaxf(c * (p.m - m), kFloor), f = ex2(d);
    return Part{m, f * p.s, f * fmaf(p.s, d, p.w)};
  };
  const Part x = at(a), y = at(b);
  return Part{m, x.s + y.s, x.w + y.w};
}

__device__ __forceinline__ Part warp_join(Part p, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    p = join(p, Part{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                     __shfl_xor_sync(0xffffffffu, p.w, o)}, c);
  return p;
}

// Log probability of logit x in a row of which p are the sums.
__device__ __forceinline__ float log_prob(float x, const Part& p, float scale) {
  if (!(p.m <= kMax)) return __int_as_float(0x7fc00000);  // a NaN or +inf in the row
  return x == neg_inf() ? x : fmaf(scale, x - p.m, -kLn2 * log2f(p.s));
}

template <typename ST>
__device__ __forceinline__ void finish(const LogprobFwd& a, int t, Part p) {
  const int k = a.target[t];
  const float l2 = log2f(p.s), nan = __int_as_float(0x7fc00000);
  const bool none = p.m == neg_inf(), bad = !(p.m <= kMax);
  float logp = bad ? nan : 0.f;
  if (k >= 0 && k < a.V)
    logp = log_prob(to_float(static_cast<const ST*>(a.logits)[t * a.ld + k]), p, a.scale);
  a.logp[t] = logp;
  a.entropy[t] = bad ? nan : none ? 0.f : kLn2 * (l2 - p.w / p.s);
  a.lse[t] = bad ? nan : none ? neg_inf() : fmaf(a.scale, p.m, kLn2 * l2);
}

// The largest of a warp's values; a NaN counts as the largest.
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename ST, bool TOP>
__global__ void __launch_bounds__(kThreads) logprob_fwd_kernel(LogprobFwd a, LogprobPlan plan) {
  __shared__ Part warps[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x / plan.splits), split = static_cast<int>(blockIdx.x - 1u * t * plan.splits);
  const ST* row = static_cast<const ST*>(a.logits) + t * a.ld;
  const float c = a.scale * kLog2e;
  pdl_wait();
  const int shift = lead(row);
  // places in the row, counted from the boundary before it
  const long long begin = 1LL * split * plan.chunk;
  const int end = static_cast<int>(min(begin + plan.chunk, 1LL * a.V + shift));
  Part p{neg_inf(), 0.f, 0.f};
  constexpr int kRun = kWarpRun * kUnroll;
  for (int i = static_cast<int>(begin) + warp * kRun; i < end; i += kWarps * kRun) {
    float v[kUnroll][kGroup];
    if (i >= shift && i + kRun <= end && i + kRun <= a.V + shift) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) load8(row + (i + u * kWarpRun + lane * kGroup - shift), v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) load_group(row, i + u * kWarpRun + lane * kGroup - shift, a.V, v[u]);
    }
    float gm = neg_inf();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float um = v[u][0];
#pragma unroll
      for (int e = 1; e < kGroup; ++e) um = max_nan(um, v[u][e]);
      gm = max_nan(gm, um);
      if (TOP && plan.seg == kWarpRun) {
        const float r = warp_max(um);
        const int run = i + u * kWarpRun;
        if (lane == 0 && run < end) a.segmax[1LL * t * plan.nseg + run / kWarpRun] = r;
      }
    }
    if (TOP && plan.seg == kRun) {
      const float r = warp_max(gm);
      if (lane == 0) a.segmax[1LL * t * plan.nseg + i / kRun] = r;
    }
    if (!(gm <= p.m)) p = join(p, Part{gm, 0.f, 0.f}, c);
    if (p.m > neg_inf()) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float s[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
          const float d = fmaxf(c * (v[u][e] - p.m), kFloor), x = ex2(d);
          s[e & 1] += x;
          w[e & 1] = fmaf(x, d, w[e & 1]);
        }
        p.s += s[0] + s[1];
        p.w += w[0] + w[1];
      }
    }
  }
  p = warp_join(p, c);
  if (lane == 0) warps[warp] = p;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kWarps; ++i) p = join(p, warps[i], c);
    if (TOP || plan.splits > 1)
      a.part[1LL * t * plan.splits + split] = make_float4(p.m, p.s, p.w, 0.f);
    else
      finish<ST>(a, t, p);
  }
}

// Larger keys are larger logits; a NaN is the largest, -0 and 0 are equal, equal logits are ordered by their place.
__device__ __forceinline__ unsigned order(float v) {
  if (v != v) return 0xffffffffu;
  const unsigned b = __float_as_uint(v + 0.f);  // -0 + 0 = 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(float v, int place) {
  return static_cast<unsigned long long>(order(v)) << 32 | (0xffffffffu - static_cast<unsigned>(place));
}
__device__ __forceinline__ int place_of(unsigned long long key) {
  return static_cast<int>(0xffffffffu - static_cast<unsigned>(key));
}

constexpr int kLongSeg = kWarpRun * kUnroll;
constexpr int kSegs = kLogprobMaxV / kLongSeg + 1;  // per row at most
// Logits that can reach the bound: K times a thread's share of K segments.
constexpr int kKept = kLogprobMaxTop * (kLogprobMaxTop * kLongSeg / kThreads);

// Of the block's threads' own keys (0: none), the K-th largest; 0 where there are fewer.
__device__ __forceinline__ unsigned long long kth(unsigned long long own, int K, unsigned long long* each,
                                                  unsigned long long* bound) {
  each[threadIdx.x] = own;
  if (threadIdx.x == 0) *bound = 0;
  __syncthreads();
  if (own) {
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < kThreads; ++j) rank += each[j] > own;
    if (rank == K - 1) *bound = own;
  }
  __syncthreads();
  return *bound;
}

// One block per row.
template <typename ST>
__global__ void __launch_bounds__(kThreads) logprob_join_kernel(LogprobFwd a, LogprobPlan plan) {
  __shared__ Part s_part;
  __shared__ unsigned long long keys[kKept], each[kThreads], s_bound;
  __shared__ int picked[kLogprobMaxTop];
  __shared__ int s_count[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x, K = a.top;
  const float c = a.scale * kLog2e;
  pdl_wait();
  if (warp == 0) {
    Part p{neg_inf(), 0.f, 0.f};
    for (int i = lane; i < plan.splits; i += 32) {
      const float4 v = a.part[1LL * t * plan.splits + i];
      p = join(p, Part{v.x, v.y, v.z}, c);
    }
    p = warp_join(p, c);
    if (lane == 0) {
      s_part = p;
      finish<ST>(a, t, p);
    }
  }
  if (K == 0) return;
  const ST* row = static_cast<const ST*>(a.logits) + t * a.ld;
  const int shift = lead(row);
  const int nseg = (a.V + shift + plan.seg - 1) / plan.seg;  // of this row
  if (threadIdx.x < 2) s_count[threadIdx.x] = 0;

  // The K best segments (all where there are fewer).
  unsigned long long own = 0;
  for (int i = threadIdx.x; i < nseg; i += kThreads) own = max(own, key_of(a.segmax[1LL * t * plan.nseg + i], i));
  unsigned long long bound = kth(own, K, each, &s_bound);
  for (int i = threadIdx.x; i < nseg; i += kThreads) {
    const unsigned long long k = key_of(a.segmax[1LL * t * plan.nseg + i], i);
    if (k >= bound) keys[atomicAdd(&s_count[0], 1)] = k;
  }
  __syncthreads();
  const int reach = s_count[0];
  for (int i = threadIdx.x; i < reach; i += kThreads) {
    const unsigned long long k = keys[i];
    int rank = 0;
    for (int j = 0; j < reach; ++j) rank += keys[j] > k;
    if (rank < K) picked[rank] = place_of(k);
  }
  __syncthreads();

  // The K largest logits of these segments.
  const int per = plan.seg / kGroup, groups = min(K, nseg) * per;
  auto walk = [&](auto&& use) {
    for (int g = threadIdx.x; g < groups; g += kThreads) {
      const int i = picked[g / per] * plan.seg + (g % per) * kGroup - shift;
      if (i >= a.V || i + kGroup <= 0) continue;
      float v[kGroup];
      load_group(row, i, a.V, v);
#pragma unroll
      for (int e = 0; e < kGroup; ++e)
        if (i + e >= 0 && i + e < a.V) use(key_of(v[e], i + e));
    }
  };
  own = 0;
  walk([&](unsigned long long k) { own = max(own, k); });
  bound = kth(own, K, each, &s_bound);
  walk([&](unsigned long long k) {
    if (k >= bound) keys[atomicAdd(&s_count[1], 1)] = k;
  });
  __syncthreads();
  const int n = s_count[1];
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long k = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > k;
    if (rank >= K) continue;
    a.top_ids[1LL * t * K + rank] = place_of(k);
    a.top_logp[1LL * t * K + rank] = log_prob(to_float(row[place_of(k)]), s_part, a.scale);
  }
}

// 2^x of the gradient: bf16 takes the hardware approximation (its 2^-22 is far below the rounding of the result), fp32
// the library's exponential of the difference, whose rounding a factor of log2 e would double.
template <typename ST>
struct Prob;
template <>
struct Prob<bf16> {
  static __device__ __forceinline__ void get(float x, float scale, float lse, float& lp, float& p) {
    lp = fmaxf(fmaf(x, scale, -lse), kFloor);
    p = ex2(lp * kLog2e);
  }
};
template <>
struct Prob<float> {
  static __device__ __forceinline__ void get(float x, float scale, float lse, float& lp, float& p) {
    lp = fmaxf(fmaf(x, scale, -lse), kFloor);
    p = expf(lp);
  }
};

template <typename ST, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) logprob_bwd_kernel(LogprobBwd a, int chunks, int chunk) {
  const int t = static_cast<int>(blockIdx.x / chunks), part = static_cast<int>(blockIdx.x - 1u * t * chunks);
  const ST* row = static_cast<const ST*>(a.logits) + t * a.ld;
  ST* out = static_cast<ST*>(a.out) + t * a.ldo;
  pdl_wait();
  const int k = a.target[t];
  const float lse = a.lse[t];
  const float dl = k >= 0 && k < a.V ? a.dlogp[t] : 0.f;
  const float de = ENTROPY ? a.dentropy[t] : 0.f, h = ENTROPY ? a.entropy[t] : 0.f;
  const int shift = lead(row), oshift = lead(out);
  const long long begin = 1LL * part * chunk;
  const int end = static_cast<int>(min(begin + chunk, 1LL * a.V + shift));
  // no gradient, or no distribution (every logit -inf)
  const bool zero = (dl == 0.f && de == 0.f) || lse == neg_inf();
  const float nan = lse - lse;  // 0, or NaN where lse is
  for (int i = static_cast<int>(begin) + threadIdx.x * kGroup; i < end; i += kThreads * kGroup * kUnroll) {
    float v[kUnroll][kGroup];
    if (!zero) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int at = i + u * kThreads * kGroup;
        if (at < end) load_group(row, at - shift, a.V, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = i + u * kThreads * kGroup - shift;
      if (at + shift >= end) break;
#pragma unroll
      for (int e = 0; e < kGroup; ++e) {
        float d = 0.f;
        if (!zero) {
          float lp, p;
          Prob<ST>::get(v[u][e], a.scale, lse, lp, p);
          d = -p * (ENTROPY ? fmaf(de, lp + h, dl) : dl) + nan;
          if (at + e == k) d += dl;
          d *= a.scale;
        }
        v[u][e] = d;
      }
      if (at >= 0 && at + kGroup <= a.V && oshift == shift) {
        store8(out + at, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < kGroup; ++e)
          if (at + e >= 0 && at + e < a.V) out[at + e] = from_float<ST>(v[u][e]);
      }
    }
  }
}

}  // namespace

LogprobPlan logprob_plan(int T, int V, int es, int sms) {
  LogprobPlan p;
  const int most = V + 16 / es - 1;  // places of a row, counted from a 16-byte boundary
  p.seg = most <= kWarpRun * kSegs ? kWarpRun : kLongSeg;
  p.nseg = (most + p.seg - 1) / p.seg;
  // One block to a row where rows fill the GPU (four blocks an SM); else a row over several, each with one load of all
  // of its threads at least.
  constexpr int step = kThreads * kGroup * kUnroll;
  const int fit = (most + step - 1) / step;
  const int want = (4 * sms + T - 1) / T;
  const int s = std::min({want, fit, kLogprobMaxSplits});
  p.chunk = (fit + s - 1) / s * step;
  p.splits = (most + p.chunk - 1) / p.chunk;
  return p;
}

template <typename ST>
cudaError_t launch_logprob_fwd(const LogprobFwd& a, const LogprobPlan& plan, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(1LL * a.T * plan.splits));
  return a.top > 0 ? launch_pdl(logprob_fwd_kernel<ST, true>, grid, dim3(kThreads), 0, st, a, plan)
                   : launch_pdl(logprob_fwd_kernel<ST, false>, grid, dim3(kThreads), 0, st, a, plan);
}

template <typename ST>
cudaError_t launch_logprob_join(const LogprobFwd& a, const LogprobPlan& plan, cudaStream_t st) {
  return launch_pdl(logprob_join_kernel<ST>, dim3(a.T), dim3(kThreads), 0, st, a, plan);
}

template <typename ST>
cudaError_t launch_logprob_bwd(const LogprobBwd& a, cudaStream_t st) {
  constexpr int chunk = kThreads * kGroup * kUnroll;
  const int chunks = (a.V + 16 / static_cast<int>(sizeof(ST)) - 1 + chunk - 1) / chunk;
  const dim3 grid(static_cast<unsigned>(1LL * a.T * chunks));
  return a.dentropy ? launch_pdl(logprob_bwd_kernel<ST, true>, grid, dim3(kThreads), 0, st, a, chunks, chunk)
                    : launch_pdl(logprob_bwd_kernel<ST, false>, grid, dim3(kThreads), 0, st, a, chunks, chunk);
}

#define LR_INSTANTIATE(ST)                                                                         \
  template cudaError_t launch_logprob_fwd<ST>(const LogprobFwd&, const LogprobPlan&, cudaStream_t);  \
  template cudaError_t launch_logprob_join<ST>(const LogprobFwd&, const LogprobPlan&, cudaStream_t); \
  template cudaError_t launch_logprob_bwd<ST>(const LogprobBwd&, cudaStream_t);
LR_INSTANTIATE(bf16)
LR_INSTANTIATE(float)
#undef LR_INSTANTIATE

}  // namespace lr
