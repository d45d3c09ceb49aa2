// Kernels of lr_logprob_fwd / lr_logprob_bwd (the mathematics is in the header).
//
// Both are bound by memory: the forward reads each logit once, the backward reads it and writes its gradient.  A block
// takes one row's chunk; a warp reads 256 consecutive logits at a time, each lane 8 of them (16 bytes of bf16, 32 of
// fp32), 64 bytes a lane in flight.  Rows may begin anywhere (an odd V leaves no row but the first on a 16-byte
// boundary): groups are cut at aligned addresses, and the first and last of a row are read element by element.
// A long row of few is cut over blocks, whose parts the join adds up in a fixed order.
//
// The largest logits: the maximum of each segment of 256 logits is kept beside the sums (a warp reduction and 4 bytes).
// By (value descending, index ascending) the K largest logits lie in the K segments whose maxima are the largest by the
// same order; so the join ranks the segments and reads K of them again.  Ranking a list takes the maxima of 64 groups of
// threads first: the K-th of these bounds what can be among the K largest, and only what reaches it is compared with each
// other (K times a group's share at most, whatever the values).
//
// Measured: 4096 rows of 131072 bf16 logits forward 171 us (6.3 TB/s, 93 % of a copy's rate; 182 with arithmetic on single
// numbers, 174 with five blocks an SM, which spill), backward 304 us (7.1 TB/s; with the exponential of fp32 566 us, bound
// by instructions).  One row of 131072 with the 20 largest: 12 us; the join is
// a chain of short steps behind one another.
#include "logprob_kernels.cuh"

#include <algorithm>

#include "f32x2.cuh"

namespace lr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 8;            // logits of a lane's load
constexpr int kWarpRun = 32 * kGroup;  // of a warp's
template <typename ST>
constexpr int kUnroll = 8 / sizeof(ST);  // groups in flight: 64 bytes a lane
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

// kUnroll groups of a lane, `stride` logits apart: all loads before the first conversion.
template <typename ST>
__device__ __forceinline__ void load_groups(const ST* p, int stride, float (*v)[kGroup]) {
  constexpr int n = sizeof(ST) / 2;  // 16-byte loads of a group
  uint4 raw[kUnroll<ST>][n];
#pragma unroll
  for (int u = 0; u < kUnroll<ST>; ++u)
#pragma unroll
    for (int i = 0; i < n; ++i) raw[u][i] = reinterpret_cast<const uint4*>(p + u * stride)[i];
#pragma unroll
  for (int u = 0; u < kUnroll<ST>; ++u) load8(reinterpret_cast<const ST*>(raw[u]), v[u]);
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
#pragma unroll 1
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

// The logit of a row's target.
template <typename ST>
__device__ __forceinline__ float target_logit(const LogprobFwd& a, int t, bool& has) {
  const int k = a.target[t];
  has = k >= 0 && k < a.V;
  return has ? to_float(static_cast<const ST*>(a.logits)[t * a.ld + k]) : 0.f;
}

__device__ __forceinline__ void finish(const LogprobFwd& a, int t, Part p, float x, bool has) {
  const float l2 = log2f(p.s), nan = __int_as_float(0x7fc00000);
  const bool none = p.m == neg_inf(), bad = !(p.m <= kMax);
  a.logp[t] = has ? log_prob(x, p, a.scale) : bad ? nan : 0.f;
  a.entropy[t] = bad ? nan : none ? 0.f : kLn2 * (l2 - p.w / p.s);
  a.lse[t] = bad ? nan : none ? neg_inf() : fmaf(a.scale, p.m, kLn2 * l2);
}

// The largest of a warp's values; a NaN counts as the largest.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <typename ST, bool TOP>
__global__ void __launch_bounds__(kThreads, sizeof(ST) == 2 ? 4 : 6) logprob_fwd_kernel(LogprobFwd a, LogprobPlan plan) {
  __shared__ Part warps[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x / plan.splits), split = static_cast<int>(blockIdx.x - 1u * t * plan.splits);
  const ST* row = static_cast<const ST*>(a.logits) + t * a.ld;
  const float c = a.scale * kLog2e;
  pdl_wait();
  pdl_trigger();
  const int shift = lead(row);
  // places in the row, counted from the boundary before it
  const long long begin = 1LL * split * plan.chunk;
  const int end = static_cast<int>(min(begin + plan.chunk, 1LL * a.V + shift));
  Part p{neg_inf(), 0.f, 0.f};
  constexpr int kU = kUnroll<ST>, kRun = kWarpRun * kU;
  for (int i = static_cast<int>(begin) + warp * kRun; i < end; i += kWarps * kRun) {
    float v[kU][kGroup];
    const int at = i + lane * kGroup - shift;
    if (i >= shift && i + kRun <= end && i + kRun <= a.V + shift) {
      load_groups(row + at, kWarpRun, v);
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) load_group(row, at + u * kWarpRun, a.V, v[u]);
    }
    float gm = neg_inf();
#pragma unroll
    for (int u = 0; u < kU; u += 2) {
      float um[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        um[w] = v[u + w][0];
#pragma unroll
        for (int e = 1; e < kGroup; ++e) um[w] = max_nan(um[w], v[u + w][e]);
        gm = max_nan(gm, um[w]);
      }
      if (TOP) {
        const int run = i + u * kWarpRun;
        float* seg = a.segmax + 1LL * t * plan.nseg + run / kLogprobSeg;
        const float r0 = warp_max(um[0]), r1 = warp_max(um[1]);
        if (lane == 0 && run < end) seg[0] = r0;
        if (lane == 0 && run + kWarpRun < end) seg[1] = r1;
      }
    }
    if (!(gm <= p.m)) p = join(p, Part{gm, 0.f, 0.f}, c);
    if (p.m > neg_inf()) {
      const uint64_t nm = f2_pack(-p.m, -p.m), cc = f2_pack(c, c);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        uint64_t s2 = 0, w2 = 0;
#pragma unroll
        for (int e = 0; e < kGroup; e += 2) {
          float d[2], s[2];
          f2_unpack(f2_mul(f2_add(f2_pack(v[u][e], v[u][e + 1]), nm), cc), d[0], d[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            d[i] = fmaxf(d[i], kFloor);
            s[i] = ex2(d[i]);
          }
          const uint64_t x = f2_pack(s[0], s[1]);
          s2 = f2_add(s2, x);
          w2 = f2_fma(x, f2_pack(d[0], d[1]), w2);
        }
        float x[2], y[2];
        f2_unpack(s2, x[0], x[1]);
        f2_unpack(w2, y[0], y[1]);
        p.s += x[0] + x[1];
        p.w += y[0] + y[1];
      }
    }
  }
  p = warp_join(p, c);
  if (lane == 0) warps[warp] = p;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 1; i < kWarps; ++i) p = join(p, warps[i], c);
    if (TOP || plan.splits > 1) {
      a.part[1LL * t * plan.splits + split] = make_float4(p.m, p.s, p.w, 0.f);
    } else {
      bool has;
      const float x = target_logit<ST>(a, t, has);
      finish(a, t, p, x, has);
    }
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
__device__ __forceinline__ float value_of(unsigned long long key) {
  const unsigned o = static_cast<unsigned>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? (o == 0xffffffffu ? 0x7fc00000u : o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int place_of(unsigned long long key) {
  return static_cast<int>(0xffffffffu - static_cast<unsigned>(key));
}

static_assert(kLogprobSeg == kWarpRun, "a segment is what a warp reads at a time");
// Logits that can reach the bound: K times the share of four threads of K segments.
constexpr int kKept = kLogprobMaxTop * (4 * kLogprobMaxTop * kLogprobSeg / kThreads);
static_assert((kLogprobMaxV / kLogprobSeg / kThreads + 1) * 4 <= kKept / kLogprobMaxTop, "segments that can reach it");

struct TopShared {
  unsigned long long keys[kKept], each[kThreads / 4], bound;
  int picked[kLogprobMaxTop];  // segments
  int count;
  Part part;
};

// Of 64 maxima of the keys of four threads each (0: none), the K-th largest; 0 where there are fewer.
__device__ __forceinline__ unsigned long long kth(unsigned long long own, int K, TopShared& s) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) own = max(own, __shfl_xor_sync(0xffffffffu, own, o));
  const int part = threadIdx.x & 3;
  if (part == 0) s.each[threadIdx.x >> 2] = own;
  __syncthreads();
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < 16; ++j) rank += s.each[16 * part + j] > own;
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (own && rank == K - 1) s.bound = own;  // four threads, the same value
  __syncthreads();
  return s.bound;
}

// Leaves in s.keys the keys that reach the K-th of the groups' maxima.  each(f) calls f for this thread's keys.
template <typename F>
__device__ __forceinline__ void reach_bound(int K, TopShared& s, F each) {
  if (threadIdx.x == 0) {
    s.bound = 0;
    s.count = 0;
  }
  unsigned long long own = 0;
  each([&](unsigned long long k) { own = max(own, k); });
  const unsigned long long bound = max(kth(own, K, s), 1ull);
  if (own >= bound)
    each([&](unsigned long long k) {
      if (k >= bound) s.keys[atomicAdd(&s.count, 1)] = k;
    });
  __syncthreads();
}

// Calls use(rank, key) for the K largest of the kept keys: 16 lanes count the larger ones of each.
template <typename F>
__device__ __forceinline__ void rank_keys(const TopShared& s, int K, F use) {
  const int part = threadIdx.x & 15, n = s.count;
#pragma unroll 1
  for (int base = 0; base < n; base += kThreads / 16) {
    const int i = base + (threadIdx.x >> 4);
    const unsigned long long k = i < n ? s.keys[i] : 0;
    int rank = 0;
#pragma unroll 2
    for (int j = part; j < n; j += 16) rank += s.keys[j] > k;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (part == 0 && i < n && rank < K) use(rank, k);
  }
}

// One block per row.
template <typename ST>
__global__ void __launch_bounds__(kThreads) logprob_join_kernel(LogprobFwd a, LogprobPlan plan) {
  __shared__ __align__(16) TopShared s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x, K = a.top;
  const float c = a.scale * kLog2e;
  pdl_wait();
  bool has = false;
  float target = 0.f;
  if (threadIdx.x == kThreads - 1) target = target_logit<ST>(a, t, has);  // asked for early, used at the end
  if (warp == 0) {
    Part p{neg_inf(), 0.f, 0.f};
#pragma unroll 1
    for (int i = lane; i < plan.splits; i += 32) {
      const float4 v = a.part[1LL * t * plan.splits + i];
      p = join(p, Part{v.x, v.y, v.z}, c);
    }
    p = warp_join(p, c);
    if (lane == 0) s.part = p;
  }
  const ST* row = static_cast<const ST*>(a.logits) + t * a.ld;
  const int shift = lead(row);
  const int nseg = (a.V + shift + kLogprobSeg - 1) / kLogprobSeg;  // of this row
  if (K > 0) {  // the K best segments (all where there are fewer)
    const float* segmax = a.segmax + 1LL * t * plan.nseg;
    reach_bound(K, s, [&](auto&& use) {
      for (int i = threadIdx.x; i < nseg; i += kThreads) use(key_of(segmax[i], i));
    });
    rank_keys(s, K, [&](int rank, unsigned long long k) { s.picked[rank] = place_of(k); });
  }
  __syncthreads();
  if (threadIdx.x == kThreads - 1) finish(a, t, s.part, target, has);
  if (K == 0) return;
  // The K largest logits of these segments.
  constexpr int kPer = kLogprobSeg / kGroup;
  const int groups = min(K, nseg) * kPer;
  reach_bound(K, s, [&](auto&& use) {
#pragma unroll 4
    for (int g = threadIdx.x; g < groups; g += kThreads) {
      const int i = s.picked[g / kPer] * kLogprobSeg + g % kPer * kGroup - shift;
      float v[kGroup];
      load_group(row, i, a.V, v);
#pragma unroll
      for (int e = 0; e < kGroup; ++e)
        if (i + e >= 0 && i + e < a.V) use(key_of(v[e], i + e));
    }
  });
  rank_keys(s, K, [&](int rank, unsigned long long k) {
    a.top_ids[1LL * t * K + rank] = place_of(k);
    a.top_logp[1LL * t * K + rank] = log_prob(value_of(k), s.part, a.scale);
  });
}

// The gradient of a row, d_j = scale (p_j (-de (lp_j + H) - dl) + [j = target] dl) = p_j (e lp_j + f) + [j = target] hit.
struct Grad {
  int k;
  float e, f, hit;
};

// e^x of the gradient: bf16 takes the hardware approximation of 2^x (its 2^-22 is far below the rounding of the result),
// fp32 the library's exponential, whose rounding a factor of log2 e would double.
template <typename ST>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (sizeof(ST) == 2) return ex2(x * kLog2e);
  else return expf(x);
}

// Up to here the rounding of lse (2^-24 of it, which p takes over as it is) is taken: 2^-14 of p for bf16, a 64th of
// the result's own rounding, and 2^-18 for fp32, what log p = 64 costs anyway.  Beyond, far_row takes longer: 4096 rows of
// 131072 in bf16 310 us on this side and 486 on the other (three passes over the logits are 475), 2048 in fp32 312 and 513,
// a single row of bf16 7 and 31.
template <typename ST>
constexpr float kFarLse = sizeof(ST) == 2 ? 1024.f : 64.f;

// Places begin .. end - 1 of a row (counted from the 16-byte boundary before it) and of its gradient: `gradient` makes a
// group of logits from place `at` on into its gradient, or all are 0 without being read.
template <typename ST, typename F>
__device__ __forceinline__ void write_gradient(const ST* row, ST* out, int V, int begin, int end, bool zero, F gradient) {
  const int shift = lead(row), oshift = lead(out);
  constexpr int kU = kUnroll<ST>, kStride = kThreads * kGroup;
  const bool whole = oshift == shift;  // both rows can be taken in aligned groups
  for (int i = begin; i < end; i += kU * kStride) {
    const int at = i + threadIdx.x * kGroup - shift;
    float v[kU][kGroup];
    if (whole && i >= shift && i + kU * kStride <= end && i + kU * kStride <= V + shift) {
      if (zero) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int n = 0; n < kGroup; ++n) v[u][n] = 0.f;
      } else {
        load_groups(row + at, kStride, v);
#pragma unroll
        for (int u = 0; u < kU; ++u) gradient(v[u], at + u * kStride);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) store8(out + at + u * kStride, v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = at + u * kStride;
        if (j + shift >= end) break;
        if (zero) {
#pragma unroll
          for (int n = 0; n < kGroup; ++n) v[u][n] = 0.f;
        } else {
          load_group(row, j, V, v[u]);
          gradient(v[u], j);
        }
        if (whole && j >= 0 && j + kGroup <= V) {
          store8(out + j, v[u]);
        } else {
#pragma unroll
          for (int n = 0; n < kGroup; ++n)
            if (j + n >= 0 && j + n < V) out[j + n] = from_float<ST>(v[u][n]);
        }
      }
    }
  }
}

__device__ __forceinline__ void add_hit(float* v, int at, const Grad& g) {
  if (static_cast<unsigned>(g.k - at) < kGroup && g.hit != 0.f) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (at + i == g.k) v[i] += g.hit;
  }
}

// A whole row whose lse does not tell its probabilities: rounded, it has lost log s (logits that share a large offset,
// or masks of the type's lowest value alone), or it is not finite.  One block takes the row's m and s again and then log p
// from differences to m, as the forward does; it reads the row twice, and before it writes any of it (the gradient may
// take the logits' place).
template <typename ST, bool ENTROPY>
__device__ __noinline__ void far_row(const ST* row, ST* out, int V, float scale, Grad g) {
  __shared__ Part warps[kWarps];
  const float c = scale * kLog2e;
  const int shift = lead(row);
  constexpr int kU = kUnroll<ST>, kStride = kThreads * kGroup;
  Part p{neg_inf(), 0.f, 0.f};
  for (int i = 0; i < V + shift; i += kU * kStride) {
    const int at = i + threadIdx.x * kGroup - shift;
    float v[kU][kGroup], m = neg_inf();
    if (i >= shift && i + kU * kStride <= V + shift) {
      load_groups(row + at, kStride, v);
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) load_group(row, at + u * kStride, V, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < kGroup; ++n) m = max_nan(m, v[u][n]);
    if (!(m <= p.m)) p = join(p, Part{m, 0.f, 0.f}, c);
    if (p.m > neg_inf()) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < kGroup; ++n) s += ex2(fmaxf(c * (v[u][n] - p.m), kFloor));
        p.s += s;
      }
    }
  }
  p = warp_join(p, c);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = p;
  __syncthreads();
  p = warps[0];
#pragma unroll 1
  for (int i = 1; i < kWarps; ++i) p = join(p, warps[i], c);
  const float log_s = kLn2 * log2f(p.s), bad = p.m <= kMax ? 0.f : __int_as_float(0x7fc00000);  // a NaN or +inf in the row
  write_gradient(row, out, V, 0, V + shift, p.m == neg_inf(), [&](float* v, int at) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const float lp = fmaxf(fmaf(scale, v[i] - p.m, -log_s), kFloor);
      v[i] = fmaf(exp_of<ST>(lp), ENTROPY ? fmaf(g.e, lp, g.f) : g.f, bad);
    }
    add_hit(v, at, g);
  });
}

template <typename ST, bool ENTROPY>
__global__ void __launch_bounds__(kThreads, 4) logprob_bwd_kernel(LogprobBwd a, int chunks, int chunk) {
  const int t = static_cast<int>(blockIdx.x / chunks), part = static_cast<int>(blockIdx.x - 1u * t * chunks);
  const ST* row = static_cast<const ST*>(a.logits) + t * a.ld;
  ST* out = static_cast<ST*>(a.out) + t * a.ldo;
  pdl_wait();
  const int k = a.target[t];
  const float lse = a.lse[t], given = a.dlogp[t];
  const float de = ENTROPY ? a.dentropy[t] : 0.f, h = ENTROPY ? a.entropy[t] : 0.f;
  const float dl = k >= 0 && k < a.V ? given : 0.f;
  Grad g;
  g.k = k;
  g.e = -de * a.scale;
  g.hit = dl * a.scale;
  g.f = fmaf(g.e, h, -g.hit);
  const bool zero = dl == 0.f && de == 0.f;  // no gradient
  if (!zero && !(fabsf(lse) <= kFarLse<ST>)) {
    if (part == 0) far_row<ST, ENTROPY>(row, out, a.V, a.scale, g);
    return;
  }
  const long long begin = 1LL * part * chunk;
  const int end = static_cast<int>(min(begin + chunk, 1LL * a.V + lead(row)));
  write_gradient(row, out, a.V, static_cast<int>(begin), end, zero, [&](float* v, int at) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const float lp = fmaxf(fmaf(v[i], a.scale, -lse), kFloor);
      v[i] = exp_of<ST>(lp) * (ENTROPY ? fmaf(g.e, lp, g.f) : g.f);
    }
    add_hit(v, at, g);
  });
}

}  // namespace

LogprobPlan logprob_plan(int T, int V, int es, int sms) {
  LogprobPlan p;
  const int most = V + 16 / es - 1;  // places of a row, counted from a 16-byte boundary
  p.nseg = (most + kLogprobSeg - 1) / kLogprobSeg;
  // One block to a row where there are eight an SM (four of bf16 or six of fp32 run at a time); else a row over several, each
  // with one load of half its threads at least.  515 rows of 50021 in fp32: 34.9 us when cut for 15 blocks an SM, 33.6 for 8, 36.5
  // for 6; 1500 rows in bf16: 43.9, 39.2, 39.1.
  const int fit = (most + 4095) / 4096;
  const int want = (8 * sms + T - 1) / T;
  const int s = std::min({want, fit, kLogprobMaxSplits});
  p.chunk = ((most + s - 1) / s + 1023) / 1024 * 1024;
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
cudaError_t launch_logprob_bwd(const LogprobBwd& a, int sms, cudaStream_t st) {
  // Chunks of up to four rounds of a block's loads, so that the row's scalars are read less often; of one where there are
  // not enough for eight blocks an SM.
  constexpr int step = kThreads * kGroup * kUnroll<ST>;
  const int steps = (a.V + 16 / static_cast<int>(sizeof(ST)) - 1 + step - 1) / step;
  const long long rounds = 1LL * a.T * steps / (8LL * sms);
  const int per = static_cast<int>(std::max(1LL, std::min({rounds, 4LL, 1LL * steps})));
  const int chunks = (steps + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(1LL * a.T * chunks));
  return a.dentropy ? launch_pdl(logprob_bwd_kernel<ST, true>, grid, dim3(kThreads), 0, st, a, chunks, per * step)
                    : launch_pdl(logprob_bwd_kernel<ST, false>, grid, dim3(kThreads), 0, st, a, chunks, per * step);
}

#define LR_INSTANTIATE(ST)                                                                         \
  template cudaError_t launch_logprob_fwd<ST>(const LogprobFwd&, const LogprobPlan&, cudaStream_t);  \
  template cudaError_t launch_logprob_join<ST>(const LogprobFwd&, const LogprobPlan&, cudaStream_t); \
  template cudaError_t launch_logprob_bwd<ST>(const LogprobBwd&, int, cudaStream_t);
LR_INSTANTIATE(bf16)
LR_INSTANTIATE(float)
#undef LR_INSTANTIATE

}  // namespace lr
