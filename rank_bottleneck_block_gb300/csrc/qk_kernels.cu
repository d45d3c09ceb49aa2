// A vector (one head of one token) lies over G lanes of a warp, a lane holding 2 U of its channels ("a slot") such
// that both channels of every pair are in the same lane: two runs of U channels, rot / 2 apart (pairs (p, p + rot/2))
// or adjacent (pairs (2p, 2p + 1)); slots past the turned channels hold 2 U neighbouring channels.  So a vector is
// read once with 16-byte loads (8-byte ones for bf16 whose dh or rot is no multiple of 16), its sums take log2 G
// shuffles, and an output may take its input's place.  A warp takes one token and a run of its heads, 32 / G at a
// time: a lane's slot stays the same, so its angles are computed once for all of them and its gains stay in registers.
#include "qk_kernels.cuh"

namespace lr {

// A run of U channels as stored: kept packed while several vectors are in flight.
template <typename ST, int U>
struct alignas(sizeof(ST) * U < 16 ? sizeof(ST) * U : 16) Run {
  ST v[U];
};

template <typename ST, int U>
__device__ __forceinline__ void get(const ST* p, Run<ST, U>& r) {
  r = *reinterpret_cast<const Run<ST, U>*>(p);
}
template <int U>
__device__ __forceinline__ void unpack(const Run<bf16, U>& r, float* v) {
#pragma unroll
  for (int i = 0; i < U; i += 2) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.v[i]));
    v[i] = f.x;
    v[i + 1] = f.y;
  }
}
template <int U>
__device__ __forceinline__ void unpack(const Run<float, U>& r, float* v) {
#pragma unroll
  for (int i = 0; i < U; ++i) v[i] = r.v[i];
}
template <int U>
__device__ __forceinline__ void put(bf16* p, const float* v) {
  Run<bf16, U> r;
#pragma unroll
  for (int i = 0; i < U; i += 2)
    *reinterpret_cast<__nv_bfloat162*>(&r.v[i]) = __floats2bfloat162_rn(v[i], v[i + 1]);
  *reinterpret_cast<Run<bf16, U>*>(p) = r;
}
template <int U>
__device__ __forceinline__ void put(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < U; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// The lane's slot: where its two runs start, and whether its channels are turned.
struct Slot {
  int o0, o1, pair;  // pair: the first of the slot's U pairs
  bool on, turned;
};
template <int U, bool ADJ, int G>
__device__ __forceinline__ Slot slot_of(const QkArgs& a) {
  const int j = threadIdx.x % G, n = a.rot / (2 * U);
  Slot s;
  s.on = j < a.dh / (2 * U);
  s.turned = s.on && j < n;
  s.pair = j * U;
  s.o0 = ADJ ? 2 * U * j : s.turned ? U * j : a.rot + 2 * U * (j - n);
  s.o1 = !ADJ && s.turned ? s.o0 + a.rot / 2 : s.o0 + U;
  return s;
}

// Cosines and sines of the slot's pairs at token t.  pos * turns wraps at 2^64, a whole number of turns, so the
// product is exact for any position; its top 32 bits, signed, are the angle in [-1/2, 1/2] turns.  For bf16 outputs
// the hardware sine and cosine serve (off by 2^-21.2 at most on [-pi, pi], against a rounding of 2^-9).
template <typename ST, int U>
__device__ __forceinline__ void slot_angles(const QkArgs& a, const Slot& sl, int t, float* c, float* s) {
  if (!sl.turned) return;
  if (a.pos == nullptr) t %= a.seq;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int p = sl.pair + i;
    const int axis = (p >= a.sec_end[0]) + (p >= a.sec_end[1]) + (p >= a.sec_end[2]);
    const long long pos = a.pos ? a.pos[static_cast<long long>(axis) * a.T + t] : t;
    const unsigned long long ph = static_cast<unsigned long long>(pos) * a.turns[p];
    const float top = static_cast<float>(static_cast<int>((ph + 0x80000000ull) >> 32));
    if constexpr (sizeof(ST) == 2) __sincosf(top * 1.46291807926715968e-9f /* 2 pi / 2^32 */, &s[i], &c[i]);
    else sincospif(top * 0x1p-31f, &s[i], &c[i]);
  }
}

// Turns the slot's pairs of (u, v), its two runs, by +angle (SIGN = 1) or -angle (-1).
template <int U, bool ADJ, int SIGN>
__device__ __forceinline__ void turn(float* u, float* v, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float& x = ADJ ? (2 * i < U ? u[2 * i] : v[2 * i - U]) : u[i];
    float& y = ADJ ? (2 * i < U ? u[2 * i + 1] : v[2 * i + 1 - U]) : v[i];
    const float sn = SIGN > 0 ? s[i] : -s[i];
    const float x1 = x * c[i] - y * sn;
    y = x * sn + y * c[i];
    x = x1;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kWarps = 8;   // most warps of a block
constexpr int kFlight = 2;  // vectors of a lane in flight
template <typename ST, int U>
constexpr int kBwdBlocks = sizeof(ST) * U > 16 ? 1 : 2;  // backward blocks an SM holds

template <typename ST, int U, bool ADJ, int G>
__global__ void __launch_bounds__(kWarps * 32) qk_fwd_kernel(const __grid_constant__ QkArgs a,
                                                             const __grid_constant__ QkPlan pl) {
  pdl_wait();
  pdl_trigger();
  constexpr int P = 32 / G;
  const int which = blockIdx.x < static_cast<unsigned>(pl.blocks[0]) ? 0 : 1;
  const QkTensor& q = a.t[which];
  const unsigned item = (blockIdx.x - (which ? pl.blocks[0] : 0)) * (blockDim.x / 32) + threadIdx.x / 32;
  const unsigned chunks = pl.chunks[which];
  const int t = static_cast<int>(item / chunks);
  if (t >= a.T) return;
  const int hn = pl.passes[which] * P, h0 = static_cast<int>(item % chunks) * hn;
  const int h1 = min(q.H, h0 + hn);
  const int sub = (threadIdx.x % 32) / G;
  const Slot sl = slot_of<U, ADJ, G>(a);
  const ST* x = static_cast<const ST*>(q.x) + t * q.ldx;
  ST* y = static_cast<ST*>(q.out) + t * q.ldo;
  const ST* g = static_cast<const ST*>(q.g);
  float c[U], s[U];
  Run<ST, U> g0 = {}, g1 = {}, r0[kFlight] = {}, r1[kFlight] = {};
  auto fetch = [&](int h, int f) {
    if (h < h1 && sl.on) {
      get(x + h * a.dh + sl.o0, r0[f]);
      get(x + h * a.dh + sl.o1, r1[f]);
    }
  };
#pragma unroll
  for (int f = 0; f < kFlight; ++f) fetch(h0 + f * P + sub, f);
  if (g && sl.on) {
    get(g + sl.o0, g0);
    get(g + sl.o1, g1);
  }
  slot_angles<ST, U>(a, sl, t, c, s);
  const float inv_dh = 1.f / static_cast<float>(a.dh);
  for (int h = h0 + sub; h < h0 + hn; h += kFlight * P) {  // the same number of rounds for every lane
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      float u[U], v[U];
      unpack<U>(r0[f], u);
      unpack<U>(r1[f], v);
      const int hf = h + f * P;
      fetch(hf + kFlight * P, f);
      if (g) {
        float ss = 0.f;
        if (sl.on) {
#pragma unroll
          for (int i = 0; i < U; ++i) ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
        }
        const float r = 1.f / sqrtf(group_sum<G>(ss) * inv_dh + a.eps);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          u[i] *= r * static_cast<float>(g0.v[i]);
          v[i] *= r * static_cast<float>(g1.v[i]);
        }
      }
      if (sl.turned) turn<U, ADJ, 1>(u, v, c, s);
      if (hf < h1 && sl.on) {
        put<U>(y + hf * a.dh + sl.o0, u);
        put<U>(y + hf * a.dh + sl.o1, v);
      }
    }
  }
}

// A warp's items: tokens x runs of heads of one tensor, blocks[] warps apart, so its gain sums stay in registers; they
// are added over the warp's lane groups, then over the block's warps, and each block leaves one row of partial sums.
// The sums over a vector's channels, mean(x^2) and mean(w x), are independent of one another and reduced together.
template <typename ST, int U, bool ADJ, int G>
__global__ void __launch_bounds__(kWarps * 32, kBwdBlocks<ST, U>) qk_bwd_kernel(const __grid_constant__ QkArgs a,
                                                                                const __grid_constant__ QkPlan pl) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float4 sums4[];
  float* sums = reinterpret_cast<float*>(sums4);  // [warps][dh]
  constexpr int P = 32 / G;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const int which = blockIdx.x < static_cast<unsigned>(pl.blocks[0]) ? 0 : 1;
  const QkTensor& q = a.t[which];
  const unsigned block = blockIdx.x - (which ? pl.blocks[0] : 0);
  const unsigned chunks = pl.chunks[which], items = chunks * a.T;
  const int hn = pl.passes[which] * P, sub = (threadIdx.x % 32) / G;
  const Slot sl = slot_of<U, ADJ, G>(a);
  const ST* g = static_cast<const ST*>(q.g);
  const float inv_dh = 1.f / static_cast<float>(a.dh);
  Run<ST, U> g0 = {}, g1 = {};
  float d0[U], d1[U];
#pragma unroll
  for (int i = 0; i < U; ++i) d0[i] = d1[i] = 0.f;
  if (g && sl.on) {
    get(g + sl.o0, g0);
    get(g + sl.o1, g1);
  }
  for (unsigned item = block * warps + warp; item < items; item += pl.blocks[which] * warps) {
    const int t = static_cast<int>(item / chunks);
    const int h0 = static_cast<int>(item % chunks) * hn;
    const int h1 = min(q.H, h0 + hn);
    const ST* x = static_cast<const ST*>(q.x) + t * q.ldx;
    const ST* dy = static_cast<const ST*>(q.dy) + t * q.lddy;
    ST* dx = static_cast<ST*>(q.out) + t * q.ldo;
    float c[U], s[U];
    Run<ST, U> x0[kFlight] = {}, x1[kFlight] = {}, y0[kFlight] = {}, y1[kFlight] = {};
    auto fetch = [&](int h, int f) {
      if (h < h1 && sl.on) {
        get(dy + h * a.dh + sl.o0, y0[f]);
        get(dy + h * a.dh + sl.o1, y1[f]);
        if (g) {
          get(x + h * a.dh + sl.o0, x0[f]);
          get(x + h * a.dh + sl.o1, x1[f]);
        }
      }
    };
#pragma unroll
    for (int f = 0; f < kFlight; ++f) fetch(h0 + f * P + sub, f);
    slot_angles<ST, U>(a, sl, t, c, s);
    for (int h = h0 + sub; h < h0 + hn; h += kFlight * P) {
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int hf = h + f * P;
        const bool on = hf < h1 && sl.on;
        float u[U], v[U], p[U], w[U];
        unpack<U>(y0[f], u);
        unpack<U>(y1[f], v);
        unpack<U>(x0[f], p);
        unpack<U>(x1[f], w);
        fetch(hf + kFlight * P, f);
        if (sl.turned) turn<U, ADJ, -1>(u, v, c, s);
        if (g) {
          float ss = 0.f, dot = 0.f;
          if (on) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
              ss = fmaf(p[i], p[i], fmaf(w[i], w[i], ss));
              dot = fmaf(u[i] * static_cast<float>(g0.v[i]), p[i],
                         fmaf(v[i] * static_cast<float>(g1.v[i]), w[i], dot));
            }
          }
          ss = group_sum<G>(ss);
          dot = group_sum<G>(dot);
          const float r = 1.f / sqrtf(ss * inv_dh + a.eps);
          const float m = dot * inv_dh * r * r;
          if (on) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
              d0[i] = fmaf(u[i], p[i] * r, d0[i]);
              d1[i] = fmaf(v[i], w[i] * r, d1[i]);
              u[i] = r * (u[i] * static_cast<float>(g0.v[i]) - p[i] * m);
              v[i] = r * (v[i] * static_cast<float>(g1.v[i]) - w[i] * m);
            }
          }
        }
        if (on) {
          put<U>(dx + hf * a.dh + sl.o0, u);
          put<U>(dx + hf * a.dh + sl.o1, v);
        }
      }
    }
  }
  if (!g) return;
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      d0[i] += __shfl_xor_sync(0xffffffffu, d0[i], o);
      d1[i] += __shfl_xor_sync(0xffffffffu, d1[i], o);
    }
  }
  if (sub == 0 && sl.on) {
    put<U>(sums + warp * a.dh + sl.o0, d0);
    put<U>(sums + warp * a.dh + sl.o1, d1);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.dh; c += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += sums[w * a.dh + c];
    q.part[static_cast<long long>(block) * a.dh + c] = v;
  }
}

// dg of both tensors from their blocks' rows, in a fixed order: 32 channels a block, every 32nd row a thread.
__global__ void __launch_bounds__(1024) qk_dg_kernel(const __grid_constant__ QkArgs a,
                                                     const __grid_constant__ QkPlan pl) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[32][33];
  const QkTensor& q = a.t[blockIdx.y];
  if (!q.g || q.H == 0) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < a.dh)
    for (int p = threadIdx.y; p < pl.blocks[blockIdx.y]; p += 32) v += q.part[static_cast<long long>(p) * a.dh + c];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = red[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < a.dh) q.dg[cc] = v;
}

// --------------------------------------------------------------- dispatch
struct QkVariant {
  int u, g;  // channels of a run, lanes of a vector
};

// Runs of 8 channels where a bf16 vector divides into them (16-byte loads), else of 4; fp32 takes 4 (16 bytes too)
// but for vectors of more than 256 channels, which then fill a warp.
static QkVariant variant(const QkArgs& a, size_t es) {
  const bool wide = a.dh % 16 == 0 && a.rot % 16 == 0 && (es == 2 || a.dh > 256);
  const int u = wide ? 8 : 4, slots = a.dh / (2 * u);
  return {u, slots <= 4 && es == 2 ? 4 : slots <= 8 ? 8 : slots <= 16 ? 16 : 32};
}

static int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// How the heads of each tensor are cut: as many passes to a warp as leave `warps` of them, so that angles and gains
// are reused; never more than 64 runs a token (tokens x runs stay below 2^30).
static void cut_heads(const QkArgs& a, int g, long long warps, QkPlan* pl) {
  long long all = 0;
  int full[2];
  for (int i = 0; i < 2; ++i) {
    full[i] = cdiv(a.t[i].H, 32 / g);
    all += 1LL * a.T * full[i];
  }
  const long long n = all / warps;
  for (int i = 0; i < 2; ++i) {
    int passes = static_cast<int>(n < 1 ? 1 : n < full[i] ? n : full[i]);
    if (passes < cdiv(full[i], 64)) passes = cdiv(full[i], 64);
    pl->chunks[i] = full[i] ? cdiv(full[i], passes) : 0;
    pl->passes[i] = full[i] ? cdiv(full[i], pl->chunks[i]) : 0;
  }
}

using QkKernel = void (*)(QkArgs, QkPlan);

template <typename ST, int U, bool ADJ>
static QkKernel pick_g(bool bwd, int g) {
  if constexpr (sizeof(ST) * U == 32) {  // fp32 runs of 8: whole warps only
    return bwd ? qk_bwd_kernel<ST, U, ADJ, 32> : qk_fwd_kernel<ST, U, ADJ, 32>;
  } else {
    switch (g) {
      case 4:
        if constexpr (sizeof(ST) == 2) return bwd ? qk_bwd_kernel<ST, U, ADJ, 4> : qk_fwd_kernel<ST, U, ADJ, 4>;
      case 8: return bwd ? qk_bwd_kernel<ST, U, ADJ, 8> : qk_fwd_kernel<ST, U, ADJ, 8>;
      case 16: return bwd ? qk_bwd_kernel<ST, U, ADJ, 16> : qk_fwd_kernel<ST, U, ADJ, 16>;
      default: return bwd ? qk_bwd_kernel<ST, U, ADJ, 32> : qk_fwd_kernel<ST, U, ADJ, 32>;
    }
  }
}

template <typename ST>
static QkKernel pick(bool bwd, bool adj, QkVariant v) {
  if (v.u == 8) return adj ? pick_g<ST, 8, true>(bwd, v.g) : pick_g<ST, 8, false>(bwd, v.g);
  return adj ? pick_g<ST, 4, true>(bwd, v.g) : pick_g<ST, 4, false>(bwd, v.g);
}

template <typename ST>
cudaError_t launch_qk_fwd(const QkArgs& a, bool adjacent, int sms, cudaStream_t st) {
  const QkVariant v = variant(a, sizeof(ST));
  QkPlan pl;
  cut_heads(a, v.g, sms * 32LL, &pl);
  const long long items = 1LL * a.T * (pl.chunks[0] + pl.chunks[1]);
  const int warps = items >= sms * 8LL * kWarps ? kWarps : items >= sms * 8LL ? 4 : 1;
  for (int i = 0; i < 2; ++i) pl.blocks[i] = cdiv(1LL * a.T * pl.chunks[i], warps);
  return launch_pdl(pick<ST>(false, adjacent, v), dim3(pl.blocks[0] + pl.blocks[1]), dim3(32 * warps), 0, st, a, pl);
}

template <typename ST>
cudaError_t launch_qk_bwd(const QkArgs& a, bool adjacent, int sms, cudaStream_t st) {
  const QkVariant v = variant(a, sizeof(ST));
  QkPlan pl;
  cut_heads(a, v.g, sms * 16LL, &pl);
  long long passes[2], items[2];
  for (int i = 0; i < 2; ++i) {
    items[i] = 1LL * a.T * pl.chunks[i];
    passes[i] = items[i] * pl.passes[i];
  }
  const int warps = items[0] + items[1] >= sms * 2LL * kWarps ? kWarps : 2;
  // two blocks an SM, shared between the tensors by their work
  const int room = sms * 2;
  for (int i = 0; i < 2; ++i) {
    long long n = (passes[i] * room + (passes[0] + passes[1]) / 2) / (passes[0] + passes[1]);
    if (n < 1) n = 1;
    if (n > cdiv(items[i], warps)) n = cdiv(items[i], warps);
    pl.blocks[i] = static_cast<int>(n < kQkMaxParts ? n : kQkMaxParts);
  }
  cudaError_t e = launch_pdl(pick<ST>(true, adjacent, v), dim3(pl.blocks[0] + pl.blocks[1]), dim3(32 * warps),
                             sizeof(float) * warps * a.dh, st, a, pl);
  if (e != cudaSuccess || (!a.t[0].g && !a.t[1].g)) return e;
  return launch_pdl(qk_dg_kernel, dim3(cdiv(a.dh, 32), 2), dim3(32, 32), 0, st, a, pl);
}

#define LR_QK_INST(ST)                                                             \
  template cudaError_t launch_qk_fwd<ST>(const QkArgs&, bool, int, cudaStream_t); \
  template cudaError_t launch_qk_bwd<ST>(const QkArgs&, bool, int, cudaStream_t);
LR_QK_INST(float)
LR_QK_INST(bf16)
#undef LR_QK_INST

}  // namespace lr
