#include "qk_kernels.cuh"

#include "small_kernels.cuh"

namespace lr {

// Angle of pair p for the positions of token t.  pos * turns wraps at 2^64, a whole number of turns, so the
// product is exact for any position; the top 32 bits, signed, are the angle in [-1/2, 1/2] turns.
__device__ __forceinline__ void turn_of(const QkArgs& a, int t, int p, float* c, float* s) {
  const int axis = (p >= a.sec_end[0]) + (p >= a.sec_end[1]) + (p >= a.sec_end[2]);
  const long long pos = a.pos ? a.pos[static_cast<long long>(axis) * a.T + t] : t % a.seq;
  const unsigned long long ph = static_cast<unsigned long long>(pos) * a.turns[p];
  const int top = static_cast<int>((ph + 0x80000000ull) >> 32);
  sincospif(static_cast<float>(top) * 0x1p-31f, s, c);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per (token, head) vector; each lane owns whole channel pairs, so an output may take its input's place.
template <typename ST, bool ADJ>
__global__ void qk_fwd_kernel(QkArgs a) {
  pdl_wait();
  pdl_trigger();
  const long long v = (blockIdx.x * 256LL + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const QkTensor& q = a.t[blockIdx.y];
  if (v >= 1LL * a.T * q.H) return;
  const int t = static_cast<int>(v / q.H), h = static_cast<int>(v % q.H);
  const ST* x = static_cast<const ST*>(q.x) + t * q.ldx + 1LL * h * a.dh;
  ST* y = static_cast<ST*>(q.out) + t * q.ldo + 1LL * h * a.dh;
  const ST* g = static_cast<const ST*>(q.g);
  float r = 1.f;
  if (g) {
    float ss = 0.f;
    for (int c = lane; c < a.dh; c += 32) {
      const float w = static_cast<float>(x[c]);
      ss = fmaf(w, w, ss);
    }
    r = 1.f / sqrtf(warp_sum(ss) / static_cast<float>(a.dh) + a.eps);
  }
  for (int p = lane; p < a.rot / 2; p += 32) {
    const int i = ADJ ? 2 * p : p, j = ADJ ? 2 * p + 1 : p + a.rot / 2;
    float c, s, u = static_cast<float>(x[i]), w = static_cast<float>(x[j]);
    if (g) {
      u *= r * static_cast<float>(g[i]);
      w *= r * static_cast<float>(g[j]);
    }
    turn_of(a, t, p, &c, &s);
    y[i] = static_cast<ST>(u * c - w * s);
    y[j] = static_cast<ST>(u * s + w * c);
  }
  for (int i = a.rot + lane; i < a.dh; i += 32) {
    float u = static_cast<float>(x[i]);
    if (g) u *= r * static_cast<float>(g[i]);
    y[i] = static_cast<ST>(u);
  }
}

// A block of 8 warps takes the vectors blockIdx.x * 8 + warp, + gridDim.x * 8, ...; the sums of dg live in
// shared memory, one row per warp, and are added in warp order at the end.
template <typename ST, bool ADJ>
__global__ void qk_bwd_kernel(QkArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float sums[];  // [8][dh]
  const QkTensor& q = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const ST* g = static_cast<const ST*>(q.g);
  float* mine = sums + warp * a.dh;
  for (int c = lane; c < a.dh; c += 32) mine[c] = 0.f;
  const long long n = 1LL * a.T * q.H;
  const int half = a.rot / 2;
  for (long long v = blockIdx.x * 8LL + warp; v < n; v += gridDim.x * 8LL) {
    const int t = static_cast<int>(v / q.H), h = static_cast<int>(v % q.H);
    const ST* x = static_cast<const ST*>(q.x) + t * q.ldx + 1LL * h * a.dh;
    const ST* dy = static_cast<const ST*>(q.dy) + t * q.lddy + 1LL * h * a.dh;
    ST* dx = static_cast<ST*>(q.out) + t * q.ldo + 1LL * h * a.dh;
    float r = 1.f, m = 0.f;
    if (g) {
      float ss = 0.f;
      for (int c = lane; c < a.dh; c += 32) {
        const float w = static_cast<float>(x[c]);
        ss = fmaf(w, w, ss);
      }
      r = 1.f / sqrtf(warp_sum(ss) / static_cast<float>(a.dh) + a.eps);
    }
    // pass 0 sums w x and dg, pass 1 writes dx
    for (int pass = g ? 0 : 1; pass < 2; ++pass) {
      float dot = 0.f;
      auto channel = [&](int i, float dn) {
        if (!g) {
          dx[i] = static_cast<ST>(dn);
          return;
        }
        const float xi = static_cast<float>(x[i]), w = dn * static_cast<float>(g[i]);
        if (pass == 0) {
          dot = fmaf(w, xi, dot);
          mine[i] += dn * (xi * r);
        } else {
          dx[i] = static_cast<ST>(r * (w - xi * m));
        }
      };
      for (int p = lane; p < half; p += 32) {
        const int i = ADJ ? 2 * p : p, j = ADJ ? 2 * p + 1 : p + half;
        const float u = static_cast<float>(dy[i]), w = static_cast<float>(dy[j]);
        float c, s;
        turn_of(a, t, p, &c, &s);
        channel(i, u * c + w * s);
        channel(j, w * c - u * s);
      }
      for (int i = a.rot + lane; i < a.dh; i += 32) channel(i, static_cast<float>(dy[i]));
      if (pass == 0) m = warp_sum(dot) * r * r / static_cast<float>(a.dh);
    }
  }
  if (!g) return;
  __syncthreads();
  for (int c = threadIdx.x; c < a.dh; c += 256) {
    float v = 0.f;
    for (int w = 0; w < 8; ++w) v += sums[w * a.dh + c];
    q.part[static_cast<long long>(blockIdx.x) * a.dh + c] = v;
  }
}

static QkArgs only(const QkArgs& a, int i) {
  QkArgs b = a;
  b.t[0] = a.t[i];
  return b;
}

template <typename ST>
cudaError_t launch_qk_fwd(const QkArgs& a, bool adjacent, cudaStream_t st) {
  for (int i = 0; i < 2; ++i) {
    if (a.t[i].H == 0) continue;
    const long long n = 1LL * a.T * a.t[i].H;
    const dim3 grid(static_cast<unsigned>((n + 7) / 8));
    cudaError_t e = adjacent ? launch_pdl(qk_fwd_kernel<ST, true>, grid, dim3(256), 0, st, only(a, i))
                             : launch_pdl(qk_fwd_kernel<ST, false>, grid, dim3(256), 0, st, only(a, i));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename ST>
cudaError_t launch_qk_bwd(const QkArgs& a, bool adjacent, cudaStream_t st) {
  for (int i = 0; i < 2; ++i) {
    if (a.t[i].H == 0) continue;
    const long long n = 1LL * a.T * a.t[i].H;
    const int blocks = static_cast<int>((n + 7) / 8 < kQkMaxParts ? (n + 7) / 8 : kQkMaxParts);
    const size_t smem = sizeof(float) * 8 * a.dh;
    cudaError_t e = adjacent ? launch_pdl(qk_bwd_kernel<ST, true>, dim3(blocks), dim3(256), smem, st, only(a, i))
                             : launch_pdl(qk_bwd_kernel<ST, false>, dim3(blocks), dim3(256), smem, st, only(a, i));
    if (e != cudaSuccess) return e;
    if (a.t[i].g) {
      e = launch_dg_finalize(a.t[i].part, blocks, a.dh, a.t[i].dg, st);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

#define LR_QK_INST(ST)                                                          \
  template cudaError_t launch_qk_fwd<ST>(const QkArgs&, bool, cudaStream_t); \
  template cudaError_t launch_qk_bwd<ST>(const QkArgs&, bool, cudaStream_t);
LR_QK_INST(float)
LR_QK_INST(bf16)
#undef LR_QK_INST

}  // namespace lr
