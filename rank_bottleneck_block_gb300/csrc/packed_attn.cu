// lr_packed_attn_bwd, the plain form: a warp per row and head (dk, dv: per row and key head), each lane four channels,
// one key (or query) at a time.
#include "packed_attn.cuh"

#include <algorithm>

namespace lr {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Channels lane, lane + 32, ... of head h of row t.
struct Vec {
  float v[4];
};
__device__ __forceinline__ Vec load(const PackedRows& x, long long t, int h, int dh) {
  Vec r;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = lane + 32 * i;
    r.v[i] = c < dh ? __bfloat162float(x.p[t * x.ld + 1LL * h * dh + c]) : 0.f;
  }
  return r;
}
__device__ __forceinline__ void store(const PackedRows& x, long long t, int h, int dh, const Vec& r) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < dh) x.p[t * x.ld + 1LL * h * dh + lane + 32 * i] = __float2bfloat16_rn(r.v[i]);
}
__device__ __forceinline__ float dot(const Vec& a, const Vec& b) {
  return warp_sum(a.v[0] * b.v[0] + a.v[1] * b.v[1] + a.v[2] * b.v[2] + a.v[3] * b.v[3]);
}
__device__ __forceinline__ void axpy(Vec& a, float f, const Vec& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a.v[i] = fmaf(f, b.v[i], a.v[i]);
}

// Checks the offsets: ws[0] = 1 where they are in order.
__global__ void check_kernel(PackedArgs a, int* ok, unsigned* err) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i <= a.nseq; i += blockDim.x) {
    const int b = i ? a.offs[i - 1] : 0, e = a.offs[i];
    if (e < b || e > a.T) bad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *ok = !bad;
    if (bad) atomicOr(err, DEV_ERR_OFFSETS);
  }
}

// The sequence of row t: false where there is none.
__device__ __forceinline__ bool sequence(const PackedArgs& a, int t, int& begin, int& end) {
  if (t < a.offs[0] || t >= a.offs[a.nseq]) return false;
  int lo = 0, hi = a.nseq;  // offs[lo] <= t < offs[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    (a.offs[mid] <= t ? lo : hi) = mid;
  }
  begin = a.offs[lo];
  end = a.offs[hi];
  return true;
}

__global__ void __launch_bounds__(32 * kWarps) dq_kernel(PackedArgs a, const int* ok, float* D) {
  const long long id = 1LL * blockIdx.x * kWarps + (threadIdx.x >> 5);
  int b, e;
  if (!*ok || id >= 1LL * a.T * a.Hq) return;
  const int t = static_cast<int>(id / a.Hq), h = static_cast<int>(id % a.Hq), hk = h / (a.Hq / a.Hk);
  if (!sequence(a, t, b, e)) return;
  const Vec q = load(a.q, t, h, a.dh), g = load(a.dout, t, h, a.dh);
  const float d = dot(g, load(a.o, t, h, a.dh)), lse = a.lse[1LL * t * a.Hq + h];
  if ((threadIdx.x & 31) == 0) D[1LL * t * a.Hq + h] = d;
  Vec dq{};
  for (int j = b; j <= t; ++j) {
    const Vec k = load(a.k, j, hk, a.dh);
    const float p = expf(a.scale * dot(q, k) - lse);
    axpy(dq, a.scale * p * (dot(g, load(a.v, j, hk, a.dh)) - d), k);
  }
  store(a.dq, t, h, a.dh, dq);
}

__global__ void __launch_bounds__(32 * kWarps) dkv_kernel(PackedArgs a, const int* ok, const float* D) {
  const long long id = 1LL * blockIdx.x * kWarps + (threadIdx.x >> 5);
  int b, e;
  if (!*ok || id >= 1LL * a.T * a.Hk) return;
  const int j = static_cast<int>(id / a.Hk), hk = static_cast<int>(id % a.Hk), G = a.Hq / a.Hk;
  if (!sequence(a, j, b, e)) return;
  const Vec k = load(a.k, j, hk, a.dh), v = load(a.v, j, hk, a.dh);
  Vec dk{}, dv{};
  for (int t = j; t < e; ++t)
    for (int h = hk * G; h < hk * G + G; ++h) {
      const Vec q = load(a.q, t, h, a.dh), g = load(a.dout, t, h, a.dh);
      const float p = expf(a.scale * dot(q, k) - a.lse[1LL * t * a.Hq + h]);
      axpy(dv, p, g);
      axpy(dk, a.scale * p * (dot(g, v) - D[1LL * t * a.Hq + h]), q);
    }
  store(a.dk, j, hk, a.dh, dk);
  store(a.dv, j, hk, a.dh, dv);
}

unsigned blocks(long long warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

}  // namespace

size_t packed_attn_bwd_ws_bytes(int T, int, int Hq, int) { return 256 + sizeof(float) * T * Hq; }

cudaError_t launch_packed_attn_bwd(const PackedArgs& a, void* ws, unsigned* err, cudaStream_t st) {
  int* ok = static_cast<int*>(ws);
  float* D = static_cast<float*>(ws) + 64;
  check_kernel<<<1, 1024, 0, st>>>(a, ok, err);
  dq_kernel<<<blocks(1LL * a.T * a.Hq), 32 * kWarps, 0, st>>>(a, ok, D);
  dkv_kernel<<<blocks(1LL * a.T * a.Hk), 32 * kWarps, 0, st>>>(a, ok, D);
  return cudaGetLastError();
}

}  // namespace lr
