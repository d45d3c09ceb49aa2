// lr_packed_attn_bwd: the lists of blocks and D = dout.o in a first launch, then dQ, dK and dV: in a launch each, or, where
// all items find an SM of their own, in one whose first blocks take dQ and whose others dK and dV.
#include <algorithm>

#include "packed_bwd_dkv.cuh"
#include "packed_bwd_dq.cuh"

namespace lr {
namespace packed {
namespace {

constexpr int kSmemBoth = dq::kSmem > dkv::kSmem ? dq::kSmem : dkv::kSmem;

// The block's shared memory; null (and an error bit) where it does not begin on a swizzled tile's boundary.
__device__ __forceinline__ uint8_t* tiles_at(uint8_t* smem, unsigned* err) {
  if (!(smem_addr(smem) & 1023u)) return smem;
  if (threadIdx.x == 0) atomicOr(err, DEV_ERR_TMEM);
  return nullptr;
}

__global__ void __launch_bounds__(kThreads, 1) packed_dq_kernel(const __grid_constant__ BwdMaps maps, const DqArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (uint8_t* smem = tiles_at(smem_raw, a.err)) dq::body(maps, a, blockIdx.x, gridDim.x, smem);
}

__global__ void __launch_bounds__(kThreads, 1) packed_dkv_kernel(const __grid_constant__ BwdMaps maps, const DkvArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (uint8_t* smem = tiles_at(smem_raw, a.err)) dkv::body(maps, a, blockIdx.x, gridDim.x, smem);
}

__global__ void __launch_bounds__(kThreads, 1)
    packed_dqkv_kernel(const __grid_constant__ BwdMaps maps, const DqArgs a, const DkvArgs b, unsigned first) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = tiles_at(smem_raw, a.err);
  if (!smem) return;
  if (blockIdx.x < first) dq::body(maps, a, blockIdx.x, first, smem);
  else dkv::body(maps, b, blockIdx.x - first, gridDim.x - first, smem);
}

struct BwdWs {
  PlanJob jobs[2];  // dQ, dK and dV
  float* D;         // [T, Hq]
};

size_t bwd_layout(int T, int nseq, int Hq, int Hk, void* base, BwdWs* w) {
  char* p = static_cast<char*>(base);
  BwdWs at{};
  at.jobs[0].tokens = kRows / (Hq / Hk);
  at.jobs[0].work = 1;
  at.jobs[1].tokens = kRows;
  at.jobs[1].work = -1;
  size_t size = 0;
  for (PlanJob& j : at.jobs) size += plan_layout(T, nseq, j.tokens, p ? p + size : nullptr, p ? &j.plan : nullptr);
  at.D = reinterpret_cast<float*>(p ? p + size : nullptr);
  size += (sizeof(float) * T * Hq + 255) / 256 * 256;
  if (w) *w = at;
  return size;
}

}  // namespace
}  // namespace packed

size_t packed_attn_bwd_ws_bytes(int T, int nseq, int Hq, int Hk) {
  return packed::bwd_layout(T, nseq, Hq, Hk, nullptr, nullptr);
}

cudaError_t launch_packed_attn_bwd(const PackedArgs& p, void* ws, unsigned* err, cudaStream_t st) {
  using namespace packed;
  cudaError_t e = configure<packed_dq_kernel, dq::kSmem>();
  if (e == cudaSuccess) e = configure<packed_dkv_kernel, dkv::kSmem>();
  if (e == cudaSuccess) e = configure<packed_dqkv_kernel, kSmemBoth>();
  if (e != cudaSuccess) return e;
  BwdWs w;
  bwd_layout(p.T, p.nseq, p.Hq, p.Hk, ws, &w);
  const int G = p.Hq / p.Hk, tq = kRows / G;
  BwdMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!encode_heads(&maps.q, p.q, p.T, p.Hq, p.dh, G, tq) || !encode_heads(&maps.dout, p.dout, p.T, p.Hq, p.dh, G, tq) ||
      !encode_heads(&maps.k, p.k, p.T, p.Hk, p.dh, 1, kRows) || !encode_heads(&maps.v, p.v, p.T, p.Hk, p.dh, 1, kRows))
    return cudaErrorInvalidValue;
  const unsigned magic = group_magic(G);
  // dQ streams K and V of a key head, dK and dV stream Q and dO of its group.
  const DqArgs a{p.dq, p.lse, w.D, p.scale, p.Hq, p.dh, G, tq, magic, taken(w.jobs[0].plan, p.Hk, 4LL * p.T * p.dh), err};
  const DkvArgs b{p.dk, p.dv, p.lse, w.D, p.scale, p.Hq, p.dh, G, tq, magic,
                  taken(w.jobs[1].plan, p.Hk, 4LL * p.T * G * p.dh), err};
  const long long na = plan_capacity(p.T, p.nseq, tq) * p.Hk, nb = plan_capacity(p.T, p.nseq, kRows) * p.Hk;
  const int sms = device_sm_count();
  e = launch_prepare(p, w.jobs, 2, w.D, err, st);
  if (e != cudaSuccess) return e;
  if (na + nb <= sms)
    return launch_as(pdl_allowed(), packed_dqkv_kernel, dim3(static_cast<unsigned>(na + nb)), dim3(kThreads), kSmemBoth, st,
                     maps, a, b, static_cast<unsigned>(na));
  e = launch_as(pdl_allowed(), packed_dq_kernel, dim3(static_cast<unsigned>(std::min<long long>(na, sms))), dim3(kThreads),
                dq::kSmem, st, maps, a);
  if (e != cudaSuccess) return e;
  return launch_as(false, packed_dkv_kernel, dim3(static_cast<unsigned>(std::min<long long>(nb, sms))), dim3(kThreads),
                   dkv::kSmem, st, maps, b);
}

}  // namespace lr
