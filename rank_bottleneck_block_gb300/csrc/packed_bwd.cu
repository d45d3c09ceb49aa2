// lr_packed_attn_bwd: the lists of blocks and D = dout.o in a first launch, then dK, dV and dQ in one: its first blocks take
// the items of dK and dV, the others those of dQ.  An SM holds one block, so those of dQ begin where the first ones find no
// more items, and fill the SMs that a few long items of dK and dV leave (one sequence of 1024 tokens, 32 over 8 heads: two
// launches took 59 us one after the other).
#include <algorithm>

#include "packed_bwd_dkv.cuh"
#include "packed_bwd_dq.cuh"

namespace lr {
namespace packed {
namespace {

constexpr int kSmem = dq::kSmem > dkv::kSmem ? dq::kSmem : dkv::kSmem;

__global__ void __launch_bounds__(kThreads, 1)
    packed_bwd_kernel(const __grid_constant__ BwdMaps maps, const DkvArgs a, const DqArgs b, unsigned first) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need it
    if (threadIdx.x == 0) atomicOr(a.err, DEV_ERR_TMEM);
    return;
  }
  if (blockIdx.x < first) dkv::body(maps, a, blockIdx.x, first, smem);
  else dq::body(maps, b, blockIdx.x - first, gridDim.x - first, smem);
}

// dK, dV of the rows of the sequences from the sums of their parts, eight channels a thread.
__global__ void __launch_bounds__(256) packed_join_kernel(PackedArgs a, const int* nblocks, int parts, const float* part_dk,
                                                          const float* part_dv) {
  const int per = a.dh / 8;
  const long long i = 1LL * blockIdx.x * 256 + threadIdx.x, row = i / per;  // row: key and head
  const int t = static_cast<int>(row / a.Hk), h = static_cast<int>(row - 1LL * t * a.Hk), c = static_cast<int>(i - row * per) * 8;
  pdl_wait();
  if (t >= a.T || *nblocks == 0 || t < a.offs[0] || t >= a.offs[a.nseq]) return;
  float k[8], v[8];
  for (int p = 0; p < parts; ++p) {
    const long long at = ((1LL * p * a.T + t) * a.Hk + h) * a.dh + c;
    float x[8], y[8];
    load8(part_dk + at, x);
    load8(part_dv + at, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      k[e] = p ? k[e] + x[e] : x[e];
      v[e] = p ? v[e] + y[e] : y[e];
    }
  }
  store8(a.dk.p + t * a.dk.ld + 1LL * h * a.dh + c, k);
  store8(a.dv.p + t * a.dv.ld + 1LL * h * a.dh + c, v);
}

// Parts of an item of dK and dV: not more items than 152 SMs (a GB300's; the size query, which asks too, needs no device), no
// part of less than four row tiles of a sequence twice as long as the average, and eight at most: a part costs some 5 us
// besides its tiles.  Whole backward: one sequence of 1024 tokens, 32 over 8 heads, 53.5 us uncut and 47.7 in parts; of
// 2048, 8 over 1, 168 and 43; eight of 128, 32 over 8, 24 uncut and 36 in four.
int dkv_parts(int T, int nseq, int Hq, int Hk) {
  const long long items = plan_capacity(T, nseq, kRows) * Hk;
  const long long tiles = 2LL * T / nseq / (kRows / (Hq / Hk));
  const long long n = std::min({152 / std::max(1LL, items), tiles / 8, 8LL});
  return static_cast<int>(std::max(1LL, n));
}

struct BwdWs {
  PlanJob jobs[2];  // dQ, dK and dV
  float* D;         // [T, Hq]
  int parts;
  float *part_dk, *part_dv;  // [parts, T, Hk, dh]
};

size_t bwd_layout(int T, int nseq, int Hq, int Hk, int dh, void* base, BwdWs* w) {
  char* p = static_cast<char*>(base);
  BwdWs at{};
  at.parts = dkv_parts(T, nseq, Hq, Hk);
  at.jobs[0].tokens = kRows / (Hq / Hk);
  at.jobs[0].work = 1;
  at.jobs[1].tokens = kRows;
  at.jobs[1].work = -1;
  size_t size = 0;
  for (PlanJob& j : at.jobs) size += plan_layout(T, nseq, j.tokens, p ? p + size : nullptr, p ? &j.plan : nullptr);
  at.D = reinterpret_cast<float*>(p ? p + size : nullptr);
  size += (sizeof(float) * T * Hq + 255) / 256 * 256;
  if (at.parts > 1) {
    const size_t each = (sizeof(float) * at.parts * T * Hk * dh + 255) / 256 * 256;
    at.part_dk = reinterpret_cast<float*>(p ? p + size : nullptr);
    at.part_dv = reinterpret_cast<float*>(p ? p + size + each : nullptr);
    size += 2 * each;
  }
  if (w) *w = at;
  return size;
}

}  // namespace
}  // namespace packed

size_t packed_attn_bwd_ws_bytes(int T, int nseq, int Hq, int Hk, int dh) {
  return packed::bwd_layout(T, nseq, Hq, Hk, dh, nullptr, nullptr);
}

cudaError_t launch_packed_attn_bwd(const PackedArgs& p, void* ws, unsigned* err, cudaStream_t st, int* launches) {
  using namespace packed;
  cudaError_t e = configure<packed_bwd_kernel, kSmem>();
  if (e != cudaSuccess) return e;
  BwdWs w;
  bwd_layout(p.T, p.nseq, p.Hq, p.Hk, p.dh, ws, &w);
  const int G = p.Hq / p.Hk, tq = kRows / G;
  BwdMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!encode_heads(&maps.q, p.q, p.T, p.Hq, p.dh, G, tq) || !encode_heads(&maps.dout, p.dout, p.T, p.Hq, p.dh, G, tq) ||
      !encode_heads(&maps.k, p.k, p.T, p.Hk, p.dh, 1, kRows) || !encode_heads(&maps.v, p.v, p.T, p.Hk, p.dh, 1, kRows))
    return cudaErrorInvalidValue;
  const unsigned magic = group_magic(G);
  // dQ streams K and V of a key head, dK and dV stream Q and dO of its group.
  const DkvArgs a{p.dk, p.dv, w.part_dk, w.part_dv, p.T, p.Hk, p.lse, w.D, p.scale, p.Hq, p.dh, G, tq, magic,
                  taken(w.jobs[1].plan, p.Hk, 4LL * p.T * G * p.dh, w.parts), err};
  const DqArgs b{p.dq, p.lse, w.D, p.scale, p.Hq, p.dh, G, tq, magic, taken(w.jobs[0].plan, p.Hk, 4LL * p.T * p.dh), err};
  const long long sms = device_sm_count();
  const unsigned na = static_cast<unsigned>(std::min(plan_capacity(p.T, p.nseq, kRows) * p.Hk * w.parts, sms));
  const unsigned nb = static_cast<unsigned>(std::min(plan_capacity(p.T, p.nseq, tq) * p.Hk, sms));
  e = launch_prepare(p, w.jobs, 2, w.D, err, st);
  if (e != cudaSuccess) return e;
  e = launch_as(pdl_allowed(), packed_bwd_kernel, dim3(na + nb), dim3(kThreads), kSmem, st, maps, a, b, na);
  *launches = w.parts == 1 ? 2 : 3;
  if (e != cudaSuccess || w.parts == 1) return e;
  const long long threads = 1LL * p.T * p.Hk * (p.dh / 8);
  return launch_as(pdl_allowed(), packed_join_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, st,
                   p, w.jobs[1].plan.nblocks, w.parts, w.part_dk, w.part_dv);
}

}  // namespace lr
