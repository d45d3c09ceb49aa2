// The launches of lr_packed_attn_bwd: the lists of blocks and D = dout.o, then dQ, then dK and dV.
#include "packed_device.cuh"

namespace lr {
namespace packed {
namespace {

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

cudaError_t launch_packed_attn_bwd(const PackedArgs& a, void* ws, unsigned* err, cudaStream_t st) {
  using namespace packed;
  BwdWs w;
  bwd_layout(a.T, a.nseq, a.Hq, a.Hk, ws, &w);
  cudaError_t e = launch_prepare(a, w.jobs, 2, w.D, err, st);
  if (e == cudaSuccess) e = launch_packed_dq(a, w.D, w.jobs[0].plan, err, st);
  if (e == cudaSuccess) e = launch_packed_dkv(a, w.D, w.jobs[1].plan, err, st);
  return e;
}

}  // namespace lr
