// Query / key norm and position rotation between the projections and attention (lr_qk_fwd / lr_qk_bwd):
// per token t and head, x in R^dh (q or k), gain g, pair p of the first rot channels, its axis a(p):
//     r = (mean_c x_c^2 + eps)^(-1/2),  n = x r g          (n = x when the tensor has no gain)
//     phase = pos[a(p)][t] * turns[p] mod 2^64             (turns in units of 2^-64 of a full turn)
//     (y_i, y_j) = (n_i cos - n_j sin, n_i sin + n_j cos)   (i, j the pair's channels; y_c = n_c for c >= rot)
// and the backward of sum(y * dy):
//     dn = rotation by -phase of dy,  dg_c = sum_{t, heads} dn_c x_c r,
//     w = dn g,  dx = r (w - x r^2 mean(w x))               (dx = dn when the tensor has no gain).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace lr {

constexpr int kQkMaxAxes = 4;
constexpr int kQkMaxParts = 4096;  // blocks per tensor that write a partial of dg

struct QkTensor {
  const void* x;   // [T, ldx], head h in columns h*dh .. h*dh + dh - 1 (may be null in a backward without norm)
  const void* dy;  // backward only
  void* out;       // y (forward) or dx (backward)
  const void* g;   // gain [dh], or null: no norm
  float* dg;       // backward: [dh], written when g is set
  float* part;     // backward: [kQkMaxParts, dh] partial sums of dg
  long long ldx, lddy, ldo;
  int H;           // 0: absent
};

struct QkArgs {
  QkTensor t[2];                    // q, k
  const unsigned long long* turns;  // [rot / 2]
  const int* pos;                   // [axes, T], or null: position t mod seq on every axis
  int T, dh, rot, seq;
  int sec_end[kQkMaxAxes - 1];      // first pair past axis 0, 1, 2 (rot / 2 when the axis is the last)
  float eps, inv_dh;
};

// How a launch cuts its work, for q and for k: blocks, the items of a lane group at most, and each token's heads into
// `chunks` items of `len` heads; item / chunks is the high word of item * magic, shifted (items are below 2^31).
struct QkPlan {
  int blocks[2], rounds[2], chunks[2], len[2], shift[2];
  unsigned magic[2];
};

// adjacent: pairs are channels (2p, 2p + 1), else (p, p + rot / 2).
template <typename ST>
cudaError_t launch_qk_fwd(const QkArgs& a, bool adjacent, int sms, cudaStream_t st);
// Writes dx of both tensors and the partial sums of dg (`plan`: how it cut the work) ...
template <typename ST>
cudaError_t launch_qk_bwd(const QkArgs& a, bool adjacent, int sms, QkPlan* plan, cudaStream_t st);
// ... and this adds them up.
cudaError_t launch_qk_dg(const QkArgs& a, const QkPlan& plan, cudaStream_t st);

}  // namespace lr
