// Causal attention over packed sequences with grouped heads (lr_packed_attn_fwd / lr_packed_attn_bwd): query head h of
// row t, key head h / G, keys j <= t of the same sequence:
//     S_tj = scale q_t.k_j,  lse_t = log sum_j exp S_tj,  o_t = sum_j exp(S_tj - lse_t) v_j
// and the backward of sum(o * dout):
//     D_t = dout_t.o_t,  P = exp(S - lse),  dS = scale P (dout_t.v_j - D_t),
//     dq_t = sum_j dS_tj k_j,  dk_j = sum dS_tj q_t,  dv_j = sum P_tj dout_t.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace lr {

struct PackedRows {
  bf16* p;       // [T, ld], head h in columns h*dh .. h*dh + dh - 1
  long long ld;  // elements
};

struct PackedArgs {
  int T, nseq, Hq, Hk, dh;
  float scale;
  const int* offs;  // [nseq + 1]
  PackedRows q, k, v, o;
  float* lse;  // [T, Hq]
  PackedRows dout, dq, dk, dv;  // backward
};

size_t packed_attn_fwd_ws_bytes(int T, int nseq, int Hq, int Hk);
size_t packed_attn_bwd_ws_bytes(int T, int nseq, int Hq, int Hk, int dh);
// launches: the kernels that were launched.
cudaError_t launch_packed_attn_fwd(const PackedArgs& a, void* ws, unsigned* err, cudaStream_t st, int* launches);
cudaError_t launch_packed_attn_bwd(const PackedArgs& a, void* ws, unsigned* err, cudaStream_t st, int* launches);

}  // namespace lr
