// Norm and rotation of queries and keys, backward: with dn = R(-theta) dy, w = dn g and r = 1/rms of x,
//     dx = r (w - x r^2 mean(w x)),  dg = sum dn x r.
// The two sums over a vector's channels, of x^2 and w x, do not depend on one another and are reduced together.  The
// gain sums stay in registers over a group's steps; they are added over the block's lane groups, each block leaves one
// row of partial sums, and a second launch adds the rows in a fixed order.
// Bound by memory: x and dy read, dx written.  Measured, 16384 tokens, 32 + 32 heads of 128: bf16 805 MB in 124.0 us
// (6.49 TB/s, 97% of the copy rate), of which the second launch takes 3 us; rotation alone 537 MB in 81 us.
#include "qk_device.cuh"

namespace lr {

template <typename ST, int U, bool ADJ, int G, bool FULL>
__global__ void __launch_bounds__(kThreads, bwd_blocks(U, sizeof(ST))) qk_bwd_kernel(
    const __grid_constant__ QkArgs a, const __grid_constant__ QkPlan pl) {
  extern __shared__ __align__(16) unsigned char smem[];
  Ring<ST, U, 4>& ring = *reinterpret_cast<Ring<ST, U, 4>*>(smem);
  const int sub = threadIdx.x % 32 / G;
  const Share sh(a, pl, 32 / G, sub);
  const QkTensor& q = a.t[sh.which];
  const Slot sl = slot_of<ST, U, ADJ, G, FULL>(a);
  const ST* g = static_cast<const ST*>(q.g);
  pdl_wait();  // what comes before reads nothing but the arguments
  pdl_trigger();
  unsigned in_item = sh.item, item = sh.item;
  int in_left = sh.rounds, in_h = 0, in_heads = 0, h = 0, heads = 0;
  const ST *in = nullptr, *in_x = nullptr;
  ST* out = nullptr;
  auto fetch = [&](int slot) {
    if (in_left > 0) {
      if (in_h == 0) {
        const Item it(sh, in_item, q.H);
        in = static_cast<const ST*>(q.dy) + it.t * q.lddy + it.h0 * a.dh + sl.o;
        in_x = static_cast<const ST*>(q.x) + it.t * q.ldx + it.h0 * a.dh + sl.o;
        in_heads = sl.on ? it.heads : 0;
        if (a.pos && sl.turned && it.heads > 0) ring.load_pos(slot, a, sl, it.t);
      }
      if (in_h < in_heads) {
        ring.load(slot, 0, in, sl);
        if (g) ring.load(slot, 2, in_x, sl);
      }
      in += a.dh;
      in_x += a.dh;
      if (++in_h == sh.len) {
        in_h = 0;
        in_item += sh.stride;
        --in_left;
      }
    }
    copies_close();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i);
  const ST* gain = ring.fill(a, g, sl);
  __syncthreads();
  f2 gx[U / 2], gy[U / 2], dgx[U / 2], dgy[U / 2], c[U / 2], s[U / 2];
#pragma unroll
  for (int k = 0; k < U / 2; ++k) {
    gx[k] = gy[k] = both(1.f);
    dgx[k] = dgy[k] = c[k] = s[k] = both(0.f);  // a lane without channels adds zeros to its group's sums
  }
  if (g && sl.on) get_pairs<ST, U, ADJ>(gain, sl, gx, gy);
  const int steps = sh.rounds * sh.len;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const int slot = i % kRing;
    fetch((slot + kAhead) % kRing);
    copies_wait<kAhead>();
    if (h == 0) {
      const Item it(sh, item, q.H);
      out = static_cast<ST*>(q.out) + it.t * q.ldo + it.h0 * a.dh + sl.o;
      heads = sl.on ? it.heads : 0;
      item += sh.stride;
      if (sl.turned && heads > 0) ring.template angles<ADJ>(slot, a, sl, it.t, c, s);
    }
    const bool on = h < heads;
    f2 U0[U / 2], V0[U / 2];  // dn
    ring.template read<ADJ>(slot, 0, U0, V0);
#pragma unroll
    for (int k = 0; k < U / 2; ++k) {
      const f2 x = U0[k], y = V0[k], yc = y * c[k];
      U0[k] = pick2<FULL>(sl.turned, fma2(x, c[k], y * s[k]), x);
      V0[k] = pick2<FULL>(sl.turned, {fmaf(-x.x, s[k].x, yc.x), fmaf(-x.y, s[k].y, yc.y)}, y);
    }
    if (g) {
      f2 X[U / 2], Y[U / 2], ss = both(0.f), dot = both(0.f);
      ring.template read<ADJ>(slot, 2, X, Y);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) {
        ss = fma2(X[k], X[k], fma2(Y[k], Y[k], ss));
        dot = fma2(U0[k] * gx[k], X[k], fma2(V0[k] * gy[k], Y[k], dot));
      }
      const float sum = group_sum<G>(ss.x + ss.y), wx = group_sum<G>(dot.x + dot.y);
      const float r = rsqrtf(sum * a.inv_dh + a.eps);
      const f2 r2 = both(r), m = both(-wx * a.inv_dh * r);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) X[k] = X[k] * r2, Y[k] = Y[k] * r2;
      if (on) {
#pragma unroll
        for (int k = 0; k < U / 2; ++k) {
          dgx[k] = fma2(U0[k], X[k], dgx[k]);
          dgy[k] = fma2(V0[k], Y[k], dgy[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < U / 2; ++k) {
        U0[k] = r2 * fma2(X[k], m, U0[k] * gx[k]);
        V0[k] = r2 * fma2(Y[k], m, V0[k] * gy[k]);
      }
    }
    if (on) put_pairs<ST, U, ADJ>(out, sl, U0, V0);
    out += a.dh;
    if (++h == sh.len) h = 0;
  }
  if (!g) return;
  copies_wait<0>();
  __syncthreads();  // the ring's memory takes the lane groups' sums, 512 floats a warp at most
  float* sums = reinterpret_cast<float*>(smem);
  constexpr int P = 32 / G, N = U / kPieces<ST, U>;
  if (sl.on) {  // X and Y at the channels they came from
    float* mine = sums + (threadIdx.x / 32 * P + sub) * a.dh;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int x = ADJ ? 2 * i : i, y = ADJ ? 2 * i + 1 : U + i;  // places among the slot's 2 U channels
      mine[sl.o + x / U * sl.apart + x % U / N * sl.hop + x % N] = i % 2 ? dgx[i / 2].y : dgx[i / 2].x;
      mine[sl.o + y / U * sl.apart + y % U / N * sl.hop + y % N] = i % 2 ? dgy[i / 2].y : dgy[i / 2].x;
    }
  }
  __syncthreads();
  for (int ch = threadIdx.x; ch < a.dh; ch += kThreads) {
    float sum = 0.f;
#pragma unroll 4
    for (int w = 0; w < kWarps * P; ++w) sum += sums[w * a.dh + ch];
    q.part[static_cast<long long>(sh.block) * a.dh + ch] = sum;
  }
}

// dg of both tensors from their blocks' rows, in a fixed order: a block sums 8 channels, a thread every 128th row.
__global__ void __launch_bounds__(1024) qk_dg_kernel(const __grid_constant__ QkArgs a,
                                                     const __grid_constant__ QkPlan pl) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][33];
  const QkTensor& q = a.t[blockIdx.y];
  if (!q.g || q.H == 0) return;
  const int c = threadIdx.x % 8, row = threadIdx.x / 8;
  float v = 0.f;
#pragma unroll 4
  for (int p = row; p < pl.blocks[blockIdx.y]; p += 128)
    v += q.part[static_cast<long long>(p) * a.dh + blockIdx.x * 8 + c];
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if (row % 4 == 0) red[c][row / 4] = v;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  v = red[threadIdx.x / 32][threadIdx.x % 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) q.dg[blockIdx.x * 8 + threadIdx.x / 32] = v;
}

template <typename ST, int U, bool ADJ, bool FULL>
static QkKernel pick_g(int g) {
  if constexpr (sizeof(ST) * U == 32) {  // fp32 runs of 8: whole warps only
    return qk_bwd_kernel<ST, U, ADJ, 32, FULL>;
  } else {
    if (sizeof(ST) == 2 && g == 4) return qk_bwd_kernel<ST, U, ADJ, sizeof(ST) == 2 ? 4 : 8, FULL>;
    if (g == 5) return qk_bwd_kernel<ST, U, ADJ, 5, FULL>;
    if (g == 8) return qk_bwd_kernel<ST, U, ADJ, 8, FULL>;
    if (g == 10) return qk_bwd_kernel<ST, U, ADJ, 10, FULL>;
    return g == 16 ? qk_bwd_kernel<ST, U, ADJ, 16, FULL> : qk_bwd_kernel<ST, U, ADJ, 32, FULL>;
  }
}

template <typename ST>
static QkKernel pick(const QkArgs& a, bool adj, QkVariant v) {
  const bool full = a.rot == a.dh;
  if (v.u == 8)
    return adj ? (full ? pick_g<ST, 8, true, true>(v.g) : pick_g<ST, 8, true, false>(v.g))
               : (full ? pick_g<ST, 8, false, true>(v.g) : pick_g<ST, 8, false, false>(v.g));
  return adj ? (full ? pick_g<ST, 4, true, true>(v.g) : pick_g<ST, 4, true, false>(v.g))
             : (full ? pick_g<ST, 4, false, true>(v.g) : pick_g<ST, 4, false, false>(v.g));
}

template <typename ST>
cudaError_t launch_qk_bwd(const QkArgs& a, bool adjacent, int sms, QkPlan* plan, cudaStream_t st) {
  QkVariant v = variant(a, sizeof(ST));
  // Small launches take the shorter runs, whose kernel needs fewer registers and twice the warps (32 + 8 heads of 128 in
  // bf16, with the launch that adds the rows: 130 tokens 5.1 us against 5.8, 600 tokens 7.6 against 8.9, 1000 tokens 9.5
  // against 10.0; 2000 tokens 14.2 against 13.9, 16384 tokens and 64 heads 126.4 against 124.4).
  const long long at_once = sms * bwd_blocks(8, 2) * (32LL / v.g) * kWarps;
  if (1LL * a.T * (a.t[0].H + a.t[1].H) <= 5 * at_once) v = variant(a, sizeof(ST), false);
  cut(a, v.g, std::min(sms * bwd_blocks(v.u, sizeof(ST)), kQkMaxParts / kMostWaves), plan);
  return launch_qk(pick<ST>(a, adjacent, v), a, *plan,
                   v.u == 8 ? Ring<ST, 8, 4>::bytes(a) : Ring<ST, 4, 4>::bytes(a), st);
}

cudaError_t launch_qk_dg(const QkArgs& a, const QkPlan& plan, cudaStream_t st) {
  return launch_pdl(qk_dg_kernel, dim3(a.dh / 8, 2), dim3(1024), 0, st, a, plan);
}

template cudaError_t launch_qk_bwd<float>(const QkArgs&, bool, int, QkPlan*, cudaStream_t);
template cudaError_t launch_qk_bwd<bf16>(const QkArgs&, bool, int, QkPlan*, cudaStream_t);

}  // namespace lr
