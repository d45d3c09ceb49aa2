// Norm and rotation of queries and keys, forward: y = r R(theta) (x g), with R(theta) g kept as four products per pair
// that are renewed once per item.
// Bound by memory: x read, y written.  Measured, 16384 tokens, 32 + 32 heads of 128: bf16 537 MB in 81.5 us (6.59 TB/s,
// 98% of the copy rate); 12483 tokens with three position axes, 20 + 4 heads: 153 MB in 26.4 us (87%: with so few heads
// to a token the angles weigh more).
#include "qk_device.cuh"

namespace lr {

template <typename ST, int U, bool ADJ, int G, bool FULL>
__global__ void __launch_bounds__(kThreads, fwd_blocks(U, sizeof(ST))) qk_fwd_kernel(
    const __grid_constant__ QkArgs a, const __grid_constant__ QkPlan pl) {
  extern __shared__ __align__(16) unsigned char smem[];
  Ring<ST, U, 2>& ring = *reinterpret_cast<Ring<ST, U, 2>*>(smem);
  const Share sh(a, pl, 32 / G, threadIdx.x % 32 / G);
  const QkTensor& q = a.t[sh.which];
  const Slot sl = slot_of<ST, U, ADJ, G, FULL>(a);
  const ST* g = static_cast<const ST*>(q.g);
  pdl_wait();  // what comes before reads nothing but the arguments
  pdl_trigger();
  unsigned in_item = sh.item, item = sh.item;
  int in_left = sh.rounds, in_h = 0, in_heads = 0, h = 0, heads = 0;
  const ST* in = nullptr;
  ST* out = nullptr;
  auto fetch = [&](int slot) {
    if (in_left > 0) {
      if (in_h == 0) {
        const Item it(sh, in_item, q.H);
        in = static_cast<const ST*>(q.x) + it.t * q.ldx + it.h0 * a.dh + sl.o;
        in_heads = sl.on ? it.heads : 0;
        if (a.pos && sl.turned && it.heads > 0) ring.load_pos(slot, a, sl, it.t);
      }
      if (in_h < in_heads) ring.load(slot, 0, in, sl);
      in += a.dh;
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
  f2 A[U / 2], B[U / 2], C[U / 2], D[U / 2];
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
      f2 gx[U / 2], gy[U / 2], c[U / 2], s[U / 2];
#pragma unroll
      for (int k = 0; k < U / 2; ++k) gx[k] = gy[k] = c[k] = both(1.f);
      if (g && sl.on) get_pairs<ST, U, ADJ>(gain, sl, gx, gy);
      if (sl.turned && heads > 0) ring.template angles<ADJ>(slot, a, sl, it.t, c, s);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) {
        A[k] = gx[k] * c[k];
        B[k] = gy[k] * -s[k];
        C[k] = gx[k] * s[k];
        D[k] = gy[k] * c[k];
      }
    }
    f2 X[U / 2], Y[U / 2];
    ring.template read<ADJ>(slot, 0, X, Y);
    float r = 1.f;
    if (g) {
      f2 ss = both(0.f);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) ss = fma2(X[k], X[k], fma2(Y[k], Y[k], ss));
      r = rsqrtf(group_sum<G>(ss.x + ss.y) * a.inv_dh + a.eps);
    }
    const f2 r2 = both(r);
#pragma unroll
    for (int k = 0; k < U / 2; ++k) {
      const f2 x = X[k] * r2, y = Y[k] * r2;
      const f2 p = x * A[k], q = y * D[k];  // all of it where the slot is not turned
      X[k] = pick2<FULL>(sl.turned, fma2(y, B[k], p), p);
      Y[k] = pick2<FULL>(sl.turned, fma2(x, C[k], q), q);
    }
    if (h < heads) put_pairs<ST, U, ADJ>(out, sl, X, Y);
    out += a.dh;
    if (++h == sh.len) h = 0;
  }
}

template <typename ST, int U, bool ADJ, bool FULL>
static QkKernel pick_g(int g) {
  if constexpr (sizeof(ST) * U == 32) {  // fp32 runs of 8: whole warps only
    return qk_fwd_kernel<ST, U, ADJ, 32, FULL>;
  } else {
    if (sizeof(ST) == 2 && g == 4) return qk_fwd_kernel<ST, U, ADJ, sizeof(ST) == 2 ? 4 : 8, FULL>;
    if (g == 5) return qk_fwd_kernel<ST, U, ADJ, 5, FULL>;
    if (g == 8) return qk_fwd_kernel<ST, U, ADJ, 8, FULL>;
    if (g == 10) return qk_fwd_kernel<ST, U, ADJ, 10, FULL>;
    return g == 16 ? qk_fwd_kernel<ST, U, ADJ, 16, FULL> : qk_fwd_kernel<ST, U, ADJ, 32, FULL>;
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
cudaError_t launch_qk_fwd(const QkArgs& a, bool adjacent, int sms, cudaStream_t st) {
  const QkVariant v = variant(a, sizeof(ST));
  QkPlan pl;
  cut(a, v.g, sms * fwd_blocks(v.u, sizeof(ST)), &pl);
  return launch_qk(pick<ST>(a, adjacent, v), a, pl, v.u == 8 ? Ring<ST, 8, 2>::bytes(a) : Ring<ST, 4, 2>::bytes(a), st);
}

template cudaError_t launch_qk_fwd<float>(const QkArgs&, bool, int, cudaStream_t);
template cudaError_t launch_qk_fwd<bf16>(const QkArgs&, bool, int, cudaStream_t);

}  // namespace lr
