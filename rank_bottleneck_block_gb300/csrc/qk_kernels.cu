// A vector (one head of one token) lies over G lanes of a warp, a lane holding 2 U of its channels ("a slot") such
// that both channels of every pair are in the same lane: two runs of U channels, rot / 2 apart (pairs (p, p + rot/2))
// or adjacent (pairs (2p, 2p + 1)); slots past the turned channels hold 2 U neighbouring channels.  So a vector is
// read once with 16-byte loads (8-byte ones for bf16 whose dh or rot is no multiple of 16), its sums take log2 G
// shuffles, and an output may take its input's place.  The vectors of a tensor are numbered token by token, head by
// head; each warp takes an equal share of consecutive ones, 32 / G at a step, and computes a lane's angles once per
// token.  Loads run kAhead steps ahead of the arithmetic through a ring in shared memory (asynchronous copies; a thread
// reads back only what it copied itself, so it waits for nothing but its own copies).  The arithmetic is on two pairs
// at a time (the f32x2 instructions).
#include "qk_kernels.cuh"

#include <algorithm>

namespace lr {

// ------------------------------------------------------ two floats at a time
struct alignas(8) f2 {
  float x, y;
};
__device__ __forceinline__ unsigned long long bits(f2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ f2 of_bits(unsigned long long r) {
  f2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return of_bits(r);
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return of_bits(r);
}
__device__ __forceinline__ f2 both(float a) { return {a, a}; }
__device__ __forceinline__ f2 operator-(f2 a) { return {-a.x, -a.y}; }

// ------------------------------------------------------------ lanes and slots
// The lane's slot: where its two runs start, and whether its channels are turned.
struct Slot {
  int o0, o1, pair, axis;  // pair: the first of the slot's U pairs; axis: theirs, or -1 if they have several
  bool on, turned;
};
__device__ __forceinline__ int axis_of(const QkArgs& a, int p) {
  return (p >= a.sec_end[0]) + (p >= a.sec_end[1]) + (p >= a.sec_end[2]);
}
template <int U, bool ADJ, int G>
__device__ __forceinline__ Slot slot_of(const QkArgs& a) {
  const int j = threadIdx.x % G, n = a.rot / (2 * U);
  Slot s;
  s.on = j < a.dh / (2 * U);
  s.turned = s.on && j < n;
  s.pair = j * U;
  s.axis = axis_of(a, s.pair);
  if (axis_of(a, s.pair + U - 1) != s.axis) s.axis = -1;
  s.o0 = ADJ ? 2 * U * j : s.turned ? U * j : a.rot + 2 * U * (j - n);
  s.o1 = !ADJ && s.turned ? s.o0 + a.rot / 2 : s.o0 + U;
  return s;
}

// The slot's channels as the first and second members of its pairs, X[i] and Y[i] (of a slot that is not turned: in
// the same order of memory).  A run of U channels is W 32-bit words.
template <typename ST, int U>
constexpr int kWords = U * static_cast<int>(sizeof(ST)) / 4;

template <typename ST, int U, bool ADJ>
__device__ __forceinline__ void pairs_of(const uint32_t* w0, const uint32_t* w1, f2* X, f2* Y) {
  float x[U], y[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if constexpr (sizeof(ST) == 4) {
      x[i] = __uint_as_float(ADJ ? (2 * i < U ? w0[2 * i] : w1[2 * i - U]) : w0[i]);
      y[i] = __uint_as_float(ADJ ? (2 * i < U ? w0[2 * i + 1] : w1[2 * i + 1 - U]) : w1[i]);
    } else if constexpr (ADJ) {
      const uint32_t w = 2 * i < U ? w0[i] : w1[i - U / 2];
      x[i] = __uint_as_float(w << 16);
      y[i] = __uint_as_float(w & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(i % 2 ? w0[i / 2] & 0xffff0000u : w0[i / 2] << 16);
      y[i] = __uint_as_float(i % 2 ? w1[i / 2] & 0xffff0000u : w1[i / 2] << 16);
    }
  }
#pragma unroll
  for (int i = 0; i < U / 2; ++i) {
    X[i] = {x[2 * i], x[2 * i + 1]};
    Y[i] = {y[2 * i], y[2 * i + 1]};
  }
}

// Words next to one another: the widest loads and stores that fit.
template <int N>
__device__ __forceinline__ void get_words(const void* p, uint32_t* w) {
  if constexpr (N == 2) {
    const uint2 q = *static_cast<const uint2*>(p);
    w[0] = q.x, w[1] = q.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 q = static_cast<const uint4*>(p)[i];
      w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void put_words(void* p, const uint32_t* w) {
  if constexpr (N == 2) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename ST, int U, bool ADJ>
__device__ __forceinline__ void get_pairs(const ST* p0, const ST* p1, f2* X, f2* Y) {
  uint32_t w0[kWords<ST, U>], w1[kWords<ST, U>];
  get_words<kWords<ST, U>>(p0, w0);
  get_words<kWords<ST, U>>(p1, w1);
  pairs_of<ST, U, ADJ>(w0, w1, X, Y);
}

// Rounds to ST and stores.
template <typename ST, int U, bool ADJ>
__device__ __forceinline__ void put_pairs(ST* p0, ST* p1, const f2* X, const f2* Y) {
  float x[U], y[U];
#pragma unroll
  for (int i = 0; i < U / 2; ++i) {
    x[2 * i] = X[i].x, x[2 * i + 1] = X[i].y;
    y[2 * i] = Y[i].x, y[2 * i + 1] = Y[i].y;
  }
  uint32_t w[2 * kWords<ST, U>];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if constexpr (sizeof(ST) == 4) {
      w[ADJ ? 2 * i : i] = __float_as_uint(x[i]);
      w[ADJ ? 2 * i + 1 : U + i] = __float_as_uint(y[i]);
    } else if constexpr (ADJ) {
      w[i] = pack(x[i], y[i]);
    } else if (i % 2 == 0) {
      w[i / 2] = pack(x[i], x[i + 1]);
      w[U / 2 + i / 2] = pack(y[i], y[i + 1]);
    }
  }
  put_words<kWords<ST, U>>(p0, w);
  put_words<kWords<ST, U>>(p1, w + kWords<ST, U>);
}

// Cosines and sines of the slot's pairs at token t.  pos * turns wraps at 2^64, a whole number of turns, so the
// product is exact for any position; its top 32 bits, signed, are the angle in [-1/2, 1/2) turns.  For bf16 outputs
// the hardware sine and cosine serve (off by 2^-21.2 at most on [-pi, pi], against a rounding of 2^-9).
template <typename ST, int U>
__device__ __forceinline__ void slot_angles(const QkArgs& a, const Slot& sl, const unsigned long long* turns, int t,
                                            int pos, f2* C, f2* S) {
  float c[U], s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const unsigned long long w = turns[sl.pair + i];
    if (sl.axis < 0 && a.pos) pos = a.pos[static_cast<long long>(axis_of(a, sl.pair + i)) * a.T + t];
    const float top = static_cast<float>(static_cast<int>((static_cast<unsigned long long>(1LL * pos) * w) >> 32));
    if constexpr (sizeof(ST) == 2) __sincosf(top * 1.46291807926715968e-9f /* 2 pi / 2^32 */, &s[i], &c[i]);
    else sincospif(top * 0x1p-31f, &s[i], &c[i]);
  }
#pragma unroll
  for (int i = 0; i < U / 2; ++i) {
    C[i] = {c[2 * i], c[2 * i + 1]};
    S[i] = {s[2 * i], s[2 * i + 1]};
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- the ring
constexpr int kWarps = 4;  // of a block
constexpr int kThreads = 32 * kWarps;
constexpr int kAhead = 3;  // steps whose loads are in flight while one is computed
constexpr int kRing = kAhead + 1;

// Blocks an SM holds; es * u: bytes of a run.
constexpr int fwd_blocks(int u, int es) { return es * u > 16 ? 4 : u == 8 ? 5 : 8; }
constexpr int bwd_blocks(int u, int es) { return es * u > 16 ? 2 : u == 8 ? 4 : 5; }

template <int B>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(B) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// For each step in flight, RUNS runs of every thread (in pieces of at most 16 bytes, a thread's pieces kThreads apart,
// so that a warp's accesses are contiguous) and its position; then the turns [rot / 2] and the gain [dh] as stored.
template <typename ST, int U, int RUNS>
struct Ring {
  static constexpr int kPiece = kWords<ST, U> < 4 ? 4 * kWords<ST, U> : 16, kPieces = 4 * kWords<ST, U> / kPiece;
  alignas(16) unsigned char data[kRing][RUNS][kPieces][kThreads][kPiece];
  int pos[kRing][kThreads];
  alignas(16) unsigned long long turns[1];

  __device__ __forceinline__ void load(int slot, int run, const ST* from) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      copy_async<kPiece>(data[slot][run][i][threadIdx.x], reinterpret_cast<const char*>(from) + i * kPiece);
  }
  template <bool ADJ>
  __device__ __forceinline__ void read(int slot, int run, f2* X, f2* Y) const {
    uint32_t w[2][kWords<ST, U>];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        get_words<kPiece / 4>(data[slot][run + r][i][threadIdx.x], w[r] + i * (kPiece / 4));
    pairs_of<ST, U, ADJ>(w[0], w[1], X, Y);
  }
  // The turns and the gain; readable after the block's next barrier.
  __device__ __forceinline__ ST* fill(const QkArgs& a, const ST* g) {
    ST* gain = reinterpret_cast<ST*>(turns + a.rot / 2);
    for (int p = threadIdx.x; p < a.rot / 2; p += kThreads) turns[p] = a.turns[p];
    if (g)
      for (int c = threadIdx.x; c < a.dh; c += kThreads) gain[c] = g[c];
    return gain;
  }
  static size_t bytes(const QkArgs& a) {
    return sizeof(Ring) - 16 + a.rot / 2 * sizeof(unsigned long long) + a.dh * sizeof(ST);
  }
};

// Where a lane group's vector of a step lies in one tensor; a step moves it by `step` elements, and by `wrap` more when
// it passes a token's last head.
template <typename ST>
struct Walk {
  ST* p;
  long long step, wrap;
  __device__ __forceinline__ Walk(ST* base, long long ld, int t, int h, int dh, int H, int step_t, int step_h)
      : p(base + t * ld + h * dh), step(step_t * ld + step_h * dh), wrap(ld - H * dh) {}
  __device__ __forceinline__ void next(bool wraps) { p += step + (wraps ? wrap : 0); }
};

// A warp's steps and its groups' first vectors.
struct Share {
  int which, steps, t, h, step_t, step_h;
  unsigned block, v, all;  // v: the group's vector, of `all`
  __device__ __forceinline__ Share(const QkArgs& a, const QkPlan& pl, int P, int sub) {
    which = blockIdx.x < static_cast<unsigned>(pl.blocks[0]) ? 0 : 1;
    block = blockIdx.x - (which ? pl.blocks[0] : 0);
    const unsigned w = block * kWarps + threadIdx.x / 32, more = pl.more[which];
    steps = pl.steps[which] + (w < more);
    v = (w * pl.steps[which] + min(w, more)) * P + sub;
    const unsigned H = a.t[which].H;
    all = H * a.T;
    t = static_cast<int>(v / H);
    h = static_cast<int>(v % H);
    step_t = pl.step_t[which];
    step_h = pl.step_h[which];
  }
};

// ----------------------------------------------------------------- forward
// y = r R(theta) (x g) with R(theta) g kept as four products per pair, renewed once per token.
template <typename ST, int U, bool ADJ, int G>
__global__ void __launch_bounds__(kThreads, fwd_blocks(U, sizeof(ST))) qk_fwd_kernel(
    const __grid_constant__ QkArgs a, const __grid_constant__ QkPlan pl) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) unsigned char smem[];
  Ring<ST, U, 2>& ring = *reinterpret_cast<Ring<ST, U, 2>*>(smem);
  constexpr int P = 32 / G;
  const Share sh(a, pl, P, threadIdx.x % 32 / G);
  const QkTensor& q = a.t[sh.which];
  const Slot sl = slot_of<U, ADJ, G>(a);
  const ST* g = static_cast<const ST*>(q.g);
  const bool fetch_pos = a.pos && sl.turned && sl.axis >= 0;
  const int* pos = a.pos + static_cast<long long>(sl.axis) * a.T;
  Walk<const ST> in(static_cast<const ST*>(q.x) + sl.o0, q.ldx, sh.t, sh.h, a.dh, q.H, sh.step_t, sh.step_h);
  Walk<ST> out(static_cast<ST*>(q.out) + sl.o0, q.ldo, sh.t, sh.h, a.dh, q.H, sh.step_t, sh.step_h);
  int in_h = sh.h, in_t = sh.t, h = sh.h, t = sh.t;
  unsigned in_v = sh.v, v = sh.v;
  int fetched = 0;
  auto fetch = [&](int slot) {
    if (fetched++ < sh.steps && in_v < sh.all && sl.on) {
      ring.load(slot, 0, in.p);
      ring.load(slot, 1, in.p + (sl.o1 - sl.o0));
      if (fetch_pos) copy_async<4>(&ring.pos[slot][threadIdx.x], pos + in_t);
    }
    copies_close();
    in_v += P;
    in_h += sh.step_h;
    const bool wraps = in_h >= q.H;
    if (wraps) in_h -= q.H;
    in_t += sh.step_t + wraps;
    in.next(wraps);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i);
  const ST* gain = ring.fill(a, g);
  __syncthreads();
  const float inv_dh = 1.f / static_cast<float>(a.dh);
  f2 A[U / 2], B[U / 2], C[U / 2], D[U / 2];
  int now = -1;
  for (int i = 0; i < sh.steps; i += kRing) {
#pragma unroll
    for (int slot = 0; slot < kRing; ++slot) {
      if (i + slot >= sh.steps) break;  // the same for all lanes of the warp
      fetch((slot + kAhead) % kRing);
      copies_wait<kAhead>();
      const bool on = v < sh.all && sl.on;
      f2 X[U / 2], Y[U / 2];
      ring.template read<ADJ>(slot, 0, X, Y);
      if (on && t != now) {
        now = t;
        f2 gx[U / 2], gy[U / 2];
#pragma unroll
        for (int k = 0; k < U / 2; ++k) gx[k] = gy[k] = both(1.f);
        if (g) get_pairs<ST, U, ADJ>(gain + sl.o0, gain + sl.o1, gx, gy);
        if (sl.turned) {
          f2 c[U / 2], s[U / 2];
          slot_angles<ST, U>(a, sl, ring.turns, t, a.pos ? ring.pos[slot][threadIdx.x] : t % a.seq, c, s);
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            A[k] = gx[k] * c[k];
            B[k] = -(gy[k] * s[k]);
            C[k] = gx[k] * s[k];
            D[k] = gy[k] * c[k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) A[k] = gx[k], D[k] = gy[k];
        }
      }
      float r = 1.f;
      if (g) {
        f2 ss = both(0.f);
        if (on) {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) ss = fma2(X[k], X[k], fma2(Y[k], Y[k], ss));
        }
        r = rsqrtf(group_sum<G>(ss.x + ss.y) * inv_dh + a.eps);
      }
      if (on) {
        const f2 r2 = both(r);
        if (sl.turned) {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            const f2 x = X[k], y = Y[k];
            X[k] = r2 * fma2(x, A[k], y * B[k]);
            Y[k] = r2 * fma2(x, C[k], y * D[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) X[k] = r2 * X[k] * A[k], Y[k] = r2 * Y[k] * D[k];
        }
        put_pairs<ST, U, ADJ>(out.p, out.p + (sl.o1 - sl.o0), X, Y);
      }
      v += P;
      h += sh.step_h;
      const bool wraps = h >= q.H;
      if (wraps) h -= q.H;
      t += sh.step_t + wraps;
      out.next(wraps);
    }
  }
}

// ---------------------------------------------------------------- backward
// The gain sums stay in registers over a warp's steps; they are added over the warp's lane groups, then over the
// block's warps, and each block leaves one row of partial sums.  The sums over a vector's channels, mean(x^2) and
// mean(w x), are independent of one another and reduced together.
template <typename ST, int U, bool ADJ, int G>
__global__ void __launch_bounds__(kThreads, bwd_blocks(U, sizeof(ST))) qk_bwd_kernel(
    const __grid_constant__ QkArgs a, const __grid_constant__ QkPlan pl) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) unsigned char smem[];
  Ring<ST, U, 4>& ring = *reinterpret_cast<Ring<ST, U, 4>*>(smem);
  constexpr int P = 32 / G;
  const int sub = threadIdx.x % 32 / G;
  const Share sh(a, pl, P, sub);
  const QkTensor& q = a.t[sh.which];
  const Slot sl = slot_of<U, ADJ, G>(a);
  const ST* g = static_cast<const ST*>(q.g);
  const bool fetch_pos = a.pos && sl.turned && sl.axis >= 0;
  const int* pos = a.pos + static_cast<long long>(sl.axis) * a.T;
  Walk<const ST> in(static_cast<const ST*>(q.dy) + sl.o0, q.lddy, sh.t, sh.h, a.dh, q.H, sh.step_t, sh.step_h);
  Walk<const ST> in_x(static_cast<const ST*>(q.x) + sl.o0, q.ldx, sh.t, sh.h, a.dh, q.H, sh.step_t, sh.step_h);
  Walk<ST> out(static_cast<ST*>(q.out) + sl.o0, q.ldo, sh.t, sh.h, a.dh, q.H, sh.step_t, sh.step_h);
  int in_h = sh.h, in_t = sh.t, h = sh.h, t = sh.t;
  unsigned in_v = sh.v, v = sh.v;
  int fetched = 0;
  auto fetch = [&](int slot) {
    if (fetched++ < sh.steps && in_v < sh.all && sl.on) {
      ring.load(slot, 0, in.p);
      ring.load(slot, 1, in.p + (sl.o1 - sl.o0));
      if (g) {
        ring.load(slot, 2, in_x.p);
        ring.load(slot, 3, in_x.p + (sl.o1 - sl.o0));
      }
      if (fetch_pos) copy_async<4>(&ring.pos[slot][threadIdx.x], pos + in_t);
    }
    copies_close();
    in_v += P;
    in_h += sh.step_h;
    const bool wraps = in_h >= q.H;
    if (wraps) in_h -= q.H;
    in_t += sh.step_t + wraps;
    in.next(wraps);
    in_x.next(wraps);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i);
  const ST* gain = ring.fill(a, g);
  __syncthreads();
  const float inv_dh = 1.f / static_cast<float>(a.dh);
  f2 gx[U / 2], gy[U / 2], dgx[U / 2], dgy[U / 2], c[U / 2], s[U / 2];
#pragma unroll
  for (int k = 0; k < U / 2; ++k) gx[k] = gy[k] = both(1.f), dgx[k] = dgy[k] = both(0.f);
  if (g && sl.on) get_pairs<ST, U, ADJ>(gain + sl.o0, gain + sl.o1, gx, gy);
  int now = -1;
  for (int i = 0; i < sh.steps; i += kRing) {
#pragma unroll
    for (int slot = 0; slot < kRing; ++slot) {
      if (i + slot >= sh.steps) break;  // the same for all lanes of the warp
      fetch((slot + kAhead) % kRing);
      copies_wait<kAhead>();
      const bool on = v < sh.all && sl.on;
      f2 U0[U / 2], V0[U / 2];  // dn
      ring.template read<ADJ>(slot, 0, U0, V0);
      if (sl.turned && v < sh.all) {
        if (t != now) {
          now = t;
          slot_angles<ST, U>(a, sl, ring.turns, t, a.pos ? ring.pos[slot][threadIdx.x] : t % a.seq, c, s);
        }
#pragma unroll
        for (int k = 0; k < U / 2; ++k) {
          const f2 x = U0[k], y = V0[k];
          U0[k] = fma2(x, c[k], y * s[k]);
          V0[k] = fma2(-x, s[k], y * c[k]);
        }
      }
      if (g) {
        f2 X[U / 2], Y[U / 2], ss = both(0.f), dot = both(0.f);
        ring.template read<ADJ>(slot, 2, X, Y);
        if (on) {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            ss = fma2(X[k], X[k], fma2(Y[k], Y[k], ss));
            dot = fma2(U0[k] * gx[k], X[k], fma2(V0[k] * gy[k], Y[k], dot));
          }
        }
        const float sum = group_sum<G>(ss.x + ss.y), wx = group_sum<G>(dot.x + dot.y);
        const float r = rsqrtf(sum * inv_dh + a.eps);
        const f2 r2 = both(r), m = both(-wx * inv_dh * r);
        if (on) {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            X[k] = X[k] * r2;
            Y[k] = Y[k] * r2;
            dgx[k] = fma2(U0[k], X[k], dgx[k]);
            dgy[k] = fma2(V0[k], Y[k], dgy[k]);
            U0[k] = r2 * fma2(X[k], m, U0[k] * gx[k]);
            V0[k] = r2 * fma2(Y[k], m, V0[k] * gy[k]);
          }
        }
      }
      if (on) put_pairs<ST, U, ADJ>(out.p, out.p + (sl.o1 - sl.o0), U0, V0);
      v += P;
      h += sh.step_h;
      const bool wraps = h >= q.H;
      if (wraps) h -= q.H;
      t += sh.step_t + wraps;
      out.next(wraps);
    }
  }
  if (!g) return;
  copies_wait<0>();
  __syncthreads();  // the ring's memory takes the warps' sums
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int k = 0; k < U / 2; ++k) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      dgx[k].x += __shfl_xor_sync(0xffffffffu, dgx[k].x, o);
      dgx[k].y += __shfl_xor_sync(0xffffffffu, dgx[k].y, o);
      dgy[k].x += __shfl_xor_sync(0xffffffffu, dgy[k].x, o);
      dgy[k].y += __shfl_xor_sync(0xffffffffu, dgy[k].y, o);
    }
  }
  if (sub == 0 && sl.on) {
    float* mine = sums + threadIdx.x / 32 * a.dh;
    put_pairs<float, U, ADJ>(mine + sl.o0, mine + sl.o1, dgx, dgy);
  }
  __syncthreads();
  for (int ch = threadIdx.x; ch < a.dh; ch += kThreads) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w) sum += sums[w * a.dh + ch];
    q.part[static_cast<long long>(sh.block) * a.dh + ch] = sum;
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

// Blocks of each tensor by its share of the steps, at most as many as the SMs hold at once, and the steps of a warp.
static void cut(const QkArgs& a, int g, int resident, int most, QkPlan* pl) {
  const int P = 32 / g;
  long long steps[2];
  for (int i = 0; i < 2; ++i) steps[i] = (1LL * a.T * a.t[i].H + P - 1) / P;
  for (int i = 0; i < 2; ++i) {
    const int H = a.t[i].H;
    long long n = (steps[i] * resident + (steps[0] + steps[1]) / 2) / (steps[0] + steps[1]);
    n = std::min(std::min(std::max(n, 1LL), static_cast<long long>(most)), (steps[i] + kWarps - 1) / kWarps);
    pl->blocks[i] = static_cast<int>(n);
    pl->steps[i] = n ? static_cast<unsigned>(steps[i] / (n * kWarps)) : 0;
    pl->more[i] = n ? static_cast<unsigned>(steps[i] % (n * kWarps)) : 0;
    pl->step_t[i] = H ? P / H : 0;
    pl->step_h[i] = H ? P % H : 0;
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

static cudaError_t launch(QkKernel kern, const QkArgs& a, const QkPlan& pl, size_t smem, cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(pl.blocks[0] + pl.blocks[1]), dim3(kThreads), smem, st, a, pl);
}

template <typename ST>
cudaError_t launch_qk_fwd(const QkArgs& a, bool adjacent, int sms, cudaStream_t st) {
  const QkVariant v = variant(a, sizeof(ST));
  QkPlan pl;
  cut(a, v.g, sms * fwd_blocks(v.u, sizeof(ST)), 1 << 30, &pl);
  return launch(pick<ST>(false, adjacent, v), a, pl, v.u == 8 ? Ring<ST, 8, 2>::bytes(a) : Ring<ST, 4, 2>::bytes(a), st);
}

template <typename ST>
cudaError_t launch_qk_bwd(const QkArgs& a, bool adjacent, int sms, cudaStream_t st) {
  const QkVariant v = variant(a, sizeof(ST));
  QkPlan pl;
  cut(a, v.g, sms * bwd_blocks(v.u, sizeof(ST)), kQkMaxParts, &pl);
  const cudaError_t e =
      launch(pick<ST>(true, adjacent, v), a, pl, v.u == 8 ? Ring<ST, 8, 4>::bytes(a) : Ring<ST, 4, 4>::bytes(a), st);
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
