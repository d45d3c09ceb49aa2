// A vector (one head of one token) lies over G lanes of a warp, a lane holding 2 U of its channels ("a slot") such
// that both channels of every pair are in the same lane: two runs of U channels, rot / 2 apart (pairs (p, p + rot/2))
// or adjacent (pairs (2p, 2p + 1)); slots past the turned channels hold 2 U neighbouring channels.  So a vector is
// read once with 16-byte loads (8-byte ones for bf16 whose dh or rot is no multiple of 16), its sums take log2 G
// shuffles, and an output may take its input's place.  A lane group takes items of one token and a run of its heads,
// head by head, and computes its angles once per item; the 32 / G groups of a warp keep step.  Loads run kAhead steps
// ahead of the arithmetic through a ring in shared memory (asynchronous copies; a thread reads back only what it
// copied itself, so it waits for nothing but its own copies).  The arithmetic is on two pairs at a time (the f32x2
// instructions).  Steps that led here, 16384 tokens, 32 + 32 heads of 128, bf16, forward / backward: a warp per vector
// with 2-byte loads 427 / 1000 us; lane groups with 16-byte loads, a warp's groups sharing a token 102 / 154; the ring
// and f32x2 92 / 128; a token for each group, and more blocks than run at once 82 / 124.
#pragma once

#include <algorithm>

#include "qk_kernels.cuh"

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

// `a` where the slot is turned, else `b`; one that is FULL has only turned slots.
template <bool FULL>
__device__ __forceinline__ f2 pick2(bool turned, f2 a, f2 b) {
  if constexpr (FULL) return a;
  return {turned ? a.x : b.x, turned ? a.y : b.y};
}

// ------------------------------------------------------------ lanes and slots
// The lane's slot: two runs of U channels in pieces of at most 16 bytes.  Piece i of run r starts at channel o + r *
// apart + i * hop, and the lanes of a group hold neighbouring pieces, so that a warp's accesses are contiguous: the
// turned channels [0, rot) go to the first rot / (2 U) lanes, the others to the rest.
template <typename ST, int U>
constexpr int kPieces = sizeof(ST) * U > 16 ? sizeof(ST) * U / 16 : 1;

struct Slot {
  int o, apart, hop;
  int axis_a, axis_b;  // position axes of its pairs: axis_b where the pair's bit of `on_b` is set, else axis_a
  unsigned on_b;
  bool on, turned, more_axes;  // more_axes: more than two
};
__device__ __forceinline__ int axis_of(const QkArgs& a, int p) {
  return (p >= a.sec_end[0]) + (p >= a.sec_end[1]) + (p >= a.sec_end[2]);
}
// Number of the slot's i-th pair: pairs (p, p + rot / 2) have their first members in run 0, and adjacent ones are
// inside a piece.
template <typename ST, int U, bool ADJ>
__device__ __forceinline__ int pair_of(const Slot& s, int i) {
  constexpr int N = U / kPieces<ST, U>;  // channels of a piece
  if constexpr (ADJ) {
    const int ch = 2 * i;
    return (s.o + ch / U * s.apart + ch % U / N * s.hop) / 2 + ch % N / 2;
  } else {
    return s.o + i / N * s.hop + i % N;
  }
}
template <typename ST, int U, bool ADJ, int G, bool FULL>
__device__ __forceinline__ Slot slot_of(const QkArgs& a) {
  constexpr int N = U / kPieces<ST, U>;
  const int j = threadIdx.x % 32 % G, n = a.rot / (2 * U);
  Slot s;
  s.on = j < a.dh / (2 * U) && threadIdx.x % 32 < 32 / G * G;  // lanes past the last group have nothing to do
  s.turned = FULL ? s.on : s.on && j < n;
  const int all = s.turned ? a.rot : a.dh - a.rot;
  s.o = s.turned ? N * j : a.rot + N * (j - n);
  s.apart = all / 2;
  s.hop = all / 2 / kPieces<ST, U>;
  s.axis_a = s.axis_b = s.turned ? axis_of(a, pair_of<ST, U, ADJ>(s, 0)) : 0;
  s.on_b = 0;
  s.more_axes = false;
  if (s.turned && a.sec_end[0] < a.rot / 2) {  // more axes than the first
#pragma unroll
    for (int i = 1; i < U; ++i) {
      const int x = axis_of(a, pair_of<ST, U, ADJ>(s, i));
      if (x == s.axis_a) continue;
      if (s.axis_b == s.axis_a) s.axis_b = x;
      if (s.axis_b == x) s.on_b |= 1u << i;
      else s.more_axes = true;
    }
  }
  return s;
}

// The slot's channels as the first and second members of its pairs, X[i] and Y[i] (of a slot that is not turned: in
// the same order of memory).  A run of U channels is kWords 32-bit words.
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

// 8 or 16 neighbouring bytes.
template <int N>
__device__ __forceinline__ void get_words(const void* p, uint32_t* w) {
  if constexpr (N == 2) {
    const uint2 q = *static_cast<const uint2*>(p);
    w[0] = q.x, w[1] = q.y;
  } else {
    const uint4 q = *static_cast<const uint4*>(p);
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  }
}
template <int N>
__device__ __forceinline__ void put_words(void* p, const uint32_t* w) {
  if constexpr (N == 2) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The slot's channels of a vector at v.
template <typename ST, int U, bool ADJ>
__device__ __forceinline__ void get_pairs(const ST* v, const Slot& s, f2* X, f2* Y) {
  constexpr int K = kPieces<ST, U>, W = kWords<ST, U> / K;
  uint32_t w[2][K * W];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < K; ++i) get_words<W>(v + s.o + r * s.apart + i * s.hop, w[r] + i * W);
  pairs_of<ST, U, ADJ>(w[0], w[1], X, Y);
}

// Rounds to ST; `p` points to the slot's first channel.
template <typename ST, int U, bool ADJ>
__device__ __forceinline__ void put_pairs(ST* p, const Slot& s, const f2* X, const f2* Y) {
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
  constexpr int K = kPieces<ST, U>, W = kWords<ST, U> / K;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < K; ++i) put_words<W>(p + r * s.apart + i * s.hop, w + (r * K + i) * W);
}

// Cosines and sines of the slot's pairs at token t.  pos * turns wraps at 2^64, a whole number of turns, so the
// product is exact for any position; its top 32 bits, signed, are the angle in [-1/2, 1/2) turns.  For bf16 outputs
// the hardware sine and cosine serve (off by 2^-21.2 at most on [-pi, pi], against a rounding of 2^-9).
template <typename ST, int U, bool ADJ>
__device__ __forceinline__ void slot_angles(const QkArgs& a, const Slot& sl, const unsigned long long* turns, int t,
                                            int pos_a, int pos_b, f2* C, f2* S) {
  float c[U], s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int p = pair_of<ST, U, ADJ>(sl, i);
    int pos = sl.on_b >> i & 1 ? pos_b : pos_a;
    if (sl.more_axes && a.pos) pos = a.pos[static_cast<long long>(axis_of(a, p)) * a.T + t];
    const float top =
        static_cast<float>(static_cast<int>((static_cast<unsigned long long>(1LL * pos) * turns[p]) >> 32));
    if constexpr (sizeof(ST) == 2) __sincosf(top * 1.46291807926715968e-9f /* 2 pi / 2^32 */, &s[i], &c[i]);
    else sincospif(top * 0x1p-31f, &s[i], &c[i]);
  }
#pragma unroll
  for (int i = 0; i < U / 2; ++i) {
    C[i] = {c[2 * i], c[2 * i + 1]};
    S[i] = {s[2 * i], s[2 * i + 1]};
  }
}

// Sum over the lane's group, the same bits in each of its lanes.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((G & (G - 1)) == 0) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {  // 5 or 10 lanes: opposite ones, then the group's first five in order
    const int lane = threadIdx.x % 32, first = lane / G * G;
    if constexpr (G == 10) v += __shfl_sync(0xffffffffu, v, first + (lane - first + 5) % 10);
    float sum = __shfl_sync(0xffffffffu, v, first);
#pragma unroll
    for (int i = 1; i < 5; ++i) sum += __shfl_sync(0xffffffffu, v, first + i);
    return sum;
  }
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

// For each step in flight, RUNS runs of every thread (a thread's pieces kThreads apart, so that a warp's accesses are
// contiguous) and its two positions; then the turns [rot / 2] and the gain [dh] as stored.
template <typename ST, int U, int RUNS>
struct Ring {
  static constexpr int K = kPieces<ST, U>, W = kWords<ST, U> / K;  // pieces of a run, words of a piece
  alignas(16) unsigned char data[kRing][RUNS][K][kThreads][4 * W];
  int pos[kRing][2][kThreads];
  alignas(16) unsigned long long turns[1];

  // Runs `run` and run + 1 from the slot's first channel on.
  __device__ __forceinline__ void load(int at, int run, const ST* p, const Slot& s) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < K; ++i)
        copy_async<4 * W>(data[at][run + r][i][threadIdx.x], p + r * s.apart + i * s.hop);
  }
  __device__ __forceinline__ void load_pos(int at, const QkArgs& a, const Slot& s, int t) {
    copy_async<4>(&pos[at][0][threadIdx.x], a.pos + static_cast<long long>(s.axis_a) * a.T + t);
    if (s.on_b) copy_async<4>(&pos[at][1][threadIdx.x], a.pos + static_cast<long long>(s.axis_b) * a.T + t);
  }
  template <bool ADJ>
  __device__ __forceinline__ void read(int at, int run, f2* X, f2* Y) const {
    uint32_t w[2][K * W];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < K; ++i) get_words<W>(data[at][run + r][i][threadIdx.x], w[r] + i * W);
    pairs_of<ST, U, ADJ>(w[0], w[1], X, Y);
  }
  template <bool ADJ>
  __device__ __forceinline__ void angles(int at, const QkArgs& a, const Slot& sl, int t, f2* C, f2* S) const {
    const int same = a.pos ? 0 : t % a.seq;
    slot_angles<ST, U, ADJ>(a, sl, turns, t, a.pos ? pos[at][0][threadIdx.x] : same,
                            a.pos ? pos[at][1][threadIdx.x] : same, C, S);
  }
  // Turns, gain, and zeros for a lane without channels; readable after the block's next barrier.
  __device__ __forceinline__ const ST* fill(const QkArgs& a, const ST* g, const Slot& s) {
    ST* gain = reinterpret_cast<ST*>(turns + a.rot / 2);
    for (int p = threadIdx.x; p < a.rot / 2; p += kThreads) turns[p] = a.turns[p];
    if (g)
      for (int c = threadIdx.x; c < a.dh; c += kThreads) gain[c] = g[c];
    if (!s.on) {
      const uint32_t zero[W] = {};
#pragma unroll 1
      for (int i = 0; i < kRing * RUNS * K; ++i) put_words<W>(data[i / (RUNS * K)][i / K % RUNS][i % K][threadIdx.x], zero);
    }
    return gain;
  }
  static size_t bytes(const QkArgs& a) {
    return sizeof(Ring) - 16 + a.rot / 2 * sizeof(unsigned long long) + a.dh * sizeof(ST);
  }
};

// A block's items: the lane group's first one, their distance, and how many rounds of them.
struct Share {
  int which, rounds, len, chunks, shift;
  unsigned block, item, stride, items, magic;
  __device__ __forceinline__ Share(const QkArgs& a, const QkPlan& pl, int P, int sub) {
    which = blockIdx.x < static_cast<unsigned>(pl.blocks[0]) ? 0 : 1;
    block = blockIdx.x - (which ? pl.blocks[0] : 0);
    len = pl.len[which];
    chunks = pl.chunks[which];
    shift = pl.shift[which];
    magic = pl.magic[which];
    items = static_cast<unsigned>(chunks) * a.T;
    const unsigned first = block * kWarps * P;  // the same rounds for all warps of a block
    stride = pl.blocks[which] * kWarps * P;
    item = first + threadIdx.x / 32 * P + sub;
    rounds = pl.rounds[which] - (first + (pl.rounds[which] - 1) * stride >= items);
  }
};

// The token and the run of heads of an item; `heads`: how many of its `len` heads there are (none past the last item).
struct Item {
  int t, h0, heads;
  __device__ __forceinline__ Item(const Share& sh, unsigned item, int H) {
    t = static_cast<int>(item);
    h0 = 0;
    if (sh.chunks > 1) {
      t = static_cast<int>(__umulhi(item, sh.magic) >> sh.shift);
      h0 = static_cast<int>(item - static_cast<unsigned>(t) * sh.chunks) * sh.len;
    }
    heads = item < sh.items ? min(sh.len, H - h0) : 0;
  }
};

// --------------------------------------------------------------- dispatch
struct QkVariant {
  int u, g;  // channels of a run, lanes of a vector
};

// Runs of 8 channels where a bf16 vector divides into them (16-byte loads) and `wide` allows, else of 4; fp32 takes 4
// (16 bytes too).  Vectors of more than 256 channels take runs of 8 in both types, and then fill a warp.
inline QkVariant variant(const QkArgs& a, size_t es, bool wide = true) {
  wide = a.dh > 256 || (wide && es == 2 && a.dh % 16 == 0 && a.rot % 16 == 0);
  const int u = wide ? 8 : 4, slots = a.dh / (2 * u);
  // 6 and 3 vectors a warp, not 4 and 2: 16 + 2 heads of 72 in bf16, 40003 tokens: 46 us against 61 (floor 31).  The
  // same count would serve 3 and 6 slots (24 of 32 lanes now); it has not been built or measured for them.
  if (slots == 5 || slots == 9 || slots == 10) return {u, slots == 5 ? 5 : 10};
  return {u, slots <= 4 && es == 2 ? 4 : slots <= 8 ? 8 : slots <= 16 ? 16 : 32};
}

inline int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

constexpr int kMostHeads = 16;  // of an item: past it the angles cost nothing any more
constexpr int kMostWaves = 4;   // blocks of a launch for each that runs at once
constexpr int kWaveSteps = 12;  // heads a lane group takes at least, where the launch has more blocks than run at once

// Cuts each token's heads into items, and gives each tensor blocks by its share of the work.  Small launches: all
// blocks run at once and a lane group takes one item, as short as lets them.  Large ones: up to kMostWaves blocks for
// each that runs at once, since SMs do not get the same share of the memory's bandwidth and a block that ends early
// makes room for another (16384 tokens, 64 heads: 95 us with one block for each that runs at once, 90, 85 and 82 us with
// two, three and four; a launch of 300,000 vectors gains nothing and pays for the blocks' starts).  Items are then as
// long as gives the fewest steps to the longest block, an item's angles counted as a step and a half.
inline void cut(const QkArgs& a, int g, int resident, QkPlan* pl) {
  const long long groups = 32 / g * kWarps;  // of a block
  long long vectors[2];
  for (int i = 0; i < 2; ++i) vectors[i] = 1LL * a.T * a.t[i].H;
  const long long all = vectors[0] + vectors[1], each = (all + resident * groups - 1) / (resident * groups);
  const long long waves = std::max(1LL, std::min<long long>(kMostWaves, each / kWaveSteps));
  const long long most = resident * waves;
  long long least = 0;
  for (int e = static_cast<int>(each <= kMostHeads ? each : kMostHeads / 2); e <= kMostHeads; ++e) {
    QkPlan p;
    long long room[2], work[2], cost = 0;
    for (int i = 0; i < 2; ++i) {
      const int H = a.t[i].H;
      p.chunks[i] = cdiv(H, e);
      p.len[i] = H ? cdiv(H, p.chunks[i]) : 0;
      room[i] = (1LL * a.T * p.chunks[i] + groups - 1) / groups;
      work[i] = room[i] * (2 * p.len[i] + 3);
    }
    const bool fits = room[0] + room[1] <= most;
    const long long share = (work[0] * most + (work[0] + work[1]) / 2) / (work[0] + work[1]);
    for (int i = 0; i < 2; ++i) {
      p.blocks[i] = static_cast<int>(fits ? room[i] : std::min(std::max(i ? most - share : share, 1LL), room[i]));
      p.rounds[i] = room[i] ? cdiv(room[i], p.blocks[i]) : 0;
      cost = std::max(cost, 1LL * p.rounds[i] * (2 * p.len[i] + 3));
    }
    if (least == 0 || cost <= least) {
      least = cost;
      *pl = p;
    }
    if (fits) break;  // longer items only leave SMs idle
  }
  for (int i = 0; i < 2; ++i) {
    // 2^(31 + L) / chunks rounded up, L = log2 of chunks rounded up: exact for 31-bit dividends
    int log = 1;
    while ((1LL << log) < pl->chunks[i]) ++log;
    pl->shift[i] = log - 1;
    pl->magic[i] =
        pl->chunks[i] > 1 ? static_cast<unsigned>(((1ULL << (31 + log)) + pl->chunks[i] - 1) / pl->chunks[i]) : 0;
  }
}

using QkKernel = void (*)(QkArgs, QkPlan);

inline cudaError_t launch_qk(QkKernel kern, const QkArgs& a, const QkPlan& pl, size_t smem, cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(pl.blocks[0] + pl.blocks[1]), dim3(kThreads), smem, st, a, pl);
}

}  // namespace lr
