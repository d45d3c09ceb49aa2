// Pieces that the packed-attention kernels share: how the sequences are cut into items, the list of them that a first
// launch makes on the device, the ring through which a block's warps receive items, and loads of head rows.
//
// A row tile is 128 rows of the matrix instruction: tq = 128 / G tokens with the G query heads of one key head each
// (token-major, rows tq G .. 127 unused).  Grouped heads then share the loads of their keys, a tile of few tokens is
// still full, and its causal edge is as long as its tokens, not as its rows.
//
// The list holds blocks of one sequence, the ones with the most work first (a counting sort by work, in bins); an item
// is a block with a key head.  Items are taken in groups of key heads whose operands stay in L2.
#pragma once

#include "attn_flash.cuh"
#include "f32x2.cuh"
#include "packed_attn.cuh"

namespace lr {
namespace packed {

using namespace flash;

constexpr int kItems = 2;  // slots of the item ring

// What the first launch leaves in the workspace.
struct Plan {
  unsigned* next;  // items taken beyond the blocks' first ones
  int* nblocks;
  int4* blocks;    // first row, length of the sequence, place of the block's first token in it, 0
  int* starts;     // [nseq + 1] blocks before each sequence
};

// The most blocks of `tokens` tokens that the sequences can have.
inline long long plan_capacity(int T, int nseq, int tokens) {
  const long long n = T / tokens + 1LL * nseq;
  return n < T ? n : T;
}
size_t plan_layout(int T, int nseq, int tokens, void* base, Plan* plan);

struct PlanJob {
  Plan plan;
  int tokens;
  int work;  // +1: a block's work grows with its place (its keys), -1: with what follows it (its queries)
};
// One launch: the lists, and (D not null) D[t, h] = dout.o of every row and head.  It starts when everything before it has
// ended, and lets the launch that follows it begin at once (that one waits for it before its first access).
cudaError_t launch_prepare(const PackedArgs& a, const PlanJob* jobs, int njobs, float* D, unsigned* err, cudaStream_t st);

// What an item needs, from its ring slot.
struct Item {
  int row0, len, t0, head;  // the sequence's first row and length, the item's first token in it, the key head
  // Tokens of a row tile of tq, the keys that some row of it sees, and the key blocks they are in.
  __device__ __forceinline__ int tokens(int tile, int tq) const { return min(tq, len - t0 - tile * tq); }  // may be < 1
  __device__ __forceinline__ int keys(int tile, int tq) const {
    const int n = tokens(tile, tq);
    return n > 0 ? t0 + tile * tq + n : 0;
  }
  __device__ __forceinline__ int nblocks(int tile, int tq) const { return (keys(tile, tq) + kRows - 1) / kRows; }
};

// The items of a launch, in the order they are taken.
struct Taken {
  const int* nblocks;
  const int4* blocks;
  unsigned* next;
  int heads, group;  // key heads, and how many are worked on together
  int parts;         // an item is this many: each with a part of what it has to go through
  // The t-th: an Item, its head negative past the end, its part in the bits above the head's 24.
  __device__ __forceinline__ int4 item(unsigned t) const {
    const unsigned n = static_cast<unsigned>(*nblocks), part = parts > 1 ? t % parts : 0;
    if (parts > 1) t /= parts;
    if (t >= n * heads) return make_int4(0, 0, 0, -1);
    const unsigned per = group * n, gi = t / per, r = t - gi * per;
    const unsigned gh = min(group, heads - static_cast<int>(gi) * group);
    int4 v = blocks[r / gh];
    v.w = static_cast<int>(gi * group + r % gh + (part << 24));
    return v;
  }
};
inline Taken taken(const Plan& plan, int heads, long long bytes_per_head, int parts = 1) {
  return Taken{plan.nblocks, plan.blocks, plan.next, heads, heads_per_group(heads, bytes_per_head), parts};
}

// Registers a thread of the kernels of 12 warps: the launch gives 168; the first four warps keep 88, the others take 208
// (88 + 2 x 208 is 3 x 168).
constexpr int kRegs = 168, kRegsFew = 88, kRegsMany = 208;
static_assert(kRegsFew + 2 * kRegsMany <= 3 * kRegs, "register split");

// Once per device: the shared memory of a kernel, and that its registers allow the split (warps would wait for them
// forever).
template <auto Kernel, int Smem>
cudaError_t configure() {
  static int done = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 32) return cudaErrorInvalidDevice;
  if (__atomic_load_n(&done, __ATOMIC_ACQUIRE) & (1 << dev)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, Kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * kThreads < 128 * kRegsFew + 256 * kRegsMany) return cudaErrorInvalidConfiguration;
  __atomic_fetch_or(&done, 1 << dev, __ATOMIC_RELEASE);
  return cudaSuccess;
}

// The tensor maps of the backward's kernels.
struct BwdMaps {
  CUtensorMap q, dout, k, v;
};

struct DqArgs {
  PackedRows dq;
  const float *lse, *D;
  float scale;
  int Hq, dh, G, tq;
  unsigned magic;
  Taken taken;
  unsigned* err;
};

struct DkvArgs {
  PackedRows dk, dv;
  float *part_dk, *part_dv;  // more than one part: their sums, [parts, T, Hk, dh]
  int T, Hk;
  const float *lse, *D;
  float scale;
  int Hq, dh, G, tq;
  unsigned magic;
  Taken taken;
  unsigned* err;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Instruction descriptor for M = 128 and a run-time N (a multiple of 16).
template <bool B_MN>
__device__ __forceinline__ uint32_t idesc_n(int n) {
  return idesc_m128<B_MN, 16>() - (2u << 17) + (static_cast<uint32_t>(n >> 3) << 17);
}

// One thread issues a tile's matrix instructions and stands still until the tensor cores take each (64 cycles at
// N = 128), so what it computes between them is lost to them: 17 instructions each made 86 cycles of it beside busy softmax
// warps, a loop over the steps 130 to 200.  The forms below come out at 64: all counts of steps are unrolled, only
// the low words of descriptors move, and the one thread is elected where it issues (not by its lane), which lets the
// compiler keep the operands in the registers of the whole warp.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ Desc(uint64_t d) : lo(static_cast<uint32_t>(d)), hi(static_cast<uint32_t>(d >> 32)) {}
  __device__ __forceinline__ Desc at(int bytes) const {  // addresses are below 2^18: no carry out of their field
    Desc d = *this;
    d.lo += static_cast<uint32_t>(bytes >> 4);
    return d;
  }
};

__device__ __forceinline__ void mma_ss1(uint32_t d, Desc a, Desc b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts1(uint32_t d, uint32_t a, Desc b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}

// d = A B^T over `steps` (1 to 8) steps of 16 channels, both K-major tiles of 64-column halves.
template <int STEPS>
__device__ __forceinline__ void mma_ss_n(uint32_t d, Desc a, Desc b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) {
    const int off = (kk >> 2) * kHalf + (kk & 3) * 32;
    mma_ss1(d, a.at(off), b.at(off), idesc, kk > 0 ? 1u : 0u);
  }
}
__device__ __forceinline__ void mma_ss(uint32_t d, Desc a, Desc b, uint32_t idesc, int steps) {
  switch (steps) {
    case 8: return mma_ss_n<8>(d, a, b, idesc);
    case 7: return mma_ss_n<7>(d, a, b, idesc);
    case 6: return mma_ss_n<6>(d, a, b, idesc);
    case 5: return mma_ss_n<5>(d, a, b, idesc);
    case 4: return mma_ss_n<4>(d, a, b, idesc);
    case 3: return mma_ss_n<3>(d, a, b, idesc);
    case 2: return mma_ss_n<2>(d, a, b, idesc);
    default: return mma_ss_n<1>(d, a, b, idesc);
  }
}

// d (+)= A B over `steps` (1 to 4) steps of 16 rows: A packed bf16 in TMEM, 8 columns a step, B an MN-major tile.
template <int STEPS>
__device__ __forceinline__ void mma_ts_n(uint32_t d, uint32_t a, Desc b, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) mma_ts1(d, a + 8 * kk, b.at(2048 * kk), idesc, kk > 0 ? 1u : acc);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, Desc b, uint32_t idesc, uint32_t acc, int steps) {
  switch (steps) {
    case 1: return mma_ts_n<1>(d, a, b, idesc, acc);
    case 2: return mma_ts_n<2>(d, a, b, idesc, acc);
    case 3: return mma_ts_n<3>(d, a, b, idesc, acc);
    default: return mma_ts_n<4>(d, a, b, idesc, acc);
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Heads of T rows: boxes of 64 channels x `heads` heads x `tokens` rows, channels beyond dh read as 0.
inline bool encode_heads(CUtensorMap* m, const PackedRows& x, int T, int H, int dh, int heads, int tokens) {
  const long long dims[3] = {dh, H, T}, strides[2] = {dh, x.ld};
  const int box[3] = {64, heads, tokens};
  return umma::encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x.p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// r / G for r < 128, G <= 128: ceil(2^16 / G) is above 2^16 / G by less than 1, which 128 times stays below 2^16 / 128.
__host__ __device__ __forceinline__ unsigned group_magic(int G) { return (65536u + G - 1) / G; }
__device__ __forceinline__ int group_div(int r, unsigned magic) {
  return static_cast<int>((static_cast<unsigned>(r) * magic) >> 16);
}

// Zeroes rows a .. b - 1 of a tile of `halves` 64-column halves (a whole warp).
__device__ __forceinline__ void zero_rows(uint8_t* tile, int a, int b, int halves) {
  const int lane = threadIdx.x & 31, per = 8 * halves;
  for (int i = lane; i < (b - a) * per; i += 32) {
    const int r = a + i / per, c = i % per;
    sts128(smem_addr(tile) + (c >> 3) * kHalf + r * 128 + ((c & 7) << 4), 0u, 0u, 0u, 0u);
  }
}

// A place in a ring of loads, and the parity of its turn there.
struct Ring {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++stage == n) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// Waits of a whole warp (the same answer in every lane).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err,
                                          unsigned code) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, code));
}

// A value that every lane holds, known to the compiler as one of the whole warp: what follows from it is computed once
// and is at hand for the matrix instructions, which take their operands from such registers.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Waits, for a limited time, for a copy or MMA in flight before the block ends (error paths).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_test(bar, parity) && global_timer_ns() - t0 < umma::kWaitLimitNs) {
  }
}

template <int R>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

}  // namespace packed
}  // namespace lr
