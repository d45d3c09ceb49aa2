// Forward of causal attention over packed sequences (tcgen05).
//
// An item is two row tiles (2 x 128 rows: consecutive tokens of a sequence with the G heads of a key head, see
// packed_device.cuh) against the keys up to their last token, 128 at a time.  Per tile t and key block j:
//
//   S_t = Q_t K_j^T            MMA, fp32 in TMEM
//   P_t = 2^(c S_t - m)        softmax warps, one row a thread, c = scale log2(e); m is the row's running maximum of
//                              c S, raised lazily; P (bf16) goes back over the first columns of S_t
//   O_t += P_t V_j             MMA with A = P from TMEM, fp32 accumulator in TMEM
//
// with l = sum 2^(c S - m) in fp32 of the unrounded terms.  m is raised only when a block's maximum passes it by more
// than 8 (powers of two), and O and l are scaled then: every formula holds for any m, and P stays below 2^8.  The two
// tiles take turns: while the softmax works on one, the tensor cores work on the other (O_0 += P_0 V_j, then the next
// S_0, then the same of tile 1), which is why an item has two.  A single tile per block left them waiting for each
// softmax.
//
// Keys past a row's token are masked in S by selection, so nothing that K holds there matters; P is 0 there, and so
// that 0 times V stays 0, rows of V past the end of the sequence are zeroed in shared memory before their product.
// Products run over the keys that any row of a tile can see, in steps of 16.
//
// Warps: 0 takes the items (the first is the block's own number, the others come from a counter) and loads them by TMA
// (Q_t per item; K_j, V_j into a ring of four 32 KB stages), 1 and 2 MMA issuers of tile 0 and 1 (1 also allocates TMEM),
// 3 idle, 4-7 and 8-11 softmax and output of tile 0 and 1.  TMEM: S_t at columns 128 t, O_t at 256 + 128 t.  Every wait is
// bounded (error word, abort flag; each role drains what it issued, and TMEM is freed).
//
// What bounds it is the issuing: a wait takes its warp some 200 cycles even when there is nothing to wait for, and a
// commit 100.  16384 tokens, 32 over 8 heads: one issuer 2354 us, one for each tile 1929, by strict turns 1530 (both at
// will, so that their instructions interleave: 1803), a step without branches between its instructions and the turn
// awaited before P 1346 (1.63 PFLOP/s).  Without its exponentials the kernel gained 8 %, without the maxima 4 %.
#include <algorithm>
#include <type_traits>

#include "packed_device.cuh"

namespace lr {
namespace packed {
namespace fwd {

constexpr int kStages = 4;
constexpr int kStageOut = 4096;  // a warp's 32 rows x 64 columns of the output
constexpr int kSmem = 1024 + 2 * kTile + kStages * kTile + 8 * kStageOut + 512;
constexpr float kLazy = 8.f;

struct Maps {
  CUtensorMap q, k, v;
};

struct Args {
  PackedRows o;
  float* lse;
  float scale;
  int Hq, dh, G, tq;  // tq: tokens of a row tile
  unsigned magic;     // of G
  Taken taken;
  const int* offs;  // every item has a block of its own, which finds it here (null: the list of the first launch)
  int nseq, T;
  unsigned* err;
};

// The t-th item of sequences cut into blocks of `tokens`, in their order (a whole warp); its head is negative where there
// is none, or where any offset is out of order.
__device__ __forceinline__ int4 own_item(const Args& a, int tokens, unsigned t) {
  const int lane = threadIdx.x & 31, heads = a.taken.heads;
  const int want = static_cast<int>(t / heads);
  int4 item = make_int4(0, 0, 0, -1);
  int count = 0;
  bool bad = false;
  for (int base = 0; base < a.nseq; base += 32) {
    const int i = base + lane;
    int b = 0, len = 0, n = 0;
    if (i < a.nseq) {
      const int e = a.offs[i + 1];
      b = a.offs[i];
      if (b < 0 || e < b || e > a.T) {
        bad = true;
      } else {
        len = e - b;
        n = (len + tokens - 1) / tokens;
      }
    }
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    const int place = want - (count + s - n);
    const unsigned mine = __ballot_sync(0xffffffffu, place >= 0 && place < n);
    if (mine) {
      const int from = __ffs(mine) - 1;
      item = make_int4(__shfl_sync(0xffffffffu, b, from), __shfl_sync(0xffffffffu, len, from),
                       __shfl_sync(0xffffffffu, place, from) * tokens, static_cast<int>(t - 1u * want * heads));
    }
    count += __shfl_sync(0xffffffffu, s, 31);
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (t == 0 && lane == 0) atomicOr(a.err, DEV_ERR_OFFSETS);
    item.w = -1;
  }
  return item;
}

// This warp's part of P (of 64 keys) is in TMEM.
__device__ __forceinline__ void p_ready(uint64_t* bar) {
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The softmax of one row over NC chunks of 32 keys of a block, and P written back, 64 keys at a time: the product of the
// first half runs while the second is computed.
template <int NC>
__device__ __forceinline__ void softmax_block(uint32_t ts, uint32_t to, int ocols, float c, int lim, bool masked,
                                              bool valid, float& m, float& l, bool first, uint64_t* p_full) {
  float x[32 * NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
  tmem_ld_wait();
  if (masked) {
#pragma unroll
    for (int i = 0; i < 32 * NC; ++i)
      if (i > lim) x[i] = -INFINITY;
  }
  float mx[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) mx[u] = max3(x[3 * u], x[3 * u + 1], x[3 * u + 2]);
#pragma unroll
  for (int i = 12; i + 1 < 32 * NC; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], x[i], x[i + 1]);
  const float bm = c * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  const bool raise = valid && (first || bm > m + kLazy);
  const float m_new = raise ? (first ? bm : fmaxf(m, bm)) : m;
  const float alpha = raise && !first ? exp2f(m - m_new) : 1.f;
  if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
    // S of this block complete implies that the product of the block before is: they are issued in that order.
    for (int cc = 0; cc < ocols; cc += 32) {
      float o[32];
      tmem_ld32(to + cc, o);
      tmem_ld_wait();
#pragma unroll
      for (int u = 0; u < 32; ++u) o[u] *= alpha;
      tmem_st32(to + cc, o);
    }
  }
  l *= alpha;
  m = m_new;
  const uint64_t cc = f2_pack(c, c), nm = f2_pack(-m, -m);
  uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    uint32_t pk[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      float a, b;
      f2_unpack(f2_fma(f2_pack(x[32 * i + 2 * u], x[32 * i + 2 * u + 1]), cc, nm), a, b);
      a = ex2_ftz(a);
      b = ex2_ftz(b);
      ls[u & 3] = f2_add(ls[u & 3], f2_pack(a, b));
      pk[u] = pack_bf16x2(a, b);
    }
    tmem_st16u(ts + 16 * i, pk);
    if (i & 1) p_ready(p_full + (i >> 1));
  }
  float s[8];
#pragma unroll
  for (int u = 0; u < 4; ++u) f2_unpack(ls[u], s[2 * u], s[2 * u + 1]);
  l += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

__global__ void __launch_bounds__(kThreads, 1) packed_fwd_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                   // [2]
  uint8_t* sKV = sQ + 2 * kTile;        // [kStages], K and V of a block by turns
  uint8_t* sO = sKV + kStages * kTile;  // [8 warps]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sO + 8 * kStageOut);
  uint64_t* q_full = bars;        // [2]
  uint64_t* q_free = bars + 2;    // [2] the tile's last S has read Q
  uint64_t* kv_full = bars + 4;   // [kStages]
  uint64_t* kv_empty = bars + 8;  // [kStages]
  uint64_t* s_full = bars + 12;   // [2]
  uint64_t* p_full = bars + 14;   // [2][2] P of 64 keys
  uint64_t* o_last = bars + 18;   // [2] the tile's last product is complete
  uint64_t* o_free = bars + 20;   // [2] its output has been read
  uint64_t* drain = bars + 22;    // [2]
  uint64_t* turn = bars + 24;     // [2] the tile's issuer may issue
  uint64_t* item_full = bars + 26;            // [kItems]
  uint64_t* item_empty = item_full + kItems;  // [kItems]
  int4* sitem = reinterpret_cast<int4*>(item_empty + kItems);  // [kItems], 16-byte aligned
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sitem + kItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kReaders = 2 + 8;  // MMA issuers, softmax warps

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_last[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&drain[i], 1);
      mbar_init(&turn[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kReaders);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int halves = a.dh > 64 ? 2 : 1, ksteps = (a.dh + 15) / 16, dh16 = ksteps * 16;
  pdl_wait();

  // Item `it` of this block; false when the wait gave up.  head < 0: there are no more.
  auto next_item = [&](int it, Item& x) -> bool {
    const int slot = it % kItems;
    if (!mbar_wait(&item_full[slot], static_cast<uint32_t>((it / kItems) & 1), abort_flag, a.err, DEV_ERR_TIMEOUT_MMA))
      return false;
    const volatile int* p = reinterpret_cast<const volatile int*>(&sitem[slot]);
    x = Item{p[0], p[1], p[2], p[3]};
    return true;
  };

  if (warp < 4) {
    regs_down<kRegsFew>();
    int4 own = make_int4(0, 0, 0, -1);
    if (warp == 0 && a.offs) own = own_item(a, 2 * a.tq, blockIdx.x);
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------ scheduler and producer
      bool ok = true;
      int g = 0, q_issued[2] = {0, 0};
      auto load_tile = [&](const CUtensorMap* map, int row, int head) {
        const int st = g % kStages;
        if (!mbar_wait(&kv_empty[st], static_cast<uint32_t>((g / kStages) & 1) ^ 1u, abort_flag, a.err,
                       DEV_ERR_TIMEOUT_PRODUCER))
          return false;
        mbar_expect_tx(&kv_full[st], halves * kHalf);
        for (int h = 0; h < halves; ++h)
          tma_load_3d(sKV + st * kTile + h * kHalf, map, &kv_full[st], 64 * h, head, row);
        ++g;
        return true;
      };
      auto load_q = [&](int tile, const Item& x) {
        if (!mbar_wait(&q_free[tile], static_cast<uint32_t>(q_issued[tile] & 1) ^ 1u, abort_flag, a.err,
                       DEV_ERR_TIMEOUT_PRODUCER))
          return false;
        mbar_expect_tx(&q_full[tile], halves * a.G * a.tq * 128);
        for (int h = 0; h < halves; ++h)
          tma_load_3d(sQ + tile * kTile + h * kHalf, &maps.q, &q_full[tile], 64 * h, x.head * a.G,
                      x.row0 + x.t0 + tile * a.tq);
        ++q_issued[tile];
        return true;
      };
      unsigned t = blockIdx.x;
      for (int it = 0; ok; ++it) {
        int4 v = own;
        if (a.offs) own.w = -1;  // the only one
        else v = a.taken.item(t);
        const int slot = it % kItems;
        ok = mbar_wait(&item_empty[slot], static_cast<uint32_t>((it / kItems) & 1) ^ 1u, abort_flag, a.err,
                       DEV_ERR_TIMEOUT_PRODUCER);
        if (!ok) break;
        sitem[slot] = v;
        mbar_arrive(&item_full[slot]);  // release: the readers see the item
        if (v.w < 0) break;
        const Item x{v.x, v.y, v.z, v.w};
        const int n1 = x.nblocks(1, a.tq), nmax = max(x.nblocks(0, a.tq), n1);
        ok = load_q(0, x);
        for (int j = 0; j < nmax && ok; ++j) {
          const int row = x.row0 + j * kRows;
          // The next item is taken as late as the loads that are left cover the counter's latency: taken earlier, it
          // would bind the last items to blocks that are still busy.
          if (!a.offs && j == max(0, nmax - 2)) t = gridDim.x + atomicAdd(a.taken.next, 1u);
          ok = load_tile(&maps.k, row, x.head);
          if (ok && j == 0 && n1 > 0) ok = load_q(1, x);
          ok = ok && load_tile(&maps.v, row, x.head);
        }
      }
      if (!ok) {  // the copies in flight end before the block does
        for (int k = max(0, g - kStages); k < g; ++k) drain_wait(&kv_full[k % kStages], (k / kStages) & 1);
        for (int t = 0; t < 2; ++t)
          if (q_issued[t]) drain_wait(&q_full[t], (q_issued[t] - 1) & 1);
      }
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------ MMA issuers, one for each tile
      const int t = uniform(warp - 1);
      const uint32_t id_s = idesc_n<false>(kRows);  // S = Q K^T: both K-major
      const uint32_t id_o = idesc_n<true>(dh16);    // O += P V: P from TMEM, V MN-major
      const uint32_t ts = uniform(tmem) + t * kRows, to = ts + 2 * kRows;
      const Desc qd = sdesc(smem_addr(sQ + t * kTile), 16, 1024), kd = sdesc(smem_addr(sKV), 16, 1024),
                 vd = sdesc(smem_addr(sKV) + kTile, kHalf, 1024);
      bool ok = true;
      uint32_t b = 0;  // key blocks so far: K of block b in stage 2 (b & 1), V in the one behind it
      uint32_t p_of = 0, p_second = 0, items = 0, turns = 0;  // the tile's blocks, second halves of P, items and turns
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return warp_wait(bar, phase & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA);
      };
      auto take_turn = [&] {
        ++turns;
        return wait(&turn[t], t ? turns + 1 : turns);
      };
      auto pass_turn = [&] {
        if (elect()) mbar_arrive(&turn[1 - t]);
      };
      for (int it = 0; ok; ++it) {
        Item x;
        ok = __all_sync(0xffffffffu, next_item(it, x));
        if (!ok) break;
        x = Item{uniform(x.row0), uniform(x.len), uniform(x.t0), uniform(x.head)};
        if (elect()) mbar_arrive(&item_empty[it % kItems]);
        if (x.head < 0) break;
        const int n = x.nblocks(t, a.tq), nmax = max(x.nblocks(0, a.tq), x.nblocks(1, a.tq));
        const int last = x.keys(t, a.tq) - (n - 1) * kRows;  // keys of the tile's last block that some row sees
        auto issue_s = [&](int j, uint32_t blk) {  // S of block j, which is the blk-th of all
          const Desc k = kd.at(2 * kTile * (blk & 1));
          if (ksteps == 8) mma_ss_n<8>(ts, qd, k, id_s);
          else mma_ss(ts, qd, k, id_s, ksteps);
          mbar_arrive(&turn[1 - t]);  // the turn passes before the commits, which take the issuer some 100 cycles each
          commit1(&s_full[t]);
          commit1(&kv_empty[2 * (blk & 1)]);
          if (j + 1 == n) commit1(&q_free[t]);
        };
        ok = (n == 0 || (wait(&q_full[t], items) && wait(&kv_full[2 * (b & 1)], b >> 1))) && take_turn();
        if (!ok) break;
        tc_fence_after();
        if (n == 0) pass_turn();
        else if (elect()) issue_s(0, b);
        for (int j = 0; j < nmax && ok; ++j, ++b) {
          uint64_t* v_full = &kv_full[2 * (b & 1) + 1];
          uint64_t* v_empty = &kv_empty[2 * (b & 1) + 1];
          if (j >= n) {  // the other tile's block: this one's part of its release, once it is there
            ok = wait(&kv_full[2 * (b & 1)], b >> 1) && wait(v_full, b >> 1) && take_turn();
            if (ok && elect()) {
              mbar_arrive(&kv_empty[2 * (b & 1)]);
              mbar_arrive(v_empty);
            }
            pass_turn();
            continue;
          }
          const Desc v = vd.at(2 * kTile * (b & 1));
          if (j + 1 < n) {
            ok = wait(v_full, b >> 1) && wait(&kv_full[2 * ((b + 1) & 1)], (b + 1) >> 1) &&
                 (j > 0 || wait(&o_free[t], items + 1)) && take_turn() && wait(&p_full[2 * t], p_of++);
            if (!ok) break;
            tc_fence_after();
            if (elect()) mma_ts_n<4>(to, ts, v, id_o, j > 0 ? 1u : 0u);
            ok = wait(&p_full[2 * t + 1], p_second++);
            if (!ok) break;
            tc_fence_after();
            if (elect()) {
              mma_ts_n<4>(to, ts + 32, v.at(4 * 2048), id_o, 1u);
              issue_s(j + 1, b + 1);
              commit1(v_empty);
            }
            continue;
          }
          ok = wait(v_full, b >> 1);
          const int steps = (last + 15) / 16, left = x.len - j * kRows;
          if (ok && left < 16 * steps) {  // rows past the sequence's end that the product's last step reads
            zero_rows(sKV + (2 * (b & 1) + 1) * kTile, left, 16 * steps, halves);  // (both issuers: the same zeroes)
            fence_async_smem();
            __syncwarp();
          }
          ok = ok && (j > 0 || wait(&o_free[t], items + 1)) && wait(&p_full[2 * t], p_of++) && take_turn();
          if (!ok) break;
          tc_fence_after();
          if (elect()) mma_ts(to, ts, v, id_o, j > 0 ? 1u : 0u, min(4, steps));
          if (steps > 4) {
            ok = wait(&p_full[2 * t + 1], p_second++);
            if (!ok) break;
            tc_fence_after();
            if (elect()) mma_ts(to, ts + 32, v.at(4 * 2048), id_o, 1u, steps - 4);
          }
          if (elect()) {
            mbar_arrive(&turn[1 - t]);
            commit1(&o_last[t]);
            commit1(v_empty);
          }
        }
        if (n > 0) ++items;
      }
      if (elect()) {
        commit1(&drain[t]);  // every MMA issued here is complete once this flips
        drain_wait(&drain[t], 0);
      }
      __syncwarp();
    }
  } else {
    regs_up<kRegsMany>();
    // ------------------------------------------------ softmax and output
    const int tile = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + tile * kRows, to = tmem + lanes + 2 * kRows + tile * kRows;
    const float c = a.scale * kLog2e;
    const int tok = group_div(row, a.magic);
    const uint32_t stage = smem_addr(sO + (warp - 4) * kStageOut);
    int s_of = 0, items_of = 0;
    for (int it = 0;; ++it) {
      Item x;
      if (!__all_sync(0xffffffffu, next_item(it, x))) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it % kItems]);
      if (x.head < 0) break;
      const int n = x.nblocks(tile, a.tq);
      if (n == 0) continue;
      const int first = x.t0 + tile * a.tq, keys = x.keys(tile, a.tq);  // the tile's first token, the keys it sees
      const int place = first + tok;
      const bool valid = tok < a.tq && place < x.len;
      float m = 0.f, l = 0.f;
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        ok = warp_wait(&s_full[tile], static_cast<uint32_t>(s_of++ & 1), abort_flag, a.err, DEV_ERR_TIMEOUT_EPILOGUE);
        if (!ok) break;
        tc_fence_after();
        const int lim = place - j * kRows;             // the last key of the block that the row sees
        const bool masked = first < j * kRows + kRows - 1;  // some row does not see all of them
        if (keys - j * kRows > 64)
          softmax_block<4>(ts, to, dh16, c, lim, masked, valid, m, l, j == 0, &p_full[2 * tile]);
        else
          softmax_block<2>(ts, to, dh16, c, lim, masked, valid, m, l, j == 0, &p_full[2 * tile]);
      }
      if (!ok) break;
      if (!warp_wait(&o_last[tile], static_cast<uint32_t>(items_of++ & 1), abort_flag, a.err, DEV_ERR_TIMEOUT_EPILOGUE))
        break;
      tc_fence_after();
      // O / l, 64 columns at a time through the warp's staging rows, so that eight lanes write 128 bytes of a row.
      const float inv = 1.f / l;
      if (valid)
        a.lse[1LL * (x.row0 + place) * a.Hq + x.head * a.G + (row - tok * a.G)] = (m + log2f(l)) * kLn2;
      for (int h = 0; h < halves; ++h) {
        float o[64];
        tmem_ld32(to + 64 * h, o);
        tmem_ld32(to + 64 * h + 32, o + 32);
        tmem_ld_wait();
        if (h + 1 == halves) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[tile]);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          sts128(stage + lane * 128 + ((u ^ (lane & 7)) << 4), pack_bf16x2(o[8 * u] * inv, o[8 * u + 1] * inv),
                 pack_bf16x2(o[8 * u + 2] * inv, o[8 * u + 3] * inv), pack_bf16x2(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                 pack_bf16x2(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
        __syncwarp();
        const int col = 64 * h + 8 * (lane & 7);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = 4 * u + (lane >> 3), full = quarter * 32 + r, t = group_div(full, a.magic);
          uint4 w;
          umma::lds128(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4), w.x, w.y, w.z, w.w);
          if (t < a.tq && first + t < x.len && col < a.dh)
            *reinterpret_cast<uint4*>(a.o.p + (x.row0 + first + t) * a.o.ld +
                                      1LL * (x.head * a.G + full - t * a.G) * a.dh + col) = w;
        }
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace fwd
}  // namespace packed

size_t packed_attn_fwd_ws_bytes(int T, int nseq, int Hq, int Hk) {
  return packed::plan_layout(T, nseq, 2 * (packed::kRows / (Hq / Hk)), nullptr, nullptr);
}

cudaError_t launch_packed_attn_fwd(const PackedArgs& p, void* ws, unsigned* err, cudaStream_t st, int* launches) {
  using namespace packed;
  using namespace packed::fwd;
  cudaError_t e = configure<packed_fwd_kernel, kSmem>();
  if (e != cudaSuccess) return e;
  const int G = p.Hq / p.Hk, tq = kRows / G;
  fwd::Maps maps;
  memset(&maps, 0, sizeof(maps));
  if (!encode_heads(&maps.q, p.q, p.T, p.Hq, p.dh, G, tq) || !encode_heads(&maps.k, p.k, p.T, p.Hk, p.dh, 1, kRows) ||
      !encode_heads(&maps.v, p.v, p.T, p.Hk, p.dh, 1, kRows))
    return cudaErrorInvalidValue;
  PlanJob job{{}, 2 * tq, 1};
  plan_layout(p.T, p.nseq, job.tokens, ws, &job.plan);
  const long long items = plan_capacity(p.T, p.nseq, 2 * tq) * p.Hk, sms = device_sm_count();
  // Where every item has an SM of its own their order does not matter, and finding one takes less than a launch that makes
  // a list (17 tokens, 32 over 8 heads: 8.2 us, with the list 10.4).
  const bool own = items <= sms && p.nseq <= 256;
  if (!own) {
    e = launch_prepare(p, &job, 1, nullptr, err, st);
    if (e != cudaSuccess) return e;
  }
  const fwd::Args a{p.o, p.lse, p.scale, p.Hq, p.dh, G, tq, group_magic(G), taken(job.plan, p.Hk, 4LL * p.T * p.dh),
                    own ? p.offs : nullptr, p.nseq, p.T, err};
  *launches = own ? 1 : 2;
  return launch_as(!own && pdl_allowed(), packed_fwd_kernel, dim3(static_cast<unsigned>(std::min(items, sms))), dim3(kThreads),
                   kSmem, st, maps, a);
}

}  // namespace lr
