// dK and dV of causal attention over packed sequences (tcgen05).
//
// An item is a block of 128 keys of one key head against the row tiles (128 rows: tokens with the G heads of the key
// head, see packed_device.cuh) from the first that holds one of its tokens to the sequence's last.  With the keys on the
// MMA rows, per row tile i:
//
//   S^T = K Q_i^T, dP^T = V dO_i^T      MMA, fp32 in TMEM
//   P^T = 2^(c S^T - lse log2 e)        element-wise warps, two threads a key; bf16 back over the columns of S^T
//   dS^T = P^T (dP^T - D)               the same over those of dP^T
//   dV += P^T dO_i, dK += dS^T Q_i      MMA with A from TMEM; dK takes the scale at the end
//
// Where there are few items, each is cut in parts of its row tiles, whose sums a further launch adds up in order
// (one sequence of 1024 tokens, 32 over 8 heads: 64 items, of which the first had 32 tiles).
//
// The heads of a group add up in the same accumulators, in a fixed order.  TMEM is full (S^T, dP^T, dV and dK, 128
// columns each; up to 64 channels dV and dK leave half of theirs unused), so S^T and dP^T have one buffer; what keeps the
// tensor cores at work is that they belong to two chains: one issuer takes dV of tile i and then S^T of tile i + 1, the
// other dK of tile i and then dP^T of tile i + 1, by turns, and the element-wise warps compute P while the second has its
// turn and dS while the first has.
//
// Rows past the end of the sequence get P = dS = 0 by selection, and rows of dO and Q there are zeroed in shared memory
// before their products.  Rows of a tile that no token has (128 is no multiple of G) stay zero from the start.
//
// Q_i is needed from S^T of tile i to dK of tile i, four turns, and dO_i from dP^T to dV, two; so Q has three stages and dO
// two (with two of both, loads came 600 cycles late for each tile).  That leaves 3 KB of shared memory: dK and dV are
// written straight from registers.
//
// Warps: 0 takes the items and loads them by TMA (K, V per item; Q_i, dO_i into their rings), 1 issuer of S^T
// and dV, which also allocates TMEM, 2 issuer of dP^T and dK, 3 loads lse and D of each tile, 4-11 element-wise and output
// (warp group h takes rows 64 h .. 64 h + 63 of a tile and columns 64 h .. of dK and dV).  TMEM: S^T at column 0, dP^T at
// 128, dV at 256, dK at 384.  Every wait is bounded (error word, abort flag; each role drains what it issued, and TMEM is
// freed).
#pragma once

#include "packed_device.cuh"

namespace lr {
namespace packed {
namespace dkv {

constexpr int kStagesQ = 3, kStagesO = 2;
constexpr int kStages = 2;  // of lse and D
constexpr int kSmem = (2 + kStagesQ + kStagesO) * kTile + kStages * 2 * kRows * 4 + 512;
static_assert(kSmem <= umma::kMaxSmem, "shared memory");

// An item's part of the row tiles of its key block; the head is taken out of the item's last word.
struct Tiles {
  int first, n, part;
  __device__ __forceinline__ Tiles(Item& x, int tq, int parts) {
    part = x.head >> 24;
    x.head &= 0xffffff;
    first = x.t0 / tq;
    const int all = (x.len + tq - 1) / tq - first, from = all * part / parts;
    n = all * (part + 1) / parts - from;
    first += from;
  }
};

// P of 64 rows (L: -lse log2 e of them) of one key from its scores, in place, and packed.  MASK: rows before `from` or from
// `rows` on do not see the key.
template <bool MASK>
__device__ __forceinline__ void exps(float* p, const float* L, float c, int from, int rows, uint32_t* w) {
  const uint64_t c2 = f2_pack(c, c);
#pragma unroll
  for (int u = 0; u < 64; u += 4) {
    const float4 l = *reinterpret_cast<const float4*>(L + u);
    f2_unpack(f2_fma(f2_pack(p[u], p[u + 1]), c2, f2_pack(l.x, l.y)), p[u], p[u + 1]);
    f2_unpack(f2_fma(f2_pack(p[u + 2], p[u + 3]), c2, f2_pack(l.z, l.w)), p[u + 2], p[u + 3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[u + e] = ex2_ftz(p[u + e]);
      if (MASK && (u + e < from || u + e >= rows)) p[u + e] = 0.f;
    }
    w[u >> 1] = pack_bf16x2(p[u], p[u + 1]);
    w[(u >> 1) + 1] = pack_bf16x2(p[u + 2], p[u + 3]);
  }
}

// dS = P (dP - D) of the same rows, packed (nD: -D of them).
template <bool MASK>
__device__ __forceinline__ void grads(const float* p, const float* d, const float* nD, int from, int rows, uint32_t* w) {
#pragma unroll
  for (int u = 0; u < 64; u += 4) {
    const float4 n = *reinterpret_cast<const float4*>(nD + u);
    float g[4];
    f2_unpack(f2_mul(f2_pack(p[u], p[u + 1]), f2_add(f2_pack(d[u], d[u + 1]), f2_pack(n.x, n.y))), g[0], g[1]);
    f2_unpack(f2_mul(f2_pack(p[u + 2], p[u + 3]), f2_add(f2_pack(d[u + 2], d[u + 3]), f2_pack(n.z, n.w))), g[2], g[3]);
    if (MASK) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (u + e < from || u + e >= rows) g[e] = 0.f;
    }
    w[u >> 1] = pack_bf16x2(g[0], g[1]);
    w[(u >> 1) + 1] = pack_bf16x2(g[2], g[3]);
  }
}

// One of `nblocks` blocks, the `block`-th.
__device__ __forceinline__ void body(const BwdMaps& maps, const DkvArgs& a, unsigned block, unsigned nblocks,
                                     uint8_t* smem) {
  uint8_t* sK = smem;
  uint8_t* sV = sK + kTile;
  uint8_t* sQ = sV + kTile;               // [kStagesQ]
  uint8_t* sdO = sQ + kStagesQ * kTile;   // [kStagesO]
  float* sL = reinterpret_cast<float*>(sdO + kStagesO * kTile);  // [kStages][128] -lse log2 e
  float* sD = sL + kStages * kRows;                            // [kStages][128] -D
  uint64_t* bars = reinterpret_cast<uint64_t*>(sD + kStages * kRows);
  uint64_t* kv_full = bars;
  uint64_t* kv_free = bars + 1;    // the item's last S^T and last dP^T have read K and V
  uint64_t* q_full = bars + 2;     // [kStagesQ]
  uint64_t* q_empty = bars + 5;    // [kStagesQ] dK of the tile is complete (it needs S^T of it, which is then too)
  uint64_t* o_full = bars + 8;     // [kStagesO]
  uint64_t* o_empty = bars + 10;   // [kStagesO] dP^T and dV of the tile are complete
  uint64_t* st_full = bars + 12;   // [kStages] lse and D
  uint64_t* st_empty = bars + 14;  // [kStages]
  uint64_t* s_full = bars + 16;
  uint64_t* dp_full = bars + 17;
  uint64_t* p_full = bars + 18;
  uint64_t* ds_full = bars + 19;
  uint64_t* acc_full = bars + 20;  // the item's last dV and dK are complete
  uint64_t* acc_free = bars + 21;  // they have been read
  uint64_t* turn = bars + 22;      // [2]
  uint64_t* drain = bars + 24;     // [2]
  uint64_t* item_full = bars + 26;            // [kItems]
  uint64_t* item_empty = item_full + kItems;  // [kItems]
  int4* sitem = reinterpret_cast<int4*>(item_empty + kItems);  // [kItems], 16-byte aligned
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sitem + kItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kReaders = 3 + 8;  // issuers, loader of lse and D, element-wise warps

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_free, 2);
    for (int i = 0; i < kStagesQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 2);
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], 8);
      mbar_init(&turn[i], 1);
      mbar_init(&drain[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 8);
    mbar_init(ds_full, 8);
    mbar_init(acc_full, 2);
    mbar_init(acc_free, 8);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kReaders);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (a.G * a.tq < kRows)  // rows that the loads never write
    for (int i = warp; i < kStagesQ + kStagesO; i += kThreads / 32) zero_rows(sQ + i * kTile, a.G * a.tq, kRows, 2);
  fence_async_smem();
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
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------ scheduler and producer
      bool ok = true;
      int g = 0, issued = 0;  // row tiles, and items
      auto wait = [&](uint64_t* bar, int phase) {
        return mbar_wait(bar, static_cast<uint32_t>(phase & 1) ^ 1u, abort_flag, a.err, DEV_ERR_TIMEOUT_PRODUCER);
      };
      auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
        for (int h = 0; h < halves; ++h) tma_load_3d(dst + h * kHalf, map, bar, 64 * h, head, row);
      };
      unsigned t = block;
      for (int it = 0; ok; ++it) {
        const int4 v = a.taken.item(t);
        const int slot = it % kItems;
        ok = wait(&item_empty[slot], it / kItems);
        if (!ok) break;
        sitem[slot] = v;
        mbar_arrive(&item_full[slot]);  // release: the readers see the item
        if (v.w < 0) break;
        Item x{v.x, v.y, v.z, v.w};
        const Tiles tiles(x, a.tq, a.taken.parts);
        if (tiles.n == 0) {
          t = nblocks + atomicAdd(a.taken.next, 1u);
          continue;
        }
        ok = wait(kv_free, issued);
        if (!ok) break;
        mbar_expect_tx(kv_full, 2 * halves * kHalf);
        load(sK, &maps.k, kv_full, x.head, x.row0 + x.t0);
        load(sV, &maps.v, kv_full, x.head, x.row0 + x.t0);
        ++issued;
        for (int i = 0; i < tiles.n && ok; ++i, ++g) {
          if (i == max(0, tiles.n - 2)) t = nblocks + atomicAdd(a.taken.next, 1u);  // late: see the forward
          const int sq = g % kStagesQ, so = g % kStagesO, bytes = halves * a.G * a.tq * 128;
          const int row = x.row0 + (tiles.first + i) * a.tq;
          ok = wait(&q_empty[sq], g / kStagesQ);
          if (!ok) break;
          mbar_expect_tx(&q_full[sq], bytes);
          load(sQ + sq * kTile, &maps.q, &q_full[sq], x.head * a.G, row);
          ok = wait(&o_empty[so], g / kStagesO);
          if (!ok) {
            drain_wait(&q_full[sq], (g / kStagesQ) & 1);
            break;
          }
          mbar_expect_tx(&o_full[so], bytes);
          load(sdO + so * kTile, &maps.dout, &o_full[so], x.head * a.G, row);
        }
      }
      if (!ok) {  // the copies in flight end before the block does
        for (int k = max(0, g - kStagesQ); k < g; ++k) drain_wait(&q_full[k % kStagesQ], (k / kStagesQ) & 1);
        for (int k = max(0, g - kStagesO); k < g; ++k) drain_wait(&o_full[k % kStagesO], (k / kStagesO) & 1);
        if (issued) drain_wait(kv_full, (issued - 1) & 1);
      }
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------ issuers: 0 of S^T and dV, 1 of dP^T and dK
      const int w = uniform(warp - 1);
      const uint32_t id_s = idesc_n<false>(kRows);  // K Q^T, V dO^T: all K-major
      const uint32_t id_g = idesc_n<true>(dh16);    // P^T dO, dS^T Q: A from TMEM, B MN-major
      const uint32_t ts = uniform(tmem) + w * kRows, tg = ts + 2 * kRows;
      const int steps = (a.tq * a.G + 15) / 16;  // of 16 rows of a tile
      const bool full = steps == 8 && ksteps == 8;
      uint8_t* sS = w ? sdO : sQ;  // B of the scores
      uint8_t* sG = w ? sQ : sdO;  // B of the gradient
      const Desc ad = sdesc(smem_addr(w ? sV : sK), 16, 1024), sd = sdesc(smem_addr(sS), 16, 1024),
                 gd = sdesc(smem_addr(sG), kHalf, 1024);
      uint64_t* bs_full = w ? o_full : q_full;
      uint64_t* bg_full = w ? q_full : o_full;
      uint64_t* bg_empty = w ? q_empty : o_empty;
      const uint32_t ns = w ? kStagesO : kStagesQ, ng = w ? kStagesQ : kStagesO;
      uint64_t* score_full = w ? dp_full : s_full;
      uint64_t* mine_full = w ? ds_full : p_full;
      bool ok = true;
      uint32_t items = 0, mine = 0, turns = 0;
      Ring s, g;  // the tile of the next score, and of the next gradient
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return warp_wait(bar, phase & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA);
      };
      auto take_turn = [&] {
        ++turns;
        return wait(&turn[w], w ? turns + 1 : turns);
      };
      // Behind a score: the turn passes first, for a commit takes its issuer some 100 cycles.
      auto score_issued = [&](bool last) {
        mbar_arrive(&turn[1 - w]);
        commit1(score_full);
        if (w) commit1(&o_empty[s.stage]);
        if (last) commit1(kv_free);
      };
      for (int it = 0; ok; ++it) {
        Item x;
        ok = __all_sync(0xffffffffu, next_item(it, x));
        if (!ok) break;
        x = Item{uniform(x.row0), uniform(x.len), uniform(x.t0), uniform(x.head)};
        if (elect()) mbar_arrive(&item_empty[it % kItems]);
        if (x.head < 0) break;
        const Tiles tiles(x, a.tq, a.taken.parts);
        if (tiles.n == 0) continue;
        const int left = min(a.tq, x.len - (tiles.first + tiles.n - 1) * a.tq) * a.G;  // rows of the last tile
        ok = wait(kv_full, items) && wait(&bs_full[s.stage], s.phase) && take_turn();
        if (!ok) break;
        tc_fence_after();
        if (elect()) {
          mma_ss(ts, ad, sd.at(s.stage * kTile), id_s, ksteps);
          score_issued(tiles.n == 1);
        }
        s.next(ns);
        ok = wait(acc_free, items + 1);
        // The operand of a gradient is there: the other issuer took a score from it in a turn before.
        for (int i = 0; ok && i + 1 < tiles.n; ++i) {
          const Desc gb = gd.at(g.stage * kTile), sb = sd.at(s.stage * kTile);
          const uint32_t acc = i > 0 ? 1u : 0u;
          // What comes last is awaited last: P behind the turn, the turn behind dS (4 x 4096 tokens, 32 over 8 heads: 1182 ->
          // 1168 us).
          ok = wait(&bs_full[s.stage], s.phase) &&
               (w ? wait(mine_full, mine) && take_turn() : take_turn() && wait(mine_full, mine));
          if (!ok) break;
          tc_fence_after();
          if (full && elect()) {
            mma_ts_n<4>(tg, ts, gb, id_g, acc);
            mma_ts_n<4>(tg, ts + 64, gb.at(4 * 2048), id_g, 1u);
            mma_ss_n<8>(ts, ad, sb, id_s);
            score_issued(i + 2 == tiles.n);
            commit1(&bg_empty[g.stage]);
          }
          if (!full && elect()) {
            mma_ts(tg, ts, gb, id_g, acc, min(4, steps));
            if (steps > 4) mma_ts(tg, ts + 64, gb.at(4 * 2048), id_g, 1u, steps - 4);
            mma_ss(ts, ad, sb, id_s, ksteps);
            score_issued(i + 2 == tiles.n);
            commit1(&bg_empty[g.stage]);
          }
          s.next(ns);
          g.next(ng);
          ++mine;
        }
        if (!ok) break;
        // The last tile, which may be a part of one.
        const Desc gb = gd.at(g.stage * kTile);
        const int lsteps = (left + 15) / 16;
        if (left < 16 * lsteps && left < a.tq * a.G) {  // rows past the sequence's end that the product's last step reads
          ok = wait(&bg_full[g.stage], g.phase);
          if (!ok) break;
          zero_rows(sG + g.stage * kTile, left, 16 * lsteps, halves);
          fence_async_smem();
          __syncwarp();
        }
        ok = wait(mine_full, mine) && take_turn();
        if (!ok) break;
        tc_fence_after();
        if (elect()) {
          mma_ts(tg, ts, gb, id_g, tiles.n > 1 ? 1u : 0u, min(4, lsteps));
          if (lsteps > 4) mma_ts(tg, ts + 64, gb.at(4 * 2048), id_g, 1u, lsteps - 4);
          mbar_arrive(&turn[1 - w]);
          commit1(acc_full);
          commit1(&bg_empty[g.stage]);
        }
        g.next(ng);
        ++mine;
        ++items;
      }
      if (elect()) {
        commit1(&drain[w]);  // every MMA issued here is complete once this flips
        drain_wait(&drain[w], 0);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------ lse and D of the tiles' rows
      bool ok = true;
      uint32_t g = 0;
      for (int it = 0; ok; ++it) {
        Item x;
        ok = __all_sync(0xffffffffu, next_item(it, x));
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[it % kItems]);
        if (x.head < 0) break;
        const Tiles tiles(x, a.tq, a.taken.parts);
        for (int i = 0; i < tiles.n && ok; ++i, ++g) {
          const int st = g % kStages, t0 = (tiles.first + i) * a.tq;
          float l[4], d[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = lane + 32 * u, tok = group_div(r, a.magic), place = t0 + tok;
            l[u] = -INFINITY;
            d[u] = 0.f;
            if (tok < a.tq && place < x.len) {
              const long long at = 1LL * (x.row0 + place) * a.Hq + x.head * a.G + (r - tok * a.G);
              l[u] = -a.lse[at] * kLog2e;
              d[u] = -a.D[at];
            }
          }
          ok = warp_wait(&st_empty[st], ((g / kStages) & 1) ^ 1u, abort_flag, a.err, DEV_ERR_TIMEOUT_PRODUCER);
          if (!ok) break;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            sL[st * kRows + lane + 32 * u] = l[u];
            sD[st * kRows + lane + 32 * u] = d[u];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&st_full[st]);
        }
      }
    }
  } else {
    regs_up<kRegsMany>();
    // ------------------------------------------------ element-wise warps and output
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;  // the key within the block
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + 64 * half, tp = ts + kRows, tv = ts + 2 * kRows;
    const float c = a.scale * kLog2e;
    uint32_t g = 0, items = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return warp_wait(bar, phase & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_EPILOGUE);
    };
    auto arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (int it = 0; ok; ++it) {
      Item x;
      ok = __all_sync(0xffffffffu, next_item(it, x));
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it % kItems]);
      if (x.head < 0) break;
      const Tiles tiles(x, a.tq, a.taken.parts);
      for (int i = 0; i < tiles.n; ++i, ++g) {
        const int st = g % kStages, t0 = (tiles.first + i) * a.tq;
        const int rows = min(a.tq, x.len - t0) * a.G - 64 * half;  // of the tile, from this thread's first
        const bool any = rows > 0;
        // The rows that see this key begin at G (key - t0); a tile before the block's last key, or past the end of the
        // sequence, is masked.
        const int from = (x.t0 + row - t0) * a.G - 64 * half;
        const bool masked = t0 < x.t0 + kRows - 1 || x.len - t0 < a.tq;
        const float* L = sL + st * kRows + 64 * half;
        const float* D = sD + st * kRows + 64 * half;
        ok = wait(&st_full[st], g / kStages) && wait(s_full, g);
        if (!ok) break;
        float p[64];
        if (any) {
          tc_fence_after();
          tmem_ld32(ts, p);
          tmem_ld32(ts + 32, p + 32);
          tmem_ld_wait();
          uint32_t w[32];
          if (masked) exps<true>(p, L, c, from, rows, w);
          else exps<false>(p, L, c, from, rows, w);
          tmem_st32u(ts, w);
          tmem_st_wait();
        }
        arrive(p_full);
        ok = wait(dp_full, g);
        if (!ok) break;
        if (any) {
          tc_fence_after();
          float d[64];
          tmem_ld32(tp, d);
          tmem_ld32(tp + 32, d + 32);
          tmem_ld_wait();
          uint32_t w[32];
          if (masked) grads<true>(p, d, D, from, rows, w);
          else grads<false>(p, d, D, from, rows, w);
          tmem_st32u(tp, w);
          tmem_st_wait();
        }
        arrive(ds_full);
        if (lane == 0) mbar_arrive(&st_empty[st]);
      }
      if (!ok) break;
      const int ncol = a.dh - 64 * half;
      const bool valid = row < x.len - x.t0;
      const long long key = x.row0 + x.t0 + row;
      if (tiles.n > 0) {
        ok = wait(acc_full, items++);
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // dV, dV, dK, dK
        const int h = k & 1;
        const float f = k < 2 ? 1.f : a.scale;
        float o[32];
        if (tiles.n > 0) {
          tmem_ld32(tv + (k >> 1) * kRows + 32 * h, o);
          tmem_ld_wait();
          if (k == 3) arrive(acc_free);
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = 0.f;
        }
        if (!valid) continue;
        const PackedRows& out = k < 2 ? a.dv : a.dk;
        bf16* to = out.p + key * out.ld + 1LL * x.head * a.dh + 64 * half + 32 * h;
        float* part = (k < 2 ? a.part_dv : a.part_dk) + ((1LL * tiles.part * a.T + key) * a.Hk + x.head) * a.dh + 64 * half + 32 * h;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (32 * h + 8 * u < ncol) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f * o[8 * u + e];
            if (a.taken.parts > 1) store8(part + 8 * u, v);
            else store8(to + 8 * u, v);
          }
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

}  // namespace dkv
}  // namespace packed
}  // namespace lr
