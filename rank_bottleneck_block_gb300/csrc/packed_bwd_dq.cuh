// dQ of causal attention over packed sequences (tcgen05).
//
// An item is one row tile (128 rows: tokens with the G heads of a key head, see packed_device.cuh) against the keys up
// to its last token, 128 at a time.  Per key block j:
//
//   S = Q K_j^T, dP = dO V_j^T          MMA, fp32 in TMEM (S in two buffers, one block ahead)
//   P = 2^(c S - lse log2 e)            element-wise warps, two threads a row, P in registers
//   dS = P (dP - D)                     written back as bf16 over the columns that S was read from
//   dQ += dS K_j                        MMA with A = dS from TMEM; the result takes the scale at the end
//
// S and dP are computed again here and not kept by the kernel of dK and dV: a kept dS takes two bytes for each pair of
// tokens and head (34 GB for one sequence of 16384 and 64 heads), and summing dQ in memory from its key blocks would
// make the sum's order depend on which finishes first.  7 products run instead of 5.
//
// Two issuers: one for S and dQ, one for dP, which follows as soon as the dP before has been read into registers.  The
// exponentials of a block need its S alone, so they run while dQ of the block before and its dP are computed.
//
// Keys past a row's token get P = dS = 0 by selection; rows of K past the end of the sequence are zeroed in shared
// memory before the product that multiplies them by those zeroes.
//
// Warps: 0 takes the items and loads them by TMA (Q, dO per item; K_j into three 32 KB stages, V_j into two), 1 issuer of
// S and dQ, which also allocates TMEM, 2 issuer of dP, 3 idle, 4-11 element-wise and output (warp group h takes keys
// 64 h .. 64 h + 63 of a block and columns 64 h .. of dQ).  TMEM: S at columns 0 and 128, dP at 256, dQ at 384.  Every
// wait is bounded (error word, abort flag; each role drains what it issued, and TMEM is freed).
#pragma once

#include "packed_device.cuh"

namespace lr {
namespace packed {
namespace dq {

constexpr int kStagesK = 3, kStagesV = 2;
constexpr int kSmem = (2 + kStagesK + kStagesV) * kTile + 512;
static_assert(kSmem <= umma::kMaxSmem, "shared memory");

// One of `nblocks` blocks, the `block`-th.
__device__ __forceinline__ void body(const BwdMaps& maps, const DqArgs& a, unsigned block, unsigned nblocks,
                                     uint8_t* smem) {
  uint8_t* sQ = smem;
  uint8_t* sdO = sQ + kTile;
  uint8_t* sK = sdO + kTile;          // [kStagesK]
  uint8_t* sV = sK + kStagesK * kTile;  // [kStagesV]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + kStagesV * kTile);
  uint64_t* qd_full = bars;
  uint64_t* qd_free = bars + 1;   // the item's last S and last dP have read Q and dO
  uint64_t* k_full = bars + 2;    // [kStagesK]
  uint64_t* k_empty = bars + 5;   // [kStagesK]
  uint64_t* v_full = bars + 8;    // [kStagesV]
  uint64_t* v_empty = bars + 10;  // [kStagesV]
  uint64_t* s_full = bars + 12;   // [2]
  uint64_t* dp_full = bars + 14;
  uint64_t* dp_free = bars + 15;  // dP is in registers
  uint64_t* ds_full = bars + 16;  // [2], as S: the element-wise warps can be a block ahead of the product
  uint64_t* dq_last = bars + 20;  // the item's last product is complete
  uint64_t* dq_free = bars + 18;  // dQ has been read
  uint64_t* drain = bars + 21;    // [2]
  uint64_t* item_full = bars + 24;            // [kItems]
  uint64_t* item_empty = item_full + kItems;  // [kItems]
  int4* sitem = reinterpret_cast<int4*>(item_empty + kItems);  // [kItems], 16-byte aligned
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sitem + kItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kReaders = 2 + 8;  // issuers, element-wise warps

  if (threadIdx.x == 0) {
    mbar_init(qd_full, 1);
    mbar_init(qd_free, 2);
    for (int i = 0; i < kStagesK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&ds_full[i], 8);
      mbar_init(&drain[i], 1);
    }
    mbar_init(dp_full, 1);
    mbar_init(dp_free, 8);
    mbar_init(dq_last, 1);
    mbar_init(dq_free, 8);
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
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------ scheduler and producer
      bool ok = true;
      int g = 0, q_issued = 0;  // key blocks, and items
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
        const Item x{v.x, v.y, v.z, v.w};
        const int n = x.nblocks(0, a.tq), row = x.row0 + x.t0;
        ok = wait(qd_free, q_issued);
        if (!ok) break;
        mbar_expect_tx(qd_full, 2 * halves * a.G * a.tq * 128);
        load(sQ, &maps.q, qd_full, x.head * a.G, row);
        load(sdO, &maps.dout, qd_full, x.head * a.G, row);
        ++q_issued;
        for (int j = 0; j < n && ok; ++j, ++g) {
          if (j == max(0, n - 2)) t = nblocks + atomicAdd(a.taken.next, 1u);  // late: see the forward
          const int sk = g % kStagesK, sv = g % kStagesV;
          ok = wait(&k_empty[sk], g / kStagesK);
          if (!ok) break;
          mbar_expect_tx(&k_full[sk], halves * kHalf);
          load(sK + sk * kTile, &maps.k, &k_full[sk], x.head, x.row0 + j * kRows);
          ok = wait(&v_empty[sv], g / kStagesV);
          if (!ok) {
            drain_wait(&k_full[sk], (g / kStagesK) & 1);
            break;
          }
          mbar_expect_tx(&v_full[sv], halves * kHalf);
          load(sV + sv * kTile, &maps.v, &v_full[sv], x.head, x.row0 + j * kRows);
        }
      }
      if (!ok) {  // the copies in flight end before the block does
        for (int k = max(0, g - kStagesK); k < g; ++k) drain_wait(&k_full[k % kStagesK], (k / kStagesK) & 1);
        for (int k = max(0, g - kStagesV); k < g; ++k) drain_wait(&v_full[k % kStagesV], (k / kStagesV) & 1);
        if (q_issued) drain_wait(qd_full, (q_issued - 1) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ issuer of S and dQ
      const uint32_t id_s = idesc_n<false>(kRows);  // S = Q K^T: both K-major
      const uint32_t id_g = idesc_n<true>(dh16);    // dQ += dS K: dS from TMEM, K MN-major
      const uint32_t tm = uniform(tmem);
      const Desc qd = sdesc(smem_addr(sQ), 16, 1024), kd = sdesc(smem_addr(sK), 16, 1024),
                 gd = sdesc(smem_addr(sK), kHalf, 1024);
      bool ok = true;
      uint32_t g = 0, items = 0;
      Ring s, k;  // K of the next S, and of the next dQ
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return warp_wait(bar, phase & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA);
      };
      for (int it = 0; ok; ++it, ++items) {
        Item x;
        ok = __all_sync(0xffffffffu, next_item(it, x));
        if (!ok) break;
        x = Item{uniform(x.row0), uniform(x.len), uniform(x.t0), uniform(x.head)};
        if (elect()) mbar_arrive(&item_empty[it % kItems]);
        if (x.head < 0) break;
        const int n = x.nblocks(0, a.tq), last = x.keys(0, a.tq) - (n - 1) * kRows;
        auto issue_s = [&](int j) {  // S of the item's block j
          const uint32_t b = g + j;
          if (!wait(&k_full[s.stage], s.phase)) return false;
          tc_fence_after();
          if (elect()) {
            const Desc kb = kd.at(s.stage * kTile);
            if (ksteps == 8) mma_ss_n<8>(tm + (b & 1) * kRows, qd, kb, id_s);
            else mma_ss(tm + (b & 1) * kRows, qd, kb, id_s, ksteps);
            commit1(&s_full[b & 1]);
            if (j + 1 == n) commit1(qd_free);
          }
          s.next(kStagesK);
          return true;
        };
        ok = wait(qd_full, items) && issue_s(0) && (n == 1 || issue_s(1));
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t b = g + j, st = k.stage;
          const int steps = j + 1 < n ? 8 : (last + 15) / 16, left = x.len - j * kRows;
          ok = (j > 0 || wait(dq_free, items + 1)) && wait(&ds_full[b & 1], b >> 1);
          if (!ok) break;
          if (left < 16 * steps) {  // rows past the sequence's end that the product's last step reads
            zero_rows(sK + st * kTile, left, 16 * steps, halves);
            fence_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (elect()) {
            const uint32_t ds = tm + (b & 1) * kRows;
            const Desc gb = gd.at(st * kTile);
            if (steps == 8) {
              mma_ts_n<4>(tm + 3 * kRows, ds, gb, id_g, j > 0 ? 1u : 0u);
              mma_ts_n<4>(tm + 3 * kRows, ds + 64, gb.at(4 * 2048), id_g, 1u);
            } else {
              mma_ts(tm + 3 * kRows, ds, gb, id_g, j > 0 ? 1u : 0u, min(4, steps));
              if (steps > 4) mma_ts(tm + 3 * kRows, ds + 64, gb.at(4 * 2048), id_g, 1u, steps - 4);
            }
            commit1(&k_empty[st]);
            if (j + 1 == n) commit1(dq_last);
          }
          k.next(kStagesK);
          if (j + 2 < n) ok = issue_s(j + 2);
        }
        g += n;
      }
      if (elect()) {
        commit1(&drain[0]);  // every MMA issued here is complete once this flips
        drain_wait(&drain[0], 0);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------ issuer of dP
      const uint32_t id_s = idesc_n<false>(kRows);
      const uint32_t tm = uniform(tmem);
      const Desc od = sdesc(smem_addr(sdO), 16, 1024), vd = sdesc(smem_addr(sV), 16, 1024);
      bool ok = true;
      uint32_t g = 0, items = 0;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return warp_wait(bar, phase & 1, abort_flag, a.err, DEV_ERR_TIMEOUT_MMA);
      };
      for (int it = 0; ok; ++it, ++items) {
        Item x;
        ok = __all_sync(0xffffffffu, next_item(it, x));
        if (!ok) break;
        x = Item{uniform(x.row0), uniform(x.len), uniform(x.t0), uniform(x.head)};
        if (elect()) mbar_arrive(&item_empty[it % kItems]);
        if (x.head < 0) break;
        const int n = x.nblocks(0, a.tq);
        ok = wait(qd_full, items);
        for (int j = 0; j < n && ok; ++j, ++g) {
          const uint32_t st = g % kStagesV;
          ok = wait(&v_full[st], g / kStagesV) && wait(dp_free, g + 1);
          if (!ok) break;
          tc_fence_after();
          if (elect()) {
            const Desc vb = vd.at(st * kTile);
            if (ksteps == 8) mma_ss_n<8>(tm + 2 * kRows, od, vb, id_s);
            else mma_ss(tm + 2 * kRows, od, vb, id_s, ksteps);
            commit1(dp_full);
            commit1(&v_empty[st]);
            if (j + 1 == n) commit1(qd_free);
          }
        }
      }
      if (elect()) {
        commit1(&drain[1]);
        drain_wait(&drain[1], 0);
      }
      __syncwarp();
    }
  } else {
    regs_up<kRegsMany>();
    // ------------------------------------------------ element-wise warps and output
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + 64 * half, tp = ts + 2 * kRows, tg = ts + 3 * kRows;
    const float c = a.scale * kLog2e;
    const int tok = group_div(row, a.magic);
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
    for (int it = 0; ok; ++it, ++items) {
      Item x;
      ok = __all_sync(0xffffffffu, next_item(it, x));
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it % kItems]);
      if (x.head < 0) break;
      const int n = x.nblocks(0, a.tq), keys = x.keys(0, a.tq), place = x.t0 + tok;
      const bool valid = tok < a.tq && place < x.len;
      float nl = 0.f, D = 0.f;
      if (valid) {
        const long long at = 1LL * (x.row0 + place) * a.Hq + x.head * a.G + (row - tok * a.G);
        nl = -a.lse[at] * kLog2e;
        D = a.D[at];
      }
      for (int j = 0; j < n; ++j, ++g) {
        const int from = j * kRows + 64 * half;   // this thread's first key
        const bool any = keys > from;             // some row of the tile sees one of the 64
        const bool masked = x.t0 < from + 63;     // some row does not see all of them
        const int lim = place - from;
        ok = wait(&s_full[g & 1], g >> 1);
        if (!ok) break;
        float p[64];
        if (any) {
          tc_fence_after();
          const uint32_t s = ts + (g & 1) * kRows;
          tmem_ld32(s, p);
          tmem_ld32(s + 32, p + 32);
          tmem_ld_wait();
          const uint64_t c2 = f2_pack(c, c), n2 = f2_pack(nl, nl);
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float e0, e1;
            f2_unpack(f2_fma(f2_pack(p[i], p[i + 1]), c2, n2), e0, e1);
            p[i] = ex2_ftz(e0);
            p[i + 1] = ex2_ftz(e1);
          }
        }
        ok = wait(dp_full, g);
        if (!ok) break;
        if (any) {
          tc_fence_after();
          float d[64];
          tmem_ld32(tp, d);
          tmem_ld32(tp + 32, d + 32);
          tmem_ld_wait();
          arrive(dp_free);
          const uint64_t nd = f2_pack(-D, -D);
          uint32_t w[32];
          if (masked) {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float d0 = i > lim ? 0.f : p[i] * (d[i] - D), d1 = i + 1 > lim ? 0.f : p[i + 1] * (d[i + 1] - D);
              w[i >> 1] = pack_bf16x2(d0, d1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              float d0, d1;
              f2_unpack(f2_mul(f2_pack(p[i], p[i + 1]), f2_add(f2_pack(d[i], d[i + 1]), nd)), d0, d1);
              w[i >> 1] = pack_bf16x2(d0, d1);
            }
          }
          tmem_st32u(ts + (g & 1) * kRows, w);
          tmem_st_wait();
        } else {
          arrive(dp_free);
        }
        arrive(&ds_full[g & 1]);
      }
      if (!ok) break;
      ok = wait(dq_last, items);
      if (!ok) break;
      tc_fence_after();
      // Straight from registers, 16 bytes at a time: shared memory is full, and an item has this once.
      bf16* out = a.dq.p + (x.row0 + place) * a.dq.ld + 1LL * (x.head * a.G + (row - tok * a.G)) * a.dh + 64 * half;
      const int ncol = a.dh - 64 * half;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float o[32];
        tmem_ld32(tg + 32 * h, o);
        tmem_ld_wait();
        if (h == 1) arrive(dq_free);
        if (!valid) continue;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (32 * h + 8 * u < ncol) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = a.scale * o[8 * u + e];
            store8(out + 32 * h + 8 * u, w);
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

}  // namespace dq
}  // namespace packed
}  // namespace lr
