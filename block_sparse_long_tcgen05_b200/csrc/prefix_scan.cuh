// Decode behind a shared prefix: block maxima of every row of the batch against the whole blocks
// of the prefix, its index keys read once for all rows.
//
// Per group a matrix product, rows x keys with K = d_idx, whose result is reduced where it falls:
// rows are the M = 128 of a tcgen05 product (up to two tiles of them against one key tile), keys
// its N = 128, and an epilogue thread owns a row, takes the maximum over each block's columns
// from TMEM and stores its ordered key. Nothing else leaves the SM.
//
// Bound by the keys' bytes up to about 128 rows (64 rows x 131072 tokens x 8 groups: 268 MB, 41 us
// at the copy rate, and 17 us of products at M = 128; takes 54), by the products beyond. A CTA stays with one
// (row tiles, group) and takes every W-th key tile, so that CTAs of all groups stream the same
// tokens' rows side by side.
#pragma once
#include "index_blockmax.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace msa {

struct PrefixScanParams {
  const int32_t* prefix;   // pages
  uint32_t* maxima;        // [rows][G][nbmax]
  int64_t num_pages;
  int n_pages, shift;      // page size 1 << shift
  int rows, G, bk, nbmax;
  int blocks;              // whole blocks of the prefix
  int tiles;               // of 128 tokens
  int pairs;               // (row tiles, group)
  int workers;             // CTAs of one pair
};

// RT: row tiles of 128 against one key tile (1 or 2).
template <int DI, int RT>
struct PrefixCfg {
  using I = IdxCfg<DI>;
  static constexpr int kStages = RT == 1 ? 5 : 4;
  static constexpr int kBuffers = RT == 1 ? 4 : 2;   // TMEM accumulators of RT * 128 columns
  static constexpr int kKOff = RT * I::kTileBytes;
  static constexpr int kBarOff = kKOff + kStages * I::kTileBytes;
  static constexpr int kSmemBytes = kBarOff + 256 + 1024;
};

constexpr int kPrefixThreads = 320;   // producer, issuer, two epilogue warpgroups

template <int DI, int RT>
// Few enough registers that a block of the sequences' own scan runs beside this one.
__global__ void __launch_bounds__(kPrefixThreads, 2)
prefix_scan_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ PrefixScanParams P) {
  using C = PrefixCfg<DI, RT>;
  using I = IdxCfg<DI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;                   // [stages]
  uint64_t* k_empty = k_full + C::kStages;       // [stages]
  uint64_t* acc_full = k_empty + C::kStages;     // [buffers]
  uint64_t* acc_empty = acc_full + C::kBuffers;  // [buffers]
  uint64_t* mma_done = acc_empty + C::kBuffers;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  WaitCtl* ctl = reinterpret_cast<WaitCtl*>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::kStages; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    // with one row tile the two epilogue warpgroups take alternate key tiles, else a row tile each
    for (int i = 0; i < C::kBuffers; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], RT == 1 ? 4 : 8); }
    mbar_init(mma_done, 1);
    wait_ctl_init(ctl);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // pairs p0, p0 + stride, ...; of each the key tiles t0, t0 + workers, ...
  const int p0 = P.workers > 1 ? static_cast<int>(blockIdx.x) % P.pairs : static_cast<int>(blockIdx.x);
  const int stride = P.workers > 1 ? P.pairs : static_cast<int>(gridDim.x);
  const int t0 = P.workers > 1 ? static_cast<int>(blockIdx.x) / P.pairs : 0;

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    const int boxes = P.shift < 7 ? 128 >> P.shift : 1;   // pages of a tile; lane l copies page l
    auto page_for = [&](int t) -> int {
      const int64_t token = static_cast<int64_t>(t) * 128 + (static_cast<int64_t>(lane) << P.shift);
      const int64_t at = token >> P.shift;
      int page = -1;
      if (lane < boxes && t < P.tiles && at < P.n_pages) {
        page = P.prefix[at];
        if (page < 0 || page >= P.num_pages) {
          record_error(MSA_ERR_DEVICE_BOUNDS, kKidPrefixScan);
          page = -1;
        }
      }
      // no page: a coordinate behind the last one, which the copy fills with zeros
      return page < 0 ? static_cast<int>(P.num_pages) : page;
    };
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
    }
    int64_t ik = 0;
    int items = 0;   // query tiles loaded
    bool ok = true;
    for (int pr = p0; pr < P.pairs && ok; pr += stride) {
      const int g = pr % P.G, rg = pr / P.G;
      if (lane == 0) {
        ok = mbar_wait(q_empty, (items & 1) ^ 1, ctl, kKidPrefixScan);
        if (ok) {
          mbar_arrive_expect_tx(q_full, RT * I::kTileBytes);
          for (int rt = 0; rt < RT; ++rt)
            for (int pnl = 0; pnl < I::kPanels; ++pnl)
              tma_load_3d(smem + rt * I::kTileBytes + pnl * I::kPanelBytes, &tm_q, q_full, pnl * I::kPanelElems, g,
                          (rg * RT + rt) * 128);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++items;
      int page = page_for(t0);
      for (int t = t0; t < P.tiles; t += P.workers, ++ik) {
        const int st = static_cast<int>(ik % C::kStages);
        const uint32_t u = static_cast<uint32_t>(ik / C::kStages);
        const int next = page_for(t + P.workers);   // its latency lies under the wait
        if (lane == 0) {
          ok = mbar_wait(&k_empty[st], (u & 1) ^ 1, ctl, kKidPrefixScan);
          if (ok) mbar_arrive_expect_tx(&k_full[st], I::kTileBytes);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        __syncwarp();
        if (!ok) break;
        if (lane < boxes) {
          uint8_t* ks = smem + C::kKOff + st * I::kTileBytes + ((lane * I::kRowBytes) << P.shift) * (boxes > 1);
          const int row = boxes > 1 ? 0 : (t * 128) & ((1 << P.shift) - 1);
          for (int pnl = 0; pnl < I::kPanels; ++pnl)
            tma_load_4d(ks + pnl * I::kPanelBytes, &tm_k, &k_full[st], pnl * I::kPanelElems, g, row, page);
        }
        page = next;
      }
    }
    if (lane == 0) {
      // drain: every copy that was started lands before the CTA ends
      for (int s = 0; s < C::kStages; ++s)
        if (ik > s) {
          const int64_t last = ((ik - 1 - s) / C::kStages) * C::kStages + s;
          mbar_wait(&k_full[s], static_cast<uint32_t>(last / C::kStages) & 1, nullptr, kKidPrefixScan);
        }
      if (items > 0) mbar_wait(q_full, (items - 1) & 1, nullptr, kKidPrefixScan);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------ MMA issuer ------------------------------
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false);
      int64_t ik = 0;
      int items = 0;
      bool ok = true;
      for (int pr = p0; pr < P.pairs && ok; pr += stride, ++items) {
        if (!mbar_wait(q_full, items & 1, ctl, kKidPrefixScan)) { ok = false; break; }
        tc_fence_after();
        for (int t = t0; t < P.tiles; t += P.workers, ++ik) {
          const int st = static_cast<int>(ik % C::kStages);
          const int ab = static_cast<int>(ik % C::kBuffers);
          if (!mbar_wait(&k_full[st], static_cast<uint32_t>(ik / C::kStages) & 1, ctl, kKidPrefixScan)) { ok = false; break; }
          if (!mbar_wait(&acc_empty[ab], (static_cast<uint32_t>(ik / C::kBuffers) & 1) ^ 1, ctl, kKidPrefixScan)) { ok = false; break; }
          tc_fence_after();
          const uint32_t k_addr = smem_u32(smem + C::kKOff + st * I::kTileBytes);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const uint32_t q_addr = smem_u32(smem + rt * I::kTileBytes);
            const uint32_t d = tmem + (ab * RT + rt) * 128;
#pragma unroll
            for (int kk = 0; kk < I::kKSteps; ++kk) {
              const uint32_t koff = (kk * 32) / I::kRowBytes * I::kPanelBytes + (kk * 32) % I::kRowBytes;
              umma_bf16(d, smem_desc(q_addr + koff, 16, I::kSbo, I::kLayout), smem_desc(k_addr + koff, 16, I::kSbo, I::kLayout),
                        idesc, kk > 0);
            }
          }
          umma_commit(&k_empty[st]);
          umma_commit(&acc_full[ab]);
        }
        umma_commit(q_empty);
      }
      umma_commit(mma_done);
      mbar_wait(mma_done, 0, nullptr, kKidPrefixScan);
    }
    __syncwarp();
  } else {
    // ------------------------------ epilogue ------------------------------
    const int group = (warp - 2) >> 2;
    const int quad = warp & 3;   // TMEM lanes this warp may read
    const int F = 128 / P.bk;
    int64_t ik = 0;
    bool ok = true;
    for (int pr = p0; pr < P.pairs && ok; pr += stride) {
      const int g = pr % P.G, rg = pr / P.G;
      const int row = (rg * RT + (RT == 1 ? 0 : group)) * 128 + quad * 32 + lane;
      uint32_t* out = P.maxima + (static_cast<int64_t>(row) * P.G + g) * P.nbmax;
      for (int t = t0; t < P.tiles; t += P.workers, ++ik) {
        if (RT == 1 && static_cast<int>(ik & 1) != group) continue;
        const int ab = static_cast<int>(ik % C::kBuffers);
        if (!mbar_wait(&acc_full[ab], static_cast<uint32_t>(ik / C::kBuffers) & 1, ctl, kKidPrefixScan)) { ok = false; break; }
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (ab * RT + (RT == 1 ? 0 : group)) * 128;
        float m = -INFINITY;
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // 64 columns at a time
          uint32_t r[2][32];
          tmem_ld32(taddr + half * 64, r[0]);
          tmem_ld32(taddr + half * 64 + 32, r[1]);
          tmem_ld_wait();
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[ab]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) m = max3f(m, __uint_as_float(r[c][j]), __uint_as_float(r[c][j + 1]));
            const int done = (half * 2 + c + 1) * 32;
            if (done % P.bk == 0) {
              const int blk = t * F + done / P.bk - 1;
              if (row < P.rows && blk < P.blocks) out[blk] = ordered_key(m);
              m = -INFINITY;
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace msa
