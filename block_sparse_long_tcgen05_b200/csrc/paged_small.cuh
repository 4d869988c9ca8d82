// Decode over a paged cache in one launch, for few and short sequences: scan, Top-k and attention
// of one (row, group) by a cluster of eight CTAs.
//
// Such a call is bound by latency: three launches and what each looks up again (lengths, pages)
// are most of it. Here a cluster's warps share out the blocks to scan and store every maximum into
// all eight CTAs' shared memory; each CTA selects for itself (the same keys, the same ids); the
// warps share out the strips of the selected blocks, and the results meet over distributed shared
// memory. One sequence of 700 tokens (2 groups): 7.8 us against 13.8 in three kernels.
#pragma once
#include "paged.cuh"

namespace msa {

constexpr int kSmallCluster = 8;
constexpr int kSmallBlocks = 256;    // of the longest sequence
constexpr int kSmallThreads = kPagedAttnWarps * 32;

struct PagedSmallParams {
  PageView view;
  const __nv_bfloat16* q_idx;   // [rows][G][DI]
  const __nv_bfloat16* ip;      // [num_pages][ps][G][DI]
  const __nv_bfloat16* q;       // [rows][G * R][D]
  const __nv_bfloat16* kp;
  const __nv_bfloat16* vp;
  int64_t i_stride, k_stride, v_stride;
  int32_t* block_ids;           // [rows][G][k]
  __nv_bfloat16* o;             // [rows][G * R][D]
  int G, R, k, bk_shift;
  float scale_log2;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrival and wait of the cluster's barrier, by all its threads; memory before the one is visible after
// the other.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int D, int NT, int DI>
__global__ void __cluster_dims__(kSmallCluster, 1, 1) __launch_bounds__(kSmallThreads, NT == 1 ? 3 : 2)
paged_small_kernel(const __grid_constant__ PagedSmallParams P) {
  constexpr int kPitch = D + 4;
  constexpr int kEight = 8 * kPitch + 16;
  constexpr int kStrip = 16 * D;
  __shared__ uint32_t maxima[kSmallBlocks];
  __shared__ int ids[32];
  __shared__ uint2 scratch[96];
  __shared__ __align__(16) float join[2 * kEight];
  __shared__ __align__(16) float mine[NT * kEight];   // this CTA's part of the result
  extern __shared__ __align__(16) uint8_t psm[];      // values: two strips a warp
  const PageView& V = P.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int rank = static_cast<int>(cluster_rank());
  const int rg = static_cast<int>(blockIdx.x) / kSmallCluster;
  const int row = rg / P.G, g = rg - row * P.G;
  const int b = row / V.S, s = row - b * V.S;
  const int worker = rank * kPagedAttnWarps + warp;
  constexpr int kWorkers = kSmallCluster * kPagedAttnWarps;
  cluster_arrive();   // every CTA runs before any stores into another's memory
  const int pos = static_cast<int>(paged_length(V, b, kKidPagedSmall)) - V.S + s;
  const int64_t head0 = static_cast<int64_t>(rg) * P.R;
  if (pos < 0) {   // a row without a token, for the whole cluster
    if (rank == 0) {
      for (int e = threadIdx.x; e < P.R * D / 8; e += kSmallThreads) reinterpret_cast<uint4*>(P.o + head0 * D)[e] = make_uint4(0, 0, 0, 0);
      if (threadIdx.x < P.k) P.block_ids[static_cast<int64_t>(rg) * P.k + threadIdx.x] = -1;
    }
    __syncthreads();
    cluster_wait();
    return;
  }
  const int bl = pos >> P.bk_shift;
  // the queries, on their way while blocks are scored
  uint4 qf[NT][D / 32];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = t * 8 + gq;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      qf[t][c] = r < P.R ? __ldg(reinterpret_cast<const uint4*>(P.q + (head0 + r) * D + c * 32 + tq * 8)) : make_uint4(0, 0, 0, 0);
  }
  const int mask = (1 << V.shift) - 1;
  if (bl + 1 > P.k && P.k > 1) {
    uint4 qv[DI / 32];   // the one query as column 0
#pragma unroll
    for (int c = 0; c < DI / 32; ++c)
      qv[c] = gq == 0 ? __ldg(reinterpret_cast<const uint4*>(P.q_idx + static_cast<int64_t>(rg) * DI + c * 32 + tq * 8))
                      : make_uint4(0, 0, 0, 0);
    const int tiles = 1 << (P.bk_shift - 4);
    const int64_t irow = static_cast<int64_t>(P.G) * DI;
    cluster_wait();
    for (int blk = worker; blk < bl; blk += kWorkers) {
      int64_t page = 0;   // lane t: of the block's tile t
      if (lane < tiles) page = page_of(V, b, (static_cast<int64_t>(blk) << P.bk_shift) + lane * 16, kKidPagedSmall);
      if (page < 0) page = 0;   // recorded; scored from the first page, and never read out of range
      float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 2
      for (int t = 0; t < tiles; ++t) {
        const int64_t pg = __shfl_sync(0xffffffffu, page, t);
        scan_tile<DI>(P.ip + pg * P.i_stride + (((blk << P.bk_shift) + t * 16) & mask) * irow + g * DI + tq * 8, irow, gq, qv, m0, m1);
      }
      scan_block_max(m0, m1);
      const uint32_t key = __shfl_sync(0xffffffffu, ordered_key(m0), 0);
      if (lane < kSmallCluster) st_cluster_u32(cluster_map(smem_u32(maxima + blk), lane), key);
    }
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      int place;
      const int id = topk_warp(maxima, bl, P.k, lane, scratch, place);
      if (lane + 1 < P.k) ids[place] = id;
      if (lane == 0) ids[P.k - 1] = bl;
    }
  } else {
    if (warp == 0) ids[lane] = bl + 1 > P.k ? bl : lane <= bl ? lane : -1;   // k = 1, or every visible block
    cluster_wait();
  }
  __syncthreads();
  if (rank == 0 && threadIdx.x < P.k) P.block_ids[static_cast<int64_t>(rg) * P.k + threadIdx.x] = ids[threadIdx.x];

  // ---- attention: strip i of the row by warp i % 32 of the cluster
  const int per_shift = P.bk_shift - 4;
  const int strips = min(P.k, bl + 1) << per_shift;
  const int64_t krow = static_cast<int64_t>(P.G) * D;
  __nv_bfloat16* ring = reinterpret_cast<__nv_bfloat16*>(psm) + warp * 2 * kStrip;
  struct Place {
    int64_t page;
    int row, seen;
  };
  auto place_of = [&](int i) {
    Place x{-1, 0, 0};
    if (i < strips) {
      const int blk = ids[i >> per_shift];
      const int t0 = (blk << P.bk_shift) + ((i & ((1 << per_shift) - 1)) << 4);
      if (blk >= 0 && t0 <= pos) x.page = page_of(V, b, t0, kKidPagedSmall);
      x.row = t0 & mask;
      x.seen = x.page >= 0 ? min(16, pos - t0 + 1) : 0;
    }
    return x;
  };
  uint4 kx[D / 32], ky[D / 32];
  auto fetch_k = [&](const Place& x) {
    if (x.seen > 0) {
      const __nv_bfloat16* ks = P.kp + x.page * P.k_stride + (x.row + gq) * krow + g * D + tq * 8;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        kx[c] = __ldg(reinterpret_cast<const uint4*>(ks + c * 32));
        ky[c] = __ldg(reinterpret_cast<const uint4*>(ks + 8 * krow + c * 32));
      }
    }
  };
  auto fetch_v = [&](const Place& x, int stage) {
    if (x.seen > 0)
      fetch_values<D>(smem_u32(ring) + stage * kStrip * 2, P.vp + x.page * P.v_stride + x.row * krow + g * D, krow, x.seen, lane);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[t][n][y] = 0.0f;
  }
  Place cur = place_of(worker);
  fetch_k(cur);
  fetch_v(cur, 0);
  int stage = 0;
  for (int i = worker; i < strips; i += kWorkers) {
    const Place next = place_of(i + kWorkers);
    __syncwarp();   // every lane is done with the stage that is refilled now
    fetch_v(next, stage ^ 1);
    if (cur.seen > 0) {
      float sc[NT][2][4];
      strip_scores<D, NT>(kx, ky, qf, sc);
      fetch_k(next);
      uint32_t pf[NT][4];
      strip_softmax<D, NT>(sc, cur.seen, P.scale_log2, gq, m, l, o, pf);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      strip_values<D, NT>(ring + stage * kStrip, lane, pf, o);
    } else {
      fetch_k(next);
    }
    cur = next;
    stage ^= 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    join_warps<D>(o[t], m[t], l[t], join, warp, gq, tq);
    for (int e = threadIdx.x; e < kEight / 4; e += kSmallThreads)
      reinterpret_cast<float4*>(mine + t * kEight)[e] = reinterpret_cast<const float4*>(join)[e];
    __syncthreads();   // the area is written again
  }
  cluster_arrive();
  cluster_wait();
  // the CTAs' parts, each CTA a share of the row's elements
  for (int e = rank * kSmallThreads + threadIdx.x; e < P.R * (D / 2); e += kSmallCluster * kSmallThreads) {
    const int r = e / (D / 2), c = (e % (D / 2)) * 2;
    const uint32_t at = smem_u32(mine + (r >> 3) * kEight);
    float2 ml[kSmallCluster], v[kSmallCluster];
    float top = -INFINITY, sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < kSmallCluster; ++w) {
      const uint32_t from = cluster_map(at, w);
      ml[w] = ld_cluster_f2(from + (8 * kPitch + 2 * (r & 7)) * 4);
      v[w] = ld_cluster_f2(from + ((r & 7) * kPitch + c) * 4);
      top = fmaxf(top, ml[w].x);
    }
#pragma unroll
    for (int w = 0; w < kSmallCluster; ++w) {
      const float f = ml[w].x == -INFINITY ? 0.0f : exp2f(ml[w].x - top);
      sum += f * ml[w].y;
      x += f * v[w].x;
      y += f * v[w].y;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;   // nothing but bad pages: zero
    *reinterpret_cast<uint32_t*>(P.o + (head0 + r) * D + c) = pack_bf16x2(x * inv, y * inv);
  }
  cluster_arrive();   // no CTA ends while another reads its memory
  cluster_wait();
}

}  // namespace msa
