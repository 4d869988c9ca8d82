// Decode over a paged cache: the Index Branch's scan, its Top-k and the sparse attention of the
// 1 to 8 newest tokens of every sequence, all reading keys and values through a page table.
//
// A sequence's token t lies in row t % ps of page table[t / ps]; a page holds ps tokens of all
// groups, [ps][G][dim]. Row (b, s) is new token s of sequence b, at position
// seqlens[b] - S + s; a row without a token (an empty or too short sequence) selects nothing
// and its output is zero.
#pragma once
#include <cuda_bf16.h>

#include "decode.cuh"
#include "ptx.cuh"

namespace msa {

struct PageView {
  const int32_t* table;      // [batch][table_stride]
  const int32_t* prefix;     // pages of the first prefix_pages * ps tokens of every sequence
  const int32_t* seqlens;
  int64_t table_stride;
  int64_t num_pages;
  int prefix_pages, max_pages, shift;   // ps = 1 << shift, 16 <= ps <= 1024
  int batch, S;
};

// Page that holds token t of sequence b (in range, or -1 after recording the error).
__device__ __forceinline__ int64_t page_of(const PageView& V, int b, int64_t t, int kernel_id) {
  const int p = static_cast<int>(t >> V.shift);
  const int64_t page = p < V.prefix_pages ? V.prefix[p] : V.table[b * V.table_stride + p];
  if (page >= 0 && page < V.num_pages) return page;
  record_error(MSA_ERR_DEVICE_BOUNDS, kernel_id);
  return -1;
}

// Length of sequence b; 0 where it is none (recorded as an error unless it is 0).
__device__ __forceinline__ int64_t paged_length(const PageView& V, int b, int kernel_id) {
  const int64_t L = V.seqlens[b];
  if (L >= 0 && L <= (static_cast<int64_t>(V.max_pages) << V.shift)) return L;
  record_error(MSA_ERR_DEVICE_BOUNDS, kernel_id);
  return 0;
}

__device__ __forceinline__ uint32_t ordered_key(float m) {
  const uint32_t u = __float_as_uint(__fadd_rn(m, 0.0f));   // -0 -> +0: equal scores, equal keys
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ------------------------------------------------------------------------------------
// Index Branch scan: block maxima of every row against the blocks before its sequence's last
// token's block, from block nb0 on. Nothing is scanned of a sequence all of whose visible
// blocks are selected anyway.
//
// Bound by the index keys' bytes. One warp takes 128 tokens of one group (32 KB at d_idx =
// 128). The keys go from memory into the registers of an m16n8k16 product as they lie: lane
// (gq, tq) loads the 16 bytes 8 tq .. 8 tq + 7 of every 32 elements of rows gq and gq + 8,
// which serve as two steps' operands, since a dot product does not mind the order of its terms
// as long as the queries' operand has the same one. The product's eight columns are the new
// tokens, so up to eight of them cost the keys' bytes once.
// ------------------------------------------------------------------------------------
struct PagedScanParams {
  PageView view;
  const __nv_bfloat16* q_idx;   // [batch][S][G][DI]
  const __nv_bfloat16* pages;   // [num_pages][ps][G][DI]
  int64_t page_stride;
  uint32_t* maxima;             // [batch * S][G][nbmax]
  int G, bk, k, nbmax, nb0;
};

constexpr int kScanMaxBatch = 4096;
constexpr int kScanThreads = 256;

template <int DI>
__global__ void __launch_bounds__(kScanThreads, 2) paged_scan_kernel(const __grid_constant__ PagedScanParams P) {
  constexpr int CH = DI / 32;
  __shared__ int ends[kScanMaxBatch];       // spans of sequences 0 .. b
  __shared__ int warp_sum[kScanThreads / 32];
  const PageView& V = P.view;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  // running total of every sequence's spans of 128 tokens
  int total = 0;
  for (int b0 = 0; b0 < V.batch; b0 += kScanThreads) {
    const int b = b0 + threadIdx.x;
    int spans = 0;
    if (b < V.batch) {
      const int64_t L = paged_length(V, b, kKidPagedScan);
      const int last = L > 0 ? static_cast<int>((L - 1) / P.bk) : 0;   // block of the last token
      if (last + 1 > P.k && last > P.nb0) spans = ((last - P.nb0) * P.bk + 127) >> 7;
    }
    int x = spans;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = total;
    for (int w = 0; w < kScanThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    if (b < V.batch) ends[b] = before + x;
    __syncthreads();
  }
  const int64_t units = static_cast<int64_t>(total) * P.G;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kScanThreads / 32) + warp; u < units;
       u += static_cast<int64_t>(gridDim.x) * (kScanThreads / 32)) {
    const int span = static_cast<int>(u / P.G), g = static_cast<int>(u - static_cast<int64_t>(span) * P.G);
    int lo = 0, hi = V.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > span) hi = mid; else lo = mid + 1;
    }
    const int b = lo;
    const int local = span - (b > 0 ? ends[b - 1] : 0);
    const int last = static_cast<int>((static_cast<int64_t>(V.seqlens[b]) - 1) / P.bk);
    const int64_t token0 = static_cast<int64_t>(P.nb0) * P.bk + static_cast<int64_t>(local) * 128;
    const int tiles = static_cast<int>(min(static_cast<int64_t>(128), static_cast<int64_t>(last) * P.bk - token0)) >> 4;
    // a span starts a page or lies inside one: lane l holds the span's page l
    int64_t my_page = 0;
    if ((lane << V.shift) < tiles * 16) my_page = page_of(V, b, token0 + (static_cast<int64_t>(lane) << V.shift), kKidPagedScan);
    if (my_page < 0) my_page = 0;   // recorded; scored from the first page, and never read out of range
    uint4 qv[CH];
    const int s = gq;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      qv[c] = s < V.S ? __ldg(reinterpret_cast<const uint4*>(
                            P.q_idx + ((static_cast<int64_t>(b) * V.S + s) * P.G + g) * DI + c * 32 + tq * 8))
                      : make_uint4(0, 0, 0, 0);
    float m0 = -INFINITY, m1 = -INFINITY;   // columns 2 tq and 2 tq + 1
    const int tiles_of_block = P.bk >> 4;
    const int mask = (1 << V.shift) - 1;
    const int64_t row = static_cast<int64_t>(P.G) * DI;
#pragma unroll 2
    for (int t = 0; t < tiles; ++t) {
      const int64_t page = __shfl_sync(0xffffffffu, my_page, (t << 4) >> V.shift);
      const __nv_bfloat16* base = P.pages + page * P.page_stride + ((token0 + t * 16) & mask) * row + g * DI + tq * 8;
      uint4 x[CH], y[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        x[c] = __ldg(reinterpret_cast<const uint4*>(base + gq * row + c * 32));
        y[c] = __ldg(reinterpret_cast<const uint4*>(base + (gq + 8) * row + c * 32));
      }
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        mma_16816(acc, {x[c].x, y[c].x, x[c].y, y[c].y}, {qv[c].x, qv[c].y});
        mma_16816(acc, {x[c].z, y[c].z, x[c].w, y[c].w}, {qv[c].z, qv[c].w});
      }
      m0 = max3f(m0, acc[0], acc[2]);
      m1 = max3f(m1, acc[1], acc[3]);
      if ((t + 1) % tiles_of_block == 0) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        const int blk = static_cast<int>((token0 + t * 16) / P.bk);
        if (gq == 0) {
          uint32_t* out = P.maxima + ((static_cast<int64_t>(b) * V.S + 2 * tq) * P.G + g) * P.nbmax + blk;
          if (2 * tq < V.S) out[0] = ordered_key(m0);
          if (2 * tq + 1 < V.S) out[static_cast<int64_t>(P.G) * P.nbmax] = ordered_key(m1);
        }
        m0 = m1 = -INFINITY;
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// Top-k of every (row, group): the local block and the k - 1 best earlier ones, equal scores
// the lower block first; ascending ids, padded with -1. One warp per (row, group), 1024 keys at
// a time in its registers (lane l: keys l, l + 32, ...); k - 1 times the best one is found by a
// warp-wide max of the keys and a min of the ids among equals, and taken out. The chosen ones of
// earlier chunks are carried as one more candidate a lane. Latency-bound.
// ------------------------------------------------------------------------------------
struct PagedTopkParams {
  PageView view;
  const uint32_t* maxima;   // [rows][G][nbmax]
  int32_t* block_ids;       // [rows][G][k]
  int G, bk, k, nbmax;
};

__global__ void __launch_bounds__(128) paged_topk_kernel(const __grid_constant__ PagedTopkParams P) {
  const PageView& V = P.view;
  const int64_t rg = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (rg >= static_cast<int64_t>(V.batch) * V.S * P.G) return;
  const int64_t row = rg / P.G;
  const int b = static_cast<int>(row / V.S), s = static_cast<int>(row % V.S);
  int32_t* out = P.block_ids + rg * P.k;
  const int64_t pos = paged_length(V, b, kKidPagedTopk) - V.S + s;
  const int bl = pos >= 0 ? static_cast<int>(pos / P.bk) : -1;
  if (bl + 1 <= P.k) {
    if (lane < P.k) out[lane] = lane <= bl ? lane : -1;
    return;
  }
  const uint32_t* src = P.maxima + rg * P.nbmax;
  uint32_t carried = 0u, carried_id = 0xffffffffu;   // lane r: the r-th best so far (key 0: none)
  for (int c0 = 0; P.k > 1 && c0 < bl; c0 += 1024) {
    uint32_t key[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) key[j] = c0 + j * 32 + lane < bl ? __ldg(src + c0 + j * 32 + lane) : 0u;
    uint32_t next = 0u, next_id = 0xffffffffu;
    uint32_t best = 0u;
    int at = -1;
    for (int r = 0; r + 1 < P.k; ++r) {
      best = carried;
      at = -1;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (key[j] > best) { best = key[j]; at = j; }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      if (top == 0u) break;
      const uint32_t id = at < 0 ? carried_id : static_cast<uint32_t>(c0 + at * 32 + lane);
      const uint32_t win = __reduce_min_sync(0xffffffffu, best == top ? id : 0xffffffffu);
      if (best == top && id == win) {
        if (at < 0) carried = 0u;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == at) key[j] = 0u;
      }
      if (lane == r) { next = top; next_id = win; }
    }
    carried = next;
    carried_id = next_id;
  }
  // ascending: an id's place is the number of smaller ones
  int place = 0;
  for (int r = 0; r + 1 < P.k; ++r) place += __shfl_sync(0xffffffffu, carried_id, r) < carried_id;
  if (lane + 1 < P.k) out[place] = static_cast<int32_t>(carried_id);
  if (lane == 0) out[P.k - 1] = bl;
}

// ------------------------------------------------------------------------------------
// Sparse attention of every (row, group) over its selected blocks. Bound by the chosen blocks'
// bytes. The block's tokens are cut into strips of 16 (a strip lies in one page); every warp
// takes every fourth strip through its own ring of asynchronous copies, and carries its own
// running maximum, sum and output, so that warps meet only once, at the end. S = Q K^T and
// O += P V are m16n8k16 products with the group's R <= 16 heads as rows (too few for tcgen05);
// a strip's probabilities go from the first product's accumulators straight into the second's
// operand, rounded to bf16 (off by at most 2^-8 of each weight, what the output is rounded to as well);
// maximum, sum and output stay in fp32.
// ------------------------------------------------------------------------------------
struct PagedAttnParams {
  PageView view;
  const __nv_bfloat16* q;      // [batch][S][G * R][D]
  const __nv_bfloat16* kp;     // [num_pages][ps][G][D]
  const __nv_bfloat16* vp;
  int64_t k_stride, v_stride;
  const int32_t* block_ids;    // [rows][G][k]
  __nv_bfloat16* o;            // [batch][S][G * R][D]
  int G, R, k, bk;
  float scale_log2;
};

constexpr int kPagedAttnWarps = 4;
constexpr int kPagedAttnRing = 3;
template <int D>
struct PagedAttnCfg {
  static constexpr int kPitch = D + 8;                       // padded: ldmatrix rows hit distinct banks
  static constexpr int kStrip = 2 * 16 * kPitch;             // elements of a strip's K and V
  static constexpr int kRingBytes = kPagedAttnWarps * kPagedAttnRing * kStrip * 2;
  static constexpr int kOutBytes = kPagedAttnWarps * (16 * D + 32) * 4;   // O, m, l of every warp (over the ring)
  static constexpr int kSmemBytes = kRingBytes > kOutBytes ? kRingBytes : kOutBytes;
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], const void* row_addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row_addr))
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], const void* row_addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row_addr))
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPagedAttnWarps * 32) paged_attn_kernel(const __grid_constant__ PagedAttnParams P) {
  using C = PagedAttnCfg<D>;
  extern __shared__ __align__(16) uint8_t psm[];
  const PageView& V = P.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int64_t rg = blockIdx.x;
  const int64_t row = rg / P.G;
  const int g = static_cast<int>(rg - row * P.G);
  const int b = static_cast<int>(row / V.S), s = static_cast<int>(row % V.S);
  const int64_t pos = paged_length(V, b, kKidPagedAttn) - V.S + s;
  const int32_t* ids = P.block_ids + rg * P.k;
  const int64_t head0 = (row * P.G + g) * P.R;

  // the warp's strips: strip i of the row is strip i % per_block of slot i / per_block
  const int per_block = P.bk >> 4;
  int slots = 0;
  if (pos >= 0) {
    const int bl = static_cast<int>(pos / P.bk);
    slots = min(P.k, bl + 1);
  }
  const int strips = slots * per_block;

  uint32_t qf[D / 16][4];
  {
    const __nv_bfloat16* q0 = P.q + head0 * D;
    auto pair = [&](int r, int col) -> uint32_t {
      return r < P.R ? *reinterpret_cast<const uint32_t*>(q0 + r * D + col) : 0u;
    };
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qf[kk][0] = pair(gq, kk * 16 + 2 * tq);
      qf[kk][1] = pair(gq + 8, kk * 16 + 2 * tq);
      qf[kk][2] = pair(gq, kk * 16 + 8 + 2 * tq);
      qf[kk][3] = pair(gq + 8, kk * 16 + 8 + 2 * tq);
    }
  }
  __nv_bfloat16* ring = reinterpret_cast<__nv_bfloat16*>(psm) + warp * kPagedAttnRing * C::kStrip;
  // starts the copies of strip i and returns how many of its tokens the row sees
  auto fetch = [&](int i, int stage) -> int {
    int seen = 0;
    if (i < strips) {
      const int blk = __ldg(ids + i / per_block);
      const int64_t t0 = static_cast<int64_t>(blk) * P.bk + (i % per_block) * 16;
      const bool in_order = blk >= 0 && t0 <= pos;   // else: behind the row's position, or no block
      int64_t page = -1;
      if (in_order) page = page_of(V, b, t0, kKidPagedAttn);
      seen = page >= 0 ? static_cast<int>(min(static_cast<int64_t>(16), pos - t0 + 1)) : 0;
      if (seen > 0) {
        const int64_t off = (t0 & ((1 << V.shift) - 1)) * P.G * D + g * D;
        const __nv_bfloat16* ks = P.kp + page * P.k_stride + off;
        const __nv_bfloat16* vs = P.vp + page * P.v_stride + off;
        __nv_bfloat16* kd = ring + stage * C::kStrip;
        __nv_bfloat16* vd = kd + 16 * C::kPitch;
#pragma unroll
        for (int e = lane; e < 16 * (D / 8); e += 32) {
          const int r = e / (D / 8), c = (e % (D / 8)) * 8;
          const bool ok = r < seen;   // rows behind the position read as zeros, whatever lies there
          const int64_t so = ok ? static_cast<int64_t>(r) * P.G * D + c : 0;
          cp_async16(kd + r * C::kPitch + c, ks + so, ok);
          cp_async16(vd + r * C::kPitch + c, vs + so, ok);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return seen;
  };

  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[n][x] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};   // rows gq and gq + 8
  int seen[kPagedAttnRing];
#pragma unroll
  for (int st = 0; st < kPagedAttnRing - 1; ++st) seen[st] = fetch(warp + st * kPagedAttnWarps, st);
  int i = warp;
  while (i < strips) {
#pragma unroll
    for (int st = 0; st < kPagedAttnRing; ++st) {   // unrolled over the ring: stage numbers are constants
      if (i >= strips) break;
      __syncwarp();   // every lane is done with the stage that is refilled now
      seen[(st + kPagedAttnRing - 1) % kPagedAttnRing] =
          fetch(i + (kPagedAttnRing - 1) * kPagedAttnWarps, (st + kPagedAttnRing - 1) % kPagedAttnRing);
      asm volatile("cp.async.wait_group %0;" ::"n"(kPagedAttnRing - 1) : "memory");
      __syncwarp();
      const int nv = seen[st];
      if (nv > 0) {
        const __nv_bfloat16* ks = ring + st * C::kStrip;
        const __nv_bfloat16* vs = ks + 16 * C::kPitch;
        float sc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[n][x] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t bf[4];
          ldsm_x4(bf, ks + ((lane & 7) + ((lane >> 4) << 3)) * C::kPitch + kk * 16 + ((lane >> 3) & 1) * 8);
          mma_16816(sc[0], qf[kk], {bf[0], bf[1]});
          mma_16816(sc[1], qf[kk], {bf[2], bf[3]});
        }
        float top[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int t = n * 8 + 2 * tq + (x & 1);
            sc[n][x] = t < nv ? sc[n][x] * P.scale_log2 : -INFINITY;
            top[x >> 1] = fmaxf(top[x >> 1], sc[n][x]);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          const float from = top[h] == -INFINITY ? 0.0f : top[h];   // every score so far is -inf
          const float keep = exp2f(m[h] - from);
          m[h] = top[h];
          top[h] = from;
          l[h] *= keep;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * h] *= keep;
            o[n][2 * h + 1] *= keep;
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            sc[n][x] = exp2f(sc[n][x] - top[x >> 1]);
            l[x >> 1] += sc[n][x];
          }
        const uint32_t pf[4] = {pack_bf16x2(sc[0][0], sc[0][1]), pack_bf16x2(sc[0][2], sc[0][3]),
                                pack_bf16x2(sc[1][0], sc[1][1]), pack_bf16x2(sc[1][2], sc[1][3])};
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t bf[4];
          ldsm_x4_trans(bf, vs + (lane & 15) * C::kPitch + n * 16 + (lane >> 4) * 8);
          mma_16816(o[2 * n], pf, {bf[0], bf[1]});
          mma_16816(o[2 * n + 1], pf, {bf[2], bf[3]});
        }
      }
      i += kPagedAttnWarps;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  __syncthreads();   // the ring's memory now takes every warp's O, m and l
  float* mine = reinterpret_cast<float*>(psm) + warp * (16 * D + 32);
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    *reinterpret_cast<float2*>(mine + gq * D + n * 8 + 2 * tq) = make_float2(o[n][0], o[n][1]);
    *reinterpret_cast<float2*>(mine + (gq + 8) * D + n * 8 + 2 * tq) = make_float2(o[n][2], o[n][3]);
  }
  if (tq == 0) {
    mine[16 * D + gq] = m[0];
    mine[16 * D + gq + 8] = m[1];
    mine[16 * D + 16 + gq] = l[0];
    mine[16 * D + 24 + gq] = l[1];
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(psm);
  for (int e = threadIdx.x; e < P.R * D / 2; e += blockDim.x) {
    const int r = e / (D / 2), c = (e % (D / 2)) * 2;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kPagedAttnWarps; ++w) top = fmaxf(top, all[w * (16 * D + 32) + 16 * D + r]);
    float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < kPagedAttnWarps; ++w) {
      const float* from = all + w * (16 * D + 32);
      const float mw = from[16 * D + r];
      const float f = mw == -INFINITY ? 0.0f : exp2f(mw - top);   // a warp without a token
      sum += f * from[16 * D + 16 + r];
      x += f * from[r * D + c];
      y += f * from[r * D + c + 1];
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;   // a row without a token: zero
    *reinterpret_cast<uint32_t*>(P.o + (head0 + r) * D + c) = pack_bf16x2(x * inv, y * inv);
  }
}

}  // namespace msa
