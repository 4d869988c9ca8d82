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
#include "step.cuh"

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
// Bound by the index keys' bytes: 8 sequences of 131073 tokens (8 groups of 128 elements, 2.15 GB) take 325 us,
// 6.6 TB/s. One warp takes 128 tokens of one group (32 KB at d_idx =
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

// Scores of 16 keys (rows gq and gq + 8 of `base`, at the lane's 16 bytes of every 64) against the queries
// in qv, maxima with what m0, m1 hold of columns 2 tq and 2 tq + 1.
template <int DI>
__device__ __forceinline__ void scan_tile(const __nv_bfloat16* base, int64_t row, int gq, const uint4 (&qv)[DI / 32], float& m0,
                                          float& m1) {
  constexpr int CH = DI / 32;
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
}
// The maxima of the block, over the keys that other lanes hold.
__device__ __forceinline__ void scan_block_max(float& m0, float& m1) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
}

template <int DI>
__global__ void __launch_bounds__(kScanThreads, 2) paged_scan_kernel(const __grid_constant__ PagedScanParams P) {
  constexpr int CH = DI / 32;
  __shared__ int ends[kScanMaxBatch];       // spans of sequences 0 .. b
  __shared__ int warp_sum[kScanThreads / 32];
  const PageView& V = P.view;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  grid_launch_dependents();
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
      scan_tile<DI>(base, row, gq, qv, m0, m1);
      if ((t + 1) % tiles_of_block == 0) {
        scan_block_max(m0, m1);
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
  grid_wait();   // nothing here depends on a prefix scan before it, but what follows does on both
}

// ------------------------------------------------------------------------------------
// Top-k of every (row, group): the local block and the k - 1 best earlier ones, equal scores
// the lower block first; ascending ids, padded with -1. One warp per (row, group). Latency-bound.
// ------------------------------------------------------------------------------------
struct PagedTopkParams {
  PageView view;
  const uint32_t* maxima;   // [rows][G][nbmax]
  int32_t* block_ids;       // [rows][G][k]
  unsigned int* arrived;    // [rows][G]: zeroed here for the attention
  __nv_bfloat16* o;         // [rows][G][width]: zeroed here where a row has no token
  int G, bk, k, nbmax, width;
};

// The k - 1 best of the keys src[0 .. n), n >= k - 1, of one warp: lane r < k - 1 returns the r-th
// best one's id, and in `place` its place among them in ascending order of ids. scratch: 96 entries of
// the warp's own in shared memory.
//
// 32 NK keys at a time (lane l: keys l, l + 32, ...), the best ones of earlier chunks carried along. The
// (k - 1)-th best of the lanes' maxima is a bound that at least k - 1 keys reach; the few keys that do
// are put side by side and each counts those before it: 3 us less than what follows, for k = 16 of 1024.
// Where more than 64 reach it (many equal scores), or few are wanted, the best one is taken out k - 1
// times instead, by a warp-wide max of the keys and a min of the ids among equals. The kernel's time, 32
// sequences of 8 groups: of 1000 blocks k = 16 takes 8.5 us by rank, 11.3 taken out one by one, k = 7 8.1 and
// 8.6, k = 4 8.1 and 8.1, k = 2 8.0 and 7.1; of 128 blocks and fewer, k = 8 7.8 and 8.1, k = 6 7.5 and 6.8.
template <int NK>
__device__ __forceinline__ int topk_warp_of(const uint32_t* src, int n, int k, int lane, uint2* scratch, int& place) {
  uint32_t carried = 0u, carried_id = 0xffffffffu;   // lane r: the r-th best so far (key 0: none)
  for (int c0 = 0; k > 1 && c0 < n; c0 += 32 * NK) {
    uint32_t key[NK];
    uint32_t best = carried;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int i = c0 + j * 32 + lane;
      key[j] = i < n ? src[i] : 0u;
      best = max(best, key[j]);
    }
    uint32_t next = 0u, next_id = 0xffffffffu;
    uint32_t bound = 0u;
    int count = 0, to = 0, total = 65;
    if (k > 6) {
      int before = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const uint32_t other = __shfl_sync(0xffffffffu, best, j);
        before += other > best || (other == best && j < lane);
      }
      bound = __shfl_sync(0xffffffffu, best, __ffs(__ballot_sync(0xffffffffu, before == k - 2)) - 1);
      count = carried >= bound && carried != 0u;
#pragma unroll
      for (int j = 0; j < NK; ++j) count += key[j] >= bound && key[j] != 0u;
      to = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += y;
      }
      total = __shfl_sync(0xffffffffu, to, 31);
    }
    if (total <= 64) {
      to -= count;
      if (carried >= bound && carried != 0u) scratch[to++] = make_uint2(carried, carried_id);
#pragma unroll
      for (int j = 0; j < NK; ++j)
        if (key[j] >= bound && key[j] != 0u) scratch[to++] = make_uint2(key[j], static_cast<uint32_t>(c0 + j * 32 + lane));
      __syncwarp();
      const uint2 a = lane < total ? scratch[lane] : make_uint2(0u, 0xffffffffu);
      const uint2 b = lane + 32 < total ? scratch[lane + 32] : make_uint2(0u, 0xffffffffu);
      int ra = 0, rb = 0;   // how many come before
      for (int j = 0; j < total; ++j) {
        const uint2 x = scratch[j];
        ra += x.x > a.x || (x.x == a.x && x.y < a.y);
        rb += x.x > b.x || (x.x == b.x && x.y < b.y);
      }
      if (lane < total && ra < k - 1) scratch[64 + ra] = a;
      if (lane + 32 < total && rb < k - 1) scratch[64 + rb] = b;
      __syncwarp();
      if (lane < k - 1 && lane < total) {
        next = scratch[64 + lane].x;
        next_id = scratch[64 + lane].y;
      }
      __syncwarp();   // the scratch is written again
    } else {
      for (int r = 0; r + 1 < k; ++r) {
        best = carried;
        int at = -1;
#pragma unroll
        for (int j = 0; j < NK; ++j)
          if (key[j] > best) { best = key[j]; at = j; }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0u) break;
        const uint32_t id = at < 0 ? carried_id : static_cast<uint32_t>(c0 + at * 32 + lane);
        const uint32_t win = __reduce_min_sync(0xffffffffu, best == top ? id : 0xffffffffu);
        if (best == top && id == win) {
          if (at < 0) carried = 0u;
#pragma unroll
          for (int j = 0; j < NK; ++j)
            if (j == at) key[j] = 0u;
        }
        if (lane == r) { next = top; next_id = win; }
      }
    }
    carried = next;
    carried_id = next_id;
  }
  // ascending: an id's place is the number of smaller ones (ids that were not found, behind a scan that
  // gave up, are -1 and take the last places)
  place = 0;
  for (int r = 0; r + 1 < k; ++r) {
    const uint32_t other = __shfl_sync(0xffffffffu, carried_id, r);
    place += other < carried_id || (other == carried_id && r < lane);
  }
  return static_cast<int>(carried_id);
}

// Up to 128 keys four a lane: of 100 blocks 7.1 us for k = 6 and 12.3 for k = 32, against 8.1 and 16.3 with 32 a
// lane; of 200 blocks, in chunks of 128, 8.6 against 8.1 (k = 6), of 1000 16 against 8.
__device__ __forceinline__ int topk_warp(const uint32_t* src, int n, int k, int lane, uint2* scratch, int& place) {
  return n <= 128 ? topk_warp_of<4>(src, n, k, lane, scratch, place) : topk_warp_of<32>(src, n, k, lane, scratch, place);
}

__global__ void __launch_bounds__(128) paged_topk_kernel(const __grid_constant__ PagedTopkParams P) {
  __shared__ uint2 scratch[4][96];
  const PageView& V = P.view;
  const int64_t rg = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (rg >= static_cast<int64_t>(V.batch) * V.S * P.G) return;
  const int64_t row = rg / P.G;
  const int b = static_cast<int>(row / V.S), s = static_cast<int>(row % V.S);
  int32_t* out = P.block_ids + rg * P.k;
  grid_launch_dependents();
  const int64_t pos = paged_length(V, b, kKidPagedTopk) - V.S + s;
  const int bl = pos >= 0 ? static_cast<int>(pos / P.bk) : -1;
  if (lane == 0) P.arrived[rg] = 0u;
  if (bl < 0)
    for (int e = lane; e < P.width / 8; e += 32) reinterpret_cast<uint4*>(P.o + rg * P.width)[e] = make_uint4(0, 0, 0, 0);
  if (bl + 1 <= P.k) {
    if (lane < P.k) out[lane] = lane <= bl ? lane : -1;
    grid_wait();
    return;
  }
  grid_wait();
  const uint32_t* src = P.maxima + rg * P.nbmax;
  int place;
  const int id = topk_warp(src, bl, P.k, lane, scratch[threadIdx.x >> 5], place);
  if (lane + 1 < P.k) out[place] = id;
  if (lane == 0) out[P.k - 1] = bl;
}

// ------------------------------------------------------------------------------------
// Sparse attention of every (row, group) over its selected blocks. Bound by the chosen blocks'
// bytes. The blocks' tokens are cut into strips of 16 (a strip lies in one page). All rows' strips
// stand in one list, and every CTA of a single resident wave takes an equal run of it, whatever
// the sequences' lengths; where a run ends inside a (row, group) its result is a part, and the
// last CTA to finish one of the parts joins them, in the list's order. (One CTA for every
// (row, group) leaves SMs idle: 8 sequences of 8 groups took 44 us, against 22 here. Clusters that
// share one wait for each other's places: 32 ragged sequences took 63 to 87 us, against 48. What is
// left above those bytes' 37 us is the chain of look-ups before the first copy, the join after the
// last, and pieces of 256 bytes every 2 KB.)
//
// A warp takes every fourth strip of the run through its own ring of asynchronous copies and carries
// its own running maximum, sum and output, so that warps meet only at the end of a (row, group).
// The products are m16n8k16, transposed so that the group's R <= 16 heads are the columns (too few
// for tcgen05's rows; one or two tiles of 8): S^T = K Q^T has the strip's tokens as rows, O^T += V^T P^T
// the output's elements. The probabilities go from the first one's accumulators into the second's
// operand through a transposition in registers (movmatrix), as two bf16 numbers each, the weight cut off and
// what that left (less than 2^-7 of it), rounded: off by at most 2^-15 + 2^-20 of each weight. Neither is negative
// or, of a positive weight, zero, so an infinite value gives an infinite output. (One number, off by 2^-8, put the outputs
// 2.1e-3 from the 64-bit ones where their own rounding is 1.7e-3; the second product costs the 16 x 4 drafted
// tokens behind 32K 3 us, 85 to 88, one short sequence 0.1 us, the other calls nothing.) Maximum, sum and
// output stay in fp32.
// ------------------------------------------------------------------------------------
struct PagedAttnParams {
  PageView view;
  const __nv_bfloat16* q;      // [batch][S][G * R][D]
  const __nv_bfloat16* kp;     // [num_pages][ps][G][D]
  const __nv_bfloat16* vp;
  int64_t k_stride, v_stride;
  const int32_t* block_ids;    // [rows][G][k]
  __nv_bfloat16* o;            // [batch][S][G * R][D]
  float* parts;                // [2 * CTAs][R][D + 2]: O, then m and l; part 2 c continues a unit, 2 c + 1 begins one
  unsigned int* arrived;       // [rows][G] parts written so far (zeroed by the Top-k)
  int G, R, k, bk_shift;       // blocks of 1 << bk_shift tokens
  float scale_log2;
};

constexpr int kPagedAttnWarps = 4;
constexpr int kPagedAttnTable = 256;   // strips looked up at a time
constexpr int kPagedAttnRing = 2;      // strips' values a warp has room for
constexpr int kPagedAttnLeast = 16;    // strips of a run, where there are enough: shorter ones cost more to join than they save
// CTAs resident on an SM. Three of 168 registers a thread; four of 128 spill (16 x 4 drafted tokens behind
// 32K: 93 us with three, 96 with four).
constexpr int kPagedAttnCtas(int nt) { return nt == 1 ? 3 : 2; }
template <int D>
struct PagedAttnCfg {
  static constexpr int kStrip = 16 * D;                      // elements of a strip's values
  static constexpr int kPitch = D + 4;                       // of a head's O in the join
  static constexpr int kEight = 8 * kPitch + 16;             // floats of 8 heads' O, m and l
  // shares of at most 18 parts (a unit has up to 256 strips, a run at least 16) of 16 heads
  static_assert(2 * kEight * 4 >= 18 * 16 * 8, "the shares fit the join's memory");
  static constexpr int kJoinOff = kPagedAttnWarps * kPagedAttnRing * kStrip * 2;
  static constexpr int kTableOff = kJoinOff + 2 * kEight * 4;
  static constexpr int kEndsOff = kTableOff + kPagedAttnTable * 16;
  static constexpr int smem_bytes(int batch) { return kEndsOff + batch * 4; }
};

__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], const void* row_addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row_addr))
               : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit elements held as a fragment (row lane / 4, columns 2 (lane % 4) ..).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Starts the copies of a strip's 16 rows of values (rows from `seen` on: zeros, whatever lies there) to
// shared address dst, 16-byte pieces c of row r at c ^ (r % 8), so that ldmatrix rows hit distinct banks.
template <int D>
__device__ __forceinline__ void fetch_values(uint32_t dst, const __nv_bfloat16* src, int64_t row, int seen, int lane) {
  constexpr int C = D / 8, STEP = 32 / C;   // pieces of a row, rows of a warp's access
  const int r0 = lane / C, c = lane % C;
  const __nv_bfloat16* s = src + r0 * row + c * 8;
  const uint32_t d = dst + r0 * D * 2, x = (c ^ r0) << 4;
#pragma unroll
  for (int i = 0; i < 16 / STEP; ++i) {   // r0 < STEP: (r0 + i STEP) % 8 is r0 | (i STEP) % 8
    const uint32_t to = d + i * STEP * D * 2 + (x ^ (((i * STEP) & 7) << 4));
    const int bytes = r0 + i * STEP < seen ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(s + i * STEP * row), "r"(bytes) : "memory");
  }
}

// S^T of a strip: keys kx, ky as they lie (rows gq and gq + 8), queries qf in the same order of elements;
// two sums whose chains are shorter.
template <int D, int NT>
__device__ __forceinline__ void strip_scores(const uint4 (&kx)[D / 32], const uint4 (&ky)[D / 32], const uint4 (&qf)[NT][D / 32],
                                             float (&sc)[NT][2][4]) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int y = 0; y < 4; ++y) sc[t][0][y] = sc[t][1][y] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mma_16816(sc[t][0], {kx[c].x, ky[c].x, kx[c].y, ky[c].y}, {qf[t][c].x, qf[t][c].y});
      mma_16816(sc[t][1], {kx[c].z, ky[c].z, kx[c].w, ky[c].w}, {qf[t][c].z, qf[t][c].w});
    }
}

// The strip's softmax against the running maximum and sum (m, l: heads 8 t + 2 tq and the next; the sum is
// of this lane's tokens), its weights P^T as operands: cut off to bf16 and, behind that, what is left;
// nv: tokens that count.
template <int D, int NT>
__device__ __forceinline__ void strip_softmax(const float (&sc)[NT][2][4], int nv, float scale_log2, int gq, float (&m)[NT][2],
                                              float (&l)[NT][2], float (&o)[NT][D / 16][4], uint32_t (&pf)[NT][4]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float x[4], top[2] = {m[t][0], m[t][1]};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      x[y] = gq + 8 * (y >> 1) < nv ? (sc[t][0][y] + sc[t][1][y]) * scale_log2 : -INFINITY;
      top[y & 1] = fmaxf(top[y & 1], x[y]);
    }
    float keep[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], off));
      const float from = top[h] == -INFINITY ? 0.0f : top[h];   // every score so far is -inf
      keep[h] = exp2f(m[t][h] - from);
      m[t][h] = top[h];
      top[h] = from;
      l[t][h] *= keep[h];
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      x[y] = exp2f(x[y] - top[y & 1]);
      l[t][y & 1] += x[y];
    }
    float rest[4];
#pragma unroll
    for (int y = 0; y < 4; ++y)   // a little more than the rest, so that no positive weight has a zero or negative one
      rest[y] = fmaf(x[y], 1.0f + 0x1p-20f, -__uint_as_float(__float_as_uint(x[y]) & 0xffff0000u));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      pf[t][h] = transpose_8x8(__byte_perm(__float_as_uint(x[2 * h]), __float_as_uint(x[2 * h + 1]), 0x7632));   // the upper halves
      pf[t][2 + h] = transpose_8x8(pack_bf16x2(rest[2 * h], rest[2 * h + 1]));
    }
    if (__any_sync(0xffffffffu, keep[0] != 1.0f || keep[1] != 1.0f)) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[t][n][y] *= keep[y & 1];
    }
  }
}

// O^T += V^T P^T, for both parts of P: the strip's values in shared memory, 16-byte pieces c of row r at c ^ (r % 8).
template <int D, int NT>
__device__ __forceinline__ void strip_values(const __nv_bfloat16* vs, int lane, const uint32_t (&pf)[NT][4], float (&o)[NT][D / 16][4]) {
  const int vr = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
  for (int n = 0; n < D / 16; ++n) {
    uint32_t af[4];
    ldsm_x4_trans(af, vs + vr * D + (((n * 2 + ((lane >> 3) & 1)) ^ (vr & 7)) * 8));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mma_16816(o[t][n], af, {pf[t][0], pf[t][1]});
      mma_16816(o[t][n], af, {pf[t][2], pf[t][3]});
    }
  }
}

// The four warps' results for eight heads into `join` (head h: O at h * pitch, maximum and sum behind the
// eight): warps 2 and 3 into 0 and 1, 1 into 0, that out. Ends with a barrier; two areas of 8 * pitch + 16.
template <int D>
__device__ __forceinline__ void join_warps(float (&o)[D / 16][4], float (&m)[2], float (&l)[2], float* join, int warp, int gq, int tq) {
  constexpr int kPitch = D + 4;   // the lanes' stores hit distinct banks
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
  auto put = [&](float* area) {
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int y = 0; y < 4; ++y) area[(2 * tq + (y & 1)) * kPitch + n * 16 + gq + 8 * (y >> 1)] = o[n][y];
    if (gq < 2) *reinterpret_cast<float2*>(area + 8 * kPitch + 2 * (2 * tq + gq)) = make_float2(gq ? m[1] : m[0], gq ? l[1] : l[0]);
  };
#pragma unroll
  for (int step = 2; step > 0; step >>= 1) {
    float* area = join + (step == 2 ? warp & 1 : 0) * (8 * kPitch + 16);
    if (warp >= step && warp < 2 * step) put(area);
    __syncthreads();
    if (warp < step) {
      float mine[2], theirs[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 ml = *reinterpret_cast<const float2*>(area + 8 * kPitch + 2 * (2 * tq + h));
        const float top = fmaxf(m[h], ml.x);
        mine[h] = m[h] == -INFINITY ? 0.0f : exp2f(m[h] - top);   // 0: a warp without a token
        theirs[h] = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
        m[h] = top;
        l[h] = l[h] * mine[h] + ml.y * theirs[h];
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int y = 0; y < 4; ++y)
          o[n][y] = o[n][y] * mine[y & 1] + area[(2 * tq + (y & 1)) * kPitch + n * 16 + gq + 8 * (y >> 1)] * theirs[y & 1];
    }
    __syncthreads();
  }
  if (warp == 0) put(join);
  __syncthreads();
}

// A place in the list of strips: strip `at` of the `n` strips of (sequence b, new token s, group g);
// `unit` is the first of them in the list. The list has fewer than 2^31 strips (4096 sequences of 8 new
// tokens, 64 groups, 256 strips), so 32 bits do: 64-bit divisions took microseconds here.
struct StripPlace {
  int b, s, g, n, at, unit, pos;
};

// Strips of one group of new token s of a sequence of length L; blocks of 1 << bk_shift tokens.
__device__ __forceinline__ int row_strips(int L, int S, int s, int k, int bk_shift) {
  const int pos = L - S + s;
  return pos < 0 ? 0 : min(k, (pos >> bk_shift) + 1) << (bk_shift - 4);
}

// ends[b]: strips of sequences 0 .. b, divided by G.
__device__ __forceinline__ StripPlace find_strip(const PagedAttnParams& P, const int* ends, int t) {
  const PageView& V = P.view;
  const int tg = static_cast<uint32_t>(t) / static_cast<uint32_t>(P.G);   // a sequence's strips are a multiple of G
  int lo = 0, hi = V.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > tg) hi = mid; else lo = mid + 1;
  }
  StripPlace x;
  x.b = lo;
  const int L = V.seqlens[lo];
  x.unit = lo > 0 ? ends[lo - 1] * P.G : 0;
  for (x.s = 0;; ++x.s) {
    x.n = row_strips(L, V.S, x.s, P.k, P.bk_shift);
    if (t < x.unit + x.n * P.G || x.s + 1 == V.S) break;
    x.unit += x.n * P.G;
  }
  x.g = static_cast<uint32_t>(t - x.unit) / static_cast<uint32_t>(x.n);
  x.unit += x.g * x.n;
  x.at = t - x.unit;
  x.pos = L - V.S + x.s;
  return x;
}

// NT: tiles of 8 heads.
template <int D, int NT>
__global__ void __launch_bounds__(kPagedAttnWarps * 32, kPagedAttnCtas(NT)) paged_attn_kernel(const __grid_constant__ PagedAttnParams P) {
  using C = PagedAttnCfg<D>;
  constexpr int kThreads = kPagedAttnWarps * 32;
  extern __shared__ __align__(16) uint8_t psm[];
  __shared__ int warp_sum[kPagedAttnWarps];
  __shared__ int is_last;
  const PageView& V = P.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  float* join = reinterpret_cast<float*>(psm + C::kJoinOff);
  longlong2* table = reinterpret_cast<longlong2*>(psm + C::kTableOff);   // first key element * 32 + tokens seen, first value element
  int* ends = reinterpret_cast<int*>(psm + C::kEndsOff);
  // running total of the sequences' strips
  int total = 0;
  for (int b0 = 0; b0 < V.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int x = 0;
    if (b < V.batch) {
      const int L = static_cast<int>(paged_length(V, b, kKidPagedAttn));
      for (int s = 0; L > 0 && s < V.S; ++s) x += row_strips(L, V.S, s, P.k, P.bk_shift);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = total;
    for (int w = 0; w < kPagedAttnWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    if (b < V.batch) ends[b] = before + x;
    __syncthreads();
  }
  const int strips = total * P.G;
  const int run = max(kPagedAttnLeast, static_cast<int>((strips + gridDim.x - 1u) / gridDim.x));
  grid_wait();   // so far only what the call was given has been read
  // (the last CTA's run may begin behind the list's end, by less than run * CTAs: no more than 2^31)
  const int begin = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * run, static_cast<int64_t>(strips)));
  const int end = min(strips, begin + min(run, strips));

  __nv_bfloat16* ring = reinterpret_cast<__nv_bfloat16*>(psm) + warp * kPagedAttnRing * C::kStrip;
  const int64_t row = static_cast<int64_t>(P.G) * D;
  // starts the copies of the values of entry i of the table
  auto fetch_v = [&](int i, int count, int stage) {
    if (i < count) {
      const longlong2 at = table[i];
      const int seen = static_cast<int>(at.x) & 31;
      if (seen > 0) fetch_values<D>(smem_u32(ring) + stage * C::kStrip * 2, P.vp + at.y, row, seen, lane);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the keys of entry i, as they lie: bytes 16 tq .. of every 64 of rows gq and gq + 8 (rows behind the
  // position hold anything; they are masked as scores)
  uint4 kx[D / 32], ky[D / 32];
  const __nv_bfloat16* k_lane = P.kp + gq * row + tq * 8;
  auto fetch_k = [&](int i, int count) {
    if (i < count) {
      const long long at = table[i].x;
      if ((at & 31) != 0) {
        const __nv_bfloat16* ks = k_lane + (at >> 5);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          kx[c] = __ldg(reinterpret_cast<const uint4*>(ks + c * 32));
          ky[c] = __ldg(reinterpret_cast<const uint4*>(ks + 8 * row + c * 32));
        }
      }
    }
  };

  uint4 qf[NT][D / 32];       // heads' queries, their elements in the keys' order
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];   // heads 8 t + 2 tq and the next
  bool begun = false;   // the unit's registers hold strips of an earlier table
  // Behind a shared prefix a run of one table takes the unit that it begins first, then the whole ones, then
  // the end of the one that another run began: so all CTAs go through low blocks first and high ones last,
  // and what rows select in common is still in L2 (64 sequences behind 128K tokens: 157 us, in the list's
  // order 164). Runs of several tables keep the list's order: batches of more than 111 rows with 8 groups and 16
  // blocks of 128 each, 55 with 32 blocks (a row's attention takes 1.12 us at 104 rows and 1.22 at 112).
  // place(i): where entry i of the table lies.
  const bool turned = V.prefix_pages > 0 && end - begin <= kPagedAttnTable;
  int head = begin, tail = begin;   // [begin, tail) ends a unit, [head, end) begins one
  if (turned && begin < end) {
    const StripPlace a = find_strip(P, ends, begin), z = find_strip(P, ends, end - 1);
    tail = a.at > 0 ? min(end, a.unit + a.n) : begin;
    head = max(tail, z.unit);
  }
  for (int sub = begin; sub < end; sub += kPagedAttnTable) {
    const int count = min(kPagedAttnTable, end - sub);
    auto place = [&](int i) {
      if (!turned) return sub + i;
      if (i < end - head) return head + i;
      i -= end - head;
      return i < head - tail ? tail + i : begin + i - (head - tail);
    };
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const StripPlace x = find_strip(P, ends, place(i));
      const int per_shift = P.bk_shift - 4;
      // (not __ldg: the Top-k may still have been writing them when this kernel began)
      const int blk = __ldcg(P.block_ids + ((static_cast<int64_t>(x.b) * V.S + x.s) * P.G + x.g) * P.k + (x.at >> per_shift));
      const int t0 = (blk << P.bk_shift) + ((x.at & ((1 << per_shift) - 1)) << 4);
      int page = -1;
      if (blk >= 0 && blk <= x.pos >> P.bk_shift && t0 <= x.pos) page = static_cast<int>(page_of(V, x.b, t0, kKidPagedAttn));
      const int seen = page >= 0 ? min(16, x.pos - t0 + 1) : 0;
      const int64_t in_page = (t0 & ((1 << V.shift) - 1)) * row + x.g * D;
      table[i] = make_longlong2((page * P.k_stride + in_page) * 32 + seen, page * P.v_stride + in_page);
    }
    __syncthreads();
    int i = warp, stage = 0;
#pragma unroll
    for (int st = 0; st < kPagedAttnRing - 1; ++st) fetch_v(warp + st * kPagedAttnWarps, count, st);
    fetch_k(warp, count);
    for (int cur = 0; cur < count;) {
      const int at = place(cur);
      const StripPlace x = find_strip(P, ends, at);
      const int stop = min(turned && cur < end - head ? end - head : count, cur + x.unit + x.n - at);
      const int64_t rg = (static_cast<int64_t>(x.b) * V.S + x.s) * P.G + x.g;
      const int64_t head0 = rg * P.R;
      if (!begun) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int r = t * 8 + gq;
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            qf[t][c] = r < P.R ? __ldg(reinterpret_cast<const uint4*>(P.q + (head0 + r) * D + c * 32 + tq * 8)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[t][n][y] = 0.0f;
          m[t][0] = m[t][1] = -INFINITY;
          l[t][0] = l[t][1] = 0.0f;
        }
      }
      for (; i < stop; i += kPagedAttnWarps) {
        __syncwarp();   // every lane is done with the stage that is refilled now
        fetch_v(i + (kPagedAttnRing - 1) * kPagedAttnWarps, count, stage == 0 ? kPagedAttnRing - 1 : stage - 1);
        const int nv = static_cast<int>(table[i].x) & 31;
        const __nv_bfloat16* vs = ring + stage * C::kStrip;
        stage = stage + 1 == kPagedAttnRing ? 0 : stage + 1;
        if (nv == 0) {
          fetch_k(i + kPagedAttnWarps, count);
          continue;
        }
        float sc[NT][2][4];
        strip_scores<D, NT>(kx, ky, qf, sc);
        fetch_k(i + kPagedAttnWarps, count);   // under this strip's softmax and values
        uint32_t pf[NT][4];
        strip_softmax<D, NT>(sc, nv, P.scale_log2, gq, m, l, o, pf);
        asm volatile("cp.async.wait_group %0;" ::"n"(kPagedAttnRing - 1) : "memory");
        __syncwarp();
        strip_values<D, NT>(vs, lane, pf, o);
      }
      cur = stop;
      begun = !turned && sub + cur < x.unit + x.n && sub + cur < end;   // the next table goes on with this unit
      if (begun) continue;

      // the warps' results, eight heads at a time
      const int first_cta = x.unit / run, last_cta = (x.unit + x.n - 1) / run;
      const bool whole = first_cta == last_cta;
      float* part = P.parts + (2 * static_cast<int64_t>(blockIdx.x) + (first_cta == blockIdx.x ? 1 : 0)) * P.R * (D + 2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        join_warps<D>(o[t], m[t], l[t], join, warp, gq, tq);
        for (int e = threadIdx.x; e < 8 * (D / 2); e += kThreads) {
          const int r8 = e / (D / 2), c = (e % (D / 2)) * 2, r = t * 8 + r8;
          if (r >= P.R) break;
          const float2 v = *reinterpret_cast<const float2*>(join + r8 * C::kPitch + c);
          const float2 ml = *reinterpret_cast<const float2*>(join + 8 * C::kPitch + 2 * r8);
          if (whole) {
            const float inv = ml.y > 0.0f ? 1.0f / ml.y : 0.0f;   // nothing but bad pages: zero
            *reinterpret_cast<uint32_t*>(P.o + (head0 + r) * D + c) = pack_bf16x2(v.x * inv, v.y * inv);
          } else {
            *reinterpret_cast<float2*>(part + r * D + c) = v;
            if (c == 0) *reinterpret_cast<float2*>(part + P.R * D + 2 * r) = ml;
          }
        }
        __syncthreads();   // the area is written again
      }
      if (whole) continue;
      // the last of the unit's CTAs to get here joins the parts
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) is_last = atomicAdd(P.arrived + rg, 1u) == static_cast<unsigned int>(last_cta - first_cta);
      __syncthreads();
      if (is_last) {
        __threadfence();
        // every part's share of each head: 2^(its maximum - the common one), over the common sum
        const int n_parts = last_cta - first_cta + 1;
        auto part_of = [&](int w) { return P.parts + (2 * static_cast<int64_t>(first_cta + w) + (w == 0 ? 1 : 0)) * P.R * (D + 2); };
        float2* share = reinterpret_cast<float2*>(join);   // [parts][R], then .x the share
        for (int e = threadIdx.x; e < n_parts * P.R; e += kThreads) {
          const int w = e / P.R;
          share[e] = __ldcg(reinterpret_cast<const float2*>(part_of(w) + P.R * D) + e - w * P.R);
        }
        __syncthreads();
        if (threadIdx.x < P.R) {
          float top = -INFINITY, sum = 0.0f;
          for (int w = 0; w < n_parts; ++w) top = fmaxf(top, share[w * P.R + threadIdx.x].x);
          for (int w = 0; w < n_parts; ++w) {
            float2& ml = share[w * P.R + threadIdx.x];
            ml.x = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
            sum += ml.x * ml.y;
          }
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
          for (int w = 0; w < n_parts; ++w) share[w * P.R + threadIdx.x].x *= inv;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < P.R * (D / 4); e += kThreads) {
          const int r = e / (D / 4), c = (e % (D / 4)) * 4;
          float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int w0 = 0; w0 < n_parts; w0 += 4) {   // four parts' loads in flight
            float2 lo[4], hi[4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (w0 + w < n_parts) {
                const float* from = part_of(w0 + w) + r * D + c;
                lo[w] = __ldcg(reinterpret_cast<const float2*>(from));
                hi[w] = __ldcg(reinterpret_cast<const float2*>(from + 2));
              }
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (w0 + w < n_parts) {
                const float f = share[(w0 + w) * P.R + r].x;
                a[0] += f * lo[w].x;
                a[1] += f * lo[w].y;
                a[2] += f * hi[w].x;
                a[3] += f * hi[w].y;
              }
          }
          *reinterpret_cast<uint2*>(P.o + (head0 + r) * D + c) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
        }
      }
      __syncthreads();   // is_last is written again by the next unit
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // the table is written again
  }
}

}  // namespace msa
