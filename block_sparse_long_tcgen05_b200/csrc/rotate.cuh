// Rotary positions, and the append of new tokens to the paged cache with the rotation on the
// way: one kernel, whose jobs are the tensors of a call.
//
// A head's first `rot` elements are pairs (x_a, x_b), element f and f + rot / 2 (halves) or
// 2f and 2f + 1 (interleaved). Pair f of a token at position p turns by p * freqs[f]:
//   y_a = s (c x_a - n x_b),  y_b = s (n x_a + c x_b),  c, n = cos, sin(p freqs[f]),
// the rest of the head is copied. The gradient is the transposed map: n changes its sign.
//
// Angles: fp32 cannot hold p * f at positions of long contexts (2^20 * 2^-24 is 1/16 rad), so
// the frequency is taken as a 64-bit fixed-point fraction of a turn and multiplied with the
// position modulo 2^64: whole turns drop out exactly. The turns a position, f / (2 pi) in fp64, are
// off by at most |f| 2^-55 (half a step of the product, and of 1 / (2 pi), which are 2^-53 and 2^-53.9
// of it), where f is negative by 2^-54 more (the step up from below 0), and the fixed point by 2^-65: the
// angle by |p| times that, 2^-55 turns a position for the usual f <= 1. Its upper 32 bits go to sincospif:
// cutting the others off is 2^-31 half turns at most, rounding what is left to fp32 2^-25.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "step.cuh"

namespace msa {

constexpr int kRotThreads = 256;
constexpr int kRotMaxJobs = 5;
constexpr int kRotGroup = 4;   // heads a thread has in flight

struct RotateJob {
  const void* src;
  void* dst;
  int64_t src_token, src_head;   // strides in elements
  int64_t dst_token, dst_head;   // within a page when paged
  int64_t dst_page;              // elements between pages
  const double* freqs;           // NULL: copied
  int heads, dim, rot;
  int head_slots;                // threads of a token's unit: each takes heads hs, hs + head_slots, ...
  unsigned int block0;           // first block of the job
  int paged;
};

struct RotateParams {
  RotateJob jobs[kRotMaxJobs];
  int count;
  int interleaved;
  float scale, sign;             // sign -1: the transposed rotation
  int64_t n;                     // tokens (rows of the tensors)
  // positions: given (rope) ...
  const void* positions;
  int positions_i64;
  // ... or of new tokens that end their sequences (append)
  const int32_t* cu_seqlens;     // [batch + 1]; NULL: `each` tokens a sequence
  int each;
  const int32_t* seqlens;
  const int32_t* page_table;
  int64_t table_stride;
  int64_t num_pages;
  int batch, max_pages, page_shift;
};

__device__ __forceinline__ float rot_in(float x) { return x; }
__device__ __forceinline__ float rot_in(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float rot_in(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T rot_out(float x);
template <>
__device__ __forceinline__ float rot_out<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rot_out<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half rot_out<__half>(float x) { return __float2half_rn(x); }

// V consecutive elements, moved as one access of V * sizeof(T) bytes (aligned to it).
template <typename T, int V>
struct alignas(sizeof(T) * V) RotVec {
  T e[V];
};

// cos and sin of 2 pi p * turns, turns given as radians per position.
__device__ __forceinline__ void rot_angle(double radians, uint64_t pos, float& c, float& n) {
  double t = radians * 0.15915494309189533576888;   // 1 / (2 pi): turns per position
  t -= floor(t);
  const uint64_t step = __double2ull_rn(t * 18446744073709551616.0);
  const int32_t top = static_cast<int32_t>(static_cast<uint32_t>((pos * step) >> 32));
  sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &n, &c);   // 2^-31: half turns
}

// One thread: V pairs (or 2 V copied elements) of one token, of heads hs, hs + head_slots, ...
// TI -> TO is the tensors' type and the result's (the same for rope, bf16 for the caches); the
// rotation is computed in fp32 and rounded once.
//
// Bound by the bytes for long inputs: 32768 tokens of 64 + 8 heads of 128 (1.21 GB) take 191 us,
// 6.3 TB/s. Two blocks an SM and four heads in flight a thread (three blocks spill: 285 us; two
// heads and three blocks: 203 us). Short inputs wait for the chain position -> angle -> store:
// 64 tokens take 3.9 us.
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kRotThreads, 2) rotate_kernel(const __grid_constant__ RotateParams P) {
  int j = 0;
  while (j + 1 < P.count && blockIdx.x >= P.jobs[j + 1].block0) ++j;
  const RotateJob& J = P.jobs[j];
  const int rot = J.freqs ? J.rot : 0;
  const int units = J.dim / (2 * V);
  const int per_token = units * J.head_slots;
  const uint64_t base = static_cast<uint64_t>(blockIdx.x - J.block0) * kRotThreads;
  // 32-bit division where the number allows it (all but calls of billions of elements)
  const int64_t first = base >> 32 ? static_cast<int64_t>(base / per_token)
                                   : static_cast<int64_t>(static_cast<uint32_t>(base) / static_cast<uint32_t>(per_token));
  const int local = static_cast<int>(base - static_cast<uint64_t>(first) * per_token) + threadIdx.x;
  const int64_t tok = first + local / per_token;
  const int in_token = local % per_token;
  const int unit = in_token % units, hs = in_token / units;

  uint64_t pos = 0;
  int64_t dst_row = tok * J.dst_token;
  if (P.positions != nullptr) {
    if (tok >= P.n) return;
    pos = P.positions_i64 ? static_cast<uint64_t>(static_cast<const int64_t*>(P.positions)[tok])
                          : static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t*>(P.positions)[tok]));
  } else {
    int seq;
    int64_t left;   // new tokens of the sequence from this one on
    if (P.cu_seqlens == nullptr) {
      seq = static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(P.each));   // n < 2^26
      left = static_cast<int64_t>(seq + 1) * P.each - tok;
    } else {
      // sequences that end at or before the block's first token, counted by the whole block
      seq = 0;
      for (int b0 = 0; b0 < P.batch; b0 += kRotThreads) {
        const int b = b0 + threadIdx.x;
        seq += __syncthreads_count(b < P.batch && P.cu_seqlens[b + 1] <= first);
      }
      while (seq < P.batch && P.cu_seqlens[seq + 1] <= tok) ++seq;
      left = seq < P.batch ? P.cu_seqlens[seq + 1] - tok : 0;
    }
    if (tok >= P.n || seq >= P.batch) return;   // rows behind the last sequence
    const int64_t len = P.seqlens[seq];
    const int64_t p = len - left;
    // equal counts: an empty sequence's rows, and those before a shorter one's first token, have no token (as
    // in the decode of the same batch)
    if (P.cu_seqlens == nullptr && p < 0 && len >= 0) return;
    if (p < 0 || (p >> P.page_shift) >= P.max_pages) {
      record_error(MSA_ERR_DEVICE_BOUNDS, kKidRotate);
      return;
    }
    pos = static_cast<uint64_t>(p);
    if (J.paged) {
      const int64_t page = P.page_table[seq * P.table_stride + (p >> P.page_shift)];
      if (page < 0 || page >= P.num_pages) {
        record_error(MSA_ERR_DEVICE_BOUNDS, kKidRotate);
        return;
      }
      dst_row = page * J.dst_page + (p & ((int64_t(1) << P.page_shift) - 1)) * J.dst_token;
    }
  }

  const int half = rot / 2;
  const bool turn = unit * V < half;
  int ea, eb;   // first elements of the two vectors
  if (!turn) {
    ea = unit * 2 * V;
    eb = ea + V;
  } else if (P.interleaved) {
    ea = unit * 2 * V;
    eb = ea + V;
  } else {
    ea = unit * V;
    eb = half + unit * V;
  }
  const TI* src = static_cast<const TI*>(J.src) + tok * J.src_token;
  TO* dst = static_cast<TO*>(J.dst) + dst_row;
  float c[V], n[V];
  // heads in groups of kRotGroup: a group's loads are all in flight before its first result is
  // stored (the stores may go where the loads come from, so the compiler cannot move them)
  for (int h0 = hs; h0 < J.heads; h0 += kRotGroup * J.head_slots) {
    RotVec<TI, V> xa[kRotGroup], xb[kRotGroup];
#pragma unroll
    for (int i = 0; i < kRotGroup; ++i) {
      const int h = h0 + i * J.head_slots;
      if (h < J.heads) {
        xa[i] = *reinterpret_cast<const RotVec<TI, V>*>(src + h * J.src_head + ea);
        xb[i] = *reinterpret_cast<const RotVec<TI, V>*>(src + h * J.src_head + eb);
      }
    }
    if (turn && h0 == hs) {   // behind the first loads
#pragma unroll
      for (int i = 0; i < V; ++i) {
        rot_angle(J.freqs[unit * V + i], pos, c[i], n[i]);
        c[i] *= P.scale;
        n[i] *= P.scale * P.sign;
      }
    }
#pragma unroll
    for (int k = 0; k < kRotGroup; ++k) {
      const int h = h0 + k * J.head_slots;
      if (h >= J.heads) break;
      float a[V], b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] = rot_in(xa[k].e[i]);
        b[i] = rot_in(xb[k].e[i]);
      }
      RotVec<TO, V> ya, yb;
      const bool neighbours = V > 1 && turn && P.interleaved;
      if constexpr (V > 1) {
        if (neighbours) {   // the vector's first V / 2 pairs lie in xa, the others in xb
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const int lo = i / 2, hi = (V + i) / 2;
            ya.e[i] = rot_out<TO>(c[lo] * a[i] - n[lo] * a[i + 1]);
            ya.e[i + 1] = rot_out<TO>(n[lo] * a[i] + c[lo] * a[i + 1]);
            yb.e[i] = rot_out<TO>(c[hi] * b[i] - n[hi] * b[i + 1]);
            yb.e[i + 1] = rot_out<TO>(n[hi] * b[i] + c[hi] * b[i + 1]);
          }
        }
      }
      if (!neighbours) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ya.e[i] = rot_out<TO>(turn ? c[i] * a[i] - n[i] * b[i] : a[i]);
          yb.e[i] = rot_out<TO>(turn ? n[i] * a[i] + c[i] * b[i] : b[i]);
        }
      }
      *reinterpret_cast<RotVec<TO, V>*>(dst + h * J.dst_head + ea) = ya;
      *reinterpret_cast<RotVec<TO, V>*>(dst + h * J.dst_head + eb) = yb;
    }
  }
}

}  // namespace msa
