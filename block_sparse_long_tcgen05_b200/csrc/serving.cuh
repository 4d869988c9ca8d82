// Host side of the serving entry points (rotary positions, paged append, paged decode): their
// argument checks, workspace layout and launches. Included by msa_api.cu after its helpers.
#pragma once

// ------------------------------- rotary positions, append -------------------------------
msa_status_t check_rope_frequencies(const double* freqs, int32_t rot, const char* name) {
  if (freqs == nullptr) return fail(MSA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(freqs) % 8 != 0) return fail(MSA_ERR_INVALID_ARG, "%s is not 8-byte aligned", name);
  if (rot < 2 || rot % 2 != 0) return fail(MSA_ERR_INVALID_ARG, "%d rotated elements: a positive even number is wanted", rot);
  return MSA_OK;
}

int dtype_bytes(int32_t dtype) { return dtype == MSA_FP32 ? 4 : 2; }

// (n: tokens; the addresses of none do not matter)
msa_status_t check_rotate_tensor(const msa_rope_tensor& t, int32_t dtype, int32_t out_dtype, int32_t rot, int64_t n,
                                 const char* name) {
  if (t.heads < 1 || t.heads > 1024) return fail(MSA_ERR_INVALID_ARG, "%s: %d heads out of range [1, 1024]", name, t.heads);
  if (t.dim < 2 || t.dim > 1024 || t.dim % 2 != 0)
    return fail(MSA_ERR_UNSUPPORTED, "%s: dim=%d unsupported (even, 2..1024)", name, t.dim);
  if (rot > t.dim) return fail(MSA_ERR_INVALID_ARG, "%s: %d rotated elements of a head of %d", name, rot, t.dim);
  if (n == 0) return MSA_OK;
  if (t.x == nullptr || t.y == nullptr) return fail(MSA_ERR_INVALID_ARG, "%s: NULL pointer", name);
  if (reinterpret_cast<uintptr_t>(t.x) % dtype_bytes(dtype) != 0 || reinterpret_cast<uintptr_t>(t.y) % dtype_bytes(out_dtype) != 0)
    return fail(MSA_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  if ((t.heads > 1 && t.y_head_stride == 0) || (n > 1 && t.y_token_stride == 0))
    return fail(MSA_ERR_INVALID_ARG, "%s: several results would go to one place (a stride of 0)", name);
  return MSA_OK;
}

// A result that goes where the input lies replaces just what its thread has read only where both have the same
// layout: element sizes and strides.
msa_status_t check_in_place(const msa_rope_tensor& t, int32_t dtype, int32_t out_dtype, int64_t n, const char* name) {
  if (n == 0 || t.x != t.y) return MSA_OK;
  if (dtype_bytes(dtype) != dtype_bytes(out_dtype) || (n > 1 && t.x_token_stride != t.y_token_stride) ||
      (t.heads > 1 && t.x_head_stride != t.y_head_stride))
    return fail(MSA_ERR_INVALID_ARG, "%s: in place only with the same strides and element size", name);
  return MSA_OK;
}

RotateJob rotate_job(const msa_rope_tensor& t, const double* freqs, int32_t rot) {
  RotateJob j{};
  j.src = t.x;
  j.dst = t.y;
  j.src_token = t.x_token_stride;
  j.src_head = t.x_head_stride;
  j.dst_token = t.y_token_stride;
  j.dst_head = t.y_head_stride;
  j.freqs = freqs;
  j.heads = t.heads;
  j.dim = t.dim;
  j.rot = freqs ? rot : 0;
  return j;
}

template <typename TI, typename TO, int V>
msa_status_t launch_rotate_v(RotateParams& P, cudaStream_t st) {
  int64_t blocks = 0;
  const int sms = num_sms();
  int64_t all = 0;   // threads at a head each
  for (int i = 0; i < P.count; ++i) all += P.n * (P.jobs[i].dim / (2 * V)) * P.jobs[i].heads;
  for (int i = 0; i < P.count; ++i) {
    RotateJob& j = P.jobs[i];
    // One angle serves all of a thread's heads, so a thread takes up to 16 of them where the call's tensors
    // still leave an SM its 512 resident threads, and one where tokens are few. Appending 8191 tokens takes
    // 72 us so, 76 with each tensor counted alone, and 133 with four times the threads.
    const int64_t each = std::min<int64_t>(16, std::max<int64_t>(1, all / (int64_t(sms) * 2 * kRotThreads)));
    j.head_slots = int((j.heads + each - 1) / each);
    j.block0 = static_cast<unsigned int>(blocks);
    const int64_t threads = P.n * (j.dim / (2 * V)) * j.head_slots;
    blocks += (threads + kRotThreads - 1) / kRotThreads;
    if (blocks > 0x7fffffff) return fail(MSA_ERR_UNSUPPORTED, "%lld tokens of %d heads are too many for one call", (long long)P.n, j.heads);
  }
  if (blocks == 0) return MSA_OK;
  ProfScope ps(kPRotate, st);
  rotate_kernel<TI, TO, V><<<unsigned(blocks), kRotThreads, 0, st>>>(P);
  MSA_CHECK_LAUNCH();
  return MSA_OK;
}

// Whether every access of the call may be one of V elements: addresses, strides, and the places
// where pairs and the copied rest begin.
template <typename TI, typename TO>
bool rotate_fits(const RotateParams& P, int V) {
  for (int i = 0; i < P.count; ++i) {
    const RotateJob& j = P.jobs[i];
    if (reinterpret_cast<uintptr_t>(j.src) % (V * sizeof(TI)) != 0 || reinterpret_cast<uintptr_t>(j.dst) % (V * sizeof(TO)) != 0 ||
        (j.src_token | j.src_head | j.dst_token | j.dst_head | j.dst_page) % V != 0 || (j.rot / 2) % V != 0 ||
        (j.dim - j.rot) % (2 * V) != 0)
      return false;
  }
  return true;
}

// The widest access that fits all tensors of the call, 16 bytes at best, else two elements, else one; the
// tensor that fits least decides for the call. The 32K prompt of 64 + 8 heads in bf16 takes 191-196 us with
// 16-byte accesses, 300 two elements at a time and 393 element by element (in fp32, whose 16 bytes are four
// elements, 362, 394 and 459); appending 8191 tokens with index keys that rotate 128 or 32 elements 77-79 us, 24
// or 20 elements 116, 14 elements 161.
template <typename TI, typename TO>
msa_status_t launch_rotate(RotateParams& P, cudaStream_t st) {
  constexpr int W = 16 / sizeof(TI);
  if (rotate_fits<TI, TO>(P, W)) return launch_rotate_v<TI, TO, W>(P, st);
  if (rotate_fits<TI, TO>(P, 2)) return launch_rotate_v<TI, TO, 2>(P, st);
  return launch_rotate_v<TI, TO, 1>(P, st);
}

msa_status_t check_dtype(int32_t dtype) {
  if (dtype != MSA_BF16 && dtype != MSA_FP16 && dtype != MSA_FP32)
    return fail(MSA_ERR_UNSUPPORTED, "dtype=%d unsupported (MSA_BF16, MSA_FP16, MSA_FP32)", dtype);
  return MSA_OK;
}

// ------------------------------- paged cache -------------------------------
msa_status_t check_paged_cache(const msa_paged_cache* c) {
  if (!c) return fail(MSA_ERR_INVALID_ARG, "cache is NULL");
  if (c->g < 1 || c->g > 64) return fail(MSA_ERR_INVALID_ARG, "g=%d out of range [1, 64]", c->g);
  if (c->d != 64 && c->d != 128) return fail(MSA_ERR_UNSUPPORTED, "d=%d unsupported (64, 128)", c->d);
  msa_status_t s;
  if ((s = check_d_idx(c->d_idx)) != MSA_OK) return s;
  const int ps = c->page_size;
  if (ps < 16 || ps > 1024 || (ps & (ps - 1)) != 0)
    return fail(MSA_ERR_UNSUPPORTED, "page_size=%d unsupported (a power of two, 16..1024)", ps);
  if (c->num_pages < 1 || c->num_pages > 0x7fffffff)
    return fail(MSA_ERR_INVALID_ARG, "num_pages=%lld out of range [1, 2^31)", (long long)c->num_pages);
  const struct { const void* p; int64_t stride; int dim; const char* name; } t[3] = {
      {c->k, c->k_page_stride, c->d, "k pages"}, {c->v, c->v_page_stride, c->d, "v pages"},
      {c->k_idx, c->k_idx_page_stride, c->d_idx, "k_idx pages"}};
  for (auto& x : t) {
    if ((s = check_ptr(x.p, x.name)) != MSA_OK) return s;
    if (x.stride < int64_t(ps) * c->g * x.dim || x.stride % 8 != 0 || x.stride > (int64_t(1) << 38))
      return fail(MSA_ERR_INVALID_ARG, "%s: page stride %lld (at least a page's elements, a multiple of 8)", x.name,
                  (long long)x.stride);
  }
  return MSA_OK;
}

int page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

msa_status_t check_sequences(const msa_paged_cache* c, int32_t batch, int32_t max_pages, int64_t table_stride,
                             const int32_t* table, const int32_t* seqlens) {
  if (batch < 1 || batch > kScanMaxBatch)
    return fail(MSA_ERR_UNSUPPORTED, "batch=%d unsupported (1..%d)", batch, kScanMaxBatch);
  if (max_pages < 1 || int64_t(max_pages) * c->page_size > kMaxN)
    return fail(MSA_ERR_INVALID_ARG, "max_pages=%d: at least one, and at most %lld tokens", max_pages, (long long)kMaxN);
  if (table_stride < max_pages) return fail(MSA_ERR_INVALID_ARG, "table_stride=%lld < max_pages=%d", (long long)table_stride, max_pages);
  const struct { const void* p; const char* name; } t[2] = {{table, "page_table"}, {seqlens, "seqlens"}};
  for (auto& x : t) {
    if (x.p == nullptr) return fail(MSA_ERR_INVALID_ARG, "%s is NULL", x.name);
    if (reinterpret_cast<uintptr_t>(x.p) % 4 != 0) return fail(MSA_ERR_INVALID_ARG, "%s is not 4-byte aligned", x.name);
  }
  return MSA_OK;
}

// CTAs of the paged attention: as many as are resident at once.
int paged_attn_ctas(int R) { return kPagedAttnCtas(R <= 8 ? 1 : 2) * num_sms(); }

// Launches a kernel of a decode; `after`: its blocks may start while the decode's kernel before it
// still runs (each waits for it where it first needs its results). The first one of a call starts
// when everything before it in the stream is done, as always.
template <typename... Params, typename... Args>
msa_status_t launch_step(void (*kernel)(Params...), int64_t grid, int threads, int smem, bool after, cudaStream_t st,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  MSA_CHECK_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
  return MSA_OK;
}

// Shared-memory limit of a kernel, set once on each device that it is launched on.
template <typename K>
msa_status_t smem_limit(std::atomic<uint64_t>& done, K kernel, int bytes) {
  int dev = 0;
  MSA_CHECK_CUDA(cudaGetDevice(&dev));
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return MSA_OK;
  const msa_status_t s = set_smem(kernel, bytes);
  if (s == MSA_OK) done.fetch_or(bit, std::memory_order_release);
  return s;
}

struct PagedLayout {
  uint32_t* maxima = nullptr;
  int32_t* block_ids = nullptr;
  float* parts = nullptr;
  unsigned int* arrived = nullptr;
  size_t bytes = 0;
};

int64_t paged_blocks(const msa_paged_cache* c, const msa_paged_decode_params* p) {
  return (int64_t(p->max_pages) * c->page_size + p->bk - 1) / p->bk;
}

PagedLayout paged_layout(void* ws, const msa_paged_cache* c, const msa_paged_decode_params* p) {
  const int64_t rows = int64_t(p->batch) * p->n_new;
  Carver cv(ws);
  PagedLayout L;
  L.maxima = static_cast<uint32_t*>(cv.take(size_t(rows) * c->g * paged_blocks(c, p) * 4));
  L.block_ids = static_cast<int32_t*>(cv.take(size_t(rows) * c->g * p->k * 4));   // used when the caller takes none
  L.parts = static_cast<float*>(cv.take(size_t(2) * paged_attn_ctas(p->hq / c->g) * (p->hq / c->g) * (c->d + 2) * 4));
  L.arrived = static_cast<unsigned int*>(cv.take(size_t(rows) * c->g * 4));
  L.bytes = cv.off;
  return L;
}

// Everything of a decode call but the tensors' addresses.
msa_status_t check_paged_shapes(const msa_paged_cache* c, const msa_paged_decode_params* p) {
  if (!c || !p) return fail(MSA_ERR_INVALID_ARG, "%s is NULL", c ? "params" : "cache");
  msa_status_t s;
  if (p->bk != 128 && p->bk != 64 && p->bk != 32) return fail(MSA_ERR_UNSUPPORTED, "bk=%d unsupported (32, 64, 128)", p->bk);
  if (p->k < 1 || p->k > 32) return fail(MSA_ERR_UNSUPPORTED, "k=%d unsupported (1..32)", p->k);
  if (p->n_new < 1 || p->n_new > 8) return fail(MSA_ERR_UNSUPPORTED, "n_new=%d unsupported (1..8 new tokens a sequence)", p->n_new);
  if ((s = check_paged_cache(c)) != MSA_OK) return s;
  if (p->hq < 1 || p->hq % c->g != 0) return fail(MSA_ERR_INVALID_ARG, "hq=%d is not a positive multiple of g=%d", p->hq, c->g);
  if (p->hq / c->g > 16) return fail(MSA_ERR_UNSUPPORTED, "hq/g=%d unsupported (at most 16)", p->hq / c->g);
  if (!(p->scale >= 0.0f) || std::isinf(p->scale)) return fail(MSA_ERR_INVALID_ARG, "scale must be finite and >= 0");
  if (p->batch < 1 || p->batch > kScanMaxBatch)
    return fail(MSA_ERR_UNSUPPORTED, "batch=%d unsupported (1..%d)", p->batch, kScanMaxBatch);
  if (p->max_pages < 1 || int64_t(p->max_pages) * c->page_size > kMaxN)
    return fail(MSA_ERR_INVALID_ARG, "max_pages=%d: at least one, and at most %lld tokens", p->max_pages, (long long)kMaxN);
  return MSA_OK;
}

template <int DI>
msa_status_t launch_paged_scan(const PagedScanParams& P, bool after, cudaStream_t st) {
  static std::once_flag once;
  static int per_sm = 0;
  std::call_once(once, [] {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, paged_scan_kernel<DI>, kScanThreads, 0) != cudaSuccess) per_sm = 0;
  });
  if (per_sm < 1) return fail(MSA_ERR_CUDA, "paged scan: no resident block");
  // at most the work of full-length sequences: eight (span, group) units a block
  const int64_t most = int64_t(P.view.batch) * ((int64_t(P.nbmax) * P.bk + 127) / 128) * P.G;
  const int64_t grid = std::min<int64_t>(int64_t(num_sms()) * per_sm, (most + 7) / 8);
  ProfScope ps(kPPagedScan, st);
  return launch_step(paged_scan_kernel<DI>, std::max<int64_t>(grid, 1), kScanThreads, 0, after, st, P);
}

template <int DI, int RT>
msa_status_t launch_prefix_scan(const CUtensorMap& tq, const CUtensorMap& tk, PrefixScanParams P, cudaStream_t st) {
  using C = PrefixCfg<DI, RT>;
  static std::atomic<uint64_t> limit{0};
  msa_status_t s;
  if ((s = smem_limit(limit, prefix_scan_kernel<DI, RT>, C::kSmemBytes)) != MSA_OK) return s;
  const int sms = num_sms();
  // (a pair's share of the SMs is rounded down: between half as many pairs as SMs and all of them, the rest idle)
  P.pairs = (P.rows + RT * 128 - 1) / (RT * 128) * P.G;
  P.workers = std::max(1, std::min(sms / P.pairs, P.tiles));
  const int grid = P.workers > 1 ? P.workers * P.pairs : std::min(sms, P.pairs);
  ProfScope ps(kPPrefixScan, st);
  return launch_step(prefix_scan_kernel<DI, RT>, grid, kPrefixThreads, C::kSmemBytes, false, st, tq, tk, P);
}

template <int DI>
msa_status_t run_prefix_scan(const msa_paged_cache* c, const void* q_idx, const PrefixScanParams& P, cudaStream_t st) {
  using I = IdxCfg<DI>;
  const CUtensorMapSwizzle sw = I::kSw64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t row = uint64_t(c->g) * DI * 2;
  CUtensorMap tq, tk;
  msa_status_t s;
  if ((s = make_map_3d(&tq, q_idx, DI, c->g, P.rows, DI * 2, row, I::kPanelElems, 1, 128, sw)) != MSA_OK) return s;
  if ((s = make_map_4d(&tk, c->k_idx, {uint64_t(DI), uint64_t(c->g), uint64_t(c->page_size), uint64_t(c->num_pages)},
                       {uint64_t(DI) * 2, row, uint64_t(c->k_idx_page_stride) * 2},
                       {uint32_t(I::kPanelElems), 1, uint32_t(std::min(c->page_size, 128)), 1}, sw)) != MSA_OK)
    return s;
  return P.rows <= 128 ? launch_prefix_scan<DI, 1>(tq, tk, P, st) : launch_prefix_scan<DI, 2>(tq, tk, P, st);
}

template <int D, int NT>
msa_status_t launch_paged_attn(const PagedAttnParams& P, cudaStream_t st) {
  using C = PagedAttnCfg<D>;
  static std::atomic<uint64_t> limit{0};
  msa_status_t s;
  if ((s = smem_limit(limit, paged_attn_kernel<D, NT>, C::smem_bytes(kScanMaxBatch))) != MSA_OK) return s;
  const int64_t most = int64_t(P.view.batch) * P.view.S * P.G * (int64_t(P.k) << (P.bk_shift - 4));   // strips
  const int64_t grid = std::min<int64_t>(paged_attn_ctas(P.R), (most + kPagedAttnLeast - 1) / kPagedAttnLeast);
  ProfScope ps(kPPagedAttn, st);
  return launch_step(paged_attn_kernel<D, NT>, grid, kPagedAttnWarps * 32, C::smem_bytes(P.view.batch), true, st, P);
}

// One launch for the whole decode. Wanted where the clusters of all (row, group)s are resident at once (they
// gain 30 to 45% there; at twice as many the three kernels are as fast, at four times faster) and a cluster
// scans the longest sequence in about the time that two more launches take. Lengths are known on the device
// alone, so the longest sequence is taken to be what the page table has room for: one of 700 tokens takes 7.7 us
// under a table of 44 pages of 16 and 14.2 under one of 1025. 16384 tokens (8 groups of 128
// index elements: 28 us against 30; at 30000 tokens 51 against 34), 256 blocks (500 blocks of 32 tokens:
// 23 against 17). `done`: whether it was launched.
template <int D, int NT, int DI>
msa_status_t try_paged_small(const PagedSmallParams& P, bool& done, cudaStream_t st) {
  constexpr int smem = kPagedAttnWarps * 2 * 16 * D * 2;
  static std::atomic<uint64_t> limit{0};
  msa_status_t s;
  if ((s = smem_limit(limit, paged_small_kernel<D, NT, DI>, smem)) != MSA_OK) return s;
  static std::once_flag once;
  static int resident = 0;   // clusters
  std::call_once(once, [] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSmallCluster);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSmallCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&resident, paged_small_kernel<D, NT, DI>, &cfg) != cudaSuccess) resident = 0;
  });
  const int64_t clusters = int64_t(P.view.batch) * P.view.S * P.G;
  done = clusters <= resident;
  if (!done) return MSA_OK;
  ProfScope ps(kPPagedSmall, st);
  paged_small_kernel<D, NT, DI><<<unsigned(clusters * kSmallCluster), kSmallThreads, smem, st>>>(P);
  MSA_CHECK_LAUNCH();
  return MSA_OK;
}

template <int D, int NT>
msa_status_t try_paged_small(int d_idx, const PagedSmallParams& P, bool& done, cudaStream_t st) {
  return d_idx == 128 ? try_paged_small<D, NT, 128>(P, done, st) : d_idx == 64 ? try_paged_small<D, NT, 64>(P, done, st)
                                                                             : try_paged_small<D, NT, 32>(P, done, st);
}

msa_status_t run_paged_decode(const msa_paged_cache* c, const msa_paged_decode_params* p, const void* q, const void* q_idx,
                              int32_t* block_ids_out, void* o, void* ws, cudaStream_t st) {
  const PagedLayout L = paged_layout(ws, c, p);
  PageView V{};
  V.table = p->page_table;
  V.prefix = p->prefix_pages;
  V.seqlens = p->seqlens;
  V.table_stride = p->table_stride;
  V.num_pages = c->num_pages;
  V.prefix_pages = p->n_prefix_pages;
  V.max_pages = p->max_pages;
  V.shift = page_shift(c->page_size);
  V.batch = p->batch;
  V.S = p->n_new;
  const float scale_log2 = (p->scale == 0.0f ? 1.0f / std::sqrt(float(c->d)) : p->scale) * 1.4426950408889634f;
  const int nbmax = int(paged_blocks(c, p));
  int32_t* ids = block_ids_out ? block_ids_out : L.block_ids;
  msa_status_t s;
  if (int64_t(p->max_pages) * c->page_size <= 16384 && nbmax <= kSmallBlocks) {
    PagedSmallParams P{};
    P.view = V;
    P.q_idx = static_cast<const __nv_bfloat16*>(q_idx);
    P.ip = static_cast<const __nv_bfloat16*>(c->k_idx);
    P.q = static_cast<const __nv_bfloat16*>(q);
    P.kp = static_cast<const __nv_bfloat16*>(c->k);
    P.vp = static_cast<const __nv_bfloat16*>(c->v);
    P.i_stride = c->k_idx_page_stride;
    P.k_stride = c->k_page_stride;
    P.v_stride = c->v_page_stride;
    P.block_ids = ids;
    P.o = static_cast<__nv_bfloat16*>(o);
    P.G = c->g;
    P.R = p->hq / c->g;
    P.k = p->k;
    P.bk_shift = page_shift(p->bk);
    P.scale_log2 = scale_log2;
    bool done = false;
    if (P.R <= 8) s = c->d == 128 ? try_paged_small<128, 1>(c->d_idx, P, done, st) : try_paged_small<64, 1>(c->d_idx, P, done, st);
    else s = c->d == 128 ? try_paged_small<128, 2>(c->d_idx, P, done, st) : try_paged_small<64, 2>(c->d_idx, P, done, st);
    if (done || s != MSA_OK) return s;
  }
  bool scanned = false;
  if (p->k > 1 && nbmax > p->k) {   // else every visible block is taken, or the local one alone
    PagedScanParams sp{};
    sp.view = V;
    sp.q_idx = static_cast<const __nv_bfloat16*>(q_idx);
    sp.pages = static_cast<const __nv_bfloat16*>(c->k_idx);
    sp.page_stride = c->k_idx_page_stride;
    sp.maxima = L.maxima;
    sp.G = c->g;
    sp.bk = p->bk;
    sp.k = p->k;
    sp.nbmax = nbmax;
    // Whole blocks of a shared prefix are scored once for all rows, where that spares reading 16 MB of keys
    // again and again (one more launch is as long: 4 sequences behind 16384 tokens of 4 groups of 64, 25 MB,
    // 19 us against 20; 2, 8 MB, 19 against 17), and where the prefix has as many blocks as are selected (a
    // sequence of fewer is not scored at all: 64 behind 1024 tokens, k = 16, 51 us against 46).
    const int prefix_blocks = int(int64_t(p->n_prefix_pages) * c->page_size / p->bk);
    const int64_t spared = int64_t(p->batch - 1) * prefix_blocks * p->bk * c->g * c->d_idx * 2;
    if (spared >= int64_t(16) << 20 && prefix_blocks >= p->k) {
      PrefixScanParams P{};
      P.prefix = p->prefix_pages;
      P.maxima = L.maxima;
      P.num_pages = c->num_pages;
      P.n_pages = p->n_prefix_pages;
      P.shift = V.shift;
      P.rows = p->batch * p->n_new;
      P.G = c->g;
      P.bk = p->bk;
      P.nbmax = nbmax;
      P.blocks = prefix_blocks;
      P.tiles = int((int64_t(P.blocks) * p->bk + 127) / 128);
      s = c->d_idx == 128 ? run_prefix_scan<128>(c, q_idx, P, st) : c->d_idx == 64 ? run_prefix_scan<64>(c, q_idx, P, st)
                                                                                   : run_prefix_scan<32>(c, q_idx, P, st);
      if (s != MSA_OK) return s;
      sp.nb0 = P.blocks;
    }
    s = c->d_idx == 128 ? launch_paged_scan<128>(sp, sp.nb0 > 0, st) : c->d_idx == 64 ? launch_paged_scan<64>(sp, sp.nb0 > 0, st)
                                                                                   : launch_paged_scan<32>(sp, sp.nb0 > 0, st);
    if (s != MSA_OK) return s;
    scanned = true;
  }
  PagedTopkParams tp{};
  tp.view = V;
  tp.maxima = L.maxima;
  tp.block_ids = ids;
  tp.G = c->g;
  tp.bk = p->bk;
  tp.k = p->k;
  tp.nbmax = nbmax;
  tp.arrived = L.arrived;
  tp.o = static_cast<__nv_bfloat16*>(o);
  tp.width = p->hq / c->g * c->d;
  const int64_t rg = int64_t(p->batch) * p->n_new * c->g;
  {
    ProfScope ps(kPPagedTopk, st);
    if ((s = launch_step(paged_topk_kernel, (rg + 3) / 4, 128, 0, scanned, st, tp)) != MSA_OK) return s;
  }
  PagedAttnParams ap{};
  ap.view = V;
  ap.q = static_cast<const __nv_bfloat16*>(q);
  ap.kp = static_cast<const __nv_bfloat16*>(c->k);
  ap.vp = static_cast<const __nv_bfloat16*>(c->v);
  ap.k_stride = c->k_page_stride;
  ap.v_stride = c->v_page_stride;
  ap.block_ids = ids;
  ap.o = static_cast<__nv_bfloat16*>(o);
  ap.parts = L.parts;
  ap.arrived = L.arrived;
  ap.G = c->g;
  ap.R = p->hq / c->g;
  ap.k = p->k;
  ap.bk_shift = page_shift(p->bk);
  ap.scale_log2 = scale_log2;
  if (ap.R <= 8) return c->d == 128 ? launch_paged_attn<128, 1>(ap, st) : launch_paged_attn<64, 1>(ap, st);
  return c->d == 128 ? launch_paged_attn<128, 2>(ap, st) : launch_paged_attn<64, 2>(ap, st);
}
