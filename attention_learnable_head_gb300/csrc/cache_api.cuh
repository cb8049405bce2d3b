// Host side of attn_sink_cache.h: validation, workspace carving and launches.  Included
// by attn_sink_api.cu after step_api.cuh, with which it shares the launch helpers.
#pragma once

namespace {

// What the entry points have in common: a paged cache of heads of 64, and a block table.
template <typename P>
int cache_validate(const P* p, int most_batch) {
  if (p == nullptr) return ATTN_SINK_ERR_INVALID_ARG;
  if (p->head_dim != kHeadDim) return ATTN_SINK_ERR_UNSUPPORTED;
  if (p->batch < 0 || p->heads_kv < 1 || p->page_size < 1 || p->num_pages < 0 ||
      p->max_pages < 0 || (long long)p->max_pages * p->page_size > (1ll << 30))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (p->batch > most_batch ||
      (long long)p->num_pages * p->page_size > ((1ll << 32) - 1) / p->heads_kv)
    return ATTN_SINK_ERR_UNSUPPORTED;
  return ATTN_SINK_OK;
}

template <typename P>
int group_validate(const P* p) {
  if (p->heads_q < 1 || p->heads_q % p->heads_kv != 0) return ATTN_SINK_ERR_INVALID_ARG;
  if ((long long)p->batch * p->heads_q >= (1ll << 31)) return ATTN_SINK_ERR_UNSUPPORTED;
  return decode_group_ok(p->heads_q / p->heads_kv) ? ATTN_SINK_OK : ATTN_SINK_ERR_UNSUPPORTED;
}

bool scale_ok(float s) { return std::isfinite(s) && s > 0.0f; }

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

// ----------------------------------------------------------------------------- decode
// The slices of a sequence's keys, and what they leave.
struct DecodeSlices {
  int splits;
  size_t off_ml, total;
};
DecodeSlices decode_slices(int splits, int batch, int heads_q) {
  DecodeSlices d;
  d.splits = splits;
  const size_t rows = (size_t)splits * batch * heads_q;
  d.off_ml = align256(rows * kHeadDim * sizeof(float));
  d.total = d.off_ml + align256(rows * sizeof(float2));
  return d;
}

// Slices of a sequence of up to `keys` keys: four rounds of the CTAs that the GPU holds at
// once, so that a last, partly filled one matters less, of kSliceLong keys or more; or, of
// few sequences, as many as it holds, of `least` keys or more.
constexpr int kSliceLong = 512;
constexpr int kSliceRounds = 4;
int decode_splits(int batch, int heads_kv, long long keys, int least, int sms) {
  const long long ctas = std::max(1ll, (long long)batch * heads_kv);
  const long long slots = kSliceCtas * (long long)sms;
  const long long rounds = std::min((kSliceRounds * slots + ctas - 1) / ctas, keys / kSliceLong);
  const long long fill = std::min(slots / ctas, (keys + least - 1) / least);
  return (int)std::max(1ll, std::min((long long)kSliceMax, std::max(rounds, fill)));
}

// The fields of SliceParams that both uses have; *tma: which copies are taken.
template <typename P>
int decode_params(const P* p, const DecodeSlices& L, const void* q, const void* k_cache,
                  const void* v_cache, const int* block_table, const int* seq_lens,
                  const float* sink, void* out, float* lse, uint8_t* ws, int* err,
                  bool own_pages, SliceParams* dp, bool* tma) {
  std::memset(dp, 0, sizeof(*dp));
  dp->q = static_cast<const __nv_bfloat16*>(q);
  dp->k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  dp->v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  dp->block_table = block_table;
  dp->seq_lens = seq_lens;
  dp->slice_o = reinterpret_cast<float*>(ws);
  dp->slice_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  dp->sink = sink;
  dp->out = static_cast<__nv_bfloat16*>(out);
  dp->lse = lse;
  dp->err = err;
  dp->batch = p->batch;
  dp->heads_q = p->heads_q;
  dp->heads_kv = p->heads_kv;
  dp->page_size = p->page_size;
  dp->num_pages = p->num_pages;
  dp->max_pages = p->max_pages;
  dp->splits = L.splits;
  dp->whole = L.splits == 1;
#ifdef ATTN_SINK_TEST_HOOKS
  dp->skip_k_tile = g_test_skip_k_tile.load();
#endif
  dp->scale_log2 = p->softmax_scale * kLog2e;
  const long long rows = (long long)p->num_pages * p->page_size;
  *tma = slice_tma_page(p->page_size) && rows > 0 && rows < (1ll << 31);
  if (!*tma) return ATTN_SINK_OK;
  dp->log2_page = log2_of(p->page_size);
  const int box = std::min(p->page_size, kSliceKeys);
  // With pages of its own for each head no more than its 128 bytes into L2: its
  // neighbour's are not wanted (64 sequences x 2048 keys read 375 MB of 269 and took 67
  // us, not 55, where L2 fetched 256 bytes)
  const CUtensorMapL2promotion promotion =
      own_pages ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  int st;
  if ((st = encode_rows(&dp->tm_k, k_cache, rows, p->heads_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        box, 1, promotion)) != ATTN_SINK_OK)
    return st;
  return encode_rows(&dp->tm_v, v_cache, rows, p->heads_kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     box, 1, promotion);
}

template <bool kShared>
auto slice_kernel(int group, bool tma) -> void (*)(SliceParams) {
  switch (group * 2 + (tma ? 1 : 0)) {
    case 2: return attn_sink_slice_kernel<1, false, kShared>;
    case 3: return attn_sink_slice_kernel<1, true, kShared>;
    case 4: return attn_sink_slice_kernel<2, false, kShared>;
    case 5: return attn_sink_slice_kernel<2, true, kShared>;
    case 8: return attn_sink_slice_kernel<4, false, kShared>;
    case 9: return attn_sink_slice_kernel<4, true, kShared>;
    case 16: return attn_sink_slice_kernel<8, false, kShared>;
    default: return attn_sink_slice_kernel<8, true, kShared>;
  }
}

template <bool kShared>
bool launch_join(const SliceParams& dp, cudaStream_t s) {
  constexpr int kRows = kJoinThreads / 32;
  const long long rows = (long long)dp.batch * dp.heads_q;
  return launch_dependent(attn_sink_join_kernel<kShared>,
                          dim3((unsigned)((rows + kRows - 1) / kRows)), kJoinThreads, 0, s, dp);
}

// ----------------------------------------------------------------------------- shared prefixes
struct SharedLayout {
  DecodeSlices own;
  int tokens, n_items, slots;
  size_t off_items, off_refs, off_ml, off_o, total;
};

// Slices of the keys behind the prefix, of which the host only knows that they are not
// more than the table holds (right for own keys that are alike: 40 sequences behind a prefix
// and 24 of 1000 to 100000 own keys take 771 us, attn_sink_decode, which cuts all, 316): one, which joins the prefix itself and needs no kernel for
// that (4 us), where the CTAs fill half of the GPU or the table is short; else of
// kSharedLong keys or more.  A block of keys takes a warp of a CTA by itself about 1 us.
constexpr int kSharedWhole = 2048;
constexpr int kSharedLong = 256;
int shared_splits(int batch, int heads_kv, long long cap, int sms) {
  if (2ll * batch * heads_kv >= kSliceCtas * (long long)sms || cap <= kSharedWhole) return 1;
  return decode_splits(batch, heads_kv, cap, kSharedLong, sms);
}

int shared_layout(const attn_sink_shared_params* p, int sms, SharedLayout* L) {
  int st = cache_validate(p, 65535);
  if (st != ATTN_SINK_OK || (st = group_validate(p)) != ATTN_SINK_OK) return st;
  if (!scale_ok(p->softmax_scale) || p->num_groups < 0 || p->num_groups > p->batch ||
      (p->num_groups == 0 && p->batch > 0))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (p->heads_kv > 65535) return ATTN_SINK_ERR_UNSUPPORTED;
  L->tokens = kBlockM / (p->heads_q / p->heads_kv);
  L->slots = kExtCtasPerSm * sms;
  // the bounds of attn_sink_shared_plan_kernel: a share's parts and one more a tile, of groups of
  // kSharedMinSeqs sequences or more (4096 sequences each in a group of its own: 702 MB of
  // workspace, 1256 where those counted too)
  const long long tiles =
      (long long)p->batch / L->tokens + std::min(p->num_groups, p->batch / kSharedMinSeqs);
  const long long items = tiles + (L->slots + p->heads_kv - 1) / p->heads_kv;
  if (items * p->heads_kv >= (1ll << 31)) return ATTN_SINK_ERR_UNSUPPORTED;   // launch grid
  L->n_items = (int)items;
  const long long cap = (long long)p->max_pages * p->page_size;
  L->own = decode_slices(shared_splits(p->batch, p->heads_kv, cap, sms), p->batch, p->heads_q);
  size_t off = L->own.total;
  L->off_items = off;
  off += align256((size_t)L->n_items * sizeof(ExtItem));
  L->off_refs = off;
  off += align256((size_t)p->batch * sizeof(SharedRef));
  const size_t parts = (size_t)L->n_items * p->heads_kv;
  L->off_ml = off;
  off += align256(parts * kBlockM * sizeof(float2));
  L->off_o = off;
  off += align256(parts * kBlockM * kHeadDim * sizeof(float));
  L->total = off;
  return ATTN_SINK_OK;
}

// ----------------------------------------------------------------------------- selection
struct SelectLayout {
  int tiles;
  size_t off_peak, off_exact, total;
};

int select_layout(const attn_sink_select_params* p, SelectLayout* L) {
  int st = cache_validate(p, 65535);
  if (st != ATTN_SINK_OK || (st = group_validate(p)) != ATTN_SINK_OK) return st;
  if (p->count < 1 || p->keep_first < 0 || p->keep_last < 0 ||
      (long long)p->keep_first + p->keep_last > p->count)
    return ATTN_SINK_ERR_INVALID_ARG;
  if ((long long)p->batch * p->heads_kv >= (1ll << 31)) return ATTN_SINK_ERR_UNSUPPORTED;
  const size_t rows = (size_t)p->batch * p->heads_kv;
  L->tiles = (p->max_pages + 15) / 16;
  L->off_peak = align256(rows * p->max_pages * sizeof(float));
  L->off_exact = L->off_peak + align256(rows * L->tiles * sizeof(unsigned));
  L->total = L->off_exact + align256(rows * p->max_pages * sizeof(unsigned long long));
  return ATTN_SINK_OK;
}

// Rows of q a sequence, on average, up to which warps keep them in registers.  The host knows
// the average alone, so this is right for sequences that are alike: one with many rows among
// many with few is read once for every 32 of them (255 single tokens on 1024 keys 53 us, a
// chunk of 512 on 16384 keys 111 us, both together 36 ms).
constexpr int kMassFewRows = 32;

// Threads of a selection's or an eviction's CTA, for rows of so many values.
int row_threads(int row) { return row <= 2048 ? 256 : row <= 8192 ? 512 : 1024; }

// ----------------------------------------------------------------------------- eviction
// Shared memory up to which a row's moves are listed there: that of four CTAs fits an SM, whose
// registers hold four of 256 threads, two of 512 or one of 1024.
constexpr size_t kEvictLists = 40 * 1024;
struct EvictLayout {
  int max_moves;
  size_t off_moves, off_from, total;
};

int evict_layout(const attn_sink_evict_params* p, EvictLayout* L) {
  int st = cache_validate(p, 65535);
  if (st != ATTN_SINK_OK) return st;
  if (p->max_keys < 0 || p->budget < 0 || p->keep_first < 0 || p->keep_last < 0 ||
      p->max_freed < 0 || (long long)p->keep_first + p->keep_last > p->budget)
    return ATTN_SINK_ERR_INVALID_ARG;
  if (p->max_keys > (1 << 30) || (long long)p->batch * p->heads_kv >= (1ll << 31) - 1 ||
      (long long)p->batch * p->max_pages >= (1ll << 31))
    return ATTN_SINK_ERR_UNSUPPORTED;
  const int behind = std::max(0, p->max_keys - p->budget);
  L->max_moves = std::min(p->budget, behind);
  const size_t rows = (size_t)p->batch * p->heads_kv;
  L->off_moves = align256(rows * sizeof(int));
  L->off_from = L->off_moves + align256(rows * L->max_moves * sizeof(int));
  L->total = L->off_from + align256(rows * L->max_moves * sizeof(int));
  return ATTN_SINK_OK;
}

auto select_kernel(int threads) -> void (*)(SelectParams) {
  return threads == 256   ? attn_sink_select_kernel<256>
         : threads == 512 ? attn_sink_select_kernel<512>
                          : attn_sink_select_kernel<1024>;
}
auto evict_kernel(int threads) -> void (*)(EvictParams) {
  return threads == 256   ? attn_sink_evict_kernel<256>
         : threads == 512 ? attn_sink_evict_kernel<512>
                          : attn_sink_evict_kernel<1024>;
}

auto prefix_kernel(bool tma) -> void (*)(ExtParams) {
  return tma ? attn_sink_extend_kernel<true, true> : attn_sink_extend_kernel<false, true>;
}

bool g_cache_attr_set[kMaxDevices] = {false};

// The shared memory limits of the kernels that keep a row in it, once per device.
int cache_attributes() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return ATTN_SINK_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  if (!g_cache_attr_set[dev]) {
    for (int group : {1, 2, 4, 8})
      for (bool tma : {false, true})
        if (cudaFuncSetAttribute(slice_kernel<false>(group, tma),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSliceSmem) != cudaSuccess ||
            cudaFuncSetAttribute(slice_kernel<true>(group, tma),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSliceSmem) != cudaSuccess)
          return ATTN_SINK_ERR_CUDA;
    for (bool tma : {false, true})
      if (cudaFuncSetAttribute(prefix_kernel(tma), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kFwdSmemBytes) != cudaSuccess)
        return ATTN_SINK_ERR_CUDA;
    for (int threads : {256, 512, 1024})
      if (cudaFuncSetAttribute(evict_kernel(threads), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               4 * kEvictStage) != cudaSuccess ||
          cudaFuncSetAttribute(select_kernel(threads), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               4 * kSelectStage) != cudaSuccess)
        return ATTN_SINK_ERR_CUDA;
    if (cudaFuncSetAttribute(attn_sink_key_mass_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMassSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(attn_sink_key_mass_few_kernel<1>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMassFewSmem) != cudaSuccess ||
        cudaFuncSetAttribute(attn_sink_key_mass_few_kernel<4>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMassFewSmem) != cudaSuccess ||
        cudaFuncSetAttribute(attn_sink_page_scores_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kScoreSmem) != cudaSuccess)
      return ATTN_SINK_ERR_CUDA;
    g_cache_attr_set[dev] = true;
  }
  return ATTN_SINK_OK;
}

}  // namespace

extern "C" {

size_t attn_sink_decode_shared_workspace_size(const attn_sink_shared_params* params) {
  SharedLayout L;
  if (shared_layout(params, sm_count_or_default(), &L) != ATTN_SINK_OK || params->batch == 0)
    return 0;
  return L.total;
}

int attn_sink_decode_shared(const attn_sink_shared_params* params, const void* q,
                            const void* k_cache, const void* v_cache, const int* block_table,
                            const int* seq_lens, const int* cu_groups, const int* prefix_lens,
                            const float* sink, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  NvtxRange range("attn_sink_decode_shared");
  SharedLayout L;
  int st = shared_layout(params, sm_count_or_default(), &L);
  if (st != ATTN_SINK_OK) return st;
  if (params->batch == 0) return ATTN_SINK_OK;
  if (q == nullptr || sink == nullptr || out == nullptr || lse == nullptr ||
      seq_lens == nullptr || cu_groups == nullptr || prefix_lens == nullptr ||
      (params->max_pages > 0 && block_table == nullptr) ||
      (params->num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, L.total)) return ATTN_SINK_ERR_WORKSPACE;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  if ((st = cache_attributes()) != ATTN_SINK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SliceParams dp;
  bool dec_tma;
  if ((st = decode_params(params, L.own, q, k_cache, v_cache, block_table, seq_lens, sink, out,
                          lse, ws, err, false, &dp, &dec_tma)) != ATTN_SINK_OK)
    return st;
  dp.cu_groups = cu_groups;
  dp.prefix_lens = prefix_lens;
  dp.num_groups = params->num_groups;
  dp.refs = reinterpret_cast<SharedRef*>(ws + L.off_refs);
  dp.prefix_o = reinterpret_cast<float*>(ws + L.off_o);
  dp.prefix_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  SharedPlan sp;
  std::memset(&sp, 0, sizeof(sp));
  ExtParams& ep = sp.e;
  ep.k_cache = dp.k_cache;
  ep.v_cache = dp.v_cache;
  ep.block_table = block_table;
  ep.seq_lens = seq_lens;
  ep.sink = sink;
  ep.out = dp.out;                         // every tile leaves sums: not written
  ep.lse = lse;
  ep.items = reinterpret_cast<ExtItem*>(ws + L.off_items);
  ep.ml_part = reinterpret_cast<float2*>(ws + L.off_ml);
  ep.o_part = reinterpret_cast<float*>(ws + L.off_o);
  ep.err = err;
  ep.batch = ep.total_q = params->batch;
  ep.heads_q = params->heads_q;
  ep.heads_kv = params->heads_kv;
  ep.group = params->heads_q / params->heads_kv;
  ep.tokens = L.tokens;
  ep.page_size = params->page_size;
  ep.num_pages = params->num_pages;
  ep.max_pages = params->max_pages;
  ep.n_items = L.n_items;
  ep.slots = L.slots;
  ep.scale_log2 = dp.scale_log2;
#ifdef ATTN_SINK_TEST_HOOKS
  ep.skip_k_tile = g_test_skip_k_tile.load();
#endif
  const long long rows = (long long)params->num_pages * params->page_size;
  const bool tma = params->page_size % 8 == 0 && rows > 0 && rows < (1ll << 31);
  ep.box = tma ? std::min(params->page_size & -params->page_size, kBlockN) : 0;
  if ((st = encode_rows(&ep.tm_q, q, params->batch, params->heads_q,
                        CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L.tokens, ep.group)) != ATTN_SINK_OK)
    return st;
  ep.tm_out = ep.tm_q;                     // unused
  if (tma &&
      ((st = encode_rows(&ep.tm_k, k_cache, rows, params->heads_kv,
                         CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ep.box)) != ATTN_SINK_OK ||
       (st = encode_rows(&ep.tm_v, v_cache, rows, params->heads_kv,
                         CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ep.box)) != ATTN_SINK_OK))
    return st;
  sp.cu_groups = cu_groups;
  sp.prefix_lens = prefix_lens;
  sp.num_groups = params->num_groups;
  sp.refs = reinterpret_cast<SharedRef*>(ws + L.off_refs);
  attn_sink_shared_plan_kernel<<<1, 32 * kSharedWarps, 0, s>>>(sp);
  if (!launched()) return ATTN_SINK_ERR_CUDA;
  const auto tiles = prefix_kernel(tma);
  if (!launch_dependent(tiles, (unsigned)L.n_items * (unsigned)params->heads_kv, kExtThreads,
                        kFwdSmemBytes, s, ep))
    return ATTN_SINK_ERR_CUDA;
  const dim3 grid(L.own.splits, params->heads_kv, params->batch);
  return launch_dependent(slice_kernel<true>(ep.group, dec_tma), grid, kSliceThreads,
                          kSliceSmem, s, dp) &&
                 (dp.whole || launch_join<true>(dp, s))
             ? ATTN_SINK_OK
             : ATTN_SINK_ERR_CUDA;
}

int attn_sink_page_bounds(const attn_sink_bounds_params* params, const void* k_cache,
                          const int* block_table, const int* cached_lens, const int* seq_lens,
                          void* bounds, void* stream) {
  NvtxRange range("attn_sink_page_bounds");
  int st = cache_validate(params, 1 << 24);
  if (st != ATTN_SINK_OK) return st;
  if (params->batch == 0) return ATTN_SINK_OK;
  if (cached_lens == nullptr || seq_lens == nullptr ||
      (params->max_pages > 0 && block_table == nullptr) ||
      (params->num_pages > 0 && (k_cache == nullptr || bounds == nullptr)) ||
      !aligned16(k_cache) || !aligned16(bounds))
    return ATTN_SINK_ERR_INVALID_ARG;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  BoundsParams bp;
  bp.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  bp.block_table = block_table;
  bp.cached = cached_lens;
  bp.seq_lens = seq_lens;
  bp.bounds = static_cast<__nv_bfloat16*>(bounds);
  bp.err = err;
  bp.batch = params->batch;
  bp.heads_kv = params->heads_kv;
  bp.page_size = params->page_size;
  bp.num_pages = params->num_pages;
  bp.max_pages = params->max_pages;
  // about eight CTAs an SM, over the sequences and the pages of each
  const int y = std::min(params->batch, 8 * sms);
  const long long warps = (long long)params->max_pages * ((params->heads_kv + 3) / 4);
  const long long x = std::min<long long>((warps + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32),
                                          std::max(1, 8 * sms / y));
  attn_sink_page_bounds_kernel<<<dim3((unsigned)std::max(x, 1ll), y), kBoundsThreads, 0,
                                 static_cast<cudaStream_t>(stream)>>>(bp);
  return launched() ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
}

size_t attn_sink_select_pages_workspace_size(const attn_sink_select_params* params) {
  SelectLayout L;
  if (select_layout(params, &L) != ATTN_SINK_OK || params->batch == 0) return 0;
  return std::max<size_t>(L.total, 256);
}

int attn_sink_select_pages(const attn_sink_select_params* params, const void* q,
                           const void* bounds, const int* block_table, const int* seq_lens,
                           int* selected, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("attn_sink_select_pages");
  SelectLayout L;
  int st = select_layout(params, &L);
  if (st != ATTN_SINK_OK) return st;
  if (params->batch == 0) return ATTN_SINK_OK;
  if (q == nullptr || seq_lens == nullptr || selected == nullptr ||
      (params->max_pages > 0 && block_table == nullptr) ||
      (params->num_pages > 0 && bounds == nullptr) || !aligned16(q) || !aligned16(bounds))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, std::max<size_t>(L.total, 256)))
    return ATTN_SINK_ERR_WORKSPACE;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  if ((st = cache_attributes()) != ATTN_SINK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SelectParams sp;
  sp.q = static_cast<const __nv_bfloat16*>(q);
  sp.bounds = static_cast<const __nv_bfloat16*>(bounds);
  sp.block_table = block_table;
  sp.seq_lens = seq_lens;
  sp.scores = reinterpret_cast<float*>(ws);
  sp.peak = reinterpret_cast<unsigned*>(ws + L.off_peak);
  sp.exact = reinterpret_cast<unsigned long long*>(ws + L.off_exact);
  sp.selected = selected;
  sp.err = err;
  sp.batch = params->batch;
  sp.heads_q = params->heads_q;
  sp.heads_kv = params->heads_kv;
  sp.group = params->heads_q / params->heads_kv;
  sp.page_size = params->page_size;
  sp.num_pages = params->num_pages;
  sp.max_pages = params->max_pages;
  sp.tiles = L.tiles;
  sp.count = params->count;
  sp.keep_first = params->keep_first;
  sp.keep_last = params->keep_last;
  // a warp for each (16 pages, kv head), up to 8 CTAs an SM over all sequences
  constexpr int kWarps = kScoreThreads / 32;
  const long long warps = (long long)std::max(1, L.tiles) * params->heads_kv;
  const long long least = (params->heads_kv + kWarps - 1) / kWarps;      // a warp a head
  const long long x = std::max(least, std::min((warps + kWarps - 1) / kWarps,
                                               8ll * sms / params->batch));
  if (x >= (1ll << 31)) return ATTN_SINK_ERR_UNSUPPORTED;
  attn_sink_page_scores_kernel<<<dim3((unsigned)x, params->batch), kScoreThreads, kScoreSmem, s>>>(
      sp);
  if (!launched()) return ATTN_SINK_ERR_CUDA;
  const int threads = row_threads(params->max_pages);
  const size_t smem = 4 * (size_t)std::min(std::max(params->max_pages, 1), kSelectStage);
  const unsigned rows = (unsigned)params->batch * (unsigned)params->heads_kv;
  return launch_dependent(select_kernel(threads), rows, threads, smem, s, sp)
             ? ATTN_SINK_OK
             : ATTN_SINK_ERR_CUDA;
}

namespace {

int pages_layout(const attn_sink_pages_params* p, int sms, DecodeSlices* L) {
  int st = cache_validate(p, 65535);
  if (st != ATTN_SINK_OK || (st = group_validate(p)) != ATTN_SINK_OK) return st;
  if (!scale_ok(p->softmax_scale) || p->count < 0 ||
      (long long)p->count * p->page_size > (1ll << 30))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (p->heads_kv > 65535) return ATTN_SINK_ERR_UNSUPPORTED;
  const long long keys = (long long)std::min(p->count, p->max_pages) * p->page_size;
  *L = decode_slices(decode_splits(p->batch, p->heads_kv, keys, kSliceThreads, sms), p->batch,
                     p->heads_q);
  return ATTN_SINK_OK;
}

}  // namespace

size_t attn_sink_decode_pages_workspace_size(const attn_sink_pages_params* params) {
  DecodeSlices L;
  if (pages_layout(params, sm_count_or_default(), &L) != ATTN_SINK_OK || params->batch == 0)
    return 0;
  return L.total;
}

int attn_sink_decode_pages(const attn_sink_pages_params* params, const void* q,
                           const void* k_cache, const void* v_cache, const int* block_table,
                           const int* seq_lens, const int* selected, const float* sink, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("attn_sink_decode_pages");
  DecodeSlices L;
  int st = pages_layout(params, sm_count_or_default(), &L);
  if (st != ATTN_SINK_OK) return st;
  if (params->batch == 0) return ATTN_SINK_OK;
  if (q == nullptr || sink == nullptr || out == nullptr || lse == nullptr ||
      seq_lens == nullptr || (params->max_pages > 0 && block_table == nullptr) ||
      (params->count > 0 && selected == nullptr) ||
      (params->num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, L.total)) return ATTN_SINK_ERR_WORKSPACE;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  if ((st = cache_attributes()) != ATTN_SINK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SliceParams dp;
  bool tma;
  if ((st = decode_params(params, L, q, k_cache, v_cache, block_table, seq_lens, sink, out, lse,
                          static_cast<uint8_t*>(workspace), err, true, &dp, &tma)) != ATTN_SINK_OK)
    return st;
  dp.selected = selected;
  dp.count = params->count;
  const dim3 grid(L.splits, params->heads_kv, params->batch);
  slice_kernel<false>(params->heads_q / params->heads_kv, tma)<<<grid, kSliceThreads, kSliceSmem, s>>>(dp);
  if (!launched()) return ATTN_SINK_ERR_CUDA;
  return L.splits == 1 || launch_join<false>(dp, s) ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
}

int attn_sink_key_mass(const attn_sink_mass_params* params, const void* q, const void* k_cache,
                       const int* block_table, const int* seq_lens, const int* cu_seqlens_q,
                       const float* lse, float* mass, void* stream) {
  NvtxRange range("attn_sink_key_mass");
  int st = cache_validate(params, 65535);
  if (st != ATTN_SINK_OK) return st;
  if (params->heads_q < 1 || params->heads_q % params->heads_kv != 0 || params->total_q < 0 ||
      params->max_keys < 0 || (params->accumulate != 0 && params->accumulate != 1) ||
      !scale_ok(params->softmax_scale))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (params->heads_q / params->heads_kv > 128 || params->heads_kv > 65535 ||
      params->total_q > (1 << 30) || params->max_keys > (1 << 30))
    return ATTN_SINK_ERR_UNSUPPORTED;
  if (params->batch == 0 || params->max_keys == 0) return ATTN_SINK_OK;
  if (seq_lens == nullptr || cu_seqlens_q == nullptr || mass == nullptr ||
      (params->total_q > 0 && (q == nullptr || lse == nullptr)) ||
      (params->max_pages > 0 && block_table == nullptr) ||
      (params->num_pages > 0 && k_cache == nullptr) || !aligned16(q) || !aligned16(k_cache))
    return ATTN_SINK_ERR_INVALID_ARG;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  if ((st = cache_attributes()) != ATTN_SINK_OK) return st;
  MassParams mp;
  std::memset(&mp, 0, sizeof(mp));
  mp.q = static_cast<const __nv_bfloat16*>(q);
  mp.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  mp.block_table = block_table;
  mp.seq_lens = seq_lens;
  mp.cu_q = cu_seqlens_q;
  mp.lse = lse;
  mp.mass = mass;
  mp.err = err;
  mp.batch = params->batch;
  mp.total_q = params->total_q;
  mp.heads_q = params->heads_q;
  mp.heads_kv = params->heads_kv;
  mp.group = params->heads_q / params->heads_kv;
  mp.page_size = params->page_size;
  mp.num_pages = params->num_pages;
  mp.max_pages = params->max_pages;
  mp.max_keys = params->max_keys;
  mp.accumulate = params->accumulate;
  mp.scale_log2 = params->softmax_scale * kLog2e;
  mp.inv_scale = 1.0f / params->softmax_scale;
#ifdef ATTN_SINK_TEST_HOOKS
  mp.skip_k_tile = g_test_skip_k_tile.load();
#endif
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long rows = (long long)params->total_q * mp.group;
  if (rows > (long long)kMassFewRows * params->batch && mp.group <= kMassMaxGroup &&
      params->softmax_scale >= kMassLeastScale && params->softmax_scale <= kMassMostScale) {
    mp.tokens = kMassRows / mp.group;
    if ((st = encode_rows(&mp.tm_q, q, params->total_q, params->heads_q,
                          CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mp.tokens, mp.group)) != ATTN_SINK_OK)
      return st;
    const dim3 grid((params->max_keys + kMassKeys - 1) / kMassKeys, params->heads_kv, params->batch);
    attn_sink_key_mass_kernel<<<grid, kMassThreads, kMassSmemBytes, s>>>(mp);
    return launched() ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
  }
  // a warp for each (32 keys, kv head), up to two rounds of the CTAs that fit at once (32 x 8192
  // keys: one 43.6 us, two 42.6, three 44.2)
  constexpr int kWarps = kMassFewThreads / 32;
  const long long warps = (params->max_keys + 31ll) / 32 * params->heads_kv;
  const long long least = (params->heads_kv + kWarps - 1) / kWarps;      // a warp a head
  const long long x = std::max(least, std::min((warps + kWarps - 1) / kWarps,
                                               4ll * sms / params->batch));
  const dim3 grid((unsigned)x, params->batch);
  if (rows <= 8ll * params->batch)
    attn_sink_key_mass_few_kernel<1><<<grid, kMassFewThreads, kMassFewSmem, s>>>(mp);
  else
    attn_sink_key_mass_few_kernel<4><<<grid, kMassFewThreads, kMassFewSmem, s>>>(mp);
  return launched() ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
}

size_t attn_sink_evict_workspace_size(const attn_sink_evict_params* params) {
  EvictLayout L;
  if (evict_layout(params, &L) != ATTN_SINK_OK || params->batch == 0) return 0;
  return L.total;
}

int attn_sink_evict(const attn_sink_evict_params* params, void* k_cache, void* v_cache,
                    const int* block_table, const int* seq_lens, const float* mass,
                    float* mass_out, int* new_lens, int* freed_pages, int* num_freed,
                    void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("attn_sink_evict");
  EvictLayout L;
  int st = evict_layout(params, &L);
  if (st != ATTN_SINK_OK) return st;
  if (num_freed == nullptr || (params->max_freed > 0 && freed_pages == nullptr))
    return ATTN_SINK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->batch == 0) {
    // no sequence: no page is freed
    if (cudaMemsetAsync(num_freed, 0, sizeof(int), s) != cudaSuccess ||
        (params->max_freed > 0 &&
         cudaMemsetAsync(freed_pages, 0xFF, (size_t)params->max_freed * sizeof(int), s) !=
             cudaSuccess))
      return ATTN_SINK_ERR_CUDA;
    return ATTN_SINK_OK;
  }
  if (seq_lens == nullptr || new_lens == nullptr || seq_lens == new_lens ||
      (params->max_keys > 0 && (mass == nullptr || mass_out == nullptr || mass == mass_out)) ||
      (params->max_pages > 0 && block_table == nullptr) ||
      (params->num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, L.total)) return ATTN_SINK_ERR_WORKSPACE;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  if ((st = cache_attributes()) != ATTN_SINK_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  EvictParams ep;
  ep.k_cache = static_cast<uint4*>(k_cache);
  ep.v_cache = static_cast<uint4*>(v_cache);
  ep.block_table = block_table;
  ep.seq_lens = seq_lens;
  ep.mass = mass;
  ep.mass_out = mass_out;
  ep.new_lens = new_lens;
  ep.freed = freed_pages;
  ep.num_freed = num_freed;
  ep.counts = reinterpret_cast<int*>(ws);
  ep.to = reinterpret_cast<int*>(ws + L.off_moves);
  ep.from = reinterpret_cast<int*>(ws + L.off_from);
  ep.err = err;
  ep.batch = params->batch;
  ep.heads_kv = params->heads_kv;
  ep.page_size = params->page_size;
  ep.num_pages = params->num_pages;
  ep.max_pages = params->max_pages;
  ep.max_keys = params->max_keys;
  ep.budget = params->budget;
  ep.keep_first = params->keep_first;
  ep.keep_last = params->keep_last;
  ep.max_freed = params->max_freed;
  ep.max_moves = L.max_moves;
  ep.stage = std::min(params->max_keys, kEvictStage);
  const unsigned rows = (unsigned)params->batch * (unsigned)params->heads_kv;
  const size_t lists = 8 * (size_t)L.max_moves;
  size_t smem = 4 * (size_t)std::max(ep.stage, 1);
  const int threads = row_threads(params->max_keys);
  ep.here = rows >= (unsigned)sms;         // enough CTAs to move the rows themselves
  ep.lists = ep.here && smem + lists <= kEvictLists;
  if (ep.lists) smem += lists;
  evict_kernel(threads)<<<rows + 1, threads, smem, s>>>(ep);
  if (!launched()) return ATTN_SINK_ERR_CUDA;
  if (ep.here) return ATTN_SINK_OK;
  // about eight CTAs an SM, over the rows and the moves of each, 64 a CTA at a time
  const unsigned y = std::min(rows, 8u * (unsigned)sms);
  const unsigned x = (unsigned)std::max(
      1, std::min((L.max_moves + 63) / 64, (int)(8u * (unsigned)sms / y)));
  return launch_dependent(attn_sink_evict_move_kernel, dim3(x, y), kMoveThreads, 0, s, ep)
             ? ATTN_SINK_OK
             : ATTN_SINK_ERR_CUDA;
}

}  // extern "C"
