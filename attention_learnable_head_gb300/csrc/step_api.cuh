// Host side of attn_sink_step.h: validation, tensor maps, workspace carving and
// launches.  Included by attn_sink_api.cu after attn_sink.h's own entry points:
// one translation unit, so that both share the device error word, the launch
// counter and the per-device state.
#pragma once

namespace {

// A launch that may begin while the kernel before it in the stream runs (the
// kernel waits for it itself: grid_dependency_wait).
template <typename P>
bool launch_dependent(void (*kernel)(P), dim3 grid, unsigned threads, size_t smem,
                      cudaStream_t s, const P& params) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
  if (e != cudaSuccess) {
    cudaGetLastError();
    g_last_cuda_error.store((int)e, std::memory_order_relaxed);
    return false;
  }
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return true;
}

// ----------------------------------------------------------------------------- plan
// Tokens a CTA of the plan writes; more CTAs per group only repeat the sums.
constexpr int kPlanTokensPerCta = 4 * kPlanThreads;
// From this many sequences on a kernel of its own sums the lengths before each group
// (and a group has one CTA, as it has by then anyway).  Device time with the CTAs' own
// sums and with that kernel: 32768 sequences of up to 1 token 44 and 27 us, of up to 40
// 120 and 185; 65536 86 and 50, 350 and 353; 131072 184 and 91, 838 and 658.
constexpr int kPlanSummed = 1 << 16;

// ----------------------------------------------------------------------------- rope
int rope_validate(const attn_sink_rope_params* p) {
  if (p == nullptr) return ATTN_SINK_ERR_INVALID_ARG;
  if (p->head_dim != kHeadDim) return ATTN_SINK_ERR_UNSUPPORTED;
  if (p->tokens < 0 || p->heads_q < 1 || p->heads_kv < 1 ||
      p->heads_q > (1 << 20) || p->heads_kv > (1 << 20))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (p->rotary_dim < 0 || p->rotary_dim > kHeadDim) return ATTN_SINK_ERR_INVALID_ARG;
  if (p->rotary_dim % 16 != 0) return ATTN_SINK_ERR_UNSUPPORTED;
  if ((p->interleaved | p->norm | p->weight_bf16) & ~1) return ATTN_SINK_ERR_INVALID_ARG;
  if (p->num_axes < 1 || p->num_axes > ATTN_SINK_ROPE_MAX_AXES) return ATTN_SINK_ERR_INVALID_ARG;
  for (int i = 0; i < p->rotary_dim / 2; ++i)
    if (p->pair_axis[i] >= p->num_axes) return ATTN_SINK_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.0f || !std::isfinite(p->amplitude))
    return ATTN_SINK_ERR_INVALID_ARG;
  return ATTN_SINK_OK;
}

// A token stride: whole 16-byte chunks, heads that do not overlap.
bool rope_stride_ok(long long stride, int heads) {
  return stride % 8 == 0 && stride >= (long long)heads * kHeadDim && stride < (1ll << 40);
}

// The grid: x CTAs, over whose warps the tokens go round, by the parts that a
// token's heads are cut into.  One part where the tokens fill the GPU (a token's
// angles are computed once); with fewer tokens the heads are spread over more
// warps, four heads at the least each.
dim3 rope_grid(const attn_sink_rope_params* p, int sms, int ctas_per_sm) {
  const long long ctas = (long long)sms * ctas_per_sm;
  const long long most = std::min((p->heads_q + 3) / 4, 65535);
  const long long parts =
      std::max<long long>(1, std::min(ctas * kRopeWarps / std::max(1, p->tokens), most));
  const long long x = std::min<long long>(((long long)p->tokens + kRopeWarps - 1) / kRopeWarps,
                                          std::max<long long>(1, ctas / parts));
  return dim3((unsigned)std::max<long long>(1, x), (unsigned)parts);
}

RopeParams rope_params(const attn_sink_rope_params* p) {
  RopeParams rp;
  std::memset(&rp, 0, sizeof(rp));
  rp.q_stride = p->q_stride;
  rp.k_stride = p->k_stride;
  rp.v_stride = p->v_stride;
  rp.tokens = p->tokens;
  rp.heads_q = p->heads_q;
  rp.heads_kv = p->heads_kv;
  rp.rotary = p->rotary_dim;
  rp.weight_bf16 = p->weight_bf16;
  rp.eps = p->eps;
  rp.amplitude = p->amplitude;
  std::memcpy(rp.pair_axis, p->pair_axis, sizeof(rp.pair_axis));
  return rp;
}

// Heads of q, k and v that a warp takes of a token at most (rope_share).
long long rope_most(const attn_sink_rope_params* p, int parts) {
  if (parts == 1) return p->heads_q + 2ll * p->heads_kv;
  auto share = [&](int heads) { return 4ll * (((heads + 3) / 4 + parts - 1) / parts); };
  return share(p->heads_q) + 2 * share(p->heads_kv);
}

template <bool kNorm, bool kInter>
void rope_launch(const RopeParams& rp, dim3 grid, bool whole, cudaStream_t s) {
  if (whole)
    attn_sink_rope_kernel<kNorm, kInter, true><<<grid, kRopeThreads, 0, s>>>(rp);
  else
    attn_sink_rope_kernel<kNorm, kInter, false><<<grid, kRopeThreads, 0, s>>>(rp);
}

template <bool kNorm, bool kInter>
void rope_bwd_launch(const RopeParams& rp, dim3 grid, bool fp32, bool whole, cudaStream_t s) {
  if (fp32 && whole)
    attn_sink_rope_bwd_kernel<kNorm, kInter, true, true><<<grid, kRopeThreads, 0, s>>>(rp);
  else if (fp32)
    attn_sink_rope_bwd_kernel<kNorm, kInter, true, false><<<grid, kRopeThreads, 0, s>>>(rp);
  else if (whole)
    attn_sink_rope_bwd_kernel<kNorm, kInter, false, true><<<grid, kRopeThreads, 0, s>>>(rp);
  else
    attn_sink_rope_bwd_kernel<kNorm, kInter, false, false><<<grid, kRopeThreads, 0, s>>>(rp);
}

// ----------------------------------------------------------------------------- extend
struct ExtendLayout {
  int tokens;        // per tile
  int n_items, max_parts, max_tiles, slots;
  bool split;                              // tiles may be cut: a join
  bool find;                               // no schedule: see ext_find
  size_t off_tiles, off_ml, off_o, total;
  // the band kernel's path (extend_window.cuh)
  int band_cols;     // 0: not taken
  long long band_rows;
  size_t off_regions, off_k, off_v, off_lost;   // off_lost: GatherParams::any_lost
};

// Windows go to the band kernel where one product covers a tile's keys (as in the
// forward), the tiles are more than the GPU holds at once or have no single launch
// (ext_find), and the sequences have enough new tokens: kExtBandTokens on average,
// below which the workspace (176 + W rows of K and V for each) is out of
// proportion; two full tiles with two heads a group, where gathering costs as much
// as it saves (with one it always did).  Device time of the band kernel's and of
// the general way behind 1024 cached keys, W = 128, 64 + 8 heads: 8 x 513 tokens 34
// and 69 us, 140 x 200 197 and 443, 32 x 64 26 and 39, 128 x 8 39.5 and 39.3, 8 x 64
// 13.4 and 12.6, 32 x 16 15.3 and 13.1, 1 x 256 (not taken) 10.8 and 9.7; 8 + 1 heads,
// 64 x 8 (not taken) 11.8 and 9.9; W = 100, 16 + 8 heads: 128 x 64 (not taken) 55 and
// 44, 128 x 200 120 and 135.
constexpr int kExtBandTokens = 8;

// Tiles that see few blocks of keys are left whole: cutting them costs a schedule, a
// join and the parts' sums on their way through memory, 8 us at the least.  Few or
// many blocks, whether there are kExtWholeCtas tiles x kv heads.  Device time whole
// and cut: 1 x 1 token (8 CTAs) on 900 keys 15 and 18 us, on 1200 16.5 and 16.8, on
// 2400 26 and 17.5; 8 x 1 (64 CTAs) on 1800 22.4 and 22.1, on 2400 26 and 22.5; 1 x
// 256 (128 CTAs) on 2400 27 and 39; 32 x 1 (256 CTAs) on 2400 31 and 41; 32 x 256
// (4096 CTAs) on 2400 258 and 264.  Keys copied one by one take twice as long, so
// half as many blocks: 1 x 2 tokens on 1100 keys in pages of one 26.5 whole, 19.9 cut.
//
// Then a CTA finds its tile by itself, in a single launch, unless it is one of many:
// the search costs each 1 us, the schedule kernel a call 4.  Found and listed, 8
// sequences of 120 new tokens (40 + 8 heads, 264 CTAs) 10.5 and 13 us, 32 x 64 (648)
// 22 and 23.4, 8 x 500 on 512 keys (1048) 41.8 and 40, 32 x 500 (3976) 139 and 127.
constexpr int kExtFindRounds = 3;  // CTAs, in what the GPU holds at once
constexpr int kExtWholeCtas = 100;
constexpr int kExtWholeFew = 10;
constexpr int kExtWholeMany = 20;

constexpr int kExtCtasPerSm = 2;   // shared memory, TMEM and registers allow two

int extend_layout(const attn_sink_extend_params* p, int sms, ExtendLayout* L) {
  if (p == nullptr) return ATTN_SINK_ERR_INVALID_ARG;
  if (p->head_dim != kHeadDim) return ATTN_SINK_ERR_UNSUPPORTED;
  if (p->batch < 0 || p->total_q < 0 || p->heads_kv < 1 || p->heads_q < 1 ||
      p->heads_q % p->heads_kv != 0 || p->page_size < 1 || p->num_pages < 0 ||
      p->max_pages < 0 || !(p->softmax_scale > 0.0f) || !std::isfinite(p->softmax_scale))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (p->batch > (1 << 24) || p->total_q > (1 << 30)) return ATTN_SINK_ERR_UNSUPPORTED;
  if ((long long)p->max_pages * p->page_size > (1ll << 30)) return ATTN_SINK_ERR_INVALID_ARG;
  // rows of the cache of one head, 128 bytes each: 512 GB
  if ((long long)p->num_pages * p->page_size > ((1ll << 32) - 1) / p->heads_kv)
    return ATTN_SINK_ERR_UNSUPPORTED;
  const int group = p->heads_q / p->heads_kv;
  if (group > kExtMaxGroup) return ATTN_SINK_ERR_UNSUPPORTED;
  L->tokens = kBlockM / group;
  L->slots = kExtCtasPerSm * sms;
  const long long shares = (3 * L->slots + p->heads_kv - 1) / p->heads_kv;
  // Blocks of keys that a tile sees at most, as the table is no wider or the window
  // touches no more; whether the tiles are cut.
  const long long span_tiles = p->total_q / L->tokens + (long long)p->batch;
  const long long most =
      std::min(((long long)p->max_pages * p->page_size + kBlockN - 1) / kBlockN,
               p->window > 0 ? ((long long)p->window + L->tokens + kBlockN - 3) / kBlockN + 1
                             : LLONG_MAX);
  const int few = p->page_size % 8 == 0 ? kExtWholeFew : kExtWholeFew / 2;   // key by key
  L->split = most > (span_tiles * p->heads_kv < kExtWholeCtas ? few : kExtWholeMany);
  L->find = !L->split && p->batch <= kExtFindMax &&
            span_tiles * p->heads_kv <= kExtFindRounds * (long long)L->slots;
  // the bounds of attn_sink_extend_plan_kernel
  const long long items = span_tiles + (L->split ? shares : 0);
  if (items * p->heads_kv >= (1ll << 31)) return ATTN_SINK_ERR_UNSUPPORTED;   // launch grid
  L->n_items = (int)items;
  L->max_parts = L->split ? (int)std::min<long long>(items, 2 * shares) : 0;
  L->max_tiles = L->max_parts / 2;         // two parts at least
  const size_t parts = (size_t)L->max_parts * p->heads_kv;
  size_t off = align256((size_t)L->n_items * sizeof(ExtItem));
  L->off_tiles = off;                      // their number, then the tiles
  off += 256 + align256((size_t)L->max_tiles * sizeof(ExtTileRef));
  L->off_ml = off;
  off += align256(parts * kBlockM * sizeof(float2));
  L->off_o = off;
  off += align256(parts * kBlockM * kHeadDim * sizeof(float));
  L->total = off;
  L->band_cols = 0;
  const long long enough = group == 2 ? 2 * L->tokens : kExtBandTokens;
  if (p->window > 0 && group > 1 && kBlockM % group == 0 &&
      (long long)L->tokens + p->window - 1 <= kBandMaxCols &&
      (p->batch > kExtFindMax || span_tiles * p->heads_kv > L->slots) &&
      p->total_q >= enough * p->batch) {
    L->band_rows = p->total_q + (long long)p->batch * (p->window - 1 + kGatherPad) + kGatherPad;
    if (L->band_rows < (1ll << 30) && span_tiles * p->heads_kv < (1ll << 30)) {
      L->band_cols = (L->tokens + p->window - 1 + 15) / 16 * 16;
      L->n_items = (int)span_tiles;        // tiles that are listed
      const size_t kv = align256((size_t)L->band_rows * p->heads_kv * kHeadDim * 2);
      off = align256((size_t)span_tiles * sizeof(int4));
      L->off_regions = off;
      off += align256((size_t)p->batch * sizeof(GatherRegion));
      L->off_k = off;
      off += kv;
      L->off_v = off;
      off += kv;
      L->off_lost = off;
      L->total = off + 256;
    }
  }
  return ATTN_SINK_OK;
}

bool g_ext_attr_set[kMaxDevices] = {false};

// The extend kernels' shared memory limit, once per device.
int extend_attributes() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return ATTN_SINK_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  if (!g_ext_attr_set[dev]) {
    if (cudaFuncSetAttribute(attn_sink_extend_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kFwdSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(attn_sink_extend_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kFwdSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(attn_sink_fwd_band_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kBandSmemMax) != cudaSuccess)
      return ATTN_SINK_ERR_CUDA;
    g_ext_attr_set[dev] = true;
  }
  return ATTN_SINK_OK;
}

// The windowed path: gather, then the band kernel with every tile a sequence.
int extend_window(const attn_sink_extend_params* p, const ExtendLayout& L, const ExtParams& ep,
                  const void* q, void* out, uint8_t* ws, int sms, cudaStream_t s) {
  GatherParams gp;
  gp.e = ep;
  gp.spans = reinterpret_cast<int4*>(ws);
  gp.regions = reinterpret_cast<GatherRegion*>(ws + L.off_regions);
  gp.k = reinterpret_cast<__nv_bfloat16*>(ws + L.off_k);
  gp.v = reinterpret_cast<uint16_t*>(ws + L.off_v);
  gp.any_lost = reinterpret_cast<int*>(ws + L.off_lost);
  gp.max_tiles = L.n_items;
  gp.rows = L.band_rows;
  FwdBandParams bp;
  std::memset(&bp, 0, sizeof(bp));
  int st;
  if ((st = encode_rows(&bp.tm_q, q, p->total_q, p->heads_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        L.tokens, ep.group)) != ATTN_SINK_OK ||
      (st = encode_rows(&bp.tm_k, gp.k, L.band_rows, p->heads_kv,
                        CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L.band_cols)) != ATTN_SINK_OK ||
      (st = encode_rows(&bp.tm_v, gp.v, L.band_rows, p->heads_kv,
                        CU_TENSOR_MAP_DATA_TYPE_FLOAT16, L.tokens + p->window - 1)) !=
          ATTN_SINK_OK ||
      (st = encode_rows(&bp.tm_out, out, p->total_q, p->heads_q,
                        CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L.tokens, ep.group)) != ATTN_SINK_OK)
    return st;
  bp.tm_out_lo = bp.tm_out;                // unused without a residual
  bp.spans = gp.spans;
  bp.any_lost = gp.any_lost;
  bp.regions = reinterpret_cast<const int4*>(gp.regions);
  bp.block_table = ep.block_table;
  bp.page_size = p->page_size;
  bp.num_pages = p->num_pages;
  bp.max_pages = p->max_pages;
  bp.sink = ep.sink;
  bp.out = ep.out;
  bp.lse = ep.lse;
  bp.err = ep.err;
  bp.total_q = p->total_q;
  bp.heads_q = p->heads_q;
  bp.heads_kv = p->heads_kv;
  bp.group = ep.group;
  while ((1 << bp.log2_group) < ep.group) ++bp.log2_group;
  bp.tokens = L.tokens;
  bp.n_cols = L.band_cols;
  bp.half0_cols = 16 * ((L.band_cols / 16 + 1) / 2);
  bp.window = p->window;
  bp.scale_log2 = ep.scale_log2;
  bp.n_tb = 1;
  bp.n_items = L.n_items * p->heads_kv;
  fast_div_init(p->heads_kv, &bp.div_hkv_mul, &bp.div_hkv_shift);
  fast_div_init(bp.n_tb, &bp.div_tb_mul, &bp.div_tb_shift);
#ifdef ATTN_SINK_TEST_HOOKS
  bp.skip_k_tile = g_test_skip_k_tile.load();
#endif
  attn_sink_gather_plan_kernel<<<1, kExtSchedThreads, 0, s>>>(gp);
  if (!launched()) return ATTN_SINK_ERR_CUDA;
  // about eight CTAs an SM, over the sequences and the rows of each
  const int y = std::min(p->batch, 8 * sms), x = std::max(1, 8 * sms / y);
  if (!launch_dependent(attn_sink_gather_kernel, dim3(x, y), kGatherThreads, 0, s, gp))
    return ATTN_SINK_ERR_CUDA;
  const int smem = std::max(80 * 1024, band_smem_bytes(L.band_cols));   // two CTAs an SM
  const int grid = (int)std::min<long long>(bp.n_items, (long long)kBandCtasPerSm * sms);
  return launch_dependent(attn_sink_fwd_band_kernel<true>, grid, kBandThreads, smem, s, bp)
             ? ATTN_SINK_OK
             : ATTN_SINK_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_sink_page_plan(const attn_sink_plan_params* params, const int* cached_lens,
                        const int* new_lens, const int* free_pages, int* block_table,
                        long long* slots, int* positions, int* cu_seqlens, int* seq_lens,
                        int* pages_needed, void* stream) {
  NvtxRange range("attn_sink_page_plan");
  if (params == nullptr || params->batch < 0 || params->page_size < 1 || params->num_pages < 0 ||
      params->max_pages < 0 || params->num_free < 0 || params->max_tokens < 0 ||
      (long long)params->max_pages * params->page_size > (1ll << 30))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (params->batch > (1 << 24)) return ATTN_SINK_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr || pages_needed == nullptr ||
      (params->batch > 0 &&
       (cached_lens == nullptr || new_lens == nullptr || seq_lens == nullptr)) ||
      (params->batch > 0 && params->max_pages > 0 && block_table == nullptr) ||
      (params->num_free > 0 && free_pages == nullptr) ||
      (params->max_tokens > 0 && (slots == nullptr || positions == nullptr)))
    return ATTN_SINK_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return ATTN_SINK_ERR_INVALID_ARG;
  // CTAs read the lengths while others write seq_lens
  if (params->batch > 0 && (seq_lens == cached_lens || seq_lens == new_lens))
    return ATTN_SINK_ERR_INVALID_ARG;
  int sms = 0;
  int* err = nullptr;
  int st;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  PlanParams pp;
  pp.cached = cached_lens;
  pp.fresh = new_lens;
  pp.free_pages = free_pages;
  pp.table = block_table;
  pp.slots = slots;
  pp.positions = positions;
  pp.cu = cu_seqlens;
  pp.lens = seq_lens;
  pp.needed = pages_needed;
  pp.err = err;
  pp.batch = params->batch;
  pp.page_size = params->page_size;
  pp.num_pages = params->num_pages;
  pp.max_pages = params->max_pages;
  pp.num_free = params->num_free;
  pp.max_tokens = params->max_tokens;
  // groups of sequences x blocks of a group's tokens, two CTAs per SM at most
  const int groups = std::max(1, (params->batch + kPlanSeqs - 1) / kPlanSeqs);
  const long long per_group = ((long long)params->max_tokens + groups - 1) / groups;
  const long long blocks = (per_group + kPlanTokensPerCta - 1) / kPlanTokensPerCta;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  pp.summed = params->batch >= kPlanSummed;
  const int y = pp.summed ? 1 : (int)std::max<long long>(
      1, std::min<long long>(blocks, std::max(1, 2 * sms / groups)));
  if (pp.summed) {
    attn_sink_plan_sum_kernel<<<1, kPlanSumThreads, 0, s>>>(pp);
    if (!launched()) return ATTN_SINK_ERR_CUDA;
  }
  attn_sink_plan_kernel<<<dim3(groups, y), kPlanThreads, 0, s>>>(pp);
  return launched() ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
}

int attn_sink_qkv_rope(const attn_sink_rope_params* params, const void* q, const void* k,
                       const void* v, const int* positions, const float* inv_freq,
                       const void* q_weight, const void* k_weight, const long long* slots,
                       void* q_out, void* k_out, void* v_out, void* k_cache, void* v_cache,
                       void* stream) {
  NvtxRange range("attn_sink_qkv_rope");
  int st = rope_validate(params);
  if (st != ATTN_SINK_OK) return st;
  if (!rope_stride_ok(params->q_stride, params->heads_q) ||
      !rope_stride_ok(params->k_stride, params->heads_kv) ||
      !rope_stride_ok(params->v_stride, params->heads_kv))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (slots != nullptr && (params->page_size < 1 || params->num_pages < 0))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (params->tokens == 0) return ATTN_SINK_OK;
  const bool to_cache = slots != nullptr && params->num_pages > 0;
  if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr ||
      (params->rotary_dim > 0 && (positions == nullptr || inv_freq == nullptr)) ||
      (params->norm && (q_weight == nullptr || k_weight == nullptr)) ||
      (to_cache && (k_cache == nullptr || v_cache == nullptr)))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(k_out) || !aligned16(v_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return ATTN_SINK_ERR_INVALID_ARG;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  RopeParams rp = rope_params(params);
  rp.q = static_cast<const __nv_bfloat16*>(q);
  rp.k = static_cast<const __nv_bfloat16*>(k);
  rp.v = static_cast<const __nv_bfloat16*>(v);
  rp.positions = positions;
  rp.inv_freq = inv_freq;
  rp.q_weight = q_weight;
  rp.k_weight = k_weight;
  rp.slots = slots;
  rp.q_out = static_cast<__nv_bfloat16*>(q_out);
  rp.k_out = static_cast<__nv_bfloat16*>(k_out);
  rp.v_out = static_cast<__nv_bfloat16*>(v_out);
  rp.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  rp.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  rp.cache_rows = slots != nullptr ? (long long)params->num_pages * params->page_size : 0;
  rp.err = err;
  const dim3 g = rope_grid(params, sms, kRopeCtas);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool whole = rope_most(params, (int)g.y) <= kRopeWhole;
  if (params->norm && params->interleaved)
    rope_launch<true, true>(rp, g, whole, s);
  else if (params->norm)
    rope_launch<true, false>(rp, g, whole, s);
  else if (params->interleaved)
    rope_launch<false, true>(rp, g, whole, s);
  else
    rope_launch<false, false>(rp, g, whole, s);
  return launched() ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
}

size_t attn_sink_qkv_rope_bwd_workspace_size(const attn_sink_rope_params* params) {
  if (rope_validate(params) != ATTN_SINK_OK || !params->norm || params->tokens == 0) return 0;
  const dim3 g = rope_grid(params, sm_count_or_default(), kRopeBwdCtas);
  return align256((size_t)g.x * g.y * 2 * kHeadDim * sizeof(float));
}

int attn_sink_qkv_rope_bwd(const attn_sink_rope_params* params, const void* q, const void* k,
                           const int* positions, const float* inv_freq, const void* q_weight,
                           const void* k_weight, const void* dq, const void* dk, const void* dv,
                           void* dq_in, void* dk_in, void* dv_in, long long dq_in_stride,
                           long long dk_in_stride, long long dv_in_stride, float* dq_weight,
                           float* dk_weight, void* workspace, size_t workspace_bytes,
                           void* stream) {
  NvtxRange range("attn_sink_qkv_rope_bwd");
  int st = rope_validate(params);
  if (st != ATTN_SINK_OK) return st;
  if (params->grad_dtype != 0 && params->grad_dtype != 1) return ATTN_SINK_ERR_INVALID_ARG;
  if (!rope_stride_ok(dq_in_stride, params->heads_q) ||
      !rope_stride_ok(dk_in_stride, params->heads_kv) ||
      (dv != nullptr && !rope_stride_ok(dv_in_stride, params->heads_kv)) ||
      (params->norm && (!rope_stride_ok(params->q_stride, params->heads_q) ||
                        !rope_stride_ok(params->k_stride, params->heads_kv))))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (params->norm && (dq_weight == nullptr || dk_weight == nullptr))
    return ATTN_SINK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->tokens == 0) {
    // no token: the weights' gradients are zero
    if (params->norm &&
        (cudaMemsetAsync(dq_weight, 0, kHeadDim * sizeof(float), s) != cudaSuccess ||
         cudaMemsetAsync(dk_weight, 0, kHeadDim * sizeof(float), s) != cudaSuccess))
      return ATTN_SINK_ERR_CUDA;
    return ATTN_SINK_OK;
  }
  if (dq == nullptr || dk == nullptr || dq_in == nullptr || dk_in == nullptr ||
      (dv == nullptr) != (dv_in == nullptr) ||
      (params->rotary_dim > 0 && (positions == nullptr || inv_freq == nullptr)) ||
      (params->norm &&
       (q == nullptr || k == nullptr || q_weight == nullptr || k_weight == nullptr)))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(dq_in) || !aligned16(dk_in) || !aligned16(dv_in))
    return ATTN_SINK_ERR_INVALID_ARG;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  const dim3 g = rope_grid(params, sms, kRopeBwdCtas);
  if (params->norm &&
      (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
       workspace_bytes < align256((size_t)g.x * g.y * 2 * kHeadDim * sizeof(float))))
    return ATTN_SINK_ERR_WORKSPACE;
  RopeParams rp = rope_params(params);
  rp.q = static_cast<const __nv_bfloat16*>(q);
  rp.k = static_cast<const __nv_bfloat16*>(k);
  rp.positions = positions;
  rp.inv_freq = inv_freq;
  rp.q_weight = q_weight;
  rp.k_weight = k_weight;
  rp.dq = dq;
  rp.dk = dk;
  rp.dv = dv;
  rp.dq_in = static_cast<__nv_bfloat16*>(dq_in);
  rp.dk_in = static_cast<__nv_bfloat16*>(dk_in);
  rp.dv_in = static_cast<__nv_bfloat16*>(dv_in);
  rp.dq_in_stride = dq_in_stride;
  rp.dk_in_stride = dk_in_stride;
  rp.dv_in_stride = dv_in_stride;
  rp.dw_part = static_cast<float*>(workspace);
  rp.err = err;
  const bool fp32 = params->grad_dtype == 1;
  const bool whole = rope_most(params, (int)g.y) <= (fp32 ? kRopeBwdWholeFp32 : kRopeBwdWhole);
  if (params->norm && params->interleaved)
    rope_bwd_launch<true, true>(rp, g, fp32, whole, s);
  else if (params->norm)
    rope_bwd_launch<true, false>(rp, g, fp32, whole, s);
  else if (params->interleaved)
    rope_bwd_launch<false, true>(rp, g, fp32, whole, s);
  else
    rope_bwd_launch<false, false>(rp, g, fp32, whole, s);
  if (!launched()) return ATTN_SINK_ERR_CUDA;
  if (params->norm) {
    const RopeSum sum{rp.dw_part, dq_weight, dk_weight, (int)(g.x * g.y)};
    if (!launch_dependent(attn_sink_rope_dw_kernel, 1, kRopeSumThreads, 0, s, sum))
      return ATTN_SINK_ERR_CUDA;
  }
  return ATTN_SINK_OK;
}

size_t attn_sink_extend_workspace_size(const attn_sink_extend_params* params) {
  ExtendLayout L;
  if (extend_layout(params, sm_count_or_default(), &L) != ATTN_SINK_OK || params->batch == 0 ||
      params->total_q == 0)
    return 0;
  return L.total;
}

int attn_sink_extend(const attn_sink_extend_params* params, const void* q, const void* k_cache,
                     const void* v_cache, const int* block_table, const int* seq_lens,
                     const int* cu_seqlens_q, const float* sink, void* out, float* lse,
                     void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("attn_sink_extend");
  ExtendLayout L;
  int st = extend_layout(params, sm_count_or_default(), &L);
  if (st != ATTN_SINK_OK) return st;
  if (params->batch == 0 || params->total_q == 0) return ATTN_SINK_OK;
  if (q == nullptr || sink == nullptr || out == nullptr || lse == nullptr ||
      seq_lens == nullptr || cu_seqlens_q == nullptr ||
      (params->max_pages > 0 && block_table == nullptr) ||
      (params->num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return ATTN_SINK_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < L.total ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return ATTN_SINK_ERR_WORKSPACE;
  int sms = 0;
  int* err = nullptr;
  if ((st = device_state(&sms, &err)) != ATTN_SINK_OK) return st;
  if ((st = extend_attributes()) != ATTN_SINK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ExtParams ep;
  std::memset(&ep, 0, sizeof(ep));
  ep.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  ep.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  ep.block_table = block_table;
  ep.seq_lens = seq_lens;
  ep.cu_q = cu_seqlens_q;
  ep.sink = sink;
  ep.out = static_cast<__nv_bfloat16*>(out);
  ep.lse = lse;
  ep.items = reinterpret_cast<ExtItem*>(ws);
  ep.n_tiles = reinterpret_cast<int2*>(ws + L.off_tiles);
  ep.tiles = reinterpret_cast<ExtTileRef*>(ws + L.off_tiles + 256);
  ep.ml_part = reinterpret_cast<float2*>(ws + L.off_ml);
  ep.o_part = reinterpret_cast<float*>(ws + L.off_o);
  ep.err = err;
  ep.batch = params->batch;
  ep.total_q = params->total_q;
  ep.heads_q = params->heads_q;
  ep.heads_kv = params->heads_kv;
  ep.group = params->heads_q / params->heads_kv;
  ep.tokens = L.tokens;
  ep.page_size = params->page_size;
  ep.num_pages = params->num_pages;
  ep.max_pages = params->max_pages;
  ep.window = params->window > 0 ? std::min(params->window, 1 << 30) : 0;   // >= any length
  ep.n_items = L.n_items;
  ep.max_parts = L.max_parts;
  ep.max_tiles = L.max_tiles;
  ep.slots = L.slots;
  ep.scale_log2 = params->softmax_scale * kLog2e;
#ifdef ATTN_SINK_TEST_HOOKS
  ep.skip_k_tile = g_test_skip_k_tile.load();
#endif
  if (L.band_cols > 0) return extend_window(params, L, ep, q, out, ws, sms, s);
  // Page sizes that are a multiple of 8 keys (whole swizzle atoms) are copied by
  // TMA, in boxes of the largest power of two that divides the page, at most a
  // block; the rows have to fit a copy's 32-bit coordinates.
  const long long rows = (long long)params->num_pages * params->page_size;
  const bool tma = params->page_size % 8 == 0 && rows > 0 && rows < (1ll << 31);
  ep.box = tma ? std::min(params->page_size & -params->page_size, kBlockN) : 0;
  if ((st = encode_rows(&ep.tm_q, q, params->total_q, params->heads_q,
                        CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L.tokens, ep.group)) != ATTN_SINK_OK ||
      (st = encode_rows(&ep.tm_out, out, params->total_q, params->heads_q,
                        CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L.tokens, ep.group)) != ATTN_SINK_OK)
    return st;
  if (tma &&
      ((st = encode_rows(&ep.tm_k, k_cache, rows, params->heads_kv,
                         CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ep.box)) != ATTN_SINK_OK ||
       (st = encode_rows(&ep.tm_v, v_cache, rows, params->heads_kv,
                         CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ep.box)) != ATTN_SINK_OK))
    return st;
  const auto kernel = tma ? attn_sink_extend_kernel<true> : attn_sink_extend_kernel<false>;
  const unsigned grid = (unsigned)L.n_items * (unsigned)params->heads_kv;
  if (L.find) {
    ep.items = nullptr;
    kernel<<<grid, kExtThreads, kFwdSmemBytes, s>>>(ep);
    return launched() ? ATTN_SINK_OK : ATTN_SINK_ERR_CUDA;
  }
  attn_sink_extend_plan_kernel<<<1, kExtSchedThreads, 0, s>>>(ep);
  if (!launched() || !launch_dependent(kernel, grid, kExtThreads, kFwdSmemBytes, s, ep) ||
      (L.split &&
       !launch_dependent(attn_sink_extend_join_kernel, kExtJoinCtas * sms, kExtJoinThreads, 0, s, ep)))
    return ATTN_SINK_ERR_CUDA;
  return ATTN_SINK_OK;
}

}  // extern "C"
