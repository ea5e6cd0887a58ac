// Host side of the token-sequence operators (declared in include/clear_attn.h): argument checks,
// tensor maps and launches. Included by clear_attn.cu.
#pragma once

#include <atomic>

#include "clear_seq_append.cuh"
#include "clear_seq_decode.cuh"
#include "clear_seq_prompt.cuh"
#include "clear_seq_prompt_bwd.cuh"

namespace {

// Launches a kernel as a programmatic dependent of the one before it in the stream: it may start early and waits for that one's
// results by griddepcontrol.wait.
template <typename... P, typename... A>
bool launch_dependent(void (*kernel)(P...), dim3 grid, int block, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

// Allows a kernel `bytes` of dynamic shared memory, once per device: `done` has a bit for each of the first 64.
bool allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done->load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done->fetch_or(bit, std::memory_order_relaxed);
  return true;
}

bool seq_strides_ok(long long s, long long per16, long long n) {
  // A stride that is used (more than one element along its axis) is a positive multiple of 16 bytes.
  return n <= 1 || (s > 0 && s % per16 == 0 && s < (1ll << 39));
}

clear_status_t check_seq_params(const clear_seq_params_t* p) {
  if (!p) return CLEAR_ERR_INVALID_ARG;
  if (p->n_seq < 1 || p->n_seq > (1 << 20) || p->n_tok < 1 || p->n_tok > (1 << 30)) return CLEAR_ERR_INVALID_ARG;
  if (p->q_heads < 1 || p->kv_heads < 1 || p->q_heads > (1 << 14) || p->q_heads % p->kv_heads) return CLEAR_ERR_INVALID_ARG;
  if (p->dtype != CLEAR_DTYPE_BF16 && p->dtype != CLEAR_DTYPE_FP16) return CLEAR_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return CLEAR_ERR_UNSUPPORTED;
  return CLEAR_OK;
}

// A [heads, tokens, d] view: 16-byte aligned, strides of used axes positive multiples of 16 bytes.
// An unused axis gets a harmless stride.
clear_status_t check_seq_view(const clear_seq_view_t* v, int heads, int n_tok, int d, SeqView* out) {
  if (!v || !aligned16(v->ptr)) return CLEAR_ERR_INVALID_ARG;
  if (!seq_strides_ok(v->head_stride, 8, heads) || !seq_strides_ok(v->token_stride, 8, n_tok)) return CLEAR_ERR_UNSUPPORTED;
  out->ptr = v->ptr;
  out->sh = heads > 1 ? v->head_stride : (long long)d;
  out->st = n_tok > 1 ? v->token_stride : (long long)d;
  return CLEAR_OK;
}

clear_status_t check_seq_cache(const clear_seq_params_t* p, const clear_seq_cache_t* c, SeqCache* out) {
  if (!c) return CLEAR_ERR_INVALID_ARG;
  if (c->dtype != p->dtype && c->dtype != CLEAR_DTYPE_E4M3) return CLEAR_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || c->page_size < 1 || c->page_size > (1 << 20) || c->max_pages < 1) return CLEAR_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !c->page_table) return CLEAR_ERR_INVALID_ARG;
  if (c->page_table_stride < c->max_pages && p->n_seq > 1) return CLEAR_ERR_INVALID_ARG;
  const bool f8 = c->dtype == CLEAR_DTYPE_E4M3;
  if (f8 && (!c->k_scale || !c->v_scale)) return CLEAR_ERR_INVALID_ARG;
  const long long per16 = f8 ? 16 : 8;
  const int n[3] = {c->n_pages, c->page_size, p->kv_heads};
  for (int i = 0; i < 3; ++i) {
    if (!seq_strides_ok(c->k_strides[i], per16, n[i]) || !seq_strides_ok(c->v_strides[i], per16, n[i])) return CLEAR_ERR_UNSUPPORTED;
    out->ks[i] = n[i] > 1 ? c->k_strides[i] : 0;
    out->vs[i] = n[i] > 1 ? c->v_strides[i] : 0;
  }
  out->k = c->k_pages;
  out->v = c->v_pages;
  out->table = c->page_table;
  out->table_stride = c->page_table_stride;
  out->max_pages = c->max_pages;
  out->n_pages = c->n_pages;
  out->page_size = c->page_size;
  out->page_div = make_fast_div(c->page_size);
  out->k_scale = f8 ? c->k_scale : nullptr;
  out->v_scale = f8 ? c->v_scale : nullptr;
  return CLEAR_OK;
}

// ---------------------------------------------------------------------------------------- append
// Tokens from which blocks are small (128 threads): enough blocks then to fill the SMs with such. Measured small and large, 24 and 8
// heads of 128, bf16: 256 tokens 4.4 and 3.9 us, 512 tokens 5.0 and 4.6, 1024 tokens 6.0 and 6.8, 8192 tokens 33 and 41; 32 and 8
// into E4M3: 256 tokens 4.9 and 4.2, 512 tokens 5.6 and 6.4, 1024 tokens 6.5 and 8.9. Few heads have small blocks anyway.
constexpr int kAppendMany = 1024;

template <typename E, bool kF8, int D, bool kHalves>
clear_status_t launch_append(const SeqAppendParams& a, cudaStream_t stream) {
  const int items = ((a.q_heads + 2 * a.kv_heads) * (D / 16) + 31) & ~31;
  const int most = a.n_tok >= kAppendMany ? 128 : kAppendMaxThreads;
  clear_seq_append_kernel<E, kF8, D, kHalves><<<a.n_tok, items < 64 ? 64 : items < most ? items : most, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? CLEAR_OK : CLEAR_ERR_CUDA;
}

template <typename E, bool kF8>
clear_status_t launch_append_d(const SeqAppendParams& a, int d, bool halves, cudaStream_t s) {
  if (d == 64) return halves ? launch_append<E, kF8, 64, true>(a, s) : launch_append<E, kF8, 64, false>(a, s);
  return halves ? launch_append<E, kF8, 128, true>(a, s) : launch_append<E, kF8, 128, false>(a, s);
}

// ---------------------------------------------------------------------------------------- decode

struct DecodeWorkspace {
  size_t ml_off, split_off, total;
};
DecodeWorkspace decode_workspace_layout(int d) {
  DecodeWorkspace w;
  w.ml_off = align256((size_t)2 * kDecMaxBlocks * kDecRows * d * sizeof(float));
  w.split_off = align256(w.ml_off + (size_t)2 * kDecMaxBlocks * kDecRows * sizeof(float2));
  w.total = align256(w.split_off + (size_t)kDecMaxBlocks * sizeof(int4));
  return w;
}

// A cache side as (128 bytes of a row, heads, rows, blocks of 128 bytes, pages), in boxes of 16 whole rows of one head,
// which land block by block. Axes of one element get a stride that passes the encoder's checks.
bool make_cache_map(CUtensorMap* m, void* base, const long long* st, const SeqCache& c, int heads, int d, int elem_bytes, int box_bytes) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const int blocks = d * elem_bytes / box_bytes;
  cuuint64_t dims[5] = {(cuuint64_t)(box_bytes / elem_bytes), (cuuint64_t)heads, (cuuint64_t)c.page_size, (cuuint64_t)blocks,
                        (cuuint64_t)c.n_pages};
  const auto bytes = [&](long long s) { return (cuuint64_t)(s > 0 ? s : d) * elem_bytes; };
  cuuint64_t strides[4] = {bytes(st[2]), bytes(st[1]), (cuuint64_t)box_bytes, bytes(st[0])};
  cuuint32_t box[5] = {(cuuint32_t)(box_bytes / elem_bytes), 1, (cuuint32_t)kDecSlice, (cuuint32_t)blocks, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, base, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             d * elem_bytes >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename E, bool kF8, int D>
clear_status_t launch_decode(SeqDecodeParams p, int num_sms, cudaStream_t stream) {
  using L1 = DecLayout<kF8, D, 1>;
  using L2 = DecLayout<kF8, D, 2>;
  CUtensorMap mk{}, mv{};
  p.tma = p.c.page_size % kDecSlice == 0;
  if (p.tma && (!make_cache_map(&mk, p.c.k, p.c.ks, p.c, p.kv_heads, D, kF8 ? 1 : 2, L1::kBox) ||
                !make_cache_map(&mv, p.c.v, p.c.vs, p.c, p.kv_heads, D, kF8 ? 1 : 2, L1::kBox)))
    return CLEAR_ERR_CUDA;
  // Up to eight heads of a group fill one tile of the matrix instruction, more take two.
  const auto kernel = p.group <= 8 ? clear_seq_decode_kernel<E, kF8, D, 1> : clear_seq_decode_kernel<E, kF8, D, 2>;
  const int smem = p.group <= 8 ? L1::kSmem : L2::kSmem;
  static std::atomic<unsigned long long> done[2];
  if (!allow_smem(reinterpret_cast<const void*>(kernel), smem, &done[p.group <= 8 ? 0 : 1])) return CLEAR_ERR_CUDA;
  const int resident = (p.group <= 8 ? L1::kPerSm : L2::kPerSm) * num_sms;
  const int blocks = resident < kDecMaxBlocks ? resident : kDecMaxBlocks;
  kernel<<<blocks, kDecThreads, smem, stream>>>(mk, mv, p);
  if (cudaGetLastError() != cudaSuccess) return CLEAR_ERR_CUDA;
  const dim3 join(blocks, p.group < kDecRows ? p.group : kDecRows);
  return launch_dependent(clear_seq_decode_join_kernel<E, D>, join, kJoinParts * D, 0, stream, p) ? CLEAR_OK : CLEAR_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------- prompt
// (d, tokens, heads) view with box 64 x 128 x 1, 128-byte swizzle.
bool make_seq_map(CUtensorMap* m, const SeqView& v, int heads, int n_tok, int d, int dtype, int rows = 128) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n_tok, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)v.st * 2, (cuuint64_t)v.sh * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, dtype == CLEAR_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, v.ptr, dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks for items of `rows` query rows: one per SM, fewer when the batch cannot have so many items.
unsigned prompt_blocks(const clear_seq_params_t* p, int rows, int heads, int num_sms) {
  const long long most = ((long long)p->n_tok / rows + p->n_seq) * heads;
  return (unsigned)(most < num_sms ? most : num_sms);
}

constexpr long long kPrSplitItems = 300;

template <typename E, int D>
clear_status_t launch_prompt_fwd(const clear_seq_params_t* sp, const SeqView& q, const SeqView& k, const SeqView& v,
                                 const SeqPromptParams& p, int num_sms, cudaStream_t stream) {
  using L = PromptLayout<D>;
  CUtensorMap mq, mk, mv;
  if (!make_seq_map(&mq, q, sp->q_heads, sp->n_tok, D, sp->dtype) || !make_seq_map(&mk, k, sp->kv_heads, sp->n_tok, D, sp->dtype) ||
      !make_seq_map(&mv, v, sp->kv_heads, sp->n_tok, D, sp->dtype))
    return CLEAR_ERR_CUDA;
  // Whole items share each key tile between 256 rows; split ones are twice as many and half as long, which pays where a block's one
  // or two long items bound the whole. Measured whole and split at d = 128 (at d = 64): one sequence of 6000 tokens, 2 heads (48 items)
  // 86 and 49 us (81 and 44); 8 heads (192) 89 and 77 (84 and 68); one of 12000, 4 heads (188) 173 and 134 (162 and 120); six
  // of 683 on average and unlike, 16 heads (256) 58 and 47; two of 2048, 24 heads (384) 65 and 74 (57 and 64); one of 4096, 32
  // heads (512) 128 and 141 (116 and 120). Between 190 and 300 items it depends on how unlike the lengths are, which the host does not
  // see: like ones lose, six of 683 each 29 and 36 us, one of 4096 with 16 heads 67 and 74. Short sequences have short items
  // already: eight of 300, 8 heads (80) 13 and 16 us.
  const bool split = ((long long)sp->n_tok + 255) / 256 * sp->q_heads < kPrSplitItems && sp->n_tok >= 512ll * sp->n_seq;
  static std::atomic<unsigned long long> done[2];
  const auto kernel = split ? clear_seq_prompt_fwd_kernel<E, D, true> : clear_seq_prompt_fwd_kernel<E, D, false>;
  if (!allow_smem(reinterpret_cast<const void*>(kernel), L::kAlloc, &done[split])) return CLEAR_ERR_CUDA;
  kernel<<<prompt_blocks(sp, split ? 128 : 256, sp->q_heads, num_sms), kPrThreads, L::kAlloc, stream>>>(mq, mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? CLEAR_OK : CLEAR_ERR_CUDA;
}

// Parts that a group's heads are split into for dK and dV: enough that every SM gets two items, where the heads allow it. One
// kv head of 16 query heads on 2048 tokens has 16 items for 148 SMs without. By the parameters alone: the workspace has room
// for the parts' fp32 sums, at most about 75000 rows in all of each of dK and dV.
int bwd_parts(const clear_seq_params_t* p) {
  constexpr long long kWanted = 2 * 148;
  const long long items = (((long long)p->n_tok + 127) / 128) * p->kv_heads;
  const long long group = p->q_heads / p->kv_heads;
  const long long parts = (kWanted + items - 1) / items;
  return (int)(parts < 1 ? 1 : parts > group ? group : parts);
}

struct PromptBwdWorkspace {
  size_t mag_g_off, mag_v_off, top_g_off, top_v_off, part1_off, part2_off, total;
};
PromptBwdWorkspace prompt_bwd_workspace_layout(const clear_seq_params_t* p) {
  PromptBwdWorkspace w;
  const int parts = bwd_parts(p);
  const size_t sums = parts > 1 ? (size_t)parts * p->kv_heads * p->n_tok * p->d * sizeof(float) : 0;
  const size_t g = align256((size_t)p->q_heads * p->n_tok * sizeof(float)), v = align256((size_t)p->kv_heads * p->n_tok * sizeof(float));
  w.mag_g_off = align256((size_t)p->q_heads * p->n_tok * sizeof(float2));  // (-lse, -D) before
  w.mag_v_off = w.mag_g_off + g;
  w.top_g_off = w.mag_v_off + v;
  w.top_v_off = w.top_g_off + g;
  w.part1_off = w.top_v_off + v;
  w.part2_off = w.part1_off + align256(sums);
  w.total = w.part2_off + align256(sums);
  return w;
}

// What n_tok tokens and any smaller number need at most: fewer tokens may take more parts. The parts change only with the number
// of 128-token tiles, and between two changes more tokens need more.
size_t prompt_bwd_workspace_most(const clear_seq_params_t* p) {
  clear_seq_params_t x = *p;
  size_t most = prompt_bwd_workspace_layout(p).total;
  for (x.n_tok = 128; x.n_tok < p->n_tok && bwd_parts(&x) > 1; x.n_tok += 128) {
    const size_t total = prompt_bwd_workspace_layout(&x).total;
    if (total > most) most = total;
  }
  return most;
}

constexpr int kTopsBlocks = 128;  // along the sequences

template <typename E, int D>
clear_status_t launch_prompt_bwd(const clear_seq_params_t* sp, const SeqView& q, const SeqView& k, const SeqView& v, const SeqView& g,
                                 const SeqView& dq, const SeqView& dk, const SeqView& dv, const SeqStatsParams& st, SeqBwdParams p,
                                 int num_sms, cudaStream_t stream) {
  using LK = PromptBwdLayout<D, true>;
  using LQ = PromptBwdLayout<D, false>;
  // Tiles that stay come 128 rows at a time, tiles that stream 64.
  CUtensorMap mq, mk, mv, mg, sq, sk, sv, sg;
  if (!make_seq_map(&mq, q, sp->q_heads, sp->n_tok, D, sp->dtype) || !make_seq_map(&mk, k, sp->kv_heads, sp->n_tok, D, sp->dtype) ||
      !make_seq_map(&mv, v, sp->kv_heads, sp->n_tok, D, sp->dtype) || !make_seq_map(&mg, g, sp->q_heads, sp->n_tok, D, sp->dtype) ||
      !make_seq_map(&sq, q, sp->q_heads, sp->n_tok, D, sp->dtype, 64) || !make_seq_map(&sk, k, sp->kv_heads, sp->n_tok, D, sp->dtype, 64) ||
      !make_seq_map(&sv, v, sp->kv_heads, sp->n_tok, D, sp->dtype, 64) || !make_seq_map(&sg, g, sp->q_heads, sp->n_tok, D, sp->dtype, 64))
    return CLEAR_ERR_CUDA;
  static std::atomic<unsigned long long> done[2];
  if (!allow_smem(reinterpret_cast<const void*>(clear_seq_prompt_bwd_kernel<E, D, true>), LK::kAlloc, &done[0]) ||
      !allow_smem(reinterpret_cast<const void*>(clear_seq_prompt_bwd_kernel<E, D, false>), LQ::kAlloc, &done[1]))
    return CLEAR_ERR_CUDA;
  constexpr bool kF16 = !std::is_same<E, Bf16>::value;
  const long long lanes = (long long)sp->n_tok * sp->q_heads * (D / 8);
  clear_seq_bwd_stats_kernel<E, D><<<(unsigned)((lanes + kStatsThreads - 1) / kStatsThreads), kStatsThreads, 0, stream>>>(st);
  if (cudaGetLastError() != cudaSuccess) return CLEAR_ERR_CUDA;
  p.out2 = dq;  // first: it settles the first rows' statistics for the other
  const unsigned q_blocks = prompt_blocks(sp, 128, sp->q_heads, num_sms);
  if (kF16) {
    const dim3 tops(sp->n_seq < kTopsBlocks ? sp->n_seq : kTopsBlocks, sp->q_heads);
    if (!launch_dependent(clear_seq_bwd_tops_kernel, tops, kTopsThreads, 0, stream, p) ||
        !launch_dependent(clear_seq_prompt_bwd_kernel<E, D, false>, q_blocks, kPrThreads, LQ::kAlloc, stream, mq, mg, sk, sv, p))
      return CLEAR_ERR_CUDA;
  } else {
    clear_seq_prompt_bwd_kernel<E, D, false><<<q_blocks, kPrThreads, LQ::kAlloc, stream>>>(mq, mg, sk, sv, p);
    if (cudaGetLastError() != cudaSuccess) return CLEAR_ERR_CUDA;
  }
  p.out1 = dv;
  p.out2 = dk;
  clear_seq_prompt_bwd_kernel<E, D, true><<<prompt_blocks(sp, 128, sp->kv_heads * p.parts, num_sms), kPrThreads, LK::kAlloc, stream>>>(mk, mv, sq, sg, p);
  if (cudaGetLastError() != cudaSuccess) return CLEAR_ERR_CUDA;
  if (p.parts > 1) {
    const long long threads = 2ll * sp->kv_heads * sp->n_tok * (D / 8);
    clear_seq_bwd_join_kernel<E, D><<<(unsigned)((threads + kStatsThreads - 1) / kStatsThreads), kStatsThreads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? CLEAR_OK : CLEAR_ERR_CUDA;
}

}  // namespace

extern "C" {

clear_status_t clear_attn_cache_append(const clear_seq_params_t* params, const clear_seq_cache_t* cache,
                                       const clear_seq_rope_t* rope, const int* seq_start, const int* seq_len,
                                       const clear_seq_view_t* q, const clear_seq_view_t* k, const clear_seq_view_t* v,
                                       const clear_seq_view_t* q_out, const clear_seq_view_t* k_out, void* stream) {
  clear_status_t st = check_seq_params(params);
  if (st != CLEAR_OK) return st;
  SeqAppendParams a{};
  if ((st = check_seq_cache(params, cache, &a.c)) != CLEAR_OK) return st;
  if (!seq_start || !seq_len || !k || !v || !q != !q_out) return CLEAR_ERR_INVALID_ARG;
  if ((st = check_seq_view(k, params->kv_heads, params->n_tok, params->d, &a.k)) != CLEAR_OK) return st;
  if ((st = check_seq_view(v, params->kv_heads, params->n_tok, params->d, &a.v)) != CLEAR_OK) return st;
  if (q && ((st = check_seq_view(q, params->q_heads, params->n_tok, params->d, &a.q)) != CLEAR_OK ||
            (st = check_seq_view(q_out, params->q_heads, params->n_tok, params->d, &a.q_out)) != CLEAR_OK))
    return st;
  if (k_out && (st = check_seq_view(k_out, params->kv_heads, params->n_tok, params->d, &a.k_out)) != CLEAR_OK) return st;
  bool halves = false;
  if (rope && rope->rot != 0) {
    if (!(rope->theta > 1.f) || !(rope->ntk > 0.f) || !std::isfinite(rope->theta) || !std::isfinite(rope->ntk)) return CLEAR_ERR_INVALID_ARG;
    if (rope->pairing != CLEAR_PAIR_ADJACENT && rope->pairing != CLEAR_PAIR_HALVES) return CLEAR_ERR_INVALID_ARG;
    if (rope->rot < 0 || rope->rot > params->d) return CLEAR_ERR_INVALID_ARG;
    if (rope->rot % 16) return CLEAR_ERR_UNSUPPORTED;
    a.rot = rope->rot;
    halves = rope->pairing == CLEAR_PAIR_HALVES;
    // Rates base^(-2i / rot) as powers of one ratio, in extended precision: 64 steps lose less than a double's last bit, and
    // 64 calls of pow would take as long as the launch.
    const long double base = (long double)rope->theta * std::pow((long double)rope->ntk, (long double)a.rot / (a.rot - 2));
    const long double ratio = std::pow(base, -2.0L / a.rot);
    long double turn = 1.0L / 6.283185307179586476925286766559L;
    for (int i = 0; i < a.rot / 2; ++i, turn *= ratio) a.turns[i] = (double)turn;
  }
  int num_sms = 0;
  if ((st = check_device(&num_sms)) != CLEAR_OK) return st;
  a.seq_start = seq_start;
  a.seq_len = seq_len;
  a.n_seq = params->n_seq;
  a.n_tok = params->n_tok;
  a.q_heads = q ? params->q_heads : 0;
  a.kv_heads = params->kv_heads;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == CLEAR_DTYPE_E4M3;
  if (params->dtype == CLEAR_DTYPE_BF16)
    return f8 ? launch_append_d<Bf16, true>(a, params->d, halves, s) : launch_append_d<Bf16, false>(a, params->d, halves, s);
  return f8 ? launch_append_d<Fp16, true>(a, params->d, halves, s) : launch_append_d<Fp16, false>(a, params->d, halves, s);
}

size_t clear_attn_decode_workspace_size(const clear_seq_params_t* params, clear_status_t* status) {
  const clear_status_t st = check_seq_params(params);
  if (status) *status = st;
  return st == CLEAR_OK ? decode_workspace_layout(params->d).total : 0;
}

clear_status_t clear_attn_decode(const clear_seq_params_t* params, const clear_seq_cache_t* cache, const int* seq_len,
                                 const clear_seq_view_t* q, const clear_seq_view_t* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  clear_status_t st = check_seq_params(params);
  if (st != CLEAR_OK) return st;
  if (params->n_tok != params->n_seq || !seq_len) return CLEAR_ERR_INVALID_ARG;
  SeqDecodeParams p{};
  if ((st = check_seq_cache(params, cache, &p.c)) != CLEAR_OK) return st;
  if ((st = check_seq_view(q, params->q_heads, params->n_tok, params->d, &p.q)) != CLEAR_OK) return st;
  if ((st = check_seq_view(o, params->q_heads, params->n_tok, params->d, &p.o)) != CLEAR_OK) return st;
  const DecodeWorkspace wl = decode_workspace_layout(params->d);
  if (!workspace || workspace_bytes < wl.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return CLEAR_ERR_WORKSPACE;
  int num_sms = 0;
  if ((st = check_device(&num_sms)) != CLEAR_OK) return st;
  p.lse = lse;
  p.seq_len = seq_len;
  p.n_seq = params->n_seq;
  p.q_heads = params->q_heads;
  p.kv_heads = params->kv_heads;
  p.group = params->q_heads / params->kv_heads;
  p.m_tiles = (p.group + kDecRows - 1) / kDecRows;
  const long long rows = (long long)cache->max_pages * cache->page_size;
  p.max_len = rows < INT_MAX ? (int)rows : INT_MAX;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)params->d));
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + wl.ml_off);
  p.split = reinterpret_cast<int4*>(ws + wl.split_off);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == CLEAR_DTYPE_E4M3, bf = params->dtype == CLEAR_DTYPE_BF16;
  if (params->d == 64) {
    if (bf) return f8 ? launch_decode<Bf16, true, 64>(p, num_sms, s) : launch_decode<Bf16, false, 64>(p, num_sms, s);
    return f8 ? launch_decode<Fp16, true, 64>(p, num_sms, s) : launch_decode<Fp16, false, 64>(p, num_sms, s);
  }
  if (bf) return f8 ? launch_decode<Bf16, true, 128>(p, num_sms, s) : launch_decode<Bf16, false, 128>(p, num_sms, s);
  return f8 ? launch_decode<Fp16, true, 128>(p, num_sms, s) : launch_decode<Fp16, false, 128>(p, num_sms, s);
}

clear_status_t clear_attn_prompt_fwd(const clear_seq_params_t* params, const int* seq_start, const clear_seq_view_t* q,
                                     const clear_seq_view_t* k, const clear_seq_view_t* v, const clear_seq_view_t* o,
                                     float* lse, void* stream) {
  clear_status_t st = check_seq_params(params);
  if (st != CLEAR_OK) return st;
  SeqView vq, vk, vv;
  SeqPromptParams p{};
  if (!seq_start) return CLEAR_ERR_INVALID_ARG;
  if ((st = check_seq_view(q, params->q_heads, params->n_tok, params->d, &vq)) != CLEAR_OK) return st;
  if ((st = check_seq_view(k, params->kv_heads, params->n_tok, params->d, &vk)) != CLEAR_OK) return st;
  if ((st = check_seq_view(v, params->kv_heads, params->n_tok, params->d, &vv)) != CLEAR_OK) return st;
  if ((st = check_seq_view(o, params->q_heads, params->n_tok, params->d, &p.o)) != CLEAR_OK) return st;
  int num_sms = 0;
  if ((st = check_device(&num_sms)) != CLEAR_OK) return st;
  p.lse = lse;
  p.seq_start = seq_start;
  p.n_seq = params->n_seq;
  p.n_tok = params->n_tok;
  p.q_heads = params->q_heads;
  p.group = params->q_heads / params->kv_heads;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)params->d));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->dtype == CLEAR_DTYPE_BF16)
    return params->d == 64 ? launch_prompt_fwd<Bf16, 64>(params, vq, vk, vv, p, num_sms, s)
                           : launch_prompt_fwd<Bf16, 128>(params, vq, vk, vv, p, num_sms, s);
  return params->d == 64 ? launch_prompt_fwd<Fp16, 64>(params, vq, vk, vv, p, num_sms, s)
                         : launch_prompt_fwd<Fp16, 128>(params, vq, vk, vv, p, num_sms, s);
}

size_t clear_attn_prompt_bwd_workspace_size(const clear_seq_params_t* params, clear_status_t* status) {
  const clear_status_t st = check_seq_params(params);
  if (status) *status = st;
  return st == CLEAR_OK ? prompt_bwd_workspace_most(params) : 0;
}

clear_status_t clear_attn_prompt_bwd(const clear_seq_params_t* params, const int* seq_start, const clear_seq_view_t* q,
                                     const clear_seq_view_t* k, const clear_seq_view_t* v, const clear_seq_view_t* o,
                                     const float* lse, const clear_seq_view_t* dO, const clear_seq_view_t* dq,
                                     const clear_seq_view_t* dk, const clear_seq_view_t* dv, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  clear_status_t st = check_seq_params(params);
  if (st != CLEAR_OK) return st;
  if (!seq_start || !lse) return CLEAR_ERR_INVALID_ARG;
  const clear_seq_view_t* views[8] = {q, k, v, o, dO, dq, dk, dv};
  SeqView w[8];
  for (int i = 0; i < 8; ++i) {
    const bool kv = i == 1 || i == 2 || i == 6 || i == 7;
    if ((st = check_seq_view(views[i], kv ? params->kv_heads : params->q_heads, params->n_tok, params->d, &w[i])) != CLEAR_OK) return st;
  }
  if (!workspace || workspace_bytes < prompt_bwd_workspace_layout(params).total ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return CLEAR_ERR_WORKSPACE;
  // The row statistics take one thread per 8 elements of o; their grid must fit.
  if ((long long)params->n_tok * params->q_heads * (params->d / 8) / kStatsThreads >= INT_MAX) return CLEAR_ERR_UNSUPPORTED;
  int num_sms = 0;
  if ((st = check_device(&num_sms)) != CLEAR_OK) return st;
  SeqStatsParams sp{};
  sp.o = w[3];
  sp.g = w[4];
  sp.v = w[2];
  sp.lse = lse;
  sp.stats = static_cast<float2*>(workspace);
  SeqBwdParams p{};
  p.stats = sp.stats;
  const PromptBwdWorkspace wl = prompt_bwd_workspace_layout(params);
  const auto at = [&](size_t off) { return reinterpret_cast<float*>(static_cast<char*>(workspace) + off); };
  p.mag_g = sp.mag_g = at(wl.mag_g_off);
  p.mag_v = sp.mag_v = at(wl.mag_v_off);
  p.top_g = at(wl.top_g_off);
  p.top_v = at(wl.top_v_off);
  p.parts = bwd_parts(params);
  p.part1 = at(wl.part1_off);
  p.part2 = at(wl.part2_off);
  p.seq_start = sp.seq_start = seq_start;
  p.n_seq = sp.n_seq = params->n_seq;
  p.n_tok = sp.n_tok = params->n_tok;
  p.q_heads = sp.q_heads = params->q_heads;
  p.kv_heads = params->kv_heads;
  p.group = sp.group = params->q_heads / params->kv_heads;
  p.scale = (float)(1.0 / std::sqrt((double)params->d));
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)params->d));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (params->dtype == CLEAR_DTYPE_BF16)
    return params->d == 64 ? launch_prompt_bwd<Bf16, 64>(params, w[0], w[1], w[2], w[4], w[5], w[6], w[7], sp, p, num_sms, s)
                           : launch_prompt_bwd<Bf16, 128>(params, w[0], w[1], w[2], w[4], w[5], w[6], w[7], sp, p, num_sms, s);
  return params->d == 64 ? launch_prompt_bwd<Fp16, 64>(params, w[0], w[1], w[2], w[4], w[5], w[6], w[7], sp, p, num_sms, s)
                         : launch_prompt_bwd<Fp16, 128>(params, w[0], w[1], w[2], w[4], w[5], w[6], w[7], sp, p, num_sms, s);
}

}  // extern "C"
