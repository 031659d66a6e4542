// rows_api.cuh - host side of mlra_prefill and mlra_decode_prefix (included by mlra_api.cu, whose
// handle, tensor maps and launch helpers it uses): argument checks, workspace, launch sequence.
#pragma once

namespace {

// Shapes of the row attention, one a set of block dims. MLRA-4 blocks (d_b = 128) run two row tiles in
// turn; at d_b = 256 a row tile's O fills half the tensor memory, so one row tile alternates two
// score buffers over 64-key tiles; at d_b = 512 two CTAs keep a half of O each and both form the
// scores (3328 FLOPs a query, key and head in place of 2176, but nothing passes between SMs).
using RowsTiny = RowShape<32, 16, 128, 32, 2, 4, 4>;
using RowsB128 = RowShape<128, 64, 128, 128, 2, 3, 2>;
using RowsB256 = RowShape<256, 64, 64, 256, 1, 3, 3>;
using RowsB512 = RowShape<512, 64, 64, 256, 1, 1, 1>;

// The per-head form (whole prompts): keys of 128 + 64, values of 128, whatever the block width
using RowsHead = RowShape<128, 64, 128, 128, 2, 2, 2, 1>;

constexpr int kMaxQueryTokens = 1 << 21;  // grid rows of the absorb kernel

template <class F>
auto with_rows(Variant v, F f) {
  switch (v) {
    case kTiny: return f(RowsTiny{});
    case kMlra2: case kMlra2Sum: return f(RowsB256{});
    case kMla: return f(RowsB512{});
    default: return f(RowsB128{});
  }
}

template <int DBB, int DH, int SUMK>
cudaError_t prep_up() {
  return prep_kernel(mlra_rows_up_kernel<UpShape<DBB, DH, SUMK>>, UpShape<DBB, DH, SUMK>::SMEM);
}
// At d_b = 128 two CTAs an SM with short rings
template <int DBB>
using ExpandShape = UpShape<DBB, 128, 1, DBB == 128 ? 2 : 4, true>;
template <int DBB>
cudaError_t prep_head() {
  cudaError_t e = prep_kernel(mlra_rows_up_kernel<ExpandShape<DBB>, true>, ExpandShape<DBB>::SMEM);
  return e == cudaSuccess ? prep_kernel(mlra_rows_kernel<RowsHead>, RowsHead::SMEM) : e;
}
cudaError_t prep_rows(Variant v) {
  cudaError_t e0 = prep_kernel(mlra_rows_plan_kernel, 0);
  if (e0 == cudaSuccess) e0 = prep_kernel(mlra_rows_merge_kernel, 0);
  if (e0 == cudaSuccess) e0 = prep_kernel(mlra_widen_pages_kernel, 0);
  if (e0 != cudaSuccess) return e0;
  cudaError_t e = with_rows(v, [](auto sh) {
    using Sh = decltype(sh);
    return prep_kernel(mlra_rows_kernel<Sh>, Sh::SMEM);
  });
  if (e != cudaSuccess) return e;
  switch (v) {
    case kTiny:
      e = prep_up<32, 32, 1>();
      return e == cudaSuccess ? prep_up<32, 32, 4>() : e;
    case kMlra2:
      e = prep_up<256, 128, 1>();
      return e == cudaSuccess ? prep_head<256>() : e;
    case kMlra2Sum: return prep_up<256, 128, 2>();
    case kMla:
      e = prep_up<512, 128, 1>();
      return e == cudaSuccess ? prep_head<512>() : e;
    case kMlra4Sum: return prep_up<128, 128, 4>();
    default:
      e = prep_up<128, 128, 1>();
      return e == cudaSuccess && v == kMlra4 ? prep_head<128>() : e;
  }
}

// The combine with prefix parts (the decode step's combine kernel, one more template flag).
template <int DB, int DH, int SUMK, int NT>
cudaError_t prep_prefix_nt() {
  using S = ProjShape<DB, DH, NT>;
  const cudaError_t e = prep_kernel(mlra_uproj_kernel<S, false, SUMK, 1>, S::SMEM4);
  return e == cudaSuccess ? prep_kernel(mlra_uproj_kernel<S, false, SUMK, 2>, S::SMEM4) : e;
}
template <int DB, int DH, int SUMK>
cudaError_t prep_prefix_proj() {
  cudaError_t e = prep_prefix_nt<DB, DH, SUMK, 16>();
  if (e == cudaSuccess) e = prep_prefix_nt<DB, DH, SUMK, 32>();
  if (e == cudaSuccess) e = prep_prefix_nt<DB, DH, SUMK, 64>();
  if constexpr (max_nt<DB>() >= 128)
    if (e == cudaSuccess) e = prep_prefix_nt<DB, DH, SUMK, 128>();
  return e;
}
cudaError_t prep_prefix(Variant v, bool summed) {
  switch (v) {
    case kTiny: return summed ? prep_prefix_proj<128, 32, 4>() : prep_prefix_proj<32, 32, 1>();
    case kMlra4: return prep_prefix_proj<128, 128, 1>();
    case kMlra4Sum: return prep_prefix_proj<512, 128, 4>();
    case kMlra2: return prep_prefix_proj<256, 128, 1>();
    case kMlra2Sum: return prep_prefix_proj<512, 128, 2>();
    case kMla: return prep_prefix_proj<512, 128, 1>();
    default: return prep_prefix_proj<128, 128, 1>();  // (E4M3 cache: for prompts only)
  }
}

template <int DB, int DH, int SUMK, int NT>
cudaError_t launch_uproj_prefix(const mlra_ctx* h, const ProjParams& pp, int batch, bool own, cudaStream_t s) {
  using S = ProjShape<DB, DH, NT>;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c =
      launch_cfg(dim3(h->cfg.h, (batch + NT - 1) / NT), dim3(kProjThreads), S::SMEM4, s, true, &attr);
  return own ? cudaLaunchKernelEx(&c, mlra_uproj_kernel<S, false, SUMK, 2>, h->map_wuv, pp)
             : cudaLaunchKernelEx(&c, mlra_uproj_kernel<S, false, SUMK, 1>, h->map_wuv, pp);
}
template <int DB, int DH, int SUMK>
cudaError_t dispatch_uproj_prefix(const mlra_ctx* h, const ProjParams& pp, int batch, bool own, cudaStream_t s) {
  switch (nt_for(batch, max_nt<DB>())) {
    case 16: return launch_uproj_prefix<DB, DH, SUMK, 16>(h, pp, batch, own, s);
    case 32: return launch_uproj_prefix<DB, DH, SUMK, 32>(h, pp, batch, own, s);
    case 64: return launch_uproj_prefix<DB, DH, SUMK, 64>(h, pp, batch, own, s);
    default:
      if constexpr (max_nt<DB>() >= 128) return launch_uproj_prefix<DB, DH, SUMK, 128>(h, pp, batch, own, s);
      return cudaErrorInvalidValue;
  }
}

// A bump allocator over the caller's workspace (base null: sizes only).
struct Carver {
  char* base;
  size_t off;
  template <class T>
  T* take(size_t count) {
    T* p = reinterpret_cast<T*>(base + off);
    off += align256(count * sizeof(T));
    return p;
  }
};

struct RowsWorkspace {
  RowPlan plan;
  float* part_o;
  float* part_lse;
};
// Plan and partial slots of the row attention over `tokens` query tokens of `seqs` sequences;
// `heads`: heads a row tile stacks.
template <class Sh>
RowsWorkspace carve_rows(const mlra_ctx* h, Carver& c, size_t tokens, size_t seqs, int heads, bool per_token) {
  const size_t tile = (size_t)Sh::NQ * (128 / heads);
  const size_t tiles = tokens / tile + seqs;
  RowsWorkspace w;
  w.plan.hdr = c.take<int>(8);
  w.plan.first = c.take<int4>((size_t)3 * h->num_sms);
  w.plan.start = c.take<long long>(tiles + 1);
  w.plan.tile = c.take<TokenTile>(tiles);
  w.plan.base = c.take<int>(seqs + 1);
  w.plan.cut = c.take<int4>((size_t)2 * h->num_sms);
  w.plan.tok = per_token ? c.take<int4>(2 * tokens) : nullptr;  // (a second record: own rows)
  w.part_lse = c.take<float>((size_t)2 * h->num_sms * Sh::ROWS);
  w.part_o = c.take<float>((size_t)2 * h->num_sms * Sh::ROWS * Sh::DV);
  return w;
}
int heads_tile_of(const mlra_ctx* h) { return h->heads_block < h->np ? h->heads_block : h->np; }

// Rows of a sequence in the per-head buffers: whole 128-token tiles.
long long seq_rows_of(int pt_stride) { return ((long long)pt_stride + 1) / 2 * kTile; }

// Whether a prompt call of these sizes takes the per-head form (unless its query is fp32): form every
// head's keys and values of the cached rows once, then attend with keys of d_h + d_rope and values of
// d_h: 640 FLOPs a query, key and head, against 640, 1152 and 3328 of the absorbed form at d_b = 128,
// 256 and 512 (where it forms the scores twice), and without its two projections' query-sided traffic.
// It costs 4 d_b d_h FLOPs and 512 bytes (of workspace too) a cached row and head. The rows' number is
// known on the device only; the host goes by the table's capacity, at most four times the query tokens,
// which holds the workspace down: a sequence with many new tokens would gain behind any context at
// d_b >= 256, and loses the form on wider tables.
// Measured, whole calls, 128 heads, per-head against absorbed, ms. One prompt of 2048, 4096, 16384
// tokens: d_b = 128: 0.24 and 0.31, 0.74 and 0.84, 9.45 and 9.13; d_b = 256: 0.27 and 0.66, 0.78 and
// 1.90, 9.42 and 20.2; d_b = 512: 0.31 and 1.93, 0.86 and 6.61 (the first two). (A few calls at a time;
// in long runs the power cap adds up to a tenth.) 1024 tokens on 4096 rows, a table at the rule's edge:
// 0.35 and 0.31, 0.39 and 0.54, 0.47 and 2.69. So at d_b = 128 long prompts and chunks of longer
// contexts lose 3 to 13 percent by it.
bool per_head_sizes(const mlra_ctx* h, int total_q, int batch, int pt_stride) {
  if (h->summed || h->fp8 || h->var == kTiny) return false;
  const long long rows = (long long)batch * seq_rows_of(pt_stride);  // a row's index is 32 bits
  return (long long)batch * pt_stride * kPage <= 4LL * total_q && rows * h->cfg.h <= 0x7fffffffLL - kTile;
}

// Few query tokens: the decode step's combine merges the attention's parts and up-projects in one
// kernel, in place of the merge and the up-projection of many tokens. Measured (four sequences of 128
// heads, contexts of 2000), both ways: d_b = 128: 28.7 and 29.0 us at 16 tokens, 32.2 and 34.9 at 32,
// 43.1 and 43.6 at 64, 59.1 and 55.4 at 128; d_b = 256: 38.6 and 38.1 at 16, 55.3 and 51.2 at 64.
constexpr int kFewTokens = 32;
bool few_tokens(const mlra_ctx* h, int total_q) { return total_q <= kFewTokens && h->d_b <= 128 && !h->summed; }

struct PrefillWorkspace {
  int* status;
  __nv_bfloat16* q_pack;
  __nv_bfloat16* o;
  float* o_few;          // few tokens: [tokens][vh][d_b], and log2 sums [tokens][vh]
  float* lse_few;
  __nv_bfloat16* pages;  // E4M3 cache only
  RowsWorkspace rows;
  size_t bytes;
};
PrefillWorkspace carve_prefill(const mlra_ctx* h, int total_q, int batch, int pt_stride, void* base) {
  Carver c = {static_cast<char*>(base), 0};
  PrefillWorkspace w;
  w.status = c.take<int>(64);
  w.q_pack = c.take<__nv_bfloat16>((size_t)total_q * h->nsub * h->np * (h->d_b + h->d_r));
  const bool few = few_tokens(h, total_q);
  w.o = few ? nullptr : c.take<__nv_bfloat16>((size_t)total_q * h->vh * h->d_b);
  w.o_few = few ? c.take<float>((size_t)total_q * h->vh * h->d_b) : nullptr;
  w.lse_few = few ? c.take<float>((size_t)total_q * h->vh) : nullptr;
  w.rows = with_rows(h->var, [&](auto sh) {
    return carve_rows<decltype(sh)>(h, c, total_q, batch, heads_tile_of(h), few);
  });
  w.pages = h->fp8 ? c.take<__nv_bfloat16>((size_t)batch * pt_stride * kPage * (h->cfg.d_c + h->d_r)) : nullptr;
  w.bytes = c.off;
  return w;
}

struct HeadWorkspace {
  int* status;
  __nv_bfloat16* kv;   // [h][rows][2 * d_h]
  __nv_bfloat16* kr;   // [rows][d_rope]
  RowsWorkspace rows;
  size_t bytes;
};
HeadWorkspace carve_head(const mlra_ctx* h, int total_q, int batch, int pt_stride, void* base) {
  Carver c = {static_cast<char*>(base), 0};
  const size_t rows = (size_t)batch * seq_rows_of(pt_stride);
  HeadWorkspace w;
  w.status = c.take<int>(64);
  w.kv = c.take<__nv_bfloat16>(rows * h->cfg.h * 2 * h->cfg.d_h);
  w.kr = c.take<__nv_bfloat16>(rows * h->d_r);
  w.rows = carve_rows<RowsHead>(h, c, total_q, batch, 1, false);
  w.bytes = c.off;
  return w;
}
size_t prefill_bytes(const mlra_ctx* h, int total_q, int batch, int pt_stride) {
  size_t a = carve_prefill(h, total_q, batch, pt_stride, nullptr).bytes;
  // Few tokens keep fp32 latents and a record a token, which more tokens do without: a call's workspace
  // holds any smaller call's as well.
  const size_t few = carve_prefill(h, total_q < kFewTokens ? total_q : kFewTokens, batch, pt_stride, nullptr).bytes;
  if (few > a) a = few;
  if (!per_head_sizes(h, total_q, batch, pt_stride)) return a;
  const size_t b = carve_head(h, total_q, batch, pt_stride, nullptr).bytes;
  return a > b ? a : b;  // (an fp32 query takes the absorbed form)
}

struct PrefixWorkspace {
  Workspace dec;       // of the decode step over the sequences' own rows (at the workspace's start)
  float* o;            // [2 * batch][vh][d_b]: of the prefixes, of the own rows
  float* lse;          // [2 * batch][vh]
  RowsWorkspace rows;
  size_t bytes;
};
PrefixWorkspace carve_prefix(const mlra_ctx* h, int batch, int groups, void* base) {
  PrefixWorkspace w;
  w.dec = carve(h, batch, base);
  Carver c = {static_cast<char*>(base), w.dec.bytes};
  w.o = c.take<float>((size_t)2 * batch * h->vh * h->d_b);
  w.lse = c.take<float>((size_t)2 * batch * h->vh);
  w.rows = with_rows(h->var, [&](auto sh) {
    return carve_rows<decltype(sh)>(h, c, batch, (size_t)groups + batch, heads_tile_of(h), true);
  });
  w.bytes = c.off;
  return w;
}

// bf16 query rows [tokens][nsub][np][width]; a box is box_cols of `heads` rows of box_tokens tokens.
bool make_rows_map(CUtensorMap* m, const void* q_pack, uint64_t width, uint64_t np, uint64_t nsub, uint64_t tokens,
                   uint32_t box_cols, uint32_t heads, uint32_t box_tokens) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  const uint64_t row = width * 2;
  cuuint64_t dims[4] = {width, np, nsub, tokens};
  cuuint64_t strides[3] = {row, row * np, row * np * nsub};
  cuuint32_t box[4] = {box_cols, heads, 1, box_tokens};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q_pack), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_for(box_cols * 2), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The parts of a launch of the row attention that both callers share.
struct RowsCall {
  const __nv_bfloat16* q_pack;
  int tokens, seqs;
  const int* cu;
  const int* lens;
  const void* pool;          // bf16 pages
  int num_pages;
  const int* page_table;     // null: identity (see RowParams)
  int pt_stride;
  const __nv_bfloat16* kv;   // per-head form: keys and values, RoPE columns
  const __nv_bfloat16* kr;
  bool causal;
  const int* own_lens;       // own rows of every token (see RowPlanParams), or null
  const int* own_table;
  int own_stride;
  RowParams rp;              // results, status (the rest is filled in here)
};

template <class Sh>
RowPlanParams plan_params(const mlra_ctx* h, const RowsCall& c, int* status) {
  RowPlanParams p = {};
  p.cu = c.cu;
  p.lens = c.lens;
  p.batch = c.seqs;
  p.total_q = c.tokens;
  p.cap_len = c.pt_stride * kPage;
  p.causal = c.causal;
  p.own_lens = c.own_lens;
  p.own = c.own_lens != nullptr ? c.tokens : 0;
  p.own_cap = c.own_stride * kPage;
  p.ctas = h->num_sms;
  p.plan = c.rp.plan;
  p.status = status;
  p.tile_tokens = Sh::NQ * (128 / (Sh::SPLIT ? 1 : heads_tile_of(h)));
  p.key_tile = Sh::KT;
  p.units = Sh::SPLIT ? h->cfg.h : h->nsub * Sh::HALVES;
  return p;
}
template <class Sh>
cudaError_t launch_plan(const mlra_ctx* h, const RowsCall& c, int* status, cudaStream_t s) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = launch_cfg(dim3(1), dim3(kPlanThreads), 0, s, true, &attr);
  return cudaLaunchKernelEx(&cfg, mlra_rows_plan_kernel, plan_params<Sh>(h, c, status));
}

template <class Sh>
cudaError_t launch_rows(const mlra_ctx* h, const RowsCall& c, cudaStream_t s) {
  const uint64_t D = h->cfg.d_c + h->d_r;
  RowParams p = c.rp;
  p.page_table = c.page_table;
  p.pt_stride = c.pt_stride;
  p.num_pages = c.num_pages;
  p.own = c.own_lens != nullptr ? c.tokens : 0;
  p.own_table = c.own_table;
  p.own_stride = c.own_stride;
  p.causal = c.causal;
  p.nsub = Sh::SPLIT ? h->cfg.h : h->nsub;
  p.chunks = Sh::SPLIT ? 1 : h->chunks;
  p.heads_tile = Sh::SPLIT ? 1 : heads_tile_of(h);
  p.tok_tile = 128 / p.heads_tile;
  p.heads_block = Sh::SPLIT ? 1 : h->heads_block;
  p.vh = h->vh;
  p.d_c = h->cfg.d_c;
  CUtensorMap mc, mr, mqc, mqr;
  if (Sh::SPLIT) {
    // keys and values of a head: rows of 2 * d_h; the queries as they came
    const uint64_t rows = (uint64_t)c.seqs * seq_rows_of(c.pt_stride), w = Sh::DB + Sh::DV;
    p.seq_rows = (int)seq_rows_of(c.pt_stride);
    p.kv_rows = (int)rows;
    if (!make_map(&mc, c.kv, rows * h->cfg.h, w, w * 2, Sh::KT, Sh::CW) ||
        !make_map(&mr, c.kr, rows, h->d_r, (uint64_t)h->d_r * 2, Sh::KT, Sh::RW) ||
        !make_rows_map(&mqc, c.q_pack, h->cfg.d_h + h->d_r, 1, h->cfg.h, c.tokens, Sh::CW, 1, 128) ||
        !make_rows_map(&mqr, c.q_pack, h->cfg.d_h + h->d_r, 1, h->cfg.h, c.tokens, Sh::RW, 1, 128))
      return cudaErrorInvalidValue;
  } else if (!make_map(&mc, c.pool, (uint64_t)c.num_pages * kPage, D, D * 2, kPage, Sh::CW) ||
             !make_map(&mr, c.pool, (uint64_t)c.num_pages * kPage, D, D * 2, kPage, Sh::RW) ||
             !make_rows_map(&mqc, c.q_pack, h->d_b + h->d_r, h->np, h->nsub, c.tokens, Sh::CW, p.heads_tile, p.tok_tile) ||
             !make_rows_map(&mqr, c.q_pack, h->d_b + h->d_r, h->np, h->nsub, c.tokens, Sh::RW, p.heads_tile, p.tok_tile)) {
    return cudaErrorInvalidValue;
  }
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = launch_cfg(dim3(h->num_sms), dim3(Sh::THREADS), Sh::SMEM, s, true, &attr);
  return cudaLaunchKernelEx(&cfg, mlra_rows_kernel<Sh>, mc, mr, mqc, mqr, p);
}

template <class Sh>
cudaError_t launch_merge(const mlra_ctx* h, const RowsCall& c, cudaStream_t s) {
  MergeParams m = {};
  m.plan = c.rp.plan;
  m.causal = c.causal;
  m.key_tile = Sh::KT;
  m.halves = Sh::HALVES;
  m.chunks = Sh::SPLIT ? 1 : h->chunks;
  m.heads_tile = Sh::SPLIT ? 1 : heads_tile_of(h);
  m.tok_tile = 128 / m.heads_tile;
  m.heads_block = Sh::SPLIT ? 1 : h->heads_block;
  m.vh = h->vh;
  m.db = Sh::DB;
  m.dv = Sh::DV;
  m.rows = Sh::ROWS;
  m.part_o = c.rp.part_o;
  m.part_lse = c.rp.part_lse;
  m.o_bf16 = c.rp.o_bf16;
  m.o_f32 = c.rp.o_f32;
  m.lse = c.rp.lse;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = launch_cfg(dim3(h->num_sms, Sh::ROWS / 8), dim3(256), 0, s, true, &attr);
  return cudaLaunchKernelEx(&cfg, mlra_rows_merge_kernel, m);
}

// Keys and values of every head for the per-head form.
template <int DBB>
cudaError_t launch_expand(const mlra_ctx* h, const UpParams& up, const __nv_bfloat16* kv, cudaStream_t s) {
  using Sh = ExpandShape<DBB>;
  CUtensorMap mc, mkv;
  const uint64_t D = h->cfg.d_c + h->d_r, w = 2 * h->cfg.d_h;
  if (!make_map(&mc, up.pool, (uint64_t)up.num_pages * kPage, D, D * 2, kPage, Sh::CW) ||
      !make_map(&mkv, kv, (uint64_t)up.kv_rows * h->cfg.h, w, w * 2, 128, 64))
    return cudaErrorInvalidValue;
  const int per_sm = 2 * (Sh::SMEM + 1024) <= 227 * 1024 ? 2 : 1;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = launch_cfg(dim3(h->num_sms * per_sm), dim3(Sh::THREADS), Sh::SMEM, s, true, &attr);
  return cudaLaunchKernelEx(&cfg, mlra_rows_up_kernel<Sh, true>, h->map_wuk, h->map_wuv, mc, mkv, up);
}

template <int DBB, int DH, int SUMK>
cudaError_t launch_up(const mlra_ctx* h, const __nv_bfloat16* o, int tokens, const UpParams& up, cudaStream_t s) {
  using Sh = UpShape<DBB, DH, SUMK>;
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return cudaErrorInvalidValue;
  CUtensorMap mo;
  cuuint64_t dims[3] = {(cuuint64_t)DBB, (cuuint64_t)h->vh, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)DBB * 2, (cuuint64_t)h->vh * DBB * 2};
  cuuint32_t box[3] = {(cuuint32_t)Sh::CW, 1, 128};
  cuuint32_t estr[3] = {1, 1, 1};
  if (fn(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(o), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_for(Sh::CW * 2), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // two CTAs an SM where shared memory holds them; no more CTAs than (head, token tile) items
  const int per_sm = 2 * (Sh::SMEM + 1024) <= 227 * 1024 ? 2 : 1;
  const long long items = (long long)up.heads * ((tokens + 127) / 128);
  const int grid = (int)(items < (long long)h->num_sms * per_sm ? items : (long long)h->num_sms * per_sm);
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = launch_cfg(dim3(grid), dim3(Sh::THREADS), Sh::SMEM, s, true, &attr);
  return cudaLaunchKernelEx(&cfg, mlra_rows_up_kernel<Sh>, h->map_wuv, h->map_wuv, mo, mo, up);
}

// bf16 absorb for every variant, with the split plan in its first row of blocks (an E4M3 cache's
// scales are in the two query scales).
template <int DB, int DH, int NT>
constexpr int plan_smem() {
  return ProjShape<DB, DH, NT>::SMEM1 > (int)sizeof(PlanShared) ? ProjShape<DB, DH, NT>::SMEM1 : (int)sizeof(PlanShared);
}
template <int DB, int DH>
cudaError_t prep_absorb_rows() {
  cudaError_t e = prep_kernel(mlra_absorb_kernel<ProjShape<DB, DH, 16>, false, true>, plan_smem<DB, DH, 16>());
  if (e == cudaSuccess) e = prep_kernel(mlra_absorb_kernel<ProjShape<DB, DH, 32>, false, true>, plan_smem<DB, DH, 32>());
  if (e == cudaSuccess) e = prep_kernel(mlra_absorb_kernel<ProjShape<DB, DH, 64>, false, true>, plan_smem<DB, DH, 64>());
  if constexpr (max_nt<DB>() >= 128)
    if (e == cudaSuccess)
      e = prep_kernel(mlra_absorb_kernel<ProjShape<DB, DH, 128>, false, true>, plan_smem<DB, DH, 128>());
  return e;
}
template <int DB, int DH, int NT>
cudaError_t launch_absorb_rows(const mlra_ctx* h, const ProjParams& pp, int tokens, cudaStream_t s) {
  using S = ProjShape<DB, DH, NT>;
  CUtensorMap mqc, mqr;
  std::memset(&mqc, 0, sizeof(mqc));
  std::memset(&mqr, 0, sizeof(mqr));
  if (!pp.q_f32) {
    const uint64_t cols = (uint64_t)DH + h->d_r;
    if (!make_q_map(&mqc, pp.q, tokens, h->cfg.h, cols, S::AW, NT, swizzle_for(S::AROWB)) ||
        !make_q_map(&mqr, pp.q, tokens, h->cfg.h, cols, h->d_r, NT, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  }
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c = launch_cfg(dim3(h->vh, (tokens + NT - 1) / NT + 1), dim3(kProjThreads), plan_smem<DB, DH, NT>(),
                                    s, true, &attr);
  return cudaLaunchKernelEx(&c, mlra_absorb_kernel<S, false, true>, h->map_wuk, mqc, mqr, pp);
}
template <int DB, int DH>
cudaError_t dispatch_absorb_plan(const mlra_ctx* h, const ProjParams& pp, int tokens, cudaStream_t s) {
  switch (nt_for(tokens, max_nt<DB>())) {
    case 16: return launch_absorb_rows<DB, DH, 16>(h, pp, tokens, s);
    case 32: return launch_absorb_rows<DB, DH, 32>(h, pp, tokens, s);
    case 64: return launch_absorb_rows<DB, DH, 64>(h, pp, tokens, s);
    default:
      if constexpr (max_nt<DB>() >= 128) return launch_absorb_rows<DB, DH, 128>(h, pp, tokens, s);
      return cudaErrorInvalidValue;
  }
}
cudaError_t dispatch_absorb_rows(const mlra_ctx* h, const ProjParams& pp, int tokens, cudaStream_t s) {
  switch (h->var) {
    case kTiny: return dispatch_absorb_plan<32, 32>(h, pp, tokens, s);
    case kMlra2: case kMlra2Sum: return dispatch_absorb_plan<256, 128>(h, pp, tokens, s);
    case kMla: return dispatch_absorb_plan<512, 128>(h, pp, tokens, s);
    default: return dispatch_absorb_plan<128, 128>(h, pp, tokens, s);
  }
}
cudaError_t prep_absorb_plan(Variant v) {
  switch (v) {
    case kTiny: return prep_absorb_rows<32, 32>();
    case kMlra2: case kMlra2Sum: return prep_absorb_rows<256, 128>();
    case kMla: return prep_absorb_rows<512, 128>();
    default: return prep_absorb_rows<128, 128>();
  }
}

ProjParams absorb_params(const mlra_ctx* h, const void* q, mlra_dtype q_dtype, int tokens, __nv_bfloat16* q_pack,
                         int* status, const EarlyTags& tags) {
  ProjParams pp = {};
  pp.q = q;
  pp.q_f32 = q_dtype == MLRA_F32;
  pp.q_pack = q_pack;
  pp.qscale = pp.qscale_rope = h->scale * kLog2e;
  pp.d_r = h->d_r;
  pp.np = h->np;
  pp.nsub = h->nsub;
  pp.chunks = h->chunks;
  pp.heads_block = h->heads_block;
  pp.batch = tokens;
  pp.h = h->vh;
  pp.q_heads = h->cfg.h;
  pp.out_heads = h->cfg.h;
  pp.out_scale = h->summed ? h->alpha : 1.f;
  pp.q_rows_per_sub = h->np;
  pp.status = status;
  pp.tags = tags;
  pp.wait_limit_ns = kWaitLimitNs;
  return pp;
}

bool rows_sizes_ok(int total_q, int batch, int pt_stride) {
  return total_q >= 0 && total_q <= kMaxQueryTokens && batch > 0 && batch <= kMaxSeqs && pt_stride > 0 &&
         (long long)pt_stride * kPage <= 0x7fffffffLL - kTile;
}

PrefixParts prefix_parts(const mlra_ctx* h, const RowsWorkspace& w, const float* o, const float* lse) {
  PrefixParts pre = {};
  pre.plan = w.plan;
  pre.chunks = h->chunks;
  pre.heads_tile = heads_tile_of(h);
  pre.tok_tile = 128 / pre.heads_tile;
  pre.o_dense = o;
  pre.lse_dense = lse;
  pre.part_o = w.part_o;
  pre.part_lse = w.part_lse;
  with_rows(h->var, [&](auto sh) {
    using Sh = decltype(sh);
    pre.halves = Sh::HALVES;
    pre.rows = Sh::ROWS;
    pre.dv = Sh::DV;
    return 0;
  });
  return pre;
}
cudaError_t dispatch_combine_prefix(const mlra_ctx* h, const ProjParams& pp, int batch, bool own, cudaStream_t s) {
  switch (h->var) {
    case kTiny:
      return h->summed ? dispatch_uproj_prefix<128, 32, 4>(h, pp, batch, own, s) : dispatch_uproj_prefix<32, 32, 1>(h, pp, batch, own, s);
    case kMlra4Sum: return dispatch_uproj_prefix<512, 128, 4>(h, pp, batch, own, s);
    case kMlra2: return dispatch_uproj_prefix<256, 128, 1>(h, pp, batch, own, s);
    case kMlra2Sum: return dispatch_uproj_prefix<512, 128, 2>(h, pp, batch, own, s);
    case kMla: return dispatch_uproj_prefix<512, 128, 1>(h, pp, batch, own, s);
    default: return dispatch_uproj_prefix<128, 128, 1>(h, pp, batch, own, s);
  }
}

// The per-head form (see per_head_sizes): expansion, plan, attention, merge.
int run_prefill_heads(mlra_handle h, const void* q, const int32_t* cu, int total_q, const void* pool, int num_pages,
                      const int32_t* page_table, int pt_stride, const int32_t* seq_lens, int batch, void* out,
                      mlra_dtype out_dtype, float* lse, void* workspace, cudaStream_t s) {
  const HeadWorkspace w = carve_head(h, total_q, batch, pt_stride, workspace);
  const EarlyTags tags = {reinterpret_cast<unsigned*>(w.status) + 1, next_call_tag()};
  UpParams up = {};
  up.heads = h->cfg.h;
  up.status = w.status;
  up.wait_limit_ns = kWaitLimitNs;
  up.tags = tags;
  up.lens = seq_lens;
  up.page_table = page_table;
  up.pt_stride = pt_stride;
  up.batch = batch;
  up.num_pages = num_pages;
  up.heads_block = h->heads_block;
  up.seq_rows = (int)seq_rows_of(pt_stride);
  up.kv_rows = batch * up.seq_rows;
  up.width = h->cfg.d_c + h->d_r;
  up.d_c = h->cfg.d_c;
  up.d_r = h->d_r;
  up.pool = static_cast<const __nv_bfloat16*>(pool);
  up.kr = w.kr;
  RowsCall c = {};
  c.q_pack = static_cast<const __nv_bfloat16*>(q);
  c.tokens = total_q;
  c.seqs = batch;
  c.cu = cu;
  c.lens = seq_lens;
  c.pt_stride = pt_stride;
  c.kv = w.kv;
  c.kr = w.kr;
  c.causal = true;
  c.rp.plan = w.rows.plan;
  c.rp.s_scale = h->scale * kLog2e;
  c.rp.o_scale = 1.f;
  c.rp.o_bf16 = out_dtype == MLRA_BF16 ? static_cast<__nv_bfloat16*>(out) : nullptr;
  c.rp.o_f32 = out_dtype == MLRA_F32 ? static_cast<float*>(out) : nullptr;
  c.rp.lse = lse;
  c.rp.lse_mul = kLn2;
  c.rp.part_o = w.rows.part_o;
  c.rp.part_lse = w.rows.part_lse;
  c.rp.status = w.status;
  c.rp.tags = tags;
  c.rp.wait_limit_ns = kWaitLimitNs;
  g_use_pdl = true;
  cudaError_t e = h->d_b == 128 ? launch_expand<128>(h, up, w.kv, s)
                : h->d_b == 256 ? launch_expand<256>(h, up, w.kv, s) : launch_expand<512>(h, up, w.kv, s);
  if (e == cudaSuccess) e = launch_plan<RowsHead>(h, c, w.status, s);
  if (e == cudaSuccess) e = launch_rows<RowsHead>(h, c, s);
  if (e == cudaSuccess) e = launch_merge<RowsHead>(h, c, s);
  return e == cudaSuccess ? MLRA_OK : MLRA_ERR_CUDA;
}

int run_prefill(mlra_handle h, const void* q, mlra_dtype q_dtype, const int32_t* cu, int total_q, const void* pool,
                int num_pages, const int32_t* page_table, int pt_stride, const int32_t* seq_lens, int batch, void* out,
                mlra_dtype out_dtype, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if (!h || !cu || !pool || !page_table || !seq_lens || !workspace || (total_q > 0 && (!q || !out)))
    return MLRA_ERR_INVALID_ARG;
  if (!rows_sizes_ok(total_q, batch, pt_stride) || num_pages <= 0) return MLRA_ERR_INVALID_ARG;
  if ((q_dtype != MLRA_F32 && q_dtype != MLRA_BF16) || (out_dtype != MLRA_F32 && out_dtype != MLRA_BF16))
    return MLRA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(pool) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return MLRA_ERR_INVALID_ARG;
  if ((long long)(total_q + 127) / 128 * h->cfg.h > 0x7fffffffLL / 2) return MLRA_ERR_UNSUPPORTED;
  if ((long long)num_pages * kPage > 0x7fffffffLL ||
      (h->fp8 && (long long)batch * pt_stride * kPage > 0x7fffffffLL))
    return MLRA_ERR_UNSUPPORTED;
  if (ws_bytes < prefill_bytes(h, total_q, batch, pt_stride)) return MLRA_ERR_WORKSPACE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return MLRA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (total_q == 0) return cudaMemsetAsync(workspace, 0, 4, s) == cudaSuccess ? MLRA_OK : MLRA_ERR_CUDA;
  if (q_dtype == MLRA_BF16 && per_head_sizes(h, total_q, batch, pt_stride))
    return run_prefill_heads(h, q, cu, total_q, pool, num_pages, page_table, pt_stride, seq_lens, batch, out, out_dtype,
                             lse, workspace, s);
  PrefillWorkspace w = carve_prefill(h, total_q, batch, pt_stride, workspace);
  const EarlyTags tags = {reinterpret_cast<unsigned*>(w.status) + 1, next_call_tag()};
  ProjParams pp = absorb_params(h, q, q_dtype, total_q, w.q_pack, w.status, tags);
  // The scores are scaled in the softmax, so that q^R goes in as it is (a bf16 query's is not
  // rounded again). An E4M3 cache's two scales go into the two query parts, relative to the larger.
  const float top = h->fp8 ? (h->latent_scale > h->rope_scale ? h->latent_scale : h->rope_scale) : 1.f;
  pp.qscale = h->fp8 ? h->latent_scale / top : 1.f;
  pp.qscale_rope = h->fp8 ? h->rope_scale / top : 1.f;
  RowsCall c = {};
  c.q_pack = w.q_pack;
  c.tokens = total_q;
  c.seqs = batch;
  c.cu = cu;
  c.lens = seq_lens;
  c.pool = h->fp8 ? static_cast<const void*>(w.pages) : pool;
  c.num_pages = h->fp8 ? batch * pt_stride : num_pages;
  c.page_table = h->fp8 ? nullptr : page_table;
  c.pt_stride = pt_stride;
  c.causal = true;
  c.rp.plan = w.rows.plan;
  c.rp.s_scale = h->scale * kLog2e * top;
  c.rp.o_scale = h->fp8 ? h->latent_scale : 1.f;
  const bool few = few_tokens(h, total_q);
  c.rp.o_bf16 = w.o;
  c.rp.o_f32 = w.o_few;
  c.rp.lse = few ? w.lse_few : lse;
  c.rp.lse_mul = few ? 1.f : kLn2;
  c.rp.part_o = w.rows.part_o;
  c.rp.part_lse = w.rows.part_lse;
  c.rp.status = w.status;
  c.rp.tags = tags;
  c.rp.wait_limit_ns = kWaitLimitNs;
  if (few) {
    pp.out = out;
    pp.out_f32 = out_dtype == MLRA_F32;
    pp.lse_out = lse;
    pp.groups = h->groups;
    pp.prefix = prefix_parts(h, w.rows, w.o_few, w.lse_few);
  }

  pp.rows = with_rows(h->var, [&](auto sh) { return plan_params<decltype(sh)>(h, c, w.status); });
  g_use_pdl = true;
  cudaError_t e = dispatch_absorb_rows(h, pp, total_q, s);
  if (e == cudaSuccess && h->fp8) {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = launch_cfg(dim3(pt_stride, batch), dim3(256), 0, s, true, &attr);
    e = cudaLaunchKernelEx(&cfg, mlra_widen_pages_kernel, static_cast<const uint8_t*>(pool), num_pages, page_table,
                           pt_stride, seq_lens, h->cfg.d_c + h->d_r, w.pages, w.status);
  }
  if (e == cudaSuccess)
    e = with_rows(h->var, [&](auto sh) {
      using Sh = decltype(sh);
      const cudaError_t r = launch_rows<Sh>(h, c, s);
      return r == cudaSuccess && !few ? launch_merge<Sh>(h, c, s) : r;
    });
  if (few) {
    if (e == cudaSuccess) e = dispatch_combine_prefix(h, pp, total_q, false, s);
  } else if (e == cudaSuccess) {
    UpParams up = {};
    up.used = w.rows.plan.hdr + 1;
    up.out = out;
    up.out_f32 = out_dtype == MLRA_F32;
    up.heads = h->cfg.h;
    up.total = total_q;
    up.out_scale = h->summed ? h->alpha : 1.f;
    up.status = w.status;
    up.wait_limit_ns = kWaitLimitNs;
    switch (h->var) {
      case kTiny: e = h->summed ? launch_up<32, 32, 4>(h, w.o, total_q, up, s) : launch_up<32, 32, 1>(h, w.o, total_q, up, s); break;
      case kMlra2: e = launch_up<256, 128, 1>(h, w.o, total_q, up, s); break;
      case kMlra2Sum: e = launch_up<256, 128, 2>(h, w.o, total_q, up, s); break;
      case kMla: e = launch_up<512, 128, 1>(h, w.o, total_q, up, s); break;
      case kMlra4Sum: e = launch_up<128, 128, 4>(h, w.o, total_q, up, s); break;
      default: e = launch_up<128, 128, 1>(h, w.o, total_q, up, s); break;
    }
  }
  return e == cudaSuccess ? MLRA_OK : MLRA_ERR_CUDA;
}

// Whether the attention kernel of a shared-prefix step takes the sequences' own rows too, each a
// sequence of one token, in place of a decode kernel before it. That saves a link of the chain and
// shares the GPU better, but a 128-row tile then holds one token's heads, and every unit of them costs
// a query load and an epilogue: for few sequences with few own rows (their number is known on the device
// only; the host goes by the table's capacity). Measured behind a prefix of 4096 rows, 128 heads, against
// the decode kernel, by sequences and own rows up to: d_b = 128: 35 and 47 us at 4 and 64, 50 and 57 at 32
// and 512, 67 and 63 at 32 and 2048, 75 and 76 at 64 and 512, 127 and 107 at 128 and 192; d_b = 256: 62 and
// 77 at 32 and 512, 99 and 105 at 64 and 512, 213 and 141 at 128 and 64; d_b = 512: 95 and 108 at 16 and
// 256, 294 and 286 at 64 and 512.
bool own_in_rows(const mlra_ctx* h, int batch, int groups, int pt_stride) {
  if (batch > 64 || groups + batch > kMaxSeqs) return false;
  return with_rows(h->var, [&](auto sh) {
    using Sh = decltype(sh);
    const long long tiles = ((long long)pt_stride * kPage + Sh::KT - 1) / Sh::KT;
    return (long long)batch * h->nsub * Sh::HALVES * (tiles + 1) <= 12LL * h->num_sms;
  });
}

int run_decode_prefix(mlra_handle h, const void* q, mlra_dtype q_dtype, const void* pool, int num_pages,
                      const int32_t* prefix_table, int prefix_stride, const int32_t* prefix_lens,
                      const int32_t* group_offsets, int groups, const int32_t* page_table, int pt_stride,
                      const int32_t* seq_lens, int batch, void* out, mlra_dtype out_dtype, float* lse,
                      void* workspace, size_t ws_bytes, void* stream) {
  if (!h || !q || !pool || !prefix_table || !prefix_lens || !group_offsets || !page_table || !seq_lens || !out ||
      !workspace)
    return MLRA_ERR_INVALID_ARG;
  if (h->fp8) return MLRA_ERR_UNSUPPORTED;
  if (!rows_sizes_ok(batch, groups, prefix_stride) || !rows_sizes_ok(batch, batch, pt_stride) || batch <= 0 ||
      num_pages <= 0)
    return MLRA_ERR_INVALID_ARG;
  if ((q_dtype != MLRA_F32 && q_dtype != MLRA_BF16) || (out_dtype != MLRA_F32 && out_dtype != MLRA_BF16))
    return MLRA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(pool) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return MLRA_ERR_INVALID_ARG;
  if ((long long)num_pages * kPage > 0x7fffffffLL) return MLRA_ERR_UNSUPPORTED;
  PrefixWorkspace w = carve_prefix(h, batch, groups, workspace);
  if (ws_bytes < w.bytes) return MLRA_ERR_WORKSPACE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return MLRA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const EarlyTags tags = {reinterpret_cast<unsigned*>(w.dec.status) + 1, next_call_tag()};
  ProjParams pp = absorb_params(h, q, q_dtype, batch, w.dec.q_pack, w.dec.status, tags);
  pp.o_part = w.dec.o_part;
  pp.lse_part = w.dec.lse_part;
  pp.out = out;
  pp.out_f32 = out_dtype == MLRA_F32;
  pp.lse_out = lse;
  const bool own = own_in_rows(h, batch, groups, pt_stride);
  pp.seq_lens = own ? nullptr : seq_lens;
  pp.pt_stride = pt_stride;
  pp.groups = h->groups;

  RowsCall c = {};
  if (own) {
    c.own_lens = seq_lens;
    c.own_table = page_table;
    c.own_stride = pt_stride;
  }
  c.q_pack = w.dec.q_pack;
  c.tokens = batch;
  c.seqs = groups;
  c.cu = group_offsets;
  c.lens = prefix_lens;
  c.pool = pool;
  c.num_pages = num_pages;
  c.page_table = prefix_table;
  c.pt_stride = prefix_stride;
  c.causal = false;
  c.rp.plan = w.rows.plan;
  c.rp.s_scale = 1.f;
  c.rp.o_scale = 1.f;
  c.rp.o_f32 = w.o;
  c.rp.lse = w.lse;
  c.rp.lse_mul = 1.f;
  c.rp.part_o = w.rows.part_o;
  c.rp.part_lse = w.rows.part_lse;
  c.rp.status = w.dec.status;
  c.rp.tags = tags;
  c.rp.wait_limit_ns = kWaitLimitNs;

  DecodeParams dp = {};
  dp.seq_lens = seq_lens;
  dp.page_table = page_table;
  dp.pt_stride = pt_stride;
  dp.batch = batch;
  dp.num_pages = num_pages;
  dp.groups = h->groups;
  dp.nsub = h->nsub;
  dp.chunks = h->chunks;
  dp.heads_block = h->heads_block;
  dp.h = h->vh;
  dp.d_c = h->cfg.d_c;
  dp.q_rows = h->heads_block < h->np ? h->heads_block : h->np;
  dp.o_scale = 1.f;
  dp.o_part = w.dec.o_part;
  dp.lse_part = w.dec.lse_part;
  dp.status = w.dec.status;
  dp.tags = tags;
  dp.wait_limit_ns = kWaitLimitNs;

  pp.prefix = prefix_parts(h, w.rows, w.o, w.lse);

  const int D = h->cfg.d_c + h->d_r;
  const int cw = h->d_b < 64 ? h->d_b : 64, rw = h->d_r < 64 ? h->d_r : 64;
  CUtensorMap mc, mr, mqc, mqr;
  const uint64_t qrows = (uint64_t)batch * h->nsub * h->np, qw = h->d_b + h->d_r;
  if (!make_map(&mc, pool, (uint64_t)num_pages * kPage, D, (uint64_t)D * 2, kPage, cw) ||
      !make_map(&mr, pool, (uint64_t)num_pages * kPage, D, (uint64_t)D * 2, kPage, rw) ||
      !make_map(&mqc, w.dec.q_pack, qrows, qw, qw * 2, dp.q_rows, cw) ||
      !make_map(&mqr, w.dec.q_pack, qrows, qw, qw * 2, dp.q_rows, rw))
    return MLRA_ERR_CUDA;

  pp.rows = with_rows(h->var, [&](auto sh) { return plan_params<decltype(sh)>(h, c, w.dec.status); });
  g_use_pdl = true;
  cudaError_t e = dispatch_absorb_rows(h, pp, batch, s);
  if (e == cudaSuccess && !own) switch (h->var) {
      case kTiny: e = launch_decode<DecTiny>(h, mc, mr, mqc, mqr, dp, s); break;
      case kMlra4: e = launch_decode<DecMlra4>(h, mc, mr, mqc, mqr, dp, s); break;
      case kMlra4Sum: e = launch_decode<DecMlra4Sum>(h, mc, mr, mqc, mqr, dp, s); break;
      case kMla: e = launch_decode<DecMla>(h, mc, mr, mqc, mqr, dp, s); break;
      default: e = launch_decode<DecMlra2>(h, mc, mr, mqc, mqr, dp, s); break;
    }
  if (e == cudaSuccess) e = with_rows(h->var, [&](auto sh) { return launch_rows<decltype(sh)>(h, c, s); });
  if (e == cudaSuccess) e = dispatch_combine_prefix(h, pp, batch, own, s);
  return e == cudaSuccess ? MLRA_OK : MLRA_ERR_CUDA;
}

}  // namespace
