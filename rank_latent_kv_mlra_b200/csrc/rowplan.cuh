// rowplan.cuh - the split of attention over many query rows: token tiles, units, and the stretch of
// units that each CTA of the attention kernel takes (see rows.cuh).
#pragma once

#include "common.cuh"

namespace mlra {

// cost of a unit beyond its key tiles, in key tiles: query load, pipeline fill and epilogue
constexpr int kUnitCost = 1;

// ---------------------------------------------------------------------------------------
// The plan
// ---------------------------------------------------------------------------------------
// A token tile: `ntok` query tokens from `tok0` (row index into the packed queries) of sequence b.
// Token i of the tile sees keys [0, lim0 + i) when causal, [0, lim0) otherwise (lim0 may be <= 0).
struct TokenTile {
  int b, tok0, ntok, lim0;
};
struct RowPlan {
  int* hdr;            // [0] token tiles, [1] tokens in use (cu[batch]), [2] bad lengths found,
                       // [3] token tiles without a key, [4, 5] length of a stretch, [6, 7] of the line
  int4* first;         // [3 * CTAs] where each CTA's stretch begins: tile, its key tiles, its begin and
                       // end on the line; the tile
  long long* start;    // [max tiles + 1] position of each tile's first unit; the last is the total
  TokenTile* tile;     // [max tiles]
  int* base;           // [batch + 1] first token tile of each sequence
  int4* tok;           // [tokens] begin of the token's tile on the line (two words), the tile's key
                       // tiles (0: none, or no sequence), the token's place in it; or null. With own
                       // rows, then the same [tokens] of those
  int4* cut;           // [2 * CTAs] the unit each CTA's stretch goes on with: first and last CTA, unit;
                       // first token, tokens (written by the attention kernel, for the merge)
};
struct RowPlanParams {
  const int* cu;       // [batch + 1] first query token of each sequence
  const int* lens;     // [batch] cached tokens of each sequence
  int batch, total_q, cap_len;
  int tile_tokens, key_tile, units;  // tokens a token tile, keys a key tile, units a token tile
  int causal;
  int ctas;            // of the attention kernel
  // `own` sequences (total_q, or 0) in front of those of cu: sequence b is token b alone and sees
  // own_lens[b] cached rows
  const int* own_lens;
  int own, own_cap;
  RowPlan plan;
  int* status;
};

__device__ __forceinline__ int tile_limit(const TokenTile& t, int causal) {
  const int l = causal ? t.lim0 + t.ntok - 1 : t.lim0;
  return l > 0 ? l : 0;
}
__device__ __forceinline__ int key_tiles(const TokenTile& t, int causal, int key_tile) {
  return (tile_limit(t, causal) + key_tile - 1) / key_tile;
}
__device__ __forceinline__ int unit_cost(int kv) { return kv > 0 ? kv + kUnitCost : 0; }

// A CTA's stretch of the line of units.
struct Stretch {
  long long lo, hi, quota;
};
__device__ __forceinline__ Stretch stretch_of(long long total, int cta, int ctas) {
  Stretch s;
  s.quota = total > 0 ? (total + ctas - 1) / ctas : 1;
  s.lo = min((long long)cta * s.quota, total);
  s.hi = min(s.lo + s.quota, total);
  return s;
}

__device__ __forceinline__ long long join64(int lo, int hi) {
  return (long long)(((unsigned long long)(unsigned)hi << 32) | (unsigned)lo);
}

constexpr int kPlanThreads = 1024;
constexpr int kMaxSeqs = 4096;
constexpr int kPlanStarts = 2048;  // positions kept in shared memory for the search at the end

// Exclusive scan over the block's threads (32 warps at most); scratch holds a value a warp. Every
// thread must have read the last call's result before the next call writes scratch: the first
// barrier sees to that.
template <class T>
__device__ __forceinline__ T warp_inclusive_scan(T x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  return x;
}
template <class T>
__device__ __forceinline__ T block_exclusive_scan(T v, T* scratch, T* total) {
  const T x = warp_inclusive_scan(v);
  __syncthreads();
  if (lane_id() == 31) scratch[warp_id()] = x;
  __syncthreads();
  // every warp scans the warps' sums
  const int nw = blockDim.x >> 5;
  const T s = warp_inclusive_scan(lane_id() < nw ? scratch[lane_id()] : T(0));
  *total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, max(warp_id() - 1, 0));
  return (warp_id() > 0 ? before : T(0)) + x - v;
}

// Shared memory of the planning block.
struct PlanShared {
  int base[kMaxSeqs + 1];   // first token tile of each sequence
  long long starts[kPlanStarts];
  long long scratch[32];
  int scratch_i[32];
  int flags[2];             // bad lengths; tiles without a key
};

// The plan, by one block (a multiple of 32 threads). Returns the bad lengths found. Bound by
// latency: a block scan for as many token tiles as there are threads.
__device__ __forceinline__ int make_row_plan(const RowPlanParams& p, PlanShared& sh) {
  int* const base = sh.base;
  long long* const starts = sh.starts;
  long long* const scratch = sh.scratch;
  int* const scratch_i = sh.scratch_i;
  int* const flags = sh.flags;
  const int threads = blockDim.x;
  if (threadIdx.x < 2) flags[threadIdx.x] = 0;
  __syncthreads();
  int bad = 0;  // 1: a length outside its table row; 2: cu not ascending within [0, total_q]
  int running = 0;
  const int seqs = p.own + p.batch;
  for (int b0 = 0; b0 < seqs; b0 += threads) {
    const int b = b0 + threadIdx.x, c = b - p.own;
    int tiles = 0;
    if (b < p.own) {
      const int n = p.own_lens[b];
      if (n < 0 || n > p.own_cap) bad |= 1;
      tiles = 1;
    } else if (b < seqs) {
      const int lo = p.cu[c], hi = p.cu[c + 1], n = p.lens[c];
      if (lo < 0 || hi < lo || hi > p.total_q || (c == 0 && lo != 0)) bad |= 2;
      else tiles = (hi - lo + p.tile_tokens - 1) / p.tile_tokens;
      if (n < 0 || n > p.cap_len) bad |= 1;
    }
    int all;
    const int first = running + block_exclusive_scan<int>(tiles, scratch_i, &all);
    if (b < seqs) base[b] = first;
    running += all;
  }
  if (bad) atomicOr(&flags[0], bad);
  if (p.plan.tok != nullptr)  // tokens of no sequence
    for (int i = threadIdx.x; i < p.total_q + p.own; i += threads) p.plan.tok[i] = make_int4(0, 0, 0, 0);
  __syncthreads();
  // packed offsets that do not ascend leave no work at all (but the own rows)
  const int tiles = (flags[0] & 2) ? p.own : running;
  if (threadIdx.x == 0) base[seqs] = running;
  __syncthreads();
  for (int b = threadIdx.x; b <= seqs; b += threads) p.plan.base[b] = base[b];
  long long pos = 0;
  for (int i0 = 0; i0 < tiles; i0 += threads) {
    const int i = i0 + threadIdx.x;
    long long cost = 0;
    TokenTile t = {0, 0, 0, 0};
    if (i < tiles) {
      int lo = 0, hi = seqs;  // last b with base[b] <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= i) lo = mid;
        else hi = mid;
      }
      const bool own = lo < p.own;
      const int c0 = own ? lo : p.cu[lo - p.own], n_q = own ? 1 : p.cu[lo - p.own + 1] - c0;
      const int cap = own ? p.own_cap : p.cap_len;
      int len = own ? p.own_lens[lo] : p.lens[lo - p.own];
      len = len < 0 ? 0 : len > cap ? cap : len;
      const int first = (i - base[lo]) * p.tile_tokens;
      t.b = lo;
      t.tok0 = c0 + first;
      t.ntok = min(p.tile_tokens, n_q - first);
      t.lim0 = p.causal ? len - n_q + first + 1 : len;
      cost = (long long)unit_cost(key_tiles(t, p.causal, p.key_tile)) * p.units;
      if (cost == 0) atomicAdd(&flags[1], 1);
    }
    long long all;
    const long long at = pos + block_exclusive_scan<long long>(cost, scratch, &all);
    if (i < tiles) {
      p.plan.start[i] = at;
      p.plan.tile[i] = t;
      if (i < kPlanStarts) starts[i] = at;
      if (p.plan.tok != nullptr)
        for (int j = 0; j < t.ntok; ++j)
          p.plan.tok[(t.b < p.own ? p.total_q : 0) + t.tok0 + j] = make_int4((int)at, (int)(at >> 32), key_tiles(t, p.causal, p.key_tile), j);
    }
    pos += all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.plan.hdr[3] = flags[1];
    p.plan.start[tiles] = pos;
    p.plan.hdr[0] = tiles;
    p.plan.hdr[1] = p.own > 0 ? p.total_q : (flags[0] & 2) ? 0 : p.cu[p.batch];
    p.plan.hdr[2] = flags[0];
    const long long quota = stretch_of(pos, 0, p.ctas).quota;
    p.plan.hdr[4] = (int)quota;
    p.plan.hdr[5] = (int)(quota >> 32);
    p.plan.hdr[6] = (int)pos;
    p.plan.hdr[7] = (int)(pos >> 32);
    if (tiles < kPlanStarts) starts[tiles] = pos;
  }
  __syncthreads();
  // where each CTA begins, so that it need not search
  for (int c = threadIdx.x; c < p.ctas; c += threads) {
    const Stretch s = stretch_of(pos, c, p.ctas);
    if (s.lo >= s.hi) continue;
    const long long* st = tiles < kPlanStarts ? starts : p.plan.start;
    int lo = 0, up = tiles;  // the last tile with start <= lo (tiles without work share their start with the next)
    while (up - lo > 1) {
      const int mid = (lo + up) >> 1;
      if (st[mid] <= s.lo) lo = mid;
      else up = mid;
    }
    const TokenTile t = p.plan.tile[lo];
    const long long at = st[lo], nx = st[lo + 1];
    p.plan.first[3 * c] = make_int4(lo, key_tiles(t, p.causal, p.key_tile), (int)at, (int)(at >> 32));
    p.plan.first[3 * c + 1] = make_int4((int)nx, (int)(nx >> 32), 0, 0);
    p.plan.first[3 * c + 2] = make_int4(t.b, t.tok0, t.ntok, t.lim0);
  }
  return flags[0];
}

// As a kernel of its own (behind the expansion, which clears the status word).
__global__ void __launch_bounds__(kPlanThreads, 1) mlra_rows_plan_kernel(const RowPlanParams p) {
  __shared__ PlanShared sh;
  grid_launch_dependents();
  // Its inputs were there before the call and its outputs are read by later kernels of the call only;
  // the kernel in front of it waited for the work before the call.
  const int bad = make_row_plan(p, sh);
  grid_dependency_wait();
  if (threadIdx.x == 0 && bad) set_status(p.status, kErrSeqLen);
}

// One unit's key tiles that lie in a stretch.
struct UnitPart {
  TokenTile t;
  int sub;            // unit within the token tile: latent block, head chunk, column half
  int kv;             // key tiles of the whole unit
  int begin, end;     // key tiles in this stretch (begin < end, or the walk has ended)
  bool valid;
};
// Walks the unit parts of a stretch in order. One warp calls it (all lanes, same results).
struct UnitWalk {
  const RowPlan* plan;
  long long pos, hi, at, nx;  // at, nx: where token tile i begins and ends on the line
  int i, tiles, units, key_tile, causal;
  TokenTile t;
  int kv;
  // whole units in turn instead of a stretch (see whole_units): CTA c takes units c, c + step, ... of
  // an order that goes through a sequence's sub-units one after the other, long units first
  int unit, step;
  __device__ __forceinline__ void load() {
    at = __ldg(plan->start + i);
    nx = __ldg(plan->start + i + 1);
    const int4 raw = __ldg(reinterpret_cast<const int4*>(plan->tile + i));
    t.b = raw.x; t.tok0 = raw.y; t.ntok = raw.z; t.lim0 = raw.w;
    kv = key_tiles(t, causal, key_tile);
  }
  __device__ __forceinline__ void init(const RowPlan* pl, int tiles_, const Stretch& s, int cta, int units_,
                                       int key_tile_, int causal_) {
    plan = pl;
    pos = s.lo;
    hi = s.hi;
    units = units_;
    key_tile = key_tile_;
    causal = causal_;
    tiles = tiles_;
    const int4 a = __ldg(pl->first + 3 * cta), b = __ldg(pl->first + 3 * cta + 1), raw = __ldg(pl->first + 3 * cta + 2);
    i = a.x;
    kv = a.y;
    at = join64(a.z, a.w);
    nx = join64(b.x, b.y);
    t.b = raw.x; t.tok0 = raw.y; t.ntok = raw.z; t.lim0 = raw.w;
  }
  __device__ __forceinline__ void init_whole(const RowPlan* pl, int tiles_, int cta, int ctas, int units_, int key_tile_,
                                             int causal_) {
    plan = pl;
    tiles = tiles_;
    units = units_;
    key_tile = key_tile_;
    causal = causal_;
    unit = cta;
    step = ctas;
    pos = hi = 0;
  }
  __device__ __forceinline__ UnitPart next_whole() {
    UnitPart u;
    u.valid = false;
    u.begin = u.end = u.kv = u.sub = 0;
    u.t = {0, 0, 0, 0};
    for (; unit < tiles * units; unit += step) {
      const int b = __ldg(&plan->tile[unit / units].b);
      const int first = __ldg(plan->base + b), n = __ldg(plan->base + b + 1) - first;
      const int r = unit - first * units;  // within the sequence's units
      i = first + n - 1 - r % n;
      const int4 raw = __ldg(reinterpret_cast<const int4*>(plan->tile + i));
      u.t.b = raw.x; u.t.tok0 = raw.y; u.t.ntok = raw.z; u.t.lim0 = raw.w;
      u.kv = u.end = key_tiles(u.t, causal, key_tile);
      if (u.kv == 0) continue;
      u.sub = r / n;
      u.valid = true;
      unit += step;
      return u;
    }
    return u;
  }
  __device__ __forceinline__ UnitPart next() {
    UnitPart u;
    u.valid = false;
    u.begin = u.end = u.kv = u.sub = 0;
    u.t = {0, 0, 0, 0};
    while (pos < hi) {
      if (pos >= nx) {
        ++i;
        load();
        continue;
      }
      const int cost = unit_cost(kv);
      u.sub = (int)((unsigned long long)(pos - at) / (unsigned)cost);
      const long long first = at + (long long)u.sub * cost;
      const long long b = pos - first - kUnitCost, e = hi - first - kUnitCost;
      u.begin = b > 0 ? (int)b : 0;
      u.end = e < kv ? (int)e : kv;
      pos = first + cost;
      if (u.end > u.begin) {
        u.t = t;
        u.kv = kv;
        u.valid = true;
        return u;
      }
    }
    return u;
  }
};

}  // namespace mlra
