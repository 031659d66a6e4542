// pages.cuh - the pages of the cache on the device: reserving, forking, freeing, compacting.
//
// The pool's state is one count a page, refs[p]: how many page-table entries hold page p (0: free).
// New pages are the lowest-numbered free ones, in the order of the requests, so every result is the
// same whatever the timing. To hand out the i-th free page without a list to keep, the first kernel
// of a call turns the counts into a bitmap of free pages with one sum for each 8192; the second
// kernel finds a page by a search over those sums and a warp's scan of one 8192-bit stretch. The
// counts are read once (4 bytes a page) and never while another block changes them.
#pragma once

#include "common.cuh"
#include "rowplan.cuh"

namespace mlra {

constexpr int kErrNoPages = -10;
constexpr int kSuperWords = 256;                 // bitmap words a sum covers
constexpr int kSuperPages = 32 * kSuperWords;    // 8192 pages
constexpr int kMaxSupers = 4096;                 // 2^25 pages
constexpr int kMaxRows = 65536;                  // rows of the page table
constexpr int kPagesThreads = 256;

enum class PageOp { kReserve, kFork, kFree };

struct PagesParams {
  int* refs;
  int num_pages;
  int* page_table;
  int pt_stride, batch;
  int* seq_lens;
  const int* ids;        // [n] sequences to grow / to free / to fork from
  const int* arg;        // [n] new lengths / sequences to fork onto
  int n;
  // workspace
  uint32_t* free_bits;   // [supers * kSuperWords] bit set: free
  int* super_free;       // [supers] free pages of each stretch
  int* rank;             // [n] pages the requests before it take
  int* first;            // [n] first page index the request writes
  int* ctl;              // [0] an error was found: nothing is changed; [1] pages taken in all
  int* status;
  // fork, compact
  char* pool;
  int row_bytes;         // bytes of a cached row
  int* remap;            // [num_pages] new place of a moved page (compact)
  int* used;             // compact: receives the number of used pages, or null
};

__device__ __forceinline__ int pages_of(int n) { return (n + kPage - 1) / kPage; }

// Checks the requests (one block). A sequence named twice, out of range, or whose lengths make no
// sense leaves the whole call without effect.
template <PageOp OP>
__device__ void check_requests(const PagesParams& p) {
  __shared__ uint32_t seen[kMaxRows / 32];
  __shared__ long long scratch[kPagesThreads / 32];
  __shared__ int bad;
  const int cap = p.pt_stride * kPage;
  if (threadIdx.x == 0) bad = 0;
  for (int i = threadIdx.x; i < (p.batch + 31) / 32; i += blockDim.x) seen[i] = 0;
  __syncthreads();
  bool wrong = false;
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
    const int id = OP == PageOp::kFork ? p.arg[i] : p.ids[i];  // the rows the call writes
    if (id < 0 || id >= p.batch) {
      wrong = true;
      continue;
    }
    if ((atomicOr(&seen[id >> 5], 1u << (id & 31)) >> (id & 31)) & 1) wrong = true;
    const int len = p.seq_lens[id];
    if (len < 0 || len > cap) wrong = true;
    if (OP == PageOp::kFork && len != 0) wrong = true;  // forks go onto empty rows
    if (OP == PageOp::kReserve && (p.arg[i] < len || p.arg[i] > cap)) wrong = true;
  }
  __syncthreads();
  if (OP == PageOp::kFork)
    for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
      const int id = p.ids[i];
      if (id < 0 || id >= p.batch || ((seen[id >> 5] >> (id & 31)) & 1) || p.seq_lens[id] < 0 || p.seq_lens[id] > cap)
        wrong = true;
    }
  if (wrong) bad = 1;
  __syncthreads();
  long long taken = 0;
  if (OP != PageOp::kFree && !bad)
    for (int i0 = 0; i0 < p.n; i0 += blockDim.x) {
      const int i = i0 + threadIdx.x;
      int need = 0, first = 0;
      if (i < p.n) {
        const int len = p.seq_lens[p.ids[i]];
        first = OP == PageOp::kFork ? len / kPage : pages_of(len);
        need = OP == PageOp::kFork ? (len % kPage != 0) : pages_of(p.arg[i]) - first;
      }
      // (64 bits: many rows may ask for more than the pool could ever hold)
      long long all;
      const long long before = block_exclusive_scan<long long>(need, scratch, &all);
      if (i < p.n) {
        p.rank[i] = (int)min(taken + before, (long long)p.num_pages);
        p.first[i] = first;
      }
      taken += all;
      __syncthreads();
    }
  if (threadIdx.x == 0) {
    p.ctl[0] = bad;
    p.ctl[1] = (int)min(taken, (long long)p.num_pages + 1);
    *p.status = bad ? kErrSeqLen : kOk;
  }
}

// Block b > 0 (b >= 0 where there are no requests to check): the bitmap of stretch b - 1, a warp
// 1024 pages. Reads 4 bytes a page.
template <bool CHECK, PageOp OP>
__global__ void __launch_bounds__(kPagesThreads) mlra_pages_scan_kernel(const PagesParams p) {
  __shared__ int sums[kPagesThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  if (CHECK && blockIdx.x == 0) {
    check_requests<OP>(p);
    return;
  }
  const int s = blockIdx.x - (CHECK ? 1 : 0);
  const int warp = warp_id(), lane = lane_id();
  const long long base = (long long)s * kSuperPages + warp * 1024;
  uint32_t word = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const long long pg = base + i * 32 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, pg < p.num_pages && p.refs[pg] == 0);
    if (lane == i) word = m;
  }
  p.free_bits[(size_t)s * kSuperWords + warp * 32 + lane] = word;
  int c = __popc(word);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  if (lane == 0) sums[warp] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int all = 0;
    for (int w = 0; w < kPagesThreads / 32; ++w) all += sums[w];
    p.super_free[s] = all;
    if (!CHECK && s == 0) *p.status = kOk;
  }
}

// Free pages before each stretch, in shared memory; returns their number in all.
__device__ __forceinline__ int load_prefix(const PagesParams& p, int* prefix, int* scratch) {
  const int supers = (p.num_pages + kSuperPages - 1) / kSuperPages;
  int running = 0;
  for (int i0 = 0; i0 < supers; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    int all;
    const int before = block_exclusive_scan<int>(i < supers ? p.super_free[i] : 0, scratch, &all);
    if (i < supers) prefix[i] = running + before;
    running += all;
    __syncthreads();
  }
  return running;
}

// The page of rank r (from 0) among the free pages (USED: among the used ones), by one warp.
template <bool USED>
__device__ __forceinline__ int select_page(const PagesParams& p, const int* prefix, int r) {
  const int supers = (p.num_pages + kSuperPages - 1) / kSuperPages;
  int lo = 0, hi = supers;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int before = USED ? mid * kSuperPages - prefix[mid] : prefix[mid];
    if (before <= r) lo = mid;
    else hi = mid;
  }
  r -= USED ? lo * kSuperPages - prefix[lo] : prefix[lo];
  const uint4* src = reinterpret_cast<const uint4*>(p.free_bits + (size_t)lo * kSuperWords) + 2 * lane_id();
  const uint4 a = src[0], b = src[1];
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  int c = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // (bits past the pool's end are zero: they would count as used, but lie behind every used page)
    if (USED) w[e] = ~w[e];
    c += __popc(w[e]);
  }
  int x = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  const unsigned m = __ballot_sync(0xffffffffu, x > r);
  const int owner = m ? __ffs(m) - 1 : 31;
  int page = 0;
  if (lane_id() == owner) {
    int k = r - (x - c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = __popc(w[e]);
      if (k >= 0 && k < n) page = lo * kSuperPages + (owner * 8 + e) * 32 + (int)__fns(w[e], 0, k + 1);
      k -= n;
    }
  }
  return __shfl_sync(0xffffffffu, page, owner);
}

// Whether the call goes ahead: requests in order, enough free pages (the last is reported here).
__device__ __forceinline__ bool go_ahead(const PagesParams& p, int free_pages) {
  if (p.ctl[0]) return false;
  if (p.ctl[1] > free_pages) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = kErrNoPages;
    return false;
  }
  return true;
}

// Grid (requests, slices): a warp a new page.
__global__ void __launch_bounds__(kPagesThreads) mlra_pages_reserve_kernel(const PagesParams p) {
  __shared__ int prefix[kMaxSupers];
  __shared__ int scratch[kPagesThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int free_pages = load_prefix(p, prefix, scratch);
  if (!go_ahead(p, free_pages)) return;
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int id = p.ids[i], len = p.arg[i], first = p.first[i], rank = p.rank[i];
    const int need = pages_of(len) - first;
    for (int x = blockIdx.y * (kPagesThreads / 32) + warp_id(); x < need; x += gridDim.y * (kPagesThreads / 32)) {
      const int page = select_page<false>(p, prefix, rank + x);
      if (lane_id() == 0) {
        p.page_table[(size_t)id * p.pt_stride + first + x] = page;
        p.refs[page] = 1;
      }
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) p.seq_lens[id] = len;
  }
}

// Copies `bytes` (a multiple of 16) with the threads first, first + stride, ...
__device__ __forceinline__ void copy_bytes(char* dst, const char* src, long long bytes, int first, int stride) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int n = (int)(bytes / 16);
  int i = first;
  for (; i + 5 * stride < n; i += 6 * stride) {
    uint4 v[6];
#pragma unroll
    for (int e = 0; e < 6; ++e) v[e] = __ldcs(s + i + e * stride);
#pragma unroll
    for (int e = 0; e < 6; ++e) __stcs(d + i + e * stride, v[e]);
  }
  for (; i < n; i += stride) __stcs(d + i, __ldcs(s + i));
}

// Grid (forks, slices): shares the source's full pages and copies the rows of its partly filled one.
__global__ void __launch_bounds__(kPagesThreads) mlra_pages_fork_kernel(const PagesParams p) {
  __shared__ int prefix[kMaxSupers];
  __shared__ int scratch[kPagesThreads / 32];
  __shared__ int new_page;
  grid_dependency_wait();
  grid_launch_dependents();
  const int free_pages = load_prefix(p, prefix, scratch);
  if (!go_ahead(p, free_pages)) return;
  const int slice = blockIdx.y * blockDim.x + threadIdx.x, slices = gridDim.y * blockDim.x;
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int src = p.ids[i], dst = p.arg[i];
    const int len = p.seq_lens[src], full = p.first[i], part = len - full * kPage;
    const int* from = p.page_table + (size_t)src * p.pt_stride;
    int* to = p.page_table + (size_t)dst * p.pt_stride;
    if (part > 0) {
      if (warp_id() == 0) {
        const int page = select_page<false>(p, prefix, p.rank[i]);
        if (lane_id() == 0) new_page = page;
      }
      __syncthreads();
      const int page = new_page, old = from[full];
      const size_t page_bytes = (size_t)kPage * p.row_bytes;
      if (old >= 0 && old < p.num_pages)
        copy_bytes(p.pool + page * page_bytes, p.pool + old * page_bytes, (long long)part * p.row_bytes, slice, slices);
      else if (slice == 0)
        set_status(p.status, kErrPageOob);
      if (slice == 0) {
        to[full] = page;
        p.refs[page] = 1;
      }
      __syncthreads();
    }
    for (int c = slice; c < full; c += slices) {
      const int page = from[c];
      to[c] = page;
      if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, 1);
      else set_status(p.status, kErrPageOob);
    }
    if (slice == 0) p.seq_lens[dst] = len;
  }
}

// One block a sequence: its entries give their pages back.
__global__ void __launch_bounds__(kPagesThreads) mlra_pages_free_kernel(const PagesParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (p.ctl[0]) return;
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int id = p.ids[i];
    const int n = pages_of(p.seq_lens[id]);
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      const int page = p.page_table[(size_t)id * p.pt_stride + c];
      if (page >= 0 && page < p.num_pages) atomicSub(p.refs + page, 1);
      else set_status(p.status, kErrPageOob);
    }
    __syncthreads();
    if (threadIdx.x == 0) p.seq_lens[id] = 0;
  }
}

// Compaction: of U used pages, the i-th that lies at U or behind moves to the i-th free one before
// U. A block a page; reads and writes each moved page once (2 * 73,728 bytes at 1152-byte rows).
__global__ void __launch_bounds__(kPagesThreads) mlra_pages_move_kernel(const PagesParams p) {
  __shared__ int prefix[kMaxSupers];
  __shared__ int scratch[kPagesThreads / 32];
  __shared__ int move[2];
  __shared__ int low_used;
  grid_dependency_wait();
  grid_launch_dependents();
  const int free_pages = load_prefix(p, prefix, scratch);
  const int U = p.num_pages - free_pages;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.ctl[1] = U;
    if (p.used != nullptr) *p.used = U;
  }
  // used pages before U
  if (U == 0 || free_pages == 0) return;
  if (warp_id() == 0) {
    const int s = U / kSuperPages, w = (U % kSuperPages) / 32;  // U < num_pages: the stretch exists
    int f = 0;
    for (int x = lane_id(); x <= w; x += 32) {
      uint32_t bits = p.free_bits[(size_t)s * kSuperWords + x];
      if (x == w) bits &= (1u << (U % 32)) - 1u;
      f += __popc(bits);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    if (lane_id() == 0) low_used = U - (prefix[s] + f);
  }
  __syncthreads();
  const int moves = U - low_used;
  const size_t page_bytes = (size_t)kPage * p.row_bytes;
  for (int i = blockIdx.x; i < moves; i += gridDim.x) {
    if (warp_id() == 0) {
      const int d = select_page<false>(p, prefix, i);
      if (lane_id() == 0) move[0] = d;
    } else if (warp_id() == 1) {
      const int s = select_page<true>(p, prefix, low_used + i);
      if (lane_id() == 0) move[1] = s;
    }
    __syncthreads();
    const int dst = move[0], src = move[1];
    copy_bytes(p.pool + dst * page_bytes, p.pool + src * page_bytes, (long long)page_bytes, threadIdx.x, blockDim.x);
    if (threadIdx.x == 0) {
      p.remap[src] = dst;
      p.refs[dst] = p.refs[src];
      p.refs[src] = 0;
    }
    __syncthreads();
  }
}
// The tables' entries follow (grid-stride over rows).
__global__ void __launch_bounds__(kPagesThreads) mlra_pages_remap_kernel(const PagesParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int U = p.ctl[1];
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    int len = p.seq_lens[b];
    if (len < 0 || len > p.pt_stride * kPage) {
      if (threadIdx.x == 0) set_status(p.status, kErrSeqLen);
      len = len < 0 ? 0 : p.pt_stride * kPage;
    }
    const int n = pages_of(len);
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      int* e = p.page_table + (size_t)b * p.pt_stride + c;
      const int page = *e;
      if (page < 0 || page >= p.num_pages) set_status(p.status, kErrPageOob);
      else if (page >= U && (((p.free_bits[page >> 5] >> (page & 31)) & 1u) == 0)) *e = p.remap[page];
    }
  }
}

}  // namespace mlra
