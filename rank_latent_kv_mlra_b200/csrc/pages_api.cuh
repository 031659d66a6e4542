// pages_api.cuh - host side of the page operators (included by mlra_api.cu).
#pragma once

namespace {

struct PagesWorkspace {
  int* status;
  int* ctl;
  uint32_t* free_bits;
  int* super_free;
  int* rank;
  int* first;
  int* remap;
  size_t bytes;
};
PagesWorkspace carve_pages(int num_pages, int batch, void* base) {
  Carver c = {static_cast<char*>(base), 0};
  const size_t supers = ((size_t)num_pages + kSuperPages - 1) / kSuperPages;
  PagesWorkspace w;
  w.status = c.take<int>(64);
  w.ctl = c.take<int>(2);
  w.free_bits = c.take<uint32_t>(supers * kSuperWords);
  w.super_free = c.take<int>(supers);
  w.rank = c.take<int>(batch);
  w.first = c.take<int>(batch);
  w.remap = c.take<int>(num_pages);
  w.bytes = c.off;
  return w;
}

bool pages_sizes_ok(int num_pages, int batch, int pt_stride) {
  return num_pages > 0 && num_pages <= kMaxSupers * kSuperPages && batch > 0 && batch <= kMaxRows && pt_stride > 0 &&
         (long long)pt_stride * kPage <= 0x7fffffffLL - kPage;
}

// Fills the parameters every page operator shares, after checking them.
int pages_params(mlra_handle h, void* pool, bool has_pool, int32_t* refs, int num_pages, int32_t* page_table,
                 int pt_stride, int batch, int32_t* seq_lens, const int32_t* ids, const int32_t* arg, int n,
                 bool has_arg, void* workspace, size_t ws_bytes, PagesParams* out) {
  if (!h || !refs || !page_table || !seq_lens || !workspace || (has_pool && !pool)) return MLRA_ERR_INVALID_ARG;
  if (!pages_sizes_ok(num_pages, batch, pt_stride) || n < 0 || n > batch) return MLRA_ERR_INVALID_ARG;
  if (n > 0 && (!ids || (has_arg && !arg))) return MLRA_ERR_INVALID_ARG;
  if ((has_pool && !aligned16(pool)) || (reinterpret_cast<uintptr_t>(workspace) & 255)) return MLRA_ERR_INVALID_ARG;
  const PagesWorkspace w = carve_pages(num_pages, batch, workspace);
  if (ws_bytes < w.bytes) return MLRA_ERR_WORKSPACE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return MLRA_ERR_INVALID_ARG;
  PagesParams p = {};
  p.refs = refs;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.pt_stride = pt_stride;
  p.batch = batch;
  p.seq_lens = seq_lens;
  p.ids = ids;
  p.arg = arg;
  p.n = n;
  p.free_bits = w.free_bits;
  p.super_free = w.super_free;
  p.rank = w.rank;
  p.first = w.first;
  p.ctl = w.ctl;
  p.remap = w.remap;
  p.status = w.status;
  p.pool = static_cast<char*>(pool);
  p.row_bytes = (h->cfg.d_c + h->d_r) * (h->fp8 ? 1 : 2);
  *out = p;
  return MLRA_OK;
}

template <class K>
cudaError_t launch_pages(K kernel, dim3 grid, const PagesParams& p, cudaStream_t s) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c = launch_cfg(grid, dim3(kPagesThreads), 0, s, true, &attr);
  return cudaLaunchKernelEx(&c, kernel, p);
}

int pages_nothing(const PagesParams& p, cudaStream_t s) {
  return cudaMemsetAsync(p.status, 0, 4, s) == cudaSuccess ? MLRA_OK : MLRA_ERR_CUDA;
}

}  // namespace
