// Device side of the paged cache's attention kernels: where a CTA's share of
// the work starts, and the page numbers ahead of a producer.
#pragma once

#include "hstu_internal.h"
#include "hstu_paged.h"
#include "hstu_ptx.cuh"

namespace hstu {
namespace {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                            int y, int z, int u) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
      : "memory");
}

template <int WARPS>
struct PagedStart {
  long long sums[WARPS];
  int e, r;
};

// Totals the work over all WARPS warps of the CTA and finds where its share
// starts; false (for all of them) when it has none.  Synchronises the CTA.
template <int WARPS>
__device__ bool paged_locate(const PagedView& p, PagedWork* w, int min_units, PagedStart<WARPS>* m,
                             unsigned* status, PagedCursor* c) {
  const int n = w->tiles * p.batch;
  const int each = (n + 32 * WARPS - 1) / (32 * WARPS);
  const int e0 = threadIdx.x * each, e1 = e0 + each < n ? e0 + each : n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sum = 0;
  for (int e = e0; e < e1; ++e) {
    const int qt = e / p.batch, b = e - qt * p.batch;
    PagedSeq s;
    if (!paged_seq(p, b, &s) && blockIdx.x == 0) atomicOr(status, kStatusBadPaged);
    sum += (long long)w->heads * paged_walk(s, qt, w->tile_rows, w->kb_shift).nb;
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) m->sums[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i < warp) before += m->sums[i];
    total += m->sums[i];
  }
  w->total = total;
  w->per = paged_share(total, gridDim.x, min_units);
  c->at = -1;
  c->u = (long long)blockIdx.x * w->per;
  if (c->u >= total) return false;
  c->u1 = c->u + w->per < total ? c->u + w->per : total;
  long long at = before + incl - sum;  // the thread's first unit
  if (at <= c->u && c->u < at + sum) {
    for (int e = e0; e < e1; ++e) {
      const int qt = e / p.batch, b = e - qt * p.batch;
      PagedSeq s;
      paged_seq(p, b, &s);
      const long long units = (long long)w->heads * paged_walk(s, qt, w->tile_rows, w->kb_shift).nb;
      if (c->u < at + units) {
        m->e = e;
        m->r = (int)(c->u - at);
        break;
      }
      at += units;
    }
  }
  __syncthreads();
  c->e = m->e;
  c->r = m->r;
  return true;
}

// Page numbers of one sequence, held by a warp: lane l has those of pages
// first + l and first + 32 + l, so that the next 32 load ahead of their use.
struct PageIds {
  int first = -64, ids = 0, next = 0;
  // Makes pages p .. p + n - 1 (n <= 32) available; `pages`: the row's valid
  // entries.  Whole-warp call.
  __device__ __forceinline__ void cover(const int32_t* row, int p, int n, int pages) {
    if (p >= first && p + n <= first + 32) return;
    const int lane = threadIdx.x & 31;
    ids = p == first + 32 ? next : (p + lane < pages ? __ldg(row + p + lane) : 0);
    first = p;
    next = p + 32 + lane < pages ? __ldg(row + p + 32 + lane) : 0;
  }
  // The number of page p, for each lane its own p (covered, or the result is unused).
  __device__ __forceinline__ int get(int p) const {
    return __shfl_sync(0xffffffffu, ids, (p - first) & 31);
  }
};

}  // namespace
}  // namespace hstu
