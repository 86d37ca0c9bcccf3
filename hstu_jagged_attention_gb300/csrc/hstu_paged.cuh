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
  int sums[WARPS];
  int e, h, i;  // entry, head and block
  int b, qt;
  PagedSeq seq;
};

// Lengths and units (0 past e1) of entries e .. e + 3, their loads in flight
// together.
struct PagedFour {
  PagedSeq seq[4];
  int units[4];
  __device__ __forceinline__ void load(const PagedView& p, const PagedWork& w, int e, int e1, bool* bad) {
    PagedRaw raw[4];
    int qt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = e + i < e1 ? e + i : e;
      qt[i] = w.tiles == 1 ? 0 : x / p.batch;
      raw[i] = paged_raw(p, x - qt[i] * p.batch);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!paged_check(p, raw[i], &seq[i])) *bad = true;
      units[i] = e + i < e1 ? w.heads * paged_walk(seq[i], qt[i], w.tile_rows, w.kb_shift).nb : 0;
    }
  }
};

// Totals the work over all WARPS warps of the CTA and finds where its share
// starts, and its first entry's lengths (in *g); false (for all of them) when
// it has none.  Synchronises the CTA.
template <int WARPS>
__device__ bool paged_locate(const PagedView& p, PagedWork* w, int min_units, PagedStart<WARPS>* m,
                             unsigned* status, PagedCursor* c, PagedSeg* g) {
  const int n = w->tiles * p.batch;
  const int each = (n + 32 * WARPS - 1) / (32 * WARPS);
  const int e0 = threadIdx.x * each, e1 = e0 + each < n ? e0 + each : n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = 0;
  bool bad = false;
  PagedFour four;
  for (int e = e0; e < e1; e += 4) {
    four.load(p, *w, e, e1, &bad);
    sum += four.units[0] + four.units[1] + four.units[2] + four.units[3];
  }
  if (bad && blockIdx.x == 0) atomicOr(status, kStatusBadPaged);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) m->sums[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i < warp) before += m->sums[i];
    total += m->sums[i];
  }
  w->total = total;
  w->per = paged_share(*w, p.batch, gridDim.x, min_units);
  c->cta = blockIdx.x;
  c->u = c->u0 = (int)blockIdx.x * w->per;
  if (c->u >= total) return false;
  c->u1 = total - c->u > w->per ? c->u + w->per : total;
  int at = before + incl - sum;  // the thread's first unit
  if (at <= c->u && c->u < at + sum) {
    for (int e = e0; e < e1; e += 4) {
      if (each > 4) four.load(p, *w, e, e1, &bad);  // else they are at hand
      bool found = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!found && c->u < at + four.units[i]) {
          found = true;
          c->e = e + i;
          g->seq = four.seq[i];
        }
        if (!found) at += four.units[i];
      }
      if (!found) continue;
      g->qt = w->tiles == 1 ? 0 : c->e / p.batch;
      g->b = c->e - g->qt * p.batch;
      g->walk = paged_walk(g->seq, g->qt, w->tile_rows, w->kb_shift);
      m->e = c->e;
      m->h = (c->u - at) / g->walk.nb;
      m->i = c->u - at - m->h * g->walk.nb;
      m->b = g->b;
      m->qt = g->qt;
      m->seq = g->seq;
      // the producers read these next
      const int page = (g->walk.block(m->i) << w->kb_shift) >> p.page_shift;
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p.page_table + (long long)g->b * p.max_pages + page));
      break;
    }
  }
  __syncthreads();
  c->e = m->e;
  c->h = m->h;
  c->i = m->i;
  c->loaded = true;
  g->b = m->b;
  g->qt = m->qt;
  g->seq = m->seq;
  g->walk = paged_walk(g->seq, g->qt, w->tile_rows, w->kb_shift);
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
