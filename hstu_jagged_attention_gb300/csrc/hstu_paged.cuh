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
  int2 sums[WARPS];  // units and blocks
  int r0, r1;        // blocks before the share and before its end
  int e, h, i;       // entry, head and unit
  PagedSeq seq;
};

// Lengths and units (0 past e1) of entries e .. e + 3, their loads in flight
// together.
struct PagedFour {
  PagedSeq seq[4];
  int units[4], nb[4];
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
      nb[i] = e + i < e1 ? paged_walk(seq[i], qt[i], w.tile_rows, w.kb_shift).nb : 0;
      units[i] = paged_units(w, nb[i]);
    }
  }
};

// Totals the work over all WARPS warps of the CTA and finds where its share
// starts, and its first entry's lengths (in *g); false (for all of them) when
// it has none.  COUNT: also its blocks, in *steps (a share without blocks is
// none).  Synchronises the CTA.
template <int WARPS, bool COUNT>
__device__ bool paged_locate(const PagedView& p, PagedWork* w, PagedStart<WARPS>* m, unsigned* status,
                             PagedCursor* c, PagedSeg* g, int* steps = nullptr) {
  const int n = w->tiles * p.batch;
  const int each = (n + 32 * WARPS - 1) / (32 * WARPS);
  const int e0 = threadIdx.x * each, e1 = e0 + each < n ? e0 + each : n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = 0, blocks = 0;
  bool bad = false;
  PagedFour four;
  for (int e = e0; e < e1; e += 4) {
    four.load(p, *w, e, e1, &bad);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum += four.units[i];
      if (COUNT) blocks += w->heads * four.nb[i];
    }
  }
  if (bad && blockIdx.x == 0) atomicOr(status, kStatusBadPaged);
  int incl = sum, bincl = blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
    if (COUNT) {
      const int y = __shfl_up_sync(0xffffffffu, bincl, o);
      if (lane >= o) bincl += y;
    }
  }
  if (lane == 31) m->sums[warp] = make_int2(incl, bincl);
  __syncthreads();
  int2 before = make_int2(0, 0), total = before;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    const int2 x = m->sums[i];
    if (i < warp) {
      before.x += x.x;
      before.y += x.y;
    }
    total.x += x.x;
    total.y += x.y;
  }
  w->total = total.x;
  w->per = paged_share(*w, p.batch, gridDim.x, 1);
  c->cta = blockIdx.x;
  c->u = c->u0 = (int)blockIdx.x * w->per;
  if (c->u >= total.x) return false;
  c->u1 = total.x - c->u > w->per ? c->u + w->per : total.x;
  if (COUNT && threadIdx.x == 0 && c->u1 == total.x) m->r1 = total.y;
  int at = before.x + incl - sum, done = before.y + bincl - blocks;  // before the thread's entries
  if ((at <= c->u && c->u < at + sum) || (COUNT && at <= c->u1 && c->u1 < at + sum)) {
    // the entries that hold the share's first unit and the one behind its last
    int nb0 = 0, r0 = 0, done0 = 0, nb1 = 0, r1 = 0, done1 = 0;
    for (int e = e0; e < e1; e += 4) {
      if (each > 4) four.load(p, *w, e, e1, &bad);  // else they are at hand
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int units = four.units[i];
        if (at <= c->u && c->u < at + units) {
          nb0 = four.nb[i];
          r0 = c->u - at;
          done0 = done;
          m->e = e + i;
          m->seq = four.seq[i];
        }
        if (COUNT && at <= c->u1 && c->u1 < at + units) {
          nb1 = four.nb[i];
          r1 = c->u1 - at;
          done1 = done;
        }
        at += units;
        if (COUNT) done += w->heads * four.nb[i];
      }
    }
    if (nb0) {
      const int h = r0 / (nb0 + w->extra), i = r0 - h * (nb0 + w->extra);
      m->h = h;
      m->i = i;
      if (COUNT) m->r0 = done0 + h * nb0 + (i < nb0 ? i : nb0);
    }
    if (COUNT && nb1) m->r1 = done1 + paged_blocks(*w, nb1, r1);
  }
  __syncthreads();
  if (COUNT) {
    *steps = m->r1 - m->r0;
    if (*steps == 0) return false;
  }
  c->e = m->e;
  c->h = m->h;
  c->i = m->i;
  c->loaded = true;
  g->qt = w->tiles == 1 ? 0 : c->e / p.batch;
  g->b = c->e - g->qt * p.batch;
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
