// Index arithmetic of the paged K/V cache, shared by its kernels and by the
// host-only entry points that enumerate the same slots and work (so that it
// is tested on a machine without a GPU).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define HSTU_HD __host__ __device__ __forceinline__
#else
#define HSTU_HD inline
#endif

namespace hstu {

// A batch of new tokens against the cache (hstu_paged_batch) with the
// cache's geometry.  The arrays are device memory in a kernel, host memory
// in the host-only entry points.
struct PagedView {
  const int32_t* q_offsets;    // batch + 1: rows of the sequences' new tokens
  const int32_t* kv_lens;      // batch: tokens in the cache, the new ones included
  const int32_t* num_targets;  // batch, or null: no candidates
  const int32_t* page_table;   // (batch, max_pages)
  int batch, max_pages, max_q, rows;
  int num_pages, page_shift;   // pages of 2^page_shift tokens
};

struct PagedSeq {
  int q0, qn;  // its rows q0 .. q0 + qn - 1 of q, k, v, out
  int kv;      // its tokens in the cache; new token i sits at kv - qn + i
  int hist;    // tokens that every candidate sees
};

// Sequence b's four words, and what they say: qn = 0 and false when they
// contradict one another or the arrays' bounds (nothing of such a sequence is
// read or written).  Apart, so that several sequences' loads can be in flight.
struct PagedRaw {
  int o0, o1, kv, nt;
};
HSTU_HD PagedRaw paged_raw(const PagedView& p, int b) {
  return PagedRaw{p.q_offsets[b], p.q_offsets[b + 1], p.kv_lens[b], p.num_targets ? p.num_targets[b] : 0};
}
HSTU_HD bool paged_check(const PagedView& p, const PagedRaw& r, PagedSeq* s) {
  s->q0 = r.o0;
  s->kv = r.kv;
  s->hist = r.kv - r.nt;
  s->qn = 0;
  // with 0 <= o0 <= o1 the difference cannot overflow
  if (r.o0 < 0 || r.o1 < r.o0 || r.o1 > p.rows) return false;
  const int n = r.o1 - r.o0;
  if (n > p.max_q || r.kv < n || r.nt < 0 || r.nt > n) return false;
  if (r.kv > 0 && ((r.kv - 1) >> p.page_shift) >= p.max_pages) return false;
  s->qn = n;
  return true;
}
HSTU_HD bool paged_seq(const PagedView& p, int b, PagedSeq* s) { return paged_check(p, paged_raw(p, b), s); }

// The pool's row of token `pos` of sequence b; -1 when its page is out of range.
HSTU_HD long long paged_slot(const PagedView& p, int b, int pos) {
  const int page = p.page_table[(long long)b * p.max_pages + (pos >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) return -1;
  return ((long long)page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// The sequence whose rows hold row t, or -1.  The guess is exact for equal
// lengths (one decode step, a dense batch); otherwise a binary search.
HSTU_HD int paged_find(const PagedView& p, int t) {
  const int total = p.q_offsets[p.batch];
  if (t >= total) return -1;
  int b = (int)((float)t * ((float)p.batch / (float)total));
  if (b > p.batch - 1) b = p.batch - 1;
  if (p.q_offsets[b] <= t && t < p.q_offsets[b + 1]) return b;
  int lo = 0, hi = p.batch;  // the last b with q_offsets[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_offsets[mid] <= t) lo = mid; else hi = mid;
  }
  return p.q_offsets[lo] <= t && t < p.q_offsets[lo + 1] ? lo : -1;
}

// The key blocks (of 2^kb_shift keys) that one tile of query rows walks:
// those that hold keys every candidate sees, 0 .. nh - 1, then the blocks d0
// .. that hold the tile's own keys and were not among them.
struct PagedWalk {
  int p0;    // position of the tile's first row
  int rows;  // its valid rows
  int nh, d0, nb;
  HSTU_HD int block(int i) const { return i < nh ? i : d0 + (i - nh); }
  HSTU_HD int end() const { return p0 + rows; }  // no row sees a key at or past it
};

HSTU_HD PagedWalk paged_walk(const PagedSeq& s, int qt, int tile_rows, int kb_shift) {
  PagedWalk w;
  w.p0 = s.kv - s.qn + tile_rows * qt;
  w.rows = s.qn - tile_rows * qt;
  if (w.rows > tile_rows) w.rows = tile_rows;
  if (w.rows <= 0) {
    w.rows = w.nh = w.d0 = w.nb = 0;
    return w;
  }
  const int p1 = w.p0 + w.rows - 1;
  const int h = s.hist < p1 + 1 ? s.hist : p1 + 1;
  w.nh = (h + (1 << kb_shift) - 1) >> kb_shift;
  w.d0 = w.p0 >> kb_shift;
  if (w.d0 < w.nh) w.d0 = w.nh;
  const int own = (p1 >> kb_shift) - w.d0 + 1;
  w.nb = w.nh + (own > 0 ? own : 0);
  return w;
}

// The work of a launch: entries (query tile qt, sequence b), qt outermost, so
// that CTAs that run at the same time on different tiles of a sequence read
// the same keys; within an entry the heads, within a head the key blocks.
// Each block is one unit, then come `extra` units without work, for what an
// item costs besides its blocks; CTA c takes units [c per, (c + 1) per): equal
// shares, whatever the lengths.  A (tile, sequence, head) whose blocks a
// share's end cuts is summed from the CTAs' parts, in their order.
struct PagedWork {
  int heads, tiles, tile_rows, kb_shift, extra;
  int most_parts;  // see paged_share
  int total, per;  // units (at most 2^30: the host checks) and units a CTA
};

// Units a CTA: an equal share, but no item cut into more than most_parts parts
// on average, which the last of its CTAs would sum alone.
HSTU_HD int paged_share(const PagedWork& w, int batch, int grid, int min_units) {
  const unsigned total = (unsigned)w.total, items = (unsigned)w.tiles * (unsigned)batch * (unsigned)w.heads;
  // ceil(total / grid), from the fp32 quotient (a few off for the largest totals)
  unsigned per = (unsigned)((float)total / (float)grid);
  while (per * (unsigned)grid < total) ++per;
  while (per > 0 && (per - 1u) * (unsigned)grid >= total) --per;
  if (items < (unsigned)grid / w.most_parts) {
    const unsigned least = (total + w.most_parts * items - 1u) / (w.most_parts * items);
    if (per < least) per = least;
  }
  return per > (unsigned)min_units ? (int)per : min_units;
}

// Units of an entry whose tile walks nb blocks, and the blocks among its
// first r units.
HSTU_HD int paged_units(const PagedWork& w, int nb) { return nb ? w.heads * (nb + w.extra) : 0; }
HSTU_HD int paged_blocks(const PagedWork& w, int nb, int r) {
  const int h = r / (nb + w.extra), i = r - h * (nb + w.extra);
  return h * nb + (i < nb ? i : nb);
}

struct PagedSeg {
  PagedSeq seq;
  PagedWalk walk;
  int b, h, qt;
  int i0, n;            // its blocks walk.block(i0) .. walk.block(i0 + n - 1)
  int c0, parts;        // the first CTA with a part of this item, and their number
};

// The segments of one CTA, units u0 .. u1 - 1: from unit i of head h of entry
// e on.  The entry's lengths are read once for all its heads; the segment
// handed to next() keeps them (`loaded`: it already holds entry e's).
struct PagedCursor {
  int cta, u, u0, u1;
  int e, h, i;
  bool loaded;
  HSTU_HD void load(const PagedView& p, const PagedWork& w, PagedSeg* g) const {
    g->qt = w.tiles == 1 ? 0 : e / p.batch;
    g->b = e - g->qt * p.batch;
    paged_seq(p, g->b, &g->seq);
    g->walk = paged_walk(g->seq, g->qt, w.tile_rows, w.kb_shift);
  }
  HSTU_HD bool next(const PagedView& p, const PagedWork& w, PagedSeg* g) {
    for (;;) {
      if (u >= u1) return false;
      if (h == w.heads) {
        h = 0;
        ++e;
        loaded = false;
      }
      if (!loaded) {
        for (;; ++e) {
          if (e >= w.tiles * p.batch) return false;
          load(p, w, g);
          if (g->walk.nb) break;
        }
        loaded = true;
      }
      if (i < g->walk.nb) break;
      u += g->walk.nb + w.extra - i;  // the share starts behind the item's blocks
      i = 0;
      ++h;
    }
    const int nb = g->walk.nb, s = u - i;  // the item's blocks and first unit
    g->h = h;
    g->i0 = i;
    g->n = nb - i < u1 - u ? nb - i : u1 - u;
    g->c0 = cta;
    g->parts = 1;
    if (s < u0 || s + nb > u1) {
      g->c0 = s / w.per;
      g->parts = (s + nb - 1) / w.per - g->c0 + 1;
    }
    u = s + nb + w.extra;  // a cut item ends the share
    i = 0;
    ++h;
    return true;
  }
};

}  // namespace hstu
