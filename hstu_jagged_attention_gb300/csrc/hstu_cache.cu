// The paged K/V cache: appending keys and values to it (with the position
// rotation), and the attention of a few new tokens over it.
//
//   append   slot = page_table[b][p / page_size] page_size + p % page_size,
//            k_pages[slot] = R_p k, v_pages[slot] = v, q_out = R_p q
//   attention
//            out[t,h,:] = inv_n sum_j silu(alpha q[t,h,:].K_j) V_j over the
//            keys j <= p(t) of the cache, candidates as in the forward
//
// (ai6s.net post section 1 for the formula; HSTU paper section 3.4: the
// history's keys and values are cached and serve every microbatch.)
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <climits>
#include <new>

#include "hstu_attn.h"
#include "hstu_internal.h"
#include "hstu_paged.cuh"
#include "hstu_ptx.cuh"

namespace hstu {
namespace {

// ------------------------------------------------------------------- append
struct AppendArgs {
  PagedView p;
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  uint16_t *k_pages, *v_pages, *q_out;
  long long page_stride;
  const float* table;  // (positions, rot): rot / 2 cosines, then as many sines; null: no rotation
  int positions, rot, pairs;
  int heads, d;
  unsigned check_ctas;
  unsigned* status;
};

struct F8 {
  float f[8];
};

__device__ __forceinline__ F8 unpack8(const uint4& p) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  F8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.f[2 * i] = __uint_as_float(w[i] << 16);
    v.f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return v;
}

__device__ __forceinline__ uint4 pack8(const F8& v) {
  return make_uint4(pack_bf16x2(v.f[0], v.f[1]), pack_bf16x2(v.f[2], v.f[3]),
                    pack_bf16x2(v.f[4], v.f[5]), pack_bf16x2(v.f[6], v.f[7]));
}

// 16 channels of one head as two vectors of 8: x = channels at c0, y = those
// at c1.  Pairs: channels 2i and 2i + 1 turn together, so each vector turns
// within itself; halves: x[i] turns with y[i].  One rounding, at the end.
__device__ __forceinline__ void turn16(uint4& x, uint4& y, const F8& cs, const F8& sn, bool pairs) {
  F8 a = unpack8(x), b = unpack8(y);
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = a.f[2 * i], a1 = a.f[2 * i + 1], b0 = b.f[2 * i], b1 = b.f[2 * i + 1];
      a.f[2 * i] = fmaf(a0, cs.f[i], -(a1 * sn.f[i]));
      a.f[2 * i + 1] = fmaf(a1, cs.f[i], a0 * sn.f[i]);
      b.f[2 * i] = fmaf(b0, cs.f[4 + i], -(b1 * sn.f[4 + i]));
      b.f[2 * i + 1] = fmaf(b1, cs.f[4 + i], b0 * sn.f[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a0 = a.f[i], b0 = b.f[i];
      a.f[i] = fmaf(a0, cs.f[i], -(b0 * sn.f[i]));
      b.f[i] = fmaf(b0, cs.f[i], a0 * sn.f[i]);
    }
  }
  x = pack8(a);
  y = pack8(b);
}

constexpr int kAppendThreads = 256;

// One thread a (token, head, 16 channels): every array is read and written
// once, with 16-byte accesses; the rotation's table is the same for all heads
// of a token and comes from L1.  Bound by memory: 65,536 tokens of 4 heads of
// 64, rotated, take 33.5 us (218 MB, 6.5 TB/s); one token for 64 sequences
// 3.0 us, the chain offsets -> lengths -> page -> store.
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  after_previous_kernel();
  const int per_head = a.d / 16, per_token = a.heads * per_head;
  PagedSeq s;
  if (blockIdx.x < a.check_ctas) {
    // The first CTAs check a sequence a thread: one that contradicts itself may
    // have no row.  (In the rows' CTAs the same check made 65,536 tokens 37.3
    // us, in CTAs behind them 34.1; so 33.6, as without it.)
    const long long b = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
    if (b < a.p.batch && !paged_seq(a.p, (int)b, &s)) atomicOr(a.status, kStatusBadPaged);
    return;
  }
  const long long unit = (long long)(blockIdx.x - a.check_ctas) * kAppendThreads + threadIdx.x;
  const long long tl = unit / per_token;
  if (tl >= a.p.rows) return;
  const int t = (int)tl, w = (int)(unit - tl * per_token);
  const int h = w / per_head, c = w - h * per_head;
  // rotated channels first, 16 a thread; then the others
  const bool turn = a.table && c < a.rot / 16;
  int c0 = 16 * c, c1 = 16 * c + 8;
  if (turn && !a.pairs) {
    c0 = 8 * c;
    c1 = a.rot / 2 + 8 * c;
  }
  const long long at = (long long)h * a.d;
  const uint16_t* kr = a.k + t * a.k_stride + at;
  const uint16_t* vr = a.v + t * a.v_stride + at;
  const int total = a.p.q_offsets[a.p.batch];
  uint4 k0 = *reinterpret_cast<const uint4*>(kr + c0), k1 = *reinterpret_cast<const uint4*>(kr + c1);
  const uint4 v0 = *reinterpret_cast<const uint4*>(vr + c0), v1 = *reinterpret_cast<const uint4*>(vr + c1);
  uint4 q0{}, q1{};
  if (a.q) {
    const uint16_t* qr = a.q + t * a.q_stride + at;
    q0 = *reinterpret_cast<const uint4*>(qr + c0);
    q1 = *reinterpret_cast<const uint4*>(qr + c1);
  }
  if (t >= total) return;  // a row behind the last sequence
  const int b = paged_find(a.p, t);
  if (b < 0 || !paged_seq(a.p, b, &s)) return;  // before the first sequence, or of one that is reported
  const int pos = s.kv - s.qn + (t - s.q0);
  const long long slot = paged_slot(a.p, b, pos);
  const int turned_at = pos < s.hist ? pos : s.hist;  // a candidate stands right behind the history
  if (slot < 0 || (a.table && turned_at >= a.positions)) {
    atomicOr(a.status, kStatusBadPaged);
    return;
  }
  if (turn) {
    const float* tab = a.table + (long long)turned_at * a.rot + 8 * c;
    F8 cs, sn;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(tab) + i);
      const float4 y = __ldg(reinterpret_cast<const float4*>(tab + a.rot / 2) + i);
      cs.f[4 * i] = x.x; cs.f[4 * i + 1] = x.y; cs.f[4 * i + 2] = x.z; cs.f[4 * i + 3] = x.w;
      sn.f[4 * i] = y.x; sn.f[4 * i + 1] = y.y; sn.f[4 * i + 2] = y.z; sn.f[4 * i + 3] = y.w;
    }
    turn16(k0, k1, cs, sn, a.pairs);
    if (a.q) turn16(q0, q1, cs, sn, a.pairs);
  }
  const long long page = slot >> a.p.page_shift;
  const long long in_page = slot & ((1 << a.p.page_shift) - 1);
  const long long to = page * a.page_stride + in_page * a.heads * a.d + at;
  *reinterpret_cast<uint4*>(a.k_pages + to + c0) = k0;
  *reinterpret_cast<uint4*>(a.k_pages + to + c1) = k1;
  *reinterpret_cast<uint4*>(a.v_pages + to + c0) = v0;
  *reinterpret_cast<uint4*>(a.v_pages + to + c1) = v1;
  if (a.q) {
    uint16_t* qo = a.q_out + (long long)t * a.heads * a.d + at;
    *reinterpret_cast<uint4*>(qo + c0) = q0;
    *reinterpret_cast<uint4*>(qo + c1) = q1;
  }
}

// ------------------------------------------------ attention of a few tokens
// A tile is up to 16 new tokens of one (sequence, head); it walks blocks of 128
// keys.  The last warp copies each block's K and V rows, page by page, into a
// ring of shared-memory stages (bulk-tensor copies, swizzled rows).  The other
// four (eight at d = 128) take a part of the keys each: S = Q K^T,
// p = silu(alpha S), O += p V on mma.sync m16n8k16, with p split into two bf16
// terms as in the forward, so that P V keeps 16 bits of p.
// Bound by memory: the cache is read once for all rows of the tile, with 1 to
// 16 operations a byte, and a 128-row tcgen05 tile would do the same reads
// with 8 times the products.  One token for 512 sequences (log-normal lengths,
// 2 heads of 64, 211 MB) takes 42 us: 3 us until the first copies are issued
// (lengths, share, page numbers: three loads one after the other), then
// 6.5 TB/s, and 1 us to join the cut items.  The first form of this kernel (64
// keys a block, 16 a warp, the shares found serially) took 50 us.
constexpr int kStepRows = 16;
constexpr int kStepKeys = 128, kStepShift = 7;
// Warps that compute: 32 keys each, two k16 steps whose chains of products
// overlap, or at d = 128 (where one step has as many products) 16.  One warp
// more than a multiple of four puts two on one of the SM's four schedulers, so
// two CTAs of five warps fit at 128 registers a thread, and at d = 128, with
// 168, one CTA of nine.
__host__ __device__ constexpr int step_warps(int d) { return d == 128 ? 8 : 4; }
__host__ __device__ constexpr int step_per_sm(int d) { return d == 128 ? 1 : 2; }

struct StepArgs {
  PagedView p;
  PagedWork w;     // total and per are found by the kernel
  int stages;
  int red_rows;    // rows of a tile that can exist: min(max_q, tile_rows)
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  float half_alpha, inv_n;
  unsigned* counters;
  float* parts;
  unsigned* status;
  unsigned long long timeout_ns;
  unsigned debug_flags;
};

struct StepWait {
  unsigned long long limit_ns;
  volatile int* abort_flag;
  unsigned* status;  // [0]: bits, [1]: the first site that gave up
};

__device__ __noinline__ void step_timeout(const StepWait& w, int site) {
  atomicOr(w.status, kStatusTimeout);
  atomicCAS(w.status + 1, 0u, (unsigned)site);
  *w.abort_flag = 1;
}

// Bounded wait; false once the CTA has given up.
__device__ __forceinline__ bool step_wait(uint32_t bar, uint32_t parity, const StepWait& w, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 3u) == 0) {
      if (*w.abort_flag) return false;
      if (globaltimer() - t0 > w.limit_ns) {
        step_timeout(w, site);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct StepCfg {
  static constexpr int WARPS = step_warps(D);
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int KEYS = kStepKeys;
  static constexpr int KW = KEYS / WARPS;       // keys of a warp: 16 or 32
  static constexpr int CH = D < 64 ? D : 64;    // channels of a swizzled row
  static constexpr int NCH = D / CH;
  static constexpr int ROWB = CH * 2;
  static constexpr int CHUNKB = KEYS * ROWB;
  static constexpr int TILEB = NCH * CHUNKB;    // a block's rows of K, or of V
  static constexpr int STAGEB = 2 * TILEB;
  static constexpr int MAX_STAGES = 16;
  // Byte of 16-byte column c of row r in a tile.  The columns' swizzle is an
  // exclusive or below the row's bytes, so with c0 < 2 even columns c away:
  // at(r, c0 + c) = at(r, c0) ^ (c << 4), within a chunk.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    const int x = ROWB == 128 ? (r & 7) : ((r >> 1) & 3);
    return (uint32_t)(r * ROWB + ((c ^ x) << 4));
  }
  // from at(r, c0), c0 < 2, to 16-byte column c0 + 2 k
  static __device__ __forceinline__ uint32_t step(uint32_t base, int k) {
    constexpr int PER = CH / 16;
    return (base ^ (uint32_t)((k % PER) << 5)) + (uint32_t)((k / PER) * CHUNKB);
  }
};

// Shared memory behind the stages: the warps' partial sums, the barriers,
// and the schedule's words.
// 8 floats between rows, so that eight rows' 8-byte stores meet all banks
__host__ __device__ constexpr int step_red_stride(int d) { return d + 8; }
__host__ __device__ constexpr int step_red_bytes(int rows, int d) {
  return step_warps(d) * rows * step_red_stride(d) * (int)sizeof(float);
}
constexpr int kStepTailBytes = 2 * 16 * 8 + 64 + 16 * 8;

template <int WARPS>
struct StepMisc {
  int abort_flag;
  unsigned last;  // bits: this CTA arrived last at the items it shares
  PagedStart<WARPS + 1> start;
};
static_assert(sizeof(StepMisc<8>) <= 64 + 16 * 8, "misc");

template <int D>
__device__ void step_produce(const CUtensorMap* tk, const CUtensorMap* tv, const StepArgs& a,
                             const PagedWork& w, PagedCursor c, PagedSeg g, uint32_t base, uint32_t full,
                             uint32_t empty, const StepWait& wt) {
  using C = StepCfg<D>;
  const int lane = threadIdx.x & 31;
  const int shift = a.p.page_shift, ps = 1 << shift;
  const int box = ps < C::KEYS ? ps : C::KEYS;
  int st = 0;
  uint32_t ph = 1, count = 0;
  bool ok = true;
  while (ok && c.next(a.p, w, &g)) {
    const int32_t* row = a.p.page_table + (long long)g.b * a.p.max_pages;
    const int end = g.walk.end();
    const int pages = (end + ps - 1) >> shift;  // of the sequence, as far as the tile sees
    PageIds ids;
    for (int i = 0; i < g.n; ++i) {
      const int tok0 = g.walk.block(g.i0 + i) << kStepShift;
      const int p0 = tok0 >> shift;
      const int valid = end - tok0 < C::KEYS ? end - tok0 : C::KEYS;
      const int npg = ps >= C::KEYS ? 1 : (valid + ps - 1) >> shift;
      ids.cover(row, p0, npg, pages);
      // npg 2 NCH <= 32 lanes copy; lane: which page of the block, which chunk of channels, K or V
      const int pg = lane / (2 * C::NCH), ch = (lane >> 1) % C::NCH;
      int page = ids.get(p0 + pg);
      const uint32_t bar = full + 8u * st;
      if (!(ok = __all_sync(0xffffffffu, step_wait(empty + 8u * st, ph, wt, kSiteStepEmpty)))) break;
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(npg * box * C::ROWB * C::NCH * 2));
      __syncwarp();
      if (pg < npg) {
        if (page < 0 || page >= a.p.num_pages) {
          // read as zeros, past the pool's end: silu(0) V = 0
          atomicOr(a.status, kStatusBadPaged);
          page = a.p.num_pages;
        }
        const uint32_t dst = base + st * C::STAGEB + (lane & 1) * C::TILEB + ch * C::CHUNKB +
                             pg * box * C::ROWB;
        tma_load_4d(dst, (lane & 1) ? tv : tk, bar, ch * C::CH, g.h,
                    ps >= C::KEYS ? (tok0 & (ps - 1)) : 0, page);
      }
      ++count;
      if (++st == a.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  // Every copy lands before the CTA ends, also where the warps that would wait
  // for it have given up.  A stage is armed again only once all of them have
  // seen its last phase complete, so each stage's last phase is the one to wait
  // for.
  if (lane == 0) {
    for (int s = 0; s < a.stages; ++s)
      if (count > (uint32_t)s) {
        const uint32_t parity = ((count - 1u - s) / a.stages) & 1u;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(full + 8u * s, parity))
          if (globaltimer() - t0 > 2000000000ull) break;
      }
  }
  __syncwarp();
}

template <int WARPS>
__device__ __forceinline__ void step_barrier() {  // the computing warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// An item whose blocks several CTAs share.
struct StepCut {
  uint16_t* out;  // its first row
  int rows, c0, parts;
};
// CTA `cta`'s part of the item that it starts, or that an earlier one does.
template <int D>
__device__ __forceinline__ float* step_part(const StepArgs& a, int cta, bool starts) {
  return a.parts + ((long long)cta * 2 + (starts ? 1 : 0)) * (kStepRows * D);
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}
// Values x .. x + 3 of an item's (rows, D) sums.
template <int D>
__device__ __forceinline__ void step_store(uint16_t* out, int heads, int x, const float4& v, float inv_n) {
  *reinterpret_cast<uint2*>(out + (long long)(x / D) * heads * D + x % D) =
      make_uint2(pack_bf16x2(v.x * inv_n, v.y * inv_n), pack_bf16x2(v.z * inv_n, v.w * inv_n));
}

// CLUSTER: the item's other parts are in the cluster's other CTAs; this CTA's
// sums stay in `red`, in the first warp's place, for step_cluster_join.
template <int D, bool CLUSTER>
__device__ void step_compute(const StepArgs& a, const PagedWork& w, PagedCursor c, PagedSeg g, uint32_t base,
                             uint32_t full, uint32_t empty, float* red, StepMisc<step_warps(D)>* m,
                             const StepWait& wt) {
  using C = StepCfg<D>;
  constexpr int KS = C::KW / 16;  // k16 steps of the P V product
  constexpr int RS = step_red_stride(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int key0 = C::KW * warp;  // this warp's keys of a block
  // ldmatrix rows: K as (keys 0-7 | 8-15) x (channels 0-7 | 8-15), V likewise, transposed
  const int mat = lane >> 3, mr = lane & 7;
  const uint32_t k_at = C::at(key0 + (mat >> 1) * 8 + mr, mat & 1);
  const uint32_t v_at = C::TILEB + C::at(key0 + (mat & 1) * 8 + mr, mat >> 1);
  const float2 ha2 = make_float2(a.half_alpha, a.half_alpha);
  int st = 0;
  uint32_t ph = 0;
  // The CTA gave up: go through the items' barriers, but touch no stage (one
  // that was not waited for is not released either) and store nothing.
  bool dead = false;
  StepCut cut0{}, cut1{};  // items shared with earlier, and with later, CTAs
  // test hook: the barrier behind the stages' is never arrived on
  if (a.debug_flags & kDebugUnsignalledWait)
    dead = !__all_sync(0xffffffffu, step_wait(full + 8u * C::MAX_STAGES - 8u, 0, wt, kSiteUnsignalledStep));
  while (c.next(a.p, w, &g)) {
    const int rows = g.walk.rows;
    uint32_t qf[D / 16][4];
    {
      const int r0 = g8, r1 = r0 + 8;
      const uint16_t* x0 =
          a.q + (long long)(g.seq.q0 + kStepRows * g.qt + r0) * a.q_stride + (long long)g.h * D + 2 * t4;
      const uint16_t* x1 = x0 + 8 * a.q_stride;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][0] = r0 < rows ? *reinterpret_cast<const uint32_t*>(x0 + 16 * kk) : 0u;
        qf[kk][1] = r1 < rows ? *reinterpret_cast<const uint32_t*>(x1 + 16 * kk) : 0u;
        qf[kk][2] = r0 < rows ? *reinterpret_cast<const uint32_t*>(x0 + 16 * kk + 8) : 0u;
        qf[kk][3] = r1 < rows ? *reinterpret_cast<const uint32_t*>(x1 + 16 * kk + 8) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][j] = 0.f;

    for (int i = 0; i < g.n && !dead; ++i) {
      const int kb = g.walk.block(g.i0 + i) << kStepShift;
      if ((dead = !__all_sync(0xffffffffu, step_wait(full + 8u * st, ph, wt, kSiteStepFull)))) break;
      const uint32_t ks = base + st * C::STAGEB + k_at, vs = base + st * C::STAGEB + v_at;
      float s[2 * KS][4];
#pragma unroll
      for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t kf[4];
          ldsm4(C::step(ks + 16 * y * C::ROWB, kk), kf);
          mma16816(s[2 * y], qf[kk], kf[0], kf[1]);
          mma16816(s[2 * y + 1], qf[kk], kf[2], kf[3]);
        }
      }
      // p = silu(alpha S) = h + h tanh(h), h = alpha S / 2; as an A operand
      // its columns are this thread's own score columns.  Rows 8 .. 15 only
      // where they exist.
      const bool masked = kb + C::KEYS > g.walk.p0 + 1 || kb + C::KEYS > g.seq.hist;
      uint32_t hi[KS][4], lo[KS][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (r == 0 || rows > 8) {
#pragma unroll
          for (int n = 0; n < 2 * KS; ++n) {
            const float2 x = __fmul2_rn(make_float2(s[n][2 * r], s[n][2 * r + 1]), ha2);
            float2 p = __ffma2_rn(x, make_float2(tanh_approx(x.x), tanh_approx(x.y)), x);
            if (masked) {
              const int pos = g.walk.p0 + 8 * r + g8, key = kb + key0 + 8 * n + 2 * t4;
              if (!(key <= pos && (key < g.seq.hist || key == pos))) p.x = 0.f;
              if (!(key + 1 <= pos && (key + 1 < g.seq.hist || key + 1 == pos))) p.y = 0.f;
            }
            const uint32_t ph2 = pack_bf16x2(p.x, p.y);
            const float2 rest = __fadd2_rn(
                p, make_float2(-__uint_as_float(ph2 << 16), -__uint_as_float(ph2 & 0xffff0000u)));
            hi[n >> 1][2 * (n & 1) + r] = ph2;
            lo[n >> 1][2 * (n & 1) + r] = pack_bf16x2(rest.x, rest.y);
          }
        } else {
#pragma unroll
          for (int n = 0; n < 2 * KS; ++n) hi[n >> 1][2 * (n & 1) + 1] = lo[n >> 1][2 * (n & 1) + 1] = 0u;
        }
      }
      // values behind the last key any row sees may be anything, NaN too
#pragma unroll
      for (int y = 0; y < KS; ++y) {
        const int live = g.walk.end() - kb - key0 - 16 * y;  // of these 16 keys
        uint32_t m0 = ~0u, m1 = ~0u;
        if (live < 16) {
          const int k0 = 2 * t4;
          m0 = (k0 < live ? 0xffffu : 0u) | (k0 + 1 < live ? 0xffff0000u : 0u);
          m1 = (k0 + 8 < live ? 0xffffu : 0u) | (k0 + 9 < live ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          constexpr int N = D / 32;  // 16-channel steps of a half: their values stay in registers
          uint32_t vf[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            ldsm4_t(C::step(vs + 16 * y * C::ROWB, half * N + n), vf[n]);
            vf[n][0] &= m0;
            vf[n][1] &= m1;
            vf[n][2] &= m0;
            vf[n][3] &= m1;
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            mma16816(o[2 * (half * N + n)], hi[y], vf[n][0], vf[n][1]);
            mma16816(o[2 * (half * N + n) + 1], hi[y], vf[n][2], vf[n][3]);
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            mma16816(o[2 * (half * N + n)], lo[y], vf[n][0], vf[n][1]);
            mma16816(o[2 * (half * N + n) + 1], lo[y], vf[n][2], vf[n][3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8u * st);
      if (++st == a.stages) {
        st = 0;
        ph ^= 1u;
      }
    }

    // the warps' sums over their keys, then out or this CTA's part
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * r + g8;
      if (row < rows) {
        float* dst = red + (warp * a.red_rows + row) * RS + 2 * t4;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
      }
    }
    step_barrier<C::WARPS>();
    if constexpr (CLUSTER) {
      for (int x = 4 * threadIdx.x; x < rows * D; x += 4 * 32 * C::WARPS) {
        float* at = red + (x / D) * RS + x % D;
        float4 v = *reinterpret_cast<const float4*>(at);
#pragma unroll
        for (int i = 1; i < C::WARPS; ++i)
          add4(v, *reinterpret_cast<const float4*>(at + i * a.red_rows * RS));
        *reinterpret_cast<float4*>(at) = v;
      }
      return;  // one segment a CTA
    }
    // one answer for the warp, whose lanes meet again in the next item's waits:
    // the copying warp may give up between two lanes' reads
    dead = __any_sync(0xffffffffu, *static_cast<volatile int*>(&m->abort_flag) != 0);
    uint16_t* out = a.out + ((long long)(g.seq.q0 + kStepRows * g.qt) * w.heads + g.h) * D;
    const bool before = g.c0 != (int)blockIdx.x;
    float* part = step_part<D>(a, blockIdx.x, !before);
    for (int x = 4 * threadIdx.x; x < rows * D; x += 4 * 32 * C::WARPS) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < C::WARPS; ++i)
        add4(v, *reinterpret_cast<const float4*>(red + (i * a.red_rows + x / D) * RS + x % D));
      if (dead) continue;
      if (g.parts == 1)
        step_store<D>(out, w.heads, x, v, a.inv_n);
      else
        __stcg(reinterpret_cast<float4*>(part + x), v);
    }
    if (g.parts > 1) {
      const StepCut cut{out, rows, g.c0, g.parts};
      if (before)
        cut0 = cut;
      else
        cut1 = cut;
    }
    step_barrier<C::WARPS>();  // red is free for the next item
  }
  if (cut0.parts == 0 && cut1.parts == 0) return;
  // The last CTA to arrive at a cut item sums its parts in the CTAs' order, so
  // that the result does not depend on who is last.  One fence a CTA, after
  // the barrier and so for all the warps' stores.
  if (threadIdx.x == 0) {
    __threadfence();
    unsigned last = 0;
    if (cut0.parts && !dead && atomicAdd(a.counters + cut0.c0, 1u) == (unsigned)(cut0.parts - 1)) last |= 1u;
    if (cut1.parts && !dead && atomicAdd(a.counters + cut1.c0, 1u) == (unsigned)(cut1.parts - 1)) last |= 2u;
    // ready for the next launch
    if (last & 1u) a.counters[cut0.c0] = 0;
    if (last & 2u) a.counters[cut1.c0] = 0;
    m->last = last;
  }
  step_barrier<C::WARPS>();
  const unsigned last = m->last;
  if (last) __threadfence();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!(last >> k & 1u)) continue;
    const StepCut cut = k ? cut1 : cut0;
    for (int x = 4 * threadIdx.x; x < cut.rows * D; x += 4 * 32 * C::WARPS) {
      float4 v = __ldcg(reinterpret_cast<const float4*>(step_part<D>(a, cut.c0, true) + x));
#pragma unroll 1
      for (int i = 1; i < cut.parts; i += 8) {  // eight loads in flight
        float4 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] = i + j < cut.parts
                     ? __ldcg(reinterpret_cast<const float4*>(step_part<D>(a, cut.c0 + i + j, false) + x))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) add4(v, y[j]);
      }
      step_store<D>(cut.out, w.heads, x, v, a.inv_n);
    }
  }
}

// Few items of few blocks: a cluster of kStepCluster CTAs an item, each with
// an equal part of its blocks.  No CTA looks for its share, and the parts meet
// in shared memory instead of behind a fence and a counter.  Bound by latency:
// one token over 513 keys, 4 heads of 64, takes 4.4 us with pages of 16 (6.2 as
// equal shares), 4.2 with pages of 64 (6.0).
constexpr int kStepCluster = 8;

// The cluster's sums, a share of the values each CTA, in the CTAs' order.
template <int D>
__device__ void step_cluster_join(const StepArgs& a, const PagedSeg& g, int rank, const float* red,
                                  const int* abort_flag) {
  using C = StepCfg<D>;
  constexpr int RS = step_red_stride(D);
  cluster_barrier();
  const uint32_t mine = smem_u32(red), flag = smem_u32(abort_flag);
  int stop = 0;
#pragma unroll
  for (int r = 0; r < kStepCluster; ++r) {
    int f;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(f) : "r"(cluster_addr(flag, r)) : "memory");
    stop |= f;
  }
  uint16_t* out = a.out + ((long long)(g.seq.q0 + kStepRows * g.qt) * a.w.heads + g.h) * D;
  for (int x = 4 * (rank * C::THREADS + (int)threadIdx.x); x < g.walk.rows * D;
       x += 4 * kStepCluster * C::THREADS) {
    float4 y[kStepCluster];
#pragma unroll
    for (int r = 0; r < kStepCluster; ++r)
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(y[r].x), "=f"(y[r].y), "=f"(y[r].z), "=f"(y[r].w)
                   : "r"(cluster_addr(mine + 4u * (uint32_t)((x / D) * RS + x % D), r))
                   : "memory");
#pragma unroll
    for (int r = 1; r < kStepCluster; ++r) add4(y[0], y[r]);
    if (!stop) step_store<D>(out, a.w.heads, x, y[0], a.inv_n);
  }
  cluster_barrier();  // no CTA leaves while another reads its sums
}

template <int D, bool CLUSTER>
__global__ void __launch_bounds__(StepCfg<D>::THREADS)
    step_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                const StepArgs a) {
  using C = StepCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* tail = smem_raw + (base - raw) + a.stages * C::STAGEB;
  float* red = reinterpret_cast<float*>(tail);
  uint8_t* after = tail + step_red_bytes(a.red_rows, D);
  const uint32_t full = smem_u32(after), empty = full + 8u * C::MAX_STAGES;
  auto* m = reinterpret_cast<StepMisc<C::WARPS>*>(after + 2 * C::MAX_STAGES * 8);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x < a.stages) {
    mbar_init(full + 8u * threadIdx.x, 1);
    mbar_init(empty + 8u * threadIdx.x, C::WARPS);
    if (threadIdx.x == 0) {
      m->abort_flag = 0;
      mbar_init(full + 8u * C::MAX_STAGES - 8u, 1);  // for the test hook alone: a.stages < MAX_STAGES
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (threadIdx.x == 32 * C::WARPS) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tv)) : "memory");
  }
  after_previous_kernel();
  PagedWork w = a.w;
  PagedCursor c;
  PagedSeg g;
  int rank = 0;
  if constexpr (CLUSTER) {
    rank = (int)blockIdx.x % kStepCluster;
    const int item = (int)blockIdx.x / kStepCluster;
    c.e = item / w.heads;
    c.h = item - c.e * w.heads;
    g.qt = c.e / a.p.batch;
    g.b = c.e - g.qt * a.p.batch;
    if (!paged_seq(a.p, g.b, &g.seq) && item == g.b * w.heads && rank == 0 && threadIdx.x == 0)
      atomicOr(a.status, kStatusBadPaged);
    g.walk = paged_walk(g.seq, g.qt, w.tile_rows, w.kb_shift);
    if (g.walk.nb == 0) return;  // the same for the whole cluster
    const int from = rank * g.walk.nb / kStepCluster, to = (rank + 1) * g.walk.nb / kStepCluster;
    w.per = 1;
    c.cta = (int)blockIdx.x;
    c.u = c.u0 = 0;
    c.u1 = to - from;
    c.i = from;
    c.loaded = true;
    g.h = c.h;
    if (to == from)  // no block of its own: its sums are zero
      for (int x = threadIdx.x; x < a.red_rows * step_red_stride(D); x += C::THREADS) red[x] = 0.f;
    __syncthreads();
  } else {
    if (!paged_locate<C::WARPS + 1, false>(a.p, &w, &m->start, a.status, &c, &g)) return;
  }
  const StepWait wt{a.timeout_ns, &m->abort_flag, a.status};
  if (warp == C::WARPS)
    step_produce<D>(&tk, &tv, a, w, c, g, base, full, empty, wt);
  else
    step_compute<D, CLUSTER>(a, w, c, g, base, full, empty, red, m, wt);
  if constexpr (CLUSTER) step_cluster_join<D>(a, g, rank, red, &m->abort_flag);
}

constexpr int step_ring_bytes(int d) { return 128 * 1024 / step_per_sm(d); }
template <int D>
constexpr int kStepBytesMost = step_ring_bytes(D) + step_red_bytes(kStepRows, D) + kStepTailBytes + 1024;

// The kernels' shared memory, once a device.
template <int D>
cudaError_t step_prepare() {
  static DeviceOnce once;
  return once.run([] {
    const cudaError_t e = cudaFuncSetAttribute(
        step_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStepBytesMost<D>);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(step_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kStepBytesMost<D>);
  });
}

// Clusters that run at once, with the most shared memory a call may ask for.
template <int D>
cudaError_t step_clusters(int* n) {
  const cudaError_t e = step_prepare<D>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kStepCluster);
  cfg.blockDim = dim3(StepCfg<D>::THREADS);
  cfg.dynamicSmemBytes = kStepBytesMost<D>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kStepCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, step_kernel<D, true>, &cfg);
}
cudaError_t step_clusters_d(int d, int* n) {
  switch (d) {
    case 32: return step_clusters<32>(n);
    case 64: return step_clusters<64>(n);
    default: return step_clusters<128>(n);
  }
}

template <int D>
cudaError_t launch_step(const CUtensorMap& tk, const CUtensorMap& tv, long long most, bool clusters,
                        StepArgs a, int sms, cudaStream_t stream) {
  using C = StepCfg<D>;
  // 128 KB of copies in flight an SM.  More make every CTA's first block wait
  // for the others' queued copies and leave more blocks to compute once the
  // last bytes have landed: 512 sequences of log-normal lengths took 42.2 us
  // with 2 stages of 32 KB a CTA, 44.2 with 3.
  constexpr int PER_SM = step_per_sm(D), RING = 128 * 1024 / PER_SM;
  a.stages = RING / C::STAGEB;
  static_assert(RING / C::STAGEB >= 2 && RING / C::STAGEB < C::MAX_STAGES, "stages");
  const int extra = step_red_bytes(a.red_rows, D) + kStepTailBytes + 1024;
  const int bytes = a.stages * C::STAGEB + extra;
  static_assert(RING == step_ring_bytes(D), "ring");
  const cudaError_t e = step_prepare<D>();
  if (e != cudaSuccess) return e;
  if (clusters)
    return launch_after_in_clusters(kStepCluster, step_kernel<D, true>,
                                    kStepCluster * a.w.tiles * a.p.batch * a.w.heads, C::THREADS, bytes,
                                    stream, tk, tv, a);
  const int grid = (int)std::min<long long>((long long)PER_SM * sms, most);
  return launch_after(step_kernel<D, false>, grid, C::THREADS, bytes, stream, tk, tv, a);
}

cudaError_t launch_step_d(int d, const CUtensorMap& tk, const CUtensorMap& tv, long long most, bool clusters,
                          const StepArgs& a, int sms, cudaStream_t s) {
  switch (d) {
    case 32: return launch_step<32>(tk, tv, most, clusters, a, sms, s);
    case 64: return launch_step<64>(tk, tv, most, clusters, a, sms, s);
    default: return launch_step<128>(tk, tv, most, clusters, a, sms, s);
  }
}

int status_of(cudaError_t e) {
  if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction)
    return HSTU_ERR_UNSUPPORTED;
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

bool bad_ptr(const void* p, unsigned align) {
  return !p || (reinterpret_cast<uintptr_t>(p) & (align - 1u));
}

// The pool as (d, heads, page_size, num_pages) with box (min(d, 64), 1,
// min(page_size, 128), 1) and the swizzle of a box row.
int make_pool_map(CUtensorMap* m, void* ptr, int num_pages, int page_size, int heads, int d,
                  long long page_stride) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)page_size,
                              (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2u, (cuuint64_t)heads * (cuuint64_t)d * 2u,
                                 (cuuint64_t)page_stride * 2u};
  const cuuint32_t box[4] = {(cuuint32_t)std::min(d, 64), 1u, (cuuint32_t)std::min(page_size, kStepKeys), 1u};
  return host_encode_map(m, ptr, 4, dims, strides, box, d >= 64);
}

}  // namespace
}  // namespace hstu

// One pool of pages with its tensor maps; immutable after creation.
struct hstu_cache {
  void *k_pages, *v_pages;
  int num_pages, page_size, page_shift, heads, d;
  long long page_stride;
  int device, sms;
  unsigned* status;
  int clusters;        // clusters of the few-token kernel that run at once
  CUtensorMap tk, tv;  // boxes of up to 128 keys, both kernels' blocks
};

namespace {

using hstu::PagedView;

constexpr long long kCounterBytes = 8192;  // one counter a CTA, rounded up

// Two parts a CTA: up to 2 CTAs an SM with tiles of 16 rows, or one with 128.
long long part_bytes(const hstu_cache* c) {
  return (long long)c->sms * 2 * HSTU_BLOCK_M * c->d * (long long)sizeof(float);
}
size_t workspace_bytes(const hstu_cache* c) { return (size_t)(kCounterBytes + part_bytes(c)); }

// The batch's fields, and (host) the view the kernels take.
int check_batch(const hstu_paged_batch* b, PagedView* v, int num_pages, int page_shift) {
  if (!b || b->batch < 0 || b->rows < 0 || b->max_q < 0 || b->max_pages < 0) return HSTU_ERR_INVALID_ARG;
  if (b->batch > 0 && b->rows > 0 &&
      (hstu::bad_ptr(b->q_offsets, 4) || hstu::bad_ptr(b->kv_lens, 4) || hstu::bad_ptr(b->page_table, 4) ||
       (b->num_targets && hstu::bad_ptr(b->num_targets, 4)) || b->max_pages < 1))
    return HSTU_ERR_INVALID_ARG;
  // token positions are 32-bit
  if (((long long)b->max_pages << page_shift) > (1LL << 30)) return HSTU_ERR_INVALID_ARG;
  // no sequence has more new tokens than there are rows
  *v = PagedView{b->q_offsets, b->kv_lens, b->num_targets, b->page_table, b->batch, b->max_pages,
                 std::min(b->max_q, b->rows), b->rows, num_pages, page_shift};
  return HSTU_OK;
}

constexpr long long kMostUnits = 1 << 30;

// Units for what an item costs besides its blocks (its queries' load, the
// pipeline's filling, its rows' way out).  With 0, 1, 2 and 3 of them, 16 x
// 4096 tokens from an empty cache (items of 1 to 32 blocks) took 300, 242, 249
// and 252 us at d = 64, and 16 ragged chunks 76.8, 73.1, 69.9 and 70.8 us at
// d = 128; 512 single tokens 43.1, 42.2, 43.1 and 44.7.
constexpr int item_units(int d) { return d == 128 ? 2 : 1; }

// Units of a launch, at most: a tile walks every block of its sequence once.
long long units_bound(const PagedView& v, int heads, int tiles, int kb_shift, int extra) {
  const long long blocks = (((long long)v.max_pages << v.page_shift) >> kb_shift) + 2 + extra;
  const long long entries = (long long)tiles * v.batch;
  return entries > INT32_MAX || entries * heads > INT32_MAX ? LLONG_MAX : entries * heads * blocks;
}

// Whether more than one tile of 16 rows goes to the 128-row tcgen05 tiles
// instead.  Those take about 4 us more to fill their pipeline and less per
// block: 32 rows, 4 heads, d = 64 took 6.9 us as 16-row tiles and 10.5 as one
// tile on 600 keys, 10.5 and 13.3 on 8 x 2000, 24.2 and 24.4 on 16 x 4096, 70
// and 61 on 64 x 4096; 64 rows 15.3 and 16.5 on 8 x 2000, 36.7 and 26.0 on
// 16 x 4096.  At d = 128 the blocks cost more: 32 rows 11.0 and 13.5 on
// 4 x 2000, 19.0 and 16.7 on 8 x 2000.  `units`: blocks of the 16-row tiles, at
// most.
bool use_tiles(const PagedView& v, int d, int sms, long long units) {
  if (v.max_q <= hstu::kStepRows) return false;
  return v.max_q > 64 || units > (d == 128 ? 5LL : 20LL) * sms;
}

// Whether 16-row tiles get a cluster of CTAs an item: where all clusters run
// at once (`clusters_at_once`), there is more than one block to share, and no
// CTA has more than 8.  The lengths are not known here, so the table's width
// bounds the blocks.  One token, 4 heads of 64, pages of 64, as clusters and as
// equal shares (either without this rule): 4.2 us and 3.9 on 64 keys, one
// block, for which seven CTAs only start and meet; 4.2 and 6.0 on 513, 6.2 and
// 7.7 on 4096, 8.9 and 9.3 on 8192, 14.6 and 13.3 on 16384; 9 sequences 17.1
// and 18.5 on 8192.
bool use_clusters(const PagedView& v, int heads, int tiles, int clusters_at_once) {
  const long long items = (long long)tiles * v.batch * heads;
  const long long blocks = (((long long)v.max_pages << v.page_shift) + hstu::kStepKeys - 1) >> hstu::kStepShift;
  return items <= clusters_at_once && blocks > 1 && blocks <= 8LL * hstu::kStepCluster;
}

int check_geometry(int num_pages, int page_size, int* shift) {
  if (num_pages < 1 || page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)))
    return HSTU_ERR_INVALID_ARG;
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  return HSTU_OK;
}

bool bad_rows(const void* p, int64_t stride, long long width) {
  return hstu::bad_ptr(p, 16) || stride < width || (stride & 7);
}

int check_device(const hstu_cache* c) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return HSTU_ERR_CUDA;
  return dev == c->device ? HSTU_OK : HSTU_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int hstu_cache_create(void* k_pages, void* v_pages, int num_pages, int page_size, int heads, int d,
                      int64_t page_stride, hstu_cache** cache) {
  if (!cache) return HSTU_ERR_INVALID_ARG;
  *cache = nullptr;
  if (d != 32 && d != 64 && d != 128) return HSTU_ERR_UNSUPPORTED;
  int shift = 0;
  if (heads < 1 || heads > (1 << 16) || check_geometry(num_pages, page_size, &shift) != HSTU_OK)
    return HSTU_ERR_INVALID_ARG;
  const long long packed = (long long)page_size * heads * d;
  if (page_stride == 0) page_stride = packed;
  if (hstu::bad_ptr(k_pages, 16) || hstu::bad_ptr(v_pages, 16) || page_stride < packed ||
      (page_stride & 7) || page_stride >= (1LL << 39))
    return HSTU_ERR_INVALID_ARG;
  hstu_cache* c = new (std::nothrow) hstu_cache{};
  if (!c) return HSTU_ERR_NO_MEMORY;
  c->k_pages = k_pages;
  c->v_pages = v_pages;
  c->num_pages = num_pages;
  c->page_size = page_size;
  c->page_shift = shift;
  c->heads = heads;
  c->d = d;
  c->page_stride = page_stride;
  int rc = hstu::host_device_check(&c->sms);
  if (rc == HSTU_OK && cudaGetDevice(&c->device) != cudaSuccess) rc = HSTU_ERR_CUDA;
  if (rc == HSTU_OK && hstu::device_status_words(&c->status) != cudaSuccess) rc = HSTU_ERR_CUDA;
  if (rc == HSTU_OK) rc = hstu::status_of(hstu::step_clusters_d(d, &c->clusters));
  if (rc == HSTU_OK)
    rc = hstu::make_pool_map(&c->tk, k_pages, num_pages, page_size, heads, d, page_stride);
  if (rc == HSTU_OK)
    rc = hstu::make_pool_map(&c->tv, v_pages, num_pages, page_size, heads, d, page_stride);
  if (rc != HSTU_OK) {
    delete c;
    return rc;
  }
  *cache = c;
  return HSTU_OK;
}

int hstu_cache_destroy(hstu_cache* cache) {
  delete cache;
  return HSTU_OK;
}

int hstu_cache_workspace(const hstu_cache* cache, size_t* bytes) {
  if (!cache || !bytes) return HSTU_ERR_INVALID_ARG;
  *bytes = workspace_bytes(cache);
  return HSTU_OK;
}

int hstu_cache_slots(const hstu_paged_batch* host_batch, int num_pages, int page_size, int64_t* host_slot,
                     int32_t* host_pos) {
  int shift = 0;
  if (check_geometry(num_pages, page_size, &shift) != HSTU_OK) return HSTU_ERR_INVALID_ARG;
  PagedView v;
  const int rc = check_batch(host_batch, &v, num_pages, shift);
  if (rc != HSTU_OK) return rc;
  if (v.rows > 0 && (!host_slot || !host_pos)) return HSTU_ERR_INVALID_ARG;
  int bad = 0;
  hstu::PagedSeq seq;
  for (int b = 0; v.rows > 0 && b < v.batch; ++b)
    if (!hstu::paged_seq(v, b, &seq)) bad = 1;
  for (int t = 0; t < v.rows; ++t) {
    host_slot[t] = -1;
    host_pos[t] = -1;
    if (v.batch == 0 || t >= v.q_offsets[v.batch]) continue;
    const int b = hstu::paged_find(v, t);
    hstu::PagedSeq s;
    if (b < 0 || !hstu::paged_seq(v, b, &s)) continue;
    const int pos = s.kv - s.qn + (t - s.q0);
    host_slot[t] = hstu::paged_slot(v, b, pos);
    host_pos[t] = pos < s.hist ? pos : s.hist;
    if (host_slot[t] < 0) bad = 1;
  }
  return bad ? HSTU_ERR_INVALID_ARG : HSTU_OK;
}

int hstu_cache_worklist(const hstu_paged_batch* host_batch, int num_pages, int page_size, int heads,
                        int tile_rows, int block_keys, int extra, int grid, int min_units, int32_t* host_dst,
                        int capacity, int* n_segments) {
  int shift = 0;
  if (check_geometry(num_pages, page_size, &shift) != HSTU_OK) return HSTU_ERR_INVALID_ARG;
  if (!n_segments || heads < 1 || tile_rows < 1 || block_keys < 1 || (block_keys & (block_keys - 1)) ||
      extra < 0 || extra > 64 || grid < 1 || min_units < 1 || capacity < 0)
    return HSTU_ERR_INVALID_ARG;
  PagedView v;
  const int rc = check_batch(host_batch, &v, num_pages, shift);
  if (rc != HSTU_OK) return rc;
  hstu::PagedWork w{};
  w.heads = heads;
  w.extra = extra;
  w.tile_rows = tile_rows;
  w.tiles = v.rows > 0 && v.batch > 0 && v.max_q > 0 ? (v.max_q - 1) / tile_rows + 1 : 0;
  while ((1 << w.kb_shift) < block_keys) ++w.kb_shift;
  if (units_bound(v, heads, w.tiles, w.kb_shift, extra) > kMostUnits) return HSTU_ERR_INVALID_ARG;
  auto units_of = [&](int e) {
    hstu::PagedSeq s;
    hstu::paged_seq(v, e % v.batch, &s);
    return hstu::paged_units(w, hstu::paged_walk(s, e / v.batch, tile_rows, w.kb_shift).nb);
  };
  for (int e = 0; e < w.tiles * v.batch; ++e) w.total += units_of(e);
  w.per = hstu::paged_share(w, v.batch, grid, min_units);
  int n = 0;
  for (int cta = 0; cta < grid && (long long)cta * w.per < w.total; ++cta) {
    hstu::PagedCursor c{};
    c.cta = cta;
    c.u = c.u0 = cta * w.per;
    c.u1 = (int)std::min<long long>((long long)c.u + w.per, w.total);
    int at = 0;
    while (at + units_of(c.e) <= c.u) at += units_of(c.e++);
    hstu::PagedSeg g;
    c.load(v, w, &g);
    c.loaded = true;
    c.h = (c.u - at) / (g.walk.nb + extra);
    c.i = c.u - at - c.h * (g.walk.nb + extra);
    while (c.next(v, w, &g)) {
      if (host_dst) {
        if (n >= capacity) return HSTU_ERR_INVALID_ARG;
        const int32_t x[8] = {cta, g.b, g.h, g.qt, g.i0, g.n, g.c0, g.parts};
        std::copy(x, x + 8, host_dst + 8 * (size_t)n);
      }
      ++n;
    }
  }
  *n_segments = n;
  return HSTU_OK;
}

int hstu_cache_append(const hstu_cache* cache, const hstu_paged_batch* batch, const void* q,
                      int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      const hstu_rotary* rotary, void* q_out, hstu_stream_t stream) {
  if (!cache) return HSTU_ERR_INVALID_ARG;
  hstu::AppendArgs a{};
  int rc = check_batch(batch, &a.p, cache->num_pages, cache->page_shift);
  if (rc != HSTU_OK) return rc;
  const int width = cache->heads * cache->d;
  if (!q != !q_out) return HSTU_ERR_INVALID_ARG;
  if (rotary && (hstu::bad_ptr(rotary->table, 16) || rotary->positions < 1 || rotary->dim < 16 ||
                 rotary->dim > cache->d || (rotary->dim & 15) ||
                 (rotary->pairs != 0 && rotary->pairs != 1)))
    return HSTU_ERR_INVALID_ARG;
  if (a.p.rows == 0 || a.p.batch == 0) return HSTU_OK;
  if (bad_rows(k, k_stride, width) || bad_rows(v, v_stride, width)) return HSTU_ERR_INVALID_ARG;
  if (q && (bad_rows(q, q_stride, width) || hstu::bad_ptr(q_out, 16))) return HSTU_ERR_INVALID_ARG;
  if ((rc = check_device(cache)) != HSTU_OK) return rc;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_pages = static_cast<uint16_t*>(cache->k_pages);
  a.v_pages = static_cast<uint16_t*>(cache->v_pages);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.page_stride = cache->page_stride;
  a.table = rotary ? rotary->table : nullptr;
  a.positions = rotary ? rotary->positions : 0;
  a.rot = rotary ? rotary->dim : 0;
  a.pairs = rotary ? rotary->pairs : 0;
  a.heads = cache->heads;
  a.d = cache->d;
  a.status = cache->status;
  const long long units = (long long)a.p.rows * (width / 16);
  a.check_ctas = ((unsigned)a.p.batch + hstu::kAppendThreads - 1) / hstu::kAppendThreads;
  const long long grid = a.check_ctas + (units + hstu::kAppendThreads - 1) / hstu::kAppendThreads;
  if (grid > 0x7fffffffLL) return HSTU_ERR_INVALID_ARG;
  return hstu::status_of(hstu::launch_after(hstu::append_kernel, (int)grid, hstu::kAppendThreads, 0,
                                            reinterpret_cast<cudaStream_t>(stream), a));
}

int hstu_attn_fwd_cache(const hstu_cache* cache, const hstu_paged_batch* batch, const void* q,
                        int64_t q_stride, float alpha, float inv_n, void* out, void* workspace,
                        hstu_stream_t stream) {
  if (!cache) return HSTU_ERR_INVALID_ARG;
  PagedView p;
  int rc = check_batch(batch, &p, cache->num_pages, cache->page_shift);
  if (rc != HSTU_OK) return rc;
  if (workspace && hstu::bad_ptr(workspace, 16)) return HSTU_ERR_INVALID_ARG;
  if (p.rows == 0 || p.batch == 0) return HSTU_OK;
  const int heads = cache->heads, d = cache->d;
  if (bad_rows(q, q_stride, (long long)heads * d) || hstu::bad_ptr(out, 16)) return HSTU_ERR_INVALID_ARG;
  if ((rc = check_device(cache)) != HSTU_OK) return rc;
  hstu::PagedWork w{};
  w.heads = heads;
  w.tile_rows = hstu::kStepRows;
  w.tiles = p.max_q > 0 ? (p.max_q - 1) / w.tile_rows + 1 : 1;  // a bound of 0: only the lengths are checked
  w.kb_shift = hstu::kStepShift;  // both kernels' blocks have 128 keys
  w.extra = item_units(d);
  const bool tiled = use_tiles(p, d, cache->sms, units_bound(p, heads, w.tiles, w.kb_shift, w.extra));
  if (tiled) {
    w.tile_rows = HSTU_BLOCK_M;
    w.tiles = (p.max_q - 1) / w.tile_rows + 1;
  }
  const long long most = units_bound(p, heads, w.tiles, w.kb_shift, w.extra);
  if (most > kMostUnits) return HSTU_ERR_INVALID_ARG;
  const bool clusters = !tiled && use_clusters(p, heads, w.tiles, cache->clusters);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap tq;
  if (tiled) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)p.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2u, (cuuint64_t)q_stride * 2u};
    const cuuint32_t box[3] = {(cuuint32_t)std::min(d, 64), 1u, (cuuint32_t)HSTU_BLOCK_M};
    if (q_stride >= (1LL << 39)) return HSTU_ERR_INVALID_ARG;
    if ((rc = hstu::host_encode_map(&tq, const_cast<void*>(q), 3, dims, strides, box, d >= 64)) != HSTU_OK)
      return rc;
  }
  char* own = nullptr;
  if (!workspace && !clusters) {
    cudaError_t e = cudaMallocAsync(reinterpret_cast<void**>(&own), workspace_bytes(cache), s);
    if (e != cudaSuccess) return e == cudaErrorMemoryAllocation ? HSTU_ERR_NO_MEMORY : HSTU_ERR_CUDA;
    if (cudaMemsetAsync(own, 0, (size_t)kCounterBytes, s) != cudaSuccess) {
      cudaFreeAsync(own, s);
      return HSTU_ERR_CUDA;
    }
    workspace = own;
  }
  unsigned* counters = static_cast<unsigned*>(workspace);
  float* parts = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes) : nullptr;
  cudaError_t e;
  if (tiled) {
    hstu::PagedFwdArgs a{};
    a.p = p;
    a.w = w;
    a.out = static_cast<uint16_t*>(out);
    a.half_alpha = 0.5f * alpha;
    a.inv_n = inv_n;
    a.counters = counters;
    a.parts = parts;
    a.timeout_ns = hstu::host_wait_timeout_ns();
    a.debug_flags = hstu::host_debug_flags();
    const int grid = (int)std::min<long long>(cache->sms, most);
    e = hstu::launch_fwd_paged(d, tq, cache->tk, cache->tv, a, grid, s);
  } else {
    hstu::StepArgs a{};
    a.p = p;
    a.w = w;
    a.red_rows = std::min(p.max_q, w.tile_rows);
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.out = static_cast<uint16_t*>(out);
    a.half_alpha = 0.5f * alpha;
    a.inv_n = inv_n;
    a.counters = counters;
    a.parts = parts;
    a.status = cache->status;
    a.timeout_ns = hstu::host_wait_timeout_ns();
    a.debug_flags = hstu::host_debug_flags();
    e = hstu::launch_step_d(d, cache->tk, cache->tv, most, clusters, a, cache->sms, s);
  }
  rc = hstu::status_of(e);
  if (own && cudaFreeAsync(own, s) != cudaSuccess && rc == HSTU_OK) rc = HSTU_ERR_CUDA;
  return rc;
}

}  // extern "C"
