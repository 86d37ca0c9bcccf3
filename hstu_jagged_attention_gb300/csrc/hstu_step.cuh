// What the kernels of few new tokens over the paged cache share, whatever the
// cache holds: their arguments, bounded waits, the products, and how the parts
// of an item that several CTAs walk become one.
#pragma once

#include "hstu_internal.h"
#include "hstu_paged.cuh"
#include "hstu_ptx.cuh"

namespace hstu {
namespace {

constexpr int kStepRows = 16;
constexpr int kStepKeys = 128, kStepShift = 7;
constexpr int kStepPerSm = 3;  // CTAs of such a kernel an SM, at most

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

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 floats between rows, so that eight rows' 8-byte stores meet all banks
__host__ __device__ constexpr int step_red_stride(int d) { return d + 8; }

template <int WARPS>
struct StepMisc {
  int abort_flag;
  unsigned last;  // bits: this CTA arrived last at the items it shares
  PagedStart<WARPS + 1> start;
};

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

// Behind a CTA's last item.
template <int D, int WARPS>
__device__ __forceinline__ void step_join(const StepArgs& a, const PagedWork& w, StepMisc<WARPS>* m,
                                          const StepCut& cut0, const StepCut& cut1, bool dead) {
  if (cut0.parts == 0 && cut1.parts == 0) return;
  // The last CTA to arrive at a cut item sums its parts in the CTAs' order, so
  // that the result does not depend on who is last.  One fence a CTA, after
  // the barrier and so for all the warps' stores.
  if (threadIdx.x < 2) {  // a thread an item: their counters' round trips overlap
    __threadfence();
    const StepCut cut = threadIdx.x ? cut1 : cut0;
    const bool last = cut.parts && !dead && atomicAdd(a.counters + cut.c0, 1u) == (unsigned)(cut.parts - 1);
    if (last) a.counters[cut.c0] = 0;  // ready for the next launch
    const unsigned both = __ballot_sync(3u, last);
    if (threadIdx.x == 0) m->last = both;
  }
  step_barrier<WARPS>();
  const unsigned last = m->last;
  if (last) __threadfence();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!(last >> k & 1u)) continue;
    const StepCut cut = k ? cut1 : cut0;
    for (int x = 4 * threadIdx.x; x < cut.rows * D; x += 4 * 32 * WARPS) {
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

// The share of this CTA, `rank` of its cluster: blocks c->i .. of its item, c->u1
// of them.  False, for the whole cluster, where the item has none.
__device__ __forceinline__ bool step_cluster_share(const StepArgs& a, int rank, PagedWork* w, PagedCursor* c,
                                                   PagedSeg* g) {
  const int item = (int)blockIdx.x / kStepCluster;
  c->e = item / w->heads;
  c->h = item - c->e * w->heads;
  g->qt = c->e / a.p.batch;
  g->b = c->e - g->qt * a.p.batch;
  if (!paged_seq(a.p, g->b, &g->seq) && item == g->b * w->heads && rank == 0 && threadIdx.x == 0)
    atomicOr(a.status, kStatusBadPaged);
  g->walk = paged_walk(g->seq, g->qt, w->tile_rows, w->kb_shift);
  if (g->walk.nb == 0) return false;
  const int from = rank * g->walk.nb / kStepCluster, to = (rank + 1) * g->walk.nb / kStepCluster;
  w->per = 1;
  c->cta = (int)blockIdx.x;
  c->u = c->u0 = 0;
  c->u1 = to - from;
  c->i = from;
  c->loaded = true;
  g->h = c->h;
  return true;
}

// Clusters that run at once, with `bytes` of shared memory a CTA.
template <class... Params>
cudaError_t clusters_at_once(void (*kernel)(Params...), int threads, int bytes, int* n) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kStepCluster);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kStepCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
}

// The cluster's sums, a share of the values each CTA, in the CTAs' order.
template <int D, int THREADS>
__device__ void step_cluster_join(const StepArgs& a, const PagedSeg& g, int rank, const float* red,
                                  const int* abort_flag) {
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
  for (int x = 4 * (rank * THREADS + (int)threadIdx.x); x < g.walk.rows * D;
       x += 4 * kStepCluster * THREADS) {
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

}  // namespace
}  // namespace hstu
