// Layer norm over a row, with the residual before it and the gate after it,
// and its gradient (HSTU paper section 3: a layer is a residual around
// Norm(A V) (.) U between two projections; section 3.1 asks for the norm).
//
//   z = residual + scale x   (or x),   xhat = (z - mean(z)) / sqrt(var(z) + eps)
//   y = (xhat gamma + beta) (.) u      (or without u)
//
//   g = dy (.) u,  a = g gamma,  du = dy (.) (xhat gamma + beta)
//   dz = rstd (a - mean(a) - xhat mean(a xhat)) + dz_in,   dx = scale dz
//   dgamma = sum over rows of g xhat,   dbeta = sum over rows of g
//
// Both are bound by memory: a few operations a byte.  A group of LANES lanes
// holds a row in registers, NV vectors of 8 channels a lane, so every array
// is read once; mean and variance are two passes over the registers, in 32
// bits.  37,611 rows of 512 with the residual take 25.7 us forward (154 MB,
// 6.0 TB/s); the gradient of 65,536 rows of 256 with the gate 30 us (168 MB),
// of which the rows 25 and the sums of dgamma and dbeta the rest.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hstu_attn.h"
#include "hstu_internal.h"
#include "hstu_ptx.cuh"

namespace {

struct NormFwdArgs {
  const uint16_t *x, *residual, *u;
  long long x_stride, residual_stride, u_stride;
  const float *gamma, *beta;
  float scale, eps;
  long long rows;
  int width;
  uint16_t *y, *z;
};

struct NormBwdArgs {
  const uint16_t *dy, *z, *u, *dz_in;
  long long dy_stride, z_stride, u_stride, dz_in_stride, du_stride;
  const float *gamma, *beta;
  float scale, eps;
  long long rows;
  int width;
  uint16_t *dz, *dx, *du;
  float* parts;  // [grid][2][width]: each CTA's dgamma and dbeta
  float *dgamma, *dbeta;  // given: the grid is one cluster, which sums them itself
};

// 8 channels of a row, as four pairs (the packed fp32 operations take pairs).
struct V8 {
  float2 f[4];
};

__device__ __forceinline__ V8 unpack(const uint4& p) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v.f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return v;
}

__device__ __forceinline__ uint32_t pack2(float2 v) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}

__device__ __forceinline__ uint4 pack(const V8& v) {
  return make_uint4(pack2(v.f[0]), pack2(v.f[1]), pack2(v.f[2]), pack2(v.f[3]));
}

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

__device__ __forceinline__ uint4 ld_row(const uint16_t* p, long long at) {
  return __ldcs(reinterpret_cast<const uint4*>(p + at));
}

__device__ __forceinline__ V8 ld_f32(const float* p, int at) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + at));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + at) + 1);
  return V8{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}

// Sums each of N values over the LANES lanes of the caller's group.  Groups of
// several warps go through `red` (2 N floats a warp, its halves used in turn
// so that one barrier a sum is enough) and meet at their own barrier.
template <int LANES, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int* turn) {
#pragma unroll
  for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (LANES > 32) {
    constexpr int W = LANES / 32;
    const int group = threadIdx.x / LANES;
    float* mine = red + (2 * group + *turn) * N * W;
    *turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) mine[i * W + (threadIdx.x / 32) % W] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(LANES) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += mine[i * W + w];
      v[i] = s;
    }
  }
}

// The next row's loads are issued before the current row is computed.
constexpr int kFwdThreads = 256;

template <int LANES, int NV, bool GATE, bool RES>
__global__ void __launch_bounds__(kFwdThreads) norm_fwd_kernel(const NormFwdArgs a) {
  hstu::after_previous_kernel();
  __shared__ float red[2 * kFwdThreads / 32];
  int turn = 0;
  const int lane = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  constexpr int GROUPS = kFwdThreads / LANES;
  const float inv_w = 1.f / (float)a.width;
  // every lane of a warp stays in the loop (its shuffles need them), with
  // its loads and stores off past the last row
  const long long step = (long long)gridDim.x * GROUPS;
  uint4 xp[NV], rp[NV], up[NV];
  auto load = [&](long long r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      xp[i] = rp[i] = make_uint4(0, 0, 0, 0);
      if (r < a.rows && c < a.width) {
        xp[i] = ld_row(a.x, r * a.x_stride + c);
        if (RES) rp[i] = ld_row(a.residual, r * a.residual_stride + c);
        if (GATE) up[i] = ld_row(a.u, r * a.u_stride + c);
      }
    }
  };
  long long r0 = (long long)blockIdx.x * GROUPS;
  load(r0 + group);
  for (; r0 < a.rows; r0 += step) {
    const long long r = r0 + group;
    const bool live = r < a.rows;
    V8 z[NV];
    uint4 uc[NV];
    float2 acc = pair(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      z[i] = unpack(xp[i]);
      uc[i] = up[i];
      if (RES) {
        const V8 rv = unpack(rp[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) z[i].f[j] = __ffma2_rn(pair(a.scale), z[i].f[j], rv.f[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = __fadd2_rn(acc, z[i].f[j]);
    }
    if (r0 + step < a.rows) load(r + step);
    if (RES) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (lane + i * LANES);
        if (live && c < a.width) *reinterpret_cast<uint4*>(a.z + r * a.width + c) = pack(z[i]);
      }
    }
    float s[1] = {acc.x + acc.y};
    group_sum<LANES, 1>(s, red, &turn);
    const float mean = s[0] * inv_w;
    acc = pair(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = 8 * (lane + i * LANES) < a.width;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[i].f[j] = __fadd2_rn(z[i].f[j], pair(-mean));
        if (in) acc = __ffma2_rn(z[i].f[j], z[i].f[j], acc);
      }
    }
    float q[1] = {acc.x + acc.y};
    group_sum<LANES, 1>(q, red, &turn);
    const float rstd = rsqrtf(fmaf(q[0], inv_w, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      if (!live || c >= a.width) continue;
      const V8 g = ld_f32(a.gamma, c), b = ld_f32(a.beta, c);
      V8 y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y.f[j] = __ffma2_rn(__fmul2_rn(z[i].f[j], pair(rstd)), g.f[j], b.f[j]);
      if (GATE) {
        const V8 u = unpack(uc[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y.f[j] = __fmul2_rn(y.f[j], u.f[j]);
      }
      *reinterpret_cast<uint4*>(a.y + r * a.width + c) = pack(y);
    }
  }
}

// The gradient's rows ahead of the one computed: each lane copies its own vectors of the next
// rows into shared memory and reads back only those, so no barrier is needed
// and the copies in flight cost no registers.  With the next row alone in
// registers, the gradient of 65,536 rows of 256 with the gate took 38.3 us.
template <int THREADS, int ARRAYS, int NV>
struct RowRing {
  static constexpr int STAGES = NV == 1 ? 4 : NV == 2 ? 3 : 2;
  static constexpr int BYTES = STAGES * ARRAYS * NV * THREADS * 16;
  uint32_t base;
  int put = 0, get = 0;
  __device__ __forceinline__ explicit RowRing(const void* smem)
      : base((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16) {}
  __device__ __forceinline__ uint32_t at(int stage, int array, int i) const {
    return base + (uint32_t)(((stage * ARRAYS + array) * NV + i) * THREADS * 16);
  }
  // 8 channels from p, or zeros
  __device__ __forceinline__ void copy(int array, int i, const uint16_t* p, bool in) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(put, array, i)), "l"(p),
                 "r"(in ? 16 : 0)
                 : "memory");
  }
  __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put + 1 == STAGES ? 0 : put + 1;
  }
  // The oldest row has landed: its vectors may be read until step().
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
  }
  __device__ __forceinline__ uint4 read(int array, int i) const {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at(get, array, i))
                 : "memory");
    return v;
  }
  __device__ __forceinline__ void step() { get = get + 1 == STAGES ? 0 : get + 1; }
};

// One CTA an SM, so that few CTAs hand over sums of dgamma and dbeta.
constexpr int kBwdThreads = 512;

template <int LANES, int NV, bool GATE, bool RES>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float red[2 * 2 * kBwdThreads / 32];
  int turn = 0;
  const int lane = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  constexpr int GROUPS = kBwdThreads / LANES;
  const float inv_w = 1.f / (float)a.width;
  hstu::after_previous_kernel();
  V8 gm[NV], bt[NV], dg[NV], db[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (lane + i * LANES);
    gm[i] = bt[i] = dg[i] = db[i] = V8{{pair(0.f), pair(0.f), pair(0.f), pair(0.f)}};
    if (c < a.width) {
      gm[i] = ld_f32(a.gamma, c);
      if (GATE) bt[i] = ld_f32(a.beta, c);
    }
  }
  extern __shared__ uint4 smem[];
  RowRing<kBwdThreads, 2 + GATE + RES, NV> ring(smem);
  constexpr int U = 2, I = 2 + GATE;  // the arrays behind z and dy
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      const bool in = r < a.rows && c < a.width;
      ring.copy(0, i, in ? a.z + r * a.z_stride + c : a.z, in);
      ring.copy(1, i, in ? a.dy + r * a.dy_stride + c : a.dy, in);
      if (GATE) ring.copy(U, i, in ? a.u + r * a.u_stride + c : a.u, in);
      if (RES) ring.copy(I, i, in && a.dz_in ? a.dz_in + r * a.dz_in_stride + c : a.z, in && a.dz_in);
    }
    ring.commit();
  };
  const long long step = (long long)gridDim.x * GROUPS;
  long long r0 = (long long)blockIdx.x * GROUPS;
#pragma unroll 1
  for (int i = 0; i < ring.STAGES - 1; ++i) fetch(r0 + i * step + group);
  for (; r0 < a.rows; r0 += step) {
    const long long r = r0 + group;
    const bool live = r < a.rows;
    // first the sums that need no statistics, then those about the mean; past
    // the row's end gamma is 0, and so is a = g gamma
    V8 z[NV], g[NV];
    uint4 dyc[NV], ic[NV];
    float2 s0 = pair(0.f), s1 = s0;
    ring.wait();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      z[i] = unpack(ring.read(0, i));
      dyc[i] = ring.read(1, i);
      g[i] = unpack(dyc[i]);
      if (RES) ic[i] = ring.read(I, i);
      if (GATE) {
        const V8 u = unpack(ring.read(U, i));
#pragma unroll
        for (int j = 0; j < 4; ++j) g[i].f[j] = __fmul2_rn(g[i].f[j], u.f[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s0 = __fadd2_rn(s0, z[i].f[j]);
        s1 = __ffma2_rn(g[i].f[j], gm[i].f[j], s1);
      }
    }
    ring.step();
    fetch(r + (ring.STAGES - 1) * step);
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    group_sum<LANES, 2>(s, red, &turn);
    const float mean = s[0] * inv_w, mean_a = s[1] * inv_w;
    s0 = s1 = pair(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = 8 * (lane + i * LANES) < a.width;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[i].f[j] = __fadd2_rn(z[i].f[j], pair(-mean));
        if (in) s0 = __ffma2_rn(z[i].f[j], z[i].f[j], s0);
        s1 = __ffma2_rn(z[i].f[j], __fmul2_rn(g[i].f[j], gm[i].f[j]), s1);
      }
    }
    float q[2] = {s0.x + s0.y, s1.x + s1.y};
    group_sum<LANES, 2>(q, red, &turn);
    const float rstd = rsqrtf(fmaf(q[0], inv_w, a.eps));
    const float mean_ax = q[1] * inv_w * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      if (!live || c >= a.width) continue;
      V8 dz, du;
      const V8 dy = unpack(dyc[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 h = __fmul2_rn(z[i].f[j], pair(rstd));
        dg[i].f[j] = __ffma2_rn(g[i].f[j], h, dg[i].f[j]);
        db[i].f[j] = __fadd2_rn(db[i].f[j], g[i].f[j]);
        const float2 x = __ffma2_rn(g[i].f[j], gm[i].f[j], pair(-mean_a));
        dz.f[j] = __fmul2_rn(__ffma2_rn(h, pair(-mean_ax), x), pair(rstd));
        if (GATE) du.f[j] = __fmul2_rn(dy.f[j], __ffma2_rn(h, gm[i].f[j], bt[i].f[j]));
      }
      if (GATE) *reinterpret_cast<uint4*>(a.du + r * a.du_stride + c) = pack(du);
      if (RES) {
        const V8 in = unpack(ic[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) dz.f[j] = __fadd2_rn(dz.f[j], in.f[j]);
      }
      *reinterpret_cast<uint4*>(a.dz + r * a.width + c) = pack(dz);
      if (RES && a.dx) {
#pragma unroll
        for (int j = 0; j < 4; ++j) dz.f[j] = __fmul2_rn(dz.f[j], pair(a.scale));
        *reinterpret_cast<uint4*>(a.dx + r * a.width + c) = pack(dz);
      }
    }
  }
  // the CTA's sums: the groups' in order, through shared memory, to its part,
  // or where the cluster's other CTAs read them
  float* acc = reinterpret_cast<float*>(smem);  // 8 floats a thread, once its copies have landed
  float* kept = acc + (GROUPS > 1 ? 8 * kBwdThreads : 0);
  float* out = a.dgamma ? kept : a.parts + (long long)blockIdx.x * 2 * a.width;
  asm volatile("cp.async.wait_all;" ::: "memory");
  // `kept` lies over the other threads' vectors too, where their copies of the
  // rows past the end (zeros) may still land; with several groups the barrier
  // in the loop stands before the first store
  if constexpr (GROUPS == 1) __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const V8& v = k ? db[i] : dg[i];
      const int c = 8 * (lane + i * LANES);
      if constexpr (GROUPS == 1) {
        if (c < a.width)
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(out + k * a.width + c + 2 * j) = v.f[j];
      } else {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[(2 * j) * kBwdThreads + threadIdx.x] = v.f[j].x;
          acc[(2 * j + 1) * kBwdThreads + threadIdx.x] = v.f[j].y;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < 8 * LANES; x += kBwdThreads) {
          const int l = x % LANES, j = x / LANES;
          const int cc = 8 * (l + i * LANES) + j;
          if (cc >= a.width) continue;
          float t = 0.f;
#pragma unroll
          for (int y = 0; y < GROUPS; ++y) t += acc[j * kBwdThreads + y * LANES + l];
          out[k * a.width + cc] = t;
        }
      }
    }
  if (!a.dgamma) return;
  // each CTA sums a share of the columns over the cluster's CTAs, in order
  hstu::cluster_barrier();
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(kept);
  for (int x = blockIdx.x * kBwdThreads + threadIdx.x; x < 2 * a.width; x += gridDim.x * kBwdThreads) {
    float t = 0.f;
    for (int r = 0; r < (int)gridDim.x; ++r) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(hstu::cluster_addr(mine + 4u * x, r)) : "memory");
      t += v;
    }
    if (x < a.width)
      a.dgamma[x] = t;
    else
      a.dbeta[x - a.width] = t;
  }
  hstu::cluster_barrier();  // no CTA leaves while another reads its sums
}

// dgamma and dbeta: the CTAs' sums in a fixed order.  A block takes 32 of the
// 2 width columns; its 16 warps take the CTAs in turn.
constexpr int kSumThreads = 512;
__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float* parts, int n, int width,
                                                               float* dgamma, float* dbeta) {
  constexpr int W = kSumThreads / 32;
  __shared__ float acc[W][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = 32 * blockIdx.x + lane;
  hstu::after_previous_kernel();
  float s = 0.f;
  if (col < 2 * width) {
    // ten loads in flight: all of a warp's share of 152 CTAs
    for (int i0 = warp; i0 < n; i0 += 10 * W) {
      float x[10];
#pragma unroll
      for (int k = 0; k < 10; ++k) {
        const int i = i0 + k * W;
        x[k] = i < n ? __ldcg(parts + (long long)i * 2 * width + col) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 10; ++k) s += x[k];
    }
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < 2 * width) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += acc[w][lane];
    if (col < width)
      dgamma[col] = t;
    else
      dbeta[col - width] = t;
  }
}

// CTAs of a launch: enough to fill the GPU, no more than there are row groups.
int norm_grid(long long rows, int groups, int per_sm, int sms) {
  return (int)std::max<long long>(1, std::min<long long>((rows + groups - 1) / groups,
                                                         (long long)per_sm * sms));
}

constexpr int kFwdPerSm = 8;

template <int LANES, int NV>
cudaError_t fwd(const NormFwdArgs& a, int sms, cudaStream_t s) {
  const int grid = norm_grid(a.rows, kFwdThreads / LANES, kFwdPerSm, sms);
  if (a.u && a.residual)
    return hstu::launch_after(norm_fwd_kernel<LANES, NV, true, true>, grid, kFwdThreads, 0, s, a);
  if (a.u)
    return hstu::launch_after(norm_fwd_kernel<LANES, NV, true, false>, grid, kFwdThreads, 0, s, a);
  if (a.residual)
    return hstu::launch_after(norm_fwd_kernel<LANES, NV, false, true>, grid, kFwdThreads, 0, s, a);
  return hstu::launch_after(norm_fwd_kernel<LANES, NV, false, false>, grid, kFwdThreads, 0, s, a);
}

// Few rows, up to two a group: one cluster of up to 8 CTAs, which sums dgamma
// and dbeta itself.  It saves the second launch, 2 us of the calling thread's
// time; on the GPU 128 rows of 256 channels (gate and residual) take 4.4 us
// either way, 256 rows 5.3 us against 4.6, and 1024 rows 10.3 against 4.6.
int cluster_ctas(long long rows, int groups) {
  if (rows > 2LL * 8 * groups) return 0;
  int n = 1;
  while (n < 8 && (long long)n * groups < rows) n *= 2;
  return n;
}

template <int LANES, int NV, bool GATE, bool RES>
cudaError_t bwd_one(const NormBwdArgs& a, int grid, int cluster, cudaStream_t s) {
  constexpr int RING = RowRing<kBwdThreads, 2 + GATE + RES, NV>::BYTES;
  constexpr int SUMS = (LANES < kBwdThreads ? 32 * kBwdThreads : 0) + 64 * LANES * NV;
  constexpr int BYTES = RING > SUMS ? RING : SUMS;
  static hstu::DeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(norm_bwd_kernel<LANES, NV, GATE, RES>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  });
  if (e != cudaSuccess) return e;
  return hstu::launch_after_in_clusters(cluster, norm_bwd_kernel<LANES, NV, GATE, RES>, grid, kBwdThreads,
                                        BYTES, s, a);
}

template <int LANES, int NV>
cudaError_t bwd(NormBwdArgs a, bool res, float* dgamma, float* dbeta, int sms, cudaStream_t s) {
  const int cluster = cluster_ctas(a.rows, kBwdThreads / LANES);
  const int grid = cluster ? cluster : norm_grid(a.rows, kBwdThreads / LANES, 1, sms);
  float* own = nullptr;
  cudaError_t e = cudaSuccess;
  if (cluster) {
    a.dgamma = dgamma;
    a.dbeta = dbeta;
  } else if (!a.parts) {
    e = cudaMallocAsync(reinterpret_cast<void**>(&own), (size_t)grid * 2u * (size_t)a.width * sizeof(float), s);
    if (e != cudaSuccess) return e;
    a.parts = own;
  }
  e = a.u && res ? bwd_one<LANES, NV, true, true>(a, grid, cluster, s)
      : a.u      ? bwd_one<LANES, NV, true, false>(a, grid, cluster, s)
      : res      ? bwd_one<LANES, NV, false, true>(a, grid, cluster, s)
                 : bwd_one<LANES, NV, false, false>(a, grid, cluster, s);
  if (e == cudaSuccess && !cluster)
    e = hstu::launch_after(norm_sum_kernel, (2 * a.width + 31) / 32, kSumThreads, 0, s, (const float*)a.parts,
                           grid, a.width, dgamma, dbeta);
  if (own) {
    const cudaError_t f = cudaFreeAsync(own, s);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

// The lanes and vectors a lane for a row of 8 nvec channels.  Forward: a warp
// holds up to 1024 channels, so that no barrier is needed.  Backward: one
// vector a lane, for the registers of the row and of its two sums (the rows
// ahead lie in shared memory); above 4096 channels a CTA's 512 lanes take two.
#define HSTU_NORM_FWD_PICK(nvec, CALL) \
  ((nvec) <= 8      ? CALL(8, 1)       \
   : (nvec) <= 16   ? CALL(16, 1)      \
   : (nvec) <= 32   ? CALL(32, 1)      \
   : (nvec) <= 64   ? CALL(32, 2)      \
   : (nvec) <= 128  ? CALL(32, 4)      \
   : (nvec) <= 256  ? CALL(256, 1)     \
   : (nvec) <= 512  ? CALL(256, 2)     \
                    : CALL(256, 4))
#define HSTU_NORM_BWD_PICK(nvec, CALL) \
  ((nvec) <= 8      ? CALL(8, 1)       \
   : (nvec) <= 16   ? CALL(16, 1)      \
   : (nvec) <= 32   ? CALL(32, 1)      \
   : (nvec) <= 64   ? CALL(64, 1)      \
   : (nvec) <= 128  ? CALL(128, 1)     \
   : (nvec) <= 256  ? CALL(256, 1)     \
   : (nvec) <= 512  ? CALL(512, 1)     \
                    : CALL(512, 2))

bool bad_ptr(const void* p, unsigned align) {
  return !p || (reinterpret_cast<uintptr_t>(p) & (align - 1u));
}
bool bad_rows(const void* p, int64_t stride, int width) {
  return bad_ptr(p, 16) || stride < width || (stride & 7);
}

int check_norm(const float* gamma, const float* beta, float scale, float eps, int64_t rows, int width) {
  if (rows < 0 || width < 8 || width > HSTU_NORM_MAX_WIDTH || (width & 7)) return HSTU_ERR_INVALID_ARG;
  if (bad_ptr(gamma, 16) || bad_ptr(beta, 16)) return HSTU_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 3.0e38f) return HSTU_ERR_INVALID_ARG;
  if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

int status_of(cudaError_t e) {
  if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction)
    return HSTU_ERR_UNSUPPORTED;
  if (e == cudaErrorMemoryAllocation) return HSTU_ERR_NO_MEMORY;
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // namespace

extern "C" {

int hstu_norm_fwd(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                  float scale, const void* u, int64_t u_stride, const float* gamma, const float* beta,
                  float eps, int64_t rows, int width, void* y, void* z, hstu_stream_t stream) {
  int rc = check_norm(gamma, beta, scale, eps, rows, width);
  if (rc != HSTU_OK) return rc;
  if (!residual != !z) return HSTU_ERR_INVALID_ARG;
  if (rows == 0) return HSTU_OK;
  if (bad_rows(x, x_stride, width) || bad_ptr(y, 16)) return HSTU_ERR_INVALID_ARG;
  if (residual && (bad_rows(residual, residual_stride, width) || bad_ptr(z, 16)))
    return HSTU_ERR_INVALID_ARG;
  if (u && bad_rows(u, u_stride, width)) return HSTU_ERR_INVALID_ARG;
  int sms = 0;
  if ((rc = hstu::host_device_check(&sms)) != HSTU_OK) return rc;
  NormFwdArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.u = static_cast<const uint16_t*>(u);
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.u_stride = u_stride;
  a.gamma = gamma;
  a.beta = beta;
  a.scale = scale;
  a.eps = eps;
  a.rows = rows;
  a.width = width;
  a.y = static_cast<uint16_t*>(y);
  a.z = static_cast<uint16_t*>(z);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define HSTU_FWD(L, N) fwd<L, N>(a, sms, s)
  return status_of(HSTU_NORM_FWD_PICK(width / 8, HSTU_FWD));
#undef HSTU_FWD
}

int hstu_norm_bwd_workspace(int width, size_t* bytes) {
  if (!bytes || width < 8 || width > HSTU_NORM_MAX_WIDTH || (width & 7)) return HSTU_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = hstu::host_device_check(&sms);
  if (rc != HSTU_OK) return rc;
  *bytes = (size_t)sms * 2u * (size_t)width * sizeof(float);
  return HSTU_OK;
}

int hstu_norm_bwd(const void* dy, int64_t dy_stride, const void* z, int64_t z_stride, const void* u,
                  int64_t u_stride, const float* gamma, const float* beta, float eps,
                  const void* dz_in, int64_t dz_in_stride, float scale, int64_t rows, int width,
                  void* dz, void* dx, void* du, int64_t du_stride, float* dgamma, float* dbeta,
                  void* workspace, hstu_stream_t stream) {
  int rc = check_norm(gamma, beta, scale, eps, rows, width);
  if (rc != HSTU_OK) return rc;
  if (!u != !du || bad_ptr(dgamma, 4) || bad_ptr(dbeta, 4)) return HSTU_ERR_INVALID_ARG;
  if (workspace && bad_ptr(workspace, 16)) return HSTU_ERR_INVALID_ARG;
  if (rows > 0) {
    if (bad_rows(dy, dy_stride, width) || bad_rows(z, z_stride, width) || bad_ptr(dz, 16))
      return HSTU_ERR_INVALID_ARG;
    if (u && (bad_rows(u, u_stride, width) || bad_rows(du, du_stride, width)))
      return HSTU_ERR_INVALID_ARG;
    if (dz_in && bad_rows(dz_in, dz_in_stride, width)) return HSTU_ERR_INVALID_ARG;
    if (dx && bad_ptr(dx, 16)) return HSTU_ERR_INVALID_ARG;
  }
  int sms = 0;
  if ((rc = hstu::host_device_check(&sms)) != HSTU_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NormBwdArgs a{};
  a.dy = static_cast<const uint16_t*>(dy);
  a.z = static_cast<const uint16_t*>(z);
  a.u = static_cast<const uint16_t*>(u);
  a.dz_in = static_cast<const uint16_t*>(dz_in);
  a.dy_stride = dy_stride;
  a.z_stride = z_stride;
  a.u_stride = u_stride;
  a.dz_in_stride = dz_in_stride;
  a.du_stride = du_stride;
  a.gamma = gamma;
  a.beta = beta;
  a.scale = scale;
  a.eps = eps;
  a.rows = rows;
  a.width = width;
  a.dz = static_cast<uint16_t*>(dz);
  a.dx = static_cast<uint16_t*>(dx);
  a.du = static_cast<uint16_t*>(du);
  a.parts = static_cast<float*>(workspace);
#define HSTU_BWD(L, N) bwd<L, N>(a, dz_in || dx, dgamma, dbeta, sms, s)
  rc = status_of(HSTU_NORM_BWD_PICK(width / 8, HSTU_BWD));
#undef HSTU_BWD
  return rc;
}

}  // extern "C"
