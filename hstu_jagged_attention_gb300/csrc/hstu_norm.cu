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
// bits.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hstu_attn.h"
#include "hstu_internal.h"

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
};

struct V8 {
  float f[8];
};

__device__ __forceinline__ V8 unpack(const uint4& p) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.f[2 * i] = __uint_as_float(w[i] << 16);
    v.f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return v;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack(const V8& v) {
  return make_uint4(pack2(v.f[0], v.f[1]), pack2(v.f[2], v.f[3]), pack2(v.f[4], v.f[5]),
                    pack2(v.f[6], v.f[7]));
}

__device__ __forceinline__ uint4 ld_row(const uint16_t* p, long long at) {
  return __ldcs(reinterpret_cast<const uint4*>(p + at));
}

__device__ __forceinline__ V8 ld_f32(const float* p, int at) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + at));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + at) + 1);
  return V8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

constexpr int kThreads = 256;

// Sums v over the LANES lanes of the caller's group, for each of N values;
// LANES > 32: over the whole CTA, by way of `red` (2 N kThreads / 32 floats,
// its halves used in turn so that one barrier a sum is enough).
template <int LANES, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int* turn) {
#pragma unroll
  for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (LANES > 32) {
    constexpr int W = LANES / 32;
    float* mine = red + (*turn ? N * W : 0);
    *turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) mine[i * W + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += mine[i * W + w];
      v[i] = s;
    }
  }
}

template <int LANES, int NV, bool GATE, bool RES>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float red[2 * 2 * (kThreads / 32)];
  int turn = 0;
  const int lane = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  constexpr int GROUPS = kThreads / LANES;
  const float inv_w = 1.f / (float)a.width;
  // every lane of a warp stays in the loop (its shuffles need them), with
  // its loads and stores off past the last row
  const long long step = (long long)gridDim.x * GROUPS;
  for (long long r0 = (long long)blockIdx.x * GROUPS; r0 < a.rows; r0 += step) {
    const long long r = r0 + group;
    const bool live = r < a.rows;
    V8 z[NV];
    uint4 up[NV];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      const bool in = live && c < a.width;
      uint4 xp = make_uint4(0, 0, 0, 0), rp = xp;
      if (in) {
        xp = ld_row(a.x, r * a.x_stride + c);
        if (RES) rp = ld_row(a.residual, r * a.residual_stride + c);
        if (GATE) up[i] = ld_row(a.u, r * a.u_stride + c);
      }
      z[i] = unpack(xp);
      if (RES) {
        const V8 rv = unpack(rp);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i].f[j] = fmaf(a.scale, z[i].f[j], rv.f[j]);
        if (in) *reinterpret_cast<uint4*>(a.z + r * a.width + c) = pack(z[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += z[i].f[j];
    }
    group_sum<LANES, 1>(s, red, &turn);
    const float mean = s[0] * inv_w;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = 8 * (lane + i * LANES) < a.width;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[i].f[j] -= mean;
        if (in) q[0] = fmaf(z[i].f[j], z[i].f[j], q[0]);
      }
    }
    group_sum<LANES, 1>(q, red, &turn);
    const float rstd = rsqrtf(fmaf(q[0], inv_w, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      if (!live || c >= a.width) continue;
      const V8 g = ld_f32(a.gamma, c), b = ld_f32(a.beta, c);
      V8 y;
#pragma unroll
      for (int j = 0; j < 8; ++j) y.f[j] = fmaf(z[i].f[j] * rstd, g.f[j], b.f[j]);
      if (GATE) {
        const V8 u = unpack(up[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) y.f[j] *= u.f[j];
      }
      *reinterpret_cast<uint4*>(a.y + r * a.width + c) = pack(y);
    }
  }
}

template <int LANES, int NV, bool GATE, bool RES>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float red[2 * 2 * (kThreads / 32)];
  int turn = 0;
  const int lane = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  constexpr int GROUPS = kThreads / LANES;
  const float inv_w = 1.f / (float)a.width;
  float dg[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.f;
  const long long step = (long long)gridDim.x * GROUPS;
  for (long long r0 = (long long)blockIdx.x * GROUPS; r0 < a.rows; r0 += step) {
    const long long r = r0 + group;
    const bool live = r < a.rows;
    uint4 zp[NV], dyp[NV], up[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      zp[i] = dyp[i] = up[i] = make_uint4(0, 0, 0, 0);
      if (live && c < a.width) {
        zp[i] = ld_row(a.z, r * a.z_stride + c);
        dyp[i] = ld_row(a.dy, r * a.dy_stride + c);
        if (GATE) up[i] = ld_row(a.u, r * a.u_stride + c);
      }
    }
    // first the sums that need no statistics, then those about the mean
    V8 z[NV], g[NV];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      z[i] = unpack(zp[i]);
      g[i] = unpack(dyp[i]);
      if (GATE) {
        const V8 u = unpack(up[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i].f[j] *= u.f[j];
      }
      if (c < a.width) {
        const V8 gm = ld_f32(a.gamma, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[0] += z[i].f[j];
          s[1] = fmaf(g[i].f[j], gm.f[j], s[1]);
        }
      }
    }
    group_sum<LANES, 2>(s, red, &turn);
    const float mean = s[0] * inv_w, mean_a = s[1] * inv_w;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      if (c < a.width) {
        const V8 gm = ld_f32(a.gamma, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          z[i].f[j] -= mean;
          q[0] = fmaf(z[i].f[j], z[i].f[j], q[0]);
          q[1] = fmaf(z[i].f[j], g[i].f[j] * gm.f[j], q[1]);
        }
      }
    }
    group_sum<LANES, 2>(q, red, &turn);
    const float rstd = rsqrtf(fmaf(q[0], inv_w, a.eps));
    const float mean_ax = q[1] * inv_w * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (lane + i * LANES);
      if (!live || c >= a.width) continue;
      const V8 gm = ld_f32(a.gamma, c);
      V8 dz;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = z[i].f[j] * rstd;
        dg[i][j] = fmaf(g[i].f[j], h, dg[i][j]);
        db[i][j] += g[i].f[j];
        dz.f[j] = rstd * (fmaf(g[i].f[j], gm.f[j], -mean_a) - h * mean_ax);
      }
      if (GATE) {
        const V8 bt = ld_f32(a.beta, c), dy = unpack(dyp[i]);
        V8 du;
#pragma unroll
        for (int j = 0; j < 8; ++j) du.f[j] = dy.f[j] * fmaf(z[i].f[j] * rstd, gm.f[j], bt.f[j]);
        *reinterpret_cast<uint4*>(a.du + r * a.du_stride + c) = pack(du);
      }
      if (RES && a.dz_in) {
        const V8 in = unpack(ld_row(a.dz_in, r * a.dz_in_stride + c));
#pragma unroll
        for (int j = 0; j < 8; ++j) dz.f[j] += in.f[j];
      }
      *reinterpret_cast<uint4*>(a.dz + r * a.width + c) = pack(dz);
      if (RES && a.dx) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dz.f[j] *= a.scale;
        *reinterpret_cast<uint4*>(a.dx + r * a.width + c) = pack(dz);
      }
    }
  }
  // the CTA's sums: the groups' in order (GROUPS > 1: through shared memory)
  float* out = a.parts + (long long)blockIdx.x * 2 * a.width;
  __shared__ float acc[GROUPS > 1 ? 16 * kThreads : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (lane + i * LANES);
    if constexpr (GROUPS == 1) {
      if (c < a.width)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          out[c + j] = dg[i][j];
          out[a.width + c + j] = db[i][j];
        }
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[(2 * j) * kThreads + threadIdx.x] = dg[i][j];
        acc[(2 * j + 1) * kThreads + threadIdx.x] = db[i][j];
      }
      __syncthreads();
      for (int k = threadIdx.x; k < 16 * LANES; k += kThreads) {
        const int l = k % LANES, jj = k / LANES;
        const int cc = 8 * (l + i * LANES) + (jj >> 1);
        if (cc >= a.width) continue;
        float s = 0.f;
        for (int gidx = 0; gidx < GROUPS; ++gidx) s += acc[jj * kThreads + gidx * LANES + l];
        out[(jj & 1) * a.width + cc] = s;
      }
    }
  }
}

// dgamma and dbeta: the CTAs' sums in a fixed order.  A block takes 32 of the
// 2 width columns; its 8 warps take the CTAs in turn.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float* parts, int n, int width,
                                                       float* dgamma, float* dbeta) {
  __shared__ float acc[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = 32 * blockIdx.x + lane;
  float s = 0.f;
  if (col < 2 * width)
    for (int i = warp; i < n; i += 8) s += parts[(long long)i * 2 * width + col];
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < 2 * width) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += acc[w][lane];
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
constexpr int kFwdPerSm = 8, kBwdPerSm = 3;

template <int LANES, int NV>
cudaError_t fwd(const NormFwdArgs& a, int sms, cudaStream_t s) {
  const int grid = norm_grid(a.rows, kThreads / LANES, kFwdPerSm, sms);
  if (a.u && a.residual)
    norm_fwd_kernel<LANES, NV, true, true><<<grid, kThreads, 0, s>>>(a);
  else if (a.u)
    norm_fwd_kernel<LANES, NV, true, false><<<grid, kThreads, 0, s>>>(a);
  else if (a.residual)
    norm_fwd_kernel<LANES, NV, false, true><<<grid, kThreads, 0, s>>>(a);
  else
    norm_fwd_kernel<LANES, NV, false, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int LANES, int NV>
cudaError_t bwd(const NormBwdArgs& a, bool res, float* dgamma, float* dbeta, int sms, cudaStream_t s) {
  const int grid = norm_grid(a.rows, kThreads / LANES, kBwdPerSm, sms);
  if (a.u && res)
    norm_bwd_kernel<LANES, NV, true, true><<<grid, kThreads, 0, s>>>(a);
  else if (a.u)
    norm_bwd_kernel<LANES, NV, true, false><<<grid, kThreads, 0, s>>>(a);
  else if (res)
    norm_bwd_kernel<LANES, NV, false, true><<<grid, kThreads, 0, s>>>(a);
  else
    norm_bwd_kernel<LANES, NV, false, false><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_sum_kernel<<<(2 * a.width + 31) / 32, 256, 0, s>>>(a.parts, grid, a.width, dgamma, dbeta);
  return cudaGetLastError();
}

// The narrowest group of lanes that holds a row of 8 nvec channels.
#define HSTU_NORM_PICK(nvec, CALL)        \
  ((nvec) <= 8      ? CALL(8, 1)          \
   : (nvec) <= 32   ? CALL(32, 1)         \
   : (nvec) <= 64   ? CALL(32, 2)         \
   : (nvec) <= 128  ? CALL(32, 4)         \
   : (nvec) <= 256  ? CALL(256, 1)        \
   : (nvec) <= 512  ? CALL(256, 2)        \
                    : CALL(256, 4))

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
  return status_of(HSTU_NORM_PICK(width / 8, HSTU_FWD));
#undef HSTU_FWD
}

int hstu_norm_bwd_workspace(int width, size_t* bytes) {
  if (!bytes || width < 8 || width > HSTU_NORM_MAX_WIDTH || (width & 7)) return HSTU_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = hstu::host_device_check(&sms);
  if (rc != HSTU_OK) return rc;
  *bytes = (size_t)kBwdPerSm * (size_t)sms * 2u * (size_t)width * sizeof(float);
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
  float* own = nullptr;
  if (!workspace) {
    const size_t bytes = (size_t)kBwdPerSm * (size_t)sms * 2u * (size_t)width * sizeof(float);
    const cudaError_t e = cudaMallocAsync(reinterpret_cast<void**>(&own), bytes, s);
    if (e != cudaSuccess) return e == cudaErrorMemoryAllocation ? HSTU_ERR_NO_MEMORY : HSTU_ERR_CUDA;
    a.parts = own;
  }
#define HSTU_BWD(L, N) bwd<L, N>(a, dz_in || dx, dgamma, dbeta, sms, s)
  rc = status_of(HSTU_NORM_PICK(width / 8, HSTU_BWD));
#undef HSTU_BWD
  if (own && cudaFreeAsync(own, s) != cudaSuccess && rc == HSTU_OK) rc = HSTU_ERR_CUDA;
  return rc;
}

}  // extern "C"
