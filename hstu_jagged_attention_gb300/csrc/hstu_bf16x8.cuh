// Eight bf16 channels as a 16-byte vector, and as floats.
#pragma once

#include "hstu_ptx.cuh"

namespace hstu {
namespace {

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

}  // namespace
}  // namespace hstu
