// kda_norm.hip - the norms around a block (include/kda_norm.h):
//     r' = r + scale * sigmoid(g) * N(z) * w_post ;  y = N(r') * w_pre
// with N(x) = x / sqrt(mean(x^2) + eps) over a row of D channels.

#include "kda_engine.h"
#include "kda_linear_impl.h"

namespace kda {
namespace {

__device__ __forceinline__ float wave_sum(float x) {
  x = row16_sum(x);
  return (readlane_f32(x, 0) + readlane_f32(x, 16)) + (readlane_f32(x, 32) + readlane_f32(x, 48));
}

// Sum over the workgroup, the same bits in every thread.
template <int NT>
__device__ __forceinline__ float block_sum(float x, float *part) {
  x = wave_sum(x);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) x += part[w];
  }
  return x;
}

// One workgroup per row, the row in registers: NG groups of E channels per
// thread, group n of thread t at channel (n NT + t) E; E = 8 with 128-bit
// accesses, E = 1 without.
template <int E>
__device__ __forceinline__ void ld_bf16(const uint16_t *p, float (&x)[E]) {
  if constexpr (E == 8) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const float4 a = unpack_bf16x4(make_uint2(u.x, u.y)), b = unpack_bf16x4(make_uint2(u.z, u.w));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    x[0] = bf16_to_f32(*p);
  }
}

template <int E>
__device__ __forceinline__ void ld_f32(const float *p, float (&x)[E]) {
  if constexpr (E == 8) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    x[0] = *p;
  }
}

template <int E>
__device__ __forceinline__ void st_any(void *base, bool bf16, int64_t i, const float (&x)[E]) {
  if (bf16) {
    uint16_t *p = static_cast<uint16_t *>(base) + i;
    if constexpr (E == 8) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f32_to_bf16(x[2 * e]) | (uint32_t)f32_to_bf16(x[2 * e + 1]) << 16;
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *p = f32_to_bf16(x[0]);
    }
  } else {
    float *p = static_cast<float *>(base) + i;
    if constexpr (E == 8) {
      reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *p = x[0];
    }
  }
}

template <int NT, int NG, int E>
__global__ __launch_bounds__(NT) void norm_kernel(NormArgs a) {
  __shared__ float part[2][NT / 64];
  const int64_t row = blockIdx.x;
  float r[NG][E], z[NG][E];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const int c = (n * NT + (int)threadIdx.x) * E;
#pragma unroll
    for (int e = 0; e < E; ++e) r[n][e] = z[n][e] = 0.0f;
    if (c < a.D) {
      if (a.resid_bf16)
        ld_bf16<E>(static_cast<const uint16_t *>(a.resid) + row * a.rs + c, r[n]);
      else
        ld_f32<E>(static_cast<const float *>(a.resid) + row * a.rs + c, r[n]);
      if (a.z) ld_bf16<E>(a.z + row * a.zs + c, z[n]);
    }
  }
  const float inv_d = 1.0f / (float)a.D;
  if (a.z) {
    float f = a.scale;
    if (a.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < E; ++e) ss = __builtin_fmaf(z[n][e], z[n][e], ss);
      f *= 1.0f / sqrtf(block_sum<NT>(ss, part[0]) * inv_d + a.eps);
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int c = (n * NT + (int)threadIdx.x) * E;
      if (c < a.D) {
        float w[E], g[E];
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = 1.0f;
        if (a.w_post) ld_f32<E>(a.w_post + c, w);
        if (a.gate) {
          ld_bf16<E>(a.gate + row * a.gs + c, g);
#pragma unroll
          for (int e = 0; e < E; ++e) w[e] *= 1.0f / (1.0f + expf(-g[e]));
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[n][e] = __builtin_fmaf(z[n][e] * f, w[e], r[n][e]);
        st_any<E>(a.resid_out, a.resid_bf16, row * a.ros + c, r[n]);
      }
    }
  }
  if (a.y) {
    float ss = 0.0f;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < E; ++e) ss = __builtin_fmaf(r[n][e], r[n][e], ss);
    const float f = 1.0f / sqrtf(block_sum<NT>(ss, part[1]) * inv_d + a.eps);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int c = (n * NT + (int)threadIdx.x) * E;
      if (c < a.D) {
        float w[E];
        ld_f32<E>(a.w_pre + c, w);
#pragma unroll
        for (int e = 0; e < E; ++e) r[n][e] = r[n][e] * f * w[e];
        st_any<E>(a.y, a.y_bf16, row * a.ys + c, r[n]);
      }
    }
  }
}

}  // namespace

const void *norm_kernel_for(int D, bool vec, int *threads) {
  *threads = 512;
  if (vec) {
    if (D <= 512 * 8) return (const void *)norm_kernel<512, 1, 8>;
    if (D <= 512 * 16) return (const void *)norm_kernel<512, 2, 8>;
    return (const void *)norm_kernel<512, 4, 8>;
  }
  if (D <= 512 * 8) return (const void *)norm_kernel<512, 8, 1>;
  return (const void *)norm_kernel<512, 32, 1>;
}

}  // namespace kda
