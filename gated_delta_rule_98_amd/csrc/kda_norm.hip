// kda_norm.hip - the norms around a block (include/kda_norm.h):
//     r' = r + scale * sigmoid(g) * N(z) * w_post ;  y = N(r') * w_pre
// with N(x) = x / sqrt(mean(x^2) + eps) over a row of D channels.
//
// One pass: a workgroup holds a row in registers, so that r, z and g are read
// once and r' and y written once; the two mean squares are sums over the
// workgroup. HBM-bound with many rows, latency-bound with few.

#include <algorithm>

#include "kda_engine.h"
#include "kda_linear_impl.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

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

// Eight consecutive channels of a row as they lie in memory, in 128-bit
// accesses: gfx950 takes them at any address, so rows need only their element's
// alignment. A row's values are touched once: streamed.
constexpr int E = 8;
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

template <bool BF16>
struct Raw {
  static constexpr int W = BF16 ? 4 : 8;
  uint32_t w[W];

  __device__ __forceinline__ void load(const void *base, int64_t i) {
    const char *p = static_cast<const char *>(base) + i * (BF16 ? 2 : 4);
#pragma unroll
    for (int x = 0; x < W / 4; ++x) {
      const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p + 16 * x));
      w[4 * x] = u[0];
      w[4 * x + 1] = u[1];
      w[4 * x + 2] = u[2];
      w[4 * x + 3] = u[3];
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (!BF16) return __uint_as_float(w[e]);
    return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
};

__device__ __forceinline__ float load_one(const void *base, bool bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(base)[i]) : static_cast<const float *>(base)[i];
}

__device__ __forceinline__ void store_one(void *base, bool bf16, int64_t i, float x) {
  if (bf16)
    static_cast<uint16_t *>(base)[i] = f32_to_bf16(x);
  else
    static_cast<float *>(base)[i] = x;
}

__device__ __forceinline__ void store(void *base, bool bf16, int64_t i, const float (&x)[E]) {
  if (bf16) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x[2 * e], x[2 * e + 1]}, bf16x2));
    __builtin_nontemporal_store((u32x4){w[0], w[1], w[2], w[3]},
                                reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(base) + i));
  } else {
    v4f_any *p = reinterpret_cast<v4f_any *>(static_cast<float *>(base) + i);
    __builtin_nontemporal_store((v4f){x[0], x[1], x[2], x[3]}, p);
    __builtin_nontemporal_store((v4f){x[4], x[5], x[6], x[7]}, p + 1);
  }
}

__device__ __forceinline__ void load_weight(const float *p, float (&w)[E]) {
  const v4f x = reinterpret_cast<const v4f_any *>(p)[0], y = reinterpret_cast<const v4f_any *>(p)[1];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = x[e];
    w[4 + e] = y[e];
  }
}

__device__ __forceinline__ float gate_of(float g) { return 1.0f / (1.0f + expf(-g)); }

// The row in registers: NG groups of 8 channels per thread, group n of thread t
// at channel 8 (n NT + t); with TAIL the D % 8 last channels are one each of the
// first threads. A workgroup walks rows gridDim.x apart: the weights stay in
// registers, and the next row is requested before this one's sums (all loads of
// the first row go out together, so one latency covers them).
template <int NT, int NG, bool RB, bool TAIL>
__global__ __launch_bounds__(NT) void norm_kernel(NormArgs a) {
  __shared__ float part[2][2][NT / 64];
  struct Row {
    Raw<RB> r[NG];
    Raw<true> z[NG], g[NG];
    float rx, zx, gx;  // the channel of the tail
  } next;
  const auto channel = [](int n) { return (n * NT + (int)threadIdx.x) * E; };
  const int whole = a.D / E * E, cx = whole + (int)threadIdx.x;
  const bool tail = TAIL && cx < a.D;
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int c = channel(n);
      if (c < whole) {
        next.r[n].load(a.resid, row * a.rs + c);
        if (a.z) next.z[n].load(a.z, row * a.zs + c);
        if (a.gate) next.g[n].load(a.gate, row * a.gs + c);
      }
    }
    next.rx = next.zx = next.gx = 0.0f;
    if (tail) {
      next.rx = load_one(a.resid, RB, row * a.rs + cx);
      if (a.z) next.zx = load_one(a.z, true, row * a.zs + cx);
      if (a.gate) next.gx = load_one(a.gate, true, row * a.gs + cx);
    }
  };
  load(blockIdx.x);
  float wo[NG][E], wp[NG][E], wox = 1.0f, wpx = 1.0f;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const int c = channel(n);
#pragma unroll
    for (int e = 0; e < E; ++e) wo[n][e] = wp[n][e] = 1.0f;
    if (c < whole) {
      if (a.w_post) load_weight(a.w_post + c, wo[n]);
      if (a.w_pre) load_weight(a.w_pre + c, wp[n]);
    }
  }
  if (tail && a.w_post) wox = a.w_post[cx];
  if (tail && a.w_pre) wpx = a.w_pre[cx];
  const float inv_d = 1.0f / (float)a.D;
  int parity = 0;  // of the row: a buffer of sums is written again two barriers after it was read
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const Row cur = next;
    if (row + gridDim.x < a.rows) load(row + gridDim.x);
    float r[NG][E], rx = cur.rx;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int e = 0; e < E; ++e) r[n][e] = channel(n) < whole ? cur.r[n].at(e) : 0.0f;
    if (a.z) {
      float f = a.scale;
      if (a.w_post) {
        float ss = cur.zx * cur.zx;
#pragma unroll
        for (int n = 0; n < NG; ++n)
          if (channel(n) < whole)
#pragma unroll
            for (int e = 0; e < E; ++e) ss = __builtin_fmaf(cur.z[n].at(e), cur.z[n].at(e), ss);
        f *= 1.0f / sqrtf(block_sum<NT>(ss, part[parity][0]) * inv_d + a.eps);
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const int c = channel(n);
        if (c < whole) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float w = a.gate ? wo[n][e] * gate_of(cur.g[n].at(e)) : wo[n][e];
            r[n][e] = __builtin_fmaf(cur.z[n].at(e) * f, w, r[n][e]);
          }
          store(a.resid_out, RB, row * a.ros + c, r[n]);
        }
      }
      if (tail) {
        rx = __builtin_fmaf(cur.zx * f, a.gate ? wox * gate_of(cur.gx) : wox, rx);
        store_one(a.resid_out, RB, row * a.ros + cx, rx);
      }
    }
    if (a.y) {
      float ss = rx * rx;
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < E; ++e) ss = __builtin_fmaf(r[n][e], r[n][e], ss);
      const float f = 1.0f / sqrtf(block_sum<NT>(ss, part[parity][1]) * inv_d + a.eps);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const int c = channel(n);
        if (c < whole) {
          float y[E];
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = r[n][e] * f * wp[n][e];
          store(a.y, a.y_bf16, row * a.ys + c, y);
        }
      }
      if (tail) store_one(a.y, a.y_bf16, row * a.ys + cx, rx * f * wpx);
    }
  }
}

template <int NT, int NG>
const void *norm_of(bool rb, bool tail) {
  if (tail) return rb ? (const void *)norm_kernel<NT, NG, true, true> : (const void *)norm_kernel<NT, NG, false, true>;
  return rb ? (const void *)norm_kernel<NT, NG, true, false> : (const void *)norm_kernel<NT, NG, false, false>;
}

}  // namespace

// Measured on MI355X at D = 4096. Up to 512 rows (two per CU) latency counts and
// a row takes 512 threads: 64 rows with every part 4.5 us, 4.9 with 256. Past
// that a row takes 256 and a workgroup several rows, 4096 workgroups at most:
// 8000 rows with every part 59.7 us (5.5 TB/s), 60.4 with 512 threads, 69 with a
// row per workgroup, its weights read for every row and no streaming hints.
constexpr int kFewRows = 512, kMostBlocks = 4096;

NormLaunch norm_launch(int rows, int D, bool rb) {
  const int groups = D / E;
  const bool tail = D % E != 0;
  const auto of = [&](const void *fn, int threads, int cap) { return NormLaunch{fn, threads, std::min(rows, cap)}; };
  if (rows <= kFewRows) {
    if (groups <= 512) return of(norm_of<512, 1>(rb, tail), 512, rows);
  } else {
    if (groups <= 256) return of(norm_of<256, 1>(rb, tail), 256, kMostBlocks);
    if (groups <= 512) return of(norm_of<256, 2>(rb, tail), 256, kMostBlocks);
  }
  if (groups <= 1024) return of(norm_of<512, 2>(rb, tail), 512, kMostBlocks / 2);
  return of(norm_of<1024, 2>(rb, tail), 1024, kMostBlocks / 4);
}

}  // namespace kda
