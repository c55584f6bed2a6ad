// kda_linear.hip - linear attention with a decay per head (include/kda_linear.h):
//     S <- a S + k v^T ;  o = S^T q .

#include "kda_engine.h"
#include "kda_linear_impl.h"

namespace kda {
namespace {

__device__ __forceinline__ void lin_put(const LinArgs &a, bool bf16, int64_t idx, float y) {
  if (bf16)
    static_cast<uint16_t *>(a.out)[idx] = f32_to_bf16(y);
  else
    static_cast<float *>(a.out)[idx] = y;
}

// One token on C columns of 16 lanes each (the column engine's layout).
template <int NV, int C>
__device__ __forceinline__ void lin_token(float4 (&s)[C][NV], const float4 (&k)[NV], const float4 (&q)[NV],
                                          const float (&vj)[C], float al, float (&o)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      s[c][e].x = __builtin_fmaf(k[e].x, vj[c], s[c][e].x * al);
      s[c][e].y = __builtin_fmaf(k[e].y, vj[c], s[c][e].y * al);
      s[c][e].z = __builtin_fmaf(k[e].z, vj[c], s[c][e].z * al);
      s[c][e].w = __builtin_fmaf(k[e].w, vj[c], s[c][e].w * al);
    }
    o[c] = lane_dot<NV>(s[c], q);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = row16_sum(o[c]);
}

// Single-token step, in place: one workgroup per (row, head, W value columns).
template <int DK, int C, bool GATE, bool BF16>
__global__ __launch_bounds__(GATE ? 1024 : 256) void lin_decode_kernel(LinArgs a) {
  constexpr int NV = DK / 64;
  const Unit u = unit_of_block(a.ntile, a.H);
  const Lane L = lane_geometry();
  const int W = C * L.slab;
  const int64_t obase = ((int64_t)u.b * a.H + u.h) * a.dv + (int64_t)u.tile * W;
  const uint16_t *kp = a.k + u.b * a.ks + (int64_t)(u.h / a.group) * DK + 4 * L.r;
  const uint16_t *qp = a.q + u.b * a.qs + (int64_t)(u.h / a.group) * DK + 4 * L.r;
  const uint16_t *vp = a.v + u.b * a.vs + (int64_t)u.h * a.dv + (int64_t)u.tile * W;
  float4 kk[NV], qq[NV];
  float vj[C];
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    kk[e] = unpack_bf16x4(*reinterpret_cast<const uint2 *>(kp + 64 * e));
    qq[e] = unpack_bf16x4(*reinterpret_cast<const uint2 *>(qp + 64 * e));
  }
#pragma unroll
  for (int c = 0; c < C; ++c) vj[c] = bf16_to_f32(vp[L.col0 + c * L.slab]);
  const float al = a.alpha[u.b * a.as + u.h];
  const int32_t slot = a.slot_ids[u.b];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    report(a.dev_err, u, KDA_DEVERR_SLOT);
    return;
  }
  float *S = a.cache + (int64_t)slot * a.slot_stride + ((int64_t)u.h * a.dv + (int64_t)u.tile * W) * DK;
  float4 s[C][NV];
  load_tile<DK, C, kDecodeLoadStream>(s, S, L);
  float gj = 0.0f, wj = 1.0f;
  if constexpr (GATE) {
    const int j = L.col0 + (L.r < C ? L.r : 0) * L.slab;
    gj = bf16_to_f32(a.gate[obase + j]);
    if (a.weight) wj = a.weight[j];
  }
  float o[C];
  lin_token<NV, C>(s, kk, qq, vj, al, o);
  store_tile<DK, C, kDecodeStoreStream>(S, s, L);
  if constexpr (GATE) {
    // the workgroup spans all dv columns: the head's mean square from the waves' partials
    __shared__ float part[kMaxWaves];
    __shared__ float raw[kMaxDv];
    store_cols<C>(raw, L, o);
    gate_partial<C>(o, part);
    __syncthreads();
    if (L.r < C) {
      const int j = L.col0 + L.r * L.slab;
      float tot = part[0];
      for (int i = 1; i < (int)(blockDim.x >> 6); ++i) tot += part[i];
      const float inv_rms = 1.0f / sqrtf(tot / (float)a.dv + a.eps);
      lin_put(a, BF16, obase + j, raw[j] * inv_rms * wj * (1.0f / (1.0f + expf(-gj))));
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (L.r == c) lin_put(a, BF16, obase + L.col0 + c * L.slab, o[c]);
  }
}

// Prompts, token by token: one workgroup per (row, head, 16 value columns).
template <int DK>
__global__ __launch_bounds__(256) void lin_prefill_kernel(LinArgs a) {
  constexpr int NV = DK / 64;
  const Unit u = unit_of_block_rows(a.ntile, a.H, a.B);
  const Lane L = lane_geometry();
  const int32_t slot = a.slot_ids[u.b], c0 = a.cu[u.b], c1 = a.cu[u.b + 1];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    report(a.dev_err, u, KDA_DEVERR_SLOT);
    return;
  }
  if (c0 < 0 || c1 < c0 || c1 > a.n_tok) {
    report(a.dev_err, u, KDA_DEVERR_SEQLEN);
    return;
  }
  const int ck = a.ckpt_pos ? a.ckpt_pos[u.b] : -1;
  if (ck > c1 - c0) {
    report(a.dev_err, u, KDA_DEVERR_CKPT);
    return;
  }
  const int64_t col = (int64_t)u.h * a.dv + u.tile * 16;
  float *S = a.cache + (int64_t)slot * a.slot_stride + col * DK;
  float *CK = ck >= 0 ? a.ckpt + ((int64_t)u.b * a.H * a.dv + col) * DK : nullptr;
  float4 s[1][NV];
  load_tile<DK, 1, false>(s, S, L);
  if (ck == 0) store_tile<DK, 1, false>(CK, s, L);
  for (int t = c0; t < c1; ++t) {
    float4 kk[NV], qq[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      const int64_t i = (int64_t)(u.h / a.group) * DK + 4 * L.r + 64 * e;
      kk[e] = unpack_bf16x4(*reinterpret_cast<const uint2 *>(a.k + t * a.ks + i));
      qq[e] = unpack_bf16x4(*reinterpret_cast<const uint2 *>(a.q + t * a.qs + i));
    }
    const float vj[1] = {bf16_to_f32(a.v[t * a.vs + col + L.col0])};
    const float al = a.alpha[t * a.as + u.h];
    float o[1];
    lin_token<NV, 1>(s, kk, qq, vj, al, o);
    if (L.r == 0) lin_put(a, a.out_bf16, (int64_t)t * a.H * a.dv + col + L.col0, o[0]);
    if (t + 1 - c0 == ck) store_tile<DK, 1, false>(CK, s, L);
  }
  store_tile<DK, 1, false>(S, s, L);
}

}  // namespace

template <int DK, int C, bool GATE>
const void *lin_decode_io(bool bf16) {
  return bf16 ? (const void *)lin_decode_kernel<DK, C, GATE, true> : (const void *)lin_decode_kernel<DK, C, GATE, false>;
}

template <int DK>
const void *lin_decode_for(int C, bool gate, bool bf16) {
  if (gate) return C == kGateSlabsDecode ? lin_decode_io<DK, kGateSlabsDecode, true>(bf16) : nullptr;
  switch (C) {
    case 1: return lin_decode_io<DK, 1, false>(bf16);
    case 2: return lin_decode_io<DK, 2, false>(bf16);
    case 4: return lin_decode_io<DK, 4, false>(bf16);
    case 8: return lin_decode_io<DK, 8, false>(bf16);
  }
  return nullptr;
}

const void *lin_decode_kernel_for(int dk, int C, bool gate, bool bf16) {
  return dk == 64 ? lin_decode_for<64>(C, gate, bf16) : dk == 128 ? lin_decode_for<128>(C, gate, bf16) : nullptr;
}

const void *lin_prefill_kernel_for(int dk) {
  return dk == 64 ? (const void *)lin_prefill_kernel<64> : (const void *)lin_prefill_kernel<128>;
}

}  // namespace kda
