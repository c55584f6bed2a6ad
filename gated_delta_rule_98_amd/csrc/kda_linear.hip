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

// Single-token step, in place: one workgroup per (row, head, W value columns),
// the state's 8 bytes per element against 5 operations: HBM-bound with many rows,
// latency-bound with few. The layout, the widths and their rule are those of
// kda_decode_step (choose_width); other widths than the rule's were within 3% at
// best. Measured on MI355X, 32 heads of 128 x 128: 64 rows 45.1 us, 6.0 TB/s (a
// plain in-place read-modify-write of the same bytes 41.3), one row 3.4.
template <int DK, int C, bool GATE, bool BF16>
__global__ __launch_bounds__(256) void lin_decode_kernel(LinArgs a) {
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

// ----------------------------------------------------------------------------
// Prompts in chunk form
// ----------------------------------------------------------------------------
//
// A row is cut into chunks of 64 tokens. With S0 the state entering a chunk,
// Gamma_t the product of its decays up to and including token t and D(t, s) the
// product of those after s up to t, the recurrence unrolls to
//     o_t = Gamma_t S0^T q_t + sum_{s <= t} D(t, s) (k_s . q_t) v_s
//     S_L = Gamma_L S0 + sum_s D(L, s) k_s v_s^T
// The decay is a scalar, so it scales scores and tokens and no triangular
// system has to be solved: the sum in S_L does not depend on S0. Long rows are
// therefore cut into segments of whole chunks that run in parallel: one kernel
// takes every segment's state sum (from a zero state), a second chains them to
// the state that enters each segment, and a third runs each segment from that
// state and writes the outputs. Rows of one segment need the third kernel only.
//
// Products on the bfloat16 matrix cores at fp32 accuracy. q, k and v are exact
// in bfloat16. The other operand of a product (the state, the decayed scores,
// the tokens scaled to the chunk's end) is fp32 and is split by truncation into
// three bfloat16 parts, 8 + 8 + 8 bits of its 24, which is exact; the three
// products are exact in fp32 and accumulate there. A bfloat16 output is the fp32
// one rounded once, so it takes all three parts too. (Two, 2^-18 of each term,
// moved one output in 400 to a neighbouring bfloat16; 16 ragged rows 98 us, 107 with
// three, 2 rows of 16384 x 64 x 64 211 and 223, 37 tokens the same.)
//
// A checkpoint cuts its row's chunks: the one that reaches it ends there, so
// the state there falls on a chunk's edge.
//
// Decay products never divide and never go through logarithms: a block of 16
// tokens holds prefix products, suffix products and its own product, and D(t, s)
// across blocks is prefix * (blocks between) * suffix. A product underflows
// only where the true value does, and 0 or a negative decay is like any other.
// Gamma and the decay to the chunk's end carry across chunks, so they are
// formed in 64 bits and rounded once.

constexpr int kLB = 16;                // block: the MFMA tile
// Decayed scores in LDS, [t][s] with s up to the end of t's half of the chunk:
// rows of 32 and of 64, padded by 8 against bank conflicts.
constexpr int kScoreElems = 32 * (32 + 8) + 32 * (64 + 8);
__device__ __forceinline__ int score_row(int tt, int m) {  // element of row 16 tt + m
  return tt < 2 ? (kLB * tt + m) * 40 : 32 * 40 + (kLB * (tt - 2) + m) * 72;
}

constexpr int kParts = 3;  // bfloat16 parts of an fp32 operand

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// (x0, x1) - (the word's two bfloat16), exact where they are the parts of x0 and
// x1 below: one dot-product instruction each. The factors (-1, 0) and (0, -1) are
// kept in registers: as a constant the compiler encodes (-1, 0) as the inline
// operand -1.0, which the instruction reads as the 32-bit -1.0, that is (0, -1).
__device__ __forceinline__ void minus_pair(uint32_t w, float &x0, float &x1) {
  uint32_t first = 0x0000bf80u, second = 0xbf800000u;
  asm("" : "+s"(first), "+s"(second));
  const bf16x2 h = __builtin_bit_cast(bf16x2, w);
  x0 = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, first), x0, false);
  x1 = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, second), x1, false);
}

// One word of two bfloat16: the upper halves of x0 (low) and x1 (high).
__device__ __forceinline__ uint32_t upper_pair(float x0, float x1) {
  return __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u);
}

// The bfloat16 parts of x, largest first, part i in words [i N/2, (i + 1) N/2):
// by truncation, 8 bits of the 24 each.
template <int N>
__device__ __forceinline__ void split_words(const float (&x)[N], uint32_t (&w)[kParts * N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float x0 = x[2 * i], x1 = x[2 * i + 1];
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      uint32_t &h = w[part * N / 2 + i];
      h = upper_pair(x0, x1);
      if (part + 1 < kParts) minus_pair(h, x0, x1);
    }
  }
}

struct Split {
  bf16x8 part[kParts];
};
__device__ __forceinline__ Split split(const float (&x)[8]) {
  uint32_t w[kParts * 4];
  split_words<8>(x, w);
  Split r;
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    r.part[i] = __builtin_bit_cast(bf16x8, (u32x4){w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]});
  return r;
}

__device__ __forceinline__ v4f mma(bf16x8 a, bf16x8 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// x, computed anew wherever this stands: keeps the compiler from hoisting
// 64-bit vector addresses out of the chunk loop (their registers would be
// spilled, and a reload waits for every load in flight) in place of a scalar
// base with a 32-bit offset.
__device__ __forceinline__ uint32_t pinned(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// An MFMA operand whose contraction index runs over tokens, from a token-major
// LDS array: lane (m, g) gets column m of its 16 at tokens 8 g .. 8 g + 7. Each
// 16-lane group reads 4 tokens x 16 columns (lane i the 4 columns 4 (i % 4) of
// token i / 4) and the transposing read hands lane i column i of the 4 tokens.
template <int PITCH>
__device__ __forceinline__ bf16x8 ld_tokens(const uint16_t *base, int tok0, int col0) {
  typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
  const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const uint16_t *p = base + (tok0 + 8 * g + (i >> 2)) * PITCH + col0 + 4 * (i & 3);
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * PITCH));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The same at tokens 4 g .. + 3 and 16 + 4 g .. + 3, where two accumulator tiles
// whose rows are tokens have theirs.
template <int PITCH>
__device__ __forceinline__ bf16x8 ld_tokens2(const uint16_t *base, int tok0, int col0) {
  typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
  const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const uint16_t *p = base + (tok0 + 4 * g + (i >> 2)) * PITCH + col0 + 4 * (i & 3);
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * PITCH));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}

// 8 channels of one token: contiguous, or the two runs of 4 at which the lane's
// accumulator registers of two 16-channel tiles stand.
__device__ __forceinline__ bf16x8 ld_run8(const uint16_t *p) {
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ bf16x8 ld_run4x2(const uint16_t *p) {
  const u32x2 a = *reinterpret_cast<const u32x2 *>(p), b = *reinterpret_cast<const u32x2 *>(p + 16);
  return __builtin_bit_cast(bf16x8, (u32x4){a.x, a.y, b.x, b.y});
}

// x moved over DPP control CTRL inside 16-lane rows, 1 where no lane is the source
template <int CTRL>
__device__ __forceinline__ float dpp_or_one(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0x3f800000, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp_or_one(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0x3ff00000, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive prefix and suffix products over a 16-lane row.
template <class T>
__device__ __forceinline__ T row_prefix(T x) {
  x = x * dpp_or_one<0x111>(x);
  x = x * dpp_or_one<0x112>(x);
  x = x * dpp_or_one<0x114>(x);
  return x * dpp_or_one<0x118>(x);
}
template <class T>
__device__ __forceinline__ T row_suffix(T x) {
  x = x * dpp_or_one<0x101>(x);
  x = x * dpp_or_one<0x102>(x);
  x = x * dpp_or_one<0x104>(x);
  return x * dpp_or_one<0x108>(x);
}

__device__ __forceinline__ double readlane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The decays of one chunk, by token.
struct ChunkDecay {
  float al[kLinChunk];   // the decay itself (1 past the chunk's end)
  float suf[kLinChunk];  // product over the token's block after it
  float gam[kLinChunk];  // Gamma: product over the chunk up to and including it
  float end[kLinChunk];  // product over the chunk after it
};

// One wave, lane = token.
__device__ __forceinline__ void put_chunk_decay(ChunkDecay &d, float al) {
  const int lane = threadIdx.x & 63, row = lane >> 4;
  const double p = row_prefix((double)al), s = row_suffix((double)al);
  const double after = dpp_or_one<0x101>(s);  // the suffix of the next lane
  const double m0 = readlane_f64(p, 15), m1 = readlane_f64(p, 31), m2 = readlane_f64(p, 47), m3 = readlane_f64(p, 63);
  const double pre = row == 0 ? 1.0 : row == 1 ? m0 : row == 2 ? m0 * m1 : m0 * m1 * m2;
  const double post = row == 0 ? m1 * m2 * m3 : row == 1 ? m2 * m3 : row == 2 ? m3 : 1.0;
  d.al[lane] = al;
  d.suf[lane] = (float)after;
  d.gam[lane] = (float)(p * pre);
  d.end[lane] = (float)(after * post);
}

// One row's tokens and segments. The segments but a row's last are full and
// numbered over all rows (full0 stand before this row's), a.more of them at most
// in a table whose rows do not overlap; a row past that is skipped and reported
// as a bad range. A row of two or more segments has a state slot for each.
struct LinRow {
  int b, full0, slot0, nseg, n;
  int32_t c0, slot;
  int err;  // 0, a device error, or -1 for a padding row
};

__device__ __forceinline__ int lin_row_check(const LinArgs &a, int b, int32_t &slot, int32_t &c0, int &n) {
  slot = a.slot_ids[b];
  c0 = a.cu[b];
  const int32_t c1 = a.cu[b + 1];
  n = 0;
  if (slot < 0) return -1;
  if (slot >= a.num_slots) return KDA_DEVERR_SLOT;
  if (c0 < 0 || c1 < c0 || c1 > a.n_tok) return KDA_DEVERR_SEQLEN;
  if (a.ckpt_pos && a.ckpt_pos[b] > c1 - c0) return KDA_DEVERR_CKPT;
  n = c1 - c0;
  return 0;
}

__device__ __forceinline__ int lin_segments(const LinArgs &a, int n) {
  return n > 0 ? (n - 1) / kLinChunk / a.seg + 1 : 1;
}

// Inclusive prefix sum over the wave: inside 16-lane rows, then the last lane
// of each row (row_bcast:15) and of each half (row_bcast:31) to the rows after it.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_prefix_sum(int x) {
  x = dpp_add<0x111, 0xF>(x);
  x = dpp_add<0x112, 0xF>(x);
  x = dpp_add<0x114, 0xF>(x);
  x = dpp_add<0x118, 0xF>(x);
  x = dpp_add<0x142, 0xA>(x);
  return dpp_add<0x143, 0xC>(x);
}

// Row `key`, or the row that holds full segment `key`, by a search over 64 rows
// at a time that every wave does for itself; false where there is none.
__device__ __forceinline__ bool lin_search(const LinArgs &a, bool full_segment, int key, LinRow &r) {
  const int lane = threadIdx.x & 63;
  int full = 0, slots = 0;
  for (int base = 0; base < a.B; base += 64) {
    const int b = base + lane;
    int32_t slot = -1, c0 = 0;
    int n = 0, err = -1, nseg = 1;
    if (b < a.B) {
      err = lin_row_check(a, b, slot, c0, n);
      nseg = lin_segments(a, n);
    }
    const int upto = wave_prefix_sum(nseg - 1);
    const uint64_t hit = __ballot(b < a.B && (full_segment ? key < full + upto : b == key));
    const uint64_t cut = __ballot(nseg > 1);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      r.b = base + l;
      r.nseg = __builtin_amdgcn_readlane(nseg, l);
      const int before = __builtin_amdgcn_readlane(upto, l) - (r.nseg - 1);
      r.full0 = full + before;
      r.slot0 = slots + before + __builtin_popcountll(cut & ((1ull << l) - 1));
      r.n = __builtin_amdgcn_readlane(n, l);
      r.c0 = __builtin_amdgcn_readlane(c0, l);
      r.slot = __builtin_amdgcn_readlane(slot, l);
      r.err = __builtin_amdgcn_readlane(err, l);
      if (r.err == 0 && r.nseg > 1 && r.full0 + r.nseg - 1 > a.more) r.err = KDA_DEVERR_SEQLEN;
      return true;
    }
    const int all = __builtin_amdgcn_readlane(upto, 63);
    full += all;
    slots += all + __builtin_popcountll(cut);
  }
  return false;
}

__device__ __forceinline__ void lin_row(const LinArgs &a, int b, LinRow &r) {
  r.b = b;
  r.full0 = r.slot0 = 0;
  r.err = lin_row_check(a, b, r.slot, r.c0, r.n);
  r.nseg = lin_segments(a, r.n);
  // where it stands matters only to a row that is cut
  if (r.nseg > 1 && a.B > 1) lin_search(a, false, b, r);
}

__device__ __forceinline__ bool lin_full_segment(const LinArgs &a, int e, LinRow &r) {
  if (a.B > 1) return lin_search(a, true, e, r);
  lin_row(a, 0, r);
  return e < r.nseg - 1;
}

// Workgroups are dispatched round-robin over the 8 XCDs. The (unit, key head)
// pairs are dealt to them in turn; the heads that share a key head stand next to
// each other in one XCD's order, so that they read its q and k through one L2.
// (Dealing whole units instead, so that a token's neighbouring heads meet in one
// L2, measured the same on one long row and 15% slower on ragged ones.)
__device__ __forceinline__ bool lin_unit_head(const LinArgs &a, int units, int &unit, int &h) {
  const int n = blockIdx.x, hk = a.H / a.group;
  int j, in_group, kh;
  divmod_uniform(n >> 3, a.group, j, in_group);
  divmod_uniform(8 * j + (n & 7), hk, unit, kh);
  h = kh * a.group + in_group;
  return unit < units;
}

// Accumulator layout of a state. Wave w holds value columns 16 w .. + 15; its
// register tile ni holds key channels 16 ni + 4 g .. + 3 of column m in lane
// (m, g).
template <int DK, int DV>
struct LinState {
  static constexpr int NI = DK / 16;
  v4f s[NI];

  __device__ static int at(int ni) {  // element of a [dv][dk] state
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    return (16 * w + (lane & 15)) * DK + 16 * ni + 4 * (lane >> 4);
  }
  __device__ static int ws_at(int ni) {  // element of a state in the workspace, in register order
    return (ni * lin_threads(DV) + (int)threadIdx.x) * 4;
  }
  __device__ __forceinline__ void load(const float *p, bool ws) {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) s[ni] = *reinterpret_cast<const v4f *>(p + (ws ? ws_at(ni) : at(ni)));
  }
  __device__ __forceinline__ void store(float *p, bool ws) const {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) *reinterpret_cast<v4f *>(p + (ws ? ws_at(ni) : at(ni))) = s[ni];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) s[ni] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  }
};

// A chunk of one token array on its way to LDS, in 16-byte pieces. Offsets from
// the chunk's first token fit 32 bits (strides are at most kLinMaxStride).
// Tokens past the chunk's n are read from its last one (so that no load waits
// behind a per-lane branch) and written as zeros.
template <int D, int NT>
struct Staged16 {
  static constexpr int N = kLinChunk * D / 8 / NT, PITCH = D + 8, STEP = NT / (D / 8);
  u32x4 x[N];

  __device__ __forceinline__ void load(const uint16_t *base, int64_t stride, int n) {
    const int t = (int)threadIdx.x / (D / 8), c = ((int)threadIdx.x % (D / 8)) * 16;
    const uint32_t st = 2 * (uint32_t)stride;  // bytes
    if (n >= kLinChunk) {
      const uint32_t off = pinned(t * st + c);
#pragma unroll
      for (int m = 0; m < N; ++m) x[m] = *at(base + (int64_t)(STEP * m) * stride, off);
    } else {
#pragma unroll
      for (int m = 0; m < N; ++m) x[m] = *at(base, pinned(min(t + STEP * m, n - 1) * st + c));
    }
  }
  __device__ static const u32x4 *at(const uint16_t *base, uint32_t bytes) {
    return reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(base) + bytes);
  }
  __device__ __forceinline__ void store(uint16_t *lds, int n) {
    const int t = (int)threadIdx.x / (D / 8), c = ((int)threadIdx.x % (D / 8)) * 8;
    if (n < kLinChunk) {
#pragma unroll
      for (int m = 0; m < N; ++m)
        if (t + STEP * m >= n) x[m] = (u32x4){0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int m = 0; m < N; ++m) *reinterpret_cast<u32x4 *>(lds + (t + STEP * m) * PITCH + c) = x[m];
  }
};

// Tokens 32 kb + 8 g .. + 7 of a column, each times its factor f, split.
__device__ __forceinline__ Split scaled_values(bf16x8 v, const float (&f)[8]) {
  const u32x4 u = __builtin_bit_cast(u32x4, v);
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16) * f[2 * e];
    x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u) * f[2 * e + 1];
  }
  return split(x);
}

// S <- Gamma_L S + sum_s end_s k_s v_s^T
template <int DK, int DV>
__device__ __forceinline__ void chunk_state(LinState<DK, DV> &S, const uint16_t *kl, const bf16x8 (&vr)[2],
                                            const ChunkDecay &d) {
  constexpr int NI = DK / 16;
  const int g = (threadIdx.x & 63) >> 4;
  const float gl = d.gam[kLinChunk - 1];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) S.s[ni] *= gl;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = d.end[32 * kb + 8 * g + e];
    const Split vs = scaled_values(vr[kb], f);
#pragma unroll
    for (int n4 = 0; n4 < NI; n4 += 4) {
      bf16x8 kt[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) kt[i] = ld_tokens<DK + 8>(kl, 32 * kb, 16 * (n4 + i));
#pragma unroll
      for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
        for (int i = 0; i < 4; ++i) S.s[n4 + i] = mma(kt[i], vs.part[x], S.s[n4 + i]);
    }
  }
}

// Chunks of a segment of n tokens with a checkpoint after cut of them: 64 tokens
// each, the one that reaches a cut inside the segment ends there.
struct LinChunks {
  int n, cut, n1, count;  // n1: chunks before the cut

  __device__ __forceinline__ LinChunks(int n_, int cut_) : n(n_), cut(cut_ > 0 && cut_ < n_ ? cut_ : n_) {
    n1 = (cut + kLinChunk - 1) / kLinChunk;
    count = n1 + (n - cut + kLinChunk - 1) / kLinChunk;
  }
  // tokens [t0, t0 + nt) of chunk c; nt = 0 past the last
  __device__ __forceinline__ void at(int c, int &t0, int &nt) const {
    t0 = c < n1 ? c * kLinChunk : cut + (c - n1) * kLinChunk;
    nt = max(0, min(kLinChunk, (c < n1 ? cut : n) - t0));
  }
};

// D(t, s) of tile (st, tt) for token t = lane's m and s = 4 g + e of their blocks.
__device__ __forceinline__ void tile_decay(const ChunkDecay &d, int st, int tt, float (&D)[4]) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const float at = d.al[kLB * tt + m];
  if (st == tt) {
    // the product after 4 g + 3 by a scan, then one factor more per step down
    const float4 as = *reinterpret_cast<const float4 *>(d.al + kLB * st + 4 * g);
    float x = row_prefix(m > 4 * g + 3 ? at : 1.0f);
    D[3] = x;
    x *= m >= 4 * g + 3 ? as.w : 1.0f;
    D[2] = x;
    x *= m >= 4 * g + 2 ? as.z : 1.0f;
    D[1] = x;
    x *= m >= 4 * g + 1 ? as.y : 1.0f;
    D[0] = x;
  } else {
    float x = row_prefix(at);
    for (int o = st + 1; o < tt; ++o) x *= d.al[kLB * o] * d.suf[kLB * o];
    const float4 sf = *reinterpret_cast<const float4 *>(d.suf + kLB * st + 4 * g);
    D[0] = x * sf.x;
    D[1] = x * sf.y;
    D[2] = x * sf.z;
    D[3] = x * sf.w;
  }
}

// ---- the state sum of every segment that another one follows ----
//
// Reads k and v once; a wave has 16 columns of the state over all key channels
// in accumulators. 8000 tokens x 32 heads of 128 x 128: 43.5 us for 126 MB read and
// 31 written (3.6 TB/s); two rows of 16384 x 32 of 64 x 64: 64 us for 242 and 7.
template <int DK, int DV>
__global__ __launch_bounds__(lin_threads(DV), 2 * DV / 64) void lin_sum_kernel(LinArgs a) {
  constexpr int NT = lin_threads(DV), NW = NT / 64;
  __shared__ __align__(16) uint16_t kl[kLinChunk * (DK + 8)];
  __shared__ __align__(16) uint16_t vl[kLinChunk * (DV + 8)];
  __shared__ __align__(16) ChunkDecay dec[NW];
  int unit, h;
  LinRow r;
  if (!lin_unit_head(a, a.more, unit, h) || !lin_full_segment(a, unit, r) || r.err) return;
  const int seg = unit - r.full0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t tok0 = (int64_t)r.c0 + (int64_t)seg * a.seg * kLinChunk;
  const uint16_t *k = a.k + tok0 * a.ks + (int64_t)(h / a.group) * DK;
  const uint16_t *v = a.v + tok0 * a.vs + (int64_t)h * DV;
  const float *al = a.alpha + tok0 * a.as + h;

  // Every chunk of a segment that another follows is full. The chunk two ahead
  // is requested while one is computed (two register sets rotate), and every NW
  // chunks each wave forms the decays of one of the next NW.
  LinState<DK, DV> S;
  S.zero();
  float total = 1.0f;
  Staged16<DK, NT> ks[2];
  Staged16<DV, NT> vs[2];
  const auto load = [&](int c, int p) {
    if (c >= a.seg) return;
    const int64_t at = (int64_t)c * kLinChunk;
    ks[p].load(k + at * a.ks, a.ks, kLinChunk);
    vs[p].load(v + at * a.vs, a.vs, kLinChunk);
  };
  const auto load_decay = [&](int c) { return c < a.seg ? al[((int64_t)c * kLinChunk + lane) * a.as] : 1.0f; };
  float an = load_decay(wave);
  const auto step = [&](int c, int p) {
    __syncthreads();
    ks[p].store(kl, kLinChunk);
    vs[p].store(vl, kLinChunk);
    if (c % NW == 0) {
      put_chunk_decay(dec[wave], an);
      an = load_decay(c + NW + wave);
    }
    __syncthreads();
    load(c + 2, p);
    const bf16x8 vr[2] = {ld_tokens<DV + 8>(vl, 0, 16 * wave), ld_tokens<DV + 8>(vl, 32, 16 * wave)};
    const ChunkDecay &d = dec[c % NW];
    chunk_state<DK, DV>(S, kl, vr, d);
    total *= d.gam[kLinChunk - 1];
  };
  load(0, 0);
  load(1, 1);
  for (int c = 0; c < a.seg; c += 2) {
    step(c, 0);
    if (c + 1 < a.seg) step(c + 1, 1);
  }
  const int64_t sh = (int64_t)(r.slot0 + seg) * a.H + h;
  S.store(a.ws + sh * (DK * DV), true);
  if (threadIdx.x == 0) a.wdec[sh] = total;
}

// ---- the state entering every segment of a row, in place of the sums ----
//
// A thread takes 4 elements through the row's segments. One row of 15 full
// segments x 32 heads of 128 x 128: 13 us, a chain of loads from the Infinity
// Cache; 16 ragged rows of 5003 tokens in all 12.5 us (a workgroup for every row and
// head, most of them of rows that are not cut).
template <int DK, int DV>
__global__ __launch_bounds__(lin_threads(DV)) void lin_scan_kernel(LinArgs a) {
  int bh, ni, b, h;
  divmod_uniform(blockIdx.x, lin_scan_parts(DK, DV), bh, ni);
  divmod_uniform(bh, a.H, b, h);
  LinRow r;
  lin_row(a, b, r);
  if (r.err || r.nseg < 2) return;
  v4f s = *reinterpret_cast<const v4f *>(a.cache + (int64_t)r.slot * a.slot_stride + (int64_t)h * (DK * DV) +
                                         LinState<DK, DV>::at(ni));
  float *w = a.ws + ((int64_t)r.slot0 * a.H + h) * (DK * DV) + LinState<DK, DV>::ws_at(ni);
  const float *dec = a.wdec + (int64_t)r.slot0 * a.H + h;
  const int64_t step = (int64_t)a.H * (DK * DV);
  for (int j = 0; j + 1 < r.nseg; ++j) {
    const v4f d = *reinterpret_cast<const v4f *>(w);
    *reinterpret_cast<v4f *>(w) = s;
    s = s * dec[(int64_t)j * a.H] + d;
    w += step;
  }
  *reinterpret_cast<v4f *>(w) = s;
}

// ---- outputs, final state and checkpoint ----
//
// 8000 tokens x 32 heads of 128 x 128, fp32 out: 88 us once the clock has settled (98
// to 115 in a process's first calls; with every chunk's inputs resident in L2 a sixth
// less), so what bounds it is mostly not HBM. A chunk of one head takes a wave 48
// MFMAs for S0^T q, 5 for the scores, 18 for their product with v and 48 for the
// state, and as many cycles of VALU work to split the fp32 operands, in phases that
// barriers keep apart. Every wave reads all of q, k and the scores from LDS, 0.5 MB a
// chunk: the LDS is busy 56% of the time (25% in bank conflicts), VALU 40%, MFMA 36%.
// 8 waves of 16 columns keep 128 registers and so two workgroups per CU. 4 waves of
// 32 columns, which would halve those reads, spilled hoisted addresses when they were
// tried (137 us); they have not been timed with the addresses pinned. The transposing
// reads' two rows apart, which takes a fifth of the conflicts away: the same within
// 1%.
template <int DK, int DV, bool BF16>
__global__ __launch_bounds__(lin_threads(DV), 2 * DV / 64) void lin_out_kernel(LinArgs a) {
  constexpr int NT = lin_threads(DV), NW = NT / 64, KB = DK / 32, T = kLinChunk / kLB;
  __shared__ __align__(16) uint16_t ql[kLinChunk * (DK + 8)];
  __shared__ __align__(16) uint16_t kl[kLinChunk * (DK + 8)];
  __shared__ __align__(16) uint16_t vl[kLinChunk * (DV + 8)];
  __shared__ __align__(16) uint16_t pl[kParts][kScoreElems];  // decayed scores, split
  __shared__ __align__(16) ChunkDecay dec[NW];  // of a group of NW chunks
  int unit, h;
  LinRow r;
  // Every row's last segment, then the full ones (measured on MI355X, the whole
  // prefill of 32 heads, bfloat16 out, us, and the other way round: 2 rows of 16384
  // tokens x 64 x 64 221, 239; 16 ragged rows of 5003 tokens in all 104, 111; 32 of
  // 8000 170, 184; 8 of 8000 149, 142, of 1000 each 134, 128).
  if (!lin_unit_head(a, a.more + a.B, unit, h)) return;
  int seg;
  if (unit >= a.B) {
    if (!lin_full_segment(a, unit - a.B, r) || r.err) return;  // reported with the row's last segment
    seg = unit - a.B - r.full0;
  } else {
    lin_row(a, unit, r);
    if (r.err) {
      if (r.err > 0 && h == 0 && threadIdx.x == 0 && a.dev_err) atomicOr(a.dev_err, r.err);
      return;
    }
    seg = r.nseg - 1;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int ck = a.ckpt_pos ? a.ckpt_pos[r.b] : -1;
  float *slot = a.cache + (int64_t)r.slot * a.slot_stride + (int64_t)h * (DK * DV);
  float *ckpt = ck >= 0 ? a.ckpt + ((int64_t)r.b * a.H + h) * (DK * DV) : nullptr;
  if (r.n == 0 && ck != 0) return;
  LinState<DK, DV> S;
  if (r.nseg > 1)
    S.load(a.ws + ((int64_t)(r.slot0 + seg) * a.H + h) * (DK * DV), true);
  else
    S.load(slot, false);
  if (ck == 0 && seg == 0) S.store(ckpt, false);
  if (r.n == 0) return;

  const int64_t full = (int64_t)a.seg * kLinChunk;
  const int first = (int)(seg * full);                    // tokens of the row before the segment
  const int n = (int)min((int64_t)(r.n - first), full);  // and in it
  const int64_t tok0 = (int64_t)r.c0 + first;
  const uint16_t *q = a.q + tok0 * a.qs + (int64_t)(h / a.group) * DK;
  const uint16_t *k = a.k + tok0 * a.ks + (int64_t)(h / a.group) * DK;
  const uint16_t *v = a.v + tok0 * a.vs + (int64_t)h * DV;
  const float *al = a.alpha + tok0 * a.as + h;
  // the tiles above the diagonal that a product over 32 tokens reads: (1, 0) and (3, 2)
  for (int i = threadIdx.x; i < kParts * 2 * kLB * kLB / 4; i += NT) {
    const int part = i >> 7, up = (i >> 6) & 1, t = (i >> 2) & 15, s = (i & 3) * 4;
    *reinterpret_cast<u32x2 *>(&pl[part][score_row(2 * up, t) + 32 * up + kLB + s]) = (u32x2){0u, 0u};
  }
  const LinChunks chunks(n, ck - first);
  Staged16<DK, NT> qs, ks;
  Staged16<DV, NT> vs;
  const auto load = [&](int c) {
    int t0, nt;
    chunks.at(c, t0, nt);
    if (nt == 0) return;
    qs.load(q + (int64_t)t0 * a.qs, a.qs, nt);
    ks.load(k + (int64_t)t0 * a.ks, a.ks, nt);
    vs.load(v + (int64_t)t0 * a.vs, a.vs, nt);
  };
  const auto load_decay = [&](int c) {
    int t0, nt;
    chunks.at(c, t0, nt);
    return lane < nt ? al[(int64_t)(t0 + lane) * a.as] : 1.0f;
  };
  float an = load_decay(wave);
  load(0);
  for (int c = 0; c < chunks.count; ++c) {
    int t0, nt;
    chunks.at(c, t0, nt);
    const ChunkDecay &d = dec[c % NW];
    __syncthreads();
    if (c % NW == 0) {  // the decays of the next NW chunks, one per wave
      put_chunk_decay(dec[wave], an);
      an = load_decay(c + NW + wave);
    }
    qs.store(ql, nt);
    ks.store(kl, nt);
    vs.store(vl, nt);
    __syncthreads();
    load(c + 1);

    // decayed scores, transposed tiles [s][t]: the ten on and below the diagonal over the waves
    for (int i = wave; i < T * (T + 1) / 2; i += NW) {
      const int tt = i >= 6 ? 3 : i >= 3 ? 2 : i >= 1 ? 1 : 0, st = i - tt * (tt + 1) / 2;
      v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        acc = mma(ld_run8(kl + (kLB * st + m) * (DK + 8) + 32 * kb + 8 * g),
                  ld_run8(ql + (kLB * tt + m) * (DK + 8) + 32 * kb + 8 * g), acc);
      float D[4], p[4];
      tile_decay(d, st, tt, D);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = st < tt || m >= 4 * g + e ? acc[e] * D[e] : 0.0f;
      uint32_t w[2 * kParts];
      split_words<4>(p, w);
#pragma unroll
      for (int x = 0; x < kParts; ++x)
        *reinterpret_cast<u32x2 *>(&pl[x][score_row(tt, m) + kLB * st + 4 * g]) = (u32x2){w[2 * x], w[2 * x + 1]};
    }

    // outputs, transposed tiles [j][t]: Gamma_t S0^T q_t
    v4f o[T];
#pragma unroll
    for (int tt = 0; tt < T; ++tt) o[tt] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = S.s[2 * kb + e / 4][e % 4];
      const Split sp = split(x);
#pragma unroll
      for (int t2 = 0; t2 < T; t2 += 2) {
        const bf16x8 q0 = ld_run4x2(ql + (kLB * t2 + m) * (DK + 8) + 32 * kb + 4 * g);
        const bf16x8 q1 = ld_run4x2(ql + (kLB * (t2 + 1) + m) * (DK + 8) + 32 * kb + 4 * g);
#pragma unroll
        for (int i = kParts - 1; i >= 0; --i) {
          o[t2] = mma(sp.part[i], q0, o[t2]);
          o[t2 + 1] = mma(sp.part[i], q1, o[t2 + 1]);
        }
      }
    }
#pragma unroll
    for (int tt = 0; tt < T; ++tt) o[tt] *= d.gam[kLB * tt + m];
    __syncthreads();

    // and sum_s D(t, s) (k_s . q_t) v_s
    const bf16x8 vr[2] = {ld_tokens<DV + 8>(vl, 0, 16 * wave), ld_tokens<DV + 8>(vl, 32, 16 * wave)};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
        for (int tt = 2 * kb; tt < T; ++tt)
          o[tt] = mma(vr[kb], ld_run8(&pl[x][score_row(tt, m) + 32 * kb + 8 * g]), o[tt]);
    const int64_t orow = (int64_t)a.H * DV;
    const int64_t obase = (tok0 + t0) * orow + (int64_t)h * DV + 16 * wave;
    constexpr int OB = BF16 ? 2 : 4;  // bytes of an output
    const uint32_t ooff = pinned(OB * (m * (uint32_t)orow + 4 * g));
    const auto put = [&](int tt) {
      char *to = static_cast<char *>(a.out) + OB * (obase + kLB * tt * orow) + ooff;
      if constexpr (BF16) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4 *>(to) = __builtin_convertvector(o[tt], bf16x4);
      } else {
        *reinterpret_cast<v4f *>(to) = o[tt];
      }
    };
    if (nt == kLinChunk) {
#pragma unroll
      for (int tt = 0; tt < T; ++tt) put(tt);
    } else {
#pragma unroll
      for (int tt = 0; tt < T; ++tt)
        if (kLB * tt + m < nt) put(tt);
    }

    chunk_state<DK, DV>(S, kl, vr, d);
    if (first + t0 + nt == ck) S.store(ckpt, false);
  }
  if (seg + 1 == r.nseg) S.store(slot, false);
}

// ----------------------------------------------------------------------------
// Short prompts of few heads: a workgroup per 16 value columns
// ----------------------------------------------------------------------------
//
// With few (row, head) pairs the kernel above leaves most CUs idle, and latency
// is what counts. Here a workgroup has 16 columns of a head and walks the whole
// row, its waves in two roles, one barrier per chunk. DK / 32 waves carry the
// state: S0^T q_t over the wave's 32 channels, to LDS, then the update. Six waves
// take the scores' products with v, up to 2 score tiles each, split in registers
// in the layout in which the product takes them: 16 tokens against 32 earlier
// ones. One chunk later four of them add up their tokens' terms and write.
// A chunk is requested two chunks ahead (two register sets rotate) and written to
// LDS one ahead. Every column tile forms the scores again, so this costs more
// work in total than the kernel above (8000 tokens x 32 heads: 337 us); lin_walks
// (kda_api.hip) says where it wins. 37 tokens x 32 heads of 128 x 128: 7.0 us
// (the kernel above 11.1), a chunk more takes 2.5 us.

constexpr int kWalkTile = 16, kWalkOutWaves = 6;

// Token-major arrays of one chunk.
template <int DK>
struct WalkTokens {
  static constexpr int PITCH = DK + 8;  // padded against bank conflicts
  uint16_t q[kLinChunk * PITCH], k[kLinChunk * PITCH], v[kLinChunk * kWalkTile];
};

// A chunk's q, k and v tile on their way from memory to LDS, in 16-byte pieces
// spread over NW waves: pieces of 64 lanes, those of k, then those of q, and two
// of v. Tokens past the chunk's nt as in Staged16.
template <int DK, int NW>
struct WalkLoad {
  static constexpr int CP = DK / 8;     // 16-byte pieces of a token = pieces of 64 lanes of an array
  static constexpr int ROWS = 64 / CP;  // tokens per piece of 64 lanes
  static constexpr int WP = 2 * CP, N = (WP + NW - 1) / NW;
  u32x4 x[N], xv;

  __device__ static const u32x4 *at(const uint16_t *base, uint32_t bytes) {
    return reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(base) + bytes);
  }
  __device__ __forceinline__ void load(const LinArgs &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                       int wave, int t0, int nt) {
    const int lane = threadIdx.x & 63, r = lane / CP, c = (lane % CP) * 16;
#pragma unroll
    for (int m = 0; m < N; ++m) {
      const int wp = wave + NW * m;
      if (WP % NW == 0 || wp < WP) {
        const bool isq = wp >= CP;
        const int row0 = (isq ? wp - CP : wp) * ROWS;
        const int64_t st = isq ? a.qs : a.ks;
        const uint16_t *base = (isq ? q : k) + (int64_t)t0 * st;
        if (nt == kLinChunk)
          x[m] = *at(base + row0 * st, pinned(r * (uint32_t)(2 * st) + c));
        else
          x[m] = *at(base, pinned(min(row0 + r, nt - 1) * (uint32_t)(2 * st) + c));
      }
    }
    if (wave < 2)
      xv = *at(v + (int64_t)t0 * a.vs, pinned(min(32 * wave + (lane >> 1), nt - 1) * (uint32_t)(2 * a.vs) + (lane & 1) * 16));
  }
  __device__ __forceinline__ void store(WalkTokens<DK> &to, int wave, int nt) {
    constexpr int PITCH = WalkTokens<DK>::PITCH;
    const int lane = threadIdx.x & 63, r = lane / CP, c = (lane % CP) * 8;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int m = 0; m < N; ++m) {
      const int wp = wave + NW * m;
      if (WP % NW == 0 || wp < WP) {
        const bool isq = wp >= CP;
        const int row = (isq ? wp - CP : wp) * ROWS + r;
        if (nt < kLinChunk && row >= nt) x[m] = zero;
        *reinterpret_cast<u32x4 *>((isq ? to.q : to.k) + row * PITCH + c) = x[m];
      }
    }
    if (wave < 2) {
      const int row = 32 * wave + (lane >> 1);
      if (nt < kLinChunk && row >= nt) xv = zero;
      *reinterpret_cast<u32x4 *>(to.v + row * kWalkTile + (lane & 1) * 8) = xv;
    }
  }
};

// The part of a state that one wave holds: 32 key channels x 16 columns, the
// accumulator layout of two MFMA tiles: channels 16 i + 4 g .. + 3 of column m.
struct WaveState {
  v4f s[2];

  // address of the wave's part of a [dv][dk] state, for this lane
  __device__ static int64_t at(int dk, int tile, int r) {
    const int lane = threadIdx.x & 63;
    return (int64_t)(kWalkTile * tile + (lane & 15)) * dk + 32 * r + 4 * (lane >> 4);
  }
  __device__ __forceinline__ void load(const float *p) {
    s[0] = *reinterpret_cast<const v4f *>(p);
    s[1] = *reinterpret_cast<const v4f *>(p + 16);
  }
  __device__ __forceinline__ void store(float *p) const {
    *reinterpret_cast<v4f *>(p) = s[0];
    *reinterpret_cast<v4f *>(p + 16) = s[1];
  }
  __device__ __forceinline__ void zero() { s[0] = s[1] = (v4f){0.0f, 0.0f, 0.0f, 0.0f}; }

  // S <- Gamma_L S + sum_s end_s k_s v_s^T over channels 32 r .. + 31
  template <int DK>
  __device__ __forceinline__ void update(const WalkTokens<DK> &x, const ChunkDecay &d, int r) {
    const int g = (threadIdx.x & 63) >> 4;
    bf16x8 kt[2][2];
    Split vs[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) kt[kb][i] = ld_tokens<DK + 8>(x.k, 32 * kb, 32 * r + 16 * i);
      const bf16x8 v = ld_tokens<kWalkTile>(x.v, 32 * kb, 0);
      const float4 f0 = *reinterpret_cast<const float4 *>(d.end + 32 * kb + 8 * g);
      const float4 f1 = *reinterpret_cast<const float4 *>(d.end + 32 * kb + 8 * g + 4);
      const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
      vs[kb] = scaled_values(v, f);
    }
    const float gl = d.gam[kLinChunk - 1];
    s[0] *= gl;
    s[1] *= gl;
#pragma unroll
    for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        s[0] = mma(kt[kb][0], vs[kb].part[x], s[0]);
        s[1] = mma(kt[kb][1], vs[kb].part[x], s[1]);
      }
  }
};

template <int DK, bool BF16>
__global__ __launch_bounds__(lin_walk_threads(DK)) void lin_walk_kernel(LinArgs a) {
  constexpr int NR = DK / 32, NW = NR + kWalkOutWaves, PITCH = DK + 8, T = kLinChunk / kLB;
  __shared__ __align__(16) WalkTokens<DK> tok[2];
  __shared__ __align__(16) ChunkDecay dec[2];
  __shared__ v4f part[2][NR][T][64];  // state terms by (chunk parity, wave, 16 tokens)
  __shared__ v4f early[2][2][64];     // products with the first 32 tokens, of tokens 48.. and 32..
  // the column tiles of a head, and the heads of a key head, are one XCD's in a row
  const int hk = a.H / a.group;
  int j, tile, in_group, row, kh;
  divmod_uniform(blockIdx.x >> 3, a.dv / kWalkTile, j, tile);
  divmod_uniform(j, a.group, j, in_group);
  divmod_uniform(8 * j + (blockIdx.x & 7), hk, row, kh);
  if (row >= a.B) return;
  const int h = kh * a.group + in_group;
  int32_t slot_id, c0;
  int n;
  const int err = lin_row_check(a, row, slot_id, c0, n);
  if (err) {
    if (err > 0 && h == 0 && tile == 0 && threadIdx.x == 0 && a.dev_err) atomicOr(a.dev_err, err);
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int ck = a.ckpt_pos ? a.ckpt_pos[row] : -1;
  if (n == 0 && ck != 0) return;
  const LinChunks chunks(n, ck);
  const int64_t tok0 = c0;
  const uint16_t *q = a.q + tok0 * a.qs + (int64_t)(h / a.group) * DK;
  const uint16_t *k = a.k + tok0 * a.ks + (int64_t)(h / a.group) * DK;
  const uint16_t *v = a.v + tok0 * a.vs + (int64_t)h * a.dv + kWalkTile * tile;
  const float *al = a.alpha + tok0 * a.as + h;

  WalkLoad<DK, NW> x[2];
  float an[2] = {1.0f, 1.0f};
  const auto load = [&](int c, int p) {
    int t0, nt;
    chunks.at(c, t0, nt);
    if (nt == 0) return;
    if (wave == NW - 1) an[p] = lane < nt ? al[(int64_t)(t0 + lane) * a.as] : 1.0f;
    x[p].load(a, q, k, v, wave, t0, nt);
  };
  const auto put = [&](int c, int p) {
    int t0, nt;
    chunks.at(c, t0, nt);
    if (nt == 0) return;
    x[p].store(tok[p], wave, nt);
    if (wave == NW - 1) put_chunk_decay(dec[p], an[p]);
  };
  if (n > 0) {
    load(0, 0);
    load(1, 1);
    put(0, 0);
  }

  if (wave < NR) {
    float *slot = a.cache + (int64_t)slot_id * a.slot_stride + (int64_t)h * (DK * a.dv) + WaveState::at(DK, tile, wave);
    float *ckpt = ck >= 0 ? a.ckpt + ((int64_t)row * a.H + h) * (DK * a.dv) + WaveState::at(DK, tile, wave) : nullptr;
    WaveState S;
    S.load(slot);
    if (ck == 0) S.store(ckpt);
    if (n == 0) return;
    __syncthreads();
    const auto step = [&](int c, int p) {
      load(c + 2, p);
      const float xs[8] = {S.s[0][0], S.s[0][1], S.s[0][2], S.s[0][3], S.s[1][0], S.s[1][1], S.s[1][2], S.s[1][3]};
      const Split sp = split(xs);
      bf16x8 qv[T];
#pragma unroll
      for (int tt = 0; tt < T; ++tt) qv[tt] = ld_run4x2(tok[p].q + (kLB * tt + m) * PITCH + 32 * wave + 4 * g);
      v4f o[T];
#pragma unroll
      for (int tt = 0; tt < T; ++tt) o[tt] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = kParts - 1; i >= 0; --i)
#pragma unroll
        for (int tt = 0; tt < T; ++tt) o[tt] = mma(sp.part[i], qv[tt], o[tt]);
#pragma unroll
      for (int tt = 0; tt < T; ++tt) part[p][wave][tt][lane] = o[tt];
      S.update<DK>(tok[p], dec[p], wave);
      int t0, nt;
      chunks.at(c, t0, nt);
      if (t0 + nt == ck) S.store(ckpt);
      put(c + 1, p ^ 1);
      __syncthreads();
    };
    for (int c = 0; c < chunks.count; c += 2) {
      step(c, 0);
      if (c + 1 < chunks.count) step(c + 1, 1);
    }
    S.store(slot);
    return;
  }

  if (n == 0) return;
  __syncthreads();
  // this wave's tokens 16 tt .. + 15 against 32 kb .. + 31; the waves of kb = tt / 2 write
  const int f = wave - NR, tt = f < 4 ? 3 - f / 2 : 5 - f, kb = f == 0 || f == 2 ? 1 : 0;
  const bool writes = kb == tt / 2;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  float gam = 0.0f;
  constexpr int OB = BF16 ? 2 : 4;  // bytes of an output
  const int64_t orow = (int64_t)a.H * a.dv;
  const auto finish = [&](int c, int p) {
    v4f o = part[p][0][tt][lane];
#pragma unroll
    for (int w = 1; w < NR; ++w) o += part[p][w][tt][lane];
    o = o * gam + acc;
    if (tt >= 2) o += early[p][3 - tt][lane];
    int t0, nt;
    chunks.at(c, t0, nt);
    if (kLB * tt + m < nt) {
      char *to = static_cast<char *>(a.out) + OB * ((tok0 + t0 + kLB * tt) * orow + (int64_t)h * a.dv + kWalkTile * tile) +
                 pinned(OB * (m * (uint32_t)orow + 4 * g));
      if constexpr (BF16) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4 *>(to) = __builtin_convertvector(o, bf16x4);
      } else {
        *reinterpret_cast<v4f *>(to) = o;
      }
    }
  };
  const auto step = [&](int c, int p) {
    load(c + 2, p);
    if (c > 0 && writes) finish(c - 1, p ^ 1);
    bf16x8 qv[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) qv[i] = ld_run8(tok[p].q + (kLB * tt + m) * PITCH + 32 * i + 8 * g);
    gam = dec[p].gam[kLB * tt + m];
    float ps[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int st = 2 * kb + i;
      float D[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      v4f sc = {0.0f, 0.0f, 0.0f, 0.0f};
      if (st <= tt) {
#pragma unroll
        for (int e = 0; e < NR; ++e)
          sc = mma(ld_run8(tok[p].k + (kLB * st + m) * PITCH + 32 * e + 8 * g), qv[e], sc);
        tile_decay(dec[p], st, tt, D);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) ps[4 * i + e] = st < tt || (st == tt && m >= 4 * g + e) ? sc[e] * D[e] : 0.0f;
    }
    const Split sp = split(ps);
    const bf16x8 vv = ld_tokens2<kWalkTile>(tok[p].v, 32 * kb, 0);
    acc = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = kParts - 1; i >= 0; --i) acc = mma(vv, sp.part[i], acc);
    if (!writes) early[p][3 - tt][lane] = acc;
    put(c + 1, p ^ 1);
    __syncthreads();
  };
  for (int c = 0; c < chunks.count; c += 2) {
    step(c, 0);
    if (c + 1 < chunks.count) step(c + 1, 1);
  }
  if (writes) finish(chunks.count - 1, (chunks.count - 1) & 1);
}

}  // namespace

template <int DK, int C, bool GATE>
const void *lin_decode_io(bool bf16) {
  return bf16 ? (const void *)lin_decode_kernel<DK, C, GATE, true> : (const void *)lin_decode_kernel<DK, C, GATE, false>;
}

template <int DK>
const void *lin_decode_for(int C, bool gate, bool bf16) {
  if (gate) return C == kLinGateSlabs ? lin_decode_io<DK, kLinGateSlabs, true>(bf16) : nullptr;
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

#define KDA_LIN_DIMS(KERNEL, ...)                                                                             \
  (dk == 64 ? dv == 64 ? (const void *)KERNEL<64, 64 __VA_ARGS__> : (const void *)KERNEL<64, 128 __VA_ARGS__>   \
            : dv == 64 ? (const void *)KERNEL<128, 64 __VA_ARGS__> : (const void *)KERNEL<128, 128 __VA_ARGS__>)

const void *lin_sum_kernel_for(int dk, int dv) { return KDA_LIN_DIMS(lin_sum_kernel); }
const void *lin_scan_kernel_for(int dk, int dv) { return KDA_LIN_DIMS(lin_scan_kernel); }
const void *lin_walk_kernel_for(int dk, bool bf16) {
  if (dk == 64) return bf16 ? (const void *)lin_walk_kernel<64, true> : (const void *)lin_walk_kernel<64, false>;
  return bf16 ? (const void *)lin_walk_kernel<128, true> : (const void *)lin_walk_kernel<128, false>;
}
const void *lin_out_kernel_for(int dk, int dv, bool bf16) {
  return bf16 ? KDA_LIN_DIMS(lin_out_kernel, , true) : KDA_LIN_DIMS(lin_out_kernel, , false);
}

}  // namespace kda
