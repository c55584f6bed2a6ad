// kda_linear_impl.h - interface of the linear-attention kernels (kda_linear.hip)
// and the block norm (kda_norm.hip) to the C ABI in kda_api.hip.

#pragma once

#include <stddef.h>
#include <stdint.h>

namespace kda {

// Arguments of the linear-attention kernels.
struct LinArgs {
  float *cache;
  int64_t num_slots, slot_stride;
  const int32_t *slot_ids, *cu, *ckpt_pos;
  const uint16_t *q, *k, *v, *gate;
  const float *alpha, *weight;
  int64_t qs, ks, vs, as;  // elements between tokens
  void *out;               // fp32, or bf16 when out_bf16
  float *ckpt;
  int32_t *dev_err;
  float eps;
  int32_t B, H, group, dv, n_tok, ntile;  // group = H / Hk heads share a key head
  int32_t out_bf16;
  // prefill: segments of seg chunks; at most `more` segments that another of their row follows
  int32_t seg, more;
  float *ws;    // states, [2 more][H][dv dk]
  float *wdec;  // decays over a segment, [2 more][H]
};

// Slabs of columns per lane of the gated single-token step, whose workgroup owns
// all dv columns of a head (waves = dv / (4 * slabs)). Measured on MI355X at 2, 4
// and 8 slabs: 13 rows x 24 heads at 64 x 128 8.3, 7.7, 7.2 us (the last 6.6 in a
// later run); 8 x 32 at 128 x 128 9.5, 8.8, 8.5; 64 x 32 46.8, 49.3, 47.7: 8 wins
// where latency counts and gives up 2% of the largest batch.
constexpr int kLinGateSlabs = 8;
const void *lin_decode_kernel_for(int dk, int C, bool gate, bool bf16);

constexpr int kLinChunk = 64;    // tokens per chunk of the prefill
// Most elements between tokens: the bytes from a chunk's first token to its last fit 32 bits.
constexpr int64_t kLinMaxStride = 1 << 24;
// Threads of its kernels: a wave per 16 value columns.
inline constexpr int lin_threads(int dv) { return 4 * dv; }
// Kernel handles of the prefill: the state sums of the segments, the states
// entering them, and the outputs.
const void *lin_sum_kernel_for(int dk, int dv);
const void *lin_scan_kernel_for(int dk, int dv);
const void *lin_out_kernel_for(int dk, int dv, bool bf16);
// The kernel for short prompts of few heads: workgroups per (row, head) and threads.
const void *lin_walk_kernel_for(int dk, bool bf16);
inline constexpr int lin_walk_tiles(int dv) { return dv / 16; }
inline constexpr int lin_walk_threads(int dk) { return 2 * dk + 6 * 64; }
// Workgroups of the scan per (row, head).
inline constexpr int lin_scan_parts(int dk, int dv) { return dk * dv / 4 / lin_threads(dv); }

// Arguments of the block norm.
struct NormArgs {
  const void *resid;
  const uint16_t *z, *gate;
  void *resid_out, *y;
  const float *w_post, *w_pre;
  int64_t rs, zs, ros, ys, gs;
  float scale, eps;
  int32_t rows, D, y_bf16;
};

// Kernel, threads and workgroups of a block norm.
struct NormLaunch {
  const void *fn;
  int threads, blocks;
};
NormLaunch norm_launch(int rows, int D, bool resid_bf16);

}  // namespace kda
