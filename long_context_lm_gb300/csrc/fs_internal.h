// fs_internal.h -- launchers shared between the kernel files and the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fs.h"

namespace fs {

struct Shape {
  int batch, H, N, d;
  int BH() const { return batch * H; }
  int C() const { return N / 32; }
  int nblk() const { return N / 128; }
};

cudaError_t launch_round_bf16(const float *src, void *dst, size_t n, cudaStream_t st);
cudaError_t launch_cell_summary(const void *k, bool f32, const Shape &sh, float *kbar,
                                float *amax, cudaStream_t st);
size_t prune_workspace_bytes(const Shape &sh);
cudaError_t launch_prune(const float *amax, const Shape &sh, int P, int W, int32_t *pool,
                         int32_t *pool_count, void *ws, cudaStream_t st);
cudaError_t launch_select(const void *q, const float *kbar, const float *amax,
                          const int32_t *pool, const int32_t *pool_count, const float *lambda,
                          const float *sigma, const Shape &sh, int K, int cap, int W,
                          bool fs_mode, int32_t *sel, float *sel_score, int *err,
                          cudaStream_t st);
// RoPE angle table (rope_table_bytes(N) of device memory, written by
// launch_rope_table) and the window operands prepared from it: kt = rotated
// keys [rows, 128] bf16 (hi | lo), v16 = values [rows, 64] fp16.
size_t rope_table_bytes(int N);
cudaError_t launch_rope_table(void *tab, int N, float rope_base, cudaStream_t st,
                              int *clear = nullptr);
// k0_prep with the cell summaries of the same keys (one read of k).
cudaError_t launch_prep_summary(const void *k, const void *v, const void *tab, const Shape &sh,
                                void *kt, void *v16, float *kbar, float *amax, int *err,
                                cudaStream_t st);
cudaError_t launch_prep(const void *k, const void *v, const void *tab, const Shape &sh, void *kt,
                        void *v16, int *err, cudaStream_t st);
// Both attention branches (window RoPE branch, NoPE readout of the selected
// cells) in one persistent tcgen05 kernel.  window: run the window branch
// (reads kt, v16, tab); sel != nullptr: run the long branch (reads the raw
// k, v cells); write_long: write RMSNorm(o_long) to `out` instead of the
// mixed output; o_long_in (window only, nullable): a precomputed long branch
// to mix in.
struct AttnArgs {
  Shape sh;
  const void *q, *k, *v;
  const void *kt, *v16, *tab;
  const int32_t *sel;
  const float *o_long_in;
  const float *mix;
  int w, K;
  float rms_eps;
  bool window, write_long;
  float *out;
  int *err;
  int *sched;  // nullable: two ints, zero at launch, left zero (q-tile tickets)
  long long *timeline;  // nullable: per CTA, global-timer ns at its start and end
};
cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t st);
// Per-CTA timeline of the calling host thread's next attention launches
// (fs_set_attention_timeline): buffer and its length in int64 entries.
void set_attention_timeline(long long *timeline, int entries);
// Bounded decode state (see k6_decode.cu): a global part (256-byte header
// whose first int is the error word, then the relative-angle tables), then
// one fixed-size block per (batch, head).  Offsets inside a head's block.
constexpr int kDecodeHeaderInts = 192;  // counts and slot lists of one head
constexpr int kDecodeTabRows = 64 + 16;  // (cos, sin)(o theta): o = r < 64, o = 64a, a < 16
struct DecodeLayout {
  int w, P, W, K, pend, nslots;
  size_t hdr, slot_cell, slot_amax, slot_kbar, slot_k, slot_v, ring_k, ring_v;
  size_t head_bytes;              // one (batch, head)
  size_t tab, global_bytes;       // angle tables inside the global part; its size
  size_t total(int BH) const { return global_bytes + (size_t)BH * head_bytes; }
};
DecodeLayout decode_layout(int w, int P, int W, int K);
size_t decode_smem_bytes(const DecodeLayout &L);
cudaError_t launch_decode_init(const void *k, const void *v, const float *kbar, const float *amax,
                               const int32_t *pool, const int32_t *pool_count, int BH, int N,
                               int N0, float rope_base, const DecodeLayout &L, void *state,
                               cudaStream_t st);
// One decode step for token t of every (batch, head).
struct DecodeArgs {
  const void *q_t, *k_t, *v_t;
  void *state;
  const float *lambda, *sigma, *mix;
  DecodeLayout L;
  int batch, H, t;
  float rms_eps;
  float *out;
  int32_t *sel_out;
};
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t st);

// Shared q / k / v projection (k7_qkv.cu): RMSNorm row scale, gain folded
// into the weights, one tcgen05 GEMM writing q, k, v [batch, H, N, 64] bf16.
struct QkvArgs {
  const void *x;      // [batch, N, D] bf16
  const float *gain;  // [D] or null (ones)
  const void *w;      // [3*H*64, D] bf16
  int batch, N, D, H;
  float eps;
  void *q, *k, *v;
  void *ws;           // qkv_workspace_bytes
  int *err;
};
size_t qkv_workspace_bytes(int M, int D, int H);
// FS-B forests (k9_fsb.cu): per (batch, head) two leaf lists (all cells;
// cells with a_c > tau), the tau forest's prefix count, then per forest the
// node means [nodes, 64] and (radius, a_max, first cell, -) [nodes].
constexpr int kFsbMaxLevels = 24;
struct FsbLayout {
  int C, levels, nodes;
  int level_off[kFsbMaxLevels];
  size_t list, hcount, mean, meta, head_bytes;
};
FsbLayout fsb_layout(int C);
cudaError_t launch_fsb(const void *q, const void *k, const float *kbar, const float *amax,
                       const float *lambda, const float *sigma, const Shape &sh, int K, int beam,
                       float tau, void *ws, int32_t *sel, cudaStream_t st);
// Gradients of the forward (k8_backward.cu), from the forward's selection.
struct BwdArgs {
  Shape sh;
  const void *q, *k, *v;   // bf16
  const float *g;          // dL/dout
  const int32_t *sel;      // the forward's selection [BH, N, K]
  const float *mix;
  int w, K;
  float rope_base, rms_eps;
  float *dq, *dk, *dv, *dmix;
  void *ws;                // backward_workspace_bytes
  int *err;                // bounded-wait failures (FS_ERR_TIMEOUT)
};
size_t backward_workspace_bytes(const Shape &sh);
cudaError_t launch_backward(const BwdArgs &a, cudaStream_t st);
cudaError_t launch_qkv(const QkvArgs &a, cudaStream_t st);

// Rotary positions (k10_rope.cu).  Two tensors; H[i] = 0: none.  Strides in
// elements between batches, heads and tokens.
struct RopeArgs {
  const void *x[2];
  void *y[2];
  int H[2];
  long long xs[2][3], ys[2][3];
  bool f32;
  int batch, N, d;
  const int32_t *pos;
  long long pos_stride;
  int pos0, inverse;
  const fs_rope_plan *plan;
};
int rope_make_plan(const fs_rope_params &p, fs_rope_plan *plan);
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st);

// Paged key/value cache (k11_cache.cu).
struct CacheRowsArgs {
  fs_cache c;
  const void *k, *v;   // append: bf16 rows
  long long ks[3], vs[3];
  void *k_out, *v_out; // read
  bool f32;            // read: fp32 rows
  const int32_t *start, *count, *path;
  int T;
};
cudaError_t launch_cache_append(const CacheRowsArgs &a, cudaStream_t st);
cudaError_t launch_cache_read(const CacheRowsArgs &a, cudaStream_t st);
cudaError_t launch_cache_accept(const CacheRowsArgs &a, cudaStream_t st);

// Attention of drafted tokens over the cache (k12_tree.cu).
struct TreeArgs {
  fs_cache c;
  const void *q;
  const int32_t *past, *count;
  const int64_t *tree;
  int H, T, window;
  float scale;
  void *out, *ws;
  long long wait_cycles;  // after which a wait gives up
};
size_t tree_workspace_bytes(const fs_cache &c, int H, int T);
cudaError_t launch_tree(const TreeArgs &a, cudaStream_t st);

// Linear attention with a decay for each head (k14_linear.cu): one sweep
//   out_t = scale (state before t, decayed, + sum over the sweep's tokens up to t)
// over the tokens of every (sequence, head), in order or in reverse.  The
// forward is one sweep; the gradients are three, with q, k, v and dout in
// other places.  A head h of the sweep reads head h / share of a tensor.
// In reverse the state enters the first token without a decay and is decayed
// once more after the last (it is lam R of the token behind).
struct LinearRows {
  const void *x;       // bf16
  long long s[3];      // elements between sequences, heads, tokens
  int share;
};
struct LinearSweep {
  LinearRows q, k, v;
  void *out;
  long long os[3];
  bool out_f32;            // parts of a sum over heads: contiguous fp32
  const float *state;      // [batch, H, d, d] or null (zeros)
  float *state_out;        // or null; may be `state`
  bool transposed;         // both are held [value][key]
  float state_mul;         // what the given state is multiplied by; its inverse for state_out
  bool reverse;
};
struct LinearArgs {
  LinearSweep sweep[3];
  int sweeps;
  int batch, H, T, d;
  const float *decay;
  const int32_t *count;
  float scale;
  long long wait_cycles;  // after which a wait of the chunked kernels gives up
};
cudaError_t launch_linear_recurrent(const LinearArgs &a, cudaStream_t st);
// The same in chunks of 128 tokens (k16_linear_tc.cu), with linear_chunk_bytes of
// scratch for states.
size_t linear_chunk_bytes(int sweeps, int batch, int H, int T, int d);
cudaError_t launch_linear_chunks(const LinearArgs &a, void *ws, int *err, cudaStream_t st);
struct LinearSumArgs {
  const float *part;   // [batch, H, T, d]
  void *out;           // bf16 [batch, H / share, T, d]
  long long os[3];
  int batch, H, share, T, d;
  const int32_t *count;
};
cudaError_t launch_linear_sum(const LinearSumArgs &a, cudaStream_t st);

// Norms around a block (k15_norm.cu).  Row strides in elements.
struct NormArgs {
  const void *x, *gate, *residual;   // gate, residual: or null
  long long xs, gs, rs;
  bool x_f32, r_f32;
  const float *gain, *next_gain;     // or null (ones)
  int M, D, groups;                  // groups 0: no norm after the block
  bool next;
  float scale, eps;
  void *z, *y;                       // forward
  long long zs, ys;
  const void *dz, *dy;               // backward: either may be null
  long long dzs, dys;
  void *dx, *dgate, *dres;           // dgate, dres: or null
  long long dxs, dgs, drs;
  float *dgain, *dnext;              // or null
  float *ws;
  int mode, per, list;               // set by the launch: how groups are added, vectors
  float inv_n, inv_D;                // (elements) of a group, floats of a team's list
  bool wide;                         // fp32 rows go 32 bytes at a time
};
size_t norm_workspace_bytes(int M, int D);
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t st);

}  // namespace fs
