// Internal interface between the C ABI (abi.hip) and the kernel launchers.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kLayoutThreads = 512;  // threads per layout workgroup

// Workspace sections (byte offsets from the workspace base, 256-aligned).
struct WsLayout {
  size_t status, num_tokens_per_expert, num_tokens_per_rank, is_token_in_rank,
      expert_offset, rank_offset, send_offset, token_slot, recv_pos, recv_token,
      recv_k, send_token, tok_mask, hist;
  size_t total;
  int nblk;  // layout workgroups (token tiles)
  int tile;  // tokens per tile
};

constexpr int kMaxPadMultiple = 1024;

// Rows of a receive buffer: T*K pairs plus at most pad-1 padding rows per
// expert segment.
inline int64_t recv_capacity(int64_t T, int K, int E, int pad) {
  return T * K + (int64_t)E * (pad - 1);
}

// layout_pairs: (t,k) pairs per layout tile (512 sizes the workspace: more
// pairs per tile means fewer tiles and a smaller histogram).  pad: expert
// segments padded to a multiple of it (sizes the per-row inverse maps).
WsLayout plan_workspace(int64_t T, int K, int E, int P, int layout_pairs = kLayoutThreads, int pad = 1);


struct LayoutArgs {
  const void* idx;
  int itype, T, K, E, P, epr, nblk, tile;
  int pad;                // expert segments padded to a multiple of this
  int R;                  // receive rows (recv_capacity)
  int* hist;              // [nblk+1][E+1+P]: per tile, bucket counts then partition token counts
  int scanned;            // hist rewritten by layout_scan_kernel: row j the counts of the tiles
                          // before j, row nblk the column totals
  unsigned long long* tok_mask;  // [T] partitions each token is sent to
  int* num_tokens_per_expert;
  int* num_tokens_per_rank;
  uint8_t* is_token_in_rank;
  int* expert_offset;
  int* rank_offset;
  int* send_offset;
  int* token_slot;
  int* recv_pos;
  int* recv_token;
  int* recv_k;
  int* send_token;        // [T*min(K,P)] token of each send row
  int* status;
};

// Dynamic LDS of the two layout kernels.
size_t layout_count_lds(int E, int P, int tile);
size_t layout_rank_lds(int E, int P, int tile, int K);

hipError_t launch_layout(const LayoutArgs& a, hipStream_t s);

// Padding rows of a padded layout: rows [expert_offset[e] + n_e,
// expert_offset[e+1]) of every expert get zero chunks (and a zero score).
// Written by extra waves of the kernel that writes the receive rows.
constexpr int kPadRows = 8;  // padding rows per fill wave

struct PadArgs {
  void* dst;                         // [R, NV] chunks
  float* scores_out;                 // [R] or null
  const int* expert_offset;          // [E+1], padded
  const int* num_tokens_per_expert;  // [E]
  int E, NV, R;
  int pad;                           // the handle's multiple (1: no padding, no fill waves)
  int ngrp;                          // segments per row
  int nblk;                          // row blocks per expert
  int nwaves;                        // fill waves: pad_fill_waves(E, pad, NV), 0 when unpadded
};

// Wavefronts of one padding fill: an expert has at most pad-1 padding rows,
// in blocks of kPadRows, and a row has one segment per 64 chunks.
inline int64_t pad_fill_waves(int E, int pad, int NV) {
  if (pad <= 1) return 0;
  return (int64_t)E * ((pad - 1 + kPadRows - 1) / kPadRows) * ((NV + 63) / 64);
}

// Token-row -> receive-row direction (dispatch, rows of the combine backward).
struct ScatterArgs {
  const void* src;        // [T, NV] chunks
  const int* recv_pos;    // [T, K]
  const float* w;         // [T, K] or null
  void* dst;              // [R, NV] chunks
  float* scores_out;      // [R] or null
  int T, K, NV, R;
  int ngrp;               // wave groups per token (set by the launcher)
  int dtype;
  bool scale;             // dst = round(w * src)
  int* status;
  PadArgs pad;            // padding rows of dst, filled by pad.nwaves waves after the token waves
};

// Receive-row -> token-row direction (combine, unscaled dispatch backward).
struct GatherArgs {
  const void* src;        // [R, NV] chunks
  const int* recv_pos;    // [T, K]
  const float* w;         // [T, K] or null (plain sum)
  void* dst;              // [T, NV] chunks
  int T, K, NV, R;
  int ngrp;               // wave groups per token (set by the launcher)
  int dtype;
  int* status;
};

// Router-weight gradient dot[t,k] = <tok[t], rcv[recv_pos[t,k]]>, one
// workgroup per token; with `gather` it also writes dst[t] = sum_k [w *] rcv.
struct DotArgs {
  const void* tok;        // [T, NV] chunks
  const void* rcv;        // [R, NV] chunks
  const int* recv_pos;    // [T, K]
  const float* w;         // [T, K] or null
  void* dst;              // [T, NV] chunks (gather only)
  float* dot_out;         // [T, K]
  int T, K, NV, R;
  int dtype;
  bool gather;
  int* status;
};

// Staged exchange: a deduplicated send buffer [send_cap, NV] per (token,
// partition) pair, rows send_offset[r] + token_slot[t,r].
struct StagedArgs {
  const void* src;        // send: x [T]; expand: S [send_cap]; reduce: y [R]; combine: Q [send_cap]
  void* dst;              // send: S; expand: recv [R]; reduce: Q; combine: out [T]
  const int* recv_pos;    // [T, K]
  const int* token_slot;  // [T, P]
  const int* send_offset; // [P+1]
  const int* rank_offset; // [P+1]
  const int* send_token;  // [send_cap]
  const unsigned long long* tok_mask;  // [T]
  const float* w;         // [T, K] or null
  float* scores_out;      // expand: [R] or null
  int T, K, P, NV, R;
  int send_cap;           // rows of the send buffer (>= send_offset[P])
  int ngrp;               // wave groups per row (set by the launcher)
  int dtype;
  bool scale;             // expand: dst = round(w * src)
  int* status;
  PadArgs pad;            // expand: padding rows of dst, filled by the grid's first pad.nwaves waves
};

// The router: scores, choice and weights of one token per wavefront, and the
// gradient back to the logits.
struct RouteArgs {
  const void* z;          // [T, E] logits
  const float* bias;      // [E] or null: added to the scores for the choice only
  int* idx;               // [T, K]
  float* w;               // [T, K]
  int T, E, K, dtype;
  int score;              // MOE_SCORE_*
  bool renorm;
  float scale;
  int groups, topk_groups;
  int per, L;             // experts per group, lanes per group (set by the launcher)
};

struct RouteBwdArgs {
  const void* z;          // [T, E] logits
  const int* idx;         // [T, K]
  const float* grad_w;    // [T, K]
  void* grad_z;           // [T, E]
  int T, E, K, dtype;
  int score;
  bool renorm;
  float scale;
};

// The balance loss of a router over sequences of tokens, and its gradient.
struct BalanceArgs {
  const void* z;          // [T, E] logits
  const void* idx;        // [T, K] int32 or int64
  const int* seq;         // [S+1] first token of each sequence, or null: one of all T
  const uint8_t* mask;    // [T] 0: not counted; or null
  float* loss;            // [2]
  int* counts;            // [S, E]
  float* probs;           // [S, E]
  int* tokens;            // [S]
  int T, E, K, S, dtype, itype, score;
  int tile;               // tokens of a workgroup (backward: of a wave; set by the launcher)
  int cols;               // second kernel: experts of a workgroup (set by the launcher)
  float *part_p, *part_z;  // partials by slot (run + sequence): [slots, E], [slots]
  int *part_c, *part_n;
  double *seq_sum, *seq_z;  // [S, columns], [S]
  const float* grad_loss;   // backward: [2]
  const void* grad_base;    // [T, E] or null
  void* grad_z;             // [T, E]
};

// The norms before and after a block (norm_kernel), and rows to 8 bits.
struct NormArgs {
  const void* x;          // [T, nch] chunks: the residual stream (quant: the rows)
  const void* y;          // [T, nch], or [R, nch] with recv_pos; null before a block
  const void* w1;         // [nch] post-norm, or null
  const void* gate;       // [T / group, nch] or null
  const void* w2;         // [nch] the norm of the (next) block, or null
  const int* recv_pos;    // [T, K] or null
  const float* w;         // [T, K] or null (plain sum)
  void* out;              // [T, nch]
  void* n;                // [T, nch]
  int8_t* q;              // [T, H] in the place of n, or null
  float* scale;           // [T]
  float* rstd;            // [T] before a block, [T, 2] after it; or null
  int* status;
  float residual, eps, offset;
  int T, nch, K, R;
  int group;              // tokens of a gate
  int dtype;
};

struct NormBwdArgs {
  const void* g;          // [T, nch] gradient of out (before a block: added to grad_x), or null
  const void* gn;         // [T, nch] gradient of n, or null
  const void* x;          // [T, nch]
  const void* y;          // [T, nch]
  const void *w1, *gate, *w2;
  const float* rstd;
  void *gx, *gy, *gw1, *gg, *gw2;  // each may be null
  float *part1, *part2, *partg;    // [runs, H]; null where not wanted
  float* means;                    // [T, 2] of a wide row after a block, where it has a norm
  float residual, offset;
  int T, nch, group, gates;
  int rows, parts, runs;  // rows of a run, runs that share a gate (1: a run holds whole gates), runs
  int dtype;
  bool block;             // after a block
};

constexpr int kNormWide = 8192;  // MOE_NORM_WIDE

void norm_bwd_plan(int64_t T, int64_t group, int nch, bool wide, int* rows, int* parts, int* runs);

// Grouped product of 8-bit rows and weights.
struct I8Args {
  const int8_t* q;        // [M, K]
  const float* qs;        // [M]
  const int8_t* w;        // [E, N, K]
  const float* ws;        // [E, N]
  const int* offset;      // [E+1] first receive row of each expert, or null: one expert, rows 0..M-1
  const int* recv_token;  // [R] or null: row p of q belongs to receive row p
  void* out;              // [R or M, N or N/2]
  int M, R, E, N;
  int kch;                // 16-byte chunks of a row of q and w
  int act;                // MOE_ACT_* or MOE_ACT_NONE
  int dtype;              // of out
};

// A whole expert layer for a few tokens (at most kFewMaxPairs pairs).
constexpr int kFewMaxPairs = 512;  // MOE_FEW_MAX_PAIRS

struct FewArgs {
  const void* x;          // [T, H]
  const void* idx;        // [T, K] int32 or int64
  const float* w;         // [T, K] or null (plain sum)
  const void* w13;        // [E, 2I, H]: gate rows, then up rows
  const void* w2;         // [E, H, I]
  float* mid;             // workspace, the activations [T*K, I], in an order of the kernels' own
  void* out;              // [T, H]
  int T, K, E, H, I;
  int itype, dtype, act;
  int pairs;              // T*K
  int hch, ich;           // 16-byte chunks of a row of H, of I
  int groups;             // distinct experts a call can have at most (set by the launcher)
  int split, part_lines;  // parts of the sum over I, 256-byte lines of a part (set by the launcher)
};

// Low-rank adapters on a layout of one adapter per token: the three kernels'
// shared arguments.
struct LowrankArgs {
  const int* expert_offset;  // [E+1]
  const int* recv_token;     // [R], -1 for a row without a token
  const void* rows;          // [T, W]: shrink and wgrad read them
  const void* bank;          // [A, r, W]
  const float* w;            // [T] or null: shrink (backward), expand and wgrad multiply by it
  float* u;                  // [R, r]: shrink writes it, expand and wgrad read it
  const float* saved;        // [R, r]: the forward's u (backward shrink with dot)
  float* dot;                // [T] or null: <raw, saved>
  const void* base;          // [T, W] or null: added by expand
  void* out;                 // [T, W] (expand), [A, r, W] (wgrad)
  int T, E, A, R, r;
  int wch;                   // 16-byte chunks of a wide row
  int dtype;
  int tiles;                 // expand: tiles of rows a wave takes (set by the launcher)
  bool backward;             // shrink: u = w * raw
};

struct Tuning {
  int chunks_per_lane;  // 1, 2, 4: consecutive 64-chunk segments per wave
  int nontemporal;      // 0, 1, 2
  int waves_per_block;  // 1, 2, 4, 8
  int layout_pairs;     // 512, 1024, 2048, 4096
  int gather_mode;      // 0: by row width (LDS-staged from 4 KiB); 1: LDS-staged (gather_lds_kernel);
                        // 2: registers (gather_kernel)
  int gather_waves;     // waves per workgroup of the LDS-staged gather: waves_per_block when
                        // that is set, else 0 (by row width, lds_gather_waves)
  // measurement: when ev_stop is set, the launch goes through
  // hipExtLaunchKernel, which binds ev_stop to the kernel's completion and,
  // when ev_start is set too, records ev_start just before the kernel; null
  // for every other launch
  hipEvent_t ev_start = nullptr;
  hipEvent_t ev_stop = nullptr;
};

// Launches a row kernel, with the tuning's measurement events when it has
// them.
template <typename F, typename... Args>
inline void launch_kernel(F kernel, dim3 grid, dim3 block, uint32_t lds, hipStream_t s, const Tuning& t,
                          Args... args) {
  if (t.ev_stop)
    hipExtLaunchKernelGGL(kernel, grid, block, lds, s, t.ev_start, t.ev_stop, 0u, args...);
  else
    hipLaunchKernelGGL(kernel, grid, block, lds, s, args...);
}

constexpr int kMaxDotWaves = 16;         // waves of one token-dot workgroup
constexpr size_t kMaxDotLds = 64 * 1024;  // LDS for its per-segment values

size_t dot_lds_bytes(int NV, int K);
int64_t row_waves(int64_t T, int NV, int cpl);

hipError_t launch_scatter(const ScatterArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_gather(const GatherArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_token_dot(const DotArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_send(const StagedArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_expand(const StagedArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_reduce_partitions(const StagedArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_combine_partitions(const StagedArgs& a, const Tuning& t, hipStream_t s);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t s);
hipError_t launch_balance(BalanceArgs a, hipStream_t s);
hipError_t launch_balance_bwd(BalanceArgs a, hipStream_t s);
int balance_runs(int64_t T);
int balance_columns(int E);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t s);
hipError_t launch_quant(const NormArgs& a, hipStream_t s);
hipError_t launch_i8(const I8Args& a, hipStream_t s);
hipError_t launch_few(const FewArgs& a, hipStream_t s);
hipError_t launch_lowrank_shrink(const LowrankArgs& a, hipStream_t s);
hipError_t launch_lowrank_expand(const LowrankArgs& a, hipStream_t s);
hipError_t launch_lowrank_pass(const LowrankArgs& shrink, const LowrankArgs& expand, hipStream_t s);
hipError_t launch_lowrank_wgrad(const LowrankArgs& a, const LowrankArgs& b, float* parts, int splits, hipStream_t s);
int lowrank_wgrad_splits(int64_t R, int A, int r, int hch, int nch, int dtype);
hipError_t launch_copy(void* dst, const void* src, size_t bytes, hipStream_t s);

}  // namespace moe
