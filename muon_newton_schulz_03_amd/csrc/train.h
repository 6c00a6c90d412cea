// Launch arguments of the training operators (layer norm, 8-bit checkpoints,
// expert weight gradients, routing), shared by the host entry points
// (train_api.cpp) and the kernels.
#pragma once

#include <cstdint>

#include <hip/hip_runtime_api.h>

namespace muon {

constexpr int kCkptGroup = 128;        // columns that share one scale byte
constexpr int kNormMaxCols = 32768;    // a row lives in one workgroup's registers
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;
// Slots of a call. The kernels count tokens and slots in 32 bits and step past the
// last one, routing by up to a workgroup's run of 2^21 tokens, weight gradients by
// a few steps of 32 slots.
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - (int64_t(1) << 22);

// A checkpoint: e4m3 codes and one power-of-two scale byte per group.
struct CkptView {
  uint8_t *codes;   // NULL: none
  uint8_t *scales;
  int64_t ld_codes, ld_scales;
};

struct NormFwdArgs {
  const void *x;
  void *y;
  const void *w, *b;  // NULL: 1, 0
  float *mean, *rstd; // may be NULL
  int64_t ld_x, ld_y;
  int64_t rows;
  int32_t cols;
  int32_t w_f32;      // w and b are float32 (else bf16)
  float eps;
  double inv_cols;    // 1 / cols
  CkptView ck;
};

struct NormBwdArgs {
  const void *dy, *x, *w;  // w NULL: 1
  const float *mean, *rstd;
  void *dx;
  void *dw, *db;           // either may be NULL
  float *part;             // [blocks][2][cols] float32
  int32_t sums;            // dw or db is wanted
  int64_t ld_dy, ld_x, ld_dx;
  int64_t rows;
  int32_t cols;
  int32_t w_f32;           // w, dw and db are float32 (else bf16)
  int32_t blocks;
};

struct CkptArgs {
  const void *in;     // save: x
  void *out;          // load: values
  int64_t ld;
  int64_t rows;
  int32_t cols;
  CkptView ck;
};

struct WgradArgs {
  const void *dy;          // slots x n
  int64_t ld_dy;
  CkptView x;              // tokens x k
  int64_t tokens, slots;
  const int32_t *offsets;  // groups + 1, or NULL: one group of every slot
  const int32_t *rows;     // slots, or NULL: slot order
  int32_t per_token;
  int32_t n, k, groups;
  void *out;               // group g at out + g * stride elements
  int64_t ld_out, stride;
  float *part;             // [splits][groups][n][k] float32, when splits > 1
  int32_t splits;
  int32_t tiles_n, tiles_k;
  int4 *order;             // groups by length (group, first slot, end), or NULL: in the given order
};

struct RouteFwdArgs {
  const void *logits;
  int64_t ld;
  int32_t tokens, experts, topk;
  int32_t renorm;
  float alpha;
  int32_t *indices;
  float *weights;
  int32_t *counts, *offsets, *rows;
  float *loss;
  // scratch of the form with several workgroups: per block and expert the
  // number of slots and the sum of probabilities, per block the counted tokens
  int32_t *hist;
  float *psum;
  int32_t *valid;
  int32_t blocks, per_block;
};

struct RouteBwdArgs {
  const void *logits;
  int64_t ld;
  int32_t tokens, experts, topk;
  int32_t renorm;
  float alpha;
  const int32_t *indices, *counts;
  const float *dweights;  // NULL: 0
  const float *dloss;     // NULL: 0
  void *dlogits;
  int64_t ld_out;
};

int norm_bwd_blocks(int64_t rows, int64_t cols);
hipError_t launch_norm_fwd(const NormFwdArgs &a, bool bf16, hipStream_t s);
hipError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, hipStream_t s);
hipError_t launch_ckpt_save(const CkptArgs &a, bool bf16, hipStream_t s);
hipError_t launch_ckpt_load(const CkptArgs &a, bool bf16, hipStream_t s);
// Fills tiles and splits of a; the float32 partials take wgrad_part_bytes, the
// order of the groups wgrad_order_bytes.
void wgrad_plan(WgradArgs &a, bool bf16);
size_t wgrad_part_bytes(const WgradArgs &a);
size_t wgrad_order_bytes(const WgradArgs &a);  // not with partials
hipError_t launch_wgrad(const WgradArgs &a, bool bf16, hipStream_t s);
void route_plan(RouteFwdArgs &a);
hipError_t launch_route_fwd(const RouteFwdArgs &a, bool bf16, hipStream_t s);
hipError_t launch_route_bwd(const RouteBwdArgs &a, bool bf16, hipStream_t s);

}  // namespace muon
