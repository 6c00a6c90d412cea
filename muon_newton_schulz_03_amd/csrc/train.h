// Launch arguments of the training operators (layer norm, 8-bit checkpoints,
// expert weight gradients, routing, products of groups of rows, the sum over a
// token's experts with dropout), shared by the host entry points
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

enum Activation : int32_t { kActSilu = 0, kActGelu = 1 };

// Slots in groups: group g's are offsets[g] .. offsets[g + 1] - 1.
struct ProductArgs {
  const void *x, *x2;      // rows of the left operand; x2: of a second product that is added (back), or NULL
  int64_t ld_x, ld_x2;
  int64_t x_rows;
  const void *w, *w2;      // weights; w2: of the gated block's second product, or x2's
  int64_t ld_w, ld_w2;
  int64_t w_stride, w2_stride;  // elements from group to group
  const int32_t *offsets;  // groups + 1, or NULL: one group of every slot
  const int32_t *rows;     // slots, or NULL: slot order
  int64_t slots;
  int32_t groups;
  int32_t gather;          // slot s reads row s of x (0), or rows[s] / gather
  int32_t scatter;         // and writes row s of out (0), or rows[s]
  int32_t back;            // weights n x k lie as rows of the sum's index
  int32_t n, k;            // columns of out, length of the sum
  void *out, *gate, *up;   // gate and up: the gated block's products, or NULL
  int64_t ld_out, ld_gate, ld_up;
  int64_t out_rows;
  int32_t act;             // Activation
  int32_t tiles_n;
  int32_t splits;          // workgroups that share a tile's sums
  int32_t thin_parts;      // whether those tiles have 32 rows instead of 64
  int32_t whole;           // of one group: the first columns whose tiles are not shared
  float *part;             // their parts when there are several
};

struct GatedGradArgs {
  const void *dh, *gate, *up;
  void *dgate, *dup;
  int64_t ld_dh, ld_gate, ld_up, ld_dgate, ld_dup;
  const int32_t *offsets;
  int64_t slots;
  int32_t groups, n;
  int32_t act;
};

constexpr int kCombineMaxTopk = 32;

struct CombineArgs {
  const void *x;           // slots x cols (backward: NULL without dweights)
  const void *res;         // forward: added, or NULL
  const void *dy;          // backward
  void *out;               // forward: y, backward: dx
  float *dweights;         // backward, or NULL
  int64_t ld_x, ld_res, ld_dy, ld_out;
  int64_t tokens;
  int32_t cols, topk;
  const float *weights;    // tokens x topk, or NULL: 1
  const int32_t *indices;  // tokens x topk, < 0: no choice; or NULL: all
  const int32_t *rows;     // backward: slots in the order of dx's rows, or NULL
  int32_t *places;         // backward: scratch, the place of each slot in rows
  const uint64_t *key;     // seed, offset; NULL: nothing is dropped
  uint32_t threshold;      // words below it are dropped
  float scale;             // 1 / (1 - p)
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
// Fills splits, thin_parts and whole of a (from its sizes, groups and the kind of product: back, and
// whether x2 and w2 are set); the parts take product_part_bytes.
void product_plan(ProductArgs &a, bool bf16);
size_t product_part_bytes(const ProductArgs &a);
hipError_t launch_product(const ProductArgs &a, bool bf16, hipStream_t s);
hipError_t launch_gated_grad(const GatedGradArgs &a, bool bf16, hipStream_t s);
hipError_t launch_combine_fwd(const CombineArgs &a, bool bf16, hipStream_t s);
hipError_t launch_combine_bwd(const CombineArgs &a, bool bf16, hipStream_t s);

}  // namespace muon
