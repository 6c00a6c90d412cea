// Which tiles a product of groups of rows takes, from its sizes, groups and type
// (host code; what the forms are: product.hip).
#pragma once

#include "train.h"

namespace muon {

constexpr int kCus = 256;
constexpr int kStreamGroups = 1024;  // that a streaming workgroup keeps the tiles of

// 256 x 256, 128 x 256, 64 x 128, 64 x 64, 32 x 64, and 32 x 64 in half the LDS
enum ProductForm : int { kLarge, kWide, kSmall, kMid, kThin, kForms, kThin2 = kForms };

// lds: the operands go straight to LDS.
ProductForm product_form(const ProductArgs &a, bool bf16, bool lds);

// Columns of tiles of `cols` columns (the gated block's two products share a tile).
inline int tiles_across(const ProductArgs &a, int cols) {
  const int wide = a.w2 && !a.back ? cols / 2 : cols;
  return (a.n + wide - 1) / wide;
}

}  // namespace muon
