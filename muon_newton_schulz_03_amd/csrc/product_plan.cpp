// The tiles of products, and whether their sums are shared out: by an estimate of
// their time.
#include "product_plan.h"

#include <algorithm>
#include <cmath>

namespace muon {
namespace {

// The form with the least time by this estimate: us for 64 bytes of the sum's
// index when the CUs have up to c tiles each, and us a tile besides, measured (at
// 2 GHz, the rate the power cap leaves) as
//              256 x 256   128 x 256       64 x 128        64 x 64        32 x 64
//   bf16       0.85 c      0.62, 0.5 c     0.22, 0.17 c    0.2, 0.13 c    0.085, 0.09 c
//   float32    3.7 c       2.08, 1.85 c    0.62, 0.5 c     0.37, 0.3 c    0.2, 0.17 c
//   a tile     3           1.2             1.8             1.3            3 (float32: 1.5)
// the first figure that of a single tile. A 256 x 256 tile skips 32-row blocks
// without slots, down to half its time; through registers it takes
// a tenth more (the others' times there are not told apart, and whether a sum is shared
// out is asked as if all went straight to LDS: the workspace's size is known from
// the sizes alone). What it chose against the next best, us:
//   one token, 8 of 128 experts 768x2048, gated     32 x 64   14.7    (64 x 64: 19)
//   64 tokens, 18432x7168, gated, nothing shared    64 x 128  133     (64 x 64: 149)
//   80 tokens, 8 of 89, 418x135, gated              128 x 256 13.7    (64 x 128: 18, 32 x 64: 40)
//   1024 tokens, 2048x2048                          64 x 128  17      (64 x 64: 21)
//   2048 tokens, 4096x4096                          128 x 256 86      (64 x 128: 98)
//   4096 tokens, 8 of 128 experts 768x2048, gated   256 x 256 280     (128 x 256: 309)
//   8192 tokens, 4095x2047 (registers)              256 x 256 203     (128 x 256: 222)
//   float32, 1024 tokens, 1024x2048                 32 x 64   39      (64 x 64: 47)
//   float32, 777 tokens, 3 of 12, 532x1024, gated   64 x 64   56      (32 x 64: 72)
//   float32, 4096 tokens, 2048x4096                 64 x 128  518     (128 x 256: 534)
struct Estimate {
  double us[kForms], shared_us;
  int splits;  // workgroups to a tile whose sums are shared out; 1 where the sum is too short, shared_us is without the second launch
  bool thin2, thin_parts;
  double least() const { return *std::min_element(us, us + kForms); }
};
Estimate estimate(const ProductArgs &a, bool bf16, bool lds) {
  const double groups = double(std::min<int64_t>(a.groups, a.slots)), slots = double(a.slots);
  const double steps = double(a.k) * (bf16 ? 2 : 4) * (a.back && a.x2 ? 2 : 1) / 64;
  // a group's last tile is half a one on average
  auto tiles = [&](int rows, int cols) {
    return (a.groups > 1 ? std::max(groups, slots / rows + groups / 2) : std::ceil(slots / rows)) * tiles_across(a, cols);
  };
  // One group's weights that no cache holds and that one or two row tiles get from
  // HBM: 5.5 TB/s, and 41 GB/s of x and weights a CU (37 in rows of 64 bytes, 52 of
  // four waves that wait for themselves alone).
  const double bytes = double(a.k) * a.n * (bf16 ? 2 : 4) * (a.w2 ? 2 : 1);
  auto cold = [&](int rows, int cols, double c, double rate) {
    return a.groups > 1 || slots > 2 * rows || bytes < 2e8 ? 0. : std::max(bytes / 5.5e6, steps * c * 64 * (rows + cols) / (rate * 1e3));
  };
  auto us_of = [&](int rows, int cols, double one, double each, double besides, double rate = 41) {
    const double c = std::ceil(tiles(rows, cols) / kCus);
    return std::max(steps * (c > 1 ? std::max(one, each * c) : one), cold(rows, cols, c, rate)) + besides * c;
  };
  const double fill = std::max(bf16 ? 0.55 : 0.5, std::min(1., slots * tiles_across(a, 256) / tiles(256, 256) / 256)) * (lds ? 1 : 1.1);
  Estimate e;
  e.us[kLarge] = bf16 ? us_of(256, 256, 0.85 * fill, 0.85 * fill, 3) : us_of(256, 256, 3.7 * fill, 3.7 * fill, 3);
  e.us[kWide] = bf16 ? us_of(128, 256, 0.62, 0.5, 1.2, 37) : us_of(128, 256, 2.08, 1.85, 1.2, 37);
  e.us[kSmall] = bf16 ? us_of(64, 128, 0.22, 0.17, 1.8) : us_of(64, 128, 0.62, 0.5, 1.8);
  e.us[kMid] = bf16 ? us_of(64, 64, 0.2, 0.13, 1.3, 37) : us_of(64, 64, 0.37, 0.3, 1.3, 37);
  e.us[kThin] = bf16 ? us_of(32, 64, 0.085, 0.09, 3, 52) : us_of(32, 64, 0.2, 0.17, 1.5, 52);
  // a streaming workgroup needs a step between two tiles, and room for the groups;
  // from sizes alone, as the workspace is asked for without the lists
  if (lds && (a.k == 0 || a.groups > kStreamGroups)) e.us[kLarge] = 1e30;
  // memory's latency asks for long loads, float32 products for two workgroups a CU:
  // 1024 tokens, 1024x2048, 40 us against 46; 64 tokens, 4096x4096, gated, 52 against 48
  e.thin2 = !bf16 && tiles(32, 64) > kCus;
  e.shared_us = 1e30;
  e.splits = 1;
  const double values = slots * a.n * (a.w2 && !a.back ? 2 : 1);
  auto share = [&](int rows, bool thin, double one, double each, double besides, double rate) {
    for (int n = 2; n <= 16 && 8 * n <= steps; ++n) {
      const double c = std::ceil(tiles(rows, 64) * n / kCus);
      const double us = std::max(std::ceil(steps / n) * std::max(one, each * c), cold(rows, 64, c, rate) / n) + besides * c + n * values * 8 / 5e6;
      if (us >= e.shared_us) continue;
      e.shared_us = us;
      e.splits = n;
      e.thin_parts = thin;
    }
  };
  e.thin_parts = false;
  share(64, false, bf16 ? 0.2 : 0.37, bf16 ? 0.13 : 0.3, 1.3, 37);
  // half of a 64-row tile's waves have nothing to do for up to 32 rows
  if (slots <= 32) share(32, true, bf16 ? 0.085 : 0.2, bf16 ? 0.09 : 0.17, bf16 ? 3 : 1.5, 52);
  return e;
}

}  // namespace

ProductForm product_form(const ProductArgs &a, bool bf16, bool lds) {
  const Estimate e = estimate(a, bf16, lds);
  const int form = int(std::min_element(e.us, e.us + kForms) - e.us);
  return form == kThin && e.thin2 ? kThin2 : ProductForm(form);
}

// A long sum with few tiles is shared out to several workgroups a tile, whose
// parts a second launch adds: 8 bytes a part and value, and what the launch costs.
// 64 tokens, 1024x8192: float32 82 -> 20 us, bf16 19 -> 13; 1 token, 2048x2304:
// float32 26 -> 13, bf16 stays at 8, two launches take 12. Up to 32 rows in 32-row
// tiles: 16 tokens, 7168x18432, float32, 146 -> 123; 5 tokens, 7168x5408, 50 -> 43. Of one group's tiles
// that go round the CUs more than a whole number of times, those left over are
// shared out, two launches of their own: 64 tokens, 18432x7168, gated, 288 tiles
// of 64 x 128 (256 of them take 92), 133 -> 107-112 us; float32, 348 tokens, 3686x4512,
// backward, 158 -> 136; 1152 tokens, 4096x7168, gated, 1130 -> 1064.
void product_plan(ProductArgs &a, bool bf16) {
  a.splits = 1;
  a.whole = 0;
  a.thin_parts = 0;
  if (a.slots == 0 || a.groups == 0) return;
  const Estimate e = estimate(a, bf16, true);
  double best = e.least();
  const double join = 5, shared = std::max(e.shared_us + join, 12.);  // the least that two launches take
  if (shared < best) {
    best = shared;
    a.splits = e.splits;
    a.thin_parts = e.thin_parts;
  }
  if (a.groups > 1) return;
  const int forms[][2] = {{256, 256}, {128, 256}, {64, 128}, {64, 64}, {32, 64}};
  for (const auto &f : forms) {
    const int64_t down = (a.slots + f[0] - 1) / f[0], across = tiles_across(a, f[1]);
    const int64_t full = down * across / kCus * kCus / down;  // columns of tiles that go round evenly
    if (full == 0 || full == across) continue;
    ProductArgs w = a, t = a;
    w.n = int32_t(full * (a.w2 && !a.back ? f[1] / 2 : f[1]));
    t.n = a.n - w.n;
    const Estimate rest = estimate(t, bf16, true);
    const double us = estimate(w, bf16, true).least() + 3 + rest.shared_us + join;
    if (us >= best) continue;
    best = us;
    a.splits = rest.splits;
    a.thin_parts = rest.thin_parts;
    a.whole = w.n;
  }
}

size_t product_part_bytes(const ProductArgs &a) {
  return a.splits > 1 ? size_t(a.splits) * size_t(a.slots) * size_t(a.n - a.whole) * (a.w2 && !a.back ? 2 : 1) * sizeof(float) : 0;
}

}  // namespace muon
