// Says what the plan makes of products, without a GPU. A line of input names one:
//   bf16 kind lds slots groups n k
// (kind 0: forward, 1: gated, 2: backward, 3: backward of both of the gated block's
// products; n, k: the product's columns and the length of its sum), a line of output
// its form, the columns that are not shared out, and the parts of the others (0: none)
// and whether those are of 32 rows. Without input, "all": every combination of type,
// kind, way of loading, form and sharing that some size of a wide grid takes.
#include <cstdio>
#include <cstring>
#include <set>
#include <tuple>

#include "product_plan.h"

using namespace muon;

namespace {

ProductArgs product(int kind, int64_t slots, int64_t groups, int64_t n, int64_t k) {
  ProductArgs a{};
  a.x_rows = 1;
  a.slots = slots;
  a.groups = int32_t(groups);
  a.n = int32_t(n);
  a.k = int32_t(k);
  a.back = kind >= 2;
  a.w2 = kind == 1 || kind == 3 ? &a : nullptr;
  a.x2 = kind == 3 ? &a : nullptr;
  return a;
}

// The form of what is not shared out, -1 where all is.
int form_of(ProductArgs a, bool bf16, bool lds) {
  if (a.splits > 1 && a.whole == 0) return -1;
  if (a.whole) a.n = a.whole;
  return product_form(a, bf16, lds);
}

void all() {
  const int slots[] = {1, 16, 33, 64, 130, 300, 1000, 2300, 5000, 9000, 20000, 65536};
  const int sizes[] = {1, 8, 72, 256, 520, 1024, 2304, 5877, 18432, 32768};
  std::set<std::tuple<int, int, int, int, int>> seen;
  for (int bf16 = 0; bf16 < 2; ++bf16)
    for (int kind = 0; kind < 4; ++kind)
      for (int lds = 0; lds < 2; ++lds)
        for (int s : slots)
          for (int n : sizes)
            for (int k : sizes)
              for (int groups : {1, 2, 16, 64, 128, 600, 1025}) {
                ProductArgs a = product(kind, s, groups, n, k);
                product_plan(a, bf16 != 0);
                const int form = form_of(a, bf16 != 0, lds != 0);
                const int type = kind == 3 ? 2 : kind;  // kernels know forward, gated and backward
                if (form >= 0) seen.emplace(bf16, type, lds, form, 0);
                if (a.splits > 1) seen.emplace(bf16, type, lds, a.thin_parts ? kThin2 : kMid, 1);
              }
  for (const auto &[b, t, l, f, p] : seen) std::printf("%d %d %d %d %d\n", b, t, l, f, p);
}

}  // namespace

int main(int argc, char **argv) {
  if (argc > 1 && !std::strcmp(argv[1], "all")) {
    all();
    return 0;
  }
  int bf16, kind, lds;
  long long slots, groups, n, k;
  while (std::scanf("%d %d %d %lld %lld %lld %lld", &bf16, &kind, &lds, &slots, &groups, &n, &k) == 7) {
    ProductArgs a = product(kind, slots, groups, n, k);
    product_plan(a, bf16 != 0);
    std::printf("%d %d %d %d\n", form_of(a, bf16 != 0, lds != 0), a.whole, a.splits > 1 ? a.splits : 0, a.thin_parts);
  }
  return 0;
}
