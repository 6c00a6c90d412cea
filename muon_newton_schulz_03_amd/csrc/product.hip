// Products of groups of rows with their own weights (gfx950): what an expert
// layer's tokens meet between the routing and the sum over each token's experts.
//   gated:     h[s, :] = act(x[t(s)] Wg_g^T) * (x[t(s)] Wu_g^T)
//   forward:   y[p(s), :] = x[q(s)] W_g^T
//   backward:  y[p(s), :] = x[q(s)] W_g  (+ x2[q(s)] W2_g, one sum)
// for the slots s of group g, offsets[g] <= s < offsets[g + 1].
//
// Weights lie as rows of the layer's outputs. A forward product sums over
// their columns: both operands have the sum's index innermost, and a fragment
// is one 16-byte LDS read. A backward product sums over their rows: the
// weights' tile goes to LDS row by row and comes back through the transposing
// LDS reads (float32: by single words).
//
// bf16 makes products of v_mfma_f32_32x32x16_bf16, float32 of
// v_mfma_f32_32x32x2_f32 (float32 products and sums; the four values of a
// fragment's 16 bytes are four products): the same bytes in LDS, the same reads.
// A sum runs in one float32 accumulator, or in two or four where as many sets of
// waves share it (64x64 and 32x64 tiles), and in up to sixteen parts of those where
// workgroups do; they are added in order, in float32, and outputs are rounded once.
//
// What bounds it. Few slots a group: the weights, each read once (32 tokens, 8 of
// 128 experts 2048x768: 60-66 us among other calls, 53 us and 290 MB at 5.5 TB/s when
// the last call's weights, of which the cache before HBM keeps a part, are the same; 64
// tokens, gated, two dense 18432x7168: 107-112 us, 4.8 TB/s).
// Many: the socket's power, at which the shader clock falls to 1.5-2 GHz, for one
// group (4096 tokens, dense 18432x7168: 1700-1810 us, 1200-1270 TFLOP/s, matrix units
// busy 69%); for many experts also what their tiles fetch again and that they
// are not full (16384 tokens, 8 of 128 experts 768x2048, gated: 850-896 us, 930 TFLOP/s,
// busy 50%, 2.34 GB read for 0.87 GB of operands). There every byte that is not moved counts: whole 128-byte
// lines of the operands in a stage took 7% off, tiles that take up the next one's
// loads before they store 3-4%. LDS reads meet no bank conflicts (under 0.1%).
// float32: the matrix units (4096 tokens, 2048x4096: 521 us, 132 TFLOP/s of 154).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lanes.h"
#include "product_plan.h"
#include "train.h"

namespace muon {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBand = 8;             // tiles of a group that take turns within one column of tiles

// A workgroup's tile: kWM x kWN waves of 32 kI x 64 (gated: 32 columns of each
// product), the 32-row blocks dealt to the wave rows in turn, so that a tile
// with few rows leaves each of them few. kK > 1: as many such sets of waves share
// the sums, each with an LDS ring of its own, and add up at the end. kStream: a
// workgroup a CU, which goes from tile to tile and loads the next one's first
// steps before it stores the last one's sums. kRow: bytes of a row in a step's LDS
// stage; 128 are a whole line, 64 leave room for a second workgroup a CU or a
// third stage.
template <int kWM_, int kWN_, int kI_, int kK_, int kStages_, int kRow_, bool kStream_>
struct Form {
  static constexpr int kRow = kRow_, kChunks = kRow / 16;  // 16-byte chunks of a row
  static constexpr int kWM = kWM_, kWN = kWN_, kI = kI_, kK = kK_, kStages = kStages_;
  static constexpr bool kStream = kStream_;
  static constexpr int kWaves = kWM * kWN * kK, kThreads = kWaves * 64;
  static constexpr int kBM = kWM * kI * 32, kBN = kWN * 64;
  static constexpr int kABytes = kBM * kRow;
  static constexpr int kStage = kABytes + kBN * kRow;  // a ring's
  static constexpr int kRing = kStages * kStage;
  static constexpr int kLds = kRing * kK + (kStream ? (4 * kBM + kStreamGroups) * 4 : 0);
  static constexpr int kOfRing = kWM * kWN;                         // waves of a ring
  static constexpr int kLoaders = kOfRing < 4 ? kOfRing : 4;        // that load it
  static constexpr int kX = kABytes / 1024 / kLoaders, kW = kBN * kRow / 1024 / kLoaders;  // their loads, a KiB each
  static_assert(kX * kLoaders * 1024 == kABytes && kW * kLoaders * 1024 == kBN * kRow);
  static constexpr int kPerSimd = kWaves >= 8 ? 2 : kWaves * (kLds > 80 * 1024 ? 1 : 2) / 4;
};
using Large = Form<2, 4, 4, 1, 2, 128, true>;    // 256 x 256, 136 KiB of LDS
using LargeAny = Form<2, 4, 4, 1, 2, 128, false>;  // the same, for operands that go through registers
using Wide = Form<1, 4, 4, 1, 3, 64, false>;     // 128 x 256, 72 KiB: two workgroups a CU
using Small = Form<2, 2, 1, 1, 3, 128, false>;   // 64 x 128, 72 KiB
using Mid = Form<2, 1, 1, 2, 3, 64, false>;      // 64 x 64, two sets of waves to a sum, 48 KiB
using Thin = Form<1, 1, 1, 4, 3, 128, false>;    // 32 x 64, four waves to a sum, 144 KiB
using Thin2 = Form<1, 1, 1, 4, 3, 64, false>;    // the same in 72 KiB: two workgroups a CU

__device__ inline float act_value(float g, int act, float &slope) {
  if (act == kActSilu) {
    // exp(-g) as a power of two, the exponent's rounding error put back
    const float t = g * -1.44269504f, lo = fmaf(g, -1.44269504f, -t) + g * -1.925963033e-8f;
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, lo * 0.693147181f, e);
    e = e == e ? e : __builtin_amdgcn_exp2f(t);  // an infinity times the correction 0
    const float s = __builtin_amdgcn_rcpf(1.f + e);
    slope = fmaf(g * s, g > 0.f ? e * s : 1.f - s, s);  // 1 - s, without cancellation
    return g * s;
  }
  const float cdf = 0.5f * erfcf(g * -0.707106781f);
  const float q = g * g, pdf = 0.398942280f * __builtin_amdgcn_exp2f(q * -0.721347520f);
  slope = fmaf(g, pdf, cdf);
  return g * cdf;
}

// ---------------------------------------------------------------------------
// tiles of groups
// ---------------------------------------------------------------------------

struct Tile {
  int32_t group;   // < 0: none
  int32_t n;       // column of tiles
  int64_t lo, hi;  // its slots
};

__device__ inline int wave_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// An offset, cut to what there is.
__device__ inline int slot_bound(const ProductArgs &a, int g) {
  const int o = a.offsets[g];
  return o < 0 ? 0 : o > int(a.slots) ? int(a.slots) : o;
}

// A group's tiles, tiles_n across and at most `rows` slots each, lie in bands of
// kBand row tiles, `first` row tiles of other groups before them.
__device__ __forceinline__ Tile group_tile(const ProductArgs &a, uint32_t id, int group, uint32_t first, uint32_t mine, int64_t lo, int64_t hi) {
  Tile t{group, 0, 0, 0};
  const uint32_t local = id - first * uint32_t(a.tiles_n);
  const uint32_t band = local / (kBand * uint32_t(a.tiles_n)), in = local - band * kBand * uint32_t(a.tiles_n);
  const uint32_t wide = mine - band * kBand < kBand ? mine - band * kBand : kBand;
  t.n = __builtin_amdgcn_readfirstlane(int(in / wide));
  const int m = __builtin_amdgcn_readfirstlane(int(band * kBand + in % wide));
  // the group's 32-row blocks, dealt evenly to its tiles: a tile of few rows
  // would wait for its weights at every step
  const int each = int((uint32_t(hi - lo + 31) / 32 + mine - 1) / mine) * 32;
  t.lo = lo + int64_t(m) * each;
  t.hi = t.lo + each < hi ? t.lo + each : hi;
  return t;
}

// The row tiles of a run of groups from g0 on: a lane counts those of `run` of
// them, whose offsets it loads at once.
constexpr int kRun = 8;
struct Count {
  int at[kRun + 1], upto;  // offsets, and the tiles up to the lane's last group
};
__device__ __forceinline__ int tiles_of(const Count &c, int r, int rows) {
  return c.at[r + 1] > c.at[r] ? (c.at[r + 1] - c.at[r] + rows - 1) / rows : 0;
}
__device__ __forceinline__ int count_tiles(Count &c, const ProductArgs &a, int g0, int run, int before, int rows, int lane) {
#pragma unroll
  for (int r = 0; r <= kRun; ++r) {
    const int g = g0 + lane * run + (r < run ? r : run);
    c.at[r] = slot_bound(a, g < a.groups ? g : a.groups);
  }
  int sum = 0;
#pragma unroll
  for (int r = 0; r < kRun; ++r) sum += tiles_of(c, r, rows);
  c.upto = before + wave_scan(sum, lane);
  return __builtin_amdgcn_readlane(c.upto, 63);
}
__device__ __forceinline__ int run_of(const ProductArgs &a) { return a.groups >= 64 * kRun ? kRun : (a.groups + 63) / 64; }

// The tiles of XCD x (every eighth workgroup runs on it): a contiguous part.
struct Part {
  uint32_t at, end;
};
__device__ __forceinline__ Part part_of(const ProductArgs &a, uint32_t total) {
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x, tiles = total * uint32_t(a.tiles_n * a.splits), per = (tiles + 7) / 8;
  const uint32_t from = (block & 7) * per, to = from + per < tiles ? from + per : tiles;
  return {from + (block >> 3), to};
}

// This workgroup's only tile, and which part of its sum.
__device__ __forceinline__ Tile find_tile(const ProductArgs &a, int rows, int lane, int &split) {
  uint32_t total = uint32_t((a.slots + rows - 1) / rows);  // row tiles
  const int run = run_of(a);
  Count c;
  if (a.offsets) {
    int before = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64 * run) before = count_tiles(c, a, g0, run, before, rows, lane);
    total = uint32_t(before);
  }
  const Part part = part_of(a, total);
  split = 0;
  if (part.at >= part.end) return Tile{-1, 0, 0, 0};
  const uint32_t id = part.at / uint32_t(a.splits);
  split = __builtin_amdgcn_readfirstlane(int(part.at - id * uint32_t(a.splits)));
  if (!a.offsets) return group_tile(a, id, 0, 0, total, 0, a.slots);
  const uint32_t row = id / uint32_t(a.tiles_n);  // in which group's tiles
  int g0 = 0;
  if (a.groups > 64 * run)
    for (int before = count_tiles(c, a, 0, run, 0, rows, lane); uint32_t(before) <= row;) {
      g0 += 64 * run;
      before = count_tiles(c, a, g0, run, before, rows, lane);
    }
  const int owner = __builtin_amdgcn_readfirstlane(__builtin_ctzll(__ballot(uint32_t(c.upto) > row)));
  int sum = 0;
#pragma unroll
  for (int r = 0; r < kRun; ++r) sum += tiles_of(c, r, rows);
  uint32_t first = 0, mine = 0, before = uint32_t(__builtin_amdgcn_readlane(c.upto - sum, owner));
  int group = 0, lo = 0, hi = 0;
#pragma unroll
  for (int r = 0; r < kRun; ++r) {
    const uint32_t n = uint32_t(__builtin_amdgcn_readlane(tiles_of(c, r, rows), owner));
    const int from = __builtin_amdgcn_readlane(c.at[r], owner), to = __builtin_amdgcn_readlane(c.at[r + 1], owner);
    const bool here = before <= row && row < before + n;
    group = here ? g0 + owner * run + r : group;
    first = here ? before : first;
    mine = here ? n : mine;
    lo = here ? from : lo;
    hi = here ? to : hi;
    before += n;
  }
  return group_tile(a, id, group, first, mine, lo, hi);
}

// A streaming workgroup keeps the tiles up to each group in LDS (`upto`).
__device__ __forceinline__ void keep_tiles(const ProductArgs &a, int *upto, int rows, int lane) {
  const int run = run_of(a);
  int before = 0;
  for (int g0 = 0; g0 < a.groups; g0 += 64 * run) {
    Count c;
    before = count_tiles(c, a, g0, run, before, rows, lane);
    int sum = c.upto;
#pragma unroll
    for (int r = kRun - 1; r >= 0; --r) {
      const int g = g0 + lane * run + r;
      if (r < run && g < a.groups) upto[g] = sum;
      sum -= tiles_of(c, r, rows);
    }
  }
}
__device__ __forceinline__ Tile kept_tile(const ProductArgs &a, const int *upto, uint32_t id, int rows, int lane) {
  if (!a.offsets) return group_tile(a, id, 0, 0, uint32_t((a.slots + rows - 1) / rows), 0, a.slots);
  const int row = int(id / uint32_t(a.tiles_n));
  int group = 0;
  for (int g0 = 0; g0 < a.groups; g0 += 64) {
    const uint64_t past = __ballot(g0 + lane < a.groups && upto[g0 + lane] > row);
    if (past) {
      group = __builtin_amdgcn_readfirstlane(g0 + __builtin_ctzll(past));
      break;
    }
  }
  const int first = group ? upto[group - 1] : 0;
  return group_tile(a, id, group, uint32_t(__builtin_amdgcn_readfirstlane(first)),
                    uint32_t(__builtin_amdgcn_readfirstlane(upto[group] - first)), slot_bound(a, group), slot_bound(a, group + 1));
}

// The entry of a slot's list, and the rows of x and of out that it stands for
// (-1: none).
__device__ inline int entry(const ProductArgs &a, int64_t s) { return a.rows ? a.rows[s] : int(s); }
__device__ inline int source_row(const ProductArgs &a, int64_t s, int v) {
  if (!a.gather) return s < a.x_rows ? int(s) : -1;
  if (v < 0) return -1;
  const int r = a.gather == 1 ? v : int(uint32_t(v) / uint32_t(a.gather));
  return r < a.x_rows ? r : -1;
}
__device__ inline int out_row(const ProductArgs &a, int64_t s, int v) {
  return !a.scatter ? int(s) : v < a.out_rows ? v : -1;  // v < 0 stays below 0
}

// ---------------------------------------------------------------------------
// the tiled kernel
// ---------------------------------------------------------------------------

// 16 bytes of a fragment: eight bf16 or four float32 of the sum's index. The
// weights come first: a lane's 16 sums are then columns of one row of x, 4 (lane
// / 32) .. + 3 of each eight, which leave from the registers.
__device__ inline void multiply(f32x16 &acc, const u32x4 &x, const u32x4 &w, __bf16) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}
__device__ inline void multiply(f32x16 &acc, const u32x4 &x, const u32x4 &w, float) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bits_f32(w[e]), bits_f32(x[e]), acc, 0, 0, 0);
}

// The 32 columns of a row that the lanes l and l + 32 hold, to p, the first n of them.
__device__ inline void store_row(__bf16 *p, const float (&f)[16], int fh, int n) {
  uint32_t d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = pack2(f[2 * i], f[2 * i + 1]);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    // the lower lane takes the first of two runs of eight columns, the upper one the second
    const auto a = __builtin_amdgcn_permlane32_swap(d[4 * g], d[4 * g + 2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d[4 * g + 1], d[4 * g + 3], false, false);
    Raw8<__bf16> r;
    r.v = u32x4{uint32_t(a[0]), uint32_t(b[0]), uint32_t(a[1]), uint32_t(b[1])};
    const int c = 16 * g + 8 * fh;
    store8(p + c, r, n - c);
  }
}
__device__ inline void store_row(float *p, const float (&f)[16], int fh, int n) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int c = 8 * g + 4 * fh;
    if (n - c >= 4) {
      *reinterpret_cast<u32x4_any *>(p + c) = u32x4{f32_bits(f[4 * g]), f32_bits(f[4 * g + 1]), f32_bits(f[4 * g + 2]), f32_bits(f[4 * g + 3])};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n - c) p[c + e] = f[4 * g + e];
    }
  }
}

// 16 bytes at any address of global memory.
template <typename T>
__device__ inline u32x4 load_whole(const T *p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) u32x4_any *>((const __attribute__((address_space(1))) char *)(p));
}
// The first min(n, 16 / sizeof(T)) elements at p, zeros behind them. kRoom: at
// least 16 bytes of the operand end at p + n; they are read whole and moved down.
template <bool kRoom, typename T>
__device__ inline u32x4 load_chunk(const T *p, int n) {
  constexpr int kE = 16 / int(sizeof(T));
  if constexpr (kRoom) {
    const int short_by = n < kE ? kE - n : 0;
    u32x4 v = load_whole(p - short_by);
    // by a chunk (all of it zeros), or 8, 4, 2 bytes
    const uint32_t by = uint32_t(short_by < kE ? short_by : kE) * uint32_t(sizeof(T));
    if (by & 16) v = u32x4{0u, 0u, 0u, 0u};
    if (by & 8) v = u32x4{v[2], v[3], 0u, 0u};
    if (by & 4) v = u32x4{v[1], v[2], v[3], 0u};
    if (sizeof(T) == 2 && (by & 2)) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    return v;
  }
  if (n >= kE) return load_whole(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < kE - 1; ++e)
    if (e < n) {
      if constexpr (sizeof(T) == 2)
        v[e / 2] |= uint32_t(reinterpret_cast<const uint16_t *>(p)[e]) << (16 * (e & 1));
      else
        v[e] = reinterpret_cast<const uint32_t *>(p)[e];
    }
  return v;
}

// Buffer resource over the 4 GiB from p (raw, untyped loads; the last dword is
// the gfx9 default format).
__device__ inline u32x4 whole(const void *p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return u32x4{uint32_t(at), uint32_t(at >> 32) & 0xffffu, 0xffffffffu, 0x00020000u};
}
// The same in every lane, said so: an operand of the assembly below has to be
// in scalar registers.
__device__ inline uint32_t scalar(uint32_t v) { return uint32_t(__builtin_amdgcn_readfirstlane(int(v))); }
__device__ inline u32x4 scalar(const u32x4 &v) { return u32x4{scalar(v[0]), scalar(v[1]), 0xffffffffu, 0x00020000u}; }
// 16 bytes a lane from the buffer straight to LDS (lane l's at lds + 16 l). In
// assembly, because the compiler would wait for all of these loads before each
// transposing LDS read; the waits that they need stand at the top of each step.
// The LDS address goes in through m0, which the compiler so knows to have set; the
// wait states: one from there to the load, five from a vector instruction that has
// written a scalar operand.
__device__ inline void to_lds(const u32x4 &r, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "{m0}"(scalar(lds)), "v"(voff), "s"(r), "s"(scalar(soff))
               : "memory");
}

// Where chunk c of a stage's row lies: at c ^ swizzle, so that 16 rows' reads of
// one chunk take all banks.
template <class F>
__device__ inline int swizzle(int row) {
  return F::kRow == 64 ? (row >> 2) & 3 : (row >> 1) & 7;
}

// Where column col of row r of a backward product's weight tile lies in its
// stage (bf16): rows of `wide` columns in runs of 32, run i of row r at place
// i ^ (r & 3) within its four (of two, i ^ (r & 1)), so that a transposing
// read, 32 columns of four consecutive rows, spreads over the banks.
template <int kBN>
__device__ inline int tr_run(int row, int run) {
  return kBN >= 128 ? (run & ~3) | ((run ^ row) & 3) : run ^ (row & 1);
}
template <int kBN>
__device__ inline int tr_at(int row, int col) {
  return row * (kBN * 2) + (tr_run<kBN>(row, col >> 5) << 6) + (col & 31) * 2;
}

// kDirect: 16-byte loads straight to LDS. Needs operands whose rows start on
// 16-byte boundaries, whole chunks in each row, and byte offsets below 2^32.
// kPart: the tile's part of a sum that several workgroups share goes to a.part, in
// slot order.
template <typename T, class F, bool kBack, bool kGated, bool kDirect, bool kPart>
__global__ __launch_bounds__(F::kThreads, F::kPerSimd) void product_kernel(const ProductArgs a) {
  constexpr int kE = 16 / int(sizeof(T));            // elements of a chunk
  constexpr int kStep = F::kRow / int(sizeof(T));  // sum indices of a step
  constexpr int kParts = F::kRow / 32;              // fragments of a row, two chunks each
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int kI = F::kI, kBN = F::kBN;
  __shared__ __attribute__((aligned(1024))) char smem[F::kLds];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // kStream: rows of x and of out of a tile's slots, for two tiles in turn, and the groups' tiles
  int *table = reinterpret_cast<int *>(smem + F::kRing * F::kK), *upto = table + 4 * F::kBM;
  Tile t;
  Part part{};
  int split = 0;
  if constexpr (F::kStream) {
    uint32_t total = uint32_t((a.slots + F::kBM - 1) / F::kBM);
    if (a.offsets) {
      if (wave == 0) keep_tiles(a, upto, F::kBM, lane);
      __syncthreads();
      total = uint32_t(__builtin_amdgcn_readfirstlane(upto[a.groups - 1]));
    }
    part = part_of(a, total);
    if (part.at >= part.end) return;
    t = kept_tile(a, upto, part.at, F::kBM, lane);
  } else {
    t = find_tile(a, F::kBM, lane, split);
    if (t.group < 0 || t.lo >= t.hi) return;
  }

  const int each = (a.k + kStep - 1) / kStep;  // steps of a part
  const int steps = kBack && a.x2 ? 2 * each : each;

  // its place in the ring's waves, and which ring
  const int lw = wave % F::kOfRing, wk = wave / F::kOfRing, wm = lw / F::kWN, wn = lw % F::kWN;
  const int fr = lane & 31, fh = lane >> 5;
  // its steps: all, or those of the workgroup's part of the sum, and of its ring's part of that
  const int of_split = kPart ? (steps + a.splits - 1) / a.splits : steps, from = split * of_split;
  const int upto_step = from + of_split < steps ? from + of_split : steps;
  const int share = upto_step > from ? (upto_step - from + F::kK - 1) / F::kK : 0;
  const int first = from + wk * share, last = first + share < upto_step ? first + share : upto_step;
  char *ring = smem + wk * F::kRing;
  f32x16 acc[kI][2];

  // the tile at hand: its slots (none where the even deal left none), first
  // column, and the wave's 32-row blocks i kWM + wm that have slots
  int count = int(t.hi - t.lo);
  int n0 = t.n * (kGated ? kBN / 2 : kBN);
  auto blocks_of = [&](int count) {
    return __builtin_amdgcn_readfirstlane(count > 0 ? ((count + 31) / 32 - wm + F::kWM - 1) / F::kWM : 0);
  };
  int live = blocks_of(count);
  const T *w = static_cast<const T *>(a.w) + t.group * a.w_stride;
  const T *w2 = static_cast<const T *>(a.w2) + t.group * a.w2_stride;
  auto list = [&](const Tile &t, int which, int r, int v) __attribute__((always_inline)) {
    const bool in = t.lo + r < t.hi;
    table[(2 * which) * F::kBM + r] = in ? source_row(a, t.lo + r, v) : -1;
    table[(2 * which + 1) * F::kBM + r] = in ? out_row(a, t.lo + r, v) : -1;
  };

  const int fa = (wm * 32 + fr) * F::kRow, fb = F::kABytes + (wn * 64 + fr) * F::kRow, fx = swizzle<F>(fr);
  int tr[2] = {0, 0};
  if constexpr (kBack && kBf16) {
    // row 8 (lane / 32) + (lane % 16) / 4 (second read: four rows on), columns
    // 16 (lane / 16 % 2) + 4 (lane % 4) of a 32-column run
#pragma unroll
    for (int j = 0; j < 2; ++j)
      tr[j] = F::kABytes + tr_at<kBN>(8 * fh + ((lane & 15) >> 2), wn * 64 + 32 * j + 16 * ((lane >> 4) & 1) + 4 * (lane & 3));
  }
  auto read_x = [&](const char *stage, int kk, u32x4 (&f)[kI], auto blocks) {
    const int ch = ((kk * 2 + fh) ^ fx) << 4;
#pragma unroll
    for (int i = 0; i < decltype(blocks)::value; ++i)
      f[i] = *reinterpret_cast<const u32x4 *>(stage + fa + i * F::kWM * 32 * F::kRow + ch);
  };
  auto read_w = [&](const char *stage, int kk, u32x4 (&f)[2]) {
    if constexpr (!kBack) {
      const int ch = ((kk * 2 + fh) ^ fx) << 4;
#pragma unroll
      for (int j = 0; j < 2; ++j) f[j] = *reinterpret_cast<const u32x4 *>(stage + fb + j * 32 * F::kRow + ch);
    } else if constexpr (kBf16) {
      typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const char *p = stage + tr[j] + kk * 16 * kBN * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * kBN * 2));
        f[j] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[j][e] = *reinterpret_cast<const uint32_t *>(stage + F::kABytes + (kk * 8 + fh * 4 + e) * kBN * 4 +
                                                        (wn * 64 + 32 * j + fr) * 4);
    }
  };
  // Zeros where the sum has ended: the tile of a part's last step is loaded whole.
  auto cut = [&](int step, int kk, u32x4 (&x)[kI], u32x4 (&v)[2]) {
    const int at = (step >= each ? step - each : step) * kStep;
    if (at + kStep <= a.k) return;
    asm volatile("");  // a branch: no selects in the other steps
    if (at + (kk * 2 + fh) * kE >= a.k) {
#pragma unroll
      for (int i = 0; i < kI; ++i) x[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 2; ++j) v[j] = u32x4{0u, 0u, 0u, 0u};
    }
  };
  auto products = [&](const u32x4 (&x)[kI], const u32x4 (&v)[2], auto blocks) {
#pragma unroll
    for (int i = 0; i < decltype(blocks)::value; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) multiply(acc[i][j], x[i], v[j], T());
  };
  // f with the number of live blocks as a constant
  auto with_blocks = [&](int live, auto f) __attribute__((always_inline)) {
    if (live <= 0)
      f(std::integral_constant<int, 0>());
    else if (kI == 1 || live == 1)
      f(std::integral_constant<int, 1>());
    else if (live == 2)
      f(std::integral_constant<int, (kI < 2 ? kI : 2)>());
    else if (live == 3)
      f(std::integral_constant<int, (kI < 3 ? kI : 3)>());
    else
      f(std::integral_constant<int, kI>());
  };

  // The sums of the tile that was, out.
  auto store = [&](const Tile &t, int count, int n0, int live, int which) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      if (i >= live) break;
      __builtin_amdgcn_sched_barrier(0);  // one block's values at a time
      const int at = (i * F::kWM + wm) * 32 + fr;
      int from, to;
      if constexpr (F::kStream) {
        from = table[(2 * which) * F::kBM + at];
        to = table[(2 * which + 1) * F::kBM + at];
      } else {
        const int64_t s = t.lo + (at < count ? at : count - 1);
        const int v = a.gather || a.scatter ? entry(a, s) : 0;
        from = source_row(a, s, v);
        to = at < count ? out_row(a, s, v) : -1;
      }
      const bool there = from >= 0;
      if constexpr (kPart) {
        const int64_t slot = t.lo + (at < count ? at : count - 1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (F::kK > 1 && !kGated && j != wk) continue;
          const int c = n0 + (kGated ? 32 * wn : 64 * wn + 32 * j), wide = kGated ? 2 * a.n : a.n;
          float f[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) f[r] = acc[i][j][r];
          store_row(a.part + (split * a.slots + slot) * wide + (kGated ? j * a.n : 0) + c, f, fh, at < count ? a.n - c : 0);
        }
        continue;
      }
      // the swaps of store_row need both lanes of a row: a row that is not stored has no columns
      const int64_t row = to < 0 ? 0 : to;
      if constexpr (kGated) {
        const int c = n0 + 32 * wn, n = to < 0 ? 0 : a.n - c;
        float g[16], u[16], h[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          g[r] = there ? acc[i][0][r] : 0.f;
          u[r] = there ? acc[i][1][r] : 0.f;
          float slope;
          h[r] = act_value(g[r], a.act, slope) * u[r];
        }
        store_row(static_cast<T *>(a.out) + row * a.ld_out + c, h, fh, n);
        if (a.gate) store_row(static_cast<T *>(a.gate) + row * a.ld_gate + c, g, fh, n);
        if (a.up) store_row(static_cast<T *>(a.up) + row * a.ld_up + c, u, fh, n);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (F::kK > 1 && j != wk) continue;
          const int c = n0 + 64 * wn + 32 * j;
          float f[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) f[r] = there ? acc[i][j][r] : 0.f;
          store_row(static_cast<T *>(a.out) + row * a.ld_out + c, f, fh, to < 0 ? 0 : a.n - c);
        }
      }
    }
  };
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  };

  if constexpr (kDirect) {
    constexpr int kX = F::kX, kW = F::kW, kAhead = F::kStages - 1;
    const bool loader = lw < F::kLoaders;
    u32x4 rx, rx2, rw, rw2;
    uint32_t vx[kX], vw[kW];
    // load l of a stage: its row in this lane, and the chunk that belongs in the lane's place
    auto load_row = [&](int l) { return l * (64 / F::kChunks) + lane / F::kChunks; };
    auto chunk = [&](int l) { return (lane & (F::kChunks - 1)) ^ swizzle<F>(load_row(l)); };
    auto cx = [&](int l) { return uint32_t(chunk(l) * kE); };  // its first sum index within a step
    constexpr int kPlaces = kBN * int(sizeof(T)) / 16;  // chunks of a backward product's stage row
    auto stage_row = [&](int q) { return uint32_t(((lw * kW + q) * 64 + lane) / kPlaces); };
    auto cw = [&](int q) { return kBack ? stage_row(q) : cx(lw * kW + q); };
    // where the tile's loads are
    auto aim = [&](int which) __attribute__((always_inline)) {
      const T *xb = static_cast<const T *>(a.x), *xb2 = static_cast<const T *>(a.x2);
      if (!a.gather) {
        xb += t.lo * a.ld_x;
        if (kBack && a.x2) xb2 += t.lo * a.ld_x;
      }
      rx = whole(xb);
      rx2 = whole(kBack && a.x2 ? xb2 : xb);
      rw = whole(w);
      rw2 = whole(kGated || (kBack && a.x2) ? w2 : w);
      if (!loader || count <= 0) return;
#pragma unroll
      for (int q = 0; q < kX; ++q) {
        const int r = load_row(lw * kX + q);
        int row = r < count ? r : count - 1;
        if (a.gather) {
          row = F::kStream ? table[(2 * which) * F::kBM + row] : source_row(a, t.lo + row, entry(a, t.lo + row));
          row = row < 0 ? 0 : row;
        }
        vx[q] = uint32_t(row * a.ld_x * int64_t(sizeof(T))) + uint32_t(chunk(lw * kX + q) * 16);
      }
#pragma unroll
      for (int q = 0; q < kW; ++q) {
        if constexpr (!kBack) {
          const int r = load_row(lw * kW + q);
          int col = kGated ? n0 + (r >> 6) * 32 + (r & 31) : n0 + r;
          col = col < a.n ? col : a.n - 1;
          vw[q] = uint32_t(col * (kGated && (r & 32) ? a.ld_w2 : a.ld_w) * int64_t(sizeof(T))) + uint32_t(chunk(lw * kW + q) * 16);
        } else {
          const int r = int(stage_row(q)), in = ((lw * kW + q) * 64 + lane) % kPlaces;
          int col = kBf16 ? tr_run<kBN>(r, in >> 2) * 32 + (in & 3) * 8 : in * 4;
          col = n0 + col < a.n ? n0 + col : n0;
          vw[q] = uint32_t((r * a.ld_w + col) * int64_t(sizeof(T)));
        }
      }
    };
    const uint32_t lds = __builtin_amdgcn_readfirstlane(
        int(uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)smem)) + wk * F::kRing));
    auto load = [&](int step, uint32_t stage) __attribute__((always_inline)) {  // stage: where it begins in the ring
      if (!loader || count <= 0) return;
      const uint32_t st = lds + stage;
      const bool second = kBack && step >= each;
      const uint32_t at = uint32_t(second ? step - each : step) * kStep;
      const uint32_t sx = at * uint32_t(sizeof(T));
      const uint32_t sw = kBack ? uint32_t(at * a.ld_w * int64_t(sizeof(T))) : sx;
      uint32_t ox[kX], ow[kW];
#pragma unroll
      for (int q = 0; q < kX; ++q) ox[q] = vx[q];
#pragma unroll
      for (int q = 0; q < kW; ++q) ow[q] = vw[q];
      if (at + kStep > uint32_t(a.k)) {  // chunks past the sum's end: the step's first
        asm volatile("");
#pragma unroll
        for (int q = 0; q < kX; ++q) ox[q] -= at + cx(lw * kX + q) >= uint32_t(a.k) ? cx(lw * kX + q) * uint32_t(sizeof(T)) : 0;
#pragma unroll
        for (int q = 0; q < kW; ++q)
          ow[q] -= at + cw(q) >= uint32_t(a.k) ? cw(q) * uint32_t(sizeof(T)) * (kBack ? uint32_t(a.ld_w) : 1u) : 0;
      }
      const u32x4 xr = scalar(second ? rx2 : rx), wr = scalar(second ? rw2 : rw), wr2 = kGated ? scalar(rw2) : wr;
#pragma unroll
      for (int q = 0; q < kX; ++q) to_lds(xr, st + (lw * kX + q) * 1024, ox[q], sx);
#pragma unroll
      for (int q = 0; q < kW; ++q)  // a load's rows are of one of the gated block's products
        to_lds(kGated && ((lw * kW + q) * (64 / F::kChunks) & 32) ? wr2 : wr, st + F::kABytes + (lw * kW + q) * 1024, ow[q], sw);
    };
    // s_waitcnt with vmcnt alone constrained: where `n` more steps follow, the next one's loads may be under way
    auto landed = [&](int n) __attribute__((always_inline)) {
      constexpr int kL = kX + kW;
      static_assert(kAhead <= 2 && kL < 64 && kParts % 2 == 0);
      if (!loader) return;
      if (n >= 1 && kAhead > 1)
        __builtin_amdgcn_s_waitcnt((kL & 15) | (kL >> 4) << 14 | 0x0F70);
      else
        __builtin_amdgcn_s_waitcnt(0x0F70);
    };
    // Loads run kStages - 1 steps ahead of the products. At the top of step s
    // the loads of the steps behind it stay under way; after the barrier, which
    // every wave reaches with its reads of step s - 1 done, the stage of that
    // step takes step s + kStages - 1. A ring of one wave needs no barrier.
    auto sums = [&](auto blocks) __attribute__((always_inline)) {
      u32x4 xf[2][kI], wf[2][2];
      uint32_t here = 0, there = kAhead * F::kStage;  // the stages of step s and of the step that is loaded
#pragma unroll 1
      for (int s = first; s < (F::kOfRing > 1 ? first + share : last); ++s) {  // the rings' waves keep step
        landed(last - 1 - s);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        if constexpr (F::kOfRing > 1) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (F::kK > 1 && F::kOfRing > 1 && s >= last) continue;
        if (s + kAhead < last) load(s + kAhead, there);
        const char *st = ring + here;
        there = here;
        here = here == (F::kStages - 1) * F::kStage ? 0 : here + F::kStage;
        if constexpr (decltype(blocks)::value > 0) {
#pragma unroll
          for (int kk = 0; kk < kParts; ++kk) {
            read_x(st, kk, xf[kk & 1], blocks);
            read_w(st, kk, wf[kk & 1]);
            if (kk) cut(s, kk - 1, xf[~kk & 1], wf[~kk & 1]);
            if (kk || s > first) products(xf[~kk & 1], wf[~kk & 1], blocks);
          }
          cut(s, kParts - 1, xf[1], wf[1]);
        }
      }
      if constexpr (decltype(blocks)::value > 0)
        if (first < last) products(xf[1], wf[1], blocks);
    };
    if constexpr (F::kStream) {
      // The last half of the waves loads nothing to LDS: it looks up the rows of
      // the tile after this one, whose entries arrive beside the products.
      static_assert(F::kThreads / 2 == F::kBM && F::kLoaders * 64 == F::kThreads / 2);
      const int r = tid - F::kBM;
      if (r >= 0) list(t, 0, r, t.lo + r < t.hi ? entry(a, t.lo + r) : -1);
      __syncthreads();
      int was_n0 = 0, was_live = -1, which = 0;  // of the tile whose sums are to be stored (-1: none yet)
      for (;;) {
        const bool more = part.at < part.end;
        if (more) {
          n0 = t.n * (kGated ? kBN / 2 : kBN);
          count = int(t.hi - t.lo);
          live = blocks_of(count);
          w = static_cast<const T *>(a.w) + t.group * a.w_stride;
          w2 = static_cast<const T *>(a.w2) + t.group * a.w2_stride;
          aim(which);
          for (int s = 0; s < kAhead && s < steps; ++s) load(s, uint32_t(s * F::kStage));
        }
        if (was_live >= 0) store(t, 0, was_n0, was_live, which ^ 1);
        if (!more) return;
        part.at += gridDim.x >> 3;
        Tile next = t;
        int v = -1;
        if (part.at < part.end) {
          next = kept_tile(a, upto, part.at, F::kBM, lane);
          if (r >= 0 && next.lo + r < next.hi) v = entry(a, next.lo + r);
        }
        clear();
        with_blocks(live, sums);
        if (r >= 0) list(next, which ^ 1, r, v);
        __builtin_amdgcn_s_waitcnt(0xC07F);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        was_n0 = n0;
        was_live = live;
        t = next;
        which ^= 1;
      }
    } else {
      aim(0);
      for (int s = 0; s < kAhead && first + s < last; ++s) load(first + s, uint32_t(s * F::kStage));
      clear();
      with_blocks(live, sums);
    }
  } else {
    // Through registers: any alignment and width. A step is loaded kDeep steps
    // ahead in whole 16-byte chunks at whatever address, which stay inside the
    // operands but for a part's last step: that one goes by elements.
    constexpr int kRt = F::kOfRing * 64, kX = F::kABytes / 16 / kRt, kW = kBN * F::kRow / 16 / kRt, kDeep = kI == 1 ? 2 : 1;
    const int rt = tid % kRt;  // the ring's threads
    auto chunk = [&](int place) { return (place & (F::kChunks - 1)) ^ swizzle<F>(place / F::kChunks); };
    constexpr int kPlaces = kBN * int(sizeof(T)) / 16;  // of a backward product's stage row
    const T *px[kX], *px2[kX], *pw[kW], *pw2[kW];
    int cx[kX], cw[kW];  // the chunk's first sum index in a step
    int nw[kW];          // columns from the chunk on
#pragma unroll
    for (int q = 0; q < kX; ++q) {
      const int place = q * kRt + rt, r = place / F::kChunks;
      int64_t row = t.lo + (r < count ? r : count - 1);
      if (a.gather) row = source_row(a, row, entry(a, row));
      row = row < 0 ? 0 : row;
      cx[q] = chunk(place) * kE;
      px[q] = static_cast<const T *>(a.x) + row * a.ld_x + cx[q];
      px2[q] = kBack ? static_cast<const T *>(a.x2) + row * a.ld_x2 + cx[q] : nullptr;
    }
#pragma unroll
    for (int q = 0; q < kW; ++q) {
      const int place = q * kRt + rt;
      if constexpr (!kBack) {
        const int r = place / F::kChunks;
        int col = kGated ? n0 + (r >> 6) * 32 + (r & 31) : n0 + r;
        col = col < a.n ? col : a.n - 1;
        cw[q] = chunk(place) * kE;
        pw[q] = (kGated && (r & 32) ? w2 + col * a.ld_w2 : w + col * a.ld_w) + cw[q];
        pw2[q] = nullptr;
        nw[q] = 0;
      } else {
        const int in = place % kPlaces;
        int col = n0 + (kBf16 ? tr_run<kBN>(place / kPlaces, in >> 2) * 32 + (in & 3) * 8 : in * 4);
        col = col < a.n ? col : n0;
        cw[q] = place / kPlaces;
        pw[q] = w + cw[q] * a.ld_w + col;
        pw2[q] = w2 + cw[q] * a.ld_w2 + col;
        nw[q] = a.n - col;
      }
    }
    struct Held {
      u32x4 x[kX], w[kW];
    };
    // rows shorter than a chunk go by elements throughout
    const bool room = a.k >= kE && (!kBack || a.n >= kE);
    auto part_of_step = [&](int at, bool second, Held &h, auto has_room) __attribute__((always_inline)) {
      constexpr bool kRoom = decltype(has_room)::value;
#pragma unroll
      for (int q = 0; q < kX; ++q) h.x[q] = load_chunk<kRoom>((second ? px2[q] : px[q]) + at, a.k - at - cx[q]);
#pragma unroll
      for (int q = 0; q < kW; ++q) {
        if constexpr (!kBack) {
          h.w[q] = load_chunk<kRoom>(pw[q] + at, a.k - at - cw[q]);
        } else {  // rows past the sum's end: the last one's place, zeros
          const int past = at + cw[q] - (a.k - 1);
          const T *p = second ? pw2[q] + (at - (past > 0 ? past : 0)) * a.ld_w2 : pw[q] + (at - (past > 0 ? past : 0)) * a.ld_w;
          const u32x4 v = load_chunk<kRoom>(p, nw[q]);
          h.w[q] = past > 0 ? u32x4{0u, 0u, 0u, 0u} : v;
        }
      }
    };
    auto fetch = [&](int step, Held &h) __attribute__((always_inline)) {
      if (step >= last) return;
      const bool second = kBack && step >= each;
      const int at = (second ? step - each : step) * kStep;
      if (!room) {
        part_of_step(at, second, h, std::false_type());
      } else if (at + kStep >= a.k) {
        part_of_step(at, second, h, std::true_type());
      } else {
#pragma unroll
        for (int q = 0; q < kX; ++q) h.x[q] = load_whole((second ? px2[q] : px[q]) + at);
#pragma unroll
        for (int q = 0; q < kW; ++q) h.w[q] = load_whole(kBack ? (second ? pw2[q] + at * a.ld_w2 : pw[q] + at * a.ld_w) : pw[q] + at);
      }
    };
    clear();
    with_blocks(live, [&](auto blocks) __attribute__((always_inline)) {
      u32x4 xf[2][kI], wf[2][2];
      Held held[kDeep];
      // the stage that a step writes was last read two steps before, ahead of the barrier between
      auto pass = [&](int s, Held &h) __attribute__((always_inline)) {
        char *st = ring + ((s - first) & 1) * F::kStage;
#pragma unroll
        for (int q = 0; q < kX; ++q) *reinterpret_cast<u32x4 *>(st + (q * kRt + rt) * 16) = h.x[q];
#pragma unroll
        for (int q = 0; q < kW; ++q) *reinterpret_cast<u32x4 *>(st + F::kABytes + (q * kRt + rt) * 16) = h.w[q];
        fetch(s + kDeep, h);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (F::kK > 1 && s >= last) return;  // this part of the sum has fewer steps
        if constexpr (decltype(blocks)::value > 0) {
#pragma unroll
          for (int kk = 0; kk < kParts; ++kk) {
            read_x(st, kk, xf[kk & 1], blocks);
            read_w(st, kk, wf[kk & 1]);
            products(xf[kk & 1], wf[kk & 1], blocks);
          }
        }
      };
#pragma unroll
      for (int d = 0; d < kDeep; ++d) fetch(first + d, held[d]);
#pragma unroll 1
      for (int s = first; s < first + share; s += kDeep) {
        pass(s, held[0]);
        if constexpr (kDeep > 1)
          if (s + 1 < first + share) pass(s + 1, held[kDeep - 1]);
      }
    });
  }

  if constexpr (F::kK > 1) {
    // The waves of a sum add up through LDS: the first (of two 32-column outputs,
    // the first two, one each) takes the others' sums to its own, in order.
    __syncthreads();
    f32x4v *part = reinterpret_cast<f32x4v *>(smem);
    static_assert(kI == 1 && F::kWaves * 8192 <= F::kRing * F::kK);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        part[((wave * 2 + j) * 4 + g) * 64 + lane] =
            f32x4v{acc[0][j][4 * g], acc[0][j][4 * g + 1], acc[0][j][4 * g + 2], acc[0][j][4 * g + 3]};
    __syncthreads();
    if (wk >= (kGated ? 1 : 2)) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (!kGated && j != wk) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4v v = part[((lw * 2 + j) * 4 + g) * 64 + lane];
#pragma unroll
        for (int p = 1; p < F::kK; ++p) v += part[(((p * F::kOfRing + lw) * 2 + j) * 4 + g) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][j][4 * g + e] = v[e];
      }
    }
  }
  if constexpr (!F::kStream) store(t, count, n0, live, 0);
}

// Adds the parts of the sums in order and makes of them what the tiled kernel
// would have: a thread takes eight columns of a slot. Its launch is what it
// costs, 4-5 us.
template <typename T, bool kGated>
__global__ __launch_bounds__(256) void join_kernel(const ProductArgs a) {
  int64_t lo = 0, hi = a.slots;
  if (a.offsets) {
    lo = slot_bound(a, 0);
    hi = slot_bound(a, a.groups);
  }
  const int64_t runs = (a.n + 7) / 8, wide = kGated ? 2 * a.n : a.n, step = a.slots * wide;
  for (int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x; u < (hi - lo) * runs; u += int64_t(gridDim.x) * 256) {
    const int64_t s = lo + u / runs;
    const int c = int(u % runs) * 8, left = a.n - c;
    const float *p = a.part + s * wide + c;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = 0; i < a.splits; ++i) {
      const Raw8<float> r = load8(p + i * step, left);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += r.get(e);
      if constexpr (kGated) {
        const Raw8<float> q = load8(p + i * step + a.n, left);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] += q.get(e);
      }
    }
    const int v = a.gather || a.scatter ? entry(a, s) : 0;
    const bool there = source_row(a, s, v) >= 0;
    const int to = out_row(a, s, v);
    if (to < 0) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = there ? f[e] : 0.f;
    if constexpr (kGated) {
      float h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[e] = there ? g[e] : 0.f;
        float slope;
        h[e] = act_value(f[e], a.act, slope) * g[e];
      }
      store8(static_cast<T *>(a.out) + to * a.ld_out + c, pack8(h, T()), left);
      if (a.gate) store8(static_cast<T *>(a.gate) + to * a.ld_gate + c, pack8(f, T()), left);
      if (a.up) store8(static_cast<T *>(a.up) + to * a.ld_up + c, pack8(g, T()), left);
    } else {
      store8(static_cast<T *>(a.out) + to * a.ld_out + c, pack8(f, T()), left);
    }
  }
}

int64_t row_tiles(const ProductArgs &a, int rows) {  // at most: a group's last one may be a part of a tile
  return a.slots / rows + std::min<int64_t>(a.offsets ? a.groups : 1, a.slots);
}

template <typename T, class F, bool kDirect, bool kPart = false>
void tiled(ProductArgs a, hipStream_t s) {
  a.tiles_n = tiles_across(a, F::kBN);
  const int64_t most = 1 << 20;
  int64_t blocks = (row_tiles(a, F::kBM) * a.tiles_n * a.splits + 7) / 8 * 8;
  if (F::kStream) blocks = std::min<int64_t>(blocks, kCus);
  const dim3 grid(unsigned(std::min(blocks, most)), unsigned((blocks + most - 1) / most));
  auto kernel = a.back ? product_kernel<T, F, true, false, kDirect, kPart>
                : a.w2 ? product_kernel<T, F, false, true, kDirect, kPart> : product_kernel<T, F, false, false, kDirect, kPart>;
  hipLaunchKernelGGL(kernel, grid, dim3(F::kThreads), 0, s, a);
}

// Whether every operand can go to LDS in aligned 16-byte chunks with 32-bit offsets.
bool direct(const ProductArgs &a, int64_t size) {
  auto fits = [&](const void *p, int64_t rows, int64_t ld, int64_t cols) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && cols * size % 16 == 0 &&
           rows * ld * size < (int64_t(1) << 32) - 4096;
  };
  const int64_t x_rows = a.gather ? a.x_rows : std::min<int64_t>(a.slots, 512);
  const int64_t wr = a.back ? a.k : a.n, wc = a.back ? a.n : a.k;
  if (!fits(a.x, x_rows, a.ld_x, a.k) || !fits(a.w, wr, a.ld_w, wc) || a.w_stride * size % 16) return false;
  if (a.w2 && (!fits(a.w2, wr, a.ld_w2, wc) || a.w2_stride * size % 16)) return false;
  if (a.x2 && (!fits(a.x2, x_rows, a.ld_x2, a.k) || a.ld_x2 != a.ld_x || a.ld_w2 != a.ld_w)) return false;
  return true;
}

template <typename T>
hipError_t product(const ProductArgs &all, hipStream_t s) {
  ProductArgs a = all;
  const bool lds = direct(a, sizeof(T));
  if (a.whole) {
    a.splits = 1;
    a.n = a.whole;
  }
  if (a.splits == 1) {
    switch (product_form(a, sizeof(T) == 2, lds)) {
      case kLarge: lds ? tiled<T, Large, true>(a, s) : tiled<T, LargeAny, false>(a, s); break;
      case kWide: lds ? tiled<T, Wide, true>(a, s) : tiled<T, Wide, false>(a, s); break;
      case kSmall: lds ? tiled<T, Small, true>(a, s) : tiled<T, Small, false>(a, s); break;
      case kMid: lds ? tiled<T, Mid, true>(a, s) : tiled<T, Mid, false>(a, s); break;
      case kThin: lds ? tiled<T, Thin, true>(a, s) : tiled<T, Thin, false>(a, s); break;
      default:  // kThin2, which bf16 does not take
        if constexpr (sizeof(T) == 4) lds ? tiled<T, Thin2, true>(a, s) : tiled<T, Thin2, false>(a, s);
    }
  }
  if (all.splits == 1) return hipGetLastError();
  hipError_t e = a.whole ? hipGetLastError() : hipSuccess;
  if (e != hipSuccess) return e;
  // the columns behind the whole tiles, or all
  a = all;
  const int64_t from = a.whole;
  a.n -= int32_t(from);
  a.w = static_cast<const T *>(a.w) + from * (a.back ? 1 : a.ld_w);
  a.w2 = a.w2 ? static_cast<const T *>(a.w2) + from * (a.back ? 1 : a.ld_w2) : nullptr;
  a.out = static_cast<T *>(a.out) + from;
  a.gate = a.gate ? static_cast<T *>(a.gate) + from : nullptr;
  a.up = a.up ? static_cast<T *>(a.up) + from : nullptr;
  if (a.thin_parts)
    lds ? tiled<T, Thin2, true, true>(a, s) : tiled<T, Thin2, false, true>(a, s);
  else
    lds ? tiled<T, Mid, true, true>(a, s) : tiled<T, Mid, false, true>(a, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t blocks = std::min<int64_t>((a.slots * ((a.n + 7) / 8) + 255) / 256, 4096);
  auto kernel = a.w2 && !a.back ? join_kernel<T, true> : join_kernel<T, false>;
  hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// the gated block's gradients before its products
// ---------------------------------------------------------------------------

// dgate = dh up act'(gate), dup = dh act(gate): a thread takes eight columns.
// Both are rounded to the operands' type here, and dx sums products of what is
// stored: the weights' gradients take the same values, and the bf16 products
// have bf16 operands in any case (a relative error of dx of 2.3e-3, where one
// rounding of dx alone has 1.7e-3). A launch of its own, not part of the
// product's loads: a slot's run of n is needed by every column tile of k. HBM
// bounds it (131072 x 768 bf16: 165-178 us, 5.6-6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void gated_grad_kernel(const GatedGradArgs a, int per_row) {
  int64_t lo = 0, hi = a.slots;
  if (a.offsets) {
    lo = a.offsets[0] < 0 ? 0 : a.offsets[0];
    hi = a.offsets[a.groups] < hi ? a.offsets[a.groups] : hi;
  }
  const int64_t row0 = lo + int64_t(blockIdx.x) * (256 / per_row) + int(threadIdx.x) / per_row;
  for (int64_t row = row0; row < hi; row += int64_t(gridDim.x) * (256 / per_row))
  for (int c = (int(threadIdx.x) % per_row + int(blockIdx.y) * per_row) * 8; c < a.n; c += int(gridDim.y) * per_row * 8) {
    const Raw8<T> dh = load8(static_cast<const T *>(a.dh) + row * a.ld_dh + c, a.n - c);
    const Raw8<T> g = load8(static_cast<const T *>(a.gate) + row * a.ld_gate + c, a.n - c);
    const Raw8<T> u = load8(static_cast<const T *>(a.up) + row * a.ld_up + c, a.n - c);
    float dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float slope;
      const float v = act_value(g.get(e), a.act, slope);
      dg[e] = dh.get(e) * u.get(e) * slope;
      du[e] = dh.get(e) * v;
    }
    store8(static_cast<T *>(a.dgate) + row * a.ld_dgate + c, pack8(dg, T()), a.n - c);
    store8(static_cast<T *>(a.dup) + row * a.ld_dup + c, pack8(du, T()), a.n - c);
  }
}

template <typename T>
hipError_t gated_grad(const GatedGradArgs &a, hipStream_t s) {
  int per_row = 8;
  while (per_row < 256 && per_row * 8 < a.n) per_row *= 2;
  const int rows = 256 / per_row;
  const int64_t blocks = std::min<int64_t>((a.slots + rows - 1) / rows, 1 << 20);
  const int across = std::min((a.n + per_row * 8 - 1) / (per_row * 8), 64);
  hipLaunchKernelGGL(gated_grad_kernel<T>, dim3(unsigned(blocks), unsigned(across)), dim3(256), 0, s, a, per_row);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product(const ProductArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? product<__bf16>(a, s) : product<float>(a, s);
}

hipError_t launch_gated_grad(const GatedGradArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? gated_grad<__bf16>(a, s) : gated_grad<float>(a, s);
}

}  // namespace muon
