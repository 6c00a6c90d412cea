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
// v_mfma_f32_32x32x2_f32 (float32 products and sums; the four 16-byte values of
// a fragment are four products): the same bytes in LDS, the same reads.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kRowBytes = 64;      // of a step in LDS: 32 bf16 or 16 float32 of the sum's index
constexpr int kTileN = 256;        // columns of a tile (gated: 128 of each product)
constexpr int kBand = 8;           // tiles of a group that take turns within one column of tiles
constexpr int kOutPitch = 64 + 4;  // floats; epilogue rows of a wave

// kWM x 4 waves of 128 x 64. One wave row: 72 KiB of LDS, two workgroups a CU.
// Two: one workgroup a CU, which reads each operand half as often from L2.
template <int kWM>
struct Form {
  static constexpr int kThreads = kWM * 256;
  static constexpr int kBM = kWM * 128;
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kStage = kABytes + kTileN * kRowBytes;
  static constexpr int kStages = kWM == 1 ? 3 : 5;
};

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

// The slots of a group, cut to what there is.
__device__ inline void group_slots(const ProductArgs &a, int g, int &lo, int &hi) {
  lo = g < a.groups ? a.offsets[g] : 0;
  hi = g < a.groups ? a.offsets[g + 1] : 0;
  lo = lo < 0 ? 0 : lo;
  hi = hi > int(a.slots) ? int(a.slots) : hi;
}

// The tile of this workgroup, of rows x tiles_n tiles of `rows` slots. The
// tiles of a group lie in bands of kBand row tiles; every eighth workgroup runs
// on one XCD, which gets a contiguous part of them.
__device__ inline Tile find_tile(const ProductArgs &a, int rows, int lane) {
  const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
  Tile t{-1, 0, 0, 0};
  uint32_t total;  // row tiles
  if (a.offsets) {
    int sum = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
      int lo, hi;
      group_slots(a, g0 + lane, lo, hi);
      sum += hi > lo ? (hi - lo + rows - 1) / rows : 0;
    }
    total = uint32_t(__builtin_amdgcn_readlane(wave_scan(sum, lane), 63));
  } else {
    total = uint32_t((a.slots + rows - 1) / rows);
  }
  const uint32_t tiles = total * uint32_t(a.tiles_n), per = (tiles + 7) / 8;
  const uint32_t id = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || id >= tiles) return t;
  const uint32_t row = id / uint32_t(a.tiles_n);  // in which group's tiles
  uint32_t first = 0, count = total;              // its row tiles
  int64_t lo = 0, hi = a.slots;
  t.group = 0;
  if (a.offsets) {
    uint32_t before = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
      int glo, ghi;
      group_slots(a, g0 + lane, glo, ghi);
      const int mine = ghi > glo ? (ghi - glo + rows - 1) / rows : 0;
      const uint32_t upto = before + uint32_t(wave_scan(mine, lane));
      const uint64_t past = __ballot(upto > row);
      if (past) {
        const int at = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
        t.group = g0 + at;
        count = uint32_t(__builtin_amdgcn_readlane(mine, at));
        first = uint32_t(__builtin_amdgcn_readlane(int(upto), at)) - count;
        lo = __builtin_amdgcn_readlane(glo, at);
        hi = __builtin_amdgcn_readlane(ghi, at);
        break;
      }
      before = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
    }
  }
  const uint32_t local = id - first * uint32_t(a.tiles_n);
  const uint32_t band = local / (kBand * uint32_t(a.tiles_n)), in = local - band * kBand * uint32_t(a.tiles_n);
  const uint32_t wide = count - band * kBand < kBand ? count - band * kBand : kBand;
  t.n = __builtin_amdgcn_readfirstlane(int(in / wide));
  const int m = __builtin_amdgcn_readfirstlane(int(band * kBand + in % wide));
  t.lo = lo + int64_t(m) * rows;
  t.hi = t.lo + rows < hi ? t.lo + rows : hi;
  return t;
}

// The row of x that slot s reads, -1: none.
__device__ inline int64_t source_row(const ProductArgs &a, int64_t s) {
  int64_t r = s;
  if (a.gather) {
    const int32_t v = a.rows ? a.rows[s] : int32_t(s);
    if (v < 0) return -1;
    r = a.gather == 1 ? v : int32_t(uint32_t(v) / uint32_t(a.gather));
  }
  return r < a.x_rows ? r : -1;
}

// ---------------------------------------------------------------------------
// the tiled kernel
// ---------------------------------------------------------------------------

// 16 bytes of a fragment: eight bf16 or four float32 of the sum's index.
__device__ inline void multiply(f32x16 &acc, const u32x4 &x, const u32x4 &w, __bf16) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), acc, 0, 0, 0);
}
__device__ inline void multiply(f32x16 &acc, const u32x4 &x, const u32x4 &w, float) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bits_f32(x[e]), bits_f32(w[e]), acc, 0, 0, 0);
}

// The first min(n, 16 / sizeof(T)) elements at p, zeros behind them.
template <typename T>
__device__ inline u32x4 load_chunk(const T *p, int n) {
  constexpr int kE = 16 / int(sizeof(T));
  if (n >= kE) return *reinterpret_cast<const u32x4_any *>(p);
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

__device__ inline __amdgpu_buffer_rsrc_t whole(const void *p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, -1, 0x00020000);
}
__device__ inline void to_lds(__amdgpu_buffer_rsrc_t r, char *lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, voff, soff, 0, 0);
}

// Where column col of row r of a backward product's weight tile lies in its
// stage (bf16): rows of 256 columns in runs of 32, run i of row r at place
// i ^ (r & 3) within its four, so that a transposing read, 32 columns of four
// consecutive rows, takes four different quarters of the banks.
__device__ inline int tr_at(int row, int col) {
  const int run = col >> 5;
  return row * (kTileN * 2) + (((run & ~3) | ((run ^ row) & 3)) << 6) + (col & 31) * 2;
}

// kDirect: 16-byte loads straight to LDS. Needs operands whose rows start on
// 16-byte boundaries, whole chunks in each row, and byte offsets below 2^32.
template <typename T, int kWM, bool kBack, bool kGated, bool kDirect>
__global__ __launch_bounds__(kWM * 256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void product_kernel(const ProductArgs a) {
  using F = Form<kWM>;
  constexpr int kE = 16 / int(sizeof(T));            // elements of a chunk
  constexpr int kStep = kRowBytes / int(sizeof(T));  // sum indices of a step
  constexpr bool kBf16 = sizeof(T) == 2;
  __shared__ __attribute__((aligned(1024))) char smem[F::kStages * F::kStage];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Tile t = find_tile(a, F::kBM, lane);
  if (t.group < 0) return;
  const int count = int(t.hi - t.lo);  // slots of the tile
  const int n0 = t.n * (kGated ? kTileN / 2 : kTileN);
  const T *w = static_cast<const T *>(a.w) + t.group * a.w_stride;
  const T *w2 = static_cast<const T *>(a.w2) + t.group * a.w2_stride;

  const int each = (a.k + kStep - 1) / kStep;  // steps of a part
  const int steps = kBack && a.x2 ? 2 * each : each;

  const int wm = kWM == 1 ? 0 : wave >> 2, wn = wave & 3;
  const int fr = lane & 31, fh = lane >> 5;
  f32x16 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // fragments: 64-byte rows of four chunks, chunk c at place c ^ (row >> 2 & 3)
  const int fa = (wm * 128 + fr) * kRowBytes, fb = F::kABytes + (wn * 64 + fr) * kRowBytes, fx = (fr >> 2) & 3;
  int tr[2] = {0, 0};
  if constexpr (kBack && kBf16) {
    // row 8 (lane / 32) + (lane % 16) / 4 (second read: four rows on), columns
    // 16 (lane / 16 % 2) + 4 (lane % 4) of a 32-column run
#pragma unroll
    for (int j = 0; j < 2; ++j)
      tr[j] = F::kABytes + tr_at(8 * fh + ((lane & 15) >> 2), wn * 64 + 32 * j + 16 * ((lane >> 4) & 1) + 4 * (lane & 3));
  }
  auto read_x = [&](const char *stage, int kk, u32x4 (&f)[4]) {
    const int ch = ((kk * 2 + fh) ^ fx) << 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const u32x4 *>(stage + fa + i * 32 * kRowBytes + ch);
  };
  auto read_w = [&](const char *stage, int kk, u32x4 (&f)[2]) {
    if constexpr (!kBack) {
      const int ch = ((kk * 2 + fh) ^ fx) << 4;
#pragma unroll
      for (int j = 0; j < 2; ++j) f[j] = *reinterpret_cast<const u32x4 *>(stage + fb + j * 32 * kRowBytes + ch);
    } else if constexpr (kBf16) {
      typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const char *p = stage + tr[j] + kk * 16 * kTileN * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * kTileN * 2));
        f[j] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[j][e] = *reinterpret_cast<const uint32_t *>(stage + F::kABytes + (kk * 8 + fh * 4 + e) * kTileN * 4 +
                                                        (wn * 64 + 32 * j + fr) * 4);
    }
  };
  // Zeros where the sum has ended: the tile of a part's last step is loaded whole.
  auto cut = [&](int step, int kk, u32x4 (&x)[4], u32x4 (&v)[2]) {
    const int at = (step >= each ? step - each : step) * kStep;
    if (at + kStep <= a.k) return;
    if (at + (kk * 2 + fh) * kE >= a.k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 2; ++j) v[j] = u32x4{0u, 0u, 0u, 0u};
    }
  };
  auto products = [&](const u32x4 (&x)[4], const u32x4 (&v)[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) multiply(acc[i][j], x[i], v[j], T());
  };
  u32x4 xf[2][4], wf[2][2];

  if (steps > 0) {
    if constexpr (kDirect) {
      // Waves 0..3 load: 2 kWM KiB of x and 4 KiB of the weights each, a KiB an instruction.
      constexpr int kX = 2 * kWM;
      const bool loader = wave < 4;
      const T *xb = static_cast<const T *>(a.x), *xb2 = static_cast<const T *>(a.x2);
      if (!a.gather) {
        xb += t.lo * a.ld_x;
        if (kBack && a.x2) xb2 += t.lo * a.ld_x;
      }
      const __amdgpu_buffer_rsrc_t rx = whole(xb), rx2 = whole(kBack && a.x2 ? xb2 : xb);
      const __amdgpu_buffer_rsrc_t rw = whole(w), rw2 = whole(kGated || (kBack && a.x2) ? w2 : w);
      uint32_t vx[kX], vw[4];
      uint32_t cx[kX], cw[4];  // the chunk's first sum index within a step
      if (loader) {
#pragma unroll
        for (int q = 0; q < kX; ++q) {
          const int r = (wave * kX + q) * 16 + (lane >> 2);
          const int c = (lane & 3) ^ ((r >> 2) & 3);
          int64_t row = r < count ? r : count - 1;
          if (a.gather) {
            row = source_row(a, t.lo + row);
            row = row < 0 ? 0 : row;
          }
          cx[q] = uint32_t(c * kE);
          vx[q] = uint32_t(row * a.ld_x * int64_t(sizeof(T))) + uint32_t(c * 16);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (!kBack) {
            const int r = (wave * 4 + q) * 16 + (lane >> 2);
            const int c = (lane & 3) ^ ((r >> 2) & 3);
            int col = kGated ? n0 + 32 * wave + (q & 1) * 16 + (lane >> 2) : n0 + r;
            col = col < a.n ? col : a.n - 1;
            cw[q] = uint32_t(c * kE);
            vw[q] = uint32_t(col * (kGated && q >= 2 ? a.ld_w2 : a.ld_w) * int64_t(sizeof(T))) + uint32_t(c * 16);
          } else {
            const int place = (wave * 4 + q) * 64 + lane;  // 16-byte places of the stage
            int r, col;
            if constexpr (kBf16) {
              r = place >> 5;
              const int run = (place & 31) >> 2;
              col = ((run & ~3) | ((run ^ r) & 3)) * 32 + (place & 3) * 8;
            } else {
              r = place >> 6;
              col = (place & 63) * 4;
            }
            col = n0 + col < a.n ? n0 + col : n0;
            cw[q] = uint32_t(r);
            vw[q] = uint32_t((r * a.ld_w + col) * int64_t(sizeof(T)));
          }
        }
      }
      auto load = [&](int step) {
        if (!loader) return;
        char *st = smem + (step % F::kStages) * F::kStage;
        const bool second = kBack && step >= each;
        const uint32_t at = uint32_t(second ? step - each : step) * kStep;
        const uint32_t sx = at * uint32_t(sizeof(T));
        const uint32_t sw = kBack ? uint32_t(at * a.ld_w * int64_t(sizeof(T))) : sx;
        uint32_t ox[kX], ow[4];
#pragma unroll
        for (int q = 0; q < kX; ++q) ox[q] = vx[q];
#pragma unroll
        for (int q = 0; q < 4; ++q) ow[q] = vw[q];
        if (at + kStep > uint32_t(a.k)) {  // chunks past the sum's end: the step's first
#pragma unroll
          for (int q = 0; q < kX; ++q) ox[q] -= at + cx[q] >= uint32_t(a.k) ? cx[q] * uint32_t(sizeof(T)) : 0;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            ow[q] -= at + cw[q] >= uint32_t(a.k) ? cw[q] * uint32_t(sizeof(T)) * (kBack ? uint32_t(a.ld_w) : 1u) : 0;
        }
#pragma unroll
        for (int q = 0; q < kX; ++q) to_lds(second ? rx2 : rx, st + (wave * kX + q) * 1024, ox[q], sx);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          to_lds(second || (kGated && q >= 2) ? rw2 : rw, st + F::kABytes + (wave * 4 + q) * 1024, ow[q], sw);
      };
      // s_waitcnt with vmcnt alone constrained: the loads of `n` steps may be under way
      auto landed = [&](int n) {
        constexpr int kL = kX + 4;
        if (!loader) return;
        if (n >= 3)
          __builtin_amdgcn_s_waitcnt((3 * kL & 15) | (3 * kL >> 4) << 14 | 0x0F70);
        else if (n == 2)
          __builtin_amdgcn_s_waitcnt((2 * kL & 15) | (2 * kL >> 4) << 14 | 0x0F70);
        else if (n == 1)
          __builtin_amdgcn_s_waitcnt((kL & 15) | (kL >> 4) << 14 | 0x0F70);
        else
          __builtin_amdgcn_s_waitcnt(0x0F70);
      };
      // Loads run kStages - 1 steps ahead of the products. At the top of step s
      // the loads of the steps behind it stay under way; after the barrier, which
      // every wave reaches with its reads of step s - 1 done, the stage of that
      // step takes step s + kStages - 1.
      constexpr int kAhead = F::kStages - 1;
      for (int s = 0; s < kAhead && s < steps; ++s) load(s);
#pragma unroll 1
      for (int s = 0; s < steps; ++s) {
        const int behind = steps - 1 - s;
        if (behind >= kAhead - 1)
          landed(kAhead - 1);
        else if (kAhead > 2 && behind == 2)
          landed(2);
        else if (behind == 1)
          landed(1);
        else
          landed(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (s + kAhead < steps) load(s + kAhead);
        const char *st = smem + (s % F::kStages) * F::kStage;
        read_x(st, 0, xf[0]);
        read_w(st, 0, wf[0]);
        if (s) products(xf[1], wf[1]);
        read_x(st, 1, xf[1]);
        read_w(st, 1, wf[1]);
        cut(s, 0, xf[0], wf[0]);
        products(xf[0], wf[0]);
        cut(s, 1, xf[1], wf[1]);
      }
      products(xf[1], wf[1]);
    } else {
      // Through registers: any alignment and width.
      constexpr int kX = F::kBM * 4 / F::kThreads, kW = 1024 / F::kThreads;
      const T *px[kX], *px2[kX];
      int cx[kX];
#pragma unroll
      for (int q = 0; q < kX; ++q) {
        const int place = q * F::kThreads + tid, r = place >> 2;
        int64_t row = t.lo + (r < count ? r : count - 1);
        if (a.gather) row = source_row(a, row);
        row = row < 0 ? 0 : row;
        cx[q] = ((place & 3) ^ ((r >> 2) & 3)) * kE;
        px[q] = static_cast<const T *>(a.x) + row * a.ld_x + cx[q];
        px2[q] = kBack ? static_cast<const T *>(a.x2) + row * a.ld_x2 + cx[q] : nullptr;
      }
      u32x4 hx[kX], hw[kW];
      auto fetch = [&](int step) {
        const bool second = kBack && step >= each;
        const int at = (second ? step - each : step) * kStep;
#pragma unroll
        for (int q = 0; q < kX; ++q) hx[q] = load_chunk((second ? px2[q] : px[q]) + at, a.k - at - cx[q]);
#pragma unroll
        for (int q = 0; q < kW; ++q) {
          const int place = q * F::kThreads + tid;
          if constexpr (!kBack) {
            const int r = place >> 2, c = ((place & 3) ^ ((r >> 2) & 3)) * kE;
            const bool up = kGated && (r >> 5 & 1);
            const int col = kGated ? n0 + 32 * (r >> 6) + (r & 31) : n0 + r;
            const T *p = up ? w2 + col * a.ld_w2 : w + col * a.ld_w;
            hw[q] = load_chunk(p + at + c, col < a.n ? a.k - at - c : 0);
          } else {
            const int r = kBf16 ? place >> 5 : place >> 6;
            const int run = (place & 31) >> 2;
            const int col = n0 + (kBf16 ? ((run & ~3) | ((run ^ r) & 3)) * 32 + (place & 3) * 8 : (place & 63) * 4);
            const T *p = second ? w2 + (at + r) * a.ld_w2 : w + (at + r) * a.ld_w;
            hw[q] = load_chunk(p + col, at + r < a.k ? a.n - col : 0);
          }
        }
      };
      fetch(0);
#pragma unroll 1
      for (int s = 0; s < steps; ++s) {
        char *st = smem + (s & 1) * F::kStage;
#pragma unroll
        for (int q = 0; q < kX; ++q) *reinterpret_cast<u32x4 *>(st + (q * F::kThreads + tid) * 16) = hx[q];
#pragma unroll
        for (int q = 0; q < kW; ++q) *reinterpret_cast<u32x4 *>(st + F::kABytes + (q * F::kThreads + tid) * 16) = hw[q];
        __syncthreads();
        if (s + 1 < steps) fetch(s + 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          read_x(st, kk, xf[kk]);
          read_w(st, kk, wf[kk]);
          products(xf[kk], wf[kk]);
        }
      }
    }
  }

  // Epilogue: 32 rows of the wave's 64 columns at a time through LDS, so that
  // a row leaves in runs of eight columns. Accumulator r of a lane is row
  // 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32.
  __syncthreads();
  float *buf = reinterpret_cast<float *>(smem) + wave * 32 * kOutPitch;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        buf[(8 * (r >> 2) + 4 * fh + (r & 3)) * kOutPitch + 32 * j + fr] = acc[i][j][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int kRuns = kGated ? 4 : 8;  // of eight columns in a row
#pragma unroll
    for (int q = 0; q < kRuns / 2; ++q) {
      const int row = (q * 64 + lane) / kRuns, col = (lane & (kRuns - 1)) * 8;
      const int at = wm * 128 + i * 32 + row;
      const int c = n0 + (kGated ? 32 : 64) * wn + col;
      if (at >= count || c >= a.n) continue;
      const int64_t s = t.lo + at;
      const bool there = source_row(a, s) >= 0;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = there ? buf[row * kOutPitch + col + e] : 0.f;
      if constexpr (kGated) {
        float u[8], h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] = there ? buf[row * kOutPitch + 32 + col + e] : 0.f;
          float slope;
          h[e] = act_value(f[e], a.act, slope) * u[e];
        }
        store8(static_cast<T *>(a.out) + s * a.ld_out + c, pack8(h, T()), a.n - c);
        if (a.gate) store8(static_cast<T *>(a.gate) + s * a.ld_gate + c, pack8(f, T()), a.n - c);
        if (a.up) store8(static_cast<T *>(a.up) + s * a.ld_up + c, pack8(u, T()), a.n - c);
      } else {
        const int64_t to = a.scatter ? a.rows[s] : s;
        if (to >= 0 && to < a.out_rows) store8(static_cast<T *>(a.out) + to * a.ld_out + c, pack8(f, T()), a.n - c);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, int kWM, bool kDirect>
void tiled(ProductArgs a, hipStream_t s) {
  using F = Form<kWM>;
  const int wide = a.w2 && !a.back ? kTileN / 2 : kTileN;
  a.tiles_n = int32_t((a.n + wide - 1) / wide);
  // a group's last tile may be a part of one
  const int64_t rows = a.slots / F::kBM + std::min<int64_t>(a.offsets ? a.groups : 1, a.slots);
  const int64_t most = 1 << 20, blocks = (rows * a.tiles_n + 7) / 8 * 8;
  const dim3 grid(unsigned(std::min(blocks, most)), unsigned((blocks + most - 1) / most));
  auto kernel = a.back ? product_kernel<T, kWM, true, false, kDirect>
                : a.w2 ? product_kernel<T, kWM, false, true, kDirect> : product_kernel<T, kWM, false, false, kDirect>;
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
hipError_t product(const ProductArgs &a, hipStream_t s) {
  if (!direct(a, sizeof(T)))
    tiled<T, 1, false>(a, s);
  else if (a.slots >= 1024 * int64_t(a.offsets ? a.groups : 1))
    tiled<T, 2, true>(a, s);
  else
    tiled<T, 1, true>(a, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// the gated block's gradients before its products
// ---------------------------------------------------------------------------

// dgate = dh up act'(gate), dup = dh act(gate): a thread takes eight columns.
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
