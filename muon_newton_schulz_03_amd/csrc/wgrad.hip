// Weight gradients of expert layers from 8-bit checkpoints (gfx950):
//   dW_g[n, k] = sum over the slots s of group g of dy[s, n] X[token(s), k],
// X the values of a checkpoint (codes times a power of two per 128 columns),
// token(s) = rows[s] / per_token.
//
// The sum runs over rows of both operands as they lie in memory (n and k
// contiguous), so both reach the matrix cores transposed: tiles go to LDS
// row by row and the fragments come back through the transposing LDS reads.
// The codes turn into bf16 on their way into LDS, one conversion that
// multiplies by the scale for two values: exact, since a value has four
// significant bits. bf16 gradients make one product. A float32 gradient is cut
// into three bf16 parts of eight significant bits each (by truncation, so
// that they add up to it exactly), three products with the same X: the sum is
// that of float32 products, at a third of the bf16 rate.
//
// Sums are float32 in the accumulators; the result is rounded once. Long sums
// with few tiles are split into `splits` runs whose float32 partials a second
// launch adds in order.
//
// A workgroup makes a 128 x 256 tile of the result in steps of 32 slots, which
// go through two LDS stages. Dense, 8192 slots into 2048x7168 bf16, it runs at
// 245 us (980 TFLOP/s) against the socket's power cap (1399 W, 2.1 GHz; a
// gradient of zeros, which toggles less, takes 226 us at 2.4 GHz): dealing loads,
// conversions and LDS traffic out between the products lost 10%, and tiles
// ordered by XCD changed nothing. float32, 16384 slots into 512x2048: 113 us, 912
// TFLOP/s of bf16 products. Many short groups, 128 of 256 slots into 768x2048:
// 195 to 215 us; the same tiles with one step each (128 groups of 32 slots) take 112,
// so that little of their first loads and last stores (403 MB of gradients, 81 us at
// 5 TB/s) runs beside products. float32, 128 groups of 32 slots: 398 us.
//
// The parts of a float32 gradient go down to 2^-133, bf16's smallest: what lies
// below in a gradient under 2^-110 is lost, and a value of X that became an infinity
// (2^128) times a part that is 0 is NaN.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBM = 128;       // tile rows (n)
constexpr int kBN = 256;       // tile columns (k)
constexpr int kBK = 32;        // slots a step
constexpr int kABytes = kBK * kBM * 2;
constexpr int kXBytes = kBK * kBN * 2;
// slot / per_token for slots below 2^31, as the high half of 2 slot * mul
// shifted down; `end`: the first slot whose token lies outside x.
struct TokenOf {
  uint32_t mul, shift, end;
};
constexpr int kOrderGroups = 512;  // more groups run in the given order
constexpr int kOutPitch = 64 + 4;  // floats; epilogue rows of a wave

template <bool kF32>
constexpr int stage_bytes() {
  return (kF32 ? 3 : 1) * kABytes + kXBytes;
}

// LDS rows hold one slot: 128 (dy) or 256 (X) bf16 in runs of 32 columns (64
// bytes), run i of row t at place i ^ (t & 3) within its four. A transposing
// read takes 32 columns of four consecutive rows: four different quarters of
// the 256-byte bank row.
// Two forms of a tile's workgroup. Four waves of 128 x 64 each read the least
// from LDS and hold two steps' loads; two workgroups fill a CU's registers.
// Eight waves of 64 x 64 hold one step's loads and one group's fragments, and
// twice as many waves hide what short groups mostly wait for: the first loads
// and the last stores of a tile.
template <int kWaves>
struct Form {
  static constexpr int kThreads = kWaves * 64;
  static constexpr int kI = kWaves == 4 ? 4 : 2;        // 32-row runs of a wave's part
  static constexpr int kR = kBK * 16 / kThreads;        // rows of a step that a thread stages
  static constexpr int kAhead = kWaves == 4 ? 1 : 0;    // groups whose fragments are read ahead
};

__device__ inline int lds_at(int row, int col, int pitch) {
  const int run = col >> 5;
  return row * pitch + (((run & ~3) | ((run ^ row) & 3)) << 6) + (col & 31) * 2;
}

struct Split3 {
  uint32_t hi, mid, lo;  // packed pairs of bf16
};
// Three bf16 parts of two floats that add up to them: eight bits each, cut
// off. An infinity or NaN is its own first part.
__device__ inline void cut3(float f, uint32_t &h, uint32_t &m, uint32_t &l) {
  const uint32_t u = f32_bits(f);
  h = u & 0xffff0000u;
  const bool special = (u & 0x7f800000u) == 0x7f800000u;
  if (special && (u & 0x007fffffu)) h |= 0x00400000u;  // NaN stays NaN
  const float r = special ? 0.f : f - bits_f32(h);
  m = f32_bits(r) & 0xffff0000u;
  l = f32_bits(r - bits_f32(m));
}
__device__ inline Split3 split3(float a, float b) {
  uint32_t h0, m0, l0, h1, m1, l1;
  cut3(a, h0, m0, l0);
  cut3(b, h1, m1, l1);
  return {h0 >> 16 | h1, m0 >> 16 | m1, l0 >> 16 | (l1 & 0xffff0000u)};
}

// Global memory, said so: the compiler then counts these loads apart from LDS
// traffic.
typedef const __attribute__((address_space(1))) char *GlobalPtr;
__device__ inline u32x4 load16(GlobalPtr p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) u32x4_any *>(p);
}

__device__ inline void store8_stream(__bf16 *p, const Raw8<__bf16> &r) {
  __builtin_nontemporal_store(r.v, reinterpret_cast<u32x4_any *>(p));
}
__device__ inline void store8_stream(float *p, const Raw8<float> &r) {
  __builtin_nontemporal_store(r.v[0], reinterpret_cast<u32x4_any *>(p));
  __builtin_nontemporal_store(r.v[1], reinterpret_cast<u32x4_any *>(p + 4));
}

// Moves a run down by `bytes` (zeros behind it).
template <int kDwords>
__device__ inline void shift_down(uint32_t (&v)[kDwords], uint32_t bytes) {
#pragma unroll
  for (int d = kDwords / 2; d >= 1; d /= 2)
    if (bytes & (4 * d)) {
#pragma unroll
      for (int i = 0; i < kDwords; ++i) v[i] = i + d < kDwords ? v[i + d] : 0u;
    }
#pragma unroll
  for (int i = 0; i < kDwords; ++i) v[i] = __builtin_amdgcn_alignbyte(i + 1 < kDwords ? v[i + 1] : 0u, v[i], bytes & 3);
}

__device__ inline uint32_t raw_word(const Raw8<__bf16> &r, int i) { return r.v[i]; }
__device__ inline uint32_t raw_word(const Raw8<float> &r, int i) { return r.v[i >> 2][i & 3]; }
__device__ inline void raw_word(Raw8<__bf16> &r, int i, uint32_t w) { r.v[i] = w; }
__device__ inline void raw_word(Raw8<float> &r, int i, uint32_t w) { r.v[i >> 2][i & 3] = w; }

// What a thread holds of a step on its way to LDS: its rows' runs of 8
// gradients, and their runs of 16 codes with their scales.
template <typename T, int kR>
struct Staged {
  Raw8<T> dy[kR];
  u32x4 codes[kR];
  uint32_t scale[kR];
  // bit r: row r adds nothing (past the group's end, or no such token); from
  // bit 4 + 4 r and 16 + 8 r: by how many bytes the run of row r was read too
  // early (codes, gradients), so as not to pass the buffer's end
  uint32_t fix;
};

__device__ inline void group_range(const WgradArgs &a, int group, int64_t &lo, int64_t &hi) {
  lo = a.offsets[group];
  hi = a.offsets[group + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi > a.slots ? a.slots : hi;
}

// The groups and their slots, the longest first (the lower index among
// equals). Long groups started last would leave most of the chip idle: 16 groups
// of 2048 slots on average, 768x2048 bf16, take 159 us in the given order and 135 in
// this one, 64 of 512 slots, 768x768 float32, 193 and 157.
__global__ __launch_bounds__(kOrderGroups) void wgrad_order_kernel(const WgradArgs a) {
  __shared__ int len[kOrderGroups];
  const int g = int(threadIdx.x);
  int64_t lo = 0, hi = 0;
  if (g < a.groups) group_range(a, g, lo, hi);
  const int mine = hi > lo ? int(hi - lo) : 0;
  len[g] = mine;
  __syncthreads();
  if (g >= a.groups) return;
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < a.groups; ++i) rank += len[i] > mine || (len[i] == mine && i < g) ? 1 : 0;
  a.order[rank] = int4{g, int(lo), int(hi), 0};
}

template <typename T, int kWaves, bool kRows, bool kPartial>
__global__ __launch_bounds__(kWaves * 64, kWaves / 2) void wgrad_kernel(const WgradArgs a, const TokenOf div) {
  using F = Form<kWaves>;
  constexpr int kI = F::kI, kR = F::kR, kAhead = F::kAhead;
  using Held = Staged<T, kR>;
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kPlanes = kF32 ? 3 : 1;
  constexpr int kStage = stage_bytes<kF32>();
  extern __shared__ __align__(256) char lds[];

  uint32_t id = blockIdx.x;
  const uint32_t tiles = uint32_t(a.tiles_n) * a.tiles_k;
  const uint32_t tile = id % tiles;
  id /= tiles;
  const int split = int(id % uint32_t(a.splits));
  int group = int(id / uint32_t(a.splits));
  const int n0 = int(tile / uint32_t(a.tiles_k)) * kBM, k0 = int(tile % uint32_t(a.tiles_k)) * kBN;

  int64_t lo = 0, hi = a.slots;
  if (a.order) {
    lo = a.order[group].y;
    hi = a.order[group].z;
    group = a.order[group].x;
  } else if (a.offsets) {
    group_range(a, group, lo, hi);
  }
  if (a.splits > 1 && hi > lo) {
    const int64_t each = ((hi - lo + a.splits - 1) / a.splits + kBK - 1) / kBK * kBK;
    lo += split * each;
    hi = lo + each < hi ? lo + each : hi;
  }
  const int len = hi > lo && a.tokens > 0 ? int(hi - lo) : 0;
  const int steps = (len + kBK - 1) / kBK;

  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  const int srow = tid >> 4;               // staged rows srow (and srow + 16) of a step
  const int dcol = n0 + (tid & 15) * 8;    // 8 gradients
  const int xcol = k0 + (tid & 15) * 16;   // 16 codes
  // this run's first slot, and where the buffers' last runs start (bytes)
  const GlobalPtr dy = GlobalPtr(a.dy) + lo * a.ld_dy * int64_t(sizeof(T));
  const int64_t dy_last = ((a.slots - 1 - lo) * a.ld_dy + a.n - 8) * int64_t(sizeof(T));
  const int64_t dy_step = a.ld_dy * kBK * int64_t(sizeof(T));
  const int32_t *rows = a.rows + lo;
  // runs that lie wholly past the tile's matrix read its first column instead
  const int dc = dcol < a.n ? dcol : 0, xc = xcol < a.k ? xcol : 0;
  int64_t dy_at[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) dy_at[r] = ((srow + 16 * r) * a.ld_dy + dc) * int64_t(sizeof(T));
  const GlobalPtr codes = GlobalPtr(static_cast<const void *>(a.x.codes)) + xc;
  const GlobalPtr scales = GlobalPtr(static_cast<const void *>(a.x.scales)) + (xc >> 7);
  const uint32_t ld_codes = uint32_t(a.x.ld_codes), ld_scales = uint32_t(a.x.ld_scales);
  // a token's run of codes stays in the buffer up to this one
  const int64_t spare = (a.tokens - 1) * a.x.ld_codes + a.k - 16 - xc;
  const int32_t safe = spare < 0 ? -1 : int32_t(spare / a.x.ld_codes);

  // the slots of a step's rows (a row past the end repeats the last)
  auto slots_of = [&](int step, uint32_t (&slot)[kR]) {
    const int st = step < steps ? step : steps - 1;
    const int most = len - 1 - st * kBK;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int at = srow + 16 * r < most ? srow + 16 * r : most;
      slot[r] = kRows ? uint32_t(rows[st * kBK + at]) : uint32_t(int32_t(lo) + st * kBK + at);
    }
  };
  // A step's loads are issued whatever their rows, and what does not count is
  // mended on the way to LDS: a load that may be skipped would make every
  // later wait one for all loads in flight. A run that reaches past its row's
  // end reads what lies behind it in the buffer (those columns' sums are not
  // stored), and one that would pass the buffer starts that much earlier.
  auto fetch = [&](int step, uint32_t (&slot)[kR], Held &st) {
    st.fix = 0;
    const int near = step < steps ? step : steps - 1;
    const GlobalPtr base = dy + near * dy_step;
    int64_t p[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) p[r] = dy_at[r];
    if (step * kBK + kBK > len || dy_last - near * dy_step < dy_step) {  // the last steps
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (step * kBK + srow + 16 * r >= len) st.fix |= 1u << r;
        const int most = len - 1 - near * kBK;
        const int at = srow + 16 * r < most ? srow + 16 * r : most;
        p[r] = (at * a.ld_dy + dc) * int64_t(sizeof(T));
        const int64_t over = p[r] - (dy_last - near * dy_step);
        if (over > 0) {
          st.fix |= uint32_t(over) << (16 + 8 * r);
          p[r] -= over;
        }
      }
    }
    uint32_t q[kR], early[kR] = {};
    bool odd = false;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      q[r] = __umulhi(slot[r] << 1, div.mul) >> div.shift;  // slot / per_token
      odd |= slot[r] >= div.end || int32_t(q[r]) > safe;
    }
    if (__any(odd)) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (slot[r] >= div.end) {  // no such token
          st.fix |= 1u << r;
          q[r] = 0;
        }
        if (int32_t(q[r]) > safe) {
          early[r] = uint32_t(int64_t(q[r]) * a.x.ld_codes - spare);
          st.fix |= early[r] << (4 + 4 * r);
        }
      }
    }
    slots_of(step + 2, slot);  // before the codes: waiting for it is not waiting for them
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if constexpr (kF32) {
        st.dy[r].v[0] = load16(base + p[r]);
        st.dy[r].v[1] = load16(base + p[r] + 16);
      } else {
        st.dy[r].v = load16(base + p[r]);
      }
      st.codes[r] = load16(codes + uint64_t(q[r]) * ld_codes - early[r]);
      st.scale[r] = uint8_t(scales[uint64_t(q[r]) * ld_scales]);
    }
  };
  auto to_lds = [&](Held &st, char *stage) {
    char *xs = stage + kPlanes * kABytes;
    if (__any(st.fix != 0)) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        constexpr int kDwords = int(sizeof(T)) * 2;
        uint32_t d[kDwords], c[4];
#pragma unroll
        for (int i = 0; i < kDwords; ++i) d[i] = raw_word(st.dy[r], i);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = st.codes[r][i];
        shift_down(c, st.fix >> (4 + 4 * r) & 15);
        shift_down(d, st.fix >> (16 + 8 * r) & 31);
        const bool none = st.fix >> r & 1;
#pragma unroll
        for (int i = 0; i < kDwords; ++i) raw_word(st.dy[r], i, none ? 0u : d[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) st.codes[r][i] = none ? 0u : c[i];
        st.scale[r] = none ? 127u : st.scale[r];  // that of another token: 0 times an infinity is no 0
      }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int row = srow + 16 * r;
      const int at = lds_at(row, dcol - n0, kBM * 2);
      if constexpr (kF32) {
        u32x4 h, m, l;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Split3 s = split3(st.dy[r].get(2 * i), st.dy[r].get(2 * i + 1));
          h[i] = s.hi;
          m[i] = s.mid;
          l[i] = s.lo;
        }
        *reinterpret_cast<u32x4 *>(stage + at) = h;
        *reinterpret_cast<u32x4 *>(stage + kABytes + at) = m;
        *reinterpret_cast<u32x4 *>(stage + 2 * kABytes + at) = l;
      } else {
        *reinterpret_cast<u32x4 *>(stage + at) = st.dy[r].v;
      }
      const float sc = scale_value(st.scale[r]);
      u32x4 v[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i >> 1][(i & 1) * 2] = decode2<0>(st.codes[r][i], sc);
        v[i >> 1][(i & 1) * 2 + 1] = decode2<1>(st.codes[r][i], sc);
      }
      const int xat = lds_at(row, xcol - k0, kBN * 2);
      *reinterpret_cast<u32x4 *>(xs + xat) = v[0];
      *reinterpret_cast<u32x4 *>(xs + xat + 16) = v[1];
    }
  };

  f32x16 acc[kI][2];
  const int wn = (wave >> 2) * 64, wk = (wave & 3) * 64;  // the wave's part of the tile
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // a lane's part of a transposing read: row 8 (lane / 32) + (lane % 16) / 4
  // (the second read of a fragment 4 rows below), columns 16 (lane / 16 % 2) +
  // 4 (lane % 4) of a 32-column run
  const int trow = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int tcol = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  int aoff[kI], xoff[2];
#pragma unroll
  for (int i = 0; i < kI; ++i) aoff[i] = lds_at(trow, wn + 32 * i + tcol, kBM * 2);
#pragma unroll
  for (int j = 0; j < 2; ++j) xoff[j] = lds_at(trow, wk + 32 * j + tcol, kBN * 2);
  typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
  auto frag = [&](const char *base, int off, int pitch) {
    typedef __attribute__((address_space(3))) const char *lds_char;
    const s16x4 p = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_char)base + off));
    const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_char)base + off + 4 * pitch));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(p, q, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // The fragments of a group (16 slots of one part of dy) are read while the
  // products of the group before run (kAhead).
  bf16x8 af[kAhead + 1][kI], bf[kAhead + 1][2];
  auto read_x = [&](const char *stage, int kk) {
#pragma unroll
    for (int j = 0; j < 2; ++j) bf[kk & kAhead][j] = frag(stage + kPlanes * kABytes + kk * 16 * kBN * 2, xoff[j], kBN * 2);
  };
  auto read_dy = [&](const char *stage, int g) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
      af[g & kAhead][i] = frag(stage + (g % kPlanes) * kABytes + (g / kPlanes) * 16 * kBM * 2, aoff[i], kBM * 2);
  };
  constexpr int kGroups = kBK / 16 * kPlanes;
  auto compute = [&](const char *stage) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int next = g + kAhead;
      if (next < kGroups) {
        if (next % kPlanes == 0) read_x(stage, next / kPlanes);
        read_dy(stage, next);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[g & kAhead][i], bf[g / kPlanes & kAhead][j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Step s is in LDS; step s + 1, loaded earlier, goes to the other stage, and
  // one further on is fetched into its registers.
  auto pass = [&](int s, int fetched, Held &st, uint32_t (&slot)[kR], char *now, char *next) {
    if constexpr (kAhead) {
      read_x(now, 0);
      read_dy(now, 0);
    }
    to_lds(st, next);
    fetch(fetched, slot, st);
    __builtin_amdgcn_sched_barrier(0);
    if (s < steps) compute(now);
    __syncthreads();
  };
  if (steps > 0) {
    uint32_t t0[kR], t1[kR];
    slots_of(0, t0);
    slots_of(1, t1);
    if constexpr (kF32 || kWaves == 8) {  // three products a step, or more waves, hide a load by themselves
      Held st;
      fetch(0, t0, st);
      to_lds(st, lds);
      fetch(1, t1, st);
      __syncthreads();
#pragma unroll 1
      for (int s = 0; s < steps; s += 2) {
        pass(s, s + 2, st, t0, lds, lds + kStage);
        pass(s + 1, s + 3, st, t1, lds + kStage, lds);
      }
    } else {
      Held s0, s1;
      fetch(0, t0, s0);
      fetch(1, t1, s1);
      to_lds(s0, lds);
      fetch(2, t0, s0);
      __syncthreads();
#pragma unroll 1
      for (int s = 0; s < steps; s += 2) {
        pass(s, s + 3, s1, t1, lds, lds + kStage);
        pass(s + 1, s + 4, s0, t0, lds + kStage, lds);
      }
    }
  }

  // Epilogue: 32 rows of the wave's 64 columns at a time through LDS, so that
  // a row leaves in runs of eight columns. Accumulator r of a lane is row
  // 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32.
  float *buf = reinterpret_cast<float *>(lds) + wave * 32 * kOutPitch;
#pragma unroll
  for (int i = 0; i < kI; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        buf[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * kOutPitch + 32 * j + (lane & 31)] = acc[i][j][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = q * 8 + (lane >> 3), col = (lane & 7) * 8;
      const int n = n0 + wn + i * 32 + row, k = k0 + wk + col;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = buf[row * kOutPitch + col + e];
      if (n < a.n && k < a.k) {
        if constexpr (kPartial) {
          float *p = a.part + ((int64_t(split) * a.groups + group) * a.n + n) * a.k + k;
          store8(p, pack8(f, float()), a.k - k);
        } else {
          T *p = static_cast<T *>(a.out) + group * a.stride + n * a.ld_out + k;
          // past the caches: the gradients of a set of experts are more than they
          // hold (128 of 768x2048: 217 us through them, 205 past)
          if (a.k - k >= 8)
            store8_stream(p, pack8(f, T()));
          else
            store8(p, pack8(f, T()), a.k - k);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Buffers that hold less than one run of the tiled kernel (gradients of fewer
// than 8 elements, codes of fewer than 16): a thread per element of the
// result.
template <typename T>
__global__ __launch_bounds__(256) void wgrad_tiny_kernel(const WgradArgs a) {
  const int64_t total = int64_t(a.groups) * a.n * a.k;
  for (int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x; u < total; u += int64_t(gridDim.x) * 256) {
    const int k = int(u % a.k), n = int(u / a.k % a.n), group = int(u / (int64_t(a.n) * a.k));
    int64_t lo = 0, hi = a.slots;
    if (a.offsets) {
      lo = a.offsets[group] < 0 ? 0 : a.offsets[group];
      hi = a.offsets[group + 1] > a.slots ? a.slots : a.offsets[group + 1];
    }
    float s = 0.f;
    for (int64_t i = lo; i < hi; ++i) {
      const int32_t slot = a.rows ? a.rows[i] : int32_t(i), token = slot / a.per_token;
      if (slot < 0 || token >= a.tokens) continue;
      const float x = bits_f32(decode2<0>(a.x.codes[token * a.x.ld_codes + k], 1.f) << 16) *
                      scale_value(a.x.scales[token * a.x.ld_scales + (k >> 7)]);
      s = fmaf(float(static_cast<const T *>(a.dy)[i * a.ld_dy + n]), x, s);
    }
    static_cast<T *>(a.out)[group * a.stride + n * a.ld_out + k] = T(s);
  }
}

// Adds the partials in split order; a thread takes eight columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void wgrad_join_kernel(const WgradArgs a) {
  const int64_t runs = (a.k + 7) / 8, total = int64_t(a.groups) * a.n * runs;
  const int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (u >= total) return;
  const int64_t row = u / runs;  // group * n + n
  const int k = int(u - row * runs) * 8;
  const int64_t group = row / a.n, n = row - group * a.n;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int64_t step = int64_t(a.groups) * a.n * a.k;
  const float *p = a.part + row * a.k + k;
#pragma unroll 8
  for (int s = 0; s < a.splits; ++s) {
    const Raw8<float> r = load8(p + s * step, a.k - k);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += r.get(e);
  }
  store8(static_cast<T *>(a.out) + group * a.stride + n * a.ld_out + k, pack8(f, T()), a.k - k);
}

template <typename T>
hipError_t wgrad(const WgradArgs &a, hipStream_t s) {
  const uint32_t work = uint32_t(a.tiles_n) * a.tiles_k * a.splits * a.groups;
  // mul = ceil(2^(31 + shift) / d) with 2^(shift - 1) < d <= 2^shift: exact up
  // to 2^31 (the excess mul d - 2^(31 + shift) < d adds less than 1 / d there)
  const uint64_t d = uint64_t(a.per_token);
  TokenOf div{0, 0, uint32_t(std::min<uint64_t>(uint64_t(a.tokens) * d, uint64_t(1) << 31))};
  while ((uint64_t(1) << div.shift) < d) ++div.shift;
  div.mul = uint32_t(((uint64_t(1) << (31 + div.shift)) + d - 1) / d);
  if (a.slots > 0 && a.tokens > 0 &&
      ((a.slots - 1) * a.ld_dy + a.n < 8 || (a.tokens - 1) * a.x.ld_codes + a.k < 16)) {
    const int64_t total = int64_t(a.groups) * a.n * a.k;
    hipLaunchKernelGGL(wgrad_tiny_kernel<T>, dim3(unsigned(std::min<int64_t>((total + 255) / 256, 1 << 20))), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (a.order) {
    hipLaunchKernelGGL(wgrad_order_kernel, dim3(1), dim3(kOrderGroups), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(work);
  auto go = [&](auto form) {
    constexpr int kWaves = decltype(form)::value;
    constexpr int kStage = stage_bytes<sizeof(T) == 4>(), kEpilogue = kWaves * 32 * kOutPitch * 4;
    constexpr int kLds = 2 * kStage > kEpilogue ? 2 * kStage : kEpilogue;
    auto kernel = a.splits == 1 ? (a.rows ? wgrad_kernel<T, kWaves, true, false> : wgrad_kernel<T, kWaves, false, false>)
                                : (a.rows ? wgrad_kernel<T, kWaves, true, true> : wgrad_kernel<T, kWaves, false, true>);
    hipLaunchKernelGGL(kernel, grid, dim3(kWaves * 64), kLds, s, a, div);
  };
  // us with four / eight waves, by slots a group:      128          512        1024
  //   bf16     64 groups into 768x2048             79 / 68    158 / 157   244 / 256
  //            16 into 2048x2048                   50 / 43     96 / 93    159 / 163
  //             1 into 2048x7168                   14 / 12     24 / 25     38 / 41
  //            32 into 256x1024 (128 tiles)        11 / 9      21 / 18     32 / 29
  //   float32  64 into 768x2048                   194 / 207   353 / 360   633 / 612
  //            16 into 2048x2048                  137 / 147   247 / 229   409 / 402
  //             1 into 2048x7168                   39 / 38     67 / 63    101 / 99
  // The rule is that of bf16 with more tiles than CUs, which gains most from it;
  // float32 and few tiles would take eight waves at 1024 slots too, for 1 to 10%.
  if (a.slots < 768 * int64_t(a.groups))
    go(std::integral_constant<int, 8>());
  else
    go(std::integral_constant<int, 4>());
  if (a.splits == 1) return hipGetLastError();
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t total = int64_t(a.groups) * a.n * ((a.k + 7) / 8);
  hipLaunchKernelGGL(wgrad_join_kernel<T>, dim3(unsigned((total + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// A sum is split where that is the shorter of both by these measured times: a
// step of 32 slots takes 0.7 us (float32 1.8) with a workgroup a CU, a third
// more with two; each split writes and reads 8 bytes an element at 5 TB/s and
// adds a load to the joining launch, which itself takes 5 us. 512 slots into
// 768x2048 take 16 us whole and 24 in four; 16384 into 512x2048 361 us whole and
// 62 in sixteen.
void wgrad_plan(WgradArgs &a, bool bf16) {
  a.tiles_n = (a.n + kBM - 1) / kBM;
  a.tiles_k = (a.k + kBN - 1) / kBN;
  a.splits = 1;
  const int64_t tiles = int64_t(a.tiles_n) * a.tiles_k * a.groups;
  const double steps = double(a.slots) / a.groups / kBK, step_us = bf16 ? 0.7 : 1.8;
  const double each_us = double(a.groups) * a.n * a.k * 8 / 5e6 + 0.1;
  double best = 0;
  for (int64_t s = 1; s * tiles <= 512 && (s == 1 || s <= steps); s *= 2) {
    const double us = steps / double(s) * step_us * (s * tiles > 256 ? 1.35 : 1.0) + (s > 1 ? 5 + double(s) * each_us : 0);
    if (s > 1 && us >= best) continue;
    best = us;
    a.splits = int32_t(s);
  }
}

size_t wgrad_part_bytes(const WgradArgs &a) {
  return a.splits > 1 ? size_t(a.splits) * a.groups * a.n * a.k * sizeof(float) : 0;
}

// Worth its launch where not all tiles are at work at once and the products
// outweigh the stores: the order brings the long groups' products together, and
// then the short ones' stores. 128 slots a group on average (32 groups of 768x2048
// float32) take 110 us in the given order and 124 by length; 256 (128 groups, bf16)
// 192 and 190.
size_t wgrad_order_bytes(const WgradArgs &a) {
  const int64_t tiles = int64_t(a.tiles_n) * a.tiles_k * a.groups;
  if (a.groups < 2 || a.groups > kOrderGroups || tiles <= 512 || a.slots < 256 * int64_t(a.groups)) return 0;
  return size_t(a.groups) * sizeof(int4);
}

hipError_t launch_wgrad(const WgradArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? wgrad<__bf16>(a, s) : wgrad<float>(a, s);
}

}  // namespace muon
