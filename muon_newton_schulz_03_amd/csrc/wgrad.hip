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
#include <hip/hip_runtime.h>

#include <algorithm>

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
constexpr int kThreads = 256;  // 4 waves, each 128 x 64 of the tile
constexpr int kABytes = kBK * kBM * 2;
constexpr int kXBytes = kBK * kBN * 2;
constexpr int kOutPitch = 64 + 4;  // floats; epilogue rows of a wave

template <bool kF32>
constexpr int stage_bytes() {
  return (kF32 ? 3 : 1) * kABytes + kXBytes;
}

// LDS rows hold one slot: 128 (dy) or 256 (X) bf16 in runs of 32 columns (64
// bytes), run i of row t at place i ^ (t & 3) within its four. A transposing
// read takes 32 columns of four consecutive rows: four different quarters of
// the 256-byte bank row.
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

constexpr uint32_t kNoToken = 0xffffffffu;

// 16 bytes from p, zeros from `end` on (the buffer's end is all that stops it).
__device__ inline u32x4 load16(const char *p, const char *end) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (p + 16 <= end) {
    v = *reinterpret_cast<const u32x4_any *>(p);
  } else {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = p + i < end ? uint8_t(p[i]) : 0u;
      v[0] = v[0] >> 8 | v[1] << 24;
      v[1] = v[1] >> 8 | v[2] << 24;
      v[2] = v[2] >> 8 | v[3] << 24;
      v[3] = v[3] >> 8 | b << 24;
    }
  }
  return v;
}

// What a thread holds of a step on its way to LDS: two rows' runs of 8
// gradients, and two rows' runs of 16 codes with their scales.
template <typename T>
struct Staged {
  Raw8<T> dy[2];
  u32x4 codes[2];
  uint32_t scale[2];
};

template <typename T, bool kPartial>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(const WgradArgs a, uint32_t token_magic) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kPlanes = kF32 ? 3 : 1;
  constexpr int kStage = stage_bytes<kF32>();
  extern __shared__ __align__(256) char lds[];

  // consecutive work (the tiles of one group) on one XCD, which shares an L2
  const uint32_t per_xcd = (gridDim.x + 7) / 8;
  uint32_t id = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  const uint32_t tiles = uint32_t(a.tiles_n) * a.tiles_k;
  const uint32_t work = tiles * a.splits * a.groups;
  if (id >= work) return;
  const uint32_t tile = id % tiles;
  id /= tiles;
  const int split = int(id % uint32_t(a.splits)), group = int(id / uint32_t(a.splits));
  const int n0 = int(tile / uint32_t(a.tiles_k)) * kBM, k0 = int(tile % uint32_t(a.tiles_k)) * kBN;

  int64_t lo = 0, hi = a.slots;
  if (a.offsets) {
    lo = a.offsets[group];
    hi = a.offsets[group + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > a.slots ? a.slots : hi;
  }
  if (a.splits > 1 && hi > lo) {
    const int64_t each = ((hi - lo + a.splits - 1) / a.splits + kBK - 1) / kBK * kBK;
    lo += split * each;
    hi = lo + each < hi ? lo + each : hi;
  }
  const int len = hi > lo ? int(hi - lo) : 0;
  const int steps = (len + kBK - 1) / kBK;

  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  const int srow = tid >> 4;               // staged rows srow and srow + 16 of a step
  const int dcol = n0 + (tid & 15) * 8;    // 8 gradients
  const int xcol = k0 + (tid & 15) * 16;   // 16 codes
  // this run's first slot; a lane's place in a step's rows
  const char *dy = static_cast<const char *>(a.dy) + lo * a.ld_dy * int64_t(sizeof(T));
  const int64_t dyoff = (srow * a.ld_dy + dcol) * int64_t(sizeof(T));
  const char *dy_end = static_cast<const char *>(a.dy) + ((a.slots - 1) * a.ld_dy + a.n) * int64_t(sizeof(T));
  const char *codes_end = reinterpret_cast<const char *>(a.x.codes) + (a.tokens - 1) * a.x.ld_codes + a.k;
  const int32_t *rows = a.rows + lo;

  // the tokens of a step's rows, one step ahead of their codes
  auto token_of = [&](int step, uint32_t (&token)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int at = step * kBK + srow + 16 * r;
      token[r] = kNoToken;
      if (at < len) {
        const uint32_t v = uint32_t(a.rows ? rows[at] : int32_t(lo) + at);
        uint32_t q = __umulhi(v, token_magic);  // v / per_token, one too few at most
        if (v - q * uint32_t(a.per_token) >= uint32_t(a.per_token)) ++q;
        if (q < uint32_t(a.tokens)) token[r] = q;
      }
    }
  };
  // Runs that reach past a row's end read what lies behind it in the buffer:
  // those columns' sums are not stored. Nothing past the buffer is read.
  auto fetch = [&](int step, const uint32_t (&token)[2], Staged<T> &st) {
    const char *base = dy + int64_t(step) * (kBK * int64_t(sizeof(T))) * a.ld_dy;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      st.dy[r] = Raw8<T>{};
      st.codes[r] = u32x4{0u, 0u, 0u, 0u};
      st.scale[r] = 127;
      if (token[r] == kNoToken) continue;
      if (dcol < a.n) {
        const char *p = base + dyoff + r * 16 * int(sizeof(T)) * a.ld_dy;
        if constexpr (kF32) {
          st.dy[r].v[0] = load16(p, dy_end);
          st.dy[r].v[1] = load16(p + 16, dy_end);
        } else {
          st.dy[r].v = load16(p, dy_end);
        }
      }
      if (xcol < a.k) {
        st.codes[r] = load16(reinterpret_cast<const char *>(a.x.codes) + int64_t(token[r]) * a.x.ld_codes + xcol, codes_end);
        st.scale[r] = a.x.scales[int64_t(token[r]) * a.x.ld_scales + (xcol >> 7)];
      }
    }
  };
  auto to_lds = [&](const Staged<T> &st, char *stage) {
    char *xs = stage + kPlanes * kABytes;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
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

  f32x16 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // a lane's part of a transposing read: row 8 (lane / 32) + (lane % 16) / 4
  // (the second read of a fragment 4 rows below), columns 16 (lane / 16 % 2) +
  // 4 (lane % 4) of a 32-column run
  const int trow = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int tcol = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  int aoff[4], xoff[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) aoff[i] = lds_at(trow, 32 * i + tcol, kBM * 2);
#pragma unroll
  for (int j = 0; j < 2; ++j) xoff[j] = lds_at(trow, wave * 64 + 32 * j + tcol, kBN * 2);
  typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
  auto frag = [&](const char *base, int off, int pitch) {
    typedef __attribute__((address_space(3))) const char *lds_char;
    const s16x4 p = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_char)base + off));
    const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_char)base + off + 4 * pitch));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(p, q, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto compute = [&](const char *stage) {
    const char *xs = stage + kPlanes * kABytes;
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
      bf16x8 bf[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) bf[j] = frag(xs + kk * 16 * kBN * 2, xoff[j], kBN * 2);
#pragma unroll
      for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 af = frag(stage + pl * kABytes + kk * 16 * kBM * 2, aoff[i], kBM * 2);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af, bf[j], acc[i][j], 0, 0, 0);
        }
    }
  };

  if (steps > 0) {
    Staged<T> st;
    uint32_t tok[2];
    token_of(0, tok);
    fetch(0, tok, st);
    token_of(1, tok);
    to_lds(st, lds);
    fetch(1, tok, st);
    token_of(2, tok);
    __syncthreads();
    // step s: LDS holds it; s + 1 goes to the other stage, s + 2 is fetched
    int at = 0;
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      to_lds(st, lds + (kStage - at));
      fetch(s + 2, tok, st);
      token_of(s + 3, tok);
      __builtin_amdgcn_sched_barrier(0);
      compute(lds + at);
      __syncthreads();
      at = kStage - at;
    }
  }

  // Epilogue: 32 rows of the wave's 64 columns at a time through LDS, so that
  // a row leaves in runs of eight columns. Accumulator r of a lane is row
  // 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32.
  float *buf = reinterpret_cast<float *>(lds) + wave * 32 * kOutPitch;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
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
      const int n = n0 + i * 32 + row, k = k0 + wave * 64 + col;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = buf[row * kOutPitch + col + e];
      if (n < a.n && k < a.k) {
        if constexpr (kPartial) {
          float *p = a.part + ((int64_t(split) * a.groups + group) * a.n + n) * a.k + k;
          store8(p, pack8(f, float()), a.k - k);
        } else {
          T *p = static_cast<T *>(a.out) + group * a.stride + n * a.ld_out + k;
          store8(p, pack8(f, T()), a.k - k);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const Raw8<float> r = load8(p + s * step, a.k - k);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += r.get(e);
  }
  store8(static_cast<T *>(a.out) + group * a.stride + n * a.ld_out + k, pack8(f, T()), a.k - k);
}

template <typename T>
hipError_t wgrad(const WgradArgs &a, hipStream_t s) {
  constexpr int kStage = stage_bytes<sizeof(T) == 4>();
  constexpr int kEpilogue = 4 * 32 * kOutPitch * 4;
  constexpr int kLds = 2 * kStage > kEpilogue ? 2 * kStage : kEpilogue;
  const uint32_t work = uint32_t(a.tiles_n) * a.tiles_k * a.splits * a.groups;
  const uint32_t magic =
      uint32_t(std::min<uint64_t>((uint64_t(1) << 32) / uint32_t(a.per_token), 0xffffffffu));
  const dim3 grid((work + 7) / 8 * 8);
  if (a.splits == 1) {
    hipLaunchKernelGGL((wgrad_kernel<T, false>), grid, dim3(kThreads), kLds, s, a, magic);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((wgrad_kernel<T, true>), grid, dim3(kThreads), kLds, s, a, magic);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t total = int64_t(a.groups) * a.n * ((a.k + 7) / 8);
  hipLaunchKernelGGL(wgrad_join_kernel<T>, dim3(unsigned((total + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Splits: enough that two workgroups a CU have work, of 128 slots at least.
void wgrad_plan(WgradArgs &a, bool bf16) {
  (void)bf16;
  a.tiles_n = (a.n + kBM - 1) / kBM;
  a.tiles_k = (a.k + kBN - 1) / kBN;
  const int64_t tiles = int64_t(a.tiles_n) * a.tiles_k * a.groups;
  const int64_t len = (a.slots + a.groups - 1) / a.groups;
  a.splits = int32_t(std::max<int64_t>(1, std::min<int64_t>(512 / tiles, len / 128)));
}

size_t wgrad_part_bytes(const WgradArgs &a) {
  return a.splits > 1 ? size_t(a.splits) * a.groups * a.n * a.k * sizeof(float) : 0;
}

hipError_t launch_wgrad(const WgradArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? wgrad<__bf16>(a, s) : wgrad<float>(a, s);
}

}  // namespace muon
