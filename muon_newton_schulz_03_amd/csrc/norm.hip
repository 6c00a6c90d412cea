// Layer norm, forward and backward (gfx950).
//
//   mu = sum x / C,  r = 1 / sqrt(sum (x - mu)^2 / C + eps),
//   y = (x - mu) r w + b;
//   xh = (x - mu) r,  h = dy w,  dx = r (h - mean(h) - xh mean(h xh)),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// Both passes are bound by memory: each element is read once into registers,
// where a row's sums are taken (centred, in float32), and written once. A
// row belongs to one wave (up to 1024 columns) or one workgroup. The forward pass
// ends the variance's sum in 64 bits and computes what lies near a border of the
// 8-bit codes again in 64 bits: of 8192x7168 codes 20 to 30 then differ from those
// of the exact output (in float32 alone 50), for less than 1 us from memory and 2 us
// of 38 where the activations are in the cache. Measured, bf16: forward with checkpoint
// 8192x7168 65 us (4.5 TB/s), backward 16384x7168 135 us with the launch that adds
// the workgroups' partial sums (5.2 TB/s; a copy of 1 GiB runs at 5.0). A backward
// pass of 333x2047 float32 is 7 + 3 us of two launches: 167 workgroups of two rows,
// which leave a third of the CUs without work, and the one that adds their sums.
//
// Above 8192 columns the backward pass does not fit its registers (two sums, this
// row, the next one and the weight): 4 to 145 of a thread's lie in memory up to
// 16384 columns, 148 to 676 above. 4096x12288 bf16 takes 71 us (4.2 TB/s), float32
// 180 (3.4); 2048x32768 bf16 500 us (0.8 TB/s), float32 870 (0.9).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

// Runs of a row whose length is a whole number of runs (kWhole) are there or
// not; else the last one may be cut. The first form has no branch but the
// lanes' own.
template <bool kWhole, typename T>
__device__ inline Raw8<T> load_run(const T *p, int n) {
  return load8(p, kWhole ? (n > 0 ? 8 : 0) : n);
}
template <bool kWhole, typename T>
__device__ inline void store_run(T *p, const Raw8<T> &r, int n) {
  store8(p, r, kWhole ? 8 : n);
}

// Sums of one or two values over the kTpr threads of a row; `slot` toggles
// between two LDS areas, so one barrier a call is enough.
template <int kTpr, int kN>
__device__ inline void row_sum(float (&v)[kN], float *lds, int &slot) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = wave_sum(v[i]);
  if constexpr (kTpr > 64) {
    constexpr int kWaves = kTpr / 64;
    float *area = lds + slot * kWaves * kN;
    slot ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < kN; ++i) area[(threadIdx.x >> 6) * kN + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[i] += area[w * kN + i];
    }
  }
}

// The sum over the kTpr threads of a row, the last two levels of a wave and the
// waves in 64 bits: their few roundings are half of what such a sum is off by.
__device__ inline double join64(uint32_t lo, uint32_t hi) { return __builtin_bit_cast(double, uint64_t(lo) | uint64_t(hi) << 32); }
template <int kTpr>
__device__ inline double row_sum64(float v, double *lds) {
  v += dpp<kQuadSwap1>(v);
  v += dpp<kQuadSwap2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  const Pair p = rows_16(v);
  const uint64_t u = __builtin_bit_cast(uint64_t, double(p.a) + double(p.b));
  const auto lo = __builtin_amdgcn_permlane32_swap(uint32_t(u), uint32_t(u), false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap(uint32_t(u >> 32), uint32_t(u >> 32), false, false);
  double s = join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
  if constexpr (kTpr > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.;
#pragma unroll
    for (int w = 0; w < kTpr / 64; ++w) s += lds[w];
  }
  return s;
}

// At most 2 kSlack where a result lies within kSlack units of its last bit of a border
// that decides its 8-bit code: the middle between two codes has its low 20 bits at
// 0x80000; bf16 results become that middle, or pass it, half a bf16 step to its sides.
// (Codes below 2^-6 of their scale have fewer bits and other middles. They are a
// step of the smallest off, at most.)
constexpr uint32_t kSlack = 4;
template <typename T>
__device__ inline uint32_t border(float f) {
  if constexpr (sizeof(T) == 2)
    return (f32_bits(f) + kSlack - 0x78000u) & 0xeffffu;
  else
    return (f32_bits(f) + kSlack - 0x80000u) & 0xfffffu;
}

// kTpr threads a row, kNv runs of 8 columns a thread.
template <typename T, bool kWf32, bool kCkpt, bool kWhole, int kTpr, int kNv>
__global__ __launch_bounds__(kTpr < 256 ? 256 : kTpr) void norm_fwd_kernel(const NormFwdArgs a) {
  constexpr int kBlock = kTpr < 256 ? 256 : kTpr;
  __shared__ float lds[2 * (kTpr / 64)];
  __shared__ double lds64[kTpr / 64];
  using W = std::conditional_t<kWf32, float, __bf16>;
  int slot = 0;
  const int t = int(threadIdx.x) % kTpr;
  const int64_t row = int64_t(blockIdx.x) * (kBlock / kTpr) + int(threadIdx.x) / kTpr;
  if (row >= a.rows) return;  // whole rows leave (one row a workgroup, or one a wave)
  const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
  T *y = static_cast<T *>(a.y) + row * a.ld_y;
  Raw8<T> xr[kNv];
  float s[1] = {0.f};
#pragma unroll
  for (int v = 0; v < kNv; ++v) {
    const int c = (v * kTpr + t) * 8;
    xr[v] = load_run<kWhole>(x + c, a.cols - c);
  }
#pragma unroll
  for (int v = 0; v < kNv; ++v)
    s[0] += ((xr[v].get(0) + xr[v].get(1)) + (xr[v].get(2) + xr[v].get(3))) +
            ((xr[v].get(4) + xr[v].get(5)) + (xr[v].get(6) + xr[v].get(7)));
  row_sum<kTpr, 1>(s, lds, slot);
  const float mean = s[0] / float(a.cols);
  // the squares as a tree: one after another, each addition would be rounded against
  // the thread's largest square, and outliers are what activations have
  float sq[kNv];
#pragma unroll
  for (int v = 0; v < kNv; ++v) {
    const int n = a.cols - (v * kTpr + t) * 8;
    sq[v] = 0.f;
    if (n <= 0) continue;
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = kWhole || i < n ? xr[v].get(i) - mean : 0.f;
    sq[v] = (fmaf(d[1], d[1], d[0] * d[0]) + fmaf(d[3], d[3], d[2] * d[2])) +
            (fmaf(d[5], d[5], d[4] * d[4]) + fmaf(d[7], d[7], d[6] * d[6]));
  }
#pragma unroll
  for (int w = 1; w < kNv; w *= 2)
#pragma unroll
    for (int v = 0; v < kNv; v += 2 * w) sq[v] += sq[v + w];
  const double var = row_sum64<kTpr>(sq[0], lds64) * a.inv_cols + double(a.eps);
  const float rstd = 1.f / sqrtf(float(var));
  const double r64 = rstd;
  float rest = float(0.5 * r64 * (1. - var * r64 * r64));
  rest = rstd > 0.f && rstd < 1e30f ? rest : 0.f;
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd + rest;
  }
#pragma unroll
  for (int v = 0; v < kNv; ++v) {
    const int c = (v * kTpr + t) * 8, n = a.cols - c;
    if (kCkpt ? !__any(n > 0) : n <= 0) break;
    float f[8];
    const float one[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    Raw8<W> w = pack8(one, W()), b{};
    if (a.w) w = load_run<kWhole>(static_cast<const W *>(a.w) + c, n);
    if (a.b) b = load_run<kWhole>(static_cast<const W *>(a.b) + c, n);
    // In float32, and the runs with a value near a border again in 64 bits: one in a
    // hundred of a wave's. (As two steps, to float32 and then to T: the compiler may
    // make one of them, which rounds other ties of the second.) Not above 16384
    // columns, where the registers for it leave one workgroup a CU (without a
    // checkpoint 2048x32768 59 us, 48 so).
    constexpr bool kAgain = kTpr * kNv <= 2048;
    uint32_t near = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = xr[v].get(i) - mean;
      f[i] = fmaf(fmaf(d, rest, d * rstd), w.get(i), b.get(i));
      near = min(near, border<T>(f[i]));
    }
    if (kAgain && near <= 2 * kSlack) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)
        __builtin_amdgcn_sched_barrier(0);  // one after another: few registers, and it is rare
        f[i] = float(fma((double(xr[v].get(i)) - double(mean)) * (r64 + double(rest)), double(w.get(i)), double(b.get(i))));
      }
    }
    const Raw8<T> r = pack8(f, T());
    if (n > 0) store_run<kWhole>(y + c, r, n);
    if constexpr (kCkpt) {
      // the checkpoint of y as stored; its groups of 128 columns are 16 lanes
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = (kWhole ? n > 0 : i < n) ? r.get(i) : 0.f;
        m = max(m, finite_mag(f[i]));
      }
      const uint32_t sb = scale_byte(row16_max(m));
      const u32x2 codes = encode8(f, scale_inverse(sb));
      if (n > 0) {
        store_codes8(a.ck.codes + row * a.ck.ld_codes + c, codes, n);
        if ((t & 15) == 0) a.ck.scales[row * a.ck.ld_scales + (c >> 7)] = uint8_t(sb);
      }
    }
  }
}

template <typename T, bool kWf32, bool kCkpt, bool kWhole>
hipError_t fwd(const NormFwdArgs &a, hipStream_t s) {
  auto go = [&](auto kernel, int tpr) {
    const int per = tpr < 256 ? 256 / tpr : 1;
    constexpr int64_t kMost = 1 << 21;  // workgroups a launch: fewer than 2^32 threads
    for (int64_t r = 0; r < a.rows; r += kMost * per) {
      NormFwdArgs part = a;
      part.rows = a.rows - r < kMost * per ? a.rows - r : kMost * per;
      part.x = static_cast<const T *>(a.x) + r * a.ld_x;
      part.y = static_cast<T *>(a.y) + r * a.ld_y;
      if (a.mean) part.mean = a.mean + r;
      if (a.rstd) part.rstd = a.rstd + r;
      if (kCkpt) {
        part.ck.codes = a.ck.codes + r * a.ck.ld_codes;
        part.ck.scales = a.ck.scales + r * a.ck.ld_scales;
      }
      hipLaunchKernelGGL(kernel, dim3(unsigned((part.rows + per - 1) / per)), dim3(tpr < 256 ? 256 : tpr), 0, s, part);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  if (a.cols <= 512) return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 64, 1>, 64);
  if (a.cols <= 1024) return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 64, 2>, 64);
  if (a.cols <= 2048) return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 256, 1>, 256);
  if (a.cols <= 4096) return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 256, 2>, 256);
  if (a.cols <= 8192) return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 256, 4>, 256);
  if (a.cols <= 16384) return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 1024, 2>, 1024);
  return go(norm_fwd_kernel<T, kWf32, kCkpt, kWhole, 1024, 4>, 1024);
}

// Each workgroup takes rows b, b + blocks, ... (kBlock / kTpr at a time) and
// keeps its columns' sums of dy xh and dy, and the weight, in registers; the
// loads of its next rows are in flight while one is reduced.
template <typename T, bool kWf32, bool kWhole, int kTpr, int kNv>
__global__ __launch_bounds__(kTpr < 256 ? 256 : kTpr) void norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int kBlock = kTpr < 256 ? 256 : kTpr;
  constexpr int kPer = kBlock / kTpr;
  using W = std::conditional_t<kWf32, float, __bf16>;
  __shared__ float lds[2 * (kTpr / 64) * 2];
  __shared__ float comb[kPer > 1 ? kTpr * kNv * 8 : 1];
  int slot = 0;
  const int t = int(threadIdx.x) % kTpr, sub = int(threadIdx.x) / kTpr;
  const float inv_c = 1.f / float(a.cols);
  Raw8<T> xn[kNv], dn[kNv];
  Raw8<W> w[kNv];
  float mn, rn;
  float aw[kNv][8], ab[kNv][8];
#pragma unroll
  for (int v = 0; v < kNv; ++v) {
    const int c = (v * kTpr + t) * 8;
    if (a.w) {
      w[v] = load_run<kWhole>(static_cast<const W *>(a.w) + c, a.cols - c);
    } else {
      const float one[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      w[v] = pack8(one, W());
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) aw[v][i] = ab[v][i] = 0.f;
  }
  // 0, in a vector register: a value known to be the same in every lane would
  // be moved to a scalar one at once, which waits for all loads before it
  int lane0 = 0;
  asm volatile("" : "+v"(lane0));
  auto fetch = [&](int64_t row) {
    const bool there = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    const T *d = static_cast<const T *>(a.dy) + row * a.ld_dy;
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      const int c = (v * kTpr + t) * 8, n = there ? a.cols - c : 0;
      xn[v] = load_run<kWhole>(x + c, n);
      dn[v] = load_run<kWhole>(d + c, n);
    }
    const int64_t at = (there ? row : 0) + lane0;
    const float m = a.mean[at], r = a.rstd[at];
    mn = there ? m : 0.f;
    rn = there ? r : 0.f;
  };
  const int64_t step = int64_t(a.blocks) * kPer;
  int64_t base = int64_t(blockIdx.x) * kPer;
  fetch(base + sub);
  for (; base < a.rows; base += step) {
    const int64_t row = base + sub;
    const float mean = mn, rstd = rn;
    Raw8<T> xr[kNv], dr[kNv];
#pragma unroll
    for (int v = 0; v < kNv; ++v) xr[v] = xn[v], dr[v] = dn[v];
    fetch(row + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kNv; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = dr[v].get(i), xh = (xr[v].get(i) - mean) * rstd, h = g * w[v].get(i);
        s[0] += h;
        s[1] = fmaf(h, xh, s[1]);
        aw[v][i] = fmaf(g, xh, aw[v][i]);
        ab[v][i] += g;
      }
    row_sum<kTpr, 2>(s, lds, slot);
    if (row < a.rows) {
      const float m0 = s[0] * inv_c, m1 = s[1] * inv_c;
      T *dx = static_cast<T *>(a.dx) + row * a.ld_dx;
#pragma unroll
      for (int v = 0; v < kNv; ++v) {
        const int c = (v * kTpr + t) * 8, n = a.cols - c;
        if (n <= 0) break;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (xr[v].get(i) - mean) * rstd;
          f[i] = rstd * (dr[v].get(i) * w[v].get(i) - m0 - xh * m1);
        }
        store_run<kWhole>(dx + c, pack8(f, T()), n);
      }
    }
  }
  if (!a.sums) return;
  float *part = a.part + int64_t(blockIdx.x) * 2 * a.cols;
  auto leave = [&](float(&acc)[kNv][8], float *to) {
    if constexpr (kPer > 1) {  // the workgroup's rows, added wave by wave
#pragma unroll
      for (int p = kPer - 1; p > 0; --p) {
        __syncthreads();
        if (sub == p)
#pragma unroll
          for (int v = 0; v < kNv; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) comb[(v * 8 + i) * kTpr + t] = acc[v][i];
        __syncthreads();
        if (sub == 0)
#pragma unroll
          for (int v = 0; v < kNv; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[v][i] += comb[(v * 8 + i) * kTpr + t];
      }
    }
    if (sub == 0)
#pragma unroll
      for (int v = 0; v < kNv; ++v) {
        const int c = (v * kTpr + t) * 8, n = a.cols - c;
        if (n > 0) store_run<kWhole>(to + c, pack8(acc[v], float()), n);
      }
  };
  leave(aw, part);
  leave(ab, part + a.cols);
}

// A tree: added one after another, each would be rounded against the largest sum.
__device__ inline float sum8(const float (&v)[8]) { return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])); }

// Sums the workgroups' partials: 32 columns a workgroup, 8 threads a column,
// each over every eighth partial, joined in a fixed order.
constexpr int kRedCols = 32, kRedSlices = 8;
__global__ __launch_bounds__(kRedCols * kRedSlices) void norm_grad_kernel(const NormBwdArgs a) {
  __shared__ float lds[kRedSlices][kRedCols];
  const int lc = int(threadIdx.x) % kRedCols, sl = int(threadIdx.x) / kRedCols;
  const int c = int(blockIdx.x) * kRedCols + lc;  // of 2 * cols: dw, then db
  float s = 0.f;
  if (c < 2 * a.cols) {
    const float *p = a.part + c;
    for (int b = sl; b < a.blocks; b += 8 * kRedSlices) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = b + j * kRedSlices;
        v[j] = at < a.blocks ? p[int64_t(at) * 2 * a.cols] : 0.f;
      }
      s += sum8(v);
    }
  }
  lds[sl][lc] = s;
  __syncthreads();
  if (sl || c >= 2 * a.cols) return;
  float v[kRedSlices];
#pragma unroll
  for (int j = 0; j < kRedSlices; ++j) v[j] = lds[j][lc];
  s = sum8(v);
  void *out = c < a.cols ? a.dw : a.db;
  const int oc = c < a.cols ? c : c - a.cols;
  if (!out) return;
  if (a.w_f32)
    static_cast<float *>(out)[oc] = s;
  else
    static_cast<__bf16 *>(out)[oc] = __bf16(s);
}

// Threads a row of the backward kernel. Wide rows: 512, so that 256 workgroups
// (whose partial sums the second launch reads) fill the chip; 16384x7168 bf16
// takes 136 us so, 165 with 256 threads and 512 workgroups.
int bwd_tpr(int64_t cols) { return cols <= 1024 ? 64 : cols <= 2048 ? 256 : cols <= 16384 ? 512 : 1024; }

template <typename T, bool kWf32, bool kWhole>
hipError_t bwd(const NormBwdArgs &a, hipStream_t s) {
  auto go = [&](auto kernel, int tpr) {
    if (a.blocks > 0) hipLaunchKernelGGL(kernel, dim3(unsigned(a.blocks)), dim3(tpr < 256 ? 256 : tpr), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.sums) return e;
    hipLaunchKernelGGL(norm_grad_kernel, dim3((2 * a.cols + kRedCols - 1) / kRedCols), dim3(kRedCols * kRedSlices), 0, s,
                       a);
    return hipGetLastError();
  };
  if (a.cols <= 512) return go(norm_bwd_kernel<T, kWf32, kWhole, 64, 1>, 64);
  if (a.cols <= 1024) return go(norm_bwd_kernel<T, kWf32, kWhole, 64, 2>, 64);
  if (a.cols <= 2048) return go(norm_bwd_kernel<T, kWf32, kWhole, 256, 1>, 256);
  if (a.cols <= 4096) return go(norm_bwd_kernel<T, kWf32, kWhole, 512, 1>, 512);
  if (a.cols <= 8192) return go(norm_bwd_kernel<T, kWf32, kWhole, 512, 2>, 512);
  if (a.cols <= 16384) return go(norm_bwd_kernel<T, kWf32, kWhole, 512, 4>, 512);
  return go(norm_bwd_kernel<T, kWf32, kWhole, 1024, 4>, 1024);
}

}  // namespace

// Workgroups of the backward pass: enough to fill the chip, but each with
// several rows, since each leaves 8 bytes a column of partial sums.
int norm_bwd_blocks(int64_t rows, int64_t cols) {
  const int per = bwd_tpr(cols) < 256 ? 256 / bwd_tpr(cols) : 1;
  const int64_t want = (rows + 2 * per - 1) / (2 * per), most = bwd_tpr(cols) < 512 ? 512 : 256;
  return int(want < most ? want : most);
}

namespace {
template <typename T, bool kWf32>
hipError_t fwd(const NormFwdArgs &a, hipStream_t s) {
  const bool ck = a.ck.codes != nullptr;
  if (a.cols % 8 == 0) return ck ? fwd<T, kWf32, true, true>(a, s) : fwd<T, kWf32, false, true>(a, s);
  return ck ? fwd<T, kWf32, true, false>(a, s) : fwd<T, kWf32, false, false>(a, s);
}
template <typename T, bool kWf32>
hipError_t bwd(const NormBwdArgs &a, hipStream_t s) {
  return a.cols % 8 == 0 ? bwd<T, kWf32, true>(a, s) : bwd<T, kWf32, false>(a, s);
}
}  // namespace

hipError_t launch_norm_fwd(const NormFwdArgs &a, bool bf16, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  if (bf16) return a.w_f32 ? fwd<__bf16, true>(a, s) : fwd<__bf16, false>(a, s);
  return a.w_f32 ? fwd<float, true>(a, s) : fwd<float, false>(a, s);
}

hipError_t launch_norm_bwd(const NormBwdArgs &a, bool bf16, hipStream_t s) {
  if (bf16) return a.w_f32 ? bwd<__bf16, true>(a, s) : bwd<__bf16, false>(a, s);
  return a.w_f32 ? bwd<float, true>(a, s) : bwd<float, false>(a, s);
}

}  // namespace muon
