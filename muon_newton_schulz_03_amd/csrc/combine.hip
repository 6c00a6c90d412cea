// The sum over a token's experts with dropout and residual, and its backward
// pass (gfx950):
//   y[t]  = res[t] + m[t] / (1 - p) * sum_j weights[t, j] x[t topk + j]
//   dx[t topk + j] = weights[t, j] d[t],  dweights[t, j] = <x[t topk + j], d[t]>,
//   d[t]  = m[t] / (1 - p) * dy[t]
// over the choices j that the token has; one choice of weight 1 is dropout
// alone. The mask m is never stored: element i of y in row order takes word
// i mod 4 of block i / 4 of the counter-based generator Philox4x32-10 (Salmon,
// Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011),
// keyed by a seed, an offset in the counter's upper half. What is dropped
// counts for nothing, whatever its value.
//
// Memory bounds both: each row of x moves once, and dy once for eight of a
// token's slots (with more of them again for the next eight, generator included). A thread takes eight columns of a token; the loads of all its
// rows go out before the generator's words are worked out, and what does not
// count is masked afterwards: a branch per row would have the loads wait for each
// other. The last run of a row starts eight columns before its end, whatever the
// width, so that every run is whole; columns that two threads hold get the same
// value from both. 16384 x 2048 bf16, 8 experts: forward 124 us (5.4 TB/s; a plain
// copy reaches 5.0-5.2), backward 226-233 us (4.9 TB/s, 4 of them for the slots'
// places); dropout of 8192 x 7168 float32 91 us (5.2 TB/s), bf16 60 us, where the
// generator's instructions count (38 without them); of 333 x 2047 float32 5.4 us
// with its call. Sums are float32 and each result is rounded once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

constexpr int kThreads = 256;

// Four words of one counter block.
// The 64-bit products and the three-way exclusive ors are one instruction each.
__device__ inline u32x4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = uint64_t(0xD2511F53u) * c0, q = uint64_t(0xCD9E8D57u) * c2;
    c0 = __builtin_amdgcn_bitop3_b32(uint32_t(q >> 32), c1, k0, 0x96);  // the exclusive or of the three
    c1 = uint32_t(q);
    c2 = __builtin_amdgcn_bitop3_b32(uint32_t(p >> 32), c3, k1, 0x96);
    c3 = uint32_t(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Which of the eight elements from `first` on are kept.
__device__ inline void kept8(uint64_t first, uint64_t offset, uint64_t seed, uint32_t threshold, bool (&k)[8]) {
  const uint64_t block = first >> 2;
  const u32x4 w0 = philox(block, offset, seed), w1 = philox(block + 1, offset, seed);
#pragma unroll
  for (int e = 0; e < 8; ++e) k[e] = (e < 4 ? w0[e] : w1[e - 4]) >= threshold;
  const int skip = int(first & 3);
  if (__ballot(skip != 0) == 0) return;  // of the whole wave, as in rows of a multiple of four
  asm volatile("");  // a branch: no third block otherwise
  const u32x4 w2 = philox(block + 2, offset, seed);
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 12; ++e) bits |= (e < 8 ? k[e < 8 ? e : 0] : w2[e & 3] >= threshold) ? 1u << e : 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) k[e] = bits >> (skip + e) & 1;
}

// A thread's run of columns: kPerRow threads make a row, kThreads / kPerRow rows
// a workgroup.
struct Run {
  int c, own;  // first column; the first of the eight that no earlier run holds
};
__device__ inline Run run_at(int c, int cols) {
  const int last = cols > 8 ? cols - 8 : 0;
  return {c < last ? c : last, c < last ? 0 : c - last};
}
// kTiny: rows of fewer than eight columns.
template <bool kTiny, typename T>
__device__ inline Raw8<T> load_run(const T *p, int cols) {
  return kTiny ? load8(p, cols) : load8(p, 8);
}
template <bool kTiny, typename T>
__device__ inline void store_run(T *p, const float (&f)[8], int cols) {
  store8(p, pack8(f, T()), kTiny ? cols : 8);
}
__device__ inline void keep(Raw8<__bf16> &r, uint32_t mask) { r.v &= mask; }
__device__ inline void keep(Raw8<float> &r, uint32_t mask) {
  r.v[0] &= mask;
  r.v[1] &= mask;
}

// The slot of a token's choice j (past its last one: that).
template <int kJ>
__device__ inline int64_t slot_of(const CombineArgs &a, int64_t t, int j) {
  return t * a.topk + (kJ == 1 || j < a.topk ? j : a.topk - 1);
}
// Weights and indices of kJ choices, all loads of one list out together.
template <int kJ>
__device__ inline void choices(const CombineArgs &a, int64_t t, int j0, float (&w)[kJ], int32_t (&idx)[kJ]) {
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    w[j] = 1.f;
    idx[j] = 0;
  }
  if (a.weights) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) w[j] = a.weights[slot_of<kJ>(a, t, j0 + j)];
  }
  if (a.indices) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) idx[j] = a.indices[slot_of<kJ>(a, t, j0 + j)];
  }
}

// kJ: rows of a token whose loads are under way together, 1, 4 or 8 (dropout has
// one row); kPerRow: 8, 64 or 256 threads, the fewest that take a row of up to
// 64, 512 or more columns in one run each (above 2048 in several).
template <typename T, int kPerRow, int kJ, bool kTiny>
__global__ __launch_bounds__(kThreads) void combine_fwd_kernel(const CombineArgs a) {
  const bool drop = a.key != nullptr;
  const uint64_t seed = drop ? a.key[0] : 0, offset = drop ? a.key[1] : 0;
  constexpr int kRows = kThreads / kPerRow;
  const T *xs = static_cast<const T *>(a.x);
  for (int64_t t = int64_t(blockIdx.x) * kRows + int(threadIdx.x) / kPerRow; t < a.tokens; t += int64_t(gridDim.x) * kRows) {
    for (int c0 = (int(threadIdx.x) % kPerRow + int(blockIdx.y) * kPerRow) * 8; c0 < a.cols; c0 += int(gridDim.y) * kPerRow * 8) {
      const int c = run_at(c0, a.cols).c;
      Raw8<T> res{};
      if (a.res) res = load_run<kTiny>(static_cast<const T *>(a.res) + t * a.ld_res + c, a.cols);
      float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      bool kept[8] = {true, true, true, true, true, true, true, true};
      for (int j0 = 0; j0 < a.topk; j0 += kJ) {
        Raw8<T> x[kJ];
        float w[kJ];
        int32_t idx[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) x[j] = load_run<kTiny>(xs + slot_of<kJ>(a, t, j0 + j) * a.ld_x + c, a.cols);
        choices(a, t, j0, w, idx);
        if (drop && j0 == 0) {
          asm volatile("");  // a branch: no words where nothing is dropped
          kept8(uint64_t(t) * uint64_t(a.cols) + c, offset, seed, a.threshold, kept);
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const bool there = idx[j] >= 0 && (kJ == 1 || j0 + j < a.topk);
          keep(x[j], there ? ~0u : 0u);
          w[j] = there ? w[j] : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[j], x[j].get(e), sum[e]);
        }
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = res.get(e) + (kept[e] ? sum[e] * a.scale : 0.f);
      store_run<kTiny>(static_cast<T *>(a.out) + t * a.ld_out + c, y, a.cols);
    }
  }
}

// The place of each slot in `rows`, for the kernel that goes by slot.
__global__ __launch_bounds__(kThreads) void places_kernel(const CombineArgs a) {
  const int64_t slots = a.tokens * a.topk;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < slots; i += int64_t(gridDim.x) * kThreads) {
    const int32_t slot = a.rows[i];
    if (slot >= 0 && slot < slots) a.places[slot] = int32_t(i);
  }
}

template <typename T, int kPerRow, int kJ, bool kTiny>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(const CombineArgs a) {
  constexpr int kWaves = kPerRow / 64, kRows = kThreads / kPerRow;  // waves of a row, rows of a workgroup
  __shared__ float part[kThreads / 64][kJ];
  const bool drop = a.key != nullptr;
  const uint64_t seed = drop ? a.key[0] : 0, offset = drop ? a.key[1] : 0;
  const int64_t slots = a.tokens * a.topk;
  const T *xs = static_cast<const T *>(a.x);
  // the waves of a workgroup stay together; rows past the last repeat it and write nothing
  for (int64_t t0 = int64_t(blockIdx.x) * kRows; t0 < a.tokens; t0 += int64_t(gridDim.x) * kRows) {
    const int64_t at = t0 + int(threadIdx.x) / kPerRow;
    const bool live = at < a.tokens;
    const int64_t t = live ? at : a.tokens - 1;
    for (int j0 = 0; j0 < a.topk; j0 += kJ) {
      // a run's loads go out before what the run before it, or the token's lists, need
      Raw8<T> dy, x[kJ];
      auto load = [&](int c0) {
        const int c = run_at(c0, a.cols).c;
        dy = load_run<kTiny>(static_cast<const T *>(a.dy) + t * a.ld_dy + c, a.cols);
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) x[j] = load_run<kTiny>(xs + slot_of<kJ>(a, t, j0 + j) * a.ld_x + c, a.cols);
        }
      };
      const int begin = int(threadIdx.x) % kPerRow * 8;
      load(begin < a.cols ? begin : 0);
      int32_t to[kJ], idx[kJ];  // row of dx, -1: none
      float w[kJ], dot[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        to[j] = int32_t(slot_of<kJ>(a, t, j0 + j));
        dot[j] = 0.f;
      }
      choices(a, t, j0, w, idx);
      if (a.rows) {  // a slot that rows does not hold has found no place: its entry is whatever was there
        int32_t back[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) to[j] = a.places[to[j]];
#pragma unroll
        for (int j = 0; j < kJ; ++j) back[j] = a.rows[to[j] >= 0 && to[j] < slots ? to[j] : 0];
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          to[j] = to[j] >= 0 && to[j] < slots && back[j] == int32_t(slot_of<kJ>(a, t, j0 + j)) ? to[j] : -1;
      }
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const bool there = live && idx[j] >= 0 && (kJ == 1 || j0 + j < a.topk);
        idx[j] = there ? 0 : -1;
        to[j] = there ? to[j] : -1;
      }
      for (int c0 = begin; c0 < a.cols; c0 += kPerRow * 8) {
        const Run run = run_at(c0, a.cols);
        bool kept[8] = {true, true, true, true, true, true, true, true};
        if (drop) {
          asm volatile("");
          kept8(uint64_t(t) * uint64_t(a.cols) + run.c, offset, seed, a.threshold, kept);
        }
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = kept[e] ? dy.get(e) * a.scale : 0.f;
        if (a.dweights) {
#pragma unroll
          for (int e = 0; e < 8; ++e) kept[e] = kept[e] && e >= run.own;
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            keep(x[j], idx[j] >= 0 ? ~0u : 0u);
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += kept[e] ? x[j].get(e) * d[e] : 0.f;
            dot[j] += s;
          }
        }
        if (c0 + kPerRow * 8 < a.cols) load(c0 + kPerRow * 8);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          if (to[j] >= 0) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = w[j] * d[e];
            store_run<kTiny>(static_cast<T *>(a.out) + int64_t(to[j]) * a.ld_out + run.c, v, a.cols);
          }
        }
      }
      if (!a.dweights) continue;
      // sums over the row's threads
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        if constexpr (kPerRow >= 64) {
          dot[j] = wave_sum(dot[j]);
        } else {
#pragma unroll
          for (int m = 1; m < kPerRow; m *= 2) dot[j] += __shfl_xor(dot[j], m);
        }
      }
      if constexpr (kWaves > 1) {
        const int wave = int(threadIdx.x) >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) part[wave][j] = dot[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          dot[j] = 0.f;
#pragma unroll
          for (int i = 0; i < kWaves; ++i) dot[j] += part[wave / kWaves * kWaves + i][j];
        }
      }
      if (live && int(threadIdx.x) % kPerRow == 0) {
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          if (j0 + j < a.topk) a.dweights[t * a.topk + j0 + j] = idx[j] >= 0 ? dot[j] : 0.f;
      }
    }
  }
}

template <bool kBack, typename T, int kPerRow, int kJ, bool kTiny>
void go(const CombineArgs &a, hipStream_t s) {
  const int64_t rows = kThreads / kPerRow;
  const unsigned blocks = unsigned(std::min<int64_t>((a.tokens + rows - 1) / rows, 1 << 20));
  if constexpr (kBack) {
    hipLaunchKernelGGL((combine_bwd_kernel<T, kPerRow, kJ, kTiny>), dim3(blocks), dim3(kThreads), 0, s, a);
  } else {
    const int across = std::min((a.cols + kPerRow * 8 - 1) / (kPerRow * 8), 64);
    hipLaunchKernelGGL((combine_fwd_kernel<T, kPerRow, kJ, kTiny>), dim3(blocks, unsigned(across)), dim3(kThreads), 0, s, a);
  }
}
template <bool kBack, typename T, int kPerRow, bool kTiny>
void by_topk(const CombineArgs &a, hipStream_t s) {
  if (a.topk == 1)
    go<kBack, T, kPerRow, 1, kTiny>(a, s);
  else if (a.topk <= 4)
    go<kBack, T, kPerRow, 4, kTiny>(a, s);
  else
    go<kBack, T, kPerRow, 8, kTiny>(a, s);
}

template <bool kBack, typename T>
hipError_t combine(const CombineArgs &a, hipStream_t s) {
  if (kBack && a.rows) {
    const int64_t blocks = std::min<int64_t>((a.tokens * a.topk + kThreads - 1) / kThreads, 4096);
    hipLaunchKernelGGL(places_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.cols < 8)
    by_topk<kBack, T, 8, true>(a, s);
  else if (a.cols <= 64)
    by_topk<kBack, T, 8, false>(a, s);
  else if (a.cols <= 512)
    by_topk<kBack, T, 64, false>(a, s);
  else
    by_topk<kBack, T, 256, false>(a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_fwd(const CombineArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? combine<false, __bf16>(a, s) : combine<false, float>(a, s);
}

hipError_t launch_combine_bwd(const CombineArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? combine<true, __bf16>(a, s) : combine<true, float>(a, s);
}

}  // namespace muon
