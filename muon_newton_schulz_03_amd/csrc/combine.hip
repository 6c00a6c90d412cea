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
// Memory bounds both: each row of x moves once, and dy once for all of a
// token's slots.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;  // rows of a token whose loads are under way together

// Four words of one counter block.
__device__ inline u32x4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = uint64_t(0xD2511F53u) * c0, q = uint64_t(0xCD9E8D57u) * c2;
    c0 = uint32_t(q >> 32) ^ c1 ^ k0;
    c1 = uint32_t(q);
    c2 = uint32_t(p >> 32) ^ c3 ^ k1;
    c3 = uint32_t(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Which of the eight elements from `first` on are kept, a bit each.
__device__ inline uint32_t kept8(uint64_t first, uint64_t offset, uint64_t seed, uint32_t threshold) {
  const uint64_t block = first >> 2;
  const int skip = int(first & 3);
  uint32_t bits = 0;
#pragma unroll
  for (int b = 0; b < 3; ++b) {
    if (b == 2 && skip == 0) break;
    const u32x4 w = philox(block + b, offset, seed);
#pragma unroll
    for (int e = 0; e < 4; ++e) bits |= (w[e] >= threshold ? 1u : 0u) << (4 * b + e);
  }
  return bits >> skip;
}

// kPerRow threads make a row (of 256; from 64 on whole waves, so that what
// belongs to a token is scalar), kThreads / kPerRow rows a workgroup.
template <int kPerRow>
__device__ inline int64_t first_token() {
  int64_t t = int64_t(blockIdx.x) * (kThreads / kPerRow) + int(threadIdx.x) / kPerRow;
  if constexpr (kPerRow >= 64) t = int64_t(blockIdx.x) * (kThreads / kPerRow) + __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kPerRow);
  return t;
}

template <typename T, int kPerRow>
__global__ __launch_bounds__(kThreads) void combine_fwd_kernel(const CombineArgs a) {
  const bool drop = a.key != nullptr;
  const uint64_t seed = drop ? a.key[0] : 0, offset = drop ? a.key[1] : 0;
  for (int64_t t = first_token<kPerRow>(); t < a.tokens; t += int64_t(gridDim.x) * (kThreads / kPerRow)) {
    for (int c = (int(threadIdx.x) % kPerRow + int(blockIdx.y) * kPerRow) * 8; c < a.cols; c += int(gridDim.y) * kPerRow * 8) {
      const int left = a.cols - c;
      Raw8<T> res{};
      if (a.res) res = load8(static_cast<const T *>(a.res) + t * a.ld_res + c, left);
      const uint32_t kept = drop ? kept8(uint64_t(t) * uint64_t(a.cols) + c, offset, seed, a.threshold) : 255u;
      float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
        Raw8<T> x[kAtOnce];
        float w[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int64_t slot = t * a.topk + j0 + j;
          const bool there = j0 + j < a.topk && (!a.indices || a.indices[slot] >= 0);
          x[j] = Raw8<T>{};
          w[j] = 0.f;
          if (there) {
            x[j] = load8(static_cast<const T *>(a.x) + slot * a.ld_x + c, left);
            w[j] = a.weights ? a.weights[slot] : 1.f;
          }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[j], x[j].get(e), sum[e]);
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = res.get(e) + (kept >> e & 1 ? sum[e] * a.scale : 0.f);
      store8(static_cast<T *>(a.out) + t * a.ld_out + c, pack8(y, T()), left);
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

template <typename T, int kPerRow>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(const CombineArgs a) {
  constexpr int kWaves = kPerRow / 64;  // of a row
  __shared__ float part[kThreads / 64][kAtOnce];
  const bool drop = a.key != nullptr;
  const uint64_t seed = drop ? a.key[0] : 0, offset = drop ? a.key[1] : 0;
  const int64_t slots = a.tokens * a.topk, step = int64_t(gridDim.x) * (kThreads / kPerRow);
  const int64_t own = first_token<kPerRow>();
  for (int64_t t0 = int64_t(blockIdx.x) * (kThreads / kPerRow); t0 < a.tokens; t0 += step) {  // the workgroup's waves stay together
    const int64_t t = own + (t0 - int64_t(blockIdx.x) * (kThreads / kPerRow));
    const bool live = t < a.tokens;
    for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
      int64_t to[kAtOnce];  // row of dx, -1: none
      float w[kAtOnce], dot[kAtOnce];
      bool there[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t slot = t * a.topk + j0 + j;
        there[j] = live && j0 + j < a.topk && (!a.indices || a.indices[slot] >= 0);
        dot[j] = w[j] = 0.f;
        to[j] = -1;
        if (there[j]) {
          w[j] = a.weights ? a.weights[slot] : 1.f;
          to[j] = slot;
          if (a.rows) {  // a slot that rows does not hold has found no place: its entry is whatever was there
            const int32_t p = a.places[slot];
            to[j] = p >= 0 && p < slots && a.rows[p] == int32_t(slot) ? p : -1;
          }
        }
      }
      if (live) {
        for (int c = int(threadIdx.x) % kPerRow * 8; c < a.cols; c += kPerRow * 8) {
          const int left = a.cols - c;
          const Raw8<T> dy = load8(static_cast<const T *>(a.dy) + t * a.ld_dy + c, left);
          Raw8<T> x[kAtOnce];
          if (a.dweights) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              x[j] = Raw8<T>{};
              if (there[j]) x[j] = load8(static_cast<const T *>(a.x) + (t * a.topk + j0 + j) * a.ld_x + c, left);
            }
          }
          const uint32_t kept = drop ? kept8(uint64_t(t) * uint64_t(a.cols) + c, offset, seed, a.threshold) : 255u;
          float d[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = kept >> e & 1 ? dy.get(e) * a.scale : 0.f;
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            if (a.dweights) {
              float s = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) s += kept >> e & 1 ? x[j].get(e) * d[e] : 0.f;
              dot[j] += s;
            }
            if (to[j] >= 0) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = w[j] * d[e];
              store8(static_cast<T *>(a.out) + to[j] * a.ld_out + c, pack8(v, T()), left);
            }
          }
        }
      }
      if (!a.dweights) continue;
      // sums over the row's threads
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
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
          for (int j = 0; j < kAtOnce; ++j) part[wave][j] = dot[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          dot[j] = 0.f;
#pragma unroll
          for (int i = 0; i < kWaves; ++i) dot[j] += part[wave / kWaves * kWaves + i][j];
        }
      }
      if (live && int(threadIdx.x) % kPerRow == 0) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (j0 + j < a.topk) a.dweights[t * a.topk + j0 + j] = there[j] ? dot[j] : 0.f;
      }
    }
  }
}


template <typename T, int kPerRow>
void fwd(const CombineArgs &a, hipStream_t s) {
  const int64_t rows = kThreads / kPerRow;
  const int64_t blocks = std::min<int64_t>((a.tokens + rows - 1) / rows, 1 << 20);
  const int across = std::min((a.cols + kPerRow * 8 - 1) / (kPerRow * 8), 64);
  hipLaunchKernelGGL((combine_fwd_kernel<T, kPerRow>), dim3(unsigned(blocks), unsigned(across)), dim3(kThreads), 0, s, a);
}

template <typename T, int kPerRow>
void bwd(const CombineArgs &a, hipStream_t s) {
  const int64_t rows = kThreads / kPerRow;
  const int64_t blocks = std::min<int64_t>((a.tokens + rows - 1) / rows, 1 << 20);
  hipLaunchKernelGGL((combine_bwd_kernel<T, kPerRow>), dim3(unsigned(blocks)), dim3(kThreads), 0, s, a);
}

template <typename T>
hipError_t forward(const CombineArgs &a, hipStream_t s) {
  if (a.cols <= 64)
    fwd<T, 8>(a, s);
  else if (a.cols <= 512)
    fwd<T, 64>(a, s);
  else
    fwd<T, 256>(a, s);
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const CombineArgs &a, hipStream_t s) {
  if (a.rows) {
    const int64_t blocks = std::min<int64_t>((a.tokens * a.topk + kThreads - 1) / kThreads, 4096);
    hipLaunchKernelGGL(places_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.cols <= 64)
    bwd<T, 8>(a, s);
  else if (a.cols <= 512)
    bwd<T, 64>(a, s);
  else
    bwd<T, 256>(a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_fwd(const CombineArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? forward<__bf16>(a, s) : forward<float>(a, s);
}

hipError_t launch_combine_bwd(const CombineArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? backward<__bf16>(a, s) : backward<float>(a, s);
}

}  // namespace muon
