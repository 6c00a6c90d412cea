// Expert routing (gfx950): softmax over the experts, the top-k choice, the
// per-expert counts and slot lists, the balance loss, and the gradient of
// loss and weights.
//
//   p = softmax(x);  choice: the k largest logits, the lower index first
//   among equals, never -inf or NaN;  weights: p of the choice, or its share
//   of the choice's sum;
//   loss = alpha E / (k n) sum_e counts_e (sum_t p_te / n)  over the n tokens
//   that have a choice;
//   d_e = dloss alpha E counts_e / (k n^2);  dx = p (d - sum p d) plus, for
//   the weights' gradient g, d + g at the choice (plain weights) or
//   w (g - sum w g) at the choice (shares).
//
// One wave holds a token's logits, expert j * 64 + lane in register j. The
// slot lists are stable (expert order, then slot order) without atomics on
// the result: workgroups count their tokens' choices, the counts are summed
// over workgroups in order, and inside a workgroup a slot's rank is the
// number of lower bits in its expert's mask of tokens.
#include <hip/hip_runtime.h>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

constexpr int kThreads = 1024;  // forward: 16 waves
constexpr int kWaves = kThreads / 64;
constexpr int kSub = 64;        // tokens ranked at a time (two mask words an expert)
constexpr float kNegInf = -__builtin_inff();

__device__ inline float wave_max(float v) {
  v = fmaxf(v, dpp<kQuadSwap1>(v));
  v = fmaxf(v, dpp<kQuadSwap2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  v = fmaxf(v, dpp<kMirror>(v));
  v = fmaxf(v, __shfl_xor(v, 16));
  v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}

template <typename T, int kJ>
__device__ inline void load_logits(const T *p, int experts, int lane, float (&x)[kJ]) {
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = j * 64 + lane;
    x[j] = e < experts ? float(p[e]) : kNegInf;
  }
}

// p[j] = softmax; returns the row's maximum (NaN ignored), and the base and
// reciprocal that give p of any logit as exp(x - base) * inv.
template <int kJ>
__device__ inline float softmax(const float (&x)[kJ], float (&p)[kJ], float &base, float &inv) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < kJ; ++j) m = fmaxf(m, x[j]);
  m = wave_max(m);
  base = m == kNegInf ? 0.f : m;  // a row of -inf: every p is 0
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    p[j] = expf(x[j] - base);
    s += p[j];
  }
  s = wave_sum(s);
  inv = s == 0.f ? 1.f : 1.f / s;
#pragma unroll
  for (int j = 0; j < kJ; ++j) p[j] *= inv;
  return m;
}

struct RouteLds {
  int hist[kRouteMaxExperts];           // counts, or running counts
  float psum[kRouteMaxExperts];
  int offs[kRouteMaxExperts + 1];
  uint32_t mask[kRouteMaxExperts][kSub / 32];
  int scan[kThreads / 64 + 1];
  int valid;
};

// The choice, weights, counts and sums of tokens [begin, end).
template <typename T, int kJ>
__device__ void route_tokens(const RouteFwdArgs &a, int begin, int end, RouteLds &lds) {
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) {
    lds.hist[e] = 0;
    lds.psum[e] = 0.f;
  }
  if (threadIdx.x == 0) lds.valid = 0;
  __syncthreads();
  float ps[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) ps[j] = 0.f;
  int valid = 0;
  for (int t = begin + wave; t < end; t += kWaves) {
    float x[kJ], p[kJ], base, inv;
    load_logits<T, kJ>(static_cast<const T *>(a.logits) + int64_t(t) * a.ld, a.experts, lane, x);
    float m = softmax<kJ>(x, p, base, inv);
#pragma unroll
    for (int j = 0; j < kJ; ++j) ps[j] += p[j];
    valid += m > kNegInf ? 1 : 0;
    int mine = -1;
    float w = 0.f, share = 0.f;
    for (int i = 0; i < a.topk; ++i) {
      if (!(m > kNegInf)) break;  // nothing left to choose
      int idx = -1;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const uint64_t b = __ballot(x[j] == m);
        if (idx < 0 && b) idx = j * 64 + __builtin_ctzll(b);
      }
      const float pw = expf(m - base) * inv;
      share += pw;
      if (lane == i) {
        mine = idx;
        w = pw;
      }
      float next = kNegInf;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        x[j] = j * 64 + lane == idx ? kNegInf : x[j];
        next = fmaxf(next, x[j]);
      }
      if (i + 1 < a.topk) m = wave_max(next);
    }
    if (a.renorm) w /= share == 0.f ? 1.f : share;
    if (lane < a.topk) {
      a.indices[int64_t(t) * a.topk + lane] = mine;
      a.weights[int64_t(t) * a.topk + lane] = w;
      if (mine >= 0) atomicAdd(&lds.hist[mine], 1);
    }
  }
  if (lane == 0 && valid) atomicAdd(&lds.valid, valid);
  for (int v = 0; v < kWaves; ++v) {  // in wave order: the same sum in every run
    if (wave == v) {
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (j * 64 + lane < a.experts) lds.psum[j * 64 + lane] += ps[j];
    }
    __syncthreads();
  }
}

// Exclusive scan of counts (a.experts of them, in LDS or global memory) into
// lds.offs.
__device__ void scan_counts(const int *counts, int experts, RouteLds &lds) {
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  const int e = int(threadIdx.x);
  const int c = e < experts ? counts[e] : 0;
  int v = c;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  if (lane == 63) lds.scan[wave] = v;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += lds.scan[w];
  if (e < experts) lds.offs[e] = before + v - c;
  if (e == experts - 1) lds.offs[experts] = before + v;
  __syncthreads();
}

// Writes the slots of tokens [begin, end) to their places: lds.offs[e] plus
// lds.hist[e], the slots of expert e that earlier tokens have.
__device__ void place_slots(const RouteFwdArgs &a, int begin, int end, RouteLds &lds) {
  for (int sub = begin; sub < end; sub += kSub) {
    for (int i = int(threadIdx.x); i < a.experts * (kSub / 32); i += kThreads) (&lds.mask[0][0])[i] = 0;
    __syncthreads();
    const int n = (end - sub < kSub ? end - sub : kSub) * a.topk;
    for (int i = int(threadIdx.x); i < n; i += kThreads) {
      const int e = a.indices[int64_t(sub) * a.topk + i], t = i / a.topk;
      if (e >= 0) atomicOr(&lds.mask[e][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    for (int i = int(threadIdx.x); i < n; i += kThreads) {
      const int e = a.indices[int64_t(sub) * a.topk + i], t = i / a.topk;
      if (e < 0) continue;
      int rank = __popc(lds.mask[e][t >> 5] & ((1u << (t & 31)) - 1));
      if (t >= 32) rank += __popc(lds.mask[e][0]);
      a.rows[lds.offs[e] + lds.hist[e] + rank] = sub * a.topk + i;
    }
    __syncthreads();
    for (int e = int(threadIdx.x); e < a.experts; e += kThreads)
      lds.hist[e] += __popc(lds.mask[e][0]) + __popc(lds.mask[e][1]);
    __syncthreads();
  }
}

__device__ inline int counted(const RouteFwdArgs &a) { return a.tokens * a.topk; }

// counts, offsets and the loss, by one workgroup: lds.offs is set, counts and
// psum hold the totals.
__device__ void finish(const RouteFwdArgs &a, const int *counts, const float *psum, int valid, RouteLds &lds) {
  const float n = float(valid > 0 ? valid : 1);
  float s = 0.f;
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) {
    s += float(counts[e]) * (psum[e] / n);
    a.offsets[e] = lds.offs[e];
  }
  s = wave_sum(s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds.psum[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x) return;
  s = 0.f;
  for (int w = 0; w < kWaves; ++w) s += lds.psum[w];
  a.offsets[a.experts] = lds.offs[a.experts];
  a.counts[a.experts] = valid;
  a.loss[0] = a.alpha * float(a.experts) / (float(a.topk) * n) * s;
}

// A few tokens: everything in one launch of one workgroup.
template <typename T, int kJ>
__global__ __launch_bounds__(kThreads) void route_one_kernel(const RouteFwdArgs a) {
  __shared__ RouteLds lds;
  route_tokens<T, kJ>(a, 0, a.tokens, lds);
  scan_counts(lds.hist, a.experts, lds);
  const int total = lds.offs[a.experts];
  for (int i = total + int(threadIdx.x); i < counted(a); i += kThreads) a.rows[i] = -1;
  const int valid = lds.valid;
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) a.counts[e] = lds.hist[e];
  __threadfence_block();  // indices written by other waves of this workgroup are read below
  finish(a, lds.hist, lds.psum, valid, lds);
  __syncthreads();
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) lds.hist[e] = 0;
  __syncthreads();
  place_slots(a, 0, a.tokens, lds);
}

// Many tokens, first launch: each workgroup's tokens, counts and sums.
template <typename T, int kJ>
__global__ __launch_bounds__(kThreads) void route_tokens_kernel(const RouteFwdArgs a) {
  __shared__ RouteLds lds;
  const int begin = int(blockIdx.x) * a.per_block;
  const int end = begin + a.per_block < a.tokens ? begin + a.per_block : a.tokens;
  route_tokens<T, kJ>(a, begin, end, lds);
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) {
    a.hist[int64_t(blockIdx.x) * a.experts + e] = lds.hist[e];
    a.psum[int64_t(blockIdx.x) * a.experts + e] = lds.psum[e];
  }
  if (threadIdx.x == 0) a.valid[blockIdx.x] = lds.valid;
}

// Second launch: over the workgroups, hist becomes its exclusive prefix sum
// and row 0 of psum the total, 16 experts a workgroup and 16 threads an
// expert, each over a run of consecutive workgroups.
constexpr int kScanExperts = 16, kScanSlices = 16;
__global__ __launch_bounds__(kScanExperts * kScanSlices) void route_scan_kernel(const RouteFwdArgs a) {
  __shared__ int cnt[kScanSlices][kScanExperts];
  __shared__ float sum[kScanSlices][kScanExperts];
  const int le = int(threadIdx.x) % kScanExperts, sl = int(threadIdx.x) / kScanExperts;
  const int e = int(blockIdx.x) * kScanExperts + le;
  const int per = (a.blocks + kScanSlices - 1) / kScanSlices;
  const int b0 = sl * per, b1 = b0 + per < a.blocks ? b0 + per : a.blocks;
  int c = 0;
  float s = 0.f;
  if (e < a.experts) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
      c += a.hist[int64_t(b) * a.experts + e];
      s += a.psum[int64_t(b) * a.experts + e];
    }
  }
  cnt[sl][le] = c;
  sum[sl][le] = s;
  __syncthreads();
  if (e < a.experts) {
    int before = 0, total = 0;
    float all = 0.f;
    for (int j = 0; j < kScanSlices; ++j) {
      before += j < sl ? cnt[j][le] : 0;
      total += cnt[j][le];
      all += sum[j][le];
    }
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
      const int h = a.hist[int64_t(b) * a.experts + e];
      a.hist[int64_t(b) * a.experts + e] = before;
      before += h;
    }
    if (sl == 0) {
      a.counts[e] = total;
      a.psum[e] = all;  // row 0: its own slice has read it
    }
  }
  if (blockIdx.x == 0) {
    __syncthreads();
    int v = 0;
    for (int b = int(threadIdx.x); b < a.blocks; b += kScanExperts * kScanSlices) v += a.valid[b];
    (&cnt[0][0])[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      v = 0;
      for (int i = 0; i < kScanExperts * kScanSlices; ++i) v += (&cnt[0][0])[i];
      a.counts[a.experts] = v;
    }
  }
}

// Third launch: the slot lists; the first workgroup also offsets and loss.
__global__ __launch_bounds__(kThreads) void route_place_kernel(const RouteFwdArgs a) {
  __shared__ RouteLds lds;
  scan_counts(a.counts, a.experts, lds);
  if (blockIdx.x == 0) finish(a, a.counts, a.psum, a.counts[a.experts], lds);
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads)
    lds.hist[e] = a.hist[int64_t(blockIdx.x) * a.experts + e];
  const int begin = int(blockIdx.x) * a.per_block;
  const int end = begin + a.per_block < a.tokens ? begin + a.per_block : a.tokens;
  const int total = lds.offs[a.experts];
  for (int i = begin * a.topk + int(threadIdx.x); i < end * a.topk; i += kThreads)
    if (i >= total) a.rows[i] = -1;
  __syncthreads();
  place_slots(a, begin, end, lds);
}

// LDS that lanes of one wave hand each other: orders the compiler's view (the
// hardware runs a wave's LDS accesses in order).
__device__ inline void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

constexpr int kBwdThreads = 256;
template <typename T, int kJ>
__global__ __launch_bounds__(kBwdThreads) void route_bwd_kernel(const RouteBwdArgs a) {
  __shared__ float extra[kBwdThreads / 64][kJ * 64];
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  float *mine = extra[wave];
  // the loss's part of d, the same for every token
  float dl[kJ];
  const float n = float(a.counts[a.experts] > 0 ? a.counts[a.experts] : 1);
  const float coef = a.dloss ? a.dloss[0] * (a.alpha * float(a.experts) / float(a.topk)) / (n * n) : 0.f;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = j * 64 + lane;
    dl[j] = a.dloss && e < a.experts ? coef * float(a.counts[e]) : 0.f;
  }
  const int waves = int(gridDim.x) * (kBwdThreads / 64);
  for (int t = int(blockIdx.x) * (kBwdThreads / 64) + wave; t < a.tokens; t += waves) {
    wave_fence();  // the last token's reads of `mine` are done
    const T *row = static_cast<const T *>(a.logits) + int64_t(t) * a.ld;
    float x[kJ], p[kJ], d[kJ], base, inv;
    load_logits<T, kJ>(row, a.experts, lane, x);
    int idx = -1;
    float g = 0.f, xi = kNegInf;
    if (a.dweights && lane < a.topk) {
      idx = a.indices[int64_t(t) * a.topk + lane];
      if (idx >= a.experts) idx = -1;
      if (idx >= 0) {
        g = a.dweights[int64_t(t) * a.topk + lane];
        xi = float(row[idx]);
      }
    }
    softmax<kJ>(x, p, base, inv);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      d[j] = dl[j];
      mine[j * 64 + lane] = 0.f;
    }
    wave_fence();
    if (a.dweights) {
      float add = g;
      if (a.renorm) {
        float w = idx >= 0 ? expf(xi - base) * inv : 0.f;
        const float share = wave_sum(w);
        w /= share == 0.f ? 1.f : share;
        add = w * (g - wave_sum(w * g));
      }
      if (idx >= 0) atomicAdd(&mine[idx], add);
    }
    wave_fence();
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (!a.renorm) d[j] += mine[j * 64 + lane];
      s = fmaf(d[j], p[j], s);
    }
    s = wave_sum(s);
    T *out = static_cast<T *>(a.dlogits) + int64_t(t) * a.ld_out;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int e = j * 64 + lane;
      float v = p[j] * (d[j] - s);
      if (a.renorm) v += mine[e];
      if (e < a.experts) out[e] = T(v);
    }
  }
}

template <typename F>
auto by_experts(int experts, F &&f) {
  if (experts <= 64) return f(std::integral_constant<int, 1>());
  if (experts <= 128) return f(std::integral_constant<int, 2>());
  if (experts <= 256) return f(std::integral_constant<int, 4>());
  if (experts <= 384) return f(std::integral_constant<int, 6>());
  if (experts <= 512) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}

template <typename T>
hipError_t route_fwd(const RouteFwdArgs &a, hipStream_t s) {
  return by_experts(a.experts, [&](auto kj) {
    constexpr int kJ = decltype(kj)::value;
    if (a.blocks == 0) {
      hipLaunchKernelGGL((route_one_kernel<T, kJ>), dim3(1), dim3(kThreads), 0, s, a);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((route_tokens_kernel<T, kJ>), dim3(unsigned(a.blocks)), dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_scan_kernel, dim3((a.experts + kScanExperts - 1) / kScanExperts),
                       dim3(kScanExperts * kScanSlices), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_place_kernel, dim3(unsigned(a.blocks)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t route_bwd(const RouteBwdArgs &a, hipStream_t s) {
  return by_experts(a.experts, [&](auto kj) {
    constexpr int kJ = decltype(kj)::value;
    const int64_t want = (int64_t(a.tokens) + 3) / 4;
    hipLaunchKernelGGL((route_bwd_kernel<T, kJ>), dim3(unsigned(want < 2048 ? want : 2048)), dim3(kBwdThreads), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

// One workgroup takes up to 128 tokens (blocks = 0: no scratch); above, each
// takes a multiple of 64, at most 1024 workgroups.
void route_plan(RouteFwdArgs &a) {
  a.blocks = 0;
  a.per_block = a.tokens;
  if (a.tokens <= 128) return;
  const int64_t subs = (int64_t(a.tokens) + kSub - 1) / kSub;
  const int64_t each = (subs + 1023) / 1024;
  a.per_block = int32_t(each * kSub);
  a.blocks = int32_t((int64_t(a.tokens) + a.per_block - 1) / a.per_block);
}

hipError_t launch_route_fwd(const RouteFwdArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? route_fwd<__bf16>(a, s) : route_fwd<float>(a, s);
}

hipError_t launch_route_bwd(const RouteBwdArgs &a, bool bf16, hipStream_t s) {
  if (a.tokens <= 0) return hipSuccess;
  return bf16 ? route_bwd<__bf16>(a, s) : route_bwd<float>(a, s);
}

}  // namespace muon
