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
// 16384 tokens to 8 of 384 experts, bf16: forward 24 us, of which the choice 15,
// the sums over workgroups 5 and the lists 4: bound by the instructions of the
// choice and by three launches, not by its 14 MB. Backward, float32, 13 us for
// 51 MB (4.0 TB/s). 32 tokens to 8 of 128, one launch: 7.6 us.
//
// Forward, 16 lanes hold a token's logits, four tokens a wave: each of the k
// rounds finds the maximum and its lowest index by lane permutations, and the
// instructions of a round serve four tokens. Backward, a wave holds one token.
// The slot lists are stable (expert order, then slot order) without atomics on
// the result: workgroups count their tokens' choices, the counts are summed
// over workgroups in order, and inside a workgroup a slot's rank is the
// number of lower bits in its expert's mask of tokens.
#include <hip/hip_runtime.h>

#include "lanes.h"
#include "train.h"

namespace muon {
namespace {

constexpr int kSub = 64;        // tokens ranked at a time (two mask words an expert)
constexpr float kNegInf = -__builtin_inff();

__device__ inline float wave_max(float v) {
  v = fmaxf(v, dpp<kQuadSwap1>(v));
  v = fmaxf(v, dpp<kQuadSwap2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  v = fmaxf(v, dpp<kMirror>(v));
  const Pair p = rows_16(v);
  const Pair q = halves_32(fmaxf(p.a, p.b));
  return fmaxf(q.a, q.b);
}

// Expert 64 j + lane in register j, -inf past the last. Every load is issued
// (past the end, of the last expert): one that a lane may skip would be waited
// for before the next.
template <typename T, int kJ>
__device__ inline void load_logits(const T *p, int experts, int lane, float (&x)[kJ]) {
  T raw[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = j * 64 + lane;
    raw[j] = p[e < experts ? e : experts - 1];
  }
#pragma unroll
  for (int j = 0; j < kJ; ++j) x[j] = j * 64 + lane < experts ? float(raw[j]) : kNegInf;
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

// A token's logits over a row of 16 lanes, in runs of eight experts: register j
// of lane l holds expert 8 l + expert_of(j).
__device__ constexpr int expert_of(int j) { return j / 8 * 128 + j % 8; }
template <typename T, int kJ>
__device__ inline void load_runs(const T *p, int experts, int l, float (&x)[kJ]) {
  Raw8<T> r[kJ / 8];
  if (experts % 8 == 0) {  // a run is there or not: past the end, the first one is read
#pragma unroll
    for (int c = 0; c < kJ / 8; ++c) {
      const int e = c * 128 + l * 8;
      r[c] = load8(p + (e < experts ? e : 0), 8);
    }
  } else {
#pragma unroll
    for (int c = 0; c < kJ / 8; ++c) r[c] = load8(p + c * 128 + l * 8, experts - c * 128 - l * 8);
  }
#pragma unroll
  for (int j = 0; j < kJ; ++j) x[j] = expert_of(j) + l * 8 < experts ? r[j / 8].get(j % 8) : kNegInf;
}

// Reductions of such a row (no traffic through LDS).
__device__ inline float row_max(float v) {
  v = fmaxf(v, dpp<kQuadSwap1>(v));
  v = fmaxf(v, dpp<kQuadSwap2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  return fmaxf(v, dpp<kMirror>(v));
}
__device__ inline float row_sum(float v) {
  v += dpp<kQuadSwap1>(v);
  v += dpp<kQuadSwap2>(v);
  v += dpp<kHalfMirror>(v);
  return v + dpp<kMirror>(v);
}
__device__ inline uint32_t row_max(uint32_t v) { return row16_max(v); }
__device__ inline uint32_t row_min(uint32_t v) {
  v = min(v, dpp<kQuadSwap1>(v));
  v = min(v, dpp<kQuadSwap2>(v));
  v = min(v, dpp<kHalfMirror>(v));
  return min(v, dpp<kMirror>(v));
}

// exp(d) for d <= 0: the product with log2 e in two parts, then the hardware's
// power of two. Ends at 2^-126, 28 decades below the smallest sum it joins.
__device__ inline float exp_sum(float d) {
  d = d < -200.f ? -200.f : d;  // -inf too; NaN stays
  const float hi = d * 1.44269502f;                               // log2 e rounded
  const float lo = fmaf(d, 1.44269502f, -hi) + d * 1.92596303e-8f;  // what the product and the constant lost
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.693147182f, e);
}

// Threads of the forward kernels: four tokens a wave; the wide forms hold 32 or
// more logits a lane and need more registers each.
template <int kJ>
constexpr int route_threads() { return kJ > 24 ? 512 : 1024; }

template <int kJ>
struct RouteLds {
  static constexpr int kWaves = route_threads<kJ>() / 64;
  int hist[kJ * 16];                    // counts, or running counts
  float psum[kJ * 16];
  int offs[kJ * 16 + 1];
  union {
    uint32_t mask[kJ * 16][kSub / 32];
    float wave_psum[kWaves][kJ * 16];
  };
  int scan[kWaves + 1];
  int valid;
};

// The choice, weights, counts and sums of tokens [begin, end).
template <typename T, int kJ>
__device__ void route_tokens(const RouteFwdArgs &a, int begin, int end, RouteLds<kJ> &lds) {
  constexpr int kThreads = route_threads<kJ>(), kWaves = kThreads / 64;
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6, l = lane & 15;
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) lds.hist[e] = 0;
  if (threadIdx.x == 0) lds.valid = 0;
  __syncthreads();
  float ps[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) ps[j] = 0.f;
  int valid = 0;
  for (int first = begin + wave * 4; first < end; first += kWaves * 4) {
    const int t = first + (lane >> 4);
    const T *logits = static_cast<const T *>(a.logits) + int64_t(t < end ? t : end - 1) * a.ld;
    float x[kJ], p[kJ], m = kNegInf, s = 0.f;
    load_runs<T, kJ>(logits, a.experts, l, x);
    // rows past the end count and choose nothing
    if (t >= end) {
#pragma unroll
      for (int j = 0; j < kJ; ++j) x[j] = kNegInf;
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) m = fmaxf(m, x[j]);
    m = row_max(m);
    const float base = m == kNegInf ? 0.f : m;  // a row of -inf: every p is 0
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      p[j] = exp_sum(x[j] - base);
      s += p[j];
    }
    s = row_sum(s);
    const float inv = s == 0.f ? 1.f : 1.f / s;
#pragma unroll
    for (int j = 0; j < kJ; ++j) ps[j] = fmaf(p[j], inv, ps[j]);
    valid += m > kNegInf ? 1 : 0;
    // choice i stays with lane i % 16 of the row
    int mine[2] = {-1, -1};
    float top[2] = {kNegInf, kNegInf};
    auto keep = [&](int i, int e, float v) {
      if (l != (i & 15)) return;
      if (i < 16) {
        mine[0] = e;
        top[0] = v;
      } else {
        mine[1] = e;
        top[1] = v;
      }
    };
    if constexpr (sizeof(T) == 2) {
      // bf16: the order of choice as one number, the value's bits (ascending with
      // it) above 1023 - e, 0 for what is never chosen. All differ, so the next
      // choice is the largest difference to this one that wraps below zero.
      uint32_t key[kJ], best = 0;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const uint32_t u = f32_bits(x[j] + 0.f) >> 16;  // -0 is 0
        const uint32_t up = u & 0x8000u ? u ^ 0xffffu : u | 0x8000u;
        key[j] = x[j] > kNegInf ? up << 10 | uint32_t(1023 - expert_of(j) - l * 8) : 0u;
        best = max(best, key[j]);
      }
      best = row_max(best);
      for (int i = 0; i < a.topk; ++i) {
        if (!__any(best != 0)) break;  // nothing left to choose
        const uint32_t up = best >> 10;
        if (best) keep(i, 1023 - int(best & 1023u), bits_f32((up & 0x8000u ? up & 0x7fffu : up ^ 0xffffu) << 16));
        uint32_t below = 0;
#pragma unroll
        for (int j = 0; j < kJ; ++j) below = max(below, key[j] - best);
        below = row_max(below);
        best = below & 0x80000000u ? best + below : 0u;
      }
    } else {
      for (int i = 0; i < a.topk; ++i) {
        if (!__any(m > kNegInf)) break;  // nothing left to choose
        uint32_t at = 0xffffu;
#pragma unroll
        for (int j = kJ - 1; j >= 0; --j) at = x[j] == m ? uint32_t(expert_of(j)) : at;
        const uint32_t e = row_min(at + uint32_t(l * 8));
        if (m > kNegInf) keep(i, int(e), m);
        const int gone = int(e) - l * 8;  // expert_of the register that holds it, in its lane
        m = kNegInf;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          x[j] = gone == expert_of(j) ? kNegInf : x[j];
          m = fmaxf(m, x[j]);
        }
        m = row_max(m);
      }
    }
    float w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = mine[h] >= 0 ? expf(top[h] - base) * inv : 0.f;
    if (a.renorm) {
      const float share = row_sum(w[0] + w[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) w[h] /= share == 0.f ? 1.f : share;
    }
    if (t < end) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 16 * h + l;
        if (i >= a.topk) break;
        a.indices[int64_t(t) * a.topk + i] = mine[h];
        a.weights[int64_t(t) * a.topk + i] = w[h];
        if (mine[h] >= 0) atomicAdd(&lds.hist[mine[h]], 1);
      }
    }
  }
  if (l == 0 && valid) atomicAdd(&lds.valid, valid);
  // the waves' sums, added in wave order: the same result in every run
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const Pair q = rows_16(ps[j]);
    const Pair h = halves_32(q.a + q.b);
    ps[j] = h.a + h.b;
    if (lane < 16) lds.wave_psum[wave][expert_of(j) + l * 8] = ps[j];
  }
  __syncthreads();
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += lds.wave_psum[w][e];
    lds.psum[e] = s;
  }
  __syncthreads();
}

// Exclusive scan of counts (a.experts of them, in LDS or global memory) into
// lds.offs.
template <int kJ>
__device__ void scan_counts(const int *counts, int experts, RouteLds<kJ> &lds) {
  // two neighbouring experts a thread: the wide forms have half the threads
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  const int e = int(threadIdx.x) * 2;
  const int c0 = e < experts ? counts[e] : 0, c = c0 + (e + 1 < experts ? counts[e + 1] : 0);
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
  const int at = before + v - c;
  if (e < experts) lds.offs[e] = at;
  if (e + 1 < experts) lds.offs[e + 1] = at + c0;
  if (e == experts - 1 || e + 1 == experts - 1) lds.offs[experts] = before + v;
  __syncthreads();
}

// Writes the slots of tokens [begin, end) to their places: lds.offs[e] plus
// lds.hist[e], the slots of expert e that earlier tokens have.
template <int kJ>
__device__ void place_slots(const RouteFwdArgs &a, int begin, int end, RouteLds<kJ> &lds) {
  constexpr int kThreads = route_threads<kJ>();
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
template <int kJ>
__device__ void finish(const RouteFwdArgs &a, const int *counts, const float *psum, int valid, RouteLds<kJ> &lds) {
  constexpr int kThreads = route_threads<kJ>(), kWaves = kThreads / 64;
  const float n = float(valid > 0 ? valid : 1);
  float s = 0.f;
  for (int e = int(threadIdx.x); e < a.experts; e += kThreads) {
    s += float(counts[e]) * (psum[e] / n);
    a.offsets[e] = lds.offs[e];
  }
  s = wave_sum(s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds.wave_psum[0][threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x) return;
  s = 0.f;
  for (int w = 0; w < kWaves; ++w) s += lds.wave_psum[0][w];
  a.offsets[a.experts] = lds.offs[a.experts];
  a.counts[a.experts] = valid;
  a.loss[0] = a.alpha * float(a.experts) / (float(a.topk) * n) * s;
}

// A few tokens: everything in one launch of one workgroup.
template <typename T, int kJ>
__global__ __launch_bounds__(route_threads<kJ>()) void route_one_kernel(const RouteFwdArgs a) {
  constexpr int kThreads = route_threads<kJ>();
  __shared__ RouteLds<kJ> lds;
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
__global__ __launch_bounds__(route_threads<kJ>()) void route_tokens_kernel(const RouteFwdArgs a) {
  constexpr int kThreads = route_threads<kJ>();
  __shared__ RouteLds<kJ> lds;
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
// and row 0 of psum the total, 16 experts a workgroup and 64 threads an
// expert, each over a run of consecutive workgroups.
constexpr int kScanExperts = 16, kScanSlices = 64;
constexpr int kMaxBlocks = 1024;
template <int kPer>  // workgroups a slice
__global__ __launch_bounds__(kScanExperts * kScanSlices) void route_scan_kernel(const RouteFwdArgs a) {
  __shared__ int cnt[kScanSlices][kScanExperts];
  __shared__ float sum[kScanSlices][kScanExperts];
  const int le = int(threadIdx.x) % kScanExperts, sl = int(threadIdx.x) / kScanExperts;
  const int e = int(blockIdx.x) * kScanExperts + le;
  const int b0 = sl * kPer, col = e < a.experts ? e : a.experts - 1;
  int h[kPer], c = 0;
  float p[kPer], s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {  // past the last workgroup: the last one's, not counted
    const int64_t at = int64_t(b0 + i < a.blocks ? b0 + i : a.blocks - 1) * a.experts + col;
    h[i] = a.hist[at];
    p[i] = a.psum[at];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (b0 + i >= a.blocks) break;
    c += h[i];
    s += p[i];
  }
  cnt[sl][le] = c;
  sum[sl][le] = s;
  __syncthreads();
  if (e < a.experts) {
    int before = 0, total = 0;
    float all = 0.f;
#pragma unroll 16
    for (int j = 0; j < kScanSlices; ++j) {
      before += j < sl ? cnt[j][le] : 0;
      total += cnt[j][le];
      all += sum[j][le];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (b0 + i >= a.blocks) break;
      a.hist[int64_t(b0 + i) * a.experts + e] = before;
      before += h[i];
    }
    if (sl == 0) {
      a.counts[e] = total;
      a.psum[e] = all;  // row 0: this thread has read it
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < 64) {
    int v = 0;
    for (int b = int(threadIdx.x); b < a.blocks; b += 64) v += a.valid[b];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    if (threadIdx.x == 0) a.counts[a.experts] = v;
  }
}

// Third launch: the slot lists; the first workgroup also offsets and loss.
template <int kJ>
__global__ __launch_bounds__(route_threads<kJ>()) void route_place_kernel(const RouteFwdArgs a) {
  constexpr int kThreads = route_threads<kJ>();
  __shared__ RouteLds<kJ> lds;
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
    dl[j] = float(a.counts[e < a.experts ? e : a.experts - 1]);  // every load issued, as for the logits
  }
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = j * 64 + lane;
    dl[j] = a.dloss && e < a.experts ? coef * dl[j] : 0.f;
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

// Registers a lane: 16 lanes hold a token in the forward kernels, 64 in the
// backward one.
template <typename F>
auto by_row(int experts, F &&f) {
  if (experts <= 128) return f(std::integral_constant<int, 8>());
  if (experts <= 256) return f(std::integral_constant<int, 16>());
  if (experts <= 384) return f(std::integral_constant<int, 24>());
  if (experts <= 512) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 64>());
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
  return by_row(a.experts, [&](auto kj) {
    constexpr int kJ = decltype(kj)::value;
    if (a.blocks == 0) {
      hipLaunchKernelGGL((route_one_kernel<T, kJ>), dim3(1), dim3(route_threads<kJ>()), 0, s, a);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((route_tokens_kernel<T, kJ>), dim3(unsigned(a.blocks)), dim3(route_threads<kJ>()), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(a.blocks <= 4 * kScanSlices ? route_scan_kernel<4> : route_scan_kernel<kMaxBlocks / kScanSlices>,
                       dim3((a.experts + kScanExperts - 1) / kScanExperts), dim3(kScanExperts * kScanSlices), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((route_place_kernel<kJ>), dim3(unsigned(a.blocks)), dim3(route_threads<kJ>()), 0, s, a);
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
  const int64_t each = (subs + kMaxBlocks - 1) / kMaxBlocks;
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
