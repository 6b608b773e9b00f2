// Routing to experts: the choice of every token's experts and their weights,
// and the gradient of the logits.
//
// Forward.  s = softmax(x) or sigmoid(x); v = s + bias; the best groups by
// the sum of their one or two largest v; the topk largest v of what is left,
// ties to the lower index; w = scale * s of the chosen, over their sum with
// renorm.  One wave takes one token: lane l holds experts l, l + 64, ... .
// The choice is the one that 64-bit scores make: v is computed and compared
// in 64 bits, since two 32-bit sigmoids plus biases can swap near neighbours.
#include "moe.hpp"
#include "sync.hpp"

namespace hocf {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// Counts of chosen experts leave a workgroup's LDS histogram through the
// workspace; the last workgroup to finish copies them out and zeroes the
// words again.  `finish` is called by every thread of every workgroup.
__device__ __forceinline__ void finish_counts(const RouteArgs& a, const uint32_t* s_hist, int* s_last) {
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    if (s_hist[e]) __hip_atomic_fetch_add(&a.ws[1 + e], s_hist[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t prev = __hip_atomic_fetch_add(&a.ws[0], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    const int last = prev == gridDim.x - 1;
    if (last) __hip_atomic_store(&a.ws[0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_last = last;
  }
  __syncthreads();
  if (!uniform(*s_last)) return;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    a.counts[e] = (int32_t)__hip_atomic_exchange(&a.ws[1 + e], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <int DT>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  constexpr int V = kRouteMaxE / 64;
  __shared__ double s_v[kRouteWaves][kRouteMaxE];
  __shared__ uint32_t s_hist[kRouteMaxE];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.E;
  const double kOff = -INFINITY;
  for (int e = threadIdx.x; e < E; e += kRouteThreads) s_hist[e] = 0;
  __syncthreads();

  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < a.T; t += (int64_t)gridDim.x * kRouteWaves) {
    double s[V], v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      const float x = e < E ? ld1<DT>(a.logits, t * a.ld + e) : -INFINITY;
      s[i] = x > -INFINITY ? (double)x : kOff;  // (NaN is off too)
    }
    uint32_t live = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) live |= (uint32_t)(s[i] > kOff) << i;
    if (a.score == kSoftmax) {
      double top = kOff, sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmax(top, s[i]);
      top = wave_max(top);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = !(live >> i & 1) ? 0.0 : s[i] == top ? 1.0 : exp(s[i] - top);
        sum += s[i];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = live >> i & 1 ? 1.0 / (1.0 + exp(-s[i])) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      const double w = s[i] + (a.bias && e < E ? (double)a.bias[e] : 0.0);
      v[i] = live >> i & 1 && w > kOff ? w : kOff;
    }
    if (a.n_group > 1) {
      const int S = E / a.n_group;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 64 * i < E) s_v[wave][lane + 64 * i] = v[i];
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
      double m1 = kOff, m2 = kOff;  // lane g: the two largest of group g
      if (lane < a.n_group)
        for (int i = 0; i < S; ++i) {
          const double w = s_v[wave][lane * S + i];
          if (w > m1) { m2 = m1; m1 = w; } else if (w > m2) m2 = w;
        }
      const double of = a.group_top == 2 && m2 > kOff ? m1 + m2 : m1;
      int ahead = 0;
      for (int g = 0; g < a.n_group; ++g) {
        const double o = __shfl(of, g, 64);
        ahead += o > of || (o == of && g < lane);
      }
      const uint64_t kept = __ballot(lane < a.n_group && ahead < a.topk_group);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        if (e < E && !(kept >> (e / S) & 1)) v[i] = kOff;
      }
      __builtin_amdgcn_wave_barrier();
    }
    double total = 0.0, mine = 0.0;
    int my_e = -1;
    for (int j = 0; j < a.topk; ++j) {
      double best = kOff, bs = 0.0;
      int at = INT_MAX;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (v[i] > best) { best = v[i]; bs = s[i]; at = lane + 64 * i; }
#pragma unroll
      for (int d = 32; d; d >>= 1) {
        const double ob = __shfl_xor(best, d, 64), os = __shfl_xor(bs, d, 64);
        const int oa = __shfl_xor(at, d, 64);
        if (ob > best || (ob == best && oa < at)) { best = ob; bs = os; at = oa; }
      }
      if (!(best > kOff)) { at = -1; bs = 0.0; }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at == lane + 64 * i) v[i] = kOff;
      total += bs;
      if (lane == j) { mine = bs; my_e = at; }
    }
    if (lane < a.topk) {
      const double w = !a.renorm ? mine : total > 0.0 ? mine / total : 0.0;
      a.experts[t * a.topk + lane] = my_e;
      a.weights[t * a.topk + lane] = (float)(w * (double)a.scale);
      if (a.counts && my_e >= 0) atomicAdd(&s_hist[my_e], 1u);
    }
  }
  if (a.counts) finish_counts(a, s_hist, &s_last);
}

int launch_moe_route(const RouteArgs& a, hipStream_t s) {
  auto kern = a.dt == kBF16 ? &route_kernel<kBF16> : &route_kernel<kF32>;
  int grid = 0;
  hipError_t e = persistent_grid(reinterpret_cast<const void*>(kern), kRouteThreads,
                                 (a.T + kRouteWaves - 1) / kRouteWaves, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kRouteThreads), 0, s, a);
  return hipGetLastError();
}

// Backward.  With p the softmax of the row and g_j = scale * dw_j:
//   softmax:             dx_e = p_e (sum over j with e_j = e of g_j  -  sum_j p_{e_j} g_j)
//   sigmoid:             dx_{e_j} = g_j s (1 - s), zero elsewhere
//   either with renorm:  w = scale * r with r the softmax of the chosen
//                        log-scores l_j, so d/dl_j = r_j (g_j - sum_k r_k g_k);
//                        l = x up to a constant for a softmax, log s for a
//                        sigmoid (dl/dx = 1 - s); zero elsewhere
// The log-score form keeps renorm exact where every chosen s underflows.
// Sums over j run in the order of the places, so results do not vary.
__device__ __forceinline__ float wave_maxf(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ float wave_sumf(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <int DT>
__global__ __launch_bounds__(kRouteThreads) void route_bwd_kernel(RouteBwdArgs a) {
  constexpr int V = kRouteMaxE / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.E;
  const float kOff = -INFINITY;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < a.T; t += (int64_t)gridDim.x * kRouteWaves) {
    // lane j: place j
    int e_j = -1;
    float x_j = kOff, g_j = 0.0f;
    if (lane < a.topk) {
      e_j = a.experts[t * a.topk + lane];
      if (e_j < -1 || e_j >= E) { report_status(a.sync, kErrBadIndex); e_j = -1; }
      if (e_j >= 0) {
        const float x = ld1<DT>(a.logits, t * a.ld + e_j);
        if (x > kOff) { x_j = x; g_j = a.dweights[t * a.topk + lane] * a.scale; }
        else e_j = -1;  // a switched-off logit has no gradient
      }
    }
    const bool dense = a.score == kSoftmax && !a.renorm;
    float p[V];
    float top = kOff, inv = 0.0f;
    if (dense) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        const float x = e < E ? ld1<DT>(a.logits, t * a.ld + e) : kOff;
        p[i] = x > kOff ? x : kOff;
        top = fmaxf(top, p[i]);
      }
      top = wave_maxf(top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = !(p[i] > kOff) ? 0.0f : p[i] == top ? 1.0f : expf(p[i] - top);
        sum += p[i];
      }
      sum = wave_sumf(sum);
      inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    // lane j: the gradient of log p_j (dense) or of x_j (sparse)
    float d_j = 0.0f, mean = 0.0f;
    const float s_j = 1.0f / (1.0f + expf(-x_j)), c_j = 1.0f / (1.0f + expf(x_j));  // sigmoid, 1 - sigmoid
    if (dense) {
      const float p_j = e_j < 0 ? 0.0f : x_j == top ? inv : expf(x_j - top) * inv;
      d_j = g_j;
      mean = wave_sumf(e_j >= 0 ? p_j * g_j : 0.0f);
    } else if (a.renorm) {
      const float l = e_j < 0 ? kOff : a.score == kSoftmax ? x_j : fminf(x_j, 0.0f) - log1pf(expf(-fabsf(x_j)));
      const float m = wave_maxf(l);
      float r = !(l > kOff) ? 0.0f : l == m ? 1.0f : expf(l - m);
      const float sum = wave_sumf(r);
      r = sum > 0.0f ? r / sum : 0.0f;
      d_j = r * (g_j - wave_sumf(r * g_j));
      if (a.score == kSigmoid) d_j *= c_j;
      if (e_j < 0) d_j = 0.0f;
    } else {
      d_j = e_j < 0 ? 0.0f : g_j * s_j * c_j;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      float d = 0.0f;
      for (int j = 0; j < a.topk; ++j) {
        const int ej = __shfl(e_j, j, 64);
        const float dj = __shfl(d_j, j, 64);
        if (ej == e) d += dj;
      }
      if (dense) d = p[i] > 0.0f ? p[i] * inv * (d - mean) : 0.0f;
      if (e < E) st1<DT>(a.dlogits, t * E + e, d);
    }
  }
}

int launch_moe_route_bwd(const RouteBwdArgs& a, hipStream_t s) {
  auto kern = a.dt == kBF16 ? &route_bwd_kernel<kBF16> : &route_bwd_kernel<kF32>;
  int grid = 0;
  hipError_t e = persistent_grid(reinterpret_cast<const void*>(kern), kRouteThreads,
                                 (a.T + kRouteWaves - 1) / kRouteWaves, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kRouteThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace hocf
