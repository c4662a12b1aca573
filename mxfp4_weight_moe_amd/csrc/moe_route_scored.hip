// Routing by scores, with a bias for balance and groups of experts, and its gradient.
//
//   p     = softmax(l) or sigmoid(l) over a token's E logits
//   key   = p + bias                          (experts are chosen by it; without a bias by the logits,
//                                              whose order p keeps)
//   group = the largest key of a group of experts, or the sum of its two largest; the `kept` best
//           groups stay
//   ids   = the k largest keys left, descending, equals to the lower id
//   gates = scale * p[ids], or scale * p[ids] / sum p[ids]
//
// The order is that of 64-bit keys: which experts a token takes does not depend on how a kernel rounds.
#include "mx_internal.hpp"
#include "moe_route.hpp"

namespace mx {

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, size_t i) {
  if constexpr (BF16)
    return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}

// A token's row: 16 lanes, four tokens a wave.
constexpr int ROUTE_LANES = 16;
template <class F>
__device__ __forceinline__ double row16(double v, F f) {
#pragma unroll
  for (int m = 1; m < ROUTE_LANES; m <<= 1) v = f(v, __shfl_xor(v, m, ROUTE_LANES));
  return v;
}

// Before: in the order of choice (NaN keys count as the lowest).
__device__ __forceinline__ bool before(double ka, int a, double kb, int b) { return ka > kb || (ka == kb && a < b); }

// Scores of a row in 64 bits.
template <bool BF16>
struct Scores {
  const void* l;
  const float* bias;
  size_t at;
  bool sigmoid;
  double top, sum;  // softmax
  __device__ __forceinline__ double logit(int e) const { return (double)logit_at<BF16>(l, at + e); }
  __device__ __forceinline__ double score(int e) const {
    const double v = logit(e);
    return sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / sum;
  }
  static __device__ __forceinline__ double ordered(double v) { return v == v ? v : -INFINITY; }
  __device__ __forceinline__ double key(int e) const { return ordered(score(e) + (bias ? (double)bias[e] : 0.0)); }
  __device__ __forceinline__ double order(int e) const { return bias ? key(e) : ordered(logit(e)); }
};

template <bool BF16>
__global__ void __launch_bounds__(64) route_scored_kernel(RouteScored a, int32_t* __restrict__ ids, float* __restrict__ gates) {
  const int lane = threadIdx.x % ROUTE_LANES;
  const int64_t t = (int64_t)blockIdx.x * (64 / ROUTE_LANES) + threadIdx.x / ROUTE_LANES;
  if (t >= a.T) return;
  Scores<BF16> s{a.logits, a.bias, (size_t)t * a.E, a.sigmoid, 0.0, 1.0};
  auto most = [](double x, double y) { return x > y ? x : (y == y ? y : x); };
  auto plus = [](double x, double y) { return x + y; };
  if (!a.sigmoid) {
    double m = -INFINITY, sum = 0.0;
    for (int e = lane; e < a.E; e += ROUTE_LANES) m = most(m, s.logit(e));
    s.top = row16(m, most);
    for (int e = lane; e < a.E; e += ROUTE_LANES) sum += exp(s.logit(e) - s.top);
    s.sum = row16(sum, plus);
    if (s.top == -INFINITY) s.top = 0.0, s.sum = 1.0;  // nothing but -Inf: every score is 0
  }
  uint64_t open = ~0ull;
  const int size = a.E / a.groups;
  if (a.groups > 1) {
    open = 0;
    double best = INFINITY;
    int last = -1;
    for (int j = 0; j < a.kept; ++j) {
      double k = -INFINITY;
      int g = 1 << 30;
      for (int c = lane; c < a.groups; c += ROUTE_LANES) {
        double one = -INFINITY, two = -INFINITY;
        for (int e = c * size; e < (c + 1) * size; ++e) {
          const double v = s.key(e);
          two = v > one ? one : (v > two ? v : two);
          one = v > one ? v : one;
        }
        const double v = a.top2 && size > 1 ? one + two : one;
        if ((j == 0 || before(best, last, v, c)) && (g == 1 << 30 || before(v, c, k, g))) k = v, g = c;
      }
#pragma unroll
      for (int m = 1; m < ROUTE_LANES; m <<= 1) {
        const double ok = __shfl_xor(k, m, ROUTE_LANES);
        const int og = __shfl_xor(g, m, ROUTE_LANES);
        if (og != 1 << 30 && (g == 1 << 30 || before(ok, og, k, g))) k = ok, g = og;
      }
      best = k, last = g;
      open |= 1ull << g;
    }
  }
  double last = INFINITY;
  int last_id = -1;
  double mine[2] = {0.0, 0.0};
  int mine_id[2] = {0, 0};
  for (int j = 0; j < a.k; ++j) {
    double k = -INFINITY;
    int id = 1 << 30;
    for (int e = lane; e < a.E; e += ROUTE_LANES) {
      if (!((open >> (e / size)) & 1)) continue;
      const double v = s.order(e);
      if ((j == 0 || before(last, last_id, v, e)) && (id == 1 << 30 || before(v, e, k, id))) k = v, id = e;
    }
#pragma unroll
    for (int m = 1; m < ROUTE_LANES; m <<= 1) {
      const double ok = __shfl_xor(k, m, ROUTE_LANES);
      const int oid = __shfl_xor(id, m, ROUTE_LANES);
      if (oid != 1 << 30 && (id == 1 << 30 || before(ok, oid, k, id))) k = ok, id = oid;
    }
    last = k, last_id = id;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (j == lane + 16 * h) mine_id[h] = id, mine[h] = s.score(id);
  }
  double sum = 0.0;
  if (a.renormalize) sum = row16(mine[0] + mine[1], plus);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 16 * h;
    if (j >= a.k) continue;
    const double p = a.renormalize ? (sum == 0.0 ? 0.0 : mine[h] / sum) : mine[h];
    ids[t * a.k + j] = mine_id[h];
    gates[t * a.k + j] = (float)((double)a.scale * p);
  }
}

int launch_route_scored(const RouteScored& a, int32_t* ids, float* gates, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + 3) / 4));
  if (a.bf16)
    hipLaunchKernelGGL(route_scored_kernel<true>, grid, dim3(64), 0, stream, a, ids, gates);
  else
    hipLaunchKernelGGL(route_scored_kernel<false>, grid, dim3(64), 0, stream, a, ids, gates);
  return hip_status(hipGetLastError());
}

// ------------------------------------------------------------------ gradient
//
// With c = scale * dgates and, renormalised, S = sum p[ids]:  dp[ids] = c, or (c - sum c p[ids] / S) / S;
//   sigmoid:  dl[ids] = dp p (1 - p), 0 elsewhere
//   softmax:  dl = p (dp - sum dp p): dense, but renormalised it is a softmax over the chosen logits,
//             dl[ids] = q (c - sum c q), 0 elsewhere
// The few chosen values are worked out in 64 bits (what is left of differences of nearly equal values),
// the rest of a dense row in 32.

// A row: one wave.  The row's dp (dense) or dl goes through the LDS, where ids place it.
template <bool BF16>
__global__ void __launch_bounds__(64) route_scored_backward_kernel(RouteScored a, const float* __restrict__ dgates,
                                                                   const int32_t* __restrict__ ids, void* __restrict__ dlogits) {
  __shared__ float row[MX_MAX_EXPERTS];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const size_t at = (size_t)t * a.E;
  const bool dense = !a.sigmoid && !a.renormalize;
  auto wave = [](double v, auto f) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = f(v, __shfl_xor(v, m, 64));
    return v;
  };
  auto plus = [](double x, double y) { return x + y; };
  auto most = [](double x, double y) { return x > y ? x : (y == y ? y : x); };
  for (int e = lane; e < a.E; e += 64) row[e] = 0.f;
  int id = -1;
  double c = 0.0, l = -INFINITY;
  if (lane < a.k) {
    id = ids[t * a.k + lane];
    c = (double)a.scale * (double)dgates[t * a.k + lane];
    if (id < 0 || id >= a.E)
      id = -1;
    else
      l = (double)logit_at<BF16>(a.logits, at + id);
  }
  double top = 0.0, sum = 1.0, p = 0.0, d = c;
  if (a.sigmoid) {
    if (id >= 0) p = 1.0 / (1.0 + exp(-l));
    if (a.renormalize) {
      const double s = wave(p, plus), cp = wave(id >= 0 ? c * p : 0.0, plus);
      d = s == 0.0 ? 0.0 : (c - cp / s) / s;
    }
    d *= p / (1.0 + exp(l));  // p (1 - p)
  } else {
    double m = l;
    if (dense)
      for (int e = lane; e < a.E; e += 64) m = most(m, (double)logit_at<BF16>(a.logits, at + e));
    top = wave(m, most);
    double z = 0.0;
    if (dense)
      for (int e = lane; e < a.E; e += 64) z += (double)__expf(logit_at<BF16>(a.logits, at + e) - (float)top);
    else if (id >= 0)
      z = exp(l - top);
    sum = wave(z, plus);
    if (top == -INFINITY) top = 0.0, sum = 1.0;  // nothing but -Inf: every score is 0
    if (id >= 0) p = exp(l - top) / sum;
    const double cp = wave(id >= 0 ? c * p : 0.0, plus);
    d = p * (c - cp);
    if (dense)
      for (int e = lane; e < a.E; e += 64)
        row[e] = (float)(-cp) * (__expf(logit_at<BF16>(a.logits, at + e) - (float)top) / (float)sum);
  }
  __syncthreads();
  if (id >= 0) row[id] = (float)d;
  __syncthreads();
  for (int e = lane; e < a.E; e += 64) {
    if constexpr (BF16)
      static_cast<uint16_t*>(dlogits)[at + e] = f32_to_bf16_rne(row[e]);
    else
      static_cast<float*>(dlogits)[at + e] = row[e];
  }
}

int launch_route_scored_backward(const RouteScored& a, const float* dgates, const int32_t* ids, void* dlogits,
                                 hipStream_t stream) {
  const dim3 grid((unsigned)a.T);
  if (a.bf16)
    hipLaunchKernelGGL(route_scored_backward_kernel<true>, grid, dim3(64), 0, stream, a, dgates, ids, dlogits);
  else
    hipLaunchKernelGGL(route_scored_backward_kernel<false>, grid, dim3(64), 0, stream, a, dgates, ids, dlogits);
  return hip_status(hipGetLastError());
}

}  // namespace mx
