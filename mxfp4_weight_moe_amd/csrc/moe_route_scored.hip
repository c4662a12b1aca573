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
// A token has 16 lanes (four tokens a wave: what a step of the choice costs beside the lanes' own work is
// paid once for four).  Its keys are made in fp32 (without a bias they are the logits, exact), cut to
// 22 bits above the expert's number, and the k + 2 largest found one by one; those few are then put in order
// by their 64-bit keys.  That is the answer unless the key of a chosen expert lies within the fp32 error
// of those that were not looked at, or two candidates' softmax scores within that of each other; then
// (and where equal keys fill the border) the row is done again entirely in 64 bits.
#include "mx_internal.hpp"
#include "moe_route.hpp"

namespace mx {

// Rows of an odd length stay whole accesses.
typedef u32x4 u32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* p, size_t i) {
  if constexpr (BF16)
    return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}

constexpr int ROUTE_LANES = 16;  // of a token
constexpr int ROUTE_ROWS = 64 / ROUTE_LANES;

template <class T, class F>
__device__ __forceinline__ T row16(T v, F f) {
#pragma unroll
  for (int m = 1; m < ROUTE_LANES; m <<= 1) v = f(v, __shfl_xor(v, m, ROUTE_LANES));
  return v;
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  max32_dpp<DPP_QUAD_XOR1, 0xF>(v);
  max32_dpp<DPP_QUAD_XOR2, 0xF>(v);
  max32_dpp<DPP_ROW_HALF_MIRROR, 0xF>(v);
  max32_dpp<DPP_ROW_MIRROR, 0xF>(v);
  return v;
}
__device__ __forceinline__ float row16_sum(float v) {
  v = row_add_step<DPP_QUAD_XOR1>(v);
  v = row_add_step<DPP_QUAD_XOR2>(v);
  v = row_add_step<DPP_ROW_HALF_MIRROR>(v);
  return row_add_step<DPP_ROW_MIRROR>(v);
}

// a before b in the order of choice.
__device__ __forceinline__ bool before(double ka, int a, double kb, int b) { return ka > kb || (ka == kb && a < b); }
// NaN counts as the lowest.
__device__ __forceinline__ double ordered(double v) { return v == v ? v : -INFINITY; }

// Scores of a row in 64 bits.
template <bool BF16>
struct Scores {
  const void* l;
  const float* bias;
  size_t at;
  bool sigmoid;
  double top, sum;  // softmax
  __device__ __forceinline__ double logit(int e) const { return (double)logit_at<BF16>(l, at + e); }
  __device__ __forceinline__ double score_of(double v) const { return sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / sum; }
  __device__ __forceinline__ double score(int e) const { return score_of(logit(e)); }
  __device__ __forceinline__ double key(int e) const { return ordered(score(e) + (bias ? (double)bias[e] : 0.0)); }
  __device__ __forceinline__ double order(int e) const { return bias ? key(e) : ordered(logit(e)); }
};

// A row in 64 bits throughout, one choice after the other: expert j's number and score go to lane
// j % 16, place j / 16.
template <bool BF16>
__device__ __attribute__((noinline)) void route_exact(const RouteScored& a, int64_t t, int lane, int (&mine_id)[2],
                                                      double (&mine)[2]) {
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
  // the best of (value, number) pairs behind the last one taken
  double last = 0.0;
  int last_id = -1;
  auto best = [&](double k, int id) {
#pragma unroll
    for (int m = 1; m < ROUTE_LANES; m <<= 1) {
      const double ok = __shfl_xor(k, m, ROUTE_LANES);
      const int oid = __shfl_xor(id, m, ROUTE_LANES);
      if (oid >= 0 && (id < 0 || before(ok, oid, k, id))) k = ok, id = oid;
    }
    last = k, last_id = id;
  };
  uint64_t open = ~0ull;
  const int size = a.E / a.groups;
  if (a.groups > 1) {
    open = 0;
    for (int j = 0; j < a.kept; ++j) {
      double k = 0.0;
      int g = -1;
      for (int c = lane; c < a.groups; c += ROUTE_LANES) {
        double one = -INFINITY, two = -INFINITY;
        for (int e = c * size; e < (c + 1) * size; ++e) {
          const double v = s.key(e);
          two = v > one ? one : (v > two ? v : two);
          one = v > one ? v : one;
        }
        const double v = a.top2 && size > 1 ? one + two : one;
        if ((j == 0 || before(last, last_id, v, c)) && (g < 0 || before(v, c, k, g))) k = v, g = c;
      }
      best(k, g);
      open |= 1ull << last_id;
    }
  }
  for (int j = 0; j < a.k; ++j) {
    double k = 0.0;
    int id = -1;
    for (int e = lane; e < a.E; e += ROUTE_LANES) {
      if (!((open >> (e / size)) & 1)) continue;
      const double v = s.order(e);
      if ((j == 0 || before(last, last_id, v, e)) && (id < 0 || before(v, e, k, id))) k = v, id = e;
    }
    best(k, id);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (j == lane + ROUTE_LANES * h) mine_id[h] = last_id, mine[h] = s.score(last_id);
  }
}

// What is added to k for the candidates that show where the border lies.
constexpr int ROUTE_MORE = 2;
// Bound of an fp32 key's distance from its 64-bit one, relative to 1 + |key|: a sigmoid score is off by
// (1.3 |l| (1 - p) p + 6 p) u < 2^-20, a softmax score, its sum of E <= 1024 terms among it, by less than
// (64 + 24) u p, and the addition of the bias by u |key|.
constexpr double ROUTE_FP32 = 0x1p-17;

// PER: logits of a lane, chunks of 4 consecutive ones, E <= 16 PER; C: candidates of a lane, k + 2 <= 16 C
// (k at most 32 with C = 3).
template <bool BF16, int PER, int C>
__global__ void __launch_bounds__(64) route_scored_kernel(RouteScored a, int32_t* __restrict__ ids, float* __restrict__ gates) {
  extern __shared__ float shared[];  // with groups: per row its keys [E], its groups' values [groups]
  const int lane = threadIdx.x % ROUTE_LANES, row = threadIdx.x / ROUTE_LANES;
  const int64_t t0 = (int64_t)blockIdx.x * ROUTE_ROWS + row, t = t0 < a.T ? t0 : a.T - 1;  // rows past the last: it again
  const size_t at = (size_t)t * a.E;
  const int E = a.E;
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const int e = 4 * (lane + ROUTE_LANES * (i / 4));
    if (e + 4 <= E) {
      if constexpr (BF16) {
        const u32x2 q = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(a.logits) + at + e);
#pragma unroll
        for (int j = 0; j < 2; ++j) l[i + 2 * j] = __uint_as_float(q[j] << 16), l[i + 2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
      } else {
        const u32x4 q = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(a.logits) + at + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) l[i + j] = __uint_as_float(q[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) l[i + j] = e + j < E ? logit_at<BF16>(a.logits, at + e + j) : -INFINITY;
    }
  }
  auto number = [&](int i) { return 4 * (lane + ROUTE_LANES * (i / 4)) + i % 4; };

  // softmax: the largest logit and the sum
  float top = 0.f, sum = 1.f;
  if (!a.sigmoid) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    top = route_value(row16_max(route_key(m)));
    if (top == -INFINITY) {
      top = 0.f;  // nothing but -Inf (or NaN, which the sum is then)
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) z += l[i] != l[i] ? l[i] : 0.f;
      sum = row16_sum(z) + 1.f;
    } else if (!a.renormalize || a.bias || a.groups > 1) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) z += __expf(l[i] - top);
      sum = row16_sum(z);
    } else {
      float z = 0.f;  // a NaN reaches every gate of its row
#pragma unroll
      for (int i = 0; i < PER; ++i) z += l[i] != l[i] || l[i] == INFINITY ? l[i] - top : 0.f;
      sum = row16_sum(z) + 1.f;
    }
  }
  const float inv = 1.f / sum;
  auto score32 = [&](float v) { return a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-v)) : __expf(v - top) * inv; };
  auto ordered32 = [](float v) { return v == v ? v : -INFINITY; };

  bool again = false;  // in 64 bits
  uint32_t comp[PER];
  const bool groups = a.groups > 1;
  if (a.bias || groups) {
    float* keys = shared + row * (E + a.groups);
    float* vals = keys + E;
    const int size = E / a.groups;
    const uint32_t magic = ((1u << 20) + size - 1) / size;  // e / size = (e * magic) >> 20 for e, size <= 1024
    float key[PER], size_of = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = number(i);
      float b = 0.f;
      if (a.bias) b = e < E ? a.bias[e] : 0.f;
      key[i] = ordered32(score32(l[i]) + b);
      if (groups && e < E) keys[e] = key[i];
      size_of = fmaxf(size_of, key[i] == -INFINITY ? 0.f : fabsf(key[i]));
    }
    if (groups) {
      __syncthreads();
      for (int g = lane; g < a.groups; g += ROUTE_LANES) {
        float one = -INFINITY, two = -INFINITY;
        for (int e = g * size; e < (g + 1) * size; ++e) {
          const float v = keys[e];
          two = fmaxf(two, fminf(one, v));
          one = fmaxf(one, v);
        }
        vals[g] = a.top2 && size > 1 ? one + two : one;
      }
      __syncthreads();
      float worst = INFINITY, next = -INFINITY;  // of the groups kept, of the others
      uint32_t lo = 0, hi = 0;
      for (int g = lane; g < a.groups; g += ROUTE_LANES) {
        const float v = vals[g];
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) rank += vals[o] > v || (vals[o] == v && o < g);
        if (rank < a.kept) {
          worst = fminf(worst, v);
          if (g < 32)
            lo |= 1u << g;
          else
            hi |= 1u << (g - 32);
        } else {
          next = fmaxf(next, v);
        }
      }
      size_of = row16(size_of, [](float x, float y) { return fmaxf(x, y); });
      auto either = [](uint32_t x, uint32_t y) { return x | y; };
      lo = row16(lo, either), hi = row16(hi, either);
      worst = row16(worst, [](float x, float y) { return fminf(x, y); });
      next = row16(next, [](float x, float y) { return fmaxf(x, y); });
      // two values of two keys each
      again = !((double)worst - (double)next > 4.0 * ROUTE_FP32 * (1.0 + (double)size_of));
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t g = ((uint32_t)number(i) * magic) >> 20;
        const float v = a.bias ? key[i] : ordered32(l[i]);
        comp[i] = ((g < 32 ? lo >> g : hi >> (g & 31)) & 1) ? route_key(v) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) comp[i] = route_key(key[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) comp[i] = route_key(ordered32(l[i]));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = number(i);
    comp[i] = e < E && comp[i] ? (comp[i] & ~1023u) | (uint32_t)(1023 - e) : 0u;
  }

  // The largest one below w, again and again: x - w wraps to the top exactly for x < w.
  uint32_t cand[C] = {};
  uint32_t w = 0;
  bool left = true;  // unless every expert is a candidate already
  const int rounds = a.k + ROUTE_MORE;
  for (int j = 0; j < rounds; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; i += 2) m = max(m, max(comp[i] - w, comp[i + 1] - w));
    w += row16_max(m);
    left = left && w != 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (j == lane + ROUTE_LANES * c) cand[c] = left ? w : 0u;
  }

  // the candidates' 64-bit keys, their order, and whether it is certain
  Scores<BF16> s{a.logits, a.bias, at, a.sigmoid, (double)top, (double)sum};
  int id[C], rank[C];
  float cl[C], cb[C];
  double key[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    id[c] = cand[c] ? 1023 - (int)(cand[c] & 1023u) : 1 << 20;
    cl[c] = cand[c] ? logit_at<BF16>(a.logits, at + id[c]) : -INFINITY;
    cb[c] = a.bias && cand[c] ? a.bias[id[c]] : 0.f;
    key[c] = a.bias ? ordered(s.score_of((double)cl[c]) + (double)cb[c]) : ordered((double)cl[c]);
    if (!cand[c]) key[c] = -INFINITY;  // its number puts it behind all others
    rank[c] = 0;
  }
  const bool rough = a.bias && !a.sigmoid;  // these scores have the fp32 sum
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = min(ROUTE_LANES, rounds - ROUTE_LANES * c);
    for (int j = 0; j < n; ++j) {
      const double ok = __shfl(key[c], j, ROUTE_LANES);
      const int oid = __shfl(id[c], j, ROUTE_LANES);
      const float ol = __shfl(cl[c], j, ROUTE_LANES), ob = __shfl(cb[c], j, ROUTE_LANES);
#pragma unroll
      for (int d = 0; d < C; ++d) {
        rank[d] += before(ok, oid, key[d], id[d]);
        if (rough && oid != id[d] && !(fabs(ok - key[d]) > 2.0 * ROUTE_FP32 * (1.0 + fabs(ok))) && !(ol == cl[d] && ob == cb[d]))
          again = again || (cand[d] != 0 && oid < 1 << 20);
      }
    }
  }
  if (left) {
    // everything that was not a candidate has an fp32 key of at most this
    const double most = (double)route_value(w | 1023u);
    const double least = a.bias ? most + ROUTE_FP32 * (1.0 + fabs(most)) : most;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (rank[c] == a.k - 1) again = again || !(key[c] > least);
  }
  const uint64_t rows = __ballot(again);
  again = ((rows >> (threadIdx.x & 48)) & 0xFFFFu) != 0;

  int out[C], out_id[C];
  double p[C];
#pragma unroll
  for (int c = 0; c < C; ++c) out[c] = rank[c], out_id[c] = id[c], p[c] = rank[c] < a.k ? s.score_of((double)cl[c]) : 0.0;
  if (again) {
    int mine_id[2] = {};
    double mine[2] = {};
    route_exact<BF16>(a, t, lane, mine_id, mine);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      out[c] = c < 2 ? lane + ROUTE_LANES * c : a.k;
      out_id[c] = c < 2 ? mine_id[c] : 0;
      p[c] = c < 2 && out[c] < a.k ? mine[c] : 0.0;
    }
  }
  if (a.renormalize) {
    double all = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) all += p[c];
    all = row16(all, [](double x, double y) { return x + y; });
#pragma unroll
    for (int c = 0; c < C; ++c) p[c] = all == 0.0 ? 0.0 : p[c] / all;
  }
  if (t0 >= a.T) return;
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (out[c] < a.k) {
      ids[t * a.k + out[c]] = out_id[c];
      gates[t * a.k + out[c]] = (float)((double)a.scale * p[c]);
    }
}

template <bool BF16, int PER>
static void route_scored(const RouteScored& a, int32_t* ids, float* gates, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + ROUTE_ROWS - 1) / ROUTE_ROWS));
  const unsigned lds = a.groups > 1 ? ROUTE_ROWS * (unsigned)(a.E + a.groups) * 4 : 0;
  if (a.k + ROUTE_MORE <= ROUTE_LANES)
    hipLaunchKernelGGL((route_scored_kernel<BF16, PER, 1>), grid, dim3(64), lds, stream, a, ids, gates);
  else
    hipLaunchKernelGGL((route_scored_kernel<BF16, PER, 3>), grid, dim3(64), lds, stream, a, ids, gates);
}

template <bool BF16>
static void route_scored(const RouteScored& a, int32_t* ids, float* gates, hipStream_t stream) {
  if (a.E <= 64)
    route_scored<BF16, 4>(a, ids, gates, stream);
  else if (a.E <= 128)
    route_scored<BF16, 8>(a, ids, gates, stream);
  else if (a.E <= 256)
    route_scored<BF16, 16>(a, ids, gates, stream);
  else if (a.E <= 384)
    route_scored<BF16, 24>(a, ids, gates, stream);
  else if (a.E <= 512)
    route_scored<BF16, 32>(a, ids, gates, stream);
  else
    route_scored<BF16, 64>(a, ids, gates, stream);
}

int launch_route_scored(const RouteScored& a, int32_t* ids, float* gates, hipStream_t stream) {
  a.bf16 ? route_scored<true>(a, ids, gates, stream) : route_scored<false>(a, ids, gates, stream);
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
