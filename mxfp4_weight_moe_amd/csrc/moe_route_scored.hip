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
// 22 to 26 bits above the expert's number, and the k + 2 largest found one by one; those few are then put in order
// by their 64-bit keys.  That is the answer unless the key of a chosen expert lies within the fp32 error
// of those that were not looked at; then (and where equal keys fill the border) the row's choice is made again, in
// 64 bits and one by one.  The same for the groups.
// Softmax's sum is taken in 64 bits (not where a gate does not need it: renormalised, without bias and groups), so
// that a gate is rounded once, whatever the experts are chosen by.  16384 x 384 16.2 us, with an fp32 sum of fp32
// exponentials 13.5, whose gates were off by up to 3 half steps; with a bias, where the candidates' order needs the sum
// in 64 bits too, 16384 x 256 13.1, 43 with fp32 exponentials and the rows that they left open made again.
//
// Bound by instructions, not memory: 16384 x 384 fp32 logits are 25 MB, 5 us to read (one choice after the other in 64
// bits took 117, passes over all of a lane's keys for each candidate 18.5); 16384 x 256 sigmoid scores with a bias 14.2,
// with groups 19.6.  A decode step is one chain of dependent steps: 4.2 us for 1 token, 8.3 for 32 with a bias and groups.
#include "mx_internal.hpp"
#include "moe_route.hpp"
#include "mx_tile.hpp"

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

// Of the lane N places on, within the row.
template <int N>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, false);  // row_ror
}
template <int N>
__device__ __forceinline__ double rotate16(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)rotate16<N>((uint32_t)(b >> 32)) << 32 | rotate16<N>((uint32_t)b));
}

// The same sum in each lane of a row: at every step two lanes add the same two values.
__device__ __forceinline__ double row16_plus(double v) {
  v += rotate16<8>(v);
  v += rotate16<4>(v);
  v += rotate16<2>(v);
  return v + rotate16<1>(v);
}

// exp(x) for x <= 0, exactly 1 at 0, of itself off by 2^-49 (beyond x = -32 by |x| 2^-54, which a sum that has a 1 in it
// does not see); below e^-800, and of NaN, 0.  2^n times a polynomial in y = x log2 e - n, |y| <= 1/2: 1 + y g(y),
// g interpolating (2^y - 1) / y at the 10 Chebyshev nodes (error 2^-50.6).  What a sum over a row takes in 64 bits, at
// some 18 instructions a term where the library's exp has its ends to look after.
__device__ __forceinline__ double exp_term(double x) {
  constexpr double LOG2E = 0x1.71547652b82fep+0, ROUND = 0x1.8p52;  // whose last place is 1
  x = __builtin_fmax(x, -800.0);
  const double n = __builtin_fma(x, LOG2E, ROUND), y = __builtin_fma(x, LOG2E, -(n - ROUND));
  double p = 0x1.e5e9f548e5725p-28;
  for (double c : {0x1.b6571de2f2351p-24, 0x1.62bfe46117445p-20, 0x1.ffcb76789860fp-17, 0x1.4309130378460p-13,
                   0x1.5d87fe908f88ap-10, 0x1.3b2ab6fba385fp-7, 0x1.c6b08d7044119p-5, 0x1.ebfbdff82c590p-3,
                   0x1.62e42fefa39f7p-1, 0x1.0000000000000p+0})
    p = __builtin_fma(p, y, c);
  return __builtin_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, n));
}

// The middle one.
__device__ __forceinline__ uint32_t median(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
// route_key for a key that is cut anyway: -0 lies right below +0 (what that may confuse is seen when the
// candidates are put in order), NaN at -Inf.
__device__ __forceinline__ uint32_t rough_key(float v) {
  const uint32_t b = __float_as_uint(__builtin_fmaxf(v, -INFINITY));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
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

// Between a row's writes to the LDS and its reads of them: its 16 lanes are of one wave, whose accesses keep
// their order.
__device__ __forceinline__ void row_written() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The best (value, number) of a row's lanes, in each of them; numbers below 0 are none.
__device__ __forceinline__ void row16_best(double& k, int& id) {
#pragma unroll
  for (int m = 1; m < ROUTE_LANES; m <<= 1) {
    const double ok = __shfl_xor(k, m, ROUTE_LANES);
    const int oid = __shfl_xor(id, m, ROUTE_LANES);
    if (oid >= 0 && (id < 0 || before(ok, oid, k, id))) k = ok, id = oid;
  }
}

// 16 / groups lanes to a group (a power of two, one at least).
__device__ __forceinline__ int group_lanes(int groups) { return groups <= 2 ? 8 : groups <= 4 ? 4 : groups <= 8 ? 2 : 1; }

// A row's keys in 64 bits, to its place in the LDS.
template <bool BF16>
__device__ __forceinline__ void exact_keys(const Scores<BF16>& s, int E, int lane, double* keys) {
  row_written();  // what was there has been read
#pragma unroll 4
  for (int e = lane; e < E; e += ROUTE_LANES) keys[e] = s.key(e);
  row_written();
}

// The groups that stay, from the keys in the LDS; vals: a place for the groups' values behind them.
__device__ __forceinline__ uint64_t exact_groups(const RouteScored& a, int lane, const double* keys, double* vals) {
  const int size = a.E / a.groups, share = group_lanes(a.groups);
  for (int c = lane / share; c < a.groups; c += ROUTE_LANES / share) {
    double one = -INFINITY, two = -INFINITY;
    for (int e = c * size + lane % share; e < (c + 1) * size; e += share) {
      const double v = keys[e];
      two = v > one ? one : (v > two ? v : two);
      one = v > one ? v : one;
    }
    for (int m = 1; m < share; m <<= 1) {
      const double o1 = __shfl_xor(one, m, ROUTE_LANES), o2 = __shfl_xor(two, m, ROUTE_LANES);
      const double lesser = o1 > one ? one : o1;
      two = o2 > two ? o2 : two;
      two = lesser > two ? lesser : two;
      one = o1 > one ? o1 : one;
    }
    vals[c] = a.top2 && size > 1 ? ordered(one + two) : one;  // +Inf and -Inf from a bias
  }
  row_written();
  uint64_t open = 0;
  for (int c = lane; c < a.groups; c += ROUTE_LANES) {
    const double v = vals[c];
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) rank += before(vals[o], o, v, c);
    if (rank < a.kept) open |= 1ull << c;
  }
  auto either = [](uint32_t x, uint32_t y) { return x | y; };
  return (uint64_t)row16((uint32_t)(open >> 32), either) << 32 | row16((uint32_t)open, either);
}

// What is added to k for the candidates that show where the border lies.
constexpr int ROUTE_MORE = 2;
// Bounds of an fp32 score's distance from its 64-bit one, u = 2^-24.  Sigmoid: the exponential is off by
// (1.3 |l| + 2) u of itself, which p (1 - p) <= 1/4 and |l| p (1 - p) < 0.23 leave 0.8 u of, the sum and its
// reciprocal by 2 u: 3 u.  Softmax: x = l - top by |x| u, so the exponential by (2.3 |x| + 2) u e^x < 3 u, and half a step
// each for the reciprocal of the 64-bit sum and the product: 6 u of the largest score.  Adding the bias rounds by
// u |key|.
constexpr float ROUTE_U = 0x1p-24f;

// PER: logits of a lane, chunks of 4 consecutive ones, E <= 16 PER; C: candidates of a lane, k + 2 <= 16 C
// (k at most 32 with C = 3).
// WHOLE of a lane's places hold an expert whatever E.
// Waves a SIMD: four up to 384 experts, which at 24 places spill 3 registers (16384 x 384 softmax 16.1 us, with three
// waves and no spill 16.6; with groups or a bias 3 to 5% the other way); three up to 512, where four would spill 50 (8192 x
// 512 softmax 13.5 for 12.3, with a bias 16.3 for 13.5); beyond, and for more than 14 chosen, what the registers allow.
template <bool BF16, int PER, int C, int WHOLE>
__global__ void __launch_bounds__(64, (C != 1 || PER > 32 ? 1 : PER > 24 ? 3 : 4))
    route_scored_kernel(RouteScored a, int32_t* __restrict__ ids, float* __restrict__ gates) {
  extern __shared__ double shared[];  // with a bias or groups: per row E + groups values
  const int lane = threadIdx.x % ROUTE_LANES, row = threadIdx.x / ROUTE_LANES;
  const int64_t t0 = (int64_t)blockIdx.x * ROUTE_ROWS + row, t = t0 < a.T ? t0 : a.T - 1;  // rows past the last: it again
  const size_t at = (size_t)t * a.E;
  const int E = a.E;
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const int e = 4 * (lane + ROUTE_LANES * (i / 4));
    if (i < WHOLE || e + 4 <= E) {
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
  constexpr uint32_t LAST = PER <= 4 ? 63 : PER <= 8 ? 127 : PER <= 16 ? 255 : PER <= 32 ? 511 : 1023;  // number

  // softmax: the largest logit, and the sum in 64 bits, which the candidates' keys and the gates are made with
  float top = 0.f;
  double sum = 1.0;
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
      sum = (double)(row16_sum(z) + 1.f);
    } else if (!a.renormalize || a.bias || a.groups > 1) {
      sum = 0.0;
      bool bad = top == INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        sum += exp_term((double)l[i] - (double)top);
        bad = bad || l[i] != l[i];
      }
      sum = row16_plus(bad ? (double)NAN : sum);
    } else {
      float z = 0.f;  // a NaN reaches every gate of its row
#pragma unroll
      for (int i = 0; i < PER; ++i) z += l[i] != l[i] || l[i] == INFINITY ? l[i] - top : 0.f;
      sum = (double)(row16_sum(z) + 1.f);
    }
  }
  const Scores<BF16> s{a.logits, a.bias, at, a.sigmoid, (double)top, sum};
  const float inv = (float)(1.0 / sum);
  auto score32 = [&](float v) { return a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-v)) : __expf(v - top) * inv; };
  auto ordered32 = [](float v) { return v == v ? v : -INFINITY; };

  bool exact = false;          // 64-bit keys are in the LDS
  double off = 0.0;            // bound of the error of an fp32 key
  double* const row_lds = shared + row * (E + a.groups);
  uint32_t comp[PER];
  const bool groups = a.groups > 1;
  uint64_t open = 0;  // groups that stay
  if (a.bias || groups) {
    float* keys = reinterpret_cast<float*>(row_lds);
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
    size_of = row16(size_of, [](float x, float y) { return fmaxf(x, y); });
    off = (double)(ROUTE_U * ((a.sigmoid ? 3.f : 6.f * inv) + size_of));
    if (groups) {
      __syncthreads();
      const int share = group_lanes(a.groups);
      for (int g = lane / share; g < a.groups; g += ROUTE_LANES / share) {
        float one = -INFINITY, two = -INFINITY;
#pragma unroll 4
        for (int e = g * size + lane % share; e < (g + 1) * size; e += share) {
          const float v = keys[e];
          two = fmaxf(two, fminf(one, v));
          one = fmaxf(one, v);
        }
        for (int m = 1; m < share; m <<= 1) {
          const float o1 = __shfl_xor(one, m, ROUTE_LANES), o2 = __shfl_xor(two, m, ROUTE_LANES);
          two = fmaxf(fmaxf(two, o2), fminf(one, o1));
          one = fmaxf(one, o1);
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
      auto either = [](uint32_t x, uint32_t y) { return x | y; };
      lo = row16(lo, either), hi = row16(hi, either);
      open = (uint64_t)hi << 32 | lo;
      worst = row16(worst, [](float x, float y) { return fminf(x, y); });
      next = row16(next, [](float x, float y) { return fmaxf(x, y); });
      // two values of two keys each, their sums rounded
      if (!((double)worst - (double)next > 8.0 * off)) {
        exact_keys(s, E, lane, row_lds);
        exact = true;
        open = exact_groups(a, lane, row_lds, row_lds + E);
        lo = (uint32_t)open, hi = (uint32_t)(open >> 32);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t g = ((uint32_t)number(i) * magic) >> 20;
        comp[i] = ((g < 32 ? lo >> g : hi >> (g & 31)) & 1) ? rough_key(a.bias ? key[i] : l[i]) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) comp[i] = rough_key(key[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) comp[i] = rough_key(l[i]);
  }
  // LAST - e below the cut: e's bits are those of the lane and of the place, apart
  const uint32_t lane_bits = (uint32_t)(~lane & 15) << 2;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t place_bits = ~(uint32_t)(64 * (i / 4) + i % 4) & (LAST & ~0x3Cu);
    uint32_t c = (comp[i] & ~LAST) | (lane_bits | place_bits);
    if (groups) c = comp[i] ? c : 0u;
    comp[i] = i < WHOLE || number(i) < E ? c : 0u;
  }

  uint32_t cand[C] = {};
  uint32_t w = 0;
  bool left = true;  // unless every expert is a candidate already
  const int rounds = a.k + ROUTE_MORE;
  bool found = false;
  if constexpr (C == 1 && PER > 4) {
    // Each lane's four largest, in order; a round takes the row's largest and moves its lane on.  Where a
    // lane is taken four times (3.5 of 100 tokens at 10 candidates) the rest of it is unknown: below, then.
    uint32_t m[4] = {};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
      for (int d = 3; d > 0; --d) m[d] = median(m[d - 1], m[d], comp[i]);
      m[0] = max(m[0], comp[i]);
    }
    for (int j = 0; j < rounds; ++j) {
      w = row16_max(m[0]);
      left = left && w != 0;
      if (j == lane) cand[0] = w;
      const bool mine = m[0] == w;
#pragma unroll
      for (int d = 0; d < 3; ++d) m[d] = mine ? m[d + 1] : m[d];
      m[3] = mine ? 0u : m[3];
    }
    found = __ballot(m[0] == 0) == 0;
  }
  if (!found) {
    // The largest one below w, again and again: x - w wraps to the top exactly for x < w.
    w = 0, left = true;
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
  }

  // the candidates' 64-bit keys, their order, and whether it is certain
  int id[C], rank[C];
  float cl[C];
  double key[C], p[C];
  bool again = false;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    id[c] = cand[c] ? (int)(LAST - (cand[c] & LAST)) : 1 << 20;
    cl[c] = cand[c] ? logit_at<BF16>(a.logits, at + id[c]) : -INFINITY;
    p[c] = s.score_of((double)cl[c]);
    key[c] = ordered(a.bias && cand[c] ? p[c] + (double)a.bias[id[c]] : (double)cl[c]);
    if (!cand[c]) key[c] = -INFINITY;  // its number puts it behind all others
    rank[c] = 0;
  }
  if (a.bias) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int d = 0; d < C; ++d)
        if (c != d) rank[d] += before(key[c], id[c], key[d], id[d]);
      unrolled<ROUTE_LANES - 1>([&](auto N) __attribute__((always_inline)) {
        const double ok = rotate16<N + 1>(key[c]);
        const int oid = (int)rotate16<N + 1>((uint32_t)id[c]);
#pragma unroll
        for (int d = 0; d < C; ++d) rank[d] += before(ok, oid, key[d], id[d]);
      });
    }
  } else {
    // the logits' own bits above the expert's number say the same in one comparison
    uint64_t whole[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      whole[c] = cand[c] ? (uint64_t)route_key(ordered32(cl[c])) << 32 | (uint32_t)(1023 - id[c]) : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int d = 0; d < C; ++d)
        if (c != d) rank[d] += whole[c] > whole[d];
      unrolled<ROUTE_LANES - 1>([&](auto N) __attribute__((always_inline)) {
        const uint64_t o = (uint64_t)rotate16<N + 1>((uint32_t)(whole[c] >> 32)) << 32 | rotate16<N + 1>((uint32_t)whole[c]);
#pragma unroll
        for (int d = 0; d < C; ++d) rank[d] += o > whole[d];
      });
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (!cand[c]) rank[c] = a.k;  // none
  }
  if (left) {
    // everything that was not a candidate has an fp32 key of at most this
    const double most = (double)route_value(w | LAST);
    const double least = a.bias ? most + off : most;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (rank[c] == a.k - 1) again = again || !(key[c] > least);
  }
  const uint64_t rows = __ballot(again);
  again = ((rows >> (threadIdx.x & 48)) & 0xFFFFu) != 0;

  int out[C], out_id[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    out[c] = rank[c], out_id[c] = id[c];
    if (rank[c] >= a.k) p[c] = 0.0;
  }
  if (again) {
    if (a.bias && !exact) exact_keys(s, E, lane, row_lds);
    double last = 0.0;
    int last_id = -1;
    auto shut = [&](int e) { return groups && !((open >> (e / (E / a.groups))) & 1); };
#pragma unroll
    for (int c = 0; c < C; ++c) out[c] = a.k;
    for (int j = 0; j < a.k; ++j) {
      double k = 0.0;
      int best = -1;
      if (a.bias) {
        for (int e = lane; e < E; e += ROUTE_LANES) {
          const double v = row_lds[e];
          if (!shut(e) && (j == 0 || before(last, last_id, v, e)) && (best < 0 || before(v, e, k, best))) k = v, best = e;
        }
      } else {
        uint32_t m = 0;  // all bits of the logits, 0 for what is taken, shut or not there
        int at_i = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const uint32_t v = comp[i] ? route_key(ordered32(l[i])) : 0u;
          if (v > m) m = v, at_i = i;
        }
        if (m) k = (double)route_value(m), best = number(at_i);
      }
      row16_best(k, best);
      last = k, last_id = best;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (number(i) == best) comp[i] = 0;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (j == lane + ROUTE_LANES * c) out[c] = j, out_id[c] = best;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) p[c] = out[c] < a.k ? s.score(out_id[c]) : 0.0;
  }
  if (a.renormalize) {
    double all = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) all += p[c];
    all = row16_plus(all);
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

template <bool BF16>
static void route_scored(const RouteScored& a, int32_t* ids, float* gates, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + ROUTE_ROWS - 1) / ROUTE_ROWS));
  const unsigned lds = a.groups > 1 || a.bias ? ROUTE_ROWS * (unsigned)(a.E + a.groups) * 8 : 0;
#define MX_ROUTE(PER, C, WHOLE) \
  hipLaunchKernelGGL((route_scored_kernel<BF16, PER, C, WHOLE>), grid, dim3(64), lds, stream, a, ids, gates)
  if (a.k + ROUTE_MORE > ROUTE_LANES) {
    if (a.E <= 256)
      MX_ROUTE(16, 3, 0);
    else if (a.E <= 512)
      MX_ROUTE(32, 3, 16);
    else
      MX_ROUTE(64, 3, 32);
  } else if (a.E <= 64) {
    MX_ROUTE(4, 1, 0);
  } else if (a.E <= 128) {
    MX_ROUTE(8, 1, 4);
  } else if (a.E <= 256) {
    MX_ROUTE(16, 1, 8);
  } else if (a.E <= 384) {
    MX_ROUTE(24, 1, 16);
  } else if (a.E <= 512) {
    MX_ROUTE(32, 1, 24);
  } else {
    MX_ROUTE(64, 1, 32);
  }
#undef MX_ROUTE
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
// Where one expert has nearly all of a row, c - sum c q is the difference of two nearly equal values, and
// with S the gates' digits go too.  So it is never formed: with q the weights of the chosen experts (p, or p / S)
// and `rest` what the others have (0 renormalised),
//   c[i] - sum c q = sum over j of (c[i] - c[j]) q[j] + c[i] rest
// in 64 bits.  The others' exponentials and their sum are fp32, which no difference is formed of; 87 below the row's
// largest logit they are 0 (in 64 bits, too, a launch took 1 us more).
// 8192 x 256 fp32 with k 8, other logits from call to call: softmax 7.1 us, 17 MB read and written (6.2 with the
// difference formed from an fp32 sum, which left no right digit where the best logit was 16 above the next);
// renormalised 7.1 (5.4 from the chosen logits alone, which do not say whether there is a NaN); sigmoid 5.1, which
// writes 8 MB alone; 32 tokens 4.0 and 3.0.  A wave a row took 10.2 where 16 lanes took 5.4: most lanes had no chosen
// value.

// exp(l - top) for l <= top, off by some 3 u of itself however far they are apart: what the difference and its product
// with log2 e lose in their roundings (1 and 1.3 |x| u of the result) is multiplied back in.  0 from 87 on.
__device__ __forceinline__ float exp_far(float l, float top) {
  const float x = l - top, b = x - l, lost = (l - (x - b)) - (top + b);
  const float t = x * 1.44269504f;  // log2 e = 1.44269504f + 1.92596299e-8f
  const float left = __builtin_fmaf(lost, 1.44269504f, __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, 1.44269504f, -t)));
  const float e = __builtin_amdgcn_exp2f(t);
  return x > -126.f ? __builtin_fmaf(e, left * 0.693147181f, e) : e;  // not for -Inf, whose left is NaN
}

// Of lane J of the row.
template <int J>
__device__ __forceinline__ double broadcast16(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, 0x150 + J, 0xF, 0xF, false);  // row_newbcast
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), 0x150 + J, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Adds the sum over the first n lanes' values j of (c - cj) qj for each of this lane's two c.
__device__ __forceinline__ void row16_pairs(const double (&c)[2], double cj, double qj, int n, double (&sum)[2]) {
  unrolled<ROUTE_LANES>([&](auto J) __attribute__((always_inline)) {
    if (J >= n) return;
    const double oc = broadcast16<J>(cj), oq = broadcast16<J>(qj);
#pragma unroll
    for (int i = 0; i < 2; ++i) sum[i] += (c[i] - oc) * oq;
  });
}

// A row has 16 lanes, as in the forward call; k of them (two values each where k > 16) hold the chosen ones.
// They write their values over the row behind it: the same wave's stores to one address keep their order.
template <bool BF16, int PER>
__global__ void __launch_bounds__(64) route_scored_backward_kernel(RouteScored a, const float* __restrict__ dgates,
                                                                   const int32_t* __restrict__ ids, void* __restrict__ dlogits) {
  constexpr int WORDS = PER > 32 ? 2 : 1;
  __shared__ uint32_t chosen[ROUTE_ROWS * ROUTE_LANES * WORDS];  // of a lane's places
  const int lane = threadIdx.x % ROUTE_LANES, row = threadIdx.x / ROUTE_LANES;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_ROWS + row;
  if (t >= a.T) return;
  const size_t at = (size_t)t * a.E;
  const int E = a.E;
  int id[2] = {-1, -1};
  double c[2] = {}, l[2] = {-INFINITY, -INFINITY}, q[2] = {}, d[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + ROUTE_LANES * h;
    if (j >= a.k) continue;
    const int e = ids[t * a.k + j];
    if (e < 0 || e >= E) continue;
    id[h] = e;
    c[h] = (double)a.scale * (double)dgates[t * a.k + j];
    l[h] = (double)logit_at<BF16>(a.logits, at + e);
  }
  // softmax: the row's logits, their exponentials, then -p sum c p (renormalised 0).  A NaN among them reaches z, and
  // from there all values of the row, as it reaches all gates of the forward call.
  float v[PER];
  float base = 0.f, z = 0.f;  // the largest logit (of nothing but -Inf 0); the sum of the exponentials that are not chosen
  if (!a.sigmoid) {
    uint32_t* const mine = chosen + (row * ROUTE_LANES + lane) * WORDS;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) mine[w] = 0;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const int e = 4 * (lane + ROUTE_LANES * (i / 4));
      if (e + 4 <= E) {
        if constexpr (BF16) {
          const u32x2 q = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(a.logits) + at + e);
#pragma unroll
          for (int j = 0; j < 2; ++j) v[i + 2 * j] = __uint_as_float(q[j] << 16), v[i + 2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
        } else {
          const u32x4 q = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(a.logits) + at + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i + j] = __uint_as_float(q[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = e + j < E ? logit_at<BF16>(a.logits, at + e + j) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i + j]);
    }
    base = route_value(row16_max(route_key(m)));
    if (base == -INFINITY) base = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = exp_far(v[i], base);
    // where a lane's logits are chosen ones: its places' bits, from the lanes that have the ids
    row_written();
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (id[h] >= 0) {
        const int place = 4 * (id[h] >> 6) + (id[h] & 3);
        atomicOr(&chosen[(row * ROUTE_LANES + ((id[h] >> 2) & 15)) * WORDS + (place >> 5)], 1u << (place & 31));
      }
    row_written();
    uint32_t taken[WORDS];
#pragma unroll
    for (int w = 0; w < WORDS; ++w) taken[w] = mine[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) z += (taken[i / 32] >> (i & 31)) & 1 ? 0.f * v[i] : v[i];
    z = row16_sum(z);
  }
  double rest = 0.0;
  // scores whose sum is 0 in 64 bits have gates 0, as in the forward call
  auto renormalize = [&]() __attribute__((always_inline)) {
    const double s = row16_plus(q[0] + q[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) q[h] = s == 0.0 ? 0.0 : q[h] / s;
  };
  if (a.sigmoid) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (id[h] >= 0) q[h] = 1.0 / (1.0 + exp(-l[h]));
    if (a.renormalize) renormalize();
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (id[h] >= 0) q[h] = exp(l[h] - (double)base);
    const double sum = row16_plus(q[0] + q[1]) + (double)z, inv = sum == 0.0 ? 1.0 : 1.0 / sum;
#pragma unroll
    for (int h = 0; h < 2; ++h) q[h] *= inv;
    if (a.renormalize)
      renormalize();
    else
      rest = (double)z * inv;
    const double cp = row16_plus(c[0] * q[0] + c[1] * q[1]);
    const float f = (float)(a.renormalize ? 0.0 * sum : -cp * inv);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] *= f;
  }
  if (a.sigmoid && !a.renormalize) {
    d[0] = c[0], d[1] = c[1];
  } else {
    d[0] = c[0] * rest, d[1] = c[1] * rest;
    row16_pairs(c, c[0], q[0], a.k, d);
    if (a.k > ROUTE_LANES) row16_pairs(c, c[1], q[1], a.k - ROUTE_LANES, d);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    d[h] *= q[h];
    if (a.sigmoid && id[h] >= 0) d[h] /= 1.0 + exp(l[h]);  // p (1 - p)
  }
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const int e = 4 * (lane + ROUTE_LANES * (i / 4));
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = a.sigmoid ? 0.f : v[i + j];
    if (e + 4 <= E) {
      if constexpr (BF16)
        *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(dlogits) + at + e) =
            u32x2{(uint32_t)f32_to_bf16_rne(o[0]) | (uint32_t)f32_to_bf16_rne(o[1]) << 16,
                  (uint32_t)f32_to_bf16_rne(o[2]) | (uint32_t)f32_to_bf16_rne(o[3]) << 16};
      else
        *reinterpret_cast<u32x4_any*>(static_cast<float*>(dlogits) + at + e) =
            u32x4{__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < E) {
          if constexpr (BF16)
            static_cast<uint16_t*>(dlogits)[at + e + j] = f32_to_bf16_rne(o[j]);
          else
            static_cast<float*>(dlogits)[at + e + j] = o[j];
        }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (id[h] >= 0) {
      if constexpr (BF16)
        static_cast<uint16_t*>(dlogits)[at + id[h]] = f32_to_bf16_rne((float)d[h]);
      else
        static_cast<float*>(dlogits)[at + id[h]] = (float)d[h];
    }
}

template <bool BF16>
static void route_scored_backward(const RouteScored& a, const float* dgates, const int32_t* ids, void* dlogits,
                                  hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + ROUTE_ROWS - 1) / ROUTE_ROWS));
#define MX_ROUTE_BWD(PER) \
  hipLaunchKernelGGL((route_scored_backward_kernel<BF16, PER>), grid, dim3(64), 0, stream, a, dgates, ids, dlogits)
  if (a.E <= 64)
    MX_ROUTE_BWD(4);
  else if (a.E <= 128)
    MX_ROUTE_BWD(8);
  else if (a.E <= 256)
    MX_ROUTE_BWD(16);
  else if (a.E <= 512)
    MX_ROUTE_BWD(32);
  else
    MX_ROUTE_BWD(64);
#undef MX_ROUTE_BWD
}

int launch_route_scored_backward(const RouteScored& a, const float* dgates, const int32_t* ids, void* dlogits,
                                 hipStream_t stream) {
  a.bf16 ? route_scored_backward<true>(a, dgates, ids, dlogits, stream)
         : route_scored_backward<false>(a, dgates, ids, dlogits, stream);
  return hip_status(hipGetLastError());
}

}  // namespace mx
