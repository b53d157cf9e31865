// Routing from given logits (softmax or sigmoid scores) and its gradient.
//
// Per token, over E logits l:
//   s = sigmoid(l)  or  softmax(l)            scores
//   b = s + bias                              what orders the experts; without
//                                             a bias the logits order them
//                                             (every score grows with its logit)
//   groups: a group's score is the sum of its 1 or 2 largest b; the
//           topk_group best groups stay (equal ones: the lower index)
//   I = the K largest of what stays (equal ones: the lower id), ascending ids
//   w = rho s_I  or  rho s_I / (sum s_I + 1e-20)
//
// Selection is decided on the values of b in 64 bits, so that it does not
// depend on how a 32-bit exponential rounds: the scores are computed in fp32
// with a known error bound, and only where the border (the K-th against the
// (K+1)-th expert, or the kept groups' last against the next) is closer than
// that bound are the candidates next to it computed again in fp64.
//
// One wavefront per token, expert 64 j + lane in slot j of lane `lane`, all
// in registers.  The K-th largest key of a set is found bit by bit, a ballot
// and a population count per slot and bit, ending at the first bit whose count
// is exactly K.  That count is what the kernel spends its time on, so with
// several slots it runs on one key a lane: first on the lanes' largest keys,
// whose K-th largest bounds the K-th largest of all from below; then the few
// keys that reach that bound move to one a lane (through LDS, ids ascending)
// and are searched again.  Where more than 64 reach it (equal keys), all slots
// are searched.
//
// Bound by the searches' instructions and, for few tokens, by one wave's chain
// of them, not by memory.  512 experts, fp32 logits, sigmoid, bias, top-22:
// 8192 tokens 10.6 us (18 MB, 1.7 TB/s), with 8 groups 16 to 19 us (a token
// whose groups need 64 bits ends last); 32 tokens 6.1 us.  Searching all slots
// instead took 20, 37 and 9.1 us.
#include <cfloat>
#include <type_traits>

#include "kernels.h"
#include "wave_device.h"

namespace lmoe {

namespace {

constexpr int kRouteWaves = 4;  // tokens per work-group

__device__ __forceinline__ float route_load(const float* p) { return *p; }
__device__ __forceinline__ float route_load(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void route_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void route_store(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// Order-preserving maps onto unsigned integers (-0 equals +0) and back.
__device__ __forceinline__ uint32_t key32(float b) {
  if (b == 0.0f) b = 0.0f;
  const uint32_t u = __float_as_uint(b);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key32_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t key64(double b) {
  if (b == 0.0) b = 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(b);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;  // key32(-inf)

template <class U, int NS>
__device__ __forceinline__ int count_ge(const U (&key)[NS], U v) {
  int c = 0;
#pragma unroll
  for (int j = 0; j < NS; ++j) c += __popcll(__ballot(key[j] >= v));
  return c;
}

// A value v that at least n of the wave's keys reach and that is either
// reached by exactly n of them or equal to the n-th largest key.  Keys of 0
// are empty; n is at most the number of others.
template <class U, int NS>
__device__ __forceinline__ U border(const U (&key)[NS], int n) {
  U v = 0;
  for (int bit = (int)sizeof(U) * 8 - 1; bit >= 0; --bit) {
    const U c = v | ((U)1 << bit);
    const int cnt = count_ge<U, NS>(key, c);
    if (cnt >= n) v = c;
    if (cnt == n) break;
  }
  return v;
}

__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return wave_reduce(v, AddOp{}); }
__device__ __forceinline__ float wave_max(float v) { return wave_reduce(v, MaxOp{}); }

// exp and 1 / x in one instruction each (2^x and 1 / x within 1 ulp; the
// argument's rounding adds 2^-24 |x log2 e| of the result).
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504f);
}
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// A logit as the kernels use it: NaN and -inf mean "not available" (-inf),
// +inf counts as the largest finite value.
__device__ __forceinline__ float clean_logit(float v) {
  return v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY;
}

// Sums of the `best` (1 or 2) largest of each group's G values in the wave's
// LDS row (fp32: half the sum of two, the same order, which cannot overflow);
// lane g returns group g's.  Each group is walked by P lanes (the
// largest power of two with n_group P <= 64), whose two largest are then
// merged; the walk starts at a different place in each group, so that groups
// a multiple of 64 apart do not meet in one LDS bank.
template <class F>
__device__ __forceinline__ F group_best(const F* row, int lane, int n_group, int G, int best) {
  int sh = 0;
  while ((n_group << (sh + 1)) <= 64) ++sh;
  const int P = 1 << sh, g = lane >> sh, i = lane & (P - 1);
  const int steps = (G + P - 1) >> sh;
  F t1 = -INFINITY, t2 = -INFINITY;
  if (g < n_group) {
    const F* at = row + g * G + i;
    int n = g % steps;
    // four reads in flight (past the last step: read again, taken as -inf)
    for (int k = 0; k < steps; k += 4) {
      F b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        b[u] = k + u < steps && i + (n << sh) < G ? at[n << sh] : -INFINITY;
        n = n + 1 == steps ? 0 : n + 1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        t2 = fmax(t2, fmin(t1, b[u]));
        t1 = fmax(t1, b[u]);
      }
    }
  }
  for (int off = 1; off < P; off <<= 1) {
    const F o1 = __shfl_xor(t1, off, 64), o2 = __shfl_xor(t2, off, 64);
    t2 = fmax(fmax(t2, o2), fmin(t1, o1));
    t1 = fmax(t1, o1);
  }
  const F half = std::is_same<F, float>::value ? F(0.5) : F(1);
  const F r = best == 2 ? half * t1 + half * t2 : t1;
  return __shfl(r, lane < n_group ? lane << sh : 0, 64);
}

// How many of the first n lanes' keys come before this lane's: larger ones,
// and equal ones of lower lanes.  Each key in turn is broadcast to all lanes,
// three instructions a key.
__device__ __forceinline__ int rank_of(uint32_t key, int n, int lane) {
  int r = 0;
  for (int i = 0; i < n; ++i) {
    const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)key, i);
    r += k > key || (k == key && i < lane);
  }
  return r;
}

// The lanes of the n largest keys (one per lane; equal keys: lower lanes).
__device__ __forceinline__ uint64_t best_lanes(uint64_t key, int n, uint64_t below) {
  const uint64_t k[1] = {key};
  const uint64_t v = border<uint64_t, 1>(k, n);
  const uint64_t gt = __ballot(key > v), eq = __ballot(key == v);
  const int room = n - __popcll(gt);
  return gt | __ballot(key == v && __popcll(eq & below) < room);
}

}  // namespace

struct RouteParams {
  int T, E, K, n_group, topk_group, best, softmax, renorm;
  float rho;
  long stride;
};

template <class LT, int NJ>
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits_kernel(
    const LT* __restrict__ logits, const float* __restrict__ bias, RouteParams p,
    int32_t* __restrict__ idx_out, float* __restrict__ w_out) {
  __shared__ float ssel[kRouteWaves][64];
  // the biased scores of the group step: 32-bit, or 64-bit where it is close
  __shared__ __attribute__((aligned(8))) char rows[kRouteWaves][NJ * 64 * 8];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wv;
  if (t >= p.T) return;
  const int E = p.E, K = p.K;
  const LT* lp = logits + (size_t)t * p.stride;
  const uint64_t below = (lane == 0) ? 0ull : (~0ull >> (64 - lane));

  float l[NJ], s[NJ], b[NJ];
  uint32_t key[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    l[j] = j * 64 + lane < E ? clean_logit(route_load(lp + j * 64 + lane)) : -INFINITY;
  float m = 0.f, inv = 1.f;
  if (p.softmax) {
    m = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) m = fmaxf(m, l[j]);
    m = wave_max(m);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = l[j] > -INFINITY ? fast_exp(l[j] - m) : 0.f;
      sum += s[j];
    }
    sum = wave_sum(sum);
    inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] *= inv;
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = l[j] > -INFINITY ? fast_rcp(1.0f + fast_exp(-l[j])) : 0.f;
  }
  // Error bound of a biased score.  A sigmoid s: the exponential is off by
  // (2^-23 + 2^-23.4 |l|) of itself, which s passes on times s (1 - s), at most
  // 1/4 and with |l| at most 0.23; the addition and the reciprocal by 2^-24
  // and 2^-23 of s: 2^-21.6 in all.  A softmax score: within 2^-19 of the
  // largest one, inv (up to 16 + 6 additions, the rounding of l - m and the
  // exponential's, times its value, and two products).  The bias addition
  // rounds by 2^-24 of its result, which is added where the border is known.
  const float serr = p.softmax ? 0x1p-19f * inv : 0x1p-21f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = j * 64 + lane;
    const bool on = l[j] > -INFINITY;
    b[j] = on ? (bias ? s[j] + bias[e] : s[j]) : -INFINITY;
    key[j] = e < E ? (on ? key32(bias ? b[j] : l[j]) : kKeyMinusInf) : 0u;
  }

  // biased scores in 64 bits (only where the border is close)
  double m64 = 0.0, inv64 = 1.0;
  bool have64 = false;
  auto prepare64 = [&]() {
    if (have64) return;
    have64 = true;
    if (!p.softmax) return;
    m64 = (double)m;
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (l[j] > -INFINITY) sum += exp((double)l[j] - m64);
    sum = wave_sum(sum);
    inv64 = sum > 0.0 ? 1.0 / sum : 0.0;
  };
  auto value64 = [&](float x, int e) -> double {
    if (!(x > -INFINITY)) return -INFINITY;
    const double v = p.softmax ? exp((double)x - m64) * inv64 : 1.0 / (1.0 + exp(-(double)x));
    return bias ? v + (double)bias[e] : v;
  };
  auto biased64 = [&](int j) { return value64(l[j], j * 64 + lane); };

  if (p.n_group > 1) {
    const int G = E / p.n_group;
    float* row = reinterpret_cast<float*>(rows[wv]);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (j * 64 + lane < E) row[j * 64 + lane] = b[j];
    wave_lds_fence();
    const bool has = lane < p.n_group;
    const float gs0 = group_best(row, lane, p.n_group, G, p.best);
    const float gs = has ? gs0 : -INFINITY;
    const uint32_t gk = has ? key32(gs) : 0u;
    const int rank = has ? rank_of(gk, p.n_group, lane) : 64;
    const uint64_t at = __ballot(rank == p.topk_group - 1);  // the last kept group
    const float gt = key32_value((uint32_t)__builtin_amdgcn_readlane((int)gk, __builtin_ctzll(at)));
    // a group's score is off by at most two scores' bounds and two roundings
    const float gerr = 4.f * serr + 0x1p-21f * fabsf(gt);
    const int over = __popcll(__ballot(has && gs >= gt + 2.f * gerr));
    const int upto = __popcll(__ballot(has && gs > gt - 2.f * gerr));
    uint64_t kept;
    if (over < p.topk_group && upto > p.topk_group) {
      // the groups next to the border are ordered by their 64-bit scores, those
      // above are in (slots that hold no expert of such a group skip the work)
      prepare64();
      const bool near = has && gs < gt + 4.f * gerr && gs > gt - 4.f * gerr;
      const uint64_t close = __ballot(near), sure = __ballot(has && gs >= gt + 4.f * gerr);
      double* row64 = reinterpret_cast<double*>(rows[wv]);
      wave_lds_fence();  // the fp32 row has been read
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = j * 64 + lane;
        if (e < E) row64[e] = (close >> (e / G)) & 1ull ? biased64(j) : (double)b[j];
      }
      wave_lds_fence();
      const double g64 = group_best(row64, lane, p.n_group, G, p.best);
      kept = sure | best_lanes(near ? key64(g64) : 0ull, p.topk_group - __popcll(sure), below);
    } else {
      kept = __ballot(rank < p.topk_group);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = j * 64 + lane;
      if (e < E && !((kept >> (e / G)) & 1ull)) {
        key[j] = 0u;
        b[j] = -INFINITY;
      }
    }
  }

  if constexpr (NJ > 1) {
    // lanes' largest keys -> a lower bound of the K-th largest of all
    uint32_t top[1] = {key[0]};
#pragma unroll
    for (int j = 1; j < NJ; ++j) top[0] = key[j] > top[0] ? key[j] : top[0];
    const uint32_t low0 = border<uint32_t, 1>(top, K);
    // with a bias also those that the scores' error may put above it
    const auto reach = [&](float b) { return 2.f * serr + 0x1p-22f * fabsf(b); };
    uint32_t low = low0;
    if (bias && low0 > kKeyMinusInf) {
      const float b0 = key32_value(low0);
      low = key32(b0 - 5.f * reach(b0));
    }
    uint64_t in[NJ];
    int n = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      in[j] = __ballot(key[j] >= low);
      n += __popcll(in[j]);
    }
    if (low > kKeyMinusInf && n <= 64) {
      // their keys, ids and scores to one a lane
      uint32_t* const ck = reinterpret_cast<uint32_t*>(rows[wv]);
      int base = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (key[j] >= low) {
          const int pos = base + __popcll(in[j] & below);
          ck[pos] = key[j];
          ck[64 + pos] = j * 64 + lane;
          ck[128 + pos] = __float_as_uint(s[j]);
        }
        base += __popcll(in[j]);
      }
      wave_lds_fence();
      const uint32_t k1[1] = {lane < n ? ck[lane] : 0u};
      const int id = ck[64 + lane];
      const float sc = __uint_as_float(ck[128 + lane]);
      // at least low0, so that no key left out lies above it (or, with a bias,
      // within 4 times the scores' error below it)
      uint32_t v = border<uint32_t, 1>(k1, K);
      v = v > low0 ? v : low0;
      const uint64_t gt = __ballot(k1[0] > v), eq = __ballot(k1[0] == v);
      bool on = k1[0] > v || (k1[0] == v && __popcll(eq & below) < K - __popcll(gt));
      if (bias) {
        const float bt = key32_value(v), kv = key32_value(k1[0]), err = reach(bt);
        const int over = __popcll(__ballot(lane < n && kv >= bt + 2.f * err));
        const int upto = __popcll(__ballot(lane < n && kv > bt - 2.f * err));
        if (over < K && upto > K) {
          // those next to the border are ordered by their 64-bit values, those
          // above are in
          prepare64();
          const bool sure = lane < n && kv >= bt + 4.f * err;
          const bool near = lane < n && !sure && kv > bt - 4.f * err;
          const uint64_t k64 = near ? key64(value64(clean_logit(route_load(lp + id)), id)) : 0ull;
          int rank = __popcll(__ballot(sure));
          for (uint64_t left = __ballot(near); left; left &= left - 1) {
            const int o = __builtin_ctzll(left);
            const uint64_t ko =
                (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k64 >> 32), o) << 32 |
                (uint32_t)__builtin_amdgcn_readlane((int)k64, o);
            rank += ko > k64 || (ko == k64 && o < lane);
          }
          on = sure || (near && rank < K);
        }
      }
      const uint64_t mk = __ballot(on);
      const float sum = wave_sum(on ? sc : 0.f);
      if (on) {
        const size_t at = (size_t)t * K + __popcll(mk & below);
        idx_out[at] = id;
        // the quotient first: at most 1, where rho / sum could overflow
        w_out[at] = (p.renorm ? sc / (sum + 1e-20f) : sc) * p.rho;
      }
      return;
    }
  }

  uint32_t v = border<uint32_t, NJ>(key, K);
  if (bias && v > kKeyMinusInf) {
    const float bt = key32_value(v);
    const float err = 2.f * serr + 0x1p-22f * fabsf(bt);
    int over = 0, upto = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      over += __popcll(__ballot(b[j] >= bt + 2.f * err));
      upto += __popcll(__ballot(b[j] > bt - 2.f * err));
    }
    if (over < K && upto > K) {
      // more than K within reach of the border: those next to it are
      // ordered by their 64-bit values, those above are in
      prepare64();
      uint64_t k64[NJ];
      int sure = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const bool in = b[j] >= bt + 4.f * err;
        sure += __popcll(__ballot(in));
        k64[j] = !in && b[j] > bt - 4.f * err ? key64(biased64(j)) : 0ull;
        key[j] = in ? 0xFFFFFFFFu : 0u;
      }
      const uint64_t v64 = border<uint64_t, NJ>(k64, K - sure);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (k64[j]) key[j] = k64[j] > v64 ? 0xFFFFFFFEu : (k64[j] == v64 ? 1u : 0u);
      v = 1u;
    }
  }

  int above = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) above += __popcll(__ballot(key[j] > v));
  int room = K - above;  // experts with key == v still to take, lowest ids first
  int base = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const uint64_t eq = __ballot(key[j] == v);
    const bool on = key[j] > v || (key[j] == v && __popcll(eq & below) < room);
    const int took = __popcll(eq);
    room -= took < room ? took : room;
    const uint64_t mk = __ballot(on);
    if (on) {
      const int pos = base + __popcll(mk & below);
      idx_out[(size_t)t * K + pos] = j * 64 + lane;
      ssel[wv][pos] = s[j];
    }
    base += __popcll(mk);
  }
  wave_lds_fence();
  const float sk = lane < K ? ssel[wv][lane] : 0.f;
  float w = sk * p.rho;
  if (p.renorm) w = (sk / (wave_sum(sk) + 1e-20f)) * p.rho;
  if (lane < K) w_out[(size_t)t * K + lane] = w;
}

// Gradient of the weights in the logits, the selection held fixed.  With
// S = sum of the selected scores + 1e-20 and D = sum dw_k s_k:
//   renormalised   ds_k = rho / S (dw_k - D / S),   otherwise ds_k = rho dw_k
//   sigmoid        dl_k = ds_k s_k (1 - s_k), zero for the others
//   softmax        dl_i = s_i (ds_i - c), c = sum ds_k s_k; renormalised, that
//                  sum is rho D / S (1 - (S - 1e-20) / S) = rho D / S 1e-20 / S,
//                  taken in that form so that nothing cancels
// ds goes without its factor 1 / S (up to 1e20), which is taken with the score or
// the slope, both at most S for a selected expert, so that nothing overflows
// that the gradient does not.
// One wavefront per token; ds goes through an LDS row to the lanes that own
// the experts.  Equal ids add up, in order; ids outside [0, E) are ignored.
// 8111 tokens x 509 experts, bf16, softmax, top-8: 9.1 us (17 MB): the ids'
// latency before their logits' (a second load, of values that the softmax form
// holds in other lanes), the look for equal ids and the row's exponentials.
template <class LT, int NJ>
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits_backward_kernel(
    const LT* __restrict__ logits, const int32_t* __restrict__ idx, const float* __restrict__ dw,
    RouteParams p, LT* __restrict__ dlogits) {
  __shared__ float row[kRouteWaves][NJ * 64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wv;
  if (t >= p.T) return;
  const int E = p.E, K = p.K;
  const LT* lp = logits + (size_t)t * p.stride;
  const int id = lane < K ? idx[(size_t)t * K + lane] : -1;
  const bool valid = id >= 0 && id < E;
  const float lk = valid ? clean_logit(route_load(lp + id)) : -INFINITY;
  // experts that are not available take no part
  const float g = lk > -INFINITY ? dw[(size_t)t * K + lane] : 0.f;

  float s[NJ];
  float m = 0.f, inv = 1.f;
  if (p.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = j * 64 + lane < E ? clean_logit(route_load(lp + j * 64 + lane)) : -INFINITY;
      m = fmaxf(m, s[j]);
    }
    m = wave_max(m);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = s[j] > -INFINITY ? fast_exp(s[j] - m) : 0.f;
      sum += s[j];
    }
    sum = wave_sum(sum);
    inv = sum > 0.f ? 1.0f / sum : 0.f;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) row[wv][j * 64 + lane] = 0.f;

  float sk, slope;  // score of slot `lane` of the selection, and (sigmoid) s (1 - s)
  if (p.softmax) {
    sk = lk > -INFINITY ? fast_exp(lk - m) * inv : 0.f;
    slope = sk;
  } else {
    const float ex = lk > -INFINITY ? fast_exp(-fabsf(lk)) : 0.f;
    const float r = 1.0f / (1.0f + ex);
    sk = lk > -INFINITY ? (lk >= 0.f ? r : ex * r) : 0.f;
    slope = ex * r * r;
  }
  float ds = p.rho * g, c = 0.f, scale = 1.f;
  if (p.renorm) {
    const float S = wave_sum(sk) + 1e-20f;
    const float D = wave_sum(g * sk);
    ds = lk > -INFINITY ? p.rho * (g - D / S) : 0.f;
    c = p.rho * (D / S) * (1e-20f / S);
    scale = 1.0f / S;
  } else if (p.softmax) {
    c = wave_sum(ds * sk);
  }
  // sigmoid: the finished gradient goes through the row; softmax: ds
  const float put = p.softmax ? ds : slope * scale * ds;
  bool dup = false;
  for (int k = 0; k + 1 < K; ++k) {
    const int o = __shfl(id, k, 64);
    dup |= lane > k && valid && o == id;
  }
  wave_lds_fence();
  if (__ballot(dup) == 0ull) {
    if (valid) row[wv][id] = put;
  } else {
    for (int k = 0; k < K; ++k) {
      if (lane == k && valid) row[wv][id] += put;
      wave_lds_fence();
    }
  }
  wave_lds_fence();
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = j * 64 + lane;
    if (e < E) {
      const float r = row[wv][e];
      const float si = s[j] * inv;
      route_store(dlogits + (size_t)t * E + e, p.softmax ? si * scale * r - si * c : r);
    }
  }
}

namespace {
template <class F>
void with_slots(int E, F f) {
  const int nj = (E + 63) / 64;
  if (nj <= 1) f(std::integral_constant<int, 1>{});
  else if (nj <= 2) f(std::integral_constant<int, 2>{});
  else if (nj <= 4) f(std::integral_constant<int, 4>{});
  else if (nj <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}
RouteParams params(const RouteProblem& r) {
  return {r.T, r.E, r.K, r.n_group, r.topk_group, r.best, r.softmax, r.renorm, r.rho, r.stride};
}
}  // namespace

hipError_t route_logits(const RouteProblem& r, const void* logits, bool bf16, const float* bias,
                        int32_t* idx, float* w, hipStream_t s) {
  const int grid = (r.T + kRouteWaves - 1) / kRouteWaves;
  const RouteParams p = params(r);
  with_slots(r.E, [&](auto nj) {
    constexpr int NJ = decltype(nj)::value;
    if (bf16)
      route_logits_kernel<uint16_t, NJ><<<grid, kRouteWaves * 64, 0, s>>>(
          static_cast<const uint16_t*>(logits), bias, p, idx, w);
    else
      route_logits_kernel<float, NJ><<<grid, kRouteWaves * 64, 0, s>>>(
          static_cast<const float*>(logits), bias, p, idx, w);
  });
  return hipGetLastError();
}

hipError_t route_logits_backward(const RouteProblem& r, const void* logits, bool bf16,
                                 const int32_t* idx, const float* dw, void* dlogits,
                                 hipStream_t s) {
  const int grid = (r.T + kRouteWaves - 1) / kRouteWaves;
  const RouteParams p = params(r);
  with_slots(r.E, [&](auto nj) {
    constexpr int NJ = decltype(nj)::value;
    if (bf16)
      route_logits_backward_kernel<uint16_t, NJ><<<grid, kRouteWaves * 64, 0, s>>>(
          static_cast<const uint16_t*>(logits), idx, dw, p, static_cast<uint16_t*>(dlogits));
    else
      route_logits_backward_kernel<float, NJ><<<grid, kRouteWaves * 64, 0, s>>>(
          static_cast<const float*>(logits), idx, dw, p, static_cast<float*>(dlogits));
  });
  return hipGetLastError();
}

}  // namespace lmoe
