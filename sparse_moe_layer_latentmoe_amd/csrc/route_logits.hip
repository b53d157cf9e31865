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
#include "route_device.h"

namespace lmoe {

namespace {
constexpr int kRouteWaves = 4;  // tokens per work-group
}

template <class LT, int NJ>
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits_kernel(
    const LT* __restrict__ logits, const float* __restrict__ bias, RouteParams p,
    int32_t* __restrict__ idx_out, float* __restrict__ w_out) {
  __shared__ float ssel[kRouteWaves][64];
  __shared__ __attribute__((aligned(8))) char rows[kRouteWaves][NJ * 64 * 8];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wv;
  if (t >= p.T) return;
  route_token<LT, NJ>(logits + (size_t)t * p.stride, bias, p, lane, ssel[wv], rows[wv],
                      idx_out + (size_t)t * p.K, w_out + (size_t)t * p.K);
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
}  // namespace

hipError_t route_logits(const RouteProblem& r, const void* logits, bool bf16, const float* bias,
                        int32_t* idx, float* w, hipStream_t s) {
  const int grid = (r.T + kRouteWaves - 1) / kRouteWaves;
  const RouteParams& p = r;
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
  const RouteParams& p = r;
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
